// cbq_step.h -- the launchers of the operators between the quantized products
// (positions, attention over the paged cache, sampling), shared by the C-ABI
// layer and their translation units.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "cbq.h"

namespace cbq {

// One head-structured tensor: value d of head h of token t at p + t*tok + h*head + d.
struct Heads {
    void *p;
    int64_t tok, head;
};

// The rotation of one call (turns: rot/2 fp64 turns a position).
struct Rotation {
    const int32_t *pos;
    const double *turns;
    int rot, off, layout;
    float mscale;
};

// x (dtype) rotated into out (the same dtype).
cudaError_t launch_rope(const Heads &x, const Heads &out, int dtype, int64_t n_tok, int heads, int dim,
                        const Rotation &r, cudaStream_t s);
// q rotated into qout, k rotated and v copied into the cache's slots.
cudaError_t launch_rope_append(const Heads &q, const Heads &k, const Heads &v, const Heads &qout, int dtype,
                               int64_t n_tok, int q_heads, const int64_t *slots, const cbq_kv_cache &cache,
                               const Rotation &r, unsigned *err, cudaStream_t s);

// One call of the tree attention (the arguments of cbq_tree_attention).
struct TreeAttention {
    const void *q;
    int64_t q_tok, q_head;
    int q_heads;
    int64_t total_tok;
    cbq_kv_cache c;
    const int32_t *table;
    int table_width, n_seq;
    const int32_t *ctx, *start;
    const int64_t *mask;
    int max_tok;
    int64_t max_len;
    float scale;
    void *out;
    int out_f32;
    float *lse;
    void *ws;
    unsigned *err;
    int stall;  // give-up test mode: the many-row kernel's first block copies nothing
};
size_t tree_attention_workspace(int n_seq, int64_t total_tok, int max_tok, int64_t max_len, int q_heads, int kv_heads,
                                int head_dim);
cudaError_t launch_tree_attention(const TreeAttention &a, cudaStream_t s);

// One call of the sampler (the arguments of cbq_sample).
struct Sample {
    const void *logits;
    int dtype, n, V;
    int64_t row_stride;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *ids;
    float *probs;
};
cudaError_t launch_sample(const Sample &a, cudaStream_t s);

}  // namespace cbq
