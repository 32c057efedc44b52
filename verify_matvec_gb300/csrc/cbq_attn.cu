// cbq_attn.cu -- attention of a tree of drafted tokens over a paged cache.
#include "cbq_device.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

namespace {

constexpr int kMaxDim = 256;

// One warp per (token, head): the lanes hold the head's values, a key at a
// time, the running maximum and sum of the softmax beside the weighted sum.
// grid (q_heads, max_tok, n_seq).
template <typename T>
__global__ void __launch_bounds__(32) k_tree_attention(TreeAttention a) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x, h = blockIdx.x, i = blockIdx.y, s = blockIdx.z, D = a.c.head_dim;
    const int64_t room = (int64_t)a.table_width * a.c.page_size;
    const int64_t b0 = a.start[s], b1 = a.start[s + 1];
    const int64_t most = a.max_len < room ? a.max_len : room;
    int64_t n = b1 - b0, ctx = a.ctx[s];
    bool cut = b0 < 0 || b1 > a.total_tok || n < 0 || n > a.max_tok || ctx < 0;
    if (b0 < 0 || b1 > a.total_tok || n < 0) n = 0;
    if (n > a.max_tok) n = a.max_tok;
    if (ctx < 0) ctx = 0;
    int64_t len = ctx + n;
    if (len > most) {
        cut = true;
        len = most;
    }
    if (cut && a.err && lane == 0) atomicOr(a.err, CBQ_DEVERR_BAD_LENGTH);
    if (i >= n) return;
    const int64_t row = b0 + i;
    const uint64_t mask = (uint64_t)a.mask[row];
    const T *q = static_cast<const T *>(a.q) + row * a.q_tok + h * a.q_head;
    const int g = h / (a.q_heads / a.c.kv_heads);
    float qv[kMaxDim / 32], acc[kMaxDim / 32];
#pragma unroll
    for (int j = 0; j < kMaxDim / 32; ++j) {
        acc[j] = 0.0f;
        qv[j] = j * 32 + lane < D ? to_f32(q[j * 32 + lane]) : 0.0f;
    }
    float top = -INFINITY, sum = 0.0f;
    for (int64_t p = 0; p < len; ++p) {
        if (p >= ctx && !(mask >> (p - ctx) & 1)) continue;
        const int64_t page = a.table[s * (int64_t)a.table_width + p / a.c.page_size];
        if (page < 0 || page >= a.c.n_pages) {
            if (a.err && lane == 0) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
            continue;
        }
        const int64_t at = page * a.c.page_stride + p % a.c.page_size * a.c.tok_stride + g * a.c.head_stride;
        const T *k = static_cast<const T *>(a.c.k) + at, *v = static_cast<const T *>(a.c.v) + at;
        float x = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxDim / 32; ++j)
            if (j * 32 + lane < D) x += qv[j] * to_f32(k[j * 32 + lane]);
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
        x *= a.scale;
        const float now = fmaxf(top, x);
        // nothing of weight so far (top is -inf): a score of -inf has none either
        const float keep = top == -INFINITY ? 0.0f : expf(top - now), w = x == -INFINITY ? 0.0f : expf(x - now);
        sum = sum * keep + w;
#pragma unroll
        for (int j = 0; j < kMaxDim / 32; ++j)
            if (j * 32 + lane < D) acc[j] = acc[j] * keep + w * to_f32(v[j * 32 + lane]);
        top = now;
    }
    const float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
    const int64_t o = (row * a.q_heads + h) * D;
    for (int j = 0; j < kMaxDim / 32; ++j) {
        const int d = j * 32 + lane;
        if (d >= D) break;
        const float r = acc[j] * inv;
        if (a.out_f32) static_cast<float *>(a.out)[o + d] = r;
        else static_cast<T *>(a.out)[o + d] = (T)r;
    }
    if (a.lse && lane == 0) a.lse[row * a.q_heads + h] = sum > 0.0f ? top + logf(sum) : (sum == 0.0f ? -INFINITY : sum);
}

}  // namespace

size_t tree_attention_workspace(int, int64_t, int, int64_t, int, int, int) { return 16; }

cudaError_t launch_tree_attention(const TreeAttention &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.q_heads, (unsigned)a.max_tok, (unsigned)a.n_seq);
    cfg.blockDim = dim3(32);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return a.c.dtype == CBQ_BF16 ? cudaLaunchKernelEx(&cfg, k_tree_attention<__nv_bfloat16>, a)
                                 : cudaLaunchKernelEx(&cfg, k_tree_attention<__half>, a);
}

}  // namespace cbq
