// cbq_rope.cu -- rotary positions of a tensor of heads, and of new tokens on
// their way into a paged cache.
//
// Pair i of a head's rotated part turns by r = 2 pi pos turns_i:
//   (a, b) -> mscale * (a cos r - b sin r, a sin r + b cos r).
// pos * turns_i is taken in fp64 and reduced to its part of a turn there (a
// position of 10^6 has turned 1.6 * 10^5 times in pair 0: fp32 would keep
// three digits of the part), then sine and cosine are fp32 (sincospif).
#include "cbq_device.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

namespace {

constexpr int kRopeThreads = 256;

// One group of heads of a token: rotated or copied, to plain strides or (cache) to the token's slot.
struct Group {
    const void *src;
    int64_t src_tok, src_head;
    void *dst;
    int64_t dst_tok, dst_head;
    int heads;
    int rotate;
    int cached;  // the destination row is the token's slot, not the token
};

struct RopeArgs {
    Group g[3];
    int n_groups;
    int64_t n_tok;
    int dim;
    Rotation r;
    const int64_t *slots;
    int64_t n_slots;
    int page_size;
    int64_t page_stride, tok_stride;
    unsigned *err;
};

// One block per token: its rot/2 sines and cosines once into shared memory,
// then the block walks the values of all its heads, a pair or a copied value
// at a time.
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(kRopeThreads) k_rope(RopeArgs a) {
    __shared__ float2 cs[CBQ_ROPE_MAX_DIM / 2];
    pdl_trigger();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int half = a.r.rot / 2;
    const double pos = (double)a.r.pos[t];
    for (int i = threadIdx.x; i < half; i += kRopeThreads) {
        double turn = pos * a.r.turns[i];
        turn -= rint(turn);
        float s, c;
        sincospif(2.0f * (float)turn, &s, &c);
        cs[i] = make_float2(c * a.r.mscale, s * a.r.mscale);
    }
    int64_t slot = 0;
    bool put = true;
    if (a.slots) {
        slot = a.slots[t];
        put = slot >= 0 && slot < a.n_slots;
        if (slot >= a.n_slots && a.err && threadIdx.x == 0) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
    }
    __syncthreads();
    for (int n = 0; n < a.n_groups; ++n) {
        const Group &g = a.g[n];
        if (g.cached && !put) continue;
        const Tin *src = static_cast<const Tin *>(g.src) + t * g.src_tok;
        Tout *dst = static_cast<Tout *>(g.dst) +
                    (g.cached ? slot / a.page_size * a.page_stride + slot % a.page_size * a.tok_stride : t * g.dst_tok);
        const int rot = g.rotate ? a.r.rot : 0;
        const int items = a.dim - rot / 2;  // pairs, then copied values
        for (int x = threadIdx.x; x < items * g.heads; x += kRopeThreads) {
            const int h = x / items, i = x - h * items;
            const Tin *from = src + h * g.src_head;
            Tout *to = dst + h * g.dst_head;
            if (i < rot / 2) {
                const int ia = a.r.off + (a.r.layout == CBQ_ROPE_HALF ? i : 2 * i);
                const int ib = ia + (a.r.layout == CBQ_ROPE_HALF ? half : 1);
                const float va = to_f32(from[ia]), vb = to_f32(from[ib]);
                to[ia] = from_f32<Tout>(va * cs[i].x - vb * cs[i].y);
                to[ib] = from_f32<Tout>(va * cs[i].y + vb * cs[i].x);
            } else {
                int d = i - rot / 2;
                if (rot && d >= a.r.off) d += rot;
                to[d] = from_f32<Tout>(to_f32(from[d]));
            }
        }
    }
}

template <typename Tin, typename Tout>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.n_tok);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rope<Tin, Tout>, a);
}

}  // namespace

cudaError_t launch_rope(const Heads &x, const Heads &out, int dtype, int64_t n_tok, int heads, int dim,
                        const Rotation &r, cudaStream_t s) {
    RopeArgs a = {};
    a.g[0] = Group{x.p, x.tok, x.head, out.p, out.tok, out.head, heads, 1, 0};
    a.n_groups = 1;
    a.n_tok = n_tok;
    a.dim = dim;
    a.r = r;
    if (dtype == CBQ_F32) return launch<float, float>(a, s);
    if (dtype == CBQ_BF16) return launch<__nv_bfloat16, __nv_bfloat16>(a, s);
    return launch<__half, __half>(a, s);
}

cudaError_t launch_rope_append(const Heads &q, const Heads &k, const Heads &v, const Heads &qout, int dtype,
                               int64_t n_tok, int q_heads, const int64_t *slots, const cbq_kv_cache &c,
                               const Rotation &r, unsigned *err, cudaStream_t s) {
    RopeArgs a = {};
    a.g[0] = Group{q.p, q.tok, q.head, qout.p, qout.tok, qout.head, q_heads, 1, 0};
    a.g[1] = Group{k.p, k.tok, k.head, c.k, 0, c.head_stride, c.kv_heads, 1, 1};
    a.g[2] = Group{v.p, v.tok, v.head, c.v, 0, c.head_stride, c.kv_heads, 0, 1};
    a.n_groups = 3;
    a.n_tok = n_tok;
    a.dim = c.head_dim;
    a.r = r;
    a.slots = slots;
    a.n_slots = c.n_pages * c.page_size;
    a.page_size = c.page_size;
    a.page_stride = c.page_stride;
    a.tok_stride = c.tok_stride;
    a.err = err;
    const bool bf = c.dtype == CBQ_BF16;
    if (dtype == CBQ_F32) return bf ? launch<float, __nv_bfloat16>(a, s) : launch<float, __half>(a, s);
    if (dtype == CBQ_BF16) return bf ? launch<__nv_bfloat16, __nv_bfloat16>(a, s) : launch<__nv_bfloat16, __half>(a, s);
    return bf ? launch<__half, __nv_bfloat16>(a, s) : launch<__half, __half>(a, s);
}

}  // namespace cbq
