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

// One group of heads of a token: rotated or copied, to plain strides or (cached) to the token's slot.
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
    int first[4];    // of a token's items, the first of each group (and the end)
    int per_head[3];
    int in_place;    // what is not rotated is there already
};

template <typename T, int V>
struct alignas(V * sizeof(T)) Vec {
    T v[V];
};

// A token's values are taken V at a time (16 bytes of input): an item is two
// such pieces whose values form pairs (half layout), one piece (pairs of
// neighbours), or one piece that is copied.  V = 1 takes any alignment: an item
// is a pair or a value.  grid (tokens, parts of a token's items): few tokens
// are spread over blocks.  Each block turns its token's rot/2 angles into sines
// and cosines once, behind the loads of its first items.
template <typename Tin, typename Tout, int V, bool kHalfLayout>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeArgs a) {
    constexpr int kItems = 2;                          // of a thread at a time
    constexpr int kPiece = !kHalfLayout && V == 1 ? 2 : V;  // values of a rotated piece
    constexpr int kTwo = kHalfLayout ? 2 : 1;
    __shared__ float2 cs[CBQ_ROPE_MAX_DIM / 2];
    pdl_trigger();
    pdl_wait();
    const int64_t t = blockIdx.x;
    const int half = a.r.rot / 2, turning = a.r.rot / (kPiece * kTwo);  // rotated items of a head
    int64_t slot_at = -1;
    if (a.slots) {
        const int64_t slot = a.slots[t];
        if (slot >= 0 && slot < a.n_slots) slot_at = slot / a.page_size * a.page_stride + slot % a.page_size * a.tok_stride;
        else if (slot >= 0 && a.err && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
    }
    const double pos = (double)a.r.pos[t];
    const int step = kItems * kRopeThreads;
    const int end = a.first[a.n_groups];
    bool known = false;
    for (int x0 = blockIdx.y * step; x0 < end; x0 += gridDim.y * step) {
        Vec<Tin, V> va[kItems], vb[kItems];
        Tout *to[kItems];
        int pair[kItems];  // the first pair of a rotated piece; -1: copied; -2: nothing
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            const int x = x0 + u * kRopeThreads + threadIdx.x;
            pair[u] = -2;
            to[u] = nullptr;
            if (x >= end) continue;
            const int n = x >= a.first[1] ? (x >= a.first[2] ? 2 : 1) : 0;
            const Group &g = a.g[n];
            if (g.cached && slot_at < 0) continue;
            const unsigned in = x - a.first[n], h = in / (unsigned)a.per_head[n], i = in - h * a.per_head[n];
            const Tin *from = static_cast<const Tin *>(g.src) + t * g.src_tok + h * g.src_head;
            Tout *dst = static_cast<Tout *>(g.dst) + (g.cached ? slot_at : t * g.dst_tok) + h * g.dst_head;
            if (g.rotate && i < (unsigned)turning) {
                const int d = a.r.off + i * kPiece;
                va[u] = *reinterpret_cast<const Vec<Tin, V> *>(from + d);
                if constexpr (kHalfLayout) vb[u] = *reinterpret_cast<const Vec<Tin, V> *>(from + d + half);
                else if constexpr (V == 1) vb[u] = *reinterpret_cast<const Vec<Tin, V> *>(from + d + 1);
                to[u] = dst + d;
                pair[u] = kHalfLayout ? i * V : i * (kPiece / 2);
            } else {
                int d = (i - (g.rotate ? turning : 0)) * V;
                if (g.rotate && d >= a.r.off) d += a.r.rot;
                va[u] = *reinterpret_cast<const Vec<Tin, V> *>(from + d);
                to[u] = dst + d;
                pair[u] = -1;
            }
        }
        if (!known) {
            known = true;
            for (int i = threadIdx.x; i < half; i += kRopeThreads) {
                double turn = pos * a.r.turns[i];
                turn -= rint(turn);
                float s, c;
                sincospif(2.0f * (float)turn, &s, &c);
                cs[i] = make_float2(c * a.r.mscale, s * a.r.mscale);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kItems; ++u) {
            if (pair[u] == -2) continue;
            Vec<Tout, V> oa, ob;
            if (pair[u] == -1) {
#pragma unroll
                for (int e = 0; e < V; ++e) oa.v[e] = from_f32<Tout>(to_f32(va[u].v[e]));
                *reinterpret_cast<Vec<Tout, V> *>(to[u]) = oa;
            } else if constexpr (kHalfLayout || V == 1) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float2 c = cs[pair[u] + e];
                    const float x = to_f32(va[u].v[e]), y = to_f32(vb[u].v[e]);
                    oa.v[e] = from_f32<Tout>(x * c.x - y * c.y);
                    ob.v[e] = from_f32<Tout>(x * c.y + y * c.x);
                }
                *reinterpret_cast<Vec<Tout, V> *>(to[u]) = oa;
                *reinterpret_cast<Vec<Tout, V> *>(to[u] + (kHalfLayout ? half : 1)) = ob;
            } else {
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float2 c = cs[pair[u] + e / 2];
                    const float x = to_f32(va[u].v[e]), y = to_f32(va[u].v[e + 1]);
                    oa.v[e] = from_f32<Tout>(x * c.x - y * c.y);
                    oa.v[e + 1] = from_f32<Tout>(x * c.y + y * c.x);
                }
                *reinterpret_cast<Vec<Tout, V> *>(to[u]) = oa;
            }
        }
    }
}

template <typename Tin, typename Tout, int V, bool kHalfLayout>
cudaError_t launch_pieces(RopeArgs a, cudaStream_t s) {
    const int piece = !kHalfLayout && V == 1 ? 2 : V, turning = a.r.rot / (piece * (kHalfLayout ? 2 : 1));
    int end = 0;
    for (int n = 0; n < 3; ++n) {
        a.first[n] = end;
        if (n >= a.n_groups) continue;
        const int copied = a.dim / V - (a.g[n].rotate ? a.r.rot / V : 0);
        a.per_head[n] = (a.g[n].rotate ? turning : 0) + (a.in_place ? 0 : copied);
        end += a.per_head[n] * a.g[n].heads;
    }
    a.first[a.n_groups] = end;
    for (int n = a.n_groups + 1; n < 4; ++n) a.first[n] = end;
    // a block a token where there are enough of them, else as many as its items fill
    const int parts = (end + 2 * kRopeThreads - 1) / (2 * kRopeThreads);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.n_tok, (unsigned)(a.n_tok >= 608 ? 1 : parts < 64 ? parts : 64));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_rope<Tin, Tout, V, kHalfLayout>, a);
}

// Whether all rows, heads and parts begin on V values (of 16 bytes of input).
template <typename Tin, typename Tout, int V>
bool whole(const RopeArgs &a) {
    const int64_t rot = a.r.layout == CBQ_ROPE_HALF ? a.r.rot / 2 : a.r.rot;
    int64_t all = a.dim | a.r.off | rot | a.page_stride | a.tok_stride;
    uintptr_t in = 0, out = 0;
    for (int n = 0; n < a.n_groups; ++n) {
        all |= a.g[n].src_tok | a.g[n].src_head | a.g[n].dst_tok | a.g[n].dst_head;
        in |= reinterpret_cast<uintptr_t>(a.g[n].src);
        out |= reinterpret_cast<uintptr_t>(a.g[n].dst);
    }
    return all % V == 0 && in % (V * sizeof(Tin)) == 0 && out % (V * sizeof(Tout)) == 0;
}

template <typename Tin, typename Tout>
cudaError_t launch(const RopeArgs &a, cudaStream_t s) {
    constexpr int V = 16 / sizeof(Tin);
    const bool half = a.r.layout == CBQ_ROPE_HALF;
    if (whole<Tin, Tout, V>(a)) return half ? launch_pieces<Tin, Tout, V, true>(a, s) : launch_pieces<Tin, Tout, V, false>(a, s);
    return half ? launch_pieces<Tin, Tout, 1, true>(a, s) : launch_pieces<Tin, Tout, 1, false>(a, s);
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
    a.in_place = x.p == out.p;
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
