// cbq_rope.cu -- rotary positions of a tensor of heads, and of new tokens on
// their way into a paged cache.
//
// Pair i of a head's rotated part turns by r = 2 pi pos turns_i:
//   (a, b) -> mscale * (a cos r - b sin r, a sin r + b cos r).
// pos * turns_i is taken in fp64 and reduced to its part of a turn there (a
// position of 10^6 has turned 1.6 * 10^5 times in pair 0: fp32 would keep
// three digits of the part), then sine and cosine are fp32 (sincospif).
//
// Bound by memory: each value is read once and written once.  8,192 tokens x 32
// heads x 128 bf16 (134 MB) take 29.3 us, 4.6 TB/s; 4,095 tokens x 48 heads into
// a cache (101 MB) 22.9 us, 4.4 TB/s; a handful of tokens 2.1 to 2.4 us, a
// launch.  Measured on the first: a value a thread 53.7 us, 16-byte pieces 39,
// with the places worked out once for the tokens of a block and their loads
// under way together 31, the sines and cosines laid out without bank conflicts
// 29 (four tokens a block for pairs of neighbours; for halves, which need twice
// the registers an item, two: four took 47).
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
// is a pair or a value.  A thread takes one item of kTok tokens: it works out
// the place once and has all their loads under way together.  grid (blocks of
// kTok tokens, parts of a token's items).  Each block turns its tokens' angles
// into sines and cosines once, behind the loads of its first items.
template <typename Tin, typename Tout, int V, bool kHalfLayout, int kTok>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeArgs a) {
    constexpr int kPiece = !kHalfLayout && V == 1 ? 2 : V;  // values of a rotated piece
    constexpr bool kTwo = kHalfLayout || V == 1;            // a rotated item is two loads
    constexpr int kPairs = V == 1 ? 1 : kHalfLayout ? V : V / 2;  // of a rotated item
    // kTok x rot/2 sines and cosines, two pairs of every item side by side, then the next two: lanes with items in a row
    // read them without bank conflicts
    extern __shared__ __align__(16) float2 cs[];
    __shared__ int64_t place[kTok];
    pdl_trigger();
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * kTok;
    const int half = a.r.rot / 2, turning = a.r.rot / (kPiece * (kHalfLayout ? 2 : 1));  // rotated items of a head
    const int tokens = a.n_tok - t0 < kTok ? (int)(a.n_tok - t0) : kTok;
    if (a.slots) {
        if (threadIdx.x < tokens) {
            const int64_t slot = a.slots[t0 + threadIdx.x];
            const bool good = slot >= 0 && slot < a.n_slots;
            if (slot >= a.n_slots && a.err && blockIdx.y == 0) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
            place[threadIdx.x] = good ? slot / a.page_size * a.page_stride + slot % a.page_size * a.tok_stride : -1;
        }
        __syncthreads();
    }
    const int end = a.first[a.n_groups];
    bool known = false;
    for (int x0 = blockIdx.y * kRopeThreads; x0 < end; x0 += gridDim.y * kRopeThreads) {
        const int x = x0 + threadIdx.x;
        const bool some = x < end;
        const int n = x >= a.first[1] ? (x >= a.first[2] ? 2 : 1) : 0;
        const Group &g = a.g[some ? n : 0];
        const unsigned each = a.per_head[some ? n : 0], in = some ? x - a.first[n] : 0, h = in / each, i = in - h * each;
        const bool turns = g.rotate && i < (unsigned)turning;
        int d = turns ? a.r.off + i * kPiece : (i - (g.rotate ? turning : 0)) * V;
        if (!turns && g.rotate && d >= a.r.off) d += a.r.rot;
        const int second = kHalfLayout ? half : 1;
        const Tin *from = static_cast<const Tin *>(g.src) + t0 * g.src_tok + h * g.src_head + d;
        Tout *to = static_cast<Tout *>(g.dst) + (g.cached ? 0 : t0 * g.dst_tok) + h * g.dst_head + d;
        Vec<Tin, V> va[kTok], vb[kTok];
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            if (!some || u >= tokens) continue;
            va[u] = *reinterpret_cast<const Vec<Tin, V> *>(from + u * g.src_tok);
            if (kTwo && turns) vb[u] = *reinterpret_cast<const Vec<Tin, V> *>(from + u * g.src_tok + second);
        }
        if (!known) {
            known = true;
            for (int j = threadIdx.x; j < tokens * half; j += kRopeThreads) {
                const int u = j / half;
                double turn = (double)a.r.pos[t0 + u] * a.r.turns[j - u * half];
                turn -= rint(turn);
                float s, c;
                sincospif(2.0f * (float)turn, &s, &c);
                const int p = j - u * half, i = p / kPairs, q = p % kPairs;
                cs[u * half + (kPairs == 1 ? p : (q / 2 * turning + i) * 2 + q % 2)] = make_float2(c * a.r.mscale, s * a.r.mscale);
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
            if (!some || u >= tokens) continue;
            const int64_t at = g.cached ? place[u] : u * g.dst_tok;
            if (at < 0) continue;
            Vec<Tout, V> oa, ob;
            float2 c[kPairs];
            if (turns) {
                if constexpr (kPairs == 1) {
                    c[0] = cs[u * half + i];
                } else {
#pragma unroll
                    for (int q = 0; q < kPairs; q += 2) {
                        const float4 y = *reinterpret_cast<const float4 *>(cs + u * half + (q / 2 * turning + i) * 2);
                        c[q] = make_float2(y.x, y.y), c[q + 1] = make_float2(y.z, y.w);
                    }
                }
            }
            if (!turns) {
#pragma unroll
                for (int e = 0; e < V; ++e) oa.v[e] = from_f32<Tout>(to_f32(va[u].v[e]));
            } else if constexpr (kTwo) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float x = to_f32(va[u].v[e]), y = to_f32(vb[u].v[e]);
                    oa.v[e] = from_f32<Tout>(x * c[e].x - y * c[e].y);
                    ob.v[e] = from_f32<Tout>(x * c[e].y + y * c[e].x);
                }
                *reinterpret_cast<Vec<Tout, V> *>(to + at + second) = ob;
            } else {
#pragma unroll
                for (int e = 0; e < V; e += 2) {
                    const float x = to_f32(va[u].v[e]), y = to_f32(va[u].v[e + 1]);
                    oa.v[e] = from_f32<Tout>(x * c[e / 2].x - y * c[e / 2].y);
                    oa.v[e + 1] = from_f32<Tout>(x * c[e / 2].y + y * c[e / 2].x);
                }
            }
            *reinterpret_cast<Vec<Tout, V> *>(to + at) = oa;
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
    const int parts = (end + kRopeThreads - 1) / kRopeThreads;
    // some tokens a block where that leaves two blocks for each of 152 SMs
    constexpr int kTok = kHalfLayout ? 2 : 4;
    const bool many = a.n_tok >= kTok * 304;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(many ? (a.n_tok + kTok - 1) / kTok : a.n_tok), (unsigned)(parts < 64 ? parts : 64));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.dynamicSmemBytes = (many ? kTok : 1) * (a.r.rot / 2) * sizeof(float2);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, k_rope<Tin, Tout, V, kHalfLayout, kTok>, a)
                : cudaLaunchKernelEx(&cfg, k_rope<Tin, Tout, V, kHalfLayout, 1>, a);
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
