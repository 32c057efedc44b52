// cbq_rope.cu -- rotary positions of a tensor of heads, and of new tokens on
// their way into a paged cache.
//
// Pair i of a head's rotated part turns by r = 2 pi pos turns_i:
//   (a, b) -> mscale * (a cos r - b sin r, a sin r + b cos r).
// pos * turns_i is taken in fp64 and reduced to its part of a turn there (a
// position of 10^6 has turned 1.6 * 10^5 times in pair 0: fp32 would keep
// three digits of the part), then the part, its sine and its cosine are fp32
// (sincospif): the part's rounding is off by an angle of at most 2^-23, which is
// what the sine and the products round by, too (against 64 bits 4.2e-8 of the
// values' size for fp32 tensors, 3.0e-8 with angles in fp64).
//
// Bound by memory: each value is read once and written once.  8,192 tokens x 32
// heads x 128 bf16 (134 MB) take 23.9 us, 5.6 TB/s; 4,095 tokens x 48 heads into
// random places of a cache (101 MB) 22.2 us, 4.5 TB/s; a handful of tokens 2.1
// to 2.2 us, a launch.  Measured on the first: a value a thread 53.7 us, 16-byte
// pieces 39, loads of two tokens under way together and sines and cosines laid
// out without bank conflicts 29, blocks that go through several tokens with the
// next ones' pieces coming meanwhile 23.9.
#include <algorithm>
#include <mutex>

#include "cbq_pipe.cuh"
#include "step/cbq_copy.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kStreamTokens = 2;  // a block, from which on k_rope_stream goes through them (1,200 tokens x 8 heads of 128 bf16:
                                  // 3.2 us, a token a block 3.9; 300 tokens, pairs: 2.7 and 2.3)

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
// is a pair or a value.
template <typename Tin, typename Tout, int V, bool kHalfLayout>
struct Item {
    static constexpr int kPiece = !kHalfLayout && V == 1 ? 2 : V;  // values of a rotated piece
    static constexpr bool kTwo = kHalfLayout || V == 1;            // a rotated item is two loads
    static constexpr int kPairs = V == 1 ? 1 : kHalfLayout ? V : V / 2;  // of a rotated item
    static constexpr int kStep = kTwo ? 2 : 4;                     // tokens of a step of k_rope_stream
    const Group &g;
    const Tin *from;  // of token 0
    Tout *to;         // of token 0, or (cached) of place 0
    int i, turning, half, second;
    bool turns;

    __device__ Item(const RopeArgs &a, int x, int n)
        : g(a.g[n]), half(a.r.rot / 2), turning(a.r.rot / (kPiece * (kHalfLayout ? 2 : 1))), second(kHalfLayout ? half : 1) {
        const unsigned each = a.per_head[n], in = x - a.first[n], h = in / each;
        i = in - h * each;
        turns = g.rotate && i < turning;
        int d = turns ? a.r.off + i * kPiece : (i - (g.rotate ? turning : 0)) * V;
        if (!turns && g.rotate && d >= a.r.off) d += a.r.rot;
        from = static_cast<const Tin *>(g.src) + h * g.src_head + d;
        to = static_cast<Tout *>(g.dst) + h * g.dst_head + d;
    }
    static __device__ int group(const RopeArgs &a, int x) { return x >= a.first[1] ? (x >= a.first[2] ? 2 : 1) : 0; }

    // Where pair p of a head lies among a token's sines and cosines: two pairs of every item side by side, then the next
    // two, so that lanes with items in a row read them without bank conflicts.
    static __device__ int place_of(int p, int turning) {
        const int i = p / kPairs, q = p % kPairs;
        return kPairs == 1 ? p : (q / 2 * turning + i) * 2 + q % 2;
    }

    // The item turned (va and vb) or copied (va) to `at`.
    __device__ void put(const Vec<Tin, V> &va, const Vec<Tin, V> &vb, const float2 *cs, Tout *at) const {
        Vec<Tout, V> oa, ob;
        if (!turns) {
#pragma unroll
            for (int e = 0; e < V; ++e) oa.v[e] = from_f32<Tout>(to_f32(va.v[e]));
            *reinterpret_cast<Vec<Tout, V> *>(at) = oa;
            return;
        }
        float2 c[kPairs];
        if constexpr (kPairs == 1) {
            c[0] = cs[i];
        } else {
#pragma unroll
            for (int q = 0; q < kPairs; q += 2) {
                const float4 y = *reinterpret_cast<const float4 *>(cs + (q / 2 * turning + i) * 2);
                c[q] = make_float2(y.x, y.y), c[q + 1] = make_float2(y.z, y.w);
            }
        }
        if constexpr (kTwo) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = to_f32(va.v[e]), y = to_f32(vb.v[e]);
                oa.v[e] = from_f32<Tout>(x * c[e].x - y * c[e].y);
                ob.v[e] = from_f32<Tout>(x * c[e].y + y * c[e].x);
            }
            *reinterpret_cast<Vec<Tout, V> *>(at + second) = ob;
        } else {
#pragma unroll
            for (int e = 0; e < V; e += 2) {
                const float x = to_f32(va.v[e]), y = to_f32(va.v[e + 1]);
                oa.v[e] = from_f32<Tout>(x * c[e / 2].x - y * c[e / 2].y);
                oa.v[e + 1] = from_f32<Tout>(x * c[e / 2].y + y * c[e / 2].x);
            }
        }
        *reinterpret_cast<Vec<Tout, V> *>(at) = oa;
    }
};

// Sine and cosine of pair p at a position, times mscale.
__device__ __forceinline__ float2 angle(const RopeArgs &a, int64_t token, int p) {
    double turn = (double)a.r.pos[token] * a.r.turns[p];
    turn -= rint(turn);
    float s, c;
    sincospif(2.0f * (float)turn, &s, &c);
    return make_float2(c * a.r.mscale, s * a.r.mscale);
}

// Where a token's row of the cache begins, -1 if it has none.
__device__ __forceinline__ int64_t cache_place(const RopeArgs &a, int64_t token, bool tell) {
    const int64_t slot = a.slots[token];
    if (slot >= a.n_slots && a.err && tell) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
    return slot >= 0 && slot < a.n_slots ? slot / a.page_size * a.page_stride + slot % a.page_size * a.tok_stride : -1;
}

// A token a block: grid (tokens, parts of a token's items).  The angles are
// taken behind the loads of the first items.
template <typename Tin, typename Tout, int V, bool kHalfLayout>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeArgs a) {
    using I = Item<Tin, Tout, V, kHalfLayout>;
    extern __shared__ __align__(16) float2 cs[];
    __shared__ int64_t place;
    pdl_trigger();
    pdl_wait();
    const int64_t t = blockIdx.x;
    if (a.slots && threadIdx.x == 0) place = cache_place(a, t, blockIdx.y == 0);
    const int end = a.first[a.n_groups];
    bool known = false;
    for (int x0 = blockIdx.y * kRopeThreads; x0 < end; x0 += gridDim.y * kRopeThreads) {
        const int x = x0 + threadIdx.x;
        const bool some = x < end;
        const I it(a, some ? x : x0, I::group(a, some ? x : x0));
        Vec<Tin, V> va, vb;
        if (some) {
            va = *reinterpret_cast<const Vec<Tin, V> *>(it.from + t * it.g.src_tok);
            if (I::kTwo && it.turns) vb = *reinterpret_cast<const Vec<Tin, V> *>(it.from + t * it.g.src_tok + it.second);
        }
        if (!known) {
            known = true;
            for (int p = threadIdx.x; p < it.half; p += kRopeThreads) cs[I::place_of(p, it.turning)] = angle(a, t, p);
            __syncthreads();
        }
        const int64_t at = !it.g.cached ? t * it.g.dst_tok : place;
        if (some && at >= 0) it.put(va, vb, cs, it.to + at);
    }
}

// Many tokens: a block goes through `each` of them in a row, kStep at a time,
// for one item a thread.  The pieces come through shared memory, kRing - 1
// steps ahead, every thread its own (it waits for its own copies and for nobody
// else's); the next step's angles are taken while this one's results are
// written.  grid (blocks of `each` tokens, parts of a token's items).
constexpr int kRing = 3;
template <typename Tin, typename Tout, int V, bool kHalfLayout>
__global__ void __launch_bounds__(kRopeThreads, 4) k_rope_stream(const __grid_constant__ RopeArgs a, int each) {
    using I = Item<Tin, Tout, V, kHalfLayout>;
    using Piece = Vec<Tin, V>;
    static_assert(sizeof(Piece) == 16, "16-byte copies");
    constexpr int kPieces = I::kTwo ? 2 : 1, kStep = I::kStep;
    extern __shared__ __align__(16) uint8_t smem[];
    Piece *ring = reinterpret_cast<Piece *>(smem) + threadIdx.x;  // [kRing][kStep][kPieces][threads]
    float2 *cs = reinterpret_cast<float2 *>(smem + kRing * kStep * kPieces * kRopeThreads * 16);  // [2][kStep][rot/2]
    __shared__ int64_t place[2][kStep];
    pdl_trigger();
    pdl_wait();
    const int64_t t0 = (int64_t)blockIdx.x * each;
    const int tokens = a.n_tok - t0 < each ? (int)(a.n_tok - t0) : each, steps = (tokens + kStep - 1) / kStep;
    const int end = a.first[a.n_groups], x = blockIdx.y * kRopeThreads + threadIdx.x;
    const bool some = x < end;
    const I it(a, some ? x : end - 1, I::group(a, some ? x : end - 1));
    const Tin *from = it.from + t0 * it.g.src_tok;
    auto fetch = [&](int i) {
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
            if (i * kStep + u >= tokens || !some) continue;
            Piece *to = ring + ((i % kRing) * kStep + u) * kPieces * kRopeThreads;
            const Tin *x = from + (i * kStep + u) * it.g.src_tok;
            copy16(smem_addr(to), x, true);
            if (I::kTwo && it.turns) copy16(smem_addr(to + kRopeThreads), x + it.second, true);
        }
        copy_commit();
    };
    auto angles = [&](int i) {
        for (int j = threadIdx.x; j < kStep * it.half; j += kRopeThreads) {
            const int u = j / it.half, p = j - u * it.half;
            if (i * kStep + u < tokens) cs[((i & 1) * kStep + u) * it.half + I::place_of(p, it.turning)] = angle(a, t0 + i * kStep + u, p);
        }
        if (a.slots && threadIdx.x < kStep && i * kStep + threadIdx.x < tokens)
            place[i & 1][threadIdx.x] = cache_place(a, t0 + i * kStep + threadIdx.x, blockIdx.y == 0);
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(i);
    angles(0);
    for (int i = 0; i < steps; ++i) {
        copy_wait<kRing - 2>();
        __syncthreads();  // this step's angles are there, and the step before has been read
#pragma unroll
        for (int u = 0; u < kStep; ++u) {
            if (i * kStep + u >= tokens || !some) continue;
            const Piece *v = ring + ((i % kRing) * kStep + u) * kPieces * kRopeThreads;
            const Piece va = v[0], vb = v[(kPieces - 1) * kRopeThreads];
            const int64_t at = it.g.cached ? place[i & 1][u] : (t0 + i * kStep + u) * it.g.dst_tok;
            if (at >= 0) it.put(va, vb, cs + ((i & 1) * kStep + u) * it.half, it.to + at);
        }
        fetch(i + kRing - 1);
        if (i + 1 < steps) angles(i + 1);
    }
}

// Dynamic shared memory of k_rope_stream, of a token's `half` pairs.
template <typename I>
constexpr size_t stream_smem(int half) {
    return (size_t)kRing * I::kStep * (I::kTwo ? 2 : 1) * kRopeThreads * 16 + 2 * I::kStep * half * sizeof(float2);
}

// Opts k_rope_stream in to the most that any rotation takes, once per device:
// the limit is the kernel's, for the calls of all host threads.
template <typename Tin, typename Tout, int V, bool kHalfLayout>
cudaError_t raise_smem() {
    static std::mutex mu;
    static bool raised[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (raised[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(k_rope_stream<Tin, Tout, V, kHalfLayout>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)stream_smem<Item<Tin, Tout, V, kHalfLayout>>(CBQ_ROPE_MAX_DIM / 2));
    raised[dev] = e == cudaSuccess;
    return e;
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
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if constexpr (V > 1) {
        const int64_t room = std::max(1, 4 * 152 / parts), each = (a.n_tok + room - 1) / room;  // four blocks for each of 152 SMs
        if (each >= kStreamTokens && parts <= 64) {
            cfg.gridDim = dim3((unsigned)((a.n_tok + each - 1) / each), (unsigned)parts);
            cfg.dynamicSmemBytes = stream_smem<Item<Tin, Tout, V, kHalfLayout>>(a.r.rot / 2);
            const cudaError_t e = raise_smem<Tin, Tout, V, kHalfLayout>();
            return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, k_rope_stream<Tin, Tout, V, kHalfLayout>, a, (int)each);
        }
    }
    cfg.gridDim = dim3((unsigned)a.n_tok, (unsigned)(parts < 64 ? parts : 64));
    cfg.dynamicSmemBytes = (a.r.rot / 2) * sizeof(float2);
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
