// cbq_kv.cu -- the paged cache between two verify steps: accepted drafts moved
// to the end of their context, and pages turned into 8 bits.
#include <algorithm>

#include "cbq_device.cuh"
#include "step/cbq_launch.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

namespace {

// ------------------------------------------------------- accepted drafts --

constexpr int kCommitThreads = 256;
constexpr int kAtOnce = 8;  // tokens whose loads are under way together

// The tokens of a sequence that move, in ascending order, as offsets into the
// cache.  A path is ascending, so a token's old place is not before its new
// one, and no move overwrites what a later one reads: a thread that takes its
// 16 bytes of all tokens in that order, eight loads ahead of their stores,
// needs no other's word and no room in between.
//
// Bound by latency (table, path, load, store one after another): 2.5 us for one
// sequence's accepted drafts in 32 layers, 7.3 for 64 sequences' of large trees
// while their 32 MB are in L2, 11.1 from memory, which would take 5.1 at its
// rate.  (The layers after one another: 15 us more.)
//
// grid (blocks of a slice of the layers' rows, keys' and values'; slices; n_seq).
template <typename V>
__global__ void __launch_bounds__(kCommitThreads) k_commit(KvCommit a, int layers_a_slice) {
    __shared__ int64_t from[CBQ_TREE_MAX], to[CBQ_TREE_MAX];
    __shared__ int32_t path[CBQ_TREE_MAX];
    __shared__ unsigned bad[2], moves[2];
    pdl_trigger();
    pdl_wait();
    const int s = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool first = blockIdx.x == 0 && blockIdx.y == 0;  // the sequence's block that reports and writes its length
    const int ctx = a.ctx[s], said = a.count[s];
    const int count = ctx < 0 ? 0 : min(max(said, 0), a.max_tok);
    if (tid < CBQ_TREE_MAX) path[tid] = tid < count ? a.path[(int64_t)s * a.max_tok + tid] : 0;
    __syncthreads();
    const int64_t room = min((int64_t)a.table_width * a.c.page_size, (int64_t)CBQ_TREE_MAX_LEN);
    if (tid < CBQ_TREE_MAX) {
        const int p = path[tid];
        const bool wrong = tid < count && (p < 0 || p >= a.max_tok || (tid > 0 && p <= path[tid - 1]) || (int64_t)ctx + p >= room);
        const unsigned who = __ballot_sync(~0u, wrong);
        if (lane == 0) bad[warp] = who;
    }
    __syncthreads();
    const int good = bad[0] ? __ffs(bad[0]) - 1 : bad[1] ? 31 + __ffs(bad[1]) : count;
    if (first && tid == 0) {
        if ((good < count || said != count || ctx < 0) && a.err) atomicOr(a.err, CBQ_DEVERR_BAD_LENGTH);
        if (a.ctx_out) a.ctx_out[s] = ctx + good;
    }
    int64_t src = 0, dst = 0;
    bool goes = false;
    if (tid < CBQ_TREE_MAX) {
        goes = tid < good && path[tid] != tid;
        if (goes) {
            const int32_t *table = a.table + (int64_t)s * a.table_width;
            const uint32_t size = a.c.page_size, p = (uint32_t)ctx + (uint32_t)path[tid], q = (uint32_t)ctx + (uint32_t)tid;
            const int ps = table[p / size], pd = table[q / size];
            goes = ps >= 0 && ps < a.c.n_pages && pd >= 0 && pd < a.c.n_pages;
            if (!goes && first && a.err) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
            src = ps * a.c.page_stride + (int64_t)(p % size) * a.c.tok_stride;
            dst = pd * a.c.page_stride + (int64_t)(q % size) * a.c.tok_stride;
        }
        const unsigned who = __ballot_sync(~0u, goes);
        if (lane == 0) moves[warp] = who;
    }
    __syncthreads();
    if (goes) {
        const int at = (warp ? __popc(moves[0]) : 0) + __popc(moves[warp] & ((1u << lane) - 1));
        from[at] = src;
        to[at] = dst;
    }
    __syncthreads();
    const int n = __popc(moves[0]) + __popc(moves[1]);
    constexpr int kEach = sizeof(V) / 2;
    const uint32_t per_head = a.c.head_dim / kEach, row = a.c.kv_heads * per_head, x = blockIdx.x * kCommitThreads + tid;
    const uint32_t of = x / row, at = x % row, layer = blockIdx.y * layers_a_slice + (of >> 1);
    if (of >> 1 >= (uint32_t)layers_a_slice || layer >= (uint32_t)a.layers) return;
    uint16_t *base = static_cast<uint16_t *>(of & 1 ? a.c.v : a.c.k) + layer * a.layer_stride + at / per_head * a.c.head_stride +
                     at % per_head * kEach;
    for (int i0 = 0; i0 < n; i0 += kAtOnce) {
        V v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (i0 + j < n) v[j] = *reinterpret_cast<const V *>(base + from[i0 + j]);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j)
            if (i0 + j < n) *reinterpret_cast<V *>(base + to[i0 + j]) = v[j];
    }
}

template <typename V>
cudaError_t launch_moves(const KvCommit &a, cudaStream_t s) {
    // (slices, so that a thread's number within its own has 32 bits: nearly always there is one)
    const int row = a.c.kv_heads * (a.c.head_dim / (int)(sizeof(V) / 2)), slice = std::min(a.layers, (1 << 30) / (2 * row));
    const int blocks = (2 * slice * row + kCommitThreads - 1) / kCommitThreads, slices = (a.layers + slice - 1) / slice;
    return launch_dependent(k_commit<V>, dim3((unsigned)blocks, (unsigned)slices, (unsigned)a.n_seq), kCommitThreads, 0, s, a, slice);
}

// ---------------------------------------------------------- 8-bit pages --

constexpr int kQuantThreads = 256, kQuantWarps = kQuantThreads / 32;
constexpr int kHeld = 8;  // 16-byte pieces of a thread that stay in registers

template <typename T>
__device__ __forceinline__ float of_bits(uint32_t b) {
    const uint16_t h = (uint16_t)b;
    return to_f32(*reinterpret_cast<const T *>(&h));
}
template <typename T>
constexpr uint32_t kInfinity = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;

// The larger magnitudes, as bits, of two 16-bit floats each.
__device__ __forceinline__ uint32_t larger(uint32_t most, uint32_t two) {
    uint32_t r;
    asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(most), "r"(two & 0x7FFF7FFFu));
    return r;
}
// The same with 0 for what is not finite.
template <typename T>
__device__ __forceinline__ uint32_t larger_finite(uint32_t most, uint32_t two) {
    if ((two & 0x7FFFu) >= kInfinity<T>) two &= 0xFFFF0000u;
    if ((two >> 16 & 0x7FFFu) >= kInfinity<T>) two &= 0xFFFFu;
    return larger(most, two);
}
// Two numbers as e4m3, the first in the low byte.  kOdd: some may not be finite, and become NaN.
template <typename T, bool kOdd>
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t two, float down) {
    const float lo = of_bits<T>(two) * down, hi = of_bits<T>(two >> 16) * down;
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    uint32_t y = r;
    if constexpr (kOdd) {
        if (fabsf(lo) == INFINITY) y = (y & 0xFF00u) | 0x7Fu;
        if (fabsf(hi) == INFINITY) y = (y & 0xFFu) | 0x7F00u;
    }
    return y;
}
// The exponent of a block's scale from the largest magnitude m 2^k, 1 <= m < 2: 448 = 1.75 * 2^8.
__device__ __forceinline__ int scale_exponent(float most) {
    if (most == 0.0f) return 0;
    int k;
    const float m = frexpf(most, &k);  // in [1/2, 1)
    return min(max(k - 9 + (m > 0.875f), -80), 120);
}
__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

// A unit is a block of tokens of one head: `warps` warps take it (1, 2, 4 or
// 8), each value read once as long as it fits their registers, which 16,384 do.
// Neighbouring units are neighbouring heads, whose rows lie side by side.
// Bound by memory: 341 pages of 48 tokens in 4 layers (402 MB read and written) 67.5
// us, 6.0 TB/s; a page of 64 in 32 layers (12.6 MB, in L2) 4.7.  A thread's pieces follow one
// another without divisions, and magnitudes are compared as integers, two at a
// time; with 96 registers a thread, two blocks an SM, 81 us.
// grid (units of a layer / units a block, layers, 2): keys, then values.
template <typename T, bool kVec>
__global__ void __launch_bounds__(kQuantThreads, 3) k_quantize(KvQuantize a, int warps, uint32_t units) {
    __shared__ uint32_t of_warp[kQuantWarps];
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dim = a.to.head_dim, block = a.to.block;
    const uint32_t heads = a.to.kv_heads, per_page = a.to.page_size / block;
    const uint32_t u = blockIdx.x * (kQuantWarps / warps) + warp / warps, i = u / (heads * per_page);
    const int h = (int)(u % heads), b = (int)(u / heads % per_page), me = warp % warps * 32 + lane, step = warps * 32;
    int64_t src = -1, dst = -1;
    if (u < units) {
        src = a.src[i], dst = a.dst[i];
        if ((src >= a.from.n_pages || dst >= a.to.n_pages)) {
            if (a.err && me == 0) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
            src = -1;
        }
    }
    const bool on = src >= 0 && dst >= 0;
    const T *x = static_cast<const T *>(blockIdx.z ? a.from.v : a.from.k) + blockIdx.y * a.from_layer + src * a.from.page_stride +
                 (int64_t)b * block * a.from.tok_stride + h * a.from.head_stride;
    uint8_t *y = static_cast<uint8_t *>(blockIdx.z ? a.to.v : a.to.k) + blockIdx.y * a.to_layer + dst * a.to.page_stride +
                 (int64_t)b * block * a.to.tok_stride + h * a.to.head_stride;
    // A thread's pieces: in token t the d-th of a row, then some rows and pieces on (no divisions).
    constexpr int kEach = kVec ? 8 : 1;
    const int per_row = dim / kEach, pieces = on ? block * per_row : 0, rows_on = step / per_row, pieces_on = step % per_row;
    struct Place {
        int t, d;
    };
    const Place first = {me / per_row, me % per_row};
    auto next = [&](Place &p) {
        p.t += rows_on;
        p.d += pieces_on;
        if (p.d >= per_row) p.d -= per_row, ++p.t;
    };
    auto load = [&](const Place &p) {
        const T *at = x + (int64_t)p.t * a.from.tok_stride + p.d * kEach;
        if constexpr (kVec) return *reinterpret_cast<const uint4 *>(at);
        else return make_uint4(*reinterpret_cast<const uint16_t *>(at), 0, 0, 0);
    };
    uint4 v[kHeld];
    Place p = first;
#pragma unroll
    for (int j = 0; j < kHeld; ++j, next(p)) v[j] = me + j * step < pieces ? load(p) : make_uint4(0, 0, 0, 0);
    // the largest magnitude of all, and only where that is not finite once more of the finite ones
    auto largest = [&](auto of) {
        uint32_t most = 0;
#pragma unroll
        for (int j = 0; j < kHeld; ++j) {
            most = of(most, v[j].x);
            if constexpr (kVec) most = of(most, v[j].y), most = of(most, v[j].z), most = of(most, v[j].w);
        }
        Place q = p;
        for (int k = me + kHeld * step; k < pieces; k += step, next(q)) {
            const uint4 w = load(q);
            most = of(most, w.x);
            if constexpr (kVec) most = of(most, w.y), most = of(most, w.z), most = of(most, w.w);
        }
        most = __reduce_max_sync(~0u, max(most & 0xFFFFu, most >> 16));
        if (warps > 1) {
            __syncthreads();
            if (lane == 0) of_warp[warp] = most;
            __syncthreads();
            for (int w = warp / warps * warps, j = 0; j < warps; ++j) most = max(most, of_warp[w + j]);
        }
        return most;
    };
    uint32_t most = largest([](uint32_t m, uint32_t two) { return larger(m, two); });
    const bool odd = most >= kInfinity<T>;
    if (warps > 1 ? __syncthreads_or(odd) : __any_sync(~0u, odd)) {
        const uint32_t finite = largest([](uint32_t m, uint32_t two) { return larger_finite<T>(m, two); });
        if (odd) most = finite;
    }
    if (!on) return;
    const int e = scale_exponent(of_bits<T>(most));
    const float down = two_to(-e);
    auto store_all = [&](auto pair) {
        auto store = [&](const Place &p, const uint4 &w) {
            uint8_t *at = y + (int64_t)p.t * a.to.tok_stride + p.d * kEach;
            if constexpr (kVec) *reinterpret_cast<uint2 *>(at) = make_uint2(pair(w.x) | pair(w.y) << 16, pair(w.z) | pair(w.w) << 16);
            else *at = (uint8_t)pair(w.x);
        };
        Place p = first;
#pragma unroll
        for (int j = 0; j < kHeld; ++j, next(p))
            if (me + j * step < pieces) store(p, v[j]);
        for (int k = me + kHeld * step; k < pieces; k += step, next(p)) store(p, load(p));
    };
    if (odd) store_all([&](uint32_t two) { return e4m3_pair<T, true>(two, down); });
    else store_all([&](uint32_t two) { return e4m3_pair<T, false>(two, down); });
    if (me == 0)
        (blockIdx.z ? a.to.v_scale : a.to.k_scale)[blockIdx.y * a.scale_layer + dst * a.to.scale_page_stride +
                                                   b * a.to.scale_block_stride + h * a.to.scale_head_stride] = two_to(e);
}

template <typename T, bool kVec>
cudaError_t launch_pages(const KvQuantize &a, cudaStream_t s) {
    const int64_t units = a.n * a.to.kv_heads * (a.to.page_size / a.to.block), pieces = (int64_t)a.to.block * a.to.head_dim / (kVec ? 8 : 1);
    int warps = 1;
    while (warps < kQuantWarps && pieces > (int64_t)warps * 32 * kHeld) warps *= 2;
    const int64_t each = kQuantWarps / warps, blocks = (units + each - 1) / each;
    return launch_dependent(k_quantize<T, kVec>, dim3((unsigned)blocks, (unsigned)a.layers, 2), kQuantThreads, 0, s, a, warps, (uint32_t)units);
}

template <typename T>
cudaError_t launch_quantize(const KvQuantize &a, cudaStream_t s) {
    // 16 bytes a load and 8 a store want whole pieces in a row, and every row on such a boundary
    const uintptr_t in = reinterpret_cast<uintptr_t>(a.from.k) | reinterpret_cast<uintptr_t>(a.from.v);
    const uintptr_t out = reinterpret_cast<uintptr_t>(a.to.k) | reinterpret_cast<uintptr_t>(a.to.v);
    const int64_t strides = a.from_layer | a.from.page_stride | a.from.tok_stride | a.from.head_stride | a.to_layer | a.to.page_stride |
                            a.to.tok_stride | a.to.head_stride;
    return in % 16 == 0 && out % 8 == 0 && strides % 8 == 0 && a.to.head_dim % 8 == 0 ? launch_pages<T, true>(a, s)
                                                                                      : launch_pages<T, false>(a, s);
}

}  // namespace

cudaError_t launch_kv_commit(const KvCommit &a, cudaStream_t s) {
    const uintptr_t ends = reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v);
    const int64_t strides = a.layer_stride | a.c.page_stride | a.c.tok_stride | a.c.head_stride | a.c.head_dim;
    return ends % 16 == 0 && strides % 8 == 0 ? launch_moves<uint4>(a, s) : launch_moves<uint16_t>(a, s);
}

cudaError_t launch_kv_quantize(const KvQuantize &a, cudaStream_t s) {
    return a.from.dtype == CBQ_BF16 ? launch_quantize<__nv_bfloat16>(a, s) : launch_quantize<__half>(a, s);
}

}  // namespace cbq
