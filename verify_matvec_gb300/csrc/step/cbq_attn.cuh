// cbq_attn.cuh -- what the kernels of the tree attention share.
#pragma once

#include <type_traits>

#include "cbq_device.cuh"
#include "step/cbq_copy.cuh"
#include "step/cbq_launch.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

constexpr int kMaxDim = 256;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// What a block needs to know of a sequence, with everything out of range cut.
struct Seq {
    int64_t row0;   // its first row of q
    int n, ctx, len;
    int from, old;  // places in 8 bits: [0, old); in 16: [from, len)
};

// In place of OldPlaces where there are none.
struct NoOldPlaces {};
__device__ __forceinline__ int chunk_of(const OldPlaces &b) { return b.chunk8; }
__device__ __forceinline__ int chunk_of(NoOldPlaces) { return 1; }
__device__ __forceinline__ int old_blocks(const OldPlaces &b) { return b.n8; }
__device__ __forceinline__ int old_blocks(NoOldPlaces) { return 0; }

__device__ __forceinline__ Seq sequence(const TreeAttention &a, int s, bool report) {
    const int64_t room = (int64_t)a.table_width * a.c.page_size;
    const int64_t b0 = __ldcg(a.start + s), b1 = __ldcg(a.start + s + 1);  // (from L2: the join reads before it waits)
    const int64_t most = a.max_len < room ? a.max_len : room;
    int64_t n = b1 - b0, ctx = __ldcg(a.ctx + s);
    bool cut = n > a.max_tok || ctx < 0;
    if (b0 < 0 || b1 > a.total_tok || n < 0) {
        n = 0;
        cut = true;
    }
    if (n > a.max_tok) n = a.max_tok;
    if (ctx < 0) ctx = 0;
    cut |= ctx + n > most;
    if (cut && report && a.err) atomicOr(a.err, CBQ_DEVERR_BAD_LENGTH);
    return Seq{b0, (int)n, (int)(ctx < most ? ctx : most), (int)(ctx + n < most ? ctx + n : most), 0, 0};
}
__device__ __forceinline__ Seq sequence(const TreeAttention &a, NoOldPlaces, int s, bool report) { return sequence(a, s, report); }

// The same where the first places are in 8 bits: the places that are cut off
// those are seen nowhere, the recent ones begin behind them all the same.
__device__ __forceinline__ Seq sequence(const TreeAttention &a, const OldPlaces &b, int s, bool report) {
    const int64_t room = (int64_t)a.table_width * a.c.page_size, room8 = (int64_t)b.table_width * b.c.page_size;
    const int64_t b0 = __ldcg(a.start + s), b1 = __ldcg(a.start + s + 1);
    int64_t n = b1 - b0, ctx = __ldcg(a.ctx + s), from = __ldcg(b.old + s);
    bool cut = n > a.max_tok || ctx < 0 || from < 0 || from > ctx || from > CBQ_TREE_MAX_LEN;
    if (b0 < 0 || b1 > a.total_tok || n < 0) {
        n = 0;
        cut = true;
    }
    n = min(n, (int64_t)a.max_tok);
    ctx = max(ctx, (int64_t)0);
    from = min(max(min(from, ctx), (int64_t)0), (int64_t)CBQ_TREE_MAX_LEN);
    const int64_t old = min(from, min(b.max_old, room8));
    const int64_t most = max(min(min(from + b.max_new, room), (int64_t)INT32_MAX - 65536), from);
    cut |= old < from || ctx + n > most;
    if (cut && report && a.err) atomicOr(a.err, CBQ_DEVERR_BAD_LENGTH);
    return Seq{b0, (int)n, (int)min(ctx, most), (int)min(ctx + n, most), (int)from, (int)old};
}

// Bits of the drafts that row's token sees, none beyond the sequence's own.
__device__ __forceinline__ uint64_t seen_drafts(const TreeAttention &a, const Seq &q, int64_t row) {
    const int k = q.len - q.ctx;
    return (uint64_t)a.mask[row] & (k >= 64 ? ~0ull : (1ull << k) - 1);
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    } else {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
}
__device__ __forceinline__ float pow2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A part's sum of weights l under its own maximum m, under the maximum m - d of
// all (d <= 0).  kFar: the maxima hold the values' scales, which the sums do not,
// so what counts of a sum may be 2^192 of such steps away: by two halves, as
// 2^d alone would be 0 below 2^-126.
template <bool kFar>
__device__ __forceinline__ float part_sum(float l, float d) {
    if (!kFar) return l * pow2(d);
    const float half = pow2(0.5f * d);
    return l * half * half;
}

__device__ __forceinline__ float log2_of(float x) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two e4m3 numbers as fp16, which holds all of them.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint16_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
    return r;
}
__device__ __forceinline__ float e4m3_f32(uint8_t b) {
    const uint32_t two = e4m3_f16x2(b);
    return __low2float(*reinterpret_cast<const __half2 *>(&two));
}

// The power of two 2^k by which a row of q is held smaller as fp16: its largest
// magnitude comes to 2^14 .. 2^15.
__device__ __forceinline__ int row_exponent(float most) {
    return most > 0.0f && most < INFINITY ? max((int)(__float_as_uint(most) >> 23) - 127 - 14, -100) : 0;
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// A scale's logarithm as the running maxima count it.
__device__ __forceinline__ float scale_log2(float v) { return fminf(fmaxf(log2_of(v), -80.0f), 120.0f); }

// The wide kernel (cbq_attn_wide.cu; head sizes 64 and 128): 256 rows of a kv
// head a block, the committed keys from c * chunk on in block c, and the drafts
// in the sequence's last; with old places, those in the first b.n8 blocks.
constexpr int kWideRows = 256;
cudaError_t launch_tree_wide(const TreeAttention &a, NoOldPlaces b, int chunk, int n_chunks, int row_tiles, float *part_o,
                             float2 *part_ml, cudaStream_t s);
cudaError_t launch_tree_wide(const TreeAttention &a, const OldPlaces &b, int chunk, int n_chunks, int row_tiles, float *part_o,
                             float2 *part_ml, cudaStream_t s);

}  // namespace cbq
