// cbq_attn.cuh -- what the kernels of the tree attention share.
#pragma once

#include <type_traits>

#include "cbq_device.cuh"
#include "step/cbq_copy.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

constexpr int kMaxDim = 256;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// What a block needs to know of a sequence, with everything out of range cut.
struct Seq {
    int64_t row0;  // its first row of q
    int n, ctx, len;
};

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
    return Seq{b0, (int)n, (int)(ctx < most ? ctx : most), (int)(ctx + n < most ? ctx + n : most)};
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

// Launches kernel<<<grid, threads, smem>>> as a programmatic dependent of the
// work ahead, in clusters of `cluster` blocks along the grid's y.
template <typename... P, typename... A>
inline cudaError_t launch_clusters(void (*kernel)(P...), dim3 grid, int cluster, int threads, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = at[1].val.clusterDim.z = 1;
    at[1].val.clusterDim.y = (unsigned)cluster;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kernel, (P)args...) : e;
}
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
    return launch_clusters(kernel, grid, 1, threads, smem, s, args...);
}

// The wide kernel (cbq_attn_wide.cu; head sizes 64 and 128): 256 rows of a kv
// head a block, the committed keys from c * chunk on in block c, and the drafts
// in the sequence's last.
constexpr int kWideRows = 256;
cudaError_t launch_tree_wide(const TreeAttention &a, int chunk, int n_chunks, int row_tiles, float *part_o,
                             float2 *part_ml, cudaStream_t s);

}  // namespace cbq
