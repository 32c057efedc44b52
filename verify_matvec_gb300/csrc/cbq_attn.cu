// cbq_attn.cu -- attention of a tree of drafted tokens over a paged cache.
//
// For each sequence and kv head the rows are its drafted tokens times the
// query heads of the group, R = n G of them, and all of them read the same
// keys: one pass over K and V serves every row,
//   o = sum_p 2^(x_p - m) v_p / sum_p 2^(x_p - m),  x = scale log2(e) q.k,
// with the running maximum m and the running sum kept per row while the keys
// stream by (each new maximum scales what was summed before).  The keys are
// cut into chunks, a block each, so that a few sequences fill the GPU; the
// chunks' (m, sum, o) of a row are joined by a second kernel, or, where there
// are few, by the blocks themselves, which are a cluster then and read one
// another's shared memory (one launch, no workspace: what short calls need).
//
// Bound by memory where the contexts are long: two sequences of 131,000 keys
// (1.07 GB, 16 rows a kv head) take 169 to 179 us, 6.0 to 6.3 TB/s.  8,191 keys of one
// sequence (34 MB, 20 rows) take 14.9 us: a block's 256 keys, the two launches
// and the join follow one another; 300 keys 6.2 us, latency throughout.  The
// products run on mma.sync: a tile of K or V serves 64 rows at most here, and
// the copies are the bound, not the products.
#include <algorithm>

#include "cbq_pipe.cuh"
#include "step/cbq_attn.cuh"

namespace cbq {

namespace {

// Any head size and any strides: one warp per (token, head), the lanes hold
// the head's values, a key at a time.  Bound by that chain: each key's look-up,
// row of k, five shuffles and row of v follow one another, some 0.9 us (5 drafts
// over 8,191 keys 7.0 ms with heads of 96, 8.2 with 192).  grid (q_heads, max_tok, n_seq).
template <typename T>
__global__ void __launch_bounds__(32) k_tree_general(TreeAttention a) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x, h = blockIdx.x, i = blockIdx.y, s = blockIdx.z, D = a.c.head_dim;
    const Seq sq = sequence(a, s, lane == 0 && h == 0 && i == 0);
    if (i >= sq.n) return;
    const int64_t row = sq.row0 + i;
    const uint64_t mask = seen_drafts(a, sq, row);
    const T *q = static_cast<const T *>(a.q) + row * a.q_tok + h * a.q_head;
    const int g = h / (a.q_heads / a.c.kv_heads);
    float qv[kMaxDim / 32], acc[kMaxDim / 32];
#pragma unroll
    for (int j = 0; j < kMaxDim / 32; ++j) {
        acc[j] = 0.0f;
        qv[j] = j * 32 + lane < D ? to_f32(q[j * 32 + lane]) : 0.0f;
    }
    float top = -INFINITY, sum = 0.0f;
    for (int p = 0; p < sq.len; ++p) {
        if (p >= sq.ctx && !(mask >> (p - sq.ctx) & 1)) continue;
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

// ------------------------------------------------- the tensor-core kernel --

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (std::is_same_v<T, __nv_bfloat16>)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of p, a place in this block's shared memory, in block r of the cluster.
__device__ __forceinline__ uint32_t peer(const void *p, uint32_t r) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(r));
    return a;
}
__device__ __forceinline__ float2 peer_load2(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 peer_load4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
}

constexpr int kMaxCluster = 8;  // blocks that join one another's parts (plan())

// Blocks of k_tree_attention that run on an SM together, for its shared memory.
constexpr int blocks_an_sm(int head_dim) { return head_dim <= 64 ? 3 : head_dim <= 128 ? 2 : 1; }

// Sizes of the kernel for head size D and 16 * WR rows a block.  Four warps:
// WR of them share out the rows, and 4 / WR the keys of a tile.  Rows of a
// tile are padded by 16 bytes, which puts the eight rows of an ldmatrix into
// different banks.
template <int D, int WR>
struct Shape {
    static constexpr int kRows = 16 * WR, kParts = 4 / WR;
    static constexpr int kTile = D > 128 && WR > 1 ? 32 : 64;  // keys of a tile
    static constexpr int kKeys = kTile / kParts;               // of them, a warp's
    static constexpr int kCopied = kTile / 4;                  // rows that a warp copies
    static constexpr int kStages = 3;
    static constexpr int kPitch = 2 * D + 16;                  // bytes of a row
    static constexpr int kTileBytes = kTile * kPitch;
    static constexpr bool kHoldQ = D <= 128;                   // q's fragments stay in registers
    static constexpr int kRing = kStages * 2 * kTileBytes;
    // q (read again for every tile where it is not held) and the parts' results; the latter two may lie in the ring
    static constexpr int kSmem = kRing + (kHoldQ ? 0 : kRows * kPitch);
    static constexpr int kResult = kParts * kRows * D * 4;
    static_assert(kResult <= kRing && kRows * kPitch <= 2 * kTileBytes, "what lies in the ring fits it");
    static_assert(kKeys % 16 == 0, "16 keys a product");
};

// Chunk c of one (sequence, kv head, row tile): see the top of the file.
// Scores and sums are fp32; the weights 2^(x-m) are rounded to the cache's 16
// bits for the product with v (the tensor cores take no mixed types), so a
// weight is off by half a step, and the sum they are divided by is not
// rounded.  For fp16, whose weights below 2^-14 lose bits, m is kept 10 lower
// than the maximum: weights reach 2^10 and keep all bits down to 2^-24.
// What a row does not see: a key's score becomes -inf (weight 0), keys
// outside the sequence are not read and are zero in shared memory, and the
// drafts' values, which some rows see and others do not, are looked over for
// NaN and infinities first (they would make 0 * v NaN): such a value row is
// zeroed and added by hand to the rows that see it.  A NaN that a row does see
// makes its sum NaN, and so its results.
template <typename T, int D, int WR>
__global__ void __launch_bounds__(128, blocks_an_sm(D))
    k_tree_attention(TreeAttention a, int chunk, int row_tiles, bool cluster, float *part_o, float2 *part_ml) {
    using S = Shape<D, WR>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t valid[S::kStages][4];
    __shared__ uint64_t drafts[S::kRows];
    __shared__ float2 ml[S::kParts][S::kRows], joined[S::kRows];
    pdl_wait();
    pdl_trigger();  // (after the wait: the join reads what this call was given before it waits)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wr = warp % WR, wk = warp / WR;
    const int kvh = blockIdx.x / row_tiles, r0 = blockIdx.x % row_tiles * S::kRows, c = blockIdx.y, s = blockIdx.z;
    const int group = a.q_heads / a.c.kv_heads;
    const Seq sq = sequence(a, s, tid == 0 && blockIdx.x == 0 && c == 0);
    const int rows = min(sq.n * group - r0, S::kRows);
    const int begin = c * chunk, end = min(sq.len, begin + chunk);
    // a row that has no keys at all is written by its first block
    if (rows <= 0 || (begin >= end && c > 0)) return;
    const bool alone = sq.len <= chunk;  // the only chunk of this sequence

    // copies: each warp brings kCopied rows of a tile; lane l < kCopied keeps the place of row l
    const int tiles = (end - begin + S::kTile - 1) / S::kTile;
    const int32_t *table = a.table + (int64_t)s * a.table_width;
    const int64_t head = kvh * a.c.head_stride;
    auto page_of = [&](int t) {  // the page of this lane's row of tile t, -1 past the end
        const int p = begin + t * S::kTile + warp * S::kCopied + lane;
        return lane < S::kCopied && p < end ? table[(uint32_t)p / (uint32_t)a.c.page_size] : -1;
    };
    auto fetch = [&](int t, int page) {
        const int slot = t % S::kStages;
        const uint32_t p = begin + t * S::kTile + warp * S::kCopied + lane;
        const bool in = lane < S::kCopied && p < (uint32_t)end, good = in && page >= 0 && page < a.c.n_pages;
        if (in && !good && a.err) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
        const int64_t at = good ? page * a.c.page_stride + (int64_t)(p % (uint32_t)a.c.page_size) * a.c.tok_stride + head : -1;
        const uint32_t bits = __ballot_sync(~0u, good);
        if (lane == 0) valid[slot][warp] = bits;
        const uint32_t ks = smem_addr(smem) + slot * 2 * S::kTileBytes + warp * S::kCopied * S::kPitch;
#pragma unroll
        for (int i = 0; i < S::kCopied * (D / 8) / 32; ++i) {
            const int x = i * 32 + lane, r = x / (D / 8), d = x % (D / 8);
            const int64_t from = __shfl_sync(~0u, at, r);
            const int64_t off = from < 0 ? 0 : from + d * 8;
            copy16(ks + r * S::kPitch + d * 16, static_cast<const T *>(a.c.k) + off, from >= 0);
            copy16(ks + S::kTileBytes + r * S::kPitch + d * 16, static_cast<const T *>(a.c.v) + off, from >= 0);
        }
    };
    static_assert(S::kCopied * (D / 8) % 32 == 0, "whole warps of copies");
    // What the first tiles and the rows need from memory is asked for together: their pages, q (row r: token r / group,
    // head r % group of the group) and the masks.
    int pages[S::kStages];
#pragma unroll
    for (int t = 0; t < S::kStages; ++t) pages[t] = t < tiles ? page_of(t) : -1;
    const float sc = fabsf(a.scale) * kLog2e;
    const bool q_whole = (reinterpret_cast<uintptr_t>(a.q) % 16 | (a.q_tok | a.q_head) % 8) == 0;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;  // (the sign of the scale goes with q)
    uint4 qv[S::kRows * (D / 8) / 128];
#pragma unroll
    for (int x = 0; x < S::kRows * (D / 8) / 128; ++x) {
        const int r = (x * 128 + tid) / (D / 8), d = (x * 128 + tid) % (D / 8);
        qv[x] = make_uint4(0, 0, 0, 0);
        if (r < rows) {
            const int tok = (r0 + r) / group, h = kvh * group + (r0 + r) % group;
            const T *from = static_cast<const T *>(a.q) + (sq.row0 + tok) * a.q_tok + h * a.q_head + d * 8;
            if (q_whole) {
                qv[x] = *reinterpret_cast<const uint4 *>(from);
            } else {
                __align__(16) T y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = from[e];
                qv[x] = *reinterpret_cast<const uint4 *>(y);
            }
        }
    }
    const uint64_t tree = tid < rows ? seen_drafts(a, sq, sq.row0 + (r0 + tid) / group) : 0;
#pragma unroll
    for (int t = 0; t < S::kStages - 1; ++t) {
        if (t < tiles) fetch(t, pages[t]);
        copy_commit();
    }
    int page = pages[S::kStages - 1];
    uint8_t *qs = S::kHoldQ ? smem + (S::kStages - 1) * 2 * S::kTileBytes : smem + S::kRing;
#pragma unroll
    for (int x = 0; x < S::kRows * (D / 8) / 128; ++x) {
        const int r = (x * 128 + tid) / (D / 8), d = (x * 128 + tid) % (D / 8);
        *reinterpret_cast<uint4 *>(qs + r * S::kPitch + d * 16) = make_uint4(qv[x].x ^ flip, qv[x].y ^ flip, qv[x].z ^ flip, qv[x].w ^ flip);
    }
    if (tid < S::kRows) drafts[tid] = tree;
    __syncthreads();
    const uint32_t q_at = smem_addr(qs) + (wr * 16 + lane % 16) * S::kPitch + lane / 16 * 16;
    uint32_t qf[S::kHoldQ ? D / 16 : 1][4];
    if constexpr (S::kHoldQ) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) ldsm4(qf[k], q_at + k * 32);
    }

    constexpr float kLower = std::is_same_v<T, __half> ? 10.0f : 0.0f;
    float o[D / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int ra = wr * 16 + lane / 4;  // this lane's rows are ra and ra + 8
    for (int t = 0; t < tiles; ++t) {
        copy_wait<S::kStages - 2>();
        __syncthreads();
        if (t + S::kStages - 1 < tiles) {
            fetch(t + S::kStages - 1, page);
            if (t + S::kStages < tiles) page = page_of(t + S::kStages);
        }
        copy_commit();
        const int slot = t % S::kStages, key0 = begin + t * S::kTile;
        uint8_t *kt = smem + slot * 2 * S::kTileBytes, *vt = kt + S::kTileBytes;

        // scores of this warp's keys
        float x[S::kKeys / 8][4] = {};
        const uint32_t k_at = smem_addr(kt) + (wk * S::kKeys + lane % 8 + lane / 16 * 8) * S::kPitch + lane / 8 % 2 * 16;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
            uint32_t qk[4];
            if constexpr (!S::kHoldQ) ldsm4(qk, q_at + k * 32);
#pragma unroll
            for (int j = 0; j < S::kKeys / 16; ++j) {
                uint32_t b[4];
                ldsm4(b, k_at + j * 16 * S::kPitch + k * 32);
                if constexpr (S::kHoldQ) {
                    mma<T>(x[2 * j], qf[k], b[0], b[1]);
                    mma<T>(x[2 * j + 1], qf[k], b[2], b[3]);
                } else {
                    mma<T>(x[2 * j], qk, b[0], b[1]);
                    mma<T>(x[2 * j + 1], qk, b[2], b[3]);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < S::kKeys / 8; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j][e] *= sc;

        // tiles with drafts, a ragged end or missing pages: the keys each row sees, bit by bit
        uint64_t there = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) there |= (uint64_t)valid[slot][w] << (w * S::kCopied);
        const bool special = key0 + S::kTile > sq.ctx || there != (S::kTile == 64 ? ~0ull : (1ull << S::kTile) - 1);
        uint64_t odd = 0;  // keys whose values are not all finite
        if (special) {
            const int known = min(max(sq.ctx - key0, 0), 64);  // committed keys of the tile
            const uint64_t old = known == 64 ? ~0ull : (1ull << known) - 1;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const uint64_t tree = drafts[ra + half * 8];
                const int gone = key0 - sq.ctx;  // drafts before this tile
                const uint64_t sees = (old | (known == 64 ? 0 : gone > 0 ? (gone < 64 ? tree >> gone : 0) : tree << known)) & there;
                const uint32_t mine = (uint32_t)(sees >> (wk * S::kKeys + lane % 4 * 2));
                const uint32_t more = S::kKeys > 32 ? (uint32_t)(sees >> (wk * S::kKeys + lane % 4 * 2 + 32)) : 0;
#pragma unroll
                for (int j = 0; j < S::kKeys / 8; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (!((j < 4 ? mine >> (j * 8 + e) : more >> (j * 8 - 32 + e)) & 1)) x[j][half * 2 + e] = -INFINITY;
            }
            if (key0 + S::kTile > sq.ctx) {
                // exponent bits all ones in any 16-bit half: NaN or infinity
                constexpr uint32_t kExp = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;
                __shared__ unsigned long long found;
                if (tid == 0) found = 0;
                __syncthreads();
                for (int i = tid; i < S::kTile * (D / 8); i += 128) {
                    const int r = i / (D / 8);
                    const uint4 v = *reinterpret_cast<const uint4 *>(vt + r * S::kPitch + i % (D / 8) * 16);
                    bool bad = false;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t y = w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
                        bad |= (y & kExp) == kExp || (y >> 16 & kExp) == kExp;
                    }
                    if (bad && key0 + r >= sq.ctx) atomicOr(&found, 1ull << r);
                }
                __syncthreads();
                odd = found;
                if (odd) {
                    for (int i = tid; i < S::kTile * (D / 8); i += 128)
                        if (odd >> (i / (D / 8)) & 1)
                            *reinterpret_cast<uint4 *>(vt + i / (D / 8) * S::kPitch + i % (D / 8) * 16) = make_uint4(0, 0, 0, 0);
                    __syncthreads();
                }
            }
        }

        // the running maximum of each row over its four lanes, and what it scales
        float shift[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            float top = -INFINITY;
#pragma unroll
            for (int j = 0; j < S::kKeys / 8; ++j) top = fmaxf(top, fmaxf(x[j][half * 2], x[j][half * 2 + 1]));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const float now = fmaxf(m[half], top - kLower);
            shift[half] = now == -INFINITY ? 0.0f : now;  // nothing seen yet: every weight stays 0
            const float keep = pow2(m[half] - shift[half]);
            m[half] = now;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < S::kKeys / 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    x[j][half * 2 + e] = pow2(x[j][half * 2 + e] - shift[half]);
                    sum += x[j][half * 2 + e];
                }
            l[half] = l[half] * keep + sum;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                o[d][half * 2] *= keep;
                o[d][half * 2 + 1] *= keep;
            }
        }
        const uint32_t v_at = smem_addr(vt) + (wk * S::kKeys + lane % 16) * S::kPitch + lane / 16 * 16;
#pragma unroll
        for (int j = 0; j < S::kKeys / 16; ++j) {
            const uint32_t p[4] = {pack2<T>(x[2 * j][0], x[2 * j][1]), pack2<T>(x[2 * j][2], x[2 * j][3]),
                                   pack2<T>(x[2 * j + 1][0], x[2 * j + 1][1]), pack2<T>(x[2 * j + 1][2], x[2 * j + 1][3])};
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                uint32_t b[4];
                ldsm4t(b, v_at + j * 16 * S::kPitch + d * 32);
                mma<T>(o[2 * d], p, b[0], b[1]);
                mma<T>(o[2 * d + 1], p, b[2], b[3]);
            }
        }
        if (odd) {  // value rows taken out above: by hand, for the rows that see them
            for (int key = wk * S::kKeys; key < (wk + 1) * S::kKeys; ++key) {
                if (!(odd >> key & 1)) continue;
                const uint32_t p = key0 + key;
                const int64_t at = table[p / (uint32_t)a.c.page_size] * a.c.page_stride +
                                   (int64_t)(p % (uint32_t)a.c.page_size) * a.c.tok_stride + head;
                const int local = key - wk * S::kKeys;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    float w = 0.0f;
#pragma unroll
                    for (int j = 0; j < S::kKeys / 8; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (j * 8 + e == (local & ~7) + (local & 1)) w = x[j][half * 2 + e];
                    w = __shfl_sync(~0u, w, (lane & ~3) | (local & 7) >> 1);
                    if (!(drafts[ra + half * 8] >> (p - sq.ctx) & 1)) continue;
#pragma unroll
                    for (int d = 0; d < D / 8; ++d)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            o[d][half * 2 + e] += w * to_f32(static_cast<const T *>(a.c.v)[at + d * 8 + lane % 4 * 2 + e]);
                }
            }
        }
    }
    copy_wait<0>();

    // join the warps that shared out the keys, then one division
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        l[half] += __shfl_xor_sync(~0u, l[half], 1);
        l[half] += __shfl_xor_sync(~0u, l[half], 2);
        if (l[half] != l[half]) m[half] = 0.0f;  // (no maximum keeps a NaN: what joins the parts must not take them for empty)
        if (lane % 4 == 0) ml[wk][ra + half * 8] = make_float2(m[half], l[half]);
    }
    __syncthreads();
    float *res = reinterpret_cast<float *>(smem);  // [part][row][D]
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = ra + half * 8;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < S::kParts; ++w) top = fmaxf(top, ml[w][r].x);
        const float f = top == -INFINITY ? 1.0f : pow2(m[half] - top);
#pragma unroll
        for (int d = 0; d < D / 8; ++d)
            *reinterpret_cast<float2 *>(res + (wk * S::kRows + r) * D + d * 8 + lane % 4 * 2) =
                make_float2(o[d][half * 2] * f, o[d][half * 2 + 1] * f);
    }
    __syncthreads();
    auto row_of = [&](int r) { return (sq.row0 + (r0 + r) / group) * a.q_heads + kvh * group + (r0 + r) % group; };
    auto put = [&](int64_t row, int d, float4 v, float top, float sum) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        if (a.out_f32)
            *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * D + d) = make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        else
            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row * D + d) = make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
        if (a.lse && d == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    };
    for (int i = tid; i < rows * (D / 4); i += 128) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int w = 0; w < S::kParts; ++w) top = fmaxf(top, ml[w][r].x);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < S::kParts; ++w) {
            if (top != -INFINITY) sum += ml[w][r].y * pow2(ml[w][r].x - top);
            const float4 y = *reinterpret_cast<const float4 *>(res + (w * S::kRows + r) * D + d);
            v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
        }
        if (!alone && cluster) {
            *reinterpret_cast<float4 *>(res + r * D + d) = v;  // (only this thread has read it)
            if (d == 0) joined[r] = make_float2(top, sum);
            continue;
        }
        const int64_t row = row_of(r);
        if (!alone) {
            const int64_t at = (int64_t)c * a.total_tok * a.q_heads + row;
            *reinterpret_cast<float4 *>(part_o + at * D + d) = v;
            if (d == 0) part_ml[at] = make_float2(top, sum);
            continue;
        }
        put(row, d, v, top, sum);
    }
    if (alone || !cluster) return;
    // the blocks of the sequence's chunks share out its values: each takes its part from all of them
    const int chunks = (sq.len + chunk - 1) / chunk;
    cluster_sync();
    for (int i = c * 128 + tid; i < rows * (D / 4); i += chunks * 128) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float2 m_of[kMaxCluster];
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int o = 0; o < kMaxCluster; ++o) {
            m_of[o] = o < chunks ? peer_load2(peer(&joined[r], o)) : make_float2(-INFINITY, 0.0f);
            top = fmaxf(top, m_of[o].x);
        }
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int o = 0; o < kMaxCluster; ++o) {
            if (o >= chunks) continue;
            const float4 y = peer_load4(peer(res + r * D + d, o));
            const float f = top == -INFINITY ? 0.0f : pow2(m_of[o].x - top);
            sum += m_of[o].y * f;
            v.x += y.x * f, v.y += y.y * f, v.z += y.z * f, v.w += y.w * f;
        }
        put(row_of(r), d, v, top, sum);
    }
    cluster_sync();  // no block leaves while another reads its shared memory
}

// The chunks of a row (token, head) joined by W warps: with many chunks and few
// rows the eight warps of a block share out those of one row (one warp going
// through 32 chunks took 18 us of a 33 us call), otherwise each takes a row of
// its own.  Eight parts' loads are under way together, each warp keeps its own
// running maximum, and what the call was given is read while the parts' kernel
// still runs (8,191 keys of one sequence 17.0 us before that, 14.6 with it).  The
// wide kernel cuts the committed keys alone (and takes the drafts with the last
// chunk).  grid (ceil(q_heads * W / 8), max_tok, n_seq).
template <typename T, int D, int W>
__global__ void __launch_bounds__(256) k_tree_join(TreeAttention a, int chunk, bool wide, const float *part_o, const float2 *part_ml) {
    constexpr int kEach = D / 32;  // values of a lane, side by side
    struct alignas(kEach * 4 < 16 ? kEach * 4 : 16) Values {
        float v[kEach];
    };
    __shared__ float tops[W], sums[W];
    __shared__ Values vals[W][W > 1 ? 32 : 1];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, w = warp % W, h = blockIdx.x * (8 / W) + warp / W, i = blockIdx.y;
    // (the parts' kernel lets this one start when what the two are given is there: only the parts have to be waited for)
    const Seq sq = sequence(a, blockIdx.z, false);
    pdl_wait();
    const int chunks = ((wide ? sq.ctx : sq.len) + chunk - 1) / chunk;
    if (i >= sq.n || h >= a.q_heads || chunks <= 1) return;  // (all warps of a row alike)
    const int64_t row = (sq.row0 + i) * a.q_heads + h, step = a.total_tok * a.q_heads;
    Values v = {};
    float top = -INFINITY, sum = 0.0f;
    for (int c0 = w; c0 < chunks; c0 += 8 * W) {  // eight parts' loads at once
        float2 p[8];
        Values y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + j * W;
            p[j] = make_float2(-INFINITY, 0.0f);
            y[j] = {};
            if (c >= chunks) continue;
            p[j] = part_ml[c * step + row];
            y[j] = reinterpret_cast<const Values *>(part_o + (c * step + row) * D)[lane];
        }
        float now = top;
#pragma unroll
        for (int j = 0; j < 8; ++j) now = fmaxf(now, p[j].x);
        if (now == -INFINITY) continue;
        const float keep = pow2(top - now);
        sum *= keep;
#pragma unroll
        for (int e = 0; e < kEach; ++e) v.v[e] *= keep;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = pow2(p[j].x - now);
            sum += p[j].y * f;
#pragma unroll
            for (int e = 0; e < kEach; ++e) v.v[e] += f * y[j].v[e];
        }
        top = now;
    }
    if constexpr (W > 1) {
        if (lane == 0) tops[w] = top, sums[w] = sum;
        vals[w][lane] = v;
        __syncthreads();
        if (w > 0) return;
#pragma unroll
        for (int o = 1; o < W; ++o) top = fmaxf(top, tops[o]);
        sum = 0.0f;
        v = {};
        if (top != -INFINITY) {
#pragma unroll
            for (int o = 0; o < W; ++o) {
                const float f = pow2(tops[o] - top);
                const Values y = vals[o][lane];
                sum += f * sums[o];
#pragma unroll
                for (int e = 0; e < kEach; ++e) v.v[e] += f * y.v[e];
            }
        }
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int64_t at = row * D + lane * kEach + j;
        if (a.out_f32) static_cast<float *>(a.out)[at] = v.v[j] * inv;
        else static_cast<T *>(a.out)[at] = from_f32<T>(v.v[j] * inv);
    }
    if (a.lse && lane == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// How a call is cut: rows of a block (16 * wr, or the wide kernel's 256), tiles
// of them, and the chunk of keys a block takes.
struct Plan {
    bool wide, cluster;  // the wide kernel; the chunks' blocks join one another
    int wr, row_tiles, chunk, n_chunks;
};

constexpr int kSms = 152;  // of a GB300 (the size of a workspace is asked for without a device, too)

// Many rows are the wide kernel's.  us by tiles of 64 rows / by the wide kernel, D = 128, 8 kv heads, one sequence: 40 rows
// at 200 keys 10.4 / 11.5, at 1,000 12.2 / 12.4, at 8,000 19.4 / 16.8; 256 rows 15.0 / 18.7, 28.5 / 23.3, 54.5 / 29.3.
// 24 sequences: 40 rows 29 / 20, 53 / 36, 204 / 154.  D = 64, 5 kv heads: 78 rows at 200 keys 8.1 / 9.8, at 8,000 15.4 /
// 14.3; 8 sequences of 384 rows 25 / 11, 152 / 85; 24 sequences of 40 rows, 8 kv heads, 12 / 16, 116 / 113.
bool wide_rows(int n_seq, int rows, int64_t max_len, int kv_heads, int head_dim) {
    if (head_dim > 128) return false;
    const bool full = (int64_t)n_seq * kv_heads * ((rows + 63) / 64) >= kSms;  // tiles of 64 rows would fill the GPU
    return head_dim > 64 ? rows > 32 && (full || max_len >= 512) : rows > 64 && (full || max_len >= 1024);
}

Plan plan(int n_seq, int max_tok, int64_t max_len, int q_heads, int kv_heads, int head_dim) {
    Plan p = {};
    const int rows = max_tok * (q_heads / kv_heads);
    p.wide = wide_rows(n_seq, rows, max_len, kv_heads, head_dim);
    int64_t n = 1;
    p.wr = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    const int block_rows = p.wide ? kWideRows : 16 * p.wr;
    p.row_tiles = (rows + block_rows - 1) / block_rows;
    const int64_t blocks = (int64_t)n_seq * kv_heads * p.row_tiles;
    if (p.wide) {
        // A chunk costs a block about 10 ns a key and 6 us for its results; the join 3 us and the way of the parts to memory
        // and back (5 TB/s): the n with the least time over all waves.  8 sequences of 256 rows x 500 keys: one chunk 20
        // us, two 26; one sequence of 128 rows x 8,000: one 75, eight 21, sixteen 19, 24 30.
        const double part_us = (double)n_seq * kv_heads * rows * head_dim * 8.0 / 5e6;
        double least = 0.0;
        for (int64_t m = 1; m <= 64; ++m) {
            const double t = (double)((blocks * m + kSms - 1) / kSms) * ((double)max_len / m * 0.01 + 6.0) + (m > 1 ? 3.0 + part_us * m : 0.0);
            if (m == 1 || t < least) least = t, n = m;
        }
        // several sequences may differ in length: no block takes much longer than others, as long as the parts' bytes stay
        // small beside the keys'
        if (n_seq > 1) n = std::max(n, max_len / std::max(2048, 32 * rows));
    } else {
        // A block takes 24 ns a key, and 1.6 us and 0.17 a row for the rest; a join by a second kernel costs 2.5 us and one
        // inside clusters 1.5.  Looked at are the most chunks that fill one wave of blocks, two, three and four: 24
        // sequences of 2,000 keys (8 kv heads, D = 128) take 47 us in 192 blocks, 53 in 384, 43 in 576 (two waves), 48 in
        // 768.  Several sequences may differ in length: half the time with half of the chunks empty counts beside the time
        // with none.  Clusters of more than eight blocks, or beyond one wave, were slower than the second kernel.
        const int64_t slots = kSms * blocks_an_sm(head_dim), most = (max_len + 63) / 64;
        const double rest = 1.6 + 0.17 * std::min(rows, block_rows);
        double least = 0.0;
        for (int64_t w = 0; w <= 4; ++w) {
            const int64_t cut = w ? std::min(most, w * slots / blocks) : 1;
            if (w && cut <= 1) continue;
            const int64_t keys = ((max_len + cut - 1) / cut + 63) / 64 * 64, m = (max_len + keys - 1) / keys;
            const bool cluster = m > 1 && m <= kMaxCluster && blocks * m <= slots;
            const double each = (double)keys * 0.024 + rest;
            double t = (double)((blocks * m + slots - 1) / slots) * each;
            if (n_seq > 1) t += 0.5 * (double)((blocks * m / 2 + slots - 1) / slots) * each;
            t += m == 1 ? 0.0 : cluster ? 1.5 : 2.5;
            if (w == 0 || t < least) least = t, n = m, p.cluster = cluster;
        }
    }
    n = std::min<int64_t>(n, 65535);  // of the grid's second axis
    int64_t chunk = (max_len + n - 1) / n;
    chunk = (chunk + 63) / 64 * 64;
    p.chunk = (int)chunk;
    p.n_chunks = (int)((max_len + p.chunk - 1) / p.chunk);
    p.cluster = p.cluster && p.n_chunks > 1;
    return p;
}

bool tiled_dim(int d) { return d == 64 || d == 128 || d == 256; }

template <typename T, int D, int WR>
cudaError_t launch_tiled(const TreeAttention &a, const Plan &p, cudaStream_t s) {
    const size_t rows = (size_t)a.total_tok * a.q_heads;
    float2 *part_ml = static_cast<float2 *>(a.ws);
    float *part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + (rows * p.n_chunks * sizeof(float2) + 15) / 16 * 16);
    const cudaError_t e = p.wide ? launch_tree_wide(a, p.chunk, p.n_chunks, p.row_tiles, part_o, part_ml, s)
                                 : launch_clusters(k_tree_attention<T, D, WR>,
                                                   dim3((unsigned)(a.c.kv_heads * p.row_tiles), (unsigned)p.n_chunks, (unsigned)a.n_seq),
                                                   p.cluster ? p.n_chunks : 1, 128, Shape<D, WR>::kSmem, s, a, p.chunk, p.row_tiles,
                                                   p.cluster, part_o, part_ml);
    if (e != cudaSuccess || p.n_chunks == 1 || p.cluster) return e;
    // (before its loads went together: a warp for each of 1,024 rows of 19 chunks 21.3 us a call, eight warps 20.4; of
    // 2,048 rows 28.0 and 30.2; a ragged batch of 5,000 rows of up to 12 chunks 62 and 65)
    const unsigned heads = (unsigned)a.q_heads, toks = (unsigned)a.max_tok, seqs = (unsigned)a.n_seq;
    return p.n_chunks > 8 && rows < 2048 ? launch_dependent(k_tree_join<T, D, 8>, dim3(heads, toks, seqs), 256, 0, s, a, p.chunk, p.wide, part_o, part_ml)
                          : launch_dependent(k_tree_join<T, D, 1>, dim3((heads + 7) / 8, toks, seqs), 256, 0, s, a, p.chunk, p.wide,
                                             part_o, part_ml);
}

template <typename T, int D>
cudaError_t launch_dim(const TreeAttention &a, const Plan &p, cudaStream_t s) {
    return p.wr == 1 ? launch_tiled<T, D, 1>(a, p, s) : p.wr == 2 ? launch_tiled<T, D, 2>(a, p, s) : launch_tiled<T, D, 4>(a, p, s);
}

template <typename T>
cudaError_t launch_type(const TreeAttention &a, cudaStream_t s) {
    // 16-byte copies want every row of k and v on a 16-byte boundary, 16-byte stores every row of out
    const uintptr_t ends = reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v) | reinterpret_cast<uintptr_t>(a.out);
    if (tiled_dim(a.c.head_dim) && ends % 16 == 0 && (a.c.page_stride | a.c.tok_stride | a.c.head_stride) % 8 == 0) {
        const Plan p = plan(a.n_seq, a.max_tok, a.max_len, a.q_heads, a.c.kv_heads, a.c.head_dim);
        if (a.c.head_dim == 64) return launch_dim<T, 64>(a, p, s);
        if (a.c.head_dim == 128) return launch_dim<T, 128>(a, p, s);
        return launch_dim<T, 256>(a, p, s);
    }
    return launch_dependent(k_tree_general<T>, dim3((unsigned)a.q_heads, (unsigned)a.max_tok, (unsigned)a.n_seq), 32, 0, s, a);
}

}  // namespace

size_t tree_attention_workspace(int n_seq, int64_t total_tok, int max_tok, int64_t max_len, int q_heads, int kv_heads,
                                int head_dim) {
    if (!tiled_dim(head_dim)) return 16;
    const Plan p = plan(n_seq, max_tok, max_len, q_heads, kv_heads, head_dim);
    if (p.n_chunks == 1 || p.cluster) return 16;
    const size_t rows = (size_t)total_tok * q_heads * p.n_chunks;
    return (rows * sizeof(float2) + 15) / 16 * 16 + rows * head_dim * sizeof(float);
}

cudaError_t launch_tree_attention(const TreeAttention &a, cudaStream_t s) {
    return a.c.dtype == CBQ_BF16 ? launch_type<__nv_bfloat16>(a, s) : launch_type<__half>(a, s);
}

}  // namespace cbq
