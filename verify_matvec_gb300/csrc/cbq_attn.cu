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
//
// Old places in 8 bits are blocks of their own, joined with the others' (chunks
// 0 .. n8 - 1 of old places, then those of 16 bits).  Half the bytes, and the
// products are the bound: mma.sync takes 512 multiplications a clock of an SM,
// and 16 rows are padded where there are fewer.  Two sequences of 131,000 keys
// (538 MB) take 106 us, 5.1 TB/s, where 16 bits take 169 to 179; 32 rows 153.
// 300 keys 6.3 us.  (A maximum that follows late, a branch where 16 keys have
// one scale, or three blocks an SM: 105, 116, 108.)
#include <algorithm>

#include "cbq_pipe.cuh"
#include "step/cbq_attn.cuh"

namespace cbq {

namespace {

// Any head size and any strides: one warp per (token, head), the lanes hold
// the head's values, a key at a time.  Bound by that chain: each key's look-up,
// row of k, five shuffles and row of v follow one another, some 0.9 us (5 drafts
// over 8,191 keys 7.0 ms with heads of 96, 8.2 with 192).  grid (q_heads, max_tok, n_seq).
template <typename T, typename Old>
__global__ void __launch_bounds__(32) k_tree_general(TreeAttention a, Old b) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x, h = blockIdx.x, i = blockIdx.y, s = blockIdx.z, D = a.c.head_dim;
    const Seq sq = sequence(a, b, s, lane == 0 && h == 0 && i == 0);
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
    // one more key, of the head's values k and v as this lane reads them
    auto see = [&](auto k, auto v) {
        float x = 0.0f;
#pragma unroll
        for (int j = 0; j < kMaxDim / 32; ++j)
            if (j * 32 + lane < D) x += qv[j] * k(j * 32 + lane);
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
        x *= a.scale;
        const float now = fmaxf(top, x);
        // nothing of weight so far (top is -inf): a score of -inf has none either
        const float keep = top == -INFINITY ? 0.0f : expf(top - now), w = x == -INFINITY ? 0.0f : expf(x - now);
        sum = sum * keep + w;
#pragma unroll
        for (int j = 0; j < kMaxDim / 32; ++j)
            if (j * 32 + lane < D) acc[j] = acc[j] * keep + w * v(j * 32 + lane);
        top = now;
    };
    auto known = [&](int64_t page, int64_t pages) {
        const bool good = page >= 0 && page < pages;
        if (!good && a.err && lane == 0) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
        return good;
    };
    if constexpr (std::is_same_v<Old, OldPlaces>) {
        for (int p = 0; p < sq.old; ++p) {
            const int64_t page = b.table[s * (int64_t)b.table_width + p / b.c.page_size];
            if (!known(page, b.c.n_pages)) continue;
            const int t = p % b.c.page_size;
            const int64_t at = page * b.c.page_stride + t * b.c.tok_stride + g * b.c.head_stride;
            const int64_t of = page * b.c.scale_page_stride + t / b.c.block * b.c.scale_block_stride + g * b.c.scale_head_stride;
            const uint8_t *k = static_cast<const uint8_t *>(b.c.k) + at, *v = static_cast<const uint8_t *>(b.c.v) + at;
            const float ks = b.c.k_scale[of], vs = b.c.v_scale[of];
            see([&](int d) { return ks * e4m3_f32(k[d]); }, [&](int d) { return vs * e4m3_f32(v[d]); });
        }
    }
    for (int p = sq.from; p < sq.len; ++p) {
        if (p >= sq.ctx && !(mask >> (p - sq.ctx) & 1)) continue;
        const int64_t page = a.table[s * (int64_t)a.table_width + p / a.c.page_size];
        if (!known(page, a.c.n_pages)) continue;
        const int64_t at = page * a.c.page_stride + p % a.c.page_size * a.c.tok_stride + g * a.c.head_stride;
        const T *k = static_cast<const T *>(a.c.k) + at, *v = static_cast<const T *>(a.c.v) + at;
        see([&](int d) { return to_f32(k[d]); }, [&](int d) { return to_f32(v[d]); });
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
    // old places: half the bytes, so twice the keys in the same ring
    static constexpr int kTile8 = 2 * kTile, kKeys8 = kTile8 / kParts, kCopied8 = kTile8 / 4, kTileBytes8 = kTile8 * D;
    static constexpr int kStages8 = kRing / (2 * kTileBytes8);
    static_assert(kStages8 >= 3, "which is without the rows' padding");
};

// The old places' share of a block's shared memory: their scales, and which of a tile there are.
template <typename S>
struct OldShared {
    float ks[S::kStages8][S::kTile8], vs[S::kStages8][S::kTile8];
    uint32_t valid[S::kStages8][4];
};

// The old places [begin, end) of a chunk, whose keys and values are e4m3 numbers
// and scales, into the running o, m and l of this lane's rows.
//   x = (scale log2(e) 2^k) ks (q 2^-k).k,   w = 2^(x - m),   l += w,
//   o += (w vs) v,                           m = max (x + log2 vs):
// the numbers of k and v go into the products as they are, as fp16, which holds
// every e4m3 number; a row of q does too, scaled to a largest magnitude of 2^14
// to 2^15 by its own power of two 2^k; the scale of a key comes to its score and
// that of a value to its weight.  The maximum is of what the weights are with
// their scales, so they stay within fp16 (and as in the kernel below, 2^10 above
// the running maximum's).  l, without them, may be larger or smaller than that by
// a block's scale, and fp32 has the room for 2^-80 <= vs <= 2^112; but not for
// the factor from one maximum to the next, 2^-192 at the least, which therefore
// goes on l in two halves here and where parts are joined (part_sum()).
// Fragments: the order of the summed axis is free as long as both sides have it,
// so a lane takes 16 bytes side by side of a key's row for four products, and
// the same 16 values of q; and the values come through a transposing load of
// 16-bit pairs, whose even and odd bytes make the fragments of the even and of
// the odd columns.
template <typename T, int D, int WR>
__device__ __forceinline__ void old_places(const TreeAttention &a, const OldPlaces &b, const Seq &sq, OldShared<Shape<D, WR>> &sh,
                                           uint8_t *smem, int begin, int end, int r0, int rows, int kvh, int s, float (&o)[D / 8][4],
                                           float (&m)[2], float (&l)[2]) {
    using S = Shape<D, WR>;
    constexpr int kPieces = D / 16;  // 16-byte pieces of a row
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, wr = warp % WR, wk = warp / WR, ra = wr * 16 + lane / 4, t4 = lane % 4;
    const int group = a.q_heads / a.c.kv_heads;
    const int tiles = (end - begin + S::kTile8 - 1) / S::kTile8;
    const int32_t *table = b.table + (int64_t)s * b.table_width;
    const int64_t head = kvh * b.c.head_stride;
    // keys are looked up in order: the next tile's key is some pages and tokens on (no divisions)
    const uint32_t size = b.c.page_size, pages_on = S::kTile8 / size, tokens_on = S::kTile8 % size;
    int p = begin + warp * S::kCopied8 + lane;  // this lane's row of the tile that is looked up next
    uint32_t entry = (uint32_t)p / size, token = (uint32_t)p % size;
    struct Look {
        int page, within;  // the id of the key's page, and the token within (-1 where there is no such key)
    };
    auto look = [&] {
        const bool key = lane < S::kCopied8 && p < end;
        const Look l = {key ? table[entry] : -1, key ? (int)token : -1};
        p += S::kTile8;
        entry += pages_on;
        token += tokens_on;
        if (token >= size) token -= size, ++entry;
        return l;
    };
    // Pieces of a row are permuted by the row: keys so that two rows of four pieces meet no bank conflict, values so that
    // eight rows of one piece meet none.
    auto place_k = [](int r, int d) { return r * D + (D > 64 ? d ^ (r & 1) * 4 : d) * 16; };
    auto place_v = [](int r, int d) { return r * D + (D > 64 ? d ^ (r & 7) : d ^ (r >> 1 & 3)) * 16; };
    auto fetch = [&](int slot, const Look &now) {
        const bool in = now.within >= 0, good = in && now.page >= 0 && now.page < b.c.n_pages;
        if (in && !good && a.err) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
        const int64_t at = good ? now.page * b.c.page_stride + now.within * b.c.tok_stride + head : -1;
        const uint32_t bits = __ballot_sync(~0u, good);
        if (lane == 0) sh.valid[slot][warp] = bits;
        if (lane < S::kCopied8) {
            const int64_t of = good ? now.page * b.c.scale_page_stride + (uint32_t)now.within / (uint32_t)b.c.block * b.c.scale_block_stride +
                                          kvh * b.c.scale_head_stride : 0;
            copy4(smem_addr(&sh.ks[slot][warp * S::kCopied8 + lane]), b.c.k_scale + of, good);
            copy4(smem_addr(&sh.vs[slot][warp * S::kCopied8 + lane]), b.c.v_scale + of, good);
        }
        const uint32_t ks = smem_addr(smem) + slot * 2 * S::kTileBytes8;
#pragma unroll
        for (int i = 0; i < S::kCopied8 * kPieces / 32; ++i) {
            const int x = i * 32 + lane, r = x / kPieces, d = x % kPieces, row = warp * S::kCopied8 + r;
            const int64_t from = __shfl_sync(~0u, at, r), off = from < 0 ? 0 : from + d * 16;
            copy16(ks + place_k(row, d), static_cast<const uint8_t *>(b.c.k) + off, from >= 0);
            copy16(ks + S::kTileBytes8 + place_v(row, d), static_cast<const uint8_t *>(b.c.v) + off, from >= 0);
        }
    };
    static_assert(S::kCopied8 * kPieces % 32 == 0, "whole warps of copies");
    Look next = look();
#pragma unroll
    for (int t = 0; t < S::kStages8 - 1; ++t) {
        const Look now = next;
        next = look();
        if (t < tiles) fetch(t, now);
        copy_commit();
    }
    // q of the two rows: 16 values side by side of each 64, as fp16
    constexpr int kSets = D / 64;
    uint32_t qf[kSets][4][4];  // [64 values][4 of them][fragment register]
    float of_row[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
        const int r = ra + half * 8;
        float v[kSets][16];
        float most = 0.0f;
        const bool whole = (reinterpret_cast<uintptr_t>(a.q) % 16 | (a.q_tok | a.q_head) % 8) == 0;
        const T *from = static_cast<const T *>(a.q) + (sq.row0 + (r0 + (r < rows ? r : 0)) / group) * a.q_tok +
                        (kvh * group + (r0 + (r < rows ? r : 0)) % group) * a.q_head + t4 * 16;
#pragma unroll
        for (int g = 0; g < kSets; ++g) {
            __align__(16) T y[16];
            if (whole) {
                *reinterpret_cast<uint4 *>(y) = *reinterpret_cast<const uint4 *>(from + g * 64);
                *reinterpret_cast<uint4 *>(y + 8) = *reinterpret_cast<const uint4 *>(from + g * 64 + 8);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = from[g * 64 + e];
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                v[g][e] = r < rows ? to_f32(y[e]) : 0.0f;
                most = fmaxf(most, fabsf(v[g][e]));
            }
        }
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
        most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
        const int k = row_exponent(most);
        const float down = two_to(-k);
        of_row[half] = a.scale * kLog2e * two_to(k);
#pragma unroll
        for (int g = 0; g < kSets; ++g)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qf[g][i][half] = pack2<__half>(v[g][i * 4] * down, v[g][i * 4 + 1] * down);
                qf[g][i][half + 2] = pack2<__half>(v[g][i * 4 + 2] * down, v[g][i * 4 + 3] * down);
            }
    }
    constexpr float kLower = 10.0f;
    for (int t = 0; t < tiles; ++t) {
        copy_wait<S::kStages8 - 2>();
        __syncthreads();
        const int slot = t % S::kStages8;
        if (t + S::kStages8 - 1 < tiles) {
            fetch(slot ? slot - 1 : S::kStages8 - 1, next);
            next = look();
        }
        copy_commit();
        const uint8_t *kt = smem + slot * 2 * S::kTileBytes8;
        const uint32_t vt = smem_addr(kt) + S::kTileBytes8;

        float x[S::kKeys8 / 8][4] = {};
#pragma unroll
        for (int j = 0; j < S::kKeys8 / 8; ++j) {
            const int r = wk * S::kKeys8 + j * 8 + lane / 4;
#pragma unroll
            for (int g = 0; g < kSets; ++g) {
                const uint4 w = *reinterpret_cast<const uint4 *>(kt + place_k(r, g * 4 + t4));
                mma<__half>(x[j], qf[g][0], e4m3_f16x2((uint16_t)w.x), e4m3_f16x2((uint16_t)(w.x >> 16)));
                mma<__half>(x[j], qf[g][1], e4m3_f16x2((uint16_t)w.y), e4m3_f16x2((uint16_t)(w.y >> 16)));
                mma<__half>(x[j], qf[g][2], e4m3_f16x2((uint16_t)w.z), e4m3_f16x2((uint16_t)(w.z >> 16)));
                mma<__half>(x[j], qf[g][3], e4m3_f16x2((uint16_t)w.w), e4m3_f16x2((uint16_t)(w.w >> 16)));
            }
        }
        // of this warp's keys, those that there are
        constexpr uint32_t kAll = S::kCopied8 == 32 ? ~0u : (1u << S::kCopied8) - 1;
        uint32_t there = kAll;
#pragma unroll
        for (int w = 0; w < S::kKeys8 / S::kCopied8; ++w) there &= sh.valid[slot][wk * (S::kKeys8 / S::kCopied8) + w];
        float2 vs[S::kKeys8 / 8];
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < S::kKeys8 / 8; ++j) {
            const int key = wk * S::kKeys8 + j * 8 + t4 * 2;
            const float2 ks = *reinterpret_cast<const float2 *>(&sh.ks[slot][key]);
            vs[j] = *reinterpret_cast<const float2 *>(&sh.vs[slot][key]);
            const float lv[2] = {scale_log2(vs[j].x), scale_log2(vs[j].y)};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[j][e] = x[j][e] * of_row[e / 2] * (e % 2 ? ks.y : ks.x);  // (in this order a score of 0 stays 0)
                if (there != kAll && !(sh.valid[slot][key / S::kCopied8] >> ((key + e % 2) % S::kCopied8) & 1)) x[j][e] = -INFINITY;
                top[e / 2] = fmaxf(top[e / 2], x[j][e] + lv[e % 2]);
            }
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            top[half] = fmaxf(top[half], __shfl_xor_sync(~0u, top[half], 1));
            top[half] = fmaxf(top[half], __shfl_xor_sync(~0u, top[half], 2));
            const float now = fmaxf(m[half], top[half] - kLower), shift = now == -INFINITY ? 0.0f : now;
            const float keep = pow2(m[half] - shift);
            const float before = keep > 0.0f ? l[half] * keep : part_sum<true>(l[half], m[half] - shift);
            m[half] = now;
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < S::kKeys8 / 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float w = pow2(x[j][half * 2 + e] - shift);
                    sum += w;
                    x[j][half * 2 + e] = w * (e ? vs[j].y : vs[j].x);
                }
            l[half] = before + sum;
#pragma unroll
            for (int d = 0; d < D / 8; ++d) {
                o[d][half * 2] *= keep;
                o[d][half * 2 + 1] *= keep;
            }
        }
#pragma unroll
        for (int j = 0; j < S::kKeys8 / 16; ++j) {
            const uint32_t p[4] = {pack2<__half>(x[2 * j][0], x[2 * j][1]), pack2<__half>(x[2 * j][2], x[2 * j][3]),
                                   pack2<__half>(x[2 * j + 1][0], x[2 * j + 1][1]), pack2<__half>(x[2 * j + 1][2], x[2 * j + 1][3])};
            const int r = wk * S::kKeys8 + j * 16 + lane % 16;
#pragma unroll
            for (int d = 0; d < kPieces; d += 2) {
                uint32_t y[4];
                ldsm4t(y, vt + place_v(r, d + lane / 16));
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t y0 = __byte_perm(y[2 * h], 0, 0x3120), y1 = __byte_perm(y[2 * h + 1], 0, 0x3120);
                    mma<__half>(o[2 * (d + h)], p, e4m3_f16x2((uint16_t)y0), e4m3_f16x2((uint16_t)y1));
                    mma<__half>(o[2 * (d + h) + 1], p, e4m3_f16x2((uint16_t)(y0 >> 16)), e4m3_f16x2((uint16_t)(y1 >> 16)));
                }
            }
        }
    }
    copy_wait<0>();
}

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
//
// Old: OldPlaces where the first places of a sequence are in 8 bits.  The
// blocks of its first n8 chunks are theirs then (old_places() above), the others
// take the rest as ever, and the parts are joined as if all were of a kind.
template <typename T, int D, int WR, typename Old>
__global__ void __launch_bounds__(128, blocks_an_sm(D))
    k_tree_attention(TreeAttention a, Old b, int chunk, int row_tiles, bool cluster, float *part_o, float2 *part_ml) {
    using S = Shape<D, WR>;
    constexpr bool kOld = std::is_same_v<Old, OldPlaces>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint32_t valid[S::kStages][4];
    __shared__ uint64_t drafts[S::kRows];
    __shared__ float2 ml[S::kParts][S::kRows], joined[S::kRows];
    pdl_wait();
    pdl_trigger();  // (after the wait: the join reads what this call was given before it waits)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kvh = blockIdx.x / row_tiles, r0 = blockIdx.x % row_tiles * S::kRows;
    const bool turned = kOld && !cluster;  // (the old places of all sequences first: their blocks take longer)
    const int c = turned ? blockIdx.z : blockIdx.y, s = turned ? blockIdx.y : blockIdx.z;
    const int group = a.q_heads / a.c.kv_heads;
    const Seq sq = sequence(a, b, s, tid == 0 && blockIdx.x == 0 && c == 0);
    const int rows = min(sq.n * group - r0, S::kRows);
    // blocks of old places that the grid has, and that this sequence needs
    const int n8 = old_blocks(b), parts8 = (sq.old + chunk_of(b) - 1) / chunk_of(b);
    const bool is8 = kOld && c < n8;
    const int parts = parts8 + (sq.len - sq.from + chunk - 1) / chunk;
    const int begin = is8 ? c * chunk_of(b) : sq.from + (c - n8) * chunk;
    const int end = is8 ? min(sq.old, begin + chunk_of(b)) : min(sq.len, begin + chunk);
    // a row that has no keys at all is written by its first block
    if (rows <= 0 || (begin >= end && !(c == n8 && parts == 0))) return;
    const bool alone = parts <= 1;  // the only chunk of this sequence
    float o[D / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    const int wr = warp % WR, wk = warp / WR, ra = wr * 16 + lane / 4;  // this lane's rows are ra and ra + 8
    if constexpr (kOld) {
        __shared__ OldShared<S> old;
        if (is8) old_places<T, D, WR>(a, b, sq, old, smem, begin, end, r0, rows, kvh, s, o, m, l);
    }
    if (!is8) {

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
    }

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
        float *to = res + (wk * S::kRows + r) * D;
        if (kOld && is8) {  // (two fragments have the even and the odd ones of 16 values)
#pragma unroll
            for (int d = 0; d < D / 16; ++d)
                *reinterpret_cast<float4 *>(to + d * 16 + lane % 4 * 4) =
                    make_float4(o[2 * d][half * 2] * f, o[2 * d + 1][half * 2] * f, o[2 * d][half * 2 + 1] * f, o[2 * d + 1][half * 2 + 1] * f);
        } else {
#pragma unroll
            for (int d = 0; d < D / 8; ++d)
                *reinterpret_cast<float2 *>(to + d * 8 + lane % 4 * 2) = make_float2(o[d][half * 2] * f, o[d][half * 2 + 1] * f);
        }
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
            if (top != -INFINITY) sum += part_sum<kOld>(ml[w][r].y, ml[w][r].x - top);
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
    const int mine = is8 ? c : parts8 + c - n8;
    auto rank_of = [&](int o) { return o < parts8 ? o : n8 + o - parts8; };
    cluster_sync();
    for (int i = mine * 128 + tid; i < rows * (D / 4); i += parts * 128) {
        const int r = i / (D / 4), d = i % (D / 4) * 4;
        float2 m_of[kMaxCluster];
        float top = -INFINITY, sum = 0.0f;
#pragma unroll
        for (int o = 0; o < kMaxCluster; ++o) {
            m_of[o] = o < parts ? peer_load2(peer(&joined[r], rank_of(o))) : make_float2(-INFINITY, 0.0f);
            top = fmaxf(top, m_of[o].x);
        }
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int o = 0; o < kMaxCluster; ++o) {
            if (o >= parts) continue;
            const float4 y = peer_load4(peer(res + r * D + d, rank_of(o)));
            const float f = top == -INFINITY ? 0.0f : pow2(m_of[o].x - top);
            if (kOld) sum += top == -INFINITY ? 0.0f : part_sum<true>(m_of[o].y, m_of[o].x - top);
            else sum += m_of[o].y * f;
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
template <typename T, int D, int W, typename Old>
__global__ void __launch_bounds__(256) k_tree_join(TreeAttention a, Old b, int chunk, bool wide, const float *part_o, const float2 *part_ml) {
    constexpr bool kOld = std::is_same_v<Old, OldPlaces>;
    constexpr int kEach = D / 32;  // values of a lane, side by side
    struct alignas(kEach * 4 < 16 ? kEach * 4 : 16) Values {
        float v[kEach];
    };
    __shared__ float tops[W], sums[W];
    __shared__ Values vals[W][W > 1 ? 32 : 1];
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, w = warp % W, h = blockIdx.x * (8 / W) + warp / W, i = blockIdx.y;
    // (the parts' kernel lets this one start when what the two are given is there: only the parts have to be waited for)
    const Seq sq = sequence(a, b, blockIdx.z, false);
    pdl_wait();
    // parts of old places, and the grid's blocks of those that this sequence did without
    const int parts8 = (sq.old + chunk_of(b) - 1) / chunk_of(b), skip = old_blocks(b) - parts8;
    const int recent = ((wide ? sq.ctx : sq.len) - sq.from + chunk - 1) / chunk;
    const int chunks = parts8 + (wide ? max(recent, 1) : recent);
    if (i >= sq.n || h >= a.q_heads || chunks <= 1) return;  // (all warps of a row alike)
    const int64_t row = (sq.row0 + i) * a.q_heads + h, step = a.total_tok * a.q_heads;
    Values v = {};
    float top = -INFINITY, sum = 0.0f;
    for (int c0 = w; c0 < chunks; c0 += 8 * W) {  // eight parts' loads at once
        float2 p[8];
        Values y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = c0 + j * W, at = c < parts8 ? c : c + skip;
            p[j] = make_float2(-INFINITY, 0.0f);
            y[j] = {};
            if (c >= chunks) continue;
            p[j] = part_ml[at * step + row];
            y[j] = reinterpret_cast<const Values *>(part_o + (at * step + row) * D)[lane];
        }
        float now = top;
#pragma unroll
        for (int j = 0; j < 8; ++j) now = fmaxf(now, p[j].x);
        if (now == -INFINITY) continue;
        const float keep = pow2(top - now);
        sum = kOld ? part_sum<true>(sum, top - now) : sum * keep;
#pragma unroll
        for (int e = 0; e < kEach; ++e) v.v[e] *= keep;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = pow2(p[j].x - now);
            sum += kOld ? part_sum<true>(p[j].y, p[j].x - now) : p[j].y * f;
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
                sum += kOld ? part_sum<true>(sums[o], tops[o] - top) : f * sums[o];
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

// The same where max_old places are in 8 bits and max_new behind them.  Blocks
// of either kind run beside one another: the recent places' fill what the old
// places' waves leave free.  A block of old places takes 12 ns a key (the wide
// kernel 10 as ever), and chunks of recent places are no longer to a block.
Plan plan_old(int n_seq, int max_tok, int64_t max_old, int64_t max_new, int q_heads, int kv_heads, int head_dim, int *n8, int *chunk8) {
    Plan p = {};
    const int rows = max_tok * (q_heads / kv_heads);
    p.wide = wide_rows(n_seq, rows, max_old + max_new, kv_heads, head_dim);
    p.wr = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    const int block_rows = p.wide ? kWideRows : 16 * p.wr;
    p.row_tiles = (rows + block_rows - 1) / block_rows;
    const int64_t blocks = (int64_t)n_seq * kv_heads * p.row_tiles, slots = p.wide ? kSms : kSms * blocks_an_sm(head_dim);
    const double old_us = p.wide ? 0.010 : 0.012, new_us = p.wide ? 0.010 : 0.024, rest = p.wide ? 6.0 : 1.6 + 0.17 * std::min(rows, block_rows);
    const double part_us = p.wide ? (double)n_seq * kv_heads * rows * head_dim * 8.0 / 5e6 : 0.0;
    auto cuts = [](int64_t keys, int64_t chunk) { return (keys + chunk - 1) / chunk; };
    auto up64 = [](int64_t keys) { return (keys + 63) / 64 * 64; };
    // several sequences may differ in length: no block takes much longer than others
    const int64_t most = n_seq > 1 && p.wide ? std::max(2048, 32 * rows) : CBQ_TREE_MAX_LEN;
    double least = 0.0;
    int64_t last = -1;
    auto look = [&](int64_t m) {  // old places in m chunks
        const int64_t c8 = max_old == 0 ? 64 : std::max<int64_t>(up64(std::min(cuts(max_old, std::max<int64_t>(m, 1)), most)), up64(cuts(max_old, 16384)));
        const int64_t m8 = cuts(max_old, c8);
        if (m8 == last) return;
        last = m8;
        int64_t c16 = max_old == 0 ? up64(cuts(max_new, std::max<int64_t>(m, 1))) : up64((int64_t)(c8 * old_us / new_us));
        c16 = std::max(std::min(c16, up64(max_new)), up64(cuts(max_new, 16384)));
        const int64_t m16 = cuts(max_new, c16), n = m8 + m16;
        const bool cluster = !p.wide && n > 1 && n <= kMaxCluster && blocks * n <= slots;
        const double t8 = c8 * old_us + rest, t16 = c16 * new_us + rest;
        auto span = [&](int64_t b8, int64_t b16) {
            const int64_t waves = cuts(b8, slots);
            const double idle = (double)(waves * slots - b8) * t8, work = (double)b16 * t16;
            return std::max(waves * t8 + std::max(work - idle, 0.0) / (double)slots, b8 ? t8 : cuts(b16, slots) * t16);
        };
        double t = span(blocks * m8, blocks * m16);
        if (n_seq > 1) t += 0.5 * span((blocks * m8 + 1) / 2, (blocks * m16 + 1) / 2);
        t += n == 1 ? 0.0 : cluster ? 1.5 : p.wide ? 3.0 + part_us * n : 2.5;
        if (p.chunk && t >= least) return;
        least = t, p.chunk = (int)c16, p.n_chunks = (int)n, p.cluster = cluster;
        *n8 = (int)m8, *chunk8 = (int)std::min<int64_t>(c8, CBQ_TREE_MAX_LEN);
    };
    for (int64_t m = 1; m < kMaxCluster; ++m) look(m);
    for (int64_t w = 1; w <= 4; ++w) {
        look((w * slots - blocks) / blocks);
        look(w * slots / blocks);
    }
    return p;
}

// Of the same limits as the last call's (or as the size of the workspace was just asked for with): the same plan.  (It
// takes the host 3 us to find.)
struct OldPlan {
    int n_seq, max_tok, q_heads, kv_heads, head_dim;
    int64_t max_old, max_new;
    Plan plan;
    int n8, chunk8;
};
const OldPlan &plan_old_again(int n_seq, int max_tok, int64_t max_old, int64_t max_new, int q_heads, int kv_heads, int head_dim) {
    static thread_local OldPlan last = {};
    if (last.n_seq != n_seq || last.max_tok != max_tok || last.max_old != max_old || last.max_new != max_new || last.q_heads != q_heads ||
        last.kv_heads != kv_heads || last.head_dim != head_dim) {
        last = OldPlan{n_seq, max_tok, q_heads, kv_heads, head_dim, max_old, max_new, {}, 0, 0};
        last.plan = plan_old(n_seq, max_tok, max_old, max_new, q_heads, kv_heads, head_dim, &last.n8, &last.chunk8);
    }
    return last;
}

// What the parts of the rows take, for the second kernel to join.
size_t parts_room(const Plan &p, int64_t total_tok, int q_heads, int head_dim) {
    if (p.n_chunks == 1 || p.cluster) return 16;
    const size_t rows = (size_t)total_tok * q_heads * p.n_chunks;
    return (rows * sizeof(float2) + 15) / 16 * 16 + rows * head_dim * sizeof(float);
}

bool tiled_dim(int d) { return d == 64 || d == 128 || d == 256; }

template <typename T, int D, int WR, typename Old>
cudaError_t launch_tiled(const TreeAttention &a, const Old &b, const Plan &p, cudaStream_t s) {
    const size_t rows = (size_t)a.total_tok * a.q_heads;
    float2 *part_ml = static_cast<float2 *>(a.ws);
    float *part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(a.ws) + (rows * p.n_chunks * sizeof(float2) + 15) / 16 * 16);
    const unsigned x = (unsigned)(a.c.kv_heads * p.row_tiles);
    const cudaError_t e = p.wide ? launch_tree_wide(a, b, p.chunk, p.n_chunks, p.row_tiles, part_o, part_ml, s)
                                 : launch_clusters(k_tree_attention<T, D, WR, Old>,
                                                   std::is_same_v<Old, OldPlaces> && !p.cluster ? dim3(x, (unsigned)a.n_seq, (unsigned)p.n_chunks)
                                                                                                : dim3(x, (unsigned)p.n_chunks, (unsigned)a.n_seq),
                                                   p.cluster ? p.n_chunks : 1, 128, Shape<D, WR>::kSmem, s, a, b, p.chunk, p.row_tiles,
                                                   p.cluster, part_o, part_ml);
    if (e != cudaSuccess || p.n_chunks == 1 || p.cluster) return e;
    // (before its loads went together: a warp for each of 1,024 rows of 19 chunks 21.3 us a call, eight warps 20.4; of
    // 2,048 rows 28.0 and 30.2; a ragged batch of 5,000 rows of up to 12 chunks 62 and 65)
    const unsigned heads = (unsigned)a.q_heads, toks = (unsigned)a.max_tok, seqs = (unsigned)a.n_seq;
    return p.n_chunks > 8 && rows < 2048 ? launch_dependent(k_tree_join<T, D, 8, Old>, dim3(heads, toks, seqs), 256, 0, s, a, b, p.chunk, p.wide, part_o, part_ml)
                          : launch_dependent(k_tree_join<T, D, 1, Old>, dim3((heads + 7) / 8, toks, seqs), 256, 0, s, a, b, p.chunk,
                                             p.wide, part_o, part_ml);
}

template <typename T, int D, typename Old>
cudaError_t launch_dim(const TreeAttention &a, const Old &b, const Plan &p, cudaStream_t s) {
    return p.wr == 1 ? launch_tiled<T, D, 1>(a, b, p, s) : p.wr == 2 ? launch_tiled<T, D, 2>(a, b, p, s) : launch_tiled<T, D, 4>(a, b, p, s);
}

template <typename T, typename Old>
cudaError_t launch_planned(const TreeAttention &a, const Old &b, const Plan &p, cudaStream_t s) {
    if (a.c.head_dim == 64) return launch_dim<T, 64>(a, b, p, s);
    if (a.c.head_dim == 128) return launch_dim<T, 128>(a, b, p, s);
    return launch_dim<T, 256>(a, b, p, s);
}

template <typename T, typename Old>
cudaError_t launch_general(const TreeAttention &a, const Old &b, cudaStream_t s) {
    return launch_dependent(k_tree_general<T, Old>, dim3((unsigned)a.q_heads, (unsigned)a.max_tok, (unsigned)a.n_seq), 32, 0, s, a, b);
}

// 16-byte copies want every row of k and v on a 16-byte boundary, 16-byte stores every row of out.
bool whole_rows(const TreeAttention &a) {
    const uintptr_t ends = reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v) | reinterpret_cast<uintptr_t>(a.out);
    return tiled_dim(a.c.head_dim) && ends % 16 == 0 && (a.c.page_stride | a.c.tok_stride | a.c.head_stride) % 8 == 0;
}

template <typename T>
cudaError_t launch_type(const TreeAttention &a, cudaStream_t s) {
    if (!whole_rows(a)) return launch_general<T>(a, NoOldPlaces{}, s);
    return launch_planned<T>(a, NoOldPlaces{}, plan(a.n_seq, a.max_tok, a.max_len, a.q_heads, a.c.kv_heads, a.c.head_dim), s);
}

template <typename T>
cudaError_t launch_type(const TreeAttention &a, OldPlaces b, cudaStream_t s) {
    const uintptr_t ends = reinterpret_cast<uintptr_t>(b.c.k) | reinterpret_cast<uintptr_t>(b.c.v);
    if (!whole_rows(a) || ends % 16 != 0 || (b.c.page_stride | b.c.tok_stride | b.c.head_stride) % 16 != 0) return launch_general<T>(a, b, s);
    const OldPlan &p = plan_old_again(a.n_seq, a.max_tok, b.max_old, b.max_new, a.q_heads, a.c.kv_heads, a.c.head_dim);
    b.n8 = p.n8;
    b.chunk8 = p.chunk8;
    return launch_planned<T>(a, b, p.plan, s);
}

}  // namespace

size_t tree_attention_workspace(int n_seq, int64_t total_tok, int max_tok, int64_t max_len, int q_heads, int kv_heads,
                                int head_dim) {
    if (!tiled_dim(head_dim)) return 16;
    return parts_room(plan(n_seq, max_tok, max_len, q_heads, kv_heads, head_dim), total_tok, q_heads, head_dim);
}

size_t tree_attention8_workspace(int n_seq, int64_t total_tok, int max_tok, int64_t max_old, int64_t max_new, int q_heads,
                                 int kv_heads, int head_dim) {
    if (!tiled_dim(head_dim)) return 16;
    return parts_room(plan_old_again(n_seq, max_tok, max_old, max_new, q_heads, kv_heads, head_dim).plan, total_tok, q_heads, head_dim);
}

cudaError_t launch_tree_attention(const TreeAttention &a, cudaStream_t s) {
    return a.c.dtype == CBQ_BF16 ? launch_type<__nv_bfloat16>(a, s) : launch_type<__half>(a, s);
}

cudaError_t launch_tree_attention8(const TreeAttention &a, const OldPlaces &b, cudaStream_t s) {
    return a.c.dtype == CBQ_BF16 ? launch_type<__nv_bfloat16>(a, b, s) : launch_type<__half>(a, b, s);
}

}  // namespace cbq
