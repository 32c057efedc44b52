// cbq_attn_wide.cu -- the tree attention's committed keys for many rows: more
// than 64 rows a kv head are bound by the matrix products, which run here on
// the 5th-generation tensor cores (tcgen05) with scores, weights and results
// in tensor memory.
//
// A block takes 256 rows of one kv head as two groups of 128 (or, where there
// are no more than 128, the even and the odd key tiles for the same rows) and
// streams K and V by.  An item is one key tile for one group; the groups take
// turns, so that one's products run while the other's weights are computed:
//   S = Q K^T (128 x 64, shared memory x shared memory), into tensor memory;
//   P = 2^(scale S - m), by the group's 128 threads, a row each, back into
//       tensor memory as 16-bit numbers;
//   O += P V (128 x D, tensor memory x shared memory).
// O is scaled down only when a row's maximum has grown by 2^8 (fp16: 2^5):
// until then the weights are just larger, and the last division takes it out.
// Roles: warps 0..3 and 4..7 the two groups, 8 and 9 the copies, 10 and 11 the
// products of a group each (waiting, issuing and committing takes a warp longer
// than the products themselves: one warp for both groups was the bound).
// Tiles lie in shared memory as 8 x 16-byte core matrices (row / 8, column /
// 16 bytes): eight rows' 16 bytes are 128 bytes in a row, so the copies of
// eight keys fill them without bank conflicts, and the same tile serves as K
// (columns are the summed axis) and as V (rows are).
#include "cbq_pipe.cuh"
#include "step/cbq_attn.cuh"

namespace cbq {

namespace {

constexpr int kGroup = 128;                   // rows of a group
constexpr int kTile = 64;                     // keys of a tile
constexpr int kStages = 5;
constexpr int kCopyWarp = 8, kMmaWarp = 10, kWideThreads = 12 * 32;  // (more warps would leave 128 registers a thread)
constexpr int kTmemCols = 512;

// Columns of tensor memory: scores, weights, results of a group.
template <int D>
struct Cols {
    static constexpr uint32_t s(int g) { return g * kTile; }
    static constexpr uint32_t p(int g) { return 2 * kTile + g * (kTile / 2); }
    static constexpr uint32_t o(int g) { return 3 * kTile + g * D; }
    static_assert(o(2) <= kTmemCols, "the tensor memory holds both groups");
};

struct WideShared {
    uint64_t full[kStages], empty[kStages];   // a tile's copies have landed; its products are done
    uint64_t scored[2], taken[2], weighed[2], summed[2];  // of a group's item: S is there, S is read, P is there, O has it
    uint64_t done[2];
    uint32_t valid[kStages][2];               // keys of a tile that exist, 32 a copying warp
    uint32_t tmem_slot;
    int abort;
    float2 ml[kGroup];
};

// Descriptor of a tile in shared memory: 16-byte units; `lead` between core
// matrices along the summed axis for rows-are-outputs operands.
__device__ __forceinline__ uint64_t tile_desc(uint32_t at, uint32_t lead, uint32_t stride) {
    return (uint64_t)((at >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((stride >> 4) & 0x3FFFu) << 32) | (1ull << 46);
}

// Instruction descriptor: fp32 sums, 16-bit operands of T, 128 x N, the second
// operand's rows along the summed axis if kRows.
template <typename T, int N, bool kRows>
constexpr uint32_t wide_idesc() {
    constexpr uint32_t f = std::is_same_v<T, __nv_bfloat16> ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | (kRows ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kGroup >> 4) << 24);
}

// The products are issued by one elected lane of a warp that stays together:
// its operands are then uniform registers as the instruction wants them (in a
// branch of one lane each had to be moved there: 100 clocks a product).
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"((int)add) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n .reg .pred p, e;\n setp.ne.b32 p, %4, 0;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"((int)add) : "memory");
}
// Arrives on the barrier once every product the elected lane issued so far is done.
__device__ __forceinline__ void commit(uint64_t &bar) {
    asm volatile(
        "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
        " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_addr(&bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

#define CBQ_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define CBQ_I8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
// 32 columns of this thread's lane; there once tm_wait_ld() returns.
__device__ __forceinline__ void tm_ld(uint32_t at, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,"
        "%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : CBQ_R8(v, 0), CBQ_R8(v, 8), CBQ_R8(v, 16), CBQ_R8(v, 24) : "r"(at) : "memory");
}
__device__ __forceinline__ void tm_st(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,"
        "%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::CBQ_I8(v, 0), CBQ_I8(v, 8), CBQ_I8(v, 16), CBQ_I8(v, 24), "r"(at) : "memory");
}
#undef CBQ_R8
#undef CBQ_I8
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The eight warps of the two groups.
__device__ __forceinline__ void groups_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// A place in the ring and how often it has come round (parities by its low bit).
struct Place {
    int slot = 0, round = 0;
    __device__ __forceinline__ void step(int by) {
        slot += by;
        if (slot >= kStages) slot -= kStages, ++round;
    }
};

// A wait of at most a second; then the call's error word says so and every
// role of the block leaves its loop.
__device__ __forceinline__ bool wait_for(WideShared &s, uint64_t &bar, uint32_t parity, unsigned *err) {
    const uint32_t b = smem_addr(&bar);
    if (mbar_try_wait(b, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
        if (*(volatile int *)&s.abort) return false;
        if (mbar_try_wait(b, parity)) return true;
        if (global_ns() - t0 > kWaitLimitNs) break;
    }
    if (err) atomicOr(err, kErrPipeTimeout);
    *(volatile int *)&s.abort = 1;
    return false;
}

// The same by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(WideShared &s, uint64_t &bar, uint32_t parity, unsigned *err) {
    return __all_sync(~0u, wait_for(s, bar, parity, err));
}

template <typename T, int D>
__global__ void __launch_bounds__(kWideThreads, 1)
    k_tree_wide(const __grid_constant__ TreeAttention a, int chunk, int n_chunks, int row_tiles, float *part_o, float2 *part_ml) {
    constexpr uint32_t kCol = 128, kRow = D / 8 * 128;       // bytes between core matrices along a row, and to the next eight rows
    constexpr int kQBytes = kGroup * D * 2, kTileBytes = kTile * D * 2;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ WideShared sh;
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kvh = blockIdx.x / row_tiles, r0 = blockIdx.x % row_tiles * kWideRows, c = blockIdx.y, s = blockIdx.z;
    const int group = a.q_heads / a.c.kv_heads;
    const Seq sq = sequence(a, s, false);  // (the drafts' kernel has reported)
    const int rows = min(sq.n * group - r0, kWideRows);
    const int begin = c * chunk, end = min(sq.ctx, begin + chunk);
    if (rows <= 0 || (begin >= end && n_chunks > 1)) {
        pdl_wait();  // what follows this kernel counts on the drafts' kernel being done
        return;
    }
    const bool split = rows <= kGroup;  // the groups share out the key tiles
    const int tiles = max(0, (end - begin + kTile - 1) / kTile), items = split ? tiles : 2 * tiles;
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem_slot)), "n"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 64 + 2);  // the copying threads' copies, and their warps' word on valid[]
            mbar_init(smem_addr(&sh.empty[i]), split ? 1 : 2);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(smem_addr(&sh.scored[g]), 1);
            mbar_init(smem_addr(&sh.taken[g]), 4);
            mbar_init(smem_addr(&sh.weighed[g]), 4);
            mbar_init(smem_addr(&sh.summed[g]), 1);
        }
        mbar_init(smem_addr(&sh.done[0]), 1);
        mbar_init(smem_addr(&sh.done[1]), 1);
        sh.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    // q of the rows, the sign of the scale with it; absent rows are zero
    const float sc = fabsf(a.scale) * kLog2e;
    const bool q_whole = (reinterpret_cast<uintptr_t>(a.q) % 16 | (a.q_tok | a.q_head) % 8) == 0;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
    for (int i = tid; i < (split ? 1 : 2) * kGroup * (D / 8); i += kWideThreads) {
        const int r = i / (D / 8), d = i % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows) {
            const int tok = (r0 + r) / group, h = kvh * group + (r0 + r) % group;
            const T *from = static_cast<const T *>(a.q) + (sq.row0 + tok) * a.q_tok + h * a.q_head + d * 8;
            if (q_whole) {
                v = *reinterpret_cast<const uint4 *>(from);
            } else {
                __align__(16) T y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = from[e];
                v = *reinterpret_cast<const uint4 *>(y);
            }
        }
        v.x ^= flip, v.y ^= flip, v.z ^= flip, v.w ^= flip;
        *reinterpret_cast<uint4 *>(smem + r / 8 * kRow + d * kCol + r % 8 * 16) = v;
    }
    proxy_fence();
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem_slot;
    const uint32_t q_at = smem_addr(smem), ring = q_at + 2 * kQBytes;

    if (warp >= kCopyWarp && warp < kMmaWarp) {
        // copies: a warp brings 32 keys of each tile; lane l keeps the place of key l
        const int cw = warp - kCopyWarp;
        const int32_t *table = a.table + (int64_t)s * a.table_width;
        const int64_t head = kvh * a.c.head_stride;
        auto page_of = [&](int t) {
            const int p = begin + t * kTile + cw * 32 + lane;
            return t < tiles && p < end ? table[(uint32_t)p / (uint32_t)a.c.page_size] : -1;
        };
        Place put;
        // lane l copies 16 bytes of key l % 8 of every eight, at columns l / 8, l / 8 + 4, ..: whole sectors are read
        const char *from0 = static_cast<const char *>(a.c.k) + lane / 8 * 16;
        const int64_t to_v = static_cast<const char *>(a.c.v) - static_cast<const char *>(a.c.k);
        const uint32_t to0 = ring + cw * 4 * kRow + lane / 8 * kCol + lane % 8 * 16;
        int page = page_of(0);
        for (int t = 0; t < tiles; ++t, put.step(1)) {
            if (t >= kStages && !warp_wait(sh, sh.empty[put.slot], (put.round - 1) & 1, a.err)) break;
            const uint32_t p = begin + t * kTile + cw * 32 + lane;
            const bool in = p < (uint32_t)end, good = in && page >= 0 && page < a.c.n_pages;
            if (in && !good && a.err) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
            const int64_t at = good ? (page * a.c.page_stride + (int64_t)(p % (uint32_t)a.c.page_size) * a.c.tok_stride + head) * 2 : -1;
            const uint32_t bits = __ballot_sync(~0u, good);
            page = page_of(t + 1);
            const uint32_t to = to0 + put.slot * 2 * kTileBytes;
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const int64_t off = __shfl_sync(~0u, at, h * 8 + lane % 8);
                const char *from = from0 + max(off, (int64_t)0);
#pragma unroll
                for (int d = 0; d < D / 32; ++d) {
                    copy16(to + h * kRow + d * 4 * kCol, from + d * 64, off >= 0);
                    copy16(to + kTileBytes + h * kRow + d * 4 * kCol, from + to_v + d * 64, off >= 0);
                }
            }
            // arrives when this thread's copies have landed.  (Their writes are handed to the tensor cores by the fence of
            // the warp that issues the products; a fence here would wait for every copy under way.)
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&sh.full[put.slot])) : "memory");
            if (lane == 0) {
                sh.valid[put.slot][cw] = bits;
                mbar_arrive(smem_addr(&sh.full[put.slot]));
            }
        }
        copy_commit();
        copy_wait<0>();
    } else if (warp >= kMmaWarp) {
        const int g = warp - kMmaWarp, by = split ? 2 : 1, last = (items - g + 1) / 2;  // items of this group
        const uint32_t at = q_at + (split ? 0 : g) * kQBytes, s_at = tmem + Cols<D>::s(g), p_at = tmem + Cols<D>::p(g);
        Place k, v;  // of the tiles of the next scores and of the next sums
        if (split && g) k.step(1), v.step(1);
        auto score = [&]() {  // the next S
            if (!warp_wait(sh, sh.full[k.slot], k.round & 1, a.err)) return false;
            proxy_fence();
            fence_after();
            const uint32_t k_at = ring + k.slot * 2 * kTileBytes;
#pragma unroll
            for (int j = 0; j < D / 16; ++j)
                mma_ss(s_at, tile_desc(at + j * 2 * kCol, kCol, kRow), tile_desc(k_at + j * 2 * kCol, kCol, kRow),
                       wide_idesc<T, kTile, false>(), j > 0);
            commit(sh.scored[g]);
            k.step(by);
            return true;
        };
        bool ok = last == 0 || score();
        for (int n = 0; n < last && ok; ++n) {
            // the group's next scores as soon as these have been read: they are there when its weights are done
            ok = n + 1 >= last || (warp_wait(sh, sh.taken[g], n & 1, a.err) && score());
            ok = ok && warp_wait(sh, sh.weighed[g], n & 1, a.err);
            if (!ok) break;
            fence_after();
            const uint32_t v_at = ring + (v.slot * 2 + 1) * kTileBytes;
#pragma unroll
            for (int j = 0; j < kTile / 16; ++j)
                mma_ts(tmem + Cols<D>::o(g), p_at + j * 8, tile_desc(v_at + j * 2 * kRow, kRow, kCol), wide_idesc<T, D, true>(), n > 0 || j > 0);
            commit(sh.summed[g]);
            commit(sh.empty[v.slot]);
            v.step(by);
        }
        // every product is done before the tensor memory is freed
        commit(sh.done[g]);
        const uint64_t t0 = global_ns();
        while (!mbar_try_wait(smem_addr(&sh.done[g]), 0u) && global_ns() - t0 < kWaitLimitNs) {}
    } else {
        // weights: thread = row of its group
        const int g = warp / 4, r = warp % 4 * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);
        constexpr float kLower = std::is_same_v<T, __half> ? 10.0f : 0.0f, kGrow = std::is_same_v<T, __half> ? 5.0f : 8.0f;
        float m = -INFINITY, l = 0.0f;  // weights are 2^(x - m): m is the maximum less kLower, or up to kGrow below that
        bool ok = true;
        int n = 0;  // items of this group so far
        Place at;
        if (split && g) at.step(1);
        for (int i = g; i < items; i += 2, ++n, at.step(split ? 2 : 1)) {
            const int slot = at.slot;
            ok = warp_wait(sh, sh.scored[g], n & 1, a.err);
            if (!ok) break;
            fence_after();
            uint32_t x[2][32];
            tm_ld(lanes + Cols<D>::s(g), x[0]);
            tm_ld(lanes + Cols<D>::s(g) + 32, x[1]);
            // which keys there are (for the copies' writes to be seen, the wait is theirs too)
            ok = warp_wait(sh, sh.full[slot], at.round & 1, a.err);
            const uint32_t there[2] = {sh.valid[slot][0], sh.valid[slot][1]};
            tm_wait_ld();
            if (!ok) break;
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.taken[g]));
            if ((there[0] & there[1]) != ~0u) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!(there[h] >> j & 1)) x[h][j] = __float_as_uint(-INFINITY);
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 64; ++j) top[j & 3] = fmaxf(top[j & 3], __uint_as_float(x[j >> 5][j & 31]));
            const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sc - kLower;
            const bool grown = now > m + kGrow || (m == -INFINITY && now > -INFINITY);
            const float keep = grown ? pow2(m - now) : 1.0f;
            if (grown) m = now, l *= keep;
            if (n > 0) {
                // the products with the weights before are done: O may be scaled, and P written
                ok = warp_wait(sh, sh.summed[g], (n - 1) & 1, a.err);
                if (!ok) break;
                fence_after();
                if (__any_sync(~0u, grown)) {
#pragma unroll
                    for (int d = 0; d < D; d += 32) {
                        uint32_t o[32];
                        tm_ld(lanes + Cols<D>::o(g) + d, o);
                        tm_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                        tm_st(lanes + Cols<D>::o(g) + d, o);
                    }
                }
            }
            const float less = m == -INFINITY ? 0.0f : -m;
            float sum[4] = {};
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float w0 = pow2(__fmaf_rn(__uint_as_float(x[j >> 4][2 * j & 31]), sc, less));
                const float w1 = pow2(__fmaf_rn(__uint_as_float(x[j >> 4][2 * j + 1 & 31]), sc, less));
                sum[j & 1] += w0;
                sum[2 + (j & 1)] += w1;
                p[j] = pack2<T>(w0, w1);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tm_st(lanes + Cols<D>::p(g), p);
            tm_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.weighed[g]));
        }
        if (ok && n > 0) ok = warp_wait(sh, sh.summed[g], (n - 1) & 1, a.err);
        fence_after();
        // Where the groups shared out the keys, group 1's part goes to group 0 through the ring.
        float *pass = reinterpret_cast<float *>(smem + 2 * kQBytes) + r * (D + 4);
        groups_sync();  // all products of both are done: the ring is free
        if (split && g == 1) {
            sh.ml[r] = make_float2(m, l);
#pragma unroll
            for (int d = 0; d < D; d += 32) {
                uint32_t o[32];
                tm_ld(lanes + Cols<D>::o(1) + d, o);
                tm_wait_ld();
#pragma unroll
                for (int j = 0; j < 32; j += 4)
                    *reinterpret_cast<uint4 *>(pass + d + j) = make_uint4(o[j], o[j + 1], o[j + 2], o[j + 3]);
            }
        }
        groups_sync();
        const int row_in = (split ? 0 : g * kGroup) + r;
        if (!(split && g == 1)) {
            const bool live = row_in < rows;
            const int64_t row = live ? (sq.row0 + (r0 + row_in) / group) * a.q_heads + kvh * group + (r0 + row_in) % group : 0;
            const int64_t step = a.total_tok * a.q_heads;
            // up to three parts of the row: this group's, the other group's, and the drafts' where this is the only chunk
            float2 other = make_float2(-INFINITY, 0.0f), draft = make_float2(-INFINITY, 0.0f);
            if (split && items > 1) other = sh.ml[r];
            pdl_wait();
            const bool last = n_chunks == 1;
            if (last && live) draft = part_ml[step + row];
            const float top = fmaxf(fmaxf(m, other.x), draft.x);
            const float f0 = n == 0 || top == -INFINITY ? 0.0f : pow2(m - top);
            const float f1 = top == -INFINITY ? 0.0f : pow2(other.x - top), f2 = top == -INFINITY ? 0.0f : pow2(draft.x - top);
            const float sum = l * f0 + other.y * f1 + draft.y * f2;
            const float inv = !last ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int d = 0; d < D; d += 32) {
                uint32_t o[32];
                tm_ld(lanes + Cols<D>::o(g) + d, o);
                tm_wait_ld();
                if (live && ok) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float v[4];
                    const float4 y = split && items > 1 ? *reinterpret_cast<const float4 *>(pass + d + j) : make_float4(0, 0, 0, 0);
                    const float4 z = last ? *reinterpret_cast<const float4 *>(part_o + (step + row) * D + d + j) : make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float ye = e == 0 ? y.x : e == 1 ? y.y : e == 2 ? y.z : y.w, ze = e == 0 ? z.x : e == 1 ? z.y : e == 2 ? z.z : z.w;
                        // (what was never written may hold anything: it is not multiplied)
                        const float own = n == 0 ? 0.0f : __uint_as_float(o[j + e]) * f0;
                        v[e] = (own + ye * f1 + ze * f2) * inv;
                    }
                    if (!last) {
                        *reinterpret_cast<float4 *>(part_o + (c * step + row) * D + d + j) = make_float4(v[0], v[1], v[2], v[3]);
                    } else if (a.out_f32) {
                        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + row * D + d + j) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
                        *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + row * D + d + j) = make_uint2(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]));
                    }
                }
                }
                __syncwarp();
            }
            if (live && ok) {
                if (!last) part_ml[c * step + row] = make_float2(top, sum);
                else if (a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
}

template <typename T, int D>
cudaError_t launch_wide(const TreeAttention &a, int chunk, int n_chunks, int row_tiles, float *part_o, float2 *part_ml, cudaStream_t s) {
    constexpr size_t kSmem = 2 * kGroup * D * 2 + kStages * 2 * kTile * D * 2;
    static_assert(kGroup * (D + 4) * 4 <= kStages * 2 * kTile * D * 2, "group 1's part fits the ring");
    return launch_dependent(k_tree_wide<T, D>, dim3((unsigned)(a.c.kv_heads * row_tiles), (unsigned)n_chunks, (unsigned)a.n_seq),
                            kWideThreads, kSmem, s, a, chunk, n_chunks, row_tiles, part_o, part_ml);
}

}  // namespace

cudaError_t launch_tree_wide(const TreeAttention &a, int chunk, int n_chunks, int row_tiles, float *part_o, float2 *part_ml, cudaStream_t s) {
    if (a.c.dtype == CBQ_BF16)
        return a.c.head_dim == 64 ? launch_wide<__nv_bfloat16, 64>(a, chunk, n_chunks, row_tiles, part_o, part_ml, s)
                                  : launch_wide<__nv_bfloat16, 128>(a, chunk, n_chunks, row_tiles, part_o, part_ml, s);
    return a.c.head_dim == 64 ? launch_wide<__half, 64>(a, chunk, n_chunks, row_tiles, part_o, part_ml, s)
                              : launch_wide<__half, 128>(a, chunk, n_chunks, row_tiles, part_o, part_ml, s);
}

}  // namespace cbq
