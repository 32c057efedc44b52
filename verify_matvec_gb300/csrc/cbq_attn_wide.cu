// cbq_attn_wide.cu -- the tree attention for many rows: from some 33 a kv head
// on the products count beside the copies, and with a few hundred they are the
// bound.  They run here on the 5th-generation tensor cores (tcgen05) with scores,
// weights and results in tensor memory.
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
// The drafts are a tile of their own, the last of a sequence: a row's weights
// follow its mask there, and a value row with NaN or infinities, which some
// rows may not see (0 * v would be NaN), is zeroed in shared memory by the
// copying warp and added by hand to the rows that see it.
// Roles: warps 0..3 and 4..7 the two groups, 8 and 9 the copies, 10 the scores'
// products and 11 the sums' (waiting, issuing and committing takes a warp as
// long as the products themselves: one warp for both was the bound).
// Tiles lie in shared memory in halves of 64 columns, 128 bytes a row, the 16-
// byte pieces of a row permuted by the row (128-byte swizzle): a copy takes
// whole 128-byte lines of four keys and meets no bank conflict, and the same
// tile serves as K (columns are the summed axis) and as V (rows are).  (With
// eight keys' 64 bytes a copy, as unpermuted core matrices want them, the
// copies were the bound: 2,100 clocks a tile for 1,700.)
//
// 8 sequences of 64 drafts x 8 heads a kv head over 16,000 keys (270 GFLOP, 543
// MB) take 254 us, 1,060 TFLOP/s, in 128 blocks on 152 SMs.  An item takes its
// SM 1,020 clocks, of which the products take 594 (S 8 x 46, both operands from
// shared memory; O 4 x 57).  24 ragged sequences of 78 rows and 64 a head (149
// MB) take 60 us: some 5 us a block beside its keys, an uneven last wave, and
// 1,120 of 1,440 blocks without keys that take their turn on an SM all the same.
#include "cbq_pipe.cuh"
#include "step/cbq_attn.cuh"

namespace cbq {

namespace {

constexpr int kGroup = 128;                   // rows of a group
constexpr int kTile = 64;                     // keys of a tile
constexpr int kStages = 5;
constexpr int kCopyWarp = 8, kScoreWarp = 10, kSumWarp = 11, kWideThreads = 12 * 32;  // (more warps would leave 128 registers a thread)
constexpr int kTmemCols = 512;

// Columns of tensor memory: a group's scores, two items' (the weights of an
// item take the place of its scores), and its results.
template <int D>
struct Cols {
    static constexpr uint32_t s(int g, int b) { return (2 * g + b) * kTile; }
    static constexpr uint32_t o(int g) { return 4 * kTile + g * D; }
    static_assert(o(2) <= kTmemCols, "the tensor memory holds both groups");
};

struct WideShared {
    uint64_t full[kStages], empty[kStages];   // a tile's copies have landed; its products are done
    // of a group's item: S is there; P is there; O has it.  Even and odd items apart: scores run two items ahead, so one
    // warp of a group may be at the next item while another is still at this one.
    uint64_t scored[2][2], weighed[2][2], summed[2][2];
    uint64_t done[2];
    uint32_t valid[kStages][2];               // keys of a tile that exist
    uint32_t odd[2];                          // drafts whose values are not all finite
    uint32_t tmem_slot;
    int abort;
    float2 ml[kGroup];
};

// Descriptor of a tile in shared memory with 128-byte rows, swizzled: eight
// rows are 1024 bytes; `lead` bytes to the next 64 columns where rows are the
// summed axis.
__device__ __forceinline__ uint64_t tile_desc(uint32_t at, uint32_t lead) {
    return (uint64_t)((at >> 4) & 0x3FFFu) | ((uint64_t)((lead >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
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
// One column, there on return.
__device__ __forceinline__ uint32_t tm_ld1(uint32_t at) {
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n tcgen05.wait::ld.sync.aligned;" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void tm_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
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
    k_tree_wide(const __grid_constant__ TreeAttention a, int chunk, int row_tiles, float *part_o, float2 *part_ml) {
    constexpr uint32_t kQHalf = kGroup * 128, kHalf = kTile * 128;  // bytes of 64 columns
    constexpr int kQBytes = kGroup * D * 2, kTileBytes = kTile * D * 2;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ WideShared sh;
    pdl_wait();
    pdl_trigger();  // (after the wait: the join reads what this call was given before it waits)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int kvh = blockIdx.x / row_tiles, r0 = blockIdx.x % row_tiles * kWideRows, c = blockIdx.y, s = blockIdx.z;
    const int group = a.q_heads / a.c.kv_heads;
    const Seq sq = sequence(a, s, threadIdx.x == 0 && blockIdx.x == 0 && c == 0);
    const int rows = min(sq.n * group - r0, kWideRows);
    const int begin = c * chunk, end = min(sq.ctx, begin + chunk);
    if (rows <= 0 || (begin >= end && c > 0)) return;
    const bool last = end == sq.ctx, alone = last && c == 0;  // with the drafts; the only chunk
    const bool split = rows <= kGroup;  // the groups share out the key tiles
    const int old_tiles = (end - begin + kTile - 1) / kTile, tiles = old_tiles + (last ? 1 : 0);
    const int items = split ? tiles : 2 * tiles;
    if (warp == kScoreWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem_slot)), "n"(kTmemCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(smem_addr(&sh.full[i]), 32 + 1);  // the copying warp's copies, and its word on valid[]
            mbar_init(smem_addr(&sh.empty[i]), 1);
        }
        for (int g = 0; g < 2; ++g) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(smem_addr(&sh.scored[g][b]), 2);  // the products, and the word of their warp, which has seen the tile's valid[]
                mbar_init(smem_addr(&sh.weighed[g][b]), 4);
                mbar_init(smem_addr(&sh.summed[g][b]), 1);
            }
        }
        mbar_init(smem_addr(&sh.done[0]), 1);
        mbar_init(smem_addr(&sh.done[1]), 1);
        sh.abort = 0;
        sh.odd[0] = sh.odd[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const float sc = fmaxf(fabsf(a.scale) * kLog2e, 1e-45f);  // (not zero: -inf times that would be NaN)
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sh.tmem_slot;
    const uint32_t q_at = smem_addr(smem), ring = q_at + 2 * kQBytes;
    const int32_t *table = a.table + (int64_t)s * a.table_width;

    const bool copies = warp >= kCopyWarp && warp < kScoreWarp;
    if (!copies) {
        // q of the rows, the sign of the scale with it; absent rows are zero
        const bool q_whole = (reinterpret_cast<uintptr_t>(a.q) % 16 | (a.q_tok | a.q_head) % 8) == 0;
        const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
        // (all loads under way at once: a second round would wait behind the copies of five tiles, some 3 us)
        constexpr int kOthers = kWideThreads - 64, kAtOnce = (2 * kGroup * (D / 8) + kOthers - 1) / kOthers;
        const int me = warp < kCopyWarp ? tid : tid - 64, pieces = (split ? 1 : 2) * kGroup * (D / 8);
        uint4 v[kAtOnce];
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const int r = (me + x * kOthers) / (D / 8), d = (me + x * kOthers) % (D / 8);
            v[x] = make_uint4(0, 0, 0, 0);
            if (r >= rows) continue;
            const T *from = static_cast<const T *>(a.q) + (sq.row0 + (r0 + r) / group) * a.q_tok + (kvh * group + (r0 + r) % group) * a.q_head + d * 8;
            if (q_whole) {
                v[x] = *reinterpret_cast<const uint4 *>(from);
            } else {
                __align__(16) T y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = from[e];
                v[x] = *reinterpret_cast<const uint4 *>(y);
            }
        }
#pragma unroll
        for (int x = 0; x < kAtOnce; ++x) {
            const int i = me + x * kOthers, r = i / (D / 8), d = i % (D / 8);
            if (i >= pieces) break;
            *reinterpret_cast<uint4 *>(smem + r / kGroup * kQBytes + d / 8 * kQHalf + r % kGroup * 128 + ((d ^ r) & 7) * 16) =
                make_uint4(v[x].x ^ flip, v[x].y ^ flip, v[x].z ^ flip, v[x].w ^ flip);
        }
        proxy_fence();
        asm volatile("bar.sync 2, %0;" ::"n"(kOthers) : "memory");
    }

    if (copies) {
        // copies: the two warps take tiles in turn (what a tile costs a warp is mostly waits and look-ups); lane l keeps
        // the places of keys l and l + 32
        const int cw = warp - kCopyWarp;
        const int64_t head = kvh * a.c.head_stride;
        // Keys are looked up in order: the page of the next tile's key is some pages and tokens on (no divisions).
        const uint32_t size = a.c.page_size, pages_on = 2 * kTile / size, tokens_on = 2 * kTile % size;
        uint32_t entry[2], token[2];  // of this lane's keys of the tile looked up next
        int p = begin + cw * kTile + lane;
#pragma unroll
        for (int e = 0; e < 2; ++e) entry[e] = (uint32_t)(p + 32 * e) / size, token[e] = (uint32_t)(p + 32 * e) % size;
        struct Look {
            int page[2], within[2];  // the id of a key's page, and the token within (-1 where there is no such key)
        };
        auto look = [&](int t) {
            Look l;
            if (t == old_tiles) {  // the drafts begin anywhere
                p = sq.ctx + lane;
#pragma unroll
                for (int e = 0; e < 2; ++e) entry[e] = (uint32_t)(p + 32 * e) / size, token[e] = (uint32_t)(p + 32 * e) % size;
            }
            const int stop = t >= tiles ? 0 : t < old_tiles ? end : sq.len;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const bool key = p + 32 * e < stop;
                l.page[e] = key ? table[entry[e]] : -1;
                l.within[e] = key ? (int)token[e] : -1;
                entry[e] += pages_on;
                token[e] += tokens_on;
                if (token[e] >= size) token[e] -= size, ++entry[e];
            }
            p += 2 * kTile;
            return l;
        };
        Place put;
        if (cw) put.step(1);
        // lane l copies piece l % 8 of the 128 bytes of keys l / 8, l / 8 + 4, ..
        const char *from0 = static_cast<const char *>(a.c.k) + lane % 8 * 16;
        const int64_t to_v = static_cast<const char *>(a.c.v) - static_cast<const char *>(a.c.k);
        const uint32_t to0 = ring + lane / 8 * 128;
        // Page ids are loaded four tiles ahead: a load returns behind the copies issued before it.
        Look next[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) next[j] = look(cw + 2 * j);
        // (in the give-up test mode no tile of the first block ever lands, and every role's wait for it runs out)
        bool ok = !(a.stall && (blockIdx.x | blockIdx.y | blockIdx.z) == 0);
        for (int t0 = cw; t0 < tiles && ok; t0 += 4) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int t = t0 + 2 * j;
                if (t >= tiles) break;
                const Look now = next[j];
                next[j] = look(t + 4);
                int64_t at[2];
                uint32_t bits[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const bool good = now.within[e] >= 0 && now.page[e] >= 0 && now.page[e] < a.c.n_pages;
                    if (now.within[e] >= 0 && !good && a.err) atomicOr(a.err, CBQ_DEVERR_BAD_SLOT);
                    at[e] = good ? (now.page[e] * a.c.page_stride + now.within[e] * a.c.tok_stride + head) * 2 : 0;
                    bits[e] = __ballot_sync(~0u, good);
                }
                if (t >= kStages) ok = warp_wait(sh, sh.empty[put.slot], (put.round - 1) & 1, a.err);
                if (!ok) break;
                const uint32_t to = to0 + put.slot * 2 * kTileBytes;
#pragma unroll
                for (int h = 0; h < 16; ++h) {
                    const int64_t off = __shfl_sync(~0u, at[h / 8], h % 8 * 4 + lane / 8);
                    const bool good = bits[h / 8] >> (h % 8 * 4 + lane / 8) & 1;
                    const char *from = from0 + off;
                    const uint32_t dst = to + h * 512 + ((lane ^ (h * 4 + lane / 8)) & 7) * 16;
#pragma unroll
                    for (int d = 0; d < D / 64; ++d) {
                        copy16(dst + d * kHalf, from + d * 128, good);
                        copy16(dst + kTileBytes + d * kHalf, from + to_v + d * 128, good);
                    }
                }
                if (t >= old_tiles) {  // the drafts: a value row with NaN or infinities is taken out
                    copy_commit();
                    copy_wait<0>();
                    __syncwarp();
                    constexpr uint32_t kExp = std::is_same_v<T, __half> ? 0x7C00u : 0x7F80u;  // all ones: not finite
#pragma unroll 1
                    for (int e = 0; e < 2; ++e) {
                        uint8_t *v = smem + 2 * kQBytes + (put.slot * 2 + 1) * kTileBytes + (e * 32 + lane) * 128;
                        bool odd = false;
#pragma unroll 4
                        for (int d = 0; d < D / 8; ++d) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(v + d / 8 * kHalf + d % 8 * 16);
#pragma unroll
                            for (int w = 0; w < 4; ++w) {
                                const uint32_t z = w == 0 ? y.x : w == 1 ? y.y : w == 2 ? y.z : y.w;
                                odd |= (z & kExp) == kExp || (z >> 16 & kExp) == kExp;
                            }
                        }
                        const uint32_t odds = __ballot_sync(~0u, odd);
                        if (odds) {
                            if (lane == 0) sh.odd[e] = odds;
                            if (odd)
                                for (int d = 0; d < D / 8; ++d)
                                    *reinterpret_cast<uint4 *>(v + d / 8 * kHalf + d % 8 * 16) = make_uint4(0, 0, 0, 0);
                            proxy_fence();
                            __syncwarp();
                        }
                    }
                }
                // arrives when this thread's copies have landed.  (Their writes are handed to the tensor cores by the fence
                // of the warp that issues the products; a fence here would wait for every copy under way.)
                asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&sh.full[put.slot])) : "memory");
                if (lane == 0) {
                    sh.valid[put.slot][0] = bits[0];
                    sh.valid[put.slot][1] = bits[1];
                    mbar_arrive(smem_addr(&sh.full[put.slot]));
                }
                put.step(2);
            }
        }
        copy_commit();
        copy_wait<0>();
    } else if (warp >= kScoreWarp) {
        // item i: group i % 2, tile i (keys shared out) or i / 2
        bool ok = true;
        Place at;
        if (warp == kScoreWarp) {
            for (int i = 0; i < items; ++i) {
                const int g = i & 1, n = i >> 1, b = n & 1;
                if (split || g == 0) {
                    ok = warp_wait(sh, sh.full[at.slot], at.round & 1, a.err);
                    if (!ok) break;
                    proxy_fence();
                }
                // into the place of the weights two items back, once they are in O
                if (n >= 2) ok = warp_wait(sh, sh.summed[g][b], (n >> 1 & 1) ^ 1, a.err);
                if (!ok) break;
                fence_after();
                if (lane == 0) mbar_arrive(smem_addr(&sh.scored[g][b]));
                const uint32_t q = q_at + (split ? 0 : g) * kQBytes, k_at = ring + at.slot * 2 * kTileBytes;
                const uint32_t s_at = tmem + Cols<D>::s(g, b);
#pragma unroll
                for (int j = 0; j < D / 16; ++j)
                    mma_ss(s_at, tile_desc(q + j / 4 * kQHalf + j % 4 * 32, 16), tile_desc(k_at + j / 4 * kHalf + j % 4 * 32, 16),
                           wide_idesc<T, kTile, false>(), j > 0);
                commit(sh.scored[g][b]);
                if (split || g == 1) at.step(1);
            }
        } else {
            for (int i = 0; i < items; ++i) {
                const int g = i & 1, n = i >> 1;
                ok = warp_wait(sh, sh.weighed[g][n & 1], n >> 1 & 1, a.err);
                if (!ok) break;
                fence_after();
                const uint32_t v_at = ring + (at.slot * 2 + 1) * kTileBytes, p_at = tmem + Cols<D>::s(g, n & 1);
#pragma unroll
                for (int j = 0; j < kTile / 16; ++j)
                    mma_ts(tmem + Cols<D>::o(g), p_at + j * 8, tile_desc(v_at + j * 2048, kHalf), wide_idesc<T, D, true>(),
                           n > 0 || j > 0);
                commit(sh.summed[g][n & 1]);
                if (split || g == 1) {
                    commit(sh.empty[at.slot]);
                    at.step(1);
                }
            }
        }
        // every product is done before the tensor memory is freed
        uint64_t &done = sh.done[warp - kScoreWarp];
        commit(done);
        const uint64_t t0 = global_ns();
        bool all = false;
        while (!(all = mbar_try_wait(smem_addr(&done), 0u)) && global_ns() - t0 < kWaitLimitNs) {}
        if (!all && a.err) atomicOr(a.err, kErrPipeTimeout);
    } else {
        // weights: thread = row of its group
        const int g = warp / 4, r = warp % 4 * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);
        constexpr float kLower = std::is_same_v<T, __half> ? 10.0f : 0.0f, kGrow = std::is_same_v<T, __half> ? 5.0f : 8.0f;
        float m = -INFINITY, l = 0.0f;  // weights are 2^(x - m): m is the maximum less kLower, or up to kGrow below that
        const int row_in = (split ? 0 : g * kGroup) + r;
        const bool live = row_in < rows;
        const int64_t tok = sq.row0 + (r0 + (live ? row_in : 0)) / group;
        const uint64_t sees = live ? seen_drafts(a, sq, tok) : 0;
        bool ok = true;
        int n = 0;  // items of this group so far
        Place at;
        if (split && g) at.step(1);
        for (int i = g; i < items; i += 2, ++n, at.step(split ? 2 : 1)) {
            const int slot = at.slot;
            ok = warp_wait(sh, sh.scored[g][n & 1], n >> 1 & 1, a.err);
            if (!ok) break;
            fence_after();
            uint32_t x[2][32];
            const uint32_t s_at = lanes + Cols<D>::s(g, 0) + (n & 1) * kTile;
            tm_ld(s_at, x[0]);
            tm_ld(s_at + 32, x[1]);
            uint32_t there[2] = {sh.valid[slot][0], sh.valid[slot][1]};
            if ((split ? i : i >> 1) >= old_tiles) there[0] &= (uint32_t)sees, there[1] &= (uint32_t)(sees >> 32);
            tm_wait_ld();
            if (!ok) break;
            if ((there[0] & there[1]) != ~0u) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!(there[h] >> j & 1)) x[h][j] = __float_as_uint(-INFINITY);
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int j = 0; j < 64; j += 2)
                top[j >> 1 & 3] = max3(top[j >> 1 & 3], __uint_as_float(x[j >> 5][j & 31]), __uint_as_float(x[j >> 5][(j & 31) + 1]));
            const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * sc - kLower;
            const bool grown = now > m + kGrow || (m == -INFINITY && now > -INFINITY);
            const float keep = grown ? pow2(m - now) : 1.0f;
            if (grown) m = now, l *= keep;
            if (n > 0 && __any_sync(~0u, grown)) {
                // O is scaled, once the products before are in it
                ok = warp_wait(sh, sh.summed[g][(n - 1) & 1], (n - 1) >> 1 & 1, a.err);
                if (!ok) break;
                fence_after();
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
            const float less = m == -INFINITY ? 0.0f : -m;
            const float2 sc2 = make_float2(sc, sc), less2 = make_float2(less, less);
            float2 sum[2] = {};
            uint32_t p[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                const float2 y = __ffma2_rn(make_float2(__uint_as_float(x[j >> 4][2 * j & 31]), __uint_as_float(x[j >> 4][(2 * j + 1) & 31])), sc2, less2);
                const float2 w = make_float2(pow2(y.x), pow2(y.y));
                sum[j & 1] = __fadd2_rn(sum[j & 1], w);
                p[j] = pack2<T>(w.x, w.y);
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            tm_st(s_at, p);
            tm_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.weighed[g][n & 1]));
        }
        if (l != l) m = 0.0f;  // (no maximum keeps a NaN: what joins the parts must not take them for empty)
        if (ok && n > 0) ok = warp_wait(sh, sh.summed[g][(n - 1) & 1], (n - 1) >> 1 & 1, a.err);
        fence_after();
        // The value rows taken out above, to the rows that see them: the weight of draft j is still in its place.
        if (ok && n > 0 && last && (split ? (tiles - 1) % 2 == g : true)) {
            for (uint64_t odd = (uint64_t)sh.odd[1] << 32 | sh.odd[0]; odd; odd &= odd - 1) {
                const int j = __ffsll((long long)odd) - 1;
                const uint32_t p = sq.ctx + j;
                const T *v = static_cast<const T *>(a.c.v) + table[p / (uint32_t)a.c.page_size] * a.c.page_stride +
                             (int64_t)(p % (uint32_t)a.c.page_size) * a.c.tok_stride + kvh * a.c.head_stride;
                const uint32_t two = tm_ld1(lanes + Cols<D>::s(g, 0) + ((n - 1) & 1) * kTile + j / 2);
                uint16_t half = (uint16_t)(j & 1 ? two >> 16 : two);
                const float w = to_f32(*reinterpret_cast<const T *>(&half));
#pragma unroll
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    tm_ld(lanes + Cols<D>::o(g) + d, o);
                    tm_wait_ld();
                    if (sees >> j & 1)
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) + w * to_f32(v[d + e]));
                    __syncwarp();
                    tm_st(lanes + Cols<D>::o(g) + d, o);
                    tm_wait_st();
                }
            }
        }
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
        if (!(split && g == 1)) {
            const int64_t row = tok * a.q_heads + kvh * group + (r0 + (live ? row_in : 0)) % group;
            float2 other = make_float2(-INFINITY, 0.0f);  // the other group's part of the row
            if (split && items > 1) other = sh.ml[r];
            const float top = fmaxf(m, other.x);
            const float f0 = n == 0 || top == -INFINITY ? 0.0f : pow2(m - top), f1 = top == -INFINITY ? 0.0f : pow2(other.x - top);
            const float sum = l * f0 + other.y * f1;
            const float inv = !alone ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
            const int64_t part = (int64_t)c * a.total_tok * a.q_heads + row;
            const int64_t to_row = (alone ? row : part) * D;
            if (split) {
#pragma unroll
                for (int d = 0; d < D; d += 32) {
                    uint32_t o[32];
                    tm_ld(lanes + Cols<D>::o(g) + d, o);
                    tm_wait_ld();
                    if (live && ok) {
#pragma unroll
                        for (int j = 0; j < 32; j += 8) {
                            float v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)  // (what was never written may hold anything: it is not multiplied)
                                v[e] = n == 0 ? 0.0f : __uint_as_float(o[j + e]) * f0;
                            if (items > 1) {
                                const float4 y0 = *reinterpret_cast<const float4 *>(pass + d + j), y1 = *reinterpret_cast<const float4 *>(pass + d + j + 4);
                                v[0] += y0.x * f1, v[1] += y0.y * f1, v[2] += y0.z * f1, v[3] += y0.w * f1;
                                v[4] += y1.x * f1, v[5] += y1.y * f1, v[6] += y1.z * f1, v[7] += y1.w * f1;
                            }
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] *= inv;
                            if (alone && !a.out_f32) {
                                *reinterpret_cast<uint4 *>(static_cast<T *>(a.out) + row * D + d + j) =
                                    make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
                            } else {
                                float4 *to = reinterpret_cast<float4 *>(alone ? static_cast<float *>(a.out) + row * D + d + j : part_o + part * D + d + j);
                                to[0] = make_float4(v[0], v[1], v[2], v[3]);
                                to[1] = make_float4(v[4], v[5], v[6], v[7]);
                            }
                        }
                    }
                    __syncwarp();
                }
            } else {
                // 32 rows x 32 values at a time, turned in shared memory (q's place, 16-byte pieces permuted by the row) so
                // that eight lanes write 128 bytes of a row: 12 sequences of 256 rows x 8,000 keys 116 us, each row by its
                // own thread 123.  (Above, where four warps write and add the other group's part, that was slower.)
                uint8_t *turn = smem + warp * 4096;
                static_assert(8 * 4096 <= 2 * kQBytes, "which has the room");
                const uint32_t lives = __ballot_sync(~0u, live && ok);
                const float f = n == 0 ? 0.0f : f0 * inv;
                int64_t at[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) at[i] = __shfl_sync(~0u, to_row, i * 4 + lane / 8) + lane % 8 * 4;
#pragma unroll
                for (int d = 0; lives && d < D; d += 32) {
                    uint32_t o[32];
                    tm_ld(lanes + Cols<D>::o(g) + d, o);
                    tm_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (n > 0)
                            v = make_float4(__uint_as_float(o[j]) * f, __uint_as_float(o[j + 1]) * f, __uint_as_float(o[j + 2]) * f,
                                            __uint_as_float(o[j + 3]) * f);
                        *reinterpret_cast<float4 *>(turn + lane * 128 + ((j / 4 ^ lane) & 7) * 16) = v;
                    }
                    __syncwarp();
                    float4 v[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] = *reinterpret_cast<const float4 *>(turn + (i * 4 + lane / 8) * 128 + ((lane ^ (i * 4 + lane / 8)) & 7) * 16);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (!(lives >> (i * 4 + lane / 8) & 1)) continue;
                        if (alone && !a.out_f32)
                            *reinterpret_cast<uint2 *>(static_cast<T *>(a.out) + at[i] + d) =
                                make_uint2(pack2<T>(v[i].x, v[i].y), pack2<T>(v[i].z, v[i].w));
                        else
                            *reinterpret_cast<float4 *>((alone ? static_cast<float *>(a.out) : part_o) + at[i] + d) = v[i];
                    }
                    __syncwarp();
                }
            }
            if (live && ok) {
                if (!alone) part_ml[part] = make_float2(top, sum);
                else if (a.lse) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
            }
        }
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kScoreWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
}

template <typename T, int D>
cudaError_t launch_wide(const TreeAttention &a, int chunk, int n_chunks, int row_tiles, float *part_o, float2 *part_ml, cudaStream_t s) {
    constexpr size_t kSmem = 2 * kGroup * D * 2 + kStages * 2 * kTile * D * 2;
    static_assert(kGroup * (D + 4) * 4 <= kStages * 2 * kTile * D * 2, "group 1's part fits the ring");
    return launch_dependent(k_tree_wide<T, D>, dim3((unsigned)(a.c.kv_heads * row_tiles), (unsigned)n_chunks, (unsigned)a.n_seq),
                            kWideThreads, kSmem, s, a, chunk, row_tiles, part_o, part_ml);
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
