// cbq_sample.cu -- one token from each row of logits: temperature, top-k,
// top-p and min-p, drawn by a given uniform number.
//
// A cluster of up to sixteen blocks takes a row; every thread reads its few
// logits once (with many rows fewer blocks a row and more logits a thread, kept
// in shared memory: less waiting for one another).  Nothing is sorted: what
// top-k and top-p keep is all above a border in the order and the first few
// equal to it.  A histogram over the row (of counts for top-k, of weights for
// top-p) finds the bin of the border, and only what can still be kept is
// listed.  Up to 256 of those one block compares with one another, each with
// all, and is done.  With more, what lies in the border's bin every block gets
// from all others and finds the border in it by itself, and the lists are
// summed up in the order of the indices.  Weights are whole numbers of 2^-45,
// so that their sums do not depend on the order of atomics and a choice is the
// same on every run.
//
// Bound by the arithmetic of the weights where a whole row is weighed (no cut,
// or top-p alone: some 40 instructions a logit, packed ones for two at a time
// among them, 10 of a row's 16 us in a block with 32 logits a thread) and otherwise by its phases' latency: a cluster's
// wait for all its blocks takes 0.5 to 0.9 us, a histogram of a row with its
// sums 3.  Many rows: a block of 1,024 threads fills an SM, so a row's load waits
// for the phases of the one before it (issue slots 61% busy while an SM has a
// block, 38% over the launch).  129,280 fp32 logits: a row with top-p alone 11 us
// where that keeps few, 19 with thousands, 29 with half of the row; five rows
// with all cuts 14.4 us (the general way, without one block that settles few:
// 20.9), 256 rows of all kinds 121.
#include <cfloat>

#include "cbq_device.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

namespace {

constexpr int kSampleThreads = 1024, kNumWarps = kSampleThreads / 32;
constexpr int kBinBits = 9, kBins = 1 << kBinBits;
constexpr int kGather = 2048;             // logits of a border's bin, from all blocks
constexpr int kMaxBlocks = 16;            // of a cluster
constexpr int kFew = kGather / 4;         // a top-k whose list will mostly fit there
constexpr int kSettle = kSampleThreads / 4;  // listed ones that one block settles, four threads each
constexpr int kTable = 256;               // steps of 2^(1/256) of the weights' table
constexpr uint64_t kOne = 1ull << 45;     // the weight 1
constexpr uint32_t kNone = 0x007FFFFFu;   // order of -inf: what is not above has no weight

// 2^(i/256) in units of 2^-46, from the eight square roots 2^(1/2) .. 2^(1/256).
struct PowTable {
    uint64_t v[kTable];
};
constexpr double root2(double x) {
    double r = x > 1.0 ? x : 1.0;
    for (int i = 0; i < 60; ++i) r = 0.5 * (r + x / r);
    return r;
}
constexpr PowTable make_table() {
    PowTable t{};
    double roots[8] = {};
    double x = 2.0;
    for (int j = 0; j < 8; ++j) {
        x = root2(x);
        roots[j] = x;  // 2^(1/2^(j+1))
    }
    for (int i = 0; i < kTable; ++i) {
        double p = 1.0;
        for (int j = 0; j < 8; ++j)
            if (i >> (7 - j) & 1) p *= roots[j];
        t.v[i] = (uint64_t)(p * 2.0 * (double)kOne + 0.5);
    }
    return t;
}
__device__ const PowTable kPow = make_table();

// Unsigned numbers in the order of the logits (no NaN, no -0 among them).
__device__ __forceinline__ uint32_t order_of(float l) {
    const uint32_t b = __float_as_uint(l);
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
}

// exp((l - top) / T) as a 2^-45 fixed-point number, by a table and a short
// polynomial (the method of P. T. P. Tang, ACM TOMS 15, 1989).  With y = (l -
// top) * log2(e)/T carried as two fp32 numbers (about 2^-44 of |y| <= 46), n =
// round(256 y) and t = (y - n/256) ln 2, |t| <= 2^-9.5: the weight is
// table[n mod 256] * (1 + (t + t^2/2 + t^3/6)) >> -floor(n/256); 1 + .. is a
// 2^-40 fixed-point number, whose rounding (2^-41) is the largest error.
// Rounding to a whole number by adding 1.5 * 2^23 keeps the conversion units,
// a quarter as wide as the others, out of it but for one conversion.
struct Scale {
    float top, hi, lo;  // hi + lo = log2(e) / T
};
// Two logits at a time: a packed instruction does the arithmetic of both.
struct Two {
    uint64_t a, b;
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ Two weigh(float la, float lb, const Scale &s, const uint64_t *table) {
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236017e-9f;
    constexpr float k40 = 1099511627776.0f, kRound = 12582912.0f;
    constexpr int kRoundBits = 0x4B400000;
    const float2 l = make_float2(la, lb), minus = both(-1.0f), hi = both(s.hi);
    const float2 d = __fadd2_rn(l, both(-s.top)), w = __fmul2_rn(d, both(-s.hi));
    const float2 z = make_float2(fminf(w.x, 50.0f), fminf(w.y, 50.0f));  // -y (NaN, which no scale times -inf would give, becomes 50 too)
    const float2 back = __fadd2_rn(d, both(s.top));                      // two-sum: d + e is the exact difference
    const float2 e = __fadd2_rn(__ffma2_rn(back, minus, l), __fadd2_rn(__ffma2_rn(d, minus, back), both(-s.top)));
    const float2 yl = __fadd2_rn(__ffma2_rn(d, hi, z), __ffma2_rn(d, both(s.lo), __fmul2_rn(e, hi)));
    const float2 nr = __ffma2_rn(z, both(-(float)kTable), both(kRound));
    const float2 r = __ffma2_rn(__fadd2_rn(nr, both(-kRound)), both(1.0f / kTable), z);  // n/256 - y, exact: they agree in their leading bits
    const float2 th = __fmul2_rn(r, both(kLn2Hi));                       // -t's larger part
    const float2 tl = __fadd2_rn(__ffma2_rn(r, both(-kLn2Hi), th), __ffma2_rn(r, both(-kLn2Lo), __fmul2_rn(yl, both(kLn2Hi))));
    const float2 t = __ffma2_rn(th, minus, tl);
    const float2 quad = __ffma2_rn(__fmul2_rn(t, t), __ffma2_rn(t, both(1.0f / 6.0f), both(0.5f)), tl);
    const float2 large = __fmul2_rn(th, both(-k40)), small = __ffma2_rn(quad, both(k40), both(kRound));
    auto whole = [&](float n256, float x, float y) {
        const int ni = __float_as_int(n256) - kRoundBits, p = __float2int_rn(x) + (__float_as_int(y) - kRoundBits);
        const uint64_t v = table[ni & (kTable - 1)];
        const uint64_t full = v + (uint64_t)((int64_t)(int32_t)(v >> 16) * p >> 24);
        return ((full >> (-(ni >> 8))) + 1) >> 1;  // (full is below 2^48: nothing from y = -50, whatever p is there)
    };
    return Two{whole(nr.x, large.x, small.x), whole(nr.y, large.y, small.y)};
}
__device__ __forceinline__ uint64_t weight(float l, const Scale &s, const uint64_t *table) { return weigh(l, l, s, table).a; }

// ------------------------------------------------------------- clusters ----

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
// The address of p, a place in this block's shared memory, in block r of the cluster.
__device__ __forceinline__ uint32_t peer(const void *p, uint32_t r) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(r));
    return a;
}
__device__ __forceinline__ void peer_store(uint32_t a, uint64_t v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void peer_store(uint32_t a, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ uint64_t peer_load(uint32_t a) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

// Sums by bin.  Weights are added in three 16-bit parts (a block adds fewer
// than 2^16 of them, so 32 bits hold each part's sum; 64-bit atomics on shared
// memory are loops), counts in part[0]; mine[] is the block's whole, all[] the
// cluster's.
struct Hist {
    union {
        uint32_t part[3][kBins];
        uint64_t all[kBins];
    };
    uint64_t mine[kBins];
};

struct alignas(16) Shared {
    uint64_t table[kTable];
    Hist hist[2];
    uint64_t swap[2][kMaxBlocks][2];  // what the blocks of the cluster tell one another
    uint64_t warp[kNumWarps], upto[kNumWarps];  // sums of the warps, and inclusive sums of those
    uint32_t key[kNumWarps], at[kNumWarps], listed[kNumWarps];
    alignas(8) uint32_t gather[kGather];  // the border's bin, of all blocks
    uint64_t above, inside, goal;
    int bin, index;
    uint32_t count;
};

// f * n, rounded down or up to a whole number, exactly; f in [0, 1].  (64-bit
// floating point is a sixty-fourth as wide as 32-bit on this GPU.)
__device__ __forceinline__ uint64_t share(uint64_t n, float f, bool up) {
    const uint32_t b = __float_as_uint(f);
    const uint64_t m = (b & 0x7FFFFFu) | (b >> 23 ? 0x800000u : 0u);
    const int s = 150 - max((int)(b >> 23), 1);  // f = m 2^-s, 23 <= s <= 149
    const uint64_t lo = n * m, hi = __umul64hi(n, m);
    uint64_t whole, rest;
    if (s < 64) {
        whole = hi << (64 - s) | lo >> s;
        rest = lo << (64 - s);
    } else {
        whole = s < 128 ? hi >> (s - 64) : 0;
        rest = lo | (s < 128 ? hi & ((1ull << (s - 64)) - 1) : hi);
    }
    return whole + (up && rest ? 1 : 0);
}

// Of a mass, how much has to be reached for the number u.
__device__ __forceinline__ uint64_t taken(uint64_t mass, float u) {
    return min(share(mass, fminf(fmaxf(u, 0.0f), 1.0f), false) + 1, mass);
}

__device__ __forceinline__ int warp_scan32(int v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
    }
    return v;
}
__device__ __forceinline__ uint64_t warp_scan(uint64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t u = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// One block's part of a row and its place in the cluster.  Warp w has the
// stretch of 32 N logits from first + 32 N w on; those that may be kept are
// listed, in order, with their place in the stretch.
template <int N>
struct Part {
    Shared &s;
    float *list;        // 32 N a warp
    uint16_t *place;
    int first, blocks, rank, warp, lane;
    int listed = 0;         // of this warp
    bool whole = false;     // all of the stretch, each in its place
    int turn = 0, use = 0;  // which of the two swap buffers and histograms is next

    // Every block gives two numbers (the same in all its threads); lane r of
    // each warp gets block r's, {0, 0} past the last.  A buffer is written again
    // two calls later: all have read it by then.
    __device__ ulonglong2 tell(uint64_t a, uint64_t b) {
        uint64_t(*to)[2] = s.swap[turn];
        turn ^= 1;
        if (threadIdx.x < (unsigned)blocks) {
            peer_store(peer(&to[rank][0], threadIdx.x), a);
            peer_store(peer(&to[rank][1], threadIdx.x), b);
        }
        cluster_sync();
        return lane < blocks ? make_ulonglong2(to[lane][0], to[lane][1]) : make_ulonglong2(0, 0);
    }

    // s.upto from a sum a warp (shuffles of 64 bits are dear: one warp does them).
    __device__ void sum_warps(uint64_t v) {
        __syncthreads();
        if (lane == 31) s.warp[warp] = v;
        __syncthreads();
        if (warp == 0) s.upto[lane] = warp_scan(s.warp[lane], lane);
        __syncthreads();
    }

    // The inclusive sum of v over the threads before and this one; *total: over
    // all.  Only the first `warps` warps have any.
    __device__ uint64_t block_scan(uint64_t v, int warps, uint64_t *total) {
        v = warp < warps ? warp_scan(v, lane) : 0;
        sum_warps(v);
        *total = s.upto[31];
        return v + (warp ? s.upto[warp - 1] : 0);
    }

    // A step of a descent: fill(add) calls add(bin, value) for what takes part,
    // bins ascending as the order descends; kWide: over all blocks of the
    // cluster, otherwise this block's.  need(total): how much to take.  Finds
    // the first bin with which that is reached: s.bin (-1: never), s.above
    // before it, s.inside in it.
    template <bool kWeights, bool kWide, typename F, typename G>
    __device__ void step(F fill, G need) {
        static_assert(kNumWarps == 32 && kBins <= kSampleThreads, "a bin a thread, a warp a lane");
        Hist &h = s.hist[use];  // last read two steps ago: a barrier lies between
        use ^= 1;
        __syncthreads();  // s.bin of the step before has been read
        if (threadIdx.x < kBins) {
#pragma unroll
            for (int p = 0; p < (kWeights ? 3 : 1); ++p) h.part[p][threadIdx.x] = 0;
        }
        if (threadIdx.x == 0) s.bin = -1;
        __syncthreads();
        fill([&](int b, uint64_t v) {
            if constexpr (kWeights) {
                atomicAdd(&h.part[0][b], (uint32_t)v & 0xFFFFu);
                atomicAdd(&h.part[1][b], (uint32_t)(v >> 16) & 0xFFFFu);
                atomicAdd(&h.part[2][b], (uint32_t)(v >> 32));
            } else {
                atomicAdd(&h.part[0][b], (uint32_t)v);
            }
        });
        __syncthreads();
        uint64_t sum = 0;
        if (threadIdx.x < kBins) {
            sum = h.part[0][threadIdx.x];
            if constexpr (kWeights)
                sum += ((uint64_t)h.part[1][threadIdx.x] << 16) + ((uint64_t)h.part[2][threadIdx.x] << 32);
            if constexpr (kWide) h.mine[threadIdx.x] = sum;
        }
        if constexpr (kWide) {
            // each block adds up a share of the bins over all blocks and hands the sums out: a load and a store a
            // thread (all bins of all blocks read by each block took twice as long: 14 bytes a clock come from others)
            cluster_sync();
            const int r = threadIdx.x & (blocks - 1), b = (rank * kBins + (int)threadIdx.x) / blocks;
            if (threadIdx.x < kBins) {
                sum = peer_load(peer(&h.mine[b], r));
                for (int o = blocks / 2; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
                peer_store(peer(&h.all[b], r), sum);
            }
            cluster_sync();
            sum = threadIdx.x < kBins ? h.all[threadIdx.x] : 0;
        }
        uint64_t total;
        const uint64_t upto = block_scan(sum, kBins / 32, &total), want = need(total);
        if (upto - sum < want && upto >= want) {
            s.bin = threadIdx.x;
            s.above = upto - sum;
            s.inside = sum;
        }
        __syncthreads();
    }

    // The border in one bin of a wide step: the logit at which the counts or
    // weights of what is listed and in_bin(logit), summed from the top after
    // `up`, reach goal.  *above: the sum above it; *inside: at it.
    template <bool kWeights, typename B, typename V>
    __device__ float border(B in_bin, V value, uint64_t goal, uint64_t up, uint64_t *above, uint64_t *inside) {
        uint32_t *own = reinterpret_cast<uint32_t *>(&s.hist[use]);  // this block's part (the next step's histogram, not yet used)
        static_assert(sizeof(Hist) >= kGather * sizeof(uint32_t) && kBins >= kSettle, "which has the room");
        if (threadIdx.x == 0) s.count = 0;
        __syncthreads();
        uint32_t lo = ~0u, hi = 0;
        for (int i = lane; i < listed; i += 32) {
            const float l = list[i];
            if (!in_bin(l)) continue;
            const uint32_t o = order_of(l), n = atomicAdd(&s.count, 1u);
            if (n < kGather) own[n] = o;
            lo = min(lo, o), hi = max(hi, o);
        }
        lo = __reduce_min_sync(~0u, lo);
        hi = __reduce_max_sync(~0u, hi);
        if (lane == 0) s.key[warp] = lo, s.at[warp] = hi;
        __syncthreads();
        lo = __reduce_min_sync(~0u, s.key[lane]);
        hi = __reduce_max_sync(~0u, s.at[lane]);
        const int count = s.count, room = kGather / blocks;
        for (int i = threadIdx.x; i < min(count, room) * blocks; i += kSampleThreads)
            peer_store(peer(&s.gather[rank * room + i / blocks], i % blocks), own[i / blocks]);
        const ulonglong2 all = tell((uint64_t)hi << 32 | lo, count);
        lo = __reduce_min_sync(~0u, lane < blocks ? (uint32_t)all.x : ~0u);
        hi = __reduce_max_sync(~0u, (uint32_t)(all.x >> 32));
        const bool fits = __all_sync(~0u, (int)all.y <= room);
        constexpr int kEach = kGather / kSampleThreads;
        uint32_t o[kEach];
        uint64_t v[kEach];
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int i = threadIdx.x + j * kSampleThreads;
            // (32 threads in a row look at one block's room, which is a multiple of that)
            const bool there = fits && i % room < (int)__shfl_sync(~0u, (uint32_t)all.y, i / room);
            o[j] = there ? s.gather[i] : 0;
            v[j] = there ? value(logit_of(o[j])) : 0;
        }
        *inside = 0;
        if (lo == hi) {  // equal ones alone: nothing to look for, but what they come to
            *inside = __reduce_add_sync(~0u, (uint32_t)all.y) * value(logit_of(lo));
        }
        while (lo < hi) {
            if (fits) {  // few: each with all (a step of a descent takes 1.4 us, and there would be three)
                uint64_t *w = s.hist[use].mine;
                if (threadIdx.x == 0) s.count = 0;
                __syncthreads();
#pragma unroll
                for (int j = 0; j < kEach; ++j) {
                    if (hi - o[j] > hi - lo || !v[j]) continue;
                    const uint32_t n = atomicAdd(&s.count, 1u);
                    if (n < kSettle) own[n] = o[j], w[n] = v[j];
                }
                __syncthreads();
                const int n = s.count, e = threadIdx.x / 4, some = warp * 8 < n ? n : 0;
                if (n <= kSettle) {
                    const uint32_t mine = e < n ? own[e] : ~0u;
                    uint64_t before = 0, equal = 0;
#pragma unroll 4
                    for (int f = threadIdx.x % 4; f < some; f += 4) {
                        const uint32_t other = own[f];
                        const uint64_t x = w[f];
                        before += other > mine ? x : 0;
                        equal += other == mine ? x : 0;
                    }
#pragma unroll
                    for (int i = 1; i < 4; i *= 2) {
                        before += __shfl_xor_sync(~0u, before, i);
                        equal += __shfl_xor_sync(~0u, equal, i);
                    }
                    if (e < n && up + before < goal && up + before + equal >= goal) {  // (equal ones: all of them)
                        s.above = up + before;
                        s.inside = equal;
                        s.index = (int)mine;
                    }
                    __syncthreads();
                    *above = s.above;
                    *inside = s.inside;
                    return logit_of((uint32_t)s.index);
                }
            }
            const int sh = max(0, 32 - __clz(hi - lo) - kBinBits);  // (hi - lo) >> sh is below kBins
            auto need = [&](uint64_t) { return goal - up; };
            if (fits) {
                step<kWeights, false>([&](auto add) {
#pragma unroll
                    for (int j = 0; j < kEach; ++j)
                        if (hi - o[j] <= hi - lo && v[j]) add((int)((hi - o[j]) >> sh), v[j]);
                }, need);
            } else {  // very many equal or near ones: the lists themselves, over all blocks
                step<kWeights, true>([&](auto add) {
                    for (int i = lane; i < listed; i += 32) {
                        const uint32_t k = hi - order_of(list[i]);
                        if (k > hi - lo || !in_bin(list[i])) continue;
                        const uint64_t x = value(list[i]);
                        if (x) add((int)(k >> sh), x);
                    }
                }, need);
            }
            const uint32_t top = hi - ((uint32_t)s.bin << sh);
            lo = top - lo < (1u << sh) ? lo : top - ((1u << sh) - 1);
            hi = top;
            up += s.above;
            *inside = s.inside;
        }
        *above = up;
        return logit_of(lo);
    }

    // The index where value(two logits) of what is listed and counts(index, logit,
    // value), summed in the order of the indices over the whole row, reaches
    // need(sum); -1 in the blocks that do not hold it.  *total: the row's sum;
    // *at: the value there.
    template <typename V, typename C, typename G>
    __device__ int walk(V value, C counts, G need, uint64_t *total, uint64_t *at) {
        const int start = first + warp * N * 32;
        uint64_t mine = 0;
        for (int i0 = 0; i0 < listed; i0 += 128) {  // two chains of arithmetic at a time (and within the stretch)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
                const int i = i0 + j * 32 + lane;
                const float la = list[i], lb = list[i + 32];
                const Two v = value(la, lb);
                mine += i < listed && counts(start + (whole ? i : (int)place[i]), la, v.a) ? v.a : 0;
                mine += i + 32 < listed && counts(start + (whole ? i + 32 : (int)place[i + 32]), lb, v.b) ? v.b : 0;
            }
        }
        // at most 2^50 a lane: the sum of a warp in two halves
        sum_warps((uint64_t)__reduce_add_sync(~0u, (uint32_t)mine & 0xFFFFFFu) +
                  ((uint64_t)__reduce_add_sync(~0u, (uint32_t)(mine >> 24)) << 24));
        if (lane == 0) s.listed[warp] = listed;
        const uint64_t block = s.upto[31], other = tell(block, 0).x;
        if (warp == 0) {
            const uint64_t upto = warp_scan(other, lane), sum = __shfl_sync(~0u, upto, 31);
            const uint64_t before = __shfl_sync(~0u, upto, rank) - block, goal = need(sum);
            if (lane == 0) s.above = before, s.inside = sum, s.goal = goal;
        }
        __syncthreads();
        uint64_t before = s.above;
        const uint64_t goal = s.goal;
        *total = s.inside;
        if (!(before < goal && before + block >= goal)) return -1;
        // this block: its threads share out the list of the warp that holds it
        const int owner = __ffs(__ballot_sync(~0u, before + s.upto[lane] >= goal)) - 1;
        before += owner ? s.upto[owner - 1] : 0;
        constexpr int kEach = (N * 32 + kSampleThreads - 1) / kSampleThreads;
        static_assert(kEach == 1, "a thread a place");
        const int to = owner - warp, n = s.listed[owner], i = threadIdx.x;
        const int where = first + owner * N * 32 + (i < n ? (whole ? i : (int)place[to * N * 32 + i]) : 0);
        uint64_t v = 0;
        if (i < n) {
            const float l = list[to * N * 32 + i];
            v = value(l, l).a;
            v = counts(where, l, v) ? v : 0;
        }
        uint64_t rest;
        const uint64_t upto = before + block_scan(v, N, &rest);
        if (upto - v < goal && upto >= goal) {
            s.index = where;
            s.inside = v;
        }
        __syncthreads();
        *at = s.inside;
        return s.index;
    }

    // What is listed, of all blocks, into the first block's gather, if it is no more than kSettle: order and index in
    // one number that is larger the earlier in the order.  The number of all, in every thread.
    __device__ int collect() {
        if (lane == 0) s.listed[warp] = listed;
        __syncthreads();
        const int upto = warp_scan32(s.listed[lane], lane), block = __shfl_sync(~0u, upto, 31);
        const int others = warp_scan32((int)tell(block, 0).x, lane), n = __shfl_sync(~0u, others, 31);
        const int to = __shfl_sync(~0u, others, rank) - block + __shfl_sync(~0u, upto, warp) - listed;
        if (n <= kSettle) {
            const uint64_t *all = reinterpret_cast<const uint64_t *>(s.gather);
            for (int i = lane; i < listed; i += 32)
                peer_store(peer(all + to + i, 0), (uint64_t)order_of(list[i]) << 32 | ~(uint32_t)(first + warp * N * 32 + place[i]));
        }
        cluster_sync();
        return n;
    }

    // The rest for those n in one block, without another word from the others: for each, what comes before it in the
    // order, and, of what is kept, before it by index.  want(mass of the first k): what top-p's must reach.
    template <typename F, typename G>
    __device__ void settle(int n, int k, F mass, G want, uint64_t least, float u, int32_t *id, float *prob) {
        uint64_t *key = reinterpret_cast<uint64_t *>(s.gather), *w = key + kSettle, *kept = w + kSettle;
        static_assert(sizeof(s.gather) >= 3 * kSettle * sizeof(uint64_t), "three numbers each");
        if (threadIdx.x < (unsigned)n) w[threadIdx.x] = mass(logit_of((uint32_t)(key[threadIdx.x] >> 32)));
        __syncthreads();
        const int e = threadIdx.x / 4, q = threadIdx.x % 4, some = warp * 8 < n ? n : 0;
        const uint64_t mine = e < n ? key[e] : ~0ull, own = e < n ? w[e] : 0;
        int place_of = 0;
        uint64_t before = 0;
#pragma unroll 4
        for (int f = q; f < some; f += 4) {
            const uint64_t other = key[f], x = w[f];
            place_of += other > mine;
            before += other > mine ? x : 0;
        }
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {
            place_of += __shfl_xor_sync(~0u, place_of, o);
            before += __shfl_xor_sync(~0u, before, o);
        }
        if (e < n && place_of == min(k, n) - 1) s.goal = before + own;
        __syncthreads();
        const bool stays = e < n && place_of < k && before < want(s.goal) && own >= least;
        if (e < n && q == 0) kept[e] = stays ? own : 0;
        __syncthreads();
        uint64_t upto = 0, total = 0;
#pragma unroll 4
        for (int f = q; f < some; f += 4) {
            const uint64_t x = kept[f];
            total += x;
            upto += (uint32_t)key[f] >= (uint32_t)mine ? x : 0;  // (the complement of the index)
        }
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {
            upto += __shfl_xor_sync(~0u, upto, o);
            total += __shfl_xor_sync(~0u, total, o);
        }
        const uint64_t goal = taken(total, u);
        if (stays && q == 0 && upto - own < goal && upto >= goal) {
            *id = (int32_t)~(uint32_t)mine;
            if (prob) *prob = (float)((double)own / (double)total);
        }
    }
};

// grid (blocks of the cluster, rows).
template <typename T, int N>
__global__ void __launch_bounds__(kSampleThreads, 1) k_sample(Sample a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    cluster_arrive();
    pdl_trigger();
    const int c = blockIdx.y, lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    if (threadIdx.x < kTable) s.table[threadIdx.x] = kPow.v[threadIdx.x];
    float *lists = reinterpret_cast<float *>(smem + sizeof(Shared));
    uint16_t *places = reinterpret_cast<uint16_t *>(lists + N * kSampleThreads);
    Part<N> row = {s, lists + warp * N * 32, places + warp * N * 32, (int)blockIdx.x * N * kSampleThreads, (int)gridDim.x,
                   (int)cluster_rank(), warp, lane};
    pdl_wait();
    const float temp = a.temperature ? a.temperature[c] : 1.0f, p = a.top_p ? a.top_p[c] : 1.0f;
    const float least = a.min_p ? a.min_p[c] : 0.0f, u = a.u[c];
    const int k = a.top_k ? a.top_k[c] : 0;
    const T *logits = static_cast<const T *>(a.logits) + c * a.row_stride;
    const int start = row.first + warp * N * 32 + lane;
    // The logits: in registers, or (32 a thread) in shared memory where the list will be, a thread reading its own.
    // NaN becomes -inf, and -0 becomes +0.
    constexpr bool kShared = N > 16;
    constexpr int kSome = N < 16 ? N : 16;  // loads under way at a time
    float held[kShared ? 1 : N];
    float best = -INFINITY;
#pragma unroll
    for (int j0 = 0; j0 < N; j0 += kSome) {
        T y[kSome];
#pragma unroll
        for (int j = 0; j < kSome; ++j) y[j] = logits[min(start + (j0 + j) * 32, a.V - 1)];
#pragma unroll
        for (int j = 0; j < kSome; ++j) {
            float l = to_f32(y[j]);
            l = start + (j0 + j) * 32 < a.V && l == l ? l + 0.0f : -INFINITY;
            best = fmaxf(best, l);
            if constexpr (kShared) row.list[(j0 + j) * 32 + lane] = l;
            else held[j0 + j] = l;
        }
    }
    auto x = [&](int j) {
        if constexpr (kShared) return row.list[j * 32 + lane];
        else return held[j];
    };

    // the top of the order
    uint32_t top = __reduce_max_sync(~0u, order_of(best));
    if (lane == 0) s.key[warp] = top;
    __syncthreads();
    cluster_wait();  // every block of the cluster runs: its shared memory may be written
    top = __reduce_max_sync(~0u, s.key[lane]);
    top = __reduce_max_sync(~0u, (uint32_t)row.tell(top, 0).x);
    if (top <= kNone || !(temp > 0.0f) || least > 1.0f) {
        // no temperature, or a min-p that the first alone meets: the first it is (if there is any)
        uint32_t at = ~0u;
#pragma unroll
        for (int j = N - 1; j >= 0; --j)
            if (x(j) == logit_of(top)) at = (uint32_t)(start + j * 32);
        at = __reduce_min_sync(~0u, at);
        if (lane == 0) s.at[warp] = at;
        __syncthreads();
        at = __reduce_min_sync(~0u, s.at[lane]);
        const ulonglong2 all = row.tell(at, 0);  // (by all lanes: a barrier of the cluster)
        at = __reduce_min_sync(~0u, lane < row.blocks ? (uint32_t)all.x : ~0u);
        if (threadIdx.x == 0 && row.rank == 0) {
            a.ids[c] = top <= kNone ? -1 : (int)at;
            if (a.probs) a.probs[c] = top <= kNone ? 0.0f : 1.0f;
        }
        return;
    }
    if (logit_of(top) == INFINITY) {  // only what is infinite has weight: as 0 among -inf
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float l = x(j) == INFINITY ? 0.0f : -INFINITY;
            if constexpr (kShared) row.list[j * 32 + lane] = l;
            else held[j] = l;
        }
        best = best == INFINITY ? 0.0f : -INFINITY;
        top = order_of(0.0f);
    }
    constexpr float kLog2eHi = 1.44269502162933349609375f, kLog2eLo = 1.925963033500011e-8f;
    Scale sc;
    sc.top = logit_of(top);
    sc.hi = fminf(kLog2eHi / temp, 1e30f);
    sc.lo = sc.hi < 1e30f && temp < INFINITY ? (__fmaf_rn(-sc.hi, temp, kLog2eHi) + kLog2eLo) / temp : 0.0f;

    // bins of 1/10.5 of a power of two of the weight; the last takes the rest
    const float cut = sc.hi * (kBins / 48.6f);
    auto t_of = [&](float l) { return l == sc.top ? 0 : min(__float2int_rz((sc.top - l) * cut), kBins - 1); };
    auto mass = [&](float l) { return weight(l, sc, s.table); };
    auto one = [](float) { return (uint64_t)1; };
    const uint64_t floor_w = least > 0.0f ? share(kOne, least, true) : 0;  // the least weight that min-p keeps

    // a histogram of the whole row, by counts for top-k or else by weights for top-p, and the bin of the border
    bool by_k = k > 0 && k < a.V;
    const bool by_p = p < 1.0f, weighed = by_p && !by_k;  // (weights first only where top-k cuts nothing)
    // For the few of a small top-k the largest logit of each thread is enough: as many of those as top-k takes lie at or
    // above a bin, so its border does, and all that is listed may be the border's (256 rows of 129,280 logits, top-k 100:
    // 153 us with every logit counted, 148 so, and then 92 as one block settles what is listed).
    bool few = by_k && k <= kFew;
    int bin = kBins - 1;
    uint64_t want = 0, above = 0, inside = 0;
    auto goal = [&](uint64_t mass_of) { return max(share(mass_of, fmaxf(p, 0.0f), true), (uint64_t)1); };
    if (few) {
        row.template step<false, true>([&](auto add) {
            if (best > -INFINITY) add(t_of(best), 1);
        }, [&](uint64_t) { return (uint64_t)k; });
        few = s.bin >= 0;
        if (few) bin = s.bin;
    }
    if (by_k && !few) {
        row.template step<false, true>([&](auto add) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (x(j) > -INFINITY) add(t_of(x(j)), 1);
        }, [&](uint64_t) { return (uint64_t)k; });
        by_k = s.bin >= 0;
        if (by_k) bin = s.bin, above = s.above;
    } else if (weighed) {
        row.template step<true, true>([&](auto add) {
#pragma unroll (kShared ? 1 : N / 4)
            for (int j0 = 0; j0 < N; j0 += 4) {  // two chains of arithmetic at a time
                float l[4];
                uint64_t v[4];
#pragma unroll
                for (int j = 0; j < 4; j += 2) {
                    l[j] = x(j0 + j), l[j + 1] = x(j0 + j + 1);
                    const Two w = weigh(l[j], l[j + 1], sc, s.table);
                    v[j] = w.a, v[j + 1] = w.b;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (v[j]) add(t_of(l[j]), v[j]);
            }
        }, [&](uint64_t total) { return want = goal(total); });
        bin = s.bin;
        above = s.above;
    }

    // The list of what may still be kept (where the logits lie in its place, it closes up behind what has been read):
    // all down to a logit that lies a little below the border's bin, or below what min-p keeps.
    const bool all_of = by_k || by_p;
    if (!all_of && !(least > 0.0f)) {
        row.whole = true;
        row.listed = N * 32;
        if constexpr (!kShared) {
#pragma unroll
            for (int j = 0; j < N; ++j) row.list[j * 32 + lane] = held[j];
        }
        __syncwarp();
    } else {
        const float down = !all_of ? (0.01f - log2f(least)) / sc.hi : bin < kBins - 1 ? (bin + 1) / cut : INFINITY;
        const float lim = fmaxf(__fsub_rd(sc.top, down * 1.00001f), -FLT_MAX);
#pragma unroll (kShared ? 8 : N)
        for (int j = 0; j < N; ++j) {
            const float l = x(j);
            const unsigned who = __ballot_sync(~0u, l >= lim);
            if (!who) continue;
            const int to = row.listed + __popc(who & ((1u << lane) - 1));
            if (l >= lim) row.list[to] = l, row.place[to] = (uint16_t)(j * 32 + lane);
            row.listed += __popc(who);
        }
        __syncwarp();
        const int n = row.collect();
        if (n <= kSettle) {
            if (row.rank == 0)
                row.settle(n, by_k ? k : a.V, mass, [&](uint64_t m) { return !by_p ? ~0ull : weighed ? want : goal(m); }, floor_w, u,
                           a.ids + c, a.probs ? a.probs + c : nullptr);
            return;
        }
    }

    float tau = -INFINITY;  // kept: above tau, and the first `ties` at it (all, if ~0)
    uint64_t ties = ~0ull;
    if (by_k) {
        tau = row.template border<false>([&](float l) { return few || t_of(l) == bin; }, one, (uint64_t)k, above, &above, &inside);
        ties = (uint64_t)k - above < inside ? (uint64_t)k - above : ~0ull;
    }
    if (by_p) {
        // with a cut among the equals at tau, those weigh `ties` times one of them: the border is looked for above them
        const bool part_of = ties != ~0ull;
        auto takes = [&](float l) { return l > tau || (l == tau && !part_of); };
        uint64_t all = 0;  // the mass of what is looked at
        if (!weighed) {
            const uint64_t rest = part_of ? ties * mass(tau) : 0;
            row.template step<true, true>([&](auto add) {
                for (int i = lane; i < row.listed; i += 32) {
                    const uint64_t v = takes(row.list[i]) ? mass(row.list[i]) : 0;
                    if (v) add(t_of(row.list[i]), v);
                }
            }, [&](uint64_t total) {
                all = total;
                return want = goal(total + rest);
            });
            bin = s.bin;
            above = s.above;
        }
        if (bin >= 0) {
            tau = row.template border<true>([&](float l) { return takes(l) && t_of(l) == bin; }, mass, want, above, &above, &inside);
            const uint64_t each = mass(tau);
            ties = 1;
            if (inside > each) ties = (want - above + each - 1) / each;  // (dear: not where there are no equal ones)
            if (ties * each >= inside) ties = ~0ull;
        } else {  // among the equals
            const uint64_t each = mass(tau);
            ties = min(ties, (want - all + each - 1) / each);
        }
    }
    int last = a.V;  // the index of the last kept one at tau
    uint64_t total, value;
    if (ties != ~0ull) {
        const int i = row.walk([](float, float) { return Two{1, 1}; }, [&](int, float l, uint64_t) { return l == tau; },
                               [&](uint64_t) { return ties; }, &total, &value);
        last = (int)__reduce_max_sync(~0u, (uint32_t)row.tell((uint64_t)(i + 1), 0).x) - 1;
    }
    const int i = row.walk([&](float x, float y) { return weigh(x, y, sc, s.table); }, [&](int at, float l, uint64_t v) {
        return (l > tau || (l == tau && at <= last)) && v >= floor_w;
    }, [&](uint64_t sum) { return taken(sum, u); }, &total, &value);
    if (i >= 0 && threadIdx.x == 0) {
        a.ids[c] = i;
        if (a.probs) a.probs[c] = (float)((double)value / (double)total);
    }
}

template <typename T, int N>
cudaError_t launch_part(const Sample &a, int blocks, cudaStream_t s) {
    constexpr int kSmem = sizeof(Shared) + N * kSampleThreads * (sizeof(float) + sizeof(uint16_t));
    cudaError_t e = cudaFuncSetAttribute(k_sample<T, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess && blocks > 8)
        e = cudaFuncSetAttribute(k_sample<T, N>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)a.n);
    cfg.blockDim = dim3(kSampleThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)blocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_sample<T, N>, a);
}

template <typename T>
cudaError_t launch(const Sample &a, cudaStream_t s) {
    // Few rows: many blocks each, for the shortest call.  Many: few blocks each, as those of a row wait for one another
    // (256 rows of 129,280 logits of all kinds: eight blocks a row 215 us, four 149, before few
    // were settled by one block; two blocks of 512 threads an SM, eight a row, were no faster than four).
    const int least = a.n <= 8 ? 8 : a.n <= 24 ? 16 : 32;  // logits a thread, where a row is long enough
    int n = 8, blocks = 1;
    while (n * blocks * kSampleThreads < a.V) {
        if (n < least || blocks == kMaxBlocks) n *= 2;
        else blocks *= 2;
    }
    return n == 8 ? launch_part<T, 8>(a, blocks, s) : n == 16 ? launch_part<T, 16>(a, blocks, s) : launch_part<T, 32>(a, blocks, s);
}
static_assert(CBQ_SAMPLE_MAX_V <= kMaxBlocks * 32 * kSampleThreads, "the longest row fits a cluster");

}  // namespace

cudaError_t launch_sample(const Sample &a, cudaStream_t s) {
    if (a.dtype == CBQ_F32) return launch<float>(a, s);
    if (a.dtype == CBQ_BF16) return launch<__nv_bfloat16>(a, s);
    return launch<__half>(a, s);
}

}  // namespace cbq
