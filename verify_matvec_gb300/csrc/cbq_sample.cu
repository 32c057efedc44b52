// cbq_sample.cu -- one token from each row of logits: temperature, top-k,
// top-p and min-p, drawn by a given uniform number.
//
// A cluster of up to eight blocks takes a row: each brings its part of the
// logits into shared memory once, as integers in the logits' order, and every
// later step reads them there.  Nothing is sorted: what top-k and top-p keep
// is all above a border in the order and the first few equal to it, and the
// border is found by histograms (of counts for top-k, of weights for top-p)
// whose bins narrow down to one value.  Weights are whole numbers of 2^-45, so
// that their sums do not depend on the order of atomics and a choice is the
// same on every run.
#include "cbq_device.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

namespace {

constexpr int kSampleThreads = 512, kNumWarps = kSampleThreads / 32;
constexpr int kBins = 1024;
constexpr int kMaxBlocks = 8;             // of a cluster
constexpr int kTable = 256;               // steps of 2^(1/256) of the weights' table
constexpr uint64_t kOne = 1ull << 45;     // the weight 1
constexpr uint32_t kNone = 0x007FFFFFu;   // order of -inf: what is not above has no weight

// 2^(i/256) in units of 2^-45, from the eight square roots 2^(1/2) .. 2^(1/256).
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
        t.v[i] = (uint64_t)(p * (double)kOne + 0.5);
    }
    return t;
}
__device__ const PowTable kPow = make_table();

// Unsigned numbers in the order of the logits; NaN below all (0).  Adding
// zero makes -0 and +0 one value, as the order wants.
__device__ __forceinline__ uint32_t order_of(float l) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    if (l != l) return 0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
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
struct Scale {
    float top, hi, lo;  // hi + lo = log2(e) / T
};
__device__ __forceinline__ uint64_t weight(float l, const Scale &s, const uint64_t *table) {
    if (l == s.top) return kOne;  // +inf at the top too
    const float d = l - s.top;
    const float y = d * s.hi;
    if (!(y > -47.0f)) return 0;
    const float back = d + s.top;                       // two-sum: d + e is the exact difference
    const float e = (l - back) + ((back - d) - s.top);
    const float yl = __fmaf_rn(d, s.hi, -y) + __fmaf_rn(d, s.lo, e * s.hi);
    const float n = rintf(y * kTable);
    const float r = __fmaf_rn(n, -1.0f / kTable, y);  // exact: y and n/256 agree in their leading bits
    constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654323148236017e-9f;
    const float th = r * kLn2Hi;
    const float tl = __fmaf_rn(r, kLn2Hi, -th) + __fmaf_rn(r, kLn2Lo, yl * kLn2Hi);
    const float t = th + tl;
    const float quad = __fmaf_rn(t * t, __fmaf_rn(t, 1.0f / 6.0f, 0.5f), tl);
    constexpr float k40 = 1099511627776.0f;
    const int p = __float2int_rn(th * k40) + __float2int_rn(quad * k40);
    const int ni = (int)n;
    const uint64_t w = table[ni & (kTable - 1)];
    const int64_t more = (int64_t)(int32_t)(w >> 15) * p >> 25;
    const uint64_t full = w + (uint64_t)more;
    const int sh = -(ni >> 8);
    return sh > 46 ? 0 : (full + ((1ull << sh) >> 1)) >> sh;
}

// ------------------------------------------------------------- clusters ----

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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
__device__ __forceinline__ uint2 peer_load2(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

// A histogram: counts in part[0], or weights in their three 16-bit parts (a
// block adds fewer than 2^16 of them, so 32 bits hold each part's sum; 64-bit
// atomics on shared memory are loops).
struct Hist {
    uint32_t part[3][kBins];
};

struct alignas(16) Shared {
    uint64_t table[kTable];
    Hist hist[2];
    uint64_t swap[2][kMaxBlocks][2];  // what the blocks of the cluster tell one another
    uint64_t warp[kNumWarps];
    uint32_t key[kNumWarps], at[kNumWarps];
    uint64_t above, inside;
    int bin, index;
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
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

// One block's part of a row and its place in the cluster.
struct Part {
    Shared &s;
    const uint32_t *x;  // the order of the logits first .. first + len
    int first, len, blocks, rank;
    int turn = 0, use = 0;  // which of the two swap buffers and histograms is next

    // f(index in the part, order), a warp to a contiguous stretch
    template <typename F>
    __device__ void each(F f) const {
        const int per = (len + kNumWarps - 1) / kNumWarps, w = threadIdx.x / 32;
        const int end = min(len, (w + 1) * per);
#pragma unroll 4
        for (int i = w * per + threadIdx.x % 32; i < end; i += 32) f(i, x[i]);
    }

    // Every block gives two numbers (of its thread 0) and gets all blocks'.
    // A buffer is written again two calls later: all blocks have read it by then.
    __device__ const uint64_t (*tell(uint64_t a, uint64_t b))[2] {
        uint64_t(*to)[2] = s.swap[turn];
        turn ^= 1;
        if (threadIdx.x < (unsigned)blocks) {
            peer_store(peer(&to[rank][0], threadIdx.x), a);
            peer_store(peer(&to[rank][1], threadIdx.x), b);
        }
        cluster_sync();
        return to;
    }

    // The block's sum of v, in every thread.
    __device__ uint64_t block_sum(uint64_t v) {
        v = warp_sum(v);
        __syncthreads();
        if (threadIdx.x % 32 == 0) s.warp[threadIdx.x / 32] = v;
        __syncthreads();
        v = 0;
#pragma unroll
        for (int i = 0; i < kNumWarps; ++i) v += s.warp[i];
        return v;
    }

    // One step of a descent: bin_of(order) in [0, kBins), or -1 for what does
    // not take part, ascending as the order descends; value(order) is counted
    // (kWeights false: at most 1) or summed.  need(total): how much to take.
    // Finds the first bin with which that is reached: s.bin (-1: never),
    // s.above before it, s.inside in it.
    template <bool kWeights, typename B, typename V, typename N>
    __device__ void step(B bin_of, V value, N need) {
        Hist &h = s.hist[use];  // last read two steps ago: a cluster barrier lies between
        use ^= 1;
        constexpr int kParts = kWeights ? 3 : 1;
        __syncthreads();  // s.bin of the step before has been read
        for (int i = threadIdx.x; i < kParts * kBins; i += kSampleThreads) h.part[0][i] = 0;
        if (threadIdx.x == 0) s.bin = -1;
        __syncthreads();
        each([&](int, uint32_t o) {
            const int b = bin_of(o);
            if (b < 0) return;
            if constexpr (kWeights) {
                const uint64_t v = value(o);
                if (!v) return;
                atomicAdd(&h.part[0][b], (uint32_t)v & 0xFFFFu);
                atomicAdd(&h.part[1][b], (uint32_t)(v >> 16) & 0xFFFFu);
                atomicAdd(&h.part[2][b], (uint32_t)(v >> 32));
            } else {
                atomicAdd(&h.part[0][b], 1u);
            }
        });
        cluster_sync();
        // every block adds up all blocks' bins (the same in each), two a thread
        uint64_t v0 = 0, v1 = 0;
        for (int r = 0; r < blocks; ++r)
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const uint2 u = peer_load2(peer(&h.part[p][2 * threadIdx.x], r));
                v0 += (uint64_t)u.x << (16 * p);
                v1 += (uint64_t)u.y << (16 * p);
            }
        const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
        uint64_t sum = warp_scan(v0 + v1, lane);
        if (lane == 31) s.warp[w] = sum;
        __syncthreads();
        uint64_t total = 0, before = 0;
#pragma unroll
        for (int i = 0; i < kNumWarps; ++i) {
            if (i < w) before += s.warp[i];
            total += s.warp[i];
        }
        sum += before;
        const uint64_t want = need(total), b0 = sum - v0 - v1, b1 = sum - v1;
        if (b0 < want && sum >= want) {
            const bool second = b1 < want;
            s.bin = 2 * threadIdx.x + (second ? 1 : 0);
            s.above = second ? b1 : b0;
            s.inside = second ? v1 : v0;
        }
        __syncthreads();
    }

    // The border of the row: the order's value at which `value` over what
    // takes(order) accepts, summed from the top, reaches need(total).  t_of
    // cuts the row into bins for a start (kept monotone by fp32's rounding);
    // then the bins are stretches of the integers, until one is left.
    // Returns false if it is never reached.  *above: the sum above the border
    // value; *inside: at it; *want: need(total).
    template <bool kWeights, typename A, typename V, typename N, typename B>
    __device__ bool border(A takes, V value, N need, B t_of, uint32_t *tau, uint64_t *above, uint64_t *inside,
                           uint64_t *want) {
        step<kWeights>([&](uint32_t o) { return takes(o) ? t_of(o) : -1; }, value,
                       [&](uint64_t total) { return *want = need(total); });
        const int first_bin = s.bin;
        if (first_bin < 0) return false;
        uint64_t up = s.above;
        *inside = s.inside;
        // the least and the greatest of the bin
        uint32_t lo = ~0u, hi = 0;
        each([&](int, uint32_t o) {
            if (takes(o) && t_of(o) == first_bin) lo = min(lo, o), hi = max(hi, o);
        });
        lo = __reduce_min_sync(~0u, lo);
        hi = __reduce_max_sync(~0u, hi);
        if (threadIdx.x % 32 == 0) s.key[threadIdx.x / 32] = lo, s.at[threadIdx.x / 32] = hi;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kNumWarps; ++i) lo = min(lo, s.key[i]), hi = max(hi, s.at[i]);
        const uint64_t(*all)[2] = tell(lo, hi);
        for (int r = 0; r < blocks; ++r) lo = min(lo, (uint32_t)all[r][0]), hi = max(hi, (uint32_t)all[r][1]);
        const uint64_t goal = *want;
        while (lo < hi) {
            const int sh = max(0, 32 - __clz(hi - lo) - 10);  // (hi - lo) >> sh is below kBins
            step<kWeights>([&](uint32_t o) { return takes(o) && o >= lo && o <= hi ? (int)((hi - o) >> sh) : -1; }, value,
                           [&](uint64_t) { return goal - up; });
            const uint32_t top = hi - ((uint32_t)s.bin << sh);
            const uint32_t low = top - lo < (1u << sh) ? lo : top - ((1u << sh) - 1);
            hi = top;
            lo = low;
            up += s.above;
            *inside = s.inside;
        }
        *tau = lo;
        *above = up;
        return true;
    }

    // The place in the part where `what`, summed in the order of the indices
    // over the whole row, reaches need; -1 in the blocks that do not hold it.
    // *total: the row's sum.  need(total) is asked once it is known.
    template <typename W, typename N>
    __device__ int walk(W what, N need, uint64_t *total) {
        const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
        uint64_t mine = 0;
        each([&](int i, uint32_t o) { mine += what(i, o); });
        mine = warp_sum(mine);
        const uint64_t block = block_sum(lane == 0 ? mine : 0);
        if (threadIdx.x == 0) s.index = -1;
        const uint64_t(*all)[2] = tell(block, 0);
        uint64_t before = 0, sum = 0;
        for (int r = 0; r < blocks; ++r) {
            if (r < rank) before += all[r][0];
            sum += all[r][0];
        }
        *total = sum;
        const uint64_t goal = need(sum);
        for (int i = 0; i < w; ++i) before += s.warp[i];
        if (before < goal && before + mine >= goal) {
            const int per = (len + kNumWarps - 1) / kNumWarps, end = min(len, (w + 1) * per);
            for (int i0 = w * per; i0 < end; i0 += 32) {
                const int i = i0 + lane;
                const uint64_t v = warp_scan(i < end ? what(i, x[i]) : 0, lane);
                const unsigned hit = __ballot_sync(~0u, before + v >= goal);
                if (hit) {
                    if (lane == 0) s.index = i0 + __ffs(hit) - 1;
                    break;
                }
                before += __shfl_sync(~0u, v, 31);
            }
        }
        __syncthreads();
        return s.index;
    }
};

// Values of type T from p on, n of them, as orders into to[]: 16 bytes a load
// where p is aligned, else one by one.
template <typename T>
__device__ __forceinline__ void bring(const T *p, int n, uint32_t *to) {
    constexpr int kVec = 16 / sizeof(T);
    int done = 0;
    if (reinterpret_cast<uintptr_t>(p) % 16 == 0) {
        done = n / kVec * kVec;
#pragma unroll 4
        for (int i = threadIdx.x * kVec; i < done; i += kSampleThreads * kVec) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p + i);
            const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
            for (int j = 0; j < kVec; j += 4)
                *reinterpret_cast<uint4 *>(to + i + j) = make_uint4(order_of(to_f32(e[j])), order_of(to_f32(e[j + 1])),
                                                                    order_of(to_f32(e[j + 2])), order_of(to_f32(e[j + 3])));
        }
    }
#pragma unroll 8
    for (int i = done + threadIdx.x; i < n; i += kSampleThreads) to[i] = order_of(to_f32(p[i]));
}

// grid (blocks of the cluster, rows); part: how many logits a block takes.
template <typename T>
__global__ void __launch_bounds__(kSampleThreads, 2) k_sample(Sample a, int part) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared &s = *reinterpret_cast<Shared *>(smem);
    uint32_t *x = reinterpret_cast<uint32_t *>(smem + sizeof(Shared));
    pdl_trigger();
    for (int i = threadIdx.x; i < kTable; i += kSampleThreads) s.table[i] = kPow.v[i];
    pdl_wait();
    const int c = blockIdx.y, lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const int first = blockIdx.x * part, len = max(0, min(part, a.V - first));
    Part row = {s, x, first, len, (int)gridDim.x, (int)cluster_rank()};
    const float temp = a.temperature ? a.temperature[c] : 1.0f, p = a.top_p ? a.top_p[c] : 1.0f;
    const float least = a.min_p ? a.min_p[c] : 0.0f, u = a.u[c];
    const int k = a.top_k ? a.top_k[c] : 0;
    bring(static_cast<const T *>(a.logits) + c * a.row_stride + first, len, x);
    cluster_sync();  // and every block of the cluster runs: its shared memory may be written

    // the first of the order
    uint32_t best = 0, at = 0;
    row.each([&](int i, uint32_t o) {
        if (o > best) best = o, at = (uint32_t)i;
    });
    const uint32_t warp_best = __reduce_max_sync(~0u, best);
    at = __reduce_min_sync(~0u, best == warp_best ? at : ~0u);
    if (lane == 0) s.key[w] = warp_best, s.at[w] = at;
    __syncthreads();
    best = 0, at = 0;
#pragma unroll
    for (int i = 0; i < kNumWarps; ++i)
        if (s.key[i] > best) best = s.key[i], at = s.at[i];
    {
        const uint64_t(*all)[2] = row.tell(best, (uint64_t)(first + at));
        best = 0, at = 0;
        for (int r = 0; r < row.blocks; ++r)
            if ((uint32_t)all[r][0] > best) best = (uint32_t)all[r][0], at = (uint32_t)all[r][1];
    }
    if (best <= kNone || !(temp > 0.0f)) {
        if (threadIdx.x == 0 && row.rank == 0) {
            a.ids[c] = best <= kNone ? -1 : (int)at;
            if (a.probs) a.probs[c] = best <= kNone ? 0.0f : 1.0f;
        }
        return;
    }
    const int top_at = (int)at;
    const double per = fmin(1.4426950408889634 / (double)temp, 1e30);
    Scale sc;
    sc.top = logit_of(best);
    sc.hi = (float)per;
    sc.lo = (float)(per - (double)sc.hi);

    // bins of 1/21 of a power of two of the weight; the last takes the rest
    const float cut = sc.hi * 21.0f;
    auto t_of = [&](uint32_t o) {
        return o == best ? 0 : min(__float2int_rz((sc.top - logit_of(o)) * cut), kBins - 1);
    };
    auto mass = [&](uint32_t o) { return weight(logit_of(o), sc, s.table); };
    uint32_t tau = kNone + 1;  // kept: above tau, and the first `ties` at it (all, if ~0)
    uint64_t ties = ~0ull, above, inside, want;
    if (k > 0 && k < a.V) {
        uint32_t to;
        if (row.border<false>([](uint32_t o) { return o > kNone; }, [](uint32_t) { return (uint64_t)1; },
                              [&](uint64_t) { return (uint64_t)k; }, t_of, &to, &above, &inside, &want)) {
            tau = to;
            ties = (uint64_t)k - above < inside ? (uint64_t)k - above : ~0ull;
        }
    }
    if (p < 1.0f) {
        // with a cut among the equals at tau, those weigh `ties` times one of them: the border is looked for above them
        const bool part_of = ties != ~0ull;
        const uint64_t rest = part_of ? ties * mass(tau) : 0;
        const uint32_t from = part_of ? tau + 1 : tau;
        uint64_t all = 0;  // the mass from there on
        auto goal = [&](uint64_t total) {
            all = total;
            const double g = ceil(fmax((double)p, 0.0) * (double)(total + rest));
            return g < 1.0 ? (uint64_t)1 : (uint64_t)g;
        };
        uint32_t to;
        if (row.border<true>([&](uint32_t o) { return o >= from; }, mass, goal, t_of, &to, &above, &inside, &want)) {
            const uint64_t one = mass(to);
            tau = to;
            ties = (want - above + one - 1) / one;
            if (ties * one >= inside) ties = ~0ull;
        } else {  // among the equals
            const uint64_t one = mass(tau);
            ties = min(ties, (want - all + one - 1) / one);
        }
    }
    int last = a.V;  // the index of the last kept one at tau
    if (ties != ~0ull) {
        uint64_t total;
        const int i = row.walk([&](int, uint32_t o) { return (uint64_t)(o == tau); }, [&](uint64_t) { return ties; }, &total);
        const uint64_t(*all)[2] = row.tell(i < 0 ? 0 : (uint64_t)(first + i) + 1, 0);
        uint64_t got = 0;
        for (int r = 0; r < row.blocks; ++r) got = max(got, all[r][0]);
        last = (int)got - 1;
    }
    const double floor_w = (double)least * (double)kOne;
    const float floor_y = least > 0.0f ? log2f(least) - 0.01f : -INFINITY;  // surely below: not weighed
    auto kept = [&](int i, uint32_t o) -> uint64_t {
        if (o < tau || (o == tau && first + i > last)) return 0;
        if ((logit_of(o) - sc.top) * sc.hi < floor_y && o != best) return 0;
        const uint64_t v = mass(o);
        return (double)v >= floor_w || !(floor_w > 0.0) || first + i == top_at ? v : 0;
    };
    uint64_t total;
    const int i = row.walk(kept, [&](uint64_t sum) {
        const uint64_t g = (uint64_t)(fmin(fmax((double)u, 0.0), 1.0) * (double)sum) + 1;
        return g < sum ? g : sum;
    }, &total);
    if (i >= 0 && threadIdx.x == 0) {
        a.ids[c] = first + i;
        if (a.probs) a.probs[c] = (float)((double)kept(i, x[i]) / (double)total);
    }
}

template <typename T>
cudaError_t launch(const Sample &a, cudaStream_t s) {
    // blocks of a row: more of them for a longer row, up to the portable eight
    const int blocks = a.V <= 4096 ? 1 : a.V <= 16384 ? 2 : a.V <= 49152 ? 4 : 8;
    const int part = ((a.V + blocks - 1) / blocks + 7) / 8 * 8;  // whole vectors, so each part is aligned as the row is
    const size_t smem = sizeof(Shared) + (size_t)part * sizeof(uint32_t);
    cudaError_t e = cudaFuncSetAttribute(k_sample<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)a.n);
    cfg.blockDim = dim3(kSampleThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)blocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_sample<T>, a, part);
}

}  // namespace

cudaError_t launch_sample(const Sample &a, cudaStream_t s) {
    if (a.dtype == CBQ_F32) return launch<float>(a, s);
    if (a.dtype == CBQ_BF16) return launch<__nv_bfloat16>(a, s);
    return launch<__half>(a, s);
}

}  // namespace cbq
