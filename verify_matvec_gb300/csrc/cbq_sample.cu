// cbq_sample.cu -- one token from each row of logits: temperature, top-k,
// top-p and min-p, drawn by a given uniform number.
#include "cbq_device.cuh"
#include "step/cbq_step.h"
#include "step/cbq_types.cuh"

namespace cbq {

namespace {

constexpr int kSampleThreads = 1024, kNumWarps = kSampleThreads / 32;
constexpr int kTable = 256;               // steps of 2^(1/256) of the weights' table
constexpr uint64_t kOne = 1ull << 45;     // the weight 1
constexpr uint32_t kNone = 0x007FFFFFu;   // order of -inf: what is not above has no weight

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
// polynomial (the method of P. T. P. Tang, ACM TOMS 15, 1989).  With y = (l - top) *
// log2(e)/T carried as two fp32 numbers (about 2^-44 of |y| <= 46), n =
// round(256 y) and t = (y - n/256) ln 2, |t| <= 2^-9.5: the weight is
// table[n mod 256] * (1 + (t + t^2/2 + t^3/6)) >> -floor(n/256); 1 + .. is a
// 2^-40 fixed-point number, whose rounding (2^-41) is the largest error.
struct Scale {
    float top, hi, lo;  // hi + lo = log2(e) / T
};
__device__ __forceinline__ uint64_t weight(float l, const Scale &s, const uint64_t *table) {
    if (l == s.top) return kOne;  // +inf at the top too
    const float d = l - s.top;
    const float back = d + s.top;                       // two-sum: d + e is the exact difference
    const float e = (l - back) + ((back - d) - s.top);
    const float y = d * s.hi;
    if (!(y > -47.0f)) return 0;
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

struct Shared {
    uint64_t table[kTable];
    uint64_t hist[256];
    uint64_t part[kNumWarps];
    uint32_t top[kNumWarps];
    uint32_t top_at[kNumWarps];
    uint64_t value;
    uint32_t digit;
    int index;
};

template <typename T>
struct Row {
    const T *x;
    int V;
    // f(index, logit) over the row, a warp to a contiguous part of it
    template <typename F>
    __device__ void part(F f) const {
        const int per = (V + kNumWarps - 1) / kNumWarps, w = threadIdx.x / 32;
        const int end = min(V, (w + 1) * per);
        for (int i = w * per + threadIdx.x % 32; i < end; i += 32) f(i, to_f32(x[i]));
    }
};

__device__ __forceinline__ uint64_t warp_sum(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
    return v;
}

// Finds, in the order of the row, the place where `what` summed from the top
// reaches `need`: the order's value *tau there and what is above it (returned).
template <typename T, typename F>
__device__ uint64_t descend(const Row<T> &row, Shared &s, uint64_t need, uint32_t *tau, F what) {
    uint32_t prefix = 0;
    uint64_t above = 0;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kSampleThreads) s.hist[i] = 0;
        __syncthreads();
        row.part([&](int, float l) {
            const uint32_t o = order_of(l);
            if (o <= kNone || (shift < 24 && (o ^ prefix) >> (shift + 8))) return;
            const uint64_t v = what(o, l);
            if (v) atomicAdd(reinterpret_cast<unsigned long long *>(&s.hist[o >> shift & 255]), (unsigned long long)v);
        });
        __syncthreads();
        if (threadIdx.x == 0) {
            uint64_t sum = above;
            int d = 255;
            for (; d > 0 && sum + s.hist[d] < need; --d) sum += s.hist[d];
            s.value = sum;
            s.digit = (uint32_t)d;
        }
        __syncthreads();
        above = s.value;
        prefix |= s.digit << shift;
        __syncthreads();
    }
    *tau = prefix;
    return above;
}

// The index where `what`, summed in the order of the indices, reaches need
// (V - 1 if it never does).
template <typename T, typename F>
__device__ int walk(const Row<T> &row, Shared &s, uint64_t need, F what) {
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
    uint64_t mine = 0;
    row.part([&](int i, float l) { mine += what(i, l); });
    mine = warp_sum(mine);
    if (lane == 0) s.part[w] = mine;
    if (threadIdx.x == 0) s.index = row.V - 1;
    __syncthreads();
    uint64_t before = 0;
    for (int i = 0; i < w; ++i) before += s.part[i];
    if (before < need && before + mine >= need) {
        const int per = (row.V + kNumWarps - 1) / kNumWarps, end = min(row.V, (w + 1) * per);
        for (int i0 = w * per; i0 < end; i0 += 32) {
            const int i = i0 + lane;
            uint64_t v = i < end ? what(i, to_f32(row.x[i])) : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint64_t u = __shfl_up_sync(~0u, v, o);
                if (lane >= o) v += u;
            }
            const unsigned hit = __ballot_sync(~0u, before + v >= need);
            if (hit) {
                if (lane == 0) s.index = i0 + __ffs(hit) - 1;
                break;
            }
            before += __shfl_sync(~0u, v, 31);
        }
    }
    __syncthreads();
    const int at = s.index;
    __syncthreads();
    return at;
}

template <typename T>
__global__ void __launch_bounds__(kSampleThreads) k_sample(Sample a) {
    __shared__ Shared s;
    pdl_trigger();
    pdl_wait();
    const int c = blockIdx.x, lane = threadIdx.x % 32, w = threadIdx.x / 32;
    const Row<T> row = {static_cast<const T *>(a.logits) + c * a.row_stride, a.V};

    // the first of the order
    uint32_t best = 0, at = 0;
    row.part([&](int i, float l) {
        const uint32_t o = order_of(l);
        if (o > best) best = o, at = (uint32_t)i;
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const uint32_t b = __shfl_xor_sync(~0u, best, o), i = __shfl_xor_sync(~0u, at, o);
        if (b > best || (b == best && i < at)) best = b, at = i;
    }
    if (lane == 0) s.top[w] = best, s.top_at[w] = at;
    for (int i = threadIdx.x; i < kTable; i += kSampleThreads) s.table[i] = (uint64_t)llrint(exp2((double)i / kTable) * (double)kOne);
    __syncthreads();
    for (int i = 0; i < kNumWarps; ++i) {
        const uint32_t b = s.top[i];
        if (b > best || (b == best && s.top_at[i] < at)) best = b, at = s.top_at[i];
    }
    const float temp = a.temperature ? a.temperature[c] : 1.0f;
    if (best <= kNone || !(temp > 0.0f)) {
        if (threadIdx.x == 0) {
            a.ids[c] = best <= kNone ? -1 : (int)at;
            if (a.probs) a.probs[c] = best <= kNone ? 0.0f : 1.0f;
        }
        return;
    }
    const int first = (int)at;
    const double per = fmin(1.4426950408889634 / (double)temp, 1e30);
    Scale sc;
    sc.top = logit_of(best);
    sc.hi = (float)per;
    sc.lo = (float)(per - (double)sc.hi);
    const int k = a.top_k ? a.top_k[c] : 0;
    const float p = a.top_p ? a.top_p[c] : 1.0f, least = a.min_p ? a.min_p[c] : 0.0f;

    uint32_t tau = kNone + 1;      // kept: above tau, and the first `ties` at it
    uint64_t ties = ~0ull;
    auto mass = [&](uint32_t, float l) { return weight(l, sc, s.table); };
    if (k > 0 && k < a.V) {
        const uint64_t above = descend(row, s, (uint64_t)k, &tau, [](uint32_t, float) { return (uint64_t)1; });
        ties = (uint64_t)k - above;
        if (tau <= kNone) tau = kNone + 1, ties = ~0ull;
    }
    if (p < 1.0f) {
        // the mass of what top-k keeps: all above tau, and `ties` times the weight at it
        uint64_t sum = 0, same = 0;
        row.part([&](int, float l) {
            const uint32_t o = order_of(l);
            if (o <= kNone || o < tau) return;
            if (o == tau) ++same;
            else sum += weight(l, sc, s.table);
        });
        sum = warp_sum(sum);
        same = warp_sum(same);
        if (lane == 0) s.part[w] = sum, s.hist[w] = same;
        __syncthreads();
        sum = same = 0;
        for (int i = 0; i < kNumWarps; ++i) sum += s.part[i], same += s.hist[i];
        __syncthreads();
        if (same < ties) ties = same;
        const uint64_t all = sum + ties * weight(logit_of(tau), sc, s.table);
        const double want = ceil(fmax((double)p, 0.0) * (double)all);
        const uint64_t need = want < 1.0 ? 1 : (uint64_t)want;
        const uint32_t from = tau;
        uint32_t to;
        const uint64_t before = descend(row, s, need, &to, [&](uint32_t o, float l) {
            return o > from ? weight(l, sc, s.table) : (uint64_t)0;
        });
        // past everything above `from`: the border is among the ties at `from`
        if (to < from) to = from;
        const uint64_t over = to == from ? sum : before;
        const uint64_t one = weight(logit_of(to), sc, s.table);
        const uint64_t m = one ? (need - over + one - 1) / one : ~0ull;
        if (to != from || m < ties) ties = m;
        tau = to;
    }
    int last = a.V;
    if (ties != ~0ull) last = walk(row, s, ties, [&](int, float l) { return (uint64_t)(order_of(l) == tau); });
    const double floor_w = (double)least * (double)kOne;
    auto kept = [&](int i, float l) -> uint64_t {
        const uint32_t o = order_of(l);
        if (o <= kNone || o < tau || (o == tau && i > last)) return 0;
        const uint64_t x = weight(l, sc, s.table);
        return (double)x >= floor_w || !(floor_w > 0.0) || i == first ? x : 0;
    };
    uint64_t sum = 0;
    row.part([&](int i, float l) { sum += kept(i, l); });
    sum = warp_sum(sum);
    if (lane == 0) s.part[w] = sum;
    __syncthreads();
    sum = 0;
    for (int i = 0; i < kNumWarps; ++i) sum += s.part[i];
    __syncthreads();
    const double u = fmin(fmax((double)a.u[c], 0.0), 1.0);
    uint64_t need = (uint64_t)(u * (double)sum) + 1;
    if (need > sum) need = sum;
    const int id = walk(row, s, need, kept);
    if (threadIdx.x == 0) {
        a.ids[c] = id;
        if (a.probs) a.probs[c] = (float)((double)kept(id, to_f32(row.x[id])) / (double)sum);
    }
}

}  // namespace

cudaError_t launch_sample(const Sample &a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.n);
    cfg.blockDim = dim3(kSampleThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (a.dtype == CBQ_F32) return cudaLaunchKernelEx(&cfg, k_sample<float>, a);
    if (a.dtype == CBQ_BF16) return cudaLaunchKernelEx(&cfg, k_sample<__nv_bfloat16>, a);
    return cudaLaunchKernelEx(&cfg, k_sample<__half>, a);
}

}  // namespace cbq
