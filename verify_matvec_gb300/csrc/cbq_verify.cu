// cbq_verify.cu -- verification of drafted trees against the target's and the
// drafter's probabilities, by given random numbers.
//
// The walk itself is a chain of a few numbers a draft: the children of the node
// it has reached are tried in turn (a child's parent is before it, so one look
// at each draft in the order of the indices is the whole walk), and only a
// refused child of a drawn draft and the last token need a pass over a row:
//   sum_x r(x),  r(x) = max(p(x) - c q(x), 0).
// A cluster of blocks takes a sequence, each a stretch of the vocabulary and
// each of its warps a stretch of that; all of them walk alike, with the same
// sums, and only those are exchanged.  The last pass leaves every warp's sum
// behind, so that the drawn token lies in one warp's stretch, which that warp
// goes through once more.
//
// What a sum can hide decides here (a token is the answer or it is not), so
// terms and sums are pairs of fp32 numbers, some 2^-48 of their size off: 64-bit
// arithmetic is a sixty-fourth as wide on this GPU and would be the bound, pairs
// cost 20 instructions a token and are not.
#include <algorithm>

#include "cbq_device.cuh"
#include "step/cbq_launch.cuh"
#include "step/cbq_step.h"

namespace cbq {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMost = 16;    // blocks of a cluster
constexpr int kTile = 128;   // tokens that a warp takes at a time, four a lane side by side

// Numbers as two, two at a time: v = hi + lo, |lo| at most half a unit of hi's
// last place.  A packed instruction does the arithmetic of both.
struct Pairs {
    float2 hi, lo;
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 less(float2 a, float2 b) { return __ffma2_rn(b, both(-1.0f), a); }  // a - b
__device__ __forceinline__ void add(Pairs &s, Pairs x) {
    const float2 t = __fadd2_rn(s.hi, x.hi), z = less(t, s.hi);
    s.lo = __fadd2_rn(s.lo, __fadd2_rn(__fadd2_rn(less(s.hi, less(t, z)), less(x.hi, z)), x.lo));
    s.hi = t;
}

// What is left of p at two tokens: max(p - c q, 0), c = ch + cl; NaN gives 0.
template <bool kOne>  // c is 1
__device__ __forceinline__ Pairs left_of(float2 p, float2 q, float ch, float cl) {
    const float2 h = kOne ? q : __fmul2_rn(q, both(ch));
    const float2 t = less(p, h), z = less(t, p);
    float2 low = less(less(p, less(t, z)), __fadd2_rn(h, z));                                    // t + low = p - h
    if (!kOne) low = __ffma2_rn(q, both(-cl), __fadd2_rn(low, __ffma2_rn(q, both(-ch), h)));     // h + the rest = ch q
    auto kept = [](float t, float low) { return t > 0.0f ? low : t == 0.0f ? fmaxf(low, 0.0f) : 0.0f; };
    return Pairs{make_float2(fmaxf(t.x, 0.0f), fmaxf(t.y, 0.0f)), make_float2(kept(t.x, low.x), kept(t.y, low.y))};
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// v at p's place in block r's shared memory.
__device__ __forceinline__ void peer_store(double *p, uint32_t r, double v) {
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.f64 [a], %2;\n}\n" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(p)), "r"(r), "d"(v) : "memory");
}

struct Shared {
    float u[CBQ_TREE_MAX], p[CBQ_TREE_MAX], q[CBQ_TREE_MAX];  // of each draft: its number, and its token's probabilities at its parent
    int token[CBQ_TREE_MAX], parent[CBQ_TREE_MAX], path[CBQ_TREE_MAX];
    int gone[CBQ_TREE_MAX];          // chosen drafts: the tokens taken out at this node
    double warp[kWarps];             // sums of the warps' stretches
    double blocks[2][kMost];         // and of the blocks', of two passes in turn
    double tiles[kWarps];            // of the owner's tiles
    double c, left, goal;
    float ch, cl;                    // c as two
    int at, n_gone, next, count, owner, hit;
    bool draws, summed, some;        // the walk has ended; the sums at hand are those of this node and c; they are not zero
};

// The walk from draft s.next on, up to where it needs a pass over a row; by one
// thread of a block.  (The sums that a draw needs are there already if the last
// child was refused: then its pass was the last.)
template <bool kDrawn>
__device__ void walk(Shared &s, int n) {
    double c = s.c, left = s.left;
    int at = s.at, i = s.next;
    for (; i < n; ++i) {
        if (s.parent[i] != at) continue;
        const double p = s.p[i], q = s.q[i], u = s.u[i];
        double rest = p;
        if (kDrawn) {
            rest = p - c * q;
        } else {
            for (int k = 0; k < s.n_gone; ++k)
                if (s.gone[k] == s.token[i]) rest = 0.0;
        }
        if (u * q * left < rest) {
            s.path[s.count++] = at = i;
            c = 0.0, left = 1.0;
            s.n_gone = 0;
            s.summed = false;
        } else if (!kDrawn) {
            if (rest > 0.0) s.gone[s.n_gone++] = s.token[i], left -= rest;
        } else if (left > 0.0) {
            c += left;
            s.summed = false;
            ++i;
            break;
        }
    }
    s.c = c, s.left = left, s.at = at, s.next = i;
    s.ch = (float)c, s.cl = (float)(c - (double)s.ch);
    s.draws = kDrawn ? s.summed || c == 0.0 : true;
}

// Four tokens side by side, as r: those of this lane of tile t of a row.
template <bool kDrawn, bool kVec>
struct Row {
    const float *p, *q;  // q null: c is 0
    int V;
    float ch, cl;
    __device__ __forceinline__ float4 load(const float *from, int t, int lane) const {
        const int i = t * kTile + lane * 4;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (kVec) {  // (every row then begins on 16 bytes, and has whole fours)
            if (i < V) v = *reinterpret_cast<const float4 *>(from + i);
        } else {
            if (i < V) v.x = from[i];
            if (i + 1 < V) v.y = from[i + 1];
            if (i + 2 < V) v.z = from[i + 2];
            if (i + 3 < V) v.w = from[i + 3];
        }
        return v;
    }
    __device__ __forceinline__ void rest(const Shared &s, int t, int lane, Pairs (&r)[2]) const {
        const float4 x = load(p, t, lane);
        const float2 a = make_float2(x.x, x.y), b = make_float2(x.z, x.w);
        if (kDrawn && q) {
            const float4 y = load(q, t, lane);
            const float2 c = make_float2(y.x, y.y), d = make_float2(y.z, y.w);
            if (ch == 1.0f && cl == 0.0f) r[0] = left_of<true>(a, c, ch, cl), r[1] = left_of<true>(b, d, ch, cl);
            else r[0] = left_of<false>(a, c, ch, cl), r[1] = left_of<false>(b, d, ch, cl);
        } else {
            // (NaN gives 0)
            r[0] = {make_float2(fmaxf(a.x, 0.0f), fmaxf(a.y, 0.0f)), make_float2(0.0f, 0.0f)};
            r[1] = {make_float2(fmaxf(b.x, 0.0f), fmaxf(b.y, 0.0f)), make_float2(0.0f, 0.0f)};
            if (!kDrawn) {
                for (int k = 0; k < s.n_gone; ++k) {
                    const int g = s.gone[k] - (t * kTile + lane * 4);
                    if (g == 0) r[0].hi.x = 0.0f;
                    if (g == 1) r[0].hi.y = 0.0f;
                    if (g == 2) r[1].hi.x = 0.0f;
                    if (g == 3) r[1].hi.y = 0.0f;
                }
            }
        }
    }
};

// The sum of a warp's numbers, by all its lanes.
__device__ __forceinline__ double warp_sum(Pairs s) {
    Pairs t = {make_float2(s.hi.x, 0.0f), make_float2(s.lo.x, 0.0f)};
    add(t, Pairs{make_float2(s.hi.y, 0.0f), make_float2(s.lo.y, 0.0f)});
#pragma unroll
    for (int o = 16; o; o >>= 1)
        add(t, Pairs{make_float2(__shfl_xor_sync(~0u, t.hi.x, o), 0.0f), make_float2(__shfl_xor_sync(~0u, t.lo.x, o), 0.0f)});
    return (double)t.hi.x + (double)t.lo.x;
}

// The token of a tile, by the warp that has it, at which the sum passes `goal`;
// the last with any weight where rounding leaves the goal behind it (-1: none).
__device__ __forceinline__ int pick(const Pairs (&r)[2], int t, int lane, double goal) {
    const float hi[4] = {r[0].hi.x, r[0].hi.y, r[1].hi.x, r[1].hi.y}, lo[4] = {r[0].lo.x, r[0].lo.y, r[1].lo.x, r[1].lo.y};
    double upto[4], sum = 0.0;
    int mine = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        upto[e] = sum += (double)hi[e] + (double)lo[e];
        if (hi[e] > 0.0f || lo[e] > 0.0f) mine = t * kTile + lane * 4 + e;
    }
    double scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double u = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += u;
    }
    const int last = (int)__reduce_max_sync(~0u, (unsigned)(mine + 1)) - 1;
    const unsigned past = __ballot_sync(~0u, scan > goal && mine >= 0);
    if (!past) return last;
    int token = mine;  // (rounding: the lane's last)
#pragma unroll
    for (int e = 3; e >= 0; --e)
        if (scan - sum + upto[e] > goal && (hi[e] > 0.0f || lo[e] > 0.0f)) token = t * kTile + lane * 4 + e;
    return __shfl_sync(~0u, token, __ffs(past) - 1);
}

// grid (1, blocks of the cluster, n_seq).
template <bool kDrawn, bool kVec>
__global__ void __launch_bounds__(kThreads, 2) k_verify(Verify a) {
    __shared__ Shared s;
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, seq = blockIdx.z, rank = blockIdx.y, blocks = gridDim.y;
    const int64_t b0 = a.start[seq], b1 = a.start[seq + 1];
    const bool inside = b0 >= 0 && b1 >= b0 && b1 <= a.total_tok;
    const int n = inside ? (int)min(b1 - b0, (int64_t)a.max_tok) : 0;
    if (rank == 0 && tid == 0 && a.err && (!inside || b1 - b0 > a.max_tok)) atomicOr(a.err, CBQ_DEVERR_BAD_LENGTH);
    int32_t *path = a.path + (int64_t)seq * a.max_tok;
    if (n == 0) {  // (for all blocks of the cluster)
        if (rank == 0) {
            for (int i = tid; i < a.max_tok; i += kThreads) path[i] = -1;
            if (tid == 0) a.count[seq] = 0, a.next[seq] = -1;
        }
        return;
    }
    cluster_arrive();
    if (tid < n) {
        const int token = a.tokens[b0 + tid], parent = a.parent[b0 + tid];
        const bool behind = tid > 0 && parent >= 0 && parent < tid, real = behind && token >= 0 && token < a.V;
        s.token[tid] = real ? token : -1;
        s.parent[tid] = behind ? parent : -1;
        s.u[tid] = a.u[b0 + tid];
        s.p[tid] = real ? a.probs[(b0 + parent) * a.probs_stride + token] : 0.0f;
        s.q[tid] = !kDrawn ? 1.0f : real ? a.draft[(b0 + parent) * a.draft_stride + token] : 0.0f;
    }
    if (tid == 0) {
        s.c = 0.0, s.left = 1.0, s.at = 0, s.next = 1, s.path[0] = 0, s.count = 1, s.n_gone = 0;
        s.summed = false;
    }
    __syncthreads();
    cluster_wait();  // every block of the cluster runs: its shared memory may be written

    const int tiles = (a.V + kTile - 1) / kTile, own = (tiles + blocks * kWarps - 1) / (blocks * kWarps);
    const int t0 = min((rank * kWarps + warp) * own, tiles), t1 = min(t0 + own, tiles);
    Row<kDrawn, kVec> row = {};
    row.V = a.V;
    int turn = 0;
    bool again = false;  // nothing was left: from p itself
    for (;;) {
        if (tid == 0) {
            if (again) s.ch = s.cl = 0.0f, s.n_gone = 0, s.summed = false;
            else walk<kDrawn>(s, n);
        }
        __syncthreads();
        const bool draws = s.draws;
        const int64_t r = b0 + s.at;
        row.p = a.probs + r * a.probs_stride;
        row.ch = s.ch;
        row.cl = s.cl;
        row.q = kDrawn && row.ch > 0.0f ? a.draft + r * a.draft_stride : nullptr;
        if (!s.summed) {
            turn ^= 1;  // (a buffer is written again two passes on: all have read it by then)
            Pairs sum = {};
#pragma unroll 4
            for (int t = t0; t < t1; ++t) {
                Pairs r[2];
                row.rest(s, t, lane, r);
                add(sum, r[0]);
                add(sum, r[1]);
            }
            const double of_warp = warp_sum(sum);
            if (lane == 0) s.warp[warp] = of_warp;
            __syncthreads();
            if (warp == 0) {
                double v = lane < kWarps ? s.warp[lane] : 0.0;
#pragma unroll
                for (int o = kWarps / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
                if (lane < blocks) peer_store(&s.blocks[turn][rank], lane, v);
            }
            cluster_arrive();
            cluster_wait();
        }
        // (what the walk and the draw go on with, in every block alike)
        if (tid == 0) {
            double total = 0.0;
            for (int o = 0; o < blocks; ++o) total += s.blocks[turn][o];
            s.left = total;
            s.some = total > 0.0;
            s.summed = true;
        }
        __syncthreads();
        if (!draws) continue;
        again = !again && !s.some && (row.ch > 0.0f || s.n_gone > 0);
        if (!again) break;
        __syncthreads();  // (all have read what the next round writes)
    }

    const bool some = s.some;
    if (rank == 0) {
        const int count = s.count;
        for (int i = tid; i < a.max_tok; i += kThreads) path[i] = i < count ? s.path[i] : -1;
        if (tid == 0) {
            a.count[seq] = count;
            if (!some) a.next[seq] = -1;
        }
    }
    if (!some) return;
    if (tid == 0) {
        const double goal = (double)fminf(fmaxf(a.u_next[seq], 0.0f), 1.0f - 0x1p-24f) * s.left;
        double before = 0.0;
        int o = 0;
        for (; o < blocks - 1 && !(goal < before + s.blocks[turn][o]); ++o) before += s.blocks[turn][o];
        int w = -1;
        if (o == rank) {
            int last = 0;
            for (int i = 0; i < kWarps && w < 0; ++i) {
                if (!(s.warp[i] > 0.0)) continue;
                last = i;
                if (goal < before + s.warp[i]) w = i;
                else before += s.warp[i];
            }
            if (w < 0) before -= s.warp[w = last];  // (rounding: the last with any weight)
        }
        s.owner = w;
        s.goal = goal - before;
    }
    __syncthreads();
    if (s.owner < 0) return;
    // the block shares out the tiles of the warp whose stretch it is
    const int o0 = min((rank * kWarps + s.owner) * own, tiles), o1 = min(o0 + own, tiles);
    double goal = s.goal;
    int last = -1;  // the last tile with any weight
    for (int base = o0; base < o1; base += kWarps) {
        const int t = base + warp;
        Pairs r[2] = {};
        if (t < o1) row.rest(s, t, lane, r);
        Pairs sum = r[0];
        add(sum, r[1]);
        const double of_tile = warp_sum(sum);
        if (lane == 0) s.tiles[warp] = of_tile;
        __syncthreads();
        int hit = -1;
        if (warp == 0) {  // (in each warp's own registers the same: one does it, and tells)
            double before = 0.0;
            for (int k = 0; k < kWarps && hit < 0; ++k) {
                if (!(s.tiles[k] > 0.0)) continue;
                last = base + k;
                if (goal < before + s.tiles[k]) hit = k;
                else before += s.tiles[k];
            }
            goal -= before;
            if (lane == 0) s.hit = hit, s.goal = goal;
        }
        __syncthreads();
        if (s.hit >= 0) {
            if (warp == s.hit) {
                const int token = pick(r, t, lane, s.goal);
                if (lane == 0) a.next[seq] = token;
            }
            return;
        }
        __syncthreads();  // (s.tiles and s.hit are written again)
    }
    if (warp == 0) {  // rounding: the last with any weight
        Pairs r[2] = {};
        if (last >= 0) row.rest(s, last, lane, r);
        const int token = pick(r, last, lane, 1e300);
        if (lane == 0) a.next[seq] = token;
    }
}

template <bool kDrawn, bool kVec>
cudaError_t launch(const Verify &a, cudaStream_t s) {
    // As many blocks as fit the GPU at a time, two an SM: a row's pass takes four of them 4 us, its exchange 1.
    const int64_t tiles = (a.V + kTile - 1) / kTile;
    int blocks = kMost;
    while (blocks > 1 && (blocks * (int64_t)a.n_seq > 2 * 152 || tiles < blocks * kWarps / 2)) blocks /= 2;
    if (blocks > 8) {
        const cudaError_t e = cudaFuncSetAttribute(k_verify<kDrawn, kVec>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    return launch_clusters(k_verify<kDrawn, kVec>, dim3(1, (unsigned)blocks, (unsigned)a.n_seq), blocks, kThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_verify(const Verify &a, cudaStream_t s) {
    const bool vec = reinterpret_cast<uintptr_t>(a.probs) % 16 == 0 && reinterpret_cast<uintptr_t>(a.draft) % 16 == 0 &&
                     (a.probs_stride | a.draft_stride | a.V) % 4 == 0;
    if (a.draft) return vec ? launch<true, true>(a, s) : launch<true, false>(a, s);
    return vec ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace cbq
