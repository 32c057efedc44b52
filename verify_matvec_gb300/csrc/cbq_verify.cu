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
// cost some 15 instructions a token and are near it.
//
// 64 binary trees of 12 over 129,280 tokens, with a drafter near the target, take
// 32 us with warm caches (the slowest of them four passes, each some 10,000 clocks
// of loads and sums in a quarter of the row, 3,000 of exchange and 2,000 of walk,
// and a draw of 6,000), 200 of 6 58 us, one of 5 7 us; trees of up to 12 whose
// drafter is farther off, and refused more often, 41, and 49 cold: latencies, with
// issue slots 15% and memory 15% busy.  (With two tiles less ahead where only p is
// read, and three operations a pair of tokens more in the differences, the 32 us
// were 37; with bulk copies into a ring of each warp's own, of 1 KB, 46.)
#include <algorithm>

#include "cbq_device.cuh"
#include "step/cbq_launch.cuh"
#include "step/cbq_step.h"

namespace cbq {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMost = 16;    // blocks of a cluster
constexpr int kTile = 128;   // tokens that a warp takes at a time, four a lane side by side

// A number as two: v = hi + lo, |lo| at most half a unit of hi's last place.
struct alignas(8) Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair normal(float hi, float lo) {  // |lo| is small beside hi
    const float s = hi + lo;
    return Pair{s, lo - (s - hi)};
}
__device__ __forceinline__ Pair plus(Pair a, Pair b) {
    const float s = a.hi + b.hi, z = s - a.hi;
    return normal(s, ((a.hi - (s - z)) + (b.hi - z)) + (a.lo + b.lo));
}
__device__ __forceinline__ Pair minus(Pair a, Pair b) { return plus(a, Pair{-b.hi, -b.lo}); }
__device__ __forceinline__ Pair times(Pair a, Pair b) {
    const float h = a.hi * b.hi, e = __fmaf_rn(a.hi, b.hi, -h);
    return normal(h, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.lo, e)));
}
__device__ __forceinline__ bool under(Pair a, Pair b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ bool some(Pair a) { return a.hi > 0.0f || (a.hi == 0.0f && a.lo > 0.0f); }

// The same, two at a time: a packed instruction does the arithmetic of both.
struct Pairs {
    float2 hi, lo;
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 less(float2 a, float2 b) { return __ffma2_rn(b, both(-1.0f), a); }  // a - b
__device__ __forceinline__ void add(Pairs &s, float2 x) {
    const float2 t = __fadd2_rn(s.hi, x), z = less(t, s.hi);
    s.lo = __fadd2_rn(s.lo, __fadd2_rn(less(s.hi, less(t, z)), less(x, z)));
    s.hi = t;
}
__device__ __forceinline__ void add(Pairs &s, Pairs x) {
    const float2 t = __fadd2_rn(s.hi, x.hi), z = less(t, s.hi);
    s.lo = __fadd2_rn(s.lo, __fadd2_rn(__fadd2_rn(less(s.hi, less(t, z)), less(x.hi, z)), x.lo));
    s.hi = t;
}

// NaN in a row, and what is below 0, count as 0.
__device__ __forceinline__ float number(float x) { return fmaxf(x, 0.0f); }

// What is left of p at two tokens: max(p - c q, 0), c = ch + cl; NaN in p gives 0, q has none.
// Only where c q <= p does the rounding of the difference count, and there it is
// (p - t) - c q.
template <bool kOne>  // c is 1
__device__ __forceinline__ Pairs left_of(float2 p, float2 q, float ch, float cl) {
    if (kOne) {  // p less the smaller of the two
        p = make_float2(fmaxf(p.x, 0.0f), fmaxf(p.y, 0.0f));
        q = make_float2(fminf(p.x, q.x), fminf(p.y, q.y));
        const float2 t = less(p, q);
        return Pairs{t, less(less(p, t), q)};
    }
    const float2 h = __fmul2_rn(q, both(ch)), t = less(p, h);
    // t + low = p - h, h + the rest = ch q
    const float2 low = __ffma2_rn(q, both(-cl), __fadd2_rn(less(less(p, t), h), __ffma2_rn(q, both(-ch), h)));
    auto kept = [](float t, float low) { return t > 0.0f ? low : t == 0.0f ? fmaxf(low, 0.0f) : 0.0f; };
    return Pairs{make_float2(fmaxf(t.x, 0.0f), fmaxf(t.y, 0.0f)), make_float2(kept(t.x, low.x), kept(t.y, low.y))};
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// v at p's place in block r's shared memory.
__device__ __forceinline__ void peer_store(Pair *p, uint32_t r, Pair v) {
    asm volatile("{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %0, %1;\n st.shared::cluster.v2.f32 [a], {%2, %3};\n}\n" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(p)), "r"(r), "f"(v.hi), "f"(v.lo) : "memory");
}

struct Shared {
    float u[CBQ_TREE_MAX], p[CBQ_TREE_MAX], q[CBQ_TREE_MAX];  // of each draft: its number, and its token's probabilities at its parent
    int token[CBQ_TREE_MAX], parent[CBQ_TREE_MAX], path[CBQ_TREE_MAX];
    int gone[CBQ_TREE_MAX];          // chosen drafts: the tokens taken out at this node
    Pair warp[kWarps];               // sums of the warps' stretches
    Pair blocks[2][kMost];           // and of the blocks', of two passes in turn
    Pair tiles[kWarps];              // of the owner's tiles
    Pair c, left, goal;
    float u_next;
    int at, n_gone, next, count, owner, hit;
    bool draws, summed, some;        // the walk has ended; the sums at hand are those of this node and c; they are not zero
};

// The walk from draft s.next on, up to where it needs a pass over a row; by one
// thread of a block.  (The sums that a draw needs are there already if the last
// child was refused: then its pass was the last.)
template <bool kDrawn>
__device__ void walk(Shared &s, int n) {
    Pair c = s.c, left = s.left;
    int at = s.at, i = s.next;
    for (; i < n; ++i) {
        if (s.parent[i] != at) continue;
        const Pair p = {s.p[i], 0.0f}, q = {s.q[i], 0.0f}, u = {s.u[i], 0.0f};
        Pair rest = p;
        if (kDrawn) {
            rest = minus(p, times(c, q));
        } else {
            for (int k = 0; k < s.n_gone; ++k)
                if (s.gone[k] == s.token[i]) rest = {0.0f, 0.0f};
        }
        if (under(times(times(u, q), left), rest)) {
            s.path[s.count++] = at = i;
            c = {0.0f, 0.0f}, left = {1.0f, 0.0f};
            s.n_gone = 0;
            s.summed = false;
        } else if (!kDrawn) {
            if (some(rest)) s.gone[s.n_gone++] = s.token[i], left = minus(left, rest);
        } else if (some(left)) {
            c = plus(c, left);
            s.summed = false;
            ++i;
            break;
        }
    }
    s.c = c, s.left = left, s.at = at, s.next = i;
    s.draws = kDrawn ? s.summed || c.hi == 0.0f : true;
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
    struct Tile {
        float4 p, q;
    };
    __device__ __forceinline__ Tile load(int t, int lane) const {
        return Tile{load(p, t, lane), kDrawn && q ? load(q, t, lane) : make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
    }
    __device__ __forceinline__ void rest(const Shared &s, int t, int lane, const Tile &x, Pairs (&r)[2]) const {
        const float2 a = make_float2(x.p.x, x.p.y), b = make_float2(x.p.z, x.p.w);
        if (kDrawn && q) {
            const float2 c = make_float2(number(x.q.x), number(x.q.y)), d = make_float2(number(x.q.z), number(x.q.w));
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

// The sums of a lane's tokens of tiles t0 .. t1 - 1: kAhead tiles are worked on
// while the next as many are on their way.
template <int kAhead, bool kBoth, bool kDrawn, bool kVec>
__device__ __forceinline__ void sum_of(const Row<kDrawn, kVec> &row, const Shared &s, int t0, int t1, int tiles, int lane, Pairs &sum) {
    float4 p[2][kAhead], q[2][kAhead];
    auto take = [&](int to, int t) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int i = t + j < t1 ? t + j : tiles;  // (past the end: zeros)
            p[to][j] = row.load(row.p, i, lane);
            if (kBoth) q[to][j] = row.load(row.q, i, lane);
        }
    };
    take(0, t0);
    for (int t = t0; t < t1; t += kAhead) {
        take(1, t + kAhead);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            Pairs r[2];
            row.rest(s, t + j, lane, {p[0][j], kBoth ? q[0][j] : float4{}}, r);
            if (kBoth) add(sum, r[0]), add(sum, r[1]);
            else add(sum, r[0].hi), add(sum, r[1].hi);
            p[0][j] = p[1][j];
            if (kBoth) q[0][j] = q[1][j];
        }
    }
}

// The sum of a warp's numbers, by all its lanes.
__device__ __forceinline__ Pair warp_sum(Pairs s) {
    Pair t = plus(Pair{s.hi.x, s.lo.x}, Pair{s.hi.y, s.lo.y});
#pragma unroll
    for (int o = 16; o; o >>= 1) t = plus(t, Pair{__shfl_xor_sync(~0u, t.hi, o), __shfl_xor_sync(~0u, t.lo, o)});
    return t;
}
// Inclusive sums over the lanes of a warp.
__device__ __forceinline__ Pair scan(Pair v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Pair u = {__shfl_up_sync(~0u, v.hi, o), __shfl_up_sync(~0u, v.lo, o)};
        if (lane >= o) v = plus(u, v);
    }
    return v;
}
// The first lane whose inclusive sum passes goal, of those with any weight; the
// last of them where rounding leaves the goal behind.  *before: the sum before it.
__device__ __forceinline__ int first_past(Pair upto, bool any, Pair goal, int lane, Pair *before) {
    const unsigned have = __ballot_sync(~0u, any), past = __ballot_sync(~0u, any && under(goal, upto));
    const int l = past ? __ffs(past) - 1 : have ? 31 - __clz(have) : 0;
    const Pair ahead = {__shfl_up_sync(~0u, upto.hi, 1), __shfl_up_sync(~0u, upto.lo, 1)};
    *before = {__shfl_sync(~0u, lane ? ahead.hi : 0.0f, l), __shfl_sync(~0u, lane ? ahead.lo : 0.0f, l)};
    return l;
}

// The token of a tile, by the warp that has it, at which the sum passes `goal`;
// the last with any weight where rounding leaves the goal behind it (-1: none).
__device__ __forceinline__ int pick(const Pairs (&r)[2], int t, int lane, Pair goal) {
    const Pair v[4] = {{r[0].hi.x, r[0].lo.x}, {r[0].hi.y, r[0].lo.y}, {r[1].hi.x, r[1].lo.x}, {r[1].hi.y, r[1].lo.y}};
    Pair upto[4];
    int mine = -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        upto[e] = e ? plus(upto[e - 1], v[e]) : normal(v[0].hi, v[0].lo);
        if (some(v[e])) mine = t * kTile + lane * 4 + e;
    }
    const Pair all = scan(upto[3], lane);
    const int last = (int)__reduce_max_sync(~0u, (unsigned)(mine + 1)) - 1;
    const unsigned past = __ballot_sync(~0u, under(goal, all) && mine >= 0);
    if (!past) return last;
    const Pair ahead = {__shfl_up_sync(~0u, all.hi, 1), __shfl_up_sync(~0u, all.lo, 1)};
    int token = mine;  // (rounding: the lane's last)
#pragma unroll
    for (int e = 3; e >= 0; --e)
        if (under(goal, lane ? plus(ahead, upto[e]) : upto[e]) && some(v[e])) token = t * kTile + lane * 4 + e;
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
        s.p[tid] = real ? number(a.probs[(b0 + parent) * a.probs_stride + token]) : 0.0f;
        s.q[tid] = !kDrawn ? 1.0f : real ? number(a.draft[(b0 + parent) * a.draft_stride + token]) : 0.0f;
    }
    if (tid == 0) {
        s.u_next = fminf(fmaxf(a.u_next[seq], 0.0f), 1.0f - 0x1p-24f);
        s.c = {0.0f, 0.0f}, s.left = {1.0f, 0.0f}, s.at = 0, s.next = 1, s.path[0] = 0, s.count = 1, s.n_gone = 0;
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
            if (again) s.c = {0.0f, 0.0f}, s.n_gone = 0, s.summed = false;
            else walk<kDrawn>(s, n);
        }
        __syncthreads();
        const bool draws = s.draws;
        const int64_t r = b0 + s.at;
        row.p = a.probs + r * a.probs_stride;
        row.ch = s.c.hi;
        row.cl = s.c.lo;
        row.q = kDrawn && row.ch > 0.0f ? a.draft + r * a.draft_stride : nullptr;
        if (!s.summed) {
            turn ^= 1;  // (a buffer is written again two passes on: all have read it by then)
            Pairs sum = {};
            if (kDrawn && row.q) sum_of<2, true>(row, s, t0, t1, tiles, lane, sum);
            else sum_of<kDrawn ? 4 : 2, false>(row, s, t0, t1, tiles, lane, sum);
            const Pair of_warp = warp_sum(sum);
            if (lane == 0) s.warp[warp] = of_warp;
            __syncthreads();
            if (warp == 0) {
                Pair v = lane < kWarps ? s.warp[lane] : Pair{0.0f, 0.0f};
#pragma unroll
                for (int o = kWarps / 2; o; o >>= 1) v = plus(v, Pair{__shfl_xor_sync(~0u, v.hi, o), __shfl_xor_sync(~0u, v.lo, o)});
                if (lane < blocks) peer_store(&s.blocks[turn][rank], lane, v);
            }
            cluster_arrive();
            cluster_wait();
        }
        // (what the walk and the draw go on with, in every block alike)
        if (warp == 0) {
            const Pair total = scan(lane < blocks ? s.blocks[turn][lane] : Pair{0.0f, 0.0f}, lane);
            if (lane == 31) {
                s.left = total;
                s.some = some(total);
                s.summed = true;
            }
        }
        __syncthreads();
        if (!draws) continue;
        again = !again && !s.some && (row.ch > 0.0f || s.n_gone > 0);
        if (!again) break;
        __syncthreads();  // (all have read what the next round writes)
    }

    const bool any = s.some;
    if (rank == 0) {
        const int count = s.count;
        for (int i = tid; i < a.max_tok; i += kThreads) path[i] = i < count ? s.path[i] : -1;
        if (tid == 0) {
            a.count[seq] = count;
            if (!any) a.next[seq] = -1;
        }
    }
    if (!any) return;
    if (warp == 0) {
        const Pair none = {0.0f, 0.0f}, of_block = lane < blocks ? s.blocks[turn][lane] : none, of_warp = lane < kWarps ? s.warp[lane] : none;
        const Pair goal = times(s.left, Pair{s.u_next, 0.0f});
        Pair before;
        int w = -1;
        const int o = first_past(scan(of_block, lane), some(of_block), goal, lane, &before);
        Pair rest = minus(goal, before);
        if (o == rank) {
            w = first_past(scan(of_warp, lane), some(of_warp), rest, lane, &before);
            rest = minus(rest, before);
        }
        if (lane == 0) s.owner = w, s.goal = rest;
    }
    __syncthreads();
    if (s.owner < 0) return;
    // the block shares out the tiles of the warp whose stretch it is
    const int o0 = min((rank * kWarps + s.owner) * own, tiles), o1 = min(o0 + own, tiles);
    Pair goal = s.goal;
    int last = -1;  // the last tile with any weight
    for (int base = o0; base < o1; base += kWarps) {
        const int t = base + warp;
        Pairs r[2] = {};
        if (t < o1) row.rest(s, t, lane, row.load(t, lane), r);
        Pairs sum = r[0];
        add(sum, r[1]);
        const Pair of_tile = warp_sum(sum);
        if (lane == 0) s.tiles[warp] = of_tile;
        __syncthreads();
        if (warp == 0) {
            const Pair v = lane < kWarps ? s.tiles[lane] : Pair{0.0f, 0.0f}, upto = scan(v, lane);
            const Pair all = {__shfl_sync(~0u, upto.hi, 31), __shfl_sync(~0u, upto.lo, 31)};
            const unsigned have = __ballot_sync(~0u, some(v));
            if (have) last = base + 31 - __clz(have);
            Pair before = all;
            const int hit = under(goal, all) ? first_past(upto, some(v), goal, lane, &before) : -1;
            goal = minus(goal, before);
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
        if (last >= 0) row.rest(s, last, lane, row.load(last, lane), r);
        const int token = pick(r, last, lane, Pair{INFINITY, 0.0f});
        if (lane == 0) a.next[seq] = token;
    }
}

template <bool kDrawn, bool kVec>
cudaError_t launch(const Verify &a, cudaStream_t s) {
    // Blocks of a sequence: what a pass costs beside the rows (walk, exchange, draw) is some 1,260 tiles' worth, and the GPU
    // takes two blocks an SM at a time.  64 trees: 4 blocks 32 us, 8 40; 200: 1 block 71, 2 58, 4 57 (chosen drafts: 41, 41
    // and 44).  With a drafter that is refused more often, passes are more and trees end farther apart: 64: 46 and 44, 200:
    // 130, 89 and 81.
    const int64_t tiles = (a.V + kTile - 1) / kTile, rows = kDrawn ? 2 : 1;
    int blocks = 1;
    double least = 0.0;
    for (int b = 1; b <= kMost && (b == 1 || tiles >= b * kWarps / 2); b *= 2) {
        const double t = std::max(1.0, (double)b * a.n_seq / (2 * 152)) * (1260.0 + (double)(tiles * rows) / b);
        if (b == 1 || t < least) least = t, blocks = b;
    }
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
