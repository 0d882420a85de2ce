// tree_verify.cu -- verification of drafted trees: which nodes the target's
// probabilities accept, from given random numbers, and the token that follows.
//
// From the last accepted node (node 0 first), with its row p of the target and q of
// the draft, the children are tried in order.  A token x drawn from q is kept with
// probability min(1, p(x) / q(x)); once it is refused the target's distribution is the
// residual max(p - q, 0), normalised, and the next child is tried against that.  The
// residual of a residual keeps its form: with s the sum of max(p - c q, 0),
//     max(max(p - c q, 0) / s - q, 0)  is  max(p - (c + s) q, 0) / s.
// So (c, s), at first (0, 1), is all there is to keep:
//     x is accepted if  u q(x) s < max(p(x) - c q(x), 0),
//     a refusal sets  c += s,  s = sum_t max(p(t) - c q(t), 0).
// After the last accepted node one more token is drawn from what is left there: the
// lowest t whose cumulative weight max(p - c q, 0) exceeds u' times the sum.  Without
// rows of a draft (tokens from a lookup, say) q is 1 at the child and 0 elsewhere: x is
// accepted if u s < p(x), and a refusal takes p(x) out of s and of the row.
//
// Weights are added as whole numbers, in units of 2^-56.  A sum is then the same in any
// order, so the split of a row over threads and CTAs changes no token, and no token on a
// border of the cumulative weights is missed by a rounding: binary32 sums move the borders
// of 128 000 tokens by 2^-24, binary64 additions run at a sixtieth of the rate.  A weight
// is d + e, the difference in binary32 and its rounding error (exact: e = (p - d) - q for
// p >= q), and falls into three whole numbers by additions alone: d + 1 has its multiple of
// 2^-23 in the low bits, what is left of it and e their multiple of 2^-44, and what is left
// then its multiple of 2^-56.  A lane adds those words over its 16 entries of a segment and
// takes the constants out once.  Each entry is rounded by itself, so the sums of a row, a
// segment, a vector and an entry agree to the last unit.  Two entries go through the
// additions of one instruction.
//
// A cluster of CTAs per sequence, one CTA for large batches, shares the row's segments
// of 512 entries.  All its CTAs walk the tree alike (one warp, from probabilities of the
// nodes' tokens that were gathered at once), and go over the row together when a sum is
// needed: at a refusal, and for the last token unless the last refusal's sums serve.
// The segments' sums stay in shared memory, so the token costs one more segment.
//
// Bound: latency.  A sum is one pass over the row by all CTAs, a warp's segments one after
// the other (issue active 29%, 1.4 TB/s), and a refusal's sum must be known before the next
// child is tried.  Graph replay: 9.3 us for one sequence of 6 nodes and 32 000 tokens; 34.3 us
// for 64 sequences of 12 nodes and 128 256 tokens in f32, which need 1.3 passes on average and
// up to 3; 16.8 us for 200 sequences of looked-up tokens out of 50 021 in bf16, of which the
// last token's segment 3.5 us.
#include <cooperative_groups.h>
#include <type_traits>

#include "attn_common.cuh"
#include "common.cuh"
#include "tree.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kNodes = PA_MAX_TREE_NODES;
constexpr int kSegment = 512;       // entries of a segment: 16 a lane
constexpr int kSegments = kMaxVocab / kSegment + 1;
constexpr int kRanks = 8;            // CTAs of a cluster at most
constexpr unsigned kAll = 0xffffffffu;
using u64 = unsigned long long;

__device__ inline float as_float(float x) { return x; }
__device__ inline float as_float(__half x) { return __half2float(x); }
__device__ inline float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A probability: NaN and negative entries count as 0, those above 1 as 1.
__device__ inline float clean(float x) { return __saturatef(x); }

// Sum of up to 16 weights d + e, d in [0, 1], |e| <= 2^-23, in units of 2^-56.
struct Sum {
    static constexpr float A = 1.f;         // [1, 2]: steps of 2^-23
    static constexpr float B = 0x1.8p-21f;  // steps of 2^-44, +- 2^-22
    static constexpr float C = 0x1.8p-33f;  // steps of 2^-56, +- 2^-34 (2^-44 at most are left)
    uint32_t a = 0, b = 0, c = 0;
    int count = 0;
    template <bool HAS_E>
    __device__ inline void add2(float d0, float d1, float e0, float e1) {
        float x0 = d0, x1 = d1;
        add2_rn(x0, x1, A, A);
        a += __float_as_uint(x0) + __float_as_uint(x1);
        add2_rn(x0, x1, -A, -A);
        sub2_rn(d0, d1, x0, x1);
        // B + d + e in steps of 2^-44, then B + d + e without it: d + e by itself would be
        // rounded by 2^-48.  Each difference is exact: of numbers that are multiples of 2^-44,
        // or that are less than that apart.  (0.6 us of the 64 sequences above.)
        x0 = d0, x1 = d1;
        add2_rn(x0, x1, B, B);
        if constexpr (HAS_E) add2_rn(x0, x1, e0, e1);
        b += __float_as_uint(x0) + __float_as_uint(x1);
        add2_rn(x0, x1, -B, -B);
        sub2_rn(d0, d1, x0, x1);
        if constexpr (HAS_E) add2_rn(d0, d1, e0, e1);
        add2_rn(d0, d1, C, C);
        c += __float_as_uint(d0) + __float_as_uint(d1);
        count += 2;
    }
    // An entry is d + e >= 0 rounded to units: never below 0.
    __device__ inline u64 value() const {
        const int64_t hi = (int32_t)(a - count * __float_as_uint(A)), mid = (int32_t)(b - count * __float_as_uint(B));
        const int64_t low = (int32_t)(c - count * __float_as_uint(C));
        return (u64)(hi * (1LL << 33) + mid * (1LL << 12) + low);
    }
};
constexpr double kUnit = 0x1p-56;
// Rows that add up to 256 and more (no probabilities) stay at the end.
__device__ inline u64 add_sat(u64 a, u64 b) {
    const u64 c = a + b;
    return c < a ? ~0ull : c;
}

// Sum over the lanes, each below 2^61, by three 32-bit ones of 27 bits.
__device__ inline u64 sum_of_lanes(u64 x) {
    const uint32_t a = __reduce_add_sync(kAll, (uint32_t)x & 0x7ffffffu);
    const uint32_t b = __reduce_add_sync(kAll, (uint32_t)(x >> 27) & 0x7ffffffu);
    const uint32_t c = __reduce_add_sync(kAll, (uint32_t)(x >> 54));
    return c < 1024 ? add_sat((u64)c << 54, ((u64)b << 27) + a) : ~0ull;
}

// max(p - c q, 0), c = hi + lo.
enum Kind { kRow, kDifference, kGeneral };  // c = 0, 1, any
struct Weights {
    Kind kind;
    float hi, lo;
    // d + e of two entries, d in the place of p.  Where d = p - rn(q hi) cancels, what the
    // product and the difference left, up to 2^-23 for c q < 1, may be the larger part of the
    // weight and have its sign: the larger of the two counts as d.  A positive weight (c q < p
    // <= 1) is off by the split of c, 2^-48 c q, and by two roundings of numbers up to 2^-23:
    // less than 2^-46.
    __device__ inline void general(float& p0, float& p1, float q0, float q1, float& e0, float& e1) const {
        float x0 = clean(q0), x1 = clean(q1), b0 = x0, b1 = x1, t0 = x0, t1 = x1, d0 = p0, d1 = p1;
        fma2_rn(b0, b1, hi, hi, 0.f, 0.f);
        fma2_rn(t0, t1, hi, hi, -b0, -b1);
        fma2_rn(x0, x1, lo, lo, t0, t1);
        sub2_rn(d0, d1, b0, b1);
        sub2_rn(p0, p1, d0, d1);
        sub2_rn(p0, p1, b0, b1);
        sub2_rn(p0, p1, x0, x1);
        const bool some0 = d0 > -p0, some1 = d1 > -p1;
        e0 = some0 ? fminf(d0, p0) : 0.f, e1 = some1 ? fminf(d1, p1) : 0.f;
        p0 = some0 ? fmaxf(d0, p0) : 0.f, p1 = some1 ? fmaxf(d1, p1) : 0.f;
    }
    template <Kind KIND>
    __device__ inline void add2(Sum& sum, float p0, float p1, float q0, float q1) const {
        p0 = clean(p0), p1 = clean(p1);
        if constexpr (KIND == kRow) {
            sum.template add2<false>(p0, p1, 0.f, 0.f);
        } else if constexpr (KIND == kDifference) {
            q0 = fminf(clean(q0), p0), q1 = fminf(clean(q1), p1);
            float d0 = p0, d1 = p1;
            sub2_rn(d0, d1, q0, q1);
            sub2_rn(p0, p1, d0, d1);
            sub2_rn(p0, p1, q0, q1);
            sum.template add2<true>(d0, d1, p0, p1);
        } else {
            float e0, e1;
            general(p0, p1, q0, q1, e0, e1);
            sum.template add2<true>(p0, p1, e0, e1);
        }
    }
    __device__ inline u64 one(float p, float q) const {
        Sum sum;  // the general form has the same d and e for c = 0 and 1
        add2<kGeneral>(sum, p, 0.f, q, 0.f);
        return sum.value();
    }
};

template <typename T>
struct Row {
    const T* at;
    int skew;  // entries from the 16-byte boundary before it
    __device__ inline Row(const void* base, int64_t offset) {
        at = static_cast<const T*>(base) + offset;
        skew = (int)((reinterpret_cast<uintptr_t>(at) & 15) / sizeof(T));
    }
};

// Vector v of COUNT, 32 lanes x N entries apart, from entry `e` of the row on.  Past L1: rows
// are read once, and may be written after this grid was launched.
template <typename T, int N, int COUNT>
__device__ inline void load_inside(const Row<T>& r, int e, uint4 (&x)[COUNT]) {
#pragma unroll
    for (int v = 0; v < COUNT; ++v) x[v] = __ldcg(reinterpret_cast<const uint4*>(r.at + e) + v * 32);
}
// N entries one by one, 0 outside the row.
template <typename T, int N>
__device__ __noinline__ uint4 load_entries(const T* at, int e, int vocab) {
    T x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = e + k >= 0 && e + k < vocab ? at[e + k] : T(0.f);
    uint4 w;
    memcpy(&w, x, 16);
    return w;
}
// The same at a row's ends, or with another skew than the vectors': all vectors inside
// the row first, together, then what lies across its ends.
template <typename T, int N, int COUNT>
__device__ inline void load_edge(const Row<T>& r, int skew, int e, int vocab, uint4 (&x)[COUNT]) {
    static_assert(N * sizeof(T) == 16, "one vector");
    bool across = false;
#pragma unroll
    for (int v = 0; v < COUNT; ++v) {
        const int at = e + v * 32 * N;
        const bool whole = skew == r.skew && at >= 0 && at + N <= vocab;
        x[v] = make_uint4(0u, 0u, 0u, 0u);
        if (whole) x[v] = __ldcg(reinterpret_cast<const uint4*>(r.at + at));
        across |= !whole && at + N > 0 && at < vocab;
    }
    if (!__any_sync(kAll, across)) return;
#pragma unroll
    for (int v = 0; v < COUNT; ++v) {
        const int at = e + v * 32 * N;
        if (at + N > 0 && at < vocab && !(skew == r.skew && at >= 0 && at + N <= vocab))
            x[v] = load_entries<T, N>(r.at, at, vocab);
    }
}

struct Shared {
    int parent[kNodes], token[kNodes];
    float p[kNodes], q[kNodes], u[kNodes];
    bool first[kNodes];        // accepted with c = 0, s = 1
    int refused[kNodes];       // tokens refused at the last accepted node (no draft)
    u64 segment[kSegments];
    u64 warp_sum[kWarps];
    u64 totals[2][kRanks];     // of every CTA's segments, by the parity of the sums' number
    int go;                    // what comes next: 0 the token, 1 a sum
    int now, num_refused;
    double c;
    int again;                 // the last sum is not the one that the token needs
};

template <typename T>
struct Verify {
    const TreeVerifyParams& p;
    Shared& sm;
    const int row0, rank, ranks;

    // Segments of a row that starts `skew` entries behind a boundary, and this CTA's.
    __device__ inline int segments(int skew) const { return (skew + p.vocab + kSegment - 1) / kSegment; }
    __device__ inline int per_cta(int skew) const { return (segments(skew) + ranks - 1) / ranks; }

    // Do segments [s, end) lie in the rows, on vectors of both?
    __device__ inline bool inside(const Row<T>& a, const Row<T>& b, int s, int end) const {
        return a.skew == b.skew && s * kSegment >= a.skew && end * kSegment - a.skew <= p.vocab;
    }

    // Entries e .. e + N - 1 without the refused tokens among them.
    template <int N>
    __device__ inline void take_out(float (&x)[N], int e, int num_refused) const {
        for (int k = 0; k < num_refused; ++k) {
            const int gone = sm.refused[k] - e;
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (j == gone) x[j] = 0.f;
        }
    }

    // Sums of the weights of row `node` by segment, and of this warp's.
    template <Kind KIND>
    __device__ void sums_of(int node, const Weights& w) {
        constexpr bool USE_Q = KIND != kRow;
        constexpr int N = 16 / (int)sizeof(T), V = kSegment / (32 * N);  // entries of a vector, vectors of a lane
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const Row<T> a(p.target, (row0 + node) * p.target_stride);
        const Row<T> b(USE_Q ? p.draft : p.target, (row0 + node) * (USE_Q ? p.draft_stride : p.target_stride));
        const int each = per_cta(a.skew), s0 = rank * each, s1 = min(s0 + each, segments(a.skew));
        const int num_refused = sm.num_refused;
        u64 mine = 0;
#pragma unroll 1
        for (int s = s0 + warp; s < s1; s += kWarps) {
            uint4 x[V], y[V];
            const int e0 = s * kSegment + lane * N - a.skew;
            if (inside(a, b, s, s + 1)) {
                load_inside<T, N>(a, e0, x);
                if (USE_Q) load_inside<T, N>(b, e0, y);
            } else {
                load_edge<T, N>(a, a.skew, e0, p.vocab, x);
                if (USE_Q) load_edge<T, N>(b, a.skew, e0, p.vocab, y);
            }
            // Refused tokens in this segment (rarely one)?
            bool some_gone = false;
            for (int k = 0; k < num_refused; ++k) some_gone |= (sm.refused[k] + a.skew) / kSegment == s;
            Sum lane_sum;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float f[N], h[N];
                unpack16(x[v], f, T());
                if (USE_Q)
                    unpack16(y[v], h, T());
                else if (some_gone)
                    take_out(f, e0 + v * 32 * N, num_refused);
#pragma unroll
                for (int k = 0; k < N; k += 2)
                    w.template add2<KIND>(lane_sum, f[k], f[k + 1], USE_Q ? h[k] : 0.f, USE_Q ? h[k + 1] : 0.f);
            }
            const u64 sum = sum_of_lanes(lane_sum.value());
            if (lane == 0) sm.segment[s - s0] = sum;
            mine = add_sat(mine, sum);
        }
        if (lane == 0) sm.warp_sum[warp] = mine;
        __syncthreads();
    }
    __device__ void sums(int node, const Weights& w) {
        if (w.kind == kRow)
            sums_of<kRow>(node, w);
        else if (w.kind == kDifference)
            sums_of<kDifference>(node, w);
        else
            sums_of<kGeneral>(node, w);
    }

    // The sum of the whole row; this CTA's and those of the CTAs before it.  Every CTA
    // writes its own to all of them, so that none reads another's memory behind the
    // cluster's barrier; the next sums go to the other half of the array.
    __device__ u64 share(const cg::cluster_group& cluster, int number, u64& own, u64& before) {
        u64* const totals = sm.totals[number & 1];
        if (threadIdx.x < 32) {
            u64 t = threadIdx.x < kWarps ? sm.warp_sum[threadIdx.x] : 0;
#pragma unroll
            for (int d = kWarps / 2; d >= 1; d >>= 1) t = add_sat(t, __shfl_xor_sync(kAll, t, d));
            t = __shfl_sync(kAll, t, 0);
            if ((int)threadIdx.x < ranks) *cluster.map_shared_rank(&totals[rank], (int)threadIdx.x) = t;
        }
        if (ranks > 1)
            cluster.sync();
        else
            __syncthreads();
        u64 total = 0;
        own = totals[rank];
        before = 0;
        for (int r = 0; r < ranks; ++r) {
            if (r < rank) before = add_sat(before, totals[r]);
            total = add_sat(total, totals[r]);
        }
        return total;
    }

    // Is x among the tokens refused at the last accepted node?  (warp)
    __device__ inline bool refused(int x, int lane) const {
        bool there = false;
        for (int k = lane; k < sm.num_refused; k += 32) there |= sm.refused[k] == x;
        return __any_sync(kAll, there);
    }

    // Inclusive sums over the lanes.
    static __device__ inline u64 scan(u64 x, int lane) {
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 up = __shfl_up_sync(kAll, x, d);
            if (lane >= d) x = add_sat(x, up);
        }
        return x;
    }

    // Of inclusive sums, the one of the lanes before `owner`.
    static __device__ inline u64 before_lane(u64 incl, int owner) {
        const u64 x = __shfl_sync(kAll, incl, owner > 0 ? owner - 1 : 0);
        return owner > 0 ? x : 0;
    }

    // The first entry of the CTA's segments whose cumulative weight exceeds `left`, less
    // than their sum, by one warp.  The sums that are searched are those that were added, so
    // each search ends at an entry, a vector and a segment that pass `left`.  (Saturated sums
    // pass it; what is before them is then not their difference to the next.)
    __device__ int find(int node, const Weights& w, u64 left, int lane) {
        constexpr int N = 16 / (int)sizeof(T), V = kSegment / (32 * N);
        const bool use_q = w.kind != kRow;
        const Row<T> a(p.target, (row0 + node) * p.target_stride);
        const Row<T> b(use_q ? p.draft : p.target, (row0 + node) * (use_q ? p.draft_stride : p.target_stride));
        const int each = per_cta(a.skew), s0 = rank * each, count = min(each, segments(a.skew) - s0);
        // The segment: a lane has some, the one that passes `left` goes through its own.
        const int share = (count + 31) / 32, k0 = lane * share, k1 = min(k0 + share, count);
        u64 mine = 0;
        for (int k = k0; k < k1; ++k) mine = add_sat(mine, sm.segment[k]);
        u64 incl = scan(mine, lane);
        int owner = __ffs(__ballot_sync(kAll, incl > left)) - 1, seg = k0;
        left -= before_lane(incl, owner);
        if (lane == owner)
            for (; seg < k1 - 1 && sm.segment[seg] <= left; ++seg) left -= sm.segment[seg];
        seg = __shfl_sync(kAll, seg, owner);
        left = __shfl_sync(kAll, left, owner);
        // The vector, then the entry.
        const int e0 = (s0 + seg) * kSegment + lane * N - a.skew;
        uint4 x[V], y[V];
        if (inside(a, b, s0 + seg, s0 + seg + 1)) {
            load_inside<T, N>(a, e0, x);
            load_inside<T, N>(b, e0, y);  // not used without a q
        } else {
            load_edge<T, N>(a, a.skew, e0, p.vocab, x);
            load_edge<T, N>(b, a.skew, e0, p.vocab, y);
        }
        int v = 0;
        u64 sum = 0;
#pragma unroll 1
        for (;; ++v) {
            uint4 xv = x[0], yv = y[0];
#pragma unroll
            for (int k = 1; k < V; ++k)
                if (k == v) xv = x[k], yv = y[k];
            float f[N], h[N];
            unpack16(xv, f, T());
            unpack16(yv, h, T());
            take_out(f, e0 + v * 32 * N, sm.num_refused);
            Sum lane_sum;
#pragma unroll
            for (int k = 0; k < N; k += 2) w.template add2<kGeneral>(lane_sum, f[k], f[k + 1], h[k], h[k + 1]);
            sum = lane_sum.value();
            const u64 all = sum_of_lanes(sum);
            if (v == V - 1 || all > left) break;
            left -= all;
        }
        incl = scan(sum, lane);
        owner = __ffs(__ballot_sync(kAll, incl > left)) - 1;
        left -= before_lane(incl, owner);
        // Its entries, a lane to each.
        const int e = (s0 + seg) * kSegment + (v * 32 + owner) * N - a.skew + lane;
        float f[1] = {0.f}, h = 0.f;
        if (lane < N && e >= 0 && e < p.vocab) {
            f[0] = as_float(a.at[e]);
            if (use_q) h = as_float(b.at[e]);
            take_out(f, e, sm.num_refused);
        }
        return __shfl_sync(kAll, e, __ffs(__ballot_sync(kAll, scan(w.one(f[0], h), lane) > left)) - 1);
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) tree_verify_kernel(const __grid_constant__ TreeVerifyParams p) {
    __shared__ Shared sm;
    const cg::cluster_group cluster = cg::this_cluster();
    const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int s = (int)blockIdx.x / ranks, tid = threadIdx.x, lane = tid & 31;
    pdl_wait_prerequisites();
    const int row0 = p.query_start[s], end = p.query_start[s + 1], n = end - row0;
    // Uniform over the cluster, as everything up to the token is.
    if (row0 < 0 || n <= 0 || end > p.num_tokens || n > kNodes) {
        if (rank == 0 && tid == 0) {
            if (n != 0 || row0 < 0 || end > p.num_tokens) set_error(p.err, PA_DEVERR_CONTEXT_LEN);
            p.accepted_lens[s] = 0;
            p.next_tokens[s] = -1;
        }
        return;
    }
    if (ranks > 1) cluster.barrier_arrive();  // waited for before the first sum is shared
    const bool drafted = p.draft != nullptr;
    bool bad = false;
    for (int i = tid; i < n; i += kThreads) {
        const int up = p.parents[row0 + i], x = p.tokens[row0 + i];
        const bool fits = up >= -1 && up < i;
        bad |= !fits || (i > 0 && (x < 0 || x >= p.vocab));
        // A node that hangs on no other, or with no token, is tried by none.
        const bool tried = fits && up >= 0 && x >= 0 && x < p.vocab;
        sm.parent[i] = tried ? up : -1;
        sm.token[i] = x;
        if (tried) {
            const float a = clean(as_float(static_cast<const T*>(p.target)[(row0 + up) * p.target_stride + x]));
            const float b = drafted ? clean(as_float(static_cast<const T*>(p.draft)[(row0 + up) * p.draft_stride + x])) : 1.f;
            const float u = p.accept_uniforms[row0 + i];
            sm.p[i] = a;
            sm.q[i] = b;
            sm.u[i] = u;
            // Exact, and off the walk's chain of dependent steps: binary64 takes long.
            sm.first[i] = (double)u * (double)b < (double)a;
        }
        if (rank == 0) p.path[row0 + i] = i == 0 ? 0 : -1;
    }
    if (rank == 0 && bad) set_error(p.err, PA_DEVERR_TREE);
    if (tid == 0) sm.num_refused = 0;
    __syncthreads();

    Verify<T> v{p, sm, row0, rank, ranks};
    // Walk (warp 0): c, s of the last accepted node, the next node to look at.
    double c = 0., sum = 1.;
    int now = 0, from = 1, count = 1, number = 0;
    bool spent = false;  // nothing is left of the target's row: the token comes from the row itself
    u64 own = 0, before = 0, total = 0;
    auto shared_sum = [&] {
        if (ranks > 1 && number == 0) cluster.barrier_wait();  // every CTA of the cluster has begun
        total = v.share(cluster, number++, own, before);
    };
    while (true) {
        if (tid < 32) {
            int go = 0;
            while (!spent) {
                int i = n;
                for (int i0 = from; i0 < n; i0 += 32) {
                    const unsigned m = __ballot_sync(kAll, i0 + lane < n && sm.parent[i0 + lane] == now);
                    if (m) {
                        i = i0 + __ffs(m) - 1;
                        break;
                    }
                }
                if (i >= n) break;
                from = i + 1;
                const bool plain = c == 0. && sum == 1.;
                const int x = sm.token[i], num_refused = sm.num_refused;
                bool accept;
                double w = 0.;
                if (drafted) {
                    accept = plain ? sm.first[i] : (double)sm.u[i] * sm.q[i] * sum < fmax(sm.p[i] - c * sm.q[i], 0.);
                } else if (plain && num_refused == 0) {
                    accept = sm.first[i];
                    w = sm.p[i];
                } else {
                    w = v.refused(x, lane) ? 0. : sm.p[i];
                    accept = (double)sm.u[i] * sum < w;
                }
                __syncwarp();  // every lane has read the list that lane 0 changes
                if (accept) {
                    if (lane == 0) {
                        if (rank == 0) p.path[row0 + count] = i;
                        sm.num_refused = 0;
                    }
                    ++count;
                    now = i;
                    c = 0.;
                    sum = 1.;
                } else if (drafted) {
                    c += sum;
                    go = 1;
                    break;
                } else {
                    sum = fmax(sum - w, 0.);
                    if (lane == 0 && w > 0.) {
                        sm.refused[num_refused] = x;
                        sm.num_refused = num_refused + 1;
                    }
                }
                __syncwarp();
            }
            if (lane == 0) {
                sm.go = go;
                sm.now = now;
                sm.c = c;
                sm.again = go || spent || !drafted || c == 0.;
            }
        }
        __syncthreads();
        const bool token = !sm.go;
        // Weights of the token: those of the last sum, or the target's row.
        const int node = sm.now;
        const double factor = sm.go || !sm.again ? sm.c : 0.;
        const float hi = (float)factor;
        const Weights w{factor == 0. ? kRow : factor == 1. ? kDifference : kGeneral, hi, (float)(factor - hi)};
        if (sm.again) {
            v.sums(node, w);
            shared_sum();
            if (token && total == 0 && sm.num_refused > 0) {
                // Nothing but refused tokens: the row itself.
                __syncthreads();
                if (tid == 0) sm.num_refused = 0;
                __syncthreads();
                v.sums(node, w);
                shared_sum();
            }
        }
        if (token) {
            if (rank == 0 && tid == 0) p.accepted_lens[s] = count;
            float u = p.sample_uniforms[s];
            u = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
            const u64 target = __umul64hi(__double2ull_rz((double)u * 18446744073709551616.), total);
            if (total == 0) {
                if (rank == 0 && tid == 0) {
                    set_error(p.err, PA_DEVERR_PROBS);
                    p.next_tokens[s] = -1;
                }
            } else if (target >= before && target - before < own && tid < 32) {
                const int x = v.find(node, w, target - before, lane);
                if (lane == 0) p.next_tokens[s] = x;
            }
            return;
        }
        // A refusal's sum.
        sum = (double)total * kUnit;
        spent = total == 0;
        __syncthreads();
    }
}

template <typename T>
cudaError_t launch_t(const TreeVerifyParams& p, int ranks, cudaStream_t stream) {
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.num_seqs * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, tree_verify_kernel<T>, p);
}

}  // namespace

cudaError_t launch_tree_verify(const TreeVerifyParams& p, int dtype, int sms, cudaStream_t stream) {
    // As many CTAs to a sequence as keep two on every SM, each with 8 segments at least.
    // (The 200 sequences above: 16.5 us so and with one CTA an SM, 21.4 with up to four; the 64
    // with draft rows: 34.7 us, 40.8 with one, 40.2 with four.)
    int ranks = 8;
    while (ranks > 1 && ((int64_t)p.num_seqs * ranks > 2LL * sms || p.vocab < ranks * 8 * kSegment)) ranks /= 2;
    switch (dtype) {
        case PA_F32: return launch_t<float>(p, ranks, stream);
        case PA_F16: return launch_t<__half>(p, ranks, stream);
        case PA_BF16: return launch_t<__nv_bfloat16>(p, ranks, stream);
        default: return cudaErrorNotSupported;
    }
}

}  // namespace pa
