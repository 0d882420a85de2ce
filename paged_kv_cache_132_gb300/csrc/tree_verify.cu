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
// p >= q), and falls into three whole numbers by additions alone: d + 2 has its multiple
// of 2^-22 in the low bits, what is left its multiples of 2^-44 and then of 2^-56.  A
// lane adds the words up and takes the constants out once per segment.
//
// A cluster of CTAs per sequence, one CTA for large batches, shares the row's segments
// of 512 entries.  All its CTAs walk the tree alike (one warp, from probabilities of the
// nodes' tokens that were gathered at once), and go over the row together when a sum is
// needed: at a refusal, and for the last token unless the last refusal's sums serve.
// The segments' sums stay in shared memory, so the token costs one more segment.
//
// Bound: HBM for batches (a row of p and mostly one of q each sequence), latency below.
#include <cooperative_groups.h>
#include <type_traits>

#include "common.cuh"
#include "tree.h"

namespace cg = cooperative_groups;

namespace pa {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kNodes = 1024;        // PA_MAX_TREE_NODES
constexpr int kSegment = 512;       // entries of a segment: 16 a lane
constexpr int kSegments = kMaxVocab / kSegment + 1;
constexpr unsigned kAll = 0xffffffffu;
using u64 = unsigned long long;

__device__ inline float as_float(float x) { return x; }
__device__ inline float as_float(__half x) { return __half2float(x); }
__device__ inline float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// A probability: NaN and negative entries count as 0, those above 1 as 1.
__device__ inline float clean(float x) { return fminf(fmaxf(x, 0.f), 1.f); }

// Sum of weights d + e, d in [0, 1], |e| <= 2^-24, in units of 2^-56.
struct Sum {
    static constexpr float A = 2.f;               // [2, 4): steps of 2^-22
    static constexpr float B = 0x1.8p-21f;        // steps of 2^-44, +- 2^-22
    static constexpr float C = 0x1.8p-33f;        // steps of 2^-56, +- 2^-34
    uint32_t a = 0, b = 0, c = 0;
    int count = 0;
    __device__ inline void add(float d, float e) {
        const float x = __fadd_rn(d, A);
        const float r = __fadd_rn(__fsub_rn(d, __fsub_rn(x, A)), e);
        const float y = __fadd_rn(r, B);
        const float z = __fadd_rn(__fsub_rn(r, __fsub_rn(y, B)), C);
        a += __float_as_uint(x);
        b += __float_as_uint(y);
        c += __float_as_uint(z);
        ++count;
    }
    __device__ inline u64 value() const {
        const int64_t hi = (int32_t)(a - count * __float_as_uint(A)), mid = (int32_t)(b - count * __float_as_uint(B)),
                      lo = (int32_t)(c - count * __float_as_uint(C));
        const int64_t v = hi * (1LL << 34) + mid * (1LL << 12) + lo;
        return v > 0 ? (u64)v : 0;
    }
};
constexpr double kUnit = 0x1p-56;
// Rows that add up to 256 and more (no probabilities) stay at the end.
__device__ inline u64 add_sat(u64 a, u64 b) {
    const u64 c = a + b;
    return c < a ? ~0ull : c;
}

// max(p - c q, 0), c = hi + lo.
struct Weights {
    bool use_q;
    float hi, lo;  // hi = 1 and lo = 0 after the first refusal
    __device__ inline void add(Sum& sum, float p, float q) const {
        p = clean(p);
        if (!use_q) {
            sum.add(p, 0.f);
        } else if (hi == 1.f && lo == 0.f) {
            const float b = fminf(fmaxf(q, 0.f), p);
            const float d = __fsub_rn(p, b);
            sum.add(d, __fsub_rn(__fsub_rn(p, d), b));
        } else {
            const float x = clean(q), b = __fmul_rn(x, hi);
            const float d = __fsub_rn(p, b);
            const float e = __fsub_rn(__fsub_rn(__fsub_rn(p, d), b), __fmaf_rn(x, lo, __fmaf_rn(x, hi, -b)));
            if (d > 0.f) sum.add(d, fmaxf(e, -d));
        }
    }
    __device__ inline u64 one(float p, float q) const {
        Sum sum;
        add(sum, p, q);
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

// N entries of a row from `e` on (a multiple of N before the skew); 0 outside it.
template <typename T, int N>
__device__ inline uint4 load_vector(const Row<T>& r, int skew, int e, int vocab) {
    static_assert(N * sizeof(T) == 16, "one vector");
    if (skew == r.skew && e >= 0 && e + N <= vocab) return __ldg(reinterpret_cast<const uint4*>(r.at + e));
    T x[N];
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = e + k >= 0 && e + k < vocab ? r.at[e + k] : T(0.f);
    uint4 w;
    memcpy(&w, x, 16);
    return w;
}

struct Shared {
    int parent[kNodes], token[kNodes];
    float p[kNodes], q[kNodes], u[kNodes];
    int refused[kNodes];    // tokens refused at the last accepted node (no draft)
    u64 segment[kSegments];
    u64 warp_sum[kWarps];
    u64 total;              // of this CTA's segments (read by the cluster)
    int go;                 // what comes next: 0 the token, 1 a sum
    int now, num_refused;
    double c;
    int again;              // the last sum is not the one that the token needs
    int use_q;
};

template <typename T>
struct Verify {
    const TreeVerifyParams& p;
    Shared& sm;
    const int row0, rank, ranks;

    // Segments of a row that starts `skew` entries behind a boundary, and this CTA's.
    __device__ inline int segments(int skew) const { return (skew + p.vocab + kSegment - 1) / kSegment; }
    __device__ inline int per_cta(int skew) const { return (segments(skew) + ranks - 1) / ranks; }

    // Sums of the weights of row `node` by segment, and of all this CTA's.  A warp has
    // eight vectors of every lane in flight: one to four segments.
    template <bool USE_Q>
    __device__ void sums_of(int node, const Weights& w) {
        constexpr int N = 16 / (int)sizeof(T), V = kSegment / (32 * N);  // entries of a vector, vectors of a lane
        constexpr int SEGS = 8 / (V * (USE_Q ? 2 : 1));
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const Row<T> a(p.target, (row0 + node) * p.target_stride);
        const Row<T> b(USE_Q ? p.draft : p.target, (row0 + node) * (USE_Q ? p.draft_stride : p.target_stride));
        const int each = per_cta(a.skew), s0 = rank * each, s1 = min(s0 + each, segments(a.skew));
        u64 mine = 0;
        for (int s = s0 + warp * SEGS; s < s1; s += kWarps * SEGS) {
            uint4 x[SEGS * V], y[SEGS * V];
#pragma unroll
            for (int v = 0; v < SEGS * V; ++v) {
                const int e = s * kSegment + (v * 32 + lane) * N - a.skew;
                x[v] = load_vector<T, N>(a, a.skew, e, p.vocab);
                if (USE_Q) y[v] = load_vector<T, N>(b, a.skew, e, p.vocab);
            }
#pragma unroll
            for (int g = 0; g < SEGS; ++g) {
                Sum lane_sum;
#pragma unroll
                for (int v = g * V; v < (g + 1) * V; ++v) {
                    float f[N], h[N];
                    unpack16(x[v], f, T());
                    if (USE_Q) unpack16(y[v], h, T());
#pragma unroll
                    for (int k = 0; k < N; ++k) w.add(lane_sum, f[k], USE_Q ? h[k] : 0.f);
                }
                u64 sum = lane_sum.value();
#pragma unroll
                for (int d = 16; d >= 1; d >>= 1) sum = add_sat(sum, __shfl_xor_sync(kAll, sum, d));
                // past the CTA's last segment: the next one's, or nothing
                if (s + g < s1) {
                    if (lane == 0) sm.segment[s + g - s0] = sum;
                    mine = add_sat(mine, sum);
                }
            }
        }
        if (lane == 0) sm.warp_sum[warp] = mine;
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 t = 0;
            for (int k = 0; k < kWarps; ++k) t = add_sat(t, sm.warp_sum[k]);
            sm.total = t;
        }
        __syncthreads();
    }
    __device__ void sums(int node, const Weights& w) {
        if (!w.use_q)
            sums_of<false>(node, w);
        else if (w.hi == 1.f && w.lo == 0.f)
            sums_of<true>(node, Weights{true, 1.f, 0.f});  // without the products
        else
            sums_of<true>(node, w);
    }

    // Is x among the tokens refused at the last accepted node?  (warp)
    __device__ inline bool refused(int x, int lane) const {
        bool there = false;
        for (int k = lane; k < sm.num_refused; k += 32) there |= sm.refused[k] == x;
        return __any_sync(kAll, there);
    }

    // The first entry of the CTA's segments whose cumulative weight exceeds `left`, by
    // one warp; entries of refused tokens weigh nothing.
    __device__ int find(int node, const Weights& w, u64 left, int lane) {
        constexpr int N = 16 / (int)sizeof(T), V = kSegment / (32 * N);
        const Row<T> a(p.target, (row0 + node) * p.target_stride);
        const Row<T> b(w.use_q ? p.draft : p.target, (row0 + node) * (w.use_q ? p.draft_stride : p.target_stride));
        const int each = per_cta(a.skew), s0 = rank * each, count = min(each, segments(a.skew) - s0);
        // this lane's segments, then the one that passes `left`
        const int share = (count + 31) / 32, k0 = lane * share, k1 = min(k0 + share, count);
        u64 mine = 0;
        for (int k = k0; k < k1; ++k) mine = add_sat(mine, sm.segment[k]);
        u64 incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 up = __shfl_up_sync(kAll, incl, d);
            if (lane >= d) incl = add_sat(incl, up);
        }
        const unsigned past = __ballot_sync(kAll, incl > left);
        if (past == 0) return -1;
        const int owner = __ffs(past) - 1;
        int seg = 0;
        if (lane == owner) {
            left -= incl - mine;
            for (seg = k0; seg < k1 - 1 && sm.segment[seg] <= left; ++seg) left -= sm.segment[seg];
        }
        seg = __shfl_sync(kAll, seg, owner);
        left = __shfl_sync(kAll, left, owner);
        int token = -1;
        for (int v = 0; v < V && token < 0; ++v) {
            const int e = (s0 + seg) * kSegment + (v * 32 + lane) * N - a.skew;
            float x[N], y[N];
            unpack16(load_vector<T, N>(a, a.skew, e, p.vocab), x, T());
            unpack16(load_vector<T, N>(b, a.skew, e, p.vocab), y, T());
            for (int k = 0; k < sm.num_refused; ++k) {
                const int gone = sm.refused[k] - e;
#pragma unroll
                for (int j = 0; j < N; ++j)
                    if (j == gone) x[j] = 0.f;
            }
            u64 sum = 0;
#pragma unroll
            for (int k = 0; k < N; ++k) sum += w.one(x[k], y[k]);
            u64 below = sum;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const u64 up = __shfl_up_sync(kAll, below, d);
                if (lane >= d) below += up;
            }
            const unsigned over = __ballot_sync(kAll, below > left);
            if (over) {
                const int at = __ffs(over) - 1;
                if (lane == at) {
                    u64 cum = below - sum;
#pragma unroll
                    for (int k = 0; k < N; ++k) {
                        cum += w.one(x[k], y[k]);
                        if (token < 0 && cum > left) token = e + k;
                    }
                }
                token = __shfl_sync(kAll, token, at);
            } else {
                left -= __shfl_sync(kAll, below, 31);
            }
        }
        return token;
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
            sm.p[i] = clean(as_float(static_cast<const T*>(p.target)[(row0 + up) * p.target_stride + x]));
            sm.q[i] = drafted ? clean(as_float(static_cast<const T*>(p.draft)[(row0 + up) * p.draft_stride + x])) : 1.f;
            sm.u[i] = p.accept_uniforms[row0 + i];
        }
        if (rank == 0) p.path[row0 + i] = i == 0 ? 0 : -1;
    }
    if (rank == 0 && bad) set_error(p.err, PA_DEVERR_TREE);
    if (tid == 0) sm.num_refused = 0;
    __syncthreads();

    Verify<T> v{p, sm, row0, rank, ranks};
    // Walk (warp 0): c, s of the last accepted node, the next node to look at.
    double c = 0., sum = 1.;
    int now = 0, from = 1, count = 1;
    bool spent = false;    // nothing is left of the target's row: the token comes from the row itself
    u64 own = 0, before = 0, total = 0;
    auto weights = [&](bool use_q, double factor) {
        const float hi = (float)factor;
        return Weights{use_q, hi, (float)(factor - hi)};
    };
    // The sums of the whole row: this CTA's, those of the CTAs before it, of all.
    auto share = [&] {
        cluster.sync();
        own = sm.total;
        before = total = 0;
        for (int r = 0; r < ranks; ++r) {
            const u64 t = *cluster.map_shared_rank(&sm.total, r);
            if (r < rank) before = add_sat(before, t);
            total = add_sat(total, t);
        }
        cluster.sync();
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
                const double u = sm.u[i], q = sm.q[i];
                double w = fmax(sm.p[i] - c * q, 0.);
                const int x = sm.token[i];
                if (!drafted) w = v.refused(x, lane) ? 0. : sm.p[i];
                if (u * q * sum < w) {
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
                    if (lane == 0 && w > 0.) sm.refused[sm.num_refused++] = x;
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
        const bool use_q = sm.go || !sm.again;
        const int node = sm.now;
        const Weights w = weights(use_q, sm.c);
        if (sm.again) {
            v.sums(node, w);
            if (token && sm.num_refused > 0) {
                // Take the refused tokens out; if nothing else is left, they are not.
                const Row<T> a(p.target, (int64_t)(row0 + node) * p.target_stride);
                const int each = v.per_cta(a.skew), s0 = rank * each;
                if (tid == 0)
                    for (int k = 0; k < sm.num_refused; ++k) {
                        const int x = sm.refused[k], seg = (x + a.skew) / kSegment - s0;
                        if (seg < 0 || seg >= each) continue;
                        const u64 gone = Weights{false, 0.f, 0.f}.one(as_float(a.at[x]), 0.f);
                        sm.segment[seg] -= min(gone, sm.segment[seg]);
                        sm.total = sm.total == ~0ull ? sm.total : sm.total - min(gone, sm.total);
                    }
                __syncthreads();
            }
            share();
            if (token && sm.num_refused > 0 && total == 0) {
                __syncthreads();
                if (tid == 0) sm.num_refused = 0;
                __syncthreads();
                v.sums(node, w);
                share();
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
