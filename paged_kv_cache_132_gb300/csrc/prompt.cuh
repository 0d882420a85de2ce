// prompt.cuh -- causal attention over whole packed prompts on the Blackwell
// tensor cores (tcgen05.mma, accumulators in tensor memory).
//
// What it computes, for token i and query head h of each packed sequence
// (KV head h / G; "PagedAttention 论文精读笔记", §2.1 attention equation and
// §5.3 prompt step, with keys and values still in the projections' rows):
//     out[i][h] = sum_{j <= i} softmax_j(scale * q[i][h] . k_j) v_j
//
// Work item: 2 * (128 / G) consecutive tokens of one (sequence, KV head), as
// two query tiles of 128 rows (row = token * G + grouped head), so both tiles
// and all G heads use every K/V tile that is loaded.  One CTA per SM takes
// items until none is left.  Keys and values stream through a ring of
// 128-position tiles; per tile j and query tile i:
//   S_i  = Q_i K_j^T      tcgen05.mma M=128 N=128 K=d, into TMEM
//   P_i  = 2^(S_i c - m)  softmax warps, one thread per row; P_i, rounded to
//                         the inputs' 16-bit type, is written over S_i
//   O_i += P_i V_j        tcgen05.mma with A = P_i from TMEM
// with c = scale * log2 e, the running maximum m in base-2 units, O_i rescaled
// only when a row's maximum grows by more than 8 (a factor of 256), and row
// sums in binary32 over the unrounded weights.  The rounding of P to 16 bits
// costs as much as the rounding of the output that follows it (half a step of
// the type on independent weights), and lets P.V run at the 16-bit rate.  In f16
// all weights of a row are 2^7 larger (2^8 by the delayed rescaling, 2^15 in all:
// half of the type's range), which the division by their sum takes out again, so
// that a weight loses bits below 2^-21 of the row's largest and rounds to 0 below
// 2^-32; without, below 2^-14 and 2^-25, and the many small weights of a long row
// were missing from its output.  bf16 has the range of binary32.
//
// Bound: tensor cores (4 d flops per row and position).  The two query tiles
// alternate on them: while one's softmax runs, the MMAs of the other (P V_j, then
// S of tile j + 1) are executed.  P_i lies over S_i because tensor memory is full
// (2 x (128 + 128) columns at d = 128), so a tile's chain is S -> softmax -> P V ->
// S; a step of both tiles takes 2080 cycles of MMAs and 2750 by the chain (softmax
// 1600: 128 exponentials a thread at 4.3 cycles, the scores' load, the maximum;
// then P V and S 1040 and their latency).  Measured: 1.59-1.76 PFLOP/s by the box
// (0.8-0.88 of the cuBLAS burst rate, 0.91-1.0 of the sustained one) for 32768
// tokens of 32 heads of 128, where power sets the clock; 0.99-1.13 PFLOP/s for 32
// prompts of 128-1024 tokens (112-128 us, by the clock), where an item is 3.5 steps
// and starting it costs a third of one.
//
// Values a query must not see: a row's weights after its own position are 0,
// but 0 * NaN is NaN on the tensor cores.  So before P.V reads a V tile that
// holds positions some row of the item does not attend (the last one or two of
// an item), a warp clears its rows after the item's last position and
// replaces non-finite elements by 0; those are added again, to the rows that do
// attend them, by the output warps.  In the tiles before, which every row of the
// item attends, the tensor cores multiply such a value by its rounded weight: an
// infinite one gives NaN where the weight has rounded to 0.  Either way it makes its
// column of the rows that attend it infinite or NaN, and nothing else.  Keys need no
// such care: masked scores are replaced.
//
// Warp roles (512 threads, registers moved between the groups by setmaxnreg):
//   warps 0, 1       MMA issuers of query tile 0 / 1 (warp 0 owns the TMEM
//                    allocation)
//   warp 2           work items, Q, K and V copies (TMA)
//   warp 3           the V tiles with masked positions (above)
//   warps 4-7, 8-11  softmax of query tile 0 / 1
//   warps 12-15      outputs: O_i / row sum, rounded once, written to memory
// Every wait is bounded; a wait that runs out sets PA_DEVERR_TIMEOUT and makes
// every role of the CTA leave, after what it issued has landed.
#pragma once

#include <cuda.h>

#include "attn_common.cuh"
#include "common.cuh"
#include "decode_common.cuh"  // kFullMask
#include "kernels.h"
#include "tcgen05.cuh"

namespace pa {

template <int D>
struct PromptShape {
    static constexpr int BM = 128;               // query rows per tile, two tiles per item
    static constexpr int BN = 128;               // key/value positions per tile
    static constexpr int HALF = 64;              // positions per K/V copy: a short last tile loads one half
    static constexpr int SLABS = D / 64;         // 64-element (128-byte) column slabs of a row
    static constexpr int SLAB = 128 * 128;       // bytes of one slab of 128 rows
    static constexpr int NSLOT = D == 128 ? 5 : 8;  // K/V ring: K_0, V_0, K_1, V_1, ... one tile per slot
    static constexpr int NITEM = 4;              // work items announced ahead of their last reader
    static constexpr int SOFTMAX_WARPS = 4;      // per query tile
    static constexpr int MMA_WARP = 0;           // first of two, one per query tile
    static constexpr int LOAD_WARP = 2;
    static constexpr int CHECK_WARP = 3;
    static constexpr int SOFTMAX_WARP = 4;       // first of eight
    static constexpr int OUT_WARP = 12;          // first of four
    static constexpr int THREADS = 512;
    static constexpr int ITEM_READERS = 8 + 4 + 2 + 1;  // softmax, output, MMA, check warps
    // Registers per thread after the split: 256 * 176 + 128 * 64 + 128 * 96
    // = 512 * 128, the launch's total.
    static constexpr int REGS_SOFTMAX = 176, REGS_OUT = 64, REGS_OTHER = 96;
    static_assert(256 * REGS_SOFTMAX + 128 * REGS_OUT + 128 * REGS_OTHER <= THREADS * 128, "register split");
    // TMEM columns: S_i (and P_i over it, two per column) at 128 i, O_i after both.
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t O_COL = 2 * BN;
    static_assert(D == 64 || D == 128, "head_dim 64 or 128");

    struct Smem {
        alignas(1024) uint8_t q[2][SLABS][SLAB];
        alignas(1024) uint8_t kv[NSLOT][SLABS][SLAB];
        float row_sum[2][BM];
        int4 item[NITEM];           // first row, length, item of the sequence, KV head; length 0: no more work
        int last_dirty;             // latest item with non-finite values in its checked tiles
        uint64_t item_full[NITEM];  // announced (load warp)
        uint64_t item_empty[NITEM]; // read by every role
        uint64_t q_full[2];         // Q_i landed
        uint64_t q_empty[2];        // last S_i of the item complete
        uint64_t kv_full[NSLOT];    // tile landed
        uint64_t kv_empty[NSLOT];   // the MMAs of both query tiles that read it complete
        uint64_t check_go[NSLOT];   // the copy of a V tile with masked positions was issued (load warp)
        uint64_t v_checked[NSLOT];  // ... and the tile is fit for P.V (check warp)
        uint64_t s_full[2];         // S_i complete
        uint64_t p_full[2][2];      // each half of P_i written (softmax warps)
        uint64_t o_full[2];         // last P_i V_j of the item complete
        uint64_t l_full[2];         // row sums written (softmax warps)
        uint64_t o_empty[2];        // O_i and the row sums read (output warps)
        uint64_t turn[2];           // MMA warp i may issue its step
        uint64_t mma_done[2];
        uint32_t tmem_base;
        int abort_flag;
    };
    static constexpr int SMEM_BYTES = (int)sizeof(Smem) + 1024;
    static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");
};

// 2^x as exp2_approx (common.cuh), free to be moved by the compiler.
__device__ __forceinline__ float prompt_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <uint32_t REGS>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <uint32_t REGS>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

__device__ __forceinline__ bool prompt_aborted(int* abort_flag) { return *reinterpret_cast<volatile int*>(abort_flag); }

// Waits for a phase of a barrier.  When the limit runs out, here or in another
// role, every wait of the CTA ends: the roles run on to the end of their item
// without data (in shared and tensor memory only: the output warps store nothing
// any more, the load warp issues nothing more) and then leave, and the CTA reports
// PA_DEVERR_TIMEOUT.  Kept short: it is inlined in some twenty places, and the
// roles' code competes for the instruction caches.
template <class Smem>
__device__ __forceinline__ void prompt_wait(const PromptParams& p, Smem& sm, uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t start = global_timer_ns();
    do {
        if (prompt_aborted(&sm.abort_flag)) return;
        if (global_timer_ns() - start > p.wait_limit_ns) *reinterpret_cast<volatile int*>(&sm.abort_flag) = 1;
    } while (!mbar_try_wait(bar, parity));
}

// The same for a barrier given by its shared-memory address (the MMA warp, whose
// every instruction between a P and its MMAs is waited for).
__device__ __forceinline__ bool try_wait_at(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
template <class Smem>
__device__ __forceinline__ void prompt_wait_at(const PromptParams& p, Smem& sm, uint32_t bar, uint32_t parity) {
    if (try_wait_at(bar, parity)) return;
    const uint64_t start = global_timer_ns();
    do {
        if (prompt_aborted(&sm.abort_flag)) return;
        if (global_timer_ns() - start > p.wait_limit_ns) *reinterpret_cast<volatile int*>(&sm.abort_flag) = 1;
    } while (!try_wait_at(bar, parity));
}

// What an item is made of, for every role alike.
struct PromptItem {
    int row0;     // first row of the sequence
    int len;      // its tokens
    int kv_head;
    int t0;       // first token of query tile 0; tile 1 starts tile_tokens later
    int end0, end1;  // positions [0, end_i) are read by tile i; 0: the tile is empty
    int first_masked;  // first K/V tile with a position some row does not attend
    __device__ __forceinline__ int end(int i) const { return i ? end1 : end0; }
    __device__ __forceinline__ int tiles(int i) const { return (end(i) + 127) >> 7; }  // its K/V tiles
    __device__ __forceinline__ int last() const { return max(end0, end1); }
};

__device__ __forceinline__ PromptItem prompt_item(const int4& it, int tile_tokens) {
    PromptItem w;
    w.row0 = it.x;
    w.len = it.y;
    w.kv_head = it.w;
    w.t0 = it.z * 2 * tile_tokens;
    w.end0 = min(w.t0 + tile_tokens, w.len);
    w.end1 = w.len > w.t0 + tile_tokens ? min(w.t0 + 2 * tile_tokens, w.len) : 0;
    w.first_masked = w.t0 >> 7;
    return w;
}

// Reader side of the item ring (one warp): the next item, or false at the end
// of the work or of the kernel.
template <class Shape>
__device__ __forceinline__ bool prompt_next_item(const PromptParams& p, typename Shape::Smem& sm, int lane, int& n,
                                                 PromptItem& w) {
    const int st = n % Shape::NITEM;
    prompt_wait(p, sm, &sm.item_full[st], (uint32_t)(n / Shape::NITEM) & 1u);
    if (__any_sync(kFullMask, prompt_aborted(&sm.abort_flag))) return false;
    const int4 it = sm.item[st];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[st]);
    ++n;
    if (it.y == 0) return false;
    w = prompt_item(it, p.tile_tokens);
    return true;
}

// ---------------------------------------------------------------------------
// load warp: work items and copies
// ---------------------------------------------------------------------------
// With a list (prompt_plan_kernel) CTA c takes item c first and then whatever
// a device counter gives it; KV heads are innermost, so CTAs at work together
// share a sequence's rows in L2.  A call with no more items than CTAs needs no
// list: CTA c finds item c itself, walking the start rows 32 sequences at a
// time.
struct PromptWalk {
    int base;    // sequences [base, base + 32) are in the lanes
    int before;  // (sequence, query tile pair) units before them
    int row0, len, nb, incl;  // this lane's sequence; inclusive sum of nb over the lanes
};

__device__ __forceinline__ void prompt_walk_load(const PromptParams& p, PromptWalk& k, int lane) {
    const int s = k.base + lane;
    k.row0 = k.len = 0;
    if (s < p.num_seqs) {
        const int a = __ldcg(p.query_start + s), b = __ldcg(p.query_start + s + 1);
        if (a < 0 || b < a || b > p.num_tokens) {
            set_error(p.err, PA_DEVERR_CONTEXT_LEN);
        } else {
            k.row0 = a;
            k.len = b - a;
        }
    }
    k.nb = (k.len + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
    k.incl = k.nb;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(kFullMask, k.incl, d);
        if (lane >= d) k.incl += up;
    }
}

// The item with number `index`; length 0 when there is none.
__device__ __forceinline__ int4 prompt_walk_to(const PromptParams& p, PromptWalk& k, int lane, int index) {
    const int unit = index / p.num_kv_heads;
    while (true) {
        const int total = __shfl_sync(kFullMask, k.incl, 31);
        if (unit < k.before + total) break;
        k.before += total;
        k.base += 32;
        if (k.base >= p.num_seqs) return make_int4(0, 0, 0, 0);
        prompt_walk_load(p, k, lane);
    }
    const int u = unit - k.before;
    const int src = __ffs(__ballot_sync(kFullMask, u < k.incl)) - 1;
    const int row0 = __shfl_sync(kFullMask, k.row0, src), len = __shfl_sync(kFullMask, k.len, src);
    const int incl = __shfl_sync(kFullMask, k.incl, src);
    return make_int4(row0, len, incl - 1 - u, index - unit * p.num_kv_heads);
}

__device__ __forceinline__ bool elect_one() {
    uint32_t lead;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(lead));
    return lead != 0;
}
// The counter's value before 1 is added (0 without a counter), and the entry of
// a unit (zeros past the list).  One block each, so that nothing but the use of
// the value waits for it.
__device__ __forceinline__ int take_item(int* counter) {
    int before;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u64 p, %1, 0;\n\t"
        "mov.b32 %0, 0;\n\t"
        "@p atom.relaxed.gpu.global.add.s32 %0, [%1], 1;\n\t}"
        : "=&r"(before)
        : "l"(counter)
        : "memory");
    return before;
}
__device__ __forceinline__ int4 load_unit(const int4* unit, bool listed) {
    int4 e;  // not through L1: written after this grid was launched
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %5, 0;\n\t"
        "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.cg.v4.s32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(e.x), "=&r"(e.y), "=&r"(e.z), "=&r"(e.w)
        : "l"(unit), "r"((unsigned)listed)
        : "memory");
    return e;
}

template <class Shape>
__device__ void prompt_load(const PromptParams& p, typename Shape::Smem& sm, int lane, const CUtensorMap* tq,
                            const CUtensorMap* tk, const CUtensorMap* tv) {
    constexpr int HALF_BYTES = Shape::HALF * 128;
    const uint32_t q_bytes = (uint32_t)(Shape::SLABS * p.tile_tokens * p.group * 128);
    uint32_t q_used = 0, q_loaded = 0;  // bit i: parity of the loads of Q_i, whether there was one
    uint32_t slot = 0, round = 0, filled = 0;
    const int total = p.items ? __ldcg(p.num_units) * p.num_kv_heads : 0;
    bool ok = true;
    auto listed = [&](int index) {
        const int unit = index / p.num_kv_heads;
        int4 e = load_unit(p.items + unit, index < total);
        e.w = index - unit * p.num_kv_heads;
        return e;
    };
    int4 next;
    if (p.items) {
        next = listed(blockIdx.x);
    } else {
        // Sequences that overlap make more items than the grid has CTAs: none is
        // computed, as with a list.
        PromptWalk walk{};
        long long rows = 0;
        for (walk.base = 0; walk.base < p.num_seqs; walk.base += 32) {
            prompt_walk_load(p, walk, lane);
            // 32 lengths of at most num_tokens each, which is below 2 * tile_tokens * SMs
            // without a list: some 38 000, the sum far below 2^31.
            rows += __reduce_add_sync(kFullMask, walk.len);
        }
        if (rows > p.num_tokens) {
            set_error(p.err, PA_DEVERR_CONTEXT_LEN);
            next = make_int4(0, 0, 0, 0);
        } else {
            walk.base = 0;
            prompt_walk_load(p, walk, lane);
            next = prompt_walk_to(p, walk, lane, blockIdx.x);
        }
    }
    // The whole warp runs the loop and one elected lane issues (as the MMA warps
    // do): a copy issued inside `if (lane == 0)` waited for its operands, and short
    // items come as fast as their copies are issued (many prompts of at most 130
    // tokens: 37.7 us so, 35.5 with the elected lane).
    for (int n = 0;; ++n) {
        const int4 it = next;
        const int st = n % Shape::NITEM;
        // The next item's number and entry arrive while this one's copies are
        // issued and waited for: 3000 cycles an item when they did not.
        int taken = 0;
        prompt_wait(p, sm, &sm.item_empty[st], ((uint32_t)(n / Shape::NITEM) & 1u) ^ 1u);
        if (__any_sync(kFullMask, prompt_aborted(&sm.abort_flag))) break;
        if (elect_one()) {
            sm.item[st] = it;
            mbar_arrive(&sm.item_full[st]);
        }
        __syncwarp();
        if (it.y == 0) break;
        const PromptItem w = prompt_item(it, p.tile_tokens);
        const int end = w.last(), nt = (end + 127) >> 7;
        // K_0, Q_0, V_0, Q_1, K_1, V_1, ...: what the item before does not hold up first
#pragma unroll 1
        for (int t = 0; t < 2 * nt; ++t) {
            // One K or V tile, in halves of 64 positions.
            const bool is_v = t & 1;
            const int j = t >> 1, row = w.row0 + j * Shape::BN;
            prompt_wait(p, sm, &sm.kv_empty[slot], round ^ 1u);
            ok = !__any_sync(kFullMask, prompt_aborted(&sm.abort_flag));
            if (!ok) break;
            if (t == 2 * nt - 2) taken = take_item(lane == 0 ? p.next_item : nullptr);
            const int halves = end - j * Shape::BN > Shape::HALF ? 2 : 1;
            const CUtensorMap* map = is_v ? tv : tk;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sm.kv_full[slot], (uint32_t)(halves * Shape::SLABS * HALF_BYTES));
#pragma unroll 1
                for (int h = 0; h < halves; ++h)
#pragma unroll
                    for (int s = 0; s < Shape::SLABS; ++s)
                        tma_load_3d_plain(sm.kv[slot][s] + h * HALF_BYTES, map, s * 64, w.kv_head,
                                          row + h * Shape::HALF, &sm.kv_full[slot]);
                if (is_v && j >= w.first_masked) mbar_arrive(&sm.check_go[slot]);
            }
            __syncwarp();
            filled |= 1u << slot;
            if (++slot == Shape::NSLOT) {
                slot = 0;
                round ^= 1u;
            }
            if (t < 2 && w.end(t)) {
                prompt_wait(p, sm, &sm.q_empty[t], ((q_used >> t) & 1u) ^ 1u);
                ok = !__any_sync(kFullMask, prompt_aborted(&sm.abort_flag));
                if (!ok) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&sm.q_full[t], q_bytes);
#pragma unroll
                    for (int s = 0; s < Shape::SLABS; ++s)
                        tma_load_3d_plain(sm.q[t][s], tq, s * 64, w.kv_head * p.group,
                                          w.row0 + w.t0 + t * p.tile_tokens, &sm.q_full[t]);
                }
                __syncwarp();
                q_used ^= 1u << t;
                q_loaded |= 1u << t;
            }
            if (t == 2 * nt - 1) next = listed((int)gridDim.x + __shfl_sync(kFullMask, taken, 0));
        }
        if (!ok) break;
    }
    pdl_launch_dependents();
    if (lane == 0) {
        // Every copy this warp issued lands before the CTA exits (bounded).
        bool drained = true;
#pragma unroll 1
        for (int i = 0; i < 2; ++i)
            if (q_loaded & (1u << i))
                drained = mbar_wait_bounded(&sm.q_full[i], ((q_used >> i) & 1u) ^ 1u, p.wait_limit_ns) && drained;
#pragma unroll 1
        for (uint32_t s = 0; s < Shape::NSLOT; ++s)
            if (filled & (1u << s))
                drained = mbar_wait_bounded(&sm.kv_full[s], s < slot ? round : round ^ 1u, p.wait_limit_ns) && drained;
        if (!drained) set_error(p.err, PA_DEVERR_TIMEOUT);
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------
// MMA issuer of query tile i (one warp)
// ---------------------------------------------------------------------------
// The whole warp runs the issue loop and one elected lane issues: descriptors
// then stay in uniform registers.  With the loop inside `if (lane == 0)` every
// MMA waited for its operands to be moved there, about 115 cycles an MMA
// against the 64 that it runs for.
__device__ __forceinline__ void commit_at(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// The operands' descriptors (smem_desc_sw128) differ in their lower halves only:
// stride 1024 bytes, version 1, 128-byte swizzle above.  Addresses / 16 stay
// below 2^14, so a step never carries out of its field.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool first) {
    asm volatile(
        "{\n\t.reg .b64 a, b;\n\t.reg .pred acc;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 acc, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, acc;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(first ? 0u : 1u), "n"(kDescHi)
        : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool first) {
    asm volatile(
        "{\n\t.reg .b64 b;\n\t.reg .pred acc;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 acc, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, acc;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(first ? 0u : 1u), "n"(kDescHi)
        : "memory");
}

template <class Shape, bool BF16>
__device__ void prompt_mma(const PromptParams& p, typename Shape::Smem& sm, uint32_t tmem, int i, int lane) {
    using Smem = typename Shape::Smem;
    constexpr int D = Shape::SLABS * 64;
    constexpr uint32_t IDESC_O = mma_idesc_f16(BF16, true, Shape::BM, D);
    constexpr uint32_t IDESC_S = mma_idesc_f16(BF16, false, Shape::BM, 128);
    constexpr uint32_t IDESC_S64 = mma_idesc_f16(BF16, false, Shape::BM, 64);
    constexpr uint32_t SLOT16 = sizeof(sm.kv[0]) >> 4, Q16 = sizeof(sm.q[0]) >> 4;
    const uint32_t base = smem_addr(&sm);
    const uint32_t q_lo = (uint32_t)smem_desc_sw128(base + offsetof(Smem, q), 16, 1024);
    const uint32_t k_lo = (uint32_t)smem_desc_sw128(base + offsetof(Smem, kv), 16, 1024);
    const uint32_t v_lo = (uint32_t)smem_desc_sw128(base + offsetof(Smem, kv), Shape::SLAB, 1024);
    auto bar = [&](size_t member, uint32_t index) { return base + (uint32_t)member + 8u * index; };
    auto wait = [&](uint32_t at, uint32_t parity) { prompt_wait_at(p, sm, at, parity); };

    // For the elected lane: S = Q K^T over the K tile's first half or all of it.
    const uint32_t s_tmem = tmem + i * Shape::BN, o_tmem = tmem + Shape::O_COL + i * D, qi_lo = q_lo + i * Q16;
    auto issue_s = [&](uint32_t slot, bool whole) {
        const uint32_t idesc = whole ? IDESC_S : IDESC_S64, b = k_lo + slot * SLOT16;
#pragma unroll
        for (int ks = 0; ks < Shape::SLABS * 4; ++ks) {
            const uint32_t off = (uint32_t)((ks >> 2) * (Shape::SLAB >> 4) + (ks & 3) * 2);
            mma_ss_lo(s_tmem, qi_lo + off, b + off, idesc, ks == 0);
        }
        commit_at(bar(offsetof(Smem, s_full), i));
    };
    // O (+)= P V over one half (64) of the V tile's positions.
    auto issue_pv = [&](uint32_t slot, int half, bool first) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            mma_ts_lo(o_tmem, s_tmem + half * 32 + ks * 8, v_lo + slot * SLOT16 + half * 512 + ks * 128, IDESC_O,
                      first && ks == 0);
    };

    uint32_t slot = 0, round = 0;         // ring position of the next tile, parity of its round
    uint32_t nq = 0, no = 0, np = 0;      // parities of the tile's Q, O and P so far
    uint32_t turn = i ^ 1;                // parity of the turn to wait for: the other warp's last one
    uint32_t checked = 0;                 // bit slot: of the slot's checked V tiles so far
    auto advance = [&] {
        if (++slot == Shape::NSLOT) {
            slot = 0;
            round ^= 1u;
        }
    };
    int n = 0;
    PromptItem w;
    bool more = prompt_next_item<Shape>(p, sm, lane, n, w);
    if (more) {
        wait(bar(offsetof(Smem, kv_full), slot), round);
        if (w.end(i)) wait(bar(offsetof(Smem, q_full), i), nq++);
        if (elect_one()) {
            if (w.end(i)) issue_s(slot, w.end(i) > 64);
            if (w.tiles(i) == 1) commit_at(bar(offsetof(Smem, q_empty), i));
            commit_at(bar(offsetof(Smem, kv_empty), slot));
        }
        __syncwarp();
        advance();
    }
    // A step: O += P V_j and S of the next K tile, which after an item's last step
    // is the first one of the next item.
    while (more) {
        const int nt = (w.last() + 127) >> 7;
        PromptItem next = w;
#pragma unroll 1
        for (int j = 0; j < nt; ++j) {
            const uint32_t vslot = slot;
            if (j >= w.first_masked) {
                wait(bar(offsetof(Smem, v_checked), vslot), (checked >> vslot) & 1u);
                checked ^= 1u << vslot;
            } else {
                wait(bar(offsetof(Smem, kv_full), vslot), round);
            }
            advance();
            const uint32_t kslot = slot, kround = round;
            const bool last = j + 1 == nt;
            if (last) more = prompt_next_item<Shape>(p, sm, lane, n, next);
            const bool has_k = !last || more;
            if (has_k) {
                wait(bar(offsetof(Smem, kv_full), kslot), kround);
                advance();
            }
            // Positions of the item from V_j on, and of what K is the tile of (<= 0: none).
            const int left = w.end(i) - j * Shape::BN;
            const bool leaves = last && more && next.end(i) > 0;
            const int left_k = last ? (leaves ? next.end(i) : 0) : left - Shape::BN;
            if (left > 0) {
                if (j == 0) wait(bar(offsetof(Smem, o_empty), i), (no++ & 1u) ^ 1u);  // read by the output warps
                wait(bar(offsetof(Smem, p_full), 2 * i), np & 1u);
            }
            // The two warps take turns: the tensor cores get one query tile's step
            // while the other's softmax runs.  What a warp does between its steps is
            // hidden behind the other's MMAs.
            wait(bar(offsetof(Smem, turn), i), turn & 1u);
            ++turn;
            if (left > 0) {
                tc_fence_after_sync();
                if (elect_one()) issue_pv(vslot, 0, j == 0);
                __syncwarp();
                wait(bar(offsetof(Smem, p_full), 2 * i + 1), np++ & 1u);
                tc_fence_after_sync();
            }
            if (leaves) wait(bar(offsetof(Smem, q_full), i), nq++ & 1u);
            if (elect_one()) {
                if (left > 64) issue_pv(vslot, 1, false);
                if (left > 0 && left <= Shape::BN) commit_at(bar(offsetof(Smem, o_full), i));
                if (left_k > 0) issue_s(kslot, left_k > 64);
                mbar_arrive(&sm.turn[i ^ 1]);
                if (left_k > 0 && left_k <= Shape::BN) commit_at(bar(offsetof(Smem, q_empty), i));
                commit_at(bar(offsetof(Smem, kv_empty), vslot));
                if (has_k) commit_at(bar(offsetof(Smem, kv_empty), kslot));
            }
            __syncwarp();
        }
        w = next;
    }
    // Nothing this warp issued may still be running when TMEM is released.
    if (elect_one()) commit_at(bar(offsetof(Smem, mma_done), i));
    __syncwarp();
    if (lane == 0 && !mbar_wait_bounded(&sm.mma_done[i], 0, p.wait_limit_ns)) set_error(p.err, PA_DEVERR_TIMEOUT);
    __syncwarp();
}

// ---------------------------------------------------------------------------
// softmax warps of query tile i (thread r = row r = TMEM lane r)
// ---------------------------------------------------------------------------
// 64 columns of this thread's TMEM lane, not waited for.  The registers hold
// nothing before tmem_wait_ld(r), which names them so that no use moves ahead.
__device__ __forceinline__ void tmem_ld_x64_async(uint32_t taddr, float (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];"
        : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]), "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]), "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]), "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31]), "=f"(r[32]), "=f"(r[33]), "=f"(r[34]), "=f"(r[35]), "=f"(r[36]), "=f"(r[37]), "=f"(r[38]), "=f"(r[39]), "=f"(r[40]), "=f"(r[41]), "=f"(r[42]), "=f"(r[43]), "=f"(r[44]), "=f"(r[45]), "=f"(r[46]), "=f"(r[47]), "=f"(r[48]), "=f"(r[49]), "=f"(r[50]), "=f"(r[51]), "=f"(r[52]), "=f"(r[53]), "=f"(r[54]), "=f"(r[55]), "=f"(r[56]), "=f"(r[57]), "=f"(r[58]), "=f"(r[59]), "=f"(r[60]), "=f"(r[61]), "=f"(r[62]), "=f"(r[63])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(float (&r)[64]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(r[0]), "+f"(r[1]), "+f"(r[2]), "+f"(r[3]), "+f"(r[4]), "+f"(r[5]), "+f"(r[6]), "+f"(r[7]), "+f"(r[8]), "+f"(r[9]), "+f"(r[10]), "+f"(r[11]), "+f"(r[12]), "+f"(r[13]), "+f"(r[14]), "+f"(r[15]), "+f"(r[16]), "+f"(r[17]), "+f"(r[18]), "+f"(r[19]), "+f"(r[20]), "+f"(r[21]), "+f"(r[22]), "+f"(r[23]), "+f"(r[24]), "+f"(r[25]), "+f"(r[26]), "+f"(r[27]), "+f"(r[28]), "+f"(r[29]), "+f"(r[30]), "+f"(r[31]), "+f"(r[32]), "+f"(r[33]), "+f"(r[34]), "+f"(r[35]), "+f"(r[36]), "+f"(r[37]), "+f"(r[38]), "+f"(r[39]), "+f"(r[40]), "+f"(r[41]), "+f"(r[42]), "+f"(r[43]), "+f"(r[44]), "+f"(r[45]), "+f"(r[46]), "+f"(r[47]), "+f"(r[48]), "+f"(r[49]), "+f"(r[50]), "+f"(r[51]), "+f"(r[52]), "+f"(r[53]), "+f"(r[54]), "+f"(r[55]), "+f"(r[56]), "+f"(r[57]), "+f"(r[58]), "+f"(r[59]), "+f"(r[60]), "+f"(r[61]), "+f"(r[62]), "+f"(r[63])
                 :
                 : "memory");
}
// Issue a store of 16 columns; tmem_wait_st() waits for all stores issued.
__device__ __forceinline__ void tmem_st_x16_async(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
                 :
                 : "r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// 16 columns of this thread's accumulator lane, times a.
__device__ __forceinline__ void prompt_scale16(uint32_t addr, float a) {
    uint32_t u[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(__uint_as_float(u[k]) * a);
    tmem_st_x16_async(addr, u);
}

// Positions after `own` (-inf: no weight).
__device__ __forceinline__ void mask64(float (&x)[64], int own) {
#pragma unroll
    for (int k = 0; k < 64; ++k) x[k] = k <= own ? x[k] : __int_as_float(0xff800000);
}

template <typename T, class Shape>
__device__ void prompt_softmax(const PromptParams& p, typename Shape::Smem& sm, uint32_t tmem, int i, int warp,
                               int lane) {
    constexpr int D = Shape::SLABS * 64;
    const int r = warp * 32 + lane;
    const int t = r / p.group;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t s_addr = tmem + lanes + i * Shape::BN, o_addr = tmem + lanes + Shape::O_COL + i * D;
    const float c = p.scale_log2;  // > 0
    const float NEG_INF = __int_as_float(0xff800000);
    uint32_t ns = 0, used = 0;     // S_i and items so far
    int n = 0;
    PromptItem w;
    while (prompt_next_item<Shape>(p, sm, lane, n, w)) {
        const int end = w.end(i), nt = w.tiles(i);
        if (!nt) continue;
        const int token = w.t0 + i * p.tile_tokens + t;
        // Rows past the tile's tokens compute something and are not stored.
        const int last = t < p.tile_tokens && token < w.len ? token : end - 1;
        float m = NEG_INF, l = 0.f;
        for (int j = 0; j < nt; ++j, ++ns) {
            prompt_wait(p, sm, &sm.s_full[i], ns & 1u);
            tc_fence_after_sync();
            float x0[64], x1[64];  // scores of positions kv0 .. kv0 + 63, kv0 + 64 .. kv0 + 127
            const int kv0 = j * Shape::BN;
            const int cols = min(Shape::BN, end - kv0);
            // The second half loads while the first one's maximum is taken.
            tmem_ld_x64_async(s_addr, x0);
            tmem_wait_ld(x0);
            tmem_ld_x64_async(s_addr + 64, x1);
            const int own = j >= w.first_masked ? last - kv0 : Shape::BN;
            float pm[8];
            if (own < 63) mask64(x0, own);
#pragma unroll
            for (int q = 0; q < 8; ++q) pm[q] = fmaxf(x0[q], x0[q + 8]);
#pragma unroll
            for (int k = 16; k < 64; k += 16)
#pragma unroll
                for (int q = 0; q < 8; ++q) pm[q] = max3(pm[q], x0[k + q], x0[k + q + 8]);
            tmem_wait_ld(x1);
            if (own < 127) mask64(x1, own - 64);
#pragma unroll
            for (int k = 0; k < 64; k += 16)
#pragma unroll
                for (int q = 0; q < 8; ++q) pm[q] = max3(pm[q], x1[k + q], x1[k + q + 8]);
            const float mx = max3(max3(pm[0], pm[1], pm[2]), max3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
            const float m_new = fmaxf(m, mx * c);
            const bool grow = m_new > m + 8.f;  // always on the first tile (m = -inf)
            float alpha = 1.f;
            if (grow) {
                alpha = prompt_exp2(m - m_new);
                m = m_new;
                l *= alpha;
            }
            // A grown maximum rescales O_i: S_i was issued after P_i V of the tile
            // before, by the same thread, so that has completed too.
            if (j > 0 && __any_sync(kFullMask, grow)) {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) prompt_scale16(o_addr + c0, alpha);
                tmem_wait_st();
            }
            // P in four pieces of 32 positions; P.V starts on the first half
            // while the second is made.
            constexpr float LARGER = std::is_same<T, __half>::value ? 7.f : 0.f;
            const float nm = m > NEG_INF ? LARGER - m : 0.f;  // no weight for scores of -inf alone
            float ps[4] = {0.f, 0.f, 0.f, 0.f};
            auto piece = [&](float* x, uint32_t addr) {
                uint32_t u[16];
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                    fma2_rn(x[k], x[k + 1], c, c, nm, nm);
                    x[k] = prompt_exp2(x[k]);
                    x[k + 1] = prompt_exp2(x[k + 1]);
                    add2_rn(ps[k & 2], ps[(k & 2) + 1], x[k], x[k + 1]);
                    u[k >> 1] = pack_rn<T>(x[k], x[k + 1]);
                }
                tmem_st_x16_async(addr, u);
            };
            auto written = [&](int half) {
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[i][half]);
            };
            piece(x0, s_addr);
            piece(x0 + 32, s_addr + 16);
            written(0);
            if (cols > 64) {
                piece(x1, s_addr + 32);
                piece(x1 + 32, s_addr + 48);
            }
            written(1);
            l += (ps[0] + ps[1]) + (ps[2] + ps[3]);
        }
        // The row sums, once the output warps have read the previous item's.
        prompt_wait(p, sm, &sm.o_empty[i], (used & 1u) ^ 1u);
        ++used;
        sm.row_sum[i][r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.l_full[i]);
    }
}

// ---------------------------------------------------------------------------
// check warp: V tiles with masked positions
// ---------------------------------------------------------------------------
// Not 0 where a 16-bit half of w is infinite or NaN: an exponent of all ones
// carries into the half's sign bit.
template <typename T>
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    else
        return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
}

// 0 * w + a on both 16-bit halves.
template <typename T>
__device__ __forceinline__ uint32_t times_zero_plus(uint32_t w, uint32_t a) {
    uint32_t d;
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(a));
    else
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w), "r"(0u), "r"(a));
    return d;
}

template <typename T, class Shape>
__device__ void prompt_check(const PromptParams& p, typename Shape::Smem& sm, int lane) {
    constexpr int CHUNKS = Shape::SLABS * 8;  // 16-byte chunks of a row
    constexpr int STEP = 32 / CHUNKS;         // rows of one pass of the warp
    const int my_chunk = lane % CHUNKS, my_row = lane / CHUNKS;
    uint32_t tiles = 0;   // ring tiles before the item
    uint32_t parity = 0;  // per slot: of its next masked V tile
    int n = 0;
    PromptItem w;
    while (prompt_next_item<Shape>(p, sm, lane, n, w)) {
        const int end = w.last(), nt = (end + 127) >> 7;
        for (int j = w.first_masked; j < nt; ++j) {
            const uint32_t tile = tiles + 2 * j + 1;  // K_0, V_0, K_1, ...
            const uint32_t slot = tile % Shape::NSLOT;
            // Issued first: before that the slot's barrier may still be two
            // phases back, which its parity does not tell from complete.
            prompt_wait(p, sm, &sm.check_go[slot], (parity >> slot) & 1u);
            prompt_wait(p, sm, &sm.kv_full[slot], (tile / Shape::NSLOT) & 1u);
            parity ^= 1u << slot;
            // Rows up to the item's first token are attended by all its rows.
            const int first = max(w.t0 + 1 - j * Shape::BN, 0);
            const int rows = min(Shape::BN, end - j * Shape::BN), all = (rows + 63) & ~63;
            // This lane's chunk of rows lane / CHUNKS, + STEP, ...
            uint8_t* const column = sm.kv[slot][my_chunk >> 3] + (my_chunk & 7) * 16;
            auto at = [&](int row) { return reinterpret_cast<uint4*>(column + row * 128); };
            for (int row = rows + my_row; row < all; row += STEP) *at(row) = make_uint4(0u, 0u, 0u, 0u);
            // 0 * v: NaN where v is infinite or NaN, and then for good in the sum.
            uint32_t acc[4] = {0u, 0u, 0u, 0u};
#pragma unroll 8
            for (int row = first + my_row; row < rows; row += STEP) {
                const uint4 v = *at(row);
                acc[0] = times_zero_plus<T>(v.x, acc[0]);
                acc[1] = times_zero_plus<T>(v.y, acc[1]);
                acc[2] = times_zero_plus<T>(v.z, acc[2]);
                acc[3] = times_zero_plus<T>(v.w, acc[3]);
            }
            if ((acc[0] | acc[1] | acc[2] | acc[3]) & 0x7fff7fffu) {
#pragma unroll 1
                for (int row = first + my_row; row < rows; row += STEP) {
                    uint32_t* v = reinterpret_cast<uint32_t*>(at(row));
#pragma unroll 1
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t bad = nonfinite2<T>(v[e]);
                        v[e] &= ~(((bad >> 31) * 0xffff0000u) | ((bad >> 15 & 1u) * 0xffffu));
                    }
                }
                atomicMax(&sm.last_dirty, n - 1);  // n: items announced so far
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.v_checked[slot]);
        }
        tiles += 2 * nt;
    }
}

// ---------------------------------------------------------------------------
// output warps
// ---------------------------------------------------------------------------
// The non-finite values that the check warp took out of V tiles: each decides
// its column of the rows that attend it.  Added to the stored output `dst` of
// the row of `token` by the thread that stored it.
template <typename T, int D>
__device__ __noinline__ void prompt_add_nonfinite(const PromptParams& p, const PromptItem& w, int token, T* dst) {
    const T* v = static_cast<const T*>(p.value) + (int64_t)w.kv_head * D;
    for (int j = w.t0 + 1; j <= token; ++j) {
        const T* row = v + (int64_t)(w.row0 + j) * p.value_stride;
        for (int c = 0; c < D; ++c) {
            const float x = (float)row[c];
            if (!isfinite(x)) dst[c] = (T)((float)dst[c] + x);
        }
    }
}

// A whole sector of a row by one thread: the rows of a warp are far apart, and
// 16-byte stores take twice as many passes of the memory pipeline, which the
// softmax warps' TMEM accesses share (32 prompts of 128-1024 tokens: 144 us; 133
// with 32 bytes; 128 to 122 without a line in L1).
__device__ __forceinline__ void store_32_bytes(void* dst, const uint32_t (&q)[8]) {
    asm volatile("st.global.L1::no_allocate.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(q[0]), "r"(q[1]), "r"(q[2]),
                 "r"(q[3]), "r"(q[4]), "r"(q[5]), "r"(q[6]), "r"(q[7])
                 : "memory");
}

// Two means of values, rounded.  A mean passes none of its values, but weights that
// were rounded up may carry one of f16 values next to the type's end beyond it
// (65504 (1 + 2^-11) rounds to infinity): a mean beyond the end is the type's largest
// value here, which an infinite one becomes as well (below).  bf16 values so large
// pass the end of binary32 in the sums first.
template <typename T>
__device__ __forceinline__ uint32_t pack_mean(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) {
        uint32_t w;
        asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
        return w;
    }
    return pack_rn<T>(a, b);
}

template <typename T, class Shape>
__device__ void prompt_output(const PromptParams& p, typename Shape::Smem& sm, uint32_t tmem, int warp, int lane) {
    constexpr int D = Shape::SLABS * 64;
    constexpr bool F16 = std::is_same<T, __half>::value;
    const int r = warp * 32 + lane;
    const int t = r / p.group, g = r - t * p.group;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    uint32_t parity = 0;  // bit i: of the next O_i
    int n = 0;
    PromptItem w;
    while (prompt_next_item<Shape>(p, sm, lane, n, w)) {
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            if (!w.end(i)) continue;
            prompt_wait(p, sm, &sm.l_full[i], (parity >> i) & 1u);
            prompt_wait(p, sm, &sm.o_full[i], (parity >> i) & 1u);
            parity ^= 1u << i;
            tc_fence_after_sync();
            // A wait that ran out left no result: the rows stay as they were.
            const bool aborted = prompt_aborted(&sm.abort_flag);
            const float l = sm.row_sum[i][r];
            const float inv = 1.f / l;  // l > 0: every row attends its own position (NaN stays NaN)
            const int token = w.t0 + i * p.tile_tokens + t;
            const bool store = t < p.tile_tokens && token < w.len && !aborted;
            const bool dirty = *reinterpret_cast<volatile int*>(&sm.last_dirty) >= n - 1;
            T* dst = static_cast<T*>(p.out) +
                     ((int64_t)(w.row0 + token) * p.num_heads + (int64_t)w.kv_head * p.group + g) * D;
            auto read = [&] {  // O_i may be written again
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.o_empty[i]);
            };
            // f16: the sums of the row's even and odd columns are not finite where one of
            // them is not; such a row's infinite means are stored again.  (16 columns at
            // a time, which leaves registers for the sums: 80.5 us for 16 prompts of
            // 128-1024 tokens of 40 heads; 82 with 32 columns, 79.4 without the check.)
            float all0 = 0.f, all1 = 0.f;
            bool again = false;
            constexpr int C = F16 ? 16 : 32;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += C) {
                uint32_t u[C];
                if constexpr (F16) {
                    tmem_ld_x16(tmem + lanes + Shape::O_COL + i * D + c0, u);
#pragma unroll
                    for (int k = 0; k < 16; k += 2)
                        add2_rn(all0, all1, __uint_as_float(u[k]), __uint_as_float(u[k + 1]));
                } else {
                    tmem_ld_x32(tmem + lanes + Shape::O_COL + i * D + c0, u);
                }
                if (c0 + C == D) {
                    if constexpr (F16) again = __any_sync(kFullMask, store && !isfinite(all0 + all1));
                    if (!again) read();
                }
                if (store) {
#pragma unroll
                    for (int k = 0; k < C; k += 16) {
                        uint32_t q[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            q[e] = pack_mean<T>(__uint_as_float(u[k + 2 * e]) * inv,
                                                __uint_as_float(u[k + 2 * e + 1]) * inv);
                        store_32_bytes(dst + c0 + k, q);
                    }
                }
            }
            if constexpr (F16) {
                if (again) {
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 2) {
                        float x0, x1;
                        asm volatile(
                            "tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];\n\t"
                            "tcgen05.wait::ld.sync.aligned;"
                            : "=f"(x0), "=f"(x1)
                            : "r"(tmem + lanes + Shape::O_COL + i * D + c0)
                            : "memory");
                        x0 *= inv, x1 *= inv;
                        if (store && isinf(x0)) dst[c0] = (T)x0;
                        if (store && isinf(x1)) dst[c0 + 1] = (T)x1;
                    }
                    read();
                }
            }
            if (store && dirty) prompt_add_nonfinite<T, D>(p, w, token, dst);
        }
    }
}

// ---------------------------------------------------------------------------
// the kernel: one CTA per SM
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(PromptShape<D>::THREADS, 1)
    prompt_kernel(const PromptParams p, const __grid_constant__ CUtensorMap tmap_q,
                  const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
    using Shape = PromptShape<D>;
    using Smem = typename Shape::Smem;
    extern __shared__ uint8_t prompt_smem_raw[];
    const uintptr_t a = reinterpret_cast<uintptr_t>(prompt_smem_raw);
    Smem& sm = *reinterpret_cast<Smem*>((a + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        prefetch_tensormap(&tmap_q);
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
        for (int s = 0; s < Shape::NITEM; ++s) {
            mbar_init(&sm.item_full[s], 1);
            mbar_init(&sm.item_empty[s], Shape::ITEM_READERS);
        }
        for (int s = 0; s < Shape::NSLOT; ++s) {
            mbar_init(&sm.kv_full[s], s == 0 && (p.debug_flags & kDebugDropFirstFill) ? 2 : 1);
            mbar_init(&sm.kv_empty[s], 2);
            mbar_init(&sm.check_go[s], 1);
            mbar_init(&sm.v_checked[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.turn[i], 1);
            mbar_init(&sm.mma_done[i], 1);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i][0], Shape::SOFTMAX_WARPS);
            mbar_init(&sm.p_full[i][1], Shape::SOFTMAX_WARPS);
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.l_full[i], Shape::SOFTMAX_WARPS);
            mbar_init(&sm.o_empty[i], 4);
        }
        sm.abort_flag = 0;
        sm.last_dirty = -1;
        fence_mbar_init();
    }
    __syncwarp();  // the allocation is one instruction of the whole warp
    if (warp == Shape::MMA_WARP) tmem_alloc(&sm.tmem_base, Shape::TMEM_COLS);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    // The kernel that wrote the start rows, q, k and v may still be finishing.
    pdl_wait_prerequisites();

    if (warp < Shape::SOFTMAX_WARP) {
        regs_dec<Shape::REGS_OTHER>();
        if (warp < Shape::LOAD_WARP)
            prompt_mma<Shape, std::is_same<T, __nv_bfloat16>::value>(p, sm, tmem, warp, lane);
        else if (warp == Shape::LOAD_WARP)
            prompt_load<Shape>(p, sm, lane, &tmap_q, &tmap_k, &tmap_v);
        else
            prompt_check<T, Shape>(p, sm, lane);
    } else if (warp < Shape::OUT_WARP) {
        regs_inc<Shape::REGS_SOFTMAX>();
        const int v = warp - Shape::SOFTMAX_WARP;
        prompt_softmax<T, Shape>(p, sm, tmem, v >> 2, v & 3, lane);
    } else {
        regs_dec<Shape::REGS_OUT>();
        prompt_output<T, Shape>(p, sm, tmem, warp - Shape::OUT_WARP, lane);
    }

    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (threadIdx.x == 0 && sm.abort_flag) set_error(p.err, PA_DEVERR_TIMEOUT);
    __syncwarp();
    if (warp == Shape::MMA_WARP) tmem_dealloc(tmem, Shape::TMEM_COLS);
}

}  // namespace pa
