// tree_attn.cuh -- attention of the nodes of drafted trees over the paged cache,
// on the Blackwell tensor cores (tcgen05.mma, accumulators in tensor memory).
//
// What it computes: the attention equation ("PagedAttention 论文精读笔记", §2.1)
// through the block tables (§5.2), for the n nodes of each sequence's tree, the
// last n of its ctx cached tokens.  Node i attends to the positions before the
// tree and to the nodes of its mask row:
//     out[i][h] = sum_j softmax_j(scale * q[i][h] . k_j) v_j,
//     j < ctx - n, or j = ctx - n + m with bit m of tree_mask[i].
//
// Work: a query tile is 128 rows (row = node * G + grouped head), 128 / G nodes.
// An item is up to two query tiles of one (sequence, KV head) over its K/V tiles
// of 128 positions.  The K/V tiles of all items stand in one list (pairs of query
// tiles outermost, so that what reads the same keys runs at the same time; then
// sequences, KV heads, tiles), and each CTA -- one per SM -- takes an equal,
// contiguous piece of it.  So every SM has the same work whatever the lengths, and
// only an item that lies across a border between CTAs is computed in parts: at most
// two per CTA, which the reduce kernel joins.  The list is never written: each CTA
// finds its piece by a prefix sum over the lengths.  Pieces are counted in half tiles,
// and an item begins with LEAD of them for what it costs beside its tiles: its first
// copies, the tile with the nodes, the outputs -- some 2 us, a tile of 64 KiB 1.43 us at
// the memory's rate.  (24 sequences of 128 to 2048 tokens of 40 KV heads: 121.7 us with a
// LEAD of 1, when CTAs of short sequences ended at 126 us and the others at 98; 117.4 with
// 2, 110.4 with 3.)
//
// Per K/V tile j and query tile:
//   S  = Q K_j^T      tcgen05.mma M=128 N=128 K=d, into TMEM
//   P  = 2^(S c - m)  softmax warps, one thread per row; P, rounded to the pools'
//                     16-bit type, is written over S
//   O += P V_j        tcgen05.mma with A = P from TMEM
// with c = scale * log2 e, the running maximum m in base-2 units, O rescaled only
// when a row's maximum grows by more than 8, row sums in binary32 over the
// unrounded weights.  In f16 all weights are 2^7 larger, which keeps seven more bits
// of the small ones; the division by their sum takes it out again.  The rounding of
// P costs half a step of the type of the weighted sum of |v|, as much as the
// output's own.
//
// Two chains S -> P -> O run in turn on the tensor cores.  A sequence of more rows
// than one query tile has two (tile 0 and 1, each K/V tile is read by both).  One
// of fewer has its single query tile in both chains, which take the K/V tiles in
// turn (even, odd) and are joined at the end: a K/V tile then costs one chain's
// time, not two, and the chain (2700 cycles) is hidden behind the other one.
//
// Bound: HBM up to about 128 rows (2 d e bytes a position and KV head against 4 d
// flops a row and position), tensor cores above.  Measured (graph replay): 64 sequences
// of 16 nodes, lognormal contexts up to 8192, 32/8 heads of 128, bf16: 93.8 us, 5.4
// TB/s; 32 of 40 to 64 nodes, 1024 to 8192 tokens: 152 us, 4.7 TB/s and 0.93 PFLOP/s at
// once; 24 of 1 to 25 nodes, 128 to 2048 tokens, 40/40 heads, f16: 111 us, 5.4 TB/s; 3 of
// 31 nodes and 30 to 33 thousand tokens, 16/4 heads of 64: 31.9 us, 3.1 TB/s.  One
// short sequence, all of it latency: 11.9 us (launch, the list's prefix sum, the first
// copies, S, softmax, P V, a part, the reduce kernel), which the others pay beside theirs.
//
// Values a row must not see: its weight is 0, but 0 * NaN is NaN on the tensor
// cores.  So before P V reads a V tile with positions of the tree, an MMA warp clears
// its rows after the context's end and replaces non-finite elements of nodes by 0;
// those are added again, to the rows that do attend them, by the output warps.
//
// K/V tiles in shared memory: [16 groups of 8 rows][d / 64 slabs][8 rows][128 bytes],
// 128-byte swizzle.  A (block, head) tile of the pool is one 4-D box of that
// (1 to 8 KiB), and both operands' descriptors take it: 8-row groups d / 64 KiB
// apart, slabs 1 KiB.
//
// Warp roles (512 threads, registers moved between the groups by setmaxnreg):
//   warps 0, 1       MMA issuers of chain 0 / 1, and while P is made, what the V tiles with
//                    nodes need (above); warp 0 owns the TMEM allocation
//   warp 2           items, Q, K and V copies (TMA)
//   warp 3           V copies at head_dim 64, idle otherwise.  (A tile's copies cost a warp
//                    some 2500 cycles, as long as 64 KiB take but twice as long as 32 KiB:
//                    19 sequences of 8192 tokens with one warp 82 us, with two 62; at
//                    head_dim 128 two are no faster.)
//   warps 4-7, 8-11  softmax of chain 0 / 1
//   warps 12-15      outputs, or an item's part
// Every wait is bounded; a wait that runs out sets PA_DEVERR_TIMEOUT and makes
// every role of the CTA leave, after what it issued has landed.
#pragma once

#include "prompt.cuh"  // TMEM, MMA, packing and barrier helpers of the prompt attention
#include "tree.h"

namespace pa {

template <int D>
struct TreeShape {
    static constexpr int BM = 128;               // query rows per tile
    static constexpr int BN = 128;               // key/value positions per tile
    static constexpr int SLABS = D / 64;         // 64-element (128-byte) column slabs of a row
    static constexpr int Q_SLAB = 128 * 128;     // bytes of one slab of 128 query rows
    static constexpr int GROUP = SLABS * 1024;   // bytes of 8 rows of keys or values
    static constexpr int TILE = 16 * GROUP;      // bytes of a K or V tile
    static constexpr int NSLOT = D == 128 ? 5 : 10;  // K/V ring: K_0, V_0, K_1, V_1, ... one tile per slot
    static constexpr int NGO = 8;                // K tiles that their warp is ahead of the V tiles' warp, and more
    static constexpr int NITEM = 4;              // items announced ahead of their last reader
    static constexpr int LEAD = D == 128 ? 3 : 4;  // an item's cost beside its tiles, in half tiles
    static constexpr int SOFTMAX_WARPS = 4;      // per chain
    static constexpr int LOAD_WARP = 2;          // and the next one, if K and V have a warp each
    static constexpr bool TWO_LOADERS = D == 64;
    static constexpr int SOFTMAX_WARP = 4;       // first of eight
    static constexpr int OUT_WARP = 12;          // first of four
    static constexpr int THREADS = 512;
    static constexpr int ITEM_READERS = 8 + 4 + 2;  // softmax, output, MMA warps
    static constexpr int REGS_SOFTMAX = 168, REGS_OUT = 80, REGS_OTHER = 96;
    static_assert(256 * REGS_SOFTMAX + 128 * REGS_OUT + 128 * REGS_OTHER <= THREADS * 128, "register split");
    // TMEM columns: S of chain i (and P over it, two per column) at 128 i, O after both.
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t O_COL = 2 * BN;
    static_assert(D == 64 || D == 128, "head_dim 64 or 128");
    static_assert(LEAD <= kTreeMaxLead, "the host's bound of the list");

    struct Smem {
        alignas(1024) uint8_t q[2][SLABS][Q_SLAB];
        alignas(1024) uint8_t kv[NSLOT][TILE];
        float row_max[2][BM];
        float row_sum[2][BM];
        int4 item[NITEM][2];        // {first row, nodes (0: no more work), ctx, KV head}, {pair, tiles from, to, sequence}
        int last_dirty;             // latest item with non-finite values among its nodes
        int scratch[16];            // sums over the warps
        int start[3];               // where this CTA's piece begins: pair, sequence, half tile of the sequence
        int start_seq[3];           // that sequence's first row, nodes, ctx
        uint64_t item_full[NITEM];  // announced (load warp)
        uint64_t item_empty[NITEM]; // read by every role
        // Who waits for a barrier waits for each of its phases in turn: a parity does not
        // tell a phase from the one two before it.  So what both chains read and what
        // only chain 0 or 1 does have barriers of their own: [0], [1], and [2] for both.
        uint64_t q_one[2];          // query tile of both chains landed in buffer 0 / 1 (taken in turn)
        uint64_t q_pair[2];         // query tile of chain 0 / 1 landed
        uint64_t q_empty[2];        // last S of the item from buffer 0 / 1 complete (two arrivals)
        uint64_t k_full[3][NSLOT];  // tile landed
        uint64_t v_full[3][NSLOT];
        uint64_t kv_empty[NSLOT];   // the MMAs that read it complete (two arrivals, both by one chain if only it does)
        uint64_t k_go[NGO];         // the copy of a K tile was issued
        uint64_t v_checked[NSLOT];  // a V tile with nodes that both chains read is fit for P V (chain 0's warp)
        uint64_t s_full[2];         // S complete
        uint64_t p_full[2][2];      // each half of P written (softmax warps)
        uint64_t o_full[2];         // last P V of the item complete
        uint64_t l_full[2];         // row maxima and sums written (softmax warps)
        uint64_t o_empty[2];        // O, maxima and sums read (output warps)
        uint64_t mma_done[2];
        uint32_t tmem_base;
        int abort_flag;
    };
    // No slack to align the base by hand: there is no static shared memory, and the
    // array is declared with the alignment.
    static constexpr int SMEM_BYTES = (int)sizeof(Smem);
    static_assert(SMEM_BYTES <= 232448, "shared memory of one CTA");
};

// As prompt_wait: when the limit runs out, here or in another role, every wait of
// the CTA ends, the roles run on to the end of their item in shared and tensor
// memory only, and leave.
template <class Smem>
__device__ __forceinline__ void tree_wait(const TreeAttnParams& p, Smem& sm, uint64_t* bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return;
    const uint64_t start = global_timer_ns();
    do {
        if (prompt_aborted(&sm.abort_flag)) return;
        if (global_timer_ns() - start > p.wait_limit_ns) *reinterpret_cast<volatile int*>(&sm.abort_flag) = 1;
    } while (!mbar_try_wait(bar, parity));
}

// ---------------------------------------------------------------------------
// sequences and items
// ---------------------------------------------------------------------------
struct TreeSeq {
    int row0, n, ctx;
    int tiles;  // K/V tiles; 0: no nodes, or lengths that break the rules
    int pairs;  // pairs of query tiles
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeAttnParams& p, int s, bool report) {
    TreeSeq q{0, 0, 0, 0, 0};
    if (s >= p.num_seqs) return q;
    const int a = __ldcg(p.query_start + s), b = __ldcg(p.query_start + s + 1), ctx = __ldcg(p.context_lens + s);
    if (a < 0 || b < a || b > p.num_tokens || b - a > p.max_nodes || ctx < b - a || ctx > p.ctx_cap) {
        if (report) set_error(p.err, PA_DEVERR_CONTEXT_LEN);
        return q;
    }
    q.row0 = a;
    q.n = b - a;
    q.ctx = ctx;
    if (q.n > 0) {
        q.tiles = (ctx + 127) >> 7;
        q.pairs = (q.n + 2 * p.tile_tokens - 1) / (2 * p.tile_tokens);
    }
    return q;
}

struct TreeItem {
    int row0, n, ctx, kv_head, pair, from, to, seq;
    int t0;           // first node of query tile 0
    int base;         // position of the first node
    bool one;         // one query tile: both chains have it, and take the K/V tiles in turn
    int first_masked; // first K/V tile with a node
    __device__ __forceinline__ int tiles() const { return to - from; }
    __device__ __forceinline__ bool whole() const { return from == 0 && to == (ctx + 127) >> 7; }
    // Has chain i any tiles?
    __device__ __forceinline__ bool used(int i) const { return i == 0 || !one || to - from > 1; }
    __device__ __forceinline__ bool own(int i, int r) const { return !one || (r & 1) == i; }
    // Barriers of the item's r-th tile.
    __device__ __forceinline__ int readers(int r) const { return one ? r & 1 : 2; }
};

// Reader side of the item ring (one warp): the next item, or false at the end
// of the work or of the kernel.
template <class Shape>
__device__ __forceinline__ bool tree_next_item(const TreeAttnParams& p, typename Shape::Smem& sm, int lane, int& n,
                                               TreeItem& w) {
    const int st = n % Shape::NITEM;
    tree_wait(p, sm, &sm.item_full[st], (uint32_t)(n / Shape::NITEM) & 1u);
    if (__any_sync(kFullMask, prompt_aborted(&sm.abort_flag))) return false;
    const int4 a = sm.item[st][0], b = sm.item[st][1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.item_empty[st]);
    ++n;
    if (a.y == 0) return false;
    w.row0 = a.x, w.n = a.y, w.ctx = a.z, w.kv_head = a.w;
    w.pair = b.x, w.from = b.y, w.to = b.z, w.seq = b.w;
    w.t0 = w.pair * 2 * p.tile_tokens;
    w.base = w.ctx - w.n;
    w.one = w.n - w.t0 <= p.tile_tokens;
    w.first_masked = w.base >> 7;
    return true;
}

// ---------------------------------------------------------------------------
// the CTA's piece of the list (all threads)
// ---------------------------------------------------------------------------
__device__ __forceinline__ int tree_warp_sum(int x) { return (int)__reduce_add_sync(kFullMask, (unsigned)x); }

// Sum of x over the CTA, and the sum over the threads before this one.
__device__ inline int tree_block_scan(int x, int* scratch, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int up = __shfl_up_sync(kFullMask, incl, d);
        if (lane >= d) incl += up;
    }
    __syncthreads();  // the scratch of the call before has been read
    if (lane == 31) scratch[warp] = incl;
    __syncthreads();
    const int w = lane < 16 ? scratch[lane] : 0;
    total = tree_warp_sum(w);
    return incl - x + tree_warp_sum(lane < warp ? w : 0);
}

// Half tiles of an item, and the tiles that begin before half tile `at` of it.
template <class Shape>
__device__ __forceinline__ int tree_item_length(int tiles) { return 2 * tiles + Shape::LEAD; }
template <class Shape>
__device__ __forceinline__ int tree_tiles_before(int at) {
    return at <= Shape::LEAD ? 0 : (at - Shape::LEAD + 1) >> 1;
}

// The list's length, the CTAs that share it (two half tiles each at least, so that a
// piece within an item has a tile), and this CTA's piece [lo, hi); sm.start is where
// it begins.  Counts stay below 2^31 (the host checks the longest list).
struct TreePiece {
    int lo, hi, total, ctas;
    // The CTA that has half tile `at` of the list.
    __device__ __forceinline__ int cta_of(int at) const { return (int)((((long long)at + 1) * ctas - 1) / total); }
};
template <class Shape>
__device__ __forceinline__ TreePiece tree_piece(const TreeAttnParams& p, typename Shape::Smem& sm) {
    int mine = 0;
    TreeSeq q = tree_seq(p, threadIdx.x, blockIdx.x == 0);
    for (int s = threadIdx.x;; q = tree_seq(p, s, blockIdx.x == 0)) {
        if (q.tiles) mine += tree_item_length<Shape>(q.tiles) * q.pairs;
        s += Shape::THREADS;
        if (s - (int)threadIdx.x >= p.num_seqs) break;
    }
    // one loop turn: q is still this thread's only sequence
    const bool single = p.num_seqs <= Shape::THREADS;
    TreePiece w;
    const int rank = tree_block_scan(mine, sm.scratch, w.total);
    const bool one_pass = single && p.max_pairs == 1;  // the sums so far are the list's
    const int total_heads = w.total;
    w.total *= p.num_kv_heads;
    w.ctas = max(1, min(p.ctas, w.total / 2));
    w.lo = w.hi = 0;
    if ((int)blockIdx.x < w.ctas) {
        w.lo = (int)((long long)blockIdx.x * w.total / w.ctas);
        w.hi = (int)(((long long)blockIdx.x + 1) * w.total / w.ctas);
    }
    if (w.lo < w.hi) {
        int before = 0;  // of the list
        bool found = false;
        for (int pair = 0; pair < p.max_pairs && !found; ++pair)
            for (int s0 = 0; s0 < p.num_seqs && !found; s0 += Shape::THREADS) {
                if (!single) q = tree_seq(p, s0 + threadIdx.x, false);
                const int x = q.pairs > pair ? tree_item_length<Shape>(q.tiles) : 0;
                int sum = total_heads, rank_here = rank;
                if (!one_pass) rank_here = tree_block_scan(x, sm.scratch, sum);
                const int first = (before + rank_here) * p.num_kv_heads;
                if (w.lo >= first && w.lo < first + x * p.num_kv_heads) {
                    sm.start[0] = pair;
                    sm.start[1] = s0 + threadIdx.x;
                    sm.start[2] = w.lo - first;
                    sm.start_seq[0] = q.row0;
                    sm.start_seq[1] = q.n;
                    sm.start_seq[2] = q.ctx;
                }
                before += sum;
                found = w.lo < before * p.num_kv_heads;
            }
    }
    __syncthreads();
    return w;
}

// ---------------------------------------------------------------------------
// copies, items and query tiles
// ---------------------------------------------------------------------------
__device__ inline void tma_load_4d(void* dst, const CUtensorMap* map, int group, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, "
        "%3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(group), "r"(smem_addr(bar))
        : "memory");
}

// KINDS: bit 0, K tiles (and with them items and query tiles); bit 1, V tiles.
template <class Shape, int KINDS>
__device__ void tree_load(const TreeAttnParams& p, typename Shape::Smem& sm, int lane, const TreePiece& piece,
                          const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv) {
    constexpr bool LEADS = KINDS & 1;
    constexpr int NSLOT = Shape::NSLOT;
    const uint32_t q_bytes = (uint32_t)(Shape::SLABS * p.tile_tokens * p.group * 128);
    const int block_size = 1 << p.block_shift;
    const uint32_t box_bytes = (uint32_t)block_size * Shape::SLABS * 128u;
    const int blocks_per_tile = 128 >> p.block_shift, groups_per_block = block_size >> 3;
    uint32_t q_loads = 0;                  // query tiles so far
    // The ring's entries are K_0, V_0, K_1, ...; with a warp for each kind, a V tile is copied
    // behind the K tile of its number (k_go).
    uint32_t q_ones = 0, q_pairs = 0;      // of them for both chains, for each one
    uint32_t number = 0;                  // tiles so far
    uint32_t slot = KINDS == 2 ? 1 : 0, round = 0;  // of the next entry
    // [kind] bit (barrier * NSLOT + slot): whether it was used, parity of its next phase
    static_assert(3 * NSLOT <= 32, "bits");
    uint32_t filled[2] = {}, parity[2] = {};
    bool ok = true, wrong = false;
    if (LEADS && lane == 0) p.splits[blockIdx.x] = make_int4(0, 0, 0, 0);

    // Half tiles left of the piece, and of the sequence (in this pair of query tiles) before
    // what is left; sequences [window, window + 32) are in the lanes once one is done.
    int left = piece.hi - piece.lo, off = 0, pair = 0, window = 0, cur = 0;
    TreeSeq mine{0, 0, 0, 0, 0};
    int row0 = 0, nodes = 0, ctx = 0;
    if (left > 0) {
        pair = sm.start[0];
        window = sm.start[1] & ~31;
        cur = sm.start[1] & 31;
        off = sm.start[2];
        row0 = sm.start_seq[0], nodes = sm.start_seq[1], ctx = sm.start_seq[2];
    }
    bool loaded = false;
    // The next item of the piece with a tile in it; false at the end.
    auto take = [&](TreeItem& w) {
        while (left > 0) {
            const int nt = (ctx + 127) >> 7, length = tree_item_length<Shape>(nt);
            if (off == length * p.num_kv_heads) {
                // the next sequence with nodes in this pair of query tiles, or in the next one
                off = 0;
                if (!loaded) mine = tree_seq(p, window + lane, false);
                loaded = true;
                unsigned later = __ballot_sync(kFullMask, mine.pairs > pair) & ~((2u << cur) - 1u);
                while (later == 0) {
                    window += 32;
                    if (window >= p.num_seqs) {
                        window = 0;
                        if (++pair >= p.max_pairs) return false;  // lengths that changed under the call
                    }
                    mine = tree_seq(p, window + lane, false);
                    later = __ballot_sync(kFullMask, mine.pairs > pair);
                }
                cur = __ffs(later) - 1;
                row0 = __shfl_sync(kFullMask, mine.row0, cur);
                nodes = __shfl_sync(kFullMask, mine.n, cur);
                ctx = __shfl_sync(kFullMask, mine.ctx, cur);
                continue;
            }
            const int head = off / length, from = off - head * length, to = min(length, from + left);
            const int start = piece.hi - left - from;  // of the item in the list
            left -= to - from;
            off += to - from;
            w.from = tree_tiles_before<Shape>(from);
            w.to = tree_tiles_before<Shape>(to);
            if (w.from == w.to) continue;
            w.row0 = row0, w.n = nodes, w.ctx = ctx;
            w.kv_head = head;
            w.pair = pair;
            w.seq = window + cur;
            w.t0 = pair * 2 * p.tile_tokens;
            w.one = nodes - w.t0 <= p.tile_tokens;
            w.first_masked = (ctx - nodes) >> 7;
            if (LEADS && w.from == 0 && w.to < nt && lane == 0)  // goes on in the next CTAs
                p.splits[blockIdx.x] =
                    make_int4(row0 + w.t0, min(2 * p.tile_tokens, nodes - w.t0), head,
                              piece.cta_of(start + Shape::LEAD + 2 * (nt - 1)) - (int)blockIdx.x + 1);
            return true;
        }
        return false;
    };
    // Lane l: the l-th block from tile j on, or -2 behind the item's last one.  32 blocks at a
    // time, and the next ones while these are used: no tile waits for the table.
    const int tiles_per_load = 32 / blocks_per_tile;
    auto blocks_from = [&](const TreeItem& w, int j) {
        const int at = j * blocks_per_tile + lane;
        const int end = min(w.to * blocks_per_tile, (w.ctx + block_size - 1) >> p.block_shift);
        return at < end ? __ldcg(p.block_tables + (int64_t)w.seq * p.max_blocks + at) : -2;
    };
    // The next item is known, and its first blocks are loading, before one's last copies.
    TreeItem w{}, next{};
    bool more = take(w);
    int ids = more ? blocks_from(w, w.from) : -2, next_ids = -2, first_ids = -2;
    for (int n = 0;; ++n) {
        if (LEADS) {
            const int st = n % Shape::NITEM;
            tree_wait(p, sm, &sm.item_empty[st], ((uint32_t)(n / Shape::NITEM) & 1u) ^ 1u);
            if (__any_sync(kFullMask, prompt_aborted(&sm.abort_flag))) break;
            if (elect_one()) {
                sm.item[st][0] = make_int4(w.row0, more ? w.n : 0, w.ctx, w.kv_head);
                sm.item[st][1] = make_int4(w.pair, w.from, w.to, w.seq);
                mbar_arrive(&sm.item_full[st]);
            }
            __syncwarp();
        }
        if (!more) break;
        bool next_more = false;
#pragma unroll 1
        for (int j = w.from; j < w.to; ++j) {
            const int r = j - w.from, sub = r & (tiles_per_load - 1);
            if (sub == 0) {
                if (r > 0) ids = next_ids;
                next_ids = blocks_from(w, j + tiles_per_load);
            }
            const int mine_id = __shfl_sync(kFullMask, ids, sub * blocks_per_tile + (lane & (blocks_per_tile - 1)));
            const int id = lane < blocks_per_tile ? mine_id : -2;
            const bool good = id >= 0 && (int64_t)id < p.num_blocks;
            wrong |= id != -2 && !good;
            const uint32_t bytes = (uint32_t)__popc(__ballot_sync(kFullMask, good)) * box_bytes;
            const int group = good ? (id * p.num_kv_heads + w.kv_head) * groups_per_block : 0;  // rows are below 2^31
            const int readers = w.readers(r);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                if (!(KINDS >> v & 1)) continue;
                uint64_t* const full = v ? &sm.v_full[readers][slot] : &sm.k_full[readers][slot];
                if (v && !LEADS) tree_wait(p, sm, &sm.k_go[number % Shape::NGO], (number / Shape::NGO) & 1u);
                tree_wait(p, sm, &sm.kv_empty[slot], round ^ 1u);
                if (v == (LEADS ? 0 : 1)) {
                    ok = !__any_sync(kFullMask, prompt_aborted(&sm.abort_flag));
                    if (!ok) break;
                }
                if (elect_one()) mbar_arrive_expect_tx(full, bytes);
                __syncwarp();
                if (good) tma_load_4d(sm.kv[slot] + lane * box_bytes, v ? tv : tk, group, full);
                __syncwarp();
                if (Shape::TWO_LOADERS && !v && elect_one()) mbar_arrive(&sm.k_go[number % Shape::NGO]);
                filled[v] |= 1u << (readers * NSLOT + slot);
                parity[v] ^= 1u << (readers * NSLOT + slot);
                slot += KINDS == 3 ? 1 : 2;
                if (slot >= NSLOT) {
                    slot -= NSLOT;
                    round ^= 1u;
                }
                // Query tiles behind the first K tile, which the item before does not hold up.
#pragma unroll 1
                for (int i = 0; !v && r == 0 && i < (w.one ? 1 : 2); ++i) {
                    const uint32_t b = q_loads & 1u;
                    tree_wait(p, sm, &sm.q_empty[b], ((q_loads >> 1) & 1u) ^ 1u);
                    ok = !__any_sync(kFullMask, prompt_aborted(&sm.abort_flag));
                    if (!ok) break;
                    uint64_t* const q_full = w.one ? &sm.q_one[b] : &sm.q_pair[i];
                    if (elect_one()) {
                        mbar_arrive_expect_tx(q_full, q_bytes);
#pragma unroll
                        for (int s = 0; s < Shape::SLABS; ++s)
                            tma_load_3d_plain(sm.q[b][s], tq, s * 64, w.kv_head * p.group,
                                              w.row0 + w.t0 + i * p.tile_tokens, q_full);
                    }
                    __syncwarp();
                    ++q_loads;
                    if (w.one) {
                        q_ones ^= 1u << b;   // parity of the next phase
                        q_ones |= 4u << b;   // used
                    } else {
                        q_pairs ^= 1u << i;
                        q_pairs |= 4u << i;
                    }
                }
                if (!ok) break;
            }
            if (!ok) break;
            ++number;
            if (r > 0) continue;
            next_more = take(next);
            first_ids = next_more ? blocks_from(next, next.from) : -2;
        }
        if (!ok) break;
        w = next;
        more = next_more;
        ids = first_ids;
    }
    if (wrong) set_error(p.err, PA_DEVERR_BLOCK_ID);
    if (LEADS) pdl_launch_dependents();
    if (lane == 0) {
        // Every copy this warp issued lands before the CTA exits (bounded).
        bool drained = true;
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
            if (q_ones >> b & 4u)
                drained = mbar_wait_bounded(&sm.q_one[b], (q_ones >> b & 1u) ^ 1u, p.wait_limit_ns) && drained;
            if (q_pairs >> b & 4u)
                drained = mbar_wait_bounded(&sm.q_pair[b], (q_pairs >> b & 1u) ^ 1u, p.wait_limit_ns) && drained;
        }
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll 1
            for (int k = 0; k < 3 * NSLOT; ++k)
                if (filled[v] >> k & 1u)
                    drained = mbar_wait_bounded(v ? &sm.v_full[0][k] : &sm.k_full[0][k], (parity[v] >> k & 1u) ^ 1u,
                                                p.wait_limit_ns) && drained;
        if (!drained) set_error(p.err, PA_DEVERR_TIMEOUT);
    }
    __syncwarp();
}

// ---------------------------------------------------------------------------
// V tiles with nodes (a warp)
// ---------------------------------------------------------------------------
// Clears rows [rows, all) of a tile and replaces non-finite elements of rows [first, rows)
// by 0; true in the lanes that found any.
template <typename T, class Shape>
__device__ __noinline__ bool tree_check_tile(uint8_t* tile, int first, int rows, int all, int lane) {
    constexpr int CHUNKS = Shape::SLABS * 8;  // 16-byte chunks of a row
    constexpr int STEP = 32 / CHUNKS;         // rows of one pass of the warp
    const int my_chunk = lane % CHUNKS, my_row = lane / CHUNKS;
    // This lane's chunk of rows my_row, + STEP, ...
    uint8_t* const column = tile + (my_chunk >> 3) * 1024 + (my_chunk & 7) * 16;
    auto at = [&](int row) { return reinterpret_cast<uint4*>(column + (row >> 3) * Shape::GROUP + (row & 7) * 128); };
    for (int row = rows + my_row; row < all; row += STEP) *at(row) = make_uint4(0u, 0u, 0u, 0u);
    // 0 * v: NaN where v is infinite or NaN, and then for good in the sum.
    uint32_t acc = 0u;
#pragma unroll 4
    for (int row = first + my_row; row < rows; row += STEP) {
        const uint4 v = *at(row);
        acc = times_zero_plus<T>(v.x, acc);
        acc = times_zero_plus<T>(v.y, acc);
        acc = times_zero_plus<T>(v.z, acc);
        acc = times_zero_plus<T>(v.w, acc);
    }
    const bool bad_here = (acc & 0x7fff7fffu) != 0;
    if (bad_here) {
#pragma unroll 1
        for (int row = first + my_row; row < rows; row += STEP) {
            uint32_t* v = reinterpret_cast<uint32_t*>(at(row));
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
                const uint32_t bad = nonfinite2<T>(v[e]);
                v[e] &= ~(((bad >> 31) * 0xffff0000u) | ((bad >> 15 & 1u) * 0xffffu));
            }
        }
    }
    return bad_here;
}

// ---------------------------------------------------------------------------
// MMA issuer of chain i (one warp; an elected lane issues)
// ---------------------------------------------------------------------------
// Upper half of a descriptor (smem_desc_sw128) with 8-row groups `stride` bytes apart.
constexpr uint32_t tree_desc_hi(uint32_t stride) { return (stride >> 4) | (1u << 14) | (2u << 29); }

template <uint32_t A_HI, uint32_t B_HI>
__device__ __forceinline__ void tree_mma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool first) {
    asm volatile(
        "{\n\t.reg .b64 a, b;\n\t.reg .pred acc;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %6};\n\t"
        "setp.ne.b32 acc, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, acc;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(first ? 0u : 1u), "n"(A_HI), "n"(B_HI)
        : "memory");
}
template <uint32_t B_HI>
__device__ __forceinline__ void tree_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool first) {
    asm volatile(
        "{\n\t.reg .b64 b;\n\t.reg .pred acc;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "setp.ne.b32 acc, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, acc;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(first ? 0u : 1u), "n"(B_HI)
        : "memory");
}

template <typename T, class Shape>
__device__ void tree_mma(const TreeAttnParams& p, typename Shape::Smem& sm, uint32_t tmem, int i, int lane) {
    using Smem = typename Shape::Smem;
    constexpr int D = Shape::SLABS * 64;
    constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr uint32_t IDESC_O = mma_idesc_f16(BF16, true, Shape::BM, D);
    constexpr uint32_t IDESC_S = mma_idesc_f16(BF16, false, Shape::BM, 128);
    constexpr uint32_t IDESC_S64 = mma_idesc_f16(BF16, false, Shape::BM, 64);
    constexpr uint32_t Q_HI = tree_desc_hi(1024), KV_HI = tree_desc_hi(Shape::GROUP);
    constexpr uint32_t SLOT16 = sizeof(sm.kv[0]) >> 4, Q16 = sizeof(sm.q[0]) >> 4;
    const uint32_t base = smem_addr(&sm);
    const uint32_t q_lo = (uint32_t)smem_desc_sw128(base + offsetof(Smem, q), 16, 0);
    const uint32_t k_lo = (uint32_t)smem_desc_sw128(base + offsetof(Smem, kv), 16, 0);
    const uint32_t v_lo = (uint32_t)smem_desc_sw128(base + offsetof(Smem, kv), 1024, 0);
    const uint32_t s_tmem = tmem + i * Shape::BN, o_tmem = tmem + Shape::O_COL + i * D;

    // For the elected lane: S = Q K^T over the K tile's first half or all of it.
    auto issue_s = [&](uint32_t qi_lo, uint32_t slot, bool all) {
        const uint32_t idesc = all ? IDESC_S : IDESC_S64, b = k_lo + slot * SLOT16;
#pragma unroll
        for (int ks = 0; ks < Shape::SLABS * 4; ++ks)
            tree_mma_ss<Q_HI, KV_HI>(s_tmem, qi_lo + (uint32_t)((ks >> 2) * (Shape::Q_SLAB >> 4) + (ks & 3) * 2),
                                     b + (uint32_t)((ks >> 2) * 64 + (ks & 3) * 2), idesc, ks == 0);
    };
    // O (+)= P V over one half (64) of the V tile's positions.
    auto issue_pv = [&](uint32_t slot, int half, bool first) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
            tree_mma_ts<KV_HI>(o_tmem, s_tmem + half * 32 + ks * 8,
                               v_lo + slot * SLOT16 + (uint32_t)((half * 4 + ks) * 2 * (Shape::GROUP >> 4)), IDESC_O,
                               first && ks == 0);
    };

    uint32_t before = 0;     // K/V tiles before the item
    uint32_t nq = 0;         // query tiles before the item
    uint32_t no = 0, np = 0; // parities of the chain's O and P so far
    // Bit slot: parity of the next phase of k_full and v_full, of this chain's own
    // barriers and of both chains', and of v_checked; bit b of q_ones: of q_one[b].
    uint32_t k_own = 0, k_both = 0, v_own = 0, v_both = 0, checked = 0, q_ones = 0, q_pairs = 0;
    int n = 0;
    TreeItem w;
    while (tree_next_item<Shape>(p, sm, lane, n, w)) {
        const int tiles = w.tiles();
        const uint32_t t = (nq + (w.one ? 0 : i)) & 1u;  // buffer of this chain's query tile
        nq += w.one ? 1 : 2;
        if (w.one) {
            tree_wait(p, sm, &sm.q_one[t], q_ones >> t & 1u);
            q_ones ^= 1u << t;
            // A chain without tiles has waited too: its arrival may not count for the
            // query tile that was in the buffer before.
            if (!w.used(i) && elect_one()) mbar_arrive(&sm.q_empty[t]);
            __syncwarp();
        } else {
            tree_wait(p, sm, &sm.q_pair[i], q_pairs++ & 1u);
        }
        uint32_t& k_par = w.one ? k_own : k_both;
        uint32_t& v_par = w.one ? v_own : v_both;
        const int readers = w.one ? i : 2;
        const int last = w.one ? (((tiles - 1) & 1) == i ? tiles - 1 : tiles - 2) : tiles - 1;  // own tile
        bool first = true;
#pragma unroll 1
        for (int r = 0; r < tiles; ++r) {
            if (!w.own(i, r)) continue;
            const uint32_t entry = 2 * (before + r), kslot = entry % Shape::NSLOT, vslot = (entry + 1) % Shape::NSLOT;
            const int cols = w.ctx - (w.from + r) * Shape::BN;
            tree_wait(p, sm, &sm.k_full[readers][kslot], k_par >> kslot & 1u);
            k_par ^= 1u << kslot;
            tc_fence_after_sync();
            if (elect_one()) {
                issue_s(q_lo + t * Q16, kslot, cols > 64);
                mma_commit(&sm.s_full[i]);
                mma_commit(&sm.kv_empty[kslot]);
                if (w.one) mma_commit(&sm.kv_empty[kslot]);
                if (r == last) {
                    mma_commit(&sm.q_empty[t]);
                    if (!w.one) mma_commit(&sm.q_empty[t]);
                }
            }
            __syncwarp();
            tree_wait(p, sm, &sm.v_full[readers][vslot], v_par >> vslot & 1u);
            v_par ^= 1u << vslot;
            if (w.from + r >= w.first_masked) {
                if (w.one || i == 0) {
                    // Rows before the first node are attended by all.
                    const int rows = min(Shape::BN, cols);
                    if (tree_check_tile<T, Shape>(sm.kv[vslot], max(w.base - (w.from + r) * Shape::BN, 0), rows,
                                                  (rows + 63) & ~63, lane))
                        atomicMax(&sm.last_dirty, n - 1);  // n: items announced so far
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (!w.one && lane == 0) mbar_arrive(&sm.v_checked[vslot]);
                } else {
                    tree_wait(p, sm, &sm.v_checked[vslot], checked >> vslot & 1u);
                    checked ^= 1u << vslot;
                }
            }
            if (first) tree_wait(p, sm, &sm.o_empty[i], (no++ & 1u) ^ 1u);  // read by the output warps
            tree_wait(p, sm, &sm.p_full[i][0], np & 1u);
            tc_fence_after_sync();
            if (elect_one()) issue_pv(vslot, 0, first);
            __syncwarp();
            tree_wait(p, sm, &sm.p_full[i][1], np++ & 1u);
            tc_fence_after_sync();
            if (elect_one()) {
                if (cols > 64) issue_pv(vslot, 1, false);
                mma_commit(&sm.kv_empty[vslot]);
                if (w.one) mma_commit(&sm.kv_empty[vslot]);
                if (r == last) mma_commit(&sm.o_full[i]);
            }
            __syncwarp();
            first = false;
        }
        before += tiles;
    }
    // Nothing this warp issued may still be running when TMEM is released.
    if (elect_one()) mma_commit(&sm.mma_done[i]);
    __syncwarp();
    if (lane == 0 && !mbar_wait_bounded(&sm.mma_done[i], 0, p.wait_limit_ns)) set_error(p.err, PA_DEVERR_TIMEOUT);
    __syncwarp();
}

// ---------------------------------------------------------------------------
// softmax warps of chain i (thread r = row r = TMEM lane r)
// ---------------------------------------------------------------------------
// Masks and tables are read past L1: they may be written after this grid was launched.
// Bit k: the row attends to node first + k of its sequence (negative: a position before
// the tree), k < 32.  `row` is its mask row, `near` the first words of it, which were
// loaded when the item began: a masked tile otherwise waits for up to three round trips.
constexpr int kTreeNear = 4;
__device__ __forceinline__ uint32_t tree_mask_bits(const TreeAttnParams& p, const uint32_t* row,
                                                   const uint32_t (&near)[kTreeNear], int first) {
    if (first <= -32) return ~0u;
    auto word = [&](int at) {
        if (at >= kTreeNear) return at < p.mask_words ? __ldcg(row + at) : 0u;
        uint32_t w = 0u;
#pragma unroll
        for (int k = 0; k < kTreeNear; ++k) w = at == k ? near[k] : w;
        return w;
    };
    if (first < 0) return (near[0] << -first) | ((1u << -first) - 1u);
    const int at = first >> 5;
    return __funnelshift_r(word(at), word(at + 1), first & 31);
}

__device__ __forceinline__ void tree_mask64(float (&x)[64], uint32_t b0, uint32_t b1) {
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        x[k] = (b0 >> k) & 1u ? x[k] : __int_as_float(0xff800000);
        x[k + 32] = (b1 >> k) & 1u ? x[k + 32] : __int_as_float(0xff800000);
    }
}

template <typename T, class Shape>
__device__ void tree_softmax(const TreeAttnParams& p, typename Shape::Smem& sm, uint32_t tmem, int i, int warp,
                             int lane) {
    constexpr int D = Shape::SLABS * 64;
    const int r = warp * 32 + lane;
    const int t = r / p.group;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t s_addr = tmem + lanes + i * Shape::BN, o_addr = tmem + lanes + Shape::O_COL + i * D;
    const float c = p.scale_log2;  // > 0
    const float NEG_INF = __int_as_float(0xff800000);
    uint32_t ns = 0, used = 0;     // S and items of the chain so far
    int n = 0;
    TreeItem w;
    while (tree_next_item<Shape>(p, sm, lane, n, w)) {
        if (!w.used(i)) continue;
        const int node = w.t0 + (w.one ? 0 : i * p.tile_tokens) + t;
        const bool valid = t < p.tile_tokens && node < w.n;
        const bool any = __any_sync(kFullMask, valid);
        // Rows without a node compute something and are not stored.
        const uint32_t* const mask = p.tree_mask + (int64_t)(w.row0 + (valid ? node : w.t0)) * p.mask_words;
        uint32_t near[kTreeNear];
#pragma unroll
        for (int k = 0; k < kTreeNear; ++k) near[k] = k < p.mask_words ? __ldcg(mask + k) : 0u;
        float m = NEG_INF, l = 0.f;
        bool begun = false;
#pragma unroll 1
        for (int j = w.from; j < w.to; ++j) {
            if (!w.own(i, j - w.from)) continue;
            const int cols = w.ctx - j * Shape::BN;
            const bool masked = j >= w.first_masked;
            uint32_t bits[4] = {~0u, ~0u, ~0u, ~0u};
            if (masked && any) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    bits[q] = tree_mask_bits(p, mask, near, j * Shape::BN + 32 * q - w.base);
                    const int here = cols - 32 * q;  // positions before the context's end
                    if (here < 32) bits[q] &= here <= 0 ? 0u : (1u << here) - 1u;
                }
            }
            tree_wait(p, sm, &sm.s_full[i], ns++ & 1u);
            tc_fence_after_sync();
            auto written = [&](int half) {
                tmem_wait_st();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[i][half]);
            };
            if (!any) {  // rows of the MMA that nobody reads
                written(0);
                written(1);
                continue;
            }
            float x0[64], x1[64];  // scores of the tile's positions 0 .. 63, 64 .. 127
            tmem_ld_x64_async(s_addr, x0);
            tmem_wait_ld(x0);
            tmem_ld_x64_async(s_addr + 64, x1);
            float pm[8];
            if (masked) tree_mask64(x0, bits[0], bits[1]);
#pragma unroll
            for (int q = 0; q < 8; ++q) pm[q] = fmaxf(x0[q], x0[q + 8]);
#pragma unroll
            for (int k = 16; k < 64; k += 16)
#pragma unroll
                for (int q = 0; q < 8; ++q) pm[q] = max3(pm[q], x0[k + q], x0[k + q + 8]);
            tmem_wait_ld(x1);
            if (masked) tree_mask64(x1, bits[2], bits[3]);
#pragma unroll
            for (int k = 0; k < 64; k += 16)
#pragma unroll
                for (int q = 0; q < 8; ++q) pm[q] = max3(pm[q], x1[k + q], x1[k + q + 8]);
            const float mx = max3(max3(pm[0], pm[1], pm[2]), max3(pm[3], pm[4], pm[5]), fmaxf(pm[6], pm[7]));
            const float m_new = fmaxf(m, mx * c);
            const bool grow = m_new > m + 8.f;  // always on the first tile with a weight (m = -inf)
            float alpha = 1.f;
            if (grow) {
                alpha = prompt_exp2(m - m_new);
                m = m_new;
                l *= alpha;
            }
            // A grown maximum rescales O: S was issued after P V of the chain's tile
            // before, by the same thread, so that has completed too.
            if (begun && __any_sync(kFullMask, grow)) {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) prompt_scale16(o_addr + c0, alpha);
                tmem_wait_st();
            }
            begun = true;
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
        // Maxima and sums, once the output warps have read the chain's last ones.
        tree_wait(p, sm, &sm.o_empty[i], (used & 1u) ^ 1u);
        ++used;
        sm.row_max[i][r] = m;
        sm.row_sum[i][r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.l_full[i]);
    }
}

// ---------------------------------------------------------------------------
// output warps
// ---------------------------------------------------------------------------
// The non-finite values of nodes that were taken out of the item's V tiles:
// each decides its column of the rows that attend it.  Added to `dst` (the stored
// output, or the stored part) by the thread that stored it.
template <typename T, int D, typename O>
__device__ __noinline__ void tree_add_nonfinite(const TreeAttnParams& p, const TreeItem& w, int node, O* dst) {
    const uint32_t* const mask = p.tree_mask + (int64_t)(w.row0 + node) * p.mask_words;
    const int32_t* const table = p.block_tables + (int64_t)w.seq * p.max_blocks;
    const int end = min(w.to * 128, w.ctx);
    for (int at = max(w.from * 128, w.base); at < end; ++at) {
        const int m = at - w.base;
        if (!((__ldcg(mask + (m >> 5)) >> (m & 31)) & 1u)) continue;
        const int id = __ldcg(table + (at >> p.block_shift));
        if (id < 0 || (int64_t)id >= p.num_blocks) continue;
        const int64_t slot = (((int64_t)id * p.num_kv_heads + w.kv_head) << p.block_shift) + (at & ((1 << p.block_shift) - 1));
        const T* v = static_cast<const T*>(p.v_cache) + slot * D;
        for (int c = 0; c < D; ++c) {
            const float x = (float)v[c];
            if (!isfinite(x)) dst[c] = (O)((float)dst[c] + x);
        }
    }
}

// Two means of values, rounded.  A mean passes none of its values, but weights that
// were rounded up may carry one of f16 values next to the type's end beyond it: a
// finite mean beyond the end is the type's largest value, an infinite one stays.
template <typename T>
__device__ __forceinline__ uint32_t tree_pack_mean(float a, float b) {
    uint32_t w = pack_mean<T>(a, b);
    if constexpr (std::is_same<T, __half>::value) {
        if (isinf(a) || isinf(b)) w = pack_rn<T>(isinf(a) ? a : fminf(fmaxf(a, -65504.f), 65504.f),
                                                 isinf(b) ? b : fminf(fmaxf(b, -65504.f), 65504.f));
    }
    return w;
}

template <typename T, class Shape>
__device__ void tree_output(const TreeAttnParams& p, typename Shape::Smem& sm, uint32_t tmem, int warp, int lane) {
    constexpr int D = Shape::SLABS * 64;
    const float NEG_INF = __int_as_float(0xff800000);
    const int r = warp * 32 + lane;
    const int t = r / p.group, g = r - t * p.group;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    uint32_t parity = 0;  // bit i: of chain i's next O
    int n = 0;
    TreeItem w;
    while (tree_next_item<Shape>(p, sm, lane, n, w)) {
        const bool whole = w.whole();
#pragma unroll 1
        for (int i = 0; i < (w.one ? 1 : 2); ++i) {
            // One query tile: chain 0's sums and, if it had any tiles, chain 1's, joined.
            const bool both = w.one && w.used(1);
            tree_wait(p, sm, &sm.l_full[i], (parity >> i) & 1u);
            tree_wait(p, sm, &sm.o_full[i], (parity >> i) & 1u);
            parity ^= 1u << i;
            if (both) {
                tree_wait(p, sm, &sm.l_full[1], (parity >> 1) & 1u);
                tree_wait(p, sm, &sm.o_full[1], (parity >> 1) & 1u);
                parity ^= 2u;
            }
            tc_fence_after_sync();
            // A wait that ran out left no result: the rows stay as they were.
            const bool aborted = prompt_aborted(&sm.abort_flag);
            float m = sm.row_max[i][r], l = sm.row_sum[i][r], a0 = 1.f, a1 = 0.f;
            if (both) {
                // A maximum of -inf: no weights (or NaN ones, which a factor of 1 keeps).
                const float m0 = m, m1 = sm.row_max[1][r];
                m = fmaxf(m0, m1);
                a0 = m0 > NEG_INF ? exp2_approx(m0 - m) : 1.f;
                a1 = m1 > NEG_INF ? exp2_approx(m1 - m) : 1.f;
                l = l * a0 + sm.row_sum[1][r] * a1;
            }
            const int tt = i * p.tile_tokens + t;  // node of the pair of query tiles
            const int node = w.t0 + tt;
            const bool store = t < p.tile_tokens && node < w.n && !aborted;
            const bool dirty = *reinterpret_cast<volatile int*>(&sm.last_dirty) >= n - 1;
            // A row without weights: 0.
            const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
            a0 *= inv, a1 *= inv;
            T* const dst = static_cast<T*>(p.out) +
                           ((int64_t)(w.row0 + node) * p.num_heads + (int64_t)w.kv_head * p.group + g) * D;
            const int64_t part = ((int64_t)blockIdx.x * 2 + (w.from == 0 ? 1 : 0)) * p.row_cap + i * Shape::BM + r;
            float* const part_dst = p.part_o + part * D;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 16) {
                uint32_t u[16];
                float x[16];
                tmem_ld_x16(tmem + lanes + Shape::O_COL + i * D + c0, u);
#pragma unroll
                for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(u[k]) * a0;
                if (both) {
                    tmem_ld_x16(tmem + lanes + Shape::O_COL + D + c0, u);
#pragma unroll
                    for (int k = 0; k < 16; ++k) x[k] = fmaf(__uint_as_float(u[k]), a1, x[k]);
                }
                if (c0 + 16 == D) {  // O may be written again
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&sm.o_empty[i]);
                        if (both) mbar_arrive(&sm.o_empty[1]);
                    }
                }
                if (!store) continue;
                uint32_t q[8];
                if (whole) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) q[e] = tree_pack_mean<T>(x[2 * e], x[2 * e + 1]);
                    store_32_bytes(dst + c0, q);
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) q[e] = __float_as_uint(x[8 * h + e]);
                        store_32_bytes(part_dst + c0 + 8 * h, q);
                    }
                }
            }
            if (store && !whole) p.part_ml[part] = make_float2(m, l);
            if (store && dirty) {
                if (whole)
                    tree_add_nonfinite<T, D>(p, w, node, dst);
                else
                    tree_add_nonfinite<T, D>(p, w, node, part_dst);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// the kernel: one CTA per SM
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(TreeShape<D>::THREADS, 1)
    tree_attn_kernel(const __grid_constant__ TreeAttnParams p, const __grid_constant__ CUtensorMap tmap_q,
                     const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v) {
    using Shape = TreeShape<D>;
    using Smem = typename Shape::Smem;
    extern __shared__ __align__(1024) uint8_t tree_smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(tree_smem_raw);
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
            for (int k = 0; k < 3; ++k) {
                mbar_init(&sm.k_full[k][s], s == 0 && (p.debug_flags & kDebugDropFirstFill) ? 2 : 1);
                mbar_init(&sm.v_full[k][s], 1);
            }
            mbar_init(&sm.kv_empty[s], 2);
            mbar_init(&sm.v_checked[s], 1);
        }
        for (int s = 0; s < Shape::NGO; ++s) mbar_init(&sm.k_go[s], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_one[i], 1);
            mbar_init(&sm.q_pair[i], 1);
            mbar_init(&sm.q_empty[i], 2);
            mbar_init(&sm.mma_done[i], 1);
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
    if (warp == 0) tmem_alloc(&sm.tmem_base, Shape::TMEM_COLS);
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = sm.tmem_base;
    // Before the lengths are read too: a caller's kernel may write them after it has let its
    // dependents start, and pieces of old lengths with items of new ones would leave parts
    // that are not there.  (1.1 us for one short sequence, 1.4 for the long ones, 0.7 or less
    // for the others, against lengths read before the wait.)
    pdl_wait_prerequisites();
    const TreePiece piece = tree_piece<Shape>(p, sm);

    if (warp < Shape::SOFTMAX_WARP) {
        regs_dec<Shape::REGS_OTHER>();
        if (warp < Shape::LOAD_WARP)
            tree_mma<T, Shape>(p, sm, tmem, warp, lane);
        else if (!Shape::TWO_LOADERS && warp == Shape::LOAD_WARP)
            tree_load<Shape, 3>(p, sm, lane, piece, &tmap_q, &tmap_k, &tmap_v);
        else if (Shape::TWO_LOADERS && warp == Shape::LOAD_WARP)
            tree_load<Shape, 1>(p, sm, lane, piece, &tmap_q, &tmap_k, &tmap_v);
        else if (Shape::TWO_LOADERS)
            tree_load<Shape, 2>(p, sm, lane, piece, &tmap_q, &tmap_k, &tmap_v);
    } else if (warp < Shape::OUT_WARP) {
        regs_inc<Shape::REGS_SOFTMAX>();
        const int v = warp - Shape::SOFTMAX_WARP;
        tree_softmax<T, Shape>(p, sm, tmem, v >> 2, v & 3, lane);
    } else {
        regs_dec<Shape::REGS_OUT>();
        tree_output<T, Shape>(p, sm, tmem, warp - Shape::OUT_WARP, lane);
    }

    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (threadIdx.x == 0) {
        p.aborted[blockIdx.x] = sm.abort_flag;
        if (sm.abort_flag) set_error(p.err, PA_DEVERR_TIMEOUT);
    }
    __syncwarp();
    if (warp == 0) tmem_dealloc(tmem, Shape::TMEM_COLS);
}

// ---------------------------------------------------------------------------
// the items that several CTAs share
// ---------------------------------------------------------------------------
// With the parts' maxima m_k, sums l_k and weighted values o_k:
//     M = max m_k,  w_k = 2^(m_k - M),  out = sum o_k w_k / sum l_k w_k.
// A warp per row; a lane holds D / 32 consecutive columns.  Part 0 is the one of the
// CTA in which the item begins, part k the first piece of the k-th CTA after it.
constexpr int kTreeReduceThreads = 256;
constexpr int kTreeReduceCtas = 8;  // of an item at most: 64 rows at a time

template <typename T, int D>
__global__ void __launch_bounds__(kTreeReduceThreads) tree_reduce_kernel(const __grid_constant__ TreeAttnParams p) {
    constexpr int VPL = D / 32;
    constexpr int PRE = 32 / VPL;  // parts whose values are loaded beside the maxima and sums
    const float NEG_INF = __int_as_float(0xff800000);
    const int lane = threadIdx.x & 31;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int4 item = __ldcg(p.splits + blockIdx.x);
    const int parts = item.w;
    if (parts == 0) return;
    // A part that is not there: the rows stay as they were.
    bool missing = false;
    for (int k = lane; k < parts; k += 32) missing |= __ldcg(p.aborted + blockIdx.x + k) != 0;
    if (__any_sync(kFullMask, missing)) return;
    auto slot = [&](int k) { return ((int64_t)(blockIdx.x + k) * 2 + (k == 0 ? 1 : 0)) * p.row_cap; };
    // Rows of the second query tile stand 128 behind the first one's.
    const int rows = item.y <= p.tile_tokens ? item.y * p.group : 128 + (item.y - p.tile_tokens) * p.group;
    for (int row = blockIdx.y * (kTreeReduceThreads / 32) + (threadIdx.x >> 5); row < rows;
         row += gridDim.y * (kTreeReduceThreads / 32)) {
        const int i = row >> 7, r = row & 127, t = r / p.group, g = r - t * p.group;
        const int node = i * p.tile_tokens + t;
        if (t >= p.tile_tokens) continue;
        float M = NEG_INF, L = 0.f, acc[VPL];
#pragma unroll
        for (int v = 0; v < VPL; ++v) acc[v] = 0.f;
        for (int k0 = 0; k0 < parts; k0 += 32) {
            const int count = min(32, parts - k0);
            float2 ml = make_float2(NEG_INF, 0.f);
            if (lane < count) ml = __ldcg(p.part_ml + slot(k0 + lane) + row);
            auto values = [&](int k, float (&o)[VPL]) {
                const float* src = p.part_o + (slot(k0 + k) + row) * D + lane * VPL;
                if constexpr (VPL == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
                    o[0] = x.x, o[1] = x.y, o[2] = x.z, o[3] = x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2*>(src));
                    o[0] = x.x, o[1] = x.y;
                }
            };
            float pre[PRE][VPL];
#pragma unroll
            for (int k = 0; k < PRE; ++k) {
#pragma unroll
                for (int v = 0; v < VPL; ++v) pre[k][v] = 0.f;
                if (k < count) values(k, pre[k]);
            }
            float cm = ml.x;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) cm = fmaxf(cm, __shfl_xor_sync(kFullMask, cm, d));
            const float m_new = fmaxf(M, cm);
            // A maximum of -inf: no weights (or NaN ones, which a factor of 1 keeps).
            const float old = M > NEG_INF ? exp2_approx(M - m_new) : 1.f;
            const float weight = ml.x > NEG_INF ? exp2_approx(ml.x - m_new) : 1.f;
            float sum = lane < count ? ml.y * weight : 0.f;
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kFullMask, sum, d);
            L = L * old + sum;
            M = m_new;
#pragma unroll
            for (int v = 0; v < VPL; ++v) acc[v] *= old;
#pragma unroll
            for (int k = 0; k < PRE; ++k) {
                if (k >= count) break;
                const float wk = __shfl_sync(kFullMask, weight, k);
#pragma unroll
                for (int v = 0; v < VPL; ++v) acc[v] = fmaf(wk, pre[k][v], acc[v]);
            }
#pragma unroll 4
            for (int k = PRE; k < count; ++k) {
                const float wk = __shfl_sync(kFullMask, weight, k);
                float o[VPL];
                values(k, o);
#pragma unroll
                for (int v = 0; v < VPL; ++v) acc[v] = fmaf(wk, o[v], acc[v]);
            }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        uint32_t* dst = reinterpret_cast<uint32_t*>(
            static_cast<T*>(p.out) +
            ((int64_t)(item.x + node) * p.num_heads + (int64_t)item.z * p.group + g) * D + lane * VPL);
        if constexpr (VPL == 4)
            *reinterpret_cast<uint2*>(dst) = make_uint2(tree_pack_mean<T>(acc[0] * inv, acc[1] * inv),
                                                        tree_pack_mean<T>(acc[2] * inv, acc[3] * inv));
        else
            *dst = tree_pack_mean<T>(acc[0] * inv, acc[1] * inv);
    }
}

template <typename T, int D>
cudaError_t launch_tree_attention_t(const TreeAttnParams& p, const CUtensorMap* tq, const CUtensorMap* tk,
                                    const CUtensorMap* tv, cudaStream_t stream) {
    using Shape = TreeShape<D>;
    constexpr int kMaxDevices = 64;
    static int configured[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(tree_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Shape::SMEM_BYTES);
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)p.ctas);
    cfg.blockDim = dim3(Shape::THREADS);
    cfg.dynamicSmemBytes = Shape::SMEM_BYTES;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<T, D>, p, *tq, *tk, *tv);
    if (e != cudaSuccess || p.ctas == 1) return e;  // one CTA shares nothing
    const int slices = (p.row_cap + kTreeReduceThreads / 32 - 1) / (kTreeReduceThreads / 32);
    cfg.gridDim = dim3((unsigned)p.ctas, (unsigned)(slices < kTreeReduceCtas ? slices : kTreeReduceCtas));
    cfg.blockDim = dim3(kTreeReduceThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, tree_reduce_kernel<T, D>, p);
}

}  // namespace pa
