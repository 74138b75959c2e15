// pkv_chunk_impl.cuh -- the chunk attention kernel: attention of each
// sequence's newest tokens over its paged cache, on the tensor cores.
//
// Mathematics.  Row by row, over steps of 128 cache positions: scores
// S = Q K^T, a running maximum m and sum l, weights P = 2^(c (S - m) + 9) with
// c = scale * log2(e), O = O * 2^(c (m_old - m)) + P V, and out = O / l.  The
// group of query heads that share a KV head are rows of one tile, so each step
// of K and V serves all of them.
//
// One CTA per SM, 12 warps, walking its share of the work (pkv_chunk_schedule.h)
// piece by piece:
//   warps 0-3, 4-7  one softmax warpgroup per slot, a row per thread
//   warps 8, 9      issue the products of a slot each
//   warp 10         walks the schedule and the block tables, issues the copies
//   warp 11         guards V where a step is not seen by every row (below)
// A slot is a tile of 128 query rows with its own S and O in tensor memory
// (P overlays S: all 512 columns are used at head_dim 128).  The two slots of a
// piece are either two query tiles that share every step of K and V, or, where
// the item has one tile, the same tile with alternate steps, joined at the end.
// While one slot's softmax runs, the other's products do.
//
// What bounds it: with 256 rows a step is 4 * 256 * 128 * D operations for
// 512 * D bytes, so long prompts are bound by the products and the softmax: a
// slot's step is its products, 1024 cycles at the tensor cores' rate, then its
// softmax, somewhat longer with the hand-overs, under the other slot's products
// (1024 tokens of 16384, groups of 4: the tensor cores are busy 73% of the time).
// At head_dim 64 the products are half of that and a step takes as long: the chain
// through one slot's S is what counts.  With one token per sequence the
// tile is nearly empty, and a step's copy from HBM takes longer than its
// products, so padding costs no time.
//
// Measured on one GB300 (head_dim 128):
//   32 heads, a prompt of 4096 tokens           138 us, 1000 TFLOP/s
//   32 heads in groups of 4, 2048 new of 32768  763 to 790 us, 1350 to 1400
//                                               TFLOP/s (power: 1500 MHz)
//   8 single tokens over 8000 to 32768, groups of 4   120 us, 6110 GB/s
//   64 x 5 tokens over 50 to 900, 32 heads      113 us, 4350 GB/s
// A call's fixed parts: 6 us until the first scores (launch, schedule, table,
// first copy), 4 us of last pieces, 5 to 13 us of the joining kernel.
//
// V is read as an operand for every row of a tile, and 0 * NaN is NaN.  So in
// steps that some row does not see whole, the guard warp clears the rows of V
// that no row of the item sees (table ends, what precedes a window) and clears
// single elements that are not finite; the epilogue adds the latter to the
// rows that do see them (they decide those elements: finite + inf = inf).
#ifndef PKV_CHUNK_IMPL_CUH
#define PKV_CHUNK_IMPL_CUH

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pkv_chunk_schedule.h"
#include "pkv_device.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

constexpr int kChunkThreads = 384;
constexpr int kChunkRows = 128;   // rows of a query tile
// Weights are 2^(c (S - m) + kWeightLift), held as fp16 for the second product:
// a row's largest is 2^9 to 2^15.5, so that one is lost only below 2^-34 of it.  At
// 1 a long context's small weights would be lost from 2^-25 on but counted in the
// sum: 131072 positions at e^-17.5 of one are 3.3e-3 of the row.
constexpr float kWeightLift = 9.f;
// log2 of how far the maximum may rise above m before O is rescaled.  Less lift and
// more room to rise saves rescaling where a tile's first step shows a few
// positions: 2 x 1000 to 4001 tokens with a window of 1024 take 78.0 us with 9 and
// 6.5, 77.5 with 8 and 7.5, 76.6 with 6 and 9.5; the others are level.
constexpr float kMostRise = 6.5f;
constexpr float kFarScore = 1048576.f;  // 2^20: an exponent in fp32 is off by up to 2^-4 from here on
constexpr int kChunkPieces = 4;   // piece descriptors in flight
// Registers per thread: 384 at launch x 168 = 64512 = 256 x 208 + 128 x 88.
constexpr int kChunkLaunchRegs = 168;

// The part of an item that a CTA begins and others end, for the joining kernel.
struct ChunkPart {
    long long start;     // the item's first unit
    ChunkShares shares;  // the cut of the line
    int valid;
    int row0;            // first query row
    int tokens;
    int kv_head;
    int lo, hi;          // positions that some row sees
    int cta1;            // the last CTA that holds it
};

struct ChunkParams {
    CUtensorMap tmap_q;  // [T][H][D] in boxes {64, group, tile_tokens}
    CUtensorMap tmap_k;  // the caches in boxes of {64, block rows, 1}
    CUtensorMap tmap_v;
    __half *out;
    const __half *value_cache;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const int32_t *query_starts;
    // A CTA's parts of items that it shares with others: part 2 * CTA + 1 of the
    // item that it begins, 2 * CTA of the one that it does not (chunk_part).
    ChunkPart *parts;      // [CTAs] of the first kind
    float2 *part_ml;       // [2 * CTAs][2 slots][128 rows] (top(), l)
    float *part_o;         // [2 * CTAs][part_rows][D], not normalised
    int32_t *status;
    ChunkShape shape;
    int num_tokens;
    int num_seqs;
    int num_heads;
    int group;
    int max_blocks_per_seq;
    int num_blocks;
    int block_shift;     // log2(block_size)
    int part_rows;
    int fits_32;         // the schedule's line (chunk_fits_32)
    float scale_log2;
    uint32_t wait_tries;
};

struct ChunkPiece {
    int row0;            // first query row of the item
    int tokens;          // its tokens
    int kv_head;
    int seq;
    int pos0;            // position of its first token (negative: sees nothing)
    int len;
    int lo, hi;          // positions that some row sees
    int all_lo, all_hi;  // positions that every row sees
    int t0, t1;          // steps of this piece
    int first[2], end[2];  // those a slot takes: first, first + stride, ... < end
    int partial;         // some of the item's steps, not all
    int part;            // then this CTA's part of it
    int single;          // one query tile: the slots take alternate steps (stride 2, else 1)
    int q_buffer;        // of a lone tile's queries (two tiles take both buffers)
    int last;            // no piece: the end
    int odd;             // the guard cleared an element that was not finite
};

// Shared-memory address of a member of the control block at shared address `ctl_at`.
#define PKV_CTL(member) (ctl_at + (uint32_t)offsetof(Control, member))

template <int D>
struct ChunkConfig {
    static constexpr int kHalves = D / 64;
    static constexpr int kHalfBytes = kChunkTile * 128;
    static constexpr int kTileBytes = kHalves * kHalfBytes;
    static constexpr int kStages = D == 128 ? 5 : 10;  // 160 KB of K and V in flight
    struct Control {
        uint64_t full[kStages], empty[kStages], edge[kStages], guard[kStages];
        uint64_t q_full[2], q_empty[2], s_full[2], p_full[2][2], o_full[2], o_free[2], o_cross[2];
        uint64_t x_full, x_empty, drain[2];
        uint64_t piece_full[kChunkPieces], piece_empty[kChunkPieces];
        ChunkPiece piece[kChunkPieces];
        float2 ml[2][kChunkRows];
        uint32_t tmem;
        int abort;
        uint32_t issued[2];  // batches of products, by slot
    };
    static constexpr size_t kSmem = (size_t)(2 + kStages) * kTileBytes + sizeof(Control);
    static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

template <int R>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

// A bounded wait of a whole warp, which leaves together: false once it has
// tried too often, or once any warp of the CTA has (the abort flag); every role
// then leaves its loop, and the CTA reports the timeout at its end.  Kept
// small, since it stands in many places: the roles' code has to share the
// instruction cache.  Addresses are those of shared memory.
__device__ __forceinline__ bool chunk_wait(uint32_t bar, uint32_t parity, uint32_t abort, uint32_t limit) {
#pragma unroll 1
    for (uint32_t i = 0; !__all_sync(kFullMask, mbar_try_wait(bar, parity)); ++i) {
        uint32_t gone;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gone) : "r"(abort) : "memory");
        if (gone || i >= limit) {
            asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1) : "memory");
            return false;
        }
    }
    return true;
}

// A bounded wait for a counter in shared memory, the same otherwise.  A try is
// two loads and a vote, far less than a suspended one: kSpinsPerTry of them count
// as one.
constexpr uint32_t kSpinsPerTry = 48;
__device__ __forceinline__ bool chunk_wait_count(uint32_t counter, uint32_t value, uint32_t abort, uint32_t limit) {
#pragma unroll 1
    for (uint32_t i = 0;; ++i) {
        uint32_t x, gone;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(x) : "r"(counter) : "memory");
        if (__all_sync(kFullMask, (int)(x - value) >= 0)) return true;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(gone) : "r"(abort) : "memory");
        if (gone || i >= limit * kSpinsPerTry) {
            asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1) : "memory");
            return false;
        }
    }
}

__device__ __noinline__ void chunk_drain(uint32_t bar, uint32_t parity) {
    mbar_wait_bounded(bar, parity, kWaitLimitNs / 8);
}

__device__ __noinline__ void chunk_report_range(int32_t *status) { report(status, PKV_ERR_OUT_OF_RANGE); }

__device__ __forceinline__ int chunk_clamp(int64_t x, int hi) { return (int)chunk_min64(chunk_max64(x, 0), hi); }

// A sequence's rows and length, clamped to what there is.
__device__ __forceinline__ ChunkSeq chunk_load_seq(const ChunkParams &p, int s, bool tell) {
    ChunkSeq q;
    const int a = __ldg(p.query_starts + s), b = __ldg(p.query_starts + s + 1), len = __ldg(p.context_lens + s);
    const int most = p.max_blocks_per_seq << p.block_shift;
    q.row0 = chunk_clamp(a, p.num_tokens);
    q.n = chunk_clamp(b, p.num_tokens) - q.row0;
    if (q.n < 0) q.n = 0;
    q.len = chunk_clamp(len, most);
    if (tell && (a != q.row0 || b != q.row0 + q.n || len != q.len)) chunk_report_range(p.status);
    return q;
}

// The schedule's closed forms, out of line, their arguments in registers (a
// reference to the parameters would be read through the caches, cold): I =
// int32_t where the line fits it.
template <typename I>
__device__ __noinline__ int64_t chunk_units(ChunkShape c, ChunkSeq s) {
    return chunk_seq_units<I>(c, s);
}

// The item of a sequence that holds unit x of its units, and x's offset in it,
// by a whole warp: 32 candidates at a time.
struct ChunkPlace {
    int kv_head, item, offset;
};

template <typename I>
__device__ __noinline__ ChunkPlace chunk_locate(ChunkShape c, ChunkSeq s, int64_t unit, int lane) {
    const int items = chunk_items(c, s);
    const I per_head = chunk_prefix<I>(c, s, items);
    I x = (I)unit;
    int head = -1;  // the last one that begins at or before x
    unsigned hits;
    do {
        const int h = head + 1 + lane;
        hits = __ballot_sync(kFullMask, h < c.num_kv_heads && h * per_head <= x);
        head += __popc(hits);
    } while (hits == kFullMask);
    x -= head * per_head;
    int lo = 0, span = items;  // the item is in [lo, lo + span)
    I before = 0;
    while (span > 1) {
        const int step = (span + 31) / 32, i = lo + lane * step;
        const I at = lane * step < span ? chunk_prefix<I>(c, s, i) : 0;
        const int who = 31 - __clz(__ballot_sync(kFullMask, lane * step < span && at <= x));
        before = __shfl_sync(kFullMask, at, who);
        lo += who * step;
        span = min(step, span - who * step);
    }
    return ChunkPlace{head, lo, (int)(x - before)};
}

// Whether some row of the item does not see all of step t.
__device__ __forceinline__ bool chunk_edge(const ChunkPiece &pc, int t) {
    return t * kChunkTile < pc.all_lo || (t + 1) * kChunkTile > pc.all_hi;
}

// Whether a position of step t is seen by some rows of the item and not by others.
__device__ __forceinline__ bool chunk_mixed(const ChunkPiece &pc, int t) {
    return max(t * kChunkTile, pc.lo) < pc.all_lo || min((t + 1) * kChunkTile, pc.hi) > pc.all_hi;
}

// Ring positions of a piece's copies relative to its first: K0 K1 V0 K2 V1 ...
__device__ __forceinline__ uint32_t chunk_v_at(int k, int n) { return k < n - 1 ? 2u * k + 2u : 2u * n - 1u; }

__device__ __forceinline__ int chunk_block(const ChunkParams &p, int seq, int logical) {
    int blk = __ldg(p.block_tables + (int64_t)seq * p.max_blocks_per_seq + logical);
    if (blk < 0 || blk >= p.num_blocks) {
        chunk_report_range(p.status);
        blk = 0;
    }
    return blk;
}

__device__ __forceinline__ bool odd_halves(uint32_t w) { return (((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u) != 0; }

__device__ __forceinline__ uint32_t clear_odd(uint32_t w) {
    if ((w & 0x7c00u) == 0x7c00u) w &= 0xffff0000u;
    if ((w & 0x7c000000u) == 0x7c000000u) w &= 0x0000ffffu;
    return w;
}

// Adds the elements of V that are not finite to the columns [c0, c0 + cols) of
// a row already written: those of the mixed steps of the piece that the row
// sees.  Rare, so plain loops.
template <int D, typename T>
__device__ __noinline__ void chunk_add_odd(const ChunkParams &p, const ChunkPiece &pc, int row_lo, int row_hi, T *row,
                                           int c0, int cols) {
    for (int t = pc.t0; t < pc.t1; ++t) {
        if (!chunk_mixed(pc, t)) continue;
        const int a = max(t * kChunkTile, row_lo), b = min((t + 1) * kChunkTile, row_hi);
        for (int pos = a; pos < b; ++pos) {
            const int64_t blk = chunk_block(p, pc.seq, pos >> p.block_shift);
            const __half *v = p.value_cache + (((blk * p.shape.num_kv_heads + pc.kv_head) << p.block_shift) +
                                               (pos & ((1 << p.block_shift) - 1))) * D;
            for (int c = c0; c < c0 + cols; ++c) {
                const __half h = v[c];
                if ((__half_as_ushort(h) & 0x7c00) == 0x7c00) row[c] = (T)((float)row[c] + __half2float(h));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// warp 10: the schedule and the copies

template <int D>
struct ChunkLoader {
    using Cfg = ChunkConfig<D>;
    using Control = typename Cfg::Control;
    const ChunkParams &p;
    Control &ctl;
    uint32_t ctl_at;  // its shared-memory address
    uint32_t q_smem, ring_smem;
    int lane;
    uint32_t ring = 0;          // ring position of the next copy
    uint32_t pieces = 0;
    uint32_t q_uses = 0, q_used = 0;         // a bit per buffer: phase, ever used
    uint32_t edge_phase = 0, edge_used = 0;  // bit per stage
    int next_buffer = 0;
    bool begun = false;  // an item that others end
    ChunkShares shares;

    __device__ bool wait(uint32_t bar, uint32_t parity) { return chunk_wait(bar, parity, PKV_CTL(abort), p.wait_tries); }

    // The positions that row `token` of the item sees: [row_begin, row_end).
    __device__ int row_end(const ChunkPiece &pc, int token) {
        return p.shape.causal ? min(max(pc.pos0 + token + 1, 0), pc.len) : pc.len;
    }
    __device__ int row_begin(const ChunkPiece &pc, int token) {
        return p.shape.window ? min(max(max(pc.pos0 + token, -1) - p.shape.window + 1, 0), pc.len) : 0;
    }

    // This lane's block of step t (-1: none of its positions is seen).
    __device__ int lookup(const ChunkPiece &pc, int t) {
        const int b = (t * kChunkTile >> p.block_shift) + lane;
        const bool mine = lane < (kChunkTile >> p.block_shift) && ((int64_t)b << p.block_shift) < pc.hi &&
                          ((int64_t)(b + 1) << p.block_shift) > pc.lo;
        return mine ? chunk_block(p, pc.seq, b) : -1;
    }

    // One tile into the next stage.  A tile that the guard goes over first
    // (edge) lands on a barrier of its own, and the products wait for the guard.
    __device__ bool copy(const CUtensorMap *map, int blk, int kv_head, bool edge) {
        const uint32_t st = ring % Cfg::kStages;
        if (!wait(PKV_CTL(empty) + 8 * st, (ring / Cfg::kStages & 1) ^ 1)) return false;
        ++ring;
        const uint32_t bar = (edge ? PKV_CTL(edge) : PKV_CTL(full)) + 8 * st;
        const unsigned live = __ballot_sync(kFullMask, blk >= 0);
        if (lane == 0) {
            mbar_arrive_expect_tx(bar, __popc(live) * ((uint32_t)D * 2 << p.block_shift));
            if (edge) mbar_arrive(PKV_CTL(full) + 8 * st);
        }
        if (edge) {
            edge_phase ^= 1u << st;
            edge_used |= 1u << st;
        }
        __syncwarp();
        if (blk >= 0) {
            const uint32_t dst = ring_smem + st * Cfg::kTileBytes + ((uint32_t)lane << p.block_shift) * 128;
            const int row = (int)(((int64_t)blk * p.shape.num_kv_heads + kv_head) << p.block_shift);
#pragma unroll
            for (int h = 0; h < Cfg::kHalves; ++h) tma_load_3d(dst + h * Cfg::kHalfBytes, map, 0, row, h, bar);
        }
        return true;
    }

    __device__ bool emit(const ChunkPiece &pc) {
        const uint32_t slot = pieces % kChunkPieces;
        if (!wait(PKV_CTL(piece_empty) + 8 * slot, (pieces / kChunkPieces & 1) ^ 1)) return false;
        ++pieces;
        if (lane == 0) {
            ctl.piece[slot] = pc;
            mbar_arrive(PKV_CTL(piece_full) + 8 * slot);
        }
        __syncwarp();
        return true;
    }

    __device__ bool load_queries(const ChunkPiece &pc) {
#pragma unroll 1
        for (int i = 0; i < (pc.single ? 1 : 2); ++i) {
            const int b = pc.single ? pc.q_buffer : i;
            if (!wait(PKV_CTL(q_empty) + 8 * b, (q_uses >> b & 1) ^ 1)) return false;
            q_uses ^= 1u << b;
            q_used |= 1u << b;
            if (lane == 0) {
                const uint32_t bar = PKV_CTL(q_full) + 8 * b;
                mbar_arrive_expect_tx(bar, (uint32_t)p.shape.tile_tokens * p.group * D * 2);
#pragma unroll
                for (int h = 0; h < Cfg::kHalves; ++h)
                    tma_load_3d(q_smem + b * Cfg::kTileBytes + h * Cfg::kHalfBytes, &p.tmap_q, h * 64,
                                pc.kv_head * p.group, pc.row0 + i * p.shape.tile_tokens, bar);
            }
            __syncwarp();
        }
        return true;
    }

    __device__ bool load(const ChunkPiece &pc) {
        const int n = pc.t1 - pc.t0;
        if (n == 0) return true;
        // The block table is read two steps ahead of the copies.
        int now = lookup(pc, pc.t0), next = n > 1 ? lookup(pc, pc.t0 + 1) : -1;
        if (pieces == 1 && !load_queries(pc)) return false;
#pragma unroll 1
        for (int t = pc.t0 - 1; t < pc.t1; ++t) {
            const int ahead = t >= pc.t0 && t + 2 < pc.t1 ? lookup(pc, t + 2) : -1;
            if (t + 1 < pc.t1 && !copy(&p.tmap_k, t < pc.t0 ? now : next, pc.kv_head, false)) return false;
            if (t < pc.t0) continue;
            // The queries only now, but for the first piece: their buffer is free when
            // the previous piece's last scores are done, and the first K can be on
            // their way before.
            if (t == pc.t0 && pieces > 1 && !load_queries(pc)) return false;
            if (!copy(&p.tmap_v, now, pc.kv_head, chunk_edge(pc, t))) return false;
            now = next;
            next = ahead;
        }
        return true;
    }

    // The next sequence at or after s that has rows; num_seqs if none.
    __device__ int next_seq(int s) {
        while (s < p.num_seqs) {
            const bool has = s + lane < p.num_seqs && chunk_load_seq(p, s + lane, false).n > 0;
            const unsigned m = __ballot_sync(kFullMask, has);
            if (m) return s + __ffs(m) - 1;
            s += 32;
        }
        return p.num_seqs;
    }

    // The share [u, end) of the line; cum = units before sequence s.
    __device__ bool walk(int s, int64_t cum, int64_t u, int64_t end) {
        if (u >= end) return true;
        ChunkShape c = p.shape;
        c.quantum_shift = chunk_quantum_shift(shares);
        ChunkSeq q = chunk_load_seq(p, s, false);
        const ChunkPlace at = p.fits_32 ? chunk_locate<int32_t>(c, q, u - cum, lane) : chunk_locate<int64_t>(c, q, u - cum, lane);
        int head = at.kv_head, item = at.item, off = at.offset, items = chunk_items(c, q);
        while (true) {
            ChunkPiece pc;
            const int w = 2 * c.tile_tokens;
            int lo, hi;
            chunk_item_range(c, q, item, &lo, &hi);
            const int cost = hi - lo + c.overhead;
            const int stop = end - u < cost - off ? off + (int)(end - u) : cost;
            const int steps = chunk_steps(lo, hi), first = lo / kChunkTile;
            const int a = chunk_step_at(c, lo, hi, off), b = chunk_step_at(c, lo, hi, stop);
            if (b > a || (steps == 0 && off == 0)) {
                pc.row0 = q.row0 + item * w;
                pc.tokens = min(w, q.n - item * w);
                pc.kv_head = head;
                pc.seq = s;
                pc.pos0 = q.len - q.n + item * w;
                pc.len = q.len;
                pc.lo = lo;
                pc.hi = hi;
                pc.all_lo = 0;
                pc.all_hi = q.len;
                if (c.causal) {
                    pc.all_hi = row_end(pc, 0);
                    if (c.window) pc.all_lo = row_begin(pc, pc.tokens - 1);
                }
                pc.t0 = first + a;
                pc.t1 = first + b;
                pc.single = pc.tokens <= c.tile_tokens;
                pc.last = 0;
                pc.q_buffer = next_buffer;  // the one that the last lone tile did not take
                next_buffer ^= 1;
                pc.odd = 0;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (pc.single) {
                        pc.first[k] = min(pc.t0 + k, pc.t1);
                        pc.end[k] = pc.t1;
                    } else {  // the steps that some row of the slot's tile sees
                        const int r0 = k * c.tile_tokens, r1 = min(r0 + c.tile_tokens, pc.tokens) - 1;
                        const int from = row_begin(pc, r0), to = row_end(pc, r1);
                        pc.first[k] = max((int)((unsigned)from / kChunkTile), pc.t0);
                        pc.end[k] = max(min((int)(((unsigned)to + kChunkTile - 1) / kChunkTile), pc.t1), pc.first[k]);
                        if (to <= from) pc.end[k] = pc.first[k];
                    }
                }
                pc.partial = b - a < steps;
                if (pc.partial) pc.part = 2 * blockIdx.x + (a == 0 ? 1 : 0);
                if (pc.partial && a == 0) {
                    begun = true;
                    if (lane == 0) {
                        ChunkPart part;
                        part.start = u - off;
                        part.shares = shares;
                        part.valid = 1;
                        part.row0 = pc.row0;
                        part.tokens = pc.tokens;
                        part.kv_head = head;
                        part.lo = lo;
                        part.hi = hi;
                        part.cta1 = chunk_share_of(shares, part.start + cost - 1);
                        p.parts[blockIdx.x] = part;
                    }
                }
                if (!emit(pc) || !load(pc)) return false;
            }
            u += stop - off;
            if (u >= end) return true;
            off = 0;
            if (++item == items) {
                item = 0;
                if (++head == c.num_kv_heads) {
                    head = 0;
                    s = next_seq(s + 1);
                    if (s >= p.num_seqs) return true;
                    q = chunk_load_seq(p, s, false);
                    items = chunk_items(c, q);
                }
            }
        }
    }

    __device__ void run(int s, int64_t cum, int64_t u, int64_t end) {
        bool ok = walk(s, cum, u, end);
        if (lane == 0 && !begun) p.parts[blockIdx.x].valid = 0;
        if (ok) {
            ChunkPiece pc = {};
            pc.last = 1;
            ok = emit(pc);
        }
        // every copy has landed and every product that reads it is complete
        for (int i = 0; ok && i < Cfg::kStages; ++i, ++ring)
            ok = wait(PKV_CTL(empty) + 8 * (ring % Cfg::kStages), (ring / Cfg::kStages & 1) ^ 1);
        for (int b = 0; ok && b < 2; ++b) ok = wait(PKV_CTL(q_empty) + 8 * b, (q_uses >> b & 1) ^ 1);
        if (!ok) {  // gave up: only the copies in flight matter now
            for (uint32_t i = 1; i <= (uint32_t)Cfg::kStages && i <= ring; ++i)
                chunk_drain(PKV_CTL(full) + 8 * ((ring - i) % Cfg::kStages), (ring - i) / Cfg::kStages & 1);
            for (int st = 0; st < Cfg::kStages; ++st)
                if (edge_used >> st & 1) chunk_drain(PKV_CTL(edge) + 8 * st, (edge_phase >> st & 1) ^ 1);
            for (int b = 0; b < 2; ++b)
                if (q_used >> b & 1) chunk_drain(PKV_CTL(q_full) + 8 * b, (q_uses >> b & 1) ^ 1);
        }
    }
};

// ---------------------------------------------------------------------------
// warps 8, 9: the products of a slot each

// A value that is the same in every lane, put in a uniform register: a warp
// reduction leaves it there, where a shuffle or a load would not.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __reduce_or_sync(kFullMask, x); }
__device__ __forceinline__ int uniform(int x) { return (int)uniform((uint32_t)x); }

template <int D>
struct ChunkProducts {
    using Cfg = ChunkConfig<D>;
    using Control = typename Cfg::Control;
    // A place in the ring: its stage and the parity of that stage's use.
    struct Place {
        uint32_t st, phase;
        __device__ void move(uint32_t by) {
            st += by;
            if (st >= Cfg::kStages) {
                st -= Cfg::kStages;
                phase ^= 1;
            }
        }
    };

    const ChunkParams &p;
    Control &ctl;
    uint32_t ctl_at;  // its shared-memory address
    uint32_t q_low, k_low, v_low;  // operand descriptors of the first buffers
    uint32_t s_tmem, o_tmem;
    int slot, lane;
    Place ring = {0, 0};        // of the piece's first copy
    uint32_t q_uses = 0, p_uses = 0, o_uses = 0, merges = 0;  // q: a bit per buffer
    uint32_t guard_phase = 0;   // a bit per stage
    uint32_t mine = 0, theirs = 0;  // batches issued so far, by this slot and (up to the piece) by the other

    __device__ bool wait(uint32_t bar, uint32_t parity) { return chunk_wait(bar, parity, PKV_CTL(abort), p.wait_tries); }

    // The slots take turns at the tensor cores, a whole batch (O of a step, S of
    // the next) at a time: run together, both slots would wait for both batches
    // and then both do their softmax, with the tensor cores idle.  A slot waits
    // until the other has issued so many batches in all.
    __device__ bool turn(uint32_t batches) {
        return chunk_wait_count(PKV_CTL(issued) + 4 * (1 - slot), batches, PKV_CTL(abort), p.wait_tries);
    }

    // S of the slot, whose K is there.
    __device__ void scores(uint32_t q_buffer, uint32_t st) {
        umma_scores<D>(s_tmem, q_low + q_buffer * (Cfg::kTileBytes >> 4), k_low + st * (Cfg::kTileBytes >> 4),
                       umma_idesc_f16(128, kChunkTile, false));
    }

    // O of the slot (+)= P V, in halves of the step's positions, each as soon as its weights are there.
    __device__ bool weighted(uint32_t st, bool begins) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            if (!wait(PKV_CTL(p_full) + 8 * (2 * slot + h), p_uses & 1)) return false;
            tc_fence_after();
            umma_weighted(o_tmem, s_tmem + 32 * h, v_low + st * (Cfg::kTileBytes >> 4) + 512 * h,
                          umma_idesc_f16(128, D, true), !begins || h);
        }
        ++p_uses;
        return true;
    }

    __device__ bool piece(const ChunkPiece &pc) {
        const int t0 = uniform(pc.t0), n = uniform(pc.t1) - t0, single = uniform(pc.single);
        if (n == 0) return true;
        const int all_lo = uniform(pc.all_lo), all_hi = uniform(pc.all_hi);
        const int first = uniform(pc.first[slot]) - t0, end = uniform(pc.end[slot]) - t0, stride = single ? 2 : 1;
        auto takes = [&](int k) { return k >= first && k < end && (!single || ((k - first) & 1) == 0); };
        const int other_first = uniform(pc.first[1 - slot]) - t0, other_end = uniform(pc.end[1 - slot]) - t0;
        // The other slot's batches in this piece: S of its first step, then one per
        // step; with alternate steps S and O of each by themselves, out of turn (its
        // O would wait for this slot's P).
        const uint32_t other_steps = other_first < other_end ? (other_end - other_first + stride - 1) / stride : 0;
        const uint32_t other = single ? 2 * other_steps : other_steps ? other_steps + 1 : 0;
        uint32_t batch = 0;
        const int last = first < end ? (single ? end - 1 - (end - 1 - first & 1) : end - 1) : -1;
        // Queries: a tile of its own each, or one tile for both.  Both warps see every
        // use of a buffer and free it, by a commit behind their last S or at once.
        const int lone = uniform(pc.q_buffer), buffer = single ? lone : slot;
#pragma unroll 1
        for (int b = 0; b < 2; ++b) {
            if (single && b != lone) continue;
            if (!wait(PKV_CTL(q_full) + 8 * b, q_uses >> b & 1)) return false;
            q_uses ^= 1u << b;
            if (b != buffer || first >= end) umma_arrive(PKV_CTL(q_empty) + 8 * b);
        }
        // Both warps go through all copies of the piece and each frees every
        // stage, by a commit where it reads it and at once where it does not: O of
        // step k, then S of step k + 1 (which overwrites P of the slot's last step).
        // Places: K of step k + 1 and V of step k (K0 K1 V0 K2 V1 ... from `ring` on).
        Place kp = ring, vp = ring;
#pragma unroll 1
        for (int k = -1; k < n; ++k) {
            const uint32_t k_st = kp.st, v_st = vp.st;
            const bool edge = k >= 0 && ((t0 + k) * kChunkTile < all_lo || (t0 + k + 1) * kChunkTile > all_hi);
            // Everything but P first, so that nothing stands between P and the products.
            const bool pv = k >= 0 && takes(k), qk = k + 1 < n && takes(k + 1);
            if (k + 1 < n && !wait(PKV_CTL(full) + 8 * k_st, kp.phase)) return false;
            if (pv) {
                if (!wait(PKV_CTL(full) + 8 * v_st, vp.phase)) return false;
                if (edge && !wait(PKV_CTL(guard) + 8 * v_st, guard_phase >> v_st & 1)) return false;
                if (k == first) {  // the previous piece's output has been read
                    if (!wait(PKV_CTL(o_free) + 8 * slot, (o_uses & 1) ^ 1)) return false;
                    if (!wait(PKV_CTL(o_cross) + 8 * slot, (merges & 1) ^ 1)) return false;
                    ++o_uses;
                }
            }
            if (pv || qk) {
                // slot 0's first batch, slot 1's first, slot 0's second ...
                if (!single && !turn(theirs + min(batch + slot, other))) return false;
                ++batch;
                if (pv && !weighted(v_st, k == first)) return false;
                tc_fence_after();
                if (qk) scores(buffer, k_st);
                ++mine;  // (a commit waits for its place behind the products)
                if (lane == 0) *(volatile uint32_t *)&ctl.issued[slot] = mine;
                // what a softmax waits for first
                if (qk) umma_commit(PKV_CTL(s_full) + 8 * slot);
                if (pv && k == last) umma_commit(PKV_CTL(o_full) + 8 * slot);
                if (pv) umma_commit(PKV_CTL(empty) + 8 * v_st);
                if (qk) umma_commit(PKV_CTL(empty) + 8 * k_st);
                if (qk && k + 1 == last) umma_commit(PKV_CTL(q_empty) + 8 * buffer);
            }
            if (k + 1 < n && !qk) umma_arrive(PKV_CTL(empty) + 8 * k_st);
            if (k >= 0 && !takes(k)) {
                if (!wait(PKV_CTL(full) + 8 * v_st, vp.phase)) return false;
                umma_arrive(PKV_CTL(empty) + 8 * v_st);
            }
            if (edge) guard_phase ^= 1u << v_st;
            kp.move(k < 0 ? 1 : 2);
            vp.move(k + 2 >= n ? 1 : 2);
        }
        if (single && n > 1) ++merges;  // the other softmax warpgroup reads this slot's output, too
        ring = vp;
        theirs += other;
        return true;
    }

    __device__ void run() {
        for (uint32_t i = 0;; ++i) {
            const uint32_t at = i % kChunkPieces;
            if (!wait(PKV_CTL(piece_full) + 8 * at, i / kChunkPieces & 1)) break;
            const ChunkPiece &pc = ctl.piece[at];
            if (uniform(pc.last)) break;
            if (!piece(pc)) break;
            umma_arrive(PKV_CTL(piece_empty) + 8 * at);
        }
        umma_commit(PKV_CTL(drain) + 8 * slot);
        chunk_drain(PKV_CTL(drain) + 8 * slot, 0);
    }
};

// ---------------------------------------------------------------------------
// warp 11: V in steps that not every row sees whole

// Rows [a, b) of a tile, 4 rows of 128 bytes at a time, 16 bytes per lane.
template <int D>
__device__ __forceinline__ void guard_clear(unsigned char *tile, int a, int b, int lane) {
#pragma unroll 1
    for (int row = a + lane / 8; row < b; row += 4)
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
            *reinterpret_cast<uint4 *>(tile + h * ChunkConfig<D>::kHalfBytes + row * 128 + lane % 8 * 16) =
                make_uint4(0, 0, 0, 0);
}

// Whether rows [a, b) hold an element that is not finite; those are cleared.
// The magnitudes' maximum, which passes NaN on, finds them at an instruction
// per two elements (rows past the end look at the last one again).
template <int D>
__device__ __forceinline__ bool guard_find(unsigned char *tile, int a, int b, int lane) {
    if (a >= b) return false;
    constexpr int kRows = D == 128 ? 4 : 8;  // 8 loads in flight
    __half2 most[4] = {};
#pragma unroll 1
    for (int r0 = a + lane / 8; r0 < b; r0 += 4 * kRows) {
        uint4 w[kRows][D / 64];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
                w[i][h] = *reinterpret_cast<const uint4 *>(tile + h * ChunkConfig<D>::kHalfBytes +
                                                           min(r0 + 4 * i, b - 1) * 128 + lane % 8 * 16);
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const __half2 *x = reinterpret_cast<const __half2 *>(&w[i][h]);
#pragma unroll
                for (int j = 0; j < 4; ++j) most[j] = __hmax2_nan(most[j], __habs2(x[j]));
            }
    }
    const __half2 all = __hmax2_nan(__hmax2_nan(most[0], most[1]), __hmax2_nan(most[2], most[3]));
    if (!__any_sync(kFullMask, odd_halves(*reinterpret_cast<const uint32_t *>(&all)))) return false;
#pragma unroll 1
    for (int row = a + lane / 8; row < b; row += 4)
#pragma unroll 1
        for (int h = 0; h < D / 64; ++h) {
            uint4 *v = reinterpret_cast<uint4 *>(tile + h * ChunkConfig<D>::kHalfBytes + row * 128 + lane % 8 * 16);
            const uint4 x = *v;
            *v = make_uint4(clear_odd(x.x), clear_odd(x.y), clear_odd(x.z), clear_odd(x.w));
        }
    return true;
}

template <int D>
__device__ void chunk_guard(const ChunkParams &p, typename ChunkConfig<D>::Control &ctl, uint32_t ctl_at,
                            unsigned char *ring, int lane) {
    using Cfg = ChunkConfig<D>;
    using Control = typename Cfg::Control;
    uint32_t ring_at = 0, phase = 0;
    for (uint32_t k = 0;; ++k) {
        const uint32_t slot = k % kChunkPieces;
        if (!chunk_wait(PKV_CTL(piece_full) + 8 * slot, k / kChunkPieces & 1, PKV_CTL(abort), p.wait_tries)) return;
        ChunkPiece &pc = ctl.piece[slot];
        if (pc.last) return;
        const int n = pc.t1 - pc.t0;
        for (int t = pc.t0; t < pc.t1; ++t) {
            if (!chunk_edge(pc, t)) continue;
            const uint32_t at = ring_at + chunk_v_at(t - pc.t0, n), st = at % Cfg::kStages;
            if (!chunk_wait(PKV_CTL(edge) + 8 * st, phase >> st & 1, PKV_CTL(abort), p.wait_tries)) return;
            phase ^= 1u << st;
            // Rows of this step: [keep_lo, keep_hi) are seen by some row of the
            // item, [all_lo, all_hi) by every one.
            const int at0 = t * kChunkTile;
            const int keep_lo = pc.lo - at0, keep_hi = pc.hi - at0, all_lo = pc.all_lo - at0, all_hi = pc.all_hi - at0;
            unsigned char *tile = ring + st * Cfg::kTileBytes;
            guard_clear<D>(tile, 0, min(keep_lo, kChunkTile), lane);
            guard_clear<D>(tile, max(keep_hi, 0), kChunkTile, lane);
            const int from = max(keep_lo, 0), to = min(keep_hi, kChunkTile);
            bool odd = guard_find<D>(tile, from, min(all_lo, to), lane);
            odd |= guard_find<D>(tile, max(max(all_hi, from), min(all_lo, to)), to, lane);
            if (odd) *(volatile int *)&pc.odd = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(PKV_CTL(guard) + 8 * st);
        }
        ring_at += 2 * n;
        __syncwarp();
        if (lane == 0) mbar_arrive(PKV_CTL(piece_empty) + 8 * slot);
    }
}

// ---------------------------------------------------------------------------
// warps 0-7: softmax and output

// The weights of a step, in place, and their sum, where exponents are so large
// that c S - c m rounded on the way would leave fp16's range (or the maximum's
// own weight at 0): the maximum is taken off the scores first, which is exact
// next to it.  Rare, so out of line; the weights of positions [0, 64) overwrite
// scores already read.
__device__ __noinline__ float chunk_far_weights(uint32_t s_at, float m, float sc) {
    float sum = 0.f;
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
        uint32_t x[2][32], w[32];
        tmem_ld32(s_at + 64 * h, x[0]);
        tmem_ld32(s_at + 64 * h + 32, x[1]);
        tmem_wait_ld();
        tmem_pin32(x[0]);
        tmem_pin32(x[1]);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t *y = &x[i / 16][2 * (i % 16)];
            const float a = ex2(fmaf(__uint_as_float(y[0]) - m, sc, kWeightLift));
            const float b = ex2(fmaf(__uint_as_float(y[1]) - m, sc, kWeightLift));
            sum += a + b;
            w[i] = pack_half2(a, b);
        }
        tmem_st32(s_at + 32 * h, w);
        tmem_wait_st();
    }
    return sum;
}

template <int D>
struct ChunkSoftmax {
    using Cfg = ChunkConfig<D>;
    using Control = typename Cfg::Control;
    const ChunkParams &p;
    Control &ctl;
    uint32_t ctl_at;  // its shared-memory address
    uint32_t tmem;  // with this warp's lanes
    int slot, row, lane;
    uint32_t s_uses = 0, o_uses = 0, merges = 0;
    float m, l;     // what the weights are relative to (an unscaled score) and their sum
    bool far;       // some row of the warp has an m whose exponent fp32 holds too coarsely

    __device__ bool wait(uint32_t bar, uint32_t parity) { return chunk_wait(bar, parity, PKV_CTL(abort), p.wait_tries); }
    __device__ void arrive(uint32_t bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    }
    // The exponent that a row's sum and output are relative to; none where it saw nothing.
    __device__ float top() { return l == 0.f ? -INFINITY : fmaf(m, p.scale_log2, -kWeightLift); }
    __device__ bool look_far() { return __any_sync(kFullMask, fabsf(m * p.scale_log2) >= kFarScore && m != -INFINITY); }
    __device__ uint32_t s_at() { return tmem + slot * kChunkTile; }
    __device__ uint32_t o_at(int s) { return tmem + 2 * kChunkTile + s * D; }

    // One step: scores -> weights, in place in tensor memory, handed over in two
    // halves, so that the second product begins under the second half's
    // exponentials: a prompt of 4096 tokens takes 148 us with the step whole, 138
    // in halves, 140 in quarters (each hand-over costs the step a wait for its stores).
    __device__ bool step(int col0, int row_lo, int row_hi, bool first, bool any) {
        if (!wait(PKV_CTL(s_full) + 8 * slot, s_uses & 1)) return false;
        ++s_uses;
        if (!any) {  // no row of this warp is one of the item's: their weights may be anything
            arrive(PKV_CTL(p_full) + 16 * slot);
            arrive(PKV_CTL(p_full) + 16 * slot + 8);
            return true;
        }
        tc_fence_after();
        // Hidden positions become -inf in place first, where there are any: the
        // common code then needs no mask.
        const bool whole = row_hi < 0 || (row_lo <= col0 && col0 + kChunkTile <= row_hi);
        if (!__all_sync(kFullMask, whole)) {
            const unsigned n = (unsigned)max(row_hi - row_lo, 0);
#pragma unroll 1
            for (int c = 0; c < kChunkTile; c += 32) {
                uint32_t x[32];
                tmem_ld32(s_at() + c, x);
                tmem_wait_ld();
                tmem_pin32(x);
                const int a = row_lo - col0 - c;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if ((unsigned)(i - a) >= n) x[i] = 0xff800000u;
                tmem_st32(s_at() + c, x);
            }
            tmem_wait_st();
        }
        const float sc = p.scale_log2;
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_at() + c * 32, s[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_pin32(s[c]);
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 64; ++i)
            top[i % 4] = fmaxf(top[i % 4], fmaxf(__uint_as_float(s[i / 16][2 * (i % 16)]),
                                                 __uint_as_float(s[i / 16][2 * (i % 16) + 1])));
        const float high = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        // What the weights are relative to moves only when the maximum rises by more
        // than a factor 2^kMostRise of the weights (fp16 carries them up to 65504), a
        // published refinement of the running maximum.
        if (first) {
            if (row_hi >= 0) m = high;
            far = look_far();
        } else {
            const bool move = row_hi >= 0 && (high - m) * sc > kMostRise;
            if (__any_sync(kFullMask, move)) {
                const float next = fmaxf(high, m), fade = move ? ex2((m - next) * sc) : 1.f;
                if (move) m = next;
                l *= fade;
                far = look_far();
                const uint64_t fade2 = pack2(fade, fade);
                // the scores' arrival means every earlier product is complete, O's last one among them
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(o_at(slot) + c * 32, o);
                    tmem_wait_ld();
                    tmem_pin32(o);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x, y;
                        unpack2(mul2(pack2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), fade2), x, y);
                        o[2 * i] = __float_as_uint(x);
                        o[2 * i + 1] = __float_as_uint(y);
                    }
                    tmem_st32(o_at(slot) + c * 32, o);
                }
            }
        }
        const float base = m == -INFINITY ? 0.f : fmaf(-m, sc, kWeightLift);  // -top()
        if (far) {
            l += chunk_far_weights(s_at(), m == -INFINITY ? 0.f : m, sc);
            tc_fence_before();
            arrive(PKV_CTL(p_full) + 16 * slot);
            arrive(PKV_CTL(p_full) + 16 * slot + 8);
            return true;
        }
        const uint64_t scale2 = pack2(sc, sc), base2 = pack2(base, base);
        uint64_t sum2[2] = {};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const uint32_t *x = &s[2 * h + i / 16][2 * (i % 16)];
                float a, b;
                unpack2(fma2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])), scale2, base2), a, b);
                a = ex2(a);
                b = ex2(b);
                sum2[i % 2] = add2(sum2[i % 2], pack2(a, b));
                w[i] = pack_half2(a, b);  // the second product's operand type; the sum has the unrounded weights
            }
            tmem_st32(s_at() + 32 * h, w);
            tmem_wait_st();
            tc_fence_before();
            arrive(PKV_CTL(p_full) + 16 * slot + 8 * h);
        }
        float x, y;
        unpack2(add2(sum2[0], sum2[1]), x, y);
        l += x + y;
        return true;
    }

    // Rows go out a thread each, in whole sectors: a store's lanes are on 32
    // different lines, so its cost goes by their number.  An output that is
    // aligned to 16 bytes only takes twice as many.
    __device__ void store_out(__half *dst, const uint32_t (&o)[32], float inv) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            w[i] = pack_half2(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
        if (reinterpret_cast<uintptr_t>(dst) & 16) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint4 *>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            return;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) store_32(dst + 16 * i, w + 8 * i);
    }
    __device__ void store_part(float *dst, const uint32_t (&o)[32]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) store_32(dst + 8 * i, o + 8 * i);
    }

    __device__ bool piece(const ChunkPiece &pc) {
        const int first = pc.first[slot], end = pc.end[slot], stride = pc.single ? 2 : 1;
        const bool merge = pc.single && pc.t1 - pc.t0 > 1;
        // this thread's row: a token of the item and a query head
        const int token = row / p.group + (pc.single ? 0 : slot * p.shape.tile_tokens);
        const int head = pc.kv_head * p.group + row % p.group;
        const bool live = row < p.shape.tile_tokens * p.group && token < pc.tokens &&
                          (slot == 0 || !pc.single || merge);
        int row_lo = 0, row_hi = -1;  // a row of no token: whatever it computes stays in its lane
        if (live) {
            row_hi = pc.len;
            if (p.shape.causal) {
                const int pos = max(pc.pos0 + token, -1);
                row_hi = min(pos + 1, pc.len);
                if (p.shape.window) row_lo = min(max(pos - p.shape.window + 1, 0), row_hi);
            }
        }
        m = 0.f;
        l = 0.f;
        const bool any = __any_sync(kFullMask, live);
#pragma unroll 1
        for (int t = first; t < end; t += stride)
            if (!step(t * kChunkTile, row_lo, row_hi, t == first, any)) return false;

        __half *out = p.out + ((int64_t)(pc.row0 + token) * p.num_heads + head) * D;
        float *part = p.part_o + ((int64_t)pc.part * p.part_rows + (pc.single ? row : slot * kChunkRows + row)) * D;
        float2 *part_ml = p.part_ml + ((int64_t)pc.part * 2 + slot) * kChunkRows + row;
        const bool mine = first < end;
        if (mine) {
            if (!wait(PKV_CTL(o_full) + 8 * slot, o_uses & 1)) return false;
            ++o_uses;
            tc_fence_after();
        }
        if (!merge) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            if (mine) {
#pragma unroll 1
                for (int c = 0; any && c < D / 32; ++c) {
                    uint32_t o[32];
                    tmem_ld32(o_at(slot) + c * 32, o);
                    tmem_wait_ld();
                    tmem_pin32(o);
                    if (live) {
                        if (!pc.partial)
                            store_out(out + c * 32, o, inv);
                        else
                            store_part(part + c * 32, o);
                    }
                }
                tc_fence_before();
                arrive(PKV_CTL(o_free) + 8 * slot);
            } else if (live && !pc.partial) {  // no step of the item is seen by this tile
#pragma unroll
                for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
            }
            if (live) {
                if (pc.partial) *part_ml = make_float2(top(), l);
                if (pc.odd && mine) {
                    if (!pc.partial)
                        chunk_add_odd<D>(p, pc, row_lo, row_hi, out, 0, D);
                    else
                        chunk_add_odd<D>(p, pc, row_lo, row_hi, part, 0, D);
                }
            }
            return true;
        }
        // One tile, alternate steps: join the slots.  Both warpgroups hold the
        // same rows, and a warp reads the other slot's O in its own lanes; each
        // writes half of the columns.
        if (!wait(PKV_CTL(x_empty), (merges & 1) ^ 1)) return false;
        ctl.ml[slot][row] = make_float2(top(), l);
        tc_fence_before();
        arrive(PKV_CTL(x_full));  // this slot's O is complete, too
        if (!wait(PKV_CTL(x_full), merges & 1)) return false;
        tc_fence_after();
        ++merges;
        const float2 a = ctl.ml[0][row], b = ctl.ml[1][row];
        arrive(PKV_CTL(x_empty));
        const float high = fmaxf(a.x, b.x), base = high == -INFINITY ? 0.f : high;
        const float fa = ex2(a.x - base), fb = ex2(b.x - base);
        const float sum = fa * a.y + fb * b.y;
        const float inv = pc.partial ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        const uint64_t fa2 = pack2(fa, fa), fb2 = pack2(fb, fb);
        const int c0 = slot * (D / 2);
#pragma unroll 1
        for (int c = 0; any && c < D / 64; ++c) {
            uint32_t oa[32], ob[32];
            tmem_ld32(o_at(0) + c0 + c * 32, oa);
            tmem_ld32(o_at(1) + c0 + c * 32, ob);
            tmem_wait_ld();
            tmem_pin32(oa);
            tmem_pin32(ob);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float x, y;
                unpack2(fma2(pack2(__uint_as_float(oa[2 * i]), __uint_as_float(oa[2 * i + 1])), fa2,
                             mul2(pack2(__uint_as_float(ob[2 * i]), __uint_as_float(ob[2 * i + 1])), fb2)), x, y);
                oa[2 * i] = __float_as_uint(x);
                oa[2 * i + 1] = __float_as_uint(y);
            }
            if (live) {
                if (!pc.partial)
                    store_out(out + c0 + c * 32, oa, inv);
                else
                    store_part(part + c0 + c * 32, oa);
            }
        }
        tc_fence_before();
        arrive(PKV_CTL(o_free) + 8 * slot);
        arrive(PKV_CTL(o_cross) + 8 * (1 - slot));
        if (live) {
            if (pc.partial) *part_ml = make_float2(high, sum);
            if (pc.odd) {
                if (!pc.partial)
                    chunk_add_odd<D>(p, pc, row_lo, row_hi, out, c0, D / 2);
                else
                    chunk_add_odd<D>(p, pc, row_lo, row_hi, part, c0, D / 2);
            }
        }
        return true;
    }

    __device__ void run() {
        for (uint32_t k = 0;; ++k) {
            const uint32_t at = k % kChunkPieces;
            if (!wait(PKV_CTL(piece_full) + 8 * at, k / kChunkPieces & 1)) return;
            const ChunkPiece &pc = ctl.piece[at];
            if (pc.last || !piece(pc)) return;
            arrive(PKV_CTL(piece_empty) + 8 * at);
        }
    }
};

// ---------------------------------------------------------------------------

template <int D>
__global__ void __launch_bounds__(kChunkThreads, 1) chunk_kernel(const __grid_constant__ ChunkParams p) {
    using Cfg = ChunkConfig<D>;
    extern __shared__ __align__(1024) unsigned char smem[];
    unsigned char *ring = smem + 2 * Cfg::kTileBytes;
    typename Cfg::Control &ctl = *reinterpret_cast<typename Cfg::Control *>(ring + Cfg::kStages * Cfg::kTileBytes);
    const uint32_t ctl_at = smem_addr(&ctl);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

    if (threadIdx.x == 0) {
        for (int i = 0; i < Cfg::kStages; ++i) {
            mbar_init(smem_addr(&ctl.full[i]), 1);
            mbar_init(smem_addr(&ctl.empty[i]), 2);  // both warps of products
            mbar_init(smem_addr(&ctl.edge[i]), 1);
            mbar_init(smem_addr(&ctl.guard[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.q_full[i]), 1);
            mbar_init(smem_addr(&ctl.q_empty[i]), 2);
            mbar_init(smem_addr(&ctl.s_full[i]), 1);
            mbar_init(smem_addr(&ctl.p_full[i][0]), 4);
            mbar_init(smem_addr(&ctl.p_full[i][1]), 4);
            mbar_init(smem_addr(&ctl.o_full[i]), 1);
            mbar_init(smem_addr(&ctl.o_free[i]), 4);
            mbar_init(smem_addr(&ctl.o_cross[i]), 4);
            mbar_init(smem_addr(&ctl.drain[i]), 1);
        }
        mbar_init(smem_addr(&ctl.x_full), 8);
        mbar_init(smem_addr(&ctl.x_empty), 8);
        for (int i = 0; i < kChunkPieces; ++i) {
            mbar_init(smem_addr(&ctl.piece_full[i]), 1);
            mbar_init(smem_addr(&ctl.piece_empty[i]), 11);  // all but the loader
        }
        ctl.abort = 0;
        ctl.issued[0] = ctl.issued[1] = 0;
        fence_barrier_init();
        prefetch_tensormap(&p.tmap_q);
        prefetch_tensormap(&p.tmap_k);
        prefetch_tensormap(&p.tmap_v);
    }
    if (warp == 8) tmem_alloc(smem_addr(&ctl.tmem), 512);
    grid_dependency_wait();
    launch_dependents();

    // Where this CTA's share starts: the units of each thread's run of
    // sequences, their running sum, and the run that holds the share's first
    // unit (the ring's memory is free until the first copy).
    int64_t *run_units = reinterpret_cast<int64_t *>(ring);
    const int per = (p.num_seqs + kChunkThreads - 1) / kChunkThreads;
    int64_t units = 0;
    for (int s = threadIdx.x * per; s < min((int)(threadIdx.x + 1) * per, p.num_seqs); ++s) {
        const ChunkSeq seq = chunk_load_seq(p, s, blockIdx.x == 0);
        units += p.fits_32 ? chunk_units<int32_t>(p.shape, seq) : chunk_units<int64_t>(p.shape, seq);
    }
    run_units[threadIdx.x] = units;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();

    if (warp >= 8) {
        regs_down<88>();
        if (warp == 10) {
            // 12 runs per lane
            int64_t mine = 0;
            for (int i = 0; i < 12; ++i) mine += run_units[lane * 12 + i];
            int64_t upto = mine;
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t x = __shfl_up_sync(kFullMask, upto, d);
                if (lane >= d) upto += x;
            }
            const int64_t total = __shfl_sync(kFullMask, upto, 31);
            const ChunkShares shares = chunk_shares(total, gridDim.x);
            const int64_t u = chunk_share(shares, blockIdx.x), end = chunk_share(shares, blockIdx.x + 1);
            int s = 0;
            int64_t cum = 0;
            if (u < end) {
                const int who = __ffs(__ballot_sync(kFullMask, upto > u)) - 1;
                cum = __shfl_sync(kFullMask, upto - mine, who);
                // the same among that lane's 12 runs
                const int64_t own = lane < 12 ? run_units[who * 12 + lane] : 0;
                int64_t up = own;
                for (int d = 1; d < 12; d <<= 1) {
                    const int64_t x = __shfl_up_sync(kFullMask, up, d);
                    if (lane >= d) up += x;
                }
                const int run = __ffs(__ballot_sync(kFullMask, cum + up > u)) - 1;
                cum += __shfl_sync(kFullMask, up - own, run);
                s = (who * 12 + run) * per;
                while (per > 1) {
                    const ChunkSeq seq = chunk_load_seq(p, s, false);
                    const int64_t x = p.fits_32 ? chunk_units<int32_t>(p.shape, seq) : chunk_units<int64_t>(p.shape, seq);
                    if (cum + x > u) break;
                    cum += x;
                    ++s;
                }
            }
            __syncwarp();
            fence_proxy_async_smem();  // the ring's memory was read and written by ordinary accesses
            ChunkLoader<D> loader{p, ctl, ctl_at, smem_addr(smem), smem_addr(ring), lane};
            loader.shares = shares;
            loader.run(s, cum, u, end);
        } else if (warp == 11) {
            chunk_guard<D>(p, ctl, ctl_at, ring, lane);
        } else {
            const int slot = uniform(warp - 8);
            const uint32_t tmem = uniform(ctl.tmem);
            const uint32_t q = uniform(smem_addr(smem)), kv = uniform(smem_addr(ring));
            ChunkProducts<D> products{p, ctl, ctl_at, umma_desc_low(q, 16), umma_desc_low(kv, 16),
                                      umma_desc_low(kv, Cfg::kHalfBytes), tmem + slot * kChunkTile,
                                      tmem + 2 * kChunkTile + slot * D, slot, lane};
            products.run();
        }
    } else {
        regs_up<208>();
        ChunkSoftmax<D> softmax{p, ctl, ctl_at, ctl.tmem + ((uint32_t)(warp % 4) << 21), warp / 4,
                                (int)threadIdx.x % kChunkRows, lane};
        softmax.run();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_free(ctl.tmem, 512);
    if (threadIdx.x == 0 && ctl.abort) report(p.status, PKV_ERR_DEVICE_TIMEOUT);
}

// The two waits on what never comes, a warp each, and how long each takes to give up.
__global__ void __launch_bounds__(64) chunk_waits_selftest_kernel(int32_t *status, uint64_t *elapsed_ns, uint32_t tries) {
    __shared__ uint64_t bar;
    __shared__ uint32_t counter, abort[2];
    const int warp = threadIdx.x / 32;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&bar), 1);
        counter = abort[0] = abort[1] = 0;
    }
    __syncthreads();
    const uint64_t t0 = global_ns();
    const bool came = warp == 0 ? chunk_wait(smem_addr(&bar), 0, smem_addr(&abort[0]), tries)
                                : chunk_wait_count(smem_addr(&counter), 1, smem_addr(&abort[1]), tries);
    if (threadIdx.x % 32 == 0) {
        elapsed_ns[warp] = global_ns() - t0;
        if (!came && abort[warp]) report(status, PKV_ERR_DEVICE_TIMEOUT);
    }
}

// Joins the parts of items cut between CTAs.  blockIdx.x is the CTA that began
// an item, blockIdx.y 32 of its tiles' rows, four per warp.  Bound by latency:
// the record, then the parts' weights and (of the first two, the usual number)
// outputs together.  The parts are taken in the order of the item's steps.  In
// calls one behind the other a prompt of 4096 tokens takes 137.6 us with this kernel
// and would take 124.0 without it, a window of 1024 77.7 and 64.8, 8 x 12 heads of
// 1500 positions 35.0 and 27.6, 8 single tokens over 8000 to 32768 120.1 and 115.0.
// (Joined inside chunk_kernel by the part that arrives last, an earlier form of
// it took longer than with this one: 158 us against 147.)  At head_dim 128 three
// CTAs per SM leave 80 registers, and 28 bytes are spilled.
constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;

template <int D>
__global__ void __launch_bounds__(kJoinThreads, 3) chunk_join_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int R = kJoinRows / (kJoinThreads / 32);
    constexpr int E = D / 32;  // columns per lane, in a row
    grid_dependency_wait();
    launch_dependents();
    const ChunkPart item = p.parts[blockIdx.x];
    if (!item.valid) return;
    ChunkShape shape = p.shape;
    shape.quantum_shift = chunk_quantum_shift(item.shares);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // The tile and this warp's rows of it.
    const int at = blockIdx.y * kJoinRows + warp * R, slot = at / kChunkRows, row0 = at % kChunkRows;
    const int token0 = slot * p.shape.tile_tokens;
    const int rows = min(p.shape.tile_tokens, item.tokens - token0) * p.group;
    if (row0 >= rows) return;
    const int last = min(R, rows - row0) - 1;  // rows past the end repeat the last one

    float top[R], sum[R], acc[R][E] = {};
#pragma unroll
    for (int r = 0; r < R; ++r) top[r] = -INFINITY, sum[r] = 0.f;
    // Parts 32 CTAs at a time: where there are more, once for the maximum first.
    const bool few = item.cta1 - (int)blockIdx.x < 32;
#pragma unroll 1
    for (int pass = few ? 1 : 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int cta = blockIdx.x; cta <= item.cta1; cta += 32) {
            int a = 0, b = 0;
            if (cta + lane <= item.cta1)
                chunk_part(shape, item.shares, cta + lane, item.start, item.lo, item.hi, &a, &b);
            const int part = 2 * (cta + lane) + (a == 0 ? 1 : 0);
            unsigned has = __ballot_sync(kFullMask, b > a);
            float2 ml[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                ml[r] = make_float2(-INFINITY, 0.f);
                if (b > a) ml[r] = p.part_ml[((int64_t)part * 2 + slot) * kChunkRows + row0 + min(r, last)];
            }
            auto load = [&](int i, float (&v)[R][E]) {
                const float *o = p.part_o + ((int64_t)__shfl_sync(kFullMask, part, i) * p.part_rows + at) * D + lane * E;
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int e = 0; e < E; e += 2) {
                        const float2 x = *reinterpret_cast<const float2 *>(o + min(r, last) * D + e);
                        v[r][e] = x.x;
                        v[r][e + 1] = x.y;
                    }
            };
            float v0[R][E], v1[R][E];
            int i0 = 0, i1 = 0;
            if (pass && has) {
                i0 = __ffs(has) - 1;
                has &= has - 1;
                i1 = has ? __ffs(has) - 1 : i0;
                load(i0, v0);
                load(i1, v1);
            }
            if (few || pass == 0) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float t = ml[r].x;
#pragma unroll
                    for (int d = 16; d; d >>= 1) t = fmaxf(t, __shfl_xor_sync(kFullMask, t, d));
                    top[r] = fmaxf(top[r], t);
                }
                if (pass == 0) continue;
            }
            unsigned seen[R];  // parts whose output counts: a row that sees nothing of a part may have none written
#pragma unroll
            for (int r = 0; r < R; ++r) {
                seen[r] = __ballot_sync(kFullMask, ml[r].y != 0.f);
                ml[r].x = ex2(ml[r].x - (top[r] == -INFINITY ? 0.f : top[r]));
                float t = ml[r].y == 0.f ? 0.f : ml[r].x * ml[r].y;
#pragma unroll
                for (int d = 16; d; d >>= 1) t += __shfl_xor_sync(kFullMask, t, d);
                sum[r] += t;
            }
            auto add = [&](int i, const float (&v)[R][E]) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float w = __shfl_sync(kFullMask, ml[r].x, i);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        if (seen[r] >> i & 1) acc[r][e] = fmaf(w, v[r][e], acc[r][e]);
                }
            };
            add(i0, v0);
            if (has) {
                add(i1, v1);
                has &= has - 1;
            }
#pragma unroll 1
            while (has) {
                const int i = __ffs(has) - 1;
                has &= has - 1;
                load(i, v0);
                add(i, v0);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = row0 + r;
        const float inv = sum[r] == 0.f ? 0.f : 1.f / sum[r];
        const int token = token0 + row / p.group, head = item.kv_head * p.group + row % p.group;
        __half *out = p.out + ((int64_t)(item.row0 + token) * p.num_heads + head) * D + lane * E;
        if (r <= last)
#pragma unroll
            for (int e = 0; e < E; e += 2)
                *reinterpret_cast<__half2 *>(out + e) = __floats2half2_rn(acc[r][e] * inv, acc[r][e + 1] * inv);
    }
}

}  // namespace pkv

#endif  // PKV_CHUNK_IMPL_CUH
