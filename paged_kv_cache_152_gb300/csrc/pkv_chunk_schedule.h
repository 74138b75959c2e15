// pkv_chunk_schedule.h -- the chunk attention's work split, shared by the
// kernel and its host check.
//
// An item is two query tiles (up to 2 * tile_tokens tokens of one sequence, all
// query heads of one KV head) and the cache positions [lo, hi) that any of its
// rows sees, in steps of 128.  Items are laid out on a line, sequence by
// sequence, KV head by KV head, item by item, each as long as its positions
// plus a fixed overhead; the line is cut into one equal share per CTA.  A
// share's cuts fall inside items, so a long context is spread over CTAs and
// causal items of different lengths balance; an item in several shares is
// written as pieces, joined afterwards.
//
// The line is never stored: the positions of item i are linear in i (up to a
// clamp at zero, and the last item's end), so the length of a sequence's first
// i items has a closed form and a share's start is found by bisection.
#ifndef PKV_CHUNK_SCHEDULE_H
#define PKV_CHUNK_SCHEDULE_H

#include <stdint.h>

#ifdef __CUDACC__
#define PKV_HD __host__ __device__ __forceinline__
#else
#define PKV_HD inline
#endif

namespace pkv {

constexpr int kChunkTile = 128;  // cache positions of a step

// A sequence's units never exceed this, so that 4096 of them fit 64 bits; only
// a call that would run for years could reach it.
constexpr int64_t kChunkMaxSeqUnits = INT64_C(1) << 50;

struct ChunkShape {
    int tile_tokens;   // tokens of one query tile (128 / group)
    int num_kv_heads;
    int causal;
    int window;        // 0: none
    int overhead;      // units of an item besides its positions, >= 1
    int quantum_shift; // items are cut at multiples of 2^this steps
};

struct ChunkSeq {
    int row0;  // first query row
    int n;     // query rows (tokens)
    int len;   // context length
};

PKV_HD int64_t chunk_max64(int64_t a, int64_t b) { return a > b ? a : b; }
PKV_HD int64_t chunk_min64(int64_t a, int64_t b) { return a < b ? a : b; }

PKV_HD int chunk_items(const ChunkShape &c, const ChunkSeq &s) {
    const unsigned w = 2u * c.tile_tokens;
    return (int)((s.n + w - 1) / w);
}

// The positions that some row of item i sees.
PKV_HD int chunk_min(int a, int b) { return a < b ? a : b; }
PKV_HD int chunk_max(int a, int b) { return a > b ? a : b; }

PKV_HD void chunk_item_range(const ChunkShape &c, const ChunkSeq &s, int64_t i, int *lo, int *hi) {
    *lo = 0;
    *hi = s.len;
    if (!c.causal) return;
    const int w = 2 * c.tile_tokens, r0 = (int)(i * w);          // below s.n
    const int r1 = s.n - r0 < w ? s.n : r0 + w;
    const int base = s.len - s.n;                                 // above -2^31
    *hi = chunk_min(chunk_max(base + r1, 0), s.len);
    if (c.window) *lo = chunk_min(chunk_max(chunk_max(base + r0, -1) - c.window + 1, 0), *hi);
}

// Units of item i (below 2^31: no context is longer than 2^30).
PKV_HD int chunk_cost(const ChunkShape &c, const ChunkSeq &s, int64_t i) {
    int lo, hi;
    chunk_item_range(c, s, i, &lo, &hi);
    return hi - lo + c.overhead;
}

// sum over k in [0, m) of max(a + k * w, 0); a > -2^31, w <= 256
template <typename I>
PKV_HD I chunk_ramp(I a, int w, I m) {
    const I k0 = a >= 0 ? 0 : (I)(((uint32_t)-a + (uint32_t)w - 1u) / (uint32_t)w);
    if (k0 >= m) return 0;
    const I n = m - k0;
    return n * a + w * (n * (k0 + m - 1) / 2);
}

// Units of a sequence's first i items of one KV head, 0 <= i <= chunk_items.
// I is int32_t where chunk_fits_32 (the usual case, and a third of the
// instructions), else int64_t.
template <typename I>
PKV_HD I chunk_prefix(const ChunkShape &c, const ChunkSeq &s, I i) {
    const I items = chunk_items(c, s);
    if (i == 0) return 0;
    if (!c.causal) return i * ((I)s.len + c.overhead);
    const int w = 2 * c.tile_tokens;
    const I base = (I)s.len - s.n;
    const I m = i < items ? i : items - 1;  // items that end at a whole tile pair
    I sum = m * c.overhead + chunk_ramp<I>(base + w, w, m);
    if (c.window) sum -= chunk_ramp<I>(base - c.window + 1, w, m);
    if (i == items) sum += chunk_cost(c, s, items - 1);
    return sum;
}

template <typename I>
PKV_HD int64_t chunk_seq_units(const ChunkShape &c, const ChunkSeq &s) {
    if (s.n <= 0) return 0;
    const I per_head = chunk_prefix<I>(c, s, chunk_items(c, s));
    if (sizeof(I) == 4) return per_head * c.num_kv_heads;
    return per_head > kChunkMaxSeqUnits / c.num_kv_heads ? kChunkMaxSeqUnits : (int64_t)per_head * c.num_kv_heads;
}

// Whether a line of num_tokens rows and num_seqs sequences, none longer than
// longest, is surely so short (2^29 units) that nothing the closed form computes
// on the way leaves 32 bits either.
PKV_HD bool chunk_fits_32(const ChunkShape &c, int num_tokens, int num_seqs, int64_t longest) {
    const int64_t items = num_tokens / (2 * c.tile_tokens) + (int64_t)num_seqs;
    const int64_t each = longest + c.overhead;
    return num_tokens < (1 << 29) && c.window <= (1 << 30) && items < (INT64_C(1) << 29) / each / c.num_kv_heads;
}

// A line of `total` units cut into `shares` equal shares: the first r of them
// have q + 1 units, the others q.
struct ChunkShares {
    int64_t q;
    int r;
};

PKV_HD ChunkShares chunk_shares(int64_t total, int shares) {
    ChunkShares s;
    if (total >> 32 == 0) {
        s.q = (uint32_t)total / (uint32_t)shares;
        s.r = (int)((uint32_t)total % (uint32_t)shares);
    } else {
        s.q = total / shares;
        s.r = (int)(total % shares);
    }
    return s;
}

// Where share k starts.
PKV_HD int64_t chunk_share(const ChunkShares &s, int k) { return s.q * k + (k < s.r ? k : s.r); }

// Where items may be cut: at multiples of 2^this steps, a sixteenth of a share
// or less (up to 8 steps).  A cut off the even share costs less than the pieces
// of a short item: 64 sequences of 5 new tokens over 50 to 900 take 126.8 us with
// cuts at every second step and 117.4 at every fourth (77 steps a share), but
// 8 x 12 heads of 1500 positions 39.8 and 42.3 (13 steps a share), 38.7 at every
// step.
PKV_HD int chunk_quantum_shift(const ChunkShares &s) {
    const int64_t sixteenth = s.q / (16 * kChunkTile);
    return sixteenth >= 8 ? 3 : sixteenth >= 4 ? 2 : sixteenth >= 2 ? 1 : 0;
}

// The share that holds unit x.
PKV_HD int chunk_share_of(const ChunkShares &s, int64_t x) {
    const int64_t longer = (s.q + 1) * s.r;
    if (s.q >> 31 == 0 && x >> 32 == 0)
        return x < longer ? (int)((uint32_t)x / (uint32_t)(s.q + 1)) : s.r + (int)((uint32_t)(x - longer) / (uint32_t)s.q);
    return x < longer ? (int)(x / (s.q + 1)) : s.r + (int)((x - longer) / s.q);
}

PKV_HD int chunk_steps(int lo, int hi) {
    return hi > lo ? (int)(((unsigned)hi + kChunkTile - 1) / kChunkTile - (unsigned)lo / kChunkTile) : 0;
}

// How many of an item's steps lie before offset x of its units.  Not
// decreasing in x, 0 at 0 and all of them at the item's cost, so the pieces
// [step_at(a), step_at(b)) of consecutive offsets partition the steps.
PKV_HD int chunk_step_at(const ChunkShape &c, int lo, int hi, int x) {
    const int steps = chunk_steps(lo, hi);
    if (x >= hi - lo + c.overhead) return steps;
    const int y = x - c.overhead;
    if (y <= 0) return 0;
    int t = (int)((unsigned)y / kChunkTile >> c.quantum_shift << c.quantum_shift);  // y < hi - lo
    if (t > steps) t = steps;
    if (t > 0 && steps - t < 1 << c.quantum_shift) t = steps;
    return t;
}

// The steps [*a, *b) that share k has of the item [lo, hi) which starts at unit
// `start`.  Where they are some but not all, they are the share's part
// (*a == 0) of that item: a share has at most one part that begins an item and
// one that does not.
PKV_HD void chunk_part(const ChunkShape &c, const ChunkShares &s, int k, int64_t start, int lo, int hi, int *a, int *b) {
    const int64_t from = chunk_share(s, k) - start, to = chunk_share(s, k + 1) - start;
    const int cost = hi - lo + c.overhead;
    *a = chunk_step_at(c, lo, hi, (int)chunk_min64(chunk_max64(from, 0), cost));
    *b = chunk_step_at(c, lo, hi, (int)chunk_min64(chunk_max64(to, 0), cost));
}

}  // namespace pkv

#endif  // PKV_CHUNK_SCHEDULE_H
