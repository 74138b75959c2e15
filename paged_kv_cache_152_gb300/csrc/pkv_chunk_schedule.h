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
    const int w = 2 * c.tile_tokens;
    return (int)(((int64_t)s.n + w - 1) / w);
}

// The positions that some of rows [r0, r1) of a sequence see.
PKV_HD void chunk_range(const ChunkShape &c, const ChunkSeq &s, int64_t r0, int64_t r1, int *lo, int *hi) {
    if (!c.causal) {
        *lo = 0;
        *hi = s.len;
        return;
    }
    const int64_t base = (int64_t)s.len - s.n;
    const int64_t h = chunk_min64(chunk_max64(base + r1, 0), s.len);
    const int64_t l = c.window ? chunk_max64(base + r0 - c.window + 1, 0) : 0;
    *hi = (int)h;
    *lo = (int)chunk_min64(l, h);
}

PKV_HD void chunk_item_range(const ChunkShape &c, const ChunkSeq &s, int64_t i, int *lo, int *hi) {
    const int64_t w = 2 * (int64_t)c.tile_tokens;
    chunk_range(c, s, i * w, chunk_min64((i + 1) * w, s.n), lo, hi);
}

PKV_HD int64_t chunk_cost(const ChunkShape &c, const ChunkSeq &s, int64_t i) {
    int lo, hi;
    chunk_item_range(c, s, i, &lo, &hi);
    return (int64_t)(hi - lo) + c.overhead;
}

// sum over k in [0, m) of max(a + k * w, 0); a > -2^31, w <= 256
PKV_HD int64_t chunk_ramp(int64_t a, int64_t w, int64_t m) {
    const int64_t k0 = a >= 0 ? 0 : (int64_t)(((uint32_t)-a + (uint32_t)w - 1u) / (uint32_t)w);
    if (k0 >= m) return 0;
    const int64_t n = m - k0;
    return n * a + w * (n * (k0 + m - 1) / 2);
}

// Units of a sequence's first i items of one KV head, 0 <= i <= chunk_items.
PKV_HD int64_t chunk_prefix(const ChunkShape &c, const ChunkSeq &s, int64_t i) {
    const int64_t items = chunk_items(c, s);
    if (i == 0) return 0;
    if (!c.causal) return i * ((int64_t)s.len + c.overhead);
    const int64_t w = 2 * (int64_t)c.tile_tokens, base = (int64_t)s.len - s.n;
    const int64_t m = i < items ? i : items - 1;  // items that end at a whole tile pair
    int64_t sum = m * c.overhead + chunk_ramp(base + w, w, m);
    if (c.window) sum -= chunk_ramp(base - c.window + 1, w, m);
    if (i == items) sum += chunk_cost(c, s, items - 1);
    return sum;
}

PKV_HD int64_t chunk_seq_units(const ChunkShape &c, const ChunkSeq &s) {
    if (s.n <= 0) return 0;
    const int64_t per_head = chunk_prefix(c, s, chunk_items(c, s));
    return per_head > kChunkMaxSeqUnits / c.num_kv_heads ? kChunkMaxSeqUnits : per_head * c.num_kv_heads;
}

// Where share k of `shares` starts on a line of `total` units.
PKV_HD int64_t chunk_share(int64_t total, int shares, int k) {
    const int64_t q = total / shares, r = total % shares;
    return q * k + (k < r ? k : r);
}

// The item of a sequence that holds unit x (0 <= x < its units) and the offset
// of x in it.
PKV_HD void chunk_find(const ChunkShape &c, const ChunkSeq &s, int64_t x, int *kv_head, int *item, int64_t *offset) {
    const int items = chunk_items(c, s);
    const int64_t per_head = chunk_prefix(c, s, items);
    const int64_t h = x / per_head;
    x -= h * per_head;
    int a = 0, b = items - 1;  // the largest a with prefix(a) <= x
    while (a < b) {
        const int mid = (int)(((int64_t)a + b + 1) / 2);
        if (chunk_prefix(c, s, mid) <= x)
            a = mid;
        else
            b = mid - 1;
    }
    *kv_head = (int)h;
    *item = a;
    *offset = x - chunk_prefix(c, s, a);
}

PKV_HD int chunk_steps(int lo, int hi) {
    return hi > lo ? (int)(((unsigned)hi + kChunkTile - 1) / kChunkTile - (unsigned)lo / kChunkTile) : 0;
}

// How many of an item's steps lie before offset x of its units.  Not
// decreasing in x, 0 at 0 and all of them at the item's cost, so the pieces
// [step_at(a), step_at(b)) of consecutive offsets partition the steps.
PKV_HD int chunk_step_at(const ChunkShape &c, int lo, int hi, int64_t x) {
    const int steps = chunk_steps(lo, hi);
    if (x >= (int64_t)(hi - lo) + c.overhead) return steps;
    const int64_t y = x - c.overhead;
    if (y <= 0) return 0;
    int t = (int)((unsigned)y / kChunkTile >> c.quantum_shift << c.quantum_shift);  // y < hi - lo
    if (t > steps) t = steps;
    if (t > 0 && steps - t < 1 << c.quantum_shift) t = steps;
    return t;
}

}  // namespace pkv

#endif  // PKV_CHUNK_SCHEDULE_H
