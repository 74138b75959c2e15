// Host check of the chunk attention's work split: for many batches and grids,
// every step of every item is in exactly one share, empty items are met once,
// a share holds at most two partial pieces, the closed-form prefix equals the
// sum, and bisection finds what a walk finds.
#include <stdio.h>
#include <stdlib.h>

#include <map>
#include <tuple>
#include <vector>

#include "pkv_chunk_schedule.h"

using namespace pkv;

#define CHECK(x)                                                       \
    do {                                                               \
        if (!(x)) {                                                    \
            printf("FAILED %s at line %d\n", #x, __LINE__);            \
            exit(1);                                                   \
        }                                                              \
    } while (0)

static unsigned long long rng_state = 88172645463325252ull;
static unsigned rnd(unsigned n) {
    rng_state ^= rng_state << 13;
    rng_state ^= rng_state >> 7;
    rng_state ^= rng_state << 17;
    return (unsigned)(rng_state >> 11) % n;
}

// A row's own visible range, from the definition.
static void row_range(const ChunkShape &c, const ChunkSeq &s, int r, int *lo, int *hi) {
    *lo = 0;
    *hi = s.len;
    if (!c.causal) return;
    const int p = s.len - s.n + r;
    *hi = p + 1 > 0 ? p + 1 : 0;
    if (c.window && p - c.window + 1 > 0) *lo = p - c.window + 1;
}

// The item of a sequence that holds unit x (0 <= x < its units) and the offset of x in it.
template <typename I>
static void find(const ChunkShape &c, const ChunkSeq &s, int64_t x, int *head, int *item, int64_t *offset) {
    const I per_head = chunk_prefix<I>(c, s, chunk_items(c, s));
    *head = (int)(x / per_head);
    x -= (int64_t)*head * per_head;
    int i = 0;
    while (i + 1 < chunk_items(c, s) && chunk_prefix<I>(c, s, i + 1) <= x) ++i;
    *item = i;
    *offset = x - chunk_prefix<I>(c, s, i);
}

template <typename I>
static void check(const ChunkShape &c, const std::vector<ChunkSeq> &seqs, int shares) {
    int64_t total = 0;
    std::vector<int64_t> cum(1, 0);
    for (const ChunkSeq &s : seqs) {
        const int items = s.n > 0 ? chunk_items(c, s) : 0;
        int64_t sum = 0;
        for (int i = 0; i < items; ++i) {
            CHECK(chunk_prefix<I>(c, s, i) == sum);
            int lo, hi, first = 1 << 30, last = 0;
            chunk_item_range(c, s, i, &lo, &hi);
            const int w = 2 * c.tile_tokens;
            for (int r = i * w; r < (i + 1) * w && r < s.n; ++r) {
                int a, b;
                row_range(c, s, r, &a, &b);
                if (b > a) {
                    if (a < first) first = a;
                    if (b > last) last = b;
                }
            }
            if (last > 0)
                CHECK(lo == first && hi == last);
            else
                CHECK(lo == hi);
            CHECK(chunk_cost(c, s, i) == hi - lo + c.overhead);
            sum += chunk_cost(c, s, i);
        }
        if (items) CHECK(chunk_prefix<I>(c, s, items) == sum);
        CHECK(chunk_seq_units<I>(c, s) == sum * c.num_kv_heads);
        total += sum * c.num_kv_heads;
        cum.push_back(total);
    }
    std::map<std::tuple<int, int, int>, int> done;   // item -> steps so far, in order of the shares
    std::map<std::tuple<int, int, int>, int> met;    // empty items
    const ChunkShares cut = chunk_shares(total, shares);
    CHECK(chunk_share(cut, 0) == 0 && chunk_share(cut, shares) == total);
    for (int k = 0; k < shares; ++k) {
        int64_t u = chunk_share(cut, k);
        const int64_t end = chunk_share(cut, k + 1);
        CHECK(end >= u);
        int partial[2] = {0, 0};
        size_t s = 0;
        while (s < seqs.size() && cum[s + 1] <= u) ++s;
        if (u >= end) continue;
        int head, item;
        int64_t off;
        find<I>(c, seqs[s], u - cum[s], &head, &item, &off);
        while (u < end) {
            int lo, hi;
            chunk_item_range(c, seqs[s], item, &lo, &hi);
            const int64_t cost = chunk_cost(c, seqs[s], item);
            CHECK(off >= 0 && off < cost);
            const int64_t b = off + (end - u) < cost ? off + (end - u) : cost;
            const int t0 = chunk_step_at(c, lo, hi, off), t1 = chunk_step_at(c, lo, hi, b);
            const int steps = chunk_steps(lo, hi);
            const auto key = std::make_tuple((int)s, head, item);
            if (steps == 0 && off == 0) ++met[key];
            // the item's parts as any share finds them
            const int64_t start = u - off;
            const int from = chunk_share_of(cut, start), to = chunk_share_of(cut, start + cost - 1);
            CHECK(from <= k && k <= to && chunk_share(cut, from) <= start && start < chunk_share(cut, from + 1));
            int at = 0;
            for (int j = from; j <= to; ++j) {
                int a, b;
                chunk_part(c, cut, j, start, lo, hi, &a, &b);
                CHECK(a == at && b >= a);
                if (j == k) CHECK(a == t0 && b == t1);
                at = b;
            }
            CHECK(at == steps);
            if (t1 > t0) {
                CHECK(done[key] == t0);
                done[key] = t1;
                if (t1 - t0 < steps) ++partial[t0 == 0];
            }
            u += b - off;
            off = 0;
            if (++item == chunk_items(c, seqs[s])) {
                item = 0;
                if (++head == c.num_kv_heads) {
                    head = 0;
                    do ++s;
                    while (s < seqs.size() && seqs[s].n == 0);
                }
            }
        }
        CHECK(partial[0] <= 1 && partial[1] <= 1);
    }
    for (size_t s = 0; s < seqs.size(); ++s)
        for (int h = 0; h < c.num_kv_heads; ++h)
            for (int i = 0; seqs[s].n > 0 && i < chunk_items(c, seqs[s]); ++i) {
                int lo, hi;
                chunk_item_range(c, seqs[s], i, &lo, &hi);
                const auto key = std::make_tuple((int)s, h, i);
                if (chunk_steps(lo, hi))
                    CHECK(done[key] == chunk_steps(lo, hi));
                else
                    CHECK(met[key] == 1);
            }
}

int main() {
    for (int round = 0; round < 4000; ++round) {
        ChunkShape c;
        c.tile_tokens = 128 / (1 + (int)rnd(16));
        c.num_kv_heads = 1 + (int)rnd(4);
        c.causal = rnd(4) != 0;
        c.window = c.causal && rnd(2) ? 1 + (int)rnd(rnd(2) ? 700 : 20) : 0;
        c.overhead = 1 + (int)rnd(400);
        c.quantum_shift = (int)rnd(4);
        std::vector<ChunkSeq> seqs;
        const int n = 1 + (int)rnd(7);
        int row = 0;
        bool any = false;
        for (int s = 0; s < n; ++s) {
            ChunkSeq q;
            q.row0 = row;
            q.len = rnd(5) ? (int)rnd(rnd(2) ? 3000 : 140) : 0;
            q.n = rnd(5) ? (int)rnd(rnd(3) ? 30 : 900) : 0;
            if (rnd(4) && q.n > q.len) q.n = q.len;
            row += q.n;
            any = any || q.n > 0;
            seqs.push_back(q);
        }
        if (!any) continue;
        const int grids[] = {1, 2, 3, 17, 152, 601};
        const int grid = grids[rnd(6)];
        int longest = 0;
        for (const ChunkSeq &q : seqs) longest = q.len > longest ? q.len : longest;
        CHECK(chunk_fits_32(c, row, n, longest));
        check<int64_t>(c, seqs, grid);
        check<int32_t>(c, seqs, grid);
    }
    // Lines that do not fit 32 bits: the closed form against a sum over items.
    for (int round = 0; round < 200; ++round) {
        ChunkShape c = {16 + (int)rnd(112), 1 + (int)rnd(16), 1, rnd(2) ? 1 + (int)rnd(1 << 30) : 0, 256, 1};
        ChunkSeq s = {0, 1 + (int)rnd(1 << 22), 1 + (int)rnd(1 << 30)};
        CHECK(!chunk_fits_32(c, 1 << 30, 1, s.len));
        int64_t sum = 0;
        for (int i = 0; i < chunk_items(c, s); ++i) sum += chunk_cost(c, s, i);
        CHECK(chunk_prefix<int64_t>(c, s, chunk_items(c, s)) == sum);
        CHECK(chunk_seq_units<int64_t>(c, s) == sum * c.num_kv_heads);
        const ChunkShares cut = chunk_shares(sum, 152);
        CHECK(chunk_share(cut, 152) == sum);
        for (int k = 0; k < 152; ++k)
            CHECK(chunk_share_of(cut, chunk_share(cut, k)) == k && chunk_share_of(cut, chunk_share(cut, k + 1) - 1) == k);
        if (chunk_fits_32(c, s.n, 1, s.len)) CHECK(chunk_prefix<int32_t>(c, s, chunk_items(c, s)) == sum);
    }
    printf("chunk schedule ok\n");
    return 0;
}
