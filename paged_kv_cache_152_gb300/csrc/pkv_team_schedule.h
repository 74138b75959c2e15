// pkv_team_schedule.h -- work split of the team decode (the 8-bit cache's and
// the selected blocks'), shared by host and device so that the host check
// (tests/cpp/test_team_schedule.cpp) runs the same code.
//
// A segment is one (sequence, KV head).  Its rows -- the context's, or with a
// block list the listed blocks' -- are cut into steps of a few rows.  A segment
// of n > 0 steps costs n + kTeamPiece units: what a piece costs besides its steps
// (queries in, the warps' outputs joined and written) is that of so many steps.
// Units are numbered sequence-major, then KV head, then position:
//
//   cum[s + 1] = cum[s] + (n(s) > 0 ? n(s) + kTeamPiece : 0),   T = cum[N] * heads,
//
// and divided among C CTAs in order.  CTA c's nominal start c T / C falls into a
// segment, and moves to the segment's start or end where that is at most
// kTeamSnap steps away, so that a short segment is not cut for a few steps.  A
// CTA's share is walked by all its warps together, one segment's part (a piece)
// after the other.
#ifndef PKV_TEAM_SCHEDULE_H
#define PKV_TEAM_SCHEDULE_H

#include <stdint.h>

#include "pkv_schedule.h"

namespace pkv {

// Measured (us) when they were chosen, before weights of two terms (chats 49.8 since,
// few 15.3, batch 178, one 17.3): 64 sequences over 50 to 900, 32 heads, int8 ("chats"), 8 of them
// ("few"), 256 over 256 to 4096, 8 heads, e4m3 ("batch"), one over 20000 ("one"),
// 4 over 5 to 100 ("tiny").
// A piece's cost of 2, 4 and 8 steps: chats 52.8, 48.3, 49.3; batch 178.6, 177.6,
// 176.6; one 16.7, 16.7, 17.7.
constexpr int kTeamPiece = 4;
// Cuts spared up to 4, 8 and 16 steps from a boundary: chats 48.2, 48.3, 47.8; few
// 14.3, 15.5, 14.0; batch 177.8, 177.6, 178.5; one 16.7, 16.7, 18.4.
constexpr int kTeamSnap = 4;
// Units that a CTA gets at the least, 3, 6 and 12: tiny 5.4, 5.4, 6.5, the others level.
constexpr int kTeamLeast = 6;

// Steps of a sequence of `rows` rows.
PKV_HD int team_steps(int64_t rows, int step_rows) { return rows <= 0 ? 0 : (int)((rows + step_rows - 1) / step_rows); }

// Rows of a sequence: the context, or at most `listed` blocks of it (a listed
// block counts as a whole one, the context's last may be anywhere in the list).
PKV_HD int64_t team_rows(int64_t context, int block_shift, int64_t listed) {
    if (listed < 0) return context;
    const int64_t blocks = (context + (int64_t(1) << block_shift) - 1) >> block_shift;
    return (blocks < listed ? blocks : listed) << block_shift;
}

PKV_HD int64_t team_units(int steps) { return steps > 0 ? (int64_t)steps + kTeamPiece : 0; }

// CTAs that get a share.
PKV_HD int64_t team_ctas(int64_t T, int64_t grid) {
    const int64_t c = T / kTeamLeast;
    return c < 1 ? 1 : c < grid ? c : grid;
}

// A place between two steps: segment s * heads + kvh, before its step `step`
// (0 <= step < n); behind the last segment: num_seqs * heads, 0.
struct TeamPlace {
    int seg;
    int step;
};

// Steps of a segment of sequence s.
PKV_HD int team_steps_of(const int64_t *cum, int s) {
    const int64_t units = cum[s + 1] - cum[s];
    return units > 0 ? (int)(units - kTeamPiece) : 0;
}

// The next segment with steps, `seg` being in sequence s (s moves along).
PKV_HD int team_next(const int64_t *cum, int num_seqs, int heads, int seg, int &s) {
    if (++seg < (s + 1) * heads) return seg;
    do ++s; while (s < num_seqs && cum[s + 1] == cum[s]);
    return s * heads;
}

// Where CTA c's share begins, 0 <= c <= C.  Never decreasing in c: of two nominal
// starts between the same two boundaries the later one is nearer to the right
// and farther from the left.  Two starts are equal only at a boundary, so the
// CTAs that share a segment are consecutive.
PKV_HD TeamPlace team_start(const int64_t *cum, int num_seqs, int heads, int64_t c, int64_t C) {
    const int64_t T = cum[num_seqs] * heads;
    const int64_t share = div_nonneg(T, C);  // c T / C without a product past 64 bits
    const int64_t at = c * share + div_nonneg(c * (T - share * C), C);
    if (at >= T) return TeamPlace{num_seqs * heads, 0};
    const int64_t row = div_nonneg(at, heads);  // cum[s] <= row < cum[s + 1]
    int s = 0, hi = num_seqs;
    while (hi - s > 1) {
        const int mid = (s + hi) >> 1;
        if (cum[mid] <= row) s = mid; else hi = mid;
    }
    const int64_t units = cum[s + 1] - cum[s];
    const int64_t off = at - cum[s] * heads;
    const int kvh = (int)div_nonneg(off, units);
    const int n = (int)(units - kTeamPiece);
    const int64_t unit = off - kvh * units;
    const int step = unit < kTeamPiece ? 0 : (int)(unit - kTeamPiece);
    TeamPlace p = {s * heads + kvh, step};
    if (step <= n - step) {
        if (step <= kTeamSnap) p.step = 0;
    } else if (n - step <= kTeamSnap) {
        p.seg = team_next(cum, num_seqs, heads, p.seg, s);
        p.step = 0;
    }
    return p;
}

}  // namespace pkv

#endif  // PKV_TEAM_SCHEDULE_H
