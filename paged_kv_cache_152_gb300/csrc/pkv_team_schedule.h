// pkv_team_schedule.h -- work split of the team decode (the 8-bit cache's and
// the selected blocks'), shared by host and device so that the host check
// (tests/cpp/test_team_schedule.cpp) runs the same code.
//
// A segment is one (sequence, KV head).  Its rows -- the context's, or with a
// block list the listed blocks' -- are cut into steps of a few rows; steps are
// numbered sequence-major, then KV head, then position:
//
//   g = cum[s] * heads + kvh * n(s) + c,   n(s) = cum[s + 1] - cum[s],
//   T = cum[N] * heads.
//
// The T steps are divided among C CTAs in order.  CTA c's nominal start c T / C
// moves to a segment boundary that lies within `snap` steps, so that a short
// segment is not cut for the sake of a few steps.  A CTA's share is walked by
// all its warps together, one segment's part (a piece) after the other.
#ifndef PKV_TEAM_SCHEDULE_H
#define PKV_TEAM_SCHEDULE_H

#include <stdint.h>

#include "pkv_schedule.h"

namespace pkv {

// Steps of a sequence of `rows` rows.
PKV_HD int64_t team_steps(int64_t rows, int step_rows) { return rows <= 0 ? 0 : (rows + step_rows - 1) / step_rows; }

// Rows of a sequence: the context, or at most `listed` blocks of it (a listed
// block counts as a whole one, the context's last may be anywhere in the list).
PKV_HD int64_t team_rows(int64_t context, int block_shift, int64_t listed) {
    if (listed < 0) return context;
    const int64_t blocks = (context + (int64_t(1) << block_shift) - 1) >> block_shift;
    return (blocks < listed ? blocks : listed) << block_shift;
}

// CTAs that get a share: each of them at least `least` steps.
PKV_HD int64_t team_ctas(int64_t T, int64_t grid, int64_t least) {
    const int64_t c = T / least;
    return c < 1 ? 1 : c < grid ? c : grid;
}

struct TeamPos {
    int s;      // sequence
    int kvh;    // KV head
    int64_t c;  // step in the segment
    int64_t n;  // the segment's steps
};

// Where step g (0 <= g < T) lies.
PKV_HD TeamPos team_locate(const int64_t *cum, int num_seqs, int heads, int64_t g) {
    const int64_t row = div_nonneg(g, heads);  // cum[s] <= row < cum[s + 1]
    int lo = 0, hi = num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] <= row) lo = mid; else hi = mid;
    }
    TeamPos p;
    p.s = lo;
    p.n = cum[lo + 1] - cum[lo];
    const int64_t off = g - cum[lo] * heads;
    p.kvh = (int)div_nonneg(off, p.n);
    p.c = off - p.kvh * p.n;
    return p;
}

// First step of CTA c's share, 0 <= c <= C.  Never decreasing in c: of two
// nominal starts between the same two boundaries the later one is nearer to the
// right and farther from the left.  A share may be empty only where two starts
// moved to the same boundary, so the CTAs that share a segment are consecutive.
PKV_HD int64_t team_start(const int64_t *cum, int num_seqs, int heads, int64_t c, int64_t C, int64_t snap) {
    const int64_t T = cum[num_seqs] * heads;
    const int64_t share = div_nonneg(T, C);  // c T / C without a product past 64 bits
    const int64_t at = c * share + div_nonneg(c * (T - share * C), C);
    if (at <= 0 || at >= T) return at <= 0 ? 0 : T;
    const TeamPos p = team_locate(cum, num_seqs, heads, at);
    const int64_t most = div_nonneg(T, 2 * C + 1);
    if (snap > most) snap = most;
    const int64_t left = p.c, right = p.n - p.c;
    if (left <= right) return left <= snap ? at - left : at;
    return right <= snap ? at + right : at;
}

}  // namespace pkv

#endif  // PKV_TEAM_SCHEDULE_H
