// Host check of the team decode's work split (pkv_team_schedule.h): the shares
// cover every step once and in order, CTAs that share a segment are consecutive,
// no segment is cut within kTeamSnap steps of its ends, and shares are even.
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "pkv_team_schedule.h"

using namespace pkv;

static int failures = 0;
#define CHECK(c)                                                          \
    do {                                                                  \
        if (!(c)) {                                                       \
            std::printf("%s:%d: %s\n", __FILE__, __LINE__, #c);           \
            if (++failures > 20) std::exit(1);                            \
        }                                                                 \
    } while (0)

static void check_split(const std::vector<int> &steps, int heads, int64_t grid, bool walk) {
    const int n = (int)steps.size();
    std::vector<int64_t> cum(n + 1, 0);
    for (int s = 0; s < n; ++s) cum[s + 1] = cum[s] + team_units(steps[s]);
    const int64_t T = cum[n] * heads;
    const int64_t C = team_ctas(T, grid);
    CHECK(C >= 1 && C <= grid);
    for (int s = 0; s < n; ++s) CHECK(team_steps_of(cum.data(), s) == steps[s]);
    // the first segment with steps
    int s0 = 0;
    while (s0 < n && steps[s0] == 0) ++s0;
    TeamPlace at = team_start(cum.data(), n, heads, 0, C);
    CHECK(at.seg == (s0 < n ? s0 : n) * heads && at.step == 0);
    int64_t next_seg = at.seg;  // what the walk has to come to next
    int next_step = 0;
    for (int64_t c = 0; c < C; ++c) {
        const TeamPlace end = team_start(cum.data(), n, heads, c + 1, C);
        CHECK(end.seg > at.seg || (end.seg == at.seg && end.step >= at.step));
        const bool empty = end.seg == at.seg && end.step == at.step;
        if (empty) CHECK(at.step == 0);
        if (end.seg < n * heads) {
            const int len = steps[end.seg / heads];
            CHECK(len > 0 && end.step < len);
            CHECK(end.step == 0 || (end.step > kTeamSnap && len - end.step > kTeamSnap));
        } else {
            CHECK(end.step == 0);
        }
        if (walk && !empty) {
            int64_t units = 0;
            int seg = at.seg, s = seg / heads, lo = at.step;
            while (seg < end.seg || (seg == end.seg && end.step > 0)) {
                const int hi = seg < end.seg ? steps[s] : end.step;
                CHECK(seg == next_seg && lo == next_step && lo < hi);
                std::vector<char> seen(hi - lo, 0);
                for (int w = 0; w < 4; ++w)
                    for (int x = lo + w; x < hi; x += 4) seen[x - lo]++;
                for (char x : seen) CHECK(x == 1);
                units += hi - lo + kTeamPiece;
                next_step = hi;
                if (hi == steps[s]) {
                    int t = s;
                    next_seg = team_next(cum.data(), n, heads, seg, t);
                    next_step = 0;
                    CHECK(next_seg == (int64_t)n * heads || steps[next_seg / heads] > 0);
                }
                if (seg == end.seg) break;
                seg = team_next(cum.data(), n, heads, seg, s);
                lo = 0;
            }
            CHECK(units <= T / C + 1 + 2 * kTeamSnap + 2 * kTeamPiece);
        }
        at = end;
    }
    CHECK(at.seg == n * heads && at.step == 0);
    if (walk) CHECK(next_seg == (int64_t)n * heads && next_step == 0);
}

int main() {
    std::mt19937 rng(5);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    for (int round = 0; round < 6000; ++round) {
        const int n = pick(1, 12), heads = pick(1, 9);
        const int top = round % 3 == 0 ? 3 : round % 3 == 1 ? 40 : 400;
        std::vector<int> steps(n);
        for (auto &s : steps) s = pick(0, 4) == 0 ? 0 : pick(1, top);
        check_split(steps, heads, pick(1, 300), true);
    }
    // long contexts: unit numbers far past 32 bits
    for (int round = 0; round < 200; ++round) {
        const int n = pick(1, 4096);
        std::vector<int> steps(n);
        for (auto &s : steps) s = pick(0, 1 << 27);
        check_split(steps, pick(1, 65536), pick(1, 4096), false);
    }
    // rows
    CHECK(team_rows(0, 4, -1) == 0 && team_rows(17, 4, -1) == 17);
    CHECK(team_rows(17, 4, 1) == 16 && team_rows(17, 4, 2) == 32 && team_rows(17, 4, 9) == 32 && team_rows(0, 4, 9) == 0);
    CHECK(team_rows(1 << 30, 7, -1) == 1 << 30 && team_rows(1 << 30, 3, 1 << 27) == 1 << 30);
    CHECK(team_steps(0, 16) == 0 && team_steps(1, 16) == 1 && team_steps(16, 16) == 1 && team_steps(17, 16) == 2);
    if (failures) return 1;
    std::printf("team schedule ok\n");
    return 0;
}
