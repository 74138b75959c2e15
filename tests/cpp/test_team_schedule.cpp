// Host check of the team decode's work split (pkv_team_schedule.h): every step
// belongs to one CTA, the walks of a CTA's eight warps cover its share, shares
// that cut a segment are consecutive, and short segments are not cut.
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

static void check_split(const std::vector<int64_t> &steps, int heads, int64_t grid, int64_t least, int64_t snap,
                        bool walk) {
    const int n = (int)steps.size();
    std::vector<int64_t> cum(n + 1, 0);
    for (int s = 0; s < n; ++s) cum[s + 1] = cum[s] + steps[s];
    const int64_t T = cum[n] * heads;
    const int64_t C = team_ctas(T, grid, least);
    CHECK(C >= 1 && C <= grid);
    int64_t last = team_start(cum.data(), n, heads, 0, C, snap);
    CHECK(last == 0);
    int64_t open = -1, open_cta = -1;  // the segment that the previous non-empty share ended inside of
    for (int64_t c = 0; c < C; ++c) {
        const int64_t a = last, b = team_start(cum.data(), n, heads, c + 1, C, snap);
        CHECK(a <= b && b <= T);
        last = b;
        if (a == b) {
            CHECK(open < 0);  // no empty share inside a segment
            continue;
        }
        const TeamPos p = team_locate(cum.data(), n, heads, a);
        const int64_t seg = (int64_t)p.s * heads + p.kvh;
        CHECK(cum[p.s] * heads + p.kvh * p.n + p.c == a && p.c < p.n && p.n == steps[p.s] && p.kvh < heads);
        CHECK((p.c > 0) == (open >= 0));
        if (p.c > 0) CHECK(open == seg && open_cta == c - 1);
        const TeamPos e = team_locate(cum.data(), n, heads, b - 1);
        const bool cut = e.c < e.n - 1;
        if (cut) CHECK(e.n > 1 && (e.c + 1 > snap || e.n - 1 - e.c > snap || snap > T / (2 * C + 1)));
        open = cut ? (int64_t)e.s * heads + e.kvh : -1;
        open_cta = c;
        if (!walk) continue;
        // pieces and steps as the kernel walks them
        std::vector<char> seen(b - a, 0);
        for (int w = 0; w < 8; ++w) {
            for (int64_t g = a + w; g < b; g += 8) seen[g - a]++;
        }
        for (char x : seen) CHECK(x == 1);
        TeamPos at = p;
        for (int64_t g = a; g < b;) {
            const int64_t seg1 = g - at.c + at.n, end = seg1 < b ? seg1 : b;
            for (int64_t x = g; x < end; ++x) {
                const TeamPos y = team_locate(cum.data(), n, heads, x);
                CHECK(y.s == at.s && y.kvh == at.kvh && y.c == at.c + (x - g));
            }
            g = end;
            at.c = 0;
            if (g < b && ++at.kvh == heads) {
                at.kvh = 0;
                do ++at.s; while (cum[at.s + 1] == cum[at.s]);
                at.n = cum[at.s + 1] - cum[at.s];
            }
        }
    }
    CHECK(last == T);
    CHECK(open < 0);
}

int main() {
    std::mt19937 rng(5);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    for (int round = 0; round < 4000; ++round) {
        const int n = pick(1, 12), heads = pick(1, 9);
        const int top = round % 3 == 0 ? 3 : round % 3 == 1 ? 40 : 400;
        std::vector<int64_t> steps(n);
        for (auto &s : steps) s = pick(0, 4) == 0 ? 0 : pick(1, top);
        check_split(steps, heads, pick(1, 200), pick(1, 16), pick(0, 12), true);
    }
    // long contexts: step numbers far past 32 bits
    for (int round = 0; round < 200; ++round) {
        const int n = pick(1, 4096);
        std::vector<int64_t> steps(n);
        for (auto &s : steps) s = (int64_t)pick(0, 1 << 26);
        check_split(steps, pick(1, 65536), pick(1, 4096), 8, 8, false);
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
