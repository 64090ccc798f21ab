// Host check of the gated forms' plan (plan.h, gated_plan) for any SM count: the
// blocks cover every token, none is empty, they are whole chunks, and there are
// no more of them than fill the GPU unless a block cannot be longer or shorter.
// Prints one line per violation and "checked <n>" at the end; exit status 1 on
// any violation. Built and run by tests/test_gated_plan.py (no GPU).

#include <cstdio>
#include <vector>

#include "plan.h"

using la::Problem;
namespace plan = la::plan;

static int g_bad = 0;
static long long g_checked = 0;

#define EXPECT(cond, ...)                    \
    do {                                     \
        if (!(cond)) {                       \
            ++g_bad;                         \
            std::printf("FAIL %s: ", #cond); \
            std::printf(__VA_ARGS__);        \
            std::printf("\n");               \
        }                                    \
    } while (0)

static void check(const Problem& p, int sms, bool backward) {
    const int per_sm = plan::gated_ctas_per_sm(p, backward);
    const plan::BlockPlan b = plan::gated_plan(p, sms, per_sm, backward);
    const bool tensor = p.d == 128 && p.dtype == 1 && !backward;
    const long long covered = (long long)b.nblk * b.block_tokens;
#define WHAT "bh=%lld N=%d d=%d dtype=%d sms=%d backward=%d: %d blocks of %d", p.bh(), p.N, p.d, p.dtype, sms, backward, b.nblk, b.block_tokens
    EXPECT(per_sm >= 1 && per_sm <= 4, WHAT);
    EXPECT(b.nblk >= 1 && b.block_tokens >= 64 && b.block_tokens % 64 == 0, WHAT);
    EXPECT(covered >= p.N && covered - b.block_tokens < p.N, WHAT);
    EXPECT(!tensor || b.block_tokens >= 256, WHAT);
    // one wave, but for heads that are more than a wave by themselves
    EXPECT((long long)b.nblk * p.bh() <= (long long)per_sm * sms || b.nblk == 1, WHAT);
    // a row of one chunk is never cut
    EXPECT(p.N > 64 || b.nblk == 1, WHAT);
    ++g_checked;
}

int main() {
    for (int sms : {1, 2, 7, 20, 66, 114, 132, 148, 160, 264})
        for (int N : {1, 2, 63, 64, 65, 127, 128, 129, 256, 257, 300, 1000, 1531, 4096, 16384, 65537, 131072, 1 << 30})
            for (auto bh : std::vector<std::pair<int, int>>{{1, 1}, {1, 3}, {2, 8}, {1, 16}, {4, 16}, {3, 37}, {5, 32}, {64, 32}})
                for (int d : {16, 32, 64, 128})
                    for (int dtype : {0, 1})
                        for (bool backward : {false, true}) check(Problem{bh.first, bh.second, N, d, dtype, 0, 1}, sms, backward);
    std::printf("checked %lld\n", g_checked);
    return g_bad ? 1 : 0;
}
