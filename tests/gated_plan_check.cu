// Host-only check of the choice between narrow tiles and split K for a gated block's
// linear of few rows (schedule.cuh), run on the CPU by tests/test_gated_plan.py: the
// sizes below were timed both ways, and the faster way is taken.  Exit status 1 if not.
#include "schedule.cuh"

#include <cstdio>

using namespace sq::sched;

struct Timed {
    int M, K, F;
    double narrow, split;  // us on 152 SMs
};
static const Timed kTimed[] = {
    {16, 4096, 800, 25.0, 22.3},    {16, 4096, 1600, 24.9, 23.1},   {16, 4096, 4800, 26.9, 29.2},
    {16, 4096, 3200, 25.7, 26.0},   {128, 4096, 3200, 26.6, 27.6},
    {16, 4096, 8192, 30.5, 35.7},   {16, 2048, 1600, 15.1, 19.8},   {16, 2048, 6400, 17.0, 24.6},
    {16, 8192, 4096, 55.3, 39.7},   {16, 8192, 8192, 61.2, 56.5},   {16, 12288, 4864, 80.9, 54.2},
    {128, 4096, 8192, 31.6, 38.6},  {128, 8192, 8192, 62.8, 60.1},  {160, 8192, 4096, 56.5, 48.5},
    {224, 8192, 4096, 56.5, 48.8},  {160, 12288, 4864, 82.1, 66.3}, {224, 12288, 4864, 82.3, 66.8},
    {8, 16384, 7000, 110.9, 90.5},  {200, 16384, 4000, 106.2, 80.2}, {8, 10240, 6500, 70.7, 59.9},
    {200, 5120, 3000, 36.5, 32.7},  {8, 5120, 5000, 37.0, 34.5},
};

int main() {
    int failures = 0;
    for (const Timed &t : kTimed) {
        int grid = 0, tile_n = 0;
        const Schedule sc = plan_gated(t.M, (t.F + 31) / 32 * 64, t.K, 152, true, &grid, &tile_n);
        const bool split = sc.sk_tiles > 0;
        if (split != (t.split < t.narrow) || (!split && tile_n != 128)) {
            std::printf("FAIL %d x %d x %d: split %d, %d columns\n", t.M, t.K, t.F, split, tile_n);
            ++failures;
        }
    }
    std::printf("%d failures\n", failures);
    return failures ? 1 : 0;
}
