// The walk of the norm-and-rotation kernels over the tokens (ops_rounds.hpp): the
// workgroups' rounds, tpi tokens each, take every token once, up to the largest
// count that a call may have.  Built with undefined-behaviour checks: an overflow of
// the position ends it.
#include <climits>
#include <cstdint>
#include <cstdio>

#include "ops_rounds.hpp"

static bool walk(int tokens, int grid, int tpi) {
    int64_t seen = 0, rounds = 0;
    for (int block = 0; block < grid; ++block) {
        int64_t before = -1;
        for (int t0 = block * tpi; t0 < tokens; t0 = apexw::next_round(t0, grid * tpi, tokens)) {
            if (t0 < 0 || t0 <= before || t0 % (grid * tpi) != block * tpi) return false;
            before = t0;
            seen += tokens - t0 < tpi ? tokens - t0 : tpi;
            if (++rounds > (int64_t)tokens / tpi + grid) return false;
        }
    }
    return seen == tokens;
}

int main() {
    const int top[] = {INT_MAX, INT_MAX - 1, INT_MAX - 3, INT_MAX - 4095, INT_MAX - 4096,
                       INT_MAX - 4097, 1 << 30};
    for (int t : top)
        if (!walk(t, 1024, 4)) return std::printf("%d tokens\n", t), 1;
    for (int t = 0; t < 9000; ++t) {
        const int rounds = (t + 3) / 4, grid = rounds < 1024 ? rounds : 1024;
        if (!walk(t, grid, 4) || !walk(t, t, 1)) return std::printf("%d tokens\n", t), 1;
    }
    std::printf("ok\n");
    return 0;
}
