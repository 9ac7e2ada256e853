// ops_rounds.hpp -- a workgroup's walk over the tokens.  Plain C++ with no HIP
// dependency: the host checks of the tests compile it with an ordinary compiler.
#pragma once

namespace apexw {

// The first token of the round after the one at t0 < tokens, `step` tokens further
// on; `tokens` where there is none.  (t0 + step itself may pass 2^31 - 1, which
// tokens may reach.)
constexpr int next_round(int t0, int step, int tokens) {
    return tokens - t0 > step ? t0 + step : tokens;
}

}  // namespace apexw
