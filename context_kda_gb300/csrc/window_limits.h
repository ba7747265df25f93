// Sizes that the window attention's forward and gradients take (host code without CUDA, so that its edges can be tested by themselves).
#pragma once

#include <cstdint>

namespace kda {

constexpr int32_t WINDOW_MAX_T = INT32_MAX - 512;    // a tile's rows behind the last token are 32-bit numbers too

// T tokens in N sequences, H query heads: a head's tiles of 128 tokens, and one more for each sequence, are blocks of one grid, with the
// sinks' pieces at most twice as many.
inline bool window_sizes_ok(int64_t T, int64_t N, int64_t H) { return T <= WINDOW_MAX_T && (T / 128 + N) * H <= INT32_MAX / 2; }

}  // namespace kda
