// How many stages a ring of steps in shared memory has (host code).
#pragma once

#include <cstdint>

namespace afx {
namespace serve {

// Stages of stage_bytes in `bytes`, `most` at the most, whose steps `warps` warps take in turn: a multiple of them, so that
// each slot belongs to one warp.  A wait for a barrier's phase knows the phase by its parity alone and also passes while the
// phase before it is open.  A warp that waits for every phase of a slot has seen the one before; with five stages and two
// warps a slot's last step was the other warp's, and steps were multiplied before their copies had come (128 tokens by
// 17,401 rows of 5120: 7 calls of 300).  Four stages take 23.4 us there.
constexpr uint32_t ring_stages(uint32_t bytes, uint32_t stage_bytes, uint32_t most, uint32_t warps) {
    const uint32_t n = bytes / stage_bytes < most ? bytes / stage_bytes : most;
    return n - n % warps;
}

}  // namespace serve
}  // namespace afx
