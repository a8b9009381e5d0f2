// Index arithmetic of the single-token serving kernels that a host program can
// run as it stands (no CUDA header).
#pragma once

namespace fdllm {

// The pass through a ring of stages in which stage s was last filled, -1 for
// never, when stage `next` of pass `round` would be the next one: the pass whose
// parity a wait for that stage's copies asks for. (A wait for the other parity
// returns at once while they are under way, and not at all once they are there.)
constexpr int last_pass(int s, int next, int round) { return s < next ? round : round - 1; }

// Tiles from that of slot `first` to that of slot len - 1, one where nothing is
// visible (first == len). Lengths reach 2^31 - 2, so nothing is rounded up first.
constexpr int tiles_of(int first, int len, int tile) {
  return len > first ? (len - 1) / tile - first / tile + 1 : 1;
}

}  // namespace fdllm
