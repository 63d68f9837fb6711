// The 4-bit KV cache row: layout, sizes and the unpacking of its codes.
//
// A pool row (slot) holds one block of 5 D / 4 bytes per KV head:
//   [0, D/2)            codes of K, 4 bits a channel
//   [D/2, D)            codes of V
//   [D, D + D/8)        (step, lo) of K's groups of 32 channels, fp16 pairs
//   [D + D/8, 5 D / 4)  (step, lo) of V's groups
// and a code c stands for lo + c * step.  Eight channels share a 32-bit
// word: channel 2j lies in bits [4j, 4j + 4), channel 2j + 1 16 bits higher,
// so (word >> 4j) & 0x000f000f is the pair (2j, 2j + 1) in the two halves of
// a packed register, and the same mask on the low or high halves of two
// words pairs one channel of two positions.  A group's 32 codes are one
// 16-byte vector with one (step, lo) word: 160 bytes per head at D = 128,
// five whole 32-byte sectors.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace specdec {

constexpr int kKv4Group = 32;
// inputs beyond this saturate: lo + 15 * step then stays finite in fp16
// (7 * 2^13, plus the roundings of lo and of 15 steps, is below 65504)
constexpr float kKv4Limit = 57344.0f;

__host__ __device__ constexpr int kv4_head_bytes(int D) { return D + D / 4; }

// Nodes of request b (all N without num_nodes; clamped to [0, N]).
__device__ __forceinline__ int kv4_nodes(const int32_t* num_nodes, int b, int N) {
  if (num_nodes == nullptr) return N;
  const int n = __ldg(num_nodes + b);
  return n < 0 ? 0 : (n > N ? N : n);
}

}  // namespace specdec
