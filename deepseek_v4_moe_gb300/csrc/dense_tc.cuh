// What the dense sublayer's tensor-core kernels share.
#pragma once
#include "common.cuh"

namespace moe {

constexpr int kBM = 128;                             // rows of a tile: the MMA's M
constexpr int kEpiWarps = 8, kThreads = 32 * (2 + kEpiWarps);
constexpr int kRingBytes = 227 * 1024 - 3072;        // what barriers and alignment leave of a CTA's shared memory

// Tile t of tm x tn, in bands of 16 row blocks, so that the CTAs at work at one time share both
// operands in L2.
__device__ __forceinline__ void band_tile(int t, int tm, int tn, int &m, int &n) {
  const int band = t / (16 * tn), first = band * 16, height = min(tm - first, 16);
  t -= band * 16 * tn;
  m = first + t % height;
  n = t / height;
}

}  // namespace moe
