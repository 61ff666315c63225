// What the dense sublayer's tensor-core kernels share.
#pragma once
#include <atomic>

#include "common.cuh"

namespace moe {

constexpr int kBM = 128;                             // rows of a tile: the MMA's M
constexpr int kEpiWarps = 8, kThreads = 32 * (2 + kEpiWarps);
constexpr int kRingBytes = 227 * 1024 - 3072;        // what barriers and alignment leave of a CTA's shared memory

// Allows a kernel its dynamic shared memory, once on each device (`done`: one bit a device).
inline cudaError_t allow_smem(const void *kernel, size_t bytes, std::atomic<unsigned long long> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Tile t of tm x tn, in bands of 16 row blocks, so that the CTAs at work at one time share both
// operands in L2.
__device__ __forceinline__ void band_tile(int t, int tm, int tn, int &m, int &n) {
  const int band = t / (16 * tn), first = band * 16, height = min(tm - first, 16);
  t -= band * 16 * tn;
  m = first + t % height;
  n = t / height;
}

}  // namespace moe
