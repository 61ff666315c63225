// Matrix product in 8-bit floating point with a scale for each block of 128, and the quantiser that makes
// its operands (sm_103a).
//
//   out[m, n] = sum_b a_scale[m, b] b_scale[n / 128, b] sum_{k in block b} a[m, k] b[n, k]
//
// The codes' products accumulate over one block of 128 k in f32 in TMEM (four tcgen05.mma kind::f8f6f4
// of 32 k each); the epilogue warps then take the block's sums, multiply them by the block's two scales
// and add them to f32 sums in registers.  So scales may be any f32 values (a block whose scales' product is no
// normal f32 value takes them one at a time), and no more than 128 products are added before a scale is applied.  Two or more TMEM buffers let the MMAs of the next blocks run
// meanwhile: a block of a 256 x 256 tile by a pair of CTAs, the widest, takes the tensor cores 512 cycles, its
// 128 x 256 sums a CTA's multiply-adds 256 and its share of shared memory's bandwidth all of it.  The epilogue
// has 168 registers a thread at 320 threads: 128 sums and two chunks of 32 columns in flight do not fit, 112
// and two of 16 do, and 256 x 224 is the tile at work at 4096 x 4096 x 4096 (times at fp8_pick_tile).
//
// A CTA (one per SM, persistent over tiles of 128 x BN; a pair of CTAs: 256 x BN):
//   warp 0     TMA producer: a ring of blocks (A 128 rows, B BN rows or half of them, 128 bytes of k each)
//   warp 1     TMEM allocator and MMA issuer
//   warps 2-9  scaled accumulation and the output: two warps for each TMEM lane quarter, half the
//              columns each
// Rows and k past an operand's end read as zeros; outputs past the end are not stored.
#include <cuda_fp8.h>
#include <string.h>

#include "common.cuh"
#include "dense.h"
#include "dense_tc.cuh"
#include "dense_vec.cuh"
#include "kernels.h"

namespace moe {
namespace {

template <int BN, int KIND>
struct Fp8Cfg {
  static constexpr bool PAIR = KIND == kPairTile, SPLIT = KIND == kSplitTile;
  static constexpr int kABytes = kBM * kScaleBlock;
  static constexpr int kBRows = PAIR ? BN / 2 : BN;  // of B in this CTA
  static constexpr int kStage = kABytes + kBRows * kScaleBlock;
  static constexpr int kBufBytes = kEpiWarps * kStageBuf;
  // what the other CTAs of a split tile send of this CTA's rows
  static constexpr int kPartBytes = SPLIT ? (kSplitMax - 1) * 32 * BN * 4 : 0;
  static constexpr int kStages = (kRingBytes - kBufBytes - kPartBytes) / kStage;
  static constexpr size_t kSmem = (size_t)kStages * kStage + kBufBytes + kPartBytes + 1024;
  static constexpr int kAcc = BN > 128 ? 2 : 4;  // TMEM buffers, one block's sums each
  static constexpr int kTmemCols = BN > 64 ? 512 : kAcc * BN;  // a power of two
  static constexpr int kPer = BN / 2;            // columns of one epilogue warp
  static constexpr int kChunk = kPer % 32 ? 16 : 32;  // columns of one TMEM load
  static_assert(kBRows % 8 == 0 && kPer % 16 == 0 && kAcc * BN <= kTmemCols, "whole swizzle groups and chunks");
};

__device__ __forceinline__ uint32_t idesc_f8(bool a_e5m2, bool b_e5m2, int M, int N) {
  return 1u << 4 | (a_e5m2 ? 1u : 0u) << 7 | (b_e5m2 ? 1u : 0u) << 10 | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(M >> 4) << 24;
}

// columns of TMEM for a whole warp, without the wait
template <int N>
__device__ __forceinline__ void tmem_ld_start(uint32_t taddr, float (&v)[N]) {
  static_assert(N == 16 || N == 32, "");
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
// waits for the loads before it; v passes through, so that nothing reads it earlier
template <int N>
__device__ __forceinline__ void tmem_ld_wait(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
// (a0, a1) += s * (v0, v1), one instruction
__device__ __forceinline__ void fma2(float &a0, float &a1, uint64_t s, float v0, float v1) {
  uint64_t a, v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(v0), "f"(v1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(s), "l"(v));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}
__device__ __forceinline__ uint64_t both(float s) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(s));
  return r;
}

// one value of a staging buffer
template <typename T>
__device__ __forceinline__ T staged(uint32_t a) {
  T v;
  if constexpr (sizeof(T) == 4) {
    uint32_t w;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(a) : "memory");
    memcpy(&v, &w, 4);
  } else {
    uint16_t w;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(w) : "r"(a) : "memory");
    memcpy(&v, &w, 2);
  }
  return v;
}

// A warp's 32 rows of N sums each to `out` from row row0 and column col on; the rows' pieces of 64 bytes
// pass through the warp's staging buffer, so that four threads store a row's piece together.
template <typename T, int N>
__device__ __forceinline__ void store_rows(const Fp8Params &p, int row0, int col, uint32_t buf, const float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  T *out = static_cast<T *>(p.out);
  constexpr int kPiece = 16 / (int)sizeof(T);  // values in 16 bytes; a row's 64 bytes are four of them
#pragma unroll
  for (int c0 = 0; c0 < N; c0 += 4 * kPiece) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int i = c0 + c * kPiece;
      if (i >= N) break;
      uint4 w;
      if constexpr (sizeof(T) == 4)
        w = make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3]));
      else
        w = make_uint4(pack2<T>(v[i], v[i + 1]), pack2<T>(v[i + 2], v[i + 3]), pack2<T>(v[i + 4], v[i + 5]),
                       pack2<T>(v[i + 6], v[i + 7]));
      sts128(buf + piece_at(lane, c), w);
    }
    __syncwarp();
    if (!p.wide) {  // single values, neighbouring threads side by side in a row
      constexpr int kRow = 4 * kPiece, kAtOnce = 32 / kRow, kBatch = 8;  // loads before the first store
      const int c = lane % kRow, left = p.m - row0;
      const bool there = c0 + c < N && col + c0 + c < p.n;
      const uint32_t from = buf + (c % kPiece) * (int)sizeof(T);
      T *dst = out + (size_t)(row0 + lane / kRow) * p.ld_out + col + c0 + c;
#pragma unroll 1
      for (int r0 = lane / kRow; r0 < 32 && r0 - lane / kRow < left; r0 += kBatch * kAtOnce) {
        T x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) x[i] = staged<T>(from + piece_at(r0 + i * kAtOnce, c / kPiece));
#pragma unroll
        for (int i = 0; i < kBatch; ++i, dst += kAtOnce * p.ld_out)
          if (there && r0 + i * kAtOnce < left) *dst = x[i];
      }
      __syncwarp();
      continue;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * i + (lane >> 2), c = c0 + (lane & 3) * kPiece, left = p.n - (col + c);
      if (row0 + r < p.m && c < N && left > 0) {
        T *dst = out + (size_t)(row0 + r) * p.ld_out + col + c;
        const uint4 w = lds128(buf + piece_at(r, lane & 3));
        if (left >= kPiece) {
          *reinterpret_cast<uint4 *>(dst) = w;
        } else {
          const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < kPiece; ++e)
            if (e < left) {
              if constexpr (sizeof(T) == 4)
                reinterpret_cast<uint32_t *>(dst)[e] = q[e];
              else
                reinterpret_cast<uint16_t *>(dst)[e] = (uint16_t)(q[e / 2] >> (16 * (e & 1)));
            }
        }
      }
    }
    __syncwarp();
  }
}

template <int BN, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                      const __grid_constant__ Fp8Params p) {
  using C = Fp8Cfg<BN, KIND>;
  constexpr bool PAIR = C::PAIR, SPLIT = C::SPLIT;
  constexpr int kRows = PAIR ? 2 * kBM : kBM;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[C::kStages], empty_bar[C::kStages], tfull_bar[C::kAcc], tempty_bar[C::kAcc];
  __shared__ __align__(8) uint64_t mma_done_bar, never_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;  // in the pair
  const int share = SPLIT ? (int)cluster_rank() : 0;  // of k
  const int first_tile = PAIR ? blockIdx.x >> 1 : SPLIT ? blockIdx.x / p.splits : blockIdx.x;
  const int tile_step = PAIR ? gridDim.x >> 1 : SPLIT ? p.tiles : gridDim.x;
  const int kb_first = SPLIT ? share * p.kb / p.splits : 0, kb_end = SPLIT ? (share + 1) * p.kb / p.splits : p.kb;
  const uint32_t stage_bytes = C::kStage - (kBM - p.a_rows) * kScaleBlock;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < C::kAcc; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], PAIR ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(&mma_done_bar, 1);
    mbar_init(&never_bar, 1);
    abort_flag = 0;
    issued = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if constexpr (PAIR) tmem_alloc_pair(&tmem_base, C::kTmemCols);
    else tmem_alloc(&tmem_base, C::kTmemCols);
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR || SPLIT) cluster_sync();  // the other CTAs run, and their barriers are initialised
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int *abort_p = &abort_flag;
  pdl_wait();     // from here on what the kernel before it wrote is read
  pdl_trigger();  // the next one may come: not earlier, as it may read before its own wait what this one waited for

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    RingPos<C::kStages> pos;
    int j = 0;
    bool ok = true;
    const uint32_t ring0 = smem_u32(ring), full0 = PAIR ? in_cta(full_bar, 0) : smem_u32(full_bar);
    for (int t = first_tile; ok && t < p.tiles; t += tile_step) {
      int m, n;
      band_tile(t, p.tiles_m, p.tiles_n, m, n);
      const int m0 = m * kRows + (int)rank * kBM, n0 = n * BN + (int)rank * C::kBRows;
      for (int kb = kb_first; kb < kb_end; ++kb, ++j, pos.next()) {
        const int s = pos.slot;
        if (!warp_wait(&empty_bar[s], pos.round ^ 1u, abort_p, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        const uint32_t a = ring0 + s * C::kStage, fb = full0 + 8 * s;
        if (rank == 0) mbar_expect_one(fb, PAIR ? 2 * stage_bytes : stage_bytes);  // both CTAs' bytes
        tma_load_2d_one<PAIR>(a, &tm_a, fb, kb * kScaleBlock, m0);
        tma_load_2d_one<PAIR>(a + C::kABytes, &tm_b, fb, kb * kScaleBlock, n0);
      }
    }
    if (lane == 0) issued = j;
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (rank == 0) {
      if (p.inject && blockIdx.x == 0)  // test hook: a wait that runs out
        (void)warp_wait(&never_bar, 0u, abort_p, p.status, p.wait_ns);
      const uint32_t idesc = idesc_f8(p.a_e5m2, p.b_e5m2, kRows, BN);
      const uint64_t a0 = smem_desc_sw128(smem_u32(ring)), b0 = a0 + (C::kABytes >> 4);
      RingPos<C::kStages> pos;
      RingPos<C::kAcc> acc;
      bool ok = true;
      for (int t = first_tile; ok && t < p.tiles; t += tile_step) {
        for (int kb = kb_first; kb < kb_end; ++kb, pos.next(), acc.next()) {
          if (!warp_wait(&tempty_bar[acc.slot], acc.round ^ 1u, abort_p, p.status, p.wait_ns) ||
              !warp_wait(&full_bar[pos.slot], pos.round, abort_p, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = pos.slot * (C::kStage >> 4), d = tmem + (uint32_t)(acc.slot * BN);
#pragma unroll
          for (int k = 0; k < kScaleBlock / 32; ++k)
            tc_mma_one<PAIR, true>(d, a0 + (at + k * 2), b0 + (at + k * 2), idesc, k ? 1u : 0u);
          tc_commit_one<PAIR>(smem_u32(&empty_bar[pos.slot]));
          tc_commit_one<PAIR>(smem_u32(&tfull_bar[acc.slot]));
        }
      }
      // every MMA this warp issued completes before TMEM is freed
      tc_commit_local_one<PAIR>(smem_u32(&mma_done_bar));
      int no_abort = 0;
      (void)wait_bounded(&mma_done_bar, 0u, &no_abort, p.status, p.wait_ns);
    }
  } else {
    // ---------------- scaled accumulation and output ----------------
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t buf = smem_u32(ring) + C::kStages * C::kStage + (warp - 2) * kStageBuf;
    const uint32_t tempty0 = PAIR ? in_cta(tempty_bar, 0) : smem_u32(tempty_bar);
    RingPos<C::kAcc> acc;
    bool ok = true;
    for (int t = first_tile; t < p.tiles; t += tile_step) {
      int m, n;
      band_tile(t, p.tiles_m, p.tiles_n, m, n);
      const int row0 = m * kRows + (int)rank * kBM + q * 32, col = n * BN + half * C::kPer;
      // the columns span at most two blocks of b_scale; the second begins at column `edge` of them
      const int blk = min(col, p.n - 1) / kScaleBlock, edge = (col / kScaleBlock + 1) * kScaleBlock - col;
      const bool two = edge < C::kPer && col + edge < p.n;
      const bool in = row0 + lane < p.m;
      const float *sa = p.a_scale + (size_t)(in ? row0 + lane : 0) * p.kb;
      const float *sb = p.b_scale + (size_t)blk * p.kb, *sb2 = two ? sb + p.kb : sb;
      float sum[C::kPer];
#pragma unroll
      for (int i = 0; i < C::kPer; ++i) sum[i] = 0.f;
      float next_a = sa[kb_first], next_b = sb[kb_first], next_b2 = sb2[kb_first];
      for (int kb = kb_first; kb < kb_end; ++kb, acc.next()) {
        const float product = next_a * next_b, product2 = next_a * next_b2;
        const uint64_t s1 = both(product), s2 = both(product2);
        const bool apart = __any_sync(0xffffffffu, !scales_multiply(next_a, next_b, product) ||
                                                       !scales_multiply(next_a, next_b2, product2));
        if (kb + 1 < kb_end) {
          next_a = sa[kb + 1];
          next_b = sb[kb + 1];
          next_b2 = sb2[kb + 1];
        }
        if (!warp_wait(&tfull_bar[acc.slot], acc.round, abort_p, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc.slot * BN + half * C::kPer);
        // rare, and so kept out of the registers of what follows (in that loop it spilled 324 bytes of the 256-column
        // tile's): the scales are read again
        if (apart) {
#pragma unroll
          for (int c = 0; c < C::kPer; c += 16) {
            const ScalePair f = scales_apart(sa[kb], (c < edge ? sb : sb2)[kb]);
            float v[16];
            tmem_ld16(tb + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c + i] = fmaf(v[i] * f.first, f.then, sum[c + i]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (PAIR) mbar_arrive_cluster(tempty0 + 8 * acc.slot);
            else mbar_arrive(&tempty_bar[acc.slot]);
          }
          continue;
        }
        constexpr int N = C::kPer / C::kChunk;
        float v[2][C::kChunk];
        tmem_ld_start(tb, v[0]);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          tmem_ld_wait(v[c & 1]);
          if (c + 1 < N) {
            tmem_ld_start(tb + (c + 1) * C::kChunk, v[(c + 1) & 1]);
          } else {  // everything is in registers: the buffer is free
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR) mbar_arrive_cluster(tempty0 + 8 * acc.slot);
              else mbar_arrive(&tempty_bar[acc.slot]);
            }
          }
          const uint64_t s = c * C::kChunk < edge ? s1 : s2;
#pragma unroll
          for (int i = 0; i < C::kChunk; i += 2)
            fma2(sum[c * C::kChunk + i], sum[c * C::kChunk + i + 1], s, v[c & 1][i], v[c & 1][i + 1]);
        }
      }
      if constexpr (SPLIT) {
        // Lane quarter q of the rows belongs to CTA q * splits / 4: it adds the others' sums to its own, in
        // the order of their ranks.
        const int owner = q * p.splits / 4, first_q = owner * 4 / p.splits;
        const uint32_t parts = smem_u32(ring) + C::kStages * C::kStage + C::kBufBytes +
                               (q - first_q) * (p.splits - 1) * 32 * BN * 4;
        auto part_at = [&](int s, int four) { return ((s * (BN / 4) + half * (C::kPer / 4) + four) * 32 + lane) * 16; };
        if (ok && owner != share) {
          const uint32_t to = in_cta_of(parts, owner);
#pragma unroll
          for (int i = 0; i < C::kPer / 4; ++i)
            st_cluster_128(to + part_at(share < owner ? share : share - 1, i), sum[4 * i], sum[4 * i + 1], sum[4 * i + 2],
                           sum[4 * i + 3]);
        }
        cluster_sync();  // every part has arrived
        if (owner != share) break;
        for (int s = 0; s < p.splits - 1; ++s)
#pragma unroll
          for (int i = 0; i < C::kPer / 4; ++i) {
            const uint4 w = lds128(parts + part_at(s, i));
            sum[4 * i] += __uint_as_float(w.x);
            sum[4 * i + 1] += __uint_as_float(w.y);
            sum[4 * i + 2] += __uint_as_float(w.z);
            sum[4 * i + 3] += __uint_as_float(w.w);
          }
      }
      if (!ok) break;
      if (p.out_type == kF32) store_rows<float>(p, row0, col, buf, sum);
      else if (p.out_type == kBF16) store_rows<__nv_bfloat16>(p, row0, col, buf, sum);
      else store_rows<__half>(p, row0, col, buf, sum);
      __syncwarp();
    }
  }
  if constexpr (SPLIT) {
    if (warp < 2) cluster_sync();  // the epilogue warps' barrier counts every thread
  }
  // Copies still in flight after an abort land before a CTA may leave (bounded; in a normal run each has
  // landed long ago).  A peer may have issued stages whose arrival the leader still owes.
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  if (threadIdx.x == 0 && rank == 0) {
    int j = issued, no_abort = 0;
    if constexpr (PAIR) {
      const int theirs = ld_cluster_s32(in_cta(&issued, 1));
      for (; j < theirs; ++j) mbar_arrive_expect_tx(&full_bar[j % C::kStages], stage_bytes);
    }
    for (int s = 0; s < C::kStages; ++s) {
      const int n = j / C::kStages + (s < j % C::kStages ? 1 : 0);
      if (n > 0) (void)wait_bounded(&full_bar[s], (uint32_t)((n - 1) & 1), &no_abort, p.status, p.wait_ns);
    }
  }
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem, C::kTmemCols);
    else tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int BN, int KIND>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &b, const Fp8Params &p, int num_sms, cudaStream_t st) {
  using C = Fp8Cfg<BN, KIND>;
  static std::atomic<unsigned long long> done{0};
  static std::atomic<int> pairs{0};
  if constexpr (C::SPLIT)
    return launch_clusters(fp8_matmul_kernel<BN, KIND>, C::kSmem, done, p.tiles, p.splits, kThreads, st, a, b, p);
  else
    return launch_tiles<C::PAIR>(fp8_matmul_kernel<BN, KIND>, C::kSmem, done, pairs, p.tiles, num_sms, st, a, b, p);
}

// ---- quantiser ----
// A block's scale is its largest magnitude over the largest code (448 or 57344); 1 for a block of
// zeros, at least 2^-126 so that it is a normal number, and with pow2 rounded up to a power of two.  A
// code is the quotient x / scale rounded to nearest even.  (A division for each value made the kernel
// arithmetic-bound: 18.9 us for 4096 x 4096 bf16.)  With the scale's reciprocal r, correctly rounded, q = x r is
// off by a last place at most, its remainder q s - x is exact in one multiply-add, and q - r (q s - x) is the
// correctly rounded quotient, with the sign of a zero (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990); of values below 2^-100, whose remainders may lie below f32's range, q
// may stay as it is.  4096 x 4096 bf16 takes 12.3 us, 11.9 with q alone, which gave 3 to 6 of 10^4 bf16 values
// another code.  The magnitudes are compared as integers, so that a NaN counts as the largest and makes the
// scale NaN.

__device__ __forceinline__ float block_scale(uint32_t amax, bool e5m2, bool pow2) {
  if (amax == 0u) return 1.f;
  float s = __fdiv_rn(__uint_as_float(amax), e5m2 ? 57344.f : 448.f);
  if (s < 1.17549435e-38f) s = 1.17549435e-38f;
  const uint32_t u = __float_as_uint(s);
  if (pow2 && (u & 0x7FFFFFu) && u < 0x7F800000u) s = __uint_as_float((u & 0x7F800000u) + 0x800000u);
  return s;
}

struct Divisor {
  float r, s;
};
// (an infinite scale: every finite value's quotient is 0)
__device__ __forceinline__ Divisor divisor(float scale) {
  return Divisor{__frcp_rn(scale), __float_as_uint(scale) == 0x7F800000u ? 0.f : scale};
}
__device__ __forceinline__ uint32_t codes2(float a, float b, const Divisor &d, bool e5m2) {
  const float2 q = __fmul2_rn(make_float2(a, b), make_float2(d.r, d.r));
  const float2 rest = __ffma2_rn(q, make_float2(d.s, d.s), make_float2(-a, -b));
  return __nv_cvt_float2_to_fp8x2(__ffma2_rn(rest, make_float2(-d.r, -d.r), q), __NV_SATFINITE,
                                  e5m2 ? __NV_E5M2 : __NV_E4M3);
}
__device__ __forceinline__ uint32_t codes4(const float *v, const Divisor &d, bool e5m2) {
  return codes2(v[0], v[1], d, e5m2) | codes2(v[2], v[3], d, e5m2) << 16;
}

// Sixteen lanes take the 128 values of a row's block, eight consecutive ones each.
template <typename T, bool WIDE>
__device__ __forceinline__ void load_part(const QuantiseParams &p, int row, int col, float (&v)[8]) {
  const T *src = static_cast<const T *>(p.x) + (size_t)row * p.ld_x + col;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.f;
  if (row >= p.rows || col >= p.k) return;
  if constexpr (WIDE) {
    load_eight<T, true>(src, 0, 1, 8, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < p.k) v[e] = to_f32(src[e]);
  }
}
template <bool WIDE>
__device__ __forceinline__ void store_part(const QuantiseParams &p, int row, int col, const Divisor &d, const float (&v)[8]) {
  if (row >= p.rows || col >= p.k) return;
  uint8_t *dst = p.codes + (size_t)row * p.ld_codes + col;
  const uint32_t a = codes4(v, d, p.e5m2), b = codes4(v + 4, d, p.e5m2);
  if constexpr (WIDE) {
    *reinterpret_cast<uint2 *>(dst) = make_uint2(a, b);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < p.k) dst[e] = (uint8_t)((e < 4 ? a : b) >> (8 * (e & 3)));
  }
}
__device__ __forceinline__ uint32_t largest(const float (&v)[8]) {
  uint32_t m = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  return m;
}

constexpr int kQuantBlocks = 4;  // neighbouring blocks of a row that 16 lanes take at a time: their loads overlap

template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) quantise_rows_kernel(const __grid_constant__ QuantiseParams p) {
  const int blocks = (p.k + kScaleBlock - 1) / kScaleBlock, per_row = (blocks + kQuantBlocks - 1) / kQuantBlocks;
  const int part = threadIdx.x & 15, step = gridDim.x * 16;
  // where this half warp begins, and by how much it moves on: rows and groups of blocks
  const long long first = (long long)blockIdx.x * 16 + (threadIdx.x >> 4);
  long long row = first / per_row;
  int group = (int)(first % per_row);
  const int rows_on = step / per_row, groups_on = step % per_row;
  pdl_wait();
  // whole warps stay in the loop for the shuffles: a half warp past the end works on nothing
  while (__any_sync(0xffffffffu, row < p.rows)) {
    const int r = row < p.rows ? (int)row : p.rows, b0 = group * kQuantBlocks;
    float v[kQuantBlocks][8];
    uint32_t m[kQuantBlocks];
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) load_part<T, WIDE>(p, r, (b0 + i) * kScaleBlock + part * 8, v[i]);
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) m[i] = largest(v[i]);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < kQuantBlocks; ++i) m[i] = max(m[i], __shfl_xor_sync(0xffffffffu, m[i], o));
#pragma unroll
    for (int i = 0; i < kQuantBlocks; ++i) {
      const float s = block_scale(m[i], p.e5m2, p.pow2);
      store_part<WIDE>(p, r, (b0 + i) * kScaleBlock + part * 8, divisor(s), v[i]);
      if (part == 0 && r < p.rows && b0 + i < blocks) p.scales[(size_t)r * blocks + b0 + i] = s;
    }
    row += rows_on;
    group += groups_on;
    if (group >= per_row) {
      group -= per_row;
      ++row;
    }
  }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) quantise_tiles_kernel(const __grid_constant__ QuantiseParams p) {
  __shared__ uint32_t largest_of[8];
  const int blocks = (p.k + kScaleBlock - 1) / kScaleBlock;
  const int tile_row = blockIdx.x / blocks, b = blockIdx.x % blocks;
  const int row = tile_row * kScaleBlock + (threadIdx.x >> 4), col = b * kScaleBlock + (threadIdx.x & 15) * 8;
  float v[8][8];
  uint32_t m = 0u;
  pdl_wait();
#pragma unroll
  for (int i = 0; i < 8; ++i) load_part<T, WIDE>(p, row + 16 * i, col, v[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, largest(v[i]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) largest_of[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, largest_of[i]);
  const float s = block_scale(m, p.e5m2, p.pow2);
  const Divisor d = divisor(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) store_part<WIDE>(p, row + 16 * i, col, d, v[i]);
  if (threadIdx.x == 0) p.scales[blockIdx.x] = s;
}

template <typename T>
cudaError_t quantise_typed(const QuantiseParams &p, int num_sms, cudaStream_t st) {
  const long long blocks = (p.k + kScaleBlock - 1) / kScaleBlock;
  if (p.tall == 1) {
    const long long per_row = (blocks + kQuantBlocks - 1) / kQuantBlocks;
    const long long ctas = (p.rows * per_row + 15) / 16, most = (long long)num_sms * 3;  // three for each SM (by registers four fit)
    const int grid = (int)(ctas < most ? ctas : most);
    return launch_pdl(p.wide ? quantise_rows_kernel<T, true> : quantise_rows_kernel<T, false>, dim3(grid), dim3(256), 0, st, p);
  }
  const int grid = (int)((p.rows + kScaleBlock - 1) / kScaleBlock * blocks);
  return launch_pdl(p.wide ? quantise_tiles_kernel<T, true> : quantise_tiles_kernel<T, false>, dim3(grid), dim3(256), 0, st, p);
}

long long fp8_tiles(const Fp8Params &p, DenseTile t) {
  const int rows = t.kind == kPairTile ? 2 * kBM : kBM;
  return (long long)((p.m + rows - 1) / rows) * ((p.n + t.bn - 1) / t.bn);
}

}  // namespace

// The tile that takes the least time (see gemm_pick_tile), from what they measured at 4096 x 4096 (us): a k
// block with 256, 224 and 128 columns on a pair 0.47, 0.42 and 0.28, with 128, 64 and 32 on a CTA by
// itself 0.305, 0.265 and 0.26; a launch 3.5 to 4.4, a further wave 0.4 and, of clusters that share a tile's
// k, which make one tile each, 4.2.  4096 rows took 59.4 in 224 columns (four waves; 60.6 since
// scales that do not multiply are told apart), 66.0 in 256, 73.3 in single CTAs' 128.
DenseTile fp8_pick_tile(const Fp8Params &p, int num_sms) {
  const struct {
    DenseTile tile;
    double k_block;
  } all[] = {{{256, kPairTile, 1}, 0.47}, {{224, kPairTile, 1}, 0.42}, {{128, kPairTile, 1}, 0.28},
             {{128, kOneTile, 1}, 0.305}, {{64, kOneTile, 1}, 0.265}, {{32, kOneTile, 1}, 0.26},
             {{64, kSplitTile, 2}, 0.265}, {{64, kSplitTile, 4}, 0.265}};
  DenseTile best = {0, kOneTile, 1};
  double least = 0;
  for (const auto &c : all) {
    const int splits = c.tile.splits;
    if (splits > p.kb) continue;
    const long long units = c.tile.kind == kPairTile || splits == 2 ? num_sms / 2 : splits == 4 ? num_sms * 36 / 152 : num_sms;
    const long long waves = (fp8_tiles(p, c.tile) + units - 1) / units;
    const bool split = c.tile.kind == kSplitTile;
    const double time = (c.tile.kind == kPairTile ? 4.0 : split ? 4.4 : 3.5) + 0.012 * c.tile.bn +
                        waves * c.k_block * ((p.kb + splits - 1) / splits) + (waves - 1) * (split ? 4.2 : 0.4);
    if (best.bn == 0 || time < least) {
      best = c.tile;
      least = time;
    }
  }
  return best;
}

cudaError_t launch_fp8_matmul(DenseTile t, const CUtensorMap &a, const CUtensorMap &b, Fp8Params p, int num_sms,
                              cudaStream_t st) {
  p.tiles_m = (p.m + (t.kind == kPairTile ? 2 : 1) * kBM - 1) / ((t.kind == kPairTile ? 2 : 1) * kBM);
  p.tiles_n = (p.n + t.bn - 1) / t.bn;
  p.tiles = p.tiles_m * p.tiles_n;
  p.splits = t.splits;
#define MOE_LAUNCH(BN, KIND) \
  if (t.bn == BN && t.kind == KIND) return launch<BN, KIND>(a, b, p, num_sms, st)
  MOE_LAUNCH(256, kPairTile);
  MOE_LAUNCH(224, kPairTile);
  MOE_LAUNCH(128, kPairTile);
  MOE_LAUNCH(128, kOneTile);
  MOE_LAUNCH(64, kOneTile);
  MOE_LAUNCH(32, kOneTile);
  MOE_LAUNCH(64, kSplitTile);
#undef MOE_LAUNCH
  return cudaErrorInvalidValue;
}

cudaError_t launch_fp8_quantise(const QuantiseParams &p, int num_sms, cudaStream_t st) {
  if (p.type == kF32) return quantise_typed<float>(p, num_sms, st);
  if (p.type == kBF16) return quantise_typed<__nv_bfloat16>(p, num_sms, st);
  return quantise_typed<__half>(p, num_sms, st);
}

}  // namespace moe
