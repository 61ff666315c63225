// Matrix products of the gated feed-forward block, forward and backward, on the 5th-generation tensor
// cores (tcgen05, TMEM, TMA), sm_103a.
//
//   forward    g = x Wg^T, u = x Wu^T, h = act(g) u                        kGateUp
//              y = h Wd^T                                                  kDown
//   backward   dh = dy Wd;  dg = dh u act'(g), du = dh act(g), h again     kHiddenGrad
//              dx = dg Wg + du Wu                                          kInputGrad
//              dWg = dg^T x, dWu = du^T x, dWd = dy^T h  (one launch)      kWeightGrad
//
// Every operand is read from the caller's row-major matrices by TMA as it lies: a matrix whose
// contraction runs along its rows' elements is a K-major operand (boxes of 64 k x 128 bytes), one
// whose contraction runs over its rows an MN-major operand (boxes of 64 columns x 64 k rows; the
// instruction descriptor's transpose bits).  Nothing is transposed in memory.  Rows, columns and k
// past a matrix's end read as zeros; outputs past the end are not stored.
//
// Products of 16-bit values are exact in f32 and accumulate in f32 in TMEM.  What is rounded to the
// 16-bit type: h (the down product's operand), dg and du (the operands of three products), the saved
// g and u, and the results.  Each is the operand type of the tensor cores, or the type of the
// caller's tensor.
//
// A CTA (one per SM, persistent over the tiles) makes tiles of 128 x BN:
//   warp 0     TMA producer: a ring of 64-wide k blocks of A (128 rows) and B (BN rows)
//   warp 1     TMEM allocator and MMA issuer (one thread)
//   warps 2-9  epilogue: two warps for each TMEM lane quarter, each every other 16 columns; the
//              accumulator is double buffered, so the next tile's MMAs run under it
// kGateUp makes BN / 2 columns of g and the same of u side by side in one accumulator, so the
// activation and the product need no second pass.
// Every wait is bounded; on expiry the CTA sets the device timeout bit, all roles leave, copies and
// MMAs in flight are waited for (bounded) and TMEM is freed.
#include "common.cuh"
#include "dense.h"
#include "dense_tc.cuh"
#include "dense_vec.cuh"

namespace moe {
namespace {

constexpr int kBK = 64;
constexpr int kABytes = kBM * kBK * 2;

template <int MODE, int BN, bool PAIR>
struct Cfg {
  static constexpr bool kAMn = MODE == kWeightGrad;
  static constexpr bool kBMn = MODE == kHiddenGrad || MODE == kInputGrad || MODE == kWeightGrad;
  // rows of B in this CTA; an MN-major operand comes in whole boxes of 64, of which the last may be used in part
  static constexpr int kBUsed = PAIR ? BN / 2 : BN, kBRows = kBMn ? (kBUsed + 63) / 64 * 64 : kBUsed;
  static constexpr int kStage = kABytes + kBRows * kBK * 2;
  static constexpr int kStages = kRingBytes / kStage;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN > 256 ? 512 : 2 * BN;  // a power of two
  static_assert(BN % 32 == 0 && kBRows % 8 == 0, "whole epilogue chunks and swizzle groups");
};

// MN-major operand in shared memory, SWIZZLE_128B: 64 columns x 8 k rows make 1024 bytes; the next 8 k
// rows follow, and the next 64 columns lie a whole box (64 columns x kBK rows) on.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((kBK * 128) >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

__device__ __forceinline__ uint32_t idesc_16(bool f16, bool a_mn, bool b_mn, int M, int N) {
  const uint32_t fmt = f16 ? 0u : 1u;
  return 1u << 4 | fmt << 7 | fmt << 10 | (a_mn ? 1u : 0u) << 15 | (b_mn ? 1u : 0u) << 16 | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(M >> 4) << 24;
}

struct Tile {
  int prob, m0, n0;  // problem (kWeightGrad), first row, first column (kGateUp: of g and of u)
};

__device__ __forceinline__ Tile tile_of(const GemmParams &p, int t, int rows, int cols) {
  Tile r;
  r.prob = 0;
  int tm = p.tiles_m, tn = p.tiles_n;
  const int each = tm * tn;
  if (t >= each * p.same) {
    t -= each * p.same;
    r.prob = p.same;
    tm = p.tiles_m_last;
    tn = p.tiles_n_last;
  } else {
    r.prob = t / each;
    t -= r.prob * each;
  }
  band_tile(t, tm, tn, r.m0, r.n0);
  r.m0 *= rows;
  r.n0 *= cols;
  return r;
}

// Sixteen consecutive values of a row of T, of which those from column `left` on do not exist (left a
// multiple of 8; the row 16-byte aligned at these columns).
template <typename T>
__device__ __forceinline__ void store16(T *dst, int left, const float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (8 * h < left)
      *reinterpret_cast<uint4 *>(dst + 8 * h) =
          make_uint4(pack2<T>(v[8 * h], v[8 * h + 1]), pack2<T>(v[8 * h + 2], v[8 * h + 3]),
                     pack2<T>(v[8 * h + 4], v[8 * h + 5]), pack2<T>(v[8 * h + 6], v[8 * h + 7]));
}
template <typename T>
__device__ __forceinline__ void load16(const T *src, int left, float (&v)[16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (8 * h < left) w = *reinterpret_cast<const uint4 *>(src + 8 * h);
    unpack2(w.x, v[8 * h], v[8 * h + 1], src);
    unpack2(w.y, v[8 * h + 2], v[8 * h + 3], src);
    unpack2(w.z, v[8 * h + 4], v[8 * h + 5], src);
    unpack2(w.w, v[8 * h + 6], v[8 * h + 7], src);
  }
}

// one thread's row of a finished tile: columns [16 * half, BN) in steps of 32
template <int MODE, int BN, typename T>
__device__ __forceinline__ void epilogue(const GemmParams &p, const Tile &tl, uint32_t tbase, int half, int row) {
  const bool last = tl.prob == p.same;
  const int m = last ? p.m_last : p.m, n = last ? p.n_last : p.n;
  const bool in = row < m;
  constexpr int kCols = MODE == kGateUp ? BN / 2 : BN;
  for (int c0 = half * 16; c0 < kCols; c0 += 32) {
    __syncwarp();  // the TMEM loads take the whole warp
    float v[16], w[16];
    tmem_ld16(tbase + c0, v);
    if constexpr (MODE == kGateUp) tmem_ld16(tbase + BN / 2 + c0, w);
    const int col = tl.n0 + c0, left = n - col;
    if (!in || left <= 0) continue;
    if constexpr (MODE == kGateUp) {
      const size_t at = (size_t)row * n + col;
      if (p.c[1]) {
        store16(static_cast<T *>(p.c[1]) + at, left, v);
        store16(static_cast<T *>(p.c[2]) + at, left, w);
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = act_value(p.act, v[j]) * w[j];
      store16(static_cast<T *>(p.c[0]) + at, left, v);
    } else if constexpr (MODE == kHiddenGrad) {
      const size_t at = (size_t)row * n + col;
      float g[16], u[16];
      load16(static_cast<const T *>(p.e[0]) + at, left, g);
      load16(static_cast<const T *>(p.e[1]) + at, left, u);
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        float a, da;
        act_both(p.act, g[j], a, da);
        g[j] = v[j] * u[j] * da;  // dg
        w[j] = a * u[j];          // h
        v[j] *= a;                // du
      }
      store16(static_cast<T *>(p.c[0]) + at, left, g);
      store16(static_cast<T *>(p.c[1]) + at, left, v);
      store16(static_cast<T *>(p.c[2]) + at, left, w);
    } else {
      store16(static_cast<T *>(p.c[tl.prob]) + (size_t)row * p.ldc[tl.prob] + col, left, v);
    }
  }
}

template <int MODE, int BN, bool PAIR>
__global__ void __launch_bounds__(kThreads, 1)
    dense_gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams p) {
  using C = Cfg<MODE, BN, PAIR>;
  constexpr int kCols = MODE == kGateUp ? BN / 2 : BN;  // output columns of a tile
  constexpr int kRows = PAIR ? 2 * kBM : kBM;           // output rows of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[C::kStages], empty_bar[C::kStages], tfull_bar[2], tempty_bar[2];
  __shared__ __align__(8) uint64_t mma_done_bar, never_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;
  const int first_tile = PAIR ? blockIdx.x >> 1 : blockIdx.x, tile_step = PAIR ? gridDim.x >> 1 : gridDim.x;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
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
  if constexpr (PAIR) cluster_sync();  // the peer's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int *abort_p = &abort_flag;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    RingPos<C::kStages> pos;
    int j = 0;
    bool ok = true;
    const uint32_t ring0 = smem_u32(ring), full0 = PAIR ? in_cta(full_bar, 0) : smem_u32(full_bar);
    for (int t = first_tile; ok && t < p.tiles; t += tile_step) {
      const Tile tl = tile_of(p, t, kRows, kCols);
      const int m0 = tl.m0 + (int)rank * kBM, n0 = tl.n0 + (MODE == kGateUp ? 0 : (int)rank * C::kBUsed);
      for (int kb = 0; kb < p.kb; ++kb, ++j, pos.next()) {
        const int s = pos.slot;
        if (!warp_wait(&empty_bar[s], pos.round ^ 1u, abort_p, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        // the second pair of matrices follows the first along k (kInputGrad)
        const int src = MODE == kWeightGrad ? tl.prob : (MODE == kInputGrad && kb >= p.kb0 ? 1 : 0);
        const int k0 = (MODE == kInputGrad && kb >= p.kb0 ? kb - p.kb0 : kb) * kBK;
        // the leader's barrier counts both CTAs' bytes
        if (rank == 0) mbar_expect_one(full0 + 8 * s, PAIR ? 2 * C::kStage : C::kStage);
        const uint32_t a = ring0 + s * C::kStage, b = a + kABytes, fb = full0 + 8 * s;
        if constexpr (C::kAMn) {
          tma_load_2d_one<PAIR>(a, &maps.a[src], fb, m0, k0);
          tma_load_2d_one<PAIR>(a + kBK * 128, &maps.a[src], fb, m0 + 64, k0);
        } else {
          tma_load_2d_one<PAIR>(a, &maps.a[src], fb, k0, m0);
        }
        if constexpr (C::kBMn) {
#pragma unroll
          for (int i = 0; i < C::kBRows / 64; ++i)
            tma_load_2d_one<PAIR>(b + i * kBK * 128, &maps.b[src], fb, n0 + 64 * i, k0);
        } else if constexpr (MODE == kGateUp) {
          if constexpr (PAIR) {  // the leader holds the gate's rows, its peer the up projection's
            tma_load_2d_one<PAIR>(b, &maps.b[rank], fb, k0, n0);
          } else {
            tma_load_2d_one<PAIR>(b, &maps.b[0], fb, k0, n0);
            tma_load_2d_one<PAIR>(b + (BN / 2) * 128, &maps.b[1], fb, k0, n0);
          }
        } else {
          tma_load_2d_one<PAIR>(b, &maps.b[0], fb, k0, n0);
        }
      }
    }
    if (lane == 0) issued = j;
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (rank == 0) {
      if (p.inject && blockIdx.x == 0)  // test hook: a wait that runs out
        (void)warp_wait(&never_bar, 0u, abort_p, p.status, p.wait_ns);
      const uint32_t idesc = idesc_16(p.f16, C::kAMn, C::kBMn, kRows, BN);
      // 16 k are 32 bytes of a K-major row, or 16 rows of 128 bytes of an MN-major box
      const uint64_t ring_d = (uint64_t)(smem_u32(ring) >> 4);
      const uint64_t a0 = (C::kAMn ? smem_desc_mn(0) : smem_desc_sw128(0)) + ring_d;
      const uint64_t b0 = (C::kBMn ? smem_desc_mn(0) : smem_desc_sw128(0)) + ring_d + (kABytes >> 4);
      constexpr int kAStep = (C::kAMn ? 2048 : 32) >> 4, kBStep = (C::kBMn ? 2048 : 32) >> 4;
      RingPos<C::kStages> pos;
      RingPos<2> acc;
      bool ok = true;
      for (int t = first_tile; ok && t < p.tiles; t += tile_step, acc.next()) {
        if (!warp_wait(&tempty_bar[acc.slot], acc.round ^ 1u, abort_p, p.status, p.wait_ns)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc.slot * BN);
        for (int kb = 0; kb < p.kb; ++kb, pos.next()) {
          if (!warp_wait(&full_bar[pos.slot], pos.round, abort_p, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = pos.slot * (C::kStage >> 4);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tc_mma_one<PAIR, false>(d, a0 + (at + k * kAStep), b0 + (at + k * kBStep), idesc, (kb | k) ? 1u : 0u);
          tc_commit_one<PAIR>(smem_u32(&empty_bar[pos.slot]));
        }
        if (ok) tc_commit_one<PAIR>(smem_u32(&tfull_bar[acc.slot]));
      }
      // every MMA this warp issued completes before TMEM is freed
      tc_commit_local_one<PAIR>(smem_u32(&mma_done_bar));
      int no_abort = 0;
      (void)wait_bounded(&mma_done_bar, 0u, &no_abort, p.status, p.wait_ns);
    }
  } else if (warp >= 2) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, half = (warp - 2) >> 2;
    int it = 0;
    for (int t = first_tile; t < p.tiles; t += tile_step, ++it) {
      const int acc = it & 1;
      int ready = 0;
      if (lane == 0)
        ready = wait_bounded(&tfull_bar[acc], (uint32_t)(it >> 1) & 1u, abort_p, p.status, p.wait_ns) ? 1 : 0;
      if (!__shfl_sync(0xffffffffu, ready, 0)) break;
      tc_fence_after();
      const Tile tl = tile_of(p, t, kRows, kCols);
      const int row = tl.m0 + (int)rank * kBM + q * 32 + lane;
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      if (p.f16)
        epilogue<MODE, BN, __half>(p, tl, tbase, half, row);
      else
        epilogue<MODE, BN, __nv_bfloat16>(p, tl, tbase, half, row);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_cluster(in_cta(&tempty_bar[acc], 0));
        else mbar_arrive(&tempty_bar[acc]);
      }
    }
  }
  // Copies still in flight after an abort land before a CTA may leave: the barriers that count them are
  // waited for (bounded; in a normal run each completed long ago).  A peer may have issued stages whose
  // arrival the leader still owes.
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();
  if (threadIdx.x == 0 && rank == 0) {
    int j = issued, no_abort = 0;
    if constexpr (PAIR) {
      const int theirs = ld_cluster_s32(in_cta(&issued, 1));
      for (; j < theirs; ++j) mbar_arrive_expect_tx(&full_bar[j % C::kStages], C::kStage);
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

int cdiv(int a, int b) { return (a + b - 1) / b; }

template <int MODE, int BN, bool PAIR>
cudaError_t launch(const GemmMaps &maps, const GemmParams &p, int num_sms, cudaStream_t st) {
  using C = Cfg<MODE, BN, PAIR>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem((const void *)dense_gemm_kernel<MODE, BN, PAIR>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {PAIR ? 2u : 1u, 1u, 1u};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 1 : 0;
  int units = num_sms;
  if constexpr (PAIR) {  // pairs that run at one time
    static std::atomic<int> pairs{0};
    units = pairs.load(std::memory_order_relaxed);
    if (!units) {
      const cudaError_t q = cudaOccupancyMaxActiveClusters(&units, dense_gemm_kernel<MODE, BN, PAIR>, &cfg);
      if (q != cudaSuccess) return q;
      if (units < 1 || units > num_sms / 2) units = num_sms / 2;
      pairs.store(units, std::memory_order_relaxed);
    }
  }
  const int busy = p.tiles < units ? p.tiles : units;
  cfg.gridDim = dim3(PAIR ? 2 * busy : busy);
  return cudaLaunchKernelEx(&cfg, dense_gemm_kernel<MODE, BN, PAIR>, maps, p);
}

long long tiles_of(int mode, const GemmParams &p, GemmTile g) {
  const int cols = mode == kGateUp ? g.bn / 2 : g.bn, rows = g.pair ? 2 * kBM : kBM;
  return (long long)cdiv(p.m, rows) * cdiv(p.n, cols) * p.same + (long long)cdiv(p.m_last, rows) * cdiv(p.n_last, cols);
}

}  // namespace

int GemmTile::b_box(int mode) const {
  if (mode == kHiddenGrad || mode == kInputGrad || mode == kWeightGrad) return 64;
  return mode == kGateUp || pair ? bn / 2 : bn;
}

// The tile whose waves over the SMs cost least.  A wave's cost in a tile's time, in units of one
// column of a 128-row tile at the tensor cores' rate: a pair's tile has its operands shared, a single
// CTA's waits for shared memory below 256 columns, and every k block has a part that does not shrink.
GemmTile gemm_pick_tile(int mode, const GemmParams &p, int num_sms) {
  const bool b_mn = mode == kHiddenGrad || mode == kInputGrad || mode == kWeightGrad;
  GemmTile best = {256, true};
  const long long pairs = num_sms / 2;
  double least = (double)((tiles_of(mode, p, best) + pairs - 1) / pairs) * 256;
  for (int bn = 256; bn >= (b_mn ? 64 : 32); bn /= 2) {
    const GemmTile g = {bn, false};
    const double cost = (double)((tiles_of(mode, p, g) + num_sms - 1) / num_sms) * (1.1 * bn + 40);
    if (cost < least) {
      best = g;
      least = cost;
    }
  }
  return best;
}

cudaError_t launch_dense_gemm(int mode, GemmTile g, const GemmMaps &maps, GemmParams p, int num_sms, cudaStream_t st) {
  const int cols = mode == kGateUp ? g.bn / 2 : g.bn, rows = g.pair ? 2 * kBM : kBM;
  p.tiles_m = cdiv(p.m, rows);
  p.tiles_n = cdiv(p.n, cols);
  p.tiles_m_last = cdiv(p.m_last, rows);
  p.tiles_n_last = cdiv(p.n_last, cols);
  p.tiles = (int)tiles_of(mode, p, g);
#define MOE_LAUNCH(MODE, BN, PAIR) \
  if (mode == MODE && g.bn == BN && g.pair == PAIR) return launch<MODE, BN, PAIR>(maps, p, num_sms, st)
#define MOE_LAUNCH_ALL(MODE)     \
  MOE_LAUNCH(MODE, 256, true);   \
  MOE_LAUNCH(MODE, 224, true);   \
  MOE_LAUNCH(MODE, 192, true);   \
  MOE_LAUNCH(MODE, 160, true);   \
  MOE_LAUNCH(MODE, 128, true);   \
  MOE_LAUNCH(MODE, 256, false);  \
  MOE_LAUNCH(MODE, 128, false);  \
  MOE_LAUNCH(MODE, 64, false)
  MOE_LAUNCH_ALL(kGateUp);
  MOE_LAUNCH(kGateUp, 32, false);
  MOE_LAUNCH_ALL(kDown);
  MOE_LAUNCH(kDown, 32, false);
  MOE_LAUNCH_ALL(kHiddenGrad);
  MOE_LAUNCH_ALL(kInputGrad);
  MOE_LAUNCH_ALL(kWeightGrad);
#undef MOE_LAUNCH_ALL
#undef MOE_LAUNCH
  return cudaErrorInvalidValue;
}

}  // namespace moe
