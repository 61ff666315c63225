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

template <int MODE, int BN>
struct Cfg {
  static constexpr bool kAMn = MODE == kWeightGrad;
  static constexpr bool kBMn = MODE == kHiddenGrad || MODE == kInputGrad || MODE == kWeightGrad;
  static constexpr int kStage = kABytes + BN * kBK * 2;
  static constexpr int kStages = kRingBytes / kStage;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
  static constexpr int kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
  static_assert(!kBMn || BN % 64 == 0, "an MN-major operand comes in 64-column boxes");
};

// MN-major operand in shared memory, SWIZZLE_128B: 64 columns x 8 k rows make 1024 bytes; the next 8 k
// rows follow, and the next 64 columns lie a whole box (64 columns x kBK rows) on.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | (uint64_t)((kBK * 128) >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1u << 46 | (uint64_t)2u << 61;
}

__device__ __forceinline__ uint32_t idesc_16(bool f16, bool a_mn, bool b_mn, int N) {
  const uint32_t fmt = f16 ? 0u : 1u;
  return 1u << 4 | fmt << 7 | fmt << 10 | (a_mn ? 1u : 0u) << 15 | (b_mn ? 1u : 0u) << 16 | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(kBM >> 4) << 24;
}

struct Tile {
  int prob, m0, n0;  // problem (kWeightGrad), first row, first column (kGateUp: of g and of u)
};

__device__ __forceinline__ Tile tile_of(const GemmParams &p, int t, int cols) {
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
  r.m0 *= kBM;
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

template <int MODE, int BN>
__global__ void __launch_bounds__(kThreads, 1)
    dense_gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams p) {
  using C = Cfg<MODE, BN>;
  constexpr int kCols = MODE == kGateUp ? BN / 2 : BN;  // output columns of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[C::kStages], empty_bar[C::kStages], tfull_bar[2], tempty_bar[2];
  __shared__ __align__(8) uint64_t mma_done_bar, never_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], kEpiWarps);
    }
    mbar_init(&mma_done_bar, 1);
    mbar_init(&never_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int *abort_p = &abort_flag;

  if (warp == 0 && lane == 0) {
    // ---------------- TMA producer ----------------
    int j = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
      const Tile tl = tile_of(p, t, kCols);
      for (int kb = 0; kb < p.kb; ++kb, ++j) {
        const int s = j % C::kStages;
        if (!mbar_wait_bounded(&empty_bar[s], (uint32_t)((j / C::kStages) & 1) ^ 1u, abort_p, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        // the second pair of matrices follows the first along k (kInputGrad)
        const int src = MODE == kWeightGrad ? tl.prob : (MODE == kInputGrad && kb >= p.kb0 ? 1 : 0);
        const int k0 = (MODE == kInputGrad && kb >= p.kb0 ? kb - p.kb0 : kb) * kBK;
        uint64_t *fb = &full_bar[s];
        mbar_arrive_expect_tx(fb, C::kStage);
        uint8_t *a = ring + (size_t)s * C::kStage, *b = a + kABytes;
        if constexpr (C::kAMn) {
          tma_load_2d(a, &maps.a[src], fb, tl.m0, k0);
          tma_load_2d(a + kBK * 128, &maps.a[src], fb, tl.m0 + 64, k0);
        } else {
          tma_load_2d(a, &maps.a[src], fb, k0, tl.m0);
        }
        if constexpr (C::kBMn) {
#pragma unroll
          for (int i = 0; i < BN / 64; ++i) tma_load_2d(b + i * kBK * 128, &maps.b[src], fb, tl.n0 + 64 * i, k0);
        } else if constexpr (MODE == kGateUp) {
          tma_load_2d(b, &maps.b[0], fb, k0, tl.n0);
          tma_load_2d(b + (BN / 2) * 128, &maps.b[1], fb, k0, tl.n0);
        } else {
          tma_load_2d(b, &maps.b[0], fb, k0, tl.n0);
        }
      }
    }
    // copies still in flight after an abort land before the CTA may leave (bounded; in a normal run
    // each has landed long ago)
    int no_abort = 0;
    for (int s = 0; s < C::kStages; ++s) {
      const int n = j / C::kStages + (s < j % C::kStages ? 1 : 0);
      if (n > 0) (void)mbar_wait_bounded(&full_bar[s], (uint32_t)((n - 1) & 1), &no_abort, p.status, p.wait_ns);
    }
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMA issuer ----------------
    if (p.inject && blockIdx.x == 0)  // test hook: a wait that runs out
      (void)mbar_wait_bounded(&never_bar, 0u, abort_p, p.status, p.wait_ns);
    const uint32_t idesc = idesc_16(p.f16, C::kAMn, C::kBMn, BN);
    int j = 0, it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x, ++it) {
      const int acc = it & 1;
      if (!mbar_wait_bounded(&tempty_bar[acc], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_p, p.status, p.wait_ns)) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(acc * BN);
      for (int kb = 0; kb < p.kb; ++kb, ++j) {
        const int s = j % C::kStages;
        if (!mbar_wait_bounded(&full_bar[s], (uint32_t)((j / C::kStages) & 1), abort_p, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = smem_u32(ring + (size_t)s * C::kStage), b = a + kABytes;
#pragma unroll
        for (int k = 0; k < kBK / 16; ++k) {
          // 16 k are 32 bytes of a K-major row, or 16 rows of 128 bytes of an MN-major box
          const uint64_t da = C::kAMn ? smem_desc_mn(a + k * 2048) : smem_desc_sw128(a + k * 32);
          const uint64_t db = C::kBMn ? smem_desc_mn(b + k * 2048) : smem_desc_sw128(b + k * 32);
          tc_mma_f16(d, da, db, idesc, (kb | k) ? 1u : 0u);
        }
        tc_commit(&empty_bar[s]);
      }
      if (ok) tc_commit(&tfull_bar[acc]);
    }
    // every MMA this thread issued completes before TMEM is freed
    tc_commit(&mma_done_bar);
    int no_abort = 0;
    (void)mbar_wait_bounded(&mma_done_bar, 0u, &no_abort, p.status, p.wait_ns);
  } else if (warp >= 2) {
    // ---------------- epilogue ----------------
    const int q = warp & 3, half = (warp - 2) >> 2;
    int it = 0;
    for (int t = blockIdx.x; t < p.tiles; t += gridDim.x, ++it) {
      const int acc = it & 1;
      int ready = 0;
      if (lane == 0)
        ready = mbar_wait_bounded(&tfull_bar[acc], (uint32_t)(it >> 1) & 1u, abort_p, p.status, p.wait_ns) ? 1 : 0;
      if (!__shfl_sync(0xffffffffu, ready, 0)) break;
      tc_fence_after();
      const Tile tl = tile_of(p, t, kCols);
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      if (p.f16)
        epilogue<MODE, BN, __half>(p, tl, tbase, half, tl.m0 + q * 32 + lane);
      else
        epilogue<MODE, BN, __nv_bfloat16>(p, tl, tbase, half, tl.m0 + q * 32 + lane);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty_bar[acc]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

int cdiv(int a, int b) { return (a + b - 1) / b; }

template <int MODE, int BN>
cudaError_t launch(const GemmMaps &maps, const GemmParams &p, int num_sms, cudaStream_t st) {
  using C = Cfg<MODE, BN>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem((const void *)dense_gemm_kernel<MODE, BN>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  dense_gemm_kernel<MODE, BN><<<p.tiles < num_sms ? p.tiles : num_sms, kThreads, C::kSmem, st>>>(maps, p);
  return cudaGetLastError();
}

}  // namespace

// The widest tile whose waves over the SMs cost least; a wave costs its tile's columns plus the part
// of a k block that does not shrink with them.
int gemm_pick_bn(int mode, const GemmParams &p, int num_sms) {
  const bool b_mn = mode == kHiddenGrad || mode == kInputGrad || mode == kWeightGrad;
  int best = 0;
  long long least = 0;
  for (int bn = 256; bn >= (b_mn ? 64 : 32); bn /= 2) {
    const long long cols = mode == kGateUp ? bn / 2 : bn;
    long long tiles = (long long)cdiv(p.m, kBM) * ((p.n + cols - 1) / cols) * p.same;
    if (p.m_last) tiles += (long long)cdiv(p.m_last, kBM) * ((p.n_last + cols - 1) / cols);
    const long long cost = (tiles + num_sms - 1) / num_sms * (bn + 32);
    if (!best || cost < least) {
      best = bn;
      least = cost;
    }
  }
  return best;
}

cudaError_t launch_dense_gemm(int mode, int bn, const GemmMaps &maps, GemmParams p, int num_sms, cudaStream_t st) {
  const int cols = mode == kGateUp ? bn / 2 : bn;
  p.tiles_m = cdiv(p.m, kBM);
  p.tiles_n = cdiv(p.n, cols);
  p.tiles_m_last = cdiv(p.m_last, kBM);
  p.tiles_n_last = cdiv(p.n_last, cols);
  p.tiles = p.tiles_m * p.tiles_n * p.same + p.tiles_m_last * p.tiles_n_last;
#define MOE_LAUNCH(MODE, BN) \
  if (mode == MODE && bn == BN) return launch<MODE, BN>(maps, p, num_sms, st)
  MOE_LAUNCH(kGateUp, 256);
  MOE_LAUNCH(kGateUp, 128);
  MOE_LAUNCH(kGateUp, 64);
  MOE_LAUNCH(kGateUp, 32);
  MOE_LAUNCH(kDown, 256);
  MOE_LAUNCH(kDown, 128);
  MOE_LAUNCH(kDown, 64);
  MOE_LAUNCH(kDown, 32);
  MOE_LAUNCH(kHiddenGrad, 256);
  MOE_LAUNCH(kHiddenGrad, 128);
  MOE_LAUNCH(kHiddenGrad, 64);
  MOE_LAUNCH(kInputGrad, 256);
  MOE_LAUNCH(kInputGrad, 128);
  MOE_LAUNCH(kInputGrad, 64);
  MOE_LAUNCH(kWeightGrad, 256);
  MOE_LAUNCH(kWeightGrad, 128);
  MOE_LAUNCH(kWeightGrad, 64);
#undef MOE_LAUNCH
  return cudaErrorInvalidValue;
}

}  // namespace moe
