// Matrix product in 8-bit floating point with a scale for each block of 128, and the quantiser that makes
// its operands (sm_103a).
//
//   out[m, n] = sum_b a_scale[m, b] b_scale[n / 128, b] sum_{k in block b} a[m, k] b[n, k]
//
// The codes' products accumulate over one block of 128 k in f32 in TMEM (four tcgen05.mma kind::f8f6f4
// of 32 k each); the epilogue warps then take the block's sums, multiply them by the block's two scales
// and add them to f32 sums in registers.  So scales may be any f32 values, and no more than 128 products
// are added before a scale is applied.  Several TMEM buffers let the MMAs of the next blocks run
// meanwhile.
//
// A CTA (one per SM, persistent over tiles of 128 x BN, BN dividing 128 so that a tile has one b_scale):
//   warp 0     TMA producer: a ring of blocks (A 128 rows, B BN rows, 128 bytes of k each)
//   warp 1     TMEM allocator and MMA issuer
//   warps 2-9  scaled accumulation and the output: two warps for each TMEM lane quarter, half the
//              columns each
// Rows and k past an operand's end read as zeros; outputs past the end are not stored.
#include <cuda_fp8.h>

#include "common.cuh"
#include "dense.h"
#include "dense_tc.cuh"
#include "dense_vec.cuh"

namespace moe {
namespace {

template <int BN>
struct Fp8Cfg {
  static constexpr int kABytes = kBM * kScaleBlock;
  static constexpr int kStage = kABytes + BN * kScaleBlock;
  static constexpr int kStages = kRingBytes / kStage;
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
  static constexpr int kAcc = 4;  // TMEM buffers, one block's sums each
  static constexpr int kTmemCols = kAcc * BN < 32 ? 32 : kAcc * BN;
  static constexpr int kPer = BN / 2;  // columns of one epilogue warp
};

__device__ __forceinline__ uint32_t idesc_f8(bool a_e5m2, bool b_e5m2, int N) {
  return 1u << 4 | (a_e5m2 ? 1u : 0u) << 7 | (b_e5m2 ? 1u : 0u) << 10 | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(kBM >> 4) << 24;
}

template <typename T, int N>
__device__ __forceinline__ void store_row(T *dst, int left, bool wide, const float (&v)[N]) {
  constexpr int per = 16 / (int)sizeof(T);
  if (wide && left >= N) {
#pragma unroll
    for (int i = 0; i < N; i += per) {
      uint4 w;
      if constexpr (sizeof(T) == 4)
        w = make_uint4(__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]),
                       __float_as_uint(v[i + 3]));
      else
        w = make_uint4(pack2<T>(v[i], v[i + 1]), pack2<T>(v[i + 2], v[i + 3]), pack2<T>(v[i + 4], v[i + 5]),
                       pack2<T>(v[i + 6], v[i + 7]));
      *reinterpret_cast<uint4 *>(dst + i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < left) dst[i] = from_f32<T>(v[i]);
  }
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_matmul_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                      const __grid_constant__ Fp8Params p) {
  using C = Fp8Cfg<BN>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[C::kStages], empty_bar[C::kStages], tfull_bar[C::kAcc], tempty_bar[C::kAcc];
  __shared__ __align__(8) uint64_t mma_done_bar, never_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < C::kAcc; ++b) {
      mbar_init(&tfull_bar[b], 1);
      mbar_init(&tempty_bar[b], kEpiWarps);
    }
    mbar_init(&mma_done_bar, 1);
    mbar_init(&never_bar, 1);
    abort_flag = 0;
    issued = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int *abort_p = &abort_flag;

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    RingPos<C::kStages> pos;
    int j = 0;
    bool ok = true;
    const uint32_t ring0 = smem_u32(ring), full0 = smem_u32(full_bar);
    for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
      int m, n;
      band_tile(t, p.tiles_m, p.tiles_n, m, n);
      for (int kb = 0; kb < p.kb; ++kb, ++j, pos.next()) {
        const int s = pos.slot;
        if (!warp_wait(&empty_bar[s], pos.round ^ 1u, abort_p, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        const uint32_t a = ring0 + s * C::kStage, fb = full0 + 8 * s;
        mbar_expect_one(fb, C::kStage);
        tma_load_2d_one<false>(a, &tm_a, fb, kb * kScaleBlock, m * kBM);
        tma_load_2d_one<false>(a + C::kABytes, &tm_b, fb, kb * kScaleBlock, n * BN);
      }
    }
    if (lane == 0) issued = j;
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (p.inject && blockIdx.x == 0)  // test hook: a wait that runs out
      (void)warp_wait(&never_bar, 0u, abort_p, p.status, p.wait_ns);
    const uint32_t idesc = idesc_f8(p.a_e5m2, p.b_e5m2, BN);
    const uint64_t a0 = smem_desc_sw128(0) + (uint64_t)(smem_u32(ring) >> 4), b0 = a0 + (C::kABytes >> 4);
    RingPos<C::kStages> pos;
    RingPos<C::kAcc> acc;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
      for (int kb = 0; kb < p.kb; ++kb, pos.next(), acc.next()) {
        if (!warp_wait(&tempty_bar[acc.slot], acc.round ^ 1u, abort_p, p.status, p.wait_ns) ||
            !warp_wait(&full_bar[pos.slot], pos.round, abort_p, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = pos.slot * (C::kStage >> 4), d = tmem + (uint32_t)(acc.slot * BN);
#pragma unroll
        for (int k = 0; k < kScaleBlock / 32; ++k)
          tc_mma_one<false, true>(d, a0 + (at + k * 2), b0 + (at + k * 2), idesc, k ? 1u : 0u);
        tc_commit_one<false>(smem_u32(&empty_bar[pos.slot]));
        tc_commit_one<false>(smem_u32(&tfull_bar[acc.slot]));
      }
    }
    // every MMA this warp issued completes before TMEM is freed
    tc_commit_one<false>(smem_u32(&mma_done_bar));
    int no_abort = 0;
    (void)wait_bounded(&mma_done_bar, 0u, &no_abort, p.status, p.wait_ns);
  } else if (warp >= 2) {
    // ---------------- scaled accumulation and output ----------------
    const int q = warp & 3, half = (warp - 2) >> 2;
    int j = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < p.tiles; t += gridDim.x) {
      int m, n;
      band_tile(t, p.tiles_m, p.tiles_n, m, n);
      const int row = m * kBM + q * 32 + lane;
      const float *sa = p.a_scale + (size_t)row * p.kb;
      const float *sb = p.b_scale + (size_t)(n * BN / kScaleBlock) * p.kb;
      const bool in = row < p.m;
      float sum[C::kPer];
#pragma unroll
      for (int i = 0; i < C::kPer; ++i) sum[i] = 0.f;
      for (int kb = 0; kb < p.kb; ++kb, ++j) {
        const int acc = j % C::kAcc;
        const float scale = in ? sa[kb] * sb[kb] : 0.f;
        int ready = 0;
        if (lane == 0)
          ready = wait_bounded(&tfull_bar[acc], (uint32_t)((j / C::kAcc) & 1), abort_p, p.status, p.wait_ns) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, ready, 0)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN + half * C::kPer);
#pragma unroll
        for (int c = 0; c < C::kPer; c += 16) {
          float v[16];
          tmem_ld16(tb + c, v);
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[c + i] = fmaf(scale, v[i], sum[c + i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty_bar[acc]);
      }
      if (!ok) break;
      const int col = n * BN + half * C::kPer, left = p.n - col;
      if (in && left > 0) {
        const size_t at = (size_t)row * p.ld_out + col;
        if (p.out_type == kF32) store_row(static_cast<float *>(p.out) + at, left, p.wide, sum);
        else if (p.out_type == kBF16) store_row(static_cast<__nv_bfloat16 *>(p.out) + at, left, p.wide, sum);
        else store_row(static_cast<__half *>(p.out) + at, left, p.wide, sum);
      }
      __syncwarp();
    }
  }
  // copies still in flight after an abort land before the CTA may leave (bounded; in a normal run each
  // has landed long ago)
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    int no_abort = 0;
    for (int s = 0; s < C::kStages; ++s) {
      const int n = issued / C::kStages + (s < issued % C::kStages ? 1 : 0);
      if (n > 0) (void)wait_bounded(&full_bar[s], (uint32_t)((n - 1) & 1), &no_abort, p.status, p.wait_ns);
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int BN>
cudaError_t launch(const CUtensorMap &a, const CUtensorMap &b, const Fp8Params &p, int num_sms, cudaStream_t st) {
  using C = Fp8Cfg<BN>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem((const void *)fp8_matmul_kernel<BN>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  fp8_matmul_kernel<BN><<<p.tiles < num_sms ? p.tiles : num_sms, kThreads, C::kSmem, st>>>(a, b, p);
  return cudaGetLastError();
}

// ---- quantiser ----
// A block's scale is its largest magnitude over the largest code (448 or 57344); 1 for a block of
// zeros, at least 2^-126 so that it is a normal number, and with pow2 rounded up to a power of two.  A
// code is x / scale rounded to nearest even.  The magnitudes are compared as integers, so that a NaN
// counts as the largest and makes the scale NaN.

__device__ __forceinline__ float block_scale(uint32_t amax, bool e5m2, bool pow2) {
  if (amax == 0u) return 1.f;
  float s = __fdiv_rn(__uint_as_float(amax), e5m2 ? 57344.f : 448.f);
  if (s < 1.17549435e-38f) s = 1.17549435e-38f;
  const uint32_t u = __float_as_uint(s);
  if (pow2 && (u & 0x7FFFFFu) && u < 0x7F800000u) s = __uint_as_float((u & 0x7F800000u) + 0x800000u);
  return s;
}

__device__ __forceinline__ uint32_t codes4(const float *v, float s, bool e5m2) {
  const __nv_fp8_interpretation_t f = e5m2 ? __NV_E5M2 : __NV_E4M3;
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[0], s), __fdiv_rn(v[1], s)), __NV_SATFINITE, f);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(v[2], s), __fdiv_rn(v[3], s)), __NV_SATFINITE, f);
  return lo | hi << 16;
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
__device__ __forceinline__ void store_part(const QuantiseParams &p, int row, int col, float s, const float (&v)[8]) {
  if (row >= p.rows || col >= p.k) return;
  uint8_t *dst = p.codes + (size_t)row * p.ld_codes + col;
  const uint32_t a = codes4(v, s, p.e5m2), b = codes4(v + 4, s, p.e5m2);
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

template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) quantise_rows_kernel(const __grid_constant__ QuantiseParams p) {
  const int blocks = (p.k + kScaleBlock - 1) / kScaleBlock;
  const long long total = (long long)p.rows * blocks, step = (long long)gridDim.x * 16;
  const int part = threadIdx.x & 15;
  // whole warps stay in the loop for the shuffles: a half warp past the end works on nothing
  for (long long base = (long long)blockIdx.x * 16 + (threadIdx.x >> 5) * 2; base < total; base += step) {
    const long long i = base + ((threadIdx.x >> 4) & 1);
    const bool in = i < total;
    const int row = in ? (int)(i / blocks) : p.rows, b = in ? (int)(i % blocks) : 0, col = b * kScaleBlock + part * 8;
    float v[8];
    load_part<T, WIDE>(p, row, col, v);
    uint32_t m = largest(v);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float s = block_scale(m, p.e5m2, p.pow2);
    store_part<WIDE>(p, row, col, s, v);
    if (in && part == 0) p.scales[i] = s;
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
#pragma unroll
  for (int i = 0; i < 8; ++i) store_part<WIDE>(p, row + 16 * i, col, s, v[i]);
  if (threadIdx.x == 0) p.scales[blockIdx.x] = s;
}

template <typename T>
cudaError_t quantise_typed(const QuantiseParams &p, int num_sms, cudaStream_t st) {
  const long long blocks = (p.k + kScaleBlock - 1) / kScaleBlock;
  if (p.tall == 1) {
    const long long ctas = (p.rows * blocks + 15) / 16, most = (long long)num_sms * 8 * 4;
    const int grid = (int)(ctas < most ? ctas : most);
    if (p.wide) quantise_rows_kernel<T, true><<<grid, 256, 0, st>>>(p);
    else quantise_rows_kernel<T, false><<<grid, 256, 0, st>>>(p);
  } else {
    const int grid = (int)((p.rows + kScaleBlock - 1) / kScaleBlock * blocks);
    if (p.wide) quantise_tiles_kernel<T, true><<<grid, 256, 0, st>>>(p);
    else quantise_tiles_kernel<T, false><<<grid, 256, 0, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

// The widest tile whose waves over the SMs cost least (see gemm_pick_bn).
int fp8_pick_bn(const Fp8Params &p, int num_sms) {
  int best = 0;
  long long least = 0;
  for (int bn = 128; bn >= 32; bn /= 2) {
    const long long tiles = (long long)((p.m + kBM - 1) / kBM) * ((p.n + bn - 1) / bn);
    const long long cost = (tiles + num_sms - 1) / num_sms * (bn + 32);
    if (!best || cost < least) {
      best = bn;
      least = cost;
    }
  }
  return best;
}

cudaError_t launch_fp8_matmul(int bn, const CUtensorMap &a, const CUtensorMap &b, Fp8Params p, int num_sms,
                              cudaStream_t st) {
  p.tiles_m = (p.m + kBM - 1) / kBM;
  p.tiles_n = (p.n + bn - 1) / bn;
  p.tiles = p.tiles_m * p.tiles_n;
  if (bn == 128) return launch<128>(a, b, p, num_sms, st);
  if (bn == 64) return launch<64>(a, b, p, num_sms, st);
  if (bn == 32) return launch<32>(a, b, p, num_sms, st);
  return cudaErrorInvalidValue;
}

cudaError_t launch_fp8_quantise(const QuantiseParams &p, int num_sms, cudaStream_t st) {
  if (p.type == kF32) return quantise_typed<float>(p, num_sms, st);
  if (p.type == kBF16) return quantise_typed<__nv_bfloat16>(p, num_sms, st);
  return quantise_typed<__half>(p, num_sms, st);
}

}  // namespace moe
