// The product of 4-bit weights and a few rows on the FP8 tensor cores (sm_103a): see few_tc.cuh.
//
// Where the matrix has more row tiles than the GPU has SMs, a CTA takes one row tile after another; otherwise the CTAs of a
// cluster share the columns of one, and their sums meet in shared memory in the order of their ranks.
// 16 tokens by 129280 x 4096 in groups of 128: 54 us, 5.1 TB/s (41 at the copy's rate); one token 46.
#include "few_tc.cuh"
#include "kernels.h"

namespace moe {
namespace {

// x as planes and groups' sums: a CTA takes a row.
template <typename T, int PLANES>
__global__ void __launch_bounds__(256) int4_planes_kernel(const __grid_constant__ Int4MatmulParams p, int tokens) {
  const int row = blockIdx.x, k8 = p.w.k / 8, block = row / tokens, token = row % tokens;
  const T *x = static_cast<const T *>(p.x) + row * p.ld_x;
  pdl_wait();
  // The product may come and fetch weights: not earlier, as what the wait was for may write them.
  pdl_trigger();
  const uint32_t most = row_max(x, k8);
  if (threadIdx.x == 0) p.back[row] = way_back(most);
  split_row<T, PLANES>(x, two_to(plane_exponent(most)), k8, p.sum_groups, 1 << (p.w.group_shift - 3),
                       p.planes + ((size_t)block * PLANES * tokens + token) * k8, (size_t)tokens * k8,
                       p.sums + (size_t)block * p.sum_groups * tokens + token, tokens);
}

template <typename T, int TOKENS, int PLANES, int GROUPS, bool ZP>
struct MatmulJob {
  using C = CodeCfg<TOKENS, PLANES, GROUPS>;
  const Int4MatmulParams &p;
  const Int4Maps &maps;
  float *sums;                    // the cluster's sums meet in it, [TOKENS][128]
  int splits, first, end, units, unit0, unit_step, block;
  struct Place {
    int unit, tile, units;
    __device__ __forceinline__ bool more() const { return unit < units; }
  };
  __device__ __forceinline__ void next(Place &a) const {
    if (++a.tile == end) {
      a.tile = first;
      a.unit += unit_step;
    }
  }
  __device__ __forceinline__ int count() const {
    return unit0 < units ? (end - first) * ((units - unit0 + unit_step - 1) / unit_step) : 0;
  }
  __device__ __forceinline__ Place begin() const { return Place{first < end ? unit0 : units, first, units}; }
  __device__ __forceinline__ void next_unit(Place &a) const { a.unit += unit_step; }
  __device__ __forceinline__ int unit_tiles() const { return end - first; }
  __device__ __forceinline__ bool skip(Place &a, int by) const { return (a.tile += by) < end; }
  __device__ __forceinline__ void weights(const Place &a, uint32_t at, uint32_t bar) const {
    tma_load_2d_one<false>(at, &maps.w, bar, a.tile * (64 * C::kHalves), a.unit * kCodeRows);
  }
  __device__ __forceinline__ void ready() const { pdl_wait(); }
  __device__ __forceinline__ void tokens(const Place &a, uint32_t at, uint32_t to, uint32_t bar) const {
#pragma unroll
    for (int h = 0; h < C::kHalves; ++h)
      tma_load_2d_one<false>(at + h * C::kB, &maps.x, bar, (a.tile * C::kHalves + h) * 128, block * C::kRows);
    tma_bulk_one(to, p.sums + ((size_t)block * p.sum_groups + a.tile * C::kAll) * TOKENS, C::kSums, bar);
  }
  struct Row {
    const uint16_t *scales;
    const uint8_t *zeros;
    int row;
  };
  __device__ __forceinline__ void row_at(Row &r, const Place &a, int row) const {
    r.row = row;
    find(r, a.unit);
    fetch(r, a.unit);
  }
  __device__ __forceinline__ void next_row(Row &r, const Place &a) const {
    find(r, a.unit + unit_step);
    fetch(r, a.unit + unit_step);
  }
  __device__ __forceinline__ void find(Row &r, int unit) const {
    const long long at = (long long)min(unit * kCodeRows + r.row, p.w.n - 1) * p.w.groups;
    r.scales = p.w.scales + at;
    r.zeros = p.w.zeros + at;
  }
  __device__ __forceinline__ void fetch(const Row &r, int unit) const {  // those of the unit after it
    if (unit + unit_step >= units) return;
    const int by = min((unit + unit_step) * kCodeRows + r.row, p.w.n - 1) - (unit * kCodeRows + r.row);
    fetch_lines(r.scales + (long long)by * p.w.groups, 2 * p.w.groups);
    if (ZP) fetch_lines(r.zeros + (long long)by * p.w.groups, p.w.groups);
  }
  struct Scales {
    uint16_t scales[C::kAll];
    uint8_t zeros[C::kAll];
    __device__ __forceinline__ float scale(int g) const { return to_f32(reinterpret_cast<const T *>(scales)[g]); }
    __device__ __forceinline__ float zero(int g) const { return ZP ? (float)(zeros[g] & 15u) : 8.f; }
  };
  __device__ __forceinline__ int last(const Place &) const { return end; }
  __device__ __forceinline__ void scales(const Row &r, const Place &a, int ahead, Scales &s) const {
#pragma unroll
    for (int g = 0; g < C::kAll; ++g) {
      const int at = min((a.tile + ahead) * C::kAll + g, p.w.groups - 1);
      s.scales[g] = r.scales[at];
      if (ZP) s.zeros[g] = r.zeros[at];
    }
  }
  __device__ __forceinline__ void finish(const Place &a, int row, int, int, int t0, const float (&acc)[C::kMine]) const {
    const int n = a.unit * kCodeRows + row, rows = min(TOKENS, p.rows - block * TOKENS);
#pragma unroll
    for (int t = 0; t < C::kMine; ++t) {
      if (t0 + t >= rows) break;
      if (splits > 1) sums[(t0 + t) * kCodeRows + row] = acc[t];
      else if (n < p.w.n) store(n, t0 + t, acc[t]);
    }
  }
  __device__ __forceinline__ void store(int n, int t, float v) const {
    const int token = block * TOKENS + t;
    static_cast<T *>(p.out)[token * p.ld_out + n] = from_f32<T>(v * 512.f * p.back[token]);
  }
};

template <typename T, int TOKENS, int PLANES, int GROUPS, bool ZP>
__global__ void __launch_bounds__(CodeCfg<TOKENS, PLANES, GROUPS>::kThreads, 1)
    int4_tc_kernel(const __grid_constant__ Int4MatmulParams p, const __grid_constant__ Int4Maps maps, int splits) {
  using C = CodeCfg<TOKENS, PLANES, GROUPS>;
  extern __shared__ char smem[];
  __shared__ __align__(8) CodeBars<C> bars;
  __shared__ float sums[TOKENS * kCodeRows];
  char *ring = smem + (-smem_u32(smem) & 1023u);
  code_setup<C>(bars);
  const int tiles = (p.w.k + 128 * C::kHalves - 1) / (128 * C::kHalves), rank = blockIdx.x % splits;
  MatmulJob<T, TOKENS, PLANES, GROUPS, ZP> job{p, maps, sums, splits, (int)((long long)tiles * rank / splits),
                                               (int)((long long)tiles * (rank + 1) / splits),
                                               (p.w.n + kCodeRows - 1) / kCodeRows, (int)blockIdx.x / splits, (int)gridDim.x / splits,
                                               (int)blockIdx.y};
  if (splits > 1 && job.first == job.end)
    for (int i = threadIdx.x; i < TOKENS * kCodeRows; i += C::kThreads) sums[i] = 0.f;
  code_pipeline<C, TOKENS, PLANES, GROUPS>(job, ring, bars, p.waits);
  if (splits > 1) {  // one row tile, whose sums meet: a part of the rows by each CTA
    cluster_sync();
    const int part = kCodeRows / splits, row0 = rank * part, rows = min(TOKENS, p.rows - job.block * TOKENS);
    for (int i = threadIdx.x; i < part * rows; i += C::kThreads) {
      const int row = row0 + i % part, t = i / part, n = job.unit0 * kCodeRows + row;
      float v = 0.f, x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)  // all loads before the first sum
        if (r < splits)
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[r]) : "r"(in_cta(&sums[t * kCodeRows + row], r)) : "memory");
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < splits) v += x[r];
      if (n < p.w.n) job.store(n, t, v);
    }
    cluster_sync();
  }
  code_end(bars);
}

template <typename T, int TOKENS, int GROUPS, bool ZP>
cudaError_t tc_launch(const Int4MatmulParams &p, const Int4Maps &maps, int num_sms, cudaStream_t st) {
  constexpr int PLANES = std::is_same<T, __half>::value ? 3 : 2;
  using C = CodeCfg<TOKENS, PLANES, GROUPS>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = launch_pdl(int4_planes_kernel<T, PLANES>, dim3(p.rows), dim3(256), 0, st, p, TOKENS);
  if (e != cudaSuccess) return e;
  const int tiles = (p.w.n + kCodeRows - 1) / kCodeRows, blocks = (p.rows + TOKENS - 1) / TOKENS;
  const int splits = code_splits((long long)tiles * blocks, num_sms);
  const int busy = splits > 1 || tiles < num_sms ? tiles : num_sms;
  return launch_code_clusters(int4_tc_kernel<T, TOKENS, PLANES, GROUPS, ZP>, C::kRing + 1024, done, dim3(busy * splits, blocks), C::kThreads, splits, st, p,
                              maps, splits);
}

template <typename T, int GROUPS, bool ZP>
cudaError_t tc_rows(const Int4MatmulParams &p, const Int4Maps &maps, int tokens, int num_sms, cudaStream_t st) {
  if constexpr (GROUPS < 4) {  // (see int4_tc_tokens)
    if (tokens == 8) return tc_launch<T, 8, GROUPS, ZP>(p, maps, num_sms, st);
    if (tokens == 16) return tc_launch<T, 16, GROUPS, ZP>(p, maps, num_sms, st);
  }
  return tc_launch<T, 32, GROUPS, ZP>(p, maps, num_sms, st);
}

template <typename T>
cudaError_t tc_typed(const Int4MatmulParams &p, const Int4Maps &maps, int tokens, int num_sms, cudaStream_t st) {
  if (p.w.group_shift == 5) return p.w.zeros ? tc_rows<T, 4, true>(p, maps, tokens, num_sms, st) : tc_rows<T, 4, false>(p, maps, tokens, num_sms, st);
  if (p.w.group_shift == 6) return p.w.zeros ? tc_rows<T, 2, true>(p, maps, tokens, num_sms, st) : tc_rows<T, 2, false>(p, maps, tokens, num_sms, st);
  return p.w.zeros ? tc_rows<T, 1, true>(p, maps, tokens, num_sms, st) : tc_rows<T, 1, false>(p, maps, tokens, num_sms, st);
}

}  // namespace

// Which form serves a call, measured on weights that come from memory (bf16, us, planes and mma.sync; n of 512 to 65536, k of
// 512 to 16384):
//   Up to 16 tokens splitting x takes a launch (4096 x 4096 in groups of 128: 7.9 and 6.0 for a token, 8.9 and 7.7 for 16),
//   which large matrices have time for (8192 x 8192: 12.8 and 18.5, 15.3 and 17.8; 65536 x 4096: 28 and 39, 34 and 50; about
//   even at 2^25: 8192 x 4096 9.9 and 10.9, 11.0 and 10.0, 16384 x 2048 8.4 and 8.1, 9.6 and 9.0), in groups of 64 larger ones
//   (8192 x 4096: 10.9 and 11.1, 11.8 and 10.6; 8192 x 8192: 15.0 and 18.6, 16.3 and 18.7), and so have long rows of more than
//   eight tokens (512 x 8192, 16 tokens: 8.8 and 13.2; with one 7.7 and 8.2).  In groups of 32 the joining of eight groups
//   takes what the conversion saves (65536 x 4096: 55 and 49, 69 and 59; 8192 x 8192: 18.8 and 20.2, 23 and 20).
//   Beyond 16 tokens mma.sync's registers leave it behind (32 tokens by 4096 x 4096: 10.0 and 15.8; 65536 x 4096: 42 and 72),
//   but for groups of 32 of many rows (8192 x 4096: 19.7 and 28; 16384 x 4096: 29.3 and 28.3; 65536 x 4096: 100 and 89; 64
//   tokens, twice 32 here, by 2048 x 4096: 13.1 and 17.5, by 4096 x 4096: 19.2 and 17.6).
// Where it is not the faster one: beyond 16 tokens at k below about 1024 in groups of 128 and 64, 2048 in groups of 32
// (4096 x 512: 7.0 and 4.0, 4096 x 1024: 7.1 and 5.8), up to 16 tokens at k of 16384 and few rows (512 x 16384, a token: 10.7
// and 14.3; 16 in groups of 32 15.4 and 25.9), and in f16 of 16 tokens in groups of 64 (65536 x 1024: 20.9 and 17.2).
int int4_tc_tokens(int rows, int n, int k, int group) {
  const long long blocks = (rows + 31) / 32;
  if (group == 32) return rows > 16 && n * blocks * blocks <= 12000 ? 32 : 0;
  if (rows > 16) return 32;
  const bool large = (long long)n * k >= (group == 128 ? 1 << 25 : 1 << 26), deep = rows > 8 && k >= 8192;
  return large || deep ? (rows <= 8 ? 8 : 16) : 0;
}

cudaError_t launch_int4_tc(const Int4MatmulParams &p, const Int4Maps &maps, int tokens, bool f16, int num_sms, cudaStream_t st) {
  return f16 ? tc_typed<__half>(p, maps, tokens, num_sms, st) : tc_typed<__nv_bfloat16>(p, maps, tokens, num_sms, st);
}

}  // namespace moe
