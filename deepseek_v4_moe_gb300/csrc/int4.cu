// Products with 4-bit weights for a few rows, and the kernels that make and widen such weights (sm_103a).
//
//   w[j, k] = (code[j, k] - zero[j, k / group]) scale[j, k / group];   out = x w^T
//
// Code minus zero is a small whole number, exact in 16 bits, so the tensor cores' products with x are exact and their sums
// in f32; a group's sum is multiplied by its scale in f32 once.  (Weights multiplied by their scales before the product
// would be rounded to 16 bits each.)
// Bound by the codes' way from memory and their conversion, 11 instructions for 8 codes.  One token by 4096 x 4096 in groups
// of 128: 6.0 us (1.3 at the copy's rate), in one wave of 256 CTAs, half of it a launch and a ring's first fill.
#include "dense_quant.cuh"
#include "few.cuh"
#include "kernels.h"

namespace moe {
namespace {

// ---- product ----

// A unit: 128 M / kw rows of the result.  The CTA's 8 warps are kw shares of k for each of 8 / kw sets of 16 M rows; a
// step of the ring holds a tile of every set and share, and the tokens' columns of every share, so that what comes from
// the L2 of x serves all sets.  The warp that is last to finish a step lets the copies of a later one into its place.
// The shares' sums meet in shared memory in their order.

constexpr int kInt4Stages = 8;             // at most
constexpr size_t kInt4Smem = 112 * 1024;  // two CTAs on an SM
struct Int4Plan {
  int log_kw, stages, box_rows;  // box_rows: tokens of a copy
  int steps, units;
  int x_bytes, stage_bytes;
};

template <typename T, int PIECES, bool ZP, int M, int NT>
__global__ void __launch_bounds__(32 * kFewWarps, 2)
    int4_matmul_kernel(const __grid_constant__ Int4MatmulParams p, const __grid_constant__ Int4Maps maps,
                       const __grid_constant__ Int4Plan plan) {
  extern __shared__ char smem[];
  __shared__ uint64_t full[kInt4Stages], never;
  __shared__ unsigned left[kInt4Stages], fills[kInt4Stages];
  __shared__ int abort_flag;
  constexpr int kWeights = kFewWarps * M * kBoxBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kw = 1 << plan.log_kw, sets = kFewWarps >> plan.log_kw, set = warp >> plan.log_kw, share = warp & (kw - 1);
  const int row_first = blockIdx.y * 8 * NT, rows = min(8 * NT, p.rows - row_first), set_rows = 16 * M;
  char *ring = smem + (-smem_u32(smem) & 1023u);
  float *parts = reinterpret_cast<float *>(ring + plan.stages * plan.stage_bytes);
  if (threadIdx.x < kInt4Stages) {
    mbar_init(&full[threadIdx.x], 1);
    left[threadIdx.x] = fills[threadIdx.x] = 0u;
    if (threadIdx.x == 0) {
      mbar_init(&never, 1);
      abort_flag = 0;
    }
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  // a step's copies, by one thread
  auto fill = [&](int stage, int unit, int step) {
    char *place = ring + stage * plan.stage_bytes;
    mbar_arrive_expect_tx(&full[stage], kWeights + plan.x_bytes);
    for (int j = 0; j < kw; ++j)
      for (int r = 0; r < sets * set_rows; r += 256)  // (a copy's most rows)
        tma_load_2d(place + (j * sets * set_rows + r) * 64, &maps.w, &full[stage], (step * kw + j) * 64, unit * sets * set_rows + r);
    tma_load_3d(place + kWeights, &maps.x, &full[stage], 0, row_first, step * kw * 4);
    fills[stage] += 1;
  };
  auto onwards = [&](int &unit, int &step, int by) {
    for (step += by; step >= plan.steps; step -= plan.steps) unit += gridDim.x;
  };
  if (threadIdx.x == 0) {
    int unit = blockIdx.x, step = 0;
    for (int s = 0; s < plan.stages && unit < plan.units; ++s, onwards(unit, step, 1)) fill(s, unit, step);
  }
  if (p.waits.inject && blockIdx.x == 0) wait_bounded(&never, 0, &abort_flag, p.waits.status, p.waits.ns);  // test hook
  Tile<T, PIECES, ZP, M, NT, (NT > 1)> t;
  t.x.set(share * 4 * plan.box_rows, plan.box_rows);
  const uint32_t w_at = smem_u32(ring) + (share * sets + set) * M * kBoxBytes, x_at = smem_u32(ring) + kWeights;
  int stage = 0, phase = 0;
  for (int unit = blockIdx.x; unit < plan.units; unit += gridDim.x) {
    const int row0 = (unit * sets + set) * set_rows;
#pragma unroll
    for (int s = 0; s < M; ++s) t.meta.row[s].at(p.w, min(row0 + 16 * s, p.w.n - 1), p.w.n - row0 - 16 * s);
    t.meta.begin(share, kw, p.w.groups);
    float acc[M][NT][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
    for (int step = 0; step < plan.steps; ++step) {
      t.meta.advance(step * kw + share);
      // (the lanes agree: one that gave up takes the warp with it)
      if (!__all_sync(0xffffffffu, wait_bounded(&full[stage], phase, &abort_flag, p.waits.status, p.waits.ns))) break;
      t.multiply(w_at + stage * plan.stage_bytes, x_at + stage * plan.stage_bytes, acc);
      __syncwarp();
      if (lane == 0) {
        unsigned before;
        asm volatile("atom.acq_rel.cta.shared::cta.inc.u32 %0, [%1], %2;"
                     : "=r"(before)
                     : "r"(smem_u32(&left[stage])), "r"(kFewWarps - 1u)
                     : "memory");
        if (before == kFewWarps - 1) {
          int u = unit, s = step;
          onwards(u, s, plan.stages);
          if (u < plan.units) fill(stage, u, s);
        }
      }
      if (++stage == plan.stages) {
        stage = 0;
        phase ^= 1;
      }
    }
    float *sums = parts + set * kw * (NT * kPartFloats);
#pragma unroll
    for (int m = 0; m < M; ++m) {
#pragma unroll
      for (int i = 0; i < NT; ++i) put_part(sums + (share * NT + i) * kPartFloats, acc[m][i]);
      warps_meet(set * kw, kw);
      const int r0 = row0 + 16 * m;
      for (int i = threadIdx.x & (32 * kw - 1); i < 16 * rows; i += 32 * kw) {
        const int row = i & 15, token = i >> 4;
        if (r0 + row >= p.w.n) continue;
        const float *at = sums + (token >> 3) * kPartFloats + part_at(row, token & 7);
        float v = at[0];
        for (int w = 1; w < kw; ++w) v += at[w * (NT * kPartFloats)];
        static_cast<T *>(p.out)[(row_first + token) * p.ld_out + r0 + row] = from_f32<T>(v);
      }
      warps_meet(set * kw, kw);
    }
  }
  // after a wait that ran out: no copy may land in memory that the CTA has left
  __syncthreads();
  if (abort_flag && threadIdx.x == 0)
    for (int s = 0, nobody = 0; s < plan.stages; ++s)
      if (fills[s]) mbar_wait_bounded(&full[s], (fills[s] - 1) & 1, &nobody, p.waits.status, p.waits.ns);
}

template <typename T, int PIECES, bool ZP, int M, int NT>
cudaError_t int4_launch(const Int4MatmulParams &p, const Int4Maps &maps, const Int4Plan &plan, int y, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = allow_smem((const void *)int4_matmul_kernel<T, PIECES, ZP, M, NT>, kInt4Smem, done);
  if (e != cudaSuccess) return e;
  const size_t smem = plan.stages * (size_t)plan.stage_bytes + kFewWarps * NT * kPartFloats * sizeof(float) + 1024;
  const int most = 2 * num_sms / y > 1 ? 2 * num_sms / y : 1;
  return launch_pdl(int4_matmul_kernel<T, PIECES, ZP, M, NT>, dim3(plan.units < most ? plan.units : most, y), dim3(32 * kFewWarps), smem,
                    st, p, maps, plan);
}

template <typename T, int PIECES, bool ZP>
cudaError_t int4_tiles(const Int4MatmulParams &p, const Int4Maps &maps, const Int4Tiles &t, int num_sms, cudaStream_t st) {
  Int4Plan plan;
  const int tiles = (p.w.k + kTileK - 1) / kTileK, set_rows = 16 * t.strips, sets = kFewWarps >> t.log_kw;
  plan.log_kw = t.log_kw;
  plan.box_rows = t.box_rows;
  plan.steps = (tiles + (1 << t.log_kw) - 1) >> t.log_kw;
  plan.units = (p.w.n + sets * set_rows - 1) / (sets * set_rows);
  plan.x_bytes = (4 << t.log_kw) * t.box_rows * 64;
  plan.stage_bytes = (kFewWarps * t.strips * kBoxBytes + plan.x_bytes + 1023) / 1024 * 1024;
  const int room = (int)kInt4Smem - 1024 - kFewWarps * t.eights * kPartFloats * 4;
  plan.stages = room / plan.stage_bytes < kInt4Stages ? room / plan.stage_bytes : kInt4Stages;
  const int y = (p.rows + 8 * t.eights - 1) / (8 * t.eights);
#define MOE_INT4(M, NT) \
  if (t.strips == M && t.eights == NT) return int4_launch<T, PIECES, ZP, M, NT>(p, maps, plan, y, num_sms, st)
  MOE_INT4(1, 1);
  MOE_INT4(4, 1);
  MOE_INT4(1, 2);
  MOE_INT4(2, 2);
  if constexpr (PIECES == 1) {  // (more than 16 tokens come here in groups of 32 only: int4_tc_tokens)
    MOE_INT4(1, 4);
    MOE_INT4(2, 4);
  }
#undef MOE_INT4
  return cudaErrorInvalidValue;
}

// ---- making and widening weights ----
//
// Symmetric: scale = max|w| / 7, code = 8 + w / scale in 1..15.  With zero points: scale = (max(w, 0) - min(w, 0)) / 15,
// zero = -min(w, 0) / scale, code = zero + w / scale in 0..15.  Quotients are rounded to nearest even; scales are rounded
// to their type first, and are 1 for zeros and at least its smallest normal value.  Eight values a lane, a group's in
// 4, 8 or 16 lanes.

// A warp's chunks of CHUNK columns of a row: row and chunk, from its number on.
template <int CHUNK>
struct RowChunks {
  long long row;
  int at, per_row, rows_on, at_on;
  __device__ __forceinline__ RowChunks(int k) {
    const int warps = blockDim.x >> 5;
    const long long first = (long long)blockIdx.x * warps + (threadIdx.x >> 5);
    const long long step = (long long)gridDim.x * warps;
    per_row = (k + CHUNK - 1) / CHUNK;
    row = first / per_row;
    at = (int)(first - row * per_row);
    rows_on = (int)(step / per_row);
    at_on = (int)(step % per_row);
  }
  __device__ __forceinline__ int column() const { return at * CHUNK; }
  __device__ __forceinline__ void next() {
    row += rows_on;
    at += at_on;
    if (at >= per_row) {
      at -= per_row;
      ++row;
    }
  }
};

// The quotients are those of dense_quant.cuh, without a division for each value (all of them divided, with a 64-bit
// division for a lane's place besides: 4096 x 2048 made and widened 22.9 us, now 14.1; each by itself, from memory, 8.9 and
// 6.1, for 3.1); a warp has its next columns' loads in flight (two ahead changed nothing).  Bound by its instructions, some
// 150 for eight values.
template <typename T, typename TS, int PER, bool ZP>  // PER: lanes of a group
__global__ void __launch_bounds__(256, 4) int4_quantise_kernel(const __grid_constant__ Int4WeightParams p) {
  constexpr float kLeast = std::is_same<TS, __half>::value ? 6.103515625e-05f : 1.17549435e-38f;
  constexpr float kInteger = 12582912.f;  // 1.5 2^23: a sum with it has the whole number nearest in its low bits
  const int lane = threadIdx.x & 31, groups = (p.k + 8 * PER - 1) / (8 * PER);
  RowChunks<256> c(p.k);
  Eight<T, true> ahead;
  auto load = [&] {
    const int col = c.column() + 8 * lane;
    ahead.load(static_cast<const T *>(p.w) + c.row * p.ld_w + col, 0, 1, c.row < p.n && col < p.k ? 8 : 0);
  };
  pdl_wait();
  load();
  while (c.row < p.n) {
    float v[8];
    ahead.get(v);
    const int col = c.column() + 8 * lane;
    const long long row = c.row;
    c.next();
    load();
    float lo = 0.f, hi = 0.f, bad = 0.f;  // bad: not 0 where a value is no number, which minima and maxima pass over
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (ZP) lo = fminf(lo, v[e]);
      hi = fmaxf(hi, ZP ? v[e] : fabsf(v[e]));
      bad = fmaf(v[e], 0.f, bad);
    }
    if (bad != 0.f) hi = __int_as_float(0x7F800000);
#pragma unroll
    for (int o = PER >> 1; o > 0; o >>= 1) {
      if (ZP) lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    float s = __fdiv_rn(ZP ? __fsub_rn(hi, lo) : hi, ZP ? 15.f : 7.f);
    s = s == 0.f ? 1.f : fmaxf(s, kLeast);
    const TS stored = from_f32<TS>(s);
    const Divisor d = divisor(to_f32(stored));
    const float zero = ZP ? fminf(fmaxf(rintf(quotient(-lo, d)), 0.f), 15.f) : 8.f, least = (ZP ? 0.f : 1.f) - zero, most = 15.f - zero;
    const uint32_t z = (uint32_t)zero;
    uint32_t w = 0;
#pragma unroll
    for (int e = 7; e >= 0; --e) {
      // rounded after the cut, whose ends are whole numbers; and not with the zero point, which would turn ties
      const float q = fminf(fmaxf(quotient(v[e], d), least), most);
      w = w << 4 | (__float_as_uint(q + kInteger) + z & 15u);
    }
    if (col < p.k) *reinterpret_cast<uint32_t *>(p.codes + row * (p.k / 2) + col / 2) = w;
    const int group = col / (8 * PER);
    if (lane % PER == 0 && group < groups) {
      static_cast<TS *>(p.scales)[row * groups + group] = stored;
      if (ZP) p.zeros[row * groups + group] = (uint8_t)z;
    }
  }
}

// Sixteen values a lane: code less zero point, exact in T, times the scale, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) int4_widen_kernel(const __grid_constant__ Int4WeightParams p) {
  const int lane = threadIdx.x & 31, groups = (p.k + p.group - 1) / p.group, shift = p.group == 32 ? 5 : p.group == 64 ? 6 : 7;
  RowChunks<512> c(p.k);
  pdl_wait();
  for (; c.row < p.n; c.next()) {
    const int col = c.column() + 16 * lane;
    if (col >= p.k) continue;
    const uint2 w = *reinterpret_cast<const uint2 *>(p.codes + c.row * (p.k / 2) + col / 2);
    const long long g = c.row * groups + (col >> shift);
    const uint32_t scale = static_cast<const uint16_t *>(p.scales)[g] * 0x10001u;
    const Zero<T> z = zero_of<T>(p.zeros ? p.zeros[g] & 15u : 8u);
    uint32_t o[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t v[4];
      widen_codes<T>(h ? w.y : w.x, z, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __half>::value) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(scale));
        else asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(v[i]) : "r"(scale));
      }
      // from pairs of columns i and i + 4 to neighbours
      o[4 * h] = __byte_perm(v[0], v[1], 0x5410);
      o[4 * h + 1] = __byte_perm(v[2], v[3], 0x5410);
      o[4 * h + 2] = __byte_perm(v[0], v[1], 0x7632);
      o[4 * h + 3] = __byte_perm(v[2], v[3], 0x7632);
    }
    uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + c.row * p.ld_out + col);
    out[0] = make_uint4(o[0], o[1], o[2], o[3]);
    out[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <typename T, typename TS>
cudaError_t quantise_launch(const Int4WeightParams &p, int num_sms, cudaStream_t st) {
  const long long ctas = ((long long)p.n * ((p.k + 255) / 256) + 7) / 8, most = 4ll * num_sms;
  const dim3 grid((unsigned)(ctas < most ? ctas : most));
  auto pick = [&](auto zp) {
    constexpr bool ZP = decltype(zp)::value;
    return p.group == 32   ? int4_quantise_kernel<T, TS, 4, ZP>
           : p.group == 64 ? int4_quantise_kernel<T, TS, 8, ZP>
                           : int4_quantise_kernel<T, TS, 16, ZP>;
  };
  return launch_pdl(p.zeros ? pick(std::true_type()) : pick(std::false_type()), grid, dim3(256), 0, st, p);
}

}  // namespace

// Strips: as many to a warp as the matrix's rows can spare (they share what is read of x).  Shares of k: as many as k has
// tiles, unless sets of rows alone keep every warp of the GPU busy.
Int4Tiles int4_pick_tiles(int rows, int n, int k, int num_sms) {
  Int4Tiles t;
  t.eights = rows <= 8 ? 1 : rows <= 16 ? 2 : 4;
  t.strips = t.eights == 1 && n >= 64 * num_sms ? 4 : t.eights >= 2 && n >= 32 * num_sms ? 2 : 1;
  const int tiles = (k + kTileK - 1) / kTileK, strips = (n + 16 * t.strips - 1) / (16 * t.strips);
  t.log_kw = 0;
  const int most = t.eights == 1 ? 3 : t.eights == 2 ? 2 : 1;  // each share has its own columns of x in a step
  while (t.log_kw < most && (2 << t.log_kw) <= tiles && (strips << t.log_kw) < 2 * kFewWarps * num_sms) ++t.log_kw;
  t.box_rows = t.eights > 1 ? 8 * t.eights : rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : 8;
  return t;
}

template <typename T>
cudaError_t launch_int4_typed(const Int4MatmulParams &p, const Int4Maps &maps, const Int4Tiles &t, int num_sms, cudaStream_t st) {
  if (p.w.group_shift == 5) return p.w.zeros ? int4_tiles<T, 1, true>(p, maps, t, num_sms, st) : int4_tiles<T, 1, false>(p, maps, t, num_sms, st);
  if (p.w.group_shift == 6) return p.w.zeros ? int4_tiles<T, 2, true>(p, maps, t, num_sms, st) : int4_tiles<T, 2, false>(p, maps, t, num_sms, st);
  return p.w.zeros ? int4_tiles<T, 4, true>(p, maps, t, num_sms, st) : int4_tiles<T, 4, false>(p, maps, t, num_sms, st);
}

cudaError_t launch_int4_matmul(const Int4MatmulParams &p, const Int4Maps &maps, const Int4Tiles &t, bool f16, int num_sms,
                               cudaStream_t st) {
  return f16 ? launch_int4_typed<__half>(p, maps, t, num_sms, st) : launch_int4_typed<__nv_bfloat16>(p, maps, t, num_sms, st);
}

cudaError_t launch_int4_quantise(const Int4WeightParams &p, int num_sms, cudaStream_t st) {
  if (p.type == kF32)
    return p.f16 ? quantise_launch<float, __half>(p, num_sms, st) : quantise_launch<float, __nv_bfloat16>(p, num_sms, st);
  if (p.type == kF16)
    return p.f16 ? quantise_launch<__half, __half>(p, num_sms, st) : quantise_launch<__half, __nv_bfloat16>(p, num_sms, st);
  return p.f16 ? quantise_launch<__nv_bfloat16, __half>(p, num_sms, st)
               : quantise_launch<__nv_bfloat16, __nv_bfloat16>(p, num_sms, st);
}

cudaError_t launch_int4_widen(const Int4WeightParams &p, int num_sms, cudaStream_t st) {
  const long long ctas = ((long long)p.n * ((p.k + 511) / 512) + 7) / 8, most = 8ll * num_sms;
  const dim3 grid((unsigned)(ctas < most ? ctas : most));
  return launch_pdl(p.f16 ? int4_widen_kernel<__half> : int4_widen_kernel<__nv_bfloat16>, grid, dim3(256), 0, st, p);
}

}  // namespace moe
