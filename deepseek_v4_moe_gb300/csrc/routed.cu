// A whole mixture-of-experts layer on a plain residual stream for a few tokens, with 16-bit weights (sm_103a), in three
// kernels:
//
//   route   l = x Wr^T
//   up      each CTA chooses the experts from l; h = weight act(x Wg_e^T) (x Wu_e^T) for every token and expert
//   down    y = sum over the experts of h Wd_e^T
//
// Bound by the chosen experts' weights on their way from memory: each is read once, for all of its tokens.  Column j of
// the tensor cores' right operand is token j for every expert (zeros where it did not choose it), so the down kernel adds
// all experts' products in its accumulators: no partial results in memory, and one order of every sum.
// One token through 256 experts of 4096 x 2048 and a shared one, six each: 65.6 us, 5.4 TB/s (52 at the copy's rate): gate and
// up read at 5.7 TB/s once they know the experts.  5 tokens through 60 experts of 1000 x 424: 22.7 us (6.6), three kernels'
// latencies.
#include "dense_tc.cuh"
#include "kernels.h"
#include "routed.cuh"

namespace moe {
namespace {

template <typename T, typename TR>
__global__ void __launch_bounds__(256) routed_logits_kernel(const __grid_constant__ RoutedParams p) {
  pdl_wait();
  pdl_trigger();
  route_logits<T, TR>(p, blockIdx.x * kRouteExperts, blockIdx.y * kRouteTokens);
}

// The weights are the left operand as they lie (128 rows x 64 columns a step, K-major, by TMA), all tokens' columns the
// right one, so that nothing but copies and one instruction for 16 columns is left: the kernels run at the pace of memory.
// (On mma.sync, a strip of 16 rows to a warp, one token of 256 experts of 4096 x 2048 took 72 to 83 us: copies of
// 16 rows x 64 bytes do not come faster than 3.2 TB/s.)
//
// Up: a tile is 64 rows of gate and 64 of up; two accumulators in TMEM, so that a tile's epilogue runs beside the next
// tile's products.  h lies by experts, [expert's place among the chosen][tokens, up to a multiple of 8][inter], with zeros
// for the tokens that have not chosen it: the down kernel's right operand, as it needs it.
// Down: a tile is 128 rows; the experts' steps are shared by the CTAs of a cluster, whose sums meet in shared memory.

constexpr int kTcThreads = 192, kTcRows = 128, kTcW = kTcRows * 128;
// NC: columns of the right operand, tokens in gate and up, two for each in down
template <int NC>
constexpr int kTcStage = kTcW + NC * 128;
template <int NC>
constexpr int kTcRing = NC == 16 ? 5 : NC == 32 ? 4 : 3;  // two CTAs on an SM: the down kernel's come while the up kernel's end
template <int NC>
constexpr size_t kTcSmem = kTcRing<NC> * kTcStage<NC> + 1024;

// what the second part of a hidden value is multiplied by, so that it is a normal number where the first one is
template <typename T>
constexpr float kLow = std::is_same<T, __half>::value ? 0x1p11f : 0x1p8f;

// NC columns of this thread's lane of an accumulator
template <int NC>
__device__ __forceinline__ void read_accumulator(uint32_t at, float (&v)[NC]) {
#pragma unroll
  for (int i = 0; i < NC; i += 16) tmem_ld16(at + i, reinterpret_cast<float(&)[16]>(v[i]));
}

// A result from the token's own experts alone, by a warp: see the down kernel's end.  (32 tokens of 64 experts of 4096 x 2048
// with a NaN in each row of the shared expert's matrix, so that every result comes here and stays NaN: 3.2 ms, for 0.48.)
template <typename T>
__device__ __noinline__ float own_experts(const RoutedParams &p, const Choice &c, int rows8, int token, int n) {
  auto eight = [](const T *at, float (&v)[8]) {
    const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(at));
    unpack2(w.x, v[0], v[1], at);
    unpack2(w.y, v[2], v[3], at);
    unpack2(w.z, v[4], v[5], at);
    unpack2(w.w, v[6], v[7], at);
  };
  float sum = 0.f;
  for (int g = 0; g < c.groups; ++g) {
    if (!(c.group_mask[g] >> token & 1)) continue;
    const int e = c.group_expert[g];
    const FewMatrix &m = e >= p.experts ? p.s_down : p.down;
    const T *w = static_cast<const T *>(m.w) + ((long long)(e >= p.experts ? e - p.experts : e) * p.hidden + n) * p.inter;
    const T *h = reinterpret_cast<const T *>(p.h) + ((long long)g * (2 * rows8) + token) * p.inter;
    for (int k = threadIdx.x % 32 * 8; k < p.inter; k += 256) {
      float a[8], b[8], low[8];
      eight(w + k, a);
      eight(h + k, b);
      eight(h + (long long)rows8 * p.inter + k, low);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(a[i], fmaf(low[i], 1.f / kLow<T>, b[i]), sum);
    }
    if (__any_sync(0xffffffffu, sum != sum)) break;  // its own
  }
  return warp_sum(sum);
}

template <bool UP, typename T, int NC>
__global__ void __launch_bounds__(kTcThreads, 2)
    routed_tc_kernel(const __grid_constant__ RoutedParams p, const __grid_constant__ RoutedMaps maps, int splits) {
  constexpr int kTcStages = kTcRing<NC>;
  extern __shared__ char smem[];
  __shared__ Choice c;
  __shared__ __align__(8) uint64_t full[kTcStages], empty[kTcStages], tfull[2], tempty[2], mma_done, never;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;
  constexpr int kTokens = UP ? NC : NC / 2;
  __shared__ float sums[UP ? 2 : 1][kTokens * (UP ? 64 : kTcRows)];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  char *ring = smem + (-smem_u32(smem) & 1023u);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kTcStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(&mma_done, 1);
    mbar_init(&never, 1);
    abort_flag = 0;
    issued = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_base, 64);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  if constexpr (UP) {
    pdl_wait();
    // The down kernel's CTAs may come, choose and fetch weights: not earlier, as they read the logits.
    pdl_trigger();
  }
  choose_groups(p, c, reinterpret_cast<uint32_t *>(ring), UP && blockIdx.x == 0);  // (the ring is not in use yet)
  volatile int *abort_p = &abort_flag;
  const Waits &w = p.waits;
  const int rows8 = (p.rows + 7) / 8 * 8, columns = UP ? rows8 : 2 * rows8, depth = UP ? p.hidden : p.inter, steps = (depth + 63) / 64;
  const int tiles = UP ? (p.inter + 63) / 64 : 1;  // of an expert
  // UP: units of an expert's tile, one after another; otherwise one tile, and this CTA's share of all experts' steps
  const int rank = UP ? 0 : blockIdx.x % splits, tile_down = UP ? 0 : blockIdx.x / splits;
  const int units = UP ? c.groups * tiles : 1, unit0 = UP ? blockIdx.x : 0, unit_step = UP ? gridDim.x : 1;
  const long long all = (long long)c.groups * steps;
  const int first = UP ? 0 : (int)(all * rank / splits), end = UP ? steps : (int)(all * (rank + 1) / splits);

  if (warp == 0) {
    // ---------------- copies ----------------
    const uint32_t ring0 = smem_u32(ring), bytes = kTcW + columns * 128;
    RingPos<kTcStages> pos;
    int j = 0, group = UP ? 0 : first / steps, k = UP ? 0 : first % steps, unit = unit0, step = first;
    auto weights = [&](int s) {
      const uint32_t at = ring0 + s * kTcStage<NC>, bar = smem_u32(&full[s]);
      mbar_expect_one(bar, bytes);
      const int e = c.group_expert[group];
      const bool shared = e >= p.experts;
      const int row = (shared ? e - p.experts : e) * (UP ? p.inter : p.hidden);
      if constexpr (UP) {
        const int r = row + (unit - group * tiles) * 64;
        tma_load_2d_one<false>(at, shared ? &maps.s_gate : &maps.gate, bar, k * 64, r);
        tma_load_2d_one<false>(at + 64 * 128, shared ? &maps.s_up : &maps.up, bar, k * 64, r);
      } else {
        tma_load_2d_one<false>(at, shared ? &maps.s_gate : &maps.gate, bar, k * 64, row + tile_down * kTcRows);
      }
    };
    auto tokens = [&](int s, int g, int kk) {
      tma_load_2d_one<false>(ring0 + s * kTcStage<NC> + kTcW, &maps.tokens, smem_u32(&full[s]), kk * 64, UP ? 0 : g * columns);
    };
    auto next = [&] {
      ++step;
      if (++k == steps) {
        k = 0;
        if (!UP) ++group;
      }
      if (UP && step == end) {
        step = 0;
        unit += unit_step;
        group = unit / tiles;
      }
    };
    if (UP) group = unit / tiles;
    if constexpr (!UP) {  // the first weights need not wait for h
      const int g0 = group, k0 = k;
      for (; j < kTcStages && step < end; ++j, next()) weights(j);
      pdl_wait();
      pdl_trigger();
      int g = g0, kk = k0;
      for (int i = 0; i < j; ++i) {
        tokens(i, g, kk);
        if (++kk == steps) {
          kk = 0;
          ++g;
        }
      }
      for (int i = 0; i < j; ++i) pos.next();
    }
    for (; unit < units && step < end; ++j, pos.next(), next()) {
      if (!warp_wait(&empty[pos.slot], pos.round ^ 1u, abort_p, w.status, w.ns)) break;
      weights(pos.slot);
      tokens(pos.slot, group, k);
    }
    if (lane == 0) issued = j;
  } else if (warp == 1) {
    // ---------------- products ----------------
    if (w.inject && blockIdx.x == 0) (void)warp_wait(&never, 0u, abort_p, w.status, w.ns);  // test hook: a wait that runs out
    const uint32_t idesc = std::is_same<T, __half>::value ? idesc_f16_f32(kTcRows, NC) : idesc_bf16_f32(kTcRows, NC);
    const uint64_t a0 = smem_desc_sw128(smem_u32(ring)), b0 = a0 + (kTcW >> 4);
    RingPos<kTcStages> pos;
    RingPos<2> acc;
    bool ok = true;
    for (int unit = unit0; ok && unit < units; unit += unit_step, acc.next()) {
      if (!warp_wait(&tempty[acc.slot], acc.round ^ 1u, abort_p, w.status, w.ns)) break;
      for (int step = first; step < end; ++step, pos.next()) {
        if (!warp_wait(&full[pos.slot], pos.round, abort_p, w.status, w.ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = pos.slot * (kTcStage<NC> >> 4), d = tmem + acc.slot * 32;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tc_mma_one<false, false>(d, a0 + (at + k * 2), b0 + (at + k * 2), idesc, step > first || k > 0 ? 1u : 0u);
        tc_commit_one<false>(smem_u32(&empty[pos.slot]));
      }
      if (ok) tc_commit_one<false>(smem_u32(&tfull[acc.slot]));
    }
    // every MMA this warp issued completes before TMEM is freed
    tc_commit_one<false>(smem_u32(&mma_done));
    int no_abort = 0;
    (void)wait_bounded(&mma_done, 0u, &no_abort, w.status, w.ns);
  } else {
    // ---------------- results ----------------
    const int q = warp & 3, row = q * 32 + lane;
    RingPos<2> acc;
    for (int unit = unit0; unit < units; unit += unit_step, acc.next()) {
      float v[kTokens];
      const bool ok = (UP || first < end) && warp_wait(&tfull[acc.slot], acc.round, abort_p, w.status, w.ns);
      if (ok) {
        tc_fence_after();
        const uint32_t at = tmem + ((uint32_t)(q * 32) << 16) + acc.slot * 32;
        if constexpr (UP) {
          read_accumulator<NC>(at, v);
        } else if constexpr (NC == 16) {  // eight tokens: both parts in one reading
          float both[16];
          read_accumulator<16>(at, both);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fmaf(both[8 + i], 1.f / kLow<T>, both[i]);
        } else {
          read_accumulator<kTokens>(at, v);
#pragma unroll
          for (int i = 0; i < kTokens; i += 16) {
            float low[16];
            read_accumulator<16>(at + rows8 + i, low);  // (past the last token what nobody reads)
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i + j] = fmaf(low[j], 1.f / kLow<T>, v[i + j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc.slot]);
      } else {
#pragma unroll
        for (int i = 0; i < kTokens; ++i) v[i] = 0.f;
      }
      if constexpr (UP) {
        float *u = sums[acc.slot];
        if (q >= 2)
#pragma unroll
          for (int t = 0; t < NC; ++t)
            if (t < p.rows) u[t * 64 + row - 64] = v[t];
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int group = unit / tiles, at = (unit - group * tiles) * 64 + row, e = c.group_expert[group];
        const uint32_t mask = c.group_mask[group];
        const float weight = weight_of(p, c, e, lane);  // this lane's token's
        if (q < 2) {
          uint16_t *h = p.h + (long long)group * (2 * rows8) * p.inter + at;
#pragma unroll
          for (int t = 0; t < NC; ++t) {
            if (t >= p.rows) break;
            T out = from_f32<T>(0.f), low = out;
            if (mask >> t & 1) {
              const float x = acts_f32(p.act, make_float2(v[t], v[t])).x * u[t * 64 + row] * __shfl_sync(0xffffffffu, weight, t);
              out = from_f32<T>(x);
              const float rest = x - to_f32(out);  // (an infinity has none)
              if (fabsf(rest) < INFINITY) low = from_f32<T>(rest * kLow<T>);
            }
            if (at < p.inter) {
              h[(long long)t * p.inter] = *reinterpret_cast<const uint16_t *>(&out);
              h[(long long)(rows8 + t) * p.inter] = *reinterpret_cast<const uint16_t *>(&low);
            }
          }
        }
      } else {
#pragma unroll
        for (int t = 0; t < kTokens; ++t)
          if (t < p.rows) sums[0][t * kTcRows + row] = v[t];
      }
    }
  }
  // Copies still in flight after an abort land before the CTA may leave (bounded; otherwise each has landed).
  tc_fence_before();
  __syncthreads();
  if (abort_flag && threadIdx.x == 0) {
    int no_abort = 0;
    for (int s = 0; s < kTcStages; ++s) {
      const int n = issued / kTcStages + (s < issued % kTcStages ? 1 : 0);
      if (n > 0) (void)wait_bounded(&full[s], (uint32_t)((n - 1) & 1), &no_abort, w.status, w.ns);
    }
  }
  if constexpr (!UP) {
    // the CTAs' sums in the order of their ranks, a part of the rows by each
    if (splits > 1) cluster_sync();
    // An infinity or a NaN of an expert's matrix is NaN as 0 times it for the tokens that have not chosen it: such results
    // are formed again.  (Without one this is a comparison for each result.)
    const int part = kTcRows / splits, row0 = rank * part, count = part * p.rows;
    for (int i0 = 0; i0 < count; i0 += kTcThreads) {
      const int i = i0 + threadIdx.x, row = row0 + i % part, t = i / part, at = tile_down * kTcRows + row;
      const bool in = i < count && at < p.hidden;
      float v = 0.f, x[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)  // all loads before the first sum
        if (in && r < splits)
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x[r]) : "r"(in_cta(&sums[0][t * kTcRows + row], r)) : "memory");
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (in && r < splits) v += x[r];
      for (unsigned again = __ballot_sync(0xffffffffu, v != v); again; again &= again - 1) {
        const int from = __ffs(again) - 1;
        const float own = own_experts<T>(p, c, rows8, __shfl_sync(0xffffffffu, t, from), __shfl_sync(0xffffffffu, at, from));
        if (lane == from) v = own;
      }
      if (in) static_cast<T *>(p.y)[t * p.ld_y + at] = from_f32<T>(v);
    }
    if (splits > 1) cluster_sync();
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
  }
}

template <typename T, int NC, int DOWN>
cudaError_t tc_launch(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, int num_sms, cudaStream_t st) {
  static std::atomic<unsigned long long> done[2];
  cudaError_t e = allow_smem((const void *)routed_tc_kernel<true, T, NC>, kTcSmem<NC>, done[0]);
  if (e == cudaSuccess)
    e = launch_pdl(p.router_f32 ? routed_logits_kernel<T, float> : routed_logits_kernel<T, T>,
                   dim3(route_ctas(p), route_turns(p)), dim3(256), 0, st, p);
  const long long groups = (p.rows * p.top_k < p.experts ? p.rows * p.top_k : p.experts) + p.shared;
  const long long units = groups * ((p.inter + 63) / 64);
  if (e == cudaSuccess)
    e = launch_pdl(routed_tc_kernel<true, T, NC>, dim3((unsigned)(units < 2 * num_sms ? units : 2 * num_sms)), dim3(kTcThreads), kTcSmem<NC>, st, p,
                   maps, 1);
  if (e != cudaSuccess) return e;
  // as many CTAs to a tile as run at one time, two on an SM (of clusters of 8, 4 and 2 on 152 SMs 32, 72 and 150)
  const int tiles = (p.hidden + kTcRows - 1) / kTcRows;
  const int splits = tiles <= num_sms * 32 / 152 ? 8 : tiles <= num_sms * 72 / 152 ? 4 : tiles <= num_sms * 150 / 152 ? 2 : 1;
  return launch_clusters(routed_tc_kernel<false, T, DOWN>, kTcSmem<DOWN>, done[1], tiles, splits, kTcThreads, st, p, down, splits);
}

template <typename T>
cudaError_t routed_typed(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, int num_sms, cudaStream_t st) {
  if (p.rows <= 8) return tc_launch<T, 16, 16>(p, maps, down, num_sms, st);
  return p.rows <= 16 ? tc_launch<T, 16, 32>(p, maps, down, num_sms, st) : tc_launch<T, 32, 64>(p, maps, down, num_sms, st);
}

}  // namespace

cudaError_t launch_routed(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, bool f16, int num_sms, cudaStream_t st) {
  return f16 ? routed_typed<__half>(p, maps, down, num_sms, st) : routed_typed<__nv_bfloat16>(p, maps, down, num_sms, st);
}

}  // namespace moe
