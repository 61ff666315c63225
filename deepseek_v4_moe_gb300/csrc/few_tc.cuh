// 4-bit weights on the FP8 tensor cores (sm_103a): the pipeline that the product of a few rows and the routed layer share.
//
// A code 0 .. 15 in a byte is the E4M3 number code 2^-9: its first eight are the subnormal numbers, the next eight have the
// smallest exponent, and both count in steps of 2^-9.  So three instructions (a mask, a shift, a mask) make eight codes an
// operand of the tensor cores, where sixteen-bit ones take 11, and the weights come from memory, through registers, into
// TMEM as the left operand.  (On mma.sync in 16 bits 16 tokens by 129280 x 4096 took 93 us, at 25 instructions for eight
// codes; mma.sync's FP8 form is made of 16-bit products, with a conversion of either operand each time: 146 us.)
//
// The right operand is split beforehand: scaled by a power of two, so that its largest magnitude lies in [128, 256), into
// p0 = e4m3(x), p1 = e4m3(32 (x - p0)) and, for f16 and the routed layer's hidden values, p2 = e4m3(32 (32 (x - p0) - p1)).
// Each plane takes four significant bits, so that two are a bf16 number and three an f16 one: exactly down to 2^-14 of the
// largest magnitude (f16: 2^-16), below that to 2^-22 of it (2^-27; two planes without the 32: 2^-17).  Half a step of three
// is 2^-14 of an f32 value.  The planes are columns of their own; a group's
// products are joined in f32, its zero point is applied to its sum of x, and its scale to the result, once for each group:
//   acc += scale (sum(code p0) + sum(code p1) / 32 + .. - zero sum(x))
//
// Roles: a warp copies (TMA), one or two issue the products, four or eight make codes operands and four or eight join the
// groups (in sets of four, of which a thread has a row; its sums of the tokens stay in registers).
// Joining is what comes before the memory: every role's warp has about 900 cycles for a tile of 128 rows x 256 columns at
// 5 TB/s, and a set of joining warps took 2050 for two.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "dense_tc.cuh"
#include "dense_vec.cuh"
#include "few.h"

namespace moe {

constexpr int kCodeRows = 128;  // of a tile; it has 256 columns, or 128 (code_halves)
constexpr int kCodeSlotsMax = 8;
constexpr float kPlane = 0.03125f;

// TOKENS: 8, 16 or 32; PLANES: 2 or 3; GROUPS of 128 columns: 1, 2 or 4
template <int TOKENS, int PLANES, int GROUPS>
struct CodeCfg {
  static constexpr int kTokens = TOKENS;
  static constexpr int kRows = TOKENS * PLANES;                 // of the right operand
  static constexpr int kN = (kRows + 15) / 16 * 16;             // columns of the sums
  static constexpr int kHalves = code_halves(TOKENS, PLANES, GROUPS), kAll = kHalves * GROUPS;  // of 128 columns; groups
  static constexpr int kW = kCodeRows * 64 * kHalves;           // bytes of codes
  static constexpr int kB = kN * 128, kSums = kAll * TOKENS * 4;
  static constexpr int kStage = kW + kHalves * kB + (kSums + 1023) / 1024 * 1024;
  static constexpr uint32_t kBytes = kW + kHalves * kRows * 128 + kSums;
  // Slots in TMEM of a tile's sums (all its groups') and of left operands.  Warps that issue products, and sets of four
  // that make operands and that join groups, take tiles in turn.  A set sees a barrier's every round only if no other set
  // uses its slot, so the numbers of slots and stages are multiples of the sets'.
  static constexpr int kD = kAll * kN <= 64 ? 4 : kAll * kN <= 192 ? 2 : 1;
  static constexpr int kIssue = kD > 1 ? 2 : 1;
  // Two sets make operands where little else is done (one token through the routed layer in groups of 128 40.8 us, with one
  // set 42.2); otherwise their instructions are missed where groups are joined (16 tokens in groups of 32 510 us, with one
  // set 487, of 128 220 and 218).
  static constexpr int kSets = TOKENS == 8 && GROUPS == 1 ? 2 : 1;
  // Sets that join take every other tile, of 32 tokens 16 each of every tile: all of them in one set have no registers for
  // the next scales (32 tokens by 129280 x 4096 in groups of 128: 80.9 us, 73.3 so; f16 79.7 and 76.0).  Two planes in
  // groups of 32 have one set, as every step is another's wait there (8192 x 8192: 37.1, in two 41.0; f16 42.4 and 41.2).
  static constexpr int kHalf = TOKENS > 16 && (GROUPS < 4 || PLANES > 2) ? 2 : 1, kTurns = kHalf == 1 && kD > 1 ? 2 : 1;
  static constexpr int kJoin = kHalf * kTurns, kMine = TOKENS / kHalf;
  static constexpr int kFit = 180 * 1024 / kStage < 12 ? 180 * 1024 / kStage : 12, kStages = kFit / 2 * 2;
  static constexpr int kRoom = (512 - kD * kAll * kN) / (32 * kHalves), kA = (kRoom < 8 ? kRoom : 8) / 2 * 2;
  static constexpr int kFirstJoin = 1 + kIssue + (1 + kIssue) % 2, kFirstMake = kFirstJoin + 4 * kJoin;  // their first warps
  static constexpr int kRing = kStages * kStage;
  static constexpr int kThreads = 32 * (kFirstMake + 4 * kSets);
  static_assert(kA >= 2 && kA <= kCodeSlotsMax && kStages >= 2, "slots");
};

// A row's power of two: what is split is x 2^e; max: the largest magnitude's bits as f32.  (Values below 2^-119 count as
// that: the sums' way back has to be a normal number.)
__device__ __forceinline__ int plane_exponent(uint32_t max) {
  const int e = 7 + 127 - (int)(max >> 23);
  return e > 126 ? 126 : e;
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

__device__ __forceinline__ float2 e4m3_pair(uint32_t c) {
  uint32_t f;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}" : "=r"(f) : "r"(c));
  return __half22float2(*reinterpret_cast<const __half2 *>(&f));
}
// the planes' codes of two scaled values, in the low 16 bits of o[plane]; returns the sum of what they stand for
template <int PLANES>
__device__ __forceinline__ float split2(float a, float b, uint32_t (&o)[PLANES]) {
  float sum = 0.f, unit = 1.f;
#pragma unroll
  for (int i = 0; i < PLANES; ++i) {
    o[i] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const float2 v = e4m3_pair(o[i]);
    sum = fmaf(v.x + v.y, unit, sum);
    a = (a - v.x) * 32.f;
    b = (b - v.y) * 32.f;
    unit *= kPlane;
  }
  return sum;
}
// Eight values' codes of each plane as they stand in the operand: even columns, then odd ones, as a word's codes leave them.
template <int PLANES>
__device__ __forceinline__ float split8(const float (&v)[8], float scale, uint2 (&o)[PLANES]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < PLANES; ++i) o[i] = make_uint2(0u, 0u);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t c[PLANES];
      sum += split2<PLANES>(v[4 * j + h] * scale, v[4 * j + 2 + h] * scale, c);
#pragma unroll
      for (int i = 0; i < PLANES; ++i) (h ? o[i].y : o[i].x) |= c[i] << (16 * j);
    }
  return sum;
}

// eight values in 16-byte pieces (a workspace is aligned to those)
template <typename T>
__device__ __forceinline__ void load_pieces(const T *x, float (&v)[8]) {
  if constexpr (std::is_same<T, float>::value) {
    const float4 a = reinterpret_cast<const float4 *>(x)[0], b = reinterpret_cast<const float4 *>(x)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    load_eight<T, true>(x, 0, 1, 8, v);
  }
}

// A row's planes (out, `apart` between two planes) and groups' sums, by a CTA of 256: k8 eights of columns of x, scaled;
// `groups` of `per` eights up to the last tile's, each sum `tokens` floats from the one before.  x none: zeros.
template <typename T, int PLANES>
__device__ __forceinline__ void split_row(const T *x, float scale, int k8, int groups, int per, uint2 *out, size_t apart, float *sums, int tokens) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, all = groups * per;
  for (int i0 = warp * 32; i0 < all; i0 += 256) {
    const int i = i0 + lane;
    float sum = 0.f;
    if (i < k8) {
      uint2 o[PLANES] = {};
      if (x) {
        float v[8];
        load_pieces(x + 8 * i, v);
        sum = split8<PLANES>(v, scale, o);
      }
#pragma unroll
      for (int k = 0; k < PLANES; ++k) out[k * apart + i] = o[k];
    }
    for (int o = per >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (i < all && i % per == 0) sums[i / per * tokens] = sum * 0x1p-9f;
  }
}
// the bits of a row's largest magnitude, by a CTA of 256
template <typename T>
__device__ __forceinline__ uint32_t row_max(const T *x, int k8) {
  __shared__ uint32_t most[8];
  uint32_t m = 0;
  for (int i = threadIdx.x; i < k8; i += 256) {
    float v[8];
    load_pieces(x + 8 * i, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(v[e]) & 0x7FFFFFFFu);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if (threadIdx.x % 32 == 0) most[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, most[i]);
  return m;
}
// what a row's sums are multiplied by; a row that is not finite gives NaN
__device__ __forceinline__ float way_back(uint32_t max) {
  return max >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : two_to(-plane_exponent(max));
}

// instruction descriptor, kind::f8f6f4: E4M3 operands (K-major), f32 sums, M x N
__device__ __forceinline__ uint32_t idesc_e4m3(int M, int N) { return 1u << 4 | (uint32_t)(N >> 3) << 17 | (uint32_t)(M >> 4) << 24; }

// D (+)= A B^T, A (128 rows x 32 columns, a byte each) in TMEM, B from shared memory; by one lane of a converged warp
__device__ __forceinline__ void mma_codes_one(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
      "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
      "r"(r[31])
      : "memory");
}
// N columns of this thread's lane in sixteens `apart` columns from one another; they have arrived after tmem_arrived
template <int N>
__device__ __forceinline__ void tmem_columns(uint32_t at, int apart, float (&v)[N]) {
  if (apart < 16) apart = 16;  // eight tokens: their planes side by side
#pragma unroll
  for (int i = 0; i < N; i += 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=f"(v[i]), "=f"(v[i + 1]), "=f"(v[i + 2]), "=f"(v[i + 3]), "=f"(v[i + 4]), "=f"(v[i + 5]), "=f"(v[i + 6]),
          "=f"(v[i + 7]), "=f"(v[i + 8]), "=f"(v[i + 9]), "=f"(v[i + 10]), "=f"(v[i + 11]), "=f"(v[i + 12]), "=f"(v[i + 13]),
          "=f"(v[i + 14]), "=f"(v[i + 15])
        : "r"(at + i / 16 * apart));
}
template <int N>
__device__ __forceinline__ void tmem_arrived(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
// two f32 multiply-adds in one instruction
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void unpair(uint64_t v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
// a piece of memory into this CTA's shared memory, by one lane of a converged warp (bytes a multiple of 16)
__device__ __forceinline__ void tma_bulk_one(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

template <typename C>
struct CodeBars {
  float join[2][C::kTurns > 1 ? C::kTokens * kCodeRows : 1];
  uint64_t full[12], empty[12], afull[kCodeSlotsMax], aempty[kCodeSlotsMax], dfull[kCodeSlotsMax], dempty[kCodeSlotsMax], mma_done[2], never;
  uint32_t tmem;
  int abort_flag, issued;
};

// The kernel's body.  A job gives this CTA's tiles, the same to every role:
//   int count();  Place begin();  place.more(), place.tile;  next(place)    its tiles, one after another through its units
//   void weights(place, at, bar)                             its codes' copy, by the converged warp
//   void ready();  void tokens(place, at, sums, bar)         what the tokens' copies wait for; they, and their groups' sums
//   next_unit(place);  int unit_tiles();  bool skip(place, tiles)   on within the unit: whether there is such a tile
//   Row; void row_at(row, place, r);  next_row(row, place)   where row r of a unit, and of the one after it, has its scales;
//                                                            the next ones are fetched into the L2
//   Scales; void scales(row, place, ahead, s); last(place)   those of the tile `ahead` tiles on; the end of such tiles
//   void finish(place, r, turn, barrier, t0, acc)            by 128 threads with a barrier for them, of tokens from t0 on;
//                                                            turn: 0 and 1, unit after unit
template <typename C, int TOKENS, int PLANES, int GROUPS, typename Job>
__device__ __forceinline__ void code_pipeline(Job &job, char *ring, CodeBars<C> &b, const Waits &w) {
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  constexpr int S = C::kStages;
  volatile int *abort_p = &b.abort_flag;
  const uint32_t ring0 = smem_u32(ring), tmem = b.tmem, tmem_d = tmem + C::kA * C::kHalves * 32;
  if (warp == 0) {
    // ---------------- copies ----------------
    RingPos<S> pos;
    int j = 0;
    auto weights = [&](const auto &p, int s) {
      mbar_expect_one(smem_u32(&b.full[s]), C::kBytes);
      job.weights(p, ring0 + s * C::kStage, smem_u32(&b.full[s]));
    };
    auto tokens = [&](const auto &p, int s) {
      const uint32_t at = ring0 + s * C::kStage + C::kW;
      job.tokens(p, at, at + C::kHalves * C::kB, smem_u32(&b.full[s]));
    };
    auto p = job.begin(), early = p;
    for (; j < S && p.more(); ++j, job.next(p)) weights(p, j);  // these need not wait for the tokens
    job.ready();
    for (int i = 0; i < j; ++i, job.next(early), pos.next()) tokens(early, i);
    for (; p.more(); ++j, pos.next(), job.next(p)) {
      if (!warp_wait(&b.empty[pos.slot], pos.round ^ 1u, abort_p, w.status, w.ns)) break;
      weights(p, pos.slot);
      tokens(p, pos.slot);
    }
    if (lane == 0) b.issued = j;
  } else if (warp <= C::kIssue) {
    // ---------------- products ----------------
    if (w.inject && blockIdx.x == 0) (void)warp_wait(&b.never, 0u, abort_p, w.status, w.ns);  // test hook: a wait that runs out
    const uint32_t idesc = idesc_e4m3(kCodeRows, C::kN);
    const uint64_t b0 = smem_desc_sw128(ring0 + C::kW);
    RingPos<S> pos(warp - 1);
    RingPos<C::kA> a(warp - 1);
    RingPos<C::kD> d(warp - 1);
    for (int i = warp - 1, tiles = job.count(); i < tiles; i += C::kIssue, pos.next(C::kIssue), a.next(C::kIssue), d.next(C::kIssue)) {
      if (!warp_wait(&b.dempty[d.slot], d.round ^ 1u, abort_p, w.status, w.ns) ||
          !warp_wait(&b.full[pos.slot], pos.round, abort_p, w.status, w.ns) ||
          !warp_wait(&b.afull[a.slot], a.round, abort_p, w.status, w.ns))
        break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 4 * C::kHalves; ++k)
        mma_codes_one(tmem_d + (d.slot * C::kAll + k * GROUPS / 4) * C::kN, tmem + a.slot * (C::kHalves * 32) + k * 8,
                      b0 + (pos.slot * (C::kStage >> 4) + k / 4 * (C::kB >> 4) + k % 4 * 2), idesc, k % (4 / GROUPS) ? 1u : 0u);
      tc_commit_one<false>(smem_u32(&b.dfull[d.slot]));
    }
    // every MMA this warp issued completes before TMEM is freed
    tc_commit_one<false>(smem_u32(&b.mma_done[warp - 1]));
    int no_abort = 0;
    (void)wait_bounded(&b.mma_done[warp - 1], 0u, &no_abort, w.status, w.ns);
  } else if (warp >= C::kFirstMake) {
    // ---------------- codes to operands ----------------
    const int set = (warp - C::kFirstMake) >> 2, q = warp & 3, row = q * 32 + lane;
    RingPos<S> pos(set);
    RingPos<C::kA> a(set);
    for (int i = set, tiles = job.count(); i < tiles; i += C::kSets, pos.next(C::kSets), a.next(C::kSets)) {
      if (!warp_wait(&b.full[pos.slot], pos.round, abort_p, w.status, w.ns) ||
          !warp_wait(&b.aempty[a.slot], a.round ^ 1u, abort_p, w.status, w.ns))
        break;
      tc_fence_after();  // the products that read this slot before are complete
      const uint32_t at = ring0 + pos.slot * C::kStage + row * (64 * C::kHalves);
#pragma unroll
      for (int h = 0; h < C::kHalves; ++h) {
        uint4 c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          c[j] = lds128(at + ((C::kHalves == 2 ? (4 * h + j) ^ (row & 7) : j ^ (row >> 1 & 3)) << 4));
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t x[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[8 * j + 2 * e] = x[e] & 0x0F0F0F0Fu;
            v[8 * j + 2 * e + 1] = x[e] >> 4 & 0x0F0F0F0Fu;
          }
        }
        tmem_store32(tmem + ((uint32_t)(q * 32) << 16) + (a.slot * C::kHalves + h) * 32, v);
      }
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&b.afull[a.slot]);
        mbar_arrive(&b.empty[pos.slot]);
      }
    }
  } else if (warp >= C::kFirstJoin) {
    // ---------------- groups' sums ----------------
    // Sets take every other tile; at the units' ends they take turns in adding the other's sums to their own and finishing.
    // What a set does for a tile bounded the pipeline (2050 cycles, one step waiting for another): so a tile's scales are
    // read during the one before, and two multiply-adds are one instruction.
    const int q = warp & 3, set = (warp - C::kFirstJoin) >> 2;
    const int late = C::kTurns > 1 ? set : 0, t_first = C::kHalf > 1 ? set * C::kMine : 0;  // its first tile and token
    constexpr int kMine = C::kMine;
    constexpr bool kAhead = kMine < 32;  // (there are no registers for it otherwise)
    RingPos<S> pos(late);
    RingPos<C::kA> a(late);
    RingPos<C::kD> d(late);
    int turn = 0, skipped = late;  // tiles before this set's first in a unit
    uint64_t acc[kMine / 2];
    auto unit = job.begin();
    typename Job::Row row;
    typename Job::Scales now, next;
    if (unit.more()) job.row_at(row, unit, q * 32 + lane);
    bool ok = true;
    for (; unit.more(); job.next_unit(unit)) {
#pragma unroll
      for (int t = 0; t < kMine / 2; ++t) acc[t] = 0u;
      auto p = unit;
      bool in = job.skip(p, skipped), read = false;  // read: the scales are those of the next tile
      for (; in; in = job.skip(p, C::kTurns)) {
        if (!read) job.scales(row, p, 0, now);
        read = kAhead && p.tile + C::kTurns < job.last(p);  // (of the same rows)
        if (read) job.scales(row, p, C::kTurns, next);
        ok = ok && warp_wait(&b.full[pos.slot], pos.round, abort_p, w.status, w.ns);
        const uint32_t sums = ring0 + pos.slot * C::kStage + C::kW + C::kHalves * C::kB;
        ok = ok && warp_wait(&b.dfull[d.slot], d.round, abort_p, w.status, w.ns);
        tc_fence_after();
        if (ok) {
          // Sixteen tokens' sums of a group at a time (of eight tokens all planes' lie in one or two sixteens), of several
          // groups where registers allow it, so that their way is waited for once.
          constexpr int kChunk = kMine < 16 ? kMine : 16, kCols = TOKENS < 16 ? C::kN : 16 * PLANES;
          constexpr int kBatch = C::kAll * kCols <= 32 ? C::kAll : kCols <= 16 ? 2 : 1;
          const uint32_t from = tmem_d + ((uint32_t)(q * 32) << 16) + d.slot * (C::kAll * C::kN);
          const uint64_t plane = pair(kPlane, kPlane);
#pragma unroll
          for (int g0 = 0; g0 < C::kAll; g0 += kBatch)
#pragma unroll
            for (int t0 = 0; t0 < kMine; t0 += kChunk) {
              float v[kBatch][kCols];
#pragma unroll
              for (int g = 0; g < kBatch; ++g) tmem_columns<kCols>(from + (g0 + g) * C::kN + t_first + t0, TOKENS, v[g]);
              tmem_arrived(reinterpret_cast<float(&)[kBatch * kCols]>(v));
              if (g0 + kBatch >= C::kAll && t0 + kChunk == kMine) {  // everything is in registers: the tile's slots are free
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                  mbar_arrive(&b.dempty[d.slot]);
                  mbar_arrive(&b.aempty[a.slot]);
                }
              }
#pragma unroll
              for (int g = 0; g < kBatch; ++g) {
                const float zero = -now.zero(g0 + g), scale = now.scale(g0 + g);
                const uint64_t z = pair(zero, zero), m = pair(scale, scale);
#pragma unroll
                for (int t4 = 0; t4 < kChunk; t4 += 4) {
                  const uint4 x4 = lds128(sums + ((g0 + g) * TOKENS + t_first + t0 + t4) * 4);
                  const uint64_t x[2] = {pair(__uint_as_float(x4.x), __uint_as_float(x4.y)), pair(__uint_as_float(x4.z), __uint_as_float(x4.w))};
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const int t = t4 + 2 * i;
                    const float *at = &v[g][(PLANES - 1) * kChunk + t];
                    uint64_t s = pair(at[0], at[1]);
#pragma unroll
                    for (int k = PLANES - 2; k >= 0; --k) s = fma2(s, plane, pair(v[g][k * kChunk + t], v[g][k * kChunk + t + 1]));
                    acc[(t0 + t) / 2] = fma2(fma2(z, x[i], s), m, acc[(t0 + t) / 2]);
                  }
                }
              }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&b.empty[pos.slot]);
        now = next;
        pos.next(C::kTurns);
        a.next(C::kTurns);
        d.next(C::kTurns);
      }
      skipped = (skipped + C::kTurns - job.unit_tiles() % C::kTurns) % C::kTurns;
      float sum[kMine];
#pragma unroll
      for (int t = 0; t < kMine; t += 2) unpair(acc[t / 2], sum[t], sum[t + 1]);
      if constexpr (C::kTurns > 1) {
        float *other = b.join[turn] + q * 32 + lane;
        if (late != turn)
#pragma unroll
          for (int t = 0; t < kMine; ++t) other[t * kCodeRows] = sum[t];
        asm volatile("bar.sync 2, %0;" ::"n"(128 * C::kTurns) : "memory");
        if (late == turn)
#pragma unroll
          for (int t = 0; t < kMine; ++t) sum[t] += other[t * kCodeRows];
      }
      if (C::kTurns == 1 || late == turn) job.finish(unit, q * 32 + lane, turn, 3 + (C::kHalf > 1 ? set : turn), t_first, sum);
      turn ^= 1;
      job.next_row(row, unit);
    }
  }
  // Copies still in flight after an abort land before the CTA may leave (bounded; otherwise each has landed).
  tc_fence_before();
  __syncthreads();
  if (b.abort_flag && threadIdx.x == 0) {
    int no_abort = 0;
    for (int s = 0; s < S; ++s) {
      const int n = b.issued / S + (s < b.issued % S ? 1 : 0);
      if (n > 0) (void)wait_bounded(&b.full[s], (uint32_t)((n - 1) & 1), &no_abort, w.status, w.ns);
    }
  }
}

// bytes of memory into the L2
__device__ __forceinline__ void fetch_lines(const void *at, int bytes) {
  for (int i = 0; i < bytes; i += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char *>(at) + i));
}

// before the pipeline, by every thread
template <typename C>
__device__ __forceinline__ void code_setup(CodeBars<C> &b) {
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&b.full[s], 1);
      mbar_init(&b.empty[s], 4 + 4 * C::kHalf);  // the warps that made its operand, and that joined its groups after the products
    }
    for (int s = 0; s < C::kA; ++s) {
      mbar_init(&b.afull[s], 4);
      mbar_init(&b.aempty[s], 4 * C::kHalf);
    }
    for (int s = 0; s < C::kD; ++s) {
      mbar_init(&b.dfull[s], 1);
      mbar_init(&b.dempty[s], 4 * C::kHalf);
    }
    for (int s = 0; s < 2; ++s) mbar_init(&b.mma_done[s], 1);
    mbar_init(&b.never, 1);
    b.abort_flag = 0;
    b.issued = 0;
    fence_mbar_init();
  }
  if (threadIdx.x >> 5 == 1) tmem_alloc(&b.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}
template <typename C>
__device__ __forceinline__ void code_end(CodeBars<C> &b) {
  __syncthreads();
  if (threadIdx.x >> 5 == 1) {
    tc_fence_after();
    tmem_dealloc(b.tmem, 512);
  }
}

// Launches clusters of `ctas` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_code_clusters(void (*kernel)(KArgs...), size_t smem, std::atomic<unsigned long long> &done, dim3 grid, int threads,
                                 int ctas, cudaStream_t st, const Args &...args) {
  const cudaError_t e = allow_smem((const void *)kernel, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)ctas, 1u, 1u};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace moe
