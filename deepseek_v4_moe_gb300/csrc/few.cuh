// What the kernels for a few rows share (sm_103a): strips of 16 rows of a weight matrix streamed through a warp and
// multiplied with up to 32 tokens.
//
// The weights are the left operand of mma.m16n8k16, the tokens its eight columns: a few tokens cost the tensor cores as
// much as one, the sums are f32, and the work left to the CUDA cores is the 4-bit weights' conversion.  (tcgen05 wants its
// left operand of 128 rows in shared or tensor memory: 4-bit weights would have to be written there in 16 bits, four
// times the bytes that come from memory, and read again.)
//
// TMA brings 64 bytes of each of a strip's rows (32 columns in 16 bits, 128 in 4), into a ring that each warp has for
// itself: no barrier is met in the loop, and one instruction takes the place of a lane's address arithmetic (with
// cp.async and the addresses in every lane 16 tokens by 129280 x 4096 took 165 us, at 1.6 instructions a cycle).
// What the weights are multiplied with comes through the L1.
// The order of k within a tile is free as long as both operands have the same one: lane 4 g + t of a warp holds columns
// 32 c + 8 t .. + 7 of row g (and g + 8), as one 16-byte read of x gives them for token g.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "dense_tc.cuh"
#include "dense_vec.cuh"
#include "few.h"

namespace moe {

constexpr int kFewWarps = 8;
constexpr int kBoxBytes = 16 * 64;       // 64 bytes of each of a strip's rows
constexpr int kPartFloats = 8 * 20;      // a strip's sums with 8 tokens, rows of 16 padded to 20 against conflicts

// boxes of a strip in a tile, and a tile's columns
template <int BITS>
constexpr int kBoxes = BITS == 16 ? 2 : 1;
template <int BITS>
constexpr int kTileK = kBoxes<BITS> * 512 / BITS;

template <typename T, bool ZERO>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  // ZERO: d is not read
  const float c0 = ZERO ? 0.f : d[0], c1 = ZERO ? 0.f : d[1], c2 = ZERO ? 0.f : d[2], c3 = ZERO ? 0.f : d[3];
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Pairs of code - zero in T from a word's codes: nibbles i and i + 4, for i = 0 .. 3.  A code in the low mantissa bits of
// 128 (bf16) or 1024 (f16) is that number plus the code; the difference to the same number plus the zero point is exact.
// f16 has mantissa bits for a code four places up as well, which is sixteen times the code: (1024 + 16 c) / 16 - (64 + z)
// in one multiply-add, so that two of three shifts are saved.
template <typename T>
struct Zero {
  uint32_t a, b;  // what is subtracted from codes in the low bits, and from codes four places up
};
template <typename T>
__device__ __forceinline__ Zero<T> zero_of(uint32_t z) {
  if constexpr (std::is_same<T, __half>::value)
    return Zero<T>{(0x6400u | z) * 0x10001u, (0xD400u | z << 4) * 0x10001u};  // 1024 + z, -(64 + z)
  else
    return Zero<T>{(0x4300u | z) * 0x10001u, 0u};  // 128 + z
}
__device__ __forceinline__ uint32_t lop_and_or(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t p;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(p) : "r"(w), "r"(mask), "r"(magic));
  return p;
}
template <typename T>
__device__ __forceinline__ void widen_codes(uint32_t w, const Zero<T> &z, uint32_t (&o)[4]) {
  if constexpr (std::is_same<T, __half>::value) {
    constexpr uint32_t kSixteenth = 0x2C002C00u;
    const uint32_t h = w >> 8;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[0]) : "r"(lop_and_or(w, 0x000F000Fu, 0x64006400u)), "r"(z.a));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[1]) : "r"(lop_and_or(w, 0x00F000F0u, 0x64006400u)), "r"(kSixteenth), "r"(z.b));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(o[2]) : "r"(lop_and_or(h, 0x000F000Fu, 0x64006400u)), "r"(z.a));
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(o[3]) : "r"(lop_and_or(h, 0x00F000F0u, 0x64006400u)), "r"(kSixteenth), "r"(z.b));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(lop_and_or(w >> (4 * i), 0x000F000Fu, 0x43004300u)), "r"(z.a));
  }
}

__device__ __forceinline__ float value16(uint32_t v, const __nv_bfloat16 *) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float value16(uint32_t v, const __half *) { return __half2float(__ushort_as_half((unsigned short)v)); }

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}

// The tokens that a lane reads the right operand of: token g of each eight, or null.
template <int NT>
struct Tokens {
  const char *row[NT];
  __device__ __forceinline__ uint4 get(int i, int k, int end) const {
    return row[i] && k < end ? *reinterpret_cast<const uint4 *>(row[i] + 2 * (long long)k) : make_uint4(0u, 0u, 0u, 0u);
  }
};

// A tile's right operand and scales in a lane's registers, and the strips' products.
template <typename T, int BITS, int M, int NT>
struct Tile;

template <typename T, int M, int NT>
struct Tile<T, 16, M, NT> {
  uint4 b[kBoxes<16>][NT];
  // x: tokens; k: first column of the tile
  __device__ __forceinline__ void fetch(const Tokens<NT> &x, int k, int end) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int c = 0; c < kBoxes<16>; ++c)
#pragma unroll
      for (int i = 0; i < NT; ++i) b[c][i] = x.get(i, k + 32 * c + 8 * t, end);
  }
  // some: bit i where eight i has tokens at all
  __device__ __forceinline__ void multiply(uint32_t place, unsigned some, float (&acc)[M][NT][4]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t at = place + g * 64 + ((t ^ (g >> 1 & 3)) << 4);
#pragma unroll
    for (int s = 0; s < M; ++s)
#pragma unroll
      for (int c = 0; c < kBoxes<16>; ++c) {
        const uint32_t box = at + (s * kBoxes<16> + c) * kBoxBytes;
        const uint4 lo = lds128(box), hi = lds128(box + 512);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (NT == 1 || some >> i & 1) {
            mma16816<T, false>(acc[s][i], lo.x, hi.x, lo.y, hi.y, b[c][i].x, b[c][i].y);
            mma16816<T, false>(acc[s][i], lo.z, hi.z, lo.w, hi.w, b[c][i].z, b[c][i].w);
          }
      }
  }
};

// A strip's scales and zero points: lane l reads row l & 15 of groups l >> 4, and + 2 (a tile has one, two or four).
struct Meta {
  const uint16_t *scales;
  const uint8_t *zeros;
  int groups;             // of a row
  __device__ __forceinline__ void at(const FewMatrix &m, long long row0, int rows_left) {
    const int lane = threadIdx.x & 31, row = lane & 15;
    const long long first = (row0 + (row < rows_left ? row : 0)) * m.groups;
    scales = m.scales + first;
    zeros = m.zeros ? m.zeros + first : nullptr;
    groups = m.groups;
  }
};

template <typename T, int M, int NT>
struct Tile<T, 4, M, NT> {
  uint4 b[4][NT];
  uint32_t scale[M][2], zero[M][2];
  __device__ __forceinline__ void fetch(const Tokens<NT> &x, int k, int end) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < NT; ++i) b[c][i] = x.get(i, k + 32 * c + 8 * t, end);
  }
  __device__ __forceinline__ void fetch_meta(const Meta (&meta)[M], int k, int shift) {
    const int lane = threadIdx.x & 31, g0 = (k >> shift) + (lane >> 4), last = meta[0].groups - 1;
#pragma unroll
    for (int s = 0; s < M; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (h == 0 || shift == 5) {
          const int g = min(g0 + 2 * h, last);
          scale[s][h] = meta[s].scales[g];
          zero[s][h] = meta[s].zeros ? meta[s].zeros[g] & 15u : 8u;
        }
  }
  __device__ __forceinline__ void order() {  // columns as the codes' pairs: 0 and 4, 1 and 5, 2 and 6, 3 and 7
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint4 v = b[c][i];
        b[c][i] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                             __byte_perm(v.y, v.w, 0x7632));
      }
  }
  __device__ __forceinline__ void multiply(uint32_t place, unsigned some, float (&acc)[M][NT][4], int shift, bool zeros) {
    const int lane = threadIdx.x & 31, g = lane >> 2, r = (lane & 7) + (lane & 8), c0 = lane >> 4;
    const T *tag = nullptr;
    const uint32_t at = place + r * 64 + ((c0 ^ (r >> 1 & 3)) << 4);
    const int per = 1 << (shift - 5);  // pieces of 32 columns in a group
    order();
#pragma unroll
    for (int s = 0; s < M; ++s) {
      uint32_t w[2][4];
      ldmatrix4(w[0], at + s * kBoxBytes);
      ldmatrix4(w[1], (at ^ 32) + s * kBoxBytes);
      Zero<T> z[2] = {zero_of<T>(8u), zero_of<T>(8u)};
      float part[NT][4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int group = c >> (shift - 5);
        if (zeros && (c & (per - 1)) == 0) {
          const uint32_t all = group < 2 ? zero[s][0] : zero[s][1];
          z[0] = zero_of<T>(__shfl_sync(0xffffffffu, all, (group & 1) * 16 + g));
          z[1] = zero_of<T>(__shfl_sync(0xffffffffu, all, (group & 1) * 16 + g + 8));
        }
        uint32_t lo[4], hi[4];
        widen_codes<T>(w[c >> 1][2 * (c & 1)], z[0], lo);
        widen_codes<T>(w[c >> 1][2 * (c & 1) + 1], z[1], hi);
        const bool begins = (c & (per - 1)) == 0;
        if (begins) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
            if (NT == 1 || some >> i & 1) mma16816<T, true>(part[i], lo[0], hi[0], lo[1], hi[1], b[c][i].x, b[c][i].y);
        } else {
#pragma unroll
          for (int i = 0; i < NT; ++i)
            if (NT == 1 || some >> i & 1) mma16816<T, false>(part[i], lo[0], hi[0], lo[1], hi[1], b[c][i].x, b[c][i].y);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (NT == 1 || some >> i & 1) mma16816<T, false>(part[i], lo[2], hi[2], lo[3], hi[3], b[c][i].z, b[c][i].w);
        if ((c & (per - 1)) == per - 1) {  // the group ends: its sums times its scale
          const uint32_t all = group < 2 ? scale[s][0] : scale[s][1];
          const float s0 = value16(__shfl_sync(0xffffffffu, all, (group & 1) * 16 + g), tag);
          const float s1 = value16(__shfl_sync(0xffffffffu, all, (group & 1) * 16 + g + 8), tag);
#pragma unroll
          for (int i = 0; i < NT; ++i)
            if (NT == 1 || some >> i & 1) {
              acc[s][i][0] = fmaf(part[i][0], s0, acc[s][i][0]);
              acc[s][i][1] = fmaf(part[i][1], s0, acc[s][i][1]);
              acc[s][i][2] = fmaf(part[i][2], s1, acc[s][i][2]);
              acc[s][i][3] = fmaf(part[i][3], s1, acc[s][i][3]);
            }
        }
      }
    }
  }
};

// A warp's sums of a strip and eight tokens in shared memory, and element (row, token) of them.
__device__ __forceinline__ void put_part(float *part, const float (&v)[4]) {
  const int lane = threadIdx.x & 31;
  *reinterpret_cast<float4 *>(part + (lane >> 2) * 20 + (lane & 3) * 4) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ int part_at(int row, int token) {
  return (row & 7) * 20 + (token >> 1) * 4 + (row >> 3) * 2 + (token & 1);
}
__device__ __forceinline__ void warps_meet(int first, int count) {  // `count` warps from warp `first` on, a power of two
  if (count == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(1 + first / count), "r"(32 * count) : "memory");
}

// Streams a job's units, one after another, through the CTA's warps.  A unit is rows of the result with all tokens: `segs`
// matrices of `tiles` tiles, dealt to 2^log_kw warps, whose sums meet in shared memory in the warps' order: the same bits
// every run.  The CTA's 8 / 2^log_kw sets of warps take neighbouring parts of a unit.  Copies run ahead across units.
//   M strips, P of them finished together;  int units, segs, tiles
//   void load_at(unit, set, seg);  void load(place, barrier, tile)       the copies' side, M * kBoxes boxes a place
//   void use_at(unit, set, seg);   void fetch(tile);  void multiply(place, acc)
//   void finish(unit, set, strip, thread, threads, sum)                  sum(strip of P, row, token)
template <int M, int P, int NT, int STAGES, int BOXES, typename Job>
__device__ __forceinline__ void stream_units(Job &job, char *smem, int log_kw, int *status, uint64_t wait_ns, bool inject) {
  constexpr int kPlace = BOXES * kBoxBytes;
  __shared__ uint64_t full[kFewWarps][STAGES];
  __shared__ uint64_t never;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, kw = 1 << log_kw, set = warp >> log_kw, mine = warp & (kw - 1);
  char *own = smem + warp * (STAGES * kPlace);
  float *parts = reinterpret_cast<float *>(smem + kFewWarps * STAGES * kPlace);
  if (threadIdx.x < kFewWarps * STAGES) mbar_init(&full[0][0] + threadIdx.x, 1);
  if (threadIdx.x == 0) {
    mbar_init(&never, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < kFewWarps * STAGES) fence_mbar_init();
  __syncthreads();
  // a place in the job's tiles that this warp has come to
  struct Place {
    int unit, seg, tile;
  };
  auto enter = [&](Place &p) {  // past the end of a matrix: the next one that has a tile for this warp
    while (p.unit < job.units && p.tile >= job.tiles) {
      p.tile -= job.tiles;
      if (++p.seg == job.segs) {
        p.seg = 0;
        p.tile = mine;
        p.unit += gridDim.x;
        if (mine >= job.segs * job.tiles) p.unit = job.units;
      }
    }
  };
  Place ahead = {(int)blockIdx.x, 0, mine};
  if (mine >= job.segs * job.tiles) ahead.unit = job.units;
  enter(ahead);
  if (ahead.unit < job.units) job.load_at(ahead.unit, set, ahead.seg);
  int begun = 0, used = 0;  // copies
  auto copy_next = [&](int stage) {
    if (ahead.unit >= job.units) return;
    if ((threadIdx.x & 31) == 0) mbar_arrive_expect_tx(&full[warp][stage], kPlace);
    __syncwarp();
    job.load(own + stage * kPlace, &full[warp][stage], ahead.tile);
    ++begun;
    ahead.tile += kw;
    if (ahead.tile >= job.tiles) {
      enter(ahead);
      if (ahead.unit < job.units) job.load_at(ahead.unit, set, ahead.seg);
    }
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s) copy_next(s);
  job.copies_begun();
  if (inject && blockIdx.x == 0) wait_bounded(&never, 0, &abort_flag, status, wait_ns);  // test hook: a wait that runs out
  int stage = 0, phase = 0;
  for (int unit = blockIdx.x; unit < job.units; unit += gridDim.x) {
    float acc[M][NT][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
    int tile = mine;
    for (int seg = 0; seg < job.segs; ++seg, tile -= job.tiles) {
      if (tile >= job.tiles) continue;
      job.use_at(unit, set, seg);
      for (; tile < job.tiles; tile += kw) {
        job.fetch(tile);
        // (the lanes agree: one that gave up takes the warp with it)
        if (!__all_sync(0xffffffffu, wait_bounded(&full[warp][stage], phase, &abort_flag, status, wait_ns))) continue;
        job.multiply(smem_u32(own) + stage * kPlace, acc);
        __syncwarp();
        ++used;
        copy_next(stage);
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    float *sums = parts + set * kw * (P * NT * kPartFloats);
#pragma unroll
    for (int m = 0; m < M; m += P) {
#pragma unroll
      for (int q = 0; q < P; ++q)
#pragma unroll
        for (int i = 0; i < NT; ++i) put_part(sums + ((mine * P + q) * NT + i) * kPartFloats, acc[m + q][i]);
      warps_meet(set * kw, kw);
      job.finish(unit, set, m, threadIdx.x & (32 * kw - 1), 32 * kw, [&](int q, int row, int token) {
        const float *at = sums + (q * NT + (token >> 3)) * kPartFloats + part_at(row, token & 7);
        float v = at[0];
        for (int w = 1; w < kw; ++w) v += at[w * (P * NT * kPartFloats)];
        return v;
      });
      warps_meet(set * kw, kw);
    }
  }
  // after a wait that ran out: no copy may land in memory that the CTA has left
  for (int nobody = 0; used < begun; ++used) {
    mbar_wait_bounded(&full[warp][stage], phase, &nobody, status, wait_ns);
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1;
    }
  }
}

}  // namespace moe
