// 4-bit weights on mma.sync (sm_103a): strips of 16 rows of the matrix streamed through a warp and multiplied with up to
// 32 tokens.
//
// The weights are the left operand of mma.m16n8k16, the tokens its eight columns: a few tokens cost the tensor cores as
// much as one, the sums are f32, and the work left to the CUDA cores is the codes' conversion to 16 bits, in registers.
// It takes x as it is, so that a product is one launch; where the conversion bounds it, few_tc.cuh's form is faster.
//
// TMA brings 64 bytes (128 columns) of each of a strip's rows into a ring, and the tokens' columns beside them: with the
// addresses in every lane 16 tokens by 129280 x 4096 took 165 us at 1.6 instructions a cycle, and with the tokens read through
// the L1 their latency stopped the warps.
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

constexpr int kTileK = 128;              // columns of a tile: a box

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
// 128 (bf16) or 1024 (f16) is that number plus the code; the difference to the same number plus the zero point is exact
// (widening codes so, without conversions: Y. J. Kim, R. Henry, R. Fahim and H. H. Awadalla, "Who Says Elephants Can't Run:
// Bringing Large Scale MoE Models into Cloud Scale Production", 2022).
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

// The right operand of a tile in shared memory: pieces of 32 columns, each `rows` tokens' 64 bytes one after another, in
// the same swizzle as the weights.  A lane's 16 bytes of a piece for its token of eight i.  ROWS8: rows is a multiple of
// 8, so that a piece is that many bytes from the one before.
template <int PIECES, bool ROWS8>
struct Operand {
  uint32_t at[ROWS8 ? 1 : PIECES];
  uint32_t pitch;  // of a piece
  // first: the tile's first line (of 64 bytes, from an address that is a multiple of 512)
  __device__ __forceinline__ void set(int first, int rows) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pitch = rows * 64;
#pragma unroll
    for (int c = 0; c < (ROWS8 ? 1 : PIECES); ++c) {
      const int line = first + c * rows + min(g, rows - 1);  // (a token that is none reads another's: nobody reads its sums)
      at[c] = line * 64 + ((t ^ (line >> 1 & 3)) << 4);
    }
  }
  __device__ __forceinline__ uint4 get(uint32_t base, int c, int i) const {
    return ROWS8 ? lds128(base + at[0] + c * pitch + i * 512) : lds128(base + at[c % (ROWS8 ? 1 : PIECES)]);
  }
};

// A strip's scales and zero points of a tile.  Lane l reads row l & 15; groups l >> 4 of the tile, and + 2 where it has
// four; where it has one, lanes from 16 on read that of this warp's next tile, and every other tile reads nothing.
// They are read one reading ahead of their use.
struct MetaRow {
  const uint16_t *scales;
  const uint8_t *zeros;
  __device__ __forceinline__ void at(const FewMatrix &m, long long row0, int rows_left) {
    const int row = threadIdx.x & 15;
    const long long first = (row0 + (row < rows_left ? row : 0)) * m.groups;
    scales = m.scales + first;
    zeros = m.zeros + first;  // (read with zero points only)
  }
};
template <int PIECES, int M, bool ZP>
struct Meta {
  static constexpr int kGroups = 4 / PIECES, kEach = kGroups == 4 ? 2 : 1;
  MetaRow row[M];
  uint32_t now[M][kEach], next[M][kEach];  // scale in the low half, zero point in the high
  int half, step, groups;                  // half: 16 in the tile that finds its scales read
  __device__ __forceinline__ void read(int tile) {
    const int lane = threadIdx.x & 31, g0 = kGroups == 1 ? tile + (lane >> 4) * step : tile * kGroups + (lane >> 4);
#pragma unroll
    for (int h = 0; h < kEach; ++h) {
      const int g = min(g0 + 2 * h, groups - 1);
#pragma unroll
      for (int s = 0; s < M; ++s) next[s][h] = row[s].scales[g] | (ZP ? (row[s].zeros[g] & 15u) << 16 : 0u);
    }
  }
  // from a warp's first tile of a matrix on; its rows are set
  __device__ __forceinline__ void begin(int tile, int step_, int groups_) {
    step = step_;
    groups = groups_;
    half = 16;
    read(tile);
  }
  __device__ __forceinline__ void advance(int tile) {
    if constexpr (kGroups == 1) {
      half ^= 16;
      if (half) return;
    }
#pragma unroll
    for (int s = 0; s < M; ++s)
#pragma unroll
      for (int h = 0; h < kEach; ++h) now[s][h] = next[s][h];
    read(tile + (kGroups == 1 ? 2 * step : step));  // (past the end: the last group's again)
  }
  // what row g, and g + 8 for eight = 8, of strip s has in group q
  __device__ __forceinline__ uint32_t get(int s, int q, int eight) const {
    return __shfl_sync(0xffffffffu, now[s][q / 2 % kEach], (kGroups == 1 ? half : (q & 1) * 16) + ((threadIdx.x & 31) >> 2) + eight);
  }
};

// columns in the order of the codes' pairs: 0 and 4, 1 and 5, 2 and 6, 3 and 7
__device__ __forceinline__ uint4 in_pairs(const uint4 v) {
  return make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                    __byte_perm(v.y, v.w, 0x7632));
}

// The products of a tile's strips.  PIECES: of 32 columns in a group, and ZP: there are zero points, at compile time, so
// that a tile's products are one run of instructions in which the strips overlap.
template <typename T, int PIECES, bool ZP, int M, int NT, bool ROWS8>
struct Tile {
  static constexpr int kGroups = 4 / PIECES;
  Operand<4, ROWS8> x;
  Meta<PIECES, M, ZP> meta;
  __device__ __forceinline__ void multiply(uint32_t place, uint32_t tokens, float (&acc)[M][NT][4]) const {
    const int lane = threadIdx.x & 31, r = lane & 15, c0 = lane >> 4;
    const T *tag = nullptr;
    const uint32_t at = place + r * 64 + ((c0 ^ (r >> 1 & 3)) << 4);
    uint32_t w[M][4];
#pragma unroll
    for (int q = 0; q < kGroups; ++q) {
      float part[M][NT][4];
      uint32_t m0[M], m1[M];
      Zero<T> z0[M], z1[M];
#pragma unroll
      for (int s = 0; s < M; ++s) {
        m0[s] = meta.get(s, q, 0);
        m1[s] = meta.get(s, q, 8);
        z0[s] = zero_of<T>(ZP ? m0[s] >> 16 : 8u);
        z1[s] = zero_of<T>(ZP ? m1[s] >> 16 : 8u);
      }
#pragma unroll
      for (int j = 0; j < PIECES; ++j) {
        const int c = q * PIECES + j;
        uint4 b[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) b[i] = in_pairs(x.get(tokens, c, i));
#pragma unroll
        for (int s = 0; s < M; ++s) {
          if (c == 0) ldmatrix4(w[s], at + s * kBoxBytes);
          if (c == 2) ldmatrix4(w[s], (at ^ 32) + s * kBoxBytes);
          uint32_t lo[4], hi[4];
          widen_codes<T>(w[s][2 * (c & 1)], z0[s], lo);
          widen_codes<T>(w[s][2 * (c & 1) + 1], z1[s], hi);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            if (j == 0) mma16816<T, true>(part[s][i], lo[0], hi[0], lo[1], hi[1], b[i].x, b[i].y);
            else mma16816<T, false>(part[s][i], lo[0], hi[0], lo[1], hi[1], b[i].x, b[i].y);
            mma16816<T, false>(part[s][i], lo[2], hi[2], lo[3], hi[3], b[i].z, b[i].w);
          }
        }
      }
      // the groups' sums times their scales
#pragma unroll
      for (int s = 0; s < M; ++s) {
        const float s0 = value16(m0[s], tag), s1 = value16(m1[s], tag);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          acc[s][i][0] = fmaf(part[s][i][0], s0, acc[s][i][0]);
          acc[s][i][1] = fmaf(part[s][i][1], s0, acc[s][i][1]);
          acc[s][i][2] = fmaf(part[s][i][2], s1, acc[s][i][2]);
          acc[s][i][3] = fmaf(part[s][i][3], s1, acc[s][i][3]);
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

}  // namespace moe
