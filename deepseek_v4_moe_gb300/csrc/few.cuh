// What the kernels for a few rows share (sm_103a): strips of 16 rows of a weight matrix streamed through a warp and
// multiplied with up to 32 tokens.
//
// The weights are the left operand of mma.m16n8k16, the tokens its eight columns: a few tokens cost the tensor cores as
// much as one, the sums are f32, and the work left to the CUDA cores is the 4-bit weights' conversion.  (tcgen05 wants its
// left operand of 128 rows in shared or tensor memory: 4-bit weights would have to be written there in 16 bits, four
// times the bytes that come from memory, and read again.)
//
// A warp copies 128 bytes of each of its rows at a time (cp.async, a ring of its own, so no barrier is met in the loop):
// 64 columns of 16-bit weights, 256 of 4-bit ones.  What the tokens are multiplied with comes from the L1.
// The order of k within a tile is free as long as both operands have the same one: lane 4 g + t of a warp holds columns
// 32 c + 8 t .. + 7 of row g (and g + 8), as one 16-byte read of x gives them for token g.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "dense_tc.cuh"
#include "dense_vec.cuh"
#include "few.h"

namespace moe {

constexpr int kFewWarps = 8;
constexpr int kStripBytes = 16 * 128;
constexpr int kMetaPitch = 32;           // a row's scales and zero points of a tile: 20 and 12 bytes
constexpr int kPartFloats = 8 * 20;      // a strip's sums with 8 tokens, rows of 16 padded to 20 against conflicts

template <int BITS>
constexpr int kTileK = 1024 / BITS;
// bytes of a ring's place: M strips, and with 4 bits their scales
template <int BITS, int M>
constexpr int kPlaceBytes = M * (kStripBytes + (BITS == 4 ? 16 * kMetaPitch : 0));

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The 16-byte piece of a row's 128 that piece c lies in: both ways of reading, 8 rows of one piece and 2 rows of 4
// neighbouring pieces, then touch every bank once.
__device__ __forceinline__ int swizzle(int row, int c) { return c ^ ((row & 1) << 2 | (row >> 1 & 3)); }

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Pairs of code - zero in T from the codes at bits 0 and 16 of w (nibbles i and i + 4 of a word shifted by 4 i): a code in
// the low mantissa bits of 128 (bf16) or 1024 (f16) is that number plus the code, and the difference is exact.
template <typename T>
constexpr uint32_t kMagic = 0x43004300u;
template <>
constexpr uint32_t kMagic<__half> = 0x64006400u;
template <typename T>
__device__ __forceinline__ uint32_t minus2(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 2) {
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value)
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
      asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
}
template <typename T>
__device__ __forceinline__ uint32_t code_pair4(uint32_t w, uint32_t offset) {
  uint32_t p;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(p) : "r"(w), "n"(0x000F000F), "n"(kMagic<T>));  // (w & mask) | magic
  return minus2<T>(p, offset);
}

__device__ __forceinline__ float value16(uint16_t v, const __nv_bfloat16 *) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float value16(uint16_t v, const __half *) {
  return __half2float(*reinterpret_cast<const __half *>(&v));
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Copies tile `tile` of the strip of rows row0 .. row0 + 15 of matrix m (its number `e` where there are several): what
// lies past its ends as zeros.  The whole warp.
template <int BITS>
__device__ __forceinline__ void copy_strip(uint32_t dst, const FewMatrix &m, int e, int row0, int tile) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  const long long row_bytes = (long long)m.k * BITS / 8;
  const int at = tile * 128 + c * 16, left = m.n - row0;
  const char *src = static_cast<const char *>(m.w) + ((long long)e * m.n + row0) * row_bytes + at;
  const bool in = at < row_bytes;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * i + (lane >> 3);
    const bool ok = in && r < left;
    cp_async16(dst + r * 128 + swizzle(r, c) * 16, ok ? src + r * row_bytes : m.w, ok ? 16 : 0);
  }
}
// its scales and zero points, each row's at dst + 32 row, as the aligned words that hold them: scales from byte 0,
// zero points from byte 20.  Words past the matrix's end are cut where it ends.
__device__ __forceinline__ void copy_meta(uint32_t dst, const FewMatrix &m, int e, int row0, int tile, int row) {
  const int g0 = (tile * 256) >> m.group_shift, g1 = min((tile * 256 + 256) >> m.group_shift, m.groups);
  const bool in = row0 + row < m.n && g0 < g1;
  const long long first = ((long long)e * m.n + row0 + row) * m.groups;
  {
    const long long b = 2 * (first + g0), end = 2 * (first + g1);
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const long long at = (b & ~3ll) + 4 * i;
      const int bytes = in ? (int)min(4ll, max(0ll, end - at)) : 0;
      if (4 * i < (2 << (8 - m.group_shift)) + 2)
        cp_async4(dst + row * kMetaPitch + 4 * i, bytes ? reinterpret_cast<const char *>(m.scales) + at : (const void *)m.scales, bytes);
    }
  }
  if (m.zeros) {
    const long long b = first + g0, end = first + g1;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long at = (b & ~3ll) + 4 * i;
      const int bytes = in ? (int)min(4ll, max(0ll, end - at)) : 0;
      if (4 * i < (1 << (8 - m.group_shift)) + 3)
        cp_async4(dst + row * kMetaPitch + 20 + 4 * i, bytes ? reinterpret_cast<const char *>(m.zeros) + at : (const void *)m.zeros, bytes);
    }
  }
}

// eight values of token column's x at column k, zeros where there are none
template <int NT>
struct Tokens {
  const char *row[NT];  // the lane's token of each eight, or null
  __device__ __forceinline__ uint4 get(int i, int k, int end) const {
    return row[i] && k < end ? *reinterpret_cast<const uint4 *>(row[i] + 2 * (long long)k) : make_uint4(0u, 0u, 0u, 0u);
  }
};

// Adds a tile's products to acc[strip][eight tokens].  `some`: bit i where eight i has tokens at all.
template <typename T, int BITS, int M, int NT>
__device__ __forceinline__ void multiply_tile(uint32_t place, const FewMatrix (&m)[M], const int (&e)[M], const int (&row0)[M], int tile,
                                              const Tokens<NT> &x, unsigned some, float (&acc)[M][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int k0 = tile * kTileK<BITS>, end = m[0].k;
  if constexpr (BITS == 16) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint4 b[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) b[i] = x.get(i, k0 + 32 * c + 8 * t, end);
#pragma unroll
      for (int s = 0; s < M; ++s) {
        const uint32_t at = place + s * kStripBytes + swizzle(g, 4 * c + t) * 16;
        const uint4 lo = lds128(at + g * 128), hi = lds128(at + (g + 8) * 128);
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (NT == 1 || some >> i & 1) {
            mma16816<T>(acc[s][i], lo.x, hi.x, lo.y, hi.y, b[i].x, b[i].y);
            mma16816<T>(acc[s][i], lo.z, hi.z, lo.w, hi.w, b[i].z, b[i].w);
          }
      }
    }
  } else {
    const T *tag = nullptr;
    const int shift = m[0].group_shift, per = 1 << (shift - 5);  // pieces of 32 columns in a group
    // where in the copied words this row's scales begin
    uint32_t sc[M][2], ze[M][2];
#pragma unroll
    for (int s = 0; s < M; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = g + 8 * h;
        // (its last two bits, so 32 of them are enough)
        const uint32_t first = ((uint32_t)e[s] * m[s].n + row0[s] + row) * m[s].groups + ((tile * 256) >> shift);
        const uint32_t base = place + M * kStripBytes + (s * 16 + row) * kMetaPitch;
        sc[s][h] = base + 2 * (first & 1);
        ze[s][h] = base + 20 + (first & 3);
      }
    float part[M][NT][4];
#pragma unroll
    for (int s = 0; s < M; ++s)
#pragma unroll
      for (int i = 0; i < NT; ++i) part[s][i][0] = part[s][i][1] = part[s][i][2] = part[s][i][3] = 0.f;
    uint32_t zero[M][2];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (k0 + 32 * c >= end) break;
      const int group = c >> (shift - 5);
      if ((c & (per - 1)) == 0) {
#pragma unroll
        for (int s = 0; s < M; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t z = m[s].zeros ? lds_u8(ze[s][h] + group) & 15u : 8u;
            zero[s][h] = kMagic<T> | z | z << 16;
          }
      }
      uint4 b[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint4 v = x.get(i, k0 + 32 * c + 8 * t, end);
        // in the order of the codes' pairs: columns 0 and 4, 1 and 5, 2 and 6, 3 and 7
        b[i] = make_uint4(__byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                          __byte_perm(v.y, v.w, 0x7632));
      }
#pragma unroll
      for (int s = 0; s < M; ++s) {
        const uint32_t at = place + s * kStripBytes + swizzle(g, c) * 16 + 4 * t;
        uint32_t lo, hi;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(lo) : "r"(at + g * 128));
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(hi) : "r"(at + (g + 8) * 128));
        uint32_t a[2][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          a[0][j] = code_pair4<T>(lo >> (4 * j), zero[s][0]);
          a[1][j] = code_pair4<T>(hi >> (4 * j), zero[s][1]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i)
          if (NT == 1 || some >> i & 1) {
            mma16816<T>(part[s][i], a[0][0], a[1][0], a[0][1], a[1][1], b[i].x, b[i].y);
            mma16816<T>(part[s][i], a[0][2], a[1][2], a[0][3], a[1][3], b[i].z, b[i].w);
          }
      }
      if ((c & (per - 1)) == per - 1 || k0 + 32 * (c + 1) >= end) {  // the group ends: its sums times its scale
#pragma unroll
        for (int s = 0; s < M; ++s) {
          const float s0 = value16((uint16_t)lds_u16(sc[s][0] + 2 * group), tag), s1 = value16((uint16_t)lds_u16(sc[s][1] + 2 * group), tag);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            acc[s][i][0] = fmaf(part[s][i][0], s0, acc[s][i][0]);
            acc[s][i][1] = fmaf(part[s][i][1], s0, acc[s][i][1]);
            acc[s][i][2] = fmaf(part[s][i][2], s1, acc[s][i][2]);
            acc[s][i][3] = fmaf(part[s][i][3], s1, acc[s][i][3]);
            part[s][i][0] = part[s][i][1] = part[s][i][2] = part[s][i][3] = 0.f;
          }
        }
      }
    }
  }
}

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

// Streams a job's units, one after another, through the CTA's warps.  A unit is rows of the result with all tokens; its
// tiles are dealt to 2^log_kw warps, whose sums meet in shared memory in the warps' order: the same bits every run.
// The CTA's 8 / 2^log_kw sets of warps take neighbouring parts of a unit.  Copies run ahead across units.
//   int units, tiles;
//   void copy(uint32_t place, int unit, int set, int tile)
//   void multiply(uint32_t place, int unit, int set, int tile, float (&acc)[M][NT][4])
//   void finish(int unit, int set, int thread, int threads, sum)   sum(strip, row, token)
template <int M, int NT, int STAGES, int PLACE, typename Job>
__device__ __forceinline__ void stream_units(Job &job, uint32_t ring, float *parts, int log_kw) {
  const int warp = threadIdx.x >> 5, kw = 1 << log_kw, set = warp >> log_kw, mine = warp & (kw - 1);
  const uint32_t own = ring + warp * (STAGES * PLACE);
  int unit_ahead = mine < job.tiles ? blockIdx.x : job.units, tile_ahead = mine;
  auto copy_next = [&](int stage) {
    if (unit_ahead < job.units) {
      job.copy(own + stage * PLACE, unit_ahead, set, tile_ahead);
      tile_ahead += kw;
      if (tile_ahead >= job.tiles) {
        tile_ahead = mine;
        unit_ahead += gridDim.x;
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES; ++s) copy_next(s);
  job.copies_begun();
  int stage = 0;
  for (int unit = blockIdx.x; unit < job.units; unit += gridDim.x) {
    float acc[M][NT][4];
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[m][i][0] = acc[m][i][1] = acc[m][i][2] = acc[m][i][3] = 0.f;
    for (int tile = mine; tile < job.tiles; tile += kw) {
      cp_wait<STAGES - 1>();
      __syncwarp();
      job.multiply(own + stage * PLACE, unit, set, tile, acc);
      __syncwarp();
      copy_next(stage);
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int i = 0; i < NT; ++i) put_part(parts + ((warp * M + m) * NT + i) * kPartFloats, acc[m][i]);
    warps_meet(set * kw, kw);
    const float *sums = parts + set * kw * (M * NT * kPartFloats);
    job.finish(unit, set, threadIdx.x & (32 * kw - 1), 32 * kw, [&](int m, int row, int token) {
      const float *at = sums + (m * NT + (token >> 3)) * kPartFloats + part_at(row, token & 7);
      float v = at[0];
      for (int w = 1; w < kw; ++w) v += at[w * (M * NT * kPartFloats)];
      return v;
    });
    warps_meet(set * kw, kw);
  }
  cp_wait<0>();
}

}  // namespace moe
