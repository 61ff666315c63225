// Matrix products of the gated feed-forward block, forward and backward, on the 5th-generation tensor
// cores (tcgen05, TMEM, TMA), sm_103a.
//
//   forward    g = x Wg^T, u = x Wu^T, h = act(g) u                        kGateUp
//              y = h Wd^T                                                  kDown
//   backward   dh = dy Wd;  dg = dh u act'(g), du = dh act(g), h again     kHiddenGrad
//              dx = dg Wg + du Wu;  dWg = dg^T x, dWu = du^T x, dWd = dy^T h     kGrads
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
//   warp 1     TMEM allocator and MMA issuer
//   warps 2-9  epilogue: two warps for each TMEM lane quarter, each every other 32 columns; the
//              accumulator is double buffered, so the next tile's MMAs run under it
// kGateUp makes BN / 2 columns of g and the same of u side by side in one accumulator, so the
// activation and the product need no second pass.  kGrads runs up to four products in one launch: its
// tiles are those of one after another, whose A is K-major (dx) or MN-major (the weights' gradients).
// Every wait is bounded; on expiry the CTA sets the device timeout bit, all roles leave, copies and
// MMAs in flight are waited for (bounded) and TMEM is freed.
#include <algorithm>

#include "common.cuh"
#include "dense.h"
#include "dense_tc.cuh"
#include "dense_vec.cuh"

namespace moe {
namespace {

constexpr int kBK = 64;
constexpr int kABytes = kBM * kBK * 2;

// How the CTAs of a cluster share a tile: not at all; a pair makes 256 rows of it (cta_group::2); or each
// takes a part of k, for few tiles with a long k.
template <int MODE, int BN, int KIND>
struct Cfg {
  static constexpr bool PAIR = KIND == kPairTile, SPLIT = KIND == kSplitTile;
  static constexpr bool kBMn = MODE == kHiddenGrad || MODE == kGrads;
  // rows of B in this CTA; an MN-major operand comes in whole boxes of 64, of which the last may be used in part
  static constexpr int kBUsed = PAIR ? BN / 2 : BN, kBRows = kBMn ? (kBUsed + 63) / 64 * 64 : kBUsed;
  static constexpr int kStage = kABytes + kBRows * kBK * 2;
  static constexpr int kBufBytes = kEpiWarps * kStageBuf;
  // what the other CTAs send of this CTA's rows: at most (kSplitMax - 1) parts of a lane quarter's rows
  static constexpr int kPartBytes = SPLIT ? (kSplitMax - 1) * 32 * BN * 4 : 0;
  static constexpr int kStages = (kRingBytes - kBufBytes - kPartBytes) / kStage;
  static constexpr size_t kSmem = (size_t)kStages * kStage + kBufBytes + kPartBytes + 1024;
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
  int prob, m0, n0;  // problem, first row, first column (kGateUp: of g and of u)
};

template <int MODE>
__device__ __forceinline__ Tile tile_of(const GemmParams &p, int t, int rows, int cols) {
  Tile r;
  r.prob = 0;
  if constexpr (MODE == kGrads) {
    int begin = 0;
    while (t >= p.problem[r.prob].end) begin = p.problem[r.prob++].end;
    t -= begin;
  }
  band_tile(t, p.problem[r.prob].tiles_m, p.problem[r.prob].tiles_n, r.m0, r.n0);
  r.m0 *= rows;
  r.n0 *= cols;
  return r;
}

// A warp's 32 rows of a tile: its columns [32 * half, kCols) in steps of 64, 32 at a time.  A thread of
// the TMEM loads has a row; rows lie far apart in memory, so what is stored (and kHiddenGrad's g and u)
// passes through shared memory, and four neighbouring threads move the 64 bytes of a row: a store that
// took 32 lines takes 8.  begin() runs while the tile's products are still made: it fetches g and u of
// the first step; each step then fetches the next one's.  The loop is kept rolled: unrolled, its code no
// longer fits the instruction caches and a tile of 256 columns took 15 us more.
template <int MODE, int BN, typename T>
struct Epilogue {
  static constexpr int kCols = MODE == kGateUp ? BN / 2 : BN;
  uint4 g[4], u[4];  // kHiddenGrad: the next step's, as they are fetched
  int row0, m, n, half;
  uint32_t buf;      // the warp's staging buffer
  uint32_t parts;    // the other CTAs' sums of this warp's rows, p.splits - 1 times 32 rows x BN
  Tile tl;
  // thread l moves piece l % 4 of rows l / 4 + 8 i
  __device__ __forceinline__ bool mine(int i, int c0, size_t ld, size_t &at) const {
    const int lane = threadIdx.x & 31, row = row0 + 8 * i + (lane >> 2), c = c0 + 8 * (lane & 3);
    at = (size_t)row * ld + tl.n0 + c;
    return row < m && c < kCols && tl.n0 + c < n;
  }
  __device__ __forceinline__ void fetch(const GemmParams &p, int c0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      size_t at;
      g[i] = u[i] = make_uint4(0u, 0u, 0u, 0u);
      if (mine(i, c0, n, at)) {
        g[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.e[0]) + at);
        u[i] = *reinterpret_cast<const uint4 *>(static_cast<const T *>(p.e[1]) + at);
      }
    }
  }
  __device__ __forceinline__ void begin(const GemmParams &p, const Tile &tile, int half_, int row0_, uint32_t buf_) {
    tl = tile;
    row0 = row0_;
    half = half_;
    buf = buf_;
    m = p.problem[tl.prob].m;
    n = p.problem[tl.prob].n;
    if constexpr (MODE == kHiddenGrad) fetch(p, half * 32);
  }
  // sixteen values as eight words of pairs
  static __device__ __forceinline__ void pack16(const float (&v)[16], uint32_t *w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack2<T>(v[2 * i], v[2 * i + 1]);
  }
  static __device__ __forceinline__ void unpack16(const uint32_t *w, float (&v)[16]) {
    const T *tag = nullptr;
#pragma unroll
    for (int i = 0; i < 8; ++i) unpack2(w[i], v[2 * i], v[2 * i + 1], tag);
  }
  // what fetch() brought, handed to the threads that have the rows
  __device__ __forceinline__ void hand_over(const uint4 (&f)[4], uint32_t (&w)[16]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < 4; ++i) sts128(buf + piece_at(8 * i + (lane >> 2), lane & 3), f[i]);
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 q = lds128(buf + piece_at(lane, c));
      w[4 * c] = q.x, w[4 * c + 1] = q.y, w[4 * c + 2] = q.z, w[4 * c + 3] = q.w;
    }
    __syncwarp();
  }
  // each thread's 32 values of its row to `out`
  __device__ __forceinline__ void emit(const uint32_t (&w)[16], void *out, size_t ld, int c0) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int c = 0; c < 4; ++c) sts128(buf + piece_at(lane, c), make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      size_t at;
      if (mine(i, c0, ld, at))
        *reinterpret_cast<uint4 *>(static_cast<T *>(out) + at) = lds128(buf + piece_at(8 * i + (lane >> 2), lane & 3));
    }
    __syncwarp();
  }
  // sixteen columns of the accumulator, with the other CTAs' parts added in order
  template <bool SPLIT>
  __device__ __forceinline__ void take(const GemmParams &p, uint32_t tbase, int col, float (&v)[16]) const {
    tmem_ld16(tbase + col, v);
    if constexpr (SPLIT)
      for (int s = 0; s < p.splits - 1; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = lds128(parts + part_at(s, col / 4 + i));
          v[4 * i] += __uint_as_float(w.x);
          v[4 * i + 1] += __uint_as_float(w.y);
          v[4 * i + 2] += __uint_as_float(w.z);
          v[4 * i + 3] += __uint_as_float(w.w);
        }
  }
  // four columns of this lane's row in part s
  static __device__ __forceinline__ uint32_t part_at(int s, int four) {
    return ((s * (BN / 4) + four) * 32 + (threadIdx.x & 31)) * 16;
  }
  template <bool SPLIT>
  __device__ __forceinline__ void finish(const GemmParams &p, uint32_t tbase) {
#pragma unroll 1
    for (int c0 = half * 32; c0 < kCols; c0 += 64) {
      uint32_t x[16], y[16], z[16];
      if constexpr (MODE == kHiddenGrad) {
        hand_over(g, x);
        hand_over(u, y);
        fetch(p, c0 + 64);
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (c0 + 16 * s >= kCols) break;  // TMEM ends here (the words left over are not stored)
        float v[16], w[16];
        take<SPLIT>(p, tbase, c0 + 16 * s, v);
        if constexpr (MODE == kGateUp) {
          take<SPLIT>(p, tbase, BN / 2 + c0 + 16 * s, w);
          pack16(v, y + 8 * s);
          pack16(w, z + 8 * s);
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = act_value(p.act, v[j]) * w[j];
          pack16(v, x + 8 * s);
        } else if constexpr (MODE == kHiddenGrad) {
          float a[16], b[16];
          unpack16(x + 8 * s, a);
          unpack16(y + 8 * s, b);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float act, slope;
            act_both(p.act, a[j], act, slope);
            a[j] = v[j] * b[j] * slope;  // dg
            w[j] = act * b[j];           // h
            v[j] *= act;                 // du
          }
          pack16(a, x + 8 * s);
          pack16(v, y + 8 * s);
          pack16(w, z + 8 * s);
        } else {
          pack16(v, x + 8 * s);
        }
      }
      if constexpr (MODE == kGateUp || MODE == kHiddenGrad) {
        emit(x, p.out[0], n, c0);
        if (p.out[1]) {
          emit(y, p.out[1], n, c0);
          emit(z, p.out[2], n, c0);
        }
      } else {
        emit(x, p.problem[tl.prob].c, p.problem[tl.prob].ldc, c0);
      }
    }
  }
};

// the epilogue warps' loop over the tiles, for one type
template <int MODE, int BN, bool PAIR, typename T>
__device__ __forceinline__ void epilogue_loop(const GemmParams &p, uint32_t tmem, uint32_t rank, int warp, int lane,
                                              int first_tile, int tile_step, uint64_t *tfull_bar, uint64_t *tempty_bar,
                                              uint32_t buf, volatile int *abort_p) {
  constexpr int kCols = MODE == kGateUp ? BN / 2 : BN, kRows = PAIR ? 2 * kBM : kBM;
  const int q = warp & 3, half = (warp - 2) >> 2;
  RingPos<2> acc;
  Epilogue<MODE, BN, T> e;
  for (int t = first_tile; t < p.tiles; t += tile_step, acc.next()) {
    const Tile tl = tile_of<MODE>(p, t, kRows, kCols);
    e.begin(p, tl, half, tl.m0 + (int)rank * kBM + q * 32, buf);
    if (!warp_wait(&tfull_bar[acc.slot], acc.round, abort_p, p.status, p.wait_ns)) break;
    tc_fence_after();
    e.template finish<false>(p, tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc.slot * BN));
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      if constexpr (PAIR) mbar_arrive_cluster(in_cta(&tempty_bar[acc.slot], 0));
      else mbar_arrive(&tempty_bar[acc.slot]);
    }
  }
}

// The epilogue of a tile whose k the cluster's CTAs share (p.splits: two or four): lane quarter q of the
// rows belongs to CTA q * splits / 4, which gets the others' sums of it and finishes it.
template <int MODE, int BN, typename T>
__device__ __forceinline__ void epilogue_split(const GemmParams &p, uint32_t tmem, int rank, int warp, int tile,
                                               uint64_t *tfull_bar, uint32_t buf, uint32_t parts0, volatile int *abort_p) {
  constexpr int kCols = MODE == kGateUp ? BN / 2 : BN;
  const int q = warp & 3, half = (warp - 2) >> 2, owner = q * p.splits / 4;
  const int first_q = owner * 4 / p.splits;  // the owner's first quarter
  const uint32_t parts = parts0 + (q - first_q) * (p.splits - 1) * 32 * BN * 4;
  const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16);
  const Tile tl = tile_of<MODE>(p, tile, kBM, kCols);
  Epilogue<MODE, BN, T> e;
  e.parts = parts;
  if (owner == rank) e.begin(p, tl, half, tl.m0 + q * 32, buf);
  const bool ok = warp_wait(tfull_bar, 0u, abort_p, p.status, p.wait_ns);
  tc_fence_after();
  if (ok && owner != rank) {
    const uint32_t to = in_cta_of(parts, owner);
    const int slot = rank < owner ? rank : rank - 1;
#pragma unroll 1
    for (int c0 = half * (BN / 2); c0 < (half + 1) * (BN / 2); c0 += 16) {
      float v[16];
      tmem_ld16(tbase + c0, v);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        st_cluster_128(to + e.part_at(slot, c0 / 4 + i), v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    }
  }
  cluster_sync();  // every part has arrived
  if (ok && owner == rank) e.template finish<true>(p, tbase);
}

template <int MODE, int BN, int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    dense_gemm_kernel(const __grid_constant__ GemmMaps maps, const __grid_constant__ GemmParams p) {
  using C = Cfg<MODE, BN, KIND>;
  constexpr bool PAIR = C::PAIR, SPLIT = C::SPLIT;
  constexpr int kCols = MODE == kGateUp ? BN / 2 : BN;  // output columns of a tile
  constexpr int kRows = PAIR ? 2 * kBM : kBM;           // output rows of a tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[C::kStages], empty_bar[C::kStages], tfull_bar[2], tempty_bar[2];
  __shared__ __align__(8) uint64_t mma_done_bar, never_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_rank() : 0u;  // in the pair
  const int part = SPLIT ? (int)cluster_rank() : 0;  // of k
  const int first_tile = PAIR ? blockIdx.x >> 1 : SPLIT ? blockIdx.x / p.splits : blockIdx.x;
  const int tile_step = PAIR ? gridDim.x >> 1 : SPLIT ? p.tiles : gridDim.x;
  // this CTA's k blocks of a tile of problem q
  auto kb_first = [&](const GemmProblem &q) { return SPLIT ? part * q.kb / p.splits : 0; };
  auto kb_end = [&](const GemmProblem &q) { return SPLIT ? (part + 1) * q.kb / p.splits : q.kb; };
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
  if constexpr (PAIR || SPLIT) cluster_sync();  // the other CTAs run, and their barriers are initialised
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  volatile int *abort_p = &abort_flag;
  pdl_wait();     // from here on what the kernel before it wrote is read
  pdl_trigger();  // the next one may come: not earlier, as it may read before its own wait what this one waited for

  if (warp == 0) {
    // ---------------- TMA producer ----------------
    RingPos<C::kStages> pos;
    int j = 0;
    bool ok = true;
    const uint32_t ring0 = smem_u32(ring), full0 = PAIR ? in_cta(full_bar, 0) : smem_u32(full_bar);
    for (int t = first_tile; ok && t < p.tiles; t += tile_step) {
      const Tile tl = tile_of<MODE>(p, t, kRows, kCols);
      const GemmProblem &q = p.problem[tl.prob];
      const bool a_mn = MODE == kGrads && q.a_mn;
      const uint32_t stage_bytes = a_mn ? C::kStage : C::kStage - (kBM - p.a_rows) * kBK * 2;
      const int m0 = tl.m0 + (int)rank * kBM, n0 = tl.n0 + (MODE == kGateUp ? 0 : (int)rank * C::kBUsed);
      const int last = kb_end(q);
      for (int kb = kb_first(q); kb < last; ++kb, ++j, pos.next()) {
        const int s = pos.slot;
        if (!warp_wait(&empty_bar[s], pos.round ^ 1u, abort_p, p.status, p.wait_ns)) {
          ok = false;
          break;
        }
        const int second = MODE == kGrads && kb >= q.kb0, k0 = (second ? kb - q.kb0 : kb) * kBK;
        const CUtensorMap *ma = &maps.a[MODE == kGrads ? q.a + second : 0], *mb = &maps.b[MODE == kGrads ? q.b + second : 0];
        // the leader's barrier counts both CTAs' bytes
        if (rank == 0) mbar_expect_one(full0 + 8 * s, PAIR ? 2 * stage_bytes : stage_bytes);
        const uint32_t a = ring0 + s * C::kStage, b = a + kABytes, fb = full0 + 8 * s;
        if (a_mn) {
          tma_load_2d_one<PAIR>(a, ma, fb, m0, k0);
          tma_load_2d_one<PAIR>(a + kBK * 128, ma, fb, m0 + 64, k0);
        } else {
          tma_load_2d_one<PAIR>(a, ma, fb, k0, m0);
        }
        if constexpr (C::kBMn) {
#pragma unroll
          for (int i = 0; i < C::kBRows / 64; ++i)
            tma_load_2d_one<PAIR>(b + i * kBK * 128, mb, fb, n0 + 64 * i, k0);
        } else if constexpr (MODE == kGateUp) {
          if constexpr (PAIR) {  // the leader holds the gate's rows, its peer the up projection's
            tma_load_2d_one<PAIR>(b, &maps.b[rank], fb, k0, n0);
          } else {
            tma_load_2d_one<PAIR>(b, &maps.b[0], fb, k0, n0);
            tma_load_2d_one<PAIR>(b + (BN / 2) * 128, &maps.b[1], fb, k0, n0);
          }
        } else {
          tma_load_2d_one<PAIR>(b, mb, fb, k0, n0);
        }
      }
    }
    if (lane == 0) issued = j;
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (rank == 0) {
      if (p.inject && blockIdx.x == 0)  // test hook: a wait that runs out
        (void)warp_wait(&never_bar, 0u, abort_p, p.status, p.wait_ns);
      // 16 k are 32 bytes of a K-major row, or 16 rows of 128 bytes of an MN-major box
      // (an address of shared memory carries the CTA's rank in its cluster above the 18 bits that count)
      const uint64_t ring_d = (smem_u32(ring) >> 4) & 0x3FFFu;
      const uint64_t b0 = (C::kBMn ? smem_desc_mn(0) : smem_desc_sw128(0)) + ring_d + (kABytes >> 4);
      constexpr int kBStep = (C::kBMn ? 2048 : 32) >> 4;
      RingPos<C::kStages> pos;
      RingPos<2> acc;
      bool ok = true;
      for (int t = first_tile; ok && t < p.tiles; t += tile_step, acc.next()) {
        const GemmProblem &q = p.problem[MODE == kGrads ? tile_of<MODE>(p, t, kRows, kCols).prob : 0];
        const bool a_mn = MODE == kGrads && q.a_mn;
        const uint32_t idesc = idesc_16(p.f16, a_mn, C::kBMn, kRows, BN);
        const uint64_t a0 = (a_mn ? smem_desc_mn(0) : smem_desc_sw128(0)) + ring_d;
        const int a_step = (a_mn ? 2048 : 32) >> 4, begin = kb_first(q), last = kb_end(q);
        if (!warp_wait(&tempty_bar[acc.slot], acc.round ^ 1u, abort_p, p.status, p.wait_ns)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(acc.slot * BN);
        for (int kb = begin; kb < last; ++kb, pos.next()) {
          if (!warp_wait(&full_bar[pos.slot], pos.round, abort_p, p.status, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t at = pos.slot * (C::kStage >> 4);
#pragma unroll
          for (int k = 0; k < kBK / 16; ++k)
            tc_mma_one<PAIR, false>(d, a0 + (at + k * a_step), b0 + (at + k * kBStep), idesc, (kb > begin || k > 0) ? 1u : 0u);
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
    const uint32_t buf = smem_u32(ring) + C::kStages * C::kStage + (warp - 2) * kStageBuf;
    if constexpr (SPLIT) {
      const uint32_t parts = smem_u32(ring) + C::kStages * C::kStage + C::kBufBytes;
      if (p.f16) epilogue_split<MODE, BN, __half>(p, tmem, part, warp, first_tile, tfull_bar, buf, parts, abort_p);
      else epilogue_split<MODE, BN, __nv_bfloat16>(p, tmem, part, warp, first_tile, tfull_bar, buf, parts, abort_p);
    } else if (p.f16) {
      epilogue_loop<MODE, BN, PAIR, __half>(p, tmem, rank, warp, lane, first_tile, tile_step, tfull_bar, tempty_bar, buf,
                                            abort_p);
    } else {
      epilogue_loop<MODE, BN, PAIR, __nv_bfloat16>(p, tmem, rank, warp, lane, first_tile, tile_step, tfull_bar, tempty_bar,
                                                   buf, abort_p);
    }
  }
  if constexpr (SPLIT) {
    if (warp < 2) cluster_sync();  // the epilogue warps' barrier counts every thread
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

template <int MODE, int BN, int KIND>
cudaError_t launch(const GemmMaps &maps, const GemmParams &p, int num_sms, cudaStream_t st) {
  using C = Cfg<MODE, BN, KIND>;
  static std::atomic<unsigned long long> done{0};
  static std::atomic<int> pairs{0};
  if constexpr (C::SPLIT)
    return launch_clusters(dense_gemm_kernel<MODE, BN, KIND>, C::kSmem, done, p.tiles, p.splits, kThreads, st, maps, p);
  else
    return launch_tiles<C::PAIR>(dense_gemm_kernel<MODE, BN, KIND>, C::kSmem, done, pairs, p.tiles, num_sms, st,
                                 maps, p);
}

// rows and columns of a tile's results
int tile_rows(DenseTile g) { return g.kind == kPairTile ? 2 * kBM : kBM; }
int tile_cols(int mode, DenseTile g) { return mode == kGateUp ? g.bn / 2 : g.bn; }
long long tiles_of(int mode, const GemmProblem &q, DenseTile g) {
  return (long long)cdiv(q.m, tile_rows(g)) * cdiv(q.n, tile_cols(mode, g));
}

}  // namespace

int gemm_b_box(int mode, DenseTile t) {
  if (mode == kHiddenGrad || mode == kGrads) return 64;
  return mode == kGateUp || t.kind == kPairTile ? t.bn / 2 : t.bn;
}

// The tile that takes the least time by what tiles measured (us on the GPU, launches replayed in a graph, bf16):
// a k block of 64 with 256, 128, 64 and 32 columns 0.339, 0.200, 0.157 and 0.147 on a CTA by itself (few columns:
// the time to issue four MMAs), 0.045 + 0.00092 for each column on a pair; the epilogue of a tile 0.25 + 0.0085 for each column
// of a plain result, 0.45 + 0.0078 of kGateUp, and 0.032 a column of kHiddenGrad, whose ten bytes for each
// value are memory's; of the two the longer, and together no less than 0.8 of their sum; a launch with its
// prologue 3.8, of pairs 5.8.  Rows that are no multiple of 128 bytes make each 128 bytes of a box two
// lines, 0.0014 for each.  Tiles go in waves over the SMs, so the widest tile is not always the fastest:
// 4096 x 4096 columns by 4096 took 83.1 us in 256 tiles of 256 columns (3.4 waves of 76 pairs), 75.6 in 304
// of 224 (4.0), and 1024 rows 29.4 in one wave of pairs, 34.8 in two of 128 columns.
//
// Few tiles with a long k leave SMs idle; then clusters of two or four CTAs share a tile's k (64 columns) and
// exchange their sums, for 2.2 more at the start and the end, and 4.2 for each further wave, as these CTAs
// make one tile each.  8 rows, hidden 4096, inter 2048: the gate and up projections 14.7 in single CTAs, 12.4
// in clusters of two; the backward pass's first product 15.5 and, in clusters of four, 11.6.
//
// Several products in one launch save a launch and share its last wave, but also the tile.  The backward
// pass of 1016 rows, hidden 224, inter 424 took 21.0 with two launches for kGrads, 13.9 with one; 4096 rows,
// hidden 4096, inter 2048 268 and 247; 8 rows, hidden 4096, inter 2048, whose dx wants clusters, 40.9 with
// two and 45.7 with one, where the model puts one ahead all the same (30.5 for 31.7 of these launches).
DenseTile gemm_pick_tile(int mode, const GemmParams &p, int num_sms, double *time) {
  const bool b_mn = mode == kHiddenGrad || mode == kGrads;
  const double per_col = mode == kGateUp ? 0.0078 : mode == kHiddenGrad ? 0.032 : 0.0085;
  const double per_tile = mode == kGateUp ? 0.45 : mode == kHiddenGrad ? 0.0 : 0.25;
  const struct {
    DenseTile tile;
    double k_block;
  } all[] = {{{256, kPairTile, 1}, 0.280}, {{224, kPairTile, 1}, 0.251}, {{192, kPairTile, 1}, 0.222},
             {{128, kPairTile, 1}, 0.163}, {{256, kOneTile, 1}, 0.339},  {{128, kOneTile, 1}, 0.200},
             {{64, kOneTile, 1}, 0.157},   {{32, kOneTile, 1}, 0.147},   {{64, kSplitTile, 2}, 0.157},
             {{64, kSplitTile, 4}, 0.157}};
  DenseTile best = {0, kOneTile, 1};
  for (const auto &c : all) {
    const int splits = c.tile.splits;
    bool fits = !(b_mn && c.tile.bn < 64);
    for (int i = 0; i < p.problems; ++i) fits = fits && splits <= p.problem[i].kb;
    // a pair's boxes have one height, whose bytes a barrier of the other CTA counts
    if (!fits || (c.tile.kind == kPairTile && p.a_rows < kBM)) continue;
    // pairs lie on the two SMs of a pair; not every SM can be in a cluster of four
    const long long units = c.tile.kind == kPairTile || splits == 2 ? num_sms / 2 : splits == 4 ? num_sms * 36 / 152 : num_sms;
    const double epilogue = per_tile + per_col * c.tile.bn;
    const double lines = p.odd_rows ? 0.0014 * (p.a_rows + (c.tile.kind == kPairTile ? c.tile.bn / 2 : c.tile.bn)) : 0.0;
    const double k_block = c.k_block > lines ? c.k_block : lines;
    double us = (c.tile.kind == kPairTile ? 5.8 : c.tile.kind == kSplitTile ? 6.0 : 3.8) + epilogue;
    long long tiles = 0, waves = 0;
    double work = 0.0, longest = 0.0, shortest = 0.0;
    for (int i = 0; i < p.problems; ++i) {  // longest k first
      const long long own = tiles_of(mode, p.problem[i], c.tile), upto = (tiles += own, (tiles + units - 1) / units);
      const double products = k_block * ((p.problem[i].kb + splits - 1) / splits);
      if (c.tile.kind == kSplitTile) {
        shortest = products + 4.2;
        longest = longest > shortest ? longest : shortest;
        work += own * shortest;
      } else {  // a wave takes as long as its first tile
        us += (upto - waves) * std::max({products, epilogue, 0.8 * (products + epilogue)});
        waves = upto;
      }
    }
    if (c.tile.kind == kSplitTile)  // a cluster for each tile, the next as one ends
      us += (tiles <= units ? longest : p.problems == 1 ? (tiles + units - 1) / units * longest
                                                        : std::max(longest, work / units + shortest)) - 4.2;
    if (best.bn == 0 || us < *time) {
      best = c.tile;
      *time = us;
    }
  }
  return best;
}

cudaError_t launch_dense_gemm(int mode, DenseTile g, const GemmMaps &maps, GemmParams p, int num_sms, cudaStream_t st) {
  p.splits = g.splits;
  p.tiles = 0;
  for (int i = 0; i < p.problems; ++i) {
    GemmProblem &q = p.problem[i];
    q.tiles_m = cdiv(q.m, tile_rows(g));
    q.tiles_n = cdiv(q.n, tile_cols(mode, g));
    q.end = p.tiles += (int)tiles_of(mode, q, g);
  }
#define MOE_LAUNCH(MODE, BN, KIND) \
  if (mode == MODE && g.bn == BN && g.kind == KIND) return launch<MODE, BN, KIND>(maps, p, num_sms, st)
#define MOE_LAUNCH_ALL(MODE)         \
  MOE_LAUNCH(MODE, 256, kPairTile);  \
  MOE_LAUNCH(MODE, 224, kPairTile);  \
  MOE_LAUNCH(MODE, 192, kPairTile);  \
  MOE_LAUNCH(MODE, 128, kPairTile);  \
  MOE_LAUNCH(MODE, 256, kOneTile);   \
  MOE_LAUNCH(MODE, 128, kOneTile);   \
  MOE_LAUNCH(MODE, 64, kOneTile);    \
  MOE_LAUNCH(MODE, 64, kSplitTile)
  MOE_LAUNCH_ALL(kGateUp);
  MOE_LAUNCH(kGateUp, 32, kOneTile);
  MOE_LAUNCH_ALL(kDown);
  MOE_LAUNCH(kDown, 32, kOneTile);
  MOE_LAUNCH_ALL(kHiddenGrad);
  MOE_LAUNCH_ALL(kGrads);
#undef MOE_LAUNCH_ALL
#undef MOE_LAUNCH
  return cudaErrorInvalidValue;
}

}  // namespace moe
