// What the dense sublayer's tensor-core kernels share.
#pragma once
#include <atomic>

#include "common.cuh"

namespace moe {

constexpr int kBM = 128;                             // rows of a tile: the MMA's M
constexpr int kEpiWarps = 8, kThreads = 32 * (2 + kEpiWarps);
constexpr int kRingBytes = 224 * 1024;  // what barriers and alignment leave of a CTA's shared memory

// mbar_wait_bounded, which reads the timer only once a barrier has stayed open for some tries: a try
// waits a while by itself, and the timer's latency would be added to every wait of a pipeline.
__device__ __forceinline__ bool wait_bounded(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *dev_status,
                                             uint64_t limit_ns) {
#pragma unroll 1
  for (int i = 0; i < 64; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  return mbar_wait_bounded(bar, parity, abort_flag, dev_status, limit_ns);
}

// Allows a kernel its dynamic shared memory, once on each device (`done`: one bit a device).
inline cudaError_t allow_smem(const void *kernel, size_t bytes, std::atomic<unsigned long long> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Tile t of tm x tn, in bands of 16 row blocks, so that the CTAs at work at one time share both
// operands in L2.
__device__ __forceinline__ void band_tile(int t, int tm, int tn, int &m, int &n) {
  const int band = t / (16 * tn), first = band * 16, height = min(tm - first, 16);
  t -= band * 16 * tn;
  m = first + t % height;
  n = t / height;
}

// ---- a pair of CTAs on one tile (cluster of 2, cta_group::2) ----

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the shared::cluster address of the same variable in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(const void *p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t in_cta_of(uint32_t shared_addr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(shared_addr), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_cluster_128(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d) : "memory");
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Arrives at a barrier of another CTA.  What it orders are TMEM loads, by the tcgen05 fences around it;
// a release at cluster scope would first wait for every memory access in flight, 1.5 us of the round
// trip of a TMEM buffer.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(addr) : "memory");
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
// ---- asynchronous operations issued by one lane of a converged warp ----
// The election is inside the instruction sequence, so the code around it is uniform over the warp and
// its descriptors and addresses stay in uniform registers: a tcgen05.mma issued from a branch that one
// lane takes cost 107 to 143 cycles of issue, N = 256 tiles 171 instead of 128; issued like this 57,
// and 128.  The elected lane is the same every time.

// a box into this CTA's shared memory, its bytes counted on the barrier at `bar` (PAIR: of this CTA or
// its peer, a shared::cluster address)
template <bool PAIR>
__device__ __forceinline__ void tma_load_2d_one(uint32_t dst, const void *tmap, uint32_t bar, int c_inner, int c_outer) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
        "{%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(tmap), "r"(bar), "r"(c_inner), "r"(c_outer)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], "
        "[%2];\n\t}" ::"r"(dst),
        "l"(tmap), "r"(bar), "r"(c_inner), "r"(c_outer)
        : "memory");
}
__device__ __forceinline__ void mbar_expect_one(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
#define MOE_MMA_ONE(GROUP, KIND)                                                    \
  asm volatile(                                                                     \
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\t"                    \
      "setp.ne.b32 p, %4, 0;\n\t"                                                   \
      "@q tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem), \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)                         \
      : "memory")
template <bool PAIR, bool FP8>
__device__ __forceinline__ void tc_mma_one(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
  if constexpr (PAIR && FP8) MOE_MMA_ONE("2", "f8f6f4");
  else if constexpr (PAIR) MOE_MMA_ONE("2", "f16");
  else if constexpr (FP8) MOE_MMA_ONE("1", "f8f6f4");
  else MOE_MMA_ONE("1", "f16");
}
#undef MOE_MMA_ONE
// arrives on the barrier (PAIR: at the same place in both CTAs) once all MMAs issued before have completed
template <bool PAIR>
__device__ __forceinline__ void tc_commit_one(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(
            bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
// the same for a barrier of this CTA only
template <bool PAIR>
__device__ __forceinline__ void tc_commit_local_one(uint32_t bar) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
  else
    tc_commit_one<false>(bar);
}
// wait_bounded by a whole warp, with one verdict
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag, int *dev_status,
                                          uint64_t limit_ns) {
  return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag, dev_status, limit_ns)) != 0;
}
// a ring position: slot and the parity of its round
template <int SLOTS>
struct RingPos {
  int slot;
  uint32_t round = 0;
  __device__ __forceinline__ RingPos(int first = 0) : slot(first) {}
  __device__ __forceinline__ void next(int by = 1) {  // (SLOTS is a multiple of `by`)
    slot += by;
    if (slot >= SLOTS) {
      slot -= SLOTS;
      round ^= 1u;
    }
  }
};

__device__ __forceinline__ void tmem_alloc_pair(uint32_t *smem_dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(smem_dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// A warp's staging buffer: 32 rows x 64 bytes, a row's in four pieces, piece c of
// row r at place c ^ (r / 2 % 4), so that both a warp writing one piece of every row and a warp writing
// whole rows side by side meet every bank once.
constexpr int kStageBuf = 32 * 64;
__device__ __forceinline__ uint32_t piece_at(int r, int c) { return r * 64 + ((c ^ (r >> 1)) & 3) * 16; }
__device__ __forceinline__ void sts128(uint32_t a, const uint4 w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 w;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(a) : "memory");
  return w;
}

// Launches a kernel over `tiles` tiles: one CTA, or one pair of CTAs, on each SM (pair) that has work.
// Its CTAs may start, and wait in pdl_wait, while the kernel before it on the stream ends.
template <bool PAIR, typename... KArgs, typename... Args>
cudaError_t launch_tiles(void (*kernel)(KArgs...), size_t smem, std::atomic<unsigned long long> &done,
                         std::atomic<int> &pairs, int tiles, int num_sms, cudaStream_t st, const Args &...args) {
  const cudaError_t e = allow_smem((const void *)kernel, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {PAIR ? 2u : 1u, 1u, 1u};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int units = num_sms;
  if constexpr (PAIR) {  // pairs that run at one time
    units = pairs.load(std::memory_order_relaxed);
    if (!units) {
      const cudaError_t q = cudaOccupancyMaxActiveClusters(&units, kernel, &cfg);
      if (q != cudaSuccess) return q;
      if (units < 1 || units > num_sms / 2) units = num_sms / 2;
      pairs.store(units, std::memory_order_relaxed);
    }
  }
  const int busy = tiles < units ? tiles : units;
  cfg.gridDim = dim3(PAIR ? 2 * busy : busy);
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Launches a kernel with a cluster of `ctas` CTAs for each tile.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), size_t smem, std::atomic<unsigned long long> &done, int tiles,
                            int ctas, int threads, cudaStream_t st, const Args &...args) {
  const cudaError_t e = allow_smem((const void *)kernel, smem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)ctas, 1u, 1u};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles * ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace moe
