// Host-side launchers of the dense feed-forward sublayer's kernels (plain residual stream).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

enum DenseType : int { kF32 = 0, kBF16 = 1, kF16 = 2 };
constexpr int kNormHiddenMax = 8192;

enum GateKind : int { kGateNone = 0, kGateVector = 1, kGateToken = 2 };

struct NormParams {
  int rows, hidden;
  int stream_type, block_type, gate_type, gate_kind, rows_per_gate;
  float scale, eps;
  const void *state, *f, *gate;  // backward: state is the stream after the block
  long long ld_state, ld_f;
  const float *w_post, *w_next;
  // forward
  void *out, *y;
  long long ld_out, ld_y;
  // backward
  const void *d_out, *d_y;
  long long ld_d_out, ld_d_y;
  void *d_state, *d_f, *d_gate;
  long long ld_d_state, ld_d_f;
  float *d_w_post, *d_w_next;
  float *part;  // workspace, laid out by norm_bwd_plan
};

// The backward pass's split of the rows: `workers` groups of threads; each takes whole chunks of
// chunk_rows rows, none of which crosses a gate row.
struct NormBwdPlan {
  int threads, groups, ctas, workers, chunk_rows, chunks_per_gate, chunks;
  int one_gate, jobs;          // a gate of one row, a chunk of it for each worker; sums over partial rows
  int depth;                   // rows of the ring; set by the launch
  size_t gate_part, floats;    // offset of the gate's partials, and the workspace's size
};
NormBwdPlan norm_bwd_plan(const NormParams &p, int num_sms);
cudaError_t launch_block_norm(const NormParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_block_norm_backward(const NormParams &p, int num_sms, cudaStream_t st);

// ---- the gated block's matrix products (dense_gemm.cu) ----

enum GemmMode : int { kGateUp = 0, kDown = 1, kHiddenGrad = 2, kGrads = 3 };
enum Activation : int { kSilu = 0, kGelu = 1 };

struct GemmMaps {
  CUtensorMap a[5], b[4];
};

// A product of a launch: c [m, n] = the sum over its pairs of matrices, a[a] b[b] over k blocks 0 .. kb0 - 1,
// a[a + 1] b[b + 1] over those from kb0 on.
struct GemmProblem {
  int m, n, kb0, kb, a, b;
  int a_mn;                   // A is MN-major (kGrads)
  int tiles_m, tiles_n, end;  // set by launch_dense_gemm; end: its last tile's number plus one
  void *c;
  long long ldc;
};
constexpr int kMaxProblems = 4;

struct GemmParams {
  GemmProblem problem[kMaxProblems];
  int problems, tiles;  // tiles: set by launch_dense_gemm
  int splits;           // CTAs that share a tile's k; set by launch_dense_gemm
  void *out[3];         // kGateUp: h, g, u; kHiddenGrad: dg, du, h
  const void *e[2];     // kHiddenGrad: the saved g and u
  int act, f16;
  int a_rows;           // rows of a K-major A's boxes; see a_box
  int odd_rows;         // a matrix has rows that are no multiple of 128 bytes
  int *status;
  uint64_t wait_ns;
  int inject;
};

// Rows of a K-major A's boxes.  A single block of fewer rows takes boxes of its own height: rows past the
// end would be filled with zeros, which costs the copy engine as much time as loading them.  The MMA
// then reads what lies in shared memory there, into accumulator rows that nothing reads.
inline int a_box(int m) { return m >= 128 ? 128 : (m + 7) / 8 * 8; }

// A tile: bn columns (kGateUp: half of them of g, half of u) of 128 rows by one CTA, of 256 by a pair, or of
// 128 by `splits` CTAs that share its k.
enum TileKind : int { kOneTile = 0, kPairTile = 1, kSplitTile = 2 };
constexpr int kSplitMax = 4;
struct DenseTile {
  int bn, kind, splits;
};
int gemm_b_box(int mode, DenseTile tile);  // rows of B's boxes
// the fastest tile for a launch, and the time that it should take in us
DenseTile gemm_pick_tile(int mode, const GemmParams &p, int num_sms, double *time);
cudaError_t launch_dense_gemm(int mode, DenseTile tile, const GemmMaps &maps, GemmParams p, int num_sms, cudaStream_t st);

// ---- FP8 with block scales (dense_fp8.cu) ----

constexpr int kScaleBlock = 128;

struct Fp8Params {
  int m, n, kb;              // kb: blocks of 128 along k
  int a_e5m2, b_e5m2, out_type;
  const float *a_scale, *b_scale;  // [m, kb], [ceil(n / 128), kb]
  void *out;
  long long ld_out;
  int wide;                  // out can be written in 16-byte pieces
  int a_rows;                // rows of A's boxes (see a_box)
  int tiles_m, tiles_n, tiles, splits;  // set by launch_fp8_matmul
  int *status;
  uint64_t wait_ns;
  int inject;
};

struct QuantiseParams {
  int rows, k, type, e5m2, pow2, tall;  // tall: rows of a block, 1 or 128
  const void *x;
  long long ld_x;
  uint8_t *codes;
  long long ld_codes;
  float *scales;             // [ceil(rows / tall), ceil(k / 128)]
  int wide;                  // x in 16-byte pieces, codes in 8-byte pieces
};

DenseTile fp8_pick_tile(const Fp8Params &p, int num_sms);
cudaError_t launch_fp8_matmul(DenseTile tile, const CUtensorMap &a, const CUtensorMap &b, Fp8Params p, int num_sms,
                              cudaStream_t st);
cudaError_t launch_fp8_quantise(const QuantiseParams &p, int num_sms, cudaStream_t st);

// ---- products for a few rows on the CUDA cores (dense_gemv.cu) ----

bool gated_gemv(int rows, int hidden, int inter);  // these kernels are the faster ones
bool fp8_gemv(int rows, int n, int k);

struct GemvParams {
  int n, k;
  int rows, splits;          // set by the launch
  int act;
  const void *x, *w[2];
  long long ld_x;
  void *out, *gate, *up;
  long long ld_out;
};

struct Fp8GemvParams {
  int n, k, kb, splits;      // splits is set by the launch
  int a_e5m2, b_e5m2;
  const uint8_t *a, *b;
  long long ld_a, ld_b;
  const float *a_scale, *b_scale;
  void *out;
  long long ld_out;
};

// up: the gate and up projections with the activation; otherwise the down projection, which starts
// while the kernel before it on the stream runs
cudaError_t launch_gated_gemv(bool up, GemvParams p, int rows, bool f16, cudaStream_t st);
cudaError_t launch_fp8_gemv(const Fp8GemvParams &p, int rows, int num_sms, int out_type, cudaStream_t st);

}  // namespace moe
