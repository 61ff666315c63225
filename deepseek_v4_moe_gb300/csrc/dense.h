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
  size_t gate_part, floats;  // offset of the gate's partials, and the workspace's size
};
NormBwdPlan norm_bwd_plan(const NormParams &p, int num_sms);
cudaError_t launch_block_norm(const NormParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_block_norm_backward(const NormParams &p, int num_sms, cudaStream_t st);

}  // namespace moe
