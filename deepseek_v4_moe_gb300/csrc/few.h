// Host-side launchers of the kernels for a few rows: products with 4-bit weights, and the routed layer without a handle.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dense.h"

namespace moe {

// A matrix [n, k] of weights, or several of them one after another (experts).  16-bit: values of the call's type, no
// scales.  4-bit: codes [n, k / 2] (the even column in the low half), scales [n, groups] of the call's type, zero points
// [n, groups] or none (8).
struct FewMatrix {
  const void *w;
  const uint16_t *scales;
  const uint8_t *zeros;
  int n, k, groups, group_shift;
};

// Halves of 128 columns that a tile of the FP8 tensor cores' form has: one where two halves' sums of all groups leave no
// room for a second tile's in TMEM (16 tokens of the routed layer in groups of 32: 566 us, 510 so; f16 599 and 559), or, of
// 32 tokens, not even for one's (in groups of 64 one half would take 937 us for 789: the tiles' fixed costs count for both
// joining sets).  groups: of 128 columns.
constexpr int code_halves(int tokens, int planes, int groups) {
  return 2 * groups * ((tokens * planes + 15) / 16 * 16) <= (tokens > 16 ? 384 : 192) ? 2 : 1;
}

// CTAs of a cluster that share a row tile's columns: as many as run at one time (of clusters of 8, 4 and 2 with an SM for
// each CTA, 12, 36 and 75 on 152 SMs: 16 tiles of 2048 x 8192 by 32 tokens took 18 us in eights, 12.5 in fours)
inline int code_splits(long long tiles, int num_sms) {
  return tiles <= num_sms * 12 / 152 ? 8 : tiles <= num_sms * 36 / 152 ? 4 : tiles <= num_sms * 75 / 152 ? 2 : 1;
}

// what a kernel with bounded waits reports to, how long they last, and whether one is to run out
struct Waits {
  int *status;
  uint64_t ns;
  int inject;
};

struct Int4MatmulParams {
  FewMatrix w;
  int rows;
  const void *x;
  void *out;
  long long ld_x, ld_out;
  Waits waits;
  // Workspace of the FP8 tensor cores' form: x as planes of codes [blocks of tokens][planes][tokens][k], the groups' sums
  // [blocks][sum_groups][tokens], what the rows' sums are multiplied by.
  uint2 *planes;
  float *sums, *back;
  int sum_groups;  // groups of a row, up to a whole tile
};
// tokens of a block in that form, for so many rows; 0: the other form serves the call
int int4_tc_tokens(int rows, int n, int k, int group);
// w: the codes, boxes of 64 bytes x the rows of a CTA's sets; x: pieces of 32 columns, boxes of those of a step's tiles.  FP8
// form: w the codes, boxes of 64 bytes for each half of a tile x 128 rows; x the planes, boxes of 128 bytes x a block's rows
struct Int4Maps {
  CUtensorMap w, x;
};
cudaError_t launch_int4_tc(const Int4MatmulParams &p, const Int4Maps &maps, int tokens, bool f16, int num_sms, cudaStream_t st);
// strips of 16 rows and eights of tokens of a warp, shares of k (2^log_kw), tokens of a copy of x
struct Int4Tiles {
  int strips, eights, log_kw, box_rows;
  int w_box() const { return 16 * strips * (8 >> log_kw) < 256 ? 16 * strips * (8 >> log_kw) : 256; }  // rows; TMA's most
  int x_box_pieces() const { return 4 << log_kw; }
};
Int4Tiles int4_pick_tiles(int rows, int n, int k, int num_sms);
cudaError_t launch_int4_matmul(const Int4MatmulParams &p, const Int4Maps &maps, const Int4Tiles &t, bool f16, int num_sms,
                               cudaStream_t st);

struct Int4WeightParams {
  int n, k, group, type;      // type: of w, or of the widened matrix
  const void *w;
  long long ld_w;
  uint8_t *codes;
  void *scales;
  uint8_t *zeros;             // or none
  int f16;                    // of the scales
  void *out;                  // widen
  long long ld_out;
};
cudaError_t launch_int4_quantise(const Int4WeightParams &p, int num_sms, cudaStream_t st);
cudaError_t launch_int4_widen(const Int4WeightParams &p, int num_sms, cudaStream_t st);

// ---- the routed layer ----

constexpr int kRoutedRows = 32;     // tokens of a call: a bit each in a group's mask
constexpr int kRoutedExperts = 512;
constexpr int kRoutedTopK = 8;
constexpr int kRoutedShared = 8;
constexpr int kHiddenPlanes = 3;    // of the 4-bit layer's hidden values, in either type

struct RoutedParams {
  int rows, hidden, inter, experts, top_k, shared;
  int softmax, normalise, act, router_f32;
  float scale;
  const void *x;
  long long ld_x;
  const void *router;
  const float *bias;
  FewMatrix gate, up, down;            // the experts'
  FewMatrix s_gate, s_up, s_down;      // the shared experts'
  void *y;
  long long ld_y;
  int32_t *indices;                    // [rows, top_k] or none
  float *weights;
  float *logits;                       // workspace: [rows, experts]
  // The hidden values, of groups: experts with tokens.
  uint16_t *h;                         // workspace: of 16-bit weights [groups, 2 parts, rows up to a multiple of 8, inter]
  float *h32;                          // workspace: of 4-bit weights [groups, rows, inter]
  int groups;                          // at most
  // Workspace of 4-bit weights: x and h32 as planes [1 or groups][planes][tokens][k], their groups' sums [1 or groups]
  // [x_groups or h_groups][tokens], what products of x are multiplied by, the largest |h| of a token, groups' tokens.
  uint2 *x_planes, *h_planes;
  float *x_sums, *h_sums, *back;
  uint32_t *h_max, *masks;
  int x_groups, h_groups;              // of a row, up to a whole tile
  Waits waits;
};
// Over all experts' rows of each matrix; of the down kernels gate and s_gate are down and s_down; boxes of 64 rows (down:
// 128).  16 bits: boxes of 128 bytes, and tokens: x, or h, boxes of 128 bytes x the tokens up to a multiple of 8 (h: twice).  4 bits:
// boxes of 64 bytes for each half of a tile, and tokens: planes, boxes of 128 bytes x routed_code_tokens' of each.
struct RoutedMaps {
  CUtensorMap gate, up, s_gate, s_up, tokens;
};
cudaError_t launch_routed(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, bool f16, int num_sms, cudaStream_t st);
inline int routed_code_tokens(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }
cudaError_t launch_routed_int4(const RoutedParams &p, const RoutedMaps &maps, const RoutedMaps &down, bool f16, int num_sms,
                               cudaStream_t st);

}  // namespace moe
