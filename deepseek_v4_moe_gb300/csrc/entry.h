// What the C entry points without a handle share: error texts, the device, checks of tensors' places.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <atomic>

#include "kernels.h"
#include "moe_ffn.h"

namespace moe {
namespace entry {

constexpr int kMaxDevices = 64;

inline int fail(int code, const char *fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  moe::set_global_error(buf);
  return code;
}

// SMs of the current device; a negative code where it is no sm_103 device
inline int current_sms() {
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    cudaGetLastError();
    return fail(MOE_FFN_ERR_CUDA, "no usable current device");
  }
  int sms = known[dev].load(std::memory_order_relaxed);
  if (sms) return sms;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return fail(MOE_FFN_ERR_CUDA, "cannot query device %d", dev);
  }
  if (major != 10 || minor != 3) return fail(MOE_FFN_ERR_UNSUPPORTED, "needs an sm_103 device, found sm_%d%d", major, minor);
  known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// A tensor argument's memory: `rows` rows of `cols` elements, `ld` elements apart; width and pitch in bytes.
struct Span {
  const void *p;
  uintptr_t end, width, pitch;
  int64_t ld;
  const char *name;
};
inline Span span(const char *name, const void *p, int64_t rows, int64_t cols, int64_t ld, int bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Span{p, p && rows > 0 ? a + (uintptr_t)((rows - 1) * ld + cols) * bytes : a, (uintptr_t)cols * bytes,
              (uintptr_t)ld * bytes, ld, name};
}
inline bool overlap(const Span &a, const Span &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (!(a.p && b.p && x < b.end && y < a.end)) return false;
  if (a.pitch != b.pitch || a.pitch == 0) return true;
  // rows at the same distance, as of two column ranges of one tensor: b's begin this far into a's pitch
  const uintptr_t into = y >= x ? (y - x) % a.pitch : (a.pitch - (x - y) % a.pitch) % a.pitch;
  return into < a.width || into + b.width > a.pitch;
}
// An output may overlap no input and no other output, but for the one input it may be itself.
inline int check_overlaps(const char *who, const Span *outs, int n_outs, const Span *ins, int n_ins, int same_out, int same_in) {
  for (int i = 0; i < n_outs; ++i) {
    for (int j = 0; j < n_ins; ++j)
      if (overlap(outs[i], ins[j]) &&
          !(i == same_out && j == same_in && outs[i].p == ins[j].p && outs[i].ld == ins[j].ld))
        return fail(MOE_FFN_ERR_ALIAS, "%s: %s overlaps %s", who, outs[i].name, ins[j].name);
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return fail(MOE_FFN_ERR_ALIAS, "%s: %s overlaps %s", who, outs[i].name, outs[j].name);
  }
  return MOE_FFN_OK;
}

inline int type_bytes(int t) { return t == MOE_FFN_F32 ? 4 : 2; }
inline bool is_type(int t) { return t == MOE_FFN_F32 || t == MOE_FFN_BF16 || t == MOE_FFN_F16; }
inline bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// A CUDA call of this one failed.  The caller learns of it here, so the runtime forgets it: an error that stayed
// recorded for the thread would be reported by its next calls too, whose work has nothing to do with it.  (One
// that the context does not recover from comes back by itself.)
inline int cuda_failed(const char *who, const char *what, cudaError_t e) {
  cudaGetLastError();
  return fail(MOE_FFN_ERR_CUDA, "%s: %s: %s", who, what, cudaGetErrorString(e));
}
inline int launched(const char *who, cudaError_t e) { return e == cudaSuccess ? MOE_FFN_OK : cuda_failed(who, "launch", e); }

// an error left by earlier work is reported with nothing enqueued
inline int pending(const char *who) {
  const cudaError_t e = cudaPeekAtLastError();
  return e == cudaSuccess ? MOE_FFN_OK
                          : fail(MOE_FFN_ERR_CUDA, "%s: a CUDA error is pending from earlier work: %s", who, cudaGetErrorString(e));
}

// A row stride holds a row, and the last row's place in memory stays far inside 64 bits: of the fewest rows
// strides may be as large as memory, of 2^30 rows 2^30 elements.
inline int check_stride(const char *who, const char *name, int64_t ld, int64_t rows, int64_t cols) {
  if (ld < cols) return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: the row stride of %s is below hidden", who, name);
  if (ld > ((int64_t)1 << 60) / rows)
    return fail(MOE_FFN_ERR_BAD_CONFIG, "%s: the row stride of %s is too large for %lld rows", who, name, (long long)rows);
  return MOE_FFN_OK;
}

constexpr int64_t kLdMax = (int64_t)1 << 36;  // a row stride in bytes stays below the tensor maps' 2^40

// What the kernels with bounded waits get besides their arguments: where they report a wait that ran out, how long one
// may last, and whether one is to run out for a test.
struct DeviceSide {
  int *status;
  uint64_t wait_ns;
  int inject;
};
int device_side(const char *who, DeviceSide *d);  // dense.cu

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn find_encode() {
  void *p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    return reinterpret_cast<EncodeTiledFn>(p);
  cudaGetLastError();
  return nullptr;
}

// A row-major matrix [outer, inner] of 1- or 2-byte elements, rows `ld` elements apart, in boxes of 128 (or 64) bytes x
// box_outer rows with the swizzle of that width; what lies past its ends reads as zeros.
inline bool encode_map(CUtensorMap *m, const void *base, int bytes, int64_t inner, int64_t outer, int64_t ld, int box_outer,
                       int box_bytes = 128) {
  static const EncodeTiledFn enc = find_encode();
  if (!enc) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)inner, (cuuint64_t)outer};
  const cuuint64_t strides[1] = {(cuuint64_t)(ld * bytes)};
  const cuuint32_t box[2] = {(cuuint32_t)(box_bytes / bytes), (cuuint32_t)box_outer};
  const cuuint32_t estr[2] = {1, 1};
  return enc(m, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
             const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A row-major matrix [rows, 32 * pieces] of 16-bit elements as pieces of 32 columns (64 bytes, in that swizzle), in boxes
// of box_rows rows of box_pieces pieces, piece after piece; what lies past its ends reads as zeros.
inline bool encode_pieces(CUtensorMap *m, const void *base, int64_t pieces, int64_t rows, int64_t ld, int box_rows, int box_pieces) {
  static const EncodeTiledFn enc = find_encode();
  if (!enc) return false;
  const cuuint64_t dims[3] = {32, (cuuint64_t)rows, (cuuint64_t)pieces};
  const cuuint64_t strides[2] = {(cuuint64_t)(ld * 2), 64};
  const cuuint32_t box[3] = {32, (cuuint32_t)box_rows, (cuuint32_t)box_pieces}, estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace entry
}  // namespace moe
