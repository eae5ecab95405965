// What the operator kernels share: launches, argument checks, conversions, mbarrier and tcgen05 helpers.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>
#include <string>
#include <utility>

#include "plan.h"
#include "reshard_ops.h"

namespace reshard {
namespace ops {

constexpr int kScaleBlock = 128;           // elements along a row (and rows, for weights) that share one scale
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyAmax = 0x1p-100f;     // an all-zero block's amax: its scale stays a normal number

// ------------------------------------------------------------------------------------------------- host side --

inline int cuda_error(cudaError_t e, const char *what) {
  return fail(e == cudaErrorMemoryAllocation ? RESHARD_ERR_OOM : RESHARD_ERR_CUDA,
              std::string(what) + ": " + cudaGetErrorString(e));
}

// Closes the body of a C entry that is a function try block: no exception leaves the library.
inline int out_of_memory() noexcept {
  try {
    return fail(RESHARD_ERR_OOM, "out of host memory");
  } catch (...) {
    return RESHARD_ERR_OOM;
  }
}
#define OPS_CATCH catch (...) { return ::reshard::ops::out_of_memory(); }

#define OPS_CUDA(call)                                            \
  do {                                                            \
    cudaError_t e_ = (call);                                      \
    if (e_ != cudaSuccess) return ::reshard::ops::cuda_error(e_, #call); \
  } while (0)

// Every violation of a call's arguments, one per line; INVALID_ARG outranks UNSUPPORTED.
class Checks {
 public:
  explicit Checks(const char *call) : call_(call) {}
  void invalid(bool bad, const char *why) { add(bad, RESHARD_ERR_INVALID_ARG, why); }
  void unsupported(bool bad, const char *why) { add(bad, RESHARD_ERR_UNSUPPORTED, why); }
  // A buffer the kernels dereference: memory of the current device, managed memory or page-locked host memory.
  void pointer(const void *p, const char *name, uintptr_t align);
  int report() const { return n_ == 0 ? RESHARD_OK : fail(code_, std::string(call_) + ": " + std::to_string(n_) + " violation(s):" + lines_); }
  bool ok() const { return n_ == 0; }

 private:
  void add(bool bad, int code, const char *why) {
    if (bad) violation(code, why);
  }
  void violation(int code, const std::string &why) {
    if (n_++ == 0 || code == RESHARD_ERR_INVALID_ARG) code_ = code;
    lines_ += "\n  " + why;
  }
  const char *call_;
  int n_ = 0, code_ = RESHARD_OK, device_ = -1;
  std::string lines_;
};

inline int element_bytes(int dtype) { return dtype == RESHARD_F32 ? 4 : dtype == RESHARD_BF16 || dtype == RESHARD_F16 ? 2 : 0; }

int device_sms(int *sms);   // multiprocessors of the current device

// Every operator kernel begins with griddepcontrol.wait (or has it after reads of what the grid before cannot have written),
// so its CTAs may be scheduled while that grid drains: of a chain of short kernels only the work itself is left, not the
// launches between them.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, int block, size_t smem, int cluster, cudaStream_t stream, Args &&...args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cfg.attrs = attr;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

#ifdef __CUDACC__
// The dynamic shared memory of a kernel, allowed once per device. regs: what its warpgroups share out among themselves; a
// build that launches with another number would wait for registers that are not there.
template <auto kernel>
int allow_smem(size_t bytes, int regs = 0) {
  static std::mutex mu;
  static uint64_t done = 0;
  int dev = 0;
  OPS_CUDA(cudaGetDevice(&dev));
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && (done >> dev & 1)) return RESHARD_OK;
  if (regs) {
    cudaFuncAttributes fa{};
    OPS_CUDA(cudaFuncGetAttributes(&fa, kernel));
    if (fa.numRegs != regs) return fail(RESHARD_ERR_UNSUPPORTED, "the kernel was built with " + std::to_string(fa.numRegs) + " registers, not " + std::to_string(regs));
  }
  OPS_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  if (dev < 64) done |= 1ull << dev;
  return RESHARD_OK;
}
#endif

// The enqueue halves of the public calls: arguments are checked by the caller.
struct Rows {                 // a quantization by rows
  const void *x;
  int dtype;
  int64_t rows, cols, stride;
  uint8_t *q;
  int64_t q_stride;
  float *scale;
  int64_t scale_row, scale_block;
  const int32_t *position = nullptr; // row r goes to rows position[r * copies + j] >= 0, j < copies; NULL: to row r
  int copies = 1;
};
int enqueue_quantize_rows(const Rows &r, cudaStream_t stream);
int enqueue_dispatch(const int32_t *ids, int64_t slots, int first, int experts, int32_t *offsets, int32_t *order,
                     int32_t *position, cudaStream_t stream);
int enqueue_combine(const float *y, int64_t y_stride, const int32_t *position, const float *weights, int64_t tokens, int k, int64_t cols,
                    void *out, int dtype, int64_t out_stride, cudaStream_t stream);

struct Product {              // out[m, n] = sum_k a[m, k] w[n, k], both as 8-bit values times block scales
  const uint8_t *a;
  int64_t a_stride;
  const float *a_scale;
  int64_t as_row, as_block;
  const void *x = nullptr;           // rows in out's type, a_stride apart, that the product quantizes itself, in place of a and
                                     // a_scale: dense and product_quantizes()
  const uint8_t *w;
  int64_t w_batch, w_stride;
  const float *w_scale;
  const int32_t *offsets = nullptr;  // groups + 1 row offsets, on the device; NULL: one group of m rows
  int groups = 1;
  const int32_t *order = nullptr;    // row r of the product is row order[r] / per_row of a's a_rows; NULL: row r. Only
                                     // where product_gathers()
  int per_row = 1;
  int64_t a_rows = 0;
  bool early = false;                // enqueued right behind a kernel of ours that wrote none of w, offsets, order
  int64_t m, n, k;
  void *out;
  int out_dtype;
  int64_t out_stride;
  // gated: w holds 2 n rows, gate then up; out is silu(gate) * up quantized by rows of 128
  bool gated = false;
  float *out_scale = nullptr;
  int64_t os_row = 0, os_block = 0;
};
int enqueue_product(const Product &p, cudaStream_t stream);
bool product_quantizes(int64_t m, int64_t k);    // whether a dense product takes rows as `x`
bool product_gathers(int64_t m, int groups);     // whether a product of m rows in so many groups can take `order`

// ----------------------------------------------------------------------------------------------- device side --

#ifdef __CUDACC__

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_enter() {
  grid_wait();
  grid_release();
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two values as e4m3 (round to nearest even, +-448 at most, NaN stays NaN); `lo` in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | (e4m3x2(c, d) << 16); }

// A block's scale and the factor its values are multiplied by, from the bits of its largest magnitude. Magnitudes are
// compared as integers, which orders NaN above infinity above every number: a block holding either gets NaN for both.
__device__ __forceinline__ void block_scale(uint32_t amax_bits, float &scale, float &inv) {
  const float a = amax_bits >= 0x7f800000u ? __int_as_float(0x7fffffff) : fmaxf(__uint_as_float(amax_bits), kTinyAmax);
  scale = __fmul_rn(a, 1.0f / kE4m3Max);
  inv = __fmul_rn(__frcp_rn(a), kE4m3Max);
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

#endif  // __CUDACC__

}  // namespace ops
}  // namespace reshard
