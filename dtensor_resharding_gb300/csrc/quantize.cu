// Values to e4m3 with one fp32 scale for each block of 128 (rows: 1 x 128; weights: 128 x 128, the layout whose scale
// tensors reshard_plan_blockwise_fp8 derives).
//
// A block's amax a = max |x| (at least 2^-100) gives the scale a * (1 / 448) and the values e4m3(x * ((1 / a) * 448)),
// rounded to nearest even. One reciprocal a block instead of a division a value; the product differs from x / scale by a
// few roundings of 32 bits, far below the 2^-4 of an e4m3 step. A block holding an infinity or NaN gets scale and values NaN.
// Both kernels read each value once, keep it in registers between the amax and the rounding, and are bound by HBM.
#include <algorithm>

#include "ops_common.cuh"
#include "values.cuh"

namespace reshard {
namespace ops {

namespace {

constexpr int kQThreads = 256;

// 8 lanes a block of 128 values, 16 each: two or four 16-byte loads, three shuffles and one 16-byte store a lane.
// 16,384 x 4096 bf16: 38.2 us, 5.3 TB/s, where a plain copy reaches 6.8 (4 lanes a block, 32 values each: the same).
template <typename T, bool Wide>
__global__ void __launch_bounds__(kQThreads) reshard_quantize_rows_kernel(Rows a, int64_t blocks, int per_row_blocks, bool wide_q) {
  grid_enter();
  const int lane = threadIdx.x & 31;
  const int64_t b = (int64_t)blockIdx.x * (kQThreads / 8) + threadIdx.x / 8;
  if (b - (lane >> 3) >= blocks) return;       // the whole warp
  const bool in = b < blocks;
  const int64_t r = !in ? 0 : blocks <= 0xffffffffll ? (uint32_t)b / (uint32_t)per_row_blocks : b / per_row_blocks;
  const int kb = in ? (int)(b - r * per_row_blocks) : 0;
  const int at = kb * kScaleBlock + (lane & 7) * 16;
  const int left = in ? (int)min((int64_t)16, a.cols - at) : 0;
  const T *const from = static_cast<const T *>(a.x) + r * a.stride + at;
  float x[16];
  if constexpr (Wide) {
    load_values<T, 16>(from, left, true, x);
  } else {
    Shifted<T, 16> s;
    uint32_t v[Shifted<T, 16>::kWords];
    s.ask(from, left, first_word(a.x));
    s.take(from, left, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = value_of<T>(v, i);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, magnitude(x[i]));
#pragma unroll
  for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
  float scale, inv;
  block_scale(m, scale, inv);
  if (!in) return;
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = e4m3x4(x[4 * i] * inv, x[4 * i + 1] * inv, x[4 * i + 2] * inv, x[4 * i + 3] * inv);
  for (int j = 0; j < a.copies; ++j) {
    const int64_t to_row = a.position ? a.position[r * a.copies + j] : r;
    if (to_row < 0) continue;
    if ((lane & 7) == 0) a.scale[to_row * a.scale_row + kb * a.scale_block] = scale;
    uint8_t *to = a.q + to_row * a.q_stride + at;
    if (wide_q && left >= 16) {
      *reinterpret_cast<uint4 *>(to) = make_uint4(q[0], q[1], q[2], q[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left) to[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
    }
  }
}

// One CTA a 128 x 128 block: 16 lanes a row, 8 values a lane in each of 8 passes, all loads in flight before the amax.
// 128 matrices of 768 x 2048 bf16: 107 us, 5.6 TB/s (values widened to 32 bits as they came: 265 us).
struct Blocks {
  const void *w;
  int64_t batch_stride, row_stride;
  int64_t rows, cols;
  uint8_t *q;
  int64_t q_batch_stride, q_row_stride;
  float *scale;
  int nb, kb;
};

// The CTA's amax, written as the block's scale and given back as the factor of its values.
__device__ __forceinline__ void block_amax(uint32_t m, uint32_t (&part)[kQThreads / 32], float *scale, float &inv) {
  m = __reduce_max_sync(kFull, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQThreads / 32; ++i) m = max(m, part[i]);
  float s;
  block_scale(m, s, inv);
  if (threadIdx.x == 0) *scale = s;
}

template <typename P>
__device__ __forceinline__ P load_stream(const P *p) {      // read once: 16 bytes at a time, not kept
  static_assert(sizeof(P) % 16 == 0, "16-byte pieces");
  P r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(P) / 16); ++i) reinterpret_cast<uint4 *>(&r)[i] = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kQThreads) reshard_quantize_blocks_kernel(Blocks a, bool wide, bool wide_q) {
  grid_enter();
  __shared__ uint32_t part[kQThreads / 32];
  const int64_t b = blockIdx.x;
  const int kb = (int)(b % a.kb), nb = (int)(b / a.kb % a.nb);
  const int64_t e = b / a.kb / a.nb;
  const int col = (threadIdx.x & 15) * 8, row0 = threadIdx.x >> 4;
  const int64_t c0 = (int64_t)kb * kScaleBlock + col;
  const int left = (int)max((int64_t)0, min((int64_t)8, a.cols - c0));
  // Whole blocks keep what they loaded as it came: eight loads in flight, and half the registers.
  if (wide && wide_q && (int64_t)(kb + 1) * kScaleBlock <= a.cols && (int64_t)(nb + 1) * kScaleBlock <= a.rows) {
    Pack<T, 8> x[8];
    const T *from = static_cast<const T *>(a.w) + e * a.batch_stride + ((int64_t)nb * kScaleBlock + row0) * a.row_stride + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = load_stream(reinterpret_cast<const Pack<T, 8> *>(from + 16 * i * a.row_stride));
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, magnitude(to_f32(x[i].v[j])));
    float inv;
    block_amax(m, part, a.scale + b, inv);
    uint8_t *to = a.q + e * a.q_batch_stride + ((int64_t)nb * kScaleBlock + row0) * a.q_row_stride + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = to_f32(x[i].v[j]) * inv;
      *reinterpret_cast<uint2 *>(to + 16 * i * a.q_row_stride) = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
    }
    return;
  }
  using S = Shifted<T, 8>;
  constexpr int kBatch = sizeof(T) == 4 ? 4 : 8;      // rows whose words are in flight together
  uint32_t v[8][S::kWords];
  const T *from = static_cast<const T *>(a.w) + e * a.batch_stride + ((int64_t)nb * kScaleBlock + row0) * a.row_stride + c0;
  const int rows = (int)min((int64_t)kScaleBlock, a.rows - (int64_t)nb * kScaleBlock) - row0;
#pragma unroll
  for (int i0 = 0; i0 < 8; i0 += kBatch) {
    S s[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) s[i].ask(from + 16 * (i0 + i) * a.row_stride, 16 * (i0 + i) < rows ? left : 0, first_word(a.w));
#pragma unroll
    for (int i = 0; i < kBatch; ++i) s[i].take(from + 16 * (i0 + i) * a.row_stride, 16 * (i0 + i) < rows ? left : 0, v[i0 + i]);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, magnitude(value_of<T>(v[i], j)));
  float inv;
  block_amax(m, part, a.scale + b, inv);
  uint8_t *to = a.q + e * a.q_batch_stride + ((int64_t)nb * kScaleBlock + row0) * a.q_row_stride + c0;
#pragma unroll
  for (int i = 0; i < 8; ++i, to += 16 * a.q_row_stride) {
    if (16 * i >= rows) break;
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = value_of<T>(v[i], j) * inv;
    const uint2 q = make_uint2(e4m3x4(x[0], x[1], x[2], x[3]), e4m3x4(x[4], x[5], x[6], x[7]));
    if (wide_q && left >= 8) {
      *reinterpret_cast<uint2 *>(to) = q;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < left) to[j] = (uint8_t)((j < 4 ? q.x : q.y) >> (8 * (j % 4)));
    }
  }
}

}  // namespace

int enqueue_quantize_rows(const Rows &r, cudaStream_t stream) {
  const int kb = (int)((r.cols + kScaleBlock - 1) / kScaleBlock);
  const int64_t blocks = r.rows * kb;
  if (blocks == 0) return RESHARD_OK;
  const dim3 grid((unsigned)((blocks + kQThreads / 8 - 1) / (kQThreads / 8)));
  const bool wide = aligned16(r.x, r.stride, element_bytes(r.dtype)), wide_q = aligned16(r.q, r.q_stride, 1);
  auto go = [&](auto t) {
    using T = decltype(t);
    return wide ? launch(reshard_quantize_rows_kernel<T, true>, grid, kQThreads, 0, 1, stream, r, blocks, kb, wide_q)
                : launch(reshard_quantize_rows_kernel<T, false>, grid, kQThreads, 0, 1, stream, r, blocks, kb, wide_q);
  };
  const cudaError_t e = r.dtype == RESHARD_F32 ? go(float()) : r.dtype == RESHARD_BF16 ? go(__nv_bfloat16()) : go(__half());
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_quantize_rows_kernel");
}

}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int reshard_quantize_rows(const void *x, int dtype, int64_t rows, int64_t cols, int64_t row_stride, void *q,
                                     int64_t q_stride, float *scale, int64_t scale_row_stride, int64_t scale_block_stride,
                                     reshard_stream_t stream) try {
  Checks c("reshard_quantize_rows");
  c.invalid(rows < 0 || cols < 0, "rows or cols < 0");
  c.invalid(!element_bytes(dtype), "dtype must be BF16, F16 or F32");
  c.invalid(row_stride < cols || q_stride < cols, "a row stride is shorter than the row");
  c.invalid(scale_row_stride < 1 || scale_block_stride < 1, "scale strides must be positive");
  c.unsupported(cols > RESHARD_MAX_EXTENT || rows > RESHARD_MAX_EXTENT || rows * ((cols + 127) / 128) > (int64_t)INT32_MAX * 32,
                "rows or cols above 2^30, or too many blocks for one launch");
  if (rows > 0 && cols > 0 && c.ok()) {
    c.pointer(x, "x", (uintptr_t)element_bytes(dtype));
    c.pointer(q, "q", 1);
    c.pointer(scale, "scale", 4);
  }
  if (!c.ok()) return c.report();
  const Rows r{x, dtype, rows, cols, row_stride, static_cast<uint8_t *>(q), q_stride, scale, scale_row_stride, scale_block_stride};
  return enqueue_quantize_rows(r, reinterpret_cast<cudaStream_t>(stream));
} OPS_CATCH

extern "C" int reshard_quantize_blocks(const void *w, int dtype, int64_t batch, int64_t rows, int64_t cols, int64_t batch_stride,
                                       int64_t row_stride, void *q, int64_t q_batch_stride, int64_t q_row_stride, float *scale,
                                       reshard_stream_t stream) try {
  Checks c("reshard_quantize_blocks");
  c.invalid(batch < 0 || rows < 0 || cols < 0, "batch, rows or cols < 0");
  c.invalid(!element_bytes(dtype), "dtype must be BF16, F16 or F32");
  c.invalid(row_stride < cols || q_row_stride < cols, "a row stride is shorter than the row");
  c.invalid(batch > 1 && (batch_stride < 0 || q_batch_stride < 0), "batch strides must not be negative");
  c.unsupported(batch > RESHARD_MAX_EXTENT || rows > RESHARD_MAX_EXTENT || cols > RESHARD_MAX_EXTENT, "an extent above 2^30");
  const int64_t nb = (rows + 127) / 128, kb = (cols + 127) / 128;
  if (c.ok()) c.unsupported(nb * kb > INT32_MAX || (nb * kb > 0 && batch > INT32_MAX / (nb * kb)), "too many blocks for one launch");
  if (batch > 0 && rows > 0 && cols > 0 && c.ok()) {
    c.pointer(w, "w", (uintptr_t)element_bytes(dtype));
    c.pointer(q, "q", 1);
    c.pointer(scale, "scale", 4);
  }
  if (!c.ok()) return c.report();
  if (batch * nb * kb == 0) return RESHARD_OK;
  const Blocks a{w, batch_stride, row_stride, rows, cols, static_cast<uint8_t *>(q), q_batch_stride, q_row_stride, scale, (int)nb, (int)kb};
  const int es = element_bytes(dtype);
  const bool wide = aligned16(w, row_stride, es) && batch_stride * es % 16 == 0;
  const bool wide_q = (reinterpret_cast<uintptr_t>(q) & 7) == 0 && q_row_stride % 8 == 0 && q_batch_stride % 8 == 0;
  const dim3 grid((unsigned)(batch * nb * kb));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == RESHARD_F32) e = launch(reshard_quantize_blocks_kernel<float>, grid, kQThreads, 0, 1, s, a, wide, wide_q);
  else if (dtype == RESHARD_BF16) e = launch(reshard_quantize_blocks_kernel<__nv_bfloat16>, grid, kQThreads, 0, 1, s, a, wide, wide_q);
  else e = launch(reshard_quantize_blocks_kernel<__half>, grid, kQThreads, 0, 1, s, a, wide, wide_q);
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_quantize_blocks_kernel");
} OPS_CATCH
