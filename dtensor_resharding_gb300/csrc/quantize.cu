// Values to e4m3 with one fp32 scale for each block of 128 (rows: 1 x 128; weights: 128 x 128, the layout whose scale
// tensors reshard_plan_blockwise_fp8 derives), and the weighted sum that ends the expert layer.
//
// A block's amax a = max |x| (at least 2^-100) gives the scale a * (1 / 448) and the values e4m3(x * ((1 / a) * 448)),
// rounded to nearest even. One reciprocal a block instead of a division a value; the product differs from x / scale by a
// few roundings of 32 bits, far below the 2^-4 of an e4m3 step. A block holding an infinity or NaN gets scale and values NaN.
// Both kernels read each value once, keep it in registers between the amax and the rounding, and are bound by HBM.
#include <algorithm>
#include <type_traits>

#include "ops_common.cuh"

namespace reshard {
namespace ops {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kQThreads = 256;

template <typename T, int N>
struct alignas(sizeof(T) * N <= 16 ? sizeof(T) * N : 16) Pack {
  T v[N];
};

// N values at p (elements from `left` on are 0); `wide`: p is aligned to 16 bytes (or to N values, if fewer) and all are in.
template <typename T, int N>
__device__ __forceinline__ void load_values(const T *p, int left, bool wide, float (&x)[N]) {
  if (wide && left >= N) {
    const Pack<T, N> r = *reinterpret_cast<const Pack<T, N> *>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(r.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = i < left ? to_f32(p[i]) : 0.0f;
  }
}

// The 16-byte words that hold N values at p, wherever p is: ask() reads them (words that hold none of the `left` values
// are not read, `any` is in their place), take() shifts the values into place and clears those from `left` on. Rows that
// start anywhere are read as fast as aligned ones this way; value by value they took three times as long.
template <typename T, int N>
struct Shifted {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  static_assert(kWords % 4 == 0, "16-byte words");
  uint32_t w[kWords + 4];
  __device__ __forceinline__ void ask(const T *p, int left, const uint8_t *any) {
    const uintptr_t skip = reinterpret_cast<uintptr_t>(p) & 15;
    const uint8_t *from = reinterpret_cast<const uint8_t *>(p) - skip;
    const int end = left > 0 ? (int)skip + min(left, N) * (int)sizeof(T) : 0;        // bytes from there to the last value
#pragma unroll
    for (int i = 0; i < kWords + 4; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(4 * i < end ? from + 4 * i : any));
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
  __device__ __forceinline__ void take(const T *p, int left, uint32_t (&v)[kWords]) {
    const uint32_t skip = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
#pragma unroll
    for (int i = 0; i < kWords + 3; ++i) w[i] = skip & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < kWords + 2; ++i) w[i] = skip & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t x = sizeof(T) < 4 ? __funnelshift_r(w[i], w[i + 1], 8 * (skip & 3)) : w[i];
      const int have = left - i * (4 / (int)sizeof(T));          // values from this word on
      v[i] = have >= 4 / (int)sizeof(T) ? x : have > 0 ? x & 0xffffu : 0;
    }
  }
};
template <typename T>
__device__ __forceinline__ float value_of(const uint32_t *v, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(v[i]);
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
  else return __half2float(__ushort_as_half((uint16_t)(v[i / 2] >> (16 * (i & 1)))));
}
// A 16-byte word that holds a tensor's first value.
__device__ __forceinline__ const uint8_t *first_word(const void *p) {
  return reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15);
}

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

// out[t] = sum_j weights[t, j] * y[position[t, j]] in the order of j, slots without a place skipped; terms and sums of 32
// bits, one rounding. One thread 8 columns of a token; bound by the read of y: 8 slots a token, 8,192 x 2048, 83 us, 6.9 TB/s (loads of
// all eight slots before the sums: three times as long).
template <typename T>
__global__ void __launch_bounds__(kQThreads)
    reshard_combine_kernel(const float *y, int64_t y_stride, const int32_t *position, const float *weights, int64_t tokens, int k, int64_t cols,
                           T *out, int64_t out_stride, int chunks, bool wide) {
  grid_enter();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= tokens * chunks) return;
  const int64_t t = tokens * chunks <= 0xffffffffll ? (uint32_t)i / (uint32_t)chunks : i / chunks;
  const int64_t c = (i - t * chunks) * 8;
  const int left = (int)min((int64_t)8, cols - c);
  float sum[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) sum[u] = 0.0f;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int p = position[t * k + j];
    if (p < 0) continue;
    const float w = weights[t * k + j];
    float x[8];
    load_values<float, 8>(y + (int64_t)p * y_stride + c, left, wide, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) sum[u] = fmaf(w, x[u], sum[u]);
  }
  T *to = out + t * out_stride + c;
  if (wide && left >= 8) {
    Pack<T, 8> r;
#pragma unroll
    for (int u = 0; u < 8; ++u) r.v[u] = from_f32<T>(sum[u]);
    *reinterpret_cast<Pack<T, 8> *>(to) = r;
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (u < left) to[u] = from_f32<T>(sum[u]);
  }
}

bool aligned16(const void *p, int64_t stride, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride * bytes) % 16 == 0;
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

int enqueue_combine(const float *y, int64_t y_stride, const int32_t *position, const float *weights, int64_t tokens, int k, int64_t cols,
                    void *out, int dtype, int64_t out_stride, cudaStream_t stream) {
  if (tokens == 0 || cols == 0) return RESHARD_OK;
  const int chunks = (int)((cols + 7) / 8), es = element_bytes(dtype);
  const int block = tokens * chunks <= 32768 ? 64 : kQThreads;      // a few tokens' columns spread over the SMs
  const dim3 grid((unsigned)((tokens * chunks + block - 1) / block));
  const bool wide = aligned16(y, y_stride, 4) && aligned16(out, out_stride, es);
  cudaError_t e;
  auto go = [&](auto t) {
    using T = decltype(t);
    return launch(reshard_combine_kernel<T>, grid, block, 0, 1, stream, y, y_stride, position, weights, tokens, k, cols,
                  static_cast<T *>(out), out_stride, chunks, wide);
  };
  if (dtype == RESHARD_F32) e = go(float());
  else if (dtype == RESHARD_BF16) e = go(__nv_bfloat16());
  else e = go(__half());
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_combine_kernel");
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
