// Rows moved by an index: tokens to their experts' places and back with weights, the gradients of both, and the lookup of
// a vocabulary's shard.
//
// With the sort (order, position) of the slots s = t * k + j that reshard_dispatch gives:
//   permute           y[position[s]] = x[t]                    its gradient  dx[t] = sum_j dy[position[s]]: combine without weights
//   combine           out[t] = sum_j w[s] y[position[s]]
//   combine backward  dy[position[s]] = w[s] dout[t],  dw[s] = <dout[t], y[position[s]]>
//   embedding         out[t] = scale * table[ids[t] - first], 0 for the rows of other shards
// A place belongs to the slot that order names and whose position it is: two slots never write one row, whatever the two
// arrays hold, and a place that belongs to none is known by reading (its gradient is 0). Places outside the rows are none.
//
// Nothing is computed that HBM would wait for: each row is read and written once, in pieces of 16 bytes, with enough of
// them in flight. Sums are fp32 in the order of j, dot products fp32 in a fixed order.
#include <algorithm>

#include "ops_common.cuh"
#include "values.cuh"

namespace reshard {
namespace ops {

namespace {

constexpr int kRowThreads = 256;
constexpr int kAhead = 4;                        // pieces of a lane in flight together
constexpr int kSpan = 32 * kAhead;               // pieces of a row that a warp moves

// Slot s's place, -1 if it has none among `rows`.
__device__ __forceinline__ int place_of(const int32_t *position, int64_t s, int64_t rows) {
  const int p = position[s];
  return p >= 0 && p < rows ? p : -1;
}

// ---------------------------------------------------------------------------------------------------------- permute --

struct Permute {
  const void *x;
  int64_t tokens, cols, stride;      // cols and strides of the kernel of whole pieces: in pieces of 16 bytes
  const int32_t *order, *position;
  int k;
  void *out;
  int64_t rows, out_stride;
  int spans;                         // warps a row (a slot's row, where rows start anywhere)
};

// Rows of whole 16-byte pieces: a warp reads 2 KB of a token's row once and writes it to each of its places.
__global__ void __launch_bounds__(kRowThreads) reshard_permute_kernel(Permute a) {
  grid_enter();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / a.spans;
  if (t >= a.tokens) return;
  const int64_t c0 = (w - t * a.spans) * kSpan + lane;
  const uint4 *const from = static_cast<const uint4 *>(a.x) + t * a.stride;
  uint4 v[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (c0 + 32 * u < a.cols) v[u] = __ldg(from + c0 + 32 * u);
  for (int j0 = 0; j0 < a.k; j0 += 32) {
    int mine = -1;
    if (j0 + lane < a.k) {
      const int64_t s = t * a.k + j0 + lane;
      mine = place_of(a.position, s, a.rows);
      if (mine >= 0 && a.order[mine] != s) mine = -1;
    }
    const int n = min(32, a.k - j0);
    for (int j = 0; j < n; ++j) {
      const int p = __shfl_sync(kFull, mine, j);
      if (p < 0) continue;
      uint4 *const to = static_cast<uint4 *>(a.out) + (int64_t)p * a.out_stride;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + 32 * u < a.cols) to[c0 + 32 * u] = v[u];
    }
  }
}

// Pieces [first, first + kSpan) of a row, copied (times `scale`, where scaled) or, without a source, zeroed.
template <typename T, bool Wide, bool Scaled>
__device__ __forceinline__ void move_span(const T *from, T *to, int64_t cols, int64_t first, int lane, float scale) {
  Eight<T, Wide> v[kAhead];
  int64_t c[kAhead];
  bool whole[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    c[u] = piece_start<T, Wide>(first + lane + 32 * u, to);
    whole[u] = c[u] >= 0 && c[u] + 8 <= cols;
    if (from && whole[u]) v[u].ask(from + c[u]);
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    if (whole[u]) {
      if (Scaled && from) {
        float x[8];
        v[u].take(from + c[u], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= scale;
        store_eight(to + c[u], x);
      } else {
        *reinterpret_cast<Pack<T, 8> *>(to + c[u]) = from ? v[u].bits(from + c[u]) : Pack<T, 8>{};
      }
    } else if (c[u] < cols) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c[u] + i >= 0 && c[u] + i < cols) to[c[u] + i] = from ? (Scaled ? from_f32<T>(to_f32(from[c[u] + i]) * scale) : from[c[u] + i]) : from_f32<T>(0.0f);
    }
  }
}

// Rows that start anywhere: a warp a piece of a slot's row, which starts elsewhere than the token's does.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) reshard_permute_any_kernel(Permute a) {
  grid_enter();
  const int64_t w = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t s = w / a.spans;
  if (s >= a.tokens * a.k) return;
  const int p = place_of(a.position, s, a.rows);
  if (p < 0 || a.order[p] != s) return;
  move_span<T, false, false>(static_cast<const T *>(a.x) + s / a.k * a.stride, static_cast<T *>(a.out) + (int64_t)p * a.out_stride, a.cols,
                             (w - s * a.spans) * kSpan, threadIdx.x & 31, 1.0f);
}

// -------------------------------------------------------------------------------------------------------- embedding --

struct Lookup {
  const void *ids;
  bool wide_ids;                     // 64 bits
  int64_t tokens;
  const void *table;
  int64_t first, rows, cols, stride;
  float scale;
  void *out;
  int64_t out_stride;
  int spans;
};

template <typename T, bool Wide, bool Scaled>
__global__ void __launch_bounds__(kRowThreads) reshard_embedding_kernel(Lookup a) {
  grid_enter();
  const int64_t w = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = w / a.spans;
  if (t >= a.tokens) return;
  const int64_t id = a.wide_ids ? static_cast<const int64_t *>(a.ids)[t] : static_cast<const int32_t *>(a.ids)[t];
  const bool here = id >= a.first && id - a.first < a.rows;
  move_span<T, Wide, Scaled>(here ? static_cast<const T *>(a.table) + (id - a.first) * a.stride : nullptr,
                             static_cast<T *>(a.out) + t * a.out_stride, a.cols, (w - t * a.spans) * kSpan, threadIdx.x & 31, a.scale);
}

// ---------------------------------------------------------------------------------------------------------- combine --

// One thread eight columns of a token; bound by the read of y: 8 slots a token, 8,192 x 2048 fp32, 83 us, 6.9 TB/s (loads of all
// eight slots before the sums: three times as long).
template <typename TY, typename TO, bool Wide>
__global__ void __launch_bounds__(kRowThreads)
    reshard_combine_kernel(const TY *y, int64_t rows, int64_t y_stride, const int32_t *position, const float *weights, int64_t tokens, int k,
                           int64_t cols, TO *out, int64_t out_stride, int pieces) {
  grid_enter();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= tokens * pieces) return;
  const int64_t t = tokens * pieces <= 0xffffffffll ? (uint32_t)i / (uint32_t)pieces : i / pieces;
  TO *const to = out + t * out_stride;
  const int64_t c = piece_start<TO, Wide>(i - t * pieces, to);
  if (c >= cols) return;
  float sum[8] = {};
  const bool whole = c >= 0 && c + 8 <= cols;
#pragma unroll 4
  for (int j = 0; j < k; ++j) {
    const int p = place_of(position, t * k + j, rows);
    if (p < 0) continue;
    const float w = weights ? weights[t * k + j] : 1.0f;
    const TY *const from = y + (int64_t)p * y_stride + c;
    float x[8];
    if (whole) {
      Eight<TY, Wide> v;
      v.ask(from);
      v.take(from, x);
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = c + u >= 0 && c + u < cols ? to_f32(from[u]) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) sum[u] = fmaf(w, x[u], sum[u]);
  }
  if (whole) {
    store_eight(to + c, sum);
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (c + u >= 0 && c + u < cols) to[c + u] = from_f32<TO>(sum[u]);
  }
}

// ------------------------------------------------------------------------------------------------- combine backward --

struct CombineBackward {
  const void *grad;                  // [tokens, cols]
  int64_t grad_stride;
  const void *y;
  int64_t rows, cols, y_stride;
  const int32_t *order, *position;
  const float *weights;              // NULL: 1
  int64_t tokens;
  int k;
  void *grad_y;                      // NULL: not asked for
  int64_t grad_y_stride;
  float *grad_weights;               // NULL: not asked for
  int pieces;
};

// A warp a slot: the token's gradient (which the k warps of a token share in L1), its row of y, one row written, and the
// dot product by shuffles. Warp i also zeroes row i of the gradient if no slot owns it.
template <typename TG, typename TY, bool Wide>
__global__ void __launch_bounds__(kRowThreads) reshard_combine_backward_kernel(CombineBackward a) {
  grid_enter();
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  const int64_t slots = a.tokens * a.k;
  if (a.grad_y && i < a.rows) {
    const int64_t s = a.order[i];      // not written behind the last place: whatever it holds there is no owner
    if (s < 0 || s >= slots || a.position[s] != i)
      for (int c = 0; c < a.pieces; c += kSpan) move_span<TY, Wide, false>(nullptr, static_cast<TY *>(a.grad_y) + i * a.grad_y_stride, a.cols, c, lane, 1.0f);
  }
  if (i >= slots) return;
  const int p = place_of(a.position, i, a.rows);
  float dot = 0.0f;
  if (p >= 0) {
    const TG *const g = static_cast<const TG *>(a.grad) + i / a.k * a.grad_stride;
    const TY *const y = a.grad_weights ? static_cast<const TY *>(a.y) + (int64_t)p * a.y_stride : nullptr;
    TY *const to = a.grad_y && a.order[p] == i ? static_cast<TY *>(a.grad_y) + (int64_t)p * a.grad_y_stride : nullptr;
    const float w = a.weights ? a.weights[i] : 1.0f;
    // Where rows start anywhere, the pieces are those of a dense gradient of y whether it is written or not, dense or not: they
    // set the order of the dot product.
    const TY *const dense = reinterpret_cast<const TY *>(p * a.cols * (int64_t)sizeof(TY));
    for (int c1 = lane; c1 < a.pieces; c1 += kSpan) {
      Eight<TG, Wide> gv[kAhead];
      Eight<TY, Wide> yv[kAhead];
      int64_t c[kAhead];
      bool whole[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        c[u] = piece_start<TY, Wide>(c1 + 32 * u, dense);
        whole[u] = c[u] >= 0 && c[u] + 8 <= a.cols;
        if (whole[u]) {
          gv[u].ask(g + c[u]);
          if (y) yv[u].ask(y + c[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        float x[8], z[8] = {};
        if (whole[u]) {
          gv[u].take(g + c[u], x);
          if (y) yv[u].take(y + c[u], z);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool in = c[u] + e >= 0 && c[u] + e < a.cols;
            x[e] = in ? to_f32(g[c[u] + e]) : 0.0f;
            z[e] = in && y ? to_f32(y[c[u] + e]) : 0.0f;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dot = fmaf(x[e], z[e], dot);
          x[e] *= w;
        }
        if (!to) continue;
        if (whole[u] && (Wide || (reinterpret_cast<uintptr_t>(to + c[u]) & 15) == 0)) {
          store_eight(to + c[u], x);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c[u] + e >= 0 && c[u] + e < a.cols) to[c[u] + e] = from_f32<TY>(x[e]);
        }
      }
    }
  }
  if (!a.grad_weights) return;
#pragma unroll
  for (int o = 16; o; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
  if (lane == 0) a.grad_weights[i] = dot;
}

int64_t warps_grid(int64_t warps) { return (warps + kRowThreads / 32 - 1) / (kRowThreads / 32); }

// Warps of a row of so many pieces.
int spans_of(int64_t pieces) { return (int)((pieces + kSpan - 1) / kSpan); }

int launched(cudaError_t e, const char *what) { return e == cudaSuccess ? RESHARD_OK : cuda_error(e, what); }

}  // namespace

int enqueue_combine(const Combine &a, cudaStream_t stream) {
  if (a.tokens == 0 || a.cols == 0) return RESHARD_OK;
  const bool wide = aligned16(a.y, a.y_stride, element_bytes(a.dtype)) && aligned16(a.out, a.out_stride, element_bytes(a.out_dtype));
  return launched(by_type(a.dtype, [&](auto y) {
    using TY = decltype(y);
    return by_type(a.out_dtype, [&](auto o) {
      using TO = decltype(o);
      const int64_t pieces = piece_count<TO>(a.cols, wide);
      const int block = a.tokens * pieces <= 32768 ? 64 : kRowThreads;      // a few tokens' columns spread over the SMs
      const dim3 grid((unsigned)((a.tokens * pieces + block - 1) / block));
      return launch(wide ? reshard_combine_kernel<TY, TO, true> : reshard_combine_kernel<TY, TO, false>, grid, block, 0, 1, stream,
                    static_cast<const TY *>(a.y), a.rows, a.y_stride, a.position, a.weights, a.tokens, a.k, a.cols, static_cast<TO *>(a.out),
                    a.out_stride, (int)pieces);
    });
  }), "launching reshard_combine_kernel");
}

namespace {

// What the calls on a sort have in common. A grid holds 2^31 - 1 CTAs.
void check_slots(Checks &c, int64_t tokens, int64_t cols, int k, int64_t rows) {
  c.invalid(tokens < 0 || cols < 0 || rows < 0 || k < 1, "tokens, cols and rows must be >= 0 and k >= 1");
  c.unsupported(tokens > RESHARD_MAX_EXTENT || cols > RESHARD_MAX_EXTENT || rows > RESHARD_MAX_SLOTS, "tokens, cols or rows above 2^30");
  if (c.ok()) {
    c.unsupported(tokens * k > RESHARD_MAX_SLOTS, "more than 2^30 slots");
    c.unsupported((double)std::max<int64_t>(tokens * k, rows) * (double)(cols / 256 + 1) > 8.0 * INT32_MAX, "too many rows and columns for one launch");
  }
}

}  // namespace
}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int reshard_permute(const void *x, int dtype, int64_t tokens, int64_t cols, int64_t row_stride, const int32_t *order,
                               const int32_t *position, int k, void *out, int64_t rows, int64_t out_stride, reshard_stream_t stream_) try {
  Checks c("reshard_permute");
  check_slots(c, tokens, cols, k, rows);
  c.invalid(!element_bytes(dtype), "dtype must be BF16, F16 or F32");
  c.invalid(row_stride < cols || out_stride < cols, "a row stride is shorter than the row");
  const int es = element_bytes(dtype);
  const bool work = tokens > 0 && cols > 0 && rows > 0;
  if (work && c.ok()) {
    c.pointer(x, "x", (uintptr_t)es);
    c.pointer(order, "order", 4);
    c.pointer(position, "position", 4);
    c.pointer(out, "out", (uintptr_t)es);
  }
  if (!c.ok()) return c.report();
  if (!work) return RESHARD_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  Permute a{x, tokens, cols, row_stride, order, position, k, out, rows, out_stride, 0};
  if (aligned16(x, row_stride, es) && aligned16(out, out_stride, es) && cols * es % 16 == 0) {
    a.cols = cols * es / 16, a.stride = row_stride * es / 16, a.out_stride = out_stride * es / 16;
    a.spans = spans_of(a.cols);
    return launched(launch(reshard_permute_kernel, dim3((unsigned)warps_grid(tokens * a.spans)), kRowThreads, 0, 1, stream, a), "launching reshard_permute_kernel");
  }
  // values are copied as they are: the types of a size share a kernel
  a.spans = spans_of(es == 4 ? piece_count<float>(cols, false) : piece_count<__half>(cols, false));
  return launched(launch(es == 4 ? reshard_permute_any_kernel<float> : reshard_permute_any_kernel<__half>,
                         dim3((unsigned)warps_grid(tokens * k * a.spans)), kRowThreads, 0, 1, stream, a), "launching reshard_permute_any_kernel");
} OPS_CATCH

extern "C" int reshard_combine(const void *y, int dtype, int64_t rows, int64_t cols, int64_t row_stride, const int32_t *position,
                               const float *weights, int64_t tokens, int k, void *out, int out_dtype, int64_t out_stride,
                               reshard_stream_t stream) try {
  Checks c("reshard_combine");
  check_slots(c, tokens, cols, k, rows);
  c.invalid(!element_bytes(dtype) || !element_bytes(out_dtype), "dtype and out_dtype must be BF16, F16 or F32");
  c.invalid(row_stride < cols || out_stride < cols, "a row stride is shorter than the row");
  if (tokens > 0 && cols > 0 && c.ok()) {
    if (rows > 0) c.pointer(y, "y", (uintptr_t)element_bytes(dtype));      // without rows no slot has a place
    c.pointer(position, "position", 4);
    if (weights) c.pointer(weights, "weights", 4);
    c.pointer(out, "out", (uintptr_t)element_bytes(out_dtype));
  }
  if (!c.ok()) return c.report();
  return enqueue_combine(Combine{y, dtype, rows, row_stride, position, weights, tokens, k, cols, out, out_dtype, out_stride},
                         reinterpret_cast<cudaStream_t>(stream));
} OPS_CATCH

extern "C" int reshard_combine_backward(const void *grad, int grad_dtype, int64_t grad_stride, const void *y, int dtype, int64_t rows,
                                        int64_t cols, int64_t row_stride, const int32_t *order, const int32_t *position,
                                        const float *weights, int64_t tokens, int k, void *grad_y, int64_t grad_y_stride,
                                        float *grad_weights, reshard_stream_t stream) try {
  Checks c("reshard_combine_backward");
  check_slots(c, tokens, cols, k, rows);
  c.invalid(!element_bytes(dtype) || !element_bytes(grad_dtype), "dtype and grad_dtype must be BF16, F16 or F32");
  c.invalid(grad_stride < cols || (grad_weights && row_stride < cols) || (grad_y && grad_y_stride < cols), "a row stride is shorter than the row");
  const int es = element_bytes(dtype);
  const int64_t warps = !c.ok() ? 0 : std::max(grad_weights || grad_y ? tokens * k : 0, grad_y ? rows : 0);
  if (warps > 0 && c.ok()) {
    if (tokens > 0) {
      if (cols > 0) c.pointer(grad, "grad", (uintptr_t)element_bytes(grad_dtype));
      if (cols > 0 && rows > 0 && grad_weights) c.pointer(y, "y", (uintptr_t)es);
      c.pointer(position, "position", 4);
      if (weights) c.pointer(weights, "weights", 4);
    }
    if (grad_y && rows > 0) {
      c.pointer(order, "order", 4);
      c.pointer(grad_y, "grad_y", (uintptr_t)es);
    }
    if (grad_weights && tokens > 0) c.pointer(grad_weights, "grad_weights", 4);
  }
  if (!c.ok()) return c.report();
  if (warps == 0) return RESHARD_OK;
  const bool wide = aligned16(grad, grad_stride, element_bytes(grad_dtype)) && (!grad_weights || aligned16(y, row_stride, es)) &&
                    (!grad_y || aligned16(grad_y, grad_y_stride, es)) && cols * es % 16 == 0;
  const CombineBackward a{grad, grad_stride, y, rows, cols, row_stride, order, position, weights, tokens, k, grad_y, grad_y_stride, grad_weights,
                          (int)(es == 4 ? piece_count<float>(cols, wide) : piece_count<__half>(cols, wide))};
  return launched(by_type(grad_dtype, [&](auto g) {
    using TG = decltype(g);
    return by_type(dtype, [&](auto t) {
      using TY = decltype(t);
      return launch(wide ? reshard_combine_backward_kernel<TG, TY, true> : reshard_combine_backward_kernel<TG, TY, false>,
                    dim3((unsigned)warps_grid(warps)), kRowThreads, 0, 1, reinterpret_cast<cudaStream_t>(stream), a);
    });
  }), "launching reshard_combine_backward_kernel");
} OPS_CATCH

extern "C" int reshard_embedding(const void *ids, int id_bits, int64_t tokens, const void *table, int dtype, int64_t first_row, int64_t rows,
                                 int64_t cols, int64_t row_stride, float scale, void *out, int64_t out_stride, reshard_stream_t stream) try {
  Checks c("reshard_embedding");
  c.invalid(tokens < 0 || rows < 0 || cols < 0 || first_row < 0, "tokens, rows, cols and first_row must be >= 0");
  c.unsupported(tokens > RESHARD_MAX_SLOTS || rows > RESHARD_MAX_EXTENT || cols > RESHARD_MAX_EXTENT, "tokens, rows or cols above 2^30");
  c.invalid(id_bits != 32 && id_bits != 64, "id_bits must be 32 or 64");
  c.invalid(!element_bytes(dtype), "dtype must be BF16, F16 or F32");
  c.invalid(row_stride < cols || out_stride < cols, "a row stride is shorter than the row");
  const int es = element_bytes(dtype);
  const bool work = tokens > 0 && cols > 0;
  if (c.ok()) c.unsupported((double)tokens * (double)(cols / 256 + 1) > 8.0 * INT32_MAX, "too many rows and columns for one launch");
  if (work && c.ok()) {
    c.pointer(ids, "ids", (uintptr_t)(id_bits / 8));
    if (rows > 0) c.pointer(table, "table", (uintptr_t)es);
    c.pointer(out, "out", (uintptr_t)es);
  }
  if (!c.ok()) return c.report();
  if (!work) return RESHARD_OK;
  const bool wide = aligned16(table, row_stride, es) && aligned16(out, out_stride, es);
  Lookup a{ids, id_bits == 64, tokens, table, first_row, rows, cols, row_stride, scale, out, out_stride, 0};
  return launched(by_type(dtype, [&](auto t) {
    using T = decltype(t);
    a.spans = spans_of(piece_count<T>(cols, wide));
    auto *kernel = wide ? scale == 1.0f ? reshard_embedding_kernel<T, true, false> : reshard_embedding_kernel<T, true, true>
                        : scale == 1.0f ? reshard_embedding_kernel<T, false, false> : reshard_embedding_kernel<T, false, true>;
    return launch(kernel, dim3((unsigned)warps_grid(tokens * a.spans)), kRowThreads, 0, 1, reinterpret_cast<cudaStream_t>(stream), a);
  }), "launching reshard_embedding_kernel");
} OPS_CATCH
