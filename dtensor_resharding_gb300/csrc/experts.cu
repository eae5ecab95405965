// The calls that put the operator kernels together: the product alone, with its rows' quantization, and the routed
// expert feed-forward. Host code only; everything is enqueued on the caller's stream in the caller's workspace.
#include <algorithm>

#include "ops_common.cuh"

namespace reshard {
namespace ops {

void Checks::pointer(const void *p, const char *name, uintptr_t align) {
  if (!p) return violation(RESHARD_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (reinterpret_cast<uintptr_t>(p) % align)
    return violation(RESHARD_ERR_INVALID_ARG, std::string(name) + " is not aligned to " + std::to_string(align) + " bytes");
  cudaPointerAttributes a{};
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return violation(RESHARD_ERR_INVALID_ARG, std::string(name) + " is not a pointer the device can dereference");
  }
  if (a.type == cudaMemoryTypeUnregistered) return violation(RESHARD_ERR_INVALID_ARG, std::string(name) + " is pageable host memory");
  if (a.type == cudaMemoryTypeDevice) {
    if (device_ < 0 && cudaGetDevice(&device_) != cudaSuccess) device_ = -1;
    if (device_ >= 0 && a.device != device_) violation(RESHARD_ERR_INVALID_ARG, std::string(name) + " is memory of device " + std::to_string(a.device));
  }
}

int device_sms(int *sms) {
  static thread_local int dev_seen = -1, seen = 0;
  int dev = 0;
  OPS_CUDA(cudaGetDevice(&dev));
  if (dev != dev_seen) {
    OPS_CUDA(cudaDeviceGetAttribute(&seen, cudaDevAttrMultiProcessorCount, dev));
    dev_seen = dev;
  }
  *sms = seen;
  return RESHARD_OK;
}

namespace {

constexpr int64_t kAlign = 256;
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t blocks_of(int64_t v) { return (v + kScaleBlock - 1) / kScaleBlock; }

// Quantized rows in a workspace: values at a 16-byte pitch, scales block by block (a block's rows side by side, so that
// the product's threads, one a row, read them in one line).
struct QuantizedRows {
  int64_t pitch, values, scales;
  QuantizedRows(int64_t rows, int64_t cols) : pitch(up(cols, 16)), values(up(rows * pitch, kAlign)), scales(up(rows * blocks_of(cols) * 4, kAlign)) {}
  int64_t bytes() const { return values + scales; }
};

struct ExpertLayout {
  int64_t slots, offsets, order, position, y;
  QuantizedRows x, h;
  ExpertLayout(int64_t tokens, int k, int experts, int64_t hidden, int64_t ffn)
      : slots(tokens * k), offsets(up(4 * (experts + 1), kAlign)), order(up(4 * slots, kAlign)), position(order),
        y(up(slots * up(hidden, 16) * 4, kAlign)), x(product_gathers(slots, experts) ? tokens : slots, hidden), h(slots, ffn) {}
  int64_t bytes() const { return offsets + order + position + y + x.bytes() + h.bytes(); }
};

void check_weight(Checks &c, const void *w, int64_t batch, int64_t batch_stride, int64_t rows, int64_t cols, int64_t stride, const char *name) {
  c.pointer(w, name, 16);
  c.invalid(stride < cols, "a weight row stride is shorter than the row");
  c.unsupported(stride % 16 != 0, "a weight row stride is not a multiple of 16 bytes (lay the rows out with a padded pitch)");
  if (batch > 1) {
    c.unsupported(batch_stride < (rows - 1) * stride + cols, "weight matrices interleave or overlap (lay them out one after another)");
    c.unsupported(batch_stride % 16 != 0, "a weight batch stride is not a multiple of 16 bytes");
  }
}

// A word as an int; what does not fit stays out of every range that the calls accept.
int as_int(int64_t v) { return (int)std::max<int64_t>(INT32_MIN, std::min<int64_t>(INT32_MAX, v)); }

// The batch stride a tensor map takes where there is one matrix only.
int64_t map_batch(int64_t batch, int64_t batch_stride, int64_t rows, int64_t stride) { return batch > 1 ? batch_stride : rows * stride; }

}  // namespace
}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int reshard_matmul_fp8(const void *a, int64_t a_stride, const float *a_scale, int64_t a_scale_row, int64_t a_scale_block,
                                  const void *w, int64_t w_batch_stride, int64_t w_stride, const float *w_scale, const int32_t *offsets,
                                  int groups, int64_t m, int64_t n, int64_t k, void *out, int out_dtype, int64_t out_stride,
                                  reshard_stream_t stream) try {
  Checks c("reshard_matmul_fp8");
  c.invalid(m < 0 || n < 0 || k < 1, "m and n must be >= 0 and k >= 1");
  c.unsupported(m > RESHARD_MAX_EXTENT || n > RESHARD_MAX_EXTENT || k > RESHARD_MAX_EXTENT, "m, n or k above 2^30");
  c.invalid(groups < 1 || (!offsets && groups != 1), "groups must be >= 1, and 1 without offsets");
  c.unsupported(groups > RESHARD_MAX_GROUPS, "more than 512 groups");
  c.invalid(!element_bytes(out_dtype), "out_dtype must be BF16, F16 or F32");
  c.invalid(a_stride < k || out_stride < n, "a row stride is shorter than the row");
  c.unsupported(a_stride % 16 != 0, "a's row stride is not a multiple of 16 bytes");
  c.invalid(a_scale_row < 0 || a_scale_block < 0, "scale strides must not be negative");
  if (m > 0 && n > 0 && c.ok()) {
    c.pointer(a, "a", 16);
    c.pointer(a_scale, "a_scale", 4);
    check_weight(c, w, groups, w_batch_stride, n, k, w_stride, "w");
    c.pointer(w_scale, "w_scale", 4);
    if (offsets) c.pointer(offsets, "offsets", 4);
    c.pointer(out, "out", (uintptr_t)element_bytes(out_dtype));
  }
  if (!c.ok()) return c.report();
  if (m == 0 || n == 0) return RESHARD_OK;
  Product p{};
  p.a = static_cast<const uint8_t *>(a), p.a_stride = a_stride, p.a_scale = a_scale, p.as_row = a_scale_row, p.as_block = a_scale_block;
  p.w = static_cast<const uint8_t *>(w), p.w_batch = map_batch(groups, w_batch_stride, n, w_stride), p.w_stride = w_stride, p.w_scale = w_scale;
  p.offsets = offsets, p.groups = groups, p.m = m, p.n = n, p.k = k;
  p.out = out, p.out_dtype = out_dtype, p.out_stride = out_stride;
  return enqueue_product(p, reinterpret_cast<cudaStream_t>(stream));
} OPS_CATCH

extern "C" int64_t reshard_linear_fp8_workspace(int64_t m, int64_t k) {
  if (m < 0 || k < 0 || m > RESHARD_MAX_EXTENT || k > RESHARD_MAX_EXTENT || product_quantizes(m, k)) return 0;
  return QuantizedRows(m, k).bytes();
}

extern "C" int reshard_linear_fp8(const void *x, int dtype, int64_t m, int64_t k, int64_t row_stride, const void *w, int64_t w_stride,
                                  const float *w_scale, int64_t n, void *out, int64_t out_stride, void *workspace, int64_t workspace_bytes,
                                  reshard_stream_t stream_) try {
  Checks c("reshard_linear_fp8");
  c.invalid(m < 0 || n < 0 || k < 1, "m and n must be >= 0 and k >= 1");
  c.unsupported(m > RESHARD_MAX_EXTENT || n > RESHARD_MAX_EXTENT || k > RESHARD_MAX_EXTENT, "m, n or k above 2^30");
  c.invalid(!element_bytes(dtype), "dtype must be BF16, F16 or F32");
  c.invalid(row_stride < k || out_stride < n, "a row stride is shorter than the row");
  if (m > 0 && n > 0 && c.ok()) {
    c.pointer(x, "x", (uintptr_t)element_bytes(dtype));
    check_weight(c, w, 1, 0, n, k, w_stride, "w");
    c.pointer(w_scale, "w_scale", 4);
    c.pointer(out, "out", (uintptr_t)element_bytes(dtype));
    if (reshard_linear_fp8_workspace(m, k) > 0) c.pointer(workspace, "workspace", kAlign);
    c.invalid(workspace_bytes < reshard_linear_fp8_workspace(m, k), "the workspace is smaller than reshard_linear_fp8_workspace");
  }
  if (!c.ok()) return c.report();
  if (m == 0 || n == 0) return RESHARD_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  Product p{};
  if (product_quantizes(m, k)) {
    p.x = x, p.a_stride = row_stride;
  } else {
    const QuantizedRows l(m, k);
    uint8_t *q = static_cast<uint8_t *>(workspace);
    float *scale = reinterpret_cast<float *>(q + l.values);
    const int rc = enqueue_quantize_rows(Rows{x, dtype, m, k, row_stride, q, l.pitch, scale, 1, m}, stream);
    if (rc) return rc;
    p.a = q, p.a_stride = l.pitch, p.a_scale = scale, p.as_row = 1, p.as_block = m;
    p.early = true;
  }
  p.w = static_cast<const uint8_t *>(w), p.w_batch = n * w_stride, p.w_stride = w_stride, p.w_scale = w_scale;
  p.m = m, p.n = n, p.k = k;
  p.out = out, p.out_dtype = dtype, p.out_stride = out_stride;
  return enqueue_product(p, stream);
} OPS_CATCH

extern "C" int64_t reshard_experts_fp8_workspace(int64_t tokens, int k, int experts, int64_t hidden, int64_t ffn, int dtype) {
  if (tokens < 0 || k < 1 || experts < 1 || hidden < 0 || ffn < 0 || !element_bytes(dtype)) return 0;
  // what the call refuses has no size, and none of the sums below passes 63 bits
  if (experts > RESHARD_MAX_GROUPS || tokens > RESHARD_MAX_SLOTS / k || hidden > RESHARD_MAX_EXTENT / 2 || ffn > RESHARD_MAX_EXTENT / 2) return 0;
  return ExpertLayout(tokens, k, experts, hidden, ffn).bytes();
}

extern "C" int reshard_experts_fp8(const void *x, int dtype, int64_t tokens, int64_t hidden, int64_t row_stride, const int32_t *ids,
                                   const float *weights, int k, int first_expert, int experts, int64_t ffn, const void *w13,
                                   int64_t w13_batch_stride, int64_t w13_stride, const float *w13_scale, const void *w2,
                                   int64_t w2_batch_stride, int64_t w2_stride, const float *w2_scale, void *out, int64_t out_stride,
                                   void *workspace, int64_t workspace_bytes, reshard_stream_t stream_) try {
  Checks c("reshard_experts_fp8");
  c.invalid(tokens < 0 || hidden < 1 || ffn < 1 || k < 1, "tokens must be >= 0, hidden, ffn and k >= 1");
  c.invalid(first_expert < 0 || experts < 1, "first_expert must be >= 0 and experts >= 1");
  c.unsupported(experts > RESHARD_MAX_GROUPS, "more than 512 experts on this side");
  c.unsupported(tokens > RESHARD_MAX_EXTENT || hidden > RESHARD_MAX_EXTENT / 2 || ffn > RESHARD_MAX_EXTENT / 2, "tokens, hidden or ffn above 2^29");
  if (c.ok()) c.unsupported(tokens * k > RESHARD_MAX_SLOTS, "more than 2^30 slots");
  c.unsupported(ffn % kScaleBlock != 0, "ffn is not a multiple of 128: a scale block would hold gate and up rows");
  c.invalid(!element_bytes(dtype), "dtype must be BF16, F16 or F32");
  c.invalid(row_stride < hidden || out_stride < hidden, "a row stride is shorter than the row");
  if (tokens > 0 && c.ok()) {
    c.pointer(x, "x", (uintptr_t)element_bytes(dtype));
    c.pointer(ids, "ids", 4);
    c.pointer(weights, "weights", 4);
    check_weight(c, w13, experts, w13_batch_stride, 2 * ffn, hidden, w13_stride, "w13");
    c.pointer(w13_scale, "w13_scale", 4);
    check_weight(c, w2, experts, w2_batch_stride, hidden, ffn, w2_stride, "w2");
    c.pointer(w2_scale, "w2_scale", 4);
    c.pointer(out, "out", (uintptr_t)element_bytes(dtype));
    c.pointer(workspace, "workspace", kAlign);
    c.invalid(workspace_bytes < reshard_experts_fp8_workspace(tokens, k, experts, hidden, ffn, dtype),
              "the workspace is smaller than reshard_experts_fp8_workspace");
  }
  if (!c.ok()) return c.report();
  if (tokens == 0) return RESHARD_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const ExpertLayout l(tokens, k, experts, hidden, ffn);
  uint8_t *at = static_cast<uint8_t *>(workspace);
  auto take = [&](int64_t bytes) { uint8_t *p = at; at += bytes; return p; };
  int32_t *offsets = reinterpret_cast<int32_t *>(take(l.offsets));
  int32_t *order = reinterpret_cast<int32_t *>(take(l.order));
  int32_t *position = reinterpret_cast<int32_t *>(take(l.position));
  float *y = reinterpret_cast<float *>(take(l.y));
  uint8_t *xq = take(l.x.values);
  float *xs = reinterpret_cast<float *>(take(l.x.scales));
  uint8_t *hq = take(l.h.values);
  float *hs = reinterpret_cast<float *>(take(l.h.scales));
  int rc = enqueue_dispatch(ids, l.slots, first_expert, experts, offsets, order, position, stream);
  if (rc) return rc;
  // Tokens are quantized once. With few rows an expert the first product gathers its rows of them; with many it reads them
  // in its own order, each written to every place it has (gathered loads, four rows each, took 566 us of 8,192 tokens'
  // product instead of 245; the copies take 28).
  const bool gathers = product_gathers(l.slots, experts);
  Rows r{x, dtype, tokens, hidden, row_stride, xq, l.x.pitch, xs, 1, gathers ? tokens : l.slots};
  if (!gathers) r.position = position, r.copies = k;
  if ((rc = enqueue_quantize_rows(r, stream))) return rc;
  Product p{};
  p.a = xq, p.a_stride = l.x.pitch, p.a_scale = xs, p.as_row = 1, p.as_block = r.scale_block;
  if (gathers) p.order = order, p.per_row = k, p.a_rows = tokens;
  p.w = static_cast<const uint8_t *>(w13), p.w_batch = map_batch(experts, w13_batch_stride, 2 * ffn, w13_stride), p.w_stride = w13_stride;
  p.w_scale = w13_scale, p.offsets = offsets, p.groups = experts, p.m = l.slots, p.n = ffn, p.k = hidden;
  p.early = true;      // behind the quantization; the sort before it has ended when that begins
  p.out = hq, p.out_stride = l.h.pitch, p.gated = true, p.out_scale = hs, p.os_row = 1, p.os_block = l.slots;
  if ((rc = enqueue_product(p, stream))) return rc;
  Product p2{};
  p2.a = hq, p2.a_stride = l.h.pitch, p2.a_scale = hs, p2.as_row = 1, p2.as_block = l.slots;
  p2.w = static_cast<const uint8_t *>(w2), p2.w_batch = map_batch(experts, w2_batch_stride, hidden, w2_stride), p2.w_stride = w2_stride;
  p2.w_scale = w2_scale, p2.offsets = offsets, p2.groups = experts, p2.m = l.slots, p2.n = hidden, p2.k = ffn;
  p2.early = true;
  // fp32 until the weighted sum: an expert's output can be beyond float16 where its share of the sum is not, and outputs that
  // cancel would leave their roundings. (16 bits there: 424 us instead of 506 for 8,192 tokens to 8 of 128 experts of 2048 x 768.)
  p2.out = y, p2.out_dtype = RESHARD_F32, p2.out_stride = up(hidden, 16);
  if ((rc = enqueue_product(p2, stream))) return rc;
  return enqueue_combine(y, up(hidden, 16), position, weights, tokens, k, hidden, out, dtype, out_stride, stream);
} OPS_CATCH

extern "C" int reshard_ops_call(int op, const reshard_word_t *a) try {
  if (!a) return fail(RESHARD_ERR_INVALID_ARG, "args is NULL");
  switch (op) {
    case RESHARD_OP_ROUTE:
      return reshard_route(reinterpret_cast<const void *>(a[0].i), as_int(a[1].i), a[2].i, as_int(a[3].i), a[4].i,
                           reinterpret_cast<const float *>(a[5].i), as_int(a[6].i), as_int(a[7].i), as_int(a[8].i), as_int(a[9].i),
                           as_int(a[10].i), as_int(a[11].i), (float)a[12].f, reinterpret_cast<float *>(a[13].i),
                           reinterpret_cast<int32_t *>(a[14].i), reinterpret_cast<reshard_stream_t>(a[15].i));
    case RESHARD_OP_ROUTE_BACKWARD:
      return reshard_route_backward(reinterpret_cast<const float *>(a[0].i), reinterpret_cast<const void *>(a[1].i),
                                    as_int(a[2].i), a[3].i, as_int(a[4].i), a[5].i, reinterpret_cast<const int32_t *>(a[6].i),
                                    as_int(a[7].i), as_int(a[8].i), as_int(a[9].i), (float)a[10].f, reinterpret_cast<void *>(a[11].i),
                                    a[12].i, reinterpret_cast<reshard_stream_t>(a[13].i));
    case RESHARD_OP_DISPATCH:
      return reshard_dispatch(reinterpret_cast<const int32_t *>(a[0].i), a[1].i, as_int(a[2].i), as_int(a[3].i),
                              reinterpret_cast<int32_t *>(a[4].i), reinterpret_cast<int32_t *>(a[5].i),
                              reinterpret_cast<int32_t *>(a[6].i), reinterpret_cast<reshard_stream_t>(a[7].i));
    case RESHARD_OP_QUANTIZE_ROWS:
      return reshard_quantize_rows(reinterpret_cast<const void *>(a[0].i), as_int(a[1].i), a[2].i, a[3].i, a[4].i,
                                   reinterpret_cast<void *>(a[5].i), a[6].i, reinterpret_cast<float *>(a[7].i), a[8].i, a[9].i,
                                   reinterpret_cast<reshard_stream_t>(a[10].i));
    case RESHARD_OP_QUANTIZE_BLOCKS:
      return reshard_quantize_blocks(reinterpret_cast<const void *>(a[0].i), as_int(a[1].i), a[2].i, a[3].i, a[4].i, a[5].i,
                                     a[6].i, reinterpret_cast<void *>(a[7].i), a[8].i, a[9].i,
                                     reinterpret_cast<float *>(a[10].i), reinterpret_cast<reshard_stream_t>(a[11].i));
    case RESHARD_OP_MATMUL_FP8:
      return reshard_matmul_fp8(reinterpret_cast<const void *>(a[0].i), a[1].i, reinterpret_cast<const float *>(a[2].i),
                                a[3].i, a[4].i, reinterpret_cast<const void *>(a[5].i), a[6].i, a[7].i,
                                reinterpret_cast<const float *>(a[8].i), reinterpret_cast<const int32_t *>(a[9].i),
                                as_int(a[10].i), a[11].i, a[12].i, a[13].i, reinterpret_cast<void *>(a[14].i), as_int(a[15].i),
                                a[16].i, reinterpret_cast<reshard_stream_t>(a[17].i));
    case RESHARD_OP_LINEAR_FP8:
      return reshard_linear_fp8(reinterpret_cast<const void *>(a[0].i), as_int(a[1].i), a[2].i, a[3].i, a[4].i,
                                reinterpret_cast<const void *>(a[5].i), a[6].i, reinterpret_cast<const float *>(a[7].i),
                                a[8].i, reinterpret_cast<void *>(a[9].i), a[10].i, reinterpret_cast<void *>(a[11].i), a[12].i,
                                reinterpret_cast<reshard_stream_t>(a[13].i));
    case RESHARD_OP_EXPERTS_FP8:
      return reshard_experts_fp8(reinterpret_cast<const void *>(a[0].i), as_int(a[1].i), a[2].i, a[3].i, a[4].i,
                                 reinterpret_cast<const int32_t *>(a[5].i), reinterpret_cast<const float *>(a[6].i),
                                 as_int(a[7].i), as_int(a[8].i), as_int(a[9].i), a[10].i, reinterpret_cast<const void *>(a[11].i),
                                 a[12].i, a[13].i, reinterpret_cast<const float *>(a[14].i),
                                 reinterpret_cast<const void *>(a[15].i), a[16].i, a[17].i,
                                 reinterpret_cast<const float *>(a[18].i), reinterpret_cast<void *>(a[19].i), a[20].i,
                                 reinterpret_cast<void *>(a[21].i), a[22].i, reinterpret_cast<reshard_stream_t>(a[23].i));
    default:
      return fail(RESHARD_ERR_INVALID_ARG, "unknown operator number");
  }
} OPS_CATCH
