// The global norm of many tensors, and their clipping: norm = sqrt(sum x^2), x * min(1, limit / (norm + 1e-6)).
//
// A list (reshard_tensors_create) keeps the tensors' places on the host. A launch takes up to kBatch of them as its argument,
// so that a call copies nothing to the device and allocates nothing there, and a captured one holds its list. A tensor is
// cut into units of one size (its head before the first 16-byte boundary belongs to the first); the CTAs of a launch share
// the units of all its tensors evenly, whatever the tensors' sizes, and look their first one up by bisection.
//
// Squares are summed over 64 bytes a thread at most in fp32, those sums in fp32 with their roundings carried along
// (two-sum), threads and CTAs in 64 bits in a fixed order: the norm is the correctly rounded one but for some 2^-24. Values
// whose squares leave fp32's range (beyond 2^50, or all of them below 2^-40) are summed in 64 bits instead.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "ops_common.cuh"
#include "values.cuh"

// The opaque list of the C ABI: host memory only.
struct reshard_tensors {
  struct Tensor {
    uintptr_t at;
    int64_t n;
    int dtype;
  };
  std::vector<Tensor> tensors;       // in the caller's order, empty ones among them
  int device = 0;
  bool overlap = false;              // some elements are in two tensors
  uintptr_t low = UINTPTR_MAX, high = 0;
  int64_t unit = 0;                  // elements
};

namespace reshard {
namespace ops {

namespace {

constexpr int kNormThreads = 256;
constexpr int kBatch = 1024;                      // tensors a launch
constexpr int kMaxCtas = 1024;                    // whose sums the workspace holds
constexpr int kUnitStep = kNormThreads * 8;       // a unit is a multiple of it
constexpr int kCtasPerSm = 4;
constexpr double kEps = 1e-6;

// Up to kBatch tensors: 28 KB of the 32 that a kernel's arguments may have.
struct Batch {
  uint64_t at[kBatch];
  uint64_t to[kBatch];               // where the clipped values go
  uint64_t n[kBatch];                // elements << 4 | type of `to` << 2 | type of `at`
  uint32_t first[kBatch + 1];        // units before the tensor's
  int count;
  int unit;
};
static_assert(sizeof(Batch) + 64 <= 32764, "a kernel's arguments");

int launched(cudaError_t e, const char *what) { return e == cudaSuccess ? RESHARD_OK : cuda_error(e, what); }

// The tensor that holds unit u.
__device__ __forceinline__ int find(const Batch &b, uint32_t u) {
  int in = 0, out = b.count;
  while (out - in > 1) {
    const int mid = (in + out) / 2;
    if (b.first[mid] <= u) in = mid;
    else out = mid;
  }
  return in;
}

// A sum of squares: fp32 with the roundings of its additions beside it, and what fp32's squares cannot hold.
struct Squares {
  float s = 0.0f, r = 0.0f;
  double d = 0.0;
  // x: up to 64 bytes' values, sq: the fp32 sum of their squares
  template <int N>
  __device__ __forceinline__ void add(float sq, const float (&x)[N]) {
    if (sq > 0x1p-80f && sq < 0x1p100f) {
      const float t = s + sq, z = t - s;
      r += (s - (t - z)) + (sq - z);
      s = t;
    } else {
      bool any = false;
#pragma unroll
      for (int i = 0; i < N; ++i) any |= x[i] != 0.0f;      // NaN too
      if (any) {
#pragma unroll
        for (int i = 0; i < N; ++i) d += (double)x[i] * (double)x[i];
      }
    }
  }
  __device__ __forceinline__ double total() const { return (double)s + (double)r + d; }
};

// The sum over the CTA's threads, in thread 0 (all threads call).
__device__ __forceinline__ double cta_sum(double v, double *part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kNormThreads / 32; ++w) v += part[w];
  return v;
}

// Elements of a tensor before its first 16-byte boundary.
template <typename T>
__device__ __forceinline__ int64_t head_of(const T *p, int64_t n) {
  return min(n, (int64_t)((-reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T)));
}

template <typename T>
__device__ __forceinline__ void add_unit(const T *p, int64_t n, int64_t unit, int step, Squares &sum) {
  constexpr int kPer = 16 / sizeof(T), kAhead = 4;
  const int tid = threadIdx.x;
  const int64_t head = head_of(p, n);
  if (unit == 0 && tid < head) {
    const float x[1] = {to_f32(p[tid])};
    sum.add(x[0] * x[0], x);
  }
  const T *const body = p + head + unit * step;
  const int m = (int)max((int64_t)0, min((int64_t)step, n - head - unit * step));
  const int words = m / kPer;
  for (int w0 = tid; w0 < words; w0 += kNormThreads * kAhead) {
    Pack<T, kPer> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int w = w0 + kNormThreads * u;
      v[u] = w < words ? *reinterpret_cast<const Pack<T, kPer> *>(body + w * kPer) : Pack<T, kPer>{};
    }
    float x[kPer * kAhead], sq[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      sq[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        x[u * kPer + i] = to_f32(v[u].v[i]);
        sq[u] = fmaf(x[u * kPer + i], x[u * kPer + i], sq[u]);
      }
    }
    sum.add((sq[0] + sq[1]) + (sq[2] + sq[3]), x);
  }
  if (tid < m - words * kPer) {
    const float x[1] = {to_f32(body[words * kPer + tid])};
    sum.add(x[0] * x[0], x);
  }
}

// Each CTA's sum of squares over its share of the launch's units; later launches of a call add to it.
__global__ void __launch_bounds__(kNormThreads, kCtasPerSm) reshard_squares_kernel(const __grid_constant__ Batch b, double *part, bool fresh) {
  grid_enter();
  __shared__ double warps[kNormThreads / 32];
  const uint32_t units = b.first[b.count];
  uint32_t u = (uint32_t)((uint64_t)units * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)((uint64_t)units * (blockIdx.x + 1) / gridDim.x);
  Squares sum;
  if (u < end) {
    int t = find(b, u);
    for (; u < end; ++u) {
      while (b.first[t + 1] <= u) ++t;
      const int64_t n = (int64_t)(b.n[t] >> 4), unit = u - b.first[t];
      const int type = (int)(b.n[t] & 3);
      if (type == RESHARD_F32) add_unit(reinterpret_cast<const float *>(b.at[t]), n, unit, b.unit, sum);
      else if (type == RESHARD_BF16) add_unit(reinterpret_cast<const __nv_bfloat16 *>(b.at[t]), n, unit, b.unit, sum);
      else add_unit(reinterpret_cast<const __half *>(b.at[t]), n, unit, b.unit, sum);
    }
  }
  const double v = cta_sum(sum.total(), warps);
  if (threadIdx.x == 0) part[blockIdx.x] = fresh ? v : part[blockIdx.x] + v;
}

// The norm from the CTAs' sums (all threads call and have it).
__device__ __forceinline__ float norm_of(const double *part, int ctas, double *warps) {
  double v = 0.0;
  for (int i = threadIdx.x; i < ctas; i += kNormThreads) v += part[i];
  return (float)sqrt(cta_sum(v, warps));
}

__global__ void __launch_bounds__(kNormThreads) reshard_norm_kernel(const double *part, int ctas, float *norm) {
  grid_enter();
  __shared__ double warps[kNormThreads / 32];
  const float v = norm_of(part, ctas, warps);
  if (threadIdx.x == 0) *norm = v;
}

template <typename T, typename TO>
__device__ __forceinline__ void clip_unit(const T *p, TO *to, int64_t n, int64_t unit, int step, float factor) {
  constexpr int kAhead = 4;
  const int tid = threadIdx.x;
  const int64_t head = head_of(to, n);
  if (unit == 0 && tid < head) to[tid] = from_f32<TO>(to_f32(p[tid]) * factor);
  const T *const from = p + head + unit * step;
  TO *const into = to + head + unit * step;
  const int m = (int)max((int64_t)0, min((int64_t)step, n - head - unit * step));
  auto body = [&](auto wide) {
    constexpr bool kWide = decltype(wide)::value;
    for (int w0 = tid * 8; w0 + 8 <= m; w0 += kNormThreads * 8 * kAhead) {
      Eight<T, kWide> v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int w = w0 + kNormThreads * 8 * u;
        if (w + 8 <= m) v[u].ask(from + w);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int w = w0 + kNormThreads * 8 * u;
        if (w + 8 > m) break;
        float x[8];
        v[u].take(from + w, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= factor;
        store_eight(into + w, x);
      }
    }
  };
  if ((reinterpret_cast<uintptr_t>(from) & 15) == 0) body(std::true_type());
  else body(std::false_type());
  const int rest = m & ~7;
  if (tid < m - rest) into[rest + tid] = from_f32<TO>(to_f32(from[rest + tid]) * factor);
}

// Every value times the factor. Under the limit in place there is nothing to do. norm: given, or NULL and found from the
// CTAs' sums, by each CTA for itself; `out` gets it. The units are taken from the last to the first, since what the sums
// read last is still in L2.
__global__ void __launch_bounds__(kNormThreads, kCtasPerSm)
    reshard_clip_kernel(const __grid_constant__ Batch b, const float *given, const double *part, int ctas, double limit, bool here, float *out) {
  grid_enter();
  __shared__ double warps[kNormThreads / 32];
  const float norm = given ? *given : norm_of(part, ctas, warps);
  if (out && blockIdx.x == 0 && threadIdx.x == 0) *out = norm;
  const double f = limit / ((double)norm + kEps);
  const float factor = f >= 1.0 || isinf(limit) ? 1.0f : (float)f;      // NaN stays
  if (here && factor == 1.0f) return;
  const uint32_t units = b.first[b.count];
  const uint32_t lo = (uint32_t)((uint64_t)units * blockIdx.x / gridDim.x);
  uint32_t u = (uint32_t)((uint64_t)units * (blockIdx.x + 1) / gridDim.x);
  if (u == lo) return;
  int t = find(b, u - 1);
  while (u-- > lo) {
    while (b.first[t] > u) --t;
    const int64_t n = (int64_t)(b.n[t] >> 4), unit = u - b.first[t];
    const int type = (int)(b.n[t] & 3), to = (int)(b.n[t] >> 2 & 3);
    auto go = [&](auto from_type, auto to_type) {
      clip_unit(reinterpret_cast<const decltype(from_type) *>(b.at[t]), reinterpret_cast<decltype(to_type) *>(b.to[t]), n, unit, b.unit, factor);
    };
    auto by_to = [&](auto from_type) {
      if (to == RESHARD_F32) go(from_type, float());
      else if (to == RESHARD_BF16) go(from_type, __nv_bfloat16());
      else go(from_type, __half());
    };
    if (type == RESHARD_F32) by_to(float());
    else if (type == RESHARD_BF16) by_to(__nv_bfloat16());
    else by_to(__half());
  }
}

// Calls f with each batch of the list that has something to do, from the last to the first where `back`.
template <typename F>
int batches(const reshard_tensors &list, const reshard_tensors *into, bool back, F &&f) {
  const int64_t count = (int64_t)list.tensors.size(), pieces = (count + kBatch - 1) / kBatch;
  Batch b;
  for (int64_t i = 0; i < pieces; ++i) {
    const int64_t at = (back ? pieces - 1 - i : i) * kBatch, end = std::min(count, at + kBatch);
    b.count = 0, b.first[0] = 0, b.unit = (int)list.unit;
    for (int64_t j = at; j < end; ++j) {
      const auto &t = list.tensors[(size_t)j];
      if (t.n == 0) continue;
      const auto &o = into ? into->tensors[(size_t)j] : t;
      const int k = b.count++;
      b.at[k] = t.at, b.to[k] = o.at, b.n[k] = (uint64_t)t.n << 4 | (uint64_t)o.dtype << 2 | (uint64_t)t.dtype;
      b.first[k + 1] = b.first[k] + (uint32_t)((t.n + list.unit - 1) / list.unit);
    }
    if (b.count == 0) continue;
    const int rc = f(b);
    if (rc) return rc;
  }
  return RESHARD_OK;
}

// The CTAs of every launch of a call on this list: as many as it has units, up to what the GPU holds at a time.
int ctas_of(const reshard_tensors &list, int *ctas) {
  int sms = 0;
  const int rc = device_sms(&sms);
  if (rc) return rc;
  int64_t units = 0;
  for (const auto &t : list.tensors) units += (t.n + list.unit - 1) / list.unit;
  *ctas = (int)std::max<int64_t>(1, std::min<int64_t>(units, std::min(kMaxCtas, sms * kCtasPerSm)));
  return RESHARD_OK;
}

void check_list(Checks &c, const reshard_tensors *list) {
  if (!list) return c.invalid(true, "the list is NULL");
  int dev = -1;
  if (list->high && cudaGetDevice(&dev) == cudaSuccess) c.invalid(dev != list->device, "a list was made on another device than the current one");
}

// Whether two lists share memory other than tensor by tensor (the same place, the same type).
bool entangled(const reshard_tensors &a, const reshard_tensors &b) {
  if (a.high <= b.low || b.high <= a.low) return false;
  struct Span {
    uintptr_t lo, hi;
    size_t i;
    bool of_b;
  };
  std::vector<Span> spans;
  for (size_t i = 0; i < a.tensors.size(); ++i) {
    const auto &x = a.tensors[i], &y = b.tensors[i];
    if (x.n == 0 || (x.at == y.at && x.dtype == y.dtype)) continue;
    spans.push_back({x.at, x.at + (uintptr_t)(x.n * element_bytes(x.dtype)), i, false});
  }
  for (size_t i = 0; i < b.tensors.size(); ++i) {
    const auto &y = b.tensors[i];
    if (y.n) spans.push_back({y.at, y.at + (uintptr_t)(y.n * element_bytes(y.dtype)), i, true});
  }
  std::sort(spans.begin(), spans.end(), [](const Span &x, const Span &y) { return x.lo < y.lo; });
  uintptr_t end[2] = {0, 0};
  for (const Span &s : spans) {
    if (s.lo < end[s.of_b ? 0 : 1]) return true;
    end[s.of_b] = std::max(end[s.of_b], s.hi);
  }
  return false;
}

int enqueue_squares(const reshard_tensors &list, double *part, int ctas, cudaStream_t stream) {
  bool fresh = true;
  return batches(list, nullptr, false, [&](const Batch &b) {
    const int rc = launched(launch(reshard_squares_kernel, dim3((unsigned)ctas), kNormThreads, 0, 1, stream, b, part, fresh), "launching reshard_squares_kernel");
    fresh = false;
    return rc;
  });
}

bool empty(const reshard_tensors &list) {
  return std::all_of(list.tensors.begin(), list.tensors.end(), [](const reshard_tensors::Tensor &t) { return t.n == 0; });
}

}  // namespace
}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int reshard_tensors_create(const void *const *at, const int64_t *elements, const int32_t *dtypes, int64_t count, reshard_tensors_t **list) try {
  Checks c("reshard_tensors_create");
  c.invalid(!list, "list is NULL");
  c.invalid(count < 0 || (count > 0 && (!at || !elements || !dtypes)), "count must be >= 0, and at, elements and dtypes not NULL");
  c.unsupported(count > RESHARD_MAX_EXTENT, "more than 2^30 tensors");
  if (!c.ok()) return c.report();
  *list = nullptr;
  reshard_tensors l;
  l.tensors.reserve((size_t)count);
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    const int es = element_bytes(dtypes[i]);
    c.invalid(!es, "a tensor's type must be BF16, F16 or F32");
    c.invalid(elements[i] < 0, "a tensor's elements must be >= 0");
    c.unsupported(elements[i] > (int64_t)1 << 40 || total > ((int64_t)1 << 40), "more than 2^40 elements");
    if (!c.ok()) break;
    if (elements[i] > 0) c.pointer(at[i], "a tensor", (uintptr_t)es);
    if (!c.ok()) break;      // one bad tensor is named, not ten thousand
    total += elements[i];
    l.tensors.push_back({reinterpret_cast<uintptr_t>(at[i]), elements[i], dtypes[i]});
  }
  if (!c.ok()) return c.report();
  // Units that give every CTA some, up to 16,384 elements: 8 pieces of 16 bytes a thread and more.
  l.unit = std::max<int64_t>(kUnitStep, std::min<int64_t>(8 * kUnitStep, total / (2 * kMaxCtas) / kUnitStep * kUnitStep));
  std::vector<std::pair<uintptr_t, uintptr_t>> spans;
  for (const auto &t : l.tensors)
    if (t.n) spans.push_back({t.at, t.at + (uintptr_t)(t.n * element_bytes(t.dtype))});
  std::sort(spans.begin(), spans.end());
  for (size_t i = 0; i < spans.size(); ++i) {
    if (i && spans[i].first < l.high) l.overlap = true;
    l.low = std::min(l.low, spans[i].first), l.high = std::max(l.high, spans[i].second);
  }
  if (!spans.empty()) OPS_CUDA(cudaGetDevice(&l.device));
  *list = new reshard_tensors(std::move(l));
  return RESHARD_OK;
} OPS_CATCH

extern "C" int reshard_tensors_destroy(reshard_tensors_t *list) {
  delete list;
  return RESHARD_OK;
}

extern "C" int64_t reshard_grad_norm_workspace(void) { return kMaxCtas * (int64_t)sizeof(double); }

extern "C" int reshard_grad_norm(const reshard_tensors_t *list, float *norm, void *workspace, int64_t workspace_bytes, reshard_stream_t stream_) try {
  Checks c("reshard_grad_norm");
  check_list(c, list);
  if (c.ok()) {
    c.pointer(norm, "norm", 4);
    c.pointer(workspace, "workspace", 8);
    c.invalid(workspace_bytes < reshard_grad_norm_workspace(), "the workspace is smaller than reshard_grad_norm_workspace");
  }
  if (!c.ok()) return c.report();
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  double *const part = static_cast<double *>(workspace);
  int ctas = 0, rc = empty(*list) ? RESHARD_OK : ctas_of(*list, &ctas);
  if (rc || (rc = enqueue_squares(*list, part, ctas, stream))) return rc;
  return launched(launch(reshard_norm_kernel, dim3(1), kNormThreads, 0, 1, stream, static_cast<const double *>(part), ctas, norm), "launching reshard_norm_kernel");
} OPS_CATCH

extern "C" int reshard_clip_grads(const reshard_tensors_t *list, const reshard_tensors_t *into, double limit, const float *norm_in, float *norm_out,
                                  void *workspace, int64_t workspace_bytes, reshard_stream_t stream_) try {
  Checks c("reshard_clip_grads");
  check_list(c, list);
  if (into) check_list(c, into);
  c.invalid(!(limit >= 0.0), "limit must be a number >= 0");
  c.invalid(norm_in && norm_out, "norm_in and norm_out: give one");
  if (c.ok()) {
    const reshard_tensors &to = into ? *into : *list;
    bool same = to.tensors.size() == list->tensors.size();
    for (size_t i = 0; same && into && i < to.tensors.size(); ++i) same = to.tensors[i].n == list->tensors[i].n;
    c.invalid(!same, "the lists' tensors must have the same numbers of elements");
    c.invalid(to.overlap, "tensors that are written must not overlap");
    if (same && into && into != list) c.invalid(entangled(*list, *into), "a tensor that is written overlaps one that is read elsewhere");
    if (norm_in) c.pointer(norm_in, "norm_in", 4);
    if (!norm_in) {
      c.pointer(norm_out, "norm_out", 4);
      c.pointer(workspace, "workspace", 8);
      c.invalid(workspace_bytes < reshard_grad_norm_workspace(), "the workspace is smaller than reshard_grad_norm_workspace");
    }
  }
  if (!c.ok()) return c.report();
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  double *const part = static_cast<double *>(workspace);
  if (empty(*list))
    return norm_in ? RESHARD_OK : launched(launch(reshard_norm_kernel, dim3(1), kNormThreads, 0, 1, stream, static_cast<const double *>(part), 0, norm_out), "launching reshard_norm_kernel");
  int ctas = 0, rc = ctas_of(*list, &ctas);
  if (rc || (!norm_in && (rc = enqueue_squares(*list, part, ctas, stream)))) return rc;
  // in place only if every tensor is its own target
  bool here = true;
  for (size_t i = 0; here && into && i < into->tensors.size(); ++i) {
    const auto &x = list->tensors[i], &y = into->tensors[i];
    here = x.n == 0 || (x.at == y.at && x.dtype == y.dtype);
  }
  return batches(*list, into, true, [&](const Batch &b) {
    const int rc = launched(launch(reshard_clip_kernel, dim3((unsigned)ctas), kNormThreads, 0, 1, stream, b, norm_in, static_cast<const double *>(part), ctas, limit,
                                   here, norm_out), "launching reshard_clip_kernel");
    norm_out = nullptr;
    return rc;
  });
} OPS_CATCH
