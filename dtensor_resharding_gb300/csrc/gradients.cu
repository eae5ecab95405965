// The global norm of many tensors, and their clipping: norm = sqrt(sum x^2), x * min(1, limit / (norm + 1e-6)).
//
// A list (reshard_tensors_create) keeps the tensors' places on the host. A launch takes some of them as its argument,
// so that a call copies nothing to the device and allocates nothing there, and a captured one holds its list. A tensor is
// cut into units of one size (its head before the first 16-byte boundary belongs to the first); the CTAs of a launch share
// the units of all its tensors evenly, whatever the tensors' sizes, and look each up by bisection.
//
// Squares are summed over 64 bytes a thread at most in fp32, those sums in fp32 with their roundings carried along
// (two-sum), threads and CTAs in 64 bits in a fixed order: the norm is the correctly rounded one but for some 2^-24. Values
// whose squares leave fp32's range (beyond 2^50, or all of them below 2^-40) are summed in 64 bits instead.
//
// Bound by HBM: 10,000 tensors of 150,000 bf16 values, norm only, 472 us, 6.4 TB/s; 384 of 1.57M clipped into fp32 720 us, of which the
// second read is what a factor of all values costs.
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
  int64_t units = 0;                 // of all tensors
};

namespace reshard {
namespace ops {

namespace {

constexpr int kNormThreads = 256;
constexpr int kMaxCtas = 1024;                    // whose sums the workspace holds, and the factor behind them
constexpr int kUnitStep = kNormThreads * 8;       // a unit is a multiple of it
constexpr int kSquaresCtas = 6, kClipCtas = 4;   // of an SM
constexpr int kFillCtas = 304;                    // two of each of 152 SMs
constexpr double kEps = 1e-6;

// A list of a few tensors goes in an argument of its size: 32 KB of one cost the host some 2 us a launch.
constexpr int kFewTensors = 96;
template <int N>
struct Places {
  uint64_t at[N];
};
struct InPlace {};

// The tensors of a launch, as one of its arguments: those have 32,764 bytes. A tensor is its address and one word: the units of
// the tensors before it (32 bits), the elements of its last unit (16), its type (2).
template <bool Moved, bool Few>      // Moved: with places of their own for the clipped values
struct Batch {
  static constexpr int kMost = Few ? kFewTensors : Moved ? 1300 : 2000;
  uint64_t at[kMost];
  uint64_t word[kMost + 1];          // the last: all units
  std::conditional_t<Moved, Places<kMost>, InPlace> to;
  int count;
  int unit;
  __host__ __device__ uint32_t first(int t) const { return (uint32_t)word[t]; }
  __host__ __device__ uint32_t units() const { return first(count); }
  __device__ __forceinline__ int type(int t) const { return (int)(word[t] >> 48); }
  __device__ __forceinline__ int64_t elements(int t) const { return (int64_t)(first(t + 1) - first(t) - 1) * unit + (int64_t)(word[t] >> 32 & 0xffff); }
  __device__ __forceinline__ uint64_t target(int t) const {
    if constexpr (Moved) return to.at[t];
    else return at[t];
  }
};
static_assert(sizeof(Batch<true, false>) + 64 <= 32764 && sizeof(Batch<false, false>) + 64 <= 32764, "a kernel's arguments");

int launched(cudaError_t e, const char *what) { return e == cudaSuccess ? RESHARD_OK : cuda_error(e, what); }

// The tensor that holds unit u.
template <typename B>
__device__ __forceinline__ int find(const B &b, uint32_t u) {
  int in = 0, out = b.count;
  while (out - in > 1) {
    const int mid = (in + out) / 2;
    if (b.first(mid) <= u) in = mid;
    else out = mid;
  }
  return in;
}

// A sum of squares: fp32 with the roundings of its additions beside it, and what fp32's squares cannot hold.
struct Squares {
  float s = 0.0f, r = 0.0f;
  double d = 0.0;
  // Adds an fp32 sum of squares; false where fp32 may not hold it: its values are to be added by add_far.
  __device__ __forceinline__ bool add(float sq) {
    if (!(sq > 0x1p-80f && sq < 0x1p100f)) return false;
    const float t = s + sq, z = t - s;
    r += (s - (t - z)) + (sq - z);
    s = t;
    return true;
  }
  __device__ __forceinline__ void add_far(float v) { d += (double)v * (double)v; }
  __device__ __forceinline__ void add_one(float v) {
    if (!add(v * v)) add_far(v);
  }
  __device__ __forceinline__ double total() const { return (double)s + (double)r + d; }
};

// The sum over the CTA's threads, in its first warp (all threads call). 64-bit additions are slow here: few lanes make them.
__device__ __forceinline__ double cta_sum(double v, double *part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < kNormThreads / 32 ? part[threadIdx.x] : 0.0;
#pragma unroll
    for (int o = kNormThreads / 64; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  }
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
  if (unit == 0 && tid < head) sum.add_one(to_f32(p[tid]));
  const T *const body = p + head + unit * step;
  const int m = (int)max((int64_t)0, min((int64_t)step, n - head - unit * step));
  const int words = m / kPer;
  for (int w0 = tid; w0 < words; w0 += kNormThreads * kAhead) {
    Words<T, kPer> v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int w = w0 + kNormThreads * u;
      v[u] = Words<T, kPer>{};
      if (w < words) v[u].load(body + w * kPer);
    }
    float sq[kAhead];
    uint32_t bits = 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float x[kPer];
      v[u].values(x);
      sq[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sq[u] = fmaf(x[i], x[i], sq[u]);
#pragma unroll
      for (int i = 0; i < 4; ++i) bits |= v[u].v[i];
    }
    if (sum.add((sq[0] + sq[1]) + (sq[2] + sq[3])) || (bits & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu)) == 0) continue;
#pragma unroll 1
    for (int u = 0; u < kAhead; ++u) {
      const int w = w0 + kNormThreads * u;
#pragma unroll 1
      for (int i = 0; w < words && i < kPer; ++i) sum.add_far(to_f32(body[w * kPer + i]));
    }
  }
  if (tid < m - words * kPer) sum.add_one(to_f32(body[words * kPer + tid]));
}

// Each CTA's sum of squares over its units of the launch, every gridDim-th; later launches of a call add to it.
template <bool Few>
__global__ void __launch_bounds__(kNormThreads, kSquaresCtas) reshard_squares_kernel(const __grid_constant__ Batch<false, Few> b, double *part, bool fresh) {
  grid_enter();
  __shared__ double warps[kNormThreads / 32];
  const uint32_t units = b.units();
  Squares sum;
  for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int t = find(b, u), type = b.type(t);
    const int64_t n = b.elements(t), unit = u - b.first(t);
    if (type == RESHARD_F32) add_unit(reinterpret_cast<const float *>(b.at[t]), n, unit, b.unit, sum);
    else if (type == RESHARD_BF16) add_unit(reinterpret_cast<const __nv_bfloat16 *>(b.at[t]), n, unit, b.unit, sum);
    else add_unit(reinterpret_cast<const __half *>(b.at[t]), n, unit, b.unit, sum);
  }
  const double v = cta_sum(sum.total(), warps);
  if (threadIdx.x == 0) part[blockIdx.x] = fresh ? v : part[blockIdx.x] + v;
}

// The norm from the CTAs' sums, in thread 0 (all threads call).
__device__ __forceinline__ float norm_of(const double *part, int ctas, double *warps) {
  double v = 0.0;
  for (int i = threadIdx.x; i < ctas; i += kNormThreads) v += part[i];
  v = cta_sum(v, warps);
  return threadIdx.x == 0 ? (float)sqrt(v) : 0.0f;
}

// What values are multiplied by. One thread computes it: a 64-bit division in each of a launch's threads, nine million for 600M
// values, took as long as the values.
__device__ __forceinline__ float factor_of(float norm, double limit) {
  const double f = limit / ((double)norm + kEps);
  return f >= 1.0 || isinf(limit) ? 1.0f : (float)f;      // NaN stays
}

__global__ void __launch_bounds__(kNormThreads) reshard_norm_kernel(const double *part, int ctas, float *norm, double limit, float *factor) {
  grid_enter();
  __shared__ double warps[kNormThreads / 32];
  const float v = norm_of(part, ctas, warps);
  if (threadIdx.x == 0) {
    *norm = v;
    if (factor) *factor = factor_of(v, limit);
  }
}

template <typename T, typename TO>
__device__ __forceinline__ void clip_unit(const T *p, TO *to, int64_t n, int64_t unit, int step, float factor) {
  constexpr int kN = kPieceOf<T, TO>, kAhead = 4;
  const int tid = threadIdx.x;
  const int64_t head = head_of(to, n);
  if (unit == 0 && tid < head) to[tid] = from_f32<TO>(to_f32(p[tid]) * factor);
  const T *const from = p + head + unit * step;
  TO *const into = to + head + unit * step;
  const int m = (int)max((int64_t)0, min((int64_t)step, n - head - unit * step));
  auto body = [&](auto wide) {
    constexpr bool kWide = decltype(wide)::value;
    for (int w0 = tid * kN; w0 + kN <= m; w0 += kNormThreads * kN * kAhead) {
      Piece<T, kN, kWide> v[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int w = w0 + kNormThreads * kN * u;
        if (w + kN <= m) v[u].ask(from + w);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int w = w0 + kNormThreads * kN * u;
        if (w + kN > m) break;
        float x[kN];
        v[u].take(from + w, x);
#pragma unroll
        for (int e = 0; e < kN; ++e) x[e] *= factor;
        store_piece(into + w, x);
      }
    }
  };
  if ((reinterpret_cast<uintptr_t>(from) & 15) == 0) body(std::true_type());
  else body(std::false_type());
  const int rest = m / kN * kN;
  if (tid < m - rest) into[rest + tid] = from_f32<TO>(to_f32(from[rest + tid]) * factor);
}

// Every value times the factor: found already, or from a norm that was given, or from the CTAs' sums, by each CTA for itself (the
// first writes the norm to `out`). Under the limit in place there is nothing to do. The units are taken from the last to the first, since
// what the sums read last is still in L2: a batch has its tensors from the last to the first. A launch has tensors of one pair of
// types: all nine pairs in one kernel spilled its registers.
template <typename T, typename TO, bool Moved, bool Few>
__global__ void __launch_bounds__(kNormThreads, (sizeof(TO) > sizeof(T) ? 6 : kClipCtas))
    reshard_clip_kernel(const __grid_constant__ Batch<Moved, Few> b, const float *found, const float *given, const double *part, int ctas, double limit, float *out) {
  grid_enter();
  __shared__ double warps[kNormThreads / 32];
  __shared__ float shared;
  float factor;
  if (found) {
    factor = *found;
  } else {
    const float norm = given ? *given : norm_of(part, ctas, warps);
    if (threadIdx.x == 0) {
      shared = factor_of(norm, limit);
      if (out && blockIdx.x == 0) *out = norm;
    }
    __syncthreads();
    factor = shared;
  }
  if (!Moved && factor == 1.0f) return;
  const uint32_t units = b.units();
  for (uint32_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int t = find(b, u);
    const uint32_t back = b.first(t + 1) - 1 - u;        // a tensor's units, too, from the last to the first
    clip_unit(reinterpret_cast<const T *>(b.at[t]), reinterpret_cast<TO *>(b.target(t)), b.elements(t), back, b.unit, factor);
  }
}

// Calls f with each batch of the list that has something to do, from the last to the first where `back`: of all its tensors,
// or of those of one type whose targets in `into` have one type.
template <bool Moved, bool Few, typename F>
int batches(const reshard_tensors &list, const reshard_tensors *into, int dtype, int to, bool back, F &&f) {
  const int64_t count = (int64_t)list.tensors.size();
  Batch<Moved, Few> b;
  b.unit = (int)list.unit, b.count = 0, b.word[0] = 0;
  for (int64_t i = 0; i < count; ++i) {
    const size_t j = (size_t)(back ? count - 1 - i : i);
    const auto &t = list.tensors[j];
    if (t.n > 0 && (!into || (t.dtype == dtype && into->tensors[j].dtype == to))) {
      const int k = b.count++;
      const uint64_t units = (uint64_t)((t.n + list.unit - 1) / list.unit);
      b.at[k] = t.at;
      if constexpr (Moved) b.to.at[k] = into->tensors[j].at;
      b.word[k] |= (uint64_t)(t.n - (int64_t)(units - 1) * list.unit) << 32 | (uint64_t)t.dtype << 48;
      b.word[k + 1] = (uint32_t)b.word[k] + units;
    }
    if (b.count == Batch<Moved, Few>::kMost || (i == count - 1 && b.count > 0)) {
      const int rc = f(b);
      if (rc) return rc;
      b.count = 0, b.word[0] = 0;
    }
  }
  return RESHARD_OK;
}

// The CTAs of the launches that sum squares: as many as the list has units, up to what the GPU holds at a time.
int ctas_of(const reshard_tensors &list, int *ctas) {
  int sms = 0;
  const int rc = device_sms(&sms);
  if (rc) return rc;
  *ctas = (int)std::max<int64_t>(1, std::min<int64_t>(list.units, std::min(kMaxCtas, sms * kSquaresCtas)));
  return RESHARD_OK;
}

void check_list(Checks &c, const reshard_tensors *list) {
  if (!list) return c.invalid(true, "the list is NULL");
  int dev = -1;
  if (list->high && cudaGetDevice(&dev) == cudaSuccess) c.invalid(dev != list->device, "a list was made on another device than the current one");
}

// Whether two lists share memory other than tensor by tensor (the same place, the same type). Lists whose ranges of addresses do not
// meet are told apart at once; others (tensors and their targets allocated in turn) are sorted in each call: 10,000 tensors cost
// the host 0.85 ms instead of 0.2.
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

template <typename F>
int by_count(const reshard_tensors &list, F &&f) {
  return list.tensors.size() <= kFewTensors ? f(std::true_type()) : f(std::false_type());
}

int enqueue_squares(const reshard_tensors &list, double *part, int ctas, cudaStream_t stream) {
  bool fresh = true;
  return by_count(list, [&](auto few) {
    constexpr bool kFew = decltype(few)::value;
    return batches<false, kFew>(list, nullptr, 0, 0, false, [&](const Batch<false, kFew> &b) {
      const int rc = launched(launch(reshard_squares_kernel<kFew>, dim3((unsigned)ctas), kNormThreads, 0, 1, stream, b, part, fresh), "launching reshard_squares_kernel");
      fresh = false;
      return rc;
    });
  });
}

int enqueue_norm(const double *part, int ctas, float *norm, double limit, float *factor, cudaStream_t stream) {
  return launched(launch(reshard_norm_kernel, dim3(1), kNormThreads, 0, 1, stream, part, ctas, norm, limit, factor), "launching reshard_norm_kernel");
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
  // Units of up to 16,384 elements (8 pieces of 16 bytes a thread, or 16), halved while there is not one for each CTA.
  l.unit = 8 * kUnitStep;
  while (l.unit > kUnitStep && total / l.unit < kFillCtas) l.unit /= 2;
  for (const auto &t : l.tensors) l.units += (t.n + l.unit - 1) / l.unit;
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

extern "C" int64_t reshard_grad_norm_workspace(void) { return (kMaxCtas + 1) * (int64_t)sizeof(double); }

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
  int ctas = 0, rc = list->units ? ctas_of(*list, &ctas) : RESHARD_OK;
  if (rc || (rc = enqueue_squares(*list, part, ctas, stream))) return rc;
  return enqueue_norm(part, ctas, norm, 0.0, nullptr, stream);
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
  if (list->units == 0) return norm_in ? RESHARD_OK : enqueue_norm(part, 0, norm_out, limit, nullptr, stream);
  int ctas = 0, rc = ctas_of(*list, &ctas);
  if (rc || (!norm_in && (rc = enqueue_squares(*list, part, ctas, stream)))) return rc;
  // in place only if every tensor is its own target
  bool here = true;
  for (size_t i = 0; here && into && i < into->tensors.size(); ++i) {
    const auto &x = list->tensors[i], &y = into->tensors[i];
    here = x.n == 0 || (x.at == y.at && x.dtype == y.dtype);
  }
  // Where every unit has a CTA on the GPU at once, each of them adds up the norm for itself; more CTAs find the factor ready.
  float *const factor = reinterpret_cast<float *>(part + kMaxCtas);
  const float *found = nullptr;
  if (!norm_in && list->units > ctas) {
    if ((rc = enqueue_norm(part, ctas, norm_out, limit, factor, stream))) return rc;
    found = factor;
  }
  bool present[4][4] = {};
  const reshard_tensors &to = into ? *into : *list;
  for (size_t i = 0; i < to.tensors.size(); ++i)
    if (to.tensors[i].n) present[list->tensors[i].dtype][to.tensors[i].dtype] = true;
  auto clip = [&](auto moved, auto few, int x, int y) {
    constexpr bool kMoved = decltype(moved)::value, kFew = decltype(few)::value;
    return batches<kMoved, kFew>(*list, &to, x, y, true, [&](const Batch<kMoved, kFew> &b) {
      // One CTA a unit, which writes faster than CTAs that stay; in place those, since most often they have nothing to do
      // (where they have: 384 of 1.57M bf16 379 us, 6.4 TB/s).
      const unsigned grid = kMoved ? b.units() : std::min((unsigned)ctas, b.units());
      const int rc = launched(by_type(x, [&](auto from_type) {
        return by_type(y, [&](auto to_type) {
          using T = decltype(from_type);
          using TO = decltype(to_type);
          if constexpr (kMoved || std::is_same_v<T, TO>)
            return launch(reshard_clip_kernel<T, TO, kMoved, kFew>, dim3(grid), kNormThreads, 0, 1, stream, b, found, norm_in, static_cast<const double *>(part), ctas, limit, norm_out);
          else
            return cudaErrorInvalidValue;        // in place the types are the same
        });
      }), "launching reshard_clip_kernel");
      norm_out = nullptr;
      return rc;
    });
  };
  for (int x = 3; x > 0; --x)
    for (int y = 3; y > 0; --y)
      if (present[x][y] && (rc = by_count(*list, [&](auto few) { return here ? clip(std::false_type(), few, x, y) : clip(std::true_type(), few, x, y); }))) return rc;
  return RESHARD_OK;
} OPS_CATCH
