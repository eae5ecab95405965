// Routing to experts: scores, selection and weights of each token, its gradient, and the order in which the chosen
// (token, expert) slots reach the experts' products.
//
// Score s of logits z: softmax(z) or sigmoid(z) = 1 / (1 + exp(-z)). Experts are ordered by s + bias; without a bias
// by z itself, which orders them as s does but has no ties that rounding made. The lowest index comes first among
// equals. With groups (equal runs of experts) only those of the `kept` groups whose `group_top` best experts have the
// largest sum of scores (+ bias) can be chosen. A logit of -inf or NaN, or a key that is one, is never chosen: the row's
// missing slots get id -1 and weight 0. Everything is computed in 32 bits.
//
// One warp holds a row in registers (E / 32 values a lane), so that a row is read once and selection is k rounds of a
// warp-wide integer maximum: keys are mapped to unsigned integers of the same order, what cannot be chosen to 0, and
// redux.sync gives the maximum and then the lowest index that has it. Bound by instruction issue (scores, groups, and the
// rounds), not by HBM, for the usual 128 to 256 experts: 16,384 x 256 fp32 in 8 groups, 8 chosen, takes 19.7 us, where the
// read alone would take 2.6; 24 x 128 takes 3.4, a launch.
#include <algorithm>
#include <cfloat>
#include <climits>

#include "ops_common.cuh"

namespace reshard {
namespace ops {

namespace {

constexpr int kRouteWarps = 4;     // rows of a CTA
constexpr uint32_t kFull = 0xffffffffu;

struct RouteArgs {
  const void *logits;
  int64_t tokens, stride;
  int experts, k, groups, kept, group_top;
  const float *bias;
  bool sigmoid, renorm;
  float scale;
};

// Unsigned integers in the order of the floats; 0 for what cannot be chosen (-inf, NaN). -0 counts as +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (!(v > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t u) { return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xffffffffu)); }

// The rounding of each step is the one its formula names: __fadd_rn keeps the compiler from fusing the sum with
// the exponential's last product, which would order near-equal scores by another rounding.
__device__ __forceinline__ float sigmoid_score(float z) { return __frcp_rn(__fadd_rn(1.0f, expf(-z))); }

__device__ __forceinline__ float warp_max(float v) {
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// A lane's V values of a row: vectors of W neighbours, dealt round the warp. e(i) is value i's expert.
template <int V, int W>
struct Lane {
  static __device__ __forceinline__ int expert(int i, int lane) { return (i / W) * 32 * W + lane * W + i % W; }
};

template <typename T, int V, int W>
__device__ __forceinline__ void load_row(const T *row, int E, int lane, float (&z)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += W) {
    const int e = Lane<V, W>::expert(i, lane);
    if (W > 1) {     // E and the row's start are multiples of W elements
      struct alignas(sizeof(T) * W) Vec { T v[W]; };
      if (e < E) {
        const Vec x = *reinterpret_cast<const Vec *>(row + e);
#pragma unroll
        for (int j = 0; j < W; ++j) z[i + j] = to_f32(x.v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) z[i + j] = -INFINITY;
      }
    } else {
      z[i] = e < E ? to_f32(row[e]) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (isnan(z[i])) z[i] = -INFINITY;
}

template <int V>
__device__ __forceinline__ float row_max(const float (&z)[V]) {
  float m = z[0];
#pragma unroll
  for (int i = 1; i < V; ++i) m = fmaxf(m, z[i]);
  m = warp_max(m);
  return m == -INFINITY ? 0.0f : m;   // a row with nothing to choose: exp(-inf - 0) = 0 everywhere
}

__device__ __forceinline__ uint32_t group_key(uint32_t best, uint32_t next) {
  return next ? order_key(fmaxf(__fadd_rn(key_value(best), key_value(next)), -FLT_MAX)) : best;      // biases of the lowest value: not -inf
}

// Bit g: group g is one of the `kept` best; total: lane g's group's key (0: nothing to choose).
__device__ __forceinline__ uint32_t best_groups(uint32_t total, int groups, int kept, int lane) {
  uint32_t mask = 0;
  for (int j = 0; j < kept; ++j) {
    const uint32_t left = lane < groups && !(mask >> lane & 1) ? total : 0;
    const uint32_t best = __reduce_max_sync(kFull, left);
    if (!best) break;
    mask |= 1u << (__ffs(__ballot_sync(kFull, left == best)) - 1);
  }
  return mask;
}

// Sets to 0 the keys of every group but the `kept` best. rank: the values that rank groups, as keys.
template <int V, int W>
__device__ __forceinline__ void keep_groups(const RouteArgs &a, int lane, const uint32_t (&rank)[V], uint32_t (&key)[V]) {
  const int size = a.experts / a.groups;
  if (W == 4 && size >= 4 && size <= 128 && (size & (size - 1)) == 0) {
    // A vector's four experts are of one group, and `lanes` neighbouring lanes hold all of it: their two best meet by
    // shuffles, for all groups of a vector index at once. 16,384 x 256 in 8 groups: 15 us more without this path.
    const int lanes = size / 4, shift = 31 - __clz(size), per = 128 >> shift;      // groups a vector index
    uint32_t total = 0;
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      uint32_t b0 = 0, b1 = 0;
#pragma unroll
      for (int i = 4 * h; i < 4 * h + 4; ++i) {
        b1 = max(b1, min(b0, rank[i]));
        b0 = max(b0, rank[i]);
      }
      for (int o = 1; o < lanes; o <<= 1) {
        const uint32_t x0 = __shfl_xor_sync(kFull, b0, o), x1 = __shfl_xor_sync(kFull, b1, o);
        b1 = max(min(b0, x0), max(b1, x1));
        b0 = max(b0, x0);
      }
      const uint32_t t = a.group_top > 1 ? group_key(b0, b1) : b0;
      const uint32_t x = __shfl_sync(kFull, t, (lane - h * per) * lanes & 31);
      if (lane >= h * per && lane < (h + 1) * per) total = x;
    }
    const uint32_t kept = best_groups(total, a.groups, a.kept, lane);
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const int g = h * per + ((lane * 4) >> shift);
      if (g > 31 || !(kept >> g & 1)) {
#pragma unroll
        for (int i = 4 * h; i < 4 * h + 4; ++i) key[i] = 0;
      }
    }
    return;
  }
  uint32_t total = 0;
  for (int g = 0; g < a.groups; ++g) {
    const int lo = g * size, hi = lo + size;
    uint32_t b0 = 0, b1 = 0;       // this lane's two best of the group
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = Lane<V, W>::expert(i, lane);
      const uint32_t u = e >= lo && e < hi ? rank[i] : 0;
      b1 = max(b1, min(b0, u));
      b0 = max(b0, u);
    }
    const uint32_t top = __reduce_max_sync(kFull, b0);
    uint32_t next = 0;
    if (a.group_top > 1 && top) {
      const uint32_t has = __ballot_sync(kFull, b0 == top);
      next = __reduce_max_sync(kFull, lane == __ffs(has) - 1 ? b1 : b0);
    }
    if (lane == g) total = group_key(top, next);
  }
  const uint32_t kept = best_groups(total, a.groups, a.kept, lane);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t g = (uint32_t)Lane<V, W>::expert(i, lane) / (uint32_t)size;
    if (g > 31 || !(kept >> g & 1)) key[i] = 0;
  }
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(kRouteWarps * 32) reshard_route_kernel(RouteArgs a, float *weights, int32_t *ids) {
  grid_enter();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const T *row = static_cast<const T *>(a.logits) + t * a.stride;
  float z[V];
  load_row<T, V, W>(row, a.experts, lane, z);

  // what the score needs of the whole row
  float top = 0.0f, total = 0.0f;
  uint32_t key[V];
  const bool whole = !a.sigmoid && (a.bias || !a.renorm), ranked = a.groups > 1 && a.group_top > 1;
  if (!a.sigmoid && (whole || ranked)) top = row_max<V>(z);
  if (whole) {
#pragma unroll
    for (int i = 0; i < V; ++i) total += expf(z[i] - top);
    total = warp_sum(total);
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < V; i += W) {
      const int e = Lane<V, W>::expert(i, lane);
      struct alignas(4 * W) Vec { float v[W]; } b{};
      if (e < a.experts) b = *reinterpret_cast<const Vec *>(a.bias + e);
#pragma unroll
      for (int j = i; j < i + W; ++j) {
        const float s = a.sigmoid ? sigmoid_score(z[j]) : __fdiv_rn(expf(z[j] - top), total);
        key[j] = z[j] > -INFINITY ? order_key(__fadd_rn(s, b.v[j - i])) : 0;
      }
    }
    if (a.groups > 1) keep_groups<V, W>(a, lane, key, key);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = order_key(z[i]);
    if (ranked) {      // sums of scores; a softmax row's common divisor changes no order
      uint32_t rank[V];
#pragma unroll
      for (int i = 0; i < V; ++i) rank[i] = key[i] ? order_key(a.sigmoid ? sigmoid_score(z[i]) : expf(z[i] - top)) : 0;
      keep_groups<V, W>(a, lane, rank, key);
    } else if (a.groups > 1) {
      keep_groups<V, W>(a, lane, key, key);
    }
  }

  // A lane holds its two best keys and where they are (of the lane's experts, less the lane's offset). The lane that gave a
  // choice moves up its second; when both are gone it looks through its keys again, at those behind the last it gave. (After every
  // choice: 22.7 us instead of 19.7 for the 256 experts above, 17.0 instead of 12.9 for 8,192 x 512, 40.4 instead of 41.5 for 32 of
  // 1,024.)
  int id = -1;              // lane j: the j-th choice
  uint32_t best0 = 0, best1 = 0;
  int at0 = 0, at1 = 0, held = 2;
  auto see = [&](uint32_t u, int at) {
    if (u > best0) {
      best1 = best0, at1 = at0;
      best0 = u, at0 = at;
    } else if (u > best1) {
      best1 = u, at1 = at;
    }
  };
#pragma unroll
  for (int i = 0; i < V; ++i) see(key[i], Lane<V, W>::expert(i, 0));
  for (int j = 0; j < a.k; ++j) {
    const uint32_t best = __reduce_max_sync(kFull, best0);
    if (!best) break;
    const uint32_t has = __ballot_sync(kFull, best0 == best);
    const int e = at0 + lane * W;
    const int first = has & (has - 1) ? __reduce_min_sync(kFull, best0 == best ? e : INT_MAX) : __shfl_sync(kFull, e, __ffs(has) - 1);
    if (best0 == best && e == first) {
      const int gone = at0;
      best0 = best1, at0 = at1;
      if (--held == 0 && j + 1 < a.k) {
        best0 = best1 = 0;
        held = 2;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int at = Lane<V, W>::expert(i, 0);
          see(key[i] < best || (key[i] == best && at > gone) ? key[i] : 0, at);
        }
      }
    }
    if (lane == j) id = first;
  }

  const float zc = id >= 0 ? to_f32(row[id]) : -INFINITY;
  float w = 0.0f;
  if (a.sigmoid) {
    if (id >= 0) w = sigmoid_score(zc);
  } else if (a.renorm) {    // relative to the largest chosen logit: no row's weights underflow together
    const float m = warp_max(zc);
    if (id >= 0) w = expf(zc - m);
  } else if (id >= 0) {
    w = __fdiv_rn(expf(zc - top), total);
  }
  if (a.renorm) {
    const float sum = warp_sum(w);
    w = sum == 0.0f ? 0.0f : __fdiv_rn(w, sum);
  }
  if (lane < a.k) {
    weights[t * a.k + lane] = w * a.scale;
    ids[t * a.k + lane] = id;
  }
}

// The gradient to the logits, with g_j the gradient to weight j times scale, over the row's valid ids i_j:
//   softmax:               d z_e = p_e (sum_j [i_j = e] g_j - sum_j g_j p_{i_j})
//   softmax, renormalised: r = softmax over the chosen logits;  d z_{i_j} = r_j (g_j - sum g r), 0 elsewhere
//   sigmoid:               d z_{i_j} = g_j s_j (1 - s_j)
//   sigmoid, renormalised: r_j = s_j / sum s;  d z_{i_j} = (g_j - sum g r) r_j (1 - s_j)
// 1 - s is computed as sigmoid(-z). The bias only selects and has no gradient. Written whole, one warp a row; bound by
// the write of the rows (and, for the whole softmax, the read of the logits) and by a row's chain of dependent loads
// (ids, then the chosen logits): 32,768 x 128 fp32, sigmoid, 9.5 us, 2.1 TB/s. Where no id repeats, zeros are written and
// the k values over them: comparing every value's expert with every id took 11.0 us there.
template <typename T, int V, int W>
__global__ void __launch_bounds__(kRouteWarps * 32)
    reshard_route_backward_kernel(RouteArgs a, const float *grad, const int32_t *ids, T *out, int64_t out_stride) {
  grid_enter();
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (t >= a.tokens) return;
  const T *row = static_cast<const T *>(a.logits) + t * a.stride;
  int id = lane < a.k ? ids[t * a.k + lane] : -1;
  if (id >= a.experts) id = -1;
  const float g = id >= 0 ? grad[t * a.k + lane] * a.scale : 0.0f;
  float zc = id >= 0 ? to_f32(row[id]) : -INFINITY;
  if (isnan(zc)) zc = -INFINITY;
  float d = 0.0f, dot = 0.0f;        // lane j: what expert i_j gets of slot j
  float p[V];
  const bool whole = !a.sigmoid && !a.renorm;
  if (whole) {
    load_row<T, V, W>(row, a.experts, lane, p);
    const float top = row_max<V>(p);
    float total = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] = expf(p[i] - top);
      total += p[i];
    }
    total = warp_sum(total);
    const float inv = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] *= inv;
    dot = warp_sum(g * (expf(zc - top) * inv));
    d = g;
  } else {
    float r = 0.0f, tail = 1.0f;
    if (a.sigmoid) {
      if (id >= 0) {
        r = sigmoid_score(zc);
        tail = sigmoid_score(-zc);
      }
    } else {
      const float m = warp_max(zc);
      if (id >= 0 && m > -INFINITY) r = expf(zc - m);
    }
    if (a.renorm) {
      const float sum = warp_sum(r);
      r = sum == 0.0f ? 0.0f : __fdiv_rn(r, sum);
      dot = warp_sum(g * r);
    }
    d = (g - dot) * r * tail;
  }
  T *to = out + t * out_stride;
  float o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.0f;
  // Zeros, and then the k values over them by their lanes; ids that repeat, and the whole softmax, are summed first.
  const uint32_t same = __match_any_sync(kFull, id);       // by every lane, whatever its id
  const bool scatter = !__any_sync(kFull, id >= 0 && __popc(same) > 1) && !whole;
  for (int j = 0; j < (scatter ? 0 : a.k); ++j) {
    const int e = __shfl_sync(kFull, id, j);
    const float v = __shfl_sync(kFull, d, j);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (Lane<V, W>::expert(i, lane) == e) o[i] += v;
  }
  if (whole) {
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = p[i] * (o[i] - dot);
  }
#pragma unroll
  for (int i = 0; i < V; i += W) {
    const int e = Lane<V, W>::expert(i, lane);
    if (e >= a.experts) continue;
    if (W > 1) {
      struct alignas(sizeof(T) * W) Vec { T v[W]; } x;
#pragma unroll
      for (int j = 0; j < W; ++j) x.v[j] = from_f32<T>(o[i + j]);
      *reinterpret_cast<Vec *>(to + e) = x;
    } else {
      to[e] = from_f32<T>(o[i]);
    }
  }
  __syncwarp();
  if (scatter && id >= 0) to[id] = from_f32<T>(d);
}

// ------------------------------------------------------------------------------------------------------ dispatch --

// The slots (token, choice) sorted by expert, in slot order within each: offsets[e] .. offsets[e + 1] are expert e's
// places, order[place] its slot, position[slot] its place (-1: no expert of this range). A counting sort by one CTA, or by
// a cluster of eight that shares its counts through distributed shared memory, in one launch without workspace: every
// warp counts the experts of a run of slots of its own; the counts of the warps and CTAs before it give each warp its
// first place of each expert; a second walk of the run places 32 slots at a time, equal ones ranked by lane
// (match.any). Counts are integers, so their atomics change nothing: the order is the same on every run. Bound by
// latency: 65,536 slots over 128 experts 12.1 us (14 with cold caches), 32,760 over 16 of them 4.7 (7) (one CTA an expert, each
// reading all ids: 117).
constexpr int kDispatchWarps = 32, kDispatchCluster = 8;

__global__ void __launch_bounds__(kDispatchWarps * 32)
    reshard_dispatch_kernel(const int32_t *ids, int slots, int first, int experts, int32_t *offsets, int32_t *order, int32_t *position) {
  grid_enter();
  extern __shared__ int32_t count[];             // [warp][expert], then [expert]: this CTA's sum
  int32_t *const sum = count + kDispatchWarps * experts;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = (int)gridDim.x, cta = (int)blockIdx.x;     // the grid is one cluster
  const int run = ((slots + ctas * kDispatchWarps * 32 - 1) / (ctas * kDispatchWarps * 32)) * 32;     // slots a warp
  const int64_t lo = (int64_t)(cta * kDispatchWarps + warp) * run;
  const int64_t hi = min(lo + run, (int64_t)slots);
  auto expert = [&](int64_t i) {       // slot i's expert here, -1 if it has none
    const int id = i < hi ? ids[i] : -1;
    return id >= first && id - first < experts ? id - first : -1;
  };
  for (int i = tid; i < kDispatchWarps * experts; i += kDispatchWarps * 32) count[i] = 0;
  __syncthreads();
  int32_t *const mine = count + warp * experts;
  for (int64_t i0 = lo + lane; i0 < hi; i0 += 8 * 32) {      // eight loads in flight
    int e[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) e[u] = expert(i0 + 32 * u);
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (e[u] >= 0) atomicAdd(&mine[e[u]], 1);
  }
  __syncthreads();
  for (int e = tid; e < experts; e += kDispatchWarps * 32) {       // counts of the warps before, and the CTA's
    int n = 0;
#pragma unroll 8
    for (int w = 0; w < kDispatchWarps; ++w) {
      const int c = count[w * experts + e];
      count[w * experts + e] = n;
      n += c;
    }
    sum[e] = n;
  }
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
  // the experts' first places: a running sum of the cluster's counts, one expert a thread, and this CTA's share of each
  __shared__ int32_t warp_sum[RESHARD_MAX_GROUPS / 32];
  int all = 0, before = 0, upto = 0;
  if (tid < (experts + 31) / 32 * 32) {
    if (tid < experts) {
      int n[kDispatchCluster];
#pragma unroll
      for (int c = 0; c < kDispatchCluster; ++c) {
        uint32_t at;
        n[c] = 0;
        if (c < ctas) {
          asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&sum[tid])), "r"(c));
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n[c]) : "r"(at));
        }
      }
#pragma unroll
      for (int c = 0; c < kDispatchCluster; ++c) {
        if (c < cta) before += n[c];
        all += n[c];
      }
    }
    upto = all;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) warp_sum[warp] = upto;
  }
  __syncthreads();
  if (tid < experts) {
    for (int w = 0; w < warp; ++w) upto += warp_sum[w];
    if (cta == 0) {
      offsets[tid] = upto - all;
      if (tid == experts - 1) offsets[experts] = upto;
    }
    sum[experts + tid] = upto - all + before;        // this CTA's first place of the expert
  }
  __syncthreads();
  for (int64_t i0 = lo; i0 < hi; i0 += 4 * 32) {
    int next[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) next[u] = expert(i0 + 32 * u + lane);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + 32 * u + lane;
      const int e = next[u];
      const uint32_t same = __match_any_sync(kFull, e);
      if (e >= 0) {
        const int at = sum[experts + e] + mine[e] + __popc(same & ((1u << lane) - 1));
        order[at] = (int32_t)i;
        position[i] = at;
      } else if (i < hi) {
        position[i] = -1;
      }
      __syncwarp();
      if (e >= 0 && (same >> lane) == 1) mine[e] += __popc(same);      // the last of each expert's lanes
      __syncwarp();
    }
  }
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");   // others may still read `sum`
}

// Calls f with the number of values a lane holds and the width of its vectors: four neighbours where E, the row
// stride and the base allow it, one otherwise.
template <typename F>
void by_shape(int experts, bool wide, F &&f) {
  if (wide) {
    if (experts <= 128) f(std::integral_constant<int, 4>(), std::integral_constant<int, 4>());
    else if (experts <= 256) f(std::integral_constant<int, 8>(), std::integral_constant<int, 4>());
    else if (experts <= 512) f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
    else f(std::integral_constant<int, 32>(), std::integral_constant<int, 4>());
  } else {
    if (experts <= 64) f(std::integral_constant<int, 2>(), std::integral_constant<int, 1>());
    else if (experts <= 256) f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
    else f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  }
}

template <typename F>
void by_type(int dtype, F &&f) {
  if (dtype == RESHARD_F32) f(float());
  else if (dtype == RESHARD_BF16) f(__nv_bfloat16());
  else f(__half());
}

bool quads(const void *p, int dtype, int experts, int64_t stride) {
  return experts % 4 == 0 && stride % 4 == 0 && (reinterpret_cast<uintptr_t>(p) % (4 * element_bytes(dtype))) == 0;
}

void check_route(Checks &c, int64_t tokens, int experts, int64_t stride, int dtype, int k, int score) {
  c.invalid(tokens < 0, "tokens < 0");
  c.invalid(experts < 1 || k < 1 || k > experts, "experts and k must be positive, k at most experts");
  c.unsupported(experts > RESHARD_ROUTE_MAX_EXPERTS || k > RESHARD_ROUTE_MAX_K, "more than 1024 experts or k above 32");
  c.invalid(stride < experts, "a row stride is shorter than the row");
  c.invalid(!element_bytes(dtype), "dtype must be BF16, F16 or F32");
  c.invalid(score != RESHARD_SCORE_SOFTMAX && score != RESHARD_SCORE_SIGMOID, "unknown score function");
  c.unsupported(tokens > (int64_t)INT32_MAX * kRouteWarps, "too many tokens for one launch");
}

}  // namespace

int enqueue_dispatch(const int32_t *ids, int64_t slots, int first, int experts, int32_t *offsets, int32_t *order,
                     int32_t *position, cudaStream_t stream) {
  // one CTA for a few slots a thread: a cluster's barriers cost more than they save there
  const int ctas = slots <= 4 * kDispatchWarps * 32 ? 1 : kDispatchCluster;
  const size_t smem = (size_t)(kDispatchWarps + 2) * experts * 4;
  int rc = allow_smem<&reshard_dispatch_kernel>((size_t)(kDispatchWarps + 2) * RESHARD_MAX_GROUPS * 4);
  if (rc) return rc;
  OPS_CUDA(launch(reshard_dispatch_kernel, dim3((unsigned)ctas), kDispatchWarps * 32, smem, ctas, stream, ids, (int)slots, first, experts,
                  offsets, order, position));
  return RESHARD_OK;
}

}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int reshard_route(const void *logits, int dtype, int64_t tokens, int experts, int64_t row_stride, const float *bias,
                             int score, int groups, int groups_kept, int group_top, int k, int renormalize, float scale,
                             float *weights, int32_t *ids, reshard_stream_t stream) try {
  Checks c("reshard_route");
  check_route(c, tokens, experts, row_stride, dtype, k, score);
  c.invalid(groups < 1 || (groups >= 1 && experts >= 1 && experts % groups), "groups must divide experts");
  c.unsupported(groups > 32, "more than 32 groups");
  c.invalid(groups_kept < 1 || groups_kept > groups, "groups_kept must be 1 .. groups");
  c.invalid(group_top != 1 && group_top != 2, "group_top must be 1 or 2");
  if (c.ok()) c.invalid((int64_t)groups_kept * (experts / groups) < k, "the kept groups hold fewer than k experts");
  if (c.ok()) c.invalid(group_top > experts / groups, "group_top exceeds a group's experts");
  if (tokens > 0 && c.ok()) {
    c.pointer(logits, "logits", (uintptr_t)element_bytes(dtype));
    if (bias) c.pointer(bias, "bias", 4);
    c.pointer(weights, "weights", 4);
    c.pointer(ids, "ids", 4);
  }
  if (!c.ok()) return c.report();
  if (tokens == 0) return RESHARD_OK;
  const RouteArgs a{logits, tokens, row_stride, experts, k, groups, groups_kept, group_top, bias,
                    score == RESHARD_SCORE_SIGMOID, renormalize != 0, scale};
  cudaError_t e = cudaSuccess;
  by_type(dtype, [&](auto t) {
    using T = decltype(t);
    by_shape(experts, quads(logits, dtype, experts, row_stride) && (reinterpret_cast<uintptr_t>(bias) & 15) == 0, [&](auto v, auto w) {
      e = launch(reshard_route_kernel<T, decltype(v)::value, decltype(w)::value>,
                 dim3((unsigned)((tokens + kRouteWarps - 1) / kRouteWarps)), kRouteWarps * 32, 0, 1,
                 reinterpret_cast<cudaStream_t>(stream), a, weights, ids);
    });
  });
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_route_kernel");
} OPS_CATCH

extern "C" int reshard_route_backward(const float *grad_weights, const void *logits, int dtype, int64_t tokens, int experts,
                                      int64_t row_stride, const int32_t *ids, int k, int score, int renormalize, float scale,
                                      void *grad_logits, int64_t grad_stride, reshard_stream_t stream) try {
  Checks c("reshard_route_backward");
  check_route(c, tokens, experts, row_stride, dtype, k, score);
  c.invalid(grad_stride < experts, "a row stride is shorter than the row");
  if (tokens > 0 && c.ok()) {
    c.pointer(grad_weights, "grad_weights", 4);
    c.pointer(logits, "logits", (uintptr_t)element_bytes(dtype));
    c.pointer(ids, "ids", 4);
    c.pointer(grad_logits, "grad_logits", (uintptr_t)element_bytes(dtype));
  }
  if (!c.ok()) return c.report();
  if (tokens == 0) return RESHARD_OK;
  const RouteArgs a{logits, tokens, row_stride, experts, k, 1, 1, 1, nullptr, score == RESHARD_SCORE_SIGMOID, renormalize != 0, scale};
  const bool wide = quads(logits, dtype, experts, row_stride) && quads(grad_logits, dtype, experts, grad_stride);
  cudaError_t e = cudaSuccess;
  by_type(dtype, [&](auto t) {
    using T = decltype(t);
    by_shape(experts, wide, [&](auto v, auto w) {
      e = launch(reshard_route_backward_kernel<T, decltype(v)::value, decltype(w)::value>,
                 dim3((unsigned)((tokens + kRouteWarps - 1) / kRouteWarps)), kRouteWarps * 32, 0, 1,
                 reinterpret_cast<cudaStream_t>(stream), a, grad_weights, ids, static_cast<T *>(grad_logits), grad_stride);
    });
  });
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_route_backward_kernel");
} OPS_CATCH

extern "C" int reshard_dispatch(const int32_t *ids, int64_t slots, int first_expert, int experts, int32_t *offsets, int32_t *order,
                                int32_t *position, reshard_stream_t stream) try {
  Checks c("reshard_dispatch");
  c.invalid(slots < 0, "slots < 0");
  c.unsupported(slots > RESHARD_MAX_SLOTS, "more than 2^30 slots");
  c.invalid(first_expert < 0 || experts < 1, "first_expert must be >= 0 and experts >= 1");
  c.unsupported(experts > RESHARD_MAX_GROUPS, "more than 512 experts on this side");
  if (c.ok()) {
    c.pointer(offsets, "offsets", 4);
    if (slots > 0) {
      c.pointer(ids, "ids", 4);
      c.pointer(order, "order", 4);
      c.pointer(position, "position", 4);
    }
  }
  if (!c.ok()) return c.report();
  return enqueue_dispatch(ids, slots, first_expert, experts, offsets, order, position, reinterpret_cast<cudaStream_t>(stream));
} OPS_CATCH
