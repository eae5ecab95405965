// The gradient of an embedding: grad_table[r] = scale * sum of grad[t] over the tokens t whose id is row r of this shard.
//
// Four launches. *Sort* (one cluster) sorts the tokens by row: a radix sort of the pairs (row, token), at most ten bits a pass,
// stable, so that a row's tokens ascend. *Zero* writes the table's zeros beside it. *Sum* takes runs of the sorted
// tokens, one thread a piece of the columns: rows that begin and end inside a run are written from there, the parts of one
// that does not are left in the workspace, and *join* adds them in the order of the runs. A token that is half of the
// text is so spread over as many CTAs as it has runs, without atomics. The order of every sum follows from the ids, the number of columns
// and the types; runs are cut from all tokens of the shard, so that other rows' tokens can regroup a row's.
// Sums are fp32, rounded once. A few tokens need no sort. Bound by the write of the table and the read of the gradients: 32,768 x
// 4096 bf16 into half of 128,000 rows 112 us (floor 97; zeros 71 with the sort's 20 beside them, sum 33); 4,095 x 2048 fp32 into 12,501 rows 27
// (zeros 16, then the sum's and the join's latency).
#include <algorithm>

#include "ops_common.cuh"
#include "values.cuh"

namespace reshard {
namespace ops {

namespace {

constexpr int64_t kAlign = 256;
int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

int launched(cudaError_t e, const char *what) { return e == cudaSuccess ? RESHARD_OK : cuda_error(e, what); }

// ------------------------------------------------------------------------------------------------------------- sort --

constexpr int kSortWarps = 32, kSortCluster = 8, kSortBits = 10;      // warps of a CTA at most

struct Sort {
  const void *ids;
  bool wide_ids;
  int64_t tokens, first, rows;
  uint2 *sorted, *other;             // (row, token) pairs; the last pass writes `sorted`
  int32_t *held;                     // how many tokens are of this shard
  int passes, bits;                  // bits a pass
};

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// Every warp has a run of the pairs in each pass: it counts their digits, the counts of the warps and CTAs before it give
// its first place of each digit, and a second walk places 32 pairs at a time, equal digits ranked by lane (match.any).
// Integer counts: the order is the same on every run. Bound by latency (two walks and three barriers a pass).
__global__ void __launch_bounds__(kSortWarps * 32) reshard_sort_rows_kernel(Sort a) {
  grid_enter();
  extern __shared__ int32_t count[];             // [warp][digit], then this CTA's sums [digit], then its first places [digit]
  __shared__ int32_t warp_sum[kSortWarps];
  const int bins = 1 << a.bits, warps = blockDim.x >> 5;
  int32_t *const sum = count + warps * bins, *const base = sum + bins;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = (int)blockIdx.x;
  int32_t *const mine = count + warp * bins;
  int64_t n = a.tokens;
  for (int pass = 0; pass < a.passes; ++pass) {
    const uint2 *const from = (a.passes - pass) & 1 ? a.other : a.sorted;
    uint2 *const to = (a.passes - pass) & 1 ? a.sorted : a.other;
    const int64_t run = (n + kSortCluster * (int)blockDim.x - 1) / (kSortCluster * (int)blockDim.x) * 32;
    const int64_t lo = (cta * warps + warp) * run, hi = min(lo + run, n);
    auto pair = [&](int64_t i) {                 // row 2^32 - 1: none
      uint2 p = make_uint2(~0u, 0);
      if (i < hi) {
        if (pass == 0) {
          const int64_t id = a.wide_ids ? static_cast<const int64_t *>(a.ids)[i] : static_cast<const int32_t *>(a.ids)[i];
          if (id >= a.first && id - a.first < a.rows) p = make_uint2((uint32_t)(id - a.first), (uint32_t)i);
        } else {
          p = __ldcg(from + i);
        }
      }
      return p;
    };
    const int shift = pass * a.bits;
    for (int i = tid; i < warps * bins; i += (int)blockDim.x) count[i] = 0;
    __syncthreads();
    for (int64_t i0 = lo + lane; i0 < hi; i0 += 4 * 32) {
      uint2 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = pair(i0 + 32 * u);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (p[u].x != ~0u) atomicAdd(&mine[p[u].x >> shift & (bins - 1)], 1);
    }
    __syncthreads();
    for (int d = tid; d < bins; d += (int)blockDim.x) {
      int s = 0;
#pragma unroll 16
      for (int w = 0; w < warps; ++w) {
        const int c = count[w * bins + d];
        count[w * bins + d] = s;
        s += c;
      }
      sum[d] = s;
    }
    cluster_barrier();
    // the digits' first places: a running sum of the cluster's counts, and this CTA's share of each
    int done = 0;
    for (int d0 = 0; d0 < bins; d0 += (int)blockDim.x) {
      const int d = d0 + tid;
      int all = 0, before = 0;
      if (d < bins) {
#pragma unroll
        for (int c = 0; c < kSortCluster; ++c) {
          uint32_t at;
          int v;
          asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&sum[d])), "r"(c));
          asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at));
          if (c < cta) before += v;
          all += v;
        }
      }
      int upto = all;
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, upto, o);
        if (lane >= o) upto += x;
      }
      __syncthreads();                           // the round before has read warp_sum
      if (lane == 31) warp_sum[warp] = upto;
      __syncthreads();
      int here = 0;
      for (int w = 0; w < warps; ++w) {
        if (w < warp) upto += warp_sum[w];
        here += warp_sum[w];
      }
      if (d < bins) base[d] = done + upto - all + before;
      done += here;
    }
    __syncthreads();
    for (int64_t i0 = lo; i0 < hi; i0 += 4 * 32) {
      uint2 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = pair(i0 + 32 * u + lane);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = p[u].x != ~0u;
        const int d = in ? (int)(p[u].x >> shift & (bins - 1)) : bins;
        const uint32_t same = __match_any_sync(kFull, d);
        if (in) to[base[d] + mine[d] + __popc(same & ((1u << lane) - 1))] = p[u];
        __syncwarp();
        if (in && (same >> lane) == 1) mine[d] += __popc(same);      // the last of each digit's lanes
        __syncwarp();
      }
    }
    n = done;
    cluster_barrier();                           // the pairs are in place, and nobody reads `sum` any more
  }
  if (cta == 0 && tid == 0) *a.held = (int32_t)n;
}

// ------------------------------------------------------------------------------------------------------------- zero --

constexpr int kZeroThreads = 256;
constexpr int64_t kZeroPiece = 32768;      // bytes of a CTA

// Zeros in `rows` rows of `bytes` bytes, `stride` apart, all a multiple of `unit` (2 or 4) bytes. Behind a sort it begins
// when that has begun, and so behind everything that came earlier on the stream; only its last CTA waits for the sort, so that the
// grid behind this one finds both done.
__global__ void __launch_bounds__(kZeroThreads) reshard_zero_kernel(uint8_t *base, int64_t rows, int64_t bytes, int64_t stride, int unit, bool behind_sort) {
  if (!behind_sort) grid_wait();
  grid_release();
  const int64_t pieces = (bytes + kZeroPiece - 1) / kZeroPiece;
  for (int64_t w = blockIdx.x; w < rows * pieces; w += gridDim.x) {
    const int64_t r = w / pieces, at = (w - r * pieces) * kZeroPiece;
    uint8_t *p = base + r * stride + at;
    int n = (int)min(kZeroPiece, bytes - at);
    auto small = [&](int i) {
      if (unit == 4) *reinterpret_cast<uint32_t *>(p + i) = 0;
      else *reinterpret_cast<uint16_t *>(p + i) = 0;
    };
    const int head = min(n, (int)(-reinterpret_cast<uintptr_t>(p) & 15));
    if ((int)threadIdx.x * unit < head) small((int)threadIdx.x * unit);
    p += head, n -= head;
#pragma unroll 8
    for (int i = threadIdx.x; i < n / 16; i += kZeroThreads) reinterpret_cast<uint4 *>(p)[i] = make_uint4(0, 0, 0, 0);
    const int tail = (n & ~15) + (int)threadIdx.x * unit;
    if (tail < n) small(tail);
  }
  if (behind_sort && blockIdx.x == gridDim.x - 1) grid_wait();
}

// -------------------------------------------------------------------------------------------------------------- sum --

constexpr int kSumThreads = 128;

// The sorted tokens go in runs, one to each CTA (of a slice of the columns): at least kMinRun tokens, and as many runs as give the
// GPU one round of CTAs, kSumCtas of each of 152 SMs, or more of fewer warps (a second round of a few CTAs took a third longer). How
// many tokens are of this shard, the device knows. (152 whatever the device has: the workspace's size is asked for without one.) Each run leaves up to two rows in the workspace. (59,088 x 176 bf16 into 25,645
// rows: 58 us, of which the sort 27; CTAs of four warps, one of them with columns, and 512 runs 68.)
constexpr int64_t kMinRun = 16, kMostRuns = 1024;
constexpr int kSumCtas = 6;
struct Slices {                      // of rows of so many columns, a piece of `values` a thread
  int threads, count;
  Slices(int64_t cols, int values) : threads(kSumThreads) {
    while (threads > 32 && threads / 2 * values >= cols) threads /= 2;
    count = (int)((cols + threads * values - 1) / (threads * values));
  }
  int64_t runs(int64_t tokens) const {
    const int64_t round = 152 * kSumCtas * (kSumThreads / threads) / count;
    return std::min((tokens + kMinRun - 1) / kMinRun, std::max<int64_t>(64, std::min(kMostRuns, round)));
  }
};

struct Sum {
  const uint2 *sorted;
  const int32_t *held;
  const void *grad;
  int64_t cols, grad_stride;
  float scale;
  void *table;
  int64_t table_stride;
  bool accumulate, wide_table;
  float *part;                       // [run][2][pitch]: of the row that a run begins inside, and of the one that it ends inside
  int64_t pitch;
  int runs;                          // at most
  int slices;                        // CTAs a run
  __device__ __forceinline__ int64_t run_of(int64_t tokens) const { return tokens <= kMinRun * runs ? kMinRun : (tokens + runs - 1) / runs; }
};

// N of a row's sums, scaled, into the table.
template <typename T, int N>
__device__ __forceinline__ void write_sums(const Sum &a, uint32_t row, int64_t c, const float (&sum)[N]) {
  T *const to = static_cast<T *>(a.table) + (int64_t)row * a.table_stride + c;
  float x[N];
  const bool whole = a.wide_table && c + N <= a.cols;
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = sum[e] * a.scale;
  if (a.accumulate) {
    float old[N];
    load_values<T, N>(to, (int)min((int64_t)N, a.cols - c), whole, old);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] += old[e];
  }
  if (whole) {
    store_piece(to, x);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < a.cols) to[e] = from_f32<T>(x[e]);
  }
}

template <typename TG, typename T, bool Wide>
__global__ void __launch_bounds__(kSumThreads, Wide ? kSumCtas : 5) reshard_sum_rows_kernel(Sum a) {
  constexpr int kN = kPieceOf<TG, T>, kRows = Wide ? 8 : 4;       // rows in flight
  grid_enter();
  const int lane = threadIdx.x & 31;
  const int64_t number = blockIdx.x / (uint32_t)a.slices;
  const int64_t c = ((int64_t)(blockIdx.x % (uint32_t)a.slices) * blockDim.x + threadIdx.x) * kN;
  const int64_t held = *a.held, run = a.run_of(held), lo = number * run, hi = min(lo + run, held);
  if (lo >= held || c - lane * kN >= a.cols) return;       // whole warps
  uint2 mine = lo + lane < hi ? a.sorted[lo + lane] : make_uint2(0, 0);
  const uint32_t before = lo > 0 ? a.sorted[lo - 1].x : ~0u;
  const uint32_t after = hi < held ? a.sorted[hi].x : ~0u;
  const TG *const grad = static_cast<const TG *>(a.grad) + c;
  const int left = (int)max((int64_t)0, min((int64_t)kN, a.cols - c));
  uint32_t row = __shfl_sync(kFull, mine.x, 0);
  bool head = before == row;
  float *const part = a.part + 2 * number * a.pitch + c;
  float sum[kN] = {};
  auto keep = [&](float *to) {
    if (left == 0) return;
#pragma unroll
    for (int e = 0; e < kN; e += 4) *reinterpret_cast<float4 *>(to + e) = make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
  };
  for (int64_t base = lo; base < hi; base += 32) {
    if (base > lo) mine = base + lane < hi ? a.sorted[base + lane] : make_uint2(0, 0);
    const int n = (int)min((int64_t)32, hi - base);
    for (int i = 0; i < n; i += kRows) {
      Piece<TG, kN, Wide> v[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        const uint32_t t = __shfl_sync(kFull, mine.y, i + u);      // i is a multiple of kRows: below 32
        if (left == kN && i + u < n) v[u].ask(grad + t * a.grad_stride);
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        if (i + u >= n) break;
        const uint32_t r = __shfl_sync(kFull, mine.x, i + u), t = __shfl_sync(kFull, mine.y, i + u);
        if (r != row) {
          if (head) keep(part);
          else if (left) write_sums<T, kN>(a, row, c, sum);
          head = false, row = r;
#pragma unroll
          for (int e = 0; e < kN; ++e) sum[e] = 0.0f;
        }
        const TG *const from = grad + t * a.grad_stride;
        float x[kN];
        if (left == kN) v[u].take(from, x);
        else load_values<TG, kN>(from, left, false, x);
#pragma unroll
        for (int e = 0; e < kN; ++e) sum[e] += x[e];
      }
    }
  }
  if (head) keep(part);
  else if (after == row) keep(part + a.pitch);
  else if (left) write_sums<T, kN>(a, row, c, sum);
}

// The rows that end in another run than they begin in: the CTAs of the run that such a row begins in.
template <typename T>
__global__ void __launch_bounds__(kSumThreads) reshard_join_rows_kernel(Sum a) {
  grid_enter();
  const int lane = threadIdx.x & 31;
  const int64_t number = blockIdx.x / (uint32_t)a.slices;
  const int64_t c = ((int64_t)(blockIdx.x % (uint32_t)a.slices) * blockDim.x + threadIdx.x) * 4;
  const int64_t held = *a.held, run = a.run_of(held), lo = number * run, hi = lo + run;
  if (hi >= held) return;
  const uint32_t row = a.sorted[hi - 1].x, after = a.sorted[hi].x, before = lo > 0 ? a.sorted[lo - 1].x : ~0u;
  // the run that the row ends in: the first whose next run begins with another row, or that is the last
  int64_t last = number + 1;
  const int64_t next = (last + lane + 1) * run;
  uint32_t ends = __ballot_sync(kFull, next >= held || a.sorted[min(next, held - 1)].x != row);
  if (after != row || before == row) return;
  while (!ends) {
    last += 32;
    const int64_t more = (last + lane + 1) * run;
    ends = __ballot_sync(kFull, more >= held || a.sorted[min(more, held - 1)].x != row);
  }
  last += __ffs(ends) - 1;
  if (c >= a.cols) return;
  float sum[4];
  load_values<float, 4>(a.part + (2 * number + 1) * a.pitch + c, 4, true, sum);
  const float *from = a.part + 2 * (number + 1) * a.pitch + c;
#pragma unroll 16
  for (int64_t r = number + 1; r <= last; ++r, from += 2 * a.pitch) {
    float x[4];
    load_values<float, 4>(from, 4, true, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += x[e];
  }
  write_sums<T, 4>(a, row, c, sum);
}

// ------------------------------------------------------------------------------------------------------- few tokens --

// Of few tokens each finds its own like: a CTA a token (and slice of the columns) compares its row with all others'; the first
// token of a row adds up the row. Without a sort and its workspace: 200 tokens of as many rows into 9,000 x 512 bf16 take 4.5 us,
// 257 by the sort 12.9 (added to a table 2.9 and 15.8). Tokens of one row (padding) are the other side: 256 of them, added up
// one after another by the CTAs of the first, take 35 us, 257 in runs 12.5.
constexpr int kFewTokens = 256;

struct FewSum {
  const void *ids;
  bool wide_ids;
  int tokens;
  int64_t first, rows;
  Sum sum;
};

template <typename TG, typename T, bool Wide>
__global__ void __launch_bounds__(kSumThreads, Wide ? kSumCtas : 5) reshard_sum_few_rows_kernel(FewSum f) {
  constexpr int kN = kPieceOf<TG, T>, kRows = Wide ? 8 : 4;
  grid_enter();
  __shared__ uint32_t like[kFewTokens / 32];     // the tokens with this one's row
  const Sum &a = f.sum;
  const int t = (int)(blockIdx.x / (uint32_t)a.slices);
  const int64_t c = ((int64_t)(blockIdx.x % (uint32_t)a.slices) * kSumThreads + threadIdx.x) * kN;
  auto row_of = [&](int i) {                     // -1: another shard's
    const int64_t id = f.wide_ids ? static_cast<const int64_t *>(f.ids)[i] : static_cast<const int32_t *>(f.ids)[i];
    return id >= f.first && id - f.first < f.rows ? id - f.first : (int64_t)-1;
  };
  const int64_t row = row_of(t);
  bool before = false;
  for (int i = threadIdx.x; i < kFewTokens; i += kSumThreads) {
    const bool same = i < f.tokens && row_of(i) == row;
    const uint32_t mask = __ballot_sync(kFull, same);
    if ((threadIdx.x & 31) == 0) like[i / 32] = mask;
    before |= same && i < t;
  }
  if (__syncthreads_or(before) || row < 0 || c >= a.cols) return;
  const TG *const grad = static_cast<const TG *>(a.grad) + c;
  const int left = (int)min((int64_t)kN, a.cols - c);
  float sum[kN] = {};
  int word = 0;
  uint32_t bits = like[0];
  auto next = [&]() {                            // the next of the row's tokens, -1 behind the last
    while (bits == 0) {
      if (++word == kFewTokens / 32) return -1;
      bits = like[word];
    }
    const int i = word * 32 + __ffs(bits) - 1;
    bits &= bits - 1;
    return i;
  };
  for (bool more = true; more;) {
    int at[kRows];
    Piece<TG, kN, Wide> v[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      at[u] = more ? next() : -1;
      more = at[u] >= 0;
      if (more && left == kN) v[u].ask(grad + at[u] * a.grad_stride);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      if (at[u] < 0) break;
      const TG *const from = grad + at[u] * a.grad_stride;
      float x[kN];
      if (left == kN) v[u].take(from, x);
      else load_values<TG, kN>(from, left, false, x);
#pragma unroll
      for (int e = 0; e < kN; ++e) sum[e] += x[e];
    }
  }
  write_sums<T, kN>(a, (uint32_t)row, c, sum);
}

struct Layout {
  int64_t sorted, held, runs, pitch, part;
  Layout(int64_t tokens, int64_t cols)
      : sorted(up(8 * tokens, kAlign)), held(kAlign), runs(Slices(cols, 8).runs(tokens)), pitch(up(cols, 8)),
        part(up(2 * runs * pitch * 4, kAlign)) {}
  int64_t bytes() const { return 2 * sorted + held + part; }
};

}  // namespace
}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int64_t reshard_embedding_backward_workspace(int64_t tokens, int64_t cols) {
  if (tokens <= kFewTokens || cols < 1 || tokens > RESHARD_MAX_SLOTS || cols > RESHARD_MAX_EXTENT) return 0;
  return Layout(tokens, cols).bytes();
}

extern "C" int reshard_embedding_backward(const void *grad, int grad_dtype, int64_t tokens, int64_t cols, int64_t grad_stride,
                                          const void *ids, int id_bits, int64_t first_row, int64_t rows, float scale, void *grad_table,
                                          int table_dtype, int64_t table_stride, int accumulate, void *workspace, int64_t workspace_bytes,
                                          reshard_stream_t stream_) try {
  Checks c("reshard_embedding_backward");
  c.invalid(tokens < 0 || rows < 0 || cols < 0 || first_row < 0, "tokens, rows, cols and first_row must be >= 0");
  c.unsupported(tokens > RESHARD_MAX_SLOTS || rows > RESHARD_MAX_EXTENT || cols > RESHARD_MAX_EXTENT, "tokens, rows or cols above 2^30");
  c.invalid(id_bits != 32 && id_bits != 64, "id_bits must be 32 or 64");
  c.invalid(!element_bytes(grad_dtype) || !element_bytes(table_dtype), "grad_dtype and table_dtype must be BF16, F16 or F32");
  c.invalid(grad_stride < cols || table_stride < cols, "a row stride is shorter than the row");
  const bool work = rows > 0 && cols > 0 && (tokens > 0 || !accumulate);      // a layout is of rows that have columns
  if (work && c.ok() && tokens > 0)
    c.unsupported(Layout(tokens, cols).runs * Slices(cols, 4).count > INT32_MAX, "too many columns for one launch");
  if (work && c.ok()) {
    c.pointer(grad_table, "grad_table", (uintptr_t)element_bytes(table_dtype));
    if (tokens > 0) {
      c.pointer(grad, "grad", (uintptr_t)element_bytes(grad_dtype));
      c.pointer(ids, "ids", (uintptr_t)(id_bits / 8));
      if (tokens > kFewTokens) c.pointer(workspace, "workspace", kAlign);
      c.invalid(workspace_bytes < reshard_embedding_backward_workspace(tokens, cols), "the workspace is smaller than reshard_embedding_backward_workspace");
    }
  }
  if (!c.ok()) return c.report();
  if (!work) return RESHARD_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int es = element_bytes(table_dtype);
  const Layout l(tokens, cols);
  uint8_t *const at = static_cast<uint8_t *>(workspace);
  int rc = RESHARD_OK;
  uint2 *const sorted = reinterpret_cast<uint2 *>(at);
  int32_t *const held = reinterpret_cast<int32_t *>(at + 2 * l.sorted);
  const bool few = tokens <= kFewTokens;
  if (!few) {
    Sort s{ids, id_bits == 64, tokens, first_row, rows, sorted, reinterpret_cast<uint2 *>(at + l.sorted), held, 1, 1};
    int need = 1;
    while (need < 30 && (rows - 1) >> need) ++need;
    s.passes = (need + kSortBits - 1) / kSortBits;
    s.bits = (need + s.passes - 1) / s.passes;
    if ((rc = allow_smem<reshard_sort_rows_kernel>((size_t)(kSortWarps + 2) * 4 << kSortBits))) return rc;
    // Half the warps take a few microseconds less for a few tokens (4,095: 10 us), all of them for many (65,536: 20 instead of 28).
    const int warps = tokens <= 16384 ? kSortWarps / 2 : kSortWarps;
    if ((rc = launched(launch(reshard_sort_rows_kernel, dim3(kSortCluster), warps * 32, (size_t)(warps + 2) * 4 << s.bits, kSortCluster, stream, s),
                       "launching reshard_sort_rows_kernel")))
      return rc;
  }
  if (!accumulate) {
    const bool dense = table_stride == cols;
    const int64_t zero_rows = dense ? 1 : rows, bytes = (dense ? rows : 1) * cols * es;
    const int64_t ctas = std::min<int64_t>(RESHARD_MAX_EXTENT, zero_rows * ((bytes + kZeroPiece - 1) / kZeroPiece));
    if ((rc = launched(launch(reshard_zero_kernel, dim3((unsigned)ctas), kZeroThreads, 0, 1, stream, static_cast<uint8_t *>(grad_table), zero_rows, bytes,
                              table_stride * es, es, !few), "launching reshard_zero_kernel")))
      return rc;
  }
  if (tokens == 0) return RESHARD_OK;
  Sum a{sorted, held, grad, cols, grad_stride, scale, grad_table, table_stride, accumulate != 0, aligned16(grad_table, table_stride, es),
        reinterpret_cast<float *>(at + 2 * l.sorted + l.held), l.pitch, 0, 0};
  const bool wide = aligned16(grad, grad_stride, element_bytes(grad_dtype));
  rc = launched(by_type(grad_dtype, [&](auto g) {
    using TG = decltype(g);
    return by_type(table_dtype, [&](auto t) {
      using T = decltype(t);
      const Slices s(cols, kPieceOf<TG, T>);
      a.slices = s.count;
      if (few) {
        a.slices = (int)((cols + kSumThreads * kPieceOf<TG, T> - 1) / (kSumThreads * kPieceOf<TG, T>));
        const FewSum f{ids, id_bits == 64, (int)tokens, first_row, rows, a};
        return launch(wide ? reshard_sum_few_rows_kernel<TG, T, true> : reshard_sum_few_rows_kernel<TG, T, false>, dim3((unsigned)(tokens * a.slices)),
                      kSumThreads, 0, 1, stream, f);
      }
      a.runs = (int)s.runs(tokens);
      return launch(wide ? reshard_sum_rows_kernel<TG, T, true> : reshard_sum_rows_kernel<TG, T, false>, dim3((unsigned)(a.runs * a.slices)), s.threads, 0,
                    1, stream, a);
    });
  }), "launching reshard_sum_rows_kernel");
  if (rc || few || a.runs == 1) return rc;
  const Slices s(cols, 4);
  a.slices = s.count;
  return launched(by_type(table_dtype, [&](auto t) {
    return launch(reshard_join_rows_kernel<decltype(t)>, dim3((unsigned)((a.runs - 1) * a.slices)), s.threads, 0, 1, stream, a);
  }), "launching reshard_join_rows_kernel");
} OPS_CATCH
