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
constexpr int kFewThreads = 64;                  // of a CTA where warps are few: spread over the SMs
constexpr int kAhead = 4;                        // pieces of a lane in flight together
constexpr int kSpan = 32 * kAhead;               // pieces of a row that a warp moves

// Slot s's place, -1 if it has none among `rows`.
__device__ __forceinline__ int place_of(const int32_t *position, int64_t s, int64_t rows) {
  const int p = position[s];
  return p >= 0 && p < rows ? p : -1;
}

// The warp's row and span where every row has `spans` warps.
struct Where {
  int64_t row, span;
  __device__ __forceinline__ explicit Where(int spans) {
    const int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
    row = w <= 0xffffffffll ? (uint32_t)w / (uint32_t)spans : w / spans;
    span = w - row * spans;
  }
};

// ---------------------------------------------------------------------------------------------------------- permute --

struct Permute {
  const void *x;
  int64_t tokens, cols, stride;      // cols and strides of the kernel of whole pieces: in pieces of 16 bytes
  const int32_t *order, *position;
  int k;
  void *out;
  int64_t rows, out_stride;
  int spans;                         // warps a row (a slot's row, where rows start anywhere); behind them, where `rest`,
  bool rest;                         // a warp 32 rows to write zeros into those that no slot owns
};

// Of the 32 rows from `first` on those that no slot owns, as bits: each lane looks one up.
__device__ __forceinline__ uint32_t unowned(const int32_t *order, const int32_t *position, int64_t slots, int64_t rows, int64_t first, int lane) {
  const int64_t i = first + lane;
  bool none = false;
  if (i < rows) {
    const int64_t s = order[i];        // not written behind the last place: whatever it holds there is no owner
    none = s < 0 || s >= slots || position[s] != i;
  }
  return __ballot_sync(kFull, none);
}

// Rows of whole 16-byte pieces: a warp reads 2 KB of a token's row once and writes it to each of its places. Bound by the writes:
// 8,192 x 2048 bf16 to 8 places each, 47 us, 6.4 TB/s. Zeros are written row after row by a warp for 32 of them: of 16,383 tokens' 8
// places of 4096 bf16, one in eight taken, 230 us (floor 178), 41 without the zeros.
__global__ void __launch_bounds__(kRowThreads) reshard_permute_kernel(Permute a) {
  grid_enter();
  const int lane = threadIdx.x & 31;
  const Where at(a.spans);
  const int64_t t = at.row;
  if (t >= a.tokens) {
    const int64_t first = ((t - a.tokens) * a.spans + at.span) * 32;
    if (!a.rest || first >= a.rows) return;
    for (uint32_t left = unowned(a.order, a.position, a.tokens * a.k, a.rows, first, lane); left; left &= left - 1) {
      uint4 *const to = static_cast<uint4 *>(a.out) + (first + __ffs(left) - 1) * a.out_stride;
      for (int64_t c = lane; c < a.cols; c += 32) to[c] = make_uint4(0, 0, 0, 0);
    }
    return;
  }
  const int64_t c0 = at.span * kSpan + lane;
  const uint4 *const from = static_cast<const uint4 *>(a.x) + t * a.stride;
  uint4 v[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u)
    if (c0 + 32 * u < a.cols) v[u] = from[c0 + 32 * u];
  for (int j0 = 0; j0 < a.k; j0 += 32) {
    int mine = -1;
    if (j0 + lane < a.k) {
      const int64_t s = t * a.k + j0 + lane;
      mine = place_of(a.position, s, a.rows);
      if (mine >= 0 && a.order[mine] != s) mine = -1;
    }
    for (uint32_t live = __ballot_sync(kFull, mine >= 0); live; live &= live - 1) {
      uint4 *const to = static_cast<uint4 *>(a.out) + (int64_t)__shfl_sync(kFull, mine, __ffs(live) - 1) * a.out_stride;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + 32 * u < a.cols) to[c0 + 32 * u] = v[u];
    }
  }
}

// Pieces [first, first + kSpan) of a row, copied (times `scale`, where scaled) or, without a source, zeroed. All lanes call.
template <typename T, bool Wide, bool Scaled>
__device__ __forceinline__ void move_span(const T *from, T *to, int64_t cols, int64_t first, int lane, float scale) {
  constexpr int kN = kPieceOf<T, T>;
  const int64_t c0 = piece_start<T, kN, Wide>(first, to);
  std::conditional_t<Wide, Words<T, kN>[kAhead], Strip<T, kN, kAhead>> v;
  if (from) {
    if constexpr (Wide) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (c0 + (32 * u + lane + 1) * kN <= cols) v[u].load(from + c0 + (32 * u + lane) * kN);
    } else {
      v.ask(from, cols, c0, lane);
    }
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int64_t c = c0 + (32 * u + lane) * kN;
    const bool whole = c >= 0 && c + kN <= cols;
    Words<T, kN> r{};
    if constexpr (Wide) {
      if (from && whole) r = v[u];
    } else {
      if (from) r = v.words(u, lane);
    }
    if (Scaled && from) {
      float x[kN];
      r.values(x);
#pragma unroll
      for (int i = 0; i < kN; ++i) x[i] *= scale;
      r.round(x);
    }
    if (whole) {
      r.store(to + c);
    } else if (c < cols) {           // the row's ends, value by value
#pragma unroll
      for (int i = 0; i < kN; ++i)
        if (c + i >= 0 && c + i < cols) to[c + i] = !from ? from_f32<T>(0.0f) : Scaled ? from_f32<T>(to_f32(from[c + i]) * scale) : from[c + i];
    }
  }
}

// Rows that start anywhere: a warp a span of a slot's row, which starts elsewhere than the token's does. Bound by instructions (shuffles,
// funnel shifts): 8,191 x 2867 bf16 to 4 places each, 53 us, floor 35.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) reshard_permute_any_kernel(Permute a) {
  grid_enter();
  const Where at(a.spans);
  const int64_t s = at.row, slots = a.tokens * a.k;
  if (s >= slots) {
    const int64_t first = ((s - slots) * a.spans + at.span) * 32;
    if (!a.rest || first >= a.rows) return;
    for (uint32_t left = unowned(a.order, a.position, slots, a.rows, first, threadIdx.x & 31); left; left &= left - 1)
      for (int c = 0; c < a.spans; ++c)
        move_span<T, false, false>(nullptr, static_cast<T *>(a.out) + (first + __ffs(left) - 1) * a.out_stride, a.cols, c * kSpan, threadIdx.x & 31, 1.0f);
    return;
  }
  const int p = place_of(a.position, s, a.rows);
  if (p < 0 || a.order[p] != s) return;
  move_span<T, false, false>(static_cast<const T *>(a.x) + s / a.k * a.stride, static_cast<T *>(a.out) + (int64_t)p * a.out_stride, a.cols, at.span * kSpan,
                             threadIdx.x & 31, 1.0f);
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

// A warp 2 KB of a token's row. Bound by the writes, and the reads of the rows that are not in L2: 32,768 tokens on a quarter of a
// vocabulary of 128,000 x 4096 bf16, 46 us, 6.3 TB/s.
template <typename T, bool Wide, bool Scaled>
__global__ void __launch_bounds__(kRowThreads) reshard_embedding_kernel(Lookup a) {
  grid_enter();
  const Where at(a.spans);
  const int64_t t = at.row;
  if (t >= a.tokens) return;
  const int64_t id = a.wide_ids ? static_cast<const int64_t *>(a.ids)[t] : static_cast<const int32_t *>(a.ids)[t];
  const bool here = id >= a.first && id - a.first < a.rows;
  move_span<T, Wide, Scaled>(here ? static_cast<const T *>(a.table) + (id - a.first) * a.stride : nullptr, static_cast<T *>(a.out) + t * a.out_stride, a.cols,
                             at.span * kSpan, threadIdx.x & 31, a.scale);
}

// ---------------------------------------------------------------------------------------------------------- combine --

// A warp a span of a token's columns. Lanes look up the places of up to 32 slots at once; those that have one are taken in
// order, kSlots rows in flight together. Bound by the read of y: 8 places a token, 8,192 x 2048 bf16, 50 us, 6.0 TB/s; where few
// slots have a place by the chain places, rows, output of each span, so that warps stay and look up the next span's places
// before this one's rows (16,383 tokens with one place of eight on average, 4096 bf16: 54 us; fp32 72, a warp a span: 86). Rows that start
// anywhere are bound by instructions (8,191 x 2867 fp16, four places each: 48 us, of 2872 columns 42; with two words read by
// each lane, without its neighbour's: 59).
template <typename TY, typename TO>
struct CombineShape {
  static constexpr int kN = kPieceOf<TY, TO>;
  static constexpr int kPieces = 16 / kN;        // 16 columns a lane
  static constexpr int kSlots = 2;
  static constexpr int kCtas = sizeof(TY) == 4 ? 3 : 4;      // of an SM: what the registers allow
};

template <typename TY, typename TO, bool Wide>
__global__ void __launch_bounds__(kRowThreads, CombineShape<TY, TO>::kCtas) reshard_combine_kernel(Combine a, int spans) {
  using Shape = CombineShape<TY, TO>;
  constexpr int kN = Shape::kN, kU = Shape::kPieces, kSlots = Shape::kSlots;
  grid_enter();
  const int lane = threadIdx.x & 31;
  const int64_t units = a.tokens * spans, step = (int64_t)gridDim.x * (blockDim.x >> 5);
  int64_t unit = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  auto row_of = [&](int64_t w) { return w <= 0xffffffffll ? (int64_t)((uint32_t)w / (uint32_t)spans) : w / spans; };
  // The lane's slot among 32 from j0 on: its place (-1: none) and weight. Those of the next unit are asked for before this one's rows.
  auto look = [&](int64_t t, int j0, int &place, float &weight) {
    const int64_t s = t * a.k + j0 + lane;
    const bool in = j0 + lane < a.k;
    place = in ? a.position[s] : -1;
    weight = in && a.weights ? a.weights[s] : 1.0f;
  };
  int next = -1;
  float next_weight = 1.0f;
  if (unit >= units) return;
  look(row_of(unit), 0, next, next_weight);
  do {
    const int64_t t = row_of(unit), span = unit - t * spans;
    int mine = next;
    float weight = next_weight;
    if (Wide && unit + step < units) look(row_of(unit + step), 0, next, next_weight);
    TO *const to = static_cast<TO *>(a.out) + t * a.out_stride;
    const int64_t c0 = piece_start<TO, kN, Wide>(span * 32 * kU, to);
    auto column = [&](int u) { return c0 + (32 * u + lane) * kN; };
    auto whole = [&](int u) { return column(u) >= 0 && column(u) + kN <= a.cols; };
    float sum[kU][kN] = {};
    for (int j0 = 0;;) {
      for (uint32_t live = __ballot_sync(kFull, mine >= 0 && mine < a.rows); live;) {
        const TY *from[kSlots];
        float w[kSlots];
        std::conditional_t<Wide, Words<TY, kN>[kU], Strip<TY, kN, kU>> v[kSlots];
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
          const int j = __ffs(live) - 1;           // -1: none left
          const int p = __shfl_sync(kFull, mine, max(j, 0));
          w[q] = __shfl_sync(kFull, weight, max(j, 0));
          from[q] = j >= 0 ? static_cast<const TY *>(a.y) + (int64_t)p * a.y_stride : nullptr;
          live &= live - 1;
          if (!from[q]) continue;
          if constexpr (Wide) {
#pragma unroll
            for (int u = 0; u < kU; ++u)
              if (whole(u)) v[q][u].load(from[q] + column(u));
          } else {
            v[q].ask(from[q], a.cols, c0, lane);
          }
        }
#pragma unroll
        for (int q = 0; q < kSlots; ++q) {
          if (!from[q]) break;
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            float x[kN];
            if constexpr (Wide) {
              if (whole(u)) {
                v[q][u].values(x);
              } else {
#pragma unroll
                for (int e = 0; e < kN; ++e) x[e] = column(u) + e < a.cols ? to_f32(from[q][column(u) + e]) : 0.0f;
              }
            } else {
              v[q].words(u, lane).values(x);
            }
#pragma unroll
            for (int e = 0; e < kN; ++e) sum[u][e] = fmaf(w[q], x[e], sum[u][e]);
          }
        }
      }
      if ((j0 += 32) >= a.k) break;
      look(t, j0, mine, weight);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (whole(u)) {
        store_piece(to + column(u), sum[u]);
      } else {
#pragma unroll
        for (int e = 0; e < kN; ++e)
          if (column(u) + e >= 0 && column(u) + e < a.cols) to[column(u) + e] = from_f32<TO>(sum[u][e]);
      }
    }
  } while (Wide && (unit += step) < units);
}

// fp32 rows of whole pieces, a few places a token: a thread eight columns, without anything shared in a warp, so that more of them
// are in flight. 4,095 x 4096 to bf16, one of eight places here, 20.9 us where warps that stay take 21.9 (after the experts' products 34
// and 36), 1,000 x 4096 with eight places 23.6 and 26.0; with 12 of them it depends (6,000 x 1000 47.9 and 50.2, 1,000 x 1000 12.7 and
// 11.9), of many tokens' share with 32 it loses (26.1 and 23.0), and 16-bit rows are 5 to 25% slower so.
constexpr int kThreadPlaces = 8;
template <typename TO>
__global__ void __launch_bounds__(kRowThreads) reshard_combine_f32_kernel(Combine a, int chunks) {
  grid_enter();
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= a.tokens * chunks) return;
  const int64_t t = a.tokens * chunks <= 0xffffffffll ? (uint32_t)i / (uint32_t)chunks : i / chunks;
  const int64_t c = (i - t * chunks) * 8;
  const int left = (int)min((int64_t)8, a.cols - c);
  float sum[8] = {};
#pragma unroll 4
  for (int j = 0; j < a.k; ++j) {
    const int p = a.position[t * a.k + j];
    if (p < 0 || p >= a.rows) continue;
    const float w = a.weights ? a.weights[t * a.k + j] : 1.0f;
    float x[8];
    load_values<float, 8>(static_cast<const float *>(a.y) + (int64_t)p * a.y_stride + c, left, true, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) sum[u] = fmaf(w, x[u], sum[u]);
  }
  TO *const to = static_cast<TO *>(a.out) + t * a.out_stride + c;
  if (left == 8) {
    store_piece(to, sum);
  } else {
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (u < left) to[u] = from_f32<TO>(sum[u]);
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
  int lanes;                         // threads a token, of the kernel of whole pieces
  int token_ctas;                    // the CTAs behind them look for rows that no slot owns
};

// Zeros in the rows of the gradient that no slot owns: a warp 32 rows, whose owners it looks up at once.
template <typename TY, bool Wide>
__device__ __forceinline__ void zero_unowned(const CombineBackward &a, int64_t first, int lane) {
  for (uint32_t left = unowned(a.order, a.position, a.tokens * a.k, a.rows, first, lane); left; left &= left - 1)
    for (int c = 0; c < a.pieces; c += kSpan)
      move_span<TY, Wide, false>(nullptr, static_cast<TY *>(a.grad_y) + (first + __ffs(left) - 1) * a.grad_y_stride, a.cols, c, lane, 1.0f);
}

// Whole pieces: `lanes` threads a token (a warp to a CTA, as many as have columns), which read its gradient once and keep the
// rows of eight slots in flight; the dot products by shuffles, then over the token's warps through shared memory. Bound by HBM:
// 8,192 x 2048 bf16, 8 places each, 96 us, 5.9 TB/s (a warp a slot, its chain of loads after one another: 225).
constexpr int kBackSlots = 8, kBackCtas = 3;     // slots in flight, CTAs of an SM
template <typename TG, typename TY>
__global__ void __launch_bounds__(kRowThreads, kBackCtas) reshard_combine_backward_kernel(CombineBackward a) {
  constexpr int kN = kPieceOf<TG, TY>;
  grid_enter();
  __shared__ float part[kRowThreads / 32][kBackSlots];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)blockIdx.x >= a.token_ctas) {
    zero_unowned<TY, true>(a, ((int64_t)((int)blockIdx.x - a.token_ctas) * (kRowThreads / 32) + warp) * 32, lane);
    return;
  }
  const int group = threadIdx.x / a.lanes, me = threadIdx.x - group * a.lanes, warps = a.lanes >> 5;
  const int64_t t = (int64_t)blockIdx.x * (kRowThreads / a.lanes) + group;
  const bool in = t < a.tokens;                    // of a whole warp
  const TG *const g = static_cast<const TG *>(a.grad) + t * a.grad_stride;
  for (int j0 = 0; j0 < a.k; j0 += kBackSlots) {
    const int64_t s = t * a.k + j0 + lane;
    const bool slot = in && lane < kBackSlots && j0 + lane < a.k;
    const int mine = slot ? place_of(a.position, s, a.rows) : -1;
    const bool own = mine >= 0 && a.grad_y && a.order[mine] == s;
    const float weight = slot && a.weights ? a.weights[s] : 1.0f;
    const uint32_t live = __ballot_sync(kFull, mine >= 0), owned = __ballot_sync(kFull, own);
    int p[kBackSlots];
    float w[kBackSlots], dot[kBackSlots];
#pragma unroll
    for (int q = 0; q < kBackSlots; ++q) {
      p[q] = __shfl_sync(kFull, mine, q);
      w[q] = __shfl_sync(kFull, weight, q);
      dot[q] = 0.0f;
    }
    if (live) {
      for (int64_t c = (int64_t)me * kN; c < a.cols; c += (int64_t)a.lanes * kN) {
        Piece<TG, kN, true> gv;
        Piece<TY, kN, true> v[kBackSlots];
        gv.ask(g + c);
        if (a.grad_weights) {
#pragma unroll
          for (int q = 0; q < kBackSlots; ++q)
            if (live >> q & 1) v[q].ask(static_cast<const TY *>(a.y) + (int64_t)p[q] * a.y_stride + c);
        }
        float x[kN];
        gv.take(g + c, x);
#pragma unroll
        for (int q = 0; q < kBackSlots; ++q) {
          if (owned >> q & 1) {
            float z[kN];
#pragma unroll
            for (int e = 0; e < kN; ++e) z[e] = x[e] * w[q];
            store_piece(static_cast<TY *>(a.grad_y) + (int64_t)p[q] * a.grad_y_stride + c, z);
          }
        }
        if (a.grad_weights) {
#pragma unroll
          for (int q = 0; q < kBackSlots; ++q) {
            if (!(live >> q & 1)) continue;
            float y[kN];
            v[q].take(nullptr, y);
#pragma unroll
            for (int e = 0; e < kN; ++e) dot[q] = fmaf(x[e], y[e], dot[q]);
          }
        }
      }
    }
    if (!a.grad_weights) continue;
    // Eight sums over the lanes: halves are exchanged until a lane has one, of the slot that its upper three bits name.
#pragma unroll
    for (int o = 16, n = kBackSlots / 2; n; o >>= 1, n >>= 1)
#pragma unroll
      for (int q = 0; q < n; ++q) {
        const float give = lane & o ? dot[q] : dot[q + n];
        dot[q] = (lane & o ? dot[q + n] : dot[q]) + __shfl_xor_sync(kFull, give, o);
      }
    dot[0] += __shfl_xor_sync(kFull, dot[0], 2);
    dot[0] += __shfl_xor_sync(kFull, dot[0], 1);
    if (warps == 1) {
      if (in && (lane & 3) == 0 && j0 + (lane >> 2) < a.k) a.grad_weights[t * a.k + j0 + (lane >> 2)] = dot[0];
      continue;
    }
    if (j0) __syncthreads();                       // the slots before have been added
    if ((lane & 3) == 0) part[warp][lane >> 2] = dot[0];
    __syncthreads();
    if (in && me < kBackSlots && j0 + me < a.k) {
      float sum = 0.0f;
      for (int i = 0; i < warps; ++i) sum += part[group * warps + i][me];
      a.grad_weights[t * a.k + j0 + me] = sum;
    }
  }
}

// Rows that start anywhere: a warp a slot (8,191 x 2867 bf16, four places each: 102 us).
template <typename TG, typename TY>
__global__ void __launch_bounds__(kRowThreads) reshard_combine_backward_any_kernel(CombineBackward a) {
  constexpr int kN = kPieceOf<TG, TY>, kU = 2;
  grid_enter();
  const int lane = threadIdx.x & 31;
  if ((int)blockIdx.x >= a.token_ctas) {
    zero_unowned<TY, false>(a, ((int64_t)((int)blockIdx.x - a.token_ctas) * (kRowThreads / 32) + (threadIdx.x >> 5)) * 32, lane);
    return;
  }
  const int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (i >= a.tokens * a.k) return;
  const int p = place_of(a.position, i, a.rows);
  float dot = 0.0f;
  if (p >= 0) {
    const TG *const g = static_cast<const TG *>(a.grad) + i / a.k * a.grad_stride;
    const TY *const y = a.grad_weights ? static_cast<const TY *>(a.y) + (int64_t)p * a.y_stride : nullptr;
    TY *const to = a.grad_y && a.order[p] == i ? static_cast<TY *>(a.grad_y) + (int64_t)p * a.grad_y_stride : nullptr;
    const float w = a.weights ? a.weights[i] : 1.0f;
    // The pieces are those of a dense gradient of y whether it is written or not, dense or not: they set the order of the dot
    // product.
    const TY *const dense = reinterpret_cast<const TY *>(p * a.cols * (int64_t)sizeof(TY));
    for (int c1 = lane; c1 < a.pieces; c1 += 32 * kU) {
      Piece<TG, kN, false> gv[kU];
      Piece<TY, kN, false> yv[kU];
      int64_t c[kU];
      bool whole[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        c[u] = piece_start<TY, kN, false>(c1 + 32 * u, dense);
        whole[u] = c[u] >= 0 && c[u] + kN <= a.cols;
        if (whole[u]) {
          gv[u].ask(g + c[u]);
          if (y) yv[u].ask(y + c[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        float x[kN], z[kN] = {};
        if (whole[u]) {
          gv[u].take(g + c[u], x);
          if (y) yv[u].take(y + c[u], z);
        } else {
#pragma unroll
          for (int e = 0; e < kN; ++e) {
            const bool in = c[u] + e >= 0 && c[u] + e < a.cols;
            x[e] = in ? to_f32(g[c[u] + e]) : 0.0f;
            z[e] = in && y ? to_f32(y[c[u] + e]) : 0.0f;
          }
        }
#pragma unroll
        for (int e = 0; e < kN; ++e) {
          dot = fmaf(x[e], z[e], dot);
          x[e] *= w;
        }
        if (!to) continue;
        if (whole[u] && (reinterpret_cast<uintptr_t>(to + c[u]) & (kN * sizeof(TY) - 1)) == 0) {
          store_piece(to + c[u], x);
        } else {
#pragma unroll
          for (int e = 0; e < kN; ++e)
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

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int launched(cudaError_t e, const char *what) { return e == cudaSuccess ? RESHARD_OK : cuda_error(e, what); }

// A launch of so many warps, in small CTAs where they would leave SMs without one.
template <typename... K, typename... A>
cudaError_t launch_warps(void (*kernel)(K...), int64_t warps, cudaStream_t stream, A &&...args) {
  const int block = warps <= 2048 ? kFewThreads : kRowThreads;
  return launch(kernel, dim3((unsigned)ceil_div(warps, block / 32)), block, 0, 1, stream, std::forward<A>(args)...);
}

}  // namespace

int enqueue_combine(const Combine &a, cudaStream_t stream) {
  if (a.tokens == 0 || a.cols == 0) return RESHARD_OK;
  int sms = 0;
  if (const int rc = device_sms(&sms)) return rc;
  const bool wide = aligned16(a.y, a.y_stride, element_bytes(a.dtype)) && aligned16(a.out, a.out_stride, element_bytes(a.out_dtype));
  if (wide && a.dtype == RESHARD_F32 && a.k <= kThreadPlaces) {
    const int chunks = (int)ceil_div(a.cols, 8);
    const int block = a.tokens * chunks <= 32768 ? kFewThreads : kRowThreads;      // a few tokens' columns spread over the SMs
    return launched(by_type(a.out_dtype, [&](auto o) {
      return launch(reshard_combine_f32_kernel<decltype(o)>, dim3((unsigned)ceil_div(a.tokens * chunks, block)), block, 0, 1, stream, a, chunks);
    }), "launching reshard_combine_f32_kernel");
  }
  return launched(by_type(a.dtype, [&](auto y) {
    using TY = decltype(y);
    return by_type(a.out_dtype, [&](auto o) {
      using TO = decltype(o);
      using Shape = CombineShape<TY, TO>;
      const int spans = (int)ceil_div(piece_count(a.cols, Shape::kN, wide), 32 * Shape::kPieces);
      const int64_t warps = a.tokens * spans;
      const int block = warps <= 2048 ? kFewThreads : kRowThreads;
      const int64_t ctas = ceil_div(warps, block / 32), stay = (int64_t)sms * Shape::kCtas * (kRowThreads / block);
      const unsigned grid = (unsigned)(wide ? std::min(ctas, stay) : ctas);      // rows that start anywhere: a warp has one span
      return launch(wide ? reshard_combine_kernel<TY, TO, true> : reshard_combine_kernel<TY, TO, false>, dim3(grid), block, 0, 1, stream, a, spans);
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
    c.unsupported((double)std::max<int64_t>(tokens * k, rows) * (double)(cols / 256 + 1) > 2.0 * INT32_MAX, "too many rows and columns for one launch");
  }
}

}  // namespace
}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int reshard_permute(const void *x, int dtype, int64_t tokens, int64_t cols, int64_t row_stride, const int32_t *order,
                               const int32_t *position, int k, void *out, int64_t rows, int64_t out_stride, int zero_rest, reshard_stream_t stream_) try {
  Checks c("reshard_permute");
  check_slots(c, tokens, cols, k, rows);
  c.invalid(!element_bytes(dtype), "dtype must be BF16, F16 or F32");
  c.invalid(row_stride < cols || out_stride < cols, "a row stride is shorter than the row");
  const int es = element_bytes(dtype);
  const bool work = (tokens > 0 || zero_rest) && cols > 0 && rows > 0;
  if (work && c.ok()) {
    if (tokens > 0) {
      c.pointer(x, "x", (uintptr_t)es);
      c.pointer(position, "position", 4);
    }
    c.pointer(order, "order", 4);
    c.pointer(out, "out", (uintptr_t)es);
  }
  if (!c.ok()) return c.report();
  if (!work) return RESHARD_OK;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  Permute a{x, tokens, cols, row_stride, order, position, k, out, rows, out_stride, 0, zero_rest != 0};
  const int64_t rest = zero_rest ? ceil_div(rows, 32) : 0;      // warps
  if (aligned16(x, row_stride, es) && aligned16(out, out_stride, es) && cols * es % 16 == 0) {
    a.cols = cols * es / 16, a.stride = row_stride * es / 16, a.out_stride = out_stride * es / 16;
    a.spans = (int)ceil_div(a.cols, kSpan);
    return launched(launch_warps(reshard_permute_kernel, tokens * a.spans + rest, stream, a), "launching reshard_permute_kernel");
  }
  // values are copied as they are: the types of a size share a kernel
  a.spans = (int)ceil_div(piece_count(cols, 16 / es, false), kSpan);
  return launched(launch_warps(es == 4 ? reshard_permute_any_kernel<float> : reshard_permute_any_kernel<__half>, tokens * k * a.spans + rest, stream, a),
                  "launching reshard_permute_any_kernel");
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
  const bool work = c.ok() && ((tokens > 0 && (grad_weights || grad_y)) || (grad_y && rows > 0));
  if (work) {
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
  if (!work) return RESHARD_OK;
  const bool wide = aligned16(grad, grad_stride, element_bytes(grad_dtype)) && (!grad_weights || aligned16(y, row_stride, es)) &&
                    (!grad_y || aligned16(grad_y, grad_y_stride, es)) && cols * es % 16 == 0;
  CombineBackward a{grad, grad_stride, y, rows, cols, row_stride, order, position, weights, tokens, k, grad_y, grad_y_stride, grad_weights, 0, 32, 0};
  return launched(by_type(grad_dtype, [&](auto g) {
    using TG = decltype(g);
    return by_type(dtype, [&](auto t) {
      using TY = decltype(t);
      constexpr int kN = kPieceOf<TG, TY>;
      while (a.lanes < kRowThreads && a.lanes * kN < cols) a.lanes *= 2;
      a.token_ctas = (int)(wide ? ceil_div(tokens, kRowThreads / a.lanes) : ceil_div(tokens * k, kRowThreads / 32));
      a.pieces = (int)std::max(piece_count(cols, kN, wide), piece_count(cols, kPieceOf<TY, TY>, wide));      // of a row, and of its zeros
      const int64_t ctas = a.token_ctas + (grad_y ? ceil_div(rows, kRowThreads) : 0);
      return launch(wide ? reshard_combine_backward_kernel<TG, TY> : reshard_combine_backward_any_kernel<TG, TY>, dim3((unsigned)ctas), kRowThreads, 0, 1,
                    reinterpret_cast<cudaStream_t>(stream), a);
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
  if (c.ok()) c.unsupported((double)tokens * (double)(cols / 256 + 1) > 2.0 * INT32_MAX, "too many rows and columns for one launch");
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
    a.spans = (int)ceil_div(piece_count(cols, kPieceOf<T, T>, wide), kSpan);
    auto *kernel = wide ? scale == 1.0f ? reshard_embedding_kernel<T, true, false> : reshard_embedding_kernel<T, true, true>
                        : scale == 1.0f ? reshard_embedding_kernel<T, false, false> : reshard_embedding_kernel<T, false, true>;
    return launch_warps(kernel, tokens * a.spans, reinterpret_cast<cudaStream_t>(stream), a);
  }), "launching reshard_embedding_kernel");
} OPS_CATCH
