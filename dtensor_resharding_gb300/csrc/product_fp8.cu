// The matrix product over 8-bit values with block scales, dense or grouped by expert, on the tcgen05 tensor cores:
//
//   out[m, n] = sum_b sa[m, b] sw[n / 128, b] (sum_{k in block b} a[m, k] w[n, k])
//
// The scales differ along K, so the inner sum of each 128-block leaves the tensor cores as fp32 (tensor memory) and is
// scaled and added in registers: out = fma(sa sw, inner, out) per block. Tensor memory holds two such partial tiles, so
// that the tensor cores work on one while the epilogue warps read the other.
//
// Two kernels, by which operand sits on the tensor cores' 128 rows:
//  - wide: 128 rows of `a` x 256 rows of `w`, persistent, for many rows a group. A thread of the eight epilogue warps
//    owns one row and 128 columns, so that one scale a block serves all of them. Bound by the tensor cores.
//  - narrow: 128 rows of `w` x 16 .. 128 rows of `a`, for few rows a group: the tile's narrow side fits the
//    rows at hand instead of padding them to 128. Bound by the read of the weights. Where the tiles alone do not fill
//    the GPU, a cluster of CTAs splits K and adds its partial tiles through distributed shared memory, in rank order.
// Both can end in silu(gate) * up, quantized by rows (the expert layer's first product): a tile then holds the 128
// columns of one quantization block and their gate and up rows.
//
// Operands come by TMA (128-byte swizzle, K along the row), rows beyond a tensor as zeros. Rows of a tile beyond its
// group's end belong to the next group: they are computed and not stored.
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "tensor_core.cuh"

namespace reshard {
namespace ops {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kBlockK = kScaleBlock;   // bytes of K a stage: one scale block, four products of 32

__device__ int g_ops_status;

struct Args {
  const float *a_scale;
  int64_t as_row, as_block;
  const float *w_scale;
  const int32_t *offsets;
  int groups, m, n, kblocks;
  int wblocks;          // blocks of w's rows in one group's scales
  void *out;
  int out_dtype;
  int64_t out_stride;
  float *out_scale;
  int64_t os_row, os_block;
};

// Offsets come from the device: kept within the rows the tensors have.
__device__ __forceinline__ int row_offset(const Args &p, int g) {
  return p.offsets ? min(max(p.offsets[g], 0), p.m) : g ? p.m : 0;
}

__device__ __forceinline__ float silu_times(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// 8 consecutive 32-bit words; p on a 32-byte boundary.
__device__ __forceinline__ void store32(void *p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
               "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// ---------------------------------------------------------------------------------------------------------- wide --

constexpr int kWideM = 128, kWideN = 256, kWideStages = 4;
constexpr int kWideStageBytes = (kWideM + kWideN) * kBlockK;
constexpr int kWideThreads = 320;        // 8 epilogue warps, the loader, the issuer

struct WideShared {
  uint64_t full[kWideStages], empty[kWideStages], done[2], taken[2], paired[2], last;
  uint32_t tmem;
  int stop;
  uint32_t amax[2][2][kWideM];
  int off[RESHARD_MAX_GROUPS + 1], tiles[RESHARD_MAX_GROUPS + 1];   // row offsets; tiles of rows before each group
};
constexpr size_t kWideSmem = 1024 + (size_t)kWideStages * kWideStageBytes + sizeof(WideShared);

struct WideTile {
  int g, row, rows, n;     // group, first row, rows of the group from there (can exceed the tile), column tile
};
__device__ __forceinline__ WideTile wide_tile(const WideShared &s, int groups, int ntiles, int64_t t) {
  int lo = 0, hi = groups - 1;          // the last group whose first tile is <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((int64_t)s.tiles[mid] * ntiles <= t) lo = mid;
    else hi = mid - 1;
  }
  const int here = s.tiles[lo + 1] - s.tiles[lo];
  const int64_t l = t - (int64_t)s.tiles[lo] * ntiles;
  const int n = (int)(l / here), m = (int)(l - (int64_t)n * here);     // row tiles first: neighbours share w's tile
  WideTile r;
  r.g = lo;
  r.row = s.off[lo] + m * kWideM;
  r.rows = s.off[lo + 1] - r.row;
  r.n = n;
  return r;
}

template <typename T>
__device__ __forceinline__ void store_row(T *to, const uint64_t (&acc)[64], int left) {
  if (left >= 128 && (reinterpret_cast<uintptr_t>(to) & 31) == 0) {
    constexpr int per = 32 / sizeof(T);
#pragma unroll
    for (int c = 0; c < 128; c += per) {
      uint32_t v[8];
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = (uint32_t)(acc[(c + j) / 2] >> (32 * (j & 1)));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = pack2<T>(lo32(acc[c / 2 + j]), hi32(acc[c / 2 + j]));
      }
      store32(to + c, v);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 128; ++c)
      if (c < left) to[c] = from_f32<T>(c & 1 ? hi32(acc[c / 2]) : lo32(acc[c / 2]));
  }
}

template <bool Gated>
__global__ void __launch_bounds__(kWideThreads, 1)
    reshard_product_wide_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw, const Args p) {
  extern __shared__ uint8_t raw[];
  uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  WideShared &s = *reinterpret_cast<WideShared *>(stages + (size_t)kWideStages * kWideStageBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Stop stop{&s.stop, &g_ops_status};
  if (tid == 0) {
    for (int i = 0; i < kWideStages; ++i) {
      bar_init(smem_addr(&s.full[i]), 1);
      bar_init(smem_addr(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&s.done[i]), 1);
      bar_init(smem_addr(&s.taken[i]), 8);
      bar_init(smem_addr(&s.paired[i]), 8);
    }
    bar_init(smem_addr(&s.last), 1);
    s.stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) tmem_alloc(smem_addr(&s.tmem), 512);
  grid_enter();
  for (int g = tid; g <= p.groups; g += kWideThreads) s.off[g] = row_offset(p, g);
  __syncthreads();
  if (warp == 0) {                     // running sum of the groups' row tiles
    int base = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      const int g = g0 + lane;
      const int own = g < p.groups ? max(0, s.off[g + 1] - s.off[g] + kWideM - 1) / kWideM : 0;
      int sum = own;
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += x;
      }
      if (g < p.groups) s.tiles[g] = base + sum - own;
      base += __shfl_sync(kFull, sum, 31);
    }
    if (lane == 0) s.tiles[p.groups] = base;
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = s.tmem;
  constexpr int kCols = Gated ? kWideN / 2 : kWideN;      // output columns of a tile
  const int ntiles = (p.n + kCols - 1) / kCols;
  const int64_t total = (int64_t)s.tiles[p.groups] * ntiles;

  if (warp == 8) {
    // ---- loader
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
        const WideTile w = wide_tile(s, p.groups, ntiles, t);
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const uint32_t st = it % kWideStages, bar = smem_addr(&s.full[st]);
          if (!(ok = bar_wait(smem_addr(&s.empty[st]), (it / kWideStages & 1) ^ 1, stop))) break;
          const uint32_t to = smem_addr(stages) + st * kWideStageBytes;
          bar_expect(bar, kWideStageBytes);
          tma_2d(to, &ma, kb * kBlockK, w.row, bar);
          const uint32_t tw = to + kWideM * kBlockK;
          if (Gated) {                 // columns 0-63: gate, 64-127: up, and the same for the tile's other half
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              tma_3d(tw + h * 16384, &mw, kb * kBlockK, w.n * kCols + h * 64, w.g, bar);
              tma_3d(tw + h * 16384 + 8192, &mw, kb * kBlockK, p.n + w.n * kCols + h * 64, w.g, bar);
            }
          } else {
            tma_3d(tw, &mw, kb * kBlockK, w.n * kCols, w.g, bar);
            tma_3d(tw + 16384, &mw, kb * kBlockK, w.n * kCols + 128, w.g, bar);
          }
        }
      }
      if (!ok)                         // stopped: what is on its way still lands in this CTA's memory
        for (uint32_t i = it > kWideStages ? it - kWideStages : 0; i < it; ++i)
          bar_drain(smem_addr(&s.full[i % kWideStages]), i / kWideStages & 1);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ---- issuer
    if (elect_one()) {
      const uint32_t idesc = instruction(kWideN);
      uint32_t it = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const uint32_t st = it % kWideStages, half = it & 1;
          if (!(ok = bar_wait(smem_addr(&s.taken[half]), (it >> 1 & 1) ^ 1, stop))) break;
          if (!(ok = bar_wait(smem_addr(&s.full[st]), it / kWideStages & 1, stop))) break;
          tc_after_sync();
          const uint32_t base = smem_addr(stages) + st * kWideStageBytes;
          const uint64_t a = operand(base), b = operand(base + kWideM * kBlockK);
#pragma unroll
          for (int k = 0; k < kBlockK / 32; ++k) mma_e4m3(tmem + half * kWideN, a + 2 * k, b + 2 * k, idesc, k > 0);
          mma_commit(smem_addr(&s.empty[st]));
          mma_commit(smem_addr(&s.done[half]));
        }
      }
      if (!ok) {
        mma_commit(smem_addr(&s.last));
        bar_drain(smem_addr(&s.last), 0);
      }
    }
    __syncwarp();
  } else {
    // ---- epilogue: a row and 128 columns a thread
    const int half_n = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + half_n * 128;
    uint32_t it = 0, tile_no = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < total; t += gridDim.x, ++tile_no) {
      const WideTile w = wide_tile(s, p.groups, ntiles, t);
      const bool in = r < w.rows;
      const float *sa = p.a_scale + (int64_t)(w.row + (in ? r : 0)) * p.as_row;
      // gated: gate and up scales of the tile's one block; otherwise this half's block
      const int wb = Gated ? w.n : min(w.n * 2 + half_n, p.wblocks - 1);
      const float *sw = p.w_scale + ((int64_t)w.g * p.wblocks + wb) * p.kblocks;
      const float *su = Gated ? sw + (int64_t)(p.n / kScaleBlock) * p.kblocks : sw;
      uint64_t acc[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) acc[i] = 0;
      float a0 = sa[0], g0 = sw[0], u0 = su[0], a1 = 0, g1 = 0, u1 = 0;
      if (p.kblocks > 1) a1 = sa[p.as_block], g1 = sw[1], u1 = su[1];
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        float a2 = 0, g2 = 0, u2 = 0;        // two blocks ahead: their latency passes under the waits
        if (kb + 2 < p.kblocks) a2 = sa[(int64_t)(kb + 2) * p.as_block], g2 = sw[kb + 2], u2 = su[kb + 2];
        const float s0 = a0 * g0, s1 = Gated ? a0 * u0 : s0;
        const uint32_t half = it & 1;
        ok = bar_wait(smem_addr(&s.done[half]), it >> 1 & 1, stop);
        if (__any_sync(kFull, !ok)) {
          ok = false;
          break;
        }
        tc_after_sync();
        uint32_t v[2][16];
        tmem_load16(from + half * kWideN, v[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_loaded(v[c & 1]);
          if (c < 7) {
            tmem_load16(from + half * kWideN + (c + 1) * 16, v[(c + 1) & 1]);
          } else {                     // the partial tile is in registers
            tc_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(smem_addr(&s.taken[half]));
          }
          const float sc = c < 4 ? s0 : s1;
#pragma unroll
          for (int i = 0; i < 8; ++i) fma2(acc[c * 8 + i], v[c & 1][2 * i], v[c & 1][2 * i + 1], sc);
        }
        a0 = a1, g0 = g1, u0 = u1;
        a1 = a2, g1 = g2, u1 = u2;
      }
      if (!ok) break;
      const int64_t row = w.row + r;
      if (!Gated) {
        const int n0 = w.n * kCols + half_n * 128, left = p.n - n0;
        if (in && left > 0) {
          const int64_t at = row * p.out_stride + n0;
          if (p.out_dtype == RESHARD_BF16) store_row(static_cast<__nv_bfloat16 *>(p.out) + at, acc, left);
          else if (p.out_dtype == RESHARD_F16) store_row(static_cast<__half *>(p.out) + at, acc, left);
          else store_row(static_cast<float *>(p.out) + at, acc, left);
        }
      } else {
        // columns c of acc: gate 0 .. 63, up 64 .. 127; this thread's 64 of the row's 128 values
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = silu_times(lo32(acc[i]), lo32(acc[32 + i])), y = silu_times(hi32(acc[i]), hi32(acc[32 + i]));
          m = max(m, max(magnitude(x), magnitude(y)));
          acc[i] = (uint64_t)__float_as_uint(y) << 32 | __float_as_uint(x);
        }
        s.amax[tile_no & 1][half_n][r] = m;
        __syncwarp();
        if (lane == 0) bar_arrive(smem_addr(&s.paired[tile_no & 1]));
        ok = bar_wait(smem_addr(&s.paired[tile_no & 1]), tile_no >> 1 & 1, stop);
        if (__any_sync(kFull, !ok)) break;
        m = max(m, s.amax[tile_no & 1][half_n ^ 1][r]);
        float scale, inv;
        block_scale(m, scale, inv);
        if (in) {
          if (half_n == 0) p.out_scale[row * p.os_row + w.n * p.os_block] = scale;
          uint8_t *to = static_cast<uint8_t *>(p.out) + row * p.out_stride + w.n * kCols + half_n * 64;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint64_t x = acc[h * 16 + 2 * i], y = acc[h * 16 + 2 * i + 1];
              q[i] = e4m3x4(lo32(x) * inv, hi32(x) * inv, lo32(y) * inv, hi32(y) * inv);
            }
            store32(to + 32 * h, q);
          }
        }
      }
    }
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp == 9) tmem_free(tmem, 512);
}

// -------------------------------------------------------------------------------------------------------- narrow --

constexpr int kNarrowM = 128;            // rows of w (of gate and of up, when gated)
constexpr int kNarrowThreads = 192;      // 4 epilogue warps, the loader, the issuer

template <int NT, bool Gated>
struct Narrow {
  static constexpr int kParts = Gated ? 2 : 1;
  static constexpr int kStageBytes = (kParts * kNarrowM + NT) * kBlockK;
  static constexpr int kStages = 110592 / kStageBytes;     // two CTAs an SM
  static constexpr int kPartial = NT * kNarrowM * 4 * kParts;   // a CTA's sums, in stage memory, for the cluster
  static constexpr int kColumns = 2 * NT * kParts < 32 ? 32 : 2 * NT * kParts;
  static_assert(kStages >= 2 && kPartial <= kStages * kStageBytes, "stages");
  struct Shared {
    uint64_t full[kStages], empty[kStages], done[2], taken[2], last;
    uint32_t tmem;
    int stop;
    int tile[4];                   // group, first row, rows, column tile
    alignas(16) float scale[4][2][kParts][NT];       // per epilogue warp, two blocks
    uint32_t amax[4][NT];
  };
  static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + sizeof(Shared);
};

template <int NT, bool Gated>
__global__ void __launch_bounds__(kNarrowThreads)
    reshard_product_narrow_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw, const Args p, const int split) {
  using C = Narrow<NT, Gated>;
  using Shared = typename C::Shared;
  constexpr int kStages = C::kStages, kParts = C::kParts;
  extern __shared__ uint8_t raw[];
  uint8_t *stages = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  Shared &s = *reinterpret_cast<Shared *>(stages + (size_t)kStages * C::kStageBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Stop stop{&s.stop, &g_ops_status};
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(smem_addr(&s.full[i]), 1);
      bar_init(smem_addr(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&s.done[i]), 1);
      bar_init(smem_addr(&s.taken[i]), 4);
    }
    bar_init(smem_addr(&s.last), 1);
    s.stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) tmem_alloc(smem_addr(&s.tmem), C::kColumns);
  grid_enter();
  const int ntiles = (p.n + kNarrowM - 1) / kNarrowM;
  const int rank = (int)(blockIdx.x % split);       // consecutive CTAs are a cluster
  if (warp == 0) {
    const int64_t t = blockIdx.x / split;
    int64_t base = 0;
    bool found = false;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
      const int x = g0 + lane;
      const int lo = x < p.groups ? row_offset(p, x) : 0, hi = x < p.groups ? row_offset(p, x + 1) : 0;
      const int own = max(0, hi - lo + NT - 1) / NT;
      int sum = own;
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, sum, o);
        if (lane >= o) sum += y;
      }
      const int64_t first = (base + sum - own) * ntiles;
      const bool mine = own > 0 && t >= first && t < first + (int64_t)own * ntiles;
      found = __any_sync(kFull, mine);
      if (mine) {
        s.tile[0] = x;
        s.tile[1] = lo + (int)((t - first) / ntiles) * NT;
        s.tile[2] = hi;
        s.tile[3] = (int)((t - first) % ntiles);
      }
      if (found) break;
      base += __shfl_sync(kFull, sum, 31);
    }
    if (!found && lane == 0) s.tile[0] = -1;
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = s.tmem;
  const int group = s.tile[0], row0 = s.tile[1], nt = s.tile[3];
  const int rows = group < 0 ? 0 : min(NT, s.tile[2] - row0);
  const int kb0 = group < 0 ? 0 : (int)((int64_t)p.kblocks * rank / split), kb1 = group < 0 ? 0 : (int)((int64_t)p.kblocks * (rank + 1) / split);
  const int wide = (rows + 15) & ~15;               // columns the products compute
  float acc[kParts][NT];
#pragma unroll
  for (int q = 0; q < kParts; ++q)
#pragma unroll
    for (int c = 0; c < NT; ++c) acc[q][c] = 0.0f;
  bool ok = true;

  if (warp == 4) {
    if (elect_one()) {
      uint32_t it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t st = it % kStages, bar = smem_addr(&s.full[st]);
        if (!(ok = bar_wait(smem_addr(&s.empty[st]), (it / kStages & 1) ^ 1, stop))) break;
        const uint32_t to = smem_addr(stages) + st * C::kStageBytes;
        bar_expect(bar, C::kStageBytes);
#pragma unroll
        for (int q = 0; q < kParts; ++q) tma_3d(to + q * kNarrowM * kBlockK, &mw, kb * kBlockK, q * p.n + nt * kNarrowM, group, bar);
        tma_2d(to + kParts * kNarrowM * kBlockK, &ma, kb * kBlockK, row0, bar);
      }
      if (!ok)
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) bar_drain(smem_addr(&s.full[i % kStages]), i / kStages & 1);
    }
    __syncwarp();
  } else if (warp == 5) {
    if (elect_one()) {
      const uint32_t idesc = instruction(wide);
      uint32_t it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const uint32_t st = it % kStages, half = it & 1;
        if (!(ok = bar_wait(smem_addr(&s.taken[half]), (it >> 1 & 1) ^ 1, stop))) break;
        if (!(ok = bar_wait(smem_addr(&s.full[st]), it / kStages & 1, stop))) break;
        tc_after_sync();
        const uint32_t base = smem_addr(stages) + st * C::kStageBytes;
        const uint64_t b = operand(base + kParts * kNarrowM * kBlockK);
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          const uint64_t a = operand(base + q * kNarrowM * kBlockK);
#pragma unroll
          for (int k = 0; k < kBlockK / 32; ++k) mma_e4m3(tmem + (half * kParts + q) * NT, a + 2 * k, b + 2 * k, idesc, k > 0);
        }
        mma_commit(smem_addr(&s.empty[st]));
        mma_commit(smem_addr(&s.done[half]));
      }
      if (!ok) {
        mma_commit(smem_addr(&s.last));
        bar_drain(smem_addr(&s.last), 0);
      }
    }
    __syncwarp();
  } else if (group >= 0) {
    // epilogue: one row of w a thread; the scales of the tile's rows of a are shared out by the warp
    constexpr int kPer = (NT + 31) / 32;
    const float *sw[kParts];
#pragma unroll
    for (int q = 0; q < kParts; ++q)
      sw[q] = p.w_scale + ((int64_t)group * p.wblocks + q * (p.n / kScaleBlock) + nt) * p.kblocks;
    float a0[kPer], a1[kPer], w0[kParts], w1[kParts];
    auto fetch = [&](int kb, float (&a)[kPer], float (&w)[kParts]) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int c = lane + 32 * i;
        a[i] = c < rows && kb < kb1 ? p.a_scale[(int64_t)(row0 + c) * p.as_row + (int64_t)kb * p.as_block] : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < kParts; ++q) w[q] = kb < kb1 ? sw[q][kb] : 0.0f;
    };
    fetch(kb0, a0, w0);
    fetch(kb0 + 1, a1, w1);
    const uint32_t from = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const uint32_t half = it & 1;
#pragma unroll
      for (int q = 0; q < kParts; ++q)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (lane + 32 * i < NT) s.scale[warp][half][q][lane + 32 * i] = a0[i] * w0[q];
#pragma unroll
      for (int i = 0; i < kPer; ++i) a0[i] = a1[i];
#pragma unroll
      for (int q = 0; q < kParts; ++q) w0[q] = w1[q];
      fetch(kb + 2, a1, w1);
      __syncwarp();
      ok = bar_wait(smem_addr(&s.done[half]), it >> 1 & 1, stop);
      if (__any_sync(kFull, !ok)) {
        ok = false;
        break;
      }
      tc_after_sync();
#pragma unroll
      for (int q = 0; q < kParts; ++q) {
#pragma unroll
        for (int c = 0; c < NT; c += 16) {
          if (c < wide) {
            uint32_t v[16];
            tmem_load16(from + (half * kParts + q) * NT + c, v);
            tmem_loaded(v);
            const float4 *sc = reinterpret_cast<const float4 *>(&s.scale[warp][half][q][c]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float4 f = sc[i];
              acc[q][c + 4 * i] = fmaf(__uint_as_float(v[4 * i]), f.x, acc[q][c + 4 * i]);
              acc[q][c + 4 * i + 1] = fmaf(__uint_as_float(v[4 * i + 1]), f.y, acc[q][c + 4 * i + 1]);
              acc[q][c + 4 * i + 2] = fmaf(__uint_as_float(v[4 * i + 2]), f.z, acc[q][c + 4 * i + 2]);
              acc[q][c + 4 * i + 3] = fmaf(__uint_as_float(v[4 * i + 3]), f.w, acc[q][c + 4 * i + 3]);
            }
          }
        }
      }
      tc_before_sync();
      __syncwarp();
      if (lane == 0) bar_arrive(smem_addr(&s.taken[half]));
    }
  }

  if (split > 1) {
    // Every CTA's products are done (its epilogue saw the last one), so its stages hold the sums from here; each rank
    // then adds every split-th row of a, over the ranks in order.
    float *part = reinterpret_cast<float *>(stages);
    if (warp < 4) {
#pragma unroll
      for (int q = 0; q < kParts; ++q)
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < rows) part[(q * NT + c) * kNarrowM + tid] = acc[q][c];
    }
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
    if (warp < 4) {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        if (c < rows && c % split == rank) {
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            float sum = 0.0f;
            for (int r = 0; r < split; ++r) {
              uint32_t at;
              float x;
              asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&part[(q * NT + c) * kNarrowM + tid])), "r"(r));
              asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(at) : "memory");
              sum += x;
            }
            acc[q][c] = sum;
          }
        }
      }
    }
    asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
  }

  if (warp < 4 && group >= 0) {
    const bool whole = !s.stop;            // a stopped CTA's sums are incomplete: nothing of them is stored
    const int n = nt * kNarrowM + tid;
    if (!Gated) {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        if (whole && c < rows && n < p.n && (split == 1 || c % split == rank)) {
          const int64_t at = (int64_t)(row0 + c) * p.out_stride + n;
          if (p.out_dtype == RESHARD_BF16) static_cast<__nv_bfloat16 *>(p.out)[at] = __float2bfloat16_rn(acc[0][c]);
          else if (p.out_dtype == RESHARD_F16) static_cast<__half *>(p.out)[at] = __float2half_rn(acc[0][c]);
          else static_cast<float *>(p.out)[at] = acc[0][c];
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        acc[0][c] = silu_times(acc[0][c], acc[kParts - 1][c]);
        const uint32_t m = __reduce_max_sync(kFull, magnitude(acc[0][c]));
        if (lane == 0) s.amax[warp][c] = m;
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        if (whole && c < rows && (split == 1 || c % split == rank)) {
          float scale, inv;
          block_scale(max(max(s.amax[0][c], s.amax[1][c]), max(s.amax[2][c], s.amax[3][c])), scale, inv);
          if (tid == 0) p.out_scale[(int64_t)(row0 + c) * p.os_row + (int64_t)nt * p.os_block] = scale;
          static_cast<uint8_t *>(p.out)[(int64_t)(row0 + c) * p.out_stride + n] = (uint8_t)e4m3x2(acc[0][c] * inv, 0.0f);
        }
      }
    }
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp == 5) tmem_free(tmem, C::kColumns);
}

// ----------------------------------------------------------------------------------------------------- host side --

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Bytes [batch, rows, cols] in boxes of box_rows x 128, 128-byte swizzle; batch 0: a plain matrix.
int encode(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t stride, int64_t batch, int64_t batch_stride, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return fail(RESHARD_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)stride, (cuuint64_t)batch_stride};
  const cuuint32_t box[3] = {(cuuint32_t)kBlockK, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, batch ? 3 : 2, const_cast<void *>(base), dims, strides, box, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(RESHARD_ERR_CUDA, "cuTensorMapEncodeTiled failed with " + std::to_string((int)r));
  return RESHARD_OK;
}

// The dynamic shared memory of a kernel, allowed once per device.
template <auto kernel>
int allow_smem(size_t bytes) {
  static std::mutex mu;
  static uint64_t done = 0;
  int dev = 0;
  OPS_CUDA(cudaGetDevice(&dev));
  std::lock_guard<std::mutex> lock(mu);
  if (dev < 64 && (done >> dev & 1)) return RESHARD_OK;
  OPS_CUDA(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes));
  if (dev < 64) done |= 1ull << dev;
  return RESHARD_OK;
}

template <bool Gated>
int enqueue_wide(const Product &p, const Args &a, int sms, cudaStream_t stream) {
  CUtensorMap ma, mw;
  int rc = encode(&ma, p.a, p.k, p.m, p.a_stride, 0, 0, kWideM);
  if (!rc) rc = encode(&mw, p.w, p.k, Gated ? 2 * p.n : p.n, p.w_stride, p.groups, p.w_batch, Gated ? 64 : 128);
  if (!rc) rc = allow_smem<&reshard_product_wide_kernel<Gated>>(kWideSmem);
  if (rc) return rc;
  const int64_t cols = Gated ? kWideN / 2 : kWideN;
  const int64_t most = (p.m / kWideM + std::min<int64_t>(p.groups, p.m)) * ((p.n + cols - 1) / cols);
  const cudaError_t e = launch(reshard_product_wide_kernel<Gated>, dim3((unsigned)std::min<int64_t>(sms, most)), kWideThreads, kWideSmem, 1,
                               stream, ma, mw, a);
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_product_wide_kernel");
}

template <int NT, bool Gated>
int enqueue_narrow(const Product &p, const Args &a, int sms, cudaStream_t stream) {
  using C = Narrow<NT, Gated>;
  CUtensorMap ma, mw;
  int rc = encode(&ma, p.a, p.k, p.m, p.a_stride, 0, 0, NT);
  if (!rc) rc = encode(&mw, p.w, p.k, Gated ? 2 * p.n : p.n, p.w_stride, p.groups, p.w_batch, kNarrowM);
  if (!rc) rc = allow_smem<&reshard_product_narrow_kernel<NT, Gated>>(C::kSmem);
  if (rc) return rc;
  const int64_t tiles = (p.m / NT + std::min<int64_t>(p.groups, p.m)) * ((p.n + kNarrowM - 1) / kNarrowM);
  // K is split while the tiles leave half of the GPU's places (two an SM) empty and a share keeps four blocks
  int split = 1;
  while (split < 8 && tiles * split * 2 <= 2 * sms && a.kblocks >= split * 8) split *= 2;
  if (tiles * split > INT32_MAX) return fail(RESHARD_ERR_UNSUPPORTED, "too many tiles for one launch");
  const cudaError_t e = launch(reshard_product_narrow_kernel<NT, Gated>, dim3((unsigned)(tiles * split)), kNarrowThreads, C::kSmem, split,
                               stream, ma, mw, a, split);
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_product_narrow_kernel");
}

template <bool Gated>
int enqueue_by_rows(const Product &p, const Args &a, cudaStream_t stream) {
  int sms = 0;
  int rc = device_sms(&sms);
  if (rc) return rc;
  const int64_t per = (p.m + p.groups - 1) / p.groups;     // rows a group, on average
  if (per <= 16) return enqueue_narrow<16, Gated>(p, a, sms, stream);
  if (per <= 32) return enqueue_narrow<32, Gated>(p, a, sms, stream);
  if (per <= 64) return enqueue_narrow<64, Gated>(p, a, sms, stream);
  return enqueue_wide<Gated>(p, a, sms, stream);
}

}  // namespace

int enqueue_product(const Product &p, cudaStream_t stream) {
  Args a{};
  a.a_scale = p.a_scale;
  a.as_row = p.as_row;
  a.as_block = p.as_block;
  a.w_scale = p.w_scale;
  a.offsets = p.offsets;
  a.groups = p.groups;
  a.m = (int)p.m;
  a.n = (int)p.n;
  a.kblocks = (int)((p.k + kBlockK - 1) / kBlockK);
  a.wblocks = (int)(((p.gated ? 2 * p.n : p.n) + kScaleBlock - 1) / kScaleBlock);
  a.out = p.out;
  a.out_dtype = p.out_dtype;
  a.out_stride = p.out_stride;
  a.out_scale = p.out_scale;
  a.os_row = p.os_row;
  a.os_block = p.os_block;
  return p.gated ? enqueue_by_rows<true>(p, a, stream) : enqueue_by_rows<false>(p, a, stream);
}

}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int reshard_ops_status(int32_t *status, int reset) {
  if (!status) return fail(RESHARD_ERR_INVALID_ARG, "status is NULL");
  OPS_CUDA(cudaDeviceSynchronize());
  int v = 0;
  OPS_CUDA(cudaMemcpyFromSymbol(&v, g_ops_status, sizeof v));
  if (reset && v) {
    const int zero = 0;
    OPS_CUDA(cudaMemcpyToSymbol(g_ops_status, &zero, sizeof zero));
  }
  *status = v;
  return RESHARD_OK;
}
