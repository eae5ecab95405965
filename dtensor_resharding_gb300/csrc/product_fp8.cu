// The matrix product over 8-bit values with block scales, dense or grouped by expert, on the tcgen05 tensor cores:
//
//   out[m, n] = sum_b sa[m, b] sw[n / 128, b] (sum_{k in block b} a[m, k] w[n, k])
//
// The scales differ along K, so the inner sum of each 128-block leaves the tensor cores as fp32 (tensor memory) and is
// scaled and added in registers: out = fma(sa sw, inner, out) per block. Tensor memory holds two such partial tiles, so
// that the tensor cores work on one while the epilogue warps read the other.
//
// Three kernels, by the rows of `a` (their sides of the choice, measured, stand at the rules below):
//  - wide: 128 rows of `a` x 256 rows of `w`, persistent, for many rows a group.
//  - narrow: 128 rows of `w` x 16 .. 64 rows of `a`: the tile's narrow side fits the rows at hand.
//  - few: up to four rows, dense: streams `w` through registers.
// Wide and narrow can end in silu(gate) * up, quantized by rows (the expert layer's first product): a tile then holds the
// 128 columns of one quantization block and their gate and up rows.
//
// Their operands come by TMA (128-byte swizzle, K along the row), rows beyond a tensor as zeros. Rows of a tile beyond its
// group's end belong to the next group: they are computed and not stored.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstddef>
#include <mutex>
#include <type_traits>

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
  const void *x;        // the few kernel's rows: values that it quantizes, or quantized ones
  int64_t x_stride;
  int cols;
  const float *w_scale;
  const int32_t *offsets;
  const int32_t *order; // NULL: row r of the product is row r of a; otherwise row order[r] / per_row
  int per_row, a_rows;
  int groups, m, n, kblocks;
  int wblocks;          // blocks of w's rows in one group's scales
  void *out;
  int out_dtype;
  int64_t out_stride;
  bool boxed;           // out has a tensor map
  float *out_scale;
  int64_t os_row, os_block;
};

// Offsets come from the device: kept within the rows the tensors have.
__device__ __forceinline__ int row_offset(const Args &p, int g) {
  return p.offsets ? min(max(p.offsets[g], 0), p.m) : g ? p.m : 0;
}

// The row of a (and of its scales) that the product's row r is. Places come from the device, too.
__device__ __forceinline__ int source_row(const Args &p, int r) {
  return p.order ? min(max(p.order[r], 0) / p.per_row, p.a_rows - 1) : r;
}

// The fast exponential and division: their error (some ulp, and 1.2 |g| ulp of the exponential for negative g) is far below
// the step of the 8-bit code that the product becomes. With expf and a rounded division the layer of 8,192 tokens takes 75 us more
// and is as far from 64 bits (0.0129 of the norm).
__device__ __forceinline__ float silu_times(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// Offsets that descend are raised to the largest before them, so that no row is of two groups and the tiles are as many as
// the host counted at most. One warp.
__device__ __forceinline__ void ascending(int *off, int groups, int lane) {
  int most = 0;
  for (int g0 = 0; g0 <= groups; g0 += 32) {
    int v = g0 + lane <= groups ? off[g0 + lane] : 0;
    for (int o = 1; o < 32; o <<= 1) v = max(v, __shfl_up_sync(kFull, v, o));
    v = max(v, most);
    if (g0 + lane <= groups) off[g0 + lane] = v;
    most = __shfl_sync(kFull, v, 31);
  }
  __syncwarp();
}

// tiles[g] = tiles of M rows before group g. One warp.
template <int M>
__device__ __forceinline__ void row_tiles(int *off, int *tiles, int groups, int lane) {
  int base = 0, down = 0;
  for (int g = lane; g < groups; g += 32) down |= off[g + 1] - off[g];
  if (__any_sync(kFull, down < 0)) ascending(off, groups, lane);
  for (int g0 = 0; g0 < groups; g0 += 32) {
    const int g = g0 + lane;
    const int own = g < groups ? (off[g + 1] - off[g] + M - 1) / M : 0;
    int sum = own;
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, sum, o);
      if (lane >= o) sum += x;
    }
    if (g < groups) tiles[g] = base + sum - own;
    base += __shfl_sync(kFull, sum, 31);
  }
  if (lane == 0) tiles[groups] = base;
}

// The last group whose first tile is at most t, by a whole warp: two looks at 32 groups each. (Halving 128 groups took a
// loader some 1,000 cycles a tile, in which its stages ran dry.)
static_assert(RESHARD_MAX_GROUPS <= 32 * 32, "two looks");
__device__ __forceinline__ int group_of(const int *tiles, int groups, uint32_t ntiles, uint32_t t, int lane) {
  auto at_most = [&](int g) { return 31 - __clz(__ballot_sync(kFull, g < groups && tiles[min(g, groups)] * ntiles <= t)); };
  const int lo = groups > 32 ? 32 * at_most(32 * lane) : 0;
  return lo + at_most(lo + lane);
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

// A CTA an SM walks over tiles: one warp loads, one issues the products, one fetches the scales, eight take the partial
// tiles out of tensor memory. A thread of those owns one row and 128 columns, so that one scale a block serves all of
// them, and adds pairs of columns with one instruction. A block's products take 512 cycles of the tensor cores and a block
// about 750: a half of tensor memory is handed from the products to the epilogue and back (two barriers each way and the
// completion of the products, 400 cycles with no work in between), and there is room for two only. 8192 x 14336 x 4096
// takes 349 us, 2.8 PFLOP/s, tensor cores 60% busy; a tile's end, 2,000 to 3,400 cycles, weighs more where K is short:
// 65,536 rows of 128 experts, 2048 x 768 without a gate 119 us into bf16, 1.7 PFLOP/s, and 150 into fp32, which the layer takes.
// Measured and not kept: 16 epilogue warps of 64 columns each (4% slower), products of 128 columns that signal the halves
// apart (6% slower), 32 columns a load (the same), w's blocks prefetched into L2 (15% slower), the next block's barrier
// looked at early (1% slower), one reciprocal for two or four gates (the same).
constexpr int kWideM = 128, kWideN = 256;
constexpr int kWideStageBytes = (kWideM + kWideN) * kBlockK;
constexpr int kWideEpi = 8;              // epilogue warps: 4 row quarters x 2 column halves
constexpr int kWideThreads = (kWideEpi + 4) * 32;        // behind a warpgroup: the issuer, the loader, the scales' loader, one idle
constexpr int kWideCols = kWideN / 2;    // columns of a thread
constexpr int kTileSlots = 8;            // tiles whose place the loader has written down: it is 6 blocks ahead at most, see the scales
// Registers a thread: at launch, of the epilogue's two warpgroups and of the other. The epilogue holds 128 sums and two loads
// of 16 columns.
constexpr int kWideRegs = 168, kWideRegsEpi = 200, kWideRegsRest = 104;
static_assert(kWideThreads * kWideRegs >= kWideEpi * 32 * kWideRegsEpi + 128 * kWideRegsRest, "more registers than the launch has");

struct WideTile {
  int g, row, rows, n;     // group, first row, rows of the group from there (can exceed the tile), column tile
};
template <bool Gated>
struct Wide {
  static constexpr int kStages = Gated ? 4 : 3;
  static constexpr int kScaleSlots = 2 * kStages;
  // An epilogue warp's 32 rows on their way out: boxes of so many bytes of each row. The gated product's, 64 bytes, leave
  // room for a fourth stage (65,536 x 768 x 2048: 212 us with three). Without a gate a fourth stage would leave 64 bytes,
  // too, of 256: 8192 x 14336 x 4096 2% faster, 65,536 x 2048 x 768 6% slower.
  static constexpr int kBox = Gated ? 64 : 128, kBoxes = Gated ? 1 : 2;
  struct Shared {
    alignas(16) uint64_t done[2];        // 16-byte pairs: the address of the other is this one's ^ 8
    alignas(16) uint64_t taken[2];
    uint64_t full[kStages], empty[kStages], paired[2], last;
    uint32_t tmem;
    int stop;
    uint32_t amax[2][2][kWideM];
    alignas(16) WideTile tile[kTileSlots];
    float a_scale[kScaleSlots][kWideM], w_scale[kScaleSlots][2];     // w: the column halves', or gate's and up's
    int off[RESHARD_MAX_GROUPS + 1], tiles[RESHARD_MAX_GROUPS + 1];   // row offsets; tiles of rows before each group
  };
  static constexpr size_t kOut = (size_t)kWideEpi * kBoxes * 32 * kBox;
  static constexpr size_t kSmem = (size_t)kStages * kWideStageBytes + kOut + sizeof(Shared);
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

__device__ __forceinline__ WideTile wide_tile(const int *off, const int *tiles, int groups, uint32_t ntiles, uint32_t t, int lane) {
  const int lo = group_of(tiles, groups, ntiles, t, lane);
  const uint32_t here = tiles[lo + 1] - tiles[lo], l = t - tiles[lo] * ntiles;
  const uint32_t n = l / here, m = l - n * here;     // row tiles first: neighbours share w's tile
  WideTile r;
  r.g = lo;
  r.row = off[lo] + m * kWideM;
  r.rows = off[lo + 1] - r.row;
  r.n = n;
  return r;
}

// An epilogue warp's 32 rows on their way to global memory: Boxes boxes of Bytes (128 or 64) of each row, in shared memory
// as a tensor map of that box and swizzle has them (16-byte pieces spread over the banks by row). A lane writes its own
// row's pieces; box_out() hands the boxes to the copy engine where all 32 rows are the group's, or else writes those that
// are. The products go on meanwhile: all CTAs finish their tiles together, and 10 MB of a round's tiles reach L2 no
// faster than it takes them (plain stores from the registers kept the epilogue 4,800 cycles a tile, a bulk copy for each
// row 3,800).
template <int Bytes>
__device__ __forceinline__ void box_put(uint8_t *box, int lane, int piece, uint4 v) {
  const int at = Bytes == 128 ? piece ^ (lane & 7) : piece ^ (lane >> 1 & 3);
  *reinterpret_cast<uint4 *>(box + lane * Bytes + at * 16) = v;
}
template <int Bytes, int Boxes>
__device__ __forceinline__ void box_out(const CUtensorMap *map, const uint8_t *box, int lane, uint8_t *out, int64_t pitch, int64_t x, int64_t row, int rows, int bytes) {
  copy_fence();
  __syncwarp();
  if (rows >= 32) {
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < Boxes; ++i)
        if (i * Bytes < bytes) tma_store_2d(map, smem_addr(box + i * 32 * Bytes), (int)x + i * Bytes, (int)row);
      bulk_commit();
    }
  } else {                       // a group's last rows
#pragma unroll 1
    for (int i = lane; i < rows * (Boxes * Bytes / 16); i += 32) {
      const int r = i / (Boxes * Bytes / 16), c = i % (Boxes * Bytes / 16), b = c / (Bytes / 16), piece = c % (Bytes / 16);
      const int at = Bytes == 128 ? piece ^ (r & 7) : piece ^ (r >> 1 & 3);
      const uint4 v = *reinterpret_cast<const uint4 *>(box + b * 32 * Bytes + r * Bytes + at * 16);
      uint8_t *to = out + (row + r) * pitch + x + c * 16;
      if (c * 16 + 16 <= bytes) {
        *reinterpret_cast<uint4 *>(to) = v;
      } else {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int e = 0; e < (bytes - c * 16) / 2; ++e) reinterpret_cast<uint16_t *>(to)[e] = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
      }
    }
    __syncwarp();
  }
}
// The boxes are free again (their last copy has been read).
__device__ __forceinline__ void box_free(int lane) {
  if (lane == 0) bulk_read();
  __syncwarp();
}

// A warp's 32 rows of 128 columns in T. boxed: out's rows start on 16 bytes (a tensor map describes it); otherwise the warp
// writes a row at a time from the boxes, an element a lane (rows from the registers, one a lane, took three times as long).
template <typename T, int Bytes, int Boxes>
__device__ __forceinline__ void store_tile(const CUtensorMap *map, bool boxed, uint8_t *box, int lane, const float2 (&sum)[kWideCols / 2], void *out, int64_t stride,
                                           int64_t n0, int64_t row, int rows, int cols) {
  constexpr int per = Boxes * Bytes / sizeof(T), piece = 16 / sizeof(T), pieces = Bytes / 16;       // columns of the boxes, of 16 bytes; those of a row of a box
#pragma unroll
  for (int c = 0; c < kWideCols; c += per) {
    if (c >= cols) break;
    box_free(lane);
#pragma unroll
    for (int j = 0; j < Boxes * pieces; ++j) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(i & 1 ? sum[(c + 4 * j + i) / 2].y : sum[(c + 4 * j + i) / 2].x);
        else v[i] = pack2<T>(sum[c / 2 + 4 * j + i].x, sum[c / 2 + 4 * j + i].y);
      }
      box_put<Bytes>(box + j / pieces * 32 * Bytes, lane, j % pieces, make_uint4(v[0], v[1], v[2], v[3]));
    }
    if (boxed) {
      box_out<Bytes, Boxes>(map, box, lane, static_cast<uint8_t *>(out), stride * (int64_t)sizeof(T), (n0 + c) * (int64_t)sizeof(T), row, rows,
                      min(per, cols - c) * (int)sizeof(T));
    } else {
      __syncwarp();
      T *to = static_cast<T *>(out) + row * stride + n0 + c;
#pragma unroll 2
      for (int r = 0; r < min(rows, 32); ++r, to += stride) {
#pragma unroll
        for (int u = 0; u < per / 32; ++u) {
          const int e = u * 32 + lane, at = e / (pieces * piece) * 32 * Bytes + r * Bytes + ((e / piece % pieces) ^ (Bytes == 128 ? r & 7 : r >> 1 & 3)) * 16;
          if (c + e < cols) to[e] = reinterpret_cast<const T *>(box + at)[e % piece];
        }
      }
    }
  }
}

template <bool Gated>
__global__ void __launch_bounds__(kWideThreads, 1)
    reshard_product_wide_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mo,
                                const __grid_constant__ Args p) {
  extern __shared__ __align__(1024) uint8_t stages[];
  using C = Wide<Gated>;
  using Shared = typename C::Shared;
  constexpr int kStages = C::kStages;
  uint8_t *const out_boxes = stages + (size_t)kStages * kWideStageBytes;
  Shared &s = *reinterpret_cast<Shared *>(out_boxes + C::kOut);
  if (smem_addr(stages) & 1023) {      // not seen: the swizzle needs it
    atomicOr(&g_ops_status, 1);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Stop stop{&s.stop, &g_ops_status};
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      bar_init(smem_addr(&s.full[i]), 33);       // the loader, and a lane's copies of scales each
      bar_init(smem_addr(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(smem_addr(&s.done[i]), 1);
      bar_init(smem_addr(&s.taken[i]), kWideEpi);
      bar_init(smem_addr(&s.paired[i]), kWideEpi);
    }
    bar_init(smem_addr(&s.last), 1);
    s.stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(smem_addr(&s.tmem), 512);
  grid_enter();
  for (int g = tid; g <= p.groups; g += kWideThreads) s.off[g] = row_offset(p, g);
  __syncthreads();
  if (warp == 4) row_tiles<kWideM>(s.off, s.tiles, p.groups, lane);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = s.tmem;
  constexpr int kCols = Gated ? kWideN / 2 : kWideN;      // output columns of a tile
  const int ntiles = (p.n + kCols - 1) / kCols;
  const uint32_t total = (uint32_t)s.tiles[p.groups] * ntiles;     // below 2^31: the caller's check

  if (warp < 4) {
    registers_down<kWideRegsRest>();
    if (warp == 1) {
      // ---- loader
      uint32_t it = 0, st = 0, phase = 1, tile_no = 0;
      bool ok = true;
      for (uint32_t t = blockIdx.x; ok && t < total; t += gridDim.x, ++tile_no) {
        const WideTile w = wide_tile(s.off, s.tiles, p.groups, ntiles, t, lane);
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const uint32_t bar = smem_addr(s.full) + st * 8;
          ok = bar_wait(smem_addr(s.empty) + st * 8, phase, stop);
          if (__any_sync(kFull, !ok)) {
            ok = false;
            break;
          }
          const uint32_t to = smem_addr(stages) + st * kWideStageBytes;
          if (lane == 0) {
            if (kb == 0) s.tile[tile_no % kTileSlots] = w;      // for the epilogue, by way of this barrier
            bar_expect(bar, kWideStageBytes);
            tma_2d(to, &ma, kb * kBlockK, w.row, bar);
            const uint32_t tw = to + kWideM * kBlockK;
            if (Gated) {                 // of each half's columns the first 64 are gate, the others up
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
          if (++st == kStages) st = 0, phase ^= 1;
        }
      }
      if (!ok && lane == 0)            // stopped: what is on its way still lands in this CTA's memory
        for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
          bar_drain(smem_addr(&s.full[i % kStages]), i / kStages & 1);
      __syncwarp();
    } else if (warp == 0) {
      // ---- issuer: the first warp, which the scheduler prefers
      // The loop is kept to a few dependent steps: they, not the products, are what a block would wait for.
      if (elect_one()) {
        const uint32_t idesc = instruction(kWideN), full = smem_addr(s.full), empty = smem_addr(s.empty);
        const uint64_t a0 = operand(smem_addr(stages));
        uint32_t st = 0, phase = 0, d = tmem, done = smem_addr(s.done), taken = smem_addr(s.taken), free_phase = 1, second = 0;
        const uint32_t mine = blockIdx.x < total ? (total - 1 - blockIdx.x) / gridDim.x + 1 : 0;
        bool ok = true;
        for (uint32_t n = mine * p.kblocks; n; --n) {
          if (!(ok = bar_wait(full + st * 8, phase, stop))) break;
          if (!(ok = bar_wait(taken, free_phase, stop))) break;
          tc_after_sync();
          const uint64_t a = a0 + st * (kWideStageBytes / 16), b = a + kWideM * kBlockK / 16;
#pragma unroll
          for (int k = 0; k < kBlockK / 32; ++k) mma_e4m3(d, a + 2 * k, b + 2 * k, idesc, k > 0);
          mma_commit(done);
          mma_commit(empty + st * 8);
          if (++st == kStages) st = 0, phase ^= 1;
          free_phase ^= second;
          second ^= 1;
          d ^= kWideN;
          done ^= 8;
          taken ^= 8;
        }
        if (!ok) {
          mma_commit(smem_addr(&s.last));
          bar_drain(smem_addr(&s.last), 0);
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // ---- scales of a stage's block, arriving with its operands. Two slots a stage: when a stage is free for block i,
      // the products of block i - kStages are done, which began after the epilogue had taken the block two before that one, so
      // the slot is free too.
      uint32_t st = 0, phase = 1, slot = 0;
      bool ok = true;
      for (uint32_t t = blockIdx.x; ok && t < total; t += gridDim.x) {
        const WideTile w = wide_tile(s.off, s.tiles, p.groups, ntiles, t, lane);
        const float *sa[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) sa[i] = p.a_scale + (int64_t)(w.row + min(lane + 32 * i, w.rows - 1)) * p.as_row;
        // lanes 0 and 1: gated, gate and up of the tile's one block; otherwise the two halves' blocks
        const int wb = Gated ? w.n + (lane & 1) * (p.n / kScaleBlock) : min(w.n * 2 + (lane & 1), p.wblocks - 1);
        const float *sw = p.w_scale + ((int64_t)w.g * p.wblocks + wb) * p.kblocks;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          ok = bar_wait(smem_addr(s.empty) + st * 8, phase, stop);
          if (__any_sync(kFull, !ok)) {
            ok = false;
            break;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            copy4(smem_addr(&s.a_scale[slot][lane + 32 * i]), sa[i]);
            sa[i] += p.as_block;
          }
          if (lane < 2) copy4(smem_addr(&s.w_scale[slot][lane]), sw + kb);
          bar_arrive_copied(smem_addr(s.full) + st * 8);
          if (++st == kStages) st = 0, phase ^= 1;
          if (++slot == C::kScaleSlots) slot = 0;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
    }
  } else {
    // ---- epilogue: a row and half of the columns a thread
    registers_up<kWideRegsEpi>();
    const int side = (warp >> 2) - 1, r = (warp & 3) * 32 + lane;
    uint8_t *const box = out_boxes + (warp - 4) * C::kBoxes * 32 * C::kBox;
    // the next block's: tensor memory, barrier, parity, scales. tries: 1 once a wait gave up, so that the others pass
    uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + side * kWideCols, done = smem_addr(s.done), phase = 0, second = 0;
    uint32_t sa = smem_addr(&s.a_scale[0][r]), sw = smem_addr(&s.w_scale[0][Gated ? 0 : side]), tries = kTries;
    const uint32_t sa_end = sa + sizeof s.a_scale;
    constexpr uint32_t kToTaken = offsetof(Shared, taken) - offsetof(Shared, done);
    for (uint32_t t = blockIdx.x, tile_no = 0; t < total; t += gridDim.x, ++tile_no) {
      float2 sum[kWideCols / 2];       // pairs of columns
#pragma unroll
      for (int i = 0; i < kWideCols / 2; ++i) sum[i] = make_float2(0.0f, 0.0f);
      uint32_t v[2][16];
      float s0, s1;
      // The first columns of a block are asked for as soon as its products are done, before the last sums of the block
      // before, and its scales with them (they came with its operands): the sums hide both.
      auto begin = [&]() {
        if (!bar_spin(done, phase, tries)) tries = 1;
        tc_after_sync();
        tmem_load(from, v[0]);
        const float a = shared_f32(sa);
        s0 = a * shared_f32(sw);
        s1 = Gated ? a * shared_f32(sw + 4) : s0;
      };
      auto block = [&](bool more) {
        const float by0 = s0, by1 = s1;
#pragma unroll
        for (int c = 0; c < kWideCols / 16; ++c) {
          tmem_loaded(v[c & 1]);
          if (c < kWideCols / 16 - 1) {
            tmem_load(from + (c + 1) * 16, v[(c + 1) & 1]);
          } else {                     // the partial tile is in registers
            tc_before_sync();
            __syncwarp();
            if (lane == 0) bar_arrive(done + kToTaken);
            from ^= kWideN;
            done ^= 8;
            phase ^= second;
            second ^= 1;
            sa += sizeof s.a_scale[0];
            sw += sizeof s.w_scale[0];
            if (sa == sa_end) sa -= sizeof s.a_scale, sw -= sizeof s.w_scale;
            if (more) begin();
          }
          const float by = c < kWideCols / 32 ? by0 : by1;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            sum[c * 8 + i] = __ffma2_rn(make_float2(__uint_as_float(v[c & 1][2 * i]), __uint_as_float(v[c & 1][2 * i + 1])), make_float2(by, by), sum[c * 8 + i]);
        }
      };
      begin();
#pragma unroll 1
      for (int kb = 1; kb < p.kblocks; ++kb) block(true);
      block(false);
      if (__any_sync(kFull, tries == 1)) break;
      const WideTile w = s.tile[tile_no % kTileSlots];
      const int64_t row0 = w.row + (warp & 3) * 32;      // the warp's rows
      const int rows = w.rows - (warp & 3) * 32;
      if (!Gated) {
        const int n0 = w.n * kCols + side * kWideCols, cols = min(kWideCols, p.n - n0);
        if (rows > 0 && cols > 0) {
          if (p.out_dtype == RESHARD_BF16) store_tile<__nv_bfloat16, C::kBox, C::kBoxes>(&mo, p.boxed, box, lane, sum, p.out, p.out_stride, n0, row0, rows, cols);
          else if (p.out_dtype == RESHARD_F16) store_tile<__half, C::kBox, C::kBoxes>(&mo, p.boxed, box, lane, sum, p.out, p.out_stride, n0, row0, rows, cols);
          else store_tile<float, C::kBox, C::kBoxes>(&mo, p.boxed, box, lane, sum, p.out, p.out_stride, n0, row0, rows, cols);
        }
      } else {
        // of the sums the first half is gate, the second up: this thread's 64 of the row's 128 values
        constexpr int kHalf = kWideCols / 4;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          sum[i] = make_float2(silu_times(sum[i].x, sum[kHalf + i].x), silu_times(sum[i].y, sum[kHalf + i].y));
          m = max(m, max(magnitude(sum[i].x), magnitude(sum[i].y)));
        }
        s.amax[tile_no & 1][side][r] = m;
        __syncwarp();
        const uint32_t paired = smem_addr(&s.paired[tile_no & 1]);
        if (lane == 0) bar_arrive(paired);
        if (!bar_spin(paired, tile_no >> 1 & 1, tries)) tries = 1;
        if (__any_sync(kFull, tries == 1)) break;
        m = max(m, s.amax[tile_no & 1][side ^ 1][r]);
        float scale, inv;
        block_scale(m, scale, inv);
        if (side == 0 && lane < rows) p.out_scale[(row0 + lane) * p.os_row + w.n * p.os_block] = scale;
        if (rows > 0) {
          box_free(lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = sum[8 * j + 2 * i], y = sum[8 * j + 2 * i + 1];
              q[i] = e4m3x4(x.x * inv, x.y * inv, y.x * inv, y.y * inv);
            }
            box_put<64>(box, lane, j, make_uint4(q[0], q[1], q[2], q[3]));
          }
          box_out<64, 1>(&mo, box, lane, static_cast<uint8_t *>(p.out), p.out_stride, w.n * kCols + side * 64, row0, rows, 64);
        }
      }
    }
    if (tries == 1) {
      s.stop = 1;
      atomicOr(&g_ops_status, 1);
    }
    bulk_done();
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp == 0) tmem_free(tmem, 512);
}

// -------------------------------------------------------------------------------------------------------- narrow --

// Few rows a group: bound by the read of the weights, so that what counts is how much of them is on the way at any time:
// two CTAs an SM with some 100 KB of stages each. The weights sit on the tensor cores' 128 rows, and a product is as wide as
// the rows at hand, to 16. Where the tiles alone do not fill the
// GPU, a cluster of CTAs splits K and adds its partial tiles through distributed shared memory, in rank order: the
// same order on every run. 16 tokens to 8 of 128 experts of 2048 x 768 each: 41 and 24 us, 389 MB, 6.0
// TB/s; 77 x 2867 x 4096 with the rows' quantization before it: 11.2 us, bound by latency (launch, first loads, the
// cluster's sum).
constexpr int kNarrowM = 128;            // rows of w (of gate and of up, when gated)
constexpr int kNarrowThreads = 192;      // 4 epilogue warps, the loader, the issuer
constexpr int kMostSplit = 8;            // CTAs of a cluster that share a tile's K
constexpr int kNarrowPerSm = 2;          // CTAs an SM

template <int NT, bool Gated>
struct Narrow {
  static constexpr int kParts = Gated ? 2 : 1;
  static constexpr int kStageBytes = (kParts * kNarrowM + NT) * kBlockK;
  static_assert(NT * kParts <= 64, "sums in the registers of a thread");
  static constexpr int kStages = 107520 / kStageBytes;
  static constexpr int kPartial = NT * kNarrowM * 4 * kParts;   // a CTA's sums, in stage memory, for the cluster
  static constexpr int kColumns = 2 * NT * kParts < 32 ? 32 : 2 * NT * kParts;
  static_assert(kStages >= 2 && kPartial <= kStages * kStageBytes, "stages");
  struct Shared {
    uint64_t full[kStages], empty[kStages], done[2], taken[2], paired[2], last;
    uint32_t tmem;
    int stop;
    alignas(16) float scale[4][2][kParts][NT];       // per epilogue warp, two blocks
    uint32_t amax[2][4][NT];
    int off[RESHARD_MAX_GROUPS + 1], tiles[RESHARD_MAX_GROUPS + 1];   // row offsets; tiles of rows before each group
  };
  static constexpr size_t kSmem = (size_t)kStages * kStageBytes + sizeof(Shared);
  static_assert(kSmem <= 115712, "shared memory of a CTA");
};

struct NarrowTile {
  int g, row, rows, n;     // group, first row, rows, column tile
};
template <int NT>
__device__ __forceinline__ NarrowTile narrow_tile(const int *off, const int *tiles, int groups, uint32_t ntiles, uint32_t t, int lane) {
  const int lo = group_of(tiles, groups, ntiles, t, lane);
  const uint32_t l = t - tiles[lo] * ntiles, m = l / ntiles;      // column tiles first: w is read in order
  NarrowTile r;
  r.g = lo;
  r.row = off[lo] + m * NT;
  r.rows = min(NT, off[lo + 1] - r.row);
  r.n = l - m * ntiles;
  return r;
}

// early: the kernel before this one on the stream wrote neither weights nor offsets nor order, and had itself waited for
// what did: their reads need not wait for its end, and the first weights are on their way while it runs.
template <int NT, bool Gated>
__global__ void __launch_bounds__(kNarrowThreads, kNarrowPerSm)
    reshard_product_narrow_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mw, const __grid_constant__ Args p,
                                  const int split, const bool early) {
  using C = Narrow<NT, Gated>;
  using Shared = typename C::Shared;
  constexpr int kStages = C::kStages, kParts = C::kParts;
  extern __shared__ __align__(1024) uint8_t stages[];
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
      bar_init(smem_addr(&s.paired[i]), 4);
    }
    bar_init(smem_addr(&s.last), 1);
    s.stop = smem_addr(stages) & 1023;       // 0: the swizzle needs it
    if (s.stop) atomicOr(&g_ops_status, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 5) tmem_alloc(smem_addr(&s.tmem), C::kColumns);
  if (!early) grid_wait();
  grid_release();
  for (int g = tid; g <= p.groups; g += kNarrowThreads) s.off[g] = row_offset(p, g);
  __syncthreads();
  if (warp == 0) row_tiles<NT>(s.off, s.tiles, p.groups, lane);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = s.tmem;
  const uint32_t ntiles = (p.n + kNarrowM - 1) / kNarrowM;
  const int rank = (int)(blockIdx.x % split);       // consecutive CTAs are a cluster
  const uint32_t first = blockIdx.x / split, step = gridDim.x / split;      // with a split, every cluster has one tile at most
  const uint32_t total = s.stop ? 0 : (uint32_t)s.tiles[p.groups] * ntiles;
  const int kb0 = (int)((int64_t)p.kblocks * rank / split), kb1 = (int)((int64_t)p.kblocks * (rank + 1) / split);
  float acc[kParts][NT];
  bool ok = true;
  auto tile = [&](uint32_t t) { return narrow_tile<NT>(s.off, s.tiles, p.groups, ntiles, t, lane); };

  if (warp == 4) {
    // ---- loader: one lane; where rows are gathered, four rows a lane
    auto weights = [&](const NarrowTile &w, int kb, uint32_t st) {
      const uint32_t to = smem_addr(stages) + st * C::kStageBytes, bar = smem_addr(s.full) + st * 8;
      bar_expect(bar, C::kStageBytes);
#pragma unroll
      for (int q = 0; q < kParts; ++q) tma_3d(to + q * kNarrowM * kBlockK, &mw, kb * kBlockK, q * p.n + w.n * kNarrowM, w.g, bar);
    };
    uint32_t sent = 0;                 // stages whose weights are on their way
    if (early) {
      for (uint32_t t = first; t < total && sent < kStages; t += step) {
        const NarrowTile w = tile(t);
        for (int kb = kb0; kb < kb1 && sent < kStages; ++kb, ++sent)
          if (lane == 0) weights(w, kb, sent);
      }
      grid_wait();
    }
    uint32_t it = 0, st = 0, phase = 1;
    for (uint32_t t = first; ok && t < total; t += step) {
      const NarrowTile w = tile(t);
      int row[4];
      if (p.order) {
#pragma unroll
        for (int i = 0; i < 4; ++i) row[i] = source_row(p, w.row + min(4 * lane + i, w.rows - 1));
      }
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        if (it >= sent) {
          ok = bar_wait(smem_addr(s.empty) + st * 8, phase, stop);
          if (__any_sync(kFull, !ok)) {
            ok = false;
            break;
          }
          if (lane == 0) weights(w, kb, st);
          __syncwarp();
        }
        const uint32_t to = smem_addr(stages) + st * C::kStageBytes + kParts * kNarrowM * kBlockK, bar = smem_addr(s.full) + st * 8;
        if (p.order) {
          if (lane < NT / 4) tma_rows4(to + lane * 4 * kBlockK, &ma, kb * kBlockK, row, bar);
        } else if (lane == 0) {
          tma_2d(to, &ma, kb * kBlockK, w.row, bar);
        }
        if (++st == kStages) st = 0, phase ^= 1;
      }
    }
    if (!ok && lane == 0)            // stopped: what is on its way still lands in this CTA's memory
      for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i) bar_drain(smem_addr(&s.full[i % kStages]), i / kStages & 1);
    __syncwarp();
  } else if (warp == 5) {
    // ---- issuer
    uint32_t st = 0, phase = 0, half = 0, free_phase = 1;
    const uint64_t a0 = operand(smem_addr(stages));
    const bool one = elect_one();      // the warp's other lanes help to find the tiles, and wait for nothing
    for (uint32_t t = first; t < total; t += step) {
      const uint32_t idesc = instruction((tile(t).rows + 15) & ~15);
      if (one) {
        for (int kb = kb0; ok && kb < kb1; ++kb) {
          if (!(ok = bar_wait(smem_addr(s.full) + st * 8, phase, stop))) break;
          if (!(ok = bar_wait(smem_addr(s.taken) + half * 8, free_phase, stop))) break;
          tc_after_sync();
          const uint64_t a = a0 + st * (C::kStageBytes / 16), b = a + kParts * kNarrowM * kBlockK / 16;
#pragma unroll
          for (int q = 0; q < kParts; ++q)
#pragma unroll
            for (int k = 0; k < kBlockK / 32; ++k)
              mma_e4m3(tmem + (half * kParts + q) * NT, a + q * kNarrowM * kBlockK / 16 + 2 * k, b + 2 * k, idesc, k > 0);
          mma_commit(smem_addr(s.empty) + st * 8);
          mma_commit(smem_addr(s.done) + half * 8);
          if (++st == kStages) st = 0, phase ^= 1;
          free_phase ^= half;
          half ^= 1;
        }
      }
    }
    if (!ok) {
      mma_commit(smem_addr(&s.last));
      bar_drain(smem_addr(&s.last), 0);
    }
    __syncwarp();
  } else {
    // ---- epilogue: one row of w a thread; the scales of the tile's rows of a are shared out by the warp
    if (early) grid_wait();
    constexpr int kPer = (NT + 31) / 32;
    const uint32_t from = tmem + ((uint32_t)(warp * 32) << 16);
    uint32_t half = 0, phase = 0, tile_no = 0;
    auto store = [&](const NarrowTile &w, int c, float v) {
      const int n = w.n * kNarrowM + tid;
      if (n >= p.n) return;
      const int64_t at = (int64_t)(w.row + c) * p.out_stride + n;
      if (p.out_dtype == RESHARD_F32) static_cast<float *>(p.out)[at] = v;
      else static_cast<uint16_t *>(p.out)[at] = p.out_dtype == RESHARD_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
    };
    auto store_gated = [&](const NarrowTile &w, int c, float h, uint32_t amax) {
      float scale, inv;
      block_scale(amax, scale, inv);
      if (tid == 0) p.out_scale[(int64_t)(w.row + c) * p.os_row + (int64_t)w.n * p.os_block] = scale;
      static_cast<uint8_t *>(p.out)[(int64_t)(w.row + c) * p.out_stride + w.n * kNarrowM + tid] = (uint8_t)e4m3x2(h * inv, 0.0f);
    };
    for (uint32_t t = first; t < total; t += step, ++tile_no) {
      const NarrowTile w = tile(t);
      const int wide = (w.rows + 15) & ~15;               // columns the products compute
      const float *sw[kParts], *sa[kPer];
#pragma unroll
      for (int q = 0; q < kParts; ++q)
        sw[q] = p.w_scale + ((int64_t)w.g * p.wblocks + q * (p.n / kScaleBlock) + w.n) * p.kblocks;
#pragma unroll
      for (int i = 0; i < kPer; ++i) sa[i] = p.a_scale + (int64_t)source_row(p, w.row + min(lane + 32 * i, w.rows - 1)) * p.as_row;
#pragma unroll
      for (int q = 0; q < kParts; ++q)
#pragma unroll
        for (int c = 0; c < NT; ++c) acc[q][c] = 0.0f;
      float a0[kPer], a1[kPer], w0[kParts], w1[kParts];
      auto fetch = [&](int kb, float (&a)[kPer], float (&b)[kParts]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) a[i] = kb < kb1 ? sa[i][(int64_t)kb * p.as_block] : 0.0f;
#pragma unroll
        for (int q = 0; q < kParts; ++q) b[q] = kb < kb1 ? sw[q][kb] : 0.0f;
      };
      fetch(kb0, a0, w0);
      fetch(kb0 + 1, a1, w1);
      for (int kb = kb0; kb < kb1; ++kb) {
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
        ok = ok && bar_wait(smem_addr(s.done) + half * 8, phase, stop);
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
              tmem_load(from + (half * kParts + q) * NT + c, v);
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
        if (lane == 0) bar_arrive(smem_addr(s.taken) + half * 8);
        phase ^= half;
        half ^= 1;
      }
      if (!ok) break;
      if (split > 1) continue;
      if (!Gated) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < w.rows) store(w, c, acc[0][c]);
      } else {
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          if (c < w.rows) {
            acc[0][c] = silu_times(acc[0][c], acc[kParts - 1][c]);
            const uint32_t m = __reduce_max_sync(kFull, magnitude(acc[0][c]));
            if (lane == 0) s.amax[tile_no & 1][warp][c] = m;
          }
        }
        __syncwarp();
        const uint32_t paired = smem_addr(&s.paired[tile_no & 1]);
        if (lane == 0) bar_arrive(paired);
        ok = bar_wait(paired, tile_no >> 1 & 1, stop);
        if (__any_sync(kFull, !ok)) {
          ok = false;
          break;
        }
        const uint32_t(&am)[4][NT] = s.amax[tile_no & 1];
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < w.rows) store_gated(w, c, acc[0][c], max(max(am[0][c], am[1][c]), max(am[2][c], am[3][c])));
      }
    }
    if (split > 1) {
      // The CTA's products are done (its epilogue saw the last one), so its stages hold the sums from here; each rank then
      // adds every split-th row of a, over the ranks in order.
      float *part = reinterpret_cast<float *>(stages);
      const NarrowTile w = first < total ? tile(first) : NarrowTile{0, 0, 0, 0};
#pragma unroll
      for (int q = 0; q < kParts; ++q)
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c < w.rows) part[(q * NT + c) * kNarrowM + tid] = acc[q][c];
      cluster_sync();
      // a loop, not unrolled: code that runs once is fetched for as long as it runs
#pragma unroll 1
      for (int c = rank; c < w.rows; c += split) {
        float x[kParts][kMostSplit], sum[kParts];
#pragma unroll
        for (int r = 0; r < kMostSplit; ++r)
#pragma unroll
          for (int q = 0; q < kParts; ++q) x[q][r] = r < split ? cluster_f32(smem_addr(&part[(q * NT + c) * kNarrowM + tid]), r) : 0.0f;
#pragma unroll
        for (int q = 0; q < kParts; ++q) {
          sum[q] = x[q][0];
#pragma unroll
          for (int r = 1; r < kMostSplit; ++r) sum[q] += x[q][r];
        }
        if (!Gated) {
          if (ok) store(w, c, sum[0]);
        } else {
          const float h = silu_times(sum[0], sum[kParts - 1]);
          const uint32_t m = __reduce_max_sync(kFull, magnitude(h));
          if (lane == 0) s.amax[0][warp][c] = m;
          asm volatile("bar.sync 1, 128;" ::: "memory");       // the four warps, each once a row
          if (ok) store_gated(w, c, h, max(max(s.amax[0][0][c], s.amax[0][1][c]), max(s.amax[0][2][c], s.amax[0][3][c])));
        }
      }
      cluster_sync();
    }
  }
  if (split > 1 && warp >= 4) {        // the cluster's barriers count every thread
    cluster_sync();
    cluster_sync();
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp == 5) tmem_free(tmem, C::kColumns);
}

// ----------------------------------------------------------------------------------------------------------- few --

constexpr int kFewRows = 8;              // columns of one warp-wide product: rows of a
constexpr int kFewMost = 4;              // rows that are worth it: every CTA quantizes them (8 rows, 4096 x 4096: 11.9 us, narrow 7.5)
constexpr int kFewN = 16;                // rows of w a CTA
constexpr int kFewWarps = 8;             // of a CTA: each has a share of K
constexpr int kFewAhead = 2;             // blocks of w on their way to a warp
constexpr int64_t kFewBytes = 64 << 10;  // of the rows of a, quantized, in shared memory

// A lane's 32 bytes of a row of w.
struct FewBytes {
  uint4 v[2];
  __device__ __forceinline__ void load(const uint8_t *p) {
    v[0] = __ldcs(reinterpret_cast<const uint4 *>(p));
    v[1] = __ldcs(reinterpret_cast<const uint4 *>(p) + 1);
  }
  __device__ __forceinline__ void load_some(const uint8_t *p, int left) {      // a row's end: what follows it is not the row's
    uint64_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll 1
      for (int j = 0; j < 8; ++j)
        if (8 * i + j < left) w[i] |= (uint64_t)p[8 * i + j] << (8 * j);
    v[0] = make_uint4((uint32_t)w[0], (uint32_t)(w[0] >> 32), (uint32_t)w[1], (uint32_t)(w[1] >> 32));
    v[1] = make_uint4((uint32_t)w[2], (uint32_t)(w[2] >> 32), (uint32_t)w[3], (uint32_t)(w[3] >> 32));
  }
};

// 16 bytes of values at p, those from `left` on 0; p may start anywhere.
template <typename X>
__device__ __forceinline__ uint4 load_piece(const X *p, int left) {
  constexpr int per = 16 / sizeof(X);
  uint64_t w[2] = {0, 0};
#pragma unroll 1
  for (int j = 0; j < min(left, per); ++j) {
    uint64_t x;
    if constexpr (sizeof(X) == 1) x = p[j];
    else if constexpr (sizeof(X) == 2) x = reinterpret_cast<const uint16_t *>(p)[j];
    else x = reinterpret_cast<const uint32_t *>(p)[j];
    const int at = j * 8 * (int)sizeof(X);
    if (at < 64) w[0] |= x << at;
    else w[1] |= x << (at - 64);
  }
  return make_uint4((uint32_t)w[0], (uint32_t)(w[0] >> 32), (uint32_t)w[1], (uint32_t)(w[1] >> 32));
}
template <typename X>
__device__ __forceinline__ void unpack(uint4 v, float *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < (int)(16 / sizeof(X)); ++j) {
    if constexpr (sizeof(X) == 4) x[j] = __uint_as_float(w[j]);
    else if constexpr (std::is_same_v<X, __nv_bfloat16>) x[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    else x[j] = __half2float(__ushort_as_half((uint16_t)(w[j / 2] >> (16 * (j & 1)))));
  }
}

// Few rows of a, dense, and often one: a matrix times a vector, bound by the read of w from HBM and, at the sizes where
// that is short, by what a kernel has to do before its first load. So no tensor memory, barriers or staging of w here:
// each warp streams w from global memory into registers, two blocks ahead, and multiplies on the warp-wide tensor
// instruction (16 x 8 x 32), whose rate is far above what the read leaves to do. Lane (g, t) holds rows g and g + 8 of w
// and row g of a at columns 32 t .. 32 t + 31 of a block: which columns a product takes from a lane is the same for both
// operands, so that a lane's bytes can be neighbours. The CTA quantizes its rows of a into shared memory (X: their type, or
// uint8_t where they come quantized) while the first loads of w are on their way: one launch for the whole call. The K
// shares of a CTA's warps are added in order. 1 x 14336 x 4096: 12.5 us, 4.7 TB/s (quantization and narrow: 14.9); of that the read
// alone would take 8.7, the start and the end the rest. Three blocks ahead spill, one takes 13.8.
template <typename X>
__global__ void __launch_bounds__(kFewWarps * 32, 3) reshard_product_few_kernel(const __grid_constant__ Args p, const uint8_t *wq, int64_t w_stride) {
  constexpr bool kGiven = std::is_same_v<X, uint8_t>;
  grid_enter();
  extern __shared__ __align__(16) uint8_t xq[];      // [row][pitch], then scales [row][block]
  __shared__ float part[kFewWarps][kFewN][kFewRows + 1];
  const int pitch = p.kblocks * kBlockK + 16;
  float *const xs = reinterpret_cast<float *>(xq + p.m * pitch);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const int n0 = blockIdx.x * kFewN;
  const int kb0 = p.kblocks * warp / kFewWarps, kb1 = p.kblocks * (warp + 1) / kFewWarps, whole = min(kb1, p.cols / kBlockK);
  const uint8_t *w0 = wq + (int64_t)min(n0 + g, p.n - 1) * w_stride + 32 * t, *w1 = wq + (int64_t)min(n0 + g + 8, p.n - 1) * w_stride + 32 * t;
  FewBytes b[kFewAhead][2];
#pragma unroll
  for (int u = 0; u < kFewAhead; ++u)
    if (kb0 + u < whole) {
      b[u][0].load(w0 + (kb0 + u) * kBlockK);
      b[u][1].load(w1 + (kb0 + u) * kBlockK);
    }

  // the rows of a: 8 lanes a block, 16 values each; the loads of two blocks a lane group are in flight together
  const bool wide = ((reinterpret_cast<uintptr_t>(p.x) | (uintptr_t)(p.x_stride * (int64_t)sizeof(X))) & 15) == 0;
  const int blocks = p.m * p.kblocks;
  constexpr int kBatch = kGiven || sizeof(X) == 2 ? 2 : 1, kPieces = kGiven ? 1 : (int)sizeof(X), kStep = kFewWarps * 4;
#pragma unroll 1
  for (int i0 = tid >> 3; i0 < (blocks + 3) / 4 * 4; i0 += kBatch * kStep) {      // four blocks a warp, all of it to the shuffles
    uint4 v[kBatch][kPieces];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kStep, r = i / p.kblocks, kb = i - r * p.kblocks, at = kb * kBlockK + (lane & 7) * 16;
      const X *from = static_cast<const X *>(p.x) + (int64_t)r * p.x_stride + at;
      const int left = i < blocks ? p.cols - at : 0;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) v[u][j] = make_uint4(0, 0, 0, 0);
      if (left >= 16 && wide) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) v[u][j] = __ldg(reinterpret_cast<const uint4 *>(from) + j);
      } else if (left > 0) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) v[u][j] = load_piece(from + j * (16 / (int)sizeof(X)), left - j * (16 / (int)sizeof(X)));
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int i = i0 + u * kStep, r = i / p.kblocks, kb = i - r * p.kblocks, at = kb * kBlockK + (lane & 7) * 16;
      if (i - (lane >> 3) >= blocks) break;            // the whole warp
      uint4 q = v[u][0];
      float scale = 0.0f;
      if constexpr (kGiven) {
        if (i < blocks) scale = p.a_scale[(int64_t)r * p.as_row + (int64_t)kb * p.as_block];
      } else {
        constexpr int per = 16 / sizeof(X);
        float x[16];
#pragma unroll
        for (int j = 0; j < kPieces; ++j) unpack<X>(v[u][j], x + j * per);
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, magnitude(x[j]));
#pragma unroll
        for (int o = 4; o; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
        float inv;
        block_scale(m, scale, inv);
        q = make_uint4(e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv), e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv),
                       e4m3x4(x[8] * inv, x[9] * inv, x[10] * inv, x[11] * inv), e4m3x4(x[12] * inv, x[13] * inv, x[14] * inv, x[15] * inv));
      }
      if (i < blocks) {
        *reinterpret_cast<uint4 *>(xq + r * pitch + at) = q;
        if ((lane & 7) == 0) xs[r * p.kblocks + kb] = scale;
      }
    }
  }
  __syncthreads();

  const float *sw = p.w_scale + (int64_t)(n0 / kScaleBlock) * p.kblocks;
  const uint8_t *mine = xq + min(g, p.m - 1) * pitch + 32 * t;
  const float *s0 = xs + min(2 * t, p.m - 1) * p.kblocks, *s1 = xs + min(2 * t + 1, p.m - 1) * p.kblocks;      // this lane's sums are of rows 2 t and 2 t + 1
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto block = [&](const FewBytes (&w)[2], int kb) {
    uint32_t q[8];
    *reinterpret_cast<uint4 *>(q) = *reinterpret_cast<const uint4 *>(mine + kb * kBlockK);
    *reinterpret_cast<uint4 *>(q + 4) = *reinterpret_cast<const uint4 *>(mine + kb * kBlockK + 16);
    const uint32_t u0[8] = {w[0].v[0].x, w[0].v[0].y, w[0].v[0].z, w[0].v[0].w, w[0].v[1].x, w[0].v[1].y, w[0].v[1].z, w[0].v[1].w};
    const uint32_t u1[8] = {w[1].v[0].x, w[1].v[0].y, w[1].v[0].z, w[1].v[0].w, w[1].v[1].x, w[1].v[1].y, w[1].v[1].z, w[1].v[1].w};
    float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; i += 2)
      asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                   : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                   : "r"(u0[i]), "r"(u1[i]), "r"(u0[i + 1]), "r"(u1[i + 1]), "r"(q[i]), "r"(q[i + 1]));
    const float f = sw[kb], f0 = s0[kb] * f, f1 = s1[kb] * f;
    acc[0] = fmaf(d[0], f0, acc[0]);
    acc[1] = fmaf(d[1], f1, acc[1]);
    acc[2] = fmaf(d[2], f0, acc[2]);
    acc[3] = fmaf(d[3], f1, acc[3]);
  };
#pragma unroll 1
  for (int kb = kb0; kb < whole; kb += kFewAhead) {
#pragma unroll
    for (int u = 0; u < kFewAhead; ++u) {
      if (kb + u < whole) {
        block(b[u], kb + u);
        if (kb + u + kFewAhead < whole) {
          b[u][0].load(w0 + (int64_t)(kb + u + kFewAhead) * kBlockK);
          b[u][1].load(w1 + (int64_t)(kb + u + kFewAhead) * kBlockK);
        }
      }
    }
  }
  if (whole < kb1) {                 // K's last block, if it is not whole, is the last warp's
    const int left = p.cols - whole * kBlockK - 32 * t;
    b[0][0].load_some(w0 + (int64_t)whole * kBlockK, left);
    b[0][1].load_some(w1 + (int64_t)whole * kBlockK, left);
    block(b[0], whole);
  }
  part[warp][g][2 * t] = acc[0];
  part[warp][g][2 * t + 1] = acc[1];
  part[warp][g + 8][2 * t] = acc[2];
  part[warp][g + 8][2 * t + 1] = acc[3];
  __syncthreads();
  const int r = tid & 15, m = tid >> 4;
  if (m < p.m && n0 + r < p.n) {
    float v = part[0][r][m];
#pragma unroll
    for (int i = 1; i < kFewWarps; ++i) v += part[i][r][m];
    const int64_t at = (int64_t)m * p.out_stride + n0 + r;
    if (p.out_dtype == RESHARD_F32) static_cast<float *>(p.out)[at] = v;
    else static_cast<uint16_t *>(p.out)[at] = p.out_dtype == RESHARD_BF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
  }
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

// Bytes [batch, rows, cols] in boxes of box_rows x box_cols (128 or 64), swizzled over as many bytes; batch 0: a plain matrix.
int encode(CUtensorMap *map, const void *base, int64_t cols, int64_t rows, int64_t stride, int64_t batch, int64_t batch_stride, int box_rows,
           int box_cols = kBlockK) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = encoder();
  if (!enc) return fail(RESHARD_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)batch};
  const cuuint64_t strides[2] = {(cuuint64_t)stride, (cuuint64_t)batch_stride};
  const cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1}, step[3] = {1, 1, 1};
  const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, batch ? 3 : 2, const_cast<void *>(base), dims, strides, box, step,
                         CU_TENSOR_MAP_INTERLEAVE_NONE, box_cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(RESHARD_ERR_CUDA, "cuTensorMapEncodeTiled failed with " + std::to_string((int)r));
  return RESHARD_OK;
}

template <bool Gated>
int enqueue_wide(const Product &p, Args a, int sms, cudaStream_t stream) {
  CUtensorMap ma, mw, mo{};
  int rc = encode(&ma, p.a, p.k, p.m, p.a_stride, 0, 0, kWideM);
  if (!rc) rc = encode(&mw, p.w, p.k, Gated ? 2 * p.n : p.n, p.w_stride, p.groups, p.w_batch, Gated ? 64 : 128);
  const int64_t es = Gated ? 1 : element_bytes(p.out_dtype), pitch = p.out_stride * es;
  // a box's column is a 32-bit number of bytes: rows of 2^31 and more are written without
  a.boxed = Gated || (((reinterpret_cast<uintptr_t>(p.out) | (uintptr_t)pitch) & 15) == 0 && p.n * es <= INT32_MAX);
  if (!rc && a.boxed) rc = encode(&mo, p.out, p.n * es, p.m, pitch, 0, 0, 32, Wide<Gated>::kBox);
  if (!rc) rc = allow_smem<&reshard_product_wide_kernel<Gated>>(Wide<Gated>::kSmem, kWideRegs);
  if (rc) return rc;
  const int64_t cols = Gated ? kWideN / 2 : kWideN;
  const int64_t most = (p.m / kWideM + std::min<int64_t>(p.groups, p.m)) * ((p.n + cols - 1) / cols);
  if (most > INT32_MAX) return fail(RESHARD_ERR_UNSUPPORTED, "too many tiles for one launch");
  const cudaError_t e = launch(reshard_product_wide_kernel<Gated>, dim3((unsigned)std::min<int64_t>(sms, most)), kWideThreads, Wide<Gated>::kSmem, 1,
                               stream, ma, mw, mo, a);
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_product_wide_kernel");
}

// K is split where the tiles leave places on the GPU empty, as far as each share keeps four blocks.
int narrow_split(int64_t tiles, int64_t places, int kblocks) {
  return (int)std::max<int64_t>(1, std::min<int64_t>({kMostSplit, places / tiles, kblocks / 4}));
}

template <int NT, bool Gated>
int enqueue_narrow(const Product &p, const Args &a, int sms, cudaStream_t stream) {
  using C = Narrow<NT, Gated>;
  CUtensorMap ma, mw;
  int rc = encode(&ma, p.a, p.k, a.a_rows, p.a_stride, 0, 0, p.order ? 1 : NT);
  if (!rc) rc = encode(&mw, p.w, p.k, Gated ? 2 * p.n : p.n, p.w_stride, p.groups, p.w_batch, kNarrowM);
  if (!rc) rc = allow_smem<&reshard_product_narrow_kernel<NT, Gated>>(C::kSmem);
  if (rc) return rc;
  const int64_t tiles = (p.offsets ? p.m / NT + std::min<int64_t>(p.groups, p.m) : (p.m + NT - 1) / NT) * ((p.n + kNarrowM - 1) / kNarrowM);
  if (tiles > INT32_MAX) return fail(RESHARD_ERR_UNSUPPORTED, "too many tiles for one launch");
  const int64_t places = (int64_t)sms * kNarrowPerSm;
  const int split = narrow_split(tiles, places, a.kblocks);
  const unsigned grid = (unsigned)(split > 1 ? tiles * split : std::min(tiles, places));
  const cudaError_t e = launch(reshard_product_narrow_kernel<NT, Gated>, dim3(grid), kNarrowThreads, C::kSmem, split, stream, ma, mw, a, split, p.early);
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_product_narrow_kernel");
}

// Whether a grouped product is narrow's, by the rows a group has on average, as far as the host knows them (m is an
// upper bound). The whole layer, narrow and wide: 128 experts of 2048 x 768, 8 rows each 115 us and 129, 12 rows 119 and 133,
// 20 rows 138 and 138, 32 rows 175 and 144; 16 experts of 4096 x 1536, 12 rows 64 and 80, 20 rows 85 and 82; 32 experts of 1024 x 512, 12
// rows 25 and 26, 32 rows 36 and 30. Their products alone into bf16: 12 rows 41 and 46, 19 and 22, 71 and 72, 40 and 38; 16 rows 41
// and 46, 23 and 22, 76 and 72, 46 and 38. Where ids range over more experts than are here the bound counts the others' slots, too: 16
// of 128 experts of 4096 x 1536, 64 tokens to 8 (4 rows each) take wide's 77 us instead of 63; from 512 tokens on wide is right (84; 91).
bool few_a_group(int64_t m, int groups) { return m <= 12 * (int64_t)groups; }

// Whether a dense product of more than 64 rows is narrow's (in tiles of 64, K split) or wide's. Wide fills the GPU only from
// 152 tiles of 128 x 256 on; below that narrow has more and shorter pieces. Both times are of this form, in ns, as
// measured. With the rows' quantization before them: 256 x 1024 x 4096 narrow 10.9 us, wide 17.6; 300 x 300 x 14336 14.4 and 49.0;
// but 400 x 4096 x 4096 24.8 and 22.2, 128 x 14336 x 1024 12.2 and 10.3.
bool narrow_is_shorter(int64_t m, int64_t n, int kblocks, int sms) {
  const int64_t tiles = (m + 63) / 64 * ((n + kNarrowM - 1) / kNarrowM), places = (int64_t)kNarrowPerSm * sms, split = narrow_split(tiles, places, kblocks);
  const int64_t ctas = tiles * split, rounds = (ctas + places - 1) / places, share = (kblocks + split - 1) / split;
  const int64_t narrow = 7000 + share * rounds * (ctas <= sms ? 550 : 900);
  const int64_t wide_tiles = (m + kWideM - 1) / kWideM * ((n + kWideN - 1) / kWideN);
  return narrow < 5000 + 390 * kblocks * ((wide_tiles + sms - 1) / sms);
}

template <bool Gated>
int enqueue_by_rows(const Product &p, const Args &a, cudaStream_t stream) {
  int sms = 0;
  int rc = device_sms(&sms);
  if (rc) return rc;
  if (p.offsets) return few_a_group(p.m, p.groups) ? enqueue_narrow<16, Gated>(p, a, sms, stream) : enqueue_wide<Gated>(p, a, sms, stream);
  if constexpr (!Gated) {
    if (p.m <= 16) return enqueue_narrow<16, false>(p, a, sms, stream);
    if (p.m <= 32) return enqueue_narrow<32, false>(p, a, sms, stream);
    if (p.m <= 64 || narrow_is_shorter(p.m, p.n, a.kblocks, sms)) return enqueue_narrow<64, false>(p, a, sms, stream);
  }
  return enqueue_wide<Gated>(p, a, sms, stream);
}

template <typename X>
int enqueue_few(const Product &p, const Args &a, cudaStream_t stream) {
  const size_t smem = (size_t)p.m * (a.kblocks * (kBlockK + 4) + 16);
  int rc = allow_smem<&reshard_product_few_kernel<X>>((size_t)(kFewBytes * 33 / 32 + 16 * kFewRows));
  if (rc) return rc;
  const cudaError_t e = launch(reshard_product_few_kernel<X>, dim3((unsigned)((p.n + kFewN - 1) / kFewN)), kFewWarps * 32, smem, 1, stream, a, p.w, p.w_stride);
  return e == cudaSuccess ? RESHARD_OK : cuda_error(e, "launching reshard_product_few_kernel");
}

}  // namespace

bool product_quantizes(int64_t m, int64_t k) { return m <= kFewMost && m * ((k + kBlockK - 1) / kBlockK * kBlockK) <= kFewBytes; }
bool product_gathers(int64_t m, int groups) { return few_a_group(m, groups); }

int enqueue_product(const Product &p, cudaStream_t stream) {
  Args a{};
  a.a_scale = p.a_scale;
  a.as_row = p.as_row;
  a.as_block = p.as_block;
  a.x = p.x ? p.x : p.a;
  a.x_stride = p.a_stride;
  a.cols = (int)p.k;
  a.w_scale = p.w_scale;
  a.offsets = p.offsets;
  a.order = p.order;
  a.per_row = p.per_row;
  a.a_rows = (int)(p.order ? p.a_rows : p.m);
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
  if (!p.offsets && !p.gated && product_quantizes(p.m, p.k)) {
    if (!p.x) return enqueue_few<uint8_t>(p, a, stream);
    if (p.out_dtype == RESHARD_F32) return enqueue_few<float>(p, a, stream);
    if (p.out_dtype == RESHARD_BF16) return enqueue_few<__nv_bfloat16>(p, a, stream);
    return enqueue_few<__half>(p, a, stream);
  }
  return p.gated ? enqueue_by_rows<true>(p, a, stream) : enqueue_by_rows<false>(p, a, stream);
}

}  // namespace ops
}  // namespace reshard

using namespace reshard;
using namespace reshard::ops;

extern "C" int reshard_ops_status(int32_t *status, int reset) try {
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
} OPS_CATCH
