// Values of a row in registers: loads and stores of eight or more neighbours, aligned or not.
#pragma once
#include <type_traits>

#include "ops_common.cuh"

namespace reshard {
namespace ops {

// Whether every row of a matrix starts on a 16-byte boundary.
inline bool aligned16(const void *p, int64_t stride, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (stride * bytes) % 16 == 0;
}

// Calls f with a value of the type that dtype names.
template <typename F>
auto by_type(int dtype, F &&f) {
  return dtype == RESHARD_F32 ? f(float()) : dtype == RESHARD_BF16 ? f(__nv_bfloat16()) : f(__half());
}

#ifdef __CUDACC__

constexpr uint32_t kFull = 0xffffffffu;

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

// The 16-byte words (8-byte ones for 8 bytes of values) that hold N values at p, wherever p is: ask() reads them (words that
// hold none of the `left` values are not read, `any` is in their place), take() shifts the values into place and clears those from
// `left` on. Rows that start anywhere are read as fast as aligned ones this way; value by value they took three times as long.
// The loads are asked for as such: as plain ones, which the compiler spreads among what follows, 16,384 x 4095 fp32 quantized by rows
// take 58.2 us instead of 56.3, 16 blocked matrices of 2045 x 2043 fp32 71.6 instead of 65.7.
template <typename T, int N>
struct Shifted {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  static constexpr int kLoad = kWords % 4 == 0 ? 4 : 2;        // 32-bit words of a load
  static_assert(kWords % kLoad == 0, "whole loads");
  uint32_t w[kWords + kLoad];
  static __device__ __forceinline__ uint32_t skip_of(const T *p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) & (4 * kLoad - 1)); }
  __device__ __forceinline__ void ask(const T *p, int left, const uint8_t *any) {
    const uint32_t skip = skip_of(p);
    const uint8_t *from = reinterpret_cast<const uint8_t *>(p) - skip;
    const int end = left > 0 ? (int)skip + min(left, N) * (int)sizeof(T) : 0;        // bytes from there to the last value
#pragma unroll
    for (int i = 0; i < kWords + kLoad; i += kLoad) {
      const uint8_t *const at = 4 * i < end ? from + 4 * i : any;
      if constexpr (kLoad == 4) {
        const uint4 v = __ldca(reinterpret_cast<const uint4 *>(at));
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(at);
        w[i] = v.x, w[i + 1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void take(const T *p, int left, uint32_t (&v)[kWords]) {
    const uint32_t skip = skip_of(p);
#pragma unroll
    for (int i = 0; i < kWords + kLoad - 1; ++i) w[i] = skip & 4 ? w[i + 1] : w[i];
    if constexpr (kLoad == 4) {
#pragma unroll
      for (int i = 0; i < kWords + 2; ++i) w[i] = skip & 8 ? w[i + 2] : w[i];
    }
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

// Rows are moved in pieces of as many neighbours as make 16 bytes of the wider of two types: a warp's loads and stores then
// cover whole sectors. (Eight floats a thread in two stores of 16 bytes, half a sector each: 604M bf16 values to fp32 took 690 us instead
// of 570.)
template <typename A, typename B>
constexpr int kPieceOf = sizeof(A) == 4 || sizeof(B) == 4 ? 4 : 8;

// N values of type T as the 32-bit words that hold them, in loads and stores of 8 or 16 bytes. Values stay words until they are
// computed with: taken apart as 16-bit registers, as they arrive, they spilled.
template <typename T, int N>
struct Words {
  static constexpr int kCount = N * (int)sizeof(T) / 4;
  static_assert(kCount == 2 || kCount % 4 == 0, "8 bytes, or 16-byte words");
  uint32_t v[kCount];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (kCount == 2) {
      const uint2 x = *reinterpret_cast<const uint2 *>(p);
      v[0] = x.x, v[1] = x.y;
    } else {
#pragma unroll
      for (int i = 0; i < kCount; i += 4) {
        const uint4 x = reinterpret_cast<const uint4 *>(p)[i / 4];
        v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
      }
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (kCount == 2) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(v[0], v[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kCount; i += 4) reinterpret_cast<uint4 *>(p)[i / 4] = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
  }
  __device__ __forceinline__ void values(float (&x)[N]) const {
    if constexpr (std::is_same_v<T, __half>) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v[i / 2]));
        x[i] = f.x, x[i + 1] = f.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = value_of<T>(v, i);
    }
  }
  __device__ __forceinline__ void round(const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      if constexpr (std::is_same_v<T, float>) {
        v[i] = __float_as_uint(x[i]);
      } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        v[i] = *reinterpret_cast<const uint32_t *>(&r);
      } else {
        const __half2 r = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        v[i] = *reinterpret_cast<const uint32_t *>(&r);
      }
    }
  }
};

// N neighbours of a row, all inside it: `Wide` rows start on 16 bytes, others anywhere. ask() starts the loads.
template <typename T, int N, bool Wide>
struct Piece {
  std::conditional_t<Wide, Words<T, N>, Shifted<T, N>> w;
  __device__ __forceinline__ void ask(const T *p) {
    if constexpr (Wide) w.load(p);
    else w.ask(p, N, reinterpret_cast<const uint8_t *>(p) - Shifted<T, N>::skip_of(p));
  }
  __device__ __forceinline__ Words<T, N> words(const T *p) {
    if constexpr (Wide) {
      return w;
    } else {
      Words<T, N> r;
      w.take(p, N, r.v);
      return r;
    }
  }
  __device__ __forceinline__ void take(const T *p, float (&x)[N]) { words(p).values(x); }
};

// U pieces of N neighbours for each lane of a warp, which lie side by side in one row that starts anywhere: piece u of lane l
// begins at p + (32 u + l) N. Every lane reads the word (of a piece's size) that its piece begins in, and has the rest from the lane
// behind it; words without a value of the row are not read. Elements outside the row hold anything. All lanes call.
template <typename T, int N, int U>
struct Strip {
  static constexpr int kCount = Words<T, N>::kCount;
  static constexpr uint32_t kBytes = 4 * kCount;
  Words<T, N> w[U], tail;
  uint32_t skip;                     // bytes of the first piece's word before it; the same for all pieces
  // row, cols: what may be read; first: lane 0's first piece
  __device__ __forceinline__ void ask(const T *row, int64_t cols, int64_t first, int lane) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(row + first), lo = reinterpret_cast<uintptr_t>(row), hi = reinterpret_cast<uintptr_t>(row + cols);
    skip = (uint32_t)(p & (kBytes - 1));
    const uintptr_t base = p - skip;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uintptr_t at = base + (uintptr_t)(32 * u + lane) * kBytes;
      if (at + kBytes > lo && at < hi) w[u].load(reinterpret_cast<const T *>(at));
    }
    const uintptr_t at = base + (uintptr_t)(32 * U) * kBytes;
    if (lane == 0 && at + kBytes > lo && at < hi) tail.load(reinterpret_cast<const T *>(at));
  }
  __device__ __forceinline__ Words<T, N> words(int u, int lane) const {
    uint32_t x[2 * kCount];
#pragma unroll
    for (int i = 0; i < kCount; ++i) {
      x[i] = w[u].v[i];
      // lane 31's neighbour is lane 0 of the next piece
      x[kCount + i] = __shfl_sync(kFull, lane == 0 ? (u + 1 < U ? w[u + 1 < U ? u + 1 : u].v[i] : tail.v[i]) : w[u].v[i], (lane + 1) & 31);
    }
    if constexpr (kCount == 4) {
      if (skip & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) x[i] = x[i + 2];
      }
    }
    if (skip & 4) {
#pragma unroll
      for (int i = 0; i < kCount + 1; ++i) x[i] = x[i + 1];
    }
    Words<T, N> r;
#pragma unroll
    for (int i = 0; i < kCount; ++i) r.v[i] = sizeof(T) == 4 ? x[i] : __funnelshift_r(x[i], x[i + 1], 8 * (skip & 3));
    return r;
  }
};

// N values rounded to T and stored at a boundary of as many.
template <typename T, int N>
__device__ __forceinline__ void store_piece(T *p, const float (&x)[N]) {
  Words<T, N> r;
  r.round(x);
  r.store(p);
}

// Where a row's piece begins, so that its place in the row that is written is a boundary of N values: where rows start
// anywhere the first piece begins that much before the row, and it and the last are written value by value.
template <typename T, int N, bool Wide>
__device__ __forceinline__ int64_t piece_start(int64_t piece, const T *row) {
  if constexpr (Wide) return piece * N;
  else return piece * N - (int64_t)((reinterpret_cast<uintptr_t>(row) & (N * sizeof(T) - 1)) / sizeof(T));
}

#endif  // __CUDACC__

// The pieces of so many values that a row of so many columns can have.
inline int64_t piece_count(int64_t cols, int values, bool wide) { return wide ? (cols + values - 1) / values : (cols + 2 * (values - 1)) / values; }

}  // namespace ops
}  // namespace reshard
