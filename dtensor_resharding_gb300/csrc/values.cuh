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

// The 16-byte words that hold N values at p, wherever p is: ask() reads them (words that hold none of the `left` values
// are not read, `any` is in their place), take() shifts the values into place and clears those from `left` on. Rows that
// start anywhere are read as fast as aligned ones this way; value by value they took three times as long.
template <typename T, int N>
struct Shifted {
  static constexpr int kWords = N * (int)sizeof(T) / 4;
  static_assert(kWords % 4 == 0, "16-byte words");
  uint32_t w[kWords + 4];
  __device__ __forceinline__ void ask(const T *p, int left, const uint8_t *any) {
    const uintptr_t skip = reinterpret_cast<uintptr_t>(p) & 15;
    const uint8_t *from = reinterpret_cast<const uint8_t *>(p) - skip;
    const int end = left > 0 ? (int)skip + min(left, N) * (int)sizeof(T) : 0;        // bytes from there to the last value
#pragma unroll
    for (int i = 0; i < kWords + 4; i += 4) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(4 * i < end ? from + 4 * i : any));
      w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
    }
  }
  __device__ __forceinline__ void take(const T *p, int left, uint32_t (&v)[kWords]) {
    const uint32_t skip = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
#pragma unroll
    for (int i = 0; i < kWords + 3; ++i) w[i] = skip & 4 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < kWords + 2; ++i) w[i] = skip & 8 ? w[i + 2] : w[i];
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

// Eight neighbours of a row, all inside it: `Wide` rows start on 16 bytes, others anywhere. ask() starts the loads.
template <typename T, bool Wide>
struct Eight {
  std::conditional_t<Wide, Pack<T, 8>, Shifted<T, 8>> w;
  __device__ __forceinline__ void ask(const T *p) {
    if constexpr (Wide) w = *reinterpret_cast<const Pack<T, 8> *>(p);
    else w.ask(p, 8, first_word(p));
  }
  __device__ __forceinline__ Pack<T, 8> bits(const T *p) {
    if constexpr (Wide) {
      return w;
    } else {
      uint32_t v[Shifted<T, 8>::kWords];
      w.take(p, 8, v);
      Pack<T, 8> r;
#pragma unroll
      for (int i = 0; i < Shifted<T, 8>::kWords; i += 4) reinterpret_cast<uint4 *>(&r)[i / 4] = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      return r;
    }
  }
  __device__ __forceinline__ void take(const T *p, float (&x)[8]) {
    const Pack<T, 8> r = bits(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(r.v[i]);
  }
};

// Eight values rounded to T and stored at a 16-byte boundary.
template <typename T>
__device__ __forceinline__ void store_eight(T *p, const float (&x)[8]) {
  Pack<T, 8> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = from_f32<T>(x[i]);
  *reinterpret_cast<Pack<T, 8> *>(p) = r;
}

// A row's columns in pieces of eight whose places in the row that is written start on 16 bytes: where rows start anywhere
// the first piece begins that much before the row, and it and the last are written value by value.
template <typename T, bool Wide>
__device__ __forceinline__ int64_t piece_start(int64_t piece, const T *row) {
  if constexpr (Wide) return piece * 8;
  else return piece * 8 - (int64_t)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
}
// The pieces that a row of so many columns can have.
template <typename T>
constexpr int64_t piece_count(int64_t cols, bool wide) {
  return wide ? (cols + 7) / 8 : (cols + 7 + (16 / (int)sizeof(T) - 1)) / 8;
}

#endif  // __CUDACC__

}  // namespace ops
}  // namespace reshard
