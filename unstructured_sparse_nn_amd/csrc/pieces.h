// pieces.h -- rows moved 16 bytes a lane, at any alignment.
#pragma once

#include "common.h"

namespace snk {

// ------------------------------------------------------------- 16-byte pieces
// Rows start at any element, so pieces are loaded and stored without an
// alignment claim; the hardware takes a 16-byte access at any address.
template <typename T> constexpr int EL = 16 / sizeof(T);
template <typename T> struct __attribute__((aligned(16))) frag { uint32_t w[4]; };

__device__ __forceinline__ float at(const frag<bf16>& f, int e) {
  return __uint_as_float(e & 1 ? f.w[e / 2] & 0xFFFF0000u : f.w[e / 2] << 16);
}
__device__ __forceinline__ float at(const frag<float>& f, int e) { return __uint_as_float(f.w[e]); }

template <typename T>
__device__ __forceinline__ frag<T> load_frag(const T* p) {
  frag<T> f;
  __builtin_memcpy(&f, p, 16);
  return f;
}
template <typename T>
__device__ __forceinline__ void store_frag(T* p, const frag<T>& f, int32_t n) {
  if (n >= EL<T>) {
    __builtin_memcpy(p, &f, 16);
  } else {
#pragma unroll
    for (int e = 0; e < EL<T> - 1; ++e)
      if (e < n) {
        const uint32_t v = f.w[e * sizeof(T) / 4] >> (8 * (e * sizeof(T) % 4));
        __builtin_memcpy(p + e, &v, sizeof(T));
      }
  }
}

// Two floats as bf16, rounded to nearest even, in one dword.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{a, b}), b2));
}
__device__ __forceinline__ frag<bf16> to_frag(const float (&v)[8]) {
  return frag<bf16>{{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                     bf16_pair(v[6], v[7])}};
}
__device__ __forceinline__ frag<float> to_frag(const float (&v)[4]) {
  return frag<float>{{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3])}};
}

__device__ __forceinline__ void floats_of(const frag<bf16>& f, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = at(f, e);
}
__device__ __forceinline__ void floats_of(const frag<float>& f, float (&v)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = at(f, e);
}

// -------------------------------------------------------------- rows by pieces
// A row of n elements is cut into cdiv(n, EL) pieces.  Piece q starts at q EL,
// the last one early enough to be whole: then only its elements from `from` on
// are its own (the piece before it has the others).  Rows shorter than a piece
// are moved element by element.
struct cut_t { int32_t at, from; };
template <typename T>
__device__ __forceinline__ cut_t cut_of(int32_t q, int32_t n) {
  const int32_t c = q * EL<T>, at = max(min(c, n - EL<T>), 0);
  return {at, c - at};
}
template <typename T>
__device__ __forceinline__ frag<T> load_cut(const T* row, cut_t c, int32_t n) {
  if (n >= EL<T>) return load_frag(row + c.at);
  frag<T> f{};
#pragma unroll
  for (int e = 0; e < EL<T> - 1; ++e)
    if (e < n) {
      uint32_t v = 0;
      __builtin_memcpy(&v, row + e, sizeof(T));
      f.w[e * sizeof(T) / 4] |= v << (8 * (e * sizeof(T) % 4));
    }
  return f;
}
template <typename T>
__device__ __forceinline__ void store_cut(T* row, cut_t c, int32_t n, const frag<T>& f) {
  if (c.from == 0 && n >= EL<T>) {
    __builtin_memcpy(row + c.at, &f, 16);
  } else {
#pragma unroll
    for (int e = 0; e < EL<T>; ++e)
      if (e >= c.from && c.at + e < n) {
        const uint32_t v = f.w[e * sizeof(T) / 4] >> (8 * (e * sizeof(T) % 4));
        __builtin_memcpy(row + c.at + e, &v, sizeof(T));
      }
  }
}

// Token numbers as the caller has them, 32 or 64 bits wide.  Those outside
// [0, n) become -1 (below) or -2 (past the end).
struct ids_t {
  const void* p;
  int32_t wide;
  __device__ __forceinline__ int32_t get(int64_t i, int32_t n) const {
    const int64_t v = wide ? static_cast<const int64_t*>(p)[i]
                           : (int64_t)static_cast<const int32_t*>(p)[i];
    return v < 0 ? -1 : v >= n ? -2 : (int32_t)v;
  }
};

// Pieces of a matrix that one launch covers with a thread each.
constexpr int64_t MAX_PIECES = (1ll << 32) - (1ll << 20);

}  // namespace snk
