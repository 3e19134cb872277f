// Pieces of 8 neighbouring elements of a row, at any alignment that the element
// type has (the device takes global accesses at any address): one or two 16-byte
// accesses, or element by element where a row ends inside the piece.
#pragma once

#include "prims.hpp"

namespace moe {

constexpr int kPiece = 8;

// 16 bytes at the alignment of an element of SIZE bytes.
template <int SIZE>
struct Any16;
template <>
struct Any16<2> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(2)));
};
template <>
struct Any16<4> {
  typedef uint32_t type __attribute__((ext_vector_type(4), aligned(4)));
};

// As 16-byte words: 8 elements of 16 bits in one, of 32 bits in two.
template <typename T>
struct Piece {
  typedef typename Any16<sizeof(T)>::type any4;
  static constexpr int kWords = (int)sizeof(T) / 2;
  uint32_t v[4 * kWords];

  // From `p`; elements from the left-th on are 0 and not read.
  __device__ __forceinline__ void load(const T* p, int left) {
    if (left >= kPiece) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const any4 t = reinterpret_cast<const any4*>(p)[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = t[j];
      }
    } else {
      T t[kPiece];
#pragma unroll
      for (int i = 0; i < kPiece; ++i) t[i] = i < left ? p[i] : (T)0.0f;
      __builtin_memcpy(v, t, sizeof(v));
    }
  }
  __device__ __forceinline__ void store(T* p, int left) const {
    if (left >= kPiece) {
#pragma unroll
      for (int i = 0; i < kWords; ++i)
        reinterpret_cast<any4*>(p)[i] = any4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    } else {
      T t[kPiece];
      __builtin_memcpy(t, v, sizeof(v));
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        if (i < left) p[i] = t[i];
    }
  }
  __device__ __forceinline__ void values(float (&f)[kPiece]) const {
    T t[kPiece];
    __builtin_memcpy(t, v, sizeof(v));
#pragma unroll
    for (int i = 0; i < kPiece; ++i) f[i] = (float)t[i];
  }
  // Rounded to nearest even.
  __device__ __forceinline__ void set(const float (&f)[kPiece]) {
    T t[kPiece];
#pragma unroll
    for (int i = 0; i < kPiece; ++i) t[i] = (T)f[i];
    __builtin_memcpy(v, t, sizeof(v));
  }
};

}  // namespace moe
