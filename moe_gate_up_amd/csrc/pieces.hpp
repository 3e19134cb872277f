// Pieces of 8 neighbouring elements of a row, at any alignment that the element
// type has (the device takes global accesses at any address): one or two 16-byte
// accesses; a row's last piece may be short.
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

  // Elements c .. c + 7 of a row of n; those behind the row are 0 and not read.  In two steps: request() makes the same
  // loads for every lane (one under a condition of the lane's would be waited for at its end), of the row's last 8 where
  // fewer are left, and settle() moves those into place.  A row that is written in place is given to it as `own`: another
  // lane may have stored the elements in front of a short piece since its request, so the lane's own are read once more.
  __device__ __forceinline__ void request(const T* row, int c, int n) {
    if (n >= kPiece) {
      const any4* from = reinterpret_cast<const any4*>(row + (uint32_t)min(c, n - kPiece));
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const any4 t = from[i];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * i + j] = t[j];
      }
    } else {
      T t[kPiece];
#pragma unroll
      for (int i = 0; i < kPiece; ++i) t[i] = c + i < n ? row[c + i] : (T)0.0f;
      __builtin_memcpy(v, t, sizeof(v));
    }
  }
  __device__ __forceinline__ void settle(int c, int n, const T* own = nullptr) {
    if (c + kPiece <= n || n < kPiece) return;
    if (own) {
      T t[kPiece];
#pragma unroll
      for (int i = 0; i < kPiece; ++i) t[i] = c + i < n ? own[c + i] : (T)0.0f;
      __builtin_memcpy(v, t, sizeof(v));
      return;
    }
    const int s = min(c + kPiece - n, kPiece);   // elements that are not the lane's come first
    constexpr int K = 4 * kWords;
#pragma unroll
    for (int step = 8; step > 0; step /= 2) {
      const int by = step * (int)sizeof(T) / 4;   // in words; 0: half a one
#pragma unroll
      for (int i = 0; i < K; ++i) {
        uint32_t moved;
        if (by == 0) moved = v[i] >> 16 | (i + 1 < K ? v[i + 1] << 16 : 0u);
        else moved = i + by < K ? v[i + by] : 0u;
        v[i] = (s & step) ? moved : v[i];
      }
    }
  }
  __device__ __forceinline__ void store(T* row, int c, int n) const { put<false>(row, c, n); }
  // As store(), past the caches: for results much larger than they are, which would push out what is still to be read.
  __device__ __forceinline__ void stream(T* row, int c, int n) const { put<true>(row, c, n); }
  template <bool STREAM>
  __device__ __forceinline__ void put(T* row, int c, int n) const {
    if (c + kPiece <= n) {
      any4* to = reinterpret_cast<any4*>(row + (uint32_t)c);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const any4 t{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        if constexpr (STREAM) __builtin_nontemporal_store(t, to + i);
        else to[i] = t;
      }
    } else {
      T t[kPiece];
      __builtin_memcpy(t, v, sizeof(v));
#pragma unroll
      for (int i = 0; i < kPiece; ++i)
        if (c + i < n) row[c + i] = t[i];
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
