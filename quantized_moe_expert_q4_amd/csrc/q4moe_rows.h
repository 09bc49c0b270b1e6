// Wide loads from rows that may start at any multiple of their element.
#pragma once
#include "q4moe_device.h"

namespace q4 {

// A matrix of `count` elements (at least one) in rows of C; T is uint16_t for bf16.
template <class T>
struct RowMatrix {
  const T* data;
  size_t count;
  int C;
  __device__ RowMatrix(const void* p, int rows, int columns)
      : data(static_cast<const T*>(p)), count((size_t)rows * columns), C(columns) {}

  // 16 bytes of a row from element c on, zeros past its end.  The last elements
  // of a row come with what follows them, those of the matrix with what
  // precedes them, so that no load leaves it.
  __device__ __forceinline__ v4u chunk(int row, int c) const {
    constexpr int kVec = 16 / sizeof(T), kBits = 8 * sizeof(T);
    const size_t at = (size_t)row * C + c;
    const int left = C - c;
    v4u r = {0, 0, 0, 0};
    if (left >= kVec) {
      __builtin_memcpy(&r, data + at, 16);
    } else if (left > 0) {
      unsigned __int128 v = 0;
      if (count >= kVec) {
        const size_t from = at + kVec <= count ? at : count - kVec;
        __builtin_memcpy(&v, data + from, 16);
        v >>= kBits * (int)(at - from);
      } else {
#pragma unroll 1
        for (int i = 0; i < left; ++i) {
          T e = data[at + i];
          uint32_t u = 0;
          __builtin_memcpy(&u, &e, sizeof(T));
          v |= (unsigned __int128)u << (kBits * i);
        }
      }
      v &= ((unsigned __int128)1 << (kBits * left)) - 1;
      __builtin_memcpy(&r, &v, 16);
    }
    return r;
  }
};

// The same for a reader that has no use for the columns past a row's end but
// may read what lies there: load() always reads 16 bytes inside the matrix, at
// the wanted place unless that leaves it; aligned() then puts them in place.
template <class T>
struct ColumnRuns {
  const T* data;
  size_t last;            // the last place of a load; a smaller matrix is read element by element
  int C;
  bool tiny;
  static constexpr int kVec = 16 / sizeof(T), kBits = 8 * sizeof(T);
  __device__ ColumnRuns(const void* p, int rows, int columns)
      : data(static_cast<const T*>(p)), last((size_t)rows * columns - kVec), C(columns),
        tiny((size_t)rows * columns < kVec) {}

  __device__ __forceinline__ v4u load(int row, int c) const {
    v4u r = {0, 0, 0, 0};
    const size_t at = (size_t)row * C + c;
    if (!tiny) __builtin_memcpy(&r, data + (at < last ? at : last), 16);
    return r;
  }

  __device__ __forceinline__ v4u aligned(v4u r, int row, int c) const {
    const size_t at = (size_t)row * C + c;
    unsigned __int128 v = 0;
    if (tiny) {
#pragma unroll 1
      for (int i = 0; i < C - c; ++i) {
        T e = data[at + i];
        uint32_t u = 0;
        __builtin_memcpy(&u, &e, sizeof(T));
        v |= (unsigned __int128)u << (kBits * i);
      }
    } else {
      __builtin_memcpy(&v, &r, 16);
      if (c < C && at > last) v >>= kBits * (int)(at - last);
    }
    __builtin_memcpy(&r, &v, 16);
    return r;
  }
};

}  // namespace q4
