// tt_rows.h -- rows of any width and alignment, eight elements at a time.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ttb {

// Eight elements of a row, on an element's boundary (int8 too: a row's last group may start on any
// byte).  A row's last group takes its last eight, whatever its width: two lanes then work the same
// columns out from the same values in the same order and store the same bits, and no load hides
// behind a branch.
// Rows narrower than eight are a variant of their own (NARROW).
template <class T>
struct Eight {
  T x[8];
};
template <bool NARROW>
__device__ __forceinline__ int64_t column(int64_t group, int64_t d) {
  return NARROW ? 0 : min(group * 8, d - 8);
}
template <bool NARROW, class T>
__device__ __forceinline__ Eight<T> get8(const T *p, int64_t d) {
  if constexpr (NARROW) {
    Eight<T> r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.x[e] = e < d ? p[e] : (T)0;
    return r;
  } else {
    typedef int words __attribute__((ext_vector_type(sizeof(Eight<T>) / 4)));
    struct __attribute__((packed, aligned(sizeof(T) < 2 ? 1 : 2))) any { words v; };
    return __builtin_bit_cast(Eight<T>, ((const any *)p)->v);
  }
}
template <bool NARROW, class T>
__device__ __forceinline__ void put8(T *p, const Eight<T> &r, int64_t d) {
  if constexpr (NARROW) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < d) p[e] = r.x[e];
  } else {
    typedef int words __attribute__((ext_vector_type(sizeof(Eight<T>) / 4)));
    struct __attribute__((packed, aligned(sizeof(T) < 2 ? 1 : 2))) any { words v; };
    ((any *)p)->v = __builtin_bit_cast(words, r);
  }
}

}  // namespace ttb
