// Rows of fp16, bf16 or fp32 elements as 16-byte vectors, shared by the kernels that move,
// combine or quantise rows.  A row starts wherever its pointer and stride put it, so vectors are
// only as aligned as one element: the memory system takes a dwordx4 access at any such address,
// and every length and stride goes through one code path.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_apq.h"

namespace moeapq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <int DT>
struct Elem;
template <>
struct Elem<MOE_DTYPE_F16> {
  using T = _Float16;
};
template <>
struct Elem<MOE_DTYPE_BF16> {
  using T = __bf16;
};
template <>
struct Elem<MOE_DTYPE_F32> {
  using T = float;
};

template <int DT>
constexpr int kElemSize = static_cast<int>(sizeof(typename Elem<DT>::T));
template <int DT>
constexpr int kPerVec = 16 / kElemSize<DT>;   // elements of one 16-byte vector

// A vector at an address aligned to one element.
template <int DT>
struct __attribute__((packed, aligned(kElemSize<DT>))) RowVec {
  u32x4 v;
};

// Streamed: read or written once in a call, so not kept in the caches (non-temporal).  A sum over
// sorted rows (8192 tokens x 8 rows of 3584 bf16) takes 96 us streamed and 112 us not.
constexpr bool kStreamed = true;

template <int DT, bool STREAMED>
__device__ __forceinline__ u32x4 load_vec(const void* p) {
  const auto* v = &static_cast<const RowVec<DT>*>(p)->v;
  return STREAMED ? __builtin_nontemporal_load(v) : *v;
}
template <int DT, bool STREAMED>
__device__ __forceinline__ void store_vec(void* p, u32x4 x) {
  auto* v = &static_cast<RowVec<DT>*>(p)->v;
  if (STREAMED)
    __builtin_nontemporal_store(x, v);
  else
    *v = x;
}

// Elements [0, n) of p, n <= kPerVec, as fp32 (exact); the rest are 0.
template <int DT, bool STREAMED = false>
__device__ __forceinline__ void load_elems(const typename Elem<DT>::T* p, int n, float (&f)[kPerVec<DT>]) {
  using T = typename Elem<DT>::T;
  constexpr int N = kPerVec<DT>;
  union {
    u32x4 v;
    T e[N];
  } u;
  u.v = u32x4{0, 0, 0, 0};
  if (n >= N) {
    u.v = load_vec<DT, STREAMED>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) u.e[i] = p[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = static_cast<float>(u.e[i]);
}

// f rounded once to the element type (nearest, ties to even) into elements [0, n) of p.
template <int DT, bool STREAMED = false>
__device__ __forceinline__ void store_elems(typename Elem<DT>::T* p, int n, const float (&f)[kPerVec<DT>]) {
  using T = typename Elem<DT>::T;
  constexpr int N = kPerVec<DT>;
  union {
    u32x4 v;
    T e[N];
  } u;
#pragma unroll
  for (int i = 0; i < N; ++i) u.e[i] = static_cast<T>(f[i]);
  if (n >= N) {
    store_vec<DT, STREAMED>(p, u.v);
  } else {
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < n) p[i] = u.e[i];
  }
}

// Calls f with the element type as a compile-time constant; dtype was checked by the entry point.
template <typename F>
inline void with_dtype(int dtype, F&& f) {
  if (dtype == MOE_DTYPE_F16)
    f(std::integral_constant<int, MOE_DTYPE_F16>{});
  else if (dtype == MOE_DTYPE_BF16)
    f(std::integral_constant<int, MOE_DTYPE_BF16>{});
  else
    f(std::integral_constant<int, MOE_DTYPE_F32>{});
}

}  // namespace moeapq
