// Token rows sorted by expert and back, with their gradients.
//
//   permute:             xs[i] = x[pairs[i] / k] for i < offsets[E];  rows[pairs[i]] = i, rows[p] = -1
//                        for a pair that names no expert
//   its gradient:        dx[t] = sum_j dxs[rows[t,j]]
//   unpermute:           y[t] = add[t] + sum_j g[t,j] ys[rows[t,j]]
//   its gradient:        dys[rows[t,j]] = g[t,j] dy[t];  dg[t,j] = <dy[t], ys[rows[t,j]]>
//
// All four only move rows: what bounds them is the traffic of the T*k sorted rows.  Nothing is
// added up across workgroups, so no atomics are needed and results do not depend on timing: a
// token's k rows are known from `rows`, the inverse of `pairs`.  Sums are fp32 in slot order,
// rounded once.
#include <type_traits>

#include "elements.hpp"
#include "internal.hpp"
#include "wave_ops.hpp"

namespace moeapq {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWaves = kRowThreads / 64;

// One wavefront per sorted position i (and per pair p = i for the pairs without an expert).
template <int SIZE>
__global__ __launch_bounds__(kRowThreads) void permute_kernel(
    const char* __restrict__ x, int64_t x_bytes, int pairs_n, int k, int E, int row_bytes,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ offsets, const int32_t* __restrict__ pairs,
    char* __restrict__ xs, int64_t xs_bytes, int32_t* __restrict__ rows) {
  constexpr int DT = SIZE == 4 ? MOE_DTYPE_F32 : MOE_DTYPE_F16;
  const int lane = threadIdx.x & 63;
  const int i = blockIdx.x * kRowWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (i >= pairs_n) return;
  if (lane == 0 && static_cast<uint32_t>(ids[i]) >= static_cast<uint32_t>(E)) rows[i] = -1;
  if (i >= offsets[E]) return;
  const int p = pairs[i];
  if (static_cast<uint32_t>(p) >= static_cast<uint32_t>(pairs_n)) return;  // not a grouping of these pairs
  if (lane == 0) rows[p] = i;
  const char* src = x + static_cast<int64_t>(p / k) * x_bytes;
  char* dst = xs + static_cast<int64_t>(i) * xs_bytes;
  const int vecs = row_bytes / 16;
#pragma unroll 4
  for (int v = lane; v < vecs; v += 64)
    reinterpret_cast<RowVec<DT>*>(dst)[v].v = reinterpret_cast<const RowVec<DT>*>(src)[v].v;
  using T = typename Elem<DT>::T;
  const int tail = (row_bytes - vecs * 16) / SIZE;
  if (lane < tail)
    reinterpret_cast<T*>(dst + vecs * 16)[lane] = reinterpret_cast<const T*>(src + vecs * 16)[lane];
}

// One wavefront per (token, 64 vectors of its row).
template <int DT>
__global__ __launch_bounds__(kRowThreads) void combine_rows_kernel(
    const typename Elem<DT>::T* __restrict__ ys, int64_t ys_stride, int T, int k, int H, int chunks,
    const int32_t* __restrict__ rows, const float* __restrict__ gates,
    const typename Elem<DT>::T* __restrict__ add, int64_t add_stride, typename Elem<DT>::T* __restrict__ y,
    int64_t y_stride) {
  constexpr int N = kPerVec<DT>;
  const int lane = threadIdx.x & 63;
  const uint32_t w = blockIdx.x * kRowWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t t = w / chunks;
  if (t >= static_cast<uint32_t>(T)) return;
  const int col = (static_cast<int>(w - t * chunks) * 64 + lane) * N;
  const int n = min(H - col, N);
  if (n <= 0) return;
  const int32_t* tr = rows + static_cast<int64_t>(t) * k;
  const float* tg = gates ? gates + static_cast<int64_t>(t) * k : nullptr;
  float acc[N] = {};
  for (int j = 0; j < k; ++j) {
    const int r = tr[j];
    if (static_cast<uint32_t>(r) >= static_cast<uint32_t>(T) * k) continue;  // the pair has no row
    float f[N];
    load_elems<DT>(ys + r * ys_stride + col, n, f);
    const float g = tg ? tg[j] : 1.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = fmaf(g, f[i], acc[i]);
  }
  if (add) {
    float f[N];
    load_elems<DT>(add + static_cast<int64_t>(t) * add_stride + col, n, f);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += f[i];
  }
  store_elems<DT>(y + static_cast<int64_t>(t) * y_stride + col, n, acc);
}

// One workgroup per token.
template <int DT>
__global__ __launch_bounds__(kRowThreads) void combine_rows_grad_kernel(
    const typename Elem<DT>::T* __restrict__ dy, int64_t dy_stride, const typename Elem<DT>::T* __restrict__ ys,
    int64_t ys_stride, int T, int k, int H, const int32_t* __restrict__ rows, const float* __restrict__ gates,
    typename Elem<DT>::T* __restrict__ dys, int64_t dys_stride, float* __restrict__ dgates) {
  constexpr int N = kPerVec<DT>;
  __shared__ float part[kRowWaves][MOE_MAX_TOPK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  for (int j = 0; j < k; ++j) {
    const int r = rows[t * k + j];
    float dot = 0.0f;
    if (static_cast<uint32_t>(r) < static_cast<uint32_t>(T) * k) {
      const float g = gates ? gates[t * k + j] : 1.0f;
      for (int col = threadIdx.x * N; col < H; col += kRowThreads * N) {
        const int n = min(H - col, N);
        float d[N], f[N];
        load_elems<DT>(dy + t * dy_stride + col, n, d);
        if (dgates) {
          load_elems<DT>(ys + r * ys_stride + col, n, f);
#pragma unroll
          for (int i = 0; i < N; ++i) dot = fmaf(d[i], f[i], dot);
        }
        if (dys) {
#pragma unroll
          for (int i = 0; i < N; ++i) d[i] *= g;
          store_elems<DT>(dys + r * dys_stride + col, n, d);
        }
      }
    }
    dot = wave_sum_f32(dpp_settled(dot));
    if (lane == 0) part[wave][j] = dot;
  }
  __syncthreads();
  const int j = threadIdx.x;
  if (dgates && j < k) dgates[t * k + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
}

}  // namespace

int launch_permute_tokens(const void* x, int dtype, int64_t x_stride, int T, int k, int E, int H,
                          const int32_t* ids, const int32_t* offsets, const int32_t* pairs, void* xs,
                          int64_t xs_stride, int32_t* rows, hipStream_t stream) {
  ProfileScope prof("permute_tokens", stream);
  const int n = T * k, size = dtype == MOE_DTYPE_F32 ? 4 : 2;
  const dim3 grid((n + kRowWaves - 1) / kRowWaves), block(kRowThreads);
  const char* src = static_cast<const char*>(x);
  char* dst = static_cast<char*>(xs);
  if (size == 4)
    hipLaunchKernelGGL(permute_kernel<4>, grid, block, 0, stream, src, x_stride * size, n, k, E, H * size, ids,
                       offsets, pairs, dst, xs_stride * size, rows);
  else
    hipLaunchKernelGGL(permute_kernel<2>, grid, block, 0, stream, src, x_stride * size, n, k, E, H * size, ids,
                       offsets, pairs, dst, xs_stride * size, rows);
  return check_launch("permute_tokens");
}

int launch_combine_rows(const char* name, const void* ys, int dtype, int64_t ys_stride, int T, int k, int H,
                        const int32_t* rows, const float* gates, const void* add, int64_t add_stride, void* y,
                        int64_t y_stride, hipStream_t stream) {
  ProfileScope prof(name, stream);
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    using E = typename Elem<DT>::T;
    const int chunks = (H + 64 * kPerVec<DT> - 1) / (64 * kPerVec<DT>);
    const uint32_t waves = static_cast<uint32_t>(T) * chunks;
    hipLaunchKernelGGL(combine_rows_kernel<DT>, dim3((waves + kRowWaves - 1) / kRowWaves), dim3(kRowThreads), 0,
                       stream, static_cast<const E*>(ys), ys_stride, T, k, H, chunks, rows, gates,
                       static_cast<const E*>(add), add_stride, static_cast<E*>(y), y_stride);
  });
  return check_launch(name);
}

int launch_combine_rows_grad(const void* dy, int dtype, int64_t dy_stride, const void* ys, int64_t ys_stride, int T,
                             int k, int H, const int32_t* rows, const float* gates, void* dys, int64_t dys_stride,
                             float* dgates, hipStream_t stream) {
  ProfileScope prof("unpermute_tokens_backward", stream);
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    using E = typename Elem<DT>::T;
    hipLaunchKernelGGL(combine_rows_grad_kernel<DT>, dim3(T), dim3(kRowThreads), 0, stream,
                       static_cast<const E*>(dy), dy_stride, static_cast<const E*>(ys), ys_stride, T, k, H, rows,
                       gates, static_cast<E*>(dys), dys_stride, dgates);
  });
  return check_launch("unpermute_tokens_backward");
}

}  // namespace moeapq
