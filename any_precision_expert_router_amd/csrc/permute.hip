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
constexpr int kTokenSlots = 4, kTokenMin = 512;   // from here on a row is read once for all its slots

// A row of `bytes` bytes, lane `at` of `step` copying it.
template <int SIZE, bool STREAMED_LOAD>
__device__ __forceinline__ void copy_row(const char* src, char* dst, int bytes, int at, int step) {
  constexpr int DT = SIZE == 4 ? MOE_DTYPE_F32 : MOE_DTYPE_F16;
  using T = typename Elem<DT>::T;
  const int vecs = bytes / 16;
#pragma unroll 4
  for (int v = at; v < vecs; v += step) store_vec<DT, kStreamed>(dst + 16 * v, load_vec<DT, STREAMED_LOAD>(src + 16 * v));
  const int tail = (bytes - vecs * 16) / SIZE;
  if (at < tail) reinterpret_cast<T*>(dst + vecs * 16)[at] = reinterpret_cast<const T*>(src + vecs * 16)[at];
}

// One wavefront per sorted position i (and per pair p = i for the pairs without an expert).  A token's
// row is read k times, from the caches after the first.  Short on latency: 16 tokens x 4 rows of 4 KiB
// take 2.4 us, against 2.7 us by token.
template <int SIZE>
__global__ __launch_bounds__(kRowThreads) void permute_gather_kernel(
    const char* __restrict__ x, int64_t x_bytes, int pairs_n, int k, int E, int row_bytes,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ offsets, const int32_t* __restrict__ pairs,
    char* __restrict__ xs, int64_t xs_bytes, int32_t* __restrict__ rows) {
  const int lane = threadIdx.x & 63;
  const int i = blockIdx.x * kRowWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (i >= pairs_n) return;
  if (lane == 0 && static_cast<uint32_t>(ids[i]) >= static_cast<uint32_t>(E)) rows[i] = -1;
  if (i >= offsets[E]) return;
  const int p = pairs[i];
  if (static_cast<uint32_t>(p) >= static_cast<uint32_t>(pairs_n)) return;  // not a grouping of these pairs
  if (lane == 0) rows[p] = i;
  copy_row<SIZE, false>(x + static_cast<int64_t>(p / k) * x_bytes, xs + static_cast<int64_t>(i) * xs_bytes, row_bytes,
                        lane, 64);
}

// One workgroup per token: its row is read once and written to its k places.  Slot j's place is found
// in its expert's part of `pairs`, which ascends, by bisection (k lanes at once).  2048 tokens x 8 rows
// of 7 KiB: 28.9 us (4.6 TB/s), 32.7 us by sorted position; 512 tokens: 8.4 and 9.2 us, 256: 6.4 and 5.0 us;
// 8192 tokens x 2 rows of 8 KiB: 46.0 and 40.6 us.  Hence the switch.
template <int SIZE>
__global__ __launch_bounds__(kRowThreads) void permute_token_kernel(
    const char* __restrict__ x, int64_t x_bytes, int pairs_n, int k, int E, int row_bytes,
    const int32_t* __restrict__ ids, const int32_t* __restrict__ offsets, const int32_t* __restrict__ pairs,
    char* __restrict__ xs, int64_t xs_bytes, int32_t* __restrict__ rows) {
  constexpr int DT = SIZE == 4 ? MOE_DTYPE_F32 : MOE_DTYPE_F16;
  using T = typename Elem<DT>::T;
  __shared__ int32_t place[MOE_MAX_TOPK];
  const int t = blockIdx.x, tid = threadIdx.x;
  if (tid < k) {
    const int p = t * k + tid, e = ids[p];
    int at = -1;
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) {
      int lo = max(offsets[e], 0), hi = min(offsets[e + 1], pairs_n);
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (pairs[mid] < p) lo = mid + 1;
        else hi = mid;
      }
      if (lo < min(offsets[e + 1], pairs_n) && pairs[lo] == p) at = lo;   // else: not a grouping of these pairs
    }
    rows[p] = at;
    place[tid] = at;
  }
  __syncthreads();
  const char* src = x + static_cast<int64_t>(t) * x_bytes;
  const int vecs = row_bytes / 16, tail = (row_bytes - vecs * 16) / SIZE;
  for (int v = tid; v < vecs; v += kRowThreads) {
    const u32x4 row = load_vec<DT, kStreamed>(src + 16 * v);
    for (int j = 0; j < k; ++j) {
      const int at = __builtin_amdgcn_readfirstlane(place[j]);
      if (at >= 0) store_vec<DT, kStreamed>(xs + static_cast<int64_t>(at) * xs_bytes + 16 * v, row);
    }
  }
  if (tid < tail) {
    const T last = reinterpret_cast<const T*>(src + vecs * 16)[tid];
    for (int j = 0; j < k; ++j) {
      const int at = __builtin_amdgcn_readfirstlane(place[j]);
      if (at >= 0) reinterpret_cast<T*>(xs + static_cast<int64_t>(at) * xs_bytes + vecs * 16)[tid] = last;
    }
  }
}

// One wavefront per (token, 64 vectors of its row): enough wavefronts for a single token's rows to be
// spread over the chip, and k independent loads a lane.  8192 tokens x 8 rows of 7 KiB with an added
// row: 96 us, 5.9 TB/s; 4099 x 10 rows of 8 KiB in fp32, ungated: 62 us, 6.0 TB/s.
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
    load_elems<DT, kStreamed>(ys + r * ys_stride + col, n, f);
    const float g = tg ? tg[j] : 1.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = fmaf(g, f[i], acc[i]);
  }
  if (add) {
    float f[N];
    load_elems<DT, kStreamed>(add + static_cast<int64_t>(t) * add_stride + col, n, f);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] += f[i];
  }
  store_elems<DT, kStreamed>(y + static_cast<int64_t>(t) * y_stride + col, n, acc);
}

// One workgroup per token.  Its dy stays in registers, kGradVecs vectors a lane at a time, while its
// rows go by once; the lanes' products are added in a fixed order.  4096 tokens x 8 rows of 7 KiB: 100 us,
// 5.0 TB/s of reads and writes in equal parts (a copy: 4.8).
constexpr int kGradVecs = 2;

template <int DT>
__global__ __launch_bounds__(kRowThreads) void combine_rows_grad_kernel(
    const typename Elem<DT>::T* __restrict__ dy, int64_t dy_stride, const typename Elem<DT>::T* __restrict__ ys,
    int64_t ys_stride, int T, int k, int H, const int32_t* __restrict__ rows, const float* __restrict__ gates,
    typename Elem<DT>::T* __restrict__ dys, int64_t dys_stride, float* __restrict__ dgates) {
  constexpr int N = kPerVec<DT>, kSpan = kRowThreads * N;
  __shared__ float part[kRowWaves][MOE_MAX_TOPK];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  for (int base = 0; base < H; base += kGradVecs * kSpan) {
    float d[kGradVecs][N];
    int col[kGradVecs], n[kGradVecs];
#pragma unroll
    for (int c = 0; c < kGradVecs; ++c) {
      col[c] = base + c * kSpan + threadIdx.x * N;
      n[c] = min(H - col[c], N);
      if (n[c] > 0) load_elems<DT, kStreamed>(dy + t * dy_stride + col[c], n[c], d[c]);
    }
    for (int j = 0; j < k; ++j) {
      const int r = rows[t * k + j];
      float dot = 0.0f;
      if (static_cast<uint32_t>(r) < static_cast<uint32_t>(T) * k) {
        const float g = gates ? gates[t * k + j] : 1.0f;
        float f[kGradVecs][N];
        if (dgates) {
#pragma unroll
          for (int c = 0; c < kGradVecs; ++c)
            if (n[c] > 0) load_elems<DT, kStreamed>(ys + r * ys_stride + col[c], n[c], f[c]);
        }
#pragma unroll
        for (int c = 0; c < kGradVecs; ++c) {
          if (n[c] <= 0) continue;
          if (dgates) {
#pragma unroll
            for (int i = 0; i < N; ++i) dot = fmaf(d[c][i], f[c][i], dot);
          }
          if (dys) {
            float o[N];
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = d[c][i] * g;
            store_elems<DT, kStreamed>(dys + r * dys_stride + col[c], n[c], o);
          }
        }
      }
      if (dgates) {
        dot = wave_sum_f32(dpp_settled(dot));
        if (lane == 0) part[wave][j] = base ? part[wave][j] + dot : dot;
      }
    }
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
  const bool by_token = k >= kTokenSlots && T >= kTokenMin;
  const dim3 grid(by_token ? T : (n + kRowWaves - 1) / kRowWaves), block(kRowThreads);
  const char* src = static_cast<const char*>(x);
  char* dst = static_cast<char*>(xs);
#define MOE_PERMUTE(KERNEL, SIZE)                                                                              \
  hipLaunchKernelGGL(KERNEL<SIZE>, grid, block, 0, stream, src, x_stride * SIZE, n, k, E, H * SIZE, ids, offsets, \
                     pairs, dst, xs_stride * SIZE, rows)
  if (by_token && size == 4) MOE_PERMUTE(permute_token_kernel, 4);
  else if (by_token) MOE_PERMUTE(permute_token_kernel, 2);
  else if (size == 4) MOE_PERMUTE(permute_gather_kernel, 4);
  else MOE_PERMUTE(permute_gather_kernel, 2);
#undef MOE_PERMUTE
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
