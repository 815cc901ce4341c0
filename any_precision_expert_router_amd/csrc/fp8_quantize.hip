// Rows quantised to e4m3 with one fp32 scale for each 128 columns, directly or through the
// SiLU gate (the step between the two products of an expert FFN).
//
//   v = x, or silu(g) * u = g / (1 + exp(-g)) * u in fp32 (not rounded before it is quantised)
//   m = max |v| over the block's finite values, at least 2^-100
//   scale = m / 448,  q = e4m3(v * (448 / m)), nearest, ties to even
//
// 448 is e4m3's largest value; |v * (448/m)| is at most 448 (1 + 2^-22), which still rounds to
// 448, so no clamp is needed.  The floor of 2^-100 keeps 448 / m and m / 448 normal fp32 numbers
// for blocks that are zero or nearly so.  A value that is not finite becomes e4m3's NaN and
// leaves the rest of its block alone.
#include <type_traits>

#include "elements.hpp"
#include "internal.hpp"
#include "wave_ops.hpp"

namespace moeapq {
namespace {

constexpr int kQuantThreads = 256;
constexpr int kQuantWaves = kQuantThreads / 64;
constexpr int kLaneCols = 8;                  // columns of one lane; 16 lanes hold a block
constexpr int kWaveCols = 64 * kLaneCols;
constexpr uint32_t kInfBits = 0x7f800000u;

// Elements [0, n) of p as fp32, n <= 8.
template <int DT>
__device__ __forceinline__ void load_cols(const typename Elem<DT>::T* p, int n, float (&f)[kLaneCols]) {
  constexpr int N = kPerVec<DT>;
#pragma unroll
  for (int h = 0; h < kLaneCols / N; ++h) {
    float part[N];
    load_elems<DT>(p + h * N, min(n - h * N, N), part);
#pragma unroll
    for (int i = 0; i < N; ++i) f[h * N + i] = part[i];
  }
}

// Maximum over the 16 lanes of a DPP row.
__device__ __forceinline__ uint32_t row_max_u32(uint32_t v) {
  v = max_dpp32<0xB1>(v);
  v = max_dpp32<0x4E>(v);
  v = max_dpp32<0x141>(v);
  return max_dpp32<0x140>(v);
}

// silu(g) * u.  exp(-g) as 2^t with the rounding of t = -g log2(e) carried along (without it the
// relative error grows as |g| 2^-24), and the quotient g / (1 + e) corrected once by its remainder:
// v is as exact as with a library exp and a division, so no more values than with those land on the
// other side of an e4m3 border (7e-5 of the values' norm on normal data, 1.1e-4 without the
// correction).  Outside +-86 the exponential is held at its value there, 1 + e is finite, and the
// quotient is g on one side and taken as 0 on the other.
__device__ __forceinline__ float silu_gate(float g, float u) {
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299112661746887e-8f, kLn2 = 0.69314718055994530942f;
  const float h = __builtin_amdgcn_fmed3f(g, -86.0f, 86.0f);
  const float t = -h * kLog2e;
  const float low = fmaf(-h, kLog2eLow, fmaf(-h, kLog2e, -t));
  float e = __builtin_amdgcn_exp2f(t);
  e = fmaf(e, low * kLn2, e);
  const float d = 1.0f + e;
  const float r = g < -86.0f ? 0.0f : __builtin_amdgcn_rcpf(d);
  const float q = g * r;
  return fmaf(fmaf(-d, q, g), r, q) * u;
}

// One wavefront per (row, 512 columns): 16 lanes hold a block, so its maximum is a DPP row's, and a
// single row still spreads over wavefronts.  15565 gated rows of 2 x 2560 bf16: 40 us, 5.0 TB/s, reads and
// the gate's 15 operations an element together.
template <int DT, bool SILU>
__global__ __launch_bounds__(kQuantThreads) void fp8_quantize_kernel(
    const typename Elem<DT>::T* __restrict__ x, int64_t x_stride, int M, int K, int chunks,
    const int32_t* __restrict__ n_rows, uint8_t* __restrict__ q, int64_t q_stride, float* __restrict__ scales) {
  const int lane = threadIdx.x & 63;
  const uint32_t w = blockIdx.x * kQuantWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t row = w / chunks;
  if (row >= static_cast<uint32_t>(M)) return;
  if (n_rows && static_cast<int>(row) >= *n_rows) return;
  const int col = (static_cast<int>(w - row * chunks) * 64 + lane) * kLaneCols;
  const int n = max(0, min(K - col, kLaneCols));
  float v[kLaneCols];
  load_cols<DT>(x + row * x_stride + col, n, v);
  if (SILU) {
    float u[kLaneCols];
    load_cols<DT>(x + row * x_stride + K + col, n, u);
#pragma unroll
    for (int i = 0; i < kLaneCols; ++i) v[i] = silu_gate(v[i], u[i]);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kLaneCols; ++i) top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
  top = row_max_u32(top);
  if (top >= kInfBits) {   // values that are not finite: NaN in e4m3, and left out of the maximum
    uint32_t finite = 0;
#pragma unroll
    for (int i = 0; i < kLaneCols; ++i) {
      const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
      if (a < kInfBits)
        finite = max(finite, a);
      else
        v[i] = __uint_as_float(0x7fc00000u);
    }
    top = row_max_u32(finite);   // the 16 lanes of a block are here together
  }
  const float m = fmaxf(__uint_as_float(top), 0x1p-100f);
  const float inv = __fdiv_rn(448.0f, m);
  u32x2 packed;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int word = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
    word = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, word, true);
    packed[h] = static_cast<uint32_t>(word);
  }
  uint8_t* dst = q + row * q_stride + col;
  if (n == kLaneCols) {
    struct __attribute__((packed, aligned(1))) Bytes { u32x2 v; };
    reinterpret_cast<Bytes*>(dst)->v = packed;
  } else {
#pragma unroll
    for (int i = 0; i < kLaneCols; ++i)
      if (i < n) dst[i] = static_cast<uint8_t>(packed[i / 4] >> (8 * (i % 4)));
  }
  if ((lane & 15) == 0 && n > 0)
    scales[static_cast<int64_t>(row) * ((K + MOE_FP8_BLOCK - 1) / MOE_FP8_BLOCK) + col / MOE_FP8_BLOCK] =
        __fdiv_rn(m, 448.0f);
}

}  // namespace

int launch_fp8_quantize(const char* name, bool silu, const void* x, int dtype, int64_t x_stride, int M, int K,
                        const int32_t* n_rows, uint8_t* q, int64_t q_stride, float* scales, hipStream_t stream) {
  ProfileScope prof(name, stream);
  const int chunks = (K + kWaveCols - 1) / kWaveCols;
  const uint64_t waves = static_cast<uint64_t>(M) * chunks;
  const dim3 grid(static_cast<uint32_t>((waves + kQuantWaves - 1) / kQuantWaves)), block(kQuantThreads);
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const auto* src = static_cast<const typename Elem<DT>::T*>(x);
    if (silu)
      hipLaunchKernelGGL((fp8_quantize_kernel<DT, true>), grid, block, 0, stream, src, x_stride, M, K, chunks, n_rows,
                         q, q_stride, scales);
    else
      hipLaunchKernelGGL((fp8_quantize_kernel<DT, false>), grid, block, 0, stream, src, x_stride, M, K, chunks, n_rows,
                         q, q_stride, scales);
  });
  return check_launch(name);
}

}  // namespace moeapq
