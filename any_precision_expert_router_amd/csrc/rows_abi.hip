// C-ABI entry points of the row operators: tokens sorted by expert and back, e4m3 quantising and
// the grouped e4m3 product.  Arguments are checked from host-visible scalars before any launch.
#include "internal.hpp"

namespace moeapq {
namespace {

constexpr int kMaxRows = MOE_MAX_TOKENS * MOE_MAX_TOPK;

int check_dtype(int dtype) {
  if (dtype < MOE_DTYPE_F16 || dtype > MOE_DTYPE_F32) return set_error(MOE_EINVAL, "unknown dtype %d", dtype);
  return MOE_OK;
}

int check_row(const char* what, int cols) {
  if (cols <= 0) return set_error(MOE_EINVAL, "need %s > 0 (got %d)", what, cols);
  if (cols > MOE_MAX_ROW) return set_error(MOE_EUNSUPPORTED, "%s=%d exceeds %d", what, cols, MOE_MAX_ROW);
  return MOE_OK;
}

int check_stride(const char* what, int64_t stride, int64_t cols) {
  if (stride < cols)
    return set_error(MOE_EINVAL, "%s row stride %lld is shorter than its %lld columns", what,
                     static_cast<long long>(stride), static_cast<long long>(cols));
  if (stride > (int64_t{1} << 40))
    return set_error(MOE_EUNSUPPORTED, "%s row stride %lld exceeds 2^40", what, static_cast<long long>(stride));
  return MOE_OK;
}

// Element pointers aligned to one element.
int check_align(const char* what, const void* p, int dtype) {
  const uintptr_t size = dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(p) & (size - 1))
    return set_error(MOE_EINVAL, "%s is not aligned to its %d-byte elements", what, static_cast<int>(size));
  return MOE_OK;
}

// T, k and H of an operator that takes no expert count.
int check_tokens(int T, int k, int H, int dtype) {
  if (int rc = check_route_args(T, MOE_MAX_EXPERTS, k)) return rc;
  if (int rc = check_row("H", H)) return rc;
  return check_dtype(dtype);
}

int quantize(const char* name, bool silu, const void* x, int dtype, int64_t x_stride, int M, int K,
             const int32_t* n_rows, uint8_t* q, int64_t q_stride, float* scales, void* stream) {
  clear_error();
  if (int rc = check_dtype(dtype)) return rc;
  if (int rc = check_row("K", K)) return rc;
  if (M < 0) return set_error(MOE_EINVAL, "M=%d < 0", M);
  if (M > kMaxRows || static_cast<int64_t>(M) * K > (int64_t{1} << 39))
    return set_error(MOE_EUNSUPPORTED, "M=%d rows of %d columns: M <= %d and M * K <= 2^39", M, K, kMaxRows);
  if (int rc = check_stride("x", x_stride, silu ? 2 * static_cast<int64_t>(K) : K)) return rc;
  if (int rc = check_stride("q", q_stride, K)) return rc;
  if (M == 0) return MOE_OK;
  if (!x || !q || !scales) return set_error(MOE_EINVAL, "NULL pointer argument");
  if (int rc = check_align("x", x, dtype)) return rc;
  return launch_fp8_quantize(name, silu, x, dtype, x_stride, M, K, n_rows, q, q_stride, scales,
                             static_cast<hipStream_t>(stream));
}

}  // namespace
}  // namespace moeapq

using namespace moeapq;

extern "C" {

int moe_permute_tokens(const void* x, int dtype, int64_t x_stride, int T, int k, int E, int H,
                       const int32_t* topk_ids, const int32_t* expert_offsets, const int32_t* sorted_pairs,
                       void* x_sorted, int64_t xs_stride, int32_t* pair_rows, void* stream) {
  clear_error();
  if (int rc = check_route_args(T, E, k)) return rc;
  if (int rc = check_row("H", H)) return rc;
  if (int rc = check_dtype(dtype)) return rc;
  if (int rc = check_stride("x", x_stride, H)) return rc;
  if (int rc = check_stride("x_sorted", xs_stride, H)) return rc;
  if (T == 0) return MOE_OK;
  if (!x || !topk_ids || !expert_offsets || !sorted_pairs || !x_sorted || !pair_rows)
    return set_error(MOE_EINVAL, "NULL pointer argument");
  if (int rc = check_align("x", x, dtype)) return rc;
  if (int rc = check_align("x_sorted", x_sorted, dtype)) return rc;
  return launch_permute_tokens(x, dtype, x_stride, T, k, E, H, topk_ids, expert_offsets, sorted_pairs, x_sorted,
                               xs_stride, pair_rows, static_cast<hipStream_t>(stream));
}

int moe_permute_tokens_backward(const void* dx_sorted, int dtype, int64_t dxs_stride, int T, int k, int H,
                                const int32_t* pair_rows, void* dx, int64_t dx_stride, void* stream) {
  clear_error();
  if (int rc = check_tokens(T, k, H, dtype)) return rc;
  if (int rc = check_stride("dx_sorted", dxs_stride, H)) return rc;
  if (int rc = check_stride("dx", dx_stride, H)) return rc;
  if (T == 0) return MOE_OK;
  if (!dx_sorted || !pair_rows || !dx) return set_error(MOE_EINVAL, "NULL pointer argument");
  if (int rc = check_align("dx_sorted", dx_sorted, dtype)) return rc;
  if (int rc = check_align("dx", dx, dtype)) return rc;
  return launch_combine_rows("permute_tokens_backward", dx_sorted, dtype, dxs_stride, T, k, H, pair_rows, nullptr,
                             nullptr, 0, dx, dx_stride, static_cast<hipStream_t>(stream));
}

int moe_unpermute_tokens(const void* y_sorted, int dtype, int64_t ys_stride, int T, int k, int H,
                         const int32_t* pair_rows, const float* gates, const void* add, int64_t add_stride,
                         void* y, int64_t y_stride, void* stream) {
  clear_error();
  if (int rc = check_tokens(T, k, H, dtype)) return rc;
  if (int rc = check_stride("y_sorted", ys_stride, H)) return rc;
  if (int rc = check_stride("y", y_stride, H)) return rc;
  if (add)
    if (int rc = check_stride("add", add_stride, H)) return rc;
  if (T == 0) return MOE_OK;
  if (!y_sorted || !pair_rows || !y) return set_error(MOE_EINVAL, "NULL pointer argument");
  if (int rc = check_align("y_sorted", y_sorted, dtype)) return rc;
  if (int rc = check_align("add", add, dtype)) return rc;
  if (int rc = check_align("y", y, dtype)) return rc;
  return launch_combine_rows("unpermute_tokens", y_sorted, dtype, ys_stride, T, k, H, pair_rows, gates, add,
                             add_stride, y, y_stride, static_cast<hipStream_t>(stream));
}

int moe_unpermute_tokens_backward(const void* dy, int dtype, int64_t dy_stride, const void* y_sorted,
                                  int64_t ys_stride, int T, int k, int H, const int32_t* pair_rows,
                                  const float* gates, void* dy_sorted, int64_t dys_stride, float* dgates,
                                  void* stream) {
  clear_error();
  if (int rc = check_tokens(T, k, H, dtype)) return rc;
  if (int rc = check_stride("dy", dy_stride, H)) return rc;
  if (dgates)
    if (int rc = check_stride("y_sorted", ys_stride, H)) return rc;
  if (dy_sorted)
    if (int rc = check_stride("dy_sorted", dys_stride, H)) return rc;
  if (T == 0) return MOE_OK;
  if (!dy || !pair_rows || (dgates && !y_sorted) || (!dy_sorted && !dgates))
    return set_error(MOE_EINVAL, "NULL pointer argument");
  if (int rc = check_align("dy", dy, dtype)) return rc;
  if (int rc = check_align("y_sorted", y_sorted, dtype)) return rc;
  if (int rc = check_align("dy_sorted", dy_sorted, dtype)) return rc;
  return launch_combine_rows_grad(dy, dtype, dy_stride, y_sorted, ys_stride, T, k, H, pair_rows, gates, dy_sorted,
                                  dys_stride, dgates, static_cast<hipStream_t>(stream));
}

int moe_fp8_quantize(const void* x, int dtype, int64_t x_stride, int M, int K, const int32_t* n_rows,
                     uint8_t* q, int64_t q_stride, float* scales, void* stream) {
  return quantize("fp8_quantize", false, x, dtype, x_stride, M, K, n_rows, q, q_stride, scales, stream);
}

int moe_fp8_quantize_silu(const void* x, int dtype, int64_t x_stride, int M, int K, const int32_t* n_rows,
                          uint8_t* q, int64_t q_stride, float* scales, void* stream) {
  return quantize("fp8_quantize_silu", true, x, dtype, x_stride, M, K, n_rows, q, q_stride, scales, stream);
}

int moe_fp8_gemm(const uint8_t* a, int64_t lda, const float* a_scales, int a_rows, const uint8_t* w,
                 const float* w_scales, int E, int M, int N, int K, const int32_t* expert_offsets,
                 const int32_t* sorted_pairs, int k, void* c, int dtype, int64_t ldc, void* stream) {
  clear_error();
  if (int rc = check_dtype(dtype)) return rc;
  if (E <= 0 || M < 0) return set_error(MOE_EINVAL, "need E > 0 and M >= 0 (E=%d M=%d)", E, M);
  if (E > MOE_MAX_EXPERTS || M > kMaxRows)
    return set_error(MOE_EUNSUPPORTED, "outside bounds: E<=%d, M<=%d (got E=%d M=%d)", MOE_MAX_EXPERTS, kMaxRows, E, M);
  if (int rc = check_row("N", N)) return rc;
  if (int rc = check_row("K", K)) return rc;
  if (K % 16) return set_error(MOE_EUNSUPPORTED, "need K %% 16 == 0 (K=%d)", K);
  if (int rc = check_stride("a", lda, K)) return rc;
  if (lda % 16 || lda > (1 << 24))
    return set_error(MOE_EUNSUPPORTED, "need lda %% 16 == 0 and lda <= 2^24 (lda=%lld)", static_cast<long long>(lda));
  if (int rc = check_stride("c", ldc, N)) return rc;
  if (!expert_offsets && E != 1) return set_error(MOE_EINVAL, "E=%d groups need expert_offsets", E);
  if (M == 0) return MOE_OK;
  if (!a || !a_scales || !w || !w_scales || !c) return set_error(MOE_EINVAL, "NULL pointer argument");
  if (a_rows <= 0 || a_rows > kMaxRows || (!sorted_pairs && a_rows < M))
    return set_error(MOE_EINVAL, "a has %d rows for M=%d", a_rows, M);
  if (sorted_pairs && (k <= 0 || k > MOE_MAX_TOPK))
    return set_error(MOE_EINVAL, "k=%d outside 1..%d", k, MOE_MAX_TOPK);
  if (sorted_pairs && a_rows * lda >= (int64_t{1} << 32))
    return set_error(MOE_EUNSUPPORTED, "gathered rows of a must lie within 4 GiB (%d rows of stride %lld)", a_rows,
                     static_cast<long long>(lda));
  if ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(w)) & 15)
    return set_error(MOE_EINVAL, "a and w must be 16-byte aligned");
  if (int rc = check_align("c", c, dtype)) return rc;
  return launch_fp8_gemm(a, lda, a_scales, a_rows, w, w_scales, E, M, N, K, expert_offsets, sorted_pairs, k, c, dtype,
                         ldc, static_cast<hipStream_t>(stream));
}

}  // extern "C"
