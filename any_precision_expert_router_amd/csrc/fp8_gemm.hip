// Matrix product in e4m3 with an fp32 scale for each block of 128, grouped by expert or plain:
//
//   c[i][n] = sum_b sa[r_i][b] sw[e][n/128][b] sum_{kk in block b} a[r_i][kk] w[e][n][kk]
//
// for the rows i of expert e's group, r_i = i or pairs[i] / k.  One 16x16x128 matrix instruction
// covers one block of 16 weight rows and 16 rows of a: its fp32 result is exact up to fp32
// accumulation, and is added to the fp32 accumulator with the product of the two scales, one FMA
// per element and block.
//
// Operand layout.  The weights are the instruction's A side (rows), a its B side (columns), so a
// lane's four results are four neighbouring columns n of one row i of c and its scale sa is one
// value.  The order of the 128 products inside a block does not matter, so lane (r, g) = (l % 16,
// l / 16) simply takes the 16-byte pieces g and g + 4 of its row's block on both sides.
#include <type_traits>

#include "elements.hpp"
#include "internal.hpp"
#include "wave_ops.hpp"

namespace moeapq {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kBlock = MOE_FP8_BLOCK;

struct GemmArgs {
  const uint8_t* a;
  int64_t lda;
  const float* a_scales;
  int a_rows;
  const uint8_t* w;
  const float* w_scales;
  int E, M, N, K, kb, nb;           // kb = blocks of K, nb = blocks of N
  const int32_t* offsets;           // [E+1] or null (one group of M rows)
  const int32_t* pairs;             // null: rows of a in place
  int k;
  void* c;
  int64_t ldc;
};

// ---- tiles of the groups ---------------------------------------------------------------------
// The rows of group e are cut into tiles of BM rows; a tile of c is (row tile, column tile), and
// all tiles are numbered group by group, inside a group column tile by column tile with the row
// tiles of one column tile side by side (they share its weights).
struct Tile {
  int e, first, rows, col_tile;     // rows <= 0: no tile
};

// Rows of group e (0 for e >= E) and the first of them, without a branch.
__device__ __forceinline__ int group_rows(const GemmArgs& g, int e, int& first) {
  const int lo = g.offsets[min(e, g.E)], hi = g.offsets[min(e + 1, g.E)];
  first = min(max(lo, 0), g.M);
  return max(min(max(hi, 0), g.M) - first, 0);
}

// Workgroups go round the 8 dies in turn, so the tiles are dealt out in 8 contiguous runs, one to
// a die: neighbouring tiles share weights or rows of a, which then are in that die's L2.
template <int BM>
__device__ __forceinline__ Tile find_tile(const GemmArgs& g, int col_tiles, uint32_t block) {
  const int lane = threadIdx.x & 63;
  Tile out{0, 0, 0, 0};
  int total = 0;
  if (g.offsets) {
    for (int e0 = 0; e0 < g.E; e0 += 64) {
      int first;
      const int n = group_rows(g, e0 + lane, first);
      total += lane_int(wave_inclusive_add((n + BM - 1) / BM), 63);
    }
  } else {
    total = (g.M + BM - 1) / BM;
  }
  const uint32_t tiles = static_cast<uint32_t>(total) * col_tiles;
  const uint32_t per = (tiles + 7) / 8;
  if (block / 8 >= per) return out;
  uint32_t t = (block % 8) * per + block / 8;
  if (t >= tiles) return out;
  if (!g.offsets) {
    out.col_tile = t / total;
    out.first = static_cast<int>(t % total) * BM;
    out.rows = min(g.M - out.first, BM);
    return out;
  }
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int first;
    const int n = group_rows(g, e0 + lane, first);
    const int mt = (n + BM - 1) / BM;
    const int upto = wave_inclusive_add(mt);
    const uint32_t all = static_cast<uint32_t>(lane_int(upto, 63)) * col_tiles;
    if (t < all) {
      const uint64_t hit = __ballot(static_cast<uint32_t>(upto) * col_tiles > t);
      const int l = __builtin_ctzll(hit);
      const int mt_l = lane_int(mt, l);
      const uint32_t in = t - static_cast<uint32_t>(lane_int(upto, l) - mt_l) * col_tiles;
      const int m = in % mt_l;
      out.e = e0 + l;
      out.col_tile = in / mt_l;
      out.first = lane_int(first, l) + m * BM;
      out.rows = min(lane_int(n, l) - m * BM, BM);
      return out;
    }
    t -= all;
  }
  return out;
}

// Row of a behind row i of c.
__device__ __forceinline__ int64_t source_row(const GemmArgs& g, int i) {
  int r = i;
  if (g.pairs) r = g.pairs[i] / g.k;
  return min(max(r, 0), g.a_rows - 1);
}

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Eight e4m3 values as fp16 (exact).
__device__ __forceinline__ f16x8 widen(int lo, int hi) {
  const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
  const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
  const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
  const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One block's products of 16 weight rows and 16 rows of a.
//
// The e4m3 instruction does not add its 128 products in fp32: it brings them to the exponent of the
// largest and drops what lies below 2^-13 of it (a second product of 2^-13 of the first survives,
// one of 2^-14 is lost).  On normal data that is a relative error of 1.5e-5, far below a 16-bit
// result's rounding (2.1e-4 for fp16, 1.7e-3 for bf16), so 16-bit results take it.  For fp32
// results (FINE) both sides are widened to fp16, which holds every e4m3 value, and the fp16
// instruction adds in fp32: 3e-8, at half the matrix rate.
template <bool FINE>
__device__ __forceinline__ f32x4 mfma_block(const i32x8& w, const i32x8& a) {
  if (!FINE) return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
  f32x4 p{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen(w[2 * i], w[2 * i + 1]), widen(a[2 * i], a[2 * i + 1]), p, 0, 0, 0);
  return p;
}

// The two 16-byte pieces g and g + 4 of one block of a row.  The last block of a row may be short:
// pieces behind the row's end are read from its start and zeroed.
template <bool TAIL>
__device__ __forceinline__ i32x8 load_pieces(const uint8_t* row, int kb, int K, int piece) {
  union {
    u32x4 half[2];
    i32x8 all;
  } u;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = kb * kBlock + (piece + 4 * h) * 16;
    const bool in = !TAIL || at < K;
    u.half[h] = *reinterpret_cast<const u32x4*>(row + (in ? at : 0));
    if (TAIL && !in) u.half[h] = u32x4{0, 0, 0, 0};
  }
  return u.all;
}

constexpr int kStreamThreads = 256;
constexpr int kStreamWaves = kStreamThreads / 64;

// Few rows: the weights go straight from memory into registers, the four wavefronts of a workgroup
// take every fourth block of K and add their results up at the end.
template <int MT, int NT, int DT>
__global__ __launch_bounds__(kStreamThreads) void fp8_gemm_stream_kernel(GemmArgs g, int col_tiles) {
  constexpr int BM = MT * 16, BN = NT * 16;
  __shared__ float part[kStreamWaves - 1][BN][BM + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, piece = lane >> 4;
  const Tile tile = find_tile<BM>(g, col_tiles, blockIdx.x);
  if (tile.rows <= 0) return;
  const int n0 = tile.col_tile * BN;
  const uint8_t* w_row[NT];
  const uint8_t* a_row[MT];
  const float* a_scale[MT];
#pragma unroll
  for (int j = 0; j < NT; ++j)
    w_row[j] = g.w + (static_cast<int64_t>(tile.e) * g.N + min(n0 + j * 16 + r, g.N - 1)) * g.K;
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t src = source_row(g, tile.first + min(i * 16 + r, tile.rows - 1));
    a_row[i] = g.a + src * g.lda;
    a_scale[i] = g.a_scales + src * g.kb;
  }
  const float* w_scale = g.w_scales + (static_cast<int64_t>(tile.e) * g.nb + n0 / kBlock) * g.kb;
  f32x4 acc[NT][MT] = {};
  auto step = [&](auto tail, int kb) {
    constexpr bool TAIL = decltype(tail)::value;
    i32x8 w[NT], a[MT];
    float s[MT];
    const float sw = w_scale[kb];
#pragma unroll
    for (int j = 0; j < NT; ++j) w[j] = load_pieces<TAIL>(w_row[j], kb, g.K, piece);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      a[i] = load_pieces<TAIL>(a_row[i], kb, g.K, piece);
      s[i] = a_scale[i][kb];
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      s[i] *= sw;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 p = mfma_block<DT == MOE_DTYPE_F32>(w[j], a[i]);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[j][i][v] = fmaf(p[v], s[i], acc[j][i][v]);
      }
    }
  };
  const int full = g.K / kBlock;
  for (int kb = wave; kb < full; kb += kStreamWaves) step(std::false_type{}, kb);
  if (full < g.kb && full % kStreamWaves == wave) step(std::true_type{}, full);
  // results of wavefronts 1-3 through LDS, added by wavefront 0 in their order
  if (wave > 0) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) part[wave - 1][j * 16 + piece * 4 + v][i * 16 + r] = acc[j][i][v];
  }
  __syncthreads();
  if (wave > 0) return;
  using T = typename Elem<DT>::T;
  T* c = static_cast<T*>(g.c);
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = i * 16 + r;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int n = n0 + j * 16 + piece * 4 + v;
        float sum = acc[j][i][v];
#pragma unroll
        for (int p = 0; p < kStreamWaves - 1; ++p) sum += part[p][j * 16 + piece * 4 + v][m];
        if (m < tile.rows && n < g.N) c[static_cast<int64_t>(tile.first + m) * g.ldc + n] = static_cast<T>(sum);
      }
  }
}

template <int MT, int NT>
int launch_stream(const GemmArgs& g, int dtype, hipStream_t stream) {
  constexpr int BM = MT * 16, BN = NT * 16;
  const int col_tiles = (g.N + BN - 1) / BN;
  // at most one partly filled row tile per group with rows
  const int64_t row_tiles = (static_cast<int64_t>(g.M) + BM - 1) / BM + (g.offsets ? min(g.E, g.M) : 0);
  const uint64_t blocks = (static_cast<uint64_t>(row_tiles) * col_tiles + 7) / 8 * 8;
  if (blocks >> 31) return set_error(MOE_EUNSUPPORTED, "moe_fp8_gemm: %llu tiles are more than one launch takes",
                                     static_cast<unsigned long long>(blocks));
  ProfileScope prof("fp8_gemm", stream);
  with_dtype(dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    hipLaunchKernelGGL((fp8_gemm_stream_kernel<MT, NT, DT>), dim3(static_cast<uint32_t>(blocks)), dim3(kStreamThreads),
                       0, stream, g, col_tiles);
  });
  return check_launch("fp8_gemm");
}

}  // namespace

int launch_fp8_gemm(const uint8_t* a, int64_t lda, const float* a_scales, int a_rows, const uint8_t* w,
                    const float* w_scales, int E, int M, int N, int K, const int32_t* offsets, const int32_t* pairs,
                    int k, void* c, int dtype, int64_t ldc, hipStream_t stream) {
  const GemmArgs g{a, lda, a_scales, a_rows, w, w_scales, E, M, N, K, (K + kBlock - 1) / kBlock,
                   (N + kBlock - 1) / kBlock, offsets, pairs, k, c, ldc};
  if (M <= 16 * E) return launch_stream<1, 2>(g, dtype, stream);
  return launch_stream<2, 2>(g, dtype, stream);
}

}  // namespace moeapq
