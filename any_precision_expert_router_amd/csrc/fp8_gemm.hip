// Matrix product in e4m3 with an fp32 scale for each block of 128, grouped by expert or plain:
//
//   c[i][n] = sum_b sa[r_i][b] sw[e][n/128][b] sum_{kk in block b} a[r_i][kk] w[e][n][kk]
//
// for the rows i of expert e's group, r_i = i or pairs[i] / k.  One 16x16x128 matrix instruction
// covers one block of 16 weight rows and 16 rows of a; its result is added to the fp32 accumulator with
// the product of the two scales, one FMA per element and block (half the instruction's own time, and
// beside it: with four FMAs to a product two wavefronts per SIMD still reach 4.0 PFLOP/s).
//
// Operand layout.  The weights are the instruction's A side (rows), a its B side (columns), so a
// lane's four results are four neighbouring columns n of one row i of c and its scale sa is one
// value.  The order of the 128 products inside a block does not matter, so lane (r, g) = (l % 16,
// l / 16) simply takes the 16-byte pieces g and g + 4 of its row's block on both sides.
//
// Three forms, chosen in launch_gemm: many rows to a group, few rows with many tiles, few with few.
#include <cstddef>
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
// The n rows of a group are cut into ceil(n / bm) tiles of equal height (rounded up to 16 rows), so
// that no tile is nearly empty; a tile of c is (row tile, column tile), and all tiles are numbered
// group by group, inside a group column tile by column tile with the row tiles of one column tile side
// by side (they share its weights).
struct Tile {
  int e, first, rows, col_tile;     // rows <= 0: no tile
};

// Rows of group e (0 for e >= E) and the first of them, without a branch.
__device__ __forceinline__ int group_rows(const GemmArgs& g, int e, int& first) {
  const int lo = g.offsets[min(e, g.E)], hi = g.offsets[min(e + 1, g.E)];
  first = min(max(lo, 0), g.M);
  return max(min(max(hi, 0), g.M) - first, 0);
}

__device__ __forceinline__ int tile_height(int n, int tiles) { return (n + tiles * 16 - 1) / (tiles * 16) * 16; }

// Row tiles of all groups together.
__device__ __forceinline__ int count_row_tiles(const GemmArgs& g, int bm) {
  if (!g.offsets) return (g.M + bm - 1) / bm;
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int first;
    total += lane_int(wave_inclusive_add((group_rows(g, e0 + lane, first) + bm - 1) / bm), 63);
  }
  return total;
}

// Tile t < row_tiles * col_tiles; every lane of the wavefront takes part.
__device__ __forceinline__ Tile tile_at(const GemmArgs& g, int bm, int row_tiles, int col_tiles, uint32_t t) {
  Tile out{0, 0, 0, 0};
  if (!g.offsets) {
    const int high = tile_height(g.M, row_tiles);
    out.col_tile = t / row_tiles;
    out.first = static_cast<int>(t % row_tiles) * high;
    out.rows = min(g.M - out.first, high);
    return out;
  }
  const int lane = threadIdx.x & 63;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int first;
    const int n = group_rows(g, e0 + lane, first);
    const int mt = (n + bm - 1) / bm;
    const int upto = wave_inclusive_add(mt);
    const uint32_t all = static_cast<uint32_t>(lane_int(upto, 63)) * col_tiles;
    if (t < all) {
      const uint64_t hit = __ballot(static_cast<uint32_t>(upto) * col_tiles > t);
      const int l = __builtin_ctzll(hit);
      const int mt_l = lane_int(mt, l);
      const uint32_t in = t - static_cast<uint32_t>(lane_int(upto, l) - mt_l) * col_tiles;
      const int n_l = lane_int(n, l), from = static_cast<int>(in % mt_l) * tile_height(n_l, mt_l);
      out.e = e0 + l;
      out.col_tile = in / mt_l;
      out.first = lane_int(first, l) + from;
      out.rows = min(n_l - from, tile_height(n_l, mt_l));
      return out;
    }
    t -= all;
  }
  return out;
}

// Workgroups go round the 8 dies in turn, so the tiles are dealt out in 8 contiguous runs, one to
// a die: neighbouring tiles share weights or rows of a, which then are in that die's L2.  Die d has
// tiles [first, end); its workgroups take them in turn.
struct TileRun {
  uint32_t first, end;
};
__device__ __forceinline__ TileRun die_tiles(uint32_t tiles, uint32_t die) {
  const uint32_t per = (tiles + 7) / 8;
  return {die * per, min((die + 1) * per, tiles)};
}

// The same, dealt out by what the tiles cost instead of by their number, for tiles of different
// heights: in units of rows, a tile's own (in steps of 32, at least 64) plus 64 for the weights' part.
// Groups of 250 and of 260 rows differ by one 256-row tile against two of 144; by number, the dies that
// got the former had the longer run (64 experts, about 256 rows each: 428 us, 411 us by cost).
__device__ __forceinline__ int tile_cost(int n, int tiles) {
  return tiles > 0 ? max((tile_height(n, tiles) + 31) / 32 * 32, 64) + 64 : 0;
}

__device__ __forceinline__ int cost_row_tiles(const GemmArgs& g, int bm) {
  const int lane = threadIdx.x & 63;
  int total = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int first;
    const int n = group_rows(g, e0 + lane, first), mt = (n + bm - 1) / bm;
    total += lane_int(wave_inclusive_add(dpp_settled(mt * tile_cost(n, mt))), 63);
  }
  return total;
}

// First tile of die d's run; `cost` is cost_row_tiles().
__device__ __forceinline__ uint32_t die_start(const GemmArgs& g, int bm, int row_tiles, int cost, int col_tiles, int d) {
  const uint32_t tiles = static_cast<uint32_t>(row_tiles) * col_tiles;
  if (d >= 8) return tiles;
  if (!g.offsets) return static_cast<uint32_t>(static_cast<uint64_t>(tiles) * d / 8);
  const uint64_t target = static_cast<uint64_t>(cost) * col_tiles * d / 8;
  const int lane = threadIdx.x & 63;
  int tiles_before = 0, cost_before = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int first;
    const int n = group_rows(g, e0 + lane, first), mt = (n + bm - 1) / bm, each = tile_cost(n, mt);
    const int cost_upto = wave_inclusive_add(dpp_settled(mt * each)), upto = wave_inclusive_add(dpp_settled(mt));
    const int cost_all = cost_before + lane_int(cost_upto, 63);
    if (static_cast<uint64_t>(cost_all) * col_tiles > target) {
      const uint64_t hit = __ballot(static_cast<uint64_t>(cost_before + cost_upto) * col_tiles > target);
      const int l = __builtin_ctzll(hit), mt_l = lane_int(mt, l), each_l = lane_int(each, l);
      const uint64_t in = target - static_cast<uint64_t>(cost_before + lane_int(cost_upto, l) - mt_l * each_l) * col_tiles;
      return static_cast<uint32_t>(tiles_before + lane_int(upto, l) - mt_l) * col_tiles +
             static_cast<uint32_t>(in / static_cast<uint32_t>(each_l));
    }
    tiles_before += lane_int(upto, 63);
    cost_before = cost_all;
  }
  return tiles;
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

// One side of a block's products: 16 rows by 128, a lane's 32 bytes.
//
// The e4m3 instruction does not add its 128 products in fp32: it brings them to the exponent of the
// largest and drops what lies below 2^-13 of it (a second product of 2^-13 of the first survives,
// one of 2^-14 is lost).  On normal data that is a relative error of 1.5e-5, far below a 16-bit
// result's rounding (2.1e-4 for fp16, 1.7e-3 for bf16), so 16-bit results take it.  For fp32
// results (FINE) both sides are widened to fp16, which holds every e4m3 value, and the fp16
// instruction adds in fp32: 3e-8, at half the matrix rate.
template <bool FINE>
struct Side {
  i32x8 v;
  __device__ __forceinline__ explicit Side(const i32x8& x) : v(x) {}
};
template <>
struct Side<true> {
  f16x8 v[4];
  Side() = default;
  __device__ __forceinline__ explicit Side(const i32x8& x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = widen(x[2 * i], x[2 * i + 1]);
  }
};

__device__ __forceinline__ f32x4 mfma_block(const Side<false>& w, const Side<false>& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, a.v, f32x4{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_block(const Side<true>& w, const Side<true>& a) {
  f32x4 p{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[i], a.v[i], p, 0, 0, 0);
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

// ---- few rows, few tiles -----------------------------------------------------------------------
// Tiles of 16 or 32 columns, so that small products still fill the chip: the weights go straight from
// memory into registers, the four wavefronts of a workgroup take every fourth block of K and add their
// results up at the end, in a fixed order.  Reading the weights bounds it (two experts of 28672 x 4096,
// one row each: 44 us, 5.4 TB/s); neighbouring lanes hold different rows, so the vector cache takes an
// access for every 16 bytes, which is what caps larger products in this form.
template <int MT, int NT, int DT>
__global__ __launch_bounds__(kStreamThreads) void fp8_gemm_stream_kernel(GemmArgs g, int col_tiles) {
  constexpr int BM = MT * 16, BN = NT * 16;
  constexpr bool kFine = DT == MOE_DTYPE_F32;
  __shared__ float part[kStreamWaves - 1][BN][BM + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, piece = lane >> 4;
  const int row_tiles = count_row_tiles(g, BM);
  const TileRun run = die_tiles(static_cast<uint32_t>(row_tiles) * col_tiles, blockIdx.x % 8);
  const uint32_t t = run.first + blockIdx.x / 8;
  if (t >= run.end) return;
  const Tile tile = tile_at(g, BM, row_tiles, col_tiles, t);
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
      const Side<kFine> as(a[i]);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const f32x4 p = mfma_block(Side<kFine>(w[j]), as);
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

// ---- many rows ---------------------------------------------------------------------------------
// A workgroup of eight wavefronts, 2 by 4, holds a tile of up to 256 rows by 256 columns; each
// wavefront has half the rows and 64 columns.  Both sides go through LDS, two stages of one block
// each, filled by direct loads.  A wavefront holds its weights of a block in registers, so their
// stage is free again after a few matrix instructions and the block after the next is asked for
// then; rows of a (which other tiles keep in the die's L2) are asked for one block ahead.
//
// What bounds it: every CU draws (rows + 256) * 128 bytes of a block through its L2 path, about 36
// bytes per cycle and CU, for rows * 256 * 128 products.  128-row tiles need 1.5 times the traffic of
// 256-row ones for the same products.  (Weights are not loaded straight into registers: a matrix
// operand wants neighbouring lanes on different rows, and the vector cache then takes one access for
// every 16 bytes instead of one for 64.)
//
// 64 experts of 5120 x 3584 with about 256 rows each: 411 us, 1.46 PFLOP/s (about 330 us without the loads,
// 290 without the products: two stages overlap them only in part).  777 rows by 11264 x 2048 in fp32:
// 48 us, 0.75 PFLOP/s.
constexpr int kTileThreads = 512, kTileWaves = kTileThreads / 64;
constexpr int kTileN = 256, kWaveN = 4;      // kWaveN: 16-column pieces of a wavefront
// Rows of the highest tile.  Accumulators fill half the registers; widening to fp16 needs the rest
// for the weights.
template <int DT>
constexpr int kTileM = DT == MOE_DTYPE_F32 ? 160 : 256;

#define MOE_LDS __attribute__((address_space(3)))

// 16 bytes per lane from rsrc + offset + uniform into LDS at lds_addr + 16 * lane.  The buffer form:
// the compiler takes the global one for a flat access and waits for every load in flight.
__device__ __forceinline__ void lds_load16(uint32_t lds_addr, __amdgpu_buffer_rsrc_t rsrc, uint32_t offset,
                                           uint32_t uniform) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (MOE_LDS void*)static_cast<uintptr_t>(lds_addr), 16, offset, uniform,
                                           0, 0);
}

// The scales of a and of the weights for kScaleBlocks blocks at a time, a row's fetched together: one
// value per row and block would take as many L2 requests as half the weights do.
constexpr int kScaleBlocks = 28, kScalePitch = kScaleBlocks + 1;   // odd: 16 rows' scales are in 16 banks

template <int BM>
struct TileLds {
  uint8_t a[2][BM * kBlock];
  uint8_t w[2][kTileN * kBlock];
  float a_scale[BM][kScalePitch];
  float w_scale[2][kScaleBlocks];   // of the tile's two 128-column halves
};

// A lane value the compiler recomputes addresses from instead of keeping them.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}

// What a wavefront loads of a tile: 1 KiB = 8 rows of a stage with each direct load, every eighth of
// them.  A stage's row is 128 bytes in 16-byte slots.  Row m of a has its piece c in slot c ^ (m % 8).
// The weights' rows are dealt to the lanes so that a lane's results are neighbouring columns; row n of
// them has its piece c in slot c ^ (n % 4 + 4 (n / (4 COLS) % 2)).  Either way the 16 rows of a fragment
// read their pieces from all banks (slot c ^ (r % 8)).
// Offsets are 32 bits: of the weights from the tile's first row, of a from the tile's first row or
// from its start if rows are gathered (the entry point keeps those below 4 GiB).
//
// COLS: 16-column pieces of a wavefront.  Its lane r of piece j is column 4 COLS (r / 4) + 4 j + r % 4.
template <int BM, int COLS>
struct Loader {
  static constexpr int kA = (BM / 8 + kTileWaves - 1) / kTileWaves, kW = kTileN / 8 / kTileWaves;
  __amdgpu_buffer_rsrc_t a_rsrc, w_rsrc;
  uint32_t a_off[kA], w_off[kW];
  uint32_t a_at, w_at;

  __device__ __forceinline__ static int lane() { return threadIdx.x & 63; }
  __device__ __forceinline__ static int wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }
  __device__ __forceinline__ static uint32_t a_chunk() { return ((lane() & 7) ^ (lane() >> 3)) * 16; }
  __device__ __forceinline__ static uint32_t w_chunk() {
    static_assert(COLS == 2 || COLS == 4, "4 COLS is 8 or 16 rows: one or two wavefronts' parts");
    return ((lane() & 7) ^ ((lane() >> 3 & 3) | ((COLS == 4 ? wave() >> 1 : wave()) & 1) << 2)) * 16;
  }

  __device__ __forceinline__ void aim(const GemmArgs& g, const Tile& tile) {
    const int nt0 = tile.col_tile * kTileN, sub = lane() >> 3;
    w_rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.w + (static_cast<int64_t>(tile.e) * g.N + nt0) * g.K),
                                               0, -1, 0x00027000);
#pragma unroll
    for (int q = 0; q < kW; ++q)
      w_off[q] = static_cast<uint32_t>(min((q * kTileWaves + wave()) * 8 + sub, g.N - 1 - nt0)) * g.K + w_chunk();
    const int64_t base = g.pairs ? 0 : source_row(g, tile.first);
    a_rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(g.a + base * g.lda), 0, -1, 0x00027000);
#pragma unroll
    for (int q = 0; q < kA; ++q) {
      const int m = min((q * kTileWaves + wave()) % (BM / 8) * 8 + sub, tile.rows - 1);
      a_off[q] = static_cast<uint32_t>((source_row(g, tile.first + m) - base) * g.lda) + a_chunk();
    }
  }
  // Direct load q of a stage, from column `uniform` + `more` on.
  __device__ __forceinline__ void load_a(int q, int stage, uint32_t uniform, uint32_t more = 0) const {
    const int part = (q * kTileWaves + wave()) % (BM / 8);   // some parts twice, the same bytes, if BM is not 64 n
    lds_load16(a_at + stage * (BM * kBlock) + part * 1024, a_rsrc, a_off[q] + more, uniform);
  }
  __device__ __forceinline__ void load_w(int q, int stage, uint32_t uniform, uint32_t more = 0) const {
    lds_load16(w_at + stage * (kTileN * kBlock) + (q * kTileWaves + wave()) * 1024, w_rsrc, w_off[q] + more, uniform);
  }
};

// Scales of blocks [kb, kb + kScaleBlocks) into LDS ([row][block] of a, [half][block] of the weights);
// the caller waits and synchronises.  In assembly, since the compiler would hold plain LDS stores
// until every direct load has landed.
template <int BM>
__device__ __forceinline__ void store_scales(const GemmArgs& g, const Tile& tile, int kb, uint32_t a_to, uint32_t w_to) {
  constexpr int kEach = (BM * kScaleBlocks + kTileThreads - 1) / kTileThreads, kGroup = kEach % 7 ? kEach : 7;
  const int tid = opaque(threadIdx.x);   // nothing of this is kept in registers between chunks
  const int n = g.kb - kb;
#pragma unroll
  for (int i0 = 0; i0 < kEach; i0 += kGroup) {
    float v[kGroup];
    uint32_t to[kGroup];
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      const int x = min(tid + (i0 + i) * kTileThreads, BM * kScaleBlocks - 1), row = x / kScaleBlocks, b = x % kScaleBlocks;
      v[i] = g.a_scales[source_row(g, tile.first + min(row, tile.rows - 1)) * g.kb + kb + min(b, n - 1)];
      to[i] = a_to + (row * kScalePitch + b) * 4;
    }
#pragma unroll
    for (int i = 0; i < kGroup; ++i) asm volatile("ds_write_b32 %0, %1" : : "v"(to[i]), "v"(v[i]) : "memory");
  }
  if (tid < 2 * kScaleBlocks) {
    const int half = tid / kScaleBlocks, i = tid % kScaleBlocks, nb = min(tile.col_tile * (kTileN / kBlock) + half, g.nb - 1);
    const float w = g.w_scales[(static_cast<int64_t>(tile.e) * g.nb + nb) * g.kb + kb + min(i, n - 1)];
    asm volatile("ds_write_b32 %0, %1" : : "v"(w_to + tid * 4), "v"(w) : "memory");
  }
}

// Results of 16 rows (lane r's row is `m`) and COLS pieces: a lane's 4 COLS neighbouring columns, from n on.
template <int COLS, int DT>
__device__ __forceinline__ void store_row(const GemmArgs& g, const Tile& tile, int m, int n, const f32x4 (&acc)[COLS]) {
  using T = typename Elem<DT>::T;
  constexpr int kVec = kPerVec<DT>;
  if (m >= tile.rows) return;
  T* row = static_cast<T*>(g.c) + static_cast<int64_t>(tile.first + m) * g.ldc + n;
#pragma unroll
  for (int q = 0; q < 4 * COLS / kVec; ++q) {
    float v[kVec];
#pragma unroll
    for (int x = 0; x < kVec; ++x) v[x] = acc[(q * kVec + x) / 4][(q * kVec + x) % 4];
    if (n + q * kVec < g.N) store_elems<DT>(row + q * kVec, g.N - n - q * kVec, v);
  }
}

// A tile's first block and the weights of its second: multiplying starts with these on their way.
template <int BM>
__device__ __forceinline__ void start_tile(const GemmArgs& g, const Loader<BM, kWaveN>& from) {
  const int full = g.K / kBlock;
  if (full == 0) return;
#pragma unroll
  for (int q = 0; q < from.kW; ++q) from.load_w(q, 0, 0);
#pragma unroll
  for (int q = 0; q < from.kA; ++q) from.load_a(q, 0, 0);
#pragma unroll
  for (int q = 0; q < from.kW; ++q) from.load_w(q, 1, min(1, full - 1) * kBlock);
}

// One tile whose first loads are on their way; leaves those of `next` (if it has rows) on theirs.
// TM: pieces of 16 rows of one wavefront.
template <int TM, int DT>
__device__ __forceinline__ void gemm_tile(const GemmArgs& g, const Tile& tile, const Tile& next, Loader<kTileM<DT>, kWaveN>& from,
                                          TileLds<kTileM<DT>>& lds) {
  constexpr bool kFine = DT == MOE_DTYPE_F32;
  constexpr int BM = kTileM<DT>;
  using Lds = TileLds<BM>;
  using Op = Side<kFine>;
  // direct loads of a block: 4 TM parts of 8 rows of a, 32 of the weights, among eight wavefronts
  constexpr int kDmaA = (TM + 1) / 2, kDmaW = Loader<BM, kWaveN>::kW;
  // products after which the block's weights are in registers everywhere, and the next one's are read
  constexpr int kSteps = TM * kWaveN, kLag = 2, kRelease = kWaveN, kNextW = kSteps - kWaveN;
  static_assert(kDmaA <= Loader<BM, kWaveN>::kA && kDmaA <= kRelease && kRelease + kDmaW <= kSteps,
                "loads of a block fit between its products");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int r = lane & 15, piece = lane >> 4;
  const int nt0 = tile.col_tile * kTileN, n0 = nt0 + wn * 16 * kWaveN, m0 = wm * 16 * TM;
  auto scales = [&](int kb) {
    store_scales<BM>(g, tile, kb, from.a_at + static_cast<uint32_t>(offsetof(Lds, a_scale)),
                     from.a_at + static_cast<uint32_t>(offsetof(Lds, w_scale)));
  };

  f32x4 acc[TM][kWaveN] = {};
  // this lane's first piece of a fragment; the other is at ^ 64
  const int slot = (piece ^ (r & 7)) << 4;
  const int a_frag = (m0 + r) * kBlock + slot, w_frag = (wn * 16 * kWaveN + (r >> 2) * 16 + (r & 3)) * kBlock + slot;
  union Piece {
    u32x4 half[2];
    i32x8 all;
  };
  auto read = [&](const uint8_t* side, int at) {
    Piece u;
    u.half[0] = *reinterpret_cast<const u32x4*>(side + at);
    u.half[1] = *reinterpret_cast<const u32x4*>(side + (at ^ 64));
    return u;
  };
  i32x8 wv[kWaveN];   // the block's weights
  auto read_w = [&](int stage, int j) { wv[j] = read(&lds.w[stage][j * 4 * kBlock], w_frag).all; };
  // One block.  The next piece of a is read one row step ahead and results are added two matrix
  // instructions after theirs, so that neither is waited for; `between(n)` comes after product n: the
  // loads of the blocks to come, and the next block's weights in place of these after their last use.
  auto multiply = [&](int kb, int stage, auto&& between) {
    const float* f = &lds.a_scale[m0 + r][kb % kScaleBlocks];
    const float sw = lds.w_scale[wn >> 1][kb % kScaleBlocks];
    auto read_a = [&](int i) { return read(&lds.a[stage][i * 16 * kBlock], a_frag).all; };
    i32x8 a[2];
    float s[2], a_scale[2];
    f32x4 p[kLag + 1];
    a[0] = read_a(0);
    a_scale[0] = f[0];
    std::conditional_t<kFine, Op, int> wide[kWaveN];
    if constexpr (kFine) {
#pragma unroll
      for (int j = 0; j < kWaveN; ++j) wide[j] = Op(wv[j]);
    }
    Op op(a[0]);
    auto add = [&](int n) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        acc[n / kWaveN][n % kWaveN][v] = fmaf(p[n % (kLag + 1)][v], s[n / kWaveN & 1], acc[n / kWaveN][n % kWaveN][v]);
    };
#pragma unroll
    for (int n = 0; n < kSteps; ++n) {
      const int i = n / kWaveN, j = n % kWaveN;
      if (j == 0) {
        op = Op(a[i & 1]);
        if (i + 1 < TM) {
          a[(i + 1) & 1] = read_a(i + 1);
          a_scale[(i + 1) & 1] = f[(i + 1) * 16 * kScalePitch];
        }
      }
      if (j == kLag) s[i & 1] = a_scale[i & 1] * sw;   // first used for the product kLag back: this row step's first
      if constexpr (kFine)
        p[n % (kLag + 1)] = mfma_block(wide[j], op);
      else
        p[n % (kLag + 1)] = mfma_block(Op(wv[j]), op);
      __builtin_amdgcn_sched_barrier(0);
      between(n);
      if (n >= kLag) add(n - kLag);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int n = kSteps - kLag; n < kSteps; ++n) add(n);
  };

  const int full = g.K / kBlock, last = full - 1;
  if (full > 0) {
    for (int kb = 0; kb <= last; ++kb) {
      if (kb % kScaleBlocks == 0) {
        if (kb > 0) {   // every wavefront is through with the scales that are replaced
          asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
          __builtin_amdgcn_s_barrier();
        }
        scales(kb);
      }
      // this block has landed (the next one's weights may be in flight), and every wavefront is through
      // with the stage that the next one's rows of a go to
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(kDmaW) : "memory");
      __builtin_amdgcn_s_barrier();
      const int stage = kb & 1, next_a = min(kb + 1, last) * kBlock, next_w = min(kb + 2, last) * kBlock;
      if (kb == 0) {
#pragma unroll
        for (int j = 0; j < kWaveN; ++j) read_w(0, j);
      }
      multiply(kb, stage, [&](int n) {
        if (n < kDmaA) from.load_a(n, stage ^ 1, next_a);
        if (n == kRelease) {   // every wavefront holds its weights of this block
          asm volatile("" : : : "memory");
          __builtin_amdgcn_s_barrier();
        }
        if (n >= kRelease && n < kRelease + kDmaW) from.load_w(n - kRelease, stage, next_w);
        if (n == kNextW - 1) {   // the next block's weights have landed everywhere
          asm volatile("s_waitcnt vmcnt(%0)" : : "n"(kDmaA + (kNextW > kRelease ? kDmaW : 0)) : "memory");
          __builtin_amdgcn_s_barrier();
        }
        if (n >= kNextW) read_w(stage ^ 1, n - kNextW);
      });
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");   // the last stages' loads
    __builtin_amdgcn_s_barrier();
  }
  // A short last block, not overlapped.  Its pieces behind the row's end are read from the block's start;
  // the weights are taken as zero there (a row of a that holds NaN gives NaN anyway).
  if (full < g.kb) {
    const uint32_t left = g.K - full * kBlock;
    if (full % kScaleBlocks == 0) scales(full);
#pragma unroll
    for (int q = 0; q < kDmaW; ++q) from.load_w(q, 0, full * kBlock, from.w_chunk() < left ? 0 : -from.w_chunk());
#pragma unroll
    for (int q = 0; q < kDmaA; ++q) from.load_a(q, 0, full * kBlock, from.a_chunk() < left ? 0 : -from.a_chunk());
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int j = 0; j < kWaveN; ++j) {
      Piece u = read(&lds.w[0][j * 4 * kBlock], w_frag);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((piece + 4 * h) * 16 >= left) u.half[h] = u32x4{0, 0, 0, 0};
      wv[j] = u.all;
    }
    multiply(full, 0, [](int) {});
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    __builtin_amdgcn_s_barrier();
  }

  // The next tile's loads go out before this one's results.
  if (next.rows > 0) {
    from.aim(g, next);
    start_tile(g, from);
  }

#pragma unroll
  for (int i = 0; i < TM; ++i) store_row<kWaveN, DT>(g, tile, m0 + i * 16 + r, n0 + piece * 4 * kWaveN, acc[i]);
}

template <int DT>
__global__ __launch_bounds__(kTileThreads, 2) void fp8_gemm_tile_kernel(GemmArgs g, int bm, int col_tiles) {
  constexpr int BM = kTileM<DT>;
  __shared__ __align__(1024) TileLds<BM> lds;
  const int row_tiles = count_row_tiles(g, bm);
  const int die = blockIdx.x % 8, cost = g.offsets ? cost_row_tiles(g, bm) : 0;
  const TileRun run{die_start(g, bm, row_tiles, cost, col_tiles, die), die_start(g, bm, row_tiles, cost, col_tiles, die + 1)};
  uint32_t t = run.first + blockIdx.x / 8;
  if (t >= run.end) return;
  Loader<BM, kWaveN> from;
  from.a_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((MOE_LDS uint8_t*)&lds.a[0][0]));
  from.w_at = from.a_at + static_cast<uint32_t>(offsetof(TileLds<BM>, w));
  Tile tile = tile_at(g, bm, row_tiles, col_tiles, t);
  from.aim(g, tile);
  start_tile(g, from);
  while (tile.rows > 0) {
    t += gridDim.x / 8;
    Tile next{0, 0, 0, 0};
    if (t < run.end) next = tile_at(g, bm, row_tiles, col_tiles, t);
    if constexpr (BM >= 256) {
      if (tile.rows > 224) gemm_tile<8, DT>(g, tile, next, from, lds);
      else if (tile.rows > 192) gemm_tile<7, DT>(g, tile, next, from, lds);
      else if (tile.rows > 160) gemm_tile<6, DT>(g, tile, next, from, lds);
    }
    if (tile.rows <= 64) gemm_tile<2, DT>(g, tile, next, from, lds);
    else if (tile.rows <= 96) gemm_tile<3, DT>(g, tile, next, from, lds);
    else if (tile.rows <= 128) gemm_tile<4, DT>(g, tile, next, from, lds);
    else if (tile.rows <= 160) gemm_tile<5, DT>(g, tile, next, from, lds);
    tile = next;
  }
}

// ---- few rows to a group, many weights ----------------------------------------------------------
// Tiles of up to 32 rows by 256 columns, each of the eight wavefronts all rows by 32 columns.  The
// weights are read once and bound it, so the stages are small enough for kFewStages of them and the
// loads run kFewStages - 1 blocks ahead.  64 experts of 5120 x 3584 with 16 rows each: 204 us, 5.8 TB/s of
// the 6.35 a pure read reaches.
constexpr int kFewM = 32, kFewStages = 4, kFewN = 2;

struct FewLds {
  uint8_t a[kFewStages][kFewM * kBlock];
  uint8_t w[kFewStages][kTileN * kBlock];
  float a_scale[kFewM][kScalePitch];
  float w_scale[2][kScaleBlocks];
};
using FewLoader = Loader<kFewM, kFewN>;

__device__ __forceinline__ void few_load(const FewLoader& from, int stage, uint32_t uniform) {
#pragma unroll
  for (int q = 0; q < from.kW; ++q) from.load_w(q, stage, uniform);
  from.load_a(0, stage, uniform);
}
__device__ __forceinline__ void few_start(const GemmArgs& g, const FewLoader& from) {
  const int full = g.K / kBlock;
  if (full == 0) return;
#pragma unroll
  for (int d = 0; d < kFewStages - 1; ++d) few_load(from, d, min(d, full - 1) * kBlock);
}

template <int TM, int DT>
__device__ __forceinline__ void few_tile(const GemmArgs& g, const Tile& tile, const Tile& next, FewLoader& from, FewLds& lds) {
  using Op = Side<DT == MOE_DTYPE_F32>;
  constexpr int kLoads = FewLoader::kW + 1;
  static_assert(FewLoader::kA == 1, "one direct load of a and kW of the weights to a stage");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, piece = lane >> 4;
  auto scales = [&](int kb) {
    store_scales<kFewM>(g, tile, kb, from.a_at + static_cast<uint32_t>(offsetof(FewLds, a_scale)),
                        from.a_at + static_cast<uint32_t>(offsetof(FewLds, w_scale)));
  };
  f32x4 acc[TM][kFewN] = {};
  const int slot = (piece ^ (r & 7)) << 4;
  const int a_frag = r * kBlock + slot, w_frag = (wave * 16 * kFewN + (r >> 2) * 4 * kFewN + (r & 3)) * kBlock + slot;
  auto multiply = [&](int kb, int stage, auto tail, uint32_t left) {
    union Piece {
      u32x4 half[2];
      i32x8 all;
    };
    auto read = [&](const uint8_t* side, int at) {
      Piece u;
      u.half[0] = *reinterpret_cast<const u32x4*>(side + at);
      u.half[1] = *reinterpret_cast<const u32x4*>(side + (at ^ 64));
      return u;
    };
    const float sw = lds.w_scale[wave * 16 * kFewN / kBlock][kb % kScaleBlocks];
    Piece w[kFewN];
#pragma unroll
    for (int j = 0; j < kFewN; ++j) {
      w[j] = read(&lds.w[stage][j * 4 * kBlock], w_frag);
      if (decltype(tail)::value) {   // pieces behind the row's end
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if ((piece + 4 * h) * 16 >= left) w[j].half[h] = u32x4{0, 0, 0, 0};
      }
    }
    const Op wo[kFewN] = {Op(w[0].all), Op(w[1].all)};
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const Op a(read(&lds.a[stage][i * 16 * kBlock], a_frag).all);
      const float s = lds.a_scale[i * 16 + r][kb % kScaleBlocks] * sw;
#pragma unroll
      for (int j = 0; j < kFewN; ++j) {
        const f32x4 p = mfma_block(wo[j], a);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][j][v] = fmaf(p[v], s, acc[i][j][v]);
      }
    }
  };
  const int full = g.K / kBlock, last = full - 1;
  if (full > 0) {
    for (int kb = 0; kb <= last; ++kb) {
      if (kb % kScaleBlocks == 0) {
        if (kb > 0) {   // every wavefront is through with the scales that are replaced
          asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
          __builtin_amdgcn_s_barrier();
        }
        scales(kb);
      }
      // this block has landed (the later ones' loads may be in flight), and every wavefront is through
      // with the stage that the one kFewStages - 1 later goes to
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"((kFewStages - 2) * kLoads) : "memory");
      __builtin_amdgcn_s_barrier();
      few_load(from, (kb + kFewStages - 1) % kFewStages, min(kb + kFewStages - 1, last) * kBlock);
      multiply(kb, kb % kFewStages, std::false_type{}, kBlock);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");   // the last stages' loads
    __builtin_amdgcn_s_barrier();
  }
  // A short last block, not overlapped (see gemm_tile).
  if (full < g.kb) {
    const uint32_t left = g.K - full * kBlock;
    if (full % kScaleBlocks == 0) scales(full);
#pragma unroll
    for (int q = 0; q < from.kW; ++q) from.load_w(q, 0, full * kBlock, from.w_chunk() < left ? 0 : -from.w_chunk());
    from.load_a(0, 0, full * kBlock, from.a_chunk() < left ? 0 : -from.a_chunk());
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" : : : "memory");
    __builtin_amdgcn_s_barrier();
    multiply(full, 0, std::true_type{}, left);
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
    __builtin_amdgcn_s_barrier();
  }
  if (next.rows > 0) {
    from.aim(g, next);
    few_start(g, from);
  }
#pragma unroll
  for (int i = 0; i < TM; ++i)
    store_row<kFewN, DT>(g, tile, i * 16 + r, tile.col_tile * kTileN + wave * 16 * kFewN + piece * 4 * kFewN, acc[i]);
}

template <int DT>
__global__ __launch_bounds__(kTileThreads, 2) void fp8_gemm_few_kernel(GemmArgs g, int col_tiles) {
  __shared__ __align__(1024) FewLds lds;
  const int row_tiles = count_row_tiles(g, kFewM);
  const TileRun run = die_tiles(static_cast<uint32_t>(row_tiles) * col_tiles, blockIdx.x % 8);
  uint32_t t = run.first + blockIdx.x / 8;
  if (t >= run.end) return;
  FewLoader from;
  from.a_at = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((MOE_LDS uint8_t*)&lds.a[0][0]));
  from.w_at = from.a_at + static_cast<uint32_t>(offsetof(FewLds, w));
  Tile tile = tile_at(g, kFewM, row_tiles, col_tiles, t);
  from.aim(g, tile);
  few_start(g, from);
  while (tile.rows > 0) {
    t += gridDim.x / 8;
    Tile next{0, 0, 0, 0};
    if (t < run.end) next = tile_at(g, kFewM, row_tiles, col_tiles, t);
    if (tile.rows > 16) few_tile<2, DT>(g, tile, next, from, lds);
    else few_tile<1, DT>(g, tile, next, from, lds);
    tile = next;
  }
}

// Workgroups for tiles of BM by BN: every group with rows may have one partly filled row tile.
int tile_blocks(const GemmArgs& g, int BM, int BN, uint32_t* blocks, int* col_tiles) {
  *col_tiles = (g.N + BN - 1) / BN;
  const int64_t row_tiles = (static_cast<int64_t>(g.M) + BM - 1) / BM + (g.offsets ? min(g.E, g.M) : 0);
  const int64_t n = (row_tiles * *col_tiles + 7) / 8 * 8;
  if (n >> 31)
    return set_error(MOE_EUNSUPPORTED, "moe_fp8_gemm: %lld tiles are more than one launch takes", static_cast<long long>(n));
  *blocks = static_cast<uint32_t>(n);
  return MOE_OK;
}

// LDS holds one workgroup of the tile kernels per compute unit: each takes tiles until its die's run
// is done.
uint32_t resident_grid(uint32_t blocks) {
  return min(blocks, static_cast<uint32_t>((device_cu_count() + 7) / 8 * 8));
}

// Rows of the highest tile: what finishes first when every compute unit takes its tiles in turn, from
// the average group's rows.  A tile's time goes with its rows plus about 64 for the weights' part (777
// rows by 11264 columns in fp32: 48 us with 160-row tiles, one round, 60 us with 96-row ones, two, 70
// us with 112-row ones, two as well, and 71 us with 64-row ones, three; 256 rows for each of 64 experts:
// 419 us with 256-row tiles, 456 us with 128-row ones).
int tile_rows(const GemmArgs& g, int most) {
  const int groups = min(g.E, g.M), n = (g.M + groups - 1) / groups;
  const int64_t cus = device_cu_count(), cols = static_cast<int64_t>(groups) * ((g.N + kTileN - 1) / kTileN);
  int best = most;
  int64_t least = INT64_MAX;
  for (int bm = most; bm >= 64; bm -= 32) {
    const int tiles = (n + bm - 1) / bm, high = ((n + tiles - 1) / tiles + 31) / 32 * 32;
    const int64_t cost = (tiles * cols + cus - 1) / cus * (max(high, 64) + 64);
    if (cost < least) {
      least = cost;
      best = bm;
    }
  }
  return best;
}

template <int DT>
int launch_tile(const GemmArgs& g, hipStream_t stream) {
  uint32_t blocks;
  int col_tiles;
  const int bm = tile_rows(g, kTileM<DT>);
  if (int rc = tile_blocks(g, bm, kTileN, &blocks, &col_tiles)) return rc;
  ProfileScope prof("fp8_gemm", stream);
  hipLaunchKernelGGL(fp8_gemm_tile_kernel<DT>, dim3(resident_grid(blocks)), dim3(kTileThreads), 0, stream, g, bm, col_tiles);
  return check_launch("fp8_gemm");
}

template <int DT>
int launch_few(const GemmArgs& g, hipStream_t stream) {
  uint32_t blocks;
  int col_tiles;
  if (int rc = tile_blocks(g, kFewM, kTileN, &blocks, &col_tiles)) return rc;
  ProfileScope prof("fp8_gemm", stream);
  hipLaunchKernelGGL(fp8_gemm_few_kernel<DT>, dim3(resident_grid(blocks)), dim3(kTileThreads), 0, stream, g, col_tiles);
  return check_launch("fp8_gemm");
}

template <int MT, int NT, int DT>
int launch_stream(const GemmArgs& g, hipStream_t stream) {
  uint32_t blocks;
  int col_tiles;
  if (int rc = tile_blocks(g, MT * 16, NT * 16, &blocks, &col_tiles)) return rc;
  ProfileScope prof("fp8_gemm", stream);
  hipLaunchKernelGGL((fp8_gemm_stream_kernel<MT, NT, DT>), dim3(blocks), dim3(kStreamThreads), 0, stream, g, col_tiles);
  return check_launch("fp8_gemm");
}

template <int DT>
int launch_gemm(const GemmArgs& g, hipStream_t stream) {
  // By the average group's rows n and the tiles there are (us, 64 experts of 5120 x 3584 bf16 results):
  //   n          24    32    48    64    96
  //   tile      241   236   244   249   263     products and the L2 path bound it
  //   few       218   252   284   341   437     weights bound it; over 32 rows they are read again
  //   stream    316   431   561   677   975     finest tiles, weights 16 bytes to a cache access
  // The first two need tiles for the whole chip: 2 experts of 28672 x 4096 (224 tiles) take 52 us as
  // few and 46 as stream, 64 rows by 4096 x 4096 (32 tiles) 20 and 13; with 256 rows there (128 tiles)
  // 21 and 40, since the stream kernel reads the weights again for every 32 rows.
  const int groups = min(g.E, g.M), n = (g.M + groups - 1) / groups, cus = device_cu_count();
  const int64_t cols = static_cast<int64_t>(groups) * ((g.N + kTileN - 1) / kTileN);
  if (n > 28 && (n + 63) / 64 * cols >= cus) return launch_tile<DT>(g, stream);
  if (n > 96 || (n + kFewM - 1) / kFewM * cols >= 2 * cus) return launch_few<DT>(g, stream);
  // 16-column tiles where 32-column ones are few: one row by 4096 x 4096 8.6 -> 6.3 us, two experts of
  // 4096 x 14336 23.4 -> 20.3 us; with 2560 tiles (2048 x 1408, 16 tokens) 21.8 -> 24.0 us instead.
  if (n <= 16 && static_cast<int64_t>(groups) * ((g.N + 31) / 32) < 2 * cus) return launch_stream<1, 1, DT>(g, stream);
  if (n <= 16) return launch_stream<1, 2, DT>(g, stream);
  return launch_stream<2, 2, DT>(g, stream);
}

}  // namespace

int launch_fp8_gemm(const uint8_t* a, int64_t lda, const float* a_scales, int a_rows, const uint8_t* w,
                    const float* w_scales, int E, int M, int N, int K, const int32_t* offsets, const int32_t* pairs,
                    int k, void* c, int dtype, int64_t ldc, hipStream_t stream) {
  const GemmArgs g{a, lda, a_scales, a_rows, w, w_scales, E, M, N, K, (K + kBlock - 1) / kBlock,
                   (N + kBlock - 1) / kBlock, offsets, pairs, k, c, ldc};
  int rc = MOE_OK;
  with_dtype(dtype, [&](auto dt) { rc = launch_gemm<decltype(dt)::value>(g, stream); });
  return rc;
}

}  // namespace moeapq
