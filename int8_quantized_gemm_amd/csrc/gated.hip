// Gated feed-forward block: both projections, the activation and the product in
// one kernel, in 16 bits with its backward pass and in block-scaled FP8.
//
//   [G | U] = x W^T + delta       x [M, K], W [2I, K] (gate rows, then up rows)
//   h       = act(G) * U          [M, I]
//   dU = dh * act(G), dG = dh * U * act'(G)
//   dx = [dG | dU] W              [M, K]
//   dW = [dG | dU]^T x            [2I, K]
//
// tile16      LDS-tiled MFMA product with float32 accumulation. An operand is
//             read either along rows (contraction index contiguous, as x and W
//             in the forward pass) or across them (contraction index the row,
//             as W in dx and both operands of dW); the second form goes
//             through the transposing LDS read, so no operand is transposed in
//             memory.
// tile16s     the same for few tiles, the contraction split over the grid where
//             they are very few (tile16_sum adds the ranges' sums); tile16s_both
//             dx and dW in one launch.
// gated_stream  a few rows: W streamed once into MFMA registers.
// gated_grad  dG and dU from dh, G and U (elementwise); f16: gated_grad_max first.
// FP8: gated8 (tiles of 256 x 256), gated8s and gated8_sum (few tiles, and K
// blocks of 32), gated8_stream (a few rows), gated_quant (codes of float32 h).
#include <type_traits>

#include "mma16.h"
#include "q8_internal.h"
#include "tile_common.h"

namespace q8 {
namespace {

// ------------------------------------------------------------------------------
// LDS-tiled product
// ------------------------------------------------------------------------------
struct T16Params {
  const void* A;     // rows m (row-major operand) or contraction rows
  const void* B;
  int64_t lda, ldb;  // elements
  uint32_t a_bytes, b_bytes;
  int64_t M, N, C;   // output rows, output columns (h columns when gated), contraction
  int64_t a_cols;    // width of A when it is read across rows (a multiple of 8)
  void* D;           // [M, ldd]
  int64_t ldd;
  // gated forward
  const uint16_t* delta;  // [M, 2N] or null
  uint16_t* gate_up;      // [M, 2N] or null
  int64_t tiles_m, tiles_n;
  int64_t whole;     // tile16: workgroups with a whole tile (the tiles after them are two halves)
  int pair;          // output (and delta / gate_up) rows 4-byte aligned, their widths even
  int S;             // tile16s: ranges of the contraction (for the host: 1 asks for one range)
  float* part;       // their sums [S][M][N, or 2N when gated], or null for S = 1
  const int32_t* exp;  // f16 gradients: the power of two taken out of A
};

// A sum of an f16 gradient with the power of two put back.
template <bool BF>
__device__ __forceinline__ float2 put_back(float2 v, int e) {
  if constexpr (BF) return v;
  else return float2{__builtin_ldexpf(v.x, e), __builtin_ldexpf(v.y, e)};
}

// Stage layout of an operand read across rows (contraction index the row):
// [64 contraction rows][ROWS columns], 16-byte chunk c of row k at position
// c ^ tr_key(k). ds_read_tr16_b64 gives lane i of a sixteen-lane group column i of
// four rows; a half-wave's two groups read rows 8g .. 8g+3 (g = 0, 1 or 2, 3),
// two chunks each, and the key spreads those eight rows over all sixteen chunk
// positions of the 256-byte bank line (rows of 256 bytes: by bits 0, 1 and 3 of
// k; rows of 128 bytes lie in alternating halves already: by bits 1 and 3).
template <int LPR>
__device__ __forceinline__ int tr_key(int k) {
  static_assert(LPR == 8 || LPR == 16, "row of 128 or 256 bytes");
  return LPR == 16 ? 2 * ((k & 3) | ((k & 8) >> 1)) : (k & 2) | ((k & 8) >> 1);
}

typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4 tr_read2(const uint8_t* p0, const uint8_t* p1) {
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Q8_AS3 s16x4*)p0);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Q8_AS3 s16x4*)p1);
  typedef int i32x2 __attribute__((ext_vector_type(2)));
  const i32x2 x = __builtin_bit_cast(i32x2, a), y = __builtin_bit_cast(i32x2, b);
  return i32x4{x[0], x[1], y[0], y[1]};
}

// ROWS rows (row-major) or columns (TR) of one operand, one 64-deep slab per
// stage. NW waves share the copies; lane l of wave load q = w + c NW writes 16
// bytes at 1024 q + 16 l. Rows and columns past the operand's end re-read its
// last ones (they reach only outputs that are not stored), so every copy lies
// inside the buffer; what lies past the contraction's end is given an offset
// beyond any buffer, which reads as zeros, in both operands.
constexpr uint32_t kNowhere = 0xFFFFFFF0u;

template <int ROWS, int NW, bool TR>
struct Operand {
  static constexpr int kLoads = ROWS * 128 / 1024 / NW;
  static constexpr int LPR = ROWS / 8;             // TR: lanes per contraction row
  static constexpr int RPL = TR ? 64 / LPR : 8;    // stage rows per load
  static_assert(ROWS * 128 % (1024 * NW) == 0 && NW % 2 == 0, "whole loads per wave");
  static_assert(!TR || (RPL * NW) % 16 == 0, "the swizzle key is the same for all of a wave's loads");
  __amdgpu_buffer_rsrc_t r;
  uint32_t voff[kLoads];
  uint32_t slab;  // bytes between slabs
  int in;         // first element of the slab that this lane copies (row-major: K offset; TR: contraction row)

  // row(i): operand row of stage row i, inside the operand (row-major);
  // col0, cols: first column of the tile and the operand's width (TR)
  template <typename F>
  __device__ __forceinline__ void init(const void* p, uint32_t bytes, int64_t ld, F&& row, int64_t col0, int64_t cols,
                                       int w, int lane) {
    r = make_rsrc(p, bytes);
    if constexpr (!TR) {
      // load q fills rows 8q .. 8q+7: physical chunk l % 8 of row 8q + l/8
      // holds logical chunk (l % 8) ^ key, and q's parity is w's
      const int chunk = (lane & 7) ^ ((4 * (w & 1) + (lane >> 4)) & 7);
#pragma unroll
      for (int c = 0; c < kLoads; ++c)
        voff[c] = (uint32_t)(row(8 * (w + c * NW) + (lane >> 3)) * ld * 2) + chunk * 16;
      slab = 128;
      in = chunk * 8;
    } else {
      const int k = RPL * w + lane / LPR;
      const int chunk = (lane % LPR) ^ tr_key<LPR>(k);
      int64_t col = col0 + chunk * 8;
      if (col > cols - 8) col = cols - 8;
#pragma unroll
      for (int c = 0; c < kLoads; ++c) voff[c] = (uint32_t)((k + c * RPL * NW) * ld * 2 + col * 2);
      slab = (uint32_t)(64 * ld * 2);
      in = k;
    }
  }
  // left: contraction elements from this slab's start to the end
  __device__ __forceinline__ void issue(int kt, int64_t left, uint8_t* lds, int w) const {
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      const bool ok = in + (TR ? c * RPL * NW : 0) < left;
      b2l16(r, ok ? voff[c] : kNowhere, kt * slab, lds + (w + c * NW) * 1024);
    }
  }
  // fragment of the sixteen rows from row, K step s (32 deep)
  __device__ __forceinline__ static i32x4 frag(const uint8_t* lds, int row, int s, int lane) {
    const int g = lane >> 4, r16 = lane & 15;
    if constexpr (!TR) {
      return *reinterpret_cast<const i32x4*>(lds + swz(row + r16, 4 * s + g));
    } else {
      const int k = 32 * s + 8 * g + (r16 >> 2);
      const int chunk = ((row >> 3) + ((r16 & 3) >> 1)) ^ tr_key<LPR>(k);
      const uint8_t* p = lds + k * (ROWS * 2) + chunk * 16 + (r16 & 1) * 8;
      return tr_read2(p, p + 4 * ROWS * 2);
    }
  }
};

// D's rows are operand A's: lane (g, r16) of a 16 x 16 block holds rows 4g .. 4g+3 of
// column r16, so adjacent lanes hold adjacent columns. Two columns per lane make
// a 4-byte store and 64-byte runs of a row; a lane that holds one row's columns
// instead (the operands exchanged) makes every lane's store a memory request
// of its own, 16 for one at the same bytes (forward of 4096 x 7168 x 2x9216 with its
// pre-activations: 50 us of requests).
__device__ __forceinline__ float swap_lanes(float v) {  // the neighbour's (lane ^ 1) value
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, true));
}

// Even lanes get (a of this lane, a of the next), odd lanes (b of the one
// before, b of this lane).
__device__ __forceinline__ float2 pair_lanes(float a, float b, bool odd) {
  const float o = swap_lanes(odd ? a : b);
  return odd ? float2{o, b} : float2{a, o};
}

// Two adjacent columns n, n+1 of a row at p (n even where the rows are 4-byte
// aligned).
template <bool BF>
__device__ __forceinline__ void store2(uint16_t* p, float2 v, int64_t n, int64_t N, bool pair) {
  const uint32_t o = pack2<BF>(v.x, v.y);
  if (pair) {
    if (n < N) *reinterpret_cast<uint32_t*>(p) = o;  // N is even
  } else {
    if (n < N) p[0] = (uint16_t)o;
    if (n + 1 < N) p[1] = (uint16_t)(o >> 16);
  }
}

template <bool BF>
__device__ __forceinline__ float2 load2(const uint16_t* p, int64_t n, int64_t N, bool pair) {
  if (pair) {
    const uint32_t o = n < N ? *reinterpret_cast<const uint32_t*>(p) : 0u;
    return float2{lo_f32<BF>(o), hi_f32<BF>(o)};
  }
  return float2{n < N ? out_bits_to_f32<BF>(p[0]) : 0.0f, n + 1 < N ? out_bits_to_f32<BF>(p[1]) : 0.0f};
}

// The same as loaded, to be used later: columns n and n + 1 of a row, column 0 (and
// 1) where n lies past the end.
__device__ __forceinline__ uint32_t load2_raw(const uint16_t* row, int64_t n, int64_t N, bool pair) {
  const uint16_t* const q = row + (n < N ? n : 0);
  if (pair) return *reinterpret_cast<const uint32_t*>(q);
  return q[0] | (uint32_t)q[n + 1 < N ? 1 : 0] << 16;
}

// Gate and up values of columns n, n+1 of row m to the outputs.
template <bool BF, int ACT>
__device__ __forceinline__ void gated_out(const T16Params& p, int64_t m, int64_t n, float2 G, float2 U, bool pair) {
  const int64_t N = p.N;
  if (p.gate_up) {
    uint16_t* q = p.gate_up + m * 2 * N + n;
    store2<BF>(q, G, n, N, pair);
    store2<BF>(q + N, U, n, N, pair);
  }
  store2<BF>(static_cast<uint16_t*>(p.D) + m * N + n, float2{act_f32<ACT>(G.x) * U.x, act_f32<ACT>(G.y) * U.y}, n, N,
             pair);
}

// One output tile of BM x BN per workgroup, both operands in 64-deep slabs of
// two halves each (A0, A1: BM/2 rows; B0, B1: BN/2 columns), two stages of LDS
// per half. A wave owns the same rows of both A halves and the same columns of
// both B halves, so a slab is four products of halves: A0 F, A0 S, A1 S, A1 F with F,
// S = B0, B1 in even slabs and B1, B0 in odd ones, so that from one product to the
// next, slabs included, only one operand changes. Each fragment is read into the
// registers of the one it follows as soon as that one's last instruction is
// out, a product (sixteen instructions) ahead of its first use:
//   product   reads meanwhile
//   A0 F      S
//   -- barrier 1: A1 has landed; A0, B0, B1 of slab k have been read, and their
//      stages are refilled with slab k + 2
//   A0 S      A1 over A0, block by block
//   A1 S
//   -- barrier 2: A0, B0, B1 of slab k + 1 have landed; A1 has been read and is
//      refilled
//   A1 F      S of slab k + 1; A0 of slab k + 1 over A1
// so the copies of a half have one and a half slabs to land, the waits count
// them and never drain them, and the eight waves meet twice a slab. (Four
// phases a slab, each reading its fragments ahead of a barrier while the other
// wave of the SIMD multiplies, measured 808 us for 4096 x 7168 x 2x9216: reading by
// four waves at a time took longer than their products.)
// The copies of slabs past the end read nothing and write zeros, which keeps
// the counts of outstanding copies the same to the last slab.
// GATED: B0 holds gate rows and B1 the up rows of the same columns, so a lane
// holds both factors of an output; N = I.
template <int BM, int BN, bool TRA, bool TRB, bool BF, bool GATED, int ACT>
__device__ __forceinline__ void tile16_body(const T16Params& p, int64_t m0, int64_t n0, uint8_t* __restrict__ a00,
                                            uint8_t* __restrict__ a01, uint8_t* __restrict__ a10,
                                            uint8_t* __restrict__ a11, uint8_t* __restrict__ b00,
                                            uint8_t* __restrict__ b01, uint8_t* __restrict__ b10,
                                            uint8_t* __restrict__ b11) {
  constexpr int WM = 2, WN = 4, NW = WM * WN;
  constexpr int HM = BM / 2, HN = BN / 2;
  constexpr int TM = HM / WM, TN = HN / WN, FM = TM / 16, FN = TN / 16;
  static_assert(FN == 2, "two column blocks per wave");
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WN, wn = w % WN;
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t M = p.M, N = p.N, C = p.C;
  typedef Operand<HM, NW, TRA> OA;
  typedef Operand<HN, NW, TRB> OB;
  constexpr int LA = OA::kLoads, LB = OB::kLoads;
  OA oa[2];
  OB ob[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    oa[h].init(p.A, p.a_bytes, p.lda, [&](int i) { return m0 + h * HM + i < M ? m0 + h * HM + i : M - 1; },
               m0 + h * HM, p.a_cols, w, lane);
    ob[h].init(p.B, p.b_bytes, p.ldb,
               [&](int i) -> int64_t {
                 // stage rows r and 16 + r of a wave's 32 hold columns 2r and 2r + 1
                 const int64_t n = n0 + (GATED ? 0 : h * HN) + i / 32 * 32 + 2 * (i % 16) + i / 16 % 2;
                 return (n < N ? n : N - 1) + (GATED && h ? N : 0);
               },
               n0 + h * HN, N, w, lane);
  }
  const int KT = (int)((C + 63) / 64);
  f32x4 acc[2][2][FM][FN];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[h][v][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  i32x4 fa[2][FM], fb[2][2][FN];  // [K step][block]; fb[half]
  auto read_b = [&](const uint8_t* lds, i32x4 (&f)[2][FN]) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < FN; ++j) f[s][j] = OB::frag(lds, wn * TN + j * 16, s, lane);
  };
  // what this wave has read is in registers, all but the last n of its copies
  // are in LDS; after the barrier that holds for every wave
  auto meet = [&](auto n) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(n)::value) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // NEXT: next is the stage of the A half that replaces fa
  auto products = [&](f32x4 (&c)[FM][FN], const i32x4 (&f)[2][FN], auto NEXT, const uint8_t* next) {
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < FN; ++j) c[i][j] = mfma16<BF>(fa[s][i], f[s][j], c[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (decltype(NEXT)::value) {
#pragma unroll
        for (int s = 0; s < 2; ++s) fa[s][i] = OA::frag(next, wm * TM + i * 16, s, lane);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto left = [&](int k) { return C - (int64_t)k * 64; };
  // slab k in the stages a0, a1, b0, b1; xa0, xf, xs: the next slab's A0 and its
  // stages of this slab's F and S
  auto slab = [&](int k, auto F, uint8_t* a0, uint8_t* a1, uint8_t* b0, uint8_t* b1, const uint8_t* xa0,
                  const uint8_t* xs) {
    constexpr int f = decltype(F)::value, s = 1 - f;
    read_b(s ? b1 : b0, fb[s]);
    products(acc[0][f], fb[f], std::false_type{}, nullptr);
    meet(std::integral_constant<int, 2 * LA + 2 * LB>{});  // A1 of this slab
    oa[0].issue(k + 2, left(k + 2), a0, w);
    ob[0].issue(k + 2, left(k + 2), b0, w);
    ob[1].issue(k + 2, left(k + 2), b1, w);
    products(acc[0][s], fb[s], std::true_type{}, a1);
    products(acc[1][s], fb[s], std::false_type{}, nullptr);
    meet(std::integral_constant<int, 2 * LA + 2 * LB>{});  // A0, B0, B1 of the next slab
    oa[1].issue(k + 2, left(k + 2), a1, w);
    read_b(xs, fb[s]);
    products(acc[1][f], fb[f], std::true_type{}, xa0);
  };
  oa[0].issue(0, left(0), a00, w);
  ob[0].issue(0, left(0), b00, w);
  ob[1].issue(0, left(0), b10, w);
  oa[1].issue(0, left(0), a10, w);
  oa[0].issue(1, left(1), a01, w);
  ob[0].issue(1, left(1), b01, w);
  ob[1].issue(1, left(1), b11, w);
  oa[1].issue(1, left(1), a11, w);
  meet(std::integral_constant<int, 3 * LA + 2 * LB>{});    // A0, B0, B1 of slab 0
  read_b(b00, fb[0]);
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[s][i] = OA::frag(a00, wm * TM + i * 16, s, lane);
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd_slab{};
  int k = 0;
  for (; k + 1 < KT; k += 2) {
    slab(k, even, a00, a10, b00, b10, a01, b11);
    slab(k + 1, odd_slab, a01, a11, b01, b11, a00, b00);
  }
  if (k < KT) slab(k, even, a00, a10, b00, b10, a01, b11);
  wait_vmem();  // no copy outlives the workgroup's LDS
  const bool pair = p.pair != 0, odd = lane & 1;
  const int64_t nw = n0 + wn * TN;
  if constexpr (!GATED) {
    uint16_t* D = static_cast<uint16_t*>(p.D);
    const int e = BF ? 0 : *p.exp;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t m = m0 + h * HM + wm * TM + i * 16 + 4 * g + r;
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float x = acc[h][v][i][0][r], y = acc[h][v][i][1][r];
            // columns read across rows lie as they are: block 0's pairs go to the
            // even lanes and block 1's to the odd ones
            const float2 o = TRB ? pair_lanes(x, y, odd) : float2{x, y};
            const int64_t n = nw + v * HN + (TRB ? (odd ? 15 + r16 : r16) : 2 * r16);
            if (m < M) store2<BF>(D + m * p.ldd + n, put_back<BF>(o, e), n, N, pair);
          }
        }
  } else {
    const int64_t n = nw + 2 * r16;
    // the next rows' delta is loaded ahead of these rows' stores, which a wait
    // for it would otherwise include
    float2 dg[2][4], du[2][4];
    auto load_delta = [&](int q, int h, int i) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        int64_t m = m0 + h * HM + wm * TM + i * 16 + 4 * g + r;
        if (m >= M) m = M - 1;
        dg[q][r] = load2<BF>(p.delta + m * 2 * N + n, n, N, pair);
        du[q][r] = load2<BF>(p.delta + m * 2 * N + N + n, n, N, pair);
      }
    };
    if (p.delta) load_delta(0, 0, 0);
#pragma unroll
    for (int b = 0; b < 2 * FM; ++b) {
      const int h = b / FM, i = b % FM, q = b & 1;
      if (p.delta && b + 1 < 2 * FM) load_delta(q ^ 1, (b + 1) / FM, (b + 1) % FM);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t m = m0 + h * HM + wm * TM + i * 16 + 4 * g + r;
        float2 G = {acc[h][0][i][0][r], acc[h][0][i][1][r]}, U = {acc[h][1][i][0][r], acc[h][1][i][1][r]};
        if (p.delta) {
          G.x += dg[q][r].x;
          G.y += dg[q][r].y;
          U.x += du[q][r].x;
          U.y += du[q][r].y;
        }
        if (m < M) gated_out<BF, ACT>(p, m, n, G, U, pair);
      }
    }
  }
}

// Tiles of 256 x 256, one workgroup per compute unit. A last round that fills at
// most half the chip is dealt out as halves of 128 rows, which take two thirds
// of a tile's time on twice the units.
struct HalfTile {
  int64_t m0, tn;
  bool half;
};
__device__ __forceinline__ HalfTile half_tile(const T16Params& p) {
  const int64_t tiles = p.tiles_m * p.tiles_n;
  int64_t b = blockIdx.x;
  const bool half = b >= p.whole;
  const int64_t lower = half && b >= tiles ? 1 : 0;  // rows 128 .. 255 of its tile
  if (lower) b -= tiles - p.whole;
  int64_t tm, tn;
  grouped_order(xcd_remap(b, tiles), p.tiles_m, p.tiles_n, 4, tm, tn);
  return {tm * 256 + lower * 128, tn, half};
}

template <bool TRA, bool TRB, bool BF, bool GATED, int ACT>
__global__ __launch_bounds__(512, 2) void tile16(T16Params p) {
  __shared__ __attribute__((aligned(1024))) uint8_t a00[128 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t a01[128 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t a10[128 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t a11[128 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t b00[128 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t b01[128 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t b10[128 * 128];
  __shared__ __attribute__((aligned(1024))) uint8_t b11[128 * 128];
  const HalfTile t = half_tile(p);
  const int64_t n0 = t.tn * (GATED ? 128 : 256);
  if (!t.half) tile16_body<256, 256, TRA, TRB, BF, GATED, ACT>(p, t.m0, n0, a00, a01, a10, a11, b00, b01, b10, b11);
  else if (t.m0 < p.M)
    tile16_body<128, 256, TRA, TRB, BF, GATED, ACT>(p, t.m0, n0, a00, a01, a10, a11, b00, b01, b10, b11);
}

// Few tiles: BM x BN per workgroup (GATED: BN/2 columns of h), 128 x 128 by eight
// waves of 64 x 32 with four stages of LDS, or, up to 64 rows, 64 x 64 by waves of
// 16 x 32 with eight stages or 64 x 128 by waves of 32 x 32 with six (seven and
// five slabs in flight: the weight stream needs some 50 KB in flight per
// compute unit); one barrier per slab; and the contraction split over the grid
// where even that leaves compute units idle (the ranges' float32 sums then go to
// part, for tile16_sum). With so little work per workgroup the barriers of a tile16
// slab cost more than its schedule gives.
constexpr int t16s_stages(int BM, int WM) { return BM == 128 ? 4 : WM == 4 ? 8 : 6; }
constexpr int t16s_stage(int BM, int WM) { return (BM + 32 * (8 / WM)) * 128; }  // A, then B

template <int BM, int WM, bool TRA, bool TRB, bool BF, bool GATED, int ACT>
__device__ __forceinline__ void tile16s_body(const T16Params& p, int64_t block, uint8_t* __restrict__ s0,
                                             uint8_t* __restrict__ s1, uint8_t* __restrict__ s2,
                                             uint8_t* __restrict__ s3, uint8_t* __restrict__ s4,
                                             uint8_t* __restrict__ s5, uint8_t* __restrict__ s6,
                                             uint8_t* __restrict__ s7) {
  constexpr int NW = 8, WN = NW / WM, BN = 32 * WN, FM = BM / WM / 16, FN = 2, NST = t16s_stages(BM, WM);
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WN, wn = w % WN;
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t tiles = p.tiles_m * p.tiles_n;
  const int64_t b = xcd_remap(block, tiles * p.S);
  const int s = (int)(b / tiles);
  int64_t tm, tn;
  grouped_order(b % tiles, p.tiles_m, p.tiles_n, 4, tm, tn);
  const int64_t m0 = tm * BM, n0 = tn * (GATED ? BN / 2 : BN);
  const int64_t M = p.M, N = p.N, C = p.C;
  typedef Operand<BM, NW, TRA> OA;
  typedef Operand<BN, NW, TRB> OB;
  OA oa;
  OB ob;
  oa.init(p.A, p.a_bytes, p.lda, [&](int i) { return m0 + i < M ? m0 + i : M - 1; }, m0, p.a_cols, w, lane);
  ob.init(p.B, p.b_bytes, p.ldb,
          [&](int i) -> int64_t {
            // a wave's 32 stage rows: gated, sixteen gate rows and the up rows of
            // the same columns; else columns 2r in row r and 2r + 1 in row 16 + r
            const int64_t n = GATED ? n0 + i / 32 * 16 + i % 16 : n0 + i / 32 * 32 + 2 * (i % 16) + i / 16 % 2;
            return (n < N ? n : N - 1) + (GATED && i / 16 % 2 ? N : 0);
          },
          n0, N, w, lane);
  const int KT = (int)((C + 63) / 64);
  const int k_b = (int)((int64_t)s * KT / p.S), k_e = (int)((int64_t)(s + 1) * KT / p.S);
  f32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto issue = [&](int kt, uint8_t* __restrict__ l) {
    const int64_t left = C - (int64_t)kt * 64;
    oa.issue(kt, left, l, w);
    ob.issue(kt, left, l + BM * 128, w);
  };
  auto step = [&](int kt, uint8_t* __restrict__ nl, const uint8_t* __restrict__ la) {
    const uint8_t* const lb = la + BM * 128;
    // this slab has landed (NST - 2 later ones may be in flight) and the slab
    // before has been read, for every wave
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NST - 2) * (OA::kLoads + OB::kLoads)) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue(kt + NST - 1, nl);
    i32x4 fb[2][FN], fa[2][FM];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < FN; ++j) fb[h][j] = OB::frag(lb, wn * 32 + j * 16, h, lane);
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[h][i] = OA::frag(la, wm * (16 * FM) + i * 16, h, lane);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma16<BF>(fa[h][i], fb[h][j], acc[i][j]);
  };
  issue(k_b, s0);
  issue(k_b + 1, s1);
  issue(k_b + 2, s2);
  if constexpr (NST > 4) {
    issue(k_b + 3, s3);
    issue(k_b + 4, s4);
  }
  if constexpr (NST > 6) {
    issue(k_b + 5, s5);
    issue(k_b + 6, s6);
  }
  for (int kt = k_b;;) {
    if constexpr (NST == 4) {
      step(kt, s3, s0);
      if (++kt >= k_e) break;
      step(kt, s0, s1);
      if (++kt >= k_e) break;
      step(kt, s1, s2);
      if (++kt >= k_e) break;
      step(kt, s2, s3);
      if (++kt >= k_e) break;
    } else if constexpr (NST == 6) {
      step(kt, s5, s0);
      if (++kt >= k_e) break;
      step(kt, s0, s1);
      if (++kt >= k_e) break;
      step(kt, s1, s2);
      if (++kt >= k_e) break;
      step(kt, s2, s3);
      if (++kt >= k_e) break;
      step(kt, s3, s4);
      if (++kt >= k_e) break;
      step(kt, s4, s5);
      if (++kt >= k_e) break;
    } else {
      step(kt, s7, s0);
      if (++kt >= k_e) break;
      step(kt, s0, s1);
      if (++kt >= k_e) break;
      step(kt, s1, s2);
      if (++kt >= k_e) break;
      step(kt, s2, s3);
      if (++kt >= k_e) break;
      step(kt, s3, s4);
      if (++kt >= k_e) break;
      step(kt, s4, s5);
      if (++kt >= k_e) break;
      step(kt, s5, s6);
      if (++kt >= k_e) break;
      step(kt, s6, s7);
      if (++kt >= k_e) break;
    }
  }
  wait_vmem();  // no copy outlives the workgroup's LDS
  const bool pair = p.pair != 0, odd = lane & 1;
  if (p.part) {
    const int64_t W = GATED ? 2 * N : N;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t m = m0 + wm * (16 * FM) + i * 16 + 4 * g + r;
        if (m >= M) continue;
        float* q = p.part + ((int64_t)s * M + m) * W;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int64_t n = GATED ? n0 + wn * 16 + r16 : n0 + wn * 32 + (TRB ? j * 16 + r16 : 2 * r16 + j);
          if (n < N) q[n + (GATED && j ? N : 0)] = acc[i][j][r];
        }
      }
    return;
  }
  uint32_t dg[FM][2], du[FM][2];  // loaded ahead of the first store, which a wait for one would include
  int e = 0;
  if constexpr (!GATED && !BF) e = *p.exp;
  if constexpr (GATED) {
    if (p.delta) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          const int64_t m = m0 + wm * (16 * FM) + i * 16 + 4 * g + r + (odd ? 1 : 0), n = n0 + wn * 16 + (r16 & ~1);
          const uint16_t* const d = p.delta + (m < M ? m : M - 1) * 2 * N;
          dg[i][r / 2] = load2_raw(d, n, N, pair);
          du[i][r / 2] = load2_raw(d + N, n, N, pair);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (GATED) {
        if (r % 2) continue;
        // even lanes take columns r16, r16 + 1 of row r, odd lanes r16 - 1, r16 of row r + 1
        float2 G = pair_lanes(acc[i][0][r], acc[i][0][r + 1], odd), U = pair_lanes(acc[i][1][r], acc[i][1][r + 1], odd);
        const int64_t m = m0 + wm * (16 * FM) + i * 16 + 4 * g + r + (odd ? 1 : 0), n = n0 + wn * 16 + (r16 & ~1);
        if (m >= M) continue;
        if (p.delta) {
          const uint32_t d = dg[i][r / 2], e = du[i][r / 2];
          G.x += lo_f32<BF>(d);
          G.y += hi_f32<BF>(d);
          U.x += lo_f32<BF>(e);
          U.y += hi_f32<BF>(e);
        }
        gated_out<BF, ACT>(p, m, n, G, U, pair);
      } else {
        const int64_t m = m0 + wm * (16 * FM) + i * 16 + 4 * g + r;
        const float x = acc[i][0][r], y = acc[i][1][r];
        const float2 o = TRB ? pair_lanes(x, y, odd) : float2{x, y};
        const int64_t n = n0 + wn * 32 + (TRB ? (odd ? 15 + r16 : r16) : 2 * r16);
        if (m < M) store2<BF>(static_cast<uint16_t*>(p.D) + m * p.ldd + n, put_back<BF>(o, e), n, N, pair);
      }
    }
}

template <int BM, int WM, bool TRA, bool TRB, bool BF, bool GATED, int ACT>
__global__ __launch_bounds__(512, 2) void tile16s(T16Params p) {
  constexpr int NST = t16s_stages(BM, WM), kStage = t16s_stage(BM, WM);
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s4[NST > 4 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s5[NST > 4 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s6[NST > 6 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s7[NST > 6 ? kStage : 16];
  tile16s_body<BM, WM, TRA, TRB, BF, GATED, ACT>(p, blockIdx.x, s0, s1, s2, s3, s4, s5, s6, s7);
}

// dx and dW in one launch, in tiles of 128 x 128 over their whole contractions: the
// workgroups with the longer one first, so that the others fill up behind them.
template <bool BF>
__global__ __launch_bounds__(512, 2) void tile16s_both(T16Params x, T16Params w, int x_first) {
  constexpr int kStage = t16s_stage(128, 2);
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[kStage];
  const int64_t nx = x.tiles_m * x.tiles_n, nw = w.tiles_m * w.tiles_n;
  const int64_t b = blockIdx.x;
  if (x_first ? b < nx : b >= nw)
    tile16s_body<128, 2, false, true, BF, false, 0>(x, x_first ? b : b - nw, s0, s1, s2, s3, s0, s0, s0, s0);
  else
    tile16s_body<128, 2, true, true, BF, false, 0>(w, x_first ? b - nx : b, s0, s1, s2, s3, s0, s0, s0, s0);
}

// Outputs from the S ranges' sums, added in order: two columns per thread.
template <bool BF, bool GATED, int ACT>
__global__ __launch_bounds__(256) void tile16_sum(T16Params p) {
  const int64_t N = p.N, W = GATED ? 2 * N : N, half = (N + 1) / 2;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.M * half) return;
  const int64_t m = i / half, n = (i - m * half) * 2;
  const bool pair = p.pair != 0, second = n + 1 < N;
  float2 x = {0.f, 0.f}, y = {0.f, 0.f};
  const float* q = p.part + m * W + n;
  for (int s = 0; s < p.S; ++s, q += p.M * W) {
    x.x += q[0];
    x.y += second ? q[1] : 0.0f;
    if constexpr (GATED) {
      y.x += q[N];
      y.y += second ? q[N + 1] : 0.0f;
    }
  }
  if constexpr (GATED) {
    if (p.delta) {
      const float2 d = load2<BF>(p.delta + m * 2 * N + n, n, N, pair), e = load2<BF>(p.delta + m * 2 * N + N + n, n, N, pair);
      x.x += d.x;
      x.y += d.y;
      y.x += e.x;
      y.y += e.y;
    }
    gated_out<BF, ACT>(p, m, n, x, y, pair);
  } else {
    store2<BF>(static_cast<uint16_t*>(p.D) + m * p.ldd + n, put_back<BF>(x, BF ? 0 : *p.exp), n, N, pair);
  }
}

// ------------------------------------------------------------------------------
// Up to sixteen rows
// ------------------------------------------------------------------------------
struct StreamParams {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* W;
  int64_t M, I, K;
  const uint16_t* delta;
  uint16_t* gate_up;
  uint16_t* h;
};

// One workgroup per eight h columns: operand 0's sixteen rows are their eight
// gate rows and eight up rows, operand 1 the activation rows. The waves split K
// and load U chunks of it before any product; partials are summed in wave order
// through LDS.
template <int NW, int U, bool BF, int ACT>
__global__ __launch_bounds__(NW * 64) void gated_stream(StreamParams p) {
  __shared__ f32x4 red[NW][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t M = p.M, I = p.I, K = p.K;
  const int64_t n0 = (int64_t)blockIdx.x * 8;
  const int64_t col = n0 + (r16 & 7) < I ? n0 + (r16 & 7) : I - 1;
  const uint16_t* wp = p.W + (col + (r16 < 8 ? 0 : I)) * K + 8 * g;
  const uint16_t* xp = p.x + (r16 < M ? r16 : M - 1) * p.ldx + 8 * g;
  const int NC = (int)((K + 31) / 32);
  const int c_b = (int)((int64_t)w * NC / NW), c_e = (int)((int64_t)(w + 1) * NC / NW);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const i32x4 zero = {0, 0, 0, 0};
  for (int c0 = c_b; c0 < c_e; c0 += U) {
    i32x4 wf[U], xf[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (int64_t)(c0 + u) * 32;
      const bool in = c0 + u < c_e && k + 8 * g < K;
      wf[u] = in ? *reinterpret_cast<const i32x4*>(wp + k) : zero;
      xf[u] = in ? *reinterpret_cast<const i32x4*>(xp + k) : zero;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) acc = mfma16<BF>(wf[u], xf[u], acc);
  }
  red[w][lane] = acc;
  __syncthreads();
  // output (m, column c of eight): gate in row c of D, up in row c + 8
  if (tid >= 128) return;
  const int c = tid & 7, m = tid >> 3;
  const int64_t n = n0 + c;
  if (m >= M || n >= I) return;
  const float* redf = reinterpret_cast<const float*>(red);
  float G = 0.f, Uv = 0.f;
#pragma unroll
  for (int ww = 0; ww < NW; ++ww) {
    const float* q = redf + ww * 256;
    G += q[((c >> 2) * 16 + m) * 4 + (c & 3)];
    Uv += q[((2 + (c >> 2)) * 16 + m) * 4 + (c & 3)];
  }
  if (p.delta) {
    G += out_bits_to_f32<BF>(p.delta[m * 2 * I + n]);
    Uv += out_bits_to_f32<BF>(p.delta[m * 2 * I + I + n]);
  }
  if (p.gate_up) {
    p.gate_up[m * 2 * I + n] = (uint16_t)f32_to_out_bits<BF>(G);
    p.gate_up[m * 2 * I + I + n] = (uint16_t)f32_to_out_bits<BF>(Uv);
  }
  p.h[m * I + n] = (uint16_t)f32_to_out_bits<BF>(act_f32<ACT>(G) * Uv);
}

// ------------------------------------------------------------------------------
// Block-scaled FP8, few tiles
// ------------------------------------------------------------------------------
// tile16s for FP8 operands (NC blocks of sixteen h columns per wave): a 128-byte slab is one K block of 128, whose product
// comes out of v_mfma_f32_16x16x128_f8f6f4 on its own and is scaled into the sums,
// or four of 32 with a v_mfma_f32_16x16x32_fp8_fp8 each, the weight as operand 0
// there, so that a lane's four values share one row scale (half the vector
// instructions per product, which bound this form). The scales of a slab are
// copied to LDS with it (held in registers, the compiler moved each one as it
// arrived, waiting for all copies before it).
struct T8Params {
  T16Params t;        // A, B, lda, ldb and C in units of two bytes
  const float* As;    // [M, KB KSUB], KSUB = 128 / bk
  const float* Ws;    // [ceil(2I/bn), KB KSUB]
  int KB, bn;         // 128-byte slabs; weight-block height
  uint8_t* q;         // codes and scales instead of D, or null
  float* qs;
  int bf16, act;
};

// Wave-uniform offset of a slab's scales. The range check compares the lane's offset
// with the buffer's size less the uniform one, which must not pass that size: a
// buffer of a few scales is shorter than the slabs copied ahead of the last. (The
// operands' sizes and slabs are multiples of 16 bytes, and kNowhere lies
// sixteen below the end of the offsets.)
__device__ __forceinline__ uint32_t scale_at(int64_t left, int off) { return left > 0 ? (uint32_t)off : 0u; }

template <int KS, int BM, int WM, int NC>
__global__ __launch_bounds__(512, 2) void gated8s(T8Params P) {
  constexpr int NW = 8, WN = NW / WM, BN = 32 * WN * NC, FM = BM / WM / 16;
  constexpr int KSUB = 128 / KS, SB = 4 * KSUB;  // K blocks and scale bytes of a row per slab
  constexpr int NST = NC == 2 ? 3 : BM == 128 ? 4 : WM == 4 ? 8 : 6;
  constexpr int kStage = (BM + BN) * 128 + BM * SB + 64 * SB;  // A, B, row scales, weight scales
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[NST > 3 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s4[NST > 4 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s5[NST > 4 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s6[NST > 6 ? kStage : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t s7[NST > 6 ? kStage : 16];
  const T16Params& p = P.t;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WN, wn = w % WN;
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t tiles = p.tiles_m * p.tiles_n;
  const int64_t b = xcd_remap(blockIdx.x, tiles * p.S);
  const int s = (int)(b / tiles);
  int64_t tm, tn;
  grouped_order(b % tiles, p.tiles_m, p.tiles_n, 4, tm, tn);
  const int64_t m0 = tm * BM, n0 = tn * (BN / 2);
  const int64_t M = p.M, N = p.N;
  const int KB = P.KB;
  typedef Operand<BM, NW, false> OA;
  typedef Operand<BN, NW, false> OB;
  OA oa;
  OB ob;
  oa.init(p.A, p.a_bytes, p.lda, [&](int i) { return m0 + i < M ? m0 + i : M - 1; }, m0, 0, w, lane);
  ob.init(p.B, p.b_bytes, p.ldb,
          [&](int i) -> int64_t {
            const int64_t n = n0 + i / 32 * 16 + i % 16;
            return (n < N ? n : N - 1) + (i / 16 % 2 ? N : 0);
          },
          n0, N, w, lane);
  // row scales: wave w copies those of rows 64 (w % (BM/64)) .. +63, so each is
  // written more than once (the same bytes to the same place, and no branch that
  // would blur the count of outstanding copies). Weight scales: float 2v is that
  // of wave column v's sixteen gate columns (one weight block), 2v + 1 of their up
  // columns.
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(P.As, (uint32_t)(M * KB * SB));
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(P.Ws, (uint32_t)((2 * N + P.bn - 1) / P.bn * KB * SB));
  const int sq = w % (BM / 64);
  const int64_t srow = m0 + sq * 64 + lane;
  const uint32_t soff = (uint32_t)((srow < M ? srow : M - 1) * KB * SB);
  const int64_t nv = n0 + lane / 2 % (WN * NC) * 16, nc = nv < N ? nv : N - 16;
  const uint32_t woff = (uint32_t)((nc + (lane % 2 ? N : 0)) / P.bn * KB * SB);
  const int k_b = (int)((int64_t)s * KB / p.S), k_e = (int)((int64_t)(s + 1) * KB / p.S);
  f32x4 acc[NC][FM][2];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < FM; ++i) acc[c][i][0] = acc[c][i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto issue = [&](int kt, uint8_t* __restrict__ l) {
    const int64_t left = p.C - (int64_t)kt * 64;
    oa.issue(kt, left, l, w);
    ob.issue(kt, left, l + BM * 128, w);
    uint8_t* const ls = l + (BM + BN) * 128;
    const uint32_t at = scale_at(left, kt * SB);
    if constexpr (KS == 128) {
      b2l4(rs, left > 0 ? soff : kNowhere, at, ls + sq * 64 * SB);
      b2l4(rw, left > 0 ? woff : kNowhere, at, ls + BM * SB);
    } else {
      b2l16(rs, left > 0 ? soff : kNowhere, at, ls + sq * 64 * SB);
      b2l16(rw, left > 0 ? woff : kNowhere, at, ls + BM * SB);
    }
  };
  auto step = [&](int kt, uint8_t* __restrict__ nl, const uint8_t* __restrict__ la) {
    const uint8_t* const lb = la + BM * 128;
    const float* const ls = reinterpret_cast<const float*>(la + (BM + BN) * 128);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((NST - 2) * (OA::kLoads + OB::kLoads + 2)) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue(kt + NST - 1, nl);
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    if constexpr (KS == 128) {
      static_assert(NC == 1, "one column block");
      f32x4 sc[FM];
#pragma unroll
      for (int i = 0; i < FM; ++i) sc[i] = *reinterpret_cast<const f32x4*>(ls + wm * (16 * FM) + i * 16 + 4 * g);
      const float cg = ls[BM + 2 * wn], cu = ls[BM + 2 * wn + 1];
      auto frag = [&](const uint8_t* l, int row) {
        const i32x4 lo = OA::frag(l, row, 0, lane), hi = OA::frag(l, row, 1, lane);
        return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
      };
      const i32x8 fg = frag(lb, wn * 32), fu = frag(lb, wn * 32 + 16);
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const i32x8 fa = frag(la, wm * (16 * FM) + i * 16);
        // zero scale operands select the unscaled instruction
        const f32x4 pg = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa, fg, z, 0, 0, 0, 0, 0, 0);
        const f32x4 pu = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fa, fu, z, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[0][i][0][r] = __builtin_fmaf(pg[r], sc[i][r] * cg, acc[0][i][0][r]);
          acc[0][i][1][r] = __builtin_fmaf(pu[r], sc[i][r] * cu, acc[0][i][1][r]);
        }
      }
    } else {
      // block q: lane group g holds bytes 32 q + 8 g .. +7 of either operand
      auto frag = [&](const uint8_t* l, int row, int q) {
        return *reinterpret_cast<const long*>(l + swz(row + r16, 2 * q + (g >> 1)) + (g & 1) * 8);
      };
      // each product is scaled into its sum two instructions behind, and the next
      // row block's fragments are read ahead of this one's products
      constexpr int PER = NC * 8;  // products of a row block: K block, column block, gate or up
      f32x4 cw[NC][2];
      long fw[NC][2][4], fa[FM][4];
      f32x4 sc[FM], pr[3];  // sc: row r16's four blocks
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          cw[c][v] = *reinterpret_cast<const f32x4*>(ls + 4 * (BM + 2 * (wn * NC + c) + v));
#pragma unroll
          for (int q = 0; q < 4; ++q) fw[c][v][q] = frag(lb, (wn * NC + c) * 32 + 16 * v, q);
        }
      auto read = [&](int i) {
        const int row = wm * (16 * FM) + i * 16;
#pragma unroll
        for (int q = 0; q < 4; ++q) fa[i][q] = frag(la, row, q);
        sc[i] = *reinterpret_cast<const f32x4*>(ls + 4 * (row + r16));
      };
      auto fold = [&](int n) {
        const int i = n / PER, q = n % PER / (2 * NC), c = n / 2 % NC, v = n % 2;
        const float m = sc[i][q] * cw[c][v][q];
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[c][i][v][r] = __builtin_fmaf(pr[n % 3][r], m, acc[c][i][v][r]);
        asm volatile("" : "+v"(acc[c][i][v]));  // folded here, not where it is next used
      };
      read(0);
#pragma unroll
      for (int n = 0; n < FM * PER; ++n) {
        const int i = n / PER, q = n % PER / (2 * NC), c = n / 2 % NC;
        if (n % PER == 0 && i + 1 < FM) read(i + 1);
        pr[n % 3] = __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(fw[c][n % 2][q], fa[i][q], z, 0, 0, 0);
        if (n >= 2) fold(n - 2);
        __builtin_amdgcn_sched_barrier(0);
      }
      fold(FM * PER - 2);
      fold(FM * PER - 1);
    }
  };
  issue(k_b, s0);
  issue(k_b + 1, s1);
  if constexpr (NST > 3) issue(k_b + 2, s2);
  if constexpr (NST > 4) {
    issue(k_b + 3, s3);
    issue(k_b + 4, s4);
  }
  if constexpr (NST > 6) {
    issue(k_b + 5, s5);
    issue(k_b + 6, s6);
  }
  for (int kt = k_b;;) {
    if constexpr (NST == 3) {
      step(kt, s2, s0);
      if (++kt >= k_e) break;
      step(kt, s0, s1);
      if (++kt >= k_e) break;
      step(kt, s1, s2);
      if (++kt >= k_e) break;
    } else if constexpr (NST == 4) {
      step(kt, s3, s0);
      if (++kt >= k_e) break;
      step(kt, s0, s1);
      if (++kt >= k_e) break;
      step(kt, s1, s2);
      if (++kt >= k_e) break;
      step(kt, s2, s3);
      if (++kt >= k_e) break;
    } else if constexpr (NST == 6) {
      step(kt, s5, s0);
      if (++kt >= k_e) break;
      step(kt, s0, s1);
      if (++kt >= k_e) break;
      step(kt, s1, s2);
      if (++kt >= k_e) break;
      step(kt, s2, s3);
      if (++kt >= k_e) break;
      step(kt, s3, s4);
      if (++kt >= k_e) break;
      step(kt, s4, s5);
      if (++kt >= k_e) break;
    } else {
      step(kt, s7, s0);
      if (++kt >= k_e) break;
      step(kt, s0, s1);
      if (++kt >= k_e) break;
      step(kt, s1, s2);
      if (++kt >= k_e) break;
      step(kt, s2, s3);
      if (++kt >= k_e) break;
      step(kt, s3, s4);
      if (++kt >= k_e) break;
      step(kt, s4, s5);
      if (++kt >= k_e) break;
      step(kt, s5, s6);
      if (++kt >= k_e) break;
      step(kt, s6, s7);
      if (++kt >= k_e) break;
    }
  }
  wait_vmem();  // no copy outlives the workgroup's LDS
  if constexpr (KS == 32) {
    // from columns 4g .. 4g+3 of row r16 to rows 4g .. 4g+3 of column r16, as the
    // products of whole slabs come, through 1280 bytes of LDS per wave
    __syncthreads();
    float* const t = reinterpret_cast<float*>(s0) + w * 320;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          *reinterpret_cast<f32x4*>(t + 20 * r16 + 4 * g) = acc[c][i][v];
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[c][i][v][r] = t[20 * (4 * g + r) + r16];
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
  }
  const bool odd = lane & 1;
  if (p.part) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t n = n0 + (wn * NC + c) * 16 + r16;
      if (n >= N) return;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int64_t m = m0 + wm * (16 * FM) + i * 16 + 4 * g + r;
          if (m >= M) continue;
          float* q = p.part + ((int64_t)s * M + m) * 2 * N + n;
          q[0] = acc[c][i][0][r];
          q[N] = acc[c][i][1][r];
        }
    }
    return;
  }
  auto out = [&](auto BF, auto A) {
    constexpr bool kBF = decltype(BF)::value;
    uint32_t dg[NC][FM][2], du[NC][FM][2];  // loaded ahead of the first store
    if (p.delta) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int r = 0; r < 4; r += 2) {
            const int64_t m = m0 + wm * (16 * FM) + i * 16 + 4 * g + r + (odd ? 1 : 0);
            const int64_t n = n0 + (wn * NC + c) * 16 + (r16 & ~1);
            const uint16_t* const d = p.delta + (m < M ? m : M - 1) * 2 * N;
            dg[c][i][r / 2] = load2_raw(d, n, N, p.pair != 0);
            du[c][i][r / 2] = load2_raw(d + N, n, N, p.pair != 0);
          }
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
          const f32x4 ag = acc[c][i][0], au = acc[c][i][1];
          float2 G = pair_lanes(ag[r], ag[r + 1], odd), U = pair_lanes(au[r], au[r + 1], odd);
          const int64_t m = m0 + wm * (16 * FM) + i * 16 + 4 * g + r + (odd ? 1 : 0);
          const int64_t n = n0 + (wn * NC + c) * 16 + (r16 & ~1);
          if (m >= M) continue;
          if (p.delta) {
            const uint32_t d = dg[c][i][r / 2], e = du[c][i][r / 2];
            G.x += lo_f32<kBF>(d);
            G.y += hi_f32<kBF>(d);
            U.x += lo_f32<kBF>(e);
            U.y += hi_f32<kBF>(e);
          }
          gated_out<kBF, decltype(A)::value>(p, m, n, G, U, p.pair != 0);
        }
  };
  act_switch(P.act, [&](auto A) {
    if (P.bf16) out(std::true_type{}, A);
    else out(std::false_type{}, A);
  });
}

// ------------------------------------------------------------------------------
// Block-scaled FP8, tiles of 256 x 256 (K blocks of 128)
// ------------------------------------------------------------------------------
// Two operands in 128-byte slabs (one K block) of two halves each, two stages of
// LDS per half, and a slab as four products of halves in the order A0 B0, A0 B1,
// A1 B1, A1 B0, each a phase: copy one half of a later slab into the stage that
// the phases before have read, read this phase's fragments, wait for what was
// read and for what the next phase reads (vmcnt, never down to zero), barrier,
// matrix instructions, barrier. A half is copied five to seven phases before it
// is read. Waves 4 to 7 run half a phase behind waves 0 to 3 (an extra barrier
// ahead of the loop): the two waves of a SIMD take turns, one in its matrix
// instructions while the other reads and waits.
// A slab's products come out of the matrix cores on their own and are scaled
// into the sums two instructions behind, in their shadow; the last two of a
// phase after its closing barrier, beside the other waves' matrix instructions.
// The weight is operand 0 here, so a lane's four values share one row scale (one
// multiplication per row block and weight block instead of four). Row scales
// travel with their half of A, the weight scales with A0. Needs the wave's 32
// gate columns, and their up columns, in one weight block each.
// H = 1, a half tile of 128 rows: two phases a slab (A0 B0, A0 B1), three stages
// of A0 and of either B half, each copied four phases before it is read; 4.5
// rounds of tiles 550 -> 533 us.
// 4096 x 7168 x 2x9216: 533 us (2.03 PFLOP/s); the two-barrier schedule of
// tile16_body needs more registers than there are (62 spilled: 907 us).
// LDS of gated8: stages of half a slab. A half of A carries its rows' scales and
// (A0) the weight scales.
constexpr int kA8 = 128 * 128 + 768, kB8 = 128 * 128;

template <int H>
__device__ __forceinline__ void gated8_body(const T8Params& P, int64_t m0, int64_t n0, uint8_t* __restrict__ a00,
                                            uint8_t* __restrict__ a01, uint8_t* __restrict__ a10,
                                            uint8_t* __restrict__ a11, uint8_t* __restrict__ b00,
                                            uint8_t* __restrict__ b01, uint8_t* __restrict__ b10,
                                            uint8_t* __restrict__ b11, uint8_t* __restrict__ b12) {
  constexpr int NW = 8, WN = 4, FM = 4, FN = 2;
  const T16Params& p = P.t;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / WN, wn = w % WN;
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t M = p.M, N = p.N;
  const int KB = P.KB;
  typedef Operand<128, NW, false> Op;
  constexpr int L = Op::kLoads;
  Op oa[2], ob[2];
  uint32_t soff[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    oa[h].init(p.A, p.a_bytes, p.lda, [&](int i) { return m0 + h * 128 + i < M ? m0 + h * 128 + i : M - 1; }, 0, 0, w,
               lane);
    ob[h].init(p.B, p.b_bytes, p.ldb, [&](int i) { return (n0 + i < N ? n0 + i : N - 1) + (h ? N : 0); }, 0, 0, w, lane);
    const int64_t m = m0 + h * 128 + (w % 2) * 64 + lane;
    soff[h] = (uint32_t)((m < M ? m : M - 1) * KB * 4);
  }
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(P.As, (uint32_t)(M * KB * 4));
  const __amdgpu_buffer_rsrc_t rw = make_rsrc(P.Ws, (uint32_t)((2 * N + P.bn - 1) / P.bn * KB * 4));
  // float 2v: wave column v's gate block, 2v + 1: its up block
  const int64_t nv = n0 + lane / 2 % WN * 32, nc = nv < N ? nv : N - 32;
  const uint32_t woff = (uint32_t)((nc + (lane % 2 ? N : 0)) / P.bn * KB * 4);
  auto left = [&](int k) { return p.C - (int64_t)k * 64; };
  auto issue_a0 = [&](int k, uint8_t* l) {
    oa[0].issue(k, left(k), l, w);
    const uint32_t at = scale_at(left(k), k * 4);
    b2l4(rs, left(k) > 0 ? soff[0] : kNowhere, at, l + 128 * 128 + w % 2 * 256);
    b2l4(rw, left(k) > 0 ? woff : kNowhere, at, l + 128 * 128 + 512);
  };
  auto issue_a1 = [&](int k, uint8_t* l) {
    oa[1].issue(k, left(k), l, w);
    b2l4(rs, left(k) > 0 ? soff[1] : kNowhere, scale_at(left(k), k * 4), l + 128 * 128 + w % 2 * 256);
  };
  constexpr int A0 = L + 2, A1 = L + 1, B = L;
  f32x4 acc[H][2][FM][FN];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int v = 0; v < 2; ++v)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[h][v][i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  i32x8 fa[FM], fb0[2][FN], fb1[FN];
  float sa[FM], wg = 0.f, wu = 0.f;
  f32x4 pr[3];
  auto frag = [&](const uint8_t* l, int row) {
    const i32x4 lo = Op::frag(l, row, 0, lane), hi = Op::frag(l, row, 1, lane);
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  auto read_a = [&](const uint8_t* l) {
#pragma unroll
    for (int i = 0; i < FM; ++i) fa[i] = frag(l, wm * 64 + i * 16);
#pragma unroll
    for (int i = 0; i < FM; ++i)
      sa[i] = reinterpret_cast<const float*>(l + 128 * 128)[wm * 64 + i * 16 + r16];
  };
  auto read_b = [&](const uint8_t* l, i32x8 (&f)[FN]) {
#pragma unroll
    for (int j = 0; j < FN; ++j) f[j] = frag(l, wn * 32 + j * 16);
  };
  auto meet = [&](auto n) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(n)::value) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  auto fold = [&](f32x4 (&c)[FM][FN], int n, float ws) {
    const int i = n / FN, j = n % FN;
    const float sc = sa[i] * ws;
#pragma unroll
    for (int r = 0; r < 4; ++r) c[i][j][r] = __builtin_fmaf(pr[n % 3][r], sc, c[i][j][r]);
    asm volatile("" : "+v"(c[i][j]));  // folded here, not where it is next used
  };
  auto products = [&](f32x4 (&c)[FM][FN], const i32x8 (&f)[FN], float ws) {
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int n = 0; n < FM * FN; ++n) {
      pr[n % 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f[n % FN], fa[n / FN], z, 0, 0, 0, 0, 0, 0);
      if (n >= 2) fold(c, n - 2, ws);
      __builtin_amdgcn_sched_barrier(0);
    }
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    fold(c, FM * FN - 2, ws);
    fold(c, FM * FN - 1, ws);
  };
  if constexpr (H == 2) {
    auto slab = [&](int k, uint8_t* a0, uint8_t* a1, uint8_t* b0, uint8_t* b1, uint8_t* xa1, const uint8_t* xb0,
                    i32x8 (&cur)[FN], i32x8 (&nxt)[FN]) {
      issue_a1(k + 1, xa1);
      read_a(a0);
      wg = reinterpret_cast<const float*>(a0 + 128 * 128 + 512)[2 * wn];
      wu = reinterpret_cast<const float*>(a0 + 128 * 128 + 512)[2 * wn + 1];
      meet(std::integral_constant<int, 2 * A1 + A0 + 2 * B>{});      // B1 of this slab
      products(acc[0][0], cur, wg);
      issue_a0(k + 2, a0);
      read_b(b1, fb1);
      meet(std::integral_constant<int, 2 * A0 + A1 + 2 * B>{});      // A1 of this slab
      products(acc[0][1], fb1, wu);
      ob[0].issue(k + 2, left(k + 2), b0, w);
      read_a(a1);
      meet(std::integral_constant<int, A0 + A1 + 2 * B>{});          // B0 of the next slab
      products(acc[1][1], fb1, wu);
      ob[1].issue(k + 2, left(k + 2), b1, w);
      read_b(xb0, nxt);
      meet(std::integral_constant<int, A0 + A1 + 4 * B>{});          // A0 of the next slab
      products(acc[1][0], cur, wg);
    };
    issue_a0(0, a00);
    ob[0].issue(0, left(0), b00, w);
    ob[1].issue(0, left(0), b10, w);
    issue_a1(0, a10);
    issue_a0(1, a01);
    ob[0].issue(1, left(1), b01, w);
    ob[1].issue(1, left(1), b11, w);
    meet(std::integral_constant<int, A0 + A1 + 3 * B>{});            // A0 and B0 of slab 0
    read_b(b00, fb0[0]);
    meet(std::integral_constant<int, A0 + A1 + 3 * B>{});
    if (wm == 1) __builtin_amdgcn_s_barrier();
    int k = 0;
    for (; k + 1 < KB; k += 2) {
      slab(k, a00, a10, b00, b10, a11, b01, fb0[0], fb0[1]);
      slab(k + 1, a01, a11, b01, b11, a10, b00, fb0[1], fb0[0]);
    }
    if (k < KB) slab(k, a00, a10, b00, b10, a11, b01, fb0[0], fb0[1]);
    if (wm == 0) __builtin_amdgcn_s_barrier();
  } else {
    auto slab = [&](int kv, uint8_t* a, uint8_t* b0, uint8_t* b1, uint8_t* xb1, const uint8_t* xb0, i32x8 (&cur)[FN],
                    i32x8 (&nxt)[FN]) {
      const int k = __builtin_amdgcn_readfirstlane(kv);  // the compiler keeps this count in a vector register
      ob[0].issue(k + 3, left(k + 3), b0, w);
      ob[1].issue(k + 2, left(k + 2), xb1, w);
      read_a(a);
      wg = reinterpret_cast<const float*>(a + 128 * 128 + 512)[2 * wn];
      wu = reinterpret_cast<const float*>(a + 128 * 128 + 512)[2 * wn + 1];
      meet(std::integral_constant<int, 2 * A0 + 4 * B>{});         // B1 of this slab, B0 of the next
      products(acc[0][0], cur, wg);
      issue_a0(k + 3, a);
      read_b(b1, fb1);
      read_b(xb0, nxt);
      meet(std::integral_constant<int, 2 * A0 + 4 * B>{});         // A of the next slab
      products(acc[0][1], fb1, wu);
    };
    ob[0].issue(0, left(0), b00, w);
    issue_a0(0, a00);
    ob[0].issue(1, left(1), b01, w);
    ob[1].issue(0, left(0), b10, w);
    issue_a0(1, a01);
    ob[0].issue(2, left(2), a11, w);
    ob[1].issue(1, left(1), b11, w);
    issue_a0(2, a10);
    meet(std::integral_constant<int, 2 * A0 + 4 * B>{});           // A and B0 of slab 0
    read_b(b00, fb0[0]);
    meet(std::integral_constant<int, 2 * A0 + 4 * B>{});
    if (wm == 1) __builtin_amdgcn_s_barrier();
    for (int k = 0;;) {
      slab(k, a00, b00, b10, b12, b01, fb0[0], fb0[1]);
      if (++k >= KB) break;
      slab(k, a01, b01, b11, b10, a11, fb0[1], fb0[0]);
      if (++k >= KB) break;
      slab(k, a10, a11, b12, b11, b00, fb0[0], fb0[1]);
      if (++k >= KB) break;
      slab(k, a00, b00, b10, b12, b01, fb0[1], fb0[0]);
      if (++k >= KB) break;
      slab(k, a01, b01, b11, b10, a11, fb0[0], fb0[1]);
      if (++k >= KB) break;
      slab(k, a10, a11, b12, b11, b00, fb0[1], fb0[0]);
      if (++k >= KB) break;
    }
    if (wm == 0) __builtin_amdgcn_s_barrier();
  }
  wait_vmem();       // no copy outlives the workgroup's LDS
  __syncthreads();   // nor meets the epilogue's use of it
  // lane (g, r16): columns 4g .. 4g+3 of row r16 of every block
  const bool bf = P.bf16 != 0, vec = p.pair != 0;
  const int64_t nw = n0 + wn * 32;
  // a wave's own 16 KB: delta's sixteen rows x 32 columns (1 KB) of every row block,
  // gate and up, copied in 64-byte runs (read by the lanes as they need it, each
  // row's eight bytes are a request: 4096 x 7168 x 2x2048 135 us against 130, 117
  // without delta)
  uint8_t* const mine = wm == 0 ? (wn == 0 ? a00 : wn == 1 ? a01 : wn == 2 ? a10 : a11)
                                : (wn == 0 ? b00 : wn == 1 ? b01 : wn == 2 ? b10 : b11);
  const bool staged = p.delta && vec && N <= 1 << 20;  // 32-bit offsets inside the tile's rows
  if (staged) {
    const int64_t last = M - 1 - m0;
    const __amdgpu_buffer_rsrc_t rd = make_rsrc(p.delta + m0 * 2 * N, (uint32_t)((last < 255 ? last + 1 : 256) * 4 * N));
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int64_t row = h * 128 + wm * 64 + i * 16 + lane / 4;
        const uint32_t off = (uint32_t)((row < last ? row : last) * 4 * N + (nw < N ? nw : N - 32) * 2 + lane % 4 * 16);
        b2l16(rd, off, 0, mine + (h * FM + i) * 2048);
        b2l16(rd, off + (uint32_t)(2 * N), 0, mine + (h * FM + i) * 2048 + 1024);
      }
    wait_vmem();
  }
  auto delta4 = [&](int h, int i, int v, int64_t m, int64_t n) {
    if (!staged) return load_bias4(p.delta + (m * 2 + v) * N, n, N, bf, vec);
    return load_bias4(mine + (h * FM + i) * 2048 + v * 1024 + r16 * 64, n - nw, 32, bf, true);
  };
  act_switch(P.act, [&](auto A) {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const int64_t m = m0 + h * 128 + wm * 64 + i * 16 + r16;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const int64_t n = nw + j * 16 + 4 * g;
          if (p.delta && m < M && n < N) {
            acc[h][0][i][j] += delta4(h, i, 0, m, n);
            acc[h][1][i][j] += delta4(h, i, 1, m, n);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[h][0][i][j][r] = act_f32<decltype(A)::value>(acc[h][0][i][j][r]) * acc[h][1][i][j][r];
        }
      }
  });
  if (!P.q) {
    // sixteen rows x 32 columns at a time through 1 KB of the same, so that eight
    // lanes store a row's 64 bytes
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        uint8_t* const ti = mine + (i & 1) * 1024;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const f32x4 v = acc[h][0][i][j];
          const uint2 o = bf ? uint2{pack2<true>(v[0], v[1]), pack2<true>(v[2], v[3])}
                             : uint2{pack2<false>(v[0], v[1]), pack2<false>(v[2], v[3])};
          *reinterpret_cast<uint2*>(ti + r16 * 64 + ((j * 4 + g) ^ (r16 & 7)) * 8) = o;
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int row = c * 8 + lane / 8, piece = lane % 8;
          const uint2 o = *reinterpret_cast<const uint2*>(ti + row * 64 + (piece ^ (row & 7)) * 8);
          const int64_t m = m0 + h * 128 + wm * 64 + i * 16 + row, n = nw + piece * 4;
          if (m < M && n < N) {
            uint16_t* q = static_cast<uint16_t*>(p.D) + m * N + n;
            if (vec) {
              *reinterpret_cast<uint2*>(q) = o;
            } else {
              q[0] = (uint16_t)o.x;
              q[1] = (uint16_t)(o.x >> 16);
              q[2] = (uint16_t)o.y;
              q[3] = (uint16_t)(o.y >> 16);
            }
          }
        }
      }
    return;
  }
  // quantized: the tile's 128 columns are one group; the four waves of a row range
  // meet their maxima in LDS
  float* const amax = reinterpret_cast<float*>(b12);  // [WN][256]
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      float a = 0.0f;
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) a = __builtin_fmaxf(a, __builtin_fabsf(acc[h][0][i][j][r]));
      a = __builtin_fmaxf(a, __shfl_xor(a, 16, 64));
      a = __builtin_fmaxf(a, __shfl_xor(a, 32, 64));
      if (g == 0) amax[wn * 256 + h * 128 + wm * 64 + i * 16 + r16] = a;
    }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      const int row = h * 128 + wm * 64 + i * 16 + r16;
      const int64_t m = m0 + row;
      if (m >= M) continue;
      float a = amax[row];
#pragma unroll
      for (int v = 1; v < WN; ++v) a = __builtin_fmaxf(a, amax[v * 256 + row]);
      const float sc = __builtin_fmaxf(a, 1e-10f) / 448.0f;
      if (wn == 0 && g == 0) P.qs[m * (N / 128) + n0 / 128] = sc;
#pragma unroll
      for (int j = 0; j < FN; ++j)
        *reinterpret_cast<uint32_t*>(P.q + m * N + nw + j * 16 + 4 * g) = fp8_codes4(acc[h][0][i][j], sc);
    }
}

__global__ __launch_bounds__(512, 2) void gated8(T8Params P) {
  __shared__ __attribute__((aligned(1024))) uint8_t a00[kA8];
  __shared__ __attribute__((aligned(1024))) uint8_t a01[kA8];
  __shared__ __attribute__((aligned(1024))) uint8_t a10[kA8];
  __shared__ __attribute__((aligned(1024))) uint8_t a11[kA8];
  __shared__ __attribute__((aligned(1024))) uint8_t b00[kB8];
  __shared__ __attribute__((aligned(1024))) uint8_t b01[kB8];
  __shared__ __attribute__((aligned(1024))) uint8_t b10[kB8];
  __shared__ __attribute__((aligned(1024))) uint8_t b11[kB8];
  __shared__ __attribute__((aligned(1024))) uint8_t b12[kB8];
  const T16Params& p = P.t;
  const HalfTile t = half_tile(p);
  const int64_t n0 = t.tn * 128;
  if (!t.half) gated8_body<2>(P, t.m0, n0, a00, a01, a10, a11, b00, b01, b10, b11, b12);
  else if (t.m0 < p.M) gated8_body<1>(P, t.m0, n0, a00, a01, a10, a11, b00, b01, b10, b11, b12);
}

// Outputs from the S ranges' sums: four columns per thread; quantized, 32 threads
// hold a group of 128 columns.
__global__ __launch_bounds__(256) void gated8_sum(T8Params P) {
  const T16Params& p = P.t;
  const int64_t N = p.N, quads = N / 4;
  const int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (v >= p.M * quads) return;  // whole groups of 32 threads: N is then a multiple of 128
  const int64_t m = v / quads, n = (v - m * quads) * 4;
  f32x4 G = {0.f, 0.f, 0.f, 0.f}, U = {0.f, 0.f, 0.f, 0.f};
  const float* q = p.part + m * 2 * N + n;
  for (int s = 0; s < p.S; ++s, q += p.M * 2 * N) {
    G += *reinterpret_cast<const f32x4*>(q);
    U += *reinterpret_cast<const f32x4*>(q + N);
  }
  const bool bf = P.bf16 != 0;
  if (p.delta) {
    G += load_bias4(p.delta + m * 2 * N, n, N, bf, p.pair != 0);
    U += load_bias4(p.delta + m * 2 * N + N, n, N, bf, p.pair != 0);
  }
  f32x4 h;
  act_switch(P.act, [&](auto A) {
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = act_f32<decltype(A)::value>(G[r]) * U[r];
  });
  if (!P.q) {
    uint16_t* o = static_cast<uint16_t*>(p.D) + m * N + n;
    const uint2 c = bf ? uint2{pack2<true>(h[0], h[1]), pack2<true>(h[2], h[3])}
                       : uint2{pack2<false>(h[0], h[1]), pack2<false>(h[2], h[3])};
    if (p.pair) {
      *reinterpret_cast<uint2*>(o) = c;
    } else {
      o[0] = (uint16_t)c.x;
      o[1] = (uint16_t)(c.x >> 16);
      o[2] = (uint16_t)c.y;
      o[3] = (uint16_t)(c.y >> 16);
    }
    return;
  }
  float a = __builtin_fmaxf(__builtin_fmaxf(__builtin_fabsf(h[0]), __builtin_fabsf(h[1])),
                            __builtin_fmaxf(__builtin_fabsf(h[2]), __builtin_fabsf(h[3])));
  a = wave_max_xor(a, 32);
  const float sc = __builtin_fmaxf(a, 1e-10f) / 448.0f;
  if (threadIdx.x % 32 == 0) P.qs[m * (N / 128) + n / 128] = sc;
  *reinterpret_cast<uint32_t*>(P.q + m * N + n) = fp8_codes4(h, sc);
}

// Sixteen rows at most, K blocks of 128: gated_stream for FP8 operands. Lane groups 0
// and 1 receive gate values, 2 and 3 up values, each with its half's weight scale.
// Quantized, h goes to part in float32 for gated_quant.
template <int NW, int R>
__global__ __launch_bounds__(NW * 64) void gated8_stream(T8Params P) {
  __shared__ f32x4 red[NW][64];
  const T16Params& p = P.t;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t I = p.N, M = p.M, K = 2 * p.C;
  const int KB = P.KB;
  const int64_t n0 = (int64_t)blockIdx.x * 8;  // I is a multiple of 16
  const int c_b = (int)((int64_t)w * KB / NW), c_e = (int)((int64_t)(w + 1) * KB / NW);
  const uint8_t* wp = static_cast<const uint8_t*>(p.B) + (n0 + (r16 & 7) + (r16 < 8 ? 0 : I)) * K + 32 * g;
  const int64_t m = r16 < M ? r16 : M - 1;
  const uint8_t* ap = static_cast<const uint8_t*>(p.A) + m * K + 32 * g;
  const float* asp = P.As + m * KB;
  // bn is a multiple of 16: one weight-scale block per half
  const float* wsp = P.Ws + ((n0 + (g < 2 ? 0 : I)) / P.bn) * KB;
  auto load32 = [](const uint8_t* q) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(q), hi = *reinterpret_cast<const i32x4*>(q + 16);
    return i32x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  };
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  const f32x4 z = {0.f, 0.f, 0.f, 0.f};
  for (int c0 = c_b; c0 < c_e; c0 += R) {
    i32x8 wf[R], af[R];
    float sa[R], sw[R];
#pragma unroll
    for (int u = 0; u < R; ++u) {
      const int c = c0 + u < c_e ? c0 + u : c_e - 1;
      wf[u] = load32(wp + (int64_t)c * 128);
      sw[u] = wsp[c];
      af[u] = load32(ap + (int64_t)c * 128);
      sa[u] = asp[c];
    }
#pragma unroll
    for (int u = 0; u < R; ++u) {
      if (c0 + u >= c_e) break;
      const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[u], af[u], z, 0, 0, 0, 0, 0, 0);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(d[r], sa[u] * sw[u], acc[r]);
    }
  }
  red[w][lane] = acc;
  __syncthreads();
  if (tid >= 128) return;
  const int c = tid & 7, row = tid >> 3;
  const int64_t n = n0 + c;
  if (row >= M) return;
  const float* redf = reinterpret_cast<const float*>(red);
  float G = 0.f, U = 0.f;
#pragma unroll
  for (int ww = 0; ww < NW; ++ww) {
    const float* q = redf + ww * 256;
    G += q[((c >> 2) * 16 + row) * 4 + (c & 3)];
    U += q[((2 + (c >> 2)) * 16 + row) * 4 + (c & 3)];
  }
  auto f32_of = [&](uint16_t h) { return P.bf16 ? bf16_bits_to_f32(h) : f16_bits_to_f32(h); };
  if (p.delta) {
    G += f32_of(p.delta[row * 2 * I + n]);
    U += f32_of(p.delta[row * 2 * I + I + n]);
  }
  float h = 0.0f;
  act_switch(P.act, [&](auto A) { h = act_f32<decltype(A)::value>(G) * U; });
  if (P.q) p.part[row * I + n] = h;
  else static_cast<uint16_t*>(p.D)[row * I + n] = (uint16_t)(P.bf16 ? f32_to_bf16_bits(h) : f32_to_f16_bits(h));
}

// Codes and scales of h [M, I] float32 in groups of 128 (one half-wave per
// group, four consecutive values per lane).
__global__ __launch_bounds__(256) void gated_quant(T8Params P) {
  const T16Params& p = P.t;
  const int64_t groups = p.M * (p.N / 128);
  const int64_t gi = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (gi >= groups) return;
  const int l = threadIdx.x & 31;
  const f32x4 v = *reinterpret_cast<const f32x4*>(p.part + gi * 128 + 4 * l);
  float a = __builtin_fmaxf(__builtin_fmaxf(__builtin_fabsf(v[0]), __builtin_fabsf(v[1])),
                            __builtin_fmaxf(__builtin_fabsf(v[2]), __builtin_fabsf(v[3])));
  a = wave_max_xor(a, 32);
  const float s = __builtin_fmaxf(a, 1e-10f) / 448.0f;
  if (l == 0) P.qs[gi] = s;
  *reinterpret_cast<uint32_t*>(P.q + gi * 128 + 4 * l) = fp8_codes4(v, s);
}

// ------------------------------------------------------------------------------
// Gradients of the pre-activations
// ------------------------------------------------------------------------------
// dgu [M, ld] = [dG | dU | 0]: rounded once to the operands' type, as the
// matrix cores take it (one 16-bit rounding per product term; the sums stay in
// float32). f16: a power of two is taken out of all of them first, so that the
// largest finite one lies in [2^14, 2^15) (a value above f16's largest would make
// a whole row of dx and of dW infinite, and gradients of 1e-6 keep four bits as
// they are); gated_grad_max finds it, the products put it back. Columns 2I .. ld
// are zeros, so dx's contraction runs over whole slabs. out: an optional second
// copy [M, 2I] without padding, as it is. Bound by memory:
// 10 M I bytes (4096 x 2x7168: 294 MB, 47 us); gated_grad_max reads 6 M I more
// (176 MB, 44 us; 1003 x 2x1021: 4.4 us). VEC: eight columns per thread (I a
// multiple of 8, 16-byte aligned rows), else one.
template <bool BF, int ACT, bool VEC>
struct GradLoad {
  static constexpr int V = VEC ? 8 : 1;
  uint32_t d[VEC ? 4 : 1], g[VEC ? 4 : 1], u[VEC ? 4 : 1];
  // columns n .. n + V - 1 of row m
  __device__ __forceinline__ GradLoad(const uint16_t* dh, const uint16_t* gu, int64_t m, int64_t n, int64_t I) {
    const uint16_t* const pd = dh + m * I + n;
    const uint16_t* const pg = gu + m * 2 * I + n;
    if constexpr (VEC) {
      const uint4 dq = *reinterpret_cast<const uint4*>(pd), gq = *reinterpret_cast<const uint4*>(pg),
                  uq = *reinterpret_cast<const uint4*>(pg + I);
      d[0] = dq.x, d[1] = dq.y, d[2] = dq.z, d[3] = dq.w;
      g[0] = gq.x, g[1] = gq.y, g[2] = gq.z, g[3] = gq.w;
      u[0] = uq.x, u[1] = uq.y, u[2] = uq.z, u[3] = uq.w;
    } else {
      d[0] = pd[0], g[0] = pg[0], u[0] = pg[I];
    }
  }
  // dG and dU of column i
  __device__ __forceinline__ float2 grad(int i) const {
    auto at = [&](const uint32_t (&w)[VEC ? 4 : 1]) {
      return i % 2 ? hi_f32<BF>(w[i / 2]) : lo_f32<BF>(w[i / 2]);
    };
    float a;
    const float da = act_grad_f32<ACT>(at(g), a), dv = at(d);
    return float2{dv * at(u) * da, dv * a};
  }
};

// f16: the largest finite |dG| and |dU| of each workgroup's columns.
// Indices in 32 bits: M ld stays below 2^31.
constexpr int kMaxima = 512, kMaxThreads = 1024;

template <int ACT, bool VEC>
__global__ __launch_bounds__(kMaxThreads) void gated_grad_max(const uint16_t* __restrict__ dh,
                                                              const uint16_t* __restrict__ gu, float* __restrict__ maxima,
                                                              int64_t M, int64_t I) {
  __shared__ float red[kMaxThreads / 64];
  typedef GradLoad<false, ACT, VEC> Load;
  const uint32_t per = (uint32_t)(I / Load::V), total = (uint32_t)M * per;
  float top = 0.0f;
  for (uint32_t i = blockIdx.x * kMaxThreads + threadIdx.x; i < total; i += gridDim.x * kMaxThreads) {
    const uint32_t m = i / per, n = (i - m * per) * Load::V;
    const Load q(dh, gu, m, n, I);
#pragma unroll
    for (int c = 0; c < Load::V; ++c) {
      const float2 v = q.grad(c);
      const float x = __builtin_fabsf(v.x), y = __builtin_fabsf(v.y);
      // a comparison with NaN is false
      if (x < __builtin_inff()) top = __builtin_fmaxf(top, x);
      if (y < __builtin_inff()) top = __builtin_fmaxf(top, y);
    }
  }
  top = wave_max_xor(top, 64);
  if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = top;
  __syncthreads();
  if (threadIdx.x >= 64) return;
  top = wave_max_xor(threadIdx.x < kMaxThreads / 64 ? red[threadIdx.x] : 0.0f, 64);
  if (threadIdx.x == 0) maxima[blockIdx.x] = top;
}

// maxima: n_max <= 512 of them (0: nothing is taken out); exp: the power of two
// that the products put back.
template <bool BF, int ACT, bool VEC>
__global__ __launch_bounds__(256) void gated_grad(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gu,
                                                  uint16_t* __restrict__ dgu, int64_t ld, uint16_t* __restrict__ out,
                                                  int64_t M, int64_t I, const float* __restrict__ maxima, int n_max,
                                                  int32_t* __restrict__ exp) {
  typedef GradLoad<BF, ACT, VEC> Load;
  constexpr int V = Load::V;
  int e = 0;
  if constexpr (!BF) {
    static_assert(kMaxima <= 512, "two maxima per thread");
    __shared__ float red[4];
    const int i = threadIdx.x, j = i + 256;
    const float top = wave_max_xor(__builtin_fmaxf(i < n_max ? maxima[i] : 0.0f, j < n_max ? maxima[j] : 0.0f), 64);
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = top;
    __syncthreads();
    const float t = __builtin_fmaxf(__builtin_fmaxf(red[0], red[1]), __builtin_fmaxf(red[2], red[3]));
    e = t > 0.0f ? __builtin_amdgcn_frexp_expf(t) - 15 : 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *exp = e;
  }
  auto rounded = [&](float a, float b) {
    if constexpr (BF) return pack2<BF>(a, b);
    else return pack2<BF>(__builtin_ldexpf(a, -e), __builtin_ldexpf(b, -e));
  };
  // threads of a row: its columns, then the padding
  const uint32_t per = (uint32_t)((ld - I) / V), total = (uint32_t)M * per;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < total; i += gridDim.x * 256) {
    const int64_t m = i / per, n = (i - (uint32_t)m * per) * V;
    if constexpr (VEC) {
      if (n >= I) {
        *reinterpret_cast<uint4*>(dgu + m * ld + I + n) = uint4{0, 0, 0, 0};
        continue;
      }
      const Load q(dh, gu, m, n, I);
      uint32_t og[4], ou[4], wg[4], wu[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 a = q.grad(2 * c), b = q.grad(2 * c + 1);
        og[c] = rounded(a.x, b.x);
        ou[c] = rounded(a.y, b.y);
        wg[c] = pack2<BF>(a.x, b.x);
        wu[c] = pack2<BF>(a.y, b.y);
      }
      *reinterpret_cast<uint4*>(dgu + m * ld + n) = uint4{og[0], og[1], og[2], og[3]};
      *reinterpret_cast<uint4*>(dgu + m * ld + I + n) = uint4{ou[0], ou[1], ou[2], ou[3]};
      if (out) {
        *reinterpret_cast<uint4*>(out + m * 2 * I + n) = uint4{wg[0], wg[1], wg[2], wg[3]};
        *reinterpret_cast<uint4*>(out + m * 2 * I + I + n) = uint4{wu[0], wu[1], wu[2], wu[3]};
      }
    } else {
      if (n >= I) {
        dgu[m * ld + I + n] = 0;
        continue;
      }
      const float2 a = Load(dh, gu, m, n, I).grad(0);
      const uint32_t o = rounded(a.x, a.y);
      dgu[m * ld + n] = (uint16_t)o;
      dgu[m * ld + I + n] = (uint16_t)(o >> 16);
      if (out) {
        const uint32_t w = pack2<BF>(a.x, a.y);
        out[m * 2 * I + n] = (uint16_t)w;
        out[m * 2 * I + I + n] = (uint16_t)(w >> 16);
      }
    }
  }
}

__global__ __launch_bounds__(256) void zero16(uint16_t* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0;
}

// ------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------
int chip_cus() {
  const int c = device_cus();
  return c > 0 ? c : 256;
}

// Which tile kernel an M x N product over slabs of 64 takes, and in how many
// ranges of them. least: the slabs that a split has to save.
struct T16Plan {
  bool big;
  int64_t tiles, whole;  // big
  int edge, cols, S;     // small: rows and columns per tile, ranges
};
constexpr int kLeast16 = 28, kLeast8 = 14, kLeast8x32 = 8;
T16Plan tile16_plan(int64_t M, int64_t N, int64_t KT, bool gated, bool can_big = true, int least = kLeast16) {
  T16Plan q{};
  const int64_t cus = chip_cus();
  q.S = 1;
  // up to 64 rows, 128 columns per tile from half the chip's units on: those
  // already draw the memory's rate, and a few tiles of 64 columns more than units
  // cost a second round (FP8 I = 9216, K = 7168: 288 tiles)
  q.edge = M <= 64 ? 64 : 128;
  q.cols = q.edge == 64 && (N * (gated ? 2 : 1) + 127) / 128 < cus / 2 ? 64 : 128;
  const int64_t cols = gated ? q.cols / 2 : q.cols;
  const int64_t small = ((M + q.edge - 1) / q.edge) * ((N + cols - 1) / cols);
  // large tiles as soon as small ones take a second round, which costs as much as
  // half a round of tiles four times their size (forward at K = 4096, small against
  // large, bf16 and FP8: 512 rows I = 4096, 256 small tiles: 35, 45 us and 35, 43;
  // I = 5504, 344: 60, 51 and 62, 42; 1000 rows I = 5504, 688: 93, 83 and 88, 63)
  if (can_big && M > 64 && small > cus) {
    q.big = true;
    q.tiles = ((M + 255) / 256) * ((N + (gated ? 127 : 255)) / (gated ? 128 : 256));
    const int64_t rest = q.tiles % cus;
    q.whole = 2 * rest <= cus ? q.tiles - rest : q.tiles;
    return q;
  }
  // ranges of at least four slabs, while they leave half the chip idle and where
  // their sums cost less (one range against several: bf16 32 x 2048, I = 2048, 32
  // slabs: 10.1 us, 13.6; FP8 200 x 1024, I = 1024, 8 slabs: 11.6, 14.7, but 64 x
  // 4096, I = 2048, 32 slabs: 17.7, 15.1; with K blocks of 32, a slower slab, 200 x
  // 2048, I = 2048, 16 slabs: 25.4, 20.2)
  int64_t s = cus / small;
  const int64_t most = (KT + 3) / 4;
  if (s > most) s = most;
  q.S = s < 1 ? 1 : s > 16 ? 16 : (int)s;
  if (KT - (KT + q.S - 1) / q.S < least) q.S = 1;
  return q;
}
int64_t slabs(int64_t C) { return (C + 63) / 64; }
size_t tile16_part_bytes(int64_t M, int64_t N, int64_t C, bool gated) {
  const T16Plan q = tile16_plan(M, N, slabs(C), gated);
  return q.S > 1 ? (size_t)q.S * (size_t)M * (size_t)(gated ? 2 * N : N) * sizeof(float) : 0;
}

template <bool TRA, bool TRB, bool BF, bool GATED, int ACT>
hipError_t launch_tile16_t(T16Params p, float* part, hipStream_t st) {
  T16Plan q = tile16_plan(p.M, p.N, slabs(p.C), GATED);
  if (p.S == 1) q.S = 1;
  p.S = q.S;
  if (q.big) {
    p.tiles_m = (p.M + 255) / 256;
    p.tiles_n = (p.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
    p.whole = q.whole;
    const int64_t grid = 2 * q.tiles - q.whole;
    if (grid > 0x7FFFFFFFLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((tile16<TRA, TRB, BF, GATED, ACT>), dim3((unsigned)grid), dim3(512), 0, st, p);
    return hipGetLastError();
  }
  const int64_t cols = GATED ? q.cols / 2 : q.cols;
  p.tiles_m = (p.M + q.edge - 1) / q.edge;
  p.tiles_n = (p.N + cols - 1) / cols;
  p.part = q.S > 1 ? part : nullptr;
  const dim3 grid((unsigned)(p.tiles_m * p.tiles_n * q.S));
  if (q.cols == 64) hipLaunchKernelGGL((tile16s<64, 4, TRA, TRB, BF, GATED, ACT>), grid, dim3(512), 0, st, p);
  else if (q.edge == 64) hipLaunchKernelGGL((tile16s<64, 2, TRA, TRB, BF, GATED, ACT>), grid, dim3(512), 0, st, p);
  else hipLaunchKernelGGL((tile16s<128, 2, TRA, TRB, BF, GATED, ACT>), grid, dim3(512), 0, st, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || q.S == 1) return e;
  const int64_t pairs = p.M * ((p.N + 1) / 2);
  hipLaunchKernelGGL((tile16_sum<BF, GATED, ACT>), dim3((unsigned)((pairs + 255) / 256)), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <bool TRA, bool TRB, bool GATED, int ACT>
hipError_t launch_tile16(const T16Params& p, bool bf, float* part, hipStream_t st) {
  return bf ? launch_tile16_t<TRA, TRB, true, GATED, ACT>(p, part, st)
            : launch_tile16_t<TRA, TRB, false, GATED, ACT>(p, part, st);
}

template <int ACT>
hipError_t launch_gated_stream(const StreamParams& p, bool bf, hipStream_t st) {
  constexpr int NW = 8, U = 8;
  const int64_t grid = (p.I + 7) / 8;
  if (grid > 0x7FFFFFFFLL) return hipErrorInvalidConfiguration;
  if (bf) hipLaunchKernelGGL((gated_stream<NW, U, true, ACT>), dim3((unsigned)grid), dim3(NW * 64), 0, st, p);
  else hipLaunchKernelGGL((gated_stream<NW, U, false, ACT>), dim3((unsigned)grid), dim3(NW * 64), 0, st, p);
  return hipGetLastError();
}

// The streaming kernels: the fewest rows, and up to sixteen where the tiles leave
// half the chip idle (16-bit K = 7168, I = 2048: 4 rows 12.4 us against 14.7, 16
// rows 15.2, 15.8; else, K = 4096, I = 5504: 16 rows 25.5 us against 17.7. FP8 K = 7168, I = 2048, 16 rows: 10.6, 13.3;
// I = 9216: 4 rows 29.3, 43.5, 16 rows 45.0, 34.9).
bool gated_streams(int64_t M, int64_t I, int64_t KT) {
  if (M <= 4 || M > 16) return M <= 4;
  return tile16_plan(M, I, KT, true, true, 0).S > 1;
}

template <int ACT>
hipError_t launch_gated_act(const GatedArgs& a, hipStream_t st) {
  const bool bf = a.dtype == Q8_BF16;
  if (gated_streams(a.M, a.I, slabs(a.K))) {
    const StreamParams p{static_cast<const uint16_t*>(a.x), a.ld_x, static_cast<const uint16_t*>(a.W), a.M, a.I, a.K,
                         static_cast<const uint16_t*>(a.delta), static_cast<uint16_t*>(a.gate_up),
                         static_cast<uint16_t*>(a.h)};
    return launch_gated_stream<ACT>(p, bf, st);
  }
  T16Params p{};
  p.A = a.x; p.lda = a.ld_x; p.a_bytes = (uint32_t)(((a.M - 1) * a.ld_x + a.K) * 2);
  p.B = a.W; p.ldb = a.K; p.b_bytes = (uint32_t)(2 * a.I * a.K * 2);
  p.M = a.M; p.N = a.I; p.C = a.K;
  p.D = a.h; p.ldd = a.I;
  p.delta = static_cast<const uint16_t*>(a.delta);
  p.gate_up = static_cast<uint16_t*>(a.gate_up);
  p.pair = a.I % 2 == 0 && ((uintptr_t)a.h | (uintptr_t)a.delta | (uintptr_t)a.gate_up) % 4 == 0;
  return launch_tile16<false, false, true, ACT>(p, bf, static_cast<float*>(a.workspace), st);
}

// dgu, and the power of two that the f16 products put back, in exp (maxima: scratch)
template <int ACT>
hipError_t launch_grad_act(const GatedGradArgs& a, uint16_t* dgu, int64_t ld, uint16_t* out, float* maxima, int32_t* exp,
                           hipStream_t st) {
  const bool vec = a.I % 8 == 0 && ((uintptr_t)a.dh | (uintptr_t)a.gate_up | (uintptr_t)out) % 16 == 0;
  const auto* dh = static_cast<const uint16_t*>(a.dh);
  const auto* gu = static_cast<const uint16_t*>(a.gate_up);
  const bool bf = a.dtype == Q8_BF16;
  int n_max = 0;
  if (!bf && (a.dx || a.dW)) {
    const int64_t blocks = (a.M * (a.I / (vec ? 8 : 1)) + kMaxThreads - 1) / kMaxThreads;
    n_max = blocks < kMaxima ? (int)blocks : kMaxima;
    hipLaunchKernelGGL((vec ? gated_grad_max<ACT, true> : gated_grad_max<ACT, false>), dim3(n_max), dim3(kMaxThreads), 0,
                       st, dh, gu, maxima, a.M, a.I);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int64_t total = a.M * (ld - a.I) / (vec ? 8 : 1);
  const int64_t blocks = (total + 255) / 256;
  const dim3 gr((unsigned)(blocks < 65536 ? blocks : 65536)), bl(256);
  const auto kern = vec ? (bf ? gated_grad<true, ACT, true> : gated_grad<false, ACT, true>)
                        : (bf ? gated_grad<true, ACT, false> : gated_grad<false, ACT, false>);
  hipLaunchKernelGGL(kern, gr, bl, 0, st, dh, gu, dgu, ld, out, a.M, a.I, maxima, n_max, exp);
  return hipGetLastError();
}

int64_t grad_ld(int64_t I) { return (2 * I + 63) / 64 * 64; }

}  // namespace

hipError_t launch_gated(const GatedArgs& a, hipStream_t st) {
  if (a.act == kSilu) return launch_gated_act<kSilu>(a, st);
  if (a.act == kGelu) return launch_gated_act<kGelu>(a, st);
  return launch_gated_act<kGeluTanh>(a, st);
}

size_t gated_bytes(int64_t M, int64_t I, int64_t K) {
  return gated_streams(M, I, slabs(K)) ? 0 : tile16_part_bytes(M, I, K, true);
}

// Whether dx and dW go out in one launch: their times in slabs of the small tile
// kernel, one after the other (the second launch costs about as much as kLaunch
// slabs, ranges' sums as kSums) against the longer contraction's tiles with the
// others behind them.
static bool one_launch(const T16Params& x, const T16Params& w) {
  const int64_t cus = chip_cus(), kLaunch = 6, kSums = 12;
  int64_t apart = kLaunch, tiles[2], len[2];
  for (int i = 0; i < 2; ++i) {
    const T16Params& p = i ? w : x;
    const T16Plan q = tile16_plan(p.M, p.N, slabs(p.C), false);
    if (q.big || q.edge != 128) return false;
    tiles[i] = ((p.M + 127) / 128) * ((p.N + 127) / 128);
    len[i] = slabs(p.C);
    apart += (tiles[i] * q.S + cus - 1) / cus * ((len[i] + q.S - 1) / q.S) + (q.S > 1 ? kSums : 0);
  }
  const int l = len[1] > len[0];  // longer contraction; at most one round of either
  const int64_t n = tiles[1 - l], d = len[1 - l], free_now = cus - tiles[l];
  int64_t t = len[l];
  while (free_now * (t / d) + tiles[l] * ((t - len[l]) / d) < n) ++t;
  return t < apart;
}

// the padded gradients of the pre-activations, the maxima and the power of two
// (f16), then the ranges' sums of dx or dW
static size_t dgu_bytes_of(int64_t M, int64_t I) { return (size_t)M * (size_t)grad_ld(I) * 2; }
constexpr size_t kMaximaBytes = kMaxima * sizeof(float) + 16;
size_t gated_grad_bytes(int64_t M, int64_t I, int64_t K) {
  if (M == 0) return 0;
  const size_t x = tile16_part_bytes(M, K, grad_ld(I), false), w = tile16_part_bytes(2 * I, K, M, false);
  return dgu_bytes_of(M, I) + kMaximaBytes + (x > w ? x : w);
}

hipError_t launch_gated_backward(const GatedGradArgs& a, hipStream_t st) {
  const bool bf = a.dtype == Q8_BF16;
  if (a.M == 0) {  // no rows: dW is an empty sum
    hipLaunchKernelGGL(zero16, dim3(1024), dim3(256), 0, st, static_cast<uint16_t*>(a.dW), 2 * a.I * a.K);
    return hipGetLastError();
  }
  const int64_t ld = grad_ld(a.I);
  uint16_t* dgu = static_cast<uint16_t*>(a.workspace);
  uint16_t* out = static_cast<uint16_t*>(a.d_gate_up);
  float* maxima = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + dgu_bytes_of(a.M, a.I));
  int32_t* exp = reinterpret_cast<int32_t*>(maxima + kMaxima);
  float* part = maxima + kMaximaBytes / sizeof(float);
  hipError_t e = a.act == kSilu   ? launch_grad_act<kSilu>(a, dgu, ld, out, maxima, exp, st)
                 : a.act == kGelu ? launch_grad_act<kGelu>(a, dgu, ld, out, maxima, exp, st)
                                  : launch_grad_act<kGeluTanh>(a, dgu, ld, out, maxima, exp, st);
  if (e != hipSuccess) return e;
  const uint32_t dgu_bytes = (uint32_t)(a.M * ld * 2);
  T16Params x{}, w{};
  x.A = dgu; x.lda = ld; x.a_bytes = dgu_bytes;
  x.B = a.W; x.ldb = a.K; x.b_bytes = (uint32_t)(2 * a.I * a.K * 2);
  x.M = a.M; x.N = a.K; x.C = ld;
  x.D = a.dx; x.ldd = a.K;
  x.pair = (uintptr_t)a.dx % 4 == 0;  // K is a multiple of 8
  w.A = dgu; w.lda = ld; w.a_bytes = dgu_bytes;
  w.B = a.x; w.ldb = a.ld_x; w.b_bytes = (uint32_t)(((a.M - 1) * a.ld_x + a.K) * 2);
  w.M = 2 * a.I; w.N = a.K; w.C = a.M; w.a_cols = ld;
  w.D = a.dW; w.ldd = a.K;
  w.pair = (uintptr_t)a.dW % 4 == 0;
  x.exp = w.exp = exp;
  const bool one = one_launch(x, w);
  // a gradient comes out the same whether or not the other is asked for
  if (one) x.S = w.S = 1;
  if (one && a.dx && a.dW) {
    for (T16Params* p : {&x, &w}) {
      p->tiles_m = (p->M + 127) / 128;
      p->tiles_n = (p->N + 127) / 128;
    }
    const dim3 grid((unsigned)(x.tiles_m * x.tiles_n + w.tiles_m * w.tiles_n)), block(512);
    const int x_first = x.C >= w.C;
    if (bf) hipLaunchKernelGGL(tile16s_both<true>, grid, block, 0, st, x, w, x_first);
    else hipLaunchKernelGGL(tile16s_both<false>, grid, block, 0, st, x, w, x_first);
    return hipGetLastError();
  }
  if (a.dx) e = launch_tile16<false, true, false, 0>(x, bf, part, st);
  if (a.dW && e == hipSuccess) e = launch_tile16<true, true, false, 0>(w, bf, part, st);
  return e;
}

// ---- block-scaled FP8 ------------------------------------------------------------
namespace {
// 256-row tiles: K blocks of 128, and the 32 columns of a wave in one weight block
T16Plan gated8_plan(int64_t M, int64_t I, int64_t K, int bn, int bk) {
  T16Plan q = tile16_plan(M, I, K / 128, true, bk == 128 && bn % 32 == 0 && I % 32 == 0,
                          bk == 128 ? kLeast8 : kLeast8x32);
  if (bk == 32 && q.cols == 128 && q.edge == 128) {
    // 256 columns per tile (64 x 64 per wave, fewer reads and barriers per product)
    // cost 1.75 rounds of 128 (4096 x 7168: I = 9216 1107 us against 1258, I = 2048
    // 253, 289; but 1000 x 4096, I = 5504, two rounds against three, 147, 134)
    const int64_t cus = chip_cus(), tm = (M + 127) / 128;
    const int64_t wide = (tm * ((I + 127) / 128) + cus - 1) / cus, narrow = (tm * ((I + 63) / 64) + cus - 1) / cus;
    if (7 * wide <= 4 * narrow) q.cols = 256;
  }
  return q;
}
bool gated8_streams(int64_t M, int64_t I, int64_t K, int bk) { return bk == 128 && gated_streams(M, I, K / 128); }

template <int KS>
void launch_gated8s(const T8Params& P, const T16Plan& q, hipStream_t st) {
  const dim3 grid((unsigned)(P.t.tiles_m * P.t.tiles_n * q.S)), block(512);
  if (q.cols == 64) hipLaunchKernelGGL((gated8s<KS, 64, 4, 1>), grid, block, 0, st, P);
  else if (q.edge == 64) hipLaunchKernelGGL((gated8s<KS, 64, 2, 1>), grid, block, 0, st, P);
  else if (KS == 32 && q.cols == 256) hipLaunchKernelGGL((gated8s<32, 128, 2, 2>), grid, block, 0, st, P);
  else hipLaunchKernelGGL((gated8s<KS, 128, 2, 1>), grid, block, 0, st, P);
}
}  // namespace

// float32 sums of K ranges, or of all of a quantized call in small tiles, or
// float32 h of a quantized call of few rows
size_t blockwise_gated_workspace_bytes(int64_t M, int64_t I, int64_t K, int bn, int bk, bool quant) {
  if (gated8_streams(M, I, K, bk)) return quant ? (size_t)M * (size_t)I * sizeof(float) : 0;
  const T16Plan q = gated8_plan(M, I, K, bn, bk);
  if (q.big || (q.S == 1 && !quant)) return 0;
  return (size_t)q.S * (size_t)M * (size_t)(2 * I) * sizeof(float);
}

hipError_t launch_blockwise_gated(const BlockGatedArgs& a, hipStream_t st) {
  T8Params P{};
  T16Params& p = P.t;
  p.A = a.A; p.lda = a.K / 2; p.a_bytes = (uint32_t)(a.M * a.K);
  p.B = a.W; p.ldb = a.K / 2; p.b_bytes = (uint32_t)(2 * a.I * a.K);
  p.M = a.M; p.N = a.I; p.C = a.K / 2;
  p.D = a.D; p.ldd = a.I;
  p.delta = static_cast<const uint16_t*>(a.delta);
  p.pair = ((uintptr_t)a.D | (uintptr_t)a.delta) % 8 == 0;
  p.part = static_cast<float*>(a.workspace);
  P.As = a.As; P.Ws = a.Ws; P.KB = (int)(a.K / 128); P.bn = a.bn;
  P.q = a.Dq; P.qs = a.Ds; P.bf16 = a.dtype == Q8_BF16; P.act = a.act;
  if (gated8_streams(a.M, a.I, a.K, a.bk)) {
    constexpr int NW = 8, R = 4;
    hipLaunchKernelGGL((gated8_stream<NW, R>), dim3((unsigned)(a.I / 8)), dim3(NW * 64), 0, st, P);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.Dq) return e;
    const int64_t groups = a.M * (a.I / 128);
    hipLaunchKernelGGL(gated_quant, dim3((unsigned)((groups + 7) / 8)), dim3(256), 0, st, P);
    return hipGetLastError();
  }
  const T16Plan q = gated8_plan(a.M, a.I, a.K, a.bn, a.bk);
  p.S = q.S;
  const int rows = q.big ? 256 : q.edge, cols = q.big ? 128 : q.cols / 2;
  p.tiles_m = (a.M + rows - 1) / rows;
  p.tiles_n = (a.I + cols - 1) / cols;
  if (p.tiles_m * p.tiles_n * (q.big ? 2 : q.S) > 0x7FFFFFFFLL) return hipErrorInvalidConfiguration;
  if (q.big) {
    p.whole = q.whole;
    hipLaunchKernelGGL(gated8, dim3((unsigned)(2 * q.tiles - q.whole)), dim3(512), 0, st, P);
    return hipGetLastError();
  }
  const bool sum = q.S > 1 || a.Dq;
  if (!sum) p.part = nullptr;
  if (a.bk == 128) launch_gated8s<128>(P, q, st);
  else launch_gated8s<32>(P, q, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !sum) return e;
  const int64_t quads = a.M * (a.I / 4);
  hipLaunchKernelGGL(gated8_sum, dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, st, P);
  return hipGetLastError();
}

}  // namespace q8
