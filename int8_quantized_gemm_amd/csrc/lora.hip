// Low-rank adapters of many requests at once, beside a shared projection.
//
//   out[m] = base[m] + s_a (x[m] A_a^T) B_a^T,   a = ids[m]   (a < 0: base[m])
//   x [M, K], A [L, R, K], B [L, N, R], base and out [M, N]
//
// V[m] = x[m] A_a^T in float32 comes first, K split over the grid, as partial
// sums [S][M][Rp] in the caller's workspace; the product of their sum with B_a
// is then added to the base.
//
// Few rows (decode): lora_shrink and lora_expand, one workgroup per tile of
// sixteen rows and adapter among them, operands straight from memory;
// lora_expand sums the partials itself.
// More: lora_shrink_tile (64 rows, operands through LDS), lora_join (sums the
// partials and splits them into two 16-bit terms, once per row) and
// lora_expand_tile (up to 256 rows by 256 columns); each workgroup works through
// the adapters among its rows, one for rows of one request.
//
// Rows are taken as they come: requests whose rows lie together cost one pass
// and no sorting launch is needed. A row's result depends on its own adapter
// and row only: products of the other rows are computed beside it in the same
// matrix instruction and dropped by a select, never by a multiplication with
// zero.
#include <type_traits>

#include "mma16.h"
#include "q8_internal.h"
#include "tile_common.h"

namespace q8 {
namespace {

constexpr int kMaxSplits = 8;  // K ranges of the shrinking product at most

struct LoraParams {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t* A;
  const uint16_t* B;
  const int32_t* ids;
  const float* scaling;
  const uint16_t* base;
  int64_t ldb;
  uint16_t* out;
  int64_t ldo;
  float* part;
  uint16_t* hi;   // terms of the scaled sums, in operand order (lora_join)
  uint16_t* lo;
  int32_t* exps;  // [M] powers of two taken out of them
  int64_t M, N, K;
  int R, Rp, L, S;
  int nb;   // blocks of sixteen rows per workgroup of lora_expand_tile
  int vec;  // out and base rows 8-byte aligned, N a multiple of 4
};

// adapter of row m: -1 for none (negative or not below L)
__device__ __forceinline__ int row_adapter(const LoraParams& p, int64_t m) {
  if (m >= p.M) return -1;
  const int a = p.ids[m];
  return (unsigned)a < (unsigned)p.L ? a : -1;
}

// One workgroup: rows [16 b, +16), the K range s of S and the blockIdx.z-th
// adapter among the rows. The waves split the K range, load the next chunks
// before the products of these, and are summed in order through LDS.
template <int RT, bool BF>
__global__ __launch_bounds__(256) void lora_shrink(LoraParams p) {
  constexpr int NW = 4;
  __shared__ f32x4 red[NW][RT][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int s = blockIdx.y;
  const int64_t K = p.K;
  // lane l < 16: the adapter of row m0 + l
  const int mine = lane < 16 ? row_adapter(p, m0 + lane) : -1;
  uint64_t todo = __ballot(mine >= 0), rows = 0;
  int a = -1;
  for (int slot = (int)blockIdx.z; todo; --slot) {
    a = __builtin_amdgcn_readfirstlane(__shfl(mine, __builtin_ctzll(todo), 64));
    rows = __ballot(mine == a);
    if (slot == 0) break;
    todo &= ~rows;
  }
  if (!todo) return;
  const int NC = (int)((K + 31) / 32);
  const int per = (NC + p.S - 1) / p.S;
  const int sb = s * per < NC ? s * per : NC, se = sb + per < NC ? sb + per : NC;
  const int c_b = sb + (int)((int64_t)w * (se - sb) / NW), c_e = sb + (int)((int64_t)(w + 1) * (se - sb) / NW);
  const int64_t mr = m0 + r16 < p.M ? m0 + r16 : p.M - 1;
  const uint16_t* xp = p.x + mr * p.ldx + 8 * g;
  const uint16_t* ap[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int rr = 16 * r + r16 < p.R ? 16 * r + r16 : p.R - 1;
    ap[r] = p.A + ((int64_t)a * p.R + rr) * K + 8 * g;
  }
  f32x4 acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
  const i32x4 zero = {0, 0, 0, 0};
  constexpr int U = RT <= 2 ? 4 : RT <= 4 ? 2 : 1;
  i32x4 af[2][U][RT], xf[2][U];
  auto load = [&](int q, int c0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = (int64_t)(c0 + u) * 32;
      const bool in = c0 + u < c_e && k + 8 * g < K;
      xf[q][u] = in ? *reinterpret_cast<const i32x4*>(xp + k) : zero;
#pragma unroll
      for (int r = 0; r < RT; ++r) af[q][u][r] = in ? *reinterpret_cast<const i32x4*>(ap[r] + k) : zero;
    }
  };
  auto products = [&](int q) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int r = 0; r < RT; ++r) acc[r] = mfma16<BF>(af[q][u][r], xf[q][u], acc[r]);
  };
  load(0, c_b);
  for (int c0 = c_b; c0 < c_e; c0 += 2 * U) {
    load(1, c0 + U);
    products(0);
    load(0, c0 + 2 * U);
    products(1);
  }
#pragma unroll
  for (int r = 0; r < RT; ++r) red[w][r][lane] = acc[r];
  __syncthreads();
  // lane (g, r16): ranks 16 r + 4g .. +3 of row m0 + r16
  for (int r = w; r < RT; r += NW) {
    f32x4 v = red[0][r][lane];
#pragma unroll
    for (int ww = 1; ww < NW; ++ww) v += red[ww][r][lane];
    if (16 * r < p.Rp && ((rows >> r16) & 1))
      *reinterpret_cast<f32x4*>(p.part + ((int64_t)s * p.M + m0 + r16) * p.Rp + 16 * r + 4 * g) = v;
  }
}

// More rows: 64 rows by all ranks per workgroup and K range, 64-deep slabs of x
// (64 rows) and A_a (16 RT rows) copied into a ring of four LDS stages, three
// slabs ahead of their products. Wave w multiplies rows 16 w .. 16 w + 15.
// 4096 x 7168, rank 64: 20 us (2.9 TB/s of x); straight from memory, where a
// fragment load touches sixteen rows, 47 us; slabs of 128 K elements copied
// together, half as many barriers, 22 us.
template <int RT, bool BF>
__global__ __launch_bounds__(256) void lora_shrink_tile(LoraParams p) {
  constexpr int NW = 4;
  constexpr int AQ = 2 * RT;                   // 1 KB copies of A per slab
  constexpr int LA = (AQ + NW - 1) / NW, LX = 2;
  constexpr int kStage = 64 * 128 + RT * 16 * 128;
  __shared__ __attribute__((aligned(1024))) uint8_t s0[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s1[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s2[kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t s3[kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  // consecutive workgroups of an XCD take one tile's K ranges, then the next
  // tile's: its L2 holds the one or two adapters of its rows, not all of them
  const int64_t b = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t m0 = b / p.S * 64;
  const int s = (int)(b % p.S);
  const int64_t K = p.K;
  const int NC = (int)((K + 63) / 64);
  const int c_b = (int)((int64_t)s * NC / p.S), c_e = (int)((int64_t)(s + 1) * NC / p.S);
  const int mine = row_adapter(p, m0 + lane);
  uint64_t todo = __ballot(mine >= 0);
  // copy q = w + 4c fills stage rows 8q .. 8q+7: lane l's chunk l % 8 of row
  // 8q + l/8 holds logical chunk (l % 8) ^ key; copies past the last one of A
  // repeat an earlier one (the same bytes to the same place), so every wave
  // counts the same number of them
  const int chunk = (lane & 7) ^ ((4 * (w & 1) + (lane >> 4)) & 7);
  // 32-bit offsets from the tile's first row; rows past the last repeat it
  const int64_t mlast = p.M - 1 - m0 < 63 ? p.M - 1 - m0 : 63;
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(p.x + m0 * p.ldx, (uint32_t)((mlast * p.ldx + K) * 2));
  uint32_t xoff[LX];
#pragma unroll
  for (int c = 0; c < LX; ++c) {
    const int64_t r = 8 * (w + NW * c) + (lane >> 3);
    xoff[c] = (uint32_t)(((r < mlast ? r : mlast) * p.ldx + chunk * 8) * 2);
  }
  while (todo) {
    const int a = __builtin_amdgcn_readfirstlane(__shfl(mine, __builtin_ctzll(todo), 64));
    const uint64_t rows = __ballot(mine == a);
    todo &= ~rows;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.A + (int64_t)a * p.R * K, (uint32_t)((int64_t)p.R * K * 2));
    uint32_t aoff[LA];
    int aq[LA];
#pragma unroll
    for (int c = 0; c < LA; ++c) {
      aq[c] = w + NW * c < AQ ? w + NW * c : w % 2;  // the swizzle key goes by q's parity, w's
      const int r = 8 * aq[c] + (lane >> 3);
      aoff[c] = (uint32_t)(((int64_t)(r < p.R ? r : p.R - 1) * K + chunk * 8) * 2);
    }
    // chunks past K, and slabs past the last, have an offset beyond any buffer:
    // they read as zeros in both operands
    auto issue = [&](int kt, uint8_t* st) {
      const bool in = (int64_t)kt * 64 + chunk * 8 < K;
#pragma unroll
      for (int c = 0; c < LX; ++c) b2l16(rx, in ? xoff[c] : 0xFFFFFFF0u, kt * 128, st + (w + NW * c) * 1024);
#pragma unroll
      for (int c = 0; c < LA; ++c) b2l16(ra, in ? aoff[c] : 0xFFFFFFF0u, kt * 128, st + 64 * 128 + aq[c] * 1024);
    };
    f32x4 acc[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) acc[r] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto step = [&](int kt, uint8_t* refill, const uint8_t* st) {
      // this slab has landed (two later ones may be in flight), for every wave;
      // and every wave has read the slab before
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * (LX + LA)) : "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      issue(kt + 3, refill);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const i32x4 xf = *reinterpret_cast<const i32x4*>(st + swz(16 * w + r16, 4 * h + g));
#pragma unroll
        for (int r = 0; r < RT; ++r)
          acc[r] = mfma16<BF>(*reinterpret_cast<const i32x4*>(st + 64 * 128 + swz(16 * r + r16, 4 * h + g)), xf, acc[r]);
      }
    };
    issue(c_b, s0);
    issue(c_b + 1, s1);
    issue(c_b + 2, s2);
    int kt = c_b;
    for (; kt + 4 <= c_e; kt += 4) {
      step(kt, s3, s0);
      step(kt + 1, s0, s1);
      step(kt + 2, s1, s2);
      step(kt + 3, s2, s3);
    }
    if (kt < c_e) step(kt, s3, s0);
    if (kt + 1 < c_e) step(kt + 1, s0, s1);
    if (kt + 2 < c_e) step(kt + 2, s1, s2);
    // no copy outlives the workgroup's LDS or meets the next adapter's
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if ((rows >> (16 * w + r16)) & 1) {
#pragma unroll
      for (int r = 0; r < RT; ++r)
        if (16 * r < p.Rp)
          *reinterpret_cast<f32x4*>(p.part + ((int64_t)s * p.M + m0 + 16 * w + r16) * p.Rp + 16 * r + 4 * g) = acc[r];
    }
  }
}

// Operand 1 of the expanding product from a row's eight float32 values: two
// 16-bit terms hi + lo, scaled by a power of two so that the row's largest
// value lies in [0.5, 1) (f16 then neither overflows nor loses small rows).
template <bool BF>
__device__ __forceinline__ void split16(const float (&v)[8], i32x4& hi, i32x4& lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = pack2<BF>(v[2 * i], v[2 * i + 1]);
    const float l0 = v[2 * i] - lo_f32<BF>(h), l1 = v[2 * i + 1] - hi_f32<BF>(h);
    hi[i] = (int)h;
    // infinite or NaN values stay what they are in hi
    lo[i] = (int)pack2<BF>(l0 - l0 == 0.0f ? l0 : 0.0f, l1 - l1 == 0.0f ? l1 : 0.0f);
  }
}

// The larger of big and |v| where v is finite: infinities and NaN stay what they
// are in any scale, and the finite values beside them need theirs.
__device__ __forceinline__ float larger_finite(float big, float v) {
  const float a = __builtin_fabsf(v);
  return a < __builtin_inff() ? __builtin_fmaxf(big, a) : big;
}

// Power of two just above big (0 where big is 0).
__device__ __forceinline__ int row_exp(float big) { return big > 0.0f ? __builtin_amdgcn_frexp_expf(big) : 0; }

// The expanding product has the rows' terms as operand 0 and B_a's rows (output
// columns) as operand 1, column 4 r16 + j of a wave's 64 in MFMA j: lane (g, r16)
// receives four adjacent columns of rows 4g .. 4g+3, and the sixteen lanes of a
// row read and write 128 consecutive bytes. (With the operands exchanged a
// lane holds one row's columns and adjacent lanes lie rows apart: every lane is
// then a memory request of its own, and base and output of 4096 x 7168 took
// twice as long.)
template <int KT>
__device__ __forceinline__ void load_b(const LoraParams& p, int a, int64_t n0, int lane, i32x4 (&bf)[KT][4]) {
  const int g = lane >> 4, r16 = lane & 15;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    int64_t n = n0 + 4 * r16 + j;
    if (n >= p.N) n = p.N - 1;
    const uint16_t* bp = p.B + ((int64_t)a * p.N + n) * p.R + 8 * g;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
      bf[kt][j] = 32 * kt + 8 * g < p.R ? *reinterpret_cast<const i32x4*>(bp + 32 * kt) : i32x4{0, 0, 0, 0};
  }
}

// Four columns n .. n+3 of row m of the base as float32.
template <bool BF, bool VEC>
__device__ __forceinline__ uint2 load_base(const LoraParams& p, int64_t m, int64_t n) {
  uint2 b = {0u, 0u};
  if (!p.base || n >= p.N) return b;
  const uint16_t* q = p.base + m * p.ldb + n;
  if constexpr (VEC) {
    b = *reinterpret_cast<const uint2*>(q);
  } else {
    b.x = q[0];
    if (n + 1 < p.N) b.x |= (uint32_t)q[1] << 16;
    if (n + 2 < p.N) b.y = q[2];
    if (n + 3 < p.N) b.y |= (uint32_t)q[3] << 16;
  }
  return b;
}

template <bool BF, bool VEC>
__device__ __forceinline__ void store_row(const LoraParams& p, int64_t m, int64_t n, const float (&v)[4], uint2 b) {
  if (n >= p.N) return;
  uint2 o;
  if (p.base) {
    o.x = pack2<BF>(v[0] + lo_f32<BF>(b.x), v[1] + hi_f32<BF>(b.x));
    o.y = pack2<BF>(v[2] + lo_f32<BF>(b.y), v[3] + hi_f32<BF>(b.y));
  } else {
    o.x = pack2<BF>(v[0], v[1]);
    o.y = pack2<BF>(v[2], v[3]);
  }
  uint16_t* q = p.out + m * p.ldo + n;
  if constexpr (VEC) {
    *reinterpret_cast<uint2*>(q) = o;
  } else {
    q[0] = (uint16_t)o.x;
    if (n + 1 < p.N) q[1] = (uint16_t)(o.x >> 16);
    if (n + 2 < p.N) q[2] = (uint16_t)o.y;
    if (n + 3 < p.N) q[3] = (uint16_t)(o.y >> 16);
  }
}

// Decode: rows [16 b, +16) x 256 columns (64 per wave) of the blockIdx.z-th
// adapter among the rows; slot 0 also stores the rows without one. The base
// and B are loaded ahead of the partial sums.
template <int KT, bool BF, bool VEC>
__global__ __launch_bounds__(256) void lora_expand(LoraParams p) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  const int64_t m0 = (int64_t)blockIdx.x * 16;
  const int64_t n0 = (int64_t)blockIdx.y * 256 + w * 64;
  const int64_t N = p.N, M = p.M;
  if (n0 >= N) return;
  const int mine = lane < 16 ? row_adapter(p, m0 + lane) : -1;
  const uint64_t live = __ballot(mine >= 0);
  const uint64_t inside = M - m0 >= 16 ? 0xFFFFull : (1ull << (M - m0)) - 1;
  uint64_t todo = live, rows = 0;
  int a = -1;
  for (int slot = (int)blockIdx.z; todo; --slot) {
    a = __builtin_amdgcn_readfirstlane(__shfl(mine, __builtin_ctzll(todo), 64));
    rows = __ballot(mine == a);
    if (slot == 0) break;
    todo &= ~rows;
  }
  if (!todo) rows = 0;
  const uint32_t store = (uint32_t)(blockIdx.z == 0 ? rows | (inside & ~live) : rows);
  if (store == 0) return;
  const int64_t n = n0 + 4 * r16;
  uint2 base[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if ((store >> (4 * g + r)) & 1) base[r] = load_base<BF, VEC>(p, m0 + 4 * g + r, n);
  f32x4 d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (rows) {
    const float sc = p.scaling ? p.scaling[a] : 1.0f;
    i32x4 bf[KT][4];
    load_b<KT>(p, a, n0, lane, bf);
    const bool in = (rows >> r16) & 1;
    float v[KT][8];
    float big = 0.0f;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      f32x4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = {0.f, 0.f, 0.f, 0.f};
      if (in && 32 * kt + 8 * g < p.R) {
        const float* q = p.part + (m0 + r16) * p.Rp + 32 * kt + 8 * g;
        for (int s = 0; s < p.S; ++s, q += M * p.Rp) {
          x0 += *reinterpret_cast<const f32x4*>(q);
          x1 += *reinterpret_cast<const f32x4*>(q + 4);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[kt][i] = x0[i] * sc;
        v[kt][4 + i] = x1[i] * sc;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) big = larger_finite(big, v[kt][i]);
    }
    big = __builtin_fmaxf(big, __shfl_xor(big, 16, 64));
    big = __builtin_fmaxf(big, __shfl_xor(big, 32, 64));
    const int e = row_exp(big);  // of row r16
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = __builtin_ldexpf(v[kt][i], -e);
      i32x4 hi, lo;
      split16<BF>(u, hi, lo);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = mfma16<BF>(lo, bf[kt][j], d[j]);
        d[j] = mfma16<BF>(hi, bf[kt][j], d[j]);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int er = __shfl(e, 4 * g + r, 64);
      const bool ok = (rows >> (4 * g + r)) & 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j][r] = ok ? __builtin_ldexpf(d[j][r], er) : 0.0f;
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if ((store >> (4 * g + r)) & 1) {
      const float v[4] = {d[0][r], d[1][r], d[2][r], d[3][r]};
      store_row<BF, VEC>(p, m0 + 4 * g + r, n, v, base[r]);
    }
}

// The rows' sums over the K ranges, scaled and split into two 16-bit terms of
// [0.5, 1) times a power of two (sixteen lanes per row, eight ranks each), in
// operand order: sixteen rows and 32 ranks are 64 lanes' sixteen bytes, so that
// lora_expand_tile loads them as they are (from rows of R values, again one
// memory request per lane). Ranks past R are zeros.
template <bool BF>
__global__ __launch_bounds__(256) void lora_join(LoraParams p) {
  const int64_t m = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int l = threadIdx.x & 15;
  const int KT = (p.R + 31) / 32;
  if (m >= p.M) return;
  f32x4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = {0.f, 0.f, 0.f, 0.f};
  // every range's loads before the first sum, and before the row's adapter is
  // known (rows without one hold nothing that is used)
  f32x4 y[kMaxSplits][2];
  if (8 * l < p.R) {
    const float* q = p.part + m * p.Rp + 8 * l;
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s) {
      const float* at = q + (int64_t)(s < p.S ? s : 0) * p.M * p.Rp;
      y[s][0] = *reinterpret_cast<const f32x4*>(at);
      y[s][1] = *reinterpret_cast<const f32x4*>(at + 4);
    }
  }
  const int a = row_adapter(p, m);
  if (a < 0) return;
  const float sc = p.scaling ? p.scaling[a] : 1.0f;
  if (8 * l < p.R) {
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s) {
      if (s >= p.S) break;
      x0 += y[s][0];
      x1 += y[s][1];
    }
  }
  float v[8], big = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = (i < 4 ? x0[i & 3] : x1[i & 3]) * sc;
    big = larger_finite(big, v[i]);
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) big = __builtin_fmaxf(big, __shfl_xor(big, d, 64));
  const int e = row_exp(big);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __builtin_ldexpf(v[i], -e);
  i32x4 hi, lo;
  split16<BF>(v, hi, lo);
  if (l >= 4 * KT) return;
  const int64_t at = (((m >> 4) * KT + (l >> 2)) * 64 + (l & 3) * 16 + (m & 15)) * 8;
  *reinterpret_cast<i32x4*>(p.hi + at) = hi;
  *reinterpret_cast<i32x4*>(p.lo + at) = lo;
  if (l == 0) p.exps[m] = e;
}

// nb blocks of sixteen rows x 256 columns (64 per wave). Each wave walks its
// blocks, the next block's base, terms and adapters loaded before
// this block's products, and keeps B_a in registers until a row of another
// adapter comes (B for every sixteen rows: 73 us instead of 46 at 4096 x 7168,
// rank 64).
template <int KT, bool BF, bool VEC>
__global__ __launch_bounds__(256) void lora_expand_tile(LoraParams p) {
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, r16 = lane & 15;
  // tile by tile, all columns of one first: an XCD's L2 then holds B of the one
  // or two adapters of its rows
  const int64_t ny = (p.N + 255) / 256;
  const int64_t b = xcd_remap(blockIdx.x, gridDim.x);
  const int64_t m0 = b / ny * (16 * p.nb);
  const int64_t n0 = b % ny * 256 + w * 64;
  const int64_t N = p.N, M = p.M;
  if (n0 >= N) return;
  const int64_t n = n0 + 4 * r16;
  struct Block {
    int id, e;  // of row r16
    i32x4 hi[KT], lo[KT];
    uint2 base[4];
  };
  auto load = [&](int t, Block& q) {
    // rows past the end repeat the last one (blocks past it the last block's
    // terms); rows without an adapter have no terms, and their products are
    // dropped
    const int64_t m = m0 + 16 * t + r16 < M ? m0 + 16 * t + r16 : M - 1;
    q.id = p.ids[m];
    q.e = p.exps[m];
    const int64_t blk = m0 + 16 * t < M ? m0 / 16 + t : (M - 1) / 16;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int64_t at = ((blk * KT + kt) * 64 + lane) * 8;
      q.hi[kt] = *reinterpret_cast<const i32x4*>(p.hi + at);
      q.lo[kt] = *reinterpret_cast<const i32x4*>(p.lo + at);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t mr = m0 + 16 * t + 4 * g + r;
      q.base[r] = load_base<BF, VEC>(p, mr < M ? mr : M - 1, n);
    }
  };
  i32x4 bf[KT][4];
  int have = -1;
  auto block = [&](int t, Block& q) {
    const int64_t mt = m0 + 16 * t;
    const int mine = mt + r16 < M && (unsigned)q.id < (unsigned)p.L ? q.id : -1;
    f32x4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint32_t todo = (uint32_t)(__ballot(mine >= 0) & 0xFFFFu);
    while (todo) {
      const int a = __builtin_amdgcn_readfirstlane(__shfl(mine, __builtin_ctz(todo), 64));
      const uint32_t rows = (uint32_t)(__ballot(mine == a) & 0xFFFFu);
      todo &= ~rows;
      if (a != have) {
        load_b<KT>(p, a, n0, lane, bf);
        have = a;
      }
      f32x4 d[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[j] = mfma16<BF>(q.lo[kt], bf[kt][j], d[j]);
          d[j] = mfma16<BF>(q.hi[kt], bf[kt][j], d[j]);
        }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int er = __shfl(q.e, 4 * g + r, 64);
        const bool ok = (rows >> (4 * g + r)) & 1;
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j][r] = ok ? __builtin_ldexpf(d[j][r], er) : acc[j][r];
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (mt + 4 * g + r < M) {
        const float v[4] = {acc[0][r], acc[1][r], acc[2][r], acc[3][r]};
        store_row<BF, VEC>(p, mt + 4 * g + r, n, v, q.base[r]);
      }
  };
  const int64_t blocks = (M - m0 + 15) / 16;
  const int T = blocks < p.nb ? (int)blocks : p.nb;
  Block q0, q1;
  load(0, q0);
  for (int t = 0; t < T; t += 2) {
    load(t + 1, q1);
    block(t, q0);
    if (t + 1 < T) {
      load(t + 2, q0);
      block(t + 1, q1);
    }
  }
}

// ------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------
int lora_rp(int R) { return (R + 15) / 16 * 16; }

// lora_shrink, else lora_shrink_tile: a workgroup per adapter of sixteen rows
// keeps up with 64-row tiles up to here, and is not slowed by rows of different
// adapters side by side (K = N = 4096, 300 rows of rank 16: 14.0 us either way with
// one adapter, 28 against 48 us with sixteen in turn; 1000 rows of rank 64: 23
// against 20 us and 101 against 86)
constexpr int64_t kSlotRows = 512;

// lora_expand, else lora_join and lora_expand_tile: one launch less while there
// are few tiles and ranks to sum the partials of (K = 2048, 517 x 1532 rank 24:
// 14.4 us against 17.4; rank 64: 17.5, 17.6; 1024 x 1532 rank 64: 21.0, 18.0;
// 517 x 7168 rank 24: 21.4, 19.7)
bool lora_direct(int64_t M, int64_t N, int R) {
  return M <= 256 || ((M + 15) / 16) * ((N + 255) / 256) * ((R + 31) / 32) <= 400;
}

// K ranges of the shrinking product (M >= 1): enough workgroups for the chip, at
// least 256 K elements per range
int lora_splits(int64_t M, int64_t K) {
  const int rows = M <= kSlotRows ? 16 : 64;
  const int64_t tiles = (M + rows - 1) / rows;
  int64_t s = (512 + tiles - 1) / tiles;
  const int64_t most = (K + 255) / 256;
  if (s > most) s = most;
  if (s > kMaxSplits) s = kMaxSplits;
  return (int)(s < 1 ? 1 : s);
}

size_t round16(size_t n) { return (n + 15) / 16 * 16; }
// one term of every row: blocks of sixteen rows by 32 ranks
size_t lora_term_bytes(int64_t M, int R) { return (size_t)((M + 15) / 16) * ((R + 31) / 32) * 1024; }
size_t lora_sum_bytes(int64_t M, int64_t K, int R) {
  return (size_t)lora_splits(M, K) * (size_t)M * (size_t)lora_rp(R) * sizeof(float);
}

template <int RT, bool BF>
hipError_t launch_shrink(const LoraParams& p, hipStream_t st) {
  if (p.M <= kSlotRows) {
    const unsigned slots = p.L < 16 ? p.L : 16;
    hipLaunchKernelGGL((lora_shrink<RT, BF>), dim3((unsigned)((p.M + 15) / 16), p.S, slots), dim3(256), 0, st, p);
  } else {
    const int64_t grid = (p.M + 63) / 64 * p.S;
    if (grid > 0x7FFFFFFFLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((lora_shrink_tile<RT, BF>), dim3((unsigned)grid), dim3(256), 0, st, p);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || lora_direct(p.M, p.N, p.R)) return e;
  hipLaunchKernelGGL((lora_join<BF>), dim3((unsigned)((p.M + 15) / 16)), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <int KT, bool BF, bool VEC>
hipError_t launch_expand_v(LoraParams p, hipStream_t st) {
  const unsigned ny = (unsigned)((p.N + 255) / 256);  // at most 65535 (checked by the front end)
  const int64_t tiles = (p.M + 15) / 16;
  if (lora_direct(p.M, p.N, p.R)) {
    const unsigned slots = p.L < 16 ? p.L : 16;
    hipLaunchKernelGGL((lora_expand<KT, BF, VEC>), dim3((unsigned)tiles, ny, slots), dim3(256), 0, st, p);
  } else {
    // the fewest blocks per workgroup with which every workgroup is resident at
    // once, three (two above rank 64) to a compute unit: 4096 x 7168, rank 64, 256
    // units, eight blocks, 896 workgroups 41 us, ten, 728 34 us
    const int cus = device_cus();
    const int64_t room = (KT <= 2 ? 3 : 2) * (int64_t)(cus > 0 ? cus : 256) / ny;
    const int64_t nb = room < 1 ? 16 : (tiles + room - 1) / room;
    p.nb = nb > 16 ? 16 : (int)nb;
    const int64_t grid = (tiles + p.nb - 1) / p.nb * ny;
    if (grid > 0x7FFFFFFFLL) return hipErrorInvalidConfiguration;
    hipLaunchKernelGGL((lora_expand_tile<KT, BF, VEC>), dim3((unsigned)grid), dim3(256), 0, st, p);
  }
  return hipGetLastError();
}

template <int KT, bool BF>
hipError_t launch_expand(const LoraParams& p, hipStream_t st) {
  return p.vec ? launch_expand_v<KT, BF, true>(p, st) : launch_expand_v<KT, BF, false>(p, st);
}

template <bool BF>
hipError_t launch_lora_t(const LoraParams& p, hipStream_t st) {
  hipError_t e;
  switch ((p.R + 15) / 16) {
    case 1: e = launch_shrink<1, BF>(p, st); break;
    case 2: e = launch_shrink<2, BF>(p, st); break;
    case 3: e = launch_shrink<3, BF>(p, st); break;
    case 4: e = launch_shrink<4, BF>(p, st); break;
    case 5: case 6: e = launch_shrink<6, BF>(p, st); break;
    default: e = launch_shrink<8, BF>(p, st); break;
  }
  if (e != hipSuccess) return e;
  switch ((p.R + 31) / 32) {
    case 1: return launch_expand<1, BF>(p, st);
    case 2: return launch_expand<2, BF>(p, st);
    case 3: return launch_expand<3, BF>(p, st);
    default: return launch_expand<4, BF>(p, st);
  }
}

}  // namespace

// partial sums, then (more than 256 rows) the two terms and the exponents
size_t lora_part_bytes(int64_t M, int64_t K, int R) {
  if (M == 0) return 0;
  size_t n = round16(lora_sum_bytes(M, K, R));
  if (M > 256) n += 2 * lora_term_bytes(M, R) + (size_t)M * 4;
  return n;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t st) {
  LoraParams p{};
  p.x = static_cast<const uint16_t*>(a.x); p.ldx = a.ld_x;
  p.A = static_cast<const uint16_t*>(a.A); p.B = static_cast<const uint16_t*>(a.B);
  p.ids = a.ids; p.scaling = a.scaling;
  p.base = static_cast<const uint16_t*>(a.base); p.ldb = a.ld_base;
  p.out = static_cast<uint16_t*>(a.out); p.ldo = a.ld_out;
  p.part = static_cast<float*>(a.workspace);
  uint8_t* q = static_cast<uint8_t*>(a.workspace) + round16(lora_sum_bytes(a.M, a.K, a.R));
  const size_t term = lora_term_bytes(a.M, a.R);
  p.hi = reinterpret_cast<uint16_t*>(q);
  p.lo = reinterpret_cast<uint16_t*>(q + term);
  p.exps = reinterpret_cast<int32_t*>(q + 2 * term);
  p.M = a.M; p.N = a.N; p.K = a.K; p.R = a.R; p.Rp = lora_rp(a.R); p.L = a.L;
  p.S = lora_splits(a.M, a.K);
  p.vec = a.N % 4 == 0 && a.ld_out % 4 == 0 && (uintptr_t)a.out % 8 == 0 &&
          (!a.base || (a.ld_base % 4 == 0 && (uintptr_t)a.base % 8 == 0));
  return a.dtype == Q8_BF16 ? launch_lora_t<true>(p, st) : launch_lora_t<false>(p, st);
}

}  // namespace q8
