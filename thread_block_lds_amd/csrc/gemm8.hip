// GEMM of two matrices in 8-bit floating point with block scales: C = A B^T (+ add).
//
//   C[m][n] = sum over groups g of 128 k:  sa(m, g) sb(n, g) sum_{k in g} A[m][k] B[n][k]   (+ add[m][n])
//
// A (M x K) and B (N x K) both keep k contiguous, so a group is 128 bytes of a row: one LDS row, one line of
// HBM, and the k depth of one v_mfma_f32_16x16x128_f8f6f4. Each group's product is formed in the matrix
// instruction from zero and added to an fp32 accumulator with one fused multiply-add by its two scales.
//
// Two arithmetics:
//   * 16-bit outputs use the 8-bit matrix instructions. Those sum eight products at a time and keep each to 2^-13 of
//     the largest of the eight (measured); on normal data the result is 1.4e-5 of its norm off, which the rounding to
//     fp16 or bf16 (2e-4, 1.7e-3) hides. Between groups everything is fp32.
//   * fp32 outputs convert both operands' codes to fp16 in registers, which is exact for e4m3 and e5m2, and use the fp16
//     instructions, whose sums are fp32 throughout.
#include <stdint.h>

#include "nt_tile.hpp"

namespace tbl {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 half2_t __attribute__((ext_vector_type(2)));

constexpr int kGroup = 128;

typedef Chunks Codes;   // the codes of 32 values as two 16-byte chunks of a row

// The same as fp16: four operands of a 16 x 16 x 32 instruction.
struct Halves {
  uint4 q[4];
};

// Two codes of a word, the lower or the upper ones.
template <int kFmt>
__device__ __forceinline__ uint32_t to_half2(uint32_t w, bool high) {
  half2_t h;
  if constexpr (kFmt == 0)
    h = high ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
  else
    h = high ? __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, 1.0f, true) : __builtin_amdgcn_cvt_scalef32_pk_f16_bf8(w, 1.0f, false);
  return __builtin_bit_cast(uint32_t, h);
}
template <int kFmt>
__device__ __forceinline__ uint4 to_halves(uint32_t a, uint32_t b) {
  return make_uint4(to_half2<kFmt>(a, false), to_half2<kFmt>(a, true), to_half2<kFmt>(b, false), to_half2<kFmt>(b, true));
}
template <int kFmt>
__device__ __forceinline__ Halves to_halves(const Codes& c) {
  return Halves{{to_halves<kFmt>(c.lo.x, c.lo.y), to_halves<kFmt>(c.lo.z, c.lo.w), to_halves<kFmt>(c.hi.x, c.hi.y),
                 to_halves<kFmt>(c.hi.z, c.hi.w)}};
}

// An operand of a group's 16 x 16 block product, as the arithmetic wants it.
template <int kFmt, bool kExact>
struct Operand;
template <int kFmt>
struct Operand<kFmt, false> {
  i32x8_t v;
  __device__ __forceinline__ void set(const Codes& c) {
    v = i32x8_t{(int)c.lo.x, (int)c.lo.y, (int)c.lo.z, (int)c.lo.w, (int)c.hi.x, (int)c.hi.y, (int)c.hi.z, (int)c.hi.w};
  }
};
template <int kFmt>
struct Operand<kFmt, true> {
  Halves v;
  __device__ __forceinline__ void set(const Codes& c) { v = to_halves<kFmt>(c); }
};

// D[n][m] over one group: lane l holds n = 4 (l / 16) .. + 3 of m = l mod 16. Which k a byte stands for does not
// matter as long as both operands agree.
template <int kFa, int kFb>
__device__ __forceinline__ f32x4_t product(const Operand<kFb, false>& b, const Operand<kFa, false>& a) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.v, a.v, f32x4_t{0, 0, 0, 0}, kFb, kFa, 0, 0, 0, 0);
}
template <int kFa, int kFb>
__device__ __forceinline__ f32x4_t product(const Operand<kFb, true>& b, const Operand<kFa, true>& a) {
  f32x4_t c = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, b.v.q[i]), __builtin_bit_cast(half8_t, a.v.q[i]), c, 0, 0, 0);
  return c;
}

// Bytes of a chunk that lie past the matrix (its row's tail may hold anything, NaN codes among it) become zero.
__device__ __forceinline__ uint4 keep_bytes(uint4 c, int n) {
  auto word = [&](uint32_t w, int at) -> uint32_t {
    const int k = n - at;
    return k >= 4 ? w : k <= 0 ? 0u : w & ((1u << (8 * k)) - 1u);
  };
  return make_uint4(word(c.x, 0), word(c.y, 4), word(c.z, 8), word(c.w, 12));
}

struct Gemm8Args {
  const uint8_t* A;
  const uint8_t* B;
  int64_t lda, ldb;
  const float* sa;
  const float* sb;
  int64_t sa_row, sa_group, sb_row, sb_group;   // floats between the scales of neighbouring (blocks of) rows and groups
  int a_shift, b_shift;                         // log2 of the rows that share a scale
  const float* add;
  void* C;
  int M, N, K, groups;
  int out;
};

// What is added to columns n .. n + 3 of row m.
__device__ __forceinline__ f32x4_t added(const Gemm8Args& a, int m, int n) {
  f32x4_t v = {0, 0, 0, 0};
  if (m >= a.M || n >= a.N) return v;
  const float* p = a.add + static_cast<int64_t>(m) * a.N + n;
  if (n + 4 <= a.N) {
    __builtin_memcpy(&v, p, 16);   // one 16-byte load, aligned or not
    return v;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < a.N) v[e] = p[e];
  return v;
}

// Four results of one row, columns n .. n + 3, rounded to the output type and written.
template <bool kF32>
__device__ __forceinline__ void put4(const Gemm8Args& a, int m, int n, f32x4_t v) {
  if (m >= a.M || n >= a.N) return;
  const int64_t at = static_cast<int64_t>(m) * a.N + n;
  const bool whole = n + 4 <= a.N;   // then one store, aligned or not
  if constexpr (kF32) {
    float* c = static_cast<float*>(a.C) + at;
    if (whole) {
      __builtin_memcpy(c, &v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) c[e] = v[e];
    }
  } else {
    uint16_t* c = static_cast<uint16_t*>(a.C) + at;
    const bool bf = a.out == 1;
    uint16_t h[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) h[e] = to_out16(v[e], bf);
    if (whole) {
      __builtin_memcpy(c, h, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (n + e < a.N) c[e] = h[e];
    }
  }
}

// A wave's sub-tile whose first row and column (of this lane) are m0 and n0. C may be add itself, so the compiler keeps every load
// behind the stores before it; the loads of four row blocks are taken together first (one at a time they cost 24 us a tile).
template <bool kF32, int TM, int TN>
__device__ __forceinline__ void put_tile(const Gemm8Args& a, int m0, int n0, f32x4_t (&acc)[TM][TN]) {
  constexpr int kAhead = TM < 4 ? TM : 4;
#pragma unroll
  for (int i0 = 0; i0 < TM; i0 += kAhead) {
    if (a.add != nullptr) {
      f32x4_t d[kAhead][TN];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) d[i][j] = added(a, m0 + (i0 + i) * 16, n0 + j * 16);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i0 + i][j] += d[i][j];
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) put4<kF32>(a, m0 + (i0 + i) * 16, n0 + j * 16, acc[i0 + i][j]);
  }
}

// The same of a wave's 16 TM x 64 sub-tile to 16 bits, two row blocks at a time through LDS (``tile``: 4 KiB, this wave's
// alone) and out as whole rows, 128 bytes of each. m0, n0: its first row and column.
template <int TM>
__device__ __forceinline__ void put_rows(const Gemm8Args& a, char* tile, int m0, int n0, f32x4_t (&acc)[TM][4]) {
  const int r = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
  const bool bf = a.out == 1;
#pragma unroll
  for (int i0 = 0; i0 < TM; i0 += 2) {
    if (a.add != nullptr) {
      f32x4_t d[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[i][j] = added(a, m0 + (i0 + i) * 16 + r, n0 + 16 * j + 4 * q);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i0 + i][j] += d[i][j];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint16_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = to_out16(acc[i0 + i][j][e], bf);
        *tile_four(tile, 16 * i + r, 16 * j + 4 * q) = make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
      }
    tile_fence();
    tile_store<2>(tile, static_cast<uint16_t*>(a.C), a.N, a.M, a.N, m0 + 16 * i0, n0, threadIdx.x & 63);
    tile_fence();
    __builtin_amdgcn_sched_barrier(0);
  }
}

// ---- tiles -----------------------------------------------------------------------------------------

// What a wave's scales are: 64 rows of A's (the first half of the waves) or of B's, one load of 4 bytes a lane and step.
struct ScaleLoad {
  const float* base;
  int64_t group;    // floats from a group to the next
  int64_t range;    // bytes that a group's rows span
  int at;           // this lane's offset
  __device__ __forceinline__ ScaleLoad(const Gemm8Args& a, int tile, int tm, int tn, int waves, int wave, int lane) {
    const bool b = wave >= waves / 2;
    const int row0 = (b ? tn : tm) * tile, row = (wave & (waves / 2 - 1)) * 64 + lane;
    const int shift = b ? a.b_shift : a.a_shift;
    const int64_t rs = b ? a.sb_row : a.sa_row;
    base = (b ? a.sb : a.sa) + (row0 >> shift) * rs;
    group = b ? a.sb_group : a.sa_group;
    range = (((tile - 1) >> shift) * rs + 1) * 4;
    at = row0 + row < (b ? a.N : a.M) ? static_cast<int>((row >> shift) * rs * 4) : kNtOut;
  }
  __device__ __forceinline__ void issue(int g, bool real, unsigned lds) const {
    load4_to_lds(make_desc(base + g * group, real ? range : 0), lds, at);
  }
};

// The group's sums of one block added to the accumulators: by the row's and the column block's scales, or (kRowB) each
// column's own.
template <bool kRowB>
__device__ __forceinline__ void add_scaled(f32x4_t& acc, const f32x4_t& p, float sa, float sb, const f32x4_t& sb4) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(p[e], kRowB ? sa * sb4[e] : sb, acc[e]);
}

// Whether two finite scales have a product beyond fp32: then a group's sum of 0 would become NaN and a small one infinite.
__device__ __forceinline__ bool beyond(float sa, float sb) {
  constexpr float inf = __builtin_huge_valf();
  return __builtin_fabsf(sa) < inf && __builtin_fabsf(sb) < inf && !(__builtin_fabsf(sa * sb) < inf);
}
// add_scaled, where scales may be beyond: those sums are taken by the smaller scale first.
template <bool kRowB>
__device__ __forceinline__ void add_scaled_wide(f32x4_t& acc, const f32x4_t& p, float sa, float sb, const f32x4_t& sb4) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float s = kRowB ? sb4[e] : sb;
    const bool wide = beyond(sa, s), less = __builtin_fabsf(s) < __builtin_fabsf(sa);
    acc[e] = wide ? __builtin_fmaf(p[e] * (less ? s : sa), less ? sa : s, acc[e]) : __builtin_fmaf(p[e], sa * s, acc[e]);
  }
}

// The loops take the product of two scales first, one multiplication a row and group instead of one a result. Where a wave's sums
// (groups g0, g0 + step, ... below g1, of the rows from m0 and columns from n0, which began at start(i, j)) are not all finite
// and its rows' largest finite scale and its columns' are beyond fp32 together, they are taken again from memory with
// add_scaled_wide. Sums that are not finite for another reason, a NaN or an infinity in a row, cost the look at the scales.
template <int kFa, int kFb, bool kRowB, bool kExact, int TM, int TN, class Start>
__device__ __forceinline__ void mend_range(const Gemm8Args& a, int g0, int g1, int step, int m0, int n0, f32x4_t (&acc)[TM][TN], Start start) {
  constexpr float inf = __builtin_huge_valf();
  float top = 0;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = __builtin_elementwise_maximum(top, __builtin_fabsf(acc[i][j][e]));   // a NaN stays
  if (__builtin_amdgcn_ballot_w64(!(top < inf)) == 0) return;
  const int r = threadIdx.x & 15, q = (threadIdx.x & 63) >> 4;
  auto scale_a = [&](int m, int g) { return a.sa[(min(m, a.M - 1) >> a.a_shift) * a.sa_row + g * a.sa_group]; };
  auto scale_b = [&](int n, int g) { return a.sb[(min(n, a.N - 1) >> a.b_shift) * a.sb_row + g * a.sb_group]; };
  // the largest finite scales of the wave's rows and columns, a row or two and a column a lane, over all of its groups
  const int lane = threadIdx.x & 63;
  float most_a = 0, most_b = 0;
  auto take = [&](float& most, float s) {
    s = __builtin_fabsf(s);
    if (s < inf) most = __builtin_fmaxf(most, s);
  };
#pragma unroll 4
  for (int g = g0; g < g1; g += step) {
#pragma unroll
    for (int m = 0; m < TM; m += 4) take(most_a, scale_a(m0 + 16 * m + (lane & (16 * TM - 1)), g));
    take(most_b, scale_b(n0 + (lane & (16 * TN - 1)), g));
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    most_a = __builtin_fmaxf(most_a, __shfl_xor(most_a, d));
    most_b = __builtin_fmaxf(most_b, __shfl_xor(most_b, d));
  }
  if (!beyond(most_a, most_b)) return;
  auto fetch = [&](const uint8_t* p, int64_t ld, int row, int rows, int g) -> Codes {   // this lane's two chunks of a row
    uint4 c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = g * kGroup + 64 * h + 16 * q;
      c[h] = make_uint4(0, 0, 0, 0);
      if (row < rows && k < a.K) c[h] = keep_bytes(*reinterpret_cast<const uint4*>(p + row * ld + k), a.K - k);
    }
    return Codes{c[0], c[1]};
  };
  // a row block at a time, with few registers: the sums of all of them are live
#pragma unroll
  for (int i = 0; i < TM; ++i) {
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = start(i, j);
#pragma unroll 1
    for (int g = g0; g < g1; g += step) {
      Operand<kFa, kExact> av;
      av.set(fetch(a.A, a.lda, m0 + 16 * i + r, a.M, g));
      const float sa = scale_a(m0 + 16 * i + r, g), sb = scale_b(n0, g);
#pragma unroll
      for (int j = 0; j < TN; ++j) {
        Operand<kFb, kExact> bv;
        bv.set(fetch(a.B, a.ldb, n0 + 16 * j + r, a.N, g));
        f32x4_t sb4 = {sb, sb, sb, sb};
        if constexpr (kRowB) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sb4[e] = scale_b(n0 + 16 * j + 4 * q + e, g);
        }
        add_scaled_wide<kRowB>(acc[i][j], product<kFa, kFb>(bv, av), sa, sb, sb4);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
}

// 256 x 256 tiles with the two-group loop of nt_tile.hpp (16-bit outputs). The scales have four slots of their own in
// LDS and are read with the operands. A compute half-period is 16 matrix instructions of 32 cycles; the
// 4 multiply-adds (kRowB: 4 products too) that follow each run beside the next one. 8192^3: 405 to 449 us, 2.45 to 2.71 PFLOP/s,
// against 3.08 of a library product of whole matrices without group scales. Bound by the board's power: the loop without the
// multiply-adds takes 376 us, and the matrix unit is busy for two thirds of the cycles of a lowered clock.
constexpr int kScaleSlot = 2 * 256 * 4;

template <int kFa, int kFb, bool kRowB>
__global__ __launch_bounds__(kNtThreads) void gemm8_tile256_kernel(Gemm8Args a, TileOrder order, Deal deal, float* __restrict__ work) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kNtStage + 4 * kScaleSlot];
  const Share share = share_of(deal, static_cast<int>(blockIdx.x));
  int tm, tn;
  order_tile(order, share.tile, tm, tn);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  NtTile t;
  t.init(lds, a.lda, a.ldb);
  const int q = t.lane >> 4, r = t.lane & 15;
  // a group that ends before its 128 values comes after the loop
  const int tail = a.K & (kGroup - 1);
  const bool odd = tail != 0 && share.s1 == a.groups;
  const int steps = share.s1 - share.s0 - (odd ? 1 : 0);
  const ScaleLoad scales(a, 256, tm, tn, 8, t.wave, t.lane);
  char* const slots = lds + 2 * kNtStage;   // step i's scales: slot i mod 4
  NtOperand oa, ob;
  i32x4_t od;
  uint64_t scale_at = reinterpret_cast<uint64_t>(scales.base + share.s0 * scales.group);
  unsigned to_slot = lds_address(slots) + t.wave * 256;
  {
    const int64_t k0 = static_cast<int64_t>(share.s0) * kGroup;
    const int kup = (a.K + 15) & ~15;   // a chunk that starts inside a row is read whole
    oa.start(a.A + static_cast<int64_t>(tm) * 256 * a.lda + k0, (min(256, a.M - tm * 256) - 1) * a.lda + kup - k0);
    ob.start(a.B + static_cast<int64_t>(tn) * 256 * a.ldb + k0, (min(256, a.N - tn * 256) - 1) * a.ldb + kup - k0);
  }
  auto advance = [&](bool real) {   // the descriptors to the next step
    oa.set(real);
    ob.set(real);
    od = make_desc(reinterpret_cast<const void*>(scale_at), real ? scales.range : 0);
    scale_at += scales.group * 4;
  };
  f32x4_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  Codes af[4], bf[4];
  float sa[4], sb = 0;
  f32x4_t sb4[4];

  // Products are used kBehind instructions after their own, in a fixed order: left to itself the compiler waits for each
  // with the matrix unit idle (493 us at 8192^3 against 462). The last three of a half-period are left to the next memory
  // half-period (settle), so the other group's instructions follow this one's without a gap.
  constexpr int kBehind = 3;
  f32x4_t p[kBehind + 1];
#pragma unroll
  for (int k = 0; k <= kBehind; ++k) p[k] = f32x4_t{0, 0, 0, 0};
  float sa_left = 0, sb_left = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) sb4[j] = f32x4_t{0, 0, 0, 0};
  bool next_real = false;
  auto column = [](int n) { return n & 4 ? 3 - (n & 3) : n & 3; };   // B forward and backward: one operand stays at every change of A
  auto settle = [&](int i0) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int m = 16 - kBehind; m < 16; ++m) add_scaled<kRowB>(acc[i0 + 3][column(m)], p[m & 3], sa_left, sa_left * sb_left, sb4[column(m)]);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](int i0) {
    Operand<kFb, false> b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j].set(bf[j]);
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      Operand<kFa, false> av;
      av.set(af[n >> 2]);
      p[n & 3] = product<kFa, kFb>(b[column(n)], av);
      __builtin_amdgcn_sched_barrier(0);
      if (n >= kBehind) {
        const int m = n - kBehind, i = m >> 2, j = column(m);
        add_scaled<kRowB>(acc[i0 + i][j], p[m & 3], sa[i], sa[i] * sb, sb4[j]);
      }
      if (n == 1 && i0 == 0) advance(next_real);
      __builtin_amdgcn_sched_barrier(0);
    }
    sa_left = sa[3];
    sb_left = sb;
  };
  auto read_scales0 = [&](int i) {
    const float* ss = reinterpret_cast<const float*>(slots + (i & 3) * kScaleSlot);
    if constexpr (kRowB) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sb4[j] = *reinterpret_cast<const f32x4_t*>(ss + 256 + t.wn * 64 + 16 * j + 4 * q);
    } else {
      sb = ss[256 + t.wn * 64];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) sa[k] = ss[t.wm * 128 + 16 * k + r];
  };
  auto read_scales1 = [&](int i) {
    const float* ss = reinterpret_cast<const float*>(slots + (i & 3) * kScaleSlot);
#pragma unroll
    for (int k = 0; k < 4; ++k) sa[k] = ss[t.wm * 128 + 64 + 16 * k + r];
  };
  auto load_scales = [&](int i) { load4_to_lds(od, to_slot + (i & 3) * kScaleSlot, scales.at); };
  auto load_first = [&](int i) {
    t.load_b<0>(ob);
    t.load_b<1>(ob);
    t.load_b<2>(ob);
    t.load_b<3>(ob);
    t.load_a<0>(oa);
    t.load_a<1>(oa);
    load_scales(i);
  };
  advance(steps > 0);
  load_first(0);
  t.load_a<2>(oa);
  t.load_a<3>(oa);
  t.stage(1, 0);
  advance(steps > 1);
  load_first(1);
  auto memory0 = [&](int s) {   // loads: step s + 1's stage
    if constexpr (kRowB) settle(4);   // the step before, whose column scales are replaced below
    bf[0] = t.b(0);
    af[0] = t.a(0);
    t.load_a<2>(oa);
    bf[1] = t.b(1);
    af[1] = t.a(1);
    bf[2] = t.b(2);
    t.load_a<3>(oa);
    af[2] = t.a(2);
    bf[3] = t.b(3);
    af[3] = t.a(3);
    read_scales0(s);
    if constexpr (!kRowB) settle(4);
  };
  auto memory1 = [&](int s) {   // loads: step s + 2's stage, which is step s's
    const int to = s & 1 ? kNtStage : -kNtStage;
    t.to_a += to;
    t.to_b += to;
    t.load_b<0>(ob);
    t.load_b<1>(ob);
    af[0] = t.a(4);
    t.load_b<2>(ob);
    af[1] = t.a(5);
    t.load_b<3>(ob);
    af[2] = t.a(6);
    t.load_a<0>(oa);
    af[3] = t.a(7);
    t.load_a<1>(oa);
    read_scales1(s);
    load_scales(s + 2);
    t.a_lo -= to;
    t.a_hi -= to;
    t.b_lo -= to;
    t.b_hi -= to;
    settle(0);
  };
  auto compute0 = [&](int s) {
    next_real = s + 2 < steps;
    multiply(0);
  };
  nt_loop<7, 2>(t.wm, steps, memory0, memory1, compute0, [&](int) { multiply(4); });
  settle(4);
  if (odd) {   // in stage 0 and slot 0; bytes of the last chunk that lie past K are cleared in LDS
    lds_barrier();   // nobody reads the stages any more
    t.rows(a.lda, a.ldb, tail);
    t.stage(0, 0);
    const int64_t k0 = static_cast<int64_t>(a.groups - 1) * kGroup;
    const int kup = (a.K + 15) & ~15;
    oa.start(a.A + static_cast<int64_t>(tm) * 256 * a.lda + k0, (min(256, a.M - tm * 256) - 1) * a.lda + kup - k0);
    ob.start(a.B + static_cast<int64_t>(tn) * 256 * a.ldb + k0, (min(256, a.N - tn * 256) - 1) * a.ldb + kup - k0);
    scale_at = reinterpret_cast<uint64_t>(scales.base + (a.groups - 1) * scales.group);
    advance(true);
    load_first(0);
    t.load_a<2>(oa);
    t.load_a<3>(oa);
    wait_loads<0>();
    lds_barrier();
    if (tail & 15) {
      char* c = lds + threadIdx.x * kNtRow + (((tail >> 4) ^ (threadIdx.x >> 1)) & 7) * 16;
      *reinterpret_cast<uint4*>(c) = keep_bytes(*reinterpret_cast<uint4*>(c), tail & 15);
      lds_barrier();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) bf[j] = t.b(j);
#pragma unroll
    for (int k = 0; k < 4; ++k) af[k] = t.a(k);
    read_scales0(0);
    multiply(0);
    settle(0);
#pragma unroll
    for (int k = 0; k < 4; ++k) af[k] = t.a(4 + k);
    read_scales1(0);
    multiply(4);
    settle(4);
  }
  mend_range<kFa, kFb, kRowB, false>(a, share.s0, share.s1, 1, tm * 256 + t.wm * 128, tn * 256 + t.wn * 64, acc, [](int, int) { return f32x4_t{0, 0, 0, 0}; });
  if (share.unit >= 0) {
    write_part(deal, work, share.unit, t.wave, t.lane, a.M - tm * 256 - t.wm * 128, acc);
    return;
  }
  wait_loads<0>();
  lds_barrier();   // nobody reads the stages any more
  put_rows(a, lds + t.wave * 4096, tm * 256 + t.wm * 128, tn * 256 + t.wn * 64, acc);
}

// Joins the parts of a split tile: a workgroup a row block of its waves.
template <int kT, bool kF32>
__global__ __launch_bounds__(kNtThreads) void gemm8_join_kernel(Gemm8Args a, TileOrder order, Deal deal, float* __restrict__ work) {
  constexpr int kRows = kT == 256 ? 128 : 32, kAcross = kT == 256 ? 4 : 2;   // of a wave; waves side by side
  const int tile = deal.whole + static_cast<int>(blockIdx.x) / (kRows / 16), i = static_cast<int>(blockIdx.x) % (kRows / 16);
  int tm, tn;
  order_tile(order, tile, tm, tn);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m0 = tm * kT + wave / kAcross * kRows + i * 16, n0 = tn * kT + wave % kAcross * 64;
  if (m0 >= a.M) return;
  f32x4_t acc[1][4];
  join_parts(deal, work, tile, i, wave, lane, acc);
  put_tile<kF32>(a, m0 + (lane & 15), n0 + 4 * (lane >> 4), acc);
}

// 128 x 128 tiles with the loop of nt_tile.hpp's Nt128 (16-bit outputs). Scales come with the operands and are read a
// step ahead; a product is added to its sum three instructions later (the last three of a step in the next one). A group takes
// 0.5 us: 777 x 4100 x 6100 30 to 31 us, one round of 231 tiles; 24 x 10240 x 6144, split three ways, 16 and 4 for joining.
constexpr int kScale128 = 2 * 128 * 4;

template <int kFa, int kFb, bool kRowB>
__global__ __launch_bounds__(kNtThreads) void gemm8_tile128_kernel(Gemm8Args a, TileOrder order, Deal deal, float* __restrict__ work) {
  __shared__ __attribute__((aligned(1024))) char lds[kNt128Stages * (kNt128Stage + kScale128)];
  int tm, tn;
  const Share share = share_of(deal, static_cast<int>(blockIdx.x));
  order_tile(order, share.tile, tm, tn);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  // the share's groups are counted from 0; ``last`` is K's last one, if it is among them
  const int groups = share.s1 - share.s0, last = share.s1 == a.groups ? groups - 1 : -1;
  const int tail = a.K & (kGroup - 1);
  Nt128 t;
  t.init(lds, a.lda, a.ldb);
  const ScaleLoad scales(a, 128, tm, tn, 4, t.wave & 3, t.lane);   // waves 4 .. 7 load the same again
  char* const slots = lds + kNt128Stages * kNt128Stage;
  const unsigned to_slot = lds_address(slots) + (t.wave & 3) * 256;
  uint64_t scale_at = reinterpret_cast<uint64_t>(scales.base + share.s0 * scales.group);
  i32x4_t od;
  NtOperand oa, ob;
  const int kup = (a.K + 15) & ~15;   // a chunk that starts inside a row is read whole
  const int64_t k0 = static_cast<int64_t>(share.s0) * kGroup;
  oa.start(a.A + static_cast<int64_t>(tm) * 128 * a.lda + k0, (min(128, a.M - tm * 128) - 1) * a.lda + kup - k0);
  ob.start(a.B + static_cast<int64_t>(tn) * 128 * a.ldb + k0, (min(128, a.N - tn * 128) - 1) * a.ldb + kup - k0);
  auto advance = [&](int g) {   // to group g, which is loaded next
    const bool real = g < groups;
    oa.set(real);
    ob.set(real);
    od = make_desc(reinterpret_cast<const void*>(scale_at), real ? scales.range : 0);
    scale_at += scales.group * 4;
    if (g == last && tail != 0) t.rows(a.lda, a.ldb, tail);
  };
  f32x4_t acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  for (int g = 0; g < kNt128Stages; ++g) {
    t.load_stage(g);
    advance(g);
    t.load_a<0>(oa);
    t.load_a<1>(oa);
    t.load_b<0>(ob);
    t.load_b<1>(ob);
    load4_to_lds(od, to_slot + g * kScale128, scales.at);
  }
  // K ends inside a chunk of its last group: that group's bytes past K are cleared in LDS, one row of either operand a thread
  auto clear_tail = [&](int g) {
    if ((tail & 15) == 0 || g != last) return;
    if (threadIdx.x < 256) {
      char* p = lds + (g & (kNt128Stages - 1)) * kNt128Stage + threadIdx.x * kNtRow + (((tail >> 4) ^ (threadIdx.x >> 1)) & 7) * 16;
      *reinterpret_cast<uint4*>(p) = keep_bytes(*reinterpret_cast<uint4*>(p), tail & 15);
    }
    lds_barrier();
  };
  struct Scales {
    float a[2], b;
    f32x4_t b4[kRowB ? 4 : 1];
  };
  const int r = t.lane & 15, q = t.lane >> 4;
  auto read_scales = [&](int g, Scales& v) {
    const float* ss = reinterpret_cast<const float*>(slots + (g & (kNt128Stages - 1)) * kScale128);
#pragma unroll
    for (int i = 0; i < 2; ++i) v.a[i] = ss[t.wm * 32 + 16 * i + r];
    v.b = ss[128 + t.wn * 64];
    if constexpr (kRowB) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v.b4[j] = *reinterpret_cast<const f32x4_t*>(ss + 128 + t.wn * 64 + 16 * j + 4 * q);
    }
  };
  constexpr int kLoads = 5;
  wait_loads<kLoads * (kNt128Stages - 1)>();
  lds_barrier();
  clear_tail(0);
  Codes af[2][2], bf[4];
  Scales sc[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) af[0][i] = t.a(i);
#pragma unroll
  for (int j = 0; j < 4; ++j) bf[j] = t.b(j);
  read_scales(0, sc[0]);
  constexpr int kBehind = 3;
  f32x4_t p[kBehind + 1];
#pragma unroll
  for (int k = 0; k <= kBehind; ++k) p[k] = f32x4_t{0, 0, 0, 0};
  sc[1] = Scales{};
  // product n of a step: column block n / 2, row block 0 1 1 0 0 1 1 0 (one operand stays at every change)
  auto row = [](int n) { return ((n + 1) >> 1) & 1; };
  auto add = [&](int n, const Scales& v) { add_scaled<kRowB>(acc[row(n)][n >> 1], p[n & 3], v.a[row(n)], v.a[row(n)] * v.b, v.b4[kRowB ? n >> 1 : 0]); };
  // step g uses ``now`` and ``mine`` and reads step g + 1's into ``next`` and, once the step before is added up, ``theirs``
  auto step = [&](int g, const Codes (&now)[2], Codes (&next)[2], Scales& mine, Scales& theirs) {
    wait_loads<kLoads * (kNt128Stages - 2)>();   // group g + 1 has landed everywhere, and group g's stage is free
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
    clear_tail(g + 1);
    t.load_stage(g & (kNt128Stages - 1));
    t.read_stage((g + 1) & (kNt128Stages - 1));
    advance(g + kNt128Stages);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int j = n >> 1;
      Operand<kFa, false> av;
      Operand<kFb, false> bv;
      av.set(now[row(n)]);
      bv.set(bf[j]);
      p[n & 3] = product<kFa, kFb>(bv, av);
      __builtin_amdgcn_sched_barrier(0);
      if (n < kBehind) add(n + 8 - kBehind, theirs);
      else add(n - kBehind, mine);
      if (n & 1) {
        bf[j] = t.b(j);   // past the last group: zeros that nobody uses
        if (j < 2) next[j] = t.a(j);
        if (j == 0) t.load_a<0>(oa);
        if (j == 1) { t.load_b<0>(ob); read_scales(g + 1, theirs); }
        if (j == 2) t.load_a<1>(oa);
        if (j == 3) { t.load_b<1>(ob); load4_to_lds(od, to_slot + (g & (kNt128Stages - 1)) * kScale128, scales.at); }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int g = 0;
  for (; g + 1 < groups; g += 2) {
    step(g, af[0], af[1], sc[0], sc[1]);
    step(g + 1, af[1], af[0], sc[1], sc[0]);
  }
  // the last three products: their scales were read over only where another step followed
  if (g < groups) {
    step(g, af[0], af[1], sc[0], sc[1]);
#pragma unroll
    for (int n = 8 - kBehind; n < 8; ++n) add(n, sc[0]);
  } else {
#pragma unroll
    for (int n = 8 - kBehind; n < 8; ++n) add(n, sc[1]);
  }
  wait_loads<0>();   // no direct load may still be writing this workgroup's LDS
  mend_range<kFa, kFb, kRowB, false>(a, share.s0, share.s1, 1, tm * 128 + t.wm * 32, tn * 128 + t.wn * 64, acc, [](int, int) { return f32x4_t{0, 0, 0, 0}; });
  if (share.unit >= 0) {
    write_part(deal, work, share.unit, t.wave, t.lane, a.M - tm * 128 - t.wm * 32, acc);
    return;
  }
  lds_barrier();   // nobody reads the stages any more
  put_rows(a, lds + t.wave * 4096, tm * 128 + t.wm * 32, tn * 128 + t.wn * 64, acc);
}

// fp32 outputs (exact products: twice the matrix cycles, and the conversions): 128 x 128 tiles, four waves of 64 x 64, two
// stages of LDS, so that two workgroups share a CU and one's loads and epilogue hide behind the other's products. Few tiles are
// split along k (exact_deal). 10240 x 6144 x 2000 with an addition: 298 to 313 us, of which 14.75 a group (16 of them, 1.09 PFLOP/s), bound
// by issue: a conversion or two and as many multiplications and multiply-adds to a matrix instruction; 40 writing, 30 adding
// (311 with the addition at the end instead of at the start). Starting half the workgroups late changed nothing.
template <int kFa, int kFb, bool kRowB>
__global__ __launch_bounds__(256, 2) void gemm8_exact_kernel(Gemm8Args a, TileOrder order, Deal deal, float* __restrict__ work) {
  constexpr int kStage = kNt128Stage + kScale128;
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  int tm, tn;
  const Share share = share_of(deal, static_cast<int>(blockIdx.x));
  order_tile(order, share.tile, tm, tn);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);

  const int tail = a.K & (kGroup - 1);                  // bytes of the last group, 0: whole
  constexpr int kInst = 4, kOperand = 128 * kGroup;
  int va[kInst], vb[kInst], at16[kInst];
#pragma unroll
  for (int j = 0; j < kInst; ++j) {
    const int row = (wave * kInst + j) * 8 + (lane >> 3);
    at16[j] = (((lane & 7) ^ (row >> 1)) & 7) * 16;
    va[j] = row * static_cast<int>(a.lda) + at16[j];
    vb[j] = row * static_cast<int>(a.ldb) + at16[j];
  }
  const ScaleLoad scales(a, 128, tm, tn, 4, wave, lane);
  const uint8_t* pa = a.A + static_cast<int64_t>(tm) * 128 * a.lda;
  const uint8_t* pb = a.B + static_cast<int64_t>(tn) * 128 * a.ldb;
  const int kup = (a.K + 15) & ~15;
  const int64_t size_a = (min(128, a.M - tm * 128) - 1) * a.lda + kup, size_b = (min(128, a.N - tn * 128) - 1) * a.ldb + kup;
  auto issue = [&](int g) {           // all of this wave's loads of group g (past the end: zero-length ones)
    const bool real = g < share.s1, last = tail != 0 && g == a.groups - 1;
    const unsigned at = lds_address(lds + (g & 1) * kStage);
    const int64_t k0 = static_cast<int64_t>(g) * kGroup;
    const i32x4_t da = make_desc(pa + k0, real ? size_a - k0 : 0), db = make_desc(pb + k0, real ? size_b - k0 : 0);
#pragma unroll
    for (int j = 0; j < kInst; ++j) load_to_lds(da, at + (wave * kInst + j) * 1024, last && at16[j] >= tail ? kNtOut : va[j]);
#pragma unroll
    for (int j = 0; j < kInst; ++j) load_to_lds(db, at + kOperand + (wave * kInst + j) * 1024, last && at16[j] >= tail ? kNtOut : vb[j]);
    scales.issue(g, real, at + 2 * kOperand + wave * 256);
  };
  const int r = lane & 15, q = lane >> 4;
  const int swz = ((q ^ (r >> 1)) & 7) * 16;
  const int hi = (swz ^ 64) - swz;    // where chunk q + 4 lies from chunk q
  const int a_rd = (wm * 64 + r) * kGroup + swz, b_rd = kOperand + (wn * 64 + r) * kGroup + swz;
  auto codes_at = [&](const char* p) -> Codes { return Codes{*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + hi)}; };
  issue(share.s0);
  // a whole tile's sums start from what is added: its loads then wait together with the first group's
  const int m0 = tm * 128 + wm * 64 + r, n0 = tn * 128 + wn * 64 + 4 * q;
  auto start = [&](int i, int j) { return a.add != nullptr && share.unit < 0 ? added(a, m0 + i * 16, n0 + j * 16) : f32x4_t{0, 0, 0, 0}; };
  f32x4_t acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = start(i, j);
  for (int g = share.s0; g < share.s1; ++g) {
    wait_loads<0>();                 // this wave's loads of group g have landed
    lds_barrier();                   // everybody's have, and nobody still reads the stage that the next loads fill
    __builtin_amdgcn_sched_barrier(0);
    issue(g + 1);
    char* stage = lds + (g & 1) * kStage;
    if (tail & 15 && g == a.groups - 1) {   // K ends inside a chunk: cleared as in the other kernels
      char* p = stage + threadIdx.x * kGroup + (((tail >> 4) ^ (threadIdx.x >> 1)) & 7) * 16;
      *reinterpret_cast<uint4*>(p) = keep_bytes(*reinterpret_cast<uint4*>(p), tail & 15);
      lds_barrier();
    }
    const float* ss = reinterpret_cast<const float*>(stage + 2 * kOperand);
    Halves bh[4], ah[2];
#pragma unroll
    for (int j = 0; j < 4; ++j) bh[j] = to_halves<kFb>(codes_at(stage + b_rd + j * 16 * kGroup));
    Codes raw = codes_at(stage + a_rd);
    float sa[4], sb = 0;
    f32x4_t sb4[kRowB ? 4 : 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) sa[i] = ss[wm * 64 + 16 * i + r];
    if constexpr (kRowB) {
#pragma unroll
      for (int j = 0; j < 4; ++j) sb4[j] = *reinterpret_cast<const f32x4_t*>(ss + 128 + wn * 64 + 16 * j + 4 * q);
    } else {
      sb = ss[128 + wn * 64];
    }
    ah[0] = to_halves<kFa>(raw);
    raw = codes_at(stage + a_rd + 16 * kGroup);
    // Row block i: 16 matrix instructions (four chains of four), each followed by a sixteenth of the next row block's
    // conversion and of the last one's scaling, in a fixed order: one wave's vector instructions then fit beside its matrix
    // instructions (left to the compiler the two alternate: 322 us at 10240 x 6144 x 2000 with an addition).
    f32x4_t p[2][4];
#pragma unroll
    for (int i = 0; i < 5; ++i) {
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int h = n >> 2, j = n & 3;
        if (i < 4) {
          const f32x4_t c = h == 0 ? f32x4_t{0, 0, 0, 0} : p[i & 1][j];
          p[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, bh[j].q[h]), __builtin_bit_cast(half8_t, ah[i & 1].q[h]), c, 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (i < 3) {   // two of the next row block's 32 codes
          const uint32_t w[8] = {raw.lo.x, raw.lo.y, raw.lo.z, raw.lo.w, raw.hi.x, raw.hi.y, raw.hi.z, raw.hi.w};
          const uint32_t two = to_half2<kFa>(w[n >> 1], n & 1);
          uint4& to = ah[(i + 1) & 1].q[n >> 2];
          if ((n & 3) == 0) to.x = two;
          else if ((n & 3) == 1) to.y = two;
          else if ((n & 3) == 2) to.z = two;
          else to.w = two;
        }
        if (i > 0) {   // one of the last row block's 16 sums
          const int jl = n >> 2, e = n & 3;
          acc[i - 1][jl][e] = __builtin_fmaf(p[(i - 1) & 1][jl][e], kRowB ? sa[i - 1] * sb4[kRowB ? jl : 0][e] : sa[i - 1] * sb, acc[i - 1][jl][e]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (i < 2) raw = codes_at(stage + a_rd + (i + 2) * 16 * kGroup);
    }
  }
  wait_loads<0>();   // no direct load may still be writing this workgroup's LDS
  mend_range<kFa, kFb, kRowB, true>(a, share.s0, share.s1, 1, tm * 128 + wm * 64, tn * 128 + wn * 64, acc, start);
  if (share.unit >= 0) {             // as two of the joining kernel's waves of 32 rows
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f32x4_t two[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) two[i][j] = acc[2 * h + i][j];
      write_part(deal, work, share.unit, (2 * wm + h) * 2 + wn, lane, a.M - tm * 128 - wm * 64 - 32 * h, two);
    }
    return;
  }
  a.add = nullptr;
  put_tile<true>(a, m0, n0, acc);
}

// ---- few rows --------------------------------------------------------------------------------------

// M <= 16 kMB rows: B is streamed from HBM straight into registers. A workgroup of eight waves takes 16 rows of B; its waves
// take the groups in turn (so the eight read 1 KiB of a row together), kDeep of them at a time with all loads in flight
// before the first product, and add their sums through LDS in order. Bound by B's bytes; one group at a time the loads'
// latency shows (24 x 10240 x 6144: 27 us). 1 x 4096 x 4096: 5.0 us in a graph, 3.3 TB/s with the launch.
constexpr int kStreamWaves = 8;

template <int kMB, int kFa, int kFb, bool kRowB, bool kF32>
__global__ __launch_bounds__(kStreamWaves * 64) void gemm8_stream_kernel(Gemm8Args a) {
  constexpr int kDeep = kMB == 1 ? 4 : kMB == 2 ? 3 : 2;
  __shared__ float sums[kStreamWaves][kMB][64 * 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, q = lane >> 4;
  const int n0 = static_cast<int>(blockIdx.x) * 16;
  constexpr int kFlags = 0x00020000;
  // ranges end after the last chunk that starts inside the matrix; rows past it read as zero
  const int kup = (a.K + 15) & ~15;
  const int64_t size_a = (a.M - 1) * a.lda + kup, size_b = (min(16, a.N - n0) - 1) * a.ldb + kup;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.A), 0, static_cast<int>(size_a), kFlags);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(a.B) + static_cast<int64_t>(n0) * a.ldb, 0,
                                                                      static_cast<int>(size_b), kFlags);
  unsigned va[kMB];
  const unsigned vb = n0 + r < a.N ? r * static_cast<unsigned>(a.ldb) + 32 * q : kNtOut;
#pragma unroll
  for (int i = 0; i < kMB; ++i) va[i] = 16 * i + r < a.M ? (16 * i + r) * static_cast<unsigned>(a.lda) + 32 * q : kNtOut;
  const float *sa[kMB], *sb;
#pragma unroll
  for (int i = 0; i < kMB; ++i) sa[i] = a.sa + (min(16 * i + r, a.M - 1) >> a.a_shift) * a.sa_row;
  sb = a.sb + (n0 >> a.b_shift) * a.sb_row;   // kRowB: row n0's, else the block's

  f32x4_t acc[kMB][1];
#pragma unroll
  for (int i = 0; i < kMB; ++i) acc[i][0] = f32x4_t{0, 0, 0, 0};
  // this lane's 32 values of a group: two neighbouring chunks
  auto fetch = [&](__amdgpu_buffer_rsrc_t rs, unsigned at, int g) -> Codes {   // kNtOut and more stays past every range
    const int k = g * kGroup + 32 * q;
    at += static_cast<unsigned>(g) * kGroup;
    Codes c;
    c.lo = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(k < a.K ? at : kNtOut), 0, 0));
    c.hi = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, static_cast<int>(k + 16 < a.K ? at + 16 : kNtOut), 0, 0));
    return c;
  };
  for (int g0 = wave; g0 < a.groups; g0 += kStreamWaves * kDeep) {
    Codes bc[kDeep], ac[kDeep][kMB];
    float as[kDeep][kMB], bs[kDeep];
    f32x4_t bs4[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int g = g0 + d * kStreamWaves, gs = min(g, a.groups - 1);
      bc[d] = fetch(rb, vb, g);
#pragma unroll
      for (int i = 0; i < kMB; ++i) {
        ac[d][i] = fetch(ra, va[i], g);
        as[d][i] = sa[i][gs * a.sa_group];
      }
      if constexpr (kRowB) {
#pragma unroll
        for (int e = 0; e < 4; ++e) bs4[d][e] = sb[min(4 * q + e, a.N - 1 - n0) + gs * a.sb_group];
      } else {
        bs[d] = sb[gs * a.sb_group];
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int g = g0 + d * kStreamWaves;
      if (g >= a.groups) break;
      if (a.K & 15 && g == a.groups - 1) {
        const int left = a.K - g * kGroup - 32 * q;
        bc[d].lo = keep_bytes(bc[d].lo, left);
        bc[d].hi = keep_bytes(bc[d].hi, left - 16);
#pragma unroll
        for (int i = 0; i < kMB; ++i) {
          ac[d][i].lo = keep_bytes(ac[d][i].lo, left);
          ac[d][i].hi = keep_bytes(ac[d][i].hi, left - 16);
        }
      }
      Operand<kFb, kF32> b;
      b.set(bc[d]);
#pragma unroll
      for (int i = 0; i < kMB; ++i) {
        Operand<kFa, kF32> av;
        av.set(ac[d][i]);
        add_scaled<kRowB>(acc[i][0], product<kFa, kFb>(b, av), as[d][i], as[d][i] * bs[d], bs4[d]);
      }
    }
  }
  mend_range<kFa, kFb, kRowB, kF32>(a, wave, a.groups, kStreamWaves, 0, n0, acc, [](int, int) { return f32x4_t{0, 0, 0, 0}; });
#pragma unroll
  for (int i = 0; i < kMB; ++i) *reinterpret_cast<f32x4_t*>(&sums[wave][i][4 * lane]) = acc[i][0];
  __syncthreads();
  if (wave < kMB) {
    f32x4_t v = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < kStreamWaves; ++w) v += *reinterpret_cast<const f32x4_t*>(&sums[w][wave][4 * lane]);
    const int m = 16 * wave + r, n = n0 + 4 * q;
    if (a.add != nullptr) v += added(a, m, n);
    put4<kF32>(a, m, n, v);
  }
}

// ---- dispatch --------------------------------------------------------------------------------------

template <int kFa, int kFb, bool kRowB, bool kF32>
hipError_t launch_stream(const Gemm8Launch& l, const Gemm8Args& a, hipStream_t s) {
  const dim3 grid((l.N + 15) / 16), block(kStreamWaves * 64);
  if (l.M <= 16) hipLaunchKernelGGL((gemm8_stream_kernel<1, kFa, kFb, kRowB, kF32>), grid, block, 0, s, a);
  else if (l.M <= 32) hipLaunchKernelGGL((gemm8_stream_kernel<2, kFa, kFb, kRowB, kF32>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((gemm8_stream_kernel<4, kFa, kFb, kRowB, kF32>), grid, block, 0, s, a);
  return hipGetLastError();
}

// fp32 outputs' tiles: fewer than the card holds at once are split along k, for one or two workgroups a CU, by what each would
// take, in us, fitted to measured launches: 1.2 a group (2 where two share a CU) and 5, joining 5 and the sums' traffic.
// Whole / two a CU / one: 200 x 2000 x 8000 70.0 / 24.8 / 23.7, 1024 x 1024 x 8192 73.7 / 32.9 / 34.0, 1500 x 1500 x 4000
// 41.8 / 36.1 / -, 2048 x 2048 x 2048 27.3 / 33.9 / -.
Deal exact_deal(int64_t tiles, int groups, double& time) {
  Deal best{static_cast<int>(tiles), static_cast<int>(tiles), 1, groups, 128};
  if (tiles > 2 * kCus) {
    time = 1e30;
    return best;
  }
  time = groups * (tiles > kCus ? 2.0 : 1.2) + 5;
  for (int slots = kCus; slots <= 2 * kCus; slots += kCus) {
    if (tiles >= slots) continue;
    const Deal d = make_deal(tiles, groups, 128, slots);
    const double t = static_cast<double>(groups) / d.parts * (d.blocks() > kCus ? 2.0 : 1.2) + 10 + d.floats() / 1e6;
    if (d.parts > 1 && t < time) {
      time = t;
      best = d;
    }
  }
  return best;
}

template <int kFa, int kFb, bool kF32>
hipError_t launch_types(const Gemm8Launch& l, const Gemm8Plan& plan, const Gemm8Args& a, hipStream_t s) {
  if (plan.kernel == 0) {
    return l.b_block == 1 ? launch_stream<kFa, kFb, true, kF32>(l, a, s) : launch_stream<kFa, kFb, false, kF32>(l, a, s);
  }
  const int t = plan.kernel;
  const int gm = (l.M + t - 1) / t, gn = (l.N + t - 1) / t;
  const TileOrder order = make_tile_order(kPanel, 1, gm, gn, gm < 8 ? gm : 8, 1, 1);
  double time;
  const Deal deal = kF32 ? exact_deal(order.tiles, a.groups, time) : make_deal(order.tiles, a.groups, t);
  const dim3 grid(static_cast<unsigned>(deal.blocks())), block(kF32 ? 256 : kNtThreads);
  if constexpr (kF32) {
    if (l.b_block == 1) hipLaunchKernelGGL((gemm8_exact_kernel<kFa, kFb, true>), grid, block, 0, s, a, order, deal, l.work);
    else hipLaunchKernelGGL((gemm8_exact_kernel<kFa, kFb, false>), grid, block, 0, s, a, order, deal, l.work);
  } else {
    if (t == 256 && l.b_block == 1) hipLaunchKernelGGL((gemm8_tile256_kernel<kFa, kFb, true>), grid, block, 0, s, a, order, deal, l.work);
    else if (t == 256) hipLaunchKernelGGL((gemm8_tile256_kernel<kFa, kFb, false>), grid, block, 0, s, a, order, deal, l.work);
    else if (l.b_block == 1) hipLaunchKernelGGL((gemm8_tile128_kernel<kFa, kFb, true>), grid, block, 0, s, a, order, deal, l.work);
    else hipLaunchKernelGGL((gemm8_tile128_kernel<kFa, kFb, false>), grid, block, 0, s, a, order, deal, l.work);
  }
  if (deal.parts > 1) {
    const unsigned split = static_cast<unsigned>(deal.tiles - deal.whole);
    if (t == 256) hipLaunchKernelGGL((gemm8_join_kernel<256, false>), dim3(split * 8), dim3(kNtThreads), 0, s, a, order, deal, l.work);
    else hipLaunchKernelGGL((gemm8_join_kernel<128, kF32>), dim3(split * 2), dim3(kNtThreads), 0, s, a, order, deal, l.work);
  }
  return hipGetLastError();
}

template <int kFa, int kFb>
hipError_t launch_formats(const Gemm8Launch& l, const Gemm8Plan& plan, const Gemm8Args& a, hipStream_t s) {
  return l.out == 2 ? launch_types<kFa, kFb, true>(l, plan, a, s) : launch_types<kFa, kFb, false>(l, plan, a, s);
}

}  // namespace

// The kernel of a shape, by what each would take, in us, fitted to measured launches (as a graph, one after another): streaming
// 4 and B's bytes at 3 (M <= 32) or 1.75 TB/s, a 128 tile 0.5 a group and 5 a round, a 256 tile 1.75 and 8; split tiles
// 5 for joining and their sums' traffic. Streaming / 128 / 256: 24 x 4096 x 4096 8.9 / 13.0 / 17.7, 24 x 10240 x 6144 25.0 /
// 18.4 / 23.8, 1024 x 4096 x 4096 - / 24.7 / 39.7, 2048 x 8192 x 8192 - / 163 / 108. Up to 16 rows streaming always wins. To fp32
// streaming / exact tiles: 24 x 4096 x 4096 8.4 / 13.9, 64 x 8192 x 8192 42.3 / 26.9.
Gemm8Plan gemm8_plan(int64_t M, int64_t N, int64_t K, int out) {
  Gemm8Plan p{0, 0};
  if (M <= 16 || N <= 0 || K <= 0) {
    if (M > 64) p.kernel = 128;
    return p;
  }
  const int groups = static_cast<int>((K + kGroup - 1) / kGroup);
  auto tiles = [&](int64_t t) { return ((M + t - 1) / t) * ((N + t - 1) / t); };
  const double stream = M > 64 ? 2e30 : 4 + N * K * (M <= 32 ? 0.33e-6 : 0.57e-6);
  if (out == 2) {
    double exact;
    const Deal d = exact_deal(tiles(128), groups, exact);
    p.kernel = stream <= exact ? 0 : 128;
    if (p.kernel) p.work_floats = d.floats();
    return p;
  }
  const Deal d256 = make_deal(tiles(256), groups, 256), d128 = make_deal(tiles(128), groups, 128);
  auto time = [&](const Deal& d, double step, double round) {
    const double rounds = (d.whole + kCus - 1) / kCus;
    return rounds * (groups * step + round) + (d.parts > 1 ? groups / d.parts * step + round + 5 + d.floats() / 1e6 : 0);
  };
  const double t256 = time(d256, 1.75, 8), t128 = time(d128, 0.5, 5);
  p.kernel = stream <= t128 && stream <= t256 ? 0 : t128 <= t256 ? 128 : 256;
  if (p.kernel) p.work_floats = (p.kernel == 128 ? d128 : d256).floats();
  return p;
}

hipError_t launch_gemm8(const Gemm8Launch& l, hipStream_t s) {
  const Gemm8Plan plan = gemm8_plan(l.M, l.N, l.K, l.out);
  Gemm8Args a;
  a.A = l.A;
  a.B = l.B;
  a.lda = l.lda;
  a.ldb = l.ldb;
  a.groups = (l.K + kGroup - 1) / kGroup;
  a.sa = l.sa;
  a.sb = l.sb;
  a.a_shift = l.a_block == 1 ? 0 : 7;
  a.b_shift = l.b_block == 1 ? 0 : 7;
  a.sa_row = l.a_block == 1 ? 1 : a.groups;
  a.sa_group = l.a_block == 1 ? l.M : 1;
  a.sb_row = l.b_block == 1 ? 1 : a.groups;
  a.sb_group = l.b_block == 1 ? l.N : 1;
  a.add = l.add;
  a.C = l.C;
  a.M = l.M;
  a.N = l.N;
  a.K = l.K;
  a.out = l.out;
  if (l.fa == 0) return l.fb == 0 ? launch_formats<0, 0>(l, plan, a, s) : launch_formats<0, 1>(l, plan, a, s);
  return l.fb == 0 ? launch_formats<1, 0>(l, plan, a, s) : launch_formats<1, 1>(l, plan, a, s);
}

}  // namespace tbl
