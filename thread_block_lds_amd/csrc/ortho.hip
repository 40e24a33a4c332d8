// Orthogonalisation of a matrix by Newton-Schulz products, as the Muon optimiser applies it to a momentum.
//
//   X = x / (|x|_F + eps);   steps times:  P = X X^T,  Q = b P + c P P,  X <- a X + Q X
//
// taken on the side that makes P the smaller square (r x r, r = min(rows, cols); c = max). Every product is
// A B^T with k contiguous in both operands: X is kept both ways, W = X (r x c) for P = W W^T and U = X^T (c x r)
// for X'^T = a U + U Q (P and Q are symmetric); the update writes both.
//
// Arithmetic: operands are fp16, sums fp32. fp16 has bf16's cost and eight times its precision; with bf16
// operands the result is 1.4 % off the exact one, with fp16 0.03-0.1 % (a bf16 output's own rounding is 0.17 %). The
// values are held at powers of two that keep them normal numbers: X at kx (rms near 1 after the
// normalisation), P at kP = 2^14 (its entries are at most 4 where the iteration is of any use), Q at kq. x itself is
// scaled by a power of two only, so 16-bit inputs enter exactly, and 1 / (|x| + eps) is applied to
// the fp32 sums of the first P and update. Two roundings are kept. The term a X multiplies what rounding adds to the small
// singular values by a in every step that follows (485 in five), so in all but the last two steps it takes X to 22 bits: U's
// remainder is kept beside it, in fp16 too. And P's and Q's diagonals (see finish).
#include <stdint.h>

#include "nt_tile.hpp"

namespace tbl {
namespace {

constexpr float kP = 16384.0f;
constexpr int kStep = 64;        // k depth of a step: 128 bytes of fp16

template <int kType>
__device__ __forceinline__ float element(const void* p, int64_t i) {
  if constexpr (kType == 0) return static_cast<float>(static_cast<const _Float16*>(p)[i]);
  else if constexpr (kType == 1) return __builtin_bit_cast(float, static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  else return static_cast<const float*>(p)[i];
}

// Elements i .. i + 7 (``left`` of them exist, the others read as 0). Whole eights are 16-byte loads at whatever
// alignment the element type has: gfx950 takes them unaligned.
template <int kType>
__device__ __forceinline__ void eight(const void* p, int64_t i, int64_t left, float (&v)[8]) {
  if (left >= 8) {
    if constexpr (kType == 2) {
      __builtin_memcpy(v, static_cast<const float*>(p) + i, 32);
    } else {
      uint32_t w[4];
      __builtin_memcpy(w, static_cast<const uint16_t*>(p) + i, 16);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h = e & 1 ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
        v[e] = kType == 0 ? static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(h))) : __builtin_bit_cast(float, h << 16);
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < left ? element<kType>(p, i + e) : 0.0f;
}

// ---- |x|^2 -----------------------------------------------------------------------------------------

constexpr int kNormParts = 1024;   // most parts of a matrix; summed in order, so the result is always the same bits
constexpr int kNormSpan = 2048;    // elements of a row that a workgroup takes at a time, eight a thread

// Part p of matrix b: the squares of the row pieces p, p + parts, ... in 64 bits.
template <int kType>
__global__ __launch_bounds__(256) void ortho_norm_kernel(const void* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                                                         int64_t batch_ld, int parts, double* __restrict__ out) {
  __shared__ double sums[4];
  const int part = static_cast<int>(blockIdx.x) % parts, b = static_cast<int>(blockIdx.x) / parts;
  const int64_t pieces = (cols + kNormSpan - 1) / kNormSpan;
  double s0 = 0, s1 = 0;
  for (int64_t i = part; i < rows * pieces; i += parts) {
    const int64_t row = i / pieces, c = (i - row * pieces) * kNormSpan + 8 * threadIdx.x;
    float v[8];
    eight<kType>(x, b * batch_ld + row * ld + c, cols - c, v);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      s0 = __builtin_fma(static_cast<double>(v[e]), static_cast<double>(v[e]), s0);
      s1 = __builtin_fma(static_cast<double>(v[e + 1]), static_cast<double>(v[e + 1]), s1);
    }
  }
  double s = s0 + s1;
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) sums[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) out[static_cast<int64_t>(b) * parts + part] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
}

// ---- x -> U, W -------------------------------------------------------------------------------------

// Scalars of a matrix that the first step's products apply: P's factor and the update's.
struct OrthoScalars {
  float p, x;
};

// How a matrix enters: 2^k brings its norm (+ eps) into [kx, 2 kx).
struct Entry {
  double norm;
  bool fine;
  int k;
  __device__ __forceinline__ Entry(double squares, float eps, float kx) {
    norm = __builtin_sqrt(squares) + static_cast<double>(eps);
    fine = norm > 0 && norm < 1e300;
    // floor(log2(norm)); squares of fp32 values sum to normal doubles
    const int e = fine ? static_cast<int>(__builtin_bit_cast(uint64_t, norm) >> 52) - 1023 : 0;
    k = static_cast<int>(__builtin_bit_cast(uint32_t, kx) >> 23) - 127 - e;
  }
  __device__ __forceinline__ OrthoScalars scalars(float kx) const {
    const double scaled = fine ? __builtin_ldexp(norm, k) : __builtin_nan("");   // 0 / 0 and inf / inf are NaN
    return OrthoScalars{static_cast<float>(kP / (scaled * scaled)), static_cast<float>(kx / scaled)};
  }
};

// 64 x 64 tiles of x, scaled by 2^k so that |x| + eps lies in [kx, 2 kx), written straight and turned as fp16 with
// zeros up to the padded row ends; lo: the remainder in U's orientation (fp32 inputs). Thread t takes eight columns of rows
// t / 8 and t / 8 + 32; the turned form goes through LDS.
constexpr int kTurnPitch = 66;

template <int kType>
__global__ __launch_bounds__(256) void ortho_enter_kernel(const void* __restrict__ x, int64_t rows, int64_t cols, int64_t ld,
                                                          int64_t batch_ld, int parts, const double* __restrict__ norms,
                                                          float eps, float kx, _Float16* __restrict__ straight, int64_t lds_,
                                                          int64_t batch_s, _Float16* __restrict__ turned, int64_t ldt,
                                                          int64_t batch_t, _Float16* __restrict__ lo, bool lo_turned,
                                                          OrthoScalars* __restrict__ scalars) {
  typedef _Float16 half8v_t __attribute__((ext_vector_type(8)));
  __shared__ double total[4];
  __shared__ _Float16 hi_t[64][kTurnPitch], lo_t[kType == 2 ? 64 : 1][kTurnPitch];
  const int b = blockIdx.z, t = threadIdx.x;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 64, c0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int row8 = t >> 3, at8 = 8 * (t & 7);
  float v[2][8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = r0 + row8 + 32 * i;
    eight<kType>(x, b * batch_ld + row * ld + c0 + at8, row < rows ? cols - c0 - at8 : 0, v[i]);
  }
  double s = 0;
  for (int i = t; i < parts; i += 256) s += norms[static_cast<int64_t>(b) * parts + i];
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if ((t & 63) == 0) total[t >> 6] = s;
  __syncthreads();
  const Entry entry((total[0] + total[1]) + (total[2] + total[3]), eps, kx);
  if (blockIdx.x == 0 && blockIdx.y == 0 && t == 0) scalars[b] = entry.scalars(kx);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = r0 + row8 + 32 * i;
    half8v_t h, l;
#pragma unroll
    for (int e8 = 0; e8 < 8; ++e8) {
      const float w = __builtin_ldexpf(v[i][e8], entry.k);
      h[e8] = static_cast<_Float16>(w);
      l[e8] = static_cast<_Float16>(w - static_cast<float>(h[e8]));
      hi_t[at8 + e8][row8 + 32 * i] = h[e8];
      if (kType == 2 && lo_turned) lo_t[at8 + e8][row8 + 32 * i] = l[e8];
    }
    if (row < rows) {
      *reinterpret_cast<half8v_t*>(straight + b * batch_s + row * lds_ + c0 + at8) = h;
      if (kType == 2 && !lo_turned) *reinterpret_cast<half8v_t*>(lo + b * batch_s + row * lds_ + c0 + at8) = l;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = row8 + 32 * i;
    if (c0 + c >= cols) continue;
    half8v_t h, l;
#pragma unroll
    for (int e8 = 0; e8 < 8; ++e8) {
      h[e8] = hi_t[c][at8 + e8];
      if constexpr (kType == 2) l[e8] = lo_t[c][at8 + e8];
    }
    *reinterpret_cast<half8v_t*>(turned + b * batch_t + (c0 + c) * ldt + r0 + at8) = h;
    if (kType == 2 && lo_turned) *reinterpret_cast<half8v_t*>(lo + b * batch_t + (c0 + c) * ldt + r0 + at8) = l;
  }
}

// ---- products --------------------------------------------------------------------------------------

enum Product : int { kGram = 0, kSquare = 1, kUpdate = 2, kLast = 3 };   // kLast: the last step's update
constexpr bool is_update(int kind) { return kind >= kUpdate; }

struct OrthoArgs {
  const _Float16* A;     // M x K, rows of lda
  const _Float16* B;     // N x K, rows of ldb
  int64_t lda, ldb, batch_a, batch_b;
  int M, N, K;           // K: padded to whole steps
  const OrthoScalars* scalars;   // nullable: the first step's factors, one of each matrix
  float f1, f2;          // kGram: P = f1 acc; kSquare: Q = f1 P + f2 acc; kUpdate: X' = f1 U + f2 acc
  const _Float16* C;     // kSquare: P; kUpdate: U (M x N, rows of ldc)
  const _Float16* lo_in; // kUpdate, nullable: U's remainder
  _Float16* lo_out;      // kUpdate, nullable: the new U's
  _Float16* D;           // P, Q or the new U, rows padded with zeros to ldc
  int64_t ldc, batch_c;
  _Float16* T;           // the transpose of D, N x M, rows of ldt: kUpdate the new W; kGram, kSquare D itself (of
  int64_t ldt, batch_t;  // the tiles above the diagonal the mirror images)
  const float* d_in;     // kSquare: what rounding took from P's diagonal, ldc of each matrix; kUpdate: from Q's
  float* d_out;          // kGram, kSquare: from D's own
  void* out;             // kLast: the result, M x N or (out_turned) N x M, instead of D and T
  int out_type, out_turned;
  float out_factor;
};

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));

// This lane, hidden from the compiler: it otherwise computes the addresses of all of a wave's sub-tiles once, and spills.
__device__ __forceinline__ int hidden_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// A wave's 16 TM x 64 sub-tile of 16-bit values turned through LDS: ``tile`` (2 KiB a row block, this wave's alone) holds it
// row-major, 128 bytes a row, 16-byte chunk c of row m at c XOR (m / 2 mod 8). Writes rows n0 .. + 63 of ``to`` (rows of ld,
// ``rows`` and ``cols`` of them exist), columns m0 .. The transposing LDS read gives a lane four rows of its column.
template <int TM>
__device__ __forceinline__ void write_turned(char* tile, uint16_t* to, int64_t ld, int rows, int cols, int n0, int m0, int lane) {
  const int i = lane & 15, g = lane >> 4;
  constexpr int kAt = TM == 1 ? 2 : 4;   // groups of eight rows a pass: with one row block the others take more columns
#pragma unroll
  for (int p = 0; p < (TM == 1 ? 2 : 2 * TM); ++p) {
    // pass p: row group (8 rows) and column block (16 columns) of this lane group
    const int rg = TM == 1 ? (g & 1) : (p >> 2) * kAt + g, cb = TM == 1 ? 2 * p + (g >> 1) : p & 3;
    const int col = 16 * cb + 4 * (i & 3);
    uint2 w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = 8 * rg + 4 * h + (i >> 2);
      char* q = tile + m * 128 + ((((col >> 3) ^ (m >> 1)) & 7) << 4) + (col & 7) * 2;
      w[h] = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)q));
    }
    const int n = n0 + 16 * cb + i, m = m0 + 8 * rg;
    if (n >= rows) continue;
    uint16_t* d = to + static_cast<int64_t>(n) * ld + m;
    if (m + 8 <= cols) {
      const uint4 v = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
      __builtin_memcpy(d, &v, 16);   // one 16-byte store, aligned or not
    } else {
      const uint32_t v[4] = {w[0].x, w[0].y, w[1].x, w[1].y};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (m + e < cols) d[e] = static_cast<uint16_t>(e & 1 ? v[e >> 1] >> 16 : v[e >> 1]);
    }
  }
}

// A wave's 16 TM x 64 values of a matrix of fp16, as whole rows: load or store p takes rows 8 p .. + 7, 128 bytes each. (As the
// matrix instructions hold them, eight bytes of 16 rows a load, the address unit took 3000 cycles for a 128 tile.)
template <int TM>
struct Rows {
  uint4 v[2 * TM];
  __device__ __forceinline__ void fetch(const _Float16* p, int64_t ld, int m0, int n0, int M, int lane) {
    const int rows = n0 < ld ? min(16 * TM, M - m0) : 0;   // ld is a multiple of 64: the 64 columns exist or do not
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<_Float16*>(p + static_cast<int64_t>(m0) * ld), 0, rows > 0 ? rows * static_cast<int>(ld) * 2 : 0, 0x00020000);
#pragma unroll
    for (int k = 0; k < 2 * TM; ++k)
      v[k] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rs, ((8 * k + (lane >> 3)) * static_cast<int>(ld) + n0 + 8 * (lane & 7)) * 2, 0, 0));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < 2 * TM; ++k) v[k] = make_uint4(0, 0, 0, 0);
  }
};

// What the epilogue combines a wave's rows with: P or U, and U's remainder.
template <int kKind, int TM>
struct Old {
  Rows<TM> c, lo;
  __device__ __forceinline__ void fetch(const OrthoArgs& a, int b, int m0, int n0) {
    if constexpr (kKind == kGram) return;
    const int lane = hidden_lane();
    c.fetch(a.C + b * a.batch_c, a.ldc, m0, n0, a.M, lane);
    if constexpr (is_update(kKind)) {
      if (a.lo_in != nullptr) lo.fetch(a.lo_in + b * a.batch_c, a.ldc, m0, n0, a.M, lane);
      else lo.clear();
    }
  }
};

// What rounding took from the diagonals of P or Q, for a wave's columns and (kSquare) rows, in LDS: this wave's alone. Issued
// before the loop, whose waits then cover the loads.
struct Kept {
  const float *rows, *cols;
  template <int kKind, int kRows>
  __device__ __forceinline__ void fetch(const OrthoArgs& a, int b, int m0, int n0, float* lds) {
    cols = lds;
    rows = lds + 64;
    if constexpr (kKind != kGram) {
      const int lane = threadIdx.x & 63;
      const i32x4_t desc = make_desc(a.d_in + b * a.ldc, ((a.N + 15) & ~15) * 4);   // of whole blocks; past them the rest is 0
      load4_to_lds(desc, lds_address(reinterpret_cast<const char*>(lds)), (n0 + lane) * 4);
      if constexpr (kKind == kSquare) {
#pragma unroll
        for (int m = 0; m < kRows; m += 64) load4_to_lds(desc, lds_address(reinterpret_cast<const char*>(lds + 64 + m)), (m0 + m + lane) * 4);
      }
    }
  }
  static constexpr int size(int rows) { return 64 + (rows + 63) / 64 * 64; }   // floats of a wave
};

template <int TM>
__device__ __forceinline__ void tile_put(char* tile, const Rows<TM>& rows, int lane) {
#pragma unroll
  for (int k = 0; k < 2 * TM; ++k) *reinterpret_cast<uint4*>(tile_chunk(tile, 8 * k + (lane >> 3), lane & 7)) = rows.v[k];
}
// A row block of fp32 results through the tile (4 KiB: 256 bytes a row, 16-byte chunk c of row m at c XOR m) to ``out``,
// M x N or turned. The loops stay loops: unrolled, all their addresses are kept at once and spill.
__device__ __forceinline__ void store_f32(char* tile, float* out, int M, int N, bool turned, int m0, int n0, const f32x4_t (&v)[4], int lane) {
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) *reinterpret_cast<f32x4_t*>(tile + i * 256 + (((4 * j + g) ^ i) << 4)) = v[j];
  tile_fence();
  if (turned) {
    float* d = out + static_cast<int64_t>(n0 + g) * M + m0 + i;
#pragma unroll 1
    for (int k = 0; k < 16; ++k, d += 4 * static_cast<int64_t>(M))
      if (m0 + i < M && n0 + 4 * k + g < N) *d = *reinterpret_cast<const float*>(tile + i * 256 + ((k ^ i) << 4) + 4 * g);
  } else {
    float* d = out + static_cast<int64_t>(m0) * N + n0 + lane;
#pragma unroll 1
    for (int k = 0; k < 16; ++k, d += N)
      if (m0 + k < M && n0 + lane < N) *d = *reinterpret_cast<const float*>(tile + k * 256 + (((lane >> 2) ^ k) << 4) + 4 * (lane & 3));
  }
  tile_fence();
}

// f(i, j, e) for the blocks of a wave's sub-tile that lie on the matrix's diagonal; its elements are those of r = 4 q + e.
template <int TM, class F>
__device__ __forceinline__ void on_diagonal(int m0, int n0, F f) {
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (m0 + 16 * i == n0 + 16 * j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) f(i, j, e);
      }
}

// The epilogue of a wave's sub-tile whose first row and column are m0 and n0. mirror: kGram, kSquare also write the
// transpose. tile: 4 KiB of LDS, this wave's alone, through which values pass between whole rows in memory and
// the matrix instructions' layout (lane: row lane mod 16 of a block, columns 4 (lane / 16) .. + 3).
template <int kKind, int TM>
__device__ __forceinline__ void finish(const OrthoArgs& a, int b, int m0, int n0, bool mirror, char* tile, f32x4_t (&acc)[TM][4],
                                       const Old<kKind, TM>& old, const Kept& kept) {
  const int lane = hidden_lane();
  const int r = lane & 15, q = lane >> 4;
  float f1 = a.f1, f2 = a.f2;
  if (a.scalars != nullptr) {
    if constexpr (kKind == kGram) f1 = a.scalars[b].p;
    if constexpr (is_update(kKind)) {
      f1 *= a.scalars[b].x;
      f2 *= a.scalars[b].x;
    }
  }
  // v = f1 acc, or f1 (old + its remainder) + f2 acc. Of P and Q the diagonals' roundings are kept: where the singular values are
  // alike, as of a wide random matrix, the diagonal's entries are too, and one rounding of them all shifts every singular value
  // (512 x 16384 to fp32 1.9e-3 off, with them 4.5e-4). With P = F + D, P P = F F + D F + F D; with Q = G + E, U Q = U G + U E.
  if constexpr (kKind == kGram) {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] *= f1;
  } else {
    // f1 + f2 D of this lane's columns of block j, and f2 D of its row of block i
    auto across = [&](int j) {
      f32x4_t v = *reinterpret_cast<const f32x4_t*>(kept.cols + 16 * j + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(f2, v[e], f1);
      return v;
    };
    auto combine = [&](const Rows<TM>& rows, float scale, auto factors) {
      tile_put<TM>(tile, rows, lane);
      tile_fence();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x4_t f = factors(j);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const half4_t v = __builtin_bit_cast(half4_t, *tile_four(tile, 16 * i + r, 16 * j + 4 * q));
          float down = 0;
          if constexpr (kKind == kSquare) down = f2 * kept.rows[16 * i + r];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(kKind == kSquare ? f[e] + down : f[e], static_cast<float>(v[e]), scale * acc[i][j][e]);
        }
      }
      tile_fence();
    };
    if (is_update(kKind) && a.lo_in != nullptr) {   // the remainder first: it is the smaller
      combine(old.lo, f2, [&](int) { return f32x4_t{f1, f1, f1, f1}; });
      combine(old.c, 1.0f, across);
    } else {
      combine(old.c, f2, across);
    }
    if constexpr (kKind == kSquare)
      on_diagonal<TM>(m0, n0, [&](int i, int j, int e) {
        if (r == 4 * q + e) acc[i][j][e] = __builtin_fmaf(f1, kept.rows[16 * i + r], acc[i][j][e]);
      });
  }

  if constexpr (kKind == kLast) {
    const int64_t o = static_cast<int64_t>(b) * a.M * a.N;
    if (a.out_type == 2) {
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        f32x4_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = acc[i][j] * a.out_factor;
        store_f32(tile, static_cast<float*>(a.out) + o, a.M, a.N, a.out_turned, m0 + 16 * i, n0, v, lane);
      }
      return;
    }
    const bool bf = a.out_type == 1;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint16_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = to_out16(acc[i][j][e] * a.out_factor, bf);
        *tile_four(tile, 16 * i + r, 16 * j + 4 * q) = make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16, h[2] | static_cast<uint32_t>(h[3]) << 16);
      }
    tile_fence();
    uint16_t* out = static_cast<uint16_t*>(a.out) + o;
    if (a.out_turned) write_turned<TM>(tile, out, a.M, a.N, a.M, n0, m0, lane);
    else tile_store<TM>(tile, out, a.N, a.M, a.N, m0, n0, lane);
  } else {
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        half4_t h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          h[e] = static_cast<_Float16>(acc[i][j][e]);
          acc[i][j][e] -= static_cast<float>(h[e]);   // the remainder
        }
        *tile_four(tile, 16 * i + r, 16 * j + 4 * q) = __builtin_bit_cast(uint2, h);
      }
    if constexpr (kKind != kUpdate)
      on_diagonal<TM>(m0, n0, [&](int i, int j, int e) {
        const int n = n0 + 16 * j + 4 * q + e;
        if (r == 4 * q + e && n < a.ldc) a.d_out[b * a.ldc + n] = acc[i][j][e];
      });
    tile_fence();
    tile_store<TM>(tile, reinterpret_cast<uint16_t*>(a.D) + b * a.batch_c, a.ldc, a.M, a.ldc, m0, n0, lane);
    if (kKind == kUpdate || mirror) write_turned<TM>(tile, reinterpret_cast<uint16_t*>(a.T) + b * a.batch_t, a.ldt, a.N, a.M, n0, m0, lane);
    if (kKind == kUpdate && a.lo_out != nullptr) {
      tile_fence();
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          half4_t l;
#pragma unroll
          for (int e = 0; e < 4; ++e) l[e] = static_cast<_Float16>(acc[i][j][e]);
          *tile_four(tile, 16 * i + r, 16 * j + 4 * q) = __builtin_bit_cast(uint2, l);
        }
      tile_fence();
      tile_store<TM>(tile, reinterpret_cast<uint16_t*>(a.lo_out) + b * a.batch_c, a.ldc, a.M, a.ldc, m0, n0, lane);
    }
  }
}

// Which tile of a product: P and Q are symmetric, so of their tile grid (g x g) only the g (g + 1) / 2 on and above the
// diagonal are computed, in panels of eight tile rows walked column by column.
struct Tiles {
  TileOrder order;
  int sym, g, count;   // count: tiles of a matrix
};
__device__ __forceinline__ void tile_of(const Tiles& t, int id, int& tm, int& tn) {
  if (!t.sym) {
    order_tile(t.order, id, tm, tn);
  } else {
    id = xcd_remap(id, t.count);
    int row = 0;   // the panel's first tile row
    for (;;) {
      const int left = t.g - row, size = left > 8 ? 8 * left - 28 : left * (left + 1) / 2;
      if (id < size) break;
      id -= size;
      row += 8;
    }
    if (id < 36) {   // its triangle
      int c = 0;
      while ((c + 1) * (c + 2) / 2 <= id) ++c;
      tm = row + id - c * (c + 1) / 2;
      tn = row + c;
    } else {
      tm = row + ((id - 36) & 7);
      tn = row + 8 + ((id - 36) >> 3);
    }
  }
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
}

// A 128 x 128 tile of D = A B^T and its epilogue. Where few tiles exist: 512 x 512, 8 to 10 us a product, of which 3.5 are the
// launch and 3 the loop; bound by latency.
template <int kKind>
__global__ __launch_bounds__(kNtThreads) void ortho_product128_kernel(OrthoArgs a, Tiles tiles) {
  __shared__ __attribute__((aligned(1024))) char lds[kNt128Stages * kNt128Stage];
  __shared__ __attribute__((aligned(16))) float diagonals[8][Kept::size(32)];
  const int b = static_cast<int>(blockIdx.x) / tiles.count;
  int tm, tn;
  tile_of(tiles, static_cast<int>(blockIdx.x) - b * tiles.count, tm, tn);
  Nt128 t;
  t.init(lds, a.lda * 2, a.ldb * 2);
  // fetched before the loop (the loads count as older than the loop's, so its waits cover them): with few steps their
  // latency would show at the end
  Old<kKind, 2> old;
  old.fetch(a, b, tm * 128 + t.wm * 32, tn * 128 + t.wn * 64);
  Kept kept;
  kept.fetch<kKind, 32>(a, b, tm * 128 + t.wm * 32, tn * 128 + t.wn * 64, diagonals[t.wave]);
  const int steps = a.K / kStep;
  NtOperand oa, ob;
  oa.start(a.A + b * a.batch_a + static_cast<int64_t>(tm) * 128 * a.lda, min(128, a.M - tm * 128) * a.lda * 2);
  ob.start(a.B + b * a.batch_b + static_cast<int64_t>(tn) * 128 * a.ldb, min(128, a.N - tn * 128) * a.ldb * 2);
  f32x4_t acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  for (int s = 0; s < kNt128Stages; ++s) {
    t.load_stage(s);
    oa.set(s < steps);
    ob.set(s < steps);
    t.load_a<0>(oa);
    t.load_a<1>(oa);
    t.load_b<0>(ob);
    t.load_b<1>(ob);
  }
  constexpr int kLoads = 4;
  wait_loads<kLoads * (kNt128Stages - 1)>();
  lds_barrier();
  Chunks af[2][2], bf[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) af[0][i] = t.a(i);
#pragma unroll
  for (int j = 0; j < 4; ++j) bf[j] = t.b(j);
  auto step = [&](int s, const Chunks (&now)[2], Chunks (&next)[2]) {
    wait_loads<kLoads * (kNt128Stages - 2)>();   // step s + 1 has landed everywhere, and step s's stage is free
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
    t.load_stage(s & (kNt128Stages - 1));
    t.read_stage((s + 1) & (kNt128Stages - 1));
    oa.set(s + kNt128Stages < steps);
    ob.set(s + kNt128Stages < steps);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, h ? bf[j].hi : bf[j].lo),
                                                             __builtin_bit_cast(half8_t, h ? now[i].hi : now[i].lo), acc[i][j], 0, 0, 0);
      bf[j] = t.b(j);   // past the last step: zeros that nobody uses
      if (j < 2) next[j] = t.a(j);
      if (j == 0) t.load_a<0>(oa);
      if (j == 1) t.load_b<0>(ob);
      if (j == 2) t.load_a<1>(oa);
      if (j == 3) t.load_b<1>(ob);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  int s = 0;
  for (; s + 1 < steps; s += 2) {
    step(s, af[0], af[1]);
    step(s + 1, af[1], af[0]);
  }
  if (s < steps) step(s, af[0], af[1]);
  wait_loads<0>();   // no direct load may still be writing this workgroup's LDS
  lds_barrier();     // nobody reads the stages any more
  finish<kKind>(a, b, tm * 128 + t.wm * 32, tn * 128 + t.wn * 64, tm != tn, lds + t.wave * (2 * 2048), acc, old, kept);
}

// The same with a 256 x 256 tile and the two-group loop of nt_tile.hpp. 8192 x 8192: the symmetric products 411 and 421 us and 14
// for joining split tiles, the update 825, the last 770: 1.3 to 1.43 PFLOP/s; a library product of the same size reaches 1.48. Bound by the
// matrix instructions at the clock that the board's power allows.
template <int kKind>
__global__ __launch_bounds__(kNtThreads) void ortho_product256_kernel(OrthoArgs a, Tiles tiles, Deal deal, float* __restrict__ work) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kNtStage];
  __shared__ __attribute__((aligned(16))) float diagonals[8][Kept::size(128)];
  const Share share = share_of(deal, static_cast<int>(blockIdx.x));
  const int b = share.tile / tiles.count;
  int tm, tn;
  tile_of(tiles, share.tile - b * tiles.count, tm, tn);
  NtTile t;
  t.init(lds, a.lda * 2, a.ldb * 2);
  Kept kept;
  kept.fetch<kKind, 128>(a, b, tm * 256 + t.wm * 128, tn * 256 + t.wn * 64, diagonals[t.wave]);
  const int steps = share.s1 - share.s0;
  NtOperand oa, ob;
  {
    const int64_t k0 = static_cast<int64_t>(share.s0) * kNtRow;
    oa.start(reinterpret_cast<const char*>(a.A + b * a.batch_a + static_cast<int64_t>(tm) * 256 * a.lda) + k0, min(256, a.M - tm * 256) * a.lda * 2 - k0);
    ob.start(reinterpret_cast<const char*>(a.B + b * a.batch_b + static_cast<int64_t>(tn) * 256 * a.ldb) + k0, min(256, a.N - tn * 256) * a.ldb * 2 - k0);
  }
  f32x4_t acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
  Chunks af[4], bf[4];
  auto load_first = [&]() {
    t.load_b<0>(ob);
    t.load_b<1>(ob);
    t.load_b<2>(ob);
    t.load_b<3>(ob);
    t.load_a<0>(oa);
    t.load_a<1>(oa);
  };
  oa.set(steps > 0);
  ob.set(steps > 0);
  load_first();
  t.load_a<2>(oa);
  t.load_a<3>(oa);
  t.stage(1, 0);
  oa.set(steps > 1);
  ob.set(steps > 1);
  load_first();
  auto memory0 = [&](int) {   // step s + 1's stage
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
  };
  auto memory1 = [&](int s) {   // step s + 2's stage is step s's
    const int to = s & 1 ? kNtStage : -kNtStage;   // from the stage of step s + 1 to the other one
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
    t.a_lo -= to;
    t.a_hi -= to;
    t.b_lo -= to;
    t.b_hi -= to;
  };
  auto multiply = [&](f32x4_t (&c)[8][4], int i0) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int j = i & 1 ? 3 - jj : jj;   // B forward and backward: one operand stays at every change of A
          c[i0 + i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, h ? bf[j].hi : bf[j].lo),
                                                                __builtin_bit_cast(half8_t, h ? af[i].hi : af[i].lo), c[i0 + i][j], 0, 0, 0);
        }
  };
  auto compute0 = [&](int s) {
    oa.set(s + 2 < steps);
    ob.set(s + 2 < steps);
    multiply(acc, 0);
  };
  nt_loop<6, 2>(t.wm, steps, memory0, memory1, compute0, [&](int) { multiply(acc, 4); });
  if (share.unit >= 0) {
    write_part(deal, work, share.unit, t.wave, t.lane, a.M - tm * 256 - t.wm * 128, acc);
    return;
  }
  lds_barrier();   // nobody reads the stages any more
  // two row blocks at a time, the next two's old values on their way; the row is hidden from the compiler, which would
  // otherwise compute all addresses before the first of them and spill
  int m = tm * 256 + t.wm * 128;
  const int n0 = tn * 256 + t.wn * 64;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    int next = m + 32;
    asm volatile("" : "+s"(next)::"memory");
    Old<kKind, 2> old;
    old.fetch(a, b, m, n0);
    f32x4_t two[2][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      two[0][j] = acc[i][j];
      two[1][j] = acc[i + 1][j];
    }
    finish<kKind, 2>(a, b, m, n0, tm != tn, lds + t.wave * (2 * 2048), two, old, kept);
    kept.rows += 32;
    tile_fence();
    m = next;
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Joins the parts of a split tile: a workgroup a row block of it.
template <int kKind>
__global__ __launch_bounds__(kNtThreads) void ortho_join_kernel(OrthoArgs a, Tiles tiles, Deal deal, float* __restrict__ work) {
  __shared__ __attribute__((aligned(1024))) char lds[8 * 4096];
  __shared__ __attribute__((aligned(16))) float diagonals[8][Kept::size(16)];
  const int tile = deal.whole + static_cast<int>(blockIdx.x) / 8, i = static_cast<int>(blockIdx.x) & 7;
  const int b = tile / tiles.count;
  int tm, tn;
  tile_of(tiles, tile - b * tiles.count, tm, tn);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  f32x4_t acc[1][4];
  if (tm * 256 + (wave >> 2) * 128 + i * 16 >= a.M) return;
  const int m0 = tm * 256 + (wave >> 2) * 128 + i * 16, n0 = tn * 256 + (wave & 3) * 64;
  Old<kKind, 1> old;
  old.fetch(a, b, m0, n0);
  Kept kept;
  kept.fetch<kKind, 16>(a, b, m0, n0, diagonals[wave]);
  join_parts(deal, work, tile, i, wave, lane, acc);
  wait_loads<0>();   // the diagonals, which only this wave reads
  finish<kKind>(a, b, m0, n0, tm != tn, lds + wave * 4096, acc, old, kept);
}

// ---- matrices with a short side --------------------------------------------------------------------
//
// r <= 128: P fits a workgroup, so a step is one launch. A matrix's rows of U are dealt to ``chunks`` workgroups of eight
// waves. Each joins all chunks' shares of P = W W^T (fp32, in order), squares it, updates its own rows of U, and leaves the
// share of the next P that its new rows make, straight from LDS. What bounds it is latency: the launch, the joining, LDS. A
// step takes 14.6 us at 16 x 128 x 1000, 11 at 128 x 128, 5.8 at 12 x 30 x 200.
//
// kR: r rounded up to 64 or 128; zeros fill the rest. Only blocks on and above P's diagonal are computed and passed on.

template <int kR>
struct Small {
  static constexpr int kBlocks = kR / 16;                     // 16 x 16 blocks across
  static constexpr int kUpper = kBlocks * (kBlocks + 1) / 2;  // on and above the diagonal: 10 or 36
  static constexpr int kWaves = 8;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kMine = (kUpper + kWaves - 1) / kWaves;   // of a wave
  // fp16 values of an LDS row: 208 or 304 bytes, odd multiples of 16 (16 rows read at one chunk touch all banks) at which
  // the four rows of a transposing read's lane group lie in different banks too
  static constexpr int kPitch = kR == 64 ? 104 : 152;
  static constexpr int kRows = 128;                           // rows of U at a time
  static constexpr int kWide = 152;                           // the pitch of their transpose
  static constexpr int64_t kShare = kUpper * 256;             // floats of a chunk's share of P
};

struct SmallArgs {
  const double* norms;
  OrthoScalars* scalars;
  _Float16* u;             // c x kR of each matrix, dense, with its remainder (lo: null where there is none yet)
  _Float16* lo;
  _Float16* lo_out;
  const float* p_in;       // chunks shares of P of each matrix
  float* p_out;
  int r, c, chunks, batch;
  float f1q, f2q, a, kq, kx;   // Q = f1q P + f2q PP; U' = a U + U Q / kq
  int first;
  void* out;               // last step
  int out_type, out_turned;
  float out_factor;        // 1 / kx
};

// Block t of the upper triangle, column by column (row <= column): the column is floor((sqrt(8 t + 1) - 1) / 2), with a half
// added under the root, where the next whole square is at least 8 away, against its rounding.
__device__ __forceinline__ void upper_block(int t, int& row, int& col) {
  col = __builtin_amdgcn_readfirstlane(static_cast<int>((__builtin_amdgcn_sqrtf(8.0f * static_cast<float>(t) + 1.5f) - 1.0f) * 0.5f));
  row = t - col * (col + 1) / 2;
}

// A wave's blocks of P; one past the last is computed as the last again and not stored.
template <int kR>
struct Blocks {
  int row[Small<kR>::kMine], col[Small<kR>::kMine], at[Small<kR>::kMine];
  bool mine[Small<kR>::kMine];
  __device__ __forceinline__ explicit Blocks(int wave) {
#pragma unroll
    for (int e = 0; e < Small<kR>::kMine; ++e) {
      const int t = wave + Small<kR>::kWaves * e;
      mine[e] = t < Small<kR>::kUpper;
      at[e] = mine[e] ? t : Small<kR>::kUpper - 1;
      upper_block(at[e], row[e], col[e]);
    }
  }
};

// A lane's eight consecutive k of one row of a 16 x 16 x 32 operand.
__device__ __forceinline__ half8_t row_operand(const _Float16* lds, int pitch, int row0, int k0) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const half8_t*>(lds + (row0 + (lane & 15)) * pitch + k0 + 8 * (lane >> 4));
}
// The same of one column: rows k0 + 8 (lane / 16) .. + 7 of column col0 + lane mod 16, by two transposing reads.
__device__ __forceinline__ half8_t column_operand(const _Float16* lds, int pitch, int k0, int col0) {
  const int lane = threadIdx.x & 63, i = lane & 15;
  const _Float16* p = lds + (k0 + 8 * (lane >> 4) + (i >> 2)) * pitch + col0 + 4 * (i & 3);
  const uint2 lo = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p));
  const uint2 hi = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * pitch)));
  return __builtin_bit_cast(half8_t, make_uint4(lo.x, lo.y, hi.x, hi.y));
}

// Adds the share of P that the kRows rows of U in LDS (kTurned: W's columns, rows of kWide) make to this wave's blocks. The
// operands are read for each block: held in registers for all of them, a wave's choice of blocks becomes a branch each.
template <int kR, bool kTurned = false>
__device__ __forceinline__ void small_gram(const _Float16* u, const Blocks<kR>& blocks, f32x4_t (&acc)[Small<kR>::kMine]) {
  typedef Small<kR> S;
#pragma unroll
  for (int k0 = 0; k0 < S::kRows; k0 += 32)
#pragma unroll
    for (int e = 0; e < S::kMine; ++e) {
      half8_t a, b;
      if constexpr (kTurned) {
        a = row_operand(u, S::kWide, 16 * blocks.row[e], k0);
        b = row_operand(u, S::kWide, 16 * blocks.col[e], k0);
      } else {
        a = column_operand(u, S::kPitch, k0, 16 * blocks.row[e]);
        b = column_operand(u, S::kPitch, k0, 16 * blocks.col[e]);
      }
      acc[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc[e], 0, 0, 0);
    }
}
template <int kR>
__device__ __forceinline__ void small_pass_on(float* share, const Blocks<kR>& blocks, f32x4_t (&acc)[Small<kR>::kMine]) {
#pragma unroll
  for (int e = 0; e < Small<kR>::kMine; ++e)
    if (blocks.mine[e]) *reinterpret_cast<f32x4_t*>(share + (blocks.at[e] * 64 + (threadIdx.x & 63)) * 4) = acc[e];
}

// Where U's remainder keeps the four values that a lane of the step kernel combines with its row m's columns 16 j + 4 q ..:
// as its registers hold them, so that loads and stores are whole lines.
template <int kR>
__device__ __forceinline__ int64_t remainder_at(int b, int c, int m, int n) {
  const int64_t pieces = (c + Small<kR>::kRows - 1) / Small<kR>::kRows;
  return ((((b * pieces + m / Small<kR>::kRows) * 8 + m % Small<kR>::kRows / 16) * Small<kR>::kBlocks + n / 16) * 64 + n % 16 / 4 * 16 + m % 16) * 4 + n % 4;
}

// A symmetric matrix's block: this lane's four values are rows 16 row + 4 (lane / 16) .. + 3, column 16 col + lane mod 16.
__device__ __forceinline__ void store_symmetric(_Float16* lds, int pitch, int row, int col, half4_t v) {
  const int lane = threadIdx.x & 63, m = 16 * col + (lane & 15), n = 16 * row + 4 * (lane >> 4);
  *reinterpret_cast<half4_t*>(lds + m * pitch + n) = v;
  if (row != col) {
#pragma unroll
    for (int e = 0; e < 4; ++e) lds[(n + e) * pitch + m] = v[e];
  }
}

// The rows of U that chunk ``part`` of ``chunks`` takes, in whole pieces of kRows.
__device__ __forceinline__ void chunk_rows(int c, int chunks, int part, int rows, int& begin, int& end) {
  const int pieces = (c + rows - 1) / rows;
  begin = static_cast<int>(static_cast<int64_t>(pieces) * part / chunks) * rows;
  end = min(c, static_cast<int>(static_cast<int64_t>(pieces) * (part + 1) / chunks) * rows);
}

// A workgroup's matrix and chunk. Workgroups go to the XCDs in turn, so matrix b's chunks are numbered to fall on one XCD (b
// mod 8): they all read the same shares, once from memory and then from its L2 (16 x 128 x 1000 97 us -> 80).
__device__ __forceinline__ bool small_place(const SmallArgs& a, int& b, int& part) {
  const int id = static_cast<int>(blockIdx.x), k = id / kNumXcds;
  b = k / a.chunks * kNumXcds + id % kNumXcds;
  part = k % a.chunks;
  return b < a.batch;
}

// x -> U (scaled as ortho_enter_kernel does), its remainder, and the shares of the first P.
template <int kType, int kR>
__global__ __launch_bounds__(Small<kR>::kThreads) void ortho_small_enter_kernel(const void* __restrict__ x, int64_t ld, int64_t batch_ld, bool tall,
                                                                int parts, float eps, SmallArgs a) {
  typedef Small<kR> S;
  __shared__ __attribute__((aligned(16))) _Float16 u[S::kRows * S::kPitch];
  __shared__ double total[S::kWaves];
  int b, part;
  if (!small_place(a, b, part)) return;
  const int t = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  double s = 0;
  for (int i = t; i < parts; i += S::kThreads) s += a.norms[static_cast<int64_t>(b) * parts + i];
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if ((t & 63) == 0) total[t >> 6] = s;
  __syncthreads();
  double squares = 0;
#pragma unroll
  for (int w = 0; w < S::kWaves; ++w) squares += total[w];
  const Entry entry(squares, eps, a.kx);
  const Blocks<kR> blocks(wave);
  if (part == 0 && t == 0) a.scalars[b] = entry.scalars(a.kx);
  int begin, end;
  chunk_rows(a.c, a.chunks, part, S::kRows, begin, end);
  f32x4_t acc[S::kMine];
#pragma unroll
  for (int e = 0; e < S::kMine; ++e) acc[e] = f32x4_t{0, 0, 0, 0};
  for (int c0 = begin; c0 < end; c0 += S::kRows) {
    // rows of x hold eight neighbouring values of a row of U (tall) or of a column of it
    constexpr int kEights = kR * S::kRows / 8 / S::kThreads;
    float v[kEights][8];
#pragma unroll
    for (int i = 0; i < kEights; ++i) {
      const int id = i * S::kThreads + t;
      const int row = tall ? c0 + id / (kR / 8) : id / (S::kRows / 8), at = tall ? id % (kR / 8) * 8 : c0 + id % (S::kRows / 8) * 8;
      const int rows = tall ? a.c : a.r, cols = tall ? a.r : a.c;
      eight<kType>(x, b * batch_ld + row * ld + at, row < rows ? cols - at : 0, v[i]);
    }
    if (c0 != begin) __syncthreads();   // the last piece's readers are done
#pragma unroll
    for (int i = 0; i < kEights; ++i) {
      const int id = i * S::kThreads + t;
      half8_t h, l;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float w = __builtin_ldexpf(v[i][e], entry.k);
        h[e] = static_cast<_Float16>(w);
        l[e] = static_cast<_Float16>(w - static_cast<float>(h[e]));
      }
      if (tall) {
        const int row = id / (kR / 8), at = id % (kR / 8) * 8;
        *reinterpret_cast<half8_t*>(u + row * S::kPitch + at) = h;
        if constexpr (kType == 2) {
          const half4_t l0 = {l[0], l[1], l[2], l[3]}, l1 = {l[4], l[5], l[6], l[7]};
          *reinterpret_cast<half4_t*>(a.lo + remainder_at<kR>(b, a.c, c0 + row, at)) = l0;
          *reinterpret_cast<half4_t*>(a.lo + remainder_at<kR>(b, a.c, c0 + row, at + 4)) = l1;
        }
      } else {
        const int n = id / (S::kRows / 8), at = id % (S::kRows / 8) * 8;
        *reinterpret_cast<half8_t*>(u + n * S::kWide + at) = h;
        if constexpr (kType == 2) {
#pragma unroll
          for (int e = 0; e < 8; ++e) a.lo[remainder_at<kR>(b, a.c, c0 + at + e, n)] = l[e];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kEights; ++i) {
      const int id = i * S::kThreads + t;
      int row, at;
      uint4 v;
      if (tall) {
        row = c0 + id / (kR / 8);
        at = id % (kR / 8) * 8;
        v = *reinterpret_cast<const uint4*>(u + id / (kR / 8) * S::kPitch + at);
      } else {   // a wave: 16 rows of U, 32 of its columns
        const int blk = i * S::kWaves + wave;
        row = c0 + 16 * (blk % 8) + (t & 15);
        at = 32 * (blk / 8) + 8 * ((t & 63) >> 4);
        v = __builtin_bit_cast(uint4, column_operand(u, S::kWide, 32 * (blk / 8), 16 * (blk % 8)));
      }
      if (row < a.c) *reinterpret_cast<uint4*>(a.u + (static_cast<int64_t>(b) * a.c + row) * kR + at) = v;
    }
    if (tall) small_gram<kR>(u, blocks, acc);
    else small_gram<kR, true>(u, blocks, acc);
  }
  small_pass_on<kR>(a.p_out + (static_cast<int64_t>(b) * a.chunks + part) * S::kShare, blocks, acc);
}

template <int kR>
__global__ __launch_bounds__(Small<kR>::kThreads) void ortho_small_step_kernel(SmallArgs a) {
  typedef Small<kR> S;
  __shared__ __attribute__((aligned(16))) _Float16 ps[kR * S::kPitch], qs[kR * S::kPitch], u[S::kRows * S::kPitch];
  __shared__ __attribute__((aligned(16))) float dp[kR], dq[kR];   // what rounding took from P's and Q's diagonals
  int b, part;
  if (!small_place(a, b, part)) return;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r = lane & 15, q = lane >> 4;
  int begin, end;
  chunk_rows(a.c, a.chunks, part, S::kRows, begin, end);

  // this wave's 16 rows of U and their remainder: the first piece's are on their way while P is joined
  uint4 rows[kR / 32];
  half4_t l4[S::kBlocks];
  auto fetch = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kR / 32; ++i) {
      const int id = i * 64 + lane, m = c0 + 16 * wave + id / (kR / 8);
      rows[i] = make_uint4(0, 0, 0, 0);
      if (m < a.c) rows[i] = *reinterpret_cast<const uint4*>(a.u + (static_cast<int64_t>(b) * a.c + m) * kR + id % (kR / 8) * 8);
    }
    const half4_t* lo = reinterpret_cast<const half4_t*>(a.lo + remainder_at<kR>(b, a.c, c0 + 16 * wave + r, 4 * q));
#pragma unroll
    for (int j = 0; j < S::kBlocks; ++j) {
      l4[j] = half4_t{0, 0, 0, 0};
      if (a.lo != nullptr) l4[j] = lo[64 * j];
    }
  };
  fetch(begin);
  const Blocks<kR> blocks(wave);

  // P: the chunks' shares added in order, rounded. Four chunks' loads are in flight together; a chunk that is not there is
  // read as the last one and not added.
  const float fp = a.first ? a.scalars[b].p : kP / (a.kx * a.kx);
  const float fx = a.first ? a.scalars[b].x : 1.0f;
  f32x4_t acc[S::kMine];
#pragma unroll
  for (int e = 0; e < S::kMine; ++e) acc[e] = f32x4_t{0, 0, 0, 0};
  const float* in = a.p_in + static_cast<int64_t>(b) * a.chunks * S::kShare;
  for (int p = 0; p < a.chunks; p += 4) {
    f32x4_t v[4][S::kMine];
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < S::kMine; ++e)
        v[k][e] = *reinterpret_cast<const f32x4_t*>(in + min(p + k, a.chunks - 1) * S::kShare + (blocks.at[e] * 64 + lane) * 4);
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < S::kMine; ++e)
        if (p + k < a.chunks) acc[e] += v[k][e];
  }
  // The diagonals' roundings are kept: where the singular values are alike, as of a wide random matrix, the diagonal's entries
  // are too, and one rounding of them all shifts every singular value (20 x 4000: 2.6e-3 off with the bf16 output's 1.7e-3).
  auto keep_diagonal = [&](float* to, int e, const f32x4_t& exact, const half4_t& rounded) {
    if (!blocks.mine[e] || blocks.row[e] != blocks.col[e]) return;
    const f32x4_t d = {exact[0] - static_cast<float>(rounded[0]), exact[1] - static_cast<float>(rounded[1]),
                       exact[2] - static_cast<float>(rounded[2]), exact[3] - static_cast<float>(rounded[3])};
    if (r >> 2 == q) to[16 * blocks.row[e] + r] = r & 2 ? (r & 1 ? d[3] : d[2]) : (r & 1 ? d[1] : d[0]);
  };
  f32x4_t whole[S::kMine];
  half4_t mine[S::kMine];
#pragma unroll
  for (int e = 0; e < S::kMine; ++e) {
    whole[e] = acc[e] * fp;
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[e][i] = static_cast<_Float16>(whole[e][i]);
    keep_diagonal(dp, e, whole[e], mine[e]);
    if (blocks.mine[e]) store_symmetric(ps, S::kPitch, blocks.row[e], blocks.col[e], mine[e]);
    acc[e] = f32x4_t{0, 0, 0, 0};
  }
  __syncthreads();
  // Q = f1q P + f2q P P; with P = F + D, F rounded and D diagonal, P P = F F + D F + F D
#pragma unroll
  for (int k0 = 0; k0 < kR; k0 += 32)
#pragma unroll
    for (int e = 0; e < S::kMine; ++e)
      acc[e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(row_operand(ps, S::kPitch, 16 * blocks.row[e], k0), row_operand(ps, S::kPitch, 16 * blocks.col[e], k0), acc[e], 0, 0, 0);
#pragma unroll
  for (int e = 0; e < S::kMine; ++e) {
    half4_t v;
    const f32x4_t down = *reinterpret_cast<const f32x4_t*>(dp + 16 * blocks.row[e] + 4 * q);
    const float across = dp[16 * blocks.col[e] + r];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[e][i] = __builtin_fmaf(a.f1q, whole[e][i], a.f2q * __builtin_fmaf(static_cast<float>(mine[e][i]), down[i] + across, acc[e][i]));
      v[i] = static_cast<_Float16>(acc[e][i]);
    }
    keep_diagonal(dq, e, acc[e], v);
    if (blocks.mine[e]) store_symmetric(qs, S::kPitch, blocks.row[e], blocks.col[e], v);
    acc[e] = f32x4_t{0, 0, 0, 0};
  }
  const float fa = a.a * fx, fq = fx / a.kq;
  for (int c0 = begin; c0 < end; c0 += S::kRows) {
#pragma unroll
    for (int i = 0; i < kR / 32; ++i) {
      const int id = i * 64 + lane;
      *reinterpret_cast<uint4*>(u + (16 * wave + id / (kR / 8)) * S::kPitch + id % (kR / 8) * 8) = rows[i];
    }
    __syncthreads();   // Q is whole (first piece), and U's rows
    f32x4_t d[S::kBlocks];
    {
      half8_t x[kR / 32];
#pragma unroll
      for (int k = 0; k < kR / 32; ++k) x[k] = row_operand(u, S::kPitch, 16 * wave, 32 * k);
#pragma unroll
      for (int j = 0; j < S::kBlocks; ++j) {
        d[j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int k = 0; k < kR / 32; ++k)
          d[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(row_operand(qs, S::kPitch, 16 * j, 32 * k), x[k], d[j], 0, 0, 0);
      }
    }
    const int row = 16 * wave + r, m = c0 + row;
    half4_t l[S::kBlocks];
#pragma unroll
    for (int j = 0; j < S::kBlocks; ++j) {
      half4_t* at = reinterpret_cast<half4_t*>(u + row * S::kPitch + 16 * j + 4 * q);
      const half4_t old = *at;
      half4_t h;
      const f32x4_t left = *reinterpret_cast<const f32x4_t*>(dq + 16 * j + 4 * q);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        d[j][e] = __builtin_fmaf(fa, static_cast<float>(old[e]) + static_cast<float>(l4[j][e]),
                                 fq * __builtin_fmaf(left[e], static_cast<float>(old[e]), d[j][e]));
        h[e] = static_cast<_Float16>(d[j][e]);
        l[j][e] = static_cast<_Float16>(d[j][e] - static_cast<float>(h[e]));
      }
      if (a.out != nullptr && a.out_type != 2) {
        const bool bf = a.out_type == 1;
        *reinterpret_cast<uint2*>(at) = make_uint2(to_out16(d[j][0] * a.out_factor, bf) | static_cast<uint32_t>(to_out16(d[j][1] * a.out_factor, bf)) << 16,
                                                   to_out16(d[j][2] * a.out_factor, bf) | static_cast<uint32_t>(to_out16(d[j][3] * a.out_factor, bf)) << 16);
      } else {
        *at = h;
      }
    }
    if (a.out == nullptr) {   // the rows from LDS, whole lines at a time; only this wave touches them
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int i = 0; i < kR / 32; ++i) {
        const int id = i * 64 + lane, mr = 16 * wave + id / (kR / 8), n = id % (kR / 8) * 8;
        if (c0 + mr < a.c)
          *reinterpret_cast<uint4*>(a.u + (static_cast<int64_t>(b) * a.c + c0 + mr) * kR + n) = *reinterpret_cast<const uint4*>(u + mr * S::kPitch + n);
      }
      if (a.lo_out != nullptr) {
        half4_t* o = reinterpret_cast<half4_t*>(a.lo_out + remainder_at<kR>(b, a.c, m, 4 * q));
#pragma unroll
        for (int j = 0; j < S::kBlocks; ++j) o[64 * j] = l[j];
      }
    }
    if (m < a.c && a.out != nullptr && a.out_type == 2) {
      float* o = static_cast<float*>(a.out) + static_cast<int64_t>(b) * a.c * a.r + (a.out_turned ? m : static_cast<int64_t>(m) * a.r);
      const int64_t step = a.out_turned ? a.c : 1;
#pragma unroll
      for (int j = 0; j < S::kBlocks; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (16 * j + 4 * q + e < a.r) o[(16 * j + 4 * q + e) * step] = d[j][e] * a.out_factor;
    }
    __syncthreads();
    if (c0 + S::kRows < end) fetch(c0 + S::kRows);
    if (a.out == nullptr) {
      small_gram<kR>(u, blocks, acc);
    } else if (a.out_type != 2) {
      // 16-bit results from LDS, eight neighbouring values of a row of the output a lane
      uint16_t* o = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(b) * a.c * a.r;
      const int cols = a.out_turned ? a.c : a.r, rows = a.out_turned ? a.r : a.c;
      const bool aligned = (cols & 7) == 0;
      constexpr int kEights = kR * S::kRows / 8 / S::kThreads;
#pragma unroll
      for (int i = 0; i < kEights; ++i) {
        uint4 v;
        int row, col;
        if (a.out_turned) {   // a wave: 16 rows of the output, 32 columns
          const int blk = i * S::kWaves + wave;
          row = 16 * (blk % S::kBlocks) + r;
          col = c0 + 32 * (blk / S::kBlocks) + 8 * q;
          v = __builtin_bit_cast(uint4, column_operand(u, S::kPitch, 32 * (blk / S::kBlocks), 16 * (blk % S::kBlocks)));
        } else {
          const int id = i * S::kThreads + t;
          row = c0 + id / (kR / 8);
          col = id % (kR / 8) * 8;
          v = *reinterpret_cast<const uint4*>(u + id / (kR / 8) * S::kPitch + col);
        }
        if (row >= rows) continue;
        uint16_t* p = o + static_cast<int64_t>(row) * cols + col;
        if (aligned && col + 8 <= cols) {
          *reinterpret_cast<uint4*>(p) = v;
        } else {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (col + e < cols) p[e] = static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
        }
      }
    }
    if (c0 + S::kRows < end) __syncthreads();   // before the next piece's rows
  }
  if (a.out == nullptr) small_pass_on<kR>(a.p_out + (static_cast<int64_t>(b) * a.chunks + part) * S::kShare, blocks, acc);
}

Tiles make_tiles(int kind, int M, int N, int t) {
  const int gm = (M + t - 1) / t, gn = (N + t - 1) / t;
  Tiles s;
  s.order = make_tile_order(kPanel, 1, gm, gn, gm < 8 ? gm : 8, 1, 1);
  s.sym = !is_update(kind);
  s.g = gm;
  s.count = s.sym ? gm * (gm + 1) / 2 : gm * gn;
  return s;
}

// The tile of a product, by what either would take, in us, fitted to measured launches: a 128 tile 0.45 a step, a 256 tile
// 1.1 to 1.5 (the more CUs are busy, the lower their clock), and what a round costs besides (the update's epilogue most);
// split tiles 5 for joining and their sums' traffic. Whole calls on r x c, all 128 / all 256 tiles: 1024 x 1024 189 / 320,
// 1024 x 4096 292 / 419, 2560 x 2560 489 / 654, 3100 x 3100 893 / 867, 2050 x 6140 712 / 728 (628 with each product's own
// choice), 4096 x 8192 2819 / 2259.
int tile_size(int kind, int M, int N, int K, int64_t batch) {
  static constexpr double kRound128[4] = {4, 5, 6, 6}, kRound256[4] = {8, 12, 15, 15};
  const double steps = K / kStep;
  const Deal d = make_deal(make_tiles(kind, M, N, 256).count * batch, K / kStep, 256);
  const double rounds = (d.whole + kCus - 1) / kCus, busy = d.blocks() < kCus ? static_cast<double>(d.blocks()) / kCus : 1;
  const double step = 1.1 + 0.4 * busy;
  const double t256 = rounds * (steps * step + kRound256[kind]) +
                      (d.parts > 1 ? steps / d.parts * step + kRound256[kind] + 5 + d.floats() / 1e6 : 0);
  const double t128 = (make_tiles(kind, M, N, 128).count * batch + kCus - 1) / kCus * (steps * 0.45 + kRound128[kind]);
  return t128 <= t256 ? 128 : 256;
}
int64_t part_floats(int kind, int M, int N, int K, int64_t batch) {
  const Tiles t = make_tiles(kind, M, N, 256);
  if (tile_size(kind, M, N, K, batch) != 256) return 0;
  return make_deal(t.count * batch, K / kStep, 256).floats();
}

template <int kKind>
hipError_t product(const OrthoArgs& a, int batch, float* work, hipStream_t s) {
  Tiles t = make_tiles(kKind, a.M, a.N, 256);
  if (tile_size(kKind, a.M, a.N, a.K, batch) == 256) {
    const Deal d = make_deal(static_cast<int64_t>(t.count) * batch, a.K / kStep, 256);
    hipLaunchKernelGGL((ortho_product256_kernel<kKind>), dim3(static_cast<unsigned>(d.blocks())), dim3(kNtThreads), 0, s, a, t, d, work);
    if (d.parts > 1)
      hipLaunchKernelGGL((ortho_join_kernel<kKind>), dim3(static_cast<unsigned>(d.tiles - d.whole) * 8), dim3(kNtThreads), 0, s, a, t, d, work);
  } else {
    t = make_tiles(kKind, a.M, a.N, 128);
    hipLaunchKernelGGL((ortho_product128_kernel<kKind>), dim3(static_cast<unsigned>(t.count) * batch), dim3(kNtThreads), 0, s, a, t);
  }
  return hipGetLastError();
}

// Parts of a matrix's norm that has ``pieces``. A launch takes less than 2^32 threads: no more than 2^20 workgroups in all.
int norm_parts(int64_t batch, int64_t pieces) {
  int64_t most = (int64_t{1} << 20) / batch;
  if (most > kNormParts) most = kNormParts;
  if (most < 1) most = 1;
  return static_cast<int>(pieces < most ? pieces : most);
}

template <int kType>
hipError_t launch_norm(const OrthoLaunch& l, int parts, double* norms, hipStream_t s) {
  const bool flat = l.ld == l.cols || l.rows == 1;   // then the matrix is one long row
  hipLaunchKernelGGL((ortho_norm_kernel<kType>), dim3(static_cast<unsigned>(l.batch * parts)), dim3(256), 0, s, l.x, flat ? 1 : l.rows,
                     flat ? l.rows * l.cols : l.cols, l.ld, l.batch_ld, parts, norms);
  return hipGetLastError();
}

template <int kType>
hipError_t launch_enter(const OrthoLaunch& l, int parts, double* norms, float kx, _Float16* straight, int64_t lds_, int64_t batch_s,
                  _Float16* turned, int64_t ldt, int64_t batch_t, _Float16* lo, bool lo_turned, OrthoScalars* scalars,
                  hipStream_t s) {
  const hipError_t e = launch_norm<kType>(l, parts, norms, s);
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>((l.cols + 63) / 64), static_cast<unsigned>((l.rows + 63) / 64), static_cast<unsigned>(l.batch));
  hipLaunchKernelGGL((ortho_enter_kernel<kType>), grid, dim3(256), 0, s, l.x, l.rows, l.cols, l.ld, l.batch_ld, parts, norms, l.eps,
                     kx, straight, lds_, batch_s, turned, ldt, batch_t, lo, lo_turned, scalars);
  return hipGetLastError();
}

template <int kType, int kR>
hipError_t launch_small(const OrthoLaunch& l, int parts, double* norms, SmallArgs a, float* share0, float* share1, hipStream_t s) {
  const hipError_t e = launch_norm<kType>(l, parts, norms, s);
  if (e != hipSuccess) return e;
  const dim3 grid(static_cast<unsigned>((a.batch + kNumXcds - 1) / kNumXcds * kNumXcds) * a.chunks);
  a.p_out = share0;
  hipLaunchKernelGGL((ortho_small_enter_kernel<kType, kR>), grid, dim3(Small<kR>::kThreads), 0, s, l.x, l.ld, l.batch_ld, l.rows > l.cols, parts, l.eps, a);
  _Float16* lo = a.lo;
  const int kept = l.steps - 3;   // as launch_ortho's
  for (int i = 0; i < l.steps; ++i) {
    a.first = i == 0;
    a.lo = i == 0 ? (kType == 2 ? lo : nullptr) : i <= kept ? lo : nullptr;
    a.lo_out = i < kept ? lo : nullptr;
    a.p_in = i & 1 ? share1 : share0;
    a.p_out = i & 1 ? share0 : share1;
    a.out = i == l.steps - 1 ? l.out : nullptr;
    hipLaunchKernelGGL((ortho_small_step_kernel<kR>), grid, dim3(Small<kR>::kThreads), 0, s, a);
  }
  return hipGetLastError();
}

int64_t up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

constexpr int64_t kSmallSide = 128;

// Chunks of a matrix with a short side: 128 rows of U each or more, evenly many, at most 16 (r > 64) or 24, since each reads all
// their shares of P, and as many as are resident at once. 1 x 100 x 4096 with at most 8 / 16 / 24: 147 / 115 / 129 us,
// 2 x 64 x 8000 123 / 83 / 79, 64 x 64 x 1000 with 4 / 8 (two rounds) 60 / 78.
int small_chunks(int64_t c, int64_t ldr, int64_t batch) {
  const int64_t pieces = up(c, 128) / 128, resident = kCus / up(batch, kNumXcds);
  int64_t most = ldr == 64 ? 24 : 16;
  if (most > resident) most = resident > 0 ? resident : 1;
  const int64_t each = (pieces + most - 1) / most;
  return static_cast<int>((pieces + each - 1) / each);
}

// Where the buffers of a call lie in its workspace, in bytes; each starts on a 256-byte boundary.
struct OrthoPlan {
  int64_t r, c, ldr, ldc;                    // W: r x ldc, U: c x ldr (fp16)
  bool small;
  int chunks;
  int64_t u0, u1, lo, w, p, q, dp, dq, norms, scalars, parts, bytes;   // small: p and q are the shares of P
};
OrthoPlan make_plan(int64_t batch, int64_t rows, int64_t cols) {
  OrthoPlan o{};
  o.r = rows < cols ? rows : cols;
  o.c = rows < cols ? cols : rows;
  o.small = o.r <= kSmallSide;
  o.ldr = o.small ? (o.r <= 64 ? 64 : 128) : up(o.r, kStep);
  o.ldc = up(o.c, kStep);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += up(bytes, 256);
    return here;
  };
  o.u0 = take(batch * o.c * o.ldr * 2);
  o.lo = take(batch * (o.small ? up(o.c, 128) : o.c) * o.ldr * 2);
  int64_t parts = o.c * ((o.r + kNormSpan - 1) / kNormSpan);   // of the norm, for either orientation
  if (parts < o.r * ((o.c + kNormSpan - 1) / kNormSpan)) parts = o.r * ((o.c + kNormSpan - 1) / kNormSpan);
  o.norms = take(batch * norm_parts(batch, parts) * 8);
  o.scalars = take(batch * 8);
  if (o.small) {
    o.chunks = small_chunks(o.c, o.ldr, batch);
    const int64_t share = (o.ldr == 64 ? Small<64>::kShare : Small<128>::kShare) * 4;
    o.p = take(batch * o.chunks * share);
    o.q = take(batch * o.chunks * share);
  } else {
    o.u1 = take(batch * o.c * o.ldr * 2);
    o.w = take(batch * o.r * o.ldc * 2);
    o.p = take(batch * o.r * o.ldr * 2);
    o.q = take(batch * o.r * o.ldr * 2);
    o.dp = take(batch * o.ldr * 4);
    o.dq = take(batch * o.ldr * 4);
    const int r = static_cast<int>(o.r), c = static_cast<int>(o.c);
    int64_t floats = part_floats(kGram, r, r, static_cast<int>(o.ldc), batch);
    for (const int64_t f : {part_floats(kSquare, r, r, static_cast<int>(o.ldr), batch), part_floats(kUpdate, c, r, static_cast<int>(o.ldr), batch)})
      if (f > floats) floats = f;
    o.parts = take(floats * 4);
  }
  o.bytes = at;
  return o;
}

// 2^floor(log2(v)) for v >= 1.
float pow2_below(double v) {
  float p = 1;
  while (p * 2.0 <= v) p *= 2;
  return p;
}

}  // namespace

int64_t ortho_workspace(int64_t batch, int64_t rows, int64_t cols) { return make_plan(batch, rows, cols).bytes; }

OrthoProduct ortho_product(int kind, int64_t batch, int64_t rows, int64_t cols) {
  const OrthoPlan o = make_plan(batch, rows, cols);
  if (o.small) return OrthoProduct{0, 1};
  const int r = static_cast<int>(o.r), M = is_update(kind) ? static_cast<int>(o.c) : r;
  const int K = static_cast<int>(kind == kGram ? o.ldc : o.ldr);
  const int tile = tile_size(kind, M, r, K, batch);
  return OrthoProduct{tile, tile == 256 ? make_deal(make_tiles(kind, M, r, 256).count * batch, K / kStep, 256).parts : 1};
}

hipError_t launch_ortho(const OrthoLaunch& l, hipStream_t s) {
  const OrthoPlan o = make_plan(l.batch, l.rows, l.cols);
  char* base = static_cast<char*>(l.work);
  auto half = [&](int64_t at) { return reinterpret_cast<_Float16*>(base + at); };
  _Float16 *u0 = half(o.u0), *u1 = half(o.u1), *lo = half(o.lo), *w = half(o.w), *p = half(o.p), *q = half(o.q);
  double* norms = reinterpret_cast<double*>(base + o.norms);
  OrthoScalars* scalars = reinterpret_cast<OrthoScalars*>(base + o.scalars);
  const int64_t bu = o.c * o.ldr, bw = o.r * o.ldc, bp = o.r * o.ldr;
  const bool tall = l.rows > l.cols;   // then x is U, else W
  // X's scale: an element of a matrix with norm 1 has rms 1 / sqrt(r c); at most 2^13, so no entry (<= 2) overflows
  double side = 1;
  while (side * side * 2 < static_cast<double>(o.r) * o.c && side < 8192) side *= 2;
  const float kx = static_cast<float>(side);
  // Q's: its entries are at most |b| 1.5 + |c| 2.25 where P's are at most 1.5
  const double most = 1.5 * __builtin_fabs(l.b) + 2.25 * __builtin_fabs(l.c);
  const float kq = most * 4096 <= 60000 ? 4096.0f : most <= 60000 ? pow2_below(60000 / most) : 1.0f;
  const int64_t pieces = l.ld == l.cols || l.rows == 1 ? (l.rows * l.cols + kNormSpan - 1) / kNormSpan : l.rows * ((l.cols + kNormSpan - 1) / kNormSpan);
  const int parts = norm_parts(l.batch, pieces);
  float* part_work = reinterpret_cast<float*>(base + o.parts);
  float *dp = reinterpret_cast<float*>(base + o.dp), *dq = reinterpret_cast<float*>(base + o.dq);
  if (o.small) {
    SmallArgs a{};
    a.norms = norms;
    a.scalars = scalars;
    a.u = u0;
    a.lo = lo;
    a.r = static_cast<int>(o.r);
    a.c = static_cast<int>(o.c);
    a.chunks = o.chunks;
    a.batch = static_cast<int>(l.batch);
    a.f1q = kq * l.b / kP;
    a.f2q = kq * l.c / (kP * kP);
    a.a = l.a;
    a.kq = kq;
    a.kx = kx;
    a.out_factor = 1 / kx;
    a.out_type = l.out_type;
    a.out_turned = !tall;
    float *share0 = reinterpret_cast<float*>(base + o.p), *share1 = reinterpret_cast<float*>(base + o.q);
    switch (l.dtype * 2 + (o.ldr == 128)) {
      case 0: return launch_small<0, 64>(l, parts, norms, a, share0, share1, s);
      case 1: return launch_small<0, 128>(l, parts, norms, a, share0, share1, s);
      case 2: return launch_small<1, 64>(l, parts, norms, a, share0, share1, s);
      case 3: return launch_small<1, 128>(l, parts, norms, a, share0, share1, s);
      case 4: return launch_small<2, 64>(l, parts, norms, a, share0, share1, s);
      default: return launch_small<2, 128>(l, parts, norms, a, share0, share1, s);
    }
  }
  // X's remainder serves the steps that two or more follow: what the last two add is multiplied by a^2 at most
  const int kept = l.steps - 3;
  _Float16* lo0 = l.dtype == 2 ? lo : nullptr;   // 16-bit inputs have no remainder
  _Float16 *straight = tall ? u0 : w, *turned = tall ? w : u0;
  const int64_t ls = tall ? o.ldr : o.ldc, lt = tall ? o.ldc : o.ldr, bs = tall ? bu : bw, bt = tall ? bw : bu;
  hipError_t e;
  switch (l.dtype) {
    case 0: e = launch_enter<0>(l, parts, norms, kx, straight, ls, bs, turned, lt, bt, lo0, !tall, scalars, s); break;
    case 1: e = launch_enter<1>(l, parts, norms, kx, straight, ls, bs, turned, lt, bt, lo0, !tall, scalars, s); break;
    default: e = launch_enter<2>(l, parts, norms, kx, straight, ls, bs, turned, lt, bt, lo0, !tall, scalars, s); break;
  }
  for (int i = 0; i < l.steps && e == hipSuccess; ++i) {
    OrthoArgs g{};
    g.A = w; g.B = w; g.lda = g.ldb = o.ldc; g.batch_a = g.batch_b = bw;
    g.M = g.N = static_cast<int>(o.r);
    g.K = static_cast<int>(o.ldc);
    g.scalars = i == 0 ? scalars : nullptr;
    g.f1 = kP / (kx * kx);
    g.d_out = dp;
    g.D = g.T = p; g.ldc = g.ldt = o.ldr; g.batch_c = g.batch_t = bp;
    if ((e = product<kGram>(g, static_cast<int>(l.batch), part_work, s)) != hipSuccess) break;
    OrthoArgs h{};
    h.A = p; h.B = p; h.lda = h.ldb = o.ldr; h.batch_a = h.batch_b = bp;
    h.M = h.N = static_cast<int>(o.r);
    h.K = static_cast<int>(o.ldr);
    h.f1 = kq * l.b / kP;
    h.f2 = kq * l.c / (kP * kP);
    h.d_in = dp;
    h.d_out = dq;
    h.C = p; h.D = h.T = q; h.ldc = h.ldt = o.ldr; h.batch_c = h.batch_t = bp;
    if ((e = product<kSquare>(h, static_cast<int>(l.batch), part_work, s)) != hipSuccess) break;
    OrthoArgs x{};
    x.A = i & 1 ? u1 : u0; x.B = q; x.lda = x.ldb = o.ldr; x.batch_a = bu; x.batch_b = bp;
    x.M = static_cast<int>(o.c);
    x.N = static_cast<int>(o.r);
    x.K = static_cast<int>(o.ldr);
    x.scalars = i == 0 ? scalars : nullptr;
    x.f1 = l.a;
    x.f2 = 1 / kq;
    x.d_in = dq;
    x.C = x.A; x.D = i & 1 ? u0 : u1; x.ldc = o.ldr; x.batch_c = bu;
    x.lo_in = i == 0 ? lo0 : i <= kept ? lo : nullptr;
    x.lo_out = i < kept ? lo : nullptr;
    x.T = w; x.ldt = o.ldc; x.batch_t = bw;
    if (i == l.steps - 1) {
      x.out = l.out;
      x.out_type = l.out_type;
      x.out_turned = !tall;
      x.out_factor = 1 / kx;
    }
    e = i == l.steps - 1 ? product<kLast>(x, static_cast<int>(l.batch), part_work, s) : product<kUpdate>(x, static_cast<int>(l.batch), part_work, s);
  }
  return e;
}

}  // namespace tbl
