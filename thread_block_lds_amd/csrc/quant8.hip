// Quantisation to 8-bit floating point with one fp32 scale for each group of values.
//
// A group is 1 x 128 values of a row (block 1) or a 128 x 128 block (block 128). With
//   most = max(2^-100, max |x| over the group),   M = 448 (e4m3) or 57344 (e5m2)
// the group's scale is most / M, rounded to fp32, and each code is the 8-bit value nearest to
// x M / most (ties to even), decided exactly: see Coder. A group that holds an infinity gets the scale inf and
// codes 0 (NaN in the place of the infinity); one that holds a NaN gets NaN in both.
//
// One pass: every value is read once, kept in registers between the maximum and the codes, and, where the
// transposed form is wanted too, quantised for both from the same registers (a 128 x 128 tile per workgroup
// holds whole groups of both directions). Bound by HBM traffic.
#include <stdint.h>

#include "internal.hpp"

namespace tbl {
namespace {

constexpr float kTiny = 0x1p-100f;
constexpr float kMost[2] = {448.0f, 57344.0f};
constexpr int kGroup = 128;

template <int kType>
struct In;   // 0: fp16, 1: bf16, 2: fp32
template <>
struct In<0> { typedef uint16_t T; };
template <>
struct In<1> { typedef uint16_t T; };
template <>
struct In<2> { typedef uint32_t T; };

// The value of an element's bits.
template <int kType>
__device__ __forceinline__ float value_of(uint32_t bits) {
  if constexpr (kType == 0) return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
  else if constexpr (kType == 1) return __builtin_bit_cast(float, bits << 16);
  else return __builtin_bit_cast(float, bits);
}

// Eight consecutive elements of a row as loaded.
template <int kType>
struct Eight {
  uint32_t w[kType == 2 ? 8 : 4];
  __device__ __forceinline__ uint32_t bits(int e) const {
    if constexpr (kType == 2) return w[e];
    else return (e & 1) ? w[e >> 1] >> 16 : w[e >> 1] & 0xFFFFu;
  }
  __device__ __forceinline__ float value(int e) const { return value_of<kType>(bits(e)); }
};

// Elements c .. c + 7 of the row at p (cols of them exist, the others read as 0). Whole eights are 16-byte loads at
// whatever alignment the element type has: gfx950 takes them unaligned.
template <int kType>
__device__ __forceinline__ Eight<kType> load_eight(const typename In<kType>::T* p, int64_t c, int64_t cols) {
  Eight<kType> v;
  if (c + 8 <= cols) {
    __builtin_memcpy(v.w, p + c, sizeof v.w);
    return v;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = c + e < cols ? p[c + e] : 0u;
    if constexpr (kType == 2) v.w[e] = b;
    else v.w[e >> 1] = (e & 1) ? v.w[e >> 1] | b << 16 : b;
  }
  return v;
}

typedef unsigned short u16x2_t __attribute__((ext_vector_type(2)));

// Magnitudes compared as unsigned bit patterns: the order of the finite ones, then inf, then NaN, so a NaN
// stays the maximum. 16-bit types: two in a register.
template <int kType>
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) {
  if constexpr (kType == 2) return max(a, b);
  else return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                                     __builtin_bit_cast(u16x2_t, b)));
}
template <int kType>
__device__ __forceinline__ uint32_t mag_bits(uint32_t w) {
  return kType == 2 ? w & 0x7FFFFFFFu : w & 0x7FFF7FFFu;
}

// The largest magnitude of eight, as one element's bits.
template <int kType>
__device__ __forceinline__ uint32_t most_of(const Eight<kType>& v) {
  uint32_t m = mag_bits<kType>(v.w[0]);
#pragma unroll
  for (int i = 1; i < (kType == 2 ? 8 : 4); ++i) m = max_bits<kType>(m, mag_bits<kType>(v.w[i]));
  if constexpr (kType != 2) m = max(m & 0xFFFFu, m >> 16);
  return m;
}

// The maximum over the 16 lanes of a row of lanes (lanes 16 i .. 16 i + 15), left in all of them.
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0xB1, 0xF, 0xF, false)));    // lane ^ 1
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x4E, 0xF, 0xF, false)));    // lane ^ 2
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x141, 0xF, 0xF, false)));   // mirror of 8
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x140, 0xF, 0xF, false)));   // mirror of 16
  return m;
}

template <int kType>
__device__ __forceinline__ float most_value(uint32_t bits) {
  const float m = value_of<kType>(bits);
  return m < kTiny ? kTiny : m;   // a NaN stays
}

// The quotient x M / most as an fp32 value that rounds to 8 bits as the exact quotient does.
//
// 16-bit inputs: with m = most 2^-e in [1, 2) and c = M 2^-e, x c is exact (8 or 11 bits times 3), and one
// correction of (x c) (1 / m) by its exact remainder gives a quotient that is exact where the true one is
// representable, else within one unit of fp32's last place. A tie between two codes has at most 5 bits, so it is
// hit exactly, and a quotient that is no tie is at least 2^-17 of its value away from one, so it never becomes
// one. fp32 inputs: the quotient in 64 bits is off by 2^-52 of its value at most and no tie is nearer than 2^-30
// unless it is hit; rounded to fp32 to odd (the last bit set where anything was dropped), it keeps the side of
// the tie that it lies on.
template <int kType, int kFmt>
struct Coder {
  float c, m, r;
  double big;
  __device__ __forceinline__ void set(float most) {
    if constexpr (kType == 2) {
      big = static_cast<double>(kMost[kFmt]) / static_cast<double>(most);
    } else {
      const bool finite = most < __builtin_huge_valf();
      const int e = finite ? static_cast<int>(__builtin_bit_cast(uint32_t, most) >> 23) - 127 : 0;
      const float down = __builtin_bit_cast(float, static_cast<uint32_t>(127 - e) << 23);   // 2^-e, e in [-100, 127]
      // e = 127 would need the subnormal 2^-127: halve twice instead
      m = finite ? (e == 127 ? most * 0x1p-126f * 0.5f : most * down) : 1.0f;
      c = finite ? (e == 127 ? kMost[kFmt] * 0x1p-126f * 0.5f : kMost[kFmt] * down) : 1.0f;
      r = finite ? 1.0f / m : (most != most ? most : 0.0f);
    }
  }
  __device__ __forceinline__ float quotient(float x) const {
    if constexpr (kType == 2) {
      const double q = static_cast<double>(x) * big;
      const float f = static_cast<float>(q);
      const double d = q - static_cast<double>(f);
      uint32_t b = __builtin_bit_cast(uint32_t, f);
      if (__builtin_fabs(d) > __builtin_fabs(q) * 0x1p-45 && !(b & 1)) b += (d > 0) == (q > 0) ? 1u : ~0u;
      return __builtin_bit_cast(float, b);
    } else {
      const float n = x * c;
      const float q = n * r;
      return __builtin_fmaf(__builtin_fmaf(-q, m, n), r, q);
    }
  }
};

template <int kFmt>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = 0;
  if constexpr (kFmt == 0) {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  }
  return static_cast<uint32_t>(w);
}

template <int kType, int kFmt>
__device__ __forceinline__ uint2 code_eight(const Eight<kType>& v, const Coder<kType, kFmt>& k) {
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = k.quotient(v.value(e));
  return make_uint2(pack4<kFmt>(q[0], q[1], q[2], q[3]), pack4<kFmt>(q[4], q[5], q[6], q[7]));
}

// Eight neighbouring codes, of which the first n stand for values that exist: the others are written as codes of 0, also where
// the group's NaN made NaN of them. kRagged: the matrix ends inside a group (where none does, leaving this out saves the
// row kernel 1 us of 34.5 at 8192 x 8192 bf16).
template <bool kRagged>
__device__ __forceinline__ uint2 kept(uint2 w, int n) {
  if (!kRagged || n >= 8) return w;
  const uint64_t m = n <= 0 ? 0 : (uint64_t{1} << (8 * n)) - 1;
  return make_uint2(w.x & static_cast<uint32_t>(m), w.y & static_cast<uint32_t>(m >> 32));
}

// Groups of 1 x 128, one direction: 16 lanes a group, a workgroup takes 16 rows x kSpan consecutive groups and
// has all its loads in flight at once. One row of 4096 takes 3.7 us, a launch's own time; bf16 8190 x 8192 39 us from memory, 5.2
// TB/s (a plain copy of as many bytes 36).
constexpr int kSpan = 4;

template <int kType, int kFmt, bool kRagged>
__global__ __launch_bounds__(256) void quant_rows_kernel(const typename In<kType>::T* __restrict__ x, int64_t rows,
                                                         int64_t cols, int64_t ld,
                                                         uint8_t* __restrict__ codes, int64_t ldc,
                                                         float* __restrict__ scale) {
  const int64_t groups = (cols + kGroup - 1) / kGroup;
  const unsigned spans = static_cast<unsigned>((groups + kSpan - 1) / kSpan);   // consecutive workgroups walk a row
  const int64_t row = static_cast<int64_t>(blockIdx.x / spans) * 16 + (threadIdx.x >> 4);
  const int64_t g0 = static_cast<int64_t>(blockIdx.x % spans) * kSpan;
  const int lane16 = threadIdx.x & 15;
  const int left = static_cast<int>(cols - g0 * kGroup) - 8 * lane16;   // values from this lane's first to the row's end
  if (row >= rows) return;   // whole rows of 16 lanes: the lane exchanges below stay inside one
  Eight<kType> v[kSpan];
#pragma unroll
  for (int s = 0; s < kSpan; ++s)
    if (g0 + s < groups) v[s] = load_eight<kType>(x + row * ld, (g0 + s) * kGroup + 8 * lane16, cols);
#pragma unroll
  for (int s = 0; s < kSpan; ++s) {
    if (g0 + s >= groups) break;
    const float most = most_value<kType>(max16(most_of<kType>(v[s])));
    Coder<kType, kFmt> k;
    k.set(most);
    *reinterpret_cast<uint2*>(codes + row * ldc + (g0 + s) * kGroup + 8 * lane16) = kept<kRagged>(code_eight<kType, kFmt>(v[s], k), left - kGroup * s);
    if (lane16 == 0) scale[(g0 + s) * rows + row] = most / kMost[kFmt];
  }
}

// A 128 x 128 tile per workgroup of 256 threads: thread t holds rows 8 (t / 16) .. + 7, columns 8 (t mod 16) .. + 7.
// kBlock 1: the row groups' codes and, with kBoth, the column groups' of the transpose; kBlock 128: one scale for
// the tile, its codes straight and (kBoth) turned. The turned bytes go through LDS, eight of a column at a time. bf16 8190 x 8192,
// rows, both ways: 57 us, 4.8 TB/s read and written, where the caches hold a part of x, 65 where they do not (a plain copy of as
// many bytes 46); fp32 4100 x 6148, blocks, both ways: 31 and 36 us (28).
constexpr int kTurn = 144;   // bytes of a turned row in LDS: 128 and a 16-byte pad

template <int kType, int kFmt, int kBlock, bool kBoth, bool kRagged>
__global__ __launch_bounds__(256) void quant_tile_kernel(const typename In<kType>::T* __restrict__ x, int64_t rows,
                                                         int64_t cols, int64_t ld,
                                                         uint8_t* __restrict__ codes, int64_t ldc,
                                                         float* __restrict__ scale, uint8_t* __restrict__ codes_t,
                                                         int64_t ldt, float* __restrict__ scale_t) {
  __shared__ __attribute__((aligned(16))) uint8_t turn[kBoth ? kGroup * kTurn : 16];
  __shared__ __attribute__((aligned(16))) uint32_t part[4][kGroup];
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kGroup, c0 = static_cast<int64_t>(blockIdx.x) * kGroup;
  const int64_t col_groups = (cols + kGroup - 1) / kGroup, row_groups = (rows + kGroup - 1) / kGroup;
  Eight<kType> v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = r0 + 8 * rg + i;
    if (row < rows) {
      v[i] = load_eight<kType>(x + row * ld, c0 + 8 * cg, cols);
    } else {
#pragma unroll
      for (int e = 0; e < (kType == 2 ? 8 : 4); ++e) v[i].w[e] = 0;
    }
  }

  const int in_cols = static_cast<int>(cols - c0) - 8 * cg, in_rows = static_cast<int>(rows - r0) - 8 * rg;
  uint2 turned[8];   // the codes of this thread's columns, eight rows each
  if constexpr (kBlock == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = r0 + 8 * rg + i;
      const float most = most_value<kType>(max16(most_of<kType>(v[i])));
      Coder<kType, kFmt> k;
      k.set(most);
      const uint2 w = kept<kRagged>(code_eight<kType, kFmt>(v[i], k), in_cols);
      if (row < rows) {
        *reinterpret_cast<uint2*>(codes + row * ldc + c0 + 8 * cg) = w;
        if (cg == 0) scale[blockIdx.x * rows + row] = most / kMost[kFmt];
      }
    }
    if constexpr (kBoth) {
      constexpr int kWords = kType == 2 ? 8 : 4;
      uint32_t cm[kWords];
#pragma unroll
      for (int e = 0; e < kWords; ++e) {
        cm[e] = mag_bits<kType>(v[0].w[e]);
#pragma unroll
        for (int i = 1; i < 8; ++i) cm[e] = max_bits<kType>(cm[e], mag_bits<kType>(v[i].w[e]));
        cm[e] = max_bits<kType>(cm[e], static_cast<uint32_t>(__shfl_xor(static_cast<int>(cm[e]), 16)));
        cm[e] = max_bits<kType>(cm[e], static_cast<uint32_t>(__shfl_xor(static_cast<int>(cm[e]), 32)));
      }
      if ((t & 63) < 16) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          part[wave][8 * cg + e] = kType == 2 ? cm[e] : (e & 1) ? cm[e >> 1] >> 16 : cm[e >> 1] & 0xFFFFu;
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int col = 8 * cg + e;
        const float most = most_value<kType>(max(max(part[0][col], part[1][col]), max(part[2][col], part[3][col])));
        Coder<kType, kFmt> k;
        k.set(most);
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = k.quotient(v[i].value(e));
        turned[e] = kept<kRagged>(make_uint2(pack4<kFmt>(q[0], q[1], q[2], q[3]), pack4<kFmt>(q[4], q[5], q[6], q[7])), in_rows);
        if (rg == 0 && c0 + col < cols) scale_t[blockIdx.y * cols + c0 + col] = most / kMost[kFmt];
      }
    }
  } else {
    uint32_t m = most_of<kType>(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = max(m, most_of<kType>(v[i]));
    m = max16(m);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
    if ((t & 63) == 0) part[0][wave] = m;
    __syncthreads();
    const float most = most_value<kType>(max(max(part[0][0], part[0][1]), max(part[0][2], part[0][3])));
    Coder<kType, kFmt> k;
    k.set(most);
    uint2 w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t row = r0 + 8 * rg + i;
      w[i] = kept<kRagged>(code_eight<kType, kFmt>(v[i], k), in_cols);
      if (row < rows) *reinterpret_cast<uint2*>(codes + row * ldc + c0 + 8 * cg) = w[i];
    }
    if (t == 0) {
      scale[blockIdx.y * col_groups + blockIdx.x] = most / kMost[kFmt];
      if constexpr (kBoth) scale_t[blockIdx.x * row_groups + blockIdx.y] = most / kMost[kFmt];
    }
    if constexpr (kBoth) {   // byte e of the eight rows: 8 x 8 bytes turned with byte permutes
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t sel = 0x0c0c0000u | static_cast<uint32_t>(e) << 8 | static_cast<uint32_t>(e + 4);
          uint32_t lo[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const uint32_t a = h ? w[2 * p].y : w[2 * p].x, b = h ? w[2 * p + 1].y : w[2 * p + 1].x;
            lo[p] = __builtin_amdgcn_perm(a, b, sel);   // byte 0: a's byte e, byte 1: b's byte e
          }
          turned[4 * h + e] = kept<kRagged>(make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16), in_rows);
        }
    }
  }
  if constexpr (kBoth) {
    // column 8 cg + e at kTurn bytes each; 16-byte chunk rg / 2 stored at chunk (rg / 2) XOR (cg / 2)
#pragma unroll
    for (int e = 0; e < 8; ++e)
      *reinterpret_cast<uint2*>(turn + (8 * cg + e) * kTurn + (((rg >> 1) ^ (cg >> 1)) << 4) + (rg & 1) * 8) = turned[e];
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int col = it * 32 + (t >> 3), chunk = t & 7;
      if (c0 + col < cols)
        *reinterpret_cast<uint4*>(codes_t + (c0 + col) * ldt + r0 + 16 * chunk) =
            *reinterpret_cast<const uint4*>(turn + col * kTurn + ((chunk ^ (col >> 4)) << 4));
    }
  }
}

template <int kType, int kFmt, bool kRagged>
hipError_t launch_typed(const Quant8Launch& a, hipStream_t s) {
  typedef typename In<kType>::T T;
  const T* x = static_cast<const T*>(a.x);
  const unsigned cg = static_cast<unsigned>((a.cols + kGroup - 1) / kGroup), rg = static_cast<unsigned>((a.rows + kGroup - 1) / kGroup);
  const bool both = a.codes_t != nullptr;
  if (a.block == 1 && !both) {
    // 2^24 workgroups, a launch's most, are 412 GB of values and codes
    const dim3 grid((cg + kSpan - 1) / kSpan * static_cast<unsigned>((a.rows + 15) / 16));
    hipLaunchKernelGGL((quant_rows_kernel<kType, kFmt, kRagged>), grid, dim3(256), 0, s, x, a.rows, a.cols, a.ld, a.codes, a.ldc, a.scale);
  } else if (a.block == 1) {
    hipLaunchKernelGGL((quant_tile_kernel<kType, kFmt, 1, true, kRagged>), dim3(cg, rg), dim3(256), 0, s, x, a.rows, a.cols, a.ld,
                       a.codes, a.ldc, a.scale, a.codes_t, a.ldt, a.scale_t);
  } else if (both) {
    hipLaunchKernelGGL((quant_tile_kernel<kType, kFmt, 128, true, kRagged>), dim3(cg, rg), dim3(256), 0, s, x, a.rows, a.cols, a.ld,
                       a.codes, a.ldc, a.scale, a.codes_t, a.ldt, a.scale_t);
  } else {
    hipLaunchKernelGGL((quant_tile_kernel<kType, kFmt, 128, false, kRagged>), dim3(cg, rg), dim3(256), 0, s, x, a.rows, a.cols, a.ld,
                       a.codes, a.ldc, a.scale, a.codes_t, a.ldt, a.scale_t);
  }
  return hipGetLastError();
}

template <int kType, int kFmt>
hipError_t launch_format(const Quant8Launch& a, hipStream_t s) {
  const bool ragged = a.cols % kGroup != 0 || (a.codes_t != nullptr && a.rows % kGroup != 0);
  return ragged ? launch_typed<kType, kFmt, true>(a, s) : launch_typed<kType, kFmt, false>(a, s);
}

}  // namespace

hipError_t launch_quant8(int dtype, int fmt, const Quant8Launch& a, hipStream_t s) {
  switch (dtype * 2 + fmt) {
    case 0: return launch_format<0, 0>(a, s);
    case 1: return launch_format<0, 1>(a, s);
    case 2: return launch_format<1, 0>(a, s);
    case 3: return launch_format<1, 1>(a, s);
    case 4: return launch_format<2, 0>(a, s);
    case 5: return launch_format<2, 1>(a, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace tbl
