// The 256 x 256 tile loop of products A B^T whose operands both keep k contiguous (the 8-bit GEMM and the
// orthogonalisation's fp16 products): 128 bytes of every row a step, 128 eight-bit or 64 sixteen-bit values.
//
// Eight waves, two per SIMD, in two groups: group 0 owns rows 0-127, group 1 rows 128-255; wave wn of a group the columns 64 wn .. + 63
// (8 x 4 blocks of 16 x 16). A step has two halves for each group: the first takes all of the wave's B and its
// first four row blocks of A into registers and multiplies them, the second its last four row blocks. Each half is a memory
// half-period (LDS reads into registers, direct loads issued) and a compute one (the matrix instructions), closed by
// barriers; group 1 runs one half-period behind, so on every SIMD one wave computes while the other fetches.
//
// LDS holds two stages of 64 KiB. B and the first row blocks of a stage are free as soon as both groups' first halves
// have read them, so their next loads go out one half earlier than the last row blocks': every load
// has six half-periods (one and a half steps) to land. Row r's 16-byte chunk c lies at chunk c XOR (r / 2 mod 8): 16
// rows read at one chunk touch all 64 banks.
#pragma once

#include "gemm_kernel.hpp"

namespace tbl {
namespace {

constexpr int kNtRow = 128;                 // bytes of a row in a step
constexpr int kNtThreads = 512;
constexpr int kNtStage = 2 * 256 * kNtRow;  // A then B
constexpr int kNtOut = 0x7FFFFFF0;          // an offset past every range

// Waits until at most N of this wave's vector-memory operations are in flight.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A lane's 32 bytes of a row: chunks q and q + 4 for lane group q = lane / 16. Which k a byte stands for does not matter as
// long as both operands agree.
struct Chunks {
  uint4 lo, hi;
};

// An operand's rows of a tile, a step at a time: the buffer descriptor of the step that is loaded next. It is moved on with
// a few scalar instructions inside a compute half-period; built anew in the memory ones, whose length counts, it cost
// 60 instructions there and a third of the loop's time.
struct NtOperand {
  uint64_t at;
  unsigned left;    // bytes from ``at`` to the end of the tile's last row
  i32x4_t desc;
  __device__ __forceinline__ void start(const void* p, int64_t bytes) {
    at = reinterpret_cast<uint64_t>(p);
    left = static_cast<unsigned>(bytes);
  }
  // real: the step exists; loads of one past the end are of zero length
  __device__ __forceinline__ void set(bool real) {
    desc = make_desc(reinterpret_cast<const void*>(at), real ? left : 0u);
    at += kNtRow;
    left -= kNtRow;
  }
};

// 16 bytes per lane from desc + voffset to LDS address base + kOffset.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
template <int kOffset>
__device__ __forceinline__ void load_to_lds_at(i32x4_t desc, unsigned base, int voffset) {
  asm volatile("s_add_u32 m0, %0, %3\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(base), "v"(voffset), "s"(desc), "n"(kOffset) : "memory", "m0", "scc");
}
#pragma clang diagnostic pop

// 4 bytes per lane from desc + voffset into LDS: lane l writes lds_addr + 4 l.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load4_to_lds(i32x4_t desc, unsigned lds_addr, int voffset) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :: "s"(__builtin_amdgcn_readfirstlane(lds_addr)), "v"(voffset), "s"(desc) : "memory", "m0");
}
#pragma clang diagnostic pop

// This wave's direct loads and LDS reads of a tile. lda, ldb in bytes.
struct NtTile {
  int lane, wave, wm, wn;
  int va[4], vb[4];
  unsigned to_a, to_b;        // LDS addresses of the next loads' rows
  const char *a_lo, *a_hi, *b_lo, *b_hi;   // this lane's chunks of the wave's first rows in the stage read next
  char* lds;

  // kept: bytes of every row that exist in the step (128 but for a step of its own at the end); later chunks read as zero
  __device__ __forceinline__ void rows(int64_t lda, int64_t ldb, int kept) {
    // instruction j of A: rows a_row(j) + lane / 8; of B: rows 32 wave + 8 j + lane / 8
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int ra = (wave >> 2) * 128 + (wave & 3) * 16 + (j & 1) * 8 + (j >> 1) * 64 + (lane >> 3), rb = 32 * wave + 8 * j + (lane >> 3);
      const int ca = (((lane & 7) ^ (ra >> 1)) & 7) * 16, cb = (((lane & 7) ^ (rb >> 1)) & 7) * 16;
      va[j] = ca < kept ? ra * static_cast<int>(lda) + ca : kNtOut;
      vb[j] = cb < kept ? rb * static_cast<int>(ldb) + cb : kNtOut;
    }
  }
  __device__ __forceinline__ void init(char* memory, int64_t lda, int64_t ldb) {
    lds = memory;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave >> 2;
    wn = wave & 3;
    rows(lda, ldb, kNtRow);
    stage(0, 0);
  }
  // The stages that the next loads fill and the next reads take.
  __device__ __forceinline__ void stage(int load, int read) {
    to_a = lds_address(lds) + load * kNtStage + ((wave >> 2) * 128 + (wave & 3) * 16) * kNtRow;
    to_b = lds_address(lds) + load * kNtStage + (256 + 32 * wave) * kNtRow;
    const int r = lane & 15, q = lane >> 4;
    const int swz = ((q ^ (r >> 1)) & 7) * 16;
    a_lo = lds + read * kNtStage + (wm * 128 + r) * kNtRow + swz;
    a_hi = lds + read * kNtStage + (wm * 128 + r) * kNtRow + (swz ^ 64);
    b_lo = a_lo + (256 + wn * 64 - wm * 128) * kNtRow;
    b_hi = a_hi + (256 + wn * 64 - wm * 128) * kNtRow;
  }
  // A's instruction j: 0, 1 the first four row blocks of either group, 2, 3 the last four
  template <int j>
  __device__ __forceinline__ void load_a(const NtOperand& a) const { load_to_lds_at<((j & 1) * 8 + (j >> 1) * 64) * kNtRow>(a.desc, to_a, va[j]); }
  template <int j>
  __device__ __forceinline__ void load_b(const NtOperand& b) const { load_to_lds_at<8 * j * kNtRow>(b.desc, to_b, vb[j]); }
  __device__ __forceinline__ Chunks a(int i) const {
    return Chunks{*reinterpret_cast<const uint4*>(a_lo + i * 16 * kNtRow), *reinterpret_cast<const uint4*>(a_hi + i * 16 * kNtRow)};
  }
  __device__ __forceinline__ Chunks b(int j) const {
    return Chunks{*reinterpret_cast<const uint4*>(b_lo + j * 16 * kNtRow), *reinterpret_cast<const uint4*>(b_hi + j * 16 * kNtRow)};
  }
};

// The loop over ``steps`` steps. memory0(s) reads the first half's operands of step s and issues the kLast loads of the last row
// blocks of step s + 1 (A's instructions 2 and 3); memory1(s) reads the last row blocks of step s and issues the kFirst
// loads of step s + 2's first half (B, A's 0 and 1, and what the user adds). Past the end loads are of zero length, so the
// counts hold. compute0(s) also moves the descriptors on to step s + 2. start() has issued step 0's loads
// and step 1's first, in this order: first half of 0, last rows of 0, first half of 1.
template <int kFirst, int kLast, class Memory0, class Memory1, class Compute0, class Compute1>
__device__ __forceinline__ void nt_loop(int group, int steps, Memory0 memory0, Memory1 memory1, Compute0 compute0, Compute1 compute1) {
  auto close = []() {
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  wait_loads<kFirst + kLast>();   // the first half's operands of step 0 have landed
  lds_barrier();
  if (group == 1) lds_barrier();  // one half-period behind
  __builtin_amdgcn_sched_barrier(0);
  for (int s = 0; s < steps; ++s) {
    memory0(s);
    wait_loads<kFirst + kLast>();   // step s's last row blocks
    close();
    compute0(s);
    close();
    memory1(s);
    wait_loads<kFirst + kLast>();   // step s + 1's first half
    close();
    compute1(s);
    close();
  }
  if (group == 0) lds_barrier();  // group 1's extra one
  wait_loads<0>();                // no direct load may still be writing this workgroup's LDS
}

// ---- a wave's results as whole rows ----------------------------------------------------------------

// A wave's tile in LDS: 128 bytes a row, 16-byte chunk c of row m at c XOR (m / 2 mod 8).
__device__ __forceinline__ char* tile_chunk(char* tile, int m, int chunk) { return tile + m * 128 + (((chunk ^ (m >> 1)) & 7) << 4); }
__device__ __forceinline__ uint2* tile_four(char* tile, int m, int n) { return reinterpret_cast<uint2*>(tile_chunk(tile, m, n >> 3) + (n & 7) * 2); }
// Between a wave's writes to its tile and its reads in another layout; its LDS operations execute in order.
__device__ __forceinline__ void tile_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}
// The tile's rows to rows m0 .. of ``to`` (rows of ld), columns n0 .. + 63; ``rows`` and ``cols`` of them exist.
template <int TM>
__device__ __forceinline__ void tile_store(char* tile, uint16_t* to, int64_t ld, int rows, int64_t cols, int m0, int n0, int lane) {
  const int n = n0 + 8 * (lane & 7);
#pragma unroll
  for (int k = 0; k < 2 * TM; ++k) {
    const int row = 8 * k + (lane >> 3), m = m0 + row;
    if (m >= rows || n >= cols) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(tile_chunk(tile, row, lane & 7));
    uint16_t* d = to + static_cast<int64_t>(m) * ld + n;
    if (n + 8 <= cols) {
      __builtin_memcpy(d, &v, 16);   // rows of any even length: one 16-byte store, aligned or not
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < cols) d[e] = static_cast<uint16_t>(e & 1 ? w[e >> 1] >> 16 : w[e >> 1]);
    }
  }
}

// ---- 128 x 128 tiles -------------------------------------------------------------------------------
//
// Eight waves of 32 x 64 (2 x 4 blocks); the same 128-byte rows and swizzle in four stages. A wave's operands of step s + 1 are
// read while it multiplies step s: a column block of B into the registers that its last product has just freed, A into
// a second set. Loads go out four steps ahead of their use, two of A and two of B a wave and step. A step takes 0.41 to 0.45 us
// with f16 operands. (Four waves of 64 x 64 read a third less from LDS, but with one wave a SIMD the compiler keeps the sums in
// accumulation registers, where adding scaled products costs a move each way.)

constexpr int kNt128Stage = 2 * 128 * kNtRow;
constexpr int kNt128Stages = 4;

struct Nt128 {
  int lane, wave, wm, wn;     // rows 32 wm .. + 31, columns 64 wn .. + 63
  int va[2], vb[2];
  unsigned to;                // LDS address of this wave's rows of A in the stage loaded next (B's 16 KiB further)
  int at, at_hi, b_at, b_hi;  // this lane's chunks of the wave's first rows of A and B within a stage
  const char* from;           // the stage read next
  char* lds;

  __device__ __forceinline__ void init(char* memory, int64_t lda, int64_t ldb) {
    lds = memory;
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    wm = wave >> 1;
    wn = wave & 1;
    rows(lda, ldb, kNtRow);
    load_stage(0);
    read_stage(0);
    const int r = lane & 15, q = lane >> 4, swz = ((q ^ (r >> 1)) & 7) * 16;
    at = (wm * 32 + r) * kNtRow + swz;
    at_hi = (wm * 32 + r) * kNtRow + (swz ^ 64);
    b_at = (128 + wn * 64 + r) * kNtRow + swz;
    b_hi = (128 + wn * 64 + r) * kNtRow + (swz ^ 64);
  }
  // kept: bytes of every row that exist in the steps loaded next; later chunks read as zero
  __device__ __forceinline__ void rows(int64_t lda, int64_t ldb, int kept) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = 16 * wave + 8 * j + (lane >> 3), c = (((lane & 7) ^ (row >> 1)) & 7) * 16;
      va[j] = c < kept ? row * static_cast<int>(lda) + c : kNtOut;
      vb[j] = c < kept ? row * static_cast<int>(ldb) + c : kNtOut;
    }
  }
  __device__ __forceinline__ void load_stage(int stage) { to = lds_address(lds) + stage * kNt128Stage + 16 * wave * kNtRow; }
  __device__ __forceinline__ void read_stage(int stage) { from = lds + stage * kNt128Stage; }
  template <int j>
  __device__ __forceinline__ void load_a(const NtOperand& a) const { load_to_lds_at<8 * j * kNtRow>(a.desc, to, va[j]); }
  template <int j>
  __device__ __forceinline__ void load_b(const NtOperand& b) const { load_to_lds_at<(128 + 8 * j) * kNtRow>(b.desc, to, vb[j]); }
  __device__ __forceinline__ Chunks a(int i) const {
    return Chunks{*reinterpret_cast<const uint4*>(from + at + i * 16 * kNtRow), *reinterpret_cast<const uint4*>(from + at_hi + i * 16 * kNtRow)};
  }
  __device__ __forceinline__ Chunks b(int j) const {
    return Chunks{*reinterpret_cast<const uint4*>(from + b_at + j * 16 * kNtRow), *reinterpret_cast<const uint4*>(from + b_hi + j * 16 * kNtRow)};
  }
};

// ---- how tiles are dealt to the compute units -------------------------------------------------------
//
// One workgroup fills a CU, so T tiles take ceil(T / 256) rounds. The tiles of a last, partial round are split along k
// into as many parts as idle CUs allow (parts of at least kMinPart steps), whose sums are joined in order by a second kernel.

constexpr int kCus = 256;
constexpr int kMinPart = 4;

struct Deal {
  int tiles;     // in all
  int whole;     // computed by one workgroup each; the others by ``parts``
  int parts;
  int steps;
  int size;      // of a tile: 128 or 256
  int blocks() const { return whole + (tiles - whole) * parts; }
  int64_t floats() const { return parts > 1 ? static_cast<int64_t>(tiles - whole) * parts * size * size : 0; }
};

inline Deal make_deal(int64_t tiles, int steps, int size, int slots = kCus) {   // slots: workgroups of a round
  Deal d{static_cast<int>(tiles), static_cast<int>(tiles), 1, steps, size};
  const int rest = static_cast<int>(tiles % slots);
  if (rest == 0) return d;
  int parts = slots / rest;
  if (parts > steps / kMinPart) parts = steps / kMinPart;
  if (parts > 16) parts = 16;
  if (parts < 2) return d;
  d.parts = parts;
  d.whole = static_cast<int>(tiles) - rest;
  return d;
}

// What a workgroup does: a tile's steps s0 .. s1 - 1, and where its sums go (unit < 0: the tile is whole).
struct Share {
  int tile, s0, s1, unit;
};
__device__ __forceinline__ Share share_of(const Deal& d, int block) {
  if (block < d.whole) return Share{block, 0, d.steps, -1};
  const int u = block - d.whole, part = u % d.parts;
  return Share{d.whole + u / d.parts, static_cast<int>(static_cast<int64_t>(d.steps) * part / d.parts),
               static_cast<int>(static_cast<int64_t>(d.steps) * (part + 1) / d.parts), u};
}

// A unit's sums: [row block of a wave][wave][column block][lane] of four floats, so writing and joining are whole lines.
// A 256 tile's waves have eight row blocks, a 128 tile's two.
__device__ __forceinline__ float4* part_at(const Deal& d, float* work, int unit, int i, int wave, int j, int lane) {
  return reinterpret_cast<float4*>(work + static_cast<int64_t>(unit) * d.size * d.size) + ((i * 8 + wave) * 4 + j) * 64 + lane;
}
// rows: how many of the wave's rows exist; blocks past them are neither written nor joined.
template <int TM>
__device__ __forceinline__ void write_part(const Deal& d, float* work, int unit, int wave, int lane, int rows, f32x4_t (&acc)[TM][4]) {
#pragma unroll
  for (int i = 0; i < TM; ++i)
    if (16 * i < rows) {
#pragma unroll
      for (int j = 0; j < 4; ++j) *part_at(d, work, unit, i, wave, j, lane) = make_float4(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]);
    }
}
// The sum of a split tile's parts, for row block i.
__device__ __forceinline__ void join_parts(const Deal& d, float* work, int tile, int i, int wave, int lane, f32x4_t (&acc)[1][4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[0][j] = f32x4_t{0, 0, 0, 0};
  const int first = (tile - d.whole) * d.parts;
  for (int p = 0; p < d.parts; ++p)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = *part_at(d, work, first + p, i, wave, j, lane);
      acc[0][j] += f32x4_t{v.x, v.y, v.z, v.w};
    }
}

}  // namespace
}  // namespace tbl
