// The paged key/value cache: layout, converts and the launch interface shared
// by the kernels that write, read and attend over it.
//
// A token's key row and value row of one head are MX blocks: 32 consecutive
// elements share a power of two 2^X (byte X + 127) and are codes of E2M1
// (4 bits) or E4M3 (8 bits).  One byte buffer holds it all:
//
//   page p, head h, tile t of the page (16 tokens):
//     base = ((p * heads + h) * page / 16 + t) * kTile
//     key codes [16 R] | value codes [16 R] | key scales [nb][16] | value scales [nb][16]
//
// with R = dim * bits / 8 the bytes of a row and nb = dim / 32.  A head's
// page is one contiguous run, a tile is what one wave reads with one load per
// 16 bytes of row, and the orders inside a tile are those of the matrix
// instructions, so attention moves codes from memory to operands without a
// shuffle.  A row's bytes are cut into segments of 64, 32 and 16 bytes (w):
//
//   keys:   [segment][piece g = 0..3][token 0..15][w / 4 bytes]
//           a lane (token, g) reads w / 4 contiguous bytes of its own token:
//           the k index of the operand that has keys as its rows
//   values: [segment][quad of tokens 0..3][c = 0..15][token of the quad][w / 16 bytes]
//           a lane (quad, c) reads four tokens of the same few elements: the
//           k index of the product with the weights runs over tokens
//
// No byte is shared by two tokens, so tokens are written independently.
#pragma once

#include "nc_device.h"

namespace nc {

constexpr int kKvTokens = 16;   // tokens of a tile

template <int FMT, int D> struct Kv {
  static constexpr int BITS = FMT == NC_E2M1 ? 4 : 8;
  static constexpr int DPB = 8 / BITS;              // elements of a byte
  static constexpr int R = D * BITS / 8;            // bytes of a row
  static constexpr int NB = D / 32;                 // blocks of a row
  static constexpr int TILE = 32 * (R + NB);        // bytes of a tile
  static constexpr int KC = 0, VC = 16 * R, KS = 32 * R, VS = 32 * R + 16 * NB;
  static constexpr int N4 = R / 64, N2 = (R % 64) / 32, N1 = (R % 32) / 16;
  static constexpr int NSEG = N4 + N2 + N1;
  static constexpr int DW = R / 16;                 // dwords of codes per lane and tile (keys, and values)
  static constexpr int w(int s) { return s < N4 ? 64 : (s < N4 + N2 ? 32 : 16); }
  static constexpr int off(int s) { return s <= N4 ? 64 * s : (s <= N4 + N2 ? 64 * N4 + 32 * (s - N4) : R); }
  static constexpr int dim0(int s) { return off(s) * DPB; }
  static constexpr int piece(int s) { return w(s) / 4 * DPB; }   // elements of a key piece
  static constexpr int lane(int s) { return w(s) / 16 * DPB; }   // elements of a value lane and token
};

// Bytes of a tile for run-time sizes (host).
inline int64_t kv_tile_bytes(int fmt, int dim) { return 32 * (int64_t)(dim * (fmt == NC_E2M1 ? 4 : 8) / 8 + dim / 32); }

// gfx950's scaled converts, codes -> two bf16 (exact: a code has at most four
// significant bits; below bf16's range the result is rounded to nearest even).
// scale: 2^X as a float whose exponent field is the scale byte (0 stands for
// 2^-127, 255 gives NaN: measured for every code and scale byte).
__device__ __forceinline__ float kv_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Codes 2i, 2i + 1 of a dword (E2M1: byte i; E4M3: half i) -> packed bf16.
template <int FMT>
__device__ __forceinline__ uint32_t kv_pair(uint32_t codes, float scale, int i) {
  bf16x2_t r;
  if constexpr (FMT == NC_E2M1) {
    switch (i) {
      case 0: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0); break;
      case 1: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1); break;
      case 2: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2); break;
      default: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3); break;
    }
  } else {
    if (i == 0) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false);
    else r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true);
  }
  return __builtin_bit_cast(uint32_t, r);
}

// Division by a number known to the host, of n < 2^31: with 2^s the power of two
// not below d and m = floor(2^32 (2^s - d) / d) + 1, n / d = (n + mulhi(n, m)) >> s
// (T. Granlund, P. L. Montgomery, "Division by Invariant Integers using
// Multiplication", PLDI 1994, section 4; the sum does not overflow here).
// Three instructions where the compiler's division takes some thirty: single-token
// calls, whose code is fetched anew by every call, spend their time on such things.
struct KvDiv {
  uint32_t d, m, s;
  __device__ __forceinline__ uint32_t quot(uint32_t n) const { return (n + __umulhi(n, m)) >> s; }
  __device__ __forceinline__ uint32_t quot(uint32_t n, uint32_t& rest) const {
    const uint32_t q = quot(n);
    rest = n - q * d;
    return q;
  }
};
inline KvDiv kv_div(uint32_t d) {
  uint32_t s = 0;
  while (s < 31 && ((uint32_t)1 << s) < d) ++s;
  return KvDiv{d, (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << s) - d)) / d + 1), s};
}

// What a cache and a view of rows are to the kernels.
struct KvCache {
  uint8_t* data;
  int64_t slots;        // pages * page
  int32_t page;         // tokens of a page, a multiple of 16
  int32_t heads;
  KvDiv by_tiles;       // tiles of a page
  KvDiv by_heads;
};
template <typename P> struct KvRows {   // element (token, head, i) at p[token * ts + head * hs + i]
  P p;
  int64_t ts, hs;
};

// One attention call (kernel argument).
struct KvAttn {
  KvCache cache;
  KvRows<const void*> q;
  KvRows<void*> out;
  float* lse;              // [total_q][lse_ts], nullable
  int64_t lse_ts;
  const int32_t* q_start;  // [batch + 1]
  const int32_t* kv_len;   // [batch]
  const int32_t* table;    // [batch][table_w] page numbers
  int32_t table_w, batch, total_q, max_q, max_kv;
  int32_t group;           // query heads of a cache head
  KvDiv by_group;
  int32_t causal, window;  // window 0: none
  float scale2;            // score scale times log2(e)
  // the split: row groups of one sequence and cache head (of a sequence with max_q queries: others have as
  // many, the last ones empty), a workgroup for each or, in the few-row kernel with shares > 0, so many
  // workgroups with equal shares of all row groups' tiles
  int32_t row_groups, shares;
  KvDiv by_row_groups, by_segments;   // row groups; segments of a sequence, heads * row groups
  float* part;             // partial results of the shares
};

// What the split of a call is, from its sizes (host): shared by the workspace
// size and the launch.
struct KvPlan {
  int32_t rows;         // rows of a workgroup: 16 or 32 (few-row kernel), kKvManyRows
  int32_t row_groups;   // row groups of one (sequence, head)
  int32_t shares;       // few rows: equal shares of the tiles, 0 for a workgroup to a row group
};

constexpr int kKvFewWaves = 4;
constexpr int kKvShareLeast = 16;  // fewest tiles of a share
constexpr int kKvManyRows = 128;   // rows of a workgroup of the many-row kernel
// Most rows of a workgroup of the few-row kernel: 32 where groups of 32 gain.
// bf16 at 256 elements does not (16 sequences of 20000 tokens, 4 heads, 32 rows,
// E4M3: 160 us against 125 for groups of 16; 32 of 2000, 8 heads, 36 rows: 144
// against 85).  At 192 they win over short keys (5 x 5 heads, 600 rows over 200
// tokens, E2M1: 19 us against 30) and lose over long ones (16 of 5500, 32 rows:
// 44 against 34): their queries and sums do not fit 256 registers (74 spilled
// for E2M1, 107 for E4M3), and the spilled ones come back at every step.  No
// rule on the keys' length chooses between the two there.
constexpr int kv_few_rows(int dtype, int dim) { return dim <= (dtype == NC_BF16 ? 192 : 128) ? 32 : 16; }

// Waves of a SIMD that the few-row kernel is compiled for: queries and sums of
// nt row tiles, and about 110 registers more.  An estimate; where it is too low
// registers spill: 74 and 107 at bf16 192 with 32 rows, 24 at bf16 256 (E4M3, its
// single tokens too), 2 to 6 at fp32 192 and at fp32 96 with 32 rows.
constexpr int kv_few_waves(int dtype, int dim, int nt) {
  const int need = (dtype == NC_BF16 ? 1 : 3) * nt * dim / 8 + nt * dim / 4 + 110;
  return need <= 168 ? 3 : need <= 256 ? 2 : 1;
}
// Workgroups of it that the card holds at once: the shares that a call is cut into.
constexpr int kKvUnits = 256;      // compute units
constexpr int kv_few_slots(int dtype, int dim, int rows) {
  const int lds = kKvFewWaves * 16 * (dim + 4) * 4 + kKvFewWaves * rows * 8, fit = 160 * 1024 / lds;
  const int waves = kv_few_waves(dtype, dim, rows / 16);
  return kKvUnits * (waves < fit ? waves : fit);
}

// Rows (query i of the sequence, head j of the group) are numbered i * group + j.
// Partial results: two places for each share and row of a group, of D
// unnormalised sums, then a maximum and a sum for each place.
inline size_t kv_part_bytes(const KvPlan& p, int dim) { return (size_t)(2 * (int64_t)p.shares * p.rows) * (size_t)(dim + 2) * 4; }

hipError_t launch_kv_write(const KvCache& c, int fmt, int dim, const KvRows<const void*>& k, const KvRows<const void*>& v,
                           int dtype, const int64_t* slots, int64_t tokens, int rule, hipStream_t stream);
hipError_t launch_kv_read(const KvCache& c, int fmt, int dim, const KvRows<void*>& k, const KvRows<void*>& v, int dtype,
                          const int64_t* slots, int64_t tokens, hipStream_t stream);
hipError_t kv_few_e2m1_bf16(const KvAttn& a, int dim, const KvPlan& p, hipStream_t stream);
hipError_t kv_few_e2m1_f32(const KvAttn& a, int dim, const KvPlan& p, hipStream_t stream);
hipError_t kv_few_e4m3_bf16(const KvAttn& a, int dim, const KvPlan& p, hipStream_t stream);
hipError_t kv_few_e4m3_f32(const KvAttn& a, int dim, const KvPlan& p, hipStream_t stream);
hipError_t kv_many_e2m1_bf16(const KvAttn& a, int dim, hipStream_t stream);
hipError_t kv_many_e2m1_f32(const KvAttn& a, int dim, hipStream_t stream);
hipError_t kv_many_e4m3_bf16(const KvAttn& a, int dim, hipStream_t stream);
hipError_t kv_many_e4m3_f32(const KvAttn& a, int dim, hipStream_t stream);
hipError_t launch_kv_join(const KvAttn& a, int dim, int dtype, const KvPlan& p, hipStream_t stream);

}  // namespace nc
