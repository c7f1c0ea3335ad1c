// Matrices of MX blocks: layout, converts and the launch interface shared by the
// kernels that write, read and multiply them and by the activations that keep
// their inputs in one.
//
// A matrix [rows, cols] is laid out for the scaled matrix instructions, whose
// operand of 32 rows and 64 columns is 32 consecutive elements a lane.  Rows go
// in strips of 32, columns in chunks of 256 (four steps of 64), both filled up
// with zeros:
//
//   codes  [strip][chunk][step 0..3] of 32 x 64 elements:
//            E2M1          [lane][16 bytes]          lane r + 32 g holds columns 32 g .. 32 g + 31 of row r
//            E4M3, E5M2    [half h][lane][16 bytes]  lane r + 32 g holds columns 32 h + 16 g .. + 15
//   scales [strip][chunk][lane][step]                lane r + 32 b: the scale byte of block b of the step
//
// which are the instruction's own orders (found by one product of random codes
// under each candidate order): a wave takes an operand with one load of 16 bytes
// a lane, from memory or LDS alike, in one run of 1 KiB, and a lane its scales of
// a chunk with one dword.
#pragma once

#include "nc_device.h"

namespace nc {

constexpr int kMxRows = 32, kMxChunk = 256, kMxStep = 64;

struct MxMat {
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows, cols;
  int32_t strips, chunks;
};

constexpr int mx_bits(int fmt) { return fmt == NC_E2M1 ? 4 : 8; }
constexpr int mx_step_bytes(int fmt) { return kMxRows * kMxStep * mx_bits(fmt) / 8; }
constexpr int mx_chunk_bytes(int fmt) { return 4 * mx_step_bytes(fmt); }
constexpr int kMxScaleBytes = 256;   // of a strip and chunk
constexpr int kMxFusedRows = 8;      // unquantised rows that the few-row product quantises itself

// A plane of fp32 or bf16 elements: row i starts at p + i * stride elements.
template <typename P> struct Plane {
  P p;
  int64_t stride;
};

// Where a piece of 16 bytes, that of column k of row r, lies in a strip's chunk.
template <int FMT> __device__ __forceinline__ int mx_piece(int r, int k) {
  if constexpr (FMT == NC_E2M1) return (k >> 6) * 1024 + (r + (k & 32)) * 16;
  else return (k >> 6) * 2048 + ((k >> 5) & 1) * 1024 + (r + 2 * (k & 16)) * 16;
}

// 2^X as a float whose exponent field is the scale byte (0 stands for 2^-127 and
// 255 for NaN in the scaled converts: measured for every code and scale byte).
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// A block's scale byte from the bits of its largest finite magnitude.  For a
// normal a = m 2^e the byte is e + 127 - emax, one more for PLUS1, one more for
// CEIL when m is above the largest value's own significand.  Subnormal a and
// anything below gives 0 (X = -127).
template <int FMT> __device__ __forceinline__ uint32_t mx_scale_byte(uint32_t a, int rule) {
  constexpr int EMAX = FMT == NC_E2M1 ? 2 : FMT == NC_E4M3 ? 8 : 15;
  constexpr uint32_t TOP = FMT == NC_E2M1 ? 0x400000u : 0x600000u;   // 1.5 and 1.75
  const int up = rule == NC_MX_PLUS1 ? 1 : (rule == NC_MX_CEIL && (a & 0x7FFFFFu) > TOP ? 1 : 0);
  const int b = (int)(a >> 23) - EMAX + up;
  return (uint32_t)(b < 0 ? 0 : b);
}

// Eight elements, as they lie in memory (fp32: 8 words, bf16: 4).
template <int DT> struct Eight { uint32_t w[DT == NC_BF16 ? 4 : 8]; };

template <int DT> __device__ __forceinline__ uint32_t bits_of(const Eight<DT>& x, int i) {
  if constexpr (DT == NC_BF16) return i & 1 ? x.w[i / 2] & 0xFFFF0000u : x.w[i / 2] << 16;
  else return x.w[i];
}

// Elements at .. at + 7 of a row of which `left` are there; past its end zeros.
// Rows may start on any element: the loads ask for no more alignment.
template <int DT> __device__ __forceinline__ Eight<DT> load8(const void* row, int64_t at, int64_t left) {
  Eight<DT> x;
  constexpr int N = DT == NC_BF16 ? 4 : 8;
  if constexpr (DT == NC_BF16) {
    const uint16_t* p = static_cast<const uint16_t*>(row) + at;
    if (left >= 8) {
      __builtin_memcpy(x.w, p, 16);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        x.w[i] = (2 * i < left ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < left ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(row) + at;
    if (left >= 8) {
      __builtin_memcpy(x.w, p, 32);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) x.w[i] = i < left ? p[i] : 0u;
    }
  }
  return x;
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

template <int DT> __device__ __forceinline__ Eight<DT> eight_of(const float (&y)[8]) {
  Eight<DT> x;
#pragma unroll
  for (int i = 0; i < (DT == NC_BF16 ? 4 : 8); ++i)
    x.w[i] = DT == NC_BF16 ? bf16_pair(y[2 * i % 8], y[(2 * i + 1) % 8]) : __float_as_uint(y[i]);
  return x;
}

// bf16 results of 32 MiB and more, what the eight L2s hold, are stored past the caches:
// they would only push out what is being read (8192 x 4096 E4M3 both ways and back 60
// us against 67, gated silu over 8192 x 11008 216 against 236; products 8192^3 E2M1 241
// against 245).  Smaller ones stay for whoever reads them next.  So do rows that do not
// start on 16 bytes, whose lines two stores share (3001 x 1357 fp32 26 us, 28 past the
// caches), and fp32, eight elements of which take two stores (a product 8192^3 to fp32
// 272 us, 323 past the caches).
template <int DT> inline bool mx_streams(const Plane<void*>& y, int64_t rows, int64_t cols) {
  return DT == NC_BF16 && rows * cols * 2 >= ((int64_t)32 << 20) && (((uintptr_t)y.p | (uintptr_t)(y.stride * 2)) & 15u) == 0;
}

template <int DT>
__device__ __forceinline__ void store8(void* row, int64_t at, int64_t left, const Eight<DT>& x, bool stream) {
  constexpr int N = DT == NC_BF16 ? 4 : 8;
  uint8_t* p = static_cast<uint8_t*>(row) + at * In<DT>::BYTES;
  if (left >= 8) {
    if (DT == NC_BF16 && stream)
      __builtin_nontemporal_store(u32x4{x.w[0], x.w[1], x.w[2], x.w[3]}, reinterpret_cast<u32x4*>(p));
    else
      __builtin_memcpy(p, x.w, 4 * N);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) {
        if constexpr (DT == NC_BF16) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(x.w[i / 2] >> (16 * (i & 1)));
        else reinterpret_cast<uint32_t*>(p)[i] = x.w[i];
      }
  }
}

// Largest finite magnitude of eight elements (fp32 bits), and what is not finite
// among them: bit 0 any, bit 1 a NaN.
template <int DT> __device__ __forceinline__ uint32_t amax8(const Eight<DT>& x, uint32_t& odd) {
  uint32_t a = 0;
  if constexpr (DT == NC_BF16) {                 // two at a time
    u16x2 m = __builtin_elementwise_max(__builtin_elementwise_max(mag16(x.w[0]), mag16(x.w[1])),
                                        __builtin_elementwise_max(mag16(x.w[2]), mag16(x.w[3])));
    a = (uint32_t)max(m.x, m.y) << 16;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, x.w[i] & kAbsMask);
  }
  odd = 0;
  if (a > kMaxFinite) {
    odd = a > kInfBits ? 3u : 1u;
    a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = bits_of<DT>(x, i) & kAbsMask;
      a = max(a, m > kMaxFinite ? 0u : m);
    }
  }
  return a;
}

// Eight elements at scale 2^X (byte sb) -> codes: .x holds E2M1's, .x and .y the
// 8-bit formats'.  The scaled converts round to nearest even and saturate (E2M1)
// or are saturated after; infinities become +-max, a NaN 0x7F (E2M1 has none:
// the caller marks the block).
template <int FMT, int DT> __device__ __forceinline__ u32x2 encode8(const Eight<DT>& x, uint32_t sb, uint32_t odd) {
  const float s = mx_scale(sb);
  if constexpr (FMT == NC_E2M1) {
    uint32_t w = 0;
    if constexpr (DT == NC_BF16) {
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x.w[0]), s, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x.w[1]), s, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x.w[2]), s, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2_t, x.w[3]), s, 3);
    } else {
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.w[0]), __uint_as_float(x.w[1]), s, 0);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.w[2]), __uint_as_float(x.w[3]), s, 1);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.w[4]), __uint_as_float(x.w[5]), s, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x.w[6]), __uint_as_float(x.w[7]), s, 3);
    }
    if (odd) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = bits_of<DT>(x, i);
        if ((b & kAbsMask) > kMaxFinite) w = (w & ~(0xFu << (4 * i))) | ((7u | ((b >> 28) & 8u)) << (4 * i));
      }
    }
    return u32x2{w, 0u};
  } else {
    u32x2 w;
    if constexpr (DT == NC_BF16) {
      const u32x4 v = {x.w[0], x.w[1], x.w[2], x.w[3]};
      w = u32x2{scvt4<FMT, NC_BF16>(v, 0, s), scvt4<FMT, NC_BF16>(v, 1, s)};
    } else {
      const u32x4 lo = {x.w[0], x.w[1], x.w[2], x.w[3]}, hi = {x.w[4], x.w[5], x.w[6], x.w[7]};
      w = u32x2{scvt4<FMT, NC_F32>(lo, 0, s), scvt4<FMT, NC_F32>(hi, 0, s)};
    }
    if (odd) {
      uint32_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) b[i] = bits_of<DT>(x, i);
      w.x = fix_nonfinite4<FMT>(w.x, b);
      w.y = fix_nonfinite4<FMT>(w.y, b + 4);
    }
    return w;
  }
}

// Codes 2i, 2i + 1 of eight -> packed bf16 at scale 2^X: exact, as a code has at
// most four significant bits (below bf16's range rounded to nearest even).
template <int FMT> __device__ __forceinline__ uint32_t mx_pair(u32x2 c, float s, int i) {
  bf16x2_t r;
  if constexpr (FMT == NC_E2M1) {
    switch (i) {
      case 0: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 0); break;
      case 1: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 1); break;
      case 2: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 2); break;
      default: r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c.x, s, 3); break;
    }
  } else {
    const uint32_t w = i < 2 ? c.x : c.y;
    if constexpr (FMT == NC_E4M3) {
      if (i & 1) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true);
      else r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
    } else {
      if (i & 1) r = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, s, true);
      else r = __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, s, false);
    }
  }
  return __builtin_bit_cast(uint32_t, r);
}

// Eight codes -> fp32 values: a code's bf16 value at scale 2^0, times 2^X (exact,
// or rounded once in fp32's subnormal range); byte 255 is NaN.
template <int FMT> __device__ __forceinline__ void decode8(u32x2 c, uint32_t sb, float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = mx_pair<FMT>(c, 1.0f, i);
    y[2 * i] = __builtin_amdgcn_ldexpf(__uint_as_float(r << 16), (int)sb - 127);
    y[2 * i + 1] = __builtin_amdgcn_ldexpf(__uint_as_float(r & 0xFFFF0000u), (int)sb - 127);
  }
  if (sb == 255u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(0x7FC00000u);
  }
}

// ---- Streaming over a matrix ----------------------------------------------------
// What the kernels that write, read and keep matrices share: a workgroup of four
// waves takes one strip and chunk, wave w rows 8 w .. 8 w + 7 of the strip, and a
// lane eight elements of each of the chunk's four steps.  A wave then touches 128
// bytes of bf16 of each row, and of the codes runs of 128 bytes; a block lies in
// four neighbouring lanes, and a lane's four scale bytes are one dword.
struct MxLane {
  int r, q;            // row of the strip; which eight of a step's 64 columns
  int64_t row, col0;   // row of the matrix, first column of the chunk
  int64_t tile;        // strip * chunks + chunk
  __device__ __forceinline__ explicit MxLane(const MxMat& m, uint32_t at = blockIdx.x) {
    const uint32_t strip = at / (uint32_t)m.chunks, chunk = at % (uint32_t)m.chunks;
    r = (int)(threadIdx.x >> 3);
    q = (int)(threadIdx.x & 7);
    row = (int64_t)strip * kMxRows + r;
    col0 = (int64_t)chunk * kMxChunk;
    tile = (int64_t)at;
  }
  __device__ __forceinline__ int64_t col(int step) const { return col0 + kMxStep * step + 8 * q; }
  // byte of this lane's eight codes of a step, in the matrix's codes; of its scales
  template <int FMT> __device__ __forceinline__ int64_t codes(int step) const {
    if constexpr (FMT == NC_E2M1) return tile * mx_chunk_bytes(FMT) + mx_piece<FMT>(r, kMxStep * step + 8 * q) + 4 * (q & 3);
    else return tile * mx_chunk_bytes(FMT) + mx_piece<FMT>(r, kMxStep * step + 8 * q) + 8 * (q & 1);
  }
  __device__ __forceinline__ int64_t scales() const { return tile * kMxScaleBytes + (r + 32 * (q >> 2)) * 4; }
};

template <int FMT> __device__ __forceinline__ void put_codes(uint8_t* p, u32x2 c) {
  if constexpr (FMT == NC_E2M1) *reinterpret_cast<uint32_t*>(p) = c.x;
  else *reinterpret_cast<u32x2*>(p) = c;
}
template <int FMT> __device__ __forceinline__ u32x2 get_codes(const uint8_t* p) {
  if constexpr (FMT == NC_E2M1) return u32x2{*reinterpret_cast<const uint32_t*>(p), 0u};
  else return *reinterpret_cast<const u32x2*>(p);
}

// max and or over the four lanes of a block (quad permutes: no LDS)
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
  return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t quad_or(uint32_t v) {
  v |= (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
  return v | (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);
}

// Quantises a lane's eight elements of a block that four lanes share.
template <int FMT, int DT> __device__ __forceinline__ u32x2 encode_quad(const Eight<DT>& x, int rule, uint32_t& sb) {
  uint32_t odd;
  const uint32_t a = quad_max(amax8<DT>(x, odd));
  sb = mx_scale_byte<FMT>(a, rule);
  const u32x2 c = encode8<FMT, DT>(x, sb, odd);
  if (FMT == NC_E2M1 && (quad_or(odd) & 2u)) sb = 255u;
  return c;
}

// ---- launches ---------------------------------------------------------------------

// One product: out = (out +) a b^T (+ bias), out [a.rows, b.rows].
struct MxProduct {
  MxMat a, b;
  const void* x;        // few rows of a linear layer: unquantised a, quantised on the way
  int64_t x_stride;
  int32_t x_dtype, rule;
  void* out;
  int64_t out_stride;
  const void* bias;     // nullable, of out's type
  int32_t out_dtype, accumulate;
  int32_t stream;       // out goes past the caches
  int32_t splits;       // parts of the columns, joined through part
  float* part;
};

hipError_t launch_mx_write(const MxMat* m, const MxMat* t, int fmt, const Plane<const void*>& x, int dtype, int rule,
                           hipStream_t stream);
hipError_t launch_mx_read(const MxMat& m, int fmt, const Plane<void*>& y, int dtype, hipStream_t stream);
// Few rows: t x t strips a workgroup, t 1 or 2 (unquantised rows: 1).  Many rows, at
// least one column: 64 w x 64 w results a workgroup, w 2 or 4.
hipError_t launch_mx_few(const MxProduct& p, int fa, int fb, int t, hipStream_t stream);
hipError_t launch_mx_many(const MxProduct& p, int fa, int fb, int w, hipStream_t stream);

struct ActForward {
  Plane<const void*> gate, up;   // up.p null: no gate
  Plane<void*> y;
  bool stream;                   // y goes past the caches
  MxMat gate_q, up_q;            // codes null: nothing is kept
  int32_t rule;
};
struct ActBackward {
  Plane<const void*> dy;
  MxMat gate_q, up_q;
  Plane<void*> dgate, dup, y;    // y.p null: not wanted
  bool stream;
};
hipError_t launch_act_forward(const ActForward& a, int act, int fmt, int dtype, hipStream_t stream);
hipError_t launch_act_backward(const ActBackward& a, int act, int fmt, int dtype, hipStream_t stream);

}  // namespace nc
