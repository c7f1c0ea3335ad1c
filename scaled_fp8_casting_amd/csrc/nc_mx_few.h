// Products with few rows, and small ones: T strips of 32 rows of a by T strips of b a
// workgroup, the chunks of 256 columns dealt to its waves in turn, operands straight
// from memory.  Their bytes bound it: those of b with few rows, else what the
// workgroups' operands overlap, which T = 2 halves.  The waves' sums meet in LDS in a
// fixed order.
//
// Up to kMxFusedRows unquantised rows (a linear layer's) are quantised on the way:
// each wave turns the columns of its own chunk into codes, in a place of its own in
// LDS where they lie as in a matrix.  Every workgroup does it again, which costs
// more the more rows there are; a kernel of its own writes more rows first.  In us,
// quantised on the way and first, bf16 rows to E2M1 or E4M3 against E2M1 weights,
// replayed from a graph over twelve matrices:
//                            6 rows        8            12           16
//   E2M1   4096 ->  4096    5.9   7.6    6.3   7.4    7.4   7.5    8.2   7.4
//          4096 -> 11008   10.3  11.9   11.0  11.4   13.2  11.8   15.3  11.5
//         11008 ->  4096   11.8  13.2   13.0  12.9   15.4  13.3   17.6  12.7
//   E4M3   4096 ->  4096    6.0   8.1    6.5   8.1    7.5   8.2    8.4   8.1
//          4096 -> 11008   10.6  13.0   11.3  12.5   13.7  13.0   15.6  12.6
//         11008 ->  4096   11.8  15.2   12.9  14.9   15.6  15.3   17.9  14.9
//
// 1 x 4096 E4M3 -> 4096 E2M1 takes 5.6 us (8.9 MB of weights; the launch and two trips
// to memory), 24 x 4096 -> 11008 E2M1 7.1 behind a write of 3.4 (24 MB at 3.4 TB/s).
#pragma once

#include "nc_mx_mul.h"

namespace nc {

// Rows in place of a matrix.
enum { kMxNoRows = -1 };   // else their nc_dtype

// `rows` rows of a chunk into a wave's place: codes, then scales, as a strip's chunk
// in a matrix.  The rows past the last keep what was there: they reach only results
// that nobody stores.
template <int FMT, int DT>
__device__ __forceinline__ void mx_quantise(uint8_t* place, const MxProduct& p, int rows, int64_t col0, int lane) {
  const int q = lane & 31;                     // eight of the chunk's 256 columns
  const int k = 8 * q;
  for (int r = lane >> 5; r < rows + (lane >> 5); r += 2) {     // both halves take every turn: quads stay whole
    const bool there = r < rows;
    const uint8_t* row = static_cast<const uint8_t*>(p.x) + (int64_t)r * p.x_stride * In<DT>::BYTES;
    const Eight<DT> v = load8<DT>(row, col0 + k, there ? p.b.cols - col0 - k : 0);
    uint32_t sb;
    const u32x2 c = encode_quad<FMT, DT>(v, p.rule, sb);
    if (there) {
      put_codes<FMT>(place + mx_piece<FMT>(r, k) + (FMT == NC_E2M1 ? 4 * (q & 3) : 8 * (q & 1)), c);
      if ((q & 3) == 0) place[mx_chunk_bytes(FMT) + (r + (k & 32)) * 4 + (k >> 6)] = (uint8_t)sb;
    }
  }
  __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

template <int FMT> struct MxChunk {            // a wave's operand of a chunk
  MxFrag<FMT> f[4];
  uint32_t scales;
  __device__ __forceinline__ void load(const uint8_t* codes, const uint8_t* s, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = mx_frag<FMT>(codes + i * mx_step_bytes(FMT), lane);
    scales = *reinterpret_cast<const uint32_t*>(s + lane * 4);
  }
};

template <int FA, int FB, bool WIDE, int S>
__device__ __forceinline__ void mx_few_step(f32x16_t& acc, const MxChunk<FA>& a, const MxChunk<FB>& b, const MxScales& xa, const MxScales& xb) {
  if constexpr (WIDE)
    acc = mx_mma_wide(mx_widen<FA>(a.f[S], (xa.block0 >> (8 * S)) & 255u, (xa.block1 >> (8 * S)) & 255u),
                      mx_widen<FB>(b.f[S], (xb.block0 >> (8 * S)) & 255u, (xb.block1 >> (8 * S)) & 255u), acc);
  else
    acc = mx_mma<FA, FB, S>(a.f[S], b.f[S], acc, xa.own, xb.own);
}

template <int FA, int FB, bool WIDE, int ROWS, int T, int WAVES>
__global__ void __launch_bounds__(64 * WAVES) mx_few(MxProduct p) {
  constexpr bool FUSED = ROWS != kMxNoRows;
  constexpr int DT = FUSED ? ROWS : NC_BF16;
  constexpr int PLACE = mx_chunk_bytes(FA) + kMxScaleBytes;
  constexpr int HALF = WAVES / 2, SIDE = 32 * T, LEAD = SIDE + 1;
  constexpr int SUMS = HALF * SIDE * LEAD * 4;
  constexpr int LDS = FUSED && WAVES * PLACE > SUMS ? WAVES * PLACE : SUMS;
  __shared__ __attribute__((aligned(16))) uint8_t lds[LDS];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = (int)(threadIdx.x & 63);
  const uint32_t across = ((uint32_t)p.b.strips + T - 1) / T;
  const int32_t strip_b = (int32_t)(blockIdx.x % across) * T, strip_a = (int32_t)(blockIdx.x / across) * T;
  uint8_t* place = lds + wave * PLACE;
  f32x16_t acc[T][T] = {};
  const int32_t chunks = p.b.chunks;
  const uint8_t *ca[T], *sa[T], *cb[T], *sb[T];
#pragma unroll
  for (int i = 0; i < T; ++i) {                  // strips past the end are the last one's again
    const int64_t ia = (int64_t)min(strip_a + i, p.a.strips - 1) * chunks, ib = (int64_t)min(strip_b + i, p.b.strips - 1) * chunks;
    ca[i] = p.a.codes + ia * mx_chunk_bytes(FA);
    sa[i] = p.a.scales + ia * kMxScaleBytes;
    cb[i] = p.b.codes + ib * mx_chunk_bytes(FB);
    sb[i] = p.b.scales + ib * kMxScaleBytes;
  }
  MxChunk<FA> a[T];
  MxChunk<FB> b[T];
  const auto load = [&](int32_t c, MxChunk<FA> (&x)[T], MxChunk<FB> (&y)[T]) {
#pragma unroll
    for (int i = 0; i < T; ++i) {
      y[i].load(cb[i] + (int64_t)c * mx_chunk_bytes(FB), sb[i] + (int64_t)c * kMxScaleBytes, lane);
      if constexpr (!FUSED) x[i].load(ca[i] + (int64_t)c * mx_chunk_bytes(FA), sa[i] + (int64_t)c * kMxScaleBytes, lane);
    }
  };
  const auto multiply = [&](MxChunk<FA> (&x)[T], MxChunk<FB> (&y)[T]) {
    MxScales xa[T], xb[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
      xa[i] = mx_scales<WIDE>(x[i].scales, lane);
      xb[i] = mx_scales<WIDE>(y[i].scales, lane);
    }
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int j = 0; j < T; ++j) {
        mx_few_step<FA, FB, WIDE, 0>(acc[i][j], x[i], y[j], xa[i], xb[j]);
        mx_few_step<FA, FB, WIDE, 1>(acc[i][j], x[i], y[j], xa[i], xb[j]);
        mx_few_step<FA, FB, WIDE, 2>(acc[i][j], x[i], y[j], xa[i], xb[j]);
        mx_few_step<FA, FB, WIDE, 3>(acc[i][j], x[i], y[j], xa[i], xb[j]);
      }
  };
  if constexpr (T == 1) {                        // the next chunk is under way while one is multiplied
    if (wave < chunks) load(wave, a, b);
    for (int32_t c = wave; c < chunks; c += WAVES) {
      MxChunk<FA> na[T];
      MxChunk<FB> nb[T];
      if (c + WAVES < chunks) load(c + WAVES, na, nb);
      if constexpr (FUSED) {
        mx_quantise<FA, DT>(place, p, (int)p.a.rows, (int64_t)c * kMxChunk, lane);
        a[0].load(place, place + mx_chunk_bytes(FA), lane);
      }
      multiply(a, b);
      b[0] = nb[0];
      if constexpr (!FUSED) a[0] = na[0];
    }
  } else {                                       // two waves a SIMD take turns
    for (int32_t c = wave; c < chunks; c += WAVES) {
      load(c, a, b);
      multiply(a, b);
    }
  }
  // The second half of the waves leave their sums, the first half add them to their
  // own; then these meet.
  if constexpr (FUSED) __syncthreads();          // the sums lie where the rows were
  float (*sums)[SIDE][LEAD] = reinterpret_cast<float (*)[SIDE][LEAD]>(lds);
  const auto leave = [&](bool add) {
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int j = 0; j < T; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = 32 * i + 8 * (e / 4) + 4 * (lane >> 5) + e % 4;
          if (!FUSED || r < p.a.rows) {
            float& y = sums[wave % HALF][r][32 * j + (lane & 31)];
            y = add ? y + acc[i][j][e] : acc[i][j][e];
          }
        }
  };
  if (wave >= HALF) leave(false);
  __syncthreads();
  if (wave < HALF) leave(true);
  __syncthreads();
  for (int i = (int)threadIdx.x; i < SIDE * SIDE / 4; i += 64 * WAVES) {
    const int r = i / (SIDE / 4), c = i % (SIDE / 4) * 4;
    const int64_t row = (int64_t)strip_a * kMxRows + r, col = (int64_t)strip_b * kMxRows + c;
    if (row < p.a.rows && col < p.b.rows) {
      float y[4] = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < HALF; ++w)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += sums[w][r][c + e];
      MxStore<4>(p, col)(row, y);
    }
  }
}

template <int FA, int FB, bool WIDE, int ROWS, int T, int WAVES> hipError_t mx_few_go(const MxProduct& p, hipStream_t stream) {
  const dim3 grid(((uint32_t)p.a.strips + T - 1) / T * (((uint32_t)p.b.strips + T - 1) / T));
  mx_few<FA, FB, WIDE, ROWS, T, WAVES><<<grid, dim3(64 * WAVES), 0, stream>>>(p);
  return hipGetLastError();
}
template <int FA, int FB, bool WIDE> hipError_t mx_few_run(const MxProduct& p, int t, hipStream_t stream) {
  if (p.x == nullptr) return t == 2 ? mx_few_go<FA, FB, WIDE, kMxNoRows, 2, 8>(p, stream) : mx_few_go<FA, FB, WIDE, kMxNoRows, 1, 8>(p, stream);
  // With a compute unit for each workgroup, sixteen waves take in more at once (1 x
  // 11008 -> 4096, 4 by 4 bits: 9.2 us against 11.4); two matrices' operands do not fit
  // their registers (32 x 11008 -> 4096 of 8 by 8 bits, called one by one: 30 us against 20 with eight
  // waves, which take 16.2 replayed from a graph).
  // So it is for 8 bits through bf16.
  constexpr int MORE = WIDE && FB != NC_E2M1 ? 8 : 16;
  if (p.b.strips <= 256 && p.b.chunks > 8)
    return p.x_dtype == NC_BF16 ? mx_few_go<FA, FB, WIDE, NC_BF16, 1, MORE>(p, stream) : mx_few_go<FA, FB, WIDE, NC_F32, 1, MORE>(p, stream);
  return p.x_dtype == NC_BF16 ? mx_few_go<FA, FB, WIDE, NC_BF16, 1, 8>(p, stream) : mx_few_go<FA, FB, WIDE, NC_F32, 1, 8>(p, stream);
}
template <int FA, int FB> hipError_t mx_few_launch(const MxProduct& p, int t, hipStream_t stream) {
  if constexpr (FA != NC_E2M1 || FB != NC_E2M1) {
    if (p.out_dtype == NC_F32) return mx_few_run<FA, FB, true>(p, t, stream);
  }
  return mx_few_run<FA, FB, false>(p, t, stream);
}

hipError_t mx_few_e2m1(const MxProduct& p, int fb, int t, hipStream_t stream);
hipError_t mx_few_e4m3(const MxProduct& p, int fb, int t, hipStream_t stream);
hipError_t mx_few_e5m2(const MxProduct& p, int fb, int t, hipStream_t stream);

}  // namespace nc
