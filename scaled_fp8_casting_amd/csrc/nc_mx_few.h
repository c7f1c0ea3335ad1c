// Products with few rows: one strip of 32 rows of a by one strip of b a
// workgroup, the chunks of 256 columns dealt to its waves in turn, operands
// straight from memory, the next chunk's under way while one is multiplied.  The
// bytes of b bound it.  The waves' sums meet in LDS in the waves' order.
//
// Up to kMxFusedRows unquantised rows (a linear layer's) are quantised on the way:
// each wave turns the columns of its own chunk into codes, in a place of its own in
// LDS where they lie as in a matrix.  Every workgroup does it again, which costs
// more the more rows there are; a kernel of its own writes more rows first.
#pragma once

#include "nc_mx_mul.h"

namespace nc {

constexpr int kMxFewWaves = 8;

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

template <int FA, int FB, bool WIDE, int ROWS>
__global__ void __launch_bounds__(64 * kMxFewWaves) mx_few(MxProduct p) {
  constexpr bool FUSED = ROWS != kMxNoRows;
  constexpr int DT = FUSED ? ROWS : NC_BF16;
  constexpr int PLACE = mx_chunk_bytes(FA) + kMxScaleBytes, SUMS = 32 * 33 * 4;
  constexpr int EACH = FUSED && PLACE > SUMS ? PLACE : SUMS;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kMxFewWaves * EACH];
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = (int)(threadIdx.x & 63);
  const uint32_t strip_b = blockIdx.x % (uint32_t)p.b.strips, strip_a = blockIdx.x / (uint32_t)p.b.strips;
  uint8_t* place = lds + wave * EACH;
  f32x16_t acc = {};
  const int32_t chunks = p.b.chunks;
  const uint8_t* cb = p.b.codes + (int64_t)strip_b * chunks * mx_chunk_bytes(FB);
  const uint8_t* sb = p.b.scales + (int64_t)strip_b * chunks * kMxScaleBytes;
  const uint8_t* ca = p.a.codes + (int64_t)strip_a * chunks * mx_chunk_bytes(FA);
  const uint8_t* sa = p.a.scales + (int64_t)strip_a * chunks * kMxScaleBytes;
  MxChunk<FA> a;
  MxChunk<FB> b;
  const auto load = [&](int32_t c, MxChunk<FA>& x, MxChunk<FB>& y) {
    y.load(cb + (int64_t)c * mx_chunk_bytes(FB), sb + (int64_t)c * kMxScaleBytes, lane);
    if constexpr (!FUSED) x.load(ca + (int64_t)c * mx_chunk_bytes(FA), sa + (int64_t)c * kMxScaleBytes, lane);
  };
  if (wave < chunks) load(wave, a, b);
  for (int32_t c = wave; c < chunks; c += kMxFewWaves) {
    MxChunk<FA> na;
    MxChunk<FB> nb;
    if (c + kMxFewWaves < chunks) load(c + kMxFewWaves, na, nb);
    if constexpr (FUSED) {
      mx_quantise<FA, DT>(place, p, (int)p.a.rows, (int64_t)c * kMxChunk, lane);
      a.load(place, place + mx_chunk_bytes(FA), lane);
    }
    const MxScales xa = mx_scales<WIDE>(a.scales, lane), xb = mx_scales<WIDE>(b.scales, lane);
    if constexpr (WIDE) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        acc = mx_mma_wide(mx_widen<FA>(a.f[s], (xa.block0 >> (8 * s)) & 255u, (xa.block1 >> (8 * s)) & 255u),
                          mx_widen<FB>(b.f[s], (xb.block0 >> (8 * s)) & 255u, (xb.block1 >> (8 * s)) & 255u), acc);
    } else {
      acc = mx_mma<FA, FB, 0>(a.f[0], b.f[0], acc, xa.own, xb.own);
      acc = mx_mma<FA, FB, 1>(a.f[1], b.f[1], acc, xa.own, xb.own);
      acc = mx_mma<FA, FB, 2>(a.f[2], b.f[2], acc, xa.own, xb.own);
      acc = mx_mma<FA, FB, 3>(a.f[3], b.f[3], acc, xa.own, xb.own);
    }
    b = nb;
    if constexpr (!FUSED) a = na;
  }
  if constexpr (FUSED) __syncthreads();          // the sums lie where the rows were
  float (*sums)[32][33] = reinterpret_cast<float (*)[32][33]>(lds);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int r = 8 * (i / 4) + 4 * (lane >> 5) + i % 4;
    if (!FUSED || r < p.a.rows) sums[wave][r][lane & 31] = acc[i];
  }
  __syncthreads();
  if (threadIdx.x < 256) {
    const int r = (int)(threadIdx.x >> 3), c = (int)(threadIdx.x & 7) * 4;
    const int64_t row = (int64_t)strip_a * kMxRows + r, col = (int64_t)strip_b * kMxRows + c;
    if (row < p.a.rows && col < p.b.rows) {
      float y[4] = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kMxFewWaves; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] += sums[w][r][c + i];
      mx_store4(p, row, col, p.b.rows - col, y);
    }
  }
}

template <int FA, int FB, bool WIDE> hipError_t mx_few_run(const MxProduct& p, hipStream_t stream) {
  const dim3 grid((uint32_t)p.a.strips * (uint32_t)p.b.strips), block(64 * kMxFewWaves);
  if (p.x == nullptr) mx_few<FA, FB, WIDE, kMxNoRows><<<grid, block, 0, stream>>>(p);
  else if (p.x_dtype == NC_BF16) mx_few<FA, FB, WIDE, NC_BF16><<<grid, block, 0, stream>>>(p);
  else mx_few<FA, FB, WIDE, NC_F32><<<grid, block, 0, stream>>>(p);
  return hipGetLastError();
}
template <int FA, int FB> hipError_t mx_few_launch(const MxProduct& p, hipStream_t stream) {
  if constexpr (FA != NC_E2M1 || FB != NC_E2M1) {
    if (p.out_dtype == NC_F32) return mx_few_run<FA, FB, true>(p, stream);
  }
  return mx_few_run<FA, FB, false>(p, stream);
}

hipError_t mx_few_e2m1(const MxProduct& p, int fb, hipStream_t stream);
hipError_t mx_few_e4m3(const MxProduct& p, int fb, hipStream_t stream);
hipError_t mx_few_e5m2(const MxProduct& p, int fb, hipStream_t stream);

}  // namespace nc
