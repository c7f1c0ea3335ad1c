// Products with few rows: one strip of 32 rows of a by one strip of b a
// workgroup, the chunks of 256 columns dealt to its waves in turn, operands
// straight from memory.  The bytes of b bound it.  The waves' sums meet in LDS in
// the waves' order.
#pragma once

#include "nc_mx_mul.h"

namespace nc {

constexpr int kMxFewWaves = 8;

// A lane's part of an operand from unquantised rows: block b of a step lies in one
// lane (E2M1) or in the two lanes r and r + 32 (16 columns each).  sb: the scale
// byte of the lane's own block, in byte S.
template <int FMT, int DT>
__device__ __forceinline__ MxFrag<FMT> mx_quantise(const void* row, int64_t col0, int64_t left, int lane, int rule, uint32_t& sb) {
  const int g = lane >> 5;
  Eight<DT> v[4];
  uint32_t odd[4];
  MxFrag<FMT> f;
  if constexpr (FMT == NC_E2M1) {
    uint32_t a = 0, any = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = load8<DT>(row, col0 + 32 * g + 8 * e, left - 32 * g - 8 * e);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a = max(a, amax8<DT>(v[e], odd[e]));
      any |= odd[e];
    }
    sb = mx_scale_byte<FMT>(a, rule);
#pragma unroll
    for (int e = 0; e < 4; ++e) f.w[0][e] = encode8<FMT, DT>(v[e], sb, odd[e]).x;
    if (any & 2u) sb = 255u;
  } else {
    uint32_t s[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = 32 * (e / 2) + 16 * g + 8 * (e % 2);
      v[e] = load8<DT>(row, col0 + k, left - k);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t a = max(amax8<DT>(v[2 * h], odd[2 * h]), amax8<DT>(v[2 * h + 1], odd[2 * h + 1]));
      a = max(a, (uint32_t)__shfl_xor((int)a, 32));
      s[h] = mx_scale_byte<FMT>(a, rule);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const u32x2 c = encode8<FMT, DT>(v[2 * h + e], s[h], odd[2 * h + e]);
        f.w[h][2 * e] = c.x;
        f.w[h][2 * e + 1] = c.y;
      }
    }
    sb = g ? s[1] : s[0];
  }
  return f;
}

template <int FA, int FB, bool WIDE>
__global__ void __launch_bounds__(64 * kMxFewWaves) mx_few(MxProduct p) {
  __shared__ float sums[kMxFewWaves][32][33];
  const int wave = (int)(threadIdx.x >> 6), lane = (int)(threadIdx.x & 63);
  const uint32_t strip_b = blockIdx.x % (uint32_t)p.b.strips, strip_a = blockIdx.x / (uint32_t)p.b.strips;
  f32x16_t acc = {};
  const uint8_t* cb = p.b.codes + (int64_t)strip_b * p.b.chunks * mx_chunk_bytes(FB);
  const uint8_t* sb = p.b.scales + (int64_t)strip_b * p.b.chunks * kMxScaleBytes;
  const uint8_t* ca = p.a.codes + (int64_t)strip_a * p.b.chunks * mx_chunk_bytes(FA);
  const uint8_t* sa = p.a.scales + (int64_t)strip_a * p.b.chunks * kMxScaleBytes;
  const int64_t row_a = (int64_t)strip_a * kMxRows + (lane & 31);
  for (int c = wave; c < p.b.chunks; c += kMxFewWaves) {
    MxFrag<FB> b[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) b[s] = mx_frag<FB>(cb + (int64_t)c * mx_chunk_bytes(FB) + s * mx_step_bytes(FB), lane);
    const MxScales xb = mx_scales<WIDE>(*reinterpret_cast<const uint32_t*>(sb + (int64_t)c * kMxScaleBytes + lane * 4), lane);
    MxFrag<FA> a[4];
    uint32_t own = 0;
    if (p.x != nullptr) {
      const int64_t left = row_a < p.a.rows ? p.b.cols - (int64_t)c * kMxChunk : 0;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t byte;
        if (p.x_dtype == NC_BF16)
          a[s] = mx_quantise<FA, NC_BF16>(static_cast<const uint16_t*>(p.x) + row_a * p.x_stride, (int64_t)c * kMxChunk + kMxStep * s,
                                          left - kMxStep * s, lane, p.rule, byte);
        else
          a[s] = mx_quantise<FA, NC_F32>(static_cast<const float*>(p.x) + row_a * p.x_stride, (int64_t)c * kMxChunk + kMxStep * s,
                                         left - kMxStep * s, lane, p.rule, byte);
        own |= byte << (8 * s);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) a[s] = mx_frag<FA>(ca + (int64_t)c * mx_chunk_bytes(FA) + s * mx_step_bytes(FA), lane);
      own = *reinterpret_cast<const uint32_t*>(sa + (int64_t)c * kMxScaleBytes + lane * 4);
    }
    const MxScales xa = mx_scales<WIDE>(own, lane);
    if constexpr (WIDE) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        acc = mx_mma_wide(mx_widen<FA>(a[s], (xa.block0 >> (8 * s)) & 255u, (xa.block1 >> (8 * s)) & 255u),
                          mx_widen<FB>(b[s], (xb.block0 >> (8 * s)) & 255u, (xb.block1 >> (8 * s)) & 255u), acc);
    } else {
      acc = mx_mma<FA, FB, 0>(a[0], b[0], acc, xa.own, xb.own);
      acc = mx_mma<FA, FB, 1>(a[1], b[1], acc, xa.own, xb.own);
      acc = mx_mma<FA, FB, 2>(a[2], b[2], acc, xa.own, xb.own);
      acc = mx_mma<FA, FB, 3>(a[3], b[3], acc, xa.own, xb.own);
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[wave][8 * (i / 4) + 4 * (lane >> 5) + i % 4][lane & 31] = acc[i];
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

template <int FA, int FB> hipError_t mx_few_launch(const MxProduct& p, hipStream_t stream) {
  const dim3 grid((uint32_t)p.a.strips * (uint32_t)p.b.strips), block(64 * kMxFewWaves);
  if ((FA != NC_E2M1 || FB != NC_E2M1) && p.out_dtype == NC_F32) mx_few<FA, FB, FA != NC_E2M1 || FB != NC_E2M1><<<grid, block, 0, stream>>>(p);
  else mx_few<FA, FB, false><<<grid, block, 0, stream>>>(p);
  return hipGetLastError();
}

hipError_t mx_few_e2m1(const MxProduct& p, int fb, hipStream_t stream);
hipError_t mx_few_e4m3(const MxProduct& p, int fb, hipStream_t stream);
hipError_t mx_few_e5m2(const MxProduct& p, int fb, hipStream_t stream);

}  // namespace nc
