// Attention over the paged cache for many rows: prompts, chunks of prompts,
// cross attention.  Definitions as in nc_kv_few.h.
//
// Matrix work and the softmax's vector work bound it, so codes are converted
// once for a workgroup of four waves and 32 rows each: every step takes 64
// keys, wave w loads tile w (prefetched one step ahead), converts it and puts
// it into LDS as operands --
//
//   keys:   [8 elements u = 0..D/8-1][key 0..63][16 bytes]
//   values: [16-key step][half h][element tile of 32][lane][quads h, 2 + h: 16 bytes]
//
// each read with 16 bytes a lane by 32x32x16 bf16 products S^T = K Q^T and
// O^T = V^T P^T.  The two halves of a wave read runs that lie 128 bytes apart
// modulo the 256 of all banks: without that shift they met in the same banks,
// a third of the kernel's cycles.  As in the few-row kernel the scores of a query lie in one
// lane (and its partner 32 lanes on) in the order the second product wants
// them.  Two LDS buffers: a step's conversion goes beside the products of the
// step before, with one barrier between steps.
#pragma once

#include "nc_kv_few.h"

namespace nc {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

__device__ __forceinline__ f32x16_t mfma32(const u32x4& a, const u32x4& b, const f32x16_t& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

constexpr int kManyWaves = 4, kManyKeys = 64;
static_assert(32 * kManyWaves == kKvManyRows, "32 rows a wave");

template <int FMT, int D> struct ManyLds {
  uint32_t k[D / 8][kManyKeys + 8][4];
  uint32_t v[kManyKeys / 16][2][D + 8][4];
  uint32_t bad[kManyWaves];        // the wave's values hold one that is not finite (steps with masks only)
};

// A wave's tile from registers to operands in LDS.
template <int FMT, int D, bool MASKED>
__device__ __forceinline__ void stage(ManyLds<FMT, D>& s, const KvRegs<FMT, D>& r, int wave, int lane, bool there, int keys) {
  using L = Kv<FMT, D>;
  const int m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int sg = 0; sg < L::NSEG; ++sg) {
    const float sc = kv_scale(r.ks[sg]);
    constexpr int DWS = 4 * L::BITS / 16;      // dwords of eight codes
#pragma unroll
    for (int st = 0; st < L::piece(sg) / 8; ++st) {
      const uint32_t* c = r.k + L::off(sg) / 16 + st * DWS;
      u32x4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = kv_pair<FMT>(c[i * DWS / 4], sc, i % (4 / DWS));
      *reinterpret_cast<u32x4*>(s.k[L::dim0(sg) / 8 + g * (L::piece(sg) / 8) + st][16 * wave + m]) = a;
    }
  }
  // tokens past the end, or on a missing page, hold anything: cleared
  uint32_t keep[2] = {~0u, ~0u}, nf = 0;
  if constexpr (MASKED) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      keep[i] = there ? (4 * g + 2 * i < keys ? 0xFFFFu : 0u) | (4 * g + 2 * i + 1 < keys ? 0xFFFF0000u : 0u) : 0u;
  }
#pragma unroll
  for (int sg = 0; sg < L::NSEG; ++sg) {
    constexpr int P4 = 2 * L::DPB;             // pairs of a dword
    const int pairs = L::lane(sg) / 2;
    float sc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i] = kv_scale((r.vs[sg] >> (8 * i)) & 255u);
#pragma unroll
    for (int pr = 0; pr < pairs; ++pr) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = i * pairs + pr;
        w[i] = kv_pair<FMT>(r.v[L::off(sg) / 16 + at / P4], sc[i], at % P4);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x2 x = {zip(w[0], w[1], h), zip(w[2], w[3], h)};
        if constexpr (MASKED) {
          x.x &= keep[0];
          x.y &= keep[1];
          nf |= not_finite16(x.x) | not_finite16(x.y);
        }
        // quad g: half g % 2, first or second eight bytes of its operand
        *reinterpret_cast<u32x2*>(&s.v[wave][g & 1][L::dim0(sg) + 32 * pr + 16 * h + m][2 * (g >> 1)]) = x;
      }
    }
  }
  if constexpr (MASKED) {
    const uint64_t any = __ballot(nf != 0);
    if (lane == 0) s.bad[wave] = any != 0;
  }
}

template <int FMT, int D, int DT> struct Many {
  using L = Kv<FMT, D>;
  static constexpr int QP = QParts<DT>::N;
  static constexpr int KS = kManyKeys / 32;    // score tiles

  u32x4 q[D / 16][QP];
  f32x16_t o[D / 32];
  float m, l;                                  // reference and sum of this lane's keys, scaled and unscaled
  int end, begin;

  template <bool MASKED>
  __device__ __forceinline__ void step(const ManyLds<FMT, D>& lds, int base, uint32_t there, float scale2, int lane) {
    const int n = lane & 31, h = lane >> 5;
    f32x16_t s[KS];
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[j][i] = 0;
#pragma unroll
    for (int st = 0; st < D / 16; ++st)
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(lds.k[2 * st + h][32 * j + n]);
#pragma unroll
        for (int c = QP - 1; c >= 0; --c) s[j] = mfma32(a, q[st][c], s[j]);
      }
    float top = -INFINITY;
    uint32_t see[KS];                          // bit i: the row sees key i of the lane's
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      see[j] = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (MASKED) {
          const int at = 32 * j + 8 * (i / 4) + 4 * h + i % 4, key = base + at;
          const bool on = key < end && key >= begin && ((there >> (at / 16)) & 1);
          see[j] |= on ? 1u << i : 0u;
          s[j][i] = on ? s[j][i] : -INFINITY;
        }
        top = fmaxf(top, s[j][i]);
      }
    }
    top = max_halves(top) * scale2;
    if (MASKED && !(top > -INFINITY)) top = -INFINITY;       // 0 scale times no key
    if (__ballot(top > m + kGrowth)) {
      const float mn = fmaxf(m, top), f = m == -INFINITY ? 0.0f : exp2_fast(m - mn);
      l *= f;
#pragma unroll
      for (int t = 0; t < D / 32; ++t) o[t] *= f;
      m = mn;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    u32x4 p[2 * KS][QP];
    float sum = 0;
#pragma unroll
    for (int j = 0; j < KS; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        float e[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          e[x] = exp2_fast(__builtin_fmaf(s[j][i + x], scale2, -ref));
          if constexpr (MASKED) e[x] = (see[j] >> (i + x)) & 1 ? e[x] : 0.0f;
          sum += e[x];
        }
        if constexpr (QP == 1) {
          p[2 * j + i / 8][0][(i % 8) / 2] = pack_bf16(e[0], e[1]);
        } else {
          uint32_t a[3], b[3];
          cut(__float_as_uint(e[0]), a);
          cut(__float_as_uint(e[1]), b);
#pragma unroll
          for (int c = 0; c < 3; ++c) p[2 * j + i / 8][c][(i % 8) / 2] = __builtin_amdgcn_perm(b[c], a[c], 0x07060302u);
        }
      }
    l += sum;
    if constexpr (MASKED) poison(lds, see, n, h);
#pragma unroll
    for (int ks = 0; ks < 2 * KS; ++ks)
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        u32x4 v = *reinterpret_cast<const u32x4*>(lds.v[ks][h][32 * t + n]);
        if constexpr (MASKED) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] &= ~whole16(not_finite16(v[i]));
        }
#pragma unroll
        for (int c = QP - 1; c >= 0; --c) o[t] = mfma32(v, p[ks][c], o[t]);
      }
  }

  // 0 times NaN is NaN: where a step has masks, values that are not finite count
  // as 0 in the product above, and rows that see one get NaN here.
  __device__ __forceinline__ void poison(const ManyLds<FMT, D>& lds, const uint32_t (&see)[KS], int n, int h) {
    uint32_t bad = 0;
#pragma unroll
    for (int w = 0; w < kManyWaves; ++w) bad |= lds.bad[w];
    if (__builtin_amdgcn_readfirstlane(bad) == 0) return;
#pragma unroll 1
    for (int ks = 0; ks < 2 * KS; ++ks) {
      const uint32_t mine = (ks < 2 ? see[0] : see[1]) >> (8 * (ks & 1));
      u32x4 vis;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        vis[i] = ((mine >> (2 * i)) & 1 ? 0x3F80u : 0u) | ((mine >> (2 * i)) & 2 ? 0x3F800000u : 0u);
#pragma unroll
      for (int t = 0; t < D / 32; ++t) {
        const u32x4 v = *reinterpret_cast<const u32x4*>(lds.v[ks][h][32 * t + n]);
        const u32x4 nf = {not_finite16(v[0]), not_finite16(v[1]), not_finite16(v[2]), not_finite16(v[3])};
        f32x16_t hit = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        hit = mfma32(nf, vis, hit);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[t][i] = hit[i] > 0.0f ? __builtin_nanf("") : o[t][i];
      }
    }
  }
};

// Waves of a SIMD that the registers leave room for: queries and sums take
// D / 4 and D / 2 registers of a bf16 call, 3 D / 4 and D / 2 of an fp32 one.
// Heads of 256 do not fit: fp32 spills 71 (E4M3) and 72 (E2M1) registers, and
// E4M3 keeps 272 bytes a lane in memory in bf16 calls too.  2 x 2048 queries over
// 4096 tokens, 8 heads of 256 x 4, take 0.60 ms in E2M1 bf16 and 1.25 in E4M3
// (fp32: 1.30 and 2.14).
constexpr int many_waves_simd(int dtype, int dim) { return dtype == NC_BF16 ? (dim <= 64 ? 3 : dim <= 128 ? 2 : 1) : (dim <= 64 ? 2 : 1); }

template <int FMT, int D, int DT>
__global__ void __launch_bounds__(64 * kManyWaves, many_waves_simd(DT, D)) kv_many(KvAttn a) {
  using L = Kv<FMT, D>;
  __shared__ __align__(16) ManyLds<FMT, D> lds[2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 31, h2 = lane >> 5;
  // workgroup -> head and sequence first (workgroups that follow each other go to different XCDs: a
  // head's rows then share one XCD's L2 when there are a multiple of 8), rows from the last ones,
  // which see the most keys with a causal mask
  //
  // Every other run of kKvUnits workgroups takes the sequences in reverse: the two workgroups of a
  // compute unit then have different lengths (8 x 448 queries over 187 .. 1500 tokens: 44 -> 39 us).
  const uint32_t all = (uint32_t)(a.batch * a.cache.heads), turn = blockIdx.x / all, bh = blockIdx.x - turn * all;
  const int rg = a.row_groups - 1 - (int)turn;
  uint32_t h;
  const int b0 = (int)a.cache.by_heads.quot(bh, h);
  const int b = (turn * all / kKvUnits) & 1 ? a.batch - 1 - b0 : b0;
  const KvSpan sp = kv_span(a, b);
  const int rows = sp.q_len * a.group, row0 = rg * kKvManyRows;
  if (row0 >= rows) return;
  const auto query = [&](int r) { return (int)a.by_group.quot((uint32_t)r); };
  const int i_lo = query(row0), i_hi = query(min(rows, row0 + kKvManyRows) - 1);
  const int any_end = kv_end(a, sp, i_hi), any_begin = kv_begin(a, kv_end(a, sp, i_lo));
  const int t0 = any_begin / 16, t1 = (any_end + 15) >> 4;

  // this wave's rows, and the keys that some of them see
  const int wrow = row0 + 32 * wave, r = wrow + n;
  const bool live = r < rows;
  const int i = live ? query(r) : 0, j = live ? r - i * a.group : 0;
  const int w_lo = query(min(wrow, rows - 1)), w_hi = query(min(rows, wrow + 32) - 1);
  const int w_any_end = wrow < rows ? kv_end(a, sp, w_hi) : 0, w_any_begin = kv_begin(a, kv_end(a, sp, w_lo));

  Many<FMT, D, DT> f;
  f.end = kv_end(a, sp, i);
  f.begin = kv_begin(a, f.end);
  f.m = -INFINITY;
  f.l = 0;
#pragma unroll
  for (int t = 0; t < D / 32; ++t)
#pragma unroll
    for (int e = 0; e < 16; ++e) f.o[t][e] = 0;
  // a negative scale is the negated query's
  const float scale2 = fabsf(a.scale2);
  const uint32_t flip = a.scale2 < 0 ? 0x80008000u : 0u;
  const int64_t at = (int64_t)(sp.q0 + i) * a.q.ts + (int64_t)((int)h * a.group + j) * a.q.hs;
#pragma unroll
  for (int st = 0; st < D / 16; ++st) {
    load_q<DT>(f.q[st], a.q.p, at + 16 * st + 8 * h2, live);
#pragma unroll
    for (int c = 0; c < Many<FMT, D, DT>::QP; ++c) f.q[st][c] ^= flip;
  }

  // Steps [0, ka) and [kb, steps) have masks for some row; those between have none: whole, seen by
  // every row, no page missing.
  const int tiles = max(t1 - t0, 0), steps = (tiles + 3) / 4;
  int ka = steps, kb = steps;
  {
    bool miss = false;
    for (int t = t0 + (int)threadIdx.x; t < t1; t += 64 * kManyWaves) miss = miss || kv_tile_at(a, b, (int)h, t) < 0;
    const int first = max(kv_begin(a, any_end) - 16 * t0, 0), last = min(kv_end(a, sp, i_lo) - 16 * t0, 16 * tiles);
    if (!__syncthreads_or(miss) && last > first) {
      ka = (first + kManyKeys - 1) / kManyKeys;
      kb = max(ka, last / kManyKeys);
    }
  }
  // Lane x looks up this wave's tile of step first + x, 64 steps at a time.
  int ids = -1;
  bool there = false;
  KvRegs<FMT, D> next;
  __shared__ uint32_t have[2][kManyWaves];
  auto look_up = [&](int k) {
    const int t = t0 + 4 * (k + lane) + wave;
    ids = t < t1 ? kv_tile_at(a, b, (int)h, t) : -1;
  };
  auto fetch = [&](int k) {                      // past the last step: the cache's first tile, unused
    const int tile = __builtin_amdgcn_readlane(ids, k & 63);
    there = tile >= 0;
    const uint8_t* p = a.cache.data + (int64_t)max(tile, 0) * L::TILE;
    load_keys<FMT, D>(next, p, lane & 15, lane >> 4);
    load_values<FMT, D>(next, p, lane & 15, lane >> 4);
  };
  auto put = [&](int k) {
    if (k >= ka && k < kb) {
      stage<FMT, D, false>(lds[k & 1], next, wave, lane, true, 16);
    } else {
      if (lane == 0) have[k & 1][wave] = there;
      stage<FMT, D, true>(lds[k & 1], next, wave, lane, there, sp.n - (t0 + 4 * k + wave) * 16);
    }
  };
  auto masked = [&](int k) {
    if (((k + 2) & 63) == 0) look_up(k + 2);
    __syncthreads();
    if (k + 1 < steps) put(k + 1);
    fetch(k + 2);
    const int base = (t0 + 4 * k) * 16;
    if (base >= w_any_end || w_any_begin - base >= kManyKeys) return;
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kManyWaves; ++w) all |= have[k & 1][w] ? 1u << w : 0u;
    f.template step<true>(lds[k & 1], base, __builtin_amdgcn_readfirstlane(all), scale2, lane);
  };
  if (steps > 0) {
    look_up(0);
    fetch(0);
    put(0);
    fetch(1);
    int k = 0;
    for (; k < ka; ++k) masked(k);
    for (; k + 1 < kb; ++k) {
      if (((k + 2) & 63) == 0) look_up(k + 2);
      __syncthreads();
      stage<FMT, D, false>(lds[(k + 1) & 1], next, wave, lane, true, 16);
      fetch(k + 2);
      f.template step<false>(lds[k & 1], 0, 0, scale2, lane);
    }
    if (k < kb) {                                // the last of them, before one that may have masks
      if (((k + 2) & 63) == 0) look_up(k + 2);
      __syncthreads();
      if (k + 1 < steps) put(k + 1);
      fetch(k + 2);
      f.template step<false>(lds[k & 1], 0, 0, scale2, lane);
      ++k;
    }
    for (; k < steps; ++k) masked(k);
  }

  // Results: of its row a lane holds, of every tile t of 32 elements, those with x = 8 e + 4 h2 + 0..3:
  // value lane x % 16, first or second of pair t as x / 16.
  const float l = add_halves(f.l);
  if (!live) return;
#pragma unroll
  for (int sg = 0; sg < L::NSEG; ++sg) {
    const int t = L::dim0(sg) / 32, dl = L::lane(sg);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = 8 * (e / 4) + 4 * h2 + e % 4;
      if (dl == 2) {                             // two lanes make four elements
        if (e % 2 == 0) {
          const f32x4_t o = {f.o[t][e], f.o[t][e + 8], f.o[t][e + 1], f.o[t][e + 9]};
          kv_result<DT>(a, sp, (int)h, r, L::dim0(sg) + 2 * c, o, f.m, l);
        }
      } else {
#pragma unroll
        for (int pp = 0; pp < dl / 4; ++pp) {
          const f32x4_t o = {f.o[t + 2 * pp][e], f.o[t + 2 * pp][e + 8], f.o[t + 2 * pp + 1][e], f.o[t + 2 * pp + 1][e + 8]};
          kv_result<DT>(a, sp, (int)h, r, L::dim0(sg) + dl * c + 4 * pp, o, f.m, l);
        }
      }
    }
  }
}

template <int FMT, int D, int DT>
hipError_t many_launch(const KvAttn& a, hipStream_t stream) {
  const int64_t grid = (int64_t)a.batch * a.cache.heads * a.row_groups;
  kv_many<FMT, D, DT><<<dim3((uint32_t)grid), dim3(64 * kManyWaves), 0, stream>>>(a);
  return hipGetLastError();
}

template <int FMT, int DT>
hipError_t many_by_dim(const KvAttn& a, int dim, hipStream_t stream) {
  switch (dim) {
    case 64: return many_launch<FMT, 64, DT>(a, stream);
    case 96: return many_launch<FMT, 96, DT>(a, stream);
    case 128: return many_launch<FMT, 128, DT>(a, stream);
    case 192: return many_launch<FMT, 192, DT>(a, stream);
    case 256: return many_launch<FMT, 256, DT>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace nc
