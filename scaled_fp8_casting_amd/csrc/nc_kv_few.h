// Attention over the paged cache for few rows: the next tokens of running
// sequences, and prompts too small to fill the card with the many-row kernel.
//
// Row r = (query i, head j of the group) of a sequence and a cache head; key
// t is seen when start(i) <= t < end(i).  With s = scale log2(e) q.k, m the
// running maximum of a row and l the running sum of 2^(s - m),
//   out = (sum_t 2^(s_t - m) v_t) / l,   lse = (m + log2 l) ln 2,
// in one pass over the cache: a new maximum m' multiplies what is there by
// 2^(m - m').  A row that sees nothing has l = 0: out = 0, lse = -inf.
//
// What bounds it is the cache's bytes, so nothing but registers lies between
// memory and the matrix instructions.  A wave takes 16 NT rows and runs over
// tiles of 16 tokens:
//
//   S^T = K Q^T   16x16x32 bf16: lane (key m, group g of k) loads its own key's
//                 codes (one load per tile and segment), converts them with
//                 their block's scale to bf16 -- exactly, a code has at most 4
//                 significant bits -- and multiplies
//   softmax       a lane has query n = lane % 16 and keys 4 g + i, so maximum and
//                 sum run over registers, then over the four groups
//   O^T = V^T P^T the weights are in place as operand: k index 8 g + e stands for
//                 key 4 g + e of the first tile (e < 4) or the second; the lane
//                 (m, g) loads quad g of both value tiles
//
// fp32 queries and weights are cut into three bf16 parts of 8 significant bits,
// exactly; products and sums are fp32.  bf16 calls round the weights to bf16
// (by 2^-8 at most, as their output is) and sum them before the rounding: one
// product with the values instead of the three of fp32 calls.  Against the
// definition the results are then 1.69e-3 of their size apart where weights kept
// whole would leave the output's own rounding, 1.66e-3 (517 tokens; 262144:
// 1.644e-3 and 1.643e-3).
//
// The waves of a workgroup take turns along the keys, two tiles at a time;
// their sums meet in LDS.  Long caches are cut over the workgroups, in shares
// that are equal however unequal the lengths are, and their sums meet in a
// second kernel.
//
// Measured, the same cache at every call, so that up to 256 MB of it may come
// from the last-level cache: the next token of one sequence, 262144 tokens of 8
// heads of 128 in E2M1 (285 MB), 51 us and 6.6 us for the second kernel; 64
// sequences of 1024 .. 8192 tokens 70 and 7 us (331 MB), where the waves wait at
// every change of sequence.  On caches that change from call to call both take
// 64 and 78 us with the launches (4.5 and 4.3 TB/s; a large copy reaches 5.1,
// reads alone 7.0).  517 tokens take 7.5 us, of which 5.6 are
// there for 32 tokens already (dependent loads: lengths, table, codes).  Wider
// steps (four tiles, 170 registers and more) left one wave a SIMD: 110 us.  The
// second kernel as the last workgroup's task needs a device-wide release from
// each of them, and took 88 and 185 us.
#pragma once

#include "nc_kv.h"

namespace nc {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ f32x4_t mfma16(const u32x4& a, const u32x4& b, const f32x4_t& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Maximum and sum over the lanes l, l ^ 32 and over l, l ^ 16, l ^ 32, l ^ 48:
// a swap of half waves (or of rows of 16 lanes) of two copies puts both
// partners' values into every lane.
__device__ __forceinline__ void swap_halves(float x, float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ void swap_rows(float x, float& a, float& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  a = __uint_as_float(r[0]);
  b = __uint_as_float(r[1]);
}
__device__ __forceinline__ float max_halves(float x) {
  float a, b;
  swap_halves(x, a, b);
  return fmaxf(a, b);
}
__device__ __forceinline__ float add_halves(float x) {
  float a, b;
  swap_halves(x, a, b);
  return a + b;
}
__device__ __forceinline__ float max_groups(float x) {
  float a, b;
  swap_rows(x, a, b);
  return max_halves(fmaxf(a, b));
}
__device__ __forceinline__ float add_groups(float x) {
  float a, b;
  swap_rows(x, a, b);
  return add_halves(a + b);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Two floats -> packed bf16, nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

// The keys of one sequence that a workgroup's rows see.
struct KvSpan {
  int n, q_len, q0;        // cached tokens, queries, first query's row in q
};
__device__ __forceinline__ KvSpan kv_span(const KvAttn& a, int b) {
  KvSpan s;
  const int64_t held = (int64_t)a.table_w * a.cache.page;
  int n = a.kv_len[b];
  n = min(max(n, 0), a.max_kv);
  s.n = held < n ? (int)held : n;
  // offsets outside q give an empty sequence, never an access outside q
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1];
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.total_q;
  s.q0 = ok ? q0 : 0;
  s.q_len = ok ? min(q1 - q0, a.max_q) : 0;
  return s;
}
// Query i sees keys [kv_begin, kv_end).
__device__ __forceinline__ int kv_end(const KvAttn& a, const KvSpan& s, int i) {
  return a.causal ? min(s.n, s.n - s.q_len + 1 + i) : s.n;
}
// max(0, end - window), without a difference that 32 bits do not hold: end may be as low as 1 - max_q.
__device__ __forceinline__ int kv_begin(const KvAttn& a, int end) { return a.window ? max(end, a.window) - a.window : 0; }

// The number of the tile (page, head, tile of the page) that holds tokens
// [16 t, 16 t + 16) of sequence b, or -1 for a page outside the cache.
__device__ __forceinline__ int kv_tile_at(const KvAttn& a, int b, int h, int t) {
  const uint32_t per = a.cache.by_tiles.d;
  uint32_t in;
  const uint32_t pg = a.cache.by_tiles.quot((uint32_t)t, in);
  if (pg >= (uint32_t)a.table_w) return -1;
  const int32_t id = a.table[(int64_t)b * a.table_w + pg];
  if (id < 0 || (int64_t)id * a.cache.page >= a.cache.slots) return -1;
  return (int)(((uint32_t)id * (uint32_t)a.cache.heads + (uint32_t)h) * per + in);
}

// Four elements of a row's result, from its sums.
template <int DT>
__device__ __forceinline__ void kv_result(const KvAttn& a, const KvSpan& sp, int h, int r, int c, const f32x4_t& o, float top,
                                          float sum) {
  uint32_t j;
  const int i = (int)a.by_group.quot((uint32_t)r, j), head = h * a.group + (int)j;
  const int64_t row = sp.q0 + i;
  const float x = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int64_t at = row * a.out.ts + head * a.out.hs + c;
  if constexpr (DT == NC_BF16)
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.out.p) + at) =
        u32x2{pack_bf16(o[0] * x, o[1] * x), pack_bf16(o[2] * x, o[3] * x)};
  else
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out.p) + at) = o * x;
  if (a.lse != nullptr && c == 0) a.lse[row * a.lse_ts + head] = (top + log2f(sum)) * kLn2;
}

template <int FMT, int D> struct KvRegs {      // one tile's codes and scales in a lane
  using L = Kv<FMT, D>;
  uint32_t k[L::DW], v[L::DW];
  uint32_t ks[L::NSEG], vs[L::NSEG];
};

template <int N>
__device__ __forceinline__ void load_dwords(uint32_t* r, const uint8_t* p) {
  if constexpr (N == 4) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = v[i];
  } else if constexpr (N == 2) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    r[0] = v.x;
    r[1] = v.y;
  } else {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

template <int FMT, int D, int S = 0>
__device__ __forceinline__ void load_keys(KvRegs<FMT, D>& r, const uint8_t* t, int m, int g) {
  using L = Kv<FMT, D>;
  if constexpr (S < L::NSEG) {
    constexpr int w = L::w(S), off = L::off(S), n = w / 16;
    load_dwords<n>(r.k + off / 16, t + L::KC + 16 * off + (g * 16 + m) * (w / 4));
    r.ks[S] = t[L::KS + ((L::dim0(S) + g * L::piece(S)) / 32) * 16 + m];
    load_keys<FMT, D, S + 1>(r, t, m, g);
  }
}
template <int FMT, int D, int S = 0>
__device__ __forceinline__ void load_values(KvRegs<FMT, D>& r, const uint8_t* t, int m, int g) {
  using L = Kv<FMT, D>;
  if constexpr (S < L::NSEG) {
    constexpr int w = L::w(S), off = L::off(S), n = w / 16;
    load_dwords<n>(r.v + off / 16, t + L::VC + 16 * off + (g * 16 + m) * (w / 4));
    r.vs[S] = *reinterpret_cast<const uint32_t*>(t + L::VS + ((L::dim0(S) + m * L::lane(S)) / 32) * 16 + 4 * g);
    load_values<FMT, D, S + 1>(r, t, m, g);
  }
}

// A float as three bf16 numbers, in the high halves: 8 significant bits are cut
// off at a time, so every part and remainder is exact.
__device__ __forceinline__ void cut(uint32_t x, uint32_t (&part)[3]) {
  part[0] = x;
  part[1] = __float_as_uint(__uint_as_float(x) - __uint_as_float(x & 0xFFFF0000u));
  part[2] = __float_as_uint(__uint_as_float(part[1]) - __uint_as_float(part[1] & 0xFFFF0000u));
}

// Queries as operands: rows of 16 lanes n, k step j of a segment: the eight
// elements that a key piece has there.
template <int DT> struct QParts { static constexpr int N = DT == NC_BF16 ? 1 : 3; };
template <int DT>
__device__ __forceinline__ void load_q(u32x4* q, const void* p, int64_t at, bool live) {
  if constexpr (DT == NC_BF16) {
    q[0] = live ? *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at) : u32x4{0, 0, 0, 0};
  } else {
    u32x4 x[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (live) {
      const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + at);
      x[0] = s[0];
      x[1] = s[1];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t a[3], b[3];
      cut(x[i >> 1][2 * (i & 1)], a);
      cut(x[i >> 1][2 * (i & 1) + 1], b);
#pragma unroll
      for (int c = 0; c < 3; ++c) q[c][i] = __builtin_amdgcn_perm(b[c], a[c], 0x07060302u);
    }
  }
}

// Halves lo (0) or hi (1) of two packed pairs.
__device__ __forceinline__ uint32_t zip(uint32_t a, uint32_t b, int hi) {
  return hi ? __builtin_amdgcn_perm(b, a, 0x07060302u) : __builtin_amdgcn_perm(b, a, 0x05040100u);
}

// Packed bf16: 1.0 in the halves that hold an infinity or NaN, and a mask of
// the halves that are not zero.
__device__ __forceinline__ uint32_t not_finite16(uint32_t x) {
  return ((x & 0x7F80u) == 0x7F80u ? 0x3F80u : 0u) | ((x & 0x7F800000u) == 0x7F800000u ? 0x3F800000u : 0u);
}
__device__ __forceinline__ uint32_t whole16(uint32_t x) {
  return (x & 0xFFFFu ? 0xFFFFu : 0u) | (x & 0xFFFF0000u ? 0xFFFF0000u : 0u);
}

// The running reference m of a row follows its maximum only when that has
// grown by more than 2^8: weights then stay below 2^8 and the sums are
// rescaled a few times per call instead of at every new maximum.
constexpr float kGrowth = 8.0f;

constexpr int kFewTiles = 2;                     // tiles of 16 keys that a wave takes at a time

template <int FMT, int D, int DT, int NT> struct Few {
  using L = Kv<FMT, D>;
  static constexpr int QP = QParts<DT>::N;       // parts of a query, and of a weight
  static constexpr int KT = kFewTiles;
  static constexpr int MT = D / 16;              // output tiles of 16 elements

  u32x4 q[NT][D / 32][QP];
  f32x4_t o[NT][MT];
  f32x4_t s[NT][KT];                             // scores
  u32x4 p[NT][QP];                               // weights
  float m[NT], l[NT];                            // reference; sum of this lane's keys
  int end[NT], begin[NT];                        // keys that the lane's row sees

  __device__ __forceinline__ void scores(const KvRegs<FMT, D> (&r)[KT]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < KT; ++j) s[t][j] = f32x4_t{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < KT; ++j)
#pragma unroll
      for (int sg = 0; sg < L::NSEG; ++sg) {
        const float sc = kv_scale(r[j].ks[sg]);
        constexpr int DWS = 4 * L::BITS / 16;    // dwords of eight codes
#pragma unroll
        for (int st = 0; st < L::piece(sg) / 8; ++st) {
          const uint32_t* c = r[j].k + L::off(sg) / 16 + st * DWS;
          u32x4 a;
#pragma unroll
          for (int i = 0; i < 4; ++i) a[i] = kv_pair<FMT>(c[i * DWS / 4], sc, i % (4 / DWS));
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c2 = QP - 1; c2 >= 0; --c2) s[t][j] = mfma16(a, q[t][L::dim0(sg) / 32 + st][c2], s[t][j]);
        }
      }
  }

  // Scores of keys that a row does not see, or of a tile that is missing (bit of `there` off): -inf.
  __device__ __forceinline__ void mask(int base, uint32_t there, int g) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < KT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = base + 16 * j + 4 * g + i;
          s[t][j][i] = key < end[t] && key >= begin[t] && ((there >> j) & 1) ? s[t][j][i] : -INFINITY;
        }
  }

  __device__ __forceinline__ void weights(float scale2) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < KT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][j][i]);
      top = max_groups(top) * scale2;
      if (__ballot(top > m[t] + kGrowth)) {
        const float mn = fmaxf(m[t], top), f = m[t] == -INFINITY ? 0.0f : exp2_fast(m[t] - mn);
        l[t] *= f;
#pragma unroll
        for (int d = 0; d < MT; ++d) o[t][d] *= f;
        m[t] = mn;
      }
      const float ref = m[t] == -INFINITY ? 0.0f : m[t];
      float sum = 0;
#pragma unroll
      for (int j = 0; j < KT; ++j) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          e[i] = exp2_fast(__builtin_fmaf(s[t][j][i], scale2, -ref));
          sum += e[i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if constexpr (QP == 1) {
            p[t][0][2 * j + i] = pack_bf16(e[2 * i], e[2 * i + 1]);
          } else {
            uint32_t x[3], y[3];
            cut(__float_as_uint(e[2 * i]), x);
            cut(__float_as_uint(e[2 * i + 1]), y);
#pragma unroll
            for (int c = 0; c < 3; ++c) p[t][c][2 * j + i] = __builtin_amdgcn_perm(y[c], x[c], 0x07060302u);
          }
        }
      }
      l[t] += sum;
    }
  }

  // Tokens past the end, or of a tile that is missing, hold anything: codes and scales cleared.
  // Whether what is left may hold a value that is not finite (a NaN code or scale, or a scale near
  // the top of bf16's range).
  static __device__ __forceinline__ bool clear(KvRegs<FMT, D> (&r)[KT], int base, uint32_t there, int n_keys, int g) {
    uint32_t odd = 0;
#pragma unroll
    for (int x = 0; x < KT; ++x) {
      const int left = (there >> x) & 1 ? n_keys - (base + 16 * x + 4 * g) : 0;      // tokens of the quad
      const uint32_t keep = left >= 4 ? ~0u : left <= 0 ? 0u : ~0u >> (32 - 8 * left);
#pragma unroll
      for (int sg = 0; sg < L::NSEG; ++sg) {
        const int n = L::w(sg) / 16;             // bytes of a token, dwords of the quad
        r[x].vs[sg] &= keep;
        // a scale byte of 240 or more: (byte & 0x7F) + 16 carries into bit 7 of bytes that have it
        odd |= r[x].vs[sg] & ((r[x].vs[sg] & 0x7F7F7F7Fu) + 0x10101010u) & 0x80808080u;
#pragma unroll
        for (int d = 0; d < n; ++d) {
          uint32_t& c = r[x].v[L::off(sg) / 16 + d];
          if (n == 4) c = left > d ? c : 0u;
          else if (n == 2) c &= left >= 2 * d + 2 ? ~0u : left == 2 * d + 1 ? 0xFFFFu : 0u;
          else c &= keep;
          if constexpr (FMT == NC_E4M3) odd |= ((c & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
        }
      }
    }
    return __ballot(odd != 0) != 0;
  }

  template <bool BY_ROW>
  __device__ __forceinline__ void values_of(const KvRegs<FMT, D> (&r)[KT], int base, uint32_t there, int n_keys, int g) {
    uint32_t keep[4];                            // tokens past the end hold anything: cleared
    if constexpr (BY_ROW) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = i / 2, key = base + 16 * j + 4 * g + 2 * (i & 1);
        const bool on = (there >> j) & 1;
        keep[i] = (on && key < n_keys ? 0xFFFFu : 0u) | (on && key + 1 < n_keys ? 0xFFFF0000u : 0u);
      }
    }
#pragma unroll
    for (int sg = 0; sg < L::NSEG; ++sg) {
      constexpr int P4 = 2 * L::DPB;             // pairs of a dword
      const int pairs = L::lane(sg) / 2;         // pairs of a lane and token
      float sc[KT][4];
#pragma unroll
      for (int x = 0; x < KT; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[x][i] = kv_scale((r[x].vs[sg] >> (8 * i)) & 255u);
#pragma unroll
      for (int pr = 0; pr < pairs; ++pr) {
        u32x4 v[2];
#pragma unroll
        for (int x = 0; x < KT; ++x) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int at = i * pairs + pr;       // the pair's place in the lane's codes
            w[i] = kv_pair<FMT>(r[x].v[L::off(sg) / 16 + at / P4], sc[x][i], at % P4);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v[h][2 * x] = zip(w[0], w[1], h);
            v[h][2 * x + 1] = zip(w[2], w[3], h);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = L::dim0(sg) / 16 + 2 * pr + h;
          if constexpr (BY_ROW) {
            u32x4 nf;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              v[h][i] &= keep[i];
              nf[i] = not_finite16(v[h][i]);
            }
            // 0 times NaN is NaN: a value that is not finite must reach the rows that see it only.
            // It counts as 0 here, and rows whose seen keys hold one get NaN.
            if (__ballot((nf[0] | nf[1] | nf[2] | nf[3]) != 0)) {
#pragma unroll
              for (int i = 0; i < 4; ++i) v[h][i] &= ~whole16(nf[i]);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                u32x4 vis;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int key = base + 16 * (i / 2) + 4 * g + 2 * (i & 1);
                  vis[i] = (key >= begin[t] && key < end[t] ? 0x3F80u : 0u) |
                           (key + 1 >= begin[t] && key + 1 < end[t] ? 0x3F800000u : 0u);
                }
                const f32x4_t hit = mfma16(nf, vis, f32x4_t{0, 0, 0, 0});
#pragma unroll
                for (int i = 0; i < 4; ++i) o[t][d][i] = hit[i] > 0.0f ? __builtin_nanf("") : o[t][d][i];
              }
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = QP - 1; c >= 0; --c) o[t][d] = mfma16(v[h], p[t][c], o[t][d]);
        }
      }
    }
  }

  __device__ __forceinline__ void values(const KvRegs<FMT, D> (&r)[KT]) {
    values_of<false>(r, 0, 0, 0, 0);
  }
  __device__ __forceinline__ void values_by_row(const KvRegs<FMT, D> (&r)[KT], int base, uint32_t there, int n_keys, int g) {
    values_of<true>(r, base, there, n_keys, g);
  }
};

// Where a workgroup's sums of a row go: the call's result, or a place among the
// partial results (D sums; maximum and sum in a list behind all of them).
template <int DT>
__device__ __forceinline__ void kv_store(const KvAttn& a, const KvSpan& sp, int h, int r, int dim, int c, const f32x4_t& o,
                                         float top, float sum, int64_t place, int64_t places) {
  if (place < 0) {
    kv_result<DT>(a, sp, h, r, c, o, top, sum);
    return;
  }
  *reinterpret_cast<f32x4_t*>(a.part + place * dim + c) = o;
  if (c == 0) {
    float* ml = a.part + places * dim + place * 2;
    ml[0] = top;
    ml[1] = sum;
  }
}

// ---- how the few-row kernel's work is shared out ----------------------------
// A segment is one (sequence, head, row group); its length is the tiles of 16
// keys that the sequence's rows reach, at least 1.  Lengths live on the device,
// so each workgroup works them out: all segments lie one after the other on a
// line, and workgroup w takes the tiles [w share, (w + 1) share) of it.  Every
// sequence has the row groups of max_q queries: groups past its own queries take
// up line but no time, so the work of the shares is equal where the sequences
// have about as many queries each (lengths may differ), and not where they differ
// (one sequence of 64 queries among 31 single tokens, 8192 tokens each, 8 heads
// of 128 x 4, E2M1: 261 us, and 84 as two calls).  Whole segments inside a share are finished there;
// the one that began before it goes to partial place 2 w, the one that goes on
// behind it to place 2 w + 1.
struct KvReach {
  KvSpan sp;
  int t0, tiles;       // first tile, tiles of a segment (0: no queries)
};
__device__ __forceinline__ KvReach kv_reach(const KvAttn& a, int b) {
  KvReach r;
  r.sp = kv_span(a, b);
  const int end = kv_end(a, r.sp, r.sp.q_len - 1);
  r.t0 = kv_begin(a, kv_end(a, r.sp, 0)) / 16;
  r.tiles = r.sp.q_len > 0 ? max(1, (end + 15) / 16 - r.t0) : 0;
  return r;
}
// The same for a sequence that is the whole wave's.
__device__ __forceinline__ KvReach kv_reach_wave(const KvAttn& a, int b) {
  const KvReach r = kv_reach(a, b);
  const auto u = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  return KvReach{{u(r.sp.n), u(r.sp.q_len), u(r.sp.q0)}, u(r.t0), u(r.tiles)};
}
__device__ __forceinline__ uint32_t scan64(uint32_t x, int lane) {   // inclusive sum over the wave
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t y = __shfl_up(x, d);
    x += lane >= d ? y : 0u;
  }
  return x;
}
// Tiles of all segments.
__device__ __forceinline__ uint32_t kv_line(const KvAttn& a, int lane) {
  uint32_t sum = 0;
  for (int b = lane; b < a.batch; b += 64) sum += (uint32_t)kv_reach(a, b).tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  return __builtin_amdgcn_readfirstlane(sum) * (uint32_t)(a.cache.heads * a.row_groups);
}
// The sequence that holds tile x of the line, and where on the line it begins.
__device__ __forceinline__ int kv_find(const KvAttn& a, uint32_t x, int lane, uint32_t& start, KvReach& at) {
  const uint32_t per = (uint32_t)(a.cache.heads * a.row_groups);
  uint32_t before = 0;
  for (int b = 0; b < a.batch; b += 64) {
    KvReach r = kv_reach(a, min(b + lane, a.batch - 1));
    const uint32_t n = b + lane < a.batch ? (uint32_t)r.tiles * per : 0u, to = before + scan64(n, lane);
    const uint64_t past = __ballot(to > x);
    if (past) {
      const int i = __builtin_ctzll(past);
      const auto of = [&](int v) { return __builtin_amdgcn_readlane(v, i); };
      start = of(to - n);
      at = KvReach{{of(r.sp.n), of(r.sp.q_len), of(r.sp.q0)}, of(r.t0), of(r.tiles)};
      return b + i;
    }
    before = __builtin_amdgcn_readlane(to, 63);
  }
  return a.batch;                                // not reached: x is inside the line
}
__device__ __forceinline__ uint32_t kv_share(const KvAttn& a, uint32_t line) {
  const uint32_t n = (line + (uint32_t)a.shares - 1) / (uint32_t)a.shares;
  return max((n + 7) & ~7u, (uint32_t)kKvShareLeast);
}

// One segment's tiles [t0, t1): the workgroup's sums into the result (place < 0)
// or a partial place.
template <int FMT, int D, int DT, int NT, int WAVES>
__device__ __forceinline__ void few_segment(const KvAttn& a, const KvSpan& sp, int b, int h, int rg, int t0, int t1, int place,
                                            float* lds) {
  using L = Kv<FMT, D>;
  using F = Few<FMT, D, DT, NT>;
  constexpr int KT = F::KT;
  const int64_t places = 2 * (int64_t)a.shares * 16 * NT;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int rows = sp.q_len * a.group, row0 = rg * 16 * NT;
  if (row0 >= rows) return;
  const int i_lo = (int)a.by_group.quot((uint32_t)row0), i_hi = (int)a.by_group.quot((uint32_t)(min(rows, row0 + 16 * NT) - 1));
  // keys that some row sees, and keys that every row sees
  const int any_end = kv_end(a, sp, i_hi), all_end = kv_end(a, sp, i_lo), all_begin = kv_begin(a, any_end);
  t0 = max(t0, kv_begin(a, all_end) / 16);
  t1 = min(t1, (any_end + 15) >> 4);

  // a negative scale is the negated query's
  const float scale2 = fabsf(a.scale2);
  const uint32_t flip = a.scale2 < 0 ? 0x80008000u : 0u;
  F f;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = row0 + 16 * t + m;
    const bool live = r < rows;
    uint32_t j;
    const int i = (int)a.by_group.quot(live ? (uint32_t)r : 0u, j);
    f.end[t] = kv_end(a, sp, i);
    f.begin[t] = kv_begin(a, f.end[t]);
    f.m[t] = -INFINITY;
    f.l[t] = 0;
#pragma unroll
    for (int d = 0; d < F::MT; ++d) f.o[t][d] = f32x4_t{0, 0, 0, 0};
    const int64_t at = (int64_t)(sp.q0 + i) * a.q.ts + (int64_t)(h * a.group + (int)j) * a.q.hs;
#pragma unroll
    for (int sg = 0; sg < L::NSEG; ++sg)
#pragma unroll
      for (int st = 0; st < L::piece(sg) / 8; ++st)
        load_q<DT>(f.q[t][L::dim0(sg) / 32 + st], a.q.p, at + L::dim0(sg) + g * L::piece(sg) + 8 * st, live);
#pragma unroll
    for (int st = 0; st < D / 32; ++st)
#pragma unroll
      for (int c = 0; c < F::QP; ++c) f.q[t][st][c] ^= flip;
  }

  // Steps of KT tiles, the waves in turn, 64 / KT steps at a time: lane i looks up the i-th tile
  // that the wave takes in them.  A step's keys and values are loaded as soon as the step before has
  // used its own; with masks or without, the code is the same but for the masking itself (a copy of
  // it for the last step of a sequence took 0.8 us more: it was fetched for that step alone).
  constexpr int STRIDE = KT * WAVES, BATCH = 64 / KT;
  const int w0 = t0 + wave * KT;                 // the wave's first tile
  const int steps = w0 < t1 ? (t1 - w0 + STRIDE - 1) / STRIDE : 0;
  for (int k0 = 0; k0 < steps; k0 += BATCH) {
    const int n = min(steps - k0, BATCH);
    const int t = w0 + (k0 + lane / KT) * STRIDE + lane % KT;
    const bool mine = lane < n * KT && t < t1;
    const int ids = mine ? kv_tile_at(a, b, h, t) : -1;
    // steps without masks: [ka, kb), if no page is missing
    const int at0 = 16 * (w0 + k0 * STRIDE);
    const int ka = all_begin > at0 ? (all_begin - at0 + 16 * STRIDE - 1) / (16 * STRIDE) : 0;
    const int whole = __ballot(mine && ids < 0) ? 0 : min(all_end, 16 * t1);
    const int kb = whole - at0 >= 16 * KT ? (whole - at0 - 16 * KT) / (16 * STRIDE) + 1 : 0;
    KvRegs<FMT, D> r[KT];
    auto tile = [&](int k, int j) {
      // a tile that is missing, or past the last step: some tile of the cache, masked or unused
      return a.cache.data + (int64_t)max(__builtin_amdgcn_readlane(ids, (k * KT + j) & 63), 0) * L::TILE;
    };
    auto keys = [&](int k) {
#pragma unroll
      for (int j = 0; j < KT; ++j) load_keys<FMT, D>(r[j], tile(k, j), m, g);
    };
    auto vals = [&](int k) {
#pragma unroll
      for (int j = 0; j < KT; ++j) load_values<FMT, D>(r[j], tile(k, j), m, g);
    };
    int base = 0;
    uint32_t there = 0;
    for (int k = 0;; ++k) {
      keys(k);
      vals(k);
      for (; k < n; ++k) {
        const bool masked = k < ka || k >= kb;
        f.scores(r);
        keys(k + 1);
        if (masked) {
          base = at0 + 16 * STRIDE * k;
          there = 0;
#pragma unroll
          for (int j = 0; j < KT; ++j) there |= __builtin_amdgcn_readlane(ids, k * KT + j) >= 0 ? 1u << j : 0u;
          f.mask(base, there, g);
        }
        f.weights(scale2);
        if (masked && F::clear(r, base, there, sp.n, g)) break;
        f.values(r);
        vals(k + 1);
      }
      if (k >= n) break;
      f.values_by_row(r, base, there, sp.n, g);  // rare: a value that is not finite and not seen by every row
    }
  }

  // Join the waves: factors from the maxima, sums one row tile at a time.
  float* ml = lds + WAVES * 16 * (D + 4);        // [wave][row][2]
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float l = add_groups(f.l[t]);
    if (g == 0) {
      ml[(wave * NT * 16 + t * 16 + m) * 2] = f.m[t];
      ml[(wave * NT * 16 + t * 16 + m) * 2 + 1] = l;
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    __syncthreads();
    float* mine_o = lds + (wave * 16 + m) * (D + 4);
#pragma unroll
    for (int sg = 0; sg < L::NSEG; ++sg)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int pr = 0; pr < L::lane(sg) / 2; ++pr) {
          const int d = L::dim0(sg) / 16 + 2 * pr;
          float* to = mine_o + L::dim0(sg) + (4 * g + i) * L::lane(sg) + 2 * pr;
          to[0] = f.o[t][d][i];
          to[1] = f.o[t][d + 1][i];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 16 * D / 4; e += 64 * WAVES) {
      const int rr = e / (D / 4), c = e % (D / 4) * 4, r = row0 + 16 * t + rr;
      if (r >= rows) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) top = fmaxf(top, ml[(w * NT * 16 + t * 16 + rr) * 2]);
      const float ref = top == -INFINITY ? 0.0f : top;
      float sum = 0;
      f32x4_t o = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        const float x = exp2_fast(ml[(w * NT * 16 + t * 16 + rr) * 2] - ref);
        sum += x * ml[(w * NT * 16 + t * 16 + rr) * 2 + 1];
        o += x * *reinterpret_cast<const f32x4_t*>(lds + (w * 16 + rr) * (D + 4) + c);
      }
      kv_store<DT>(a, sp, h, r, D, c, o, top, sum, place < 0 ? place : place * (16 * NT) + 16 * t + rr, places);
    }
  }
}


template <int FMT, int D, int DT, int NT, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, kv_few_waves(DT, D, NT)) kv_few(KvAttn a) {
  // one row tile's sums of every wave, then every row's maximum and sum
  __shared__ __align__(16) float lds[WAVES * 16 * (D + 4) + WAVES * 16 * NT * 2];
  const uint32_t per = (uint32_t)(a.cache.heads * a.row_groups);
  uint32_t x, to, start = 0, seg;                // tiles [x, to) of the line; segment seg of sequence b begins at start
  int b;
  KvReach r;
  if (a.shares == 0) {                           // a workgroup for each segment
    b = (int)a.by_segments.quot(blockIdx.x, seg);
    r = kv_reach_wave(a, b);
    x = 0;
    to = (uint32_t)r.tiles;
    if (to == 0) return;
  } else {
    const int lane = threadIdx.x & 63;
    const uint32_t line = kv_line(a, lane), share = kv_share(a, line);
    x = blockIdx.x * share;
    to = min(line, x + share);
    if (x >= to) return;
    b = kv_find(a, x, lane, start, r);
    seg = (x - start) / (uint32_t)r.tiles;
    start += seg * (uint32_t)r.tiles;
  }
  for (;;) {
    const uint32_t end = start + (uint32_t)r.tiles, stop = min(end, to);
    uint32_t rg;
    const int h = (int)a.by_row_groups.quot(seg, rg);
    const int place = x == start && stop == end ? -1 : 2 * (int)blockIdx.x + (x == start ? 1 : 0);
    few_segment<FMT, D, DT, NT, WAVES>(a, r.sp, b, h, (int)rg, r.t0 + (int)(x - start), r.t0 + (int)(stop - start), place, lds);
    x = start = stop;
    if (x >= to) return;
    if (++seg == per) {
      seg = 0;
      do {                                       // x is inside the line, so there is another sequence
        if (++b >= a.batch) return;
        r = kv_reach_wave(a, b);
      } while (r.tiles == 0);
    }
    __syncthreads();                             // before the sums in LDS are overwritten
  }
}

template <int FMT, int D, int DT, int NT, int WAVES>
hipError_t few_launch(const KvAttn& a, hipStream_t stream) {
  const int64_t grid = a.shares > 0 ? a.shares : (int64_t)a.batch * a.cache.heads * a.row_groups;
  kv_few<FMT, D, DT, NT, WAVES><<<dim3((uint32_t)grid), dim3(64 * WAVES), 0, stream>>>(a);
  return hipGetLastError();
}

template <int FMT, int D, int DT>
hipError_t few_by_rows(const KvAttn& a, const KvPlan& p, hipStream_t stream) {
  if constexpr (kv_few_waves(DT, D, 1) >= 2)
    if (p.rows == 16 && p.shares == 0) return few_launch<FMT, D, DT, 1, 2 * kKvFewWaves>(a, stream);
  if (p.rows == 16) return few_launch<FMT, D, DT, 1, kKvFewWaves>(a, stream);
  if constexpr (kv_few_rows(DT, D) == 32)
    if (p.rows == 32) return few_launch<FMT, D, DT, 2, kKvFewWaves>(a, stream);
  return hipErrorInvalidValue;
}

template <int FMT, int DT>
hipError_t few_by_dim(const KvAttn& a, int dim, const KvPlan& p, hipStream_t stream) {
  switch (dim) {
    case 64: return few_by_rows<FMT, 64, DT>(a, p, stream);
    case 96: return few_by_rows<FMT, 96, DT>(a, p, stream);
    case 128: return few_by_rows<FMT, 128, DT>(a, p, stream);
    case 192: return few_by_rows<FMT, 192, DT>(a, p, stream);
    case 256: return few_by_rows<FMT, 256, DT>(a, p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace nc
