// Writing keys and values into the paged cache, and reading them back.
//
// Both move each byte once, so HBM bandwidth bounds them.  A lane takes eight
// elements of one row (16 bytes of bf16) -- a quarter of a block, so the
// block's largest magnitude is two lane exchanges away -- of the key and of
// the value.  Lanes run over the chunks of a row, then over sixteen consecutive
// tokens, then heads: when the tokens' slots follow each other, as in a prompt,
// a workgroup (256 lanes) moves whole tiles and no cache line of the cache is
// shared by workgroups on two XCDs.
#include "nc_kv.h"

namespace nc {
namespace {

// The block's scale byte from the bits of its largest finite magnitude.  For
// a normal a = m 2^e the byte is e + 127 - emax, one more for PLUS1, one more
// for CEIL when m is above the largest value's own significand.  Subnormal a
// and anything below gives 0 (X = -127).
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t a, int rule) {
  constexpr int EMAX = FMT == NC_E2M1 ? 2 : 8;
  constexpr uint32_t TOP = FMT == NC_E2M1 ? 0x400000u : 0x600000u;   // 1.5 and 1.75
  const int up = rule == NC_MX_PLUS1 ? 1 : (rule == NC_MX_CEIL && (a & 0x7FFFFFu) > TOP ? 1 : 0);
  const int b = (int)(a >> 23) - EMAX + up;
  return (uint32_t)(b < 0 ? 0 : b);
}

// Eight elements (fp32 bits) of a block that four lanes share -> codes; the
// block's scale byte in sb.  Infinities saturate.  E4M3 holds a NaN as 0x7F;
// E2M1 has none, so a block with one gets scale byte 255, which reads as NaN.
template <int FMT>
__device__ __forceinline__ u32x2 encode8(uint32_t (&x)[8], int rule, uint32_t& sb) {
  uint32_t a = 0;
  bool nf = false, nan = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t m = x[i] & kAbsMask;
    nf = nf || m > kMaxFinite;
    nan = nan || m > kInfBits;
    a = max(a, m > kMaxFinite ? 0u : m);
  }
  a = max(a, (uint32_t)__shfl_xor((int)a, 1));
  a = max(a, (uint32_t)__shfl_xor((int)a, 2));
  sb = scale_byte<FMT>(a, rule);
  const float s = kv_scale(sb);
  if constexpr (FMT == NC_E2M1) {
    // measured against the definition at every scale: round to nearest even, saturating
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x[0]), __uint_as_float(x[1]), s, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x[2]), __uint_as_float(x[3]), s, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x[4]), __uint_as_float(x[5]), s, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x[6]), __uint_as_float(x[7]), s, 3);
    uint32_t any = nan ? 1u : 0u;
    any |= (uint32_t)__shfl_xor((int)any, 1);
    any |= (uint32_t)__shfl_xor((int)any, 2);
    if (nf) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if ((x[i] & kAbsMask) > kMaxFinite) w = (w & ~(0xFu << (4 * i))) | ((7u | ((x[i] >> 28) & 8u)) << (4 * i));
    }
    if (any) sb = 255u;
    return u32x2{w, 0u};
  } else {
    const u32x4 lo = {x[0], x[1], x[2], x[3]}, hi = {x[4], x[5], x[6], x[7]};
    u32x2 w = {scvt4<NC_E4M3, NC_F32>(lo, 0, s), scvt4<NC_E4M3, NC_F32>(hi, 0, s)};
    if (nf) {
      w.x = fix_nonfinite4<NC_E4M3>(w.x, x);
      w.y = fix_nonfinite4<NC_E4M3>(w.y, x + 4);
    }
    return w;
  }
}

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t at, uint32_t (&x)[8]) {
  if constexpr (DT == NC_BF16) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = v[i] << 16;
      x[2 * i + 1] = v[i] & 0xFFFF0000u;
    }
  } else {
    const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const float*>(p) + at);
    const u32x4 a = q[0], b = q[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  }
}

// Where eight elements starting at e0 = 8 * chunk of a row lie in a tile.  All
// eight are in one segment (segments are multiples of 32 elements), in one
// key piece, and in 8 / lane(s) neighbouring value lanes.
template <int FMT, int D>
struct Place {
  using L = Kv<FMT, D>;
  int w, koff, voff, vstep;
  __device__ __forceinline__ Place(int e0, int tok) {
    constexpr int D4 = L::dim0(L::N4), D2 = L::dim0(L::N4 + L::N2);   // first elements past the 64- and 32-byte segments
    const int b0 = e0 / L::DPB;
    int s0;                                                          // byte the segment starts at
    if (e0 < D4) {
      w = 64;
      s0 = b0 & ~63;
    } else if (e0 < D2) {
      w = 32;
      s0 = 64 * L::N4;
    } else {
      w = 16;
      s0 = 64 * L::N4 + 32 * L::N2;
    }
    const int r = b0 - s0, pw = w / 4, wl = w / 16;
    koff = L::KC + 16 * s0 + ((r / pw) * 16 + tok) * pw + r % pw;
    voff = L::VC + 16 * s0 + (tok / 4) * 4 * w + (r / wl) * 4 * wl + (tok & 3) * wl;
    vstep = 4 * wl;
  }
};

// The bytes of eight elements to and from their places: keys are contiguous,
// values in runs of wl = 4, 2 or 1 bytes, vstep apart.
template <int FMT>
__device__ __forceinline__ void put_key(uint8_t* p, u32x2 c) {
  if constexpr (FMT == NC_E2M1) *reinterpret_cast<uint32_t*>(p) = c.x;
  else *reinterpret_cast<u32x2*>(p) = c;
}
template <int FMT>
__device__ __forceinline__ u32x2 get_key(const uint8_t* p) {
  if constexpr (FMT == NC_E2M1) return u32x2{*reinterpret_cast<const uint32_t*>(p), 0u};
  else return *reinterpret_cast<const u32x2*>(p);
}
template <int FMT>
__device__ __forceinline__ void put_value(uint8_t* p, int w, int step, u32x2 c) {
  if (w == 64) {
    *reinterpret_cast<uint32_t*>(p) = c.x;
    if constexpr (FMT == NC_E4M3) *reinterpret_cast<uint32_t*>(p + step) = c.y;
  } else if (w == 32) {
#pragma unroll
    for (int i = 0; i < (FMT == NC_E2M1 ? 2 : 4); ++i)
      *reinterpret_cast<uint16_t*>(p + i * step) = (uint16_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1)));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i * step] = (uint8_t)(c.x >> (8 * i));
  }
}
template <int FMT>
__device__ __forceinline__ u32x2 get_value(const uint8_t* p, int w, int step) {
  u32x2 c = {0u, 0u};
  if (w == 64) {
    c.x = *reinterpret_cast<const uint32_t*>(p);
    if constexpr (FMT == NC_E4M3) c.y = *reinterpret_cast<const uint32_t*>(p + step);
  } else if (w == 32) {
#pragma unroll
    for (int i = 0; i < (FMT == NC_E2M1 ? 2 : 4); ++i) {
      const uint32_t v = *reinterpret_cast<const uint16_t*>(p + i * step);
      if (i < 2) c.x |= v << (16 * (i & 1));
      else c.y |= v << (16 * (i & 1));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c.x |= (uint32_t)p[i * step] << (8 * i);
  }
  return c;
}

// Lane -> (token, head, chunk of eight elements); false past the end.  The
// caller's checks keep the count of lanes below 2^32.
template <int D>
__device__ __forceinline__ bool item(const KvCache& c, int64_t tokens, int64_t& token, int& head, int& chunk) {
  const uint32_t i = blockIdx.x * (uint32_t)kThreads + threadIdx.x;
  const uint32_t row = i / (D / 8);
  chunk = (int)(i % (D / 8));
  uint32_t h;
  const uint32_t run = c.by_heads.quot(row / kKvTokens, h);
  head = (int)h;
  token = (int64_t)run * kKvTokens + row % kKvTokens;
  return token < tokens;
}

// The tile and the token inside it of a slot; false for a slot outside the cache.
template <int FMT, int D>
__device__ __forceinline__ bool place_of(const KvCache& c, int64_t slot, int head, int64_t& base, int& tok) {
  if (slot < 0 || slot >= c.slots) return false;
  uint32_t tile;
  const uint32_t page = c.by_tiles.quot((uint32_t)slot / kKvTokens, tile);     // slots are below 2^31
  base = (int64_t)((page * (uint32_t)c.heads + (uint32_t)head) * c.by_tiles.d + tile) * Kv<FMT, D>::TILE;
  tok = (int)((uint32_t)slot % kKvTokens);
  return true;
}

template <int FMT, int D, int DT>
NC_STREAM_KERNEL kv_write(KvCache c, KvRows<const void*> k, KvRows<const void*> v, const int64_t* slots, int64_t tokens,
                          int rule) {
  using L = Kv<FMT, D>;
  int64_t token, base = 0;
  int head, chunk, tok = 0;
  // the four lanes of a block have the same token and head, so they leave together
  if (!item<D>(c, tokens, token, head, chunk)) return;
  if (!place_of<FMT, D>(c, slots[token], head, base, tok)) return;
  uint32_t xk[8], xv[8], sk, sv;
  load8<DT>(k.p, token * k.ts + head * k.hs + chunk * 8, xk);
  load8<DT>(v.p, token * v.ts + head * v.hs + chunk * 8, xv);
  const u32x2 ck = encode8<FMT>(xk, rule, sk), cv = encode8<FMT>(xv, rule, sv);
  const Place<FMT, D> at(8 * chunk, tok);
  uint8_t* t = c.data + base;
  put_key<FMT>(t + at.koff, ck);
  put_value<FMT>(t + at.voff, at.w, at.vstep, cv);
  if ((chunk & 3) == 0) {
    t[L::KS + (chunk >> 2) * 16 + tok] = (uint8_t)sk;
    t[L::VS + (chunk >> 2) * 16 + tok] = (uint8_t)sv;
  }
}

// The rows read are four times the codes: stored past the caches they leave them
// to the codes (131072 tokens of 8 heads of 128, E2M1 to bf16: 94 us against 142).
__device__ __forceinline__ void stream16(void* p, u32x4 v) { __builtin_nontemporal_store(v, static_cast<u32x4*>(p)); }

template <int FMT, int DT>
__device__ __forceinline__ void store8(void* p, int64_t at, u32x2 c, uint32_t sb) {
  const float s = kv_scale(sb);
  if constexpr (DT == NC_BF16) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = FMT == NC_E2M1 ? kv_pair<FMT>(c.x, s, i) : kv_pair<FMT>(i < 2 ? c.x : c.y, s, i & 1);
    stream16(static_cast<uint16_t*>(p) + at, r);
  } else {
    // a code's bf16 value at scale 2^0 (exact), times 2^X (exact in fp32, or rounded once in its
    // subnormal range); byte 255 is NaN
    float y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = FMT == NC_E2M1 ? kv_pair<FMT>(c.x, 1.0f, i) : kv_pair<FMT>(i < 2 ? c.x : c.y, 1.0f, i & 1);
      y[2 * i] = __builtin_amdgcn_ldexpf(__uint_as_float(r << 16), (int)sb - 127);
      y[2 * i + 1] = __builtin_amdgcn_ldexpf(__uint_as_float(r & 0xFFFF0000u), (int)sb - 127);
    }
    if (sb == 255u) {
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(0x7FC00000u);
    }
    u32x4* q = reinterpret_cast<u32x4*>(static_cast<float*>(p) + at);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      stream16(q + h, u32x4{__float_as_uint(y[4 * h]), __float_as_uint(y[4 * h + 1]), __float_as_uint(y[4 * h + 2]),
                            __float_as_uint(y[4 * h + 3])});
  }
}

template <int FMT, int D, int DT>
NC_STREAM_KERNEL kv_read(KvCache c, KvRows<void*> k, KvRows<void*> v, const int64_t* slots, int64_t tokens) {
  using L = Kv<FMT, D>;
  int64_t token, base = 0;
  int head, chunk, tok = 0;
  if (!item<D>(c, tokens, token, head, chunk)) return;
  u32x2 ck = {0u, 0u}, cv = {0u, 0u};
  uint32_t sk = 127u, sv = 127u;                 // a slot outside the cache reads as zeros
  if (place_of<FMT, D>(c, slots[token], head, base, tok)) {
    const Place<FMT, D> at(8 * chunk, tok);
    const uint8_t* t = c.data + base;
    ck = get_key<FMT>(t + at.koff);
    cv = get_value<FMT>(t + at.voff, at.w, at.vstep);
    sk = t[L::KS + (chunk >> 2) * 16 + tok];
    sv = t[L::VS + (chunk >> 2) * 16 + tok];
  }
  store8<FMT, DT>(k.p, token * k.ts + head * k.hs + chunk * 8, ck, sk);
  store8<FMT, DT>(v.p, token * v.ts + head * v.hs + chunk * 8, cv, sv);
}

int64_t grid_of(int64_t tokens, int heads, int dim) {
  return ((tokens + kKvTokens - 1) / kKvTokens * kKvTokens * heads * (dim / 8) + kThreads - 1) / kThreads;
}

// fn(FMT, D, DT) as compile-time values
template <int FMT, int D, typename Fn>
hipError_t by_dtype(int dtype, Fn fn) {
  return dtype == NC_BF16 ? fn.template operator()<FMT, D, NC_BF16>() : fn.template operator()<FMT, D, NC_F32>();
}
template <int FMT, typename Fn>
hipError_t by_dim(int dim, int dtype, Fn fn) {
  switch (dim) {
    case 64: return by_dtype<FMT, 64>(dtype, fn);
    case 96: return by_dtype<FMT, 96>(dtype, fn);
    case 128: return by_dtype<FMT, 128>(dtype, fn);
    case 192: return by_dtype<FMT, 192>(dtype, fn);
    case 256: return by_dtype<FMT, 256>(dtype, fn);
  }
  return hipErrorInvalidValue;
}
template <typename Fn>
hipError_t by_all(int fmt, int dim, int dtype, Fn fn) {
  return fmt == NC_E2M1 ? by_dim<NC_E2M1>(dim, dtype, fn) : by_dim<NC_E4M3>(dim, dtype, fn);
}

struct Write {
  const KvCache& c;
  const KvRows<const void*>&k, &v;
  const int64_t* slots;
  int64_t tokens;
  int rule;
  int64_t grid;
  hipStream_t stream;
  template <int FMT, int D, int DT> hipError_t operator()() const {
    kv_write<FMT, D, DT><<<dim3((uint32_t)grid), dim3(kThreads), 0, stream>>>(c, k, v, slots, tokens, rule);
    return hipGetLastError();
  }
};
struct Read {
  const KvCache& c;
  const KvRows<void*>&k, &v;
  const int64_t* slots;
  int64_t tokens, grid;
  hipStream_t stream;
  template <int FMT, int D, int DT> hipError_t operator()() const {
    kv_read<FMT, D, DT><<<dim3((uint32_t)grid), dim3(kThreads), 0, stream>>>(c, k, v, slots, tokens);
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_kv_write(const KvCache& c, int fmt, int dim, const KvRows<const void*>& k, const KvRows<const void*>& v,
                           int dtype, const int64_t* slots, int64_t tokens, int rule, hipStream_t stream) {
  return by_all(fmt, dim, dtype, Write{c, k, v, slots, tokens, rule, grid_of(tokens, c.heads, dim), stream});
}

hipError_t launch_kv_read(const KvCache& c, int fmt, int dim, const KvRows<void*>& k, const KvRows<void*>& v, int dtype,
                          const int64_t* slots, int64_t tokens, hipStream_t stream) {
  return by_all(fmt, dim, dtype, Read{c, k, v, slots, tokens, grid_of(tokens, c.heads, dim), stream});
}

}  // namespace nc
