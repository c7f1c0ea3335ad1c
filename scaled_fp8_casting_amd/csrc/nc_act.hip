// Activations that keep their inputs as MX blocks, and their gradients from what
// was kept.
//
//   forward:  y = f(gate) up;  gate and up quantised
//   backward: dgate = dy up f'(gate), dup = dy f(gate), and y again where wanted,
//             with gate and up as they were kept
//
// f: silu z s(z) with s(z) = 1 / (1 + e^-z); gelu z Phi(z); gelu_tanh
// z s(2 c (z + 0.044715 z^3)), c = sqrt(2 / pi) (0.5 (1 + tanh u) = s(2 u));
// relu2 max(z, 0)^2.  Derivatives: s + z s (1 - s); Phi + z phi(z); s + z s (1 - s)
// 2 c (1 + 3 * 0.044715 z^2); 2 max(z, 0).  All in fp32; z = -inf gives NaN where
// the formula does (-inf times 0).
//
// Each byte moves once, so HBM bandwidth bounds them: gated silu over 8192 x 11008 bf16
// kept in E4M3 129 us forward (5.7 TB/s), 159 us backward with y again (5.7).
#include <cfloat>
#include <type_traits>

#include "nc_mx.h"

namespace nc {
namespace {

// z cut to [-most, most]: where a factor next to it is 0 already, infinities and
// overflows would make NaN of the product.
__device__ __forceinline__ float within(float z, float most) { return fminf(fmaxf(z, -most), most); }
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

template <int ACT> __device__ __forceinline__ void act_of(float z, float& f, float& df) {
  if constexpr (ACT == NC_ACT_SILU) {
    const float s = sigmoid(z);
    f = z * s;
    df = s * (1.0f + within(z, FLT_MAX) * (1.0f - s));
  } else if constexpr (ACT == NC_ACT_GELU) {
    const float phi = 0.5f * erfcf(z * -0.70710678118654752f);
    f = z * phi;
    df = phi + within(z, FLT_MAX) * (expf(-0.5f * z * z) * 0.39894228040143268f);
  } else if constexpr (ACT == NC_ACT_GELU_TANH) {
    constexpr float c2 = 1.5957691216057308f, k = 0.044715f;   // 2 sqrt(2 / pi)
    const float n = within(z, 16.0f);            // s is 0 or 1 from there on
    const float s = z == z ? sigmoid(c2 * (n + k * n * n * n)) : z;
    f = z * s;
    df = s + n * s * (1.0f - s) * (c2 * (1.0f + 3.0f * k * n * n));
  } else {
    const float r = z > 0.0f ? z : (z != z ? z : 0.0f);
    f = r * r;
    df = 2.0f * r;
  }
}

// What was kept, as fp32.  Blocks of fp32's largest values (a mask's lowest ones) may round
// up to 2^128, which is finite but past fp32: it counts as fp32's largest number, one
// rounding away, so that a factor of 0 next to it gives 0.
template <int FMT> __device__ __forceinline__ void kept8(u32x2 c, uint32_t sb, float (&y)[8]) {
  constexpr uint32_t EMAX = FMT == NC_E2M1 ? 2 : FMT == NC_E4M3 ? 8 : 15;
  decode8<FMT>(c, sb, y);
  if (sb + EMAX >= 255u) {                       // 2^EMAX 2^(sb - 127) is past fp32
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((__float_as_uint(y[i]) & kAbsMask) == kInfBits) y[i] = copysignf(FLT_MAX, y[i]);
  }
}

template <int DT> __device__ __forceinline__ void floats(const Eight<DT>& x, float (&y)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(bits_of<DT>(x, i));
}
template <int DT> __device__ __forceinline__ const uint8_t* row_of(const Plane<const void*>& x, int64_t row) {
  return static_cast<const uint8_t*>(x.p) + row * x.stride * In<DT>::BYTES;
}
template <int DT> __device__ __forceinline__ uint8_t* row_of(const Plane<void*>& x, int64_t row) {
  return static_cast<uint8_t*>(x.p) + row * x.stride * In<DT>::BYTES;
}

// STEPS: how many of a chunk's four steps a workgroup takes.  One where there would be
// few workgroups of four: a thread's elements follow each other, and their functions
// are long.  In us, with four and with one: gelu over 1001 x 1365 fp32 9.5 and 7.2,
// gelu_tanh's gradient over 100 x 4096 7.1 and 3.6; over rows of 4096 columns, gated, E4M3,
// replayed from a graph:
//   chunks                  512         1024         2048         4096         8192        16384
//   silu    bf16       13.6 12.7    20.5 19.2    32.6 30.6    57.4 57.1   104.3 109.5  197.2 218.6
//   gelu    bf16       16.2 14.8    25.3 23.2    39.7 38.0    72.7 72.0   131.6 138.9  255.1 269.8
//   relu2   bf16       11.2 10.8    17.7 18.0    29.1 31.9    53.7 59.6   102.1 115.1  196.0 228.7
//   gelu    fp32       19.1 16.7    30.3 27.7    52.5 51.3    93.9 96.9   175.9 188.5  346.0 376.9
//   gradient, y again:
//   silu    bf16       15.0 12.6    21.5 21.8    37.2 36.6    66.8 72.0   127.8 139.6  249.8 276.2
//   gelu    bf16       17.8 15.4    26.9 25.5    41.5 43.1    78.0 80.6   147.9 156.1  282.7 304.0
//   relu2   bf16       12.2 13.0    21.2 20.9    34.3 35.9    64.8 70.3   124.0 137.8  251.6 274.0
// One number for all: relu2 would gain 3 us at 2048 chunks from four, silu loses 2.
template <int STEPS> struct ActPart {
  int s0;
  MxLane at;
  __device__ __forceinline__ explicit ActPart(const MxMat& m) : s0(STEPS == 4 ? 0 : (int)(blockIdx.x & 3)), at(m, STEPS == 4 ? blockIdx.x : blockIdx.x >> 2) {}
  __device__ __forceinline__ void put_scales(const MxMat& m, uint32_t scales) const {
    if ((at.q & 3) != 0) return;
    if constexpr (STEPS == 4) *reinterpret_cast<uint32_t*>(m.scales + at.scales()) = scales;
    else m.scales[at.scales() + s0] = (uint8_t)scales;
  }
  __device__ __forceinline__ uint32_t get_scales(const MxMat& m) const {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(m.scales + at.scales());
    return STEPS == 4 ? w : w >> (8 * s0);
  }
};

template <int ACT, int FMT, int DT, bool GATED, int STEPS>
NC_STREAM_KERNEL act_forward(ActForward a) {
  const ActPart<STEPS> part(a.gate_q);
  const MxLane& at = part.at;
  const int s0 = part.s0;
  const bool there = at.row < a.gate_q.rows;
  Eight<DT> g[STEPS], u[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t left = there ? a.gate_q.cols - at.col(s0 + s) : 0;
    g[s] = load8<DT>(row_of<DT>(a.gate, at.row), at.col(s0 + s), left);
    if constexpr (GATED) u[s] = load8<DT>(row_of<DT>(a.up, at.row), at.col(s0 + s), left);
  }
  if (a.gate_q.codes != nullptr) {
    uint32_t sg = 0, su = 0;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
      uint32_t sb;
      put_codes<FMT>(a.gate_q.codes + at.codes<FMT>(s0 + s), encode_quad<FMT, DT>(g[s], a.rule, sb));
      sg |= sb << (8 * s);
      if constexpr (GATED) {
        put_codes<FMT>(a.up_q.codes + at.codes<FMT>(s0 + s), encode_quad<FMT, DT>(u[s], a.rule, sb));
        su |= sb << (8 * s);
      }
    }
    part.put_scales(a.gate_q, sg);
    if constexpr (GATED) part.put_scales(a.up_q, su);
  }
  if (!there) return;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    float z[8], w[8], y[8];
    floats<DT>(g[s], z);
    if constexpr (GATED) floats<DT>(u[s], w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, df;
      act_of<ACT>(z[i], f, df);
      y[i] = GATED ? f * w[i] : f;
    }
    store8<DT>(row_of<DT>(a.y, at.row), at.col(s0 + s), a.gate_q.cols - at.col(s0 + s), eight_of<DT>(y), a.stream);
  }
}

template <int ACT, int FMT, int DT, bool GATED, int STEPS>
NC_STREAM_KERNEL act_backward(ActBackward a) {
  const ActPart<STEPS> part(a.gate_q);
  const MxLane& at = part.at;
  const int s0 = part.s0;
  if (at.row >= a.gate_q.rows) return;
  Eight<DT> dy[STEPS];
  u32x2 g[STEPS], u[STEPS];
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    dy[s] = load8<DT>(row_of<DT>(a.dy, at.row), at.col(s0 + s), a.gate_q.cols - at.col(s0 + s));
    g[s] = get_codes<FMT>(a.gate_q.codes + at.codes<FMT>(s0 + s));
    if constexpr (GATED) u[s] = get_codes<FMT>(a.up_q.codes + at.codes<FMT>(s0 + s));
  }
  const uint32_t sg = part.get_scales(a.gate_q);
  uint32_t su = 0;
  if constexpr (GATED) su = part.get_scales(a.up_q);
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int64_t col = at.col(s0 + s), left = a.gate_q.cols - col;
    float d[8], z[8], w[8], dz[8], dw[8], y[8];
    floats<DT>(dy[s], d);
    kept8<FMT>(g[s], (sg >> (8 * s)) & 255u, z);
    if constexpr (GATED) kept8<FMT>(u[s], (su >> (8 * s)) & 255u, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f, df;
      act_of<ACT>(z[i], f, df);
      dz[i] = d[i] * (GATED ? w[i] * df : df);   // w df first: d w may pass fp32 where df is 0 or small
      dw[i] = d[i] * f;
      y[i] = GATED ? f * w[i] : f;
    }
    store8<DT>(row_of<DT>(a.dgate, at.row), col, left, eight_of<DT>(dz), a.stream);
    if constexpr (GATED) store8<DT>(row_of<DT>(a.dup, at.row), col, left, eight_of<DT>(dw), a.stream);
    if (a.y.p != nullptr) store8<DT>(row_of<DT>(a.y, at.row), col, left, eight_of<DT>(y), a.stream);
  }
}

template <int ACT, int FMT, typename Fn> hipError_t by_dtype(int dtype, Fn fn) {
  return dtype == NC_BF16 ? fn.template operator()<ACT, FMT, NC_BF16>() : fn.template operator()<ACT, FMT, NC_F32>();
}
template <int ACT, typename Fn> hipError_t by_format(int fmt, int dtype, Fn fn) {
  return fmt == NC_E2M1 ? by_dtype<ACT, NC_E2M1>(dtype, fn)
       : fmt == NC_E4M3 ? by_dtype<ACT, NC_E4M3>(dtype, fn) : by_dtype<ACT, NC_E5M2>(dtype, fn);
}
template <typename Fn> hipError_t by_act(int act, int fmt, int dtype, Fn fn) {
  switch (act) {
    case NC_ACT_SILU: return by_format<NC_ACT_SILU>(fmt, dtype, fn);
    case NC_ACT_GELU: return by_format<NC_ACT_GELU>(fmt, dtype, fn);
    case NC_ACT_GELU_TANH: return by_format<NC_ACT_GELU_TANH>(fmt, dtype, fn);
    case NC_ACT_RELU2: return by_format<NC_ACT_RELU2>(fmt, dtype, fn);
  }
  return hipErrorInvalidValue;
}

constexpr uint32_t kFewChunks = 4096;              // measured above

// fn(steps of a workgroup as a constant, workgroups)
template <typename Fn> void by_steps(const MxMat& m, Fn fn) {
  const uint32_t chunks = (uint32_t)m.strips * (uint32_t)m.chunks;
  if (chunks < kFewChunks) fn(std::integral_constant<int, 1>{}, dim3(4 * chunks));
  else fn(std::integral_constant<int, 4>{}, dim3(chunks));
}

struct Forward {
  ActForward a;
  hipStream_t stream;
  template <int ACT, int FMT, int DT> hipError_t operator()() {
    a.stream = mx_streams<DT>(a.y, a.gate_q.rows, a.gate_q.cols);
    by_steps(a.gate_q, [&](auto steps, dim3 grid) {
      if (a.up.p != nullptr) act_forward<ACT, FMT, DT, true, decltype(steps)::value><<<grid, dim3(kThreads), 0, stream>>>(a);
      else act_forward<ACT, FMT, DT, false, decltype(steps)::value><<<grid, dim3(kThreads), 0, stream>>>(a);
    });
    return hipGetLastError();
  }
};
struct Backward {
  ActBackward a;
  hipStream_t stream;
  template <int ACT, int FMT, int DT> hipError_t operator()() {
    const int64_t rows = a.gate_q.rows, cols = a.gate_q.cols;
    a.stream = mx_streams<DT>(a.dgate, rows, cols) && (a.dup.p == nullptr || mx_streams<DT>(a.dup, rows, cols)) &&
               (a.y.p == nullptr || mx_streams<DT>(a.y, rows, cols));
    by_steps(a.gate_q, [&](auto steps, dim3 grid) {
      if (a.up_q.codes != nullptr) act_backward<ACT, FMT, DT, true, decltype(steps)::value><<<grid, dim3(kThreads), 0, stream>>>(a);
      else act_backward<ACT, FMT, DT, false, decltype(steps)::value><<<grid, dim3(kThreads), 0, stream>>>(a);
    });
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_act_forward(const ActForward& a, int act, int fmt, int dtype, hipStream_t stream) {
  return by_act(act, fmt, dtype, Forward{a, stream});
}
hipError_t launch_act_backward(const ActBackward& a, int act, int fmt, int dtype, hipStream_t stream) {
  return by_act(act, fmt, dtype, Backward{a, stream});
}

}  // namespace nc
