// Writing matrices of MX blocks and reading them back.
//
// Both move each byte once, so HBM bandwidth bounds them: 8192 x 11008 bf16 to E4M3 55
// us (4.9 TB/s) and back 45.5 (6.0), 8192 x 4096 both ways 29 us (4.7).
#include "nc_mx.h"

namespace nc {
namespace {

// Rows only: no exchange but the block's maximum, which lies in four lanes.
template <int FMT, int DT>
NC_STREAM_KERNEL mx_write_rows(MxMat m, Plane<const void*> x, int rule) {
  const MxLane at(m);
  const bool there = at.row < m.rows;
  const uint8_t* row = static_cast<const uint8_t*>(x.p) + at.row * x.stride * In<DT>::BYTES;
  Eight<DT> v[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) v[s] = load8<DT>(row, at.col(s), there ? m.cols - at.col(s) : 0);
  uint32_t scales = 0;
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    uint32_t sb;
    const u32x2 c = encode_quad<FMT, DT>(v[s], rule, sb);
    put_codes<FMT>(m.codes + at.codes<FMT>(s), c);
    scales |= sb << (8 * s);
  }
  if ((at.q & 3) == 0) *reinterpret_cast<uint32_t*>(m.scales + at.scales()) = scales;
}

// Columns, and rows of the same read: a workgroup takes 64 rows (one step of the
// transposed matrix) by 256 columns (a chunk of the rows' matrix) through LDS.
// Two rounds of 32 rows are read as in mx_write_rows and left in LDS; then each
// thread has one column, whose two blocks of 32 rows it reads down, and writes 16
// bytes a piece: 512 in a run.  Four workgroups share the lines of the transposed
// scales (a byte of each dword): they follow each other on one XCD.
template <int FMT, int DT>
NC_STREAM_KERNEL mx_write_both(MxMat m, MxMat t, Plane<const void*> x, int rule) {
  constexpr int N = DT == NC_BF16 ? 4 : 8;
  __shared__ uint32_t tile[64][kMxChunk * In<DT>::BYTES / 4];
  const int64_t rows = t.cols, cols = t.rows;
  const uint32_t across = (uint32_t)((cols + kMxChunk - 1) / kMxChunk);
  // blocks b, b + 8, b + 16, b + 24 (one XCD) are the four steps of a chunk of t
  const uint32_t unit = blockIdx.x / 32 * 8 + blockIdx.x % 8;
  const uint32_t chunk = unit / across, band = unit % across;
  const int step = (int)(blockIdx.x / 8 % 4);
  if (chunk >= (uint32_t)t.chunks) return;
  const int64_t row0 = (int64_t)chunk * kMxChunk + kMxStep * step, col0 = (int64_t)band * kMxChunk;
  const int r = (int)(threadIdx.x >> 3), q = (int)(threadIdx.x & 7);
  Eight<DT> x8[2][4];                            // all on the way before the first is used
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = row0 + 32 * h + r;
    const uint8_t* p = static_cast<const uint8_t*>(x.p) + row * x.stride * In<DT>::BYTES;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t c = col0 + kMxStep * s + 8 * q;
      x8[h][s] = load8<DT>(p, c, row < rows ? cols - c : 0);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t row = row0 + 32 * h + r;
    const Eight<DT>(&v)[4] = x8[h];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < N; ++i) tile[32 * h + r][(kMxStep * s + 8 * q) * In<DT>::BYTES / 4 + i] = v[s].w[i];
    if (m.codes != nullptr && row / kMxRows < m.strips) {
      const int64_t at = row / kMxRows * m.chunks + band;
      uint32_t scales = 0;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t sb;
        const u32x2 c = encode_quad<FMT, DT>(v[s], rule, sb);
        const int k = kMxStep * s + 8 * q;
        put_codes<FMT>(m.codes + at * mx_chunk_bytes(FMT) + mx_piece<FMT>(r, k) + (FMT == NC_E2M1 ? 4 * (q & 3) : 8 * (q & 1)), c);
        scales |= sb << (8 * s);
      }
      if ((q & 3) == 0) *reinterpret_cast<uint32_t*>(m.scales + at * kMxScaleBytes + (r + 32 * (q >> 2)) * 4) = scales;
    }
  }
  __syncthreads();
  const int c = (int)threadIdx.x;
  const int64_t strip = col0 / kMxRows + c / kMxRows;
  if (strip >= t.strips) return;
  const int64_t at = strip * t.chunks + chunk;
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    Eight<DT> v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int k = 32 * b + 8 * e + i * 8 / N;
        if constexpr (DT == NC_BF16) {
          const uint16_t* lo = reinterpret_cast<const uint16_t*>(tile[k]) + c;
          const uint16_t* hi = reinterpret_cast<const uint16_t*>(tile[k + 1]) + c;
          v[e].w[i] = (uint32_t)*lo | (uint32_t)*hi << 16;
        } else {
          v[e].w[i] = tile[k][c];
        }
      }
    uint32_t a = 0, odd[4], any = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a = max(a, amax8<DT>(v[e], odd[e]));
      any |= odd[e];
    }
    uint32_t sb = mx_scale_byte<FMT>(a, rule);
    u32x2 w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = encode8<FMT, DT>(v[e], sb, odd[e]);
    if (FMT == NC_E2M1 && (any & 2u)) sb = 255u;
    uint8_t* codes = t.codes + at * mx_chunk_bytes(FMT);
    const int k = kMxStep * step + 32 * b;
    if constexpr (FMT == NC_E2M1) {
      *reinterpret_cast<u32x4*>(codes + mx_piece<FMT>(c % kMxRows, k)) = u32x4{w[0].x, w[1].x, w[2].x, w[3].x};
    } else {
      *reinterpret_cast<u32x4*>(codes + mx_piece<FMT>(c % kMxRows, k)) = u32x4{w[0].x, w[0].y, w[1].x, w[1].y};
      *reinterpret_cast<u32x4*>(codes + mx_piece<FMT>(c % kMxRows, k + 16)) = u32x4{w[2].x, w[2].y, w[3].x, w[3].y};
    }
    t.scales[at * kMxScaleBytes + (c % kMxRows + 32 * b) * 4 + step] = (uint8_t)sb;
  }
}

template <int FMT, int DT>
NC_STREAM_KERNEL mx_read(MxMat m, Plane<void*> y, bool stream) {
  const MxLane at(m);
  if (at.row >= m.rows) return;
  uint8_t* row = static_cast<uint8_t*>(y.p) + at.row * y.stride * In<DT>::BYTES;
  u32x2 c[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) c[s] = get_codes<FMT>(m.codes + at.codes<FMT>(s));
  const uint32_t scales = *reinterpret_cast<const uint32_t*>(m.scales + at.scales());
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const uint32_t sb = (scales >> (8 * s)) & 255u;
    Eight<DT> v;
    if constexpr (DT == NC_BF16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v.w[i] = mx_pair<FMT>(c[s], mx_scale(sb), i);
    } else {
      float f[8];
      decode8<FMT>(c[s], sb, f);
      v = eight_of<DT>(f);
    }
    store8<DT>(row, at.col(s), m.cols - at.col(s), v, stream);
  }
}

// fn<FMT, DT>()
template <int FMT, typename Fn> hipError_t by_dtype(int dtype, Fn fn) {
  return dtype == NC_BF16 ? fn.template operator()<FMT, NC_BF16>() : fn.template operator()<FMT, NC_F32>();
}
template <typename Fn> hipError_t by_format(int fmt, int dtype, Fn fn) {
  return fmt == NC_E2M1 ? by_dtype<NC_E2M1>(dtype, fn) : fmt == NC_E4M3 ? by_dtype<NC_E4M3>(dtype, fn) : by_dtype<NC_E5M2>(dtype, fn);
}

struct WriteRows {
  const MxMat& m;
  const Plane<const void*>& x;
  int rule;
  hipStream_t stream;
  template <int FMT, int DT> hipError_t operator()() const {
    mx_write_rows<FMT, DT><<<dim3((uint32_t)m.strips * (uint32_t)m.chunks), dim3(kThreads), 0, stream>>>(m, x, rule);
    return hipGetLastError();
  }
};
struct WriteBoth {
  const MxMat &m, &t;
  const Plane<const void*>& x;
  int rule;
  hipStream_t stream;
  template <int FMT, int DT> hipError_t operator()() const {
    const uint32_t units = (uint32_t)t.chunks * (uint32_t)((t.rows + kMxChunk - 1) / kMxChunk);
    mx_write_both<FMT, DT><<<dim3((units + 7) / 8 * 32), dim3(kThreads), 0, stream>>>(m, t, x, rule);
    return hipGetLastError();
  }
};
struct Read {
  const MxMat& m;
  const Plane<void*>& y;
  hipStream_t stream;
  template <int FMT, int DT> hipError_t operator()() const {
    mx_read<FMT, DT><<<dim3((uint32_t)m.strips * (uint32_t)m.chunks), dim3(kThreads), 0, stream>>>(m, y, mx_streams<DT>(y, m.rows, m.cols));
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_mx_write(const MxMat* m, const MxMat* t, int fmt, const Plane<const void*>& x, int dtype, int rule,
                           hipStream_t stream) {
  if (t == nullptr) return by_format(fmt, dtype, WriteRows{*m, x, rule, stream});
  const MxMat none = {};
  return by_format(fmt, dtype, WriteBoth{m != nullptr ? *m : none, *t, x, rule, stream});
}

hipError_t launch_mx_read(const MxMat& m, int fmt, const Plane<void*>& y, int dtype, hipStream_t stream) {
  return by_format(fmt, dtype, Read{m, y, stream});
}

}  // namespace nc
