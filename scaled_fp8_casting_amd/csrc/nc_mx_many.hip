// The many-row product by its operands' formats, and the join of its splits.
#include "nc_mx_many.h"

namespace nc {
namespace {

// Sums the splits' parts in their order, four results a thread.
NC_STREAM_KERNEL mx_join(MxProduct p) {
  const int64_t rows = p.a.rows, cols = p.b.rows, across = (cols + 3) / 4;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = i / across, col = i % across * 4;
  if (row >= rows) return;
  const int64_t left = cols - col;
  float y[4] = {0, 0, 0, 0};
  for (int32_t s = 0; s < p.splits; ++s) {
    const float* q = p.part + ((int64_t)s * rows + row) * cols + col;
    if (left >= 4) {
      float v[4];
      __builtin_memcpy(v, q, 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] += v[e];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) y[e] += q[e];
    }
  }
  MxStore<4>(p, col)(row, y);
}

}  // namespace

hipError_t launch_mx_many(const MxProduct& p, int fa, int fb, int w, hipStream_t stream) {
  const hipError_t e = fa == NC_E2M1 ? mx_many_e2m1(p, fb, w, stream) : fa == NC_E4M3 ? mx_many_e4m3(p, fb, w, stream) : mx_many_e5m2(p, fb, w, stream);
  if (e != hipSuccess || p.splits == 1) return e;
  const int64_t threads = p.a.rows * ((p.b.rows + 3) / 4);
  mx_join<<<dim3((uint32_t)((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace nc
