// Joining the partial results of attention chunks: out = sum_c 2^(m_c - m) o_c
// / sum_c 2^(m_c - m) l_c in a fixed order.  A workgroup takes one row; its
// threads are D / 4 columns of four elements times P lines of chunks, each
// line in one pass with a running maximum, the lines joined in LDS.
#include "nc_kv_few.h"

namespace nc {
namespace {

constexpr int kJoinThreads = 256;

template <int D, int DT>
__global__ void __launch_bounds__(kJoinThreads) kv_join(KvAttn a) {
  constexpr int COLS = D / 4, P = kJoinThreads / COLS;
  __shared__ __align__(16) float lds[P * (D + 2)];
  const int rows_all = a.max_q * a.group;
  const uint32_t r = blockIdx.x % (uint32_t)rows_all, bh = blockIdx.x / (uint32_t)rows_all;
  const int h = bh % a.cache.heads, b = bh / a.cache.heads;
  const KvSpan sp = kv_span(a, b);
  if ((int)r >= sp.q_len * a.group) return;
  const int col = threadIdx.x % COLS, line = threadIdx.x / COLS;
  const int64_t n = (int64_t)a.batch * a.cache.heads * a.chunks * rows_all;
  float top = -INFINITY, sum = 0;
  f32x4_t o = {0, 0, 0, 0};
  if (line < P) {
    for (int c = line; c < a.chunks; c += P) {
      const int64_t at = ((int64_t)bh * a.chunks + c) * rows_all + r;
      const float mc = a.part[n * D + at * 2], lc = a.part[n * D + at * 2 + 1];
      if (mc == -INFINITY && lc == 0.0f) continue;     // nothing seen there
      const f32x4_t oc = *reinterpret_cast<const f32x4_t*>(a.part + at * D + 4 * col);
      const float mn = fmaxf(top, mc), ref = mn == -INFINITY ? 0.0f : mn;
      const float x = exp2_fast(top - ref), y = exp2_fast(mc - ref);
      sum = sum * x + lc * y;
      o = o * x + oc * y;
      top = mn;
    }
    *reinterpret_cast<f32x4_t*>(lds + line * D + 4 * col) = o;
    if (col == 0) {
      lds[P * D + 2 * line] = top;
      lds[P * D + 2 * line + 1] = sum;
    }
  }
  __syncthreads();
  if (line != 0) return;
  top = -INFINITY;
#pragma unroll
  for (int i = 0; i < P; ++i) top = fmaxf(top, lds[P * D + 2 * i]);
  const float ref = top == -INFINITY ? 0.0f : top;
  sum = 0;
  o = f32x4_t{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const float x = exp2_fast(lds[P * D + 2 * i] - ref);
    sum += x * lds[P * D + 2 * i + 1];
    o += x * *reinterpret_cast<const f32x4_t*>(lds + i * D + 4 * col);
  }
  kv_result<DT>(a, sp, h, (int)r, 4 * col, o, top, sum);
}

template <int D>
hipError_t join(const KvAttn& a, int dtype, hipStream_t stream) {
  const dim3 grid((uint32_t)((int64_t)a.batch * a.cache.heads * a.max_q * a.group));
  if (dtype == NC_BF16) kv_join<D, NC_BF16><<<grid, dim3(kJoinThreads), 0, stream>>>(a);
  else kv_join<D, NC_F32><<<grid, dim3(kJoinThreads), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_join(const KvAttn& a, int dim, int dtype, hipStream_t stream) {
  switch (dim) {
    case 64: return join<64>(a, dtype, stream);
    case 96: return join<96>(a, dtype, stream);
    case 128: return join<128>(a, dtype, stream);
    case 192: return join<192>(a, dtype, stream);
    case 256: return join<256>(a, dtype, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace nc
