// Joining partial results: out = sum_c 2^(m_c - m) o_c / sum_c 2^(m_c - m) l_c
// in a fixed order.  A workgroup takes one row; its threads are D / 4 columns
// of four elements times P lines of partial results, the lines joined in LDS.
#include "nc_kv_few.h"

namespace nc {
namespace {

constexpr int kJoinThreads = 256;

// Places first, first + 1 * step, ... of a row, n of them; `head` is the first
// place (it may lie off the run).
struct KvParts {
  int64_t head, first, step, places;
  int n;
};

template <int D, int DT>
__device__ __forceinline__ void join_row(const KvAttn& a, const KvSpan& sp, int h, int r, const KvParts& p) {
  constexpr int COLS = D / 4, P = kJoinThreads / COLS;
  __shared__ __align__(16) float lds[P * (D + 2)];
  const int col = threadIdx.x % COLS, line = threadIdx.x / COLS;
  const float* ml = a.part + p.places * D;
  float top = -INFINITY, sum = 0;
  f32x4_t o = {0, 0, 0, 0};
  if (line < P) {
#pragma unroll 4
    for (int c = line; c < p.n; c += P) {
      const int64_t at = c == 0 ? p.head : p.first + (c - 1) * p.step;
      const float mc = ml[at * 2], lc = ml[at * 2 + 1];
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
  const int lines = min(P, p.n);
  top = -INFINITY;
  for (int i = 0; i < lines; ++i) top = fmaxf(top, lds[P * D + 2 * i]);
  const float ref = top == -INFINITY ? 0.0f : top;
  sum = 0;
  o = f32x4_t{0, 0, 0, 0};
  for (int i = 0; i < lines; ++i) {
    const float x = exp2_fast(lds[P * D + 2 * i] - ref);
    sum += x * lds[P * D + 2 * i + 1];
    o += x * *reinterpret_cast<const f32x4_t*>(lds + i * D + 4 * col);
  }
  kv_result<DT>(a, sp, h, r, 4 * col, o, top, sum);
}

// A row of every segment; those that lie in one share are finished already.
template <int D, int DT>
__global__ void __launch_bounds__(kJoinThreads) kv_join(KvAttn a, int rows) {
  const int rows_all = a.max_q * a.group, lane = threadIdx.x & 63;
  const int r = (int)(blockIdx.x % (uint32_t)rows_all);
  const uint32_t bh = blockIdx.x / (uint32_t)rows_all;
  uint32_t head;
  const int b = (int)a.cache.by_heads.quot(bh, head), h = (int)head;
  const KvReach reach = kv_reach(a, b);
  if (r >= reach.sp.q_len * a.group) return;
  // where the segment lies on the line
  uint32_t all = 0, before = 0;
  for (int i = lane; i < a.batch; i += 64) {
    const uint32_t n = (uint32_t)kv_reach(a, i).tiles;
    all += n;
    before += i < b ? n : 0u;
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    all += __shfl_xor(all, d);
    before += __shfl_xor(before, d);
  }
  const uint32_t per = (uint32_t)(a.cache.heads * a.row_groups);
  const uint32_t share = kv_share(a, all * per);
  const uint32_t start = before * per + ((uint32_t)h * a.row_groups + (uint32_t)(r / rows)) * (uint32_t)reach.tiles;
  const uint32_t g0 = start / share, g1 = (start + (uint32_t)reach.tiles - 1) / share;
  if (g0 == g1) return;
  KvParts p;
  p.places = 2 * (int64_t)a.shares * rows;
  p.head = (int64_t)(2 * g0 + 1) * rows + r % rows;
  p.step = 2 * rows;
  p.first = (int64_t)(2 * g0 + 2) * rows + r % rows;
  p.n = (int)(g1 - g0) + 1;
  join_row<D, DT>(a, reach.sp, h, r, p);
}

template <int D, int DT>
hipError_t join(const KvAttn& a, const KvPlan& p, hipStream_t stream) {
  const dim3 grid((uint32_t)((int64_t)a.batch * a.cache.heads * a.max_q * a.group));
  kv_join<D, DT><<<grid, dim3(kJoinThreads), 0, stream>>>(a, p.rows);
  return hipGetLastError();
}
template <int D>
hipError_t join_by_dtype(const KvAttn& a, int dtype, const KvPlan& p, hipStream_t stream) {
  return dtype == NC_BF16 ? join<D, NC_BF16>(a, p, stream) : join<D, NC_F32>(a, p, stream);
}

}  // namespace

hipError_t launch_kv_join(const KvAttn& a, int dim, int dtype, const KvPlan& p, hipStream_t stream) {
  switch (dim) {
    case 64: return join_by_dtype<64>(a, dtype, p, stream);
    case 96: return join_by_dtype<96>(a, dtype, p, stream);
    case 128: return join_by_dtype<128>(a, dtype, p, stream);
    case 192: return join_by_dtype<192>(a, dtype, p, stream);
    case 256: return join_by_dtype<256>(a, dtype, p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace nc
