// The C-ABI of MX matrices, their products and the activations that keep their
// inputs in them: argument checks, the choice of kernel, launches.  No allocation,
// no state.
#include <algorithm>

#include "nc_mx.h"
#include "nc_mx_plan.h"

using namespace nc;

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool valid_fmt(int32_t f) { return f == NC_E2M1 || f == NC_E4M3 || f == NC_E5M2; }
bool valid_dtype(int32_t d) { return d == NC_F32 || d == NC_BF16; }
bool valid_rule(int32_t r) { return r == NC_MX_OCP || r == NC_MX_PLUS1 || r == NC_MX_CEIL; }
bool valid_act(int32_t a) { return a == NC_ACT_SILU || a == NC_ACT_GELU || a == NC_ACT_GELU_TANH || a == NC_ACT_RELU2; }
int64_t strips_of(int64_t rows) { return (rows + kMxRows - 1) / kMxRows; }
int64_t chunks_of(int64_t cols) { return (cols + kMxChunk - 1) / kMxChunk; }
nc_status hip_status(hipError_t e) { return e == hipSuccess ? NC_OK : NC_E_HIP; }

nc_status check_sizes(int64_t rows, int64_t cols, int32_t fmt) {
  if (!valid_fmt(fmt)) return NC_E_UNSUPPORTED;
  if (rows < 0 || cols < 0 || rows > INT32_MAX || cols > INT32_MAX) return NC_E_ARG;
  return strips_of(rows) * chunks_of(cols) <= kMostTiles ? NC_OK : NC_E_ARG;
}

nc_status check_matrix(const nc_mx_matrix* m) {
  if (m == nullptr) return NC_E_ARG;
  const nc_status s = check_sizes(m->rows, m->cols, m->fmt);
  if (s != NC_OK || m->rows == 0 || m->cols == 0) return s;
  if (m->data == nullptr) return NC_E_ARG;
  return aligned16(m->data) ? NC_OK : NC_E_ALIGN;
}

MxMat matrix_of(uint8_t* data, int64_t rows, int64_t cols, int32_t fmt) {
  const int64_t strips = strips_of(rows), chunks = chunks_of(cols);
  return MxMat{data, data != nullptr ? data + strips * chunks * mx_chunk_bytes(fmt) : nullptr, rows, cols, (int32_t)strips, (int32_t)chunks};
}
MxMat matrix_of(const nc_mx_matrix* m) { return matrix_of(m->data, m->rows, m->cols, m->fmt); }
bool empty(const nc_mx_matrix* m) { return m->rows == 0 || m->cols == 0; }

nc_status check_plane(const nc_plane* x, nc_dtype dtype, int64_t least) {
  if (x == nullptr || x->data == nullptr || x->stride < least) return NC_E_ARG;
  return ((uintptr_t)x->data & (dtype == NC_BF16 ? 1u : 3u)) == 0 ? NC_OK : NC_E_ALIGN;
}
Plane<const void*> input(const nc_plane* x) { return x != nullptr ? Plane<const void*>{x->data, x->stride} : Plane<const void*>{}; }
Plane<void*> output(const nc_plane* x) { return x != nullptr ? Plane<void*>{x->data, x->stride} : Plane<void*>{}; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t bytes_of(int64_t rows, int64_t cols, int32_t fmt) {
  return (size_t)(strips_of(rows) * chunks_of(cols)) * (size_t)(mx_chunk_bytes(fmt) + kMxScaleBytes);
}

nc_status check_out(const nc_mx_out* o, int64_t rows, int64_t cols) {
  if (o == nullptr) return NC_E_ARG;
  if (!valid_dtype(o->dtype)) return NC_E_UNSUPPORTED;
  if (rows == 0 || cols == 0) return NC_OK;
  const nc_plane p = {o->data, o->stride};
  const nc_status s = check_plane(&p, (nc_dtype)o->dtype, rows > 1 ? cols : 0);
  if (s != NC_OK) return s;
  return ((uintptr_t)o->bias & (o->dtype == NC_BF16 ? 1u : 3u)) == 0 ? NC_OK : NC_E_ALIGN;
}

void set_out(MxProduct& p, const nc_mx_out* o) {
  p.out = o->data;
  p.out_stride = o->stride;
  p.bias = o->bias;
  p.out_dtype = o->dtype;
  p.accumulate = o->accumulate != 0;
}

size_t part_bytes(int64_t rows_a, int64_t rows_b, int32_t splits) { return splits > 1 ? round256((size_t)(rows_a * rows_b) * 4 * splits) : 0; }

// For every plan of so many or fewer rows: no more than kMostSplitTiles tiles of
// 128 x 128, nor more splits than chunks allow.
size_t most_part_bytes(int64_t rows_a, int64_t rows_b, int64_t chunks) {
  const int64_t splits = std::min<int64_t>(kMostSplitTiles, chunks / kSplitChunks);
  if (splits < 2) return 0;
  return round256((size_t)std::min<double>((double)kMostSplitTiles * 128 * 128 * 4, (double)rows_a * (double)rows_b * 4 * (double)splits));
}

nc_status product(MxProduct& p, int32_t fa, int32_t fb, void* ws, size_t ws_bytes, hipStream_t stream) {
  MxPlan plan = plan_of(p.a.rows, p.b.rows, p.b.chunks, fa, fb, p.out_dtype == NC_F32);
  if (p.x != nullptr) plan = MxPlan{1, 0, 1};
  p.splits = plan.splits;
  p.part = (float*)ws;
  p.stream = p.out_dtype == NC_BF16 && mx_streams<NC_BF16>(Plane<void*>{p.out, p.out_stride}, p.a.rows, p.b.rows);
  if (part_bytes(p.a.rows, p.b.rows, plan.splits) > ws_bytes) return NC_E_WORKSPACE;
  if (plan.t > 0) {
    const int64_t side = 32 * plan.t;
    if (((p.a.rows + side - 1) / side) * ((p.b.rows + side - 1) / side) > kMostTiles / 2) return NC_E_ARG;   // 512 threads
    return hip_status(launch_mx_few(p, fa, fb, plan.t, stream));
  }
  if (((p.a.rows + 127) / 128) * ((p.b.rows + 127) / 128) > kMostTiles) return NC_E_ARG;
  return hip_status(launch_mx_many(p, fa, fb, plan.w, stream));
}

}  // namespace

extern "C" {

size_t nc_mx_bytes(int64_t rows, int64_t cols, int32_t fmt) {
  return check_sizes(rows, cols, fmt) == NC_OK ? bytes_of(rows, cols, fmt) : 0;
}

nc_status nc_mx_write(const nc_mx_matrix* m, const nc_mx_matrix* t, const nc_plane* x, nc_dtype dtype, nc_mx_rule rule,
                      void* stream) {
  if (!valid_dtype(dtype) || !valid_rule(rule)) return NC_E_UNSUPPORTED;
  if (m == nullptr && t == nullptr) return NC_E_ARG;
  nc_status s = NC_OK;
  if (m != nullptr && (s = check_matrix(m)) != NC_OK) return s;
  if (t != nullptr && (s = check_matrix(t)) != NC_OK) return s;
  if (m != nullptr && t != nullptr && (m->rows != t->cols || m->cols != t->rows || m->fmt != t->fmt)) return NC_E_SHAPE;
  if (t != nullptr && chunks_of(t->cols) * chunks_of(t->rows) > kMostTiles / 4 - 8) return NC_E_ARG;
  const nc_mx_matrix* any = m != nullptr ? m : t;
  if (empty(any)) return NC_OK;
  if ((s = check_plane(x, dtype, 0)) != NC_OK) return s;
  const MxMat mm = m != nullptr ? matrix_of(m) : MxMat{}, tt = t != nullptr ? matrix_of(t) : MxMat{};
  return hip_status(launch_mx_write(m != nullptr ? &mm : nullptr, t != nullptr ? &tt : nullptr, any->fmt, input(x), dtype, rule,
                                    (hipStream_t)stream));
}

nc_status nc_mx_read(const nc_mx_matrix* m, const nc_plane* y, nc_dtype dtype, void* stream) {
  if (!valid_dtype(dtype)) return NC_E_UNSUPPORTED;
  nc_status s = check_matrix(m);
  if (s != NC_OK || empty(m)) return s;
  if ((s = check_plane(y, dtype, m->rows > 1 ? m->cols : 0)) != NC_OK) return s;
  return hip_status(launch_mx_read(matrix_of(m), m->fmt, output(y), dtype, (hipStream_t)stream));
}

size_t nc_mx_workspace_bytes(const nc_mx_matrix* b, int64_t rows, int32_t x_fmt) {
  if (b == nullptr || check_sizes(b->rows, b->cols, b->fmt) != NC_OK || rows < 0 || rows > INT32_MAX) return 0;
  if (x_fmt >= 0 && rows <= kMxFusedRows) return 0;   // nothing written first, no splits
  const size_t part = most_part_bytes(rows, b->rows, chunks_of(b->cols));
  if (x_fmt < 0) return part;
  return check_sizes(rows, b->cols, x_fmt) == NC_OK ? part + round256(bytes_of(rows, b->cols, x_fmt)) : 0;
}

nc_status nc_mx_matmul(const nc_mx_matrix* a, const nc_mx_matrix* b, const nc_mx_out* out, void* ws, size_t ws_bytes,
                       void* stream) {
  nc_status s = check_matrix(a);
  if (s != NC_OK || (s = check_matrix(b)) != NC_OK) return s;
  if (a->cols != b->cols) return NC_E_SHAPE;
  if ((s = check_out(out, a->rows, b->rows)) != NC_OK) return s;
  if (a->rows == 0 || b->rows == 0) return NC_OK;
  MxProduct p = {};
  p.a = matrix_of(a);
  p.b = matrix_of(b);
  set_out(p, out);
  if (ws_bytes > 0 && (ws == nullptr || !aligned16(ws))) return NC_E_WORKSPACE;
  return product(p, a->fmt, b->fmt, ws, ws_bytes, (hipStream_t)stream);
}

nc_status nc_mx_linear(const nc_plane* x, int64_t rows, nc_dtype x_dtype, nc_fmt x_fmt, nc_mx_rule rule,
                       const nc_mx_matrix* w, const nc_mx_out* out, void* ws, size_t ws_bytes, void* stream) {
  if (!valid_dtype(x_dtype) || !valid_rule(rule)) return NC_E_UNSUPPORTED;
  nc_status s = check_matrix(w);
  if (s != NC_OK || (s = check_sizes(rows, w->cols, x_fmt)) != NC_OK) return s;
  if ((s = check_out(out, rows, w->rows)) != NC_OK) return s;
  if (rows == 0 || w->rows == 0) return NC_OK;
  if (w->cols > 0 && (s = check_plane(x, x_dtype, 0)) != NC_OK) return s;
  if (ws_bytes > 0 && (ws == nullptr || !aligned16(ws))) return NC_E_WORKSPACE;
  MxProduct p = {};
  p.b = matrix_of(w);
  set_out(p, out);
  if (rows <= kMxFusedRows) {
    p.a = matrix_of(nullptr, rows, w->cols, x_fmt);
    p.x = w->cols > 0 ? x->data : nullptr;
    p.x_stride = w->cols > 0 ? x->stride : 0;
    p.x_dtype = x_dtype;
    p.rule = rule;
    return product(p, x_fmt, w->fmt, ws, ws_bytes, (hipStream_t)stream);
  }
  const size_t need = round256(bytes_of(rows, w->cols, x_fmt));
  if (ws_bytes < need) return NC_E_WORKSPACE;
  p.a = matrix_of((uint8_t*)ws, rows, w->cols, x_fmt);
  if (w->cols > 0) {
    const hipError_t e = launch_mx_write(&p.a, nullptr, x_fmt, input(x), x_dtype, rule, (hipStream_t)stream);
    if (e != hipSuccess) return hip_status(e);
  }
  return product(p, x_fmt, w->fmt, (uint8_t*)ws + need, ws_bytes - need, (hipStream_t)stream);
}

nc_status nc_act_forward(nc_act act, int64_t rows, int64_t cols, const nc_plane* gate, const nc_plane* up,
                         const nc_plane* y, nc_dtype dtype, const nc_mx_matrix* gate_q, const nc_mx_matrix* up_q,
                         nc_mx_rule rule, void* stream) {
  if (!valid_act(act) || !valid_dtype(dtype) || !valid_rule(rule)) return NC_E_UNSUPPORTED;
  nc_status s = check_sizes(rows, cols, NC_E4M3);
  if (s != NC_OK) return s;
  if ((gate_q == nullptr ? up_q != nullptr : (up_q != nullptr) != (up != nullptr))) return NC_E_ARG;
  if (gate_q != nullptr && (s = check_matrix(gate_q)) != NC_OK) return s;
  if (up_q != nullptr && (s = check_matrix(up_q)) != NC_OK) return s;
  if (gate_q != nullptr && (gate_q->rows != rows || gate_q->cols != cols)) return NC_E_SHAPE;
  if (up_q != nullptr && (up_q->rows != rows || up_q->cols != cols || up_q->fmt != gate_q->fmt)) return NC_E_SHAPE;
  if (rows == 0 || cols == 0) return NC_OK;
  if ((s = check_plane(gate, dtype, 0)) != NC_OK) return s;
  if (up != nullptr && (s = check_plane(up, dtype, 0)) != NC_OK) return s;
  if ((s = check_plane(y, dtype, rows > 1 ? cols : 0)) != NC_OK) return s;
  ActForward a = {};
  a.gate = input(gate);
  a.up = input(up);
  a.y = output(y);
  a.gate_q = gate_q != nullptr ? matrix_of(gate_q) : matrix_of(nullptr, rows, cols, NC_E4M3);
  if (up_q != nullptr) a.up_q = matrix_of(up_q);
  a.rule = rule;
  return hip_status(launch_act_forward(a, act, gate_q != nullptr ? gate_q->fmt : NC_E4M3, dtype, (hipStream_t)stream));
}

nc_status nc_act_backward(nc_act act, const nc_plane* dy, nc_dtype dtype, const nc_mx_matrix* gate_q,
                          const nc_mx_matrix* up_q, const nc_plane* dgate, const nc_plane* dup, const nc_plane* y,
                          void* stream) {
  if (!valid_act(act) || !valid_dtype(dtype)) return NC_E_UNSUPPORTED;
  nc_status s = check_matrix(gate_q);
  if (s != NC_OK) return s;
  if (up_q != nullptr && (s = check_matrix(up_q)) != NC_OK) return s;
  if ((up_q != nullptr) != (dup != nullptr)) return NC_E_ARG;
  if (up_q != nullptr && (up_q->rows != gate_q->rows || up_q->cols != gate_q->cols || up_q->fmt != gate_q->fmt)) return NC_E_SHAPE;
  if (empty(gate_q)) return NC_OK;
  const int64_t least = gate_q->rows > 1 ? gate_q->cols : 0;
  if ((s = check_plane(dy, dtype, 0)) != NC_OK || (s = check_plane(dgate, dtype, least)) != NC_OK) return s;
  if (dup != nullptr && (s = check_plane(dup, dtype, least)) != NC_OK) return s;
  if (y != nullptr && (s = check_plane(y, dtype, least)) != NC_OK) return s;
  ActBackward a = {};
  a.dy = input(dy);
  a.gate_q = matrix_of(gate_q);
  if (up_q != nullptr) a.up_q = matrix_of(up_q);
  a.dgate = output(dgate);
  a.dup = output(dup);
  a.y = output(y);
  return hip_status(launch_act_backward(a, act, gate_q->fmt, dtype, (hipStream_t)stream));
}

}  // extern "C"
