"""scaled_fp8_casting_amd: the scaled FP8 cast on MI355X (gfx950).

A thin Python binding over libnarrowcast's C-ABI (include/narrowcast.h).
Functions carry the C names and only marshal arguments: torch tensors
provide device memory and the current HIP stream; every step of the cast
runs in the library's HIP kernels.  There is no CPU fallback: calls raise if
the library is not built or a tensor is not on the GPU.

Device buffers used by the calls, as torch tensors:

* counts: int64 [count, 5] -- n_finite, n_clip, n_underflow, n_nonfinite,
  then amax (fp32 bits in the low 32 bits of the fifth word);
* stats:  float64 [count, 6] -- sum e, |e|, e^2, sign(x) e, x e, x^2;
* state:  int32 [count, 6] -- k, a_ref bits, has_ref, n_hist, head, step;
* hist:   float32 [count, window];
* loss scale: int32 [2] -- s_log2, clean_steps.

The key/value cache (new_kv_cache, nc_kv_write, nc_kv_read, nc_kv_attention)
keeps keys and values as MX blocks of E2M1 or E4M3 codes in pages.
"""

import ctypes
import math
import struct
from operator import attrgetter
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import (NC_BF16, NC_E2M1, NC_E4M3, NC_E5M2, NC_EST_CURRENT, NC_EST_EMA, NC_EST_MAX_WINDOW,  # noqa: F401
                   NC_EST_MOST_RECENT, NC_F32, NC_MX_CEIL, NC_MX_OCP, NC_MX_PLUS1, NC_W_BF16, NC_W_FP16,
                   NcKvAttn, NcKvCache, NcKvRows, NcPolicy, NcSwampPolicy, NcTensor, NcUpdateTensor)

COUNT_FIELDS = ("n_finite", "n_clip", "n_underflow", "n_nonfinite")
STAT_FIELDS = ("sum_e", "sum_abs_e", "sum_e2", "sum_dir_e", "sum_xe", "sum_x2")
STATE_FIELDS = ("k", "a_ref_bits", "has_ref", "n_hist", "head", "step")

FMT = {"e4m3": NC_E4M3, "e5m2": NC_E5M2}
MX_RULE = {"ocp": NC_MX_OCP, "plus1": NC_MX_PLUS1, "ceil": NC_MX_CEIL}
MX_AXIS = {"rows": 0, "cols": 1}
EST = {"current": NC_EST_CURRENT, "most_recent": NC_EST_MOST_RECENT, "max_window": NC_EST_MAX_WINDOW,
       "ema": NC_EST_EMA}


class NarrowcastError(RuntimeError):
    def __init__(self, status: int, call: str):
        msg = _lib.load().nc_status_string(status).decode()
        super().__init__(f"{call}: status {status}: {msg}")
        self.status = status


def _check(status: int, call: str):
    if status != 0:
        raise NarrowcastError(status, call)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return NC_F32
    if t.dtype == torch.bfloat16:
        return NC_BF16
    raise TypeError(f"input dtype {t.dtype} (float32 or bfloat16 expected)")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected (no CPU path)")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: Optional[torch.Tensor], name: str, dtype: torch.dtype, rows: int, width: Optional[int] = None):
    """Raise ValueError unless t is a contiguous `dtype` tensor holding at least
    `rows` rows of `width` elements (or `rows` elements when width is None):
    the kernels write (or read) that many, so a smaller buffer would be
    overrun on the GPU."""
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: contiguous tensor expected")
    if width is None:
        if t.numel() < rows:
            raise ValueError(f"{name}: {t.numel()} elements, at least {rows} needed")
    elif t.dim() != 2 or t.shape[1] != width or t.shape[0] < rows:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected ({rows}, {width}) or more rows")


def tensors(xs: Sequence[Optional[torch.Tensor]], codes: Sequence[Optional[torch.Tensor]],
            cols: Optional[Sequence[int]] = None, scales: Optional[Sequence[torch.Tensor]] = None,
            n: Optional[Sequence[int]] = None, axis: str = "rows"):
    """A host array of nc_tensor descriptors (contiguous device tensors).

    Before any pointer is taken, the sizes are checked against what the
    kernels will touch: every input has the first input's dtype (fp32 or
    bf16), every code buffer is uint8 with exactly as many elements as its
    input, every scale buffer uint8 with one byte per 32 elements, and the
    per-tensor lists have one entry per tensor.  A mismatch raises
    ValueError."""
    count = len(codes)
    for name, lst in (("xs", xs), ("cols", cols), ("scales", scales), ("n", n)):
        if lst is not None and len(lst) != count:
            raise ValueError(f"{name}: {len(lst)} entries for {count} tensors")
    if axis not in MX_AXIS:
        raise ValueError(f"axis {axis!r}")
    dt0 = None
    if xs is not None and count:
        dt0 = xs[0].dtype
        _dtype_code(xs[0])
    ns = []
    for i in range(count):
        x = xs[i] if xs is not None else None
        c = codes[i]
        if x is not None and x.dtype != dt0:
            raise ValueError(f"xs[{i}]: dtype {x.dtype}, but xs[0] is {dt0} (one dtype per call)")
        for t in (x, c):
            if t is not None and not t.is_contiguous():
                raise ValueError("contiguous tensors expected")
        ni = n[i] if n is not None else (x.numel() if x is not None else c.numel())
        if x is not None and x.numel() != ni:
            raise ValueError(f"xs[{i}]: {x.numel()} elements, n = {ni}")
        if c is not None:
            if c.dtype != torch.uint8:
                raise ValueError(f"codes[{i}]: dtype {c.dtype}, expected torch.uint8")
            if c.numel() != ni:
                raise ValueError(f"codes[{i}]: {c.numel()} elements for {ni} inputs")
        if scales is not None:
            sc = scales[i]
            if sc.dtype != torch.uint8 or not sc.is_contiguous():
                raise ValueError(f"scales[{i}]: contiguous torch.uint8 expected")
            if sc.numel() != ni // 32:
                raise ValueError(f"scales[{i}]: {sc.numel()} bytes for {ni // 32} blocks of 32")
        ns.append(ni)
    arr = (NcTensor * max(count, 1))()
    for i in range(count):
        x = xs[i] if xs is not None else None
        c = codes[i]
        arr[i].x = _ptr(x) if x is not None and x.numel() else None
        arr[i].codes = _ptr(c) if c is not None and c.numel() else None
        arr[i].n = ns[i]
        arr[i].cols = cols[i] if cols is not None else 0
        arr[i].scales = _ptr(scales[i]) if scales is not None and scales[i].numel() else None
        arr[i].mx_axis = MX_AXIS[axis]
    return arr, count


# -- device buffers ---------------------------------------------------------

def new_counts(count: int, device="cuda") -> torch.Tensor:
    return torch.zeros((count, 5), dtype=torch.int64, device=device)


def new_stats(count: int, device="cuda") -> torch.Tensor:
    return torch.zeros((count, 6), dtype=torch.float64, device=device)


def new_state(count: int, device="cuda") -> torch.Tensor:
    return torch.zeros((count, 6), dtype=torch.int32, device=device)


def new_history(count: int, window: int, device="cuda") -> torch.Tensor:
    return torch.zeros((count, window), dtype=torch.float32, device=device)


def new_loss_scale(s_log2: int, device="cuda") -> torch.Tensor:
    return torch.tensor([s_log2, 0], dtype=torch.int32, device=device)


def policy(fmt="e4m3", est="max_window", window=16, margin=0, hysteresis=True, interval=1,
           skip_on_nonfinite=False, ls_enable=False, ls_growth_interval=2000, ls_log2_min=0,
           ls_log2_max=24, ema_alpha=0.0625) -> NcPolicy:
    return NcPolicy(FMT[fmt] if isinstance(fmt, str) else fmt, EST[est] if isinstance(est, str) else est,
                    window, margin, int(hysteresis), interval, int(skip_on_nonfinite), int(ls_enable),
                    ls_growth_interval, ls_log2_min, ls_log2_max, ema_alpha)


def counts_list(counts: torch.Tensor):
    """Host view of a counts tensor: one dict per tensor (amax as a float)."""
    rows = counts.cpu().tolist()
    out = []
    for r in rows:
        d = dict(zip(COUNT_FIELDS, r[:4]))
        d["amax_bits"] = r[4] & 0xFFFFFFFF
        d["amax"] = struct.unpack("<f", struct.pack("<I", d["amax_bits"]))[0]
        out.append(d)
    return out


def workspace_bytes(desc, count: int) -> int:
    return int(_lib.load().nc_workspace_bytes(desc, count))


def new_workspace(desc, count: int, device="cuda") -> torch.Tensor:
    """Device workspace for the calls that reduce (amax, casts, statistics);
    torch's allocator returns 256-byte aligned memory."""
    return torch.empty(max(workspace_bytes(desc, count), 16), dtype=torch.uint8, device=device)


def _check_cast_outputs(count, st, out, ls, stats, ws):
    _need(st, "st", torch.int32, count, 6)
    _need(out, "out", torch.int64, count, 5)
    _need(ls, "ls", torch.int32, 2)
    _need(stats, "stats", torch.float64, count, 6)
    _need(ws, "ws", torch.uint8, 0)


def _ws(ws, desc, count):
    return new_workspace(desc, count) if ws is None else ws


# -- the C-ABI calls ----------------------------------------------------------

def nc_amax(xs: Sequence[torch.Tensor], out: torch.Tensor, ls: Optional[torch.Tensor] = None,
            ws: Optional[torch.Tensor] = None, stream=None):
    _need(out, "out", torch.int64, len(xs), 5)
    _need(ls, "ls", torch.int32, 2)
    _need(ws, "ws", torch.uint8, 0)
    desc, count = tensors(xs, [None] * len(xs))
    dt = _dtype_code(xs[0]) if xs else NC_F32
    ws = _ws(ws, desc, count)
    _check(_lib.load().nc_amax(desc, count, dt, _ptr(ls), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)),
           "nc_amax")


def nc_scale_update(pol: NcPolicy, st: torch.Tensor, in_counts: torch.Tensor,
                    hist: Optional[torch.Tensor] = None, ls: Optional[torch.Tensor] = None,
                    stream=None):
    count = st.shape[0]
    _need(st, "st", torch.int32, count, 6)
    _need(in_counts, "in_counts", torch.int64, count, 5)
    _need(hist, "hist", torch.float32, count * pol.window)
    _need(ls, "ls", torch.int32, 2)
    _check(_lib.load().nc_scale_update(ctypes.byref(pol), count, _ptr(st), _ptr(hist),
                                       _ptr(in_counts), _ptr(ls), _stream(stream)), "nc_scale_update")


def nc_cast_tensor(xs: Sequence[torch.Tensor], codes: Sequence[torch.Tensor], fmt, st: torch.Tensor,
                   out: torch.Tensor, ls: Optional[torch.Tensor] = None,
                   stats: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                   stream=None):
    _check_cast_outputs(len(codes), st, out, ls, stats, ws)
    desc, count = tensors(xs, codes)
    dt = _dtype_code(xs[0]) if xs else NC_F32
    f = FMT[fmt] if isinstance(fmt, str) else fmt
    ws = _ws(ws, desc, count)
    _check(_lib.load().nc_cast_tensor(desc, count, dt, f, _ptr(st), _ptr(ls), _ptr(out), _ptr(stats),
                                      _ptr(ws), ws.numel(), _stream(stream)), "nc_cast_tensor")


def nc_cast_tensor_static(xs: Sequence[torch.Tensor], codes: Sequence[torch.Tensor], fmt, st: torch.Tensor,
                          out: torch.Tensor, ls: Optional[torch.Tensor] = None,
                          stats: Optional[torch.Tensor] = None, stream=None):
    """nc_cast_tensor without a workspace: the library's static per-GPU
    scratch serves instead, so nothing is allocated (for callers that cannot
    allocate).  Calls that overlap on one GPU race on that scratch."""
    _check_cast_outputs(len(codes), st, out, ls, stats, None)
    desc, count = tensors(xs, codes)
    dt = _dtype_code(xs[0]) if xs else NC_F32
    f = FMT[fmt] if isinstance(fmt, str) else fmt
    _check(_lib.load().nc_cast_tensor_static(desc, count, dt, f, _ptr(st), _ptr(ls), _ptr(out), _ptr(stats),
                                             _stream(stream)), "nc_cast_tensor_static")


def nc_cast_tensor_sr(xs: Sequence[torch.Tensor], codes: Sequence[torch.Tensor], fmt, st: torch.Tensor,
                      out: torch.Tensor, seed: int, offset: int, ls: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None, stream=None):
    _check_cast_outputs(len(codes), st, out, ls, None, ws)
    desc, count = tensors(xs, codes)
    dt = _dtype_code(xs[0]) if xs else NC_F32
    f = FMT[fmt] if isinstance(fmt, str) else fmt
    ws = _ws(ws, desc, count)
    _check(_lib.load().nc_cast_tensor_sr(desc, count, dt, f, _ptr(st), _ptr(ls), seed & (2 ** 64 - 1),
                                         offset & (2 ** 64 - 1), _ptr(out), _ptr(ws), ws.numel(),
                                         _stream(stream)), "nc_cast_tensor_sr")


def nc_cast_mx(xs: Sequence[torch.Tensor], codes: Sequence[torch.Tensor], scales: Sequence[torch.Tensor],
               cols: Sequence[int], fmt, rule, out: torch.Tensor, stats: Optional[torch.Tensor] = None,
               ws: Optional[torch.Tensor] = None, stream=None, axis: str = "rows"):
    _check_cast_outputs(len(codes), None, out, None, stats, ws)
    desc, count = tensors(xs, codes, cols=cols, scales=scales, axis=axis)
    dt = _dtype_code(xs[0]) if xs else NC_BF16
    f = FMT[fmt] if isinstance(fmt, str) else fmt
    r = MX_RULE[rule] if isinstance(rule, str) else rule
    ws = _ws(ws, desc, count)
    _check(_lib.load().nc_cast_mx(desc, count, dt, f, r, _ptr(out), _ptr(stats), _ptr(ws), ws.numel(),
                                  _stream(stream)), "nc_cast_mx")


def nc_dequant(codes: Sequence[torch.Tensor], ys: Sequence[torch.Tensor], fmt,
               st: Optional[torch.Tensor] = None, scales: Optional[Sequence[torch.Tensor]] = None,
               cols: Optional[Sequence[int]] = None, stream=None, axis: str = "rows"):
    count = len(codes)
    if len(ys) != count:
        raise ValueError(f"ys: {len(ys)} entries for {count} tensors")
    for i, y in enumerate(ys):
        if y.dtype != torch.bfloat16 or not y.is_contiguous():
            raise TypeError("dequant output must be contiguous bfloat16")
        if y.numel() != codes[i].numel():
            raise ValueError(f"ys[{i}]: {y.numel()} elements for {codes[i].numel()} codes")
    _need(st, "st", torch.int32, count, 6)
    desc, count = tensors(None, codes, cols=cols, scales=scales, axis=axis)
    f = FMT[fmt] if isinstance(fmt, str) else fmt
    yp = (ctypes.c_void_p * max(count, 1))(*[_ptr(y) if y.numel() else None for y in ys])
    _check(_lib.load().nc_dequant(desc, count, f, _ptr(st), yp, NC_BF16, _stream(stream)), "nc_dequant")


def nc_cast_stats(xs: Sequence[torch.Tensor], codes: Sequence[torch.Tensor], fmt, out: torch.Tensor,
                  ws: Optional[torch.Tensor] = None, st: Optional[torch.Tensor] = None,
                  ls: Optional[torch.Tensor] = None,
                  scales: Optional[Sequence[torch.Tensor]] = None, cols: Optional[Sequence[int]] = None,
                  stream=None, axis: str = "rows"):
    _need(out, "out", torch.float64, len(codes), 6)
    _need(st, "st", torch.int32, len(codes), 6)
    _need(ls, "ls", torch.int32, 2)
    _need(ws, "ws", torch.uint8, 0)
    desc, count = tensors(xs, codes, cols=cols, scales=scales, axis=axis)
    dt = _dtype_code(xs[0]) if xs else NC_F32
    f = FMT[fmt] if isinstance(fmt, str) else fmt
    ws = _ws(ws, desc, count)
    _check(_lib.load().nc_cast_stats(desc, count, dt, f, _ptr(st), _ptr(ls), _ptr(out), _ptr(ws),
                                     ws.numel(), _stream(stream)), "nc_cast_stats")


# -- the update/step-ratio ("swamping") monitor -------------------------------

WFMT = {"bf16": NC_W_BF16, "fp16": NC_W_FP16}
SWAMP_FIELDS = ("n_considered", "n_zero", "n_below", "n_noop", "n_excluded")


def update_tensors(ws: Sequence[torch.Tensor], ds: Sequence[torch.Tensor],
                   flags: Optional[Sequence[Optional[torch.Tensor]]] = None):
    """A host array of nc_update_tensor descriptors (contiguous fp32 device tensors)."""
    count = len(ws)
    if len(ds) != count or (flags is not None and len(flags) != count):
        raise ValueError("one update (and flag buffer) per weight tensor")
    for i in range(count):
        w, d = ws[i], ds[i]
        for t in (w, d):
            if t.dtype != torch.float32 or not t.is_contiguous():
                raise TypeError("weights and updates must be contiguous float32")
        if w.numel() != d.numel():
            raise ValueError("a weight tensor and its update differ in size")
        if flags is not None and flags[i] is not None:
            _need(flags[i], f"flags[{i}]", torch.uint8, w.numel())
            if flags[i].numel() != w.numel():
                raise ValueError(f"flags[{i}]: {flags[i].numel()} bytes for {w.numel()} elements")
    arr = (NcUpdateTensor * max(count, 1))()
    for i in range(count):
        w, d = ws[i], ds[i]
        arr[i].w = _ptr(w) if w.numel() else None
        arr[i].d = _ptr(d) if d.numel() else None
        f = flags[i] if flags is not None else None
        arr[i].flags = _ptr(f) if f is not None and f.numel() else None
        arr[i].n = w.numel()
    return arr, count


def new_swamp_counts(count: int, device="cuda") -> torch.Tensor:
    return torch.zeros((count, 5), dtype=torch.int64, device=device)


def new_swamp_state(count: int, device="cuda") -> torch.Tensor:
    return torch.zeros((count, 4), dtype=torch.int32, device=device)


def swamp_policy(window=8, num=1, den=2) -> NcSwampPolicy:
    return NcSwampPolicy(window, num, den, 0)


def swamp_counts_list(counts: torch.Tensor):
    return [dict(zip(SWAMP_FIELDS, r)) for r in counts.cpu().tolist()]


def new_swamp_workspace(ws: Sequence[torch.Tensor], ds: Sequence[torch.Tensor], device="cuda") -> torch.Tensor:
    desc, count = update_tensors(ws, ds)
    return torch.empty(max(int(_lib.load().nc_swamp_workspace_bytes(desc, count)), 16), dtype=torch.uint8,
                       device=device)


def nc_swamp_watch(ws: Sequence[torch.Tensor], ds: Sequence[torch.Tensor], wfmt, out: torch.Tensor,
                   flags: Optional[Sequence[Optional[torch.Tensor]]] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    _need(out, "out", torch.int64, len(ws), 5)
    _need(workspace, "workspace", torch.uint8, 0)
    desc, count = update_tensors(ws, ds, flags)
    lib = _lib.load()
    if workspace is None:
        workspace = new_swamp_workspace(ws, ds)
    f = WFMT[wfmt] if isinstance(wfmt, str) else wfmt
    _check(lib.nc_swamp_watch(desc, count, f, _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)),
           "nc_swamp_watch")


def nc_swamp_window(pol: NcSwampPolicy, st: torch.Tensor, in_counts: torch.Tensor, stream=None):
    _need(st, "st", torch.int32, st.shape[0], 4)
    _need(in_counts, "in_counts", torch.int64, st.shape[0], 5)
    _check(_lib.load().nc_swamp_window(ctypes.byref(pol), st.shape[0], _ptr(st), _ptr(in_counts),
                                       _stream(stream)), "nc_swamp_window")


# -- the key/value cache -------------------------------------------------------

KV_FMT = {"e2m1": NC_E2M1, "e4m3": NC_E4M3}
_I32_MAX = 2 ** 31 - 1


class KvCache:
    """Keys and values of past tokens as MX blocks, in pages.

    data is one uint8 tensor of `pages` rows, a page each; pages may be copied
    as rows, and another tensor may take its place.  `page` tokens a page (a
    multiple of 16), `heads` key/value heads of `dim` elements (64, 96, 128, 192
    or 256), fmt "e2m1" or "e4m3"; these are fixed."""

    def __init__(self, data: torch.Tensor, page: int, heads: int, dim: int, fmt: str):
        self._page, self._heads, self._dim, self._fmt = int(page), int(heads), int(dim), fmt
        self.data = data

    page, heads, dim, fmt = (property(attrgetter(name)) for name in ("_page", "_heads", "_dim", "_fmt"))
    device, data = (property(attrgetter(name)) for name in ("_device", "_data"))
    pages = property(lambda self: self._data.shape[0])

    @data.setter
    def data(self, data: torch.Tensor):
        each = kv_page_bytes(self._page, self._heads, self._dim, self._fmt)
        if data.dtype != torch.uint8 or data.dim() != 2 or data.shape[1] != each or not data.is_contiguous():
            raise ValueError(f"data: shape {tuple(data.shape)} of {data.dtype}, expected contiguous "
                             f"torch.uint8 (pages, {each})")
        pages, fmt = data.shape[0], KV_FMT[self._fmt]
        if pages and _lib.load().nc_kv_cache_bytes(pages, self._page, self._heads, self._dim, fmt) == 0:
            raise ValueError(f"{pages} pages: pages * page and pages * page / 16 * heads stay below 2^31")
        self._data, self._at, self._bytes, self._device = data, data.data_ptr(), data.numel(), data.device
        self._gpu = data.device.index if data.device.type == "cuda" else None
        self._descriptor = NcKvCache(self._at if pages else None, pages, self._page, self._heads, self._dim, fmt)

    @property
    def descriptor(self) -> NcKvCache:
        """What the calls pass on.  A tensor may be resized in place, so data is looked at every time."""
        d = self._data
        if d.data_ptr() != self._at or d.numel() != self._bytes:
            self.data = d
        return self._descriptor


def kv_page_bytes(page: int, heads: int, dim: int, fmt: str) -> int:
    """Bytes of one page of a cache."""
    if fmt not in KV_FMT:
        raise ValueError(f"fmt {fmt!r}: one of {sorted(KV_FMT)}")
    if page <= 0 or page % 16:
        raise ValueError(f"page {page}: a positive multiple of 16")
    if heads < 1 or dim not in (64, 96, 128, 192, 256):
        raise ValueError(f"heads {heads}, dim {dim}: at least one head of 64, 96, 128, 192 or 256 elements")
    # the library takes 32 bits of either, and ctypes would drop the rest of a longer number
    each = 0 if max(page, heads) > _I32_MAX else int(_lib.load().nc_kv_cache_bytes(1, page, heads, dim, KV_FMT[fmt]))
    if each == 0:
        raise ValueError(f"page {page}, heads {heads}: too large")
    return each


def new_kv_cache(pages: int, page: int, heads: int, dim: int, fmt: str = "e2m1", device="cuda") -> KvCache:
    """A cache of `pages` pages, every token zero."""
    return KvCache(torch.zeros((pages, kv_page_bytes(page, heads, dim, fmt)), dtype=torch.uint8, device=device), page,
                   heads, dim, fmt)


_KV_DTYPE = {torch.float32: (NC_F32, 4), torch.bfloat16: (NC_BF16, 8)}     # code, elements of 16 bytes


def _rows(t: torch.Tensor, name: str, shape: tuple, dtype: torch.dtype, unit: int, dev: torch.device):
    """Pointer, token and head stride of [tokens, heads, dim] rows: strides that are multiples of 16 bytes,
    elements adjacent.  The pointer is checked to be the device's by the caller."""
    if t.dtype is not dtype or t.shape != shape or t.device != dev:
        raise ValueError(f"{name}: shape {tuple(t.shape)} of {t.dtype} on {t.device}, expected {tuple(shape)} of "
                         f"{dtype} on {dev}")
    ts, hs, one = t.stride()
    at = t.data_ptr()
    if one != 1 or (ts | hs) & (unit - 1) or at & 15:
        ts, hs = ts if shape[0] > 1 else 0, hs if shape[1] > 1 else 0     # torch gives an axis of length 1 any stride
        if one != 1 or (ts | hs) & (unit - 1) or at & 15:
            raise ValueError(f"{name}: strides {t.stride()}: rows of adjacent elements that start on 16 bytes expected")
    return at, ts, hs


def _spread(t: torch.Tensor, name: str):
    """Raise ValueError where an output's rows share memory."""
    if t.is_contiguous():
        return
    at = 0
    for size, stride in sorted(((n, s) for n, s in zip(t.shape, t.stride()) if n > 1), key=lambda x: x[1]):
        if stride <= at:
            raise ValueError(f"{name}: strides {t.stride()}: its rows overlap")
        at += (size - 1) * stride


def _kv_stream(stream, gpu: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(gpu)           # torch.cuda.current_stream(gpu), without its object
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _kv_call(cache: KvCache, name: str, call, *args):
    """The library's call with the cache's GPU as the current one: a default stream's number is 0 on every GPU,
    and means the current one's."""
    if torch._C._cuda_getDevice() == cache._gpu:  # torch.cuda.current_device(), for a GPU that is in use
        status = call(*args)
    else:
        with torch.cuda.device(cache.device):
            status = call(*args)
    if status:
        _check(status, name)


def _kv_tokens(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor):
    """Checks of a write or read; the call's arguments from the cache to the slots."""
    c = cache.descriptor                         # first: it looks at data anew
    dt, dev = k.dtype, cache._device
    code, unit = _KV_DTYPE.get(dt, (None, 0))
    if code is None:
        raise TypeError(f"dtype {dt} (float32 or bfloat16 expected)")
    if slots.dtype is not torch.int64 or slots.dim() != 1 or slots.device != dev or not slots.is_contiguous():
        raise ValueError(f"slots: shape {tuple(slots.shape)} of {slots.dtype} on {slots.device}, expected contiguous "
                         f"torch.int64, one entry a token, on {dev}")
    tokens = slots.numel()
    shape = (tokens, cache._heads, cache._dim)
    ks, vs = _rows(k, "k", shape, dt, unit, dev), _rows(v, "v", shape, dt, unit, dev)
    if cache._gpu is None:
        raise ValueError("device tensor expected (no CPU path)")
    return c, NcKvRows(*ks), NcKvRows(*vs), tokens, code, slots.data_ptr()


def nc_kv_write(cache: KvCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, rule="ceil", stream=None):
    """Quantise keys and values [tokens, heads, dim] into the cache at `slots`
    (int64, page * cache.page + offset; distinct; -1 skips a token).  k and v
    may be slices of a fused projection."""
    r = MX_RULE[rule] if isinstance(rule, str) else rule
    args = _kv_tokens(cache, k, v, slots)
    _kv_call(cache, "nc_kv_write", _lib.load().nc_kv_write, *args, r, _kv_stream(stream, cache._gpu))


def nc_kv_read(cache: KvCache, slots: torch.Tensor, k_out: torch.Tensor, v_out: torch.Tensor, stream=None):
    """The keys and values at `slots`, as fp32 or bf16 [tokens, heads, dim]."""
    _spread(k_out, "k")
    _spread(v_out, "v")
    args = _kv_tokens(cache, k_out, v_out, slots)
    _kv_call(cache, "nc_kv_read", _lib.load().nc_kv_read, *args, _kv_stream(stream, cache._gpu))


def kv_workspace_bytes(cache: KvCache, q: torch.Tensor, batch: int, max_q: int, max_kv: int) -> int:
    if max(q.shape[1], batch, max_q, max_kv) > _I32_MAX:
        raise ValueError(f"q_heads {q.shape[1]}, batch {batch}, max_q {max_q}, max_kv {max_kv}: at most 2^31 - 1 each")
    return int(_lib.load().nc_kv_workspace_bytes(cache.descriptor, _dtype_code(q), q.shape[1], batch, max_q, max_kv))


def new_kv_workspace(cache: KvCache, q: torch.Tensor, batch: int, max_q: int, max_kv: int) -> torch.Tensor:
    """Device workspace for nc_kv_attention at these or smaller batch, max_q and
    max_kv, whatever the window; calls that run concurrently need workspaces of
    their own."""
    return torch.empty(max(kv_workspace_bytes(cache, q, batch, max_q, max_kv), 16), dtype=torch.uint8,
                       device=cache.device)


def nc_kv_attention(cache: KvCache, q: torch.Tensor, out: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
                    table: torch.Tensor, max_q: int, max_kv: int, causal: bool = True, window: int = 0,
                    scale: Optional[float] = None, lse: Optional[torch.Tensor] = None,
                    ws: Optional[torch.Tensor] = None, stream=None):
    """Attention of queries q [rows, q_heads, dim] over the cache, into out (as q).

    Sequence b has the rows q_start[b] .. q_start[b + 1] - 1 of q (int32,
    batch + 1) and kv_len[b] cached tokens (int32) on the pages table[b] (int32
    [batch, pages]).  max_q and max_kv bound both on the host; the work is split
    as if every sequence had max_q queries, so prompts and single tokens are
    faster as two calls.  causal: the queries are the sequence's last tokens; else each sees the whole cache
    (cross attention).  window: tokens that a query sees at most, 0 for all.
    scale: 1 / sqrt(dim) where None.  lse (fp32 [rows, q_heads]) receives
    log sum exp of the scores; a query that sees nothing gets out 0, lse -inf."""
    c = cache.descriptor                         # first: it looks at data anew
    dt, dev, shape = q.dtype, cache._device, q.shape
    if dt not in _KV_DTYPE:
        raise TypeError(f"q: dtype {dt} (float32 or bfloat16 expected)")
    if len(shape) != 3 or shape[2] != cache._dim:
        raise ValueError(f"q: shape {tuple(shape)}, expected (rows, q_heads, {cache.dim})")
    rows, q_heads, _ = shape
    if q_heads == 0 or q_heads % cache._heads:
        raise ValueError(f"q: {q_heads} heads, a multiple of the cache's {cache.heads} expected")
    code, unit = _KV_DTYPE[dt]
    qs, os = _rows(q, "q", shape, dt, unit, dev), _rows(out, "out", shape, dt, unit, dev)
    _spread(out, "out")
    batch = kv_len.numel()
    i32 = torch.int32
    if kv_len.dtype is not i32 or kv_len.dim() != 1 or kv_len.device != dev or not kv_len.is_contiguous():
        raise ValueError(f"kv_len: shape {tuple(kv_len.shape)} of {kv_len.dtype} on {kv_len.device}, expected contiguous "
                         f"torch.int32 (batch,) on {dev}")
    if q_start.dtype is not i32 or q_start.shape != (batch + 1,) or q_start.device != dev or not q_start.is_contiguous():
        raise ValueError(f"q_start: shape {tuple(q_start.shape)} of {q_start.dtype} on {q_start.device}, expected "
                         f"contiguous torch.int32 ({batch + 1},) on {dev}")
    pages = table.shape
    if table.dtype is not i32 or len(pages) != 2 or pages[0] != batch or table.device != dev or not table.is_contiguous():
        raise ValueError(f"table: shape {tuple(table.shape)} of {table.dtype} on {table.device}, expected contiguous "
                         f"torch.int32 ({batch}, pages) on {dev}")
    if window > _I32_MAX:                        # more than any sequence has tokens
        window = _I32_MAX
    # the call's 32-bit sizes, of which ctypes would keep the low bits: none negative or above 2^31 - 1
    if (max_q | max_kv | window | rows | q_heads | batch | pages[1]) >> 31:
        raise ValueError(f"max_q {max_q}, max_kv {max_kv}, window {window}, {rows} rows, {q_heads} heads, batch {batch}, "
                         f"{pages[1]} pages: none may be negative or above 2^31 - 1")
    if scale is None:
        scale = 1.0 / math.sqrt(cache.dim)
    elif not math.isfinite(scale):
        raise ValueError(f"scale {scale}: a finite number expected")
    lat, lts = None, 0
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != (rows, q_heads) or lse.device != dev \
                or (q_heads > 1 and lse.stride(1) != 1):
            raise ValueError(f"lse: shape {tuple(lse.shape)} of {lse.dtype} on {lse.device}, expected torch.float32 "
                             f"({rows}, {q_heads}) on {dev}, heads adjacent")
        _spread(lse, "lse")
        lat, lts = lse.data_ptr(), (lse.stride(0) if rows > 1 else 0)
    if ws is not None and (ws.dtype is not torch.uint8 or ws.device != dev or not ws.is_contiguous()):
        raise ValueError(f"ws: dtype {ws.dtype} on {ws.device}, expected contiguous torch.uint8 on {dev}")
    if cache._gpu is None:
        raise ValueError("device tensor expected (no CPU path)")
    if rows == 0 or batch == 0 or max_q == 0:
        return
    if ws is None:
        need = int(_lib.load().nc_kv_workspace_bytes(c, code, q_heads, batch, max_q, max_kv))
        if need:
            # on the call's own stream: freed memory is handed out again in that stream's order
            on = torch.cuda.current_stream(dev) if stream is None else (
                stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=dev))
            with torch.cuda.stream(on):
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
    a = NcKvAttn(*qs, *os, lat, lts, q_start.data_ptr(), kv_len.data_ptr(), table.data_ptr(), pages[1], batch, rows,
                 q_heads, max_q, max_kv, 1 if causal else 0, window, scale)
    wat, wn = (None, 0) if ws is None else (ws.data_ptr(), ws.numel())
    _kv_call(cache, "nc_kv_attention", _lib.load().nc_kv_attention, c, a, code, wat, wn, _kv_stream(stream, cache._gpu))
