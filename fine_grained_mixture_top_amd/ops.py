"""Single operators around the experts' products (include/moe_ops.h): tokens
sorted by expert and back, E4M3 products with a scale per block of 128, SwiGLU
quantized for the next product.

Argument marshalling only, as in ``binding``: torch tensors in caller-owned
device memory, ``MoEError`` on a non-zero status.  Tensors whose type, shape,
layout or device an operator cannot take raise ``ValueError`` before the call.
Codes are ``torch.float8_e4m3fn`` or ``torch.uint8`` tensors.  Calls run on
``stream``, or on the current stream of the tensors' device.

    plan = ops.Plan(T, K, E)                      # buffers, kept between calls
    ops.moe_sort(plan, topk_idx)                  # int32 [T, K]
    ops.moe_permute_fp8(plan, x, xq, xs)          # rows by expert, 8-bit
    ops.moe_fp8_mm(plan, xq, xs, w1q, w1s, h)     # h [cap, 2n]
    ops.moe_swiglu_fp8(h, aq, as_, plan=plan)
    ops.moe_fp8_mm(plan, aq, as_, w2q, w2s, y)
    ops.moe_unpermute(plan, y, topk_gate, o)      # o [T, d]
"""
from __future__ import annotations

import ctypes

import torch

from . import binding as B

(MOE_OPS_K_SORT, MOE_OPS_K_PERMUTE, MOE_OPS_K_PERMUTE_FP8, MOE_OPS_K_UNPERMUTE, MOE_OPS_K_UNPERMUTE_BWD,
 MOE_OPS_K_QUANT_ROWS, MOE_OPS_K_QUANT_WEIGHTS, MOE_OPS_K_QUANT_COLS, MOE_OPS_K_FP8_MM, MOE_OPS_K_FP8_WGRAD,
 MOE_OPS_K_SWIGLU_FP8, MOE_OPS_K_SWIGLU_BWD) = range(29, 41)
KERNEL_NAMES = B.KERNEL_NAMES + ["sort", "permute", "permute_fp8", "unpermute", "unpermute_bwd", "quant_rows",
                                 "quant_weights", "quant_cols", "fp8_mm", "fp8_wgrad", "swiglu_fp8", "swiglu_bwd_rows"]
MOE_MM_GATHER = 1
MOE_MM_SB_OUT_MAJOR = 2

BLOCK = 128
E4M3 = torch.float8_e4m3fn
_CODES = (E4M3, torch.uint8)
_DTYPE = {torch.float32: B.MOE_F32, torch.bfloat16: B.MOE_BF16}


class MoePlanDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("K", ctypes.c_int32), ("E", ctypes.c_int32), ("align", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("reserved", ctypes.c_uint32), ("profile", ctypes.POINTER(B.MoeProfile))]


class MoePlan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("offsets", "counts", "row_token", "slot_row")]


class MoeMmDesc(ctypes.Structure):
    _fields_ = [("a_rows", ctypes.c_int32), ("rows", ctypes.c_int32), ("rows_used", ctypes.c_int32),
                ("E", ctypes.c_int32), ("K", ctypes.c_int32), ("N", ctypes.c_int32), ("out", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("profile", ctypes.POINTER(B.MoeProfile))]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded HIP library with the operators' signatures (raises when it has not been built)."""
    global _lib
    if _lib is None:
        L = B.lib()
        vp, sz, i32, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64
        pd, pp = ctypes.POINTER(MoePlanDesc), ctypes.POINTER(MoePlan)
        pm, prof = ctypes.POINTER(MoeMmDesc), ctypes.POINTER(B.MoeProfile)
        sig = {
            "moe_plan_rows": ([pd], sz),
            "moe_sort_workspace_bytes": ([pd], sz),
            "moe_sort": ([pd, vp, pp, vp, sz, vp], i32),
            "moe_permute": ([pd, pp, i32, i32, vp, vp, vp], i32),
            "moe_permute_fp8": ([pd, pp, i32, i32, vp, vp, vp, vp], i32),
            "moe_permute_bwd": ([pd, pp, i32, i32, vp, vp, vp], i32),
            "moe_unpermute": ([pd, pp, i32, i32, vp, vp, vp, vp], i32),
            "moe_unpermute_bwd": ([pd, pp, i32, i32, vp, vp, vp, vp, vp, vp], i32),
            "moe_fp8_quant_rows": ([pd, pp, i32, i64, i32, vp, vp, vp, prof, vp], i32),
            "moe_fp8_quant_weights": ([i32, i32, i32, i32, vp, vp, vp, vp, prof, vp], i32),
            "moe_fp8_quant_cols": ([pd, pp, i32, i32, i32, vp, vp, vp, vp], i32),
            "moe_fp8_mm": ([pm, vp, vp, vp, vp, pp, vp, vp], i32),
            "moe_fp8_wgrad": ([pd, pp, i32, i32, i32, vp, vp, vp, vp, vp, vp], i32),
            "moe_swiglu_fp8": ([pd, pp, i32, i64, i32, vp, vp, vp, vp, prof, vp], i32),
            "moe_swiglu_bwd": ([pd, pp, i32, i64, i32, vp, vp, vp, prof, vp], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes, fn.restype = args, res
        _lib = L
    return _lib


def blocks(n: int) -> int:
    """Blocks of 128 along a length (the last one may be shorter)."""
    return -(-n // BLOCK)


def _need(name, t, dtypes, shape, device):
    """The address of a contiguous tensor of one of the types, of the shape, on the device."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.device == device:
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} is not one of {', '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} where {tuple(shape)} is needed")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    raise ValueError(f"{name}: on {t.device}, the call is on {device}")


_VALUES = (torch.float32, torch.bfloat16)
_F32 = (torch.float32,)


_INT32 = 2 ** 31 - 1  # ctypes cuts a larger size off without a word


def _shape(name, t, dims=2):
    """The sizes of a tensor of `dims` dimensions, a row's within 32 bits (_need checks the rest)."""
    if isinstance(t, torch.Tensor):
        s = t.shape
        if len(s) == dims:
            if s[1] > _INT32 or s[-1] > _INT32:
                raise ValueError(f"{name}: shape {tuple(s)}, sizes past 32 bits")
            return s
    raise ValueError(f"{name}: a {dims}-dimensional tensor is needed")


# the current stream's handle without building a Stream object (2 us a call), and
# the current device without the check that the GPU is in use (a tensor is on it
# by then), where this torch has them
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(fn, device, stream, *args):
    """fn(*args, stream) with `device` current; raises on a non-zero status."""
    if device.type != "cuda":
        raise ValueError(f"{fn}: the call is on {device}, a GPU is needed")
    index = device.index
    if index is not None and index != _current_device():
        with torch.cuda.device(device):
            return _call(fn, device, stream, *args)
    if stream is None:
        handle = _raw_stream(index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    else:
        if stream.device != device:
            raise ValueError(f"stream on {stream.device}, the call is on {device}")
        handle = stream.cuda_stream
    status = getattr(_lib or lib(), fn)(*args, handle)
    if status:
        raise B.MoEError(fn, status)


class Plan:
    """Which rows belong to which expert: the sizes of a call sequence, the
    plan's device buffers (written by ``moe_sort``) and its workspace.

    offsets [E+1], counts [E], row_token [cap], slot_row [T, K] (int32).  align:
    every expert's segment starts at a multiple of it (128 for the weight
    gradients).  A plan belongs to one sequence of calls at a time."""

    def __init__(self, T: int, K: int, E: int, align: int = 1, device="cuda"):
        device = torch.device(device)
        if device.type == "cuda" and device.index is None:
            device = torch.device("cuda", torch.cuda.current_device())
        if max(T, K, E, align) > _INT32 or min(T, K, E, align) < -_INT32:
            raise B.MoEError("moe_plan_rows", B.MOE_ESHAPE)
        self.T, self.K, self.E, self.align, self.device = T, K, E, align, device
        self.desc = MoePlanDesc(T, K, E, align, 0, 0, None)
        self.cap = int(lib().moe_plan_rows(ctypes.byref(self.desc)))
        if self.cap == 0 and T != 0:
            raise B.MoEError("moe_plan_rows", B.MOE_EINVAL if min(T, K, E, align) < 1 else B.MOE_ESHAPE)
        z = lambda *n: torch.zeros(n, dtype=torch.int32, device=device)  # noqa: E731
        self.offsets, self.counts, self.row_token, self.slot_row = z(E + 1), z(E), z(self.cap), z(T, K)
        self.ws = torch.empty(max(int(lib().moe_sort_workspace_bytes(ctypes.byref(self.desc))), 256),
                              dtype=torch.uint8, device=device)
        self.c = MoePlan(self.offsets.data_ptr(), self.counts.data_ptr(), self.row_token.data_ptr(),
                         self.slot_row.data_ptr())
        self._d, self._p = ctypes.byref(self.desc), ctypes.byref(self.c)

    def attach(self, profiler: B.Profiler):
        """Records launch timing of the calls that take this plan."""
        profiler.attach(self.desc)

    def detach(self):
        self.desc.profile = None


def _plan_or_none(plan):
    return (None, None) if plan is None else (plan._d, plan._p)


def _profile(plan):
    return None if plan is None else plan.desc.profile


def _plan_rows(name, plan, R, device):
    if plan is not None and (R != plan.cap or device != plan.device):
        raise ValueError(f"{name}: {R} rows on {device}, the plan has {plan.cap} on {plan.device}")


def moe_sort(plan: Plan, expert_idx, stream=None):
    """Sorts the choices expert_idx [T, K] (int32; ids outside 0..E-1 are dropped) into the plan."""
    idx = _need("expert_idx", expert_idx, (torch.int32,), (plan.T, plan.K), plan.device)
    _call("moe_sort", plan.device, stream, plan._d, idx, plan._p, plan.ws.data_ptr(), plan.ws.numel())


def moe_permute(plan: Plan, x, xp, stream=None):
    """xp[slot_row[t, k]] = x[t]."""
    d = _shape("x", x)[1]
    px = _need("x", x, _VALUES, (plan.T, d), plan.device)
    pxp = _need("xp", xp, (x.dtype,), (plan.cap, d), plan.device)
    _call("moe_permute", plan.device, stream, plan._d, plan._p, _DTYPE[x.dtype], d, px, pxp)


def moe_permute_fp8(plan: Plan, x, q, s, stream=None):
    """The rows of moe_permute as codes q [cap, d] and scales s [cap, ceil(d/128)]."""
    d = _shape("x", x)[1]
    px = _need("x", x, _VALUES, (plan.T, d), plan.device)
    pq = _need("q", q, _CODES, (plan.cap, d), plan.device)
    ps = _need("s", s, _F32, (plan.cap, blocks(d)), plan.device)
    _call("moe_permute_fp8", plan.device, stream, plan._d, plan._p, _DTYPE[x.dtype], d, px, pq, ps)


def moe_permute_bwd(plan: Plan, dxp, dx, stream=None):
    """dx[t] = sum over k of dxp[slot_row[t, k]]."""
    d = _shape("dxp", dxp)[1]
    pg = _need("dxp", dxp, _VALUES, (plan.cap, d), plan.device)
    px = _need("dx", dx, (dxp.dtype,), (plan.T, d), plan.device)
    _call("moe_permute_bwd", plan.device, stream, plan._d, plan._p, _DTYPE[dxp.dtype], d, pg, px)


def moe_unpermute(plan: Plan, y, w, o, stream=None):
    """o[t] = sum over k of w[t, k] y[slot_row[t, k]] (w fp32)."""
    d = _shape("y", y)[1]
    py = _need("y", y, _VALUES, (plan.cap, d), plan.device)
    pw = _need("w", w, _F32, (plan.T, plan.K), plan.device)
    po = _need("o", o, (y.dtype,), (plan.T, d), plan.device)
    _call("moe_unpermute", plan.device, stream, plan._d, plan._p, _DTYPE[y.dtype], d, py, pw, po)


def moe_unpermute_bwd(plan: Plan, d_o, y, w, dy, dw, stream=None):
    """dy[slot_row[t, k]] = w[t, k] d_o[t]; dw[t, k] = <d_o[t], y[slot_row[t, k]]> (0 for a dropped choice).
    dw None: y is not read (may be None); dy None: w is not read."""
    d = _shape("d_o", d_o)[1]
    dt = (d_o.dtype,)
    pdo = _need("d_o", d_o, _VALUES, (plan.T, d), plan.device)
    py = None if y is None else _need("y", y, dt, (plan.cap, d), plan.device)
    pw = None if w is None else _need("w", w, _F32, (plan.T, plan.K), plan.device)
    pdy = None if dy is None else _need("dy", dy, dt, (plan.cap, d), plan.device)
    pdw = None if dw is None else _need("dw", dw, _F32, (plan.T, plan.K), plan.device)
    if (pdy is None and pdw is None) or (pdw is not None and py is None) or (pdy is not None and pw is None):
        raise ValueError("dy needs w, dw needs y, and one of dy and dw is needed")
    _call("moe_unpermute_bwd", plan.device, stream, plan._d, plan._p, _DTYPE[d_o.dtype], d, pdo, py, pw, pdy, pdw)


def moe_fp8_quant_rows(src, q, s, plan: Plan = None, stream=None):
    """src [R, C] -> codes q [R, C] and scales s [R, ceil(C/128)]; with a plan (R = plan.cap) its rows only."""
    R, C = _shape("src", src)
    _plan_rows("src", plan, R, src.device)
    p = _need("src", src, _VALUES, (R, C), src.device)
    pq = _need("q", q, _CODES, (R, C), src.device)
    ps = _need("s", s, _F32, (R, blocks(C)), src.device)
    d, c = _plan_or_none(plan)
    _call("moe_fp8_quant_rows", src.device, stream, d, c, _DTYPE[src.dtype], R, C, p, pq, ps, _profile(plan))


def moe_fp8_quant_weights(w, q, qt, s, stream=None):
    """w [E, K, N] -> codes q [E, K, N] and qt [E, N, K] (either may be None), scales s per 128 x 128 block."""
    E, K, N = _shape("w", w, 3)
    if q is None and qt is None:
        raise ValueError("one of q and qt is needed")
    p = _need("w", w, _VALUES, (E, K, N), w.device)
    pq = None if q is None else _need("q", q, _CODES, (E, K, N), w.device)
    pt = None if qt is None else _need("qt", qt, _CODES, (E, N, K), w.device)
    ps = _need("s", s, _F32, (E, blocks(K), blocks(N)), w.device)
    _call("moe_fp8_quant_weights", w.device, stream, _DTYPE[w.dtype], E, K, N, p, pq, pt, ps, None)


def column_buffers(plan: Plan, C: int):
    """Buffers of moe_fp8_quant_cols for C columns: codes [cap//128, C, 128], scales [cap//128, C]."""
    n = plan.cap // BLOCK
    return (torch.zeros((n, C, BLOCK), dtype=torch.uint8, device=plan.device).view(E4M3),
            torch.zeros((n, C), dtype=torch.float32, device=plan.device))


def moe_fp8_quant_cols(plan: Plan, src, q, s, gather: bool = False, stream=None):
    """Blocks of 128 rows per column and segment: src [cap, C], or with gather [T, C] read through row_token;
    q [cap//128, C, 128], s [cap//128, C].  The plan's align is a multiple of 128."""
    C = _shape("src", src)[1]
    p = _need("src", src, _VALUES, (plan.T if gather else plan.cap, C), plan.device)
    n = plan.cap // BLOCK
    pq = _need("q", q, _CODES, (n, C, BLOCK), plan.device)
    ps = _need("s", s, _F32, (n, C), plan.device)
    _call("moe_fp8_quant_cols", plan.device, stream, plan._d, plan._p, _DTYPE[src.dtype], C, int(gather), p, pq, ps)


_mm_descs = {}  # (sizes, type, flags) -> descriptor without a profile: building one takes 1.5 us


def _mm_desc(profile, *key):
    if profile:
        return MoeMmDesc(*key, 0, profile)
    d = _mm_descs.get(key)
    if d is None:
        if len(_mm_descs) >= 1024:
            _mm_descs.clear()
        d = _mm_descs[key] = MoeMmDesc(*key, 0, None)
    return d


def moe_fp8_mm(plan, a, sa, b, sb, c, gather: bool = False, sb_out_major: bool = False, stream=None):
    """c[r] = (a sa)[r] (b sb)[e]^T for the rows r of expert e's segment.

    a [cap, K] codes (gather: [T, K], row r reads a's row row_token[r]), sa [., ceil(K/128)]; b [E, N, K]
    codes; sb [E, ceil(K/128), ceil(N/128)], or with sb_out_major [E, ceil(N/128), ceil(K/128)]; c [cap, N]
    fp32 or bf16.  plan None: dense, a [R, K], b [N, K] or [1, N, K], c [R, N]."""
    rows_a, K = _shape("a", a)
    rows, N = _shape("c", c)
    if rows_a > _INT32 or rows > _INT32:
        raise ValueError(f"a and c: {rows_a} and {rows} rows, sizes past 32 bits")
    dev = a.device
    if plan is None:
        if gather:
            raise ValueError("gather needs a plan")
        E, want, profile = 1, rows, None
    else:
        E, want, profile = plan.E, plan.T if gather else plan.cap, plan.desc.profile
        _plan_rows("c", plan, rows, dev)
    kb, nb = blocks(K), blocks(N)
    shape_b, shape_sb = (N, K), (nb, kb) if sb_out_major else (kb, nb)
    if plan is not None or (isinstance(b, torch.Tensor) and b.dim() == 3):
        shape_b = (E, *shape_b)
    if plan is not None or (isinstance(sb, torch.Tensor) and sb.dim() == 3):
        shape_sb = (E, *shape_sb)
    pa = _need("a", a, _CODES, (want, K), dev)
    psa = _need("sa", sa, _F32, (want, kb), dev)
    pb = _need("b", b, _CODES, shape_b, dev)
    psb = _need("sb", sb, _F32, shape_sb, dev)
    pc = _need("c", c, _VALUES, (rows, N), dev)
    flags = (MOE_MM_GATHER if gather else 0) | (MOE_MM_SB_OUT_MAJOR if sb_out_major else 0)
    used = 0 if plan is None else plan.T * plan.K
    d = _mm_desc(profile, rows_a, rows, used, E, K, N, _DTYPE[c.dtype], flags)
    _call("moe_fp8_mm", dev, stream, ctypes.byref(d), pa, psa, pb, psb, None if plan is None else plan._p, pc)


def moe_fp8_wgrad(plan: Plan, a, sa, b, sb, dw, stream=None):
    """dw[e] = sum over expert e's rows of (a sa)^T (b sb): a [cap//128, M, 128], sa [cap//128, M], b and sb
    likewise with N columns, from moe_fp8_quant_cols; dw [E, M, N] fp32 or bf16."""
    M = _shape("a", a, 3)[1]
    N = _shape("b", b, 3)[1]
    n = plan.cap // BLOCK
    pa = _need("a", a, _CODES, (n, M, BLOCK), plan.device)
    psa = _need("sa", sa, _F32, (n, M), plan.device)
    pb = _need("b", b, _CODES, (n, N, BLOCK), plan.device)
    psb = _need("sb", sb, _F32, (n, N), plan.device)
    pw = _need("dw", dw, _VALUES, (plan.E, M, N), plan.device)
    _call("moe_fp8_wgrad", plan.device, stream, plan._d, plan._p, M, N, _DTYPE[dw.dtype], pa, psa, pb, psb, pw)


def moe_swiglu_fp8(h, q, s, a=None, plan: Plan = None, stream=None):
    """A = silu(G) U of h [R, 2n] = [G | U] -> codes q [R, n], scales s [R, ceil(n/128)]; a [R, n] (h's type)
    when given.  With a plan (R = plan.cap) its rows only."""
    R, n2 = _shape("h", h)
    n = n2 // 2
    _plan_rows("h", plan, R, h.device)
    ph = _need("h", h, _VALUES, (R, 2 * n), h.device)
    pq = _need("q", q, _CODES, (R, n), h.device)
    ps = _need("s", s, _F32, (R, blocks(n)), h.device)
    pa = None if a is None else _need("a", a, (h.dtype,), (R, n), h.device)
    d, c = _plan_or_none(plan)
    _call("moe_swiglu_fp8", h.device, stream, d, c, _DTYPE[h.dtype], R, n, ph, pq, ps, pa, _profile(plan))


def moe_swiglu_bwd(da, h, dh, plan: Plan = None, stream=None):
    """dh [R, 2n] = (da U s (1 + G (1 - s)), da silu(G)), s = sigmoid(G), from da [R, n] and h [R, 2n]."""
    R, n2 = _shape("h", h)
    n = n2 // 2
    _plan_rows("h", plan, R, h.device)
    ph = _need("h", h, _VALUES, (R, 2 * n), h.device)
    pa = _need("da", da, (h.dtype,), (R, n), h.device)
    pd = _need("dh", dh, (h.dtype,), (R, 2 * n), h.device)
    d, c = _plan_or_none(plan)
    _call("moe_swiglu_bwd", h.device, stream, d, c, _DTYPE[h.dtype], R, n, pa, ph, pd, _profile(plan))
