"""Host-side checks of the single operators' C ABI and binding (no GPU):
exports, constants, sizes, refusals before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

from fine_grained_mixture_top_amd import binding as B
from fine_grained_mixture_top_amd import ops

import ops_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_ops.h")
P = 4096  # an aligned address that no refused call touches


def desc(T=8, K=2, E=4, align=1, flags=0, reserved=0):
    return ops.MoePlanDesc(T, K, E, align, flags, reserved, None)


def plan(**kw):
    a = dict(offsets=P, counts=P, row_token=P, slot_row=P)
    a.update(kw)
    return ops.MoePlan(*[a[f] for f in ("offsets", "counts", "row_token", "slot_row")])


def ref(x):
    return ctypes.byref(x)


def test_header_functions_and_constants():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    lib = ops.lib()
    assert len(names) == 15
    for n in names:
        assert hasattr(lib, n) and getattr(lib, n).argtypes is not None, n
    consts = dict(re.findall(r"#define\s+(MOE_[A-Z0-9_]+)\s+(\d+)u?", text))
    assert len(consts) == 14
    for k, v in consts.items():
        assert getattr(ops, k) == int(v), k
    assert len(ops.KERNEL_NAMES) == ops.MOE_OPS_K_SWIGLU_BWD + 1


def test_plan_sizes():
    lib = ops.lib()
    assert lib.moe_plan_rows(ref(desc())) == 16
    assert lib.moe_plan_rows(ref(desc(T=5, K=2, E=8, align=128))) == 10 + 8 * 127
    assert lib.moe_plan_rows(ref(desc(T=1, K=2, E=8, align=128))) == 2 + 2 * 127  # at most T*K segments have rows
    assert lib.moe_plan_rows(ref(desc(T=0))) == 0
    assert lib.moe_sort_workspace_bytes(ref(desc())) == 0
    n = lib.moe_sort_workspace_bytes(ref(desc(T=40000, K=8, E=300)))
    assert n > 0 and n % 256 == 0


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), B.MOE_EINVAL), (dict(K=0), B.MOE_EINVAL), (dict(E=0), B.MOE_EINVAL), (dict(align=0), B.MOE_EINVAL),
    (dict(flags=1), B.MOE_EINVAL), (dict(reserved=1), B.MOE_EINVAL), (dict(T=1 << 24), B.MOE_ESHAPE),
    (dict(K=1025), B.MOE_ESHAPE), (dict(E=1025), B.MOE_ESHAPE), (dict(align=257), B.MOE_ESHAPE),
    (dict(T=(1 << 24) - 1, K=65), B.MOE_ESHAPE),
])
def test_plan_descriptors_refused(kw, code):
    lib, d, p = ops.lib(), desc(**kw), plan()
    assert lib.moe_plan_rows(ref(d)) == 0 and lib.moe_sort_workspace_bytes(ref(d)) == 0
    assert lib.moe_sort(ref(d), P, ref(p), P, 1 << 30, None) == code
    assert lib.moe_permute(ref(d), ref(p), B.MOE_BF16, 128, P, P, None) == code
    assert lib.moe_unpermute_bwd(ref(d), ref(p), B.MOE_BF16, 128, P, P, P, P, P, None) == code
    assert lib.moe_fp8_quant_cols(ref(d), ref(p), B.MOE_BF16, 128, 0, P, P, P, None) == code
    assert lib.moe_fp8_wgrad(ref(d), ref(p), 128, 128, B.MOE_BF16, P, P, P, P, P, None) == code


def test_sort_refusals():
    lib, d, p = ops.lib(), desc(), plan()
    assert lib.moe_sort(None, P, ref(p), P, 0, None) == B.MOE_EINVAL
    assert lib.moe_sort(ref(d), None, ref(p), P, 0, None) == B.MOE_EINVAL
    assert lib.moe_sort(ref(d), P, None, P, 0, None) == B.MOE_EINVAL
    for f in ("offsets", "counts", "row_token", "slot_row"):
        assert lib.moe_sort(ref(d), P, ref(plan(**{f: 0})), P, 0, None) == B.MOE_EINVAL
    big = desc(T=40000, K=8, E=300)
    need = lib.moe_sort_workspace_bytes(ref(big))
    assert lib.moe_sort(ref(big), P, ref(p), P, need - 1, None) == B.MOE_EWORKSPACE
    assert lib.moe_sort(ref(big), P, ref(p), P + 16, need, None) == B.MOE_EINVAL
    assert lib.moe_sort(ref(big), P, ref(p), None, need, None) == B.MOE_EINVAL


def test_row_moves_refused():
    lib, d, p = ops.lib(), desc(), plan()
    for dt, width, code in ((7, 128, B.MOE_EDTYPE), (B.MOE_BF16, 0, B.MOE_EINVAL), (B.MOE_BF16, 24, B.MOE_ESHAPE),
                            (B.MOE_BF16, (1 << 20) + 16, B.MOE_ESHAPE)):
        assert lib.moe_permute(ref(d), ref(p), dt, width, P, P, None) == code
        assert lib.moe_permute_fp8(ref(d), ref(p), dt, width, P, P, P, None) == code
        assert lib.moe_permute_bwd(ref(d), ref(p), dt, width, P, P, None) == code
        assert lib.moe_unpermute(ref(d), ref(p), dt, width, P, P, P, None) == code
        assert lib.moe_unpermute_bwd(ref(d), ref(p), dt, width, P, P, P, P, P, None) == code
    bf = B.MOE_BF16
    for x, y in ((None, P), (P, None), (P + 8, P), (P, P + 8)):
        assert lib.moe_permute(ref(d), ref(p), bf, 128, x, y, None) == B.MOE_EINVAL
        assert lib.moe_permute_bwd(ref(d), ref(p), bf, 128, x, y, None) == B.MOE_EINVAL
        assert lib.moe_permute_fp8(ref(d), ref(p), bf, 128, x, y, P, None) == B.MOE_EINVAL
        assert lib.moe_unpermute(ref(d), ref(p), bf, 128, x, P, y, None) == B.MOE_EINVAL
    assert lib.moe_unpermute(ref(d), ref(p), bf, 128, P, None, P, None) == B.MOE_EINVAL
    bwd = lambda *a: lib.moe_unpermute_bwd(ref(d), ref(p), bf, 128, *a, None)  # noqa: E731
    assert bwd(P, P, P, None, None) == B.MOE_EINVAL      # nothing to write
    assert bwd(P, None, P, P, P) == B.MOE_EINVAL         # dw without y
    assert bwd(P, P, None, P, P) == B.MOE_EINVAL         # dy without w
    assert bwd(None, P, P, P, P) == B.MOE_EINVAL
    assert bwd(P, P, P, P + 4, P) == B.MOE_EINVAL
    assert lib.moe_permute(ref(d), ref(plan(slot_row=0)), bf, 128, P, P, None) == B.MOE_EINVAL
    # no tokens: nothing to do, whatever the buffers
    assert lib.moe_permute(ref(desc(T=0)), ref(plan(slot_row=0, row_token=0)), bf, 128, None, None, None) == B.MOE_OK


def test_quantizers_refused():
    lib, d, p, bf = ops.lib(), desc(align=128), plan(), B.MOE_BF16
    rows = lib.moe_plan_rows(ref(d))
    q = lambda *a: lib.moe_fp8_quant_rows(*a, None, None)  # noqa: E731
    assert q(None, None, 9, 4, 128, P, P, P) == B.MOE_EDTYPE
    assert q(None, None, bf, -1, 128, P, P, P) == B.MOE_EINVAL
    assert q(None, None, bf, 4, 100, P, P, P) == B.MOE_ESHAPE
    assert q(None, None, bf, 1 << 37, 128, P, P, P) == B.MOE_ESHAPE
    assert q(None, None, bf, 4, 128, None, P, P) == B.MOE_EINVAL
    assert q(None, None, bf, 4, 128, P, P + 1, P) == B.MOE_EINVAL
    assert q(None, None, bf, 4, 128, P, P, None) == B.MOE_EINVAL
    assert q(None, None, bf, 0, 128, None, None, None) == B.MOE_OK
    assert q(ref(d), None, bf, rows, 128, P, P, P) == B.MOE_EINVAL      # a descriptor without its plan
    assert q(None, ref(p), bf, rows, 128, P, P, P) == B.MOE_EINVAL
    assert q(ref(d), ref(p), bf, rows - 1, 128, P, P, P) == B.MOE_EINVAL  # not the plan's rows
    w = lambda *a: lib.moe_fp8_quant_weights(*a, None, None)  # noqa: E731
    assert w(9, 2, 128, 128, P, P, P, P) == B.MOE_EDTYPE
    assert w(bf, 0, 128, 128, P, P, P, P) == B.MOE_EINVAL
    assert w(bf, 2, 120, 128, P, P, P, P) == B.MOE_ESHAPE
    assert w(bf, 2, 128, 8, P, P, P, P) == B.MOE_ESHAPE
    assert w(bf, 1025, 128, 128, P, P, P, P) == B.MOE_ESHAPE
    assert w(bf, 1024, 1 << 20, 1 << 20, P, P, P, P) == B.MOE_ESHAPE
    assert w(bf, 2, 128, 128, P, None, None, P) == B.MOE_EINVAL
    assert w(bf, 2, 128, 128, P, P + 8, None, P) == B.MOE_EINVAL
    c = lambda dd, *a: lib.moe_fp8_quant_cols(ref(dd), ref(p), *a, None)  # noqa: E731
    assert c(desc(align=64), bf, 128, 0, P, P, P) == B.MOE_ESHAPE
    assert c(desc(align=192), bf, 128, 0, P, P, P) == B.MOE_ESHAPE
    assert c(d, bf, 24, 0, P, P, P) == B.MOE_ESHAPE
    assert c(d, bf, 128, 0, P, None, P) == B.MOE_EINVAL
    s = lambda *a: lib.moe_swiglu_fp8(*a, None, None)  # noqa: E731
    assert s(None, None, 5, 4, 128, P, P, P, None) == B.MOE_EDTYPE
    assert s(None, None, bf, 4, 24, P, P, P, None) == B.MOE_ESHAPE
    assert s(None, None, bf, 4, 128, P, P, P, P + 2) == B.MOE_EINVAL
    assert s(ref(d), ref(p), bf, 4, 128, P, P, P, None) == B.MOE_EINVAL
    b = lambda *a: lib.moe_swiglu_bwd(*a, None, None)  # noqa: E731
    assert b(None, None, bf, 4, 8, P, P, P) == B.MOE_ESHAPE
    assert b(None, None, bf, 4, 128, P, None, P) == B.MOE_EINVAL
    assert b(None, None, bf, 0, 128, None, None, None) == B.MOE_OK


def mm(a_rows=8, rows=8, rows_used=0, E=2, K=128, N=128, out=B.MOE_BF16, flags=0, reserved=0):
    return ops.MoeMmDesc(a_rows, rows, rows_used, E, K, N, out, flags, reserved, None)


@pytest.mark.parametrize("kw,code", [
    (dict(flags=4), B.MOE_EINVAL), (dict(reserved=1), B.MOE_EINVAL), (dict(a_rows=-1), B.MOE_EINVAL),
    (dict(rows=-1, a_rows=-1), B.MOE_EINVAL), (dict(rows_used=-1), B.MOE_EINVAL), (dict(rows_used=9), B.MOE_EINVAL), (dict(E=0), B.MOE_EINVAL), (dict(out=3), B.MOE_EDTYPE),
    (dict(K=0), B.MOE_EINVAL), (dict(K=72), B.MOE_ESHAPE), (dict(N=24), B.MOE_ESHAPE),
    (dict(K=(1 << 20) + 16), B.MOE_ESHAPE), (dict(E=1025), B.MOE_ESHAPE), (dict(K=1 << 16, N=1 << 15), B.MOE_ESHAPE),
    (dict(a_rows=9), B.MOE_EINVAL), (dict(a_rows=0, flags=ops.MOE_MM_GATHER), B.MOE_EINVAL),
    (dict(a_rows=1 << 24, K=128, flags=ops.MOE_MM_GATHER), B.MOE_ESHAPE),
])
def test_mm_refused(kw, code):
    assert ops.lib().moe_fp8_mm(ref(mm(**kw)), P, P, P, P, ref(plan()), P, None) == code


def test_mm_pointers_refused():
    lib, p = ops.lib(), plan()
    call = lambda d, *a, pl=p: lib.moe_fp8_mm(ref(d), *a[:4], pl and ref(pl), a[4], None)  # noqa: E731
    for i in range(5):
        for bad in ((None, P + 2) if i in (1, 3) else (None, P + 8)):
            a = [P] * 5
            a[i] = bad
            assert call(mm(), *a) == B.MOE_EINVAL
    assert call(mm(), *[P] * 5, pl=None) == B.MOE_EINVAL                 # several experts without a plan
    assert call(mm(E=1, flags=ops.MOE_MM_GATHER), *[P] * 5, pl=None) == B.MOE_EINVAL
    assert call(mm(), *[P] * 5, pl=plan(counts=0)) == B.MOE_EINVAL
    assert call(mm(flags=ops.MOE_MM_GATHER), *[P] * 5, pl=plan(row_token=0)) == B.MOE_EINVAL
    assert call(mm(rows=0, a_rows=0), *[None] * 5) == B.MOE_OK
    assert lib.moe_fp8_mm(None, P, P, P, P, ref(p), P, None) == B.MOE_EINVAL


def test_wgrad_refused():
    lib, p, bf = ops.lib(), plan(), B.MOE_BF16
    call = lambda d, M, N, out, *a: lib.moe_fp8_wgrad(ref(d), ref(p), M, N, out, *a, None)  # noqa: E731
    d = desc(align=128)
    assert call(desc(align=1), 128, 128, bf, *[P] * 5) == B.MOE_ESHAPE
    assert call(d, 128, 128, 5, *[P] * 5) == B.MOE_EDTYPE
    assert call(d, 24, 128, bf, *[P] * 5) == B.MOE_ESHAPE
    assert call(d, 128, 24, bf, *[P] * 5) == B.MOE_ESHAPE
    for i in range(5):
        a = [P] * 5
        a[i] = None
        assert call(d, 128, 128, bf, *a) == B.MOE_EINVAL
        a[i] = P + (2 if i in (1, 3) else 8)
        assert call(d, 128, 128, bf, *a) == B.MOE_EINVAL


def test_binding_refuses_tensors():
    """Types, shapes, layouts and devices that an operator cannot take never reach the library."""
    p = ops.Plan(4, 2, 8, align=128, device="cpu")
    idx = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="expert_idx"):
        ops.moe_sort(p, idx.long())
    with pytest.raises(ValueError, match="shape"):
        ops.moe_sort(p, idx[:3])
    with pytest.raises(ValueError, match="contiguous"):
        ops.moe_sort(p, torch.zeros(2, 4, dtype=torch.int32).t())
    with pytest.raises(ValueError, match="GPU"):
        ops.moe_sort(p, idx)  # a plan on the host
    with pytest.raises(ValueError, match="GPU"):
        ops.moe_permute(p, torch.zeros(4, 32), torch.zeros(p.cap, 32))
    with pytest.raises(ValueError, match="float16|float32"):
        ops.moe_permute(p, torch.zeros(4, 32, dtype=torch.float16), torch.zeros(p.cap, 32))
    with pytest.raises(B.MoEError):
        ops.Plan(4, 0, 8, device="cpu")
    with pytest.raises(B.MoEError):
        ops.Plan(1 << 24, 1, 8, device="cpu")
    assert ops.Plan(0, 2, 8, device="cpu").cap == 0


def test_sizes_past_32_bits_refused():
    """Sizes that the C interface holds in 32 bits are refused, never cut off (tensors without memory)."""
    n = 2 ** 32 + 16  # 16 in 32 bits

    def t(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="meta")
    for kw in (dict(T=2 ** 32 + 8), dict(K=2 ** 32 + 1), dict(E=2 ** 32 + 4), dict(align=2 ** 32 + 1), dict(T=8 - 2 ** 32)):
        with pytest.raises(B.MoEError):
            ops.Plan(**{**dict(T=8, K=1, E=4, align=1, device="meta"), **kw})
    p = ops.Plan(1, 1, 1, align=128, device="meta")
    q, s = t(1, n, dtype=torch.uint8), t(1, ops.blocks(n), dtype=torch.float32)
    for call in (lambda: ops.moe_permute(p, t(1, n), t(p.cap, n)), lambda: ops.moe_permute_bwd(p, t(p.cap, n), t(1, n)),
                 lambda: ops.moe_permute_fp8(p, t(1, n), q, s), lambda: ops.moe_unpermute(p, t(p.cap, n), s, t(1, n)),
                 lambda: ops.moe_unpermute_bwd(p, t(1, n), None, s, None, None),
                 lambda: ops.moe_fp8_quant_rows(t(1, n), q, s), lambda: ops.moe_fp8_quant_cols(p, t(p.cap, n), q, s),
                 lambda: ops.moe_fp8_quant_weights(t(1, n, 16), q, None, s),
                 lambda: ops.moe_fp8_quant_weights(t(1, 16, n), q, None, s),
                 lambda: ops.moe_swiglu_fp8(t(1, 2 * n), q, s), lambda: ops.moe_swiglu_bwd(t(1, n), t(1, 2 * n), t(1, 2 * n)),
                 lambda: ops.moe_fp8_mm(None, q, s, q, s, t(1, 16)), lambda: ops.moe_fp8_mm(None, q, s, q, s, t(1, n)),
                 lambda: ops.moe_fp8_mm(None, t(n, 16, dtype=torch.uint8), t(n, 1, dtype=torch.float32),
                                        t(16, 16, dtype=torch.uint8), t(1, 1, dtype=torch.float32), t(n, 16)),
                 lambda: ops.moe_fp8_wgrad(p, t(1, n, 128), s, t(1, 16, 128), s, t(1, n, 16))):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_reference_encoder():
    """The tests' own E4M3 encoder: every code's value encodes to itself, midpoints go to the even code."""
    v = R.e4m3_values()
    codes = torch.tensor([c for c in range(256) if c & 0x7f != 0x7f])
    assert torch.equal(R.encode(v[codes]).long(), codes)
    pos = v[:127]
    mid = (pos[:-1] + pos[1:]) / 2
    lo = torch.arange(126)
    assert torch.equal(R.encode(mid).long(), torch.where(lo % 2 == 0, lo, lo + 1))
    assert torch.equal(R.encode(mid * (1 + 1e-12))[1:].long(), lo[1:] + 1)
    x = torch.randn(4096, generator=torch.Generator().manual_seed(1)).clamp(-448, 448)
    assert torch.equal(R.encode(x.double()), x.to(torch.float8_e4m3fn).view(torch.uint8))
