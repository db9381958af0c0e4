"""Host-side checks of the C ABI and binding of include/moe_step_ops.h (no GPU):
exports, constants, sizes, refusals before anything is launched."""
import ctypes
import os
import re

import pytest
import torch

from fine_grained_mixture_top_amd import binding as B
from fine_grained_mixture_top_amd import ops

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_step_ops.h")
P = 4096  # an aligned address that no refused call touches


def ref(x):
    return ctypes.byref(x)


def test_header_functions_and_constants():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    lib = ops.lib()
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", text))
    assert names
    for n in names:
        assert hasattr(lib, n) and getattr(lib, n).argtypes is not None, n
    consts = dict(re.findall(r"#define\s+(MOE_[A-Z0-9_]+)\s+(\d+)u?", text))
    ids = [int(v) for k, v in consts.items() if k.startswith("MOE_STEP_K_")]
    assert sorted(ids) == list(range(len(ops.KERNEL_NAMES), len(ops.STEP_KERNEL_NAMES)))
    for k, v in consts.items():
        assert getattr(ops, k) == int(v), k


def bdesc(T=8, E=4, K=2, dtype=B.MOE_F32, flags=0, reserved=0):
    return ops.MoeBalanceDesc(T, E, K, dtype, flags, reserved, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), B.MOE_EINVAL), (dict(K=0), B.MOE_EINVAL), (dict(E=0), B.MOE_EINVAL), (dict(dtype=2), B.MOE_EDTYPE),
    (dict(flags=1), B.MOE_EINVAL), (dict(reserved=1), B.MOE_EINVAL), (dict(T=1 << 24), B.MOE_ESHAPE),
    (dict(K=1025), B.MOE_ESHAPE), (dict(E=1025), B.MOE_ESHAPE), (dict(T=(1 << 24) - 1, K=65), B.MOE_ESHAPE),
])
def test_balance_descriptors_refused(kw, code):
    lib, d = ops.lib(), bdesc(**kw)
    assert lib.moe_balance_workspace_bytes(ref(d)) == 0
    assert lib.moe_balance(ref(d), P, P, None, P, P, P, P, P, P, 1 << 30, None) == code
    assert lib.moe_balance_bwd(ref(d), P, P, P, P, P, None, None, None, P, None) == code


def test_balance_refusals():
    lib, d = ops.lib(), bdesc(T=3000, E=64)
    need = lib.moe_balance_workspace_bytes(ref(d))
    assert need > 0 and need % 256 == 0
    good = [P, P, None, P, P, P, P, P, P, need]
    for i in (0, 1, 3, 4, 5, 6, 7, 8):
        bad = list(good)
        bad[i] = None
        assert lib.moe_balance(ref(d), *bad, None) == B.MOE_EINVAL, i
        if i != 2:
            bad[i] = P + 1
            assert lib.moe_balance(ref(d), *bad, None) == B.MOE_EINVAL, i
    assert lib.moe_balance(ref(d), *good[:-1], need - 1, None) == B.MOE_EWORKSPACE
    assert lib.moe_balance(None, *good, None) == B.MOE_EINVAL
    good = [P, P, P, P, P, None, None, None, P]
    for i in (0, 1, 2, 3, 4, 8):
        bad = list(good)
        bad[i] = None
        assert lib.moe_balance_bwd(ref(d), *bad, None) == B.MOE_EINVAL, i
        bad[i] = P + 2 if i else P + 1
        assert lib.moe_balance_bwd(ref(d), *bad, None) == B.MOE_EINVAL, i
    for gates in ((P, None, None), (None, P, P), (P, P, None), (P, None, P)):
        assert lib.moe_balance_bwd(ref(d), *good[:5], *gates, P, None) == B.MOE_EINVAL
    # no tokens: nothing to do
    assert lib.moe_balance_bwd(ref(bdesc(T=0)), *[None] * 9, None) == B.MOE_OK


def test_balance_binding_refuses():
    for kw, code in ((dict(T=-1, K=1, E=1), B.MOE_EINVAL), (dict(T=1, K=0, E=1), B.MOE_EINVAL),
                     (dict(T=1 << 24, K=1, E=1), B.MOE_ESHAPE), (dict(T=1, K=1, E=1025), B.MOE_ESHAPE),
                     (dict(T=1 << 40, K=1, E=1), B.MOE_ESHAPE)):
        with pytest.raises(B.MoEError) as e:
            ops.Balance(**kw, device="cpu")
        assert e.value.status == code
    b = ops.Balance(6, 2, 4, device="cpu")
    z, idx, dz = torch.zeros(6, 4), torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, 4)
    d = torch.ones(2)
    with pytest.raises(ValueError, match="a GPU is needed"):
        ops.moe_balance(b, z, idx)
    with pytest.raises(ValueError, match="logits"):
        ops.moe_balance(b, z.half(), idx)
    with pytest.raises(ValueError, match="logits"):
        ops.moe_balance(b, torch.zeros(4, 6).t(), idx)
    with pytest.raises(ValueError, match="expert_idx"):
        ops.moe_balance(b, z, idx.long())
    with pytest.raises(ValueError, match="valid"):
        ops.moe_balance(b, z, idx, valid=torch.ones(6))
    with pytest.raises(ValueError, match="dz"):
        ops.moe_balance_bwd(b, z, d, dz.bfloat16())
    with pytest.raises(ValueError, match="d_loss"):
        ops.moe_balance_bwd(b, z, torch.ones(3), dz)
    with pytest.raises(ValueError, match="all three or none"):
        ops.moe_balance_bwd(b, z, d, dz, idx, torch.ones(6, 2))
    with pytest.raises(ValueError, match="a tensor is needed"):
        ops.moe_balance_bwd(b, None, d, dz)


def odesc(E=2, M=64, N=96, dtype=B.MOE_BF16, steps=5, eps=1e-7, scale=1.0, flags=0, reserved=0, coef=(3.4445, -4.775, 2.0315)):
    c = None if coef is None else (ctypes.c_float * (3 * max(steps, 1)))(*(list(coef) * max(steps, 1)))
    d = ops.MoeOrthoDesc(E, M, N, dtype, steps, eps, scale, flags, reserved, c, None)
    d.keep = c
    return d


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), B.MOE_EINVAL), (dict(M=0), B.MOE_EINVAL), (dict(N=-1), B.MOE_EINVAL), (dict(steps=0), B.MOE_EINVAL),
    (dict(coef=None), B.MOE_EINVAL), (dict(dtype=3), B.MOE_EDTYPE), (dict(flags=1), B.MOE_EINVAL), (dict(reserved=1), B.MOE_EINVAL),
    (dict(E=1025), B.MOE_ESHAPE), (dict(steps=65), B.MOE_ESHAPE), (dict(M=16385, N=16385), B.MOE_ESHAPE),
    (dict(M=1, N=1 << 23), B.MOE_ESHAPE), (dict(M=1 << 30, N=1 << 30), B.MOE_ESHAPE), (dict(eps=-1.0), B.MOE_EINVAL),
    (dict(eps=float("nan")), B.MOE_EINVAL), (dict(scale=float("inf")), B.MOE_EINVAL), (dict(coef=(1.0, float("nan"), 0.0)), B.MOE_EINVAL),
])
def test_ortho_descriptors_refused(kw, code):
    lib, d = ops.lib(), odesc(**kw)
    assert lib.moe_orthogonalize_workspace_bytes(ref(d)) == 0
    assert lib.moe_orthogonalize(ref(d), P, P, P, 1 << 40, None) == code


def test_ortho_refusals():
    lib, d = ops.lib(), odesc()
    need = lib.moe_orthogonalize_workspace_bytes(ref(d))
    assert need > 0 and need % 256 == 0
    assert lib.moe_orthogonalize(None, P, P, P, need, None) == B.MOE_EINVAL
    for bad in ((None, P, P), (P, None, P), (P, P, None), (P + 1, P, P), (P, P + 1, P), (P, P, P + 16)):
        assert lib.moe_orthogonalize(ref(d), *bad, need, None) == B.MOE_EINVAL
    assert lib.moe_orthogonalize(ref(d), P, P, P, need - 1, None) == B.MOE_EWORKSPACE
    assert lib.moe_orthogonalize(ref(odesc(dtype=B.MOE_F32)), P + 2, P, P, 1 << 40, None) == B.MOE_EINVAL
    # the workspace grows with the matrices at a time, not with all of them
    big = [lib.moe_orthogonalize_workspace_bytes(ref(odesc(E=e, M=4096, N=4096))) for e in (17, 34, 1024)]
    assert big[0] == big[1] and big[2] <= big[0]


def test_ortho_binding_refuses():
    for kw, code in ((dict(E=0, M=1, N=1), B.MOE_EINVAL), (dict(E=1, M=1, N=1, steps=65), B.MOE_ESHAPE),
                     (dict(E=1, M=1 << 40, N=1), B.MOE_ESHAPE), (dict(E=1, M=20000, N=20000), B.MOE_ESHAPE),
                     (dict(E=1, M=4, N=4, eps=-1.0), B.MOE_EINVAL), (dict(E=1, M=4, N=4, scale=float("nan")), B.MOE_EINVAL),
                     (dict(E=1, M=4, N=4, coef=(1.0, 1e39, 0.0)), B.MOE_EINVAL)):
        with pytest.raises(B.MoEError) as e:
            ops.Ortho(**kw, device="cpu")
        assert e.value.status == code
    for kw in (dict(dtype=torch.float16), dict(coef=(1.0, 2.0)), dict(coef=[(1.0, 2.0, 3.0)] * 4), dict(coef=[(1.0, 2.0)] * 5)):
        with pytest.raises(ValueError):
            ops.Ortho(1, 4, 4, device="cpu", **kw)
    h = ops.Ortho(2, 4, 6, device="cpu")
    g = torch.zeros(2, 4, 6, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="a GPU is needed"):
        ops.moe_orthogonalize(h, g, torch.zeros_like(g))
    with pytest.raises(ValueError, match="g: dtype"):
        ops.moe_orthogonalize(h, g.float(), g)
    with pytest.raises(ValueError, match="g: shape"):
        ops.moe_orthogonalize(h, g[0], g)
    with pytest.raises(ValueError, match="o: not contiguous"):
        ops.moe_orthogonalize(h, g, torch.zeros(2, 6, 4, dtype=torch.bfloat16).transpose(1, 2))


def mdesc(a_rows=8, rows=8, used=0, E=2, K=64, N=48, out=B.MOE_BF16, flags=0, reserved=0):
    return ops.MoeMmDesc(a_rows, rows, used, E, K, N, out, flags, reserved, None)


PLAN = ops.MoePlan(P, P, P, P)


@pytest.mark.parametrize("kw,code", [
    (dict(a_rows=-1), B.MOE_EINVAL), (dict(rows=-1), B.MOE_EINVAL), (dict(used=9), B.MOE_EINVAL), (dict(E=0), B.MOE_EINVAL),
    (dict(K=0), B.MOE_EINVAL), (dict(N=0), B.MOE_EINVAL), (dict(K=48), B.MOE_ESHAPE), (dict(N=24), B.MOE_ESHAPE), (dict(E=1025), B.MOE_ESHAPE),
    (dict(K=(1 << 20) + 32), B.MOE_ESHAPE), (dict(K=1 << 16, N=1 << 15), B.MOE_ESHAPE), (dict(out=5), B.MOE_EDTYPE), (dict(flags=2), B.MOE_EINVAL),
    (dict(reserved=1), B.MOE_EINVAL), (dict(a_rows=9), B.MOE_EINVAL), (dict(a_rows=1 << 24, flags=1), B.MOE_ESHAPE),
    (dict(a_rows=0, flags=1), B.MOE_EINVAL),
])
def test_mxfp4_mm_descriptors_refused(kw, code):
    assert ops.lib().moe_mxfp4_mm(ref(mdesc(**kw)), P, P, P, ref(PLAN), P, None) == code


def test_mxfp4_refusals():
    lib, bf = ops.lib(), B.MOE_BF16
    mm = lambda d, *a: lib.moe_mxfp4_mm(ref(d), *a, None)  # noqa: E731
    assert lib.moe_mxfp4_mm(None, P, P, P, ref(PLAN), P, None) == B.MOE_EINVAL
    for bad in ((None, P, P, ref(PLAN), P), (P, None, P, ref(PLAN), P), (P, P, None, ref(PLAN), P), (P, P, P, ref(PLAN), None),
                (P + 8, P, P, ref(PLAN), P), (P, P + 8, P, ref(PLAN), P), (P, P, P, ref(PLAN), P + 8), (P, P, P, None, P)):
        assert mm(mdesc(), *bad) == B.MOE_EINVAL
    assert mm(mdesc(flags=1), P, P, P, ref(ops.MoePlan(P, P, 0, P)), P) == B.MOE_EINVAL
    assert mm(mdesc(), P, P, P, ref(ops.MoePlan(0, P, P, P)), P) == B.MOE_EINVAL
    assert mm(mdesc(E=1, flags=1), P, P, P, None, P) == B.MOE_EINVAL
    assert mm(mdesc(a_rows=0, rows=0), None, None, None, ref(PLAN), None) == B.MOE_OK
    w = lambda *a: lib.moe_mxfp4_quant_weights(*a, None, None)  # noqa: E731
    assert w(4, 1, 32, 16, P, P, P) == B.MOE_EDTYPE
    for E, K, N, code in ((0, 32, 16, B.MOE_EINVAL), (1, 0, 16, B.MOE_EINVAL), (1, 16, 16, B.MOE_ESHAPE), (1, 32, 8, B.MOE_ESHAPE),
                          (1025, 32, 16, B.MOE_ESHAPE), (1024, 1 << 20, 1 << 20, B.MOE_ESHAPE)):
        assert w(bf, E, K, N, P, P, P) == code
    for bad in ((None, P, P), (P, None, P), (P, P, None), (P + 8, P, P), (P, P + 8, P)):
        assert w(bf, 1, 32, 16, *bad) == B.MOE_EINVAL


def test_mxfp4_binding_refuses():
    z = lambda *n, dtype=torch.uint8: torch.zeros(*n, dtype=dtype)  # noqa: E731
    bf = torch.bfloat16
    a, q, s, c = z(4, 64, dtype=bf), z(1, 16, 32), z(1, 16, 2), z(4, 16, dtype=bf)
    with pytest.raises(ValueError, match="a GPU is needed"):
        ops.moe_mxfp4_mm(None, a, q, s, c)
    with pytest.raises(ValueError, match="a: dtype"):
        ops.moe_mxfp4_mm(None, a.float(), q, s, c)
    with pytest.raises(ValueError, match="multiple of 32"):
        ops.moe_mxfp4_mm(None, z(4, 48, dtype=bf), q, s, c)
    with pytest.raises(ValueError, match="q: shape"):
        ops.moe_mxfp4_mm(None, a, q[..., :31].contiguous(), s, c)
    with pytest.raises(ValueError, match="s: dtype"):
        ops.moe_mxfp4_mm(None, a, q, s.float(), c)
    with pytest.raises(ValueError, match="gather needs a plan"):
        ops.moe_mxfp4_mm(None, a, q, s, c, gather=True)
    with pytest.raises(ValueError, match="c: not contiguous"):
        ops.moe_mxfp4_mm(None, a, q, s, z(16, 4, dtype=bf).t())
    with pytest.raises(ValueError, match="multiple of 32"):
        ops.moe_mxfp4_quant_weights(z(1, 48, 16, dtype=bf), z(1, 16, 24), z(1, 16, 1))
    with pytest.raises(ValueError, match="q: shape"):
        ops.moe_mxfp4_quant_weights(z(1, 64, 16, dtype=bf), z(1, 64, 16), s)
