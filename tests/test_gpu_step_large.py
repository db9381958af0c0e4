"""Orthogonalised updates whose smaller side is above 128, in every kind of tile: scales, spoiled
matrices, addresses, what lies around results and workspace, captured graphs.  (test_gpu_step_ops.py
has these for the forms up to 128 rows.)"""
import pytest
import torch

from fine_grained_mixture_top_amd import ops

import step_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def within(buf, at, t):
    """A contiguous copy of t inside buf, from element `at` on."""
    out = buf[at:at + t.numel()].view(t.shape)
    out.copy_(t)
    return out


# tiles of 64, 64, 128 with three stages ahead, 128 with one, 256 (bf16)
SIZES = [(4, 130, 200), (4, 257, 161), (40, 300, 290), (64, 257, 300), (342, 300, 260)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,M,N", SIZES)
def test_orthogonalize_any_scale(E, M, N, dtype):
    """Powers of two leave the results as they are, up to the ends of the type."""
    w = randn(gen(1), E, M, N).to(DT[dtype])
    h = ops.Ortho(E, M, N, dtype=DT[dtype], eps=0.0)
    o, one = torch.empty_like(w), torch.empty_like(w)
    ops.moe_orthogonalize(h, w, one)
    assert bool(torch.isfinite(one).all())
    for p in (-90, 60, 120):
        ops.moe_orthogonalize(h, (w.double() * 2.0 ** p).to(DT[dtype]), o)
        assert torch.equal(o, one), p


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,M,N", SIZES)
def test_orthogonalize_spoiled_matrices_stay_alone(E, M, N, dtype):
    w = randn(gen(2), E, M, N).to(DT[dtype])
    h, o, clean = ops.Ortho(E, M, N, dtype=DT[dtype]), torch.empty_like(w), torch.empty_like(w)
    ops.moe_orthogonalize(h, w, clean)
    w[1, M - 1, 7], w[2, 0, N - 1] = float("nan"), float("-inf")
    ops.moe_orthogonalize(h, w, o)
    assert bool(torch.isnan(o[1:3]).all())
    assert torch.equal(o[0], clean[0]) and torch.equal(o[3:], clean[3:])
    w[1:3] = 0.0
    ops.moe_orthogonalize(h, w, o)  # (what they left in the workspace is without effect)
    assert not o[1:3].any() and torch.equal(o[0], clean[0]) and torch.equal(o[3:], clean[3:])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,M,N", SIZES + [(2, 256, 192), (342, 264, 272)])
def test_orthogonalize_addresses_and_what_lies_around(E, M, N, dtype):
    """Buffers aligned to their element alone; nothing written before or behind them."""
    w = randn(gen(3), E, M, N).to(DT[dtype])
    h, o = ops.Ortho(E, M, N, dtype=DT[dtype]), torch.empty_like(w)
    ops.moe_orthogonalize(h, w, o)
    src = torch.full((w.numel() + 1,), 5.0, dtype=w.dtype, device="cuda")
    dst = torch.full((w.numel() + 70,), 3.0, dtype=w.dtype, device="cuda")
    odd_w, odd_o = within(src, 1, w), within(dst, 3, torch.zeros_like(w))
    ops.moe_orthogonalize(h, odd_w, odd_o)
    assert torch.equal(o, odd_o) and torch.equal(odd_w, w)
    assert bool((dst[:3] == 3).all()) and bool((dst[3 + w.numel():] == 3).all()) and float(src[0]) == 5


SMOOTH_AFTER = [(3.4445, -4.7750, 2.0315)] * 4 + [R.SMOOTH] * 8


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E,M,N,coef", [
    (1, 64, 200, 5), (3, 1000, 128, 5), (3, 40, 100, SMOOTH_AFTER), (1, 130, 200, 1), (1, 130, 200, 5), (3, 257, 161, 7),
    (2, 200, 300, SMOOTH_AFTER), (40, 300, 290, 5), (64, 257, 300, 6), (342, 300, 260, 5),
])
def test_orthogonalize_workspace(E, M, N, coef, dtype):
    """The bytes that moe_orthogonalize_workspace_bytes names are all that is used, whatever they hold: one step,
    one group of steps, two and more."""
    w = randn(gen(4), E, M, N).to(DT[dtype])
    if isinstance(coef, int):
        h = ops.Ortho(E, M, N, dtype=DT[dtype], steps=coef)
    else:
        h = ops.Ortho(E, M, N, dtype=DT[dtype], steps=len(coef), coef=coef)
    need = h.ws.numel()
    o, again = torch.empty_like(w), torch.empty_like(w)
    ops.moe_orthogonalize(h, w, o)
    assert bool(torch.isfinite(o).all())
    buf = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    at = -buf.data_ptr() % 256 + 256
    h.ws = buf[at:at + need]
    ops.moe_orthogonalize(h, w, again)
    assert torch.equal(o, again)
    assert bool((buf[:at] == 255).all()) and bool((buf[at + need:] == 255).all())
    if isinstance(coef, int):
        ref = R.ortho_ref(w[E - 1], coef, [R.QUINTIC] * coef)
        tol = R.ortho_tolerance(w.dtype, coef, [R.QUINTIC]) + R.HALF[w.dtype]
        assert float((o[E - 1].double() - ref).norm()) <= tol * float(ref.norm())


def test_orthogonalize_two_large_calls_captured():
    """Two handles in one graph, a tall and a wide update, replayed beside eager calls on another stream."""
    a, b = randn(gen(5), 3, 400, 170, dtype=torch.bfloat16), randn(gen(6), 2, 140, 300)
    ha, hb = ops.Ortho(3, 400, 170), ops.Ortho(2, 140, 300, dtype=torch.float32)
    ea, eb = ops.Ortho(3, 400, 170), ops.Ortho(2, 140, 300, dtype=torch.float32)
    oa, ob, wa, wb = torch.empty_like(a), torch.empty_like(b), torch.empty_like(a), torch.empty_like(b)

    def work():
        ops.moe_orthogonalize(ha, a, oa)
        ops.moe_orthogonalize(hb, b, ob)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for i in range(3):
        a.copy_(randn(gen(70 + i), 3, 400, 170))
        b.copy_(randn(gen(80 + i), 2, 140, 300))
        s.wait_stream(torch.cuda.current_stream())
        ops.moe_orthogonalize(ea, a, wa, stream=s)
        ops.moe_orthogonalize(eb, b, wb, stream=s)
        oa.fill_(3), ob.fill_(3)
        graph.replay()  # (beside the other stream's calls, each with a workspace of its own)
        s.synchronize()
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb), i
