"""The operators of include/moe_step_ops.h on the GPU against float64 references
(step_ref.py): sizes from nothing to large, odd lengths, masks that leave rows
empty, non-finite values in places that must not be read, buffers that must stay
as they were, other streams, captured graphs.  Tolerances are error bounds derived
in step_ref.py and beside their use."""
import pytest
import torch

from fine_grained_mixture_top_amd import binding as B
from fine_grained_mixture_top_amd import ops

import step_ref as R

pytestmark = pytest.mark.gpu

NEG = float("-inf")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def offset(t, by):
    """A contiguous copy of t whose address is `by` elements past an allocation's start."""
    buf = torch.zeros(t.numel() + by, dtype=t.dtype, device=t.device)
    out = buf[by:by + t.numel()].view(t.shape)
    out.copy_(t)
    return out


# ---------------------------------------------------------------- balance

def check_balance(b, z, idx, valid):
    r = R.balance_ref(z, idx, valid)
    assert int(b.tokens) == r["n"]
    assert torch.equal(b.counts.long(), r["counts"])
    steps = R.balance_steps(z)
    R.within(b.load, r["load"], r["load"] * steps * 2.0 ** -23, "load")
    R.within(b.lse, r["lse"], R.lse_bound(r["lse"]), "lse")
    # E products of counts and means: E additions at most, few factors more; the z loss: as many additions as the means'
    lse = torch.where(r["counting"], r["lse"], torch.zeros_like(r["lse"])).abs()
    per = 1.0 / max(r["n"], 1)
    bound = torch.stack([r["loss"][0] * (steps + z.shape[1] + 8) * 2.0 ** -23,
                         r["loss"][1] * steps * 2.0 ** -23 + (2 * lse * R.lse_bound(lse)).sum() * per])
    R.within(b.loss, r["loss"], bound, "loss")
    return r


def top(z, K):
    return torch.topk(z.float(), K, dim=1).indices.to(torch.int32)


BALANCE = [  # T, E, K, dtype, share of padded tokens, masked experts, offset of the logits' address
    (0, 8, 2, "f32", 0.0, 0, 0), (1, 1, 1, "f32", 0.0, 0, 0), (1, 128, 8, "bf16", 0.0, 0, 0), (3, 7, 3, "f32", 0.0, 1, 0),
    (17, 16, 4, "f32", 0.3, 0, 1), (130, 60, 6, "bf16", 0.2, 3, 0), (512, 16, 4, "f32", 0.0, 0, 0),
    (129, 127, 5, "f32", 0.1, 2, 0), (129, 128, 8, "bf16", 0.1, 2, 3), (1000, 1000, 8, "f32", 0.0, 10, 0),
    (333, 1023, 8, "bf16", 0.5, 1, 0), (333, 1024, 2, "bf16", 0.0, 0, 0), (4099, 60, 6, "bf16", 0.2, 3, 0),
    (8200, 1024, 8, "f32", 0.0, 0, 0), (32768, 128, 8, "f32", 0.0, 0, 0), (70001, 24, 3, "f32", 0.05, 0, 0),
    (5000, 4, 4, "bf16", 0.0, 3, 0), (2500, 2, 1, "f32", 0.9, 1, 0), (5000, 520, 8, "f32", 0.0, 0, 0),
    (5000, 516, 8, "bf16", 0.0, 0, 0), (2049, 301, 7, "bf16", 0.0, 0, 0), (2049, 301, 7, "f32", 0.0, 0, 0),
]


def balance_case(T, E, K, dtype, pad, masked, off, seed):
    g = gen(seed)
    z = 2.0 * randn(g, T, E) + randn(g, E)
    if masked and T:
        z.scatter_(1, torch.rand(T, E, generator=g, device="cuda").topk(masked, 1).indices, NEG)
        z[torch.rand(T, generator=g, device="cuda") < 0.1] = NEG
    z = offset(z.to(DT[dtype]), off)
    idx = top(z, K)
    idx[torch.rand(T, K, generator=g, device="cuda") < 0.1] = -1
    idx[torch.rand(T, K, generator=g, device="cuda") < 0.05] = E
    valid = torch.rand(T, generator=g, device="cuda") >= pad if pad else None
    return g, z, idx, valid


@pytest.mark.parametrize("T,E,K,dtype,pad,masked,off", BALANCE)
def test_balance(T, E, K, dtype, pad, masked, off):
    g, z, idx, valid = balance_case(T, E, K, dtype, pad, masked, off, 11)
    b = ops.Balance(T, K, E)
    for t in (b.counts, b.tokens, b.load, b.lse, b.loss):
        t.fill_(-7)
    b.ws.fill_(255)
    ops.moe_balance(b, z, idx, valid)
    r = check_balance(b, z, idx, valid)
    first = [t.clone() for t in (b.counts, b.load, b.lse, b.loss)]
    d_loss = torch.tensor([0.7, -0.3], device="cuda")
    dz = offset(torch.full_like(z, 9.0), off)
    ops.moe_balance_bwd(b, z, d_loss, dz)
    want, bound = R.balance_bwd_ref(z, idx, r, d_loss)
    R.within(dz, want, bound + want.abs() * R.HALF[z.dtype] + 1e-38, "dz")
    gate, d_gate = torch.softmax(randn(g, T, K), 1), randn(g, T, K, std=1e-2)
    gone = (idx < 0) | (idx >= E)
    gate[gone], d_gate[gone] = float("nan"), float("inf")  # what a dropped choice holds is without effect
    ops.moe_balance_bwd(b, z, d_loss, dz, idx, gate, d_gate)
    want, bound = R.balance_bwd_ref(z, idx, r, d_loss, gate, d_gate)
    R.within(dz, want, bound + want.abs() * R.HALF[z.dtype] + 1e-38, "dz with gates")
    ops.moe_balance(b, z, idx, valid)
    assert all(torch.equal(x, y) for x, y in zip(first, (b.counts, b.load, b.lse, b.loss)))


@pytest.mark.parametrize("T,E,K", [(50, 12, 40), (20, 300, 200), (9, 5, 1024), (2500, 24, 33)])
def test_balance_more_choices_than_lanes(T, E, K):
    """Experts chosen many times by one token."""
    g = gen(T)
    z, idx = randn(g, T, E), torch.randint(-1, E + 1, (T, K), generator=g, device="cuda", dtype=torch.int32)
    b = ops.Balance(T, K, E)
    ops.moe_balance(b, z, idx)
    r = check_balance(b, z, idx, None)
    d_loss, dz = torch.tensor([0.7, -0.3], device="cuda"), torch.empty_like(z)
    gate, d_gate = torch.softmax(randn(g, T, K), 1), randn(g, T, K)
    ops.moe_balance_bwd(b, z, d_loss, dz, idx, gate, d_gate)
    want, bound = R.balance_bwd_ref(z, idx, r, d_loss, gate, d_gate)
    # (up to K values join an element: rounding of every partial sum, none above the sum of magnitudes)
    there = (idx >= 0) & (idx < E)
    gd = torch.where(there, gate * d_gate.abs(), 0.0).double()
    mag = torch.zeros_like(bound).scatter_add_(1, torch.where(there, idx, 0).long(), gd + gate.double() * gd.sum(1, keepdim=True))
    R.within(dz, want, bound + K * 2.0 ** -23 * mag + want.abs() * 2.0 ** -24 + 1e-38, "dz")


def test_balance_nothing_counts():
    b = ops.Balance(40, 2, 12)
    z = torch.full((40, 12), float("nan"), device="cuda")
    z[:20] = NEG
    valid = torch.zeros(40, dtype=torch.uint8, device="cuda")
    valid[:20] = 1  # valid, but every expert masked
    idx = torch.zeros(40, 2, dtype=torch.int32, device="cuda")
    ops.moe_balance(b, z, idx, valid)
    assert int(b.tokens) == 0 and not b.counts.any() and not b.load.any() and not b.loss.any()
    assert bool((b.lse == NEG).all())
    dz = torch.full_like(z, 5.0)
    ops.moe_balance_bwd(b, z, torch.ones(2, device="cuda"), dz)
    assert not dz.any()


def test_balance_spoiled_token_stays_in_its_row():
    g = gen(3)
    z = randn(g, 300, 40)
    z[7, 3], z[9, 0] = float("nan"), float("inf")
    b = ops.Balance(300, 4, 40)
    idx = torch.randint(0, 40, (300, 4), generator=g, device="cuda", dtype=torch.int32)
    ops.moe_balance(b, z, idx)
    assert int(b.tokens) == 300 and bool(torch.isnan(b.loss).all()) and bool(torch.isnan(b.load).all())
    rows = torch.isnan(b.lse) | torch.isinf(b.lse)
    assert rows.nonzero().flatten().tolist() == [7, 9]
    dz = torch.empty_like(z)
    ops.moe_balance_bwd(b, z, torch.ones(2, device="cuda"), dz)
    bad = ~torch.isfinite(dz).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 9]
    # marked as not valid they change nothing
    valid = torch.ones(300, dtype=torch.bool, device="cuda")
    valid[7] = valid[9] = False
    ops.moe_balance(b, z, idx, valid)
    check_balance(b, torch.where(valid[:, None], z, torch.zeros_like(z)), idx, valid)


def test_balance_large_logits_and_ties():
    z = torch.tensor([[3e38, -3e38, 3e38, 0.0], [-3.4e38, -3.4e38, -3.4e38, -3.4e38], [88.0, 89.0, -100.0, NEG]], device="cuda")
    idx = torch.tensor([[0, 2], [0, 1], [1, 1]], dtype=torch.int32, device="cuda")  # the last: one expert twice
    b = ops.Balance(3, 2, 4)
    ops.moe_balance(b, z, idx)
    assert b.counts.tolist() == [2, 3, 1, 0]
    p = torch.softmax(z.double(), 1)
    R.within(b.load, p.mean(0), 1e-6, "load")
    d_loss = torch.tensor([1.0, 0.0], device="cuda")
    dz = torch.empty_like(z)
    gate, d_gate = torch.full((3, 2), 0.5, device="cuda"), torch.tensor([[1.0, 0.0]] * 3, device="cuda")
    ops.moe_balance_bwd(b, z[:], d_loss, dz, idx, gate, d_gate)
    f = b.counts.double() * 4 / (9 * 2)
    want = p * (f - (p * f).sum(1, keepdim=True))
    want[0, 0] += 0.25
    want[0, 2] -= 0.25
    want[1, 0] += 0.25
    want[1, 1] -= 0.25  # (the last token's two choices cancel)
    # (row 1: the log-sum-exp of equal logits of -3.4e38 is -3.4e38 itself, their p are 1/4 all the same)
    R.within(dz, want, 1e-6)


def test_balance_gradient_against_differences():
    g = gen(5)
    T, E, K = 40, 12, 3
    z = randn(g, T, E)
    z[::7, 2] = NEG
    idx = top(z, K)
    valid = torch.rand(T, generator=g, device="cuda") > 0.2
    b = ops.Balance(T, K, E)
    ops.moe_balance(b, z, idx, valid)
    d_loss = torch.tensor([1.3, 0.2], device="cuda")
    gate = torch.softmax(torch.gather(z, 1, idx.long()), 1)
    d_gate = randn(g, T, K, std=0.1)
    dz = torch.empty_like(z)
    ops.moe_balance_bwd(b, z, d_loss, dz, idx, gate, d_gate)

    def total(zz):
        r = R.balance_ref(zz, idx, valid)
        gates = torch.softmax(torch.gather(zz, 1, idx.long()), 1)
        return float((d_loss.double() * r["loss"]).sum() + (gates * d_gate.double()).sum())

    h = 1e-5
    for t, e in [(0, 0), (0, 2), (3, 5), (14, 1), (21, 11), (39, 7)] + [(5, int(idx[5, k])) for k in range(K)]:
        up, down = z.double().clone(), z.double().clone()
        up[t, e] += h
        down[t, e] -= h
        # the difference's error: h^2 times a third derivative of order 1, and 1e-16 / h
        assert abs(float(dz[t, e]) - (total(up) - total(down)) / (2 * h)) < 1e-6, (t, e)


def replay(work, outs, eager):
    """Captures work() and checks every replay of three against eager(), with eager work between them."""
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
        want = eager(i)
        for o in outs:
            o.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), i


@pytest.mark.parametrize("T,E", [(100, 16), (3000, 96)])
def test_balance_captured_and_on_another_stream(T, E):
    g = gen(6)
    K = 4
    z, idx = randn(g, T, E), torch.zeros(T, K, dtype=torch.int32, device="cuda")
    b, b2 = ops.Balance(T, K, E), ops.Balance(T, K, E)
    d_loss, dz = torch.ones(2, device="cuda"), torch.zeros(T, E, device="cuda")

    def work():
        ops.moe_balance(b, z, idx)
        ops.moe_balance_bwd(b, z, d_loss, dz)

    def eager(i):
        z.copy_(randn(gen(60 + i), T, E))
        idx.copy_(top(z, K))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        d2 = torch.empty_like(dz)
        ops.moe_balance(b2, z, idx, stream=s)
        ops.moe_balance_bwd(b2, z, d_loss, d2, stream=s)
        s.synchronize()
        return b2.counts, b2.load, b2.lse, b2.loss, d2

    replay(work, (b.counts, b.load, b.lse, b.loss, dz), eager)


def test_balance_profile():
    b = ops.Balance(300, 2, 64)
    z, idx = torch.zeros(300, 64, device="cuda"), torch.zeros(300, 2, dtype=torch.int32, device="cuda")
    prof = B.Profiler(4)
    b.attach(prof)
    ops.moe_balance(b, z, idx)
    ops.moe_balance_bwd(b, z, torch.ones(2, device="cuda"), torch.empty_like(z))
    torch.cuda.synchronize()
    b.detach()
    rec = prof.records()
    prof.close()
    assert [ops.STEP_KERNEL_NAMES[k] for k, _ in rec] == ["balance", "balance_bwd"] and all(ms >= 0 for _, ms in rec)


# ---------------------------------------------------------------- orthogonalised updates

def update(g, M, N, kind="gauss"):
    w = randn(g, M, N)
    if kind == "low":  # a few large directions and small noise, as weight gradients have them
        r = max(1, min(M, N) // 16)
        w = 0.01 * w + randn(g, M, r) @ randn(g, r, N)
    return w


def check_ortho(o, ref, tol, what=""):
    """The error's norm, and every row's: a result's rounding is at most half a step of each value; a row may
    hold more than its share of the rest, not 8 times the largest row's."""
    half = R.HALF[o.dtype]
    off = o.double() - ref
    assert bool(torch.isfinite(o).all()), what
    n = float(ref.norm())
    assert float(off.norm()) <= (tol + half) * n + 1e-300, (what, float(off.norm()) / n, tol)
    rows = ref.norm(dim=1)
    bad = off.norm(dim=1) > half * rows + 8 * tol * rows.max() + 1e-300
    assert not bad.any(), (what, bad.nonzero().flatten()[:8].tolist())


ORTHO = [  # E, M, N, dtype, steps, coefficients, spectrum
    (1, 1, 1, "f32", 5, R.QUINTIC, "gauss"), (1, 1, 7, "bf16", 5, R.QUINTIC, "gauss"), (2, 3, 2, "f32", 5, R.QUINTIC, "gauss"),
    (3, 1, 300, "bf16", 3, R.QUINTIC, "gauss"), (2, 300, 1, "f32", 2, R.QUINTIC, "gauss"),
    (3, 63, 65, "bf16", 5, R.QUINTIC, "low"), (3, 65, 63, "f32", 5, R.QUINTIC, "low"), (2, 64, 64, "bf16", 1, R.QUINTIC, "gauss"),
    (1, 1536, 128, "f32", 5, R.QUINTIC, "low"), (1, 1537, 127, "bf16", 5, R.QUINTIC, "low"), (2, 130, 257, "bf16", 5, R.QUINTIC, "gauss"),
    (5, 40, 2000, "bf16", 4, R.QUINTIC, "gauss"), (2, 720, 1040, "f32", 5, R.QUINTIC, "low"), (2, 1040, 720, "bf16", 5, R.QUINTIC, "low"),
    (2, 40, 200, "bf16", 12, R.SMOOTH, "gauss"), (2, 200, 40, "bf16", 12, R.SMOOTH, "gauss"),
    (2, 40, 200, "bf16", 20, R.SMOOTH, "gauss"), (2, 200, 40, "bf16", 20, R.SMOOTH, "gauss"), (2, 41, 199, "f32", 12, R.SMOOTH, "gauss"),
    (1, 256, 1024, "bf16", 10, R.SMOOTH, "gauss"), (70, 16, 48, "bf16", 5, R.QUINTIC, "low"), (40, 1030, 1033, "f32", 2, R.QUINTIC, "low"),
    (36, 1033, 1027, "bf16", 3, R.QUINTIC, "low"),
]


@pytest.mark.parametrize("E,M,N,dtype,steps,coef,kind", ORTHO)
def test_orthogonalize(E, M, N, dtype, steps, coef, kind):
    g = gen(E + M + N)
    w = torch.stack([update(g, M, N, kind) for _ in range(E)]).to(DT[dtype])
    if E > 1:
        w[1] = 0.0  # an expert without rows
    h = ops.Ortho(E, M, N, dtype=DT[dtype], steps=steps, coef=coef, scale=0.2)
    h.ws.fill_(255)
    o = torch.full_like(w, 7.0)
    ops.moe_orthogonalize(h, w, o)
    for e in range(E) if E < 8 else (0, 1, 2, E // 2, E - 2, E - 1):
        ref = R.ortho_ref(w[e], steps, [coef] * steps, scale=0.2)
        if e == 1:
            assert not o[e].any()
            continue
        smallest = 0.0
        if coef == R.SMOOTH:
            s = torch.linalg.svdvals(w[e].double().cpu())
            smallest = float(s.min() / w[e].double().norm())
        check_ortho(o[e], ref, R.ortho_tolerance(w.dtype, steps, [coef], smallest), e)
    again = torch.empty_like(o)
    ops.moe_orthogonalize(h, w, again)
    assert torch.equal(o, again)


def test_orthogonalize_more_matrices_than_at_a_time():
    """160 matrices of 1100 x 1101 go through the workspace in two parts."""
    g = gen(8)
    E, M, N = 160, 1100, 1101
    w = randn(g, E, M, N, dtype=torch.bfloat16)
    h = ops.Ortho(E, M, N, steps=2)
    assert h.ws.numel() < 5 * E * 1152 * 1152 * 4
    o = torch.empty_like(w)
    ops.moe_orthogonalize(h, w, o)
    for e in (0, 79, 80, 81, 153, 154, 159):
        check_ortho(o[e], R.ortho_ref(w[e], 2, [R.QUINTIC] * 2), R.ortho_tolerance(w.dtype, 2, [R.QUINTIC]), e)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orthogonalize_any_size_of_values(dtype):
    """Results do not depend on the update's scale, up to the ends of its type."""
    g = gen(9)
    w = update(g, 50, 70, "low").to(DT[dtype])
    h = ops.Ortho(1, 50, 70, dtype=DT[dtype], eps=0.0)
    o, one = torch.empty(1, 50, 70, dtype=DT[dtype], device="cuda"), torch.empty(1, 50, 70, dtype=DT[dtype], device="cuda")
    ops.moe_orthogonalize(h, w[None].contiguous(), one)
    for p in (-100, -60, 60, 124 - int(w.float().abs().max().log2().ceil())):
        ops.moe_orthogonalize(h, (w.double() * 2.0 ** p).to(DT[dtype])[None].contiguous(), o)
        assert torch.equal(o, one), p  # (powers of two)
    tiny = ops.Ortho(1, 50, 70, dtype=DT[dtype], eps=1.0)
    small = (w.double() * 2.0 ** -70).to(DT[dtype])
    ops.moe_orthogonalize(tiny, small[None].contiguous(), o)  # far below eps: the steps' linear part
    ref = small.double() * 3.4445 ** 5
    assert float((o[0].double() - ref).norm() / ref.norm()) < R.HALF[DT[dtype]] + 1e-5


def test_orthogonalize_spoiled_matrix_stays_alone():
    g = gen(10)
    w = randn(g, 4, 60, 90, dtype=torch.bfloat16)
    h, o, clean = ops.Ortho(4, 60, 90), torch.empty_like(w), torch.empty_like(w)
    ops.moe_orthogonalize(h, w, clean)
    w[1, 5, 7], w[2, 0, 0] = float("nan"), float("-inf")
    ops.moe_orthogonalize(h, w, o)
    assert bool(torch.isnan(o[1]).all()) and bool(torch.isnan(o[2]).all())
    assert torch.equal(o[0], clean[0]) and torch.equal(o[3], clean[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_orthogonalize_addresses(dtype):
    """Matrices whose addresses are aligned to their element alone."""
    g = gen(12)
    for M, N in ((33, 65), (64, 96)):
        w = randn(g, 2, M, N, dtype=DT[dtype])
        h, o = ops.Ortho(2, M, N, dtype=DT[dtype]), torch.empty_like(w)
        ops.moe_orthogonalize(h, w, o)
        odd = offset(torch.zeros_like(w), 3)
        ops.moe_orthogonalize(h, offset(w, 1), odd)
        assert torch.equal(o, odd)


def test_orthogonalize_leaves_what_lies_around():
    g = gen(13)
    buf = torch.full((2, 50, 66), 3.0, device="cuda")
    flat = buf.view(-1)
    o = flat[64:64 + 2 * 33 * 65].view(2, 33, 65)
    w = randn(g, 2, 33, 65)
    keep = w.clone()
    ops.moe_orthogonalize(ops.Ortho(2, 33, 65, dtype=torch.float32), w, o)
    assert torch.equal(w, keep)
    assert bool((flat[:64] == 3).all()) and bool((flat[64 + 2 * 33 * 65:] == 3).all())


def test_orthogonalize_two_captured_calls():
    """Two handles in one graph, a tall and a wide update, replayed beside eager calls on another stream."""
    g = gen(14)
    a, b = randn(g, 3, 200, 70, dtype=torch.bfloat16), randn(g, 2, 70, 200)
    ha, hb = ops.Ortho(3, 200, 70), ops.Ortho(2, 70, 200, dtype=torch.float32)
    ea, eb = ops.Ortho(3, 200, 70), ops.Ortho(2, 70, 200, dtype=torch.float32)
    oa, ob = torch.empty_like(a), torch.empty_like(b)

    def work():
        ops.moe_orthogonalize(ha, a, oa)
        ops.moe_orthogonalize(hb, b, ob)

    def eager(i):
        a.copy_(randn(gen(70 + i), 3, 200, 70))
        b.copy_(randn(gen(80 + i), 2, 70, 200))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        wa, wb = torch.empty_like(a), torch.empty_like(b)
        ops.moe_orthogonalize(ea, a, wa, stream=s)
        ops.moe_orthogonalize(eb, b, wb, stream=s)
        s.synchronize()
        return wa, wb

    replay(work, (oa, ob), eager)


def test_orthogonalize_coefficients_per_step():
    g = gen(15)
    coef = [(3.0, -3.2, 1.2), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0)]
    for dtype in (torch.float32, torch.bfloat16):
        w = randn(g, 1, 48, 100, dtype=dtype)
        o = torch.empty_like(w)
        ops.moe_orthogonalize(ops.Ortho(1, 48, 100, dtype=dtype, steps=3, coef=coef), w, o)
        # differences of any of these maps on 0 .. 1.25 are below 4
        check_ortho(o[0], R.ortho_ref(w[0], 3, coef), R.ortho_tolerance(dtype, 3, [R.QUINTIC]))


# ---------------------------------------------------------------- MXFP4 weights

def weights(g, E, K, N, dtype=torch.float32, std=0.02):
    return randn(g, E, K, N, dtype=dtype, std=std)


def quantized(w):
    E, K, N = w.shape
    q = torch.full((E, N, K // 2), 0xaa, dtype=torch.uint8, device="cuda")
    s = torch.full((E, N, K // 32), 0xaa, dtype=torch.uint8, device="cuda")
    ops.moe_mxfp4_quant_weights(w, q, s)
    return q, s


@pytest.mark.parametrize("E,K,N,dtype", [(1, 32, 16, "f32"), (3, 96, 48, "bf16"), (2, 128, 64, "f32"), (1, 160, 80, "bf16"),
                                         (5, 736, 1040, "f32"), (2, 2048, 512, "bf16"), (1, 64, 4112, "bf16")])
def test_mxfp4_weights(E, K, N, dtype):
    g = gen(K + N)
    w = weights(g, E, K, N)
    w.view(-1)[::7] *= 2.0 ** 12
    w[0, :32, 0] = 0.0
    # borders between two codes, in a block whose largest value, 6, sets the scale to 1
    ties = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5.0, 7.5, -7.5,
                         0.0, -0.0] + [0.1] * 13, device="cuda")
    w[0, :32, 1] = ties
    w[0, :32, 2] = ties * 2.0 ** -128  # subnormal numbers
    w[0, :32, 3] = ties * 2.0 ** 125
    w[0, :32, 4] = 1e-45
    w = w.to(DT[dtype])
    q, s = quantized(w)
    rq, rs = R.mxfp4_codes(w)
    assert torch.equal(s, rs)
    assert torch.equal(q, rq)


def test_mxfp4_weights_not_finite():
    g = gen(21)
    w = weights(g, 2, 96, 32)
    w[0, 40, 3], w[1, 95, 31] = float("inf"), float("nan")
    q, s = quantized(w)
    rq, rs = R.mxfp4_codes(w)
    assert torch.equal(s, rs) and torch.equal(q, rq) and int((s == 255).sum()) == 2


def segments(T, K, E, drop, seed, align=1, lo=0):
    g = gen(seed)
    idx = torch.randint(lo, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    idx[torch.rand(T, K, generator=g, device="cuda") < drop] = -1
    plan = ops.Plan(T, K, E, align=align)
    ops.moe_sort(plan, idx)
    return plan


def check_mm(plan, a, q, s, c, gather, poison):
    """Every segment's rows, and the rows of none as they were."""
    offsets, counts, token = plan.offsets.tolist(), plan.counts.tolist(), plan.row_token.long()
    mine = torch.zeros(plan.cap, dtype=torch.bool, device="cuda")
    for e in range(plan.E):
        if not counts[e]:
            continue
        at = slice(offsets[e], offsets[e] + counts[e])
        mine[at] = True
        x = (a[token[at]] if gather else a[at]).double()
        w = R.mxfp4_values(q[e], s[e])
        ref, got = x @ w.t(), c[at].double()
        # where the magnitudes add up past fp32's largest number, below 2^128, a partial sum may pass it, and
        # opposite ones make it a NaN: the definition's value is no fp32 number there
        past = (x.abs() @ w.abs().t() >= 2.0 ** 128) & torch.isfinite(ref)
        ref, got = ref.masked_fill(past, 0.0), got.masked_fill(past, 0.0)
        R.within(got, ref, R.mxfp4_mm_bound(x, w, a.shape[1], ref, c.dtype).masked_fill(past, 0.0), e)
    assert bool((c[~mine] == poison).all())


MM = [  # T, K, E, align, drop, reduction, columns, result, gathered
    (1, 1, 1, 1, 0.0, 32, 16, "bf16", False), (1, 8, 16, 1, 0.0, 7168, 64, "bf16", True), (3, 2, 5, 16, 0.3, 96, 48, "f32", True),
    (40, 4, 300, 1, 0.1, 288, 80, "bf16", True), (37, 3, 8, 1, 0.15, 736, 1040, "f32", False), (64, 8, 128, 1, 0.0, 256, 512, "bf16", True),
    (200, 2, 3, 1, 0.0, 1024, 272, "bf16", False), (200, 2, 3, 1, 0.2, 32, 16, "f32", True), (301, 5, 7, 128, 0.1, 160, 528, "bf16", True),
    (1000, 2, 4, 1, 0.0, 224, 256, "f32", True), (129, 1, 1, 1, 0.0, 64, 272, "bf16", False), (4000, 3, 24, 1, 0.05, 512, 320, "bf16", True),
    (2500, 4, 1000, 1, 0.0, 128, 32, "bf16", True), (6000, 1, 2, 256, 0.0, 2048, 768, "f32", False), (50, 6, 1024, 1, 0.5, 64, 48, "f32", False),
    (700, 8, 64, 1, 0.0, 1056, 144, "bf16", True), (900, 8, 600, 1, 0.0, 96, 304, "bf16", True),
    (9000, 1, 2, 1, 0.1, 160, 4112, "f32", True), (2300, 4, 2, 16, 0.0, 224, 4112, "bf16", False), (9100, 1, 1, 1, 0.0, 32, 4096, "bf16", False),
]


@pytest.mark.parametrize("T,K,E,align,drop,d,N,out,gather", MM)
def test_mxfp4_mm(T, K, E, align, drop, d, N, out, gather):
    plan = segments(T, K, E, drop, T + E, align)
    g = gen(d + N)
    q, s = quantized(weights(g, E, d, N, dtype=torch.bfloat16))
    a = randn(g, T if gather else plan.cap, d, dtype=torch.bfloat16)
    if not gather:  # rows of no segment are never read
        mine = torch.zeros(plan.cap, dtype=torch.bool, device="cuda")
        for o, n in zip(plan.offsets.tolist(), plan.counts.tolist()):
            mine[o:o + n] = True
        a[~mine] = float("nan")
    c = torch.full((plan.cap, N), -7.25, dtype=DT[out], device="cuda")
    ops.moe_mxfp4_mm(plan, a, q, s, c, gather=gather)
    check_mm(plan, a, q, s, c, gather, -7.25)
    again = torch.full_like(c, -7.25)
    ops.moe_mxfp4_mm(plan, a, q, s, again, gather=gather)
    assert torch.equal(c, again)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 100, 300])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_mxfp4_mm_dense(rows, out):
    g = gen(rows)
    q, s = quantized(weights(g, 1, 416, 208))
    a = randn(g, rows, 416, dtype=torch.bfloat16)
    c = torch.empty(rows, 208, dtype=DT[out], device="cuda")
    ops.moe_mxfp4_mm(None, a, q[0], s[0], c)
    w, x = R.mxfp4_values(q[0], s[0]), a.double()
    R.within(c, x @ w.t(), R.mxfp4_mm_bound(x, w, 416, x @ w.t(), c.dtype))
    ops.moe_mxfp4_mm(None, torch.empty(0, 416, dtype=torch.bfloat16, device="cuda"), q, s, c[:0])


@pytest.mark.parametrize("T", [4, 600, 9000, 70000])
def test_mxfp4_mm_keeps_what_is_not_finite_in_its_place(T):
    """NaN and infinity in a row stay in that row, a block without a number in its column and expert; scale
    codes from one end to the other; tokens that do not exist count as zeros."""
    E, d, N = 3, 160, 64
    plan = segments(T, 2, E, 0.0, 5)
    g = gen(T)
    q, s = quantized(weights(g, E, d, N))
    s[0, 5, 4], s[1, 6, 0], s[2, 7, 1], s[1, 8] = 255, 0, 252, 1
    a = randn(g, T, d, dtype=torch.bfloat16)
    a[1, 3] = float("nan")
    a[2, 159] = float("inf")
    q[:, :, 79] = 0x11  # (no zero meets the infinity)
    c = torch.full((plan.cap, N), -7.25, device="cuda")
    ops.moe_mxfp4_mm(plan, a, q, s, c, gather=True)
    check_mm(plan, a, q, s, c, True, -7.25)
    ghosts = plan.row_token.clone()
    lost = torch.arange(plan.cap, device="cuda") % 3 == 0
    plan.row_token[lost] = T + 7
    plan.row_token[0] = -1
    c2 = torch.full_like(c, -7.25)
    ops.moe_mxfp4_mm(plan, a, q, s, c2, gather=True)
    keep = ~lost
    assert torch.equal(c2[keep].nan_to_num(7, 8, 9), c[keep].nan_to_num(7, 8, 9))
    e0 = slice(int(plan.offsets[0]), int(plan.offsets[0] + plan.counts[0]))
    z = c2[lost]
    assert bool(((z == 0) | torch.isnan(z)).all())  # zeros, NaN in the spoiled block's column
    assert bool((torch.isnan(c2[e0][lost[e0]]).nonzero()[:, 1] == 5).all())
    plan.row_token.copy_(ghosts)


def test_mxfp4_mm_captured_and_on_another_stream():
    """Decode through two products, captured: sort, product, product back; and a few hundred rows."""
    g = gen(31)
    for T in (3, 500, 6000):
        E, K, d, n = 6, 2, 192, 96
        w1, w2 = quantized(weights(g, E, d, n)), quantized(weights(g, E, n, d))
        x, idx = randn(g, T, d, dtype=torch.bfloat16), torch.zeros(T, K, dtype=torch.int32, device="cuda")
        pa, pb = ops.Plan(T, K, E), ops.Plan(T, K, E)
        h, y = torch.zeros(pa.cap, n, dtype=torch.bfloat16, device="cuda"), torch.zeros(pa.cap, d, device="cuda")

        def work(p=pa, h=h, y=y, stream=None):
            ops.moe_sort(p, idx, stream=stream)
            ops.moe_mxfp4_mm(p, x, *w1, h, gather=True, stream=stream)
            ops.moe_mxfp4_mm(p, h, *w2, y, stream=stream)

        def eager(i):
            x.copy_(randn(gen(90 + i), T, d))
            idx.copy_(torch.randint(0, E, (T, K), generator=gen(95 + i), device="cuda"))
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            h2, y2 = torch.zeros_like(h), torch.zeros_like(y)
            work(pb, h2, y2, s)
            s.synchronize()
            return h2, y2

        replay(work, (h, y), eager)


def test_mxfp4_profile():
    q, s = quantized(torch.ones(1, 32, 16, device="cuda"))
    plan = ops.Plan(2, 1, 1)
    ops.moe_sort(plan, torch.zeros(2, 1, dtype=torch.int32, device="cuda"))
    prof = B.Profiler(2)
    plan.attach(prof)
    ops.moe_mxfp4_mm(plan, torch.ones(2, 32, dtype=torch.bfloat16, device="cuda"), q, s, torch.empty(2, 16, device="cuda"))
    torch.cuda.synchronize()
    plan.detach()
    rec = prof.records()
    prof.close()
    assert [ops.STEP_KERNEL_NAMES[k] for k, _ in rec] == ["mxfp4_mm"]
