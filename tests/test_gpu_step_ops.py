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
