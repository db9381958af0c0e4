"""The single operators of include/moe_ops.h on the GPU against float64
references (ops_ref.py): sizes from nothing to several tiles, odd lengths,
dropped and doubled choices, empty experts, non-finite values in places that
must not be read, buffers that must stay as they were, other streams, captured
graphs.  Tolerances are error bounds derived in ops_ref.py and beside their use."""
import numpy as np
import pytest
import torch

from fine_grained_mixture_top_amd import binding as B
from fine_grained_mixture_top_amd import ops

import ops_ref as R

pytestmark = pytest.mark.gpu

POISON = -7.25  # exact in every type


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def choices(g, T, K, E, drop=0.0, lo=0):
    idx = torch.randint(lo, E, (T, K), generator=g, device="cuda", dtype=torch.int32)
    if drop:
        idx[torch.rand(T, K, generator=g, device="cuda") < drop] = -1
    return idx


def sorted_plan(idx, E, align=1):
    p = ops.Plan(idx.shape[0], idx.shape[1], E, align=align)
    p.row_token.fill_(-77)
    ops.moe_sort(p, idx)
    return p


def check_plan(p, idx, E, align):
    r = R.plan_ref(idx.cpu(), E, align)
    assert p.cap == r["cap"]
    np.testing.assert_array_equal(p.offsets.cpu().numpy(), r["offsets"])
    np.testing.assert_array_equal(p.counts.cpu().numpy(), r["counts"])
    np.testing.assert_array_equal(p.slot_row.cpu().numpy(), r["slot_row"])
    end = r["offsets"][-1]
    got = p.row_token.cpu().numpy()
    np.testing.assert_array_equal(got[:end], r["row_token"][:end])
    assert (got[end:] == -77).all()  # behind the last segment: as it was
    return r


SORTS = [  # T, K, E, align, share dropped
    (0, 4, 8, 1, 0.0), (1, 1, 1, 1, 0.0), (1, 8, 256, 1, 0.0), (1, 8, 256, 128, 0.0), (3, 5, 2, 16, 0.3),
    (7, 64, 1000, 1, 0.1), (513, 8, 1024, 7, 0.0), (512, 8, 64, 256, 0.5), (513, 8, 64, 128, 0.0),
    (5000, 3, 1, 1, 0.0), (9001, 6, 129, 128, 0.2), (70000, 8, 128, 1, 0.0), (70001, 8, 1024, 3, 0.1),
    (2, 1024, 7, 1, 0.0),
]


@pytest.mark.parametrize("T,K,E,align,drop", SORTS)
def test_sort(T, K, E, align, drop):
    idx = choices(gen(T + K), T, K, E, drop)
    check_plan(sorted_plan(idx, E, align), idx, E, align)


def test_sort_ids_out_of_range_and_skew():
    """Ids that are no expert drop their choice; all choices on one expert; no choice at all."""
    E = 16
    idx = choices(gen(1), 3000, 4, E)
    bad = torch.tensor([-1, E, E + 1, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    idx.view(-1)[:: 7] = bad.repeat(2000)[: idx.view(-1)[:: 7].numel()]
    check_plan(sorted_plan(idx, E, 128), idx, E, 128)
    one = torch.full((3000, 4), E - 1, dtype=torch.int32, device="cuda")
    check_plan(sorted_plan(one, E, 128), one, E, 128)
    none = torch.full((3000, 4), E, dtype=torch.int32, device="cuda")
    check_plan(sorted_plan(none, E, 128), none, E, 128)


def test_sort_same_plan_again():
    """A plan sorted again, with fewer rows than before, holds the new choices alone."""
    E, p = 32, ops.Plan(6000, 2, 32, align=16)
    for drop, seed in ((0.0, 1), (0.8, 2), (0.0, 3)):
        idx = choices(gen(seed), 6000, 2, E, drop)
        p.row_token.fill_(-77)
        ops.moe_sort(p, idx)
        check_plan(p, idx, E, 16)


MOVES = [  # T, K, E, d, align, share dropped, type
    (1, 8, 256, 7168, 1, 0.0, "bf16"), (1, 1, 1, 16, 1, 0.0, "f32"), (33, 3, 7, 48, 16, 0.4, "bf16"),
    (257, 8, 64, 2048, 128, 0.1, "bf16"), (100, 9, 5, 1040, 1, 0.2, "f32"), (4100, 2, 16, 528, 1, 0.0, "bf16"),
    (19, 40, 8, 272, 3, 0.3, "f32"), (256, 11, 9, 2576, 1, 0.2, "bf16"), (300, 3, 12, 4112, 16, 0.1, "bf16"),
    (7, 17, 30, 5008, 1, 0.2, "f32"),
]


def move_case(T, K, E, d, align, drop, dtype):
    g = gen(T * K + d)
    idx = choices(g, T, K, E, drop)
    p = sorted_plan(idx, E, align)
    return g, p, R.plan_ref(idx.cpu(), E, align), R.DT[dtype]


def untouched(buf, rows, value=POISON):
    """The rows of buf outside `rows` still hold the poison."""
    keep = torch.ones(buf.shape[0], dtype=torch.bool, device=buf.device)
    keep[rows] = False
    assert (buf[keep].double() == value).all()


@pytest.mark.parametrize("T,K,E,d,align,drop,dtype", MOVES)
def test_permute(T, K, E, d, align, drop, dtype):
    g, p, r, dt = move_case(T, K, E, d, align, drop, dtype)
    x = randn(g, T, d, dtype=dt)
    xp = torch.full((p.cap, d), POISON, dtype=dt, device="cuda")
    ops.moe_permute(p, x, xp)
    slots = torch.from_numpy(r["slot_row"]).cuda()
    t, k = torch.nonzero(slots >= 0, as_tuple=True)
    assert torch.equal(xp[slots[t, k]], x[t])
    untouched(xp, slots[t, k])
    # quantized on the way: the codes and scales of the token's row
    q = torch.full((p.cap, d), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((p.cap, ops.blocks(d)), POISON, device="cuda")
    ops.moe_permute_fp8(p, x, q, s)
    rq, rs = R.quant_rows_ref(x)
    assert torch.equal(q[slots[t, k]], rq[t]) and torch.equal(s[slots[t, k]], rs[t])
    untouched(q, slots[t, k], 0x11)
    untouched(s, slots[t, k])


@pytest.mark.parametrize("T,K,E,d,align,drop,dtype", MOVES)
def test_unpermute_and_gradients(T, K, E, d, align, drop, dtype):
    g, p, r, dt = move_case(T, K, E, d, align, drop, dtype)
    slots = torch.from_numpy(r["slot_row"]).cuda()
    kept = slots >= 0
    y = randn(g, p.cap, d, dtype=dt)
    y[torch.from_numpy(r["row_token"]).cuda() < 0] = float("nan")   # rows of no choice
    w = torch.randn(T, K, generator=g, device="cuda")
    w[~kept] = float("nan")                                         # weights of dropped choices
    do = randn(g, T, d, dtype=dt)
    y64 = torch.where(kept[..., None], y[slots.clamp(min=0)].double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    w64 = torch.where(kept, w, torch.zeros_like(w)).double()

    o = torch.full((T, d), POISON, dtype=dt, device="cuda")
    ops.moe_unpermute(p, y, w, o)
    prod = w64[..., None] * y64
    # K fused multiply-adds, one rounding each of at most the sum of magnitudes; then the type's
    ref = prod.sum(1)
    R.within(o, ref, K * 2.0 ** -24 * prod.abs().sum(1) * 1.001 + R.HALF[dt] * ref.abs() * 1.01, "o")

    dx = torch.full((T, d), POISON, dtype=dt, device="cuda")
    ops.moe_permute_bwd(p, y, dx)
    ref = y64.sum(1)
    R.within(dx, ref, K * 2.0 ** -24 * y64.abs().sum(1) * 1.001 + R.HALF[dt] * ref.abs() * 1.01, "dx")

    dy = torch.full((p.cap, d), POISON, dtype=dt, device="cuda")
    dw = torch.full((T, K), POISON, device="cuda")
    ops.moe_unpermute_bwd(p, do, y, w, dy, dw)
    t, k = torch.nonzero(kept, as_tuple=True)
    rows = slots[t, k]
    assert torch.equal(dy[rows], (w[t, k, None] * do[t].float()).to(dt))  # one fp32 product, rounded once
    untouched(dy, rows)
    dots = do.double()[:, None] * y64
    # d fused multiply-adds and a tree of at most 9 additions
    R.within(dw, dots.sum(2), (d + 9) * 2.0 ** -24 * dots.abs().sum(2) * 1.001, "dw")
    assert (dw[~kept] == 0).all()

    # either gradient alone is the same
    dy2, dw2 = torch.full_like(dy, POISON), torch.full_like(dw, POISON)
    ops.moe_unpermute_bwd(p, do, None, w, dy2, None)
    ops.moe_unpermute_bwd(p, do, y, None, None, dw2)
    assert torch.equal(dy, dy2) and torch.equal(dw, dw2)


def test_unpermute_gradients_against_differences():
    """d<o, do>/dw and /dy by central differences of the forward call (fp32, every choice)."""
    T, K, E, d = 5, 3, 4, 32
    g = gen(3)
    idx = choices(g, T, K, E, 0.2)
    p = sorted_plan(idx, E)
    y, w, do = randn(g, p.cap, d, dtype=torch.float32), torch.rand(T, K, generator=g, device="cuda"), \
        randn(g, T, d, dtype=torch.float32)
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    ops.moe_unpermute_bwd(p, do, y, w, dy, dw)

    def loss(y, w):
        o = torch.empty(T, d, device="cuda")
        ops.moe_unpermute(p, y, w, o)
        return float((o.double() * do.double()).sum())

    # linear in w and in y: the difference quotient is exact but for the forward's rounding, which is at
    # most (K + 1) 2^-24 of sum |do| sum |w y| per evaluation
    h = 0.25
    rows = p.slot_row.long()
    mag = (do.double().abs()[:, None] * y.double()[rows.clamp(min=0)].abs() * (w.abs() + h).double()[..., None]).sum()
    eps = 2 * (K + 1) * 2.0 ** -24 * float(mag) * 1.1 / (2 * h)
    for t in range(T):
        for k in range(K):
            a, b = w.clone(), w.clone()
            a[t, k] += h
            b[t, k] -= h
            assert abs((loss(y, a) - loss(y, b)) / (2 * h) - float(dw[t, k])) <= eps + 1e-5 * abs(float(dw[t, k]))
    for r, j in ((0, 0), (3, 17), (p.cap - 1, 31)):
        a, b = y.clone(), y.clone()
        a[r, j] += h
        b[r, j] -= h
        assert abs((loss(a, w) - loss(b, w)) / (2 * h) - float(dy[r, j])) <= eps + 1e-5 * abs(float(dy[r, j]))


# ---------------------------------------------------------------- quantizers

def hard_rows(g, Rn, C, dtype):
    """Rows with zero blocks, tiny, huge and single-value blocks."""
    x = randn(g, Rn, C, dtype=torch.float32)
    x[0::5] *= 1e-38
    x[1::5] *= 1e30
    x[2::5] = 0
    if Rn > 3:
        x[3, :] = 0
        x[3, C // 2] = -448.0
    return x.to(dtype)


@pytest.mark.parametrize("Rn,C,dtype", [(1, 16, "bf16"), (5, 128, "bf16"), (7, 144, "f32"), (130, 1040, "bf16"),
                                        (33, 7168, "f32"), (3, 112, "bf16")])
def test_quant_rows(Rn, C, dtype):
    x = hard_rows(gen(Rn + C), Rn, C, R.DT[dtype])
    q = torch.full((Rn, C), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((Rn, ops.blocks(C)), POISON, device="cuda")
    ops.moe_fp8_quant_rows(x, q, s)
    rq, rs = R.quant_rows_ref(x)
    assert torch.equal(s, rs)
    assert torch.equal(R.decode(q), R.decode(rq))  # (a zero may carry either sign)


def test_quant_rows_of_a_plan_and_non_finite():
    T, K, E, C = 300, 3, 9, 272
    g = gen(5)
    idx = choices(g, T, K, E, 0.2)
    p = sorted_plan(idx, E, 16)
    tok = p.row_token.long().cpu()
    tok[int(p.offsets[-1]):] = -1
    rows = torch.nonzero(tok >= 0)[:, 0].cuda()
    x = randn(g, p.cap, C)
    x[rows[4], 130] = float("nan")
    x[rows[5], 3] = float("-inf")
    q = torch.full((p.cap, C), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((p.cap, ops.blocks(C)), POISON, device="cuda")
    ops.moe_fp8_quant_rows(x, q, s, plan=p)
    untouched(q, rows, 0x11)
    untouched(s, rows)
    ok = torch.ones(len(rows), ops.blocks(C), dtype=torch.bool, device="cuda")
    ok[4, 1] = ok[5, 0] = False
    assert torch.isnan(s[rows][~ok]).all()
    x[rows[4], 130] = x[rows[5], 3] = 0.0
    rq, rs = R.quant_rows_ref(x[rows])
    assert torch.equal(s[rows][ok], rs[ok])
    wide = torch.repeat_interleave(ok, 128, 1)[:, :C]
    assert torch.equal(q[rows][wide], rq[wide])


@pytest.mark.parametrize("E,K,N,dtype", [(1, 16, 16, "bf16"), (2, 128, 256, "f32"), (3, 272, 144, "bf16"),
                                         (5, 1040, 528, "bf16"), (2, 96, 2048, "f32")])
def test_quant_weights(E, K, N, dtype):
    g = gen(K + N)
    w = randn(g, E, K, N, dtype=R.DT[dtype], std=0.02)
    w[0, :16] = 0
    q = torch.full((E, K, N), 0x11, dtype=torch.uint8, device="cuda")
    qt = torch.full((E, N, K), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((E, ops.blocks(K), ops.blocks(N)), POISON, device="cuda")
    ops.moe_fp8_quant_weights(w, q, qt, s)
    for e in range(E):
        for i in range(s.shape[1]):
            for j in range(s.shape[2]):
                at = (e, slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                rq, rs = R.block_codes(w[at])
                assert float(s[e, i, j]) == float(rs)
                assert torch.equal(R.decode(q[at]), R.decode(rq))
    assert torch.equal(qt, q.transpose(1, 2))
    for keep in (0, 1):  # one layout alone
        q1, s1 = torch.zeros_like(q if keep == 0 else qt), torch.zeros_like(s)
        ops.moe_fp8_quant_weights(w, q1 if keep == 0 else None, q1 if keep else None, s1)
        assert torch.equal(q1, qt if keep else q) and torch.equal(s1, s)


COLS = [(1, 1, 4, 16, 128), (300, 3, 9, 272, 128), (300, 3, 9, 144, 256), (1000, 2, 3, 1040, 128)]


@pytest.mark.parametrize("T,K,E,C,align", COLS)
@pytest.mark.parametrize("gather", [False, True])
def test_quant_cols(T, K, E, C, align, gather):
    g = gen(T + C)
    idx = choices(g, T, K, E, 0.1 if T > 1 else 0.0)
    p = sorted_plan(idx, E, align)
    r = R.plan_ref(idx.cpu(), E, align)
    src = randn(g, T if gather else p.cap, C)
    if not gather:
        src[torch.from_numpy(r["row_token"]).cuda() < 0] = float("nan")  # between the segments
    q, s = ops.column_buffers(p, C)
    q = q.view(torch.uint8)
    q.fill_(0x11)
    s.fill_(POISON)
    ops.moe_fp8_quant_cols(p, src, q, s, gather=gather)
    end = int(r["offsets"][-1]) // 128
    assert (q[end:] == 0x11).all() and (s[end:] == POISON).all()
    for b in range(end):
        tok = torch.from_numpy(r["row_token"][128 * b:128 * b + 128]).cuda()
        rows = tok if gather else torch.arange(128 * b, 128 * b + 128, device="cuda")
        v = torch.where((tok >= 0)[:, None], src[rows.clamp(min=0)].float(), torch.zeros((), device="cuda"))
        rq, rs = R.quant_rows_ref(v.t().contiguous())
        assert torch.equal(s[b], rs[:, 0])
        assert torch.equal(R.decode(q[b]), R.decode(rq))


# ---------------------------------------------------------------- products

def codes(g, *shape):
    """Every finite code, magnitudes log-uniform as the format spreads them."""
    c = torch.randint(0, 255, shape, generator=g, device="cuda", dtype=torch.int32)
    c = torch.where((c & 0x7f) == 0x7f, c - 1, c)
    return c.to(torch.uint8)


def weights_ref(b, sb):
    """b [N, K] codes, sb [ceil(K/128), ceil(N/128)] -> float64 [K, N]."""
    return R.values(b, torch.repeat_interleave(sb.t(), 128, 0)[:b.shape[0]]).t().contiguous()


def mm_case(g, rows_a, E, K, N):
    a, sa = codes(g, rows_a, K), torch.rand(rows_a, ops.blocks(K), generator=g, device="cuda") + 0.1
    b, sb = codes(g, E, N, K), torch.rand(E, ops.blocks(K), ops.blocks(N), generator=g, device="cuda") + 0.1
    return a, sa, b, sb


def check_mm(p, r, a, sa, b, sb, c, K, dt, gather):
    for e in range(p.E):
        n = int(r["counts"][e])
        if n == 0:
            continue
        rows = torch.arange(int(r["offsets"][e]), int(r["offsets"][e]) + n, device="cuda")
        take = torch.from_numpy(r["row_token"]).cuda()[rows] if gather else rows
        av, wv = R.values(a[take], sa[take]), weights_ref(b[e], sb[e])
        ref = av @ wv
        R.within(c[rows], ref, R.mm_bound(av.abs(), wv.abs(), K, ref, dt), f"expert {e}")


PRODUCTS = [  # T, K choices, E, reduction, columns, align, dropped, type, gathered
    (1, 1, 1, 16, 16, 1, 0.0, "f32", False), (1, 8, 256, 512, 256, 1, 0.0, "bf16", True),
    (1, 8, 64, 2048, 512, 128, 0.0, "bf16", False), (16, 8, 64, 1040, 272, 1, 0.1, "bf16", True),
    (37, 5, 6, 272, 144, 1, 0.3, "f32", False), (100, 3, 3, 128, 1040, 16, 0.0, "bf16", True),
    (200, 2, 5, 400, 128, 128, 0.0, "f32", True), (700, 4, 8, 1024, 512, 1, 0.0, "bf16", False),
    (3001, 2, 9, 656, 336, 1, 0.4, "f32", True), (4096, 2, 4, 256, 768, 128, 0.0, "bf16", True),
    (900, 1, 1, 384, 256, 1, 0.0, "bf16", False), (64, 1, 1000, 144, 48, 1, 0.0, "f32", False),
    # every workgroup walks several tiles: one block of the reduction a tile, a ragged one, several
    (4111, 2, 4, 128, 2064, 1, 0.1, "bf16", True), (4111, 2, 4, 272, 2064, 1, 0.1, "bf16", True),
    (4111, 2, 3, 16, 2304, 128, 0.0, "bf16", False), (5003, 2, 8, 640, 4096, 1, 0.3, "bf16", False),
    (4111, 2, 4, 128, 1040, 1, 0.1, "f32", True), (4111, 2, 4, 400, 1040, 1, 0.1, "f32", False),
    (6007, 2, 40, 384, 1296, 1, 0.2, "bf16", True), (6007, 2, 40, 112, 1296, 1, 0.2, "bf16", True),
    (400, 2, 20, 1040, 2064, 1, 0.0, "bf16", True), (300, 2, 20, 1040, 400, 1, 0.0, "f32", True),
    (150, 1, 10, 528, 272, 1, 0.0, "bf16", False),
    # many experts with few rows: a workgroup's next tile is many experts further on
    (128, 4, 256, 400, 144, 1, 0.1, "bf16", True), (128, 4, 256, 272, 144, 1, 0.0, "f32", False),
    (3200, 2, 160, 400, 656, 1, 0.2, "bf16", True), (3200, 2, 160, 128, 656, 1, 0.2, "bf16", False),
    (1920, 2, 160, 400, 656, 1, 0.2, "f32", True), (1920, 2, 160, 128, 656, 128, 0.2, "f32", True),
    (2000, 8, 1000, 144, 272, 1, 0.5, "bf16", True),
    # the widest tiles, two to a workgroup: one block of the reduction, a ragged one, a short one
    (7777, 2, 4, 128, 1808, 1, 0.1, "bf16", True), (7777, 2, 4, 272, 1808, 1, 0.1, "bf16", True),
    (7777, 2, 3, 16, 2000, 128, 0.0, "bf16", False), (4300, 2, 3, 400, 2320, 1, 0.1, "f32", True),
    (4300, 2, 3, 400, 2320, 128, 0.0, "f32", False), (7680, 2, 60, 400, 640, 1, 0.1, "bf16", True),
    (7680, 2, 60, 656, 640, 128, 0.0, "bf16", False),
]


@pytest.mark.parametrize("T,K,E,Kd,N,align,drop,dtype,gather", PRODUCTS)
def test_product(T, K, E, Kd, N, align, drop, dtype, gather):
    g = gen(T + Kd + N)
    idx = choices(g, T, K, E, drop, lo=1 if E > 4 else 0)  # expert 0 of many stays empty
    p = sorted_plan(idx, E, align)
    r = R.plan_ref(idx.cpu(), E, align)
    dt = R.DT[dtype]
    a, sa, b, sb = mm_case(g, T if gather else p.cap, E, Kd, N)
    if not gather:
        sa[torch.from_numpy(r["row_token"]).cuda() < 0] = float("nan")  # rows of no segment
    c = torch.full((p.cap, N), POISON, dtype=dt, device="cuda")
    ops.moe_fp8_mm(p, a, sa, b, sb, c, gather=gather)
    check_mm(p, r, a, sa, b, sb, c, Kd, dt, gather)
    slots = torch.from_numpy(r["slot_row"]).cuda()
    untouched(c, slots[slots >= 0])
    # the scales' other layout gives the same bits, and so does the same call again
    c2 = torch.full_like(c, POISON)
    ops.moe_fp8_mm(p, a, sa, b, sb.transpose(1, 2).contiguous(), c2, gather=gather, sb_out_major=True)
    assert torch.equal(c, c2)


@pytest.mark.parametrize("rows,Kd,N,dtype", [(0, 128, 128, "bf16"), (1, 4096, 1024, "bf16"), (3, 16, 48, "f32"),
                                             (17, 2064, 144, "f32"), (129, 640, 384, "bf16"), (600, 1024, 528, "f32"),
                                             (5000, 512, 1024, "bf16")])
def test_product_dense(rows, Kd, N, dtype):
    g = gen(rows + Kd)
    dt = R.DT[dtype]
    a, sa, b, sb = mm_case(g, rows, 1, Kd, N)
    c = torch.full((rows, N), POISON, dtype=dt, device="cuda")
    ops.moe_fp8_mm(None, a, sa, b[0], sb[0], c)
    av, wv = R.values(a, sa), weights_ref(b[0], sb[0])
    ref = av @ wv
    R.within(c, ref, R.mm_bound(av.abs(), wv.abs(), Kd, ref, dt))


def test_product_rows_do_not_leak():
    """A row's NaN or infinite scale, or a NaN code, spoils that row alone; a weight block's spoils its columns."""
    g = gen(11)
    rows, Kd, N = 300, 384, 400
    a, sa, b, sb = mm_case(g, rows, 1, Kd, N)
    clean = torch.empty(rows, N, device="cuda")
    ops.moe_fp8_mm(None, a, sa, b, sb, clean)
    sa[7, 1] = float("nan")
    a[100, 383] = 0x7f
    sa[299, 0] = float("inf")
    c = torch.empty_like(clean)
    ops.moe_fp8_mm(None, a, sa, b, sb, c)
    spoiled = torch.zeros(rows, dtype=torch.bool, device="cuda")
    spoiled[[7, 100, 299]] = True
    assert torch.equal(c[~spoiled], clean[~spoiled])
    assert not torch.isfinite(c[spoiled]).any()
    sb[0, 2, 1] = float("nan")
    ops.moe_fp8_mm(None, a, sa, b, sb, c)
    assert torch.isnan(c[:, 128:256]).all()
    assert torch.equal(c[~spoiled][:, :128], clean[~spoiled][:, :128])
    assert torch.equal(c[~spoiled][:, 256:], clean[~spoiled][:, 256:])


def test_product_of_a_broken_plan_stays_in_its_buffers():
    """Segments that reach past the buffers, or tokens that do not exist, are cut off, never followed."""
    g = gen(12)
    T, K, E, Kd, N = 40, 2, 4, 256, 128
    idx = choices(g, T, K, E)
    p = sorted_plan(idx, E)
    p.counts[E - 1] += 1000
    p.row_token[3] = 10 ** 6
    p.row_token[4] = -5
    a, sa, b, sb = mm_case(g, T, E, Kd, N)
    c = torch.full((p.cap + 64, N), POISON, device="cuda")
    ops.moe_fp8_mm(p, a, sa, b, sb, c[:p.cap], gather=True)
    torch.cuda.synchronize()
    assert (c[p.cap:] == POISON).all() and (c[3:5] == 0).all()


# One size for every kernel of the product (256 CUs): T, K choices, E, reduction, columns, type, gathered; the
# reduction ends in a short block, rows and columns inside a tile.
KERNELS = {
    "16 rows x 32": (12, 2, 4, 400, 272, "bf16", True), "16 rows x 64": (18, 2, 4, 400, 272, "f32", True),
    "32 rows x 64": (40, 2, 4, 400, 272, "bf16", False), "64 x 128": (300, 2, 4, 400, 272, "bf16", True),
    "128 x 128": (1500, 2, 2, 400, 2064, "bf16", True), "256 x 256": (2100, 2, 3, 400, 2064, "bf16", False),
    "256 x 256 gathered": (2600, 2, 3, 400, 2320, "bf16", True), "64 x 128 fp32": (300, 2, 4, 400, 272, "f32", False),
    "128 x 256 fp32": (1500, 2, 2, 400, 2064, "f32", True),
}
DENSE = {  # rows, reduction, columns, type
    "16 rows x 32": (5, 400, 272, "f32"), "16 rows x 64": (9, 400, 272, "bf16"), "32 rows x 64": (20, 400, 272, "bf16"),
    "64 x 128": (300, 400, 272, "bf16"), "128 x 128": (1900, 400, 4064, "bf16"), "256 x 256": (4000, 400, 4064, "bf16"),
    "64 x 128 fp32": (300, 400, 272, "f32"), "128 x 256 fp32": (4000, 400, 4064, "f32"),
}
NAN_CODE = 0x7f


@pytest.mark.parametrize("kernel", KERNELS)
def test_rows_of_tokens_that_do_not_exist_are_zeros(kernel):
    """Whatever a's first row holds, and the other rows are what they are without such tokens."""
    T, K, E, Kd, N, dtype, _ = KERNELS[kernel]
    g = gen(13)
    p = sorted_plan(choices(g, T, K, E), E)
    a, sa, b, sb = mm_case(g, T, E, Kd, N)
    a[0] = NAN_CODE
    sa[0] = float("nan")
    clean = torch.full((p.cap, N), POISON, dtype=R.DT[dtype], device="cuda")
    ops.moe_fp8_mm(p, a, sa, b, sb, clean, gather=True)
    assert torch.isnan(clean[p.row_token == 0]).all()
    gone = torch.zeros(p.cap, dtype=torch.bool, device="cuda")
    gone[[1, p.cap // 2, p.cap - 2]] = True
    p.row_token[gone] = torch.tensor([10 ** 6, -5, T], dtype=torch.int32, device="cuda")
    c = torch.full_like(clean, POISON)
    ops.moe_fp8_mm(p, a, sa, b, sb, c, gather=True)
    assert (c[gone] == 0).all()
    assert torch.equal(c[~gone].nan_to_num(nan=POISON), clean[~gone].nan_to_num(nan=POISON))


def spoil(a, sa, b, sb, Kd):
    """NaN and infinities in some rows of a, one column and one column block of b's first expert -> those rows."""
    rows = [1, len(a) // 2, len(a) - 2, len(a) - 1]
    sa[rows[0], 1] = float("nan")
    a[rows[1], Kd - 1] = NAN_CODE
    sa[rows[2], -1] = float("inf")
    a[rows[3], 0] = 0x80 | NAN_CODE
    b[0, 5, Kd - 1] = NAN_CODE
    sb[0, -1, 1] = float("nan")
    return rows


def check_spoiled(c, clean, bad_rows, first):
    """bad_rows are not finite; rows of the first expert (`first`) are NaN in columns 5 and 128..255; the rest as clean."""
    assert not torch.isfinite(c[bad_rows]).any()
    cols = torch.zeros(c.shape[1], dtype=torch.bool, device="cuda")
    cols[5] = cols[128:256] = True
    assert torch.isnan(c[first][:, cols]).all()
    good = ~bad_rows[:, None] & ~(first[:, None] & cols)
    assert torch.equal(c[good], clean[good])


@pytest.mark.parametrize("kernel", KERNELS)
def test_product_contains_what_is_not_finite(kernel):
    T, K, E, Kd, N, dtype, gather = KERNELS[kernel]
    g = gen(14)
    p = sorted_plan(choices(g, T, K, E), E)
    a, sa, b, sb = mm_case(g, T if gather else p.cap, E, Kd, N)
    clean = torch.empty(p.cap, N, dtype=R.DT[dtype], device="cuda")
    ops.moe_fp8_mm(p, a, sa, b, sb, clean, gather=gather)
    rows = spoil(a, sa, b, sb, Kd)
    c = torch.empty_like(clean)
    ops.moe_fp8_mm(p, a, sa, b, sb, c, gather=gather)
    bad = torch.zeros(len(a), dtype=torch.bool, device="cuda")
    bad[rows] = True
    check_spoiled(c, clean, bad[p.row_token.long()] if gather else bad,
                  torch.arange(p.cap, device="cuda") < p.counts[0])


@pytest.mark.parametrize("kernel", DENSE)
def test_dense_product_contains_what_is_not_finite(kernel):
    rows, Kd, N, dtype = DENSE[kernel]
    g = gen(15)
    a, sa, b, sb = mm_case(g, rows, 1, Kd, N)
    clean = torch.empty(rows, N, dtype=R.DT[dtype], device="cuda")
    ops.moe_fp8_mm(None, a, sa, b, sb, clean)
    av, wv = R.values(a, sa), weights_ref(b[0], sb[0])
    ref = av @ wv
    R.within(clean, ref, R.mm_bound(av.abs(), wv.abs(), Kd, ref, R.DT[dtype]))
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[spoil(a, sa, b, sb, Kd)] = True
    c = torch.empty_like(clean)
    ops.moe_fp8_mm(None, a, sa, b, sb, c)
    check_spoiled(c, clean, bad, torch.ones(rows, dtype=torch.bool, device="cuda"))


WGRADS = [  # T, K, E, M, N, align, dropped, type, gathered
    (1, 1, 4, 16, 16, 128, 0.0, "f32", True), (5, 2, 3, 144, 272, 128, 0.0, "bf16", True),
    (300, 3, 9, 272, 144, 128, 0.2, "f32", False), (300, 2, 5, 256, 512, 256, 0.0, "bf16", True),
    (3000, 2, 3, 528, 400, 128, 0.0, "f32", True), (0, 2, 3, 128, 128, 128, 0.0, "bf16", False),
    # more tiles than workgroups, several experts without rows
    (90, 1, 80, 512, 528, 128, 0.3, "bf16", True), (90, 1, 80, 512, 528, 256, 0.3, "f32", True),
    (2000, 3, 40, 528, 512, 128, 0.0, "bf16", False), (6000, 3, 2, 2064, 2048, 128, 0.0, "bf16", True),
    (900, 2, 40, 752, 512, 128, 0.1, "bf16", True), (60, 1, 90, 384, 512, 128, 0.2, "bf16", False),
]


@pytest.mark.parametrize("T,K,E,M,N,align,drop,dtype,gather", WGRADS)
def test_wgrad(T, K, E, M, N, align, drop, dtype, gather):
    g = gen(T + M + N)
    idx = choices(g, T, K, E, drop, lo=1 if E > 4 else 0)
    p = sorted_plan(idx, E, align)
    r = R.plan_ref(idx.cpu(), E, align)
    dt = R.DT[dtype]
    x, dy = randn(g, T if gather else p.cap, M), randn(g, p.cap, N, std=1e-3)
    (xq, xs), (yq, ys) = ops.column_buffers(p, M), ops.column_buffers(p, N)
    ops.moe_fp8_quant_cols(p, x, xq, xs, gather=gather)
    ops.moe_fp8_quant_cols(p, dy, yq, ys)
    dw = torch.full((E, M, N), POISON, dtype=dt, device="cuda")
    ops.moe_fp8_wgrad(p, xq, xs, yq, ys, dw)
    for e in range(E):
        b0, nb = int(r["offsets"][e]) // 128, -(-int(r["counts"][e]) // 128)
        ref, mag = torch.zeros(M, N, dtype=torch.float64, device="cuda"), torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for b in range(b0, b0 + nb):
            xv, yv = R.decode(xq[b]) * xs[b].double()[:, None], R.decode(yq[b]) * ys[b].double()[:, None]
            ref += xv @ yv.t()
            mag += xv.abs() @ yv.abs().t()
        # as mm_bound, with the product of the two scales rounded once more per block
        bound = R.mm_steps(128 * nb, 3, dt) * mag + R.HALF[dt] * ref.abs() * (1 + 2.0 ** -7)
        R.within(dw[e], ref, bound, f"expert {e}")


# One size for every tile of the weight gradient: T, K, E, M, N, type
WTILES = {"192 x 256": (900, 2, 40, 752, 512, "bf16"), "128 x 128": (900, 2, 40, 528, 400, "bf16"),
          "64 x 128": (900, 2, 9, 272, 144, "bf16"), "128 x 64 fp32": (900, 2, 9, 272, 144, "f32")}


@pytest.mark.parametrize("tile", WTILES)
def test_wgrad_contains_what_is_not_finite(tile):
    """A value of x or dy that is not finite spoils its column's row or column of its own expert's gradient alone."""
    T, K, E, M, N, dtype = WTILES[tile]
    g = gen(16)
    p = sorted_plan(choices(g, T, K, E), E, 128)
    x, dy = randn(g, p.cap, M), randn(g, p.cap, N)
    bufs = ops.column_buffers(p, M) + ops.column_buffers(p, N)

    def wgrad():
        dw = torch.full((E, M, N), POISON, dtype=R.DT[dtype], device="cuda")
        ops.moe_fp8_quant_cols(p, x, *bufs[:2])
        ops.moe_fp8_quant_cols(p, dy, *bufs[2:])
        ops.moe_fp8_wgrad(p, *bufs, dw)
        return dw
    clean = wgrad()
    off = p.offsets.tolist()
    x[off[1], 7], x[off[E - 1], M - 1], dy[off[2] + 1, 33] = float("nan"), float("inf"), float("-inf")
    bad = torch.zeros(E, M, N, dtype=torch.bool, device="cuda")
    bad[1, 7] = bad[E - 1, M - 1] = bad[2, :, 33] = True
    dw = wgrad()
    assert torch.isnan(dw[bad]).all() and torch.equal(dw[~bad], clean[~bad])


# Scales whose products leave fp32's normal range, beside results that do not.  a's scales go by row (column of
# x), b's by column block (column of dy); tiny codes or zeros where both scales are large, so that results stay finite.
EA, EB = (-60, 80, -120, 0, 100, 118), (-100, 50, 118, 0)


def hard_scales(g, shape, exps, dim):
    e = torch.tensor(exps, device="cuda").repeat(shape[dim])[:shape[dim]]
    m = 1 + torch.rand(shape, generator=g, device="cuda")
    return m * torch.exp2(e.float()).view([-1 if i == dim else 1 for i in range(len(shape))]), e


def check_hard(c, ref, mag, steps, blocks, dt, apart, sa, sb):
    """Sums' and result's rounding as for any scales; below the smallest normal number a result is a multiple of
    2^-149 (fp32; each block's sum may round to one) or 2^-133 (bf16).  Where the kernel does not keep the scales
    apart, their product (sa [rows, blocks] by sb [blocks, columns]) is off by up to 2^-150 below the normal numbers,
    times at most 128 * 448 * 448 < 2^24.7: 2^-125 a block; and past the largest number nothing is asked.  Nor is it
    of results past the largest number."""
    ok = mag < 3e38
    small = blocks * 2.0 ** -149 + (2.0 ** -133 if dt == torch.bfloat16 else 0.0)
    if not apart:
        for i in range(blocks):
            ok &= torch.isfinite(sa[:, i, None] * sb[None, i])
        small += blocks * 2.0 ** -125
    bound = steps * mag + R.HALF[dt] * ref.abs() * (1 + 2.0 ** -7) + small
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    R.within(torch.where(ok, c.double(), zero), torch.where(ok, ref, zero), bound)


@pytest.mark.parametrize("kernel", KERNELS)
def test_product_of_scales_past_the_normal_range(kernel):
    T, K, E, Kd, N, dtype, gather = KERNELS[kernel]
    apart = dtype == "f32" or "rows x" in kernel
    g, dt = gen(17), R.DT[dtype]
    p = sorted_plan(choices(g, T, K, E), E)
    a, _, b, _ = mm_case(g, T if gather else p.cap, E, Kd, N)
    sa, ea = hard_scales(g, (len(a), ops.blocks(Kd)), EA, 0)
    sb, eb = hard_scales(g, (E, ops.blocks(Kd), ops.blocks(N)), EB, 2)
    a[ea >= 80] = a[ea >= 80] & 0x81  # 2^-9, 0 and their negatives
    a[ea == 100] = 0
    tiny = torch.repeat_interleave(eb, 128)[:N] == 50
    b[:, tiny] = b[:, tiny] & 0x81
    c = torch.full((p.cap, N), POISON, dtype=dt, device="cuda")
    ops.moe_fp8_mm(p, a, sa, b, sb, c, gather=gather)
    for e in range(E):
        r0 = int(p.offsets[e])
        rows = torch.arange(r0, r0 + int(p.counts[e]), device="cuda")
        take = p.row_token[rows].long() if gather else rows
        av, wv = R.values(a[take], sa[take]), weights_ref(b[e], sb[e])
        # (per block: the scales' product, its product with the block's, its power of two and the sum)
        check_hard(c[rows], av @ wv, av.abs() @ wv.abs(), R.mm_steps(Kd, 4, dt), ops.blocks(Kd), dt, apart,
                   sa[take], torch.repeat_interleave(sb[e], 128, 1)[:, :N])


@pytest.mark.parametrize("tile", WTILES)
def test_wgrad_of_scales_past_the_normal_range(tile):
    T, K, E, M, N, dtype = WTILES[tile]
    g, dt = gen(18), R.DT[dtype]
    p = sorted_plan(choices(g, T, K, E), E, 128)
    nb = p.cap // 128
    a, b = codes(g, nb, M, 128), codes(g, nb, N, 128)
    sa, ea = hard_scales(g, (nb, M), EA, 1)
    sb, eb = hard_scales(g, (nb, N), EB, 1)
    a[:, ea >= 80] = a[:, ea >= 80] & 0x81
    a[:, ea == 100] = 0
    b[:, eb == 50] = b[:, eb == 50] & 0x81
    dw = torch.full((E, M, N), POISON, dtype=dt, device="cuda")
    ops.moe_fp8_wgrad(p, a, sa, b, sb, dw)
    off, counts = p.offsets.tolist(), p.counts.tolist()
    for e in range(E):
        b0, n = off[e] // 128, -(-counts[e] // 128)
        ref, mag = torch.zeros(M, N, dtype=torch.float64, device="cuda"), torch.zeros(M, N, dtype=torch.float64, device="cuda")
        for i in range(b0, b0 + n):
            xv, yv = R.decode(a[i]) * sa[i].double()[:, None], R.decode(b[i]) * sb[i].double()[:, None]
            ref += xv @ yv.t()
            mag += xv.abs() @ yv.abs().t()
        check_hard(dw[e], ref, mag, R.mm_steps(128 * n, 4, dt), n, dt, dtype == "f32", sa[b0:b0 + n].t(), sb[b0:b0 + n])


# ---------------------------------------------------------------- SwiGLU

def swiglu64(h, n):
    g, u = h[:, :n].double(), h[:, n:].double()
    s = torch.sigmoid(g)
    return g, u, s


@pytest.mark.parametrize("Rn,n,dtype", [(1, 16, "bf16"), (7, 144, "f32"), (300, 256, "bf16"), (65, 1040, "f32")])
def test_swiglu(Rn, n, dtype):
    gn = gen(Rn + n)
    dt = R.DT[dtype]
    h = randn(gn, Rn, 2 * n, dtype=dt, std=3.0)
    h[0, 0], h[0, 1], h[0, 2] = 200.0, -200.0, 0.0
    q = torch.full((Rn, n), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((Rn, ops.blocks(n)), POISON, device="cuda")
    a = torch.full((Rn, n), POISON, dtype=dt, device="cuda")
    ops.moe_swiglu_fp8(h, q, s, a)
    g, u, sg = swiglu64(h, n)
    ref = g * sg * u
    # the exponential's argument rounds by |g| 2^-24 log2(e) ln 2 and the exponential and the reciprocal by
    # about a step (2^-23) each; one addition, two products
    rel = (g.abs() + 8) * 2.0 ** -23
    err = rel * ref.abs() + 1e-37
    R.within(a, ref, err + R.HALF[dt] * ref.abs() * 1.01, "a")
    wide = torch.repeat_interleave(s.double(), 128, 1)[:, :n]
    amax = torch.stack([ref[:, c:c + 128].abs().amax(1) for c in range(0, n, 128)], 1)
    R.within(s, amax / 448, amax / 448 * ((g.abs().max() + 9) * 2.0 ** -23) + R.TINY, "s")
    # a code is off by at most half a step: 2^-4 of the value, or 2^-10 of the scale below 2^-6
    R.within(R.decode(q) * wide, ref, ref.abs() * 2.0 ** -4 * 1.001 + wide * 2.0 ** -10 + err, "q")
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    ops.moe_swiglu_fp8(h, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("Rn,n,dtype", [(1, 16, "bf16"), (7, 144, "f32"), (300, 256, "bf16"), (65, 1040, "f32")])
def test_swiglu_bwd(Rn, n, dtype):
    gn = gen(Rn + n)
    dt = R.DT[dtype]
    h, da = randn(gn, Rn, 2 * n, dtype=dt, std=3.0), randn(gn, Rn, n, dtype=dt)
    h[0, 0], h[0, 1], h[0, 2] = 200.0, -200.0, 0.0
    dh = torch.full((Rn, 2 * n), POISON, dtype=dt, device="cuda")
    ops.moe_swiglu_bwd(da, h, dh)
    g, u, s = swiglu64(h, n)
    d = da.double()
    rel = (g.abs() + 8) * 2.0 ** -23
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    # 1 - s and 1 + g (1 - s) cancel: an error of s counts |g| s more
    bg = (d * u * s).abs() * (rel * (1 + (g * (1 - s)).abs() + (g * s).abs()) + 4 * 2.0 ** -24 * (1 + g.abs()))
    R.within(dh[:, :n], dg, bg + R.HALF[dt] * dg.abs() * 1.01 + 1e-37, "dg")
    R.within(dh[:, n:], du, rel * du.abs() + R.HALF[dt] * du.abs() * 1.01 + 1e-37, "du")


def test_swiglu_bwd_against_differences():
    """dh by central differences of sum(da * A) in float64 of the formula."""
    gn = gen(2)
    h, da = randn(gn, 4, 64, dtype=torch.float32), randn(gn, 4, 32, dtype=torch.float32)
    dh = torch.empty_like(h)
    ops.moe_swiglu_bwd(da, h, dh)
    step = 1e-4
    for i, j in ((0, 0), (1, 31), (2, 32), (3, 63)):
        v = []
        for sgn in (1, -1):
            x = h.double().clone()
            x[i, j] += sgn * step
            g, u, s = swiglu64(x, 32)
            v.append(float((da.double() * g * s * u).sum()))
        # a third derivative of order one times step^2, and the kernel's rounding
        assert abs((v[0] - v[1]) / (2 * step) - float(dh[i, j])) <= 1e-6 + 1e-5 * abs(float(dh[i, j]))


# The sigmoid's relative error: the hardware exponential's last place (2^-23, its argument in two parts is exact to
# 2^-40) and the sum that joins the parts (2^-24), the denominator's rounding and the reciprocal's after its Newton
# step (2^-24 each): 5 * 2^-24, whatever g is, where it is a normal number; below 2^-126 it may be 0.
SIGMOID = 5 * 2.0 ** -24


def wide_gates(gn, Rn, n, dt):
    h = randn(gn, Rn, 2 * n, dtype=torch.float32)
    h[:, :n] = (torch.rand(Rn, n, generator=gn, device="cuda") - 0.5) * 174.0  # -87..87
    return h.to(dt)


def type_step(dt):
    """What the result's type adds: nothing to fp32 sums; to bf16 half a step of the value, and below 2^-126, where a
    result is a multiple of 2^-133, half of that."""
    return (R.HALF[dt] * 1.01, 2.0 ** -134) if dt == torch.bfloat16 else (0.0, 0.0)


@pytest.mark.parametrize("Rn,n,dtype", [(64, 256, "f32"), (33, 400, "bf16")])
def test_swiglu_error_does_not_grow_with_the_gate(Rn, n, dtype):
    gn, dt = gen(19), R.DT[dtype]
    h = wide_gates(gn, Rn, n, dt)
    q, s = torch.empty(Rn, n, dtype=torch.uint8, device="cuda"), torch.empty(Rn, ops.blocks(n), device="cuda")
    a = torch.empty(Rn, n, dtype=dt, device="cuda")
    ops.moe_swiglu_fp8(h, q, s, a)
    g, u, sg = swiglu64(h, n)
    ref = g * sg * u
    err = (SIGMOID + 2 * 2.0 ** -24) * 1.001 * ref.abs() + 2.0 ** -140  # two products
    half, tiny = type_step(dt)
    R.within(a, ref, err + half * ref.abs() + tiny, "a")
    # a block's scale is off as its largest value is, and rounds once
    amax = torch.stack([ref[:, c:c + 128].abs().amax(1) for c in range(0, n, 128)], 1)
    R.within(s, (amax / 448).clamp(min=R.TINY), (SIGMOID + 3 * 2.0 ** -24) * 1.001 * amax / 448 + 2.0 ** -140, "s")
    wide = torch.repeat_interleave(s.double(), 128, 1)[:, :n]
    R.within(R.decode(q) * wide, ref, ref.abs() * 2.0 ** -4 * 1.001 + wide * 2.0 ** -10 + err, "q")


@pytest.mark.parametrize("Rn,n,dtype", [(64, 256, "f32"), (33, 400, "bf16")])
def test_swiglu_bwd_error_does_not_grow_with_the_gate(Rn, n, dtype):
    gn, dt = gen(20), R.DT[dtype]
    h, da = wide_gates(gn, Rn, n, dt), randn(gn, Rn, n, dtype=dt)
    dh = torch.empty_like(h)
    ops.moe_swiglu_bwd(da, h, dh)
    g, u, s = swiglu64(h, n)
    d, step = da.double(), 2.0 ** -24
    half, tiny = type_step(dt)
    du = d * g * s
    R.within(dh[:, n:], du, (SIGMOID + 2 * step) * 1.001 * du.abs() + half * du.abs() + tiny + 2.0 ** -140, "du")
    # t = 1 - s is off by s SIGMOID and a rounding, m = g t by g times that and a rounding, q = 1 + m by a rounding
    # more; d u s q: the sigmoid's error and three products
    t, q = 1 - s, 1 + g * (1 - s)
    eq = g.abs() * (s * SIGMOID + 2 * step * t) + step * q.abs()
    dg = d * u * s * q
    bound = (d * u * s).abs() * (q.abs() * (SIGMOID + 3 * step) + eq) * 1.001 + half * dg.abs() + tiny + 2.0 ** -140
    R.within(dh[:, :n], dg, bound, "dg")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_swiglu_of_the_farthest_gates(dtype):
    """Gates down to the type's lowest value give zeros, up to its largest the gate itself, with finite gradients."""
    dt, n = R.DT[dtype], 16
    big = torch.finfo(dt).max
    gates = torch.tensor([-big, -1e30, -1e4, -200.0, -105.0, -90.0, -88.0, -87.5, 0.0, -0.0, 88.0, 90.0, 200.0, 1e4, 1e30, big],
                         device="cuda")
    h = torch.ones(1, 2 * n, device="cuda")
    h[0, :n] = gates
    h = h.to(dt)
    q, s = torch.empty(1, n, dtype=torch.uint8, device="cuda"), torch.empty(1, 1, device="cuda")
    a, dh, da = torch.empty(1, n, dtype=dt, device="cuda"), torch.empty_like(h), torch.ones(1, n, dtype=dt, device="cuda")
    ops.moe_swiglu_fp8(h, q, s, a)
    ops.moe_swiglu_bwd(da, h, dh)
    g = h[:, :n].double()
    ref = g * torch.sigmoid(g)
    # a sigmoid below 2^-126 may be 0: at most 105 * 2^-126 of these sums (farther gates: less than 2^-149 of them)
    tol = ref.abs() * 1e-6 + R.HALF[dt] * ref.abs() * (dt == torch.bfloat16) + 105 * 2.0 ** -126
    R.within(a, ref, tol, "a")
    R.within(dh[:, n:], ref, tol, "du")
    sg = torch.sigmoid(g)
    dg = sg * (1 + g * (1 - sg))
    R.within(dh[:, :n], dg, dg.abs() * 1e-5 + R.HALF[dt] * dg.abs() * (dt == torch.bfloat16) + 105 * 2.0 ** -126, "dg")
    assert float(s) == float(torch.tensor(big, dtype=torch.float32) / torch.tensor(448.0))


def test_swiglu_of_a_plan():
    """Only the plan's rows are read and written."""
    T, K, E, n = 200, 3, 7, 144
    g = gen(9)
    idx = choices(g, T, K, E, 0.3)
    p = sorted_plan(idx, E, 16)
    r = R.plan_ref(idx.cpu(), E, 16)
    slots = torch.from_numpy(r["slot_row"]).cuda()
    rows = slots[slots >= 0]
    h, da = randn(g, p.cap, 2 * n), randn(g, p.cap, n)
    q = torch.full((p.cap, n), 0x11, dtype=torch.uint8, device="cuda")
    s = torch.full((p.cap, 2), POISON, device="cuda")
    a, dh = torch.full((p.cap, n), POISON, dtype=torch.bfloat16, device="cuda"), torch.full_like(h, POISON)
    ops.moe_swiglu_fp8(h, q, s, a, plan=p)
    ops.moe_swiglu_bwd(da, h, dh, plan=p)
    q2, s2, a2, dh2 = torch.empty_like(q), torch.empty_like(s), torch.empty_like(a), torch.empty_like(dh)
    ops.moe_swiglu_fp8(h, q2, s2, a2)
    ops.moe_swiglu_bwd(da, h, dh2)
    for got, full, poison in ((q, q2, 0x11), (s, s2, POISON), (a, a2, POISON), (dh, dh2, POISON)):
        assert torch.equal(got[rows], full[rows])
        untouched(got, rows, poison)


# ---------------------------------------------------------------- together

class Experts:
    """Buffers and calls of an FP8 expert layer, forward and backward, as a program would write it."""

    def __init__(self, T, K, E, d, n, w1, w2):
        self.p = ops.Plan(T, K, E, align=128)
        cap, bf = self.p.cap, torch.bfloat16

        def q(*shape):
            return torch.zeros(*shape, dtype=torch.uint8, device="cuda").view(ops.E4M3)

        def f(*shape):
            return torch.zeros(*shape, device="cuda")

        def h(*shape):
            return torch.zeros(*shape, dtype=bf, device="cuda")

        self.w1q, self.w1t, self.w1s = q(E, d, 2 * n), q(E, 2 * n, d), f(E, ops.blocks(d), ops.blocks(2 * n))
        self.w2q, self.w2t, self.w2s = q(E, n, d), q(E, d, n), f(E, ops.blocks(n), ops.blocks(d))
        ops.moe_fp8_quant_weights(w1, self.w1q, self.w1t, self.w1s)
        ops.moe_fp8_quant_weights(w2, self.w2q, self.w2t, self.w2s)
        self.xq, self.xs = q(T, d), f(T, ops.blocks(d))
        self.h, self.a, self.aq, self.as_ = h(cap, 2 * n), h(cap, n), q(cap, n), f(cap, ops.blocks(n))
        self.y, self.o = h(cap, d), h(T, d)
        self.dy, self.dyq, self.dys, self.dw = h(cap, d), q(cap, d), f(cap, ops.blocks(d)), f(T, K)
        self.da, self.dh = h(cap, n), h(cap, 2 * n)
        self.dhq, self.dhs = q(cap, 2 * n), f(cap, ops.blocks(2 * n))
        self.dxp, self.dx = h(cap, d), h(T, d)
        self.cx, self.cdh = ops.column_buffers(self.p, d), ops.column_buffers(self.p, 2 * n)
        self.ca, self.cdy = ops.column_buffers(self.p, n), ops.column_buffers(self.p, d)
        self.dw1, self.dw2 = h(E, d, 2 * n), h(E, n, d)

    def forward(self, x, idx, w):
        p = self.p
        ops.moe_sort(p, idx)
        ops.moe_fp8_quant_rows(x, self.xq, self.xs)
        ops.moe_fp8_mm(p, self.xq, self.xs, self.w1t, self.w1s, self.h, gather=True)
        ops.moe_swiglu_fp8(self.h, self.aq, self.as_, self.a, plan=p)
        ops.moe_fp8_mm(p, self.aq, self.as_, self.w2t, self.w2s, self.y)
        ops.moe_unpermute(p, self.y, w, self.o)

    def backward(self, x, w, do):
        p = self.p
        ops.moe_unpermute_bwd(p, do, self.y, w, self.dy, self.dw)
        ops.moe_fp8_quant_rows(self.dy, self.dyq, self.dys, plan=p)
        ops.moe_fp8_mm(p, self.dyq, self.dys, self.w2q, self.w2s, self.da, sb_out_major=True)
        ops.moe_swiglu_bwd(self.da, self.h, self.dh, plan=p)
        ops.moe_fp8_quant_rows(self.dh, self.dhq, self.dhs, plan=p)
        ops.moe_fp8_mm(p, self.dhq, self.dhs, self.w1q, self.w1s, self.dxp, sb_out_major=True)
        ops.moe_permute_bwd(p, self.dxp, self.dx)
        ops.moe_fp8_quant_cols(p, x, *self.cx, gather=True)
        ops.moe_fp8_quant_cols(p, self.dh, *self.cdh)
        ops.moe_fp8_wgrad(p, *self.cx, *self.cdh, self.dw1)
        ops.moe_fp8_quant_cols(p, self.a, *self.ca)
        ops.moe_fp8_quant_cols(p, self.dy, *self.cdy)
        ops.moe_fp8_wgrad(p, *self.ca, *self.cdy, self.dw2)

    def results(self):
        return [self.o, self.dw, self.dx, self.dw1, self.dw2]


def layer_case(T=600, K=3, E=8, d=512, n=256, seed=21, drop=0.1):
    g = gen(seed)
    x, do = randn(g, T, d), randn(g, T, d)
    w1, w2 = randn(g, E, d, 2 * n, std=0.05), randn(g, E, n, d, std=0.05)
    idx = choices(g, T, K, E, drop)
    w = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), 1)
    return x, do, w1, w2, idx, w


def layer64(x, do, w1, w2, idx, w):
    """The layer and its gradients in float64 without any quantization."""
    T, d = x.shape
    E, n = w1.shape[0], w2.shape[1]
    x, do, w1, w2, w = (t.double() for t in (x, do, w1, w2, w))
    o, dx, dw = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(w)
    dw1, dw2 = torch.zeros_like(w1), torch.zeros_like(w2)
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        if not len(t):
            continue
        g, u, s = swiglu64(x[t] @ w1[e], n)
        a = g * s * u
        y = a @ w2[e]
        o.index_add_(0, t, w[t, k, None] * y)
        dw[t, k] = (do[t] * y).sum(1)
        dy = w[t, k, None] * do[t]
        da = dy @ w2[e].t()
        dh = torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], 1)
        dx.index_add_(0, t, dh @ w1[e].t())
        dw1[e], dw2[e] = x[t].t() @ dh, a.t() @ dy
    return [o, dw, dx, dw1, dw2]


def test_layer_forward_and_backward():
    """The operators as one FP8 layer.  A value's code is off by up to 2^-4 of it, 2^-4 / sqrt(3) in the mean
    square at worst; the result of a chain of m such products is off by about sqrt(2 m) of that relative to its
    norm: up to three products deep (dx, dw1), six quantized operands, 0.09."""
    x, do, w1, w2, idx, w = layer_case()
    L = Experts(600, 3, 8, 512, 256, w1, w2)
    L.forward(x, idx, w)
    L.backward(x, w, do)
    for name, got, ref in zip(("o", "dw", "dx", "dw1", "dw2"), L.results(), layer64(x, do, w1, w2, idx, w)):
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel <= 0.09, (name, rel)
    first = [t.clone() for t in L.results()]
    L.forward(x, idx, w)
    L.backward(x, w, do)
    for a, b in zip(first, L.results()):
        assert torch.equal(a, b)  # bit for bit the same again


def test_layer_from_moe_route():
    """moe_route's selection feeds the sort: the plan's rows are the routing's, and the gates its weights."""
    T, d, E, n, K = 512, 256, 16, 128, 4
    g = gen(8)
    x, wr = randn(g, T, d), randn(g, d, E, std=0.1)
    desc = B.make_desc(T, d, E, n, K)
    rt = B.Routing(desc)
    B.moe_route(desc, x, wr, None, rt, B.workspace(desc, B.MOE_WS_ROUTE))
    p = ops.Plan(T, K, E)
    ops.moe_sort(p, rt.topk_idx.view(T, K))
    assert torch.equal(p.offsets, rt.offsets) and torch.equal(p.counts, rt.counts)
    assert torch.equal(p.row_token, rt.row_token[:p.cap])
    y, o = randn(g, p.cap, d), torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    ops.moe_unpermute(p, y, rt.topk_gate.view(T, K), o)
    ref = torch.zeros(T, d, dtype=torch.float64, device="cuda")
    ref.index_add_(0, rt.row_token[:p.cap].long(), y.double() * rt.row_gate[:p.cap].double()[:, None])
    R.within(o, ref, 2.0 ** -8 * ref.abs() * 1.01 + (K + 4) * 2.0 ** -23 * 8 * 4, "o")


def test_layer_on_another_stream():
    """On a stream that is not current, after work queued on it alone."""
    x, do, w1, w2, idx, w = layer_case(T=300)
    L = Experts(300, 3, 8, 512, 256, w1, w2)
    L.forward(x, idx, w)
    ref = L.o.clone()
    st = torch.cuda.Stream()
    xs, o = torch.zeros_like(x), torch.zeros_like(ref)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(20_000_000)
        xs.copy_(x)
    p = L.p
    ops.moe_sort(p, idx, stream=st)
    ops.moe_fp8_quant_rows(xs, L.xq, L.xs, stream=st)
    ops.moe_fp8_mm(p, L.xq, L.xs, L.w1t, L.w1s, L.h, gather=True, stream=st)
    ops.moe_swiglu_fp8(L.h, L.aq, L.as_, L.a, plan=p, stream=st)
    ops.moe_fp8_mm(p, L.aq, L.as_, L.w2t, L.w2s, L.y, stream=st)
    ops.moe_unpermute(p, L.y, w, o, stream=st)
    st.synchronize()
    assert torch.equal(o, ref)


def test_layer_captured():
    """A captured forward and backward, replayed with new inputs between eager calls on other plans."""
    x, do, w1, w2, idx, w = layer_case()
    L, M = Experts(600, 3, 8, 512, 256, w1, w2), Experts(600, 3, 8, 512, 256, w1, w2)
    bufs = [t.clone() for t in (x, do, idx, w)]
    L.forward(bufs[0], bufs[2], bufs[3])  # first use outside the capture
    L.backward(bufs[0], bufs[3], bufs[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward(bufs[0], bufs[2], bufs[3])
        L.backward(bufs[0], bufs[3], bufs[1])
    for seed in (31, 32, 33):
        nx, ndo, _, _, nidx, nw = layer_case(seed=seed, drop=0.1 * (seed - 31))
        M.forward(nx, nidx, nw)
        M.backward(nx, nw, ndo)
        ref = [t.clone() for t in M.results()]
        for b, v in zip(bufs, (nx, ndo, nidx, nw)):
            b.copy_(v)
        for t in L.results():
            t.fill_(POISON)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(L.results(), ref):
            assert torch.equal(a, b)


def test_two_layers_at_once():
    """Two layers on two streams, several rounds without waiting, give what each gives alone."""
    cases = [layer_case(T=600, seed=41), layer_case(T=350, seed=42, drop=0.3)]
    layers = [Experts(c[0].shape[0], 3, 8, 512, 256, c[2], c[3]) for c in cases]
    refs = []
    for L, (x, do, _, _, idx, w) in zip(layers, cases):
        L.forward(x, idx, w)
        L.backward(x, w, do)
        refs.append([t.clone() for t in L.results()])
        for t in L.results():
            t.fill_(POISON)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for L, (x, do, _, _, idx, w), st in zip(layers, cases, streams):
            with torch.cuda.stream(st):
                L.forward(x, idx, w)
                L.backward(x, w, do)
    torch.cuda.synchronize()
    for L, ref in zip(layers, refs):
        for a, b in zip(L.results(), ref):
            assert torch.equal(a, b)


def test_rows_past_32_bits():
    """Row buffers of several GiB: bytes and elements behind 2^31 (and 2^32) are reached like the first ones."""
    T, K, E, d = 180000, 8, 8, 2048
    g = gen(77)
    idx = choices(g, T, K, E)
    p = sorted_plan(idx, E, 128)
    x = randn(g, T, d)
    slots = p.slot_row.long()
    rows = torch.cat([torch.randint(0, T * K, (150,), generator=g, device="cuda"),
                      torch.topk(slots.view(-1), 150).indices])           # slots, the farthest rows among them
    t, r = rows // K, slots.view(-1)[rows]
    assert int(r.max()) * d > 2 ** 31
    xp = torch.empty(p.cap, d, dtype=torch.bfloat16, device="cuda")
    ops.moe_permute(p, x, xp)
    assert torch.equal(xp[r], x[t])
    q, s = torch.empty(p.cap, d, dtype=torch.uint8, device="cuda"), torch.empty(p.cap, d // 128, device="cuda")
    ops.moe_permute_fp8(p, x, q, s)
    rq, rs = R.quant_rows_ref(x[t])
    assert torch.equal(R.decode(q[r]), R.decode(rq)) and torch.equal(s[r], rs)
    q2, s2 = torch.empty_like(q), torch.empty_like(s)
    ops.moe_fp8_quant_rows(xp, q2, s2, plan=p)
    assert torch.equal(q2[r], q[r]) and torch.equal(s2[r], s[r])
    del q2, s2

    N = 1040
    b, sb = codes(g, E, N, d), torch.rand(E, d // 128, ops.blocks(N), generator=g, device="cuda") + 0.1
    c = torch.full((p.cap, N), POISON, dtype=torch.bfloat16, device="cuda")
    ops.moe_fp8_mm(p, q, s, b, sb, c)
    e = idx.view(-1)[rows].long()
    for i in range(E):
        m = e == i
        av, wv = R.values(q[r[m]], s[r[m]]), weights_ref(b[i], sb[i])
        ref = av @ wv
        R.within(c[r[m]], ref, R.mm_bound(av.abs(), wv.abs(), d, ref, torch.bfloat16), f"expert {i}")

    w = torch.rand(T, K, generator=g, device="cuda")
    o = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    ops.moe_unpermute(p, xp, w, o)
    ref = (w[t].double().sum(1))[:, None] * x[t].double()
    R.within(o[t], ref, (K + 1) * 2.0 ** -23 * ref.abs() + 2.0 ** -8 * ref.abs() * 1.01, "o")
    dw = torch.empty(T, K, device="cuda")
    dyp = torch.empty_like(xp)
    ops.moe_unpermute_bwd(p, x, xp, w, dyp, dw)
    dots = x[t].double().square().sum(1)
    R.within(dw[t, 0], dots, (d + 9) * 2.0 ** -24 * dots * 1.001, "dw")
    assert torch.equal(dyp[r], (w.view(-1)[rows, None] * x[t].float()).bfloat16())
    del dyp

    # the last expert's weight gradient, a few of its values
    (cq, cs), (yq, ys) = ops.column_buffers(p, d), ops.column_buffers(p, 16)
    assert cq.numel() > 2 ** 31
    dy = randn(g, p.cap, 16)
    ops.moe_fp8_quant_cols(p, x, cq, cs, gather=True)
    ops.moe_fp8_quant_cols(p, dy, yq, ys)
    gw = torch.empty(E, d, 16, device="cuda")
    ops.moe_fp8_wgrad(p, cq, cs, yq, ys, gw)
    b0, n = int(p.offsets[E - 1]) // 128, int(p.counts[E - 1])
    nb = -(-n // 128)
    cols = torch.tensor([0, 700, d - 1], device="cuda")
    xv = R.decode(cq[b0:b0 + nb][:, cols]) * cs[b0:b0 + nb][:, cols].double()[..., None]
    yv = R.decode(yq[b0:b0 + nb]) * ys[b0:b0 + nb].double()[..., None]
    xv, yv = xv.transpose(0, 1).reshape(3, -1), yv.transpose(0, 1).reshape(16, -1)
    ref, mag = xv @ yv.t(), xv.abs() @ yv.abs().t()
    R.within(gw[E - 1][cols], ref, R.mm_steps(128 * nb, 3, torch.float32) * mag + 2.0 ** -24 * ref.abs() * 1.001, "dw")


def test_profile_names_the_launches():
    p = ops.Plan(64, 2, 8)
    prof = B.Profiler(8)
    p.attach(prof)
    x = torch.zeros(64, 128, dtype=torch.bfloat16, device="cuda")
    ops.moe_sort(p, choices(gen(1), 64, 2, 8))
    ops.moe_permute(p, x, torch.zeros(p.cap, 128, dtype=torch.bfloat16, device="cuda"))
    p.detach()
    ops.moe_sort(p, choices(gen(1), 64, 2, 8))
    torch.cuda.synchronize()
    rec = prof.records()
    assert [ops.KERNEL_NAMES[k] for k, _ in rec] == ["sort", "permute"] and all(ms >= 0 for _, ms in rec)
    prof.close()
