"""The operators of include/moe_step_ops.h in float64, written from their
formulas (nothing shared with the kernels), and the error bounds their results
are held to.

Rounding to a type is off by at most half a step: bf16 2^-8, fp32 2^-24 of the
value.  A sum of fp32 terms is off by at most its chain of additions times 2^-24
of the sum of magnitudes."""
import torch

NEG = float("-inf")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def within(got, ref, bound, what=""):
    """Equal infinities and NaNs, everything else inside its bound."""
    got, ref = got.double(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), (what, "NaN")
    inf = torch.isinf(ref)
    assert torch.equal(got[inf], ref[inf]), (what, "inf")
    fine = torch.isfinite(ref)
    assert bool(torch.isfinite(got[fine]).all()), (what, "not finite")
    off = (got - ref).abs()[fine]
    bound = bound.expand_as(ref)[fine] if isinstance(bound, torch.Tensor) else torch.full_like(off, bound)
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(off[bad].max()), float((off / bound.clamp(min=1e-300))[bad].max()))


# ---------------------------------------------------------------- balance

def balance_ref(z, idx, valid=None):
    """Everything moe_balance gives, in float64, and p with zeros for tokens that do not count."""
    T, E = z.shape
    K = idx.shape[1]
    z = z.double()
    counting = (z > NEG).any(1) | torch.isnan(z).any(1)
    if valid is not None:
        counting = counting & valid.bool()
    p, lse = torch.zeros_like(z), torch.full((T,), NEG, dtype=torch.float64, device=z.device)
    if counting.any():
        p[counting] = torch.softmax(z[counting], 1)
        lse[counting] = torch.logsumexp(z[counting], 1)
    n = int(counting.sum())
    counts = torch.zeros(E, dtype=torch.int64, device=z.device)
    for k in range(K):
        e = idx[:, k].long()
        e = e[counting & (e >= 0) & (e < E)]
        counts += torch.bincount(e, minlength=E)
    per = 1.0 / n if n else 0.0
    load = p.sum(0) * per
    loss = torch.stack([(counts.double() * load).sum() * per * E / K, (lse[counting] ** 2).sum() * per])
    return dict(counts=counts, n=n, load=load, lse=lse, loss=loss, p=p, counting=counting)


def spread(z):
    """The largest distance of a finite logit from its row's maximum."""
    z = z.double()
    m = z.amax(1, keepdim=True)
    d = torch.where(torch.isfinite(z) & torch.isfinite(m), m - z, torch.zeros_like(z))
    return float(d.max()) if d.numel() else 0.0


def balance_steps(z):
    """Relative error of a mean probability in steps of 2^-23.  An exponential of x = z - max: x and x log2(e)
    round and log2(e) itself is rounded, |x| 2^-24 each, and the instruction 2^-23; the row's sum and its
    reciprocal: at most 16 additions in a lane, 6 between lanes, 2 more.  Then a lane's sum over its rows
    (at most T / 2048 + 64, or for the one-workgroup form T L / 512 <= 64 as T E <= 2^14), 6 between lanes, 8
    waves, 512 / 16 lines and 16 of their sums, the multiplication by 1 / n."""
    return 2 * spread(z) + 24 + z.shape[0] / 2048 + 64 + 6 + 8 + 32 + 16 + 4


def lse_bound(lse):
    """max + ln(2) log2(sum): the sum's relative error is at most sum_i p_i (2 |x_i| + 24) 2^-23, and sum p |x| is at
    most the entropy, ln 1024 < 7; the logarithm's instruction, its constant and the addition: 2^-22 of 7 + |lse|."""
    return torch.where(torch.isfinite(lse), (lse.abs() + 7) * 2.0 ** -22 + 38 * 2.0 ** -23, torch.zeros_like(lse))


def balance_bwd_ref(z, idx, ref, d_loss, gate=None, d_gate=None):
    """(dz, its bound without the result's rounding) in float64."""
    T, E = z.shape
    K = idx.shape[1]
    n = max(ref["n"], 1)
    gb, gz = float(d_loss[0]), float(d_loss[1])
    p, f = ref["p"], ref["counts"].double() * (gb * E / (n * n * K))
    lse = torch.where(ref["counting"], ref["lse"], torch.zeros_like(ref["lse"]))
    inner = (p * f).sum(1, keepdim=True)
    dz = p * (f - inner + (2.0 * gz / n) * lse[:, None])
    mag = p * (f.abs() + (p * f.abs()).sum(1, keepdim=True) + abs(2.0 * gz / n) * lse.abs()[:, None])
    # p: its exponent's three roundings and lse's error; the sums: E terms at most 16 in a lane and 6 lanes; products
    # (above 32 lse is not used for p)
    finite = lse.abs().max().clamp(max=32.0) if T else 0.0
    bound = mag * ((3 * spread(z) + 4 * float(finite) + 14 + 38 + 24 + 16) * 2.0 ** -23)
    if gate is not None:
        there = (idx >= 0) & (idx < E)
        g = torch.where(there, gate.double(), 0.0)
        d = torch.where(there, d_gate.double(), 0.0)
        v = g * (d - (g * d).sum(1, keepdim=True))
        m = g.abs() * (d.abs() + (g * d).abs().sum(1, keepdim=True))
        at = torch.where(there, idx, torch.zeros_like(idx)).long()
        dz = dz.scatter_add(1, at, v)
        # the inner sum: K terms; the products; then up to K values join an element
        bound = bound.scatter_add(1, at, m * ((2 * K + 8) * 2.0 ** -23)) + dz.abs() * K * 2.0 ** -24
    return dz, bound


# ---------------------------------------------------------------- orthogonalised updates

QUINTIC = (3.4445, -4.7750, 2.0315)
SMOOTH = (1.875, -1.25, 0.375)  # x (15 - 10 x^2 + 3 x^4) / 8: rises to 1 and stays there


def ortho_ref(g, steps, coef, eps=1e-7, scale=1.0):
    """One matrix in float64; coef [steps][3]."""
    x = g.double()
    x = x / (x.norm() + eps) if x.any() else x
    for i in range(steps):
        a, b, c = coef[i]
        y = x @ x.t()
        x = a * x + b * (y @ x) + c * (y @ (y @ x))
    return scale * x


def ortho_tolerance(dtype, steps, coef, smallest=0.0):
    """Error of a result before its rounding, relative to its Frobenius norm.

    A step's map of the singular values, f(s) = s p(s^2), carries an error of X on by at most its steepest
    difference, which is below 4 for QUINTIC on 0 .. 1.25 (3.9 at 1.2, a = 3.44 at 0) and a = 1.875 for SMOOTH;
    for SMOOTH, concave and at most 1, all steps together carry it on by at most 1 / `smallest`, X_0's smallest
    singular value.  One step a group: a step is off by 2^-22 of X's norm, three products' parts and sums.
      Several steps a group (bf16): what A's sums and parts lost, 2 * 2^-24 of its largest singular value, grows by
    a^2 with every step that A itself goes through, the last P of the group sees it times |b| / a, and the ones before
    it lose less by a^2 each."""
    a, b, _ = coef[0]
    steep = 4.0 if tuple(coef[0]) == QUINTIC else a
    each = steep ** steps / (steep - 1)
    if smallest:
        each = min(each, steps / smallest)
    tol = each * 2.0 ** -22
    if dtype == torch.bfloat16:
        group = 1
        while group < steps and a ** (group + 1) <= 512:
            group += 1
        grown = 2 * abs(b) / a * a ** (2 * (group - 1)) * 2.0 ** -24 / (1 - a ** -2)
        tol += grown * -(-steps // group)
    return tol


# ---------------------------------------------------------------- MXFP4 weights

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def power(e):
    """2^e in float64 from its bits (a GPU's pow may be off by a step)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def mxfp4_values(q, s):
    """float64 values [..., K] of codes [..., K/2] and scale codes [..., K/32]."""
    t = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=q.device)
    v = torch.stack([t[(q & 15).long()], t[(q >> 4).long()]], -1).flatten(-2)
    f = power(s.long() - 127)
    f = torch.where(s == 255, torch.full_like(f, float("nan")), f)
    return v * torch.repeat_interleave(f, 32, -1)


def mxfp4_codes(w):
    """q [E, N, K/2], s [E, N, K/32] of w [E, K, N], by the definition in float64."""
    E, K, N = w.shape
    v = w.double().transpose(1, 2).reshape(E, N, K // 32, 32)
    m = v.abs().amax(-1)
    finite = torch.isfinite(v).all(-1)
    e = torch.frexp(torch.where(finite, m, torch.ones_like(m)))[1] - 1 - 2
    e = torch.where(m > 0, e, torch.full_like(e, -127)).clamp(min=-127)
    a = v.abs() * power(-e)[..., None]
    mags = torch.tensor(E2M1, dtype=torch.float64, device=w.device)
    near = (a[..., None] - mags).abs()
    best = near.amin(-1, keepdim=True)
    # of two equally near values the one with the even code; from 6 on: 6
    even = torch.arange(8, device=w.device) % 2 == 0
    c = torch.where(near == best, torch.where(even, 0, 1), 2).argmin(-1)
    c = torch.where(finite[..., None], c + 8 * torch.signbit(v).long(), torch.zeros_like(c)).view(E, N, K)
    s = torch.where(finite, e + 127, torch.full_like(e, 255))
    return (c[..., ::2] + 16 * c[..., 1::2]).to(torch.uint8), s.to(torch.uint8)


def mxfp4_mm_bound(a, w, K, ref, out):
    """Every one of the K exact products, and 16 sums of the waves', may round once in fp32 (one step each, 2^-23, so
    that an adder which cuts off is covered), and the result once in its type."""
    return (K + 16) * 2.0 ** -23 * (a.abs() @ w.abs().t()) + HALF[out] * ref.abs() * (1 + 2.0 ** -7) + 1e-37
