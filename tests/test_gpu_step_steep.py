"""bf16 updates whose singular values fall steeply, as those of weight gradients do: several
steps on A = X X^T alone enlarge what A lost in its sums and its two fp16 parts.  Every
kind of tile of the products, against float64, with the error held apart from the
result's own rounding."""
import math

import pytest
import torch

from fine_grained_mixture_top_amd import ops

import step_ref as R

pytestmark = pytest.mark.gpu


def spectrum(kind, m):
    i = torch.arange(1, m + 1, dtype=torch.float64, device="cuda")
    if kind == "squares":
        return i ** -2
    large, rest = {"one": (1, 1e-3), "two": (2, 1e-3), "sixteen": (16, 1e-2)}[kind]
    return torch.where(i <= large, 1.0, rest)


KINDS = ("one", "two", "squares", "sixteen")


def steep(kind, M, N, g, dtype=torch.bfloat16):
    m, k = min(M, N), max(M, N)
    u = torch.linalg.qr(torch.randn(m, m, generator=g, device="cuda", dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(k, m, generator=g, device="cuda", dtype=torch.float64))[0]
    w = (u * spectrum(kind, m)) @ v.t()
    return (w if M <= N else w.t()).contiguous().to(dtype)


def lost(m, k, steps=5):
    """What several steps on A alone may add to a result, relative to its norm.

    An element of A is off by at most 2^-23 in its two parts (2^-24 and less in root mean square) and by its
    sum's roundings: one for every eight products, half a step 2^-25 .. 2^-24 of the sum so far (root mean square of
    a step's half at most 2^-25), which grows evenly: 2^-25 sqrt(k / 8 / 3).  Together 2^-25 sqrt(k / 24 + 4) of an element, and for
    one large direction over all rows (elements about 1 / m) that over sqrt(m) of what a small direction's A has.  There every
    step's P = a + b A + .. loses |b| / a of A's error, grown by a^2 with every step before:
    |b| / a (1 + a^2 + .. + a^(2 steps - 2)).  The matrices of later steps are rounded too, 1 / a^2 of that and less
    each: a factor of two covers these and chance."""
    a, b, _ = R.QUINTIC
    grown = -b / a * (a ** (2 * steps) - 1) / (a * a - 1)
    return 2 * grown * 2.0 ** -25 * math.sqrt((k / 24 + 4) / m)


def check(o, w, steps, tol, what):
    """|o - ref|^2 is the rounding's and the rest's.  The rounding's sum of squares is that of the rounded reference but for
    chance: squares of evenly spread errors vary by 0.9 of their mean; four standard deviations."""
    ref = R.ortho_ref(w, steps, [R.QUINTIC] * steps)
    off, own = float((o.double() - ref).norm()), float((ref.to(o.dtype).double() - ref).norm())
    chance = own * own * 4 * 0.9 * math.sqrt(2 / ref.numel())
    rest = math.sqrt(max(off * off - own * own - chance, 0.0)) / float(ref.norm())
    assert rest <= tol, (what, rest, tol)


@pytest.mark.parametrize("E,M,N", [
    (1, 160, 160), (1, 200, 1536), (1, 1536, 256),            # tiles of 64
    (4, 1024, 1024),                                          # 128, three stages ahead
    (128, 256, 1536), (24, 720, 1040), (24, 1040, 721),       # 128, one stage ahead
    (342, 300, 320), (342, 320, 300),                         # 256
    (4, 128, 1536), (4, 1000, 100), (4, 64, 640), (4, 17, 300),  # up to 128 rows
])
def test_steep_spectra(E, M, N):
    g = torch.Generator("cuda").manual_seed(E + M + N)
    made = [steep(kind, M, N, g) for kind in KINDS]
    w = torch.stack([made[e % len(KINDS)] for e in range(E)]) if E > 1 else None
    tol = lost(min(M, N), max(M, N))
    if E == 1:
        h = ops.Ortho(1, M, N)
        for kind, one in zip(KINDS, made):
            o = torch.empty_like(one)[None]
            ops.moe_orthogonalize(h, one[None], o)
            check(o[0], one, 5, tol, kind)
        return
    o = torch.empty_like(w)
    ops.moe_orthogonalize(ops.Ortho(E, M, N), w, o)
    for e in (0, 1, 2, 3, E - 4, E - 3, E - 2, E - 1):
        check(o[e], w[e], 5, tol, (e, KINDS[e % len(KINDS)]))


@pytest.mark.parametrize("M,N", [(129, 50000), (40000, 200), (130, 9000)])
def test_steep_spectra_of_long_matrices(M, N):
    """Sums over a long side lose more (`lost` for 129 x 50000 without its factor of two: 3.3e-3); they are taken in
    pieces, or steps in smaller groups, so that no more than 1.5e-3 is added."""
    g = torch.Generator("cuda").manual_seed(M + N)
    h = ops.Ortho(1, M, N)
    for kind in KINDS:
        w = steep(kind, M, N, g)
        o = torch.empty_like(w)[None]
        ops.moe_orthogonalize(h, w[None], o)
        check(o[0], w, 5, 1.5e-3, kind)


@pytest.mark.parametrize("E,M,N", [(1, 129, 4000), (1, 1000, 100), (24, 300, 320), (342, 320, 300)])
def test_steep_spectra_in_fp32(E, M, N):
    """Step by step: every step is off by 2^-22 of X's norm and carries that on, as for any other spectrum."""
    g = torch.Generator("cuda").manual_seed(E + M + N)
    made = [steep(kind, M, N, g, torch.float32) for kind in KINDS]
    w = torch.stack([made[e % len(KINDS)] for e in range(max(E, len(KINDS)))])
    o = torch.empty_like(w)
    ops.moe_orthogonalize(ops.Ortho(len(w), M, N, dtype=torch.float32), w, o)
    for e in range(4):
        ref = R.ortho_ref(w[e], 5, [R.QUINTIC] * 5)
        tol = R.ortho_tolerance(torch.float32, 5, [R.QUINTIC]) + R.HALF[torch.float32]
        assert float((o[e].double() - ref).norm()) <= tol * float(ref.norm()), KINDS[e]


CUBELESS = (1.25, 0.0, -0.25)  # s (5 - s^4) / 4: rises to 1 and stays there


@pytest.mark.parametrize("E,M,N,coef,steps", [
    (1, 1, 40, R.SMOOTH, 64), (3, 500, 1, R.SMOOTH, 40), (1, 2, 300, R.SMOOTH, 40), (1, 30, 100, CUBELESS, 64),
    (1, 140, 200, CUBELESS, 64), (1, 140, 200, R.SMOOTH, 40), (30, 300, 170, CUBELESS, 40),
])
def test_many_steps(E, M, N, coef, steps):
    """Steps without end, in groups that neither lose more nor hold a larger Q than a few do: the singular values
    are 1 in the end, and more steps only mend what the ones before lost.  One dominant direction, which what
    the last groups add is not seen behind: each may add 1.5e-3, and three of those are a bound."""
    g = torch.Generator("cuda").manual_seed(M + N + steps)
    w = torch.stack([steep("one", M, N, g) for _ in range(E)])
    o = torch.empty_like(w)
    ops.moe_orthogonalize(ops.Ortho(E, M, N, steps=steps, coef=coef), w, o)
    for e in range(E):
        ref = R.ortho_ref(w[e], steps, [coef] * steps)
        off = float((o[e].double() - ref).norm())
        assert off <= (R.HALF[o.dtype] + 3 * 1.5e-3) * float(ref.norm()), (e, off / float(ref.norm()))
