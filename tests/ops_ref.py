"""The operators of include/moe_ops.h in float64, written from their formulas
(loops over experts and blocks; nothing shared with the kernels), and the
error bounds their results are held to.

Rounding to a type is off by at most half a step: bf16 2^-8, fp32 2^-24, E4M3
2^-4 of the value."""
import numpy as np
import torch

TINY = 2.0 ** -126
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def plan_ref(idx, E, align):
    """offsets, counts, row_token (-1 between segments), slot_row by counting."""
    T, K = idx.shape
    of = [[] for _ in range(E)]
    for s, e in enumerate(idx.reshape(-1).tolist()):
        if 0 <= e < E:
            of[e].append(s)
    cap = T * K + min(E, T * K) * (align - 1)
    offsets, row_token, slot_row = [0], np.full(cap, -1, np.int64), np.full(T * K, -1, np.int64)
    for rows in of:
        at = offsets[-1]
        for j, s in enumerate(rows):
            row_token[at + j], slot_row[s] = s // K, at + j
        offsets.append(at + -(-len(rows) // align) * align)
    return dict(offsets=np.array(offsets), counts=np.array([len(r) for r in of]), row_token=row_token,
                slot_row=slot_row.reshape(T, K), cap=cap)


def e4m3_values():
    """The value of every code, from the format: 1 sign, 4 exponent (bias 7), 3 mantissa bits, 0x7f NaN."""
    v = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        x = float("nan") if (c & 0x7f) == 0x7f else x
        v.append(-x if c & 0x80 else x)
    return torch.tensor(v, dtype=torch.float64)


def decode(codes):
    """Codes (uint8 or float8 tensor) as float64 values."""
    return e4m3_values().to(codes.device)[codes.view(torch.uint8).long()]


def encode(v):
    """Codes of float64 values in [-448, 448]: nearest, ties to the even code."""
    pos = e4m3_values()[:127].to(v.device)  # ascending magnitudes, codes 0..126
    a = v.abs().clamp(max=448.0)
    hi = torch.searchsorted(pos, a).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - pos[lo], pos[hi] - a
    take_lo = (dl < dh) | ((dl == dh) & (lo % 2 == 0))
    c = torch.where(take_lo, lo, hi)
    return (c + 128 * torch.signbit(v).long()).to(torch.uint8)


def scale_of(amax):
    """max(amax / 448, 2^-126) in fp32.  The quotient is taken in float64 and rounded once more, which gives
    the fp32 quotient's bits (53 >= 2 * 24 + 2); torch's own fp32 division by a number multiplies by the
    rounded reciprocal on the GPU."""
    return torch.clamp((amax.double() / 448.0).float(), min=TINY)


def block_codes(x):
    """One block (any shape, float tensor) -> codes, scale (fp32), by the definition's fp32 steps."""
    x = x.float()
    amax = x.abs().max()
    if not torch.isfinite(x).all():
        return None, torch.full((), float("nan"), device=x.device)
    s = scale_of(amax)
    return encode((x * (1.0 / s)).double()), s


def quant_rows_ref(x):
    """codes [R, C], scales [R, ceil(C/128)] of finite x, all rows of a block column at once."""
    q, s = torch.empty(x.shape, dtype=torch.uint8, device=x.device), []
    for c0 in range(0, x.shape[1], 128):
        v = x[:, c0:c0 + 128].float()
        sc = scale_of(v.abs().amax(1))
        q[:, c0:c0 + 128] = encode((v * (1.0 / sc)[:, None]).double())
        s.append(sc)
    return q, torch.stack(s, 1)


def values(q, s):
    """float64 values of codes [R, C] with scales [R, ceil(C/128)]."""
    return decode(q) * torch.repeat_interleave(s.double(), 128, 1)[:, :q.shape[1]]


def mm_steps(K, per_block, out):
    """|error| of a product's sums relative to sum |a b|: every one of the K products and `per_block` more
    operations per block may round once in fp32 (one step each, 2^-23, so that a truncating adder is covered).
    A bf16 result comes from the 8-bit matrix cores: they align eight neighbouring products to the largest
    of them, whose leading power of two is 2^E, and keep multiples of 2^(E - 13).  Seven products may lose
    less than one such unit each, and 2^E is at most the largest |a b| of the eight, hence at most their
    sum: less than 7 * 2^-13 of sum |a b|."""
    return (K + per_block * -(-K // 128)) * 2.0 ** -23 + (7 * 2.0 ** -13 if out == torch.bfloat16 else 0.0)


def mm_bound(a_abs, b_abs, K, ref, out):
    """|error| an element may have: its sums' (two operations per block join the block's), and its type's rounding."""
    return mm_steps(K, 2, out) * (a_abs @ b_abs) + HALF[out] * (ref.abs() * (1 + 2.0 ** -7)) + 1e-300


def within(got, ref, bound, what=""):
    """Every element finite where the reference is and inside its bound."""
    got, ref = got.double(), ref.double()
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((got - ref).abs()[bad].max()),
                           float((((got - ref).abs()) / bound.clamp(min=1e-300))[bad].max()))
