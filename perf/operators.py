"""Cases of the operators around the experts' products: tokens sorted by expert
and back, the 8-bit product with a scale per block of 128, and SwiGLU with its
result quantized for the next product.

``run`` computes a case in plain torch operations, or with ``own`` set through
``fine_grained_mixture_top_amd.ops``.

Conventions (those of include/moe_ops.h): expert ids outside 0..E-1 are
dropped; expert e's rows start at offsets[e], a multiple of ``align``; an E4M3
block has the scale s = max(amax / 448, 2^-126) and the codes e4m3(x * (1 / s)),
with s, 1 / s and the product in fp32.  Buffers that an operator fills in part
start as zeros here, so that the rest of them compares equal.
"""
import math

import torch

own = False

TINY = 2.0 ** -126  # smallest scale
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a served batch, the production-shaped layer's width and experts
        dict(name="dispatch-one-token", op="dispatch", T=1, K=8, E=256, d=7168, align=1, dtype="bf16", drop=0.0, skew=0.0),
        # one training step's tokens of the 7B-shaped layer, segments padded for the weight gradients
        dict(name="dispatch-train", op="dispatch", T=32768, K=8, E=128, d=1536, align=128, dtype="bf16", drop=0.0, skew=0.5),
        # prefill of a ragged batch into 8-bit rows, a tenth of the choices dropped (a capacity limit, or other ranks' experts)
        dict(name="dispatch-fp8-ragged", op="dispatch_fp8", T=4099, K=4, E=64, d=2048, align=1, dtype="bf16", drop=0.1, skew=0.3),
        # a small served batch's outputs gathered back
        dict(name="combine-decode", op="combine", T=8, K=8, E=256, d=7168, align=1, dtype="bf16", drop=0.0, skew=0.0, weighted=True),
        # the backward of a training step's combination: row and weight gradients
        dict(name="combine-bwd-train", op="combine_bwd", T=16384, K=8, E=128, d=2048, align=1, dtype="bf16", drop=0.05, skew=0.3),
        # decode: few rows, most experts touched, the weights' bytes are the work
        dict(name="product-decode", op="product", T=16, K=8, E=256, d=2048, n=512, align=1, out="bf16", gather=True, drop=0.0, skew=0.0),
        # the OLMoE-shaped layer's up-projection in training or prefill
        dict(name="product-up", op="product", T=32768, K=8, E=64, d=2048, n=2048, align=1, out="bf16", gather=True, drop=0.0, skew=0.2),
        # input gradient from bf16 output gradients, odd sizes, some experts without rows, fp32 result
        dict(name="product-dgrad-ragged", op="dgrad", T=1001, K=3, E=24, d=1040, n=720, align=1, out="f32", drop=0.2, skew=1.5),
        # weight gradient of an up-projection of the granularity sweep, both operands quantized along the rows
        dict(name="wgrad-train", op="wgrad", T=16384, K=4, E=64, d=2048, n=1024, align=128, out="bf16", drop=0.0, skew=0.2),
        # the weights quantized after an optimizer step, both layouts
        dict(name="weights-step", op="weights", E=64, d=2048, n=1024, dtype="bf16"),
        # between the two products of the 7B-shaped layer
        dict(name="swiglu-train", op="swiglu", R=262144, n=256, dtype="bf16"),
        # the activation's gradient for a short ragged batch
        dict(name="swiglu-bwd-ragged", op="swiglu_bwd", R=2999, n=1040, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dispatch", "dispatch_fp8", "combine", "combine_bwd", "product", "product", "dgrad", "wgrad", "weights",
                     "swiglu", "swiglu_bwd"])
    if op == "weights":
        return dict(op=op, E=_log(rng, 1, 64), d=16 * _log(rng, 8, 160), n=16 * _log(rng, 4, 128),
                    dtype=rng.choice(["bf16", "f32"]))
    if op in ("swiglu", "swiglu_bwd"):
        return dict(op=op, R=_log(rng, 1, 60000), n=16 * _log(rng, 4, 128), dtype=rng.choice(["bf16", "f32"]))
    E = 8 * _log(rng, 1, 32)
    K = rng.randint(1, min(8, E))
    c = dict(op=op, T=_log(rng, 1, 16384), K=K, E=E, d=16 * _log(rng, 8, 200), drop=rng.choice([0.0, 0.0, 0.15]),
             skew=round(rng.uniform(0.0, 0.6), 2))
    if op in ("dispatch", "dispatch_fp8", "combine", "combine_bwd"):
        c["align"] = rng.choice([1, 1, 16, 128])
        c["dtype"] = "bf16" if op == "dispatch_fp8" else rng.choice(["bf16", "bf16", "f32"])
        if op == "combine":
            c["weighted"] = rng.random() < 0.7
        return c
    c["d"] = 16 * _log(rng, 8, 128)
    c["n"] = 16 * _log(rng, 4, 128)
    c["E"] = E = min(E, 64)
    c["T"] = min(c["T"], 8192)
    c["out"] = rng.choice(["bf16", "bf16", "f32"])
    c["align"] = 128 if op == "wgrad" else rng.choice([1, 1, 128])
    if op == "product":
        c["gather"] = rng.random() < 0.5
    return c


# ---------------------------------------------------------------- inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _cap(c):
    return c["T"] * c["K"] + min(c["E"], c["T"] * c["K"]) * (c["align"] - 1)


def _blocks(n):
    return (n + 127) // 128


def _choices(c, g):
    """Experts of every token, distinct within a token as a router's top-K gives them."""
    T, K, E = c["T"], c["K"], c["E"]
    bias = -c["skew"] * torch.log(1.0 + torch.arange(E, device="cuda", dtype=torch.float32))
    bias = bias[torch.randperm(E, generator=g, device="cuda")]
    idx = torch.topk(torch.randn(T, E, generator=g, device="cuda") + bias, K, dim=1).indices.to(torch.int32)
    if c["drop"]:
        idx = torch.where(torch.rand(T, K, generator=g, device="cuda") < c["drop"], torch.full_like(idx, -1), idx)
    return idx.contiguous()


def _inputs(c, seed):
    g = torch.Generator("cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    s = dict(case=dict(c))
    op = c["op"]
    if "K" in c:
        s["idx"] = _choices(c, g)
        cap = _cap(c)
    if op in ("dispatch", "dispatch_fp8"):
        s["x"] = normal(c["T"], c["d"], dtype=_DT[c["dtype"]])
    elif op == "combine":
        s["y"] = normal(cap, c["d"], dtype=_DT[c["dtype"]])
        s["w"] = torch.softmax(torch.randn(c["T"], c["K"], generator=g, device="cuda"), 1) if c["weighted"] else None
    elif op == "combine_bwd":
        s["do"] = normal(c["T"], c["d"], dtype=_DT[c["dtype"]])
        s["y"] = normal(cap, c["d"], dtype=_DT[c["dtype"]])
        s["w"] = torch.softmax(torch.randn(c["T"], c["K"], generator=g, device="cuda"), 1)
    elif op == "product":
        rows = c["T"] if c["gather"] else cap
        s["a"], s["sa"] = _quant_rows(normal(rows, c["d"]))
        _, s["b"], s["sb"] = _quant_weights(normal(c["E"], c["d"], c["n"], std=0.02))
    elif op == "dgrad":
        s["dy"] = normal(cap, c["n"])
        s["b"], _, s["sb"] = _quant_weights(normal(c["E"], c["d"], c["n"], std=0.02))
    elif op == "wgrad":
        s["x"], s["dy"] = normal(c["T"], c["d"]), normal(cap, c["n"])
    elif op == "weights":
        s["w"] = normal(c["E"], c["d"], c["n"], std=0.02, dtype=_DT[c["dtype"]])
    elif op in ("swiglu", "swiglu_bwd"):
        s["h"] = normal(c["R"], 2 * c["n"], dtype=_DT[c["dtype"]])
        if op == "swiglu_bwd":
            s["da"] = normal(c["R"], c["n"], dtype=_DT[c["dtype"]])
    return s


def prepare(case, seed):
    c = case
    s = _inputs(c, seed)
    op = c["op"]
    if "K" in c and not op.startswith("dispatch"):
        s["rows"] = _sort(s["idx"], c)
        s["most"] = max(1, int(s["rows"]["counts"].max()))  # rows of the fullest expert
    if own:
        _prepare_own(s, c)
    return s


# ---------------------------------------------------------------- plain forms

def _sort(idx, c):
    """The rows of every expert: a stable sort of the slots by expert."""
    T, K, E, align = c["T"], c["K"], c["E"], c["align"]
    cap = _cap(c)
    flat = idx.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.argsort(key, stable=True)
    sk = key[order]
    counts = torch.bincount(key, minlength=E + 1)[:E]
    zero = torch.zeros(1, dtype=torch.long, device=idx.device)
    first = torch.cat([zero, torch.cumsum(counts, 0)])
    offsets = torch.cat([zero, torch.cumsum((counts + align - 1) // align * align, 0)])
    row = offsets[sk] + torch.arange(T * K, device=idx.device) - first[sk]
    kept = sk < E
    slot_row = torch.full((T * K,), -1, dtype=torch.long, device=idx.device)
    slot_row[order] = torch.where(kept, row, torch.full_like(row, -1))
    row_token = torch.zeros(cap + 1, dtype=torch.long, device=idx.device)
    row_token = torch.where(torch.arange(cap + 1, device=idx.device) < offsets[E], row_token - 1, row_token)
    row_token[torch.where(kept, row, torch.full_like(row, cap))] = torch.div(order, K, rounding_mode="floor")
    return dict(offsets=offsets.int(), counts=counts.int(), row_token=row_token[:cap].int(),
                slot_row=slot_row.int().view(T, K))


def _spread(values, rows, cap):
    """values [n, ...] at the rows given, -1 for none, in zeros [cap, ...]."""
    out = torch.zeros((cap + 1,) + tuple(values.shape[1:]), dtype=values.dtype, device=values.device)
    rows = rows.reshape(-1).long()
    out[torch.where(rows < 0, torch.full_like(rows, cap), rows)] = values
    return out[:cap]


def _pick(values, rows):
    """values[rows] in fp32, zeros where a row is -1."""
    got = values.float()[rows.long().clamp(min=0)]
    return torch.where((rows >= 0).unsqueeze(-1), got, torch.zeros_like(got))


def _scale(amax):
    # (a tensor of 448: dividing by a number multiplies by its rounded reciprocal on the GPU)
    return torch.clamp(amax / torch.full_like(amax, 448.0), min=TINY)


def _codes(x, inv):
    return torch.clamp(x * inv, -448.0, 448.0).to(E4M3)


def _pad(x, dim, to):
    short = -x.shape[dim] % to
    if not short:
        return x
    shape = list(x.shape)
    shape[dim] = short
    return torch.cat([x, torch.zeros(shape, dtype=x.dtype, device=x.device)], dim)


def _quant_rows(x):
    R, C = x.shape
    v = _pad(x.float(), 1, 128).view(R, -1, 128)
    s = _scale(v.abs().amax(2))
    return _codes(v, (1.0 / s).unsqueeze(2)).view(R, -1)[:, :C].contiguous(), s


def _quant_weights(w):
    """codes [E, d, n], codes [E, n, d], scales [E, d/128, n/128]."""
    E, d, n = w.shape
    v = _pad(_pad(w.float(), 1, 128), 2, 128).view(E, _blocks(d), 128, _blocks(n), 128)
    s = _scale(v.abs().amax(4).amax(2))
    q = _codes(v, (1.0 / s)[:, :, None, :, None]).view(E, 128 * _blocks(d), 128 * _blocks(n))[:, :d, :n]
    return q.contiguous(), q.transpose(1, 2).contiguous(), s


def _wide(s, n):
    """A scale per 128 values as one per value."""
    return s.repeat_interleave(128, dim=-1)[..., :n]


def _table(rows, most):
    """[E, most] row numbers and which of them are there."""
    at = torch.arange(most, device=rows["counts"].device)[None, :]
    there = at < rows["counts"][:, None]
    return torch.where(there, rows["offsets"][:-1, None] + at, torch.zeros_like(rows["offsets"][:-1, None] + at)).long(), there


def _grouped(a, w, rows, most, cap, out, gather):
    """a fp32 rows times w [E, K, N] fp32 by segment."""
    r, there = _table(rows, most)
    take = rows["row_token"].long()[r].clamp(min=0) if gather else r
    c = torch.bmm(a[take], w).to(out)
    return _spread(c.view(-1, c.shape[2]), torch.where(there, r, torch.full_like(r, -1)), cap)


def _columns(x, r, there):
    """Rows r [E, most] of x with the codes of each column's blocks of 128 rows as the values they stand for."""
    v = x.float()[r]
    v = torch.where(there.unsqueeze(-1), v, torch.zeros_like(v))
    E, most, C = v.shape
    v = _pad(v, 1, 128).view(E, -1, 128, C)
    s = _scale(v.abs().amax(2, keepdim=True))
    return (_codes(v, 1.0 / s).float() * s).view(E, -1, C)


def _dgrad_plain(s, c):
    dy, sy = _quant_rows(s["dy"])
    w = s["b"].float() * _wide(_wide(s["sb"], c["n"]).transpose(1, 2), c["d"]).transpose(1, 2)
    return _grouped(dy.float() * _wide(sy, c["n"]), w.transpose(1, 2).contiguous(), s["rows"], s["most"], _cap(c), _DT[c["out"]],
                    False)


def _plain(s):
    c = s["case"]
    op = c["op"]
    if op in ("dispatch", "dispatch_fp8"):
        rows = _sort(s["idx"], c)
        if op == "dispatch":
            return dict(rows, xp=_spread(s["x"].repeat_interleave(c["K"], 0), rows["slot_row"], _cap(c)))
        q, sc = _quant_rows(s["x"])
        q = _spread(q.view(torch.uint8).repeat_interleave(c["K"], 0), rows["slot_row"], _cap(c))
        return dict(rows, q=q.view(E4M3), s=_spread(sc.repeat_interleave(c["K"], 0), rows["slot_row"], _cap(c)))
    if op == "combine":
        y = _pick(s["y"], s["rows"]["slot_row"])
        y = y * s["w"].unsqueeze(-1) if s["w"] is not None else y
        return y.sum(1).to(s["y"].dtype)
    if op == "combine_bwd":
        slots = s["rows"]["slot_row"]
        do = s["do"].float().unsqueeze(1)
        dy = (do * s["w"].unsqueeze(-1)).to(s["do"].dtype)
        return dict(dy=_spread(dy.view(-1, c["d"]), slots, _cap(c)), dw=(do * _pick(s["y"], slots)).sum(2))
    if op == "product":
        a = s["a"].float() * _wide(s["sa"], c["d"])
        w = s["b"].float() * _wide(_wide(s["sb"].transpose(1, 2), c["d"]).transpose(1, 2), c["n"]).transpose(1, 2)
        return _grouped(a, w.transpose(1, 2).contiguous(), s["rows"], s["most"], _cap(c), _DT[c["out"]], c["gather"])
    if op == "dgrad":
        return _dgrad_plain(s, c)
    if op == "wgrad":
        r, there = _table(s["rows"], s["most"])
        x = _columns(s["x"], s["rows"]["row_token"].long()[r].clamp(min=0), there)
        dy = _columns(s["dy"], r, there)
        return torch.bmm(x.transpose(1, 2).contiguous(), dy).to(_DT[c["out"]])
    if op == "weights":
        return _quant_weights(s["w"])
    h = s["h"].float()
    g, u = h[:, :c["n"]], h[:, c["n"]:]
    sg = 1.0 / (1.0 + torch.exp(-g))
    if op == "swiglu":
        return _quant_rows(g * sg * u)
    da = s["da"].float()
    return torch.cat([da * u * sg * (1.0 + g * (1.0 - sg)), da * g * sg], 1).to(s["h"].dtype)


# ---------------------------------------------------------------- the framework's operators

def _prepare_own(s, c):
    """The plan and buffers that a program keeps between calls."""
    from fine_grained_mixture_top_amd import ops
    op = c["op"]

    def zeros(*shape, dtype):
        return torch.zeros(*shape, dtype=dtype, device="cuda")

    if "K" in c:
        s["plan"] = p = ops.Plan(c["T"], c["K"], c["E"], align=c["align"])
        cap = p.cap
        if not op.startswith("dispatch"):
            ops.moe_sort(p, s["idx"])
    if op == "dispatch":
        s["xp"] = zeros(cap, c["d"], dtype=s["x"].dtype)
    elif op == "dispatch_fp8":
        s["q"], s["s"] = zeros(cap, c["d"], dtype=torch.uint8).view(E4M3), zeros(cap, _blocks(c["d"]), dtype=torch.float32)
    elif op == "combine":
        s["o"] = zeros(c["T"], c["d"], dtype=s["y"].dtype)
    elif op == "combine_bwd":
        s["dy"], s["dw"] = zeros(cap, c["d"], dtype=s["y"].dtype), zeros(c["T"], c["K"], dtype=torch.float32)
    elif op == "product":
        s["c"] = zeros(cap, c["n"], dtype=_DT[c["out"]])
    elif op == "dgrad":
        s["q"], s["s"] = zeros(cap, c["n"], dtype=torch.uint8).view(E4M3), zeros(cap, _blocks(c["n"]), dtype=torch.float32)
        s["c"] = zeros(cap, c["d"], dtype=_DT[c["out"]])
    elif op == "wgrad":
        s["xq"], s["xs"] = ops.column_buffers(p, c["d"])
        s["yq"], s["ys"] = ops.column_buffers(p, c["n"])
        s["c"] = zeros(c["E"], c["d"], c["n"], dtype=_DT[c["out"]])
    elif op == "weights":
        s["q"] = zeros(c["E"], c["d"], c["n"], dtype=torch.uint8).view(E4M3)
        s["qt"] = zeros(c["E"], c["n"], c["d"], dtype=torch.uint8).view(E4M3)
        s["s"] = zeros(c["E"], _blocks(c["d"]), _blocks(c["n"]), dtype=torch.float32)
    elif op == "swiglu":
        s["q"] = zeros(c["R"], c["n"], dtype=torch.uint8).view(E4M3)
        s["s"] = zeros(c["R"], _blocks(c["n"]), dtype=torch.float32)
    else:
        s["dh"] = zeros(c["R"], 2 * c["n"], dtype=s["h"].dtype)


def _own(s):
    from fine_grained_mixture_top_amd import ops
    op, p = s["case"]["op"], s.get("plan")
    if op == "dispatch":
        ops.moe_sort(p, s["idx"])
        ops.moe_permute(p, s["x"], s["xp"])
        return dict(offsets=p.offsets, counts=p.counts, row_token=p.row_token, slot_row=p.slot_row, xp=s["xp"])
    if op == "dispatch_fp8":
        ops.moe_sort(p, s["idx"])
        ops.moe_permute_fp8(p, s["x"], s["q"], s["s"])
        return dict(offsets=p.offsets, counts=p.counts, row_token=p.row_token, slot_row=p.slot_row, q=s["q"], s=s["s"])
    if op == "combine":
        if s["w"] is None:
            ops.moe_permute_bwd(p, s["y"], s["o"])
        else:
            ops.moe_unpermute(p, s["y"], s["w"], s["o"])
        return s["o"]
    if op == "combine_bwd":
        ops.moe_unpermute_bwd(p, s["do"], s["y"], s["w"], s["dy"], s["dw"])
        return dict(dy=s["dy"], dw=s["dw"])
    if op == "product":
        ops.moe_fp8_mm(p, s["a"], s["sa"], s["b"], s["sb"], s["c"], gather=s["case"]["gather"])
        return s["c"]
    if op == "dgrad":
        ops.moe_fp8_quant_rows(s["dy"], s["q"], s["s"], plan=p)
        ops.moe_fp8_mm(p, s["q"], s["s"], s["b"], s["sb"], s["c"], sb_out_major=True)
        return s["c"]
    if op == "wgrad":
        ops.moe_fp8_quant_cols(p, s["x"], s["xq"], s["xs"], gather=True)
        ops.moe_fp8_quant_cols(p, s["dy"], s["yq"], s["ys"])
        ops.moe_fp8_wgrad(p, s["xq"], s["xs"], s["yq"], s["ys"], s["c"])
        return s["c"]
    if op == "weights":
        ops.moe_fp8_quant_weights(s["w"], s["q"], s["qt"], s["s"])
        return s["q"], s["qt"], s["s"]
    if op == "swiglu":
        ops.moe_swiglu_fp8(s["h"], s["q"], s["s"])
        return s["q"], s["s"]
    ops.moe_swiglu_bwd(s["da"], s["h"], s["dh"])
    return s["dh"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    op = c["op"]
    if op in ("swiglu", "swiglu_bwd"):
        e = 2 if c["dtype"] == "bf16" else 4
        R, n = c["R"], c["n"]
        if op == "swiglu":
            return dict(bytes=R * (2 * n * e + n + 4 * _blocks(n)), flops=R * n * 8)
        return dict(bytes=R * n * 5 * e, flops=R * n * 14)
    if op == "weights":
        e = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=c["E"] * (c["d"] * c["n"] * (e + 2) + 4 * _blocks(c["d"]) * _blocks(c["n"])),
                    flops=2 * c["E"] * c["d"] * c["n"])
    T, K, E, d = c["T"], c["K"], c["E"], c["d"]
    rows = T * K * (1.0 - c["drop"])
    plan = 4 * (2 * T * K + rows + 2 * E + 1)
    touched = min(E, E * (1.0 - (1.0 - 1.0 / E) ** rows)) if rows else 0  # experts with rows, at an even spread
    if op in ("dispatch", "dispatch_fp8"):
        e = 2 if c["dtype"] == "bf16" else 4
        out = d * e if op == "dispatch" else d + 4 * _blocks(d)
        return dict(bytes=plan + T * d * e + rows * out, flops=0 if op == "dispatch" else 2 * T * d)
    if op == "combine":
        e = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=4 * T * K * (2 if c["weighted"] else 1) + (rows + T) * d * e, flops=2 * rows * d)
    if op == "combine_bwd":
        e = 2 if c["dtype"] == "bf16" else 4
        return dict(bytes=12 * T * K + (2 * rows + T) * d * e, flops=3 * rows * d)
    n = c["n"]
    o = 2 if c["out"] == "bf16" else 4
    if op == "product":
        src = T if c["gather"] else rows
        return dict(bytes=src * (d + 4 * _blocks(d)) + touched * (d * n + 4 * _blocks(d) * _blocks(n)) + rows * n * o,
                    flops=2 * rows * d * n)
    if op == "dgrad":
        return dict(bytes=rows * n * 2 + touched * (d * n + 4 * _blocks(d) * _blocks(n)) + rows * d * o, flops=2 * rows * d * n)
    return dict(bytes=T * d * 2 + rows * n * 2 + E * d * n * o, flops=2 * rows * d * n)


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3_64(v):
    """The E4M3 value nearest to v (float64), ties to the even one, at most 448."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)


def _block_64(v):
    """One block: (values of its codes, scale); the scale and the scaled values are fp32 numbers by definition."""
    m = v.abs().amax()
    s = torch.clamp((m.float().double() / 448.0).float(), min=TINY)
    return _e4m3_64((v.float() * (1.0 / s)).double()), s.double()


def _rows_64(x):
    """Codes' values and scales of x [R, C], block by block along C."""
    q, s = torch.empty_like(x, dtype=torch.float64), []
    for c0 in range(0, x.shape[1], 128):
        v = x[:, c0:c0 + 128]
        sc = torch.clamp((v.abs().amax(1).float().double() / 448.0).float(), min=TINY)
        q[:, c0:c0 + 128] = _e4m3_64((v.float() * (1.0 / sc)[:, None]).double())
        s.append(sc.double())
    return q, torch.stack(s, 1)


def _value_64(q, s):
    """q [R, C] times its scales [R, C/128]."""
    v = q.double().clone()
    for b in range(s.shape[1]):
        v[:, 128 * b:128 * b + 128] *= s[:, b:b + 1].double()
    return v


def _plan_64(idx, c):
    """Rows by counting, on the host."""
    ids = idx.reshape(-1).tolist()
    E, K, align = c["E"], c["K"], c["align"]
    of = [[] for _ in range(E)]
    for i, e in enumerate(ids):
        if 0 <= e < E:
            of[e].append(i)
    offsets, row_token, slot_row = [0], [0] * _cap(c), [-1] * len(ids)
    for e in range(E):
        at = offsets[-1]
        for j, i in enumerate(of[e]):
            row_token[at + j], slot_row[i] = i // K, at + j
        end = at + -(-len(of[e]) // align) * align
        for j in range(at + len(of[e]), end):
            row_token[j] = -1
        offsets.append(end)
    return offsets, [len(v) for v in of], row_token, slot_row


def exact(case, seed):
    c = case
    op = c["op"]
    s = _inputs(c, seed)
    if op in ("swiglu", "swiglu_bwd"):
        h, n = s["h"].double(), c["n"]
        g, u = h[:, :n], h[:, n:]
        sig = torch.sigmoid(g)
        if op == "swiglu":
            return _rows_64(g * sig * u)
        da = s["da"].double()
        return torch.cat([da * u * (sig + g * sig * (1.0 - sig)), da * (g * sig)], 1)
    if op == "weights":
        if c["E"] * _blocks(c["d"]) * _blocks(c["n"]) > 20000:
            return None
        w = s["w"].double()
        q, sc = torch.empty_like(w), torch.empty(c["E"], _blocks(c["d"]), _blocks(c["n"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            for i in range(sc.shape[1]):
                for j in range(sc.shape[2]):
                    at = (e, slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                    q[at], sc[e, i, j] = _block_64(w[at])
        return q, q.transpose(1, 2).contiguous(), sc
    offsets, counts, row_token, slot_row = _plan_64(s["idx"], c)
    T, K, E, cap = c["T"], c["K"], c["E"], _cap(c)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32)

    slots = torch.tensor(slot_row, device="cuda").view(T, K)
    if op in ("dispatch", "dispatch_fp8"):
        plan = dict(offsets=ints(offsets), counts=ints(counts), row_token=ints(row_token), slot_row=ints(slot_row).view(T, K))
        x = s["x"].double()
        vals = dict(xp=x) if op == "dispatch" else dict(zip(("q", "s"), _rows_64(x)))
        for name, v in vals.items():
            out = torch.zeros(cap, v.shape[1], dtype=torch.float64, device="cuda")
            for k in range(K):
                kept = slots[:, k] >= 0
                out[slots[kept, k]] = v[kept]
            plan[name] = out
        return plan
    if op == "combine":
        o = torch.zeros(T, c["d"], dtype=torch.float64, device="cuda")
        for k in range(K):
            kept = slots[:, k] >= 0
            v = s["y"][slots[kept, k]].double()
            o[kept] += v if s["w"] is None else v * s["w"][kept, k].double()[:, None]
        return o
    if op == "combine_bwd":
        dy = torch.zeros(cap, c["d"], dtype=torch.float64, device="cuda")
        dw = torch.zeros(T, K, dtype=torch.float64, device="cuda")
        for k in range(K):
            kept = slots[:, k] >= 0
            do = s["do"][kept].double()
            dy[slots[kept, k]] = do * s["w"][kept, k].double()[:, None]
            dw[kept, k] = (do * s["y"][slots[kept, k]].double()).sum(1)
        return dict(dy=dy, dw=dw)
    token = torch.tensor(row_token, device="cuda")
    if op == "wgrad":
        out = torch.zeros(E, c["d"], c["n"], dtype=torch.float64, device="cuda")
        for e in range(E):
            r0, m = offsets[e], counts[e]
            for b in range(0, m, 128):
                at = slice(r0 + b, r0 + min(m, b + 128))
                x, sx = _rows_64(s["x"][token[at]].double().t())
                y, sy = _rows_64(s["dy"][at].double().t())
                out[e] += (x * sx) @ (y * sy).t()
        return out
    out = torch.zeros(cap, c["n"] if op == "product" else c["d"], dtype=torch.float64, device="cuda")
    for e in range(E):
        at = slice(offsets[e], offsets[e] + counts[e])
        if not counts[e]:
            continue
        if op == "product":
            take = token[at] if c["gather"] else torch.arange(at.start, at.stop, device="cuda")
            a = _value_64(s["a"][take], s["sa"][take])
            w = _value_64(s["b"][e], torch.repeat_interleave(s["sb"][e].t(), 128, 0)[:c["n"]])
        else:
            a = _value_64(*_rows_64(s["dy"][at].double()))
            w = _value_64(s["b"][e], torch.repeat_interleave(s["sb"][e], 128, 0)[:c["d"]])
        out[at] = a @ w.t()
    return out
