"""Operators of the state-space-duality layer: what is measured, on which sizes.

A layer is  norm -> in-projection -> short convolution + SSM -> norm -> out-projection.  The operators are the
root-mean-square norm with the residual's addition (and an 8-bit output with scales), its gradient, the short
convolution over packed prompts, the multi-head SSM over packed prompts, and both for one token per request, with
the requests' states in pools indexed by slot.

`run` computes an operator in plain torch operations, or (own = True) through selective_state_space_55_amd.
"""
import math
import random

import torch

own = False
EPS = 1e-5
IO = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = torch.float32


# ---------------------------------------------------------------- cases


def listed():
    return [
        # a decode batch between two layers: norm of the 1.4B width feeding a block-scaled 8-bit in-projection
        dict(name="norm-decode-mx8", op="norm_fwd", rows=16, dim=2048, io="bf16", res="f32", quant="mx"),
        # a prefill batch: 2.8B width, residual kept in bf16, row-scaled 8-bit output
        dict(name="norm-prefill-row8", op="norm_fwd", rows=32768, dim=2560, io="bf16", res="bf16", quant="row"),
        # training the 130M width in fp32, a short batch
        dict(name="norm-train-130m", op="norm_bwd", rows=2048, dim=768, io="f32", res="f32"),
        # training the 1.4B width: bf16 activations, fp32 residual stream
        dict(name="norm-train-1.4b", op="norm_bwd", rows=32768, dim=2048, io="bf16", res="f32"),
        # a few short prompts of a small model
        dict(name="conv-ragged", op="conv", total=333, nseq=5, heads=24, headdim=64, dstate=128, groups=1, K=4, io="bf16"),
        # the 28-sequence packed prefill of the 1.4B layer (inner width 4096)
        dict(name="conv-prefill", op="conv", total=32768, nseq=28, heads=64, headdim=64, dstate=128, groups=1, K=4, io="bf16"),
        # one prompt of a small model
        dict(name="prompt-one", op="ssd", total=509, nseq=1, heads=24, headdim=64, dstate=128, groups=1, gated=True, euler=False),
        # the 28-sequence packed prefill of the 1.4B layer
        dict(name="prompt-mix", op="ssd", total=32768, nseq=28, heads=64, headdim=64, dstate=128, groups=1, gated=True, euler=False),
        # one long document, wider heads, two groups of B and C
        dict(name="prompt-long", op="ssd", total=20000, nseq=1, heads=32, headdim=128, dstate=64, groups=2, gated=True, euler=True),
        # one user's next token, 2.8B layer (inner width 5120)
        dict(name="step-one", op="step", batch=1, pad=0, heads=80, headdim=64, dstate=128, groups=1, K=4, io="bf16", euler=False),
        # a small fp32 model's padded batch
        dict(name="step-padded", op="step", batch=37, pad=11, heads=24, headdim=96, dstate=64, groups=2, K=4, io="f32", euler=True),
        # a full decode batch of the 2.8B layer
        dict(name="step-batch", op="step", batch=256, pad=0, heads=80, headdim=64, dstate=128, groups=1, K=4, io="bf16", euler=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "conv", "ssd", "step"])
    if op in ("norm_fwd", "norm_bwd"):
        c = dict(op=op, rows=_log(rng, 1, 16384), dim=_log(rng, 65, 5120), io=rng.choice(["bf16", "bf16", "f32"]))
        if rng.random() < 0.5:
            c["dim"] = max(8, c["dim"] // 8 * 8)
        c["res"] = rng.choice(["f32", c["io"], "none"])
        if op == "norm_fwd":
            c["quant"] = rng.choice(["none", "row", "mx"])
        return c
    c = dict(op=op, heads=_log(rng, 2, 64), headdim=rng.choice([32, 64, 64, 96, 128]), dstate=rng.choice([64, 128]))
    c["groups"] = rng.choice([g for g in (1, 1, 2, 4) if c["heads"] % g == 0])
    while c["heads"] * c["headdim"] > 5120:
        c["heads"] -= c["groups"]
    if op == "conv":
        total = _log(rng, 1, 16384)
        return c | dict(total=total, nseq=rng.randint(1, min(total, 40)), K=rng.choice([2, 3, 4, 4]), io=rng.choice(["bf16", "f32"]))
    if op == "ssd":
        total = _log(rng, 1, 16384)
        return c | dict(total=total, nseq=rng.randint(1, min(total, 40)), gated=rng.random() < 0.7, euler=rng.random() < 0.5)
    batch = _log(rng, 1, 256)
    return c | dict(batch=batch, pad=rng.randint(0, batch // 4), K=rng.choice([2, 3, 4, 4]), io=rng.choice(["bf16", "bf16", "f32"]),
                    euler=rng.random() < 0.5)


def _lengths(case):
    """Sequence lengths of a packed case: spread over a factor of 30, at least one token each."""
    r, n = random.Random(case["total"] * 1009 + case["nseq"]), case["nseq"]
    weight = [math.exp(r.uniform(0, math.log(30))) for _ in range(n)]
    lens = [1 + int((case["total"] - n) * w / sum(weight)) for w in weight]
    lens[0] += case["total"] - sum(lens)
    return lens


def _positions(case, n):
    """Tokens that a request has behind it: a third are new, the others continue."""
    r = random.Random(n * 31 + case["heads"])
    return [0 if i % 3 == 1 else r.choice([1, 2, 5, r.randint(3, 9000)]) for i in range(n)]


def _widths(case):
    inner = case["heads"] * case["headdim"]
    return inner, inner + 2 * case["groups"] * case["dstate"]


def work(case):
    op, e = case["op"], {"bf16": 2, "f32": 4, "none": 0}
    if op == "norm_fwd":
        n, io, res = case["rows"] * case["dim"], e[case["io"]], e[case["res"]]
        out = 1 if case["quant"] != "none" else io
        scales = {"none": 0, "row": 4 * case["rows"], "mx": case["rows"] * -(-case["dim"] // 32)}[case["quant"]]
        return {"bytes": n * (io + 2 * res + out) + 4 * case["dim"] + scales + 4 * case["rows"], "flops": 6 * n}
    if op == "norm_bwd":
        n, io, res = case["rows"] * case["dim"], e[case["io"]], e[case["res"]]
        apart = case["res"] not in ("none", case["io"])  # the residual's gradient has a type of its own
        return {"bytes": n * (2 * io + (2 * res if res else io) + (res if apart else 0)) + 8 * case["dim"] + 4 * case["rows"], "flops": 12 * n}
    inner, width = _widths(case)
    state = inner * case["dstate"] * 4
    if op == "conv":
        io, k = e[case["io"]], case["K"]
        return {"bytes": case["total"] * width * 2 * io + case["nseq"] * 2 * (k - 1) * width * io + 4 * width * (k + 1),
                "flops": case["total"] * width * (2 * k + 6)}
    if op == "ssd":
        a_token = 2 * (inner * (3 if case["gated"] else 2) + 2 * case["groups"] * case["dstate"] + case["heads"])
        started = sum(p > 0 for p in _positions(case, case["nseq"]))
        return {"bytes": case["total"] * a_token + (case["nseq"] + started) * state, "flops": case["total"] * inner * case["dstate"] * 4}
    rows, io = case["batch"] - case["pad"], e[case["io"]]
    a_row = 2 * state + io * (2 * inner + case["heads"] + width * (case["K"] + 1))
    return {"bytes": rows * a_row + 4 * width * (case["K"] + 1), "flops": rows * inner * case["dstate"] * 5}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, dtype=F32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int64, device="cuda")

    op = case["op"]
    s = {"case": case}
    if op in ("norm_fwd", "norm_bwd"):
        rows, dim, io = case["rows"], case["dim"], IO[case["io"]]
        res = IO.get(case["res"])
        s["weight"] = 1 + normal(dim, scale=0.1)
        if op == "norm_fwd":
            s["x"] = normal(rows, dim, dtype=io)
            s["residual"] = normal(rows, dim, dtype=res, scale=3.0) if res else None
        else:
            s["r"] = normal(rows, dim, dtype=res or io, scale=3.0)
            s["rstd"] = torch.rsqrt(s["r"].double().square().mean(1) + EPS).float()
            s["dy"] = normal(rows, dim, dtype=io)
            s["dres"] = normal(rows, dim, dtype=res) if res else None
        return s
    H, P, N, G = case["heads"], case["headdim"], case["dstate"], case["groups"]
    inner, width = _widths(case)
    s["A_log"] = torch.log(1 + 15 * torch.rand(H, generator=g, device="cuda"))
    s["D"] = normal(H)
    s["dt_bias"] = torch.log(torch.expm1(0.001 + 0.099 * torch.rand(H, generator=g, device="cuda")))
    n = case["batch"] if op == "step" else case["nseq"]
    slots = torch.randperm(n + 3, generator=g, device="cuda")[:n]
    s["positions"] = ints(_positions(case, n))
    if op in ("conv", "step"):
        s["conv_weight"], s["conv_bias"] = normal(width, case["K"], scale=0.5), normal(width, scale=0.1)
        s["conv_state"] = normal(n + 3, case["K"], width, dtype=IO[case["io"]])
    if op in ("ssd", "step"):
        s["state"] = normal(n + 3, H, P, N, scale=0.1)
    if op == "step":
        if case["pad"]:  # a captured batch that is not full: its last rows hold no request
            slots[n - case["pad"]:] = -1
        proj = normal(n, inner + width + H, dtype=IO[case["io"]])  # z | x B C | dt, as one in-projection gives them
        s["z"], s["xbc"], s["dt"] = proj[:, :inner].unflatten(1, (H, P)), proj[:, inner:inner + width], proj[:, inner + width:]
        s["y"] = torch.zeros(n, H, P, dtype=IO[case["io"]], device="cuda")
    else:
        total, lens = case["total"], _lengths(case)
        cu = [0]
        for length in lens:
            cu.append(cu[-1] + length)
        s["cu"], s["longest"] = ints(cu), max(lens)
        if op == "conv":
            s["xbc"] = normal(total, width, dtype=IO[case["io"]])
        else:
            u = normal(total, width)
            u = (u * torch.sigmoid(u)).bfloat16()  # x | B | C as the convolution leaves them
            s["x"] = u[:, :inner].unflatten(1, (H, P))
            s["B"] = u[:, inner:inner + G * N].unflatten(1, (G, N))
            s["C"] = u[:, inner + G * N:].unflatten(1, (G, N))
            s["dt"] = normal(total, H, dtype=torch.bfloat16)
            s["z"] = normal(total, H, P, dtype=torch.bfloat16) if case["gated"] else None
    s["slots"] = slots
    return s


# ---------------------------------------------------------------- the operators


def run(s):
    if own:
        return _own(s)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "conv": _conv, "ssd": _ssd, "step": _step}[s["case"]["op"]](s)


def _own(s):
    import selective_state_space_55_amd as m

    c, op = s["case"], s["case"]["op"]
    rule = "euler" if c.get("euler") else "zoh"
    if op == "norm_fwd":
        quant = None if c["quant"] == "none" else c["quant"]
        return m.rms_norm_fwd(s["x"], s["weight"], s["residual"], eps=EPS, quant=quant, return_rstd=True)
    if op == "norm_bwd":
        return m.rms_norm_bwd(s["dy"], s["r"], s["weight"], s["rstd"], s["dres"])
    if op == "conv":
        u = m.ssd_conv_fwd_varlen(s["xbc"], s["conv_weight"], s["cu"], bias=s["conv_bias"], conv_state=s["conv_state"],
                                  slots=s["slots"], positions=s["positions"])
        return u, s["conv_state"]
    if op == "ssd":
        y = m.ssd_fwd_varlen(s["x"], s["dt"], s["A_log"], s["B"], s["C"], s["cu"], D=s["D"], z=s["z"], dt_bias=s["dt_bias"],
                             state=s["state"], slots=s["slots"], positions=s["positions"], discretization=rule)
        return y, s["state"]
    y = m.ssd_step(s["xbc"], s["dt"], s["A_log"], s["conv_weight"], s["conv_state"], s["state"], s["positions"], slots=s["slots"],
                   D=s["D"], z=s["z"], dt_bias=s["dt_bias"], conv_bias=s["conv_bias"], out=s["y"], discretization=rule)
    return y, s["conv_state"], s["state"]


def _silu(v):
    return v * torch.sigmoid(v)


def _quantise(y, quant):
    """e4m3 values and their scales: one fp32 per row (largest magnitude / 448), or one power of two per 32 columns, the
    smallest that keeps the block's magnitudes within 448; 1 where all are zero."""
    if quant == "row":
        top = y.abs().amax(1)
        scale = torch.where(top > 0, top / 448, torch.ones_like(top))
        return (y / scale[:, None]).to(torch.float8_e4m3fn), scale
    rows, dim = y.shape
    blocks = torch.nn.functional.pad(y, (0, -dim % 32)).view(rows, -1, 32)
    top = blocks.abs().amax(2)
    m, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    k = torch.where(top > 0, (e - 9 + (m > 0.875)).clamp(-127, 127), torch.zeros_like(e))
    scale = torch.ldexp(torch.ones_like(top), k)
    q = (blocks / scale[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(rows, -1)[:, :dim], scale.to(torch.float8_e8m0fnu)


def _norm_fwd(s):
    c, x = s["case"], s["x"].float()
    r = x if s["residual"] is None else x + s["residual"].float()
    rstd = torch.rsqrt(r.square().mean(1) + EPS)
    y = r * rstd[:, None] * s["weight"]
    out = (y.to(s["x"].dtype),) if c["quant"] == "none" else _quantise(y, c["quant"])
    if s["residual"] is not None:
        out += (r.to(s["residual"].dtype),)
    return out + (rstd,)


def _norm_bwd(s):
    dy, r, rstd = s["dy"].float(), s["r"].float(), s["rstd"][:, None]
    xh, g = r * rstd, dy * s["weight"]
    dr = rstd * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["dres"] is not None:
        dr = dr + s["dres"].float()
    out = {"dx": dr.to(s["dy"].dtype), "dweight": (dy * xh).double().sum(0).float()}
    if s["dres"] is not None:
        out["dresidual"] = dr.to(s["dres"].dtype)
    return out


def _conv(s):
    x, cu, pos, slots, ring = s["xbc"], s["cu"], s["positions"], s["slots"], s["conv_state"]
    total, K = x.shape[0], s["case"]["K"]
    t = torch.arange(total, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    back = torch.arange(K - 1, -1, -1, device="cuda")  # how far behind the token each tap looks
    local = (t - cu[seq])[:, None] - back
    at = pos[seq][:, None] + local
    here = x[(t[:, None] - back).clamp(min=0)].float()
    kept = ring[slots[seq][:, None], at.remainder(K)].float()
    v = torch.where((local >= 0)[:, :, None], here, torch.where((at >= 0)[:, :, None], kept, torch.zeros_like(kept)))
    u = _silu((v * s["conv_weight"].t()).sum(1) + s["conv_bias"]).to(x.dtype)
    lens = cu[1:] - cu[:-1]
    last = torch.arange(1, K, device="cuda")
    some = last <= lens[:, None]
    row = (pos + lens)[:, None] - last
    ring[slots[:, None].expand_as(some)[some], row.remainder(K)[some]] = x[(cu[1:, None] - last)[some]]
    return u, ring


def _ssd(s):
    Q = 64
    cu, slots, pos, euler = s["cu"], s["slots"], s["positions"], s["case"]["euler"]
    total, H, P = s["x"].shape
    G, N = s["B"].shape[1:]
    S, L = slots.numel(), -(-s["longest"] // Q) * Q
    C = L // Q
    lens = cu[1:] - cu[:-1]
    place = torch.arange(L, device="cuda")
    valid = place < lens[:, None]
    token = (cu[:-1, None] + place).clamp(max=total - 1)

    def chunks(v):  # (total, a, b) -> (S, C, a, Q, b)
        return v[token].float().unflatten(1, (C, Q)).transpose(2, 3)

    x, B, Cm = chunks(s["x"]), chunks(s["B"]), chunks(s["C"])
    A = -torch.exp(s["A_log"])
    step = torch.nn.functional.softplus(s["dt"][token].float() + s["dt_bias"]) * valid[:, :, None]
    weight = step if euler else torch.expm1(step * A) / A
    weight = weight.unflatten(1, (C, Q)).transpose(2, 3)  # (S, C, H, Q)
    cum = (step * A).double().unflatten(1, (C, Q)).transpose(2, 3).cumsum(3)
    gap = cum[..., :, None] - cum[..., None, :]
    causal = torch.ones(Q, Q, dtype=torch.bool, device="cuda").tril()
    M = torch.exp(torch.where(causal, gap, -torch.inf).float()) * weight[..., None, :]
    M = M.unflatten(2, (G, H // G)) * (Cm @ B.transpose(3, 4))[:, :, :, None]
    y = M.flatten(2, 3) @ x
    # each chunk's own state, then the state that enters each chunk: sums over the chunks before it
    scaled = x * (torch.exp(cum[..., -1:] - cum).float() * weight)[..., None]
    Bh, Ch = B.repeat_interleave(H // G, 2), Cm.repeat_interleave(H // G, 2)
    own_state = (scaled.transpose(3, 4) @ Bh).permute(0, 2, 1, 3, 4).flatten(3)  # (S, H, C, P N)
    until = cum[..., -1].permute(0, 2, 1).cumsum(2)  # (S, H, C)
    entry = torch.nn.functional.pad(until, (1, 0))  # before chunk c, and at the end
    gap = entry[..., :, None] - until[..., None, :]
    before = torch.ones(C + 1, C, dtype=torch.bool, device="cuda").tril(-1)
    started = torch.where((pos > 0)[:, None, None, None], s["state"][slots], torch.zeros((), device="cuda"))
    states = torch.exp(torch.where(before, gap, -torch.inf)).float() @ own_state
    states = states + torch.exp(entry).float()[..., None] * started.flatten(2)[:, :, None]
    h_in = states[:, :, :C].unflatten(3, (P, N)).permute(0, 2, 1, 4, 3)  # (S, C, H, N, P)
    y = y + torch.exp(cum).float()[..., None] * (Ch @ h_in)
    y = y + s["D"][:, None, None] * x
    y = y.transpose(2, 3).flatten(1, 2)[valid]
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][slots] = states[:, :, C].unflatten(2, (P, N))
    return y.bfloat16(), s["state"]


def _step(s):
    c, K = s["case"], s["case"]["K"]
    H, P, N, G = c["heads"], c["headdim"], c["dstate"], c["groups"]
    keep = c["batch"] - c["pad"]  # the rows that hold a request
    slots, pos, x = s["slots"][:keep], s["positions"][:keep], s["xbc"][:keep]
    back = torch.arange(K - 1, 0, -1, device="cuda")
    at = pos[:, None] - back
    kept = torch.where((at >= 0)[:, :, None], s["conv_state"][slots[:, None], at.remainder(K)].float(), torch.zeros((), device="cuda"))
    v = torch.cat([kept, x[:, None].float()], 1)
    u = _silu((v * s["conv_weight"].t()).sum(1) + s["conv_bias"])
    s["conv_state"][slots, pos.remainder(K)] = x
    xs = u[:, :H * P].unflatten(1, (H, P))
    B = u[:, H * P:H * P + G * N].unflatten(1, (G, N)).repeat_interleave(H // G, 1)
    C = u[:, H * P + G * N:].unflatten(1, (G, N)).repeat_interleave(H // G, 1)
    A = -torch.exp(s["A_log"])
    step = torch.nn.functional.softplus(s["dt"][:keep].float() + s["dt_bias"])
    weight = step if c["euler"] else torch.expm1(step * A) / A
    h = torch.where((pos > 0)[:, None, None, None], s["state"][slots], torch.zeros((), device="cuda"))
    h = torch.exp(step * A)[:, :, None, None] * h + (weight[:, :, None] * xs)[..., None] * B[:, :, None]
    s["state"][slots] = h
    y = (h * C[:, :, None]).sum(3) + s["D"][:, None] * xs
    s["y"][:keep] = (y * _silu(s["z"][:keep].float())).to(s["y"].dtype)
    return s["y"], s["conv_state"], s["state"]


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd, "conv": _exact_conv, "ssd": _exact_ssd, "step": _exact_step}[case["op"]](s)


def _exact_norm_fwd(s):
    r = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
    rstd = 1 / torch.sqrt((r * r).sum(1) / r.shape[1] + EPS)
    y = r * rstd.unsqueeze(1) * s["weight"].double()
    quant = s["case"]["quant"]
    out = []
    if quant == "none":
        out.append(y)
    else:
        block = y.shape[1] if quant == "row" else 32
        qs, scales = [], []
        for part in y.split(block, 1):
            top = part.abs().amax(1, keepdim=True)
            scale = top / 448 if quant == "row" else torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-127, 127))
            scale = torch.where(top == 0, torch.ones_like(scale), scale)
            v = part / scale
            # e4m3: 3 bits behind the first, steps of 2^-9 below 2^-6
            unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            qs.append(torch.round(v / unit) * unit)
            scales.append(scale)
        out += [torch.cat(qs, 1), torch.cat(scales, 1) if quant == "mx" else scales[0].squeeze(1)]
    if s["residual"] is not None:
        out.append(r)
    return out + [rstd]


def _exact_norm_bwd(s):
    """By differentiating y = r w / sqrt(...) with the given 1 / sqrt(...): d rstd / d r = -rstd^3 r / dim."""
    dy, r, w, rstd = s["dy"].double(), s["r"].double(), s["weight"].double(), s["rstd"].double().unsqueeze(1)
    d_rstd = (dy * w * r).sum(1, keepdim=True)
    dr = dy * w * rstd - d_rstd * rstd ** 3 * r / r.shape[1]
    out = {"dweight": torch.mv((r * dy).t(), rstd.squeeze(1))}
    if s["dres"] is not None:
        dr += s["dres"].double()
        out["dresidual"] = dr
    return out | {"dx": dr}


def _exact_conv(s):
    x, w, K = s["xbc"].double(), s["conv_weight"].double(), s["case"]["K"]
    ring, us = s["conv_state"].double(), []
    cu, slots, pos = s["cu"].tolist(), s["slots"].tolist(), s["positions"].tolist()
    for i, slot in enumerate(slots):
        past = [ring[slot, q % K] if q >= 0 else torch.zeros_like(x[0]) for q in range(pos[i] - K + 1, pos[i])]
        v = torch.cat([torch.stack(past), x[cu[i]:cu[i + 1]]])
        n = cu[i + 1] - cu[i]
        a = s["conv_bias"].double() + sum(w[:, k] * v[k:k + n] for k in range(K))
        us.append(a / (1 + torch.exp(-a)))
        for j in range(1, min(n, K - 1) + 1):
            ring[slot, (pos[i] + n - j) % K] = x[cu[i + 1] - j]
    return torch.cat(us), ring


def _exact_ssd(s):
    """The recurrence itself, a token of every sequence at a time."""
    cu, lens = s["cu"][:-1], s["cu"][1:] - s["cu"][:-1]
    H, G = s["x"].shape[1], s["B"].shape[1]
    A = -torch.exp(s["A_log"].double())
    step = s["dt"].double() + s["dt_bias"].double()
    step = torch.clamp(step, min=0) + torch.log1p(torch.exp(-step.abs()))
    a = torch.exp(step * A)
    w = step if s["case"]["euler"] else torch.expm1(step * A) / A
    h = s["state"].double()[s["slots"]] * (s["positions"] > 0).double()[:, None, None, None]
    y = torch.zeros_like(s["x"], dtype=torch.float64)
    order = torch.argsort(lens, descending=True)  # the sequences still running are the first ones
    lens, cu, h = lens[order], cu[order], h[order]
    left = lens.tolist()
    for t in range(left[0]):
        n = sum(v > t for v in left)
        at = cu[:n] + t
        xt = s["x"][at].double()
        Bt, Ct = (v[at].double().repeat_interleave(H // G, 1) for v in (s["B"], s["C"]))
        h[:n].mul_(a[at][:, :, None, None]).add_((w[at][:, :, None] * xt)[..., None] * Bt[:, :, None])
        y[at] = torch.matmul(h[:n], Ct[..., None]).squeeze(3) + s["D"].double()[:, None] * xt
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z / (1 + torch.exp(-z))
    state = s["state"].double()
    state[s["slots"][order]] = h
    return y, state


def _exact_step(s):
    c, K = s["case"], s["case"]["K"]
    H, P, N, G = c["heads"], c["headdim"], c["dstate"], c["groups"]
    ring, state, y = s["conv_state"].double(), s["state"].double(), s["y"].double()
    A, slots, pos = -torch.exp(s["A_log"].double()), s["slots"].tolist(), s["positions"].tolist()
    w, bias = s["conv_weight"].double(), s["conv_bias"].double()
    for i, slot in enumerate(slots):
        if slot < 0:
            continue
        p, new = pos[i], s["xbc"][i].double()
        a = bias + w[:, K - 1] * new
        for back in range(1, K):
            if p >= back:
                a = a + w[:, K - 1 - back] * ring[slot, (p - back) % K]
        ring[slot, p % K] = new
        u = a / (1 + torch.exp(-a))
        x, B, C = u[:H * P].view(H, P), u[H * P:H * P + G * N].view(G, N), u[H * P + G * N:].view(G, N)
        d = s["dt"][i].double() + s["dt_bias"].double()
        d = torch.clamp(d, min=0) + torch.log1p(torch.exp(-d.abs()))
        wt = d if c["euler"] else torch.expm1(d * A) / A
        h = torch.exp(d * A).view(G, -1, 1, 1) * (state[slot] if p > 0 else 0 * state[slot]).view(G, H // G, P, N)
        h = h + (wt[:, None] * x).view(G, -1, P, 1) * B.view(G, 1, 1, N)
        state[slot] = h.view(H, P, N)
        o = (h @ C.view(G, 1, N, 1)).view(H, P) + s["D"].double()[:, None] * x
        z = s["z"][i].double()
        y[i] = o * z / (1 + torch.exp(-z))
    return y, ring, state
