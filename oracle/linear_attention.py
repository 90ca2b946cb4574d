"""fp64 definitions of linear attention with a fixed decay per head, of its gradient and of the group norm that follows
it, in plain torch on the CPU.

Each is the formula, sequence by sequence and token by token; nothing is shared with the HIP library.  The `_sums`
forms are the same sums over absolute values, which is what a rounding of one term is measured against.
"""
from __future__ import annotations

import torch


def _d(t):
    return None if t is None else t.detach().cpu().double()


def sequence(q, k, v, log_decay, state, scale):
    """(o, S after): one sequence, q and k (L, H, K), v (L, H, V), state (H, V, K)."""
    lam, o = torch.exp(log_decay)[:, None, None], []
    for t in range(q.shape[0]):
        state = lam * state + v[t][:, :, None] * k[t][:, None, :]
        o.append(scale * (state * q[t][:, None, :]).sum(2))
    return (torch.stack(o) if o else v), state


def sequence_grad(do, q, k, v, log_decay, state, d_state, scale):
    """(dq, dk, dv, d state): the gradient of sequence, by its recurrence from the last token to the first."""
    lam = torch.exp(log_decay)[:, None, None]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(q.shape[0]):
        state = lam * state + v[t][:, :, None] * k[t][:, None, :]
        dq[t] = scale * (state * do[t][:, :, None]).sum(1)
    r = d_state
    for t in reversed(range(q.shape[0])):
        r = r + scale * do[t][:, :, None] * q[t][:, None, :]
        dk[t] = (r * v[t][:, :, None]).sum(1)
        dv[t] = (r * k[t][:, None, :]).sum(2)
        r = lam * r
    return dq, dk, dv, r


def forward(q, k, v, log_decay, cu, state=None, slots=None, positions=None, scale=1.0, sums=False):
    """(o, state after): packed q, k (total, H, K), v (total, H, V); rows of o outside every sequence are NaN.  state (entries,
    H, V, K): the entries of the sequences, or with slots a pool."""
    q, k, v, ld = _d(q), _d(k), _d(v), _d(log_decay)
    if sums:
        q, k, v, scale = q.abs(), k.abs(), v.abs(), abs(scale)
    n = len(cu) - 1
    H, K, V = q.shape[1], q.shape[2], v.shape[2]
    after = torch.zeros(n, H, V, K, dtype=torch.float64) if state is None else _d(state).clone()
    if sums:
        after = after.abs()
    before = after.clone()
    o = torch.full_like(v, float("nan"))
    for s in range(n):
        a, b = int(cu[s]), int(cu[s + 1])
        entry = s if slots is None else int(slots[s])
        kept = 0 <= entry < after.shape[0]
        if slots is not None and a == b:
            continue
        h = torch.zeros(H, V, K, dtype=torch.float64)
        if kept and (positions is None or int(positions[s]) > 0):
            h = before[entry]
        o[a:b], h = sequence(q[a:b], k[a:b], v[a:b], ld, h, scale)
        if kept:
            after[entry] = h
    return o, after


def backward(do, q, k, v, log_decay, cu, state=None, d_state=None, scale=1.0, sums=False):
    """(dq, dk, dv, d state): packed, state and d_state (nseq, H, V, K)."""
    do, q, k, v, ld, state, d_state = _d(do), _d(q), _d(k), _d(v), _d(log_decay), _d(state), _d(d_state)
    n = len(cu) - 1
    zeros = torch.zeros(n, q.shape[1], v.shape[2], q.shape[2], dtype=torch.float64)
    state, d_state = zeros if state is None else state, zeros if d_state is None else d_state
    if sums:
        do, q, k, v, state, d_state, scale = do.abs(), q.abs(), k.abs(), v.abs(), state.abs(), d_state.abs(), abs(scale)
    dq, dk, dv = (torch.full_like(t, float("nan")) for t in (q, k, v))
    dh = zeros.clone()
    for s in range(n):
        i = slice(int(cu[s]), int(cu[s + 1]))
        dq[i], dk[i], dv[i], dh[s] = sequence_grad(do[i], q[i], k[i], v[i], ld, state[s], d_state[s], scale)
    return dq, dk, dv, dh


def step(q, k, v, log_decay, state, positions, slots=None, scale=1.0, sums=False):
    """(o, state after): a token of every row; rows without a slot are NaN in o."""
    n = q.shape[0]
    slots = list(range(n)) if slots is None else [int(x) for x in slots]
    o, after = forward(q, k, v, log_decay, list(range(n + 1)), state, slots, positions, scale, sums)
    o[[not 0 <= s < state.shape[0] for s in slots]] = float("nan")
    return o, after


def _silu(v):
    return v / (1 + torch.exp(-v))


def group_norm(x, groups, weight=None, bias=None, z=None, eps=1e-5, center=True, silu=False):
    """y, in 64 bits (of tensors that are; autograd runs through it)."""
    g = x.reshape(x.numel() // x.shape[-1], groups, x.shape[-1] // groups)
    mean = g.mean(2, keepdim=True) if center else torch.zeros_like(g[:, :, :1])
    d = g - mean
    n = (d / torch.sqrt((d * d).mean(2, keepdim=True) + eps)).reshape(x.shape)
    n = n if weight is None else n * weight
    n = n if bias is None else n + bias
    return n * _silu(z) if z is not None else _silu(n) if silu else n


def group_norm_grad(dy, x, groups, weight=None, bias=None, z=None, eps=1e-5, center=True, silu=False):
    """A dict of dx, dz, dweight, dbias, as there are, each with the sums over absolute values that its terms add up to, by the
    formulas."""
    dy, x, w, b, z = _d(dy), _d(x), _d(weight), _d(bias), _d(z)
    dim, width = x.shape[-1], x.shape[-1] // groups
    rows = x.numel() // dim
    g = x.reshape(rows, groups, width)
    d = g - g.mean(2, keepdim=True) if center else g
    rstd = 1 / torch.sqrt((d * d).mean(2, keepdim=True) + eps)
    xh = (d * rstd).reshape(rows, dim)
    n = (xh if w is None else xh * w) + (0 if b is None else b)
    dy = dy.reshape(rows, dim)
    out, dn = {}, dy
    if z is not None:
        z = z.reshape(rows, dim)
        s = 1 / (1 + torch.exp(-z))
        out["dz"] = dy * n * s * (1 + z * (1 - s))
        # (xh is off by what its mean is: roundings of 1, not of xh)
        size = (xh.abs() + 1) * (1 if w is None else w.abs()) + (0 if b is None else b.abs())
        out["dz_sums"] = dy.abs() * size * s * (1 + z.abs() * (1 - s))
        dn = dy * z * s
    elif silu:
        s = 1 / (1 + torch.exp(-n))
        dn = dy * s * (1 + n * (1 - s))
    # what dn's own rounding is measured against: its derivative by n is bounded by 1/2, n is off by its terms
    slack = dy.abs() * (1 + n.abs()) if silu else dn.abs()
    out["dweight"], out["dweight_sums"] = (dn * xh).sum(0), (slack * (xh.abs() + 1)).sum(0)
    out["dbias"], out["dbias_sums"] = dn.sum(0), slack.sum(0)
    wt = torch.ones(dim, dtype=torch.float64) if w is None else w
    h = (dn * wt).reshape(rows, groups, width)
    ha = (slack * wt.abs()).reshape(rows, groups, width)
    x3 = xh.reshape(rows, groups, width)
    dx = h - x3 * (h * x3).mean(2, keepdim=True) - (h.mean(2, keepdim=True) if center else 0)
    dxa = ha + (x3.abs() + 1) * (ha * (x3.abs() + 1)).mean(2, keepdim=True) + (ha.mean(2, keepdim=True) if center else 0)
    out["dx"], out["dx_sums"] = (dx * rstd).reshape(x.shape), (dxa * rstd).reshape(x.shape)
    for name in ("dz", "dz_sums"):
        if name in out:
            out[name] = out[name].reshape(x.shape)
    return out
