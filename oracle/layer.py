"""fp64 definitions of the state-space-duality layer's operators, in plain torch on the CPU: the
convolution and the SSM over packed sequences, both for one token per request, and the
root-mean-square norm with its 8-bit outputs and its gradient.

Each is the formula, sequence by sequence and token by token; nothing is shared with
the HIP library.  The SSM functions also return the same sums over absolute values,
which is what a rounding of one term is measured against.
"""
from __future__ import annotations

import torch


def _d(t):
    return None if t is None else t.detach().cpu().double()


def _silu(v):
    return v / (1 + torch.exp(-v))


def conv_varlen(x, weight, cu, bias=None, ring=None, slots=None, positions=None, silu=True):
    """(u, ring after) for packed x (total, width); rows of u outside every sequence are NaN."""
    x, w = _d(x), _d(weight)
    K = w.shape[1]
    ring = None if ring is None else _d(ring).clone()
    old = None if ring is None else ring.clone()
    u = torch.full_like(x, float("nan"))
    cu = [int(v) for v in cu]
    for s in range(len(cu) - 1):
        slot = -1 if slots is None else int(slots[s])
        kept = ring is not None and 0 <= slot < ring.shape[0]
        pos = max(int(positions[s]), 0) if kept else 0
        for t in range(cu[s], cu[s + 1]):
            a = torch.zeros(x.shape[1], dtype=torch.float64) if bias is None else _d(bias).clone()
            for k in range(K):
                at = t - (K - 1) + k
                p = pos + at - cu[s]
                if at >= cu[s]:
                    a += w[:, k] * x[at]
                elif p >= 0 and kept:
                    a += w[:, k] * old[slot, p % K]
            u[t] = _silu(a) if silu else a
        n = cu[s + 1] - cu[s]
        if kept:
            for i in range(1, min(n, K - 1) + 1):
                ring[slot, (pos + n - i) % K] = x[cu[s + 1] - i]
    return u, ring


def _decay(dt, A_log, dt_bias, softplus, euler):
    d = _d(dt) + (0 if dt_bias is None else _d(dt_bias))
    if softplus:
        d = d.clamp(min=0) + torch.log1p(torch.exp(-d.abs()))
    A = -torch.exp(_d(A_log))
    return torch.exp(d * A), (d if euler else torch.expm1(d * A) / A)


def ssd_varlen(x, dt, A_log, B, C, cu, D=None, z=None, dt_bias=None, state=None, slots=None, positions=None,
               softplus=True, euler=False):
    """(y, state after, |y| sums, |state| sums): packed x (total, H, P), B and C (total, G, N)."""
    x, B, C = _d(x), _d(B), _d(C)
    total, H, P = x.shape
    G, N = B.shape[1:]
    a, w = _decay(dt, A_log, dt_bias, softplus, euler)
    y, ya = torch.full_like(x, float("nan")), torch.zeros_like(x)
    state = None if state is None else _d(state).clone()
    sa = None if state is None else state.abs()
    cu = [int(v) for v in cu]
    for s in range(len(cu) - 1):
        if cu[s] == cu[s + 1]:
            continue
        slot = -1 if slots is None else int(slots[s])
        kept = state is not None and 0 <= slot < state.shape[0]
        h = torch.zeros(H, P, N, dtype=torch.float64)
        if kept and int(positions[s]) > 0:
            h = state[slot].clone()
        ha = h.abs()
        for t in range(cu[s], cu[s + 1]):
            Bt, Ct = B[t].repeat_interleave(H // G, 0), C[t].repeat_interleave(H // G, 0)
            wx = w[t][:, None] * x[t]
            h = a[t][:, None, None] * h + wx[:, :, None] * Bt[:, None, :]
            ha = a[t][:, None, None] * ha + wx.abs()[:, :, None] * Bt.abs()[:, None, :]
            y[t] = (h * Ct[:, None, :]).sum(2)
            ya[t] = (ha * Ct.abs()[:, None, :]).sum(2)
        if kept:
            state[slot], sa[slot] = h, ha
    if D is not None:
        y = y + _d(D)[:, None] * x
        ya = ya + (_d(D)[:, None] * x).abs()
    if z is not None:
        gate = _silu(_d(z))
        y, ya = y * gate, ya * gate.abs()
    return y, state, ya, sa


def ssd_step(xbc, dt, A_log, conv_weight, conv_state, state, positions, slots=None, D=None, z=None, dt_bias=None,
             conv_bias=None, softplus=True, euler=False):
    """(y, ring after, state after, |y| sums, |state| sums): a token of every row, u not rounded in between.
    Rows without a slot are NaN in y."""
    batch = xbc.shape[0]
    nslots, H, P, N = state.shape
    G = (xbc.shape[1] - H * P) // (2 * N)
    slots = list(range(batch)) if slots is None else [int(v) for v in slots]
    y = torch.full((batch, H, P), float("nan"), dtype=torch.float64)
    ya = torch.zeros_like(y)
    ring, st = _d(conv_state).clone(), _d(state).clone()
    sa = st.abs()
    for i in range(batch):
        if not 0 <= slots[i] < nslots:
            continue
        one = [0, 1]
        u, ring = conv_varlen(xbc[i:i + 1], conv_weight, one, conv_bias, ring, [slots[i]], [positions[i]])
        x = u[:, :H * P].view(1, H, P)
        B, C = u[:, H * P:H * P + G * N].view(1, G, N), u[:, H * P + G * N:].view(1, G, N)
        yi, after, yai, sai = ssd_varlen(x, dt[i:i + 1], A_log, B, C, one, D, None if z is None else z[i:i + 1], dt_bias, st,
                                         [slots[i]], [positions[i]], softplus, euler)
        y[i], ya[i], st = yi[0], yai[0], after
        sa[slots[i]] = sai[slots[i]]
    return y, ring, st, ya, sa


def rms_norm(x, weight, residual=None, eps=1e-5):
    """(y, r, rstd)"""
    r = _d(x) + (0 if residual is None else _d(residual))
    rstd = 1 / torch.sqrt((r * r).mean(-1) + eps)
    return r * rstd[..., None] * _d(weight), r, rstd


def e4m3(v):
    """v rounded to the nearest e4m3 value (ties to even), as fp64; |v| <= 448."""
    unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / unit) * unit


def row_scale(y):
    top = y.abs().amax(-1)
    return torch.where(top == 0, torch.ones_like(top), top / 448)


def block_scale(y):
    """The smallest power of two that keeps 32 columns' magnitudes within 448 (1 where they are 0)."""
    out = []
    for part in y.split(32, -1):
        top = part.abs().amax(-1)
        out.append(torch.where(top == 0, torch.ones_like(top), torch.exp2(torch.ceil(torch.log2(top / 448)).clamp(-127, 127))))
    return torch.stack(out, -1)


def rms_norm_bwd(dy, r, weight, rstd, d_residual=None):
    """(dr, dweight, |dr| sums, |dweight| sums)"""
    dy, r, w, rstd = _d(dy), _d(r), _d(weight), _d(rstd)[..., None]
    xh, g = r * rstd, dy * w
    dr = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
    dra = rstd * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    if d_residual is not None:
        dr, dra = dr + _d(d_residual), dra + _d(d_residual).abs()
    n = r.shape[-1]
    dw, dwa = (dy * xh).reshape(-1, n).sum(0), (dy * xh).abs().reshape(-1, n).sum(0)
    return dr, dw, dra, dwa
