"""Linear attention with a fixed decay and the group norm on the CPU: the 64-bit definitions against autograd and against
differences, and what the C ABI and the binding refuse (the pointers are fake; every call fails before a launch)."""
import ctypes
import itertools

import pytest
import torch

import selective_state_space_55_amd as mscan
from oracle import linear_attention as la

OK, ENULL, ESHAPE, EDTYPE, EALIGN, EUNSUP, EWS, EHIP = range(8)
P = 0x10000
BAD = ctypes.c_size_t(-1).value


@pytest.fixture(scope="module")
def lib():
    return mscan.load_library()


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


# ---------------------------------------------------------------- the definitions


@pytest.mark.parametrize("carried", [False, True])
def test_gradient_against_autograd_and_differences(carried):
    H, K, V, cu = 2, 3, 4, [0, 5, 5, 6, 13]
    T, n, c = cu[-1], 4, 0.7
    ld = torch.tensor([-0.1, -0.9], dtype=torch.float64)
    q, k, v, do = rand(T, H, K, seed=1), rand(T, H, K, seed=2), rand(T, H, V, seed=3), rand(T, H, V, seed=4)
    h0 = rand(n, H, V, K, seed=5) if carried else torch.zeros(n, H, V, K, dtype=torch.float64)
    dh = rand(n, H, V, K, seed=6) if carried else torch.zeros_like(h0)

    def loss(q, k, v, h0):
        total = 0.0
        for s in range(n):
            i = slice(cu[s], cu[s + 1])
            o, h = la.sequence(q[i], k[i], v[i], ld, h0[s], c)
            total = total + (o * do[i]).sum() + (h * dh[s]).sum()
        return total

    args = [t.clone().requires_grad_() for t in (q, k, v, h0)]
    want = torch.autograd.grad(loss(*args), args)
    got = la.backward(do, q, k, v, ld, cu, h0, dh, c)
    for g, w in zip(got, want):
        assert torch.allclose(g, w, rtol=1e-12, atol=1e-12)
    # a central difference of a quadratic form's parts: exact but for 64-bit rounding over the step
    for i, t in enumerate((q, k, v, h0)):
        step = rand(*t.shape, seed=10 + i)
        at = [q, k, v, h0]
        up, down = list(at), list(at)
        up[i], down[i] = t + 1e-4 * step, t - 1e-4 * step
        assert abs(float((loss(*up) - loss(*down)) / 2e-4 - (got[i] * step).sum())) < 1e-8


def test_chunks_of_the_definition_join():
    """Two halves with the state carried between them are the whole, both ways."""
    H, K, V, T = 2, 4, 3, 11
    ld = torch.tensor([-0.02, -0.5], dtype=torch.float64)
    q, k, v, do = rand(T, H, K, seed=1), rand(T, H, K, seed=2), rand(T, H, V, seed=3), rand(T, H, V, seed=4)
    o, h = la.forward(q, k, v, ld, [0, T])
    o1, h1 = la.forward(q[:6], k[:6], v[:6], ld, [0, 6])
    o2, h2 = la.forward(q[6:], k[6:], v[6:], ld, [0, T - 6], h1)
    assert torch.allclose(torch.cat([o1, o2]), o) and torch.allclose(h2, h)
    whole = la.backward(do, q, k, v, ld, [0, T])
    second = la.backward(do[6:], q[6:], k[6:], v[6:], ld, [0, T - 6], h1)
    first = la.backward(do[:6], q[:6], k[:6], v[:6], ld, [0, 6], None, second[3])
    for i in range(3):
        assert torch.allclose(torch.cat([first[i], second[i]]), whole[i])


@pytest.mark.parametrize("form,center,affine", itertools.product(("none", "silu", "gate"), (True, False), ("", "w", "wb")))
def test_group_norm_gradient_against_autograd(form, center, affine):
    rows, groups, width = 4, 3, 5
    x, dy = rand(rows, groups * width, seed=1), rand(rows, groups * width, seed=2)
    z = rand(rows, groups * width, seed=3) if form == "gate" else None
    w = 1 + 0.1 * rand(groups * width, seed=4) if "w" in affine else None
    b = rand(groups * width, seed=5) if "b" in affine else None
    leaves = {n: t.clone().requires_grad_() for n, t in (("dx", x), ("dz", z), ("dweight", w), ("dbias", b)) if t is not None}
    y = la.group_norm(leaves["dx"], groups, leaves.get("dweight"), leaves.get("dbias"), leaves.get("dz"), 1e-5, center, form == "silu")
    want = dict(zip(leaves, torch.autograd.grad(y, list(leaves.values()), dy)))
    got = la.group_norm_grad(dy, x, groups, w, b, z, 1e-5, center, form == "silu")
    for name, value in want.items():
        assert torch.allclose(got[name], value, rtol=1e-10, atol=1e-10), name
    step = rand(*x.shape, seed=9)
    up, down = (la.group_norm(x + e * step, groups, w, b, z, 1e-5, center, form == "silu") for e in (1e-5, -1e-5))
    assert abs(float(((up - down) / 2e-5 * dy).sum() - (got["dx"] * step).sum())) < 1e-6


# ---------------------------------------------------------------- refusals


def fwd(lib, q=P, k=P, v=P, ld=P, cu=P, h0=None, h1=None, slots=None, pos=None, o=P, nseq=2, total=10, H=4, K=64, V=128,
        longest=0, nslots=4, qs=256, ks=256, vs=512, scale=1.0, io=1, ws=P, wsb=1 << 40):
    return lib.mamba_linear_attention_fwd(q, k, v, ld, cu, h0, h1, slots, pos, o, nseq, total, H, K, V, longest, nslots, qs, ks, vs,
                                          scale, io, ws, wsb, None)


def bwd(lib, do=P, q=P, k=P, v=P, ld=P, cu=P, h0=None, dh1=None, dq=P, dk=P, dv=P, dh0=None, nseq=2, total=10, H=4, K=64, V=128,
        longest=0, gs=512, qs=256, ks=256, vs=512, scale=1.0, io=1, ws=P, wsb=1 << 40):
    return lib.mamba_linear_attention_bwd(do, q, k, v, ld, cu, h0, dh1, dq, dk, dv, dh0, nseq, total, H, K, V, longest, gs, qs, ks,
                                          vs, scale, io, ws, wsb, None)


COMMON = [
    (dict(q=None), ENULL), (dict(k=None), ENULL), (dict(v=None), ENULL), (dict(ld=None), ENULL),
    (dict(nseq=0), ESHAPE), (dict(total=-1), ESHAPE), (dict(H=0), ESHAPE), (dict(K=0), ESHAPE), (dict(V=0), ESHAPE),
    (dict(longest=-1), ESHAPE), (dict(qs=248), ESHAPE), (dict(ks=248), ESHAPE), (dict(vs=504), ESHAPE),
    (dict(cu=None, nseq=3), ESHAPE),   # ten tokens are not three equal sequences
    (dict(total=1 << 55), ESHAPE),
    (dict(K=60), EUNSUP), (dict(V=124), EUNSUP), (dict(K=264, qs=2000, ks=2000), EUNSUP), (dict(V=264, vs=2000), EUNSUP),
    (dict(H=1 << 18, K=128), EUNSUP), (dict(qs=(1 << 24) + 8), EUNSUP), (dict(vs=(1 << 24) + 8), EUNSUP),
    (dict(nseq=1 << 30), EUNSUP), (dict(io=0), EUNSUP), (dict(scale=float("inf")), EUNSUP), (dict(scale=float("nan")), EUNSUP),
    (dict(io=7), EDTYPE),
    (dict(qs=260), EALIGN), (dict(ks=260), EALIGN), (dict(vs=516), EALIGN), (dict(q=P + 8), EALIGN), (dict(k=P + 2), EALIGN),
    (dict(v=P + 8), EALIGN), (dict(ld=P + 2), EALIGN), (dict(cu=P + 4), EALIGN), (dict(h0=P + 8), EALIGN),
]


@pytest.mark.parametrize("bad,code", COMMON + [
    (dict(o=None), ENULL), (dict(slots=P), ENULL), (dict(o=P + 8), EALIGN), (dict(h1=P + 8), EALIGN),
    (dict(h0=P, slots=P + 4), EALIGN), (dict(h0=P, pos=P + 4), EALIGN), (dict(nslots=-1), ESHAPE), (dict(nslots=1 << 60), ESHAPE)])
def test_forward_refusals(lib, bad, code):
    assert fwd(lib, **bad) == code


@pytest.mark.parametrize("bad,code", COMMON + [
    (dict(do=None), ENULL), (dict(dq=None), ENULL), (dict(dk=None), ENULL), (dict(dv=None), ENULL), (dict(gs=504), ESHAPE),
    (dict(gs=516), EALIGN), (dict(do=P + 8), EALIGN), (dict(dq=P + 8), EALIGN), (dict(dk=P + 8), EALIGN), (dict(dv=P + 8), EALIGN),
    (dict(dh0=P + 8), EALIGN), (dict(dh1=P + 8), EALIGN)])
def test_backward_refusals(lib, bad, code):
    assert bwd(lib, **bad) == code


def test_nothing_to_do_launches_nothing(lib):
    assert fwd(lib, total=0) == OK and bwd(lib, total=0) == OK
    assert fwd(lib, total=0, q=None, k=None, v=None, o=None, h0=P, h1=P, slots=P, pos=P) == OK


def test_workspace(lib):
    f, b = lib.mamba_linear_attention_fwd_workspace_size, lib.mamba_linear_attention_bwd_workspace_size
    for size in (f, b):
        assert size(0, 10, 4, 64, 64, 1, 0) == BAD and size(1, 10, 4, 60, 64, 1, 0) == BAD and size(1, 10, 4, 64, 512, 1, 0) == BAD
        assert size(3, 10, 4, 64, 64, 0, 0) == BAD and size(1, 10, 4, 64, 64, 1, -1) == BAD
        assert size(1, 1 << 20, 4, 64, 64, 1, 64) == 0     # known to be short: not cut
        assert size(600, 600 * 64, 8, 64, 64, 0, 0) == 0   # fills the GPU by itself
        assert 0 < size(1, 1 << 20, 4, 64, 128, 1, 0) < BAD and 0 < size(1, 1 << 20, 4, 64, 128, 0, 0) < BAD
    for call, size in ((fwd, f), (bwd, b)):
        need = size(1, 1 << 20, 4, 64, 128, 1, 0)
        big = dict(nseq=1, total=1 << 20)
        assert call(lib, ws=None, **big) == EWS
        assert call(lib, wsb=need - 1, **big) == EWS
        assert call(lib, ws=P + 128, **big) == EWS
    # a state a piece, not a sequence: one long prompt beside many short ones
    state = 4 * 64 * 128 * 4
    assert f(4001, 8096, 4, 64, 128, 1, 0) <= state * 2 * (8096 // 64) + 512


def step(lib, q=P, k=P, v=P, ld=P, state=P, slots=P, pos=P, o=P, batch=3, H=4, K=64, V=128, nslots=4, qs=256, ks=256, vs=512,
         scale=1.0, io=1):
    return lib.mamba_linear_attention_step(q, k, v, ld, state, slots, pos, o, batch, H, K, V, nslots, qs, ks, vs, scale, io, None)


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), ENULL), (dict(k=None), ENULL), (dict(v=None), ENULL), (dict(ld=None), ENULL), (dict(state=None), ENULL),
    (dict(pos=None), ENULL), (dict(o=None), ENULL), (dict(batch=0), ESHAPE), (dict(nslots=-1), ESHAPE), (dict(qs=255), ESHAPE),
    (dict(vs=511), ESHAPE), (dict(nslots=1 << 60), ESHAPE), (dict(K=4), EUNSUP), (dict(K=264, qs=2000, ks=2000), EUNSUP),
    (dict(V=257, vs=2000), EUNSUP), (dict(batch=1 << 30), EUNSUP), (dict(scale=float("nan")), EUNSUP), (dict(io=2), EDTYPE),
    (dict(q=P + 1), EALIGN), (dict(io=0, v=P + 2), EALIGN), (dict(state=P + 8), EALIGN), (dict(pos=P + 4), EALIGN),
    (dict(slots=P + 4), EALIGN), (dict(ld=P + 2), EALIGN)])
def test_step_refusals(lib, bad, code):
    assert step(lib, **bad) == code


def gn(lib, x=P, w=P, b=P, z=None, eps=1e-5, y=P, rows=4, groups=3, width=8, zs=24, center=1, silu=0, io=1):
    return lib.mamba_group_norm_fwd(x, w, b, z, eps, y, rows, groups, width, zs, center, silu, io, None)


def gn_bwd(lib, dy=P, x=P, w=P, b=P, z=None, eps=1e-5, y=P, dz=None, dw=P, db=P, rows=4, groups=3, width=8, zs=24, center=1,
           silu=0, io=1, ws=P, wsb=1 << 40):
    return lib.mamba_group_norm_bwd(dy, x, w, b, z, eps, y, dz, dw, db, rows, groups, width, zs, center, silu, io, ws, wsb, None)


NORM = [
    (dict(x=None), ENULL), (dict(y=None), ENULL), (dict(rows=-1), ESHAPE), (dict(groups=0), ESHAPE), (dict(width=0), ESHAPE),
    (dict(width=8193), EUNSUP), (dict(groups=1 << 22), EUNSUP), (dict(rows=1 << 33), EUNSUP), (dict(eps=-1.0), EUNSUP),
    (dict(eps=float("nan")), EUNSUP), (dict(z=P, dz=P, silu=1), EUNSUP), (dict(z=P, dz=P, zs=23), ESHAPE), (dict(io=3), EDTYPE),
    (dict(x=P + 1), EALIGN), (dict(y=P + 1), EALIGN), (dict(w=P + 2), EALIGN), (dict(b=P + 1), EALIGN), (dict(z=P + 1, dz=P), EALIGN),
]


@pytest.mark.parametrize("bad,code", NORM)
def test_norm_refusals(lib, bad, code):
    assert gn(lib, **{k: v for k, v in bad.items() if k != "dz"}) == code
    assert gn_bwd(lib, **bad) == code


@pytest.mark.parametrize("bad,code", [
    (dict(dy=None), ENULL), (dict(z=P), ENULL), (dict(dz=P), ENULL), (dict(dy=P + 1), EALIGN), (dict(dw=P + 2), EALIGN),
    (dict(db=P + 1), EALIGN), (dict(ws=None), EWS), (dict(ws=P + 16), EWS), (dict(wsb=10), EWS)])
def test_norm_gradient_refusals(lib, bad, code):
    assert gn_bwd(lib, **bad) == code


def test_norm_of_no_rows(lib):
    assert gn(lib, rows=0, x=None, y=None) == OK and gn_bwd(lib, rows=0, dy=None, x=None, y=None, dw=None, db=None) == OK


def test_exports(lib):
    for name in mscan.EXPORTED_LINEAR_ATTENTION:
        assert hasattr(lib, name)


def test_binding_needs_device_tensors():
    t, s = torch.zeros(2, 3, 1, 8, dtype=torch.bfloat16), torch.zeros(1)
    for call in (lambda: mscan.linear_attention_fwd(t, t, t, s), lambda: mscan.linear_attention_bwd(t, t, t, t, s),
                 lambda: mscan.linear_attention_fwd_varlen(t[0], t[0], t[0], s, torch.zeros(2, dtype=torch.int64)),
                 lambda: mscan.linear_attention_step(t[0], t[0], t[0], s, torch.zeros(3, 1, 8, 8), torch.zeros(3, dtype=torch.int64)),
                 lambda: mscan.group_norm_fwd(t, 2), lambda: mscan.group_norm_bwd(t, t, 2)):
        with pytest.raises(ValueError, match="device tensors"):
            call()
