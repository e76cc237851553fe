"""Norm, rotation and linear attention without a GPU: the oracle's own pins (gradients against
differences, closed forms) and what the calls refuse."""
import ctypes

import numpy as np
import pytest

from conftest import ROOT  # noqa: F401
from oracle import layer as L

FAKE = 0x10000  # 16-byte aligned, never dereferenced: validation fails first


@pytest.fixture(scope="module")
def cp():
    import __graft_entry__
    __graft_entry__.build()
    import blockwise_online_softmax_cpattn_gb300 as mod
    return mod


# ---------------------------------------------------------------------------
# oracle
# ---------------------------------------------------------------------------
def _difference(f, x, step=1e-6):
    """Central differences of a scalar function, entry by entry."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        up = f()
        x[i] = keep - step
        down = f()
        x[i] = keep
        g[i] = (up - down) / (2 * step)
    return g


@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("norm", [True, False])
def test_rotation_gradients_against_differences(pairing, norm):
    rng = np.random.default_rng(0)
    x, dy = rng.normal(size=(2, 2, 2, 3, 8))
    w = rng.normal(size=8) if norm else None
    pos, f = [0, 3, 1000], [1.0, 0.01]
    loss = lambda: (L.rotate_fwd(x, w, 1e-3, pos, f, 4, pairing) * dy).sum()  # noqa: E731
    dx, dw = L.rotate_bwd(x, w, 1e-3, pos, f, 4, pairing, dy)
    # differences: step^2 times a third derivative and 1e-16 over the step
    assert np.allclose(dx, _difference(loss, x), atol=1e-7)
    if norm:
        assert np.allclose(dw, _difference(loss, w), atol=1e-7)


def test_rotation_keeps_lengths_and_adds_up():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(1, 1, 4, 16))
    f = 10000.0 ** (-np.arange(8) / 8)
    for pairing in ("halves", "neighbours"):
        y = L.turn(x, [5, 5, 5, 5], f, 16, pairing)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        assert np.allclose(L.turn(y, [2] * 4, f, 16, pairing), L.turn(x, [7] * 4, f, 16, pairing))
        assert np.allclose(L.turn(y, [5] * 4, f, 16, pairing, inverse=True), x)


def test_linear_recurrence_is_the_weighted_sum():
    rng = np.random.default_rng(2)
    B, H, G, T, D = 2, 4, 2, 9, 8
    q = rng.normal(size=(B, H, T, D))
    k, v = rng.normal(size=(2, B, G, T, D))
    S0 = rng.normal(size=(B, H, D, D))
    ld = np.array([-0.5, -1e-3, 0.0, -np.inf])
    o, S = L.linear_fwd(q, k, v, ld, 0.3, S0)
    i = np.arange(T)
    for h in range(H):
        r = np.exp(ld[h])
        w = np.where(i[:, None] >= i, np.power(r, np.maximum(i[:, None] - i, 0)), 0)
        g = h // 2
        ref = ((q[:, h] @ k[:, g].transpose(0, 2, 1)) * w) @ v[:, g]
        ref += np.power(r, i + 1)[:, None] * (q[:, h] @ S0[:, h])
        assert np.allclose(o[:, h], 0.3 * ref)


def test_linear_gradients_against_differences():
    rng = np.random.default_rng(3)
    B, H, G, T, D = 1, 2, 1, 3, 4
    q, do = rng.normal(size=(2, B, H, T, D))
    k, v = rng.normal(size=(2, B, G, T, D))
    S0, dS1 = rng.normal(size=(2, B, H, D, D))
    ld = np.array([-0.3, -0.01])

    def loss():
        o, S1 = L.linear_fwd(q, k, v, ld, 0.5, S0)
        return (o * do).sum() + (S1 * dS1).sum()

    grads = L.linear_bwd(q, k, v, ld, 0.5, do, S0, dS1)
    for x, g in zip((q, k, v, S0), grads):
        assert np.allclose(g, _difference(loss, x), atol=1e-7)


def test_steps_and_lengths_are_the_whole_sequence():
    rng = np.random.default_rng(4)
    B, H, T, D = 3, 2, 7, 4
    q, k, v = rng.normal(size=(3, B, H, T, D))
    ld = [-0.2, -2.0]
    o, S1 = L.linear_fwd(q, k, v, ld, 1.0)
    part, S = L.linear_fwd(q, k, v, ld, 1.0, lengths=[4, 4, 4])
    assert np.array_equal(part[:, :, :4], o[:, :, :4]) and not part[:, :, 4:].any()
    for t in range(4, T):
        y, S = L.linear_step(q[:, :, t], k[:, :, t], v[:, :, t], ld, 1.0, S)
        assert np.allclose(y, o[:, :, t])
    assert np.allclose(S, S1)
    _, S = L.linear_fwd(q, k, v, ld, 1.0, lengths=[0, -3, 99])
    assert not S[:2].any() and np.allclose(S[2], S1[2])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def _rot(mod, **kw):
    base = dict(B=2, H_q=4, H_kv=2, T=64, D=64, cp=2, layout="zigzag", dtype="bf16", norm=1)
    base.update(kw)
    return mod.make_rotate_desc(**base)


def fake(n):
    """n distinct aligned pointers."""
    return [FAKE * (i + 1) for i in range(n)]


def _fwd(cp, d, **kw):
    a = dict(zip(("q", "k", "v", "qw", "kw", "f", "qo", "ko", "vo"), fake(9)), pos=None)
    a.update(kw)
    return cp.cpattn_rotate_fwd(d, a["q"], a["k"], a["v"], a["qw"], a["kw"], a["f"], a["pos"], a["qo"],
                                a["ko"], a["vo"], 0)


def _bwd(cp, d, **kw):
    names = ("q", "k", "qw", "kw", "f", "dqo", "dko", "dvo", "dq", "dk", "dv", "dqw", "dkw", "ws")
    a = dict(zip(names, fake(14)), pos=None, n=1 << 30)
    a.update(kw)
    return cp.cpattn_rotate_bwd(d, a["q"], a["k"], a["qw"], a["kw"], a["f"], a["pos"], a["dqo"], a["dko"],
                                a["dvo"], a["dq"], a["dk"], a["dv"], a["dqw"], a["dkw"], a["ws"], a["n"], 0)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 1), (dict(H_q=0), 1), (dict(H_kv=-1), 1), (dict(T=0), 1), (dict(D=0), 1), (dict(cp=0), 1),
    (dict(T=66), 1),                       # zigzag: T % (2 cp)
    (dict(T=65, layout="contiguous"), 1),  # T % cp
    (dict(layout=9), 1), (dict(dtype=9), 1), (dict(pairing=9), 1), (dict(norm=2), 1),
    (dict(natural_in=3), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
    (dict(rot=-8), 1), (dict(rot=72), 1),
    (dict(rot=12), 2), (dict(D=60, rot=0), 2), (dict(D=136, rot=0), 2), (dict(H_q=1 << 15), 2),
    (dict(B=1 << 20, T=4096), 2),
])
def test_rotation_descriptors(cp, kw, code):
    d = _rot(cp, **kw)
    assert _fwd(cp, d) == code
    assert _bwd(cp, d) == code
    assert cp.cpattn_rotate_bwd_workspace(d) == 0


def test_rotation_arguments(cp):
    d = _rot(cp)
    for name in ("q", "k", "qo", "ko", "v", "vo"):
        assert _fwd(cp, d, **{name: 32 * FAKE + 8}) == 1, name
        if name not in ("v", "vo"):
            assert _fwd(cp, d, **{name: None}) == 1, name
    assert _fwd(cp, d, v=None) == 1 and _fwd(cp, d, vo=None) == 1  # both or neither
    assert _fwd(cp, d, f=None) == 1 and _fwd(cp, d, f=FAKE + 4) == 1
    assert _fwd(cp, d, pos=FAKE + 2) == 1 and _fwd(cp, d, qw=FAKE + 2) == 1
    for name in ("q", "k", "dqo", "dko", "dq", "dk", "ws"):
        assert _bwd(cp, d, **{name: None}) == 1, name
        assert _bwd(cp, d, **{name: 32 * FAKE + 8}) == 1, name
    assert _bwd(cp, d, dv=None) == 1 and _bwd(cp, d, dqw=FAKE + 2) == 1
    assert _bwd(cp, d, n=cp.cpattn_rotate_bwd_workspace(d) - 1) == 1
    plain = _rot(cp, norm=0)
    assert cp.cpattn_rotate_bwd_workspace(plain) == 16
    assert _bwd(cp, plain, q=None, k=None) == 1            # weights' gradients without a norm


def test_rotation_outputs_that_meet(cp):
    """The permuting call is not made in place, and no two outputs are one."""
    d = _rot(cp, natural_in=1)
    q, k, v = fake(3)
    assert _fwd(cp, d, qo=q) == 1 and _fwd(cp, d, ko=q) == 1 and _fwd(cp, d, vo=v) == 1
    assert _fwd(cp, _rot(cp), qo=7 * FAKE, ko=7 * FAKE) == 1
    assert _bwd(cp, d, dq=6 * FAKE) == 1 and _bwd(cp, d, dk=11 * FAKE) == 1   # (dq_out; dv)
    assert _bwd(cp, _rot(cp), dq=10 * FAKE) == 1


def test_rotation_in_place_only_row_by_row(cp):
    """Where tokens stay, an output may be its own input, but no other and by the same strides."""
    d = _rot(cp)
    q, k, v = fake(3)
    assert _fwd(cp, d, qo=k) == 1 and _fwd(cp, d, ko=q) == 1 and _fwd(cp, d, vo=k) == 1
    assert _fwd(cp, d, qo=4 * FAKE) == 1                     # (a weight)
    assert _bwd(cp, d, dq=q) == 1 and _bwd(cp, d, dk=k) == 1  # the forward's inputs
    assert _bwd(cp, d, dqw=32 * FAKE, dkw=32 * FAKE) == 1 and _bwd(cp, d, ws=q) == 1
    i = (ctypes.c_int64 * 3)(64 * 64 * 4, 64 * 64, 64)
    o = (ctypes.c_int64 * 3)(64 * 64 * 4, 64, 64 * 4)
    p = fake(6)
    assert cp._lib.cpattn_rotate_fwd(ctypes.byref(d), p[0], i, p[1], None, None, None, None, None, p[5], None,
                                     p[0], o, p[4], None, None, None, 0) == 1


def test_rotation_strides(cp):
    """Off the 16-byte grid, negative, or an output whose rows would meet."""
    d = _rot(cp)
    lib = cp._lib.cpattn_rotate_fwd

    def call(in_strides, out_strides):
        i = (ctypes.c_int64 * 3)(*in_strides)
        o = (ctypes.c_int64 * 3)(*out_strides)
        p = fake(5)
        return lib(ctypes.byref(d), p[0], i, p[1], None, None, None, None, None, p[2], None, p[3], o, p[4],
                   None, None, None, 0)

    ok = (64 * 64 * 4, 64 * 64, 64)
    for bad in ((ok[0] + 4, ok[1], ok[2]), (ok[0], ok[1] + 4, ok[2]), (ok[0], ok[1], 68), (-ok[0], ok[1], 64)):
        assert call(bad, ok) == 1
        assert call(ok, bad) == 1
    assert call(ok, (0, ok[1], 64)) == 1 and call(ok, (ok[0], 32, 64)) == 1


@pytest.mark.parametrize("kw,code", [
    (dict(H_q=3, H_kv=2), 1), (dict(T=502), 1), (dict(D=192), 2), (dict(D=60), 2), (dict(causal=0), 2),
    (dict(scale=0.0), 1), (dict(dtype=5), 1), (dict(B=0), 1), (dict(a2a=3, cp=2), 1), (dict(B=1 << 24), 2),
])
def test_linear_descriptors(cp, kw, code):
    base = dict(B=1, H_q=4, H_kv=2, T=512, D=64, cp=2, layout="zigzag", dtype="bf16")
    base.update(kw)
    d = cp.make_desc(**base)
    assert cp.cpattn_linear_fwd(d, FAKE, FAKE, FAKE, FAKE, None, None, FAKE, None, FAKE, 1 << 40, 0) == code
    assert cp.cpattn_linear_bwd(d, FAKE, FAKE, FAKE, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, None, FAKE,
                                1 << 40, 0) == code
    assert cp.cpattn_linear_workspace(d) == 0 and cp.cpattn_linear_bwd_workspace(d) == 0
    d.T, d.cp = 1, 1
    if kw.keys() & {"T", "a2a"} == set():
        assert cp.cpattn_linear_step(d, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, n_states=1, stream=0) in (1, 2)


def test_linear_arguments(cp):
    d = cp.make_desc(1, 4, 2, 4096, 64, 2, "zigzag", "bf16")
    fwd = lambda *a, n=1 << 40: cp.cpattn_linear_fwd(d, *a, n, 0)  # noqa: E731
    p = fake(6)
    good = [p[0], p[1], p[2], p[3], None, None, p[4], None, p[5]]
    for i in (0, 1, 2, 3, 6, 8):
        for bad in (None, 64 * FAKE + 2):
            assert fwd(*good[:i], bad, *good[i + 1:]) == 1, i
    for i in (4, 5, 7):
        assert fwd(*good[:i], 64 * FAKE + 2, *good[i + 1:]) == 1, i
    for x in p[:3]:                                     # o or the state over an input
        assert fwd(*good[:6], x, *good[7:]) == 1 and fwd(*good[:7], x, good[8]) == 1
    s = 40 * FAKE                                       # o over state_in; the workspace over anything
    assert fwd(*good[:5], s, s, *good[7:]) == 1 and fwd(*good[:5], s, *good[6:8], s) == 1
    assert fwd(*good[:7], s, s) == 1 and fwd(*good[:8], p[3]) == 1 and fwd(*good[:8], p[4]) == 1
    n = cp.cpattn_linear_workspace(d)
    assert n > 16 and fwd(*good, n=n - 1) == 1
    bwd = lambda *a, n=1 << 40: cp.cpattn_linear_bwd(d, *a, n, 0)  # noqa: E731
    good = fake(12)
    for i in (0, 1, 2, 3, 5, 7, 8, 9, 11):
        for bad in (None, 64 * FAKE + 2):
            assert bwd(*good[:i], bad, *good[i + 1:]) == 1, i
    for i in (4, 6, 10):
        assert bwd(*good[:i], 64 * FAKE + 2, *good[i + 1:]) == 1, i
    for i in (7, 8, 9, 10):                             # an output over an input or another output
        for x in good[:3] + good[4:7] + [y for j, y in enumerate(good[7:11], 7) if j != i]:
            assert bwd(*good[:i], x, *good[i + 1:]) == 1, i
    for x in good[:11]:
        assert bwd(*good[:11], x) == 1
    assert bwd(*good, n=cp.cpattn_linear_bwd_workspace(d) - 1) == 1
    small = cp.make_desc(1, 4, 2, 4096, 64, 2, "zigzag", "bf16", scale=2.0 ** -65)
    assert cp.cpattn_linear_bwd(small, *good, 1 << 40, 0) == 2   # 1 / scale times the state's gradient
    # shared key heads: the query heads' own gradients
    same = cp.make_desc(1, 4, 4, 4096, 64, 2, "zigzag", "bf16")
    assert cp.cpattn_linear_bwd_workspace(d) >= cp.cpattn_linear_bwd_workspace(same) + 2 * 4 * 4 * 4096 * 64


def test_step_arguments(cp):
    d = cp.make_desc(3, 4, 2, 1, 64, 1, "contiguous", "bf16")
    lib = cp._lib.cpattn_linear_step

    p = fake(7)

    def call(q=p[0], ts=256, hs=64, ld=p[3], slots=None, s0=p[4], s1=p[5], o=p[6], n=3, desc=d):
        return lib(ctypes.byref(desc), n, q, ts, hs, p[1], 128, 64, p[2], 128, 64, ld, slots, s0, s1, o, 0)

    assert call(q=None) == 1 and call(q=FAKE + 8) == 1 and call(ts=252) == 1 and call(hs=60) == 1
    assert call(ts=-256) == 1 and call(ld=None) == 1 and call(slots=64 * FAKE + 2) == 1 and call(n=-1) == 1
    assert call(s0=None) == 1 and call(s1=64 * FAKE + 4) == 1 and call(o=None) == 1
    assert call(o=p[1]) == 1 and call(s1=p[0]) == 1 and call(o=p[5]) == 1 and call(o=p[4]) == 1
    assert call(o=p[3]) == 1 and call(slots=p[5]) == 1
    for kw in (dict(T=2), dict(T=2, cp=2), dict(a2a=2, cp=2, T=2)):
        base = dict(B=3, H_q=4, H_kv=2, T=1, D=64, cp=1, layout="contiguous", dtype="bf16")
        base.update(kw)
        assert call(desc=cp.make_desc(**base)) == 1, kw


def test_binding_checks_tensors(cp):
    """Wrong types, shapes and strides raise before the library is called."""
    import torch
    d = _rot(cp, eps=-1.0)  # (refused by the library: nothing would run)
    q, k = torch.zeros(2, 4, 64, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    w = torch.zeros(64, dtype=torch.bfloat16)
    here = cp._here()
    if here != -1:
        pytest.skip("a GPU is here: CPU tensors are refused by their device")
    run = lambda q=q, k=k, f=f, w=w, pos=None: cp.cpattn_rotate_fwd(  # noqa: E731
        d, q, k, None, w, w, f, pos, q if torch.is_tensor(q) else None, k, None, 0)
    assert run() == cp.ERR_INVALID_ARG
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[0]), dict(q=q.transpose(2, 3)), dict(f=f.float()),
                dict(f=f[:31]), dict(w=w.float()), dict(w=w[:63]), dict(pos=torch.zeros(2, 64)),
                dict(pos=torch.zeros(2, 32, dtype=torch.int32))):
        with pytest.raises(ValueError):
            run(**bad)
    d = cp.make_desc(1, 4, 2, 64, 64, 1, "contiguous", "bf16", scale=-1.0)
    q, k = torch.zeros(1, 4, 64, 64, dtype=torch.bfloat16), torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    ld, S, ws = torch.zeros(4), torch.zeros(1, 4, 64, 64), torch.zeros(64)
    n = torch.zeros(1, dtype=torch.int32)
    run = lambda q=q, ld=ld, S=S, n=n: cp.cpattn_linear_fwd(d, q, k, k, ld, n, S, q, None, ws, stream=0)  # noqa: E731
    assert run() == cp.ERR_INVALID_ARG
    for bad in (dict(q=q.float()), dict(q=q[:, :, :32]), dict(ld=ld.double()), dict(ld=ld[:3]), dict(S=S.bfloat16()),
                dict(S=S[:, :2]), dict(n=n.long())):
        with pytest.raises(ValueError):
            run(**bad)
