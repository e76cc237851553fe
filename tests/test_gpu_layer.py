"""GPU: norm and rotation before attention, linear attention and its single-token step, against
the float64 oracle.

Tolerances (half a step of a rounding: bf16 2^-8, float32 2^-24 of the value).

Rotation, forward.  u = w x r: r = rsqrt of a sum of D squares, off by less than 2^-19 (D
additions of 2^-24 each in chains of at most 20, rsqrtf 2^-22); cosine and sine off by less
than 2^-21 (sincospif, and an angle off by 2^-25); so y is off by at most 2^-18 (|u_a| + |u_b|)
of its pair, and its own rounding.
Backward.  With h = w g and n = x r, dx = r (h - n mean(h n)) is off by at most
2^-17 r (|h_a| + |h_b| + |n| mean(|h| |n|)) and its rounding; dw, a sum of N rows of terms off by
2^-17, is off by 2^-17 and N 2^-24 of the sum of magnitudes.

Linear attention.  Everything is bounded by the same sums with magnitudes in place of values
(A: the oracle run on |q|, |k|, |v|, |S|).  On the tensor cores P, the state as an operand and
the weighted keys are rounded to bf16 (keys to two such numbers, 2^-16), so an output is off by at
most two such roundings, 2 * 2^-8 A (second order and float32: 2^-12 A), and its own.  States handed
out carry 24 bits of every product (here 16 would pass, 2^-16; by norm they are held to 24 in
test_gpu_layer_edges.py), float32 folds (2^-22 each chunk) and weights off by 2^-17: 2^-14 A.  In
float32 throughout: at most T + D additions in a chain, weights off by 2^-17:
(2^-24 (T + D) + 2^-16) A.  Gradients are the same sums.
A power of a decay below float32's least normal number, 2^-126, may count as 0: that is off by at
most 2^-126 of the same sums without decay, here fewer than 2^12 terms below 2^8 each (a decay of
e^-200 leaves a gradient of 1e-87 in float64 and 0 in float32), so by less than 2^-100."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT
from gpu_helpers import cp_mod, dev
from oracle import layer as L
from oracle import layouts as OL
from test_gpu_canary import Guarded, check_all

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def f64(t):
    return t.double().cpu().numpy()


def draw(rng, shape, dtype, scale=1.0):
    """Random numbers of the type, on the GPU, and as the oracle takes them."""
    t = torch.from_numpy((rng.normal(size=shape) * scale).astype(np.float32)).to(DT[dtype])
    return t.to(dev()), f64(t)


def checked(cp, status):
    cp.check(status)
    cp.check(cp.cpattn_check())


def within(got, ref, bound, what=""):
    err = np.abs(got - ref)
    bad = ~(err <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(err / np.maximum(bound, 1e-300))),
                           np.argwhere(bad)[:3].tolist())


def positions(T, cp, layout):
    return np.asarray(OL.positions(T, cp, layout))


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------
def pair_sum(u, rot, pairing):
    """|a| + |b| of every channel's pair (|u| of the others)."""
    s = np.abs(u)
    i, j = (slice(0, rot // 2), slice(rot // 2, rot)) if pairing == "halves" else (slice(0, rot, 2), slice(1, rot, 2))
    both = s[..., i] + s[..., j]
    s[..., i] = s[..., j] = both
    return s


def rotation_case(cp, B, Hq, Hkv, T, D, dtype, ranks=1, layout="contiguous", rot=None, pairing="halves",
                  norm=True, natural=1, pos=None, eps=1e-6, strides="fused", values=True, seed=0, f=None,
                  stream=None, weights=True):
    """Runs forward and backward; compares everything, canaries and untouched channels among it."""
    rng = np.random.default_rng(seed)
    rot = D if rot is None else rot
    d = cp.make_rotate_desc(B, Hq, Hkv, T, D, cp=ranks, layout=layout, dtype=dtype, rot=rot, pairing=pairing,
                            norm=int(norm), natural_in=natural, eps=eps)
    W = Hq + 2 * Hkv

    def split(x):
        if strides == "fused":      # [B, T, heads, D]
            y = x.view(B, T, W, D).transpose(1, 2)
        else:                       # [B, heads, T, D]
            y = x.view(B, W, T, D)
        return y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]

    x, _ = draw(rng, (B * T * W * D,), dtype, 2.0)
    q, k, v = split(x)
    ws = [None, None]
    if norm and weights:
        ws = [draw(rng, (D,), dtype)[0] for _ in range(2)]
    if f is None:
        f = 10000.0 ** (-2 * np.arange(rot // 2) / max(rot, 1))
    inv_freq = torch.from_numpy(np.asarray(f, np.float64)).to(dev())
    slot_pos = positions(T, ranks, layout)
    p_dev = None if pos is None else torch.from_numpy(np.asarray(pos, np.int32)).to(dev())
    p = slot_pos if pos is None else np.asarray(pos)
    order = slot_pos if natural else np.arange(T)   # the projection's token of every slot
    outs = {n: Guarded((B, h, T, D), DT[dtype]) for n, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    checked(cp, cp.cpattn_rotate_fwd(d, q, k, v if values else None, ws[0], ws[1], inv_freq, p_dev,
                                     outs["q"].t, outs["k"].t, outs["v"].t if values else None, stream=stream))
    check_all(outs, ["q", "k"] + (["v"] if values else []))
    half = HALF[dtype]
    w64 = [None if not norm else np.ones(D) if w is None else f64(w) for w in ws]
    for n, src, w in (("q", q, w64[0]), ("k", k, w64[1])):
        a = f64(src)[:, :, order]
        ref = L.rotate_fwd(a, w, eps, p, f, rot, pairing)
        u = a if w is None else a / np.sqrt((a * a).mean(-1, keepdims=True) + eps) * w
        within(f64(outs[n].t), ref, 2.0 ** -18 * pair_sum(u, rot, pairing) + half * np.abs(ref), n)
    if values:
        assert np.array_equal(f64(outs["v"].t), f64(v)[:, :, order])

    dys = [draw(rng, (B, h, T, D), dtype) for h in (Hq, Hkv, Hkv)]
    raw = Guarded((B * T * W * D,), DT[dtype])
    dq, dk, dv = split(raw.t)
    dws = {n: Guarded((D,), torch.float32) for n in ("dqw", "dkw")}
    work = Guarded((cp.cpattn_rotate_bwd_workspace(d),), torch.uint8)
    run = lambda: checked(cp, cp.cpattn_rotate_bwd(  # noqa: E731
        d, q if norm else None, k if norm else None, ws[0], ws[1], inv_freq, p_dev, dys[0][0], dys[1][0],
        dys[2][0] if values else None, dq, dk, dv if values else None, dws["dqw"].t if norm else None,
        dws["dkw"].t if norm else None, work.t, stream=stream))
    run()
    first = raw.t.clone(), dws["dqw"].t.clone(), dws["dkw"].t.clone()
    run()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8))
               for a, b in zip(first, (raw.t, dws["dqw"].t, dws["dkw"].t)))  # bitwise
    check_all({"dx": raw, "ws": work, **dws}, (["dqw", "dkw"] if norm else []))
    N = None
    for n, src, out, (_, dy), w in (("dqw", q, dq, dys[0], w64[0]), ("dkw", k, dk, dys[1], w64[1])):
        a = f64(src)[:, :, order]
        ref, dw = L.rotate_bwd(a, w, eps, p, f, rot, pairing, dy)
        got = f64(out)[:, :, order]
        if w is None:
            bound = 2.0 ** -18 * pair_sum(dy, rot, pairing) + half * np.abs(ref)
        else:
            g = L.turn(dy, p, f, rot, pairing, inverse=True)
            gs = pair_sum(g, rot, pairing)   # (turning back mixes errors of the pair)
            r = 1 / np.sqrt((a * a).mean(-1, keepdims=True) + eps)
            nn, h = np.abs(a * r), gs * np.abs(w)
            bound = 2.0 ** -17 * r * (h + nn * (h * nn).mean(-1, keepdims=True)) + half * np.abs(ref)
            N = a.shape[0] * a.shape[1] * a.shape[2]
            mag = (gs * nn).sum((0, 1, 2))
            within(f64(dws[n].t), dw, (2.0 ** -17 + N * 2.0 ** -24) * mag, n)
        within(got, ref, bound, n[:2])
    if values:
        assert np.array_equal(f64(dv)[:, :, order], dys[2][1])
    else:
        untouched = f64(split(raw.t)[2])
        assert np.isnan(untouched).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("D,rot", [(128, 128), (64, 32), (8, 8), (96, 24), (40, 40), (128, 0), (112, 16)])
def test_rotation(dtype, pairing, norm, D, rot):
    rotation_case(cp_mod(), 2, 3, 2, 37, D, dtype, rot=rot, pairing=pairing, norm=norm, seed=D + rot)


@pytest.mark.parametrize("layout,ranks,T", [("contiguous", 1, 1), ("contiguous", 3, 33), ("zigzag", 2, 44), ("zigzag", 8, 1024)])
@pytest.mark.parametrize("natural", [0, 1])
@pytest.mark.parametrize("strides", ["fused", "heads"])
def test_rotation_orders(layout, ranks, T, natural, strides):
    rotation_case(cp_mod(), 1, 4, 2, T, 64, "bf16", ranks=ranks, layout=layout, natural=natural, strides=strides)


@pytest.mark.parametrize("B,T,Hq,Hkv", [(1, 1, 1, 1), (3, 2, 32, 4), (1, 700, 40, 8), (5, 61, 1, 7)])
def test_rotation_sizes(B, T, Hq, Hkv):
    """From a single row to more than every warp takes at once; heads that do not divide."""
    rotation_case(cp_mod(), B, Hq, Hkv, T, 128, "bf16")
    rotation_case(cp_mod(), B, Hq, Hkv, T, 64, "f32", values=False, norm=B != 3)


def test_rotation_without_weights():
    rotation_case(cp_mod(), 1, 2, 2, 9, 64, "bf16", weights=False)


def test_rotation_of_far_and_odd_positions():
    """Positions of 32 bits, of both signs; frequencies from 1 turn in 6 to 1 in 10^9, 0 and above 2."""
    pos = np.array([[0, 1, -1, 131071, 1 << 24, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 123456789]])
    f = np.array([1.0, 0.999999, 0.1, 1e-3, 1e-5, 1e-9, 0.0, 1.9999999])
    rotation_case(cp_mod(), 1, 2, 1, 9, 16, "f32", pos=pos, f=f, norm=False)
    # above 2 the last places of the fixed-point number go: 2^(e-64) a position
    f = np.array([2.0, 3.7, 100.0, 1000.25, 0.5, 0.25, 7.0, 8.0])
    rotation_case(cp_mod(), 1, 2, 1, 9, 16, "f32", pos=pos, f=f, norm=False)


def test_rotation_of_tiny_and_huge_rows():
    cp = cp_mod()
    d = cp.make_rotate_desc(1, 3, 1, 1, 64, dtype="f32", rot=0, eps=0.0)
    x = torch.ones(1, 3, 1, 64, device=dev()) * torch.tensor([1e-15, 1.0, 1e15], device=dev()).view(1, 3, 1, 1)
    k = torch.ones(1, 1, 1, 64, device=dev())
    y, ko = torch.empty_like(x), torch.empty_like(k)
    checked(cp, cp.cpattn_rotate_fwd(d, x, k, None, None, None, None, None, y, ko, None))
    assert torch.allclose(y, torch.ones_like(y), rtol=2.0 ** -19, atol=0)
    d.eps = 1e-6
    x.zero_()  # a row of zeros stays one
    checked(cp, cp.cpattn_rotate_fwd(d, x, k, None, None, None, None, None, y, ko, None))
    assert not y.any()


def test_rotation_in_place_and_packed_tokens():
    """A server's tokens, [n, heads, D], each at its own position; output over input."""
    cp = cp_mod()
    rng = np.random.default_rng(5)
    n, Hq, Hkv, D = 45, 6, 2, 128
    x, x64 = draw(rng, (n, Hq + 2 * Hkv, D), "bf16")
    pos = rng.integers(0, 10 ** 6, (1, n)).astype(np.int32)
    f = 1e6 ** (-2 * np.arange(64) / 128)
    d = cp.make_rotate_desc(1, Hq, Hkv, n, D)
    w, w64 = draw(rng, (D,), "bf16")
    view = lambda a, b: x[:, a:b].transpose(0, 1).unsqueeze(0)  # noqa: E731
    q, k, v = view(0, Hq), view(Hq, Hq + Hkv), view(Hq + Hkv, Hq + 2 * Hkv)
    checked(cp, cp.cpattn_rotate_fwd(d, q, k, v, w, w, torch.from_numpy(f).to(dev()),
                                     torch.from_numpy(pos).to(dev()), q, k, v))
    heads = x64.transpose(1, 0, 2)[None]
    ref = L.rotate_fwd(heads[:, :Hq + Hkv], w64, 1e-6, pos, f, D, "halves")
    got = f64(x).transpose(1, 0, 2)[None]
    u = pair_sum(heads[:, :Hq + Hkv] / np.sqrt((heads[:, :Hq + Hkv] ** 2).mean(-1, keepdims=True) + 1e-6) * w64, D, "halves")
    within(got[:, :Hq + Hkv], ref, 2.0 ** -18 * u + HALF["bf16"] * np.abs(ref))
    assert np.array_equal(got[:, Hq + Hkv:], heads[:, Hq + Hkv:])


@pytest.mark.parametrize("dtype,D,norm", [("bf16", 128, 1), ("f32", 48, 1), ("bf16", 64, 0)])
def test_rotation_backward_in_place(dtype, D, norm):
    """Gradients over the upstream gradients: the same numbers as apart from them."""
    cp = cp_mod()
    rng = np.random.default_rng(7)
    d = cp.make_rotate_desc(2, 3, 2, 700, D, dtype=dtype, norm=norm)
    shapes = [(2, h, 700, D) for h in (3, 2, 2)]
    x = [draw(rng, sh, dtype)[0] for sh in shapes]
    dy = [draw(rng, sh, dtype)[0] for sh in shapes]
    f = torch.from_numpy(100.0 ** (-np.arange(D // 2) / D)).to(dev())
    ws = torch.empty(cp.cpattn_rotate_bwd_workspace(d), dtype=torch.uint8, device=dev())
    dw = [torch.empty(D, device=dev()) for _ in range(4)]

    def run(out, dws):
        checked(cp, cp.cpattn_rotate_bwd(d, x[0] if norm else None, x[1] if norm else None, None, None, f, None,
                                         *dy, *out, dws[0] if norm else None, dws[1] if norm else None, ws))

    apart = [torch.empty_like(t) for t in dy]
    run(apart, dw[:2])
    run(dy, dw[2:])
    for a, b in zip(apart, dy):
        assert torch.equal(a, b)
    if norm:
        assert torch.equal(dw[0], dw[2]) and torch.equal(dw[1], dw[3])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(1, 128), (5, 128), (33, 64), (3, 48)])
def test_rotation_without_epsilon(dtype, T, D):
    """A warp whose slots are not all of the batch divides nothing by nothing."""
    rotation_case(cp_mod(), 1, 3, 2, T, D, dtype, eps=0.0)


def test_rotation_past_32_bits():
    """Strides and offsets of more than 2^31 elements."""
    cp = cp_mod()
    big = torch.empty(2 ** 31 + 2 ** 12, dtype=torch.bfloat16, device=dev())
    q = big.as_strided((2, 1, 3, 64), (2 ** 31, 192, 64, 1))
    rng = np.random.default_rng(6)
    x, x64 = draw(rng, (2, 1, 3, 64), "bf16")
    q.copy_(x)
    f = 100.0 ** (-np.arange(32) / 32)
    d = cp.make_rotate_desc(2, 1, 1, 3, 64, norm=0)
    out = torch.empty_like(x)
    checked(cp, cp.cpattn_rotate_fwd(d, q, x, None, None, None, torch.from_numpy(f).to(dev()), None, q, out, None))
    ref = L.rotate_fwd(x64, None, 0, np.arange(3), f, 64, "halves")
    for y in (out, q):
        within(f64(y), ref, 2.0 ** -18 * pair_sum(x64, 64, "halves") + HALF["bf16"] * np.abs(ref))
    del big, q
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------
def spread_decays(H):
    """From a memory of one token to one that hardly fades."""
    return -np.exp2(-np.arange(H) * 9.0 / max(H - 1, 1)).astype(np.float32)


class LinearCase:
    def __init__(self, B, Hq, Hkv, T, D, dtype, ranks=1, layout="contiguous", a2a=1, ld=None, state=True,
                 lengths=None, scale=None, seed=0):
        self.cp = cp_mod()
        self.d = self.cp.make_desc(B, Hq, Hkv, T, D, ranks, layout, dtype, a2a=a2a, scale=scale)
        self.scale = float(self.d.scale)
        rng = np.random.default_rng(seed)
        self.dtype, self.T, self.D, self.a2a = dtype, T, D, a2a
        self.shape_q, self.shape_kv = (B, Hq, T, D), (B, Hkv, T, D)
        self.slots = np.argsort(positions(T, ranks // a2a, layout))  # slot of every natural position
        self.ld = spread_decays(Hq) if ld is None else np.asarray(ld, np.float32)
        self.ld_dev = torch.from_numpy(self.ld).to(dev())
        self.lengths = lengths
        self.len_dev = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=dev())
        self.q, q = self._tensor(rng, self.shape_q)
        self.k, k = self._tensor(rng, self.shape_kv)
        self.v, v = self._tensor(rng, self.shape_kv)
        self.do, do = self._tensor(rng, self.shape_q)
        self.nat = q, k, v, do
        self.S0 = self.dS1 = s0 = ds1 = None
        if state:
            (self.S0, s0), (self.dS1, ds1) = (self._state(rng, B, Hq, D) for _ in range(2))
        self.states = s0, ds1
        # where the products run: on tensor cores or in float32
        self.tc = dtype == "bf16" and D in (64, 128) and (layout == "contiguous" or T // (ranks // a2a) // 2 >= 16)

    def _tensor(self, rng, shape):
        """Natural order for the oracle; layout order, head-sharded for a2a > 1, on the GPU."""
        t = torch.from_numpy(rng.normal(size=shape).astype(np.float32)).to(DT[self.dtype])
        x = t[:, :, torch.from_numpy(np.argsort(self.slots))].to(dev())
        return self._shard(x), f64(t)

    def _shard(self, x):
        B, H = x.shape[:2]
        return x.view(B, self.a2a, H // self.a2a, *x.shape[2:]).transpose(0, 1).contiguous()

    def unshard(self, x, tokens=True):
        """[a2a * B][H / a2a].. -> float64 [B][H].., tokens in natural order."""
        B = self.shape_q[0]
        x = f64(x)
        x = x.reshape(self.a2a, B, -1, *x.shape[-2:]).swapaxes(0, 1)
        x = x.reshape(B, -1, *x.shape[-2:])
        return x[:, :, self.slots] if tokens else x

    def _state(self, rng, B, H, D):
        t = torch.from_numpy(rng.normal(size=(B, H, D, D)).astype(np.float32))
        return self._shard(t.to(dev())), f64(t)

    def bounds(self, ref, A, dtype):
        half = HALF[dtype] * np.abs(ref)
        if self.tc:
            return (2 * 2.0 ** -8 + 2.0 ** -12) * A + half + 2.0 ** -100
        return (2.0 ** -24 * (self.T + self.D) + 2.0 ** -16) * A + half + 2.0 ** -100

    def state_bounds(self, ref, A):
        return (2.0 ** -14 if self.tc else 2.0 ** -24 * (self.T + self.D) + 2.0 ** -16) * A + 2.0 ** -100

    def forward(self, out=None, state_out=None, ws=None, stream=None):
        cp = self.cp
        o = torch.empty_like(self.q) if out is None else out
        ws = torch.empty(cp.cpattn_linear_workspace(self.d), dtype=torch.uint8, device=dev()) if ws is None else ws
        cp.check(cp.cpattn_linear_fwd(self.d, self.q, self.k, self.v, self.ld_dev, self.len_dev, self.S0, o,
                                      state_out, ws, stream=stream))
        return o

    def check_forward(self):
        cp = self.cp
        o = Guarded(tuple(self.q.shape), DT[self.dtype])
        B, H = self.q.shape[1] * self.a2a, self.q.shape[2]
        S1 = Guarded((self.a2a * self.shape_q[0], self.q.shape[2], self.D, self.D), torch.float32)
        ws = Guarded((cp.cpattn_linear_workspace(self.d),), torch.uint8)
        self.forward(o.t, S1.t, ws.t)
        cp.check(cp.cpattn_check())
        q, k, v, _ = self.nat
        ref, S = L.linear_fwd(q, k, v, self.ld, self.scale, self.states[0], self.lengths)
        mag = lambda x: None if x is None else np.abs(x)  # noqa: E731
        A, AS = L.linear_fwd(mag(q), mag(k), mag(v), self.ld, self.scale, mag(self.states[0]), self.lengths)
        got = self.unshard(o.t)
        n = [self.T] * self.shape_q[0] if self.lengths is None else [min(max(x, 0), self.T) for x in self.lengths]
        for b, m in enumerate(n):
            within(got[b, :, :m], ref[b, :, :m], self.bounds(ref, A, self.dtype)[b, :, :m], "o")
            assert np.isnan(got[b, :, m:]).all()          # rows behind the end: as they were
        within(self.unshard(S1.t, False), S, self.state_bounds(S, AS), "state")
        check_all({"o": o, "state": S1, "ws": ws}, ["state"])
        first = o.t.clone(), S1.t.clone()
        self.forward(o.t, S1.t, ws.t)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, (o.t, S1.t)))
        # without the state out: its own roundings, the same bounds
        plain = Guarded(tuple(self.q.shape), DT[self.dtype])
        self.forward(plain.t, None, ws.t)
        cp.check(cp.cpattn_check())
        got = self.unshard(plain.t)
        for b, m in enumerate(n):
            within(got[b, :, :m], ref[b, :, :m], self.bounds(ref, A, self.dtype)[b, :, :m], "o alone")

    def backward(self, outs, ws, stream=None):
        cp = self.cp
        cp.check(cp.cpattn_linear_bwd(self.d, self.q, self.k, self.v, self.ld_dev, self.S0, self.do, self.dS1,
                                      outs[0], outs[1], outs[2], outs[3], ws, stream=stream))

    def check_backward(self, dstate=True):
        cp = self.cp
        bufs = {n: Guarded(tuple(x.shape), DT[self.dtype]) for n, x in (("dq", self.q), ("dk", self.k), ("dv", self.v))}
        if dstate:
            bufs["dstate"] = Guarded((self.a2a * self.shape_q[0], self.q.shape[2], self.D, self.D), torch.float32)
        bufs["ws"] = Guarded((cp.cpattn_linear_bwd_workspace(self.d),), torch.uint8)
        outs = [bufs[n].t for n in ("dq", "dk", "dv")] + [bufs["dstate"].t if dstate else None]
        self.backward(outs, bufs["ws"].t)
        cp.check(cp.cpattn_check())
        check_all(bufs, [n for n in bufs if n != "ws"])
        q, k, v, do = self.nat
        refs = L.linear_bwd(q, k, v, self.ld, self.scale, do, *self.states)
        mag = [None if x is None else np.abs(x) for x in (q, k, v, do, *self.states)]
        As = L.linear_bwd(*mag[:3], self.ld, self.scale, mag[3], *mag[4:])
        for n, ref, A in zip(("dq", "dk", "dv"), refs, As):
            within(self.unshard(bufs[n].t), ref, self.bounds(ref, A, self.dtype), n)
        if dstate:
            within(self.unshard(bufs["dstate"].t, False), refs[3], self.state_bounds(refs[3], As[3]), "dstate")
        first = [x.clone() for x in outs if x is not None]
        self.backward(outs, bufs["ws"].t)
        assert all(torch.equal(a, b) for a, b in zip(first, [x for x in outs if x is not None]))


SHAPES = [
    # B, Hq, Hkv, T, D, dtype, ranks, layout, a2a
    (1, 2, 2, 1, 128, "bf16", 1, "contiguous", 1),
    (2, 2, 1, 2, 64, "bf16", 1, "contiguous", 1),
    (1, 2, 2, 127, 128, "bf16", 1, "contiguous", 1),
    (1, 3, 1, 128, 128, "bf16", 1, "contiguous", 1),
    (2, 2, 2, 129, 64, "bf16", 1, "contiguous", 1),
    (1, 2, 1, 255, 128, "bf16", 3, "contiguous", 1),
    (1, 4, 2, 1000, 128, "bf16", 1, "contiguous", 1),    # runs
    (1, 2, 1, 1025, 64, "bf16", 1, "contiguous", 1),
    (2, 4, 2, 1024, 128, "bf16", 4, "zigzag", 1),
    (1, 8, 4, 512, 64, "bf16", 4, "zigzag", 2),          # head-sharded: decays by the whole head number
    (1, 2, 2, 320, 128, "bf16", 2, "zigzag", 1),         # halves of 80 tokens: a chunk each
    (2, 4, 2, 1200, 128, "bf16", 3, "zigzag", 1),        # of 200: a whole and a partial one, and runs
    (1, 4, 4, 528, 64, "bf16", 4, "zigzag", 2),          # of 132
    (1, 2, 1, 520, 128, "bf16", 2, "zigzag", 1),         # of 130
    (1, 2, 2, 512, 64, "bf16", 16, "zigzag", 1),         # of 16
    (1, 2, 2, 120, 64, "bf16", 4, "zigzag", 1),          # of 15: float32
    (1, 2, 1, 200, 32, "bf16", 1, "contiguous", 1),
    (1, 2, 2, 1, 128, "f32", 1, "contiguous", 1),
    (2, 4, 2, 63, 128, "f32", 1, "contiguous", 1),
    (1, 2, 2, 64, 64, "f32", 1, "contiguous", 1),
    (1, 2, 1, 65, 24, "f32", 1, "contiguous", 1),
    (1, 2, 2, 700, 128, "f32", 1, "contiguous", 1),
    (1, 2, 1, 660, 72, "f32", 3, "zigzag", 1),
    (2, 4, 4, 96, 8, "f32", 4, "zigzag", 4),
]


def ids(s):
    return "-".join(str(x) for x in s)


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("state", [False, True])
def test_linear_forward(shape, state):
    B, Hq, Hkv, T, D, dtype, ranks, layout, a2a = shape
    LinearCase(B, Hq, Hkv, T, D, dtype, ranks, layout, a2a, state=state).check_forward()


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
@pytest.mark.parametrize("state", [False, True])
def test_linear_backward(shape, state):
    B, Hq, Hkv, T, D, dtype, ranks, layout, a2a = shape
    LinearCase(B, Hq, Hkv, T, D, dtype, ranks, layout, a2a, state=state).check_backward(dstate=state)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64), ("f32", 40)])
@pytest.mark.parametrize("T", [5, 300, 900])
def test_linear_lengths(dtype, D, T):
    """Padded rows: empty, negative, one token, off and on the chunk's grid, whole, beyond; what the
    padding holds, NaN and infinities, does not matter."""
    lengths = [0, 1, T, -7, T + 100, T - 1, min(128, T), min(257, T)]
    c = LinearCase(len(lengths), 2, 1, T, D, dtype, lengths=lengths)
    for b, n in enumerate(lengths):
        n = min(max(n, 0), T)
        for i, x in enumerate((c.q, c.k, c.v)):
            x.view(len(lengths), -1, T, D)[b, :, n:] = (float("nan"), float("inf"), float("-inf"))[(i + b) % 3]
    c.check_forward()


@pytest.mark.parametrize("T,ranks", [(320, 2), (1200, 3), (1024, 4)])
def test_linear_lengths_in_zigzag_order(T, ranks):
    """Positions, not slots, count; rows that end in every kind of chunk."""
    h = T // ranks // 2
    lengths = [0, 1, h - 1, h, h + 1, 2 * h + min(h, 129), T - 1, T]
    c = LinearCase(len(lengths), 2, 1, T, 64, "bf16", ranks, "zigzag", lengths=lengths)
    slots = torch.from_numpy(c.slots).to(dev())
    for b, n in enumerate(lengths):
        for x in (c.q, c.k, c.v):
            x[0][b][:, slots[n:]] = float("nan")
    c.check_forward()


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_linear_extreme_decays(dtype, D):
    """None at all, so strong that a token sees itself alone, and what counts as 0."""
    ld = [0.0, -float("inf"), -1e-7, -30.0, -200.0, 3.0, float("nan"), -0.69314718]
    c = LinearCase(1, 8, 8, 520, D, dtype, ld=ld)
    c.check_forward()
    c.check_backward()


def test_linear_long_memory():
    """Without decay over 16 chunks and several runs, in float32 states."""
    c = LinearCase(1, 1, 1, 2100, 128, "bf16", ld=[0.0])
    c.check_forward()


@pytest.mark.parametrize("dtype,D,T", [("bf16", 128, 900), ("bf16", 128, 100), ("f32", 64, 500)])
def test_linear_state_in_place(dtype, D, T):
    """state_out over state_in, also where several runs of a sequence read it."""
    c = LinearCase(1, 2, 2, T, D, dtype)
    S1 = torch.empty_like(c.S0)
    o = c.forward(None, S1).clone()
    keep = c.S0.clone()
    got = c.forward(None, c.S0)
    c.cp.check(c.cp.cpattn_check())
    assert torch.equal(got, o) and torch.equal(c.S0, S1) and not torch.equal(keep, S1)


def test_linear_in_parts_is_the_whole():
    """A prompt in two calls that hand the state on."""
    cp = cp_mod()
    B, H, T, D, cut = 1, 3, 700, 128, 333
    c = LinearCase(B, H, H, T, D, "bf16", state=False)
    q, k, v = (x.view(B, H, T, D) for x in (c.q, c.k, c.v))
    S = torch.zeros(B, H, D, D, device=dev())
    parts = []
    for a, b in ((0, cut), (cut, T)):
        d = cp.make_desc(B, H, H, b - a, D, 1, "contiguous", "bf16")
        x = [y[:, :, a:b].contiguous() for y in (q, k, v)]
        o = torch.empty_like(x[0])
        ws = torch.empty(cp.cpattn_linear_workspace(d), dtype=torch.uint8, device=dev())
        checked(cp, cp.cpattn_linear_fwd(d, *x, c.ld_dev, None, S, o, S, ws))
        parts.append(f64(o))
    nat = c.nat[:3]
    ref, S1 = L.linear_fwd(*nat, c.ld, c.scale)
    A, AS = L.linear_fwd(*map(np.abs, nat), c.ld, c.scale)
    within(np.concatenate(parts, 2), ref, c.bounds(ref, A, "bf16"))
    within(f64(S), S1, c.state_bounds(S1, AS))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_past_32_bits(dtype):
    """More than 2^31 elements a tensor: the last heads are right."""
    cp = cp_mod()
    H, T, D = 16400, 1024, 128
    assert H * T * D > 2 ** 31
    d = cp.make_desc(1, H, H, T, D, 1, "contiguous", dtype)
    x = torch.zeros(1, H, T, D, dtype=DT[dtype], device=dev())
    rng = np.random.default_rng(8)
    last, nat = draw(rng, (1, 2, T, D), dtype)
    x[:, -2:] = last
    ld = np.full(H, -0.05, np.float32)
    o = torch.empty_like(x)
    ws = torch.empty(cp.cpattn_linear_workspace(d), dtype=torch.uint8, device=dev())
    checked(cp, cp.cpattn_linear_fwd(d, x, x, x, torch.from_numpy(ld).to(dev()), None, None, o, None, ws))
    ref, _ = L.linear_fwd(nat, nat, nat, ld[:2], float(d.scale))
    A, _ = L.linear_fwd(np.abs(nat), np.abs(nat), np.abs(nat), ld[:2], float(d.scale))
    tol = 2 * 2.0 ** -8 + 2.0 ** -12 if dtype == "bf16" else 2.0 ** -24 * (T + D) + 2.0 ** -16
    within(f64(o[:, -2:]), ref, tol * A + HALF[dtype] * np.abs(ref))
    assert not o[:, :-2].any()
    del x, o, ws
    torch.cuda.empty_cache()


def test_linear_timeout_is_reported_and_context_survives():
    cp = cp_mod()
    c = LinearCase(1, 2, 2, 700, 128, "bf16")
    for backward in (False, True):
        c.d.debug_fault = 1
        if backward:
            outs = [torch.empty_like(x) for x in (c.q, c.k, c.v, c.S0)]
            c.backward(outs, torch.empty(cp.cpattn_linear_bwd_workspace(c.d), dtype=torch.uint8, device=dev()))
        else:
            c.forward()
        assert cp.cpattn_check() == cp.ERR_TIMEOUT
        assert cp.cpattn_check() == cp.OK
        c.d.debug_fault = 0
        c.check_forward()


# ---------------------------------------------------------------------------
# a token at a time
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("n,Hq,Hkv,D,dtype", [(1, 1, 1, 8, "f32"), (1, 4, 2, 128, "bf16"), (3, 2, 1, 64, "bf16"),
                                             (70, 32, 4, 64, "bf16"), (5, 3, 3, 24, "f32"), (40, 32, 32, 128, "f32"),
                                             (50, 30, 10, 72, "bf16")])
@pytest.mark.parametrize("in_place", [False, True])
def test_step(n, Hq, Hkv, D, dtype, in_place):
    """Permuted slots, requests left out, states without one; rows of a fused projection."""
    cp = cp_mod()
    rng = np.random.default_rng(n + D)
    d = cp.make_desc(n, Hq, Hkv, 1, D, 1, "contiguous", dtype)
    x, x64 = draw(rng, (n, Hq + 2 * Hkv, D), dtype)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    ld = spread_decays(Hq)
    n_states = n + 3
    S = Guarded((n_states, Hq, D, D), torch.float32)
    S.t.copy_(torch.from_numpy(rng.normal(size=(n_states, Hq, D, D)).astype(np.float32)))
    S64 = f64(S.t)
    out = S if in_place else Guarded((n_states, Hq, D, D), torch.float32)
    slots = rng.permutation(n_states)[:n]
    left_out = []
    if n > 2:
        slots[1], slots[2] = -1, n_states
        left_out = [1, 2]
    o = Guarded((n, Hq, D), DT[dtype])
    checked(cp, cp.cpattn_linear_step(d, q, k, v, torch.from_numpy(ld).to(dev()),
                                      torch.from_numpy(slots.astype(np.int32)).to(dev()), S.t, out.t, o.t))
    check_all({"S": S, "out": out, "o": o})
    live = [b for b in range(n) if b not in left_out]
    args = [f64(t)[live] for t in (q, k, v)]
    ref, S1 = L.linear_step(*args, ld, float(d.scale), S64[slots[live]])
    A, AS = L.linear_step(*map(np.abs, args), ld, float(d.scale), np.abs(S64[slots[live]]))
    within(f64(o.t)[live], ref, (2.0 ** -24 * (D + 16) + 2.0 ** -20) * A + HALF[dtype] * np.abs(ref))
    assert np.isnan(f64(o.t)[left_out]).all()
    got = f64(out.t)
    within(got[slots[live]], S1, 2.0 ** -20 * AS)
    rest = sorted(set(range(n_states)) - set(slots[live].tolist()))
    assert np.array_equal(got[rest], S64[rest]) if in_place else np.isnan(got[rest]).all()


def test_step_without_slots_and_decay_of_zero():
    cp = cp_mod()
    rng = np.random.default_rng(1)
    d = cp.make_desc(2, 2, 2, 1, 64, 1, "contiguous", "f32")
    x, x64 = draw(rng, (2, 6, 64), "f32")
    S, S64 = draw(rng, (2, 2, 64, 64), "f32")
    o = torch.empty(2, 2, 64, device=dev())
    ld = np.array([-np.inf, 1.0], np.float32)
    checked(cp, cp.cpattn_linear_step(d, x[:, :2], x[:, 2:4], x[:, 4:], torch.from_numpy(ld).to(dev()), None, S, S, o))
    ref, S1 = L.linear_step(x64[:, :2], x64[:, 2:4], x64[:, 4:], ld, float(d.scale), S64)
    A, AS = L.linear_step(*(np.abs(y) for y in (x64[:, :2], x64[:, 2:4], x64[:, 4:])), ld, float(d.scale), np.abs(S64))
    within(f64(o), ref, 2.0 ** -16 * A)
    within(f64(S), S1, 2.0 ** -20 * AS)


def test_step_past_32_bits():
    """A state behind 2^31 numbers."""
    cp = cp_mod()
    H, D = 64, 128
    n_states = 2 ** 31 // (H * D * D) + 2
    S = torch.empty(n_states, H, D, D, device=dev())
    S[-1] = 1.0
    S[0] = 2.0
    d = cp.make_desc(1, H, H, 1, D, 1, "contiguous", "f32", scale=1.0)
    q = torch.ones(1, H, D, device=dev())
    kv = torch.zeros(1, H, D, device=dev())
    o = torch.empty(1, H, D, device=dev())
    slots = torch.tensor([n_states - 1], dtype=torch.int32, device=dev())
    checked(cp, cp.cpattn_linear_step(d, q, kv, kv, torch.zeros(H, device=dev()), slots, S, S, o))
    assert bool((o == D).all()) and bool((S[0] == 2).all()) and bool((S[-1] == 1).all())
    del S
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------
# streams, graphs, the debug build, other devices
# ---------------------------------------------------------------------------
def test_another_stream_and_captured_calls():
    """Forward and backward on a stream of their own, and two captured graphs that share one
    workspace, replayed in turn on new inputs."""
    cp = cp_mod()
    cases = [LinearCase(1, 2, 1, 900, 128, "bf16", seed=i) for i in range(2)]
    n = max(cp.cpattn_linear_workspace(cases[0].d), cp.cpattn_linear_bwd_workspace(cases[0].d))
    ws = torch.empty(n, dtype=torch.uint8, device=dev())
    side = torch.cuda.Stream()

    def outputs(c):
        return [torch.empty_like(x) for x in (c.q, c.S0, c.q, c.k, c.v, c.S0)]

    def step(c, out, stream=None):
        c.forward(out[0], out[1], ws, stream)
        c.backward(out[2:], ws, stream)

    refs = []
    for c in cases:
        out = outputs(c)
        step(c, out)
        refs.append([x.clone() for x in out])
    torch.cuda.synchronize()
    outs = [outputs(c) for c in cases]
    side.wait_stream(torch.cuda.current_stream())
    step(cases[0], outs[0], side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], refs[0]))
    graphs = []
    for c, out in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(c, out)
        graphs.append(g)
    for x in outs[0] + outs[1]:
        x.fill_(float("nan"))
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    cp.check(cp.cpattn_check())
    for out, ref in zip(outs, refs):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    # new inputs under the first graph
    for a, b in zip((cases[0].q, cases[0].k, cases[0].v, cases[0].do, cases[0].S0, cases[0].dS1),
                    (cases[1].q, cases[1].k, cases[1].v, cases[1].do, cases[1].S0, cases[1].dS1)):
        a.copy_(b)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs[0], refs[1]))


def test_two_streams_at_once():
    """Calls side by side, each with its own workspace: what each gives alone."""
    cp = cp_mod()
    cases = [LinearCase(1, 4, 2, 3000, 128, "bf16", seed=1), LinearCase(2, 4, 4, 640, 64, "bf16", 2, "zigzag", seed=2),
             LinearCase(1, 2, 2, 900, 128, "f32", seed=3)]
    refs, outs, wss = [], [], []
    for c in cases:
        n = max(cp.cpattn_linear_workspace(c.d), cp.cpattn_linear_bwd_workspace(c.d))
        wss.append(torch.empty(n, dtype=torch.uint8, device=dev()))
        ref = [torch.empty_like(x) for x in (c.q, c.S0, c.q, c.k, c.v, c.S0)]
        c.forward(ref[0], ref[1], wss[-1])
        c.backward(ref[2:], wss[-1])
        refs.append(ref)
        outs.append([torch.empty_like(x) for x in ref])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for c, out, ws, st in zip(cases, outs, wss, streams):
            c.forward(out[0], out[1], ws, st)
            c.backward(out[2:], ws, st)
    torch.cuda.synchronize()
    cp.check(cp.cpattn_check())
    for out, ref in zip(outs, refs):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 40)])
def test_linear_on_16_byte_boundaries(dtype, D):
    """Tensors that begin 16 bytes behind a coarser boundary."""
    cp = cp_mod()
    c = LinearCase(1, 2, 1, 700, D, dtype, seed=4)
    ws = torch.empty(max(cp.cpattn_linear_workspace(c.d), cp.cpattn_linear_bwd_workspace(c.d)), dtype=torch.uint8,
                     device=dev())

    def off(x):
        n = 16 // x.element_size()
        y = torch.empty(x.numel() + n, dtype=x.dtype, device=dev())[n:].view(x.shape)
        return y.copy_(x)

    def run():
        out = [off(torch.zeros_like(x)) if shifted else torch.empty_like(x) for x in (c.q, c.S0, c.q, c.k, c.v, c.S0)]
        c.forward(out[0], out[1], ws)
        c.backward(out[2:], ws)
        cp.check(cp.cpattn_check())
        return out

    shifted = False
    ref = run()
    shifted = True
    c.q, c.k, c.v, c.do, c.S0, c.dS1 = (off(x) for x in (c.q, c.k, c.v, c.do, c.S0, c.dS1))
    assert c.q.data_ptr() % 32 == 16
    for a, b in zip(run(), ref):
        assert torch.equal(a, b)


def test_rotation_captured():
    cp = cp_mod()
    rng = np.random.default_rng(3)
    d = cp.make_rotate_desc(1, 4, 2, 300, 128)
    q, k = draw(rng, (1, 4, 300, 128), "bf16")[0], draw(rng, (1, 2, 300, 128), "bf16")[0]
    f = torch.ones(64, dtype=torch.float64, device=dev())
    w = draw(rng, (128,), "bf16")[0]
    qo, ko, dq, dk = (torch.empty_like(x) for x in (q, k, q, k))
    dw = torch.zeros(2, 128, device=dev())
    ws = torch.empty(cp.cpattn_rotate_bwd_workspace(d), dtype=torch.uint8, device=dev())

    def step():
        cp.check(cp.cpattn_rotate_fwd(d, q, k, None, w, w, f, None, qo, ko, None))
        cp.check(cp.cpattn_rotate_bwd(d, q, k, w, w, f, None, qo, ko, None, dq, dk, None, dw[0], dw[1], ws))

    step()
    ref = [x.clone() for x in (qo, ko, dq, dk, dw)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        for x in (qo, ko, dq, dk, dw):
            x.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((qo, ko, dq, dk, dw), ref))


def test_tensors_of_another_device_are_refused():
    cp = cp_mod()
    d = cp.make_desc(1, 2, 2, 8, 64, 1, "contiguous", "bf16")
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device=dev())
    ld, ws = torch.zeros(2, device=dev()), torch.zeros(1024, device=dev())
    for bad in (x.cpu(), ):
        with pytest.raises(ValueError):
            cp.cpattn_linear_fwd(d, bad, x, x, ld, None, None, x, None, ws)
    with pytest.raises(ValueError):
        cp.cpattn_linear_fwd(d, x, x, x, ld.cpu(), None, None, x, None, ws)
    r = cp.make_rotate_desc(1, 2, 2, 8, 64, norm=0, rot=0)
    with pytest.raises(ValueError):
        cp.cpattn_rotate_fwd(r, x, x.cpu(), None, None, None, None, None, x, x, None)


def test_under_bounds_checks():
    """The linear kernels of the CPATTN_DEBUG build check every row they compute."""
    import __graft_entry__
    __graft_entry__._build_lib().build(debug=True)
    env = dict(os.environ, CPATTN_DEBUG_LIB="1")
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_layer.py", "-m", "gpu", "-x", "-q", "-k",
                        "linear_forward or linear_backward or linear_lengths", "-p", "no:cacheprovider"], cwd=ROOT,
                       env=env, capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]


# ---------------------------------------------------------------------------
# as they are used
# ---------------------------------------------------------------------------
def _close(got, ref, tol, what):
    """Norms: chains of kernels, whose roundings to bf16 between them are independent."""
    e = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert e <= tol, (what, e)


@pytest.mark.parametrize("kind", ["softmax", "linear"])
def test_training_step_from_the_projection_and_back(kind):
    """A fused projection through norm, rotation and the zigzag order into attention, and its
    gradient back to the projection and the norms' weights, against float64 autograd.
    Tolerance: q, k and the gradients between the kernels are rounded to bf16 (2^-8 each at most,
    uniform: 2^-8 / sqrt(3) of the norm), through at most six such roundings and attention's own
    three: 2^-8 / sqrt(3) * 3 = 2^-7.2; twice that."""
    cp = cp_mod()
    rng = np.random.default_rng(11)
    B, Hq, Hkv, T, D, ranks = 1, 4, 2, 512, 64, 2
    W = Hq + 2 * Hkv
    x, _ = draw(rng, (B, T, W, D), "bf16")
    wq, wk = (draw(rng, (D,), "bf16", 0.2)[0] + 1 for _ in range(2))
    f = 10000.0 ** (-2 * np.arange(D // 2) / D)
    do, _ = draw(rng, (B, Hq, T, D), "bf16")           # natural order
    pos = positions(T, ranks, "zigzag")
    ld = spread_decays(Hq)

    # float64
    X = x.double().cpu().requires_grad_()
    WQ, WK = (w.double().cpu().requires_grad_() for w in (wq, wk))
    heads = X.transpose(1, 2)
    ang = torch.arange(T, dtype=torch.float64)[:, None] * torch.from_numpy(f)
    cos, sin = torch.cos(ang), torch.sin(ang)

    def prep(h, w):
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * w
        a, b = h[..., :D // 2], h[..., D // 2:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)

    Q, K = prep(heads[:, :Hq], WQ), prep(heads[:, Hq:Hq + Hkv], WK)
    V = heads[:, Hq + Hkv:]
    K, V = K.repeat_interleave(Hq // Hkv, 1), V.repeat_interleave(Hq // Hkv, 1)
    i = torch.arange(T)
    S = Q @ K.transpose(-1, -2) / D ** 0.5
    if kind == "softmax":
        P = torch.softmax(S.masked_fill(i[:, None] < i, float("-inf")), -1)
    else:
        e = (i[:, None] - i).clamp(min=0)
        P = S * torch.exp(torch.from_numpy(ld).double()[:, None, None] * e) * (i[:, None] >= i)
    O = P @ V
    O.backward(do.double().cpu())

    # the library
    rd = cp.make_rotate_desc(B, Hq, Hkv, T, D, cp=ranks, layout="zigzag", natural_in=1)
    split = lambda t: (t[:, :, :Hq].transpose(1, 2), t[:, :, Hq:Hq + Hkv].transpose(1, 2),  # noqa: E731
                       t[:, :, Hq + Hkv:].transpose(1, 2))
    q, k, v = (torch.empty(B, h, T, D, dtype=torch.bfloat16, device=dev()) for h in (Hq, Hkv, Hkv))
    fd = torch.from_numpy(f).to(dev())
    cp.check(cp.cpattn_rotate_fwd(rd, *split(x), wq, wk, fd, None, q, k, v))
    d = cp.make_desc(B, Hq, Hkv, T, D, ranks, "zigzag", "bf16")
    o, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))
    dol = do[:, :, torch.from_numpy(pos).to(dev())].contiguous()
    if kind == "softmax":
        lse = torch.empty(B, Hq, T, device=dev())
        ws = torch.empty(cp.cpattn_ring_bwd_workspace(d), dtype=torch.uint8, device=dev())
        cp.check(cp.cpattn_ring_fwd(d, q, k, v, o, lse))
        cp.check(cp.cpattn_ring_bwd(d, q, k, v, o, lse, dol, dq, dk, dv, ws))
    else:
        ldd = torch.from_numpy(ld).to(dev())
        ws = torch.empty(max(cp.cpattn_linear_workspace(d), cp.cpattn_linear_bwd_workspace(d)), dtype=torch.uint8,
                         device=dev())
        cp.check(cp.cpattn_linear_fwd(d, q, k, v, ldd, None, None, o, None, ws))
        cp.check(cp.cpattn_linear_bwd(d, q, k, v, ldd, None, dol, None, dq, dk, dv, None, ws))
    dx = torch.empty_like(x)
    dw = torch.empty(2, D, device=dev())
    ws = torch.empty(cp.cpattn_rotate_bwd_workspace(rd), dtype=torch.uint8, device=dev())
    xq, xk, _ = split(x)
    cp.check(cp.cpattn_rotate_bwd(rd, xq, xk, wq, wk, fd, None, dq, dk, dv, *split(dx), dw[0], dw[1], ws))
    cp.check(cp.cpattn_check())
    tol = 2.0 ** -6.2
    back = torch.from_numpy(np.argsort(pos)).to(dev())
    _close(f64(o[:, :, back]), O.detach().numpy(), tol, "o")
    _close(f64(dx), X.grad.numpy(), tol, "dx")
    _close(f64(dw[0]), WQ.grad.numpy(), tol, "dwq")
    _close(f64(dw[1]), WK.grad.numpy(), tol, "dwk")


def test_serving_prompts_then_tokens():
    """Padded prompts leave states; single tokens, rotated at their own positions, go on from them;
    a request ends and its slot is skipped.  Against the whole sequences in float64.
    Tolerance as above, of fewer roundings."""
    cp = cp_mod()
    rng = np.random.default_rng(12)
    B, H, G, T, D, new = 3, 4, 2, 300, 64, 5
    lengths = [300, 1, 177]
    f = 10000.0 ** (-2 * np.arange(D // 2) / D)
    fd = torch.from_numpy(f).to(dev())
    ld = spread_decays(H)
    ldd = torch.from_numpy(ld).to(dev())
    W = H + 2 * G
    x, x64 = draw(rng, (B, T + new, W, D), "bf16")   # row b: its prompt, padding, then its new tokens
    w, w64 = draw(rng, (D,), "bf16")
    split = lambda t: (t[:, :, :H].transpose(1, 2), t[:, :, H:H + G].transpose(1, 2), t[:, :, H + G:].transpose(1, 2))  # noqa: E731
    q, k, v = (torch.empty(B, h, T, D, dtype=torch.bfloat16, device=dev()) for h in (H, G, G))
    rd = cp.make_rotate_desc(B, H, G, T, D)
    cp.check(cp.cpattn_rotate_fwd(rd, *split(x[:, :T]), w, w, fd, None, q, k, v))
    d = cp.make_desc(B, H, G, T, D, 1, "contiguous", "bf16")
    n = torch.tensor(lengths, dtype=torch.int32, device=dev())
    o = torch.zeros_like(q)
    S = torch.zeros(B, H, D, D, device=dev())
    ws = torch.empty(cp.cpattn_linear_workspace(d), dtype=torch.uint8, device=dev())
    cp.check(cp.cpattn_linear_fwd(d, q, k, v, ldd, n, None, o, S, ws))
    rt = cp.make_rotate_desc(1, H, G, B, D)
    ds = cp.make_desc(B, H, G, 1, D, 1, "contiguous", "bf16")
    steps = torch.full((new, B, H, D), 7.0, dtype=torch.bfloat16, device=dev())
    slots = torch.arange(B, dtype=torch.int32, device=dev())
    for t in range(new):
        if t == 3:
            slots[1] = -1                           # the second request is over
        tok = x[:, T + t].contiguous()
        h = lambda a, b: tok[:, a:b].transpose(0, 1).unsqueeze(0)  # noqa: E731
        pos = (n + t).view(1, B)
        cp.check(cp.cpattn_rotate_fwd(rt, h(0, H), h(H, H + G), None, w, w, fd, pos, h(0, H), h(H, H + G), None))
        cp.check(cp.cpattn_linear_step(ds, tok[:, :H], tok[:, H:H + G], tok[:, H + G:], ldd, slots, S, S, steps[t]))
    cp.check(cp.cpattn_check())
    for b in range(B):
        rows = np.concatenate([x64[b, :lengths[b]], x64[b, T:]]).transpose(1, 0, 2)[None]
        m = rows.shape[2]
        qq = L.rotate_fwd(rows[:, :H], w64, 1e-6, np.arange(m), f, D, "halves")
        kk = L.rotate_fwd(rows[:, H:H + G], w64, 1e-6, np.arange(m), f, D, "halves")
        ref, _ = L.linear_fwd(qq, kk, rows[:, H + G:], ld, float(d.scale))
        _close(f64(o[b, :, :lengths[b]]), ref[0, :, :lengths[b]], 2.0 ** -6.7, "prompt")
        live = new if b != 1 else 3
        _close(f64(steps[:live, b]), ref[0, :, lengths[b]:lengths[b] + live].transpose(1, 0, 2), 2.0 ** -6.7, "tokens")
    assert bool((steps[3:, 1] == 7).all())


def test_rotated_tokens_into_the_cache():
    """A decoding step's rotated keys and values go into the paged cache as they lie."""
    cp = cp_mod()
    rng = np.random.default_rng(13)
    n, Hq, Hkv, D = 21, 4, 2, 64
    x, _ = draw(rng, (n, Hq + 2 * Hkv, D), "bf16")
    d = cp.make_rotate_desc(1, Hq, Hkv, n, D, norm=0)
    f = torch.from_numpy(100.0 ** (-np.arange(32) / 32)).to(dev())
    pos = torch.arange(n, dtype=torch.int32, device=dev()).flip(0).contiguous().view(1, n)
    h = lambda a, b: x[:, a:b].transpose(0, 1).unsqueeze(0)  # noqa: E731
    cp.check(cp.cpattn_rotate_fwd(d, h(0, Hq), h(Hq, Hq + Hkv), None, None, None, f, pos, h(0, Hq), h(Hq, Hq + Hkv), None))
    cd = cp.make_cache_desc(Hq, Hkv, D, 16, 4)
    slots = torch.randperm(64, device=dev())[:n].int()
    caches = [torch.zeros(cp.cpattn_cache_bytes(cd), dtype=torch.uint8, device=dev()) for _ in range(2)]
    k, v = x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    cp.check(cp.cpattn_cache_append(cd, n, k, v, slots, caches[0]))
    cp.check(cp.cpattn_cache_append(cd, n, k.contiguous(), v.contiguous(), slots, caches[1]))
    cp.check(cp.cpattn_check())
    assert torch.equal(*caches) and bool(caches[0].any())
