"""GPU: norm, rotation and linear attention at the edges of what their documentation promises.
Tolerances are derived beside each test (half a step of a rounding: bf16 2^-8, float32 2^-24)."""
import numpy as np
import pytest
import torch

from gpu_helpers import cp_mod, dev
from oracle import layer as L
from test_gpu_layer import LinearCase, checked, draw, f64, pair_sum, rotation_case, spread_decays, within

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# padding
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_padding_never_shows(D, state):
    """What lies behind a row's end, zeros or NaN and infinities, changes no bit: many heads, each
    in several runs, rows that end at every remainder of eight inside a run that others start from."""
    cp = cp_mod()
    B, Hq, T = 18, 4, 1200
    d = cp.make_desc(B, Hq, Hq, T, D, 1, "contiguous", "bf16")
    # the runs' sums are in the workspace: there is more than one run
    assert cp.cpattn_linear_workspace(d) > 2 * 4 * B * Hq * D * D
    ends = [1, 2, 3, 4, 5, 6, 7, 60, 61, 100, 121, 127, 129, 252, 333, 500, 636, 1199]
    gen = torch.Generator(dev()).manual_seed(1)
    x = [torch.randn(B, Hq, T, D, device=dev(), generator=gen).bfloat16() for _ in range(3)]
    ld = torch.from_numpy(spread_decays(Hq)).to(dev())
    lengths = torch.tensor(ends, dtype=torch.int32, device=dev())
    ws = torch.empty(cp.cpattn_linear_workspace(d), dtype=torch.uint8, device=dev())
    tails = [torch.arange(T, device=dev()) >= n for n in ends]

    def run(fills):
        for t, fill in zip(x, fills):
            for b, tail in enumerate(tails):
                t[b, :, tail] = fill
        o = torch.zeros_like(x[0])
        S = torch.zeros(B, Hq, D, D, device=dev()) if state else None
        checked(cp, cp.cpattn_linear_fwd(d, *x, ld, lengths, None, o, S, ws))
        return o, S

    ref, S0 = run((0.0, 0.0, 0.0))
    assert ref.isfinite().all()
    nan, inf = float("nan"), float("inf")
    for fills in ((nan, nan, nan), (nan, inf, -inf), (inf, nan, 1e38)) * 8:
        o, S = run(fills)
        assert torch.equal(o, ref)
        if state:
            assert torch.equal(S, S0)


# ---------------------------------------------------------------------------
# angles
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("pairing", ["halves", "neighbours"])
def test_angles_and_their_turns(pairing):
    """Cosines and sines themselves, forward and backward: rows whose pairs are (1, 0) and (0, 1).

    The angle is off by less than 2^-25 and sincospif by a unit in the last place (2^-23 of the
    value); the products with 1 and 0 are exact.  The oracle's own angle in float64, below 2^18, is off
    by 2^-35.  Angles near every quarter turn are among them, where one of the two is small."""
    cp = cp_mod()
    T, D, half = 1024, 64, 32
    rng = np.random.default_rng(2)
    near = np.concatenate([2 ** -np.arange(0.0, 16.0), 1.9999999 * rng.random(half - 16)])
    f = np.where(near > 0, near, 1.0)
    # the first positions: those whose angle at f = 1 is nearest to a quarter turn's multiple
    p = np.arange(1, 131072)
    off = np.abs(p / (np.pi / 2) - np.round(p / (np.pi / 2)))
    pos = np.concatenate([p[np.argsort(off)[:T // 2]], rng.integers(-131072, 131072, T - T // 2 - 2), [0, -1]])
    first = np.zeros(D)
    first[:half if pairing == "halves" else D:1 if pairing == "halves" else 2] = 1
    x = torch.from_numpy(np.stack([first, 1 - first])).float().to(dev())[None, :, None].expand(1, 2, T, D)
    d = cp.make_rotate_desc(1, 2, 1, T, D, dtype="f32", pairing=pairing, norm=0)
    q, k = x.contiguous(), x[:, :1].contiguous()
    inv_freq, p_dev = torch.from_numpy(f).to(dev()), torch.from_numpy(pos.astype(np.int32))[None].to(dev())
    t = pos[:, None] * f
    c, s = np.cos(t), np.sin(t)

    def compare(got, s):
        got = got.double().cpu().numpy()[0]
        a, b = (slice(0, half), slice(half, D)) if pairing == "halves" else (slice(0, D, 2), slice(1, D, 2))
        for have, want, slope in ((got[0][:, a], c, s), (got[0][:, b], s, c), (got[1][:, a], -s, c), (got[1][:, b], c, s)):
            err = np.abs(have - want)
            bound = 2.0 ** -25 * np.abs(slope) + 2.0 ** -23 * np.abs(want) + 2.0 ** -34
            assert (err <= bound).all(), (err / bound).max()

    qo, ko = torch.empty_like(q), torch.empty_like(k)
    checked(cp, cp.cpattn_rotate_fwd(d, q, k, None, None, None, inv_freq, p_dev, qo, ko, None))
    compare(qo, s)
    ws = torch.empty(cp.cpattn_rotate_bwd_workspace(d), dtype=torch.uint8, device=dev())
    checked(cp, cp.cpattn_rotate_bwd(d, None, None, None, None, inv_freq, p_dev, q, k, None, qo, ko, None, None, None, ws))
    compare(qo, -s)


# ---------------------------------------------------------------------------
# long sums
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sums_over_long_runs_off_the_tensor_cores(dtype):
    """One run of 65536 tokens that add up without decay, each the same: the errors of a single
    accumulator all point one way (up to 1e-3 of the sum).

    A chunk's sum has 64 terms, a run's one a chunk, each rounded once: (64 + T / 64) 2^-24 of the
    sum; an output is a product over D channels of it and two of at most max(D, 64) terms, its
    weights and the scale.  All terms are positive, so this is relative to the values."""
    cp = cp_mod()
    H, T, D = 152, 65536, 8
    d = cp.make_desc(1, H, H, T, D, 1, "contiguous", dtype)
    assert cp.cpattn_linear_workspace(d) == cp.cpattn_linear_bwd_workspace(d) == 16  # one run a head
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    half = 2.0 ** -24 if dtype == "f32" else 2.0 ** -8
    gen = torch.Generator().manual_seed(5)
    rows = [(0.5 + torch.rand(H, D, generator=gen)).to(dt) for _ in range(4)]
    q, k, v, do = (x.to(dev())[None, :, None].expand(1, H, T, D).contiguous() for x in rows)
    ld = torch.zeros(H, device=dev())
    o, dq, dk, dv = (torch.empty_like(q) for _ in range(4))
    S, dS = (torch.empty(1, H, D, D, device=dev()) for _ in range(2))
    ws = torch.empty(16, dtype=torch.uint8, device=dev())
    checked(cp, cp.cpattn_linear_fwd(d, q, k, v, ld, None, None, o, S, ws))
    checked(cp, cp.cpattn_linear_bwd(d, q, k, v, ld, None, do, None, dq, dk, dv, dS, ws))
    q, k, v, do = (x.double() for x in rows)
    scale, sums = float(d.scale), (64 + T / 64) * 2.0 ** -24
    outs = sums + (D + 2 * 64 + 8) * 2.0 ** -24 + half

    def close(got, ref, tol):
        err = (got.double().cpu() / ref - 1).abs().max().item()
        assert err <= tol, (err, tol)

    kv, qdo = k[:, :, None] * v[:, None], q[:, :, None] * do[:, None]
    close(S[0], T * kv, sums + 2.0 ** -22)
    close(dS[0], scale * T * qdo, sums + 2.0 ** -22)
    t = torch.arange(T, dtype=torch.float64)[None, :, None]
    for h in range(0, H, 19):
        at = slice(h, h + 1)
        close(o[0, at], scale * (t + 1) * torch.einsum("hd,hde->he", q[at], kv[at])[:, None], outs)
        close(dq[0, at], scale * (t + 1) * torch.einsum("he,hde->hd", do[at], kv[at])[:, None], outs)
        close(dk[0, at], scale * (T - t) * torch.einsum("he,hde->hd", v[at], qdo[at])[:, None], outs)
        close(dv[0, at], scale * (T - t) * torch.einsum("hd,hde->he", k[at], qdo[at])[:, None], outs)


# ---------------------------------------------------------------------------
# roundings on the tensor cores, by norm
# ---------------------------------------------------------------------------
def by_chunks(a, b, c, ld, scale):
    """out_i = scale sum over j <= i of r^(i-j) (a_i . b_j) c_j in float64, and the sum of
    r^(T-1-j) b_j c_j^T, by chunks of 256 on the GPU."""
    B, H, T, D = a.shape
    out = torch.empty(B, H, T, D, dtype=torch.float64, device=a.device)
    S = torch.zeros(B, H, D, D, dtype=torch.float64, device=a.device)
    ld = ld.double()[:, None]
    for at in range(0, T, 256):
        x, y, z = (u[:, :, at:at + 256].double() for u in (a, b, c))
        n = x.shape[2]
        i = torch.arange(n, device=a.device, dtype=torch.float64)
        w = torch.exp(ld[:, :, None] * (i[:, None] - i).clamp(min=0)) * (i[:, None] >= i)
        out[:, :, at:at + n] = scale * ((x @ y.transpose(-1, -2) * w) @ z + torch.exp(ld * (i + 1))[..., None] * (x @ S))
        S = torch.exp(ld * n)[..., None] * S + (y * torch.exp(ld * (n - 1 - i))[..., None]).transpose(-1, -2) @ z
    return out, S


def off(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


@pytest.mark.parametrize("H,T,D", [(32, 2048, 128), (8, 8192, 128), (12, 4096, 64), (4, 2048, 64)])
@pytest.mark.parametrize("memory", [256, 16384])
def test_outputs_by_norm(H, T, D, memory):
    """Outputs and gradients of sequences in several runs, with memories short and long, with the
    states handed out and without.

    A rounding to bf16 is off by 2^-8 / sqrt(3) * sqrt(3 / 8 / ln 2) = 1.66e-3 of a number, root mean
    square.  An output has its own, and each term of its sum one more, of the weighted score or of
    the state as an operand, independent of each other: 1.66e-3 sqrt(2) = 2.35e-3 of the norm.  Keys in
    two numbers add 1e-5, keys in one up to another 1.66e-3: 2.87e-3 in all."""
    cp = cp_mod()
    d = cp.make_desc(1, H, H, T, D, 1, "contiguous", "bf16")
    assert cp.cpattn_linear_workspace(d) > 16  # runs
    gen = torch.Generator(dev()).manual_seed(3)
    q, k, v, do = (torch.randn(1, H, T, D, device=dev(), generator=gen).bfloat16() for _ in range(4))
    ld = -torch.logspace(0, -np.log10(memory), H, device=dev())
    ws = torch.empty(max(cp.cpattn_linear_workspace(d), cp.cpattn_linear_bwd_workspace(d)), dtype=torch.uint8, device=dev())
    flip = lambda x: x.flip(2)  # noqa: E731
    scale = float(d.scale)
    want = {"o": by_chunks(q, k, v, ld, scale)[0], "dq": by_chunks(do, v, k, ld, scale)[0],
            "dk": flip(by_chunks(flip(v), flip(do), flip(q), ld, scale)[0]),
            "dv": flip(by_chunks(flip(k), flip(q), flip(do), ld, scale)[0])}
    for state in (False, True):
        S, dS = (torch.empty(1, H, D, D, device=dev()) if state else None for _ in range(2))
        got = {n: torch.empty_like(q) for n in want}
        checked(cp, cp.cpattn_linear_fwd(d, q, k, v, ld, None, None, got["o"], S, ws))
        checked(cp, cp.cpattn_linear_bwd(d, q, k, v, ld, None, do, None, got["dq"], got["dk"], got["dv"], dS, ws))
        for n in want:
            assert off(got[n], want[n]) < 2.4e-3, (n, state, off(got[n], want[n]))


@pytest.mark.parametrize("H,T,D", [(32, 2048, 128), (12, 4096, 64), (152, 1024, 128), (152, 1000, 64), (3, 100, 128)])
def test_states_handed_out_by_norm(H, T, D):
    """state_out and dstate_in, from sequences in several runs and in one.

    Keys in two bf16 numbers would leave (1.66e-3)^2 = 2.7e-6 of each product, in three 5e-9.  What is
    left is float32's: a chunk's sum rounds 24 times (three parts of eight steps), the state once a chunk,
    and memories here span a few chunks; taken as 2^-23 each and half of them one way, 2e-7 to 4e-7."""
    cp = cp_mod()
    d = cp.make_desc(1, H, H, T, D, 1, "contiguous", "bf16")
    gen = torch.Generator(dev()).manual_seed(4)
    q, k, v, do = (torch.randn(1, H, T, D, device=dev(), generator=gen).bfloat16() for _ in range(4))
    ld = -torch.logspace(-0.5, -2.5, H, device=dev())
    ws = torch.empty(max(cp.cpattn_linear_workspace(d), cp.cpattn_linear_bwd_workspace(d)), dtype=torch.uint8, device=dev())
    S, dS = (torch.empty(1, H, D, D, device=dev()) for _ in range(2))
    o, dq, dk, dv = (torch.empty_like(q) for _ in range(4))
    checked(cp, cp.cpattn_linear_fwd(d, q, k, v, ld, None, None, o, S, ws))
    checked(cp, cp.cpattn_linear_bwd(d, q, k, v, ld, None, do, None, dq, dk, dv, dS, ws))
    assert off(S, by_chunks(q, k, v, ld, 1.0)[1]) < 5e-7
    # sum of r^(i+1) q_i dO_i^T: the state of the reversed sequence, decayed once more
    ref = by_chunks(q.flip(2), q.flip(2), do.flip(2), ld, 1.0)[1] * torch.exp(ld.double())[:, None, None]
    assert off(dS, float(d.scale) * ref) < 5e-7


# ---------------------------------------------------------------------------
# norm and rotation: many rows (eight pairs a lane in the backward pass, then in both)
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T,D,kw", [(1500, 128, {}), (2900, 128, {}), (2900, 128, {"pairing": "neighbours", "rot": 96}),
                                    (2900, 96, {"rot": 32}), (2900, 112, {"pairing": "neighbours", "rot": 16}),
                                    (2900, 128, {"norm": False, "rot": 64})])
def test_rotation_of_many_rows(T, D, kw):
    rotation_case(cp_mod(), 1, 40, 8, T, D, "bf16", seed=T + D, **kw)


@pytest.mark.parametrize("D", [128, 64])
def test_rotation_of_packed_tokens_in_float32(D):
    """A server's tokens in float32, [n, heads, D], each at its own position; output over input."""
    cp = cp_mod()
    rng = np.random.default_rng(6)
    n, Hq, Hkv = 45, 6, 2
    x, x64 = draw(rng, (n, Hq + 2 * Hkv, D), "f32")
    pos = rng.integers(0, 10 ** 6, (1, n)).astype(np.int32)
    f = 1e6 ** (-2 * np.arange(D // 2) / D)
    w, w64 = draw(rng, (D,), "f32")
    d = cp.make_rotate_desc(1, Hq, Hkv, n, D, dtype="f32")
    q, k, v = (x[:, a:b].transpose(0, 1).unsqueeze(0) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    checked(cp, cp.cpattn_rotate_fwd(d, q, k, v, w, w, torch.from_numpy(f).to(dev()), torch.from_numpy(pos).to(dev()),
                                     q, k, v))
    heads, got = x64.transpose(1, 0, 2)[None], f64(x).transpose(1, 0, 2)[None]
    turned = heads[:, :Hq + Hkv]
    ref = L.rotate_fwd(turned, w64, 1e-6, pos, f, D, "halves")
    # 2^-18 of the pair for the norm, the cosine and the sine (an angle off by 2^-25), and the rounding
    u = pair_sum(turned / np.sqrt((turned ** 2).mean(-1, keepdims=True) + 1e-6) * w64, D, "halves")
    within(got[:, :Hq + Hkv], ref, 2.0 ** -18 * u + 2.0 ** -24 * np.abs(ref))
    assert np.array_equal(got[:, Hq + Hkv:], heads[:, Hq + Hkv:])


# ---------------------------------------------------------------------------
# waits that run out, in the kernels of other sizes and orders
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,T,ranks,layout", [(64, 700, 1, "contiguous"), (128, 1200, 3, "zigzag"), (64, 528, 2, "zigzag")])
def test_timeouts_of_other_kernels(D, T, ranks, layout):
    """The first chunk's loads never count as done: the status says so, and the next call is right."""
    c = LinearCase(1, 2, 2, T, D, "bf16", ranks, layout)
    cp = c.cp
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
# gradients of padded rows
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 40)])
def test_gradients_of_padded_rows(dtype, D):
    """With dO = 0 behind the rows' ends and no dstate_out: the gradients of the rows cut there, and
    zeros behind."""
    T, ends = 700, [1, 130, 640, 700]
    c = LinearCase(len(ends), 2, 1, T, D, dtype)
    for b, n in enumerate(ends):
        c.do[0, b, :, n:] = 0
    outs = [torch.empty_like(x) for x in (c.q, c.k, c.v, c.S0)]
    ws = torch.empty(c.cp.cpattn_linear_bwd_workspace(c.d), dtype=torch.uint8, device=dev())
    c.dS1 = None
    c.backward(outs, ws)
    c.cp.check(c.cp.cpattn_check())
    got = [c.unshard(x) for x in outs[:3]] + [c.unshard(outs[3], False)]
    for b, n in enumerate(ends):
        cut = lambda x: x[b:b + 1, :, :n]  # noqa: E731
        q, k, v, do = map(cut, c.nat)
        S0 = c.states[0][b:b + 1]
        ref = L.linear_bwd(q, k, v, c.ld, c.scale, do, S0)
        A = L.linear_bwd(*map(np.abs, (q, k, v)), c.ld, c.scale, np.abs(do), np.abs(S0))
        for i, name in enumerate(("dq", "dk", "dv")):
            within(got[i][b:b + 1, :, :n], ref[i], c.bounds(ref[i], A[i], dtype), name)
            assert not got[i][b, :, n:].any()
        within(got[3][b:b + 1], ref[3], c.state_bounds(ref[3], A[3]), "dstate")
