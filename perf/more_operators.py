"""Workloads of what stands around attention in a layer, and of the attention whose memory
does not grow with the sequence:

  rotate       queries and keys of a fused projection: RMS norm of each head, rotation by
               position, and the move into the attention's token order, values along
               (cpattn_rotate_fwd)
  rotate_bwd   its gradients: of the projection's output and of the norms' weights
               (cpattn_rotate_bwd)
  linear       linear attention with a decay for each head, whole sequences
               (cpattn_linear_fwd)
  linear_bwd   its gradients (cpattn_linear_bwd)
  step         one token of many requests over their states (cpattn_linear_step)

Every case runs either in plain form (elementary torch operations) or, with ``own`` set,
through the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
THETA = 1e6
CHUNK = 128   # tokens that the plain form of linear attention takes at a time
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a busy server: 64 tokens, each at a position of its own
        {"name": "rotate_decode_64", "op": "rotate", "B": 1, "T": 64, "H_q": 32, "H_kv": 4, "D": 128,
         "cp": 1, "layout": "contiguous", "dtype": "bf16", "rot": 128, "pairing": "halves",
         "norm": True, "served": True},
        # a long prompt's fused projection on its way into the ring, zigzag over four ranks
        {"name": "rotate_prompt_32768", "op": "rotate", "B": 1, "T": 32768, "H_q": 32, "H_kv": 4,
         "D": 128, "cp": 4, "layout": "zigzag", "dtype": "bf16", "rot": 128, "pairing": "halves",
         "norm": True, "served": False},
        # a training step's gradients on their way back to the projection
        {"name": "rotate_bwd_8192", "op": "rotate_bwd", "B": 1, "T": 8192, "H_q": 32, "H_kv": 8,
         "D": 128, "cp": 8, "layout": "zigzag", "dtype": "bf16", "rot": 128, "pairing": "halves",
         "norm": True, "served": False},
        # the same of a small float32 model, an odd length, half of the channels rotated
        {"name": "rotate_bwd_f32_1021", "op": "rotate_bwd", "B": 3, "T": 1021, "H_q": 12, "H_kv": 12,
         "D": 64, "cp": 1, "layout": "contiguous", "dtype": "f32", "rot": 32, "pairing": "neighbours",
         "norm": True, "served": False},
        # a training step's forward pass, tokens in the ring's order
        {"name": "linear_8192", "op": "linear", "B": 1, "T": 8192, "H_q": 32, "H_kv": 32, "D": 128,
         "cp": 8, "layout": "zigzag", "dtype": "bf16", "ragged": False, "state": False},
        # prompts of different lengths, padded, one row unused, that go on from earlier states
        {"name": "linear_ragged_1021", "op": "linear", "B": 8, "T": 1021, "H_q": 12, "H_kv": 12,
         "D": 64, "cp": 1, "layout": "contiguous", "dtype": "bf16", "ragged": True, "state": True},
        # one very long prompt, few heads
        {"name": "linear_131072", "op": "linear", "B": 1, "T": 131072, "H_q": 8, "H_kv": 8, "D": 128,
         "cp": 1, "layout": "contiguous", "dtype": "bf16", "ragged": False, "state": True},
        # float32 all through
        {"name": "linear_f32_1500", "op": "linear", "B": 2, "T": 1500, "H_q": 8, "H_kv": 8, "D": 128,
         "cp": 1, "layout": "contiguous", "dtype": "f32", "ragged": False, "state": True},
        # a training step's backward pass, keys and values shared by four heads each
        {"name": "linear_bwd_8192", "op": "linear_bwd", "B": 1, "T": 8192, "H_q": 32, "H_kv": 8,
         "D": 128, "cp": 8, "layout": "zigzag", "dtype": "bf16", "ragged": False, "state": False},
        # the same of a small model, a batch
        {"name": "linear_bwd_4x1024", "op": "linear_bwd", "B": 4, "T": 1024, "H_q": 12, "H_kv": 12,
         "D": 64, "cp": 4, "layout": "zigzag", "dtype": "bf16", "ragged": False, "state": True},
        # one user: latency of a decoding step, heads as the one of the cache has them
        {"name": "step_1", "op": "step", "B": 1, "H_q": 32, "H_kv": 8, "D": 128, "dtype": "bf16"},
        # one decoding step of a busy server
        {"name": "step_128", "op": "step", "B": 128, "H_q": 32, "H_kv": 32, "D": 128, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above."""
    op = rng.choice(["rotate", "rotate_bwd", "linear", "linear", "linear_bwd", "step"])
    H_q, H_kv, D = rng.choice([(32, 32, 128), (32, 8, 128), (32, 4, 128), (8, 8, 128), (12, 12, 64),
                               (16, 2, 64)])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "step":
        return {"op": op, "B": _log_int(rng, 1, 128 * 32 * 16384 // (H_q * D * D)), "H_q": H_q,
                "H_kv": H_kv, "D": D, "dtype": dtype}
    cp, layout = rng.choice([(1, "contiguous"), (1, "contiguous"), (2, "zigzag"), (4, "contiguous"),
                             (4, "zigzag"), (8, "zigzag")])
    most = 8192 * 32 if op != "rotate" else 32768 * 32
    if dtype == "f32" and op in ("linear", "linear_bwd"):
        most //= 8
    B = rng.choice([1, 1, 2, 3, 8])
    T = _log_int(rng, 1, most // (B * H_q))
    if layout == "zigzag":
        T = max(1, T // (256 * cp)) * 256 * cp if rng.random() < 0.7 else max(1, T // (2 * cp)) * 2 * cp
        if T * B > most // H_q:
            B = 1
    else:
        T = max(1, T // cp) * cp
    c = {"op": op, "B": B, "T": T, "H_q": H_q, "H_kv": H_kv, "D": D, "cp": cp, "layout": layout,
         "dtype": dtype}
    if op in ("rotate", "rotate_bwd"):
        c.update(rot=rng.choice([D, D, D // 2, D // 4]), pairing=rng.choice(["halves", "neighbours"]),
                 norm=rng.random() < 0.7, served=False)
        if op == "rotate" and rng.random() < 0.3:
            c.update(B=1, T=min(T, 4096), cp=1, layout="contiguous", served=True)
    else:
        c.update(ragged=op == "linear" and layout == "contiguous" and T >= 8 and rng.random() < 0.4,
                 state=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(_DT[dtype])


def _lengths(c):
    """Tokens of every row of a padded batch; a batch's first row is unused."""
    return [int(c["T"] * ((i + (c["B"] == 1)) * 0.6180339887498949 % 1.0)) for i in range(c["B"])]


def _positions(T, cp, layout):
    """Natural position of every slot of the layout order."""
    p = torch.arange(T, device=DEV)
    if layout == "zigzag":
        parts = p.view(2 * cp, -1)
        p = torch.stack([parts[:cp], parts[cp:].flip(0)], 1).reshape(-1)
    return p


def _split(x, c):
    """Queries, keys and values of a fused projection [B, T, (H_q + 2 H_kv) D], as views
    [B, H, T, D]."""
    v = x.view(c["B"], c["T"], c["H_q"] + 2 * c["H_kv"], c["D"]).transpose(1, 2)
    return v[:, :c["H_q"]], v[:, c["H_q"]:c["H_q"] + c["H_kv"]], v[:, c["H_q"] + c["H_kv"]:]


def _decays(H):
    """log of the decay of every head: from a memory of a few tokens to one of hundreds."""
    return -torch.exp2(-8.0 * (torch.arange(H, device=DEV, dtype=torch.float64) + 1) / H).float()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": c}
    lib = None
    if own:
        import blockwise_online_softmax_cpattn_gb300 as lib
        st["lib"] = lib
    B, H_q, H_kv, D, dt = c["B"], c["H_q"], c["H_kv"], c["D"], c["dtype"]

    if c["op"] in ("rotate", "rotate_bwd"):
        T, W = c["T"], (H_q + 2 * H_kv) * D
        st["x"] = _normal(gen, (B, T, W), dt, 2.0)
        st["wq"] = 1 + _normal(gen, (D,), dt, 0.2) if c["norm"] else None
        st["wk"] = 1 + _normal(gen, (D,), dt, 0.2) if c["norm"] else None
        i = torch.arange(c["rot"] // 2, device=DEV, dtype=torch.float64)
        st["inv_freq"] = THETA ** (-2 * i / c["rot"])
        st["pos"] = None
        if c["served"]:
            st["pos"] = torch.randint(0, 131072, (B, T), generator=gen, device=DEV, dtype=torch.int32)
        if c["op"] == "rotate":
            if c["served"]:   # packed tokens, as the cache's calls take them
                st["out"] = [torch.zeros(B, T, h, D, dtype=_DT[dt], device=DEV).transpose(1, 2)
                             for h in (H_q, H_kv, H_kv)]
            else:
                st["out"] = [torch.zeros(B, h, T, D, dtype=_DT[dt], device=DEV)
                             for h in (H_q, H_kv, H_kv)]
        else:
            st["dy"] = [_normal(gen, (B, h, T, D), dt) for h in (H_q, H_kv, H_kv)]
            st["dx"] = torch.zeros(B, T, W, dtype=_DT[dt], device=DEV)
            st["dw"] = [torch.zeros(D, device=DEV) if c["norm"] else None for _ in range(2)]
        if own:
            st["desc"] = lib.make_rotate_desc(B, H_q, H_kv, T, D, cp=c["cp"], layout=c["layout"],
                                              dtype=dt, rot=c["rot"], pairing=c["pairing"],
                                              norm=int(c["norm"]), natural_in=1, eps=EPS)
            if c["op"] == "rotate_bwd":
                st["ws"] = torch.empty(lib.cpattn_rotate_bwd_workspace(st["desc"]),
                                       dtype=torch.uint8, device=DEV)
        return st

    st["ld"] = _decays(H_q)
    st["scale"] = 1.0 / math.sqrt(D)
    if c["op"] == "step":
        x = _normal(gen, (B, H_q + 2 * H_kv, D), dt)
        st["q"], st["k"], st["v"] = x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:]
        st["S"] = torch.randn((B, H_q, D, D), generator=gen, device=DEV)
        st["S_out"] = torch.zeros_like(st["S"])
        st["o"] = torch.zeros(B, H_q, D, dtype=_DT[dt], device=DEV)
        st["slots"] = torch.randperm(B, generator=gen, device=DEV).int()
        if own:
            st["desc"] = lib.make_desc(B, H_q, H_kv, 1, D, 1, "contiguous", dt)
        return st

    T = c["T"]
    st["q"] = _normal(gen, (B, H_q, T, D), dt)
    st["k"] = _normal(gen, (B, H_kv, T, D), dt)
    st["v"] = _normal(gen, (B, H_kv, T, D), dt)
    st["S0"] = torch.randn((B, H_q, D, D), generator=gen, device=DEV) if c["state"] else None
    if c["op"] == "linear":
        st["lengths"] = None
        if c["ragged"]:
            st["rows"] = _lengths(c)   # the host of such a program knows them too
            st["lengths"] = torch.tensor(st["rows"], dtype=torch.int32, device=DEV)
        st["o"] = torch.zeros_like(st["q"])
        st["S1"] = torch.zeros(B, H_q, D, D, device=DEV) if c["state"] else None
    else:
        st["do"] = _normal(gen, (B, H_q, T, D), dt)
        st["dS1"] = torch.randn((B, H_q, D, D), generator=gen, device=DEV) if c["state"] else None
        st["dS0"] = torch.zeros(B, H_q, D, D, device=DEV) if c["state"] else None
        st["dq"], st["dk"], st["dv"] = (torch.zeros_like(st[n]) for n in ("q", "k", "v"))
    if own:
        st["desc"] = lib.make_desc(B, H_q, H_kv, T, D, c["cp"], c["layout"], dt)
        size = (lib.cpattn_linear_workspace if c["op"] == "linear" else
                lib.cpattn_linear_bwd_workspace)(st["desc"])
        st["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rotate": _own_rotate, "rotate_bwd": _own_rotate_bwd, "linear": _own_linear,
                "linear_bwd": _own_linear_bwd, "step": _own_step}[op](state)
    return {"rotate": _plain_rotate, "rotate_bwd": _plain_rotate_bwd, "linear": _plain_linear,
            "linear_bwd": _plain_linear_bwd, "step": _plain_step}[op](state)


def _own_rotate(s):
    lib, (q, k, v), out = s["lib"], _split(s["x"], s["case"]), s["out"]
    lib.check(lib.cpattn_rotate_fwd(s["desc"], q, k, v, s["wq"], s["wk"], s["inv_freq"], s["pos"],
                                    out[0], out[1], out[2]))
    return tuple(out)


def _own_rotate_bwd(s):
    lib, c = s["lib"], s["case"]
    q, k, _ = _split(s["x"], c)
    dq, dk, dv = _split(s["dx"], c)
    lib.check(lib.cpattn_rotate_bwd(s["desc"], q, k, s["wq"], s["wk"], s["inv_freq"], s["pos"],
                                    *s["dy"], dq, dk, dv, s["dw"][0], s["dw"][1], s["ws"]))
    return (s["dx"], *s["dw"]) if c["norm"] else s["dx"]


def _own_linear(s):
    lib = s["lib"]
    lib.check(lib.cpattn_linear_fwd(s["desc"], s["q"], s["k"], s["v"], s["ld"], s["lengths"], s["S0"],
                                    s["o"], s["S1"], s["ws"]))
    return (s["o"], s["S1"]) if s["case"]["state"] else s["o"]


def _own_linear_bwd(s):
    lib = s["lib"]
    lib.check(lib.cpattn_linear_bwd(s["desc"], s["q"], s["k"], s["v"], s["ld"], s["S0"], s["do"],
                                    s["dS1"], s["dq"], s["dk"], s["dv"], s["dS0"], s["ws"]))
    out = (s["dq"], s["dk"], s["dv"])
    return out + (s["dS0"],) if s["case"]["state"] else out


def _own_step(s):
    lib = s["lib"]
    lib.check(lib.cpattn_linear_step(s["desc"], s["q"], s["k"], s["v"], s["ld"], s["slots"], s["S"],
                                     s["S_out"], s["o"]))
    return s["o"], s["S_out"]


# -- plain forms -------------------------------------------------------------
def _cos_sin(s):
    """[B or 1, T, rot / 2] for the slots of the attention's order; angles in 64 bits."""
    c = s["case"]
    p = s["pos"] if s["pos"] is not None else _positions(c["T"], c["cp"], c["layout"])[None]
    a = p.double()[..., None] * s["inv_freq"]
    return torch.cos(a).float(), torch.sin(a).float()


def _turn(x, cos, sin, c):
    """Rotates the first rot channels of [B, H, T, D]."""
    r, half = c["rot"], c["rot"] // 2
    cos, sin = cos[:, None], sin[:, None]
    y = x.clone()
    if c["pairing"] == "halves":
        a, b = x[..., :half], x[..., half:r]
        y[..., :half], y[..., half:r] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    return y


def _plain_rotate(s):
    c = s["case"]
    order = _positions(c["T"], c["cp"], c["layout"])
    cos, sin = _cos_sin(s)
    out = []
    for x, w in zip(_split(s["x"], c), (s["wq"], s["wk"], None)):
        x = x[:, :, order]
        if len(out) < 2:
            x = x.float()
            if c["norm"]:
                x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
            x = _turn(x, cos, sin, c)
        out.append(x.to(_DT[c["dtype"]]))
    return tuple(out)


def _plain_rotate_bwd(s):
    c = s["case"]
    order = _positions(c["T"], c["cp"], c["layout"])
    cos, sin = _cos_sin(s)
    dx = torch.empty_like(s["x"])
    dws = []
    for x, d, dy, w in zip(_split(s["x"], c), _split(dx, c), s["dy"], (s["wq"], s["wk"], None)):
        g = dy.float()
        if len(dws) < 2:
            g = _turn(g, cos, -sin, c)
            dw = None
            if c["norm"]:
                x = x[:, :, order].float()
                r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
                n = x * r
                dw = (g * n).sum((0, 1, 2))
                h = g * w.float()
                g = r * (h - n * (h * n).mean(-1, keepdim=True))
            dws.append(dw)
        d[:, :, order] = g.to(d.dtype)
    return (dx, *dws) if c["norm"] else dx


def _powers(ld, n):
    """decay ** e for e = 0 .. n, [H, n + 1]."""
    return torch.exp(ld.double()[:, None] * torch.arange(n + 1, device=DEV, dtype=torch.float64)).float()


def _mix(a, b, c, ld, M, late):
    """out_r = sum over s <= r of decay^(r-s) (a_r . b_s) c_s, with what went before in M
    [B, H, D, D]; [B, H, T, D] float32.  Also returns M behind the last token.  late: M counts
    from the first token itself, not from the one before it."""
    B, H, T, D = a.shape
    n = -(-T // CHUNK)
    pad = n * CHUNK - T
    a, b, c = (torch.nn.functional.pad(x, (0, 0, 0, pad)).view(B, H, n, CHUNK, D) for x in (a, b, c))
    p = _powers(ld, CHUNK + 1)
    i = torch.arange(CHUNK, device=DEV)
    e = i[:, None] - i[None]
    w = torch.where(e >= 0, p[:, e.clamp(min=0)], torch.zeros((), device=DEV))
    out = ((a @ b.transpose(-1, -2)) * w[None, :, None]) @ c
    late = int(late)
    U = (b * p[:, CHUNK - 1 - i + late][None, :, None, :, None]).transpose(-1, -2) @ c
    if pad:
        last = CHUNK - pad
        e = (last - 1 - i + late).clamp(min=0)
        U[:, :, -1] = (b[:, :, -1] * p[:, e][None, ..., None]).transpose(-1, -2) @ c[:, :, -1]
    M = torch.zeros(B, H, D, D, device=DEV) if M is None else M
    before = []
    for k in range(n):
        before.append(M)
        M = p[:, CHUNK - pad if k == n - 1 else CHUNK][None, :, None, None] * M + U[:, :, k]
    before = torch.stack(before, 2)
    out += p[:, i + 1 - late][None, :, None, :, None] * (a @ before)
    return out.view(B, H, n * CHUNK, D)[:, :, :T], M


def _shared(x, H_q):
    return x.float().repeat_interleave(H_q // x.shape[1], 1)


def _plain_linear(s):
    c = s["case"]
    H, T = c["H_q"], c["T"]
    order = _positions(T, c["cp"], c["layout"])
    back = torch.argsort(order)
    q, k, v = (_shared(s[n][:, :, back], H) for n in ("q", "k", "v"))
    if not c["ragged"]:
        o, S1 = _mix(q, k, v, s["ld"], s["S0"], False)
        o = (o * s["scale"])[:, :, order].to(_DT[c["dtype"]])
        return (o, S1) if c["state"] else o
    o = torch.zeros_like(s["q"])
    S1 = []
    for b, n in enumerate(s["rows"]):
        S = s["S0"][b:b + 1] if c["state"] else torch.zeros(1, H, c["D"], c["D"], device=DEV)
        if n:
            x, S = _mix(q[b:b + 1, :, :n], k[b:b + 1, :, :n], v[b:b + 1, :, :n], s["ld"], S, False)
            o[b, :, :n] = (x[0] * s["scale"]).to(o.dtype)
        S1.append(S)
    return (o, torch.cat(S1)) if c["state"] else o


def _plain_linear_bwd(s):
    c = s["case"]
    H, G, sc = c["H_q"], c["H_kv"], s["scale"]
    order = _positions(c["T"], c["cp"], c["layout"])
    back = torch.argsort(order)
    q, k, v, do = (_shared(s[n][:, :, back], H) for n in ("q", "k", "v", "do"))
    S0 = s["S0"].transpose(-1, -2) if c["state"] else None
    dq, _ = _mix(do, v, k, s["ld"], S0, False)
    q, k, v, do = (x.flip(2) for x in (q, k, v, do))
    R = s["dS1"] / sc if c["state"] else None
    dv, R0 = _mix(k, q, do, s["ld"], R, True)
    dk, _ = _mix(v, do, q, s["ld"], R.transpose(-1, -2) if c["state"] else None, True)
    out = []
    for x in (dq, dk.flip(2), dv.flip(2)):
        x = x * sc
        if out:
            x = x.view(c["B"], G, H // G, c["T"], c["D"]).sum(2)
        out.append(x[:, :, order].to(_DT[c["dtype"]]))
    return tuple(out) + (R0 * sc,) if c["state"] else tuple(out)


def _plain_step(s):
    c = s["case"]
    H = c["H_q"]
    q, k, v = (_shared(s[n], H) for n in ("q", "k", "v"))
    rows = s["slots"].long()
    S = _powers(s["ld"], 1)[:, 1][None, :, None, None] * s["S"][rows] + k[..., None] * v[..., None, :]
    o = (q[..., None] * S).sum(2) * s["scale"]
    S_out = torch.empty_like(S)
    S_out[rows] = S
    return o.to(_DT[c["dtype"]]), S_out


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    c = case
    B, H_q, H_kv, D = c["B"], c["H_q"], c["H_kv"], c["D"]
    elt = 2 if c["dtype"] == "bf16" else 4
    T = c.get("T", 1)
    rows, rows_kv = B * H_q * T, B * H_kv * T
    if c["op"] in ("rotate", "rotate_bwd"):
        moved = 2 if c["op"] == "rotate" else (3 if c["norm"] else 2)
        return {"bytes": elt * D * ((rows + rows_kv) * moved + 2 * rows_kv),
                "flops": (rows + rows_kv) * D * (8 if c["op"] == "rotate" else 16)}
    states = 4 * B * H_q * D * D
    if c["op"] == "step":
        return {"bytes": 2 * states + elt * D * (2 * rows + 2 * rows_kv), "flops": 5 * B * H_q * D * D}
    if c["op"] == "linear":
        if c["ragged"]:
            n = sum(_lengths(c))
            rows, rows_kv = H_q * n, H_kv * n
        return {"bytes": elt * D * (2 * rows + 2 * rows_kv) + (2 * states if c["state"] else 0),
                "flops": 4 * D * D * rows}
    return {"bytes": elt * D * (3 * rows + 4 * rows_kv) + (3 * states if c["state"] else 0),
            "flops": 10 * D * D * rows}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
BLOCK = 96   # tokens at a time; another cut than the plain form's


def _exact_rotation(s, x, inverse):
    """x [B, H, T, D] in the attention's order, as complex numbers times e^(i angle)."""
    c = s["case"]
    r = c["rot"]
    if s["pos"] is not None:
        p = s["pos"].double()
    else:
        p = torch.empty(c["T"], dtype=torch.float64, device=DEV)
        T, cp = c["T"], c["cp"]
        for rank in range(cp):
            n = T // cp
            if c["layout"] == "contiguous":
                p[rank * n:(rank + 1) * n] = torch.arange(rank * n, (rank + 1) * n, device=DEV)
            else:
                h = n // 2
                late = (2 * cp - 1 - rank) * h
                p[rank * n:rank * n + h] = torch.arange(rank * h, (rank + 1) * h, device=DEV)
                p[rank * n + h:(rank + 1) * n] = torch.arange(late, late + h, device=DEV)
        p = p[None]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       p[:, None, :, None] * s["inv_freq"] * (-1 if inverse else 1))
    head = x[..., :r]
    if c["pairing"] == "halves":
        z = torch.complex(head[..., :r // 2].contiguous(), head[..., r // 2:].contiguous()) * turn
        head = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(head.reshape(*head.shape[:-1], r // 2, 2).contiguous()) * turn
        head = torch.view_as_real(z).flatten(-2)
    return torch.cat([head, x[..., r:]], -1)


def _natural(c):
    """Slots of the layout order, by natural position."""
    T, cp = c["T"], c["cp"]
    if c["layout"] == "contiguous":
        return list(range(T))
    h = T // (2 * cp)
    slots = []
    for chunk in range(2 * cp):
        first = 2 * chunk * h if chunk < cp else (2 * (2 * cp - 1 - chunk) + 1) * h
        slots += range(first, first + h)
    return slots


def _exact_rotate(s):
    c = s["case"]
    slots = torch.tensor(_natural(c), device=DEV)
    xs = []
    for j, x in enumerate(_split(s["x"].double(), c)):
        y = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        y[:, :, slots] = x
        if j < 2:
            if c["norm"]:
                w = (s["wq"] if j == 0 else s["wk"]).double()
                y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS) * w
            y = _exact_rotation(s, y, False)
        xs.append(y)
    return tuple(xs)


def _exact_rotate_bwd(s):
    c = s["case"]
    slots = torch.tensor(_natural(c), device=DEV)
    dx, dws = [], []
    for j, x in enumerate(_split(s["x"].double(), c)):
        g = s["dy"][j].double()
        if j < 2:
            g = _exact_rotation(s, g, True)[:, :, slots]
            if c["norm"]:
                w = (s["wq"] if j == 0 else s["wk"]).double()
                ms = x.square().mean(-1, keepdim=True) + EPS
                dws.append((g * x / ms.sqrt()).sum((0, 1, 2)))
                g = g * w
                g = g / ms.sqrt() - x * (g * x).mean(-1, keepdim=True) / ms ** 1.5
        else:
            g = g[:, :, slots]
        dx.append(g)
    dx = torch.cat(dx, 1).transpose(1, 2).flatten(2)
    return (dx, *dws) if c["norm"] else dx


def _exact_pass(s, q, k, v, S, do=None):
    """The recurrence over [H, T, D] of one batch row, in blocks; with do given, the states
    behind every block's start come back instead of the outputs."""
    ld = s["ld"].double()[:, None, None]
    T = q.shape[1]
    outs, states = [], []
    for t in range(0, T, BLOCK):
        n = min(BLOCK, T - t)
        states.append(S)
        i = torch.arange(n, device=DEV, dtype=torch.float64)
        w = torch.exp(ld * (i[:, None] - i).clamp(min=0)).tril()
        qb, kb, vb = q[:, t:t + n], k[:, t:t + n], v[:, t:t + n]
        if do is None:
            seen = torch.einsum("hid,hjd->hij", qb, kb) * w
            outs.append(s["scale"] * (torch.einsum("hij,hjd->hid", seen, vb)
                                      + torch.exp(ld * (i[:, None] + 1)) * torch.einsum("hid,hde->hie", qb, S)))
        S = torch.exp(ld * n) * S + torch.einsum("hjd,hje->hde", kb * torch.exp(ld * (n - 1 - i[:, None])), vb)
    return (torch.cat(outs, 1) if do is None else states), S


def _exact_linear(s, b, n, slots):
    c = s["case"]
    H, D = c["H_q"], c["D"]
    q, k, v = (s[m][b].double()[:, slots[:n]].repeat_interleave(H // s[m].shape[1], 0) for m in "qkv")
    S = s["S0"][b].double() if c["state"] else torch.zeros(H, D, D, dtype=torch.float64, device=DEV)
    o = torch.zeros(H, c["T"], D, dtype=torch.float64, device=DEV)
    if n:
        x, S = _exact_pass(s, q, k, v, S)
        o[:, slots[:n]] = x
    return o, S


def _exact_linear_bwd(s, b, slots):
    c = s["case"]
    H, G, D, T = c["H_q"], c["H_kv"], c["D"], c["T"]
    q, k, v, do = (s[m][b].double()[:, slots].repeat_interleave(H // s[m].shape[1], 0)
                   for m in ("q", "k", "v", "do"))
    zero = torch.zeros(H, D, D, dtype=torch.float64, device=DEV)
    states, _ = _exact_pass(s, q, k, v, s["S0"][b].double() if c["state"] else zero, do)
    dS = s["dS1"][b].double() if c["state"] else zero
    do = do * s["scale"]
    ld = s["ld"].double()[:, None, None]
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    for blk in reversed(range(len(states))):
        t = blk * BLOCK
        n = min(BLOCK, T - t)
        i = torch.arange(n, device=DEV, dtype=torch.float64)
        w = torch.exp(ld * (i[:, None] - i).clamp(min=0)).tril()
        at, S = slice(t, t + n), states[blk]
        since, left = torch.exp(ld * (i[:, None] + 1)), torch.exp(ld * (n - 1 - i[:, None]))
        p = (q[:, at] @ k[:, at].mT) * w
        dp = (do[:, at] @ v[:, at].mT) * w
        dq[:, at] = dp @ k[:, at] + since * (do[:, at] @ S.mT)
        dk[:, at] = dp.mT @ q[:, at] + left * (v[:, at] @ dS.mT)
        dv[:, at] = p.mT @ do[:, at] + left * (k[:, at] @ dS)
        dS = torch.exp(ld * n) * dS + (q[:, at] * since).mT @ do[:, at]
    out = []
    for x, heads in ((dq, H), (dk, G), (dv, G)):
        y = torch.empty(heads, T, D, dtype=torch.float64, device=DEV)
        y[:, slots] = x.view(heads, H // heads, T, D).sum(1)
        out.append(y)
    return out + ([dS] if c["state"] else [])


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rotate":
        return _exact_rotate(s)
    if c["op"] == "rotate_bwd":
        return _exact_rotate_bwd(s)
    if c["op"] == "step":
        rows = s["slots"].long()
        rep = c["H_q"] // c["H_kv"]
        q, k, v = (s[n].double() for n in "qkv")
        o = torch.empty(q.shape, dtype=torch.float64, device=DEV)
        S_out = torch.empty(s["S"].shape, dtype=torch.float64, device=DEV)
        for h in range(c["H_q"]):
            S = torch.exp(s["ld"][h].double()) * s["S"][rows, h].double()
            S += torch.einsum("bd,be->bde", k[:, h // rep], v[:, h // rep])
            o[:, h] = s["scale"] * torch.einsum("bd,bde->be", q[:, h], S)
            S_out[rows, h] = S
        return o, S_out
    slots = torch.tensor(_natural(c), device=DEV)
    if c["op"] == "linear":
        parts = [_exact_linear(s, b, s["rows"][b] if c["ragged"] else c["T"], slots)
                 for b in range(c["B"])]
    else:
        parts = [_exact_linear_bwd(s, b, slots) for b in range(c["B"])]
    out = tuple(torch.stack(x) for x in zip(*parts))
    return out if c["state"] or c["op"] == "linear_bwd" else out[0]
