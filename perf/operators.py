"""Workloads of the 4-bit key/value cache: its planning, its filling and reading, and
the attention of new tokens over it.

Every case runs either in plain form (elementary torch operations) or, with ``own``
set, through the library's calls:

  plan    request lengths -> pages taken and returned, block table, query offsets,
          slot of every new token (cpattn_cache_plan)
  append  key/value rows quantised into their slots and read back
          (cpattn_cache_append, cpattn_cache_read)
  attn    new tokens of many requests over their cached keys (cpattn_cache_attn)

A group of ``group`` channels of one token and K/V head is held as 4-bit codes c and
two bfloat16 numbers a, z; it stands for round_bf16(a * (1 + c / 16) + z).
"""
import math

import torch

own = False

DEV = "cuda"
TILE = 16   # tokens of a tile: the unit in which a page's rows are laid out
TINY = 2.0 ** -100   # a group whose a is below this is stored with a = 0
HUGE = 2.0 ** 120    # stored values are held within +- this


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decoding step of a busy server: every request grows by a token
        {"name": "plan_decode_64", "op": "plan", "requests": 64, "page": 64, "min_old": 1,
         "max_old": 8000, "max_new": 1, "ended": 0, "pages_left": 64},
        # a batch of prompts comes in while finished requests leave and drafts roll back
        {"name": "plan_prompts_700", "op": "plan", "requests": 700, "page": 16, "min_old": 0,
         "max_old": 4000, "max_new": 1000, "ended": 90, "pages_left": 16000},
        # the new keys and values of one decoding step, slices of a fused projection
        {"name": "append_decode_64", "op": "append", "tokens": 64, "H_q": 32, "H_kv": 8, "D": 128,
         "group": 64, "page": 64, "dtype": "bf16", "fused": True, "holes": 3},
        # a prompt's keys and values as the ring leaves them, [H, T, D]
        {"name": "append_prompt_32768", "op": "append", "tokens": 32768, "H_q": 32, "H_kv": 8,
         "D": 128, "group": 64, "page": 64, "dtype": "bf16", "fused": False, "holes": 0},
        # float32, small heads, an odd number of tokens and a padded tail
        {"name": "append_f32_5003", "op": "append", "tokens": 5003, "H_q": 12, "H_kv": 12, "D": 64,
         "group": 32, "page": 48, "dtype": "f32", "fused": False, "holes": 500},
        # one user: latency of a decoding step
        {"name": "decode_1x4096", "op": "attn", "requests": 1, "H_q": 32, "H_kv": 8, "D": 128,
         "group": 64, "page": 64, "min_len": 4095, "max_len": 4095, "n_q": 1, "idle": 0,
         "dtype": "bf16"},
        # a busy server: ragged lengths, two slots of the batch unused
        {"name": "decode_128_ragged", "op": "attn", "requests": 128, "H_q": 32, "H_kv": 8, "D": 128,
         "group": 64, "page": 64, "min_len": 100, "max_len": 16000, "n_q": 1, "idle": 2,
         "dtype": "bf16"},
        # one very long context, a head of its own for every query head
        {"name": "decode_1x131072", "op": "attn", "requests": 1, "H_q": 8, "H_kv": 8, "D": 128,
         "group": 128, "page": 128, "min_len": 131071, "max_len": 131071, "n_q": 1, "idle": 0,
         "dtype": "bf16"},
        # many short conversations on a small model
        {"name": "decode_256_small", "op": "attn", "requests": 256, "H_q": 12, "H_kv": 12, "D": 64,
         "group": 32, "page": 16, "min_len": 3, "max_len": 1023, "n_q": 1, "idle": 0,
         "dtype": "bf16"},
        # float32 all through, sixteen requests
        {"name": "decode_f32_16", "op": "attn", "requests": 16, "H_q": 32, "H_kv": 4, "D": 128,
         "group": 64, "page": 32, "min_len": 700, "max_len": 9000, "n_q": 1, "idle": 0,
         "dtype": "f32"},
        # drafts of up to five tokens a request checked in one pass
        {"name": "draft_32x5", "op": "attn", "requests": 32, "H_q": 32, "H_kv": 4, "D": 128,
         "group": 64, "page": 64, "min_len": 500, "max_len": 12000, "n_q": 5, "idle": 0,
         "dtype": "bf16"},
        # the next chunk of a long prompt over what is cached
        {"name": "prompt_chunk_2048", "op": "attn", "requests": 1, "H_q": 32, "H_kv": 8, "D": 128,
         "group": 64, "page": 64, "min_len": 30000, "max_len": 30000, "n_q": 2048, "idle": 0,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges above."""
    kind = rng.choice(["plan", "append", "attn", "attn"])
    if kind == "plan":
        r = _log_int(rng, 1, 700)
        new = _log_int(rng, 1, 1000)
        return {"op": "plan", "requests": r, "page": rng.choice([16, 32, 48, 64, 128, 256]),
                "min_old": rng.choice([0, 1, 50]), "max_old": _log_int(rng, 100, 4000),
                "max_new": new, "ended": rng.randint(0, r // 4),
                "pages_left": _log_int(rng, 1, 20000)}
    H_q, H_kv, D = rng.choice([(32, 8, 128), (32, 4, 128), (8, 8, 128), (12, 12, 64), (16, 2, 64)])
    group = rng.choice([g for g in (32, 64, 128) if g <= D])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "append":
        n = _log_int(rng, 1, 30000)
        return {"op": "append", "tokens": n, "H_q": H_q, "H_kv": H_kv, "D": D, "group": group,
                "page": page, "dtype": dtype, "fused": rng.choice([True, False]),
                "holes": rng.randint(0, n // 8)}
    n_q = rng.choice([1, 1, 1, 2, 3, 4, 7, 16, _log_int(rng, 17, 1500)])
    longest = _log_int(rng, 20, 100000 if n_q <= 16 else 20000)
    # at most about 400,000 cached tokens, and at most 12,000 query rows of long contexts
    most = max(1, min(256, 400000 // longest, 1500 // n_q))
    r = _log_int(rng, 1, most)
    return {"op": "attn", "requests": r, "H_q": H_q, "H_kv": H_kv, "D": D, "group": group,
            "page": page, "min_len": rng.choice([0, 1, longest // 3]), "max_len": longest,
            "n_q": n_q, "idle": rng.randint(0, r // 8), "dtype": dtype}


def _spread(n, lo, hi):
    """n whole numbers over [lo, hi], more of them short than long."""
    return [lo + int((hi - lo + 0.999) * ((i + 1) * 0.6180339887498949 % 1.0) ** 1.5)
            for i in range(n)]


def _shapes(c):
    """The new tokens and cached lengths of an attention case's requests: the same numbers
    for every seed, in an order of the seed's own.  One request: the longest."""
    r, idle = c["requests"], c["idle"]
    ctx = [c["max_len"]] if r == 1 else _spread(r - idle, c["min_len"], c["max_len"])
    n_q = [c["n_q"]] if r == 1 else _spread(r - idle, max(1, c["n_q"] // 2), c["n_q"])
    return n_q, [a + b for a, b in zip(ctx, n_q)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _dt(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def _block_bytes(c):
    """Bytes of one page of one K/V head."""
    return c["page"] // TILE * _tile_bytes(c)


def _tile_bytes(c):
    return 2 * TILE * (c["D"] // 2 + 4 * (c["D"] // c["group"]))


def _order(n, g):
    return torch.randperm(n, generator=g, device=DEV)


def _prepare_plan(c, g):
    r, page = c["requests"], c["page"]
    old = torch.tensor(_spread(r, c["min_old"], c["max_old"]), device=DEV)[_order(r, g)]
    grow = r - c["ended"]
    add = torch.tensor(_spread(grow, min(1, c["max_new"]), c["max_new"]) + [-1] * c["ended"], device=DEV)
    add = add[_order(r, g)]
    # of the requests that shrink every third only takes a few drafted tokens back
    back = (add < 0) & (torch.arange(r, device=DEV) % 3 == 0)
    new = torch.where(add >= 0, old + add, torch.where(back, (old - 5).clamp(min=0), 0))
    tokens = sum(_spread(grow, min(1, c["max_new"]), c["max_new"]))
    cols = -(-(c["max_old"] + c["max_new"]) // page)
    used = -(-old // page)
    held = r * (-(-c["max_old"] // page))
    n_pages = held + c["pages_left"]
    ids = _order(n_pages, g).to(torch.int32)
    col = torch.arange(cols, device=DEV)
    table = torch.where(col[None] < used[:, None],
                        ids[(torch.arange(r, device=DEV)[:, None] * (held // r) + col).clamp(max=n_pages - 1)], -1)
    free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    free[: c["pages_left"]] = ids[held:]
    i32 = lambda x: x.to(torch.int32).contiguous()  # noqa: E731
    n_slots = tokens + 13  # a padded batch
    return {"old": i32(old), "new": i32(new), "table": i32(table), "free": free,
            "n_free": torch.full((1,), c["pages_left"], dtype=torch.int32, device=DEV),
            "n_free_out": torch.zeros(1, dtype=torch.int32, device=DEV),
            "len_out": torch.zeros(r, dtype=torch.int32, device=DEV),
            "q_start": torch.zeros(r + 1, dtype=torch.int32, device=DEV),
            "slots": torch.zeros(n_slots, dtype=torch.int32, device=DEV), "n_pages": n_pages}


def _prepare_append(c, g):
    n, H_q, H, D = c["tokens"], c["H_q"], c["H_kv"], c["D"]
    # channels of different sizes, some of them large, as keys have them
    size = torch.exp(0.5 * torch.randn(H, D, generator=g, device=DEV))
    size = torch.where(torch.rand(H, D, generator=g, device=DEV) < 0.02, 8 * size, size)
    kf = torch.randn(n, H, D, generator=g, device=DEV) * size
    vf = torch.randn(n, H, D, generator=g, device=DEV)
    if c["fused"]:
        qkv = torch.zeros(n, H_q + 2 * H, D, dtype=_dt(c), device=DEV)
        k, v = qkv[:, H_q:H_q + H], qkv[:, H_q + H:]
    else:
        k, v = (torch.empty(H, n, D, dtype=_dt(c), device=DEV).transpose(0, 1) for _ in range(2))
    k.copy_(kf)
    v.copy_(vf)
    n_pages = -(-n // c["page"]) + 3
    # runs of 16 tokens land in pages of their own order
    slots = _order(n_pages, g)[:, None] * c["page"] + torch.arange(c["page"], device=DEV)
    slots = slots.reshape(-1)[:n].to(torch.int32)
    if c["holes"]:
        slots[_order(n, g)[: c["holes"]]] = -1
    cache = torch.zeros(n_pages, H, _block_bytes(c), dtype=torch.uint8, device=DEV)
    return {"k": k, "v": v, "slots": slots.contiguous(), "cache": cache, "n_pages": n_pages,
            "k_out": torch.empty(n, H, D, dtype=_dt(c), device=DEV),
            "v_out": torch.empty(n, H, D, dtype=_dt(c), device=DEV)}


def _prepare_attn(c, g):
    H_q, H, D, G, page, r = c["H_q"], c["H_kv"], c["D"], c["group"], c["page"], c["requests"]
    n_q, length = _shapes(c)
    n_q = torch.tensor(n_q + [0] * c["idle"], device=DEV)
    length = torch.tensor(length + [0] * c["idle"], device=DEV)
    at = _order(r, g)
    n_q, length = n_q[at], length[at]
    # an unused slot of the batch still holds a query row, over a cache of no tokens
    n_q = torch.where(length == 0, 1, n_q)
    n = sum(_shapes(c)[0]) + c["idle"]
    most = c["max_len"] + c["n_q"]
    cols = -(-most // page)
    used = -(-length // page)
    n_pages = int(used.sum()) + 2
    ids = _order(n_pages, g)
    first = torch.cumsum(used, 0) - used
    col = torch.arange(cols, device=DEV)
    table = torch.where(col[None] < used[:, None], ids[(first[:, None] + col).clamp(max=n_pages - 1)], -1)
    tiles = n_pages * H * (page // TILE)
    cache = torch.randint(0, 256, (tiles, 2, TILE * (D // 2 + 4 * D // G)), dtype=torch.uint8, generator=g,
                          device=DEV)
    step = 0.2 + 0.25 * torch.rand(tiles, 2, TILE * (D // G), generator=g, device=DEV)
    z = -(7.5 + torch.randn(tiles, 2, TILE * (D // G), generator=g, device=DEV)) * step - 16 * step
    az = torch.stack([16 * step, z], -1).to(torch.bfloat16).contiguous()
    cache[:, :, TILE * (D // 2):] = az.view(torch.uint8).reshape(tiles, 2, -1)
    qkv = torch.randn(n, H_q + 2 * H, D, generator=g, device=DEV).to(_dt(c))
    start = torch.zeros(r + 1, dtype=torch.int32, device=DEV)
    start[1:] = torch.cumsum(n_q, 0)
    return {"q": qkv[:, :H_q], "q_start": start, "len": length.to(torch.int32), "n_pages": n_pages,
            "table": table.to(torch.int32).contiguous(),
            "cache": cache.view(n_pages, H, _block_bytes(c)),
            "o": torch.empty(n, H_q, D, dtype=_dt(c), device=DEV),
            "lse": torch.empty(n, H_q, dtype=torch.float32, device=DEV)}


def prepare(case, seed):
    c = dict(case)
    s = {"plan": _prepare_plan, "append": _prepare_append, "attn": _prepare_attn}[c["op"]](c, _gen(seed))
    s["case"] = c
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_plan(c, s):
    page, r = c["page"], c["requests"]
    table, free, n_free = s["table"].long(), s["free"].long(), s["n_free"].long()
    cols = table.shape[1]
    old, new = (x.long().clamp(0, cols * page) for x in (s["old"], s["new"]))
    p_old, p_new = -(-old // page), -(-new // page)
    col = torch.arange(cols, device=DEV)[None]
    # pages past a request's new end go back, in the order of the requests
    back = (col >= p_new[:, None]) & (col < p_old[:, None])
    at = torch.cumsum(back.reshape(-1), 0).reshape(back.shape)
    room = torch.cat([free, free.new_zeros(1)])
    room.scatter_(0, torch.where(back, n_free + at - 1, len(free)).reshape(-1), table.reshape(-1))
    free = room[:-1]
    have = n_free + at[-1, -1]
    # and are taken from the list's end, by the requests in order as long as they last
    need = (p_new - p_old).clamp(min=0)
    end = torch.cumsum(need, 0)
    served = (need == 0) | (end <= have)
    take = (col >= p_old[:, None]) & (col < p_new[:, None]) & served[:, None]
    rank = (end - need)[:, None] + col - p_old[:, None]
    table = torch.where(take, free[(have - 1 - rank).clamp(0, len(free) - 1)], table)
    left = have - torch.where(served, need, 0).sum()
    add = (new - old).clamp(min=0)
    start = torch.cat([add.new_zeros(1), torch.cumsum(add, 0)])
    i = torch.arange(s["slots"].shape[0], device=DEV)
    req = torch.searchsorted(start[1:], i, right=True).clamp(max=r - 1)
    pos = old[req] + i - start[req]
    slot = table[req, (pos // page).clamp(max=cols - 1)] * page + pos % page
    slot = torch.where((i < start[-1]) & served[req], slot, -1)
    return [x.to(torch.int32) for x in (table, free, left.reshape(1), torch.where(served, new, old), start, slot)]


def _plain_group(x, c):
    """(c, a, z) of the groups of x [n, H, D] as the cache holds them, in float32."""
    n, H, D = x.shape
    x = x.float()
    x = torch.where(torch.isnan(x), 0.0, x).clamp(-HUGE, HUGE).reshape(n, H, D // c["group"], c["group"])
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    a = ((hi - lo) * torch.tensor(16 / 15, dtype=torch.float32, device=DEV)).to(torch.bfloat16).float()
    a = torch.where(a < TINY, 0.0, a)
    z = (lo - a).to(torch.bfloat16).float()
    # the codes are chosen next to a border: d against a * (33 + 2 j) / 32, in 64 bits
    d = (x - z).double()
    code = torch.ceil(d / a.double() * 16 - 16.5).clamp(0, 15)
    return torch.where(a == 0, 0.0, code).float(), a, z


def _value(code, a, z):
    return (a * (1 + code / 16) + z).to(torch.bfloat16)


def _plain_append(c, s):
    live = ((s["slots"] >= 0) & (s["slots"] < s["n_pages"] * c["page"]))[:, None, None]
    return [torch.where(live, _value(*_plain_group(s[x], c)).reshape(s[x].shape).to(_dt(c)), 0) for x in ("k", "v")]


def _plain_rows(c, s):
    """Keys and values of every request's pages, [2][requests, tokens, H, D] in float32."""
    H, D, G, page = c["H_kv"], c["D"], c["group"], c["page"]
    r, cols = s["table"].shape
    pages = s["cache"][s["table"].long().clamp(0, s["n_pages"] - 1)]
    t = pages.reshape(r, cols, H, page // TILE, 2, TILE * (D // 2 + 4 * D // G))
    words = t[..., : TILE * D // 2].contiguous().view(torch.int32).reshape(*t.shape[:5], TILE, D // 8)
    az = t[..., TILE * D // 2:].contiguous().view(torch.bfloat16).float().reshape(*t.shape[:5], TILE, D // G, 2)
    # keys: a word is turned left by three bits; values: the token 2 t + e of eight is in row t + 4 e
    k = ((words[..., 0, :, :] >> 3) & 0x1FFFFFFF) | (words[..., 0, :, :] << 29)
    row = torch.arange(TILE, device=DEV)
    row = row // 8 * 8 + row % 8 // 2 + row % 2 * 4
    v = words[..., 1, :, :][..., row, :]
    w = torch.stack([k, v])
    par = torch.stack([az[..., 0, :, :, :], az[..., 1, :, :, :][..., row, :, :]])
    dim = torch.arange(8, device=DEV)
    shift = (4 * (dim // 2 + dim % 2 * 4)).to(torch.int32)
    code = ((w[..., None] >> shift) & 15).float().reshape(*w.shape[:-1], D // G, G)
    x = (par[..., :1] * (1 + code / 16) + par[..., 1:]).to(torch.bfloat16).float()
    # [2, r, cols, H, tiles, TILE, D/G, G] -> [2, r, tokens, H, D]
    return x.reshape(2, r, cols, H, page, D).transpose(3, 4).reshape(2, r, cols * page, H, D)


def _plain_attn(c, s):
    H_q, H, D = c["H_q"], c["H_kv"], c["D"]
    rep, r = H_q // H, c["requests"]
    k, v = _plain_rows(c, s)
    most = c["n_q"]
    start, length = s["q_start"].long(), s["len"].long()
    n_q = start[1:] - start[:-1]
    j = torch.arange(most, device=DEV)
    rows = (start[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)
    live = j[None] < n_q[:, None]
    q = s["q"].float()[rows].reshape(r, most, H, rep, D)
    score = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(r, H, rep * most, D), k.permute(0, 2, 3, 1))
    score = score.reshape(r, H, rep, most, -1) * (1.0 / math.sqrt(D))
    key = torch.arange(k.shape[1], device=DEV)
    sees = key[None, None] <= (length - n_q)[:, None, None] + j[None, :, None]
    sees = sees & (key < length[:, None])[:, None]
    score = score.masked_fill_(~sees[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((key < length[:, None])[..., None, None], v, 0.0)
    o = torch.matmul(p.reshape(r, H, rep * most, -1), v.permute(0, 2, 1, 3)).reshape(r, H, rep, most, D)
    o = o / torch.where(total == 0, 1.0, total)
    lse = top[..., 0] + total[..., 0].log()
    # back to the packed rows
    at = torch.where(live, rows, s["q"].shape[0]).reshape(-1)
    out = o.new_zeros(s["q"].shape[0] + 1, H_q, D)
    out[at] = o.permute(0, 3, 1, 2, 4).reshape(r * most, H_q, D)
    out_lse = lse.new_zeros(s["q"].shape[0] + 1, H_q)
    out_lse[at] = lse.permute(0, 3, 1, 2).reshape(r * most, H_q)
    return [out[:-1].to(_dt(c)), out_lse[:-1]]


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _handle(c, s):
    """The descriptor and workspace that a program keeps beside its cache."""
    import blockwise_online_softmax_cpattn_gb300 as cp
    if c["op"] == "plan":
        d = cp.make_cache_desc(1, 1, 128, c["page"], s["n_pages"])
        size = cp.cpattn_cache_plan_workspace(d, c["requests"])
    else:
        d = cp.make_cache_desc(c["H_q"], c["H_kv"], c["D"], c["page"], s["n_pages"], group=c["group"],
                               dtype=c["dtype"])
        size = cp.cpattn_cache_attn_workspace(d)
    s["handle"] = cp, d, torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)


def _own(c, s):
    if "handle" not in s:
        _handle(c, s)
    cp, d, ws = s["handle"]
    if c["op"] == "plan":
        cp.check(cp.cpattn_cache_plan(d, c["requests"], s["table"].shape[1], s["old"], s["new"], s["table"],
                                      s["free"], s["n_free"], s["n_free_out"], s["len_out"], s["q_start"],
                                      s["slots"], s["slots"].shape[0], ws))
        return [s[x] for x in ("table", "free", "n_free_out", "len_out", "q_start", "slots")]
    if c["op"] == "append":
        n = c["tokens"]
        cp.check(cp.cpattn_cache_append(d, n, s["k"], s["v"], s["slots"], s["cache"]))
        cp.check(cp.cpattn_cache_read(d, n, s["slots"], s["cache"], s["k_out"], s["v_out"]))
        return [s["k_out"], s["v_out"]]
    cp.check(cp.cpattn_cache_attn(d, c["requests"], s["table"].shape[1], s["q"].shape[0], c["n_q"], s["q"],
                                  s["q_start"], s["len"], s["table"], s["cache"], s["o"], s["lse"], ws))
    return [s["o"], s["lse"]]


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"plan": _plain_plan, "append": _plain_append, "attn": _plain_attn}[c["op"]](c, state)


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "plan":
        grow = c["requests"] - c["ended"]
        tokens = sum(_spread(grow, min(1, c["max_new"]), c["max_new"]))
        # lengths in and out, the offsets, a slot a token, a page taken or returned: two numbers
        pages = tokens // c["page"] + c["ended"] * c["max_old"] // (2 * c["page"])
        return {"bytes": 16 * c["requests"] + 4 * tokens + 8 * pages, "flops": 0}
    rows = c["H_kv"] * c["D"] * (4 if c["dtype"] == "f32" else 2)
    held = 2 * c["H_kv"] * (c["D"] // 2 + 4 * (c["D"] // c["group"]))
    if c["op"] == "append":
        live = c["tokens"] - c["holes"]
        # rows in, codes out, codes in, rows out, two slot maps
        return {"bytes": live * (2 * rows + 2 * held) + c["tokens"] * (2 * rows + 8), "flops": 0}
    n_q, length = _shapes(c)
    elt = 4 if c["dtype"] == "f32" else 2
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(n_q, length))
    n = sum(n_q) + c["idle"]
    return {"bytes": sum(length) * held + n * c["H_q"] * (2 * c["D"] * elt + 4) + 4 * c["requests"],
            "flops": 4 * c["D"] * c["H_q"] * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_append(c, s):
    import numpy as np
    f32 = np.float32
    outs = []
    live = s["slots"].cpu().numpy() >= 0
    for name in ("k", "v"):
        x = s[name].float().cpu().numpy()
        x = x.reshape(-1, c["group"])
        lo, hi = x.min(1), x.max(1)
        to_bf16 = lambda y: torch.from_numpy(y).to(torch.bfloat16).double().numpy()  # noqa: E731
        a = to_bf16((hi - lo) * f32(16 / 15))
        a[a < TINY] = 0
        z = to_bf16(lo - a.astype(f32))
        d = (x - z.astype(f32)[:, None]).astype(np.float64)
        code = np.zeros(d.shape)
        for j in range(15):  # how many of the fifteen borders the value is above
            code += d > a[:, None] * ((33 + 2 * j) / 32)
        code[a == 0] = 0
        y = a[:, None] * (16 + code) / 16 + z[:, None]
        y = torch.from_numpy(y).to(torch.bfloat16).double().reshape(s[name].shape)
        y[torch.from_numpy(~live)] = 0
        outs.append(y)
    return outs


def _exact_attn(c, s):
    H_q, H, D, G, page = c["H_q"], c["H_kv"], c["D"], c["group"], c["page"]
    table, length, start = s["table"].tolist(), s["len"].tolist(), s["q_start"].tolist()
    n = s["q"].shape[0]
    o = torch.zeros(n, H_q, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(n, H_q, dtype=torch.float64, device=DEV)
    block = s["cache"].view(s["n_pages"], H, page // TILE, 2, -1)
    for r, L in enumerate(length):
        b, e = start[r], start[r + 1]
        if L == 0:
            lse[b:e] = -math.inf
            continue
        used = torch.tensor(table[r][: -(-L // page)], device=DEV)
        mine = block[used]                                     # [pages, H, tiles, 2, bytes]
        kv = []
        for which in (0, 1):
            t = mine[:, :, :, which]
            by = t[..., : TILE * D // 2].reshape(*t.shape[:3], TILE, D // 8, 4).long()
            word = by[..., 0] + (by[..., 1] << 8) + (by[..., 2] << 16) + (by[..., 3] << 24)
            if which == 0:
                word = (word >> 3) | ((word & 7) << 29)
            par = t[..., TILE * D // 2:].contiguous().view(torch.bfloat16).double()
            par = par.reshape(*t.shape[:3], TILE, D // G, 2)
            val = torch.empty(*word.shape, 8, dtype=torch.float64, device=DEV)
            for d in range(8):
                val[..., d] = 1 + ((word >> (4 * (d // 2) + 16 * (d % 2))) & 15) / 16
            val = val.reshape(*t.shape[:3], TILE, D // G, G)
            val = (val * par[..., :1] + par[..., 1:]).to(torch.bfloat16).double()
            val = val.reshape(*t.shape[:3], TILE, D)
            if which == 1:
                back = [t8 for h in (0, 8) for t8 in (h, h + 4, h + 1, h + 5, h + 2, h + 6, h + 3, h + 7)]
                val = val[..., back, :]
            kv.append(val.transpose(1, 2).reshape(-1, H, TILE, D).transpose(1, 2).reshape(-1, H, D)[:L])
        k, v = kv
        i = torch.arange(b, e, device=DEV) - b
        hidden = torch.arange(L, device=DEV)[None] > (L - (e - b) + i)[:, None]
        for h in range(H):
            q = s["q"][b:e, h * H_q // H:(h + 1) * H_q // H].double()
            sc = torch.einsum("nrd,ld->rnl", q, k[:, h]) / math.sqrt(D)
            sc.masked_fill_(hidden[None], -math.inf)
            lse[b:e, h * H_q // H:(h + 1) * H_q // H] = torch.logsumexp(sc, -1).T
            o[b:e, h * H_q // H:(h + 1) * H_q // H] = torch.einsum("rnl,ld->nrd", torch.softmax(sc, -1), v[:, h])
    return [o, lse]


def exact(case, seed):
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return (_exact_append if case["op"] == "append" else _exact_attn)(s["case"], s)
