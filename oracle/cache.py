"""The 4-bit key/value cache in plain numpy: the definition of its format, its block
tables and its attention, in float64 except where the format itself fixes float32 or
bfloat16 roundings.  Test infrastructure only."""
import numpy as np

TILE = 16


def round_bf16(x):
    """float64 -> the nearest bfloat16 (ties to even), as float64.  Normal range only."""
    m, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.rint(m * 256.0) / 256.0, e)


def bf16_bits(x):
    """Bit patterns of float64 values that are bfloat16 numbers."""
    return (np.asarray(x, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint32)


def bits_bf16(b):
    return (np.asarray(b, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


def quantise(x, group):
    """x [..., D] float32 -> codes [..., D] (0..15), a, z [..., D / group] (float64)."""
    x = np.asarray(x, dtype=np.float32)
    x = np.where(np.isnan(x), np.float32(0), np.clip(x, np.float32(-2.0 ** 120), np.float32(2.0 ** 120)))
    g = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    lo, hi = g.min(-1), g.max(-1)
    a = round_bf16((hi - lo) * np.float32(16 / 15))
    a = np.where(a < 2.0 ** -100, 0.0, a)
    z = round_bf16(lo - a.astype(np.float32))
    d = (g - z.astype(np.float32)[..., None]).astype(np.float64)
    borders = a[..., None, None] * (33 + 2 * np.arange(15)) / 32
    codes = (d[..., None] > borders).sum(-1)
    codes = np.where(a[..., None] == 0, 0, codes)
    return codes.reshape(x.shape), a, z


def values(codes, a, z):
    """The numbers the cache stands for, as float64 (each is a bfloat16 number)."""
    group = codes.shape[-1] // a.shape[-1]
    g = codes.reshape(*a.shape, group)
    return round_bf16(a[..., None] * (1 + g / 16) + z[..., None]).reshape(codes.shape)


def v_row(t):
    return (t & 8) | ((t >> 1) & 3) | ((t & 1) << 2)


def _words(codes, is_v):
    """[..., D] codes -> [..., D / 8] words."""
    c = codes.reshape(*codes.shape[:-1], -1, 8).astype(np.uint64)
    w = np.zeros(c.shape[:-1], np.uint64)
    for ch in range(8):
        w |= c[..., ch] << np.uint64(4 * (ch // 2 + 4 * (ch % 2)))
    if not is_v:
        w = ((w << np.uint64(3)) | (w >> np.uint64(29))) & np.uint64(0xFFFFFFFF)
    return w.astype(np.uint32)


def half_tile(D, group):
    return TILE * (D // 2 + 4 * (D // group))


def _row_at(cache, page_tokens, D, group, slot, h, is_v):
    """(words, az) views of one row of `cache` [n_pages, H_kv, block] uint8."""
    page, off = divmod(int(slot), page_tokens)
    half = half_tile(D, group)
    base = (off // TILE) * 2 * half + is_v * half
    r = v_row(off % TILE) if is_v else off % TILE
    block = cache[page, h]
    w = block[base + r * D // 2: base + (r + 1) * D // 2].view(np.uint32)
    p = base + TILE * D // 2 + r * 4 * (D // group)
    return w, block[p: p + 4 * (D // group)].view(np.uint32)


def append(cache, page_tokens, group, k, v, slots):
    """k, v [n, H_kv, D] float32 into `cache` in place."""
    n, H, D = k.shape
    for is_v, x in ((0, k), (1, v)):
        codes, a, z = quantise(x, group)
        w = _words(codes, is_v)
        az = bf16_bits(a) | (bf16_bits(z) << 16)
        for i, s in enumerate(slots):
            if 0 <= s < cache.shape[0] * page_tokens:
                for h in range(H):
                    row, par = _row_at(cache, page_tokens, D, group, s, h, is_v)
                    row[:] = w[i, h]
                    par[:] = az[i, h]


def read(cache, page_tokens, group, D, slots):
    """Rows of the slots, k and v [n, H_kv, D] float64; zeros outside the cache."""
    H = cache.shape[1]
    out = np.zeros((2, len(slots), H, D))
    words = np.zeros((2, len(slots), H, D // 8), np.uint32)
    az = np.zeros((2, len(slots), H, D // group), np.uint32)
    live = np.array([0 <= s < cache.shape[0] * page_tokens for s in slots], bool)
    for i, s in enumerate(slots):
        if live[i]:
            for h in range(H):
                for is_v in (0, 1):
                    words[is_v, i, h], az[is_v, i, h] = _row_at(cache, page_tokens, D, group, s, h, is_v)
    words[0] = (words[0] >> np.uint32(3)) | (words[0] << np.uint32(29))
    codes = np.stack([(words >> np.uint32(4 * (ch // 2 + 4 * (ch % 2)))) & np.uint32(15) for ch in range(8)], -1)
    codes = codes.reshape(2, len(slots), H, D)
    with np.errstate(invalid="ignore"):
        out = values(codes, bits_bf16(az & np.uint32(0xFFFF)), bits_bf16(az >> np.uint32(16)))
    out[:, ~live] = 0
    return out[0], out[1]


def plan(page, len_old, len_new, table, free_list, n_free, n_slots):
    """One request after the other.  Returns (table, free_list, n_free, len_out, q_start, slots)."""
    table, free = table.copy(), free_list.copy()
    R, cols = table.shape
    old = np.clip(len_old, 0, cols * page)
    new = np.clip(len_new, 0, cols * page)
    top = int(n_free)
    for r in range(R):  # give back
        for p in range(-(-new[r] // page), -(-old[r] // page)):
            free[top] = table[r, p]
            top += 1
    have, wanted = top, 0
    len_out = new.copy()
    q_start, slots = [0], []
    for r in range(R):  # take
        po, pn = -(-old[r] // page), -(-new[r] // page)
        need = max(pn - po, 0)
        served = need == 0 or wanted + need <= have
        wanted += need
        if served:
            for p in range(po, pn):
                top -= 1
                table[r, p] = free[top]
        else:
            len_out[r] = old[r]
        for pos in range(old[r], new[r]):
            slots.append(table[r, pos // page] * page + pos % page if served else -1)
        q_start.append(q_start[-1] + max(new[r] - old[r], 0))
    slots = (slots + [-1] * n_slots)[:n_slots]
    return table, free, top, len_out, np.array(q_start), np.array(slots, dtype=np.int64)


def attention(q, k, v, seen, scale):
    """One request and K/V head: q [n, D], k, v [L, D] float64, query i sees the keys
    [0, seen[i]).  Returns (o, lse, sum p |v| / sum p, max scale * sum |q| |k|)."""
    n, D = q.shape
    L = k.shape[0]
    s = scale * (q @ k.T)
    hidden = np.arange(L)[None, :] >= np.asarray(seen)[:, None]
    s = np.where(hidden, -np.inf, s)
    m = s.max(1, initial=-np.inf)
    p = np.exp(s - np.where(np.isinf(m), 0.0, m)[:, None])
    p[hidden] = 0
    tot = p.sum(1)
    safe = np.where(tot == 0, 1.0, tot)[:, None]
    with np.errstate(divide="ignore"):
        lse = np.where(tot == 0, -np.inf, m + np.log(tot))
    size = scale * (np.abs(q) @ np.abs(k).T).max(initial=0.0) if L else 0.0
    return p @ v / safe, lse, p @ np.abs(v) / safe, size
