"""GPU: the 4-bit key/value cache against the oracle's plain numpy form.

Tolerances of the attention.  The cache's values are bf16 numbers on both sides, so
what differs is: the scores, sums of D float32 products with at most 2^-23 of the
running sum lost at each step, off by ds <= 2^-23 (D + 8) max(scale sum |q||k|); with
them every probability by a factor within 1 +- 2 ds (numerator and sum), the
exponential and the sums in float32 by less than 2^-17 of it (sums of up to 2^6 steps a
thread); on the bf16 path P rounded to bf16, 2^-8 of each term.  So o is off by at most
(2 ds + 2^-17 [+ 2^-8]) sum p |v|, plus its own rounding to bf16, 2^-8 |o|.  lse is off by
ds + 2^-20 (1 + |lse|).
A probability below float32's least normal number, 2^-126 of the row's largest (which is at
least 1 in the kernel's units, and so is the sum), may count as zero: where all the weight is
on keys whose value is 0 that is what is left of o, at most 2^-126 sum |v|."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from conftest import ROOT
from gpu_helpers import cp_mod, dev
from oracle import cache as OC
from test_gpu_canary import Guarded, check_all

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(dev())


def make_cache(cp, d, rng=None, fill=None):
    n = cp.cpattn_cache_bytes(d)
    block = n // (d.n_pages * d.H_kv)
    if fill is None:
        c = rng.integers(0, 256, n, dtype=np.uint8)
    else:
        c = np.full(n, fill, np.uint8)
    return c.reshape(d.n_pages, d.H_kv, block)


def to_dt(x, dtype):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.float32 if dtype == "f32" else torch.bfloat16)


def f32_of(t):
    return t.float().cpu().numpy()


def checked(cp, status):
    cp.check(status)
    cp.check(cp.cpattn_check())


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
def _rows_run(cp, d, dtype, k, v, slots, layout, seed=0):
    """Appends into a cache of random bytes; returns it, the oracle's, and the rows read."""
    rng = np.random.default_rng(seed)
    cache = make_cache(cp, d, rng)
    n, H, D = k.shape
    kt, vt = to_dt(k, dtype), to_dt(v, dtype)
    ref = cache.copy()
    OC.append(ref, d.page, d.group, f32_of(kt), f32_of(vt), slots)
    if layout == "fused":       # slices of a projection [n, H + 2 H, D]
        buf = torch.zeros(n, 3 * H, D, dtype=kt.dtype, device=dev())
        kd, vd = buf[:, H:2 * H], buf[:, 2 * H:]
    elif layout == "heads":     # the ring's [H, n, D]
        kd, vd = (torch.zeros(H, n, D, dtype=kt.dtype, device=dev()).transpose(0, 1) for _ in range(2))
    else:
        kd, vd = (torch.zeros(n, H, D, dtype=kt.dtype, device=dev()) for _ in range(2))
    kd.copy_(kt)
    vd.copy_(vt)
    c = torch.from_numpy(cache).to(dev())
    s = i32(slots)
    st = cp.cpattn_cache_append(d, n, kd, vd, s, c)
    cp.check(st)
    code = cp.cpattn_check()
    ko, vo = torch.full_like(kd, 7.0), torch.full_like(vd, 7.0)
    checked(cp, cp.cpattn_cache_read(d, n, s, c, ko, vo))
    return c.cpu().numpy(), ref, f32_of(ko), f32_of(vo), code


@pytest.mark.parametrize("D,group", [(128, 32), (128, 64), (128, 128), (64, 32), (64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["plain", "fused", "heads"])
def test_append_and_read(D, group, dtype, layout):
    cp = cp_mod()
    rng = np.random.default_rng(D + group)
    d = cp.make_cache_desc(6, 3, D, 48, 5, group=group, dtype=dtype)
    n = 101
    k = rng.normal(size=(n, 3, D)) * np.exp(rng.normal(size=(3, D)))
    v = rng.normal(size=(n, 3, D)) + 3
    slots = rng.permutation(5 * 48)[:n]
    slots[5], slots[77], slots[100] = -1, 5 * 48, 2 ** 31 - 1
    got, ref, ko, vo, code = _rows_run(cp, d, dtype, k, v, slots, layout)
    assert code == cp.OK
    assert np.array_equal(got, ref)  # every byte, those of other slots among them
    rk, rv = OC.read(ref, d.page, group, D, slots)
    assert np.array_equal(ko, rk) and np.array_equal(vo, rv)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 1000])
def test_append_lengths(n):
    cp = cp_mod()
    rng = np.random.default_rng(n)
    d = cp.make_cache_desc(1, 1, 64, 16, 64, group=32)
    k, v = rng.normal(size=(2, n, 1, 64))
    got, ref, ko, vo, _ = _rows_run(cp, d, "bf16", k, v, rng.permutation(1024)[:n], "plain")
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_hard_values(dtype):
    """Constant groups, ties, tiny and huge spreads, large offsets, zeros of both signs."""
    cp = cp_mod()
    rng = np.random.default_rng(9)
    d = cp.make_cache_desc(1, 1, 64, 16, 2, group=32, dtype=dtype)
    k = np.zeros((12, 1, 64), np.float32)
    k[0] = 0.75
    k[1, 0, ::2] = -0.0
    k[2] = np.tile(np.arange(32) / 2, 2)           # a step of 31/30: codes at and near borders
    k[3] = np.tile(np.arange(32) // 2, 2)          # 0 .. 15: a = 16, every value at a code
    k[4] = np.tile(np.arange(32) / 2 - 0.25, 2)
    k[5] = rng.normal(size=64) * 2.0 ** 118
    k[6] = rng.normal(size=64) * 2.0 ** -98        # around the least spread that is kept
    k[7] = rng.normal(size=64) * 2.0 ** -110
    k[8] = 1000 + rng.integers(0, 8, 64)
    k[9] = 2.0 ** 120 * np.where(np.arange(64) % 2, 1, -1)
    k[10] = -5 + 2.0 ** -8 * rng.integers(0, 3, 64)
    k[11, 0, 3] = 1e-30
    got, ref, ko, vo, code = _rows_run(cp, d, dtype, k, k[::-1].copy(), np.arange(12), "plain")
    assert code == cp.OK
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_reports_what_it_cannot_hold(dtype):
    cp = cp_mod()
    rng = np.random.default_rng(4)
    d = cp.make_cache_desc(1, 1, 64, 16, 2, group=32, dtype=dtype)
    base = rng.normal(size=(5, 1, 64)).astype(np.float32)
    for bad in (np.nan, np.inf, -np.inf, 2.0 ** 121, -3e38):
        k = base.copy()
        k[2, 0, 40] = bad
        got, ref, ko, vo, code = _rows_run(cp, d, dtype, k, base, np.arange(5), "plain")
        assert code == cp.ERR_RANGE
        assert np.array_equal(got, ref)
        assert np.isfinite(ko).all()
    # a skipped token is not looked at
    got, ref, ko, vo, code = _rows_run(cp, d, dtype, k, base, np.array([0, 1, -1, 3, 4]), "plain")
    assert code == cp.OK and np.array_equal(got, ref)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_on_16_byte_boundaries(dtype):
    """Rows that lie on 16-byte boundaries and on no wider ones."""
    cp = cp_mod()
    rng = np.random.default_rng(21)
    d = cp.make_cache_desc(2, 2, 64, 16, 8, group=32, dtype=dtype)
    n, vec = 50, 4 if dtype == "f32" else 8
    kt, vt = (to_dt(x, dtype) for x in rng.normal(size=(2, n, 2, 64)))
    slots = rng.permutation(128)[:n]
    bufs = [torch.full((n, 2 * 64 + vec), 7.0, dtype=kt.dtype, device=dev()) for _ in range(4)]
    kd, vd, ko, vo = (b[:, vec:].unflatten(1, (2, 64)) for b in bufs)
    assert all(x.data_ptr() % 32 == 16 for x in (kd, vd, ko, vo))
    kd.copy_(kt)
    vd.copy_(vt)
    c, s = torch.zeros(cp.cpattn_cache_bytes(d), dtype=torch.uint8, device=dev()), i32(slots)
    checked(cp, cp.cpattn_cache_append(d, n, kd, vd, s, c))
    ref = np.zeros(tuple(make_cache(cp, d, fill=0).shape), np.uint8)
    OC.append(ref, 16, 32, f32_of(kt), f32_of(vt), slots)
    assert np.array_equal(c.cpu().numpy().reshape(ref.shape), ref)
    checked(cp, cp.cpattn_cache_read(d, n, s, c, ko, vo))
    for got, want, buf in zip((ko, vo), OC.read(ref, 16, 32, 64, slots), bufs[2:]):
        assert np.array_equal(f32_of(got), want)
        assert (buf[:, :vec] == 7.0).all()      # the gaps between rows


def test_append_of_one_slot_twice_touches_no_other():
    cp = cp_mod()
    rng = np.random.default_rng(22)
    d = cp.make_cache_desc(1, 1, 128, 32, 4)
    n = 300
    k, v = (to_dt(x, "bf16") for x in rng.normal(size=(2, n, 1, 128)))
    slots = rng.integers(0, 100, n)
    ref = make_cache(cp, d, rng)
    c, s, kd, vd = torch.from_numpy(ref.copy()).to(dev()), i32(slots), k.to(dev()), v.to(dev())
    checked(cp, cp.cpattn_cache_append(d, n, kd, vd, s, c))
    once = np.flatnonzero(np.bincount(slots, minlength=128)[slots] == 1)
    OC.append(ref, 32, 64, f32_of(k)[once], f32_of(v)[once], slots[once])
    keep = np.array([x for x in range(128) if (slots == x).sum() < 2])
    for got, want in zip(OC.read(c.cpu().numpy(), 32, 64, 128, keep), OC.read(ref, 32, 64, 128, keep)):
        assert np.array_equal(got, want, equal_nan=True)


def test_append_past_32_bits():
    """A cache of over 4 GB: the last page's bytes."""
    cp = cp_mod()
    d = cp.make_cache_desc(8, 8, 128, 64, 60000, group=64)
    assert cp.cpattn_cache_bytes(d) > 1 << 32
    c = torch.zeros(60000, 8, 64 * 144, dtype=torch.uint8, device=dev())
    rng = np.random.default_rng(6)
    k, v = to_dt(rng.normal(size=(3, 8, 128)), "bf16"), to_dt(rng.normal(size=(3, 8, 128)), "bf16")
    slots = np.array([60000 * 64 - 1, 59999 * 64, 5])
    s = i32(slots)
    kd, vd = k.to(dev()), v.to(dev())
    checked(cp, cp.cpattn_cache_append(d, 3, kd, vd, s, c))
    ref = np.zeros((2, 8, 64 * 144), np.uint8)
    OC.append(ref, 64, 64, f32_of(k), f32_of(v), np.array([64 + 63, 64, 5]))
    assert np.array_equal(c[59999].cpu().numpy(), ref[1])
    assert np.array_equal(c[0].cpu().numpy(), ref[0])
    assert not c[1:59999].any()
    # and attention over it: one request on the far page
    q = to_dt(rng.normal(size=(1, 8, 128)), "bf16").to(dev())
    o, ws = torch.empty_like(q), torch.empty(cp.cpattn_cache_attn_workspace(d), dtype=torch.uint8, device=dev())
    checked(cp, cp.cpattn_cache_attn(d, 1, 1, 1, 1, q, i32([0, 1]), i32([1]), i32([[59999]]), c, o, None, ws))
    ko, vo = torch.empty_like(q), torch.empty_like(q)
    checked(cp, cp.cpattn_cache_read(d, 1, i32([59999 * 64]), c, ko, vo))
    assert torch.equal(o, vo)  # one key: its value


@pytest.mark.parametrize("page,n_q", [(16 * 900000, 1), (16 * 900001, 2), (16 * 900000, 60)])
def test_a_page_past_32_bits(page, n_q):
    """A page whose bytes pass 32 bits: its last tokens through append, read and attention.  All
    other keys are zeros and all other values too, so the answer is a sum of few terms."""
    cp = cp_mod()
    rng = np.random.default_rng(31)
    d = cp.make_cache_desc(1, 1, 128, page, 1, group=32, causal=0, scale=1.0)
    assert cp.cpattn_cache_bytes(d) > 1 << 31
    c = torch.zeros(cp.cpattn_cache_bytes(d), dtype=torch.uint8, device=dev())
    n = 20
    slots = i32(page - n + np.arange(n))
    k, v = np.zeros((n, 1, 128)), rng.normal(size=(n, 1, 128))
    k[7, 0, :32] = 1.0
    kd, vd = to_dt(k, "bf16").to(dev()), to_dt(v, "bf16").to(dev())
    checked(cp, cp.cpattn_cache_append(d, n, kd, vd, slots, c))
    ko, vo = torch.empty_like(kd), torch.empty_like(vd)
    checked(cp, cp.cpattn_cache_read(d, n, slots, c, ko, vo))
    assert np.array_equal(f32_of(ko), k)
    vals = OC.values(*OC.quantise(f32_of(vd), 32))
    assert np.array_equal(f32_of(vo), vals)
    # the score of the one key: 32 q; q is bf16 and its products and their sum are exact
    q = np.zeros((n_q, 1, 128))
    q[:, 0, :32] = 0.5 + np.arange(n_q)[:, None] / 128
    qd = to_dt(q, "bf16").to(dev())
    o, lse = torch.empty(n_q, 1, 128, dtype=torch.bfloat16, device=dev()), torch.empty(n_q, 1, device=dev())
    ws = torch.empty(cp.cpattn_cache_attn_workspace(d), dtype=torch.uint8, device=dev())
    checked(cp, cp.cpattn_cache_attn(d, 1, 1, n_q, n_q, qd, i32([0, n_q]), i32([page]), i32([[0]]), c, o, lse, ws))
    w = np.ones((n_q, n))
    w[:, 7] = np.exp(32 * f32_of(qd)[:, 0, 0].astype(np.float64))
    total = w.sum(1) + (page - n)
    ref = w @ vals[:, 0].astype(np.float64) / total[:, None]
    size = w @ np.abs(vals[:, 0]).astype(np.float64) / total[:, None]
    # as at the head of this file, with exact scores; sums of up to 2^18 equal terms a thread in
    # float32, each off by 2^-24 of the sum so far
    got = o[:, 0].double().cpu().numpy()
    sums = 2.0 ** -24 * 2.0 ** 18
    assert np.all(np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -17 + sums) * size + 2.0 ** -8 * np.abs(ref) * 1.02)
    assert np.all(np.abs(lse[:, 0].double().cpu().numpy() - np.log(total)) <= sums + 2.0 ** -17)


@pytest.mark.parametrize("n_q", [1, 60])
def test_every_piece_of_a_page_past_32_bits_counts(n_q):
    """Values that grow along a page of 14.4 million tokens, scores of zero: o is their mean, lse the
    logarithm of their number.  A CTA's piece is 1/152 of the sum, 2^-7.2; the spans lose 2^-13 of it
    at most, some 160 joins two roundings each, 2^-16.  P is 1, so its sum is exact."""
    cp = cp_mod()
    page, D, group = 16 * 900000, 128, 32
    d = cp.make_cache_desc(1, 1, D, page, 1, group=group, causal=0, o_dtype="f32")
    g = torch.Generator(device=dev())
    g.manual_seed(7)
    tiles = page // 16
    c = torch.randint(0, 256, (tiles, 2, 16 * (D // 2 + 4 * (D // group))), dtype=torch.uint8, generator=g, device=dev())
    codes = c[:, 1, : 16 * (D // 2)].view(torch.int32).reshape(tiles, 16, D // 8)
    a = 2.0 ** (torch.arange(tiles, device=dev()) * 6 // tiles)     # 1 .. 32, a sixth of the page each
    az = torch.zeros(tiles, 2, 16 * (D // group), 2, device=dev())
    az[..., 0] = a[:, None, None]
    c[:, :, 16 * (D // 2):] = az.to(torch.bfloat16).view(torch.uint8).reshape(tiles, 2, -1)
    total = torch.zeros(D, dtype=torch.float64, device=dev())
    for ch in range(8):   # channel 2p + e of a word in bits 4 (p + 4e)
        x = (codes >> (4 * (ch // 2 + 4 * (ch % 2)))) & 15
        total[ch::8] = ((16 + x).sum(1).double() * a[:, None].double()).sum(0) / 16
    ref = (total / page).cpu().numpy()
    q = torch.zeros(n_q, 1, D, dtype=torch.bfloat16, device=dev())
    o, lse = torch.empty(n_q, 1, D, device=dev()), torch.empty(n_q, 1, device=dev())
    ws = torch.empty(cp.cpattn_cache_attn_workspace(d), dtype=torch.uint8, device=dev())
    checked(cp, cp.cpattn_cache_attn(d, 1, 1, n_q, n_q, q, i32([0, n_q]), i32([page]), i32([[0]]), c.reshape(-1), o,
                                     lse, ws))
    err = np.abs(o[:, 0].double().cpu().numpy() - ref)
    assert np.all(err <= (2.0 ** -13 + 2.0 ** -16) * ref), (err / ref).max()
    assert np.abs(lse.double().cpu().numpy() - np.log(page)).max() <= 2.0 ** -20 * (1 + np.log(page))


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
def _plan_state(rng, R, cols, page, n_pages, old):
    used = -(-old // page)
    ids = rng.permutation(n_pages)
    table = rng.integers(-5, n_pages + 5, (R, cols))     # stale entries past a request's end
    at = 0
    for r in range(R):
        table[r, : used[r]] = ids[at: at + used[r]]
        at += used[r]
    free = np.full(n_pages, -7)
    free[: n_pages - at] = ids[at:]
    return table, free, n_pages - at


def _plan_run(cp, page, n_pages, old, new, table, free, n_free, n_slots, alias=False):
    R, cols = table.shape
    d = cp.make_cache_desc(1, 1, 64, page, n_pages)
    o, n, t, f = i32(old), i32(new), i32(table), i32(free)
    nf = i32([n_free])
    nfo = nf if alias else i32([-1])
    lens = o if alias else i32(np.full(R, -1))
    start, slots = i32(np.full(R + 1, -1)), i32(np.full(max(n_slots, 1), -9))
    ws = torch.full((cp.cpattn_cache_plan_workspace(d, R),), 0xA5, dtype=torch.uint8, device=dev())
    checked(cp, cp.cpattn_cache_plan(d, R, cols, o, n, t, f, nf, nfo, lens, start, slots, n_slots, ws))
    got = [x.cpu().numpy() for x in (t, f, nfo, lens, start, slots)]
    ref = OC.plan(page, np.asarray(old), np.asarray(new), table, free, n_free, n_slots)
    assert np.array_equal(got[0], ref[0])
    assert got[2][0] == ref[2]
    assert np.array_equal(got[1][: ref[2]], ref[1][: ref[2]])
    assert np.array_equal(got[3], ref[3]) and np.array_equal(got[4], ref[4])
    assert np.array_equal(got[5][:n_slots], ref[5])
    assert n_slots or got[5][0] == -9


@pytest.mark.parametrize("R,cols,page,grow,slack,extra", [
    (1, 1, 16, 0, 0, 0), (1, 8, 16, 50, 9, 3), (2, 6, 32, 40, 20, 0), (7, 9, 48, 60, 40, 17),
    (33, 12, 16, 100, 300, 5), (64, 40, 64, 1, 64, 0), (64, 8, 16, 90, 20, 1), (300, 6, 16, 70, 100, 64),
    (1023, 3, 16, 4, 900, 0), (1024, 3, 16, 3, 50, 1), (1025, 3, 16, 20, 3000, 7), (2500, 5, 32, 50, 800, 9),
    (40, 200, 16, 2000, 9000, 100), (3, 3000 // 16, 16, 2900, 400, 0),
])
@pytest.mark.parametrize("shrink", [0.0, 0.4])
def test_plan(R, cols, page, grow, slack, extra, shrink):
    cp = cp_mod()
    rng = np.random.default_rng(R * 7 + cols)
    cap = cols * page
    old = np.minimum(rng.integers(0, max(1, cap - grow) + 1, R), cap)
    new = np.minimum(old + rng.integers(0, grow + 1, R), cap)
    down = rng.random(R) < shrink
    new = np.where(down, rng.integers(0, old + 1), new)
    new = np.where(down & (rng.random(R) < 0.5), 0, new)
    n_pages = int((-(-old // page)).sum()) + slack + 1
    table, free, n_free = _plan_state(rng, R, cols, page, n_pages, old)
    tokens = int(np.maximum(new - old, 0).sum())
    for n_slots in {tokens + extra, tokens // 2}:
        for alias in (False, True):
            _plan_run(cp, page, n_pages, old, new, table, free, n_free, n_slots, alias)


def test_plan_runs_out_of_pages():
    """Exactly enough, one too few, none; requests that need no page go on."""
    cp = cp_mod()
    rng = np.random.default_rng(1)
    old = np.array([16, 10, 32, 0, 5, 31])
    new = np.array([40, 12, 33, 64, 5, 32])   # 2, 0, 1, 4, 0, 0 pages
    for slack in (0, 1, 2, 3, 6, 7, 8):
        n_pages = int((-(-old // 16)).sum()) + slack
        table, free, n_free = _plan_state(rng, 6, 6, 16, n_pages, old)
        assert n_free == slack
        _plan_run(cp, 16, n_pages, old, new, table, free, n_free, 120)


def test_plan_clamps_lengths():
    cp = cp_mod()
    rng = np.random.default_rng(2)
    old, new = np.array([-3, 5, 2 ** 31 - 1, -2 ** 31]), np.array([7, 2 ** 31 - 1, 10, -1])
    table, free, n_free = _plan_state(rng, 4, 3, 16, 20, np.clip(old, 0, 48))
    _plan_run(cp, 16, 20, old, new, table, free, n_free, 60)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Case:
    """Requests with random cached bytes, their tables, queries and the oracle's answer."""

    def __init__(self, cp, H_q=8, H_kv=2, D=128, group=64, page=64, n_q=(1,), kv_len=(100,), dtype="bf16",
                 o_dtype=None, causal=1, seed=0, tail=3, spare=2, fused=True, offset=0.0, holes=()):
        rng = np.random.default_rng(seed)
        self.cp, self.n_q, self.kv_len, self.tail = cp, np.array(n_q), np.array(kv_len), tail
        R = len(n_q)
        used = np.maximum(-(-self.kv_len // page), 0)
        cols = int(max(1, used.max())) + spare
        n_pages = int(used.sum()) + 3
        self.d = d = cp.make_cache_desc(H_q, H_kv, D, page, n_pages, group=group, dtype=dtype, o_dtype=o_dtype,
                                        causal=causal)
        ids = rng.permutation(n_pages)
        table = np.full((R, cols), 2 ** 31 - 1)           # entries past the end: not pages
        table[:, -1] = -1
        at = 0
        for r in range(R):
            table[r, : used[r]] = ids[at: at + used[r]]
            at += used[r]
        for r, c in holes:
            table[r, c] = -1 if c % 2 else n_pages
        self.table = table
        # rows nothing was appended to hold bytes that decode to NaN
        cache = make_cache(cp, d, fill=0xFF)
        for r in range(R):
            n = self.kv_len[r]
            if n > 0:
                pos = np.arange(n)
                slots = np.where((table[r, pos // page] >= 0) & (table[r, pos // page] < n_pages),
                                 table[r, pos // page] * page + pos % page, -1)
                k = rng.normal(size=(n, H_kv, D)) * 1.5
                v = rng.normal(size=(n, H_kv, D)) + offset
                OC.append(cache, page, group, k.astype(np.float32), v.astype(np.float32), slots)
        self.cache = cache
        n = int(self.n_q.sum()) + tail
        q = to_dt(rng.normal(size=(n, H_q, D)), dtype)
        self.q = f32_of(q).astype(np.float64)
        if fused:
            buf = torch.zeros(n, H_q + 2 * H_kv, D, dtype=q.dtype, device=dev())
            self.qd = buf[:, :H_q]
            self.qd.copy_(q)
        else:
            self.qd = q.to(dev())
        self.start = np.concatenate([[0], np.cumsum(self.n_q)])
        self.dev = [i32(self.start), i32(self.kv_len), i32(table), torch.from_numpy(cache).to(dev())]
        self.o = torch.full((n, H_q, D), 77.0, device=dev(),
                            dtype=torch.float32 if d.o_dtype == cp.F32 else torch.bfloat16)
        self.lse = torch.full((n, H_q), 77.0, dtype=torch.float32, device=dev())
        self.ws = torch.full((cp.cpattn_cache_attn_workspace(d),), 0xFF, dtype=torch.uint8, device=dev())

    def run(self, lse=True, max_q=None):
        R, cols = self.table.shape
        return self.cp.cpattn_cache_attn(self.d, R, cols, self.qd.shape[0], max_q or max(1, int(self.n_q.max())),
                                         self.qd, *self.dev[:3], self.dev[3], self.o,
                                         self.lse if lse else None, self.ws)

    def expect(self):
        d = self.d
        n, rep = int(self.n_q.sum()), d.H_q // d.H_kv
        o, lse = np.zeros((n, d.H_q, d.D)), np.full((n, d.H_q), -np.inf)
        pv, ds, self.flushed = np.zeros_like(o), np.zeros((n, d.H_q)), 0.0
        for r in range(len(self.n_q)):
            b, e, L = self.start[r], self.start[r + 1], max(int(self.kv_len[r]), 0)
            if L == 0 or b == e:
                continue
            pos = np.arange(L)
            pg = self.table[r, pos // d.page].astype(np.int64)
            live = (pg >= 0) & (pg < d.n_pages)
            k, v = OC.read(self.cache, d.page, d.group, d.D, np.where(live, pg * d.page + pos % d.page, -1))
            seen = np.arange(e - b) + 1 + L - (e - b) if d.causal else np.full(e - b, L)
            k, v = k[live], v[live]
            self.flushed = max(self.flushed, 2.0 ** -126 * np.abs(v).sum(0).max(initial=0.0))
            below = np.concatenate([[0], np.cumsum(live)])
            seen = below[np.clip(seen, 0, L)]
            for h in range(d.H_q):
                res = OC.attention(self.q[b:e, h], k[:, h // rep], v[:, h // rep], seen, d.scale)
                o[b:e, h], lse[b:e, h], pv[b:e, h] = res[:3]
                ds[b:e, h] = 2.0 ** -23 * (d.D + 8) * res[3]
        return o, lse, pv, ds

    def compare(self, lse=True):
        n = int(self.n_q.sum())
        got, got_lse = self.o.double().cpu().numpy(), self.lse.double().cpu().numpy()
        o, ref_lse, pv, ds = self.expect()
        bf16 = self.d.dtype == self.cp.BF16
        tol = (2 * ds[..., None] + 2.0 ** -17 + (2.0 ** -8 if bf16 else 0)) * pv + self.flushed
        if self.d.o_dtype == self.cp.BF16:
            tol = tol + 2.0 ** -8 * (np.abs(o) + tol)
        assert np.all(np.abs(got[:n] - o) <= tol), np.max(np.abs(got[:n] - o) - tol)
        assert np.all(got[n:] == 77.0)            # rows behind the last sequence
        if lse:
            empty = np.isinf(ref_lse)
            assert np.array_equal(np.isneginf(got_lse[:n]), empty)
            fine = ~empty
            diff = np.abs(got_lse[:n][fine] - ref_lse[fine])
            assert np.all(diff <= ds[fine] + 2.0 ** -20 * (1 + np.abs(ref_lse[fine]))), diff.max()
            assert np.all(got_lse[n:] == 77.0)
        else:
            assert np.all(got_lse == 77.0)

    def check(self, **kw):
        checked(self.cp, self.run(**kw))
        self.compare(lse=kw.get("lse", True))
        return self


LENS = (1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 0, 511)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,group,page", [(128, 64, 64), (128, 32, 16), (128, 128, 48), (64, 32, 32), (64, 64, 128)])
def test_attn_decode_lengths(dtype, D, group, page):
    Case(cp_mod(), D=D, group=group, page=page, n_q=[1] * len(LENS), kv_len=LENS, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H_q,H_kv", [(1, 1), (3, 3), (4, 2), (6, 2), (8, 1), (20, 4), (10, 1), (17, 1), (40, 2)])
def test_attn_heads(dtype, H_q, H_kv):
    Case(cp_mod(), H_q=H_q, H_kv=H_kv, n_q=[1, 1, 2], kv_len=[70, 33, 150], dtype=dtype, seed=H_q).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [1, 0])
@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (4, 4, 64), (8, 1, 64)])
def test_attn_several_tokens(dtype, causal, H_q, H_kv, D):
    """Ragged numbers of new tokens; requests without any; more new tokens than cached ones
    (rows before the sequence's start see nothing); a request of only new tokens."""
    n_q = [3, 0, 1, 5, 17, 9, 40, 2, 33]
    kv = [50, 20, 1, 5, 100, 4, 300, 0, 33]
    Case(cp_mod(), H_q=H_q, H_kv=H_kv, D=D, group=32, n_q=n_q, kv_len=kv, dtype=dtype, causal=causal).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q,kv", [([130], [130]), ([257], [1000]), ([64, 300, 1], [64, 301, 700]),
                                    ([128, 128], [128, 256]), ([200, 1, 90], [150, 9, 1200])])
def test_attn_prompts(dtype, n_q, kv):
    Case(cp_mod(), H_q=4, H_kv=2, n_q=n_q, kv_len=kv, dtype=dtype, page=48).check()


@pytest.mark.parametrize("D,group,page", [(128, 128, 128), (128, 32, 16), (64, 64, 64), (64, 32, 48)])
@pytest.mark.parametrize("causal", [1, 0])
def test_attn_prompt_formats(D, group, page, causal):
    Case(cp_mod(), H_q=6, H_kv=2, D=D, group=group, page=page, n_q=[150, 61], kv_len=[190, 700], causal=causal,
         seed=3).check()


@pytest.mark.parametrize("n_q", [1, 6, 150])
def test_attn_float32_output_of_bf16(n_q):
    Case(cp_mod(), n_q=[n_q, n_q], kv_len=[400, 150], o_dtype="f32", seed=5).check()


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("n_q", [12, 16, 40])
def test_attn_many_items_of_a_cta(n_q, seed):
    """Wide drafts: a CTA meets many items of odd and even numbers of tiles, of one half and of
    two, one after the other, call behind call."""
    rng = np.random.default_rng(seed)
    R = 24
    kv = rng.integers(1, 9, R) * 128 - rng.integers(0, 128, R)
    kv[rng.integers(0, R, 3)] = 0
    nq = rng.integers(1, n_q + 1, R)
    nq[:2] = n_q
    c = Case(cp_mod(), H_q=32, H_kv=4, n_q=nq, kv_len=kv, seed=seed, page=32)
    for _ in range(60):
        cp_mod().check(c.run())
    c.check()


@pytest.mark.parametrize("n_q", [1, 100])
def test_attn_without_lse(n_q):
    Case(cp_mod(), n_q=[n_q], kv_len=[130], fused=False).check(lse=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n_q", [1, 3, 200])
def test_attn_long(dtype, n_q):
    """One request over all SMs: the pieces of a row meet again."""
    Case(cp_mod(), H_q=4, H_kv=1, n_q=[n_q], kv_len=[9001], dtype=dtype, offset=2.0).check()


@pytest.mark.parametrize("max_q", [1, 4, 64, 5000])
def test_attn_max_q_only_chooses_the_kernel(max_q):
    Case(cp_mod(), n_q=[1, 30, 2], kv_len=[40, 500, 90], page=16).check(max_q=max_q)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_a_mixed_batch_in_two_calls(dtype):
    """Decoding requests and, from a later request on, chunks of prompts: rows that the other call
    computes are left as they are."""
    c = Case(cp_mod(), n_q=[1, 1, 2, 1, 150, 77], kv_len=[300, 5, 64, 1100, 400, 77], dtype=dtype)
    start, lens, table = c.dev[:3]
    cols, n = c.table.shape[1], c.qd.shape[0]
    call = lambda a, b, max_q: checked(c.cp, c.cp.cpattn_cache_attn(  # noqa: E731
        c.d, b - a, cols, n, max_q, c.qd, start[a:], lens[a:], table[a:], c.dev[3], c.o, c.lse, c.ws))
    call(0, 4, 2)
    assert (c.o[5:] == 77.0).all() and (c.lse[5:] == 77.0).all()
    first = c.o[:5].clone()
    call(4, 6, 150)
    assert torch.equal(c.o[:5], first)
    c.compare()


@pytest.mark.parametrize("n_q", [1, 150])
def test_attn_pages_outside_the_cache_hold_no_key(n_q):
    """Entries that are no pages, among them all of a request's, and a hole in the middle."""
    holes = [(0, 1), (1, 0), (1, 1), (2, 3), (2, 4)]
    Case(cp_mod(), n_q=[n_q] * 3, kv_len=[50, 32, 200], page=16, holes=holes, spare=1).check()


@pytest.mark.parametrize("n_q", [1, 130])
def test_attn_peaked_and_flat_rows(n_q):
    """Scores far apart (the running maximum moves by hundreds) and all equal."""
    c = Case(cp_mod(), n_q=[n_q] * 2, kv_len=[300, 400], fused=False)
    c.q[: n_q] *= 40
    c.q[n_q: 2 * n_q] = 0
    c.qd.copy_(to_dt(c.q, "bf16"))
    c.q = f32_of(c.qd).astype(np.float64)
    c.check()


@pytest.mark.parametrize("n_q", [1, 130])
def test_attn_nan_query_stays_in_its_row(n_q):
    c = Case(cp_mod(), n_q=[n_q, n_q], kv_len=[200, 333], fused=False)
    checked(c.cp, c.run())
    o, lse = c.o.clone(), c.lse.clone()
    c.qd[n_q // 2, 3, 5] = float("nan")
    checked(c.cp, c.run())
    keep = torch.ones(o.shape[:2], dtype=torch.bool, device=dev())
    keep[n_q // 2, 3] = False
    assert torch.equal(c.o[keep], o[keep]) and torch.equal(c.lse[keep], lse[keep])
    assert c.o[n_q // 2, 3].isnan().all() and c.lse[n_q // 2, 3].isnan()


@pytest.mark.parametrize("dtype,n_q", [("bf16", 1), ("bf16", 4), ("bf16", 150), ("f32", 2)])
def test_attn_is_deterministic_and_replays(dtype, n_q):
    """Eager twice, on another stream, and from a graph: the same bits."""
    c = Case(cp_mod(), n_q=[n_q] * 3, kv_len=[1200, 37, 3000], dtype=dtype)
    checked(c.cp, c.run())
    o, lse = c.o.clone(), c.lse.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.o.fill_(77.0)
        cp_mod().check(c.run())
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cp_mod().check(c.run())
    for _ in range(2):
        c.o.fill_(77.0)
        c.lse.fill_(77.0)
        c.ws.fill_(0xFF)
        g.replay()
        checked(c.cp, 0)
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R", [32, 33, 257, 700])
def test_attn_many_requests(dtype, R):
    rng = np.random.default_rng(R)
    kv = rng.integers(0, 40, R)
    kv[rng.integers(0, R, 3)] = 500
    Case(cp_mod(), H_q=4, H_kv=2, D=64, group=32, page=16, n_q=rng.integers(0, 3, R), kv_len=kv, dtype=dtype,
         seed=R).check()


def test_attn_many_prompts():
    rng = np.random.default_rng(3)
    n_q = rng.integers(0, 30, 280)
    Case(cp_mod(), H_q=4, H_kv=1, D=64, group=64, page=16, n_q=n_q, kv_len=n_q + rng.integers(0, 100, 280)).check()


@pytest.mark.parametrize("H_q,n_q", [(8, 1), (9, 1), (4, 2), (3, 3), (4, 12), (7, 7), (1, 48), (1, 49), (16, 3), (17, 3)])
def test_attn_rows_where_kernels_change(H_q, n_q):
    Case(cp_mod(), H_q=H_q, H_kv=1, n_q=[n_q, 1, n_q], kv_len=[n_q, 300, 1100], seed=H_q).check()


@pytest.mark.parametrize("dtype,n_q", [("bf16", 2), ("bf16", 100), ("f32", 2)])
def test_attn_clamps_what_it_is_told(dtype, n_q):
    """Offsets outside the rows and lengths outside the table."""
    c = Case(cp_mod(), n_q=[n_q, n_q, n_q], kv_len=[90, 320, 150], dtype=dtype, tail=0)
    cap = c.table.shape[1] * c.d.page
    c.dev[0].copy_(i32([-5, n_q, 2 * n_q, 2 ** 31 - 1]))
    c.dev[1].copy_(i32([-7, 2 ** 31 - 1, 150]))
    c.kv_len = np.array([0, cap, 150])
    c.check()
    # a request that ends before it begins has no rows
    c = Case(cp_mod(), n_q=[n_q, 0, 0], kv_len=[90, 300, 150], dtype=dtype, tail=0)
    c.dev[0].copy_(i32([0, n_q, n_q - 1, -2 ** 31]))
    c.check()


def test_attn_graphs_that_share_a_workspace():
    """Captured calls of all kernels on one workspace, replayed in turn, and eager ones between."""
    cp = cp_mod()
    cases = [Case(cp, n_q=[1] * 3, kv_len=[1200, 37, 3000]), Case(cp, n_q=[5] * 2, kv_len=[900, 2000], seed=1),
             Case(cp, n_q=[150, 20], kv_len=[1500, 1024], seed=2), Case(cp, n_q=[2], kv_len=[2500], dtype="f32", seed=3)]
    ws = max((c.ws for c in cases), key=lambda x: x.numel())
    graphs = []
    for c in cases:
        c.ws = ws
        c.check()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            cp.check(c.run())
        graphs.append(g)
    want = [(c.o.clone(), c.lse.clone()) for c in cases]
    for i in (0, 1, 0, 2, 3, 0, 2, 2, 1, 3, 1, 0):
        cases[i].o.fill_(77.0)
        cases[i].lse.fill_(77.0)
        graphs[i].replay()
        cp.check(cases[(i + 1) % 4].run())
    checked(cp, 0)
    for c, (o, lse) in zip(cases, want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


@pytest.mark.parametrize("n_q", [(1, 1), (1, 150), (150, 130)])
def test_attn_on_two_streams(n_q):
    """Two calls at once, each with a workspace of its own."""
    cp = cp_mod()
    cases = [Case(cp, n_q=[n, n], kv_len=[2000, 900], seed=n) for n in n_q]
    for c in cases:
        c.check()
    want = [(c.o.clone(), c.lse.clone()) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                cp.check(c.run())
    torch.cuda.synchronize()
    checked(cp, 0)
    for c, (o, lse) in zip(cases, want):
        assert torch.equal(c.o, o) and torch.equal(c.lse, lse)


def test_attn_with_a_device_side_batch_that_changes():
    """A captured call follows lengths and tables that change between replays."""
    c = Case(cp_mod(), n_q=[1] * 5, kv_len=[300, 5, 0, 129, 64], tail=0)
    cp_mod().check(c.run())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cp_mod().check(c.run())
    for lens in ([300, 5, 0, 129, 64], [1, 0, 0, 0, 0], [0, 4, 0, 17, 33], [299, 1, 0, 128, 63]):
        c.kv_len = np.array(lens)
        c.dev[1].copy_(i32(lens))
        g.replay()
        checked(c.cp, 0)
        c.compare()


def _long_run(dtype, rows, L, R, n_q=1, D=128, group=64, page=64, qs=0.0, seed=0):
    """R requests of n_q tokens and `rows` query heads over the same pages of L tokens, causal,
    float32 results.  Values are positive and of many sizes, so that sums use every bit they have;
    queries of size qs.  Returns o, lse and, of a few rows, (their index, o, lse, ds) in 64 bits."""
    cp = cp_mod()
    rng = np.random.default_rng(seed)
    n_pages = -(-L // page)
    d = cp.make_cache_desc(rows, 1, D, page, n_pages, group=group, dtype=dtype, o_dtype="f32")
    cache = make_cache(cp, d, rng).reshape(-1, 2, 16 * (D // 2 + 4 * (D // group)))
    az = np.zeros((cache.shape[0], 2, 16 * (D // group), 2), np.float32)
    az[:, 0] = 2.0, -2.9375                            # keys within +-1
    az[:, 1, :, 0] = np.exp(rng.normal(size=az.shape[:1] + az.shape[2:3]))
    cache[:, :, 16 * (D // 2):] = OC.bf16_bits(OC.round_bf16(az)).astype("<u2").view(np.uint8).reshape(
        cache.shape[0], 2, -1)
    cache = cache.reshape(n_pages, 1, -1)
    q = to_dt(qs * rng.normal(size=(R * n_q, rows, D)), dtype)
    o, lse = torch.empty(R * n_q, rows, D, device=dev()), torch.empty(R * n_q, rows, device=dev())
    ws = torch.empty(cp.cpattn_cache_attn_workspace(d), dtype=torch.uint8, device=dev())
    table = i32(np.arange(n_pages))[None].repeat(R, 1)
    checked(cp, cp.cpattn_cache_attn(d, R, n_pages, R * n_q, n_q, q.to(dev()), i32(np.arange(R + 1) * n_q),
                                     i32(np.full(R, L)), table, torch.from_numpy(cache).to(dev()), o, lse, ws))
    k, v = OC.read(cache, page, group, D, np.arange(L))
    out = []
    for t in rng.integers(0, R * n_q, 6 if qs or n_q > 1 else 1):
        h = int(rng.integers(0, rows))
        ref, ref_lse, _, size = OC.attention(f32_of(q[t:t + 1, h]).astype(np.float64), k[:, 0], v[:, 0],
                                               [L - n_q + t % n_q + 1], d.scale)
        out.append((int(t), h, ref[0], ref_lse[0], 2.0 ** -23 * (D + 8) * size))
    return o, lse, out


@pytest.mark.parametrize("rows,D,group", [(8, 128, 64), (3, 128, 32), (8, 64, 64)])
def test_attn_float32_sums_over_long_runs(rows, D, group):
    """A warp that walks 750 units of a request.  What the sums may lose, of sum p |v| and of sum p
    alike: 64 additions a span, each rounded to nearest, 2^-18; 24 folds of two roundings, 2^-18.4;
    a tile's three products on the tensor cores, 3 2^-23; the exponential, 2^-21: below 2^-17, so o
    is off by at most 2^-16 sum p |v| and what the scores are (2 ds)."""
    o, lse, rows64 = _long_run("f32", rows, 24000, 5000, D=D, group=group, qs=0.003)
    for t, h, ref, ref_lse, ds in rows64:
        err = np.abs(o[t, h].double().cpu().numpy() - ref)
        assert np.all(err <= (2 * ds + 2.0 ** -16) * ref), (err / ref).max()
        assert abs(lse[t, h].item() - ref_lse) <= ds + 2.0 ** -17 + 2.0 ** -20 * (1 + abs(ref_lse))


@pytest.mark.parametrize("rows,D,L", [(8, 128, 200000), (16, 128, 200000), (5, 64, 150000), (13, 64, 150000)])
def test_attn_sums_over_long_runs(rows, D, L):
    """Scores of zero: P is 1 and its sum exact.  O may lose 2^-23 of its sum at each of the 512
    steps that a span has on the tensor cores, 2^-14 in all; the folds of the spans (25) two
    roundings each, below 2^-18.  (One sum of all the steps would be 1e-3 too small.)"""
    o, lse, rows64 = _long_run("bf16", rows, L, 5000, D=D)
    for t, h, ref, ref_lse, _ in rows64:
        err = np.abs(o[t, h].double().cpu().numpy() - ref)
        assert np.all(err <= (2.0 ** -14 + 2.0 ** -17) * ref), (err / ref).max()
        assert abs(lse[t, h].item() - ref_lse) <= 2.0 ** -20 * (1 + abs(ref_lse))


@pytest.mark.parametrize("rows,n_q,R,D,group,L", [(4, 20000, 1, 128, 64, 220000), (4, 16, 400, 128, 128, 180000),
                                                  (6, 9, 400, 64, 32, 150001), (4, 20000, 1, 64, 64, 150000)])
def test_attn_prompt_sums_over_long_runs(rows, n_q, R, D, group, L):
    """As above, of many rows (halves of items that share the tokens, and that share the rows): a
    span has 1024 steps, 2^-13."""
    o, lse, rows64 = _long_run("bf16", rows, L, R, n_q=n_q, D=D, group=group)
    for t, h, ref, ref_lse, _ in rows64:
        err = np.abs(o[t, h].double().cpu().numpy() - ref)
        assert np.all(err <= (2.0 ** -13 + 2.0 ** -17) * ref), (err / ref).max()
        assert abs(lse[t, h].item() - ref_lse) <= 2.0 ** -20 * (1 + abs(ref_lse))


@pytest.mark.parametrize("dtype,rows,n_q,R,D,qs", [("bf16", 8, 1, 3000, 128, 3.0), ("bf16", 16, 1, 3000, 64, 1.0),
                                                   ("f32", 8, 1, 3000, 128, 3.0), ("f32", 4, 500, 6, 64, 1.0),
                                                   ("bf16", 4, 300, 30, 128, 3.0), ("bf16", 4, 16, 310, 128, 1.0),
                                                   ("bf16", 4, 300, 30, 64, 1.0), ("bf16", 4, 16, 310, 64, 3.0)])
def test_attn_spans_with_maxima_of_their_own(dtype, rows, n_q, R, D, qs):
    """Scores that differ, so that every span has its own maximum.  As at the head of this file, and
    what the spans may lose (2^-13 at most, float32 2^-17; of the probabilities' sum 2^-17)."""
    o, lse, rows64 = _long_run(dtype, rows, 60017, R, n_q=n_q, D=D, qs=qs)
    tol = 2.0 ** -16 if dtype == "f32" else 2.0 ** -8 + 2.0 ** -13 + 2.0 ** -16
    for t, h, ref, ref_lse, ds in rows64:
        err = np.abs(o[t, h].double().cpu().numpy() - ref)
        assert np.all(err <= (2 * ds + tol) * ref), (err / ref).max()
        assert abs(lse[t, h].item() - ref_lse) <= ds + 2.0 ** -17 + 2.0 ** -20 * (1 + abs(ref_lse))


# ---------------------------------------------------------------------------
# bounded waits, buffers' ends, the bounds-checked build
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("hook,dtype,n_q,kv", [(1, "bf16", [1, 1], [1200, 300]), (1, "bf16", [4, 1], [1200, 300]),
                                               (1, "f32", [2], [700]), (2, "bf16", [150, 20], [1200, 300]),
                                               (2, "bf16", [30], [2000]), (3, "bf16", [1], [9001]),
                                               (3, "f32", [3], [4000])])
def test_attn_timeout_is_reported_and_context_survives(hook, dtype, n_q, kv):
    """A wait that nothing ends runs out (50 ms), is reported once, and the next call is right."""
    c = Case(cp_mod(), H_q=4, H_kv=1, n_q=n_q, kv_len=kv, dtype=dtype)
    c.d.debug_fault = hook
    c.cp.check(c.run())
    assert c.cp.cpattn_check() == c.cp.ERR_TIMEOUT
    assert c.cp.cpattn_check() == c.cp.OK
    c.d.debug_fault = 0
    c.o.fill_(77.0)
    c.lse.fill_(77.0)
    c.check()


@pytest.mark.parametrize("nan_first", [True, False])
def test_a_value_out_of_range_hides_no_timeout(nan_first):
    """A NaN appended before (or after) a wait that runs out: both are reported, the fault first."""
    c = Case(cp_mod(), H_q=4, H_kv=1, n_q=[1], kv_len=[700])
    k = torch.full((1, 1, 128), float("nan"), dtype=torch.bfloat16, device=dev())
    last = i32([c.d.n_pages * c.d.page - 1])
    append = lambda: c.cp.check(c.cp.cpattn_cache_append(c.d, 1, k, k, last, c.dev[3].clone()))  # noqa: E731
    if nan_first:
        append()
    c.d.debug_fault = 1
    c.cp.check(c.run())
    c.d.debug_fault = 0
    if not nan_first:
        append()
    assert [c.cp.cpattn_check() for _ in range(3)] == [c.cp.ERR_TIMEOUT, c.cp.ERR_RANGE, c.cp.OK]
    append()
    assert [c.cp.cpattn_check() for _ in range(2)] == [c.cp.ERR_RANGE, c.cp.OK]


@pytest.mark.parametrize("dtype,n_q,kv,D", [("bf16", [1, 2], [100, 3001], 128), ("bf16", [4, 5], [77, 2000], 64),
                                            ("bf16", [130, 61], [400, 1500], 128), ("f32", [1, 3], [900, 50], 64)])
def test_calls_stay_in_their_buffers(dtype, n_q, kv, D):
    """Every output and workspace between guard bytes, every row written."""
    cp = cp_mod()
    rng = np.random.default_rng(5)
    R, H_q, H, page, cols = 2, 8, 2, 16, -(-max(kv) // 16)
    n_pages = sum(-(-x // page) for x in kv)
    d = cp.make_cache_desc(H_q, H, D, page, n_pages, group=32, dtype=dtype)
    tdt = torch.float32 if dtype == "f32" else torch.bfloat16
    i, n, new = torch.int32, sum(n_q), sum(kv)
    b = dict(table=Guarded((R, cols), i), free=Guarded((n_pages,), i), n_free=Guarded((1,), i), lens=Guarded((R,), i),
             start=Guarded((R + 1,), i), slots=Guarded((new,), i),
             plan_ws=Guarded((cp.cpattn_cache_plan_workspace(d, R),), torch.uint8),
             cache=Guarded((cp.cpattn_cache_bytes(d),), torch.uint8), k=Guarded((new, H, D), tdt),
             v=Guarded((new, H, D), tdt), o=Guarded((n, H_q, D), tdt), lse=Guarded((n, H_q), torch.float32),
             ws=Guarded((cp.cpattn_cache_attn_workspace(d),), torch.uint8))
    t = {name: g.t for name, g in b.items()}
    t["free"].copy_(i32(rng.permutation(n_pages)))
    t["n_free"].fill_(n_pages)
    t["lens"].zero_()
    checked(cp, cp.cpattn_cache_plan(d, R, cols, t["lens"], i32(kv), t["table"], t["free"], t["n_free"], t["n_free"],
                                     t["lens"], t["start"], t["slots"], new, t["plan_ws"]))
    assert t["lens"].tolist() == kv and t["n_free"].item() == 0
    k, v = (to_dt(rng.normal(size=(new, H, D)), dtype).to(dev()) for _ in range(2))
    checked(cp, cp.cpattn_cache_append(d, new, k, v, t["slots"], t["cache"]))
    checked(cp, cp.cpattn_cache_read(d, new, t["slots"], t["cache"], t["k"], t["v"]))
    q = to_dt(rng.normal(size=(n, H_q, D)), dtype).to(dev())
    checked(cp, cp.cpattn_cache_attn(d, R, cols, n, max(n_q), q, i32(np.concatenate([[0], np.cumsum(n_q)])), t["lens"],
                                     t["table"], t["cache"], t["o"], t["lse"], t["ws"]))
    check_all(b, written=("k", "v", "o", "lse"))


@pytest.mark.skipif(os.environ.get("CPATTN_DEBUG_LIB") == "1", reason="is that build")
def test_the_bounds_checked_build():
    import __graft_entry__
    __graft_entry__._build_lib().build(debug=True)
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_cache.py", "-m", "gpu", "-x", "-q", "-p",
                        "no:cacheprovider"], cwd=ROOT, env=dict(os.environ, CPATTN_DEBUG_LIB="1"), capture_output=True,
                       text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_a_server_step_by_step():
    """Prompts, decoding steps, drafts taken back and requests that end, through plan,
    append and attention, against rows kept aside."""
    cp = cp_mod()
    rng = np.random.default_rng(11)
    H_q, H, D, page, R, cols, n_pages = 8, 2, 64, 16, 4, 12, 40
    d = cp.make_cache_desc(H_q, H, D, page, n_pages, group=32)
    cache = torch.full((cp.cpattn_cache_bytes(d),), 0xFF, dtype=torch.uint8, device=dev())
    table, free = i32(np.full((R, cols), -1)), i32(np.arange(n_pages))
    n_free, lens = i32([n_pages]), i32(np.zeros(R))
    start, slots_all = i32(np.zeros(R + 1)), i32(np.zeros(200))
    ws = torch.empty(max(cp.cpattn_cache_plan_workspace(d, R), cp.cpattn_cache_attn_workspace(d)),
                     dtype=torch.uint8, device=dev())
    kept = [[np.zeros((0, H, D)), np.zeros((0, H, D))] for _ in range(R)]
    targets = [[37, 90, 1, 16], [38, 91, 2, 17], [43, 96, 7, 22], [40, 92, 3, 22], [41, 0, 4, 23],
               [0, 60, 5, 24], [80, 61, 6, 25]]
    old = [0] * R
    for new in targets:
        add = [max(b - a, 0) for a, b in zip(old, new)]
        n = sum(add)
        checked(cp, cp.cpattn_cache_plan(d, R, cols, lens, i32(new), table, free, n_free, n_free, lens, start,
                                         slots_all, 200, ws))
        assert lens.tolist() == list(new)
        qkv = to_dt(rng.normal(size=(max(n, 1), H_q + 2 * H, D)), "bf16").to(dev())
        q, k, v = qkv[:, :H_q], qkv[:, H_q:H_q + H], qkv[:, H_q + H:]
        cp.check(cp.cpattn_cache_append(d, n, k, v, slots_all, cache))
        o = torch.zeros(max(n, 1), H_q, D, dtype=torch.bfloat16, device=dev())
        checked(cp, cp.cpattn_cache_attn(d, R, cols, n, max(add + [1]), q, start, lens, table, cache, o, None, ws))
        at = 0
        for r in range(R):
            rows = slice(at, at + add[r])
            at += add[r]
            for x, t in zip((0, 1), (k, v)):
                new_rows = OC.values(*OC.quantise(f32_of(t[rows]), 32))
                kept[r][x] = np.concatenate([kept[r][x][: min(old[r], new[r])], new_rows])
            for h in range(H_q):
                ref, _, pv, _ = OC.attention(f32_of(q[rows])[:, h].astype(np.float64), kept[r][0][:, h // 4],
                                             kept[r][1][:, h // 4], np.arange(add[r]) + 1 + old[r], d.scale)
                got = o[rows, h].double().cpu().numpy()
                assert np.all(np.abs(got - ref) <= 2.0 ** -8 * (np.abs(ref) + 1.02 * pv) + 2.0 ** -12 * pv)
        old = new
    held = sum(-(-x // page) for x in old)
    assert n_free.item() == n_pages - held


def test_state_of_another_device_is_refused():
    """(a CPU tensor stands for one)"""
    c = Case(cp_mod(), n_q=[1], kv_len=[20])
    cache, k, slots = c.dev[3].cpu(), torch.zeros(2, 2, 128, dtype=torch.bfloat16, device=dev()), i32([0, 1])
    with pytest.raises(ValueError, match="current device"):
        c.cp.cpattn_cache_attn(c.d, 1, c.table.shape[1], c.qd.shape[0], 1, c.qd, *c.dev[:3], cache, c.o, c.lse, c.ws)
    with pytest.raises(ValueError, match="current device"):
        c.cp.cpattn_cache_append(c.d, 2, k, k, slots, cache)
    with pytest.raises(ValueError, match="current device"):
        c.cp.cpattn_cache_read(c.d, 2, slots, cache, k, k)
    x, ws = i32(np.zeros(8)), torch.zeros(4096, dtype=torch.uint8, device=dev())
    with pytest.raises(ValueError, match="current device"):
        c.cp.cpattn_cache_plan(c.cp.make_cache_desc(1, 1, 64, 16, 8), 2, 2, x, x, x.cpu(), *[x] * 6, 2, ws)


def test_a_captured_decoding_step():
    """plan, append, read and attention of one step in a graph, replayed token by token: the
    same cache, table and results as eager calls."""
    cp = cp_mod()
    rng = np.random.default_rng(14)
    H_q, H, D, page, R, cols, n_pages, steps = 8, 2, 128, 16, 3, 4, 12, 20
    d = cp.make_cache_desc(H_q, H, D, page, n_pages)
    first = rng.integers(1, 20, R)
    rows = to_dt(rng.normal(size=(steps, R, H_q + 2 * H, D)), "bf16").to(dev())
    prompt = to_dt(rng.normal(size=(int(first.sum()), 2 * H, D)), "bf16").to(dev())

    def server():
        s = dict(cache=torch.zeros(cp.cpattn_cache_bytes(d), dtype=torch.uint8, device=dev()),
                 table=i32(np.full((R, cols), -1)), free=i32(np.arange(n_pages)), n_free=i32([n_pages]),
                 lens=i32(np.zeros(R)), new=i32(first), start=i32(np.zeros(R + 1)), slots=i32(np.zeros(80)),
                 x=torch.zeros(R, H_q + 2 * H, D, dtype=torch.bfloat16, device=dev()),
                 o=torch.zeros(R, H_q, D, dtype=torch.bfloat16, device=dev()), lse=torch.zeros(R, H_q, device=dev()),
                 back=torch.zeros(2, R, H, D, dtype=torch.bfloat16, device=dev()),
                 ws=torch.zeros(max(cp.cpattn_cache_plan_workspace(d, R), cp.cpattn_cache_attn_workspace(d)),
                                dtype=torch.uint8, device=dev()))
        plan(s)
        cp.check(cp.cpattn_cache_append(d, prompt.shape[0], prompt[:, :H], prompt[:, H:], s["slots"], s["cache"]))
        return s

    def plan(s):
        cp.check(cp.cpattn_cache_plan(d, R, cols, s["lens"], s["new"], s["table"], s["free"], s["n_free"], s["n_free"],
                                      s["lens"], s["start"], s["slots"], 80, s["ws"]))

    def step(s):
        torch.add(s["lens"], 1, out=s["new"])
        plan(s)
        q, k, v = s["x"][:, :H_q], s["x"][:, H_q:H_q + H], s["x"][:, H_q + H:]
        cp.check(cp.cpattn_cache_append(d, R, k, v, s["slots"], s["cache"]))
        cp.check(cp.cpattn_cache_read(d, R, s["slots"], s["cache"], s["back"][0], s["back"][1]))
        cp.check(cp.cpattn_cache_attn(d, R, cols, R, 1, q, s["start"], s["lens"], s["table"], s["cache"], s["o"],
                                      s["lse"], s["ws"]))

    a, b = server(), server()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    for i in range(steps):
        for s in (a, b):
            s["x"].copy_(rows[i])
        step(a)
        g.replay()
        checked(cp, 0)
        for name in ("table", "n_free", "lens", "start", "slots", "cache", "back", "o", "lse"):
            assert torch.equal(a[name], b[name]), (i, name)
    assert a["lens"].tolist() == [int(x) + steps for x in first]


def test_ring_prompt_then_sharded_decoding():
    """A prompt through the ring; its keys and values into the caches of cp ranks, from the
    layout-order tensors; the next token attends to every rank's shard and the partial
    results are merged: the same as one cache that holds all of it."""
    cp = cp_mod()
    rng = np.random.default_rng(12)
    H_q, H, D, T, ranks, page = 8, 2, 128, 512, 4, 64
    q, k, v = (to_dt(rng.normal(size=(1, h, T, D)), "bf16").to(dev()) for h in (H_q, H, H))
    rd = cp.make_desc(1, H_q, H, T, D, ranks)
    ql, kl, vl = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    cp.check(cp.cpattn_layout_batch(cp.ZIGZAG_FWD, rd, [q, k, v], [ql, kl, vl], [H_q, H, H]))
    o, lse = torch.empty_like(ql), torch.empty(1, H_q, T, dtype=torch.float32, device=dev())
    checked(cp, cp.cpattn_ring_fwd(rd, ql, kl, vl, o, lse))
    c = T // ranks
    d = cp.make_cache_desc(H_q, H, D, page, c // page, causal=0, o_dtype="f32")
    whole = cp.make_cache_desc(H_q, H, D, page, T // page)
    big = torch.zeros(cp.cpattn_cache_bytes(whole), dtype=torch.uint8, device=dev())
    cp.check(cp.cpattn_cache_append(whole, T, k[0].transpose(0, 1), v[0].transpose(0, 1), i32(np.arange(T)), big))
    new_q = to_dt(rng.normal(size=(1, H_q, D)), "bf16").to(dev())
    ws = torch.empty(cp.cpattn_cache_attn_workspace(d), dtype=torch.uint8, device=dev())
    acc, acc_lse = torch.zeros(1, H_q, D, device=dev()), torch.full((1, H_q), -np.inf, device=dev())
    for r in range(ranks):
        mine = torch.zeros(cp.cpattn_cache_bytes(d), dtype=torch.uint8, device=dev())
        rows = slice(r * c, (r + 1) * c)   # the rank's zigzag rows, wherever they lie in the sequence
        cp.check(cp.cpattn_cache_append(d, c, kl[0, :, rows].transpose(0, 1), vl[0, :, rows].transpose(0, 1),
                                        i32(np.arange(c)), mine))
        po, pl = torch.empty(1, H_q, D, device=dev()), torch.empty(1, H_q, device=dev())
        cp.check(cp.cpattn_cache_attn(d, 1, c // page, 1, 1, new_q, i32([0, 1]), i32([c]),
                                      i32(np.arange(c // page)[None]), mine, po, pl, ws))
        cp.check(cp.cpattn_merge(H_q, D, acc, acc_lse, po, pl, acc, acc_lse))
    one, one_lse = torch.empty(1, H_q, D, dtype=torch.bfloat16, device=dev()), torch.empty(1, H_q, device=dev())
    checked(cp, cp.cpattn_cache_attn(whole, 1, T // page, 1, 1, new_q, i32([0, 1]), i32([T]),
                                     i32(np.arange(T // page)[None]), big, one, one_lse, ws))
    # both sides round P (2^-8 of sum p |v|, at most max |v| = the largest cached value), one
    # of them its result; scores within 2^-23 (D + 8) of sums of at most scale sum |q||k|
    kr, vr = torch.empty(T, H, D, dtype=torch.bfloat16, device=dev()), torch.empty(T, H, D, dtype=torch.bfloat16, device=dev())
    checked(cp, cp.cpattn_cache_read(whole, T, i32(np.arange(T)), big, kr, vr))
    for h in range(H_q):
        ref, rl, pv, size = OC.attention(f32_of(new_q[:, h]).astype(np.float64), f32_of(kr[:, h // 4]).astype(np.float64),
                                         f32_of(vr[:, h // 4]).astype(np.float64), [T], d.scale)
        ds = 2.0 ** -23 * (D + 8) * size
        tol = (2 * ds + 2.0 ** -17 + 2.0 ** -8) * pv
        assert np.all(np.abs(acc[:, h].double().cpu().numpy() - ref) <= tol)
        assert np.all(np.abs(one[:, h].double().cpu().numpy() - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))
        for got in (acc_lse, one_lse):
            assert abs(got[0, h].item() - rl[0]) <= ds + 2.0 ** -20 * (1 + abs(rl[0]))


def test_cached_prefix_through_the_ring():
    """The rows of a cached prefix, read back head-major, are the ring's keys and values."""
    cp = cp_mod()
    rng = np.random.default_rng(13)
    H, D, T, page = 2, 64, 256, 16
    d = cp.make_cache_desc(2, H, D, page, T // page + 2, group=32)
    cache = torch.zeros(cp.cpattn_cache_bytes(d), dtype=torch.uint8, device=dev())
    k, v = (to_dt(rng.normal(size=(T, H, D)), "bf16").to(dev()) for _ in range(2))
    slots = i32((rng.permutation(T // page)[:, None] * page + np.arange(page)).reshape(-1))
    cp.check(cp.cpattn_cache_append(d, T, k, v, slots, cache))
    kr, vr = (torch.empty(1, H, T, D, dtype=torch.bfloat16, device=dev()) for _ in range(2))
    checked(cp, cp.cpattn_cache_read(d, T, slots, cache, kr[0].transpose(0, 1), vr[0].transpose(0, 1)))
    ref = OC.values(*OC.quantise(f32_of(k), 32))
    assert np.array_equal(f32_of(kr[0].transpose(0, 1)), ref)
    rd = cp.make_desc(1, 2, H, T, D, 1, layout="contiguous")
    q = to_dt(rng.normal(size=(1, 2, T, D)), "bf16").to(dev())
    o, lse = torch.empty_like(q), torch.empty(1, 2, T, dtype=torch.float32, device=dev())
    checked(cp, cp.cpattn_ring_fwd(rd, q, kr, vr, o, lse))
    # the cache's own attention of the same queries over the same rows
    at = i32(slots.cpu().numpy().reshape(-1, page)[:, 0][None] // page)
    o2, lse2 = torch.empty(T, 2, D, dtype=torch.bfloat16, device=dev()), torch.empty(T, 2, device=dev())
    ws = torch.empty(cp.cpattn_cache_attn_workspace(d), dtype=torch.uint8, device=dev())
    checked(cp, cp.cpattn_cache_attn(d, 1, T // page, T, T, q[0].transpose(0, 1), i32([0, T]), i32([T]), at, cache, o2,
                                     lse2, ws))
    diff = (o2.transpose(0, 1)[None].float() - o.float()).abs()
    # each side: P rounded (2^-8 of sum p |v| <= max |v|) and its result (2^-8 |o|)
    assert diff.max().item() <= 4 * 2.0 ** -8 * vr.float().abs().max().item()
    assert (lse2.T[None] - lse).abs().max().item() <= 2.0 ** -14
