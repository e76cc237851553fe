"""The 4-bit key/value cache without a GPU: the oracle's own pins, and what the calls refuse."""
import numpy as np
import pytest

from conftest import ROOT  # noqa: F401
from oracle import cache as OC

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
def test_bf16_rounding_matches_torch():
    import torch
    x = np.random.default_rng(0).normal(size=4096).astype(np.float32)
    x = np.concatenate([x, np.float32([0.0, -0.0, 1.00390625, 1.01171875, 3.0, -2.0 ** 100])])
    ref = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert np.array_equal(OC.round_bf16(x), ref)
    assert np.array_equal(OC.bits_bf16(OC.bf16_bits(ref)), ref)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("shift", [0.0, 40.0])
def test_quantised_values_are_near(group, shift):
    x = (np.random.default_rng(1).normal(size=(50, 128)) + shift).astype(np.float32)
    codes, a, z = OC.quantise(x, group)
    y = OC.values(codes, a, z)
    assert codes.min() >= 0 and codes.max() <= 15
    # half a step a / 32; the ends of the range move with the rounding of z and a (half a
    # bf16 step of each, 2^-8); the value's own rounding to bf16, 2^-8
    a_, z_ = np.repeat(a, group, 1), np.repeat(z, group, 1)
    assert np.all(np.abs(y - x) <= a_ / 32 + 2.0 ** -8 * (np.abs(z_) + 2 * a_ + np.abs(y)))
    # the least and the most of a group take the end codes unless rounding moved the ends
    assert (codes.reshape(50, -1, group).min(-1) <= 1).all()


def test_constant_and_tiny_groups():
    x = np.full((1, 64), 0.75, np.float32)
    codes, a, z = OC.quantise(x, 32)
    assert not codes.any() and not a.any() and np.array_equal(OC.values(codes, a, z), x)
    x[0, 5] = 0.75 + 2.0 ** -20
    codes, a, z = OC.quantise(x, 32)
    assert np.all(np.abs(OC.values(codes, a, z) - x) <= 2.0 ** -8)


def test_rows_survive_the_layout():
    rng = np.random.default_rng(2)
    D, group, page, H = 64, 32, 48, 3
    cache = rng.integers(0, 256, (4, H, page // 16 * 2 * OC.half_tile(D, group)), dtype=np.uint8)
    before = cache.copy()
    k, v = rng.normal(size=(2, 20, H, D)).astype(np.float32)
    slots = rng.permutation(4 * page)[:20]
    slots[3], slots[7] = -1, 4 * page
    OC.append(cache, page, group, k, v, slots)
    for x, y in zip((k, v), OC.read(cache, page, group, D, slots)):
        ref = OC.values(*OC.quantise(x, group))
        ref[[3, 7]] = 0
        assert np.array_equal(y, ref)
    other = [s for s in range(4 * page) if s not in set(slots.tolist())]
    for x, y in zip(OC.read(before, page, group, D, other), OC.read(cache, page, group, D, other)):
        assert np.array_equal(x, y, equal_nan=True)


def test_plan_hands_every_page_out_once():
    rng = np.random.default_rng(3)
    page, R, cols, n_pages = 16, 9, 8, 60
    ids = rng.permutation(n_pages)
    old = rng.integers(0, 100, R)
    used = -(-old // page)
    table = np.full((R, cols), -1)
    at = 0
    for r in range(R):
        table[r, : used[r]] = ids[at: at + used[r]]
        at += used[r]
    free = np.full(n_pages, -1)
    free[: n_pages - at] = ids[at:]
    new = np.clip(old + rng.integers(-60, 60, R), 0, cols * page)
    t, f, nf, lens, start, slots = OC.plan(page, old, new, table, free, n_pages - at, 400)
    held = np.concatenate([t[r, : -(-lens[r] // page)] for r in range(R)])
    assert sorted(np.concatenate([held, f[:nf]])) == list(range(n_pages))
    live = slots[slots >= 0]
    assert len(set(live.tolist())) == len(live)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------
def _desc(cp, **kw):
    base = dict(H_q=8, H_kv=2, D=128, page=64, n_pages=100)
    base.update(kw)
    return cp.make_cache_desc(**base)


BAD_DESC = [
    (dict(H_q=7), 1), (dict(H_kv=0), 1), (dict(H_q=-8), 1), (dict(D=96), 2), (dict(D=0), 1),
    (dict(group=16), 1), (dict(D=64, group=128), 1), (dict(page=0), 1), (dict(page=24), 1),
    (dict(page=-16), 1), (dict(n_pages=0), 1), (dict(n_pages=1 << 30), 2), (dict(dtype=7), 1),
    (dict(dtype="f32", o_dtype="bf16"), 1), (dict(o_dtype=9), 1), (dict(scale=0.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(causal=2), 1),
    (dict(debug_fault=-1), 1), (dict(debug_fault=4), 1),
]


@pytest.mark.parametrize("kw,code", BAD_DESC)
def test_bad_descriptors(cp, kw, code):
    d = _desc(cp, **kw)
    big = 1 << 40
    assert cp.cpattn_cache_bytes(d) == 0
    assert cp.cpattn_cache_plan_workspace(d, 4) == 0
    assert cp.cpattn_cache_attn_workspace(d) == 0
    assert cp.cpattn_cache_plan(d, 4, 4, *[FAKE] * 9, 0, FAKE, big, 0) == code
    assert cp.cpattn_cache_append(d, 4, FAKE, FAKE, FAKE, FAKE, 0) == code
    assert cp.cpattn_cache_read(d, 4, FAKE, FAKE, FAKE, FAKE, 0) == code
    assert cp.cpattn_cache_attn(d, 4, 4, 4, 1, *[FAKE] * 8, big, 0) == code


def test_sizes(cp):
    assert cp.cpattn_cache_bytes(_desc(cp)) == 100 * 2 * 64 * 144
    assert cp.cpattn_cache_bytes(_desc(cp, D=64, group=32, page=48)) == 100 * 2 * 48 * 80
    # beyond 32 bits
    assert cp.cpattn_cache_bytes(_desc(cp, H_kv=8, n_pages=1 << 24)) == (1 << 24) * 8 * 64 * 144


def test_plan_refuses(cp):
    d = _desc(cp)
    need = cp.cpattn_cache_plan_workspace(d, 4)
    assert need > 0 and need % 256 == 0

    def call(n_req=4, max_pages=4, at=None, n_slots=4, ws=FAKE, size=need):
        p = [FAKE] * 9
        if at is not None:
            p[at[0]] = at[1]
        return cp.cpattn_cache_plan(d, n_req, max_pages, *p, n_slots, ws, size, 0)

    assert call(n_req=0) == 1 and call(n_req=-1) == 1 and call(max_pages=0) == 1 and call(n_slots=-1) == 1
    for i in range(9):
        assert call(at=(i, 0)) == 1
        assert call(at=(i, FAKE + 2)) == 1
    assert call(ws=0) == 1 and call(ws=FAKE + 8) == 1 and call(size=need - 1) == 1
    assert call(max_pages=1 << 30) == 2                       # n_req * max_pages past 32 bits
    assert call(n_req=1, max_pages=1 << 26, size=1 << 30) == 2   # a row's tokens past 32 bits
    # sums of a length and a page, or of a count and a loop's step, past 32 bits
    assert call(n_req=1, max_pages=(1 << 25) - 1, size=1 << 30) == 2
    assert call(n_req=1, max_pages=(1 << 24) + 1, size=1 << 30) == 2
    assert call(n_req=(1 << 24) + 1, max_pages=1, size=1 << 40) == 2


def test_rows_refuse(cp):
    d = _desc(cp)
    for call in (lambda n, k, v, s, c: cp.cpattn_cache_append(d, n, k, v, s, c, 0),
                 lambda n, k, v, s, c: cp.cpattn_cache_read(d, n, s, c, k, v, 0)):
        assert call(0, 0, 0, 0, 0) == 0  # nothing to do
        assert call(-1, FAKE, FAKE, FAKE, FAKE) == 1
        for i in range(4):
            for bad in (0, FAKE + 2):
                p = [FAKE] * 4
                p[i] = bad
                assert call(4, *p) == 1
    lib = cp._lib
    import ctypes
    for ts, hs in ((128, 128 + 4), (100, 128), (1024, 64), (-1024, 128), (0, 128), (260, 128)):
        assert lib.cpattn_cache_append(ctypes.byref(d), 4, FAKE, ts, hs, FAKE, 256, 128, FAKE, FAKE, 0) == 1
        assert lib.cpattn_cache_append(ctypes.byref(d), 4, FAKE, 256, 128, FAKE, ts, hs, FAKE, FAKE, 0) == 1
        assert lib.cpattn_cache_read(ctypes.byref(d), 4, FAKE, FAKE, FAKE, ts, hs, FAKE, 256, 128, 0) == 1
        assert lib.cpattn_cache_read(ctypes.byref(d), 4, FAKE, FAKE, FAKE, 256, 128, FAKE, ts, hs, 0) == 1


def test_attention_refuses(cp):
    d = _desc(cp)
    need = cp.cpattn_cache_attn_workspace(d)
    assert need > 0 and need % 256 == 0

    def call(n_req=4, max_pages=4, n=4, max_q=1, at=None, size=need):
        p = [FAKE] * 8
        if at is not None:
            p[at[0]] = at[1]
        return cp.cpattn_cache_attn(d, n_req, max_pages, n, max_q, *p, size, 0)

    assert call(n=0) == 0  # nothing to do
    assert call(n_req=0) == 1 and call(max_pages=0) == 1 and call(n=-1) == 1 and call(max_q=0) == 1
    for i in (0, 1, 2, 3, 4, 5, 7):  # q, q_start, kv_len, table, cache, o, workspace
        assert call(at=(i, 0)) == 1
        assert call(at=(i, FAKE + 2)) == 1
    assert call(at=(6, FAKE + 2)) == 1  # lse may be null, not misaligned
    assert call(size=need - 1) == 1
    assert call(max_pages=1 << 30) == 2
    assert call(n_req=1, max_pages=1 << 26) == 2
    assert call(n_req=1, max_pages=(1 << 25) - 1) == 2
    assert call(n_req=1, max_pages=(1 << 24) + 1) == 2
    assert call(n_req=(1 << 24) + 1, max_pages=1) == 2
    assert call(n=1 << 29) == 2


def test_binding_checks_tensors(cp):
    import torch
    d = _desc(cp)
    i32 = torch.zeros(64, dtype=torch.int32)
    k = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cache = torch.zeros(cp.cpattn_cache_bytes(d), dtype=torch.uint8)
    with pytest.raises(ValueError):
        cp.cpattn_cache_append(d, 4, k, k, i32.long(), cache, 0)
    with pytest.raises(ValueError):
        cp.cpattn_cache_append(d, 5, k, k, i32, cache, 0)
    with pytest.raises(ValueError):
        cp.cpattn_cache_append(d, 4, k.float(), k, i32, cache, 0)
    with pytest.raises(ValueError):
        cp.cpattn_cache_append(d, 4, k.transpose(1, 2), k, i32, cache, 0)
    with pytest.raises(ValueError):
        cp.cpattn_cache_append(d, 4, k, k, i32, cache[:-1], 0)
    with pytest.raises(ValueError):
        cp.cpattn_cache_plan(d, 4, 20, i32, i32, i32, i32, i32, i32, i32, i32, i32, 4, cache, 1 << 20, 0)
    q = torch.zeros(4, 8, 128, dtype=torch.bfloat16)
    o, lse = torch.zeros_like(q), torch.zeros(4, 8)
    ok = [q, i32, i32, i32, cache, o, lse, cache]
    for at, bad in ((0, q.float()), (5, o.float()), (5, o[:3]), (6, lse.double()), (6, lse[:3]), (1, i32[:2])):
        args = list(ok)
        args[at] = bad
        with pytest.raises(ValueError):
            cp.cpattn_cache_attn(d, 4, 2, 4, 1, *args, 1 << 30, 0)


def test_binding_checks_every_tensors_device(cp, monkeypatch):
    """Each argument of each call as the only tensor, a CPU one where device 0 is current."""
    import torch
    monkeypatch.setattr(cp, "_here", lambda: 0)
    d = _desc(cp)
    i32 = torch.zeros(128, dtype=torch.int32)
    k, q = (torch.zeros(4, h, 128, dtype=torch.bfloat16) for h in (2, 8))
    cache, ws = torch.zeros(cp.cpattn_cache_bytes(d), dtype=torch.uint8), torch.zeros(1 << 20, dtype=torch.uint8)
    calls = [(lambda a: cp.cpattn_cache_plan(d, 4, 2, *a[:9], 4, a[9], 1 << 20, 0), [i32] * 9 + [ws]),
             (lambda a: cp.cpattn_cache_append(d, 4, *a, 0), [k, k, i32, cache]),
             (lambda a: cp.cpattn_cache_read(d, 4, *a, 0), [i32, cache, k, k]),
             (lambda a: cp.cpattn_cache_attn(d, 4, 2, 4, 1, *a, 1 << 30, 0),
              [q, i32, i32, i32, cache, q, torch.zeros(4, 8), ws])]
    for call, tensors in calls:
        for i, t in enumerate(tensors):
            with pytest.raises(ValueError, match="current device"):
                call([t if j == i else FAKE for j in range(len(tensors))])


def test_range_has_a_status_string(cp):
    assert cp.cpattn_status_string(cp.ERR_RANGE) not in ("", "unknown status")
