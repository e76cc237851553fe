"""GPU: norm, rotation and linear attention at the edges of what their documentation promises.
Tolerances are derived beside each test (half a step of a rounding: bf16 2^-8, float32 2^-24)."""
import numpy as np
import pytest
import torch

from gpu_helpers import cp_mod, dev
from test_gpu_layer import checked, spread_decays

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
