"""Linear attention without a GPU: what a bound on its states can tell apart."""
import numpy as np
import torch


def test_bound_on_states_tells_two_parts_from_three():
    """Weighted keys as two bf16 numbers leave an error that the bound on states (5e-7 of their norm)
    does not let pass; as three they do not."""
    rng = np.random.default_rng(0)
    T, D = 512, 32
    k, v = (torch.from_numpy(rng.normal(size=(T, D))).bfloat16().double() for _ in range(2))
    weighted = (k * torch.exp(-0.01 * torch.arange(T - 1, -1, -1).double())[:, None]).float().double()
    ref = weighted.T @ v
    parts, left, errors = torch.zeros_like(weighted), weighted.clone(), []
    for _ in range(3):
        part = left.bfloat16().double()
        parts, left = parts + part, left - part
        errors.append(((parts.T @ v - ref).norm() / ref.norm()).item())
    assert errors[0] > 1e-3 and errors[1] > 4 * 5e-7 and errors[2] < 5e-8, errors
