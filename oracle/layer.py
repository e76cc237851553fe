"""Norm, rotation and linear attention in plain numpy, float64: the definitions of what stands
around and beside softmax attention.  Test infrastructure only.

Tensors are [B, H, T, D]; linear attention takes its tokens in natural order."""
import numpy as np


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------
def turn(x, pos, inv_freq, rot, pairing, inverse=False):
    """Rotates the first rot channels of x at positions pos ([T] or [B, T])."""
    pos = np.asarray(pos, np.float64)
    t = np.atleast_2d(pos)[:, None, :, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(t), np.sin(t) * (-1 if inverse else 1)
    y = np.array(x, np.float64)
    if pairing == "halves":
        i, j = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        i, j = slice(0, rot, 2), slice(1, rot, 2)
    a, b = np.array(x[..., i], np.float64), np.array(x[..., j], np.float64)
    y[..., i], y[..., j] = a * c - b * s, a * s + b * c
    return y


def rotate_fwd(x, w, eps, pos, inv_freq, rot, pairing):
    """w: the norm's weights, None for a rotation alone."""
    x = np.asarray(x, np.float64)
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return turn(x, pos, inv_freq, rot, pairing)


def rotate_bwd(x, w, eps, pos, inv_freq, rot, pairing, dy):
    """Gradients of x and (with the norm) of w."""
    g = turn(dy, pos, inv_freq, rot, pairing, inverse=True)
    if w is None:
        return g, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n, h = x * r, g * w
    return r * (h - n * (h * n).mean(-1, keepdims=True)), (g * n).sum((0, 1, 2))


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------
def decays(log_decay):
    """The decay of every head; a positive or NaN logarithm counts as 0."""
    ld = np.array(log_decay, np.float64)
    ld[np.isnan(ld)] = 0
    return np.exp(np.minimum(ld, 0))


def _shared(x, H):
    return np.repeat(np.asarray(x, np.float64), H // x.shape[1], 1)


def linear_fwd(q, k, v, log_decay, scale, S0=None, lengths=None):
    """S_t = r S_(t-1) + k_t v_t^T, o_t = scale q_t S_t.  Returns o (0 behind a row's length) and
    the states behind the last token."""
    B, H, T, D = q.shape
    q, k, v, r = np.asarray(q, np.float64), _shared(k, H), _shared(v, H), decays(log_decay)[:, None, None]
    o = np.zeros((B, H, T, D))
    S = np.zeros((B, H, D, D)) if S0 is None else np.array(S0, np.float64)
    n = [T] * B if lengths is None else [min(max(int(x), 0), T) for x in lengths]
    for b in range(B):
        for t in range(n[b]):
            S[b] = r * S[b] + k[b, :, t, :, None] * v[b, :, t, None, :]
            o[b, :, t] = scale * np.einsum("hd,hde->he", q[b, :, t], S[b])
    return o, S


def linear_bwd(q, k, v, log_decay, scale, do, S0=None, dS1=None):
    """dq, dk, dv (summed over the query heads of a key head) and the gradient of S0."""
    B, H, T, D = q.shape
    G = k.shape[1]
    q, do, r = np.asarray(q, np.float64), np.asarray(do, np.float64), decays(log_decay)[:, None, None]
    k, v = _shared(k, H), _shared(v, H)
    states = np.zeros((T + 1, B, H, D, D))
    if S0 is not None:
        states[0] = S0
    for t in range(T):
        states[t + 1] = r * states[t] + k[:, :, t, :, None] * v[:, :, t, None, :]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dS = np.zeros((B, H, D, D)) if dS1 is None else np.array(dS1, np.float64)
    for t in reversed(range(T)):
        dS = dS + scale * q[:, :, t, :, None] * do[:, :, t, None, :]
        dq[:, :, t] = scale * np.einsum("bhde,bhe->bhd", states[t + 1], do[:, :, t])
        dk[:, :, t] = np.einsum("bhde,bhe->bhd", dS, v[:, :, t])
        dv[:, :, t] = np.einsum("bhde,bhd->bhe", dS, k[:, :, t])
        dS = r * dS
    group = lambda x: x.reshape(B, G, H // G, T, D).sum(2)  # noqa: E731
    return dq, group(dk), group(dv), dS


def linear_step(q, k, v, log_decay, scale, S):
    """One token: q [n, H, D], k and v [n, H_kv, D], S [n, H, D, D]."""
    H = q.shape[1]
    k, v = _shared(k, H), _shared(v, H)
    S = decays(log_decay)[:, None, None] * np.asarray(S, np.float64) + k[..., None] * v[..., None, :]
    return scale * np.einsum("nhd,nhde->nhe", np.asarray(q, np.float64), S), S
