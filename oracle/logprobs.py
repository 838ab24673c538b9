"""Float64 definitions of the log probabilities of given tokens, their entropy, the largest
alternatives and the gradient, and of gradient clipping: plain numpy, no code shared with
the HIP path.

Row n of logits z with token t (negative: none):
  lse = log sum exp z,  logp = z[t] - lse (0 without a token),  H = -sum p log p,
  dz = p (gz - gl - ge (log p + H)) + gl [v = t].
A row with no finite logit: lse = logp = -inf, H = 0, dz = 0.  A row with NaN or +inf: NaN,
alternatives -1.  A token at or past the vocabulary: logp and the gradient row NaN."""
import numpy as np


def _row_state(z):
    """(bad rows, empty rows, lse, ln p); ln p from differences to the maximum, as the sum
    m + ln S of a row near the lowest value would lose ln S."""
    bad = ~(z < np.inf).all(axis=1)
    empty = ~bad & (z == -np.inf).all(axis=1)
    m = np.where(bad | empty, 0.0, np.where(np.isfinite(z), z, -np.inf).max(axis=1))
    with np.errstate(divide="ignore", invalid="ignore"):
        ln_s = np.log(np.exp(z - m[:, None]).sum(axis=1))
        lp = (z - m[:, None]) - np.where(empty, 0.0, ln_s)[:, None]
    lse = np.where(empty, -np.inf, m + ln_s)
    lse[bad] = np.nan
    lp[bad] = np.nan
    return bad, empty, lse, lp


def forward(z, tokens, top=0):
    """dict of logp, entropy, lse [N] and, with top, top_idx, top_logp [N, top] (float64)."""
    z = np.asarray(z, np.float64)
    N, V = z.shape
    bad, empty, lse, lp = _row_state(z)
    with np.errstate(invalid="ignore"):
        p = np.exp(lp)
        H = -np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0).sum(axis=1)
    H = np.where(empty, 0.0, H)
    H[bad] = np.nan
    logp = np.zeros(N)
    for n, t in enumerate(np.asarray(tokens)):
        if bad[n] or t >= V:
            logp[n] = np.nan
        elif t >= 0:
            logp[n] = lp[n, t]
    out = dict(logp=logp, entropy=H, lse=lse)
    if top:
        order = np.argsort(np.where(bad[:, None], 0.0, -z), axis=1, kind="stable")[:, :top]
        out["top_idx"] = np.where(bad[:, None], -1, order)
        tl = np.take_along_axis(lp, order, axis=1)
        tl[bad] = np.nan
        out["top_logp"] = tl
    return out


def gradient(z, tokens, g_logp=None, g_entropy=None, g_lse=None):
    """dz [N, V] (float64) for upstream gradients of logp, entropy and lse."""
    z = np.asarray(z, np.float64)
    N, V = z.shape
    tokens = np.asarray(tokens)
    zero = np.zeros(N)
    gl, ge, gz = (zero if g is None else np.asarray(g, np.float64) for g in (g_logp, g_entropy, g_lse))
    gl = np.where(tokens < 0, 0.0, gl)
    bad, empty, _, lp = _row_state(z)
    f = forward(z, tokens)
    with np.errstate(invalid="ignore"):
        p = np.exp(lp)
        inner = np.where(p > 0, lp, 0.0) + f["entropy"][:, None]
        dz = p * ((gz - gl)[:, None] - ge[:, None] * inner)
    for n in range(N):
        if 0 <= tokens[n] < V:
            dz[n, tokens[n]] += gl[n]
    dz[empty] = 0.0
    dz[bad | (tokens >= V)] = np.nan
    return dz


def head_forward(h, W, tokens):
    return forward(np.asarray(h, np.float64) @ np.asarray(W, np.float64).T, tokens)


def head_gradient(h, W, tokens, g_logp=None, g_entropy=None, g_lse=None):
    """(dh, dW) in float64 for z = h W^T."""
    h, W = np.asarray(h, np.float64), np.asarray(W, np.float64)
    dz = gradient(h @ W.T, tokens, g_logp, g_entropy, g_lse)
    return dz @ W, dz.T @ h


def clip(grads, max_norm):
    """(norm, clipped) of a list of arrays: scaled by max_norm / norm where the finite norm
    exceeds max_norm, else as they were."""
    norm = float(np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads)))
    s = max_norm / norm if np.isfinite(norm) and norm > max_norm else 1.0
    return norm, [np.asarray(g, np.float64) * s for g in grads]
