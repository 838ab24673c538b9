"""Shared by the tests of the log probabilities: seeded rows and derived tolerances."""
import numpy as np

U = 2.0 ** -24  # half a step of float32, relative


def np64(t):
    return t.detach().double().cpu().numpy()


def make_rows(torch, N, V, dtype, seed, masked=False, pad=0, scale=2.5, levels=0):
    """Logits [N, V] inside rows of V + pad elements, with a likely token per row."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    z = torch.randn((N, V), generator=g, device="cuda") * scale
    if levels:  # few values: many equal logits
        z = (z * levels).round() / levels
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
    z.scatter_add_(1, tokens[:, None], 12.0 * torch.rand((N, 1), generator=g, device="cuda"))
    if masked:
        z.masked_fill_(torch.rand((N, V), generator=g, device="cuda") < 0.3, float("-inf"))
    wide = torch.full((N, V + pad), 7.0, device="cuda", dtype=dtype)
    wide[:, :V] = z.to(dtype)
    return wide[:, :V], tokens


# How far the float32 parts may take the results from float64, worst case, for a row with
# p_v and d_v = z_v - max, A = sum p |d|, B = sum p d^2:
#  * a term exp(d) errs by 2.5 U |d| (the difference, its product with log2 e and that
#    constant are each rounded) + 2 U (one step of the hardware's 2^x);
#  * up to 32 terms are added in float32: 31 U; sums of those are float64;
#  * a lane rescales its sums when its maximum rises (at most once a step, 20 steps for the
#    rows here) and 6 + 2 + 6 joins follow: 2 U each, and 2.5 U of the |d| that they cover,
#    once more at most.
# So S errs by U (5 A + 101) relative, ln S by as much, and T / S (terms weighted by |d|) by
# U (5 B + 101 A) + A U (5 A + 101) <= U (10 B + 202 A) as A^2 <= B.  A result is rounded once.
def row_tolerances(z):
    """(tolerance of lse and ln S, tolerance of the entropy) per row, before rounding."""
    with np.errstate(invalid="ignore", over="ignore"):
        m = np.where(np.isfinite(z), z, -np.inf).max(axis=1, initial=-np.inf)
        m = np.where(np.isfinite(m), m, 0.0)
        d = np.maximum(z - m[:, None], -200.0)
        p = np.exp(d)
        s = np.maximum(p.sum(1), 1e-300)
        A, B = (p * -d).sum(1) / s, (p * d * d).sum(1) / s
    lse = U * (5 * A + 101)
    return np.nan_to_num(lse, nan=1e-5), np.nan_to_num(lse + U * (10 * B + 202 * A), nan=1e-4)


def close(name, got, want, tol):
    """|got - want| <= tol + one rounding to float32, NaN and infinities equal."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, name
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{name}: NaN places"
    fin = np.isfinite(want)
    assert np.array_equal(got[~fin & ~np.isnan(want)], want[~fin & ~np.isnan(want)]), f"{name}: inf"
    off = np.abs(got - want)[fin] - np.broadcast_to(tol, want.shape)[fin] - U * np.abs(want)[fin]
    assert off.size == 0 or off.max() <= 0, f"{name}: {off.max():.3g} past the tolerance"


def check_forward(outs, z, f, top):
    """Outputs of token_logprobs (tensors) against the float64 dict f for logits z."""
    tl, th = row_tolerances(z)
    close("logp", np64(outs[0]), f["logp"], tl)
    close("entropy", np64(outs[1]), f["entropy"], th)
    close("lse", np64(outs[2]), f["lse"], tl)
    if top:
        assert np.array_equal(outs[3].cpu().numpy(), f["top_idx"]), "top_idx"
        close("top_logp", np64(outs[4]), f["top_logp"], tl[:, None])


def grad_tolerance(z, dz, g, tokens, entropy, half_step):
    """Per-element tolerance of dz: ln p errs by U (5 A + 101 + 3 (|ln p| + ln S)), so p by as
    much relative; the bracket (gz - gl - ge (ln p + H)) by that times |ge| and three
    roundings of its parts; the result is rounded to its type (half_step)."""
    tl, th = row_tolerances(z)
    with np.errstate(invalid="ignore", over="ignore"):
        m = np.where(np.isfinite(z), z, -np.inf).max(axis=1, initial=-np.inf)
        m = np.where(np.isfinite(m), m, 0.0)
        s = np.exp(np.maximum(z - m[:, None], -800.0)).sum(1)
        lp = np.maximum(z - m[:, None] - np.log(np.maximum(s, 1e-300))[:, None], -200.0)
    lp = np.nan_to_num(lp)
    p = np.exp(lp)
    gl, ge, gz = (np.zeros(len(z)) if x is None else np.abs(x) for x in g)
    H = np.nan_to_num(np.abs(entropy))
    e_lp = tl[:, None] + U * 3 * (np.abs(lp) + np.log(np.maximum(s, 1.0))[:, None])
    size = (gz + gl)[:, None] + ge[:, None] * (np.abs(lp) + H[:, None])
    tol = p * (size * (e_lp + 6 * U) + ge[:, None] * (e_lp + th[:, None]))
    hot = np.zeros_like(p)
    ok = (tokens >= 0) & (tokens < z.shape[1])
    hot[np.arange(len(z))[ok], tokens[ok]] = gl[ok] * 2 * U
    return tol + hot + half_step * np.abs(np.nan_to_num(dz)) + 1e-38
