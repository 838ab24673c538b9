"""Log probabilities of given tokens from hidden states on the GPU, and their gradients,
against the float64 definitions; the operators together as a training step uses them."""
import numpy as np
import pytest

import output_head_kl_amd as kd
from logprobs_util import close, np64, row_tolerances
from oracle import logprobs as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(torch, N, d, V, dtype, seed, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    h = torch.randn((N, d), generator=g, device="cuda").to(dt)
    W = (torch.randn((V, d), generator=g, device="cuda") * (scale / d ** 0.5)).to(dt)
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
    if N > 2:
        tokens[1] = -1
        tokens[2] = V - 1
    return h, W, tokens


def z_tolerance(h, W):
    """z is a float32 sum of d products (exact for bf16, rounded for float32): worst case
    (d + 1) U sum |h W|; the sums' errors are of random sign, so sqrt(d + 1) of them with a
    factor of 6 bounds every one of the elements compared here."""
    d = h.shape[1]
    return 6 * (d + 1) ** 0.5 * U * np.sqrt((h ** 2).sum(1)[:, None] * (W ** 2).sum(1)[None]).max(1)


def check_forward(h, W, tokens, outs):
    """A shift of z by dz changes lse and the given token's z by at most dz each, the entropy
    by at most sum p |ln p + H| dz <= 2 (H + 1) dz or so for the rows here (A bounds it)."""
    hn, Wn, tk = np64(h), np64(W), tokens.cpu().numpy()
    z = hn @ Wn.T
    f = ref.forward(z, tk)
    ez = z_tolerance(hn, Wn)
    tl, th = row_tolerances(z)
    # the reference point of a partial is max * log2 e rounded: U |max| more
    shift = 4 * U * np.abs(z).max(1)
    close("logp", np64(outs[0]), f["logp"], tl + 2 * ez + shift)
    A = np.abs(z - z.max(1)[:, None])
    p = np.exp(z - f["lse"][:, None])
    close("entropy", np64(outs[1]), f["entropy"], th + (p * (A + f["entropy"][:, None] + 2)).sum(1) * 2 * (ez + shift))
    close("lse", np64(outs[2]), f["lse"], tl + ez + shift)
    return f


def check_grad(name, got, want, dtype):
    """bf16: dz is rounded once (2^-9 of its size at most, so 2^-9 / sqrt 3 or less in the
    2-norm as roundings are spread evenly), its sums keep that in the 2-norm, and the result
    is rounded once more: 2 * 2^-9; 2^-7 leaves room for cancelling sums.  float32: z's error
    of about 1e-6 |z| <= 1e-5 enters p and so dz relatively, with the sums' own sqrt(n) U."""
    got, want = np64(got), np.asarray(want)
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
    assert rel <= (2.0 ** -7 if dtype == "bf16" else 1e-5), f"{name}: {rel:.3g}"


SIZES = [(1, 8, 1, 2048), (1, 64, 2, 2048), (3, 64, 383, 2048), (5, 72, 385, 2), (17, 264, 3001, 2048),
         (1, 512, 20000, 2048), (64, 256, 5003, 2048), (65, 256, 5003, 64), (300, 136, 2050, 128),
         (700, 264, 3001, 300), (33, 72, 66001, 2048), (20, 264, 70000, 2048), (64, 40, 65537, 64),
         (16, 136, 66000, 2048)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,d,V,chunk", SIZES)
def test_forward(torch_cuda, dtype, N, d, V, chunk):
    torch = torch_cuda
    h, W, tokens = make(torch, N, d, V, dtype, 3 * N + V)
    outs = kd.head_logprobs(h, W, tokens, chunk=chunk)
    check_forward(h, W, tokens, outs)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,d,V,chunk", [s for s in SIZES if s[2] > 2])
@pytest.mark.parametrize("which", ["logp", "all"])
def test_gradients(torch_cuda, dtype, N, d, V, chunk, which):
    torch = torch_cuda
    h, W, tokens = make(torch, N, d, V, dtype, 5 * N + V)
    g = torch.Generator(device="cuda").manual_seed(9)
    up = [torch.randn(N, generator=g, device="cuda") if which == "all" or n == 0 else None
          for n in range(3)]
    hx, wx = h.detach().requires_grad_(), W.detach().requires_grad_()
    outs = kd.head_logprobs(hx, wx, tokens, chunk=chunk)
    used = [(o, k) for o, k in zip(outs, up) if k is not None]
    torch.autograd.backward([o for o, _ in used], [k for _, k in used])
    dh, dW = ref.head_gradient(np64(h), np64(W), tokens.cpu().numpy(),
                               *[None if k is None else np64(k) for k in up])
    assert hx.grad.dtype == h.dtype and wx.grad.dtype == W.dtype
    check_grad("dh", hx.grad, dh, dtype)
    check_grad("dW", wx.grad, dW, dtype)
    if N > 2 and which == "logp":
        assert (hx.grad[1] == 0).all()  # no token: no gradient


@pytest.mark.parametrize("N,d,V,chunk", [
    (300, 72, 70001, 2048),  # vocabulary tiles of 384 rows, a ragged last one
    (700, 264, 40000, 300),  # the same in three chunks, the last of 100 rows
    (1100, 264, 2050, 1100),  # dh from W or a copy of it, 264 hidden units
    (1100, 512, 2050, 600),  # two chunks of different length
    (1030, 1000, 1999, 515),
    (4200, 264, 1111, 2100),  # above 4096 tokens dh always reads a copy of W
    (4200, 512, 777, 1500)])
def test_tiles_of_both_heights(torch_cuda, N, d, V, chunk):
    """bf16 above 64 tokens: the products choose 256 or 384 rows of W (or of its copy) a tile."""
    test_forward(torch_cuda, "bf16", N, d, V, chunk)
    test_gradients(torch_cuda, "bf16", N, d, V, chunk, "all")


@pytest.mark.parametrize("N,d,V,chunk", [
    (1000, 1000, 16380, 4096),  # tiles of 128 x 128 in all four products
    (300, 72, 70001, 150),  # of 64 x 64, in two chunks
    (1000, 264, 16380, 512)])  # of both, the last chunk shorter
def test_float32_tiles_of_both_sizes(torch_cuda, N, d, V, chunk):
    test_forward(torch_cuda, "f32", N, d, V, chunk)
    test_gradients(torch_cuda, "f32", N, d, V, chunk, "all")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,d,V", [(300, 8, 1), (300, 64, 2), (70, 8, 5), (65, 72, 40), (1, 8, 1),
                                   (64, 16, 17)])
def test_vocabularies_smaller_than_a_tile(torch_cuda, dtype, N, d, V):
    test_forward(torch_cuda, dtype, N, d, V, 4096)
    if V > 2:
        test_gradients(torch_cuda, dtype, N, d, V, 4096, "all")


@pytest.mark.parametrize("dw", ["bf16", "f32"])
@pytest.mark.parametrize("N,d,V", [(1, 8, 3), (1, 1000, 513), (5, 136, 2050), (16, 520, 700),
                                   (17, 264, 3001), (33, 1032, 1111), (48, 64, 20000),
                                   (64, 264, 5003)])
def test_few_tokens_gradients_are_rounded_once(torch_cuda, N, d, V, dw):
    """bf16, up to 64 tokens: dz enters the products to 2^-16 of its size (a bf16 number and
    the bf16 of what it leaves), so an element of dh or dW is off by one rounding to its type
    plus that, z's own error through p, and the float32 sums' (of random sign, so 6 sqrt n U of
    the terms' sizes for n of them)."""
    torch = torch_cuda
    h, W, tokens = make(torch, N, d, V, "bf16", 77 + N)
    g = torch.Generator(device="cuda").manual_seed(4)
    gl, ge, gz = (torch.randn(N, generator=g, device="cuda") for _ in range(3))
    outs = kd._ops._head_logprobs(h, W, tokens, 4096, None, None, True)
    dt = torch.bfloat16 if dw == "bf16" else torch.float32
    dh, dW = kd.head_logprobs_bwd(h, W, tokens, outs[1], outs[0][1], gl, ge, gz, dW_dtype=dt)
    assert dW.dtype == dt
    hn, Wn, tk = np64(h), np64(W), tokens.cpu().numpy()
    z = hn @ Wn.T
    f = ref.forward(z, tk)
    dz = ref.gradient(z, tk, np64(gl), np64(ge), np64(gz))
    lp = z - f["lse"][:, None]
    tl, th = row_tolerances(z)
    ez = z_tolerance(hn, Wn) + 4 * U * np.abs(z).max(1)
    size = (np.abs(np64(gl)) + np.abs(np64(gz)))[:, None] + \
        np.abs(np64(ge))[:, None] * (np.abs(lp) + f["entropy"][:, None] + 1)
    A = (np.exp(lp) * np.abs(z - z.max(1)[:, None])).sum(1) + f["entropy"] + 2
    err = np.exp(lp) * size * (2 * ez * A + tl + th + 16 * U)[:, None] + 2.0 ** -16 * np.abs(dz)
    err[np.arange(N)[tk >= 0], tk[tk >= 0]] += 2 * U * np.abs(np64(gl))[tk >= 0]
    mag = np.abs(dz) + err
    for name, got, want, e, half in (
            ("dh", dh, dz @ Wn, err @ np.abs(Wn) + 6 * V ** 0.5 * U * (mag @ np.abs(Wn)), 2.0 ** -8),
            ("dW", dW, dz.T @ hn, err.T @ np.abs(hn) + 6 * (2 * N) ** 0.5 * U * (mag.T @ np.abs(hn)),
             2.0 ** -8 if dw == "bf16" else U)):
        off = np.abs(np64(got) - want) - half * (np.abs(want) + e) - e
        assert off.max() <= 0, f"{name}: {off.max():.3g} past the tolerance"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 70])
def test_heads_past_32_bit_offsets(torch_cuda, dtype, N):
    """W and dW of 2.17e9 elements; the reference is float64 on the GPU, in parts of W."""
    torch = torch_cuda
    d, V, part = 4096, 530000, 53000
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(8)
    h = torch.randn((N, d), generator=g, device="cuda").to(dt)
    W = torch.empty((V, d), dtype=dt, device="cuda")
    for v in range(0, V, part):
        W[v:v + part] = torch.randn((part, d), generator=g, device="cuda") * (2 / d ** 0.5)
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda")
    tokens[0], tokens[1], tokens[2] = V - 1, -1, V - 4000
    up = torch.randn(N, generator=g, device="cuda")
    hx, wx = h.detach().requires_grad_(), W.detach().requires_grad_()
    outs = kd.head_logprobs(hx, wx, tokens)
    dh, dW = torch.autograd.grad(outs[0], (hx, wx), up)
    z = torch.cat([h.double() @ W[v:v + part].double().t() for v in range(0, V, part)], 1)
    lse = z.logsumexp(1)
    ez = 6 * (d + 1) ** 0.5 * U * float((h.double().norm(dim=1)[:, None] * 2.3).max())
    given = tokens >= 0
    logp = torch.where(given, z.gather(1, tokens.clamp(min=0)[:, None])[:, 0] - lse, 0.0)
    assert (outs[2].double() - lse).abs().max().item() <= ez + 1e-5
    assert (outs[0].double() - logp).abs().max().item() <= 2 * ez + 2e-5
    dz = -(z - lse[:, None]).exp() * (up.double() * given)[:, None]
    dz[given.nonzero()[:, 0], tokens[given]] += up.double()[given]
    want = sum(dz[:, v:v + part] @ W[v:v + part].double() for v in range(0, V, part))
    check_grad("dh", dh, np64(want), dtype)
    for rows in (slice(V - 4096, V), slice(260000, 264000), slice(0, 500)):
        check_grad("dW", dW[rows], np64(dz[:, rows].t() @ h.double()), dtype)


def test_infinite_logits_make_the_row_invalid(torch_cuda):
    """An infinite weight: -inf or +inf logits, so NaN in the row's results, status set."""
    torch = torch_cuda
    for N, V in ((3, 500), (3, 70000), (300, 500)):
        for sign in (-1.0, 1.0):
            h, W, tokens = make(torch, N, 64, V, "bf16", 5)
            h[:, 0] = 1.0
            W[V // 2, 0] = sign * float("inf")
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            for out in kd.head_logprobs(h, W, tokens, status=status):
                assert out.isnan().all(), (N, V, sign)
            assert status.item() == 2


@pytest.mark.parametrize("size", [9.0, 16.0])
def test_confident_tokens_keep_their_small_gradients(torch_cuda, size):
    """p of the given token near one: its dz = g (1 - p) is rounded once, not a difference of
    two rounded numbers (which would be off by many times its size).  The other 776 logits
    are about N(0, 4), their exponentials sum to about 776 e^2 = 5700: the given token's
    ln p is about -ln(1 + 5700 / e^size), -0.53 at 9 and -6e-4 at 16."""
    torch = torch_cuda
    N, d, V = 40, 64, 777
    h, W, tokens = make(torch, N, d, V, "bf16", 13)
    tokens = torch.arange(N, device="cuda") * 19
    W = W.clone()
    W[tokens] = (h.float() * (size / h.float().norm(dim=1, keepdim=True) ** 2)).to(W.dtype)
    hx = h.detach().requires_grad_()
    logp, _, _ = kd.head_logprobs(hx, W, tokens)
    assert logp.median().item() > -2 * np.log(1 + 5700 / np.exp(size))
    logp.sum().backward()
    dh, _ = ref.head_gradient(np64(h), np64(W), tokens.cpu().numpy(), np.ones(N))
    check_grad("dh", hx.grad, dh, "bf16")


def test_against_differences(torch_cuda):
    """Central differences of the GPU's forward along random directions, float32: the step
    leaves h^2 / 6 of a third derivative of order one, rounding 2e-6 N / h."""
    torch = torch_cuda
    h, W, tokens = make(torch, 6, 32, 50, "f32", 17)
    g = torch.randn(6, device="cuda").double()

    def value(a, b):
        o = kd.head_logprobs(a, b, tokens)
        return g @ (o[0].double() + 0.5 * o[1].double() - 0.25 * o[2].double())

    hx, wx = h.clone().requires_grad_(), W.clone().requires_grad_()
    value(hx, wx).backward()
    for i in range(4):
        a, b = torch.randn_like(h), torch.randn_like(W)
        a, b = a / a.norm(), b / b.norm()
        with torch.no_grad():
            num = (value(h + 0.02 * a, W + 0.02 * b) - value(h - 0.02 * a, W - 0.02 * b)) / 0.04
        want = (hx.grad.double() * a).sum() + (wx.grad.double() * b).sum()
        assert abs(num.item() - want.item()) < 4e-3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_chunks_groups_and_repeats(torch_cuda, dtype):
    """The forward does not depend on the chunk at all; dh and dW only in the order of float32
    sums; smaller dW groups and a repeat give the same bits of dh."""
    torch = torch_cuda
    h, W, tokens = make(torch, 1000, 136, 1999, dtype, 23)
    up = torch.randn(1000, device="cuda")
    st = torch.empty((1000, 2), device="cuda")
    want = None
    for chunk in (1000, 300, 64, 1):
        if chunk == 1 and dtype == "f32":
            continue
        outs = kd.head_logprobs(h, W, tokens, chunk=chunk)
        if want is None:
            want = outs
            z = h.double() @ W.double().t()
            m = z.max(1).values
            st = torch.stack([m, (z - m[:, None]).exp().sum(1).log()], 1).float().contiguous()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
    base = kd.head_logprobs_bwd(h, W, tokens, st, want[1], up, up, up, chunk=300)
    for group in (16384, 600, 0):
        dh, dW = kd.head_logprobs_bwd(h, W, tokens, st, want[1], up, up, up, chunk=300,
                                      dw_group_tokens=group)
        assert torch.equal(dh, base[0])
        assert (dW - base[1]).norm() <= 1e-5 * base[1].norm()
    only, none = kd.head_logprobs_bwd(h, W, tokens, st, want[1], up, up, up, chunk=300, want_dW=False)
    assert none is None and torch.equal(only, base[0])
    none, only = kd.head_logprobs_bwd(h, W, tokens, st, want[1], up, up, up, chunk=300, want_dh=False)
    assert none is None and torch.equal(only, base[1])


def test_frozen_head(torch_cuda):
    torch = torch_cuda
    h, W, tokens = make(torch, 20, 64, 500, "bf16", 29)
    hx, wx = h.detach().requires_grad_(), W.detach().requires_grad_()
    a, = torch.autograd.grad(kd.head_logprobs(hx, W, tokens)[0].sum(), hx)
    b, = torch.autograd.grad(kd.head_logprobs(h, wx, tokens)[0].sum(), wx)
    c = torch.autograd.grad(kd.head_logprobs(hx, wx, tokens)[0].sum(), (hx, wx))
    assert torch.equal(a, c[0]) and torch.equal(b, c[1])


@pytest.mark.parametrize("N", [3, 400])
def test_invalid_tokens_and_states(torch_cuda, N):
    torch = torch_cuda
    h, W, tokens = make(torch, N, 64, 700, "bf16", 31)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    clean = kd.head_logprobs(h, W, tokens, status=status)
    assert status.item() == 0
    tokens[0] = 700
    outs = kd.head_logprobs(h, W, tokens, status=status)
    assert status.item() == 2 and torch.isnan(outs[0]).nonzero().tolist() == [[0]]
    assert torch.equal(outs[1], clean[1]) and torch.equal(outs[2], clean[2])
    tokens[0] = 1
    h = h.clone()
    h[2, 5] = float("nan")
    status.zero_()
    outs = kd.head_logprobs(h, W, tokens, status=status)
    assert status.item() == 2
    for o in outs:
        assert torch.isnan(o).nonzero().tolist() == [[2]]


def test_no_rows(torch_cuda):
    torch = torch_cuda
    h = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    W = torch.ones((30, 64), device="cuda", dtype=torch.bfloat16, requires_grad=True)
    outs = kd.head_logprobs(h, W, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert all(o.shape == (0,) for o in outs)
    outs[0].sum().backward()
    assert h.grad.shape == (0, 64) and (W.grad == 0).all()


@pytest.mark.parametrize("N", [2, 300])
def test_recorded_and_replayed_and_other_streams(torch_cuda, N):
    torch = torch_cuda
    h, W, tokens = make(torch, N, 136, 3001, "bf16", 37)
    hx, wx = h.detach().requires_grad_(), W.detach().requires_grad_()
    up = torch.randn(N, device="cuda")

    def step():
        o = kd.head_logprobs(hx, wx, tokens, chunk=128)
        return (*o, *torch.autograd.grad((o[0], o[1]), (hx, wx), (up, up)))

    want = [t.detach().clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kd.head_logprobs(h, W, tokens, chunk=128, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs))
    for seed in (0, 1, 2):
        a, b, t = make(torch, N, 136, 3001, "bf16", 100 + seed)
        with torch.no_grad():
            hx.copy_(a)
            wx.copy_(b)
        tokens.copy_(t)
        want = [t.detach().clone() for t in step()]
        for graph, outs in graphs:
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(outs, want):
                assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_agrees_with_the_logits_form_and_the_loss(torch_cuda, dtype):
    """The same numbers from logits; and the KL loss with one teacher entry of probability one
    per row is the mean of -logp, its dh and dW those of this operator."""
    torch = torch_cuda
    N, d, V = 200, 264, 3001
    h, W, tokens = make(torch, N, d, V, dtype, 41)
    tokens = tokens.clamp(min=0)
    hx, wx = h.detach().requires_grad_(), W.detach().requires_grad_()
    logp, H, lse = kd.head_logprobs(hx, wx, tokens)
    (-logp.mean()).backward()
    a = kd.token_logprobs(h.float() @ W.float().t(), tokens)
    for x, y in zip((logp, H, lse), a):
        assert (x - y).abs().max().item() < 5e-5
    loss, dh, dW = kd.fwd_bwd(h, W, tokens.int()[:, None].contiguous(), torch.ones((N, 1), device="cuda"))
    assert abs(loss.item() + logp.mean().item()) < 1e-5
    tol = 1e-2 if dtype == "bf16" else 1e-5
    for x, y in ((hx.grad, dh), (wx.grad, dW)):
        assert (x.double() - y.double()).norm() <= tol * y.double().norm()


def test_a_training_step_of_all_operators(torch_cuda):
    """KL to the teacher's cached top K plus hard-label and entropy terms on the same head,
    gradients added up and clipped, against float64; then scored through the logits."""
    import oracle
    torch = torch_cuda
    N, d, V, K = 300, 136, 2001, 8
    h, W, tokens = make(torch, N, d, V, "f32", 43)
    teacher = torch.randn((N, V), device="cuda") * 3
    idx, p, _ = kd.teacher_topk(teacher, K=K)
    hx, wx = h.clone().requires_grad_(), W.clone().requires_grad_()
    logp, H, _ = kd.head_logprobs(hx, wx, tokens)
    loss = kd.chunked_kl_loss(hx, wx, idx, p) - 0.5 * logp.mean() - 0.1 * H.mean()
    loss.backward()
    r = oracle.forward_backward(np64(h), np64(W), idx.cpu().numpy(), np64(p), np.ones(N, np.uint8))
    f = ref.head_forward(np64(h), np64(W), tokens.cpu().numpy())
    dh, dW = ref.head_gradient(np64(h), np64(W), tokens.cpu().numpy(), np.full(N, -0.5 / N),
                               np.full(N, -0.1 / N))
    want = r["loss"] - 0.5 * f["logp"].mean() - 0.1 * f["entropy"].mean()
    assert abs(loss.item() - want) < 1e-5 * abs(want)
    norm, clipped = ref.clip([r["dh"] + dh, r["dW"] + dW], 0.01)
    got = kd.clip_grads([hx.grad, wx.grad], 0.01)
    assert abs(got.item() - norm) < 1e-5 * norm
    for x, y in zip((hx.grad, wx.grad), clipped):
        check_grad("clipped", x, y, "f32")
    with torch.no_grad():
        wx -= wx.grad
        scored = kd.token_logprobs(hx @ wx.t(), tokens, top=5)
        assert (scored[0] - kd.head_logprobs(hx, wx, tokens)[0]).abs().max() < 5e-5
