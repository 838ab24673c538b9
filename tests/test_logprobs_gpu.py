"""Log probabilities of given tokens from logits, on the GPU, against the float64 definitions
in oracle/logprobs.py: sizes from one to a full vocabulary, both types, row strides and
alignments, masks, equal logits, invalid rows and tokens, streams, graphs, offsets past 2^32
bytes; the gradient against the formula and against differences."""
import threading

import numpy as np
import pytest

import output_head_kl_amd as kd
from logprobs_util import check_forward, close, grad_tolerance, make_rows, np64
from oracle import logprobs as ref

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _dt(torch, name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _check(torch, logits, tokens, top):
    outs = kd.token_logprobs(logits, tokens, top=top)
    z = np64(logits)
    f = ref.forward(z, tokens.cpu().numpy(), top)
    check_forward(outs, z, f, top)
    return outs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,top,pad", [
    (1, 1, 1, 0), (1, 2, 2, 0), (5, 7, 7, 0), (3, 8, 1, 0), (4, 9, 5, 3), (2, 63, 63, 1),
    (3, 64, 64, 0), (2, 65, 64, 0), (1, 1000, 20, 0), (7, 4097, 50, 1), (1, 8192, 64, 0),
    (2, 8193, 3, 2), (37, 32003, 20, 61), (1, 128256, 20, 0), (3, 200001, 64, 0),
    (300, 5003, 8, 5), (600, 2050, 5, 0), (1100, 9001, 1, 0)])
def test_sizes(torch_cuda, dtype, N, V, top, pad):
    torch = torch_cuda
    logits, tokens = make_rows(torch, N, V, _dt(torch, dtype), 11 * N + V, pad=pad)
    outs = _check(torch, logits, tokens, top)
    plain = kd.token_logprobs(logits, tokens.int())  # without alternatives, int32 tokens
    for a, b in zip(plain, outs[:3]):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V", [(5, 3001), (700, 3001)])
def test_masked_rows(torch_cuda, dtype, N, V):
    torch = torch_cuda
    logits, tokens = make_rows(torch, N, V, _dt(torch, dtype), 5, masked=True)
    low = torch.finfo(logits.dtype).min
    logits[0] = float("-inf")                 # nothing left
    logits[1] = low                           # the lowest value everywhere: uniform
    logits[2, 1:] = float("-inf")             # one token left
    logits[2, 0] = -3.0
    logits[3].masked_fill_(torch.isinf(logits[3]), low)
    tokens[2], tokens[4] = 0, -1
    outs = _check(torch, logits, tokens, 20)
    assert outs[2][0].item() == float("-inf") and outs[0][2].item() == 0.0
    assert outs[3][2].tolist() == list(range(20))
    assert abs(outs[1][1].item() - np.log(V)) < 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,levels", [(2, 100000, 1), (900, 3000, 2), (1, 3000, 4)])
def test_equal_logits_go_to_the_lowest_index(torch_cuda, dtype, N, V, levels):
    torch = torch_cuda
    logits, tokens = make_rows(torch, N, V, _dt(torch, dtype), 17, levels=levels)
    logits[0] = 0.0
    logits[0, 1::2] = -0.0                    # equal to +0
    _check(torch, logits, tokens, 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,V,pad", [(8, 150001, 1), (24, 100003, 0), (9, 262144, 3), (120, 130008, 0)])
@pytest.mark.parametrize("top", [1, 20, 64])
def test_long_rows_in_pieces(torch_cuda, dtype, N, V, pad, top):
    """Rows long enough to be split over workgroups: pieces without a finite logit, candidates
    in one piece only, equal ones in all, NaN in one piece, the given token anywhere."""
    torch = torch_cuda
    logits, tokens = make_rows(torch, N, V, _dt(torch, dtype), N + V, masked=True, pad=pad)
    logits[0] = float("-inf")
    logits[1, : V - 70] = float("-inf")       # all of it in the last piece
    logits[2, 70:] = float("-inf")            # in the first
    logits[3] = 1.5                           # equal everywhere
    logits[4] = torch.finfo(logits.dtype).min
    logits[5, V // 2] = float("nan")
    logits[6, V - 1] = float("inf")
    logits[7, : V // 2] = float("-inf")
    tokens[1], tokens[2], tokens[3], tokens[4] = V - 1, 0, V // 3, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = kd.token_logprobs(logits, tokens, top=top, status=status)
    z = np64(logits)
    check_forward(outs, z, ref.forward(z, tokens.cpu().numpy(), top), top)
    assert status.item() == 2


def test_rows_that_rise_and_fall(torch_cuda):
    """Every step raises the running maximum, or none does after the first."""
    torch = torch_cuda
    up = torch.linspace(-40, 40, 40000, device="cuda").repeat(520, 1)
    for z in (up, up.flip(1).contiguous()):
        for n in (520, 2):
            _check(torch, z[:n].bfloat16(), torch.arange(n, device="cuda") * 7, 20)


def test_wide_range_and_large_offsets(torch_cuda):
    """Values to 1e38, and rows far from zero: the results follow the differences only."""
    torch = torch_cuda
    z, tokens = make_rows(torch, 6, 4001, torch.float32, 23)
    z = z.contiguous()
    z[0] *= 1e36
    z[1, 5] = -3.4e38
    z[2] += 1000.0
    _check(torch, z, tokens, 9)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [4, 800])
def test_invalid_rows_and_tokens_stay_in_their_rows(torch_cuda, dtype, N):
    torch = torch_cuda
    V = 2500
    logits, tokens = make_rows(torch, N, V, _dt(torch, dtype), 31)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kd.token_logprobs(logits, tokens, top=5, status=status)
    assert status.item() == 0
    for place, value in ((0, float("nan")), (V - 1, float("nan")), (1234, float("inf"))):
        bad = logits.clone()
        bad[1, place] = value
        bad[3, ::3] = float("nan")
        status.zero_()
        outs = kd.token_logprobs(bad, tokens, top=5, status=status)
        assert status.item() == 2
        z = np64(bad)
        check_forward(outs, z, ref.forward(z, tokens.cpu().numpy(), 5), 5)
    for t in (V, V + 70000, 2 ** 40):
        off = tokens.clone()
        off[2] = t
        status.zero_()
        outs = kd.token_logprobs(logits, off, top=5, status=status)
        assert status.item() == 2 and torch.isnan(outs[0]).nonzero().tolist() == [[2]]
        assert torch.isfinite(outs[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_every_alignment(torch_cuda, dtype):
    """Views that begin at any element of an allocation, rows of odd strides."""
    torch = torch_cuda
    flat = torch.randn(3 * 4111 + 64, device="cuda").to(_dt(torch, dtype))
    for first in range(9):
        z = flat[first:].as_strided((3, 4100 - first), (4111, 1))
        tokens = torch.tensor([0, 4000, 77], device="cuda")
        _check(torch, z, tokens, 6)
        g = torch.tensor([1.0, -2.0, 0.5], device="cuda")
        x = z.detach().requires_grad_()
        logp, H, _ = kd.token_logprobs(x, tokens)
        (logp @ g + H @ g).backward()
        zz, gg = np64(z), np64(g)
        dz = ref.gradient(zz, tokens.cpu().numpy(), gg, gg)
        tol = grad_tolerance(zz, dz, (gg, gg, None), tokens.cpu().numpy(), np64(H), HALF[dtype])
        assert (np.abs(np64(x.grad) - dz) <= tol).all()


def test_rows_past_32_bit_offsets(torch_cuda):
    torch = torch_cuda
    ld = 2 ** 31 + 40
    flat = torch.empty(2 * ld + 5000, dtype=torch.bfloat16, device="cuda")
    z = flat.as_strided((3, 5000), (ld, 1))
    rows, tokens = make_rows(torch, 3, 5000, torch.bfloat16, 41)
    z.copy_(rows)
    a, b = kd.token_logprobs(z, tokens, top=4), kd.token_logprobs(rows, tokens, top=4)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    x, y = z.detach().requires_grad_(), rows.detach().requires_grad_()
    for t in (x, y):
        kd.token_logprobs(t, tokens)[0].sum().backward()
    assert torch.equal(x.grad, y.grad)


def test_no_rows(torch_cuda):
    torch = torch_cuda
    x = torch.empty((0, 50), device="cuda", requires_grad=True)
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    outs = kd.token_logprobs(x, t, top=3)
    assert [tuple(o.shape) for o in outs] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    outs[0].sum().backward()
    assert x.grad.shape == (0, 50)


# ---- the gradient -----------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["logp", "entropy", "lse", "all"])
@pytest.mark.parametrize("N,V,pad", [(1, 1, 0), (1, 5, 0), (3, 8, 8), (5, 8191, 1), (2, 70001, 0),
                                     (530, 1999, 3)])
def test_gradient(torch_cuda, dtype, which, N, V, pad):
    torch = torch_cuda
    logits, tokens = make_rows(torch, N, V, _dt(torch, dtype), 7 * N + V, pad=pad, masked=V > 8)
    if N > 2:
        logits[1] = float("-inf")
        tokens[2] = -1
    gen = torch.Generator(device="cuda").manual_seed(3)
    g = [torch.randn(N, generator=gen, device="cuda") if which in (n, "all") else None
         for n in ("logp", "entropy", "lse")]
    x = logits.detach().requires_grad_()
    outs = kd.token_logprobs(x, tokens, top=min(V, 2))
    used = [(o, k) for o, k in zip(outs[:3], g) if k is not None]
    torch.autograd.backward([o for o, _ in used], [k for _, k in used])
    z, tk = np64(logits), tokens.cpu().numpy()
    gn = [None if k is None else np64(k) for k in g]
    dz = ref.gradient(z, tk, *gn)
    tol = grad_tolerance(z, dz, gn, tk, np64(outs[1]), HALF[dtype])
    off = np.abs(np64(x.grad) - dz) - tol
    assert off.max() <= 0, f"{off.max():.3g} past the tolerance"
    if N > 2:
        assert (x.grad[1] == 0).all()


def test_gradient_against_differences(torch_cuda):
    """Central differences of the GPU's own forward in float32: the step h = 0.05 leaves
    h^2 / 6 |f'''| <= 4.2e-4 * 6 (three derivatives of p are at most 6 p in size, weights of
    one), rounding 1e-6 / h = 2e-5."""
    torch = torch_cuda
    z, tokens = make_rows(torch, 3, 17, torch.float32, 51)
    z = z.contiguous()
    g = torch.tensor([0.7, -0.4, 1.0], device="cuda")
    x = z.detach().requires_grad_()

    def value(t):
        logp, H, lse = kd.token_logprobs(t, tokens)
        return (logp.double() @ g.double() + 0.3 * (H.double() @ g.double())
                + 0.2 * (lse.double() @ g.double()))

    value(x).backward()
    for n in range(3):
        for v in range(17):
            e = torch.zeros_like(z)
            e[n, v] = 0.05
            with torch.no_grad():
                num = (value(z + e) - value(z - e)) / 0.1
            assert abs(num.item() - x.grad[n, v].item()) < 3e-3


def test_gradient_in_place_and_into_padded_rows(torch_cuda):
    torch = torch_cuda
    logits, tokens = make_rows(torch, 9, 777, torch.bfloat16, 61, pad=23)
    g = torch.randn(9, device="cuda")
    x = logits.detach().requires_grad_()
    logp, H, _ = kd.token_logprobs(x, tokens)
    logp.backward(g)
    z = logits.double()
    m = z.max(1).values
    stats = torch.stack([m, (z - m[:, None]).exp().sum(1).log()], 1).float()
    wide = torch.full((9, 900), 5.0, dtype=torch.bfloat16, device="cuda")
    kd.token_logprobs_bwd(logits, tokens, stats, H.detach(), g, out=wide[:, :777])
    assert torch.equal(wide[:, :777], x.grad) and (wide[:, 777:] == 5.0).all()
    whole = logits.as_strided((9, 800), (800, 1))
    kd.token_logprobs_bwd(logits, tokens, stats, H.detach(), g, out=logits)
    assert torch.equal(logits, x.grad) and (whole[:, 777:] == 7.0).all()


def test_gradients_too_large_for_the_cache(torch_cuda):
    """A gradient of more than 256 MB is stored past the cache: the same bits as in parts."""
    torch = torch_cuda
    for V in (128256, 128255):  # rows of an odd length are not aligned
        z, tokens = make_rows(torch, 1100, V, torch.bfloat16, 65)
        g = torch.randn(1100, device="cuda")

        def grad(a, b):
            x = z[a:b].detach().requires_grad_()
            logp, H, _ = kd.token_logprobs(x, tokens[a:b])
            return torch.autograd.grad((logp, H), x, (g[a:b], g[a:b]))[0]

        whole = grad(0, 1100)
        for a in range(0, 1100, 550):
            assert torch.equal(whole[a:a + 550], grad(a, a + 550))


def test_invalid_rows_have_nan_gradients(torch_cuda):
    torch = torch_cuda
    z, tokens = make_rows(torch, 4, 333, torch.float32, 71)
    z = z.contiguous()
    z[1, 3] = float("nan")
    tokens[2] = 333
    z.requires_grad_()
    kd.token_logprobs(z, tokens)[0].sum().backward()
    nan = torch.isnan(z.grad)
    assert nan[1].all() and nan[2].all() and not nan[0].any() and not nan[3].any()


def test_second_backward_and_changed_logits(torch_cuda):
    torch = torch_cuda
    z, tokens = make_rows(torch, 4, 333, torch.float32, 81)
    x = z.contiguous().requires_grad_()
    loss = kd.token_logprobs(x, tokens)[0].sum()
    loss.backward(retain_graph=True)
    once = x.grad.clone()
    loss.backward()
    assert torch.equal(x.grad, 2 * once)
    y = x.detach().clone().requires_grad_()
    yy = y * 1.0
    loss = kd.token_logprobs(yy, tokens)[0].sum()
    with torch.no_grad():
        yy.add_(1.0)
    with pytest.raises(RuntimeError, match="modified"):
        loss.backward()


# ---- streams, graphs, threads ----------------------------------------------------------------
def test_same_bits_every_time_and_on_other_streams(torch_cuda):
    torch = torch_cuda
    for N in (3, 900):
        logits, tokens = make_rows(torch, N, 30011, torch.bfloat16, 91, masked=True)
        want = kd.token_logprobs(logits, tokens, top=33)
        side = torch.cuda.Stream()
        for stream in (None, side, side.cuda_stream):
            side.wait_stream(torch.cuda.current_stream())
            got = kd.token_logprobs(logits, tokens, top=33, stream=stream)
            torch.cuda.current_stream().wait_stream(side)
            for a, b in zip(got, want):
                assert torch.equal(a, b)
            for t in got:
                t.record_stream(torch.cuda.current_stream())


@pytest.mark.parametrize("N", [2, 600])
def test_recorded_and_replayed(torch_cuda, N):
    torch = torch_cuda
    V = 20011
    logits, tokens = make_rows(torch, N, V, torch.bfloat16, 101)
    x = logits.contiguous().requires_grad_()
    g = torch.randn(N, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        outs = kd.token_logprobs(x, tokens, top=7, status=status)
        grad, = torch.autograd.grad((outs[0], outs[1]), x, (g, g))
        return (*outs, grad)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = step()
        graphs.append((graph, outs))
    for seed in (1, 2, 3):
        rows, t = make_rows(torch, N, V, torch.bfloat16, 200 + seed, masked=seed == 2)
        with torch.no_grad():
            x.copy_(rows)
        tokens.copy_(t)
        want = [o.detach().clone() for o in step()]
        for graph, outs in graphs:
            for o in outs:
                o.detach().fill_(3)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(outs, want):
                assert torch.equal(a, b)
    assert status.item() == 0


def test_two_threads_on_their_own_streams(torch_cuda):
    torch = torch_cuda
    cases = [make_rows(torch, n, 60001, torch.bfloat16, 300 + n) for n in (2, 40)]
    want = [kd.token_logprobs(z, t, top=20) for z, t in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = kd.token_logprobs(*cases[i], top=20)
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not wrong


def test_given_workspace_is_enough_and_not_exceeded(torch_cuda):
    torch = torch_cuda
    logits, tokens = make_rows(torch, 3, 50021, torch.bfloat16, 111)
    need = kd.token_logprobs_workspace_bytes(3, 50021, 9)
    assert need > 0
    buf = torch.full((need + 512,), 171, dtype=torch.uint8, device="cuda")
    a = kd.token_logprobs(logits, tokens, top=9, workspace=buf[:need])
    b = kd.token_logprobs(logits, tokens, top=9)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert (buf[need:] == 171).all()
    with pytest.raises(kd.KDError, match="KD_E_WORKSPACE"):
        kd.token_logprobs(logits, tokens, top=9, workspace=buf[:need - 1])


def test_agrees_with_the_teacher_producer(torch_cuda):
    """The alternatives are the teacher top-K producer's tokens with ln of its probabilities."""
    torch = torch_cuda
    z, tokens = make_rows(torch, 50, 9001, torch.bfloat16, 121)
    z = z.contiguous()
    idx, p, lse = kd.teacher_topk(z, K=20)
    outs = kd.token_logprobs(z, tokens, top=20)
    assert torch.equal(outs[3], idx)
    close("p", np64(outs[4].exp()), np64(p), 2e-5 * np64(p))
    close("lse", np64(outs[2]), np64(lse), 1e-5)
