"""The global gradient norm and clipping on the GPU against float64: many sizes, types and
alignments, no clipping, nothing finite, streams, graphs."""
import numpy as np
import pytest

import output_head_kl_amd as kd
from oracle import logprobs as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def make(torch, sizes, kinds, seed=0, scale=0.01):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=g, device="cuda") * scale).to(
        torch.bfloat16 if k == "b" else torch.float32) for n, k in zip(sizes, kinds)]


def check(torch, grads, max_norm, out):
    """Squares are float64 products of float32 values: the norm is right to its rounding, the
    scale to one more, an output to its own rounding (bf16 2^-8, fp32 2^-24) on top."""
    before = [g.double().cpu().numpy() for g in grads]
    norm, want = ref.clip(before, max_norm)
    got = kd.clip_grads(grads, max_norm, out=out)
    assert abs(got.item() - norm) <= 2 * U * norm
    for w, b, t in zip(want, before, grads if out is None else out):
        half = 2.0 ** -8 if t.dtype == torch.bfloat16 else U
        x = t.double().cpu().numpy()
        if norm <= max_norm:
            assert np.array_equal(x, b)
        else:
            assert (np.abs(x - w) <= (half + 3 * U) * np.abs(w) + 1e-44).all()
    return got


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("factor", [0.0, 0.3, 3.0])
@pytest.mark.parametrize("sizes,kinds", [
    ([1], "f"), ([1], "b"), ([3, 1, 7], "bfb"), ([8191, 8192, 8193], "fbf"),
    ([100003, 5, 0, 64 * 1024], "bffb"), ([4097] * 200, "fb" * 100), ([30000001], "b"),
    ([20000003, 77], "fb"), ([77, 70000003], "ff")])
def test_values(torch_cuda, sizes, kinds, factor, inplace):
    torch = torch_cuda
    grads = make(torch, sizes, kinds, sum(sizes))
    norm = 0.01 * sum(sizes) ** 0.5
    if sizes == [1]:
        norm = abs(grads[0].float().item())
    check(torch, grads, factor * norm, None if inplace else [torch.full_like(g, 9) for g in grads])


def test_every_alignment(torch_cuda):
    torch = torch_cuda
    for dt in (torch.bfloat16, torch.float32):
        a, b = torch.randn(9000, device="cuda").to(dt), torch.zeros(9100, device="cuda", dtype=dt)
        for i in range(9):
            b.fill_(5)
            grads, out = [a[i:i + 8500 + i]], [b[3 * i % 9:][:8500 + i]]
            check(torch, grads, 1.0, out)
            rest = b.clone()
            rest[3 * i % 9:][:8500 + i] = 5
            assert (rest == 5).all()


def test_huge_tiny_and_not_finite(torch_cuda):
    """Squares beyond float32's range; a norm that is not finite leaves everything as it was."""
    torch = torch_cuda
    check(torch, [torch.full((1000,), 1e30, device="cuda")], 1.0, None)
    check(torch, [torch.full((1000,), 1e-30, device="cuda")], 1e-32, None)
    for bad in (float("inf"), float("nan")):
        g = make(torch, [5000, 300], "fb", 3)
        g[1][7] = bad
        keep = [t.clone() for t in g]
        out = [torch.zeros_like(t) for t in g]
        n = kd.clip_grads(g, 0.1, out=out)
        assert not torch.isfinite(n).item()
        kd.clip_grads(g, 0.1)
        for a, b, c in zip(g, keep, out):
            assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
            assert torch.equal(c.nan_to_num(7.0), b.nan_to_num(7.0))
    g = [torch.full((100,), 3e38, device="cuda")]  # the norm passes float32's range
    assert kd.clip_grads(g, 1.0).item() == float("inf") and (g[0] == 3e38).all()


def test_norm_alone_and_empty(torch_cuda):
    torch = torch_cuda
    g = make(torch, [1000, 0, 77], "fbb", 5)
    want = ref.clip([t.double().cpu().numpy() for t in g], 1.0)[0]
    assert abs(kd.grad_norm(g).item() - want) <= 2 * U * want
    assert abs(kd.grad_norm([g[0], g[0]]).item() - kd.grad_norm(g[0]).item() * 2 ** 0.5) < 1e-6
    e = torch.empty(0, device="cuda")
    assert kd.grad_norm(e).item() == 0 and kd.clip_grads([e], 0.0, out=[e]).item() == 0


def test_refused(torch_cuda):
    torch = torch_cuda
    g = torch.ones(64, 64, device="cuda")
    for bad in ([g, g], [g, g[3]], [g.view(-1)[:100], g.view(-1)[99:]]):
        with pytest.raises(kd.KDError, match="share memory"):
            kd.clip_grads(bad, 1.0)
    with pytest.raises(kd.KDError, match="shares memory"):
        kd.clip_grads([g.view(-1)[:64]], 1.0, out=[g.view(-1)[1:65]])
    with pytest.raises(ValueError, match="contiguous"):
        kd.clip_grads([g.t()], 1.0)
    with pytest.raises(TypeError, match="float16"):
        kd.clip_grads([g.half()], 1.0)
    with pytest.raises(ValueError, match="shape"):
        kd.clip_grads([g], 1.0, out=[g[0].clone()])
    with pytest.raises(ValueError, match="is on cpu"):
        kd.clip_grads([g, torch.ones(3)], 1.0)
    with pytest.raises(kd.KDError, match="max_norm"):
        kd.clip_grads([g], -1.0)
    assert (g == 1).all()


def test_autograd_sees_the_write(torch_cuda):
    torch = torch_cuda
    a = torch.ones(10, device="cuda", requires_grad=True)
    b = a * 2
    c = b.exp()
    kd.clip_grads([c.detach()], 0.1)
    with pytest.raises(RuntimeError, match="modified"):
        c.sum().backward()


def test_same_bits_on_other_streams_and_in_graphs(torch_cuda):
    torch = torch_cuda
    g = make(torch, [700001, 33, 4096], "fbf", 9)
    keep = [t.clone() for t in g]
    out = [torch.empty_like(t) for t in g]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    n = kd.clip_grads(g, 0.5, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    n.record_stream(torch.cuda.current_stream())
    want = [t.clone() for t in (n, *out)]
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nn = kd.clip_grads(g, 0.5)
        graphs.append((graph, nn))
    for seed in (0, 1, 2):
        if seed:
            for t, k in zip(keep, make(torch, [700001, 33, 4096], "fbf", 20 + seed)):
                t.copy_(k)
            want = [kd.clip_grads(keep, 0.5, out=out), *out]
            want = [t.clone() for t in want]
        for graph, nn in graphs:
            for t, k in zip(g, keep):
                t.copy_(k)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip((nn, *g), want):
                assert torch.equal(a, b)
