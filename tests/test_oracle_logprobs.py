"""Pins of the float64 definitions in oracle/logprobs.py: torch's float64 log_softmax and
autograd, finite differences, hand-computed rows."""
import numpy as np
import pytest
import torch

from oracle import logprobs as ref


def _case(seed=0, N=6, V=11):
    rng = np.random.default_rng(seed)
    z = rng.normal(size=(N, V)) * 2.0
    tokens = rng.integers(0, V, N)
    tokens[1] = -1
    return z, tokens, rng


def test_hand_computed_rows():
    z = np.log(np.array([[1.0, 2.0, 1.0], [3.0, 1.0, 0.0]]) + 0.0, where=[[1, 1, 1], [1, 1, 0]],
               out=np.full((2, 3), -np.inf))
    f = ref.forward(z, [1, 2], top=2)
    assert np.allclose(f["lse"], np.log(4.0))
    assert np.isclose(f["logp"][0], np.log(0.5)) and f["logp"][1] == -np.inf
    assert np.allclose(f["entropy"], [1.5 * np.log(2.0), -(0.75 * np.log(0.75) + 0.25 * np.log(0.25))])
    assert f["top_idx"].tolist() == [[1, 0], [0, 1]]


def test_against_torch_log_softmax_and_autograd():
    z, tokens, rng = _case()
    x = torch.tensor(z, requires_grad=True)
    lp = torch.log_softmax(x, 1)
    t = torch.tensor(tokens)
    logp = torch.where(t < 0, torch.zeros(()).double(), lp[torch.arange(6), t.clamp(min=0)])
    H = -(lp.exp() * lp).sum(1)
    lse = torch.logsumexp(x, 1)
    f = ref.forward(z, tokens)
    for a, b in ((f["logp"], logp), (f["entropy"], H), (f["lse"], lse)):
        assert np.allclose(a, b.detach().numpy(), atol=1e-13)
    g = [rng.normal(size=6) for _ in range(3)]
    (torch.tensor(g[0]) @ logp + torch.tensor(g[1]) @ H + torch.tensor(g[2]) @ lse).backward()
    assert np.allclose(ref.gradient(z, tokens, *g), x.grad.numpy(), atol=1e-13)


def test_gradient_against_differences():
    z, tokens, rng = _case(3, 3, 5)
    g = [rng.normal(size=3) for _ in range(3)]

    def value(zz):
        f = ref.forward(zz, tokens)
        return g[0] @ f["logp"] + g[1] @ f["entropy"] + g[2] @ f["lse"]

    dz = ref.gradient(z, tokens, *g)
    for n in range(3):
        for v in range(5):
            e = np.zeros_like(z)
            e[n, v] = 1e-5
            assert abs((value(z + e) - value(z - e)) / 2e-5 - dz[n, v]) < 1e-9


def test_empty_masked_and_invalid_rows():
    z = np.array([[-np.inf] * 4, [0.0, -np.inf, 0.0, -np.inf], [0.0, np.nan, 0.0, 0.0],
                  [0.0, np.inf, 0.0, 0.0], [0.0] * 4])
    tokens = np.array([2, 0, 0, 0, 4])
    f = ref.forward(z, tokens, top=3)
    assert f["lse"][0] == -np.inf and f["logp"][0] == -np.inf and f["entropy"][0] == 0
    assert f["top_idx"][0].tolist() == [0, 1, 2] and (f["top_logp"][0] == -np.inf).all()
    assert np.isclose(f["logp"][1], -np.log(2.0)) and f["top_idx"][1].tolist() == [0, 2, 1]
    for n in (2, 3):
        assert np.isnan([f["lse"][n], f["logp"][n], f["entropy"][n]]).all()
        assert (f["top_idx"][n] == -1).all() and np.isnan(f["top_logp"][n]).all()
    assert np.isnan(f["logp"][4]) and np.isclose(f["lse"][4], np.log(4.0))
    dz = ref.gradient(z, tokens, np.ones(5), np.ones(5))
    assert (dz[0] == 0).all() and np.isnan(dz[2:]).all()
    assert np.allclose(dz[1], [0.5, 0, -0.5, 0])


def test_head_is_the_logits_form_of_the_product():
    rng = np.random.default_rng(5)
    h, W = rng.normal(size=(4, 3)), rng.normal(size=(7, 3))
    tokens = np.array([0, 6, -1, 3])
    g = [rng.normal(size=4) for _ in range(3)]
    hx, wx = torch.tensor(h, requires_grad=True), torch.tensor(W, requires_grad=True)
    (hx @ wx.t()).backward(torch.tensor(ref.gradient(h @ W.T, tokens, *g)))
    dh, dW = ref.head_gradient(h, W, tokens, *g)
    assert np.allclose(dh, hx.grad.numpy()) and np.allclose(dW, wx.grad.numpy())
    assert np.allclose(ref.head_forward(h, W, tokens)["lse"], torch.logsumexp(hx @ wx.t(), 1).detach())


@pytest.mark.parametrize("max_norm", [0.0, 2.5, 5.0, 9.0])
def test_clip(max_norm):
    grads = [np.array([3.0]), np.zeros((0, 2)), np.array([[0.0, 4.0]])]
    norm, out = ref.clip(grads, max_norm)
    assert norm == 5.0
    s = min(1.0, max_norm / 5.0)
    assert out[0][0] == 3.0 * s and out[2][0, 1] == 4.0 * s
