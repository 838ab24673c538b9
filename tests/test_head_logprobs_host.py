"""Refusals of the log probabilities from hidden states, without a GPU."""
import ctypes

import pytest
import torch

import output_head_kl_amd as kd

OK, E_ARG, E_INDEX, E_WORKSPACE, E_UNSUPPORTED, E_HIP = range(6)
A = 4096


def fwd(h=A, W=A, dtype=1, tokens=A, bits=64, N=4, d=64, V=64, chunk=2, logp=A, entropy=A, lse=A,
        stats=A, status=A, ws=A, ws_bytes=1 << 40):
    return kd._lib().kd_head_logprobs(h, W, dtype, tokens, bits, N, d, V, chunk, logp, entropy,
                                      lse, stats, status, ws, ws_bytes, None)


def bwd(h=A, W=A, dtype=1, tokens=A, bits=64, N=4, d=64, V=64, chunk=2, stats=A, entropy=A, gl=A,
        ge=A, gz=A, dh=A, dW=A, wt=0, ws=A, ws_bytes=1 << 40):
    return kd._lib().kd_head_logprobs_bwd(h, W, dtype, tokens, bits, N, d, V, chunk, stats,
                                          entropy, gl, ge, gz, dh, dW, wt, ws, ws_bytes, None)


COMMON = [
    (dict(dtype=2), E_ARG), (dict(bits=8), E_ARG), (dict(N=-1), E_ARG), (dict(d=0), E_ARG),
    (dict(V=0), E_ARG), (dict(chunk=0), E_ARG), (dict(d=60), E_UNSUPPORTED),
    (dict(d=(1 << 20) + 8), E_UNSUPPORTED), (dict(V=(1 << 24) + 1), E_UNSUPPORTED),
    (dict(N=1 << 23, chunk=1 << 23), E_UNSUPPORTED), (dict(N=(1 << 40) + 1), E_UNSUPPORTED),
    (dict(h=None), E_ARG), (dict(W=None), E_ARG), (dict(tokens=None), E_ARG),
    (dict(h=A + 8), E_ARG), (dict(W=A + 8), E_ARG), (dict(tokens=A + 4), E_ARG),
    (dict(ws=None), E_WORKSPACE), (dict(ws=A + 64), E_ARG), (dict(ws_bytes=64), E_WORKSPACE)]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(logp=None), E_ARG), (dict(entropy=None), E_ARG), (dict(lse=None), E_ARG),
    (dict(lse=A + 2), E_ARG), (dict(stats=A + 4), E_ARG), (dict(status=A + 1), E_ARG)])
def test_forward_refusals(change, code):
    assert fwd(**change) == code and kd._lib().kd_last_error() != b""


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(dh=None, dW=None), E_ARG), (dict(stats=None), E_ARG), (dict(entropy=None), E_ARG),
    (dict(dh=A + 8), E_ARG), (dict(dW=A + 8), E_ARG), (dict(gl=A + 2), E_ARG),
    (dict(stats=A + 4), E_ARG), (dict(wt=2), E_ARG), (dict(dtype=0, wt=1), E_ARG)])
def test_backward_refusals(change, code):
    assert bwd(**change) == code and kd._lib().kd_last_error() != b""


@pytest.mark.parametrize("place", ["h in dh", "W in dh", "h in dW", "W in dW", "dh in dW"])
def test_results_in_the_operands_are_refused(place):
    far = {name: 1 << (30 + 2 * i) for i, name in enumerate(("h", "W", "dh", "dW"))}
    inner, outer = place.split(" in ")
    at = dict(far, **{inner: far[outer] + 128})  # inside the other's 4 x 64 or 64 x 64 elements
    assert bwd(**at) == E_ARG and b"share memory" in kd._lib().kd_last_error()


def test_more_threads_than_a_launch_has_are_refused():
    for f in (fwd, bwd):
        assert f(N=1 << 22, chunk=1 << 22, V=(1 << 16) + 1) == E_UNSUPPORTED


def test_no_rows_need_nothing():
    assert fwd(N=0, h=None, tokens=None, logp=None, entropy=None, lse=None) == OK
    assert bwd(N=0, h=None, tokens=None, stats=None, entropy=None, dW=None) == OK


def test_workspace_bytes():
    f = kd.head_logprobs_workspace_bytes
    assert f(32768, 2048, 128256) == f(262144, 2048, 128256) < 32 << 20  # one chunk's partials
    b = kd.head_logprobs_bwd_workspace_bytes
    assert b(32768, 2048, 128256, dw_group_tokens=0) < b(32768, 2048, 128256)
    out = ctypes.c_size_t(0)
    lib = kd._lib()
    assert lib.kd_head_logprobs_workspace_bytes(1, 12, 5, 1, 1, ctypes.byref(out)) == E_UNSUPPORTED
    assert lib.kd_head_logprobs_workspace_bytes(1, 16, 5, 1, 1, None) == E_ARG
    assert lib.kd_head_logprobs_bwd_workspace_bytes(1, 16, 5, 1, 1, 0, -1, ctypes.byref(out)) == E_ARG


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_tensors_off_the_gpu_are_refused(device):
    h, W = torch.zeros((3, 8), device=device), torch.zeros((5, 8), device=device)
    t = torch.zeros(3, dtype=torch.int64, device=device)
    s = torch.zeros((3, 2), device=device)
    for f in (lambda: kd.head_logprobs(h, W, t), lambda: kd.head_logprobs_bwd(h, W, t, s, s[:, 0])):
        with pytest.raises(ValueError, match="CUDA"):
            f()
