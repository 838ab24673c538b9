"""Refusals of the log-probability calls, without a GPU: the binding's checks before the
library is used, and the library's host-side checks before any device work."""
import ctypes

import pytest
import torch

import output_head_kl_amd as kd

OK, E_ARG, E_INDEX, E_WORKSPACE, E_UNSUPPORTED, E_HIP = range(6)
A = 4096  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    return kd._lib()


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_tensors_off_the_gpu_are_refused(monkeypatch, device):
    class NoLibrary:
        def __getattr__(self, name):
            raise AssertionError(f"the library was used ({name})")

    monkeypatch.setattr(kd, "_LIB", NoLibrary())
    z = torch.zeros((3, 8), device=device)
    t = torch.zeros(3, dtype=torch.int64, device=device)
    s = torch.zeros((3, 2), device=device)
    for call in (lambda: kd.token_logprobs(z, t), lambda: kd.token_logprobs(z.requires_grad_(), t),
                 lambda: kd.token_logprobs_bwd(z, t, s, s[:, 0])):
        with pytest.raises(ValueError, match="CUDA|on "):
            call()


def _fwd(lib, logits=A, dtype=1, ld=64, tokens=A, bits=64, N=4, V=64, top=3, logp=A, entropy=A,
         lse=A, stats=A, idx=A, tlp=A, status=A, ws=A, ws_bytes=1 << 20):
    return lib.kd_token_logprobs(logits, dtype, ld, tokens, bits, N, V, top, logp, entropy, lse,
                                 stats, idx, tlp, status, ws, ws_bytes, None)


def _bwd(lib, logits=A, dtype=1, ld=64, tokens=A, bits=64, N=4, V=64, stats=A, entropy=A, gl=A,
         ge=A, gz=A, out=1 << 20, ld_d=64):
    return lib.kd_token_logprobs_bwd(logits, dtype, ld, tokens, bits, N, V, stats, entropy, gl, ge,
                                     gz, out, ld_d, None)


COMMON = [
    (dict(dtype=2), E_ARG), (dict(dtype=-1), E_ARG), (dict(bits=16), E_ARG), (dict(N=-1), E_ARG),
    (dict(V=0), E_ARG), (dict(ld=63), E_ARG), (dict(ld=-64), E_ARG), (dict(logits=None), E_ARG),
    (dict(tokens=None), E_ARG), (dict(logits=A + 1), E_ARG), (dict(dtype=0, logits=A + 2), E_ARG),
    (dict(tokens=A + 4), E_ARG), (dict(bits=32, tokens=A + 2), E_ARG),
    (dict(V=1 << 29, ld=1 << 29), E_UNSUPPORTED), (dict(N=1 << 24), E_UNSUPPORTED),
    (dict(ld=(1 << 36) + 1), E_UNSUPPORTED)]


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(top=-1), E_ARG), (dict(top=65), E_ARG), (dict(top=65, V=100, ld=100), E_UNSUPPORTED),
    (dict(logp=None), E_ARG), (dict(entropy=None), E_ARG), (dict(lse=None), E_ARG),
    (dict(idx=None), E_ARG), (dict(tlp=None), E_ARG), (dict(logp=A + 2), E_ARG),
    (dict(stats=A + 4), E_ARG), (dict(status=A + 1), E_ARG), (dict(tlp=A + 2), E_ARG),
    (dict(V=100000, ld=100000, ws=None), E_WORKSPACE), (dict(V=100000, ld=100000, ws=A + 128), E_ARG),
    (dict(V=100000, ld=100000, ws_bytes=100), E_WORKSPACE)])
def test_forward_refusals(lib, change, code):
    assert _fwd(lib, **change) == code
    assert kd._lib().kd_last_error() != b""


@pytest.mark.parametrize("change,code", COMMON + [
    (dict(ld_d=63), E_ARG), (dict(ld_d=(1 << 36) + 1), E_ARG), (dict(stats=None), E_ARG),
    (dict(entropy=None), E_ARG), (dict(out=None), E_ARG), (dict(out=A + 1), E_ARG),
    (dict(stats=A + 4), E_ARG), (dict(gl=A + 2), E_ARG),
    (dict(out=A + 2), E_ARG), (dict(out=A - 128), E_ARG), (dict(out=A, ld_d=65), E_ARG),
    (dict(out=A + 2 * 64 * 4 - 2), E_ARG),
    (dict(N=(1 << 24) - 1, V=(1 << 29) - 1, ld=1 << 29, ld_d=1 << 29, out=1 << 62), E_UNSUPPORTED)])
def test_backward_refusals(lib, change, code):
    assert _bwd(lib, **change) == code


def test_more_threads_than_a_launch_has_are_refused(lib):
    """(2^24 - 1) rows of two pieces of 8192 elements, 256 threads each: over 2^32."""
    assert _bwd(lib, N=(1 << 24) - 1, V=8193, ld=8200, ld_d=8200, out=1 << 62) == E_UNSUPPORTED


def test_no_rows_need_nothing(lib):
    assert _fwd(lib, N=0, logits=None, tokens=None, logp=None, entropy=None, lse=None, idx=None,
                tlp=None, ws=None) == OK
    assert _bwd(lib, N=0, logits=None, tokens=None, stats=None, entropy=None, out=None) == OK


def test_workspace_sizes(lib):
    b = ctypes.c_size_t(0)
    f = lib.kd_token_logprobs_workspace_bytes
    assert f(4096, 128256, 8, 1, ctypes.byref(b)) == OK and b.value == 0
    assert f(1, 128256, 8, 1, ctypes.byref(b)) == OK and b.value > 0
    assert kd.token_logprobs_workspace_bytes(1, 128256, 64) > b.value
    for args in ((-1, 5, 1, 1), (1, 0, 1, 1), (1, 5, -1, 1), (1, 5, 1, 2)):
        assert f(*args, ctypes.byref(b)) == E_ARG
    assert f(1, 100, 65, 1, ctypes.byref(b)) == E_UNSUPPORTED
    assert f(1, 100, 1, 1, None) == E_ARG
