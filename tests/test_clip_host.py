"""Refusals of gradient clipping, without a GPU."""
import ctypes

import pytest
import torch

import output_head_kl_amd as kd

OK, E_ARG, E_INDEX, E_WORKSPACE, E_UNSUPPORTED, E_HIP = range(6)
A = 1 << 20


def call(grads, outs, numel, types, max_norm=1.0, norm=A, ws=A, ws_bytes=1 << 20, n=None):
    n = len(grads) if n is None else n
    arr = lambda t, v: None if v is None else (t * len(v))(*v)  # noqa: E731
    return kd._lib().kd_clip_grads(arr(ctypes.c_void_p, grads), arr(ctypes.c_void_p, outs),
                                   arr(ctypes.c_int64, numel), arr(ctypes.c_int32, types), n,
                                   max_norm, norm, ws, ws_bytes, None)


@pytest.mark.parametrize("args,kw,code", [
    (([A], None, [8], [1]), dict(max_norm=-1.0), E_ARG),
    (([A], None, [8], [1]), dict(max_norm=float("nan")), E_ARG),
    (([A], None, [8], [1]), dict(norm=None), E_ARG),
    (([A], None, [8], [1]), dict(norm=A + 2), E_ARG),
    (([A], None, [8], [1]), dict(ws=None), E_WORKSPACE),
    (([A], None, [8], [1]), dict(ws=A + 64), E_ARG),
    (([A], None, [8], [1]), dict(ws_bytes=8), E_WORKSPACE),
    (([A], None, [8], [2]), {}, E_ARG),
    (([A], None, [-8], [1]), {}, E_ARG),
    (([A], None, [1 << 45], [1]), {}, E_UNSUPPORTED),
    (([A, A], None, [1 << 44, 1], [1, 1]), {}, E_UNSUPPORTED),
    (([A], None, [8], [1]), dict(n=-1), E_ARG),
    (([None], None, [8], [1]), {}, E_ARG),
    (([A], [None], [8], [1]), {}, E_ARG),
    (([A + 1], None, [8], [1]), {}, E_ARG),
    (([A + 2], None, [8], [0]), {}, E_ARG),
    (([A], [A + 1026], [8], [0]), {}, E_ARG),
    # the same tensor twice, and tensors that touch
    (([A, A], None, [8, 8], [1, 1]), {}, E_ARG),
    (([A, A + 1024, A + 30], None, [16, 8, 8], [1, 1, 1]), {}, E_ARG),
    (([A, A + 4096], [A + 8192, A + 8200], [16, 8], [1, 1]), {}, E_ARG),
    (([A, A + 4096], [A + 8192, A], [16, 8], [1, 1]), {}, E_ARG),     # another's gradient
    (([A], [A + 2], [16], [1]), {}, E_ARG),                            # shifted by one
    (([A, A + 4096], [A, A + 4090], [16, 8], [1, 1]), {}, E_ARG),
])
def test_refusals(args, kw, code):
    assert call(*args, **kw) == code
    assert kd._lib().kd_last_error() != b""


def test_workspace_bytes():
    b = ctypes.c_size_t(0)
    f = kd._lib().kd_clip_grads_workspace_bytes
    sizes = (ctypes.c_int64 * 3)(0, 1, 10 ** 9)
    assert f(sizes, 3, ctypes.byref(b)) == OK and 0 < b.value < 1 << 20
    assert f(None, 0, ctypes.byref(b)) == OK and b.value == 256
    assert f(None, 1, ctypes.byref(b)) == E_ARG and f(sizes, 3, None) == E_ARG


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_tensors_off_the_gpu_are_refused(device):
    g = torch.zeros(4, device=device)
    for f in (lambda: kd.grad_norm([g]), lambda: kd.clip_grads(g, 1.0),
              lambda: kd.clip_grads([g], 1.0, out=[g])):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(ValueError, match="no tensors"):
        kd.clip_grads([], 1.0)
