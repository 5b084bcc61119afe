"""The gradient norm's and the clipped step's host side: workspace and refusals.
No call here reaches a CUDA API."""
import ctypes

import pytest

import zero_sharded_mixed_bucket_gb300 as zg

A = 1 << 20            # an aligned address, never read


def _plan(*sizes, bits=32):
    return zg.zero_adamw_plan([zg.adamw_tensor(grad=A, master=A, m=A, v=A, m_scale=A, v_scale=A, numel=n) for n in sizes], zg.ZERO_FP16, bits)


def _refused(status, f, *args):
    with pytest.raises(zg.ZeroError) as e:
        f(*args)
    assert e.value.status == status and str(e.value)


def test_workspace():
    assert zg.zero_adamw_norm_workspace(_plan()) == zg.zero_adamw_norm_workspace(_plan(1)) > 0
    assert zg.zero_adamw_norm_workspace(_plan(1 << 33)) <= 1 << 20
    p = _plan(100)
    p.n_chunks += 1
    _refused(zg.ZERO_EINVAL, zg.zero_adamw_norm_workspace, p)
    assert zg.lib().zero_adamw_norm_workspace(None, ctypes.byref(ctypes.c_int64())) == zg.ZERO_EINVAL
    assert zg.lib().zero_adamw_norm_workspace(ctypes.byref(_plan(1)), None) == zg.ZERO_EINVAL


def test_norm_refusals():
    p, f = _plan(100), zg.zero_adamw_norm
    _refused(zg.ZERO_EINVAL, f, p, A, float("inf"), 1.0, A, A, A)
    _refused(zg.ZERO_EINVAL, f, p, A, float("nan"), 1.0, A, A, A)
    _refused(zg.ZERO_EINVAL, f, p, A, 1.0, float("nan"), A, A, A)
    _refused(zg.ZERO_ENOMEM, f, p, None, 1.0, 1.0, A, A, A)
    _refused(zg.ZERO_ENOMEM, f, p, A, 1.0, 1.0, None, A, A)
    _refused(zg.ZERO_ENOMEM, f, p, A, 1.0, 1.0, A, A, None)
    _refused(zg.ZERO_EALIGN, f, p, A + 4, 1.0, 1.0, A, A, A)
    _refused(zg.ZERO_EALIGN, f, p, A, 1.0, 1.0, A + 2, A, A)
    _refused(zg.ZERO_EALIGN, f, p, A, 1.0, 1.0, A, A + 2, A)
    _refused(zg.ZERO_EALIGN, f, p, A, 1.0, 1.0, A, A, A + 8)
    p.numel += 1
    _refused(zg.ZERO_EINVAL, f, p, A, 1.0, 1.0, A, A, A)
    _refused(zg.ZERO_EINVAL, zg.zero_adamw_clip, p, A, A)


@pytest.mark.parametrize("bits", [8, 32])
def test_clip_and_step_refusals(bits):
    p, hp = _plan(100, bits=bits), zg.zero_adamw_t(t=1, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, grad_scale=1.0)
    _refused(zg.ZERO_ENOMEM, zg.zero_adamw_clip, p, A, None)
    _refused(zg.ZERO_ENOMEM, zg.zero_adamw_clip, p, None, A)
    _refused(zg.ZERO_EALIGN, zg.zero_adamw_clip, p, A, A + 1)
    f = zg.zero_adamw_step_clipped
    _refused(zg.ZERO_ENOMEM, f, p, A, hp, None, None)
    _refused(zg.ZERO_EALIGN, f, p, A, hp, A + 2, None)
    _refused(zg.ZERO_EALIGN, f, p, A, hp, A, A + 2)
    _refused(zg.ZERO_ENOMEM, f, p, None, hp, A, None)
    hp.t = 0
    _refused(zg.ZERO_EINVAL, f, p, A, hp, A, None)


def test_empty_list_is_no_launch():
    hp = zg.zero_adamw_t(t=1, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, grad_scale=1.0)
    zg.zero_adamw_clip(_plan(), None, A)
    zg.zero_adamw_step_clipped(_plan(), None, hp, A)
