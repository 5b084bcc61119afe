"""The list-of-tensors AdamW step's host side: plans and refusals.  No call
here reaches a CUDA API."""
import ctypes
import os
import re

import pytest

import zero_sharded_mixed_bucket_gb300 as zg
from tests.conftest import ROOT

A = 1 << 20            # an aligned address, never read


def _t(numel=10, **k):
    d = {"grad": A, "master": A, "m": A, "v": A, "param": A}
    d.update(k)
    return zg.adamw_tensor(numel=numel, **d)


def _refused(status, f, *args):
    with pytest.raises(zg.ZeroError) as e:
        f(*args)
    assert e.value.status == status and str(e.value)


def test_struct_sizes_match_header():
    text = open(os.path.join(ROOT, "include", "zero_gb300.h"), encoding="utf-8").read()
    for name, cls in (("zero_adamw_tensor", zg.zero_adamw_tensor_t), ("zero_adamw_plan", zg.zero_adamw_plan_t),
                      ("zero_adamw", zg.zero_adamw_t)):
        m = re.search(r"(\d+) bytes\. \*/\s*typedef struct %s \{" % name, text)
        assert m and ctypes.sizeof(cls) == int(m.group(1)), name


@pytest.mark.parametrize("dtype,e", [(zg.ZERO_FP16, 2), (zg.ZERO_BF16, 2), (zg.ZERO_FP32, 4)])
@pytest.mark.parametrize("bits,per", [(32, 24), (8, 12)])
def test_plan(dtype, e, bits, per):
    sizes = [1, 0, 256, 257, 100_003]
    p = zg.zero_adamw_plan([_t(n) for n in sizes], dtype, bits)
    assert p.n_tensors == 5 and p.numel == sum(sizes)
    assert p.flat_elems == 256 + 0 + 256 + 512 + 100_096
    assert p.hbm_bytes == sum(sizes) * (2 * e + per)
    assert p.table_bytes > 0
    empty = zg.zero_adamw_plan([], dtype, bits)
    assert empty.n_tensors == empty.numel == empty.n_chunks == 0


def test_plan_refusals():
    _refused(zg.ZERO_EINVAL, zg.zero_adamw_plan, [_t(-1)])
    _refused(zg.ZERO_EINVAL, zg.zero_adamw_plan, [_t()], 3)
    _refused(zg.ZERO_EUNSUPPORTED, zg.zero_adamw_plan, [_t()], zg.ZERO_FP16, 16)
    _refused(zg.ZERO_EUNSUPPORTED, zg.zero_adamw_plan, [_t(1 << 40), _t(1)])
    _refused(zg.ZERO_EINVAL, zg.zero_adamw_plan, [_t(weight_decay=float("nan"))])
    with pytest.raises(zg.ZeroError):
        zg._check(zg.lib().zero_adamw_plan(None, 3, zg.ZERO_FP16, 32, ctypes.byref(zg.zero_adamw_plan_t())))


def test_table_refusals():
    t = [_t()]
    p = zg.zero_adamw_plan(t)
    I = zg.zero_adamw_table_init
    _refused(zg.ZERO_ENOMEM, I, p, t, None)
    _refused(zg.ZERO_EALIGN, I, p, t, A + 8)
    _refused(zg.ZERO_EINVAL, I, p, [], A)
    _refused(zg.ZERO_EINVAL, I, p, [_t(5000)], A)
    for k in ("grad", "master", "m", "v"):
        _refused(zg.ZERO_ENOMEM, I, p, [_t(**{k: None})], A)
        _refused(zg.ZERO_EALIGN, I, p, [_t(**{k: A + 1})], A)
    _refused(zg.ZERO_EALIGN, I, p, [_t(param=A + 1)], A)
    p8 = zg.zero_adamw_plan(t, zg.ZERO_FP16, 8)
    _refused(zg.ZERO_ENOMEM, I, p8, t, A)                      # no scale bytes
    p.table_bytes += 4
    _refused(zg.ZERO_EINVAL, I, p, t, A)


def test_step_refusals():
    p = zg.zero_adamw_plan([_t()])
    ok = {"t": 1, "lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "grad_scale": 1.0}
    for k, v in (("t", 0), ("t", -3), ("beta1", 1.0), ("beta1", -0.1), ("beta2", 1.0), ("beta2", float("nan")),
                 ("eps", -1.0), ("eps", float("nan")), ("lr", float("inf")), ("grad_scale", float("nan"))):
        _refused(zg.ZERO_EINVAL, zg.zero_adamw_step, p, A, zg.zero_adamw_t(**{**ok, k: v}))
    _refused(zg.ZERO_ENOMEM, zg.zero_adamw_step, p, None, zg.zero_adamw_t(**ok))
    _refused(zg.ZERO_EALIGN, zg.zero_adamw_step, p, A + 4, zg.zero_adamw_t(**ok))
    _refused(zg.ZERO_EALIGN, zg.zero_adamw_step, p, A, zg.zero_adamw_t(**ok), A + 2)
    _refused(zg.ZERO_ENOMEM, zg.zero_adamw_check, p, A, None)
    _refused(zg.ZERO_EALIGN, zg.zero_adamw_check, p, A, A + 1)
    _refused(zg.ZERO_EINVAL, zg.zero_adamw_states, p, A, A, A)
    p8 = zg.zero_adamw_plan([_t(m_scale=A, v_scale=A)], zg.ZERO_BF16, 8)
    _refused(zg.ZERO_ENOMEM, zg.zero_adamw_states, p8, A, None, A)
    _refused(zg.ZERO_EALIGN, zg.zero_adamw_states, p8, A, A, A + 2)


@pytest.mark.parametrize("numel,flat,chunks", [(1 << 62, 1 << 62, 3), (4300, 1 << 20, 3), (4300, 4608, 1), (4300, 4608, 40)])
def test_plans_that_no_list_has(numel, flat, chunks):
    """Counts that agree with one another, but not with any list of two tensors:
    with more chunks than the table was filled for, what lies past it would be read."""
    p = zg.zero_adamw_plan([_t(4200), _t(100)], zg.ZERO_BF16, 32)
    assert (p.numel, p.flat_elems, p.n_chunks) == (4300, 4608, 3)
    p.table_bytes += 4 * (chunks - 3)
    p.numel, p.flat_elems, p.n_chunks, p.hbm_bytes = numel, flat, chunks, (numel * 28 + (1 << 63)) % (1 << 64) - (1 << 63)
    hp = zg.zero_adamw_t(t=1, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, grad_scale=1.0)
    _refused(zg.ZERO_EINVAL, zg.zero_adamw_step, p, A, hp)
    _refused(zg.ZERO_EINVAL, zg.zero_adamw_check, p, A, A)
