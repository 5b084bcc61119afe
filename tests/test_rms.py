"""The root-mean-square norm's host side: plans and refusals.  No call here
reaches a CUDA API."""
import ctypes
import os
import re

import pytest

import zero_sharded_mixed_bucket_gb300 as zg
from tests.conftest import ROOT

A = 1 << 20            # an aligned address, never read


def _refused(status, f, *args, **kw):
    with pytest.raises(zg.ZeroError) as e:
        f(*args, **kw)
    assert e.value.status == status and str(e.value)


def test_struct_size_matches_header():
    text = open(os.path.join(ROOT, "include", "zero_gb300.h"), encoding="utf-8").read()
    m = re.search(r"(\d+) bytes\. \*/\s*typedef struct zero_rms_plan \{", text)
    assert m and ctypes.sizeof(zg.zero_rms_plan_t) == int(m.group(1))


@pytest.mark.parametrize("dtype,e", [(zg.ZERO_FP16, 2), (zg.ZERO_BF16, 2), (zg.ZERO_FP32, 4)])
@pytest.mark.parametrize("block,cols", [(0, 0), (32, 25), (128, 7)])
def test_plan(dtype, e, block, cols):
    p = zg.zero_rms_plan(1003, 771, dtype, 776, 0, block)
    assert (p.rows, p.dim, p.x_stride, p.y_stride, p.block, p.scale_cols) == (1003, 771, 776, 771, block, cols)
    out = 771 + cols if block else 771 * e
    assert p.hbm_bytes_forward == 1003 * (3 * 771 * e + 4 + out) + 771 * e
    assert p.hbm_bytes_backward == 1003 * (4 * 771 * e + 4) + 2 * 771 * e
    assert 1 <= p.blocks <= 152 * 16 and p.workspace_bytes == 16 + p.blocks * 771 * 4
    assert zg.zero_rms_plan(0, 1, dtype).blocks == 0


def test_plan_refusals():
    _refused(zg.ZERO_EINVAL, zg.zero_rms_plan, -1, 8)
    _refused(zg.ZERO_EINVAL, zg.zero_rms_plan, 1, 0)
    _refused(zg.ZERO_EINVAL, zg.zero_rms_plan, 1, 8, 3)
    _refused(zg.ZERO_EINVAL, zg.zero_rms_plan, 1, 8, 0, 7)
    _refused(zg.ZERO_EINVAL, zg.zero_rms_plan, 1, 8, 0, 0, 7)
    _refused(zg.ZERO_EUNSUPPORTED, zg.zero_rms_plan, 1, 8, 0, 0, 0, 64)
    _refused(zg.ZERO_EUNSUPPORTED, zg.zero_rms_plan, 1, (1 << 20) + 1)
    _refused(zg.ZERO_EUNSUPPORTED, zg.zero_rms_plan, (1 << 40) + 1, 8)
    _refused(zg.ZERO_EUNSUPPORTED, zg.zero_rms_plan, 1 << 30, 8, 0, 1 << 40)
    with pytest.raises(zg.ZeroError):
        zg._check(zg.lib().zero_rms_plan(1, 8, 0, 0, 0, 0, None))


def test_forward_refusals():
    p, q = zg.zero_rms_plan(4, 64), zg.zero_rms_plan(4, 64, block=32)
    f = zg.zero_rms_forward
    _refused(zg.ZERO_EINVAL, f, p, A, None, A, -1.0, None, A)
    _refused(zg.ZERO_EINVAL, f, p, A, None, A, float("nan"), None, A)
    _refused(zg.ZERO_EINVAL, f, p, A, None, A, 1e-5, A, A)                    # h without a residual
    _refused(zg.ZERO_EINVAL, f, p, A, None, A, 1e-5, None, A, A, A)           # 8 bits without a block
    _refused(zg.ZERO_ENOMEM, f, p, None, None, A, 1e-5, None, A)
    _refused(zg.ZERO_ENOMEM, f, p, A, None, A, 1e-5, None, None)
    _refused(zg.ZERO_ENOMEM, f, p, A, A, A, 1e-5, None, A)                    # a residual without h
    _refused(zg.ZERO_ENOMEM, f, q, A, None, A, 1e-5, None, None, A, None)
    for k in range(6):
        v = [A, A, A, A, A, A]
        v[k] += 2 if k == 5 else 1
        _refused(zg.ZERO_EALIGN, f, p, v[0], v[1], v[2], 1e-5, v[3], v[4], None, None, v[5])
    p.dim = 65
    _refused(zg.ZERO_EINVAL, f, p, A, None, A, 1e-5, None, A)
    _refused(zg.ZERO_EINVAL, f, None_plan(), A, None, A, 1e-5, None, A)


def None_plan():
    return zg.zero_rms_plan_t()


def test_values_and_backward_refusals():
    p, q = zg.zero_rms_plan(4, 64), zg.zero_rms_plan(4, 64, block=32)
    _refused(zg.ZERO_EINVAL, zg.zero_rms_values, p, A, A, A)
    _refused(zg.ZERO_ENOMEM, zg.zero_rms_values, q, None, A, A)
    _refused(zg.ZERO_ENOMEM, zg.zero_rms_values, q, A, None, A)
    _refused(zg.ZERO_ENOMEM, zg.zero_rms_values, q, A, A, None)
    _refused(zg.ZERO_EALIGN, zg.zero_rms_values, q, A, A, A + 1)
    b = zg.zero_rms_backward
    _refused(zg.ZERO_ENOMEM, b, p, None, None, A, A, A, A, A, A)
    _refused(zg.ZERO_ENOMEM, b, p, A, None, None, A, A, A, A, A)
    _refused(zg.ZERO_ENOMEM, b, p, A, None, A, A, None, A, A, A)
    _refused(zg.ZERO_ENOMEM, b, p, A, None, A, A, A, A, A, None)
    for k in range(8):
        v = [A] * 8
        v[k] += 8 if k == 7 else 2 if k == 4 else 1
        _refused(zg.ZERO_EALIGN, b, p, *v)


def test_no_rows_is_no_launch():
    p = zg.zero_rms_plan(0, 64, block=32)
    zg.zero_rms_forward(p, None, None, None, 1e-5, None, None)
    zg.zero_rms_values(p, None, None, None)
    zg.zero_rms_backward(p, None, None, None, None, None)
