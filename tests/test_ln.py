"""Layer norm's host side: plans and refusals.  No call here reaches a CUDA API."""
import ctypes
import os
import re

import pytest

import zero_sharded_mixed_bucket_gb300 as zg
from tests.conftest import ROOT


def test_struct_size_matches_header():
    text = open(os.path.join(ROOT, "include", "zero_gb300.h"), encoding="utf-8").read()
    m = re.search(r"(\d+) bytes\. \*/\s*typedef struct zero_ln_plan \{", text)
    assert ctypes.sizeof(zg.zero_ln_plan_t) == int(m.group(1))


@pytest.mark.parametrize("rows,dim,dtype,e", [(1, 1, zg.ZERO_FP16, 2), (7, 768, zg.ZERO_BF16, 2), (1003, 771, zg.ZERO_FP32, 4)])
def test_plan_sizes(rows, dim, dtype, e):
    p = zg.zero_ln_plan(rows, dim, dtype)
    assert (p.x_stride, p.y_stride) == (dim, dim)
    assert p.hbm_bytes_forward == 2 * rows * dim * e + 8 * rows + 2 * dim * e
    assert p.hbm_bytes_backward == 3 * rows * dim * e + 8 * rows + 3 * dim * e
    assert p.workspace_bytes >= p.blocks * dim * 8 and p.workspace_bytes % 4 == 0
    q = zg.zero_ln_plan(rows, dim, dtype, dim + 3, dim + 8)
    assert (q.x_stride, q.y_stride) == (dim + 3, dim + 8)


@pytest.mark.parametrize("args,status", [
    ((-1, 8), zg.ZERO_EINVAL), ((4, 0), zg.ZERO_EINVAL), ((4, 8, 9), zg.ZERO_EINVAL),
    ((4, 8, zg.ZERO_FP16, 7), zg.ZERO_EINVAL), ((4, 8, zg.ZERO_FP16, 0, 5), zg.ZERO_EINVAL),
    ((4, (1 << 20) + 1), zg.ZERO_EUNSUPPORTED), (((1 << 40) + 1, 8), zg.ZERO_EUNSUPPORTED),
    ((1 << 40, 8, zg.ZERO_FP16, 1 << 40), zg.ZERO_EUNSUPPORTED),
])
def test_plan_refusals(args, status):
    with pytest.raises(zg.ZeroError) as e:
        zg.zero_ln_plan(*args)
    assert e.value.status == status and "zero_ln_plan" in str(e.value)


def _refused(status, f, *args):
    with pytest.raises(zg.ZeroError) as e:
        f(*args)
    assert e.value.status == status


def test_call_refusals():
    p = zg.zero_ln_plan(4, 64, zg.ZERO_BF16)
    F, B, A = zg.zero_ln_forward, zg.zero_ln_backward, 1 << 20        # A: an aligned address, never read
    _refused(zg.ZERO_ENOMEM, F, p, None, A, A, 1e-5, A)
    _refused(zg.ZERO_ENOMEM, F, p, A, A, A, 1e-5, None)
    _refused(zg.ZERO_EINVAL, F, p, A, A, A, -1.0, A)
    _refused(zg.ZERO_EINVAL, F, p, A, A, A, float("nan"), A)
    for k in (0, 1, 2, 4):
        args = [A, A, A, 1e-5, A]
        if k != 3:
            args[k] = A + 1
        _refused(zg.ZERO_EALIGN, F, p, *args)
    _refused(zg.ZERO_EALIGN, F, p, A, A, A, 1e-5, A, A + 2)
    _refused(zg.ZERO_ENOMEM, B, p, None, A, A, A, A, A)
    _refused(zg.ZERO_ENOMEM, B, p, A, A, A, None, A, A)
    _refused(zg.ZERO_ENOMEM, B, p, A, A, A, A, A, A, A, None, None)
    _refused(zg.ZERO_EALIGN, B, p, A, A, A, A, A, A + 1)
    _refused(zg.ZERO_EALIGN, B, p, A, A, A, A, A, A, A, A, A + 8)
    p.blocks += 1
    _refused(zg.ZERO_EINVAL, F, p, A, A, A, 1e-5, A)
    _refused(zg.ZERO_EINVAL, B, p, A, A, A, A, A, A, A, A, A)


def test_plan_byte_counts_stay_in_range():
    """Rows and widths that are each allowed: the counts of bytes are right, or the plan is refused."""
    for rows, dim in ((1 << 40, (1 << 20) - 1), (1 << 40, 1 << 19), (1 << 39, (1 << 20) - 3), (1 << 38, 1 << 20)):
        for dtype, e in ((zg.ZERO_FP32, 4), (zg.ZERO_BF16, 2)):
            try:
                p = zg.zero_ln_plan(rows, dim, dtype)
            except zg.ZeroError as err:
                assert err.status == zg.ZERO_EUNSUPPORTED and rows * dim > 1 << 58
                continue
            assert p.hbm_bytes_forward == 2 * rows * dim * e + 8 * rows + 2 * dim * e
            assert p.hbm_bytes_backward == 3 * rows * dim * e + 8 * rows + 3 * dim * e
