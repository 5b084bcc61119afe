"""Log probabilities' host side: plans and refusals.  No call here reaches a
CUDA API."""
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
    m = re.search(r"(\d+) bytes\. \*/\s*typedef struct zero_lp_plan \{", text)
    assert m and ctypes.sizeof(zg.zero_lp_plan_t) == int(m.group(1))


@pytest.mark.parametrize("n,v,d,top", [(0, 10, 8, 0), (1, 50257, 4096, 8), (8192, 50257, 768, 0), (20_000, 50257, 64, 32), (5, 1 << 24, 8, 32)])
def test_plan(n, v, d, top):
    p, c = zg.zero_lp_plan(n, v, d, zg.ZERO_BF16, top=top), zg.zero_ce_plan(n, v, d, zg.ZERO_BF16)
    assert (p.tokens, p.vocab, p.hidden, p.top, p.piece, p.splits) == (n, v, d, top, c.piece, c.splits)
    assert p.flops_forward == 2 * n * v * d and p.flops_backward == 6 * n * v * d
    assert p.workspace_bytes >= c.workspace_bytes and p.rows % 256 == 0 and p.rows >= 256
    strips = -(-v // 256) * 2
    assert p.workspace_bytes <= max(c.workspace_bytes, (5 << 29) + min(n, 256) * strips * (12 + 512))
    if n > 3:
        assert p.workspace_bytes >= min(n, p.rows) * (strips * 12 + (4 * v if top else 0))


def test_plan_refusals():
    P, BF = zg.zero_lp_plan, zg.ZERO_BF16
    _refused(zg.ZERO_EUNSUPPORTED, P, 4, 10, 8, zg.ZERO_FP32)
    _refused(zg.ZERO_EUNSUPPORTED, P, 4, 10, 8, BF, top=33)
    _refused(zg.ZERO_EINVAL, P, 4, 10, 8, BF, top=-1)
    _refused(zg.ZERO_EINVAL, P, -1, 10, 8, BF)
    _refused(zg.ZERO_EINVAL, P, 4, 0, 8, BF)
    _refused(zg.ZERO_EALIGN, P, 4, 10, 33, BF)
    _refused(zg.ZERO_EUNSUPPORTED, P, (1 << 24) + 1, 10, 8, BF)
    assert zg.lib().zero_lp_plan(1, 1, 8, BF, 0, 0, 0, 0, None) == zg.ZERO_EINVAL
    assert P(4, 10, 8, BF, top=32).top == 32          # more than there are entries


def test_forward_refusals():
    p, q, F = zg.zero_lp_plan(4, 100, 64, top=3), zg.zero_lp_plan(4, 100, 64), zg.zero_lp_forward
    ok = [A, A, A, 1.0, A, A, A, A, A, A]             # x w targets scale logp lse entropy top_logp top_index workspace
    for k in (0, 1, 2, 4, 5, 7, 8, 9):
        a = list(ok)
        a[k] = None
        _refused(zg.ZERO_ENOMEM, F, p, *a)
    for k, off in ((0, 8), (1, 2), (2, 4), (4, 2), (5, 2), (6, 1), (7, 2), (8, 4), (9, 8)):
        a = list(ok)
        a[k] = A + off
        _refused(zg.ZERO_EALIGN, F, p, *a)
    for scale in (0.0, -1.0, float("inf"), float("nan"), 3e38):
        _refused(zg.ZERO_EINVAL, F, p, A, A, A, scale, A, A, A, A, A, A)
    _refused(zg.ZERO_EINVAL, F, q, *ok)               # alternatives that the plan has not
    p.rows += 256
    _refused(zg.ZERO_EINVAL, F, p, *ok)


def test_backward_and_status_refusals():
    p, B = zg.zero_lp_plan(4, 100, 64), zg.zero_lp_backward
    ok = [A, A, A, 1.0, A, A, A, A, 1.0, A, A, A]     # x w targets scale lse entropy dlogp dentropy grad_scale dx dw workspace
    for k in (0, 1, 2, 4, 5, 11):
        a = list(ok)
        a[k] = None
        _refused(zg.ZERO_ENOMEM, B, p, *a)
    for k, off in ((0, 8), (1, 8), (2, 4), (4, 2), (5, 2), (6, 2), (7, 1), (9, 8), (10, 2), (11, 8)):
        a = list(ok)
        a[k] = A + off
        _refused(zg.ZERO_EALIGN, B, p, *a)
    for k, bad in ((3, 0.0), (3, float("nan")), (8, float("inf")), (8, float("nan"))):
        a = list(ok)
        a[k] = bad
        _refused(zg.ZERO_EINVAL, B, p, *a)
    _refused(zg.ZERO_ENOMEM, zg.zero_lp_status, p, None)
    _refused(zg.ZERO_EALIGN, zg.zero_lp_status, p, A + 4)
    p.splits += 1
    _refused(zg.ZERO_EINVAL, B, p, *ok)
    _refused(zg.ZERO_EINVAL, zg.zero_lp_status, p, A)
