"""Cross entropy over a vocabulary, host side: plans and refusals.  No call
here reaches a CUDA API."""
import ctypes
import os
import re

import pytest

import zero_sharded_mixed_bucket_gb300 as zg
from tests.conftest import ROOT

A = 1 << 20            # an aligned address, never read


def _refused(status, f, *args):
    with pytest.raises(zg.ZeroError) as e:
        f(*args)
    assert e.value.status == status and str(e.value)


def test_struct_size_matches_header():
    text = open(os.path.join(ROOT, "include", "zero_gb300.h"), encoding="utf-8").read()
    m = re.search(r"(\d+) bytes\. \*/\s*typedef struct zero_ce_plan \{", text)
    assert ctypes.sizeof(zg.zero_ce_plan_t) == int(m.group(1))


@pytest.mark.parametrize("n,v,d", [(1, 1, 8), (1, 50257, 4096), (8192, 50257, 768), (300, 257, 64), (0, 10, 8)])
def test_plan(n, v, d):
    p = zg.zero_ce_plan(n, v, d, zg.ZERO_BF16)
    assert (p.x_stride, p.w_stride) == (d, d)
    assert p.flops_forward == 2 * n * v * d and p.flops_backward == 3 * p.flops_forward
    assert p.piece % 256 == 0 and 256 <= p.piece <= (v + 255) // 256 * 256
    assert 1 <= p.splits <= 32
    # no logits in memory: G of a piece, not of the vocabulary, where that is large
    assert n * p.piece * 2 <= (1 << 29) + n * 512
    assert zg.zero_ce_plan(n, v, d, zg.ZERO_BF16, piece=100).piece == 256
    assert p.workspace_bytes >= n * p.piece * 2


def test_plan_refusals():
    P, BF = zg.zero_ce_plan, zg.ZERO_BF16
    _refused(zg.ZERO_EUNSUPPORTED, P, 4, 10, 8, zg.ZERO_FP32)
    _refused(zg.ZERO_EINVAL, P, 4, 10, 8, 7)
    _refused(zg.ZERO_EINVAL, P, -1, 10, 8, BF)
    _refused(zg.ZERO_EINVAL, P, 4, 0, 8, BF)
    _refused(zg.ZERO_EINVAL, P, 4, 10, 0, BF)
    _refused(zg.ZERO_EALIGN, P, 4, 10, 33, BF)
    _refused(zg.ZERO_EALIGN, P, 4, 10, 8, BF, 12)
    _refused(zg.ZERO_EALIGN, P, 4, 10, 8, BF, 8, 20)
    _refused(zg.ZERO_EINVAL, P, 4, 10, 16, BF, 8)
    _refused(zg.ZERO_EINVAL, P, 4, 10, 16, BF, 0, 8)
    _refused(zg.ZERO_EINVAL, P, 4, 10, 16, BF, 0, 0, -256)
    _refused(zg.ZERO_EUNSUPPORTED, P, (1 << 24) + 1, 10, 8, BF)
    _refused(zg.ZERO_EUNSUPPORTED, P, 4, (1 << 24) + 1, 8, BF)
    assert P(4, 10, 33, BF, 40, 40).hidden == 33


def test_call_refusals():
    p = zg.zero_ce_plan(4, 100, 64, zg.ZERO_FP16)
    F, B = zg.zero_ce_forward, zg.zero_ce_backward
    ok = [A] * 7
    for k in (0, 1, 2, 3, 4, 6):
        a = list(ok)
        a[k] = None
        _refused(zg.ZERO_ENOMEM, F, p, *a)
    for k, off in ((0, 8), (1, 2), (2, 4), (3, 2), (4, 1), (5, 2), (6, 8)):
        a = list(ok)
        a[k] = A + off
        _refused(zg.ZERO_EALIGN, F, p, *a)
    ok = [A, A, A, A, None, 1.0, A, A, A]                      # x w targets lse dloss scale dx dw workspace
    for k in (0, 1, 2, 3, 8):
        a = list(ok)
        a[k] = None
        _refused(zg.ZERO_ENOMEM, B, p, *a)
    for k, off in ((0, 8), (1, 8), (2, 4), (3, 2), (4, 2), (6, 8), (7, 2), (8, 8)):
        a = list(ok)
        a[k] = A + off
        _refused(zg.ZERO_EALIGN, B, p, *a)
    _refused(zg.ZERO_EINVAL, B, p, A, A, A, A, None, float("inf"), A, A, A)
    _refused(zg.ZERO_ENOMEM, zg.zero_ce_status, p, None)
    _refused(zg.ZERO_EALIGN, zg.zero_ce_status, p, A + 4)
    p.splits += 1
    for f, a in ((F, [A] * 7), (B, ok), (zg.zero_ce_status, [A])):
        _refused(zg.ZERO_EINVAL, f, p, *a)


@pytest.mark.parametrize("piece", [1 << 62, (1 << 63) - 256, (1 << 63) - 1])
def test_plan_of_a_huge_piece(piece):
    p, q = zg.zero_ce_plan(8, 1000, 64, zg.ZERO_BF16, piece=piece), zg.zero_ce_plan(8, 1000, 64, zg.ZERO_BF16, piece=1024)
    assert bytes(p) == bytes(q) and p.piece == 1024


def test_plan_counts_stay_in_range():
    """Sizes that are each allowed, but whose product is not."""
    for n, v, d in ((1 << 24, 1 << 22, 1 << 18), (1 << 24, 1 << 22, 1 << 13), (1 << 24, 8, 1 << 20), (1 << 20, 1 << 20, 1 << 20),
                    (8, 1 << 24, 1 << 20), (1 << 24, 1 << 22, 4096), (1 << 20, 1 << 18, 1 << 20)):
        try:
            p = zg.zero_ce_plan(n, v, d, zg.ZERO_BF16)
        except zg.ZeroError as e:
            assert e.status == zg.ZERO_EUNSUPPORTED and n * v * d >= 1 << 57
            continue
        assert p.flops_forward == 2 * n * v * d and p.flops_backward == 6 * n * v * d
        assert p.workspace_bytes >= n * p.piece * 2
        tiles = -(-n // 256) * -(-v // 256)
        assert tiles / 76 * -(-d // 64) < 1 << 31            # K-blocks that one pair of SMs counts
    _refused(zg.ZERO_EUNSUPPORTED, zg.zero_ce_plan, 1 << 24, 1 << 22, 1 << 18, zg.ZERO_BF16)
    assert zg.zero_ce_plan(1 << 20, 1 << 18, 1 << 14, zg.ZERO_BF16).flops_forward == 1 << 53
