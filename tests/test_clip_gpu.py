"""The gradient norm of a list, clipping and the clipped step on the GPU.

Bound of the norm: squares of up to 32 values are summed in binary32, so the sum of
squares is off by 33 half units in the last place at most, its root by half
of that; the result rounds to binary32 once."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucket_gb300 as zg
from tests.test_adamw_gpu import DT, SIZES, Tensors, _bits, _hp

pytestmark = pytest.mark.gpu

F, U = np.float32, 2.0 ** -24


class Norm:
    def __init__(self, plan):
        self.norm = torch.full((2,), -7.0, device="cuda")
        self.flag = torch.full((1,), 9, dtype=torch.int32, device="cuda")
        self.ws = torch.full((zg.zero_adamw_norm_workspace(plan),), 0xFF, dtype=torch.uint8, device="cuda")

    def of(self, T, scale, most, flag=True, stream=None):
        zg.zero_adamw_norm(T.plan, T.table, scale, most, self.norm, self.flag if flag else None, self.ws, stream)
        return float(self.norm[0]), float(self.norm[1]), int(self.flag[0])


def _norm64(T, scale):
    return abs(float(F(scale))) * float(np.sqrt(sum((T.host(k, "grad").astype(np.float64) ** 2).sum() for k in range(len(T.sizes)))))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shifts", [(0,), (1, 0, 3)])
@pytest.mark.parametrize("sizes", SIZES + [[], [0], [5_000_011, 1]], ids=str)
def test_norm(sizes, shifts, dtype):
    T = Tensors(sizes, dtype, 32, seed=3, shifts=shifts)
    N = Norm(T.plan)
    want = _norm64(T, 0.125)
    for most in (0.0, -1.0, 2 * want + 1, 0.25 * want):
        norm, factor, flag = N.of(T, -0.125, most)
        assert abs(norm - want) <= want * U * 18 and flag == 0
        f64 = min(1.0, most / (want + 1e-6)) if most > 0 else 1.0
        assert abs(factor - f64) <= f64 * U * 20
        assert f64 < 1.0 or factor == 1.0
    again = Norm(T.plan)
    again.of(T, -0.125, 0.25 * want)
    assert torch.equal(again.norm, N.norm)            # equal bits
    N.flag.fill_(9)
    assert N.of(T, 0.125, 1.0, flag=False)[2] == 9
    assert T.guards_kept()


def _filled(dtype, n, shift=0):
    return Tensors([n, 40, 0, 5000], dtype, 32, seed=1, shifts=(shift,))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [3e38, 1e30, 1e19, 1e-19, 1e-25, 1e-37, 1e-39])
def test_norm_where_squares_leave_binary32(size, dtype):
    """Squares that overflow or underflow binary32, in batches of their own, together with ordinary ones, alone."""
    T = _filled(dtype, 9001)
    for what in ("all", "some", "one"):
        for k in (0, 1, 3):
            g = T.view[k]["grad"]
            g.copy_(torch.randn(g.numel(), device="cuda", generator=torch.Generator(device="cuda").manual_seed(k)) if what == "some"
                    else torch.zeros_like(g))
            if what == "one":
                g[-1] = size
            else:
                g[:: 1 if what == "all" else 97] = size
        N = Norm(T.plan)
        scale = 1.0 if size < 1 else 2.0 ** -20       # the norm itself stays in range
        norm, _, flag = N.of(T, scale, 1.0)
        want = _norm64(T, scale)
        assert flag == 0 and abs(norm - want) <= want * U * 18 + 2.0 ** -150, what


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_norm_of_gradients_that_are_not_finite(bad, shift, dtype):
    T = _filled(dtype, 70_001, shift)
    N = Norm(T.plan)
    for k, at in ((0, 0), (0, 70_000), (1, 39), (3, 4097)):
        g = T.view[k]["grad"]
        old = g[at].clone()
        g[at] = bad
        norm, factor, flag = N.of(T, 1.0, 1.0)
        check = torch.zeros(1, dtype=torch.int32, device="cuda")
        zg.zero_adamw_check(T.plan, T.table, check, torch.cuda.current_stream())
        assert flag == 1 == int(check)
        assert (np.isnan(norm) and np.isnan(factor)) if np.isnan(bad) else (norm == np.inf and factor == 0)
        g[at] = old
        assert N.of(T, 1.0, 1.0)[2] == 0


@pytest.mark.parametrize("n", [9001, 500_001])        # one block alone, and two kernels
@pytest.mark.parametrize("most", [0.0, -1.0, float("inf"), float("-inf")])
def test_no_clipping_whatever_the_gradients(most, n):
    """A max_norm <= 0 or infinite: the factor is 1, also of gradients that are not finite; norm and flag say what they are."""
    T = _filled("fp32", n)
    N = Norm(T.plan)
    for bad in (None, float("inf"), float("-inf"), float("nan")):
        if bad is not None:
            T.view[3]["grad"][4097] = bad
        norm, factor, flag = N.of(T, 1.0, most)
        assert factor == 1.0 and flag == (bad is not None)
        assert np.isnan(norm) if bad != bad else norm == np.inf if bad else np.isfinite(norm)
        norm, factor, flag = N.of(T, 0.0, most)       # 0 times an infinity is NaN, as the formula has it
        assert factor == 1.0 and flag == (bad is not None) and (np.isnan(norm) if bad else norm == 0)
    norm, factor, flag = N.of(T, 0.0, 1.0)
    assert np.isnan(norm) and np.isnan(factor) and flag == 1


def test_norm_of_zeros():
    T = _filled("bf16", 9001)
    for k in (0, 1, 3):
        T.view[k]["grad"].fill_(-0.0)
    assert Norm(T.plan).of(T, 1.0, 1.0) == (0.0, 1.0, 0)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shifts", [(0,), (1, 0, 3)])
def test_clip_in_place(shifts, dtype):
    T = Tensors([1, 4097, 0, 12_345, 8192], dtype, 32, seed=4, shifts=shifts)
    N = Norm(T.plan)
    old = [v["grad"].clone() for v in T.view]
    N.of(T, 1.0, 0.0)
    zg.zero_adamw_clip(T.plan, T.table, N.norm, torch.cuda.current_stream())     # factor 1
    assert all(torch.equal(a, v["grad"]) for a, v in zip(old, T.view))
    norm, factor, _ = N.of(T, 1.0, 0.5)
    assert factor < 1
    zg.zero_adamw_clip(T.plan, T.table, N.norm, torch.cuda.current_stream())
    for a, v in zip(old, T.view):
        assert torch.equal((a.float() * N.norm[1]).to(a.dtype), v["grad"])
    norm, _, _ = N.of(T, 1.0, 0.0)
    assert abs(norm - 0.5) <= 0.5 * torch.finfo(DT[dtype][1]).eps + 1e-5         # each value rounded to its type; the 1e-6 beside the norm
    assert T.guards_kept()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("bits", [8, 32])
def test_clipped_step_is_the_step_of_scaled_gradients(bits, dtype):
    """Bit for bit: the two factors' product, rounded once, is the gradients' scale."""
    sizes = [1, 4097, 0, 12_345, 256]
    A, B = (Tensors(sizes, dtype, bits, seed=6, shifts=(0, 1)) for _ in range(2))
    N = Norm(A.plan)
    _, factor, _ = N.of(A, 0.125, 0.01)
    assert 0 < factor < 1
    s = torch.cuda.current_stream()
    zg.zero_adamw_step_clipped(A.plan, A.table, _hp(), N.norm, None, s)
    zg.zero_adamw_step(B.plan, B.table, _hp(grad_scale=float(F(factor) * F(0.125))), None, s)
    plain = Tensors(sizes, dtype, bits, seed=6, shifts=(0, 1))
    zg.zero_adamw_step(plain.plan, plain.table, _hp(), None, s)
    for a, b in zip(A.view, B.view):
        for name in a:
            assert torch.equal(a[name], b[name]), name
    assert not torch.equal(A.view[1]["m"], plain.view[1]["m"])
    assert A.guards_kept()
    # the flag stops it
    old = [{k: t.clone() for k, t in v.items()} for v in A.view]
    A.view[3]["grad"][7] = float("inf")
    N.of(A, 0.125, 0.01)
    zg.zero_adamw_step_clipped(A.plan, A.table, _hp(t=4), N.norm, N.flag, s)
    for a, b in zip(A.view, old):
        assert all(torch.equal(a[n], b[n]) for n in a if n != "grad")


def test_graph_replays_and_streams():
    """The norm and the step captured once, replayed over changing gradients; two lists' norms at the same time."""
    T, P = (Tensors([400_003, 2, 640], "bf16", 32, seed=8) for _ in range(2))
    N, M = Norm(T.plan), Norm(P.plan)
    st, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            s = torch.cuda.current_stream()
            zg.zero_adamw_norm(T.plan, T.table, 0.125, 0.5, N.norm, N.flag, N.ws, s)
            zg.zero_adamw_step_clipped(T.plan, T.table, _hp(), N.norm, N.flag, s)
    for turn in range(3):
        for X in (T, P):
            X.view[0]["grad"].copy_(torch.randn(400_003, device="cuda", generator=torch.Generator(device="cuda").manual_seed(turn)) * 10 ** turn)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(other):
            M.of(P, 0.125, 0.5, stream=other)
            zg.zero_adamw_step_clipped(P.plan, P.table, _hp(), M.norm, M.flag, other)
        torch.cuda.synchronize()
        assert torch.equal(N.norm, M.norm) and abs(float(N.norm[0]) - _norm64(T, 0.125)) <= _norm64(T, 0.125) * U * 18
        for a, b in zip(T.view, P.view):
            assert all(torch.equal(a[n], b[n]) for n in a)


def test_offsets_past_32_bits():
    """One tensor of 2^32 + 5000 bfloat16 gradients, which alone are read."""
    n = (1 << 32) + 5000
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1 << 31, (1 << 32) + 17, n - 1], device="cuda")
    g[at] = 3.0
    rec = [zg.adamw_tensor(grad=g, master=g, m=g, v=g, numel=n)]
    plan = zg.zero_adamw_plan(rec, zg.ZERO_BF16, 32)
    table = torch.empty(plan.table_bytes, dtype=torch.uint8, device="cuda")
    zg.zero_adamw_table_init(plan, rec, table, torch.cuda.current_stream())
    N = Norm(plan)
    zg.zero_adamw_norm(plan, table, 1.0, 1.5, N.norm, N.flag, N.ws)
    assert float(N.norm[0]) == 6.0
    zg.zero_adamw_clip(plan, table, N.norm, torch.cuda.current_stream())
    assert bool((g[at].float() == (3.0 * N.norm[1]).bfloat16().float()).all())
    zg.zero_adamw_norm(plan, table, 1.0, 0.0, N.norm, N.flag, N.ws)
    assert abs(float(N.norm[0]) - 1.5) < 1.5 * 2.0 ** -8
