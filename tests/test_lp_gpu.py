"""Log probabilities, entropies, alternatives and gradients on the GPU against
their definitions in 64 bits.

Tolerances: those of cross entropy's tests for a logit, a row's lse and the
gradients' products; for the entropy, log S - T / S with S = sum e, T = sum e d: a
logit's error times sum p |log p + H|, and of each sum its chain of
additions, exp2's 2^-21 and its argument's rounding, |d| 2^-23, on
the magnitudes 1 + sum p |d| + sum p d^2 that those act on."""
import os

import pytest
import torch

import zero_sharded_mixed_bucket_gb300 as zg
from tests.launches import launches
from tests.test_ce_gpu import DT, GUARD, _e, _guards_kept, _rows

pytestmark = pytest.mark.gpu


class Job:
    def __init__(self, n, v, d, dtype, pad=0, piece=0, top=0, scale=1.0, seed=0, ignore=0.2, spread=1.5, grid=False):
        self.n, self.v, self.d, self.top, self.scale = n, v, d, top, scale
        self.code, self.dt, self.u = DT[dtype]
        g = torch.Generator(device="cuda").manual_seed(seed + n + 7 * v + 13 * d)
        stride = (d + 7) // 8 * 8 + pad
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        (self.fx0, self.x), (self.fw0, self.w) = _rows(n, d, stride, self.dt), _rows(v, d, stride, self.dt)
        x, w = r(n, d), r(v, d) * (spread / d ** 0.5)
        if grid:                                      # multiples of powers of two: every sum is exact
            step = 2.0 ** -10
            x, w = (x * 16).round().clamp(-127, 127) / 16, (w / step).round().clamp(-127, 127) * step
        self.x.copy_(x)
        self.w.copy_(w)
        self.t = torch.randint(0, v, (n,), device="cuda", generator=g)
        drop = torch.rand(n, device="cuda", generator=g)
        self.t[drop < ignore] = -100
        self.t[drop < ignore / 4] = v                 # past the end counts as no target too
        if n > 1:
            self.t[0], self.t[1] = v - 1, 0
        self.plan = zg.zero_lp_plan(n, v, d, self.code, stride, stride, piece, top)
        self.ws = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda").fill_(0xFF)
        self.logp, self.lse, self.ent = (torch.full((n,), GUARD, device="cuda") for _ in range(3))
        self.tl = torch.full((n, top), GUARD, device="cuda") if top else None
        self.ti = torch.full((n, top), -77, dtype=torch.int64, device="cuda") if top else None
        (self.fx, self.dx), (self.fw, self.dw) = _rows(n, d, stride, self.dt), _rows(v, d, stride, self.dt)
        self.g = g

    def forward(self, stream=None):
        zg.zero_lp_forward(self.plan, self.x, self.w, self.t, self.scale, self.logp, self.lse, self.ent, self.tl, self.ti, self.ws,
                           stream or torch.cuda.current_stream())

    def backward(self, dlogp, dent, scale=1.0, stream=None):
        zg.zero_lp_backward(self.plan, self.x, self.w, self.t, self.scale, self.lse, self.ent, dlogp, dent, scale, self.dx, self.dw,
                            self.ws, stream or torch.cuda.current_stream())

    def define(self):
        x, w = self.x.double(), self.w.double()
        self.s32 = float(torch.tensor(self.scale, dtype=torch.float32))
        self.z = (x @ w.t()) * self.s32
        self.counted = (self.t >= 0) & (self.t < self.v)
        self.at = torch.where(self.counted, self.t, 0)[:, None]
        self.want_lse = torch.logsumexp(self.z, 1)
        self.lp = self.z - self.want_lse[:, None]
        self.p = torch.exp(self.lp)
        self.want_logp = torch.where(self.counted, self.lp.gather(1, self.at)[:, 0], 0.0)
        self.want_ent = torch.special.entr(self.p).sum(1)
        # error of one scaled logit, of a row's lse, of its entropy
        self.ez = _e(self.d) * (x.abs() @ w.abs().t()) * self.s32
        chain = 256 + self.v / 256 + 16
        self.elog = self.ez.amax(1) + 2.0 ** -21 + chain * 2.0 ** -24 + 6 * 2.0 ** -24 * (1 + self.z.abs().amax(1))
        dist = self.z - self.z.amax(1, keepdim=True)
        act = 1 + (self.p * dist.abs()).sum(1) + (self.p * dist * dist).sum(1)
        spread = (self.p * (self.lp + self.want_ent[:, None]).abs()).sum(1)
        self.eent = 1.1 * self.ez.amax(1) * spread + 4 * (2.0 ** -21 + chain * 2.0 ** -24) * act

    def check_forward(self):
        self.define()
        assert ((self.lse.double() - self.want_lse).abs() <= self.elog).all()
        tol = 2 * self.elog + 2.0 ** -23 * self.want_logp.abs()
        assert ((self.logp.double() - self.want_logp).abs() <= torch.where(self.counted, tol, 0.0)).all()
        off = (self.ent.double() - self.want_ent).abs()
        assert (off <= self.eent).all(), "worst %g of the tolerance" % float((off / self.eent).max())
        if self.top:
            k = min(self.top, self.v)
            assert (self.ti[:, k:] == -1).all() and (self.tl[:, k:] == -float("inf")).all()
            ti, tl = self.ti[:, :k], self.tl[:, :k]
            assert ((ti >= 0) & (ti < self.v)).all()
            assert (ti.sort(1).values.diff(dim=1) > 0).all()             # distinct
            z, slack = self.z.gather(1, ti), 2 * self.ez.amax(1, keepdim=True)
            assert (z.diff(dim=1) <= slack).all()
            rest = self.z.scatter(1, ti, -float("inf")).amax(1, keepdim=True)
            assert (z[:, -1:] >= rest - slack).all()
            assert ((tl.double() - (z - self.want_lse[:, None])).abs() <= 2 * self.elog[:, None] + 2.0 ** -23 * (z - self.want_lse[:, None]).abs()).all()
            same = ti == self.at                                          # the given token among them: the same log probability
            assert (tl[same & self.counted[:, None]] == self.logp[:, None].expand(-1, k)[same & self.counted[:, None]]).all()

    def check_backward(self, a, b):
        """a, b: row factors (float64) of G: scale and the gradients' scale included."""
        x, w = self.x.double(), self.w.double()
        a = torch.where(self.counted, a, 0.0)[:, None]
        b = b[:, None]
        inner = self.lp + self.want_ent[:, None]
        onehot = torch.zeros_like(self.z).scatter_(1, self.at, 1.0) * self.counted[:, None]
        G = a * (onehot - self.p) - b * torch.where(self.p > 0, self.p * inner, 0.0)
        most = float((a.abs() + 4 * b.abs()).max()) if self.n else 0.0
        ep = self.ez + self.elog[:, None] + 2.0 ** -20 + 4 * 2.0 ** -24 * self.z.abs()      # relative, of p; absolute, of log p
        eG = self.p * ep * (a.abs() + b.abs() * (inner.abs() + 1)) + b.abs() * self.p * (self.eent[:, None] + 8 * 2.0 ** -24 * (inner.abs() + self.want_ent[:, None])) \
            + G.abs() * (1.01 * self.u + 8 * 2.0 ** -24) + most * 2.0 ** -25 * (2.0 ** -14 if self.u == 2.0 ** -11 else 0)
        for got, full, f, ef, o in ((self.dx, self.fx, G, eG, w), (self.dw, self.fw, G.t(), eG.t(), x)):
            want = f @ o
            tol = ef @ o.abs() * 1.01 + 1.5 * _e(f.shape[1]) * (f.abs() @ o.abs()) + 1.01 * self.u * want.abs() \
                + (2.0 ** -25 if self.u == 2.0 ** -11 else 0) + 1e-38
            off = (got.double() - want).abs()
            assert (off <= tol).all(), "worst %g of the tolerance" % float((off / tol).max())
            assert _guards_kept(full, got)


SHAPES = [  # tokens, vocab, hidden, pad, piece, top, scale
    (1, 1, 8, 0, 0, 1, 1.0), (1, 2, 8, 8, 0, 5, 1.0), (1, 257, 64, 0, 0, 8, 0.7), (1, 1000, 768, 0, 256, 32, 1.0), (1, 50257, 256, 0, 0, 8, 1.0),
    (2, 3, 1, 0, 0, 4, 1.0), (2, 5000, 72, 0, 0, 3, 1.3), (3, 1000, 72, 0, 512, 20, 1.0), (3, 9, 33, 8, 0, 0, 2.0),
    (1, 700, 40_000, 0, 0, 9, 1.0), (3, 300, 11_000, 0, 0, 2, 1.0), (4, 2, 8, 0, 0, 2, 1.0), (5, 300, 33, 8, 256, 7, 1.25), (64, 256, 64, 0, 0, 1, 1.0), (128, 256, 128, 0, 0, 32, 1.0),
    (129, 513, 136, 8, 256, 8, 0.5), (127, 255, 200, 0, 0, 0, 1.0), (257, 2049, 264, 0, 768, 20, 1.0), (300, 4099, 100, 0, 1024, 5, 1.0),
    (20, 50257, 64, 0, 0, 32, 1.0), (1025, 1031, 520, 0, 0, 4, 1.0), (600, 3001, 1600, 0, 1280, 0, 1.25), (600, 50257, 64, 0, 0, 8, 1.0),
    (700, 50257, 40, 0, 0, 32, 0.8), (1500, 50257, 72, 8, 0, 20, 1.0), (3000, 23_000, 33, 0, 0, 8, 1.0), (2000, 16500, 72, 0, 0, 20, 1.0), (5000, 2, 64, 0, 0, 2, 1.0),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,v,d,pad,piece,top,scale", SHAPES)
def test_forward_and_gradients(n, v, d, pad, piece, top, scale, dtype):
    j = Job(n, v, d, dtype, pad, piece, top, scale)
    j.forward()
    j.check_forward()
    dl = torch.randn(n, device="cuda", generator=j.g) / n
    de = torch.randn(n, device="cuda", generator=j.g) / n
    j.backward(dl, de, 64.0)
    j.check_backward(dl.double() * 64 * j.s32, de.double() * 64 * j.s32)
    j.backward(dl, None, 64.0)
    j.check_backward(dl.double() * 64 * j.s32, torch.zeros_like(dl.double()))
    j.backward(None, de, 64.0)
    j.check_backward(torch.zeros_like(dl.double()), de.double() * 64 * j.s32)
    zg.zero_lp_status(j.plan, j.ws)
    assert _guards_kept(j.fx0, j.x) and _guards_kept(j.fw0, j.w)


def _order(j):
    z = (j.x.double() @ j.w.double().t())
    k = min(j.top, j.v)
    return torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,v,top", [(1, 4000, 32), (2, 700, 8), (3, 50257, 20), (4, 1000, 8), (40, 50257, 8), (600, 50257, 20), (1023, 30000, 1), (600, 50257, 32),
                                     (1400, 50257, 8), (1400, 50001, 32)])
def test_order_of_alternatives(n, v, top, dtype):
    """Logits on a grid, exact in every order of summing: the alternatives in the order of a stable sort, ties included."""
    j = Job(n, v, 48, dtype, top=top, grid=True, scale=1.25)
    j.w[v // 2:v // 2 + min(300, v // 2)] = j.w[:min(300, v // 2)]            # equal logits far apart
    j.w[5:7] = j.w[3:5]                                                        # and near
    j.forward()
    assert torch.equal(j.ti, _order(j))


@pytest.mark.parametrize("n", [1, 3, 20, 600, 1400])
@pytest.mark.parametrize("what", ["rising", "falling", "equal", "rising in strips"])
def test_alternatives_of_sorted_logits(n, what):
    """Vocabularies whose logits rise (every entry is the best yet), fall, or are all the same."""
    v, top = 50_000, 20
    j = Job(n, v, 16, "bf16", top=top)
    i = torch.arange(v, device="cuda")
    i = {"rising": i, "falling": v - 1 - i, "equal": 0 * i, "rising in strips": i % 128}[what]
    j.x.zero_()
    j.w.zero_()
    j.x[:, 0] = 1
    j.x[:, 1] = 1
    j.w[:, 0] = (i // 256).to(j.dt)
    j.w[:, 1] = (i % 256).to(j.dt) / 256
    j.forward()
    assert torch.equal(j.ti, _order(j))
    j.define()
    assert ((j.lse.double() - j.want_lse).abs() <= j.elog).all() and ((j.ent.double() - j.want_ent).abs() <= j.eent).all()


@pytest.mark.parametrize("n,v,d,top,sample", [
    (800, 50257, 16, 8, False), (1400, 50257, 16, 8, True), (1300, 50257, 16, 16, False), (1400, 50257, 16, 16, True),
    (1600, 50257, 16, 20, False), (2048, 50257, 16, 20, True), (2048, 50257, 16, 32, False), (2670, 50257, 16, 32, False),
    (2700, 50257, 16, 32, True), (2048, 50257, 1024, 1, False), (4000, 50257, 1024, 8, False), (4100, 50257, 1024, 8, True),
    (20_000, 10_240, 16, 8, False), (20_000, 10_241, 16, 8, True), (2, 50257, 16, 8, None)])
def test_which_logits_are_kept(n, v, d, top, sample):
    """All, up to a number of them that goes by the alternatives and the hidden size, or a sample's: two kernels more."""
    j = Job(n, v, d, "bf16", top=top)
    assert launches(j.forward) == (2 if sample is None else 6 if sample else 4)
    assert n * v <= 1 << 29                           # one pass over the rows


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,v,top", [(1700, 50257, 20), (2800, 50001, 32)])
def test_order_of_alternatives_by_sample(n, v, top, dtype):
    """The order of a stable sort, ties included, where only a sample's logits are kept."""
    j = Job(n, v, 48, dtype, top=top, grid=True, scale=1.25)
    j.w[v // 2:v // 2 + 300] = j.w[:300]
    j.w[5:7] = j.w[3:5]
    assert launches(j.forward) == 6
    j.forward()
    assert torch.equal(j.ti, _order(j))


@pytest.mark.parametrize("what", ["rising", "falling", "equal", "rising in strips"])
def test_alternatives_of_sorted_logits_by_sample(what):
    test_alternatives_of_sorted_logits(1800, what)
    assert launches(Job(1800, 50_000, 16, "bf16", top=20).forward) == 6


def test_gradients_against_differences():
    j = Job(40, 300, 48, "bf16", ignore=0.1, scale=1.25)
    dl, de = torch.randn(40, device="cuda", generator=j.g), torch.randn(40, device="cuda", generator=j.g)
    j.forward()
    j.backward(dl, de)
    counted, at = (j.t >= 0) & (j.t < j.v), torch.where((j.t >= 0) & (j.t < j.v), j.t, 0)[:, None]

    def f(x, w):
        lp = torch.log_softmax(1.25 * (x @ w.t()), 1)
        return (lp.gather(1, at)[:, 0] * dl.double())[counted].sum() - ((lp.exp() * lp).sum(1) * de.double()).sum()

    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = j.x.double(), j.w.double()
    for grad, k in ((j.dx, 0), (j.dw, 1)):
        for _ in range(8):
            d = torch.randn((x, w)[k].shape, device="cuda", generator=g, dtype=torch.float64)
            hi = f(x + 1e-4 * d, w) if k == 0 else f(x, w + 1e-4 * d)
            lo = f(x - 1e-4 * d, w) if k == 0 else f(x, w - 1e-4 * d)
            got = (grad.double() * d).sum()
            assert abs(got - (hi - lo) / 2e-4) <= 2.0 ** -6 * grad.double().norm() * 6


def test_rows_in_pieces():
    """More rows than one forward pass takes at a time: each row as if alone."""
    j = Job(11_000, 50257, 24, "fp16", top=32, grid=True)
    assert j.plan.rows < 11_000
    j.forward()
    assert torch.equal(j.ti[-700:], _order(j)[-700:]) and torch.equal(j.ti[:50], _order(j)[:50])
    few = Job(11_000, 50257, 24, "fp16", grid=True)
    few.forward()
    for a, b in ((j.lse, few.lse), (j.logp, few.logp), (j.ent, few.ent)):
        assert torch.equal(a, b)
    want = torch.log_softmax(j.x.double() @ j.w.double().t(), 1)
    assert (j.tl.double() - want.gather(1, j.ti)).abs().max() < 1e-5


def test_confident_rows():
    """A likely token's log probability and entropy keep their digits: neither is the difference of large numbers."""
    for n in (1, 3, 70):
        j = Job(n, 1000, 64, "bf16", top=2)
        j.x.zero_()
        j.w.zero_()
        j.x[:, 0] = 8
        j.w[7, 0] = 3                                 # a logit of 24 against 999 of 0
        j.t.fill_(7)
        j.forward()
        e = 999 * torch.exp(torch.tensor(-24.0, dtype=torch.float64))
        logp = -torch.log1p(e)
        ent = torch.log1p(e) + e * 24 / (1 + e)
        # S = 1 + e in binary32: e to half a unit of 1, T = 24 e to its own
        assert abs(float(j.logp[0]) - float(logp)) <= 2.0 ** -24 * 1.01
        assert abs(float(j.ent[0]) - float(ent)) <= 2.0 ** -24 * 1.01 + float(ent) * 2.0 ** -18
        assert int(j.ti[0, 0]) == 7 and int(j.ti[0, 1]) == 0


@pytest.mark.parametrize("n", [1, 3, 20, 600, 1400])
def test_infinite_and_nan_logits(n):
    """-infinity is no alternative and adds nothing; a NaN or +infinity spoils its own row's log probability and entropy."""
    v = 50257
    j = Job(n, v, 16, "bf16", top=5, grid=True, ignore=0.0)
    j.x[:, 0] = 0
    j.x[0, 0] = 1
    j.w[100:200, 0] = -float("inf")                   # row 0's logits there are -infinity, the others' 0 * inf: NaN
    j.forward()
    z = j.x[0].double() @ j.w.double().t()
    assert (z[100:200] == -float("inf")).all()
    lp = torch.log_softmax(z, 0)
    p = lp.exp()
    assert abs(float(j.lse[0]) - float(torch.logsumexp(z, 0))) < 1e-5
    assert abs(float(j.ent[0]) - float(-(p * lp)[p > 0].sum())) < 1e-4
    assert torch.equal(j.ti[0], torch.sort(z, descending=True, stable=True).indices[:5])
    if n > 1:
        assert j.logp[1:].isnan().all() and j.ent[1:].isnan().all() and j.lse[1:].isnan().all() and j.tl[1:].isnan().all()
        rest = (j.x[1:, 1:].double() @ j.w[:, 1:].double().t())
        rest[:, 100:200] = -float("inf")
        assert torch.equal(j.ti[1:], torch.sort(rest, dim=1, descending=True, stable=True).indices[:, :5])
    j.w[100:200, 0] = float("inf")
    j.forward()
    assert j.logp[0].isnan() and j.ent[0].isnan()
    j.w[:, 0] = -float("inf")                         # nothing is left of row 0
    j.forward()
    assert (j.ti[0] == -1).all() and j.logp[0].isnan()


@pytest.mark.parametrize("n", [1, 3, 70])
def test_logits_of_the_lowest_value(n):
    """Entries masked by bfloat16's lowest value: probability 0, nothing in the entropy, no gradient."""
    j = Job(n, 1000, 64, "bf16", top=4, ignore=0.0)
    j.x[:, 0] = 1
    j.w[:, 0] = 0
    j.w[300:900] = 0
    j.w[300:900, 0] = torch.finfo(torch.bfloat16).min
    j.t.fill_(5)
    j.forward()
    keep = torch.cat([torch.arange(300), torch.arange(900, 1000)]).cuda()
    lp = torch.log_softmax(j.x.double() @ j.w[keep].double().t(), 1)
    assert (j.logp.double() - lp[:, 5]).abs().max() < 1e-5 and (j.ent.double() + (lp.exp() * lp).sum(1)).abs().max() < 1e-4
    assert torch.isin(j.ti, keep).all()
    one = torch.ones(n, device="cuda")
    j.backward(one, one)
    assert j.dw.isfinite().all() and (j.dw[300:900] == 0).all()
    j.t.fill_(400)                                    # a masked entry given: its log probability is what the logits say
    j.forward()
    assert (j.logp < -3e38).all()


@pytest.mark.parametrize("dtype", list(DT))
def test_gradients_lose_no_more_than_G_rounded_once(dtype):
    """G scaled and rounded to the operands' type, all else in 64 bits: the kernels are next to that.

    What is left is binary32's: a G_iv is relatively off by some 2^-18 (a logit's sum, exp2), so about one in 2^-18 / (2 u) of them, and
    of the results, falls on the other side of a border and is a whole step 2 u off: sqrt(2^-18 * 2 u) of the norm, 1.7e-4 in bfloat16
    and 6.1e-5 in binary16, under a quarter of what the two roundings (some u / 2 each) take."""
    n, v, d = 300, 5000, 256
    j = Job(n, v, d, dtype, scale=1.25)
    dl, de = torch.randn(n, device="cuda", generator=j.g) / n, torch.full((n,), 0.01 / n, device="cuda")
    j.forward()
    j.backward(dl, de, 1024.0)
    j.define()
    a = torch.where(j.counted, dl.double() * 1024 * j.s32, 0.0)[:, None]
    b = de.double()[:, None] * 1024 * j.s32
    onehot = torch.zeros_like(j.z).scatter_(1, j.at, 1.0) * j.counted[:, None]
    G = a * (onehot - j.p) - b * j.p * (j.lp + j.want_ent[:, None])
    unit = float((a.abs() + 4 * b.abs()).max()) / (2.0 ** 14 if dtype == "fp16" else 1.0)
    R = (G / unit).float().to(j.dt).double() * unit
    for got, exact, near in ((j.dx, G @ j.w.double(), R @ j.w.double()), (j.dw, G.t() @ j.x.double(), R.t() @ j.x.double())):
        near = near.to(j.dt).double()
        lost = (near - exact).norm()
        assert (got.double() - near).norm() <= lost / 4
        assert lost <= 1.5 * j.u * exact.norm()       # two roundings, half a step each at most: u each


def test_tokens_without_a_target_and_factors_of_zero():
    j = Job(300, 700, 64, "bf16", ignore=1.0)
    j.t.fill_(-100)
    j.forward()
    assert (j.logp == 0).all()
    j.check_forward()
    j.backward(torch.full((300,), float("nan"), device="cuda"), None)          # no target: no factor
    assert (j.dx == 0).all() and (j.dw == 0).all()
    j.backward(None, None)
    assert (j.dx == 0).all() and (j.dw == 0).all()


def test_one_nonfinite_factor():
    j = Job(200, 500, 64, "bf16", ignore=0.0)
    j.forward()
    j.define()
    for bad in (float("nan"), float("inf")):
        for which in (0, 1):
            f = [torch.ones(200, device="cuda"), torch.ones(200, device="cuda")]
            f[which][17] = bad
            j.backward(*f)
            keep = torch.arange(200, device="cuda") != 17
            assert j.dx[17].isnan().all() and j.dx[keep].isfinite().all() and j.dw.isnan().any()


def test_no_tokens():
    j = Job(0, 300, 24, "bf16", top=3)
    j.forward()
    j.backward(None, None)
    assert (j.dw == 0).all() and _guards_kept(j.fw, j.dw)
    zg.zero_lp_status(j.plan, j.ws)


def test_same_bits_each_time_and_outputs_left_out():
    j = Job(1400, 50257, 72, "bf16", top=8)
    dl = torch.randn(1400, device="cuda")
    out = []
    for _ in range(3):
        j.ws.fill_(0xFF)
        j.forward()
        j.backward(dl, dl)
        out.append([t.clone() for t in (j.logp, j.lse, j.ent, j.tl, j.ti, j.dx, j.dw)])
    assert all(torch.equal(a, b) for o in out[1:] for a, b in zip(out[0], o))
    j.dx.fill_(1)
    zg.zero_lp_backward(j.plan, j.x, j.w, j.t, 1.0, j.lse, j.ent, dl, dl, 1.0, None, j.dw, j.ws, torch.cuda.current_stream())
    assert (j.dx == 1).all() and torch.equal(j.dw, out[0][6])
    j.dw.fill_(1)
    zg.zero_lp_backward(j.plan, j.x, j.w, j.t, 1.0, j.lse, j.ent, dl, dl, 1.0, j.dx, None, j.ws, torch.cuda.current_stream())
    assert (j.dw == 1).all() and torch.equal(j.dx, out[0][5])
    zg.zero_lp_forward(j.plan, j.x, j.w, j.t, 1.0, j.logp, j.lse, None, j.tl, j.ti, j.ws, torch.cuda.current_stream())
    assert torch.equal(j.logp, out[0][0])


@pytest.mark.parametrize("n", [1, 130, 1400])
def test_streams_and_graphs(n):
    j, k = Job(n, 50257, 64, "bf16", top=8), Job(n, 50257, 64, "bf16", top=8)
    dl = torch.randn(n, device="cuda")
    j.forward()
    j.backward(dl, dl)
    torch.cuda.synchronize()
    st, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            k.forward()
            k.backward(dl, dl)
    other = torch.cuda.Stream()
    want = [t.clone() for t in (j.logp, j.ent, j.tl, j.ti, j.dx, j.dw)]
    for _ in range(3):
        k.ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        j.forward(other)                              # at the same time, with a workspace of its own
        j.backward(dl, dl, stream=other)
        torch.cuda.synchronize()
        for q in (j, k):
            assert all(torch.equal(a, b) for a, b in zip(want, (q.logp, q.ent, q.tl, q.ti, q.dx, q.dw)))


@pytest.mark.parametrize("top,n,v", [(0, 130, 600), (8, 130, 600), (8, 1400, 50257)])
def test_bounded_wait_is_reported(top, n, v):
    """The first block's first copy is announced but not made (test hook)."""
    j = Job(n, v, 128, "bf16", top=top)
    os.environ["ZERO_TEST_WITHHOLD_TILE"] = "1"
    try:
        j.forward()
    finally:
        del os.environ["ZERO_TEST_WITHHOLD_TILE"]
    with pytest.raises(zg.ZeroError) as e:
        zg.zero_lp_status(j.plan, j.ws)
    assert e.value.status == zg.ZERO_ETIMEOUT and j.logp[j.t >= 0][0].isnan() and j.lse.isnan().all() and j.ent.isnan().all()
    if top:
        assert j.tl.isnan().all() and (j.ti == -1).all()
    j.forward()
    zg.zero_lp_status(j.plan, j.ws)
    j.check_forward()
    os.environ["ZERO_TEST_WITHHOLD_TILE"] = "1"
    try:
        j.backward(torch.ones(n, device="cuda"), None)
    finally:
        del os.environ["ZERO_TEST_WITHHOLD_TILE"]
    with pytest.raises(zg.ZeroError):
        zg.zero_lp_status(j.plan, j.ws)
    assert j.dx.isnan().all() and j.dw.isnan().all()


def test_status_of_a_backward_pass_without_outputs():
    """Nothing is computed, so nothing has run out: neither a workspace of any contents nor an earlier call's error is reported."""
    j = Job(130, 600, 64, "bf16")
    one = torch.ones(130, device="cuda")
    none = lambda: zg.zero_lp_backward(j.plan, j.x, j.w, j.t, 1.0, j.lse, j.ent, one, one, 1.0, None, None, j.ws,  # noqa: E731
                                       torch.cuda.current_stream())
    none()                                            # the workspace is 0xFF everywhere
    zg.zero_lp_status(j.plan, j.ws)
    os.environ["ZERO_TEST_WITHHOLD_TILE"] = "1"
    try:
        j.forward()
    finally:
        del os.environ["ZERO_TEST_WITHHOLD_TILE"]
    with pytest.raises(zg.ZeroError):
        zg.zero_lp_status(j.plan, j.ws)
    none()
    zg.zero_lp_status(j.plan, j.ws)
    j.forward()
    j.check_forward()


@pytest.mark.parametrize("n", [2, 70])
def test_offsets_past_32_bits(n):
    """A weight whose rows lie past 2^32 values."""
    v, d, stride = 300, 64, 1 << 24
    full = torch.empty(v * stride, dtype=torch.bfloat16, device="cuda")
    w = full.view(v, stride)[:, :d]
    j = Job(n, v, d, "bf16", top=4)
    w.copy_(j.w)
    p = zg.zero_lp_plan(n, v, d, zg.ZERO_BF16, j.plan.x_stride, stride, 0, 4)
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    j.forward()
    out = [torch.empty_like(t) for t in (j.logp, j.lse, j.ent, j.tl, j.ti)]
    zg.zero_lp_forward(p, j.x, w, j.t, 1.0, *out, ws, torch.cuda.current_stream())
    assert all(torch.equal(a, b) for a, b in zip(out, (j.logp, j.lse, j.ent, j.tl, j.ti)))
    dl = torch.ones(n, device="cuda")
    j.backward(dl, dl)
    dx = torch.empty_strided(j.dx.shape, j.dx.stride(), dtype=j.dt, device="cuda")
    zg.zero_lp_backward(p, j.x, w, j.t, 1.0, j.lse, j.ent, dl, dl, 1.0, dx, None, ws, torch.cuda.current_stream())
    assert torch.equal(dx, j.dx)


@pytest.mark.parametrize("n,d", [(70, 64), (70, 61), (1100, 64)])
def test_gradient_of_a_weight_past_32_bits(n, d):
    """dw with rows past 2^32 values, by tiled copies, one by one (rows that do not end on 16 bytes) and summed over parts of the
    tokens: the bits of the same rows side by side, and nothing beside them."""
    v, stride = 300, 1 << 24
    j = Job(n, v, d, "bf16")
    w, dw = (torch.empty(v * stride, dtype=torch.bfloat16, device="cuda").view(v, stride) for _ in range(2))
    w[:, :d].copy_(j.w)
    dw[:, :d + 64].fill_(GUARD)
    p = zg.zero_lp_plan(n, v, d, zg.ZERO_BF16, j.plan.x_stride, stride)
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    dl = torch.randn(n, device="cuda", generator=j.g)
    j.forward()
    j.backward(dl, dl)
    dx = torch.empty_strided(j.dx.shape, j.dx.stride(), dtype=j.dt, device="cuda")
    zg.zero_lp_backward(p, j.x, w, j.t, 1.0, j.lse, j.ent, dl, dl, 1.0, dx, dw, ws, torch.cuda.current_stream())
    assert torch.equal(dx, j.dx) and torch.equal(dw[:, :d], j.dw) and (dw[:, d:d + 64] == GUARD).all()
    j.define()
    j.check_backward(dl.double(), dl.double())
    # no tokens, and a pass whose wait ran out
    zg.zero_lp_backward(zg.zero_lp_plan(0, v, d, zg.ZERO_BF16, j.plan.x_stride, stride), None, None, None, 1.0, None, None, None, None, 1.0,
                        None, dw, ws, torch.cuda.current_stream())
    assert (dw[:, :d] == 0).all() and (dw[:, d:d + 64] == GUARD).all()
    os.environ["ZERO_TEST_WITHHOLD_TILE"] = "1"
    try:
        zg.zero_lp_backward(p, j.x, w, j.t, 1.0, j.lse, j.ent, dl, dl, 1.0, None, dw, ws, torch.cuda.current_stream())
    finally:
        del os.environ["ZERO_TEST_WITHHOLD_TILE"]
    with pytest.raises(zg.ZeroError):
        zg.zero_lp_status(p, ws)
    assert dw[:, :d].isnan().all() and (dw[:, d:d + 64] == GUARD).all()


@pytest.mark.parametrize("n", [1, 3, 20, 600, 1400])
def test_infinite_logits_are_the_first_alternatives(n):
    """+infinity is a number: the lowest such indices come first, with NaN as their log probability; other rows' NaN are none."""
    j = Job(n, 50257, 16, "bf16", top=5, grid=True, ignore=0.0)
    j.x[:, 0] = 0
    j.x[0, 0] = 1
    j.w[100:103, 0] = float("inf")
    j.w[40_000:40_200, 0] = float("inf")
    j.forward()
    assert j.ti[0].tolist() == [100, 101, 102, 40_000, 40_001] and j.tl[0].isnan().all()
    assert j.logp[0].isnan() and j.lse[0].isnan() and j.ent[0].isnan()
    if n > 1:                                         # 0 times infinity
        rest = j.x[1:, 1:].double() @ j.w[:, 1:].double().t()
        rest[:, 100:103] = rest[:, 40_000:40_200] = -float("inf")
        assert torch.equal(j.ti[1:], torch.sort(rest, dim=1, descending=True, stable=True).indices[:, :5])


@pytest.mark.parametrize("top,n,v", [(0, 300, 600), (3, 1400, 50257)])
def test_results_after_a_wait_that_ran_out(top, n, v):
    """NaN, but for what says nothing of the logits: logp of tokens without a target is 0, the alternatives' indices are -1."""
    j = Job(n, v, 128, "bf16", top=top, ignore=0.4)
    os.environ["ZERO_TEST_WITHHOLD_TILE"] = "1"
    try:
        j.forward()
    finally:
        del os.environ["ZERO_TEST_WITHHOLD_TILE"]
    counted = (j.t >= 0) & (j.t < v)
    assert 0 < int(counted.sum()) < n
    assert j.logp[counted].isnan().all() and (j.logp[~counted] == 0).all()
    assert j.lse.isnan().all() and j.ent.isnan().all() and (not top or (j.tl.isnan().all() and (j.ti == -1).all()))
    with pytest.raises(zg.ZeroError):
        zg.zero_lp_status(j.plan, j.ws)
