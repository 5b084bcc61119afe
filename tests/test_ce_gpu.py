"""Cross entropy over a vocabulary on the GPU against its definition in 64 bits.

Tolerances, derived.  A product of K 16-bit values is exact in binary32; the
tensor cores add 16 of them at a time to the accumulator, each step off by at
most 2^-22 of the magnitudes so far, so a sum is off by at most
(K/16 + 2) 2^-22 sum |a b| =: e(K) sum |a b|.  exp2 is good to 2^-21 here, a
token's sum over the vocabulary has at most 256 + V/256 additions in a chain,
and the exponents' bases are rounded at 2^-24 of the largest logit.  G is
rounded once to the operand type (u: 2^-11 binary16, 2^-8 bfloat16), the
outputs once more.  Each bound below is the sum of those, carried through the
products elementwise."""
import os

import pytest
import torch

import zero_sharded_mixed_bucket_gb300 as zg

pytestmark = pytest.mark.gpu

DT = {"fp16": (zg.ZERO_FP16, torch.float16, 2.0 ** -11), "bf16": (zg.ZERO_BF16, torch.bfloat16, 2.0 ** -8)}
GUARD = -77.0


def _e(k):
    return (k / 16 + 2) * 2.0 ** -22


def _rows(rows, width, stride, dt):
    full = torch.full((max(rows, 1) * stride + 128,), GUARD, dtype=dt, device="cuda")
    return full, full[64:64 + max(rows, 1) * stride].view(-1, stride)[:rows, :width]


def _guards_kept(full, view):
    keep = torch.ones_like(full, dtype=torch.bool)
    keep.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((full[keep] == GUARD).all())


class Job:
    def __init__(self, n, v, d, dtype, pad=0, piece=0, seed=0, ignore=0.2, spread=1.5):
        self.n, self.v, self.d = n, v, d
        self.code, self.dt, self.u = DT[dtype]
        g = torch.Generator(device="cuda").manual_seed(seed + n + 7 * v + 13 * d)
        stride = (d + 7) // 8 * 8 + pad
        r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
        _, self.x = _rows(n, d, stride, self.dt)
        _, self.w = _rows(v, d, stride, self.dt)
        self.x.copy_(r(n, d))
        self.w.copy_(r(v, d) * (spread / d ** 0.5))
        self.t = torch.randint(0, v, (n,), device="cuda", generator=g)
        drop = torch.rand(n, device="cuda", generator=g)
        self.t[drop < ignore] = -100
        self.t[drop < ignore / 4] = v            # past the end counts as no target too
        if n > 1:
            self.t[0], self.t[1] = v - 1, 0
        self.plan = zg.zero_ce_plan(n, v, d, self.code, stride, stride, piece)
        self.ws = torch.empty(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda").fill_(0xFF)
        self.loss, self.lse = (torch.full((n,), GUARD, device="cuda") for _ in range(2))
        self.total = torch.full((2,), GUARD, device="cuda")
        (self.fx, self.dx), (self.fw, self.dw) = _rows(n, d, stride, self.dt), _rows(v, d, stride, self.dt)

    def forward(self):
        zg.zero_ce_forward(self.plan, self.x, self.w, self.t, self.loss, self.lse, self.total, self.ws,
                           torch.cuda.current_stream())

    def backward(self, scale=1.0, dloss=None, lse=None):
        zg.zero_ce_backward(self.plan, self.x, self.w, self.t, self.lse if lse is None else lse, dloss, scale, self.dx,
                            self.dw, self.ws, torch.cuda.current_stream())

    def define(self):
        x, w = self.x.double(), self.w.double()
        self.z = x @ w.t()
        self.counted = (self.t >= 0) & (self.t < self.v)
        self.want_lse = torch.logsumexp(self.z, 1)
        at = torch.where(self.counted, self.t, 0)[:, None]
        self.onehot = torch.zeros_like(self.z).scatter_(1, at, 1.0) * self.counted[:, None]
        self.want_loss = torch.where(self.counted, self.want_lse - self.z.gather(1, at)[:, 0], 0.0)
        # error of one logit, of a row's lse
        self.ez = _e(self.d) * (x.abs() @ w.abs().t())
        chain = 256 + self.v / 256 + 16
        self.elog = self.ez.amax(1) + 2.0 ** -21 + chain * 2.0 ** -24 + 6 * 2.0 ** -24 * (1 + self.z.abs().amax(1))

    def check_forward(self):
        self.define()
        assert ((self.lse.double() - self.want_lse).abs() <= self.elog).all()
        tol = 2 * self.elog + 2.0 ** -23 * self.want_loss.abs()
        assert ((self.loss.double() - self.want_loss).abs() <= torch.where(self.counted, tol, 0.0)).all()
        c = int(self.counted.sum())
        assert self.total[1] == c
        want = float(self.want_loss.sum() / max(c, 1))
        assert abs(float(self.total[0]) - want) <= float(tol.max()) + (self.n / 1024 + 16) * 2.0 ** -24 * abs(want)

    def check_backward(self, s):
        """s: row factors (float64) of G."""
        x, w = self.x.double(), self.w.double()
        s = torch.where(self.counted, s, 0.0)[:, None]
        p = torch.exp(self.z - self.want_lse[:, None])
        G = s * (p - self.onehot)
        most = float(s.abs().max()) if self.n else 0.0
        eG = s.abs() * p * (self.ez + self.elog[:, None] + 2.0 ** -20 + 4 * 2.0 ** -24 * self.z.abs()) \
            + G.abs() * (1.01 * self.u + 8 * 2.0 ** -24) + most * 2.0 ** -25 * (2.0 ** -14 if self.u == 2.0 ** -11 else 0)
        for got, full, a, ea, b in ((self.dx, self.fx, G, eG, w), (self.dw, self.fw, G.t(), eG.t(), x)):
            want = a @ b
            K = a.shape[1]
            tol = ea @ b.abs() * 1.01 + 1.5 * _e(K) * (a.abs() @ b.abs()) + 1.01 * self.u * want.abs() \
                + (2.0 ** -25 if self.u == 2.0 ** -11 else 0) + 1e-38
            off = (got.double() - want).abs()
            assert (off <= tol).all(), "worst %g of the tolerance" % float((off / tol).max())
            assert _guards_kept(full, got)


SHAPES = [  # tokens, vocab, hidden, pad, piece
    (1, 1, 8, 0, 0), (1, 2, 8, 8, 0), (1, 257, 64, 0, 0), (1, 1000, 768, 0, 256), (2, 3, 1, 0, 0), (3, 1000, 72, 0, 512),
    (5, 300, 33, 8, 256), (64, 256, 64, 0, 0), (128, 256, 128, 0, 0), (129, 513, 136, 8, 256), (127, 255, 200, 0, 0),
    (256, 2048, 256, 0, 0), (257, 2049, 264, 0, 768), (300, 4099, 100, 0, 1024), (1000, 700, 1000, 0, 0),
    (20, 50257, 64, 0, 0), (1025, 1031, 520, 0, 0), (600, 3001, 1600, 0, 1280),
    (3000, 100, 264, 0, 0), (2500, 700, 33, 8, 256), (5000, 2, 64, 0, 0),   # dw's product in parts
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,v,d,pad,piece", SHAPES)
def test_loss_and_gradients(n, v, d, pad, piece, dtype):
    j = Job(n, v, d, dtype, pad, piece)
    j.forward()
    j.check_forward()
    j.backward(scale=64.0)
    c = max(1, int(j.counted.sum()))
    j.check_backward(torch.full((n,), 64.0 / c, device="cuda", dtype=torch.float64))
    zg.zero_ce_status(j.plan, j.ws)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("n,v,d,pad,piece", [(3, 1000, 72, 0, 512), (200, 3000, 160, 0, 1024), (130, 257, 64, 8, 0)])
def test_gradients_of_a_weighted_sum(n, v, d, pad, piece, dtype):
    """dloss given per token, of either sign, over six decades, zero in places."""
    j = Job(n, v, d, dtype, pad, piece)
    j.forward()
    j.define()
    g = torch.Generator(device="cuda").manual_seed(3)
    dl = torch.randn(n, device="cuda", generator=g) * 10 ** (6 * torch.rand(n, device="cuda", generator=g) - 3)
    dl[::5] = 0
    j.backward(scale=0.5, dloss=dl)
    # rows far below the largest factor lose precision to G's absolute spacing in binary16 only
    j.check_backward(dl.double() * 0.5)


def test_gradients_against_differences():
    """Central differences of the 64-bit loss along random directions: the
    loss is smooth on the scale of 1e-4 steps (error ~1e-8), so what is left is
    the gradients' own rounding: bfloat16, 2^-8 a value, independent."""
    j = Job(40, 300, 48, "bf16", ignore=0.1)
    j.forward()
    j.backward()
    t, counted = j.t, (j.t >= 0) & (j.t < j.v)

    def f(x, w):
        z = x @ w.t()
        l = torch.logsumexp(z, 1) - z.gather(1, torch.where(counted, t, 0)[:, None])[:, 0]
        return l[counted].sum() / counted.sum()

    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = j.x.double(), j.w.double()
    for grad, k in ((j.dx, 0), (j.dw, 1)):
        for _ in range(8):
            d = torch.randn((x, w)[k].shape, device="cuda", generator=g, dtype=torch.float64)
            hi = f(x + 1e-4 * d, w) if k == 0 else f(x, w + 1e-4 * d)
            lo = f(x - 1e-4 * d, w) if k == 0 else f(x, w - 1e-4 * d)
            got = (grad.double() * d).sum()
            assert abs(got - (hi - lo) / 2e-4) <= 2.0 ** -6 * grad.double().norm() * 6


def test_same_bits_each_time_and_outputs_left_out():
    j = Job(300, 5000, 192, "bf16", piece=2048)
    j.forward()
    j.backward(8.0)
    first = [t.clone() for t in (j.loss, j.lse, j.total, j.dx, j.dw)]
    j.ws.fill_(0x7F)
    j.forward()
    j.backward(8.0)
    for a, b in zip(first, (j.loss, j.lse, j.total, j.dx, j.dw)):
        assert torch.equal(a, b)
    dx, dw = torch.empty_like(j.dx), torch.empty_like(j.dw)
    st = torch.cuda.current_stream()
    dx, dw = (torch.zeros_like(t.as_strided(t.shape, t.stride())) for t in (j.dx, j.dw))
    zg.zero_ce_backward(j.plan, j.x, j.w, j.t, j.lse, None, 8.0, dx, None, j.ws, st)
    zg.zero_ce_backward(j.plan, j.x, j.w, j.t, j.lse, None, 8.0, None, dw, j.ws, st)
    assert torch.equal(dx, first[3]) and torch.equal(dw, first[4])
    zg.zero_ce_forward(j.plan, j.x, j.w, j.t, j.loss, j.lse, None, j.ws, st)
    assert torch.equal(j.loss, first[0])


def test_pieces_do_not_change_the_loss_and_hardly_the_gradient():
    a, b = Job(150, 4000, 128, "fp16"), Job(150, 4000, 128, "fp16", piece=256)
    assert b.plan.piece == 256 and a.plan.piece == 4096
    for j in (a, b):
        j.forward()
        j.backward(16.0)
    assert torch.equal(a.loss, b.loss) and torch.equal(a.dw, b.dw)
    assert (a.dx.double() - b.dx.double()).norm() <= 2.0 ** -11 * a.dx.double().norm()


@pytest.mark.parametrize("dtype", list(DT))
def test_no_token_has_a_loss(dtype):
    j = Job(70, 500, 64, dtype)
    j.t.fill_(-100)
    j.forward()
    j.check_forward()
    assert not j.loss.any() and j.total.tolist() == [0.0, 0.0]
    j.backward(1024.0)
    assert not j.dx.any() and not j.dw.any()
    j.backward(1024.0, dloss=torch.ones(70, device="cuda"))
    assert not j.dx.any() and not j.dw.any()


def test_no_tokens():
    j = Job(0, 500, 64, "bf16", pad=8)
    j.forward()
    j.backward()
    assert j.total.tolist() == [0.0, 0.0] and not j.dw.any() and _guards_kept(j.fw, j.dw)


def test_one_entry_vocabulary():
    j = Job(33, 1, 64, "bf16")
    j.t[:] = 0
    j.forward()
    assert not j.loss.any()
    j.backward()
    # p = exp(z - lse) = 1 up to exp2's 2^-21 and the base's rounding
    assert (j.dx.float().abs() <= 2.0 ** -18 * (1 + j.lse.abs()[:, None]) * j.w.float().abs().max()).all()


def test_large_logits():
    """Logits of several hundred: the maximum is taken off before exp, and a
    target far below it has a finite loss."""
    j = Job(65, 900, 64, "bf16", spread=80.0)
    j.forward()
    j.check_forward()
    assert j.lse.max() > 150 and j.loss.isfinite().all() and j.loss.max() > 100
    j.backward()
    j.check_backward(torch.full((65,), 1.0 / int(j.counted.sum()), device="cuda", dtype=torch.float64))


def test_nonfinite_tokens_stay_apart():
    j = Job(140, 600, 64, "bf16", ignore=0.0)
    j.forward()
    clean = j.loss.clone()
    j.x[3, 5], j.x[130, 0] = float("nan"), float("inf")
    j.forward()
    assert not j.loss[3].isfinite() and not j.loss[130].isfinite()
    keep = torch.ones(140, dtype=torch.bool, device="cuda")
    keep[3] = keep[130] = False
    assert torch.equal(j.loss[keep], clean[keep])
    j.t[3] = j.t[130] = -100                # without a target such a token has no loss and no gradient of its own
    j.forward()
    j.backward()
    assert j.loss[3] == 0 and j.total[0].isfinite() and not j.dx[3].any() and not j.dx[130].any()
    assert j.dx[keep].isfinite().all()


def test_minus_infinity_in_a_logit():
    """An entry of the vocabulary that a weight of -inf masks: probability 0."""
    j = Job(10, 300, 64, "bf16", ignore=0.0)
    j.x.copy_(j.x.abs() + 0.1)
    j.w[17] = -float("inf")
    j.t[:] = 5
    j.forward()
    w = j.w.double()
    z = j.x.double() @ torch.cat([w[:17], w[18:]]).t()
    want = torch.logsumexp(z, 1)
    assert ((j.lse.double() - want).abs() <= 1e-4).all()


def test_runs_on_the_given_stream():
    j = Job(256, 3000, 256, "bf16")
    j.forward()
    j.backward()
    want = [j.loss.clone(), j.dx.clone(), j.dw.clone()]
    src = j.x.clone()
    j.x.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(8):
            big = big @ big * 1e-3
        j.x.copy_(src)
        j.forward()
        j.backward()
    torch.cuda.synchronize()
    for a, b in zip(want, (j.loss, j.dx, j.dw)):
        assert torch.equal(a, b)


def test_captured_in_a_graph():
    j = Job(100, 2000, 128, "bf16")
    j.forward()
    j.backward()
    want = [j.loss.clone(), j.dx.clone(), j.dw.clone()]
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        j.forward()
        j.backward()
    for t in (j.loss, j.dx, j.dw):
        t.zero_()
    gr.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (j.loss, j.dx, j.dw)):
        assert torch.equal(a, b)


def test_bounded_wait_is_reported():
    """The first block's first copy is announced but not made (test hook): its
    waits run out after seconds, the call reports it and the GPU goes on."""
    j = Job(130, 600, 128, "bf16")
    os.environ["ZERO_TEST_WITHHOLD_TILE"] = "1"
    try:
        j.forward()
    finally:
        del os.environ["ZERO_TEST_WITHHOLD_TILE"]
    with pytest.raises(zg.ZeroError) as e:
        zg.zero_ce_status(j.plan, j.ws)
    assert e.value.status == zg.ZERO_ETIMEOUT and j.loss[0].isnan()
    j.forward()
    zg.zero_ce_status(j.plan, j.ws)
    j.check_forward()


@pytest.mark.parametrize("n", [2, 70])
def test_offsets_past_32_bits(n):
    """A weight of 2^23 + 5 rows of 576 values: 4.8e9 values, 9.7 GB."""
    v, d = 2 ** 23 + 5, 576
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.empty(v, d, dtype=torch.bfloat16, device="cuda")
    for a in range(0, v, 1 << 20):
        w[a:a + (1 << 20)] = torch.randn(min(1 << 20, v - a), d, device="cuda", generator=g) * 0.05
    x = torch.randn(n, d, device="cuda", generator=g).bfloat16()
    t = torch.randint(v - 1000, v, (n,), device="cuda", generator=g)
    p = zg.zero_ce_plan(n, v, d, zg.ZERO_BF16)
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    loss, lse, dx, dw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    zg.zero_ce_forward(p, x, w, t, loss, lse, None, ws)
    zg.zero_ce_backward(p, x, w, t, lse, None, 1.0, dx, dw, ws)
    z = torch.cat([x.double() @ w[a:a + (1 << 19)].double().t() for a in range(0, v, 1 << 19)], 1)
    want = torch.logsumexp(z, 1)
    # one logit is off by e(d) sum |x w| < 1e-3 here (sum |x w| < 40), the rest by less
    assert ((lse.double() - want).abs() <= 1e-3).all()
    assert ((loss.double() - (want - z.gather(1, t[:, None])[:, 0])).abs() <= 2e-3).all()
    G = torch.softmax(z, 1)
    G[torch.arange(n), t] -= 1
    G /= n
    for a, b in ((0, 300), (2 ** 22 - 100, 2 ** 22 + 100), (v - 1000, v)):
        ref = G[:, a:b].t() @ x.double()
        assert (dw[a:b].double() - ref).norm() <= 2.0 ** -7 * ref.norm() + 1e-12
    ref = sum(G[:, a:a + (1 << 19)] @ w[a:a + (1 << 19)].double() for a in range(0, v, 1 << 19))
    assert (dx.double() - ref).norm() <= 2.0 ** -7 * ref.norm()


def test_tiny_upstream_gradients():
    """dloss down to binary32's subnormals: the row factors' inverse stays finite."""
    j = Job(40, 300, 64, "bf16")
    j.forward()
    for d in (1e-30, 1e-39, 0.0):
        j.backward(1.0, dloss=torch.full((40,), d, device="cuda"))
        assert j.dx.isfinite().all() and j.dw.isfinite().all()


@pytest.mark.parametrize("n", [2, 64])
def test_gradients_of_confident_tokens(n):
    """Hidden states along their targets' weights: z_t = 25, every product of
    the same sign, the rest near 0, so p_t - 1 is -5e-9 and the whole gradient
    about that.  What may be left is the logit's change from the loss to its
    gradient: none where both sum alike (n > 3), but lse's rounding, 2^-20 at 25,
    and exp's; where the loss of up to 3 tokens is summed apart, 32 steps a part,
    each cut by half of 2^-23 on average, of a sum that is half the part's."""
    v, d = 300, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    w = (torch.randn(v, d, device="cuda", generator=g) / 64).bfloat16()
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    x = (25 * w[t].float()).bfloat16()
    p = zg.zero_ce_plan(n, v, d, zg.ZERO_BF16)
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    loss, lse, dx, dw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(x), torch.empty_like(w)
    zg.zero_ce_forward(p, x, w, t, loss, lse, None, ws)
    zg.zero_ce_backward(p, x, w, t, lse, torch.ones(n, device="cuda"), 1.0, dx, dw, ws)
    z = x.double() @ w.double().t()
    assert 20 < z.gather(1, t[:, None]).min() and z.gather(1, t[:, None]).max() < 32
    G = torch.softmax(z, 1)
    G[torch.arange(n), t] -= 1
    assert G.abs().max() < 1e-6
    off = 2.0 ** -19 if n > 3 else 16 * 2.0 ** -23 * 32 / 2
    rest = 2.0 ** -10 * G.abs().sum(1)               # the others' relative errors, far above theirs
    assert ((dx.double() - G @ w.double()).abs() <= (off + rest)[:, None] * w.double().abs().max()).all()
    assert ((dw.double() - G.t() @ x.double()).abs() <= n * (off + rest.max()) * x.double().abs().max()).all()


def test_long_sums_are_not_cut_short():
    """dw over 131072 tokens, all products of one sign.  The tensor cores cut
    their running sums toward zero, by up to 2^-23 at each of 64 steps of 16
    in 1024 values; longer sums are added to nearest.  So the mean error of the
    gradients, over 2.6 million of them whose own roundings average out
    (2^-11 / 1600), stays below 64 * 2^-23 and exp's 2^-21."""
    n, v, d = 131072, 2048, 1280
    p = zg.zero_ce_plan(n, v, d, zg.ZERO_FP16)
    g = torch.Generator(device="cuda").manual_seed(2)
    x = (0.5 + torch.rand(n, d, device="cuda", generator=g)).half()
    w = (torch.randn(v, d, device="cuda", generator=g) * 0.02).half()
    t = torch.zeros(n, dtype=torch.int64, device="cuda")     # entry 0 alone has negative products
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    loss, lse, dw = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(w)
    zg.zero_ce_forward(p, x, w, t, loss, lse, None, ws)
    zg.zero_ce_backward(p, x, w, t, lse, None, 2048.0, None, dw, ws)
    want = torch.zeros(v, d, dtype=torch.float64, device="cuda")
    for a in range(0, n, 16384):
        q = torch.softmax(x[a:a + 16384].double() @ w.double().t(), 1)
        want += q.t() @ x[a:a + 16384].double()
    want = want[1:] * (2048.0 / n)
    assert want.min() > 2.0 ** -13                           # normal numbers
    off = ((dw[1:].double() - want) / want).mean()
    assert off.abs() <= 64 * 2.0 ** -23 + 2.0 ** -21 + 6 * 2.0 ** -11 / 1600


@pytest.mark.parametrize("dtype", list(DT))
def test_one_nonfinite_upstream_gradient(dtype):
    """An infinity or NaN in dloss, or a dloss that overflows with the scale,
    is its own token's: the others' dx is what it is without."""
    j = Job(130, 300, 64, dtype)
    j.t[:8] = torch.tensor([1, 2, 3, -100, 4, 5, 6, 7], device="cuda")
    j.forward()
    j.define()
    g = torch.Generator(device="cuda").manual_seed(5)
    clean = 0.5 + torch.rand(130, device="cuda", generator=g)
    for bad, scale in ((float("inf"), 2.0), (-float("inf"), 2.0), (float("nan"), 2.0), (1e38, 64.0)):
        dl = clean.clone()
        dl[2] = 0.0                                  # without the bad one
        j.backward(scale, dloss=dl)
        j.check_backward(dl.double() * scale)
        want = j.dx.clone()
        dl[2] = bad
        j.backward(scale, dloss=dl)
        assert not j.dx[2].isfinite().any() and not j.dw.isfinite().any()
        keep = torch.arange(130, device="cuda") != 2
        assert torch.equal(j.dx[keep], want[keep]), (bad, scale)
        dl[2], dl[3] = 1.0, bad                      # and at a token without a target it counts for nothing
        j.backward(scale, dloss=dl)
        dl[3] = 1.0
        got = j.dx.clone(), j.dw.clone()
        j.backward(scale, dloss=dl)
        assert torch.equal(got[0], j.dx) and torch.equal(got[1], j.dw)


@pytest.mark.parametrize("n,piece", [(3, 0), (140, 256)])
def test_tokens_without_a_target_have_no_gradient_whatever_w_holds(n, piece):
    """A weight of -inf masks an entry of the vocabulary: its products with
    probabilities of 0 are NaN, and so is dx, but not of a token whose gradient
    is 0 by itself."""
    j = Job(n, 600, 64, "bf16", piece=piece, ignore=0.0)
    j.x.copy_(j.x.abs() + 0.1)
    j.w[17] = -float("inf")
    j.t[:] = 5
    j.t[n - 1], j.t[1] = -100, 600
    j.forward()
    assert j.lse.isfinite().all() and j.loss[1] == 0 and j.loss[n - 1] == 0
    for dl in (None, torch.ones(n, device="cuda")):
        j.dx.fill_(GUARD)
        j.backward(8.0, dloss=dl)
        assert not j.dx[1].any() and not j.dx[n - 1].any()
        assert j.dx[0].isnan().all() and _guards_kept(j.fx, j.dx)


@pytest.mark.parametrize("hook,n,v,d,with_dx", [("1", 130, 600, 128, False), ("1", 130, 600, 128, True),
                                                ("2", 130, 600, 128, False), ("2", 2500, 700, 33, False),
                                                ("2", 2500, 700, 33, True)])
def test_bounded_wait_of_the_gradients_is_seen(hook, n, v, d, with_dx):
    """A wait that runs out in the product that makes G (1) or in dw's (2; one
    part, or several): the call reports it, and no gradient of an earlier step is
    left to be taken for this one's, with dx or without."""
    j = Job(n, v, d, "bf16")
    j.forward()
    j.dw.fill_(0.5)
    j.dx.fill_(0.5)
    os.environ["ZERO_TEST_WITHHOLD_TILE"] = hook
    try:
        zg.zero_ce_backward(j.plan, j.x, j.w, j.t, j.lse, None, 1.0, j.dx if with_dx else None, j.dw, j.ws,
                            torch.cuda.current_stream())
    finally:
        del os.environ["ZERO_TEST_WITHHOLD_TILE"]
    with pytest.raises(zg.ZeroError) as e:
        zg.zero_ce_status(j.plan, j.ws)
    assert e.value.status == zg.ZERO_ETIMEOUT
    assert j.dw.isnan().all() and _guards_kept(j.fw, j.dw)
    assert j.dx.isnan().all() if with_dx else (j.dx == 0.5).all()
    j.backward()
    zg.zero_ce_status(j.plan, j.ws)
    assert j.dx.isfinite().all() and j.dw.isfinite().all()


def test_status_of_a_backward_pass_without_outputs():
    """Nothing is computed, so nothing has run out: neither a workspace of any contents nor an earlier call's error is reported."""
    j = Job(130, 600, 64, "bf16")
    none = lambda: zg.zero_ce_backward(j.plan, j.x, j.w, j.t, j.lse, None, 1.0, None, None, j.ws, torch.cuda.current_stream())  # noqa: E731
    none()                                            # the workspace is 0xFF everywhere
    zg.zero_ce_status(j.plan, j.ws)
    os.environ["ZERO_TEST_WITHHOLD_TILE"] = "1"
    try:
        j.forward()
    finally:
        del os.environ["ZERO_TEST_WITHHOLD_TILE"]
    with pytest.raises(zg.ZeroError):
        zg.zero_ce_status(j.plan, j.ws)
    none()
    zg.zero_ce_status(j.plan, j.ws)
    j.forward()
    j.check_forward()


@pytest.mark.parametrize("dtype", list(DT))
def test_tiny_upstream_gradients_against_the_definition(dtype):
    """dloss far below 1, as it is (bfloat16) and scaled up (binary16)."""
    j = Job(40, 300, 64, dtype)
    j.forward()
    j.define()
    g = torch.Generator(device="cuda").manual_seed(6)
    dl = (1 + torch.rand(40, device="cuda", generator=g)) * 1e-30
    scale = 1.0 if dtype == "bf16" else 2.0 ** 100
    j.backward(scale, dloss=dl)
    j.check_backward(dl.double() * scale)
    assert j.dx[0].any() and j.dw[0].any()
