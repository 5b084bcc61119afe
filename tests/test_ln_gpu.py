"""Layer norm on the GPU against its definition in 64 bits.

Tolerances, derived: u is the output type's unit roundoff (2^-11 binary16,
2^-8 bfloat16, 2^-24 binary32; binary16 also has an absolute 2^-25 below its
normals), and a binary32 sum of n terms in which no term passes through more
than `depth` additions is off by at most depth * 2^-24 times the sum of the
magnitudes.  A row's sum is split over at least 32 lanes and joined by a
tree, so depth = dim / 32 + 40 bounds it; a column's sum has at most `rows`
additions.  Products and differences add a few roundings each (the constants
below count them)."""
import pytest
import torch

import zero_sharded_mixed_bucket_gb300 as zg

pytestmark = pytest.mark.gpu

DT = {"fp16": (zg.ZERO_FP16, torch.float16, 2.0 ** -11, 2.0 ** -25),
      "bf16": (zg.ZERO_BF16, torch.bfloat16, 2.0 ** -8, 0.0),
      "fp32": (zg.ZERO_FP32, torch.float32, 2.0 ** -24, 0.0)}
E32 = 2.0 ** -24
GUARD = -77.0


def _buf(rows, dim, stride, dtype, shift=0):
    """rows x dim view, `stride` apart, starting `shift` values into a guarded buffer."""
    full = torch.full((max(rows, 1) * stride + 64 + shift,), GUARD, dtype=dtype, device="cuda")
    at = 32 + shift
    return full, full[at:at + max(rows, 1) * stride].view(-1, stride)[:rows, :dim]


def _guards_kept(full, view):
    keep = torch.ones_like(full, dtype=torch.bool)
    keep.as_strided(view.shape, view.stride(), view.storage_offset()).fill_(False)
    return bool((full[keep] == GUARD).all())


def _inputs(rows, dim, dtype, xs, ys, shift, seed=0, scale=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[dtype][1]
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    _, x = _buf(rows, dim, xs, dt, shift)
    _, dy = _buf(rows, dim, ys, dt, shift)
    x.copy_(r(rows, dim) * scale + r(dim))
    dy.copy_(r(rows, dim))
    return x, dy, (1 + 0.3 * r(dim)).to(dt), (0.2 * r(dim)).to(dt)


def _definition(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = 1 / torch.sqrt(var + eps)
    h = (x - mean[:, None]) * rstd[:, None]
    return mean, rstd, h, h * (1 if w is None else w.double()) + (0 if b is None else b.double())


def _within(got, want, tol, what):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), "%s: %d values off, worst %g of the tolerance" % (
        what, int(bad.sum()), float(((got.double() - want).abs() / tol).max()))


SHAPES = [  # rows, dim, x pad, y pad, shift of the first row in values
    (1, 768, 0, 0, 0), (1, 1, 0, 0, 0), (5, 1, 3, 0, 1), (3, 2, 0, 0, 0), (7, 17, 0, 0, 0), (4, 33, 7, 1, 0),
    (300, 64, 0, 0, 0), (33, 255, 1, 0, 0), (257, 1000, 0, 24, 0), (64, 1600, 0, 0, 0), (130, 4096, 0, 0, 0),
    (19, 4096, 8, 8, 8), (19, 4096, 0, 0, 1), (1003, 771, 5, 5, 0), (9, 8192, 0, 0, 0), (6, 8200, 0, 0, 0),
    (3, 16384, 0, 0, 0), (2, 20000, 0, 0, 0), (2, 70001, 0, 0, 0), (2500, 96, 0, 0, 0), (9000, 8, 0, 0, 0),
    # rows on 4-byte boundaries, and rows of a block of 512 threads
    (300, 134, 0, 0, 0), (37, 770, 0, 0, 2), (611, 1438, 0, 2, 0), (11, 5806, 0, 0, 0), (350, 10460, 0, 0, 0),
    (5, 13001, 1, 1, 0), (170, 12000, 0, 0, 0), (3, 30002, 0, 0, 0), (2, 32768, 0, 0, 0),
]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,dim,xp,yp,shift", SHAPES)
def test_forward(rows, dim, xp, yp, shift, dtype):
    code, dt, u, tiny = DT[dtype]
    xs, ys, eps = dim + xp, dim + yp, 1e-5
    x, _, w, b = _inputs(rows, dim, dtype, xs, ys, shift, seed=rows + dim)
    full, y = _buf(rows, dim, ys, dt, shift)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    plan = zg.zero_ln_plan(rows, dim, code, xs, ys)
    zg.zero_ln_forward(plan, x, w, b, eps, y, mean, rstd, torch.cuda.current_stream())
    m, r, h, want = _definition(x, w, b, eps)
    depth = dim / 32 + 40
    dm = (depth + 2) * E32 * x.double().abs().mean(1)
    _within(mean, m, dm + 1e-38, "mean")
    # var: the mean's error enters squared and through its own rounding
    dr = r * ((depth + 8) * E32 + 0.5 * (r * dm) ** 2 * 2)
    _within(rstd, r, dr, "rstd")
    dh = r[:, None] * dm[:, None] + h.abs() * (dr / r + 4 * E32)[:, None]
    tol = w.double().abs() * dh + 2 * E32 * (w.double() * h).abs() + u * want.abs() * 1.01 + E32 * want.abs() + tiny + 1e-38
    _within(y, want, tol + u * (w.double().abs() * dh), "y")
    assert _guards_kept(full, y)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,dim,xp,yp,shift", SHAPES)
def test_backward(rows, dim, xp, yp, shift, dtype):
    code, dt, u, tiny = DT[dtype]
    xs, ys = dim + xp, dim + yp
    x, dy, w, b = _inputs(rows, dim, dtype, xs, ys, shift, seed=rows * 3 + dim)
    m, r, _, _ = _definition(x, w, b, 1e-5)
    mean, rstd = m.float(), r.float()
    full, dx = _buf(rows, dim, xs, dt, shift)
    fw, dw = _buf(1, dim, dim, dt, shift)
    fb, db = _buf(1, dim, dim, dt, shift)
    plan = zg.zero_ln_plan(rows, dim, code, xs, ys)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream()
    zg.zero_ln_backward(plan, dy, x, w, mean, rstd, dx, dw, db, ws, st)
    # the formula at the given statistics
    m, r = mean.double(), rstd.double()
    h = (x.double() - m[:, None]) * r[:, None]
    g = dy.double() * w.double()
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    want = (g - c1 - h * c2) * r[:, None]
    depth = dim / 32 + 40
    d1 = (depth + 3) * E32 * g.abs().mean(1, keepdim=True)
    d2 = (depth + 6) * E32 * (g * h).abs().mean(1, keepdim=True)
    tol = r[:, None] * (d1 + h.abs() * d2 + 6 * E32 * (g.abs() + c1.abs() + (h * c2).abs())) * (1 + u)
    _within(dx, want, tol + 1.01 * u * want.abs() + tiny + 1e-38, "dx")
    _within(dw[0], (dy.double() * h).sum(0), (rows + 8) * E32 * (dy.double() * h).abs().sum(0) * (1 + u)
            + 1.01 * u * (dy.double() * h).sum(0).abs() + tiny + 1e-38, "dweight")
    _within(db[0], dy.double().sum(0), (rows + 2) * E32 * dy.double().abs().sum(0) * (1 + u)
            + 1.01 * u * dy.double().sum(0).abs() + tiny + 1e-38, "dbias")
    assert _guards_kept(full, dx) and _guards_kept(fw, dw) and _guards_kept(fb, db)
    # the same call again gives the same bits, and outputs may be left out
    again = [torch.empty_like(t) for t in (dw[0], db[0])]
    dx2 = torch.empty_strided(dx.shape, dx.stride(), dtype=dt, device="cuda")
    zg.zero_ln_backward(plan, dy, x, w, mean, rstd, dx2, again[0], None, ws, st)
    zg.zero_ln_backward(plan, dy, x, w, mean, rstd, None, None, again[1], ws, st)
    bits = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
    assert torch.equal(bits(again[0]), bits(dw[0])) and torch.equal(bits(again[1]), bits(db[0]))
    assert torch.equal(bits(dx2), bits(dx))


def test_gradient_against_differences():
    """The fp32 kernels' gradients against central differences of the 64-bit
    forward definition: step 1e-4 of O(1) inputs, truncation ~1e-8 of the
    third derivative, so 1e-4 of the gradient's size is generous."""
    rows, dim = 6, 40
    x, dy, w, b = _inputs(rows, dim, "fp32", dim, dim, 0, seed=4)
    plan = zg.zero_ln_plan(rows, dim, zg.ZERO_FP32)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zg.zero_ln_forward(plan, x, w, b, 1e-5, y, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    zg.zero_ln_backward(plan, dy, x, w, mean, rstd, dx, dw, db, ws)
    f = lambda x, w, b: (_definition(x, w, b, 1e-5)[3] * dy.double()).sum()  # noqa: E731
    args = [x.double(), w.double(), b.double()]
    g = torch.Generator(device="cuda").manual_seed(1)
    for k, grad in enumerate((dx, dw, db)):
        for _ in range(8):
            d = torch.randn(args[k].shape, device="cuda", generator=g, dtype=torch.float64)
            hi, lo = list(args), list(args)
            hi[k], lo[k] = args[k] + 1e-4 * d, args[k] - 1e-4 * d
            want = (f(*hi) - f(*lo)) / 2e-4
            got = (grad.double() * d).sum()
            assert abs(got - want) <= 1e-4 * (grad.double().norm() * d.norm())


@pytest.mark.parametrize("dtype", list(DT))
def test_without_weight_or_bias_or_statistics(dtype):
    code, dt, u, tiny = DT[dtype]
    x, dy, w, b = _inputs(11, 200, dtype, 200, 200, 0)
    plan = zg.zero_ln_plan(11, 200, code)
    y, ones, zeros = torch.empty_like(x), torch.ones_like(w), torch.zeros_like(b)
    want = torch.empty_like(x)
    for ww, bb in ((None, None), (w, None), (None, b)):
        zg.zero_ln_forward(plan, x, ww, bb, 1e-5, y)
        zg.zero_ln_forward(plan, x, ones if ww is None else ww, zeros if bb is None else bb, 1e-5, want)
        assert torch.equal(y, want)
    mean, rstd = torch.empty(11, device="cuda"), torch.empty(11, device="cuda")
    zg.zero_ln_forward(plan, x, None, None, 1e-5, y, mean, rstd)
    dx, dx1 = torch.empty_like(x), torch.empty_like(x)
    zg.zero_ln_backward(plan, dy, x, None, mean, rstd, dx)
    zg.zero_ln_backward(plan, dy, x, ones, mean, rstd, dx1)
    assert torch.equal(dx, dx1)


def test_constant_rows_and_nonfinite_rows_stay_apart():
    rows, dim = 9, 520
    x, dy, w, b = _inputs(rows, dim, "fp32", dim, dim, 0)
    x[2] = 3.0                       # no variance: y is the bias
    plan = zg.zero_ln_plan(rows, dim, zg.ZERO_FP32)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    zg.zero_ln_forward(plan, x, w, b, 1e-5, y, mean, rstd)
    assert torch.equal(y[2], b) and mean[2] == 3.0
    clean = y.clone()
    x[4, 7], x[5, 0], x[6, 519] = float("nan"), float("inf"), -float("inf")
    zg.zero_ln_forward(plan, x, w, b, 1e-5, y, mean, rstd)
    assert y[4:7].isnan().all()
    keep = [0, 1, 2, 3, 7, 8]
    assert torch.equal(y[keep], clean[keep])


def test_no_rows():
    plan = zg.zero_ln_plan(0, 100, zg.ZERO_BF16)
    dw, db = (torch.full((100,), 5.0, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    zg.zero_ln_forward(plan, None, None, None, 1e-5, None)
    zg.zero_ln_backward(plan, None, None, None, None, None, None, dw, db, ws)
    assert not dw.any() and not db.any()


def test_rows_past_32_bit_offsets():
    """Rows whose element offsets pass 2^31 (and byte offsets 2^32)."""
    rows, dim, stride = 3, 64, (1 << 30) + 8
    full = torch.empty(2 * stride + dim, dtype=torch.bfloat16, device="cuda")
    x = full.as_strided((rows, dim), (stride, 1))
    src = torch.randn(rows, dim, device="cuda").bfloat16()
    x.copy_(src)
    y, y1 = torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16), torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16)
    zg.zero_ln_forward(zg.zero_ln_plan(rows, dim, zg.ZERO_BF16, stride, dim), x, None, None, 1e-5, y)
    zg.zero_ln_forward(zg.zero_ln_plan(rows, dim, zg.ZERO_BF16), src, None, None, 1e-5, y1)
    assert torch.equal(y, y1)


def test_runs_on_the_given_stream():
    """Work queued behind a slow producer on a side stream sees its results."""
    x, _, w, b = _inputs(512, 2048, "bf16", 2048, 2048, 0)
    late, y, want = torch.zeros_like(x), torch.empty_like(x), torch.empty_like(x)
    plan = zg.zero_ln_plan(512, 2048, zg.ZERO_BF16)
    zg.zero_ln_forward(plan, x, w, b, 1e-5, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(8):
            big = big @ big * 1e-3
        late.copy_(x)
    zg.zero_ln_forward(plan, late, w, b, 1e-5, y, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("rows,dim,shift", [(5, 48, 0), (9, 768, 0), (9, 771, 1), (5, 2000, 0), (3, 4096, 1), (3, 9000, 1)])
@pytest.mark.parametrize("size,up", [(1e-22, 1.0), (1e-12, 1e-6), (1e10, 1e6), (1e17, 1e-12)])
def test_backward_of_rows_of_any_size(rows, dim, shift, size, up):
    """1/rstd far from 1: xhat is of order 1 whatever x's size, and no power of
    rstd beyond the first belongs in the result."""
    x, dy, w, b = _inputs(rows, dim, "fp32", dim, dim, shift)
    x *= size
    dy *= up
    m, r, _, _ = _definition(x, None, None, 0.0)
    mean, rstd = m.float(), r.float()
    plan = zg.zero_ln_plan(rows, dim, zg.ZERO_FP32)
    (_, dx), (_, dw), (_, db) = _buf(rows, dim, dim, torch.float32, shift), _buf(1, dim, dim, torch.float32), _buf(1, dim, dim, torch.float32)
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    zg.zero_ln_backward(plan, dy, x, w, mean, rstd, dx, dw, db, ws)
    m, r = mean.double(), rstd.double()
    h = (x.double() - m[:, None]) * r[:, None]
    g = dy.double() * w.double()
    c1, c2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    want = (g - c1 - h * c2) * r[:, None]
    depth = dim / 32 + 40
    d1 = (depth + 3) * E32 * g.abs().mean(1, keepdim=True)
    d2 = (depth + 6) * E32 * (g * h).abs().mean(1, keepdim=True)
    tol = r[:, None] * (d1 + h.abs() * d2 + 6 * E32 * (g.abs() + c1.abs() + (h * c2).abs()))
    _within(dx, want, tol + 1.01 * E32 * want.abs(), "dx")
    _within(dw[0], (dy.double() * h).sum(0), (rows + 8) * E32 * (dy.double() * h).abs().sum(0), "dweight")
    _within(db[0], dy.double().sum(0), (rows + 2) * E32 * dy.double().abs().sum(0), "dbias")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("dim", [56, 104, 208, 2256, 4280, 8560, 60, 61, 95, 191, 3000, 9000, 9001, 16872])
def test_constant_rows_have_no_variance(dim, dtype):
    """Rows of one value, a whole number whose sums are exact in binary32: the
    mean is that number, y the bias and rstd 1/sqrt(eps), whatever dim is and
    however small eps (an error of one unit in the mean's last place is 0.02 of a
    standard deviation at eps = 1e-5)."""
    code, dt, u, tiny = DT[dtype]
    x, _, w, b = _inputs(5, dim, dtype, dim, dim, 0)
    for k, c in enumerate((1000, -1000, 500, 7, 0)):
        x[k] = c
    plan = zg.zero_ln_plan(5, dim, code)
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    for eps in (1e-5, 1e-12):
        zg.zero_ln_forward(plan, x, w, b, eps, y, mean, rstd)
        assert mean.tolist() == [1000.0, -1000.0, 500.0, 7.0, 0.0]
        assert torch.equal(y, b.expand(5, dim))
        assert ((rstd.double() * eps ** 0.5 - 1).abs() <= 4 * E32).all()
