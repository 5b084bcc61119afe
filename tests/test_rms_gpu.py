"""The root-mean-square norm on the GPU, against its formulas in 64 bits.

Bounds: a row's mean square is a binary32 sum whose longest chain of additions
is `_chain(dim)`, so it is off by that many half units in the last place at
most, and 1/sqrt of it by half of that and rsqrtf's own 2 units; the products
after it round once each; the result is rounded to its type once."""
import numpy as np
import pytest
import torch

import zero_sharded_mixed_bucket_gb300 as zg
from tests.launches import launches

pytestmark = pytest.mark.gpu

DT = {"fp16": (zg.ZERO_FP16, torch.float16), "bf16": (zg.ZERO_BF16, torch.bfloat16), "fp32": (zg.ZERO_FP32, torch.float32)}
EPS, GUARD, U = 1e-5, -77.0, 2.0 ** -24


def _chain(dim):
    """Additions in a row: a lane's own (64 values, or dim / 512 of a long row), the lanes' tree, the warps'."""
    return (dim if dim < 64 else 64 if dim <= 32768 else dim // 512 + 4) + 5 + 16


def _half(dt):
    return torch.finfo(dt).eps / 2


def _least(dt):
    """Half the distance of the type's smallest numbers."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2


class Rows:
    """(n, d) values, rows `stride` apart, in a guarded buffer `shift` values off a 16-byte boundary."""

    def __init__(self, n, d, stride, shift, dt, values=None, guard=GUARD):
        self.full = torch.full((n * stride + 64 + shift,), guard, dtype=dt, device="cuda")
        self.v = self.full[32 + shift:].as_strided((n, d), (stride, 1))
        self.guard, self.n, self.d = guard, n, d
        if values is not None:
            self.v.copy_(values)

    def kept(self):
        mask = torch.ones_like(self.full, dtype=torch.bool)
        mask.as_strided(self.v.shape, self.v.stride(), self.v.storage_offset()).fill_(False)
        return bool((self.full[mask] == self.guard).all())


def _setup(n, d, dtype, xpad=0, ypad=0, shift=0, seed=0, scale=2.0, block=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 7 * n + d)
    code, dt = DT[dtype]
    r = lambda k, *size: torch.randn(*size, device="cuda", generator=g) * k  # noqa: E731
    xs, ys = d + xpad, d + ypad
    s = {"x": Rows(n, d, xs, shift, dt, r(scale, n, d)), "r": Rows(n, d, xs, shift, dt, r(1.5 * scale, n, d)),
         "w": (1 + r(0.3, d)).to(dt), "h": Rows(n, d, xs, shift, dt), "y": Rows(n, d, ys, shift, dt),
         "rstd": torch.full((n,), GUARD, device="cuda"), "plan": zg.zero_rms_plan(n, d, code, xs, ys, block), "dt": dt}
    if block:
        s["q"] = Rows(n, d, ys, shift, torch.uint8, guard=0xA5)
        s["q_scale"] = torch.full((n, s["plan"].scale_cols), 0xA5, dtype=torch.uint8, device="cuda")
    return s


def _want(h, w, dim):
    h = h.double()
    rstd = 1 / torch.sqrt((h * h).mean(1) + EPS)
    return rstd, h * rstd[:, None] * (1 if w is None else w.double())


def _close_y(y, y64, dt, dim):
    tol = y64.abs() * (_half(dt) * 1.001 + U * (_chain(dim) / 2 + 8)) + _least(dt)
    return bool(((y.double() - y64).abs() <= tol).all())


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 8), (9, 16), (33, 31), (700, 64), (701, 65), (130, 96), (67, 128), (66, 129), (40, 255),
          (37, 256), (257, 768), (255, 771), (31, 1000), (64, 2048), (13, 2049), (1, 4096), (9, 4096), (7, 4097), (5, 8192),
          (5, 8200), (3, 10007), (3, 16384), (2, 16391), (2, 32768), (2, 40001), (1, 100_000),
          (160, 9001), (310, 16391), (306, 32800)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad,shift", [((0, 0), 0), ((8, 16), 0), ((1, 3), 0), ((2, 2), 2), ((0, 0), 1)], ids=str)
@pytest.mark.parametrize("n,d", SHAPES)
def test_forward_and_backward(n, d, pad, shift, dtype):
    s = _setup(n, d, dtype, *pad, shift)
    dt, p, st = s["dt"], s["plan"], torch.cuda.current_stream()
    zg.zero_rms_forward(p, s["x"].v, s["r"].v, s["w"], EPS, s["h"].v, s["y"].v, None, None, s["rstd"], st)
    want_h = (s["x"].v.float() + s["r"].v.float()).to(dt)
    assert torch.equal(s["h"].v, want_h)
    rstd64, y64 = _want(want_h, s["w"], d)
    assert bool(((s["rstd"].double() - rstd64).abs() <= rstd64 * U * (_chain(d) / 2 + 6)).all())
    assert _close_y(s["y"].v, y64, dt, d)
    assert all(s[k].kept() for k in ("x", "r", "h", "y"))
    # backward, from the statistics as given
    g = torch.Generator(device="cuda").manual_seed(n)
    dy = Rows(n, d, p.y_stride, shift, dt, torch.randn(n, d, device="cuda", generator=g))
    dh = Rows(n, d, p.x_stride, shift, dt, torch.randn(n, d, device="cuda", generator=g))
    dx = Rows(n, d, p.x_stride, shift, dt)
    dw = torch.full((d,), GUARD, dtype=dt, device="cuda")
    ws = torch.full((p.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")
    zg.zero_rms_backward(p, dy.v, dh.v, s["h"].v, s["w"], s["rstd"], dx.v, dw, ws, st)
    rstd = s["rstd"].double()[:, None]
    xhat, gw = want_h.double() * rstd, dy.v.double() * s["w"].double()
    m, mag = (gw * xhat).mean(1, keepdim=True), (gw * xhat).abs().mean(1, keepdim=True)
    dx64 = rstd * (gw - xhat * m) + dh.v.double()
    tol = dx64.abs() * _half(dt) * 1.001 + _least(dt) + U * (rstd * (8 * gw.abs() + xhat.abs() * (_chain(d) + 8) * mag) + 2 * dx64.abs())
    assert bool(((dx.v.double() - dx64).abs() <= tol).all())
    dw64, dmag = (dy.v.double() * xhat).sum(0), (dy.v.double() * xhat).abs().sum(0)
    tol = dw64.abs() * _half(dt) * 1.001 + _least(dt) + U * dmag * (n + 64)       # a lane's rows one after another, then the blocks
    assert bool(((dw.double() - dw64).abs() <= tol).all())
    assert dx.kept() and dy.kept() and dh.kept()
    # without the stream's gradient, into dh itself, and each output alone
    alone = torch.full((d,), GUARD, dtype=dt, device="cuda")
    zg.zero_rms_backward(p, dy.v, None, s["h"].v, s["w"], s["rstd"], None, alone, ws, st)
    assert torch.equal(alone, dw)
    zg.zero_rms_backward(p, dy.v, dh.v, s["h"].v, s["w"], s["rstd"], dh.v, None, None, st)
    assert torch.equal(dh.v, dx.v) and dh.kept()
    plain = Rows(n, d, p.x_stride, shift, dt)
    zg.zero_rms_backward(p, dy.v, None, s["h"].v, s["w"], s["rstd"], plain.v, None, None, st)
    plain64 = rstd * (gw - xhat * m)
    tol = plain64.abs() * _half(dt) * 1.001 + _least(dt) + U * (rstd * (8 * gw.abs() + xhat.abs() * (_chain(d) + 8) * mag) + 2 * plain64.abs())
    assert bool(((plain.v.double() - plain64).abs() <= tol).all())


@pytest.mark.parametrize("n,d", [(1, 8196), (5, 8193), (160, 9001), (3, 12288), (310, 10_000), (320, 16384)])
def test_long_binary32_rows_backward_wherever_they_start(n, d):
    """Rows of 8193 to 16384 values on 16-byte boundaries take the kernel that the same rows off them take: one pass and a join, equal bits."""
    stride = (d + 3) // 4 * 4
    p = zg.zero_rms_plan(n, d, zg.ZERO_FP32, stride, stride)
    g = torch.Generator(device="cuda").manual_seed(d)
    value = [torch.randn(n, d, device="cuda", generator=g) for _ in range(3)]
    w, rstd = torch.randn(d, device="cuda", generator=g), torch.rand(n, device="cuda", generator=g) + 0.5
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    out = []
    for shift in (0, 1):
        h, dy, dh = (Rows(n, d, stride, shift, torch.float32, v) for v in value)
        dx, dw = Rows(n, d, stride, shift, torch.float32), torch.full((d,), GUARD, device="cuda")
        assert (h.v.data_ptr() % 16 == 0) == (shift == 0)
        call = lambda s: zg.zero_rms_backward(p, dy.v, dh.v, h.v, w, rstd, dx.v, dw, ws, s)  # noqa: E731
        assert launches(call) == 2
        call(torch.cuda.current_stream())
        assert dx.kept()
        out.append((dx.v.clone(), dw))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


def _codes(y64, block):
    """Scale bytes and the values that codes stand for, from 64-bit results; and where a scale is within binary32's error of the next."""
    n, d = y64.shape
    b = torch.nn.functional.pad(y64, (0, -d % block)).view(n, -1, block)
    most = b.abs().amax(2)
    e = torch.ceil(torch.log2(most.clamp(min=2.0 ** -140) / 448)).clamp(min=-127)
    near = (torch.log2(most.clamp(min=2.0 ** -140) / 448) - torch.round(torch.log2(most.clamp(min=2.0 ** -140) / 448))).abs() < 1e-5
    return (e + 127).long(), near


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("block", [32, 128])
@pytest.mark.parametrize("pad,shift", [((0, 0), 0), ((8, 16), 0), ((1, 3), 0), ((2, 2), 2)], ids=str)
@pytest.mark.parametrize("n,d", [(1, 1), (3, 31), (5, 32), (6, 33), (33, 96), (17, 128), (16, 129), (130, 768), (31, 771), (1, 4096),
                                 (9, 4096), (5, 4100), (4, 8192), (3, 8200), (3, 16384), (2, 16391), (2, 40001)])
def test_8bit_results(n, d, pad, shift, block, dtype):
    s = _setup(n, d, dtype, *pad, shift, block=block)
    dt, p, st = s["dt"], s["plan"], torch.cuda.current_stream()
    if n > 2:
        s["x"].v[1] = 0
        s["r"].v[1] = 0                               # a row of zeros
    zg.zero_rms_forward(p, s["x"].v, s["r"].v, s["w"], EPS, s["h"].v, s["y"].v, s["q"].v, s["q_scale"], s["rstd"], st)
    _, y64 = _want(s["h"].v, s["w"], d)
    assert _close_y(s["y"].v, y64, dt, d)
    e, near = _codes(y64, block)
    got = s["q_scale"].long()
    assert bool(((got == e) | (near & ((got - e).abs() <= 1))).all())
    values = Rows(n, d, p.y_stride, shift, torch.bfloat16)
    zg.zero_rms_values(p, s["q"].v, s["q_scale"], values.v, st)
    unit = torch.exp2(got.double() - 127).repeat_interleave(block, 1)[:, :d]
    code = torch.empty(n, d, dtype=torch.uint8, device="cuda").copy_(s["q"].v)
    stands = code.view(torch.float8_e4m3fn).double() * unit
    assert torch.equal(values.v.double(), stands)
    # e4m3: half of 2^-3 of a binade, 2^-9 apart below 2^-6
    tol = y64.abs() * (2.0 ** -4 + U * (_chain(d) / 2 + 8)) + unit * 2.0 ** -10 * 1.001
    assert bool(((stands - y64).abs() <= tol).all())
    assert all(s[k].kept() for k in ("x", "r", "h", "y", "q")) and values.kept()
    # the 8-bit results alone, without a residual or a weight
    q2, sc2 = Rows(n, d, p.y_stride, shift, torch.uint8, guard=0xA5), torch.empty_like(s["q_scale"])
    zg.zero_rms_forward(p, s["h"].v, None, None, EPS, None, None, q2.v, sc2, None, st)
    _, y64 = _want(s["h"].v, None, d)
    unit = torch.exp2(sc2.double() - 127).repeat_interleave(block, 1)[:, :d]
    code.copy_(q2.v)
    assert bool(((code.view(torch.float8_e4m3fn).double() * unit - y64).abs() <= y64.abs() * (2.0 ** -4 + U * (_chain(d) / 2 + 8)) + unit * 2.0 ** -10 * 1.001).all())
    assert q2.kept()


@pytest.mark.parametrize("d", [256, 771])
def test_8bit_blocks_that_are_not_finite_and_the_scale_range(d):
    """An infinity or a NaN spoils its own row's blocks as the formula has it; scales at both ends of a byte."""
    p = zg.zero_rms_plan(4, d, zg.ZERO_FP32, block=128)
    x = torch.randn(4, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    w = torch.ones(d, device="cuda")
    w[:128] = 2.0 ** 120
    w[128:256] = 2.0 ** -126
    x[1, 5] = float("nan")
    x[2, 130] = float("inf")                          # rstd 0: 0 elsewhere, inf * 0 there
    q, sc = torch.empty(4, d, dtype=torch.uint8, device="cuda"), torch.empty(4, p.scale_cols, dtype=torch.uint8, device="cuda")
    y, v = torch.empty_like(x), torch.empty(4, d, dtype=torch.bfloat16, device="cuda")
    zg.zero_rms_forward(p, x, None, w, EPS, None, y, q, sc, None)
    zg.zero_rms_values(p, q, sc, v)
    assert bool((sc[1] == 255).all()) and bool(v[1].isnan().all()) and bool(y[1].isnan().all())
    assert int(sc[2, 0]) == 0 and bool((v[2, :128] == 0).all())
    assert int(sc[2, 1]) == 255 and bool(v[2, 128:256].isnan().all())
    _, y64 = _want(x[[0, 3]], w, d)
    e, near = _codes(y64, 128)
    assert bool((near | (sc[[0, 3]].long() == e)).all()) and int(sc[0, 1]) == 0 and int(sc[0, 0]) > 235
    unit = torch.exp2(sc[[0, 3]].double() - 127).repeat_interleave(128, 1)[:, :d]
    got = q[[0, 3]].view(torch.float8_e4m3fn).double() * unit
    assert bool(((got - y64).abs() <= y64.abs() * 2.0 ** -4 * 1.001 + unit * 2.0 ** -10 * 1.001 + 2.0 ** -149).all())
    # read out: exact but below bfloat16's smallest numbers, to the nearest of those
    off = (v[[0, 3]].double() - got).abs()
    assert bool((off <= 2.0 ** -134).all()) and bool((off[got.abs() >= 2.0 ** -126] == 0).all())


def test_every_code_and_scale_read_out():
    """All 256 codes under scale bytes from 0 to 255, 16 codes at a time and one by one."""
    scales = torch.tensor(list(range(0, 16)) + list(range(100, 150)) + list(range(230, 256)), dtype=torch.uint8, device="cuda")
    n = len(scales)
    for d, stride in ((256, 256), (256, 257), (255, 255)):
        p = zg.zero_rms_plan(n, d, zg.ZERO_BF16, y_stride=stride, block=128)
        q = torch.zeros(n, stride, dtype=torch.uint8, device="cuda")
        q[:, :d] = torch.arange(d, device="cuda").to(torch.uint8)
        v = torch.full((n, stride), GUARD, dtype=torch.bfloat16, device="cuda")
        zg.zero_rms_values(p, q, scales[:, None].expand(n, 2).contiguous(), v)
        want = q[:, :d].contiguous().view(torch.float8_e4m3fn).double() * torch.exp2(scales.double() - 127)[:, None]
        want[scales == 255] = float("nan")
        got = v[:, :d].double()
        assert torch.equal(got.isnan(), want.isnan()) and bool((v[:, d:] == GUARD).all())
        fine = ~want.isnan()
        big = fine & (want.abs() > torch.finfo(torch.bfloat16).max)
        assert bool((got[big] == want[big].sign() * float("inf")).all())
        fine &= ~big
        assert bool(((got - want).abs()[fine] <= 2.0 ** -134).all()) and torch.equal(got[fine & (want.abs() >= 2.0 ** -126)], want[fine & (want.abs() >= 2.0 ** -126)])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [64, 771, 768, 4096, 20_001, 40_000])
def test_stream_updated_in_place(d, dtype):
    """h may be the residual, or x, itself."""
    a, b = _setup(9, d, dtype), _setup(9, d, dtype)
    zg.zero_rms_forward(a["plan"], a["x"].v, a["r"].v, a["w"], EPS, a["h"].v, a["y"].v, None, None, a["rstd"])
    for own in ("r", "x"):
        b = _setup(9, d, dtype)
        zg.zero_rms_forward(b["plan"], b["x"].v, b["r"].v, b["w"], EPS, b[own].v, b["y"].v, None, None, b["rstd"])
        assert torch.equal(b[own].v, a["h"].v) and torch.equal(b["y"].v, a["y"].v) and torch.equal(b["rstd"], a["rstd"])
        assert b[own].kept()


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d,pad", [(256, 0), (4096, 0), (257, 1), (4097, 0), (40_000, 0)])
def test_stream_of_any_bit_patterns(d, pad, dtype):
    """x + residual is the binary32 sum rounded once, for every exponent, subnormal numbers, infinities and NaN."""
    code, dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(d)
    kind = torch.int32 if dtype == "fp32" else torch.int16
    lim = torch.iinfo(kind)
    bits = lambda: torch.randint(lim.min, lim.max + 1, (64, d + pad), device="cuda", generator=g, dtype=torch.int64).to(kind).view(dt)  # noqa: E731
    x, r = bits(), bits()
    r[::4] = -x[::4]                                  # sums of 0
    r[1::4] = (x[1::4].float() * 2.0 ** -9).to(dt)    # sums between two numbers
    h, y = torch.empty_like(x), torch.empty_like(x)
    p = zg.zero_rms_plan(64, d, code, d + pad, d + pad)
    zg.zero_rms_forward(p, x, r, None, EPS, h, y)
    want = (x.float() + r.float()).to(dt)[:, :d]
    got = h[:, :d]
    assert torch.equal(got.isnan(), want.isnan())
    keep = ~want.isnan()
    assert torch.equal(got[keep].view(kind), want[keep].view(kind))


def test_gradients_against_differences():
    """Central differences of sum(c y) + sum(k h) in binary64 of the formula, through the kernels' gradients in binary32."""
    n, d = 3, 40
    g = torch.Generator(device="cuda").manual_seed(5)
    h, w, c, k = (torch.randn(*size, device="cuda", generator=g) for size in ((n, d), (d,), (n, d), (n, d)))
    p = zg.zero_rms_plan(n, d, zg.ZERO_FP32)
    y, rstd, dx, dw = torch.empty_like(h), torch.empty(n, device="cuda"), torch.empty_like(h), torch.empty_like(w)
    zg.zero_rms_forward(p, h, None, w, EPS, None, y, None, None, rstd)
    zg.zero_rms_backward(p, c, k, h, w, rstd, dx, dw, torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda"))
    loss = lambda h, w: float((c.double() * h * w / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)).sum() + (k.double() * h).sum())  # noqa: E731
    step = 1e-5
    for i in range(0, n * d, 7):
        e = torch.zeros(n * d, dtype=torch.float64, device="cuda")
        e[i] = step
        e = e.view(n, d)
        diff = (loss(h.double() + e, w.double()) - loss(h.double() - e, w.double())) / (2 * step)
        assert abs(diff - float(dx.view(-1)[i])) < 1e-4
    for i in range(0, d, 5):
        e = torch.zeros(d, dtype=torch.float64, device="cuda")
        e[i] = step
        diff = (loss(h.double(), w.double() + e) - loss(h.double(), w.double() - e)) / (2 * step)
        assert abs(diff - float(dw[i])) < 1e-4


def test_no_rows_and_no_outputs():
    p = zg.zero_rms_plan(0, 100, zg.ZERO_FP32)
    dw = torch.full((100,), GUARD, device="cuda")
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    zg.zero_rms_backward(p, None, None, None, None, None, None, dw, ws)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("d", [1000, 20_000])
def test_offsets_past_32_bits(d, odd, dtype):
    """Rows 2^31 values apart: only three exist, the rest of the buffer is never touched."""
    code, dt = DT[dtype]
    stride = (1 << 31) + (16 if dtype == "bf16" else 4) + odd
    big = torch.empty(2 * stride + d, dtype=dt, device="cuda")
    v = big.as_strided((3, d), (stride, 1))
    x = torch.randn(3, d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).to(dt)
    v.copy_(x)
    p = zg.zero_rms_plan(3, d, code, stride, 0, 128)
    y, q, sc, rstd = torch.empty(3, d, dtype=dt, device="cuda"), torch.empty(3, d, dtype=torch.uint8, device="cuda"), \
        torch.empty(3, p.scale_cols, dtype=torch.uint8, device="cuda"), torch.empty(3, device="cuda")
    zg.zero_rms_forward(p, v, None, None, EPS, None, y, q, sc, rstd)
    _, y64 = _want(x, None, d)
    assert _close_y(y, y64, dt, d)
    if dtype == "bf16":                               # codes and values as far apart
        f = zg.zero_rms_plan(3, d, code, stride, stride, 128)
        fq, fv = (torch.empty(2 * stride + d, dtype=t, device="cuda").as_strided((3, d), (stride, 1)) for t in (torch.uint8, torch.bfloat16))
        near = torch.empty(3, d, dtype=torch.bfloat16, device="cuda")
        zg.zero_rms_forward(f, v, None, None, EPS, None, None, fq, sc, rstd)
        zg.zero_rms_values(f, fq, sc, fv)
        zg.zero_rms_values(p, q, sc, near)
        assert torch.equal(fq, q) and torch.equal(fv, near)
        del fq, fv
    dw = torch.empty(d, dtype=dt, device="cuda")
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
    far = torch.empty(2 * stride + d, dtype=dt, device="cuda").as_strided((3, d), (stride, 1))
    zg.zero_rms_backward(p, y, None, v, None, rstd, far, dw, ws)
    want = rstd.double()[:, None] * (y.double() - x.double() * rstd.double()[:, None] * (y.double() * x.double() * rstd.double()[:, None]).mean(1, keepdim=True))
    mag = rstd.double()[:, None] * y.double().abs()
    assert bool(((far.double() - want).abs() <= want.abs() * _half(dt) * 1.001 + U * (_chain(d) + 100) * mag + U).all())


def test_streams_graphs_and_repeats():
    s = _setup(300, 771, "bf16", 5, 5)
    p, st = s["plan"], torch.cuda.Stream()
    dy = torch.randn(300, 776, device="cuda").bfloat16()[:, :771]
    dx, dw = torch.empty(300, 776, device="cuda", dtype=torch.bfloat16)[:, :771], torch.empty(771, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")

    def both(stream):
        zg.zero_rms_forward(p, s["x"].v, s["r"].v, s["w"], EPS, s["h"].v, s["y"].v, None, None, s["rstd"], stream)
        zg.zero_rms_backward(p, dy, None, s["h"].v, s["w"], s["rstd"], dx, dw, ws, stream)

    both(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [t.clone() for t in (s["y"].v, dx, dw)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        both(st)
        st.synchronize()
        with torch.cuda.graph(graph, stream=st):
            both(torch.cuda.current_stream())
    for t in (s["y"].v, dx, dw):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((s["y"].v, dx, dw), want))


def test_two_streams_at_once():
    """Calls with workspaces of their own, at the same time."""
    jobs = []
    for k in range(2):
        s = _setup(2000, 1600, "fp16", seed=k)
        dy = torch.randn(2000, 1600, device="cuda").half()
        out = [torch.empty(2000, 1600, device="cuda", dtype=torch.float16), torch.empty(1600, device="cuda", dtype=torch.float16)]
        jobs.append((s, dy, out, torch.empty(s["plan"].workspace_bytes, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    results = []
    for turn in range(2):
        for s, dy, out, ws, st in jobs:
            stream = torch.cuda.current_stream() if turn == 0 else st
            for _ in range(1 if turn == 0 else 20):
                zg.zero_rms_forward(s["plan"], s["x"].v, s["r"].v, s["w"], EPS, s["h"].v, s["y"].v, None, None, s["rstd"], stream)
                zg.zero_rms_backward(s["plan"], dy, None, s["h"].v, s["w"], s["rstd"], out[0], out[1], ws, stream)
        torch.cuda.synchronize()
        results.append([t.clone() for s, _, out, _, _ in jobs for t in (s["y"].v, *out)])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("d", [16, 31, 64, 120, 128, 136, 300, 771, 1024, 2040, 4096, 4100, 8192, 8200, 12_289, 16_384, 16_392, 33_000, 40_001])
def test_same_bits_wherever_rows_start(d, dtype):
    """Small multiples of powers of two, whose sums are exact in every order: rows on 16-byte boundaries, and the same rows off them, come out
    with equal bits.  Squares: multiples of 1/4 up to 16, 40001 of them below 2^24 / 4; dy w xhat: multiples of 1/8 up to 3/2."""
    n, stride = 37, (d + 15) // 16 * 16
    code, dt = DT[dtype]
    g = torch.Generator(device="cuda").manual_seed(d)
    k = lambda lo, hi, unit, *size: (torch.randint(lo, hi + 1, size, device="cuda", generator=g) * unit).to(dt)  # noqa: E731
    x, r, dy, dh, w = k(-4, 4, 0.5, n, d), k(-4, 4, 0.5, n, d), k(-1, 1, 1.0, n, d), k(-8, 8, 0.25, n, d), k(1, 3, 0.5, d)
    given = torch.exp2(torch.randint(-1, 1, (n,), device="cuda", generator=g).float())
    out = []
    for shift in (0, 1):
        p = zg.zero_rms_plan(n, d, code, stride, stride, 32)
        a, b, gy, gh = (Rows(n, d, stride, shift, dt, v) for v in (x, r, dy, dh))
        h, y, dx, plain = (Rows(n, d, stride, shift, dt) for _ in range(4))
        q, vals = Rows(n, d, stride, shift, torch.uint8, guard=0xA5), Rows(n, d, stride, shift, torch.bfloat16)
        sc = torch.empty(n, p.scale_cols, dtype=torch.uint8, device="cuda")
        rstd, dw = torch.empty(n, device="cuda"), torch.empty(d, dtype=dt, device="cuda")
        ws = torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda")
        assert (a.v.data_ptr() % 16 == 0) == (shift == 0)
        zg.zero_rms_forward(p, a.v, b.v, w, EPS, h.v, y.v, q.v, sc, rstd)
        zg.zero_rms_values(p, q.v, sc, vals.v)
        zg.zero_rms_backward(p, gy.v, gh.v, h.v, w, given, dx.v, dw, ws)
        zg.zero_rms_backward(p, gy.v, None, h.v, w, given, plain.v, None, None)
        assert all(t.kept() for t in (h, y, q, vals, dx, plain))
        out.append([t.v.clone() for t in (h, y, q, vals, dx, plain)] + [sc, rstd, dw])
    for name, a, b in zip(("h", "y", "q", "values", "dx", "dx without dh", "scales", "rstd", "dw"), *out):
        assert torch.equal(a, b), name


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("d", [1000, 9000, 20_000])
def test_gradients_of_rows_past_32_bits(d, odd, dtype):
    """h, dy, dh and dx with rows 2^31 values apart: dx and dw have the bits of the same rows side by side."""
    code, dt = DT[dtype]
    far, near = (1 << 31) + (16 if dtype == "bf16" else 4) + odd, (d + 15) // 16 * 16 + odd
    g = torch.Generator(device="cuda").manual_seed(d)
    value = [torch.randn(3, d, device="cuda", generator=g).to(dt) for _ in range(3)]
    w, rstd = torch.randn(d, device="cuda", generator=g).to(dt), torch.rand(3, device="cuda", generator=g) + 0.5
    out = []
    for stride in (near, far):
        p = zg.zero_rms_plan(3, d, code, stride, stride)
        h, dy, dx = (torch.empty(2 * stride + d, dtype=dt, device="cuda").as_strided((3, d), (stride, 1)) for _ in range(3))
        h.copy_(value[0])
        dy.copy_(value[1])
        dx.copy_(value[2])                            # dh is written over
        dw = torch.empty(d, dtype=dt, device="cuda")
        zg.zero_rms_backward(p, dy, dx, h, w, rstd, dx, dw, torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda"))
        out.append((dx.clone(memory_format=torch.contiguous_format), dw))
        del h, dy, dx
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    dw64 = (value[1].double() * value[0].double() * rstd.double()[:, None]).sum(0)
    mag = (value[1].double() * value[0].double() * rstd.double()[:, None]).abs().sum(0)
    assert bool(((out[1][1].double() - dw64).abs() <= dw64.abs() * _half(dt) * 1.001 + U * mag * 70).all())
