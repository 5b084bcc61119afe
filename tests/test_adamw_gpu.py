"""The list-of-tensors AdamW step on the GPU.

Binary32 moments: bit for bit against the CPU oracle of the sharded step (the
decay applied to the weights first), and against the formula in 64 bits.
8-bit moments: bit for bit against a binary32 restatement in numpy (IEEE
operations in the documented order), and the stored values against the
formula in 64 bits -- always a neighbouring code, right on average."""
import numpy as np
import pytest
import torch

import oracle
import zero_sharded_mixed_bucket_gb300 as zg

pytestmark = pytest.mark.gpu

DT = {"fp16": (zg.ZERO_FP16, torch.float16, oracle.FP16), "bf16": (zg.ZERO_BF16, torch.bfloat16, oracle.BF16),
      "fp32": (zg.ZERO_FP32, torch.float32, oracle.FP32)}
F = np.float32
GUARD8, GUARDF = 0xA5, -77.0


def _bits(t):
    return t.detach().cpu().contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16).numpy()


class Tensors:
    """A list of tensors, each in guarded buffers `shift` values off a 16-byte boundary."""

    def __init__(self, sizes, dtype, bits, seed=0, shifts=(0,), decay=(0.1, 0.0), param=True, scale=1.0):
        rng = np.random.default_rng(seed)
        self.sizes, self.bits, self.dtype = sizes, bits, dtype
        self.code, dt, self.odt = DT[dtype]
        self.full, self.view, self.rec = [], [], []
        self.decay = [F(decay[k % len(decay)]) for k in range(len(sizes))]
        for k, n in enumerate(sizes):
            shift = shifts[k % len(shifts)]
            full, view = {}, {}

            def put(name, values, kind):
                t = torch.full((n + 64 + shift,), GUARD8 if kind == torch.uint8 else GUARDF, dtype=kind, device="cuda")
                t[32 + shift:32 + shift + n] = torch.from_numpy(values).to("cuda").to(kind)
                full[name], view[name] = t, t[32 + shift:32 + shift + n]

            mag = (10.0 ** rng.uniform(-4, 0, n)).astype(F) * F(scale)
            put("grad", rng.standard_normal(n).astype(F) * mag, dt)
            put("master", rng.standard_normal(n).astype(F) * F(0.02), torch.float32)
            if param:
                put("param", np.zeros(n, F), dt)
            if bits == 32:
                put("m", rng.standard_normal(n).astype(F) * F(1e-3), torch.float32)
                put("v", rng.random(n).astype(F) * F(1e-5), torch.float32)
            else:
                nb = -(-n // 256)
                put("m", rng.integers(0, 256, n).astype(np.uint8), torch.uint8)
                put("v", rng.integers(0, 256, n).astype(np.uint8), torch.uint8)
                for q in ("m_scale", "v_scale"):
                    t = torch.full((nb + 64,), GUARD8, dtype=torch.uint8, device="cuda")
                    t[32:32 + nb] = torch.from_numpy(rng.integers(108, 118, nb).astype(np.uint8)).to("cuda")
                    full[q], view[q] = t, t[32:32 + nb]
            self.full.append(full)
            self.view.append(view)
            self.rec.append(zg.adamw_tensor(numel=n, weight_decay=float(self.decay[k]), **view))
        self.plan = zg.zero_adamw_plan(self.rec, self.code, bits)
        self.table = torch.empty(max(self.plan.table_bytes, 16), dtype=torch.uint8, device="cuda")
        zg.zero_adamw_table_init(self.plan, self.rec, self.table, torch.cuda.current_stream())
        self.starts = np.concatenate([[0], np.cumsum([-(-n // 256) * 256 for n in sizes])]).astype(np.int64)

    def host(self, k, name):
        t = self.view[k][name]
        return t.float().cpu().numpy() if t.dtype != torch.uint8 else t.cpu().numpy()

    def guards_kept(self):
        for full, view in zip(self.full, self.view):
            for name, t in full.items():
                keep = torch.ones_like(t, dtype=torch.bool)
                a = view[name].storage_offset()
                keep[a:a + view[name].numel()] = False
                if not bool((t[keep] == (GUARD8 if t.dtype == torch.uint8 else GUARDF)).all()):
                    return False
        return True


def _hp(**k):
    d = {"t": 3, "lr": 1e-2, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "grad_scale": 0.125, "seed": 77}
    d.update(k)
    return zg.zero_adamw_t(**d)


def _keep(hp, decay):
    return F(1.0 - float(F(hp.lr)) * float(decay))


SIZES = [[1], [7], [4096], [4097], [0, 5, 0, 8192 + 3, 256], [255, 256, 257, 1, 12_345], [3] * 70, [100_003, 2, 640]]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shifts", [(0,), (1, 0, 3)])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_binary32_moments(sizes, shifts, dtype):
    T = Tensors(sizes, dtype, 32, seed=len(sizes), shifts=shifts)
    old = [{n: T.host(k, n) for n in T.view[k]} for k in range(len(sizes))]
    hp = _hp()
    zg.zero_adamw_step(T.plan, T.table, hp, None, torch.cuda.current_stream())
    torch.cuda.synchronize()
    for k, n in enumerate(sizes):
        if n == 0:
            continue
        o = old[k]
        w, m, v = (o["master"] * _keep(hp, T.decay[k])).copy(), o["m"].copy(), o["v"].copy()
        g = T.view[k]["grad"].cpu()
        g = g.numpy().view(np.uint32) if dtype == "fp32" else g.view(torch.int16).numpy().view(np.uint16)
        ref = oracle.step([np.ascontiguousarray(g)], w, m, v, dtype=T.odt, lr=hp.lr, beta1=hp.beta1, beta2=hp.beta2,
                          eps=hp.eps, t=hp.t - 1, loss_scale=8.0)
        for name, want in (("master", w), ("m", m), ("v", v)):
            assert np.array_equal(_bits(T.view[k][name]), want.view(np.int32)), (k, name)
        p = T.view[k]["param"]
        assert np.array_equal(_bits(p).view(np.uint32 if dtype == "fp32" else np.uint16), ref["p16"]), (k, "param")
        # the formula in 64 bits: a dozen binary32 roundings, of the weight and of the update
        g64 = o["grad"].astype(np.float64) * 0.125
        b1, b2 = float(F(hp.beta1)), float(F(hp.beta2))
        m64 = b1 * o["m"].astype(np.float64) + (1 - b1) * g64
        v64 = b2 * o["v"].astype(np.float64) + (1 - b2) * g64 * g64
        step = float(F(hp.lr)) * (m64 / (1 - b1 ** 3)) / (np.sqrt(v64 / (1 - b2 ** 3)) + float(F(hp.eps)))
        w64 = o["master"].astype(np.float64) * (1 - float(F(hp.lr)) * float(T.decay[k])) - step
        mag = float(F(hp.lr)) * ((b1 * np.abs(o["m"]) + (1 - b1) * np.abs(g64)) / (1 - b1 ** 3)) / (np.sqrt(v64 / (1 - b2 ** 3)))
        assert (np.abs(T.host(k, "master") - w64) <= 2.0 ** -24 * (3 * np.abs(o["master"]) + 3 * np.abs(w64) + 12 * mag)).all()
    assert T.guards_kept()


# ---- 8-bit moments: a binary32 restatement ------------------------------------------
def _value(code, least):
    """Magnitude codes relative to the scale (float64, exact): least = -exponent of the least normal."""
    e, f = code >> 4, (code & 15) / 16.0
    return np.where(e == 0, f * 2.0 ** -least, (1 + f) * 2.0 ** (e.astype(np.float64) - 1 - least))


def _unpack(o):
    s = lambda q: np.repeat(2.0 ** (o[q].astype(np.float64) - 127), 256)[:o["m"].size]  # noqa: E731
    m = _value(o["m"] & 127, 6) * s("m_scale") * np.where(o["m"] > 127, -1.0, 1.0)
    return m.astype(F), (_value(o["v"], 14) * s("v_scale")).astype(F)


def _random(n, start, hp):
    i = np.arange(start, start + n, dtype=np.uint64)
    j, u = i >> np.uint64(1), np.uint64(0xFFFFFFFF)
    k = lambda x: np.uint64(x)  # noqa: E731
    h = ((j & u) * k(0x9E3779B1) + (j >> k(32)) * k(0x6A09E667) + k((hp.seed + hp.t * 0x510E527F) & 0xFFFFFFFF)) & u
    h = ((h ^ (h >> k(15))) * k(0xBB67AE85)) & u
    h = ((h ^ (h >> k(15))) * k(0xA54FF53B)) & u
    h ^= h >> k(16)
    return np.where(i & k(1), h >> k(16), h & k(0xFFFF)).astype(np.int64)


def _codes(x, rnd, least, most, floor):
    """Stochastic codes and scale bytes of x >= 0 (binary32), by exact integer arithmetic on a 2^-(least+23) grid."""
    n = x.size
    b = np.zeros(-(-n // 256) * 256, F)
    b[:n] = x
    e = np.minimum((b.view(np.int32).reshape(-1, 256).max(1) + (1 << 19)) >> 23, 253)
    y = (x.astype(np.float64) * np.repeat(2.0 ** (127.0 - e), 256)[:n]).astype(F)
    base = F(2.0 ** -least)
    low = y < base
    bits = np.where(low, y + base, y).astype(F).view(np.int32).astype(np.int64)
    c = ((bits + rnd * 8) >> 19) - (127 - least) * 16 + np.where(low, 0, 16)
    c = np.minimum(c, most)
    return (np.maximum(c, (x > 0).astype(np.int64)) if floor else c), e


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("shifts", [(0,), (1, 0, 3)])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_8bit_moments(sizes, shifts, dtype):
    T = Tensors(sizes, dtype, 8, seed=len(sizes) + 1, shifts=shifts)
    old = [{n: T.host(k, n) for n in T.view[k]} for k in range(len(sizes))]
    hp = _hp(t=12)
    zg.zero_adamw_step(T.plan, T.table, hp, None, torch.cuda.current_stream())
    torch.cuda.synchronize()
    b1, b2 = F(hp.beta1), F(hp.beta2)
    bc1, bc2 = 1 - float(b1) ** 12, 1 - float(b2) ** 12
    for k, n in enumerate(sizes):
        if n == 0:
            continue
        o = old[k]
        g = o["grad"] * F(0.125)
        m0, r0 = _unpack(o)
        m = m0 * b1 + g * (F(1) - b1)
        r = np.sqrt((r0 * r0) * b2 + (g * g) * (F(1) - b2))
        w = o["master"] * _keep(hp, T.decay[k]) - (m * F(float(F(hp.lr)) / bc1)) / (r * F(1 / np.sqrt(bc2)) + F(hp.eps))
        assert w.dtype == F
        rnd = _random(n, int(T.starts[k]), hp)
        cm, em = _codes(np.abs(m), rnd, 6, 127, False)
        cr, er = _codes(r, rnd, 14, 255, True)
        cm = cm + np.where((m < 0) & (cm > 0), 128, 0)
        assert np.array_equal(T.host(k, "m_scale"), em) and np.array_equal(T.host(k, "v_scale"), er)
        assert np.array_equal(T.host(k, "m"), cm) and np.array_equal(T.host(k, "v"), cr)
        assert np.array_equal(_bits(T.view[k]["master"]), w.view(np.int32))
        assert torch.equal(T.view[k]["param"].cpu(), torch.from_numpy(w).to(DT[dtype][1]))
        # against 64 bits: the stored value is a neighbour of the exact one (codes
        # are 1/16 of a binade apart at most; below the least normal evenly
        # spaced; the largest code is 1.9375)
        g64 = o["grad"].astype(np.float64) * 0.125
        m64 = float(b1) * m0.astype(np.float64) + (1 - float(b1)) * g64
        r64 = np.sqrt(float(b2) * r0.astype(np.float64) ** 2 + (1 - float(b2)) * g64 ** 2)
        st = {q: T.host(k, q) for q in ("m", "v", "m_scale", "v_scale")}
        ms, rs = (x.astype(np.float64) for x in _unpack(st))
        for got, want, e, least in ((ms, m64, em, 6), (rs, r64, er, 14)):
            unit = np.repeat(2.0 ** (e - 127.0), 256)[:n]
            gap = 2.0 ** np.floor(np.log2(np.maximum(np.abs(want) / unit, 2.0 ** -least))) / 16 * unit
            assert (np.abs(got - want) <= gap * (1 + 1e-5) + 1e-6 * np.abs(want)).all()
            assert (np.abs(want) <= 1.9375 * unit * (1 + 1e-6)).all()
    # read out: the same values, exactly
    flat = [torch.full((T.plan.flat_elems,), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    zg.zero_adamw_states(T.plan, T.table, flat[0], flat[1])
    for k, n in enumerate(sizes):
        a = int(T.starts[k])
        want = _unpack({q: T.host(k, q) for q in ("m", "v", "m_scale", "v_scale")}) if n else (np.zeros(0, F),) * 2
        for t, x in zip(flat, want):
            assert np.array_equal(t[a:a + n].float().cpu().numpy(), x)
            assert bool((t[a + n:int(T.starts[k + 1])] == 9.0).all())
    assert T.guards_kept()


def test_rounding_is_right_on_average():
    """Over 400 seeds the mean stored moment equals the exact one: the error of
    the mean of S bounded steps of size <= gap has a deviation below
    gap / (2 sqrt(S)); 6 deviations, over 2000 values."""
    n, S = 2000, 400
    sums = [np.zeros(n), np.zeros(n)]
    for s in range(S):
        T = Tensors([n], "fp32", 8, seed=5)
        if s == 0:
            o = {q: T.host(0, q) for q in T.view[0]}
        zg.zero_adamw_step(T.plan, T.table, _hp(seed=s * 7919, t=1 + s % 5))
        for acc, x in zip(sums, _unpack({q: T.host(0, q) for q in ("m", "v", "m_scale", "v_scale")})):
            acc += x
    st = {q: T.host(0, q) for q in ("m_scale", "v_scale")}
    b1, b2 = float(F(0.9)), float(F(0.999))
    m0, r0 = (x.astype(np.float64) for x in _unpack(o))
    g = o["grad"].astype(np.float64) * 0.125
    for acc, want, q, least in ((sums[0], b1 * m0 + (1 - b1) * g, "m_scale", 6),
                                (sums[1], np.sqrt(b2 * r0 * r0 + (1 - b2) * g * g), "v_scale", 14)):
        unit = np.repeat(2.0 ** (st[q] - 127.0), 256)[:n]
        y = np.abs(want) / unit
        gap = 2.0 ** np.floor(np.log2(np.maximum(y, 2.0 ** -least))) / 16 * unit
        inside = y >= (2.0 ** -18 if least == 14 else 0)   # a nonzero r below the least code is stored as that code
        off = np.abs(acc / S - want)[inside]
        assert (off <= (6 * gap / (2 * np.sqrt(S)) + 1e-5 * np.abs(want))[inside]).all()


def test_zero_blocks_zero_gradients_and_nonzero_roots():
    T = Tensors([600], "fp32", 8, seed=2)
    v = T.view[0]
    v["grad"].zero_()
    v["m"].zero_()
    v["v"].zero_()
    w = v["master"].clone()
    hp = _hp()
    zg.zero_adamw_step(T.plan, T.table, hp)
    assert not v["m"].any() and not v["v"].any() and not v["m_scale"].any() and not v["v_scale"].any()
    assert torch.equal(v["master"], w * float(_keep(hp, T.decay[0])))     # 0 / (0 + eps): only the decay
    # one large and one tiny gradient in a block: the tiny one's root is not stored as zero
    v["grad"][0], v["grad"][1] = 1e4, 1e-9
    zg.zero_adamw_step(T.plan, T.table, hp)
    assert v["v"][1] == 1 and v["v"][0] > 200 and v["v"][2] == 0


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("dtype", list(DT))
def test_check_and_skip(bits, dtype):
    T = Tensors([5000, 3, 300, 1], dtype, bits, shifts=(0, 1))
    flag = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    zg.zero_adamw_check(T.plan, T.table, flag)
    assert flag.item() == 0
    for k, at, bad in ((0, 4999, float("nan")), (1, 2, float("inf")), (3, 0, -float("inf"))):
        keep = T.view[k]["grad"][at].clone()
        T.view[k]["grad"][at] = bad
        zg.zero_adamw_check(T.plan, T.table, flag)
        assert flag.item() == 1
        before = [{n: t.clone() for n, t in f.items()} for f in T.full]
        zg.zero_adamw_step(T.plan, T.table, _hp(), flag)
        for f, b in zip(T.full, before):
            for n in f:
                assert torch.equal(f[n].view(torch.uint8), b[n].view(torch.uint8))
        T.view[k]["grad"][at] = keep
    zg.zero_adamw_check(T.plan, T.table, flag)
    w = T.view[0]["master"].clone()
    zg.zero_adamw_step(T.plan, T.table, _hp(), flag)
    assert flag.item() == 0 and not torch.equal(w, T.view[0]["master"])


def test_same_bits_each_time_and_without_parameters():
    out = []
    for _ in range(2):
        T = Tensors([70_000, 9], "bf16", 8, seed=3, param=False)
        for t in range(1, 4):
            zg.zero_adamw_step(T.plan, T.table, _hp(t=t))
        out.append(T)
    for a, b in zip(out[0].full, out[1].full):
        for n in a:
            assert torch.equal(a[n], b[n])
    assert out[0].guards_kept()


def test_8bit_moments_follow_a_decaying_gradient():
    """sqrt(v) must come down when gradients do, although a step moves it by
    less than a code's spacing: after 3000 steps of gradients 100 times
    smaller, beta2 = 0.999 leaves 5 % of the old v."""
    n = 4096
    T = Tensors([n], "fp32", 8, seed=1, decay=(0.0,))
    v = T.view[0]
    for name in ("m", "v", "m_scale", "v_scale"):
        v[name].zero_()
    v["grad"].fill_(1.0)
    t = 0
    for t in range(1, 1001):
        zg.zero_adamw_step(T.plan, T.table, _hp(t=t, grad_scale=1.0, lr=0.0))
    r0 = _unpack({q: T.host(0, q) for q in ("m", "v", "m_scale", "v_scale")})[1].mean()
    want0 = np.sqrt(1 - 0.999 ** 1000)
    assert abs(r0 - want0) < 0.05 * want0
    v["grad"].fill_(0.01)
    for t in range(1001, 4001):
        zg.zero_adamw_step(T.plan, T.table, _hp(t=t, grad_scale=1.0, lr=0.0))
    r1 = _unpack({q: T.host(0, q) for q in ("m", "v", "m_scale", "v_scale")})[1].astype(np.float64)
    want1 = np.sqrt((1 - 0.999 ** 1000) * 0.999 ** 3000 + 1e-4 * (1 - 0.999 ** 3000))
    # rounding up or down with the right chance adds a random walk: each step's
    # variance is at most (move per step) * gap, so v's relative excess stays below
    # gap^2-sized terms, a few percent, and the mean over 4096 values is tight
    assert abs(np.sqrt((r1 ** 2).mean()) - want1) < 0.1 * want1


@pytest.mark.parametrize("bits", [8, 32])
def test_offsets_past_32_bits(bits):
    """A tensor of 2^33 + 777 values: the values around 2^32 and at the end as in
    a short list (8 bits: with the same random numbers, which go by a value's
    place)."""
    n, zero = 2 ** 33 + 777, torch.uint8 if bits == 8 else torch.float32
    if bits == 32:
        n = 2 ** 32 + 777
    grad = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    master = torch.zeros(n, device="cuda")
    m, v = (torch.zeros(n, dtype=zero, device="cuda") for _ in range(2))
    sc = [torch.zeros(-(-n // 256), dtype=torch.uint8, device="cuda") for _ in range(2)] if bits == 8 else [None, None]
    g = torch.Generator(device="cuda").manual_seed(0)
    marks = [2 ** 32 - 512, (n - 1500) // 256 * 256]
    for a in marks:
        k = min(1024, n - a)
        grad[a:a + k] = torch.randn(k, device="cuda", generator=g).bfloat16()
        master[a:a + k] = torch.randn(k, device="cuda", generator=g)
    old = [(grad[a:a + 1024].float().cpu().numpy(), master[a:a + 1024].cpu().numpy()) for a in marks]
    rec = [zg.adamw_tensor(grad=grad, master=master, m=m, v=v, numel=n, m_scale=sc[0], v_scale=sc[1])]
    plan = zg.zero_adamw_plan(rec, zg.ZERO_BF16, bits)
    table = torch.empty(plan.table_bytes, dtype=torch.uint8, device="cuda")
    zg.zero_adamw_table_init(plan, rec, table)
    hp = _hp(t=1, grad_scale=1.0)
    zg.zero_adamw_step(plan, table, hp)
    b1, b2 = F(hp.beta1), F(hp.beta2)
    for a, (g0, w0) in zip(marks, old):
        k = g0.size
        m1, v1 = g0 * (F(1) - b1), (g0 * g0) * (F(1) - b2)
        if bits == 32:
            assert np.array_equal(m[a:a + k].cpu().numpy(), m1) and np.array_equal(v[a:a + k].cpu().numpy(), v1)
            continue
        r1 = np.sqrt(v1)
        w1 = w0 - (m1 * F(float(F(hp.lr)) / (1 - float(b1)))) / (r1 * F(1 / np.sqrt(1 - float(b2))) + F(hp.eps))
        rnd = _random(k, a, hp)
        cm, em = _codes(np.abs(m1), rnd, 6, 127, False)
        cr, er = _codes(r1, rnd, 14, 255, True)
        assert np.array_equal(m[a:a + k].cpu().numpy(), cm + np.where((m1 < 0) & (cm > 0), 128, 0))
        assert np.array_equal(v[a:a + k].cpu().numpy(), cr)
        assert np.array_equal(master[a:a + k].cpu().numpy(), w1)
        assert np.array_equal(sc[0][a // 256:a // 256 + em.size].cpu().numpy(), em)
    del grad, master, m, v, sc
    torch.cuda.empty_cache()


def _step8(T, hp):
    """The 8-bit step of a list in binary32 (t = hp.t), compared with the kernel's bit for bit."""
    old = [{n: T.host(k, n) for n in T.view[k]} for k in range(len(T.sizes))]
    zg.zero_adamw_step(T.plan, T.table, hp)
    b1, b2 = F(hp.beta1), F(hp.beta2)
    bc1, bc2 = 1 - float(b1) ** hp.t, 1 - float(b2) ** hp.t
    with np.errstate(all="ignore"):
        for k, n in enumerate(T.sizes):
            o = old[k]
            g = o["grad"] * F(hp.grad_scale)
            m0, r0 = _unpack(o)
            m = m0 * b1 + g * (F(1) - b1)
            r = np.sqrt((r0 * r0) * b2 + (g * g) * (F(1) - b2))
            w = o["master"] * _keep(hp, T.decay[k]) - (m * F(float(F(hp.lr)) / bc1)) / (r * F(1 / np.sqrt(bc2)) + F(hp.eps))
            rnd = _random(n, int(T.starts[k]), hp)
            cm, em = _codes(np.abs(m), rnd, 6, 127, False)
            cr, er = _codes(r, rnd, 14, 255, True)
            cm = cm + np.where((m < 0) & (cm > 0), 128, 0)
            assert np.array_equal(T.host(k, "m_scale"), em) and np.array_equal(T.host(k, "v_scale"), er)
            assert np.array_equal(T.host(k, "m"), cm) and np.array_equal(T.host(k, "v"), cr)
            assert np.array_equal(T.host(k, "master"), w, equal_nan=True)


@pytest.mark.parametrize("shifts", [(0,), (1,)])
def test_8bit_scales_of_the_whole_range(shifts):
    """Blocks of every scale byte, gradients from 1e-20 to 1e18: those whose
    decoding or encoding takes two factors, and the last scale, which cuts."""
    n = 253 * 256 * 3 - 100
    T = Tensors([n], "fp32", 8, seed=9, shifts=shifts)
    v, rng = T.view[0], np.random.default_rng(10)
    nb = v["m_scale"].numel()
    v["m_scale"].copy_(torch.from_numpy((1 + np.arange(nb) % 253).astype(np.uint8)))
    v["v_scale"].copy_(torch.from_numpy((1 + rng.permutation(nb) % 253).astype(np.uint8)))
    size = np.repeat(10.0 ** rng.uniform(-20, 18, nb), 256)[:n] * (np.repeat(rng.random(nb), 256)[:n] < 0.7)
    v["grad"].copy_(torch.from_numpy((rng.standard_normal(n) * size).astype(F)))
    for t in (5, 6):
        _step8(T, _hp(t=t))
        out = [torch.zeros(T.plan.flat_elems, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        zg.zero_adamw_states(T.plan, T.table, *out)
        for got, want in zip(out, _unpack({q: T.host(0, q) for q in ("m", "v", "m_scale", "v_scale")})):
            got = got[:n].float().cpu().numpy()
            normal = np.abs(want) >= 2.0 ** -126
            assert np.array_equal(got[normal], want[normal])
            assert (np.abs(got - want) < 2.0 ** -133).all()          # bfloat16's subnormals
    assert T.guards_kept()
    big = T.host(0, "m_scale") > 133
    assert big.any() and (T.host(0, "v_scale") > 141).any() and (T.host(0, "v_scale") == 253).any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_8bit_block_of_a_nonfinite_gradient(bad):
    """A NaN or infinity that is not checked for takes its block of 256 with it:
    the last scale, the largest codes at the value, the least nonzero root
    beside it; the neighbouring blocks are what they are without."""
    T, clean = Tensors([1000], "fp32", 8, seed=11), Tensors([1000], "fp32", 8, seed=11)
    T.view[0]["grad"][300] = bad
    _step8(T, _hp())
    zg.zero_adamw_step(clean.plan, clean.table, _hp())
    v, c = T.view[0], clean.view[0]
    assert v["m_scale"][1] == 253 and v["v_scale"][1] == 253
    assert v["m"][300] == (255 if bad < 0 else 127) and v["v"][300] == 255 and not v["master"][300].isfinite()
    keep = torch.ones(1000, dtype=torch.bool)
    keep[256:512] = False
    for q in ("m", "v", "master", "param"):
        assert torch.equal(v[q][keep.cuda()], c[q][keep.cuda()])
    assert not v["m"][301:512].any() and (v["v"][301:512] == 1).all()
    rest = torch.arange(1000) != 300
    assert torch.equal(v["master"][rest.cuda()], c["master"][rest.cuda()])


def test_binary32_weights_past_32_bits():
    """The weights, too, of values around 2^32 in one tensor."""
    n = 2 ** 32 + 2000
    grad, master = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    marks = [2 ** 31 - 512, 2 ** 32 - 512, n - 1024]
    g = torch.Generator(device="cuda").manual_seed(0)
    for a in marks:
        grad[a:a + 1024] = torch.randn(1024, device="cuda", generator=g).bfloat16()
        master[a:a + 1024] = torch.randn(1024, device="cuda", generator=g)
    g0, w0 = ([t[a:a + 1024].clone() for a in marks] for t in (grad, master))
    rec = [zg.adamw_tensor(grad=grad, master=master, m=m, v=v, numel=n, weight_decay=0.1)]
    plan = zg.zero_adamw_plan(rec, zg.ZERO_BF16, 32)
    table = torch.empty(plan.table_bytes, dtype=torch.uint8, device="cuda")
    zg.zero_adamw_table_init(plan, rec, table)
    zg.zero_adamw_step(plan, table, _hp(t=1, grad_scale=1.0))
    # the same values as a short list
    for k, a in enumerate(marks):
        ts = {"grad": g0[k], "master": w0[k].clone(), "m": torch.zeros(1024, device="cuda"), "v": torch.zeros(1024, device="cuda")}
        r = [zg.adamw_tensor(numel=1024, weight_decay=0.1, **ts)]
        p = zg.zero_adamw_plan(r, zg.ZERO_BF16, 32)
        tab = torch.empty(p.table_bytes, dtype=torch.uint8, device="cuda")
        zg.zero_adamw_table_init(p, r, tab)
        zg.zero_adamw_step(p, tab, _hp(t=1, grad_scale=1.0))
        for q, big in (("master", master), ("m", m), ("v", v)):
            assert torch.equal(ts[q], big[a:a + 1024]), (k, q)
        assert not torch.equal(ts["master"], w0[k])
    del grad, master, m, v
    torch.cuda.empty_cache()
