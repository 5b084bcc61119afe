"""The training-end operators: what is timed, the plain forms, and the definitions in 64 bits.

Three operators that sit between a transformer's last block and the sharded
optimizer state, on sizes of the parameter lists this repository benchmarks
(a 50257-row embedding; d = 768, 1600 and 4096; 12 and 48 layers):

  ln        layer norm of rows, forward, and backward with the reduction of
            the weight's and the bias's gradient
  ce        softmax cross entropy of x W^T over a large vocabulary, loss only
            or loss with the gradients of x and W
  adamw     one AdamW step over a list of tensors, with the moments in 32
            bits or in 8 (the 8-bit form also reads its moments out, as a
            checkpoint does: what is stored is returned as the values it
            stands for)

`run` computes the plain form (elementary torch operations in 32 bits, rounded
once) unless `own` is set, when it calls this package's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5
IGNORE = -100


def f32(x):
    """The nearest binary32 value."""
    return float(np.float32(x))


def _esize(case):
    return 4 if case["dtype"] == "fp32" else 2


def _model_list(vocab, d, layers):
    """Parameter tensors of the benchmarked lists, embedding first: per layer 12 d^2 + 4 d values."""
    return [vocab * d] + [3 * d * d, d * d, 4 * d * d, 4 * d * d, d, d, d, d] * layers


# ---- cases --------------------------------------------------------------------
def listed():
    return [
        # one token of a d = 768 model: a single row, where only latency counts
        {"name": "ln_fwd_one_row", "op": "ln_fwd", "rows": 1, "dim": 768, "pad": 0, "dtype": "bf16"},
        # a training batch of 8192 tokens through a d = 4096 model's layer norm
        {"name": "ln_fwd_8192x4096", "op": "ln_fwd", "rows": 8192, "dim": 4096, "pad": 0, "dtype": "bf16"},
        # odd sizes and a padded row stride, fp32 training
        {"name": "ln_bwd_odd_fp32", "op": "ln_bwd", "rows": 1003, "dim": 771, "pad": 5, "dtype": "fp32"},
        # batch 32 x sequence 1024 x hidden 1600, the activation checkpoint this repository partitions
        {"name": "ln_bwd_32768x1600", "op": "ln_bwd", "rows": 32768, "dim": 1600, "pad": 0, "dtype": "fp16"},
        # scoring one token against the whole vocabulary (the weight is read once)
        {"name": "ce_loss_one_token", "op": "ce_fwd", "tokens": 1, "vocab": 50257, "hidden": 4096, "pad": 0, "dtype": "bf16"},
        # evaluating a ragged batch
        {"name": "ce_loss_1023", "op": "ce_fwd", "tokens": 1023, "vocab": 50257, "hidden": 1600, "pad": 0, "dtype": "fp16"},
        # a training step's loss and gradients, d = 768
        {"name": "ce_train_8192x768", "op": "ce_train", "tokens": 8192, "vocab": 50257, "hidden": 768, "pad": 0, "dtype": "bf16"},
        # the same at d = 4096: the largest product
        {"name": "ce_train_8192x4096", "op": "ce_train", "tokens": 8192, "vocab": 50257, "hidden": 4096, "pad": 0, "dtype": "bf16"},
        # the vectors of two layers alone: a few small tensors, latency
        {"name": "adamw32_vectors", "op": "adamw", "bits": 32, "list": "vectors", "dtype": "fp32"},
        # every tensor of the 12-layer d = 768 list
        {"name": "adamw32_12x768", "op": "adamw", "bits": 32, "list": "12x768", "dtype": "fp16"},
        {"name": "adamw8_12x768", "op": "adamw", "bits": 8, "list": "12x768", "dtype": "bf16"},
        # every tensor of the 48-layer d = 1600 list, 1.56e9 values
        {"name": "adamw8_48x1600", "op": "adamw", "bits": 8, "list": "48x1600", "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "ce_fwd", "ce_train", "adamw32", "adamw8"])
    if op.startswith("ln"):
        dim = _log(rng, 16, 16384)
        rows = _log(rng, 1, max(1, min(65536, 32768 * 1600 // dim)))
        return {"op": op, "rows": rows, "dim": dim, "pad": rng.choice([0, 0, 1, 8]),
                "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    if op.startswith("ce"):
        hidden = 8 * _log(rng, 8, 512)
        vocab = _log(rng, 2, 65536)
        tokens = _log(rng, 1, min(16384, 8192 * 50257 * 4096 // (hidden * vocab), (8192 * 50257) // vocab))
        return {"op": op, "tokens": tokens, "vocab": vocab, "hidden": hidden, "pad": rng.choice([0, 0, 8]),
                "dtype": rng.choice(["fp16", "bf16"])}
    count = _log(rng, 1, 300)
    return {"op": "adamw", "bits": 32 if op == "adamw32" else 8, "list": "drawn", "count": count,
            "most": _log(rng, 8, 2_000_000), "pick": rng.randrange(1 << 30), "dtype": rng.choice(["fp16", "bf16", "fp32"])}


def _numels(case):
    if case["list"] == "vectors":
        return [768] * 8
    if case["list"] == "12x768":
        return _model_list(50257, 768, 12)
    if case["list"] == "48x1600":
        return _model_list(50257, 1600, 48)
    g = torch.Generator().manual_seed(case["pick"])
    u = torch.rand(case["count"], generator=g, dtype=torch.float64)
    return [max(1, int(n)) for n in torch.exp(u * math.log(case["most"])).tolist()]


# ---- inputs -------------------------------------------------------------------
def _rows(g, n, width, pad, dtype, scale=1.0):
    """(n, width) values in a buffer whose rows are width + pad apart."""
    full = torch.zeros(n, width + pad, device="cuda", dtype=dtype)
    full[:, :width] = torch.randn(n, width, device="cuda", generator=g) * scale
    return full[:, :width]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"].startswith("ln"):
        n, d, pad = case["rows"], case["dim"], case["pad"]
        x = _rows(g, n, d, pad, dt, 2.0)
        x += 0.5 * torch.randn(d, device="cuda", generator=g).to(dt)       # channels have means of their own
        w = (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt)
        b = (0.1 * torch.randn(d, device="cuda", generator=g)).to(dt)
        s = {"case": case, "x": x, "w": w, "b": b}
        if case["op"] == "ln_bwd":
            s["dy"] = _rows(g, n, d, pad, dt)
            x32 = x.float()
            s["mean"] = x32.mean(1)
            s["rstd"] = torch.rsqrt(x32.var(1, unbiased=False) + EPS)
        if own:
            import zero_sharded_mixed_bucket_gb300 as zg
            s["zg"], s["plan"] = zg, zg.zero_ln_plan(n, d, _zdtype(zg, case), d + pad, d + pad)
            if case["op"] == "ln_fwd":
                s["out"] = [torch.empty_strided(x.shape, x.stride(), device="cuda", dtype=dt),
                            torch.empty(n, device="cuda"), torch.empty(n, device="cuda")]
            else:
                s["out"] = [torch.empty_strided(x.shape, x.stride(), device="cuda", dtype=dt),
                            torch.empty_like(w), torch.empty_like(b)]
            s["ws"] = torch.empty(s["plan"].workspace_bytes, device="cuda", dtype=torch.uint8)
        return s
    if case["op"].startswith("ce"):
        n, v, d, pad = case["tokens"], case["vocab"], case["hidden"], case["pad"]
        x = _rows(g, n, d, pad, dt)                                        # a layer norm's output
        w = _rows(g, v, d, pad, dt, 1.5 / math.sqrt(d))
        t = torch.randint(0, v, (n,), device="cuda", generator=g)
        t = torch.where(torch.rand(n, device="cuda", generator=g) < 0.1, IGNORE, t)  # padding tokens
        t[0] = v - 1
        s = {"case": case, "x": x, "w": w, "t": t, "scale": 1024.0}        # the loss scale of mixed precision
        if own:
            import zero_sharded_mixed_bucket_gb300 as zg
            s["zg"], s["plan"] = zg, zg.zero_ce_plan(n, v, d, _zdtype(zg, case), d + pad, d + pad)
            s["out"] = [torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(2, device="cuda")]
            if case["op"] == "ce_train":
                s["out"] += [torch.empty_strided(a.shape, a.stride(), device="cuda", dtype=dt) for a in (x, w)]
            s["ws"] = torch.empty(s["plan"].workspace_bytes, device="cuda", dtype=torch.uint8)
        return s
    sizes = _numels(case)
    starts, total = [], 0
    for k in sizes:                     # every tensor starts at a multiple of 256 values of the flat buffers
        starts.append(total)
        total += -(-k // 256) * 256
    used = torch.zeros(total, device="cuda", dtype=torch.bool)
    for a, k in zip(starts, sizes):
        used[a:a + k] = True
    f = {"master": torch.randn(total, device="cuda", generator=g).mul_(0.02).mul_(used)}
    f["grad"] = torch.randn(total, device="cuda", generator=g).mul_(1e-3 * 1024).mul_(used).to(dt)
    f["param"] = f["master"].to(dt)
    if case["bits"] == 32:
        f["m"] = torch.randn(total, device="cuda", generator=g).mul_(3e-4).mul_(used)
        f["v"] = torch.rand(total, device="cuda", generator=g).mul_(1e-6).mul_(used)
    else:
        f["m"] = torch.randint(0, 256, (total,), device="cuda", generator=g, dtype=torch.uint8).mul_(used)
        f["v"] = torch.randint(100, 256, (total,), device="cuda", generator=g, dtype=torch.uint8).mul_(used)
        f["m_scale"] = torch.randint(114, 118, (total // 256,), device="cuda", generator=g, dtype=torch.uint8)
        f["v_scale"] = torch.randint(116, 119, (total // 256,), device="cuda", generator=g, dtype=torch.uint8)
    decay = [0.1 if k > 16384 else 0.0 for k in sizes]                     # vectors are not decayed
    s = {"case": case, "flat": f, "sizes": sizes, "starts": starts, "decay": decay,
         "hp": {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "grad_scale": 1.0 / 1024, "t": 7, "seed": 20240229}}
    if own:
        import zero_sharded_mixed_bucket_gb300 as zg
        tensors = []
        for a, k, wd in zip(starts, sizes, decay):
            p = {n: f[n][a:] for n in ("grad", "param", "master", "m", "v")}
            if case["bits"] == 8:
                p.update({n: f[n][a // 256:] for n in ("m_scale", "v_scale")})
            tensors.append(zg.adamw_tensor(numel=k, weight_decay=wd, **p))
        s["zg"], s["plan"] = zg, zg.zero_adamw_plan(tensors, _zdtype(zg, case), case["bits"])
        s["table"] = torch.empty(s["plan"].table_bytes, device="cuda", dtype=torch.uint8)
        zg.zero_adamw_table_init(s["plan"], tensors, s["table"], torch.cuda.current_stream())
        s["own_hp"] = zg.zero_adamw_t(**s["hp"])
        if case["bits"] == 8:
            s["out"] = [torch.zeros(total, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    return s


def _zdtype(zg, case):
    return {"fp16": zg.ZERO_FP16, "bf16": zg.ZERO_BF16, "fp32": zg.ZERO_FP32}[case["dtype"]]


# ---- one pass -----------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"ln_fwd": _own_ln_fwd, "ln_bwd": _own_ln_bwd, "ce_fwd": _own_ce, "ce_train": _own_ce,
                "adamw": _own_adamw}[op](s)
    return {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "ce_fwd": _ce, "ce_train": _ce, "adamw": _adamw}[op](s)


def _own_ln_fwd(s):
    y, mean, rstd = s["out"]
    s["zg"].zero_ln_forward(s["plan"], s["x"], s["w"], s["b"], EPS, y, mean, rstd, torch.cuda.current_stream())
    return {"y": y, "mean": mean, "rstd": rstd}


def _own_ln_bwd(s):
    dx, dw, db = s["out"]
    s["zg"].zero_ln_backward(s["plan"], s["dy"], s["x"], s["w"], s["mean"], s["rstd"], dx, dw, db, s["ws"],
                             torch.cuda.current_stream())
    return {"dx": dx, "dw": dw, "db": db}


def _own_ce(s):
    loss, lse, total = s["out"][:3]
    st = torch.cuda.current_stream()
    s["zg"].zero_ce_forward(s["plan"], s["x"], s["w"], s["t"], loss, lse, total, s["ws"], st)
    r = {"loss": loss, "lse": lse, "mean": total[0]}
    if s["case"]["op"] == "ce_train":
        r["dx"], r["dw"] = s["out"][3:]
        s["zg"].zero_ce_backward(s["plan"], s["x"], s["w"], s["t"], lse, None, s["scale"], r["dx"], r["dw"], s["ws"], st)
    return r


def _own_adamw(s):
    zg, f, st = s["zg"], s["flat"], torch.cuda.current_stream()
    zg.zero_adamw_step(s["plan"], s["table"], s["own_hp"], None, st)
    r = {"master": f["master"], "param": f["param"]}
    if s["case"]["bits"] == 32:
        return {**r, "m": f["m"], "v": f["v"]}
    zg.zero_adamw_states(s["plan"], s["table"], s["out"][0], s["out"][1], st)
    return {**r, "m": s["out"][0], "root_v": s["out"][1]}


def _ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    y = c * rstd[:, None] * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _ln_bwd(s):
    xhat = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dy"].float()
    db, dw = dy.sum(0), (dy * xhat).sum(0)
    g = dy * s["w"].float()
    dx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    dt = s["x"].dtype
    return {"dx": dx.to(dt), "dw": dw.to(dt), "db": db.to(dt)}


def _ce(s):
    x, w, t = s["x"].float(), s["w"].float(), s["t"]
    counted = (t >= 0) & (t < w.shape[0])
    at = torch.where(counted, t, 0)[:, None]
    z = x @ w.t()
    top = z.max(1, keepdim=True).values
    lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
    loss = torch.where(counted, lse - z.gather(1, at)[:, 0], 0.0)
    n = counted.sum().clamp(min=1)
    r = {"loss": loss, "lse": lse, "mean": loss.sum() / n}
    if s["case"]["op"] == "ce_train":
        z = torch.exp(z - lse[:, None])
        z.scatter_add_(1, at, torch.full_like(at, -1, dtype=z.dtype))
        z *= (counted * (s["scale"] / n))[:, None]
        r["dx"], r["dw"] = (z @ w).to(s["x"].dtype), (z.t() @ x).to(s["x"].dtype)
    return r


# 8-bit moments.  A block of 256 values has a scale 2^(e-127), e the exponent
# field of its largest magnitude plus one code step (253 at most), so that the
# largest too can round up.  A magnitude y < 31/16, relative to it, is a float
# with four bits of fraction: m has a sign and three bits of exponent
# (least normal 2^-6), sqrt(v) has four (least normal 2^-14); below the least
# normal the codes are evenly spaced.  Rounding is stochastic, its 16 random
# bits hashed from the seed, the step and the value's place in the list.
def _hash16(n, start, mixed):
    """Random 16-bit numbers of values start .. start+n-1 (start even)."""
    i = torch.arange(start, start + n, device="cuda")
    j, u = i >> 1, 0xFFFFFFFF
    h = ((j & u) * 0x9E3779B1 + (j >> 32) * 0x6A09E667 + mixed) & u
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & u
    h = ((h ^ (h >> 15)) * 0xA54FF53B) & u
    h = h ^ (h >> 16)
    return torch.where((i & 1) == 1, h >> 16, h & 0xFFFF)


def _decode(code, least):
    """Values of magnitude codes, relative to the block's scale; least: exponent field of the least normal."""
    c = code.int()
    low = c < 16
    y = ((c + least * 16 - 16 * (~low).int()) << 19).view(torch.float32)
    return torch.where(low, y - 2.0 ** (least - 127), y)


def _encode(y, rnd, least, most):
    low = y < 2.0 ** (least - 127)
    bits = torch.where(low, y + 2.0 ** (least - 127), y).view(torch.int32)
    c = ((bits + (rnd << 3).int()) >> 19) - least * 16 + 16 * (~low).int()
    return c.clamp(max=most)


def _blocks(x, fill=0):
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % 256), value=fill).view(-1, 256)


def _power(e):
    """2^(e-127) for exponent fields 1..254, and 0 for 0."""
    return (e << 23).view(torch.float32)


def _block_scale(x):
    return ((_blocks(x).view(torch.int32).max(1).values + (1 << 19)) >> 23).clamp(max=253)


def _adamw_one(f, a, n, decay, h, bits):
    """The step on the tensor at [a, a + n) of the flat buffers, in place."""
    b1, b2 = f32(h["beta1"]), f32(h["beta2"])
    c1, c2 = 1 - b1 ** h["t"], 1 - b2 ** h["t"]
    g = f["grad"][a:a + n].float() * f32(h["grad_scale"])
    w = f["master"][a:a + n] * f32(1 - f32(h["lr"]) * f32(decay))
    m, v = f["m"][a:a + n], f["v"][a:a + n]
    if bits == 32:
        m1 = m * b1 + g * f32(1 - b1)
        v1 = v * b2 + (g * g) * f32(1 - b2)
        d = torch.sqrt(v1 / f32(c2)) + f32(h["eps"])
        w = w - (m1 / f32(c1) / d) * f32(h["lr"])
        m.copy_(m1)
        v.copy_(v1)
    else:
        k = slice(a // 256, a // 256 + -(-n // 256))
        size_m, size_v = (_power(f[q][k].int())[:, None].expand(-1, 256).reshape(-1)[:n] for q in ("m_scale", "v_scale"))
        m0 = _decode(m & 127, 121) * size_m
        m0 = torch.where(m > 127, -m0, m0)
        r0 = _decode(v, 113) * size_v
        m1 = m0 * b1 + g * f32(1 - b1)
        r1 = torch.sqrt((r0 * r0) * b2 + (g * g) * f32(1 - b2))
        d = r1 * f32(1 / math.sqrt(c2)) + f32(h["eps"])
        w = w - (m1 * f32(f32(h["lr"]) / c1)) / d
        rnd = _hash16(n, a, (h["seed"] + h["t"] * 0x510E527F) & 0xFFFFFFFF)
        em, ev = _block_scale(m1.abs()), _block_scale(r1)
        wide = lambda e: _power(254 - e)[:, None].expand(-1, 256).reshape(-1)[:n]  # noqa: E731
        cm = _encode(m1.abs() * wide(em), rnd, 121, 127)
        cv = torch.maximum(_encode(r1 * wide(ev), rnd, 113, 255), (r1 > 0).int())
        m.copy_(cm + 128 * ((m1 < 0) & (cm > 0)))
        v.copy_(cv)
        f["m_scale"][k], f["v_scale"][k] = em.to(torch.uint8), ev.to(torch.uint8)
    f["master"][a:a + n] = w
    f["param"][a:a + n] = w.to(f["param"].dtype)


def _adamw(s):
    f, bits = s["flat"], s["case"]["bits"]
    for a, n, decay in zip(s["starts"], s["sizes"], s["decay"]):
        _adamw_one(f, a, n, decay, s["hp"], bits)
    r = {"master": f["master"], "param": f["param"]}
    if bits == 32:
        return {**r, "m": f["m"], "v": f["v"]}
    size = lambda q: _power(f[q].int())[:, None]  # noqa: E731
    m = (_decode(f["m"] & 127, 121).view(-1, 256) * size("m_scale")).view(-1)
    m = torch.where(f["m"] > 127, -m, m)
    return {**r, "m": m.bfloat16(), "root_v": (_decode(f["v"], 113).view(-1, 256) * size("v_scale")).view(-1).bfloat16()}


# ---- work ---------------------------------------------------------------------
def work(case):
    e = _esize(case)
    if case["op"].startswith("ln"):
        n, d = case["rows"], case["dim"]
        if case["op"] == "ln_fwd":
            return {"bytes": 2 * n * d * e + 2 * d * e + 8 * n, "flops": 8 * n * d}
        return {"bytes": 3 * n * d * e + 3 * d * e + 8 * n, "flops": 14 * n * d}
    if case["op"].startswith("ce"):
        n, v, d = case["tokens"], case["vocab"], case["hidden"]
        if case["op"] == "ce_fwd":
            return {"bytes": (n + v) * d * e + 16 * n, "flops": 2 * n * v * d}
        return {"bytes": 2 * (n + v) * d * e + 16 * n, "flops": 6 * n * v * d}
    n = sum(_numels(case))
    # gradient in, parameter out, master weight in and out, both moments in and out; 8-bit moments also come back as values
    return {"bytes": n * (2 * e + 24 if case["bits"] == 32 else 2 * e + 16), "flops": n * (16 if case["bits"] == 32 else 40)}


# ---- the definitions in 64 bits -------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("ln"):
        x = s["x"].double()
        if case["op"] == "ln_fwd":
            var, mean = torch.var_mean(x, 1, correction=0)
            rstd = (var + EPS) ** -0.5
            y = torch.addcmul(s["b"].double(), (x - mean[:, None]) / (var + EPS).sqrt()[:, None], s["w"].double())
            return {"y": y, "mean": mean, "rstd": rstd}
        # with the statistics as given, the backward pass is the product with the row's projection
        dy, w = s["dy"].double(), s["w"].double()
        mean, rstd = s["mean"].double(), s["rstd"].double()
        h = torch.einsum("rd,r->rd", x - mean[:, None], rstd)
        q = dy * w / x.shape[1]
        dx = x.shape[1] * q - q.sum(1)[:, None] - h * torch.einsum("rd,rd->r", q, h)[:, None]
        return {"dx": dx * rstd[:, None], "dw": torch.einsum("rd,rd->d", dy, h), "db": torch.einsum("rd->d", dy)}
    if case["op"].startswith("ce"):
        x, w, t = s["x"].double(), s["w"].double(), s["t"]
        n, v = x.shape[0], w.shape[0]
        good = [(t >= 0) & (t < v)][0]
        number = max(1, int(good.sum()))
        r = {"loss": torch.zeros(n, device="cuda", dtype=torch.float64), "lse": torch.zeros(n, device="cuda", dtype=torch.float64)}
        train = case["op"] == "ce_train"
        if train:
            r["dx"], r["dw"] = torch.zeros_like(x), torch.zeros_like(w)
        for a in range(0, n, 2048):
            b = slice(a, min(a + 2048, n))
            z = torch.mm(x[b], w.T)
            r["lse"][b] = torch.logsumexp(z, 1)
            i = torch.nonzero(good[b])[:, 0]
            r["loss"][b][i] = r["lse"][b][i] - z[i, t[b][i]]
            if train:
                p = torch.softmax(z, 1)
                p[i, t[b][i]] -= 1
                p[~good[b]] = 0
                r["dx"][b] = torch.mm(p, w) * (s["scale"] / number)
                r["dw"] += torch.mm(p.T, x[b]) * (s["scale"] / number)
        r["mean"] = r["loss"].sum() / number
        return r
    f, h = s["flat"], s["hp"]
    single = {k: f32(q) if isinstance(q, float) else q for k, q in h.items()}
    bias1, bias2 = -math.expm1(h["t"] * math.log(single["beta1"])), -math.expm1(h["t"] * math.log(single["beta2"]))
    keep = torch.ones(f["master"].numel(), device="cuda", dtype=torch.float32)
    for a, n, decay in zip(s["starts"], s["sizes"], s["decay"]):
        keep[a:a + n] = 1 - single["lr"] * f32(decay)
    out = {"master": torch.empty_like(f["master"], dtype=torch.float64)}
    out["param"] = out["master"]
    names = ("m", "v") if case["bits"] == 32 else ("m", "root_v")
    out.update({k: torch.empty_like(f["master"], dtype=torch.float64) for k in names})
    step = 1 << 26
    for a in range(0, keep.numel(), step):
        c = slice(a, min(a + step, keep.numel()))
        g = f["grad"][c].double() * single["grad_scale"]
        if case["bits"] == 32:
            m, v = f["m"][c].double(), f["v"][c].double()
        else:
            m = _value64(f["m"][c] & 127, f["m_scale"][a // 256:], 6) * (1.0 - 2.0 * (f["m"][c] >= 128))
            v = _value64(f["v"][c], f["v_scale"][a // 256:], 14) ** 2
        m = torch.lerp(g, m, single["beta1"])
        v = torch.lerp(g.square(), v, single["beta2"])
        out["master"][c] = f["master"][c].double() * keep[c] - single["lr"] * (m / bias1) / ((v / bias2).sqrt() + single["eps"])
        if case["bits"] == 32:
            out["m"][c], out["v"][c] = m, v
        else:
            rnd = _hash16(m.numel(), a, (h["seed"] + h["t"] * 0x510E527F) & 0xFFFFFFFF).double() / 65536
            out["m"][c] = _stored64(m.abs(), rnd, 6, 1.9375) * m.sign()
            out["root_v"][c] = _stored64(v.sqrt(), rnd, 14, 1.9375, True)
    return out


def _value64(code, scale, deep):
    """Codes to values: fraction f of 16, exponent e: (16 + f) / 16 2^(e - 1 - deep), or f / 16 2^-deep where e is 0."""
    e, f = (code >> 4).double(), (code & 15).double() / 16
    y = torch.where(e == 0, f * 2.0 ** -deep, (1 + f) * torch.exp2(e - 1 - deep))
    return y * torch.exp2(scale[: -(-code.numel() // 256)].double() - 127).repeat_interleave(256)[: code.numel()]


def _stored64(x, rnd, deep, most, floor=False):
    """What x >= 0 is stored as: the next code below, or above with the chance of its distance, in blocks of 256."""
    b = x.view(-1, 256)
    top = b.max(1, keepdim=True).values
    unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -126) * (32 / 31))))
    y = b / unit
    gap = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -deep)))) / 16
    y = (torch.floor(y / gap + rnd.view(-1, 256)) * gap).clamp(max=most)
    if floor:
        y = torch.where((b > 0) & (y == 0), 2.0 ** -(deep + 4), y)
    return (y * unit).view(-1)
