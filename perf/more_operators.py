"""Root-mean-square norm, log probabilities, gradient norm: what is timed, the plain forms, the definitions in 64 bits.

Three operators beside layer norm, cross entropy and AdamW, on sizes of the
parameter lists this repository benchmarks (a 50257-row embedding; d = 768,
1600 and 4096; 12 and 48 layers):

  rms_fwd   root-mean-square norm of rows with the residual's addition, to 16
            or 32 bits or to 8 bits with a scale per block (which are read out
            as the values they stand for)
  rms_bwd   its gradients: of the residual stream and of the weight
  lp        log probabilities of given tokens over a large vocabulary, the
            entropy, and the most likely alternatives
  lp_train  log probabilities and entropy with the gradients of x and W
  norm      the global norm of a list's gradients, whether one is not finite,
            and the factor that clips them
  clip      the norm and the AdamW step that takes the gradients clipped

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


# ---- cases --------------------------------------------------------------------
def listed():
    return [
        # one token of a d = 4096 model, into the 8-bit operand of the next product: latency alone
        {"name": "rms_one_row_8bit", "op": "rms_fwd", "rows": 1, "dim": 4096, "pad": 0, "residual": True, "block": 128, "dtype": "bf16"},
        # a training batch of 8192 tokens through a d = 4096 block's norm
        {"name": "rms_8192x4096", "op": "rms_fwd", "rows": 8192, "dim": 4096, "pad": 0, "residual": True, "block": 0, "dtype": "bf16"},
        # the same batch into 8 bits
        {"name": "rms_8192x4096_8bit", "op": "rms_fwd", "rows": 8192, "dim": 4096, "pad": 0, "residual": True, "block": 128, "dtype": "bf16"},
        # odd sizes and a padded row stride, fp32 training
        {"name": "rms_bwd_odd_fp32", "op": "rms_bwd", "rows": 1003, "dim": 771, "pad": 5, "residual": True, "dtype": "fp32"},
        # batch 32 x sequence 1024 x hidden 1600, the activation checkpoint this repository partitions
        {"name": "rms_bwd_32768x1600", "op": "rms_bwd", "rows": 32768, "dim": 1600, "pad": 0, "residual": True, "dtype": "fp16"},
        # one generated token scored against the whole vocabulary, with 8 alternatives (the weight is read once)
        {"name": "lp_one_token", "op": "lp", "tokens": 1, "vocab": 50257, "hidden": 4096, "pad": 0, "top": 8, "scale": 1.0, "dtype": "bf16"},
        # scoring a ragged batch at temperature 0.8, with 20 alternatives
        {"name": "lp_1023_top20", "op": "lp", "tokens": 1023, "vocab": 50257, "hidden": 1600, "pad": 0, "top": 20, "scale": 1.25, "dtype": "fp16"},
        # scoring a batch of 8192 tokens at d = 4096, with 8 alternatives
        {"name": "lp_8192x4096", "op": "lp", "tokens": 8192, "vocab": 50257, "hidden": 4096, "pad": 0, "top": 8, "scale": 1.0, "dtype": "bf16"},
        # a policy-gradient step with an entropy bonus, d = 768
        {"name": "lp_train_8192x768", "op": "lp_train", "tokens": 8192, "vocab": 50257, "hidden": 768, "pad": 0, "top": 0, "scale": 1.0, "dtype": "bf16"},
        # the gradients of two layers' vectors alone: latency
        {"name": "norm_vectors", "op": "norm", "list": "vectors", "dtype": "fp32"},
        # the gradients of the 48-layer d = 1600 list, 1.56e9 values
        {"name": "norm_48x1600", "op": "norm", "list": "48x1600", "dtype": "bf16"},
        # a clipped step of the 12-layer d = 768 list
        {"name": "clip_12x768", "op": "clip", "list": "12x768", "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rms_fwd", "rms_bwd", "lp", "lp_train", "norm", "clip"])
    if op.startswith("rms"):
        dim = _log(rng, 16, 16384)
        rows = _log(rng, 1, max(1, min(65536, 32768 * 1600 // dim)))
        c = {"op": op, "rows": rows, "dim": dim, "pad": rng.choice([0, 0, 1, 8]), "residual": rng.random() < 0.7,
             "dtype": rng.choice(["fp16", "bf16", "fp32"])}
        return {**c, "block": rng.choice([0, 32, 128])} if op == "rms_fwd" else c
    if op.startswith("lp"):
        hidden = 8 * _log(rng, 8, 512)
        vocab = _log(rng, 2, 65536)
        most = 8192 * 50257 * 4096 // (hidden * vocab) // (1 if op == "lp" else 3)
        tokens = _log(rng, 1, min(16384, most, (8192 * 50257) // vocab))
        return {"op": op, "tokens": tokens, "vocab": vocab, "hidden": hidden, "pad": rng.choice([0, 0, 8]),
                "top": min(vocab, rng.choice([0, 1, 5, 8, 20, 32])) if op == "lp" else 0, "scale": rng.choice([1.0, 1.0, 1.25, 0.5]),
                "dtype": rng.choice(["fp16", "bf16"])}
    return {"op": op, "list": "drawn", "count": _log(rng, 1, 300), "most": _log(rng, 8, 2_000_000),
            "pick": rng.randrange(1 << 30), "dtype": rng.choice(["fp16", "bf16", "fp32"])}


def _numels(case):
    if case["list"] == "vectors":
        return [768] * 8
    if case["list"] == "drawn":
        g = torch.Generator().manual_seed(case["pick"])
        u = torch.rand(case["count"], generator=g, dtype=torch.float64)
        return [max(1, int(n)) for n in torch.exp(u * math.log(case["most"])).tolist()]
    layers, d = (int(q) for q in case["list"].split("x"))
    return [50257 * d] + [3 * d * d, d * d, 4 * d * d, 4 * d * d, d, d, d, d] * layers


# ---- inputs -------------------------------------------------------------------
def _rows(g, n, width, pad, dtype, scale=1.0):
    """(n, width) values in a buffer whose rows are width + pad apart."""
    full = torch.zeros(n, width + pad, device="cuda", dtype=dtype)
    full[:, :width] = torch.randn(n, width, device="cuda", generator=g) * scale
    return full[:, :width]


def _grid_rows(g, n, width, pad, dtype, std):
    """The same, as whole multiples (8 bits at most) of a power of two, as values from an 8-bit checkpoint are.

    Products and their sums are then exact in 32 bits in every order, so that which alternative is the more
    likely is decided by the values, not by a sum's rounding.
    """
    step = 2.0 ** (math.floor(math.log2(std)) - 4)
    full = torch.zeros(n, width + pad, device="cuda", dtype=dtype)
    full[:, :width] = (torch.randn(n, width, device="cuda", generator=g) * (std / step)).round_().clamp_(-255, 255) * step
    return full[:, :width]


def _like(x):
    return torch.empty_strided(x.shape, x.stride(), device="cuda", dtype=x.dtype)


def _zdtype(zg, case):
    return {"fp16": zg.ZERO_FP16, "bf16": zg.ZERO_BF16, "fp32": zg.ZERO_FP32}[case["dtype"]]


def _prepare_rms(case, g):
    dt = DTYPES[case["dtype"]]
    n, d, pad = case["rows"], case["dim"], case["pad"]
    s = {"case": case, "w": (1 + 0.2 * torch.randn(d, device="cuda", generator=g)).to(dt)}
    x = _rows(g, n, d, pad, dt, 2.0)
    if case["op"] == "rms_fwd":
        s["x"] = x                                                         # a block's output, and the stream it joins
        s["r"] = _rows(g, n, d, pad, dt, 3.0) if case["residual"] else None
    else:
        s["h"], s["dy"] = x, _rows(g, n, d, pad, dt)
        s["dh"] = _rows(g, n, d, pad, dt) if case["residual"] else None    # the stream's own gradient
        s["rstd"] = torch.rsqrt(x.float().square().mean(1) + EPS)
    if own:
        import zero_sharded_mixed_bucket_gb300 as zg
        block = case.get("block", 0)
        s["zg"], s["plan"] = zg, zg.zero_rms_plan(n, d, _zdtype(zg, case), d + pad, d + pad, block)
        if case["op"] == "rms_bwd":
            s["out"] = [_like(x), torch.empty_like(s["w"])]
            s["ws"] = torch.empty(s["plan"].workspace_bytes, device="cuda", dtype=torch.uint8)
            return s
        s["h"], s["rstd"] = _like(x) if case["residual"] else None, torch.empty(n, device="cuda")
        if block:
            s["q"] = torch.empty_strided(x.shape, x.stride(), device="cuda", dtype=torch.uint8)
            s["q_scale"] = torch.empty(n, -(-d // block), device="cuda", dtype=torch.uint8)
            s["y"] = torch.empty_strided(x.shape, x.stride(), device="cuda", dtype=torch.bfloat16)
        else:
            s["y"] = _like(x)
    return s


def _prepare_lp(case, g):
    dt = DTYPES[case["dtype"]]
    n, v, d, pad = case["tokens"], case["vocab"], case["hidden"], case["pad"]
    x = _grid_rows(g, n, d, pad, dt, 1.0)                                  # a norm's output
    w = _grid_rows(g, v, d, pad, dt, 1.5 / math.sqrt(d))
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    t = torch.where(torch.rand(n, device="cuda", generator=g) < 0.1, IGNORE, t)  # padding tokens
    t[0] = v - 1
    s = {"case": case, "x": x, "w": w, "t": t}
    train = case["op"] == "lp_train"
    if train:                                                              # advantages and an entropy bonus, means over the tokens
        s["dlogp"] = torch.randn(n, device="cuda", generator=g) / n
        s["dent"] = torch.full((n,), 0.01 / n, device="cuda")
        s["grad_scale"] = 1024.0                                           # the loss scale of mixed precision
    if own:
        import zero_sharded_mixed_bucket_gb300 as zg
        s["zg"], s["plan"] = zg, zg.zero_lp_plan(n, v, d, _zdtype(zg, case), d + pad, d + pad, top=case["top"])
        s["out"] = [torch.empty(n, device="cuda") for _ in range(3)]
        if case["top"]:
            s["top"] = [torch.empty(n, case["top"], device="cuda"), torch.empty(n, case["top"], device="cuda", dtype=torch.int64)]
        if train:
            s["grads"] = [_like(x), _like(w)]
        s["ws"] = torch.empty(s["plan"].workspace_bytes, device="cuda", dtype=torch.uint8)
    return s


def _prepare_list(case, g):
    dt = DTYPES[case["dtype"]]
    sizes = _numels(case)
    starts, total = [], 0
    for k in sizes:                     # every tensor starts at a multiple of 256 values of the flat buffers
        starts.append(total)
        total += -(-k // 256) * 256
    used = torch.zeros(total, device="cuda", dtype=torch.bool)
    for a, k in zip(starts, sizes):
        used[a:a + k] = True
    f = {"grad": torch.randn(total, device="cuda", generator=g).mul_(1e-2 * 1024).mul_(used).to(dt)}
    step = case["op"] == "clip"
    if step:
        f["master"] = torch.randn(total, device="cuda", generator=g).mul_(0.02).mul_(used)
        f["param"] = f["master"].to(dt)
        f["m"] = torch.randn(total, device="cuda", generator=g).mul_(3e-4).mul_(used)
        f["v"] = torch.rand(total, device="cuda", generator=g).mul_(1e-6).mul_(used)
    decay = [0.1 if k > 16384 else 0.0 for k in sizes]                     # vectors are not decayed
    s = {"case": case, "flat": f, "sizes": sizes, "starts": starts, "decay": decay, "max_norm": 1.0,
         "hp": {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "grad_scale": 1.0 / 1024, "t": 7, "seed": 0}}
    if own:
        import zero_sharded_mixed_bucket_gb300 as zg
        if not step:                    # the list is AdamW's, whose other buffers the norm leaves alone: one stands for all
            f["master"] = f["m"] = f["v"] = torch.empty(total, device="cuda")
        tensors = [zg.adamw_tensor(numel=k, weight_decay=wd, **{q: b[a:] for q, b in f.items()})
                   for a, k, wd in zip(starts, sizes, decay)]
        s["zg"], s["plan"] = zg, zg.zero_adamw_plan(tensors, _zdtype(zg, case), 32)
        s["table"] = torch.empty(s["plan"].table_bytes, device="cuda", dtype=torch.uint8)
        zg.zero_adamw_table_init(s["plan"], tensors, s["table"], torch.cuda.current_stream())
        s["own_hp"] = zg.zero_adamw_t(**s["hp"])
        s["norm"], s["flag"] = torch.empty(2, device="cuda"), torch.empty(1, device="cuda", dtype=torch.int32)
        s["ws"] = torch.empty(zg.zero_adamw_norm_workspace(s["plan"]), device="cuda", dtype=torch.uint8)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"].startswith("rms"):
        return _prepare_rms(case, g)
    return _prepare_lp(case, g) if case["op"].startswith("lp") else _prepare_list(case, g)


# ---- one pass -----------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rms_fwd": _own_rms_fwd, "rms_bwd": _own_rms_bwd, "lp": _own_lp, "lp_train": _own_lp,
                "norm": _own_list, "clip": _own_list}[op](s)
    return {"rms_fwd": _rms_fwd, "rms_bwd": _rms_bwd, "lp": _lp, "lp_train": _lp, "norm": _norm, "clip": _clip}[op](s)


def _own_rms_fwd(s):
    zg, st, block = s["zg"], torch.cuda.current_stream(), s["case"]["block"]
    q, q_scale = (s["q"], s["q_scale"]) if block else (None, None)
    zg.zero_rms_forward(s["plan"], s["x"], s["r"], s["w"], EPS, s["h"], None if block else s["y"], q, q_scale, s["rstd"], st)
    if block:
        zg.zero_rms_values(s["plan"], q, q_scale, s["y"], st)
    r = {"y": s["y"], "rstd": s["rstd"]}
    return {**r, "h": s["h"]} if s["case"]["residual"] else r


def _own_rms_bwd(s):
    dx, dw = s["out"]
    s["zg"].zero_rms_backward(s["plan"], s["dy"], s["dh"], s["h"], s["w"], s["rstd"], dx, dw, s["ws"], torch.cuda.current_stream())
    return {"dx": dx, "dw": dw}


def _own_lp(s):
    zg, c, st = s["zg"], s["case"], torch.cuda.current_stream()
    logp, lse, entropy = s["out"]
    top, index = s["top"] if c["top"] else (None, None)
    zg.zero_lp_forward(s["plan"], s["x"], s["w"], s["t"], c["scale"], logp, lse, entropy, top, index, s["ws"], st)
    r = {"logp": logp, "lse": lse, "entropy": entropy}
    if c["top"]:
        r["top"], r["index"] = top, index
    if c["op"] == "lp_train":
        r["dx"], r["dw"] = s["grads"]
        zg.zero_lp_backward(s["plan"], s["x"], s["w"], s["t"], c["scale"], lse, entropy, s["dlogp"], s["dent"], s["grad_scale"],
                            r["dx"], r["dw"], s["ws"], st)
    return r


def _own_list(s):
    zg, st, h = s["zg"], torch.cuda.current_stream(), s["hp"]
    zg.zero_adamw_norm(s["plan"], s["table"], h["grad_scale"], s["max_norm"], s["norm"], s["flag"], s["ws"], st)
    r = {"norm": s["norm"][0], "factor": s["norm"][1], "flag": s["flag"]}
    if s["case"]["op"] == "clip":
        zg.zero_adamw_step_clipped(s["plan"], s["table"], s["own_hp"], s["norm"], s["flag"], st)
        r.update({q: s["flat"][q] for q in ("master", "param", "m", "v")})
    return r


# ---- plain forms ----------------------------------------------------------------
# 8-bit values: e4m3 (448 the largest) times 2^(e-127), one byte e per block of a row,
# the least power of two that keeps the block's largest magnitude within 448.
def _to_8bit(y, block):
    n, d = y.shape
    b = torch.nn.functional.pad(y, (0, -d % block)).view(n, -1, block)
    bits = b.abs().amax(2).view(torch.int32)
    e = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp(min=0)
    e = torch.where(bits == 0, 0, e)
    up = ((254 - e) << 23).view(torch.float32)[:, :, None]
    q = (b * up).to(torch.float8_e4m3fn)
    return (q.float() / up).view(n, -1)[:, :d]


def _rms_fwd(s):
    c, dt = s["case"], DTYPES[s["case"]["dtype"]]
    h = s["x"].float()
    r = {}
    if c["residual"]:
        r["h"] = (h + s["r"].float()).to(dt)                               # the stream, as the next block reads it
        h = r["h"].float()
    r["rstd"] = torch.rsqrt((h * h).mean(1) + EPS)
    y = h * r["rstd"][:, None] * s["w"].float()
    return {"y": _to_8bit(y, c["block"]).bfloat16() if c["block"] else y.to(dt), **r}


def _rms_bwd(s):
    dt = s["h"].dtype
    xhat = s["h"].float() * s["rstd"][:, None]
    dy = s["dy"].float()
    g = dy * s["w"].float()
    dx = (g - xhat * (g * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(dt), "dw": (dy * xhat).sum(0).to(dt)}


def _keys(z):
    """Whole numbers in the order of alternatives: by logit, then the lower index first."""
    i = (z + 0.0).view(torch.int32)
    i = torch.where(i < 0, i ^ 0x7FFFFFFF, i).long()
    return i * (1 << 32) + (0x7FFFFFFF - torch.arange(z.shape[1], device="cuda"))


def _lp(s):
    c, x, w, t = s["case"], s["x"].float(), s["w"].float(), s["t"]
    n, v, k = x.shape[0], w.shape[0], c["top"]
    counted = (t >= 0) & (t < v)
    at = torch.where(counted, t, 0)[:, None]
    z = x @ w.t()
    r = {}
    if k:
        first = [torch.topk(_keys(z[a:a + 1024]), k, dim=1).values for a in range(0, n, 1024)]
        r["index"] = 0x7FFFFFFF - (torch.cat(first) & 0xFFFFFFFF)
        r["top"] = z.gather(1, r["index"]) * c["scale"]
    z *= c["scale"]
    most = z.max(1, keepdim=True).values
    given = z.gather(1, at)[:, 0]
    z -= most
    e = torch.exp(z)
    total = e.sum(1)
    r["lse"] = torch.log(total) + most[:, 0]
    r["logp"] = torch.where(counted, given - r["lse"], 0.0)
    r["entropy"] = torch.log(total) - (e * z).sum(1) / total
    if k:
        r["top"] -= r["lse"][:, None]
    if c["op"] == "lp_train":
        a = torch.where(counted, s["dlogp"], 0.0)
        e /= total[:, None]
        z -= torch.log(total)[:, None]                                     # log p
        z += r["entropy"][:, None]
        z *= s["dent"][:, None]
        z += a[:, None]
        z *= -e
        z.scatter_add_(1, at, a[:, None])
        z *= s["grad_scale"] * c["scale"]
        r["dx"], r["dw"] = (z @ w).to(s["x"].dtype), (z.t() @ x).to(s["x"].dtype)
    return r


def _norm(s):
    f, gs = s["flat"], f32(s["hp"]["grad_scale"])
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for a, n in zip(s["starts"], s["sizes"]):
        g = f["grad"][a:a + n].float() * gs
        total += (g * g).sum()
    norm = torch.sqrt(total)
    factor = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm.float(), "factor": factor.float(), "flag": (~torch.isfinite(norm)).int().view(1)}


def _clip(s):
    f, h, r = s["flat"], s["hp"], _norm(s)
    b1, b2 = f32(h["beta1"]), f32(h["beta2"])
    c1, c2 = 1 - b1 ** h["t"], 1 - b2 ** h["t"]
    for a, n, decay in zip(s["starts"], s["sizes"], s["decay"]):
        g = f["grad"][a:a + n].float() * (r["factor"] * f32(h["grad_scale"]))
        w = f["master"][a:a + n] * f32(1 - f32(h["lr"]) * f32(decay))
        m = f["m"][a:a + n].mul_(b1).add_(g * f32(1 - b1))
        v = f["v"][a:a + n].mul_(b2).add_((g * g) * f32(1 - b2))
        w = w - (m / f32(c1) / (torch.sqrt(v / f32(c2)) + f32(h["eps"]))) * f32(h["lr"])
        f["master"][a:a + n] = w
        f["param"][a:a + n] = w.to(f["param"].dtype)
    return {**r, **{q: f[q] for q in ("master", "param", "m", "v")}}


# ---- work ---------------------------------------------------------------------
def work(case):
    e = _esize(case)
    if case["op"].startswith("rms"):
        n, d = case["rows"], case["dim"]
        if case["op"] == "rms_bwd":
            return {"bytes": (4 if case["residual"] else 3) * n * d * e + 2 * d * e + 4 * n, "flops": 11 * n * d}
        stream = (3 if case["residual"] else 1) * n * d * e + d * e + 4 * n
        if case["block"]:               # codes and scales out, and the values read out
            return {"bytes": stream + 3 * n * d + n * -(-d // case["block"]), "flops": 7 * n * d}
        return {"bytes": stream + n * d * e, "flops": 5 * n * d}
    if case["op"].startswith("lp"):
        n, v, d = case["tokens"], case["vocab"], case["hidden"]
        if case["op"] == "lp":
            return {"bytes": (n + v) * d * e + (20 + 12 * case["top"]) * n, "flops": 2 * n * v * d}
        return {"bytes": 2 * (n + v) * d * e + 28 * n, "flops": 6 * n * v * d}
    n = sum(_numels(case))
    # the step: gradient in, parameter out, master weight and both moments in and out
    return {"bytes": n * e, "flops": 3 * n} if case["op"] == "norm" else {"bytes": n * (2 * e + 24), "flops": 20 * n}


# ---- the definitions in 64 bits -------------------------------------------------
def _exact_rms(s):
    c, w = s["case"], s["w"].double()
    if c["op"] == "rms_bwd":
        h, dy, rstd = s["h"].double(), s["dy"].double(), s["rstd"].double()
        n = torch.einsum("rd,r->rd", h, rstd)
        q = dy * w
        dx = torch.einsum("rd,r->rd", q, rstd) - torch.einsum("rd,r->rd", n, rstd * torch.einsum("rd,rd->r", q, n) / h.shape[1])
        return {"dx": dx if s["dh"] is None else dx + s["dh"].double(), "dw": torch.einsum("rd,rd->d", dy, n)}
    h, out = s["x"].double(), {}
    if c["residual"]:
        out["h"] = (h + s["r"].double()).to(s["x"].dtype).double()         # a stored value: rounded by definition
        h = out["h"]
    size = (torch.linalg.vector_norm(h, dim=1) ** 2 / h.shape[1] + EPS).sqrt()
    y = h / size[:, None] * w
    if c["block"]:
        b = torch.nn.functional.pad(y, (0, -y.shape[1] % c["block"])).unflatten(1, (-1, c["block"]))
        most = b.abs().amax(2, keepdim=True)
        unit = torch.exp2(torch.ceil(torch.log2(most / 448)).clamp(min=-127))
        b = b / unit
        gap = torch.exp2(torch.floor(torch.log2(b.abs().clamp(min=2.0 ** -6)))) / 8
        y = (torch.round(b / gap) * gap * unit).flatten(1)[:, : y.shape[1]]
    return {"y": y, "rstd": 1 / size, **out}


def _exact_lp(s):
    c, x, w, t = s["case"], s["x"].double(), s["w"].double(), s["t"]
    n, v, k = x.shape[0], w.shape[0], c["top"]
    good = (t >= 0) & (t < v)
    zeros = lambda *size: torch.zeros(size, device="cuda", dtype=torch.float64)  # noqa: E731
    r = {"logp": zeros(n), "lse": zeros(n), "entropy": zeros(n)}
    if k:
        r["top"], r["index"] = zeros(n, k), torch.zeros(n, k, device="cuda", dtype=torch.int64)
    train = c["op"] == "lp_train"
    if train:
        r["dx"], r["dw"] = torch.zeros_like(x), torch.zeros_like(w)
    for a in range(0, n, 1024):
        b = slice(a, min(a + 1024, n))
        z = torch.mm(x[b], w.T)
        if k:
            high, i = torch.sort(z, dim=1, descending=True, stable=True)
            r["index"][b] = i[:, :k]
        z *= c["scale"]
        lp = torch.log_softmax(z, 1)
        if k:
            r["top"][b] = lp.gather(1, i[:, :k])
        p = lp.exp()
        r["lse"][b] = torch.logsumexp(z, 1)
        r["entropy"][b] = torch.special.entr(p).sum(1)
        i = torch.nonzero(good[b])[:, 0]
        r["logp"][b][i] = lp[i, t[b][i]]
        if train:
            up = torch.where(good[b], s["dlogp"][b], 0.0).double()
            d = torch.special.entr(p) - p * (r["entropy"][b][:, None])      # of the entropy
            d = d * s["dent"][b].double()[:, None] - p * up[:, None]
            d[i, t[b][i]] += up[i]
            d *= s["grad_scale"] * c["scale"]
            r["dx"][b] = torch.mm(d, w)
            r["dw"] += torch.mm(d.T, x[b])
    return r


def _exact_list(s):
    f, h = s["flat"], s["hp"]
    gs = f32(h["grad_scale"])
    square = sum(float(f["grad"][a:a + n].double().square().sum()) for a, n in zip(s["starts"], s["sizes"]))
    norm = torch.tensor(math.sqrt(square) * gs, device="cuda", dtype=torch.float64)
    factor = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    out = {"norm": norm, "factor": torch.tensor(factor, device="cuda", dtype=torch.float64),
           "flag": torch.zeros(1, device="cuda", dtype=torch.int32)}
    if s["case"]["op"] == "norm":
        return out
    one = {k: f32(q) if isinstance(q, float) else q for k, q in h.items()}
    bias1, bias2 = -math.expm1(h["t"] * math.log(one["beta1"])), -math.expm1(h["t"] * math.log(one["beta2"]))
    keep = torch.ones(f["master"].numel(), device="cuda", dtype=torch.float32)
    for a, n, decay in zip(s["starts"], s["sizes"], s["decay"]):
        keep[a:a + n] = 1 - one["lr"] * f32(decay)
    g = f["grad"].double() * (gs * factor)
    out["m"] = torch.lerp(g, f["m"].double(), one["beta1"])
    out["v"] = torch.lerp(g.square(), f["v"].double(), one["beta2"])
    out["master"] = f["master"].double() * keep - one["lr"] * (out["m"] / bias1) / ((out["v"] / bias2).sqrt() + one["eps"])
    out["param"] = out["master"]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"].startswith("rms"):
        return _exact_rms(s)
    return _exact_lp(s) if case["op"].startswith("lp") else _exact_list(s)
