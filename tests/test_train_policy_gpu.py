"""The example that trains by policy gradient: the whole path's gradients, the
clipped step and the alternatives against the same model in 64 bits; the same
captured in a graph; a projection that reads the norm's 8-bit results."""
import importlib.util
import os

import pytest
import torch

import zero_sharded_mixed_bucket_gb300 as zg
from tests.conftest import ROOT

pytestmark = pytest.mark.gpu


def _example():
    spec = importlib.util.spec_from_file_location("train_policy", os.path.join(ROOT, "examples", "train_policy.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _job(tokens=90, vocab=700, hidden=136, **kw):
    M = _example()
    p = M.Policy(vocab, hidden, tokens, loss_scale=64.0, beta=0.1, temperature=0.8, **kw)
    g = torch.Generator(device="cuda").manual_seed(3)
    p.master["norm"] += 0.1 * torch.randn(hidden, device="cuda", generator=g)
    p.master["weight"] *= 4                           # states whose actions are not all alike
    for k in p.param:
        p.param[k].copy_(p.master[k])
    x, residual, good = next(M.batches(vocab, hidden, tokens))
    actions = torch.where(torch.rand(tokens, device="cuda", generator=g) < 0.2, -100, good)
    return M, p, x, residual, actions, torch.randn(tokens, device="cuda", generator=g), torch.randn(tokens, hidden, device="cuda", generator=g).bfloat16()


def _model(p, x, residual, actions, adv, dh):
    """The loss in 64 bits, from the stream as it is stored: its gradients, log probabilities and entropies."""
    q = {k: v.double().requires_grad_() for k, v in p.param.items()}
    h = (x.float() + residual.float()).bfloat16().double().requires_grad_()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + p.eps) * q["norm"]
    lp = torch.log_softmax(p.logit_scale * (y @ q["weight"].t()), 1)
    counted = actions >= 0
    logp = torch.where(counted, lp.gather(1, torch.where(counted, actions, 0)[:, None])[:, 0], 0.0)
    ent = -(lp.exp() * lp).sum(1)
    loss = -(adv.double() * logp).mean() - p.beta * ent.mean()
    (p.scale * loss + (dh.double() * h).sum()).backward()
    return h.grad, q["norm"].grad, q["weight"].grad, logp.detach(), ent.detach(), lp.detach()


@pytest.mark.parametrize("top", [0, 5])
def test_gradients_of_the_whole_path(top):
    """The path rounds y, G, dy and each result to bfloat16 (2^-8 each, independent errors): 2^-6 of a gradient's norm covers the four.
    y's rounding moves a logit by 2^-9 sum |y w|, at most a few times over the square root of its terms: 0.02 of a log probability."""
    M, p, x, residual, actions, adv, dh = _job(top=top)
    logp, ent = p.forward(x, residual, actions)
    dx = p.backward(actions, adv, dh)
    want = _model(p, x, residual, actions, adv, dh)
    assert (logp.double() - want[3]).abs().max() < 0.02 and (ent.double() - want[4]).abs().max() < 0.02
    for got, ref in ((dx, want[0]), (p.grad["norm"], want[1]), (p.grad["weight"], want[2])):
        assert (got.double() - ref).norm() <= 2.0 ** -6 * ref.norm()
    if top:
        z = want[5].gather(1, p.top_index)
        assert (z.diff(dim=1) < 0.04).all() and (z[:, 0] >= want[5].amax(1) - 0.04).all()
        assert (p.top_logp.double() - z).abs().max() < 0.02


def test_clipped_update():
    """One step: the norm of what the gradients hold, and AdamW's first step of them clipped."""
    M, p, x, residual, actions, adv, dh = _job(max_norm=0.01)
    p.forward(x, residual, actions)
    p.backward(actions, adv)
    old = {k: w.clone() for k, w in p.master.items()}
    assert p.update() and p.t == 1
    g = {k: v.double() / 64 for k, v in p.grad.items()}
    norm = sum((v * v).sum() for v in g.values()).sqrt()
    assert abs(float(p.norm[0]) - norm) < 1e-5 * norm and float(p.norm[1]) < 1
    factor = 0.01 / (float(norm) + 1e-6)
    for k in old:
        c = g[k] * factor
        want = old[k].double() * (1 - 3e-3 * (0.01 if k == "weight" else 0)) - 3e-3 * c / (c.abs() + 1e-8)
        big = c.abs() > 1e-6                          # elsewhere eps decides, and the factor's rounding with it
        assert (p.master[k].double() - want)[big].abs().max() < 1e-6
        assert torch.equal(p.param[k], p.master[k].bfloat16())


def test_overflowed_step_is_skipped():
    M, p, x, residual, actions, adv, dh = _job()
    p.scale = 2.0 ** 130
    old = {k: w.clone() for k, w in p.master.items()}
    p.forward(x, residual, actions)
    with pytest.raises(zg.ZeroError):                 # the scale itself is out of binary32's range
        p.backward(actions, adv)
    p.scale = 2.0 ** 127
    adv *= 2.0 ** 20
    p.backward(actions, adv)
    assert not p.update() and p.scale == 2.0 ** 126
    assert all(torch.equal(w, old[k]) for k, w in p.master.items())


def test_captured_whole():
    """The whole step captured and replayed over new batches, against the same calls made one by one."""
    M, p, x, residual, actions, adv, _ = _job(top=3)
    q = _job(top=3)[1]

    def step(o):
        s = torch.cuda.current_stream()
        o.forward(x, residual, actions)
        o.backward(actions, adv)
        zg.zero_adamw_norm(o.adamw, o.table, 1 / 64, 0.5, o.norm, o.flag, o.norm_ws, s)
        zg.zero_adamw_step_clipped(o.adamw, o.table, zg.zero_adamw_t(t=1, grad_scale=1 / 64, seed=0, **o.hp), o.norm, o.flag, s)

    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            step(q)
    data = M.batches(700, 136, 90, seed=9)
    for _ in range(3):
        a, b, c = next(data)
        x.copy_(a), residual.copy_(b), actions.copy_(c)
        torch.cuda.synchronize()
        graph.replay()
        step(p)
        torch.cuda.synchronize()
        for k in p.master:
            assert torch.equal(p.master[k], q.master[k]) and torch.equal(p.param[k], q.param[k])
        assert torch.equal(p.top_index, q.top_index) and torch.equal(p.norm, q.norm)


def test_captured_behind_copies_and_another_stream():
    """Inputs that a copy and another stream's kernel write just before, in a graph and in a row of calls: each call sees
    its own, and what is read out just after is its result."""
    n, d, v = 300, 512, 1000
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    rounds = [(r(n, d).bfloat16(), r(n, d).bfloat16(), r(n)) for _ in range(3)]
    x, res, dl = (torch.zeros_like(t) for t in rounds[0])
    w, weight = r(v, d).bfloat16() / 16, (1 + r(d) / 8).bfloat16()
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    e = lambda *s: torch.empty(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    h, y, vals, dx, dw, dxn, dwn = e(n, d), e(n, d), e(n, d), e(n, d), e(v, d), e(n, d), e(d)
    q, qs, rstd = torch.empty(n, d, dtype=torch.uint8, device="cuda"), torch.empty(n, d // 32, dtype=torch.uint8, device="cuda"), torch.empty(n, device="cuda")
    logp, lse, ent, tl, ti = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty(n, 4, device="cuda"), torch.empty(n, 4, dtype=torch.int64, device="cuda")
    rp, lp = zg.zero_rms_plan(n, d, zg.ZERO_BF16, block=32), zg.zero_lp_plan(n, v, d, zg.ZERO_BF16, top=4)
    rw, lw = (torch.empty(p.workspace_bytes, dtype=torch.uint8, device="cuda") for p in (rp, lp))
    out = [torch.empty_like(o) for o in (vals, logp, ent, tl, ti, dxn, dwn, dw)]
    side = torch.cuda.Stream()

    def step(k):
        s = torch.cuda.current_stream()
        side.wait_stream(s)
        with torch.cuda.stream(side):
            torch.mul(rounds[k][0], 1, out=x)
        res.copy_(rounds[k][1])
        dl.copy_(rounds[k][2])
        s.wait_stream(side)
        zg.zero_rms_forward(rp, x, res, weight, 1e-5, h, y, q, qs, rstd, s)
        zg.zero_rms_values(rp, q, qs, vals, s)
        zg.zero_lp_forward(lp, y, w, t, 1.0, logp, lse, ent, tl, ti, lw, s)
        zg.zero_lp_backward(lp, y, w, t, 1.0, lse, ent, dl, dl, 1.0, dx, dw, lw, s)
        zg.zero_rms_backward(rp, dx, None, h, weight, rstd, dxn, dwn, rw, s)
        for o, f in zip(out, (vals, logp, ent, tl, ti, dxn, dwn, dw)):
            o.copy_(f)
        for f in (x, res, dl, vals, logp, ent, tl, ti, dxn, dwn, dw):
            f.zero_()

    want = []
    for k in range(3):
        step(k)
        torch.cuda.synchronize()
        want.append([o.clone() for o in out])
    hs = (rounds[0][0].float() + rounds[0][1].float()).bfloat16().double()
    y64 = hs * torch.rsqrt((hs * hs).mean(1, keepdim=True) + 1e-5) * weight.double()
    z = y64.bfloat16().double() @ w.double().t()
    assert (want[0][1].double() - torch.log_softmax(z, 1).gather(1, t[:, None])[:, 0]).abs().max() < 0.05     # a y next to a border rounds either way
    for turn in range(20):                            # one behind the other, no wait between
        step(turn % 3)
        got = [o.clone() for o in out]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[19 % 3]))
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(st):
        with torch.cuda.graph(graph, stream=st):
            step(2)
            step(1)
    for o in out:
        o.zero_()
    torch.cuda.synchronize()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want[1]))


@pytest.mark.parametrize("block", [32, 128])
def test_projection_of_8bit_results(block):
    """The norm into 8 bits, read out as values, scored: what a product with 8-bit operands would see.  Each value is off by 2^-4 of itself
    at most, independently, so a logit by 2^-4 sqrt(sum (y w)^2) times a few: six of those."""
    n, d, v = 70, 256, 1000
    g = torch.Generator(device="cuda").manual_seed(4)
    x, r = (torch.randn(n, d, device="cuda", generator=g).bfloat16() for _ in range(2))
    w = (torch.randn(v, d, device="cuda", generator=g) / 16).bfloat16()
    t = torch.randint(0, v, (n,), device="cuda", generator=g)
    p, lp = zg.zero_rms_plan(n, d, zg.ZERO_BF16, block=block), zg.zero_lp_plan(n, v, d, zg.ZERO_BF16, top=3)
    h, y, vals = (torch.empty_like(x) for _ in range(3))
    q, sc = torch.empty(n, d, dtype=torch.uint8, device="cuda"), torch.empty(n, p.scale_cols, dtype=torch.uint8, device="cuda")
    ws = torch.empty(lp.workspace_bytes, dtype=torch.uint8, device="cuda")
    zg.zero_rms_forward(p, x, r, None, 1e-5, h, y, q, sc)
    zg.zero_rms_values(p, q, sc, vals)
    out = []
    for a in (y, vals):
        o = [torch.empty(n, device="cuda") for _ in range(3)] + [torch.empty(n, 3, device="cuda"), torch.empty(n, 3, dtype=torch.int64, device="cuda")]
        zg.zero_lp_forward(lp, a, w, t, 1.0, *o, ws)
        out.append(o)
    lsm = torch.log_softmax(vals.double() @ w.double().t(), 1)
    assert (out[1][0].double() - lsm.gather(1, t[:, None])[:, 0]).abs().max() < 1e-4
    spread = 2.0 ** -4 * ((y.double() ** 2) @ (w.double() ** 2).t()).sqrt().amax(1)
    assert ((out[0][0] - out[1][0]).double().abs() < 6 * 2 * spread).all()


def test_example_runs():
    M = _example()
    assert len(M.main(["--steps", "3", "--vocab", "300", "--hidden", "64", "--tokens", "128"])) == 3
    assert len(M.main(["--steps", "2", "--vocab", "300", "--hidden", "72", "--tokens", "50", "--top", "0", "--dtype", "fp16"])) == 2
