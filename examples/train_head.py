"""Train the end of a language model: layer norm, vocabulary projection, loss.

Hidden states go through a layer norm and a [vocab, hidden] projection; one
step is

    zero_ln_forward -> zero_ce_forward -> zero_ce_backward -> zero_ln_backward
    -> zero_adamw_check -> zero_adamw_step

in mixed precision: 16-bit parameters and gradients (the loss scaled), binary32
master weights, the moments in 8 or 32 bits, a step with an overflowed gradient
skipped and the scale halved.  The hidden states are synthetic: a fixed random
vector per token of the vocabulary, plus noise, so the loss falls from log
vocab towards what the noise leaves.

    python examples/train_head.py [--steps 60] [--vocab 8192] [--hidden 768] [--tokens 2048] [--bits 8]
"""
import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import zero_sharded_mixed_bucket_gb300 as zg  # noqa: E402

DTYPES = {"fp16": (zg.ZERO_FP16, torch.float16), "bf16": (zg.ZERO_BF16, torch.bfloat16)}


class Head:
    """Layer norm weight and bias and projection weight, with their optimizer state."""

    def __init__(self, vocab, hidden, tokens, dtype="bf16", bits=8, loss_scale=1024.0, device="cuda", seed=0):
        code, dt = DTYPES[dtype]
        self.scale, self.t, self.eps, self.hp = loss_scale, 0, 1e-5, dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8)
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = {"ln_weight": torch.ones(hidden, device=device), "ln_bias": torch.zeros(hidden, device=device),
                       "weight": torch.randn(vocab, hidden, device=device, generator=g) * 0.02}
        self.param = {k: w.to(dt) for k, w in self.master.items()}
        self.grad = {k: torch.zeros_like(p) for k, p in self.param.items()}
        kind = torch.uint8 if bits == 8 else torch.float32
        self.m = {k: torch.zeros(w.shape, dtype=kind, device=device) for k, w in self.master.items()}
        self.v = {k: torch.zeros(w.shape, dtype=kind, device=device) for k, w in self.master.items()}
        blocks = {k: -(-w.numel() // 256) for k, w in self.master.items()}
        self.scales = {k: [torch.zeros(n, dtype=torch.uint8, device=device) for _ in range(2)] for k, n in blocks.items()}
        # the list of tensors: the projection decays, the vectors do not
        tensors = [zg.adamw_tensor(grad=self.grad[k], param=self.param[k], master=w, m=self.m[k], v=self.v[k],
                                   numel=w.numel(), weight_decay=0.01 if w.dim() > 1 else 0.0,
                                   m_scale=self.scales[k][0] if bits == 8 else None,
                                   v_scale=self.scales[k][1] if bits == 8 else None)
                   for k, w in self.master.items()]
        self.adamw = zg.zero_adamw_plan(tensors, code, bits)
        self.table = torch.empty(self.adamw.table_bytes, dtype=torch.uint8, device=device)
        zg.zero_adamw_table_init(self.adamw, tensors, self.table, torch.cuda.current_stream())
        self.flag = torch.zeros(1, dtype=torch.int32, device=device)
        # activations and workspaces of a batch
        self.ln = zg.zero_ln_plan(tokens, hidden, code)
        self.ce = zg.zero_ce_plan(tokens, vocab, hidden, code)
        self.y, self.dy, self.dx = (torch.empty(tokens, hidden, dtype=dt, device=device) for _ in range(3))
        self.mean, self.rstd, self.loss, self.lse = (torch.empty(tokens, device=device) for _ in range(4))
        self.total = torch.empty(2, device=device)
        self.ln_ws = torch.empty(self.ln.workspace_bytes, dtype=torch.uint8, device=device)
        self.ce_ws = torch.empty(self.ce.workspace_bytes, dtype=torch.uint8, device=device)

    def forward(self, x, targets):
        """Loss of every token, its mean and the number of tokens that have one (on the device)."""
        s, p = torch.cuda.current_stream(), self.param
        zg.zero_ln_forward(self.ln, x, p["ln_weight"], p["ln_bias"], self.eps, self.y, self.mean, self.rstd, s)
        zg.zero_ce_forward(self.ce, self.y, p["weight"], targets, self.loss, self.lse, self.total, self.ce_ws, s)
        return self.loss, self.total

    def backward(self, x, targets):
        """Gradients of loss_scale times the mean loss; returns that of x."""
        s, p, g = torch.cuda.current_stream(), self.param, self.grad
        zg.zero_ce_backward(self.ce, self.y, p["weight"], targets, self.lse, None, self.scale, self.dy, g["weight"],
                            self.ce_ws, s)
        zg.zero_ln_backward(self.ln, self.dy, x, p["ln_weight"], self.mean, self.rstd, self.dx, g["ln_weight"],
                            g["ln_bias"], self.ln_ws, s)
        return self.dx

    def update(self):
        """AdamW on every tensor unless a gradient is inf or NaN; whether it was applied."""
        s = torch.cuda.current_stream()
        zg.zero_adamw_check(self.adamw, self.table, self.flag, s)
        hp = zg.zero_adamw_t(t=self.t + 1, grad_scale=1.0 / self.scale, seed=self.t, **self.hp)
        zg.zero_adamw_step(self.adamw, self.table, hp, self.flag, s)
        if self.flag.item():
            zg.zero_ce_status(self.ce, self.ce_ws, s)     # raises if the gradients did not finish
            self.scale = max(1.0, self.scale / 2)
            return False
        self.t += 1
        return True

    def step(self, x, targets):
        _, total = self.forward(x, targets)
        self.backward(x, targets)
        self.update()
        return total[0]


def batches(vocab, hidden, tokens, dtype="bf16", device="cuda", noise=0.5, seed=1):
    """Endless (hidden states, targets): a vector per vocabulary entry plus noise, one token in ten without a target."""
    g = torch.Generator(device=device).manual_seed(seed)
    table = torch.randn(vocab, hidden, device=device, generator=g)
    while True:
        t = torch.randint(0, vocab, (tokens,), device=device, generator=g)
        x = table[t] + noise * torch.randn(tokens, hidden, device=device, generator=g)
        t = torch.where(torch.rand(tokens, device=device, generator=g) < 0.1, -100, t)
        yield x.to(DTYPES[dtype][1]), t


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--vocab", type=int, default=8192)
    ap.add_argument("--hidden", type=int, default=768)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    ap.add_argument("--dtype", default="bf16", choices=sorted(DTYPES))
    a = ap.parse_args(argv)
    head = Head(a.vocab, a.hidden, a.tokens, a.dtype, a.bits)
    data = batches(a.vocab, a.hidden, a.tokens, a.dtype)
    losses = []
    for k in range(a.steps):
        losses.append(float(head.step(*next(data))))
        if k % 10 == 0 or k == a.steps - 1:
            print("step %4d  loss %.4f  (log vocab %.4f)  loss scale %g" % (k, losses[-1], math.log(a.vocab), head.scale))
    return losses


if __name__ == "__main__":
    main()
