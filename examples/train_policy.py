"""Train the end of a language model by policy gradient: norm, log probabilities, clipped step.

A block's output joins the residual stream and goes through a root-mean-square
norm and a [vocab, hidden] projection; one step is

    zero_rms_forward -> zero_lp_forward -> zero_lp_backward -> zero_rms_backward
    -> zero_adamw_norm -> zero_adamw_step_clipped

on the loss -mean(advantage * log p(action)) - beta * mean(entropy), in mixed
precision as in train_head.py, with the gradients' global norm clipped and a step
with an overflowed gradient skipped.  The task is synthetic: every state has one
good action, and an action's advantage is 1 if it is that one.

    python examples/train_policy.py [--steps 60] [--vocab 1024] [--hidden 256] [--tokens 2048] [--top 4]
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import zero_sharded_mixed_bucket_gb300 as zg  # noqa: E402

DTYPES = {"fp16": (zg.ZERO_FP16, torch.float16), "bf16": (zg.ZERO_BF16, torch.bfloat16)}


class Policy:
    """Norm weight and projection weight, with their optimizer state."""

    def __init__(self, vocab, hidden, tokens, dtype="bf16", top=0, loss_scale=1024.0, max_norm=1.0, beta=0.01, temperature=1.0,
                 device="cuda", seed=0):
        code, dt = DTYPES[dtype]
        self.scale, self.max_norm, self.beta, self.t, self.eps = loss_scale, max_norm, beta, 0, 1e-5
        self.logit_scale, self.hp = 1.0 / temperature, dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8)
        g = torch.Generator(device=device).manual_seed(seed)
        self.master = {"norm": torch.ones(hidden, device=device), "weight": torch.randn(vocab, hidden, device=device, generator=g) * 0.02}
        self.param = {k: w.to(dt) for k, w in self.master.items()}
        self.grad = {k: torch.zeros_like(p) for k, p in self.param.items()}
        self.m, self.v = ({k: torch.zeros_like(w) for k, w in self.master.items()} for _ in range(2))
        tensors = [zg.adamw_tensor(grad=self.grad[k], param=self.param[k], master=w, m=self.m[k], v=self.v[k], numel=w.numel(),
                                   weight_decay=0.01 if w.dim() > 1 else 0.0) for k, w in self.master.items()]
        self.adamw = zg.zero_adamw_plan(tensors, code, 32)
        self.table = torch.empty(self.adamw.table_bytes, dtype=torch.uint8, device=device)
        zg.zero_adamw_table_init(self.adamw, tensors, self.table, torch.cuda.current_stream())
        self.norm, self.flag = torch.zeros(2, device=device), torch.zeros(1, dtype=torch.int32, device=device)
        self.norm_ws = torch.empty(zg.zero_adamw_norm_workspace(self.adamw), dtype=torch.uint8, device=device)
        # activations and workspaces of a batch
        self.rms, self.lp = zg.zero_rms_plan(tokens, hidden, code), zg.zero_lp_plan(tokens, vocab, hidden, code, top=top)
        self.h, self.y, self.dy, self.dx = (torch.empty(tokens, hidden, dtype=dt, device=device) for _ in range(4))
        self.rstd, self.logp, self.lse, self.entropy, self.dlogp = (torch.empty(tokens, device=device) for _ in range(5))
        self.dentropy = torch.full((tokens,), -beta / tokens, device=device)
        self.top_logp = torch.empty(tokens, top, device=device) if top else None
        self.top_index = torch.empty(tokens, top, dtype=torch.int64, device=device) if top else None
        self.rms_ws = torch.empty(self.rms.workspace_bytes, dtype=torch.uint8, device=device)
        self.lp_ws = torch.empty(self.lp.workspace_bytes, dtype=torch.uint8, device=device)

    def forward(self, x, residual, actions):
        """Log probability of every action and entropy of every state; the most likely actions are in top_index."""
        s, p = torch.cuda.current_stream(), self.param
        zg.zero_rms_forward(self.rms, x, residual, p["norm"], self.eps, self.h, self.y, None, None, self.rstd, s)
        zg.zero_lp_forward(self.lp, self.y, p["weight"], actions, self.logit_scale, self.logp, self.lse, self.entropy, self.top_logp,
                           self.top_index, self.lp_ws, s)
        return self.logp, self.entropy

    def backward(self, actions, advantages, dh=None):
        """Gradients of loss_scale times the loss; returns that of x and of the stream (dh: what reaches the stream besides)."""
        s, p, g = torch.cuda.current_stream(), self.param, self.grad
        torch.mul(advantages, -1.0 / advantages.numel(), out=self.dlogp)
        zg.zero_lp_backward(self.lp, self.y, p["weight"], actions, self.logit_scale, self.lse, self.entropy, self.dlogp, self.dentropy,
                            self.scale, self.dy, g["weight"], self.lp_ws, s)
        zg.zero_rms_backward(self.rms, self.dy, dh, self.h, p["norm"], self.rstd, self.dx, g["norm"], self.rms_ws, s)
        return self.dx

    def update(self):
        """A clipped AdamW step unless a gradient is inf or NaN; whether it was applied."""
        s = torch.cuda.current_stream()
        zg.zero_adamw_norm(self.adamw, self.table, 1.0 / self.scale, self.max_norm, self.norm, self.flag, self.norm_ws, s)
        hp = zg.zero_adamw_t(t=self.t + 1, grad_scale=1.0 / self.scale, seed=0, **self.hp)
        zg.zero_adamw_step_clipped(self.adamw, self.table, hp, self.norm, self.flag, s)
        if self.flag.item():
            zg.zero_lp_status(self.lp, self.lp_ws, s)     # raises if the gradients did not finish
            self.scale = max(1.0, self.scale / 2)
            return False
        self.t += 1
        return True


def batches(vocab, hidden, tokens, dtype="bf16", device="cuda", noise=0.5, seed=1):
    """Endless (block outputs, stream, good actions): a vector per action plus noise, half of it in the stream."""
    g = torch.Generator(device=device).manual_seed(seed)
    table = torch.randn(vocab, hidden, device=device, generator=g)
    while True:
        good = torch.randint(0, vocab, (tokens,), device=device, generator=g)
        x = noise * torch.randn(tokens, hidden, device=device, generator=g)
        yield (0.5 * table[good] + x).to(DTYPES[dtype][1]), (0.5 * table[good] - 0.5 * x).to(DTYPES[dtype][1]), good


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--vocab", type=int, default=1024)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--top", type=int, default=4)
    ap.add_argument("--dtype", default="bf16", choices=sorted(DTYPES))
    a = ap.parse_args(argv)
    policy = Policy(a.vocab, a.hidden, a.tokens, a.dtype, a.top)
    g = torch.Generator(device="cuda").manual_seed(2)
    data, rewards = batches(a.vocab, a.hidden, a.tokens, a.dtype), []
    for k in range(a.steps):
        x, residual, good = next(data)
        # half of the actions tried are the good ones, the others any
        tried = torch.where(torch.rand(a.tokens, device="cuda", generator=g) < 0.5, good,
                            torch.randint(0, a.vocab, (a.tokens,), device="cuda", generator=g))
        policy.forward(x, residual, tried)
        policy.backward(tried, (tried == good).float())
        policy.update()
        rewards.append(float((policy.top_index[:, 0] == good).float().mean()) if a.top else float(policy.entropy.mean()))
        if k % 10 == 0 or k == a.steps - 1:
            print("step %4d  good action first %.3f  entropy %.3f  gradient norm %.3f" %
                  (k, rewards[-1], float(policy.entropy.mean()), float(policy.norm[0])))
    return rewards


if __name__ == "__main__":
    main()
