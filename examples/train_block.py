"""Trains the adapters, router and norm of one MoE block,

    out = h + FFN(layer_norm(h)),

on synthetic data: every step runs layer norm, router, balance loss, routing plan, expert
FFN, their backward passes and one AdamW step over all trained tensors (8-bit moments for
the per-expert factors, 32-bit for the rest).  The target is the same block with other
adapters, so the loss can fall.

    python examples/train_block.py [--steps N] [--tokens T]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_ffn_top_gb300 as m  # noqa: E402
from synth import Shape, make_inputs  # noqa: E402

FACTORS = ("A1", "A3", "B1", "B3", "A2", "B2")
BF16, F32 = torch.bfloat16, torch.float32


class Block:
    """Buffers and weights of the block, and its training step."""

    def __init__(self, shp: Shape, seed: int = 0, balance: float = 0.01, lr: float = 2e-3):
        self.shp, self.balance = shp, balance
        T, H, E, k, A = shp.T, shp.H, shp.E, shp.k, shp.A
        inp = {n: v.cuda() for n, v in make_inputs(shp, seed=seed).items() if torch.is_tensor(v)}
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.h = inp["x"]
        self.w = {n: inp[n] for n in ("W1", "W3", "W2") + FACTORS}
        self.Wr = (torch.randn(A, E, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
        self.gamma, self.beta = torch.ones(H, device="cuda"), torch.zeros(H, device="cuda")
        self.d = m.make_dims(T, H, shp.I, E, k, shp.r, A, shp.scale)
        self.ws = m.Workspaces.allocate(self.d)
        self.rsc, self.bsc, self.nsc = m.router_scratch(self.d), m.balance_scratch(self.d), m.layernorm_scratch(T, H)
        f = dict(device="cuda", dtype=F32)
        self.xn, self.y, self.dxn, self.dh = (torch.empty(T, H, dtype=BF16, device="cuda") for _ in range(4))
        self.mean, self.rstd = torch.empty(T, **f), torch.empty(T, **f)
        self.ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.rw, self.dw = torch.empty(T, k, **f), torch.empty(T, k, **f)
        self.logits, self.dl = torch.empty(T, E, **f), torch.empty(T, E, **f)
        self.aux, self.prob = torch.empty(A, **f), torch.empty(A, E, **f)
        self.counts = torch.empty(A, E, dtype=torch.int32, device="cuda")
        self.grads = m.alloc_grads(self.d)
        self.dWr, self.dgamma, self.dbeta = torch.empty(A, E, H, **f), torch.empty(H, **f), torch.empty(H, **f)
        self.step = 0
        # the trained tensors: bf16 operands with fp32 masters, fp32 norm weights without decay
        entries = [self._entry(self.w[n], self.grads["d" + n], lr, 0.01, eight=n in ("B1", "B3", "A2")) for n in FACTORS]
        entries.append(self._entry(self.Wr, self.dWr, lr, 0.01))
        entries += [self._entry(self.gamma, self.dgamma, lr, 0.0), self._entry(self.beta, self.dbeta, lr, 0.0)]
        self.trained = m.AdamWTensors(entries)
        self.all_grads = list(self.grads.values()) + [self.dWr, self.dgamma, self.dbeta]

    @staticmethod
    def _entry(p, g, lr, decay, eight=False):
        n = p.numel()
        e = dict(p=p, g=g, lr=lr, weight_decay=decay)
        if p.dtype != F32:
            e["master"] = p.to(F32)
        if eight:
            e.update(m=torch.zeros(n, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                     m_scale=torch.zeros(-(-n // 256), device="cuda"), v_scale=torch.zeros(-(-n // 256), device="cuda"))
        else:
            e.update(m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda"))
        return e

    def forward(self) -> torch.Tensor:
        m.moe_lora_layernorm_forward(self.h, self.gamma, self.beta, self.xn, self.mean, self.rstd)
        m.moe_lora_router_forward(self.d, self.xn, self.Wr, self.ids, self.rw, self.logits, self.rsc)
        m.moe_lora_plan(self.d, self.ids, None, self.ws.plan)
        m.moe_lora_forward(self.d, self.ws.plan, self.xn, self.rw, self.w, self.y, self.ws.saved, self.ws.fwd)
        return self.h + self.y

    def train_step(self, target: torch.Tensor):
        """One step; returns (mean squared error, balance loss), both on the device."""
        diff = (self.forward() - target).float()
        loss = diff.square().mean()
        dout = (diff * (2.0 / diff.shape[1])).to(BF16)
        # loss and gradient of the balance term in one pass over the logits
        m.moe_lora_balance_loss(self.d, self.logits, self.ids, None, self.balance * self.shp.T, self.aux, self.counts,
                                self.prob, self.bsc, dlogits=self.dl)
        m.moe_lora_backward(self.d, self.ws.plan, self.ws.saved, self.xn, self.rw, dout, self.w, self.dxn, self.dw,
                            self.grads, self.ws.bwd)
        m.moe_lora_router_backward_aux(self.d, self.xn, self.Wr, self.ids, self.rw, self.dw, self.dl, None, self.dWr,
                                       self.dxn, self.rsc)
        m.moe_lora_layernorm_backward(self.h, self.gamma, self.mean, self.rstd, self.dxn, dout, self.dh, self.dgamma,
                                      self.dbeta, self.nsc)  # dout: the residual stream's own gradient
        norm = torch.stack(torch._foreach_norm(self.all_grads)).norm()
        self.step += 1
        m.moe_lora_adamw_step(self.trained, self.step, beta2=0.99, grad_scale=(100.0 / norm).clamp(max=1.0))
        return loss, self.aux / self.shp.T


def train(shp: Shape, steps: int, seed: int = 0):
    """Losses and balance losses of `steps` steps."""
    target = Block(shp, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    for n in ("B1", "B3", "B2"):
        target.w[n].add_((0.1 * torch.randn(target.w[n].shape, generator=g, device="cuda")).to(BF16))
    want = target.forward()
    block = Block(shp, seed=seed)
    out = [block.train_step(want) for _ in range(steps)]
    assert m.moe_lora_get_error(block.d, block.ws.plan) == 0
    assert m.moe_lora_router_get_error(block.rsc) == 0
    assert m.moe_lora_balance_get_error(block.d, block.bsc) == 0
    return [float(a) for a, _ in out], [float(b) for _, b in out]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--tokens", type=int, default=1024)
    a = ap.parse_args()
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    losses, aux = train(Shape(T=a.tokens, H=512, I=256, E=16, k=2, r=16), a.steps)
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}  balance {aux[i]:.6f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.5f}  balance {aux[-1]:.6f}")


if __name__ == "__main__":
    main()
