"""Trains the adapters, router and norm of one MoE block and a frozen head on rewards,

    logits = (h + FFN(layer_norm(h))) head^T,

on synthetic data: log probabilities of the tokens under the policy that drew them and under a
reference model, then per step the clipped policy loss with its KL term and its gradient to the
logits, the block's backward pass, one Muon step over the factors and one AdamW step over the
router and the norm.

    python examples/policy_block.py [--steps N] [--tokens T] [--vocab V]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import moe_expert_ffn_top_gb300 as m  # noqa: E402
from synth import Shape  # noqa: E402
from train_block import BF16, F32, FACTORS, Block  # noqa: E402


class PolicyBlock(Block):
    """The block of train_block under a head, with what a policy step needs."""

    def __init__(self, shp: Shape, vocab: int, seed: int = 0, lr: float = 2e-3):
        super().__init__(shp, seed=seed, lr=lr)
        T, H = shp.T, shp.H
        g = torch.Generator(device="cuda").manual_seed(seed + 5)
        self.head = (torch.randn(vocab, H, generator=g, device="cuda") * H ** -0.5).to(BF16)
        self.logits_v = torch.empty(T, vocab, dtype=BF16, device="cuda")
        self.targets = torch.randint(0, vocab, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.targets[torch.rand(T, generator=g, device="cuda") < 0.2] = -1  # the prompts
        self.advantages = torch.randn(T, generator=g, device="cuda")
        f = dict(device="cuda", dtype=F32)
        self.old, self.ref, self.logp = (torch.empty(T, **f) for _ in range(3))
        self.loss, self.stats = torch.empty(1, **f), torch.empty(1, 4, **f)
        self.psc, self.err = m.policy_scratch(T), torch.zeros(1, dtype=torch.int32, device="cuda")
        factors = [self._entry(self.w[n], self.grads["d" + n], lr, 0.01) for n in FACTORS]
        self.muon = m.MuonTensors([{k: e[k] for k in ("p", "master", "g", "m", "lr", "weight_decay")} for e in factors])
        self.rest = m.AdamWTensors([self._entry(self.Wr, self.dWr, lr, 0.01), self._entry(self.gamma, self.dgamma, lr, 0.0),
                                    self._entry(self.beta, self.dbeta, lr, 0.0)])

    def score(self, out: torch.Tensor) -> None:
        """Log probabilities of the targets into `out`, and the logits they come from."""
        torch.matmul(self.forward(), self.head.T, out=self.logits_v)
        m.moe_lora_token_logp_forward(self.logits_v, self.targets, out, err=self.err)

    def policy_step(self) -> torch.Tensor:
        """One step; returns the loss, on the device.  The gradient takes the logits' place."""
        torch.matmul(self.forward(), self.head.T, out=self.logits_v)
        m.moe_lora_policy_loss(self.logits_v, self.targets, self.advantages, self.old, self.ref, self.loss, self.stats, self.psc,
                               kl_coef=0.05, logp=self.logp, dlogits=self.logits_v, err=self.err)
        self.dout = torch.matmul(self.logits_v, self.head)
        m.moe_lora_backward(self.d, self.ws.plan, self.ws.saved, self.xn, self.rw, self.dout, self.w, self.dxn, self.dw,
                            self.grads, self.ws.bwd)
        m.moe_lora_router_backward(self.d, self.xn, self.Wr, self.ids, self.rw, self.dw, None, self.dWr, self.dxn, self.rsc)
        m.moe_lora_layernorm_backward(self.h, self.gamma, self.mean, self.rstd, self.dxn, self.dout, self.dh, self.dgamma,
                                      self.dbeta, self.nsc)
        self.step += 1
        m.moe_lora_muon_step(self.muon)
        m.moe_lora_adamw_step(self.rest, self.step)
        return self.loss.clone()


def train(shp: Shape, vocab: int, steps: int, seed: int = 0):
    """Losses of `steps` steps, and the block."""
    block = PolicyBlock(shp, vocab, seed)
    block.score(block.old)
    block.ref.copy_(block.old)  # the reference model is where the policy starts
    losses = [block.policy_step() for _ in range(steps)]
    assert m.moe_lora_get_error(block.d, block.ws.plan) == 0
    assert m.moe_lora_router_get_error(block.rsc) == 0
    assert m.moe_lora_muon_get_error(block.muon) == 0
    assert int(block.err) == 0
    return [float(x) for x in losses], block


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    losses, block = train(Shape(T=a.tokens, H=512, I=256, E=16, k=2, r=16), a.vocab, a.steps)
    kl, clipped, ratio, entropy = block.stats[0].tolist()
    for i in range(0, a.steps, max(1, a.steps // 10)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"step {a.steps - 1:4d}  loss {losses[-1]:.5f}  kl {kl:.5f}  clipped {clipped:.3f}  ratio {ratio:.3f}  entropy {entropy:.3f}")


if __name__ == "__main__":
    main()
