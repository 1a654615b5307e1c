"""The post-training operators together, as a program uses them: the example's step, its gradient
to the hidden states, a preference step on the same logits."""
import os
import sys

import pytest
import torch

import moe_expert_ffn_top_gb300 as m
import post_ref as ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    yield


def test_example_runs_and_its_gradient_is_the_definitions():
    import policy_block
    from synth import Shape
    losses, b = policy_block.train(Shape(T=256, H=512, I=256, E=16, k=2, r=16), 1000, 3)
    assert all(map(torch.isfinite, torch.tensor(losses)))
    before = {n: b.w[n].clone() for n in policy_block.FACTORS}
    hidden = b.forward()
    logits = torch.matmul(hidden, b.head.T)
    r = ref.tokens(logits, b.targets, 1.0)
    kl = torch.tensor(0.05).item()
    wl, ws, wd, lt, st, dtol = ref.policy(r, b.advantages, b.old, b.ref, None, [0, 256], None, 1.0, 0.2, 0.2, kl)
    loss = b.policy_step()
    assert (loss.double() - wl).abs() <= lt
    assert ((b.stats[0].double() - ws[0]).abs() <= st[0]).all()
    # the gradient to the hidden states: bf16 dlogits (half a step each), products rounded once to bf16
    want = wd @ b.head.double()
    size = wd.abs() @ b.head.double().abs()
    assert ((b.dout.double() - want).abs() <= 2 ** -8 * (want.abs() + size) + dtol @ b.head.double().abs() + 1e-12).all()
    for n in policy_block.FACTORS:
        assert torch.isfinite(b.w[n].float()).all() and not torch.equal(before[n], b.w[n])


def test_preference_step():
    """Reference sums, then log probabilities, loss and the gradient to the logits, against 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, n, seq = 90, 5000, torch.tensor([0, 20, 45, 60, 88], device="cuda")
    x, x0 = (torch.randn(T, n, generator=g, device="cuda") for _ in range(2))
    y = torch.randint(0, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[30:35] = -1
    lp, lse, sums, dl, sc = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty(4, device="cuda"), torch.zeros(T, device="cuda"), m.preference_scratch(2)
    loss, stats = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
    m.moe_lora_token_logp_forward(x0, y, lp)
    m.moe_lora_preference_loss(lp, y, seq, None, loss, stats, sc, seq_logp=sums)  # the reference model's sums
    m.moe_lora_token_logp_forward(x, y, lp, lse)
    m.moe_lora_preference_loss(lp, y, seq, sums, loss, stats, sc, beta=0.1, dlogp=dl)
    dx = torch.empty_like(x)
    m.moe_lora_token_logp_backward(x, y, lse, dl, dx)
    r0, r = ref.tokens(x0, y, 1.0), ref.tokens(x, y, 1.0)
    c0, c = (torch.where(v["ok"], v["logp"], 0.0) for v in (r0, r))
    s0 = ref.preference(c0, y, seq, None, [0, 2], None, 0.1, "sigmoid", 0.0, 0.0, False)[2]
    b32 = torch.tensor(0.1).item()
    wl, ws, _, wd = ref.preference(c, y, seq, s0, [0, 2], None, b32, "sigmoid", 0.0, 0.0, False)
    # a sum of 25 log probabilities, each within its tolerance; beta times that reaches the loss
    serr = 4 * 30 * float((r["tol"]["logp"] + r0["tol"]["logp"]).max())
    assert abs(float(loss) - float(wl)) <= b32 * serr + 1e-6
    hot = torch.zeros_like(r["p"]).scatter_(1, r["y"], 1.0)
    want = torch.where(r["ok"], torch.nan_to_num(wd).cuda(), 0.0)[:, None] * (hot - r["p"])
    tol = (want.abs() + r["p"] * b32) * (b32 * serr + float(r["tol"]["p"].max())) + 1e-9
    assert ((dx.double() - want).abs() <= tol).all()
    assert (dx[88:] == 0).all() and (dx[30:35] == 0).all()


def test_two_calls_at_once():
    """Calls on two streams, each with a workspace of its own, against the same calls one after the other."""
    g = torch.Generator(device="cuda").manual_seed(8)

    def problem(rows, n, shape):
        x = torch.randn(rows, n, generator=g, device="cuda").bfloat16()
        y = torch.randint(0, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
        adv, old = torch.randn(rows, generator=g, device="cuda"), -torch.rand(rows, generator=g, device="cuda") * 9
        u = torch.randn(*shape, generator=g, device="cuda")
        return x, y, adv, old, u

    def outputs(p):
        x, _, _, _, u = p
        out = dict(loss=torch.empty(1, device="cuda"), stats=torch.empty(1, 4, device="cuda"), d=torch.empty_like(x), p=torch.zeros_like(u),
                   m=torch.zeros_like(u))
        return out, m.policy_scratch(x.shape[0]), m.MuonTensors([dict(p=out["p"], g=u, m=out["m"], lr=0.1)])

    def call(p, out, sc, t):
        x, y, adv, old, _ = p
        for _ in range(5):
            m.moe_lora_policy_loss(x, y, adv, old, None, out["loss"], out["stats"], sc, dlogits=out["d"])
            m.moe_lora_muon_step(t)
    ps = [problem(40, 30000, (64, 16, 500)), problem(700, 9000, (9, 700, 128))]
    want = [outputs(p) for p in ps]
    for p, o in zip(ps, want):
        call(p, *o)
    got, streams = [outputs(p) for p in ps], [torch.cuda.Stream() for _ in ps]
    torch.cuda.synchronize()
    for p, o, s in zip(ps, got, streams):
        with torch.cuda.stream(s):
            call(p, *o)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(a[0][k], b[0][k]) for k in a[0])
