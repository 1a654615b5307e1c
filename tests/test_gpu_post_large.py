"""Post-training operators where offsets pass 32 bits: the last rows and matrices of large tensors."""
import math

import pytest
import torch

import moe_expert_ffn_top_gb300 as m
import post_ref as ref
from train_ops_ref import TINY_OF, UNIT

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    yield
    torch.cuda.empty_cache()


def test_logits_past_32_bits():
    rows, n = 17000, 131072  # 2.2e9 elements
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(rows, n, dtype=BF, device="cuda")
    y = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    some = torch.tensor([0, 8191, 16383, 16384, rows - 1], device="cuda")
    x[some] = (2 * torch.randn(len(some), n, generator=g, device="cuda")).to(BF)
    y[some] = torch.randint(0, n, (len(some),), generator=g, device="cuda", dtype=torch.int32)
    r = ref.tokens(x[some], y[some], 1.0)
    old = torch.zeros(rows, device="cuda")
    old[some] = r["logp"].float()
    adv = torch.ones(rows, device="cuda")
    lp, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    m.moe_lora_token_logp_forward(x, y, lp, lse)
    assert ((lp[some].double() - r["logp"]).abs() <= r["tol"]["logp"]).all() and int((lp != 0).sum()) == len(some)
    d = torch.full_like(x, 3.0)
    dlogp = adv * 0.5
    m.moe_lora_token_logp_backward(x, y, lse, dlogp, d)
    hot = torch.zeros_like(r["p"]).scatter_(1, r["y"], 1.0)
    want = 0.5 * (hot - r["p"])
    # lse is rounded to fp32 here, which the probabilities follow
    tol = 0.5 * (r["p"] * (r["tol"]["p"] + 8 * 2.0 ** -24 * r["lse"].abs()[:, None]) + 4 * 2.0 ** -24 * (hot + r["p"]))
    assert ((d[some].double() - want).abs() <= tol + UNIT[BF] * (want.abs() + tol) + TINY_OF[BF]).all()
    assert int(torch.count_nonzero(d.view(-1, n).abs().amax(1))) == len(some)
    loss, stats = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
    m.moe_lora_policy_loss(x, y, adv, old, None, loss, stats, m.policy_scratch(rows), dlogits=d)
    wl, ws, wd, lt, st, dtol = ref.policy(r, adv[some], old[some], None, None, [0, len(some)], None, 1.0, 0.2, 0.2, 0.0)
    assert (loss.double() - wl).abs() <= lt and ((stats[0].double() - ws[0]).abs() <= st[0]).all()
    assert ((d[some].double() - wd).abs() <= dtol + UNIT[BF] * (wd.abs() + dtol) + TINY_OF[BF]).all()
    assert int(torch.count_nonzero(d.abs().amax(1))) == len(some)


@pytest.mark.parametrize("rows,cols", [(128, 2048), (2048, 128)])
def test_matrices_past_32_bits(rows, cols):
    batch = 8200  # 2.15e9 elements
    g = torch.Generator(device="cuda").manual_seed(2)
    grad = torch.zeros(batch, rows, cols, dtype=BF, device="cuda")
    some = [0, 4000, 8191, batch - 1]
    for i in some:
        grad[i] = torch.randn(rows, cols, generator=g, device="cuda").to(BF)
    p, mom = torch.zeros_like(grad), torch.zeros(batch, rows, cols, device="cuda")
    t = m.MuonTensors([dict(p=p, g=grad, m=mom, lr=-1.0, scale=1.0)])
    m.moe_lora_muon_step(t, momentum=0.5)
    assert m.moe_lora_muon_get_error(t) == 0
    for i in some:
        want = ref.newton_schulz(grad[i].float(), 5, (3.4445, -4.7750, 2.0315), 1e-7)
        # elements: bf16's rounding, and the 2-norm's bound for the whole matrix
        assert ((p[i].double() - want).abs() <= UNIT[BF] * want.abs() + 2e-5 * float(want.norm()) + TINY_OF[BF]).all()
        assert torch.equal(mom[i], 0.5 * grad[i].float())
    assert int(torch.count_nonzero(p.view(batch, -1).abs().amax(1))) == len(some)
    assert math.isclose(float(mom[batch - 2].abs().sum()), 0.0)
