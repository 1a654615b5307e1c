"""GPU tests of the training-step operators where a promise of include/moe_lora.h once did not
hold."""
import pytest
import torch

import moe_expert_ffn_top_gb300 as m
from test_gpu_train_ops import F32, _balance, _gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    yield


@pytest.mark.parametrize("T,E,dt", [(256, 16, F32), (256, 128, torch.bfloat16), (130, 127, torch.float16),
                                    (8200, 60, F32), (9000, 96, F32)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_balance_non_finite_dloss_leaves_dead_tokens_alone(T, E, dt, bad):
    """An overflowed loss scale reaches the live tokens' gradient; a token without a live route, and a row
    of -inf, keep theirs of 0 (one launch and three)."""
    g = _gen(T + E)
    logits = torch.randn(T, E, generator=g, device="cuda").to(dt)
    ids = torch.topk(logits.float(), 2, dim=1).indices.to(torch.int32).contiguous()
    ids[torch.rand(T, generator=g, device="cuda") < 0.3] = -1
    ids[3], ids[5] = -1, 1
    logits[5] = float("-inf")
    dead = (ids < 0).all(1)
    fine = _balance(logits, ids, None)
    got = _balance(logits, ids, None, dloss=torch.full((1,), bad, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(got[:3], fine[:3]))  # loss, counts and prob do not use it
    assert (got[3][dead] == 0).all() and (got[3][5] == 0).all()
    live = ~dead
    live[5] = False
    # p and f_e - <p, f> are finite and as a rule not 0: infinity stays infinite, NaN spreads
    assert not torch.isfinite(got[3][live]).any()


@pytest.mark.parametrize("rows,n,dt,launches", [
    (64, 577, F32, 1), (128, 577, F32, 1), (129, 577, F32, 2), (192, 577, F32, 2), (347, 577, F32, 2),
    (32, 4096, torch.bfloat16, 1), (33, 4096, torch.bfloat16, 2), (96, 4096, torch.bfloat16, 2)])
def test_norm_backward_adds_its_weight_gradients_only_where_a_team_has_one_row(rows, n, dt, launches):
    """One cluster of sixteen blocks does so (16 rows of 8 teams of 577 fp32 columns, of 2 teams of 4,096
    bf16 columns); with more rows it took 1 to 2.6 us longer than the two launches."""
    x = torch.randn(rows, n, generator=_gen(rows), device="cuda").to(dt)
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dx, dg, db = torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    sc = m.layernorm_scratch(rows, n)
    m.moe_lora_launch_count(True)
    m.moe_lora_layernorm_backward(x, None, mean, rstd, x, None, dx, dg, db, sc)
    assert m.moe_lora_launch_count(True) == launches
    # mean 0, rstd 1: h = dy = x; at most 347 squares, each rounding one unit
    want = (x.double() ** 2).sum(0)
    assert ((dg.double() - want).abs() <= (rows + 2) * 2.0 ** -24 * want).all()
    assert ((db.double() - x.double().sum(0)).abs() <= (rows + 2) * 2.0 ** -24 * x.double().abs().sum(0)).all()
