"""GPU tests of the training-step operators at sizes where blocks work through many rows,
chunks or tensors: the kernels that large batches run.  Row counts follow the GPU's number of
SMs.  Definitions and tolerances are those of test_gpu_train_ops."""
import pytest
import torch

import moe_expert_ffn_top_gb300 as m
import test_gpu_train_ops as base
from test_gpu_train_ops import BF, F32, HF, _balance, _check_balance, _entry, _gen, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    yield


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ------------------------------------------------------------------ layer norm
# Aligned rows stream from 4 * teams rows per SM on; teams of a block (256 threads): 32 of 8 threads
# for narrow rows, 4 of 64 for 4,096 bf16 columns, one for 16,384.  One row more than the blocks
# share evenly.
@pytest.mark.parametrize("per_sm,n,dt,wdt,pad", [
    (17, 4096, BF, BF, 0),      # every slot of every thread full, 8 vectors a thread
    (9, 16384, BF, F32, 0),     # one team
    (17, 4000, BF, BF, 0),      # slots past the end of the row
    (5, 16000, HF, HF, 16),     # one team, rows apart
    (133, 64, BF, BF, 0), (133, 128, HF, F32, 8), (133, 200, BF, BF, 0), (133, 320, BF, F32, 0), (133, 384, BF, BF, 0),
    (133, 440, HF, HF, 8), (65, 1000, BF, BF, 0),  # 1 to 8 vectors a thread
    (17, 2560, F32, F32, 0), (17, 3000, F32, BF, 4), (17, 3584, F32, F32, 0), (17, 4096, F32, F32, 0),  # 10 to 16
    (9, 5000, F32, F32, 0), (133, 192, F32, F32, 0), (133, 256, F32, BF, 0),  # fp32, two teams; 6 and 8 vectors
    (17, 4095, BF, BF, 0), (17, 3001, F32, F32, 2), (133, 203, HF, F32, 3),  # rows off the 16-byte grid
])
def test_norm_forward_of_many_rows(per_sm, n, dt, wdt, pad):
    base.test_norm_forward(per_sm * _sms() + 1, n, dt, wdt, True, True, pad)


@pytest.mark.parametrize("dres", [False, True])
@pytest.mark.parametrize("per_sm,n,dt,wdt,pad", [
    (20, 4096, BF, F32, 0),     # two teams, ten rows each, partial rows of the weight gradients
    (17, 2048, F32, F32, 0), (65, 200, BF, BF, 0),
    (33, 577, F32, F32, 0),     # rows off the 16-byte grid, alike
    (20, 1000, HF, F32, 3),     # with dres the tensors' rows lie on the grid in different ways
    (5, 16384, BF, F32, 0), (5, 12004, F32, F32, 0),  # two slices, a cluster each
    (1, 70000, BF, F32, 0),     # nine slices in two launches
])
def test_norm_backward_of_many_rows(per_sm, n, dt, wdt, pad, dres):
    base.test_norm_backward(per_sm * _sms() + 1, n, dt, wdt, True, True, pad, dres, True)


def test_norm_in_place_of_many_rows():
    """y in place of x in the streamed forward, whose rows are read ahead (rows on the grid and off it)."""
    for n in (1024, 1027):
        x = torch.randn(65 * _sms() + 3, n, generator=_gen(n), device="cuda").bfloat16()
        y = torch.empty_like(x)
        m.moe_lora_layernorm_forward(x, None, None, y)
        m.moe_lora_layernorm_forward(x, None, None, x)
        assert torch.equal(x, y)


# ------------------------------------------------------------------ balance loss
def _routes(T, E, k, g, masked):
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    ids[torch.rand(T, k, generator=g, device="cuda") < masked] = -1
    return ids.contiguous()


@pytest.mark.parametrize("T,E,k,dt,masked,pad", [
    (9001, 256, 6, F32, 0.2, 0), (9001, 160, 8, BF, 0.5, 8), (8300, 130, 4, BF, 0.2, 2), (8300, 127, 8, HF, 0.2, 0),
    (8300, 60, 4, HF, 0.9, 4), (9001, 33, 4, F32, 0.2, 0), (3001, 384, 8, F32, 0.2, 4), (1501, 1024, 6, F32, 0.2, 0),
    (1501, 1023, 3, BF, 0.2, 1)])
def test_balance_in_three_launches(T, E, k, dt, masked, pad):
    """More than 2^19 logits or 2^13 tokens, rows of every alignment."""
    g = _gen(T + E)
    _, logits = _rows(T, E, E + pad, dt, g, scale=2.0)
    ids = _routes(T, E, k, g, masked)
    m.moe_lora_launch_count(True)
    got = _balance(logits, ids, None)
    assert m.moe_lora_launch_count(True) == 3
    assert got[4] == 0
    _check_balance(logits, ids, [0, T], got)
    fwd = _balance(logits, ids, None, grad=False)
    assert all(torch.equal(a, b) for a, b in zip(fwd[:3], got[:3]))


@pytest.mark.parametrize("E,dt", [(96, F32), (96, BF), (60, HF), (33, F32)])
def test_balance_adapters_of_all_sizes_equal_their_own_runs(E, dt):
    """A large adapter makes three launches of them all; small ones beside it (empty, without a live
    route, of one block, eight and sixteen) equal their own single launch bit for bit."""
    k = 5
    sizes = [128, 0, 8960, 2560, 256, 1280, 30]  # the third has more than 2^13 tokens, the fifth no live route
    offs = [sum(sizes[:i]) for i in range(len(sizes) + 1)]
    T, A = offs[-1], len(sizes)
    g = _gen(E)
    logits = (2 * torch.randn(T, E, generator=g, device="cuda")).to(dt)
    ids = _routes(T, E, k, g, 0.3)
    ids[offs[4]:offs[5]] = -1
    dloss = torch.rand(A, generator=g, device="cuda") + 0.5
    m.moe_lora_launch_count(True)
    got = _balance(logits, ids, offs, dloss=dloss, A=A)
    assert m.moe_lora_launch_count(True) == 3
    assert got[4] == 0
    _check_balance(logits, ids, offs, got, dloss=dloss)
    for a, n in enumerate(sizes):
        lo, hi = offs[a], offs[a + 1]
        if n == 0:
            assert float(got[0][a]) == 0 and (got[1][a] == 0).all() and (got[2][a] == 0).all()
            continue
        one = _balance(logits[lo:hi].clone(), ids[lo:hi].clone(), None, dloss=dloss[a:a + 1].clone())
        assert m.moe_lora_launch_count(True) == (3 if n > 1 << 13 else 1)
        for x, y in zip(one[:4], (got[0][a:a + 1], got[1][a:a + 1], got[2][a:a + 1], got[3][lo:hi])):
            assert torch.equal(x, y)


# ------------------------------------------------------------------ AdamW
def _many(eight, p_dt, g_dt, master, seed):
    """One tensor of 3 M elements and forty odd ones: several thousand chunks of 2,048 elements."""
    g = _gen(seed)
    sizes = [3_000_003] + [50_001 + 3_737 * i for i in range(40)]
    return [_entry(n, p_dt, g_dt, eight, master, g, lr=1e-3 * (1 + i % 3), wd=0.01 * (i % 4))
            for i, n in enumerate(sizes)]


def _new_gradients(es, seed):
    g = _gen(seed)
    for i, e in enumerate(es):
        e["g"].copy_(10.0 ** -(i % 5) * torch.randn(e["g"].numel(), generator=g, device="cuda"))


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("p_dt,g_dt,master", [(BF, F32, True), (BF, BF, False), (F32, HF, False)])
def test_adamw_of_many_chunks(p_dt, g_dt, master, eight):
    """Every block takes chunks of several tensors in turn: equal to slices of one tensor at a time, each
    less than the launch's blocks take at once, bit for bit (three steps, moments not zero)."""
    a, b = (_many(eight, p_dt, g_dt, master, 31) for _ in range(2))
    part = 2048 * 2 * _sms()  # elements: fewer chunks than blocks
    assert sum(e["p"].numel() for e in a) > 5 * 2048 * 4 * _sms()  # five chunks a block (of four per SM at most)
    whole, parts = m.AdamWTensors(a), []
    for e in b:
        for lo in range(0, e["p"].numel(), part):
            hi = min(lo + part, e["p"].numel())
            cut = {k: t[lo // 256:-(-hi // 256)] if k.endswith("scale") else t[lo:hi] for k, t in e.items()
                   if torch.is_tensor(t)}
            parts.append(m.AdamWTensors([dict(cut, lr=e["lr"], weight_decay=e["weight_decay"])]))
    scale = torch.full((1,), 0.5, device="cuda")
    for step in (1, 2, 3):
        for es in (a, b):
            _new_gradients(es, 40 + step)
        m.moe_lora_adamw_step(whole, step, grad_scale=scale)
        for t in parts:
            m.moe_lora_adamw_step(t, step, grad_scale=scale)
    for x, y in zip(a, b):
        for key in x:
            assert not torch.is_tensor(x[key]) or torch.equal(x[key], y[key]), key


# ------------------------------------------------------------------ all of them
def _calls():
    """Calls whose kernels stream, and the tensors that they write."""
    rows, n, T, E, k = 65 * _sms() + 1, 256, 9000, 96, 4
    g = _gen(50)
    x = torch.randn(rows, n, generator=g, device="cuda").bfloat16()
    gamma, beta = torch.randn(n, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda")
    logits, ids = torch.randn(T, E, generator=g, device="cuda"), _routes(T, E, k, g, 0.1)
    d = m.make_dims(T=T, H=512, I=64, E=E, k=k, r=8, A=2)
    offs = [0, 128, T]
    bsc, nsc = m.balance_scratch(d), m.layernorm_scratch(rows, n)
    f = dict(device="cuda")
    out = dict(y=torch.empty_like(x), mean=torch.empty(rows, **f), rstd=torch.empty(rows, **f), dx=torch.empty_like(x),
               dg=torch.empty(n, **f), db=torch.empty(n, **f), loss=torch.empty(2, **f),
               counts=torch.empty(2, E, dtype=torch.int32, device="cuda"), prob=torch.empty(2, E, **f),
               dl=torch.empty(T, E, **f))
    es = _many(False, BF, F32, True, 32) + _many(True, BF, F32, True, 33)
    ten = m.AdamWTensors(es)

    def run():
        m.moe_lora_layernorm_forward(x, gamma, beta, out["y"], out["mean"], out["rstd"])
        m.moe_lora_layernorm_backward(x, gamma, out["mean"], out["rstd"], out["y"], x, out["dx"], out["dg"], out["db"],
                                      nsc)
        m.moe_lora_balance_loss(d, logits, ids, offs, 0.01, out["loss"], out["counts"], out["prob"], bsc, out["dl"])
        m.moe_lora_adamw_step(ten, 2)

    return run, out, [e[k] for e in es for k in ("p", "master", "m", "v")]


def test_streamed_calls_in_a_graph():
    """Replays of all operators captured together (three launches of the balance loss, overlapped) equal the
    calls; the AdamW step goes on from its state."""
    run, out, state = _calls()
    start = [t.clone() for t in state]
    for _ in range(2):
        run()
    torch.cuda.synchronize()
    want = [t.clone() for t in list(out.values()) + state]
    for t, s in zip(state, start):
        t.copy_(s)
    run2, out2, state2 = _calls()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run2()
    for _ in range(2):
        for t in out2.values():
            t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(list(out2.values()) + state2, want))


def test_streamed_calls_do_not_allocate_on_the_device():
    run = _calls()[0]
    run()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        run()
    torch.cuda.synchronize()
    assert torch.cuda.mem_get_info()[0] == free
