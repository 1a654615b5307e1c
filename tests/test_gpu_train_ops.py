"""GPU tests of the training-step operators against 64-bit definitions: layer norm
forward and backward, the router's balance loss, AdamW with 32- and 8-bit moments.

Tolerances are the rounding of the output's type plus, for the fp32 arithmetic behind
it, a bound of one rounding unit per operation and per addition of the longest chain
(train_ops_ref.CHAIN) times the size of the terms."""
import math

import pytest
import torch

import moe_expert_ffn_top_gb300 as m
import train_ops_ref as ref
from train_ops_ref import CHAIN, TINY_OF, U32, UNIT

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    yield


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(rows, n, ld, dtype, g, fill=float("nan"), scale=1.0, shift=0.0):
    """Random rows inside a wider buffer; what lies between the rows is `fill`."""
    b = torch.full((rows, ld), fill, dtype=dtype, device="cuda")
    b[:, :n] = (torch.randn(rows, n, generator=g, device="cuda") * scale + shift).to(dtype)
    return b, b[:, :n]


def _within(name, got, want, tol):
    got, want, tol = got.double().cpu(), want.double().cpu(), tol.double().cpu() if torch.is_tensor(tol) else tol
    off = (got - want).abs()
    assert torch.isfinite(got).all(), name
    assert (off <= tol).all(), (name, float((off / tol).max()))


# ------------------------------------------------------------------ layer norm
NORM = [  # rows, n, dtype, weight type, gamma, beta, extra columns between rows
    (1, 1, F32, F32, True, True, 0), (3, 2, BF, F32, True, True, 0), (1, 4096, BF, BF, True, True, 0),
    (5, 7, HF, HF, True, True, 1), (33, 64, BF, BF, True, False, 0), (130, 577, F32, F32, True, True, 3),
    (29, 1024, HF, F32, False, False, 8), (17, 1027, BF, BF, True, True, 5), (300, 2048, BF, F32, True, True, 8),
    (41, 2049, HF, F32, True, True, 6), (64, 4096, F32, F32, True, True, 0), (9, 8192, BF, BF, False, True, 0),
    (3, 12000, HF, HF, True, True, 0), (2, 16384, BF, BF, True, True, 16), (4, 16385, BF, F32, True, True, 0),
    (2, 40000, F32, F32, True, True, 0), (3, 70000, BF, F32, True, True, 0), (2, 70001, HF, BF, True, True, 0),
    (400, 9858, BF, BF, True, True, 8), (330, 8185, HF, F32, True, True, 7), (1300, 130, BF, F32, True, True, 1), (700, 256, F32, BF, True, True, 0), (1500, 96, BF, HF, True, True, 4),
]


@pytest.mark.parametrize("rows,n,dt,wdt,with_g,with_b,pad", NORM)
def test_norm_forward(rows, n, dt, wdt, with_g, with_b, pad):
    g = _gen(rows * 7 + n)
    _, x = _rows(rows, n, n + pad, dt, g, scale=2.0, shift=0.7)
    yb, y = _rows(rows, n, n + pad, dt, g, fill=5.0)
    gamma = (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(wdt) if with_g else None
    beta = torch.randn(n, generator=g, device="cuda").to(wdt) if with_b else None
    mean, rstd = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    m.moe_lora_layernorm_forward(x, gamma, beta, y, mean, rstd, 1e-5)
    y0 = torch.full_like(yb, 5.0)[:, :n]
    m.moe_lora_layernorm_forward(x, gamma, beta, y0, eps=1e-5)  # without the statistics
    wy, wmean, wrstd = ref.norm_fwd(x, gamma, beta, 1e-5)
    xd = x.double()
    amean = xd.abs().mean(1)
    _within("mean", mean, wmean, CHAIN * U32 * amean)
    dev = (xd - wmean[:, None]).abs()
    # relative error of the variance: its own chain, and twice the rounding of x - mean
    dvar = CHAIN * U32 + 4 * U32 * ((xd.abs() + amean[:, None]) * dev).mean(1) * CHAIN * wrstd ** 2
    _within("rstd", rstd, wrstd, wrstd * (dvar + 4 * U32))
    ga = 1.0 if gamma is None else gamma.double().abs()
    tol = (CHAIN * U32 * amean + 2 * U32 * xd.abs().amax(1))[:, None] * wrstd[:, None] * ga \
        + (dvar[:, None] + 8 * U32) * wy.abs() + (0.0 if beta is None else (dvar[:, None] + 8 * U32) * beta.double().abs())
    _within("y", y, wy, tol * (1 + UNIT[dt]) + UNIT[dt] * wy.abs() + TINY_OF[dt])
    assert torch.equal(y, y0)
    if pad:
        assert (yb[:, n:] == 5.0).all()  # nothing is written between the rows


@pytest.mark.parametrize("dres,wgrad", [(False, True), (True, True), (True, False)])
@pytest.mark.parametrize("rows,n,dt,wdt,with_g,with_b,pad", NORM)
def test_norm_backward(rows, n, dt, wdt, with_g, with_b, pad, dres, wgrad):
    g = _gen(rows * 5 + n)
    _, x = _rows(rows, n, n + pad, dt, g, scale=2.0, shift=0.7)
    _, dy = _rows(rows, n, n + pad, dt, g)
    dr = _rows(rows, n, n + 2 * pad, dt, g)[1] if dres else None
    dxb, dx = _rows(rows, n, n + pad, dt, g, fill=5.0)
    gamma = (1 + 0.3 * torch.randn(n, generator=g, device="cuda")).to(wdt) if with_g else None
    xf = x.float()
    mean = xf.mean(1)
    rstd = 1 / torch.sqrt((xf - mean[:, None]).square().mean(1) + 1e-5)
    dg = torch.full((n,), float("nan"), device="cuda") if wgrad else None
    db = torch.full((n,), float("nan"), device="cuda") if wgrad and with_b else None
    sc = m.layernorm_scratch(rows, n).fill_(0xFF) if wgrad or n > 8192 else None
    args = (x, gamma, mean, rstd, dy, dr)
    m.moe_lora_layernorm_backward(*args, dx, dg, db, sc)
    wdx, wdg, wdb, size, sg, sb = ref.norm_bwd(x, gamma, mean, rstd, dy, dr)
    _within("dx", dx, wdx, UNIT[dt] * wdx.abs() + (CHAIN + 16) * U32 * size + TINY_OF[dt])
    # rows are added in slices: a chain of at most 2 * CHAIN at these row counts
    if wgrad:
        _within("dgamma", dg, wdg, (2 * CHAIN + 8) * U32 * sg + 1e-30)
    if db is not None:
        _within("dbeta", db, wdb, 2 * CHAIN * U32 * sb + 1e-30)
    if pad:
        assert (dxb[:, n:] == 5.0).all()
    # the same bits again, and in place of dy
    dx2 = torch.zeros_like(dxb)[:, :n]
    dg2, db2 = (None if t is None else torch.empty_like(t) for t in (dg, db))
    m.moe_lora_layernorm_backward(*args, dx2, dg2, db2, sc)
    assert torch.equal(dx, dx2) and (dg is None or torch.equal(dg, dg2)) and (db is None or torch.equal(db, db2))
    dyc = torch.zeros(rows, n + pad, dtype=dt, device="cuda")[:, :n]  # dy's strides: the same calls bit for bit
    dyc.copy_(dy)
    m.moe_lora_layernorm_backward(x, gamma, mean, rstd, dyc, dr, dyc, dg2, db2, sc)
    assert torch.equal(dx, dyc) and (dg is None or torch.equal(dg, dg2)) and (db is None or torch.equal(db, db2))


def test_norm_in_place_and_on_another_stream():
    g = _gen(3)
    x = torch.randn(257, 768, generator=g, device="cuda").bfloat16()
    y = torch.empty_like(x)
    m.moe_lora_layernorm_forward(x, None, None, y)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.moe_lora_layernorm_forward(x, None, None, x)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(x, y)


def test_norm_gradients_match_differences():
    """Every gradient against central differences of the 64-bit forward."""
    g = _gen(11)
    rows, n, h = 4, 24, 1e-4
    x, dy = (torch.randn(rows, n, generator=g, device="cuda") for _ in range(2))
    gamma, beta = (torch.randn(n, generator=g, device="cuda") for _ in range(2))
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    m.moe_lora_layernorm_forward(x, gamma, beta, y, mean, rstd)
    dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
    m.moe_lora_layernorm_backward(x, gamma, mean, rstd, dy, None, dx, dg, db, m.layernorm_scratch(rows, n))
    loss = lambda a, b, c: (ref.norm_fwd(a, b, c, 1e-5)[0] * dy.double()).sum()  # noqa: E731
    args = [x.double(), gamma.double(), beta.double()]
    for k, got in ((0, dx), (1, dg), (2, db)):
        want = torch.zeros_like(args[k]).flatten()
        for i in range(want.numel()):
            d = torch.zeros_like(want)
            d[i] = h
            up, dn = ([a + s * d.view_as(a) if j == k else a for j, a in enumerate(args)] for s in (1, -1))
            want[i] = (loss(*up) - loss(*dn)) / (2 * h)
        # third derivatives of the norm at unit scale are O(100): h^2 * 100 = 1e-6, and fp32 arithmetic
        _within("d%d" % k, got.flatten(), want, 1e-5 * (1 + want.abs().max()))


def test_norm_special_values():
    """A constant row has rstd = 1/sqrt(eps) and y = beta; NaN or infinity spoil their own row only."""
    x = torch.full((4, 640), 3.0, device="cuda").bfloat16()
    x[1, 5], x[2, 639] = float("nan"), float("inf")
    beta = torch.arange(640, device="cuda").bfloat16()
    y, mean, rstd = torch.empty_like(x), torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    m.moe_lora_layernorm_forward(x, None, beta, y, mean, rstd, 1e-4)
    assert torch.equal(y[0], beta) and torch.equal(y[3], beta)
    assert y[1].isnan().all() and y[2].isnan().all()
    assert abs(float(rstd[0]) - 100.0) <= 1e-4 and float(mean[3]) == 3.0


@pytest.mark.parametrize("wgrad", [True, False])
def test_norm_no_rows(wgrad):
    x = torch.empty(0, 64, device="cuda")
    e = torch.empty(0, device="cuda")
    m.moe_lora_layernorm_forward(x, None, None, x, e, e)
    dg = torch.full((64,), 7.0, device="cuda") if wgrad else None
    m.moe_lora_layernorm_backward(x, None, e, e, x, None, x, dg, None, m.layernorm_scratch(0, 64) if wgrad else None)
    if wgrad:
        assert (dg == 0).all()


def test_norm_offsets_past_32_bits():
    """Rows of a buffer of more than 2^32 elements."""
    ld, n, rows = (1 << 30) + 8, 512, 5
    b = torch.empty(rows * ld, dtype=BF, device="cuda")
    x = b.as_strided((rows, n), (ld, 1))
    x.copy_(torch.randn(rows, n, generator=_gen(1), device="cuda"))
    xc = x.contiguous()
    y, yc = torch.empty_like(xc), torch.empty_like(xc)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    m.moe_lora_layernorm_forward(x, None, None, y, mean, rstd)
    m.moe_lora_layernorm_forward(xc, None, None, yc)
    assert torch.equal(y, yc)
    dy = torch.randn(rows, n, generator=_gen(2), device="cuda").bfloat16()
    dx, dxc = torch.empty_like(dy), torch.empty_like(dy)
    m.moe_lora_layernorm_backward(x, None, mean, rstd, dy, None, dx)
    m.moe_lora_layernorm_backward(xc, None, mean, rstd, dy, None, dxc)
    assert torch.equal(dx, dxc)


# ------------------------------------------------------------------ balance loss
def _balance(logits, ids, offsets, coef=0.01, dloss=None, grad=True, A=1):
    T, E = logits.shape
    d = m.make_dims(T=T, H=64, I=64, E=E, k=ids.shape[1], r=8, A=A)
    sc = m.balance_scratch(d).fill_(0xFF)
    loss = torch.full((A,), float("nan"), device="cuda")
    counts = torch.full((A, E), -9, dtype=torch.int32, device="cuda")
    prob = torch.full((A, E), float("nan"), device="cuda")
    dl = torch.full((T, E), float("nan"), device="cuda") if grad else None
    m.moe_lora_balance_loss(d, logits, ids, offsets, coef, loss, counts, prob, sc, dl, dloss)
    return loss, counts, prob, dl, m.moe_lora_balance_get_error(d, sc)


def _check_balance(logits, ids, offsets, got, coef=0.01, dloss=None):
    loss, counts, prob, dl, _ = got
    A = len(offsets) - 1
    wl, wc, wp, wd = ref.balance(logits.float().cpu(), ids.cpu(), offsets, coef, dloss)
    assert torch.equal(counts.cpu(), wc)
    # a probability: the exponent's argument (its rounding times its size) and exp, sum, quotient
    l = logits.float()
    span = torch.where(torch.isfinite(l), l, 0.0).abs().amax().item() * 2
    rel = (CHAIN + 2 * span + 16) * U32
    _within("prob", prob, wp, rel * wp + 1e-30)
    _within("loss", loss, wl, 2 * rel * wl + 1e-30)
    if dl is not None:
        E = logits.shape[1]
        f = wc.double() / wc.sum(1, keepdim=True).clamp(min=1)
        # |dl| <= g p max(f, s), s <= max f; each term to `rel`
        live = ((ids >= 0) & (ids < E)).any(1).cpu()
        p = torch.where(live[:, None], torch.softmax(l.double().cpu(), 1).nan_to_num(0.0), 0.0)
        tol = torch.zeros_like(wd)
        for a in range(A):
            lo, hi = offsets[a], offsets[a + 1]
            N = max(1, int(live[lo:hi].sum()))
            g = (1.0 if dloss is None else float(dloss[a])) * coef * E / N
            tol[lo:hi] = 2 * rel * g * p[lo:hi] * float(f[a].max())
        _within("dlogits", dl, wd, tol + 1e-30)
        assert (dl.cpu()[~live] == 0).all()


@pytest.mark.parametrize("T,E,k,dt,mask,pad", [
    (1, 1, 1, F32, 0.0, 0), (1, 16, 2, F32, 0.0, 0), (2, 3, 3, BF, 0.0, 0), (63, 8, 1, F32, 0.3, 0),
    (64, 60, 4, BF, 0.2, 4), (65, 127, 8, HF, 0.5, 1), (256, 16, 2, F32, 0.0, 0), (500, 256, 6, F32, 0.2, 0),
    (1030, 128, 8, BF, 0.9, 8), (333, 384, 8, F32, 0.2, 0), (200, 512, 32, HF, 0.1, 0), (130, 1024, 6, F32, 0.2, 12),
    (97, 1023, 3, F32, 0.2, 0), (3000, 33, 4, F32, 0.2, 3)])
def test_balance(T, E, k, dt, mask, pad):
    g = _gen(T + E)
    _, logits = _rows(T, E, E + pad, dt, g, scale=2.0)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :min(k, E)].to(torch.int32)
    if k > E:
        ids = torch.cat([ids, torch.full((T, k - E), -1, dtype=torch.int32, device="cuda")], 1)
    ids[torch.rand(ids.shape, generator=g, device="cuda") < mask] = -1
    ids = ids.contiguous()
    got = _balance(logits, ids, None)
    assert got[4] == 0
    _check_balance(logits, ids, [0, T], got)
    fwd = _balance(logits, ids, None, grad=False)
    assert all(torch.equal(a, b) for a, b in zip(fwd[:3], got[:3]))


def test_balance_many_tokens():
    """More tokens than one block's chunk per adapter slice; counts and the mean against whole-tensor sums."""
    T, E, k = 70001, 64, 4
    g = _gen(5)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    loss, counts, prob, dl, err = _balance(logits, ids, None)
    wc = torch.bincount(ids.flatten().long(), minlength=E)
    assert err == 0 and torch.equal(counts[0].long(), wc)
    p = torch.softmax(logits.double(), 1)
    f = wc.double() / (T * k)
    rel = (2 * CHAIN + 32) * U32
    _within("prob", prob[0], p.mean(0), rel * p.mean(0))
    _within("loss", loss[0], 0.01 * E * (f * p.mean(0)).sum(), 2 * rel * 0.02)
    want = 0.01 * E / T * p * (f - (p @ f)[:, None])
    _within("dlogits", dl, want, 2 * rel * 0.01 * E / T * p * f.max())


@pytest.mark.parametrize("dt", [F32, BF])
def test_balance_adapters_equal_their_own_runs(dt):
    """Ragged and empty adapter ranges; every adapter's results equal its standalone run bit for bit."""
    E, k = 96, 5
    offs = [0, 128, 128, 1280, 1408, 6400, 6700]
    T, A = offs[-1], len(offs) - 1
    g = _gen(9)
    logits = torch.randn(T, E, generator=g, device="cuda").to(dt)
    ids = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    ids[torch.rand(T, k, generator=g, device="cuda") < 0.3] = -1
    ids[128:1280] = -1  # an adapter without a live route
    ids = ids.contiguous()
    dloss = torch.rand(A, generator=g, device="cuda") + 0.5
    got = _balance(logits, ids, offs, dloss=dloss, A=A)
    small = [0, 128, 128, 1280, 1408]
    _check_balance(logits[:1408], ids[:1408], small,
                   (got[0][:4], got[1][:4], got[2][:4], got[3][:1408], 0), dloss=dloss)
    for a in range(A):
        lo, hi = offs[a], offs[a + 1]
        if hi == lo:
            assert float(got[0][a]) == 0 and (got[1][a] == 0).all() and (got[2][a] == 0).all()
            continue
        one = _balance(logits[lo:hi].clone(), ids[lo:hi].clone(), None, dloss=dloss[a:a + 1].clone())
        for x, y in zip(one[:4], (got[0][a:a + 1], got[1][a:a + 1], got[2][a:a + 1], got[3][lo:hi])):
            assert torch.equal(x, y)
    assert float(got[0][2]) == 0 and (got[3][128:1280] == 0).all()


@pytest.mark.parametrize("T,masked", [(256, 0), (256, 0.02), (4096, 0.2), (16_384, 0), (20_824, 0.2)])
def test_balance_gradient_of_even_counts(T, masked):
    """Every expert selected: the counts differ by masked routes alone, and the gradient is what their
    small differences leave.  Its error is relative to those, not to the counts; even counts give 0."""
    E = 8
    g = _gen(21)
    logits = torch.randn(T, E, generator=g, device="cuda").bfloat16()
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1).int()
    ids[torch.rand(T, E, generator=g, device="cuda") < masked] = -1
    _, counts, _, dl, err = _balance(logits, ids, [0, T])
    assert err == 0
    if not masked:
        assert (counts == T).all() and not dl.any()
        return
    _, wc, _, wd = ref.balance(logits.float().cpu(), ids.cpu(), [0, T], 0.01, None)
    assert torch.equal(counts.cpu(), wc)
    l = logits.double().cpu()
    live = (ids >= 0).any(1).cpu()
    f = (wc[0].double() / wc.sum() - 1 / E).abs()  # dl = g p (f_e - <p, f>) with f less 1/E as well
    p = torch.softmax(l, 1) * live[:, None]
    rel = (CHAIN + 4 * l.abs().amax() + 16) * U32  # as in _check_balance
    _within("dlogits", dl, wd, 2 * rel * 0.01 * E / int(live.sum()) * p * (f + (p * f).sum(1, keepdim=True)) + 1e-30)


def test_balance_masked_values():
    """-inf logits have no probability, a row of them nothing at all; rows without a live route are not
    looked at; out-of-range ids are dropped and flagged."""
    T, E = 70, 40
    g = _gen(2)
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[:, 7] = float("-inf")
    logits[3] = float("-inf")
    logits[4] = torch.finfo(F32).min
    ids = torch.randint(0, E, (T, 2), generator=g, device="cuda", dtype=torch.int32)
    ids[10:20] = -1
    logits[12], logits[13], logits[14] = float("nan"), float("inf"), float("-inf")
    ids[20, 0], ids[21, 1], ids[22] = E, -5, 1 << 30
    got = _balance(logits, ids, None)
    assert got[4] == m.MOE_LORA_DEV_BAD_ID
    fine = logits.clone()
    fine[10:20] = 0
    fine[4] = 0  # equal logits of any size: the same probabilities
    _check_balance(fine, ids, [0, T], got)
    finite7 = got[3][:, 7].clone()
    finite7[4] = 0  # the one row whose logit 7 is finite
    assert (got[3][3] == 0).all() and (finite7 == 0).all() and (got[3][10:20] == 0).all()
    none = _balance(logits, torch.full_like(ids, -1), None)
    assert float(none[0]) == 0 and (none[1] == 0).all() and (none[2] == 0).all() and (none[3] == 0).all()


def test_balance_nothing():
    loss, counts, prob, _, err = _balance(torch.empty(0, 16, device="cuda"),
                                          torch.empty(0, 2, dtype=torch.int32, device="cuda"), None)
    assert err == 0 and float(loss) == 0 and (counts == 0).all() and (prob == 0).all()


def test_balance_gradient_matches_differences():
    """dlogits against central differences of the loss with the counts held, in 64 bits."""
    T, E, h = 5, 12, 1e-4
    g = _gen(4)
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids = torch.topk(logits, 3, dim=1).indices.to(torch.int32).contiguous()
    dl = _balance(logits, ids, None, coef=1.0)[3]
    x = logits.double().cpu()
    f = ref.balance(x, ids.cpu(), [0, T], 1.0, None)[1][0].double() / (3 * T)
    loss = lambda l: E * (f * torch.softmax(l, 1).mean(0)).sum()  # noqa: E731
    want = torch.zeros(T * E).double()
    for i in range(T * E):
        d = torch.zeros(T * E).double()
        d[i] = h
        want[i] = (loss(x + d.view(T, E)) - loss(x - d.view(T, E))) / (2 * h)
    # second-order error h^2 times a third derivative below E, and fp32 arithmetic
    _within("dl", dl.flatten(), want, E * h * h + 1e-6)


def test_router_backward_with_the_balance_gradient():
    """dlogits, dW_r and grad-x gain the balance loss's part; without one the results are those of
    moe_lora_router_backward bit for bit."""
    from synth import make_router_inputs
    T, H, E, k = 300, 256, 64, 4
    inp = make_router_inputs(T, H, E, k, seed=1, device="cuda")
    d = m.make_dims(T, H, 256, E, k, 16)
    sc = m.router_scratch(d)
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w, lg = torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    m.moe_lora_router_forward(d, inp["x"], inp["Wr"], ids, w, lg, sc)
    dw = torch.randn(T, k, generator=_gen(1), device="cuda")
    aux = _balance(lg, ids, None, coef=5.0)[3]

    def back(fn, *a):
        dl, dWr = torch.empty(T, E, device="cuda"), torch.empty(E, H, device="cuda")
        dx = torch.zeros(T, H, dtype=BF, device="cuda")
        fn(d, inp["x"], inp["Wr"], ids, w, dw, *a, dl, dWr, dx, sc)
        assert m.moe_lora_router_get_error(sc) == 0
        return dl, dWr, dx

    old = back(m.moe_lora_router_backward)
    assert all(torch.equal(a, b) for a, b in zip(old, back(m.moe_lora_router_backward_aux, None)))
    dl, dWr, dx = back(m.moe_lora_router_backward_aux, aux)
    _within("dlogits", dl, old[0].double() + aux.double(), 2 * U32 * (old[0].abs() + aux.abs()) + 1e-30)
    b = dl.bfloat16().double()  # the operand of both products
    want = b.T @ inp["x"].double()
    _within("dWr", dWr, want, (T + 8) * U32 * (b.abs().T @ inp["x"].double().abs()))
    want = b @ inp["Wr"].double()
    _within("dx", dx, want, UNIT[BF] * want.abs() + (E + 8) * U32 * (b.abs() @ inp["Wr"].double().abs()))


# ------------------------------------------------------------------ AdamW
def _entry(n, p_dt, g_dt, eight, master, g, lr=1e-3, wd=0.0):
    w = 0.05 * torch.randn(n, generator=g, device="cuda")
    e = dict(p=w.to(p_dt), g=(0.01 * torch.randn(n, generator=g, device="cuda")).to(g_dt), lr=lr, weight_decay=wd)
    if master:
        e["master"] = w
    if eight:
        e.update(m=torch.zeros(n, dtype=torch.uint8, device="cuda"), v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                 m_scale=torch.zeros(-(-n // 256), device="cuda"), v_scale=torch.zeros(-(-n // 256), device="cuda"))
    else:
        e.update(m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda"))
    return e


def _values(codes, scale):
    return ref.e4m3_values()[codes.long().cpu()] * scale.double().cpu().repeat_interleave(256)[:codes.numel()]


def _moments(e):
    if "m_scale" not in e:
        return e["m"].double().cpu(), e["v"].double().cpu()
    return _values(e["m"], e["m_scale"]), _values(e["v"], e["v_scale"]) ** 2


SIZES = [1, 2, 7, 8, 255, 256, 257, 1000, 4096, 5003, 70001]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("p_dt,g_dt,master", [(F32, F32, False), (BF, F32, True), (HF, BF, True), (BF, BF, False),
                                              (F32, HF, False), (HF, HF, False)])
def test_adamw_steps(p_dt, g_dt, master, eight):
    """Five steps over tensors of many lengths, each checked from the state before it."""
    g = _gen(7)
    es = [_entry(n, p_dt, g_dt, eight, master, g, lr=1e-3 * (1 + i % 3), wd=0.1 * (i % 2)) for i, n in enumerate(SIZES)]
    ten = m.AdamWTensors(es)
    scale = torch.full((1,), 0.5, device="cuda")
    for step in range(1, 6):
        before = [(e["master" if master else "p"].double().cpu(), *_moments(e)) for e in es]
        for e in es:
            e["g"].copy_(0.01 * torch.randn(e["g"].numel(), generator=g, device="cuda"))
        m.moe_lora_adamw_step(ten, step, 0.9, 0.99, 1e-8, grad_scale=scale)
        for e, (w0, m0, v0) in zip(es, before):
            gr = e["g"].double().cpu() * 0.5
            w, mm, vv = ref.adamw32(w0, gr, m0, v0, step, 0.9, 0.99, 1e-8, e["lr"], e["weight_decay"])
            # moments: two products and a sum; the update: ten roundings of a quotient whose parts err by 4
            mt, vt = 4 * U32 * (m0.abs() + gr.abs()), 8 * U32 * vv
            um = e["lr"] * (mt / (1 - 0.9 ** step)) / ((vv / (1 - 0.99 ** step)).sqrt() + 1e-8)
            wt = 4 * U32 * w0.abs() + um + 16 * U32 * (w - w0).abs() + 8 * U32 * w.abs()
            if master:
                _within("master", e["master"], w, wt)
                assert torch.equal(e["p"], e["master"].to(p_dt))
            else:
                _within("p", e["p"], w, wt + UNIT[p_dt] * (w.abs() + wt) + TINY_OF[p_dt])
            gm, gv = _moments(e)
            if not eight:
                _within("m", gm, mm, mt)
                _within("v", gv, vv, vt)
                continue
            for got, want, sc, tol in ((gm, mm, e["m_scale"], mt), (gv.sqrt(), vv.sqrt(), e["v_scale"], 8 * U32 * vv.sqrt())):
                n = want.numel()
                s = sc.double().cpu().repeat_interleave(256)[:n]
                top = torch.nn.functional.pad(want.abs(), (0, -n % 256)).view(-1, 256).amax(1)
                _within("scale", sc, top / 448, 16 * U32 * top / 448 + mt.max() / 448)
                # half a step of E4M3: 2^-4 of the value, 2^-10 of the scale below 2^-6 of it
                _within("code", got, want, torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-5) + 2 * tol)


def test_adamw_eight_bit_rounding_is_nearest_even():
    """Zero gradient and beta 1 -> the stored moment is the old one times beta1, rounded to the nearest
    code (ties to even): checked code by code against all 256 values."""
    n = 4096
    g = _gen(8)
    e = _entry(n, F32, F32, True, False, g)
    e["g"].copy_(torch.randn(n, generator=g, device="cuda"))
    ten = m.AdamWTensors([e])
    m.moe_lora_adamw_step(ten, 1, 0.0, 0.0, 1e-8)  # m = g, r = |g|
    vals = ref.e4m3_values()
    keep = ~vals.isnan()
    codes = torch.arange(256)[keep]
    for c, s, sign in ((e["m"], e["m_scale"], 1), (e["v"], e["v_scale"], 0)):
        want = e["g"].cpu() if sign else e["g"].cpu().abs()
        top = want.abs().view(-1, 256).amax(1)
        assert torch.equal(s.cpu(), top * torch.tensor(1 / 448))  # fp32 products, as the header gives them
        x = (want.view(-1, 256) * (top.reciprocal() * 448)[:, None]).double().view(-1)
        dist = (x[:, None] - vals[keep][None, :]).abs()
        best = dist.amin(1, keepdim=True)
        even = (codes & 1) == 0
        near = (dist == best) & (even[None, :] | ((dist == best).sum(1, keepdim=True) == 1))
        got = torch.searchsorted(codes, c.cpu().long())
        assert near[torch.arange(n), got].all()


def test_adamw_special_values():
    """A non-finite gradient spoils its own element only, in 32 and in 8 bits; zero gradients leave zero
    states; blocks of zeros and of vanishing values are stored as zeros."""
    g = _gen(3)
    for eight in (False, True):
        a, b = (_entry(1000, BF, F32, eight, True, _gen(4)) for _ in range(2))
        a["g"][10], a["g"][300], a["g"][999] = float("nan"), float("inf"), float("-inf")
        b["g"][[10, 300, 999]] = 0.0
        z = _entry(300, F32, F32, eight, False, g, wd=0.0)
        z["g"].zero_()
        t = _entry(300, F32, F32, eight, False, g)
        t["g"].fill_(1e-36)
        keep = z["p"].clone()
        m.moe_lora_adamw_step(m.AdamWTensors([a, b, z, t]), 1)
        ok = torch.ones(1000, dtype=torch.bool, device="cuda")
        ok[[10, 300, 999]] = False
        for key in ("p", "master", "m", "v"):
            assert torch.equal(a[key][ok], b[key][ok]), (eight, key)
        assert a["master"][[10, 300, 999]].isnan().all()
        if eight:
            assert (a["m"][[10, 300, 999]] & 0x7F == 0x7F).all() and (a["v"][[10, 300, 999]] & 0x7F == 0x7F).all()
            assert torch.equal(a["m_scale"], b["m_scale"]) and torch.equal(a["v_scale"], b["v_scale"])
            assert (t["m_scale"] == 0).all() and (t["m"] == 0).all() and (t["v"] & 0x7F != 0x7F).all()
        assert torch.equal(z["p"], keep) and not z["m"].any() and not z["v"].any()


def test_adamw_many_tensors():
    """More tensors than one launch takes, both state kinds mixed: equal to one tensor at a time, bit for bit."""
    def make():
        g = _gen(6)
        return [_entry(1 + (37 * i) % 600, (F32, BF)[i % 2], F32, i % 3 == 0, i % 2 == 1, g, wd=0.01 * (i % 5))
                for i in range(800)]
    a, b = make(), make()
    m.moe_lora_launch_count(True)
    m.moe_lora_adamw_step(m.AdamWTensors(a), 3)
    assert m.moe_lora_launch_count(True) == 3
    for e in b:
        m.moe_lora_adamw_step(m.AdamWTensors([e]), 3)
    for x, y in zip(a, b):
        for key in x:
            assert not torch.is_tensor(x[key]) or torch.equal(x[key], y[key])


def test_adamw_scales_inside_an_array():
    """The block scales of several tensors in one array, at any multiple of four bytes."""
    def make():
        g = _gen(5)
        es = [_entry(n, BF, F32, True, True, g) for n in (257, 1000, 300, 64)]
        return es
    a, b = make(), make()
    ms, vs = torch.zeros(16, device="cuda"), torch.zeros(16, device="cuda")
    at = 1
    for e in b:
        k = e["m_scale"].numel()
        e["m_scale"], e["v_scale"] = ms[at:at + k], vs[at:at + k]
        at += k
    for step in (1, 2):
        m.moe_lora_adamw_step(m.AdamWTensors(a), step)
        m.moe_lora_adamw_step(m.AdamWTensors(b), step)
    for x, y in zip(a, b):
        assert all(torch.equal(x[k], y[k]) for k in ("p", "master", "m", "v", "m_scale", "v_scale"))


def test_adamw_empty_and_lr():
    e0 = dict(p=torch.empty(0, device="cuda"), g=torch.empty(0, device="cuda"), m=torch.empty(0, device="cuda"),
              v=torch.empty(0, device="cuda"))
    e1 = _entry(64, F32, F32, False, False, _gen(1))
    keep = e1["p"].clone()
    ten = m.AdamWTensors([e0, e1])
    ten.set_lr(0.0)
    m.moe_lora_adamw_step(ten, 1)
    assert torch.equal(e1["p"], keep) and e1["m"].any()
    m.moe_lora_adamw_step(m.AdamWTensors([]), 1)


def test_adamw_eight_bits_follow_32_bits():
    """A quadratic: both state kinds reach the minimum, the weights within a few percent of the way."""
    n, steps = 2048, 200
    g = _gen(12)
    target = torch.randn(n, generator=g, device="cuda")
    es = []
    for eight in (False, True):
        e = _entry(n, F32, F32, eight, False, _gen(13), lr=0.05)
        e["p"].zero_()
        es.append(e)
    ten = m.AdamWTensors(es)
    for s in range(1, steps + 1):
        for e in es:
            torch.sub(e["p"], target, out=e["g"])
        ten.set_lr(0.05 * (1 - s / (steps + 1)))
        m.moe_lora_adamw_step(ten, s, 0.9, 0.99)
    start = float(target.norm())
    assert float((es[0]["p"] - target).norm()) <= 0.05 * start
    assert float((es[1]["p"] - target).norm()) <= 0.10 * start


def test_training_calls_do_not_allocate_on_the_device():
    """No call allocates device memory: free memory is the same after a round of all of them."""
    x = torch.randn(64, 256, device="cuda").bfloat16()
    y, mean, rstd = torch.empty_like(x), torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    dg, db = torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
    sc = m.layernorm_scratch(64, 256)
    ten = m.AdamWTensors([_entry(3000, F32, F32, k, False, _gen(1)) for k in (False, True)])

    def calls():
        m.moe_lora_layernorm_forward(x, None, None, y, mean, rstd)
        m.moe_lora_layernorm_backward(x, None, mean, rstd, x, None, y, dg, db, sc)
        m.moe_lora_adamw_step(ten, 1)
        torch.cuda.synchronize()

    calls()
    free = torch.cuda.mem_get_info()[0]
    for _ in range(3):
        calls()
    assert torch.cuda.mem_get_info()[0] == free


def test_training_calls_in_a_graph():
    """Every call can be captured in a CUDA graph; a replay equals the call."""
    g = _gen(14)
    x = torch.randn(200, 512, generator=g, device="cuda").bfloat16()
    gamma, beta = torch.randn(512, generator=g, device="cuda"), torch.randn(512, generator=g, device="cuda")
    T, E, k = 200, 64, 4
    logits = torch.randn(T, E, generator=g, device="cuda")
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    d = m.make_dims(T=T, H=512, I=64, E=E, k=k, r=8)
    bsc, nsc = m.balance_scratch(d), m.layernorm_scratch(200, 512)
    out = dict(y=torch.empty_like(x), mean=torch.empty(200, device="cuda"), rstd=torch.empty(200, device="cuda"),
               dx=torch.empty_like(x), dg=torch.empty(512, device="cuda"), db=torch.empty(512, device="cuda"),
               loss=torch.empty(1, device="cuda"), counts=torch.empty(1, E, dtype=torch.int32, device="cuda"),
               prob=torch.empty(1, E, device="cuda"), dl=torch.empty(T, E, device="cuda"))

    def calls():
        m.moe_lora_layernorm_forward(x, gamma, beta, out["y"], out["mean"], out["rstd"])
        m.moe_lora_layernorm_backward(x, gamma, out["mean"], out["rstd"], out["y"], None, out["dx"], out["dg"],
                                      out["db"], nsc)
        m.moe_lora_balance_loss(d, logits, ids, None, 0.01, out["loss"], out["counts"], out["prob"], bsc, out["dl"])

    calls()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in out.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        for t in out.values():
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[n]) for n in out)
    assert math.isfinite(float(want["loss"]))


def test_training_example_learns():
    """The example's block: the loss falls, two runs agree bit for bit."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    shp = ex.Shape(T=300, H=512, I=256, E=16, k=2, r=16)
    losses, aux = ex.train(shp, 60)
    assert all(math.isfinite(v) for v in losses + aux)
    assert losses[-1] < 0.5 * losses[0], (losses[0], losses[-1])
    again, _ = ex.train(shp, 5)
    assert again == losses[:5]
