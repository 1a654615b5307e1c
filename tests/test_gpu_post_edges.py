"""Post-training operators at the ends of their arguments' ranges, against 64-bit definitions."""
import math

import pytest
import torch

import moe_expert_ffn_top_gb300 as m
import post_ref as ref
from post_ref import U32
from train_ops_ref import TINY_OF, UNIT

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from moe_expert_ffn_top_gb300 import _build
    _build.build()
    torch.cuda.set_device(0)
    yield


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _within(name, got, want, tol):
    off = (got.double() - want.double()).abs()
    assert (off <= tol).all(), (name, float((off - tol).max()), float(off.max()))


def _corrected(seq, T):
    out, at = [], 0
    for v in seq:
        at = min(max(at, v), T)
        out.append(at)
    return out


BAD_SEQ = [([0, 10, 5, 20, 30], 20), ([-4, 10, 12, 15, 20], 20), ([0, 1 << 60, 3, 4, 5], 20), ([0, 5, 9, -(1 << 60), 20], 20),
           ([0, 40, 50, 60, 3, 5, 8, 9, 80], 100), ([7, 30, 2, 9, 4, 60, 50, 55, 70], 90), ([30, 30, 29, 29, 28, 90, 10, 100, 90], 95), ([5, 2, 3], 50), ([0, 9000, 4000, 12000, 15000], 20000)]


def _check_offsets(seq, T, average=False, scratch=None):
    g = _gen(T + len(seq))
    lp, y = -torch.rand(T, generator=g, device="cuda"), torch.where(torch.rand(T, generator=g, device="cuda") < 0.2, -1, 1).to(torch.int32)
    P = len(seq) // 2
    good = _corrected(seq, T)
    scratch = m.preference_scratch(P) if scratch is None else scratch
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = torch.full((T,), 5.0, device="cuda")
    loss, stats, sl = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"), torch.empty(2 * P, device="cuda")
    beta = torch.tensor(0.1).item()
    m.moe_lora_preference_loss(lp, y, torch.tensor(seq, device="cuda"), None, loss, stats, scratch, beta=beta, average=average, seq_logp=sl,
                               dlogp=d, err=err)
    assert int(err) == (m.MOE_LORA_DEV_BAD_ID if good != list(seq) else 0)
    wl, ws, wt, wd = ref.preference(lp, y, good, None, [0, P], None, beta, "sigmoid", 0.0, 0.0, average)
    _within("sums", sl.cpu(), wt, 4 * U32 * wt.abs())
    assert abs(float(loss) - float(wl)) <= 1e-5 * (1 + abs(float(wl)))
    inside = ~torch.isnan(wd)
    assert (d.cpu()[~inside] == 5.0).all()
    # x is off by beta times the sums' rounding, and the loss's slope by that much
    size = float(wt.abs().max())
    _within("dlogp", d.cpu()[inside], wd[inside], beta / P * (32 * U32 + beta * 8 * U32 * size))


@pytest.mark.parametrize("seq,T", BAD_SEQ)
@pytest.mark.parametrize("average", [False, True])
def test_offsets_that_go_back(seq, T, average):
    """An offset below one before it, or past the tokens, counts as the nearest that is not; no token belongs to two pairs."""
    _check_offsets(seq, T, average)


@pytest.mark.parametrize("pairs", [200, 300, 2047, 2048, 2049, 5000, 9000])
def test_offsets_that_go_back_in_long_lists(pairs):
    """The largest offset so far may lie far before a pair's own."""
    g = torch.Generator().manual_seed(pairs)
    base = torch.randint(0, 6, (2 * pairs + 1,), generator=g).cumsum(0)
    T = int(base[-1])
    scratch = m.preference_scratch(pairs)  # a call does not see what an earlier list was
    for at, to in ((None, 0), (3, T // 3), (2 * pairs // 2, T * 3 // 4), (min(4095, 2 * pairs - 1), int(base[min(4095, 2 * pairs - 1)]) + 40), (2 * pairs - 1, 1 << 50),
                   (min(4096, 2 * pairs), 2), (None, 0)):
        seq = base.clone()
        if at is not None:
            seq[at] = to
        _check_offsets(seq.tolist(), T, scratch=scratch)


# ------------------------------------------------------------------ Muon
@pytest.mark.parametrize("shape", [(16, 200), (200, 16), (64, 300), (300, 64), (128, 640), (31, 90), (13, 77)])
def test_smallest_norms(shape):
    """A matrix whose |u| is at most 2^-60 counts as 0, one above takes a whole step, whatever eps leaves of it."""
    sizes = (-57.5, -58.5, -59.5, -59.9, -60.1, -60.5, -61.5, -62.5, -63.5, -64.5, -66.0, -72.0, -80.0)
    u = torch.randn(len(sizes), *shape, generator=_gen(sum(shape)), device="cuda").double()
    u = (u / u.flatten(1).norm(dim=1)[:, None, None] * (2.0 ** torch.tensor(sizes, dtype=torch.float64, device="cuda"))[:, None, None]).float()
    p, mom = torch.zeros_like(u), torch.zeros_like(u)
    t = m.MuonTensors([dict(p=p, g=u, m=mom, lr=-1.0, scale=1.0)])
    m.moe_lora_muon_step(t, momentum=0.0, nesterov=False, eps=1e-30)
    want = ref.newton_schulz(u, 5, (3.4445, -4.7750, 2.0315), 1e-30)
    assert torch.equal(mom, u)
    for i, size in enumerate(sizes):
        if size <= -60:
            assert (p[i] == 0).all(), size
        else:
            # 2e-4 as for the hardest spectra: at 2^-60 the squares' sums keep 2^-29 of |u|^2 in steps of the smallest number
            assert float((p[i].double() - want[i]).norm() / want[i].norm()) <= 2e-4, size


def test_norm_at_the_border():
    for eps in (1e-30, 1e-7):
        u = torch.tensor([2.0 ** -60, 2.0 ** -60 * (1 + 2.0 ** -20), -(2.0 ** -59)], device="cuda").view(3, 1, 1)
        p = torch.zeros_like(u)
        t = m.MuonTensors([dict(p=p, g=u, m=torch.zeros_like(u), lr=-1.0, scale=1.0)])
        m.moe_lora_muon_step(t, momentum=0.0, nesterov=False, eps=eps)
        want = ref.newton_schulz(u, 5, (3.4445, -4.7750, 2.0315), eps)
        assert float(p[0]) == 0.0
        assert ((p[1:].double() - want[1:]).abs() <= 2e-4 * want[1:].abs()).all()


@pytest.mark.parametrize("eps", [1e-7, 1e-3, 1.0])
@pytest.mark.parametrize("shape", [(16, 200), (200, 16), (64, 300), (300, 64), (128, 640), (31, 90), (1, 7)])
def test_norms_below_eps(shape, eps):
    """X keeps its relative precision where |u| is far below eps: neighbours of one tile, each of another size."""
    sizes = (30.0, 3.0, 1.0, 0.2, 0.03, 1e-3, 1e-5, 1e-7, 1e-10, 0.5)
    u = torch.randn(len(sizes), *shape, generator=_gen(sum(shape)), device="cuda").double()
    u = (u / u.flatten(1).norm(dim=1)[:, None, None] * (eps * torch.tensor(sizes, dtype=torch.float64, device="cuda"))[:, None, None]).float()
    small = u[[i for i, v in enumerate(sizes) if v <= 1e-5]].clone()  # whose singular values stay below 4 with the last coefficients
    for u, steps, coefs in ((u, 5, (3.4445, -4.7750, 2.0315)), (u, 1, (3.4445, -4.7750, 2.0315)), (small, 5, (8.0, -12.0, 4.9))):
        p = torch.zeros_like(u)
        t = m.MuonTensors([dict(p=p, g=u, m=torch.zeros_like(u), lr=-1.0, scale=1.0)])
        m.moe_lora_muon_step(t, momentum=0.0, nesterov=False, eps=eps, steps=steps, coefs=coefs)
        want = ref.newton_schulz(u, steps, coefs, eps)
        off = (p.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
        # factors to 2^-22 and fp32 sums, as for the hardest spectra
        assert float(off.max()) <= 2e-4, off.tolist()


# ------------------------------------------------------------------ preference loss
@pytest.mark.parametrize("kind,smooth", [("sigmoid", 0.0), ("sigmoid", 0.1), ("hinge", 0.0), ("squared", 0.0)])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("each,length", [(1, 5), (120, 7), (2, 3000)])
def test_infinite_log_probabilities(kind, smooth, average, each, length):
    """A masked token's log probability of -inf makes its sequence's sum -inf: losses and gradients by the definition.
    Adapters: chosen answers of that kind, rejected ones, and neither."""
    P, T = 3 * each, 2 * 3 * each * length
    lp = -torch.rand(T, generator=_gen(each), device="cuda") - 0.1
    y = torch.ones(T, dtype=torch.int32, device="cuda")
    seq = torch.arange(0, T + 1, length, device="cuda")
    rows = lp.view(P, 2, length)
    rows[:each, 0, length // 2] = -INF
    rows[each:2 * each, 1, length - 1] = -INF
    y.view(P, 2, length)[2 * each:, :, 0] = -1
    rows[2 * each:, :, 0] = -INF  # tokens without a target may hold anything
    beta = torch.tensor(0.2).item()
    smooth = torch.tensor(smooth).item()
    loss, stats = torch.full((3,), 9.0, device="cuda"), torch.full((3, 4), 9.0, device="cuda")
    sl, dl = torch.full((2 * P,), 9.0, device="cuda"), torch.full((T,), 9.0, device="cuda")
    m.moe_lora_preference_loss(lp, y, seq, None, loss, stats, m.preference_scratch(P, 3), beta=beta, kind=kind, label_smoothing=smooth, average=average,
                               pair_offsets=[0, each, 2 * each, P], seq_logp=sl, dlogp=dl)
    clean = torch.where(y > 0, lp, 0.0).double().view(P, 2, length).sum(2)
    n = torch.full((P, 1), length if average else 1, device="cuda")
    if average:
        n[2 * each:] = length - 1
    s = clean / n
    assert (sl.view(P, 2)[:each, 0] == -INF).all() and (sl.view(P, 2)[each:2 * each, 1] == -INF).all()
    fin = torch.isfinite(s)
    # a sum of `length` values in pairs of fp32 numbers, a division, one rounding
    _within("sums", sl.view(P, 2)[fin], s[fin], 4 * U32 * s[fin].abs())
    h = s[:, 0] - s[:, 1]
    x = beta * h
    if kind == "sigmoid":
        l = (1 - smooth) * torch.where(x < 0, -x, 0.0) + (smooth * torch.where(x > 0, x, 0.0) if smooth else 0.0) + torch.log1p(torch.exp(-x.abs()))
        d = beta * (smooth - 1 / (1 + torch.exp(x)))
    elif kind == "hinge":
        l, d = (1 - x).clamp(min=0), torch.where(x < 1, -beta, 0.0)
    else:
        l, d = (h - 0.5 / beta) ** 2, 2 * (h - 0.5 / beta)
    want = l.view(3, each).mean(1)
    for a in range(3):
        if math.isinf(float(want[a])):
            assert float(loss[a]) == INF, a
        else:
            assert abs(float(loss[a]) - float(want[a])) <= 1e-5 * (1 + abs(float(want[a]))), a
    assert float(stats[0, 0]) == 0 and abs(float(stats[1, 0]) - 1) <= 4 * U32 and float(stats[0, 1]) == -INF and float(stats[1, 2]) == -INF
    assert float(stats[0, 3]) == -INF and float(stats[1, 3]) == INF
    assert torch.isfinite(stats[2]).all() and torch.isfinite(stats[0, 2]) and torch.isfinite(stats[1, 1])
    g = (d / each)[:, None] / n
    g = torch.stack([g[:, 0], -g[:, 0]], 1)[:, :, None].expand(P, 2, length)
    g = torch.where(y.view(P, 2, length) > 0, g, 0.0)
    got = dl.view(P, 2, length).double()
    # by its formula: sigma, two products, a division; (h - 1 / (2 beta)) for the squared kind
    assert (torch.isnan(got) == False).all() and torch.equal(torch.isinf(got), torch.isinf(g))  # noqa: E712
    assert (torch.sign(got) == torch.sign(g)).all()
    f = torch.isfinite(g)
    assert ((got[f] - g[f]).abs() <= 2e-5 * g[f].abs() + 1e-6 / each).all()


# ------------------------------------------------------------------ logits far from 0
# type, common offset, spread around it, inverse temperature
FAR = [(F32, -1e6, 3.0, 1.0), (F32, 1e6, 3.0, 1.0), (F32, 3e7, 30.0, 1.0), (F32, -2e7, 30.0, 0.9), (BF, -12.0, 3.0, 1e5), (BF, 0.0, 3.0, 1e6), (BF, -9.0, 2.0, 1e6),
       (HF, -5.0, 1.0, 1e6), (HF, 3e4, 1e3, 1e6), (F32, -300.0, 20.0, 1e5), (F32, 3e9, 3e3, 1.0), (F32, -3e9, 3e3, 1.0), (F32, 3e9, 3e3, 1.3),
       (F32, 1e12, 1e6, 1.7), (BF, 1e30, 1e28, 1.0), (BF, -1e30, 1e28, 1.0), (F32, 4e10, 1e6, 1e-6), (F32, -2e37, 1e31, 1.0), (F32, 5e37, 1e33, 1.0)]


def _far_rows(rows, n, dt, offset, spread, seed):
    """Rows around an offset; in some, two entries share the largest value, and some have masked entries."""
    g = _gen(seed)
    x = (offset + spread * torch.randn(rows, n, generator=g, device="cuda").double()).to(dt)
    y = torch.randint(0, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
    top = x.argmax(1)
    y[::3] = top[::3].to(torch.int32)
    x[1::4, 3 % n] = x.amax(1)[1::4]
    x[2::4, n // 2:] = torch.finfo(dt).min
    x[3::4, : n // 2] = -INF
    y[2::4] %= n // 2
    y[3::4] = y[3::4] % (n - n // 2) + n // 2
    y[rows // 2] = -1
    return g, x, y


def _tokens(x, y, it):
    """ref.tokens, with entries of -inf as such, and one rounding more in every exponent than it allows (from x c of 2^31
    on a target's distance from the largest logit is formed first, then multiplied)."""
    z = x.double() * it
    r = ref.tokens(torch.where(torch.isinf(x), torch.finfo(F32).min, x.double()), y, it)
    p = r["p"]
    far = torch.where(p > 0, (z.amax(1, keepdim=True) - z).abs(), 0.0)
    one = U32 * (p * far).sum(1)
    r["tol"]["p"] = r["tol"]["p"] + U32 * far + one[:, None]
    r["tol"]["logp"] = r["tol"]["logp"] + one + U32 * torch.where(torch.isfinite(r["logp"]), r["logp"].abs(), 0.0)
    r["tol"]["lse"] = r["tol"]["lse"] + one
    r["tol"]["entropy"] = r["tol"]["entropy"] + one + U32 * (p * far * far).sum(1)
    return r


@pytest.mark.parametrize("rows,n", [(9, 300), (9, 5000), (5, 40000), (130, 5003), (2500, 1501)])
@pytest.mark.parametrize("dt,offset,spread,it", FAR)
def test_far_logits(rows, n, dt, offset, spread, it):
    """Softmax does not depend on a common offset: log probabilities, entropies, policy loss and its gradient."""
    it = torch.tensor(it).item()
    g, x, y = _far_rows(rows, n, dt, offset, spread, rows + n)
    r = _tokens(x, y, it)
    out = [torch.full((rows,), 9.0, device="cuda") for _ in range(3)]
    m.moe_lora_token_logp_forward(x, y, *out, inv_temp=it)
    for name, got in zip(("logp", "lse", "entropy"), out):
        _within(name, got, torch.where(r["ok"], r[name], 0.0), torch.where(r["ok"], r["tol"][name], 0.0))
    alone = torch.full((rows,), 9.0, device="cuda")
    m.moe_lora_token_logp_forward(x, y, alone, inv_temp=it)
    _within("logp alone", alone, torch.where(r["ok"], r["logp"], 0.0), torch.where(r["ok"], r["tol"]["logp"], 0.0))
    # the ratio is near 1 for half of the rows, and far below its border for the others
    lp = r["logp"].clamp(-1e30, 0)
    old = (lp + 0.1 * torch.randn(rows, generator=g, device="cuda").clamp(-1, 1)).float()
    old[1::2] = -0.5 * torch.rand(rows, generator=g, device="cuda")[1::2]
    adv = torch.rand(rows, generator=g, device="cuda") + 0.1
    r["logp"] = lp
    # ratios that fp32 holds, of log probabilities that fp32 holds
    keep = ((out[0].double() - old.double()).abs() < 60) & (r["tol"]["logp"] < 1e-3)
    w = torch.where(keep, torch.rand(rows, generator=g, device="cuda") + 0.1, 0.0)
    loss, stats, d = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"), torch.full_like(x, 9.0)
    m.moe_lora_policy_loss(x, y, adv, old, None, loss, stats, m.policy_scratch(rows), weight=w, dlogits=d, inv_temp=it, clip_low=1.0, clip_high=1e30)
    wl, ws, wd, lt, st, dtol = ref.policy(r, adv, old, None, w, [0, rows], None, it, 1.0, 1e30, 0.0)
    _within("loss", loss, wl, lt)
    _within("stats", stats, ws, st)
    big = torch.finfo(dt).max
    wd = wd.clamp(-big, big)
    # an exponential below 2^-126 is 0, and the sum at least 2^-65 (the reference may miss the maximum by 64, half a
    # unit of fp32 below 2^31, and is rounded up): a probability below 2^-61 may be lost
    lost = 2.0 ** -61 * (w * adv * it).double() * torch.exp((lp - old.double()).clamp(max=60))
    _within("dlogits", d.clamp(-big, big), wd, dtol + UNIT[dt] * (wd.abs() + dtol) + torch.where(wd != 0, TINY_OF[dt] + lost[:, None], 0.0))


@pytest.mark.parametrize("rows,n,pad", [(9, 300, 0), (9, 5000, 3), (5, 40000, 0), (130, 5003, 0), (2500, 1501, 0)])
@pytest.mark.parametrize("dt,offset,spread,it", FAR)
def test_far_logits_backward(rows, n, pad, dt, offset, spread, it):
    """The gradient where fp32 holds lse coarsely, against the definition's own lse; into strided rows and in place."""
    it = torch.tensor(it).item()
    g, x, y = _far_rows(rows, n, dt, offset, spread, rows + n)
    buf = torch.full((rows, n + pad), 7.0, dtype=dt, device="cuda")
    buf[:, :n] = x
    x = buf[:, :n]
    r = _tokens(x, y, it)
    lp, lse = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    m.moe_lora_token_logp_forward(x, y, lp, lse, inv_temp=it)
    dlogp = torch.randn(rows, generator=g, device="cuda")
    dlogp[rows // 3] = 0.0
    d = torch.full((rows, n + pad), 5.0, dtype=dt, device="cuda")
    m.moe_lora_token_logp_backward(x, y, lse, dlogp, d[:, :n], inv_temp=it)
    coef = torch.where(r["ok"], dlogp.double() * it, 0.0)[:, None]
    hot = torch.zeros_like(r["p"]).scatter_(1, r["y"], 1.0)
    want = torch.where(coef != 0, coef * (hot - r["p"]), 0.0)
    tol = coef.abs() * (r["p"] * r["tol"]["p"] + 3 * U32 * (hot + r["p"]))
    tol = tol + 2.0 ** -61 * coef.abs()  # as above
    # |lse| below 1,024 is used as saved
    tol = tol + coef.abs() * r["p"] * torch.where(r["lse"].abs() < 1025, r["tol"]["lse"], 0.0)[:, None]
    big = torch.finfo(dt).max
    want = want.clamp(-big, big)
    _within("dlogits", d[:, :n].clamp(-big, big), want, torch.where(coef != 0, tol + UNIT[dt] * (want.abs() + tol) + TINY_OF[dt], 0.0))
    if pad:
        assert (d[:, n:] == 5.0).all()
    m.moe_lora_token_logp_backward(x, y, lse, dlogp, x, inv_temp=it)
    assert torch.equal(x, d[:, :n])
    if pad:
        assert (buf[:, n:] == 7.0).all()


@pytest.mark.parametrize("dt", [F32, BF, HF])
@pytest.mark.parametrize("rows,n", [(6, 300), (6, 5000), (5, 40000), (2500, 1501)])
def test_masked_rows_backward(rows, n, dt):
    """Rows of nothing but masks are uniform in the backward as in the forward and the policy loss."""
    for it in (1.0, 0.25, 1e4):
        x = torch.randn(rows, n, generator=_gen(n), device="cuda").to(dt)
        x[0::3] = torch.finfo(dt).min
        x[1::3] = -INF
        y = torch.randint(0, n, (rows,), generator=_gen(n + 1), device="cuda", dtype=torch.int32)
        lp, lse, ent = (torch.empty(rows, device="cuda") for _ in range(3))
        m.moe_lora_token_logp_forward(x, y, lp, lse, ent, inv_temp=it)
        dlogp = torch.randn(rows, generator=_gen(3), device="cuda")
        d, dp = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
        m.moe_lora_token_logp_backward(x, y, lse, dlogp, d, inv_temp=it)
        flat = torch.arange(rows, device="cuda") % 3 < 2
        hot = torch.zeros(rows, n, dtype=torch.float64, device="cuda").scatter_(1, y.long()[:, None], 1.0)
        coef = dlogp.double()[:, None] * it
        want = coef * (hot - 1.0 / n)
        # n equal terms: their sum, a quotient, two products and the output's rounding
        tol = coef.abs() * (hot + 1.0 / n) * 300 * U32
        _within("masked", d[flat], want[flat], (tol + UNIT[dt] * (want.abs() + tol) + TINY_OF[dt])[flat])
        assert (ent[flat].double() - math.log(n)).abs().max() <= 1e-4
        assert ((lp[0::3].double() + math.log(n)).abs() <= 1e-5 * math.log(n)).all() and (lp[1::3] == -INF).all()
        # the policy loss's gradient on the same rows: ratio 1 and advantages that make the same factor
        m.moe_lora_policy_loss(x, y, -dlogp, lp.nan_to_num(neginf=0.0), None, torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"),
                               m.policy_scratch(rows), weight=torch.ones(rows, device="cuda"), dlogits=dp, inv_temp=it)
        i = slice(0, rows, 3)
        _within("policy", dp[i], want[i], (tol + UNIT[dt] * (want.abs() + tol) + TINY_OF[dt])[i])


# ------------------------------------------------------------------ sums over tokens and pairs
# Pairs of fp32 numbers: a chain of k <= 24 additions leaves at most k 2^-24 of the terms' size in the lower number, whose
# own additions are each off by 2^-24 of that: k^2 2^-48 < 2^-38 in all.
PAIRS_KEEP = 2.0 ** -38


@pytest.mark.parametrize("rows,adapters", [(64, 1), (50, 3), (700, 1), (20000, 2), (30000, 1)])
def test_policy_sums_that_cancel(rows, adapters):
    """Terms of either sign: with the ratios at 1 they are the advantages, and only their sum's rounding is left."""
    n = 16
    g = _gen(rows)
    x = torch.randn(rows, n, generator=g, device="cuda")
    y = torch.randint(0, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
    adv = torch.randn(rows, generator=g, device="cuda") * 2.0 ** torch.randint(-8, 13, (rows,), generator=g, device="cuda")
    half = rows // 2
    adv[half:2 * half] = -adv[:half].flip(0) + 1e-3 * torch.rand(half, generator=g, device="cuda")
    offs = [0] + [rows * a // adapters // 2 * 2 for a in range(1, adapters)] + [rows]
    loss, stats, lp = torch.empty(adapters, device="cuda"), torch.empty(adapters, 4, device="cuda"), torch.empty(rows, device="cuda")
    w = torch.full((rows,), 2.0 ** -12, device="cuda")
    kw = dict(weight=w, adapter_offsets=offs if adapters > 1 else None, logp=lp)
    m.moe_lora_policy_loss(x, y, adv, torch.zeros(rows, device="cuda"), None, loss, stats, m.policy_scratch(rows, adapters), **kw)
    old = lp.clone()
    m.moe_lora_policy_loss(x, y, adv, old, None, loss, stats, m.policy_scratch(rows, adapters), **kw)
    assert torch.equal(old, lp)
    for a in range(adapters):
        v = -adv[offs[a]:offs[a + 1]].double() * 2.0 ** -12
        assert abs(float(loss[a]) - float(v.sum())) <= 2 * U32 * abs(float(v.sum())) + PAIRS_KEEP * float(v.abs().sum()), a
        assert abs(float(stats[a, 2]) - (offs[a + 1] - offs[a]) * 2.0 ** -12) <= U32 * rows * 2.0 ** -12


@pytest.mark.parametrize("pairs", [16, 256, 512, 16384])
def test_preference_sums_that_cancel(pairs):
    g = _gen(pairs)
    lp = -torch.rand(2 * pairs, generator=g, device="cuda") * 2.0 ** torch.randint(0, 12, (2 * pairs,), generator=g, device="cuda")
    v = lp.view(pairs, 2)
    half = pairs // 2
    v[half:, 0], v[half:, 1] = v[:half, 1].flip(0), v[:half, 0].flip(0) + 1e-4
    h32 = v[:, 0] - v[:, 1]
    loss, stats = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
    m.moe_lora_preference_loss(lp, torch.ones(2 * pairs, dtype=torch.int32, device="cuda"), torch.arange(2 * pairs + 1, device="cuda"), None, loss, stats,
                               m.preference_scratch(pairs), beta=0.5)
    for got, want in ((stats[0, 1], 0.5 * v[:, 0].double()), (stats[0, 2], 0.5 * v[:, 1].double()), (stats[0, 3], h32.double())):
        assert abs(float(got) - float(want.mean())) <= 2 * U32 * abs(float(want.mean())) + PAIRS_KEEP * float(want.abs().mean())


# ------------------------------------------------------------------ a token's terms
@pytest.mark.parametrize("rows,n", [(8, 200), (8, 9000), (300, 9000)])
def test_ratio_past_fp32_without_advantage(rows, n):
    """exp(logp - old) may pass fp32's range; times an advantage of 0 it has no part in loss and gradient."""
    x = torch.randn(rows, n, generator=_gen(rows), device="cuda")
    y = torch.arange(rows, device="cuda", dtype=torch.int32) % n
    adv = torch.randn(rows, generator=_gen(2), device="cuda")
    old = torch.full((rows,), -9.0, device="cuda")
    far = torch.arange(rows, device="cuda") % 4 == 1
    adv[far], old[far] = 0.0, -200.0
    near = torch.where(far, -9.0, old)
    res = []
    for o in (old, near):
        loss, stats, d = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"), torch.full_like(x, 9.0)
        m.moe_lora_policy_loss(x, y, adv, o, None, loss, stats, m.policy_scratch(rows), dlogits=d)
        res.append((loss, stats[0, :2], stats[0, 3], d))
    assert all(torch.equal(a, b) for a, b in zip(*res)) and torch.isfinite(res[0][0]).all()
    assert (res[0][3][far] == 0).all()


@pytest.mark.parametrize("rows,n", [(8, 200), (8, 9000), (300, 9000)])
def test_kl_without_weight(rows, n):
    """With kl_coef 0 a reference model only reports: loss and gradient are those without it, however far it lies."""
    x = torch.randn(rows, n, generator=_gen(rows), device="cuda")
    y = torch.arange(rows, device="cuda", dtype=torch.int32) % n
    x[1, 1] = -INF  # a masked target: its logp is -inf, its ratio 0
    adv, old = torch.randn(rows, generator=_gen(2), device="cuda"), torch.full((rows,), -9.0, device="cuda")
    rlp = torch.full((rows,), -9.0, device="cuda")
    res = []
    for r in (rlp + 150.0, rlp, None):
        loss, stats, d = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"), torch.full_like(x, 9.0)
        m.moe_lora_policy_loss(x, y, adv, old, r, loss, stats, m.policy_scratch(rows), dlogits=d)
        res.append((loss, stats[0, 1:], d))
        if r is not None:
            assert float(stats[0, 0]) == INF
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(*res)) and torch.isfinite(res[0][2]).all() and torch.isfinite(res[0][0]).all()


@pytest.mark.parametrize("dt", [F32, BF, HF])
@pytest.mark.parametrize("rows,n", [(300, 200), (40, 5003), (20, 40000)])
def test_log_probabilities_of_certain_tokens(rows, n, dt):
    """Never above 0; entropies never below it."""
    g = _gen(n)
    x = torch.randn(rows, n, generator=g, device="cuda")
    y = torch.randint(0, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
    at = torch.arange(rows, device="cuda")
    x[at, y.long()] += torch.linspace(5, 60, rows, device="cuda")
    x = x.to(dt)
    for it in (1.0, 0.7, 30.0):
        it = torch.tensor(it).item()
        lp, ent = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        m.moe_lora_token_logp_forward(x, y, lp, None, ent, inv_temp=it)
        r = ref.tokens(x, y, it)
        assert (lp <= 0).all() and (ent >= 0).all(), (float(lp.max()), float(ent.min()))
        _within("logp", lp, r["logp"], r["tol"]["logp"])
        _within("entropy", ent, r["entropy"], r["tol"]["entropy"])


@pytest.mark.parametrize("rows,n", [(8, 200), (8, 9000), (300, 9000)])
def test_weight_zero_whatever_its_values(rows, n):
    """Tokens of weight 0 may hold anything in every input; the others' results are those of a batch without them."""
    x = torch.randn(rows, n, generator=_gen(rows), device="cuda")
    y = torch.arange(rows, device="cuda", dtype=torch.int32) % n
    adv, old = torch.randn(rows, generator=_gen(2), device="cuda"), torch.full((rows,), -9.0, device="cuda")
    rlp, w = old + 0.3, torch.rand(rows, generator=_gen(3), device="cuda") + 0.1
    off = torch.arange(rows, device="cuda") % 4 == 2
    w[off] = 0.0
    res = []
    for bad in (False, True):
        a, o, r, v, t = adv.clone(), old.clone(), rlp.clone(), x.clone(), y.clone()
        if bad:
            a[off], o[off], r[off] = math.nan, -INF, INF
            v[off] = torch.where(torch.rand(n, generator=_gen(5), device="cuda") < 0.5, INF, math.nan)
        else:
            t[off] = -1
        loss, stats, d = torch.empty(2, device="cuda"), torch.empty(2, 4, device="cuda"), torch.full_like(v, 9.0)
        m.moe_lora_policy_loss(v, t, a, o, r, loss, stats, m.policy_scratch(rows, 2), weight=w, adapter_offsets=[0, rows // 2, rows], kl_coef=0.1, dlogits=d)
        res.append((loss, stats, d))
    assert all(torch.equal(a, b) for a, b in zip(*res)) and all(torch.isfinite(v).all() for v in res[1])


@pytest.mark.parametrize("dt", [F32, BF, HF])
@pytest.mark.parametrize("rows,n,adapters", [(300, 5003, 3), (2500, 1501, 2), (70, 40000, 4), (40, 300, 1)])
def test_masked_vocabulary_in_the_policy_gradient(rows, n, adapters, dt):
    """Masked entries (-inf and the type's lowest value) and masked targets, with counted means and several adapters; in place too."""
    g = _gen(rows)
    x = (2 * torch.randn(rows, n, generator=g, device="cuda")).to(dt)
    y = torch.randint(0, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
    hide = torch.rand(rows, n, generator=g, device="cuda") < 0.5
    hide.scatter_(1, y.long()[:, None], False)
    x = torch.where(hide, torch.where(torch.arange(rows, device="cuda")[:, None] % 2 == 0, -INF, torch.finfo(dt).min), x.float()).to(dt)
    y[5::7] = -1
    gone = torch.arange(rows, device="cuda") % 11 == 3
    x[gone, y.clamp(min=0)[gone].long()] = -INF  # masked targets: logp -inf, ratio 0
    r = _tokens(x, y, 1.0)
    gone = gone & (y >= 0)
    old = (torch.where(gone, -8.0, r["logp"]) + 0.1 * torch.randn(rows, generator=g, device="cuda")).float()
    adv = torch.randn(rows, generator=g, device="cuda")
    offs = [0] + [rows * (a + 1) // adapters - 1 for a in range(adapters - 1)] + [rows]
    loss, stats, d = torch.empty(adapters, device="cuda"), torch.empty(adapters, 4, device="cuda"), torch.full_like(x, 9.0)
    lp = torch.empty(rows, device="cuda")
    kw = dict(adapter_offsets=offs if adapters > 1 else None, logp=lp)
    m.moe_lora_policy_loss(x, y, adv, old, None, loss, stats, m.policy_scratch(rows, adapters), dlogits=d, **kw)
    assert (lp[gone] == -INF).all()
    r["logp"] = torch.where(gone, -1e5, r["logp"])  # a ratio of 0 in 64 bits too
    r["tol"]["logp"] = torch.where(gone, 0.0, r["tol"]["logp"])
    low, high = 0.2, 0.2
    wl, ws, wd, lt, st, dtol = ref.policy(r, adv, old, None, None, offs, None, 1.0, low, high, 0.0)
    _within("loss", loss, wl, lt)
    _within("stats", stats, ws, st)
    _within("dlogits", d, wd, torch.where(wd != 0, dtol + UNIT[dt] * (wd.abs() + dtol) + TINY_OF[dt], dtol))
    assert (d[hide] == 0).all() and (d[gone] == 0).all()
    x2 = x.clone()
    m.moe_lora_policy_loss(x2, y, adv, old, None, loss, stats, m.policy_scratch(rows, adapters), dlogits=x2, **kw)
    assert torch.equal(x2, d)


def test_edges_captured_and_on_another_stream():
    """Far rows, coarse lse, bad offsets and small norms replayed from a graph: equal bits to eager calls, word and workspace reset."""
    T, n = 130, 9000
    x = torch.randn(T, n, generator=_gen(1), device="cuda")
    x[::3] *= 1e10
    x[1::3] -= 1e6
    x[2::6] = -INF
    y = torch.randint(0, n, (T,), generator=_gen(2), device="cuda", dtype=torch.int32)
    seq = torch.arange(0, T + 1, 10, device="cuda")[:13].clone()
    seq[4] = 3
    u = torch.randn(5, 16, 90, generator=_gen(3), device="cuda") * torch.tensor([1e-25, 1e-12, 1e-8, 1.0, 1e8], device="cuda")[:, None, None]
    sc, err = m.preference_scratch(6), torch.zeros(1, dtype=torch.int32, device="cuda")

    def buffers():
        z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        b = dict(lp=z(T), lse=z(T), ent=z(T), loss=z(1), stats=z(1, 4), sl=z(12), dl=z(T), d=torch.zeros_like(x), p=torch.zeros_like(u), m=torch.zeros_like(u))
        return b, m.MuonTensors([dict(p=b["p"], g=u, m=b["m"], lr=0.5)])

    def call(b, t):
        m.moe_lora_token_logp_forward(x, y, b["lp"], b["lse"], b["ent"])
        b["lp"].clamp_(min=-50)
        m.moe_lora_preference_loss(b["lp"], y, seq, None, b["loss"], b["stats"], sc, seq_logp=b["sl"], dlogp=b["dl"], err=err)
        m.moe_lora_token_logp_backward(x, y, b["lse"], b["dl"], b["d"])
        m.moe_lora_muon_step(t)
    want, got = buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(*got)
    torch.cuda.current_stream().wait_stream(side)
    call(*want)
    assert all(torch.equal(want[0][k], got[0][k]) for k in want[0]) and int(err) == m.MOE_LORA_DEV_BAD_ID
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(*got)
    for to in (3, 40, 1 << 50, 40):
        seq[4] = to
        err.zero_()
        x[5:9].normal_(generator=_gen(to % 1000))
        graph.replay()
        bits = int(err)
        err.zero_()
        call(*want)
        assert bits == int(err) == (0 if to == 40 else m.MOE_LORA_DEV_BAD_ID)
        assert all(torch.equal(want[0][k], got[0][k]) for k in want[0]) and torch.isfinite(want[0]["d"]).all()


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Before any launch: calls go to the current device."""
    x, y, v = torch.zeros(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, device="cuda")
    one, four, seq = torch.zeros(1, device="cuda"), torch.zeros(1, 4, device="cuda"), torch.tensor([0, 2, 4], device="cuda")
    psc, fsc = m.policy_scratch(4), m.preference_scratch(1)
    t = m.MuonTensors([dict(p=x.clone(), g=x, m=x.clone())])
    calls = [lambda: m.moe_lora_token_logp_forward(x, y, v), lambda: m.moe_lora_token_logp_backward(x, y, v, v, x),
             lambda: m.moe_lora_policy_loss(x, y, v, v, None, one, four, psc), lambda: m.moe_lora_preference_loss(v, y, seq, None, one, four, fsc),
             lambda: m.moe_lora_muon_step(t)]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
