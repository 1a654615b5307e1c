"""GPU tests of the token log probabilities, the policy loss and the preference loss against
64-bit definitions.

Tolerances are the rounding of the output's type plus, for the fp32 arithmetic behind it, one
rounding unit per operation and per addition of the longest chain (post_ref)."""
import math

import pytest
import torch

import moe_expert_ffn_top_gb300 as m
import post_ref as ref
from post_ref import CHAIN, U32
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
    got, want = got.double(), want.double().to(got.device)
    tol = tol.to(got.device) if torch.is_tensor(tol) else tol
    assert torch.isfinite(got).all(), name
    off = (got - want).abs()
    assert (off <= tol).all(), (name, float((off / tol).max()))


def _poisoned(scratch):
    """A workspace whose contents do not matter, but for the 16 bytes that are cleared once."""
    scratch[16:].fill_(0xFF)
    return scratch


def _inputs(rows, n, dt, pad, masked, seed, spread=3.0):
    g = _gen(seed)
    buf = torch.full((rows, n + pad), float("nan"), dtype=dt, device="cuda")
    buf[:, :n] = (spread * torch.randn(rows, n, generator=g, device="cuda") + 1.5).to(dt)
    targets = torch.randint(0, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
    targets[torch.rand(rows, generator=g, device="cuda") < masked] = -1
    return g, buf, buf[:, :n], targets


SHAPES = [  # rows, n, type, columns between rows, masked, inv_temp
    (1, 1, F32, 0, 0, 1.0), (3, 2, BF, 0, 0, 1.0), (5, 7, HF, 1, 0.3, 1.3), (9, 100, BF, 0, 0.3, 1.0), (1, 32000, BF, 0, 0, 1.25),
    (4, 513, F32, 3, 0.2, 0.5), (1000, 129, BF, 1, 0.5, 1.0), (33, 1024, HF, 0, 0, 2.0), (300, 4096, F32, 0, 0.1, 1.0),
    (7, 4097, BF, 0, 0.1, 1.0), (300, 4095, HF, 2, 0.4, 0.7), (170, 8192, BF, 8, 0, 1.0), (160, 16385, BF, 0, 0.1, 1.0), (40, 50257, HF, 0, 0.3, 1.0),
    (170, 33000, BF, 5, 0.1, 1.0), (3, 65536, F32, 0, 0, 1.0), (20, 131072, BF, 0, 0.1, 1.0), (156, 70001, F32, 0, 0.6, 1.0),
    (3, 262144, BF, 0, 0, 1.0), (2, 524288, HF, 0, 0, 1.0), (2, 524287, F32, 1, 0, 1.0), (50, 151936, BF, 0, 0.2, 0.9),
]


@pytest.mark.parametrize("rows,n,dt,pad,masked,it", SHAPES)
def test_token_logp(rows, n, dt, pad, masked, it):
    g, buf, x, y = _inputs(rows, n, dt, pad, masked, rows * 3 + n)
    out = [torch.full((rows,), float("nan"), device="cuda") for _ in range(3)]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.moe_lora_token_logp_forward(x, y, *out, inv_temp=it, err=err)
    alone = torch.full((rows,), float("nan"), device="cuda")
    m.moe_lora_token_logp_forward(x, y, alone, inv_temp=it)
    r = ref.tokens(x, y, torch.tensor(it, dtype=F32).item())
    for name, got in zip(("logp", "lse", "entropy"), out):
        _within(name, got, torch.where(r["ok"], r[name], 0.0), torch.where(r["ok"], r["tol"][name], 0.0))
    _within("logp alone", alone, torch.where(r["ok"], r["logp"], 0.0), torch.where(r["ok"], r["tol"]["logp"], 0.0))
    assert int(err) == 0
    # backward, into strided rows and in place
    dlogp = torch.randn(rows, generator=g, device="cuda")
    dlogp[rows // 2] = 0.0
    db = torch.full((rows, n + pad), 5.0, dtype=dt, device="cuda")
    lse = out[1]
    m.moe_lora_token_logp_backward(x, y, lse, dlogp, db[:, :n], inv_temp=it)
    it32 = torch.tensor(it, dtype=F32).item()
    z = x.double() * it32
    p = torch.exp(z - lse.double()[:, None])
    coef = torch.where(r["ok"], dlogp.double() * it32, 0.0)[:, None]
    hot = torch.zeros_like(p).scatter_(1, r["y"], 1.0)
    want = torch.where(coef != 0, coef * (hot - p), 0.0)
    far = (z - lse.double()[:, None]).abs()
    tol = coef.abs() * U32 * (p * (3 * far + 8) + 3 * (hot + p))
    _within("dlogits", db[:, :n], want, torch.where(coef != 0, tol + UNIT[dt] * (want.abs() + tol) + TINY_OF[dt], 0.0))
    if pad:
        assert (db[:, n:] == 5.0).all()
    m.moe_lora_token_logp_backward(x, y, lse, dlogp, x, inv_temp=it)
    assert torch.equal(x, db[:, :n])


@pytest.mark.parametrize("rows,n,dt,pad,masked,it", SHAPES)
@pytest.mark.parametrize("with_ref,weighted,adapters", [(True, False, 1), (False, True, 3), (True, True, 1), (True, False, 4)])
def test_policy_loss(rows, n, dt, pad, masked, it, with_ref, weighted, adapters):
    g, buf, x, y = _inputs(rows, n, dt, pad, masked, rows * 5 + n)
    it = torch.tensor(it, dtype=F32).item()
    low, high, beta = 0.2, 0.3, 0.05
    r = ref.tokens(x, y, it)
    step = 0.4 * torch.randn(rows, generator=g, device="cuda")
    for edge in (math.log(1 - low), math.log(1 + high)):  # ratios on a border of the clip would test the comparison alone
        step = torch.where((step - edge).abs() < 2e-3, edge + 4e-3, step)
    old = (r["logp"] - step).float()
    adv = torch.randn(rows, generator=g, device="cuda")
    rlp = (r["logp"] + 0.5 * torch.randn(rows, generator=g, device="cuda")).float() if with_ref else None
    w = torch.rand(rows, generator=g, device="cuda") if weighted else None
    if weighted and rows > 2:
        w[1] = 0.0
    cut = sorted(torch.randint(0, rows + 1, (adapters - 1,), generator=torch.Generator().manual_seed(n)).tolist())
    offs = [0] + cut + [rows] if adapters > 1 else None
    dloss = torch.rand(adapters, generator=g, device="cuda") + 0.5
    loss, stats = torch.full((adapters,), float("nan"), device="cuda"), torch.full((adapters, 4), float("nan"), device="cuda")
    logp = torch.full((rows,), float("nan"), device="cuda")
    sc = _poisoned(m.policy_scratch(rows, adapters))
    db = torch.full((rows, n + pad), 5.0, dtype=dt, device="cuda")
    kw = dict(clip_low=low, clip_high=high, kl_coef=beta, weight=w, adapter_offsets=offs, inv_temp=it)
    m.moe_lora_policy_loss(x, y, adv, old, rlp, loss, stats, sc, logp=logp, dlogits=db[:, :n], dloss=dloss, **kw)
    wl, ws, wd, lt, st, dtol = ref.policy(r, adv, old, rlp, w, offs or [0, rows], dloss, it, low, high, torch.tensor(beta, dtype=F32).item())
    _within("logp", logp, torch.where(r["ok"], r["logp"], 0.0), torch.where(r["ok"], r["tol"]["logp"], 0.0))
    _within("loss", loss, wl, lt)
    _within("stats", stats, ws, st)
    _within("dlogits", db[:, :n], wd, torch.where(wd != 0, dtol + UNIT[dt] * (wd.abs() + dtol) + TINY_OF[dt], dtol))
    if pad:
        assert (db[:, n:] == 5.0).all()
    # without the gradient: the same loss; each adapter alone: the same up to rounding; in place of the logits: the same bits
    l2, s2 = torch.empty_like(loss), torch.empty_like(stats)
    m.moe_lora_policy_loss(x, y, adv, old, rlp, l2, s2, sc, **kw)
    assert torch.equal(loss, l2) and torch.equal(stats, s2)
    for a in range(adapters if offs else 0):
        i = slice(offs[a], offs[a + 1])
        if i.start % 4 or i.start * x.stride(0) * x.element_size() % 16 or i.start == i.stop:
            continue  # 16-byte aligned starts only
        l1, s1 = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
        m.moe_lora_policy_loss(x[i], y[i], adv[i], old[i], None if rlp is None else rlp[i], l1, s1, m.policy_scratch(i.stop - i.start),
                               clip_low=low, clip_high=high, kl_coef=beta, weight=None if w is None else w[i], inv_temp=it)
        _within("loss alone", l1, wl[a:a + 1], lt[a:a + 1])
        _within("stats alone", s1, ws[a:a + 1], st[a:a + 1])
    m.moe_lora_policy_loss(x, y, adv, old, rlp, l2, s2, sc, dlogits=x, dloss=dloss, **kw)
    assert torch.equal(x, db[:, :n]) and torch.equal(loss, l2)


def test_special_logits():
    """Masked vocabulary (-inf and the type's lowest value), rows of nothing else, NaN and infinity."""
    for dt in (F32, BF, HF):
        low = torch.finfo(dt).min
        for n in (300, 5000, 40000):
            x = torch.randn(8, n, device="cuda", generator=_gen(n)).to(dt)
            x[0, 5:] = -INF
            x[1, :] = low
            x[2, 1:] = low
            x[3, :] = -INF
            x[4, n - 1] = INF
            x[5, n // 2] = float("nan")
            x[6, 3] = -INF
            y = torch.tensor([2, 7, 0, 1, 1, 1, 3, -1], dtype=torch.int32, device="cuda")
            x[7] = float("nan")  # a row without a target may hold anything
            lp, lse, ent = (torch.zeros(8, device="cuda") for _ in range(3))
            m.moe_lora_token_logp_forward(x, y, lp, lse, ent)
            z = x[0, :5].double()
            assert abs(float(lp[0]) - float(z[2] - z.logsumexp(0))) < 1e-5
            p = torch.softmax(z, 0)
            assert abs(float(ent[0]) + float((p * p.log()).sum())) < 1e-5
            assert abs(float(lp[1]) + math.log(n)) < 1e-5 * math.log(n) and abs(float(ent[1]) - math.log(n)) < 1e-4
            # one exponential, to 2 units of its last place, and its logarithm: differences of 4 units of at most 1
            assert abs(float(lp[2])) <= 8 * U32 and abs(float(ent[2])) <= 8 * U32
            assert float(lp[3]) == -INF and abs(float(ent[3]) - math.log(n)) < 1e-4  # all the same
            assert torch.isnan(lp[4:6]).all() and torch.isnan(ent[4:6]).all()
            assert float(lp[6]) == -INF and math.isfinite(float(lse[6]))
            assert float(lp[7]) == 0 and float(lse[7]) == 0 and float(ent[7]) == 0
            # the gradient at masked places is 0, and other rows do not see the bad ones
            d = torch.full_like(x, 7.0)
            loss, stats = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
            y2 = torch.where(torch.arange(8, device="cuda") < 3, y, -1)
            m.moe_lora_policy_loss(x, y2, torch.ones(8, device="cuda"), lp.clone(), None, loss, stats, m.policy_scratch(8), dlogits=d)
            assert (d[0, 5:] == 0).all() and (d[2, 1:] == 0).all() and (d[3:] == 0).all() and torch.isfinite(d.float()).all()
            assert math.isfinite(float(loss))


def test_bad_targets_are_flagged_and_masked():
    x = torch.randn(6, 1000, device="cuda", generator=_gen(1))
    y = torch.tensor([5, 1000, -2, -1, 999, 1 << 30], dtype=torch.int32, device="cuda")
    clean = torch.tensor([5, -1, -1, -1, 999, -1], dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, b = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    m.moe_lora_token_logp_forward(x, clean, b, err=err)
    assert int(err) == 0
    m.moe_lora_token_logp_forward(x, y, a, err=err)
    assert torch.equal(a, b) and int(err) == m.MOE_LORA_DEV_BAD_ID
    m.moe_lora_token_logp_forward(x, y, a)  # without a word nothing is noted
    outs = []
    for t in (y, clean):
        err.zero_()
        l, s, d = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"), torch.empty_like(x)
        m.moe_lora_policy_loss(x, t, torch.ones(6, device="cuda"), b, b, l, s, m.policy_scratch(6), kl_coef=0.1, dlogits=d, err=err)
        outs.append((l, s, d, int(err)))
    assert all(torch.equal(p, q) for p, q in zip(outs[0][:3], outs[1][:3])) and [o[3] for o in outs] == [1, 0]


def test_no_rows():
    x, e = torch.empty(0, 100, device="cuda"), torch.empty(0, device="cuda")
    y = torch.empty(0, dtype=torch.int32, device="cuda")
    for w in (None, e):
        loss, stats = torch.full((2,), 3.0, device="cuda"), torch.full((2, 4), 3.0, device="cuda")
        m.moe_lora_policy_loss(x, y, e, e, None, loss, stats, m.policy_scratch(0, 2), adapter_offsets=[0, 0, 0], weight=w, dlogits=torch.empty_like(x))
        assert (loss == 0).all() and (stats == 0).all()
    m.moe_lora_token_logp_forward(x, y, e)


def test_gradients_match_differences():
    """Policy gradient, and the log probabilities' under the preference loss, against central differences."""
    n, T = 40, 12
    g = _gen(8)
    x = torch.randn(T, n, generator=g, device="cuda")
    y = torch.randint(0, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    y[3] = -1
    r = ref.tokens(x, y, 1.0)
    old = (r["logp"] + 0.05 * torch.randn(T, generator=g, device="cuda")).float()
    adv, rlp = torch.randn(T, generator=g, device="cuda"), (r["logp"] - 0.3).float()
    d, loss, stats = torch.empty_like(x), torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
    m.moe_lora_policy_loss(x, y, adv, old, rlp, loss, stats, m.policy_scratch(T), kl_coef=0.1, dlogits=d)

    def f(v):
        return float(ref.policy(ref.tokens(v, y, 1.0), adv, old, rlp, None, [0, T], None, 1.0, 0.2, 0.2, 0.1)[0])
    seq = torch.tensor([0, 2, 5, 9, 12], device="cuda")

    def fp(v):
        q = ref.tokens(v, y, 1.0)
        return float(ref.preference(torch.where(q["ok"], q["logp"], 0.0), y, seq, None, [0, 2], None, 0.3, "sigmoid", 0.1, 0.2, True)[0])
    lp, lse, dlp = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.zeros(T, device="cuda")
    m.moe_lora_token_logp_forward(x, y, lp, lse)
    m.moe_lora_preference_loss(lp, y, seq, None, loss, stats, m.preference_scratch(2), beta=0.3, label_smoothing=0.1, margin=0.2, average=True, dlogp=dlp)
    dp = torch.empty_like(x)
    m.moe_lora_token_logp_backward(x, y, lse, dlp, dp)
    h = 1e-5
    for i, j in [(0, 0), (1, int(y[1])), (4, 7), (8, int(y[8])), (11, 39), (3, 4)]:
        for fn, got in ((f, d), (fp, dp)):
            a, b = x.double().clone(), x.double().clone()
            a[i, j] += h
            b[i, j] -= h
            diff = (fn(a) - fn(b)) / (2 * h)
            # the difference's own error: h^2 times a third derivative of at most a few, and 2^-52 / h
            assert abs(float(got[i, j]) - diff) < 1e-6 + 2e-5 * abs(diff), (i, j)


# ------------------------------------------------------------------ preference loss
PAIRS = [  # lengths of the sequences, adapters' first pairs
    ([1, 1], None), ([0, 0], None), ([5, 0, 3, 7], None), ([40, 33, 1, 0, 300, 257, 64, 65], [0, 1, 4]),
    ([2000, 1700, 900, 1024], [0, 0, 2]), ([3000, 5000], None), ([7] * 2100, [0, 1025, 1025, 1050]),
]


@pytest.mark.parametrize("kind", ["sigmoid", "squared", "hinge"])
@pytest.mark.parametrize("average,with_ref,smooth", [(False, True, 0.1), (True, False, 0.0), (True, True, 0.5)])
@pytest.mark.parametrize("lens,offs", PAIRS)
def test_preference_loss(lens, offs, kind, average, with_ref, smooth):
    g = _gen(len(lens) + sum(lens))
    P, A = len(lens) // 2, 1 if offs is None else len(offs) - 1
    seq = torch.tensor([0] + lens, device="cuda").cumsum(0) + 3  # tokens ahead of the first sequence, and behind the last
    T = int(seq[-1]) + 5
    y = torch.where(torch.rand(T, generator=g, device="cuda") < 0.3, -1, 7).to(torch.int32)
    lp = -torch.rand(T, generator=g, device="cuda") * 4
    lp[y < 0] = float("nan")  # not read as values
    rf = None
    clean = torch.where(y < 0, 0.0, lp)
    if with_ref:
        tot = ref.preference(clean, y, seq, None, offs or [0, P], None, 0.2, kind, smooth, 0.1, average)[2]
        rf = (tot + torch.randn(2 * P, generator=torch.Generator().manual_seed(1)).double()).float().cuda()
    dloss = torch.rand(A, generator=g, device="cuda") + 0.5
    loss, stats = torch.full((A,), float("nan"), device="cuda"), torch.full((A, 4), float("nan"), device="cuda")
    sl, dl = torch.full((2 * P,), float("nan"), device="cuda"), torch.full((T,), 5.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(beta=0.2, kind=kind, label_smoothing=smooth, margin=0.1, average=average, pair_offsets=offs, err=err)
    m.moe_lora_preference_loss(lp, y, seq, rf, loss, stats, _poisoned(m.preference_scratch(P, A)), seq_logp=sl, dlogp=dl, dloss=dloss, **kw)
    b32 = torch.tensor(0.2, dtype=F32).item()
    s32, m32 = torch.tensor(smooth, dtype=F32).item(), torch.tensor(0.1, dtype=F32).item()
    wl, ws, wt, wd = ref.preference(clean, y, seq, None if rf is None else rf.cpu(), offs or [0, P], dloss, b32, kind, s32, m32, average)
    assert int(err) == 0
    # A thread's own fp32 sum has at most len / 128 + 1 additions, the rest is in 64 bits
    size = max([float(clean[a:b].abs().sum()) for a, b in zip(seq[:-1].tolist(), seq[1:].tolist())] + [1.0])
    serr = (max(lens) / 128 + 2) * U32 * size
    if average:
        serr = (max(lens) / 128 + 2) * U32 * 4
    _within("seq_logp", sl, wt, serr + U32 * wt.abs())
    hmax = float(wt.abs().max()) * 2 + (0 if rf is None else float(rf.abs().max()) * 2) + 10
    slope = max(b32, 2 * (hmax + 2.5)) if kind == "squared" else b32  # of the loss in h
    lerr = slope * 2 * serr + 16 * U32 * (1 + (hmax + 2.5) ** 2 if kind == "squared" else 1 + b32 * hmax)
    _within("loss", loss, wl, lerr + CHAIN * U32 * wl.abs() + 1e-30)
    right = (stats[:, 0].double().cpu() - ws[:, 0]).abs()
    assert (right <= 4 * U32).all()  # no distance lies within rounding of 0 here
    _within("rewards", stats[:, 1:], ws[:, 1:], 2 * serr + CHAIN * U32 * (hmax + 1))
    inside = ~torch.isnan(wd)
    assert (dl.cpu()[~inside] == 5.0).all()
    derr = (2 * 2 * serr if kind == "squared" else b32 * b32 * 2 * serr) * float(dloss.max())
    _within("dlogp", dl.cpu()[inside], wd[inside], derr + 32 * U32 * (wd[inside].abs() + (b32 if kind != "squared" else 2 * (hmax + 2.5))))
    l2 = torch.empty_like(loss)
    m.moe_lora_preference_loss(lp, y, seq, rf, l2, stats, m.preference_scratch(P, A), **kw)
    assert torch.equal(loss, l2)
    for a in range(A if offs else 0):  # each adapter's pairs alone
        i0, i1 = offs[a], offs[a + 1]
        if i0 == i1:
            assert float(loss[a]) == 0
            continue
        l1, s1 = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda")
        m.moe_lora_preference_loss(lp, y, seq[2 * i0:2 * i1 + 1].clone(), None if rf is None else rf[2 * i0:2 * i1].clone(), l1, s1,
                                   m.preference_scratch(i1 - i0), **dict(kw, pair_offsets=None))
        if (T // (2 * P) >= 1024) == (T // (2 * (i1 - i0)) >= 1024):  # the same block size: the same bits
            assert torch.equal(l1, loss[a:a + 1]) and torch.equal(s1[0], stats[a])


def test_preference_bad_offsets():
    """Offsets that go back or past the end are flagged, and nothing outside is touched."""
    lp, y = -torch.ones(20, device="cuda"), torch.ones(20, dtype=torch.int32, device="cuda")
    for seq in ([0, 10, 5, 20, 30], [-4, 10, 12, 15, 20], [0, 1 << 60, 3, 4, 5], [0, 5, 9, -(1 << 60), 20]):
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        d = torch.full((20,), 5.0, device="cuda")
        loss, stats, sl = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"), torch.empty(4, device="cuda")
        m.moe_lora_preference_loss(lp, y, torch.tensor(seq, device="cuda"), None, loss, stats, m.preference_scratch(2), seq_logp=sl, dlogp=d, err=err)
        assert int(err) == m.MOE_LORA_DEV_BAD_ID and torch.isfinite(sl).all() and math.isfinite(float(loss))


def test_no_pairs():
    e, y = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    loss, stats = torch.full((1,), 3.0, device="cuda"), torch.full((1, 4), 3.0, device="cuda")
    m.moe_lora_preference_loss(e, y, torch.zeros(1, dtype=torch.int64, device="cuda"), None, loss, stats, m.preference_scratch(0))
    assert float(loss) == 0 and (stats == 0).all()


def test_streams_and_graphs():
    """On a side stream, and captured and replayed on new inputs, each against an eager call."""
    T, n = 300, 20000
    _, _, x, y = _inputs(T, n, BF, 0, 0.2, 4)
    adv = torch.randn(T, device="cuda", generator=_gen(2))
    lp = torch.empty(T, device="cuda")
    m.moe_lora_token_logp_forward(x, y, lp)
    bufs = lambda: (torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"), torch.empty_like(x), torch.empty(T, device="cuda"))  # noqa: E731

    def call(b, sc):
        m.moe_lora_policy_loss(x, y, adv, lp, lp, b[0], b[1], sc, kl_coef=0.1, dlogits=b[2], logp=b[3])
        m.moe_lora_preference_loss(b[3], y, seq, None, l2, s2, psc, dlogp=dlp)
    seq = torch.arange(0, T + 1, T // 6, device="cuda")
    l2, s2, dlp, psc = torch.empty(1, device="cuda"), torch.empty(1, 4, device="cuda"), torch.zeros(T, device="cuda"), m.preference_scratch(3)
    want, sc = bufs(), m.policy_scratch(T)
    call(want, sc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, sc2 = bufs(), m.policy_scratch(T)
    with torch.cuda.stream(side):
        call(got, sc2)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph, got = torch.cuda.CUDAGraph(), bufs()
    with torch.cuda.graph(graph):
        call(got, sc2)
    for seed in (5, 6):
        x.copy_(torch.randn(T, n, device="cuda", generator=_gen(seed)))
        graph.replay()
        call(want, sc)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
