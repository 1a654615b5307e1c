"""Cases of the post-training operators: token log probabilities (forward and backward), the
clipped policy loss with a KL term and its gradient, the preference loss over pairs of packed
sequences, and the Muon step over the layer's factors.  `run` computes a case in plain fp32
torch operations, or with `own` set through the package's entry points; `exact` computes the
definition in 64 bits."""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.04
BETA, MARGIN, SMOOTH = 0.1, 0.0, 0.05
MOMENTUM, NS_STEPS, NS_EPS = 0.95, 5, 1e-7
NS_A, NS_B, NS_C = 3.4445, -4.7750, 2.0315


# ------------------------------------------------------------------ cases
def _logp(op, tokens, vocab, dtype, masked, temp=1.0, pad=0, entropy=False):
    # `masked`: share of tokens without a target (prompts, padding); `pad`: columns of the buffer past the vocabulary
    c = {"op": op, "tokens": tokens, "vocab": vocab, "dtype": dtype, "masked": masked, "temp": temp, "pad": pad}
    if op == "logp_fwd":
        c["entropy"] = entropy
    return c


def _policy(tokens, vocab, dtype, masked, adapters=1, ref=True, weighted=False, grad=True, temp=1.0, pad=0):
    return {"op": "policy", "tokens": tokens, "vocab": vocab, "dtype": dtype, "masked": masked, "adapters": adapters,
            "ref": ref, "weighted": weighted, "grad": grad, "temp": temp, "pad": pad}


def _pref(pairs, mean_len, kind, average, masked, adapters=1, ref=True):
    return {"op": "pref", "pairs": pairs, "mean_len": mean_len, "kind": kind, "average": average, "masked": masked,
            "adapters": adapters, "ref": ref}


def _muon(hidden, inter, experts, rank, adapters, param, grad, nesterov=True, decay=0.01):
    return {"op": "muon", "hidden": hidden, "inter": inter, "experts": experts, "rank": rank, "adapters": adapters,
            "param": param, "grad": grad, "nesterov": nesterov, "decay": decay}


def listed():
    return [
        # a sampler's log probabilities of one decoding step of a small batch: all latency
        dict(_logp("logp_fwd", 4, 32000, "bf16", 0.0, temp=0.7), name="logp_fwd_decode"),
        # a reference model's pass over a training batch, with entropies for the log
        dict(_logp("logp_fwd", 16384, 65536, "bf16", 0.1, entropy=True), name="logp_fwd_batch"),
        # an odd vocabulary, rows off the 16-byte grid, half of the tokens are prompts
        dict(_logp("logp_bwd", 1031, 50257, "f16", 0.5), name="logp_bwd_odd"),
        # the preference loss's way back to the logits of a training batch
        dict(_logp("logp_bwd", 16384, 65536, "bf16", 0.1), name="logp_bwd_batch"),
        # a test-size model in fp32
        dict(_policy(64, 4096, "f32", 0.2), name="policy_tiny_f32"),
        # 16 adapters, each with its own loss, share a batch; odd vocabulary inside a padded buffer
        dict(_policy(2048, 50257, "bf16", 0.4, adapters=16, pad=47), name="policy_16_adapters"),
        # a large vocabulary, per-sequence weights, sampled at a temperature
        dict(_policy(8192, 151936, "bf16", 0.3, weighted=True, temp=0.8), name="policy_large"),
        # a handful of short pairs
        dict(_pref(4, 50, "sigmoid", False, 0.3), name="pref_tiny"),
        # many long pairs of four adapters, length-normalised without a reference model
        dict(_pref(1024, 700, "sigmoid", True, 0.3, adapters=4, ref=False), name="pref_batch"),
        # the smallest training configuration's factors
        dict(_muon(512, 256, 16, 16, 1, "master_bf16", "f32"), name="muon_tiny"),
        # 16 adapters' factors, bf16 without master copies, bf16 gradients
        dict(_muon(2048, 768, 128, 8, 16, "bf16", "bf16"), name="muon_16_adapters"),
        # all factors of the production layer
        dict(_muon(4096, 2048, 256, 128, 1, "master_bf16", "f32"), name="muon_production"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _vocab(rng, lo=100, hi=200000):
    v = _log(rng, lo, hi)
    return max(64, v // 64 * 64) if rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["logp_fwd", "logp_bwd", "policy", "policy", "pref", "muon"])
    if op in ("logp_fwd", "logp_bwd", "policy"):
        vocab = _vocab(rng)
        tokens = _log(rng, 1, min(32768, (1 << 29) // vocab))
        dtype, masked, temp = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([0.0, 0.1, 0.5, 0.9]), rng.choice([1.0, 1.0, 0.6])
        pad = rng.choice([0, 0, 8, 5])
        if op != "policy":
            return _logp(op, tokens, vocab, dtype, masked, temp, pad, rng.random() < 0.5)
        return _policy(tokens, vocab, dtype, masked, rng.choice([1, 1, 3, 16]), rng.random() < 0.7, rng.random() < 0.5,
                       rng.random() < 0.8, temp, pad)
    if op == "pref":
        pairs = _log(rng, 1, 2000)
        return _pref(pairs, _log(rng, 5, min(4000, 1000000 // pairs)), rng.choice(["sigmoid", "squared", "hinge"]),
                     rng.random() < 0.5, rng.choice([0.0, 0.3, 0.7]), rng.choice([1, 1, 2, 8]), rng.random() < 0.7)
    hidden, inter = rng.choice([512, 1024, 2048, 4096, 1000]), rng.choice([256, 768, 1408, 2048, 300])
    rank, adapters = rng.choice([8, 16, 32, 64, 128, 24]), rng.choice([1, 1, 4])
    most = (1 << 26) // (3 * inter * rank * adapters)
    return _muon(hidden, inter, _log(rng, 1, max(1, min(256, most))), rank, adapters,
                 rng.choice(["f32", "master_bf16", "master_f16", "bf16"]), rng.choice(["f32", "bf16", "f16"]),
                 rng.random() < 0.7, rng.choice([0.0, 0.01, 0.1]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _chunks(rows, per_row):
    step = max(1, (1 << 26) // per_row)
    return [(i, min(rows, i + step)) for i in range(0, rows, step)]


def _prepare_logits(c, g):
    """Logits of a model at work: most targets well ahead of the rest, the others anywhere."""
    T, V, dt = c["tokens"], c["vocab"], DT[c["dtype"]]
    buf = torch.zeros(T, V + c["pad"], dtype=dt, device="cuda")
    logits = buf[:, :V]
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    ahead = torch.where(_rand(g, T) < 0.8, math.log(V) + 3 + 2 * _randn(g, T), 0.0)
    targets_masked = torch.where(_rand(g, T) < c["masked"], -1, targets).to(torch.int32)
    logp = torch.empty(T, device="cuda")
    lse = torch.empty(T, device="cuda")
    for lo, hi in _chunks(T, V):
        x = 2 * _randn(g, hi - lo, V)
        x[torch.arange(hi - lo, device="cuda"), targets[lo:hi]] += ahead[lo:hi]
        logits[lo:hi] = x.to(dt)
        z = logits[lo:hi].float() / c["temp"]
        lse[lo:hi] = torch.logsumexp(z, 1)
        logp[lo:hi] = z[torch.arange(hi - lo, device="cuda"), targets[lo:hi]] - lse[lo:hi]
    return {"logits": logits, "targets": targets_masked, "scale": 1.0 / c["temp"]}, logp, lse


def _like(t):
    b = torch.zeros(t.shape[0], t.stride(0) if t.shape[0] > 1 else t.shape[1], dtype=t.dtype, device=t.device)
    return b[:, :t.shape[1]]


def _prepare_logp(c, g):
    s, _, lse = _prepare_logits(c, g)
    T = c["tokens"]
    s["logp"], s["entropy"] = torch.empty(T, device="cuda"), torch.empty(T, device="cuda") if c.get("entropy") else None
    if c["op"] == "logp_fwd":
        s["lse"] = torch.empty(T, device="cuda")
    else:  # what a loss over sequences sends back
        s.update(lse=torch.where(s["targets"] >= 0, lse, 0.0), dlogp=_randn(g, T) / T, dlogits=_like(s["logits"]))
    return s


def _offsets(n, parts):
    """Uneven ranges of n, the last one empty where there are several."""
    return [n * a * (a + 1) // (parts * (parts - 1)) if parts > 1 else n * a for a in range(parts)] + [n]


def _prepare_policy(c, g):
    s, logp, _ = _prepare_logits(c, g)
    T, A = c["tokens"], c["adapters"]
    # the policy has moved a little since the samples were drawn; no ratio lies on a border of the clip
    step = 0.15 * _randn(g, T)
    for edge in (math.log(1 - CLIP_LOW), math.log(1 + CLIP_HIGH)):
        step = torch.where((step - edge).abs() < 2e-3, edge + 4e-3, step)
    s["old"] = logp - step
    s["ref"] = logp + 0.3 * _randn(g, T) if c["ref"] else None
    s["adv"] = _randn(g, T)
    s["weight"] = _rand(g, T) / T if c["weighted"] else None
    s["offsets"] = _offsets(T, A)
    s["first"] = torch.tensor(s["offsets"][1:], device="cuda")
    s["dloss"] = 0.5 + _rand(g, A)
    s.update(loss=torch.empty(A, device="cuda"), stats=torch.empty(A, 4, device="cuda"), logp=torch.empty(T, device="cuda"),
             dlogits=_like(s["logits"]) if c["grad"] else None)
    return s


def _prepare_pref(c, g):
    P, A = c["pairs"], c["adapters"]
    # a packed batch of answers of log-normal lengths, short ones among them
    share = torch.exp(0.6 * _randn(g, 2 * P)).double().cumsum(0)
    seq = torch.zeros(2 * P + 1, dtype=torch.int64, device="cuda")
    seq[1:] = (share / share[-1] * (2 * P * c["mean_len"])).round().long()
    T = 2 * P * c["mean_len"] + 7  # and the batch's padding behind the last sequence
    targets = torch.where(_rand(g, T) < c["masked"], -1, 1).to(torch.int32)
    live = targets >= 0
    logp = torch.where(live, -torch.exp(_randn(g, T) - 0.5), 0.0)
    sums = torch.zeros(T + 1, dtype=torch.float64, device="cuda")
    sums[1:] = logp.double().cumsum(0)
    total = sums[seq[1:]] - sums[seq[:-1]]
    s = {"logp": logp, "targets": targets, "seq": seq, "pairs": _offsets(P, A),
         "ref": (total + 3 * _randn(g, 2 * P)).float() if c["ref"] else None, "dloss": 0.5 + _rand(g, A)}
    if c["ref"] and c["average"]:
        cnt = torch.zeros(T + 1, dtype=torch.int64, device="cuda")
        cnt[1:] = live.long().cumsum(0)
        s["ref"] = s["ref"] / (cnt[seq[1:]] - cnt[seq[:-1]]).clamp(min=1)
    s.update(loss=torch.empty(A, device="cuda"), stats=torch.empty(A, 4, device="cuda"), seq_logp=torch.empty(2 * P, device="cuda"),
             dlogp=torch.zeros(T, device="cuda"))
    return s


def _factors(c):
    """Shapes of the trained factors: leading axes are matrices of their own."""
    H, I, E, r, A = c["hidden"], c["inter"], c["experts"], c["rank"], c["adapters"]
    return [(A, r, H), (A, r, H), (A, E, I, r), (A, E, I, r), (A, E, r, I), (A, H, r)]


def _prepare_muon(c, g):
    s = {"lr": 1e-3, "decay": c["decay"], "nesterov": c["nesterov"], "scale": torch.full((1,), 0.7, device="cuda"),
         "grad": [], "m": [], "param": [], "master": [] if c["param"].startswith("master") else None}
    low = {"f32": torch.float32, "bf16": torch.bfloat16, "master_bf16": torch.bfloat16, "master_f16": torch.float16}[c["param"]]
    for shape in _factors(c):
        rows, cols = shape[-2:]
        lead = shape[:-2]
        size = torch.exp(2 * _rand(g, *lead, 1, 1) - 9)  # matrices of very different size
        strong = torch.matmul(_randn(g, *lead, rows, 2), _randn(g, *lead, 2, cols))  # a gradient's few strong directions
        s["grad"].append((size * (_randn(g, *shape) + strong)).to(DT[c["grad"]]))
        s["m"].append(size * (0.3 * _randn(g, *shape) + 0.5 * strong))
        w = 0.02 * _randn(g, *shape)
        s["param"].append(w.to(low))
        if s["master"] is not None:
            s["master"].append(w)
    return s


_PREPARE = {"logp_fwd": _prepare_logp, "logp_bwd": _prepare_logp, "policy": _prepare_policy, "pref": _prepare_pref,
            "muon": _prepare_muon}


def prepare(case, seed):
    s = _PREPARE[case["op"]](case, _gen(seed))
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _plain_stats(s):
    z = s["logits"].float() * s["scale"]
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total))[:, 0]
    live = s["targets"] >= 0
    at = s["targets"].clamp(min=0).long()[:, None]
    # target minus maximum first: both are of the logits' size, and their difference is what counts
    logp = (z.gather(1, at) - top - torch.log(total))[:, 0]
    return z, e / total, lse, torch.where(live, logp, 0.0), live, at


def _plain_logp_fwd(s):
    z, p, lse, logp, live, _ = _plain_stats(s)
    out = {"logp": logp, "lse": torch.where(live, lse, 0.0)}
    if s["entropy"] is not None:
        out["entropy"] = torch.where(live, -(p * (z - lse[:, None])).sum(1), 0.0)
    return out


def _plain_grad(s, p, coef, at):
    """coef * (onehot - p) by rows."""
    d = -p * coef[:, None]
    d.scatter_add_(1, at, coef[:, None])
    return d.to(s["logits"].dtype)


def _plain_logp_bwd(s):
    live = s["targets"] >= 0
    p = torch.exp(s["logits"].float() * s["scale"] - s["lse"][:, None])
    at = s["targets"].clamp(min=0).long()[:, None]
    return {"dlogits": _plain_grad(s, p, torch.where(live, s["dlogp"] * s["scale"], 0.0), at)}


def _plain_policy(s):
    z, p, lse, logp, live, at = _plain_stats(s)
    A = len(s["offsets"]) - 1
    of = torch.bucketize(torch.arange(z.shape[0], device="cuda"), s["first"], right=True)
    member = ((of[None, :] == torch.arange(A, device="cuda")[:, None]) & live[None, :]).double()
    if s["weight"] is None:
        w = torch.where(live, 1 / member.sum(1).clamp(min=1).float()[of], 0.0)
    else:
        w = torch.where(live, s["weight"], 0.0)
    rho = torch.exp(logp - s["old"])
    adv = s["adv"]
    clipped = ((adv > 0) & (rho > 1 + CLIP_HIGH)) | ((adv < 0) & (rho < 1 - CLIP_LOW))
    loss = -torch.minimum(rho * adv, rho.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * adv)
    g = torch.where(clipped, 0.0, -rho * adv)
    kl = torch.zeros_like(rho)
    if s["ref"] is not None:
        d = s["ref"] - logp
        kl = torch.expm1(d) - d
        loss = loss + KL * kl
        g = g - KL * torch.expm1(d)
    entropy = -(p * (z - lse[:, None])).sum(1)
    terms = torch.stack([loss, kl, clipped.float(), rho, entropy], 1)
    sums = member @ (w[:, None] * torch.where(live[:, None], terms, 0.0)).double()
    out = {"loss": sums[:, 0].float(), "stats": sums[:, 1:].float(), "logp": logp}
    if s["dlogits"] is not None:
        out["dlogits"] = _plain_grad(s, p, torch.where(live, w * g * s["dloss"][of] * s["scale"], 0.0), at)
    return out


def _sums(v, offsets):
    """Sums of a vector between offsets."""
    run = torch.zeros(len(v) + 1, dtype=v.dtype, device="cuda")
    torch.cumsum(v, 0, out=run[1:])
    return run[offsets[1:]] - run[offsets[:-1]]


def _plain_pref(s):
    c, P = s["case"], (len(s["seq"]) - 1) // 2
    A = c["adapters"]
    live = s["targets"] >= 0
    seq_logp = _sums(s["logp"].double(), s["seq"])
    n = _sums(live.double(), s["seq"]).clamp(min=1) if c["average"] else torch.ones(2 * P, device="cuda", dtype=torch.float64)
    seq_logp = seq_logp / n
    r = seq_logp - s["ref"].double() if s["ref"] is not None else seq_logp
    h = r[0::2] - r[1::2]
    delta = BETA * h - MARGIN
    if c["kind"] == "sigmoid":
        soft = torch.log1p(torch.exp(-delta.abs()))
        loss = (1 - SMOOTH) * (soft + (-delta).clamp(min=0)) + SMOOTH * (soft + delta.clamp(min=0))
        dh = BETA * (1 / (1 + torch.exp(-delta)) - (1 - SMOOTH))
    elif c["kind"] == "squared":
        off = h - 1 / (2 * BETA)
        loss, dh = off * off, 2 * off
    else:
        loss, dh = (1 - delta).clamp(min=0), torch.where(delta < 1, -BETA, 0.0)
    of = torch.bucketize(torch.arange(P, device="cuda"), torch.tensor(s["pairs"][1:], device="cuda"), right=True)
    member = (of[None, :] == torch.arange(A, device="cuda")[:, None]).double()
    count = member.sum(1).clamp(min=1)
    terms = torch.stack([loss, (delta > 0).double(), BETA * r[0::2], BETA * r[1::2], h], 1)
    mean = (member @ terms / count[:, None]).float()
    per = (dh * s["dloss"].double()[of] / count[of])[:, None] / torch.stack([n[0::2], -n[1::2]], 1)
    dlogp = torch.zeros_like(s["logp"])
    packed = 2 * P * c["mean_len"]
    dlogp[:packed] = torch.repeat_interleave(per.reshape(-1).float(), s["seq"][1:] - s["seq"][:-1], output_size=packed)
    return {"loss": mean[:, 0], "stats": mean[:, 1:], "seq_logp": seq_logp.float(), "dlogp": torch.where(live, dlogp, 0.0)}


def _plain_muon(s):
    for i, grad in enumerate(s["grad"]):
        g = grad.float() * s["scale"]
        m = MOMENTUM * s["m"][i] + (1 - MOMENTUM) * g
        u = (1 - MOMENTUM) * g + MOMENTUM * m if s["nesterov"] else m
        tall = u.shape[-2] > u.shape[-1]
        x = u.transpose(-1, -2) if tall else u
        x = x / (torch.sqrt((x * x).sum((-1, -2), keepdim=True)) + NS_EPS)
        for _ in range(NS_STEPS):
            a = torch.matmul(x, x.transpose(-1, -2))
            x = NS_A * x + torch.matmul(NS_B * a + NS_C * torch.matmul(a, a), x)
        if tall:
            x = x.transpose(-1, -2)
        w = s["master"][i] if s["master"] is not None else s["param"][i].float()
        w = w * (1 - s["lr"] * s["decay"]) - s["lr"] * math.sqrt(max(1.0, u.shape[-2] / u.shape[-1])) * x
        s["param"][i], s["m"][i] = w.to(s["param"][i].dtype), m
        if s["master"] is not None:
            s["master"][i] = w
    return _muon_outputs(s)


def _muon_outputs(s):
    return {k: list(s[k]) for k in ("param", "master", "m") if s[k] is not None}


# ------------------------------------------------------------------ the framework's operators
def _own_logp_fwd(s, m):
    m.moe_lora_token_logp_forward(s["logits"], s["targets"], s["logp"], s["lse"], s["entropy"], inv_temp=s["scale"])
    return {k: s[k] for k in ("logp", "lse", "entropy") if s[k] is not None}


def _own_logp_bwd(s, m):
    m.moe_lora_token_logp_backward(s["logits"], s["targets"], s["lse"], s["dlogp"], s["dlogits"], inv_temp=s["scale"])
    return {"dlogits": s["dlogits"]}


def _own_policy(s, m):
    if "scratch" not in s:  # a program keeps one workspace for its sizes
        s["scratch"] = m.policy_scratch(s["logits"].shape[0], len(s["offsets"]) - 1)
    m.moe_lora_policy_loss(s["logits"], s["targets"], s["adv"], s["old"], s["ref"], s["loss"], s["stats"], s["scratch"],
                           clip_low=CLIP_LOW, clip_high=CLIP_HIGH, kl_coef=KL, weight=s["weight"], adapter_offsets=s["offsets"],
                           logp=s["logp"], dlogits=s["dlogits"], dloss=s["dloss"], inv_temp=s["scale"])
    return {k: s[k] for k in ("loss", "stats", "logp", "dlogits") if s[k] is not None}


def _own_pref(s, m):
    c = s["case"]
    if "scratch" not in s:
        s["scratch"] = m.preference_scratch(c["pairs"], c["adapters"])
    m.moe_lora_preference_loss(s["logp"], s["targets"], s["seq"], s["ref"], s["loss"], s["stats"], s["scratch"], beta=BETA,
                               kind=c["kind"], label_smoothing=SMOOTH, margin=MARGIN, average=c["average"],
                               pair_offsets=s["pairs"], seq_logp=s["seq_logp"], dlogp=s["dlogp"], dloss=s["dloss"])
    return {k: s[k] for k in ("loss", "stats", "seq_logp", "dlogp")}


def _own_muon(s, m):
    if "tensors" not in s:  # a program lists its tensors once
        s["tensors"] = m.MuonTensors([dict(p=p, g=s["grad"][i], m=s["m"][i], lr=s["lr"], weight_decay=s["decay"],
                                           master=s["master"][i] if s["master"] is not None else None)
                                      for i, p in enumerate(s["param"])])
    m.moe_lora_muon_step(s["tensors"], momentum=MOMENTUM, nesterov=s["nesterov"], steps=NS_STEPS, coefs=(NS_A, NS_B, NS_C),
                         eps=NS_EPS, grad_scale=s["scale"])
    return _muon_outputs(s)


_PLAIN = {"logp_fwd": _plain_logp_fwd, "logp_bwd": _plain_logp_bwd, "policy": _plain_policy, "pref": _plain_pref, "muon": _plain_muon}
_OWN = {"logp_fwd": _own_logp_fwd, "logp_bwd": _own_logp_bwd, "policy": _own_policy, "pref": _own_pref, "muon": _own_muon}


def run(state):
    op = state["case"]["op"]
    if own:
        import moe_expert_ffn_top_gb300 as m
        return _OWN[op](state, m)
    return _PLAIN[op](state)


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] in ("logp_fwd", "logp_bwd", "policy"):
        live = max(1.0, c["tokens"] * (1 - c["masked"]))  # rows without a target are not read, their gradient is written
        row, T = c["vocab"] * SIZE[c["dtype"]], c["tokens"]
        if c["op"] == "logp_fwd":
            return {"bytes": live * row + T * (16 if c["entropy"] else 12), "flops": 4 * live * c["vocab"]}
        if c["op"] == "logp_bwd":
            return {"bytes": live * row + T * row + 12 * T, "flops": 4 * live * c["vocab"]}
        vecs = 4 * T * (4 + (1 if c["ref"] else 0) + (1 if c["weighted"] else 0))
        return {"bytes": live * row + (T * row if c["grad"] else 0) + vecs, "flops": (10 if c["grad"] else 6) * live * c["vocab"]}
    if c["op"] == "pref":
        T = 2 * c["pairs"] * c["mean_len"]
        return {"bytes": 12 * T + 24 * c["pairs"], "flops": 6 * T}
    n = flops = 0
    for shape in _factors(c):
        short, long_ = sorted(shape[-2:])
        batch = math.prod(shape[:-2])
        n += batch * short * long_
        # the Gram matrix, the product with the polynomial, and the polynomial itself: three products a step
        flops += batch * (4 * short * short * long_ + 6 * NS_STEPS * short ** 3)
    low = 4 if c["param"] == "f32" else 2
    weights = 8 + low if c["param"].startswith("master") else 2 * low
    return {"bytes": n * (SIZE[c["grad"]] + 8 + weights), "flops": flops}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rows(s, fn):
    """fn(z, targets, rows) over slices of the live rows, z the scaled logits in 64 bits."""
    rows = torch.nonzero(s["targets"] >= 0)[:, 0]
    for lo, hi in _chunks(len(rows), 4 * s["logits"].shape[1]):
        r = rows[lo:hi]
        fn(s["logits"][r].double() * s["scale"], s["targets"][r].long(), r)


def _exact_token(s):
    T = s["logits"].shape[0]
    logp, lse, ent = (torch.zeros(T, dtype=torch.float64, device="cuda") for _ in range(3))

    def rows(z, y, r):
        l = torch.logsumexp(z, 1)
        lse[r] = l
        logp[r] = z.gather(1, y[:, None])[:, 0] - l
        ent[r] = l - (torch.exp(z - l[:, None]) * z).sum(1)
    _exact_rows(s, rows)
    return logp, lse, ent


def _exact_dlogits(s, lse, coef):
    d = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")

    def rows(z, y, r):
        hot = torch.zeros_like(z)
        hot[torch.arange(len(y), device="cuda"), y] = 1
        d[r] = coef[r][:, None] * (hot - torch.exp(z - lse[r][:, None]))
    _exact_rows(s, rows)
    return d


def _exact_logp(c, s):
    if c["op"] == "logp_bwd":  # the saved lse is an input
        return {"dlogits": _exact_dlogits(s, s["lse"].double(), s["dlogp"].double() * s["scale"])}
    logp, lse, ent = _exact_token(s)
    return {"logp": logp, "lse": lse, "entropy": ent} if c["entropy"] else {"logp": logp, "lse": lse}


def _exact_policy(c, s):
    logp, lse, ent = _exact_token(s)
    T, A = c["tokens"], c["adapters"]
    loss, stats, coef = [], [], torch.zeros(T, dtype=torch.float64, device="cuda")
    for a in range(A):
        i = slice(s["offsets"][a], s["offsets"][a + 1])
        on = (s["targets"][i] >= 0).double()
        w = on * s["weight"][i].double() if c["weighted"] else on / max(1.0, float(on.sum()))
        rho, adv = torch.exp(logp[i] - s["old"][i].double()), s["adv"][i].double()
        low, high = 1 - CLIP_LOW, 1 + CLIP_HIGH
        cut = ((adv > 0) & (rho > high)) | ((adv < 0) & (rho < low))
        obj = torch.where(adv > 0, rho.clamp(max=high), rho.clamp(min=low)) * adv
        kl, g = torch.zeros_like(rho), torch.where(cut, 0.0, -adv * rho)
        if c["ref"]:
            d = s["ref"][i].double() - logp[i]
            kl = torch.exp(d) - 1 - d
            g = g + KL * (1 - torch.exp(d))
        loss.append((w * (KL * kl - obj)).sum())
        stats.append(torch.stack([(w * v).sum() for v in (kl, cut.double(), rho, ent[i])]))
        coef[i] = float(s["dloss"][a]) * w * g * s["scale"]
    out = {"loss": torch.stack(loss), "stats": torch.stack(stats), "logp": logp}
    if c["grad"]:
        out["dlogits"] = _exact_dlogits(s, lse, coef)
    return out


def _exact_pref(c, s):
    P, A, seq = c["pairs"], c["adapters"], s["seq"].tolist()
    logp, live = s["logp"].double().cpu(), (s["targets"] >= 0).cpu()
    ref = s["ref"].double().cpu() if c["ref"] else torch.zeros(2 * P, dtype=torch.float64)
    dloss = s["dloss"].double().cpu()
    norm = [max(1, int(live[a:b].sum())) if c["average"] else 1 for a, b in zip(seq, seq[1:])]
    total = [float(logp[a:b].sum()) / n for a, b, n in zip(seq, seq[1:], norm)]
    dlogp = torch.zeros_like(logp)
    loss, stats = torch.zeros(A).double(), torch.zeros(A, 4).double()
    for a in range(A):
        n = s["pairs"][a + 1] - s["pairs"][a]
        for i in range(s["pairs"][a], s["pairs"][a + 1]):
            rc, rr = total[2 * i] - float(ref[2 * i]), total[2 * i + 1] - float(ref[2 * i + 1])
            h = rc - rr
            x = BETA * h - MARGIN
            if c["kind"] == "sigmoid":
                lp, ln = (math.log1p(math.exp(-x)) if x > 0 else -x + math.log1p(math.exp(x))), \
                         (math.log1p(math.exp(x)) if x < 0 else x + math.log1p(math.exp(-x)))
                l = (1 - SMOOTH) * lp + SMOOTH * ln
                d = BETA * (-(1 - SMOOTH) * math.exp(-ln) + SMOOTH * math.exp(-lp))
            elif c["kind"] == "squared":
                l, d = (h - 0.5 / BETA) ** 2, 2 * (h - 0.5 / BETA)
            else:
                l, d = max(0.0, 1 - x), -BETA if x < 1 else 0.0
            loss[a] += l / n
            stats[a] += torch.tensor([float(x > 0), BETA * rc, BETA * rr, h]).double() / n
            d *= float(dloss[a]) / n
            for j, sign in ((2 * i, 1), (2 * i + 1, -1)):
                span = slice(seq[j], seq[j + 1])
                dlogp[span] = torch.where(live[span], sign * d / norm[j], 0.0)
    return {"loss": loss, "stats": stats, "seq_logp": torch.tensor(total).double(), "dlogp": dlogp}


def _exact_muon(c, s):
    f64 = torch.float64
    out = {"param": [], "master": [], "m": []}
    for i, grad in enumerate(s["grad"]):
        rows, cols = grad.shape[-2:]
        g = grad.to(f64) * s["scale"].to(f64)
        m = s["m"][i].to(f64)
        m += (1 - MOMENTUM) * (g - m)
        u = torch.lerp(g, m, MOMENTUM) if s["nesterov"] else m
        o = torch.empty(u.shape, dtype=f64, device="cuda")
        flat, res = u.reshape(-1, rows, cols), o.view(-1, rows, cols)
        for b, e in _chunks(len(flat), rows * cols):
            x = flat[b:e]
            x = x / (torch.linalg.vector_norm(x, dim=(1, 2))[:, None, None] + NS_EPS)
            for _ in range(NS_STEPS):
                k = x @ x.mT if rows <= cols else x.mT @ x
                q = NS_B * k + NS_C * (k @ k)
                x = NS_A * x + (q @ x if rows <= cols else x @ q)
            res[b:e] = x
        w = (s["master"][i] if s["master"] is not None else s["param"][i]).to(f64)
        w = w - s["lr"] * (s["decay"] * w + max(1.0, rows / cols) ** 0.5 * o)
        for k, v in (("param", w), ("master", w), ("m", m)):
            out[k].append(v)
    if s["master"] is None:
        out.pop("master")
    return out


def exact(case, seed):
    s = prepare(case, seed)
    fn = {"logp_fwd": _exact_logp, "logp_bwd": _exact_logp, "policy": _exact_policy, "pref": _exact_pref, "muon": _exact_muon}
    return fn[case["op"]](case, s)
