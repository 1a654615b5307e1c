"""Cases of the training-step operators around the expert layer: layer norm (forward and
backward), the router's balance loss with its gradient, and the AdamW step over many
tensors.  `run` computes a case in plain fp32 torch operations, or with `own` set through
the package's entry points; `exact` computes the definition in 64 bits."""
import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5                      # layer norm
BETA1, BETA2, ADAM_EPS = 0.9, 0.999, 1e-8
STEP = 100                      # optimizer step number: bias corrections matter at this point
BLOCK = 256                     # elements that share one scale of an 8-bit state
E4M3_MAX = 448.0
TINY = 2.0 ** -100              # blocks whose largest value is below are stored as zeros


# ------------------------------------------------------------------ cases
def _norm(op, rows, n, dtype, weight, bias=True, pad=0, dres=False, wgrad=True):
    c = {"op": op, "rows": rows, "n": n, "dtype": dtype, "weight": weight, "bias": bias, "pad": pad}
    if op == "norm_bwd":
        c.update(dres=dres, wgrad=wgrad)
    return c


def _balance(tokens, experts, topk, adapters, dtype, grad, masked):
    return {"op": "balance", "tokens": tokens, "experts": experts, "topk": topk, "adapters": adapters,
            "dtype": dtype, "grad": grad, "masked": masked}


def _adamw(hidden, inter, experts, rank, adapters, param, grad, bits, decay=0.01, odd=0):
    # `odd` elements more in every tensor: lengths that end inside a scale block
    return {"op": "adamw", "hidden": hidden, "inter": inter, "experts": experts, "rank": rank, "adapters": adapters,
            "param": param, "grad": grad, "bits": bits, "decay": decay, "odd": odd}


def listed():
    return [
        # one token in front of the router: a decoding step, all latency
        dict(_norm("norm_fwd", 1, 4096, "bf16", "bf16"), name="norm_fwd_one_token"),
        # a ragged token count at a width that no vector load divides, rows inside a wider buffer
        dict(_norm("norm_fwd", 1029, 2049, "f16", "f32", pad=6), name="norm_fwd_odd_width"),
        # the production batch of the expert layer
        dict(_norm("norm_fwd", 65536, 4096, "bf16", "bf16"), name="norm_fwd_production"),
        # a small fp32 model, odd sizes, no residual: the weight's reduction counts as much as dx
        dict(_norm("norm_bwd", 347, 577, "f32", "f32"), name="norm_bwd_small_f32"),
        # the production batch, the residual stream's gradient added in the same pass
        dict(_norm("norm_bwd", 65536, 4096, "bf16", "f32", dres=True), name="norm_bwd_production"),
        # the smallest training configuration
        dict(_balance(256, 16, 2, 1, "f32", True, 0.0), name="balance_tiny"),
        # counts and loss alone, as logged in evaluation; half-precision logits, odd expert count, masked routes
        dict(_balance(2047, 60, 4, 1, "bf16", False, 0.2), name="balance_eval_masked"),
        # 16 adapters with a router each share one layer
        dict(_balance(16384, 128, 8, 16, "f32", True, 0.0), name="balance_16_adapters"),
        # the production batch
        dict(_balance(65536, 256, 6, 1, "f32", True, 0.0), name="balance_production"),
        # the smallest training configuration's factors, bf16 operands with fp32 master copies
        dict(_adamw(512, 256, 16, 16, 1, "master_bf16", "f32", 32), name="adamw_tiny"),
        # 16 adapters' factors as 96 tensors of odd lengths, bf16 without master, bf16 gradients
        dict(_adamw(2048, 768, 128, 8, 16, "bf16", "bf16", 32, odd=3), name="adamw_16_adapters"),
        # all factors of the production layer, 8-bit states
        dict(_adamw(4096, 2048, 256, 128, 1, "master_bf16", "f32", 8), name="adamw_production_8bit"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance", "adamw"])
    if op in ("norm_fwd", "norm_bwd"):
        n = _log(rng, 64, 16384)
        if rng.random() < 0.5:  # widths of models are multiples of 64; the rest are whatever comes
            n = max(64, n // 64 * 64)
        rows = _log(rng, 1, min(65536, (1 << 27) // n))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        return _norm(op, rows, n, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.8, rng.choice([0, 0, 8, 5]),
                     rng.random() < 0.5, rng.random() < 0.8)
    if op == "balance":
        experts = rng.choice([8, 16, 60, 64, 127, 128, 160, 256, 384, 512])
        tokens = _log(rng, 1, min(65536, (1 << 23) // experts))
        adapters = rng.choice([1, 1, 2, 16])
        if tokens < 128 * adapters:
            adapters = 1
        return _balance(tokens, experts, rng.randint(1, min(8, experts)), adapters,
                        rng.choice(["f32", "f32", "bf16", "f16"]), rng.random() < 0.7, rng.choice([0.0, 0.2, 0.9]))
    hidden, inter = rng.choice([512, 1024, 2048, 4096]), rng.choice([256, 768, 1408, 2048])
    rank, adapters = rng.choice([8, 16, 32, 64]), rng.choice([1, 1, 4, 16])
    most = (1 << 26) // (3 * inter * rank * adapters)
    return _adamw(hidden, inter, _log(rng, 1, max(1, min(256, most))), rank, adapters,
                  rng.choice(["f32", "master_bf16", "master_f16", "bf16"]), rng.choice(["f32", "bf16", "f16"]),
                  rng.choice([32, 8, 8]), rng.choice([0.0, 0.01, 0.1]), rng.choice([0, 0, 1, 3, 100]))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rows(t, pad):
    """`t` as rows of a buffer that is `pad` elements wider."""
    if not pad:
        return t.contiguous()
    b = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b[:, :t.shape[1]]


def _prepare_norm(c, g):
    rows, n, dt, wdt = c["rows"], c["n"], DT[c["dtype"]], DT[c["weight"]]
    # hidden states: a few columns much larger than the rest, and a mean that is not zero
    col = 1 + 4 * (torch.rand(n, generator=g, device="cuda") < 0.01).float()
    x = _rows((_randn(g, rows, n) * col + 0.3).to(dt), c["pad"])
    s = {"x": x, "gamma": (1 + 0.1 * _randn(g, n)).to(wdt), "beta": (0.1 * _randn(g, n)).to(wdt) if c["bias"] else None}
    if c["op"] == "norm_fwd":
        s.update(y=_rows(torch.zeros(rows, n, dtype=dt, device="cuda"), c["pad"]),
                 mean=torch.empty(rows, device="cuda"), rstd=torch.empty(rows, device="cuda"))
        return s
    xf = x.float()
    mean = xf.mean(1)
    var = (xf - mean[:, None]).square().mean(1)
    s.update(mean=mean, rstd=1 / torch.sqrt(var + EPS), dy=_rows(_randn(g, rows, n).to(dt), c["pad"]),
             dres=_randn(g, rows, n).to(dt) if c["dres"] else None, dx=torch.empty(rows, n, dtype=dt, device="cuda"))
    if c["wgrad"]:
        s.update(dgamma=torch.empty(n, device="cuda"), dbeta=torch.empty(n, device="cuda") if c["bias"] else None)
    return s


def _adapter_offsets(c):
    """First token of each adapter: uneven ranges that start at multiples of 128."""
    T, A = c["tokens"], c["adapters"]
    tiles = T // 128
    return [min(tiles, a * tiles // A + (a % 2 if tiles >= 4 * A else 0)) * 128 for a in range(A)] + [T]


def _prepare_balance(c, g):
    T, E, k, A = c["tokens"], c["experts"], c["topk"], c["adapters"]
    # a router at work: some experts are preferred
    logits = (_randn(g, T, E) + 0.7 * _randn(g, E)).to(DT[c["dtype"]])
    ids = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32)
    if c["masked"]:
        ids[torch.rand(T, k, generator=g, device="cuda") < c["masked"]] = -1
    offsets = _adapter_offsets(c)
    s = {"logits": logits, "ids": ids, "offsets": offsets, "first": torch.tensor(offsets[:-1], device="cuda"), "coef": 0.01,
         "loss": torch.empty(A, device="cuda"), "counts": torch.empty(A, E, dtype=torch.int32, device="cuda"),
         "prob": torch.empty(A, E, device="cuda")}
    if c["grad"]:
        s.update(dloss=0.5 + torch.rand(A, generator=g, device="cuda"), dlogits=torch.empty(T, E, device="cuda"))
    return s


def _factors(c):
    """(name, elements) of the trained tensors of the expert layer, adapter by adapter, and of its router."""
    H, I, E, r, o = c["hidden"], c["inter"], c["experts"], c["rank"], c["odd"]
    one = [("A1", r * H), ("A3", r * H), ("B1", E * I * r), ("B3", E * I * r), ("A2", E * r * I), ("B2", H * r)]
    return [(n, e + o) for _ in range(c["adapters"]) for n, e in one]


def _quantise(x):
    """Blocks of 256 of a flat fp32 tensor as E4M3 values and their fp32 scales."""
    b = x.view(-1, BLOCK)
    finite = torch.isfinite(b)
    top = torch.where(finite, b.abs(), 0.0).amax(1)
    some = top >= TINY
    inv = torch.where(some, E4M3_MAX / top, 0.0)
    q = torch.where(finite, b * inv[:, None], torch.nan).to(torch.float8_e4m3fn)
    return q.view(-1), torch.where(some, top / E4M3_MAX, 0.0)


def _prepare_adamw(c, g):
    # one arena for each kind of data, tensors at multiples of 256 elements, zeros between them
    sizes = [e for _, e in _factors(c)]
    starts, end = [], 0
    for e in sizes:
        starts.append(end)
        end += -(-e // BLOCK) * BLOCK
    used = torch.zeros(end, dtype=torch.bool, device="cuda")
    for at, e in zip(starts, sizes):
        used[at:at + e] = True
    fill = lambda t: torch.where(used, t, 0.0)  # noqa: E731
    w = fill(0.02 * _randn(g, end))
    # gradients of very different sizes from tensor to tensor and element to element
    size = torch.exp(2 * torch.rand(end // BLOCK, generator=g, device="cuda") - 9)
    grad = fill(_randn(g, end) * size.repeat_interleave(BLOCK))
    m = fill(0.3 * grad + 0.1 * _randn(g, end) * size.repeat_interleave(BLOCK))
    v = fill((0.5 * grad).square() + (0.1 * size.square()).repeat_interleave(BLOCK))
    s = {"grad": grad.to(DT[c["grad"]]), "starts": starts, "sizes": sizes, "decay": c["decay"], "lr": 1e-4, "step": STEP,
         "scale": torch.full((1,), 0.7, device="cuda"), "param_kind": c["param"], "bits": c["bits"]}
    low = {"f32": torch.float32, "bf16": torch.bfloat16, "master_bf16": torch.bfloat16, "master_f16": torch.float16}[c["param"]]
    s["param"] = w.to(low)
    if c["param"].startswith("master"):
        s["master"] = w
    if c["bits"] == 32:
        s.update(m=m, v=v)
    else:
        s["m"], s["m_scale"] = _quantise(m)
        s["r"], s["r_scale"] = _quantise(torch.sqrt(v))
    return s


def prepare(case, seed):
    g = _gen(seed)
    make = {"norm_fwd": _prepare_norm, "norm_bwd": _prepare_norm, "balance": _prepare_balance, "adamw": _prepare_adamw}
    s = make[case["op"]](case, g)
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
    y = d * rstd[:, None] * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_bwd(s):
    dy = s["dy"].float()
    h = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    u = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (u - u.mean(1, keepdim=True) - h * (u * h).mean(1, keepdim=True))
    if s["dres"] is not None:
        dx = dx + s["dres"].float()
    out = {"dx": dx.to(s["x"].dtype)}
    if "dgamma" in s:
        out["dgamma"] = (dy * h).sum(0)
        if s["beta"] is not None:
            out["dbeta"] = dy.sum(0)
    return out


def _plain_balance(s):
    logits, ids = s["logits"].float(), s["ids"].long()
    (T, E), A = logits.shape, len(s["offsets"]) - 1
    of = torch.bucketize(torch.arange(T, device="cuda"), s["first"], right=True) - 1  # adapter of each token
    routed = ids >= 0
    slot = torch.where(routed, of[:, None] * E + ids, 0).view(-1)
    counts = torch.zeros(A * E, dtype=torch.long, device="cuda").scatter_add_(0, slot, routed.long().view(-1)).view(A, E)
    live = routed.any(1)
    p = torch.where(live[:, None], torch.softmax(logits, 1), 0.0)
    member = (of[None, :] == torch.arange(A, device="cuda")[:, None]) & live[None, :]
    tokens = member.sum(1).clamp(min=1).float()
    prob = (member.float() @ p) / tokens[:, None]
    f = counts.float() / counts.sum(1, keepdim=True).clamp(min=1).float()
    out = {"loss": s["coef"] * E * (f * prob).sum(1), "counts": counts.to(torch.int32), "prob": prob}
    if "dlogits" in s:
        ft = f[of]
        w = (s["dloss"] * (s["coef"] * E) / tokens)[of]
        out["dlogits"] = w[:, None] * (p * (ft - (p * ft).sum(1, keepdim=True)))
    return out


def _plain_adamw(s):
    bc1, bc2 = 1 - BETA1 ** s["step"], 1 - BETA2 ** s["step"]
    g = s["grad"].float() * s["scale"]
    if s["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        r = (s["r"].float().view(-1, BLOCK) * s["r_scale"][:, None]).view(-1)
        v = r * r
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + ((1 - BETA2) * g) * g
    r = torch.sqrt(v)
    w = s["master"] if "master" in s else s["param"].float()
    w = w * (1 - s["lr"] * s["decay"]) - (s["lr"] / bc1) * (m / (r * (1 / math.sqrt(bc2)) + ADAM_EPS))
    s["param"] = w.to(s["param"].dtype)
    if "master" in s:
        s["master"] = w
    if s["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["m_scale"] = _quantise(m)
        s["r"], s["r_scale"] = _quantise(r)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    names = ["param"] + (["master"] if "master" in s else [])
    return {k: s[k] for k in names + (["m", "v"] if s["bits"] == 32 else ["m", "m_scale", "r", "r_scale"])}


# ------------------------------------------------------------------ the framework's operators
def _own_norm_fwd(s, m):
    m.moe_lora_layernorm_forward(s["x"], s["gamma"], s["beta"], s["y"], s["mean"], s["rstd"], EPS)
    return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}


def _own_norm_bwd(s, m):
    if "scratch" not in s:  # a program keeps one workspace for its sizes
        s["scratch"] = m.layernorm_scratch(*s["x"].shape)
    dgamma, dbeta = s.get("dgamma"), s.get("dbeta")
    m.moe_lora_layernorm_backward(s["x"], s["gamma"], s["mean"], s["rstd"], s["dy"], s["dres"], s["dx"], dgamma, dbeta,
                                  s["scratch"])
    return {k: t for k, t in (("dx", s["dx"]), ("dgamma", dgamma), ("dbeta", dbeta)) if t is not None}


def _own_balance(s, m):
    if "dims" not in s:  # a program has the layer's sizes and keeps a workspace for them
        T, E = s["logits"].shape
        s["dims"] = m.make_dims(T=T, H=512, I=256, E=E, k=s["ids"].shape[1], r=16, A=len(s["offsets"]) - 1)
        s["scratch"] = m.balance_scratch(s["dims"])
    m.moe_lora_balance_loss(s["dims"], s["logits"], s["ids"], s["offsets"], s["coef"], s["loss"], s["counts"], s["prob"],
                            s["scratch"], dlogits=s.get("dlogits"), dloss=s.get("dloss"))
    return {k: s[k] for k in ("loss", "counts", "prob", "dlogits") if k in s}


def _own_adamw(s, m):
    if "tensors" not in s:  # a program lists its tensors once
        def part(key, i, blocks=False):
            at, e = s["starts"][i], s["sizes"][i]
            if key not in s:
                return None
            return s[key][at // BLOCK:at // BLOCK - (-e // BLOCK)] if blocks else s[key][at:at + e]
        b8 = s["bits"] == 8
        s["tensors"] = m.AdamWTensors([
            dict(p=part("param", i), g=part("grad", i), master=part("master", i), m=part("m", i),
                 v=part("r" if b8 else "v", i), m_scale=part("m_scale", i, True) if b8 else None,
                 v_scale=part("r_scale", i, True) if b8 else None, lr=s["lr"], weight_decay=s["decay"])
            for i in range(len(s["sizes"]))])
    m.moe_lora_adamw_step(s["tensors"], s["step"], BETA1, BETA2, ADAM_EPS, grad_scale=s["scale"])
    return _adamw_outputs(s)


def run(state):
    op = state["case"]["op"]
    if own:
        import moe_expert_ffn_top_gb300 as m
        return {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "balance": _own_balance, "adamw": _own_adamw}[op](state, m)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance, "adamw": _plain_adamw}[op](state)


# ------------------------------------------------------------------ work
def work(case):
    c = case
    if c["op"] in ("norm_fwd", "norm_bwd"):
        e, s, w = c["rows"] * c["n"], SIZE[c["dtype"]], c["n"] * SIZE[c["weight"]]
        if c["op"] == "norm_fwd":
            return {"bytes": 2 * e * s + w * (2 if c["bias"] else 1) + 8 * c["rows"], "flops": 8 * e}
        grads = 4 * c["n"] * (2 if c["bias"] else 1) if c["wgrad"] else 0
        return {"bytes": (4 if c["dres"] else 3) * e * s + w + 8 * c["rows"] + grads, "flops": 14 * e}
    if c["op"] == "balance":
        T, E, A = c["tokens"], c["experts"], c["adapters"]
        return {"bytes": T * E * (SIZE[c["dtype"]] + (4 if c["grad"] else 0)) + 4 * T * c["topk"] + 8 * A * E + 4 * A,
                "flops": (9 if c["grad"] else 5) * T * E}
    n = sum(e for _, e in _factors(c))
    low = 4 if c["param"] == "f32" else 2
    weights = 8 + low if c["param"].startswith("master") else 2 * low
    states = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (SIZE[c["grad"]] + weights + states), "flops": 15 * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_norm(c, s):
    x = s["x"].double()
    n = x.shape[1]
    if c["op"] == "norm_fwd":
        mu = x.sum(1, keepdim=True) / n
        x -= mu
        rstd = ((x ** 2).sum(1, keepdim=True) / n + EPS) ** -0.5
        y = x * rstd * s["gamma"].double()
        return {"y": y + s["beta"].double() if c["bias"] else y, "mean": mu[:, 0], "rstd": rstd[:, 0]}
    # the saved statistics are inputs of the backward
    rstd = s["rstd"].double().unsqueeze(1)
    h = (x - s["mean"].double().unsqueeze(1)) * rstd
    dy = s["dy"].double()
    out = {"dgamma": torch.einsum("ij,ij->j", dy, h), "dbeta": dy.sum(0)} if c["wgrad"] else {}
    if not c["bias"]:
        out.pop("dbeta", None)
    dy = dy * s["gamma"].double()
    dx = (dy - (dy.sum(1, keepdim=True) + h * torch.einsum("ij,ij->i", dy, h).unsqueeze(1)) / n) * rstd
    out["dx"] = dx + s["dres"].double() if c["dres"] else dx
    return out


def _exact_balance(c, s):
    E, A = c["experts"], c["adapters"]
    loss, counts, prob = [], [], []
    dl = torch.zeros(c["tokens"], E, dtype=torch.float64, device="cuda")
    for a in range(A):
        lo, hi = s["offsets"][a], s["offsets"][a + 1]
        ids, l = s["ids"][lo:hi], s["logits"][lo:hi].double()
        on = (ids >= 0).any(1)
        e = torch.exp(l - l.amax(1, keepdim=True)) if hi > lo else l
        p = e / e.sum(1, keepdim=True) * on[:, None]
        cnt = torch.stack([(ids == j).sum() for j in range(E)]) if hi > lo else torch.zeros(E, device="cuda")
        N, R = max(1, int(on.sum())), max(1, int(cnt.sum()))
        P, f = p.sum(0) / N, cnt.double() / R
        loss.append(s["coef"] * E * torch.dot(f, P))
        counts.append(cnt)
        prob.append(P)
        if c["grad"]:
            dl[lo:hi] = float(s["dloss"][a]) * s["coef"] * E / N * (p * f - p * (p @ f)[:, None])
    out = {"loss": torch.stack(loss), "prob": torch.stack(prob)}
    return dict(out, dlogits=dl) if c["grad"] else out


def _exact_e4m3(b):
    """Rows of 256 to the nearest E4M3 values (ties to even) and scales, in 64 bits."""
    top = b.abs().amax(1, keepdim=True)
    q = torch.where(top >= TINY, b / torch.where(top >= TINY, top, 1.0) * E4M3_MAX, 0.0)
    _, e = torch.frexp(q)                             # |q| in [2^(e-1), 2^e)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)  # three bits after the leading one, 2^-9 below 2^-6
    return torch.round(q / step) * step, torch.where(top >= TINY, top / E4M3_MAX, 0.0)


def _exact_adamw(c, s):
    f64 = torch.float64
    g = s["grad"].to(f64) * s["scale"].to(f64)
    if c["bits"] == 32:
        m, v = s["m"].to(f64), s["v"].to(f64)
    else:
        m = s["m"].to(f64) * s["m_scale"].to(f64).repeat_interleave(BLOCK)
        v = (s["r"].to(f64) * s["r_scale"].to(f64).repeat_interleave(BLOCK)) ** 2
    m += (1 - BETA1) * (g - m)
    v += (1 - BETA2) * (g ** 2 - v)
    hat_m, hat_r = m / (1 - BETA1 ** STEP), (v / (1 - BETA2 ** STEP)) ** 0.5
    w = (s["master"] if "master" in s else s["param"]).to(f64)
    w = w - s["lr"] * (s["decay"] * w + hat_m / (hat_r + ADAM_EPS))
    out = {"param": w, "master": w} if "master" in s else {"param": w}
    if c["bits"] == 32:
        return dict(out, m=m, v=v)
    (qm, sm), (qr, sr) = _exact_e4m3(m.view(-1, BLOCK)), _exact_e4m3((v ** 0.5).view(-1, BLOCK))
    return dict(out, m=qm.view(-1), m_scale=sm.view(-1), r=qr.view(-1), r_scale=sr.view(-1))


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_fwd": _exact_norm, "norm_bwd": _exact_norm, "balance": _exact_balance, "adamw": _exact_adamw}[case["op"]](case, s)
