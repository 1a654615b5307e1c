"""64-bit definitions of the post-training operators (token log probabilities, policy and
preference losses, Muon) for the tests, with the sizes that their tolerances are made of."""
import math

import torch

U32 = 2.0 ** -24
CHAIN = 256  # longest chain of additions behind one fp32 sum: a thread's own values, then warp, block, cluster


def tokens(logits, targets, inv_temp):
    """logp, lse, entropy of every row as if it had a target (0 where it has none), the
    probabilities, and tolerances of the three.  A probability carries the rounding of its
    exponent (three roundings relative to its distance from the maximum), of the exponential
    (4 units) and of the sum (its chain, and its terms' own errors)."""
    z = logits.double() * inv_temp
    n = z.shape[1]
    ok = (targets >= 0) & (targets < n)
    y = torch.where(ok, targets, 0).long()[:, None]
    top = z.amax(1, keepdim=True)
    top = torch.where(torch.isinf(top) & (top < 0), torch.zeros_like(top), top)
    d = z - top
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    p = e / s
    far = torch.where(p > 0, d.abs(), 0.0)
    ent = s.log()[:, 0] - (p * torch.where(p > 0, d, 0.0)).sum(1)
    logp = (d.gather(1, y) - s.log())[:, 0]
    lse = (top + s.log())[:, 0]
    avg, sq = (p * far).sum(1), (p * far * far).sum(1)
    sum_err = U32 * (CHAIN + 8 + 3 * avg)
    zy = d.gather(1, y)[:, 0].abs()
    tol = {"logp": sum_err + U32 * (4 * zy + 4 * logp.abs() + 4), "lse": sum_err + U32 * (4 * lse.abs() + 4 * top[:, 0].abs() + 4),
           "entropy": sum_err + U32 * ((2 * CHAIN + 16) * (avg + 1) + 8 * sq + 8), "p": sum_err[:, None] + U32 * (3 * far + 8)}
    return {"ok": ok, "y": y, "p": p, "logp": logp, "lse": lse, "entropy": ent, "tol": tol}


def policy(r, adv, old, ref, weight, offsets, dloss, inv_temp, low, high, beta):
    """loss [A], stats [A,4], dlogits of the rows r = tokens(...), and the tolerances of the three."""
    A, T = len(offsets) - 1, len(adv)
    ok = r["ok"] if weight is None else r["ok"] & (weight != 0)
    adv, old = adv.double(), old.double()
    lerr = r["tol"]["logp"] + U32 * ((r["logp"] - old).abs() + 1)
    rho = torch.exp(r["logp"] - old)
    rerr = rho * (lerr + 4 * U32)
    lo, hi = float(torch.tensor(1.0) - torch.tensor(low)), float(torch.tensor(1.0) + torch.tensor(high))
    cut = ((adv > 0) & (rho > hi)) | ((adv < 0) & (rho < lo))
    l = -torch.minimum(rho * adv, rho.clamp(lo, hi) * adv)
    g = torch.where(cut, torch.zeros_like(rho), -rho * adv)
    err = rerr * adv.abs() + 4 * U32 * l.abs()
    gerr = err.clone()
    kl = torch.zeros_like(rho)
    klerr = torch.zeros_like(rho)
    if ref is not None:
        d = ref.double() - r["logp"]
        em = torch.expm1(d)
        kl = em - d
        derr = r["tol"]["logp"] + U32 * d.abs()
        klerr = em.abs() * derr + 4 * U32 * (em.abs() + d.abs())
        l = l + beta * kl
        g = g - beta * em
        err = err + beta * klerr + 2 * U32 * l.abs()
        gerr = gerr + beta * (torch.exp(d) * derr + 4 * U32 * em.abs())
    z = torch.zeros(T, dtype=torch.float64, device=adv.device)
    pick = lambda v: torch.where(ok, v, z)  # noqa: E731
    loss, stats, ltol, stol, coef, ctol = [], [], [], [], z.clone(), z.clone()
    for a in range(A):
        i = slice(offsets[a], offsets[a + 1])
        n = max(1, int(ok[i].sum()))
        w = torch.where(ok[i], torch.full_like(z[i], 1.0 / n) if weight is None else weight[i].double(), z[i])
        terms = [(l, err), (kl, klerr), (cut.double(), z), (rho, rerr), (r["entropy"], r["tol"]["entropy"])]
        sums = [(w * pick(v)[i]).sum() for v, _ in terms]
        tols = [(w.abs() * (pick(e)[i] + (CHAIN + 6) * U32 * pick(v)[i].abs())).sum() + 1e-30 for v, e in terms]
        loss.append(sums[0]), stats.append(torch.stack(sums[1:])), ltol.append(tols[0]), stol.append(torch.stack(tols[1:]))
        up = 1.0 if dloss is None else float(dloss[a])
        coef[i] = up * w * pick(g)[i] * inv_temp
        ctol[i] = (up * w * inv_temp).abs() * pick(gerr)[i] + 8 * U32 * coef[i].abs()
    hot = torch.zeros_like(r["p"])
    hot.scatter_(1, r["y"], 1.0)
    dl = coef[:, None] * (hot - r["p"])
    dl[~ok] = 0
    dtol = ctol[:, None] * (hot + r["p"]) + coef.abs()[:, None] * (r["p"] * r["tol"]["p"] + 3 * U32 * (hot + r["p"]))
    dtol[~ok] = 0
    return torch.stack(loss), torch.stack(stats), dl, torch.stack(ltol), torch.stack(stol), dtol


def preference(logp, targets, seq, ref, offsets, dloss, beta, kind, smooth, margin, average):
    """loss [A], stats [A,4], seq_logp [2P], dlogp [tokens] (NaN where no sequence is), by loops on the host."""
    seq, logp, live = [int(v) for v in seq], logp.double().cpu(), (targets >= 0).cpu()
    P, A = len(seq) // 2, len(offsets) - 1
    norm = [max(1, int(live[a:b].sum())) if average else 1 for a, b in zip(seq, seq[1:])]
    s = [float((logp[a:b] * live[a:b]).sum()) / n for a, b, n in zip(seq, seq[1:], norm)]
    rw = [v - (0.0 if ref is None else float(ref[j])) for j, v in enumerate(s)]
    loss, stats = torch.zeros(A).double(), torch.zeros(A, 4).double()
    dlogp = torch.full_like(logp, math.nan)
    for a in range(A):
        pairs = range(offsets[a], offsets[a + 1])
        for i in pairs:
            h = rw[2 * i] - rw[2 * i + 1]
            x = beta * h - margin
            sig = lambda v: 1 / (1 + math.exp(-v)) if v >= 0 else math.exp(v) / (1 + math.exp(v))  # noqa: E731
            soft = lambda v: max(v, 0.0) + math.log1p(math.exp(-abs(v)))  # noqa: E731
            if kind == "sigmoid":
                l, d = (1 - smooth) * soft(-x) + smooth * soft(x), beta * (smooth * sig(x) - (1 - smooth) * sig(-x))
            elif kind == "squared":
                l, d = (h - 0.5 / beta) ** 2, 2 * (h - 0.5 / beta)
            else:
                l, d = max(0.0, 1 - x), -beta if x < 1 else 0.0
            loss[a] += l / len(pairs)
            stats[a] += torch.tensor([float(x > 0), beta * rw[2 * i], beta * rw[2 * i + 1], h]).double() / len(pairs)
            up = (1.0 if dloss is None else float(dloss[a])) / len(pairs)
            for j, sign in ((2 * i, 1.0), (2 * i + 1, -1.0)):
                dlogp[seq[j]:seq[j + 1]] = live[seq[j]:seq[j + 1]] * (sign * up * d / norm[j])
    return loss, stats, torch.tensor(s).double(), dlogp


def newton_schulz(u, steps, coefs, eps):
    """X of every matrix of u [..., rows, cols] in 64 bits."""
    u = u.double()
    tall = u.shape[-2] > u.shape[-1]
    x = u.mT if tall else u
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + eps)
    a, b, c = coefs
    for _ in range(steps):
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.mT if tall else x


def muon(w, m, g, scale_g, momentum, nesterov, steps, coefs, eps, lr, wd, scale):
    """w and m after a step, and X."""
    g = g.double() * scale_g
    m = momentum * m.double() + (1 - momentum) * g
    u = (1 - momentum) * g + momentum * m if nesterov else m
    x = newton_schulz(u, steps, coefs, eps)
    return w.double() * (1 - lr * wd) - lr * scale * x, m, x
