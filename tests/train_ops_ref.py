"""64-bit definitions of the training-step operators (layer norm, balance loss, AdamW) for
the tests, and the rounding units their tolerances are made of."""
import torch

U32 = 2.0 ** -24
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY_OF = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
# Longest chain of additions behind one fp32 sum of the kernels at the tested sizes: a
# thread's own values, then the warp's, then the block's.  Each addition adds at most
# one rounding unit of the sum of magnitudes.
CHAIN = 256


def norm_fwd(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    y = (x - mean) * rstd
    if gamma is not None:
        y = y * gamma.double()
    if beta is not None:
        y = y + beta.double()
    return y, mean[:, 0], rstd[:, 0]


def norm_bwd(x, gamma, mean, rstd, dy, dres):
    """dx, dgamma, dbeta and, for the tolerances, the sizes of the terms behind each."""
    x, dy = x.double(), dy.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    h = (x - mean) * rstd
    u = dy * gamma.double() if gamma is not None else dy
    a, b = u.mean(1, keepdim=True), (u * h).mean(1, keepdim=True)
    dx = rstd * (u - a - h * b)
    size = rstd * (u.abs() + u.abs().mean(1, keepdim=True) + h.abs() * (u * h).abs().mean(1, keepdim=True))
    # h itself carries the rounding of x - mean
    hs = (x.abs() + mean.abs()) * rstd
    size = size + rstd * (hs * b.abs() + h.abs() * (u.abs() * hs).mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
        size = size + dres.double().abs()
    return dx, (dy * h).sum(0), dy.sum(0), size, (dy.abs() * (h.abs() + hs)).sum(0), dy.abs().sum(0)


def balance(logits, ids, offsets, coef, dloss):
    """loss [A], counts [A,E], prob [A,E], dlogits [T,E] by loops over adapters and tokens."""
    T, E = logits.shape
    A = len(offsets) - 1
    loss, counts, prob = torch.zeros(A).double(), torch.zeros(A, E, dtype=torch.int32), torch.zeros(A, E).double()
    dl = torch.zeros(T, E).double()
    for a in range(A):
        live, ps = [], {}
        for t in range(offsets[a], offsets[a + 1]):
            good = [e for e in ids[t].tolist() if 0 <= e < E]
            for e in good:
                counts[a, e] += 1
            if good:
                live.append(t)
                l = logits[t].double()
                top = l.max()
                p = torch.exp(l - (top if top > float("-inf") or top != top else torch.zeros(())))
                z = p.sum()
                ps[t] = p / z if z != 0 else p
                prob[a] += ps[t]
        if not live:
            continue
        f = counts[a].double() / counts[a].sum()
        prob[a] /= len(live)
        loss[a] = coef * E * (f * prob[a]).sum()
        up = 1.0 if dloss is None else float(dloss[a])
        for t in live:
            dl[t] = up * coef * E / len(live) * ps[t] * (f - (ps[t] * f).sum())
    return loss, counts, prob, dl


def e4m3_values():
    """The 256 values of an E4M3 code (sign, 4 exponent bits of bias 7, 3 mantissa bits; S.1111.111 = NaN)."""
    out = []
    for c in range(256):
        s, e, f = c >> 7, (c >> 3) & 15, c & 7
        v = float("nan") if (e, f) == (15, 7) else (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
        out.append(-v if s else v)
    return torch.tensor(out, dtype=torch.float64)


def adamw32(w, g, m, v, step, b1, b2, eps, lr, wd):
    """One step in 64 bits."""
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    mh, vh = m / (1 - b1 ** step), v / (1 - b2 ** step)
    return w * (1 - lr * wd) - lr * mh / (vh.sqrt() + eps), m, v
