"""64-bit models of the attention's forward and backward pass and of rotary
positions with per-head norms, from the formulas, on whatever device the
inputs are on. Beside each value comes the sum of the absolute terms it is made
of, which the tests' tolerances go by."""
import math

import torch


def attention(q, k, v, sinks, cu_q, cu_k, hkv, scale, causal, window):
    """(out, lse) in 64 bits of q [T, Hq, d], k, v ragged HND; differentiable."""
    T, hq, d = q.shape
    G = hq // hkv
    outs, lses = [], []
    for a, b, s, t in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        lq, lk = b - a, t - s
        see = visible(lq, lk, causal, window, q.device)
        kk = k[hkv * s:hkv * t].view(hkv, lk, d).repeat_interleave(G, 0)
        vv = v[hkv * s:hkv * t].view(hkv, lk, d).repeat_interleave(G, 0)
        l = torch.einsum("ihd,hjd->hij", q[a:b], kk) * scale
        l = l.masked_fill(~see, -math.inf)
        if sinks is not None:
            l = torch.cat([l, sinks.view(hq, 1, 1).expand(hq, lq, 1)], 2)
        lse = torch.logsumexp(l, 2)
        w = torch.exp(l - lse.masked_fill(lse == -math.inf, 0.0)[..., None])[..., :lk]
        outs.append(torch.einsum("hij,hjd->ihd", w, vv))
        lses.append(lse.t())
    return torch.cat(outs), torch.cat(lses)


def visible(lq, lk, causal, window, dev):
    i = torch.arange(lq, device=dev)[:, None] + lk - lq
    j = torch.arange(lk, device=dev)[None, :]
    see = torch.ones((lq, lk), dtype=torch.bool, device=dev)
    if causal:
        see &= j <= i
        if window > 0:
            see &= j > i - window
    return see


def attention_gradients(dout, q, k, v, out, lse, sinks, cu_q, cu_k, hkv, scale, causal, window,
                        dlse=None):
    """{name: (gradient, tolerance)} as functions of what the forward pass left.

    Rounding. The weight P_ij and dS_ij are rounded to bf16 (2^-8 of each) and
    the result once more (2^-8 of it). In 32 bits, a sum of d products is off
    by at most d 2^-24 <= 2^-17 of its absolute terms; an exponent, with
    logits and log-sum-exp below 2^6 in magnitude and 2^-17 of the logit's terms
    (below 2^6 too, for these inputs), moves a weight by less than 2^-10 of it;
    sums over keys or rows add less than 2^-12 (below 2^12 terms).
    """
    f = [x.double() for x in (dout, q, k, v, out, lse)]
    dout, q, k, v, out, lse = f
    T, hq, d = q.shape
    G = hq // hkv
    rel = 2.0 ** -8 + 2.0 ** -10 + 2.0 ** -11
    delta = (dout * out).sum(-1)
    delta_abs = (dout * out).abs().sum(-1)
    if dlse is not None:
        delta = delta - dlse.double()
        delta_abs = delta_abs + dlse.double().abs()
    z = {n: (torch.zeros_like(x), torch.zeros_like(x)) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    for a, b, s, t in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        lq, lk = b - a, t - s
        see = visible(lq, lk, causal, window, q.device)
        for h in range(hq):
            r = slice(hkv * s + (h // G) * lk, hkv * s + (h // G + 1) * lk)
            l = scale * (q[a:b, h] @ k[r].T)
            p = torch.where(see, torch.exp(l - lse[a:b, h, None]), 0.0)
            e = p * (dout[a:b, h] @ v[r].T - delta[a:b, h, None])
            # what dS may be off by: its own rounding, and that of the difference's terms
            off = rel * e.abs() + 2.0 ** -16 * p * (
                dout[a:b, h].abs() @ v[r].abs().T + delta_abs[a:b, h, None])
            for name, at, val, tol in (
                    ("dq", (slice(a, b), h), scale * (e @ k[r]), scale * (off @ k[r].abs())),
                    ("dk", r, scale * (e.T @ q[a:b, h]), scale * (off.T @ q[a:b, h].abs())),
                    ("dv", r, p.T @ dout[a:b, h], rel * (p.T @ dout[a:b, h].abs()))):
                z[name][0][at] += val
                z[name][1][at] += tol
    res = {n: (val, tol + 2.0 ** -8 * val.abs() + 1e-30) for n, (val, tol) in z.items()}
    if sinks is not None:
        w = torch.exp(sinks.double() - lse)
        res["dsinks"] = (-(w * delta).sum(0), (w * (2.0 ** -12 * delta.abs() + 2.0 ** -16 * delta_abs)
                                               ).sum(0) + 1e-30)
    return res


# ----------------------------------------------------------------------------
class Rotation:
    """x -> R x and its transpose in 64 bits, by the definition."""

    def __init__(self, inv_freq, factor, interleaved, positions):
        n = len(inv_freq)
        i = torch.arange(n, device=positions.device)
        self.first = 2 * i if interleaved else i
        self.second = 2 * i + 1 if interleaved else n + i
        angle = positions.double()[:, None] * torch.tensor(inv_freq, dtype=torch.float64,
                                                           device=positions.device)
        self.cos, self.sin = factor * angle.cos()[:, None], factor * angle.sin()[:, None]
        self.factor = abs(factor)

    def __call__(self, x, back=False):
        a, b = x[..., self.first], x[..., self.second]
        sin = -self.sin if back else self.sin
        y = x.clone()
        y[..., self.first] = a * self.cos - b * sin
        y[..., self.second] = b * self.cos + a * sin
        return y

    def size(self, x):
        """The absolute terms of each element of R x (or of its transpose).

        An angle that is off by t moves a cos - b sin by up to t (|a sin| + |b cos|),
        which may be large where both terms are small (cos and b near 0). In
        32 bits t is at most pi 2^-24 (the angle's fraction of a turn has 24
        bits), and cos and sin are off by less than 2^-23 themselves: together
        less than 2^-21 (|a| + |b|), that is 2^-4 (|a| + |b|) at 2^-17 of the terms."""
        a, b = x[..., self.first].abs(), x[..., self.second].abs()
        y = x.abs()
        angle = 2.0 ** -4 * self.factor * (a + b)
        y[..., self.first] = a * self.cos.abs() + b * self.sin.abs() + angle
        y[..., self.second] = b * self.cos.abs() + a * self.sin.abs() + angle
        return y


def norm(x, w, eps):
    x = x.double()
    if w is None:
        return x
    return w.double() * x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)


def rotated(x, w, eps, rot):
    """(y, sum of absolute terms) of norm and rotation."""
    n = norm(x, w, eps)
    return rot(n), rot.size(n)


def rotated_gradients(g, x, w, eps, rot):
    """(dx, its absolute terms, dw, its absolute terms) given dL/dy = g."""
    back, size = rot(g.double(), back=True), rot.size(g.double())
    if w is None:
        return back, size, None, None
    x, w = x.double(), w.double()
    rs = torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * rs
    u = w * back
    dx = rs * (u - xh * (u * xh).mean(-1, keepdim=True))
    us = w.abs() * size
    dxs = rs * (us + xh.abs() * (us * xh.abs()).mean(-1, keepdim=True))
    return dx, dxs, (back * xh).sum((0, 1)), (size * xh.abs()).sum((0, 1))


def hnd_rows(cu, hkv, dev="cpu"):
    """Ragged HND rows [tokens, Hkv] of the tokens of each sequence."""
    rows = []
    for a, b in zip(cu[:-1], cu[1:]):
        h = torch.arange(hkv)[None, :] * (b - a)
        rows.append(hkv * a + torch.arange(b - a)[:, None] + h)
    return torch.cat(rows).to(dev) if rows else torch.zeros((0, hkv), dtype=torch.long, device=dev)
