"""The few-token layer and the 8-bit operators in 64 bits (torch on the CPU), with bounds on
what fp32 arithmetic may be off by.  Shared by the GPU tests of moe_few_tokens* and moe_int8_*."""
import math

import torch

U32 = 2.0 ** -24  # half a step of fp32, relative
BF16 = 2.0 ** -8  # half a step of bf16, relative


def codes64(v):
    """(codes, scales) of rows: scale = max|v| / 127, code = round-half-even(127 v / max|v|)."""
    v = v.double()
    a = v.abs().amax(-1, keepdim=True)
    q = torch.where(a > 0, torch.round(127.0 * v / torch.where(a > 0, a, torch.ones_like(a))), torch.zeros_like(v))
    return q, (a / 127.0).squeeze(-1)


def act64(u, kind):
    """Activation of the last axis and a bound factor: |act(u + e) - act(u)| <= slope * |e| elementwise."""
    if kind == "swiglu":
        g, up = u.chunk(2, -1)
        return g * torch.sigmoid(g) * up
    if kind == "gelu":
        return 0.5 * u * (1.0 + torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
    return u


def act_error(u, du, kind):
    """Bound on the fp32 activation's error where u is known within du: GELU and SiLU have slopes within
    1.13 and 1.1.  GELU's exp argument a = 2 sqrt(2/pi) (u + 0.044715 u^3), |a| <= 1.6 |u| + 0.072 |u|^3, takes
    five roundings of terms of one sign and one more inside exp (6 |a| 2^-24); ex2 is within 2 steps, 1 + e one
    rounding, the division 2 steps (9 of 2^-24): below (8 |a| + 16) 2^-24 relative.  SiLU's argument takes
    the one rounding: below (2 |g| + 16) 2^-24.  Past |a| = 90 the result is 0 or u to fp32."""
    if kind == "swiglu":
        g, up = u.chunk(2, -1)
        dg, dup = du.chunk(2, -1)
        s = g * torch.sigmoid(g)
        return 1.1 * dg * (up.abs() + dup) + s.abs() * dup + (g.abs().clamp(max=90) + 8) * 2 * U32 * (s * up).abs()
    if kind == "gelu":
        h = act64(u, "gelu").abs()
        a = (1.6 * u.abs() + 0.072 * u.abs() ** 3).clamp(max=90)
        return 1.13 * du + (8 * a + 16) * U32 * h + 1e-37
    return du


def route64(x, w_r, bias, offset, n, k, scale):
    z = x.double() @ w_r.double().T
    if offset is not None:
        z[:, :n] += offset.double()
    s = torch.sigmoid(z)
    sel = s[:, :n] + bias.double()
    top = torch.sort(sel, dim=1, descending=True, stable=True)
    idx = top.indices[:, :k]
    margin = (top.values[:, k - 1] - top.values[:, k]).min().item() if k < n else math.inf
    gap = (top.values[:, :k].diff(dim=1).abs().min().item() if k > 1 else math.inf)
    who = torch.cat([idx, torch.arange(n, w_r.shape[0]).expand(x.shape[0], -1)], 1)
    kept = torch.gather(s, 1, who)
    return idx, kept / kept.sum(1, keepdim=True) * scale, who, min(margin, gap)


def few64(x, w_r, bias, offset, w1, w2, n, k, scale, act, w1s=None, w2s=None):
    """Outputs, gates, indices, smallest selection gap, and a bound on |kernel - out| for every element.

    The bound: bf16 rounding of the result, plus what fp32 may do before it -- a sum of m products is within
    m 2^-24 of the sum of their magnitudes; gates are within 2^-18; the bf16 path keeps 16 bits of each hidden
    value (2^-16); an 8-bit hidden code may fall on the other side where its quotient is within its error of
    a half-integer, which moves the result by one code."""
    T, d = x.shape
    idx, gates, who, gap = route64(x, w_r, bias, offset, n, k, scale)
    out = torch.zeros(T, d, dtype=torch.float64)
    err = torch.zeros(T, d, dtype=torch.float64)
    int8 = w1s is not None
    for t in range(T):
        for j in range(who.shape[1]):
            e = int(who[t, j])
            g = gates[t, j]
            W1, W2 = w1[e].double(), w2[e].double()
            f = W2.shape[1]
            if int8:
                q, sx = codes64(x[t:t + 1])
                u = ((W1 @ q[0]) * sx * w1s[e].double())
                du = 6 * U32 * u.abs()  # the scales' own rounding and two products
            else:
                u = W1 @ x[t].double()
                du = (d + 4) * U32 * (W1.abs() @ x[t].double().abs())
            h = act64(u, act)
            dh = act_error(u, du, act)
            if int8:
                qh, sh = codes64(h[None])
                a = h.abs().max()
                quot = 127.0 * h / a if a > 0 else h * 0
                dq = 127.0 / a * (dh + quot.abs() / 127.0 * dh.max()) + 8 * U32 * quot.abs() if a > 0 else h * 0
                flips = ((quot - torch.floor(quot) - 0.5).abs() <= dq).double()
                y = (W2 @ qh[0]) * sh * w2s[e].double()
                rel = 6 * U32 + (dh.max() / a if a > 0 else 0.0)
                dy = rel * y.abs() + (W2.abs() @ flips) * sh * w2s[e].double()
            else:
                y = W2 @ h
                dy = W2.abs() @ (dh + 2.0 ** -16 * h.abs()) + (2 * f + 4) * U32 * (W2.abs() @ h.abs())
            out[t] += g * y
            err[t] += g * dy + g * y.abs() * (2.0 ** -18 + 16 * U32)
    return out, gates, idx, gap, err + BF16 * (out.abs() + err) + 1e-38
