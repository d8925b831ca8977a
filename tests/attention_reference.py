"""Plain float64 forms of the operators of an attention layer, on the CPU, and
what their float32 evaluation may be off by.

Error bounds.  U = 2^-24 is half a step of float32 and ``half_step`` that of a
type, both relative to the value.  A sum of n products is off by at most
(n + 1) U times the sum of their sizes; exp2, log2 and the reciprocal are taken
as good to 2 U each.  With bfloat16 inputs the weights P and the gradients dS
are rounded to bfloat16 (a relative ``half_step``) before the products that
take them.  Every bound is a size computed in float64 times such a count; none
was fitted to a result.
"""
import math

import torch

F = torch.float64
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def weight_step(dtype):
    """The rounding of weights before a product: none in float32."""
    return half_step(dtype) if dtype is torch.bfloat16 else 0.0


def to64(t):
    return None if t is None else t.detach().cpu().to(F)


# ---------------------------------------------------------------------- rotary


def rotary(x, inv_freq, positions, layout, scale, back=False):
    """x[tokens, heads, D] in float64; positions [tokens]."""
    r = 2 * inv_freq.numel()
    a = positions.to(F)[:, None] * inv_freq.to(F)
    c, s = scale * torch.cos(a)[:, None], scale * torch.sin(a)[:, None] * (-1 if back else 1)
    y = x.clone()
    one, two = ((slice(0, r // 2), slice(r // 2, r)) if layout == "half" else
                (slice(0, r, 2), slice(1, r, 2)))
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., one] * s + x[..., two] * c
    return y


def rotary_bound(x, y, r, layout, scale, dtype):
    """Two products and a sum of values of a pair, sine and cosine good to 4 U of 1 (the part of
    a turn is rounded to float32: pi U; the functions to 2 U) with the factor's product 1 more:
    10 U of the pair's sizes covers all; then the rounding to the type."""
    one, two = ((slice(0, r // 2), slice(r // 2, r)) if layout == "half" else
                (slice(0, r, 2), slice(1, r, 2)))
    e = torch.zeros_like(y)
    size = scale * (x[..., one].abs() + x[..., two].abs())
    e[..., one] = 10 * U * size
    e[..., two] = 10 * U * size
    return e + half_step(dtype) * (y.abs() + e) * (e > 0)


# ------------------------------------------------------------------- attention


def spans(starts, lengths, rows, batch, most):
    """[(first row in the flat tensor, tokens)] of every sequence."""
    if starts is not None:
        s = [min(max(int(v), 0), rows) for v in starts]
        return [(a, max(0, b - a)) for a, b in zip(s, s[1:])]
    n = [most] * batch if lengths is None else [min(max(int(v), 0), most) for v in lengths]
    return [(i * most, v) for i, v in enumerate(n)]


def one_head(q, k, v, causal, scale):
    """(weights, o, lse) of q[nq,D], k, v [nk,D]."""
    nq, nk = q.shape[0], k.shape[0]
    s = scale * (q @ k.t())
    if causal:
        i = torch.arange(nq)[:, None] + nk - nq
        s = s.masked_fill(torch.arange(nk)[None] > i, -math.inf)
    m = s.amax(-1, keepdim=True) if nk else s.new_full((nq, 1), -math.inf)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total == 0, torch.ones_like(total), total)
    return s, p, p @ v, (m + torch.log(total))[:, 0]


def score_error(q, k, s, lse, scale):
    """Relative error of exp(s - x) where x is good to its own rounding: the product's sum, the
    scale and base change (3 roundings of s and of what is subtracted) and exp2."""
    d = q.shape[1]
    size = scale * (q.abs() @ k.abs().t())
    seen = torch.where(torch.isinf(s), torch.zeros_like(s), s)
    top = torch.where(torch.isinf(lse), torch.zeros_like(lse), lse)[:, None]
    return ((d + 2) * size + 3 * (seen.abs() + top.abs() + size.amax(-1, keepdim=True)) + 2) * U


def attention(q, k, v, q_spans, k_spans, causal, scale, dtype, dout=None):
    """Flat q[rows,H,D], k, v [rows,G,D] in float64: a dict with o, lse and, with dout, dq, dk,
    dv, and a dict with the bounds of their errors."""
    h, g = q.shape[1], k.shape[1]
    rep = h // g
    out = {"o": torch.zeros_like(q), "lse": q.new_full(q.shape[:2], -math.inf)}
    err = {"o": torch.zeros_like(q), "lse": q.new_zeros(q.shape[:2])}
    if dout is not None:
        for name, t in (("dq", q), ("dk", k), ("dv", v)):
            out[name], err[name] = torch.zeros_like(t), torch.zeros_like(t)
    ws, hs = weight_step(dtype), half_step(dtype)
    for (q0, nq), (k0, nk) in zip(q_spans, k_spans):
        if nq == 0 or nk == 0:
            continue
        rows, keys = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for j in range(h):
            a, b, c = q[rows, j], k[keys, j // rep], v[keys, j // rep]
            s, p, o, lse = one_head(a, b, c, causal, scale)
            e = score_error(a, b, s, lse, scale)
            # sums over nk terms, scaled down at most once a tile, joined once more
            sums = (nk + nk // 32 + 8) * U
            pv = p @ c.abs()
            eo = (p * (e + ws)) @ c.abs() + ((p * e).sum(-1, keepdim=True) + 2 * sums + 4 * U) * pv
            none = torch.isinf(lse)
            el = (p * e).sum(-1) + sums + 4 * U * (1 + torch.where(none, torch.zeros_like(lse), lse).abs())
            out["o"][rows, j], out["lse"][rows, j] = o, lse
            err["o"][rows, j] = eo + hs * (o.abs() + eo)
            err["lse"][rows, j] = el
            if dout is None:
                continue
            t = dout[rows, j]
            d = a.shape[1]
            dp = t @ c.t()
            delta = (t * o).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            ep = e + el[:, None] + 2 * U * torch.where(none, torch.zeros_like(lse), lse).abs()[:, None]
            edp = (d + 1) * U * (t.abs() @ c.abs().t())
            ed = (t.abs() * err["o"][rows, j]).sum(-1, keepdim=True) + \
                (d + 1) * U * (t * o).abs().sum(-1, keepdim=True)
            eds = p * (edp + ed + 2 * U * (dp.abs() + delta.abs())) + ds.abs() * (ep + ws)
            nsum = (nq * rep + 8) * U
            one = p * (ep + ws)
            out["dv"][keys, j // rep] += p.t() @ t
            err["dv"][keys, j // rep] += one.t() @ t.abs() + nsum * (p.t() @ t.abs())
            out["dq"][rows, j] = scale * (ds @ b)
            err["dq"][rows, j] = scale * (eds @ b.abs() + (nk + 8) * U * (ds.abs() @ b.abs()))
            out["dk"][keys, j // rep] += scale * (ds.t() @ a)
            err["dk"][keys, j // rep] += scale * (eds.t() @ a.abs() + nsum * (ds.abs().t() @ a.abs()))
    if dout is not None:
        for name in ("dq", "dk", "dv"):
            err[name] += hs * (out[name].abs() + err[name])
    return out, err


def step(q, k, v, k_cache, v_cache, lengths, k_prefix, v_prefix, scale, dtype):
    """One token of every sequence in float64: (o, bound, the caches after it)."""
    b, h, d = q.shape
    rows, g = k_cache.shape[1], k.shape[1]
    o, err = torch.zeros_like(q), torch.zeros_like(q)
    kc, vc = k_cache.clone(), v_cache.clone()
    for i in range(b):
        n = min(max(int(lengths[i]), 0), rows)
        ks, vs = [k_cache[i, :n], k[i:i + 1]], [v_cache[i, :n], v[i:i + 1]]
        if k_prefix is not None:
            ks, vs = [k_prefix] + ks, [v_prefix] + vs
        ks, vs = torch.cat(ks), torch.cat(vs)
        one, e = attention(q[i:i + 1], ks, vs, [(0, 1)], [(0, ks.shape[0])], False, scale, dtype)
        o[i], err[i] = one["o"][0], e["o"][0]
        if n < rows:
            kc[i, n], vc[i, n] = k[i], v[i]
    return o, err, kc, vc
