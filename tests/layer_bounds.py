"""Gradients of the operators around the SSD by their formulas in float64, each
with a bound of what a float32 evaluation may be off by.

The bounds follow the values: an error is carried through the same recurrence
or sum as the value it belongs to, so they stay tight over long sequences
(what has decayed away takes its error with it).  U = 2^-24; the counts are
those of layer_reference: the sigmoid is off by a relative (2 |v| + 8) U, the
time step by (3 |raw| + 10) U with softplus and U without, the decay
a = exp(d A) by (|d A| (cd + 3) + 3) U with cd the time step's count.  FIRST
covers the products of two errors.  TINY is float32's smallest normal number:
the exponential gives 0 for results below it, so a decay is also off by TINY,
and with it what it multiplies by TINY times that (64 states at time steps of
0.7 reach exp(-90) = 8e-40 in one token).
"""
import torch

from layer_reference import F, U, conv, grads, half_step, lengths_of, norm, norm_terms, silu, softplus

FIRST = 1 + 2.0 ** -8
TINY = 2.0 ** -126


def _rounded(want, err, dtype):
    return err + half_step(dtype) * (want.abs() + err)


def scan_gradients(u, dt, A, B, C, D, z, dt_bias, init, lengths, use_softplus, dy, dfinal, dtype):
    """{name: (gradient, bound)} of selective_scan; inputs float64 (D, z, dt_bias, init and
    dfinal may be None).  States and their gradients are carried over chunks,
    which adds the decay over a chunk and a second sum: twice the recurrence's bound,
    as in scan_bounds."""
    b, n, ch = u.shape
    ns, groups = A.shape[1], B.shape[2]
    lens = torch.tensor(lengths_of(lengths, b, n))
    live = (torch.arange(n) < lens[:, None])[..., None]
    keep = lambda v: torch.where(live, v, torch.zeros_like(v))
    raw = keep(dt if dt_bias is None else dt + dt_bias)
    d = keep(softplus(raw) if use_softplus else raw)
    cd = 3 * raw.abs() + 10 if use_softplus else torch.ones_like(raw)
    u, dy = keep(u), keep(dy)
    z = None if z is None else keep(z)
    Bs, Cs = (torch.where(live[..., None], v, torch.zeros_like(v)).repeat_interleave(ch // groups, 2)
              for v in (B, C))
    zero = u.new_zeros((b, ch, ns))
    h0 = zero if init is None else init
    w = d * u
    sg = None if z is None else 1 / (1 + torch.exp(-z))
    q = dy if z is None else dy * z * sg
    rq = torch.zeros_like(q) if z is None else 2 * z.abs() + 12
    Dv = u.new_zeros(ch) if D is None else D

    hs, eh = [h0], [zero]           # states before token t, and their errors
    for t in range(n):
        dA = d[:, t, :, None] * A
        a, c3 = torch.exp(dA), cd[:, t, :, None] + 3
        term = w[:, t, :, None] * Bs[:, t]
        new = a * hs[-1] + term
        e = a * eh[-1] + U * ((dA.abs() * c3 + 3) * (a * hs[-1]).abs() + c3 * term.abs() + new.abs())
        e = e + TINY * (1 + hs[-1].abs())
        on = live[:, t, :, None]
        hs.append(torch.where(on, new, hs[-1]))
        eh.append(torch.where(on, e, eh[-1]))
    ag, ea = (zero if dfinal is None else dfinal), zero
    out = {k: [None] * n for k in ("g", "eg", "m", "em", "h", "eh")}
    for t in range(n - 1, -1, -1):
        on = live[:, t, :, None]
        dA = d[:, t, :, None] * A
        a, c3 = torch.exp(dA), cd[:, t, :, None] + 3
        qC = q[:, t, :, None] * Cs[:, t]
        g = ag + qC
        eg = ea + U * (rq[:, t, :, None] * qC.abs() + g.abs())
        nag = a * g
        nea = a * eg + U * (dA.abs() * c3 + 4) * nag.abs() + TINY * (1 + g.abs())
        # what a kernel holds: the recurrence's error twice (chunks), and a rounding
        full = lambda e, v: 2 * e + U * v.abs()
        m, hp = nag * hs[t], full(eh[t], hs[t])
        em = full(nea, nag) * hs[t].abs() + nag.abs() * hp + U * m.abs()
        for k, v in (("g", g), ("eg", full(eg, g)), ("m", m), ("em", em), ("h", hs[t + 1]),
                     ("eh", full(eh[t + 1], hs[t + 1]))):
            out[k][t] = torch.where(on, v, zero)
        ag, ea = torch.where(on, nag, ag), torch.where(on, nea, ea)
    g, eg, m, em, h, eh = (torch.stack(out[k], 1) for k in ("g", "eg", "m", "em", "h", "eh"))

    gB, egB = (g * Bs).sum(-1), (eg * Bs.abs()).sum(-1) + (ns + 4) * U * (g * Bs).abs().sum(-1)
    gA = (m * A).sum(-1)
    egA = (em * A.abs()).sum(-1) + (ns + 8) * U * (m * A).abs().sum(-1)
    dd = gB * u + gA
    edd = egB * u.abs() + egA + 2 * U * ((gB * u).abs() + gA.abs())
    if use_softplus:
        s = keep(1 / (1 + torch.exp(-raw)))
        edd = (edd + (3 * raw.abs() + 10) * U * dd.abs()) * s
        dd = dd * s
    else:
        dd, edd = keep(dd), keep(edd)
    du = gB * d + Dv * q
    edu = egB * d.abs() + (cd + 2) * U * (gB * d).abs() + (rq + 2) * U * (Dv * q).abs()
    # an element of a sum over tokens passes a chunk's 64 tokens at most, then the parts of
    # the batch's chunks (16 tokens at least): eight at a time by a tree, every sixteenth
    # eight in a row, up to seven single ones, and 16 wavefronts; one over channels 16
    # lanes by halves, four wavefronts and the channel tiles
    over_tokens = 64 + 3 + b * -(-n // 16) // 128 + 1 + 7 + 16
    over_channels = 8 + -(-(ch // groups) // 64)

    def by_group(v, e):
        v, e = (x.view(b, n, groups, -1, ns) for x in (v, e))
        return v.sum(3), e.sum(3) + over_channels * U * v.abs().sum(3)

    def over_time(v, e):
        dims = tuple(range(2))
        return v.sum(dims), e.sum(dims) + over_tokens * U * v.abs().sum(dims)

    gw, qh = g * w[..., None], h * q[..., None]
    r = {"du": (du, edu), "ddt": (dd, edd)}
    r["dA"] = over_time(m * d[..., None],
                        em * d.abs()[..., None] + (cd[..., None] + 1) * U * (m * d[..., None]).abs())
    r["dB"] = by_group(gw, eg * w.abs()[..., None] + (cd[..., None] + 2) * U * gw.abs())
    r["dC"] = by_group(qh, eh * q.abs()[..., None] + (rq[..., None] + 1) * U * qh.abs())
    r["dD"] = None if D is None else over_time(q * u, (rq + 2) * U * (q * u).abs())
    r["dz"] = None
    if z is not None:
        s = (h * Cs).sum(-1) + Dv * u
        es = (eh * Cs.abs()).sum(-1) + (ns + 6) * U * ((h * Cs).abs().sum(-1) + (Dv * u).abs())
        slope = sg * (1 + z * (1 - sg))
        eslope = U * (2 * z.abs() + 12) * (1 + z.abs()) * sg
        v = dy * s * slope
        r["dz"] = v, dy.abs() * (es * slope.abs() + s.abs() * eslope) + 3 * U * v.abs()
    r["ddt_bias"] = None if dt_bias is None else over_time(dd, edd)
    r["dinit"] = ag, 2 * ea + U * ag.abs()
    for k, v in r.items():
        if v is not None:
            want, err = v[0], FIRST * v[1]
            r[k] = want, _rounded(want, err, dtype) if k in ("du", "ddt", "dB", "dC", "dz") else err
    return r


def conv_gradients(x, weight, bias, init, lengths, act, dy, dfinal, dtype):
    """{name: (gradient, bound)} of conv1d.  The recomputed sum is off by W + 2
    roundings (through silu's curvature of at most 0.5), its slope and the products
    by (3 |p| + 20) U, dx's sum by W + 2; the weights' sums pass a tile's 32 tokens,
    its four wavefronts and the parts of the batch's tiles (32 tokens at least)."""
    b, n, c = x.shape
    w = weight.shape[1]
    start = x.new_zeros(b, w - 1, c) if init is None else init
    a = [x, weight, bias, start]
    want = grads(lambda *v: conv(*v, lengths, act), a, (dy, dfinal))
    sizes = [None if v is None else v.abs() for v in a]
    slope = 1.1 if act else 1.0
    eg = dy.abs() * 2 * U
    if act:
        p, _ = conv(*a, lengths, False)
        ps, _ = conv(*sizes, lengths, False)
        eg = dy.abs() * (0.5 * (w + 2) * U * ps + slope * (3 * p.abs() + 20) * U)
    plain = lambda *v: conv(*v, lengths, False)
    big = grads(plain, sizes, (slope * dy.abs(), dfinal.abs()))
    off = grads(plain, sizes, (eg, 0 * dfinal))
    r = {}
    for i, name in enumerate(("dx", "dweight", "dbias", "dinit")):
        if a[i] is None:
            r[name] = None
            continue
        if name in ("dx", "dinit"):
            r[name] = want[i], _rounded(want[i], off[i] + (w + 2) * U * big[i], dtype)
        else:
            r[name] = want[i], off[i] + (36 + b * -(-n // 32)) * U * big[i]
    return r


def norm_gradients(x, weight, bias, z, groups, kind, eps, dy, dtype):
    """{name: (gradient, bound)} of norm.  With d = dy w, dv = rstd (d - mean(d) -
    xh mean(d xh)) is off by rstd times [n + 4 roundings of the means' terms, and xh's
    error in each of its two places] and rstd's own relative error; dx and dz add the
    gate's (3 |z| + 24) U.  dweight and dbias pass at most rows + 12 additions."""
    rows = x.shape[0]
    want = grads(lambda *v: norm(*v, groups, kind, eps), (x, weight, bias, z), (dy,))
    xh, e, rstd, er = norm_terms(x, z, groups, kind, eps)
    n = x.shape[1] // groups
    d = (dy * weight).view(xh.shape).abs()
    mean = lambda v: v.mean(-1, keepdim=True)
    sizes = d + (mean(d) if kind == "layer" else 0) + xh.abs() * mean(d * xh.abs())
    off = (n + 4) * U * sizes + e * mean(d * xh.abs()) + xh.abs() * mean(d * e)
    edv = (rstd * (off + (er + 4 * U) * sizes)).reshape(x.shape)
    big = (rstd * sizes).reshape(x.shape)
    xhf, ef = xh.reshape(x.shape), e.reshape(x.shape)
    r = {"dz": None}
    if z is None:
        r["dx"] = want[0], _rounded(want[0], edv, dtype)
    else:
        g = (3 * z.abs() + 24) * U
        r["dx"] = want[0], _rounded(want[0], (edv + g * big) * silu(z).abs(), dtype)
        r["dz"] = want[3], _rounded(want[3], (edv + g * big) * x.abs() * 1.1, dtype)
    r["dweight"] = want[1], (dy.abs() * ef).sum(0) + (rows + 12) * U * (dy * xhf).abs().sum(0)
    r["dbias"] = None if bias is None else (want[2], (rows + 12) * U * dy.abs().sum(0))
    return r
