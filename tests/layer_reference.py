"""Plain float64 forms of the operators around the SSD (convolution, selective
scan, norm), differentiable, on the CPU, and what their float32 evaluation may
be off by.

Error bounds.  U = 2^-24 is half a step of float32 (relative to the value) and
``half_step`` that of the output's type.  A sum of n products is off by at
most (n + 1) U times the sum of their sizes; exp2 and the reciprocal are taken
as good to 2 U each, and the exponential's argument, rounded on its way in,
adds its own size times 2 U.  The sigmoid is then off by a relative
(2 |v| + 8) U.  Every bound below is a size computed in float64 times such a
count; none was fitted to a result.
"""
import torch

F = torch.float64
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def silu(v):
    return v / (1 + torch.exp(-v))


def to64(t):
    return None if t is None else t.detach().cpu().to(F)


def lengths_of(lengths, b, n):
    if lengths is None:
        return [n] * b
    return [min(max(int(v), 0), n) for v in lengths]


# ---------------------------------------------------------------------- conv1d


def conv(x, weight, bias, init, lengths=None, act=True):
    """(y, final state) of x[B,L,C] in float64; zeros behind a sequence's length."""
    b, n, c = x.shape
    w = weight.shape[1]
    if init is None:
        init = x.new_zeros((b, w - 1, c))
    ys, finals = [], []
    for i, m in enumerate(lengths_of(lengths, b, n)):
        rows = torch.cat([init[i], x[i, :m]])
        finals.append(rows[m:])
        p = x.new_zeros((m, c)) if bias is None else bias.expand(m, c)
        for k in range(w):
            p = p + weight[:, k] * rows[k:k + m]
        ys.append(torch.cat([silu(p) if act else p, x.new_zeros((n - m, c))]))
    return torch.stack(ys), torch.stack(finals)


def conv_bound(x, weight, bias, init, lengths, act, dtype):
    """Largest error of y: the sum's W + 2 roundings on the sum of the terms'
    sizes (silu's slope is at most 1.1), the sigmoid's, two products, and the
    rounding to the output's type."""
    w = weight.shape[1]
    size, _ = conv(x.abs(), weight.abs(), None if bias is None else bias.abs(),
                   None if init is None else init.abs(), lengths, act=False)
    p, _ = conv(x, weight, bias, init, lengths, act=False)
    y = silu(p) if act else p
    err = 1.1 * (w + 2) * U * size + (2 * p.abs() + 12) * U * y.abs()
    return err + half_step(dtype) * (y.abs() + err)


# --------------------------------------------------------------- selective scan


def softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def scan(u, dt, A, B, C, D, z, dt_bias, init, lengths=None, use_softplus=True):
    """(y, final state) of the recurrence, token by token; u, dt, z [B,L,D]."""
    b, n, ch = u.shape
    per = ch // B.shape[2]
    raw = dt if dt_bias is None else dt + dt_bias
    d = softplus(raw) if use_softplus else raw
    h = u.new_zeros((b, ch, A.shape[1])) if init is None else init
    lens = torch.tensor(lengths_of(lengths, b, n))
    ys = []
    for t in range(n):
        live = (t < lens)[:, None, None]
        Bt, Ct = (v[:, t].repeat_interleave(per, 1) for v in (B, C))
        new = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * u[:, t])[..., None] * Bt
        h = torch.where(live, new, h)
        s = (h * Ct).sum(-1)
        if D is not None:
            s = s + D * u[:, t]
        if z is not None:
            s = s * silu(z[:, t])
        ys.append(torch.where(live[..., 0], s, torch.zeros_like(s)))
    return torch.stack(ys, 1), h


def scan_bounds(u, dt, A, B, C, D, z, dt_bias, init, lengths, use_softplus, dtype):
    """Largest errors of (y, final state).  The time step d is off by a relative
    cd U: 3 |raw| + 10 with softplus (the sum with its bias, the exponential's
    argument, the series), 1 without.  The decay exp(d A) is then off by a
    relative (|d A| (cd + 3) + 3) U and the input term by (cd + 3) U, and the
    state's error follows the same recurrence as the state.  Chunks that are
    carried add the decay over a chunk (the same relative error, summed) and a
    second sum: twice the recurrence's bound covers both."""
    b, n, ch = u.shape
    per = ch // B.shape[2]
    raw = dt if dt_bias is None else dt + dt_bias
    d = softplus(raw) if use_softplus else raw
    cd = 3 * raw.abs() + 10 if use_softplus else torch.ones_like(raw)
    lens = torch.tensor(lengths_of(lengths, b, n))
    h = u.new_zeros((b, ch, A.shape[1])) if init is None else init
    e = torch.zeros_like(h)
    out = []
    for t in range(n):
        live = (t < lens)[:, None, None]
        Bt, Ct = (v[:, t].repeat_interleave(per, 1) for v in (B, C))
        dA = d[:, t, :, None] * A
        a = torch.exp(dA)
        term = (d[:, t] * u[:, t])[..., None] * Bt
        new = a * h + term
        grown = a * e + U * ((dA.abs() * (cd[:, t, :, None] + 3) + 3) * (a * h).abs()
                             + (cd[:, t, :, None] + 3) * term.abs() + new.abs())
        e = torch.where(live, grown, e)
        h = torch.where(live, new, h)
        size = (h * Ct).abs().sum(-1)
        s = (h * Ct).sum(-1)
        if D is not None:
            size = size + (D * u[:, t]).abs()
            s = s + D * u[:, t]
        err = 2 * (e * Ct.abs()).sum(-1) + (A.shape[1] + 8) * U * size
        if z is not None:
            zt = z[:, t]
            err = err * silu(zt).abs() + (2 * zt.abs() + 12) * U * (s * silu(zt)).abs()
            s = s * silu(zt)
        err = err + half_step(dtype) * (s.abs() + err)
        out.append(torch.where(live[..., 0], err, torch.zeros_like(err)))
    return torch.stack(out, 1), 2 * e + U * h.abs()


def scan_gradient_sizes(u, dt, A, B, C, D, z, dt_bias, init, lengths, use_softplus, dy, dfinal):
    """The backward formulas with every term by its size: what a rounding's
    relative error multiplies.  Order as the inputs."""
    b, n, ch = u.shape
    ns, groups = A.shape[1], B.shape[2]
    raw = dt if dt_bias is None else dt + dt_bias
    d = softplus(raw) if use_softplus else raw
    lens = torch.tensor(lengths_of(lengths, b, n))
    live = (torch.arange(n) < lens[:, None])[..., None]
    d = torch.where(live, d, torch.zeros_like(d)).abs()
    u, dy = (torch.where(live, v, torch.zeros_like(v)).abs() for v in (u, dy))
    Bs, Cs = (torch.where(live[..., None], v, torch.zeros_like(v)).abs().repeat_interleave(
        ch // groups, 2) for v in (B, C))
    a = torch.exp(-d[..., None] * A.abs())
    h, hs = init.abs(), [init.abs()]
    for t in range(n):
        h = a[:, t] * h + (d * u)[:, t, :, None] * Bs[:, t]
        hs.append(h)
    hs = torch.stack(hs, 1)
    q = dy if z is None else dy * silu(z).abs()
    g, gs = dfinal.abs(), []
    for t in range(n - 1, -1, -1):
        g = g + q[:, t, :, None] * Cs[:, t]
        gs.append(g)
        g = a[:, t] * g
    gs = torch.stack(gs[::-1], 1)
    m = gs * a * hs[:, :-1]
    gB = (gs * Bs).sum(-1)
    Ds = torch.zeros(ch, dtype=F) if D is None else D.abs()
    ddt = (m * A.abs()).sum(-1) + gB * u
    y = (hs[:, 1:] * Cs).sum(-1) + Ds * u
    by_group = (b, n, groups, -1, ns)
    return (gB * d + Ds * q, ddt, (m * d[..., None]).sum((0, 1)),
            (gs * (d * u)[..., None]).view(by_group).sum(3),
            (hs[:, 1:] * q[..., None]).view(by_group).sum(3), (q * u).sum((0, 1)),
            None if z is None else 1.1 * dy * y * (1 + z.abs() / 4), ddt.sum((0, 1)), g)


# ------------------------------------------------------------------------ norm


def norm(x, weight, bias, z, groups, kind, eps):
    v = x if z is None else x * silu(z)
    g = v.reshape(x.shape[0], groups, -1)
    if kind == "layer":
        g = g - g.mean(-1, keepdim=True)
    xh = g / torch.sqrt((g * g).mean(-1, keepdim=True) + eps)
    y = xh.reshape(x.shape) * weight
    return y if bias is None else y + bias


def norm_terms(x, z, groups, kind, eps):
    """(xh, its error's bound, 1 / standard deviation), [R, groups, D / groups].
    The statistics are sums of n float32 terms by a tree whose depth is at most
    n (n U of their size); the centred value carries the mean's error.  Each
    value of v is off by (2 |z| + 11) U with a gate."""
    v = x if z is None else x * silu(z)
    ev = 0 * v if z is None else (2 * z.abs() + 11) * U * v.abs()
    g = v.reshape(x.shape[0], groups, -1)
    eg = ev.reshape(g.shape)
    n = g.shape[-1]
    if kind == "layer":
        eg = eg + eg.mean(-1, keepdim=True) + (n + 2) * U * g.abs().mean(-1, keepdim=True)
        g = g - g.mean(-1, keepdim=True)
        eg = eg + U * g.abs()
    var = (g * g).mean(-1, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    # relative error of rstd: half of the variance's, and the root's own
    ervar = ((n + 3) * U * var + 2 * (g.abs() * eg).mean(-1, keepdim=True) +
             (eg * eg).mean(-1, keepdim=True)) * rstd * rstd
    er = 0.5 * ervar + 4 * U
    xh = g * rstd
    return xh, eg * rstd + (er + 2 * U) * xh.abs(), rstd, er


def norm_bound(x, weight, bias, z, groups, kind, eps, dtype):
    xh, e, _, _ = norm_terms(x, z, groups, kind, eps)
    y = norm(x, weight, bias, z, groups, kind, eps)
    err = e.reshape(x.shape) * weight.abs() + 2 * U * (xh.reshape(x.shape) * weight).abs()
    err = err + 2 * U * y.abs()
    return err + half_step(dtype) * (y.abs() + err)


# -------------------------------------------------------------------- gradients


def grads(fn, leaves, cotangents):
    """Gradients of sum(out * cotangent) with respect to the leaves (None stays None)."""
    ls = [None if v is None else v.clone().requires_grad_() for v in leaves]
    outs = fn(*ls)
    outs = outs if isinstance(outs, tuple) else (outs,)
    loss = sum((o * c).sum() for o, c in zip(outs, cotangents) if c is not None)
    live = [v for v in ls if v is not None]
    got = iter(torch.autograd.grad(loss, live, allow_unused=True))
    out = []
    for v in ls:
        if v is None:
            out.append(None)
        else:
            d = next(got)
            out.append(torch.zeros_like(v) if d is None else d)
    return out


def within(name, got, ref, bound):
    """Every element of got within bound of ref; reports the worst one."""
    got = got.detach().cpu().to(F)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), f"{name}: not finite"
    over = (got - ref).abs() - bound
    worst = int(over.argmax())
    assert over.max() <= 0, (f"{name}: element {worst} is {got.flatten()[worst]:.9g}, "
                             f"{ref.flatten()[worst]:.9g} wanted, off by more than "
                             f"{bound.expand_as(ref).flatten()[worst]:.3g}")
