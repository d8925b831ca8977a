"""The operators around the SSD together, as a layer uses them: convolution,
SSD or selective scan and norm in a run with their gradients, prompts carried
on token by token, padded batches, streams, graphs, long strides."""

import pytest
import torch

import layer_reference as ref
from gpu_helpers import TOL, say
from layer_reference import F, to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m2():
    import state_space_sequence_02_amd as lib
    return lib


def _gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return lambda *shape: torch.randn(shape, generator=g)


def _near(name, got, want, tol):
    got = got.detach().cpu().to(F)
    err = (got - want).abs().max() / want.abs().max()
    assert err <= tol, (name, float(err), tol)


# ------------------------------------------------- convolution, SSD, gated norm


def _ssd64(x, dt, A, B, C, D, h):
    """The SSD recurrence token by token: x [B,L,H,P], B and C [B,L,G,N]."""
    per = x.shape[2] // B.shape[2]
    ys = []
    for t in range(x.shape[1]):
        Bt, Ct = (v[:, t].repeat_interleave(per, 1) for v in (B, C))
        h = torch.exp(dt[:, t] * A)[..., None, None] * h + \
            (dt[:, t, :, None] * x[:, t])[..., None] * Bt[:, :, None]
        ys.append((h * Ct[:, :, None]).sum(-1) + D[:, None] * x[:, t])
    return torch.stack(ys, 1), h


def test_ssd_layer_and_its_gradients(m2):
    """proj -> conv1d (x, B, C in one call) -> ssd -> gated norm, float32, against
    the float64 layer and its autograd gradients, at the float32 bar of the SSD
    tests.  The projection's gradient is written in place by the operators."""
    b, n, H, P, N, G, W = 2, 70, 4, 16, 16, 2, 4
    inner, bc = H * P, G * N
    conv = inner + 2 * bc
    r = _gen(1)
    proj = r(b, n, inner + conv)          # z, then x B C
    wc, bias = r(conv, W) / 2, 0.1 * r(conv)
    dt, A, D = 0.1 * r(b, n, H).abs(), -r(H).abs() - 0.1, r(H)
    wn, dy = 1 + 0.1 * r(inner), r(b, n, inner)

    g = {k: v.cuda() for k, v in dict(proj=proj, wc=wc, bias=bias, dt=dt, A=A, D=D, wn=wn,
                                      dy=dy).items()}
    z, xbc = g["proj"][..., :inner], g["proj"][..., inner:]
    (x, B, C), _ = m2.conv1d_forward(xbc, g["wc"], g["bias"], parts=(inner, bc, bc))
    x, B, C = x.view(b, n, H, P), B.view(b, n, G, N), C.view(b, n, G, N)
    y, _ = m2.ssd_forward(x, g["dt"], g["A"], B, C, g["D"], None, chunk_size=64)
    out = m2.norm_forward(y.view(b, n, inner), g["wn"], None, z, ngroups=G)

    gn = m2.norm_backward(y.view(b, n, inner), g["wn"], None, z, g["dy"], ngroups=G)
    gs = m2.ssd_backward(x, g["dt"], g["A"], B, C, g["D"], None, gn["dx"].view(b, n, H, P),
                         chunk_size=64)
    dproj = torch.full_like(g["proj"], float("nan"))
    dproj[..., :inner] = gn["dz"]
    dims = m2.make_conv_dims(b, n, conv, W, (inner, bc, bc), torch.float32,
                             x_stride=inner + conv, dx_stride=inner + conv)
    size = m2.mamba2_conv1d_backward_workspace_bytes(dims)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    dwc, dbias = torch.empty_like(g["wc"]), torch.empty_like(g["bias"])
    m2.mamba2_conv1d_backward(dims, xbc, g["wc"], g["bias"], None, None, gs["dx"].flatten(2),
                              gs["dB"].flatten(2), gs["dC"].flatten(2), None,
                              dproj[..., inner:], dwc, dbias, None, ws, size)
    torch.cuda.synchronize()

    def layer(proj, wc, bias, dt, A, D, wn):
        v, _ = ref.conv(proj[..., inner:], wc, bias, None)
        x, B, C = v.split((inner, bc, bc), -1)
        y, _ = _ssd64(x.view(b, n, H, P), dt, A, B.view(b, n, G, N), C.view(b, n, G, N), D,
                      x.new_zeros(b, H, P, N))
        return ref.norm(y.reshape(b * n, inner), wn, None, proj[..., :inner].reshape(b * n, inner),
                        G, "rms", 1e-5).view(b, n, inner)

    leaves = [to64(v) for v in (proj, wc, bias, dt, A, D, wn)]
    _near("out", out, layer(*leaves), TOL["f32"])
    want = ref.grads(layer, leaves, (to64(dy),))
    for name, got, w in zip(("proj", "wc", "bias", "dt", "A", "D", "wn"),
                            (dproj, dwc, dbias, gs["ddt"], gs["dA"], gs["dD"], gn["dweight"]),
                            want):
        _near(name, got, w, TOL["f32"])


# --------------------------------------------- convolution, selective scan, norm


class ScanLayer:
    """x -> conv1d -> dt, B, C by projections -> selective scan with gate -> layer norm."""

    def __init__(self, seed, d=96, n=16, rank=8, dtype=torch.float32):
        r = _gen(seed)
        self.d, self.n, self.rank = d, n, rank
        c = lambda t: t.cuda()
        self.wc, self.bc = c(r(d, 4) / 2), c(0.1 * r(d))
        self.wx = c(r(d, rank + 2 * n) / d ** 0.5).to(dtype)
        self.wdt = c(r(rank, d) / rank ** 0.5).to(dtype)
        self.dt_bias = c(r(d) - 3)
        self.A = c(-torch.exp(0.5 * r(d, n)))
        self.D = c(r(d))
        self.wn, self.bn = c(1 + 0.1 * r(d)), c(0.1 * r(d))

    def _split(self, u):
        # 8 columns of rank, then B and C: column ranges of the projection's rows
        p = u @ self.wx
        k = self.rank
        return ((p[..., :k] @ self.wdt).contiguous(), p[..., k:k + self.n].unsqueeze(-2),
                p[..., k + self.n:].unsqueeze(-2))

    def prompt(self, m2, x, z, conv_state=None, state=None, lengths=None):
        u, conv_state = m2.conv1d_forward(x, self.wc, self.bc, conv_state, lengths=lengths)
        dt, B, C = self._split(u)
        y, state = m2.selective_scan_forward(u, dt, self.A, B, C, self.D, z, self.dt_bias, state,
                                             lengths=lengths)
        return m2.norm_forward(y, self.wn, self.bn, kind="layer"), conv_state, state

    def step(self, m2, x, z, conv_state, state):
        u = m2.conv1d_step(x, self.wc, self.bc, conv_state)
        dt, B, C = self._split(u)
        B, C = B.clone(), C.clone()  # the step's base pointers: 16-byte aligned
        y = m2.selective_scan_step(u, dt, self.A, B, C, self.D, z, self.dt_bias, state)
        return m2.norm_forward(y, self.wn, self.bn, kind="layer")


@pytest.mark.parametrize("dtype,tol", [(torch.float32, TOL["f32"]), (torch.bfloat16, TOL["bf16"])])
def test_prompt_then_steps_is_the_longer_prompt(m2, dtype, tol):
    layer = ScanLayer(3, dtype=dtype)
    r = _gen(4)
    x, z = (r(3, 190, layer.d).to(dtype).cuda() for _ in range(2))
    whole, wc, ws = layer.prompt(m2, x, z)
    first, cs, st = layer.prompt(m2, x[:, :180].contiguous(), z[:, :180].contiguous())
    outs = [first]
    for t in range(180, 185):
        outs.append(layer.step(m2, x[:, t].contiguous(), z[:, t].contiguous(), cs, st)[:, None])
    # and a second prompt carried on from the steps' states
    rest, cs, st = layer.prompt(m2, x[:, 185:].contiguous(), z[:, 185:].contiguous(), cs, st)
    got = torch.cat(outs + [rest], 1)
    _near("outputs", got, to64(whole), tol)
    assert torch.equal(cs, wc)
    _near("state", st, to64(ws), tol)


def test_padded_batch_is_its_sequences(m2):
    """A padded batch (one sequence empty) gives each sequence's own outputs and
    states, zeros behind them, and carries on from those states; what stands in
    the padding does not matter."""
    layer = ScanLayer(5)
    r = _gen(6)
    n, lens = 150, [150, 0, 3, 77]
    x, z = r(4, n, layer.d).cuda(), r(4, n, layer.d).cuda()
    lengths = torch.tensor(lens, dtype=torch.int32).cuda()
    for fill in (float("nan"), float("inf"), 0.0):
        px, pz = x.clone(), z.clone()
        for i, m in enumerate(lens):
            px[i, m:] = fill
            pz[i, m:] = fill
        cs0, st0 = r(4, 3, layer.d).cuda(), r(4, layer.d, layer.n).cuda()
        u, cs = m2.conv1d_forward(px, layer.wc, layer.bc, cs0, lengths=lengths)
        dt, B, C = layer._split(u)
        y, st = m2.selective_scan_forward(u, dt, layer.A, B, C, layer.D, pz, layer.dt_bias, st0,
                                          lengths=lengths)
        for i, m in enumerate(lens):
            assert (u[i, m:] == 0).all() and (y[i, m:] == 0).all()
            if m == 0:
                assert torch.equal(cs[i], cs0[i]) and torch.equal(st[i], st0[i])
                continue
            ui, ci = m2.conv1d_forward(x[i:i + 1, :m], layer.wc, layer.bc, cs0[i:i + 1].clone())
            assert torch.equal(ui[0], u[i, :m]) and torch.equal(ci[0], cs[i])
            yi, si = m2.selective_scan_forward(
                u[i:i + 1, :m].contiguous(), dt[i:i + 1, :m].contiguous(), layer.A,
                B[i:i + 1, :m].clone(), C[i:i + 1, :m].clone(), layer.D,
                z[i:i + 1, :m].contiguous(), layer.dt_bias, st0[i:i + 1].clone())
            _near("y", y[i, :m], to64(yi[0]), TOL["f32"])
            _near("state", st[i], to64(si[0]), TOL["f32"])


def test_ssd_decode_from_convolution_step(m2):
    """conv1d_step's parts are what decode_step takes."""
    b, H, P, N, G = 3, 4, 32, 64, 2
    inner, bc = H * P, G * N
    r = _gen(7)
    io = torch.bfloat16
    xs = r(b, 6, inner + 2 * bc).to(io).cuda()
    w, bias = (r(inner + 2 * bc, 4) / 2).cuda(), r(inner + 2 * bc).cuda()
    dt = (0.1 * r(b, 6, H).abs()).to(io).cuda()
    A, D = -r(H).abs().cuda(), r(H).cuda()
    (x, B, C), _ = m2.conv1d_forward(xs, w, bias, parts=(inner, bc, bc))
    y, fin = m2.ssd_forward(x.view(b, 6, H, P), dt, A, B.view(b, 6, G, N), C.view(b, 6, G, N), D,
                            None, chunk_size=64)
    cs = torch.zeros(b, 3, inner + 2 * bc, dtype=io, device="cuda")
    st = torch.zeros(b, H, P, N, device="cuda")
    for t in range(6):
        x1, B1, C1 = m2.conv1d_step(xs[:, t], w, bias, cs, parts=(inner, bc, bc))
        y1 = m2.decode_step(x1.view(b, H, P), dt[:, t].clone(), A, B1.view(b, G, N),
                            C1.view(b, G, N), D, st, chunk_size=64)
        _near("y", y1, to64(y[:, t]), TOL["bf16"])
    _near("state", st, to64(fin), TOL["bf16"])


# -------------------------------------------------- gradients against differences


def test_gradients_are_differences(m2):
    """The operators' float32 gradients along random directions against central
    differences of the float64 forms (step 1e-5: their own error is of the
    order of 1e-10 relative; the float32 sums' 1e-4 is the SSD tests' bar)."""
    r = _gen(9)
    b, n, ch, ns = 2, 40, 32, 5
    wt, bias, h0 = r(ch, 4), r(ch), r(b, 3, ch)
    x, dyc, dfc = r(b, n, ch), r(b, n, ch), r(b, 3, ch)
    scan = [ref.silu(r(b, n, ch)), 0.5 * r(b, n, ch), -r(ch, ns).abs() - 0.1, r(b, n, 1, ns),
            r(b, n, 1, ns), r(ch), r(b, n, ch), r(ch) - 2, r(b, ch, ns)]
    dfs = r(b, ch, ns)
    nx, nw, nb, nz = r(n, ch), r(ch), r(ch), r(n, ch)
    c = lambda ts: [t.cuda() for t in ts]
    gc = m2.conv1d_backward(*c((x, wt, bias, h0)), dyc.cuda(), dfc.cuda())
    gs = m2.selective_scan_backward(*c(scan), dyc.cuda(), dfs.cuda())
    gn = m2.norm_backward(*c((nx, nw, nb, nz)), dyc[0].contiguous().cuda(), kind="layer", ngroups=4)

    def along(fn, leaves, cots, grads):
        leaves = [to64(v) for v in leaves]
        loss = lambda ls: sum((o * to64(k)).sum() for o, k in zip(fn(*ls), cots))
        for i, g in enumerate(grads):
            v = r(*leaves[i].shape).to(F)
            up, down = ([l + s * v if k == i else l for k, l in enumerate(leaves)]
                        for s in (1e-5, -1e-5))
            diff = (loss(up) - loss(down)) / 2e-5
            got = (g.cpu().to(F) * v).sum()
            size = (g.cpu().to(F) * v).abs().sum()
            assert abs(got - diff) <= TOL["f32"] * size, (i, float(got), float(diff))

    along(lambda *a: ref.conv(*a), (x, wt, bias, h0), (dyc, dfc),
          [gc[k] for k in ("dx", "dweight", "dbias", "dinit")])
    along(lambda *a: ref.scan(*a), scan, (dyc, dfs),
          [gs[k] for k in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinit")])
    along(lambda x, w, bb, z: (ref.norm(x, w, bb, z, 4, "layer", 1e-5),), (nx, nw, nb, nz),
          (dyc[0],), [gn[k] for k in ("dx", "dweight", "dbias", "dz")])


# -------------------------------------------------------------- calls and their order


def _everything(m2, seed, dtype=torch.bfloat16):
    """Inputs of one call of every operator, and a function that makes the calls."""
    layer = ScanLayer(seed, d=128, dtype=dtype)
    r = _gen(seed + 100)
    b, n = 2, 333
    t = {k: r(b, n, layer.d).to(dtype).cuda() for k in ("x", "z", "dy")}
    t["cs"] = r(b, 3, layer.d).to(dtype).cuda()
    t["st"] = r(b, layer.d, layer.n).cuda()
    t["lens"] = torch.tensor([n, 200], dtype=torch.int32).cuda()
    t["B"], t["C"] = (r(b, n, 2, layer.n).to(dtype).cuda() for _ in range(2))
    t["dt"] = r(b, n, layer.d).to(dtype).cuda()
    one = {k: t[k][:, 0].clone() for k in ("x", "z", "dt", "B", "C")}

    def calls(**kw):
        L = layer
        out = []
        u, cs = m2.conv1d_forward(t["x"], L.wc, L.bc, t["cs"], lengths=t["lens"], **kw)
        y, st = m2.selective_scan_forward(u, t["dt"], L.A, t["B"], t["C"], L.D, t["z"], L.dt_bias,
                                          t["st"], lengths=t["lens"], **kw)
        o = m2.norm_forward(y, L.wn, L.bn, t["z"], ngroups=2, kind="layer", **kw)
        gn = m2.norm_backward(y, L.wn, L.bn, t["z"], t["dy"], ngroups=2, kind="layer", **kw)
        gs = m2.selective_scan_backward(u, t["dt"], L.A, t["B"], t["C"], L.D, t["z"], L.dt_bias,
                                        t["st"], gn["dx"], st, lengths=t["lens"], **kw)
        gc = m2.conv1d_backward(t["x"], L.wc, L.bc, t["cs"], gs["du"], cs, lengths=t["lens"], **kw)
        c1 = m2.conv1d_step(one["x"], L.wc, L.bc, cs, **kw)
        s1 = m2.selective_scan_step(c1, one["dt"], L.A, one["B"], one["C"], L.D, one["z"],
                                    L.dt_bias, st, **kw)
        out += [u, cs, y, st, o, c1, s1]
        for g in (gn, gs, gc):
            out += list(g.values())
        return out

    return t, calls


def test_same_call_same_bits(m2):
    _, calls = _everything(m2, 20)
    first = calls()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, calls()))


def test_other_streams(m2):
    """A call on another stream (given, or the current one), two calls at once on
    two streams: the same bits."""
    _, calls = _everything(m2, 21)
    _, other = _everything(m2, 22)
    want, wother = calls(), other()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        got1 = calls(stream=s1)
        with torch.cuda.stream(s2):
            got2 = other()
        got3 = calls(stream=s2.cuda_stream)
        torch.cuda.synchronize()
        with torch.cuda.stream(s2):
            got4 = calls(stream=0)  # the default stream, from another current one
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(want, got4))
        assert all(torch.equal(p, q) for p, q in zip(want, got1))
        assert all(torch.equal(p, q) for p, q in zip(wother, got2))
        assert all(torch.equal(p, q) for p, q in zip(want, got3))


def test_captured_and_replayed(m2):
    """Every operator captured into a graph, two graphs side by side, replayed on
    new inputs with eager work between: each replay is the eager result."""
    runs = [_everything(m2, s) for s in (23, 24)]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for t, calls in runs:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            calls()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(calls())
        graphs.append(g)
    r = _gen(25)
    for i in range(4):
        for t, _ in runs:
            for k in ("x", "z", "dy", "dt", "B", "C"):
                t[k].copy_(r(*t[k].shape).to(t[k].dtype))
        eager = [calls() for _, calls in runs]
        order = (0, 1) if i % 2 else (1, 0)
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        for got, want in zip(outs, eager):
            assert all(torch.equal(p, q) for p, q in zip(got, want)), i


# --------------------------------------------------------- offsets beyond 32 bits


def test_rows_far_apart(m2):
    """Column ranges of very wide rows: the last rows lie beyond 2^31 elements."""
    n, wide, c = 20000, 1 << 17, 64
    say("rows far apart")
    rows = torch.empty(n, wide, dtype=torch.bfloat16, device="cuda")
    assert rows.numel() > 1 << 31
    r = _gen(30)
    near = r(1, n, c).to(torch.bfloat16).cuda()
    far = rows[:, 8:8 + c].unsqueeze(0)
    far.copy_(near)
    w = r(c, 4).cuda()
    a, fa = m2.conv1d_forward(near, w)
    b, fb = m2.conv1d_forward(far, w)
    assert torch.equal(a, b) and torch.equal(fa, fb)
    ga, gb = (m2.conv1d_backward(v, w, None, None, a) for v in (near, far))
    assert torch.equal(ga["dx"], gb["dx"]) and torch.equal(ga["dweight"], gb["dweight"])
    wn = r(c).cuda()
    assert torch.equal(m2.norm_forward(near, wn, None, near), m2.norm_forward(far, wn, None, far))
    ga, gb = (m2.norm_backward(v, wn, None, v, a) for v in (near, far))
    assert torch.equal(ga["dx"], gb["dx"]) and torch.equal(ga["dz"], gb["dz"])
    A = -torch.ones(c, 16, device="cuda")
    Bn, Bf = (v[..., :16].unsqueeze(-2) for v in (near.clone(), far))
    Bn = Bn.contiguous()
    (ya, sa), (yb, sb) = (m2.selective_scan_forward(near, near, A, B, B, None, z)
                          for B, z in ((Bn, near), (Bf, far)))
    assert torch.equal(ya, yb) and torch.equal(sa, sb)
    ga, gb = (m2.selective_scan_backward(near, near, A, B, B, None, z, None, None, a)
              for B, z in ((Bn, near), (Bf, far)))
    assert all(torch.equal(ga[k], gb[k]) for k in ("du", "ddt", "dA", "dB", "dC", "dz"))


def test_long_sequence_of_many_channels(m2):
    """More than 2^31 elements of u: decays of at least e^-0.3 a token leave nothing of
    what lies 512 tokens back, so the last tokens are those of a short call."""
    n, ch, ns = (1 << 20) + 37, 2080, 4
    say("long sequence")
    g = torch.Generator(device="cuda")
    g.manual_seed(31)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.bfloat16)
    u, dt = rn(1, n, ch), rn(1, n, ch)
    assert u.numel() > 1 << 31
    B, C = rn(1, n, 1, ns), rn(1, n, 1, ns)
    A = -torch.ones(ch, ns, device="cuda")
    bias = torch.full((ch,), 2.5, device="cuda")
    y, fin = m2.selective_scan_forward(u, dt, A, B, C, None, None, bias)
    k = 600
    tail = [v[:, -k:].clone() for v in (u, dt, B, C)]  # a view may start off 16 bytes
    ys, fs = m2.selective_scan_forward(tail[0], tail[1], A, tail[2], tail[3], None, None, bias)
    _near("final", fin, to64(fs), TOL["f32"])
    _near("y", y[:, -64:], to64(ys[:, -64:]), TOL["bf16"])
    del y
    w = torch.ones(ch, 4, device="cuda")
    c, cf = m2.conv1d_forward(u, w)
    cs, csf = m2.conv1d_forward(tail[0], w)
    assert torch.equal(c[:, -64:], cs[:, -64:]) and torch.equal(cf, csf)
    gl = m2.conv1d_backward(u, w, None, None, c)
    gt = m2.conv1d_backward(tail[0], w, None, None, cs)
    assert torch.equal(gl["dx"][:, -64:], gt["dx"][:, -64:])
