"""The feed-forward and residual-norm operators on the GPU against their
64-bit definitions, elementwise, with bounds from the arithmetic (ffn_testlib)."""
import pytest

import mot_dit_b200 as W

torch = pytest.importorskip("torch")
import ffn_testlib as T  # noqa: E402

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
CODE = {BF: W.BF16, FP: W.FP32}
ACT = {n: i for i, n in enumerate(W.ACTS)}


def _ws(nbytes):
    return torch.full((max(nbytes, 1),), 255, dtype=torch.uint8, device="cuda") if nbytes else None  # (NaN patterns)


@pytest.fixture(autouse=True)
def _no_timeout():
    yield
    W.ops_check_status()


# rows: one token, a few, ragged tiles, several row tiles; features and
# reductions that no tile or vector divides; long reductions with few tiles
# (cluster split), many tiles (CTA pairs).
LINEAR = [
    # M, N, K, act, type, out, residual, save z
    (1, 1, 1, "none", BF, BF, False, False),
    (1, 64, 64, "silu", BF, FP, True, True),
    (1, 1000, 1536, "gelu_tanh", BF, BF, False, False),
    (3, 77, 130, "gelu_erf", BF, BF, True, True),
    (16, 384, 6144, "none", BF, FP, True, False),
    (17, 40, 72, "relu", BF, BF, True, True),
    (129, 200, 328, "sigmoid", BF, FP, True, True),
    (130, 4111, 200, "gelu_tanh", BF, BF, True, True),
    (200, 264, 511, "silu", BF, BF, False, True),
    (1088, 1536, 768, "none", BF, FP, True, False),
    (2100, 2049, 136, "gelu_tanh", BF, BF, True, False),
    (2560, 2560, 256, "silu", BF, BF, False, True),
    (1, 33, 65, "gelu_tanh", FP, FP, True, True),
    (70, 129, 1030, "silu", FP, FP, True, False),
    (260, 516, 96, "gelu_erf", FP, FP, False, True),
    (1500, 2000, 70, "relu", FP, FP, True, True),
]


@pytest.mark.parametrize("M,N,K,act,t,o,res,save", LINEAR)
def test_linear(M, N, K, act, t, o, res, save):
    n = T.normals(M + N + K)
    x, w, b = n(M, K, dtype=t), n(N, K, std=K ** -0.5, dtype=t), n(N, std=0.3)
    r = n(M, N, dtype=o) if res else None
    (y, oky), (z, okz) = T.guarded((M, N), o), T.guarded((M, N), t)
    W.op_linear_act(CODE[t], x, w, b, y, M, N, K, act=ACT[act], residual=r, z=z if save else None, out_dtype=CODE[o])
    z64, ez, y64, ey = T.linear64(x, w, b, r, act, o)
    T.within(y, y64, ey)
    oky()
    if save:
        T.within(z, z64, ez)
        okz()
    y2 = torch.empty_like(y)
    W.op_linear_act(CODE[t], x, w, b, y2, M, N, K, act=ACT[act], residual=r, out_dtype=CODE[o])
    assert torch.equal(y, y2)  # the same bits, with or without z
    if res:  # in place on the residual
        W.op_linear_act(CODE[t], x, w, b, r, M, N, K, act=ACT[act], residual=r, out_dtype=CODE[o])
        assert torch.equal(r, y2)


@pytest.mark.parametrize("t", [BF, FP])
@pytest.mark.parametrize("sx,sw,sy", [(1, 0, 0), (0, 3, 0), (0, 0, 1), (1, 1, 1)])
def test_linear_unaligned(t, sx, sw, sy):
    """Operands and outputs that start off a 16-byte boundary."""
    M, N, K = 150, 136, 200
    n = T.normals(sx * 100 + sw * 10 + sy)
    put = lambda v, s: torch.cat([torch.zeros(s, dtype=v.dtype, device="cuda"), v.flatten()])[s:].view(v.shape)  # noqa: E731
    x, w = put(n(M, K, dtype=t), sx), put(n(N, K, std=K ** -0.5, dtype=t), sw)
    b, r = put(n(N), sy), put(n(M, N, dtype=t), sy)
    (y, oky), (z, okz) = T.guarded((M, N), t, sy), T.guarded((M, N), t, sy)
    W.op_linear_act(CODE[t], x, w, b, y, M, N, K, act=ACT["silu"], residual=r, z=z)
    z64, ez, y64, ey = T.linear64(x, w, b, r, "silu", t)
    T.within(y, y64, ey)
    T.within(z, z64, ez)
    oky(), okz()


LINEAR_BWD = [
    (1, 1, 1, "silu", BF, BF),
    (1, 65, 64, "none", BF, BF),
    (33, 64, 64, "none", BF, BF),
    (33, 64, 64, "none", BF, FP),
    (100, 71, 200, "gelu_tanh", BF, FP),
    (257, 4111, 264, "gelu_tanh", BF, BF),
    (1000, 129, 67, "gelu_erf", BF, BF),
    (8448, 64, 72, "silu", BF, BF),
    (64, 72, 3000, "sigmoid", BF, FP),
    (2049, 1544, 1100, "relu", BF, BF),
    (40, 33, 65, "silu", FP, FP),
    (2048, 36, 40, "none", FP, FP),
    (300, 777, 321, "gelu_tanh", FP, FP),
]


@pytest.mark.parametrize("M,N,K,act,t,o", LINEAR_BWD)
def test_linear_backward(M, N, K, act, t, o):
    n = T.normals(M + 3 * N + K)
    x, w, dy = n(M, K, dtype=t), n(N, K, std=K ** -0.5, dtype=t), n(M, N, dtype=o)
    z = n(M, N, dtype=t, std=1.5) if act != "none" else None
    (dx, ok1), (dw, ok2), (db, ok3) = T.guarded((M, K), t), T.guarded((N, K), t), T.guarded((N,), FP)
    need = W.op_linear_act_workspace(CODE[t], M, N, K, act=ACT[act], dy_dtype=CODE[o])
    call = lambda a, b, c: W.op_linear_act_backward(CODE[t], x, w, z, dy, a, b, c, M, N, K, act=ACT[act],  # noqa: E731
                                                    dy_dtype=CODE[o], workspace=_ws(need))
    call(dx, dw, db)
    (dx64, ex), [((dw64, ew), (db64, eb))] = T.linear_grad64(x, w, z, dy, act)
    T.within(dx, dx64, ex)
    T.within(dw, dw64, ew)
    T.within(db, db64, eb)
    ok1(), ok2(), ok3()
    # each gradient alone, within the same bounds
    a, b, c = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    call(a, None, None), call(None, b, None), call(None, None, c)
    T.within(a, dx64, ex), T.within(b, dw64, ew)
    assert torch.equal(c, db)


GATED = [
    (1, 1, 1, "silu", BF, True, True),
    (1, 64, 64, "silu", BF, False, False),
    (1, 1000, 1536, "gelu_tanh", BF, True, False),
    (5, 33, 71, "sigmoid", BF, True, True),
    (140, 100, 200, "relu", BF, False, True),
    (129, 777, 136, "gelu_erf", BF, True, True),
    (1088, 1536, 256, "silu", BF, True, True),
    (2600, 2200, 128, "gelu_tanh", BF, False, False),
    (64, 40, 4096, "silu", BF, True, True),
    (150, 130, 201, "none", BF, True, True),
    (3, 20, 33, "silu", FP, True, True),
    (130, 300, 200, "gelu_erf", FP, False, True),
    (1000, 1100, 60, "gelu_tanh", FP, True, False),
]


@pytest.mark.parametrize("M,F,K,act,t,bias,save", GATED)
def test_gated(M, F, K, act, t, bias, save):
    n = T.normals(M + F + K)
    x, wg, wu = n(M, K, dtype=t), n(F, K, std=K ** -0.5, dtype=t), n(F, K, std=K ** -0.5, dtype=t)
    bg, bu = (n(F, std=0.3), n(F, std=0.3)) if bias else (None, None)
    (a, ok1), (g, ok2), (u, ok3) = (T.guarded((M, F), t) for _ in range(3))
    kw = dict(act=ACT[act], bias_g=bg, bias_u=bu)
    W.op_gated(CODE[t], x, wg, wu, a, M, F, K, g=g if save else None, u=u if save else None, **kw)
    (a64, ea), (g64, eg), (u64, eu) = T.gated64(x, wg, wu, bg, bu, act)
    T.within(a, a64, ea)
    ok1()
    if save:
        T.within(g, g64, eg), T.within(u, u64, eu)
        ok2(), ok3()
    a2 = torch.empty_like(a)
    W.op_gated(CODE[t], x, wg, wu, a2, M, F, K, **kw)
    assert torch.equal(a, a2)


GATED_BWD = [
    (1, 1, 1, "silu", BF, True),
    (33, 64, 64, "silu", BF, True),
    (100, 71, 200, "gelu_tanh", BF, False),
    (300, 333, 67, "gelu_erf", BF, True),
    (2112, 1024, 768, "silu", BF, True),
    (8448, 40, 64, "sigmoid", BF, True),
    (50, 2000, 72, "relu", BF, True),
    (264, 777, 321, "silu", FP, True),
    (20, 33, 65, "gelu_tanh", FP, False),
]


@pytest.mark.parametrize("M,F,K,act,t,bias", GATED_BWD)
def test_gated_backward(M, F, K, act, t, bias):
    n = T.normals(M + 3 * F + K)
    x, wg, wu = n(M, K, dtype=t), n(F, K, std=K ** -0.5, dtype=t), n(F, K, std=K ** -0.5, dtype=t)
    g, u, da = n(M, F, dtype=t, std=1.5), n(M, F, dtype=t), n(M, F, dtype=t)
    outs = [T.guarded(s, d) for s, d in (((M, K), t), ((F, K), t), ((F, K), t), ((F,), FP), ((F,), FP))]
    dx, dwg, dwu, dbg, dbu = (o[0] for o in outs)
    ws = _ws(W.op_gated_workspace(CODE[t], M, F, K))
    call = lambda a, b, c, d, e: W.op_gated_backward(CODE[t], x, wg, wu, g, u, da, a, b, c, M, F, K, act=ACT[act],  # noqa: E731
                                                     dbias_g=d, dbias_u=e, workspace=ws)
    call(dx, dwg, dwu, dbg if bias else None, dbu if bias else None)
    (dx64, ex), [((g64, eg), (bg64, ebg)), ((u64, eu), (bu64, ebu))] = T.gated_grad64(x, wg, wu, g, u, da, act)
    T.within(dx, dx64, ex), T.within(dwg, g64, eg), T.within(dwu, u64, eu)
    if bias:
        T.within(dbg, bg64, ebg), T.within(dbu, bu64, ebu)
        c, d = torch.empty_like(dbg), torch.empty_like(dbu)
        call(None, None, None, c, d)
        assert torch.equal(c, dbg) and torch.equal(d, dbu)
    for _, ok in outs:
        ok()
    a, b, c = torch.empty_like(dx), torch.empty_like(dwg), torch.empty_like(dwu)
    call(a, None, None, None, None), call(None, b, c, None, None)
    T.within(a, dx64, ex), T.within(b, g64, eg), T.within(c, u64, eu)


NORM = [
    # M, per, D, types (stream, compute), post, gate, mod, gain, alpha
    (1, 0, 1, FP, BF, True, True, True, True, 1.0),
    (1, 0, 768, FP, BF, True, True, True, True, 1.0),
    (5, 0, 3, FP, BF, True, False, False, False, 1.0),
    (37, 10, 33, BF, BF, True, True, True, True, 0.5),
    (100, 34, 64, FP, BF, False, True, True, False, 1.0),
    (300, 1, 264, FP, BF, True, True, True, True, 1.0),
    (700, 100, 1536, FP, BF, True, True, True, False, 1.0),
    (333, 0, 1537, BF, BF, True, True, True, True, -1.25),
    (90, 30, 520, BF, BF, False, False, False, False, 1.0),
    (61, 0, 4096, FP, BF, True, True, False, True, 1.0),
    (40, 20, 8192, FP, BF, True, True, True, True, 1.0),
    (23, 8, 5003, BF, BF, True, True, True, True, 1.0),
    (50, 25, 100, FP, FP, True, True, True, True, 1.0),
    (65, 0, 2049, FP, FP, False, True, True, True, 1.0),
]


def _norm_case(M, per, D, r, t, post, gate, mod, gain):
    n = T.normals(M + D)
    p = per or M
    G = -(-M // p)
    table = n(G, 3, D, std=0.5)
    v = dict(post_gain=n(D, std=0.2, mean=1.0) if post else None, gate=table[:, 0] if gate else None,
             gain=n(D, std=0.2, mean=1.0) if gain else None, scale=table[:, 1] if mod else None,
             shift=table[:, 2] if mod else None)
    return n, p, G, n(M, D, std=2.0, dtype=r), n(M, D, std=0.7, dtype=t), v


def _d(v):
    return {k: None if x is None else x.double() for k, x in v.items()}


@pytest.mark.parametrize("M,per,D,r,t,post,gate,mod,gain,alpha", NORM)
def test_residual_norm(M, per, D, r, t, post, gate, mod, gain, alpha):
    n, p, G, x, y, v = _norm_case(M, per, D, r, t, post, gate, mod, gain)
    (s, ok1), (h, ok2) = T.guarded((M, D), r), T.guarded((M, D), t)
    kw = dict(post_norm=post, alpha=alpha, rows_per_group=per, ld_mod=3 * D, res_dtype=CODE[r], **v)
    W.op_residual_norm(CODE[t], x, y, s, h, M, D, **kw)
    s64, h64 = T.norm64(x.double(), y.double(), post, alpha=alpha, per=p, **_d(v))
    # p carries the statistic's error: D + 8 additions and roundings; s two more
    rel = (D + 16) * 2.0 ** -24
    part = (s64 - alpha * x.double()).abs()
    es = rel * part + 2.0 ** -22 * (s64.abs() + (alpha * x.double()).abs())
    T.within(s, s64, es + T.H[r] * (s64.abs() + es))
    # h = s r m + b: r's error is that of the mean of s^2, which the errors of s shift by their own share
    rms = (s64 * s64).mean(1, keepdim=True).add(T.EPS).sqrt()
    mul = torch.ones(M, D, device="cuda", dtype=torch.float64)
    if gain:
        mul = mul * v["gain"].double()
    if mod:
        mul = mul * (1 + T.spread(v["scale"], M, p))
    shift = es.norm(dim=1, keepdim=True) / (D ** 0.5 * rms)
    eh = mul.abs() / rms * (es + s64.abs() * (rel + 2 * shift)) + 2.0 ** -21 * (h64.abs() + (s64 / rms * mul).abs())
    T.within(h, h64, eh + T.H[t] * (h64.abs() + eh))
    ok1(), ok2()
    s2, h2 = x.clone(), y.clone()  # in place
    W.op_residual_norm(CODE[t], s2, h2, s2, h2, M, D, **kw)
    assert torch.equal(s2, s) and torch.equal(h2, h)


@pytest.mark.parametrize("M,per,D,r,t,post,gate,mod,gain,alpha", NORM)
def test_residual_norm_backward(M, per, D, r, t, post, gate, mod, gain, alpha):
    n, p, G, s, y, v = _norm_case(M, per, D, r, t, post, gate, mod, gain)
    dh, ds = n(M, D, dtype=t), n(M, D, dtype=r)
    outs = {"dx": T.guarded((M, D), r), "dy": T.guarded((M, D), t)}
    for k, x in v.items():
        if x is not None:
            outs["d" + k] = T.guarded(tuple(x.shape), FP)
    kw = dict(post_norm=post, alpha=alpha, rows_per_group=per, ld_mod=3 * D, res_dtype=CODE[r],
              **{k: x for k, x in v.items() if k != "shift"})
    ws = _ws(W.op_residual_norm_workspace(M, D, per))
    W.op_residual_norm_backward(CODE[t], s, y, ds, dh, outs["dx"][0], outs["dy"][0], M, D, workspace=ws, **kw,
                                **{k: o[0] for k, o in outs.items() if k not in ("dx", "dy")})
    # the definition's gradient at the point whose stream value is s
    vd = {k: None if x is None else x.double().requires_grad_() for k, x in v.items()}
    yd = y.double().requires_grad_()
    with torch.no_grad():
        s0, _ = T.norm64(torch.zeros_like(s).double(), yd, post, alpha=alpha, per=p, **vd)
    xd = ((s.double() - s0) / alpha).requires_grad_()
    s64, h64 = T.norm64(xd, yd, post, alpha=alpha, per=p, **vd)
    names = [k for k in vd if vd[k] is not None]
    got = torch.autograd.grad([s64, h64], [xd, yd] + [vd[k] for k in names], [ds.double(), dh.double()])
    want = dict(zip(["dx", "dy"] + ["d" + k for k in names], got))
    # Error bound: every factor of dv, dy and the column terms carries at most rel; the sums over a row and
    # the expansion of mean(dp post_gain q) are bounded with absolute values throughout.
    rel = (D + 32) * 2.0 ** -23
    one = torch.ones(M, D, device="cuda", dtype=torch.float64)
    rows = lambda x: one if x is None else T.spread(x, M, p)  # noqa: E731
    vec = lambda x: one if x is None else one * x.double()  # noqa: E731
    with torch.no_grad():
        S, Y, DH, DS = s.double().abs(), y.double().abs(), dh.double().abs(), ds.double().abs()
        mul = (vec(v["gain"]) * (1 + T.spread(v["scale"], M, p)) if mod else vec(v["gain"])).abs()
        w = (rows(v["gate"]) * vec(v["post_gain"])).abs()
        r_ = 1 / ((S * S).mean(1, keepdim=True) + T.EPS).sqrt()
        ry = 1 / ((Y * Y).mean(1, keepdim=True) + T.EPS).sqrt() if post else one[:, :1]
        mag = lambda a, b: (a * b).mean(1, keepdim=True)  # noqa: E731
        c = r_ ** 3 * mag(DH * mul, S)
        dv = DS + r_ * DH * mul + S * c
        dy = ry * (dv * w + Y * ry ** 2 * mag(dv * w, Y)) if post else dv * w
        q = Y * ry
        cols = {"dx": abs(alpha) * dv, "dy": dy}
        grp = lambda a: torch.stack([a[i * p:(i + 1) * p].sum(0) for i in range(G)])  # noqa: E731
        cols["dgate"] = grp(dv * q * vec(v["post_gain"]).abs())
        cols["dpost_gain"] = (dv * q * rows(v["gate"]).abs()).sum(0)
        cols["dscale"] = grp(DH * S * r_ * vec(v["gain"]).abs())
        cols["dshift"] = grp(DH)
        cols["dgain"] = (DH * S * r_ * ((1 + rows(v["scale"])).abs() if mod else 1)).sum(0)
    for k, (o, ok) in outs.items():
        row = k in ("dx", "dy")
        e = (rel + (0 if row else M * 2.0 ** -24)) * cols[k]
        T.within(o, want[k].reshape(o.shape), e + T.H[o.dtype] * (want[k].reshape(o.shape).abs() + e))
        ok()
    # in place on the gradients, without the parameter gradients: the same bits
    a, b = ds.clone(), dh.clone()
    W.op_residual_norm_backward(CODE[t], s, y, a, b, a, b, M, D, **kw)
    assert torch.equal(a, outs["dx"][0]) and torch.equal(b, outs["dy"][0])
    # no gradient from the stream
    a, b, zero = torch.empty_like(ds), torch.empty_like(dh), torch.zeros_like(ds)
    a2, b2 = torch.empty_like(ds), torch.empty_like(dh)
    W.op_residual_norm_backward(CODE[t], s, y, None, dh, a, b, M, D, **kw)
    W.op_residual_norm_backward(CODE[t], s, y, zero, dh, a2, b2, M, D, **kw)
    assert torch.equal(a, a2) and torch.equal(b, b2)


@pytest.mark.parametrize("r,t", [(FP, BF), (BF, BF), (FP, FP)])
@pytest.mark.parametrize("scale", [1e-8, 1.0, 1e13, 1e15, 1e17])
@pytest.mark.parametrize("D", [96, 4100])
def test_residual_norm_backward_of_any_magnitude(D, scale, r, t):
    """A stream of large or small rows, and no gradient from it: dx = r (dn - n mean(dn n)) alone."""
    M = 33
    n = T.normals(D)
    s, y, dh, gain = n(M, D, std=scale, dtype=r), n(M, D, dtype=t), n(M, D, dtype=t), n(D, mean=1.0)
    (dx, ok1), (dy, ok2) = T.guarded((M, D), r), T.guarded((M, D), t)
    W.op_residual_norm_backward(CODE[t], s, y, None, dh, dx, dy, M, D, gain=gain, res_dtype=CODE[r])
    S, dn = s.double(), dh.double() * gain.double()
    rs = 1 / ((S * S).mean(1, keepdim=True) + T.EPS).sqrt()
    want = rs * dn - S * rs ** 3 * (dn * S).mean(1, keepdim=True)
    # the statistic and the mean: D additions and a few roundings of either term
    e = (D + 32) * 2.0 ** -23 * (rs * dn.abs() + S.abs() * rs ** 3 * (dn * S).abs().mean(1, keepdim=True))
    T.within(dx, want, e + T.H[r] * (want.abs() + e))
    T.within(dy, want, e + T.H[t] * (want.abs() + e))
    ok1(), ok2()
    # the same of the post-norm: dy = r_y (dv - q mean(dv q)), q = y r_y, from a stream of ordinary size
    s, y, ds = n(M, D, dtype=r), n(M, D, std=scale, dtype=t), n(M, D, dtype=r)
    W.op_residual_norm_backward(CODE[t], s, y, ds, dh, dx, dy, M, D, post_norm=True, gain=gain, res_dtype=CODE[r])
    S, Y = s.double(), y.double()
    rs, ry = (1 / ((v * v).mean(1, keepdim=True) + T.EPS).sqrt() for v in (S, Y))
    dv = ds.double() + rs * dn - S * rs ** 3 * (dn * S).mean(1, keepdim=True)
    want = ry * (dv - Y * ry ** 2 * (dv * Y).mean(1, keepdim=True))
    size = ds.double().abs() + rs * dn.abs() + S.abs() * rs ** 3 * (dn * S).abs().mean(1, keepdim=True)
    e = (D + 32) * 2.0 ** -22 * ry * (size + Y.abs() * ry ** 2 * (size * Y.abs()).mean(1, keepdim=True))
    T.within(dy, want, e + T.H[t] * (want.abs() + e))


@pytest.mark.parametrize("r,t", [(FP, BF), (BF, BF), (FP, FP)])
@pytest.mark.parametrize("M,per,D", [(19, 7, 4001), (13, 5, 8191), (700, 350, 4001), (1, 0, 7681)])
def test_residual_norm_wide_odd(M, per, D, r, t):
    """Wide rows without vector accesses, 16 and 24 columns a thread, in every type: both directions."""
    test_residual_norm(M, per, D, r, t, True, True, True, True, 0.75)
    test_residual_norm_backward(M, per, D, r, t, True, True, True, True, 0.75)


# ----------------------------------------------------------- more of each
@pytest.mark.parametrize("M,N,K,o,res", [
    (300, 200, 2000, FP, True),    # a segmented reduction, ragged
    (1088, 384, 6144, FP, True),   # seven segments
    (2600, 1100, 1000, FP, False),  # two segments on CTA pairs
    (32, 500, 1537, FP, True),     # segments behind the loader warps
    (16, 4200, 520, BF, True),     # few tokens, two feature groups a block
    (2, 640, 6144, FP, False),     # few tokens, a group shared by a cluster
    (9, 100, 333, BF, True),       # few tokens, rows at any alignment
])
def test_linear_forms(M, N, K, o, res):
    n = T.normals(M + N + K)
    x, w, b = n(M, K, dtype=BF), n(N, K, std=K ** -0.5, dtype=BF), n(N)
    r = n(M, N, dtype=o) if res else None
    y, ok = T.guarded((M, N), o)
    W.op_linear_act(W.BF16, x, w, b, y, M, N, K, residual=r, out_dtype=CODE[o])
    _, _, y64, ey = T.linear64(x, w, b, r, "none", o)
    T.within(y, y64, ey)
    ok()
    if o == FP:  # the accumulation's truncations stay near fp32's own roundings
        assert ((y.double() - y64).norm() / y64.norm()).item() < 1e-6


@pytest.mark.parametrize("N", [1, 8, 31, 32, 33, 64, 65, 80, 95, 96, 97, 128, 160])
def test_linear_fp32_narrow(N):
    """fp32 layers with fewer columns than a tile, at few rows and many."""
    for M, K in ((9, 200), (140, 67), (1000, 320), (40, 1536)):
        n = T.normals(M + N + K)
        x, w, b, r = n(M, K), n(N, K, std=K ** -0.5), n(N), n(M, N)
        (y, ok1), (z, ok2) = T.guarded((M, N), FP), T.guarded((M, N), FP)
        W.op_linear_act(W.FP32, x, w, b, y, M, N, K, act=ACT["silu"], residual=r, z=z)
        z64, ez, y64, ey = T.linear64(x, w, b, r, "silu", FP)
        T.within(y, y64, ey), T.within(z, z64, ez)
        ok1(), ok2()
        (dx, ok1), (dw, ok2), db = T.guarded((M, K), FP), T.guarded((N, K), FP), torch.empty(N, device="cuda")
        W.op_linear_act_backward(W.FP32, x, w, z, r, dx, dw, db, M, N, K, act=ACT["silu"],
                                 workspace=_ws(W.op_linear_act_workspace(W.FP32, M, N, K, act=ACT["silu"])))
        (dx64, ex), [((dw64, ew), (db64, eb))] = T.linear_grad64(x, w, z, r, "silu")
        T.within(dx, dx64, ex), T.within(dw, dw64, ew), T.within(db, db64, eb)
        ok1(), ok2()


@pytest.mark.parametrize("M,N,K,t", [(9000, 100, 72, BF), (9000, 70, 130, BF), (40, 5000, 200, BF), (5128, 271, 74, FP), (43, 3000, 520, FP)])
def test_gradients_in_pieces(M, N, K, t):
    """Few tiles and a long reduction: it is cut into pieces that are added afterwards."""
    n = T.normals(M + N)
    x, w, dy, z = n(M, K, dtype=t), n(N, K, std=K ** -0.5, dtype=t), n(M, N, dtype=t), n(M, N, dtype=t)
    (dx, ok1), (dw, ok2), db = T.guarded((M, K), t), T.guarded((N, K), t), torch.empty(N, device="cuda")
    ws = _ws(W.op_linear_act_workspace(CODE[t], M, N, K, act=ACT["silu"]))
    W.op_linear_act_backward(CODE[t], x, w, z, dy, dx, dw, db, M, N, K, act=ACT["silu"], workspace=ws)
    (dx64, ex), [((dw64, ew), (db64, eb))] = T.linear_grad64(x, w, z, dy, "silu")
    T.within(dx, dx64, ex), T.within(dw, dw64, ew), T.within(db, db64, eb)
    ok1(), ok2()
    a, b = torch.empty_like(dx), torch.empty_like(dw)
    W.op_linear_act_backward(CODE[t], x, w, z, dy, a, b, db, M, N, K, act=ACT["silu"], workspace=ws)
    assert torch.equal(a, dx) and torch.equal(b, dw)
    wu, u = n(N, K, std=K ** -0.5, dtype=t), n(M, N, dtype=t)
    outs = [torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(dw)]
    W.op_gated_backward(CODE[t], x, w, wu, z, u, dy, *outs, M, N, K, workspace=_ws(W.op_gated_workspace(CODE[t], M, N, K)))
    (dx64, ex), [((g64, eg), _), ((u64, eu), _)] = T.gated_grad64(x, w, wu, z, u, dy, "silu")
    T.within(outs[0], dx64, ex), T.within(outs[1], g64, eg), T.within(outs[2], u64, eu)


@pytest.mark.parametrize("M,F,K", [(256, 8192, 1024), (16, 8192, 1536), (64, 8192, 2048), (640, 10816, 512), (2048, 13568, 64),
                                   (70, 8127, 1030)])
def test_gated_backward_across_the_seam(M, F, K):
    """The input gradient sums over two operand pairs in pieces, one of which crosses from the first to the second after
    an odd number of k-blocks: alone and with the other gradients."""
    n = T.normals(M + 3 * F + K)
    x, wg, wu = n(M, K, dtype=BF), n(F, K, std=K ** -0.5, dtype=BF), n(F, K, std=K ** -0.5, dtype=BF)
    g, u, da = n(M, F, dtype=BF, std=1.5), n(M, F, dtype=BF), n(M, F, dtype=BF)
    outs = [T.guarded(s, d) for s, d in (((M, K), BF), ((F, K), BF), ((F, K), BF), ((F,), FP), ((F,), FP))]
    dx, dwg, dwu, dbg, dbu = (o[0] for o in outs)
    ws = _ws(W.op_gated_workspace(W.BF16, M, F, K))
    (dx64, ex), [((g64, eg), (bg64, ebg)), ((u64, eu), (bu64, ebu))] = T.gated_grad64(x, wg, wu, g, u, da, "silu")
    W.op_gated_backward(W.BF16, x, wg, wu, g, u, da, dx, None, None, M, F, K, workspace=ws)
    T.within(dx, dx64, ex)
    alone = dx.clone()
    W.op_gated_backward(W.BF16, x, wg, wu, g, u, da, dx, dwg, dwu, M, F, K, dbias_g=dbg, dbias_u=dbu, workspace=ws)
    T.within(dx, dx64, ex), T.within(dwg, g64, eg), T.within(dwu, u64, eu)
    T.within(dbg, bg64, ebg), T.within(dbu, bu64, ebu)
    T.within(alone, dx64, ex)
    for _, ok in outs:
        ok()
    W.ops_check_status()


@pytest.mark.parametrize("t", [BF, FP])
def test_backward_unaligned(t):
    """Every operand of the backward passes off a 16-byte boundary, one by one and together."""
    M, N, K = 150, 136, 200
    put = lambda v, s: torch.cat([torch.zeros(s, dtype=v.dtype, device="cuda"), v.flatten()])[s:].view(v.shape)  # noqa: E731
    for which in ("x", "w", "dy", "z", "out", "all"):
        n = T.normals(9)
        off = lambda k: 1 if which in (k, "all") else 0  # noqa: E731
        x, w = put(n(M, K, dtype=t), off("x")), put(n(N, K, std=K ** -0.5, dtype=t), off("w"))
        dy, z, u = put(n(M, N, dtype=t), off("dy")), put(n(M, N, dtype=t), off("z")), put(n(M, N, dtype=t), off("z"))
        (dx, ok1), (dw, ok2), (du, ok3) = (T.guarded(s, t, off("out")) for s in ((M, K), (N, K), (N, K)))
        db = torch.empty(N, device="cuda")
        for act, pre in (("none", None), ("gelu_tanh", z)):
            W.op_linear_act_backward(CODE[t], x, w, pre, dy, dx, dw, db, M, N, K, act=ACT[act],
                                     workspace=_ws(W.op_linear_act_workspace(CODE[t], M, N, K, act=ACT[act])))
            (dx64, ex), [((dw64, ew), (db64, eb))] = T.linear_grad64(x, w, pre, dy, act)
            T.within(dx, dx64, ex), T.within(dw, dw64, ew), T.within(db, db64, eb)
        W.op_gated_backward(CODE[t], x, w, w, z, u, dy, dx, dw, du, M, N, K, workspace=_ws(W.op_gated_workspace(CODE[t], M, N, K)))
        (dx64, ex), [((g64, eg), _), ((u64, eu), _)] = T.gated_grad64(x, w, w, z, u, dy, "silu")
        T.within(dx, dx64, ex), T.within(dw, g64, eg), T.within(du, u64, eu)
        ok1(), ok2(), ok3()


@pytest.mark.parametrize("D", [7, 64, 1000, 4100, 8000])
@pytest.mark.parametrize("t", [BF, FP])
def test_residual_norm_unaligned(D, t):
    """Streams and outputs off a 16-byte boundary give the bits that a row's own arithmetic gives elsewhere."""
    M = 9
    n = T.normals(D)
    put = lambda v, s: torch.cat([torch.zeros(s, dtype=v.dtype, device="cuda"), v.flatten()])[s:].view(v.shape)  # noqa: E731
    x, y, g, ds, dh = n(M, D, dtype=t), n(M, D, dtype=t), n(D), n(M, D, dtype=t), n(M, D, dtype=t)
    kw = dict(post_norm=True, gain=g, res_dtype=CODE[t])
    want, got = [], []
    for s, out in ((0, want), (1, got)):
        (sv, ok1), (h, ok2), (dx, ok3), (dy, ok4) = (T.guarded((M, D), t, s) for _ in range(4))
        W.op_residual_norm(CODE[t], put(x, s), put(y, s), sv, h, M, D, **kw)
        W.op_residual_norm_backward(CODE[t], put(x, s), put(y, s), put(ds, s), put(dh, s), dx, dy, M, D, **kw)
        ok1(), ok2(), ok3(), ok4()
        out += [sv, h, dx, dy]
    for a, b in zip(want, got):  # (the order of a row's sums differs: a step or two)
        assert torch.isfinite(b).all()
        assert (a.double() - b.double()).norm() <= 2 * T.H[t] * a.double().norm() + 1e-5 * a.double().norm()


def test_first_call_in_a_capture():
    """A process whose first call of the operators is a captured one."""
    import subprocess
    import sys
    code = """
import torch, sys
import mot_dit_b200 as W
torch.cuda.init()
n = lambda *s: torch.randn(*s, device="cuda").bfloat16()
x, w, y, a, h = n(200, 256), n(512, 256), n(200, 512), n(200, 512), n(200, 256)
s = torch.randn(200, 256, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    st = torch.cuda.current_stream()
    W.op_gated(W.BF16, x, w, w, a, 200, 512, 256, stream=st)
    W.op_linear_act(W.BF16, x, w, None, y, 200, 512, 256, act=2, stream=st)
    W.op_residual_norm(W.BF16, s, x, s, h, 200, 256, post_norm=True, stream=st)
g.replay()
torch.cuda.synchronize()
z = x.double() @ w.double().t()
want = torch.nn.functional.silu(z)
assert ((y.double() - want).norm() / want.norm()).item() < 2.0 ** -7
assert ((a.double() - want * z).norm() / (want * z).norm()).item() < 2.0 ** -7
print("captured first")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


def test_a_failed_call_spoils_no_later_one():
    """A status check inside a capture is refused (it would synchronise), and so is a call on a stream whose capture it
    ended; neither leaves an error for the calls after them."""
    import subprocess
    import sys
    code = """
import torch
import mot_dit_b200 as W
x, w, y = torch.randn(64, 256, device="cuda"), torch.randn(128, 256, device="cuda"), torch.empty(64, 128, device="cuda")
db = torch.ones(8, device="cuda")
torch.cuda.synchronize()
st = torch.cuda.Stream()
g = torch.cuda.CUDAGraph()
with torch.cuda.stream(st):
    g.capture_begin()
    for call in (W.ops_check_status, lambda: W.op_linear_act_backward(W.FP32, None, None, None, None, None, None, db, 0, 8, 256, stream=st)):
        try:
            call()
            raise SystemExit("not refused")
        except W.WamError as e:
            assert e.status == 4, e
    try:
        g.capture_end()
    except RuntimeError:
        pass
W.op_linear(W.FP32, x, w, torch.zeros(128, device="cuda"), y, 64, 128, 256)
W.ops_check_status()
want = x.double() @ w.double().t()
assert ((y.double() - want).norm() / want.norm()).item() < 1e-5
print("later call ok")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "later call ok" in r.stdout, r.stdout + r.stderr[-2000:]


def test_fp32_products_are_fp32():
    """Three parts an operand: the sums are as near as an fp32 matrix product's, at any scale of the operands."""
    M, N, K = 200, 300, 1500
    n = T.normals(5)
    for scale in (1.0, 1e-20, 1e15):
        x, w = n(M, K, std=scale), n(N, K, std=1 / scale)
        y = torch.empty(M, N, device="cuda")
        W.op_linear_act(W.FP32, x, w, None, y, M, N, K)
        want = x.double() @ w.double().t()
        assert ((y.double() - want).norm() / want.norm()).item() < 1e-6


@pytest.mark.parametrize("M,N,K", [(1100, 2000, 16384), (1100, 2000, 5400), (300, 200, 40000), (64, 64, 100000)])
def test_fp32_products_of_long_reductions(M, N, K):
    """The error relative to the result does not grow with the reduction: its accumulators' chains are no longer than
    those of K = 1500 (errors of independent chains add up as the chains do), and the fp32 additions of the K / 768
    chains are off by 2^-24 each, 4e-8 sqrt(K / 768) of the result together: half of the bound at K = 100000."""
    n = T.normals(M + K)
    x, w, y = n(M, K), n(N, K, std=K ** -0.5), torch.empty(M, N, device="cuda")
    W.op_linear_act(W.FP32, x, w, None, y, M, N, K)
    want = x.double() @ w.double().t()
    assert ((y.double() - want).norm() / want.norm()).item() < 1e-6
    _, _, y64, ey = T.linear64(x, w, None, None, "none", FP)
    T.within(y, y64, ey)


@pytest.mark.parametrize("M,F,K", [(1100, 1000, 6000), (2100, 20, 5500), (300, 3000, 12000)])
def test_gated_fp32_of_long_reductions(M, F, K):
    """A gated layer's two halves through several rounds, in tiles of either width."""
    n = T.normals(M + F)
    x, wg, wu = n(M, K), n(F, K, std=K ** -0.5), n(F, K, std=K ** -0.5)
    (a, ok1), (g, ok2), (u, ok3) = (T.guarded((M, F), FP) for _ in range(3))
    W.op_gated(W.FP32, x, wg, wu, a, M, F, K, g=g, u=u)
    (a64, ea), (g64, eg), (u64, eu) = T.gated64(x, wg, wu, None, None, "silu")
    T.within(a, a64, ea), T.within(g, g64, eg), T.within(u, u64, eu)
    for got, want in ((g, g64), (u, u64)):
        assert ((got.double() - want).norm() / want.norm()).item() < 1e-6
    ok1(), ok2(), ok3()
    a2 = torch.empty_like(a)
    W.op_gated(W.FP32, x, wg, wu, a2, M, F, K)
    assert torch.equal(a, a2)


@pytest.mark.parametrize("M,F,K", [(1000, 8127, 1100), (64, 20000, 700), (20000, 300, 200)])
def test_gated_backward_fp32_of_long_reductions(M, F, K):
    """Rounds of a reduction over two operand pairs, whole and in pieces, and of the weights' over many rows."""
    n = T.normals(M + F)
    x, wg, wu = n(M, K), n(F, K, std=K ** -0.5), n(F, K, std=K ** -0.5)
    g, u, da = n(M, F, std=1.5), n(M, F), n(M, F)
    outs = [T.guarded(s, FP) for s in ((M, K), (F, K), (F, K), (F,), (F,))]
    W.op_gated_backward(W.FP32, x, wg, wu, g, u, da, *(o[0] for o in outs[:3]), M, F, K, dbias_g=outs[3][0], dbias_u=outs[4][0],
                        workspace=_ws(W.op_gated_workspace(W.FP32, M, F, K)))
    dx, [(dwg, dbg), (dwu, dbu)] = T.gated_grad64(x, wg, wu, g, u, da, "silu")
    for (got, ok), (want, e) in zip(outs, (dx, dwg, dwu, dbg, dbu)):
        T.within(got, want, e)
        ok()
    for (got, _), (want, _) in zip(outs[:3], (dx, dwg, dwu)):
        assert ((got.double() - want).norm() / want.norm()).item() < 1.5e-6  # (1e-6 as above, and dg's own roundings)


@pytest.mark.parametrize("t", [BF, FP])
def test_linear_special_values(t):
    """A row with a NaN or an infinity spoils itself only; infinite pre-activations have their limits."""
    M, N, K = 140, 64, 96
    n = T.normals(3)
    x, w = n(M, K, dtype=t), n(N, K, dtype=t)
    clean = torch.empty(M, N, dtype=t, device="cuda")
    W.op_linear_act(CODE[t], x, w, None, clean, M, N, K, act=ACT["silu"])
    x[7, 3], x[90, 5] = float("nan"), float("inf")
    y = torch.empty_like(clean)
    W.op_linear_act(CODE[t], x, w, None, y, M, N, K, act=ACT["silu"])
    bad = ~torch.isfinite(y)
    assert torch.isnan(y[7]).all() and bad[90].any()
    keep = [i for i in range(M) if i not in (7, 90)]
    assert torch.equal(y[keep], clean[keep])
    z = torch.tensor([[float("inf"), float("-inf"), 1e30, -1e30, 0.0, -0.0, 100.0, -100.0]], device="cuda").to(t)
    z = torch.nn.functional.pad(z, (0, 56))
    dy = torch.ones(1, N, dtype=t, device="cuda")
    for name, limit in (("silu", [1, 0, 1, 0]), ("gelu_tanh", [1, 0, 1, 0]), ("gelu_erf", [1, 0, 1, 0]), ("sigmoid", [0, 0, 0, 0]),
                        ("relu", [1, 0, 1, 0])):
        db = torch.empty(N, device="cuda")
        ws = _ws(W.op_linear_act_workspace(CODE[t], 1, N, K, act=ACT[name]))
        W.op_linear_act_backward(CODE[t], None, None, z, dy, None, None, db, 1, N, K, act=ACT[name], workspace=ws)
        assert torch.isfinite(db).all() and db[:4].tolist() == limit, (name, db[:4])


@pytest.mark.parametrize("act", W.ACTS)
def test_gradients_against_differences(act):
    """fp32: central differences of the forward operators themselves."""
    M, N, K = 6, 24, 32
    n = T.normals(11)
    x, w, b, dy = n(M, K), n(N, K, std=K ** -0.5), n(N, std=0.3), n(M, N)
    if act == "relu":  # (no pre-activation within a step of the corner)
        b = b + 0.0
    run = lambda x_, w_: (W.op_linear_act(W.FP32, x_, w_, b, y, M, N, K, act=ACT[act], z=z), (y.double() * dy.double()).sum().item())[1]  # noqa: E731
    y, z = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    run(x, w)
    z0 = z.clone()
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    W.op_linear_act_backward(W.FP32, x, w, z0, dy, dx, dw, db, M, N, K, act=ACT[act],
                             workspace=_ws(W.op_linear_act_workspace(W.FP32, M, N, K, act=ACT[act])))
    h = 2.0 ** -7
    for (src, grad, at) in ((x, dx, (2, 5)), (x, dx, (5, 31)), (w, dw, (3, 7)), (w, dw, (23, 0))):
        lo, hi = src.clone(), src.clone()
        lo[at] -= h
        hi[at] += h
        if act == "relu":
            run(hi if src is x else x, hi if src is w else w)
            z1 = z.clone()
            run(lo if src is x else x, lo if src is w else w)
            if ((z1 > 0) != (z > 0)).any():  # a corner between the two points: no difference quotient
                continue
        diff = (run(hi if src is x else x, hi if src is w else w) - run(lo if src is x else x, lo if src is w else w)) / (2 * h)
        # third derivatives times h^2 / 6 of up to N terms, and fp32 rounding over 2 h
        assert abs(diff - grad[at].item()) < 1e-3 * (1 + abs(diff)), (act, at, diff, grad[at].item())


def test_zero_rows():
    n = T.normals(1)
    w = n(24, 32, dtype=BF)
    e = torch.empty(0, 32, dtype=BF, device="cuda")
    o = torch.empty(0, 24, dtype=BF, device="cuda")
    W.op_linear_act(W.BF16, e, w, None, o, 0, 24, 32)
    W.op_gated(W.BF16, e, w, w, o, 0, 24, 32)
    dw, db = torch.full((24, 32), 5.0, dtype=BF, device="cuda"), torch.full((24,), 5.0, device="cuda")
    W.op_linear_act_backward(W.BF16, e, w, o, o, e.clone(), dw, db, 0, 24, 32, act=2)
    assert not dw.any() and not db.any()
    d2, d3, b2, b3 = torch.ones_like(dw), torch.ones_like(dw), torch.ones_like(db), torch.ones_like(db)
    W.op_gated_backward(W.BF16, e, w, w, o, o, o, e.clone(), d2, d3, 0, 24, 32, dbias_g=b2, dbias_u=b3)
    assert not d2.any() and not d3.any() and not b2.any() and not b3.any()
    g = torch.ones(32, device="cuda")
    z = torch.empty(0, 32, device="cuda")
    W.op_residual_norm(W.BF16, z, e, z.clone(), e.clone(), 0, 32)
    W.op_residual_norm_backward(W.BF16, z, e, z, e, z.clone(), e.clone(), 0, 32, post_norm=True, dpost_gain=g)
    assert not g.any()


def _block(stream, s, M=70, D=264, F=520, G=2):
    """A feed-forward half of a block, forward and backward, with the operators alone; s: its buffers."""
    per = -(-M // G)
    kw = dict(stream=stream)
    W.op_gated(W.BF16, s["h"], s["wg"], s["wu"], s["a"], M, F, D, g=s["g"], u=s["u"], **kw)
    W.op_linear_act(W.BF16, s["a"], s["wd"], s["bd"], s["y"], M, D, F, **kw)
    mod = dict(post_norm=True, post_gain=s["pg"], gate=s["table"][:, 0], gain=s["gain"], scale=s["table"][:, 1], rows_per_group=per,
               ld_mod=3 * D)
    W.op_residual_norm(W.BF16, s["x"], s["y"], s["s"], s["h2"], M, D, shift=s["table"][:, 2], **mod, **kw)
    W.op_residual_norm_backward(W.BF16, s["s"], s["y"], s["ds"], s["dh2"], s["dx"], s["dy"], M, D, dpost_gain=s["dpg"], dgate=s["dgate"],
                                dgain=s["dgain"], dscale=s["dscale"], dshift=s["dshift"], workspace=s["ws1"], **mod, **kw)
    W.op_linear_act_backward(W.BF16, s["a"], s["wd"], None, s["dy"], s["da"], s["dwd"], s["dbd"], M, D, F, workspace=s["ws2"], **kw)
    W.op_gated_backward(W.BF16, s["h"], s["wg"], s["wu"], s["g"], s["u"], s["da"], s["dh"], s["dwg"], s["dwu"], M, F, D,
                        workspace=s["ws3"], **kw)


def _block_state(seed, M=70, D=264, F=520, G=2):
    n = T.normals(seed)
    b = lambda *sh: torch.full(sh, float("nan"), dtype=BF, device="cuda")  # noqa: E731
    f = lambda *sh: torch.full(sh, float("nan"), device="cuda")  # noqa: E731
    return dict(h=n(M, D, dtype=BF), x=n(M, D), wg=n(F, D, std=D ** -0.5, dtype=BF), wu=n(F, D, std=D ** -0.5, dtype=BF),
                wd=n(D, F, std=F ** -0.5, dtype=BF), bd=n(D, std=0.1), pg=n(D, mean=1.0, std=0.1), gain=n(D, mean=1.0, std=0.1),
                table=n(G, 3, D, std=0.5), ds=n(M, D), dh2=n(M, D, dtype=BF), a=b(M, F), g=b(M, F), u=b(M, F), y=b(M, D), s=f(M, D),
                h2=b(M, D), dx=f(M, D), dy=b(M, D), dpg=f(D), dgate=f(G, D), dgain=f(D), dscale=f(G, D), dshift=f(G, D), da=b(M, F),
                dwd=b(D, F), dbd=f(D), dh=b(M, D), dwg=b(F, D), dwu=b(F, D), ws1=_ws(W.op_residual_norm_workspace(M, D, -(-M // G))),
                ws2=_ws(W.op_linear_act_workspace(W.BF16, M, D, F)), ws3=_ws(W.op_gated_workspace(W.BF16, M, F, D)))


def test_block_against_autograd():
    """The operators together against the definition's gradient in 64 bits.  Every stage rounds to bf16 once or twice
    (2^-8 each); eight such roundings lie on the longest way, and errors pass through factors of about one."""
    M, D, G = 70, 264, 2
    s = _block_state(0)
    _block(None, s)
    leaf = {k: s[k].double().requires_grad_() for k in ("h", "x", "wg", "wu", "wd", "bd", "pg", "gain", "table")}
    a = torch.nn.functional.silu(leaf["h"] @ leaf["wg"].t()) * (leaf["h"] @ leaf["wu"].t())
    y = a @ leaf["wd"].t() + leaf["bd"]
    tb = leaf["table"]
    st, h2 = T.norm64(leaf["x"], y, True, leaf["pg"], tb[:, 0], leaf["gain"], tb[:, 1], tb[:, 2], 1.0, M // G)
    grads = dict(zip(leaf, torch.autograd.grad([st, h2], list(leaf.values()), [s["ds"].double(), s["dh2"].double()])))
    got = dict(h="dh", x="dx", wg="dwg", wu="dwu", wd="dwd", bd="dbd", pg="dpg", gain="dgain")
    pairs = [(s["s"], st), (s["h2"], h2)] + [(s[v], grads[k]) for k, v in got.items()]
    pairs += [(s[k], grads["table"][:, i]) for i, k in enumerate(("dgate", "dscale", "dshift"))]
    for x, want in pairs:
        assert torch.isfinite(x).all()
        assert ((x.double() - want).norm() / want.norm()).item() < 8 * 2.0 ** -8


def test_block_captured_and_on_streams():
    """A captured block replays to the eager bits with new inputs; two streams with their own workspaces do not disturb
    each other; tensors made on one stream are used on another."""
    keys = ("s", "h2", "dx", "dy", "dpg", "dgate", "dgain", "dscale", "dshift", "dwd", "dbd", "dh", "dwg", "dwu")
    want = {}
    for seed in (1, 2):
        s = _block_state(seed)
        _block(None, s)
        want[seed] = {k: s[k].clone() for k in keys}
    s = _block_state(1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _block(torch.cuda.current_stream(), s)
    for seed in (2, 1, 2):
        new = _block_state(seed)
        for k in ("h", "x", "wg", "wu", "wd", "bd", "pg", "gain", "table", "ds", "dh2"):
            s[k].copy_(new[k])
        g.replay()
        torch.cuda.synchronize()
        for k in keys:
            assert torch.equal(s[k], want[seed][k]), (seed, k)
    s1, s2 = _block_state(1), _block_state(2)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    a.wait_stream(torch.cuda.current_stream()), b.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        _block(a, s1)
        _block(b, s2)
    torch.cuda.synchronize()
    for k in keys:
        assert torch.equal(s1[k], want[1][k]) and torch.equal(s2[k], want[2][k]), k
