"""64-bit definitions of the feed-forward and residual-norm operators, with
elementwise error bounds of the kernels' arithmetic.

Half a rounding step is H[type] relative to the value.  A sum of K products
in fp32 is off by at most K 2^-23 sum |a b| (the tensor core may truncate, so a
whole step is counted per addition).  The activations have |act'| < 1.2 and are
evaluated to a few fp32 steps (counted as 2^-18 of |z| + 1: exp's argument error
grows with |z| but the result then vanishes or saturates)."""
from __future__ import annotations

import math

import torch

H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS = 1e-6
ACT_ERR = 2.0 ** -18


def act64(z, name):
    f = torch.nn.functional
    return {"none": lambda: z, "relu": lambda: f.relu(z), "sigmoid": lambda: torch.sigmoid(z), "silu": lambda: f.silu(z),
            "gelu_tanh": lambda: f.gelu(z, approximate="tanh"), "gelu_erf": lambda: f.gelu(z)}[name]()


def dact64(z, name):
    z = z.detach().clone().requires_grad_()
    return torch.autograd.grad(act64(z, name).sum(), z)[0]


def product(a, b, terms=None):
    """a b^T in 64 bits and the bound of its fp32 sum's error."""
    a, b = a.double(), b.double()
    return a @ b.t(), (terms or a.shape[1]) * 2.0 ** -23 * (a.abs() @ b.abs().t())


def within(got, want, bound):
    """Every element finite and within its bound (an absolute floor covers exact zeros)."""
    got = got.double()
    assert torch.isfinite(got).all(), "non-finite output"
    off = (got - want).abs() - bound - 1e-30
    worst = off.max().item()
    assert worst <= 0, f"off by {((got - want).abs() / (bound + 1e-30)).max().item():.3g} bounds (max {worst:.3g} past its bound)"


def linear64(x, w, bias, res, act, out_type):
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -23 * z.abs()
    y = act64(z, act)
    ey = 1.2 * ez + (0 if act == "none" else ACT_ERR * (z.abs() + 1))
    if res is not None:
        y = y + res.double()
        ey = ey + 2.0 ** -23 * y.abs()
    return z, ez + H[x.dtype] * (z.abs() + ez), y, ey + H[out_type] * (y.abs() + ey)


def linear_grad64(x, w, z, dy, act):
    """(dx, dw, db) and their bounds; dz is rounded to the compute type."""
    t = x.dtype
    d, zd = dy.double(), None if z is None else z.double()
    der = torch.ones_like(d) if z is None else dact64(zd, act)
    dz = d * der
    ez = d.abs() * (0 if z is None else ACT_ERR * (zd.abs() + 1)) + 2.0 ** -23 * dz.abs()  # before rounding
    return _grads(x, [(dz, ez, w)], t)


def _grads(x, sides, t):
    dx = edx = 0
    out = []
    terms = sum(d.shape[1] for d, _, _ in sides)
    for d, e, w in sides:
        er = e + (H[t] * (d.abs() + e) if t != torch.float32 else 0)  # the product's operand
        wa = w.double()
        dx = dx + d @ wa
        edx = edx + er @ wa.abs() + terms * 2.0 ** -23 * ((d.abs() + er) @ wa.abs())
        xd = x.double()
        dw, edw = d.t() @ xd, er.t() @ xd.abs() + d.shape[0] * 2.0 ** -23 * ((d.abs() + er).t() @ xd.abs())
        db, edb = d.sum(0), e.sum(0) + d.shape[0] * 2.0 ** -24 * (d.abs() + e).sum(0)
        out.append(((dw, edw + H[t] * (dw.abs() + edw)), (db, edb + 2.0 ** -24 * db.abs())))
    return (dx, edx + H[t] * (dx.abs() + edx)), out


def gated64(x, wg, wu, bg, bu, act):
    t = x.dtype
    (g, eg), (u, eu) = product(x, wg), product(x, wu)
    if bg is not None:
        g, eg = g + bg.double(), eg + 2.0 ** -23 * (g + bg.double()).abs()
    if bu is not None:
        u, eu = u + bu.double(), eu + 2.0 ** -23 * (u + bu.double()).abs()
    f = act64(g, act)
    ef = 1.2 * eg + (0 if act == "none" else ACT_ERR * (g.abs() + 1))
    a = f * u
    ea = ef * (u.abs() + eu) + f.abs() * eu + 2.0 ** -23 * a.abs()
    return (a, ea + H[t] * (a.abs() + ea)), (g, eg + H[t] * (g.abs() + eg)), (u, eu + H[t] * (u.abs() + eu))


def gated_grad64(x, wg, wu, g, u, da, act):
    g, u, da, t = g.double(), u.double(), da.double(), x.dtype
    f, df = act64(g, act), dact64(g, act)
    ea = 0 if act == "none" else ACT_ERR * (g.abs() + 1)
    dg, du = da * u * df, da * f
    return _grads(x, [(dg, (da * u).abs() * ea + 2.0 ** -22 * dg.abs(), wg), (du, da.abs() * ea + 2.0 ** -23 * du.abs(), wu)], t)


def spread(v, M, per):
    return None if v is None else v.double().repeat_interleave(per, 0)[:M]


def norm64(x, y, post, post_gain, gate, gain, scale, shift, alpha, per):
    """(s, h) with gradients attached to whatever of the inputs carries them (all 64-bit)."""
    M = x.shape[0]
    rms = lambda v: v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)  # noqa: E731
    rows = lambda v: v.repeat_interleave(per, 0)[:M]  # noqa: E731
    p = rms(y) if post else y
    if post_gain is not None:
        p = p * post_gain
    s = alpha * x + (p * rows(gate) if gate is not None else p)
    h = rms(s)
    if gain is not None:
        h = h * gain
    if scale is not None:
        h = h * (1 + rows(scale))
    if shift is not None:
        h = h + rows(shift)
    return s, h


def normals(seed, dev="cuda"):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def make(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g, device=dev) * std + mean).to(dtype)
    return make


def guarded(shape, dtype, shift=0):
    """A NaN-filled output inside a larger buffer of NaNs, `shift` elements past
    an aligned address; returns (the output, a check that nothing around it was written)."""
    n, pad = math.prod(shape), 512
    buf = torch.full((n + 2 * pad + shift,), float("nan"), dtype=dtype, device="cuda")
    lo = pad + shift

    def intact():
        assert torch.isnan(buf[:lo]).all() and torch.isnan(buf[lo + n:]).all(), "bytes around an output were written"
    return buf[lo:lo + n].view(shape), intact
