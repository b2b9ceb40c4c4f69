"""Argument checks and workspace sizes of the feed-forward and residual-norm
operators, on a host without a GPU: every refusal comes before a device call."""
import ctypes as C

import numpy as np
import pytest

import mot_dit_b200 as W

P = 1 << 20  # addresses that are only compared
M, N, K, D = 8, 64, 32, 64


def _lin(**kw):
    a = dict(dtype=W.BF16, out=W.FP32, x=P, w=2 * P, b=3 * P, r=0, y=4 * P, z=0, M=M, N=N, K=K, act=0)
    a.update(kw)
    return W.lib().wam_op_linear_act(a["dtype"], a["out"], a["x"], a["w"], a["b"], a["r"], a["y"], a["z"], a["M"], a["N"], a["K"],
                                     a["act"], None)


@pytest.mark.parametrize("bad", [
    dict(dtype=7), dict(out=3), dict(dtype=W.FP32, out=W.BF16), dict(act=-1), dict(act=6), dict(M=-1), dict(N=0), dict(K=0),
    dict(N=1 << 25), dict(x=0), dict(w=0), dict(y=0), dict(x=P + 1), dict(y=4 * P + 2), dict(b=3 * P + 2), dict(z=4 * P + 1),
    dict(y=P), dict(y=2 * P + 64), dict(z=4 * P), dict(r=4 * P + 4), dict(y=3 * P - 4),
])
def test_linear_refusals(bad):
    assert _lin(**bad) == 1


def test_zero_rows_need_no_device():
    assert _lin(M=0) == 0
    assert W.lib().wam_op_gated(W.BF16, P, 2 * P, 3 * P, None, None, 4 * P, None, None, 0, N, K, 2, None) == 0


def _lin_bwd(**kw):
    a = dict(dtype=W.BF16, dyt=W.BF16, x=P, w=2 * P, z=3 * P, dy=4 * P, dx=5 * P, dw=6 * P, db=7 * P, M=M, N=N, K=K, act=2, ws=8 * P,
             nb=1 << 19)
    a.update(kw)
    return W.lib().wam_op_linear_act_backward(a["dtype"], a["dyt"], a["x"], a["w"], a["z"], a["dy"], a["dx"], a["dw"], a["db"], a["M"],
                                              a["N"], a["K"], a["act"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("bad", [
    dict(dtype=2), dict(dtype=W.FP32), dict(act=9), dict(z=0), dict(dy=0), dict(x=0), dict(w=0), dict(dx=0, dw=0, db=0), dict(ws=0),
    dict(nb=16), dict(ws=8 * P + 16), dict(dx=P), dict(dw=4 * P), dict(dw=5 * P), dict(db=8 * P), dict(M=-2), dict(K=-1), dict(dx=5 * P + 1),
])
def test_linear_backward_refusals(bad):
    assert _lin_bwd(**bad) == 1


def _gated(**kw):
    a = dict(dtype=W.BF16, x=P, wg=2 * P, wu=3 * P, bg=0, bu=0, a=4 * P, g=5 * P, u=6 * P, M=M, F=N, K=K, act=2)
    a.update(kw)
    return W.lib().wam_op_gated(a["dtype"], a["x"], a["wg"], a["wu"], a["bg"], a["bu"], a["a"], a["g"], a["u"], a["M"], a["F"], a["K"],
                                a["act"], None)


@pytest.mark.parametrize("bad", [
    dict(dtype=5), dict(act=6), dict(x=0), dict(wg=0), dict(wu=0), dict(a=0), dict(g=0), dict(u=0), dict(a=5 * P), dict(u=5 * P),
    dict(a=P), dict(F=0), dict(K=0), dict(M=-1), dict(g=5 * P + 1),
])
def test_gated_refusals(bad):
    assert _gated(**bad) == 1


def _gated_bwd(**kw):
    a = dict(x=P, wg=2 * P, wu=3 * P, g=4 * P, u=5 * P, da=6 * P, dx=7 * P, dwg=8 * P, dwu=9 * P, dbg=10 * P, dbu=11 * P, M=M, F=N, K=K,
             act=2, ws=12 * P, nb=1 << 19)
    a.update(kw)
    return W.lib().wam_op_gated_backward(W.BF16, *[a[k] for k in ("x", "wg", "wu", "g", "u", "da", "dx", "dwg", "dwu", "dbg", "dbu", "M",
                                                                  "F", "K", "act", "ws", "nb")], None)


@pytest.mark.parametrize("bad", [
    dict(x=0), dict(wg=0), dict(g=0), dict(u=0), dict(da=0), dict(dwg=0), dict(dbu=0), dict(dx=0, dwg=0, dwu=0, dbg=0, dbu=0), dict(ws=0),
    dict(nb=0), dict(dx=6 * P), dict(dwu=8 * P), dict(act=-1), dict(M=-1), dict(F=0),
])
def test_gated_backward_refusals(bad):
    assert _gated_bwd(**bad) == 1


def _norm(**kw):
    a = dict(dtype=W.BF16, rt=W.FP32, x=P, y=2 * P, s=3 * P, h=4 * P, M=M, D=D, al=1.0, post=1, pg=5 * P, gate=6 * P, gain=7 * P,
             scale=8 * P, shift=9 * P, per=4, ld=D)
    a.update(kw)
    return W.lib().wam_op_residual_norm(*[a[k] for k in ("dtype", "rt", "x", "y", "s", "h", "M", "D", "al", "post", "pg", "gate", "gain",
                                                         "scale", "shift", "per", "ld")], None)


@pytest.mark.parametrize("bad", [
    dict(dtype=4), dict(rt=4), dict(dtype=W.FP32, rt=W.BF16), dict(x=0), dict(y=0), dict(s=0), dict(h=0), dict(D=0), dict(D=8193),
    dict(M=-1), dict(per=-1), dict(post=0), dict(ld=D - 1), dict(s=P + 4), dict(h=P), dict(s=6 * P), dict(s=2 * P), dict(x=P + 2),
    dict(gate=6 * P + 1), dict(h=3 * P),
])
def test_norm_refusals(bad):
    assert _norm(**bad) == 1


def _norm_bwd(**kw):
    a = dict(dtype=W.BF16, rt=W.FP32, s=P, y=2 * P, ds=3 * P, dh=4 * P, dx=5 * P, dy=6 * P, M=M, D=D, al=1.0, post=1, pg=7 * P, gate=8 * P,
             gain=9 * P, scale=10 * P, per=4, ld=D, dpg=11 * P, dgate=12 * P, dgain=13 * P, dscale=14 * P, dshift=15 * P, ws=16 * P,
             nb=1 << 19)
    a.update(kw)
    return W.lib().wam_op_residual_norm_backward(*[a[k] for k in (
        "dtype", "rt", "s", "y", "ds", "dh", "dx", "dy", "M", "D", "al", "post", "pg", "gate", "gain", "scale", "per", "ld", "dpg", "dgate",
        "dgain", "dscale", "dshift", "ws", "nb")], None)


@pytest.mark.parametrize("bad", [
    dict(dtype=3), dict(dtype=W.FP32, rt=W.BF16), dict(s=0), dict(y=0), dict(dh=0), dict(dx=0), dict(dy=0), dict(ws=0), dict(nb=8),
    dict(post=0), dict(dx=4 * P), dict(dy=3 * P), dict(dx=3 * P + 4), dict(dgate=13 * P), dict(dscale=4 * P), dict(D=9000), dict(ld=3),
    dict(dy=5 * P), dict(dgain=16 * P),
])
def test_norm_backward_refusals(bad):
    assert _norm_bwd(**bad) == 1


def test_workspace_sizes():
    # nothing but the partial sums when the incoming gradient is the operand itself
    small = W.op_linear_act_workspace(W.BF16, 1000, 512, 256)
    assert 0 < small < 1000 * 512 * 2
    assert W.op_linear_act_workspace(W.BF16, 1000, 512, 256, act=2) >= small + 1000 * 512 * 2
    assert W.op_linear_act_workspace(W.BF16, 1000, 513, 256) >= 1000 * 520 * 2  # rows padded to 16 bytes
    assert W.op_linear_act_workspace(W.BF16, 1000, 512, 257) >= (1000 + 512) * 264 * 2  # operands copied
    assert W.op_linear_act_workspace(W.FP32, 1000, 513, 257, act=1) < 1000 * 520 * 4 + 16 * 513 * 257 * 4
    # a narrow layer over many rows: its weight gradient's reduction in pieces
    assert W.op_linear_act_workspace(W.BF16, 8192, 128, 128) >= 2 * 128 * 128 * 4
    assert W.op_gated_workspace(W.BF16, 100, 200, 64) >= 2 * 100 * 200 * 2
    assert W.op_residual_norm_workspace(0, 64) == 0
    assert W.op_residual_norm_workspace(100, 64, 1) == 100 * 3 * 64 * 4
    n = C.c_size_t(0)
    for f, a in ((W.lib().wam_op_gated_workspace, (W.BF16, -1, 8, 8)), (W.lib().wam_op_gated_workspace, (9, 8, 8, 8)),
                 (W.lib().wam_op_linear_act_workspace, (W.FP32, 8, 8, 8, 0, W.BF16)),
                 (W.lib().wam_op_residual_norm_workspace, (8, 0, 0))):
        assert f(*a, C.byref(n)) == 1 and f(*a, None) == 1


def test_binding_checks_tensors():
    """Tensors of another type, size, layout or device are refused before the library is called."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(M, K, dtype=torch.bfloat16)
    ok = dict(x=P, w=2 * P, bias=3 * P, y=4 * P)
    for name, t in (("x", x), ("y", np.zeros(3))):
        with pytest.raises((W.WamError, AttributeError)):
            W.op_linear_act(W.BF16, *[{**ok, name: t}[k] for k in ("x", "w", "bias", "y")], M, N, K)
    with pytest.raises(W.WamError):
        W.op_gated(W.BF16, x, 2 * P, 3 * P, 4 * P, M, N, K)
    with pytest.raises(W.WamError):
        W.op_residual_norm(W.BF16, P, 2 * P, 3 * P, 4 * P, M, D, gate=torch.zeros(2, D), rows_per_group=4)
    with pytest.raises(W.WamError):
        W.op_gated_backward(W.BF16, P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 8 * P, 9 * P, M, N, K, workspace=torch.zeros(1 << 20))


BIG = 1 << 32


@pytest.mark.parametrize("call", [
    lambda: W.op_linear_act_workspace(W.BF16, BIG + M, N, K), lambda: W.op_linear_act_workspace(W.BF16, M, N, K, act=BIG),
    lambda: W.op_gated_workspace(W.BF16, M, BIG + N, K), lambda: W.op_gated_workspace(BIG + W.BF16, M, N, K),
    lambda: W.op_residual_norm_workspace(BIG + M, D), lambda: W.op_residual_norm_workspace(M, D, BIG + 1),
    lambda: W.op_linear_act(W.BF16, P, 2 * P, 3 * P, 4 * P, BIG, N, K), lambda: W.op_linear_act(W.BF16, P, 2 * P, 3 * P, 4 * P, M, N, -K),
    lambda: W.op_linear_act_backward(W.BF16, P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, M, BIG + N, K, workspace=8 * P),
    lambda: W.op_gated(W.BF16, P, 2 * P, 3 * P, 4 * P, BIG, N, K),
    lambda: W.op_gated_backward(W.BF16, P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, 7 * P, 8 * P, 9 * P, M, N, BIG + K, workspace=10 * P),
    lambda: W.op_residual_norm(W.BF16, P, 2 * P, 3 * P, 4 * P, BIG, D),
    lambda: W.op_residual_norm(W.BF16, P, 2 * P, 3 * P, 4 * P, M, D, gate=5 * P, rows_per_group=4, ld_mod=BIG + D),
    lambda: W.op_residual_norm_backward(W.BF16, P, 2 * P, 3 * P, 4 * P, 5 * P, 6 * P, BIG, D),
])
def test_binding_refuses_what_32_bits_cannot_hold(call):
    """ctypes would pass a size's low 32 bits on (a workspace for 16 rows where 2^32 + 16 were asked for)."""
    with pytest.raises(W.WamError) as e:
        call()
    assert e.value.status == 1
    assert W.op_residual_norm_workspace(M, D, 1) == M * 3 * D * 4  # (and ordinary sizes pass)
