"""A layer's operators without a GPU: their argument checks (in the library and in
the binding) fire before anything touches a device, and the plain forms the GPU
tests compare with are the published generator and the formulas' derivatives."""
import inspect
import os
import re

import numpy as np
import pytest
import torch

import _layer
import zero_dp_partitioned_amd as zdp
from zero_dp_partitioned_amd import build

A = 1 << 20  # an aligned address that is never read: the checks come first
BIG = 2 ** 62
F32, F16, BF16 = zdp.DT_F32, zdp.DT_F16, zdp.DT_BF16


@pytest.fixture(scope="module")
def lib():
    return zdp.load()


def refuse(call, bad, rc):
    for kw in bad:
        assert call(**kw) == rc, kw
        assert zdp.last_error()


def caller(fn, **ok):
    """fn with these arguments, in this order, and any of them replaced."""
    def call(**kw):
        assert set(kw) <= set(ok)
        return fn(*{**ok, **kw}.values(), None)
    return call


def test_norm_refusals(lib):
    call = caller(lib.zero_layer_norm, x=A, dt=F32, rows=4, cols=40, x_ld=40, weight=A, bias=A, w_dt=F32, eps=1e-5, y=A,
                  y_ld=40, mean=A, rstd=A)
    refuse(call, (dict(rows=-1), dict(cols=-1), dict(dt=0), dict(dt=4), dict(w_dt=F16), dict(dt=F16, w_dt=BF16),
                  dict(x_ld=39), dict(y_ld=39), dict(x=None), dict(y=None), dict(weight=None), dict(mean=None),
                  dict(rstd=None), dict(eps=-1e-9), dict(eps=float("nan")), dict(eps=float("inf")), dict(x_ld=BIG),
                  dict(y_ld=BIG), dict(rows=BIG)), zdp.ERR_INVALID_ARG)
    refuse(call, (dict(x=A + 2), dict(y=A + 1), dict(dt=F16, x=A + 1), dict(weight=A + 2), dict(bias=A + 3),
                  dict(mean=A + 2), dict(rstd=A + 2)), zdp.ERR_ALIGNMENT)
    refuse(call, (dict(cols=2 ** 20 + 1, x_ld=2 ** 21, y_ld=2 ** 21),), zdp.ERR_UNSUPPORTED)
    assert call(rows=0, x=None, y=None, mean=None, rstd=None) == zdp.OK
    assert call(cols=0, x=None, y=None, weight=None) == zdp.OK


@pytest.mark.parametrize("eps", [3.5e38, 1e39, 1e300])
def test_an_eps_past_fp32_is_refused(lib, eps):
    """It would be infinity, and every row its bias."""
    call = caller(lib.zero_layer_norm, x=A, dt=F32, rows=0, cols=40, x_ld=40, weight=A, bias=A, w_dt=F32, eps=eps, y=A,
                  y_ld=40, mean=A, rstd=A)
    assert call() == zdp.ERR_INVALID_ARG and "eps" in zdp.last_error()
    assert call(eps=3.4e38) == call(eps=1e-45) == call(eps=5e-324) == call(eps=0.0) == zdp.OK


def test_norm_backward_refusals(lib):
    ws = zdp.workspace_bytes(1)
    call = caller(lib.zero_layer_norm_backward, dy=A, dy_ld=40, x=A, x_ld=40, dt=F32, rows=4, cols=40, weight=A, w_dt=F32,
                  mean=A, rstd=A, res=A, res_ld=40, dx=A, dx_ld=40, dw=A, db=A, dw_dt=F32, accumulate=0, ws=A, ws_bytes=ws)
    refuse(call, (dict(rows=-1), dict(cols=-1), dict(dt=0), dict(w_dt=F16), dict(dw_dt=0), dict(dy_ld=39), dict(x_ld=39),
                  dict(dx_ld=39), dict(res_ld=39), dict(dy=None), dict(x=None), dict(dx=None), dict(weight=None),
                  dict(mean=None), dict(rstd=None), dict(dy_ld=BIG), dict(x_ld=BIG), dict(dx_ld=BIG), dict(res_ld=BIG)),
           zdp.ERR_INVALID_ARG)
    refuse(call, (dict(dy=A + 2), dict(x=A + 2), dict(dx=A + 2), dict(res=A + 2), dict(weight=A + 2), dict(mean=A + 2),
                  dict(rstd=A + 1), dict(dw=A + 2), dict(db=A + 2), dict(dw_dt=F16, dw=A + 1)), zdp.ERR_ALIGNMENT)
    refuse(call, (dict(ws=None), dict(ws=A + 128), dict(ws_bytes=ws - 1)), zdp.ERR_WORKSPACE)
    wide = dict(cols=2 ** 20 + 1, dy_ld=2 ** 21, x_ld=2 ** 21, res_ld=2 ** 21, dx_ld=2 ** 21)
    refuse(call, (wide,), zdp.ERR_UNSUPPORTED)
    none = dict(rows=0, dy=None, x=None, dx=None, res=None, weight=None, mean=None, rstd=None)
    assert call(**none, dw=None, db=None, dw_dt=0, ws=None) == zdp.OK
    assert call(cols=0) == zdp.OK


def test_dropout_refusals(lib):
    call = caller(lib.zero_dropout, x=A, dt=F32, rows=4, cols=40, x_ld=40, res=A, res_ld=40, y=A, y_ld=40, p=0.5, seed=1,
                  offset=2, counter=A, first=3)
    refuse(call, (dict(rows=-1), dict(cols=-1), dict(dt=0), dict(dt=4), dict(x_ld=39), dict(res_ld=39), dict(y_ld=39),
                  dict(x=None), dict(y=None), dict(x_ld=BIG), dict(res_ld=BIG), dict(y_ld=BIG), dict(p=-1e-9), dict(p=1.0),
                  dict(p=1 - 2.0 ** -34), dict(p=float("nan")), dict(p=float("inf")), dict(first=-1),
                  dict(first=2 ** 63 - 160)), zdp.ERR_INVALID_ARG)
    refuse(call, (dict(x=A + 2), dict(y=A + 2), dict(res=A + 1), dict(counter=A + 4), dict(dt=BF16, x=A + 1)),
           zdp.ERR_ALIGNMENT)
    assert call(rows=0, x=None, y=None, res=None, counter=None) == zdp.OK
    assert call(cols=0, x=None, y=None, res=None, first=2 ** 63 - 1) == zdp.OK


def test_binding_refuses_host_tensors():
    x, w, v = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4)
    with pytest.raises(ValueError, match="device tensor"):
        zdp.layer_norm(x, w, w, x)
    with pytest.raises(ValueError, match="device tensor"):
        zdp.layer_norm_backward(x, x, w, v, v, x)
    with pytest.raises(ValueError, match="device tensor"):
        zdp.dropout(x, x, 0.5, 1)


@pytest.fixture
def host(monkeypatch):
    """The binding's checks on host tensors: -1 is their device, and what would be called is recorded."""
    calls = []
    monkeypatch.setattr(zdp, "_device_of", lambda t, name: -1)
    monkeypatch.setattr(zdp, "_call", lambda fn, device, stream, *args: calls.append((fn.__name__, args)))
    return calls


def refused(error, fn, *args, match=None, **kw):
    with pytest.raises(error, match=match):
        fn(*args, **kw)


def test_norm_binding_checks(host):
    x, y = torch.zeros(4, 8), torch.zeros(4, 8)
    w, v = torch.zeros(8), torch.zeros(4)
    f = zdp.layer_norm
    f(x, w, None, y)
    f(x[:, 2:5], w[:3], w[:3], y[:, 1:4], mean=v, rstd=v)
    assert [a[1][2:5] for a in host] == [(4, 8, 8), (4, 3, 8)]
    refused(ValueError, f, x, w[:7], None, y, match="weight")
    refused(ValueError, f, x, w, w[:7], y, match="bias")
    refused(TypeError, f, x, None, None, y)
    refused(TypeError, f, x, w, w.half(), y, match="bias")
    refused(TypeError, f, x, w.half(), None, y, match="weight")
    refused(TypeError, f, x.half(), w.bfloat16(), None, y.half(), match="weight")
    refused(TypeError, f, x, w, None, y.half(), match="y")
    refused(ValueError, f, x, w, None, y[:3], match="y")
    refused(ValueError, f, x.t(), w[:4], None, y.t().contiguous(), match="dense")
    refused(ValueError, f, x, w, None, y, mean=v, match="together")
    refused(ValueError, f, x, w, None, y, mean=v[:3], rstd=v, match="mean")
    refused(TypeError, f, x, w, None, y, mean=v, rstd=v.double(), match="rstd")
    refused(ValueError, f, x, w, None, y, mean=v, rstd=torch.zeros(8)[::2], match="contiguous")
    assert len(host) == 2


def test_norm_backward_binding_checks(host):
    x = torch.zeros(4, 8)
    w, v, ws = torch.zeros(8), torch.zeros(4), torch.zeros(16, dtype=torch.uint8)
    f = zdp.layer_norm_backward
    f(x, x, w, v, v, x)
    f(x, x, w, v, v, x, w.half(), w.half(), workspace=ws, dresidual=x, accumulate=True)
    f(x, x, w, v, v, x, None, w.bfloat16(), workspace=ws)
    assert len(host) == 3
    refused(ValueError, f, x, x, w, v, v, x, w, match="workspace")
    refused(TypeError, f, x, x, w, v, v, x, w, workspace=ws.float(), match="workspace")
    refused(TypeError, f, x, x, w, v, v, x, w, w.half(), workspace=ws, match="dbias")
    refused(ValueError, f, x, x, w, v, v, x, w[:7], workspace=ws, match="dweight")
    refused(TypeError, f, x, x, w, None, v, x, match="mean")
    refused(ValueError, f, x, x, w, v[:3], v, x, match="mean")
    refused(ValueError, f, x[:3], x, w, v, v, x, match="dy")
    refused(TypeError, f, x.half(), x, w, v, v, x, match="dy")
    refused(TypeError, f, x, x, w, v, v, x, dresidual=x.half(), match="dresidual")
    refused(ValueError, f, x, x, w, v, v, x[:, :7], match="dx")
    assert len(host) == 3


def test_dropout_binding_checks(host):
    x = torch.zeros(4, 8)
    f = zdp.dropout
    f(x, x, 0.5, -1, 2 ** 64 + 5)
    assert host[0][1][10:12] == (2 ** 64 - 1, 5)
    f(x.view(2, 2, 8), x.view(2, 2, 8), 0.5, 1)
    assert host[1][1][2:5] == (1, 32, 32)
    f(x[:, 1:4], x[:, 2:5], 0.5, 1, residual=x[:, :3])
    assert host[2][1][2:5] == (4, 3, 8)
    f(x, x, 0.5, 1, counter=torch.zeros(1, dtype=torch.int64))
    refused(ValueError, f, x, x[:3], 0.5, 1, match="y")
    refused(ValueError, f, x, x.view(-1), 0.5, 1, match="y")
    refused(TypeError, f, x, x.half(), 0.5, 1, match="y")
    refused(TypeError, f, x, None, 0.5, 1, match="y")
    refused(TypeError, f, x, x, 0.5, 1, residual=x.half(), match="residual")
    refused(ValueError, f, x, x, 0.5, 1, residual=x[:, :7], match="residual")
    refused(ValueError, f, x.t(), x, 0.5, 1)
    refused(ValueError, f, x.view(2, 2, 8)[:, :, :4], torch.zeros(2, 2, 4), 0.5, 1, match="contiguous")
    refused(ValueError, f, x, x, 0.5, 1, first=2 ** 64, match="first")  # would wrap to 0
    refused(ValueError, f, x, x, 0.5, 1, first=-1, match="first")
    refused(TypeError, f, x, x, 0.5, 1, counter=torch.zeros(1), match="counter")
    refused(ValueError, f, x, x, 0.5, 1, counter=torch.zeros(2, dtype=torch.int64), match="counter")
    assert len(host) == 4


def test_gated_refusals(lib):
    call = caller(lib.zero_gated_product, x=A, dt=F16, m=5, d=40, x_ld=40, wg=A, wu=A, f=7, w_ld=40, act=0, h=A, h_ld=7,
                  gate=A, up=A, pre_ld=7)
    refuse(call, (dict(m=-1), dict(d=-1), dict(f=-1), dict(dt=F32), dict(dt=0), dict(act=-1), dict(act=5), dict(x_ld=39),
                  dict(w_ld=39), dict(h_ld=6), dict(pre_ld=6), dict(x=None), dict(wg=None), dict(wu=None), dict(h=None),
                  dict(gate=None), dict(up=None), dict(x_ld=BIG), dict(w_ld=BIG), dict(h_ld=BIG), dict(pre_ld=BIG)),
           zdp.ERR_INVALID_ARG)
    refuse(call, (dict(x=A + 1), dict(wg=A + 1), dict(wu=A + 1), dict(h=A + 1), dict(gate=A + 1), dict(up=A + 1)),
           zdp.ERR_ALIGNMENT)
    refuse(call, (dict(m=2 ** 31), dict(f=2 ** 31, h_ld=2 ** 31, pre_ld=2 ** 31), dict(d=2 ** 31, x_ld=2 ** 31, w_ld=2 ** 31),
                  dict(x_ld=4_194_304), dict(w_ld=4_194_304)), zdp.ERR_UNSUPPORTED)
    assert call(m=0, x=None, h=None, gate=None, up=None) == zdp.OK
    assert call(f=0, wg=None, wu=None, h=None, gate=None, up=None) == zdp.OK


def test_gated_backward_refusals(lib):
    ws = zdp.workspace_bytes(1)
    call = caller(lib.zero_gated_product_backward, dh=A, dh_ld=7, x=A, dt=BF16, m=5, d=40, x_ld=40, wg=A, wu=A, f=7, w_ld=40,
                  act=0, gate=A, up=A, pre_ld=7, dgate=A, dup=A, dpre_ld=7, dx=A, dx_ld=40, dwg=A, dwu=A, dw_ld=40,
                  dw_dt=F32, accumulate=0, ws=A, ws_bytes=ws)
    refuse(call, (dict(m=-1), dict(d=-1), dict(f=-1), dict(dt=F32), dict(act=9), dict(dh_ld=6), dict(x_ld=39), dict(w_ld=39),
                  dict(pre_ld=6), dict(dpre_ld=6), dict(dx_ld=39), dict(dw_ld=39), dict(dw_dt=F16), dict(dw_dt=0),
                  dict(dh=None), dict(x=None), dict(wg=None), dict(wu=None), dict(gate=None), dict(up=None),
                  dict(dgate=None), dict(dup=None), dict(dwg=None), dict(dwu=None), dict(dh_ld=BIG), dict(x_ld=BIG),
                  dict(w_ld=BIG), dict(pre_ld=BIG), dict(dpre_ld=BIG), dict(dx_ld=BIG), dict(dw_ld=BIG)),
           zdp.ERR_INVALID_ARG)
    refuse(call, (dict(dh=A + 1), dict(x=A + 1), dict(wg=A + 1), dict(wu=A + 1), dict(gate=A + 1), dict(up=A + 1),
                  dict(dgate=A + 1), dict(dup=A + 1), dict(dx=A + 1), dict(dwg=A + 2), dict(dwu=A + 2)), zdp.ERR_ALIGNMENT)
    refuse(call, (dict(ws=None), dict(ws=A + 128), dict(ws_bytes=ws - 1)), zdp.ERR_WORKSPACE)
    refuse(call, (dict(m=2 ** 31), dict(x_ld=4_194_304), dict(w_ld=4_194_304), dict(dpre_ld=4_194_304)),
           zdp.ERR_UNSUPPORTED)


def test_gated_binding_checks(host):
    def h16(*s):
        return torch.zeros(*s, dtype=torch.float16)
    x, w, h = h16(5, 8), h16(7, 8), h16(5, 7)
    f = zdp.gated_product
    f(x, w, w, h)
    f(x, w, w, h, "relu", gate=h, up=h)
    f(x[:, 1:4], w[:, :3], w[:, 2:5], h, "sigmoid")
    assert [a[1][9] for a in host] == [0, 3, 4] and host[2][1][4] == 8
    refused(ValueError, f, x, w, w, h, "tanh", match="act")
    refused(TypeError, f, x.float(), w.float(), w.float(), h.float(), match="x")
    refused(TypeError, f, x, w.bfloat16(), w, h, match="w_gate")
    refused(TypeError, f, x, w, w.bfloat16(), h, match="w_up")
    refused(ValueError, f, x, w, w[:6], h, match="w_up")
    refused(ValueError, f, x, w[:, :7], w[:, :7], h, match="w_gate")
    refused(ValueError, f, x, w, h16(7, 9)[:, :8], h, match="elements apart")
    refused(ValueError, f, x, w, w, h[:4], match="out")
    refused(ValueError, f, x, w, w, h, gate=h, match="together")
    refused(ValueError, f, x, w, w, h, gate=h, up=h16(5, 8)[:, :7], match="elements apart")
    refused(ValueError, f, x, w, w, h.t(), match="out")
    assert len(host) == 3


def test_gated_backward_binding_checks(host):
    def h16(*s):
        return torch.zeros(*s, dtype=torch.float16)
    x, w, h, ws = h16(5, 8), h16(7, 8), h16(5, 7), torch.zeros(16, dtype=torch.uint8)
    f = zdp.gated_product_backward
    f(h, x, w, w, h, h, h, h, ws)
    f(h, x, w, w, h, h, h, h, ws, dx=x, dw_gate=w.float(), dw_up=w.float(), act="gelu", accumulate=True)
    assert host[1][1][24] is True and host[1][1][23] == F32
    refused(ValueError, f, h, x, w, w, h, h, h, h, None, match="workspace")
    refused(ValueError, f, h, x, w, w, h, h, h, h, ws, dw_gate=w, match="together")
    refused(TypeError, f, h, x, w, w, h, h, h, h, ws, dw_gate=w.bfloat16(), dw_up=w.bfloat16(), match="dw_gate")
    refused(TypeError, f, h, x, w, w, h, h, h, h, ws, dw_gate=w, dw_up=w.float(), match="dw_up")
    refused(ValueError, f, h, x, w, w, h, h, h, h, ws, dw_gate=w, dw_up=w[:6], match="dw_up")
    refused(ValueError, f, h, x, w, w, h, h, h, h, ws, dx=h, match="dx")
    refused(ValueError, f, h[:4], x, w, w, h, h, h, h, ws, match="dout")
    refused(ValueError, f, h, x, w, w, h, h[:, :6], h, h, ws, match="up")
    refused(ValueError, f, h, x, w, w, h, h, h, h16(5, 8)[:, 1:], ws, match="elements apart")
    refused(ValueError, f, h, x, w, w, h, h, h, h, ws, act="swish", match="act")
    assert len(host) == 2


def test_the_binding_passes_what_the_library_takes(lib):
    """Each call's arguments, counted: the binding gives as many as the entry point has."""
    for name in ("layer_norm", "layer_norm_backward", "dropout", "gated_product", "gated_product_backward"):
        assert "stream" in inspect.signature(getattr(zdp, name)).parameters
        assert getattr(lib, f"zero_{name}").argtypes


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def test_the_generator_gives_the_published_words():
    """The known answers that its authors publish for Philox4x32-10: all zeros, all ones, and digits of pi."""
    ones = 0xFFFFFFFF
    c = [[0] * 4, [ones] * 4, [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]]
    k = [(0, 0), (ones, ones), (0xA4093822, 0x299F31D0)]
    want = [[0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8], [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD],
            [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]]
    for ci, ki, wi in zip(c, k, want):
        assert _layer.philox(np.array([ci], np.uint64), ki)[0].tolist() == wi


def test_kept_is_the_same_from_any_start():
    whole = _layer.kept(1000, 0.3, 5, 6, 2 ** 34 + 1)
    for a in (1, 2, 3, 4, 501):
        assert (_layer.kept(1000 - a, 0.3, 5, 6, 2 ** 34 + 1 + a) == whole[a:]).all()


def test_the_norm_s_gradient_is_its_slope():
    g = np.random.default_rng(0)
    x, w, b, dy = g.normal(size=(3, 11)), g.normal(size=11), g.normal(size=11), g.normal(size=(3, 11))
    _, mean, rstd = _layer.norm(x, w, b, 1e-5)
    dx, dw, db = _layer.norm_grad(dy, x, w, mean, rstd)
    e, h = [g.normal(size=t.shape) for t in (x, w, b)], 1e-5
    up, down = (_layer.norm(x + s * h * e[0], w + s * h * e[1], b + s * h * e[2], 1e-5)[0] for s in (1, -1))
    slope = ((up - down) / (2 * h) * dy).sum()
    assert abs((dx * e[0]).sum() + (dw * e[1]).sum() + (db * e[2]).sum() - slope) < 1e-7


def test_the_pieces_that_both_products_keep_are_the_same():
    """gated_product.hip and mx_product.hip each deal tiles to the XCDs and fetch to LDS in asm of their own: a change to
    one is a change to both, but for the operands' type."""
    def pieces(name):
        with open(os.path.join(build.CSRC, name)) as f:
            text = f.read()
        deal = re.search(r"void tile_of\([^{]*\{\n(.*?)^\}", text, re.S | re.M)[1]
        fetch = re.search(r"void fetch_to_lds_if\([^{]*\{\n(.*?)^\}", text, re.S | re.M)[1]
        grant = re.search(r"  int dev = 0;\n(.*?granted\.fetch_or[^\n]*\n  \}\n)", text, re.S)[1]
        return deal, fetch, grant
    for mine, other in zip(pieces("gated_product.hip"), pieces("mx_product.hip")):
        assert mine == other
