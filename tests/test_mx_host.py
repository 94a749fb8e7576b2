"""The microscaled 4-bit calls without a GPU: their argument checks (in the
library and in the binding) fire before anything touches a device, and the
plain numpy form the GPU tests compare with has the format's properties."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import _mx
import zero_dp_partitioned_amd as zdp
from zero_dp_partitioned_amd import build

A = 1 << 20  # an aligned address that is never read: the checks come first
BIG = 2 ** 62


@pytest.fixture(scope="module")
def lib():
    return zdp.load()


def _quantize(lib, src=A, dt=zdp.DT_F32, rows=4, cols=40, src_ld=40, codes=A, scales=A, ld=2, codes_t=A, scales_t=A,
              ld_t=1):
    return lib.zero_mx_quantize(src, dt, rows, cols, src_ld, codes, scales, ld, codes_t, scales_t, ld_t, None)


@pytest.mark.parametrize("kw, rc", [
    (dict(rows=-1), zdp.ERR_INVALID_ARG), (dict(cols=-1, src_ld=1), zdp.ERR_INVALID_ARG),
    (dict(dt=0), zdp.ERR_INVALID_ARG), (dict(dt=4), zdp.ERR_INVALID_ARG),
    (dict(src_ld=39), zdp.ERR_INVALID_ARG), (dict(src=None), zdp.ERR_INVALID_ARG),
    (dict(src=A + 2), zdp.ERR_ALIGNMENT), (dict(src=A + 1, dt=zdp.DT_BF16), zdp.ERR_ALIGNMENT),
    (dict(codes=None), zdp.ERR_INVALID_ARG), (dict(scales_t=None), zdp.ERR_INVALID_ARG),
    (dict(codes=None, scales=None, codes_t=None, scales_t=None), zdp.ERR_INVALID_ARG),
    (dict(ld=1), zdp.ERR_INVALID_ARG), (dict(ld_t=0), zdp.ERR_INVALID_ARG),
    (dict(codes=A + 8), zdp.ERR_ALIGNMENT), (dict(codes_t=A + 1), zdp.ERR_ALIGNMENT),
    (dict(src_ld=BIG), zdp.ERR_INVALID_ARG), (dict(ld=BIG), zdp.ERR_INVALID_ARG), (dict(ld_t=BIG), zdp.ERR_INVALID_ARG),
])
def test_quantize_refusals(lib, kw, rc):
    assert _quantize(lib, **kw) == rc
    assert zdp.last_error()


@pytest.mark.parametrize("rows, cols", [(0, 5), (5, 0), (0, 0)])
def test_empty_quantize_is_ok(lib, rows, cols):
    assert _quantize(lib, src=None, rows=rows, cols=cols) == zdp.OK


def test_writeback_refusals(lib):
    f = lib.zero_mx_cast_writeback
    assert f(A, -1, A, A, 0, None) == zdp.ERR_INVALID_ARG
    assert f(A, 8, A, A, -32, None) == zdp.ERR_INVALID_ARG
    assert f(A, 8, A, A, 33, None) == zdp.ERR_INVALID_ARG
    assert f(None, 8, A, A, 0, None) == zdp.ERR_INVALID_ARG
    assert f(A, 8, None, A, 32, None) == zdp.ERR_INVALID_ARG
    assert f(A, 8, A, None, 32, None) == zdp.ERR_INVALID_ARG
    assert f(A + 2, 8, A, A, 0, None) == zdp.ERR_ALIGNMENT
    assert f(A, 8, A + 4, A, 0, None) == zdp.ERR_ALIGNMENT
    assert f(None, 0, None, None, 64, None) == zdp.OK


def test_dequantize_refusals(lib):
    f = lib.zero_mx_dequantize
    ok = dict(codes=A, scales=A, rows=4, cols=40, ld=2, out=A, dt=zdp.DT_F16, out_ld=40)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["codes"], a["scales"], a["rows"], a["cols"], a["ld"], a["out"], a["dt"], a["out_ld"], None)

    for kw in (dict(rows=-1), dict(cols=-1), dict(ld=1), dict(out_ld=39), dict(dt=9), dict(codes=None),
               dict(scales=None), dict(out=None), dict(ld=BIG), dict(out_ld=BIG)):
        assert call(**kw) == zdp.ERR_INVALID_ARG, kw
    assert call(codes=A + 8) == zdp.ERR_ALIGNMENT
    assert call(out=A + 1) == zdp.ERR_ALIGNMENT
    assert call(rows=0, codes=None, scales=None, out=None) == zdp.OK


def _ptrs(*values):
    return (ctypes.c_void_p * len(values))(*values)


def test_reduce_refusals(lib):
    f = lib.zero_mx_reduce_grad_segment
    ws = zdp.workspace_bytes(1)

    def call(codes=_ptrs(A, A), scales=_ptrs(A, A), n_d=2, n=100, avg=A, w=A, wb=ws, group=0, state=A):
        return f(codes, scales, n_d, n, avg, w, wb, group, state, None)

    assert call(n=-1) == zdp.ERR_INVALID_ARG
    assert call(avg=None) == zdp.ERR_INVALID_ARG
    assert call(avg=A + 2) == zdp.ERR_ALIGNMENT
    assert call(state=None) == zdp.ERR_INVALID_ARG
    assert call(w=None) == zdp.ERR_WORKSPACE
    assert call(wb=ws - 1) == zdp.ERR_WORKSPACE
    assert call(w=A + 128) == zdp.ERR_WORKSPACE
    assert call(group=zdp.MAX_GROUPS) == zdp.ERR_WORKSPACE
    assert call(codes=None) == zdp.ERR_INVALID_ARG
    assert call(n_d=0) == zdp.ERR_INVALID_ARG
    assert call(n_d=zdp.MAX_REPLICAS + 1) == zdp.ERR_UNSUPPORTED
    assert call(codes=_ptrs(A, None)) == zdp.ERR_INVALID_ARG
    assert call(scales=_ptrs(None, A)) == zdp.ERR_INVALID_ARG
    assert call(codes=_ptrs(A, A + 8)) == zdp.ERR_ALIGNMENT
    even = [A + 64 * r for r in range(65)]
    odd = even[:64] + [A]
    assert call(codes=_ptrs(*odd), scales=_ptrs(*even), n_d=65) == zdp.ERR_UNSUPPORTED
    assert call(codes=_ptrs(*even), scales=_ptrs(*odd), n_d=65) == zdp.ERR_UNSUPPORTED


def test_product_refusals(lib):
    f = lib.zero_mx_product
    ok = dict(a=A, sa=A, lda=3, b=A, sb=A, ldb=3, m=5, n=7, kb=3, out=A, dt=zdp.DT_F32, ldo=7)

    def call(**kw):
        a = {**ok, **kw}
        return f(a["a"], a["sa"], a["lda"], a["b"], a["sb"], a["ldb"], a["m"], a["n"], a["kb"], a["out"], a["dt"],
                 a["ldo"], None)

    for kw in (dict(m=-1), dict(n=-1), dict(kb=-1), dict(lda=2), dict(ldb=2), dict(ldo=6), dict(dt=0), dict(a=None),
               dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(lda=BIG), dict(ldb=BIG),
               dict(ldo=BIG)):
        assert call(**kw) == zdp.ERR_INVALID_ARG, kw
    for kw in (dict(a=A + 8), dict(b=A + 4), dict(out=A + 2), dict(out=A + 1, dt=zdp.DT_F16)):
        assert call(**kw) == zdp.ERR_ALIGNMENT, kw
    assert call(m=2 ** 31) == zdp.ERR_UNSUPPORTED
    assert call(n=2 ** 31, ldo=2 ** 31) == zdp.ERR_UNSUPPORTED
    assert call(lda=2 ** 20) == zdp.ERR_UNSUPPORTED
    assert call(ldb=2 ** 20) == zdp.ERR_UNSUPPORTED
    assert call(m=0, a=None, sa=None, out=None) == zdp.OK


def _mx_tensors(rows, kb):
    return torch.zeros(rows, 16 * kb, dtype=torch.uint8), torch.zeros(rows, kb, dtype=torch.uint8)


def test_binding_refuses_host_tensors():
    c, s = _mx_tensors(4, 2)
    x = torch.zeros(4, 40)
    with pytest.raises(ValueError):
        zdp.mx_quantize(x, c, s)
    with pytest.raises(ValueError):
        zdp.mx_dequantize(c, s, x)
    with pytest.raises(ValueError):
        zdp.mx_product(c, s, c, s, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        zdp.mx_cast_writeback(torch.zeros(8), c.view(-1), s.view(-1))


def test_binding_row_checks():
    dev = -1  # the host
    f = zdp._need_rows
    x = torch.zeros(6, 10)
    types = zdp._mx_types()
    assert f(x, "x", types, dev) == (6, 10, 10)
    assert f(x[:, 2:7], "x", types, dev) == (6, 5, 10)
    assert f(x[1:2], "x", types, dev) == (1, 10, 10)
    with pytest.raises(ValueError, match="expected device 0"):
        f(x, "x", types, 0)
    with pytest.raises(ValueError, match="not dense"):
        f(x.t(), "x", types, dev)
    with pytest.raises(ValueError, match="overlap"):
        f(x[:1].expand(6, 10), "x", types, dev)
    with pytest.raises(TypeError):
        f(x.double(), "x", types, dev)
    with pytest.raises(TypeError):
        f([1], "x", types, dev)
    with pytest.raises(ValueError, match="dimensions"):
        f(x[0], "x", types, dev)


def test_binding_matrix_checks():
    dev = -1
    c, s = _mx_tensors(6, 4)
    f = zdp._need_mx
    assert f(c, s, "A", dev, 6, 97) == (6, 4, 4)
    assert f(c[:, 16:48], s[:, 1:3], "A", dev, 6, 64) == (6, 2, 4)
    with pytest.raises(ValueError, match="blocks a row"):
        f(c, s, "A", dev, 6, 96)
    with pytest.raises(ValueError, match="rows"):
        f(c, s, "A", dev, 5)
    with pytest.raises(ValueError, match="do not match"):
        f(c[:, :48], s, "A", dev)
    with pytest.raises(ValueError, match="16 to 1"):
        f(c[:, 16:48], s[:, 1:3].contiguous(), "A", dev)
    with pytest.raises(TypeError):
        f(c.to(torch.int8), s, "A", dev)


def test_binding_flat_checks():
    dev = -1
    c, s = torch.zeros(16 * 5, dtype=torch.uint8), torch.zeros(5, dtype=torch.uint8)
    f = zdp._need_flat
    assert f(c, s, "v", dev, 64, 96) == (5, 5)
    assert f(c, s, "v", dev, 64, 70) == (5, 5)
    for offset, n in ((64, 97), (32 * 5, 1), (33, 1), (-32, 32)):
        with pytest.raises(ValueError):
            f(c, s, "v", dev, offset, n)
    with pytest.raises(ValueError):
        f(c[:-1], s, "v", dev, 64, 96)


def test_view_of_a_tensor_in_a_flat_vector():
    c, s = torch.arange(16 * 12, dtype=torch.uint8), torch.arange(12, dtype=torch.uint8)
    vc, vs = zdp.mx_view(c, s, 64, 3, 96)
    assert vc.shape == (3, 48) and vs.shape == (3, 3)
    assert vc.data_ptr() == c.data_ptr() + 32 and vs.data_ptr() == s.data_ptr() + 2
    for bad in ((33, 3, 96), (64, 3, 95), (64, 4, 96), (-32, 1, 32)):
        with pytest.raises(ValueError):
            zdp.mx_view(c, s, *bad)


@pytest.mark.parametrize("bad", [(0, -1, 32), (64, -2, 96), (0, 1, -32), (64, -1, -32)])
def test_view_of_fewer_than_no_values_is_refused(bad):
    """Slices with a negative end would silently be the vector without its last blocks."""
    c, s = torch.zeros(16 * 12, dtype=torch.uint8), torch.zeros(12, dtype=torch.uint8)
    with pytest.raises(ValueError):
        zdp.mx_view(c, s, *bad)


def test_the_plain_form_is_the_nearest_code():
    """Brute force: every code's value against the plain form's choice."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=(50, 64)) * np.exp2(rng.integers(-20, 20, (50, 1)))
    x[3, 5:20] = [k / 8 for k in range(15)]
    codes, scales = _mx.quantize(x)
    v = _mx.decode(codes, scales)
    s = np.ldexp(1.0, scales.astype(int) - 127).repeat(32, 1)
    best = np.min(np.abs(np.abs(x)[..., None] - _mx.GRID * s[..., None]), -1)
    np.testing.assert_array_equal(np.abs(np.abs(x) - np.abs(v)), best)
    assert (np.abs(x).reshape(50, 2, 32).max(-1) / np.ldexp(1.0, scales.astype(int) - 127) < 8).all()
    assert (np.abs(x).reshape(50, 2, 32).max(-1) / np.ldexp(1.0, scales.astype(int) - 127) >= 4).all()


def test_the_plain_form_at_the_edges():
    x = np.zeros((6, 32))
    x[1, 3] = 2.0 ** -149
    x[2, 0], x[2, 1] = np.finfo(np.float32).max, -1.0
    x[3, 7] = np.nan
    x[4, 0] = -np.inf
    x[5, :8] = [5.0, 2.5, 3.5, 0.25, 0.75, 1.25, 1.75, -7.9]
    codes, scales = _mx.quantize(x)
    assert scales[:, 0].tolist() == [0, 0, 252, 255, 255, 127]
    assert not codes[0].any() and not codes[1].any() and not codes[3].any() and not codes[4].any()
    v = _mx.decode(codes, scales)
    assert v[2, 0] == 6 * 2.0 ** 125 and np.isnan(v[3]).all() and np.isnan(v[4]).all()
    assert v[5, :8].tolist() == [4.0, 2.0, 4.0, 0.0, 1.0, 1.0, 2.0, -6.0]


def test_a_matrix_is_no_flat_vector():
    """The rows of a 32 x 40 matrix are padded to whole blocks: read as a vector, the padding would be values."""
    dev = -1
    c, s = _mx_tensors(32, 2)
    f = zdp._need_flat
    for codes, scales in ((c, s), (c.view(-1), s), (c, s.view(-1)), (c.view(4, 8, 32), s.view(-1))):
        with pytest.raises(ValueError, match="dimensions"):
            f(codes, scales, "v", dev, 0, 1280)
    assert f(c.view(-1), s.view(-1), "v", dev, 0, 1280) == (40, 64)
    with pytest.raises(ValueError, match="dimensions"):
        f(torch.tensor(0, dtype=torch.uint8), s.view(-1), "v", dev, 0, 0)


def _functions(path):
    """{name: text} of the functions of a source file that begin in the first column."""
    with open(path) as f:
        text = f.read()
    return {m[2]: m[0] for m in re.finditer(r"^(template <[^\n]*>\n)?\w[^\n;]*?\b(\w+)\([^;{]*\{\n.*?^\}", text, re.S | re.M)}


def test_the_pieces_kept_twice_are_the_same():
    """mx_device.h repeats what kernels.hip keeps to itself (encodings, norm partials): a change to one is a change to
    both, or the 4-bit average's norm and flag are no longer those of the 16-bit one."""
    mine, steps = (_functions(os.path.join(build.CSRC, f)) for f in ("mx_device.h", "kernels.hip"))
    both = set(mine) & set(steps)
    assert both >= {"ld_stream", "st_stream", "decode16", "encode16", "account", "write_block_partial", "route_partials"}
    for name in sorted(both):
        assert mine[name] == steps[name], f"{name} differs between mx_device.h and kernels.hip"


def test_the_binding_does_without_torch_s_private_names(monkeypatch):
    """The 4-bit calls find the current device and stream through torch's public calls where it lacks the faster ones."""
    class Stream:
        def __init__(self, device):
            self.cuda_stream = 70 + device

    for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
        monkeypatch.delattr(torch._C, name)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    types = zdp._MxTypes()
    assert types.stream(2) == 72 and types.device() == 3


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """A launch goes to its stream's device, where the tensors' memory need not be mapped."""
    class Stream:
        def __init__(self, device):
            self.device_index, self.cuda_stream = device, 7

    calls = []
    monkeypatch.setattr(zdp._mx(), "device", lambda: 0)
    with pytest.raises(ValueError, match="device 1"):
        zdp._call(lambda *a: calls.append(a) or zdp.OK, 0, Stream(1), 3)
    assert not calls
    zdp._call(lambda *a: calls.append(a) or zdp.OK, 0, Stream(0), 3)
    assert calls == [(3, 7)]
