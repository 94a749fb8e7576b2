"""A layer's operators together, as a training step uses them: a residual sublayer
x + dropout(act(norm(x) wg^T) * (norm(x) wu^T)) whose weights are tensors of the
flat 16-bit vector and whose gradients go into the gradient copy of it that
zero_adam_step reads. Also in graphs, on several streams, and at offsets past 32 bits."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _layer
import zero_dp_partitioned_amd as zdp
from _gpu_helpers import DEV

pytestmark = pytest.mark.gpu

M, D = 200, 136  # the block's width is its input's, so that the sum with x needs no product more
SCALE = 64.0     # loss scale
SEED = 12345
ACT = "silu"


class Sublayer:
    """Weights in a flat fp16 vector, gradients in a copy of it, the step's state, and the activations."""

    def __init__(self, seed):
        g = torch.Generator(device=DEV).manual_seed(seed)
        shapes = {"nw": (D,), "nb": (D,), "wg": (D, D), "wu": (D, D)}
        n = sum(int(np.prod(s)) for s in shapes.values())
        self.flat = (torch.randn(n, generator=g, device=DEV) * 0.1).half()
        self.grad = torch.zeros_like(self.flat)
        self.p, self.g, at = {}, {}, 0
        for name, s in shapes.items():
            k = int(np.prod(s))
            self.p[name], self.g[name] = self.flat[at:at + k].view(s), self.grad[at:at + k].view(s)
            at += k
        self.p["nw"] += 1
        self.master = self.flat.float()
        self.m, self.v = torch.zeros_like(self.master), torch.zeros_like(self.master)
        self.state, self.ws = zdp.new_state(SCALE), zdp.new_workspace(1)
        self.group = zdp.Group(self.master, self.m, self.v, replicas=[self.grad], flat_param=self.flat, lr=1e-2)
        self.x = (torch.randn(M, D, generator=g, device=DEV)).half()
        self.dy = (torch.randn(M, D, generator=g, device=DEV) * SCALE * 0.01).half()
        self.counter = torch.zeros(1, dtype=torch.int64, device=DEV)
        self.norm, self.h, self.gate, self.up, self.y, self.dh, self.dn, self.dx = (torch.empty_like(self.x) for _ in range(8))
        self.mean, self.rstd = torch.empty(M, device=DEV), torch.empty(M, device=DEV)

    def forward(self):
        p = self.p
        zdp.layer_norm(self.x, p["nw"], p["nb"], self.norm, mean=self.mean, rstd=self.rstd)
        zdp.gated_product(self.norm, p["wg"], p["wu"], self.h, ACT, gate=self.gate, up=self.up)
        zdp.dropout(self.h, self.y, 0.2, SEED, residual=self.x, counter=self.counter)

    def backward(self):
        p, g = self.p, self.g
        zdp.dropout(self.dy, self.dh, 0.2, SEED, counter=self.counter)
        zdp.gated_product_backward(self.dh, self.norm, p["wg"], p["wu"], self.gate, self.up, self.gate, self.up, self.ws,
                                   dx=self.dn, dw_gate=g["wg"], dw_up=g["wu"], act=ACT)
        zdp.layer_norm_backward(self.dn, self.x, p["nw"], self.mean, self.rstd, self.dx, g["nw"], g["nb"],
                                workspace=self.ws, dresidual=self.dy)

    def step(self):
        self.forward()
        self.backward()
        zdp.adam_step([self.group], self.ws, self.state)
        self.counter += 1

    def held(self):
        return [self.y, self.dx, self.grad, self.flat, self.master, self.m, self.v, self.state, self.counter]


def exact(s, offset):
    """y, dx and the flat gradient in 64 bits, from the weights as they are (numpy)."""
    p = {k: v.double().cpu().numpy() for k, v in s.p.items()}
    x, dy = s.x.double().cpu().numpy(), s.dy.double().cpu().numpy()
    n, mean, rstd = _layer.norm(x, p["nw"], p["nb"], 1e-5)
    gate, up = n @ p["wg"].T, n @ p["wu"].T
    sig = 1 / (1 + np.exp(-gate))
    keep = _layer.kept(M * D, 0.2, SEED, offset).reshape(M, D) / 0.8
    y = x + keep * gate * sig * up
    dh = dy * keep
    dg, du = dh * up * (sig + gate * sig * (1 - sig)), dh * gate * sig
    dn = dg @ p["wg"] + du @ p["wu"]
    dx, dnw, dnb = _layer.norm_grad(dn, x, p["nw"], mean, rstd, dy)
    return y, dx, np.concatenate([dnw, dnb, (dg.T @ n).ravel(), (du.T @ n).ravel()])


def test_training_steps():
    """Three steps. On the way from x to a gradient at most eight tensors are rounded to fp16, each by at most 2^-11
    of its values; none of the functions between them magnifies a relative error more than twice in the 2-norm here,
    so the results are held to 16 * 2^-11 in the 2-norm (a wrong mask, sign or term is far outside)."""
    s = Sublayer(1)
    for k in range(3):
        s.forward()
        s.backward()
        y, dx, grad = exact(s, k)
        for got, want, what in ((s.y, y, "y"), (s.dx, dx, "dx"), (s.grad, grad, "gradient")):
            got = got.double().cpu().numpy()
            off = np.linalg.norm(got - want) / np.linalg.norm(want)
            assert off <= 16 * 2.0 ** -11, f"step {k}: {what} off by {off}"
        before = s.flat.clone()
        zdp.adam_step([s.group], s.ws, s.state)
        s.counter += 1
        st = zdp.read_state(s.state)
        assert st["step"] == k + 1 and not st["overflow"]
        norm = np.linalg.norm(s.grad.double().cpu().numpy()) / SCALE
        assert abs(st["grad_norm"] - norm) <= 1e-6 * norm  # the step read the gradients that the operators wrote
        assert not torch.equal(before, s.flat) and torch.equal(s.flat, s.master.half())


def test_overflow_reaches_the_step():
    """A gradient past fp16's range sets the step's flag."""
    s = Sublayer(2)
    s.dy.fill_(60000.0)
    s.step()
    st = zdp.read_state(s.state)
    assert st["overflow"] == 1


def test_steps_in_a_graph():
    """Captured steps, replayed with eager work between the replays, give the eager steps' bits."""
    a, b = Sublayer(3), Sublayer(3)
    a.step()
    b.step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.step()
    for k in range(4):
        b.step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(a.held(), b.held())):
            assert torch.equal(p, q), f"replay {k}: buffer {i} differs from the eager step"


def test_two_graphs_and_two_streams():
    """Independent sublayers, each with its own workspace, at once: captured in two graphs, and eager on two streams."""
    pairs = [(Sublayer(k), Sublayer(k)) for k in (4, 5)]
    streams, graphs = [torch.cuda.Stream() for _ in pairs], []
    for a, b in pairs:
        a.step()
        b.step()
    for (a, _), s in zip(pairs, streams):
        s.wait_stream(torch.cuda.current_stream())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            a.step()
    for k in range(3):
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (_, b), s in zip(pairs, streams):
            with torch.cuda.stream(s):
                b.step()
        torch.cuda.synchronize()
        for a, b in pairs:
            assert all(torch.equal(p, q) for p, q in zip(a.held(), b.held())), k


def test_a_named_stream():
    s, want = Sublayer(6), Sublayer(6)
    want.forward()
    torch.cuda.synchronize()
    side, p = torch.cuda.Stream(), s.p
    zdp.layer_norm(s.x, p["nw"], p["nb"], s.norm, mean=s.mean, rstd=s.rstd, stream=side)
    zdp.gated_product(s.norm, p["wg"], p["wu"], s.h, ACT, gate=s.gate, up=s.up, stream=side)
    zdp.dropout(s.h, s.y, 0.2, SEED, residual=s.x, stream=side)
    side.synchronize()
    assert torch.equal(s.y, want.y)


def test_first_calls_of_a_process_are_captured():
    """Every variant, in a process where no call came before the capture."""
    script = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_layer_first_capture.py")
    r = subprocess.run([sys.executable, script], capture_output=True, text=True, timeout=110)
    assert r.returncode == 0 and "first calls captured: ok" in r.stdout, r.stdout[-1000:] + r.stderr[-3000:]


# --------------------------------------------------------------------------
# offsets past 32 bits
# --------------------------------------------------------------------------

def test_dropout_past_2_to_the_32_elements():
    n, tail = 2 ** 32 + 4099, 4096 + 1003
    x = torch.ones(n, dtype=torch.bfloat16, device=DEV)
    zdp.dropout(x, x, 0.5, 9, 1)
    mask = torch.from_numpy(_layer.kept(tail, 0.5, 9, 1, n - tail)).to(DEV)
    assert torch.equal(x[n - tail:] != 0, mask)
    assert torch.equal(x[:4096] != 0, torch.from_numpy(_layer.kept(4096, 0.5, 9, 1)).to(DEV))


def test_rows_far_apart():
    """Three rows, more than 2^31 elements from one to the next, against the same rows side by side."""
    rows, cols, ld = 3, 1000, 2 ** 31 + 24
    big = torch.zeros(2 * ld + cols, dtype=torch.bfloat16, device=DEV)
    far = big.as_strided((rows, cols), (ld, 1))
    g = torch.Generator(device=DEV).manual_seed(1)
    x, dy, w = (torch.randn(*s, generator=g, device=DEV).bfloat16() for s in ((rows, cols), (rows, cols), (cols,)))
    mean, rstd, ws = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV), zdp.new_workspace(1)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    zdp.layer_norm(x, w, w, y, mean=mean, rstd=rstd)
    far.copy_(x)
    zdp.layer_norm(far, w, w, dx)
    assert torch.equal(dx, y)
    zdp.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, workspace=ws)
    got, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    zdp.layer_norm_backward(dy, far, w, mean, rstd, got, dw2, db2, workspace=ws)
    assert torch.equal(got, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    zdp.layer_norm_backward(dy, x, w, mean, rstd, far, dw2, db2, workspace=ws)
    assert torch.equal(far, dx)
    zdp.dropout(x, y, 0.5, 1)
    zdp.dropout(x, far, 0.5, 1)
    assert torch.equal(far, y)
    wg, wu = (torch.randn(cols, 64, generator=g, device=DEV).bfloat16() for _ in range(2))
    t = x[:, :64].contiguous()
    zdp.gated_product(t, wg, wu, y)
    zdp.gated_product(t, wg, wu, far)  # outputs may lie any distance apart
    assert torch.equal(far, y)


@pytest.mark.parametrize("ld", [4_194_296, 4_194_303])
def test_operands_whose_rows_lie_as_far_apart_as_they_may(ld):
    """600 rows, 2.5e9 elements from the first to the last: tiles start past 2^32 bytes, and rows of a tile lie 2^31 apart."""
    m, d, f = 600, 200, 300
    g = torch.Generator(device=DEV).manual_seed(2)
    x, wg, wu, dh, gate = (torch.randn(*s, generator=g, device=DEV).half() for s in ((m, d), (f, d), (f, d), (m, f), (m, f)))
    big = torch.zeros((m - 1) * ld + f, dtype=x.dtype, device=DEV)
    ws = zdp.new_workspace(1)

    def run(x, wg, wu, dg, du):
        h, dx = torch.empty(m, f, dtype=x.dtype, device=DEV), torch.empty(m, d, dtype=x.dtype, device=DEV)
        a, b = torch.empty(f, d, device=DEV), torch.empty(f, d, device=DEV)
        zdp.gated_product(x, wg, wu, h)
        zdp.gated_product_backward(dh, x, wg, wu, gate, gate, dg, du, ws, dx=dx, dw_gate=a, dw_up=b)
        return h, dx, a, b
    near = run(x, wg, wu, torch.empty_like(dh), torch.empty_like(dh))
    far = big.as_strided((m, d), (ld, 1))
    far.copy_(x)
    assert all(torch.equal(p, q) for p, q in zip(near, run(far, wg, wu, torch.empty_like(dh), torch.empty_like(dh))))
    both = big.as_strided((f, d), (ld, 1)), big[1_000:].as_strided((f, d), (ld, 1))
    for t, w in zip(both, (wg, wu)):
        t.copy_(w)
    assert all(torch.equal(p, q) for p, q in zip(near, run(x, *both, torch.empty_like(dh), torch.empty_like(dh))))
    dg, du = big.as_strided((m, f), (ld, 1)), torch.zeros_like(big).as_strided((m, f), (ld, 1))
    assert all(torch.equal(p, q) for p, q in zip(near, run(x, wg, wu, dg, du)))


def test_a_large_tile_s_rows_as_far_apart_as_they_may():
    """256 rows of a tile, 2^31 bytes from the first to the last, in the forward pass and in dx."""
    m, d, f, ld = 2560, 72, 2048, 4_194_296
    g = torch.Generator(device=DEV).manual_seed(2)
    x, wg, wu = (torch.randn(*s, generator=g, device=DEV).half() for s in ((m, d), (f, d), (f, d)))
    big = torch.zeros((m - 1) * ld + m, dtype=x.dtype, device=DEV)
    near, far = torch.empty(m, f, dtype=x.dtype, device=DEV), torch.empty(m, f, dtype=x.dtype, device=DEV)
    zdp.gated_product(x, wg, wu, near)
    spread = big.as_strided((m, d), (ld, 1))
    spread.copy_(x)
    zdp.gated_product(spread, wg, wu, far)
    assert torch.equal(near, far)
    # dx of 2560 x 2560 from dgate and dup with 72 columns, far apart
    dh, gate = (torch.randn(m, d, generator=g, device=DEV).half() for _ in range(2))
    w = torch.randn(d, m, generator=g, device=DEV).half()
    xx, ws = torch.zeros(m, m, dtype=x.dtype, device=DEV), zdp.new_workspace(1)
    a, b = torch.empty_like(xx), torch.empty_like(xx)
    zdp.gated_product_backward(dh, xx, w, w, gate, gate, torch.empty_like(dh), torch.empty_like(dh), ws, dx=a)
    du = torch.zeros_like(big).as_strided((m, d), (ld, 1))
    zdp.gated_product_backward(dh, xx, w, w, gate, gate, spread, du, ws, dx=b)
    assert torch.equal(a, b)


def test_refusals_on_the_device():
    x, w, v = torch.zeros(4, 64, device=DEV).half(), torch.zeros(8, 64, device=DEV).half(), torch.zeros(64, device=DEV)
    h, ws = torch.zeros(4, 8, device=DEV).half(), zdp.new_workspace(1)
    with pytest.raises(ValueError):
        zdp.layer_norm(x, v.cpu(), None, x)
    with pytest.raises(ValueError):
        zdp.dropout(x, x.cpu(), 0.5, 1)
    with pytest.raises(zdp.ZeroError):
        zdp.dropout(x, x, 1.0, 1)
    with pytest.raises(zdp.ZeroError):
        zdp.layer_norm(x, v, None, x, eps=-1.0)
    with pytest.raises(ValueError):
        zdp.gated_product(x, w, w[:7], h)
    with pytest.raises(zdp.ZeroError) as e:  # a workspace too small
        zdp.gated_product_backward(h, x, w, w, h, h, h.clone(), h.clone(), ws[:1 << 20], dx=x.clone())
    assert e.value.code == zdp.ERR_WORKSPACE
    with pytest.raises(zdp.ZeroError) as e:  # rows too far apart for an operand
        big = torch.zeros(4_194_304 + 64, dtype=torch.float16, device=DEV)
        zdp.gated_product(big.as_strided((2, 64), (4_194_304, 1)), w, w, h[:2])
    assert e.value.code == zdp.ERR_UNSUPPORTED
