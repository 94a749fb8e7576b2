"""A program whose first calls of a layer's operators are captured ones: every
kernel variant enters a graph before any eager call has asked for its LDS, and
the graph's replays are compared with eager calls afterwards. Run by
test_gpu_sublayer.py in a process of its own."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import zero_dp_partitioned_amd as zdp  # noqa: E402

# m, d, f: single tokens; the small tile with one and two stages in flight, masked and split; the middle and the large tile
SIZES = [(1, 200, 300), (3, 200, 300), (33, 40, 300), (33, 520, 33), (70, 2048, 4096), (600, 640, 520), (2000, 1500, 200),
         (1300, 2600, 2600), (1301, 2603, 2601), (4000, 2560, 72), (1500, 1600, 640)]


def main():
    torch.manual_seed(1)
    cases, ws = [], zdp.new_workspace(1)
    for dt in (torch.float16, torch.bfloat16):
        for m, d, f in SIZES:
            x, wg, wu = (torch.randn(r, d, device="cuda").to(dt) for r in (m, f, f))
            h, g, u, dg, du = (torch.empty(m, f, dtype=dt, device="cuda") for _ in range(5))
            dh = torch.randn(m, f, device="cuda").to(dt)
            wide = torch.float32 if m % 2 else dt
            dwg, dwu = torch.empty(f, d, dtype=wide, device="cuda"), torch.empty(f, d, dtype=wide, device="cuda")
            cases.append((x, wg, wu, h, g, u, dh, dg, du, torch.empty_like(x), dwg, dwu))

    def calls():
        for x, wg, wu, h, g, u, dh, dg, du, dx, dwg, dwu in cases:
            zdp.gated_product(x, wg, wu, h, "gelu_tanh", gate=g, up=u)
            zdp.gated_product_backward(dh, x, wg, wu, g, u, dg, du, ws, dx=dx, dw_gate=dwg, dw_up=dwu, act="gelu_tanh")

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    outs = [c[k] for c in cases for k in (3, 4, 5, 7, 8, 9, 10, 11)]
    for replay in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        calls()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, outs)):
            if not (torch.equal(a, b) and bool(a.any())):
                sys.exit(f"replay {replay}: output {k} {tuple(a.shape)} {a.dtype} differs from the eager call")
    print("first calls captured: ok", flush=True)


if __name__ == "__main__":
    main()
