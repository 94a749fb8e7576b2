"""A program whose first calls of the 4-bit product are captured ones: every kernel
variant enters a graph before any eager call has asked for its LDS, and the
graph's replays are compared with eager calls afterwards. Run by
test_gpu_mx.py in a process of its own."""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import zero_dp_partitioned_amd as zdp  # noqa: E402

# m, n: 32 x 32 tiles of eight and of four waves, 64 x 64, 128 x 128, 256 x 256
SIZES = [(40, 50), (600, 600), (900, 900), (1800, 1900), (3400, 3400)]
DTYPES = [torch.float16, torch.bfloat16, torch.float32]


def main():
    torch.manual_seed(1)
    kb, cases = 20, []
    for m, n in SIZES:
        ops = []
        for rows in (m, n):
            ops += [torch.randint(0, 256, (rows, 16 * kb), dtype=torch.uint8, device="cuda"),
                    torch.randint(118, 126, (rows, kb), dtype=torch.uint8, device="cuda")]
        cases += [(ops, torch.empty(m, n, dtype=dt, device="cuda")) for dt in DTYPES]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for ops, out in cases:
            zdp.mx_product(*ops, out)
    for replay in range(3):
        for _, out in cases:
            out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for ops, out in cases:
            want = torch.empty_like(out)
            zdp.mx_product(*ops, want)
            if not (torch.equal(out, want) and bool(out.any())):
                sys.exit(f"replay {replay}: {tuple(out.shape)} {out.dtype} differs from the eager call")
    print("first calls captured: ok", flush=True)


if __name__ == "__main__":
    main()
