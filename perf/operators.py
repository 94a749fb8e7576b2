"""Cases of the microscaled 4-bit (MXFP4) operators, and their plain forms.

The format: blocks of 32 values share one power of two, held as a biased exponent byte (E8M0: 2^(byte - 127),
255 = NaN), and each value is an E2M1 code (0 0.5 1 1.5 2 3 4 6 with a sign), two codes a byte, the even
element in the low nibble. The block's exponent is floor(log2(max |v|)) - 2; the codes round to nearest
even and saturate at 6.

What is held in 4 bits comes back as the values it stands for, so the quantising cases write the codes and widen
them again, as a rank does that writes its slice and reads the gathered vector.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 32
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
PER_VALUE = 17 / 32  # bytes a value takes: 16 bytes of codes and one of scale for 32


def _ceil(n, m):
    return (n + m - 1) // m


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the smallest shard (787,971 parameters over 4 ranks, the last rank's slice): launch-bound
        {"name": "writeback_tiny", "kind": "writeback", "n": 196_899, "offset": 591_072, "dtype": "f16"},
        # rank 63 of 64 of a 7.5B-parameter vector, segments aligned to a block: offsets past 2^32
        {"name": "writeback_7.5b", "kind": "writeback", "n": 117_186_240, "offset": 7_382_813_760, "dtype": "bf16"},
        # one token's activations on their way into a product
        {"name": "quantise_token", "kind": "quantise", "rows": 1, "cols": 4096, "dtype": "bf16", "both": False},
        # a ragged batch at GPT-2 1.5B's width, both ways, as a training step of a layer needs
        {"name": "quantise_ragged", "kind": "quantise", "rows": 1001, "cols": 1600, "dtype": "f16", "both": True},
        # 8192 tokens at LLaMA-3 8B's MLP width, both ways
        {"name": "quantise_train", "kind": "quantise", "rows": 8192, "cols": 14336, "dtype": "bf16", "both": True},
        # four copies of the smallest shard
        {"name": "average_tiny", "kind": "average", "n": 196_993, "copies": 4},
        # eight copies of a 117M shard (7.5B over 64 ranks), one for each GPU of a node
        {"name": "average_7.5b", "kind": "average", "n": 117_187_500, "copies": 8},
        # one token through LLaMA-3 8B's MLP projection: reads the weights once
        {"name": "product_token", "kind": "product", "m": 1, "n": 14336, "k": 4096, "dtype": "bf16"},
        # a small odd batch through GPT-2 1.5B's MLP output projection
        {"name": "product_batch", "kind": "product", "m": 45, "n": 1600, "k": 6400, "dtype": "f16"},
        # GPT-2 1.5B's tied head on a ragged batch: an odd vocabulary
        {"name": "product_head", "kind": "product", "m": 1001, "n": 50257, "k": 1600, "dtype": "bf16"},
        # forward of LLaMA-3 8B's MLP projection over 8192 tokens
        {"name": "product_forward", "kind": "product", "m": 8192, "n": 14336, "k": 4096, "dtype": "bf16"},
        # its weight gradient: the contraction runs over the tokens, the gradient stays fp32
        {"name": "product_wgrad", "kind": "product", "m": 14336, "n": 4096, "k": 8192, "dtype": "f32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["writeback", "quantise", "average", "product"])
    if kind == "writeback":
        return {"kind": kind, "n": _log(rng, 1, 117_000_000), "offset": BLOCK * rng.randrange(0, 230_000_000),
                "dtype": rng.choice(["f16", "bf16", "f32"])}
    if kind == "quantise":
        rows, cols = _log(rng, 1, 8192), _log(rng, 1, 14336)
        return {"kind": kind, "rows": rows, "cols": cols, "dtype": rng.choice(["f16", "bf16", "f32"]),
                "both": rng.random() < 0.5}
    if kind == "average":
        copies = rng.choice([1, 2, 3, 4, 7, 8])
        return {"kind": kind, "n": _log(rng, 1, 117_000_000), "copies": copies}
    m, k = _log(rng, 1, 8192), _log(rng, 32, 14336)
    n = _log(rng, 1, min(50257, 8192 * 14336 * 4096 // (m * k)))
    return {"kind": kind, "m": m, "n": n, "k": k, "dtype": rng.choice(["f16", "bf16", "f32"])}


def work(case):
    kind = case["kind"]
    if kind == "writeback":  # master read, codes written and read, values written
        n = case["n"]
        return {"bytes": n * (4 + 2 * PER_VALUE + BYTES[case["dtype"]]), "flops": 2 * n}
    if kind == "quantise":  # source read; for each way codes written and read, values written
        n, ways, s = case["rows"] * case["cols"], 2 if case["both"] else 1, BYTES[case["dtype"]]
        return {"bytes": n * (s + ways * (2 * PER_VALUE + s)), "flops": 2 * n * ways}
    if kind == "average":
        n, c = case["n"], case["copies"]
        return {"bytes": n * (c * PER_VALUE + 4), "flops": n * (c + 3)}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": (m + n) * _ceil(k, BLOCK) * 17 + m * n * BYTES[case["dtype"]], "flops": 2 * m * n * k}


# --------------------------------------------------------------------------
# plain forms (fp32)
# --------------------------------------------------------------------------

def _blocks(x):
    """[rows, cols] as fp32 [rows, blocks, 32], the last block filled with zeros."""
    rows, cols = x.shape
    x = x.float()
    if cols % BLOCK:
        x = torch.cat([x, x.new_zeros(rows, BLOCK - cols % BLOCK)], 1)
    return x.reshape(rows, -1, BLOCK)


def _exponents(blocks):
    """The blocks' shared exponents: floor(log2(max |v|)) - 2, at least -126 here (no block is that small)."""
    amax = blocks.abs().amax(-1, keepdim=True)
    return (torch.frexp(amax).exponent - 3).clamp_min(-126)


def _power(e):
    return ((e.int() + 127) << 23).view(torch.float32)


def _round(r):
    """The E2M1 values nearest to r, ties to even, saturating at 6."""
    a = r.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step).clamp_max(6.0) * torch.sign(r)


def _values(x):
    """[rows, cols] rounded to the format along its rows, as fp32 values."""
    b = _blocks(x)
    s = _power(_exponents(b))
    return (_round(b / s) * s).reshape(x.shape[0], -1)[:, :x.shape[1]]


def _encode(x):
    """[rows, cols] -> codes [rows, 16 * blocks] and scales [rows, blocks]."""
    b = _blocks(x)
    e = _exponents(b)
    q = _round(b / _power(e))
    mag = torch.bucketize(q.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=q.device), out_int32=True)
    code = (mag + 8 * (q < 0)).to(torch.uint8).reshape(x.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (e[..., 0] + 127).to(torch.uint8)


def _pairs(dtype):
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=dtype, device=DEV)
    grid = torch.cat([grid, -grid])
    byte = torch.arange(256, device=DEV)
    return torch.stack([grid[byte & 15], grid[byte >> 4]], 1)


def _decode(codes, scales, dtype=torch.float32):
    """codes [..., 16 * blocks], scales [..., blocks] -> values [..., 32 * blocks]."""
    v = _pairs(dtype)[codes.int()].reshape(*scales.shape, BLOCK)
    return (v * _power(scales.int() - 127).to(dtype)[..., None]).reshape(*scales.shape[:-1], -1)


def _plain(s):
    kind = s["kind"]
    if kind == "writeback":
        return _values(s["master"][None])[0].to(s["out"].dtype)
    if kind == "quantise":
        x = s["x"]
        got = [_values(x).to(x.dtype)]
        if s["both"]:
            got.append(_values(x.t()).to(x.dtype))
        return got
    if kind == "average":
        v = _decode(s["codes"], s["scales"])[:, :s["n"]]
        avg = v.sum(0) / v.shape[0]
        g = avg * (1.0 / s["loss_scale"])
        norm = g.double().square().sum().sqrt().float().reshape(1)
        return {"avg": avg, "norm": norm, "overflow": (~torch.isfinite(avg)).any().int().reshape(1)}
    a, b = _decode(s["a_codes"], s["a_scales"]), _decode(s["b_codes"], s["b_scales"])
    return (a @ b.t()).to(s["out"].dtype)


# --------------------------------------------------------------------------
# the framework's calls
# --------------------------------------------------------------------------

def _kernels(s):
    import zero_dp_partitioned_amd as zdp
    kind = s["kind"]
    if kind == "writeback":
        zdp.mx_cast_writeback(s["master"], s["codes"], s["scales"], s["offset"])
        zdp.mx_dequantize(s["codes"], s["scales"], s["out"], offset=s["offset"])
        return s["out"]
    if kind == "quantise":
        zdp.mx_quantize(s["x"], s["codes"], s["scales"], s["codes_t"], s["scales_t"])
        zdp.mx_dequantize(s["codes"], s["scales"], s["out"])
        if not s["both"]:
            return [s["out"]]
        zdp.mx_dequantize(s["codes_t"], s["scales_t"], s["out_t"])
        return [s["out"], s["out_t"]]
    if kind == "average":
        if "state" not in s:  # a program makes these once
            s["state"], s["workspace"] = zdp.new_state(s["loss_scale"]), zdp.new_workspace(1)
        st, ws = s["state"], s["workspace"]
        zdp.mx_reduce_grad_segment(s["code_copies"], s["scale_copies"], s["avg"], ws, 0, st)
        zdp.grad_norm_overflow(None, ws, 1, st)
        norm, flag = zdp.StepState.grad_norm.offset, zdp.StepState.overflow.offset
        return {"avg": s["avg"], "norm": st[norm:norm + 4].view(torch.float32),
                "overflow": st[flag:flag + 4].view(torch.int32)}
    zdp.mx_product(s["a_codes"], s["a_scales"], s["b_codes"], s["b_scales"], s["out"])
    return s["out"]


def run(state):
    return _kernels(state) if own else _plain(state)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _empty(rows, cols):
    b = _ceil(cols, BLOCK)
    return (torch.empty(rows, 16 * b, dtype=torch.uint8, device=DEV), torch.empty(rows, b, dtype=torch.uint8, device=DEV))


def _normal(gen, *shape, sigma=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device=DEV) * sigma).to(dtype)


def _inputs(case, seed):
    """The arrays drawn from the seed."""
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind = case["kind"]
    if kind == "writeback":  # master weights
        return {"master": _normal(gen, case["n"], sigma=0.02)}
    if kind == "quantise":  # activations, each token at its own size
        x = _normal(gen, case["rows"], case["cols"]) * torch.exp(_normal(gen, case["rows"], 1))
        return {"x": x.to(TYPES[case["dtype"]])}
    if kind == "average":  # gradients times a loss scale, quantised by the ranks that sent them
        got = [_encode(_normal(gen, 1, case["n"], sigma=1e-3 * 1024.0)) for _ in range(case["copies"])]
        return {"codes": torch.cat([c for c, _ in got]), "scales": torch.cat([s for _, s in got])}
    a = _encode(_normal(gen, case["m"], case["k"]))
    b = _encode(_normal(gen, case["n"], case["k"], sigma=0.02))
    return {"a_codes": a[0], "a_scales": a[1], "b_codes": b[0], "b_scales": b[1]}


def prepare(case, seed):
    s = {"kind": case["kind"], **_inputs(case, seed)}
    kind = case["kind"]
    if kind == "writeback":  # the whole flat vector in 4 bits; the rank writes its slice
        blocks = case["offset"] // BLOCK + _ceil(case["n"], BLOCK)
        s |= {"offset": case["offset"], "codes": torch.empty(16 * blocks, dtype=torch.uint8, device=DEV),
              "scales": torch.empty(blocks, dtype=torch.uint8, device=DEV),
              "out": torch.empty(case["n"], dtype=TYPES[case["dtype"]], device=DEV)}
    elif kind == "quantise":
        x = s["x"]
        s["both"] = case["both"]
        s["codes"], s["scales"] = _empty(*x.shape)
        s["codes_t"], s["scales_t"] = _empty(x.shape[1], x.shape[0]) if case["both"] else (None, None)
        s["out"] = torch.empty_like(x)
        s["out_t"] = x.new_empty(x.shape[1], x.shape[0]) if case["both"] else None
    elif kind == "average":
        s |= {"n": case["n"], "loss_scale": 1024.0, "code_copies": list(s["codes"].unbind(0)),
              "scale_copies": list(s["scales"].unbind(0)), "avg": torch.empty(case["n"], device=DEV)}
    else:
        s["out"] = torch.empty(case["m"], case["n"], dtype=TYPES[case["dtype"]], device=DEV)
    return s


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _nearest(x):
    """[rows, cols] float64 -> the format's values, by comparing with the midpoints between its magnitudes."""
    rows, cols = x.shape
    pad = torch.zeros(rows, _ceil(cols, BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    pad[:, :cols] = x
    b = pad.view(rows, -1, BLOCK)
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -120))) - 2)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    y = (b / scale).abs()
    low, high = torch.bucketize(y, mid, out_int32=True), torch.bucketize(y, mid, right=True, out_int32=True)
    index = torch.where(low % 2 == 0, low, high)  # they differ at a midpoint only: the even code
    return (torch.copysign(grid[index], b) * scale).view(rows, -1)[:, :cols]


def _wide(codes, scales):
    """codes [rows, 16 * blocks], scales [rows, blocks] -> float64 values [rows, 32 * blocks]."""
    rows = codes.shape[0]
    nibble = torch.stack([codes % 16, codes // 16], -1).reshape(rows, -1).int()
    mag, sign = nibble % 8, 1 - 2 * (nibble // 8)
    exp, man = mag // 2, mag % 2
    v = torch.where(exp == 0, man * 0.5, (1 + man * 0.5) * 2.0 ** (exp - 1).double()) * sign
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1)


def exact(case, seed):
    s, kind = _inputs(case, seed), case["kind"]
    if kind == "writeback":
        return _nearest(s["master"].double()[None])[0]
    if kind == "quantise":
        x = s["x"].double()
        return [_nearest(x)] + ([_nearest(x.t().contiguous())] if case["both"] else [])
    if kind == "average":
        total = torch.zeros(case["n"], dtype=torch.float64, device=DEV)
        for c, e in zip(s["codes"], s["scales"]):
            total += _wide(c[None], e[None])[0, :case["n"]]
        avg = total / case["copies"]
        return {"avg": avg, "norm": (torch.linalg.vector_norm(avg) / 1024.0).reshape(1), "overflow": None}
    return _wide(s["a_codes"], s["a_scales"]) @ _wide(s["b_codes"], s["b_scales"]).t()
