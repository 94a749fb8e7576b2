"""The wait states around the product's fetches to LDS, in the assembly that the
compiler writes for mx_product.hip (no GPU: the file is only compiled).

The fetches stand in inline asm, where the compiler counts no wait states. The
hardware wants one between a scalar write of m0 and a load to LDS, which takes
its LDS base from m0, and five between a vector instruction's write of a scalar
register and a load that reads that register as its base. A fetch that comes
too early can take the value from before, and its piece then lands elsewhere in
LDS or comes from elsewhere."""
import os
import re
import subprocess

import pytest

from zero_dp_partitioned_amd import build

M0_STATES, BASE_STATES = 1, 5


def _sregs(op):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", op) or re.fullmatch(r"s(\d+)", op)
    return set(range(int(m[1]), int(m[m.lastindex]) + 1)) if m else set()


class _Listing:
    """The instructions of an assembly text, with the jumps to each label."""

    def __init__(self, text):
        self.ins, self.jumps = [], {}
        for line in text.split("\n"):
            t = line.split(";")[0].strip()
            if t.endswith(":") or (t and not t.startswith(".")):
                name, _, rest = t.partition(" ") if " " in t else t.partition("\t")
                self.ins.append((name, [o.strip() for o in rest.split(",")] if rest else []))
                if re.match(r"s_c?branch", name):
                    self.jumps.setdefault(self.ins[-1][1][0], []).append(len(self.ins))

    def before(self, i, states, done=0):
        """(instruction, wait states since) for those at most `states` back from instruction i, over every way to it."""
        while i > 0 and done < states:
            i -= 1
            name, ops = self.ins[i]
            if name.endswith(":"):
                for j in self.jumps.get(name[:-1], ()):
                    yield from self.before(j, states, done)
            else:
                yield name, ops, done
                if name in ("s_branch", "s_endpgm"):
                    return
                done += int(ops[0], 0) + 1 if name == "s_nop" else 1

    def early_fetches(self):
        """(fetches, what comes too soon before one of them)."""
        n, early = 0, []
        for i, (name, ops) in enumerate(self.ins):
            if not re.match(r"(global|buffer)_load_(lds_\w+|\w+_lds)", name):
                continue
            n += 1
            base = set().union(*(_sregs(o.split()[0]) for o in ops))
            for was, to, done in self.before(i, BASE_STATES):
                if was.startswith("s_") and to[:1] == ["m0"] and done < M0_STATES:
                    early.append((was, to, name, ops))
                if was.startswith("v_") and any(_sregs(o) & base for o in to[:2 if "_co_" in was or "div" in was else 1]):
                    early.append((was, to, name, ops))
        return n, early


def test_the_reader_finds_planted_hazards():
    """Small texts with a known answer: the plain order, both kinds, over a jump, and what keeps the distance."""
    load = "\tglobal_load_lds_dwordx4 v1, s[6:7]\n"
    nops = "\ts_nop 3\n"
    for text, found in ((nops + "\ts_mov_b32 m0, s2\n" + load, True), ("\ts_mov_b32 m0, s2\n\ts_nop 0\n" + load, False),
                        ("\tv_readfirstlane_b32 s7, v3\n" + nops + load, True),
                        ("\tv_readfirstlane_b32 s8, v3\n" + load, False),
                        ("\tv_readlane_b32 s6, v3, 2\n\ts_nop 4\n" + load, False),
                        (".L1:\n" + load + "\tv_readfirstlane_b32 s6, v3\n\ts_cbranch_scc1 .L1\n\ts_endpgm\n", True)):
        n, early = _Listing(text).early_fetches()
        assert n == 1 and bool(early) == found, text


def test_every_asm_that_writes_m0_says_so():
    """What an asm overwrites stands in its list, or the compiler may keep a value there across it."""
    with open(os.path.join(build.CSRC, "mx_product.hip")) as f:
        blocks = [b for b in re.findall(r"\basm volatile\((.*?)\);", f.read(), re.S) if re.search(r"\bm0,", b)]
    assert len(blocks) == 2
    for b in blocks:
        assert '"m0"' in b.rsplit(":", 1)[1], b


def test_every_fetch_to_lds_keeps_its_wait_states(tmp_path):
    out = tmp_path / "mx_product.s"
    cmd = [build.hipcc(), *build.COMMON, *build.DEVICE, "-x", "hip", "--cuda-device-only", "-S",
           os.path.join(build.CSRC, "mx_product.hip"), "-o", str(out)]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    except FileNotFoundError:
        pytest.skip("hipcc not found")
    assert r.returncode == 0, r.stderr[-3000:]
    n, early = _Listing(out.read_text()).early_fetches()
    assert n > 0, "no fetch to LDS in the product's kernels"
    assert not early, f"of {n} fetches some come too early, the first: {early[0]}"
