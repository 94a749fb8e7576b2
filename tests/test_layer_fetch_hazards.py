"""The wait states around the gated product's fetches to LDS, in the assembly that
the compiler writes for gated_product.hip (no GPU: the file is only compiled),
read as for the 4-bit product, and what its asm says that it overwrites."""
import os
import re
import subprocess

import pytest

from test_mx_fetch_hazards import _Listing
from zero_dp_partitioned_amd import build

SOURCE = os.path.join(build.CSRC, "gated_product.hip")


def test_every_asm_that_writes_m0_or_scc_says_so():
    """What an asm overwrites stands in its list, or the compiler may keep a value there across it."""
    with open(SOURCE) as f:
        blocks = re.findall(r"\basm volatile\((.*?)\);", f.read(), re.S)
    m0 = [b for b in blocks if re.search(r"\bm0,", b)]
    scc = [b for b in blocks if "s_cmp" in b]
    assert len(m0) == 1 and len(scc) == 2
    for name, found in (('"m0"', m0), ('"scc"', scc), ('"memory"', blocks)):
        for b in found:
            assert name in b.rsplit(":", 1)[1], b


def test_every_fetch_to_lds_keeps_its_wait_states(tmp_path):
    out = tmp_path / "gated_product.s"
    cmd = [build.hipcc(), *build.COMMON, *build.DEVICE, "-x", "hip", "--cuda-device-only", "-S", SOURCE, "-o", str(out)]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    except FileNotFoundError:
        pytest.skip("hipcc not found")
    assert r.returncode == 0, r.stderr[-3000:]
    text = out.read_text()
    n, early = _Listing(text).early_fetches()
    assert n > 0, "no fetch to LDS in the product's kernels"
    assert not early, f"of {n} fetches some come too early, the first: {early[0]}"
    # no kernel keeps an array in scratch memory or spills: such loads would count among the fetches that a wait counts
    spills = [int(x) for x in re.findall(r"\.vgpr_spill_count:\s*(\d+)", text)]
    scratch = [int(x) for x in re.findall(r"\.private_segment_fixed_size:\s*(\d+)", text)]
    assert spills and not any(spills) and not any(scratch), (spills, scratch)
