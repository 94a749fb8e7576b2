"""Which launches the gated product's backward pass takes (csrc/gated_route.h, host
only: built with g++): at sizes where dx and dw were timed in one launch and in
two, the rule takes the faster way or one nearly as fast."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
ROOM = 2 ** 22  # floats of scratch: 16 MiB

# (m, d, f): us of the whole backward pass with dx and dw apart, and together, on one MI355X (fp16)
MEASURED = {
    (4096, 1024, 1024): (66.1, 114.8), (8192, 512, 512): (48.5, 176.4), (2048, 768, 3000): (87.4, 99.2),
    (1500, 1600, 640): (38.2, 42.5), (3953, 672, 2624): (111.3, 148.6), (6659, 272, 288): (40.7, 134.3),
    (4296, 456, 496): (43.8, 94.4), (2000, 2048, 2048): (92.0, 103.8), (1000, 1024, 4096): (65.4, 71.7),
    (2000, 1024, 4096): (105.5, 118.8), (600, 800, 3200): (42.4, 47.3), (3922, 744, 2808): (147.2, 156.1),
    (1500, 1600, 6400): (218.8, 176.0), (2048, 1600, 6400): (245.2, 231.9), (500, 1600, 6400): (96.1, 84.8),
    (1001, 1600, 6400): (145.2, 141.0), (1024, 2560, 6912): (228.6, 186.1), (529, 3752, 2440): (113.9, 70.6),
    (1153, 1960, 5184): (183.0, 142.6), (708, 1384, 12944): (239.7, 181.7), (291, 3384, 2080): (54.3, 49.2),
    (153, 3344, 7920): (119.1, 100.0), (1470, 1720, 6536): (247.5, 187.1), (1500, 1608, 1000): (52.3, 45.8),
    (2079, 1000, 3776): (132.5, 91.1), (1408, 1584, 1504): (69.9, 44.9), (3267, 584, 3600): (159.2, 105.3),
    (2550, 1024, 2856): (119.4, 82.3), (647, 3408, 608): (38.3, 28.8), (474, 4216, 504): (34.0, 24.5),
    (2960, 344, 19952): (391.4, 350.9), (1576, 776, 17120): (376.0, 312.6), (2787, 1088, 13440): (481.3, 453.2),
    (3159, 384, 19256): (385.0, 410.0), (1031, 2712, 520): (37.5, 49.6), (1648, 312, 3392): (56.2, 74.7),
    (451, 776, 976): (40.6, 31.8), (712, 2704, 280): (35.0, 28.3), (666, 2816, 256): (41.5, 26.8),
    (558, 2224, 336): (41.7, 31.9), (1203, 1648, 576): (47.7, 37.4), (1777, 336, 344): (33.8, 52.7),
    (1043, 264, 704): (31.5, 39.4), (1870, 1000, 976): (58.1, 72.2), (903, 880, 256): (29.6, 36.8),
    (2118, 1088, 1032): (55.1, 57.3), (256, 4096, 4096): (65.7, 65.3), (8033, 328, 17136): (930.4, 820.4),
}


@pytest.fixture(scope="module")
def routes(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("g++ not found")
    exe = tmp_path_factory.mktemp("routes") / "gated_routes"
    cmd = ["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
           os.path.join(ROOT, "tests", "c_abi", "gated_routes.cpp"), "-o", str(exe)]
    b = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert b.returncode == 0, b.stderr[-3000:]

    def run(sizes):
        r = subprocess.run([str(exe), str(ROOM)], input="\n".join("%d %d %d" % s for s in sizes), capture_output=True, text=True,
                           timeout=300)
        assert r.returncode == 0, r.stderr[-3000:]
        names = ("together", "splits", "dx_blocks", "tiles", "forward", "forward_splits", "dx", "dx_splits", "dw", "dw_splits")
        return [dict(zip(names, map(int, line.split()))) for line in r.stdout.split("\n")[:len(sizes)]]
    return run


def test_the_way_taken_is_the_faster_one(routes):
    """Within 5 %: two timings of one size on two cards differ by 3."""
    for (size, (apart, together)), r in zip(MEASURED.items(), routes(list(MEASURED))):
        took, other = (together, apart) if r["together"] else (apart, together)
        assert took <= 1.05 * other, f"{size}: {took} us where the other way takes {other}"


def test_one_launch_s_blocks_fit_the_card(routes):
    """dx's blocks, of which each takes a CU, and the partial sums they leave."""
    sizes = [(m, d, f) for m in (65, 200, 1001, 8192, 70_000) for d in (256, 264, 1600, 8192) for f in (256, 1000, 6400, 28_672)]
    for (m, d, f), r in zip(sizes, routes(sizes)):
        if r["together"]:
            assert 0 < r["dx_blocks"] <= 256 and r["splits"] * m * d <= max(ROOM, m * d) and 0 < r["tiles"] <= 1024, (m, d, f)


def test_splits_fit_the_scratch_and_the_contraction(routes):
    sizes = [(m, d, f) for m in (1, 5, 64, 128, 300, 5000, 2 ** 31 - 1) for d in (1, 8, 100, 130, 2048, 2 ** 22)
             for f in (1, 64, 4096, 200_000)]
    for (m, d, f), r in zip(sizes, routes(sizes)):
        assert r["forward_splits"] == 1
        assert r["dx_splits"] >= 1 and (r["dx_splits"] == 1 or (r["dx_splits"] * m * d <= ROOM and r["dx_splits"] * 4 * 64 <= 2 * f + 512))
        assert r["dw_splits"] >= 1 and (r["dw_splits"] == 1 or (r["dw_splits"] * 2 * f * d <= ROOM and r["dw_splits"] * 4 * 64 <= m + 256))


def test_tiles_fit_their_operands(routes):
    """A tile along the columns is moved back to end with its operand, so it may not be wider."""
    sizes = [(m, d, f) for m in (1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 2000) for d in (1, 127, 128, 129, 255, 256, 257, 2000)
             for f in (1, 64, 127, 128, 255, 256, 3000)]
    side = {0: 256, 1: 128, 2: 0}
    for (m, d, f), r in zip(sizes, routes(sizes)):
        assert d >= side[r["dx"]] and d >= side[r["dw"]] and f >= side[r["dw"]], (m, d, f)
        assert not r["together"] or (d >= 256 and f >= 256)
