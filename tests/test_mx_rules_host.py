"""Which kernel the sizes of the GPU tests select, asked from the library's
own rules: every tile of every product is tested."""
import os
import shutil
import subprocess

import pytest

from test_gpu_mx_tiles import PARTS, TILES
from test_host_sanitize import CSRC, ROOT


def test_tiles_of_the_gpu_tests(tmp_path):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = str(tmp_path / "mx_rules")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-I" + CSRC,
                    os.path.join(ROOT, "tests", "mx_rules.cpp"), "-o", exe], check=True,
                   capture_output=True, timeout=120)
    sizes = [(m, c, i) for what, tile, m, c, i in TILES] + [(m, c, i) for m, c, i, t, p in PARTS]
    out = subprocess.run([exe] + [str(v) for s in sizes for v in s], check=True,
                         capture_output=True, text=True, timeout=60).stdout.split("\n")
    got = [tuple(int(v) for v in line.split()) for line in out if line]
    assert len(got) == len(sizes)
    at = {"matmul": 0, "linear": 1, "grad": 2}
    for (what, tile, m, c, i), g in zip(TILES, got):
        assert g[at[what]] == tile, (what, m, c, i, g)
        if what == "grad":
            assert g[3] == 1, (m, c, i, g)
    for (m, c, i, tile, parts), g in zip(PARTS, got[len(TILES):]):
        assert (g[2], g[3]) == (tile, parts), (m, c, i, g)
    assert {(w, t) for w, t, *_ in TILES} == {(w, t) for w in at for t in (64, 128, 256)}
    assert {(t, p) for *_, t, p in PARTS} >= {(64, 2), (128, 2), (256, 2), (256, 3)}
