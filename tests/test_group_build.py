"""Checks of the gfx950 code of the products by 4-bit weights and of the experts'
calls, from the compiler's own listing and remarks (hipcc cross-compiles on a machine
without a GPU): no kernel uses scratch memory, and the tiles wait for their loads to LDS
before every barrier that hands what they brought to other waves, for all but those
that come after them."""
import re
import subprocess

import pytest

from dtensor_layout_movement_amd import build as B
from test_block_build import waited


def listing(name, folder):
    out = folder / (name + ".s")
    flags = [f for f in B.HIP_FLAGS if f not in ("-fPIC", "-Wall")]
    cmd = [B.hipcc(), *flags, "--cuda-device-only", "-S", "-Rpass-analysis=kernel-resource-usage", "-I", B.INCLUDE,
           "-I", B.CSRC, f"{B.CSRC}/{name}.hip", "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    return out.read_text(), res.stderr


@pytest.mark.parametrize("name", ["group_quantize", "group_matmul", "group_tiles", "expert_route"])
def test_no_scratch(name, tmp_path):
    _, remarks = listing(name, tmp_path)
    sizes = re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+)", remarks, re.S)
    assert sizes
    for kernel, size in sizes:
        assert size == "0", kernel


def test_tiles_wait_for_their_loads_before_every_barrier(tmp_path):
    text, _ = listing("group_tiles", tmp_path)
    found = 0
    for name, body in re.findall(r"^(\S+group_tilesI\S+):\s+; @\1\n(.*?)\.Lfunc_end", text, re.S | re.M):
        lines = [line.split(";")[0].strip() for line in body.splitlines()]
        lines = [line for line in lines if line]
        bm, bn, wm, wn = map(int, re.search(r"group_tilesILi\d+ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
        threads, heights = 64 * wm * wn, {bm, min(bm, 128)}  # tiles of 256 rows have half tiles too
        # behind the a that a step waits for there is at least one step of it, and, while the
        # weight's next three are young, those
        left = {0} | {h * 8 // threads for h in heights} | {(h * 8 + bn * 6) // threads for h in heights}
        counts = [waited(lines, i) for i, line in enumerate(lines) if line.startswith("s_barrier")]
        assert counts and set(counts) <= left, (name, counts, left)
        found += 1
    assert found == 9  # three tiles, three result types
