"""Checks of the block-scaled products' gfx950 code, from the compiler's own listing
(hipcc cross-compiles on a machine without a GPU): loads that go straight to LDS
are waited for before every barrier that hands what they brought to other
waves, in the code as it is built."""
import re
import subprocess

import pytest

from dtensor_layout_movement_amd import build as B


@pytest.fixture(scope="module", params=["block_matmul", "block_grad"])
def kernels(request, tmp_path_factory):
    """The instructions of each kernel that loads to LDS, by its name."""
    out = tmp_path_factory.mktemp("isa") / (request.param + ".s")
    flags = [f for f in B.HIP_FLAGS if f not in ("-fPIC", "-Wall")]
    cmd = [B.hipcc(), *flags, "--cuda-device-only", "-S", "-I", B.INCLUDE, "-I", B.CSRC,
           f"{B.CSRC}/{request.param}.hip", "-o", str(out)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    found = {}
    for name, body in re.findall(r"^(\S+):\s+; @\1\n(.*?)\.Lfunc_end", out.read_text(), re.S | re.M):
        lines = [line.split(";")[0].strip() for line in body.splitlines()]
        lines = [line for line in lines if line]
        if any(line.startswith("buffer_load") and line.endswith(" lds") for line in lines):
            found[name] = lines
    return found


def waited(lines, at):
    """The vmcnt of the wait that stands before the barrier at `at` in straight-line
    code with no load between them; None if there is none."""
    for line in reversed(lines[:at]):
        m = re.match(r"s_waitcnt .*vmcnt\((\d+)\)", line)
        if m:
            return int(m.group(1))
        if re.match(r"buffer_load|global_load|s_cbranch|s_branch|s_barrier|\.L", line):
            return None
    return None


def test_loads_to_lds_are_waited_for_before_every_barrier(kernels):
    assert kernels
    for name, lines in kernels.items():
        # a ring's step leaves the loads of the two steps after it under way
        m = re.search(r"matmul_ringILi\d+ELb[01]ELb[01]ELi(\d)E", name)
        left = {0} if not m else {0, 2 * (max(2, int(m.group(1))) * 16 + 64) * 8 // 256}
        counts = [waited(lines, i) for i, line in enumerate(lines) if line.startswith("s_barrier")]
        assert counts and set(counts) <= left, (name, counts)
