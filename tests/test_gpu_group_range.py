"""GPU tests of products by group-scaled 4-bit weights whose scales lie at the ends of
their range, in every form, against plain 64-bit forms (group_reference.py); the
tolerances are those of test_gpu_groups.py.

Every shape here ends inside a step of the tiles (64 columns, three steps of the weight at
a time), so that they multiply what lies behind a row's last group by zeros.
"""
import numpy as np
import pytest
import torch

import dtensor_layout_movement_amd as R
import group_reference as ref
from test_gpu_blocks import DTYPES, Plain, stream, workspace
from test_gpu_groups import PARTS, Grouped, check

pytestmark = pytest.mark.gpu

# few rows; tiles of 64 rows with shared contractions and without, of 128 and of 256
FORMS = [(5, 70), (40, 70), (40, 17000), (130, 16400), (257, 24500)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def some(n, g):
    """Rows of the weight around the tiles' edges, and others."""
    at = torch.cat([torch.arange(min(n, 9)), torch.arange(max(0, n - 9), n), torch.randint(0, n, (90,), generator=g)] +
                   [torch.arange(e - 4, e + 5) for e in (64, 128, 256, 384, 512)])
    return torch.unique(at[at < n])


def multiply(x, b, src):
    """The binary32 product of x (values in src's type) by b."""
    m, n, k = x.shape[0], b.rows, b.cols
    a, o = Plain(m, k, DTYPES[src], value=x.to(DTYPES[src])), Plain(m, n, torch.float32)
    keep, args = workspace(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
    R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
    torch.cuda.synchronize()
    o.check_rest()
    return a.view.cpu().double().numpy(), o.view


def weight_rows(b, at):
    return ref.values(b.payload.cpu()[at][:, :b.width], b.scales.cpu()[at][:, :b.groups], len(at), b.cols)


@pytest.mark.parametrize("src", list(DTYPES))
@pytest.mark.parametrize("k", [264, 330, 1000])
@pytest.mark.parametrize("m,n", FORMS)
def test_largest_scales_of_rows_whose_sums_are_finite(m, n, k, src):
    """Every third row has the scale 2^127 throughout and magnitudes up to 1; the rows
    behind it have all codes.  Under that scale theirs would be infinite."""
    g = torch.Generator().manual_seed(m + k)
    b = Grouped(n, k).fill(n + k, 120, 130)
    b.payload[:n:3, :b.width] &= 0x99  # magnitudes of 0 and 1/2, signs
    b.payload[:n:3, 3:7] = 0x2A  # -1 and 1
    b.scales[:n:3, :b.groups] = 254
    av, got = multiply(torch.randn(m, k, generator=g) * 2.0 ** -12, b, src)
    at = some(n, g)
    bv = weight_rows(b, at)
    check(got.cpu()[:, at], av @ bv.T, np.abs(av) @ np.abs(bv).T, k * PARTS[src] + 1, "f32", (m, n, k))
    assert bool(torch.isfinite(got).all())
