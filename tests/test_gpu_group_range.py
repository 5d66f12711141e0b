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


@pytest.mark.parametrize("src", list(DTYPES))
@pytest.mark.parametrize("m,n", FORMS)
def test_elements_past_binary32_are_infinite_and_stay_in_their_columns(m, n, src):
    """4 and 6 under the scale 2^126, 2 and more under 2^127: as they read back.  The sums
    that have one are infinite or NaN, the others as ever."""
    k, g = 300, torch.Generator().manual_seed(m)
    b = Grouped(n, k).fill(n, 120, 130)
    at = some(n, g)
    big = at[1::4]
    b.payload[big, 48:64] = 0  # of one group
    for i, (scale, code) in enumerate([(253, 6), (253, 15), (254, 4), (254, 13), (254, 6), (254, 7)]):
        b.scales[big[i::6], 3] = scale
        b.payload[big[i::6], 53] = code << 4
    av, got = multiply(torch.randn(m, k, generator=g).abs() + 0.5, b, src)
    back = Plain(n, k, torch.float32)
    R.reshard_group_dequantize(b.m, back.m, stream())
    torch.cuda.synchronize()
    infinite = torch.isinf(back.view)
    assert infinite.sum() == len(big) and bool(infinite[big, 107].all())
    got = got.cpu()
    lost = torch.zeros(n, dtype=torch.bool)
    lost[big] = True
    assert torch.equal(torch.isfinite(got), ~lost.expand(m, n))
    rest = at[~lost[at]]
    bv = weight_rows(b, rest)
    check(got[:, rest], av @ bv.T, np.abs(av) @ np.abs(bv).T, k * PARTS[src] + 1, "f32")


@pytest.mark.parametrize("src", list(DTYPES))
@pytest.mark.parametrize("m,n", FORMS)
def test_elements_below_the_normal_range_are_multiplied_exactly(m, n, src):
    """Scale bytes 0 to 2, elements from 2^-128 on, by large elements of a: terms above
    2^-126."""
    k, g = 300, torch.Generator().manual_seed(m)
    b = Grouped(n, k).fill(n, 0, 3)
    x = (1 + torch.rand(m, k, generator=g)) * torch.randn(m, k, generator=g).sign() * (2.0 ** 14 if src == "f16" else 2.0 ** 100)
    av, got = multiply(x, b, src)
    at = some(n, g)
    bv = weight_rows(b, at)
    # (the elements of a are multiples of 2^4 at least: every part's term is 2^-124 or more)
    want, mass = av @ bv.T, np.abs(av) @ np.abs(bv).T
    check(got.cpu()[:, at], want, mass, k * PARTS[src] + 1, "f32")


def test_magnitudes_that_round_to_two_to_the_128_read_back_as_infinite():
    top = torch.tensor([3.5 * 2.0 ** 126, -3.4028234663852886e38, float(np.nextafter(np.float32(3.5 * 2.0 ** 126), np.float32(0))),
                        3.0 * 2.0 ** 126, 2.0 ** 127, 1.0])
    src, h, back = Plain(6, 1, torch.float32, value=top[:, None]), Grouped(6, 1), Plain(6, 1, torch.float32)
    R.reshard_group_quantize(src.m, h.m, stream())
    R.reshard_group_dequantize(h.m, back.m, stream())
    torch.cuda.synchronize()
    inf = float("inf")
    assert back.view.flatten().tolist() == [inf, -inf, 3.0 * 2.0 ** 126, 3.0 * 2.0 ** 126, 2.0 ** 127, 1.0]
    assert h.scales[:6, 0].tolist() == [253, 253, 253, 252, 252, 125]
