"""GPU tests of the experts' calls at the sizes whose kernels others do not take: rows of
more than 16 and more than 128 MiB, which pass the caches, and more tokens than one launch
takes.  Formulas in 64 bits on rows and tokens drawn from all of them; the tolerances are
those of test_gpu_experts.py."""
import numpy as np
import pytest
import torch

import dtensor_layout_movement_amd as R
import group_reference as ref
from test_gpu_blocks import DTYPES, Plain, stream
from test_gpu_experts import sort_fast
from test_gpu_groups import check

pytestmark = pytest.mark.gpu

BITS = {"bf16": torch.int16, "f16": torch.int16, "f32": torch.int32}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


# (more than so many MiB of rows, tokens, choices, columns) of 4-byte elements; 16-bit ones have twice the tokens.  Rows of 1027
# columns have workgroups of their own, those of 131 share them; both start off the 16-byte
# grid and end inside a piece.
LARGE = [(16, 560, 9, 1027), (128, 4000, 9, 1027), (16, 9000, 4, 131), (128, 70000, 4, 131)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("mib,tokens,choices,cols", LARGE)
def test_rows_that_pass_the_caches(mib, tokens, choices, cols, dtype):
    t = DTYPES[dtype]
    size = torch.finfo(t).bits // 8
    tokens = tokens * 4 // size
    n = tokens * choices
    assert mib < n * cols * size / 2 ** 20 < 8 * mib
    g = torch.Generator().manual_seed(tokens)
    ids = torch.randint(0, 20, (tokens, choices), generator=g)
    ids[torch.rand(ids.shape, generator=g) < 0.1] = -1
    ids[5] = -1  # a token without a row
    position = sort_fast(ids.numpy(), 2, 15)[1]  # some experts are not held
    p = torch.from_numpy(position).to(torch.int32).cuda()
    dev = torch.Generator(device="cuda").manual_seed(1)
    make = lambda rows: Plain(rows, cols, t, stride=cols + 3, offset=1)

    def randoms(m):
        m.view.copy_(torch.randn(m.rows, cols, device="cuda", generator=dev))
        return m

    x, y, dout = randoms(make(tokens)), randoms(make(n)), randoms(make(tokens))
    held = torch.zeros(n, dtype=torch.bool, device="cuda")
    held[torch.from_numpy(position[position >= 0]).cuda()] = True
    y.view[~held] = float("nan")  # not read
    weights = Plain(tokens, choices, torch.float32, value=torch.rand(tokens, choices, generator=g))
    pick = torch.unique(torch.cat([torch.arange(9), torch.arange(tokens - 5, tokens), torch.randint(0, tokens, (60,), generator=g)]))
    pos = position[pick]
    rows_of = [(i, j, int(r)) for (i, j), r in np.ndenumerate(pos) if r >= 0]
    at = [r for _, _, r in rows_of]
    bits = BITS[dtype]

    rows = make(n)
    idle = rows.view[~held].view(torch.uint8).clone()
    R.reshard_expert_gather(x.m, p.data_ptr(), choices, rows.m, stream())
    torch.cuda.synchronize()
    assert torch.equal(rows.view[at].view(bits), x.view[pick[[i for i, _, _ in rows_of]]].view(bits))
    assert torch.equal(rows.view[~held].view(torch.uint8), idle)
    # all of them: a row that was written holds its token's bits
    token = torch.zeros(n, dtype=torch.int64, device="cuda")
    token[p[p >= 0].long()] = torch.arange(tokens, device="cuda").repeat_interleave(choices)[(p >= 0).flatten()]
    assert torch.equal(rows.view[held].view(bits), x.view[token[held]].view(bits))
    rows.check_rest()

    # the picked tokens' rows, one behind the other, for the plain forms
    small = np.full(pos.shape, -1)
    for q, (i, j, _) in enumerate(rows_of):
        small[i, j] = q
    yv = y.view[at].double().cpu().numpy()
    wv, dv = weights.view.cpu().double().numpy()[pick], dout.view[pick].double().cpu().numpy()
    for w in (weights.m, None):
        out = make(tokens)
        R.reshard_expert_combine(y.m, p.data_ptr(), choices, w, out.m, stream())
        torch.cuda.synchronize()
        want, mass = ref.combine(yv, small, wv if w else None)
        check(out.view[pick], want, mass, 2 * choices, dtype, "combine")
        assert bool((out.view[5] == 0).all()) and bool(torch.isfinite(out.view).all())
        out.check_rest()

    drows, dweights = make(n), Plain(tokens, choices, torch.float32, stride=choices + 1)
    R.reshard_expert_combine_grad(dout.m, y.m, p.data_ptr(), choices, weights.m, drows.m, dweights.m, stream())
    torch.cuda.synchronize()
    want, dw, mass = ref.combine_grad(dv, yv, small, wv, np.zeros_like(yv))
    check(drows.view[at], want, np.abs(want), 1, dtype, "rows")
    check(dweights.view[pick], dw, mass, 2 * cols, "f32", "weights")
    assert torch.equal(drows.view[~held].view(torch.uint8), idle)
    assert bool((dweights.view[p < 0] == 0).all()) and bool(torch.isfinite(dweights.view).all())
    for m in (drows, dweights, x, y, dout):
        m.check_rest()


MOST = (1 << 23) - 1  # workgroups of a launch


def few_kept(tokens, choices, near):
    """Positions of which only those of the tokens around `near` and a few others have rows."""
    g = torch.Generator().manual_seed(tokens % 1000)
    keep = torch.unique(torch.cat([torch.arange(3), torch.arange(near - 20, min(tokens, near + 20)),
                                   torch.randint(0, tokens, (40,), generator=g), torch.arange(tokens - 3, tokens)]))
    position = torch.full((tokens, choices), -1, dtype=torch.int32, device="cuda")
    n = len(keep) * choices
    position[keep.cuda()] = torch.randperm(n, generator=g).to(torch.int32).view(-1, choices).cuda()
    return keep, position, n


@pytest.mark.parametrize("tokens,choices,cols,near", [
    (MOST + 1000, 2, 512, MOST),  # a workgroup a token
    ((1 << 30) - 8, 1, 9, ((1 << 31) - (1 << 20)) // 2),  # two pieces a token, 2^31 - 2^20 of them a launch
])
def test_more_tokens_than_one_launch_takes(tokens, choices, cols, near):
    keep, position, n = few_kept(tokens, choices, near)
    x = torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator().manual_seed(1)
    vals = torch.randn(len(keep), cols, generator=g).bfloat16()
    x[keep.cuda()] = vals.cuda()
    rows = Plain(n, cols, torch.bfloat16)
    X = R.matrix(tokens, cols, R.DTYPE_BF16, x.data_ptr(), cols)
    R.reshard_expert_gather(X, position.data_ptr(), choices, rows.m, stream())
    torch.cuda.synchronize()
    pos = position[keep.cuda()].cpu().numpy()
    for j in range(choices):
        assert torch.equal(rows.view[pos[:, j].tolist()].cpu(), vals)
    rows.check_rest()
    # and back: x receives the sums, zeros where there is no row
    weights = torch.rand(tokens, choices, device="cuda") if choices > 1 else None
    W = None if weights is None else R.matrix(tokens, choices, R.DTYPE_F32, weights.data_ptr(), choices)
    x.fill_(3.0)
    R.reshard_expert_combine(rows.m, position.data_ptr(), choices, W, X, stream())
    torch.cuda.synchronize()
    want, mass = ref.combine(rows.view.cpu().double().numpy(), pos, None if W is None else weights[keep.cuda()].cpu().double().numpy())
    check(x[keep.cuda()], want, mass, 2 * choices, "bf16")
    x[keep.cuda()] = 0
    for part in x.split(1 << 26):
        assert not bool(part.any())


def test_gradients_of_more_tokens_than_one_launch_takes():
    tokens, choices, cols = MOST + 1000, 2, 8
    keep, position, n = few_kept(tokens, choices, MOST)
    g = torch.Generator(device="cuda").manual_seed(1)
    dout = torch.randn(tokens, cols, device="cuda", generator=g)
    weights = torch.rand(tokens, choices, device="cuda", generator=g)
    dweights = torch.full((tokens, choices), 7.0, device="cuda")
    rows, drows = (Plain(n, cols, torch.float32, value=torch.randn(n, cols)) for _ in range(2))
    m = lambda t: R.matrix(t.shape[0], t.shape[1], R.DTYPE_F32, t.data_ptr(), t.shape[1])
    R.reshard_expert_combine_grad(m(dout), rows.m, position.data_ptr(), choices, m(weights), drows.m, m(dweights), stream())
    torch.cuda.synchronize()
    at, pos = keep.cuda(), position[keep.cuda()].cpu().numpy()
    dr, dw, mass = ref.combine_grad(dout[at].cpu().double().numpy(), rows.view.cpu().double().numpy(), pos,
                                    weights[at].cpu().double().numpy(), np.zeros((n, cols)))
    check(drows.view, dr, np.abs(dr), 1, "f32", "rows")
    check(dweights[at], dw, mass, 2 * cols, "f32", "weights")
    dweights[at] = 0
    assert not bool(dweights.any())
    drows.check_rest()
