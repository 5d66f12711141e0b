"""GPU tests of tokens sorted by expert, their rows moved there and back, and the
gradients, against plain 64-bit forms (group_reference.py).

Tolerances.  Sorting and gathering are exact.  A token's sum adds one product for each
choice: with c of them at most 2 c roundings of 2^-24 relative to the sum of the
terms' magnitudes, and half a step of the type.  A weight's gradient adds one product
a column: cols roundings of that kind and one each for the products, and half a step.
A gradient row is one product, rounded to binary32 and then to the type.
"""
import numpy as np
import pytest
import torch

import dtensor_layout_movement_amd as R
import group_reference as ref
from test_gpu_blocks import CANARY, DTYPES, Plain, stream, workspace
from test_gpu_groups import PARTS, Grouped, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def sort(ids, first, experts):
    """Offsets and positions (device tensors) of a 2-d tensor of choices."""
    tokens, choices = ids.shape
    code = R.DTYPE_I64 if ids.dtype == torch.int64 else R.DTYPE_I32
    offsets = torch.full((experts + 3,), -77, dtype=torch.int32, device="cuda")
    position = torch.full((tokens * choices + 2,), -77, dtype=torch.int32, device="cuda")
    ids = ids.cuda()
    keep, args = workspace(R.reshard_expert_sort_workspace(tokens, choices, experts))
    R.reshard_expert_sort(ids.data_ptr(), code, tokens, choices, first, experts, offsets.data_ptr(),
                          position.data_ptr(), *args, stream())
    torch.cuda.synchronize()
    assert bool((offsets[experts + 1:] == -77).all()) and bool((position[tokens * choices:] == -77).all())
    assert bool((keep[args[1]:] == CANARY).all())
    return offsets[:experts + 1], position[:tokens * choices].view(tokens, choices)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,choices,first,experts,total", [
    (0, 3, 0, 5, 5), (1, 1, 0, 1, 1), (1, 8, 0, 64, 64), (63, 1, 0, 2, 2), (65, 3, 7, 40, 50), (1024, 1, 0, 1000, 1024),
    (1025, 1, 5, 1, 9), (512, 8, 0, 64, 64), (513, 8, 0, 64, 64), (1000, 5, 100, 1024, 1300), (4096, 8, 0, 64, 64),
    (70000, 2, 3, 3, 8), (3000, 64, 0, 17, 64)])
def test_sort_is_stable_and_leaves_others_out(tokens, choices, first, experts, total, dtype):
    g = torch.Generator().manual_seed(tokens + choices)
    ids = torch.randint(0, total, (tokens, choices), generator=g)
    ids[torch.rand(ids.shape, generator=g) < 0.3] = first + experts // 2  # a popular one
    ids[torch.rand(ids.shape, generator=g) < 0.05] = -1
    offsets, position = sort(ids.to(dtype), first, experts)
    want = ref.sort(ids.numpy(), first, experts) if ids.numel() <= 40000 else sort_fast(ids.numpy(), first, experts)
    assert np.array_equal(offsets.cpu().numpy(), want[0])
    assert np.array_equal(position.cpu().numpy(), want[1])


def sort_fast(ids, first, experts):
    flat = ids.reshape(-1) - first
    held = (flat >= 0) & (flat < experts)
    order = np.argsort(np.where(held, flat, experts), kind="stable")
    position = np.empty(flat.shape, np.int64)
    position[order] = np.arange(len(flat))
    counts = np.bincount(flat[held], minlength=experts)
    return np.concatenate([[0], np.cumsum(counts)]), np.where(held, position, -1).reshape(ids.shape)


def test_numbers_at_the_ends_of_their_type_are_no_experts():
    big = torch.tensor([[2**63 - 1, -2**63], [5, 2**40], [2**32 + 5, -2**32 + 5], [6, 4]])
    offsets, position = sort(big, 5, 2)
    assert offsets.tolist() == [0, 1, 2]
    assert position.tolist() == [[-1, -1], [0, -1], [-1, -1], [1, -1]]
    small = torch.tensor([[2**31 - 1, -2**31], [5, 6]], dtype=torch.int32)
    assert sort(small, 5, 2)[1].tolist() == [[-1, -1], [0, 1]]


def test_one_expert_gets_everything_and_none_gets_anything():
    for n in (100, 5000):
        offsets, position = sort(torch.full((n, 2), 3), 0, 7)
        assert offsets.tolist() == [0, 0, 0, 0] + [2 * n] * 4
        assert torch.equal(position.cpu().flatten(), torch.arange(2 * n, dtype=torch.int32))
        offsets, position = sort(torch.full((n, 2), 9), 0, 7)
        assert offsets.tolist() == [0] * 8 and bool((position == -1).all())


# --------------------------------------------------------------------- moving


def case(tokens, choices, total, experts, n_rows=None, seed=0):
    """Positions of random choices; all rows, or fewer than the choices need."""
    g = torch.Generator().manual_seed(seed + tokens)
    ids = torch.rand(tokens, total, generator=g).argsort(dim=1)[:, :choices]
    if tokens > 3:
        ids[2] = -1  # a token without any row
    offsets, position = ref.sort(ids.numpy(), 0, experts)
    n = n_rows if n_rows is not None else tokens * choices
    return position, n, torch.from_numpy(position).to(torch.int32).cuda()


CASES = [(1, 1, 1, 1, 1), (1, 8, 64, 64, 7168), (3, 2, 4, 4, 1), (5, 3, 5, 5, 7), (40, 8, 16, 12, 33), (17, 64, 64, 50, 130),
         (130, 5, 9, 9, 515), (300, 8, 32, 32, 1024), (7, 9, 12, 12, 3001)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,choices,total,experts,cols", CASES)
def test_gather_copies_bits(tokens, choices, total, experts, cols, dtype):
    for extra, n_rows in ((0, None), (3, None), (0, max(1, tokens * choices // 2))):
        position, n, p = case(tokens, choices, total, experts, n_rows)
        size = torch.empty((), dtype=DTYPES[dtype]).element_size()
        x = Plain(tokens, cols, DTYPES[dtype], stride=cols + extra, offset=extra)
        bits = torch.int32 if size == 4 else torch.int16
        raw = torch.randint(-2**31 if size == 4 else -2**15, 2**31 if size == 4 else 2**15, (tokens, cols),
                            generator=torch.Generator().manual_seed(cols))
        x.view.view(bits).copy_(raw.to(bits))
        rows = Plain(n, cols, DTYPES[dtype], stride=cols + extra, offset=extra)
        want = ref.gather(raw.numpy(), position, rows.view.view(bits).cpu().long().numpy())
        R.reshard_expert_gather(x.m, p.data_ptr(), choices, rows.m, stream())
        torch.cuda.synchronize()
        assert np.array_equal(rows.view.view(bits).cpu().long().numpy(), want)
        rows.check_rest()
        x.check_rest()


def inputs(position, n, cols, dtype, weights_dtype, extra, seed):
    g = torch.Generator().manual_seed(seed)
    tokens, choices = position.shape
    rows = Plain(n, cols, DTYPES[dtype], stride=cols + extra, offset=extra,
                 value=torch.randn(n, cols, generator=g).to(DTYPES[dtype]))
    used = {p for _, _, p in ref.kept(position, n)}
    for r in range(n):
        if r not in used:
            rows.view[r] = float("nan")  # not read
    w = torch.rand(tokens, choices, generator=g)
    w[torch.from_numpy(position < 0)] = float("nan")  # nor are these
    weights = Plain(tokens, choices, DTYPES[weights_dtype], stride=choices + extra, offset=extra,
                    value=w.to(DTYPES[weights_dtype]))
    return rows, weights


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,choices,total,experts,cols", CASES)
def test_combine_adds_the_choices_that_have_a_row(tokens, choices, total, experts, cols, dtype):
    for extra, n_rows, wt in ((0, None, "f32"), (3, None, dtype), (0, max(1, tokens * choices // 2), "bf16"), (1, None, None)):
        position, n, p = case(tokens, choices, total, experts, n_rows)
        rows, weights = inputs(position, n, cols, dtype, wt or "f32", extra, cols)
        out = Plain(tokens, cols, DTYPES[dtype], stride=cols + extra, offset=extra)
        R.reshard_expert_combine(rows.m, p.data_ptr(), choices, weights.m if wt else None, out.m, stream())
        torch.cuda.synchronize()
        want, mass = ref.combine(rows.view.cpu().double().numpy(), position, weights.view.cpu().double().numpy() if wt else None)
        check(out.view, want, mass, 2 * choices, dtype, (extra, n_rows, wt))
        if tokens > 3:
            assert bool((out.view[2] == 0).all())
        out.check_rest()
        rows.check_rest()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("tokens,choices,total,experts,cols", CASES)
def test_combine_grad_matches_the_formulas(tokens, choices, total, experts, cols, dtype):
    for extra, n_rows, wt, dt in ((0, None, "f32", "f32"), (3, None, dtype, "bf16"), (0, max(1, tokens * choices // 2), "f16", dtype),
                                  (1, None, None, "f16")):
        position, n, p = case(tokens, choices, total, experts, n_rows)
        rows, weights = inputs(position, n, cols, dtype, wt or "f32", extra, cols)
        dout = Plain(tokens, cols, DTYPES[dtype], stride=cols + extra, offset=extra,
                     value=torch.randn(tokens, cols, generator=torch.Generator().manual_seed(1)).to(DTYPES[dtype]))
        drows = Plain(n, cols, DTYPES[dtype], stride=cols + extra, offset=extra)
        dweights = Plain(tokens, choices, DTYPES[dt], stride=choices + extra, offset=extra)
        before = drows.view.cpu()
        both = (rows.m, p.data_ptr(), choices, weights.m if wt else None)
        R.reshard_expert_combine_grad(dout.m, *both, drows.m, dweights.m, stream())
        torch.cuda.synchronize()
        y = np.nan_to_num(rows.view.cpu().double().numpy())
        dv, wv = dout.view.cpu().double().numpy(), weights.view.cpu().double().numpy() if wt else None
        want, dw, mass = ref.combine_grad(dv, y, position, wv, before.double().numpy())
        used = [r for _, _, r in ref.kept(position, n)]
        check(drows.view[used], want[used], np.abs(want[used]), 1, dtype, "rows")
        idle = [r for r in range(n) if r not in set(used)]
        assert torch.equal(drows.view[idle].cpu().view(torch.uint8), before[idle].view(torch.uint8))
        check(dweights.view, dw, mass, 2 * cols, dt, "weights")
        dropped = torch.from_numpy(~((position >= 0) & (position < n)))
        assert bool((dweights.view.cpu()[dropped] == 0).all())
        for m in (drows, dweights, rows, dout):
            m.check_rest()
        # each alone gives the same bits
        one, other = Plain(n, cols, DTYPES[dtype]), Plain(tokens, choices, DTYPES[dt])
        R.reshard_expert_combine_grad(dout.m, None, *both[1:], one.m, None, stream())
        R.reshard_expert_combine_grad(dout.m, *both, None, other.m, stream())
        torch.cuda.synchronize()
        assert torch.equal(one.view[used], drows.view[used]) and torch.equal(other.view, dweights.view)


def test_gradients_agree_with_differences():
    """Along random directions, in fp32: the sum is linear in rows and in weights, so
    that a difference over any step is exact up to roundings."""
    tokens, choices, cols = 20, 3, 50
    position, n, p = case(tokens, choices, 6, 6)
    g = torch.Generator().manual_seed(3)
    y, d = torch.randn(n, cols, generator=g), torch.randn(tokens, cols, generator=g)
    w, e = torch.rand(tokens, choices, generator=g), torch.randn(tokens, choices, generator=g)
    r = torch.randn(n, cols, generator=g)

    def forward(rows, weights):
        a, b, o = (Plain(*t.shape, torch.float32, value=t) for t in (rows, weights, d))
        R.reshard_expert_combine(a.m, p.data_ptr(), choices, b.m, o.m, stream())
        torch.cuda.synchronize()
        return float((o.view.cpu().double() * d.double()).sum())

    dout, rows, weights = (Plain(*t.shape, torch.float32, value=t) for t in (d, y, w))
    drows, dweights = Plain(n, cols, torch.float32, value=torch.zeros(n, cols)), Plain(tokens, choices, torch.float32)
    R.reshard_expert_combine_grad(dout.m, rows.m, p.data_ptr(), choices, weights.m, drows.m, dweights.m, stream())
    torch.cuda.synchronize()
    # 20 x 50 sums of 3 terms of size about 1, each off by 6 roundings of 2^-24, times d
    tol = 4 * tokens * cols * choices * 6 * 2.0 ** -24 * 4
    assert abs((forward(y + r, w) - forward(y - r, w)) / 2 - float((drows.view.cpu().double() * r.double()).sum())) < tol
    assert abs((forward(y, w + e) - forward(y, w - e)) / 2 - float((dweights.view.cpu().double() * e.double()).sum())) < tol


def test_no_tokens_no_columns_and_no_rows():
    p = torch.full((8,), 0, dtype=torch.int32, device="cuda")
    for tokens, cols, n in ((0, 5, 3), (4, 0, 3), (4, 5, 0)):
        x, rows, out = (Plain(r, cols, torch.float32) for r in (tokens, n, tokens))
        w = Plain(tokens, 2, torch.float32, value=torch.ones(tokens, 2))
        dw = Plain(tokens, 2, torch.float32)
        R.reshard_expert_gather(x.m, p.data_ptr(), 2, rows.m, stream())
        R.reshard_expert_combine(rows.m, p.data_ptr(), 2, w.m, out.m, stream())
        drows = Plain(n, cols, torch.float32)
        R.reshard_expert_combine_grad(x.m, rows.m, p.data_ptr(), 2, w.m, drows.m, dw.m, stream())
        torch.cuda.synchronize()
        if n == 0:
            assert bool((out.view == 0).all())
        if n == 0 or cols == 0:
            assert bool((dw.view == 0).all())
        for m in (x, out, dw):
            m.check_rest()


def test_positions_outside_the_rows_are_left_out():
    p = torch.tensor([[0, -5], [2**31 - 1, 2], [-2**31, 3]], dtype=torch.int32, device="cuda")
    x, rows = Plain(3, 40, torch.float32, value=torch.ones(3, 40)), Plain(3, 40, torch.float32)
    before = rows.view.clone()
    R.reshard_expert_gather(x.m, p.data_ptr(), 2, rows.m, stream())
    out = Plain(3, 40, torch.float32)
    torch.cuda.synchronize()
    assert bool((rows.view[0] == 1).all()) and bool((rows.view[2] == 1).all())
    assert torch.equal(rows.view[1].view(torch.uint8), before[1].view(torch.uint8))
    rows.check_rest()
    R.reshard_expert_combine(rows.m, p.data_ptr(), 2, None, out.m, stream())
    torch.cuda.synchronize()
    assert bool((out.view[:2] == 1).all()) and bool((out.view[2] == 0).all())


# ------------------------------------------------------------ a run of them all


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens", [1, 50, 700])
def test_a_layer_of_experts_and_its_way_back(tokens, dtype):
    """Sort, gather, two products by 4-bit weights, combine, and the gradients of the
    way back; eager, and captured and replayed on new inputs."""
    experts, first, total, choices, hidden, inner = 12, 2, 16, 4, 136, 72
    g = torch.Generator().manual_seed(tokens)
    t = DTYPES[dtype]
    n = tokens * choices
    w_up, w_down = torch.randn(experts * inner, hidden, generator=g) * 0.1, torch.randn(experts * hidden, inner, generator=g) * 0.1
    held = []
    for w in (w_up, w_down):
        src, h = Plain(*w.shape, torch.float32, value=w), Grouped(*w.shape)
        R.reshard_group_quantize(src.m, h.m, stream())
        held.append(h)
    up, down = held
    ids = torch.empty(tokens, choices, dtype=torch.int64, device="cuda")
    offsets = torch.empty(experts + 1, dtype=torch.int32, device="cuda")
    position = torch.empty(tokens, choices, dtype=torch.int32, device="cuda")
    x, out, dout = (Plain(tokens, hidden, t) for _ in range(3))
    rows, y, drows = (Plain(n, hidden, t) for _ in range(3))
    mid = Plain(n, inner, t)
    weights, dweights = Plain(tokens, choices, torch.float32), Plain(tokens, choices, torch.float32)
    rooms = [workspace(k) for k in (R.reshard_expert_sort_workspace(tokens, choices, experts),
                                    R.reshard_expert_matmul_workspace(rows.m, up.m, experts, mid.m),
                                    R.reshard_expert_matmul_workspace(mid.m, down.m, experts, y.m))]

    def layer():
        R.reshard_expert_sort(ids.data_ptr(), R.DTYPE_I64, tokens, choices, first, experts, offsets.data_ptr(),
                              position.data_ptr(), *rooms[0][1], stream())
        R.reshard_expert_gather(x.m, position.data_ptr(), choices, rows.m, stream())
        R.reshard_expert_matmul(rows.m, up.m, offsets.data_ptr(), experts, mid.m, *rooms[1][1], stream())
        R.reshard_expert_matmul(mid.m, down.m, offsets.data_ptr(), experts, y.m, *rooms[2][1], stream())
        R.reshard_expert_combine(y.m, position.data_ptr(), choices, weights.m, out.m, stream())
        R.reshard_expert_combine_grad(dout.m, y.m, position.data_ptr(), choices, weights.m, drows.m, dweights.m, stream())

    def fill(seed):
        g = torch.Generator().manual_seed(seed)
        ids.copy_(torch.rand(tokens, total, generator=g).argsort(dim=1)[:, :choices])
        x.view.copy_(torch.randn(tokens, hidden, generator=g).to(t))
        dout.view.copy_(torch.randn(tokens, hidden, generator=g).to(t))
        weights.view.copy_(torch.rand(tokens, choices, generator=g))

    def verify():
        off, pos = ref.sort(ids.cpu().numpy(), first, experts)
        assert np.array_equal(offsets.cpu().numpy(), off) and np.array_equal(position.cpu().numpy(), pos)
        xv = x.view.cpu().double().numpy()
        gathered = ref.gather(xv, pos, np.zeros((n, hidden)))
        uv, dv = up.values(), down.values()
        midv, yv = mid.view.cpu().double().numpy(), y.view.cpu().double().numpy()
        for e in range(experts):  # each step against the step before it, as the device holds it
            r = slice(off[e], off[e + 1])
            a, b = uv[e * inner:(e + 1) * inner], dv[e * hidden:(e + 1) * hidden]
            check(mid.view[r], gathered[r] @ a.T, np.abs(gathered[r]) @ np.abs(a).T, hidden * PARTS[dtype] + 1, dtype)
            check(y.view[r], midv[r] @ b.T, np.abs(midv[r]) @ np.abs(b).T, inner * PARTS[dtype] + 1, dtype)
        wv = weights.view.cpu().double().numpy()
        want, mass = ref.combine(yv, pos, wv)
        check(out.view, want, mass, 2 * choices, dtype)
        gd, gw, gm = ref.combine_grad(dout.view.cpu().double().numpy(), yv, pos, wv, np.zeros((n, hidden)))
        check(drows.view[:off[-1]], gd[:off[-1]], np.abs(gd[:off[-1]]), 1, dtype)
        check(dweights.view, gw, gm, 2 * hidden, "f32")

    fill(1)
    layer()
    torch.cuda.synchronize()
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for seed in (2, 3, 4):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        verify()
        layer()  # eager work between the replays
        torch.cuda.synchronize()
        verify()


def test_two_streams_with_workspaces_of_their_own():
    tokens, choices, experts = 3000, 4, 30
    jobs = []
    for s in range(2):
        st = torch.cuda.Stream()
        ids = torch.randint(0, experts, (tokens, choices), generator=torch.Generator().manual_seed(s)).cuda()
        keep, args = workspace(R.reshard_expert_sort_workspace(tokens, choices, experts))
        jobs.append((st, ids, args, keep, torch.empty(experts + 1, dtype=torch.int32, device="cuda"),
                     torch.empty(tokens * choices, dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(5):
        for st, ids, args, _, offsets, position in jobs:
            R.reshard_expert_sort(ids.data_ptr(), R.DTYPE_I64, tokens, choices, 0, experts, offsets.data_ptr(),
                                  position.data_ptr(), *args, st.cuda_stream)
    torch.cuda.synchronize()
    for _, ids, _, _, offsets, position in jobs:
        want = sort_fast(ids.cpu().numpy(), 0, experts)
        assert np.array_equal(offsets.cpu().numpy(), want[0])
        assert np.array_equal(position.cpu().numpy().reshape(tokens, choices), want[1])
