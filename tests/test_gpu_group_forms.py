"""GPU tests of the products by group-scaled 4-bit weights in the forms that only shapes
like these take (the contraction has at least 8 groups; more than 16 rows a weight on
average, counting a's rows over the experts; 256 tiles of 128 x 128 and more than 64 rows
a weight; 192 tiles of 256 x 256 and, for experts, 192 rows each).  Plain forms and
tolerances are those of test_gpu_groups.py."""
import numpy as np
import pytest
import torch

import dtensor_layout_movement_amd as R
import group_reference as ref
from dtensor_layout_movement_amd import workloads as W
from dtensor_layout_movement_amd.quantized import QuantizedPlan
from test_gpu_blocks import CANARY, DTYPES, Plain, stream, workspace
from test_gpu_groups import PARTS, Grouped, check, expert_product
from test_gpu_group_range import FORMS, some, weight_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


# ------------------------------------------------------------- experts' tiles

# what is left of an expert's rows behind its whole tiles, and experts without rows between
LEFT = [1, 64, 0, 65, 128, 129, 255, 0, 256, 257]


@pytest.mark.parametrize("src,out", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("height,n,spare", [(64, 130, 10), (128, 1900, 200), (256, 3300, 800)])
def test_experts_rows_end_anywhere_in_a_tile(height, n, spare, src, out):
    """Ten experts' 1155 rows; the rows behind them, which are not used, make the buffer's
    average 116, 135 and 195 an expert."""
    expert_product(LEFT, n, 264, src, out, spare=spare)
    expert_product(LEFT[::-1], n, 330, src, out, spare=spare - 3, start=3, seed=1, extra=5)


@pytest.mark.parametrize("height,m,n", [(64, 200, 300), (128, 300, 6600), (256, 600, 10200)])
@pytest.mark.parametrize("src", list(DTYPES))
def test_offsets_that_make_no_sense_stay_inside_the_matrices_in_tiles(height, m, n, src):
    """They are cut to the rows there are; a range that ends before it begins has none.
    Where the ranges that are left do not overlap, their rows are right."""
    k, g = 264, torch.Generator().manual_seed(m)
    x = torch.randn(m, k, generator=g)
    for lists in ([-5, 10, 4000, 2**31 - 1], [30, 10, 20, 5], [-2**31, -1, -1, 3], [m - 1, m + 1, m + 1, 2 * m],
                  [0, m, 0, m], [m, 5, m, 5]):
        a, b, o = Plain(m, k, DTYPES[src], value=x.to(DTYPES[src])), Grouped(3 * n, k).fill(1, 120, 128), Plain(m, n, torch.float32)
        where = torch.tensor(lists, dtype=torch.int32, device="cuda")
        keep, args = workspace(R.reshard_expert_matmul_workspace(a.m, b.m, 3, o.m))
        before = o.view.clone()
        R.reshard_expert_matmul(a.m, b.m, where.data_ptr(), 3, o.m, *args, stream())
        torch.cuda.synchronize()
        o.check_rest()
        a.check_rest()
        assert bool((keep[args[1]:] == CANARY).all())
        lo = [min(max(v, 0), m) for v in lists[:3]]
        hi = [min(max(v, at), m) for v, at in zip(lists[1:], lo)]
        owners = torch.zeros(m, dtype=torch.int64)
        for e in range(3):
            owners[lo[e]:hi[e]] += 1
        assert torch.equal(o.view.cpu()[owners == 0].view(torch.uint8), before.cpu()[owners == 0].view(torch.uint8))
        at, av = some(n, g), a.view.cpu().double().numpy()
        for e in range(3):
            rows = [r for r in range(lo[e], hi[e]) if owners[r] == 1]
            if rows and bool((owners <= 1).all()):
                bv = weight_rows(b, e * n + at)
                check(o.view.cpu()[rows][:, at], av[rows] @ bv.T, np.abs(av[rows]) @ np.abs(bv).T, k * PARTS[src] + 1, "f32",
                      (lists, e))


def test_experts_products_in_tiles_repeat_and_are_the_same_in_a_graph():
    for src, n, spare in (("bf16", 130, 10), ("f32", 1900, 200), ("f16", 3300, 800)):
        m, k, experts = sum(LEFT) + spare, 264, len(LEFT)
        g = torch.Generator().manual_seed(n)
        a, o = Plain(m, k, DTYPES[src], value=torch.randn(m, k, generator=g).to(DTYPES[src])), Plain(m, n, torch.float32)
        b = Grouped(experts * n, k).fill(3, 120, 128)
        counts = [torch.tensor([0] + c, dtype=torch.int32).cumsum(0).to(torch.int32).cuda() for c in (LEFT, LEFT[::-1])]
        where = counts[0].clone()
        keep, args = workspace(R.reshard_expert_matmul_workspace(a.m, b.m, experts, o.m))
        run = lambda: R.reshard_expert_matmul(a.m, b.m, where.data_ptr(), experts, o.m, *args, stream())
        wants = []
        for c in counts:
            where.copy_(c)
            o.view.zero_()
            run()
            torch.cuda.synchronize()
            wants.append(o.view.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for i in (0, 1, 0, 1):  # other offsets between replays
            where.copy_(counts[i])
            o.view.zero_()
            keep.fill_(CANARY)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o.view, wants[i])


# --------------------------------------- infinities, NaN and exactness in every form


@pytest.mark.parametrize("src", list(DTYPES))
@pytest.mark.parametrize("m,n", FORMS)
@pytest.mark.parametrize("k", [297, 1000])
def test_infinities_and_nan_stay_in_their_rows_and_columns_in_every_form(k, m, n, src):
    """A NaN scale in a row beside a tile's edge and in the short last group of others."""
    g = torch.Generator().manual_seed(m + k)
    x = torch.randn(m, k, generator=g).abs() + 0.5
    x[0, 3], x[2, k - 1], x[4, 0] = float("inf"), float("nan"), -float("inf")
    if m > 128:
        x[127, 70], x[128, 71] = float("nan"), float("inf")
    a, b, o = Plain(m, k, DTYPES[src], value=x.to(DTYPES[src])), Grouped(n, k).fill(5, 124, 130), Plain(m, n, torch.float32)
    b.payload[:n, 1] = 0x22  # columns 2 and 3: ones
    lost = [r for r in (7, 63, 127, 256, n - 1) if r < n]
    b.scales[7, 2] = 255
    for r in lost[1:]:
        b.scales[r, b.groups - 1] = 255
    keep, args = workspace(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
    R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
    torch.cuda.synchronize()
    at = some(n, g)
    assert set(lost) <= set(at.tolist())
    with np.errstate(invalid="ignore"):
        want = a.view.cpu().double().numpy() @ weight_rows(b, at).T
    got = o.view.cpu().double()[:, at].numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and inf.any()
    assert np.isnan(got[:, np.isin(at.numpy(), lost)]).all()
    assert np.isfinite(got[[1, 3]][:, ~np.isin(at.numpy(), lost)]).all()


@pytest.mark.parametrize("src", ["f16", "f32"])
@pytest.mark.parametrize("n", [9, 11100, 24600])
def test_elements_are_used_unrounded_in_every_form(n, src):
    """One element of a in each of 288 rows, times weights of one, gives it back: tiles of
    64 that share contractions, of 128 and of 256."""
    k = 288
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(k, generator=g) * torch.exp2(torch.randint(-14, 12, (k,), generator=g).float())).to(DTYPES[src])
    if src == "f16":
        x[:4] = torch.tensor([6e-8, 65504.0, 1.2e-7, -6.1e-5])
    else:
        x[:3] = torch.tensor([3.4028234e38, -1.1754944e-20, 1e-30])
    a, o = Plain(k, k, DTYPES[src], value=torch.diag(x)), Plain(k, n, torch.float32)
    b = Grouped(n, k)
    b.payload[:n, :b.width], b.scales[:n, :b.groups] = 0x22, 127
    keep, args = workspace(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
    R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
    torch.cuda.synchronize()
    assert torch.equal(o.view, x.float().cuda()[:, None].expand(k, n))


# ------------------------------------------------- what a refit leaves is multiplied


@pytest.mark.parametrize("tokens", [3, 50])
def test_a_refits_weights_are_multiplied_where_they_arrive(tokens):
    """weight() of a plan describes a rank's shard as the products take it: a matrix cut
    along its rows, one cut along its columns, and a stack of experts cut along them."""
    g = torch.Generator().manual_seed(tokens)
    T = W.TensorSpec
    specs = [T("rows", (300, 288), torch.bfloat16, (3,), (0,), (2,), (0,)),
             T("cols", (130, 512), torch.float32, (2,), (0,), (2,), (1,)),
             T("experts", (6, 40, 288), torch.bfloat16, (2,), (1,), (3,), (0,))]
    whole = [(torch.randn(*s.shape, generator=g) * 0.1).to(s.dtype) for s in specs]

    def parts(t, side):
        mesh, place = getattr(specs[t], side + "_mesh"), getattr(specs[t], side + "_placements")
        return list(torch.tensor_split(whole[t], mesh[0], dim=place[0]))

    plan = QuantizedPlan(specs, R.DTYPE_FP4_E2M1)
    try:
        src = [[p.contiguous().cuda() for p in parts(t, "src")] for t in range(len(specs))]
        bufs = {(side, what): [[torch.full((max(1, r * c),), CANARY, dtype=torch.uint8, device="cuda")
                                for r, c in getattr(plan, what + "_shapes")(t, side)] for t in range(len(specs))]
                for side in ("src", "dst") for what in ("payload", "scale")}
        ptrs = {key: [[b.data_ptr() for b in per] for per in v] for key, v in bufs.items()}
        bound = plan.bind([[s.data_ptr() for s in per] for per in src], ptrs["src", "payload"], ptrs["src", "scale"],
                          ptrs["dst", "payload"], ptrs["dst", "scale"])
        plan.execute(bound, stream())
        for t, spec in enumerate(specs):
            for rank, part in enumerate(parts(t, "dst")):
                w = plan.weight(t, rank, ptrs["dst", "payload"][t][rank], ptrs["dst", "scale"][t][rank])
                held = ref.quantize(part.reshape(-1, part.shape[-1]))[0]
                k, experts = w.cols, part.shape[0] if part.dim() == 3 else 0
                n = w.rows // max(1, experts)
                a = Plain(tokens, k, torch.bfloat16, value=torch.randn(tokens, k, generator=g).bfloat16())
                o = Plain(tokens, n, torch.float32)
                av = a.view.cpu().double().numpy()
                if experts:
                    ends = [0] + [tokens * (e + 1) // experts for e in range(experts)]
                    where = torch.tensor(ends, dtype=torch.int32, device="cuda")
                    keep, args = workspace(R.reshard_expert_matmul_workspace(a.m, w, experts, o.m))
                    R.reshard_expert_matmul(a.m, w, where.data_ptr(), experts, o.m, *args, stream())
                else:
                    ends = [0, tokens]
                    keep, args = workspace(R.reshard_group_matmul_workspace(a.m, w, o.m))
                    R.reshard_group_matmul(a.m, w, o.m, *args, stream())
                torch.cuda.synchronize()
                for e in range(len(ends) - 1):
                    r, v = slice(ends[e], ends[e + 1]), held[e * n:(e + 1) * n]
                    check(o.view[r], av[r] @ v.T, np.abs(av[r]) @ np.abs(v).T, k + 1, "f32", (spec.name, rank, e))
                o.check_rest()
    finally:
        plan.close()
