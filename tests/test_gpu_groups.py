"""GPU tests of the group-scaled 4-bit matrices and their products against plain
64-bit forms (group_reference.py).

Tolerances.  Quantizing and reading back are exact up to the one rounding the format
defines: compared bit for bit.  A product multiplies exactly (an fp16 or fp32 element
of a as two or three parts that add up to it) and adds K terms, or K times the parts,
in binary32 in some order: each sum is off by at most that many times 2^-24 of the
sum of the terms' magnitudes S (first order; a part's magnitudes add up to less than
twice the element's, and all but the first are below 2^-7 of it, so that S grows by
less than 1%, which the count of the terms, one above that of the additions, and the
rounding that no chain of additions exhausts leave room for).  The result's type adds half a step.
"""
import numpy as np
import pytest
import torch

import dtensor_layout_movement_amd as R
import group_reference as ref
from group_reference import GROUP
from dtensor_layout_movement_amd import workloads as W
from dtensor_layout_movement_amd.quantized import QuantizedPlan
from test_gpu_blocks import CANARY, DTYPES, Plain, stream, workspace

pytestmark = pytest.mark.gpu

PARTS = {"bf16": 1, "f16": 2, "f32": 3}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


class Grouped:
    """A group-scaled matrix with spare stride and canaries around."""

    def __init__(self, rows, cols, extra=0, extra_scales=0):
        self.rows, self.cols, self.groups = rows, cols, -(-cols // GROUP)
        self.width = self.groups * GROUP // 2
        self.payload = torch.full((rows + 2, self.width + 16 * extra), CANARY, dtype=torch.uint8, device="cuda")
        self.scales = torch.full((rows + 2, self.groups + extra_scales), CANARY, dtype=torch.uint8, device="cuda")
        self.m = R.matrix(rows, cols, R.DTYPE_FP4_E2M1, self.payload.data_ptr(), 2 * self.payload.stride(0), 1,
                          self.scales.data_ptr(), self.scales.stride(0))
        self.m.keep = self.payload, self.scales

    def check_rest(self):
        codes = torch.stack((self.payload & 15, self.payload >> 4), dim=-1).flatten(1)
        assert bool((codes[:self.rows, self.cols:2 * self.width] == 0).all())
        assert bool((self.payload[:self.rows, self.width:] == CANARY).all())
        assert bool((self.payload[self.rows:] == CANARY).all())
        assert bool((self.scales[:self.rows, self.groups:] == CANARY).all())
        assert bool((self.scales[self.rows:] == CANARY).all())

    def fill(self, seed, low=100, high=140):
        """Random codes, zeros behind the last column, and scale bytes."""
        g = torch.Generator().manual_seed(seed)
        codes = torch.randint(0, 16, (self.rows, 2 * self.width), generator=g)
        codes[:, self.cols:] = 0
        self.payload[:self.rows, :self.width] = (codes[:, 0::2] | codes[:, 1::2] << 4).to(torch.uint8).cuda()
        self.scales[:self.rows, :self.groups] = torch.randint(low, high, (self.rows, self.groups), generator=g).to(
            torch.uint8).cuda()
        return self

    def values(self):
        return ref.values(self.payload, self.scales, self.rows, self.cols)


def values_of(shape, kind, seed, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if kind == "wide":  # magnitudes over the whole range, subnormals and rows of zeros among them
        x = x * torch.exp2(torch.randint(-145, 122, (shape[0], 1), generator=g).float())
        x[:: 7] = 0
    elif kind == "special":
        for v in (float("inf"), -float("inf"), float("nan")):
            x[torch.rand(shape, generator=g) < 0.004] = v
        x[torch.rand(shape, generator=g) < 0.02] = -0.0
    elif kind == "border":  # largest values at and just above 6 * 2^e, ties between 4-bit values
        x = torch.round(x.clamp(-5, 5) * 8) / 8
        x[:, ::GROUP] = 6.0 * torch.exp2(torch.randint(-1, 3, (shape[0], 1), generator=g).float())
        x[1::2, ::GROUP] = torch.nextafter(x[1::2, ::GROUP], torch.tensor(float("inf")))
    return x.to(dtype)


SHAPES = [(1, 1), (1, 32), (3, 31), (5, 33), (64, 64), (65, 100), (130, 300), (301, 515)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_quantize_matches_the_definition(shape, dtype):
    rows, cols = shape
    for i, kind in enumerate(("normal", "wide", "special", "border")):
        x = values_of(shape, kind, 10 * rows + i, DTYPES[dtype])
        src = Plain(rows, cols, DTYPES[dtype], stride=cols + (3 if i % 2 else 0), offset=i, value=x)
        dst = Grouped(rows, cols, extra=i % 2, extra_scales=i)
        R.reshard_group_quantize(src.m, dst.m, stream())
        torch.cuda.synchronize()
        want, scales = ref.quantize(x)
        assert np.array_equal(dst.scales[:rows, :dst.groups].cpu().numpy(), scales), kind
        got = dst.values()
        assert np.array_equal(got, want, equal_nan=True), kind
        assert np.array_equal(np.signbit(got)[~np.isnan(got)], np.signbit(want)[~np.isnan(want)]), kind
        dst.check_rest()
        src.check_rest()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dequantize_rounds_each_value_once(shape, dtype):
    """Every code under every scale byte, 255 (NaN) and 0 among them."""
    rows, cols = shape
    h = Grouped(rows, cols, extra=2, extra_scales=1).fill(rows + cols, 0, 256)
    out = Plain(rows, cols, DTYPES[dtype], stride=cols + 5, offset=3)
    R.reshard_group_dequantize(h.m, out.m, stream())
    torch.cuda.synchronize()
    with np.errstate(over="ignore"):
        want = torch.from_numpy(h.values().astype(np.float32)).to(DTYPES[dtype])  # binary32 holds it, or it is infinite
    got = out.view.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)])
    if dtype != "f16":  # exact
        fin = np.isfinite(want.double().numpy())
        assert np.array_equal(want.double().numpy()[fin], h.values()[fin])
    out.check_rest()


# ------------------------------------------------------------------ products


def room(need):
    keep, args = workspace(need)
    return keep, args


def tolerance(terms, mass, want, dtype):
    t = DTYPES[dtype]
    info = torch.finfo(t)
    return terms * 2.0 ** -24 * mass + info.eps / 2 * (np.abs(want) + terms * 2.0 ** -24 * mass) + \
        info.smallest_normal * info.eps / 2


def check(got, want, mass, terms, dtype, name=""):
    got = got.double().cpu().numpy()
    tol = tolerance(terms, mass, want, dtype)
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
    top = torch.finfo(DTYPES[dtype]).max
    over = np.abs(want) + tol >= top  # may round to infinity
    bad = ~(off <= tol) & ~over
    assert not bad.any(), (name, np.argwhere(bad)[:5], got[bad][:5], want[bad][:5], tol[bad][:5])
    assert (np.isfinite(got) | over).all()


def product(m, n, k, src, out, seed=0, extra=0, offset=0):
    g = torch.Generator().manual_seed(seed + m + 3 * n + 7 * k)
    x = torch.randn(m, k, generator=g)
    x[:, ::17] *= 20
    a = Plain(m, k, DTYPES[src], stride=k + extra, offset=offset, value=x.to(DTYPES[src]))
    b = Grouped(n, k, extra=extra % 3, extra_scales=extra).fill(seed + n, 118, 128)
    o = Plain(m, n, DTYPES[out], stride=n + extra, offset=offset)
    keep, args = room(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
    R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
    torch.cuda.synchronize()
    av, bv = a.view.cpu().double().numpy(), b.values()
    check(o.view, av @ bv.T, np.abs(av) @ np.abs(bv).T, k * PARTS[src] + 1, out, (m, n, k, src, out))
    o.check_rest()
    a.check_rest()
    assert bool((keep[args[1]:] == CANARY).all())


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 16, 32), (2, 17, 33), (4, 15, 127), (15, 64, 128), (16, 33, 129),
                                   (17, 130, 256), (33, 16, 1000), (64, 200, 96), (65, 31, 300), (130, 257, 161),
                                   (300, 129, 513)])
@pytest.mark.parametrize("src", list(DTYPES))
def test_product_of_every_kind_of_size(m, n, k, src):
    for out in DTYPES:
        product(m, n, k, src, out)
    product(m, n, k, src, src, seed=1, extra=5, offset=3)


@pytest.mark.parametrize("src,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("m,n,k", [(1, 2048, 4096), (5, 513, 7168), (48, 1030, 2050), (257, 1100, 640), (1030, 520, 520),
                                   (700, 8200, 288)])
def test_larger_products(m, n, k, src, out):
    product(m, n, k, src, out)


@pytest.mark.parametrize("m,n,k", [(0, 5, 40), (5, 0, 40), (3, 5, 0), (300, 257, 0), (0, 0, 0)])
def test_products_without_rows_columns_or_contraction(m, n, k):
    for src in DTYPES:
        a, b, o = Plain(m, k, DTYPES[src]), Grouped(n, k), Plain(m, n, torch.bfloat16, stride=n + 3, offset=1)
        keep, args = room(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
        R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
        torch.cuda.synchronize()
        assert bool((o.view == 0).all())
        o.check_rest()


@pytest.mark.parametrize("m", [1, 20, 300])
@pytest.mark.parametrize("src", list(DTYPES))
def test_infinities_and_nan_stay_in_their_rows_and_columns(m, src):
    n, k = 70, 200
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(m)).abs() + 0.5
    x[0, 3] = float("inf")
    if m > 5:
        x[2, 199], x[4, 0] = float("nan"), -float("inf")
    a, b, o = Plain(m, k, DTYPES[src], value=x.to(DTYPES[src])), Grouped(n, k).fill(5, 124, 130), Plain(m, n, torch.float32)
    codes = b.payload[:n, :b.width]
    codes[:, 1] = 0x22  # columns 2 and 3: ones
    b.scales[7, 2] = 255
    b.scales[11, 6] = 255  # the short last group
    keep, args = room(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
    R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
    torch.cuda.synchronize()
    with np.errstate(invalid="ignore"):
        want = a.view.cpu().double().numpy() @ b.values().T
    got = o.view.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]) and inf.any()
    assert np.isnan(want[:, 7]).all() and np.isnan(want[:, 11]).all()


@pytest.mark.parametrize("src", ["f16", "f32"])
def test_elements_are_used_unrounded(src):
    """One column of a after the other times a weight of ones gives the element back."""
    k = 96
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(k, generator=g) * torch.exp2(torch.randint(-14, 12, (k,), generator=g).float())).to(DTYPES[src])
    if src == "f16":
        x[:4] = torch.tensor([6e-8, 65504.0, 1.2e-7, -6.1e-5])
    else:
        x[:3] = torch.tensor([3.4028234e38, -1.1754944e-20, 1e-30])
    for m in (k, 4 * k):  # small and large forms
        a = Plain(m, k, DTYPES[src], value=torch.diag(x).repeat(m // k, 1))
        b = Grouped(9, k)
        b.payload[:9, :b.width], b.scales[:9, :b.groups] = 0x22, 127
        o = Plain(m, 9, torch.float32)
        keep, args = room(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
        R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
        torch.cuda.synchronize()
        assert torch.equal(o.view.cpu(), x.float().repeat(m // k)[:, None].expand(m, 9))


# ----------------------------------------------------------- experts' products


def expert_product(counts, n, k, src, out, spare=0, start=0, seed=0, extra=0):
    """counts: rows of each expert; spare rows behind the last, start rows before the first."""
    experts, total = len(counts), start + sum(counts) + spare
    offsets = start + np.concatenate([[0], np.cumsum(counts)])
    g = torch.Generator().manual_seed(seed + n)
    a = Plain(total, k, DTYPES[src], stride=k + extra, offset=extra, value=torch.randn(total, k, generator=g).to(DTYPES[src]))
    if spare:
        a.view[total - spare:] = float("nan")  # not used
    b = Grouped(experts * n, k, extra=extra % 3, extra_scales=extra).fill(seed, 120, 128)
    o = Plain(total, n, DTYPES[out], stride=n + extra, offset=extra)
    before = o.raw.clone()
    where = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    keep, args = room(R.reshard_expert_matmul_workspace(a.m, b.m, experts, o.m))
    R.reshard_expert_matmul(a.m, b.m, where.data_ptr(), experts, o.m, *args, stream())
    torch.cuda.synchronize()
    av, bv = a.view.cpu().double().numpy(), b.values()
    for e in range(experts):
        rows = slice(offsets[e], offsets[e + 1])
        w = bv[e * n:(e + 1) * n]
        check(o.view[rows], av[rows] @ w.T, np.abs(av[rows]) @ np.abs(w).T, k * PARTS[src] + 1, out, (e, counts))
    o.view[offsets[0]:offsets[-1]].view(torch.uint8).fill_(CANARY) if extra == 0 and total else o.view[
        offsets[0]:offsets[-1]].copy_(o.flat[:1].expand(offsets[-1] - offsets[0], n) if total else o.view)
    o.check_rest()
    if extra == 0:
        assert torch.equal(o.raw, before)  # rows without an expert are as they were


COUNTS = {
    "one token": [0, 1, 0, 0, 1],
    "one expert": [37],
    "all to the last": [0] * 66 + [70],
    "empty ones between": [3, 0, 0, 17, 0, 16, 1, 0, 33, 0],
    "none": [0, 0, 0],
    "many small": [1, 2] * 70,
    "large and small": [300, 1, 0, 129, 16, 64, 65],
}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("src,out", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32")])
def test_expert_products(name, src, out):
    expert_product(COUNTS[name], 33, 161, src, out)
    expert_product(COUNTS[name], 64, 256, src, out, spare=19, seed=1)


@pytest.mark.parametrize("src", list(DTYPES))
def test_expert_products_of_strided_and_offset_matrices(src):
    expert_product([5, 0, 40, 200], 130, 300, src, src, spare=3, start=4, extra=5)
    expert_product([150, 90], 300, 700, src, "f32", start=70)


def test_offsets_that_make_no_sense_stay_inside_the_matrices():
    """They are cut to the rows there are; a range that ends before it begins has none."""
    m, n, k = 40, 33, 70
    for lists in ([-5, 10, 4000, 2**31 - 1], [30, 10, 20, 5], [-2**31, -1, -1, 3], [39, 41, 41, 100]):
        a, b, o = Plain(m, k, torch.bfloat16, value=torch.ones(m, k)), Grouped(3 * n, k).fill(1), Plain(m, n, torch.float32)
        where = torch.tensor(lists, dtype=torch.int32, device="cuda")
        keep, args = room(R.reshard_expert_matmul_workspace(a.m, b.m, 3, o.m))
        R.reshard_expert_matmul(a.m, b.m, where.data_ptr(), 3, o.m, *args, stream())
        torch.cuda.synchronize()
        o.check_rest()


def test_products_repeat_bit_for_bit_and_are_the_same_in_a_graph():
    for m, n, k in ((3, 300, 2000), (40, 600, 4096), (600, 1100, 512)):
        a = Plain(m, k, torch.bfloat16, value=torch.randn(m, k, generator=torch.Generator().manual_seed(m)).bfloat16())
        b, o = Grouped(n, k).fill(3, 118, 128), Plain(m, n, torch.float32)
        keep, args = room(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
        R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
        torch.cuda.synchronize()
        want = o.view.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
        for _ in range(3):
            o.view.zero_()
            keep.fill_(CANARY)  # the workspace needs no preparation
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(o.view, want)


def test_quantizing_into_columns_of_one_buffer():
    """Two weights' payloads side by side: neither touches the other's bytes."""
    rows, cols = 33, 70
    pay = torch.full((rows, 112), CANARY, dtype=torch.uint8, device="cuda")
    sc = torch.full((rows, 7), CANARY, dtype=torch.uint8, device="cuda")
    x = values_of((rows, cols), "normal", 4, torch.float32)
    src = Plain(rows, cols, torch.float32, value=x)
    for at in (0, 1):
        R.reshard_group_quantize(src.m, R.matrix(rows, cols, R.DTYPE_FP4_E2M1, pay.data_ptr() + 64 * at, 224, 1,
                                                 sc.data_ptr() + 4 * at, 7), stream())
    torch.cuda.synchronize()
    want, scales = ref.quantize(x)
    for at in (0, 1):
        assert np.array_equal(ref.values(pay[:, 64 * at:64 * at + 48], sc[:, 4 * at:4 * at + 3], rows, cols), want)
    assert bool((pay[:, 48:64] == CANARY).all()) and bool((sc[:, 3] == CANARY).all())


# --------------------------------------------------------------- refit to 4 bits

T, RR = W.TensorSpec, W.R
LISTS = {
    "rows cut anywhere to columns": [T("w", (301, 512), torch.bfloat16, (4,), (0,), (2,), (1,))],
    "columns with an edge, replicas": [T("w", (130, 511), torch.float32, (2,), (1,), (2, 3), (RR, 0))],
    "a stack of experts": [T("e", (6, 40, 96), torch.float16, (3, 2), (0, 1), (2, 3), (0, 2))],
    "several": [T("a", (33, 70), torch.float32, (1,), (0,), (1,), (0,)), T("b", (4, 5, 64), torch.bfloat16, (4,), (0,), (2,), (2,))],
}


@pytest.mark.parametrize("name", list(LISTS))
def test_every_destination_rank_holds_its_part_of_the_quantized_whole(name):
    specs = LISTS[name]

    def parts(spec, side):
        h = R.layout_create(spec.shape, R.dtype_code(spec.dtype), getattr(spec, side + "_mesh"), getattr(spec, side + "_placements"))
        try:
            return [tuple(slice(*R.reshard_layout_shard_runs(h, r, d)[0]) for d in range(len(spec.shape)))
                    for r in range(R.reshard_layout_num_ranks(h))]
        finally:
            R.reshard_layout_destroy(h)

    whole = [values_of((int(np.prod(s.shape[:-1])), s.shape[-1]), "normal" if s.dtype != torch.float32 else "special", t, s.dtype)
             .view(s.shape) for t, s in enumerate(specs)]
    src = [[w[box].contiguous().cuda() for box in parts(s, "src")] for s, w in zip(specs, whole)]
    plan = QuantizedPlan(specs, R.DTYPE_FP4_E2M1)
    try:
        bufs = {(side, what): [[torch.full((max(1, r * c),), CANARY, dtype=torch.uint8, device="cuda")
                                for r, c in getattr(plan, what + "_shapes")(t, side)] for t in range(len(specs))]
                for side in ("src", "dst") for what in ("payload", "scale")}
        ptrs = {k: [[b.data_ptr() for b in per] for per in v] for k, v in bufs.items()}
        bound = plan.bind([[s.data_ptr() for s in per] for per in src], ptrs["src", "payload"], ptrs["src", "scale"],
                          ptrs["dst", "payload"], ptrs["dst", "scale"])
        plan.execute(bound, stream())
        torch.cuda.synchronize()
        for t, (s, w) in enumerate(zip(specs, whole)):
            want, scales = ref.quantize(w.reshape(-1, s.shape[-1]))
            want, scales = want.reshape(s.shape), scales.reshape(*s.shape[:-1], -1)
            for rank, box in enumerate(parts(s, "dst")):
                part = want[box].reshape(-1, want[box].shape[-1])
                rows, cols = plan.shard_shapes(t, "dst")[rank]
                assert part.shape == (rows, cols)
                q = bufs["dst", "payload"][t][rank].view(plan.payload_shapes(t, "dst")[rank])
                sc = bufs["dst", "scale"][t][rank].view(plan.scale_shapes(t, "dst")[rank])
                assert np.array_equal(ref.values(q, sc, rows, cols), part, equal_nan=True), (t, rank)
                groups = slice(box[-1].start // GROUP, -(-box[-1].stop // GROUP))
                assert np.array_equal(sc.cpu().numpy(), scales[(*box[:-1], groups)].reshape(rows, -1))
    finally:
        plan.close()


# ---------------------------------------------- every form, by the shapes that take it


@pytest.mark.parametrize("src", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", [(16, 3300, 2100), (16, 13000, 640), (64, 300, 6000), (70, 260, 20000), (65, 33000, 256),
                                   (257, 50000, 232), (2000, 6400, 320)])
def test_forms_of_the_products(m, n, k, src):
    """Few rows with 16 to 64 columns a workgroup, tiles of 64 with shared contractions, of
    128, of 256 with half tiles; checked on rows and columns drawn from all of it."""
    g = torch.Generator().manual_seed(m + n)
    a = Plain(m, k, DTYPES[src], value=torch.randn(m, k, generator=g).to(DTYPES[src]))
    b, o = Grouped(n, k).fill(n, 120, 128), Plain(m, n, torch.float32)
    keep, args = room(R.reshard_group_matmul_workspace(a.m, b.m, o.m))
    R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
    torch.cuda.synchronize()
    rows = torch.unique(torch.cat([torch.arange(min(m, 3)), torch.arange(max(0, m - 3), m), torch.randint(0, m, (60,), generator=g)]))
    cols = torch.unique(torch.cat([torch.arange(min(n, 40)), torch.arange(max(0, n - 40), n), torch.randint(0, n, (400,), generator=g)]))
    av = a.view.cpu()[rows].double().numpy()
    bv = ref.values(b.payload.cpu()[cols][:, :b.width], b.scales.cpu()[cols][:, :b.groups], len(cols), k)
    check(o.view.cpu()[rows][:, cols], av @ bv.T, np.abs(av) @ np.abs(bv).T, k * PARTS[src] + 1, "f32", (m, n, k))
    assert bool(torch.isfinite(o.view).all())
    o.check_rest()
    # the same call in a graph, replayed with eager work between
    want = o.view.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.reshard_group_matmul(a.m, b.m, o.m, *args, stream())
    for _ in range(2):
        o.view.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.view, want)


def test_rows_far_apart_take_the_form_that_has_no_limit():
    """More than 2^22 bytes from row to row of the payload (here of one row more than
    fits): many rows of a go sixteen at a time."""
    m, n, k = 40, 3, 256
    stride = (1 << 23) + 64  # elements
    pay = torch.full((3 * stride // 2,), CANARY, dtype=torch.uint8, device="cuda")
    sc = torch.full((n, 8), 127, dtype=torch.uint8, device="cuda")
    small = Grouped(n, k).fill(9, 127, 128)
    for r in range(n):
        pay[r * stride // 2:r * stride // 2 + k // 2] = small.payload[r, :k // 2]
    a = Plain(m, k, torch.bfloat16, value=torch.randn(m, k, generator=torch.Generator().manual_seed(1)).bfloat16())
    o, want = Plain(m, n, torch.float32), Plain(m, n, torch.float32)
    b = R.matrix(n, k, R.DTYPE_FP4_E2M1, pay.data_ptr(), stride, 1, sc.data_ptr(), 8)
    keep, args = room(R.reshard_group_matmul_workspace(a.m, b, o.m))
    R.reshard_group_matmul(a.m, b, o.m, *args, stream())
    torch.cuda.synchronize()
    av, bv = a.view.cpu().double().numpy(), small.values()
    check(o.view, av @ bv.T, np.abs(av) @ np.abs(bv).T, k + 1, "f32")


def test_weights_past_four_gigabytes():
    """A payload whose last rows lie past 2^32 bytes, in both kinds of forms."""
    n, k = 300000, 32768
    pay = torch.zeros(n, k // 2, dtype=torch.uint8, device="cuda")
    sc = torch.full((n, k // 32), 127, dtype=torch.uint8, device="cuda")
    assert pay.numel() > 1 << 32
    last = Grouped(64, k).fill(4, 127, 128)
    pay[n - 64:] = last.payload[:64, :k // 2]
    b = R.matrix(n, k, R.DTYPE_FP4_E2M1, pay.data_ptr(), k, 1, sc.data_ptr(), k // 32)
    for m in (2, 300):
        a = Plain(m, k, torch.bfloat16, value=torch.randn(m, k, generator=torch.Generator().manual_seed(m)).bfloat16())
        o = Plain(m, n, torch.bfloat16)
        keep, args = room(R.reshard_group_matmul_workspace(a.m, b, o.m))
        R.reshard_group_matmul(a.m, b, o.m, *args, stream())
        torch.cuda.synchronize()
        av, bv = a.view.cpu().double().numpy(), last.values()
        check(o.view[:, n - 64:], av @ bv.T, np.abs(av) @ np.abs(bv).T, k + 1, "bf16")
        assert bool((o.view[:, :n - 64] == 0).all())
