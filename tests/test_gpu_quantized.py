"""GPU tests of the 8-bit refit over kinds of layouts: every destination rank's
payload and scales are those of quantizing the whole tensor, bit for bit."""
import numpy as np
import pytest
import torch

import block_reference as ref
import dtensor_layout_movement_amd as R
from block_reference import BLOCK, E4M3, E5M2
from dtensor_layout_movement_amd import workloads as W
from dtensor_layout_movement_amd.quantized import QuantizedPlan
from test_gpu_blocks import byte_buffers, stream, values_of

pytestmark = pytest.mark.gpu

T, RR = W.TensorSpec, W.R
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a visible MI355X")
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def indices(spec, side):
    """Per rank, the global indices of its rows and columns."""
    mesh, pl = getattr(spec, side + "_mesh"), getattr(spec, side + "_placements")
    h = R.layout_create(spec.shape, R.dtype_code(spec.dtype), mesh, pl, getattr(spec, side + "_split"))
    try:
        return [[np.concatenate([np.arange(lo, hi) for lo, hi in R.reshard_layout_shard_runs(h, r, d)] or
                                [np.arange(0)]) for d in range(2)]
                for r in range(R.reshard_layout_num_ranks(h))]
    finally:
        R.reshard_layout_destroy(h)


LISTS = {
    "rows to columns": [T("w", (512, 1024), BF16, (4,), (0,), (2,), (1,))],
    "columns to rows, both edges cut": [T("w", (300, 500), F32, (1,), (0,), (1,), (1,))],
    "edge blocks on the last ranks": [T("w", (511, 200), F16, (2,), (0,), (4,), (0,))],
    "columns with an edge": [T("w", (130, 1023), BF16, (4,), (1,), (2, 2), (RR, 1))],
    "replicas on both sides": [T("w", (256, 384), BF16, (2, 2), (RR, 0), (3, 2), (RR, 0))],
    "replicas to replicas": [T("w", (200, 300), F32, (3,), (RR,), (2,), (RR,))],
    "two mesh dims on two sides": [T("w", (512, 512), F32, (2, 2), (0, 1), (2, 2), (1, 0))],
    "strided rows": [T("w", (1024, 256), BF16, (2, 4), (0, 0), (2, 2), (RR, 1), src_split=(4, 1))],
    "strided on both sides": [T("w", (2048, 128), F16, (2, 2), (0, 0), (2, 4), (0, 0), src_split=(2, 1), dst_split=(4, 1))],
    "several tensors and types": [T("a", (256, 128), F32, (2,), (0,), (1,), (0,)), T("b", (128, 640), BF16, (1,), (0,), (5,), (1,)),
                                  T("c", (1, 1), F16, (1,), (0,), (1,), (1,)), T("d", (129, 257), F16, (2,), (RR,), (2,), (RR,))],
}


@pytest.mark.parametrize("fmt", [E4M3, E5M2])
@pytest.mark.parametrize("name", list(LISTS))
def test_every_destination_rank_holds_its_part_of_the_quantized_whole(name, fmt):
    specs = LISTS[name]
    whole = [values_of(s.shape, ("wide", "special", "border", "normal")[t % 4] if s.dtype == F32 else "normal", t, s.dtype)
             for t, s in enumerate(specs)]
    src = [[w[torch.from_numpy(r)][:, torch.from_numpy(c)].contiguous().cuda() for r, c in indices(s, "src")]
           for s, w in zip(specs, whole)]
    plan = QuantizedPlan(specs, fmt)
    try:
        bufs = {(side, what): [byte_buffers(getattr(plan, what + "_shapes")(t, side)) for t in range(len(specs))]
                for side in ("src", "dst") for what in ("payload", "scale")}
        ptrs = {k: [[b.data_ptr() for b in per] for per in v] for k, v in bufs.items()}
        bound = plan.bind([[s.data_ptr() for s in per] for per in src], ptrs["src", "payload"], ptrs["src", "scale"],
                          ptrs["dst", "payload"], ptrs["dst", "scale"])
        for _ in range(2):
            plan.execute(bound, stream())
        torch.cuda.synchronize()
        for t, (s, w) in enumerate(zip(specs, whole)):
            want, scales = ref.quantize(w, BLOCK, fmt)
            for rank, (rows, cols) in enumerate(indices(s, "dst")):
                assert plan.shard_shapes(t, "dst")[rank] == (len(rows), len(cols))
                q = bufs["dst", "payload"][t][rank].view(plan.payload_shapes(t, "dst")[rank])
                sc = bufs["dst", "scale"][t][rank].view(plan.scale_shapes(t, "dst")[rank])
                part = want[np.ix_(rows, cols)]
                assert np.array_equal(ref.values(q, sc, len(rows), len(cols), BLOCK, fmt), part, equal_nan=True), (t, rank)
                assert np.array_equal(sc.cpu().numpy(), scales[np.ix_(rows[::BLOCK] // BLOCK, cols[::BLOCK] // BLOCK)])
                assert bool((q[:, len(cols):] == 0).all())
        for per, w, s in zip(src, whole, specs):  # the sources are read only
            for x, (r, c) in zip(per, indices(s, "src")):
                y = w[torch.from_numpy(r)][:, torch.from_numpy(c)]
                assert torch.equal(x.cpu().view(torch.uint8), y.contiguous().view(torch.uint8))
    finally:
        plan.close()
