"""CPU tests of the group-scaled 4-bit operators and of tokens sorted by expert:
their refusals (every one is decided on the host, before any device call) and the
plain 64-bit reference."""
import numpy as np
import pytest
import torch

import dtensor_layout_movement_amd as R
import group_reference as ref
from test_blocks import BAD, NULL, P, held, plain, refused

F, H, I4 = R.DTYPE_F32, R.DTYPE_BF16, R.DTYPE_FP4_E2M1
OUT = dict(data=7 * P)


def grouped(rows, cols, data=2 * P, stride=None, scales=3 * P, scale_stride=None, block_rows=1):
    return R.matrix(rows, cols, I4, data, stride, block_rows, scales, scale_stride)


def no_gpu(call, *args):
    """A valid call gets as far as the device."""
    if not torch.cuda.is_available():
        refused(R.ERR_HIP, "hipGetDevice", call, *args)


def test_strides_of_a_described_matrix_default_to_the_smallest():
    m = grouped(4, 65)
    assert (m.row_stride, m.scale_stride, m.block_rows) == (96, 3, 1)
    assert R.reshard_dtype_size(I4) == 0  # no layout holds it
    with pytest.raises(R.ReshardError, match="dtype"):
        R.reshard_layout_create((32, 32), I4, (1,), (0,))


@pytest.mark.parametrize("src,dst,status,text", [
    (plain(4, 70, dtype=R.DTYPE_I32), grouped(4, 70), BAD, "src: dtype"),
    (held(4, 70), grouped(4, 70, data=5 * P), BAD, "src: dtype"),
    (grouped(4, 70), grouped(4, 70, data=5 * P), BAD, "src: dtype"),
    (plain(4, 70), plain(4, 70, data=5 * P), BAD, "dst: dtype"),
    (plain(4, 70), held(4, 70), BAD, "dst: dtype"),
    (plain(4, 70), grouped(4, 71), BAD, "differ in shape"),
    (plain(-1, 70), grouped(4, 70), BAD, "out of range"),
    (plain(4, 70, stride=69), grouped(4, 70), BAD, "row_stride"),
    (plain(4, 70), grouped(4, 70, stride=64), BAD, "row_stride"),
    (plain(4, 70), grouped(4, 70, stride=112), BAD, "row_stride"),
    (plain(4, 70), grouped(4, 70, scale_stride=2), BAD, "scale_stride"),
    (plain(4, 70), grouped(4, 70, block_rows=128), BAD, "block_rows"),
    (plain(4, 70), R.matrix(4, 70, I4, 2 * P, 96, 0, 3 * P, 3), BAD, "block_rows"),
    (plain(4, 70, data=0), grouped(4, 70), NULL, "src: data"),
    (plain(4, 70), grouped(4, 70, data=0), NULL, "dst: data"),
    (plain(4, 70), grouped(4, 70, scales=0), NULL, "dst: scales"),
    (plain(4, 70, data=P + 1), grouped(4, 70), BAD, "misaligned"),
    (plain(4, 70), grouped(4, 70, data=2 * P + 8), BAD, "misaligned"),
    (plain(4, 70), grouped(4, 70, data=P + 512), BAD, "overlap"),
    (plain(4, 70), grouped(4, 70, scales=P + 559), BAD, "overlap"),
    (plain(4, 70), grouped(4, 70, scales=2 * P + 191), BAD, "overlap"),
])
def test_quantize_refusals(src, dst, status, text):
    refused(status, text, R.reshard_group_quantize, src, dst)


def test_neighbours_in_memory_are_no_overlap():
    no_gpu(R.reshard_group_quantize, plain(4, 70), grouped(4, 70, data=P + 560))
    no_gpu(R.reshard_group_quantize, plain(4, 70), grouped(4, 70, scales=2 * P + 192))
    # payloads of two weights as columns of one buffer
    no_gpu(R.reshard_group_dequantize, grouped(4, 64, stride=128), plain(4, 64, data=5 * P))


@pytest.mark.parametrize("src,dst,status,text", [
    (plain(4, 70), plain(4, 70, data=5 * P), BAD, "src: dtype"),
    (held(4, 70), plain(4, 70, data=5 * P), BAD, "src: dtype"),
    (grouped(4, 70), grouped(4, 70, data=5 * P), BAD, "dst: dtype"),
    (grouped(4, 70), plain(5, 70), BAD, "differ in shape"),
    (grouped(4, 70), plain(4, 70, data=2 * P), BAD, "overlap"),
    (grouped(4, 70), plain(4, 70, data=3 * P - 2), BAD, "overlap"),
])
def test_dequantize_refusals(src, dst, status, text):
    refused(status, text, R.reshard_group_dequantize, src, dst)


W = dict(data=5 * P, scales=6 * P)


@pytest.mark.parametrize("a,b,out,status,text", [
    (held(5, 70), grouped(9, 70, **W), plain(5, 9, **OUT), BAD, "a: dtype"),
    (grouped(5, 70), grouped(9, 70, **W), plain(5, 9, **OUT), BAD, "a: dtype"),
    (plain(5, 70), held(9, 70, 128, **W), plain(5, 9, **OUT), BAD, "b: dtype"),
    (plain(5, 70), plain(9, 70, data=5 * P), plain(5, 9, **OUT), BAD, "b: dtype"),
    (plain(5, 70), grouped(9, 71, **W), plain(5, 9, **OUT), BAD, "contraction"),
    (plain(5, 70), grouped(9, 70, **W), plain(9, 5, **OUT), BAD, "out is not"),
    (plain(5, 70), grouped(9, 70, **W), grouped(5, 9, data=7 * P, scales=8 * P), BAD, "out: dtype"),
    (plain(5, 70), grouped(9, 70, **W), plain(5, 9), BAD, "out overlaps a"),
    (plain(5, 70), grouped(9, 70, **W), plain(5, 9, data=6 * P), BAD, "out overlaps b"),
    (plain(5, 70), grouped(9, 70, data=0, scales=6 * P), plain(5, 9, **OUT), NULL, "b: data"),
    (plain(5, 70), grouped(9, 70, data=5 * P, scales=0), plain(5, 9, **OUT), NULL, "b: scales"),
    (plain(5, 70, data=0), grouped(9, 70, **W), plain(5, 9, **OUT), NULL, "a: data"),
])
def test_matmul_refusals(a, b, out, status, text):
    refused(status, text, R.reshard_group_matmul, a, b, out, 8 * P, 1 << 30)


@pytest.mark.parametrize("offsets,experts,b,out,status,text", [
    (4 * P, 0, grouped(18, 70, **W), plain(5, 9, **OUT), BAD, "experts is not"),
    (4 * P, -2, grouped(18, 70, **W), plain(5, 9, **OUT), BAD, "experts is not"),
    (4 * P, 1025, grouped(1025, 70, **W), plain(5, 1, **OUT), BAD, "experts is not"),
    (4 * P, 2, grouped(19, 70, **W), plain(5, 9, **OUT), BAD, "equal rows"),
    (4 * P, 2, grouped(18, 70, **W), plain(5, 18, **OUT), BAD, "out is not"),
    (0, 2, grouped(18, 70, **W), plain(5, 9, **OUT), NULL, "offsets"),
    (4 * P + 2, 2, grouped(18, 70, **W), plain(5, 9, **OUT), BAD, "offsets: misaligned"),
    (7 * P + 80, 2, grouped(18, 70, **W), plain(5, 9, **OUT), BAD, "out overlaps offsets"),
])
def test_expert_matmul_refusals(offsets, experts, b, out, status, text):
    refused(status, text, R.reshard_expert_matmul, plain(5, 70), b, offsets, experts, out, 8 * P, 1 << 30)


def test_workspaces_are_asked_for_and_checked():
    # fp32 rows are cut into parts in memory where large tiles read them
    a, b, o = R.matrix(700, 300, F, 0), R.matrix(8192, 300, I4, 0, None, 1), R.matrix(700, 8192, H, 0)
    need = R.reshard_group_matmul_workspace(a, b, o)
    assert R.reshard_expert_matmul_workspace(a, R.matrix(4 * 8192, 300, I4, 0, None, 1), 4, o) >= 0
    refused(BAD, "contraction", R.reshard_group_matmul_workspace, R.matrix(700, 301, F, 0), b, o)
    refused(BAD, "experts is not", R.reshard_expert_matmul_workspace, a, b, 0, o)
    if need:
        a, b, o = plain(700, 300, F), grouped(8192, 300, data=1 << 40, scales=1 << 41), plain(700, 8192, data=1 << 42)
        refused(BAD, "workspace of", R.reshard_group_matmul, a, b, o, 1 << 43, need - 1)
        refused(BAD, "workspace is NULL", R.reshard_group_matmul, a, b, o, 0, need)
        refused(BAD, "workspace is misaligned", R.reshard_group_matmul, a, b, o, (1 << 43) + 8, need)
        refused(BAD, "overlaps the workspace", R.reshard_group_matmul, a, b, o, 1 << 42, need)


@pytest.mark.parametrize("change,status,text", [
    (dict(ids_dtype=R.DTYPE_I16), BAD, "ids: dtype"),
    (dict(ids_dtype=F), BAD, "ids: dtype"),
    (dict(choices=0), BAD, "choices"),
    (dict(choices=65), BAD, "choices"),
    (dict(tokens=-1), BAD, "tokens"),
    (dict(tokens=1 << 28), BAD, "tokens"),
    (dict(tokens=1 << 62), BAD, "tokens"),
    (dict(experts=0), BAD, "experts"),
    (dict(experts=1025), BAD, "experts"),
    (dict(first=-1), BAD, "first"),
    (dict(first=1 << 41), BAD, "first"),
    (dict(ids=0), NULL, "ids"),
    (dict(ids=P + 4), BAD, "ids: misaligned"),
    (dict(offsets=0), NULL, "offsets"),
    (dict(offsets=5 * P + 2), BAD, "offsets: misaligned"),
    (dict(position=0), NULL, "position"),
    (dict(position=P + 100), BAD, "position overlaps ids"),
    (dict(position=5 * P + 32), BAD, "offsets overlaps position"),
    (dict(room=(0, 0), tokens=5000), BAD, "workspace of 0"),
    (dict(room=(9 * P + 8, 1 << 20), tokens=5000), BAD, "workspace is misaligned"),
])
def test_sort_refusals(change, status, text):
    c = dict(ids=P, ids_dtype=R.DTYPE_I64, tokens=20, choices=5, first=0, experts=8, offsets=5 * P, position=7 * P,
             room=(9 * P, 1 << 20))
    c.update(change)
    room = c.pop("room")
    refused(status, text, R.reshard_expert_sort, *c.values(), *room)


def test_sort_workspace():
    assert R.reshard_expert_sort_workspace(0, 8, 64) == 0
    assert R.reshard_expert_sort_workspace(1, 8, 64) == 0
    assert 0 < R.reshard_expert_sort_workspace(1 << 24, 64, 1024) <= 1 << 20
    refused(BAD, "experts", R.reshard_expert_sort_workspace, 4, 8, 2000)
    refused(BAD, "choices", R.reshard_expert_sort_workspace, 4, 80, 64)


@pytest.mark.parametrize("x,position,choices,rows,status,text", [
    (plain(4, 70), 5 * P, 2, plain(8, 71, data=7 * P), BAD, "columns"),
    (plain(4, 70), 5 * P, 2, plain(8, 70, F, data=7 * P), BAD, "dtype"),
    (plain(4, 70), 5 * P, 2, held(8, 70), BAD, "rows: dtype"),
    (held(4, 70), 5 * P, 2, plain(8, 70, data=7 * P), BAD, "x: dtype"),
    (plain(4, 70), 5 * P, 0, plain(8, 70, data=7 * P), BAD, "choices"),
    (plain(4, 70), 0, 2, plain(8, 70, data=7 * P), NULL, "position"),
    (plain(4, 70), 5 * P + 1, 2, plain(8, 70, data=7 * P), BAD, "position: misaligned"),
    (plain(4, 70), 5 * P, 2, plain(8, 70), BAD, "rows overlaps x"),
    (plain(4, 70), 7 * P + 1116, 2, plain(8, 70, data=7 * P), BAD, "rows overlaps position"),
    (plain(4, 70), 5 * P, 2, plain(8, 70, data=0), NULL, "rows: data"),
])
def test_gather_refusals(x, position, choices, rows, status, text):
    refused(status, text, R.reshard_expert_gather, x, position, choices, rows)


@pytest.mark.parametrize("rows,position,choices,weights,out,status,text", [
    (plain(8, 70), 5 * P, 2, None, plain(4, 71, data=7 * P), BAD, "columns"),
    (plain(8, 70), 5 * P, 2, None, plain(4, 70, F, data=7 * P), BAD, "dtype"),
    (plain(8, 70), 5 * P, 2, plain(4, 3, data=9 * P), plain(4, 70, data=7 * P), BAD, "weights: is not tokens x choices"),
    (plain(8, 70), 5 * P, 2, plain(4, 2, R.DTYPE_I32, data=9 * P), plain(4, 70, data=7 * P), BAD, "weights: dtype"),
    (plain(8, 70), 5 * P, 2, plain(4, 2, data=0), plain(4, 70, data=7 * P), NULL, "weights: data"),
    (plain(8, 70), 5 * P, 2, plain(4, 2, data=7 * P), plain(4, 70, data=7 * P), BAD, "out overlaps weights"),
    (plain(8, 70), 5 * P, 65, None, plain(4, 70, data=7 * P), BAD, "choices"),
    (plain(8, 70), 0, 2, None, plain(4, 70, data=7 * P), NULL, "position"),
    (plain(8, 70), 5 * P, 2, None, plain(4, 70), BAD, "out overlaps rows"),
    (plain(8, 70, data=0), 5 * P, 2, None, plain(4, 70, data=7 * P), NULL, "rows: data"),
])
def test_combine_refusals(rows, position, choices, weights, out, status, text):
    refused(status, text, R.reshard_expert_combine, rows, position, choices, weights, out)


D, Y, DR, DW, PW = plain(4, 70), plain(8, 70, data=2 * P), plain(8, 70, data=3 * P), plain(4, 2, F, data=4 * P), plain(4, 2, F, data=6 * P)


@pytest.mark.parametrize("dout,rows,position,weights,drows,dweights,status,text", [
    (D, Y, 5 * P, PW, None, None, BAD, "neither"),
    (D, None, 5 * P, PW, DR, DW, BAD, "rows: matrix is NULL"),
    (D, plain(8, 71, data=2 * P), 5 * P, PW, DR, DW, BAD, "rows and dout differ in columns"),
    (D, plain(8, 70, F, data=2 * P), 5 * P, PW, DR, DW, BAD, "rows and dout differ in dtype"),
    (D, Y, 5 * P, PW, plain(8, 71, data=3 * P), DW, BAD, "drows and dout differ in columns"),
    (D, Y, 5 * P, PW, plain(8, 70, F, data=3 * P), DW, BAD, "drows and dout differ in dtype"),
    (D, Y, 5 * P, PW, plain(9, 70, data=3 * P), DW, BAD, "drows and rows differ"),
    (D, Y, 5 * P, plain(4, 3, F, data=6 * P), DR, DW, BAD, "weights: is not"),
    (D, Y, 5 * P, PW, DR, plain(5, 2, F, data=4 * P), BAD, "dweights: is not"),
    (D, Y, 5 * P, PW, Y, DW, BAD, "overlaps"),
    (D, Y, 5 * P, PW, DR, plain(4, 2, F, data=6 * P), BAD, "overlaps weights"),
    (D, Y, 0, PW, DR, DW, NULL, "position"),
    (D, plain(8, 70, data=0), 5 * P, PW, DR, DW, NULL, "rows: data"),
])
def test_combine_grad_refusals(dout, rows, position, weights, drows, dweights, status, text):
    refused(status, text, R.reshard_expert_combine_grad, dout, rows, position, 2, weights, drows, dweights)


def test_valid_calls_get_as_far_as_the_device():
    no_gpu(R.reshard_group_quantize, plain(4, 70), grouped(4, 70))
    no_gpu(R.reshard_group_dequantize, grouped(4, 70), plain(4, 70))
    no_gpu(R.reshard_group_matmul, plain(5, 70), grouped(9, 70, **W), plain(5, 9, **OUT), 8 * P, 1 << 30)
    no_gpu(R.reshard_expert_matmul, plain(5, 70), grouped(18, 70, **W), 4 * P, 2, plain(5, 9, **OUT), 8 * P, 1 << 30)
    no_gpu(R.reshard_expert_sort, P, R.DTYPE_I32, 20, 5, 0, 8, 5 * P, 7 * P)
    no_gpu(R.reshard_expert_sort, 0, R.DTYPE_I32, 0, 5, 0, 8, 5 * P, 0)  # no tokens: offsets of zero are written
    no_gpu(R.reshard_expert_gather, plain(4, 70), 5 * P, 2, plain(8, 70, data=7 * P))
    no_gpu(R.reshard_expert_combine, plain(8, 70), 5 * P, 2, None, plain(4, 70, data=7 * P))
    no_gpu(R.reshard_expert_combine, plain(8, 70), 5 * P, 2, PW, plain(4, 70, data=7 * P))
    no_gpu(R.reshard_expert_combine_grad, D, Y, 5 * P, 2, PW, DR, DW)
    no_gpu(R.reshard_expert_combine_grad, D, None, 5 * P, 2, PW, DR, None)
    no_gpu(R.reshard_expert_combine_grad, D, Y, 5 * P, 2, None, None, DW)


@pytest.mark.parametrize("rows,ok", [((1 << 27) - 16, True), (1 << 30, False)])
def test_products_of_more_workgroups_than_one_launch_takes_are_refused(rows, ok):
    w, out = grouped(rows, 100, scales=1 << 50), R.matrix(1, rows, H, P)
    if ok:
        assert R.reshard_group_matmul_workspace(plain(1, 100), w, out) >= 0
    else:
        refused(BAD, "too many tiles", R.reshard_group_matmul_workspace, plain(1, 100), w, out)


def test_reference_rounds_ties_to_even_codes():
    v = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    assert list(ref.round_to_format(v)) == [0, 2, 2, 4, 4, 6, 6]
    assert list(ref.round_to_format(np.nextafter(v, 0))) == [0, 1, 2, 3, 4, 5, 6]
    assert list(ref.round_to_format(np.nextafter(v, 9))) == [1, 2, 3, 4, 5, 6, 7]
    x = torch.tensor([[6.0] + [0.0] * 31 + [6.0000005] + [1.0] * 3])
    got, scales = ref.quantize(x)
    assert list(scales[0]) == [127, 128] and got[0, 32] == 6.0 and got[0, 33] == 1.0
    assert ref.quantize(torch.zeros(1, 5))[1][0, 0] == 127


def test_reference_sorts_in_order():
    ids = np.array([[3, 1], [1, 9], [-1, 3], [1, 3]])
    offsets, position = ref.sort(ids, 1, 3)
    assert list(offsets) == [0, 3, 3, 6]
    assert position.tolist() == [[3, 0], [1, -1], [-1, 4], [2, 5]]


# ------------------------------------------------------------- refit to 4 bits

from dtensor_layout_movement_amd import workloads as WL  # noqa: E402
from dtensor_layout_movement_amd.quantized import QuantizedPlan  # noqa: E402

T, BF, RR = WL.TensorSpec, torch.bfloat16, WL.R


def test_four_bit_plan_shapes():
    p = QuantizedPlan([T("up", (1000, 511), BF, (3,), (0,), (2, 2), (RR, 1)),
                       T("experts", (8, 40, 96), torch.float32, (4, 2), (0, 1), (2, 3), (0, 2))], R.DTYPE_FP4_E2M1)
    try:
        assert p.shard_shapes(0, "src") == [(334, 511), (334, 511), (332, 511)]  # rows are cut anywhere
        assert p.payload_shapes(0, "dst") == [(1000, 128)] * 4 and p.scale_shapes(0, "dst") == [(1000, 8)] * 4
        assert p.shard_shapes(0, "dst") == [(1000, 256), (1000, 255)] * 2
        assert p.shard_shapes(1, "src") == [(40, 96)] * 8 and p.shard_shapes(1, "dst") == [(160, 32)] * 6
        assert p.payload_shapes(1, "dst") == [(160, 16)] * 6 and p.scale_shapes(1, "dst") == [(160, 1)] * 6
        m = p.weight(1, 0, P, 2 * P)
        assert (m.rows, m.cols, m.dtype, m.block_rows, m.row_stride, m.scale_stride) == (160, 32, I4, 1, 32, 1)
        st = R.reshard_plan_stats(p.plan)
        assert st["bytes_written"] == 2 * 1000 * (256 + 16) + 8 * 40 * (48 + 3)
    finally:
        p.close()


@pytest.mark.parametrize("spec,text", [
    (T("c", (256, 300), BF, (1,), (0,), (2,), (1,)), "inside a block of 32"),
    (T("s", (2, 2, 64, 64), BF, (1,), (0,), (1,), (0,)), "2-d weights are quantized, and 3-d"),
    (T("p", (256, 256), BF, (2,), (WL.P,), (1,), (0,)), "Partial"),
    (T("i", (256, 256), torch.int32, (1,), (0,), (1,), (0,)), "dtype"),
])
def test_four_bit_plan_refusals(spec, text):
    with pytest.raises(ValueError, match=text):
        QuantizedPlan([spec], R.DTYPE_FP4_E2M1)


@pytest.mark.parametrize("wl", [WL.ffn_up(), WL.ffn_refit(4), WL.moe_experts()], ids=lambda w: w.name)
def test_four_bit_plan_takes_the_workloads(wl):
    p = QuantizedPlan(wl.tensors, R.DTYPE_FP4_E2M1)
    try:
        direct = sum(2 * int(np.prod(spec.shape)) for spec in wl.tensors)
        assert R.reshard_plan_stats(p.plan)["bytes_read"] == direct // 4 + direct // 64
    finally:
        p.close()
