"""CPU tests of the block-scaled 8-bit operators: their refusals (every one is
decided on the host, before any device call) and the plain 64-bit reference
against torch's own 8-bit casts."""
import numpy as np
import pytest
import torch

import block_reference as ref
import dtensor_layout_movement_amd as R
from dtensor_layout_movement_amd import workloads as W
from dtensor_layout_movement_amd.quantized import QuantizedPlan

P = 0x100000  # addresses that no call below gets as far as using
F, H, E = R.DTYPE_F32, R.DTYPE_BF16, R.DTYPE_FP8_E4M3


def plain(rows, cols, dtype=H, data=P, stride=None):
    return R.matrix(rows, cols, dtype, data, stride)


def held(rows, cols, block_rows=1, data=2 * P, stride=None, scales=3 * P, scale_stride=None, dtype=E):
    return R.matrix(rows, cols, dtype, data, stride, block_rows, scales, scale_stride)


def refused(status, text, call, *args):
    with pytest.raises(R.ReshardError) as e:
        call(*args)
    assert e.value.status == status and text in str(e.value), str(e.value)


BAD, NULL = R.ERR_INVALID_ARGUMENT, R.ERR_NULL_SHARD


@pytest.mark.parametrize("src,dst,status,text", [
    (plain(4, 130, dtype=R.DTYPE_I32), held(4, 130), BAD, "src: dtype"),
    (plain(4, 130, dtype=R.DTYPE_F64), held(4, 130), BAD, "src: dtype"),
    (held(4, 130), held(4, 130, data=5 * P), BAD, "src: dtype"),
    (plain(4, 130), plain(4, 130, data=5 * P), BAD, "dst: dtype"),
    (plain(4, 130), held(4, 131), BAD, "differ in shape"),
    (plain(-1, 130), held(4, 130), BAD, "out of range"),
    (plain(2**31, 130), held(4, 130), BAD, "out of range"),
    (plain(4, 130, stride=129), held(4, 130), BAD, "row_stride"),
    (plain(4, 130, stride=-130), held(4, 130), BAD, "row_stride"),
    (plain(4, 130), held(4, 130, stride=144), BAD, "row_stride"),
    (plain(4, 130), held(4, 130, stride=264), BAD, "row_stride"),
    (plain(4, 130), held(4, 130, scale_stride=1), BAD, "scale_stride"),
    (plain(4, 130), held(4, 130, block_rows=64, stride=256, scale_stride=2), BAD, "block_rows"),
    (R.matrix(4, 130, H, P, 130, 1), held(4, 130), BAD, "block_rows"),
    (plain(4, 130, data=0), held(4, 130), NULL, "src: data"),
    (plain(4, 130), held(4, 130, data=0), NULL, "dst: data"),
    (plain(4, 130), held(4, 130, scales=0), NULL, "dst: scales"),
    (plain(4, 130, data=P + 1), held(4, 130), BAD, "misaligned"),
    (plain(4, 130), held(4, 130, data=2 * P + 8), BAD, "misaligned"),
    (plain(4, 130), held(4, 130, data=P + 512), BAD, "overlap"),
    (plain(4, 130), held(4, 130, scales=P), BAD, "overlap"),
    (plain(4, 130), held(4, 130, scales=2 * P + 1000), BAD, "overlap"),
])
def test_quantize_refusals(src, dst, status, text):
    refused(status, text, R.reshard_block_quantize, src, dst)


@pytest.mark.parametrize("dst,dst_t,status,text", [
    (held(200, 130, 128), held(130, 201, 128, data=5 * P, scales=6 * P), BAD, "transposed"),
    (held(200, 130, 1), held(130, 200, 128, data=5 * P, scales=6 * P), BAD, "128 rows"),
    (held(200, 130, 128), held(130, 200, 1, data=5 * P, scales=6 * P), BAD, "128 rows"),
    (held(200, 130, 128), held(130, 200, 128, data=5 * P, scales=6 * P, dtype=R.DTYPE_FP8_E5M2), BAD, "dtype"),
    (held(200, 130, 128), held(130, 200, 128, data=2 * P, scales=6 * P), BAD, "overlap"),
    (held(200, 130, 128), held(130, 200, 128, data=5 * P, scales=3 * P), BAD, "overlap"),
    (held(200, 130, 128), held(130, 200, 128, data=0, scales=3 * P), NULL, "dst_t"),
])
def test_transpose_refusals(dst, dst_t, status, text):
    refused(status, text, R.reshard_block_quantize, plain(200, 130), dst, dst_t)


@pytest.mark.parametrize("src,dst,status,text", [
    (plain(4, 130), plain(4, 130, data=5 * P), BAD, "src: dtype"),
    (held(4, 130), held(4, 130, data=5 * P), BAD, "dst: dtype"),
    (held(4, 130), plain(5, 130), BAD, "differ in shape"),
    (held(4, 130), plain(4, 130, data=2 * P), BAD, "overlap"),
    (held(4, 130), plain(4, 130, data=3 * P - 2), BAD, "overlap"),
    (held(4, 130), plain(4, 130, F, data=P + 2), BAD, "misaligned"),
])
def test_dequantize_refusals(src, dst, status, text):
    refused(status, text, R.reshard_block_dequantize, src, dst)


OUT = dict(data=7 * P)


@pytest.mark.parametrize("a,b,out,room,status,text", [
    (held(5, 130), plain(9, 130), plain(5, 9, **OUT), (0, 0), BAD, "b: dtype"),
    (held(5, 130), held(9, 131, 128, data=5 * P, scales=6 * P), plain(5, 9, **OUT), (0, 0), BAD, "contraction"),
    (held(5, 130), held(9, 130, 128, data=5 * P, scales=6 * P), plain(9, 5, **OUT), (0, 0), BAD, "out is not"),
    (held(5, 130), held(9, 130, 128, data=5 * P, scales=6 * P), held(5, 9, data=7 * P), (0, 0), BAD, "out: dtype"),
    (held(5, 130), held(9, 130, 128, data=5 * P, scales=6 * P), plain(5, 9, data=2 * P), (0, 0), BAD, "out overlaps a"),
    (held(5, 130), held(9, 130, 128, data=5 * P, scales=6 * P), plain(5, 9, data=6 * P), (0, 0), BAD, "out overlaps b"),
    (held(5, 130), held(9, 130, 128, data=0, scales=6 * P), plain(5, 9, **OUT), (0, 0), NULL, "b: data"),
    (plain(500, 130), held(9, 130, 128, data=5 * P, scales=6 * P), plain(500, 9, **OUT), (0, 0), BAD, "workspace of 0"),
    (plain(500, 130), held(9, 130, 128, data=5 * P, scales=6 * P), plain(500, 9, **OUT), (0, 1 << 20), BAD, "workspace is"),
    (plain(500, 130), held(9, 130, 128, data=5 * P, scales=6 * P), plain(500, 9, **OUT), (8 * P + 4, 1 << 20), BAD,
     "misaligned"),
    (plain(500, 130), held(9, 130, 128, data=5 * P, scales=6 * P), plain(500, 9, **OUT), (7 * P - 64, 1 << 20), BAD,
     "overlaps the workspace"),
])
def test_matmul_refusals(a, b, out, room, status, text):
    refused(status, text, R.reshard_block_matmul, a, b, out, *room)


def test_matmul_same_handle_twice_is_refused_as_an_overlap():
    x = plain(130, 130)
    refused(BAD, "overlap", R.reshard_block_matmul, x, held(130, 130, 128), x, 8 * P, 1 << 20)


def test_columns_of_one_larger_matrix_do_not_overlap():
    """a in the left, out in the right columns of rows of 512 elements: accepted as
    far as the device; one element more of either is not."""
    w = held(128, 256, 128, data=5 * P, scales=6 * P)
    room = (8 * P, 1 << 20)
    left = R.matrix(40, 256, H, P, 512)
    for out, ok in ((R.matrix(40, 128, H, P + 512, 512), True), (R.matrix(40, 128, H, P + 768, 512), True),
                    (R.matrix(40, 128, H, P + 510, 512), False), (R.matrix(40, 128, H, P + 770, 512), False),
                    (R.matrix(40, 128, H, P - 256, 512), True), (R.matrix(40, 128, H, P - 254, 512), False)):
        if not ok:
            refused(BAD, "out overlaps a", R.reshard_block_matmul, left, w, out, *room)
        elif not torch.cuda.is_available():
            refused(R.ERR_HIP, "hipGetDevice", R.reshard_block_matmul, left, w, out, *room)


@pytest.mark.parametrize("dy,x,dw,status,text", [
    (held(5, 9, data=5 * P), held(5, 130), plain(9, 130, **OUT), BAD, "dy: dtype"),
    (plain(5, 9), plain(5, 130), plain(9, 130, **OUT), BAD, "x: dtype"),
    (plain(6, 9), held(5, 130), plain(9, 130, **OUT), BAD, "contraction"),
    (plain(5, 9), held(5, 130), plain(130, 9, **OUT), BAD, "dw is not"),
    (plain(5, 9), held(5, 130), plain(9, 130), BAD, "dw overlaps dy"),
    (plain(5, 9), held(5, 130), plain(9, 130, data=0), NULL, "dw: data"),
    (plain(5, 9), held(5, 130, scales=0), plain(9, 130, **OUT), NULL, "x: scales"),
])
def test_grad_refusals(dy, x, dw, status, text):
    refused(status, text, R.reshard_block_grad, dy, x, dw, False, 8 * P, 1 << 30)


def test_workspace_queries_check_shapes_and_need_no_pointers():
    a, b, o = R.matrix(500, 300, H, 0), R.matrix(70, 300, E, 0, None, 128), R.matrix(500, 70, H, 0)
    assert R.reshard_block_matmul_workspace(a, b, o) >= 500 * 384 + 500 * 3
    q = R.matrix(500, 300, E, 0, None, 1)
    assert R.reshard_block_matmul_workspace(q, b, o) >= 0
    assert R.reshard_block_grad_workspace(o, q, R.matrix(70, 300, F, 0)) >= 0
    refused(BAD, "contraction", R.reshard_block_matmul_workspace, R.matrix(500, 301, H, 0), b, o)
    refused(BAD, "dw is not", R.reshard_block_grad_workspace, o, q, R.matrix(71, 300, F, 0))


def test_strides_of_matrices_without_elements_mean_nothing():
    # no contraction: a and b have no elements, and rows any distance apart
    a, b = R.matrix(70, 0, E, None, 1 << 40, 1, None, -5), R.matrix(9, 0, E, None, 1 << 24, 128, None, 0)
    assert R.reshard_block_matmul_workspace(a, b, plain(70, 9)) == 0
    # no columns of out: b has no elements
    b = R.matrix(0, 130, E, None, 1 << 24, 128, None, 0)
    assert R.reshard_block_matmul_workspace(held(70, 130), b, R.matrix(70, 0, H, None, -1)) == 0
    # with elements on both sides the limit holds
    refused(BAD, "2^23", R.reshard_block_matmul_workspace, held(70, 130), held(9, 130, 128, stride=1 << 24), plain(70, 9))


@pytest.mark.parametrize("rows,ok", [((1 << 27) - 16, True), ((1 << 27) - 15, False), (1 << 30, False)])
def test_products_of_more_workgroups_than_one_launch_takes_are_refused(rows, ok):
    """2^23 - 1 at most, with few rows one for each 16 columns of out."""
    w, out = held(rows, 100, 128), R.matrix(1, rows, H, P)
    if ok:
        assert R.reshard_block_matmul_workspace(plain(1, 100), w, out) == 0
    else:
        refused(BAD, "too many tiles", R.reshard_block_matmul_workspace, plain(1, 100), w, out)
        refused(BAD, "too many tiles", R.reshard_block_matmul, plain(1, 100), w, out)


@pytest.mark.parametrize("rows,ok", [((1 << 27) - 128, True), ((1 << 27) - 127, False), (1 << 30, False)])
def test_weights_of_more_blocks_than_one_launch_takes_are_refused(rows, ok):
    """2^23 - 1 blocks of 128 x 128 at most, here eight for each 128 rows."""
    src, dst = plain(rows, 1024), held(rows, 1024, 128, data=1 << 45, scales=1 << 50)
    if not ok:
        refused(BAD, "too many tiles", R.reshard_block_quantize, src, dst)
    elif not torch.cuda.is_available():
        refused(R.ERR_HIP, "hipGetDevice", R.reshard_block_quantize, src, dst)


def test_valid_calls_fail_cleanly_without_a_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is visible")
    refused(R.ERR_HIP, "hipGetDevice", R.reshard_block_quantize, plain(4, 130), held(4, 130))
    refused(R.ERR_HIP, "hipGetDevice", R.reshard_block_dequantize, held(4, 130), plain(4, 130))
    w = held(9, 130, 128, data=5 * P, scales=6 * P)
    refused(R.ERR_HIP, "hipGetDevice", R.reshard_block_matmul, held(5, 130), w, plain(5, 9, **OUT))
    refused(R.ERR_HIP, "hipGetDevice", R.reshard_block_grad, plain(5, 9), held(5, 130), plain(9, 130, **OUT), False,
            8 * P, 1 << 30)


def test_reference_decodes_and_rounds_as_torch_does():
    codes = torch.arange(256, dtype=torch.uint8)
    for fmt, t in ((ref.E4M3, torch.float8_e4m3fn), (ref.E5M2, torch.float8_e5m2)):
        table = ref.decode_table(fmt)
        want = codes.view(t).float().double().numpy()
        assert np.array_equal(table, want, equal_nan=True)
        g = torch.Generator().manual_seed(5)
        x = torch.randn(20000, generator=g) * torch.exp2(torch.randint(-20, 9, (20000,), generator=g).float())
        x = x.clamp(-ref.TOP[fmt], ref.TOP[fmt])
        fin = table[np.isfinite(table)]
        ties = (np.sort(fin)[1:] + np.sort(fin)[:-1]) / 2  # midpoints of neighbouring values
        x = torch.cat([x, torch.from_numpy(ties).float()])
        assert np.array_equal(ref.round_to_format(x.double().numpy(), fmt), x.to(t).float().double().numpy())


# ---------------------------------------------------------------- refit plans

T = W.TensorSpec
BF, RR = torch.bfloat16, W.R


def test_quantized_plan_shapes():
    with_edge = T("up", (1000, 300), BF, (2,), (0,), (2, 2), (RR, 1))  # rows cut at 500: inside a block
    with pytest.raises(ValueError, match="inside a block"):
        QuantizedPlan([with_edge])
    p = QuantizedPlan([T("up", (1000, 511), BF, (1,), (0,), (2, 2), (RR, 1)),
                       T("down", (512, 1024), torch.float32, (2,), (1,), (4,), (0,))])
    try:
        assert p.payload_shapes(0, "dst") == [(1000, 256)] * 4
        assert p.shard_shapes(0, "dst") == [(1000, 256), (1000, 255)] * 2  # columns cut at 256, the edge at 511
        assert p.scale_shapes(0, "dst") == [(8, 2)] * 4
        assert p.payload_shapes(1, "src") == [(512, 512)] * 2 and p.scale_shapes(1, "dst") == [(1, 8)] * 4
        st = R.reshard_plan_stats(p.plan)
        assert st["bytes_written"] == 2 * (1000 * 512 + 8 * 4) + 512 * 1024 + 4 * 8
        assert p.bytes_moved() > st["bytes_read"] + st["bytes_written"]
    finally:
        p.close()


@pytest.mark.parametrize("spec,text", [
    (T("e", (4, 256, 256), BF, (1,), (0,), (1,), (0,)), "2-d"),
    (T("i", (256, 256), torch.int32, (1,), (0,), (1,), (0,)), "dtype"),
    (T("p", (256, 256), BF, (2,), (W.P,), (1,), (0,)), "Partial"),
    (T("c", (256, 300), BF, (1,), (0,), (2,), (1,)), "inside a block"),
])
def test_quantized_plan_refusals(spec, text):
    with pytest.raises(ValueError, match=text):
        QuantizedPlan([spec])


def test_quantized_plan_refuses_other_formats_and_empty_lists():
    with pytest.raises(ValueError, match="FP8"):
        QuantizedPlan([T("u", (256, 256), BF, (1,), (0,), (1,), (0,))], dtype=R.DTYPE_BF16)
    with pytest.raises(ValueError, match="at least one"):
        QuantizedPlan([])


@pytest.mark.parametrize("wl", [W.ffn_up(), W.ffn_refit(4), W.ffn_up_fsdp2_tp()], ids=lambda w: w.name)
def test_quantized_plan_takes_the_dense_workloads(wl):
    p = QuantizedPlan(wl.tensors)
    try:
        for t, spec in enumerate(wl.tensors):
            for side in ("src", "dst"):
                assert all(c % 128 == 0 for _, c in p.payload_shapes(t, side))
        direct = sum(2 * spec.shape[0] * spec.shape[1] for spec in wl.tensors)
        assert R.reshard_plan_stats(p.plan)["bytes_read"] < 0.51 * direct  # a byte an element, and the scales
    finally:
        p.close()
