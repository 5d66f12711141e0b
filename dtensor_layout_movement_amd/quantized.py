"""Refit of trained weights to an 8-bit or a 4-bit inference layout.

The pages mention that the refit supports precision modes and say nothing more
(the news.bpdata.com and techfeed.io write-ups, closing remarks on the refit
guide).  The reading taken here: the trainer holds fp32, bf16 or fp16 weights,
the inference engine 8-bit ones with a power-of-two scale for each block of
128 x 128 (the block-scaled format of ``include/reshard.h``), or 4-bit ones with
one for each group of 32 columns (the group-scaled format), experts stacked in
front among them.  Every source shard is quantized where it lies and one reshard
then moves payload and scales, so that the move carries one byte an element, or
half of one, instead of two or four, and every destination replica receives the
same bytes.

Blocks must not be cut: every shard's runs start at a multiple of 128 (of 32 along
the columns of a 4-bit weight, whose rows may be cut anywhere) and end at one or
at the tensor's edge, on both sides; other layouts are refused.  The result is
then that of quantizing the whole tensor.
"""
from __future__ import annotations

from . import reshard as R

FLOATS = (R.DTYPE_F32, R.DTYPE_BF16, R.DTYPE_F16)


def _blocks(n: int, block: int = R.BLOCK) -> int:
    return -(-n // block)


class QuantizedPlan:
    """Plan for a list of 2-d weights, with ``DTYPE_FP4_E2M1`` of 3-d stacks of experts'
    too (objects with name, shape, dtype, src_mesh,
    src_placements, dst_mesh, dst_placements and optionally src_split / dst_split,
    e.g. workloads.TensorSpec; out_dtype is not looked at).

    The caller owns all buffers, as for a plain plan.  Per tensor: the source
    shards (contiguous, the spec's dtype), a payload and a scale buffer for each
    source rank, and a payload and a scale buffer for each destination rank, of
    ``payload_shapes`` and ``scale_shapes`` (one byte an element, contiguous;
    payload columns are rounded up to whole blocks).  In 4 bits a shard of a stack is
    one matrix, its experts' rows one below the other, and its payload's columns count
    bytes of two elements.
    """

    def __init__(self, specs, dtype: int = R.DTYPE_FP8_E4M3):
        self.specs = list(specs)
        self.dtype = dtype
        # columns and rows of a block, columns of a block's payload in bytes
        self._cols, self._rows, self._bytes = (
            (R.GROUP, 1, R.GROUP // 2) if dtype == R.DTYPE_FP4_E2M1 else (R.BLOCK, R.BLOCK, R.BLOCK))
        self.plan = None
        self._layouts = []
        try:
            self._build()
        except Exception:
            self.close()
            raise

    def _layout(self, *args):
        h = R.layout_create(*args)
        self._layouts.append(h)
        return h

    def _build(self):
        if not self.specs:
            raise ValueError("need at least one tensor")
        if self.dtype not in (R.DTYPE_FP8_E4M3, R.DTYPE_FP8_E5M2, R.DTYPE_FP4_E2M1):
            raise ValueError("dtype is not FP8_E4M3, FP8_E5M2 or FP4_E2M1")
        stacks = self.dtype == R.DTYPE_FP4_E2M1
        payload, scales = {"src": [], "dst": []}, {"src": [], "dst": []}
        self._shapes = {"src": [], "dst": []}  # per tensor, per rank: (rows, cols) of the shard
        for spec in self.specs:
            if len(spec.shape) != 2 and not (stacks and len(spec.shape) == 3):
                raise ValueError(f"{spec.name}: only 2-d weights are quantized" + (", and 3-d stacks" if stacks else ""))
            if R.dtype_code(spec.dtype) not in FLOATS:
                raise ValueError(f"{spec.name}: dtype is not F32, BF16 or F16")
            if R.PARTIAL in tuple(spec.src_placements):
                raise ValueError(f"{spec.name}: Partial contributions cannot be quantized before they are added")
            *lead, n, k = spec.shape
            grid = (*lead, _blocks(n, self._rows), _blocks(k, self._cols))
            for side in ("src", "dst"):
                mesh, pl = getattr(spec, side + "_mesh"), getattr(spec, side + "_placements")
                split = getattr(spec, side + "_split", None)
                whole = self._layout(spec.shape, R.dtype_code(spec.dtype), mesh, pl, split)
                held = self._layout((*lead, n, grid[-1] * self._bytes), R.DTYPE_U8 if stacks else self.dtype, mesh, pl,
                                    split)
                scale = self._layout(grid, R.DTYPE_U8, mesh, pl, split)
                shapes = []
                for rank in range(R.reshard_layout_num_ranks(whole)):
                    self._check_cuts(spec, side, rank, whole, held, scale)
                    *outer, rows, cols = R.local_shape(whole, rank, len(spec.shape))
                    for m in outer:
                        rows *= m
                    shapes.append((rows, cols))
                self._shapes[side].append(shapes)
                payload[side].append(held)
                scales[side].append(scale)
        self.plan = R.reshard_plan_create_batched(payload["src"] + scales["src"], payload["dst"] + scales["dst"])
        load = R.reshard_plan_src_load(self.plan)
        # source ranks whose shard the move reads (of replicated shards, one or a few)
        self._read, at = [], 0
        for shapes in self._shapes["src"]:
            self._read.append([load[at + r] > 0 for r in range(len(shapes))])
            at += len(shapes)
        for t, shapes in enumerate(self._shapes["src"]):
            for r in range(len(shapes)):
                self._read[t][r] |= load[at + r] > 0
            at += len(shapes)

    def _check_cuts(self, spec, side, rank, whole, held, scale):
        last = len(spec.shape) - 1
        for dim, extent in enumerate(spec.shape):
            block = self._cols if dim == last else self._rows if dim == last - 1 else 1
            runs = R.reshard_layout_shard_runs(whole, rank, dim)
            for lo, hi in runs:
                if lo % block or (hi % block and hi != extent):
                    raise ValueError(f"{spec.name}: {side} rank {rank} cuts dim {dim} at [{lo}, {hi}), inside a "
                                     f"block of {block}")
            blocks = [(lo // block, _blocks(hi, block)) for lo, hi in runs]
            payload = [(lo * self._bytes, hi * self._bytes) for lo, hi in blocks] if dim == last else runs
            if (R.reshard_layout_shard_runs(held, rank, dim) != payload or
                    R.reshard_layout_shard_runs(scale, rank, dim) != blocks):
                raise ValueError(f"{spec.name}: {side} rank {rank} splits dim {dim} and its blocks differently")

    # ------------------------------------------------------------- buffers

    def shard_shapes(self, t: int, side: str):
        """(rows, cols) of each rank's shard; side is "src" or "dst"."""
        return list(self._shapes[side][t])

    def payload_shapes(self, t: int, side: str):
        """(rows, bytes of a row) of each rank's payload."""
        return [(r, _blocks(c, self._cols) * self._bytes) for r, c in self._shapes[side][t]]

    def scale_shapes(self, t: int, side: str):
        return [(_blocks(r, self._rows), _blocks(c, self._cols)) for r, c in self._shapes[side][t]]

    def weight(self, t: int, rank: int, payload: int, scales: int, side: str = "dst") -> R.Matrix:
        """The block- or group-scaled matrix of a rank's shard, as the products take it."""
        r, c = self._shapes[side][t][rank]
        blocks = _blocks(c, self._cols)
        return R.matrix(r, c, self.dtype, payload, blocks * self._cols, self._rows, scales, blocks)

    def bind(self, src, src_payload, src_scales, dst_payload, dst_scales):
        """Handles for ``execute``, reusable as long as the buffers live.  Each
        argument: a list per tensor of device addresses, one per rank (0 or None
        for an empty shard)."""
        jobs = []
        for t, spec in enumerate(self.specs):
            code = R.dtype_code(spec.dtype)
            for rank, (r, c) in enumerate(self._shapes["src"][t]):
                if self._read[t][rank]:
                    jobs.append((R.matrix(r, c, code, src[t][rank]),
                                 self.weight(t, rank, src_payload[t][rank], src_scales[t][rank], "src")))
        flat = lambda *lists: R.pointer_array([p for per in lists for ranks in per for p in ranks])
        return jobs, flat(src_payload, src_scales), flat(dst_payload, dst_scales)

    # ------------------------------------------------------------- execute

    def bytes_moved(self) -> int:
        """Bytes read and written by one execute, quantization included."""
        st = R.reshard_plan_stats(self.plan)
        total = st["bytes_read"] + st["bytes_written"]
        for t, spec in enumerate(self.specs):
            size = R.reshard_dtype_size(R.dtype_code(spec.dtype))
            for read, (r, c) in zip(self._read[t], self._shapes["src"][t]):
                if read:
                    blocks = _blocks(c, self._cols)
                    total += r * c * size + r * blocks * self._bytes + _blocks(r, self._rows) * blocks
        return total

    def execute(self, bound, stream: int):
        """Quantize every source shard that is read, then move payload and scales,
        all on one stream (a raw hipStream_t address; 0 = the null stream)."""
        jobs, src, dst = bound
        for plain, held in jobs:
            if self.dtype == R.DTYPE_FP4_E2M1:
                R.reshard_group_quantize(plain, held, stream)
            else:
                R.reshard_block_quantize(plain, held, None, stream)
        R.reshard_execute(self.plan, src, dst, stream)

    def close(self):
        if self.plan is not None:
            R.reshard_plan_destroy(self.plan)
        for h in self._layouts:
            R.reshard_layout_destroy(h)
        self.plan = None
        self._layouts = []
