"""Block-scaled 8-bit operators: the measured cases and their plain forms.

A block-scaled matrix holds one 8-bit float per element and one power of two
per block of 128 columns (of one row for activations and gradients, of 128 rows
for weights).  With amax the largest finite magnitude of a block and top the
format's largest value (448 for e4m3, 57344 for e5m2) the block's exponent is
the smallest e >= -127 with amax <= top * 2^e (0 for a block of zeros), and an
element is held as x / 2^e rounded to nearest, ties to even.

Four uses:

  restore   an activation checkpoint saved in 8 bits and read back
  weights   a weight quantized in blocks of 128 x 128, with its transpose
  project   y = x^ W^^T, x quantized within the call, W quantized beforehand
  backward  of that projection: dx = dy^ W^ (dy quantized within the call) and
            dw = dy^T x^ from the 8-bit checkpoint of x

``^`` marks the values that the 8-bit form stands for.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token's hidden state saved and restored: latency
        {"name": "restore_token", "kind": "restore", "rows": 1, "cols": 4096, "type": "bf16"},
        # the FFN activations of a 4096-token micro-batch
        {"name": "restore_ffn", "kind": "restore", "rows": 4096, "cols": 14336, "type": "bf16"},
        # an odd fp32 tensor: columns end inside a block, rows start off the 16-byte grid
        {"name": "restore_ragged_f32", "kind": "restore", "rows": 5000, "cols": 3001, "type": "f32"},
        # an up-projection's fp32 master weight quantized for a refit and for the backward pass
        {"name": "weights_ffn_f32", "kind": "weights", "rows": 14336, "cols": 4096, "type": "f32"},
        # an uneven weight: both sides end inside a block
        {"name": "weights_ragged", "kind": "weights", "rows": 5000, "cols": 3001, "type": "bf16"},
        # rollout decoding, one sequence: the up-projection of a single token
        {"name": "project_token", "kind": "project", "m": 1, "n": 14336, "k": 4096, "type": "bf16"},
        # rollout decoding of 33 sequences: the down-projection, long contraction, few outputs
        {"name": "project_decode_batch", "kind": "project", "m": 33, "n": 4096, "k": 14336, "type": "bf16"},
        # a short prompt over an uneven weight in fp16
        {"name": "project_ragged_f16", "kind": "project", "m": 301, "n": 5000, "k": 3001, "type": "f16"},
        # a training micro-batch or a long prompt through the up-projection
        {"name": "project_prompt", "kind": "project", "m": 4096, "n": 14336, "k": 4096, "type": "bf16"},
        # a short micro-batch through a key projection
        {"name": "backward_kv", "kind": "backward", "m": 257, "n": 1024, "k": 4096, "type": "bf16"},
        # an uneven weight, gradients in fp32
        {"name": "backward_ragged_f32", "kind": "backward", "m": 301, "n": 5000, "k": 3001, "type": "f32"},
        # the up-projection's backward pass over a training micro-batch
        {"name": "backward_ffn", "kind": "backward", "m": 4096, "n": 14336, "k": 4096, "type": "bf16"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("restore", "weights", "project", "project", "backward"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if kind in ("restore", "weights"):
        # up to the bytes of the largest listed one in 32 bits
        cols = _spread(rng, 64, 14336)
        rows = _spread(rng, 1, max(2, min(16384, 14336 * 4096 // 2 // cols)))
        return {"kind": kind, "rows": rows, "cols": cols, "type": dtype}
    k = _spread(rng, 128, 14336)
    n = _spread(rng, 128, 14336 * 4096 // max(4096, k))
    m = _spread(rng, 1, 4096 if kind == "project" or dtype == "bf16" else 1024)
    return {"kind": kind, "m": m, "n": n, "k": k, "type": dtype}


def _up(n):
    return -(-n // BLOCK) * BLOCK


# ------------------------------------------------------------- plain forms


def _power(e):
    """2^e in float32 for integers -127 <= e <= 127, exactly (by its bits)."""
    p = (e.to(torch.int32).clamp(min=-126) + 127 << 23).view(torch.float32)
    return torch.where(e < -126, p * 0.5, p)


def _quantize(x, block_rows):
    """Payload (e4m3, as a float8 tensor of the padded width) and exponents of x."""
    rows, cols = x.shape
    R, C = -(-rows // block_rows), -(-cols // BLOCK)
    p = torch.zeros(R * block_rows, C * BLOCK, dtype=torch.float32, device=x.device)
    p[:rows, :cols] = x
    blocks = p.view(R, block_rows, C, BLOCK)
    mag = blocks.abs()
    amax = torch.where(torch.isfinite(mag), mag, 0.0).amax(dim=(1, 3))
    frac, top = torch.frexp(amax)
    e = top - 9 + (frac > 0.875).to(top.dtype)
    e = torch.where(amax > 0, e.clamp(min=-127), torch.zeros_like(e))
    inverse = _power(-e)
    q = (blocks * inverse[:, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(R * block_rows, C * BLOCK)[:rows], e


def _values(q, e, block_rows, cols):
    """The float32 values of a payload q (rows x padded) under the exponents e."""
    s = _power(e).repeat_interleave(block_rows, 0)[: q.shape[0]].repeat_interleave(BLOCK, 1)
    return (q.float() * s)[:, :cols]


def _held(data, exponents):
    """A payload and scales as bytes (e4m3, 2^(byte - 127)) back as tensors."""
    return data.view(torch.float8_e4m3fn), exponents.to(torch.int32) - 127


# ------------------------------------------------------------------ inputs


def _activations(rows, cols, dtype, g, scale=1.0):
    """Normal values with a few large channels, as hidden states have."""
    x = torch.randn(rows, cols, device="cuda", generator=g)
    channel = torch.rand(cols, device="cuda", generator=g)
    x.mul_(torch.where(channel > 0.99, 20.0, 1.0) * scale)
    return x.to(dtype)


def _bytes(q, e):
    return q.view(torch.uint8).contiguous(), (e + 127).to(torch.uint8).contiguous()


def _empty(rows, cols, block_rows=None):
    """Room for a payload of padded width and its scales (or a plain matrix)."""
    C = -(-cols // BLOCK)
    return (torch.empty(rows, C * BLOCK, dtype=torch.uint8, device="cuda"),
            torch.empty(-(-rows // block_rows), C, dtype=torch.uint8, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype, kind = TYPES[case["type"]], case["kind"]
    s = {"case": case}
    if kind in ("restore", "weights"):
        rows, cols = case["rows"], case["cols"]
        if kind == "restore":
            s["x"] = _activations(rows, cols, dtype, g)
            s["q"], s["scales"] = _empty(rows, cols, 1)
            s["out"] = torch.empty_like(s["x"])
        else:
            s["x"] = (torch.randn(rows, cols, device="cuda", generator=g) * 0.02).to(dtype)
            s["q"], s["scales"] = _empty(rows, cols, BLOCK)
            s["qt"], s["scales_t"] = _empty(cols, rows, BLOCK)
            s["out"] = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
            s["out_t"] = torch.empty(cols, rows, dtype=torch.bfloat16, device="cuda")
        return s
    m, n, k = case["m"], case["n"], case["k"]
    w = torch.randn(n, k, device="cuda", generator=g) * 0.02
    if kind == "project":
        s["x"] = _activations(m, k, dtype, g)
        s["w"], s["w_scales"] = _bytes(*_quantize(w, BLOCK))
        s["out"] = torch.empty(m, n, dtype=dtype, device="cuda")
        return s
    s["wt"], s["wt_scales"] = _bytes(*_quantize(w.t().contiguous(), BLOCK))
    s["x"], s["x_scales"] = _bytes(*_quantize(_activations(m, k, dtype, g), 1))
    s["dy"] = _activations(m, n, dtype, g, 1e-3)
    s["dx"] = torch.empty(m, k, dtype=dtype, device="cuda")
    s["dw"] = torch.empty(n, k, dtype=dtype if dtype != torch.float16 else torch.float32, device="cuda")
    return s


# --------------------------------------------------------------- one pass


def _own(s):
    """The handles that a user's program keeps: matrix descriptions and a workspace."""
    import dtensor_layout_movement_amd as R

    def plain(t):
        return R.matrix(t.shape[0], t.shape[1], R.dtype_code(t.dtype), t.data_ptr(), t.stride(0))

    def held(rows, cols, q, scales, block_rows):
        return R.matrix(rows, cols, R.DTYPE_FP8_E4M3, q.data_ptr(), q.stride(0), block_rows, scales.data_ptr(),
                        scales.stride(0))

    case, kind = s["case"], s["case"]["kind"]
    h = {"R": R}
    if kind in ("restore", "weights"):
        rows, cols = case["rows"], case["cols"]
        h["x"], h["out"] = plain(s["x"]), plain(s["out"])
        h["q"] = held(rows, cols, s["q"], s["scales"], 1 if kind == "restore" else BLOCK)
        if kind == "weights":
            h["qt"], h["out_t"] = held(cols, rows, s["qt"], s["scales_t"], BLOCK), plain(s["out_t"])
        return h
    m, n, k = case["m"], case["n"], case["k"]
    if kind == "project":
        h["x"], h["w"], h["out"] = plain(s["x"]), held(n, k, s["w"], s["w_scales"], BLOCK), plain(s["out"])
        need = R.reshard_block_matmul_workspace(h["x"], h["w"], h["out"])
    else:
        h["dy"], h["dx"], h["dw"] = plain(s["dy"]), plain(s["dx"]), plain(s["dw"])
        h["wt"], h["x"] = held(k, n, s["wt"], s["wt_scales"], BLOCK), held(m, k, s["x"], s["x_scales"], 1)
        need = max(R.reshard_block_matmul_workspace(h["dy"], h["wt"], h["dx"]),
                   R.reshard_block_grad_workspace(h["dy"], h["x"], h["dw"]))
    h["room"] = torch.empty(max(1, need), dtype=torch.uint8, device="cuda")
    h["workspace"] = (h["room"].data_ptr(), need)
    return h


def run(s):
    case, kind = s["case"], s["case"]["kind"]
    if own:
        h = s.get("own")
        if h is None:
            h = s["own"] = _own(s)
        R, stream = h["R"], torch.cuda.current_stream().cuda_stream
        if kind == "restore":
            R.reshard_block_quantize(h["x"], h["q"], None, stream)
            R.reshard_block_dequantize(h["q"], h["out"], stream)
            return s["out"]
        if kind == "weights":
            R.reshard_block_quantize(h["x"], h["q"], h["qt"], stream)
            R.reshard_block_dequantize(h["q"], h["out"], stream)
            R.reshard_block_dequantize(h["qt"], h["out_t"], stream)
            return s["out"], s["out_t"]
        if kind == "project":
            R.reshard_block_matmul(h["x"], h["w"], h["out"], *h["workspace"], stream)
            return s["out"]
        R.reshard_block_matmul(h["dy"], h["wt"], h["dx"], *h["workspace"], stream)
        R.reshard_block_grad(h["dy"], h["x"], h["dw"], False, *h["workspace"], stream)
        return s["dx"], s["dw"]
    if kind == "restore":
        q, e = _quantize(s["x"], 1)
        return _values(q, e, 1, case["cols"]).to(s["x"].dtype)
    if kind == "weights":
        q, e = _quantize(s["x"], BLOCK)
        w = _values(q, e, BLOCK, case["cols"]).to(torch.bfloat16)
        return w, w.t().contiguous()
    if kind == "project":
        q, e = _quantize(s["x"], 1)
        x = _values(q, e, 1, case["k"])
        w = _values(*_held(s["w"], s["w_scales"]), BLOCK, case["k"])
        return (x @ w.t()).to(s["x"].dtype)
    q, e = _quantize(s["dy"], 1)
    dy = _values(q, e, 1, case["n"])
    wt = _values(*_held(s["wt"], s["wt_scales"]), BLOCK, case["n"])
    x = _values(*_held(s["x"], s["x_scales"]), 1, case["k"])
    return (dy @ wt.t()).to(s["dx"].dtype), (s["dy"].float().t() @ x).to(s["dw"].dtype)


# -------------------------------------------------------------------- work


def work(case):
    size = 4 if case["type"] == "f32" else 2
    if case["kind"] == "restore":
        r, c = case["rows"], case["cols"]
        # read x, write the saved bytes and scales, write the restored values
        return {"bytes": r * c * (2 * size + 1) + r * _up(c) // BLOCK, "flops": 3 * r * c}
    if case["kind"] == "weights":
        r, c = case["rows"], case["cols"]
        # read w, write both orientations, write both restored
        return {"bytes": r * c * (size + 2 + 4), "flops": 4 * r * c}
    m, n, k = case["m"], case["n"], case["k"]
    if case["kind"] == "project":
        return {"bytes": m * k * size + n * k + m * n * size, "flops": 2 * m * n * k}
    return {"bytes": m * n * size + n * k + m * k + m * k * size + n * k * (2 if case["type"] == "bf16" else 4),
            "flops": 4 * m * n * k}


# --------------------------------------------------- the definition in 64 bits


def _two_to(e):
    """2^e in float64 for whole -1022 <= e <= 1023, from the exponent field."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _rounded(x, block_rows):
    """x as its e4m3 blocks hold it, straight from the definition."""
    rows, cols = x.shape
    x = x.double()
    out = torch.empty_like(x)
    pad = torch.nn.functional.pad(x.abs(), (0, _up(cols) - cols, 0, -rows % block_rows))
    amax = pad.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, block_rows)).amax(dim=(1, 3))
    e = torch.ceil(torch.log2(amax.clamp(min=2.0**-300) / 448.0)).clamp(min=-400)
    # the logarithm may land on the wrong side of a border
    e = torch.where(448.0 * _two_to(e - 1) >= amax, e - 1, e)
    e = torch.where(448.0 * _two_to(e) < amax, e + 1, e)
    unit = torch.where(amax > 0, _two_to(e.clamp(min=-127)), torch.ones_like(amax))
    unit = unit.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]
    v = x / unit
    # e4m3: three mantissa bits down to 2^-6, steps of 2^-9 below
    step = _two_to(torch.floor(torch.log2(v.abs().clamp(min=2.0**-6))) - 3)
    step = torch.where(v.abs() >= 16 * step, 2 * step, step)
    step = torch.where((v.abs() < 8 * step) & (step > 2.0**-9), step / 2, step)
    torch.mul(torch.round(v / step) * step, unit, out=out)
    return out


def _decoded(data, scales, block_rows, cols):
    """The bytes' values from the e4m3 bit fields."""
    table = []
    for b in range(256):
        sign, field, frac = (-1.0 if b & 128 else 1.0), b >> 3 & 15, b & 7
        v = frac * 2.0**-9 if field == 0 else (8 + frac) * 2.0 ** (field - 10)
        table.append(float("nan") if field == 15 and frac == 7 else sign * v)
    table = torch.tensor(table, dtype=torch.float64, device=data.device)
    unit = _two_to(scales.long() - 127)
    rows = torch.arange(data.shape[0], device=data.device) // block_rows
    columns = torch.arange(cols, device=data.device)
    return table[data[:, :cols].long()] * unit[rows][:, columns // BLOCK]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "restore":
        return _rounded(s["x"], 1)
    if kind == "weights":
        w = _rounded(s["x"], BLOCK)
        return w, w.t().contiguous()
    if kind == "project":
        return _rounded(s["x"], 1) @ _decoded(s["w"], s["w_scales"], BLOCK, case["k"]).t()
    dx = _rounded(s["dy"], 1) @ _decoded(s["wt"], s["wt_scales"], BLOCK, case["n"]).t()
    return dx, s["dy"].double().t() @ _decoded(s["x"], s["x_scales"], 1, case["k"])
