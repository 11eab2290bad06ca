"""What is measured of the feed-forward operators: the cases, their inputs, the operators'
plain forms and 64-bit values, and the library's calls.

Operators (include/rec_attn.h):
  ffn         gated feed-forward block of packed token rows, (act(x Wg') * (x Wu')) Wo'
              (rec_attn_ffn_fwd)
  ffn_train   the same with its backward pass: y, dx, dw_in, dw_out (rec_attn_ffn_fwd +
              rec_attn_ffn_bwd)
  quantize    rows or weights to e4m3 with a power-of-two scale for each 1 x 128 or
              128 x 128 block (rec_attn_scaled_quantize)
  matmul      product of two e4m3 matrices with a scale for each block of 128
              (rec_attn_scaled_matmul)
  ffn_scaled  the feed-forward block with e4m3 weights, its rows quantized on the way
              (rec_attn_ffn_scaled_fwd)

`own` selects the library's calls; otherwise `run` computes the operators in elementary
torch operations, in 32 bits, rounded once.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
TOP = 448.0  # the largest e4m3 value
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def ffn_case(kind, rows, width, hidden, act="silu", dtype="bf16"):
    return {"kind": kind, "rows": rows, "width": width, "hidden": hidden, "act": act, "dtype": dtype}


def quantize_case(rows, width, block_rows, dtype="bf16"):
    return {"kind": "quantize", "rows": rows, "width": width, "block_rows": block_rows, "dtype": dtype}


def matmul_case(rows, cols, depth):
    return {"kind": "matmul", "rows": rows, "cols": cols, "depth": depth}


def listed():
    cases = {
        # one token through the block of a 512-wide ranking transformer: the smallest call, latency
        "ffn_one_token": ffn_case("ffn", 1, 512, 1024),
        # a few tokens through a wide block: the weights' bytes
        "ffn_wide_tokens": ffn_case("ffn", 24, 4096, 8192),
        # one request with a 20K-token history and its target
        "ffn_history": ffn_case("ffn", 20001, 512, 1024),
        # a training step on 16 such histories
        "train_histories": ffn_case("ffn_train", 320016, 512, 1024),
        # a training step on a ragged batch with a wider hidden state, sizes off the tiles
        "train_wide": ffn_case("ffn_train", 5003, 1408, 4104, "gelu"),
        # a training step in fp32 on one ragged request
        "train_fp32": ffn_case("ffn_train", 1850, 512, 1024, "silu", "fp32"),
        # activations of the 16 histories to e4m3, a scale for each row's 128 values
        "quantize_rows": quantize_case(320016, 512, 1),
        # a weight matrix to e4m3 when a model is loaded, a scale for each 128 x 128 block
        "quantize_weights": quantize_case(4104, 8192, 128, "fp32"),
        # one token through an e4m3 projection: the weights' bytes
        "matmul_one_token": matmul_case(1, 4096, 4096),
        # a batch of prompts through a wide e4m3 projection
        "matmul_prompts": matmul_case(16387, 8192, 4096),
        # a few tokens through the wide block with e4m3 weights
        "ffn_scaled_tokens": ffn_case("ffn_scaled", 24, 4096, 8192),
        # serving the 16 histories with e4m3 weights
        "ffn_scaled_histories": ffn_case("ffn_scaled", 320016, 512, 1024),
    }
    return [{"name": n, **c} for n, c in cases.items()]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["ffn", "ffn_train", "quantize", "matmul", "ffn_scaled"])
    if kind == "quantize":
        dtype = "bf16" if rng.random() < 0.6 else "fp32"
        width = 16 * _spread(rng, 4, 512)
        rows = min(_spread(rng, 1, 320016), 320016 * 512 // width)
        return quantize_case(rows, width, rng.choice([1, 128]), dtype)
    if kind == "matmul":
        depth, cols = 16 * _spread(rng, 4, 512), 8 * _spread(rng, 4, 1024)
        return matmul_case(min(_spread(rng, 1, 32768), 16387 * 8192 * 4096 // (depth * cols)), cols, depth)
    act = rng.choice(["silu", "gelu"])
    fp32 = kind != "ffn_scaled" and rng.random() < 0.2
    if kind == "ffn_scaled":
        width, hidden = 16 * _spread(rng, 4, 256), 128 * _spread(rng, 1, 64)
    else:
        width, hidden = 8 * _spread(rng, 8, 512), 8 * _spread(rng, 8, 1024)
    most = (2000 * 512 * 1024 if fp32 else 320016 * 512 * 1024) // (width * hidden)
    rows = max(1, min(_spread(rng, 1, 4000 if fp32 else 320016), most))
    return ffn_case(kind, rows, width, hidden, act, "fp32" if fp32 else "bf16")


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    kind, r = case["kind"], case["rows"]
    if kind == "quantize":
        n, size = r * case["width"], 2 if case["dtype"] == "bf16" else 4
        scales = -(-r // case["block_rows"]) * _blocks(case["width"])
        return {"bytes": n * (size + 1) + 4 * scales, "flops": 3 * n}
    if kind == "matmul":
        n, k = case["cols"], case["depth"]
        scales = (r + _blocks(n)) * _blocks(k)
        return {"bytes": (r + n) * k + 2 * r * n + 4 * scales, "flops": 2 * r * n * k}
    w, h = case["width"], case["hidden"]
    if kind == "ffn_scaled":
        return {"bytes": 4 * r * w + 3 * w * h + 4 * 3 * _blocks(w) * _blocks(h), "flops": 6 * r * w * h}
    size = 2 if case["dtype"] == "bf16" else 4
    if kind == "ffn":
        return {"bytes": size * (2 * r * w + 3 * w * h), "flops": 6 * r * w * h}
    # x, dy and the weights read; y, dx and the weights' gradients written; three products forward, six backward
    return {"bytes": size * (4 * r * w + 6 * w * h), "flops": 18 * r * w * h}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dtype = DTYPES[case.get("dtype", "bf16")]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def rows_of(n, width):
        # rows behind a norm with gains: columns of unlike size, a few of them large
        gain = 0.5 + torch.rand(width, generator=gen, device=DEV)
        gain[torch.randint(0, width, (max(1, width // 64),), generator=gen, device=DEV)] *= 8
        return normal(n, width) * gain

    s = {"case": case}
    kind = case["kind"]
    if kind == "quantize":
        x = rows_of(case["rows"], case["width"]) if case["block_rows"] == 1 else \
            normal(case["rows"], case["width"]) / math.sqrt(case["width"])
        s["x"] = x.to(dtype)
        return s
    if kind == "matmul":
        # the activations and weights that a program holds in e4m3
        s["a"], s["a_scale"] = _quantize(rows_of(case["rows"], case["depth"]).bfloat16().float(), 1)
        s["b"], s["b_scale"] = _quantize(normal(case["cols"], case["depth"]) / math.sqrt(case["depth"]), BLOCK)
        return s
    r, w, h = case["rows"], case["width"], case["hidden"]
    w_in, w_out = normal(2 * h, w) / math.sqrt(w), normal(w, h) / math.sqrt(h)
    s["x"] = (rows_of(r, w) if kind == "ffn_scaled" else normal(r, w)).to(dtype)
    if kind == "ffn_scaled":
        s["w_in"], s["w_in_scale"] = _quantize(w_in, BLOCK)
        s["w_out"], s["w_out_scale"] = _quantize(w_out, BLOCK)
        return s
    s["w_in"], s["w_out"] = w_in.to(dtype), w_out.to(dtype)
    if kind == "ffn_train":
        s["dy"] = normal(r, w).to(dtype)
    return s


# ------------------------------------------------------------------ plain forms
def _largest(x, block_rows):
    """The largest absolute value of each block_rows x 128 block."""
    rows, width = x.shape
    nr, nw = -(-rows // block_rows), _blocks(width)
    a = x.abs()
    if nw * BLOCK != width or nr * block_rows != rows:
        p = a.new_zeros(nr * block_rows, nw * BLOCK)
        p[:rows, :width] = a
        a = p
    return a.reshape(nr, block_rows, nw, BLOCK).amax((1, 3))


def _spread_scale(scale, block_rows, rows, width):
    """A block's scale at each of its values."""
    return scale.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :width]


def _quantize(x, block_rows):
    """e4m3 values and scales: the least power of two that brings a block's largest value to at
    most 448 (1 for a block of zeros)."""
    top = _largest(x, block_rows)
    part, e = torch.frexp(top)  # top = part 2^e, part in [0.5, 1); 448 = 0.875 2^9
    e = (e - 9 + (part > 0.875).int()).clamp_min(-126)
    scale = torch.where(top > 0, ((e + 127) << 23).view(torch.float32), 1.0)  # (the exponent's bits: exact)
    return (x / _spread_scale(scale, block_rows, *x.shape)).to(torch.float8_e4m3fn), scale


def _dequantize(q, scale, block_rows):
    return q.float() * _spread_scale(scale, block_rows, *q.shape)


def _act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _act_slope(g, act):
    if act == "silu":
        sig = torch.sigmoid(g)
        return sig * (1 + g * (1 - sig))
    return 0.5 * (1 + torch.erf(g * math.sqrt(0.5))) + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)


def _plain(s):
    c = s["case"]
    kind = c["kind"]
    if kind == "quantize":
        q, scale = _quantize(s["x"].float(), c["block_rows"])
        return {"values": q, "scale": scale}
    if kind == "matmul":
        return (_dequantize(s["a"], s["a_scale"], 1) @ _dequantize(s["b"], s["b_scale"], BLOCK).T).bfloat16()
    h = c["hidden"]
    if kind == "ffn_scaled":
        x = _dequantize(*_quantize(s["x"].float(), 1), 1)
        pre = x @ _dequantize(s["w_in"], s["w_in_scale"], BLOCK).T
        inner = _dequantize(*_quantize(_act(pre[:, :h], c["act"]) * pre[:, h:], 1), 1)
        return (inner @ _dequantize(s["w_out"], s["w_out_scale"], BLOCK).T).bfloat16()
    dtype = DTYPES[c["dtype"]]
    x, w_in, w_out = s["x"].float(), s["w_in"].float(), s["w_out"].float()
    pre = x @ w_in.T
    g, u = pre[:, :h], pre[:, h:]
    a = _act(g, c["act"])
    inner = a * u
    y = (inner @ w_out.T).to(dtype)
    if kind == "ffn":
        return y
    dy = s["dy"].float()
    dh = dy @ w_out
    dpre = torch.cat((dh * u * _act_slope(g, c["act"]), dh * a), 1)
    return {"y": y, "dx": (dpre @ w_in).to(dtype), "dw_in": (dpre.T @ x).to(dtype), "dw_out": (dy.T @ inner).to(dtype)}


# ------------------------------------------------------------------ the library's calls
def _own(s):
    from generative_recommender_ranking_gb300 import binding as bd
    c = s["case"]
    kind = c["kind"]
    if kind == "quantize":
        x, br = s["x"], c["block_rows"]
        q = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=DEV)
        scale = torch.empty(-(-x.shape[0] // br), _blocks(x.shape[1]), device=DEV)
        bd.rec_attn_scaled_quantize(x, q, scale, block_rows=br)
        return {"values": q, "scale": scale}
    if kind == "matmul":
        y = torch.empty(c["rows"], c["cols"], dtype=torch.bfloat16, device=DEV)
        bd.rec_attn_scaled_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], y)
        return y
    x = s["x"]
    y = torch.empty_like(x)
    if kind == "ffn_scaled":
        bd.rec_attn_ffn_scaled_fwd(x, s["w_in"], s["w_in_scale"], s["w_out"], s["w_out_scale"], y, activation=c["act"])
        return y
    bd.rec_attn_ffn_fwd(x, s["w_in"], s["w_out"], y, activation=c["act"])
    if kind == "ffn":
        return y
    dx, dw_in, dw_out = torch.empty_like(x), torch.empty_like(s["w_in"]), torch.empty_like(s["w_out"])
    bd.rec_attn_ffn_bwd(x, s["w_in"], s["w_out"], s["dy"], dx, dw_in, dw_out, activation=c["act"])
    return {"y": y, "dx": dx, "dw_in": dw_in, "dw_out": dw_out}


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------ 64-bit values
def _e4m3(v):
    """v (64 bits) at the nearest e4m3 value, ties to even: 8 steps an octave from 2^-6 on, equal
    steps below."""
    step = _power((torch.frexp(v)[1] - 1).clamp_min(-6) - 3)
    return torch.round(v / step) * step


def _power(e):
    """2^e in 64 bits, from its exponent's bits (a power function's rounding would move ties)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _blockwise(x, block_rows):
    """(e4m3 values, scales) of x in 64 bits."""
    values, scales = torch.empty_like(x), x.new_empty(-(-x.shape[0] // block_rows), _blocks(x.shape[1]))
    turn = BLOCK * max(1, 4194304 // (BLOCK * x.shape[1]))
    for r in range(0, x.shape[0], turn):
        part = x[r:r + turn]
        for b in range(scales.shape[1]):
            block = part[:, b * BLOCK:(b + 1) * BLOCK]
            top = block.abs().amax(1)
            if block_rows > 1:
                short = -top.shape[0] % block_rows
                top = torch.cat((top, top.new_zeros(short))).view(-1, block_rows).amax(1)
            e = torch.ceil(torch.log2(torch.where(top > 0, top, TOP) / TOP))
            # (the logarithm is off by a step at the powers of two themselves)
            e = torch.where(top > TOP * _power(e), e + 1, torch.where(top <= TOP * _power(e - 1), e - 1, e))
            unit = _power(e.clamp_min(-126))
            unit = torch.where(top > 0, unit, 1.0)
            first = r // block_rows
            scales[first:first + unit.shape[0], b] = unit
            unit = unit.repeat_interleave(block_rows)[:part.shape[0], None]
            values[r:r + turn, b * BLOCK:(b + 1) * BLOCK] = _e4m3(block / unit)
    return values, scales


def _held(q, scale, block_rows):
    """The 64-bit values that e4m3 blocks stand for."""
    v = q.float().double() if q.dtype != torch.float64 else q.clone()
    for b in range(scale.shape[1]):
        v[:, b * BLOCK:(b + 1) * BLOCK] *= scale[:, b].double().repeat_interleave(block_rows)[:v.shape[0], None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "quantize":
        values, scale = _blockwise(s["x"].double(), case["block_rows"])
        return {"values": values, "scale": scale}
    if kind == "matmul":
        return _held(s["a"], s["a_scale"], 1) @ _held(s["b"], s["b_scale"], BLOCK).T
    scaled = kind == "ffn_scaled"
    if scaled:
        w_in, w_out = _held(s["w_in"], s["w_in_scale"], BLOCK), _held(s["w_out"], s["w_out_scale"], BLOCK)
    else:
        w_in, w_out = s["w_in"].double(), s["w_out"].double()
    w_gate, w_up = w_in.chunk(2)
    rows, train = case["rows"], kind == "ffn_train"
    y = w_out.new_empty(rows, case["width"])
    dx, dw_gate, dw_up, dw_out = torch.empty_like(y), 0, 0, 0
    for r in range(0, rows, 32768):
        x = s["x"][r:r + 32768].double()
        if scaled:
            x = _held(*_blockwise(x, 1), 1)
        g, u = x @ w_gate.T, x @ w_up.T
        if case["act"] == "silu":
            p = 1 / (1 + torch.exp(-g))     # act(g) = g p(g)
            slope = p + g * p * (1 - p)
        else:
            p = torch.special.erfc(-g / math.sqrt(2)) / 2
            slope = p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
        inner = g * p * u
        if scaled:
            inner = _held(*_blockwise(inner, 1), 1)
        y[r:r + 32768] = inner @ w_out.T
        if train:
            dy = s["dy"][r:r + 32768].double()
            dh = dy @ w_out
            dg, du = dh * u * slope, dh * g * p
            dx[r:r + 32768] = dg @ w_gate + du @ w_up
            dw_gate, dw_up, dw_out = dw_gate + dg.T @ x, dw_up + du.T @ x, dw_out + dy.T @ inner
    return {"y": y, "dx": dx, "dw_in": torch.cat((dw_gate, dw_up)), "dw_out": dw_out} if train else y
