"""The 8-bit linear-layer operators of fp4q and the cases they are measured on.

Three operators make one path: the RMS norm (with the residual's addition) that ends in E4M3
codes with a scale per 128 channels, the quantizer that gives other activations (a scale per
row and 128 channels) and weights (a scale per 128 x 128 tile) the same form, and the matrix
product of two such operands.  A scale is the fp32 value A / 448 (A the block's largest
magnitude), or the smallest power of two that is not below it, held as an E8M0 byte; neither
is ever below 2^-126, and a block with a NaN or an infinity has the scale NaN.

`run` computes an operator in plain torch operations in fp32, or, with `own` set, calls the
framework; `exact` computes it in fp64 from the definition.
"""

import math

import torch

own = False

_E4M3_MAX = 448.0
_BLOCK = 128
_EPS = 1e-6
_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# the cost of a drawn case stays within the largest listed one of its operator
_NORM_MAX = 16384 * 8192
_QUANT_MAX = 32768 * 14336
_GEMM_MAX = 8192 ** 3


def _norm(name, M, K, scale, dtype="bf16", residual=True, pad=0):
    return {"name": name, "op": "norm", "M": M, "K": K, "scale": scale, "dtype": dtype, "residual": residual, "pad": pad}


def _quant(name, M, K, scale, rows, dtype="bf16", pad=0):
    return {"name": name, "op": "quant", "M": M, "K": K, "scale": scale, "rows": rows, "dtype": dtype, "pad": pad}


def _gemm(name, M, N, K, scale, dtype="bf16"):
    return {"name": name, "op": "gemm", "M": M, "N": N, "K": K, "scale": scale, "dtype": dtype}


def listed():
    return [
        # one token of one sequence before its projection: latency alone
        _norm("norm_decode_1x4096", 1, 4096, "f32"),
        # a decode batch of the widest rows
        _norm("norm_decode_16x14336", 16, 14336, "e8m0"),
        # a ragged chunk whose input is a column slice of a wider tensor and whose last block is short
        _norm("norm_ragged_333x5008", 333, 5008, "f32", dtype="fp16", pad=24),
        # a long prefill: memory bandwidth alone
        _norm("norm_prefill_16384x8192", 16384, 8192, "f32"),
        # the input of the down projection in a decode batch
        _quant("rows_decode_16x14336", 16, 14336, "f32", 1),
        # the same in a long prefill
        _quant("rows_prefill_32768x14336", 32768, 14336, "e8m0", 1),
        # a projection's weights, once when they are loaded
        _quant("weight_14336x4096", 14336, 4096, "f32", 128),
        # one token through the up projection: the weights are read once
        _gemm("gemm_decode_1x14336x4096", 1, 14336, 4096, "f32"),
        # a decode batch through the down projection: few output tiles, a long sum
        _gemm("gemm_decode_16x4096x14336", 16, 4096, 14336, "e8m0"),
        # a ragged chunk through odd sizes in all three directions
        _gemm("gemm_ragged_333x4104x5008", 333, 4104, 5008, "f32", dtype="fp16"),
        # a prefill through a square projection
        _gemm("gemm_prefill_8192x8192x8192", 8192, 8192, 8192, "f32"),
        # a prefill through the up projection, scales in powers of two
        _gemm("gemm_prefill_4096x14336x4096", 4096, 14336, 4096, "e8m0"),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def _channels(rng):
    """A row length: half the time whole blocks of 128, else any multiple of 16."""
    return _BLOCK * _spread(rng, 1, 112) if rng.random() < 0.5 else 16 * _spread(rng, 1, 896)


def draw(rng):
    op = rng.choice(["norm", "quant", "gemm", "gemm"])
    scale = rng.choice(["f32", "e8m0"])
    pad = rng.choice([0, 0, 8 * rng.randint(1, 16)])
    if op == "norm":
        K = _channels(rng)
        M = _spread(rng, 1, min(16384, _NORM_MAX // K))
        c = _norm("", M, K, scale, rng.choice(["bf16", "bf16", "fp16"]), rng.random() < 0.75, pad)
    elif op == "quant":
        K = _channels(rng)
        M = _spread(rng, 1, min(32768, _QUANT_MAX // K))
        c = _quant("", M, K, scale, rng.choice([1, 128]), rng.choice(["bf16", "bf16", "fp16"]), pad)
    else:
        K, N = _channels(rng), _spread(rng, 1, 14336)
        M = _spread(rng, 1, min(8192, _GEMM_MAX // (K * N)))
        c = _gemm("", M, N, K, scale, rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    del c["name"]
    return c


# ---------------------------------------------------------------- plain forms

def _padded(v, rows):
    """v [M, K] with zeros up to whole blocks of `rows` x 128, as [M / rows, rows, K / 128, 128]."""
    M, K = v.shape
    v = torch.nn.functional.pad(v, (0, -K % _BLOCK, 0, -M % rows))
    return v.view(v.shape[0] // rows, rows, v.shape[1] // _BLOCK, _BLOCK)


def _quantize_plain(v, rows, scale):
    """fp32 v [M, K] -> E4M3 codes [M, K] and scales [ceil(M / rows), ceil(K / 128)]."""
    M, K = v.shape
    t = _padded(v, rows)
    a = t.abs().amax((1, 3))
    if scale == "f32":
        s = (a / torch.full_like(a, _E4M3_MAX)).clamp_min(2.0 ** -126)   # a quotient: a number would be inverted first
        s = torch.where(torch.isfinite(a), s, torch.nan)
        out = s
    else:
        m, e = torch.frexp(a)                       # a = m 2^e, m in [1/2, 1); 448 = (7/8) 2^9
        byte = (e - 9 + (m > 0.875) + 127).clamp(1, 254)
        byte = torch.where(a > 0, byte, 1)
        byte = torch.where(torch.isfinite(a), byte, 255)
        s = torch.where(torch.isfinite(a), torch.exp2((byte - 127).float()), torch.nan)
        out = byte.to(torch.uint8).view(torch.float8_e8m0fnu)
    q = (t / s[:, None, :, None]).clamp(-_E4M3_MAX, _E4M3_MAX)
    q = q.reshape(t.shape[0] * rows, -1)[:M, :K].contiguous()
    return q.to(torch.float8_e4m3fn), out


def _norm_plain(st):
    h = st["x"].float()
    stored = None
    if st["residual"] is not None:
        h = h + st["residual"].float()
        stored = h.to(st["x"].dtype)
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + _EPS) * st["weight"].float()
    return _quantize_plain(y, 1, st["scale"]) + (stored,)


def _gemm_plain(st):
    a, b = st["a_codes"].float(), st["b_codes"].float()
    sa, sb = st["a_scales"].float(), st["b_scales"].float()
    N, K = b.shape
    a = a * sa.repeat_interleave(_BLOCK, 1)[:, :K]
    b = b * sb.repeat_interleave(_BLOCK, 0)[:N].repeat_interleave(_BLOCK, 1)[:, :K]
    return (a @ b.t()).to(st["dtype"])


# ---------------------------------------------------------------- inputs

def _activations(g, M, K, dtype, pad):
    """N(0, 1) entries with a factor for each row (log-normal) and 0.5 % of the channels x 50, as a
    column slice of a wider tensor where pad is not zero."""
    x = torch.randn((M, K + pad), generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn((M, 1), generator=g, device="cuda"))
    cols = torch.randperm(K, generator=g, device="cuda")[:max(1, round(0.005 * K))]
    x[:, cols] *= 50.0
    return x.to(dtype)[:, :K]


def _weights(g, N, K, dtype, pad):
    """Laplace(0, 0.02) entries with 0.5 % of the input channels x 10."""
    u = torch.rand((N, K + pad), generator=g, device="cuda", dtype=torch.float32) - 0.5
    w = -0.02 * u.sign() * torch.log1p(-(2.0 * u).abs().clamp_max(1 - 2.0 ** -20))
    cols = torch.randperm(K, generator=g, device="cuda")[:max(1, round(0.005 * K))]
    w[:, cols] *= 10.0
    return w.to(dtype)[:, :K]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, K, scale = case["M"], case["K"], case["scale"]
    dtype = _DTYPES[case["dtype"]]
    st = {"op": case["op"], "scale": scale, "dtype": dtype}
    s_dtype = torch.float32 if scale == "f32" else torch.float8_e8m0fnu
    kb = -(-K // _BLOCK)
    if case["op"] == "gemm":
        # operands as the quantizer leaves them; D is a buffer that a server keeps
        N = case["N"]
        st["a_codes"], st["a_scales"] = _quantize_plain(_activations(g, M, K, torch.bfloat16, 0).float(), 1, scale)
        st["b_codes"], st["b_scales"] = _quantize_plain(_weights(g, N, K, torch.bfloat16, 0).float(), 128, scale)
        st["out"] = torch.empty((M, N), dtype=dtype, device="cuda")
        return st
    rows = 1
    if case["op"] == "norm":
        st["x"] = _activations(g, M, K, dtype, case["pad"])
        st["residual"] = _activations(g, M, K, dtype, case["pad"]) if case["residual"] else None
        st["weight"] = (1.0 + 0.1 * torch.randn(K, generator=g, device="cuda")).to(dtype)
        st["stored"] = torch.empty((M, K), dtype=dtype, device="cuda") if case["residual"] else None
    else:
        rows = st["rows"] = case["rows"]
        make = _activations if rows == 1 else _weights
        st["x"] = make(g, M, K, dtype, case["pad"])
    st["codes"] = torch.empty((M, K), dtype=torch.float8_e4m3fn, device="cuda")
    st["scales"] = torch.empty((-(-M // rows), kb), dtype=s_dtype, device="cuda")
    return st


def run(state):
    st = state
    if own:
        from microscaling_fp4_quantization_b200 import fp4q as F
        fmt = F.FP4Q_FP8_SCALE_F32 if st["scale"] == "f32" else F.FP4Q_FP8_SCALE_E8M0
        if st["op"] == "norm":
            codes, scales, stored = F.add_rmsnorm_fp8(st["x"], st["residual"], st["weight"], _EPS, scale_format=fmt,
                                                      residual_out=st["stored"], codes=st["codes"],
                                                      scales=st["scales"])
            return {"codes": codes, "scales": scales, "residual": stored}
        if st["op"] == "quant":
            codes, scales = F.quantize_fp8(st["x"], block_rows=st["rows"], scale_format=fmt, codes=st["codes"],
                                           scales=st["scales"])
            return {"codes": codes, "scales": scales}
        return {"d": F.gemm_fp8(st["a_codes"], st["a_scales"], st["b_codes"], st["b_scales"], out_dtype=st["dtype"],
                                out=st["out"])}
    if st["op"] == "norm":
        codes, scales, stored = _norm_plain(st)
        return {"codes": codes, "scales": scales, "residual": stored}
    if st["op"] == "quant":
        codes, scales = _quantize_plain(st["x"].float(), st["rows"], st["scale"])
        return {"codes": codes, "scales": scales}
    return {"d": _gemm_plain(st)}


def work(case):
    M, K = case["M"], case["K"]
    kb = -(-K // _BLOCK)
    sb = 4 if case["scale"] == "f32" else 1
    if case["op"] == "norm":
        # x in, codes and scales out, the weight; with a residual, that in and the sum out.  Per element:
        # the addition, a square and its sum, two products, the maximum, the division
        per = 7 if case["residual"] else 3
        return {"bytes": M * K * per + 2 * K + M * kb * sb, "flops": 7 * M * K}
    if case["op"] == "quant":
        rows = case["rows"]
        return {"bytes": 3 * M * K + -(-M // rows) * kb * sb, "flops": 2 * M * K}
    N = case["N"]
    out = 4 if case["dtype"] == "fp32" else 2
    return {"bytes": M * K + N * K + (M + -(-N // _BLOCK)) * kb * sb + M * N * out, "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definition in 64 bits

def _e4m3_exact(v):
    """The E4M3 value nearest to v (ties to the even code), at most 448 in magnitude: steps of
    2^(e-3) for magnitudes in [2^e, 2^(e+1)), e >= -6."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp_min(-6) - 3)
    return (torch.round(v / step) * step).clamp(-_E4M3_MAX, _E4M3_MAX)


def _quantize_exact(v, rows, scale):
    M, K = v.shape
    kb = -(-K // _BLOCK)
    cols = torch.arange(K, device=v.device) // _BLOCK
    per_col = torch.zeros((-(-M // rows), K), dtype=v.dtype, device=v.device)
    row = torch.arange(M, device=v.device) // rows
    per_col = per_col.scatter_reduce(0, row[:, None].expand(M, K), v.abs(), "amax") if rows > 1 else v.abs()
    a = torch.zeros((per_col.shape[0], kb), dtype=v.dtype, device=v.device)
    a = a.scatter_reduce(1, cols[None].expand(per_col.shape[0], K), per_col, "amax")
    s = (a / _E4M3_MAX).clamp_min(2.0 ** -126)
    if scale == "f32":
        s = s.float().double()                     # the codes are taken with the scale that is stored
    else:
        m, e = torch.frexp(s)                      # 2^ceil(log2 s): 2^(e-1) where s is a power of two
        s = torch.ldexp(torch.ones_like(s), torch.where(m == 0.5, e - 1, e))
    q = _e4m3_exact(v / s[row][:, cols])
    return q, s


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "gemm":
        N, K = st["b_codes"].shape
        k = torch.arange(K, device="cuda") // _BLOCK
        n = torch.arange(N, device="cuda") // _BLOCK
        a = st["a_codes"].double() * st["a_scales"].double()[:, k]
        b = st["b_codes"].double() * st["b_scales"].double()[n][:, k]
        return {"d": torch.matmul(a, b.transpose(0, 1))}
    x = st["x"].double()
    if case["op"] == "quant":
        q, s = _quantize_exact(x, case["rows"], case["scale"])
        return {"codes": q, "scales": s}
    h = x if st["residual"] is None else x + st["residual"].double()
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / h.shape[1] + _EPS) * st["weight"].double()
    q, s = _quantize_exact(y, 1, case["scale"])
    return {"codes": q, "scales": s, "residual": None if st["residual"] is None else h}
