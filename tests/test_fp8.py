"""The 8-bit operators on the GPU against the CPU oracle: the quantizer (bit for bit), the residual
RMS norm, the GEMM, and a run of the three together.

Tolerances, from the arithmetic (u = 2^-24):
 - quantizer: every step is correctly rounded, so codes and scales are equal.
 - norm: residual_out is one fp32 addition and one rounding: equal.  y: h is off by u; the square sum by
   2 u for its terms and u for each addition on the longest path (8 C in a thread's chunks, C for the
   chunks, 1 + 10 across threads, C <= 4: 47), the mean and eps by u each, of all of which the root
   halves: 26 u; root and the two products 3 u.  So y is off by less than 30 u, a scale by 31 u, and with
   the scale that was stored (its quotient rounded once or twice) a code's quotient by less than 33 u.
 - GEMM: an MMA adds 32 exact products to the accumulator; each of these 33 terms is taken to lose at
   most 2^-24 of the largest, so four MMAs lose 132 u S_j in block j, S_j = sum |a b|.  A block's scales
   are multiplied (u), it is added by one rounding, and so is every later block and the split's sums (8 at
   most): (132 + kb + 10) u sum_j s_j S_j, and half a step of the result's type."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as o

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def F(cuda_device):
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def activations(M, K, seed, dtype=BF16, pad=0, outliers=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, K + pad)).astype(np.float32) * np.exp(rng.normal(0, 1, (M, 1))).astype(np.float32)
    if outliers:
        x[:, rng.choice(K, max(1, K // 200), replace=False)] *= 50
    return torch.from_numpy(x).to(dtype).cuda()[:, :K]


def np32(t):
    return t.float().cpu().numpy()


def np_codes(t):
    return t.view(torch.uint8).cpu().numpy()


def np_scales(t):
    return t.cpu().numpy() if t.dtype == torch.float32 else t.view(torch.uint8).cpu().numpy()


def synced(F):
    torch.cuda.synchronize()
    assert F.fp4q_device_status() == F.FP4Q_OK


# ---------------------------------------------------------------- quantizer

QUANT_SHAPES = [(1, 16), (1, 128), (3, 144), (5, 4096), (129, 272), (256, 384), (333, 5008), (1, 32784), (700, 16)]


def check_quantized(F, x, rows, fmt, codes, scales):
    ref_c, ref_s = o.quantize(np32(x), rows, fmt)
    assert np.array_equal(np_scales(scales), ref_s, equal_nan=fmt == o.F32)
    assert np.array_equal(np_codes(codes), ref_c)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
@pytest.mark.parametrize("M,K", QUANT_SHAPES)
def test_quantizer(F, M, K, fmt, rows):
    for dtype, pad in ((BF16, 0), (FP16, 24)):
        x = activations(M, K, M + K, dtype, pad)
        codes, scales = F.quantize_fp8(x, rows, fmt)
        synced(F)
        check_quantized(F, x, rows, fmt, codes, scales)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=["bf16", "fp16"])
def test_quantizer_at_the_edges(F, dtype, fmt, rows):
    """Blocks of zeros (of both signs), of the smallest and the largest values, with a NaN, with an
    infinity; values on midpoints of the codes; block maxima on and next to powers of two times 448."""
    K = 128 * 12
    x = torch.zeros((4, K))
    f = torch.finfo(dtype)
    x[:, 128:256] = -0.0
    x[:, 256:384] = f.smallest_normal * torch.linspace(-1, 1, 128)
    x[:, 384:512] = f.max * torch.linspace(-1, 1, 128)
    x[:, 512:640] = torch.linspace(-3, 3, 128)
    x[1, 520] = float("nan")
    x[:, 640:768] = torch.linspace(-3, 3, 128)
    x[2, 700] = float("-inf")
    mids = torch.tensor(o._MIDPOINTS[o._MIDPOINTS >= 0.25][:127], dtype=torch.float32)
    x[:, 768:896] = torch.cat([mids, torch.zeros(128 - mids.numel())])
    x[:, 768] = 448.0
    for i, top in enumerate((448.0, 452.0, 444.0, 224.0)):
        x[:, 896 + 128 * i:1024 + 128 * i] = torch.linspace(-1, 1, 128) * 100
        x[:, 900 + 128 * i] = top
    x[:, 1408:] = torch.linspace(0, 1, 128) * 2.0 ** -14
    x = x.to(dtype).cuda()
    codes, scales = F.quantize_fp8(x, rows, fmt)
    synced(F)
    xn = np32(x)
    ref_c, ref_s = o.quantize(xn, rows, fmt)
    assert np.array_equal(np_scales(scales), ref_s, equal_nan=fmt == o.F32)
    got = np_codes(codes)
    # below a scale of 2^-90 the quotient may be one ulp off, which the code of a midpoint shows
    tiny = o.spread(o.scale_values(ref_s), rows, 4, K) < 2.0 ** -90
    assert np.array_equal(got[~tiny], ref_c[~tiny])
    s = o.spread(o.scale_values(ref_s), rows, 4, K)
    q = xn.astype(np.float64) / s
    lo, hi = o.e4m3_decode(o.e4m3_encode(q - np.abs(q) * 4 * U)), o.e4m3_decode(o.e4m3_encode(q + np.abs(q) * 4 * U))
    v = o.e4m3_decode(got)
    assert np.all((lo <= v) & (v <= hi) | ~tiny)


def test_quantizer_writes_its_outputs_only(F):
    from gpu_util import Guarded
    x = activations(37, 272, 5)
    for rows, n in ((1, 37 * 3), (128, 3)):
        c, s = Guarded(37 * 272), Guarded(n * 4)
        F.fp4q_quantize_fp8(0, 0, rows, x, 272, 37, 272, c.view, s.view)
        synced(F)
        c.check("codes"), s.check("scales")
        ref_c, ref_s = o.quantize(np32(x), rows, 0)
        assert np.array_equal(c.numpy().reshape(37, 272), ref_c)
        assert np.array_equal(s.numpy().view(np.float32).reshape(ref_s.shape), ref_s)


# ---------------------------------------------------------------- norm

def check_norm(F, x, r, w, eps, fmt, codes, scales, stored):
    M, K = x.shape
    xn, rn = np32(x), None if r is None else np32(r)
    if r is not None:
        assert torch.equal(stored.cpu(), (x.float().cpu() + r.float().cpu()).to(x.dtype))
    _, y = o.rmsnorm(xn, rn, np32(w), eps)
    A = o.blocks_amax(y, 1)
    got_s = np_scales(scales)
    sv = o.scale_values(got_s)
    if fmt == o.F32:
        want = np.maximum(A / 448, 2.0 ** -126)
        assert np.all(np.abs(sv - want) <= 31 * U * want)
    else:
        lo, hi = o.scale_of(A * (1 - 31 * U), fmt)[0], o.scale_of(A * (1 + 31 * U), fmt)[0]
        assert np.all((lo <= got_s) & (got_s <= hi))
    q = y / o.spread(sv, 1, M, K)
    v = o.e4m3_decode(np_codes(codes))
    lo = o.e4m3_decode(o.e4m3_encode(q - np.abs(q) * 33 * U))
    hi = o.e4m3_decode(o.e4m3_encode(q + np.abs(q) * 33 * U))
    assert np.all((lo <= v) & (v <= hi))


NORM_SHAPES = [(1, 16), (1, 128), (2, 144), (5, 496), (3, 512), (7, 528), (1, 4096), (300, 4096), (4, 8192), (3, 8208),
               (16, 14336), (2, 16384), (2, 16400), (1, 32768), (1000, 272)]


@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
@pytest.mark.parametrize("M,K", NORM_SHAPES)
def test_norm(F, M, K, fmt):
    for dtype, pad, res in ((BF16, 0, True), (FP16, 40, True), (BF16, 8, False)):
        x = activations(M, K, M + K, dtype, pad)
        r = activations(M, K, M + K + 1, dtype, pad) if res else None
        w = (1 + 0.1 * torch.randn(K, generator=torch.Generator().manual_seed(K))).to(dtype).cuda()
        codes, scales, stored = F.add_rmsnorm_fp8(x, r, w, 1e-5, fmt)
        synced(F)
        assert (stored is None) == (r is None)
        check_norm(F, x, r, w, 1e-5, fmt, codes, scales, stored)


def test_norm_in_place(F):
    """The sum stored over the residual and over x, with strided rows: what lies between rows stays."""
    M, K = 65, 1040
    x, r = activations(M, K, 1, BF16, 16), activations(M, K, 2, BF16, 8)
    w = torch.ones(K, dtype=BF16, device="cuda")
    ref = F.add_rmsnorm_fp8(x, r, w, 1e-6)
    for which in ("residual", "x"):
        x2, r2 = x._base.clone()[:, :K], r._base.clone()[:, :K]
        out = r2 if which == "residual" else x2
        tail = out._base[:, K:].clone()
        got = F.add_rmsnorm_fp8(x2, r2, w, 1e-6, residual_out=out)
        synced(F)
        assert got[2].data_ptr() == out.data_ptr()
        for a, b in zip(got[:2] + (out,), ref):
            assert torch.equal(a.view(torch.uint8) if a.element_size() == 1 else a,
                               b.view(torch.uint8) if b.element_size() == 1 else b)
        assert torch.equal(out._base[:, K:], tail)
        other, orig = (x2, x) if which == "residual" else (r2, r)
        assert torch.equal(other, orig)


def test_norm_rows_stand_alone(F):
    """A row's result depends on that row alone: zeros, a NaN, an infinity in others change nothing, and
    the row of zeros (eps > 0) gives zero codes at the smallest scale."""
    M, K = 9, 1024
    x, r = activations(M, K, 3), activations(M, K, 4)
    w = torch.ones(K, dtype=BF16, device="cuda")
    ref = F.add_rmsnorm_fp8(x, r, w, 1e-6)
    x2, r2 = x.clone(), r.clone()
    x2[2], r2[2] = 0, 0
    x2[4, 7] = float("nan")
    r2[6, 1000] = float("inf")
    codes, scales, stored = F.add_rmsnorm_fp8(x2, r2, w, 1e-6)
    synced(F)
    c, s, c0, s0 = np_codes(codes), np_scales(scales), np_codes(ref[0]), np_scales(ref[1])
    for i in (0, 1, 3, 5, 7, 8):
        assert np.array_equal(c[i], c0[i]) and np.array_equal(s[i], s0[i]) and torch.equal(stored[i], ref[2][i])
    assert np.all(c[2] & 0x7F == 0) and np.all(s[2] == np.float32(2.0 ** -126))
    assert np.all(c[4] == 0x7F) and np.all(np.isnan(s[4]))
    # 1 / sqrt(inf) = 0: finite entries become 0, the infinity NaN
    assert np.isnan(s[6, 1000 // 128]) and np.all(s[6, :7] == np.float32(2.0 ** -126))
    assert np.isnan(np32(stored)[4, 7]) and np.isinf(np32(stored)[6, 1000])


# ---------------------------------------------------------------- GEMM

GEMM_SHAPES = [  # few rows: one, a batch, each tile of tokens, an odd N, K below and off a block
    (1, 128, 128), (1, 1, 16), (1, 4096, 4096), (16, 1000, 2064), (17, 257, 144), (32, 129, 1040), (33, 4104, 512),
    (64, 256, 4096), (5, 7, 8208),
    # many rows: both tiles, ragged in all directions
    (65, 130, 144), (128, 256, 128), (129, 257, 1040), (200, 33, 5008), (333, 4104, 784), (1000, 8200, 400),
    (2500, 2056, 272)]


def make_operands(F, M, N, K, fmt, seed):
    a = F.quantize_fp8(activations(M, K, seed), 1, fmt)
    rng = np.random.default_rng(seed + 1)
    w = torch.from_numpy(rng.laplace(0, 0.02, (N, K)).astype(np.float32)).to(BF16).cuda()
    return a, F.quantize_fp8(w, 128, fmt)


def check_gemm(d, a, b, K):
    A, B = o.operand(np_codes(a[0]), np_scales(a[1]), 1), o.operand(np_codes(b[0]), np_scales(b[1]), 128)
    ref, mag = A @ B.T, np.abs(A) @ np.abs(B).T
    kb = -(-K // 128)
    half = torch.finfo(d.dtype).eps / 2
    # fp16 results below its smallest normal number are off by half of a fixed step
    bound = (132 + kb + 10) * U * mag + half * np.maximum(np.abs(ref), torch.finfo(d.dtype).smallest_normal)
    err = np.abs(d.double().cpu().numpy() - ref)
    assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_gemm(F, M, N, K, fmt):
    a, b = make_operands(F, M, N, K, fmt, M + N + K)
    for dtype in (BF16, FP16, F32):
        d = F.gemm_fp8(*a, *b, out_dtype=dtype)
        again = F.gemm_fp8(*a, *b, out_dtype=dtype)
        synced(F)
        check_gemm(d, a, b, K)
        assert torch.equal(d, again)


@pytest.mark.parametrize("M,N,K", [(1, 300, 1040), (16, 512, 2048), (40, 130, 400), (130, 1000, 528), (700, 6000, 512)])
def test_gemm_of_small_integers_is_exact(F, M, N, K):
    """Codes in {-2 .. 2} and scales that are powers of two in [1/4, 4]: every sum is exact in fp32, in
    whatever order it is taken, so the result is equal to the product."""
    rng = np.random.default_rng(K + M)
    kb = -(-K // 128)
    qa, qb = rng.integers(-2, 3, (M, K)).astype(np.float32), rng.integers(-2, 3, (N, K)).astype(np.float32)
    ea, eb = rng.integers(-2, 3, (M, kb)), rng.integers(-2, 3, (-(-N // 128), kb))
    ac, bc = (torch.from_numpy(q).cuda().to(torch.float8_e4m3fn) for q in (qa, qb))
    A = qa.astype(np.float64) * o.spread(np.exp2(ea), 1, M, K)
    B = qb.astype(np.float64) * o.spread(np.exp2(eb), 128, N, K)
    for make in (lambda e: torch.from_numpy(np.exp2(e).astype(np.float32)).cuda(),
                 lambda e: torch.from_numpy((e + 127).astype(np.uint8)).cuda().view(torch.float8_e8m0fnu)):
        d = F.gemm_fp8(ac, make(ea), bc, make(eb), out_dtype=F32)
        synced(F)
        assert np.array_equal(d.double().cpu().numpy(), A @ B.T)


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
def test_gemm_carries_nan(F, M, fmt):
    """A NaN code spoils its row (of A) or column (of B), a NaN scale likewise, and nothing else."""
    N, K = 300, 400
    a, b = make_operands(F, M, N, K, fmt, 8)
    ref = F.gemm_fp8(*a, *b, out_dtype=F32)
    ac, sa, bc, sb = a[0].clone(), a[1].clone(), b[0].clone(), b[1].clone()
    ac.view(torch.uint8)[1, 390] = 0x7F
    bc.view(torch.uint8)[7, 3] = 0xFF
    if fmt == o.F32:
        sa[2, 1], sb[1, 3] = float("nan"), float("nan")
    else:
        sa.view(torch.uint8)[2, 1], sb.view(torch.uint8)[1, 3] = 255, 255
    d = F.gemm_fp8(ac, sa, bc, sb, out_dtype=F32)
    synced(F)
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[1:3], bad[:, 7], bad[:, 128:256] = True, True, True
    assert torch.equal(torch.isnan(d), bad)
    assert torch.equal(d[~bad], ref[~bad])


def test_gemm_of_the_extreme_scale_bytes(F):
    """E8M0 byte 0 is 2^-127 and byte 254 is 2^127: their product with codes of one is exact."""
    M, N, K = 4, 130, 128
    one = torch.ones((M, K), device="cuda").to(torch.float8_e4m3fn)
    b = torch.ones((N, K), device="cuda").to(torch.float8_e4m3fn)
    for x, y in ((0, 254), (254, 0), (0, 127), (127, 254 - 7), (127, 0)):
        sa = torch.full((M, 1), x, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        sb = torch.full((2, 1), y, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        d = F.gemm_fp8(one, sa, b, sb, out_dtype=F32)
        synced(F)
        assert torch.all(d.double() == 128 * 2.0 ** (x + y - 254)), (x, y)


def test_gemm_writes_its_output_only(F):
    from gpu_util import Guarded
    for M, N, K, dt, size in ((3, 70, 144, 0, 2), (130, 257, 272, 2, 4), (130, 264, 272, 1, 2)):
        a, b = make_operands(F, M, N, K, 0, 3)
        d = Guarded(M * N * size)
        F.fp4q_gemm_fp8(0, dt, a[0], a[1], b[0], b[1], M, N, K, d.view)
        synced(F)
        d.check("d")


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("M", [1, 48, 300])
@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
def test_a_layer(F, M, fmt):
    """norm -> up projection -> quantizer -> down projection, on a stream of its own and captured into a
    graph that is replayed on new inputs: the replays give what the calls give."""
    H, I = 1040, 2064
    w = (1 + 0.1 * torch.randn(H)).to(BF16).cuda()
    up = F.quantize_fp8(activations(I, H, 1, outliers=False) * 0.02, 128, fmt)
    down = F.quantize_fp8(activations(H, I, 2, outliers=False) * 0.02, 128, fmt)
    x, r = activations(M, H, 3), activations(M, H, 4)

    def layer():
        c, s, stored = F.add_rmsnorm_fp8(x, r, w, 1e-6, fmt)
        h = F.gemm_fp8(c, s, *up)
        c2, s2 = F.quantize_fp8(h, 1, fmt)
        return c, s, stored, h, c2, s2, F.gemm_fp8(c2, s2, *down)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = layer()
    torch.cuda.current_stream().wait_stream(side)
    synced(F)
    c, s, stored, h, c2, s2, d = eager
    check_norm(F, x, r, w, 1e-6, fmt, c, s, stored)
    check_gemm(h, (c, s), up, H)
    check_quantized(F, h, 1, fmt, c2, s2)
    check_gemm(d, (c2, s2), down, I)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer()
    for seed in (3, 20):
        x.copy_(activations(M, H, seed))
        r.copy_(activations(M, H, seed + 1))
        graph.replay()
        want = layer()
        synced(F)
        for a, b in zip(captured, want):
            assert torch.equal(a.view(torch.uint8) if a.element_size() == 1 else a,
                               b.view(torch.uint8) if b.element_size() == 1 else b)


def test_calls_on_two_streams(F):
    """Calls on two streams at once share nothing."""
    args = [make_operands(F, M, 4104, 4096, 0, M) for M in (4, 300)]
    ref = [F.gemm_fp8(*a, *b) for a, b in args]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in args]
    outs = [[], []]
    for _ in range(10):
        for i, (a, b) in enumerate(args):
            outs[i].append(F.gemm_fp8(*a, *b, out=torch.empty_like(ref[i]), stream=streams[i]))
    synced(F)
    for i in range(2):
        assert all(torch.equal(d, ref[i]) for d in outs[i])


def test_empty_calls(F):
    e = torch.empty((0, 256), dtype=BF16, device="cuda")
    c, s = F.quantize_fp8(e)
    assert c.shape == (0, 256) and s.shape == (0, 2)
    w = torch.ones(256, dtype=BF16, device="cuda")
    c, s, r = F.add_rmsnorm_fp8(e, e, w, 1e-6)
    assert c.shape == (0, 256) and r.shape == (0, 256)
    b = F.quantize_fp8(activations(40, 256, 1), 128)
    assert F.gemm_fp8(c, s, *b).shape == (0, 40)
    z = F.quantize_fp8(torch.empty((3, 0), dtype=BF16, device="cuda"))
    assert z[0].shape == (3, 0) and z[1].shape == (3, 0)
    synced(F)


def test_refusals_of_the_tensor_calls(F):
    x = activations(4, 256, 1)
    w = torch.ones(256, dtype=BF16, device="cuda")
    bad = [lambda: F.quantize_fp8(x.float()), lambda: F.quantize_fp8(x.cpu()), lambda: F.quantize_fp8(x.t()),
           lambda: F.quantize_fp8(x, 64), lambda: F.quantize_fp8(x, 1, 7),
           lambda: F.quantize_fp8(x, codes=torch.empty((4, 256), dtype=torch.uint8, device="cuda")),
           lambda: F.add_rmsnorm_fp8(x, x.half(), w, 1e-6), lambda: F.add_rmsnorm_fp8(x, x[:3], w, 1e-6),
           lambda: F.add_rmsnorm_fp8(x, None, w.half(), 1e-6), lambda: F.add_rmsnorm_fp8(x, None, w[:128], 1e-6),
           lambda: F.add_rmsnorm_fp8(x, None, w, 1e-6, residual_out=x)]
    c, s = F.quantize_fp8(x)
    bc, bs = F.quantize_fp8(x, 128)
    _, s8 = F.quantize_fp8(x, 1, 1)
    bad += [lambda: F.gemm_fp8(c, s8, bc, bs), lambda: F.gemm_fp8(c, s, bc, s), lambda: F.gemm_fp8(c[:, :128], s, bc, bs),
            lambda: F.gemm_fp8(c, s, bc, bs, out_dtype=torch.float64),
            lambda: F.gemm_fp8(c, s, bc, bs, out=torch.empty((4, 5), dtype=BF16, device="cuda"))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call, status in ((lambda: F.quantize_fp8(activations(4, 24, 1)), F.FP4Q_ERR_SHAPE),
                         (lambda: F.add_rmsnorm_fp8(x, None, w, -1.0), F.FP4Q_ERR_ARG),
                         (lambda: F.add_rmsnorm_fp8(x[:3], x[:3], w, 1e-6, residual_out=x[1:]), F.FP4Q_ERR_ARG)):
        with pytest.raises(F.Fp4qError) as e:
            call()
        assert e.value.status == status
    torch.cuda.synchronize()
