"""Every kernel of the 8-bit GEMM at the sizes that pick it, sizes past 32-bit offsets, and the calls the
documentation allows at their edges.  Tolerances as in test_fp8.py."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as o
from test_fp8 import (BF16, F32, FP16, activations, check_gemm, check_quantized, make_operands, np32, np_codes,
                      np_scales, synced)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def F(cuda_device):
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


# (M, N, K): few rows split over 1 .. 8 CTAs and over several tiles of tokens; 128 x 128 and 256 x 128
# tiles; the widest tiles; each with whole and with short last blocks, odd numbers of blocks, and more
# tiles than are resident at once
SHAPES = [(1, 19000, 272), (2, 128, 2048), (3, 250, 1536), (16, 384, 1536), (16, 640, 5008), (9, 1300, 1040),
          (20, 1000, 1040), (32, 2300, 2064), (33, 128, 4096), (64, 500, 1296), (100, 260, 2048), (150, 1300, 784),
          (70, 16000, 272), (130, 10000, 144), (1000, 2050, 400), (700, 4104, 1040), (640, 12000, 272), (1030, 4360, 1168),
          (3000, 3100, 656)]


@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gemm_variants(F, M, N, K, fmt):
    a, b = make_operands(F, M, N, K, fmt, M + N)
    d = F.gemm_fp8(*a, *b, out_dtype=F32)
    again = F.gemm_fp8(*a, *b, out_dtype=F32)
    synced(F)
    check_gemm(d, a, b, K)
    assert torch.equal(d, again)


@pytest.mark.parametrize("M,N,K", [(2000, 4500, 528), (640, 12000, 272)])
@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
def test_wide_tiles_of_small_integers_are_exact(F, M, N, K, fmt):
    """As test_gemm_of_small_integers_is_exact, on the kernels for many rows; a few NaN scales spoil their
    rows and columns and nothing else."""
    g = torch.Generator(device="cuda").manual_seed(K)
    kb = -(-K // 128)
    qa = torch.randint(-2, 3, (M, K), generator=g, device="cuda").float()
    qb = torch.randint(-2, 3, (N, K), generator=g, device="cuda").float()
    ea = torch.randint(-2, 3, (M, kb), generator=g, device="cuda")
    eb = torch.randint(-2, 3, (-(-N // 128), kb), generator=g, device="cuda")
    k = torch.arange(K, device="cuda") // 128
    n = torch.arange(N, device="cuda") // 128
    ref = (qa.double() * torch.exp2(ea.double())[:, k]) @ (qb.double() * torch.exp2(eb.double())[n][:, k]).T
    ac, bc = qa.to(torch.float8_e4m3fn), qb.to(torch.float8_e4m3fn)
    if fmt == o.F32:
        sa, sb = torch.exp2(ea.float()), torch.exp2(eb.float())
    else:
        sa, sb = ((e + 127).to(torch.uint8).view(torch.float8_e8m0fnu) for e in (ea, eb))
    d = F.gemm_fp8(ac, sa, bc, sb, out_dtype=F32)
    synced(F)
    assert torch.equal(d.double(), ref)
    if fmt == o.F32:
        sa[M - 1, kb - 1] = float("nan")
        sb[1, 0] = float("nan")
    else:
        sa.view(torch.uint8)[M - 1, kb - 1] = 255
        sb.view(torch.uint8)[1, 0] = 255
    d = F.gemm_fp8(ac, sa, bc, sb, out_dtype=F32)
    synced(F)
    bad = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    bad[M - 1], bad[:, 128:256] = True, True
    assert torch.equal(torch.isnan(d), bad)
    assert torch.equal(d[~bad].double(), ref[~bad])


def test_wide_tiles_at_the_extreme_scale_bytes(F):
    """E8M0 bytes 0 and 254 on the kernel whose scales the tensor core applies."""
    M, N, K = 2560, 2240, 128
    one = torch.ones((M, K), device="cuda").to(torch.float8_e4m3fn)
    b = torch.ones((N, K), device="cuda").to(torch.float8_e4m3fn)
    for x, y in ((0, 254), (254, 0), (0, 127), (127, 247), (127, 0)):
        sa = torch.full((M, 1), x, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        sb = torch.full((-(-N // 128), 1), y, dtype=torch.uint8, device="cuda").view(torch.float8_e8m0fnu)
        d = F.gemm_fp8(one, sa, b, sb, out_dtype=F32)
        synced(F)
        assert torch.all(d.double() == 128 * 2.0 ** (x + y - 254)), (x, y)


def test_arrays_at_the_least_alignment(F):
    """D on 16 bytes but not on 32, E8M0 scales on single bytes, fp32 scales on 4: the results are those of
    aligned arrays, and what lies around D stays."""
    for M, N, K in ((5, 264, 1040), (700, 4104, 1040), (2500, 2056, 512)):
        for fmt in (o.F32, o.E8M0):
            a, b = make_operands(F, M, N, K, fmt, 6)
            ref = F.gemm_fp8(*a, *b)

            def shifted(t, by):
                raw = torch.zeros(t.numel() * t.element_size() + 64, dtype=torch.uint8, device="cuda")
                raw[by:by + t.numel() * t.element_size()] = t.contiguous().view(torch.uint8).flatten()
                return raw[by:by + t.numel() * t.element_size()]

            by = 4 if fmt == o.F32 else 1
            sa, sb = shifted(a[1], by), shifted(b[1], by)
            raw = torch.full((M * N * 2 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
            F.fp4q_gemm_fp8(fmt, F.FP4Q_DTYPE_BF16, a[0], sa, b[0], sb, M, N, K, raw.data_ptr() + 16)
            synced(F)
            assert torch.equal(raw[16:16 + M * N * 2].view(BF16).view(M, N), ref)
            assert torch.all(raw[:16] == 0xA5) and torch.all(raw[16 + M * N * 2:] == 0xA5)


@pytest.mark.parametrize("dtype", [BF16, FP16, F32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
@pytest.mark.parametrize("M,N,K", [(5, 1301, 272), (150, 1299, 784), (150, 1302, 784), (333, 4102, 1040),
                                   (333, 4109, 1040), (640, 12001, 272), (1025, 4358, 400), (3000, 3099, 656),
                                   (2049, 6, 272), (700, 1, 528)])
def test_rows_of_no_alignment_are_exact(F, M, N, K, fmt, dtype):
    """N that leaves D's rows without 16-byte alignment, odd and even, on the kernels for few, some and many
    rows.  Small integers and scales of one, so that every sum is exact in fp32 and each output is its one
    rounding; what lies around D stays."""
    g = torch.Generator(device="cuda").manual_seed(N)
    kb = -(-K // 128)
    a = torch.randint(-2, 3, (M, K), generator=g, device="cuda").float()
    b = torch.randint(-2, 3, (N, K), generator=g, device="cuda").float()
    ref = (a.double() @ b.double().T).to(dtype)
    ac, bc = a.to(torch.float8_e4m3fn), b.to(torch.float8_e4m3fn)
    if fmt == o.F32:
        sa, sb = (torch.ones((r, kb), device="cuda") for r in (M, -(-N // 128)))
    else:
        sa, sb = (torch.full((r, kb), 127, dtype=torch.uint8, device="cuda") for r in (M, -(-N // 128)))
    size = ref.element_size()
    code = {BF16: F.FP4Q_DTYPE_BF16, FP16: F.FP4Q_DTYPE_FP16, F32: F.FP4Q_DTYPE_F32}[dtype]
    raw = torch.full((M * N * size + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    F.fp4q_gemm_fp8(fmt, code, ac, sa, bc, sb, M, N, K, raw.data_ptr() + 16)
    synced(F)
    end = 16 + M * N * size
    assert torch.equal(raw[16:end].view(dtype).view(M, N), ref)
    assert torch.all(raw[:16] == 0xA5) and torch.all(raw[end:] == 0xA5)


@pytest.mark.parametrize("residual", [False, True], ids=["alone", "residual"])
@pytest.mark.parametrize("K", [16, 528, 4096, 5008, 8192, 14336, 16384, 16400, 32768])
def test_norm_of_a_row_is_the_same_in_any_batch(F, K, residual):
    """One token, a few and more than there are SMs: the square sum of a row keeps its order, to the bit."""
    M = 700
    x, r = activations(M, K, K), activations(M, K, K + 1)
    w = activations(1, K, K + 2)[0]
    ref = F.add_rmsnorm_fp8(x, r if residual else None, w, 1e-6)
    for lo, hi in ((0, 1), (3, 20), (40, 188), (100, 249), (699, 700)):
        part = F.add_rmsnorm_fp8(x[lo:hi], r[lo:hi] if residual else None, w, 1e-6)
        synced(F)
        assert torch.equal(part[1], ref[1][lo:hi])
        assert torch.equal(part[0].view(torch.uint8), ref[0][lo:hi].view(torch.uint8))
        if residual:
            assert torch.equal(part[2], ref[2][lo:hi])


@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
def test_norm_of_zeros_without_eps(F, fmt):
    """0 / sqrt(0 + 0) is NaN throughout the row, and in that row alone."""
    x = activations(3, 528, 1)
    x[1] = 0
    w = torch.ones(528, dtype=BF16, device="cuda")
    codes, scales, _ = F.add_rmsnorm_fp8(x, None, w, 0.0, fmt)
    synced(F)
    c = np_codes(codes)
    assert np.all(c[1] & 0x7F == 0x7F) and np.all(c[[0, 2]] & 0x7F != 0x7F)
    assert torch.all(torch.isnan(scales.float()[1])) and not torch.any(torch.isnan(scales.float()[[0, 2]]))


def test_quantize_past_32_bit_offsets(F):
    """More than 2^32 bytes of input and 2^31 of codes: rows from the start, around the borders and the end."""
    M, K = 140000, 16384
    x = torch.empty((M, K), dtype=BF16, device="cuda")
    step = 10000
    for i in range(0, M, step):
        x[i:i + step] = torch.randn((step, K), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda")
    rows = [0, 65535, 65536, 131071, 131072, M - 128, M - 1]
    for block_rows in (1, 128):
        codes, scales = F.quantize_fp8(x, block_rows, o.E8M0)
        synced(F)
        if block_rows == 1:
            check_quantized(F, x[rows], 1, o.E8M0, codes[rows], scales[rows])
        else:
            for t in (0, 511, 512, 1023, 1024, M // 128 - 1):
                check_quantized(F, x[128 * t:128 * t + 128], 128, o.E8M0, codes[128 * t:128 * t + 128], scales[t:t + 1])
        del codes, scales
    # the same rows as a strided view whose distance between rows passes 32 bits
    del x
    wide = torch.zeros((3, 1 << 31), dtype=BF16, device="cuda")
    wide[:, :400] = activations(3, 400, 2)
    v = wide[:, :400]
    codes, scales = F.quantize_fp8(v)
    w = torch.ones(400, dtype=BF16, device="cuda")
    n = F.add_rmsnorm_fp8(v, v, w, 1e-6, residual_out=v)
    synced(F)
    ref = F.add_rmsnorm_fp8(activations(3, 400, 2), activations(3, 400, 2), w, 1e-6)
    check_quantized(F, activations(3, 400, 2), 1, o.F32, codes, scales)
    assert np.array_equal(np_codes(n[0]), np_codes(ref[0])) and np.array_equal(np_scales(n[1]), np_scales(ref[1]))
    assert torch.equal(v, ref[2])


@pytest.mark.parametrize("fmt", [o.F32, o.E8M0], ids=["f32", "e8m0"])
def test_gemm_past_32_bit_offsets(F, fmt):
    """D of more than 2^32 elements, and codes of more than 2^31 bytes, on sampled rows."""
    M, N, K = 70000, 65536, 16
    a, b = make_operands(F, M, 128, K, fmt, 5)
    bc, bs = b[0].view(torch.uint8).repeat(N // 128, 1).view(torch.float8_e4m3fn), b[1]
    bs = bs.repeat(N // 128, 1) if fmt == o.F32 else bs.view(torch.uint8).repeat(N // 128, 1).view(torch.float8_e8m0fnu)
    d = F.gemm_fp8(*a, bc, bs)
    synced(F)
    rows = [0, 32767, 32768, 65535, 65536, M - 1]
    part = (a[0][rows].contiguous(), a[1][rows].contiguous())
    ref = F.gemm_fp8(*part, *b)
    check_gemm(ref, part, b, K)
    for i, r in enumerate(rows):
        assert torch.equal(d[r].view(N // 128, 128), ref[i].expand(N // 128, 128))
    del d, a, bc, bs
    M, N, K = 140000, 130, 16384
    ac = torch.empty((M, K), dtype=torch.float8_e4m3fn, device="cuda")
    src, b = make_operands(F, 1000, N, K, fmt, 7)
    for i in range(0, M, 1000):
        ac[i:i + 1000] = src[0]
    sa = src[1].repeat(M // 1000, 1) if fmt == o.F32 else \
        src[1].view(torch.uint8).repeat(M // 1000, 1).view(torch.float8_e8m0fnu)
    d = F.gemm_fp8(ac, sa, *b)
    synced(F)
    assert torch.equal(d, d[:1000].repeat(M // 1000, 1))
    check_gemm(d[:1000], src, b, K)


def test_two_graphs_replayed_at_once(F):
    """Two graphs of the same calls on two streams, replayed together: they share nothing."""
    def build(seed, M):
        x, r = activations(M, 2064, seed), activations(M, 2064, seed + 1)
        w = torch.ones(2064, dtype=BF16, device="cuda")
        b = F.quantize_fp8(activations(3000, 2064, seed + 2), 128)
        call = lambda: (lambda n: (n[2], F.gemm_fp8(n[0], n[1], *b)))(F.add_rmsnorm_fp8(x, r, w, 1e-6))
        want = call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = call()
        return g, got, want, (x, r, w, b)   # a graph does not keep its inputs alive
    graphs = [build(1, 7), build(10, 300)]
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(10):
        for (g, _, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    synced(F)
    for _, got, want, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_operands_may_repeat(F):
    """The same tensor as x and residual, and the same codes as A and B."""
    x = activations(128, 256, 3)
    w = torch.ones(256, dtype=BF16, device="cuda")
    c, s, stored = F.add_rmsnorm_fp8(x, x, w, 1e-6)
    assert torch.equal(stored, x + x)
    codes, scales = F.quantize_fp8(x, 1)
    tile = torch.full((1, 2), 0.5, device="cuda")
    d = F.gemm_fp8(codes, scales, codes, tile, out_dtype=F32)
    synced(F)
    check_gemm(d, (codes, scales), (codes, tile), 256)


def test_streams_given_by_hand(F):
    x = activations(4, 256, 1)
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        torch.cuda.synchronize()
        c, sc = F.quantize_fp8(x, stream=s)
        torch.cuda.synchronize()
        check_quantized(F, x, 1, o.F32, c, sc)


def test_norm_of_large_rows_saturates_as_documented(F):
    """A row whose square sum passes fp32's range: 1 / sqrt(inf) = 0, so zero codes."""
    x = torch.full((2, 256), 1e30, dtype=BF16, device="cuda")
    x[1] = 1.0
    c, s, _ = F.add_rmsnorm_fp8(x, None, torch.ones(256, dtype=BF16, device="cuda"), 0.0)
    synced(F)
    assert np.all(np_codes(c)[0] == 0) and np.all(np_codes(c)[1] == 0x7E)
    h = torch.full((1, 256), 60000.0, dtype=FP16, device="cuda")
    _, _, stored = F.add_rmsnorm_fp8(h, h, torch.ones(256, dtype=FP16, device="cuda"), 1e-6)
    assert torch.all(torch.isinf(stored)) and np.all(np.isinf(np32(stored)))
