"""The tensor calls with a stream given by hand: they run on it, and what they allocate belongs to it."""

import pytest
import torch

pytestmark = pytest.mark.gpu

M, H, N = 512, 2048, 4096
BF16 = torch.bfloat16
DELAY = 100_000_000   # cycles, some 50 ms: the host queues the rest of a test meanwhile


@pytest.fixture(scope="module")
def F(cuda_device):
    from microscaling_fp4_quantization_b200 import fp4q
    return fp4q


def values(rows, cols, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((rows, cols), generator=g, device="cuda").to(BF16)


def same(a, b):
    as_bytes = lambda t: t.contiguous().view(torch.uint8)
    return torch.equal(as_bytes(a), as_bytes(b))


@pytest.fixture(scope="module")
def operands(F):
    x, r, w = values(M, H, 1), values(M, H, 2), values(1, H, 3)[0]
    b = F.quantize_fp8(values(N, H, 4), 128)
    plan = F.fp4q_plan_create(F.FP4Q_NVFP4, 16, 16, F.FP4Q_SCALE_NV_DYNAMIC)
    a = F.quantize_fp8(x)
    torch.cuda.synchronize()
    return x, r, w, a, b, plan


def calls(F, operands):
    x, r, w, a, b, plan = operands
    return {"quantize": lambda s, x=x: F.quantize_fp8(x, stream=s),
            "tiles": lambda s, x=x: F.quantize_fp8(x, 128, F.FP4Q_FP8_SCALE_E8M0, stream=s),
            "norm": lambda s, x=x: F.add_rmsnorm_fp8(x, r, w, 1e-6, stream=s),
            "product": lambda s, x=x: (F.gemm_fp8(*a, *b, stream=s),),
            "rotate": lambda s, x=x: F.rotate_quantize(plan, x, stream=s)}


NAMES = ["quantize", "tiles", "norm", "product", "rotate"]


def handle_of(kind, stream):
    return stream if kind == "object" else stream.cuda_stream


@pytest.mark.parametrize("kind", ["object", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_allocated_on_the_call_s_stream(F, operands, name, kind):
    """A freed output goes back to the given stream: the current stream's next tensor of its size lies
    elsewhere, so nothing that is queued there can write over what the given stream still reads."""
    side = torch.cuda.Stream()
    out = calls(F, operands)[name](handle_of(kind, side))
    sizes = [t.numel() * t.element_size() for t in out]
    places = [(t.data_ptr(), t.data_ptr() + n) for t, n in zip(out, sizes)]
    torch.cuda.synchronize()
    del out
    for n in sizes:
        again = torch.empty(n, dtype=torch.uint8, device="cuda")
        at = again.data_ptr()
        assert not any(at < hi and lo < at + n for lo, hi in places)


@pytest.mark.parametrize("kind", ["object", "handle"])
def test_a_chain_whose_intermediates_are_dropped(F, operands, kind):
    """Norm and product on a side stream, the codes and scales dropped before the product has run, and the
    current stream's memory filled meanwhile."""
    x, r, w, _, b, _ = operands
    c, s, _ = F.add_rmsnorm_fp8(x, r, w, 1e-6)
    want = F.gemm_fp8(c, s, *b)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c, s, stored = F.add_rmsnorm_fp8(x, r, w, 1e-6, stream=handle_of(kind, side))
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
    d = F.gemm_fp8(c, s, *b, stream=handle_of(kind, side))
    shapes = [c.numel(), s.numel() * 4]
    del c, s, stored
    fills = [torch.full((n,), 0x7F, dtype=torch.uint8, device="cuda") for n in shapes for _ in range(4)]
    torch.cuda.synchronize()
    assert F.fp4q_device_status() == F.FP4Q_OK
    assert same(d, want)
    assert all(bool((t == 0x7F).all()) for t in fills)


@pytest.mark.parametrize("kind", ["object", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads_is_left_alone(F, operands, name, kind):
    """Tensors freed while the current stream has yet to read them: a call on another stream does not take
    their memory."""
    call = calls(F, operands)[name]
    side = torch.cuda.Stream()
    want = call(None)
    sizes = [t.numel() * t.element_size() for t in want]
    torch.cuda.synchronize()
    for _ in range(2):
        kept = []
        held = [torch.full((n,), 0x2B, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda._sleep(DELAY)
        kept = [h.clone() for h in held]
        del held
        got = call(handle_of(kind, side))
        torch.cuda.synchronize()
        assert all(bool((t == 0x2B).all()) for t in kept)
        assert all(same(a, b) for a, b in zip(got, want))
        del kept, got


@pytest.mark.parametrize("kind", ["object", "handle", "legacy default"])
@pytest.mark.parametrize("name", ["quantize", "tiles", "norm", "rotate"])
def test_calls_run_on_the_given_stream(F, operands, name, kind):
    """The input is written late on the given stream: a call on any other would read what was there before."""
    call = calls(F, operands)[name]
    new = values(M, H, 9)
    want = call(None, new)
    x = operands[0].clone()
    side = torch.cuda.default_stream() if kind == "legacy default" else torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
        x.copy_(new)
    got = call(0 if kind == "legacy default" else handle_of(kind, side), x)
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["object", "handle"])
@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_error_pass_waits_for_the_given_stream(F, fmt, kind):
    """The energies come back as numbers: they are read once the given stream has them."""
    if fmt == "nvfp4":
        plan = F.fp4q_plan_create(F.FP4Q_NVFP4, 16, 16, F.FP4Q_SCALE_NV_DYNAMIC)
    else:
        plan = F.fp4q_plan_create(F.FP4Q_MXFP4, 32, 32, F.FP4Q_SCALE_FLOOR_OCP)
    new = values(M, H, 12)
    want = F.quant_error(plan, new)
    x = values(M, H, 11)
    assert F.quant_error(plan, x) != want   # (and leaves other energies in the memory that is reused)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(DELAY)
        x.copy_(new)
    assert F.quant_error(plan, x, stream=handle_of(kind, side)) == want


def test_a_stream_of_another_device_is_refused(F, operands):
    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 1), 0
    for name in NAMES:
        with pytest.raises(ValueError):
            calls(F, operands)[name](Elsewhere())
    with pytest.raises(ValueError):
        F.quant_error(operands[-1], operands[0], stream=Elsewhere())


def test_a_captured_call_on_a_given_stream(F, operands):
    """A call with the capturing stream given allocates from the graph's memory, and replays."""
    x, _, _, _, b, _ = operands
    live = x.clone()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        c, s = F.quantize_fp8(live, stream=side)
        d = F.gemm_fp8(c, s, *b, stream=side.cuda_stream)
    for seed in (21, 22):
        live.copy_(values(M, H, seed))
        graph.replay()
        want = F.gemm_fp8(*F.quantize_fp8(live), *b)
        torch.cuda.synchronize()
        assert same(d, want)
