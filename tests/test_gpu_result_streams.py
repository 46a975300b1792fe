"""Results that a call on a given stream allocates: they take no block that the
current stream still reads, and theirs is not taken while it reads them."""
import pytest

import fp8_device_reference as ref
import glq_inputs as gi
from gpu_helpers import Device

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SLEEP = 100_000_000  # cycles, about 50 ms


@pytest.fixture(scope="module")
def glq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import e8_lattice_codebook_b200 as glq
    return glq


def _calls(glq):
    gen = torch.Generator("cuda").manual_seed(61)
    x = torch.randn(24, 264, generator=gen, device="cuda").to(torch.bfloat16)
    linear = glq.Fp8Linear(*ref.random_weight(gen, 264, 264))
    experts = []
    for m, n in ((136, 264), (136, 264), (264, 136)):
        made = [ref.random_weight(gen, m, n) for _ in range(4)]
        experts += [torch.stack([w.view(torch.uint8) for w, _ in made]).view(torch.float8_e4m3fn),
                    torch.stack([s for _, s in made])]
    moe = glq.Fp8Moe(*experts, topk=2)
    logits = torch.randn(24, 4, generator=gen, device="cuda")
    q, s = glq.fp8_quantize(x)
    return {
        "quantize": lambda st: glq.fp8_quantize(x, stream=st)[0].view(torch.uint8),
        "linear": lambda st: linear(x, stream=st),
        "quantized": lambda st: linear.forward_quantized(q, s, stream=st),
        "dequant": lambda st: linear.dequant(stream=st),
        "moe": lambda st: moe(x, logits, stream=st),
    }


def _check(call):
    want = call(None).clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)  # loads what it needs
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    for _ in range(3):
        # a block that the current stream has yet to read, given back to the allocator
        block = torch.full_like(want, 3)
        torch.cuda._sleep(SLEEP)
        kept = block.clone()
        where = block.data_ptr()
        del block
        got = call(side)
        assert got.data_ptr() != where
        side.synchronize()
        # a result that the current stream reads late, given back while it has not
        torch.cuda._sleep(SLEEP)
        late = got.clone()
        where = got.data_ptr()
        del got
        again = call(side)
        assert again.data_ptr() != where
        torch.cuda.synchronize()
        assert torch.equal(again, want) and torch.equal(late, want)
        assert torch.equal(kept, torch.full_like(want, 3))


@pytest.mark.parametrize("name", ["quantize", "linear", "quantized", "dequant", "moe"])
def test_fp8_results(glq, name):
    _check(_calls(glq)[name])


def test_lattice_results(glq):
    L = gi.make_layer(62, 0, 264, 256, 3)
    layer = Device().layer(L)
    x = torch.randn(24, 256, generator=torch.Generator("cuda").manual_seed(62), device="cuda").to(torch.bfloat16)
    _check(lambda st: layer(x, stream=st))
    _check(lambda st: layer(x[:2], out_dtype=torch.float32, stream=st))
    _check(lambda st: layer.dequant(stream=st))
    _check(lambda st: layer.rht_input(x, stream=st))


def test_captured_on_a_given_stream(glq):
    """Calls on a stream that was forked from the capturing one, their results dropped while capturing or kept."""
    gen = torch.Generator("cuda").manual_seed(63)
    x = torch.randn(24, 264, generator=gen, device="cuda").to(torch.bfloat16)
    linear = glq.Fp8Linear(*ref.random_weight(gen, 264, 264))
    L = gi.make_layer(63, 0, 256, 264, 2)
    lattice = Device().layer(L)
    linear.reserve(24)
    lattice.reserve(24)
    want = lattice(linear(linear(x)))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        linear(x, stream=side)
        q, s = glq.fp8_quantize(linear(x, stream=side), stream=side)
        y = lattice(linear.forward_quantized(q, s, stream=side), stream=side)
        del q, s
        torch.cuda.current_stream().wait_stream(side)
        z = y + 0
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        want = lattice(linear(linear(x)))
        graph.replay()
        assert torch.equal(y, want) and torch.equal(z, want)
    torch.cuda.synchronize()
