"""The 8-bit float linear layer where a CTA takes tile after tile: stages,
accumulators and the buffers between CTAs are used again.  Against the
definition in 64 bits (tests/fp8_device_reference.py), on the device."""
import pytest

import fp8_device_reference as ref
from test_gpu_fp8 import LINEAR

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def glq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import e8_lattice_codebook_b200 as glq
    return glq


@pytest.fixture(scope="module")
def layer_of(glq):
    last = {}  # one layer at a time

    def make(m, n):
        if (m, n) not in last:
            last.clear()
            gen = torch.Generator("cuda").manual_seed(m + 3 * n)
            w, s = ref.random_weight(gen, m, n)
            last[m, n] = glq.Fp8Linear(w, s), w, s
        return last[m, n]

    yield make
    last.clear()


def _x(B, n, dtype):
    gen = torch.Generator("cuda").manual_seed(7 * B + n)
    x = torch.randn(B, n, generator=gen, device="cuda")
    x[:, ::37] *= 20.0
    return x.to(dtype)


def _check(layer, w, s, x, out):
    y = layer(x, out_dtype=out)
    layer.check()
    assert y.dtype == out
    want, bound = ref.linear(x, w, s, out)
    bad = ref.not_within(y, want, bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist())
    assert torch.equal(y, layer(x, out_dtype=out))  # and the same bits again


@pytest.mark.parametrize("m,n,B", [(9600, 8200, b) for b in (1, 2, 5, 16, 17, 32, 33, 64)] +
                         [(12160, 12296, b) for b in (1, 4, 29, 47)] + [(22400, 8200, b) for b in (1, 15)])
def test_parts_of_several_tiles(layer_of, m, n, B):
    """Clusters that split K and take more than one tile: the parts' buffers are written again."""
    layer, w, s = layer_of(m, n)
    plan = layer.plan(B)
    assert plan["kernel"] == 0 and plan["cluster"] > 1 and plan["items"] > plan["clusters"], plan
    _check(layer, w, s, _x(B, n, torch.bfloat16), torch.float32 if B & 1 else torch.bfloat16)


@pytest.mark.parametrize("m,n,B", [(20488, 264, b) for b in (1, 4, 5, 8, 9, 17, 33, 64)] +
                         [(38408, 1544, b) for b in (1, 3, 16, 32, 64)])
def test_several_tiles(layer_of, m, n, B):
    """CTAs that share no tile and take several in turn."""
    layer, w, s = layer_of(m, n)
    plan = layer.plan(B)
    assert plan["kernel"] == 0 and plan["cluster"] == 1 and plan["items"] > plan["clusters"], plan
    _check(layer, w, s, _x(B, n, torch.float16), torch.float32 if B & 1 else torch.float16)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m,n,B", [(4096, 264, 2048), (4104, 1160, 2049), (10120, 520, 700)])
def test_several_tiles_of_many_tokens(layer_of, m, n, B, out):
    layer, w, s = layer_of(m, n)
    plan = layer.plan(B)
    assert plan["kernel"] == 1 and plan["ksplit"] == 1 and plan["items"] > plan["clusters"], plan
    _check(layer, w, s, _x(B, n, torch.bfloat16), DT[out])


@pytest.mark.parametrize("m,n,B,out", [(6400, 16392, 66, "f16"), (5120, 12296, 257, "f32")])
def test_several_parts_of_many_tokens(layer_of, m, n, B, out):
    """K split over pairs that take several of the parts."""
    layer, w, s = layer_of(m, n)
    plan = layer.plan(B)
    assert plan["kernel"] == 1 and plan["ksplit"] > 1 and plan["items"] > plan["clusters"], plan
    _check(layer, w, s, _x(B, n, torch.float16), DT[out])


@pytest.fixture(scope="module")
def poison(glq):
    """Leaves NaN weights, tokens and scales wherever the kernels keep theirs."""
    bad = torch.full((2048, 2048), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    layer = glq.Fp8Linear(bad, torch.full((16, 16), float("nan")))
    x = torch.full((520, 2048), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer.reserve(520)

    def run():
        for B in (520, 64, 32, 16, 8, 1):
            assert torch.isnan(layer(x[:B])).all()

    return run


@pytest.mark.parametrize("m,n,B", LINEAR)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32")])
def test_nothing_is_left_of_other_calls(layer_of, poison, m, n, B, dt, out):
    """Sizes that leave rows, columns or tokens of a tile unused, after calls that were NaN everywhere."""
    layer, w, s = layer_of(m, n)
    poison()
    _check(layer, w, s, _x(B, n, DT[dt]), DT[out])


def test_rows_of_an_output_after_others(layer_of, poison, glq):
    layer, w, s = layer_of(264, 904)
    x = _x(17, 904, torch.float16)
    q, sc = glq.fp8_quantize(x)
    rows = torch.full((21, 264), 7.0, device="cuda", dtype=torch.float16)
    poison()
    layer.forward_quantized(q, sc, out=rows[2:19])
    want, bound = ref.linear(x, w, s, torch.float16)
    assert not ref.not_within(rows[2:19], want, bound).any()
    assert torch.all(rows[:2] == 7) and torch.all(rows[19:] == 7)
