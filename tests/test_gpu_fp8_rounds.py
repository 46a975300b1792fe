"""The 8-bit float linear layer where a CTA takes tile after tile: stages,
accumulators and the buffers between CTAs are used again.  Against the
definition in 64 bits (tests/fp8_device_reference.py), on the device."""
import pytest

import fp8_device_reference as ref

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
