"""The mixture-of-experts layer where a CTA takes more blocks than it has stages:
every stage, accumulator and barrier is used again, over tiles of several rows
and experts.  Against the definition in 64 bits, on the device."""
import pytest

import fp8_device_reference as ref
from test_gpu_moe import SIZES

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

MOST_STAGES = 32  # a stage of 16 tokens takes 16 of 512 columns of tensor memory


@pytest.fixture(scope="module")
def glq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import e8_lattice_codebook_b200 as glq
    return glq


@pytest.fixture(scope="module")
def experts_of():
    last = {}

    def make(E, d, inter):
        if (E, d, inter) not in last:
            last.clear()
            gen = torch.Generator("cuda").manual_seed(E + d + inter)
            out = []
            for m, n in ((inter, d), (inter, d), (d, inter)):
                made = [ref.random_weight(gen, m, n) for _ in range(E)]
                out.append((torch.stack([w.view(torch.uint8) for w, _ in made]).view(torch.float8_e4m3fn),
                            torch.stack([s for _, s in made])))
            last[E, d, inter] = out
        return last[E, d, inter]

    yield make
    last.clear()


def _inputs(T, E, d, forced, dtype):
    """Tokens and logits; the first `forced` tokens choose expert 3 before all others."""
    gen = torch.Generator("cuda").manual_seed(100 * T + E)
    x = torch.randn(T, d, generator=gen, device="cuda")
    x[:, ::41] *= 10.0
    logits = torch.randn(T, E, generator=gen, device="cuda")
    if forced:
        logits[:forced, 3] = 9.0
    return x.to(dtype), logits


# T, E, k, d, inter, forced, fullest: between which two numbers of tokens the fullest expert has
CASES = [
    (1, 8, 8, 4000, 2008, 0, (1, 1)), (4, 8, 5, 4000, 2008, 0, (1, 4)),       # roundings in each CTA
    (5, 8, 4, 4000, 2008, 0, (1, 5)), (16, 8, 3, 4000, 2008, 0, (1, 16)),     # shared, 16 tokens
    (20, 8, 2, 4000, 2008, 0, (1, 16)), (20, 8, 2, 4000, 2008, 20, (17, 20)),  # the larger kernel: 16 and 32 tokens
    (64, 8, 2, 4000, 2008, 40, (33, 64)), (64, 8, 8, 4000, 2008, 0, (64, 64)),  # 64
    (64, 128, 8, 2048, 768, 0, (1, 16)), (64, 128, 8, 2048, 768, 30, (17, 32)),  # many experts of a few tokens
    (150, 8, 2, 4000, 2008, 0, (30, 80)),                                     # slices of 64
]


@pytest.mark.parametrize("T,E,k,d,inter,forced,fullest", CASES)
def test_more_blocks_than_stages(glq, experts_of, T, E, k, d, inter, forced, fullest):
    experts = experts_of(E, d, inter)
    x, logits = _inputs(T, E, d, forced, torch.float16 if T & 1 else torch.bfloat16)
    chosen = torch.bincount(torch.topk(logits, k).indices.flatten(), minlength=E)
    assert fullest[0] <= int(chosen.max()) <= fullest[1]
    blocks = lambda v: -(-v // 128)  # noqa: E731
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    first = int((chosen > 0).sum()) * 2 * blocks(inter) * blocks(d)
    assert first > MOST_STAGES * sms
    (gate, gs), (up, us), (down, ds) = experts
    layer = glq.Fp8Moe(gate, gs, up, us, down, ds, k, renormalize=k != 4)
    for out in (torch.float32, x.dtype):
        y = layer(x, logits, out_dtype=out)
        layer.check()
        want, bound = ref.moe(x, logits, *experts, k, k != 4, 0, 1.0)
        bad = ref.not_within(y, want, bound + ref.half_step(out) * want.abs() + ref.smallest(out))
        assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist())
        assert torch.equal(y, layer(x, logits, out_dtype=out))  # the same bits again


@pytest.mark.parametrize("T,E,k,d,inter", SIZES)
def test_nothing_is_left_of_other_calls(glq, experts_of, T, E, k, d, inter):
    """After calls that were NaN everywhere: unused rows of a tile, places of no token, sums of no expert."""
    experts = experts_of(E, d, inter)
    (gate, gs), (up, us), (down, ds) = experts
    layer = glq.Fp8Moe(gate, gs, up, us, down, ds, k)
    for n in (64, 16, 4):
        x, logits = _inputs(n, E, d, 0, torch.bfloat16)
        assert torch.isnan(layer(torch.full_like(x, float("nan")), logits)).all()
    x, logits = _inputs(T, E, d, 0, torch.bfloat16)
    y = layer(x, logits, out_dtype=torch.float32)
    layer.check()
    want, bound = ref.moe(x, logits, *experts, k, True, 0, 1.0)
    bad = ref.not_within(y, want, bound + ref.half_step(y.dtype) * want.abs() + ref.smallest(y.dtype))
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist())
