"""The mixture-of-experts layer's weights from scores far from zero, against the
definition in 64 bits (tests/fp8_device_reference.py)."""
import pytest

import fp8_device_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def glq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import e8_lattice_codebook_b200 as glq
    return glq


def _experts(gen, E, d, inter):
    out = []
    for m, n in ((inter, d), (inter, d), (d, inter)):
        made = [ref.random_weight(gen, m, n) for _ in range(E)]
        out.append((torch.stack([w.view(torch.uint8) for w, _ in made]).view(torch.float8_e4m3fn),
                    torch.stack([s for _, s in made])))
    return out


def _layer(glq, experts, topk, **options):
    (gate, gs), (up, us), (down, ds) = experts
    return glq.Fp8Moe(gate, gs, up, us, down, ds, topk, **options)


def _check(y, x, logits, experts, topk, renormalize, scoring, scale):
    want, bound = ref.moe(x, logits, *experts, topk, renormalize, scoring, scale)
    bound = bound + ref.half_step(y.dtype) * want.abs() + ref.smallest(y.dtype)
    bad = ref.not_within(y, want, bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:5].tolist())


@pytest.mark.parametrize("T", [3, 12, 40])  # every way through the kernel: roundings in each CTA, shared, a larger tile
def test_renormalized_sigmoid_over_the_range(glq, T):
    """Scores below fp32's smallest number have a quotient; all at 1, and both mixed."""
    gen = torch.Generator("cuda").manual_seed(41)
    experts = _experts(gen, 10, 136, 136)
    layer = _layer(glq, experts, 4, renormalize=True, scoring=glq.GLQ_MOE_SIGMOID, routed_scale=2.5)
    x = torch.randn(T, 136, generator=gen, device="cuda").to(torch.bfloat16)
    noise = torch.randn(T, 10, generator=gen, device="cuda")
    for shift in (-1e6, -1000.0, -100.0, -95.0, -90.0, -87.5, -30.0, 0.0, 30.0, 100.0, 1e6):
        logits = noise + shift
        y = layer(x, logits, out_dtype=torch.float32)
        layer.check()
        _check(y, x, logits, experts, 4, True, 1, 2.5)
    logits = 60 * noise                       # from one that vanishes to 1
    logits[0] = torch.finfo(torch.float32).min
    logits[1] = -100.0                        # equal, and far below
    _check(layer(x, logits, out_dtype=torch.float32), x, logits, experts, 4, True, 1, 2.5)


def test_infinite_scores(glq):
    """An infinite logit: its sigmoid is 1, its softmax is none."""
    gen = torch.Generator("cuda").manual_seed(42)
    experts = _experts(gen, 6, 136, 136)
    x = torch.randn(5, 136, generator=gen, device="cuda").to(torch.float16)
    logits = torch.randn(5, 6, generator=gen, device="cuda")
    logits[1, 3] = float("inf")
    as_one = logits.clone()
    as_one[1, 3] = 1e4                        # sigmoid: exactly 1 in 64 bits
    for renormalize in (False, True):
        layer = _layer(glq, experts, 2, renormalize=renormalize, scoring=glq.GLQ_MOE_SIGMOID)
        y = layer(x, logits, out_dtype=torch.float32)
        _check(y, x, as_one, experts, 2, renormalize, 1, 1.0)
        y = _layer(glq, experts, 2, renormalize=renormalize)(x, logits, out_dtype=torch.float32)
        assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2, 3, 4]]).all()
