"""The bounded wait between the CTAs of the mixture-of-experts kernel, on the GPU,
without a fault: one CTA of the grid never arrives, the others give up after a
short limit, and the layer works again once check() has told of it."""
import time

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


@pytest.mark.parametrize("on_side", [False, True])
def test_wait_runs_out_and_the_layer_recovers(glq, on_side):
    gen = torch.Generator("cuda").manual_seed(71)
    experts = []
    for m, n in ((136, 264), (136, 264), (264, 136)):
        made = [ref.random_weight(gen, m, n) for _ in range(6)]
        experts += [torch.stack([w.view(torch.uint8) for w, _ in made]).view(torch.float8_e4m3fn),
                    torch.stack([s for _, s in made])]
    layer = glq.Fp8Moe(*experts, topk=2)
    x = {T: torch.randn(T, 264, generator=gen, device="cuda").to(torch.bfloat16) for T in (2, 9)}  # two and four barriers
    logits = {T: torch.randn(T, 6, generator=gen, device="cuda") for T in x}
    want = {T: layer(x[T], logits[T]) for T in x}
    layer.check()
    torch.cuda.synchronize()
    side = torch.cuda.Stream() if on_side else None
    for _ in range(2):
        layer.selftest_wait(2, 2_000_000, stream=side)  # every CTA arrives
        layer.check(stream=side)
        t0 = time.time()
        layer.selftest_wait(1, 2_000_000, stream=side)  # about 1 ms
        with pytest.raises(glq.GlqError) as e:
            layer.check(stream=side)
        assert e.value.status == 9 and time.time() - t0 < 2.0
        layer.check(stream=side)  # cleared
        for T in x:
            y = layer(x[T], logits[T], stream=side)
            layer.check(stream=side)
            assert torch.equal(y, want[T])
    for bad in ((0, 10), (3, 10), (1, 0)):
        with pytest.raises(glq.GlqError) as e:
            layer.selftest_wait(*bad)
        assert e.value.status == 1
