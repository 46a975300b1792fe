"""The mixture-of-experts layer against its definition in 64 bits
(tests/fp8_reference.py), through the public binding."""
import numpy as np
import pytest

import fp8_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def glq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import e8_lattice_codebook_b200 as glq
    return glq


def _f64(t):
    return t.detach().cpu().double().numpy()


class Experts:
    def __init__(self, gen, E, d, inter):
        make = lambda m, n: [ref.random_weight(gen, m, n) for _ in range(E)]  # noqa: E731
        self.raw = [make(inter, d), make(inter, d), make(d, inter)]
        self.values = [[ref.weight_values(w, s) for w, s in m] for m in self.raw]
        self.E, self.d, self.inter = E, d, inter

    def layer(self, glq, topk, **options):
        args = []
        for m in self.raw:
            args += [torch.stack([w.view(torch.uint8) for w, _ in m]).view(torch.float8_e4m3fn).cuda(),
                     torch.stack([s for _, s in m]).cuda()]
        return glq.Fp8Moe(*args, topk=topk, **options)

    def check(self, y, x, logits, topk, renormalize=True, scoring=0, routed_scale=1.0):
        want, bound = ref.moe(_f64(x), _f64(logits), *self.values, topk, renormalize, scoring, routed_scale)
        bound += ref.half_step(y.dtype) * np.abs(want) + ref.smallest(y.dtype)
        got = _f64(y)
        bad = ~(np.abs(got - want) <= bound)
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], np.abs(got - want).max(), np.abs(want).max())


def _inputs(gen, T, E, d, dtype):
    x = torch.randn(T, d, generator=gen, dtype=torch.float64)
    x[:, ::41] *= 10.0
    return x.to(dtype), torch.randn(T, E, generator=gen, dtype=torch.float32)


SIZES = [  # T, E, k, d, inter: one block; widths that end inside a block; every token tile; all experts; many per lane
    (1, 1, 1, 8, 8), (1, 8, 2, 256, 128), (3, 5, 5, 136, 264), (7, 64, 6, 320, 200), (16, 8, 3, 512, 384), (17, 12, 4, 264, 136),
    (32, 6, 2, 128, 520), (33, 9, 4, 392, 264), (64, 4, 2, 256, 256), (64, 130, 8, 136, 72), (5, 300, 16, 72, 40), (1, 512, 16, 64, 16),
    # the largest tables in shared memory, for each token tile
    (64, 512, 16, 16, 8), (32, 512, 16, 8, 16), (16, 512, 16, 16, 16), (4, 9, 9, 264, 136),
]


@pytest.mark.parametrize("T,E,k,d,inter", SIZES)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32")])
def test_layer(glq, T, E, k, d, inter, dt, out):
    gen = torch.Generator().manual_seed(T + 5 * E + 7 * d)
    ex = Experts(gen, E, d, inter)
    layer = ex.layer(glq, k)
    x, logits = _inputs(gen, T, E, d, DT[dt])
    y = layer(x.cuda(), logits.cuda(), out_dtype=DT[out])
    layer.check()
    ex.check(y, x, logits, k)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("scoring", [0, 1])
@pytest.mark.parametrize("ldt", ["f32", "bf16"])
def test_scores(glq, renormalize, scoring, ldt):
    gen = torch.Generator().manual_seed(31)
    ex = Experts(gen, 10, 136, 136)
    layer = ex.layer(glq, 4, renormalize=renormalize, scoring=scoring, routed_scale=2.5)
    x, logits = _inputs(gen, 9, 10, 136, torch.bfloat16)
    logits = (3 * logits).to(DT[ldt])
    ex.check(layer(x.cuda(), logits.cuda()), x, logits, 4, renormalize, scoring, 2.5)


def test_ties_masks_and_empty_tokens(glq):
    gen = torch.Generator().manual_seed(32)
    ex = Experts(gen, 40, 136, 136)
    layer = ex.layer(glq, 3)
    x, logits = _inputs(gen, 8, 40, 136, torch.float16)
    low, high = torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    logits[0] = 0.25                     # all equal: 0, 1, 2
    logits[1, 5:] = 0.0
    logits[1, 9] = -0.0                  # -0 and 0 are equal
    logits[1, :5] = -1.0
    logits[2] = -float("inf")            # no expert: y = 0
    logits[3, 1:] = -float("inf")        # fewer than topk
    logits[4] = low                      # the type's lowest value is still a choice
    logits[5, 3:] = float("nan")         # NaN is none
    logits[6, 7] = 80.0                  # all others vanish
    logits[7] = -high
    logits[7, 33] = high
    clean = torch.nan_to_num(logits, nan=-float("inf"), posinf=high, neginf=-float("inf"))
    y = layer(x.cuda(), logits.cuda())
    layer.check()
    assert torch.count_nonzero(y[2]) == 0
    ex.check(y, x, clean, 3)
    none = torch.full_like(logits, -float("inf"))
    out = torch.full((8, 136), 7.0, dtype=torch.float16, device="cuda")
    layer(x.cuda(), none.cuda(), out=out)
    assert torch.count_nonzero(out) == 0
    ex.check(layer(x.cuda(), clean.cuda()), x, clean, 3)  # and the next call is whole again


def test_nan_stays_in_its_token(glq):
    gen = torch.Generator().manual_seed(33)
    ex = Experts(gen, 6, 264, 136)
    layer = ex.layer(glq, 2)
    x, logits = _inputs(gen, 20, 6, 264, torch.bfloat16)
    clean = layer(x.cuda(), logits.cuda())
    x[4, 100], x[11, 3] = float("nan"), float("inf")
    logits[15, 2] = float("inf")
    y = layer(x.cuda(), logits.cuda())
    bad = [4, 11, 15]
    keep = [t for t in range(20) if t not in bad]
    assert torch.isnan(y[bad]).all()
    assert torch.isfinite(y[keep]).all()
    # token 15 may use an expert it did not use before, which moves the shares of the CTAs
    ex.check(y[keep], x[keep], logits[keep], 2)
    ex.check(clean[keep], x[keep], logits[keep], 2)


def test_more_than_one_slice_and_calls_in_turn(glq):
    gen = torch.Generator().manual_seed(34)
    ex = Experts(gen, 8, 136, 264)
    layer = ex.layer(glq, 2)
    for T in (1, 150, 64, 16, 70, 2):
        x, logits = _inputs(gen, T, 8, 136, torch.bfloat16)
        y = layer(x.cuda(), logits.cuda())
        ex.check(y, x, logits, 2)
        assert torch.equal(y, layer(x.cuda(), logits.cuda()))  # the same bits again
    layer.check()


def test_one_expert_for_all(glq):
    gen = torch.Generator().manual_seed(35)
    ex = Experts(gen, 4, 264, 392)
    layer = ex.layer(glq, 1)
    x, logits = _inputs(gen, 64, 4, 264, torch.bfloat16)
    logits[:, 2] += 100
    ex.check(layer(x.cuda(), logits.cuda()), x, logits, 1)


@pytest.mark.parametrize("fullest", [15, 16, 17, 32, 33, 63])
def test_fullest_expert(glq, fullest):
    """One expert with a given number of the 64 tokens beside many with a few: every token tile, full and one over."""
    gen = torch.Generator().manual_seed(38)
    ex = Experts(gen, 48, 264, 136)
    layer = ex.layer(glq, 2)
    x, logits = _inputs(gen, 64, 48, 264, torch.bfloat16)
    logits[:, 7] = -float("inf")
    logits[torch.randperm(64, generator=gen)[:fullest], 7] = 9.0
    chosen = torch.bincount(torch.topk(logits, 2).indices.flatten(), minlength=48)
    assert chosen[7] == fullest and chosen.sort().values[-2] < 15
    ex.check(layer(x.cuda(), logits.cuda()), x, logits, 2)
    layer.check()


def test_streams_graphs_and_reservation(glq):
    gen = torch.Generator().manual_seed(36)
    ex = Experts(gen, 16, 264, 136)
    layer, other = ex.layer(glq, 4), ex.layer(glq, 2, renormalize=False)
    w, s = ref.random_weight(gen, 264, 264)
    linear = glq.Fp8Linear(w.cuda(), s.cuda())
    x, logits = (t.cuda() for t in _inputs(gen, 24, 16, 264, torch.bfloat16))

    def block():  # a layer's products together, as a model runs them
        h = linear(x)
        return h, other(layer(h, logits), logits)

    want = block()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = layer(linear(x, stream=side), logits, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, layer(want[0], logits))
    glq.glq_workspace_release(torch.cuda.current_device())
    y = torch.zeros(24, 264, device="cuda", dtype=torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(glq.GlqError) as e:
            layer(x, logits, out=y)
        y.add_(1)
    assert e.value.status == 11
    for m in (layer, other, linear):
        m.reserve(24)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block()
    for _ in range(3):
        x.copy_(torch.randn_like(x))
        logits.copy_(torch.randn_like(logits))
        want = block()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    layer.check()
    other.check()


def test_refusals(glq):
    gen = torch.Generator().manual_seed(37)
    ex = Experts(gen, 4, 136, 72)
    layer = ex.layer(glq, 2)
    x, logits = (t.cuda() for t in _inputs(gen, 3, 4, 136, torch.bfloat16))
    assert layer(x[:0], logits[:0]).shape == (0, 136)
    for a, b in ((x[:, :128], logits), (x.cpu(), logits), (x, logits[:2]), (x, logits[:, :3]), (x, logits.cpu()), (x.t(), logits)):
        with pytest.raises(ValueError):
            layer(a, b)
    for a, b, kw in ((x.float(), logits, {}), (x, logits.half(), {}), (x, logits, {"out_dtype": torch.float16})):
        with pytest.raises(glq.GlqError) as e:
            layer(a, b, **kw)
        assert e.value.status == 3
    for k in (0, 5, 17):
        with pytest.raises(glq.GlqError) as e:
            ex.layer(glq, k)
        assert e.value.status == 2
    for kw in ({"scoring": 2}, {"routed_scale": float("nan")}):
        with pytest.raises(glq.GlqError) as e:
            ex.layer(glq, 2, **kw)
        assert e.value.status == 1
    config, _ = glq.glq_moe_info(layer.handle)
    assert (config["experts"], config["d"], config["inter"], config["topk"]) == (4, 136, 72, 2)
