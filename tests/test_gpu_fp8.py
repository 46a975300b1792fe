"""The 8-bit float linear layer and its activation rounding against their
definition in 64 bits (tests/fp8_reference.py), through the public binding."""
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


def _x(gen, B, n, dtype):
    x = torch.randn(B, n, generator=gen, dtype=torch.float64)
    x[:, ::37] *= 20.0
    return x.to(dtype)


def _f64(t):
    return t.detach().cpu().double().numpy()


def _layer(glq, gen, m, n):
    w, s = ref.random_weight(gen, m, n)
    return glq.Fp8Linear(w.cuda(), s.cuda()), w, s


def _check(y, xd, w, s, dtype):
    xv, wv = ref.values(_f64(xd)), ref.weight_values(w, s)
    want = xv @ wv.T
    got = _f64(y)
    assert got.shape == want.shape
    bad = np.abs(got - want) > ref.linear_bound(xv, wv, want, dtype)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5], np.abs(got - want).max())


@pytest.mark.parametrize("B,n,dt", [(1, 8, "bf16"), (1, 5120, "bf16"), (3, 136, "f16"), (33, 960, "f32"), (31, 256, "bf16"),
                                    (257, 1000, "f16")])
def test_quantize_is_exact(glq, B, n, dt):
    gen = torch.Generator().manual_seed(B * 1000 + n)
    x = _x(gen, B, n, DT[dt])
    x[0, : min(n, 128)] = 0           # a group of zeros
    if B > 2:
        x[1] *= 1e-4                  # fp16: subnormals
        x[2, 1:8] = x[2, 0] * torch.tensor([1, 3, 5, 7, 9, 11, 13]).to(x.dtype) / 64  # near ties
    q, s = glq.fp8_quantize(x.cuda())
    wq, ws = ref.quantize(_f64(x))
    np.testing.assert_array_equal(_f64(s), ws)
    np.testing.assert_array_equal(_f64(q.float()), wq)


def test_quantize_extremes(glq):
    x = torch.zeros(6, 256, dtype=torch.float32)
    x[0, :] = 1e-38
    x[1, :] = 3e38
    x[2, 5] = float("nan")
    x[3, 7], x[3, 8] = float("inf"), 1.0
    x[4, 200] = -float("inf")
    x[5, 0] = -448.0
    q, s = glq.fp8_quantize(x.cuda())
    q, s = q.float().cpu(), s.cpu()
    # 1e-38 * 448 * 2^110 = 0.005815; e4m3's subnormals are 2^-9 apart there: 2.98 steps, so 3
    assert s[0, 0] == np.float32(2.0 ** -110 / 448) and torch.all(q[0] == 3 * 2.0 ** -9)
    assert torch.isfinite(s[:, 1]).all() and torch.all(q[1] == 448)
    assert torch.isnan(q[2, :128]).all() and torch.isnan(s[0, 2]) and torch.all(q[2, 128:] == 0)
    assert torch.isnan(q[3, 7]) and q[3, 8] == 0 and torch.isinf(s[0, 3])
    assert torch.isnan(q[4, 200]) and torch.isinf(s[1, 4]) and torch.all(q[4, :128] == 0)
    assert q[5, 0] == -448 and s[0, 5] == 1


LINEAR = [  # m, n, B: one block, ends inside a block, fewer blocks than SMs, many tiles; each token tile
    (8, 8, 1), (128, 128, 16), (136, 264, 5), (960, 960, 1), (2560, 960, 2), (8, 4096, 7), (4096, 1024, 16),
    (264, 1160, 17), (1024, 512, 32), (200, 392, 33), (1032, 648, 64), (392, 520, 65), (640, 2048, 100), (256, 256, 128),
    (520, 136, 129), (384, 1032, 300), (1536, 1024, 512), (776, 776, 1000),
    # K split over pairs: 2 to 8 parts, ends inside a block, an odd number of row blocks
    (128, 4096, 66), (392, 3080, 200), (1032, 2056, 257),
]


@pytest.mark.parametrize("m,n,B", LINEAR)
@pytest.mark.parametrize("dt,out", [("bf16", "bf16"), ("f16", "f32")])
def test_linear(glq, m, n, B, dt, out):
    gen = torch.Generator().manual_seed(m + 3 * n + 7 * B)
    layer, w, s = _layer(glq, gen, m, n)
    x = _x(gen, B, n, DT[dt])
    y = layer(x.cuda(), out_dtype=DT[out])
    layer.check()
    _check(y, x, w, s, DT[out])


def test_linear_f16_and_batches_in_turn(glq):
    """One layer, every token tile in turn and back: nothing of one call is left for the next."""
    gen = torch.Generator().manual_seed(5)
    layer, w, s = _layer(glq, gen, 1160, 1160)
    for B in (1, 300, 16, 64, 2, 130, 40, 1):
        x = _x(gen, B, 1160, torch.float16)
        y = layer(x.cuda())
        _check(y, x, w, s, torch.float16)
        assert torch.equal(y, layer(x.cuda()))  # the same bits again
    layer.check()


def test_long_batch_in_slices(glq):
    gen = torch.Generator().manual_seed(6)
    layer, w, s = _layer(glq, gen, 72, 136)
    x = _x(gen, 8192 + 77, 136, torch.bfloat16)
    y = layer(x.cuda())
    _check(y, x, w, s, torch.bfloat16)
    q, sc = glq.fp8_quantize(x.cuda())
    assert torch.equal(layer.forward_quantized(q, sc), y)
    layer.check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("m,n", [(392, 1160), (16384, 6400)])
def test_rounding_inside_and_in_front(glq, m, n, dt):
    """Few tokens, rounded by the product (the smaller layer: up to 8, the larger: up to 4) or before it: the same bits."""
    gen = torch.Generator().manual_seed(9)
    layer, _, _ = _layer(glq, gen, m, n)
    for B in range(1, 11):
        x = _x(gen, B, n, DT[dt])
        if B > 2:
            x[B - 1, 5], x[1, n - 1] = float("nan"), float("inf")
        y = layer(x.cuda())
        want = layer.forward_quantized(*glq.fp8_quantize(x.cuda()), out_dtype=DT[dt])
        assert torch.equal(torch.nan_to_num(y, nan=7.0), torch.nan_to_num(want, nan=7.0))
        assert torch.equal(torch.isnan(y), torch.isnan(want))
    layer.check()


@pytest.mark.parametrize("B", [1, 16, 17, 100, 400])
def test_quantized_input_gives_the_same(glq, B):
    gen = torch.Generator().manual_seed(B)
    layer, w, s = _layer(glq, gen, 520, 904)
    x = _x(gen, B, 904, torch.bfloat16).cuda()
    q, sc = glq.fp8_quantize(x)
    for dt in ("bf16", "f32"):
        assert torch.equal(layer.forward_quantized(q, sc, out_dtype=DT[dt]), layer(x, out_dtype=DT[dt]))
    y = layer.forward_quantized(q, sc, out_dtype=torch.float16)
    _check(y, x, w, s, torch.float16)


def test_dequant_and_strided_weights(glq):
    gen = torch.Generator().manual_seed(9)
    w, s = ref.random_weight(gen, 264, 392)
    wide = torch.zeros(264, 400, dtype=torch.uint8)
    wide[:, :392] = w.view(torch.uint8)
    strided = wide.cuda().view(torch.float8_e4m3fn)[:, :392]
    for given in (w, w.cuda(), strided, w.t().contiguous().t()):  # CPU, packed, row stride, columns first
        layer = glq.Fp8Linear(given, s)
        np.testing.assert_array_equal(_f64(layer.dequant()), ref.weight_values(w, s).astype(np.float32))
    assert glq.glq_fp8_info(layer.handle)[:2] == (264, 392)


@pytest.mark.parametrize("B", [3, 40, 200])
def test_nan_and_inf_stay_in_their_token(glq, B):
    gen = torch.Generator().manual_seed(12)
    layer, w, s = _layer(glq, gen, 264, 520)
    x = _x(gen, B, 520, torch.bfloat16)
    clean = layer(x.cuda())
    x[0, 3] = float("nan")
    x[2, 300] = float("inf")
    y = layer(x.cuda())
    keep = [b for b in range(B) if b not in (0, 2)]
    assert torch.isnan(y[0]).all() and torch.isnan(y[2]).all()
    assert torch.equal(y[keep], clean[keep])
    assert torch.equal(layer(x[keep].cuda())[0], clean[1])  # and nothing of it is left in shared memory


def test_streams_and_graphs(glq):
    gen = torch.Generator().manual_seed(21)
    layer, w, s = _layer(glq, gen, 1032, 1544)
    other, w2, s2 = _layer(glq, gen, 264, 1032)
    xs = [_x(gen, B, 1544, torch.bfloat16).cuda() for B in (1, 70, 600)]
    want = [other(layer(x)) for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = [other(layer(x, stream=side), stream=side) for x in xs]
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    layer.reserve(600)
    other.reserve(600)
    held = glq.glq_workspace_info(torch.cuda.current_device())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [other(layer(x)) for x in xs]
    for k in range(3):
        for x in xs:
            x.copy_(torch.randn_like(x))
        want = [other(layer(x)) for x in xs]
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), k
    assert glq.glq_workspace_info(torch.cuda.current_device()) == held
    layer.check()


def test_capture_needs_a_reservation(glq):
    gen = torch.Generator().manual_seed(22)
    layer, _, _ = _layer(glq, gen, 264, 264)
    x = torch.randn(40, 264, device="cuda").half()
    y = torch.empty(40, 264, device="cuda", dtype=torch.float16)
    layer(x[:1])  # the launch paths are warm
    glq.glq_workspace_release(torch.cuda.current_device())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(glq.GlqError) as e:
            layer(x, out=y)
        y.zero_()
    assert e.value.status == 11
    graph.replay()
    assert torch.count_nonzero(y) == 0


def test_empty_batch_and_out(glq):
    gen = torch.Generator().manual_seed(23)
    layer, w, s = _layer(glq, gen, 264, 264)
    assert layer(torch.empty(0, 264, device="cuda", dtype=torch.bfloat16)).shape == (0, 264)
    q, sc = glq.fp8_quantize(torch.empty(0, 264, device="cuda"))
    assert q.shape == (0, 384) and sc.shape == (3, 0)
    assert layer.forward_quantized(q, sc).shape == (0, 264)
    x = _x(gen, 5, 264, torch.float16)
    rows = torch.full((9, 264), 7.0, device="cuda", dtype=torch.float16)
    layer(x.cuda(), out=rows[2:7])
    _check(rows[2:7], x, w, s, torch.float16)
    assert torch.all(rows[:2] == 7) and torch.all(rows[7:] == 7)  # the rows around are left


def test_refusals(glq):
    gen = torch.Generator().manual_seed(24)
    layer, w, s = _layer(glq, gen, 264, 264)
    x = torch.zeros(4, 264, device="cuda", dtype=torch.bfloat16)
    for bad in (x.cpu(), x[:, :256], x.t(), x.float()[:, ::2], x[0]):
        with pytest.raises(ValueError):
            layer(bad)
    with pytest.raises(glq.GlqError) as e:
        layer(x.float())
    assert e.value.status == 3
    with pytest.raises(glq.GlqError) as e:
        layer(x, out_dtype=torch.float16)
    assert e.value.status == 3
    with pytest.raises(ValueError):
        layer(x, out=torch.empty(4, 256, device="cuda", dtype=torch.bfloat16))
    q, sc = glq.fp8_quantize(x)
    for bad in ((q[:, :264], sc), (q, sc[:, :2]), (q, sc.double()), (q.view(torch.uint8), sc), (q, sc.cpu())):
        with pytest.raises(ValueError):
            layer.forward_quantized(*bad)
    for bad in ((w.float(), s), (w, s[:1]), (w[:260], s), (w[:, :260], s)):
        with pytest.raises((ValueError, glq.GlqError)):
            glq.Fp8Linear(*bad)
    with pytest.raises(glq.GlqError) as e:
        glq.fp8_quantize(torch.zeros(2, 12, device="cuda"))
    assert e.value.status == 2


def test_wait_runs_out_and_reports(glq):
    gen = torch.Generator().manual_seed(25)
    layer, w, s = _layer(glq, gen, 136, 264)
    layer.selftest_wait(1, 2_000_000)  # an arrival that never comes: about 1 ms
    with pytest.raises(glq.GlqError) as e:
        layer.check()
    assert e.value.status == 9
    layer.check()  # cleared
    layer.selftest_wait(2, 2_000_000)
    layer.check()
    x = _x(gen, 3, 264, torch.bfloat16)
    _check(layer(x.cuda()), x, w, s, torch.bfloat16)  # the context is whole
    for bad in ((0, 10), (3, 10), (1, 0)):
        with pytest.raises(glq.GlqError) as e:
            layer.selftest_wait(*bad)
        assert e.value.status == 1


def test_no_layer_while_capturing(glq):
    gen = torch.Generator().manual_seed(26)
    w, s = (t.cuda() for t in ref.random_weight(gen, 136, 136))
    y = torch.zeros(8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(glq.GlqError) as e:
            glq.Fp8Linear(w, s)
        y.add_(1)
    assert e.value.status == 11
    graph.replay()
    assert torch.all(y == 1)  # the capture was not disturbed
