"""Where the binding allocates a call's result when it is given a stream: on
that stream, whose kernel writes it, with the current stream recorded as a
reader.  With fakes of torch's allocator and streams, without a GPU."""
import contextlib
import types

import pytest
import torch

import e8_lattice_codebook_b200 as glq
from e8_lattice_codebook_b200 import shard


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


class World:
    """The current stream, and tensors that know where they were allocated."""

    def __init__(self):
        self.main, self.side = Stream(1), Stream(2)
        self.now = self.main
        self.launches = []
        world = self

        class Tensor:
            is_cuda, device = True, torch.device("cuda", 0)

            def __init__(self, shape, dtype, on):
                self.shape, self.dtype, self.on, self.recorded = tuple(shape), dtype, on, []

            dim = lambda t: len(t.shape)  # noqa: E731
            size = lambda t, i: t.shape[i]  # noqa: E731
            is_contiguous = lambda t: True  # noqa: E731
            get_device = lambda t: 0  # noqa: E731
            data_ptr = lambda t: 1 << 20  # noqa: E731
            record_stream = lambda t, s: t.recorded.append(s)  # noqa: E731

            def new_empty(t, shape, dtype=None):
                return Tensor(shape, dtype or t.dtype, world.now)

            def numel(t):
                return t.shape[0] * t.shape[1]

            def __getitem__(t, at):
                return t

        @contextlib.contextmanager
        def stream(s):
            before, world.now = world.now, s
            yield
            world.now = before

        self.Tensor = Tensor
        cuda = types.SimpleNamespace(Stream=Stream, ExternalStream=lambda raw, device: {1: self.main, 2: self.side}[raw],
                                     current_device=lambda: 0, current_stream=lambda d=None: world.now, stream=stream,
                                     device=lambda i: contextlib.nullcontext())
        self.torch = types.SimpleNamespace(
            cuda=cuda, float16=torch.float16, bfloat16=torch.bfloat16, device=torch.device, float32=torch.float32, float8_e4m3fn=torch.float8_e4m3fn,
            empty=lambda shape, dtype, device: Tensor(shape, dtype, world.now), _C=types.SimpleNamespace(_cuda_getDevice=lambda: 0))

    def layer(self, cls, **fields):
        layer = cls.__new__(cls)
        layer.__dict__.update(handle=0, _index=0, device=torch.device("cuda", 0), **fields)
        return layer


@pytest.fixture
def world(monkeypatch):
    w = World()
    monkeypatch.setattr(glq, "_torch", lambda: w.torch)
    monkeypatch.setattr(shard, "_torch", lambda: w.torch, raising=False)
    monkeypatch.setattr(glq, "_raw_stream", lambda i: w.now.cuda_stream)
    monkeypatch.setattr(glq, "_E4M3_F32", None)
    monkeypatch.setattr(glq, "_DTYPE_CODES", {})
    for name in ("glq_linear", "glq_dequant_reference", "glq_rht_input", "glq_rht_input_operand", "glq_rht_output"):
        monkeypatch.setattr(glq, name, lambda *a: w.launches.append(a[-1]))
    monkeypatch.setattr(shard, "glq_linear", lambda *a: w.launches.append(a[-1]))
    for name in ("glq_fp8_quantize", "glq_fp8_linear", "glq_fp8_linear_quantized", "glq_fp8_dequant", "glq_moe_forward"):
        monkeypatch.setattr(glq, name, lambda *a: w.launches.append(a[-1]))
    return w


def _fp8_calls(w):
    bf16, x = torch.bfloat16, w.Tensor((5, 264), torch.bfloat16, w.main)
    linear = w.layer(glq.Fp8Linear, m=136, n=264)
    moe = w.layer(glq.Fp8Moe, d=264, inter=136, experts=4, topk=2)
    q, s = w.Tensor((5, 384), torch.float8_e4m3fn, w.main), w.Tensor((3, 5), torch.float32, w.main)
    logits = w.Tensor((5, 4), torch.float32, w.main)
    return {
        "quantize": (lambda st: glq.fp8_quantize(x, stream=st), [x], [torch.float8_e4m3fn, torch.float32]),
        "linear": (lambda st: linear(x, stream=st), [x], [bf16]),
        "linear, f32": (lambda st: linear(x, out_dtype=torch.float32, stream=st), [x], [torch.float32]),
        "quantized": (lambda st: linear.forward_quantized(q, s, stream=st), [q, s], [bf16]),
        "dequant": (lambda st: linear.dequant(stream=st), [], [torch.float32]),
        "moe": (lambda st: moe(x, logits, stream=st), [x, logits], [bf16]),
    }


CALLS = ["quantize", "linear", "linear, f32", "quantized", "dequant", "moe"]


def _check(w, calls, name):
    run, inputs, dtypes = calls[name]
    bare = types.SimpleNamespace(cuda_stream=2)  # another library's
    for given, other in ((w.side, True), (bare, True), (w.main, False), (None, False)):
        for t in inputs:
            t.recorded.clear()
        w.launches.clear()
        outs = run(given)
        outs = outs if isinstance(outs, tuple) else (outs,)
        assert [o.dtype for o in outs] == dtypes
        assert w.launches == [(given or w.main).cuda_stream]
        for o in outs:
            assert o.on is (w.side if other else w.main), name
            assert (w.main in o.recorded) == other
        for t in inputs:
            assert (w.side in t.recorded) == other


@pytest.mark.parametrize("name", CALLS)
def test_fp8_results(world, name):
    _check(world, _fp8_calls(world), name)


def _lattice_calls(w):
    bf16, f32, x = torch.bfloat16, torch.float32, w.Tensor((5, 264), torch.bfloat16, w.main)
    layer = w.layer(glq.GlqLinear, m=136, n=264)
    part = w.layer(shard.RowParallelLinear, m=136, n=264)
    return {
        "lattice": (lambda st: layer(x, stream=st), [x], [bf16]),
        "lattice dequant": (lambda st: layer.dequant(stream=st), [], [f32]),
        "rht in": (lambda st: layer.rht_input(x, stream=st), [x], [f32]),
        "rht operand": (lambda st: layer.rht_input_operand(x, stream=st), [x], [torch.float16, f32]),
        "rht out": (lambda st: layer.rht_output(x, stream=st), [x], [f32]),
        "part": (lambda st: part.partial(x, stream=st), [x], [f32]),
    }


@pytest.mark.parametrize("name", ["lattice", "lattice dequant", "rht in", "rht operand", "rht out", "part"])
def test_lattice_results(world, name):
    _check(world, _lattice_calls(world), name)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_collective_is_on_the_given_stream(world, monkeypatch, dtype):
    """A shard's sum over the ranks follows the part on its stream, and the rounding follows the sum."""
    monkeypatch.setattr(torch.distributed, "all_reduce", lambda t, **k: world.launches.append(world.now.cuda_stream))
    monkeypatch.setattr(shard, "glq_cast", lambda *a: world.launches.append(a[-1]))
    x = world.Tensor((5, 264), torch.bfloat16, world.main)
    layer = world.layer(shard.RowParallelLinear, m=136, n=264, rank=0, world=2, group=None)
    steps = 2 + (dtype != torch.float32)
    for given in (world.side, world.main, None):
        world.launches.clear()
        y = layer(x, out_dtype=dtype, stream=given)
        assert world.launches == [(given or world.main).cuda_stream] * steps
        assert y.on is (given or world.main) and y.dtype == dtype
        assert (world.main in y.recorded) == (given is world.side) == (world.side in x.recorded)
        x.recorded.clear()
        assert world.now is world.main
