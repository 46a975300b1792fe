"""Reading and clearing a layer's error word happens on the stream that check()
is given, and is over when it returns; so is the making of a layer."""
import numpy as np
import pytest

import fp8_device_reference as ref
import glq_inputs as gi
from gpu_helpers import Device, to_torch_x, tolerance
from oracle import glq_oracle as orc

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def glq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import e8_lattice_codebook_b200 as glq
    return glq


def _layers(glq):
    w, s = ref.random_weight(torch.Generator("cuda").manual_seed(51), 136, 264)
    fp8 = glq.Fp8Linear(w, s)
    lattice = Device().layer(gi.make_layer(51, 0, 64, 256, 2))
    return [(fp8, lambda n, st: fp8.selftest_wait(n, 200_000, stream=st)),
            (lattice, lambda n, st: lattice.selftest_wait(0, n, 200_000, stream=st))]


def test_check_uses_its_stream_alone(glq):
    side = torch.cuda.Stream()
    for layer, wait in _layers(glq):
        wait(1, side)  # the first use of a kernel loads it, which waits for the device
        with pytest.raises(glq.GlqError):
            layer.check(stream=side)
        torch.cuda.synchronize()
        torch.cuda._sleep(1_000_000_000)  # about half a second on the default stream
        busy = torch.cuda.Event()
        busy.record()
        outcomes = []
        for arrivals in (1, 2, 1, 2):  # runs out, completes, and again
            wait(arrivals, side)
            try:
                layer.check(stream=side)
                outcomes.append(0)
            except glq.GlqError as e:
                outcomes.append(e.status)
        still_busy = not busy.query()
        torch.cuda.synchronize()
        assert outcomes == [9, 0, 9, 0]
        assert still_busy  # nothing of a check waited for, or was put behind, the default stream's work
        layer.check()


def test_layer_is_made_when_the_call_returns(glq):
    """A call on a stream that waits for no other, straight after the layer was made."""
    L = gi.make_layer(52, 0, 1024, 1024, 3)
    xb = gi.make_x(52, 0, 4, L.n, "bf16")
    x, y = to_torch_x(xb, "bf16"), torch.empty(4, L.m, device="cuda")
    ref_y = orc.linear(L.m, L.n, L.bpw, L.idx1, L.idx2, L.weight_scale, L.resid_scale, L.s_in, L.s_out, xb, True,
                       cb2=L.cb2_f16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        layer = Device().layer(L)
        layer(x, out=y, stream=side)
        layer.check(stream=side)
        assert np.max(np.abs(y.cpu().numpy().astype(np.float64) - ref_y)) <= tolerance(ref_y)
