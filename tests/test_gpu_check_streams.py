"""Reading and clearing a layer's error word happens on the stream that check()
is given, and is over when it returns."""
import pytest

import fp8_device_reference as ref
import glq_inputs as gi
from gpu_helpers import Device

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
