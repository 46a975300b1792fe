"""Host-side checks of the 8-bit float operators that need no GPU: refusals
that precede any CUDA call, and the 64-bit definition the GPU tests use
against torch's own e4m3 rounding."""
import ctypes

import numpy as np
import pytest
import torch

import fp8_reference as ref
from e8_lattice_codebook_b200 import build as glq_build


@pytest.fixture(scope="module")
def lib():
    glq_build.build()
    import e8_lattice_codebook_b200 as glq
    return glq._L()


P = 1 << 20  # an aligned address that no refused call reads


@pytest.mark.parametrize("args,status", [
    ((P, 0, -1, 128, P, P, None), 2), ((P, 0, 1, 0, P, P, None), 2), ((P, 0, 1, 12, P, P, None), 2),
    ((P, 0, 1, (1 << 20) + 8, P, P, None), 2), ((P, 0, 65535 * 32 + 1, 128, P, P, None), 2), ((P, 3, 1, 128, P, P, None), 3),
    ((None, 0, 1, 128, P, P, None), 1), ((P, 0, 1, 128, None, P, None), 1), ((P, 0, 1, 128, P, None, None), 1),
    ((P + 2, 0, 1, 128, P, P, None), 1), ((P, 0, 1, 128, P + 8, P, None), 1), ((P, 0, 0, 128, None, None, None), 0),
])
def test_quantize_refusals(lib, args, status):
    assert lib.glq_fp8_quantize(*args) == status


@pytest.mark.parametrize("m,n,w,ldw,s,status", [
    (0, 8, P, 8, P, 2), (8, 0, P, 8, P, 2), (12, 8, P, 8, P, 2), (8, 12, P, 16, P, 2), (8, 16, P, 8, P, 2),
    (8, 16, P, 20, P, 2), ((1 << 20) + 8, 8, P, 8, P, 2), (8, 8, None, 8, P, 1), (8, 8, P, 8, None, 1), (8, 8, P + 4, 8, P, 1),
])
def test_create_refusals(lib, m, n, w, ldw, s, status):
    h = ctypes.c_void_p(5)
    assert lib.glq_fp8_create(m, n, w, ldw, s, None, ctypes.byref(h)) == status
    assert not h.value
    assert lib.glq_fp8_create(m, n, w, ldw, s, None, None) == 1


def test_null_handles(lib):
    assert lib.glq_fp8_linear(None, P, 0, P, 0, 1, None) == 1
    assert lib.glq_fp8_linear_quantized(None, P, P, P, 0, 1, None) == 1
    assert lib.glq_fp8_dequant(None, P, None) == 1
    assert lib.glq_fp8_reserve(None, 1) == 1
    assert lib.glq_fp8_check(None, None) == 1
    assert lib.glq_fp8_destroy(None) == 1
    assert lib.glq_fp8_info(None, None, None, None) == 1


@pytest.mark.parametrize("change,status", [
    ({"experts": 0}, 2), ({"experts": 513}, 2), ({"d": 12}, 2), ({"inter": 0}, 2), ({"topk": 0}, 2), ({"topk": 9}, 2),
    ({"experts": 20, "topk": 17}, 2), ({"experts": 16, "d": 1 << 20, "inter": 1 << 20}, 2), ({"scoring": 2}, 1), ({"routed_scale": float("inf")}, 1),
])
def test_moe_create_refusals(lib, change, status):
    import e8_lattice_codebook_b200 as glq
    base = dict(experts=8, d=128, inter=128, topk=2, scoring=0, renormalize=1, routed_scale=1.0)
    h = ctypes.c_void_p(5)
    assert lib.glq_moe_create(glq.MoeConfig(**{**base, **change}), P, P, P, P, P, P, None, ctypes.byref(h)) == status
    assert not h.value
    config = glq.MoeConfig(**base)
    for i in range(6):
        w = [P] * 6
        w[i] = None
        assert lib.glq_moe_create(config, *w, None, ctypes.byref(h)) == 1
    assert lib.glq_moe_create(None, P, P, P, P, P, P, None, ctypes.byref(h)) == 1
    assert lib.glq_moe_forward(None, P, 0, P, 0, P, 0, 1, None) == 1
    assert lib.glq_moe_reserve(None, 1) == 1
    assert lib.glq_moe_check(None, None) == 1
    assert lib.glq_moe_destroy(None) == 1
    assert lib.glq_moe_info(None, None, None) == 1


def test_reference_routes_ties_to_the_lowest_index():
    rows = np.array([[0.0, 1.0, 1.0, 1.0], [-np.inf, -np.inf, 2.0, -np.inf], [np.nan, 0.0, np.nan, 0.0], [-np.inf] * 4])
    got = ref.route(rows, 2, True, 0, 1.0)
    assert [[e for e, _ in r] for r in got] == [[1, 2], [2], [1, 3], []]
    assert got[0][0][1] == 0.5 and got[1][0][1] == 1.0
    every = ref.route(rows[:1], 1, False, 0, 2.0)[0][0][1]
    assert abs(every - 2 * np.e / (1 + 3 * np.e)) < 1e-15


def test_reference_rounds_as_the_format_does():
    """Every e4m3 value, the points half way between two, and their neighbours."""
    v = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (v[1:] + v[:-1]) / 2
    z = torch.cat([v, mid, mid * (1 - 2 ** -20), mid * (1 + 2 ** -20)])
    z = torch.cat([z, -z])
    np.testing.assert_array_equal(ref.e4m3_round(z.numpy()), z.float().to(torch.float8_e4m3fn).double().numpy())
    assert ref.e4m3_round(np.array([1e9]))[0] == 448
