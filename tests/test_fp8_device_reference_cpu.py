"""The 64-bit definitions that run on a device, on the CPU against those of
fp8_reference.py; their comparison, and the refusals of the test entries."""
import numpy as np
import pytest
import torch

import fp8_device_reference as dev
import fp8_reference as ref


def test_comparison_refuses_nan_and_values_outside():
    want = torch.tensor([1.0, -2.0, 0.0, 5.0, 5.0], dtype=torch.float64)
    bound = torch.tensor([0.5, 0.5, 0.0, 0.25, 0.25], dtype=torch.float64)
    got = torch.tensor([1.5, float("nan"), 0.0, 5.25 + 2.0 ** -20, float("inf")])
    assert dev.not_within(got, want, bound).tolist() == [False, True, False, True, True]


@pytest.mark.parametrize("m,n,B", [(136, 264, 5), (8, 8, 1), (264, 520, 17)])
def test_linear_is_the_same(m, n, B):
    gen = torch.Generator().manual_seed(m + n)
    w, s = dev.random_weight(gen, m, n)
    x = torch.randn(B, n, generator=gen).to(torch.bfloat16)
    x[:, ::37] *= 20
    if B > 4:
        x[4, :128] = 0
    xd = x.double().numpy()
    np.testing.assert_array_equal(dev.values(x.double()).numpy(), ref.values(xd))
    wv = ref.weight_values(w, s)
    np.testing.assert_array_equal(dev.weight_values(w, s).numpy(), wv)
    y, bound = dev.linear(x, w, s, torch.bfloat16)
    want = ref.values(xd) @ wv.T
    # two orders of a sum of at most 1000 doubles
    np.testing.assert_allclose(y.numpy(), want, rtol=0, atol=1e-12 * np.abs(want).max())
    np.testing.assert_allclose(bound.numpy(), ref.linear_bound(ref.values(xd), wv, want, torch.bfloat16), rtol=1e-9)


@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("scoring", [0, 1])
def test_moe_is_the_same(renormalize, scoring):
    gen = torch.Generator().manual_seed(3)
    E, d, inter, T = 5, 136, 200, 7
    raw = [[dev.random_weight(gen, *shape) for _ in range(E)] for shape in ((inter, d), (inter, d), (d, inter))]
    stacked = [(torch.stack([w.view(torch.uint8) for w, _ in m]).view(torch.float8_e4m3fn), torch.stack([s for _, s in m]))
               for m in raw]
    x, logits = torch.randn(T, d, generator=gen).to(torch.float16), torch.randn(T, E, generator=gen)
    logits[2] = 0.5
    got = dev.moe(x, logits, *stacked, 3, renormalize, scoring, 2.5)
    want = ref.moe(x.double().numpy(), logits.double().numpy(), *[[ref.weight_values(w, s) for w, s in m] for m in raw], 3,
                   renormalize, scoring, 2.5)
    for a, b in zip(got, want):
        np.testing.assert_allclose(a.numpy(), b, rtol=1e-9, atol=1e-12 * np.abs(b).max())


def test_sigmoid_weights_far_below_zero():
    """Scores that vanish in doubles have weights all the same: they depend on differences alone there."""
    l = torch.tensor([[-1000.0, -1001.0, -1002.0]])
    ids, w = dev.route(l, 2, True, 1, 1.0)
    assert ids.tolist() == [[0, 1]]
    np.testing.assert_allclose(w.numpy(), [[1 / (1 + np.exp(-1)), 1 / (1 + np.e)]], rtol=1e-12)


def test_null_handles():
    from e8_lattice_codebook_b200 import build as glq_build
    glq_build.build()
    import e8_lattice_codebook_b200 as glq
    assert glq._L().glq_fp8_plan(None, 1, None, None, None, None, None) == 1
    assert glq._L().glq_moe_selftest_wait(None, 1, 10, None) == 1
