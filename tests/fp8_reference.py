"""The 8-bit float operators from their definition, in 64 bits, on the CPU:
plain loops and products, sharing no code with the library."""
import numpy as np
import torch

TOP, FLOOR, G = 448.0, 2.0 ** -110, 128


def e4m3_round(z: np.ndarray) -> np.ndarray:
    """Doubles to the nearest e4m3 value, half to even, saturating."""
    a = np.minimum(np.abs(z), TOP)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, TOP), z)


def quantize(x: np.ndarray):
    """x [B][n] doubles -> (values [B][G*128], scales [G][B]) as doubles."""
    B, n = x.shape
    groups = -(-n // G)
    q, s = np.zeros((B, groups * G)), np.zeros((groups, B))
    with np.errstate(all="ignore"):
        for g in range(groups):
            v = x[:, g * G:(g + 1) * G]
            a = np.maximum(np.max(np.abs(v), axis=1, initial=0.0), FLOOR)  # NaN if any is
            s[g] = (a / TOP).astype(np.float32)
            inv = (TOP / a).astype(np.float32).astype(np.float64)
            z = (v * inv[:, None]).astype(np.float32).astype(np.float64)
            q[:, g * G:g * G + v.shape[1]] = e4m3_round(z)
    return q, s


def values(x: np.ndarray) -> np.ndarray:
    """What the rounded activations stand for."""
    q, s = quantize(x)
    return (q * np.repeat(s.T, G, axis=1))[:, :x.shape[1]]


def weight_values(w: torch.Tensor, scales: torch.Tensor) -> np.ndarray:
    m, n = w.shape
    s = scales.cpu().double().numpy()
    return w.cpu().float().double().numpy() * np.repeat(np.repeat(s, G, 0)[:m], G, 1)[:, :n]


def random_weight(gen, m, n, gain=None):
    """e4m3 weights and scales (CPU tensors) of a Gaussian matrix."""
    w = torch.randn(m, n, generator=gen, dtype=torch.float64) * (n ** -0.5 if gain is None else gain)
    rb, cb = -(-m // G), -(-n // G)
    s = torch.zeros(rb, cb, dtype=torch.float32)
    q = torch.zeros(m, n, dtype=torch.float64)
    for r in range(rb):
        for c in range(cb):
            blk = w[r * G:(r + 1) * G, c * G:(c + 1) * G]
            s[r, c] = float(blk.abs().max()) / TOP
            q[r * G:(r + 1) * G, c * G:(c + 1) * G] = blk / s[r, c].double()
    return q.float().to(torch.float8_e4m3fn), s


def half_step(dtype) -> float:
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def smallest(dtype) -> float:
    """The largest absolute error of one rounding among subnormals."""
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def linear_bound(xv, wv, ref, dtype):
    """How far y may be from ref = xv wv^T.  fp32: each of a sum's n products
    (exact in fp32) is added once, with at most one unit of the last place of
    the running sum lost (2^-23, the tensor core cuts rather than rounds), the
    blocks' sums and scales take three roundings more each; then one rounding
    to dtype."""
    mag = np.abs(xv) @ np.abs(wv).T
    n = xv.shape[1]
    terms = min(n, G) + 4 * (-(-n // G)) + 4
    return half_step(dtype) * np.abs(ref) + terms * 2.0 ** -23 * mag + smallest(dtype)
