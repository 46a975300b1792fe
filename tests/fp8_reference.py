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


# ---------------------------------------------------------------------------
# Mixture of experts
# ---------------------------------------------------------------------------

def route(logits: np.ndarray, topk: int, renormalize: bool, scoring: int, scale: float):
    """[(expert, weight), ...] per token: the largest logits, the lowest index
    first among equals, never -inf or NaN."""
    out = []
    for row in logits:
        ok = [e for e in range(len(row)) if row[e] > -np.inf]
        best = sorted(ok, key=lambda e: (-row[e], e))[:topk]
        if scoring == 0:
            top = max((row[e] for e in ok), default=0.0)
            w = {e: np.exp(row[e] - top) for e in ok}
            total = sum(w[e] for e in (best if renormalize else ok))
        else:
            w = {e: 1.0 / (1.0 + np.exp(-row[e])) for e in best}
            total = sum(w[e] for e in best) if renormalize else 1.0
        out.append([(e, w[e] / total * scale) for e in best])
    return out


def _between(h, err):
    """How far the values held for h may be apart when h itself is known to
    +-err: (held values, bound).  A value near the middle of two e4m3 values
    may fall to either."""
    n = h.shape[1]
    q, s = quantize(h.astype(np.float32).astype(np.float64))
    held = (q * np.repeat(s.T, G, axis=1))[:, :n]
    bound = np.zeros_like(held)
    for g in range(0, n, G):
        v, e = np.abs(h[:, g:g + G]), err[:, g:g + G]
        a = np.maximum(v.max(axis=1, keepdims=True), FLOOR)
        rel = np.max(e, axis=1, keepdims=True) / a + 2.0 ** -22  # of the scale
        z = v * TOP / a
        dz = e * TOP / a + z * rel
        lo, hi = e4m3_round(np.maximum(z - dz, 0)), e4m3_round(z + dz)
        bound[:, g:g + G] = (np.abs(hi - lo) + hi * rel) * a / TOP
    return held, bound


def moe(x, logits, gate, up, down, topk, renormalize, scoring, scale):
    """(y, bound): the layer in 64 bits and how far fp32 arithmetic may be from
    it before y's own rounding.  gate, up, down: lists of weight values."""
    xv = values(x)
    y, bound = np.zeros_like(x), np.zeros_like(x)
    n_x, n_h = x.shape[1], gate[0].shape[0]
    terms = lambda n: (min(n, G) + 4 * (-(-n // G)) + 8) * 2.0 ** -23  # noqa: E731  (as linear_bound, split sums)
    for t, chosen in enumerate(route(logits, topk, renormalize, scoring, scale)):
        for e, p in chosen:
            v = xv[t:t + 1]
            g, u = v @ gate[e].T, v @ up[e].T
            eg, eu = (terms(n_x) * (np.abs(v) @ np.abs(w[e]).T) for w in (gate, up))
            sig = 1.0 / (1.0 + np.exp(-g))
            h = g * sig * u
            # |silu'| <= 1.1; exp, sum, quotient and product lose a few units each
            eh = 1.1 * eg * np.abs(u) + np.abs(g * sig) * eu + 1.1 * eg * eu + np.abs(h) * (np.abs(g) + 16) * 2.0 ** -23
            held, b = _between(h, eh)
            y[t] += p * (held @ down[e].T)[0]
            mag = np.abs(held) @ np.abs(down[e]).T
            ep = (logits.shape[1] + 16 + np.abs(logits[t][np.isfinite(logits[t])]).max(initial=0.0)) * 2.0 ** -23
            bound[t] += p * ((b @ np.abs(down[e]).T) + (terms(n_h) + topk * 2.0 ** -23 + ep) * mag)[0]
    return y, bound
