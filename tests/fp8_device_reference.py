"""The definitions of fp8_reference.py as torch operations in 64 bits, which run
on the tensors' device: for layers of real size.  The error bounds are the
same ones, with the same derivations."""
import torch

TOP, FLOOR, G = 448.0, 2.0 ** -110, 128


def not_within(got, want, bound):
    """Where got is further than bound from want; a NaN always is."""
    return ~((got.double() - want).abs() <= bound)


def e4m3_round(z):
    """Doubles to the nearest e4m3 value, half to even, saturating."""
    a = z.abs().clamp(max=TOP)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=TOP), z)


def values(x):
    """What the rounded activations x [B][n] (doubles) stand for."""
    B, n = x.shape
    v = torch.nn.functional.pad(x, (0, -n % G)).view(B, -1, G)
    a = v.abs().amax(2, keepdim=True).clamp(min=FLOOR)
    q = e4m3_round((v * (TOP / a).float().double()).float().double())
    return (q * (a / TOP).float().double()).view(B, -1)[:, :n]


def weight_values(w, scales):
    """e4m3 weights [..., m, n] times their block scales, in doubles."""
    m, n = w.shape[-2:]
    return w.double() * scales.double().repeat_interleave(G, -2)[..., :m, :].repeat_interleave(G, -1)[..., :n]


def random_weight(gen, m, n):
    """e4m3 weights and scales of a Gaussian matrix, on the generator's device."""
    w = torch.randn(m, n, generator=gen, device=gen.device) * n ** -0.5
    rb, cb = -(-m // G), -(-n // G)
    s = torch.nn.functional.pad(w.abs(), (0, -n % G, 0, -m % G)).view(rb, G, cb, G).amax((1, 3)) / TOP
    w /= s.repeat_interleave(G, 0)[:m].repeat_interleave(G, 1)[:, :n]
    return w.to(torch.float8_e4m3fn), s


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def smallest(dtype):
    return torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2


def terms(n, more):
    """Units of 2^-23 that a sum over n products may lose, as linear_bound counts them."""
    return (min(n, G) + 4 * (-(-n // G)) + more) * 2.0 ** -23


def linear(x, w, scales, dtype):
    """(y, bound) of the layer for x [B][n], y rounded to dtype."""
    xv, wv = values(x.double()), weight_values(w, scales)
    want = xv @ wv.t()
    return want, half_step(dtype) * want.abs() + terms(x.shape[1], 4) * (xv.abs() @ wv.abs().t()) + smallest(dtype)


def route(logits, topk, renormalize, scoring, scale):
    """(experts [T][topk], weights [T][topk]) of finite logits; ties go to the
    lowest index."""
    l = logits.double()
    best = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :topk]
    chosen = l.gather(1, best)
    if scoring == 0:
        w = torch.exp(chosen - l.amax(1, keepdim=True))
        total = w.sum(1, keepdim=True) if renormalize else torch.exp(l - l.amax(1, keepdim=True)).sum(1, keepdim=True)
        return best, w / total * scale
    log_w = torch.nn.functional.logsigmoid(chosen)  # the quotient of scores that vanish in doubles is a number yet
    if renormalize:
        log_w = log_w - torch.logsumexp(log_w, 1, keepdim=True)
    return best, torch.exp(log_w) * scale


def _held(h, err):
    """(values held for h, how far they may be when h is known to +-err)."""
    m, n = h.shape
    held = values(h.float().double())
    pad = lambda t: torch.nn.functional.pad(t, (0, -n % G)).view(m, -1, G)  # noqa: E731
    v, e = pad(h.abs()), pad(err)
    a = v.amax(2, keepdim=True).clamp(min=FLOOR)
    rel = e.amax(2, keepdim=True) / a + 2.0 ** -22  # of the scale
    z = v * TOP / a
    dz = e * TOP / a + z * rel
    lo, hi = e4m3_round((z - dz).clamp(min=0)), e4m3_round(z + dz)
    return held, (((hi - lo).abs() + hi * rel) * a / TOP).view(m, -1)[:, :n]


def moe(x, logits, gate, up, down, topk, renormalize, scoring, scale):
    """(y, bound before y's own rounding); gate, up, down: (weights, scales)."""
    xv = values(x.double())
    experts, weights = route(logits, topk, renormalize, scoring, scale)
    y, bound = torch.zeros_like(xv), torch.zeros_like(xv)
    for e in experts.unique().tolist():
        t, c = (experts == e).nonzero(as_tuple=True)
        gw, uw, dw = (weight_values(w[e], s[e]) for w, s in (gate, up, down))
        v, p = xv[t], weights[t, c][:, None]
        g, u = v @ gw.t(), v @ uw.t()
        eg, eu = (terms(x.shape[1], 8) * (v.abs() @ w.abs().t()) for w in (gw, uw))
        act = g * torch.sigmoid(g)
        h = act * u
        # |silu'| <= 1.1; exp, sum, quotient and product lose a few units each
        eh = 1.1 * eg * u.abs() + act.abs() * eu + 1.1 * eg * eu + h.abs() * (g.abs() + 16) * 2.0 ** -23
        held, b = _held(h, eh)
        ep = (logits.shape[1] + 16 + logits[t].double().abs().amax(1, keepdim=True)) * 2.0 ** -23
        mag = held.abs() @ dw.abs().t()
        y.index_add_(0, t, p * (held @ dw.t()))
        bound.index_add_(0, t, p * (b @ dw.abs().t() + (terms(gw.shape[0], 8) + topk * 2.0 ** -23 + ep) * mag))
    return y, bound
