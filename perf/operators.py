"""The 8-bit floating point operators, in their plain form and through the package.

Three operators that belong together: the quantiser of activations (one scale
for each token and group of 128 columns), the linear layer whose weights are
e4m3 with one scale for each 128 x 128 block, and a mixture-of-experts layer
for a few tokens whose experts are such layers.

`run` computes a case from what `prepare` made: with `own` false in elementary
fp32 operations, with `own` true through e8_lattice_codebook_b200.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
TOP = 448.0          # largest e4m3 value
FLOOR = 2.0 ** -110  # smallest group maximum a scale is made from
G = 128              # columns (and weight rows) that share a scale

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one token's hidden state before a shared q/k/v or gate/up product
        {"name": "quantize-1x5120", "op": "quantize", "B": 1, "n": 5120, "x": "bf16"},
        # the MLP activations of a prefill batch; 2048 x 11008 is the SmolLM3-3B-shaped width
        {"name": "quantize-2048x11008", "op": "quantize", "B": 2048, "n": 11008, "x": "f16"},
        # the smallest layer, one token: SmolLM2-360M-shaped, columns that end inside a block
        {"name": "linear-960x960-b1", "op": "linear", "m": 960, "n": 960, "B": 1, "x": "f16", "y": "f16"},
        # single-token decode of the largest layer of the 24B-class set
        {"name": "linear-32768x5120-b1", "op": "linear", "m": 32768, "n": 5120, "B": 1, "x": "bf16", "y": "bf16"},
        # batched decode, long reduction, fp32 out (a partial sum or logits)
        {"name": "linear-4096x14336-b13", "op": "linear", "m": 4096, "n": 14336, "B": 13, "x": "bf16", "y": "f32"},
        # a short ragged prompt between decode and prefill
        {"name": "linear-11008x2048-b77", "op": "linear", "m": 11008, "n": 2048, "B": 77, "x": "f16", "y": "f16"},
        # a prompt on a short layer: few output tiles
        {"name": "linear-2560x960-b333", "op": "linear", "m": 2560, "n": 960, "B": 333, "x": "bf16", "y": "bf16"},
        # prefill from activations that were quantised once for several layers
        {"name": "quantized-4096x14336-b2048", "op": "quantized", "m": 4096, "n": 14336, "B": 2048, "x": "bf16", "y": "bf16"},
        # the largest prefill batch of the benchmark
        {"name": "linear-14336x4096-b8192", "op": "linear", "m": 14336, "n": 4096, "B": 8192, "x": "bf16", "y": "bf16"},
        # one token through a layer of many small experts
        {"name": "moe-t1-e128k8-2048x768", "op": "moe", "T": 1, "E": 128, "k": 8, "d": 2048, "i": 768, "x": "bf16", "renorm": True},
        # a few concurrent requests; an expert width that ends inside a block
        {"name": "moe-t7-e64k6-2560x960", "op": "moe", "T": 7, "E": 64, "k": 6, "d": 2560, "i": 960, "x": "f16", "renorm": False},
        # the largest decode batch, every expert in use
        {"name": "moe-t64-e32k4-4096x2048", "op": "moe", "T": 64, "E": 32, "k": 4, "d": 4096, "i": 2048, "x": "bf16", "renorm": True},
    ]


def _spread(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    x = rng.choice(["f16", "bf16"])
    op = rng.choice(["quantize", "linear", "linear", "quantized", "moe", "moe"])
    if op == "moe":
        E = _spread(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        while True:
            d, i = _spread(rng, 512, 4096, 8), _spread(rng, 256, 2048, 8)
            if E * d * i <= 32 * 4096 * 2048:
                break
        return {"op": "moe", "T": _spread(rng, 1, 64), "E": E, "k": k, "d": d, "i": i, "x": x, "renorm": rng.random() < 0.5}
    while True:
        B, n, m = _spread(rng, 1, 8192), _spread(rng, 256, 16384, 8), _spread(rng, 256, 32768, 8)
        if op == "quantize" and B * n <= 2048 * 11008:
            return {"op": op, "B": B, "n": n, "x": x}
        if op != "quantize" and m * n <= 32768 * 5120 and B * m * n <= 8192 * 4096 * 14336:
            return {"op": op, "m": m, "n": n, "B": B, "x": x, "y": rng.choice([x, x, "f32"])}


def _weights(gen, experts, rows, cols):
    """Gaussian weights [experts][rows][cols] as e4m3 and their fp32 block scales."""
    w = torch.randn(experts, rows, cols, generator=gen, device="cuda")
    w *= cols ** -0.5
    rb, cb = -(-rows // G), -(-cols // G)
    pad = torch.nn.functional.pad(w.abs(), (0, cb * G - cols, 0, rb * G - rows))
    top = pad.view(experts, rb, G, cb, G).amax((2, 4))
    del pad
    s = top / TOP
    w /= _blocks(s, rows, cols)
    return w.to(E4M3), s


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    st = {"case": dict(case)}
    tokens, width = (case["T"], case["d"]) if case["op"] == "moe" else (case["B"], case["n"])
    x = torch.randn(tokens, width, generator=gen, device="cuda")
    # a few channels much larger than the rest, as hidden states have them
    x *= 1.0 + 19.0 * (torch.rand(width, generator=gen, device="cuda") < 0.01)
    st["x"] = x.to(DTYPES[case["x"]])
    if case["op"] in ("linear", "quantized"):
        w, s = _weights(gen, 1, case["m"], case["n"])
        st["w"], st["ws"] = w[0], s[0]
    if case["op"] == "moe":
        E, d, i = case["E"], case["d"], case["i"]
        st["gate"], st["up"], st["down"] = _weights(gen, E, i, d), _weights(gen, E, i, d), _weights(gen, E, d, i)
        st["logits"] = torch.randn(tokens, E, generator=gen, device="cuda")
    return st


def prepare(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "quantized":  # the caller has these in hand: one quantisation serves several layers
        st["q"], st["s"] = _quantize(st["x"])
    if own:  # a program lays its weights out once and keeps the layer
        import e8_lattice_codebook_b200 as glq

        if case["op"] in ("linear", "quantized"):
            st["layer"] = glq.Fp8Linear(st.pop("w"), st.pop("ws"))
        elif case["op"] == "moe":
            gate, up, down = st.pop("gate"), st.pop("up"), st.pop("down")
            st["layer"] = glq.Fp8Moe(*gate, *up, *down, topk=case["k"], renormalize=case["renorm"])
    return st


def _blocks(s, rows, cols):
    """Block scales [..., rows/128, cols/128] spread over [..., rows, cols]."""
    return s.repeat_interleave(G, -2)[..., :rows, :].repeat_interleave(G, -1)[..., :cols]


def _quantize(x):
    """e4m3 values [tokens][columns rounded up to 128] and scales [groups][tokens]."""
    tokens, n = x.shape
    groups = -(-n // G)
    v = torch.nn.functional.pad(x.float(), (0, groups * G - n)).view(tokens, groups, G)
    top = v.abs().amax(-1).clamp_min(FLOOR)
    full = torch.full_like(top, TOP)  # a tensor: a scalar operand would be multiplied by its rounded inverse
    q = (v * (full / top).unsqueeze(-1)).to(E4M3)
    return q.view(tokens, groups * G), (top / full).t().contiguous()


def _values(q, s, n):
    """The fp32 values that quantised activations stand for."""
    return q[:, :n].float() * s.t().repeat_interleave(G, -1)[:, :n]


def _requantized(h):
    """h [..., n] in fp32, rounded to the e4m3 values it is held in."""
    flat = h.reshape(-1, h.shape[-1])
    return _values(*_quantize(flat), flat.shape[-1]).view(h.shape)


def _dequantized(w, s):
    return w.float() * _blocks(s, w.shape[-2], w.shape[-1])


def _moe(st):
    case, x, logits = st["case"], st["x"], st["logits"].float()
    T, E, k = case["T"], case["E"], case["k"]
    # a stable sort: ties go to the lowest index
    order = torch.sort(logits, dim=-1, descending=True, stable=True).indices[:, :k]
    p = torch.exp(logits - logits.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).gather(1, order)
    if case["renorm"]:
        p = p / p.sum(-1, keepdim=True)
    xv = _requantized(x.float())
    few = T * k <= E  # the chosen experts' weights alone, else every expert over every token
    pick = order.reshape(-1) if few else slice(None)
    rows = xv.repeat_interleave(k, 0).unsqueeze(1) if few else xv.unsqueeze(0)
    (gw, gs), (uw, us), (dw, ds) = ((w.view(torch.uint8)[pick].view(E4M3), s[pick]) for w, s in (st["gate"], st["up"], st["down"]))
    g = rows @ _dequantized(gw, gs).transpose(1, 2)
    u = rows @ _dequantized(uw, us).transpose(1, 2)
    h = _requantized(g / (1.0 + torch.exp(-g)) * u)
    y = h @ _dequantized(dw, ds).transpose(1, 2)
    if few:
        y = (y.view(T, k, -1) * p.unsqueeze(-1)).sum(1)
    else:
        mix = torch.zeros(T, E, device=x.device).scatter_(1, order, p)
        y = (y * mix.t().unsqueeze(-1)).sum(0)
    return y.to(x.dtype)


def run(st):
    case = st["case"]
    if own:
        import e8_lattice_codebook_b200 as glq

        if case["op"] == "quantize":
            return glq.fp8_quantize(st["x"])
        if case["op"] == "linear":
            return st["layer"](st["x"], out_dtype=DTYPES[case["y"]])
        if case["op"] == "quantized":
            return st["layer"].forward_quantized(st["q"], st["s"], out_dtype=DTYPES[case["y"]])
        return st["layer"](st["x"], st["logits"])
    if case["op"] == "quantize":
        return _quantize(st["x"])
    if case["op"] == "moe":
        return _moe(st)
    q, s = (st["q"], st["s"]) if case["op"] == "quantized" else _quantize(st["x"])
    return (_values(q, s, case["n"]) @ _dequantized(st["w"], st["ws"]).t()).to(DTYPES[case["y"]])


def work(case):
    if case["op"] == "quantize":
        v = case["B"] * case["n"]
        return {"bytes": 3 * v + 4 * case["B"] * -(-case["n"] // G), "flops": 3 * v}
    if case["op"] == "moe":
        T, E, k, d, i = (case[c] for c in ("T", "E", "k", "d", "i"))
        used = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token chose, on average
        scales = 4 * (2 * -(-i // G) * -(-d // G) + -(-d // G) * -(-i // G))
        return {"bytes": used * (3 * d * i + scales) + T * (4 * d + 4 * E), "flops": 6 * T * k * d * i}
    m, n, B = case["m"], case["n"], case["B"]
    x = B * n + 4 * B * -(-n // G) if case["op"] == "quantized" else 2 * B * n
    return {"bytes": m * n + 4 * -(-m // G) * -(-n // G) + x + B * m * (4 if case["y"] == "f32" else 2), "flops": 2 * B * m * n}


# ---------------------------------------------------------------------------
# The definition in 64 bits.  A held value is what its format holds: scales
# and the quantiser's two roundings before e4m3 are fp32 by definition, all
# else is a double.
# ---------------------------------------------------------------------------

def _exact_held(v):
    """(e4m3 values, scales) of rows v [tokens][n] (doubles), both as doubles."""
    n = v.shape[1]
    qs, ss = [], []
    for c in range(0, n, G):
        part = v[:, c:c + G]
        a = part.abs().max(dim=1, keepdim=True).values.clamp(min=FLOOR)
        inv = (TOP / a).float().double()
        z = (part * inv).float().double()
        # e4m3: 3 mantissa bits, exponents from -6; half to even
        e = torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6)))
        step = torch.exp2(e - 3)
        qs.append((torch.round(z / step) * step).clamp(-TOP, TOP))
        ss.append((a / TOP).float().double())
    return qs, ss


def _exact_rows(v):
    """Rows v as the doubles that their held values stand for."""
    qs, ss = _exact_held(v)
    return torch.cat([q * s for q, s in zip(qs, ss)], dim=1)


def _exact_weight(w, s):
    out = w.to(torch.float64)
    for r in range(s.shape[0]):
        for c in range(s.shape[1]):
            out[r * G:(r + 1) * G, c * G:(c + 1) * G] *= s[r, c].double()
    return out


def exact(case, seed):
    st = _inputs(case, seed)
    x = st["x"].double()
    if case["op"] == "quantize":
        qs, ss = _exact_held(x)
        q = torch.zeros(x.shape[0], len(qs) * G, dtype=torch.float64, device=x.device)
        q[:, :x.shape[1]] = torch.cat(qs, dim=1)
        return q, torch.cat(ss, dim=1).t().contiguous()
    xv = _exact_rows(x)
    if case["op"] != "moe":
        return xv @ _exact_weight(st["w"], st["ws"]).T
    logits = st["logits"].double()
    chosen = {}
    for t, row in enumerate(logits.tolist()):
        best = sorted(range(len(row)), key=lambda e: (-row[e], e))[:case["k"]]
        total = math.fsum(math.exp(row[e]) for e in (best if case["renorm"] else range(len(row))))
        for e in best:
            chosen.setdefault(e, []).append((t, math.exp(row[e]) / total))
    y = torch.zeros_like(x)
    for e, uses in chosen.items():
        rows = torch.tensor([t for t, _ in uses], device=x.device)
        weight = torch.tensor([p for _, p in uses], dtype=torch.float64, device=x.device)
        gate, up, down = (_exact_weight(st[w][0][e], st[w][1][e]) for w in ("gate", "up", "down"))
        g, u = xv[rows] @ gate.T, xv[rows] @ up.T
        h = _exact_rows((g * torch.sigmoid(g) * u).float().double())
        y.index_add_(0, rows, weight[:, None] * (h @ down.T))
    return y
