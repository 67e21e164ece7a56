"""Cases of the 8-bit floating-point linear layers: what is timed, its plain form and its exact value.

Scheme.  A group is 128 consecutive input channels of one row (activations) or
128 output x 128 input channels (weights).  Its scale is the least power of two
2^e, e >= -126, with amax <= 448 * 2^e, and its codes are e4m3(v * 2^-e), round
half to even.  A layer is out = bf16(x . w^T + bias) on what the codes stand for.

  linear   bf16 rows through one weight matrix
  grouped  rows sorted by expert, each span through its expert's matrix
  gated    rows [gate | up] through silu(gate) * up, then a linear layer
  experts  grouped (gate and up), silu(gate) * up, grouped (down): one feed-forward of experts
"""
import math

import torch

own = False

BLOCK = 128


def listed():
    return [
        # one token through a small projection: the smallest call, latency
        {"name": "linear 1 token", "op": "linear", "M": 1, "N": 2048, "K": 2048, "bias": True, "pad": 0},
        # a decode batch: the weights' bytes
        {"name": "linear 16 tokens", "op": "linear", "M": 16, "N": 8192, "K": 4096, "bias": False, "pad": 0},
        # a short prompt, channels that end inside blocks, rows of a wider buffer
        {"name": "linear odd", "op": "linear", "M": 77, "N": 1000, "K": 1176, "bias": True, "pad": 24},
        # a chunk of a prompt
        {"name": "linear 300 tokens", "op": "linear", "M": 300, "N": 4096, "K": 4096, "bias": False, "pad": 0},
        # a long prompt: the tensor cores
        {"name": "linear 8192 tokens", "op": "linear", "M": 8192, "N": 8192, "K": 4096, "bias": True, "pad": 0},
        # a decode batch of 16 tokens, 4 experts each
        {"name": "grouped 64 rows", "op": "grouped", "E": 32, "active": 24, "M": 64, "N": 2048, "K": 2048},
        # small experts with odd sizes, some of them empty
        {"name": "grouped odd", "op": "grouped", "E": 9, "active": 7, "M": 501, "N": 328, "K": 200},
        # a prompt over many experts, ragged
        {"name": "grouped 16384 rows", "op": "grouped", "E": 64, "active": 60, "M": 16384, "N": 2048, "K": 2048},
        # one token's down projection
        {"name": "gated 1 token", "op": "gated", "M": 1, "N": 4096, "K": 8192},
        # a prompt's down projection
        {"name": "gated 4096 tokens", "op": "gated", "M": 4096, "N": 4096, "K": 8192},
        # feed-forward of experts, a decode batch and a prompt
        {"name": "experts 32 rows", "op": "experts", "E": 32, "active": 16, "M": 32, "N": 2048, "K": 1024},
        {"name": "experts 8192 rows", "op": "experts", "E": 32, "active": 32, "M": 8192, "N": 2048, "K": 1024},
    ]


def draw(rng):
    def size(lo, hi):  # spread over the logarithm, half of them rounded to a usual size
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return v if rng.random() < 0.5 or v < 64 else v // 64 * 64

    op = rng.choice(["linear", "grouped", "gated", "experts"])
    if op == "linear":
        return {"op": op, "M": size(1, 8192), "N": size(64, 8192), "K": size(64, 4096), "bias": rng.random() < 0.5,
                "pad": rng.choice([0, 8, 40])}
    if op == "gated":
        return {"op": op, "M": size(1, 4096), "N": size(64, 4096), "K": size(64, 8192)}
    m, e = size(1, 16384 if op == "grouped" else 8192), rng.randint(2, 64 if op == "grouped" else 32)
    return {"op": op, "E": e, "active": rng.randint(min(m, (e + 1) // 2), min(m, e)), "M": m, "N": size(64, 2048),
            "K": size(64, 2048 if op == "grouped" else 1024)}


# ---------------------------------------------------------------- inputs

def _random(shape, scale, gen):
    return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)


def _rows(m, k, pad, gen):
    """Activations: rows of different size, a few input channels far above the others; `pad` more columns behind."""
    x = torch.randn((m, k + pad), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((m, 1), generator=gen, device="cuda"))
    x *= torch.where(torch.rand((1, k + pad), generator=gen, device="cuda") < 0.01, 12.0, 1.0)
    return x.to(torch.bfloat16)[:, :k]


def _counts(case, seed):
    """Rows of each expert: `active` experts drawn without order, at least one row each, the rest by skewed weights."""
    gen = torch.Generator().manual_seed(seed)
    e, active, m = case["E"], case["active"], case["M"]
    who = torch.randperm(e, generator=gen)[:active]
    weight = torch.exp(0.6 * torch.randn(active, generator=gen))
    more = torch.multinomial(weight, max(1, m - active), replacement=True, generator=gen)[:m - active]
    counts = torch.zeros(e, dtype=torch.int64)
    counts[who] = 1 + torch.bincount(more, minlength=active)
    return counts


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, m, n, k = case["op"], case["M"], case["N"], case["K"]
    if op == "linear":
        bias = _random((n,), 0.5, gen) if case["bias"] else None
        return {"x": _rows(m, k, case["pad"], gen), "w": _random((1, n, k), k ** -0.5, gen), "bias": bias}
    if op == "gated":
        return {"x": _rows(m, 2 * k, 0, gen), "w": _random((1, n, k), k ** -0.5, gen)}
    counts = _counts(case, seed)
    d = {"counts": counts}
    if op == "grouped":
        return dict(d, x=_rows(m, k, 0, gen), w=_random((case["E"], n, k), k ** -0.5, gen))
    # experts: n model channels, k hidden ones (w gives gate and up, w2 the way back)
    return dict(d, x=_rows(m, n, 0, gen), w=_random((case["E"], 2 * k, n), n ** -0.5, gen),
                w2=_random((case["E"], n, k), k ** -0.5, gen))


# ------------------------------------------------------------ plain form

def _exponents(amax):
    """Least e >= -126 with amax <= 448 * 2^e, from amax = f * 2^p with 0.5 <= f < 1 and 448 = 0.875 * 2^9."""
    f, p = torch.frexp(amax)
    return torch.clamp(torch.where(f <= 0.875, p - 9, p - 8), min=-126)


def _quantised(v, rows):
    """Codes of v [..., R, C] in groups of rows x 128, and the power of two of each group."""
    r, c = v.shape[-2:]
    rb, cb = -(-r // rows), -(-c // BLOCK)
    v = torch.nn.functional.pad(v.float(), (0, cb * BLOCK - c, 0, rb * rows - r))
    g = v.reshape(*v.shape[:-2], rb, rows, cb, BLOCK)
    e = _exponents(g.abs().amax(dim=(-3, -1), keepdim=True))
    return torch.ldexp(g, -e).to(torch.float8_e4m3fn), torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _values(codes, scale, r, c):
    """What codes and scales stand for, in 32 bits, [..., r, c]."""
    v = codes.float() * scale
    v = v.reshape(*v.shape[:-4], v.shape[-4] * v.shape[-3], v.shape[-2] * v.shape[-1])
    return v[..., :r, :c]


def _act(v):
    return _values(*_quantised(v, 1), *v.shape[-2:])


def _silu_mul(h):
    g, u = h.float().chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _grouped(v, s, w, n, k):
    """Rows of each expert padded to the longest, one batched product, and back."""
    padded = torch.zeros((s["E"], s["most"], v.shape[-1]), device=v.device)
    padded[s["expert"], s["place"]] = v
    return torch.bmm(padded, _values(*w, n, k).transpose(1, 2))[s["expert"], s["place"]]


def _run_plain(s):
    op, n, k = s["op"], s["N"], s["K"]
    if op == "linear":
        y = _act(s["x"]) @ _values(*s["wq"], n, k)[0].t()
        return (y + s["bias"].float() if s["bias"] is not None else y).to(torch.bfloat16)
    if op == "gated":
        return (_act(_silu_mul(s["x"])) @ _values(*s["wq"], n, k)[0].t()).to(torch.bfloat16)
    if op == "grouped":
        return _grouped(_act(s["x"]), s, s["wq"], n, k).to(torch.bfloat16)
    h = _grouped(_act(s["x"]), s, s["wq"], 2 * k, n).to(torch.bfloat16)
    return _grouped(_act(_silu_mul(h)), s, s["wq2"], n, k).to(torch.bfloat16)


# -------------------------------------------------------------- the calls

def _prepare_own(s, w, w2):
    from video_vae_decode_b200 import qvae

    s["qvae"] = qvae
    s["packed"] = qvae.fp8_quantize_weights(w)
    if w2 is not None:
        s["packed2"] = qvae.fp8_quantize_weights(w2)
    m, n, k = s["M"], s["N"], s["K"]
    s["out"] = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
    s["workspace"] = qvae.fp8_workspace(m, n if s["op"] == "experts" else k)
    if s["op"] == "experts":
        s["h"] = torch.empty((m, 2 * k), dtype=torch.bfloat16, device="cuda")
        s["workspace2"] = qvae.fp8_workspace(m, k)


def _run_own(s):
    q, op = s["qvae"], s["op"]
    if op == "linear":
        return q.linear_fp8_fused(s["x"], s["packed"], s["bias"], out=s["out"], workspace=s["workspace"])
    if op == "gated":
        return q.linear_fp8_fused(s["x"], s["packed"], silu_mul=True, out=s["out"], workspace=s["workspace"])
    if op == "grouped":
        return q.linear_fp8_grouped_fused(s["x"], s["offsets"], s["packed"], out=s["out"], workspace=s["workspace"])
    h = q.linear_fp8_grouped_fused(s["x"], s["offsets"], s["packed"], out=s["h"], workspace=s["workspace"])
    return q.linear_fp8_grouped_fused(h, s["offsets"], s["packed2"], silu_mul=True, out=s["out"],
                                      workspace=s["workspace2"])


def prepare(case, seed):
    d = _inputs(case, seed)
    s = {"op": case["op"], "M": case["M"], "N": case["N"], "K": case["K"], "x": d["x"], "bias": d.get("bias")}
    if "counts" in d:
        counts = d["counts"]
        ends = torch.cumsum(counts, 0)
        s["offsets"] = torch.cat([ends.new_zeros(1), ends]).to(torch.int32).cuda()
        s["E"], s["most"] = case["E"], int(counts.max())
        s["expert"] = torch.repeat_interleave(torch.arange(case["E"]), counts).cuda()
        s["place"] = (torch.arange(case["M"]) - torch.repeat_interleave(ends - counts, counts)).cuda()
    if own:
        _prepare_own(s, d["w"], d.get("w2"))
    else:
        s["wq"] = _quantised(d["w"], BLOCK)
        if "w2" in d:
            s["wq2"] = _quantised(d["w2"], BLOCK)
    return s


def run(s):
    return _run_own(s) if own else _run_plain(s)


def work(case):
    op, m, n, k = case["op"], case["M"], case["N"], case["K"]
    a = case.get("active", 1)

    def weights(rows, cols):
        return rows * cols + -(-rows // BLOCK) * -(-cols // BLOCK)

    if op == "linear":
        return {"bytes": 2 * m * k + weights(n, k) + 2 * m * n + (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    if op == "gated":
        return {"bytes": 4 * m * k + weights(n, k) + 2 * m * n, "flops": 2 * m * n * k}
    if op == "grouped":
        return {"bytes": 2 * m * k + a * weights(n, k) + 2 * m * n + 4 * (case["E"] + 1), "flops": 2 * m * n * k}
    return {"bytes": 2 * m * n + a * (weights(2 * k, n) + weights(n, k)) + 2 * m * n + 4 * (case["E"] + 1),
            "flops": 6 * m * n * k}


# ------------------------------------------------------------------ exact

def _exact_codes(v, rows):
    """What v [R, C], in 64 bits, stands for after quantisation, from the definition of e4m3: 3 mantissa bits, least
    normal exponent -6."""
    r, c = v.shape
    rb, cb = -(-r // rows), -(-c // 128)
    big = torch.zeros((rb * rows, cb * 128), dtype=torch.float64, device=v.device)
    big[:r, :c] = v.double()
    t = big.view(rb, rows, cb, 128)
    amax = t.abs().amax(3, keepdim=True).amax(1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(torch.clamp(amax / 448, min=2.0 ** -126))))
    u = t / scale
    top = torch.floor(torch.log2(torch.clamp(u.abs(), min=2.0 ** -6)))
    step = torch.exp2(top - 3)
    return (torch.round(u / step) * step * scale).reshape(rb * rows, cb * 128)[:r, :c]


def _exact_product(x, w):
    return _exact_codes(x, 1) @ _exact_codes(w, 128).t()


def _exact_gate(h, k):
    h = h.double()
    return h[:, :k] * torch.sigmoid(h[:, :k]) * h[:, k:]


def exact(case, seed):
    d = _inputs(case, seed)
    op, k = case["op"], case["K"]
    if op == "linear":
        y = _exact_product(d["x"], d["w"][0])
        return y if d["bias"] is None else y + d["bias"].double()
    if op == "gated":
        return _exact_product(_exact_gate(d["x"], k), d["w"][0])
    spans = torch.split(d["x"], d["counts"].tolist())
    y = [_exact_product(x, w) for x, w in zip(spans, d["w"]) if x.shape[0]]
    if op == "experts":  # the hidden rows are stored in bf16 between the two products
        w2 = [w for x, w in zip(spans, d["w2"]) if x.shape[0]]
        y = [_exact_product(_exact_gate(h.to(torch.bfloat16), k), w) for h, w in zip(y, w2)]
    return torch.cat(y)
