"""Operators with one scale per 128 values, as they are used in an expert layer: what is measured.

Five operators and their sizes:

  quantize      bf16 -> E4M3: activations with a scale per row and 128 columns, weights with a scale per 128x128 block
                (and the transposed copy that the input gradient's product reads)
  gemm          E4M3 product with those scales, weight K-major
  grouped_gemm  the same for ragged row ranges, each with its expert's weight
  wgrad         weight gradients of the experts, dW_g = dY_g^T X_g, over ragged row ranges
  swiglu        silu(gate) * up and its backward pass, each with the quantizer of its result

A case's group sizes follow from the case alone, its values from the seed.
"""

import collections
import math
import random

import torch

own = False

GROUP = 128
E4M3_MAX = 448.0


def _blocks(n):
    return (n + GROUP - 1) // GROUP


# ---- the cases ---------------------------------------------------------------------------
def listed():
    return [
        # the activations of eight sequences, one token each, before a projection: latency
        {"name": "quantize_rows_8x8192", "op": "quantize_rows", "rows": 8, "cols": 8192},
        # a training step lays out the experts' weights once, both ways round; the last blocks are partial
        {"name": "quantize_weights_8x4112x2064", "op": "quantize_weights", "groups": 8, "rows": 4112, "cols": 2064},
        # decode: the weight is streamed once for eight tokens
        {"name": "gemm_8x8192x8192", "op": "gemm", "m": 8, "n": 8192, "k": 8192},
        # a chunk of a prompt with sizes that fill no tile and a partial last block
        {"name": "gemm_1017x2064x1552", "op": "gemm", "m": 1017, "n": 2064, "k": 1552},
        # the square product
        {"name": "gemm_4096x4096x4096", "op": "gemm", "m": 4096, "n": 4096, "k": 4096},
        # prompts of 8192 tokens through a wide projection
        {"name": "gemm_8192x28672x8192", "op": "gemm", "m": 8192, "n": 28672, "k": 8192},
        # decode through 64 experts: most have one or two rows, some none
        {"name": "grouped_64x96x4096x2048", "op": "grouped_gemm", "groups": 64, "m": 96, "n": 4096, "k": 2048},
        # 8192 rows over 16 experts, two of them empty
        {"name": "grouped_16x8192x4096x7168", "op": "grouped_gemm", "groups": 16, "m": 8192, "n": 4096, "k": 7168},
        # gradients of a few rows: every expert's gradient is written, little is computed
        {"name": "wgrad_8x333x1040x528", "op": "wgrad", "groups": 8, "m": 333, "n": 1040, "k": 528},
        # a training step's gradients
        {"name": "wgrad_16x8192x4096x2048", "op": "wgrad", "groups": 16, "m": 8192, "n": 4096, "k": 2048},
        # between the experts' two products, forward
        {"name": "swiglu_8192x2048", "op": "swiglu", "rows": 8192, "d": 2048},
        # and backward
        {"name": "swiglu_backward_8192x2048", "op": "swiglu_backward", "rows": 8192, "d": 2048},
    ]


def _spread(rng, low, high, step=1):
    """A multiple of `step` from [low, high], spread evenly over its logarithm."""
    n = math.exp(rng.uniform(math.log(low), math.log(high + 0.999)))
    return max(low, min(high, int(n) // step * step)) if n >= step else low


def draw(rng):
    op = rng.choice(["quantize_rows", "quantize_weights", "gemm", "grouped_gemm", "wgrad", "swiglu", "swiglu_backward"])
    if op == "quantize_rows":
        return {"op": op, "rows": _spread(rng, 1, 16384), "cols": _spread(rng, 128, 8192, 16)}
    if op == "quantize_weights":
        return {"op": op, "groups": _spread(rng, 1, 16), "rows": _spread(rng, 256, 4096, 16),
                "cols": _spread(rng, 256, 4096, 16)}
    if op == "gemm":
        return {"op": op, "m": _spread(rng, 1, 8192), "n": _spread(rng, 256, 16384, 16),
                "k": _spread(rng, 256, 8192, 16)}
    if op == "grouped_gemm":
        return {"op": op, "groups": _spread(rng, 2, 64), "m": _spread(rng, 1, 8192),
                "n": _spread(rng, 256, 4096, 16), "k": _spread(rng, 256, 4096, 16)}
    if op == "wgrad":
        return {"op": op, "groups": _spread(rng, 1, 16), "m": _spread(rng, 16, 16384),
                "n": _spread(rng, 256, 4096, 16), "k": _spread(rng, 256, 2048, 16)}
    return {"op": op, "rows": _spread(rng, 1, 16384), "d": _spread(rng, 128, 4096, 16)}


def _group_sizes(case):
    """Rows per group: uneven popularity, and two groups of eight or more left empty."""
    G, M = case["groups"], case["m"]
    rng = random.Random("%d,%d,%d,%d" % (G, M, case["n"], case["k"]))
    empty = set(rng.sample(range(G), 2)) if G >= 8 else set()
    share = [0.0 if g in empty else math.exp(rng.gauss(0.0, 0.7)) for g in range(G)]
    rows = collections.Counter(rng.choices(range(G), weights=share, k=M))
    return [rows[g] for g in range(G)]


# ---- inputs ------------------------------------------------------------------------------
def _normal(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(torch.bfloat16)


def _activations(gen, rows, cols):
    """Unit normal rows with a few strong channels, as activations have them."""
    channel = 1.0 + 15.0 * (torch.rand(cols, generator=gen, device="cuda") < 0.005).float()
    return (torch.randn(rows, cols, generator=gen, device="cuda") * channel).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    state = {"op": op}
    if op == "quantize_rows":
        state["x"] = _activations(gen, case["rows"], case["cols"])
    elif op == "quantize_weights":
        state["w"] = _normal(gen, case["groups"], case["rows"], case["cols"], std=0.02)
    elif op == "gemm":
        state["a"], state["sa"] = _quantize_rows(_activations(gen, case["m"], case["k"]))
        q, s = _quantize_blocks(_normal(gen, 1, case["n"], case["k"], std=0.02))
        state["bt"], state["sbt"] = q[0], s[0]
    elif op in ("grouped_gemm", "wgrad"):
        sizes = _group_sizes(case)
        ends = torch.tensor([0] + sizes, device="cuda").cumsum(0)
        state["offsets"] = ends.to(torch.int32)
        state["longest"] = max(sizes)  # for the plain form's padding
        if op == "grouped_gemm":
            state["a"], state["sa"] = _quantize_rows(_activations(gen, case["m"], case["k"]))
            state["bt"], state["sbt"] = _quantize_blocks(
                _normal(gen, case["groups"], case["n"], case["k"], std=0.02))
        else:
            state["dy"] = _normal(gen, case["m"], case["n"], std=0.01)
            state["x"] = _activations(gen, case["m"], case["k"])
    else:
        state["gu"] = _normal(gen, case["rows"], 2 * case["d"], std=1.5)
        if op == "swiglu_backward":
            state["dy"] = _normal(gen, case["rows"], case["d"], std=0.01)
    return state


# ---- plain forms ---------------------------------------------------------------------------
def _quantize(x, amax):
    """Codes of x with the scale amax / 448, shaped to broadcast against x."""
    s = amax / torch.full_like(amax, E4M3_MAX)  # by a tensor: a plain number would be a product with 1/448
    t = torch.where(s > 0, x / s, torch.zeros_like(x))
    return t.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), s


def _quantize_rows(x):
    rows, cols = x.shape
    nb = _blocks(cols)
    p = torch.zeros(rows, nb * GROUP, device=x.device)
    p[:, :cols] = x.float()
    p = p.view(rows, nb, GROUP)
    q, s = _quantize(p, p.abs().amax(2, keepdim=True))
    return q.view(rows, -1)[:, :cols].contiguous(), s.view(rows, nb)


def _quantize_blocks(w):
    G, rows, cols = w.shape
    rb, cb = _blocks(rows), _blocks(cols)
    p = torch.zeros(G, rb * GROUP, cb * GROUP, device=w.device)
    p[:, :rows, :cols] = w.float()
    p = p.view(G, rb, GROUP, cb, GROUP)
    q, s = _quantize(p, p.abs().amax((2, 4), keepdim=True))
    return q.view(G, rb * GROUP, cb * GROUP)[:, :rows, :cols].contiguous(), s.view(G, rb, cb)


def _rows_of(q, s):
    """The values that codes with a scale per row and 128 columns stand for."""
    return q.float() * s.repeat_interleave(GROUP, 1)[:, :q.shape[1]]


def _blocks_of(q, s):
    """The values that codes [G, rows, cols] with a scale per 128x128 block stand for."""
    return q.float() * s.repeat_interleave(GROUP, 1).repeat_interleave(GROUP, 2)[:, :q.shape[1], :q.shape[2]]


def _padded(x, offsets, longest):
    """[rows, cols] -> [G, longest, cols] with zeros behind each group's rows, and every row's place there."""
    row = torch.arange(x.shape[0], device=x.device)
    group = torch.searchsorted(offsets[1:].long(), row, right=True)
    place = row - offsets.long()[group]
    p = torch.zeros(offsets.shape[0] - 1, longest, x.shape[1], device=x.device)
    p[group, place] = x
    return p, group, place


def _plain(state):
    op = state["op"]
    if op == "quantize_rows":
        q, s = _quantize_rows(state["x"])
        return {"q": q, "scales": s}
    if op == "quantize_weights":
        q, s = _quantize_blocks(state["w"])
        return {"q": q, "scales": s, "qt": q.transpose(1, 2).contiguous(), "scales_t": s.transpose(1, 2).contiguous()}
    if op == "gemm":
        w = _blocks_of(state["bt"][None], state["sbt"][None])[0]
        return torch.matmul(_rows_of(state["a"], state["sa"]), w.t()).to(torch.bfloat16)
    if op == "grouped_gemm":
        p, group, place = _padded(_rows_of(state["a"], state["sa"]), state["offsets"], state["longest"])
        w = _blocks_of(state["bt"], state["sbt"])
        return torch.bmm(p, w.transpose(1, 2))[group, place].to(torch.bfloat16)
    if op == "wgrad":
        dy = _padded(state["dy"].float(), state["offsets"], state["longest"])[0]
        x = _padded(state["x"].float(), state["offsets"], state["longest"])[0]
        return torch.bmm(dy.transpose(1, 2), x)
    gu = state["gu"].float()
    d = gu.shape[1] // 2
    g, u = gu[:, :d], gu[:, d:]
    sigma = 1.0 / (1.0 + torch.exp(-g))
    if op == "swiglu":
        q, s = _quantize_rows(g * sigma * u)
        return {"q": q, "scales": s}
    dy = state["dy"].float()
    dgu = torch.cat([dy * u * (sigma * (1.0 + g * (1.0 - sigma))), dy * (g * sigma)], 1)
    q, s = _quantize_rows(dgu)
    return {"dgu": dgu.to(torch.bfloat16), "q": q, "scales": s}


# ---- the framework's calls -----------------------------------------------------------------
def _framework(state):
    import fp8_block_scaled_03_amd as fp8bs
    e4m3 = torch.float8_e4m3fn
    op = state["op"]
    if op == "quantize_rows":
        q, s = fp8bs.quantize_tg128(state["x"])
        return {"q": q.view(e4m3), "scales": s}
    if op == "quantize_weights":
        q, s, qt, st = fp8bs.quantize_b128(state["w"], transposed=True)
        return {"q": q.view(e4m3), "scales": s, "qt": qt.view(e4m3), "scales_t": st}
    if op == "gemm":
        return fp8bs.gemm_tg128_nt(state["a"], state["sa"], state["bt"], state["sbt"])
    if op == "grouped_gemm":
        return fp8bs.grouped_gemm_tg128_nt(state["a"], state["sa"], state["bt"], state["sbt"], state["offsets"])
    if op == "wgrad":
        return fp8bs.grouped_wgrad(state["dy"], state["x"], state["offsets"])
    if op == "swiglu":
        q, s = fp8bs.swiglu_quantize_tg128(state["gu"])
        return {"q": q.view(e4m3), "scales": s}
    dgu, q, s = fp8bs.swiglu_backward_quantize_tg128(state["gu"], state["dy"])
    return {"dgu": dgu, "q": q.view(e4m3), "scales": s}


def run(state):
    if own:
        return _framework(state)
    return _plain(state)


# ---- what a pass cannot do without -----------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "quantize_rows":
        r, c = case["rows"], case["cols"]
        return {"bytes": 3 * r * c + 4 * r * _blocks(c), "flops": 2 * r * c}
    if op == "quantize_weights":
        n = case["groups"] * case["rows"] * case["cols"]
        return {"bytes": 4 * n + 8 * case["groups"] * _blocks(case["rows"]) * _blocks(case["cols"]), "flops": 2 * n}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        scales = 4 * _blocks(k) * (m + _blocks(n))
        return {"bytes": m * k + n * k + scales + 2 * m * n, "flops": 2 * m * n * k}
    if op == "grouped_gemm":
        m, n, k = case["m"], case["n"], case["k"]
        live = sum(1 for s in _group_sizes(case) if s)
        scales = 4 * _blocks(k) * (m + live * _blocks(n))
        return {"bytes": m * k + live * n * k + scales + 2 * m * n, "flops": 2 * m * n * k}
    if op == "wgrad":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * (n + k) + 4 * case["groups"] * n * k, "flops": 2 * m * n * k}
    r, d = case["rows"], case["d"]
    if op == "swiglu":
        return {"bytes": 5 * r * d + 4 * r * _blocks(d), "flops": 6 * r * d}
    return {"bytes": 12 * r * d + 4 * r * _blocks(2 * d), "flops": 16 * r * d}


# ---- the definitions in 64 bits --------------------------------------------------------------
def _nearest_e4m3(t):
    """The E4M3 value nearest to t (64 bits, within +-448), ties to the even one."""
    exponent = (torch.frexp(t.abs())[1] - 1).clamp(min=-6).double()
    step = torch.pow(2.0, exponent - 3.0)
    return torch.round(t / step) * step


def _codes64(x, amax):
    s = amax / torch.full_like(amax, E4M3_MAX)
    held = s.float().double()  # the scale as it is stored
    # the quotient is an fp32 one by definition: quotients of bf16 values often lie on a border between two codes
    t = torch.where(held > 0, x / held, torch.zeros_like(x)).float().double()
    return _nearest_e4m3(t.clamp(-E4M3_MAX, E4M3_MAX)), s


def _codes64_of_rows(x):
    parts = [_codes64(p, p.abs().amax(1, keepdim=True)) for p in x.split(GROUP, 1)]
    return torch.cat([p[0] for p in parts], 1), torch.cat([p[1] for p in parts], 1)


def _values64(q, s, rows_per_scale):
    """The values of codes [rows, cols] with a scale per `rows_per_scale` rows and 128 columns."""
    row = torch.arange(q.shape[0], device=q.device) // rows_per_scale
    col = torch.arange(q.shape[1], device=q.device) // GROUP
    return q.double() * s.double()[row][:, col]


def exact(case, seed):
    state = prepare(case, seed)
    op = state["op"]
    if op == "quantize_rows":
        q, s = _codes64_of_rows(state["x"].double())
        return {"q": q, "scales": s}
    if op == "quantize_weights":
        w = state["w"].double()
        bands = []
        for band in w.split(GROUP, 1):
            parts = [_codes64(p, p.abs().amax((1, 2), keepdim=True)) for p in band.split(GROUP, 2)]
            bands.append((torch.cat([p[0] for p in parts], 2), torch.cat([p[1] for p in parts], 2)))
        q = torch.cat([b[0] for b in bands], 1)
        s = torch.cat([b[1] for b in bands], 1)
        return {"q": q, "scales": s, "qt": q.transpose(1, 2), "scales_t": s.transpose(1, 2)}
    if op == "gemm":
        return _values64(state["a"], state["sa"], 1) @ _values64(state["bt"], state["sbt"], GROUP).t()
    if op in ("grouped_gemm", "wgrad"):
        ends = [0]
        for n in _group_sizes(case):
            ends.append(ends[-1] + n)
        if op == "grouped_gemm":
            a = _values64(state["a"], state["sa"], 1)
            return torch.cat([a[b:e] @ _values64(state["bt"][g], state["sbt"][g], GROUP).t()
                              for g, (b, e) in enumerate(zip(ends, ends[1:]))])
        dy, x = state["dy"].double(), state["x"].double()
        return torch.stack([dy[b:e].t() @ x[b:e] for b, e in zip(ends, ends[1:])])
    gu = state["gu"].double()
    g, u = gu.chunk(2, 1)
    silu = g * torch.sigmoid(g)
    if op == "swiglu":
        q, s = _codes64_of_rows(silu * u)
        return {"q": q, "scales": s}
    dy = state["dy"].double()
    slope = torch.sigmoid(g) + silu * torch.sigmoid(-g)
    dgu = torch.cat([dy * u * slope, dy * silu], 1)
    q, s = _codes64_of_rows(dgu)
    return {"dgu": dgu, "q": q, "scales": s}
