"""The 8-bit floating point layers that stand beside the 1-bit ones, and the
rows of a mixture-of-experts layer on their way to the experts and back, with
what each is measured on:

- "quantize": rows (or 128 x 128 blocks of weights) to 8 bits with a power of
  two for each 128 positions;
- "linear": the product of 8-bit weights (a scale for each 128 x 128 block)
  with 8-bit activations (a scale for each 128 positions), or with 16-bit ones
  that the call quantizes, with bias, activation or gate, and residual;
- "grouped": the same per expert on ragged runs of gathered rows;
- "sort", "join", "grad": rows sorted by expert, back with the router's weights
  (or without them, which is the gradient of the sort), and the gradients of
  the weighted join.

A case is run in plain torch operations in 32 bits (`own` false) or through
the library's entry points (`own` true).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16,
          "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1}
#: The largest finite value of each 8-bit type.
TOPS = {"e4m3": 448.0, "e5m2": 57344.0}


# ------------------------------------------------------------------ the cases
def _quantize(name, rows, K, dtype, to="e4m3", blocks=False):
    return {"name": name, "op": "quantize", "rows": rows, "K": K, "dtype": dtype, "to": to, "blocks": blocks}


def _linear(name, m, K, B, dtype, out, scales, act="none", gated=False, bias=False, residual=False,
            outliers=False):
    return {"name": name, "op": "linear", "m": m, "K": K, "B": B, "dtype": dtype, "out": out, "scales": scales,
            "act": act, "gated": gated, "bias": bias, "residual": residual, "outliers": outliers}


def _grouped(name, E, k, T, m, K, dtype, out, scales, act="none", gated=False, bias=False, skew=1.0):
    return {"name": name, "op": "grouped", "E": E, "k": k, "T": T, "m": m, "K": K, "dtype": dtype, "out": out,
            "scales": scales, "act": act, "gated": gated, "bias": bias, "skew": skew, "residual": False}


def _rows(name, op, E, k, T, n, dtype, weighted=True, residual=False, padded=0.0):
    return {"name": name, "op": op, "E": E, "k": k, "T": T, "n": n, "dtype": dtype, "weighted": weighted,
            "residual": residual, "padded": padded}


def listed():
    return [
        # the activations of a decoding batch: latency
        _quantize("quantize-batch", 24, 4096, "bf16"),
        # a long prompt on its way into an 8B-class down projection
        _quantize("quantize-prompt", 4096, 14336, "f16"),
        # one new token through an attention output projection, residual added
        _linear("token-residual", 4096, 4096, 1, "bf16", "bf16", "e8m0", residual=True),
        # sixteen sequences through an 8B-class gate and up projection, scales as a checkpoint holds them
        _linear("tokens16-gated", 28672, 4096, 16, "bf16", "bf16", "f32", act="silu", gated=True, outliers=True),
        # a prompt of 512 tokens through 8192 x 8192, quantized before, everything the epilogue offers
        _linear("prompt512", 8192, 8192, 512, "e4m3", "f16", "f32", act="gelu", bias=True, residual=True),
        # sizes that no tile divides, gradients in e5m2, float32 results
        _linear("grad-odd", 1281, 5125, 777, "e5m2", "f32", "e8m0"),
        # a long prompt through the gate and up projection: the largest
        _linear("prompt4096-gated", 28672, 4096, 4096, "bf16", "bf16", "e8m0", act="silu", gated=True),
        # a decoding batch of 24 tokens into 8 of 64 experts
        _grouped("experts-batch", 64, 8, 24, 2816, 2048, "bf16", "bf16", "f32", act="silu", gated=True),
        # a prompt of 2048 tokens into 64 experts, unevenly loaded, rows quantized before
        _grouped("experts-prompt", 64, 8, 2048, 2816, 2048, "e4m3", "bf16", "e8m0", act="silu", gated=True),
        # a decoding batch back from its experts: latency
        _rows("join-batch", "join", 64, 8, 24, 2048, "bf16", residual=True),
        # a prompt's rows sorted by expert, some of its tokens padding
        _rows("sort-prompt", "sort", 64, 8, 4096, 2048, "bf16", padded=0.03),
        # the gradients of a prompt's join
        _rows("join-grad-prompt", "grad", 64, 8, 2048, 2048, "bf16"),
    ]


#: What a drawn case may cost at most: the largest listed products, weights held in 32 bits by the plain form, rows moved.
MOST_FLOPS = 2 * 28672 * 4096 * 4096
MOST_WEIGHTS = 64 * 2816 * 2048
MOST_VALUES = 4096 * 8 * 2048


def _log(rng, low, high, step=1):
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step
    return min(max(v, low), high)


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "linear", "grouped", "grouped", "sort", "join", "grad"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "quantize":
        K = _log(rng, 128, 28672)
        rows = min(_log(rng, 1, 16384), 4096 * 14336 // K)
        case = _quantize("", rows, K, rng.choice(["f32", "f16", "bf16"]), rng.choice(["e4m3", "e4m3", "e5m2"]))
        if rng.random() < 0.25:
            case["to"], case["blocks"] = "e4m3", True
    elif op in ("linear", "grouped"):
        dtype = rng.choice(["f16", "bf16", "e4m3", "e4m3", "e5m2"])
        out = rng.choice(["f16", "bf16", "f32"])
        scales = rng.choice(["e8m0", "f32"])
        act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
        gated = flag()
        step = 2 if gated else 1
        if op == "linear":
            B, m, K = _log(rng, 1, 4096), _log(rng, 512, 28672, step), _log(rng, 512, 28672)
            K = max(512, min(K, MOST_FLOPS // (2 * m * B), MOST_WEIGHTS // m))
            case = _linear("", m, K, B, dtype, out, scales, act, gated, flag(), flag(), flag())
        else:
            E = _log(rng, 4, 128)
            k, T = rng.randint(1, min(E, 8)), _log(rng, 1, 2048)
            m, K = _log(rng, 512, 8192, step), _log(rng, 512, 8192)
            m = max(512, min(m, MOST_WEIGHTS // (512 * E) // 2 * 2))
            K = max(512, min(K, MOST_FLOPS // (4 * m * T * k), MOST_WEIGHTS // (m * E)))
            case = _grouped("", E, k, T, m, K, dtype, out, scales, act, gated, flag(), rng.choice([0.0, 1.0]))
    else:
        E = _log(rng, 4, 512)
        k, n = rng.randint(1, min(E, 10)), _log(rng, 512, 8192)
        T = max(1, min(_log(rng, 1, 16384), MOST_VALUES // (k * n)))
        dtype = rng.choice(["f32", "f16", "bf16"] + (["e4m3"] if op == "sort" else []))
        case = _rows("", op, E, k, T, n, dtype, op == "grad" or flag(), op == "join" and flag(),
                     rng.choice([0.0, 0.1]))
    del case["name"]
    return case


def _blocks(n):
    return (n + 127) // 128


def work(case):
    """Every input read once and every output written once; of the experts, those that some token goes to (even loads)."""
    op = case["op"]
    if op == "quantize":
        rows, K = case["rows"], case["K"]
        held = _blocks(rows) if case["blocks"] else rows
        return {"bytes": rows * K * (SIZES[case["dtype"]] + 1) + held * _blocks(K), "flops": 2 * rows * K}
    if op in ("linear", "grouped"):
        m, K = case["m"], case["K"]
        width = m // 2 if case["gated"] else m
        matrix = m * K + _blocks(m) * _blocks(K) * (1 if case["scales"] == "e8m0" else 4) + (4 * m if case["bias"] else 0)
        if op == "linear":
            tokens, rows, matrices, extra = case["B"], case["B"], 1, 0
        else:
            T, E, k = case["T"], case["E"], case["k"]
            tokens, rows, matrices, extra = T, T * k, E * (1.0 - (1.0 - k / E) ** T), 4 * (E + 1) + 4 * T * k
        held = K * SIZES[case["dtype"]] + (_blocks(K) if case["dtype"] in TOPS else 0)
        moved = matrices * matrix + tokens * held + rows * width * SIZES[case["out"]] + extra
        if case["residual"]:
            moved += rows * width * SIZES[case["out"]]
        return {"bytes": int(moved), "flops": 2 * rows * m * K}
    T, k, n, size = case["T"], case["k"], case["n"], SIZES[case["dtype"]]
    rows = T * k
    moved = (T + rows) * n * size + 4 * rows + (4 * rows if case["weighted"] and op != "sort" else 0)
    if op == "grad":       # dy and z read, dz and the weights' gradients written, positions, weights and rows read
        return {"bytes": moved + rows * n * size + 8 * rows, "flops": 3 * rows * n}
    return {"bytes": moved + (T * n * size if case["residual"] else 0), "flops": 2 * rows * n if op == "join" else 0}


# ------------------------------------------------------------------ 8 bits in plain operations
def _power(e):
    """2^e in float32 for integers -126 <= e <= 127."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _exponents(largest, to):
    """The smallest e with largest <= top 2^e, 0 for zeros."""
    part, e = torch.frexp(largest)            # largest = part 2^e, part in [1/2, 1); top = 7/8 2^9 or 7/8 2^16
    e = e - (9 if to == "e4m3" else 16) + (part > 0.875)
    return torch.where(largest > 0, e, torch.zeros_like(e))


def _padded(x, *multiples):
    pads = []
    for size, by in zip(reversed(x.shape), reversed(multiples)):
        pads += [0, -size % by]
    return torch.nn.functional.pad(x, pads)


def _to_rows(x, to):
    """x [rows][K] -> values [rows][K in whole 128], exponents uint8 [rows][blocks]."""
    g = _padded(x.float(), 1, 128).unflatten(-1, (-1, 128))
    e = _exponents(g.abs().amax(-1), to)
    values = (g * _power(-e).unsqueeze(-1)).flatten(-2).to(DTYPES[to])
    return values, (e + 127).to(torch.uint8)


def _block_view(w):
    """[..][m][K], both in whole 128, -> [..][m / 128][128][K / 128][128]."""
    return w.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))


def _to_blocks(w, to="e4m3"):
    """w [..][m][K] -> values [..][m][K in whole 128], exponents uint8 [..][ceil(m / 128)][K / 128]."""
    m = w.shape[-2]
    g = _block_view(_padded(w.float(), 128, 128))
    e = _exponents(g.abs().amax(-1).amax(-2), to)
    values = (g * _power(-e)[..., :, None, :, None]).flatten(-4, -3).flatten(-2)[..., :m, :]
    return values.to(DTYPES[to]).contiguous(), (e + 127).to(torch.uint8)


def _from_rows(values, exps):
    return (values.float().unflatten(-1, (-1, 128)) * _power(exps.int() - 127).unsqueeze(-1)).flatten(-2)


def _from_blocks(values, scales):
    m = values.shape[-2]
    s = scales if scales.dtype == torch.float32 else _power(scales.int() - 127)
    s = s.repeat_interleave(128, dim=-2)[..., :m, :]
    return (values.float().unflatten(-1, (-1, 128)) * s.unsqueeze(-1)).flatten(-2)


# ------------------------------------------------------------------ the inputs
def _values(gen, rows, K, outliers=False):
    a = torch.randn(rows, K, generator=gen, device="cuda")
    if outliers:  # about one position in a hundred twenty times the others, the same for every token
        a *= torch.where(torch.rand(K, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    return a


def _with_pitch(exps):
    """Exponents whose rows lie whole words apart, as the library keeps them."""
    rows, blocks = exps.shape[-2:]
    held = torch.full((*exps.shape[:-1], blocks + -blocks % 4), 127, dtype=torch.uint8, device=exps.device)
    held[..., :blocks] = exps
    return held[..., :blocks]


def _weights(gen, lead, m, K, kind):
    """8-bit weights as a model holds them, matrix by matrix, and their scales."""
    values, scales = [], []
    for _ in range(lead or 1):
        w = torch.randn(m, K, generator=gen, device="cuda") * 0.02 * (torch.rand(m, 1, generator=gen, device="cuda") + 0.5)
        if kind == "e8m0":
            v, s = _to_blocks(w)
        else:                               # any scale: the block's largest value becomes 448
            g = _block_view(_padded(w, 128, 128))
            s = g.abs().amax(-1).amax(-2) / 448.0
            s = torch.where(s > 0, s, torch.ones_like(s))
            v = (g / s[:, None, :, None]).clamp(-448.0, 448.0).flatten(-4, -3).flatten(-2)[:m].to(DTYPES["e4m3"])
        values.append(v)
        scales.append(s)
    values, scales = (torch.stack(values), torch.stack(scales)) if lead else (values[0], scales[0])
    return values.contiguous(), _with_pitch(scales) if kind == "e8m0" else scales.contiguous()


def _routing(gen, T, E, k, skew, padded):
    """What the router gives: weights [T][k], sorted positions [T][k], tokens [T k], run ends [E + 1]."""
    logits = torch.randn(T, E, generator=gen, device="cuda") * 1.5 + torch.randn(E, generator=gen, device="cuda") * skew
    top, ids = torch.topk(logits, k, dim=1)
    weight = torch.softmax(top, dim=1)
    live = (torch.rand(T, 1, generator=gen, device="cuda") >= padded).expand(T, k)
    flat = torch.where(live, ids, torch.full_like(ids, E)).reshape(-1)
    key, perm = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda")).to(torch.int32)
    pos = torch.empty_like(perm)
    pos[perm] = torch.arange(T * k, device="cuda")
    pos = torch.where(flat < E, pos, torch.full_like(pos, -1)).reshape(T, k).to(torch.int32)
    rows = torch.where(key < E, torch.div(perm, k, rounding_mode="floor"), torch.full_like(perm, -1)).to(torch.int32)
    return torch.where(live, weight, torch.zeros_like(weight)).contiguous(), pos, rows, offsets


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": dict(case)}
    op = case["op"]
    if op == "quantize":
        x = _values(gen, case["rows"], case["K"], not case["blocks"])
        st["x"] = (x * 0.02 if case["blocks"] else x).to(DTYPES[case["dtype"]])
        return st
    if op in ("linear", "grouped"):
        m, K = case["m"], case["K"]
        lead = case["E"] if op == "grouped" else 0
        st["w"], st["scales"] = _weights(gen, lead, m, K, case["scales"])
        st["bias"] = torch.randn((lead, m) if lead else (m,), generator=gen, device="cuda") if case["bias"] else None
        if op == "grouped":
            _, _, st["rows"], st["offsets"] = _routing(gen, case["T"], lead, case["k"], case["skew"], 0.0)
            st["cap"] = int(st["offsets"].diff().max())     # the plain form pads each expert's rows to this
            held, tokens = case["T"], case["T"] * case["k"]
        else:
            held, tokens = case["B"], case["B"]
        a = _values(gen, held, K, case.get("outliers", False))
        if case["dtype"] in TOPS:
            st["a"], exps = _to_rows(a, case["dtype"])
            st["exps"] = _with_pitch(exps)
        else:
            st["a"] = a.to(DTYPES[case["dtype"]])
        width = m // 2 if case["gated"] else m
        st["residual"] = (torch.randn(tokens, width, generator=gen, device="cuda").to(DTYPES[case["out"]])
                          if case["residual"] else None)
        return st
    T, k, n = case["T"], case["k"], case["n"]
    st["weight"], st["pos"], st["rows"], _ = _routing(gen, T, case["E"], k, 1.0, case["padded"])
    if op == "sort":
        st["x"] = torch.randn(T, n, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        return st
    st["z"] = torch.randn(T * k, n, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
    extra = op == "grad" or case["residual"]
    st["dy" if op == "grad" else "residual"] = (
        torch.randn(T, n, generator=gen, device="cuda").to(DTYPES[case["dtype"]]) if extra else None)
    return st


# ------------------------------------------------------------------ the plain forms
def _activated(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _expert_rows(st, a, w):
    """z [R][m]: row r of the sorted order through its own expert's matrix."""
    case, off = st["case"], st["offsets"].long()
    R = case["T"] * case["k"]
    r = torch.arange(R, device=a.device)
    expert = torch.searchsorted(off[1:], r, right=True)
    source = st["rows"].long()
    if R < case["E"]:          # few rows: each row's own matrix
        z = torch.bmm(w[expert], a[source].unsqueeze(-1)).squeeze(-1)
    else:                      # each expert's rows padded to the longest run
        at = off[:-1, None] + torch.arange(st["cap"], device=a.device)
        x = torch.where((at < off[1:, None]).unsqueeze(-1), a[source[at.clamp(max=R - 1)]], 0.0)
        z = torch.bmm(w, x.transpose(1, 2).contiguous()).transpose(1, 2)[expert, r - off[expert]]
    return z if st["bias"] is None else z + st["bias"][expert]


def _products(st):
    case = st["case"]
    a = _from_rows(st["a"], st["exps"]) if "exps" in st else _from_rows(*_to_rows(st["a"], "e4m3"))
    w = _from_blocks(st["w"], st["scales"])
    if case["op"] == "grouped":
        z = _expert_rows(st, a, w)
    else:
        z = torch.matmul(a, w.t())
        z = z if st["bias"] is None else z + st["bias"]
    if case["gated"]:
        half = case["m"] // 2
        y = _activated(z[:, :half], case["act"]) * z[:, half:]
    else:
        y = _activated(z, case["act"])
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(DTYPES[case["out"]])


def _moved(st):
    """sort, join and grad."""
    case, rows, pos = st["case"], st["rows"].long(), st["pos"].long()
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "sort":
        x = st["x"].float()
        return torch.where((rows >= 0)[:, None], x[rows.clamp(min=0)], 0.0).to(dtype)
    z, live = st["z"].float(), pos >= 0
    picked = torch.where(live.unsqueeze(-1), z[pos.clamp(min=0)], 0.0)          # [T][k][n]
    if case["op"] == "join":
        y = (picked * st["weight"].unsqueeze(-1) if case["weighted"] else picked).sum(1)
        return (y if st["residual"] is None else y + st["residual"].float()).to(dtype)
    dy = st["dy"].float()
    dz = torch.zeros(z.shape[0] + 1, z.shape[1], device=z.device)                # the last row takes what goes nowhere
    dz[torch.where(live, pos, z.shape[0]).flatten()] = (st["weight"].unsqueeze(-1) * dy.unsqueeze(1)).flatten(0, 1)
    return {"dz": dz[:-1].to(dtype), "dweight": (picked * dy.unsqueeze(1)).sum(-1)}


def _plain(st):
    case = st["case"]
    if case["op"] == "quantize":
        values, exps = _to_blocks(st["x"], case["to"]) if case["blocks"] else _to_rows(st["x"], case["to"])
        return {"values": values, "exps": exps}
    return _products(st) if case["op"] in ("linear", "grouped") else _moved(st)


def _own(st):
    from bit_lifted_gemv_amd import lq
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        if case["blocks"]:
            q = lq.quantize8_blocks(st["x"])
            return {"values": q.values, "exps": q.scales}
        q = lq.quantize8(st["x"], DTYPES[case["to"]])
        return {"values": q.values, "exps": q.exps}
    if op in ("linear", "grouped"):
        w = lq.Blocks8(st["w"], st["scales"])
        a = lq.Rows8(st["a"], st["exps"]) if "exps" in st else st["a"]
        out = DTYPES[case["out"]]
        if op == "linear":
            return lq.gemm8(w, a, bias=st["bias"], act=case["act"], gated=case["gated"],
                            residual=st["residual"], out_dtype=out)
        return lq.gemm8_grouped(w, a, st["offsets"], rows=st["rows"], bias=st["bias"], act=case["act"],
                                gated=case["gated"], out_dtype=out)
    if op == "sort":
        return lq.sort_rows(st["x"], st["rows"])
    if op == "join":
        return lq.join_rows(st["z"], st["pos"], st["weight"] if case["weighted"] else None, residual=st["residual"])
    dz, dweight = lq.join_rows_grad(st["dy"], st["z"], st["pos"], st["weight"], st["rows"])
    return {"dz": dz, "dweight": dweight}


def run(state):
    """One pass.  quantize: per row and 128 positions (or per 128 x 128 block) the smallest power of two that brings
    the largest value within the 8-bit type, and the values divided by it and rounded to nearest even;
    linear: z = sum over blocks of scale(weights) scale(activations) (weights . activations) + bias, act(z) + residual,
    or act(z_i) z_{i + m/2} + residual; 16-bit activations are quantized to e4m3 first;
    grouped: row r of the sorted order is token rows[r] through the expert e with offsets[e] <= r < offsets[e + 1];
    sort: row r is token rows[r], zeros for -1;
    join: token t gets sum_j weight[t][j] z[pos[t][j]] + residual (weight 1 without weights; nothing for -1);
    grad: dz[pos[t][j]] = weight[t][j] dy[t] (zeros in rows that no token has), dweight[t][j] = dy[t] . z[pos[t][j]]."""
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definition in 64 bits
#: Double-precision products beyond this take too long.
EXACT_FLOPS = 5e14


def _rounded(y, to):
    """float64 values to the nearest of the 8-bit type's, ties to the even one."""
    bits, lowest = (3, -6) if to == "e4m3" else (2, -14)
    exponent = torch.floor(torch.log2(y.abs().clamp(min=2.0**-60)))
    exponent = torch.where(torch.exp2(exponent) > y.abs(), exponent - 1, exponent)      # log2 may round up
    unit = torch.exp2(exponent.clamp(min=lowest) - bits)
    return torch.round(y / unit) * unit


def _scale(largest, to):
    """2^e, e the smallest integer with largest <= top 2^e (1 for zeros), float64."""
    ratio = largest.double() / TOPS[to]
    e = torch.ceil(torch.log2(ratio.clamp(min=1e-300)))
    e = torch.where(torch.exp2(e - 1) >= ratio, e - 1, e)
    e = torch.where(torch.exp2(e) < ratio, e + 1, e)
    return torch.where(largest > 0, torch.exp2(e), torch.ones_like(e))


def _exact_rows(x, to):
    """The 8-bit values of rows and the scale of each position, float64."""
    K = x.shape[1]
    blocks = [x[:, lo:lo + 128].double() for lo in range(0, K, 128)]
    scale = [_scale(b.abs().max(1, keepdim=True).values, to) for b in blocks]
    values = torch.cat([_rounded(b / s, to) for b, s in zip(blocks, scale)], dim=1)
    return values, torch.cat([s.expand_as(b) for b, s in zip(blocks, scale)], dim=1)


def _exact_act(z, act):
    z = z.double()
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":   # (1 + tanh u) / 2 = 1 / (1 + exp(-2 u))
        return z * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z**3))
    return z


def _exact_product(case, values, scales, bias, a):
    """One matrix: a [n][K] in float64, weights expanded a block of rows at a time."""
    K, m = a.shape[1], case["m"]
    parts = []
    for lo in range(0, m, 128):
        w = values[lo:lo + 128, :K].double()
        s = scales[lo // 128].double()
        s = s if scales.dtype == torch.float32 else torch.exp2(s - 127.0)
        parts.append(a @ (w * s.repeat_interleave(128)[:K]).T)
    z = torch.cat(parts, dim=1)
    z = z if bias is None else z + bias.double()
    if case["gated"]:
        return _exact_act(z[:, :m // 2], case["act"]) * z[:, m // 2:]
    return _exact_act(z, case["act"])


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        if not case["blocks"]:
            values, _ = _exact_rows(st["x"], case["to"])
        else:
            x = st["x"].double()
            values = torch.empty_like(x)
            for lo in range(0, case["rows"], 128):
                for at in range(0, case["K"], 128):
                    b = x[lo:lo + 128, at:at + 128]
                    values[lo:lo + 128, at:at + 128] = _rounded(b / _scale(b.abs().max(), case["to"]), case["to"])
        return {"values": torch.nn.functional.pad(values, (0, -case["K"] % 128)), "exps": None}
    if op in ("linear", "grouped"):
        if work(case)["flops"] > EXACT_FLOPS:
            return None
        K = case["K"]
        if "exps" in st:
            a = st["a"].double()[:, :K] * torch.exp2(st["exps"].double() - 127.0).repeat_interleave(128, dim=1)[:, :K]
        else:
            values, scale = _exact_rows(st["a"], "e4m3")
            a = values * scale
        if op == "linear":
            y = _exact_product(case, st["w"], st["scales"], st["bias"], a)
        else:
            ends = st["offsets"].tolist()
            y = torch.cat([_exact_product(case, st["w"][e], st["scales"][e], None if st["bias"] is None else st["bias"][e],
                                          a[st["rows"][ends[e]:ends[e + 1]].long()])
                           for e in range(case["E"]) if ends[e + 1] > ends[e]])
        return y if st["residual"] is None else y + st["residual"].double()
    T, k, n = case["T"], case["k"], case["n"]
    if op == "sort":
        x = torch.cat([st["x"].double(), torch.zeros(1, n, device="cuda", dtype=torch.float64)])
        return x[st["rows"].long()]                        # -1 is the row of zeros
    z = torch.cat([st["z"].double(), torch.zeros(1, n, device="cuda", dtype=torch.float64)])
    if op == "join":
        y = torch.zeros(T, n, device="cuda", dtype=torch.float64)
        for j in range(k):
            row = z[st["pos"][:, j].long()]
            y += row * st["weight"][:, j:j + 1].double() if case["weighted"] else row
        return y if st["residual"] is None else y + st["residual"].double()
    dy, dz = st["dy"].double(), torch.zeros_like(z)
    dweight = torch.zeros(T, k, device="cuda", dtype=torch.float64)
    for j in range(k):
        p = st["pos"][:, j].long()
        dweight[:, j] = (dy * z[p]).sum(1)
        dz[p] = st["weight"][:, j:j + 1].double() * dy     # -1 goes to the last row, dropped
    return {"dz": dz[:-1], "dweight": dweight}
