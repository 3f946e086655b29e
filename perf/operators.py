"""The products around a lifted 1-bit layer that a language model needs besides
lq_gemv and lq_gemm, with what each is measured on:

- "linear": the product with bias, activation (gated or not) and residual in
  its epilogue, from one token to long prompts;
- "grouped": the products of a mixture-of-experts layer, one 1-bit matrix per
  expert and ragged runs of rows (rows gathered from the tokens on the way in);
- "join": the same products on the way out, each token's expert rows added
  with the router's weights, and the residual;
- "route": the router's choice of experts and the sorted order of the rows.

A case is run in plain torch operations in 32 bits (`own` false) or through
the library's entry points (`own` true).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------ the cases
def _linear(name, m, K, B, dtype, out, act="none", gated=False, bias=False, residual=False,
            outliers=False):
    return {"name": name, "op": "linear", "m": m, "K": K, "B": B, "dtype": dtype, "out": out,
            "act": act, "gated": gated, "bias": bias, "residual": residual, "outliers": outliers}


def _experts(name, op, E, k, T, m, K, dtype, act="none", gated=False, bias=False, residual=False,
             skew=1.0):
    return {"name": name, "op": op, "E": E, "k": k, "T": T, "m": m, "K": K, "dtype": dtype,
            "out": dtype, "act": act, "gated": gated, "bias": bias, "residual": residual,
            "skew": skew}


def _route(name, T, E, k, dtype, renorm, padded):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "renorm": renorm,
            "padded": padded}


def listed():
    return [
        # one new token through an attention output projection (4096 x 4096 at 20/8), residual added
        _linear("token-residual", 4096, 10240, 1, "bf16", "bf16", residual=True),
        # five sequences in flight through a 70B-class down projection (8192 x 28672 at 19/8)
        _linear("tokens5-down", 8192, 68096, 5, "f16", "f16", residual=True),
        # sixteen sequences through an 8B-class gate and up projection (2 x 14336 rows of 4096 at 16/8)
        _linear("tokens16-gated", 28672, 8192, 16, "bf16", "bf16", act="silu", gated=True, outliers=True),
        # a prompt of 512 tokens through 8192 x 8192 at 40/16, everything the epilogue offers
        _linear("prompt512", 8192, 20480, 512, "f16", "f16", act="gelu", bias=True, residual=True),
        # sizes that no tile divides, float32 results
        _linear("prompt-odd", 1281, 5128, 777, "f16", "f32", act="relu", bias=True),
        # a long prompt through the gate and up projection: the largest
        _linear("prompt4096-gated", 28672, 8192, 4096, "bf16", "bf16", act="silu", gated=True),
        # one new token to 8 of 64 experts (2 x 1408 rows of 2048 at 16/8): latency
        _experts("experts-token", "grouped", 64, 8, 1, 2816, 4096, "bf16", act="silu", gated=True),
        # a decoding batch of 24 tokens on its way out of the experts
        _experts("join-batch", "join", 64, 8, 24, 2048, 2816, "bf16", residual=True),
        # a prompt of 2048 tokens into 64 experts, unevenly loaded
        _experts("experts-prompt", "grouped", 64, 8, 2048, 2816, 4096, "bf16", act="silu", gated=True),
        # few large experts: 1500 tokens out of 2 of 8 (4096 x 14336 at 16/8), with a bias each
        _experts("join-prompt", "join", 8, 2, 1500, 4096, 28672, "f16", bias=True, residual=True),
        # the router of a decoding batch
        _route("route-batch", 24, 64, 8, "f32", True, 0.0),
        # the router of a long prompt batch with padding tokens that go to no expert
        _route("route-prompt", 16384, 256, 8, "bf16", True, 0.03),
    ]


#: What a drawn case may cost at most: the largest listed one's products, and the largest signs held in 32 bits.
MOST_FLOPS = 2 * 28672 * 8192 * 4096
MOST_SIGNS = 28672 * 8192 * 4


def _log(rng, low, high, step=1):
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high))) / step)) * step
    return min(max(v, low), high)


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "join", "route"])
    dtype = rng.choice(["f16", "bf16"])
    act = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"])
    flag = lambda: rng.random() < 0.5  # noqa: E731
    if op == "route":
        E = _log(rng, 4, 512)
        return {k: v for k, v in _route("", _log(rng, 1, 16384), E, rng.randint(1, min(E, 10)),
                                        rng.choice(["f32", "f16", "bf16"]), flag(),
                                        rng.choice([0.0, 0.1])).items() if k != "name"}
    gated = op != "join" and flag()
    step = 2 if gated else 1
    if op == "linear":
        B, m = _log(rng, 1, 4096), _log(rng, 512, 28672, step)
        K = _log(rng, 1024, 68096, 8)
        K = max(1024, min(K, MOST_FLOPS // (2 * m * B) // 8 * 8, MOST_SIGNS // m // 8 * 8))
        case = _linear("", m, K, B, dtype, rng.choice([dtype, dtype, "f32"]), act, gated, flag(),
                       flag(), flag())
    else:
        E = _log(rng, 4, 128)
        k, T = rng.randint(1, min(E, 8)), _log(rng, 1, 2048)
        m, K = _log(rng, 512, 8192, step), _log(rng, 1024, 28672, 8)
        K = max(1024, min(K, MOST_FLOPS // (4 * m * T * k) // 8 * 8, MOST_SIGNS // (m * E) // 8 * 8))
        case = _experts("", op, E, k, T, m, K, dtype, act if op == "grouped" else "none", gated,
                        flag(), op == "join" and flag(), rng.choice([0.0, 1.0]))
    del case["name"]
    return case


def work(case):
    """Every input read once and every output written once; of the experts, those that some token goes to (even loads)."""
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * SIZES[case["dtype"]] + T + T * k * 16 + 4 * (E + 1), "flops": 3 * T * E}
    m, K = case["m"], case["K"]
    width = m // 2 if case["gated"] else m
    matrix = m * ((K + 7) // 8) + 4 * m + (4 * m if case["bias"] else 0)
    if case["op"] == "linear":
        rows, held, tokens, matrices = case["B"], case["B"], case["B"], 1
        extra = 0
    else:
        T, E, k = case["T"], case["E"], case["k"]
        rows, matrices = T * k, E * (1.0 - (1.0 - k / E) ** T)
        held, tokens = (T, rows) if case["op"] == "grouped" else (rows, T)
        extra = 4 * (E + 1) + (4 * rows if case["op"] == "grouped" else 8 * rows)
    moved = matrices * matrix + 2 * held * K + tokens * width * SIZES[case["out"]] + extra
    if case["residual"]:
        moved += tokens * width * SIZES[case["out"]]
    return {"bytes": int(moved), "flops": 2 * rows * m * K}


# ------------------------------------------------------------------ the inputs
def _signs(gen, *shape):
    """Packed words of random signs, a row's words rounded up to whole 128-byte lines."""
    *lead, K = shape
    ldw = ((K + 31) // 32 + 31) // 32 * 32
    return torch.randint(-2**31, 2**31, (*lead, ldw), generator=gen, device="cuda", dtype=torch.int64).to(torch.int32)


def _values(gen, rows, K, dtype, outliers=False):
    a = torch.randn(rows, K, generator=gen, device="cuda")
    if outliers:  # about one position in a hundred twenty times the others, the same for every token
        a *= torch.where(torch.rand(K, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    return a.to(DTYPES[dtype])


def _logits(gen, T, E, skew):
    """Router logits: some experts are liked more than others by every token."""
    liked = torch.randn(E, generator=gen, device="cuda") * skew
    return torch.randn(T, E, generator=gen, device="cuda") * 1.5 + liked


def _routing(logits, k, valid, renorm):
    """The router in plain operations: see run()."""
    T, E = logits.shape
    x = logits.float()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    top = torch.gather(x, 1, order)
    p = torch.exp(top - top[:, :1])
    total = p.sum(1, keepdim=True) if renorm else torch.exp(x - top[:, :1]).sum(1, keepdim=True)
    weight = p / total
    if valid is not None:
        live = valid.bool()[:, None]
        order = torch.where(live, order, torch.full_like(order, E))
        weight = torch.where(live, weight, torch.zeros_like(weight))
    flat = order.reshape(-1)
    key, perm = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(key, torch.arange(E + 1, device=key.device)).to(torch.int32)
    pos = torch.empty_like(perm)
    pos[perm] = torch.arange(T * k, device=perm.device)
    pos = torch.where(flat < E, pos, torch.full_like(pos, -1)).reshape(T, k)
    rows = torch.where(key < E, torch.div(perm, k, rounding_mode="floor"), torch.full_like(perm, -1))
    ids = torch.where(order < E, order, torch.full_like(order, -1))
    return {"ids": ids.to(torch.int32), "weight": weight, "pos": pos.to(torch.int32),
            "rows": rows.to(torch.int32), "offsets": offsets}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": dict(case)}
    if case["op"] == "route":
        st["logits"] = _logits(gen, case["T"], case["E"], 1.0).to(DTYPES[case["dtype"]])
        st["valid"] = (torch.rand(case["T"], generator=gen, device="cuda") >= case["padded"]).to(torch.uint8) if case["padded"] else None
        return st
    m, K = case["m"], case["K"]
    lead = (m,) if case["op"] == "linear" else (case["E"], m)
    st["w"] = _signs(gen, *lead, K)
    st["s"] = torch.rand(*lead, generator=gen, device="cuda") * 0.02 + 0.01
    st["bias"] = torch.randn(*lead, generator=gen, device="cuda") if case["bias"] else None
    if case["op"] == "linear":
        held, tokens = case["B"], case["B"]
    else:
        T, k = case["T"], case["k"]
        r = _routing(_logits(gen, T, case["E"], case["skew"]), k, None, True)
        st["offsets"], st["rows"], st["pos"], st["weight"] = r["offsets"], r["rows"], r["pos"], r["weight"]
        st["cap"] = int(r["offsets"].diff().max())   # the plain form pads each expert's rows to this
        held, tokens = (T, T * k) if case["op"] == "grouped" else (T * k, T)
    st["a"] = _values(gen, held, K, case["dtype"], case.get("outliers", False))
    width = m // 2 if case["gated"] else m
    st["residual"] = torch.randn(tokens, width, generator=gen, device="cuda").to(DTYPES[case["out"]]) if case["residual"] else None
    return st


# ------------------------------------------------------------------ the plain forms
def _unpacked(w, K):
    """Packed words [..][ldw] -> signs [..][K], float32."""
    bits = (w.unsqueeze(-1) >> torch.arange(32, device=w.device, dtype=torch.int32)) & 1
    return bits.flatten(-2)[..., :K].float() * 2.0 - 1.0


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


def _finished(z, case):
    """Activation of the product's rows [.., m]: act(z), or act(first half) * second half."""
    if not case["gated"]:
        return _activated(z, case["act"])
    half = case["m"] // 2
    return _activated(z[..., :half], case["act"]) * z[..., half:]


def _expert_rows(st):
    """z [R][m]: row r of the sorted order through its own expert's matrix."""
    case, a, off = st["case"], st["a"].float(), st["offsets"].long()
    R, K = case["T"] * case["k"], case["K"]
    r = torch.arange(R, device=a.device)
    expert = torch.searchsorted(off[1:], r, right=True)
    source = st["rows"].long() if case["op"] == "grouped" else r
    if R < case["E"]:          # few rows: each row's own matrix
        z = torch.bmm(_unpacked(st["w"][expert], K), a[source].unsqueeze(-1)).squeeze(-1)
    else:                      # each expert's rows padded to the longest run
        at = off[:-1, None] + torch.arange(st["cap"], device=a.device)
        x = torch.where((at < off[1:, None]).unsqueeze(-1), a[source[at.clamp(max=R - 1)]], 0.0)
        z = torch.bmm(_unpacked(st["w"], K), x.transpose(1, 2).contiguous())
        z = z.transpose(1, 2)[expert, r - off[expert]]
    z = z * st["s"][expert]
    return z if st["bias"] is None else z + st["bias"][expert]


def _plain(st):
    case = st["case"]
    if case["op"] == "route":
        return _routing(st["logits"], case["k"], st["valid"], case["renorm"])
    if case["op"] == "linear":
        z = torch.matmul(st["a"].float(), _unpacked(st["w"], case["K"]).t()) * st["s"]
        y = _finished(z if st["bias"] is None else z + st["bias"], case)
    elif case["op"] == "grouped":
        y = _finished(_expert_rows(st), case)
    else:
        y = (_expert_rows(st)[st["pos"].long()] * st["weight"].unsqueeze(-1)).sum(1)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return y.to(DTYPES[case["out"]])


def _own(st):
    from bit_lifted_gemv_amd import lq
    case = st["case"]
    if case["op"] == "route":
        r = lq.route(st["logits"], case["k"], valid=st["valid"], renorm=case["renorm"])
        return {"ids": r.ids, "weight": r.weight, "pos": r.pos, "rows": r.rows, "offsets": r.offsets}
    out = DTYPES[case["out"]]
    if case["op"] == "linear":
        return lq.gemm_ep(st["w"], st["s"], st["a"], bias=st["bias"], act=case["act"],
                          gated=case["gated"], residual=st["residual"], out_dtype=out)
    if case["op"] == "grouped":
        return lq.gemm_grouped(st["w"], st["s"], st["a"], st["offsets"], rows=st["rows"],
                               bias=st["bias"], act=case["act"], gated=case["gated"], out_dtype=out)
    return lq.gemm_join(st["w"], st["s"], st["a"], st["offsets"], st["pos"], st["weight"],
                        bias=st["bias"], residual=st["residual"], out_dtype=out)


def run(state):
    """One pass.  With z = s * (signs . a) + bias per row of the weights:
    linear: act(z) + residual, or act(z_i) z_{i + m/2} + residual;
    grouped: row r of the sorted order is token rows[r] through the expert e with
    offsets[e] <= r < offsets[e + 1]; activation as linear;
    join: token t gets sum_j weight[t][j] z[pos[t][j]] + residual;
    route: the k largest logits (ties to the lowest expert), their softmax weights (over the chosen ones,
    or over all), and the order of (token, choice) pairs sorted by expert."""
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definition in 64 bits
#: Double-precision products beyond this take too long.
EXACT_FLOPS = 5e14


def _exact_product(words, K, x):
    """x [n][K] against packed rows [m][ldw] -> [n][m], both in float64, some rows at a time."""
    x = x.double()
    parts = []
    place = torch.tensor([1 << i for i in range(32)], device=words.device, dtype=torch.int64)
    for lo in range(0, words.shape[0], 2048):
        w = words[lo:lo + 2048].long() & 0xFFFFFFFF
        bit = torch.bitwise_and(w[:, :, None], place).ne(0).reshape(w.shape[0], -1)[:, :K]
        sign = torch.where(bit, 1.0, -1.0).to(torch.float64)
        parts.append(x @ sign.T)
    return torch.cat(parts, dim=1)


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


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "route":
        x = st["logits"].double()
        T, E, k = case["T"], case["E"], case["k"]
        best = torch.topk(x, k, dim=1).values          # the values; which of equal ones does not matter here
        over = best if case["renorm"] else x
        weight = torch.exp(best - torch.logsumexp(over, dim=1, keepdim=True))
        if st["valid"] is not None:
            weight = weight * st["valid"].double()[:, None]
        return {"ids": None, "weight": weight, "pos": None, "rows": None, "offsets": None}
    if work(case)["flops"] > EXACT_FLOPS:
        return None
    m, K = case["m"], case["K"]

    def one(words, s, bias, x):
        z = _exact_product(words, K, x) * s.double()
        z = z if bias is None else z + bias.double()
        if case["gated"]:
            return _exact_act(z[:, :m // 2], case["act"]) * z[:, m // 2:]
        return _exact_act(z, case["act"])

    if case["op"] == "linear":
        y = one(st["w"], st["s"], st["bias"], st["a"])
    else:
        ends = st["offsets"].tolist()
        pieces = []
        for e in range(case["E"]):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                x = st["a"][st["rows"][lo:hi].long()] if case["op"] == "grouped" else st["a"][lo:hi]
                pieces.append(one(st["w"][e], st["s"][e], None if st["bias"] is None else st["bias"][e], x))
        y = torch.cat(pieces)
        if case["op"] == "join":
            total = torch.zeros(case["T"], m, device=y.device, dtype=torch.float64)
            for j in range(case["k"]):
                total += st["weight"][:, j:j + 1].double() * y[st["pos"][:, j].long()]
            y = total
    return y if st["residual"] is None else y + st["residual"].double()
