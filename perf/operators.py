"""Measured cases of the microscaled (MX) operators.

Four operators that one quantised expert layer chains:

* ``quant``    rows -> microscaled codes (4-bit E2M1 or 8-bit E4M3 elements, one power-of-two E8M0
               scale for each 32 consecutive elements) and, for 4 bits, back to values;
* ``norm``     residual addition, root-mean-square norm and the normed rows in 8 microscaled bits;
* ``product``  rows grouped by expert times each expert's 4-bit microscaled weights;
* ``forward``  the expert MLP on such rows: gate/up product, SiLU-and-mul, requantisation, down
               product and the router-weighted sum over each token's experts.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once), or with
``own`` through the library's calls.  ``exact`` restates the definition in 64 bits.

The block rule of both quantisers: with a = max |v| of a block, e = floor(log2 a) - emax clamped to
[-127, 127] (emax = 2 for E2M1, 8 for E4M3; a = 0 gives -127); scale code e + 127; element = v / 2^e
rounded to nearest even and clamped to the largest finite element (6, 448).
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 32
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # load time: the gate/up weights of a 64-expert layer (E=64, 2I=2816, H=2048), to 4 bits and back
        {"name": "quant4-weights", "op": "quant", "rows": 64 * 2816, "cols": 2048, "dtype": "bf16", "bits": 4},
        # activations of an odd batch from a float32 producer
        {"name": "quant8-rows", "op": "quant", "rows": 517, "cols": 1408, "dtype": "f32", "bits": 8},
        # one decoded token between attention and the experts: latency
        {"name": "norm-token", "op": "norm", "T": 1, "H": 4096, "dtype": "bf16", "bits": 8, "residual": True, "y": True,
         "strided": False},
        # a prompt's rows, with the 16-bit normed rows for the router beside the 8-bit ones
        {"name": "norm-prompt", "op": "norm", "T": 8192, "H": 4096, "dtype": "bf16", "bits": 8, "residual": True, "y": True,
         "strided": False},
        # an odd batch out of a wider buffer, an odd width, 8-bit rows only
        {"name": "norm-ragged", "op": "norm", "T": 517, "H": 2080, "dtype": "f16", "bits": 8, "residual": True, "y": False,
         "strided": True},
        # a dense layer on one token: one read of the weights
        {"name": "product-token", "op": "product", "R": 1, "E": 1, "K": 4096, "N": 4096, "bits": 8, "skew": 0.0},
        # decode, 64 tokens on two of eight experts, the down projection's shape (K=14336)
        {"name": "product-decode", "op": "product", "R": 128, "E": 8, "K": 14336, "N": 4096, "bits": 8, "skew": 0.0},
        # many small experts, skewed load, an odd number of outputs, 4-bit rows
        {"name": "product-ragged", "op": "product", "R": 3001, "E": 64, "K": 2048, "N": 2817, "bits": 4, "skew": 0.7},
        # prefill, 4096 tokens on two of eight experts, the gate/up projection's shape
        {"name": "product-prefill", "op": "product", "R": 8192, "E": 8, "K": 4096, "N": 28672, "bits": 8, "skew": 0.2},
        # the whole expert MLP: decode of 64 tokens, eight large experts
        {"name": "forward-decode", "op": "forward", "T": 64, "E": 8, "k": 2, "H": 4096, "I": 14336, "bits": 8, "bias": "none"},
        # many small experts with a popularity like Zipf's (some get no token)
        {"name": "forward-fine", "op": "forward", "T": 512, "E": 128, "k": 8, "H": 2048, "I": 768, "bits": 8, "bias": "zipf"},
        # prefill of 4096 tokens, 4-bit activations
        {"name": "forward-prefill", "op": "forward", "T": 4096, "E": 8, "k": 2, "H": 4096, "I": 14336, "bits": 4,
         "bias": "normal"},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _multiple(rng, lo, hi, m, avoid=()):
    n = max(lo, min(hi, _spread(rng, lo, hi) // m * m))
    return n + m if n in avoid else n


def _seconds(case):
    w = work(case)
    return w["bytes"] / 6.5e12 + w["flops"] / 2e15


def draw(rng):
    op = rng.choice(["quant", "norm", "product", "product", "forward", "forward"])
    most = max(_seconds(c) for c in listed() if c["op"] == op)
    while True:
        bits = rng.choice([4, 8])
        if op == "quant":
            c = {"op": op, "rows": _spread(rng, 1, 200000), "cols": _multiple(rng, 32, 14336, 32, (3072,)),
                 "dtype": rng.choice(["bf16", "f16", "f32"]), "bits": bits}
            fits = c["rows"] * c["cols"] <= 3.7e8
        elif op == "norm":
            c = {"op": op, "T": _spread(rng, 1, 8192), "H": _multiple(rng, 64, 14336, 32, (3072,)),
                 "dtype": rng.choice(["bf16", "f16"]), "bits": 8, "residual": rng.random() < 0.75,
                 "y": rng.random() < 0.5, "strided": rng.random() < 0.5}
            fits = c["T"] * c["H"] <= 3.4e7
        elif op == "product":
            c = {"op": op, "R": _spread(rng, 1, 8192), "E": _spread(rng, 1, 128), "K": _multiple(rng, 128, 14336, 128, (3072,)),
                 "N": _spread(rng, 32, 28672), "bits": bits, "skew": rng.choice([0.0, 0.3, 0.7])}
            fits = c["E"] * c["N"] * c["K"] <= 9.5e8 and 3072 not in (c["R"], c["N"])
        else:
            E = _spread(rng, 1, 128)
            c = {"op": op, "T": _spread(rng, 1, 4096), "E": E, "k": rng.randint(1, min(E, 8)),
                 "H": _multiple(rng, 128, 4096, 128, (3072,)), "I": _multiple(rng, 128, 14336, 128, (1536, 3072)),
                 "bits": bits, "bias": rng.choice(["none", "normal"])}
            # (the plain form pads every expert to the fullest one's rows)
            fits = E * c["H"] * c["I"] <= 4.8e8 and c["T"] != 3072 and c["T"] * E * max(c["H"], 2 * c["I"]) <= 2e9
        if fits and _seconds(c) <= most:
            return c


# ----------------------------------------------------- inputs of a program --
def _loads(case, g):
    """Rows of each expert: popularity rank^-skew, drawn."""
    p = torch.arange(1, case["E"] + 1, dtype=torch.float64) ** -case["skew"]
    p = p[torch.randperm(case["E"], generator=g)]
    return torch.bincount(torch.multinomial(p, case["R"], replacement=True, generator=g), minlength=case["E"])


def _logits(case, g):
    """Router logits, with a bias for each expert where the load is uneven."""
    lg = torch.randn(case["T"], case["E"], generator=g)
    if case["bias"] == "normal":
        lg += torch.randn(case["E"], generator=g)
    elif case["bias"] == "zipf":
        lg += -2.2 * torch.log(torch.randperm(case["E"], generator=g) + 1.0)
    return lg


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}
    row = case["bits"] / 8 + 1 / BLOCK  # bytes of one microscaled element
    w4 = 0.5 + 1 / BLOCK
    g = torch.Generator().manual_seed(0)
    if op == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["dtype"]] + row + (2 if case["bits"] == 4 else 0)), "flops": 4.0 * n}
    if op == "norm":
        n = case["T"] * case["H"]
        return {"bytes": n * (2 + (4 if case["residual"] else 0) + (2 if case["y"] else 0) + row) + 2 * case["H"], "flops": 8.0 * n}
    if op == "product":
        touched = int((_loads(case, g) > 0).sum())
        return {"bytes": case["R"] * (case["K"] * row + case["N"] * 2) + touched * case["N"] * case["K"] * w4 + 4 * case["E"],
                "flops": 2.0 * case["R"] * case["K"] * case["N"]}
    ids = _logits(case, g).topk(case["k"], dim=1).indices
    touched = len(torch.unique(ids))
    T, k, H, I = case["T"], case["k"], case["H"], case["I"]
    return {"bytes": touched * 3 * H * I * w4 + T * (H * row + H * 2 + 8 * k), "flops": 6.0 * T * k * H * I}


def prepare(case, seed):
    gd = torch.Generator(device=DEV).manual_seed(1000 + int(seed))
    gc = torch.Generator().manual_seed(1000 + int(seed))
    op, s = case["op"], dict(case)

    def rand(*shape):
        return torch.randn(*shape, generator=gd, device=DEV)

    def hidden(rows, cols):
        """Rows of a residual stream: some channels are far louder than the others."""
        return rand(rows, cols) * torch.exp(0.7 * rand(cols))

    def weights(E, N, K):
        q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
        sc = torch.empty(E, N, K // BLOCK, dtype=torch.uint8, device=DEV)
        for e in range(E):
            q[e], sc[e] = _quantise(rand(N, K) * 0.02, 4)
        return q, sc

    if op == "quant":
        x = rand(case["rows"], case["cols"])
        x *= 0.02 if case["bits"] == 4 else torch.exp(0.7 * rand(case["cols"]))
        s["x"] = x.to(DTYPES[case["dtype"]])
    elif op == "norm":
        T, H, dt = case["T"], case["H"], DTYPES[case["dtype"]]
        wide = H + 64 if case["strided"] else H
        s["x"] = rand(T, wide).to(dt)[:, :H]
        s["residual_in"] = hidden(T, wide).to(dt)[:, :H] if case["residual"] else None
        s["weight"] = (1 + 0.2 * rand(H)).to(dt)
    elif op == "product":
        loads = _loads(case, gc)
        s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), loads.cumsum(0)]).to(torch.int32).to(DEV)
        s["most"] = int(loads.max())
        s["a"], s["a_scale"] = _quantise(hidden(case["R"], case["K"]), case["bits"])
        s["w"], s["w_scale"] = weights(case["E"], case["N"], case["K"])
    else:
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        top = _logits(case, gc).softmax(1).topk(k, dim=1)
        s["topk_w"] = (top.values / top.values.sum(1, keepdim=True)).to(DEV)
        s["topk_ids"] = top.indices.to(torch.int32).to(DEV)
        s["most"] = int(torch.bincount(top.indices.reshape(-1), minlength=E).max())
        s["a"], s["a_scale"] = _quantise(hidden(T, H), case["bits"])
        s["w13"], s["s13"] = weights(E, 2 * I, H)
        s["w2"], s["s2"] = weights(E, H, I)
    return s


# ------------------------------------------------------------- plain forms --
def _power(e):
    """2^e as float32, for whole e of [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(v, bits):
    """float32 [..., K] -> (codes uint8 [..., K * bits / 8], scale codes uint8 [..., K / 32])."""
    b = v.float().unflatten(-1, (-1, BLOCK))
    a = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(a).exponent - 1 - (2 if bits == 4 else 8)
    e = torch.where(a == 0, -127, e).clamp(-127, 127)
    t = (b * _power(-e)).flatten(-2)
    scale = (e + 127).squeeze(-1).to(torch.uint8)
    if bits == 8:
        return t.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale
    m = t.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = (torch.round(m / step) * step).clamp(max=6)
    code = torch.where(m < 2, 2 * m, torch.where(m < 4, m + 2, m / 2 + 4)).to(torch.uint8) + 8 * torch.signbit(t).to(torch.uint8)
    return code[..., 0::2] | code[..., 1::2] << 4, scale


def _values(q, scale, bits):
    """The float32 values that codes and scale codes stand for."""
    if bits == 8:
        v = q.view(torch.float8_e4m3fn).float()
    else:
        mag = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=q.device)
        one = torch.cat([mag, -mag])
        pair = torch.stack([one.repeat(16), one.repeat_interleave(16)], 1)  # both elements of each byte
        v = torch.nn.functional.embedding(q.int(), pair).flatten(-2)
    s = scale.to(torch.int32)
    p = torch.where(s == 0, 2.0 ** -127, (s << 23).view(torch.float32))
    return (v.unflatten(-1, (-1, BLOCK)) * p.unsqueeze(-1)).flatten(-2)


def _grouped(rows, w, expert, place, most):
    """rows [R, K] times the transpose of w [E, N, K][expert of the row]."""
    padded = torch.zeros(w.shape[0], most, rows.shape[1], device=rows.device)
    padded[expert, place] = rows
    return torch.bmm(padded, w.transpose(1, 2))[expert, place]


def _plain(s):
    op, bits = s["op"], s["bits"]
    if op == "quant":
        q, scale = _quantise(s["x"], bits)
        if bits == 4:
            return {"values": _values(q, scale, 4).to(torch.bfloat16)}
        return {"codes": q.view(torch.float8_e4m3fn), "scale": scale.view(torch.float8_e8m0fnu)}
    if op == "norm":
        h = s["x"].float()
        if s["residual_in"] is not None:
            h = h + s["residual_in"].float()
        y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
        q, scale = _quantise(y, bits)
        out = {"codes": q.view(torch.float8_e4m3fn), "scale": scale.view(torch.float8_e8m0fnu)}
        if s["residual_in"] is not None:
            out["residual"] = h.to(s["x"].dtype)
        if s["y"]:
            out["y"] = y.to(s["x"].dtype)
        return out
    a = _values(s["a"], s["a_scale"], bits)
    if op == "product":
        w = _values(s["w"], s["w_scale"], 4)
        r = torch.arange(s["R"], device=a.device)
        expert = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
        return _grouped(a, w, expert, r - s["offsets"][expert], s["most"]).to(torch.bfloat16)
    I = s["I"]
    expert, order = torch.sort(s["topk_ids"].reshape(-1).long(), stable=True)
    place = torch.arange(len(order), device=a.device) - torch.searchsorted(expert, expert)
    h = _grouped(a[order // s["k"]], _values(s["w13"], s["s13"], 4), expert, place, s["most"])
    act = h[:, :I] / (1 + torch.exp(-h[:, :I])) * h[:, I:]
    act = _values(*_quantise(act, bits), bits)
    y = _grouped(act, _values(s["w2"], s["s2"], 4), expert, place, s["most"])
    slots = torch.empty_like(y)
    slots[order] = y
    return (slots.unflatten(0, (-1, s["k"])) * s["topk_w"].unsqueeze(-1)).sum(1).to(torch.bfloat16)


# ------------------------------------------------------------ one pass -----
def run(state):
    if not own:
        return _plain(state)
    import weight_quantized_moe_gb300 as mq
    op, bits = state["op"], state["bits"]
    if op == "quant":
        q, scale = mq.moe_quantize_mx(state["x"], bits=bits)
        if bits == 4:
            return {"values": mq.moe_dequantize_mx(q, scale, bits=4, dtype=torch.bfloat16)}
        return {"codes": q.view(torch.float8_e4m3fn), "scale": scale.view(torch.float8_e8m0fnu)}
    if op == "norm":
        q, scale, residual, y = mq.moe_rmsnorm_mx(state["x"], state["weight"], eps=EPS, residual=state["residual_in"],
                                                  bits=bits, want_y=state["y"])
        out = {"codes": q.view(torch.float8_e4m3fn), "scale": scale.view(torch.float8_e8m0fnu)}
        if residual is not None:
            out["residual"] = residual
        if y is not None:
            out["y"] = y
        return out
    if op == "product":
        return mq.moe_mx_product(state["a"], state["a_scale"], state["w"], state["w_scale"],
                                 expert_offsets=state["offsets"], a_bits=bits)
    return mq.moe_mx_forward(state["a"], state["a_scale"], state["w13"], state["s13"], state["w2"], state["s2"],
                             state["topk_w"], state["topk_ids"], a_bits=bits)


# --------------------------------------------------------------- 64 bits ---
def exact(case, seed):
    s = prepare(case, seed)
    op, bits, f64 = s["op"], s["bits"], torch.float64

    def to_codes(v):
        """(element values, scale values, what they stand for) of the block rule."""
        b = v.reshape(*v.shape[:-1], -1, BLOCK)
        a = b.abs().max(dim=-1, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a))))
        # (log2 may round up to a whole number just below it)
        e = torch.where(a < torch.exp2(e), e - 1, e) - (2 if bits == 4 else 8)
        e = torch.where(a > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
        p = torch.exp2(e)
        t = b / p
        m = t.abs()
        if bits == 4:
            r = torch.zeros_like(m)
            below = 0.0
            # halfway points, and whether a tie goes up (to the element with an even last bit)
            for value, half, up in ((0.5, 0.25, 0), (1, 0.75, 1), (1.5, 1.25, 0), (2, 1.75, 1), (3, 2.5, 0), (4, 3.5, 1), (6, 5, 0)):
                r += (value - below) * ((m >= half) if up else (m > half))
                below = value
        else:
            x = torch.frexp(m)[1].to(f64) - 1
            u = torch.exp2(x.clamp(min=-6) - 3)
            r = (torch.round(m / u) * u).clamp(max=448)
        r = torch.copysign(r, t)
        return r.reshape(v.shape), p.squeeze(-1), (r * p).reshape(v.shape)

    def stands_for(q, scale, nbits):
        if nbits == 8:
            v = q.view(torch.float8_e4m3fn).to(f64)
        else:
            lut = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=f64, device=q.device)
            v = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=f64, device=q.device)
            v[..., 0::2] = lut[(q & 15).long()]
            v[..., 1::2] = lut[(q >> 4).long()]
        return v * torch.exp2(scale.to(f64) - 127).repeat_interleave(BLOCK, -1)

    if op == "quant":
        if bits == 4:
            out = torch.empty(s["x"].shape, dtype=f64, device=DEV)
            for i in range(0, out.shape[0], 16384):
                out[i:i + 16384] = to_codes(s["x"][i:i + 16384].to(f64))[2]
            return {"values": out}
        codes, scale, _ = to_codes(s["x"].to(f64))
        return {"codes": codes, "scale": scale}
    if op == "norm":
        h = s["x"].to(f64) + (0 if s["residual_in"] is None else s["residual_in"].to(f64))
        y = h / torch.sqrt((h * h).sum(-1, keepdim=True) / s["H"] + EPS) * s["weight"].to(f64)
        codes, scale, _ = to_codes(y)
        out = {"codes": codes, "scale": scale}
        if s["residual_in"] is not None:
            out["residual"] = h
        if s["y"]:
            out["y"] = y
        return out
    a = stands_for(s["a"], s["a_scale"], bits)
    if op == "product":
        at = s["offsets"].tolist()
        out = torch.zeros(s["R"], s["N"], dtype=f64, device=DEV)
        for e in range(s["E"]):
            if at[e + 1] > at[e]:
                out[at[e]:at[e + 1]] = a[at[e]:at[e + 1]] @ stands_for(s["w"][e], s["w_scale"][e], 4).T
        return out
    out = torch.zeros(s["T"], s["H"], dtype=f64, device=DEV)
    for e in range(s["E"]):
        t, j = torch.nonzero(s["topk_ids"] == e, as_tuple=True)
        if len(t):
            h = a[t] @ stands_for(s["w13"][e], s["s13"][e], 4).T
            act = to_codes(torch.sigmoid(h[:, :s["I"]]) * h[:, :s["I"]] * h[:, s["I"]:])[2]
            y = act @ stands_for(s["w2"][e], s["s2"][e], 4).T
            out.index_add_(0, t, y * s["topk_w"][t, j].to(f64).unsqueeze(1))
    return out
