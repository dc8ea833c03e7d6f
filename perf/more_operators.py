"""Measured cases of the 16-bit grouped product, its gradients, and low-rank adapters beside it.

Three operators for layers whose experts (or dense projections) hold bf16 or f16 weights:

* ``product``  rows grouped by expert times each expert's weights, out[r] = W[e(r)] a[r];
* ``grad``     both gradients of that product: da[r] = W[e(r)]^T dy[r] and dW[e] = sum over e's rows of dy[r] a[r]^T;
* ``lora``     low-rank adapters of many requests in one call, beside a projection that is already computed:
               out[r] = base[r] + s[l] B[l, e] (A[l, e] x[r]), l the row's adapter (or none), e its expert.

``run`` computes a case in its plain form (elementary torch operations in 32 bits, rounded once), or with
``own`` through the library's calls.  ``exact`` restates the definition in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # a dense layer on one token: one read of the weights
        {"name": "product-token", "op": "product", "R": 1, "E": 1, "K": 4096, "N": 4096, "dtype": "bf16", "out": "bf16",
         "skew": 0.0},
        # decode, 64 tokens on two of eight experts, the gate/up projection's shape
        {"name": "product-decode", "op": "product", "R": 128, "E": 8, "K": 4096, "N": 28672, "dtype": "bf16", "out": "bf16",
         "skew": 0.0},
        # 512 tokens on eight of 128 small experts, popularity like Zipf's (some get no row)
        {"name": "product-fine", "op": "product", "R": 4096, "E": 128, "K": 2048, "N": 1536, "dtype": "f16", "out": "f16",
         "skew": 1.0},
        # odd counts: rows, outputs and a row length that fills no tile, float32 results
        {"name": "product-ragged", "op": "product", "R": 3001, "E": 64, "K": 2056, "N": 2817, "dtype": "bf16", "out": "f32",
         "skew": 0.7},
        # prefill, 4096 tokens on two of eight experts, the gate/up projection's shape
        {"name": "product-prefill", "op": "product", "R": 8192, "E": 8, "K": 4096, "N": 28672, "dtype": "bf16", "out": "bf16",
         "skew": 0.2},
        # a training step's backward pass through a small batch, float32 weight gradients to accumulate into
        {"name": "grad-ragged", "op": "grad", "R": 517, "E": 16, "K": 1408, "N": 2048, "dtype": "f16", "out": "f32", "skew": 0.7},
        # many small experts, 512 tokens on eight of 128
        {"name": "grad-fine", "op": "grad", "R": 4096, "E": 128, "K": 2048, "N": 1536, "dtype": "bf16", "out": "bf16", "skew": 1.0},
        # a training step's backward pass through the gate/up projection: 4096 tokens on two of eight experts
        {"name": "grad-train", "op": "grad", "R": 8192, "E": 8, "K": 4096, "N": 28672, "dtype": "bf16", "out": "bf16", "skew": 0.2},
        # one decoded token with an adapter: latency
        {"name": "lora-token", "op": "lora", "R": 1, "E": 1, "K": 4096, "N": 4096, "L": 16, "r": 16, "dtype": "bf16", "run": 1,
         "none": 0.0},
        # decode, 64 requests on 48 adapters
        {"name": "lora-decode", "op": "lora", "R": 64, "E": 1, "K": 4096, "N": 4096, "L": 48, "r": 16, "dtype": "bf16", "run": 1,
         "none": 0.1},
        # prompts of several requests in one batch, high rank
        {"name": "lora-prompts", "op": "lora", "R": 4099, "E": 1, "K": 4096, "N": 4096, "L": 16, "r": 64, "dtype": "bf16", "run": 400,
         "none": 0.1},
        # adapters of the experts' gate/up projection: 512 tokens on eight of 64 experts
        {"name": "lora-experts", "op": "lora", "R": 4096, "E": 64, "K": 2048, "N": 2816, "L": 6, "r": 32, "dtype": "f16", "run": 100,
         "none": 0.2},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _eights(rng, lo, hi):
    return max(lo, min(hi, _spread(rng, lo, hi) // 8 * 8))


def _seconds(case):
    w = work(case)
    return w["bytes"] / 6.5e12 + w["flops"] / 1.8e15


def draw(rng):
    op = rng.choice(["product", "product", "grad", "grad", "lora", "lora"])
    most = max(_seconds(c) for c in listed() if c["op"] == op)
    while True:
        dtype = rng.choice(["bf16", "f16"])
        c = {"op": op, "R": _spread(rng, 1, 8192), "E": _spread(rng, 1, 128), "K": _eights(rng, 64, 14336)}
        if op == "lora":
            E = c["E"] = c["E"] if rng.random() < 0.4 else 1
            c |= {"N": _spread(rng, 32, 14336), "L": _spread(rng, 1, 64), "r": rng.choice([8, 16, 24, 32, 64, 128]),
                  "dtype": dtype, "run": rng.choice([1, 30, 500]), "none": rng.choice([0.0, 0.2])}
            fits = E * c["L"] * c["r"] * (c["K"] + c["N"]) <= 1e9 and c["R"] * max(c["K"], c["N"]) <= 3.4e7
        else:
            c |= {"N": _spread(rng, 32, 28672) if op == "product" else _eights(rng, 32, 28672), "dtype": dtype,
                  "out": rng.choice([dtype, dtype, "f32"]), "skew": rng.choice([0.0, 0.3, 0.7, 1.0])}
            fits = c["E"] * c["N"] * c["K"] <= 9.5e8
        # (the plain form pads every group to the fullest one's rows)
        if fits and c["R"] * c["E"] * max(c["K"], c["N"]) <= 4e9 and _seconds(c) <= most:
            return c


# ----------------------------------------------------- inputs of a program --
def _loads(case, g):
    """Rows of each expert: popularity rank^-skew, drawn."""
    p = torch.arange(1, case["E"] + 1, dtype=torch.float64) ** -case.get("skew", 0.3)
    p = p[torch.randperm(case["E"], generator=g)]
    return torch.bincount(torch.multinomial(p, case["R"], replacement=True, generator=g), minlength=case["E"])


def _adapters(case, g):
    """Each row's adapter, -1 for none: tokens of a request stand together, also among an expert's rows."""
    R, L = case["R"], case["L"]
    requests = max(1, round(R / case["run"]))
    of = torch.randint(L, (requests,), generator=g)
    of = torch.where(torch.rand(requests, generator=g) < case["none"], -1, of)
    token = torch.sort(torch.randint(requests, (R,), generator=g)).values if case["run"] > 1 else torch.arange(R) % requests
    return of[token]


def _expert_rows(loads):
    return torch.repeat_interleave(torch.arange(len(loads)), loads)


def _row_adapters(case, loads, g):
    """Adapters of rows in expert order: each expert's rows are a choice of the tokens, in their order."""
    ids = _adapters(case, g)
    if case["E"] == 1:
        return ids
    mixed = torch.randperm(case["R"], generator=g)
    key = _expert_rows(loads) * case["R"] + mixed
    return ids[torch.sort(key).values % case["R"]]


def work(case):
    op, R, E, K, N = (case[n] for n in ("op", "R", "E", "K", "N"))
    g = torch.Generator().manual_seed(0)
    loads = _loads(case, g)
    touched = int((loads > 0).sum())
    out = 4 if case.get("out") == "f32" else 2
    if op == "product":
        return {"bytes": 2 * R * K + 2 * touched * N * K + out * R * N + 4 * E, "flops": 2.0 * R * K * N}
    if op == "grad":
        return {"bytes": 2 * R * (2 * K + N) + 2 * touched * N * K + out * E * N * K + 4 * E, "flops": 4.0 * R * K * N}
    ids = _row_adapters(case, loads, g)
    has = ids >= 0
    groups = len(torch.unique(_expert_rows(loads)[has] * case["L"] + ids[has]))
    live = int(has.sum())
    return {"bytes": 2 * live * K + 2 * groups * case["r"] * (K + N) + 4 * R * N + 4 * R, "flops": 2.0 * live * case["r"] * (K + N)}


def prepare(case, seed):
    gd = torch.Generator(device=DEV).manual_seed(2000 + int(seed))
    gc = torch.Generator().manual_seed(2000 + int(seed))
    op, R, E, K, N, dt = case["op"], case["R"], case["E"], case["K"], case["N"], DTYPES[case["dtype"]]
    s = dict(case)

    def rand(*shape):
        return torch.randn(*shape, generator=gd, device=DEV)

    def weights(n, rows, cols, scale):
        w = torch.empty(n, rows, cols, dtype=dt, device=DEV)
        for e in range(n):
            w[e] = rand(rows, cols) * scale
        return w

    loads = _loads(case, gc)
    s["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), loads.cumsum(0)]).to(torch.int32).to(DEV)
    s["a"] = (rand(R, K) * torch.exp(0.5 * rand(K))).to(dt)  # normed rows: some channels are louder
    if op == "lora":
        ids = _row_adapters(case, loads, gc)
        group = torch.where(ids >= 0, _expert_rows(loads) * case["L"] + ids, E * case["L"])
        s["most"] = int(torch.bincount(group).max())
        s["adapters"] = ids.to(torch.int32).to(DEV)
        s["lora_a"] = weights(case["L"] * E, case["r"], K, K ** -0.5).unflatten(0, (case["L"], E))
        s["lora_b"] = weights(case["L"] * E, N, case["r"], 0.3 * case["r"] ** -0.5).unflatten(0, (case["L"], E))
        s["scaling"] = (0.5 + torch.rand(case["L"], generator=gc)).to(DEV)
        s["base"] = rand(R, N).to(dt)
        return s
    s["most"] = int(loads.max())
    s["w"] = weights(E, N, K, 0.02)
    if op == "grad":
        s["dy"] = (rand(R, N) * 1e-2).to(dt)
    return s


# ------------------------------------------------------------- plain forms --
def _places(group):
    """(rows in group order, their groups, each one's place within its group)."""
    ordered, order = torch.sort(group, stable=True)
    return order, ordered, torch.arange(len(order), device=group.device) - torch.searchsorted(ordered, ordered)


def _expert_of(s):
    r = torch.arange(s["R"], device=s["a"].device)
    return torch.searchsorted(s["offsets"][1:].long(), r, right=True)


def _padded(rows, groups, most, group, place):
    p = torch.zeros(groups, most, rows.shape[1], device=rows.device)
    p[group, place] = rows.float()
    return p


def _plain(s):
    op, E, most = s["op"], s["E"], s["most"]
    expert = _expert_of(s)
    dt = s["a"].dtype
    if op == "lora":
        L = s["L"]
        l = s["adapters"].long()
        order, group, place = _places(torch.where(l >= 0, expert * L + l, E * L))
        live = int(L * E)
        a = s["lora_a"].transpose(0, 1).flatten(0, 1).float()  # [E L, r, K]
        b = s["lora_b"].transpose(0, 1).flatten(0, 1).float()
        x = _padded(s["a"][order], live + 1, most, group, place)[:live]
        delta = torch.bmm(torch.bmm(x, a.transpose(1, 2)), b.transpose(1, 2))
        delta = delta * s["scaling"].repeat(E)[:, None, None]
        delta = torch.cat([delta, torch.zeros_like(delta[:1])])[group, place]
        out = torch.empty_like(delta)
        out[order] = s["base"][order].float() + delta
        return {"out": out.to(dt)}
    _, group, place = _places(expert)
    a = _padded(s["a"], E, most, group, place)
    if op == "product":
        out = torch.bmm(a, s["w"].float().transpose(1, 2))[group, place]
        return {"out": out.to(DTYPES[s["out"]])}
    dy = _padded(s["dy"], E, most, group, place)
    return {"da": torch.bmm(dy, s["w"].float())[group, place].to(dt),
            "dw": torch.bmm(dy.transpose(1, 2), a).to(DTYPES[s["out"]])}


# ------------------------------------------------------------ one pass -----
def run(state):
    if not own:
        return _plain(state)
    import weight_quantized_moe_gb300 as mq
    op = state["op"]
    if op == "product":
        return {"out": mq.moe_grouped_product(state["a"], state["w"], expert_offsets=state["offsets"],
                                              out_dtype=DTYPES[state["out"]])}
    if op == "grad":
        da, dw = mq.moe_grouped_product_grad(state["dy"], state["a"], state["w"], expert_offsets=state["offsets"],
                                             dw_dtype=DTYPES[state["out"]])
        return {"da": da, "dw": dw}
    return {"out": mq.moe_lora_product(state["a"], state["lora_a"], state["lora_b"], state["adapters"], base=state["base"],
                                       expert_offsets=state["offsets"], scaling=state["scaling"])}


# --------------------------------------------------------------- 64 bits ---
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    at = s["offsets"].tolist()
    R, E, K, N = s["R"], s["E"], s["K"], s["N"]
    if s["op"] == "product":
        out = torch.zeros(R, N, dtype=f64, device=DEV)
        for e in range(E):
            rows = slice(at[e], at[e + 1])
            if at[e + 1] > at[e]:
                out[rows] = s["a"][rows].to(f64) @ s["w"][e].to(f64).T
        return {"out": out}
    if s["op"] == "grad":
        da = torch.zeros(R, K, dtype=f64, device=DEV)
        dw = torch.zeros(E, N, K, dtype=f64, device=DEV)
        for e in range(E):
            rows = slice(at[e], at[e + 1])
            if at[e + 1] > at[e]:
                dy = s["dy"][rows].to(f64)
                da[rows] = dy @ s["w"][e].to(f64)
                dw[e] = dy.T @ s["a"][rows].to(f64)
        return {"da": da, "dw": dw}
    out = s["base"].to(f64)
    ids = s["adapters"].cpu()
    row_expert = torch.bucketize(torch.arange(R), torch.tensor(at[1:]), right=True)
    for e, l in {(int(e), int(l)) for e, l in zip(row_expert, ids) if l >= 0}:
        rows = torch.nonzero((row_expert == e) & (ids == l)).flatten().to(DEV)
        h = s["a"][rows].to(f64) @ s["lora_a"][l, e].to(f64).T
        out[rows] += s["scaling"][l].to(f64) * (h @ s["lora_b"][l, e].to(f64).T)
    return {"out": out}
