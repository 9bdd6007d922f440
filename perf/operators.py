"""What the low-rank adapter calls and the whole mixture-of-experts layer cost, case by case.

Two sets of operators that a decoder's serving step puts together:

* low-rank adapters of many requests beside a shared packed projection
  (``q8_linear_lora``, ``q8_linear_fused_gate_up_silu_lora``) and beside a product that is
  there already (``lora_add``, ``lora_gate_up_silu``):
      y[t] = W x[t] + s_a B_a (A_a x[t]),  a = the row's adapter (none: -1);
* the whole mixture-of-experts layer of a few tokens (``q8_moe_layer``):
      y[t] = sum_j p_j W_down[e_j] (SiLU(W_gate[e_j] x[t]) * (W_up[e_j] x[t])),
  the e_j and p_j from the softmax top-k of the router's logits.

With ``own`` false every operator is computed in its plain form from elementary torch
operations in float32; with ``own`` true by this package's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
QK, BLOCK = 32, 34  # a Q8_0 block: binary16 scale, 32 int8 quants
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # One request's next token through the 8B block's fused q/k/v projection: latency.
        {"name": "lora_qkv_m1", "op": "lora_linear", "m": 1, "k": 4096, "n": 6144, "parts": "4096,1024,1024",
         "adapters": 1, "rank": 16, "type": "bf16", "ranks": False, "none": 0.0},
        # A decode batch of sixteen requests on eight adapters, two rows without one, through q/k/v.
        {"name": "lora_qkv_m16", "op": "lora_linear", "m": 16, "k": 4096, "n": 6144, "parts": "4096,1024,1024",
         "adapters": 8, "rank": 16, "type": "bf16", "ranks": False, "none": 0.1},
        # The 8B block's fused gate and up of a small decode batch, each projection with its own adapter.
        {"name": "lora_gate_up_m8", "op": "lora_gate_up", "m": 8, "k": 4096, "f": 12288, "parts": "12288,12288",
         "adapters": 4, "rank": 32, "type": "bf16", "ranks": True, "none": 0.0},
        # The 8B block's down projection, a batch of five, high ranks in binary16.
        {"name": "lora_down_m5", "op": "lora_linear", "m": 5, "k": 12288, "n": 4096, "parts": "4096",
         "adapters": 3, "rank": 64, "type": "fp16", "ranks": False, "none": 0.0},
        # A big decode batch on a small odd-sized projection, float32 adapters of several ranks.
        {"name": "lora_odd_m83", "op": "lora_linear", "m": 83, "k": 1024, "n": 2001, "parts": "1500,501",
         "adapters": 17, "rank": 24, "type": "fp32", "ranks": True, "none": 0.3},
        # A prompt batch's adapters beside a projection that has been computed: long and ragged.
        {"name": "lora_add_m2048", "op": "lora_add", "m": 2048, "k": 4096, "n": 6144, "parts": "4096,1024,1024",
         "adapters": 6, "rank": 32, "type": "bf16", "ranks": True, "none": 0.1},
        # The same beside gate and up, with the activation behind them.
        {"name": "lora_act_m611", "op": "lora_act", "m": 611, "k": 4096, "f": 12288, "parts": "12288,12288",
         "adapters": 3, "rank": 16, "type": "fp16", "ranks": False, "none": 0.0},
        # One token through the 30B-A3B layer: latency.
        {"name": "moe_a3b_m1", "op": "moe", "m": 1, "experts": 128, "top": 8, "h": 2048, "f": 768,
         "normalize": True, "top_p": 1.0},
        # A few tokens (drafted ones, or a small batch), experts dropped below the cumulative share.
        {"name": "moe_a3b_m5", "op": "moe", "m": 5, "experts": 128, "top": 8, "h": 2048, "f": 768,
         "normalize": True, "top_p": 0.9},
        # A decode batch of sixteen.
        {"name": "moe_a3b_m16", "op": "moe", "m": 16, "experts": 128, "top": 8, "h": 2048, "f": 768,
         "normalize": True, "top_p": 1.0},
        # The largest batch listed: four routed tokens for each expert on average.
        {"name": "moe_a3b_m64", "op": "moe", "m": 64, "experts": 128, "top": 8, "h": 2048, "f": 768,
         "normalize": True, "top_p": 1.0},
        # Few wide experts, two of eight chosen, their probabilities not divided by their sum.
        {"name": "moe_e8_m7", "op": "moe", "m": 7, "experts": 8, "top": 2, "h": 1280, "f": 1792,
         "normalize": False, "top_p": 1.0},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora_linear", "lora_gate_up", "lora_add", "lora_act", "moe", "moe", "moe"])
    if op == "moe":
        while True:
            experts = _log_int(rng, 4, 256)
            top = rng.randint(1, min(8, experts))
            h, f = 256 * _log_int(rng, 1, 16), 256 * _log_int(rng, 1, 8)
            # below eight routed tokens an expert, the layer's float32 range
            m = _log_int(rng, 1, max(1, min(64, (8 * experts - 1) // top)))
            if experts * h * f <= 128 * 2048 * 768:
                return {"op": op, "m": m, "experts": experts, "top": top, "h": h, "f": f,
                        "normalize": rng.random() < 0.7, "top_p": rng.choice([1.0, 1.0, 0.95, 0.7])}
    while True:
        k = 256 * _log_int(rng, 1, 48)
        n = _log_int(rng, 64, 16384)
        if n * k <= 4096 * 12288 * 2:
            break
    case = {"op": op, "m": _log_int(rng, 1, 2048) if op in ("lora_add", "lora_act") else _log_int(rng, 1, 100), "k": k}
    if op in ("lora_gate_up", "lora_act"):
        case["f"], parts = n, [n, n]
    else:
        cut = sorted(rng.randint(1, n - 1) for _ in range(rng.choice([0, 1, 2])))
        case["n"], parts = n, [b - a for a, b in zip([0] + cut, cut + [n]) if b > a]
    case["parts"] = ",".join(str(p) for p in parts)
    case.update(adapters=_log_int(rng, 1, 32), rank=8 * rng.randint(1, 8), type=rng.choice(sorted(TYPES)),
                ranks=rng.random() < 0.5, none=rng.choice([0.0, 0.1, 0.5]))
    return case


def _parts(case):
    return [int(p) for p in case["parts"].split(",")]


# ----------------------------------------------------------------------------- inputs


def _packed(gen, rows, k):
    """Q8_0 bytes of weights of about N(0, 0.02^2), as quantizing a trained matrix gives them."""
    blocks = torch.empty((rows, k // QK, BLOCK), dtype=torch.uint8, device=DEV)
    scale = (0.02 / 40) * (0.75 + 0.5 * torch.rand((rows, k // QK), generator=gen, device=DEV))
    blocks[..., :2] = scale.half().unsqueeze(-1).view(torch.uint8)
    # the sum of two uniform draws: a bell of standard deviation about 40 over [-126, 126]
    q = torch.randint(-49, 50, (rows, k), generator=gen, device=DEV, dtype=torch.int8)
    q += torch.randint(-49, 50, (rows, k), generator=gen, device=DEV, dtype=torch.int8)
    blocks[..., 2:] = q.view(torch.uint8).view(rows, k // QK, QK)
    return blocks.view(-1)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    m, s = case["m"], dict(case)
    if case["op"] == "moe":
        e, h, f = case["experts"], case["h"], case["f"]
        s["router"] = 0.02 * normal(e, h)
        s["gate_up"] = _packed(gen, e * 2 * f, h)
        s["down"] = _packed(gen, e * h, f)
        s["x"] = normal(m, h)
        return s
    k, rank, count, parts = case["k"], case["rank"], case["adapters"], _parts(case)
    n = sum(parts)
    s["x"] = normal(m, k)
    s["a"] = (normal(count, len(parts) * rank, k) / math.sqrt(k)).to(TYPES[case["type"]])
    s["b"] = (0.1 * normal(count, n, rank)).to(TYPES[case["type"]])
    s["scale"] = 0.5 + 1.5 * torch.rand(count, generator=gen, device=DEV)
    s["ranks"] = (torch.randint(1, rank + 1, (count,), generator=gen, device=DEV, dtype=torch.int32)
                  if case["ranks"] else None)
    adapter = torch.randint(0, count, (m,), generator=gen, device=DEV, dtype=torch.int32)
    s["adapter"] = torch.where(torch.rand(m, generator=gen, device=DEV) < case["none"], -1, adapter).to(torch.int32)
    s["parts"] = parts
    if case["op"] in ("lora_linear", "lora_gate_up"):
        s["w"] = _packed(gen, n, k)
    else:
        s["y"] = normal(m, n)  # the shared projection's output
    return s


# -------------------------------------------------------------------------- plain form


def _unpack(packed, rows, k):
    b = packed.view(-1, BLOCK)
    d = b[:, :2].contiguous().view(torch.float16).float()
    q = b[:, 2:].contiguous().view(torch.int8).float()
    return (q * d).view(-1, rows, k)


def _silu_mul(gu, f):
    g = gu[..., :f]
    return g / (1 + torch.exp(-g)) * gu[..., f:]


def _delta(s):
    """Every adapter's first product for every row; a row keeps its own adapter's alone."""
    count, n, rank = s["b"].shape
    parts = s["parts"]
    ids = torch.arange(count, device=DEV)
    keep = (s["adapter"][:, None] == ids).float() * s["scale"]
    u = (s["x"] @ s["a"].float().reshape(-1, s["a"].shape[2]).T).view(-1, count, len(parts), rank)
    u = u * keep[:, :, None, None]
    if s["ranks"] is not None:
        u = u * (torch.arange(rank, device=DEV) < s["ranks"][:, None])[None, :, None, :]
    rows = s["b"].float().split(parts, dim=1)
    return torch.cat([u[:, :, i].reshape(-1, count * rank) @ r.transpose(1, 2).reshape(count * rank, -1)
                      for i, r in enumerate(rows)], dim=1)


def _choose(s):
    """The chosen experts and their weights, [m][top]; a slot behind the top-p cut has weight 0."""
    logits = s["x"].double() @ s["router"].double().T
    p, idx = torch.sort(torch.softmax(logits, dim=1), dim=1, descending=True, stable=True)
    p, idx = p[:, :s["top"]], idx[:, :s["top"]]
    if s["top_p"] < 1:
        before = torch.cumsum(p, dim=1) - p
        p = p * (before < s["top_p"] * p.sum(dim=1, keepdim=True))
    if s["normalize"]:
        p = p / p.sum(dim=1, keepdim=True)
    return idx, p.float()


def _mixture(s):
    idx, p = _choose(s)
    e, h, f, m, x = s["experts"], s["h"], s["f"], s["m"], s["x"]
    if idx.numel() <= e:  # the chosen experts' weights, one copy a pair
        pair = idx.reshape(-1)
        gu = _unpack(s["gate_up"].view(e, -1)[pair], 2 * f, h)
        hid = _silu_mul(torch.bmm(gu, x.repeat_interleave(s["top"], dim=0)[:, :, None])[:, :, 0], f)
        out = torch.bmm(_unpack(s["down"].view(e, -1)[pair], h, f), hid[:, :, None])
        return (out.view(m, -1, h) * p[:, :, None]).sum(dim=1)
    weight = torch.zeros((m, e), device=DEV).scatter_(1, idx, p)
    hid = _silu_mul((x @ _unpack(s["gate_up"], 2 * f, h).view(-1, h).T).view(m, e, 2 * f), f)
    hid = (hid * weight[:, :, None]).view(m, e * f)
    return hid @ _unpack(s["down"], h, f).transpose(1, 2).reshape(e * f, h)


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "moe":
        return _mixture(s)
    if s["op"] in ("lora_linear", "lora_gate_up"):
        y = s["x"] @ _unpack(s["w"], sum(s["parts"]), s["k"])[0].T + _delta(s)
    else:
        y = s["y"] + _delta(s)
    return _silu_mul(y, s["f"]) if s["op"] in ("lora_gate_up", "lora_act") else y


def _run_own(s):
    import block_quantized_weight_linear_amd as q8

    if s["op"] == "moe":
        return q8.q8_moe_layer(s["router"], s["gate_up"], s["down"], s["experts"], s["f"], s["h"], s["x"], s["top"],
                               normalize=s["normalize"], top_p=s["top_p"])
    lora = (s["a"], s["b"], s["adapter"])
    more = {"scale": s["scale"], "ranks": s["ranks"], "sections": s["parts"]}
    if s["op"] == "lora_linear":
        return q8.q8_linear_lora(s["w"], s["n"], s["k"], s["x"], *lora, **more)
    if s["op"] == "lora_gate_up":
        return q8.q8_linear_fused_gate_up_silu_lora(s["w"], s["f"], s["k"], s["x"], *lora, **more)
    if s["op"] == "lora_add":
        return q8.lora_add(s["y"], s["x"], *lora, **more)
    return q8.lora_gate_up_silu(s["y"], s["x"], *lora, **more)


# -------------------------------------------------------------------------------- work


def work(case):
    m = case["m"]
    if case["op"] == "moe":
        e, top, h, f = case["experts"], case["top"], case["h"], case["f"]
        used = e * (1 - (1 - top / e) ** m)  # experts that m tokens choose, on average
        weights = 3 * f * h
        return {"bytes": used * weights * BLOCK / QK + 4 * e * h + 8 * m * h,
                "flops": 2 * m * (top * weights + e * h)}
    k, rank, parts, size = case["k"], case["rank"], _parts(case), TYPES[case["type"]].itemsize
    n = sum(parts)
    rows = m * (1 - case["none"])
    used = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** rows)
    share = (rank + 1) / (2 * rank) if case["ranks"] else 1.0  # of the padded rank, on average
    out = case["f"] if "f" in case else n
    base = n * k * BLOCK / QK if case["op"] in ("lora_linear", "lora_gate_up") else 4 * m * n
    flops = 2 * m * n * k if case["op"] in ("lora_linear", "lora_gate_up") else 0
    return {"bytes": base + used * share * size * rank * (len(parts) * k + n) + 4 * m * (k + out),
            "flops": flops + 2 * rows * share * rank * (len(parts) * k + n)}


# ------------------------------------------------------------------------------- exact


def _exact_weight(packed, rows, k):
    block = packed.reshape(rows, k // QK, BLOCK)
    quants = block[:, :, 2:].to(torch.int16)
    quants = torch.where(quants > 127, quants - 256, quants).to(torch.float64)
    return torch.mul(quants, block[:, :, :2].contiguous().view(torch.float16).to(torch.float64)).reshape(rows, k)


def _exact_act(gate, up):
    return gate * torch.sigmoid(gate) * up


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"].to(torch.float64)
    if case["op"] == "moe":
        e, h, f, top = case["experts"], case["h"], case["f"], case["top"]
        prob = torch.softmax(torch.matmul(x, s["router"].to(torch.float64).t()), 1).cpu()
        y = torch.zeros((case["m"], h), dtype=torch.float64, device=DEV)
        given = {}
        for t in range(case["m"]):
            order = sorted(range(e), key=lambda i: (-prob[t, i].item(), i))[:top]
            total, kept, so_far = sum(prob[t, i].item() for i in order), [], 0.0
            for i in order:
                if not kept or case["top_p"] >= 1 or so_far < case["top_p"] * total:
                    kept.append(i)
                so_far += prob[t, i].item()
            by = sum(prob[t, i].item() for i in kept) if case["normalize"] else 1.0
            for i in kept:
                given.setdefault(i, []).append((t, prob[t, i].item() / by))
        gate_up, down = s["gate_up"].reshape(e, -1), s["down"].reshape(e, -1)
        for i, pairs in given.items():
            rows = torch.tensor([t for t, _ in pairs], device=DEV)
            share = torch.tensor([w for _, w in pairs], dtype=torch.float64, device=DEV)
            both = torch.matmul(x[rows], _exact_weight(gate_up[i], 2 * f, h).t())
            hidden = _exact_act(both[:, :f], both[:, f:])
            y.index_add_(0, rows, share[:, None] * torch.matmul(hidden, _exact_weight(down[i], h, f).t()))
        return y
    n, rank = sum(s["parts"]), case["rank"]
    if "w" in s:
        y = torch.matmul(x, _exact_weight(s["w"], n, case["k"]).t())
    else:
        y = s["y"].to(torch.float64)
    of_row = s["adapter"].tolist()
    for t, i in enumerate(of_row):
        if i < 0:
            continue
        r = int(s["ranks"][i]) if s["ranks"] is not None else rank
        at = 0
        for p, size in enumerate(s["parts"]):
            inner = torch.mv(s["a"][i, p * rank:p * rank + r].to(torch.float64), x[t])
            y[t, at:at + size] += s["scale"][i].to(torch.float64) * torch.mv(
                s["b"][i, at:at + size, :r].to(torch.float64), inner)
            at += size
    return _exact_act(y[:, :n // 2], y[:, n // 2:]) if "f" in case else y
