"""What the block-scaled 8-bit floating-point linears cost, case by case.

Weights and activations are e4m3 codes with one float32 scale for each block of 128: a weight
block is 128 rows x 128 inputs, an activation block 128 inputs of one row.

* ``f8_quantize_act`` / ``f8_quantize_weight``: codes and scales of float rows or matrices;
* ``f8_linear``: y[t][n] = sum_b sx[t][b] sw[n/128][b] sum_{i in b} qx[t][i] qw[n][i];
* ``f8_linear_fused_gate_up_silu``: h = SiLU(g) * u with [g u] = x . W^T, and [g u] where it is kept;
* ``f8_linear_backward``: dx = dy . W and dW = dy^T . x;
* ``f8_linear_fused_gate_up_silu_backward``: the same two products behind the activation's gradient.

With ``own`` false every operator is computed in its plain form from elementary torch
operations in float32; with ``own`` true by this package's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
BLOCK = 128
TOP = 448.0  # e4m3's largest value
TINY = 2.0 ** -116  # a block whose largest magnitude is below this is coded as zeros
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------ cases


def listed():
    return [
        # The input of a decode batch's projection, float32 as the packed linears take it: latency.
        {"name": "quantize_act_m16", "op": "quantize_act", "m": 16, "k": 4096, "type": "fp32", "pow2": False},
        # A gate projection's master weights after a step of training, scales that are powers of two.
        {"name": "quantize_weight", "op": "quantize_weight", "n": 12288, "k": 4096, "type": "fp32", "pow2": True},
        # One request's next token through the 8B block's fused q/k/v projection: latency.
        {"name": "linear_m1", "op": "linear", "m": 1, "n": 6144, "k": 4096, "type": "bf16"},
        # A decode batch through the 8B block's down projection, float32 outputs.
        {"name": "linear_down_m37", "op": "linear", "m": 37, "n": 4096, "k": 12288, "type": "fp32"},
        # A short prompt on a small odd-sized projection, its last block of inputs cut short.
        {"name": "linear_odd_m300", "op": "linear", "m": 300, "n": 2001, "k": 1040, "type": "fp16"},
        # A prompt batch through the 8B block's fused q/k/v projection.
        {"name": "linear_m4096", "op": "linear", "m": 4096, "n": 6144, "k": 4096, "type": "bf16"},
        # A small decode batch through the 8B block's gate and up.
        {"name": "gate_up_m8", "op": "gate_up", "m": 8, "f": 12288, "k": 4096, "type": "bf16", "keep": False},
        # The same of a training batch, which keeps the gate and up rows for its backward pass.
        {"name": "gate_up_m2048", "op": "gate_up", "m": 2048, "f": 12288, "k": 4096, "type": "bf16", "keep": True},
        # Gradients of a few rows in float32 through an odd-sized projection.
        {"name": "linear_back_odd_m77", "op": "linear_back", "m": 77, "n": 2001, "k": 1040, "type": "fp32"},
        # Gradients of a training batch through the 8B block's down projection.
        {"name": "linear_back_m2048", "op": "linear_back", "m": 2048, "n": 4096, "k": 12288, "type": "bf16"},
        # Gradients of one expert's share of a batch through its gate and up, binary16.
        {"name": "gate_up_back_m130", "op": "gate_up_back", "m": 130, "f": 768, "k": 2048, "type": "fp16"},
        # The largest: gradients of a training batch through the 8B block's gate and up.
        {"name": "gate_up_back_m4096", "op": "gate_up_back", "m": 4096, "f": 12288, "k": 4096, "type": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize_act", "quantize_weight", "linear", "linear", "linear", "gate_up", "gate_up",
                     "linear_back", "gate_up_back"])
    kind = rng.choice(sorted(TYPES))
    while True:
        m, n, k = _log_int(rng, 1, 4096), _log_int(rng, 48, 16384), 16 * _log_int(rng, 4, 768)
        rows = 2 * n if op.startswith("gate_up") else n
        if rows * k <= 24576 * 4096 and m * rows * k <= 2048 * 24576 * 4096:
            break
    if op == "quantize_act":
        return {"op": op, "m": m, "k": k, "type": kind, "pow2": rng.random() < 0.5}
    if op == "quantize_weight":
        return {"op": op, "n": n, "k": k, "type": kind, "pow2": rng.random() < 0.5}
    if op == "gate_up":
        return {"op": op, "m": m, "f": n, "k": k, "type": kind, "keep": rng.random() < 0.5}
    if op == "gate_up_back":
        return {"op": op, "m": m, "f": n, "k": k, "type": kind}
    return {"op": op, "m": m, "n": n, "k": k, "type": kind}


# ----------------------------------------------------------------------------- inputs


def _blocks(size):
    return (size + BLOCK - 1) // BLOCK


def _whole(x, rows, cols):
    """x with zeros up to whole blocks of `rows` rows and `cols` columns."""
    n, k = x.shape
    return torch.nn.functional.pad(x, (0, -k % cols, 0, -n % rows))


def _quantize(x, rows, pow2):
    """Codes (e4m3) and scales of blocks of `rows` rows and 128 columns, every step in float32."""
    n, k = x.shape
    x = _whole(x.float(), rows, BLOCK)
    x = x.view(x.shape[0] // rows, rows, x.shape[1] // BLOCK, BLOCK)
    top = x.abs().amax(dim=(1, 3))
    if pow2:
        part, power = torch.frexp(top)  # top = part 2^power, 1/2 <= part < 1; 448 = 7/8 2^9
        scale = torch.ldexp(torch.ones_like(top), power - 9 + (part > 0.875).int())
        by = 1.0 / scale
    else:
        largest = torch.full_like(top, TOP)  # quotients of tensors: rounded once, no reciprocal
        scale, by = top / largest, largest / top
    scale, by = scale.masked_fill(top < TINY, 0.0), by.masked_fill(top < TINY, 0.0)
    code = (x * by[:, None, :, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return code.view(-1, x.shape[2] * BLOCK)[:n, :k].contiguous(), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = dict(case)
    kind, k = TYPES[case["type"]], case["k"]

    def inputs(rows):  # activations: one column in 64 several times larger than the rest
        return normal(rows, k) * torch.where(torch.rand(k, generator=gen, device=DEV) < 1 / 64, 8.0, 1.0)

    if case["op"] == "quantize_act":
        s["x"] = inputs(case["m"]).to(kind)
        return s
    if case["op"] == "quantize_weight":
        s["x"] = (0.02 * normal(case["n"], k)).to(kind)
        return s
    m, parts = case["m"], [case["f"]] * 2 if "f" in case else [case["n"]]
    s["parts"] = parts
    coded = [_quantize(0.02 * normal(n, k), BLOCK, False) for n in parts]
    s["wq"], s["wd"] = torch.cat([q for q, _ in coded]), torch.cat([d for _, d in coded])
    s["xq"], s["xd"] = _quantize(inputs(m), 1, False)
    if case["op"] == "linear_back":
        s["dy"] = (0.1 * normal(m, case["n"])).to(kind)
    if case["op"] == "gate_up_back":
        s["gu"] = (1.5 * normal(m, 2 * case["f"])).to(kind)
        s["dh"] = (0.1 * normal(m, case["f"])).to(kind)
    return s


# -------------------------------------------------------------------------- plain form


def _spread(d, rows, n, k):
    """A scale for each element of [n][k] from one for each block of `rows` x 128."""
    return d.repeat_interleave(rows, dim=0)[:n].repeat_interleave(BLOCK, dim=1)[:, :k]


def _weight(s):
    k, at, first, whole = s["k"], 0, 0, []
    for n in s["parts"]:
        d = s["wd"][first:first + _blocks(n)]
        whole.append(s["wq"][at:at + n].float() * _spread(d, BLOCK, n, k))
        at, first = at + n, first + _blocks(n)
    return torch.cat(whole)


def _input(s):
    return s["xq"].float() * _spread(s["xd"], 1, s["m"], s["k"])


def run(state):
    s = state
    if own:
        return _run_own(s)
    kind, op = TYPES[s["type"]], s["op"]
    if op == "quantize_act":
        return _quantize(s["x"], 1, s["pow2"])
    if op == "quantize_weight":
        return _quantize(s["x"], BLOCK, s["pow2"])
    w, x = _weight(s), _input(s)
    if op == "linear":
        return (x @ w.T).to(kind)
    if op == "gate_up":
        gu = x @ w.T
        g, u = gu[:, :s["f"]], gu[:, s["f"]:]
        h = (g / (1 + torch.exp(-g)) * u).to(kind)
        return (h, gu.to(kind)) if s["keep"] else h
    if op == "linear_back":
        dy = s["dy"].float()
    else:
        g, u, dh = s["gu"][:, :s["f"]].float(), s["gu"][:, s["f"]:].float(), s["dh"].float()
        sig = 1 / (1 + torch.exp(-g))
        dy = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * g * sig], dim=1)
    return (dy @ w).to(kind), (dy.T @ x).to(kind)


def _run_own(s):
    import block_quantized_weight_linear_amd as q8

    op = s["op"]
    if op == "quantize_act":
        return q8.f8_quantize_act(s["x"], pow2=s["pow2"])
    if op == "quantize_weight":
        return q8.f8_quantize_weight(s["x"], pow2=s["pow2"])
    operands = (s["wq"], s["wd"], s["xq"], s["xd"])
    if op == "linear":
        return q8.f8_linear(*operands, dtype=TYPES[s["type"]])
    if op == "gate_up":
        return q8.f8_linear_fused_gate_up_silu(*operands, dtype=TYPES[s["type"]], keep_gate_up=s["keep"])
    if op == "linear_back":
        return q8.f8_linear_backward(*operands, s["dy"])
    return q8.f8_linear_fused_gate_up_silu_backward(*operands, s["gu"], s["dh"])


# -------------------------------------------------------------------------------- work


def work(case):
    size, k = TYPES[case["type"]].itemsize, case["k"]
    if case["op"] == "quantize_act":
        m = case["m"]
        return {"bytes": m * k * (size + 1) + 4 * m * _blocks(k), "flops": 3 * m * k}
    if case["op"] == "quantize_weight":
        n = case["n"]
        return {"bytes": n * k * (size + 1) + 4 * _blocks(n) * _blocks(k), "flops": 3 * n * k}
    m = case["m"]
    n = 2 * case["f"] if "f" in case else case["n"]
    parts = [case["f"]] * 2 if "f" in case else [n]
    given = (m + n) * k + 4 * _blocks(k) * (m + sum(_blocks(p) for p in parts))
    if case["op"] in ("linear", "gate_up"):
        out = n if case["op"] == "linear" else case["f"] + (n if case["keep"] else 0)
        return {"bytes": given + m * out * size, "flops": 2 * m * n * k}
    grads = m * n * size if case["op"] == "linear_back" else m * (n + case["f"]) * size
    return {"bytes": given + grads + (m + n) * k * size, "flops": 4 * m * n * k}


# ------------------------------------------------------------------------------- exact

_E4M3 = None


def _code_values():
    """The 256 codes' values: sign, four bits of exponent (bias 7), three of fraction."""
    global _E4M3
    if _E4M3 is None:
        table = []
        for c in range(256):
            e, f = c >> 3 & 15, c & 7
            v = math.nan if c & 127 == 127 else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
            table.append(-v if c >> 7 else v)
        _E4M3 = torch.tensor(table, dtype=torch.float64, device=DEV)
    return _E4M3


def _exact_values(codes):
    return _code_values()[codes.view(torch.uint8).int()]


def _nearest_code_value(v):
    """The e4m3 value nearest to each of v (at most 448 in magnitude), ties to the even code."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.round(v / step) * step


def _exact_quantized(x, rows, pow2):
    n, k = x.shape
    values = torch.zeros((n, k), dtype=torch.float64, device=DEV)
    scales = torch.zeros((-(-n // rows), -(-k // BLOCK)), dtype=torch.float64, device=DEV)
    whole = x.to(torch.float64)
    for b in range(scales.shape[1]):
        cols = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
        part = whole[:, cols]
        top = part.abs().max(dim=1).values
        if rows > 1:
            top = torch.stack([t.max() for t in top.split(rows)])
        live = top >= TINY
        # the definition rounds each quotient and each product to float32
        if pow2:
            scale = torch.exp2(torch.ceil(torch.log2(torch.where(live, top, 1.0) / TOP)))
            by = 1 / scale
        else:
            scale = (top / TOP).to(torch.float32).to(torch.float64)
            by = (TOP / torch.where(live, top, 1.0)).to(torch.float32).to(torch.float64)
        scales[:, b] = torch.where(live, scale, 0.0)
        by = torch.where(live, by, 0.0).repeat_interleave(rows)[:n, None]
        product = (part * by).to(torch.float32).to(torch.float64)
        values[:, cols] = _nearest_code_value(torch.clamp(product, -TOP, TOP))
    return values, scales


def _exact_matrix(codes, d, rows):
    v = _exact_values(codes)
    for b in range(d.shape[1]):
        v[:, b * BLOCK:(b + 1) * BLOCK] *= d[:, b].to(torch.float64).repeat_interleave(rows)[:v.shape[0], None]
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("quantize_act", "quantize_weight"):
        return _exact_quantized(s["x"], 1 if op == "quantize_act" else BLOCK, case["pow2"])
    x = _exact_matrix(s["xq"], s["xd"], 1)
    if "f" not in case:
        w = _exact_matrix(s["wq"], s["wd"], BLOCK)
        if op == "linear":
            return torch.matmul(x, w.t())
        dy = s["dy"].to(torch.float64)
        return torch.matmul(dy, w), torch.matmul(dy.t(), x)
    f = case["f"]
    half = s["wd"].shape[0] // 2
    gate = _exact_matrix(s["wq"][:f], s["wd"][:half], BLOCK)
    up = _exact_matrix(s["wq"][f:], s["wd"][half:], BLOCK)
    if op == "gate_up":
        g, u = torch.matmul(x, gate.t()), torch.matmul(x, up.t())
        h = g * torch.sigmoid(g) * u
        return (h, torch.hstack((g, u))) if case["keep"] else h
    gu = s["gu"].to(torch.float64)
    g, u, dh = gu[:, :f], gu[:, f:], s["dh"].to(torch.float64)
    sig = torch.sigmoid(g)
    dg, du = dh * u * (sig + g * sig * (1 - sig)), dh * g * sig
    return torch.matmul(dg, gate) + torch.matmul(du, up), torch.vstack((torch.matmul(dg.t(), x), torch.matmul(du.t(), x)))
