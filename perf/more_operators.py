"""Serving an MoE layer, as it is measured: the experts' products in 8-bit
integers and the whole expert layer for a few tokens, each in its plain form
(elementary torch operations in float32, float64 where a value is rounded to
an integer) and as calls of this package.

A case is a dict; ``op`` names the operator:

* ``linear8``: rows grouped by expert, quantised row by row, then
  Y = act((Xq Wq^T) sx sw + b) + R with weights held in 8-bit integers and a
  scale for each output channel;
* ``gated8``: the same rows, H = act((Xq Gq^T) sx sg) * ((Xq Uq^T) sx su);
* ``decode``: for each of a few tokens, the sum over its chosen experts of
  w_j Wd[e_j] (act(Wg[e_j] x) * (Wu[e_j] x)); weights in bf16, or (``int8``) in
  8-bit integers with a scale for each channel.  Choices outside the experts
  that are here take no part.

A row's scale is max |x| / 127 in float32 and its values are x over that
scale, rounded to the nearest integer, ties to even; a row of zeros has the
scale 0.
"""

import math

import torch

own = False

ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "relu", "none")


# ---- cases ------------------------------------------------------------------

def _linear(rows, tail, groups, empty, inner, out, act, spread, bias, residual, dtype="bf16"):
    return {"op": "linear8", "rows": rows, "tail": tail, "groups": groups, "empty": empty, "inner": inner, "out": out,
            "act": act, "spread": spread, "bias": bias, "residual": residual, "dtype": dtype}


def _gated(rows, tail, groups, empty, hidden, inner, act, spread, dtype="bf16"):
    return {"op": "gated8", "rows": rows, "tail": tail, "groups": groups, "empty": empty, "hidden": hidden,
            "inner": inner, "act": act, "spread": spread, "dtype": dtype}


def _decode(tokens, topk, experts, ranks, hidden, inner, act, int8):
    return {"op": "decode", "tokens": tokens, "topk": topk, "experts": experts, "ranks": ranks, "hidden": hidden,
            "inner": inner, "act": act, "int8": int8}


def listed():
    cases = [
        # The down projection of a decode step on one rank of eight: 24 rows,
        # each of another expert, 8 of the 32 experts without any.
        ("linear8-decode", _linear(24, 0, 32, 8, 2048, 7168, "none", 0.0, False, False)),
        # A prompt's dense projection with the whole epilogue (one group, a last
        # partial block of rows): bound by the products.
        ("linear8-dense", _linear(8000, 0, 1, 0, 4096, 8192, "gelu", 0.0, True, True)),
        # Ragged groups of float32 rows with odd widths, unused rows behind.
        ("linear8-odd", _linear(3001, 39, 9, 2, 2001, 1111, "silu", 0.3, True, False, "f32")),
        # A small batch on two experts: few rows, few tiles.
        ("gated8-small", _gated(40, 8, 2, 0, 1024, 512, "gelu_tanh", 0.0)),
        # One rank's share of 4096 tokens, top-8 of 256 experts over 8 ranks.
        ("gated8-rank", _gated(4096, 0, 32, 0, 7168, 2048, "silu", 0.5)),
        # A long prompt on few experts: bound by the products.
        ("gated8-prompt", _gated(16384, 0, 8, 0, 4096, 4096, "silu", 0.2)),
        # One sequence's token on a small layer: latency counts.
        ("decode-small", _decode(1, 8, 64, 1, 2048, 1024, "silu", False)),
        # One sequence's token on the full widths, every weight read once.
        ("decode-one", _decode(1, 8, 32, 1, 7168, 2048, "silu", False)),
        # A decode step of 64 sequences on one rank of eight: seven choices in
        # eight are other ranks', the others meet on 32 experts.
        ("decode-rank", _decode(64, 8, 32, 8, 7168, 2048, "silu", False)),
        # The widths of neither a power of two nor whole 16-byte rows.
        ("decode-odd", _decode(5, 3, 12, 2, 1001, 333, "gelu", False)),
        # Weights in 8 bits: one token, and a step of 16 sequences.
        ("decode8-one", _decode(1, 8, 32, 1, 7168, 2048, "silu", True)),
        ("decode8-batch", _decode(16, 4, 32, 1, 4096, 2048, "gelu_tanh", True)),
    ]
    return [{"name": n, **c} for n, c in cases]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row width: mostly multiples of 64, then multiples of 16, then any."""
    n = _log(rng, lo, hi)
    kind = rng.random()
    if kind < 0.5:
        return max(64, n // 64 * 64)
    if kind < 0.8:
        return max(16, n // 16 * 16)
    return n


# The largest listed products, in operations, and the largest listed layer, in
# weights of one matrix and in weights that tokens meet.
_MOST = 1.0e12
_MOST_WEIGHTS = 32 * 7168 * 2048
_MOST_MET = 64 * 8 * 7168 * 2048


def draw(rng):
    op = rng.choice(["linear8", "gated8", "decode", "decode"])
    if op == "decode":
        hidden, inner = _width(rng, 256, 7168), _width(rng, 64, 4096)
        experts = _log(rng, 1, max(1, min(128, _MOST_WEIGHTS // (hidden * inner))))
        ranks = rng.choice([1, 1, 2, 8])
        topk = rng.randint(1, min(8, experts * ranks))
        tokens = _log(rng, 1, max(1, min(64, _MOST_MET // (topk * hidden * inner))))
        return _decode(tokens, topk, experts, ranks, hidden, inner, rng.choice(ACTIVATIONS[:4]), rng.random() < 0.5)
    groups = _log(rng, 1, 32)
    empty = rng.randint(0, groups // 3)
    a, b = _width(rng, 64, 7168), _width(rng, 64, 4096)
    rows = _log(rng, 1, max(2, min(32768, int(_MOST / (a * b * (4 if op == "gated8" else 2))))))
    tail = rng.choice([0, 0, rng.randint(1, 300)])
    act, spread, dtype = rng.choice(ACTIVATIONS[:4]), rng.choice([0.0, 0.3, 1.0]), rng.choice(["bf16", "bf16", "f32"])
    if op == "gated8":
        return _gated(rows, tail, groups, empty, a, b, act, spread, dtype)
    if rng.random() < 0.5:
        a, b = b, a
    return _linear(rows, tail, groups, empty, a, b, rng.choice([act, "none"]), spread, rng.random() < 0.5,
                   rng.random() < 0.5, dtype)


# ---- sizes ------------------------------------------------------------------

def _sizes(case):
    """Rows of each group that has any, largest first; then the empty ones."""
    live = case["groups"] - case["empty"]
    share = [1.0 / (i + 1) ** case["spread"] for i in range(live)]
    total = sum(share)
    cut = [int(case["rows"] * s / total) for s in share]
    for i in range(case["rows"] - sum(cut)):
        cut[i % live] += 1
    return cut + [0] * case["empty"]


def work(case):
    """Bytes with every input read once and every output written once (the
    weights of groups without rows, and of experts without tokens, are not
    read), and the products' operations."""
    if case["op"] == "decode":
        t, k, h, f = case["tokens"], case["topk"], case["hidden"], case["inner"]
        # Choices that are here, and the experts that they are expected to meet
        # (all experts are equally likely, a token's are distinct).
        met = t * k / case["ranks"]
        live = case["experts"] * (1.0 - (1.0 - k / (case["experts"] * case["ranks"])) ** t)
        size = 1 if case["int8"] else 2
        scales = live * (2 * f + h) * 4 if case["int8"] else 0
        return {"bytes": live * 3 * h * f * size + scales + t * (2 * h * 2 + 8 * k), "flops": met * 3 * 2 * h * f}
    n, size = case["rows"], 2 if case["dtype"] == "bf16" else 4
    live = sum(1 for s in _sizes(case) if s)
    if case["op"] == "gated8":
        h, f = case["hidden"], case["inner"]
        return {"bytes": n * (size * h + 2 * f) + live * 2 * f * (h + 4), "flops": 2 * n * 2 * h * f}
    a, b = case["inner"], case["out"]
    return {"bytes": n * (size * a + 2 * b * (1 + case["residual"])) + live * b * (a + 4 + 2 * case["bias"]),
            "flops": 2 * n * a * b}


# ---- inputs -----------------------------------------------------------------

def _normal(gen, shape, scale=1.0, dtype=torch.bfloat16):
    """Normal values, drawn one leading slice at a time where that is large."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out if len(shape) == 3 else [out]:
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    return out


def _weights8(gen, groups, out, inner):
    """Normal weights held in 8 bits, as a channel whose largest is near four
    deviations is, and the channels' scales, some larger than others."""
    q = torch.empty(groups, out, inner, dtype=torch.int8, device="cuda")
    for part in q:
        part.copy_((torch.randn(part.shape, generator=gen, device="cuda") * 32).round_().clamp_(-127, 127))
    s = torch.exp(0.3 * torch.randn(groups, out, generator=gen, device="cuda")) * (inner ** -0.5 / 32)
    return q, s


def _rows(gen, case, width):
    """Rows whose sizes differ from one to the next."""
    n = case["rows"] + case["tail"]
    x = torch.randn(n, width, generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn(n, 1, generator=gen, device="cuda"))
    return x.to(torch.bfloat16) if case["dtype"] == "bf16" else x


def _offsets(case, seed):
    """Host and device offsets of the groups: the sizes in the seed's order."""
    sizes = _sizes(case)
    order = torch.randperm(len(sizes), generator=torch.Generator().manual_seed(seed + 17)).tolist()
    host = [0]
    for i in order:
        host.append(host[-1] + sizes[i])
    return host, torch.tensor(host, dtype=torch.int32, device="cuda")


def _inputs(case, seed):
    """The operator's inputs alone, from the case and the seed."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "decode":
        t, k, g, h, f = case["tokens"], case["topk"], case["experts"], case["hidden"], case["inner"]
        s["x"] = _normal(gen, (t, h))
        # Scores over the experts of every rank; this one's come first, in the
        # middle or last, and the others' have ids below 0 or past the end.
        scores = torch.randn(t, g * case["ranks"], generator=gen, device="cuda")
        top = torch.sort(torch.softmax(scores, 1), dim=1, descending=True, stable=True)
        s["idx"] = (top.indices[:, :k] - g * (seed % case["ranks"])).int().contiguous()
        s["w"] = (top.values[:, :k] / top.values[:, :k].sum(dim=1, keepdim=True)).contiguous()
        if case["int8"]:
            s["w_gate"], s["s_gate"] = _weights8(gen, g, f, h)
            s["w_up"], s["s_up"] = _weights8(gen, g, f, h)
            s["w_down"], s["s_down"] = _weights8(gen, g, h, f)
        else:
            s["w_gate"], s["w_up"] = _normal(gen, (g, f, h), h ** -0.5), _normal(gen, (g, f, h), h ** -0.5)
            s["w_down"] = _normal(gen, (g, h, f), f ** -0.5)
        return s
    g = case["groups"]
    s["host"], s["offsets"] = _offsets(case, seed)
    if case["op"] == "gated8":
        s["x"] = _rows(gen, case, case["hidden"])
        s["w_gate"], s["s_gate"] = _weights8(gen, g, case["inner"], case["hidden"])
        s["w_up"], s["s_up"] = _weights8(gen, g, case["inner"], case["hidden"])
        return s
    s["x"] = _rows(gen, case, case["inner"])
    s["w_q"], s["s_w"] = _weights8(gen, g, case["out"], case["inner"])
    s["bias"] = _normal(gen, (g, case["out"])) if case["bias"] else None
    s["residual"] = _normal(gen, (case["rows"] + case["tail"], case["out"])) if case["residual"] else None
    return s


def prepare(case, seed):
    """Inputs, output buffers, and the quantised rows' buffers or the workspace
    that a program keeps between steps."""
    s = _inputs(case, seed)
    if case["op"] == "decode":
        s["y"] = torch.zeros_like(s["x"])
        if own:
            import reduce_rank_buffers_amd as rrb
            s["work"] = torch.empty(rrb.moe_decode_workspace(case["tokens"], case["topk"], case["hidden"], case["inner"]),
                                    dtype=torch.uint8, device="cuda")
        return s
    n = case["rows"] + case["tail"]
    s["q"] = torch.zeros(s["x"].shape, dtype=torch.int8, device="cuda")
    s["s_x"] = torch.zeros(n, dtype=torch.float32, device="cuda")
    s["y"] = torch.zeros(n, case["inner" if case["op"] == "gated8" else "out"], dtype=torch.bfloat16, device="cuda")
    return s


# ---- one pass ---------------------------------------------------------------

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _own_linear(s):
    import reduce_rank_buffers_amd as rrb
    rrb.quantize_rows(s["x"], s["q"], s["s_x"], offsets=s["offsets"])
    rrb.expert_linear_int8(s["q"], s["s_x"], s["offsets"], s["w_q"], s["s_w"], s["y"], bias=s["bias"],
                           activation=s["case"]["act"], residual=s["residual"])
    return [s["y"]]


def _own_gated(s):
    import reduce_rank_buffers_amd as rrb
    rrb.quantize_rows(s["x"], s["q"], s["s_x"], offsets=s["offsets"])
    rrb.expert_gated_int8(s["q"], s["s_x"], s["offsets"], s["w_gate"], s["s_gate"], s["w_up"], s["s_up"], s["y"],
                          activation=s["case"]["act"])
    return [s["y"]]


def _own_decode(s):
    import reduce_rank_buffers_amd as rrb
    scales = (s["s_gate"], s["s_up"], s["s_down"]) if s["case"]["int8"] else None
    rrb.moe_decode(s["x"], s["idx"], s["w"], s["w_gate"], s["w_up"], s["w_down"], s["y"],
                   activation=s["case"]["act"], scales=scales, workspace=s["work"])
    return [s["y"]]


_OWN = {"linear8": _own_linear, "gated8": _own_gated, "decode": _own_decode}


def _act(name, x):
    if name == "none":
        return x
    if name == "relu":
        return x * (x > 0).to(x.dtype)
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _quantized(x):
    """Rows as integers (in float32), and their scales."""
    scale = (x.abs().max(dim=1, keepdim=True).values.double() / 127.0).float()
    div = torch.where(scale == 0, torch.ones_like(scale), scale)
    return torch.round(x.double() / div.double()).float(), scale


def _groups(s):
    return [(e, a, b) for e, (a, b) in enumerate(zip(s["host"], s["host"][1:])) if b > a]


def _plain_linear(s):
    q, scale = _quantized(s["x"])
    for e, a, b in _groups(s):
        pre = (q[a:b] @ s["w_q"][e].float().T) * scale[a:b] * s["s_w"][e]
        if s["bias"] is not None:
            pre = pre + s["bias"][e].float()
        y = _act(s["case"]["act"], pre)
        if s["residual"] is not None:
            y = y + s["residual"][a:b].float()
        s["y"][a:b] = y.to(torch.bfloat16)
    return [s["y"]]


def _plain_gated(s):
    q, scale = _quantized(s["x"])
    for e, a, b in _groups(s):
        gate = (q[a:b] @ s["w_gate"][e].float().T) * scale[a:b] * s["s_gate"][e]
        up = (q[a:b] @ s["w_up"][e].float().T) * scale[a:b] * s["s_up"][e]
        s["y"][a:b] = (_act(s["case"]["act"], gate) * up).to(torch.bfloat16)
    return [s["y"]]


def _plain_decode(s):
    c = s["case"]
    x = s["x"].float()[:, :, None]
    y = torch.zeros(c["tokens"], c["hidden"], device="cuda")
    here = (s["idx"] >= 0) & (s["idx"] < c["experts"])
    at = torch.where(here, s["idx"], torch.zeros_like(s["idx"])).long()

    def product(w, scale, e, v):
        z = (s[w][e].float() @ v)[:, :, 0]
        return z * s[scale][e] if c["int8"] else z

    for j in range(c["topk"]):
        e = at[:, j]
        h = _act(c["act"], product("w_gate", "s_gate", e, x)) * product("w_up", "s_up", e, x)
        z = product("w_down", "s_down", e, h[:, :, None])
        y = y + torch.where(here[:, j:j + 1], s["w"][:, j:j + 1] * z, torch.zeros_like(z))
    s["y"].copy_(y)
    return [s["y"]]


_PLAIN = {"linear8": _plain_linear, "gated8": _plain_gated, "decode": _plain_decode}


# ---- the definition in 64 bits ----------------------------------------------

def _phi(name, x):
    """The activations as torch's own functions define them."""
    from torch.nn import functional as F
    return {"none": lambda v: v, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name](x)


def exact(case, seed):
    s = _inputs(case, seed)
    linear = torch.nn.functional.linear
    if case["op"] == "decode":
        x, w = s["x"].double(), s["w"].double()
        y = torch.zeros_like(x)

        def weight(name, e):
            m = s["w_" + name][e].double()
            return m * s["s_" + name][e].double()[:, None] if case["int8"] else m

        for e in range(case["experts"]):
            share = (w * (s["idx"] == e)).sum(dim=1)
            t = share.nonzero()[:, 0]
            if t.numel():
                h = _phi(case["act"], linear(x[t], weight("gate", e))) * linear(x[t], weight("up", e))
                y[t] += share[t, None] * linear(h, weight("down", e))
        return [y]
    # The scale is the float32 nearest to max |x| / 127 by definition.
    x = s["x"].double()
    scale = torch.linalg.vector_norm(x, float("inf"), dim=1, keepdim=True).div(127).to(torch.float32).double()
    xq = torch.nan_to_num(x / scale, nan=0.0).round() * scale
    y = torch.zeros(s["x"].shape[0], case["inner" if case["op"] == "gated8" else "out"], dtype=torch.float64,
                    device="cuda")
    for e, (a, b) in enumerate(zip(s["host"], s["host"][1:])):
        if a == b:
            continue
        if case["op"] == "gated8":
            gate, up = (linear(xq[a:b], s["w_" + p][e].double() * s["s_" + p][e].double()[:, None])
                        for p in ("gate", "up"))
            y[a:b] = _phi(case["act"], gate) * up
            continue
        bias = s["bias"][e].double() if case["bias"] else None
        y[a:b] = _phi(case["act"], linear(xq[a:b], s["w_q"][e].double() * s["s_w"][e].double()[:, None], bias))
        if case["residual"]:
            y[a:b] += s["residual"][a:b].double()
    return [y]
