"""The expert step of an MoE layer, as it is measured: the gate, the experts'
gated feed-forward, the experts' product with its epilogue, and the combine's
gradient, each in its plain form (elementary torch operations in float32) and
as calls of this package.

A case is a dict; ``op`` names the operator:

* ``gate``: routing scores [tokens, experts] -> the top-k experts of each
  token and their softmax weights, or (``back``) the scores' gradient;
* ``gated``: rows grouped by expert, H = act(X Wg^T) * (X Wu^T), or (``back``)
  the gradients of X, Wg and Wu;
* ``linear``: rows grouped by expert, Y = act(X W^T + b) + R, or (``back``)
  the gradients of X, W and b;
* ``combine_back``: the gradient of the weighted sum over each token's expert
  rows, for the rows and for the weights.

Group sizes follow from the case (``spread``: sizes fall off as
1/(i+1)^spread over the groups that are not ``empty``); which expert gets
which size follows from the seed.
"""

import math

import torch

own = False

ACTIVATIONS = ("silu", "gelu", "gelu_tanh", "relu", "none")


# ---- cases ------------------------------------------------------------------

def _gate(tokens, experts, topk, dtype, renorm, masked, back=False):
    return {"op": "gate", "tokens": tokens, "experts": experts, "topk": topk, "dtype": dtype, "renorm": renorm,
            "masked": masked, "back": back}


def _gated(rows, tail, groups, empty, hidden, inner, act, spread, save=False, back=False):
    return {"op": "gated", "rows": rows, "tail": tail, "groups": groups, "empty": empty, "hidden": hidden,
            "inner": inner, "act": act, "spread": spread, "save": save, "back": back}


def _linear(rows, tail, groups, empty, inner, out, act, spread, bias, residual, save=False, back=False):
    return {"op": "linear", "rows": rows, "tail": tail, "groups": groups, "empty": empty, "inner": inner, "out": out,
            "act": act, "spread": spread, "bias": bias, "residual": residual, "save": save, "back": back}


def _combine(tokens, ranks, hidden, experts, topk):
    return {"op": "combine_back", "tokens": tokens, "ranks": ranks, "hidden": hidden, "experts": experts, "topk": topk}


def listed():
    cases = [
        # One decode step of 16 sequences: the smallest call, latency only.
        ("gate-decode", _gate(16, 256, 8, "f32", False, 0.0)),
        # A prompt batch with a quarter of the experts masked out per token.
        ("gate-prompt", _gate(32768, 256, 8, "bf16", True, 0.25)),
        # The training step's gradient of the scores.
        ("gate-back", _gate(16384, 128, 6, "f32", False, 0.0, back=True)),
        # Decode on one rank of eight: 32 of 256 experts, 24 of them hit by one
        # row each; the weights are all that is read.
        ("gated-decode", _gated(24, 0, 32, 8, 7168, 2048, "silu", 0.0)),
        # One rank's share of 4096 tokens, top-8 of 256 experts over 8 ranks:
        # about 128 rows per expert, uneven.
        ("gated-rank", _gated(4096, 0, 32, 0, 7168, 2048, "silu", 0.5)),
        # Training forward with a few experts per rank: bound by the products;
        # keeps both projections for the backward pass.
        ("gated-train", _gated(16384, 0, 8, 0, 4096, 4096, "silu", 0.2, save=True)),
        # Training backward at ragged sizes: an odd inner width, empty experts,
        # unused rows behind the last one.
        ("gated-back", _gated(12007, 89, 9, 2, 4088, 2001, "gelu_tanh", 0.3, back=True)),
        # The down projection of the same decode step.
        ("linear-decode", _linear(24, 0, 32, 8, 2048, 7168, "none", 0.0, False, False)),
        # A dense projection with the whole epilogue (one group, a last partial
        # block of rows).
        ("linear-dense", _linear(8000, 0, 1, 0, 4096, 8192, "gelu", 0.0, True, True)),
        # The down projection's training backward.
        ("linear-back", _linear(8192, 0, 16, 0, 2048, 7168, "none", 0.4, True, False, back=True)),
        # A small batch's combine gradient, and the full workload's.
        ("combine-back-small", _combine(128, 1, 4096, 64, 4)),
        ("combine-back", _combine(4096, 8, 7168, 256, 8)),
    ]
    return [{"name": n, **c} for n, c in cases]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row width: mostly multiples of 64, then multiples of 8, then any."""
    n = _log(rng, lo, hi)
    kind = rng.random()
    if kind < 0.5:
        return max(64, n // 64 * 64)
    if kind < 0.8:
        return max(8, n // 8 * 8)
    return n


# The largest listed products, in operations.
_MOST = 1.0e12


def draw(rng):
    op = rng.choice(["gate", "gated", "gated", "linear", "linear", "combine_back"])
    if op == "gate":
        experts = rng.choice([_log(rng, 4, 1024), 64, 128, 256])
        topk = rng.randint(1, min(16, experts))
        tokens = _log(rng, 1, 32768 * 256 // max(256, experts))
        return _gate(tokens, experts, topk, rng.choice(["f32", "bf16"]), rng.random() < 0.5,
                     rng.choice([0.0, 0.0, 0.25, 0.9]), rng.random() < 0.4)
    if op == "combine_back":
        ranks = rng.choice([1, 2, 4, 8])
        experts = ranks * rng.choice([2, 8, 32])
        topk = rng.randint(1, min(8, experts))
        hidden = _width(rng, 64, 7168)
        tokens = ranks * _log(rng, 1, max(2, min(4096, 4096 * 7168 // hidden) // ranks))
        return _combine(tokens, ranks, hidden, experts, topk)
    back = rng.random() < 0.45
    groups = _log(rng, 1, 32)
    empty = rng.randint(0, groups // 3)
    a, b = _width(rng, 64, 7168), _width(rng, 64, 4096)
    per_row = a * b * (4 if op == "gated" else 2) * (2 if back else 1)
    rows = _log(rng, 1, max(2, min(32768, int(_MOST / per_row))))
    tail = rng.choice([0, 0, rng.randint(1, 300)])
    act, spread = rng.choice(ACTIVATIONS[:4]), rng.choice([0.0, 0.3, 1.0])
    if op == "gated":
        return _gated(rows, tail, groups, empty, a, b, act, spread, rng.random() < 0.5, back)
    if rng.random() < 0.5:
        a, b = b, a
    return _linear(rows, tail, groups, empty, a, b, rng.choice([act, "none"]), spread, rng.random() < 0.5,
                   rng.random() < 0.5 and not back, rng.random() < 0.3 and not back, back)


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


def _grad_activation(case):
    return case["op"] == "linear" and case["act"] != "none"


def work(case):
    """Bytes with every input read once and every output written once (the
    weights of groups without rows are not read), and the products' operations."""
    op = case["op"]
    if op == "gate":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        size = 4 if case["dtype"] == "f32" else 2
        if case["back"]:
            return {"bytes": t * (2 * e * size + 8 * k), "flops": 6 * t * e}
        return {"bytes": t * (e * size + 8 * k), "flops": 4 * t * e}
    if op == "combine_back":
        t, k, h = case["tokens"], case["topk"], case["hidden"]
        return {"bytes": t * h * 2 * (1 + 2 * k) + t * k * 12, "flops": 3 * t * k * h}
    n, groups = case["rows"], case["groups"]
    live = sum(1 for s in _sizes(case) if s)
    if op == "gated":
        h, f = case["hidden"], case["inner"]
        weights = 2 * 2 * h * f
        if case["back"]:
            return {"bytes": 2 * n * (2 * h + 3 * f) + live * weights + groups * weights,
                    "flops": 2 * n * 4 * h * f}
        return {"bytes": 2 * n * (h + f * (3 if case["save"] else 1)) + live * weights, "flops": 2 * n * 2 * h * f}
    a, b = case["inner"], case["out"]
    weights = 2 * a * b
    if case["back"]:
        pre = b if _grad_activation(case) else 0
        return {"bytes": 2 * n * (2 * a + b + pre) + live * weights + groups * (weights + 2 * b * case["bias"]),
                "flops": 2 * n * 2 * a * b}
    rows = a + b * (1 + case["residual"] + case["save"])
    return {"bytes": 2 * n * rows + live * (weights + 2 * b * case["bias"]), "flops": 2 * n * a * b}


# ---- inputs -----------------------------------------------------------------

def _normal(gen, shape, scale=1.0, dtype=torch.bfloat16):
    """Normal values, drawn one leading slice at a time where that is large."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    parts = out if len(shape) == 3 else [out]
    for part in parts:
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * scale)
    return out


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
    op = case["op"]
    s = {"case": case}
    if op == "gate":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        logits = _normal(gen, (t, e), 1.0, torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        if case["masked"]:
            logits.masked_fill_(torch.rand(t, e, generator=gen, device="cuda") < case["masked"], float("-inf"))
        s["logits"] = logits
        if case["back"]:
            s["idx"] = torch.sort(logits.float(), dim=1, descending=True, stable=True).indices[:, :k].int().contiguous()
            s["d_w"] = _normal(gen, (t, k), 1.0, torch.float32)
        return s
    if op == "combine_back":
        t, k, h, e = case["tokens"], case["topk"], case["hidden"], case["experts"]
        logits = torch.randn(t, e, generator=gen, device="cuda")
        top = torch.sort(torch.softmax(logits, 1), dim=1, descending=True, stable=True)
        s["idx"] = top.indices[:, :k].int().contiguous()
        s["w"] = top.values[:, :k].contiguous()
        s["d_y"] = _normal(gen, (t, h))
        s["z"] = _normal(gen, (t * k, h))
        # The arena row of each (token, choice): by expert, then by token.
        pair = s["idx"].long() * t + torch.arange(t, device="cuda")[:, None]
        s["slot"] = torch.argsort(torch.argsort(pair.reshape(-1))).reshape(t, k)
        return s
    n = case["rows"] + case["tail"]
    g = case["groups"]
    s["host"], s["offsets"] = _offsets(case, seed)
    if op == "gated":
        h, f = case["hidden"], case["inner"]
        s["x"] = _normal(gen, (n, h))
        s["w_gate"] = _normal(gen, (g, f, h), h ** -0.5)
        s["w_up"] = _normal(gen, (g, f, h), h ** -0.5)
        if case["back"]:
            s["gate"], s["up"], s["d_h"] = _normal(gen, (n, f)), _normal(gen, (n, f)), _normal(gen, (n, f))
        return s
    a, b = case["inner"], case["out"]
    s["x"] = _normal(gen, (n, a))
    s["w"] = _normal(gen, (g, b, a), a ** -0.5)
    s["bias"] = _normal(gen, (g, b)) if case["bias"] else None
    s["residual"] = _normal(gen, (n, b)) if case["residual"] else None
    if case["back"]:
        s["d_y"] = _normal(gen, (n, b))
        s["pre"] = _normal(gen, (n, b)) if _grad_activation(case) else None
    return s


def prepare(case, seed):
    """Inputs, output buffers and (where the framework's calls are measured)
    the routed plan and workspace that a program keeps between steps."""
    s = _inputs(case, seed)
    op = case["op"]
    zeros = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")
    if op == "gate":
        t, e, k = case["tokens"], case["experts"], case["topk"]
        if case["back"]:
            s["d_logits"] = torch.zeros_like(s["logits"])
        else:
            s["out_idx"], s["out_w"] = zeros(t, k, dtype=torch.int32), zeros(t, k, dtype=torch.float32)
    elif op == "combine_back":
        s["d_z"], s["d_w"] = torch.zeros_like(s["z"]), torch.zeros_like(s["w"])
        if own:
            import reduce_rank_buffers_amd as rrb
            r, t = case["ranks"], case["tokens"]
            s["plan"] = rrb.MoeDevicePlan(r, t, case["hidden"], case["experts"], case["topk"], "combine")
            s["plan"].route(s["idx"], s["w"])
            s["d_y_ranks"] = list(s["d_y"].reshape(r, t // r, case["hidden"]).unbind(0))
    elif op == "gated":
        n, f = case["rows"] + case["tail"], case["inner"]
        if case["back"]:
            s["d_x"], s["d_w_gate"], s["d_w_up"] = (torch.zeros_like(s[q]) for q in ("x", "w_gate", "w_up"))
            if own:
                import reduce_rank_buffers_amd as rrb
                s["work"] = torch.empty(rrb.expert_gated_backward_workspace(n, case["hidden"], f, case["groups"]),
                                        dtype=torch.uint8, device="cuda")
        else:
            s["h"] = zeros(n, f)
            s["gate"], s["up"] = (zeros(n, f), zeros(n, f)) if case["save"] else (None, None)
    else:
        n, b = case["rows"] + case["tail"], case["out"]
        if case["back"]:
            s["d_x"], s["d_weight"] = torch.zeros_like(s["x"]), torch.zeros_like(s["w"])
            s["d_bias"] = torch.zeros_like(s["bias"]) if case["bias"] else None
            if own:
                import reduce_rank_buffers_amd as rrb
                s["work"] = torch.empty(rrb.expert_linear_backward_workspace(n, case["inner"], b, case["groups"]),
                                        dtype=torch.uint8, device="cuda")
        else:
            s["y"] = zeros(n, b)
            s["pre_out"] = zeros(n, b) if case["save"] else None
    return s


# ---- one pass ---------------------------------------------------------------

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _kept(*outputs):
    return [t for t in outputs if t is not None]


def _own_gate(s):
    import reduce_rank_buffers_amd as rrb
    renorm = s["case"]["renorm"]
    if s["case"]["back"]:
        rrb.moe_gate_backward(s["logits"], s["idx"], s["d_w"], s["d_logits"], renormalize=renorm)
        return [s["d_logits"]]
    rrb.moe_gate(s["logits"], s["out_idx"], s["out_w"], renormalize=renorm)
    return [s["out_idx"], s["out_w"]]


def _own_gated(s):
    import reduce_rank_buffers_amd as rrb
    act = s["case"]["act"]
    if s["case"]["back"]:
        rrb.expert_gated_backward(s["d_h"], s["x"], s["offsets"], s["w_gate"], s["w_up"], s["gate"], s["up"],
                                  activation=act, d_x=s["d_x"], d_w_gate=s["d_w_gate"], d_w_up=s["d_w_up"],
                                  workspace=s["work"])
        return [s["d_x"], s["d_w_gate"], s["d_w_up"]]
    rrb.expert_gated(s["x"], s["offsets"], s["w_gate"], s["w_up"], s["h"], activation=act, save_gate=s["gate"],
                     save_up=s["up"])
    return _kept(s["h"], s["gate"], s["up"])


def _own_linear(s):
    import reduce_rank_buffers_amd as rrb
    act = s["case"]["act"]
    if s["case"]["back"]:
        rrb.expert_linear_backward(s["d_y"], s["x"], s["offsets"], s["w"], pre=s["pre"], activation=act,
                                   d_x=s["d_x"], d_w=s["d_weight"], d_bias=s["d_bias"], workspace=s["work"])
        return _kept(s["d_x"], s["d_weight"], s["d_bias"])
    rrb.expert_linear(s["x"], s["offsets"], s["w"], s["y"], bias=s["bias"], activation=act, residual=s["residual"],
                      save_pre=s["pre_out"])
    return _kept(s["y"], s["pre_out"])


def _own_combine_back(s):
    ranks = s["case"]["ranks"]
    s["plan"].backward(s["d_y_ranks"], [s["z"]] + [None] * (ranks - 1), [s["d_z"]] + [None] * (ranks - 1),
                       d_weights=s["d_w"])
    return [s["d_z"], s["d_w"]]


_OWN = {"gate": _own_gate, "gated": _own_gated, "linear": _own_linear, "combine_back": _own_combine_back}


def _act(name, x):
    """The activation and its derivative."""
    if name == "none":
        return x, torch.ones_like(x)
    if name == "relu":
        on = (x > 0).to(x.dtype)
        return x * on, on
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return x * s, s * (1.0 + x * (1.0 - s))
    if name == "gelu":
        c = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * c, c + x * torch.exp(-0.5 * x * x) * math.sqrt(0.5 / math.pi)
    c = math.sqrt(2.0 / math.pi)
    th = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1.0 + th), 0.5 * (1.0 + th) + 0.5 * x * (1.0 - th * th) * c * (1.0 + 3 * 0.044715 * x * x)


def _masked_exp(logits):
    """exp(l - max) per row, and its sum; a row of -inf alone gives zeros, and
    the sum 1 in its place."""
    top = logits.max(dim=1, keepdim=True).values
    e = torch.exp(logits - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = e.sum(dim=1, keepdim=True)
    return e, torch.where(total == 0, torch.ones_like(total), total)


def _plain_gate(s):
    c = s["case"]
    logits = s["logits"].float()
    e, total = _masked_exp(logits)
    if not c["back"]:
        idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :c["topk"]]
        sel = torch.gather(e, 1, idx)
        if c["renorm"]:
            total = sel.sum(dim=1, keepdim=True)
            total = torch.where(total == 0, torch.ones_like(total), total)
        return [idx.int(), sel / total]
    idx = s["idx"].long()
    sel = torch.gather(e, 1, idx)
    if c["renorm"]:
        total = sel.sum(dim=1, keepdim=True)
        total = torch.where(total == 0, torch.ones_like(total), total)
        w = sel / total
        d = torch.zeros_like(e).scatter(1, idx, w * (s["d_w"] - (w * s["d_w"]).sum(dim=1, keepdim=True)))
    else:
        p = e / total
        mean = (sel / total * s["d_w"]).sum(dim=1, keepdim=True)
        d = p * (torch.zeros_like(e).scatter(1, idx, s["d_w"]) - mean)
    return [d.to(s["logits"].dtype)]


def _groups(s):
    return [(e, a, b) for e, (a, b) in enumerate(zip(s["host"], s["host"][1:]))]


def _plain_gated(s):
    c = s["case"]
    if not c["back"]:
        for e, a, b in _groups(s):
            if a == b:
                continue
            x = s["x"][a:b].float()
            gate, up = x @ s["w_gate"][e].float().T, x @ s["w_up"][e].float().T
            s["h"][a:b] = (_act(c["act"], gate)[0] * up).to(torch.bfloat16)
            if c["save"]:
                s["gate"][a:b], s["up"][a:b] = gate.to(torch.bfloat16), up.to(torch.bfloat16)
        return _kept(s["h"], s["gate"], s["up"])
    for e, a, b in _groups(s):
        x, d_h = s["x"][a:b].float(), s["d_h"][a:b].float()
        f, df = _act(c["act"], s["gate"][a:b].float())
        d_gate, d_up = d_h * s["up"][a:b].float() * df, d_h * f
        s["d_w_gate"][e] = (d_gate.T @ x).to(torch.bfloat16)
        s["d_w_up"][e] = (d_up.T @ x).to(torch.bfloat16)
        s["d_x"][a:b] = (d_gate @ s["w_gate"][e].float() + d_up @ s["w_up"][e].float()).to(torch.bfloat16)
    return [s["d_x"], s["d_w_gate"], s["d_w_up"]]


def _plain_linear(s):
    c = s["case"]
    if not c["back"]:
        for e, a, b in _groups(s):
            if a == b:
                continue
            pre = s["x"][a:b].float() @ s["w"][e].float().T
            if c["bias"]:
                pre = pre + s["bias"][e].float()
            y = _act(c["act"], pre)[0]
            if c["residual"]:
                y = y + s["residual"][a:b].float()
            s["y"][a:b] = y.to(torch.bfloat16)
            if c["save"]:
                s["pre_out"][a:b] = pre.to(torch.bfloat16)
        return _kept(s["y"], s["pre_out"])
    for e, a, b in _groups(s):
        d = s["d_y"][a:b].float()
        if s["pre"] is not None:
            d = d * _act(c["act"], s["pre"][a:b].float())[1]
        s["d_weight"][e] = (d.T @ s["x"][a:b].float()).to(torch.bfloat16)
        s["d_x"][a:b] = (d @ s["w"][e].float()).to(torch.bfloat16)
        if c["bias"]:
            s["d_bias"][e] = d.sum(dim=0).to(torch.bfloat16)
    return _kept(s["d_x"], s["d_weight"], s["d_bias"])


def _plain_combine_back(s):
    d_y = s["d_y"].float()
    for j in range(s["case"]["topk"]):
        at = s["slot"][:, j]
        s["d_w"][:, j] = (d_y * s["z"][at].float()).sum(dim=1)
        s["d_z"][at] = (s["w"][:, j:j + 1] * d_y).to(torch.bfloat16)
    return [s["d_z"], s["d_w"]]


_PLAIN = {"gate": _plain_gate, "gated": _plain_gated, "linear": _plain_linear, "combine_back": _plain_combine_back}


# ---- the definition in 64 bits ----------------------------------------------

def _phi(name, x):
    """The activations as torch's own functions define them, for autograd."""
    from torch.nn import functional as F
    return {"none": lambda v: v, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}[name](x)


def _softmax64(logits):
    """Softmax of the finite scores of each row (0 where there are none)."""
    x = logits.double()
    p = torch.softmax(x.masked_fill(x == float("-inf"), -1e300), dim=1)
    return p * (x != float("-inf"))


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "gate":
        k = case["topk"]
        if not case["back"]:
            keys = s["logits"].double()
            idx = torch.sort(-keys, dim=1, stable=True).indices[:, :k]
            w = torch.gather(_softmax64(s["logits"]), 1, idx)
            if case["renorm"]:
                w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
            return [idx.int(), w]
        with torch.enable_grad():
            leaf = s["logits"].double().masked_fill(s["logits"] == float("-inf"), -1e4).requires_grad_()
            real = (s["logits"] != float("-inf")).double()
            w = torch.gather(torch.softmax(leaf, 1) * real, 1, s["idx"].long())
            if case["renorm"]:
                w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
            (w * s["d_w"].double()).sum().backward()
        return [leaf.grad * real]
    if op == "combine_back":
        flat = s["slot"].reshape(-1)
        rows = s["d_y"].double().repeat_interleave(case["topk"], dim=0)
        d_z = torch.empty(s["z"].shape, dtype=torch.float64, device="cuda")
        d_z[flat] = rows * s["w"].double().reshape(-1, 1)
        d_w = torch.linalg.vecdot(rows, s["z"][flat].double()).reshape(s["w"].shape)
        return [d_z, d_w]
    n = case["rows"] + case["tail"]
    zeros = lambda like, *shape: torch.zeros(shape or like.shape, dtype=torch.float64, device="cuda")
    at = [slice(a, b) for a, b in zip(s["host"], s["host"][1:])]
    if op == "gated":
        if not case["back"]:
            gate, up = zeros(None, n, case["inner"]), zeros(None, n, case["inner"])
            for e, r in enumerate(at):
                x = s["x"][r].double()
                gate[r] = torch.nn.functional.linear(x, s["w_gate"][e].double())
                up[r] = torch.nn.functional.linear(x, s["w_up"][e].double())
            h = _phi(case["act"], gate) * up
            return [h, gate, up] if case["save"] else [h]
        with torch.enable_grad():
            gate, up = s["gate"].double().requires_grad_(), s["up"].double().requires_grad_()
            (_phi(case["act"], gate) * up).backward(s["d_h"].double())
        d_x, d_wg, d_wu = zeros(s["x"]), zeros(s["w_gate"]), zeros(s["w_up"])
        for e, r in enumerate(at):
            x = s["x"][r].double()
            d_x[r] = torch.cat([gate.grad[r], up.grad[r]], 1) @ torch.cat([s["w_gate"][e], s["w_up"][e]], 0).double()
            d_wg[e], d_wu[e] = gate.grad[r].T @ x, up.grad[r].T @ x
        return [d_x, d_wg, d_wu]
    if not case["back"]:
        pre, y = zeros(None, n, case["out"]), zeros(None, n, case["out"])
        for e, r in enumerate(at):
            bias = s["bias"][e].double() if case["bias"] else None
            pre[r] = torch.nn.functional.linear(s["x"][r].double(), s["w"][e].double(), bias)
            y[r] = _phi(case["act"], pre[r])
            if case["residual"]:
                y[r] += s["residual"][r].double()
        return [y, pre] if case["save"] else [y]
    d = s["d_y"].double()
    if s["pre"] is not None:
        with torch.enable_grad():
            leaf = s["pre"].double().requires_grad_()
            _phi(case["act"], leaf).backward(d)
        d = leaf.grad
    d_x, d_w = zeros(s["x"]), zeros(s["w"])
    d_b = zeros(s["bias"]) if case["bias"] else None
    for e, r in enumerate(at):
        d_x[r] = d[r] @ s["w"][e].double()
        d_w[e] = d[r].T @ s["x"][r].double()
        if case["bias"]:
            d_b[e] = torch.ones(1, d[r].shape[0], dtype=torch.float64, device="cuda").matmul(d[r])[0]
    return _kept(d_x, d_w, d_b)
