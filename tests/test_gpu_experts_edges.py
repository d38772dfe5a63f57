"""GPU tests of the experts' calls at their edges: what lies around the
operands, far tails, sizes past one launch, overlapping tensors, replayed
steps.  Against the binary64 oracle, with the bounds of
tests/test_gpu_experts.py (its docstring derives them)."""

import numpy as np
import pytest
import torch

from tests import test_gpu_experts as T
from tests.gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Fenced:
    """Puts CPU tensors on the GPU with 64 KiB of NaN bit patterns before and
    behind them (any element there that reached a sum would show)."""

    def __init__(self, shift=0):
        self.shift = shift

    def __call__(self, t):
        if t is None:
            return None
        side = 65536 // t.element_size()
        buf = torch.full((t.numel() + 2 * side + 8,), float("nan"), dtype=t.dtype, device=DEV)
        out = buf[side + self.shift:side + self.shift + t.numel()].reshape(t.shape)
        out.copy_(t)
        return out


@pytest.mark.parametrize("i", [8, 64, 72, 128, 200])
@pytest.mark.parametrize("sizes,o", [([2500, 0, 130, 1], 4104), ([64] * 16, 1032), ([1, 0, 3], 264)])
def test_short_reductions(sizes, o, i, monkeypatch):
    """Reductions of one to four steps, where the steps loaded ahead lie past
    the end: nothing from around the operands reaches a result."""
    require_gpu()
    monkeypatch.setattr(T, "Shifted", Fenced)
    T._say(f"short reductions {len(sizes)} groups {i} {o}")
    T._forward_linear(T.Problem(60, sizes, i, o), "none", True, True, True)
    T._forward_gated(T.Problem(61, sizes, i, o // 2), "silu", True)
    T._backward_linear(T.Problem(62, sizes, o, i), "relu")
    T._backward_gated(T.Problem(63, sizes, o, i), "silu")


def test_gelu_far_tail():
    """x Phi(x) and its slope relative to themselves, for every bf16 from -12.5
    to -1/16.  Phi within 1.1e-6 of the formula and z^2, z = |x| / sqrt 2 <= 8.9,
    rounded to fp32 three times before e^(-z^2): 79 * 2^-22 and the
    exponential's own argument, 114 * 2^-24, together below 2^-14; the slope's
    two terms likewise, and one rounding to bf16 each."""
    require_gpu()
    bits = torch.arange(0xBD80, 0xC149, dtype=torch.int32).to(torch.int16)
    x = bits.view(BF).reshape(-1, 1).to(DEV)
    one = torch.ones(1, 1, 1, dtype=BF, device=DEV)
    y, d_x = torch.empty_like(x), torch.empty_like(x)
    T.rrb.expert_linear(x, None, one, y, activation="gelu")
    T.rrb.expert_linear_backward(torch.ones_like(x), x, None, one, pre=x, activation="gelu", d_x=d_x)
    nx = T._np(x)
    assert nx.min() == -12.5 and nx.max() == -0.0625
    want, slope = T.OE.act("gelu", nx), T.OE.act_grad("gelu", nx)
    T._check("act", y, want, 2.0 ** -14 * np.abs(want))
    phi = want / nx
    T._check("slope", d_x, slope, 2.0 ** -14 * (phi + np.abs(slope - phi)))


@pytest.mark.parametrize("name", T.ACTS)
@pytest.mark.parametrize("o", [64, 37])
def test_bias_gradient_of_cancelling_rows(name, o):
    """Column sums that nearly cancel: 100 rows of dZ = dY act'(pre), and three
    more that take their sum back to 2^-20 of it.  dZ in fp32 is off by 2^-19
    (1 + |pre|) |dY|, a sum of N terms by N 2^-24 of their magnitudes' in any
    order; rounding each dZ to bf16 first would be off by 40 times as
    much and more."""
    require_gpu()
    rng = T._rng(64, o)
    rows, G = 100, 2
    off = np.array([0, rows + 3, 2 * (rows + 3)], np.int32)
    N = int(off[-1])
    bf = lambda a: torch.from_numpy(a).to(BF).double().numpy()
    d, pre = bf(rng.standard_normal((N, o))), bf(rng.standard_normal((N, o)))
    slope = lambda: T.OE.act_grad(name, pre)
    for e in range(G):
        r = slice(int(off[e]), int(off[e + 1]))
        pre[r][rows:] = 4.0
        d[r][rows:] = 0.0
        for q in range(3):
            d[r][rows + q] = bf(-(d[r] * slope()[r]).sum(axis=0) / slope()[r][rows + q])
    x, w = torch.ones(N, 8, dtype=BF, device=DEV), torch.ones(G, o, 8, dtype=BF, device=DEV)
    put = lambda a: torch.from_numpy(a).to(BF).to(DEV)
    d_b = torch.full((G, o), -7.25, dtype=BF, device=DEV)
    T.rrb.expert_linear_backward(put(d), x, put_off(off), w, pre=put(pre), activation=name, d_bias=d_b)
    dz = d * slope()
    sums = lambda a: np.stack([a[int(off[e]):int(off[e + 1])].sum(axis=0) for e in range(G)])
    assert (np.abs(sums(dz)) <= 2.0 ** -20 * sums(np.abs(dz))).all()
    bound = 2.0 ** -19 * sums(np.abs(d) * (1 + np.abs(pre))) + (rows + 3) * 2.0 ** -24 * sums(np.abs(dz))
    T._check("d_bias", d_b, sums(dz), bound)


def put_off(off):
    return torch.from_numpy(off).to(DEV)


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
@pytest.mark.parametrize("sizes,o", [([20000, 0, 1, 3000], 64), ([5000], 37), ([300] * 12, 130), ([9000, 40], 8)])
@pytest.mark.parametrize("lead,tail", [(0, 0), (3, 5)])
def test_bias_gradient_of_long_groups(name, sizes, o, lead, tail):
    """Groups whose rows are split over workgroups, alone and with the other
    gradients: the same bits, from call to call too."""
    require_gpu()
    p = T.Problem(65, sizes, 8, o, lead=lead, tail=tail)
    T._backward_linear(p, name)
    d, pre = p.rows(o), p.rows(o)
    got = [p.out(p.G, o) for _ in range(3)]
    d_x, d_w = p.out(p.N, 8), p.out(p.G, o, 8)
    for q, kw in zip(got, ({}, {"d_x": d_x, "d_w": d_w}, {})):
        T.rrb.expert_linear_backward(d, p.x, p.d_off, p.w, pre=pre, activation=name, d_bias=q, **kw)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    nd = T._np(d)
    err = np.zeros_like(nd)
    if name != "none":
        err = np.abs(nd) * T.ACT * (1 + np.abs(T._np(pre)))
        nd = nd * T.OE.act_grad(name, T._np(pre))
    sums = lambda a: np.stack([np.nan_to_num(a[p.off[e]:p.off[e + 1]]).sum(axis=0) for e in range(p.G)])
    T._check("d_bias", got[0], sums(nd), sums(err) + (np.diff(p.off).max() + 64) * 2.0 ** -24 * sums(np.abs(nd)))


def test_gate_of_the_most_tokens():
    """2^26 - 1 tokens, the most that the gate takes, at a wave per token: a
    score of 1 in a row of zeros, at a different expert for each token.  Weights
    and gradients are then two values each, known to E 2^-23 relative (the bound
    of tests/test_gpu_experts.py's gate); bf16 gradients add half a step."""
    require_gpu()
    N, E = (1 << 26) - 1, 264
    T._say(f"gate of {N} tokens, {N * E * 2 >> 30} GiB of scores, twice")
    hot = (torch.arange(N, dtype=torch.int32, device=DEV) * 7 % E).reshape(N, 1)
    logits, d_logits = torch.zeros(N, E, dtype=BF, device=DEV), torch.empty(N, E, dtype=BF, device=DEV)
    step = 1 << 22
    for a in range(0, N, step):
        logits[a:a + step].scatter_(1, hot[a:a + step].long(), 1.0)
    idx, w = torch.full((N, 1), -1, dtype=torch.int32, device=DEV), torch.full((N, 1), -1.0, device=DEV)
    T.rrb.moe_gate(logits, idx, w)
    assert torch.equal(idx, hot)
    p = np.e / (np.e + E - 1)
    rel = (E + 10) * 2.0 ** -23
    assert abs(w.min().item() - p) <= rel * p and abs(w.max().item() - p) <= rel * p
    T.rrb.moe_gate_backward(logits, idx, torch.ones_like(w), d_logits)
    other = p / np.e * -p
    for a in range(0, N, step):
        d, h = d_logits[a:a + step], hot[a:a + step].long()
        for got, want in ((d.gather(1, h), p * (1 - p)), (d.scatter_(1, h, d[0, (h[0, 0] + 1) % E].item()), other)):
            for v in (got.min().item(), got.max().item()):
                assert abs(v - want) <= (T.HALF + 6 * rel) * abs(want), (a, v, want)
    del logits, d_logits, d
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate_gradients_in_the_scores_place(dtype, renorm):
    require_gpu()
    for N, E, k in T.GATES:
        logits = T._scores(N, E, "masked", dtype).to(DEV)
        idx, w = torch.empty(N, k, dtype=torch.int32, device=DEV), torch.empty(N, k, device=DEV)
        T.rrb.moe_gate(logits, idx, w, renormalize=renorm)
        d_w = torch.from_numpy(T._rng(66, N, E).standard_normal((N, k)).astype(np.float32)).to(DEV)
        want = torch.empty_like(logits)
        T.rrb.moe_gate_backward(logits, idx, d_w, want, renormalize=renorm)
        T.rrb.moe_gate_backward(logits, idx, d_w, logits, renormalize=renorm)
        assert torch.equal(logits, want), (N, E, k)


def test_gate_refuses_overlaps():
    require_gpu()
    buf = torch.zeros(4096, device=DEV)
    logits = buf[:1024].reshape(16, 64)
    idx, w = torch.zeros(16, 4, dtype=torch.int32, device=DEV), torch.zeros(16, 4, device=DEV)
    for call in (lambda: T.rrb.moe_gate(logits, idx, buf[1000:1064].reshape(16, 4)),
                 lambda: T.rrb.moe_gate(logits, idx, idx.view(torch.float32)),
                 lambda: T.rrb.moe_gate_backward(logits, idx, w, buf[64:1088].reshape(16, 64))):
        with pytest.raises(T.rrb.RrbError) as e:
            call()
        assert "overlaps" in str(e.value)


def test_plans_refuse_overlaps():
    """Offsets in a plan's workspace, and the combine's gradient over its
    inputs, its weights or the workspace; neither call then writes."""
    require_gpu()
    N, h, E, k = 32, 64, 8, 2
    rng = T._rng(67)
    idx, w = torch.from_numpy(T._choices(rng, N, E, k)).to(DEV), torch.rand(N, k, device=DEV)
    comb = T.rrb.MoeDevicePlan(1, N, h, E, k, "combine")
    comb.route(idx, w)
    dy, z = T._bf16(rng, (N, h)).to(DEV), T._bf16(rng, (N * k, h)).to(DEV)
    dz, dw = torch.zeros_like(z), torch.zeros(N, k, device=DEV)
    ws = comb._ws.view(torch.int32)
    keep = comb._ws.clone()
    at = ws.numel() // 2
    calls = [lambda: comb.expert_offsets(ws[at:at + E + 1]),
             lambda: comb.backward([dy], [z], [z], d_weights=dw),
             lambda: comb.backward([z], None, [z]),
             lambda: comb.backward([dy], [z], [dz], d_weights=w, weights=w),
             lambda: comb.backward([dy], [z], [dz], d_weights=ws[at:at + N * k].view(torch.float32))]
    for call in calls:
        with pytest.raises(T.rrb.RrbError) as e:
            call()
        assert "overlaps" in str(e.value)
    assert torch.equal(comb._ws, keep)
    comb.backward([dy], [z], [dz], d_weights=dw)
    want_z, want_w = T.OE.combine_grad(T._np(dy), T._np(z), T._slots(idx.cpu().numpy(), E), T._np(w))
    T._check("dz", dz, want_z, T.ADD * np.abs(want_z), T.HALF * 1.01)


@pytest.mark.parametrize("h,shift", [(8, 0), (8, 1), (5, 0)])
def test_combine_backward_of_more_tokens_than_a_launch(h, shift):
    """More than 2^23 tokens, which a launch takes: both kernels' later slices
    (whole 16-byte rows, and rows off those boundaries), every row and weight.
    dz is one fp32 product rounded to bf16, so equal; dw sums h products."""
    require_gpu()
    N, E = (1 << 23) + 77, 4
    T._say(f"combine gradient of {N} tokens, width {h}, shift {shift}")
    gen = torch.Generator(device=DEV).manual_seed(68)
    idx = torch.randint(0, E, (N, 1), generator=gen, dtype=torch.int32, device=DEV)
    w = torch.rand(N, 1, generator=gen, device=DEV)
    put = T.Shifted(shift)
    dy, z = (put(torch.randn(N, h, generator=gen, device=DEV).to(BF)) for _ in range(2))
    plan = T.rrb.MoeDevicePlan(1, N, h, E, 1, "combine")
    plan.route(idx, w)
    dz, dw = put(torch.full((N, h), -7.25, dtype=BF)), torch.full((N, 1), -7.0, device=DEV)
    plan.backward([dy], [z], [dz], d_weights=dw)
    order = torch.sort(idx[:, 0], stable=True).indices  # token of each arena row
    assert torch.equal(dz, (w * dy.float()).to(BF)[order])
    terms = dy.float()[order].double() * z.double()
    got = dw[order, 0].double()
    assert ((got - terms.sum(dim=1)).abs() <= (h + 2) * T.ADD * terms.abs().sum(dim=1)).all()


@pytest.mark.parametrize("N,h,f,E,k,R", [(64, 64, 96, 8, 2, 2), (256, 136, 72, 16, 4, 4), (1, 48, 40, 16, 4, 1)])
def test_moe_step_replayed_by_itself(N, h, f, E, k, R):
    """The whole step captured, and replayed three times on new inputs with
    every output, intermediate and the plan's routing made useless before: the
    replay alone has to bring all of it back, equal to an eager step's."""
    require_gpu()
    rng = T._rng(69, N, h, f)
    x, dy = T._bf16(rng, (N, h)).to(DEV), T._bf16(rng, (N, h)).to(DEV)
    logits = torch.zeros(N, E, device=DEV)
    wg, wu = (T._bf16(rng, (E, f, h), h ** -0.5).to(DEV) for _ in range(2))
    wd = T._bf16(rng, (E, h, f), f ** -0.5).to(DEV)
    n = N * k
    new = lambda *s, dtype=BF: torch.zeros(s, dtype=dtype, device=DEV)
    disp = T.rrb.MoeDevicePlan(R, N, h, E, k, "dispatch")
    comb = T.rrb.MoeDevicePlan(R, N, h, E, k, "combine", share=disp)
    shards = lambda t: list(t.reshape(R, N // R, h).unbind(0))
    arena = lambda t: [t] + [None] * (R - 1)
    idx, off = new(N, k, dtype=torch.int32), new(E + 1, dtype=torch.int32)
    w, d_w, d_logits = (new(N, c, dtype=torch.float32) for c in (k, k, E))
    xe, z, d_z, d_xe = (new(n, h) for _ in range(4))
    g, u, hh, d_h = (new(n, f) for _ in range(4))
    y, d_x, d_wg, d_wu, d_wd = new(N, h), new(N, h), new(E, f, h), new(E, f, h), new(E, h, f)
    ones = torch.ones(N, k, device=DEV)

    def step():
        T.rrb.moe_gate(logits, idx, w, renormalize=True)
        disp.route(idx, w)
        disp.expert_offsets(off)
        disp.run(shards(x), arena(xe))
        T.rrb.expert_gated(xe, off, wg, wu, hh, save_gate=g, save_up=u)
        T.rrb.expert_linear(hh, off, wd, z)
        comb.run(arena(z), shards(y))
        comb.backward(shards(dy), arena(z), arena(d_z), d_weights=d_w)
        T.rrb.expert_linear_backward(d_z, hh, off, wd, d_x=d_h, d_w=d_wd)
        T.rrb.expert_gated_backward(d_h, xe, off, wg, wu, g, u, d_x=d_xe, d_w_gate=d_wg, d_w_up=d_wu)
        comb.run(arena(d_xe), shards(d_x), weights=ones)
        T.rrb.moe_gate_backward(logits, idx, d_w, d_logits, renormalize=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    made = (idx, off, w, d_w, d_logits, xe, z, d_z, d_xe, g, u, hh, d_h, y, d_x, d_wg, d_wu, d_wd)
    other = torch.arange(k, dtype=torch.int32, device=DEV).expand(N, k).contiguous()
    for q in range(3):
        x.copy_(T._bf16(T._rng(70, q), (N, h)))
        logits.copy_(torch.from_numpy(T._rng(71, q).standard_normal((N, E)).astype(np.float32)))
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in made]
        disp.route(other, torch.full((N, k), float("nan"), device=DEV))
        for t in made:
            t.fill_(float("nan") if t.is_floating_point() else 0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(eager, made)):
            assert torch.equal(a, b), (q, i)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
def test_gate_gradient_of_experts_far_below_the_largest(dtype):
    """Renormalised over chosen experts whose scores lie far below the row's
    largest, which is not among them (its entry is passed over): the softmax
    over the chosen alone, against the oracle with the others masked."""
    require_gpu()
    for E in (5, 300):
        l = np.full((3, E), -1.0)
        l[:, 0] = 200.0, 1000.0, 90.0
        l[:, 1:4] = [1.0, 0.0, -2.0]
        idx = np.array([[-1, 1, 2], [3, 99999, 1], [2, 3, 1]], np.int32)
        d_w = T._rng(72, E).standard_normal((3, 3)).astype(np.float32)
        logits = torch.from_numpy(l).to(dtype).to(DEV)
        out = torch.full((3, E), -7.0, dtype=dtype, device=DEV)
        T.rrb.moe_gate_backward(logits, torch.from_numpy(idx).to(DEV), torch.from_numpy(d_w).to(DEV), out,
                                renormalize=True)
        for t in range(3):
            used = (idx[t] >= 0) & (idx[t] < E)
            masked = np.full((1, E), -np.inf)
            masked[0, idx[t][used]] = l[t, idx[t][used]]
            want = T.OE.gate_grad(masked, idx[t:t + 1, used], d_w[t:t + 1, used].astype(np.float64), True)
            # weights below 1 known to (k + |l - m| + 8) 2^-23 <= 2^-19, times two terms of |dw|
            T._check("d_logits", out[t:t + 1], want, np.full_like(want, 2.0 ** -17 * np.abs(d_w[t]).max()))


@pytest.mark.parametrize("name", ["none", "gelu"])
def test_bias_gradient_of_one_group_among_many(name):
    """All rows in one of 64 groups; the others' gradients are 0."""
    require_gpu()
    T._backward_linear(T.Problem(73, [0] * 40 + [9000] + [0] * 23, 16, 72), name)
