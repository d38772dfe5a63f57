"""GPU parity of the MoE gate, the experts' products and their gradients
against the binary64 oracle.

Tolerances.  Inputs are bf16 (or fp32) values, taken exactly by both sides.
A product sums K exact fp32 products in fp32 in some order: off by at most
K 2^-23 sum |a b| (one half step, 2^-24, per product and per addition, and the
few partial sums' joins).  One rounding to bf16 is off by at most 2^-8 of the
value.  An activation f and its slope are computed in fp32 from an argument
known to 2^-23 relative, so off by at most 2^-19 (1 + |x|) absolute and a
slope of at most 1.13; those errors and a factor's own are carried through by
the product rule.  Gradients round the projections' gradients to bf16 first:
2^-8 of each term, so at most 2^-8 sum |terms| in the result, and for
independent roundings about 2^-8 / sqrt 3 of its norm, twice 2^-8 with the
final rounding being far above it for the tens of elements compared.
"""

import ctypes
import sys

import numpy as np
import pytest
import torch

import reduce_rank_buffers_amd as rrb
from oracle import experts as OE
from tests.gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HALF = 2.0 ** -8     # half a step of bf16
ADD = 2.0 ** -23     # a product and an addition in fp32
ACT = 2.0 ** -19
TINY = 1e-37         # below it fp32 has lost precision


def _say(*a):
    print(*a, file=sys.stderr, flush=True)


def _rng(*key):
    return np.random.default_rng([77, *key])


def _bf16(rng, shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(BF)


def _np(t):
    return t.detach().cpu().double().numpy()


class Shifted:
    """Puts CPU tensors on the GPU; with shift, `shift` elements into a larger
    buffer, so that rows lose their alignment."""

    def __init__(self, shift=0):
        self.shift = shift

    def __call__(self, t):
        if t is None:
            return None
        buf = torch.empty(t.numel() + self.shift + 8, dtype=t.dtype, device=DEV)
        out = buf[self.shift:self.shift + t.numel()].reshape(t.shape)
        out.copy_(t)
        return out


def _check(what, got, want, bound, rms=None):
    """Every element within its bound, and the norm of the errors within rms
    of the result's norm."""
    got = _np(got)
    ok = ~np.isnan(want)
    err = np.abs(got - want)[ok]
    over = err - (bound + HALF * np.abs(want) + TINY)[ok]
    assert np.isfinite(got[ok]).all(), f"{what}: not finite"
    assert over.size == 0 or over.max() <= 0, f"{what}: off by {err[over.argmax()]} at {want[ok][over.argmax()]}"
    if rms is not None and err.size >= 64:
        assert np.sqrt((err ** 2).sum()) <= rms * np.sqrt((want[ok] ** 2).sum()) + TINY, f"{what}: norm of errors"


def _offsets(sizes, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(sizes)]).astype(np.int32)


class Problem:
    """Rows grouped by `sizes`, `lead` unused rows before and `tail` behind."""

    def __init__(self, seed, sizes, i, o, lead=0, tail=0, shift=0):
        rng = _rng(seed, i, o, *sizes)
        self.off = _offsets(sizes, lead)
        self.N, self.G, self.i, self.o = int(self.off[-1]) + tail, len(sizes), i, o
        self.put = Shifted(shift)
        self.rng = rng
        x = _bf16(rng, (self.N, i))
        used = np.zeros(self.N, bool)
        for e, r in OE.groups(self.off):
            used[r] = True
        self.used = used
        x[~torch.from_numpy(used)] = float("nan")  # rows of no group: never read
        self.x, self.d_off = self.put(x), torch.from_numpy(self.off).to(DEV)
        self.w, self.w2 = self.weight(), self.weight()

    def weight(self):
        w = _bf16(self.rng, (self.G, self.o, self.i), self.i ** -0.5)
        for e in range(self.G):
            if self.off[e + 1] <= self.off[e]:
                w[e] = float("nan")  # weights without rows: never read
        return self.put(w)

    def rows(self, width, scale=1.0):
        t = _bf16(self.rng, (self.N, width), scale)
        t[~torch.from_numpy(self.used)] = float("nan")
        return self.put(t)

    def out(self, *shape):
        return self.put(torch.full(shape, -7.25, dtype=BF))

    def untouched(self, what, t):
        assert (_np(t)[~self.used] == -7.25).all(), f"{what}: rows of no group were written"


def _abs_linear(p, a, w):
    """sum |a| |w| per output, the scale of a product's error."""
    return np.nan_to_num(OE.linear(np.abs(a), p.off, np.abs(w))[0])


SHAPES = [
    # sizes, in, out
    ([1], 8, 8), ([1], 1, 1), ([2], 7, 5), ([3, 0, 1], 64, 64), ([0, 0, 0], 64, 72), ([17], 64, 16),
    ([5, 128, 0, 129, 1], 72, 136), ([130, 7], 200, 264), ([33, 20], 13, 39), ([64, 64], 128, 128),
    ([16, 0, 15, 1, 31], 256, 48), ([300], 333, 250), ([100, 0, 28], 1032, 24), ([4] * 70, 40, 24),
    ([1] * 200, 24, 16), ([260, 3, 511], 320, 520), ([1000], 96, 600),
]
ACTS = list(OE.ACTIVATIONS)


def _ids(s):
    return f"{len(s[0])}x{max(s[0])}-{s[1]}-{s[2]}"


def _forward_linear(p, name, bias, residual, save):
    b = p.put(_bf16(p.rng, (p.G, p.o))) if bias else None
    r = p.rows(p.o) if residual else None
    y, pre = p.out(p.N, p.o), p.out(p.N, p.o) if save else None
    rrb.expert_linear(p.x, p.d_off, p.w, y, bias=b, activation=name, residual=r, save_pre=pre)
    torch.cuda.synchronize()
    x, w = _np(p.x), _np(p.w)
    nb, nr = _np(b) if bias else None, _np(r) if residual else None
    want, wpre = OE.linear(x, p.off, w, nb, name, nr)
    e = (p.i + 1) * ADD * (_abs_linear(p, x, w) + (np.abs(wpre) if bias else 0))
    if save:
        _check("pre", pre, wpre, e, HALF)
        p.untouched("pre", pre)
    e = 1.13 * e + (0 if name == "none" else ACT * (1 + np.abs(wpre)))
    if residual:
        e = e + ADD * (np.abs(want) + np.abs(nr))
    _check("out", y, want, e, 1.5 * HALF)
    p.untouched("out", y)


@pytest.mark.parametrize("shape", SHAPES, ids=_ids)
@pytest.mark.parametrize("lead,tail,shift", [(0, 0, 0), (3, 5, 0), (0, 2, 1)])
def test_linear(shape, lead, tail, shift):
    require_gpu()
    k = SHAPES.index(shape) + lead + shift
    p = Problem(1, *shape, lead=lead, tail=tail, shift=shift)
    _forward_linear(p, ACTS[k % 5], k % 2 == 0, k % 3 == 0, k % 4 < 2)


@pytest.mark.parametrize("name", ACTS)
def test_linear_epilogues(name):
    require_gpu()
    for bias in (False, True):
        for residual in (False, True):
            _forward_linear(Problem(2, [40, 0, 90], 64, 136), name, bias, residual, True)


def test_linear_in_place_residual():
    require_gpu()
    p = Problem(3, [150, 20], 72, 200)
    y = p.rows(p.o)
    keep = _np(y)
    rrb.expert_linear(p.x, p.d_off, p.w, y, residual=y)
    want = OE.linear(_np(p.x), p.off, _np(p.w), None, "none", keep)[0]
    _check("out", y, want, (p.i + 2) * ADD * (_abs_linear(p, _np(p.x), _np(p.w)) + np.abs(keep)))


@pytest.mark.parametrize("shape", SHAPES, ids=_ids)
@pytest.mark.parametrize("lead,tail,shift", [(0, 0, 0), (3, 5, 0), (0, 2, 1)])
def test_gated(shape, lead, tail, shift):
    require_gpu()
    k = SHAPES.index(shape) + lead + shift
    _forward_gated(Problem(4, *shape, lead=lead, tail=tail, shift=shift), ACTS[k % 5], k % 2)


def _forward_gated(p, name, save):
    h = p.out(p.N, p.o)
    g, u = (p.out(p.N, p.o), p.out(p.N, p.o)) if save else (None, None)
    rrb.expert_gated(p.x, p.d_off, p.w, p.w2, h, activation=name, save_gate=g, save_up=u)
    torch.cuda.synchronize()
    x, wg, wu = _np(p.x), _np(p.w), _np(p.w2)
    want, ng, nu = OE.gated(x, p.off, wg, wu, name)
    eg, eu = p.i * ADD * _abs_linear(p, x, wg), p.i * ADD * _abs_linear(p, x, wu)
    if g is not None:
        _check("gate", g, ng, eg, HALF)
        _check("up", u, nu, eu, HALF)
        p.untouched("gate", g)
        p.untouched("up", u)
    e = np.abs(nu) * (1.13 * eg + ACT * (1 + np.abs(ng))) + np.abs(OE.act(name, ng)) * eu + ADD * np.abs(want)
    _check("out", h, want, e, 1.5 * HALF)
    p.untouched("out", h)


def _grad_bounds(p, d, d_err, x, w):
    """Bounds of dX and dW for dZ = d known to d_err, rounded to bf16."""
    e = np.nan_to_num(d_err) + HALF * np.nan_to_num(np.abs(d))
    ax, aw, ad = np.nan_to_num(np.abs(x)), np.nan_to_num(np.abs(w)), np.nan_to_num(np.abs(d))
    bx, bw, _ = OE.linear_grad(e, ax, p.off, aw)
    sx, sw, _ = OE.linear_grad(ad, ax, p.off, aw)
    rows = np.diff(p.off).max() + 1
    return np.nan_to_num(bx) + p.o * ADD * np.nan_to_num(sx), bw + rows * ADD * sw


@pytest.mark.parametrize("shape", SHAPES, ids=_ids)
@pytest.mark.parametrize("lead,tail,shift", [(0, 0, 0), (3, 5, 0), (0, 2, 1)])
def test_linear_backward(shape, lead, tail, shift):
    require_gpu()
    k = SHAPES.index(shape) + lead + shift
    _backward_linear(Problem(5, *shape, lead=lead, tail=tail, shift=shift), ACTS[k % 5])


def _backward_linear(p, name):
    d, pre = p.rows(p.o), p.rows(p.o) if name != "none" else None
    d_x, d_w, d_b = p.out(p.N, p.i), p.out(p.G, p.o, p.i), p.out(p.G, p.o)
    rrb.expert_linear_backward(d, p.x, p.d_off, p.w, pre=pre, activation=name, d_x=d_x, d_w=d_w, d_bias=d_b)
    torch.cuda.synchronize()
    nd, x, w = _np(d), _np(p.x), _np(p.w)
    npre = _np(pre) if pre is not None else None
    wx, ww, wb = OE.linear_grad(nd, x, p.off, w, npre, name)
    dz = nd * (OE.act_grad(name, npre) if pre is not None else 1.0)
    err = np.abs(nd) * ACT * (1 + np.abs(npre)) if pre is not None else np.zeros_like(nd)
    bx, bw = _grad_bounds(p, dz, err, x, w)
    _check("d_x", d_x, wx, bx, 2 * HALF)
    _check("d_w", d_w, ww, bw, 2 * HALF)
    ez, az = np.nan_to_num(err) + HALF * np.nan_to_num(np.abs(dz)), np.nan_to_num(np.abs(dz))
    bb = OE.linear_grad(ez, np.zeros_like(x), p.off, np.zeros_like(w))[2]
    sb = OE.linear_grad(az, np.zeros_like(x), p.off, np.zeros_like(w))[2]
    _check("d_bias", d_b, wb, bb + (np.diff(p.off).max() + 1) * ADD * sb, 2 * HALF)
    p.untouched("d_x", d_x)


@pytest.mark.parametrize("shape", SHAPES, ids=_ids)
@pytest.mark.parametrize("lead,tail,shift", [(0, 0, 0), (3, 5, 0), (0, 2, 1)])
def test_gated_backward(shape, lead, tail, shift):
    require_gpu()
    k = SHAPES.index(shape) + lead + shift
    _backward_gated(Problem(6, *shape, lead=lead, tail=tail, shift=shift), ACTS[(k + 1) % 5])


def _backward_gated(p, name):
    d, g, u = p.rows(p.o), p.rows(p.o), p.rows(p.o)
    d_x, d_wg, d_wu = p.out(p.N, p.i), p.out(p.G, p.o, p.i), p.out(p.G, p.o, p.i)
    rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, g, u, activation=name, d_x=d_x, d_w_gate=d_wg, d_w_up=d_wu)
    torch.cuda.synchronize()
    nd, ng, nu, x, wg, wu = (_np(t) for t in (d, g, u, p.x, p.w, p.w2))
    wx, wwg, wwu = OE.gated_grad(nd, x, p.off, wg, wu, ng, nu, name)
    dg, du = nd * nu * OE.act_grad(name, ng), nd * OE.act(name, ng)
    bxg, bwg = _grad_bounds(p, dg, np.abs(nd * nu) * ACT * (1 + np.abs(ng)) + ADD * np.abs(dg), x, wg)
    bxu, bwu = _grad_bounds(p, du, np.abs(nd) * ACT * (1 + np.abs(ng)) + ADD * np.abs(du), x, wu)
    # both halves accumulate in one sum: twice the additions
    sx = np.nan_to_num(OE.linear_grad(np.nan_to_num(np.abs(dg)), np.abs(x), p.off, np.nan_to_num(np.abs(wg)))[0])
    sx = sx + np.nan_to_num(OE.linear_grad(np.nan_to_num(np.abs(du)), np.abs(x), p.off, np.nan_to_num(np.abs(wu)))[0])
    _check("d_x", d_x, wx, bxg + bxu + 2 * p.o * ADD * sx, 2 * HALF)
    _check("d_w_gate", d_wg, wwg, bwg, 2 * HALF)
    _check("d_w_up", d_wu, wwu, bwu, 2 * HALF)
    p.untouched("d_x", d_x)


# Enough tiles for the larger tile shapes: whole tiles, tiles of at most 128
# rows, one row, empty groups; a reduction that ends inside a step and outputs
# that end inside a tile.
RAGGED = [2500, 0, 100, 1300, 129, 1, 2900, 256, 128, 700]


@pytest.mark.parametrize("i,o", [(200, 4104), (64, 4104), (136, 8200), (2056, 1032), (1029, 2050)])
@pytest.mark.parametrize("lead,tail", [(0, 0), (7, 9)])
def test_large_forward(i, o, lead, tail):
    require_gpu()
    _say(f"large forward {i} -> {o}")
    _forward_linear(Problem(50, RAGGED, i, o, lead, tail), ACTS[i % 5], True, True, lead == 0)
    _forward_gated(Problem(51, RAGGED, i, o // 2, lead, tail), ACTS[(i + 2) % 5], lead == 0)


@pytest.mark.parametrize("i,o", [(4104, 200), (4104, 201), (8200, 64), (2056, 1027), (4099, 1031)])
@pytest.mark.parametrize("lead,tail", [(0, 0), (7, 9)])
def test_large_backward(i, o, lead, tail):
    require_gpu()
    _say(f"large backward {i} <- {o}")
    _backward_linear(Problem(52, RAGGED, i, o, lead, tail), ACTS[o % 5])
    _backward_gated(Problem(53, RAGGED, i, o, lead, tail), ACTS[(o + 2) % 5])


@pytest.mark.parametrize("sizes,i,o", [([1, 0, 3, 1, 2, 60, 1, 9], 2048, 4096), ([64] * 32, 1024, 1024),
                                       ([40, 100] * 16, 512, 2048), ([1] * 300, 256, 512)])
def test_few_rows(sizes, i, o):
    """Shapes where the smaller tiles are taken: decode and short batches."""
    require_gpu()
    _forward_linear(Problem(54, sizes, i, o), "silu", True, False, True)
    _forward_gated(Problem(55, sizes, i, o), "gelu", False)
    _backward_gated(Problem(56, sizes, i, o // 4), "silu")


def test_arena_past_4_gib():
    """Rows and weights whose byte offsets pass 2^32: the last rows' outputs
    and the last group's gradient against the oracle on those alone."""
    require_gpu()
    N, i, o = 280000, 8192, 64
    _say(f"arena of {N * i * 2 >> 20} MiB")
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = torch.empty(N, i, dtype=BF, device=DEV)
    for a in range(0, N, 40000):
        x[a:a + 40000] = torch.randn(min(40000, N - a), i, generator=gen, device=DEV).to(BF)
    off = torch.tensor([0, N - 100, N], dtype=torch.int32, device=DEV)
    w = (torch.randn(2, o, i, generator=gen, device=DEV) * i ** -0.5).to(BF)
    y, d_w = torch.empty(N, o, dtype=BF, device=DEV), torch.empty_like(w)
    rrb.expert_linear(x, off, w, y)
    at = slice(N - 300, N)
    nx, nw = _np(x[at]), _np(w)
    want = np.concatenate([nx[:200] @ nw[0].T, nx[200:] @ nw[1].T])
    scale = np.concatenate([np.abs(nx[:200]) @ np.abs(nw[0]).T, np.abs(nx[200:]) @ np.abs(nw[1]).T])
    _check("out", y[at], want, i * ADD * scale, HALF * 1.01)
    rrb.expert_linear_backward(y, x, off, w, d_w=d_w)
    ny = _np(y[N - 100:])
    _check("d_w", d_w[1], ny.T @ nx[200:], 101 * ADD * (np.abs(ny).T @ np.abs(nx[200:])), HALF * 1.01)
    d_x = x  # in place of the inputs, which nothing reads any more
    rrb.expert_linear_backward(y, torch.empty_like(x), off, w, d_x=d_x)
    ny = _np(y[at])
    want = np.concatenate([ny[:200] @ nw[0], ny[200:] @ nw[1]])
    scale = np.concatenate([np.abs(ny[:200]) @ np.abs(nw[0]), np.abs(ny[200:]) @ np.abs(nw[1])])
    _check("d_x", d_x[at], want, (o + 1) * ADD * scale, HALF * 1.01)
    del x, d_x, y
    G, i, o = 40, 8192, 8192
    w = torch.empty(G, o, i, dtype=BF, device=DEV)
    for e in range(G):
        w[e] = (torch.randn(o, i, generator=gen, device=DEV) * i ** -0.5).to(BF)
    x = torch.randn(2 * G, i, generator=gen, device=DEV).to(BF)
    off = torch.arange(0, 2 * G + 1, 2, dtype=torch.int32, device=DEV)
    y = torch.empty(2 * G, o, dtype=BF, device=DEV)
    rrb.expert_linear(x, off, w, y)
    nx, nw = _np(x[-2:]), _np(w[-1])
    _check("out", y[-2:], nx @ nw.T, i * ADD * (np.abs(nx) @ np.abs(nw).T), HALF * 1.01)


def test_gradients_against_differences():
    """The kernels' gradients along random directions against differences of
    the forward definition: <grad, v> = (L(p + hv) - L(p - hv)) / 2h, L = the
    sum of out * d.  The gradient's error is at most 2 * 2^-8 of its norm (as
    above), so off by at most that times |v| |grad|; the difference's own
    error at h = 1e-4 is far below it."""
    require_gpu()
    p = Problem(7, [30, 0, 45], 40, 24)
    x, wg, wu = _np(p.x), np.nan_to_num(_np(p.w)), np.nan_to_num(_np(p.w2))
    for name in ACTS:
        _, ng, nu = OE.gated(x, p.off, wg, wu, name)
        g, u = (torch.from_numpy(v).to(BF).to(DEV) for v in (ng, nu))
        d = p.rows(p.o)
        nd = _np(d)
        outs = p.out(p.N, p.i), p.out(p.G, p.o, p.i), p.out(p.G, p.o, p.i)
        rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, g, u, activation=name, d_x=outs[0], d_w_gate=outs[1],
                                  d_w_up=outs[2])
        for at in range(3):
            grad = _np(outs[at])
            for trial in range(4):
                v = _rng(8, at, trial).standard_normal(grad.shape)
                arg = [x, wg, wu]

                def loss(h):
                    a = list(arg)
                    a[at] = a[at] + h * v
                    if name == "relu":  # the kink: keep the slope of the point
                        gg, uu = OE.linear(a[0], p.off, a[1])[0], OE.linear(a[0], p.off, a[2])[0]
                        return (np.where(ng > 0, gg, 0.0) * uu * nd).sum()
                    return (OE.gated(a[0], p.off, a[1], a[2], name)[0] * nd).sum()

                slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
                # saved projections are rounded: 2^-8 of each, in g and in u
                limit = 4 * HALF * np.sqrt((grad ** 2).sum()) * np.sqrt((v ** 2).sum())
                assert abs((grad * v).sum() - slope) <= limit, (name, at, trial)


def test_values_do_not_leak():
    """NaN and infinity in one group's rows, weights or gradients stay in that
    group; a NaN row stays a row."""
    require_gpu()
    for sizes, i, o in (([70, 60, 130], 64, 72), ([9, 3, 8], 40, 33)):
        p = Problem(9, sizes, i, o)
        d, g, u = p.rows(o), p.rows(o), p.rows(o)
        clean = [p.out(p.N, o), p.out(p.N, i), p.out(p.G, o, i), p.out(p.G, o, i)]
        dirty = [torch.empty_like(t) for t in clean]

        def run(o_):
            rrb.expert_gated(p.x, p.d_off, p.w, p.w2, o_[0])
            rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, g, u, d_x=o_[1], d_w_gate=o_[2], d_w_up=o_[3])

        run(clean)
        mid = slice(sizes[0], sizes[0] + sizes[1])
        p.x[mid] = float("inf")
        d[mid] = float("nan")
        p.w[1] = float("nan")
        run(dirty)
        keep = np.ones(p.N, bool)
        keep[mid] = False
        for a, b in zip(clean[:2], dirty[:2]):
            assert torch.equal(a[torch.from_numpy(keep)], b[torch.from_numpy(keep)])
        for a, b in zip(clean[2:], dirty[2:]):
            assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
            assert not torch.isfinite(b[1].float()).any()
        q = Problem(10, sizes, i, o)
        a, b = q.out(q.N, o), q.out(q.N, o)
        rrb.expert_linear(q.x, q.d_off, q.w, a)
        q.x[5, 3] = float("nan")
        rrb.expert_linear(q.x, q.d_off, q.w, b)
        assert torch.isnan(b[5].float()).all()
        a[5] = b[5] = 0
        assert torch.equal(a, b)


@pytest.mark.parametrize("name", ACTS)
def test_extreme_arguments(name):
    """Activations and slopes at large, tiny and zero arguments (a 1 x 1
    product passes the argument through exactly), against the oracle."""
    require_gpu()
    v = np.array([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 3, -3, 9, -9, 20, -20, 88, -88, 120, -120, 1e4, -1e4,
                  1e20, -1e20, 3e38, -3e38], np.float32)
    x = torch.from_numpy(v).to(BF).reshape(-1, 1).to(DEV)
    one = torch.ones(1, 1, 1, dtype=BF, device=DEV)
    y, d_x = torch.empty_like(x), torch.empty_like(x)
    rrb.expert_linear(x, None, one, y, activation=name)
    rrb.expert_linear_backward(torch.ones_like(x), x, None, one, pre=x, activation=name, d_x=d_x)
    nx = _np(x)
    with np.errstate(over="ignore", invalid="ignore"):
        want, slope = OE.act(name, nx), OE.act_grad(name, nx)
    # far out the exact values: x or 0, slope 1 or 0
    big = np.abs(nx) > 1e3
    neg = 0.0 if name != "none" else 1.0
    want = np.where(big, np.where(nx > 0, nx, neg * nx), want)
    slope = np.where(big, np.where(nx > 0, 1.0, neg), slope)
    _check("act", y, want, ACT * np.abs(want) + (0 if name in ("none", "relu") else ACT * np.minimum(np.abs(nx), 1)))
    _check("slope", d_x, slope, np.full_like(slope, ACT * 4) + HALF * np.abs(slope))


def test_offsets_are_clamped():
    """Offsets outside the arena or decreasing: nothing outside the outputs is
    written (guards around them keep their values)."""
    require_gpu()
    p = Problem(11, [40, 40, 48], 64, 40)
    for bad in ([0, 500, 2 ** 31 - 1, 128], [-5, 30, 60, 128], [100, 20, 90, 64], [2 ** 31 - 1] * 4, [-9] * 4):
        off = torch.tensor(bad, dtype=torch.int32, device=DEV)
        bufs = []

        def guarded(*shape):
            n = int(np.prod(shape))
            b = torch.full((n + 4096,), 3.5, dtype=BF, device=DEV)
            bufs.append((b, n))
            return b[2048:2048 + n].reshape(shape)

        h, dx, dw, du = (guarded(*s) for s in ((p.N, p.o), (p.N, p.i), (p.G, p.o, p.i), (p.G, p.o, p.i)))
        rrb.expert_gated(p.x, off, p.w, p.w2, h)
        rrb.expert_gated_backward(h, p.x, off, p.w, p.w2, h, h, d_x=dx, d_w_gate=dw, d_w_up=du)
        torch.cuda.synchronize()
        for b, n in bufs:
            assert (b[:2048] == 3.5).all() and (b[2048 + n:] == 3.5).all()


def test_no_rows():
    require_gpu()
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    x, y = torch.empty(0, 16, dtype=BF, device=DEV), torch.empty(0, 24, dtype=BF, device=DEV)
    w = torch.full((2, 24, 16), float("nan"), dtype=BF, device=DEV)
    rrb.expert_gated(x, off, w, w, y)
    rrb.expert_linear(x, off, w, y)
    g, u, b = torch.ones_like(w), torch.ones_like(w), torch.ones(2, 24, dtype=BF, device=DEV)
    rrb.expert_gated_backward(y, x, off, w, w, y, y, d_x=x, d_w_gate=g, d_w_up=u)
    assert not g.any() and not u.any()
    g.fill_(1)
    rrb.expert_linear_backward(y, x, off, w, d_x=x, d_w=g, d_bias=b)
    assert not g.any() and not b.any()
    rrb.expert_linear_backward(y, x, off, w, d_x=x)
    rrb.expert_gated_backward(y, x, off, w, w, y, y, d_x=x)


def test_partial_gradients():
    """Any subset of the gradients, and the caller's workspace: the same bits."""
    require_gpu()
    p = Problem(12, [50, 80], 64, 48)
    d, g, u = p.rows(p.o), p.rows(p.o), p.rows(p.o)
    full = p.out(p.N, p.i), p.out(p.G, p.o, p.i), p.out(p.G, p.o, p.i)
    rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, g, u, d_x=full[0], d_w_gate=full[1], d_w_up=full[2])
    ws = torch.full((rrb.expert_gated_backward_workspace(p.N, p.i, p.o, p.G),), 255, dtype=torch.uint8, device=DEV)
    a, b, c = p.out(p.N, p.i), p.out(p.G, p.o, p.i), p.out(p.G, p.o, p.i)
    rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, g, u, d_x=a, workspace=ws)
    rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, g, u, d_w_gate=b, d_w_up=c, workspace=ws)
    assert torch.equal(a, full[0]) and torch.equal(b, full[1]) and torch.equal(c, full[2])
    with pytest.raises(ValueError):
        rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, g, u, d_x=a, workspace=ws[:-1])
    full = p.out(p.N, p.i), p.out(p.G, p.o, p.i), p.out(p.G, p.o)
    rrb.expert_linear_backward(d, p.x, p.d_off, p.w, pre=g, activation="silu", d_x=full[0], d_w=full[1],
                               d_bias=full[2])
    for at, what in enumerate(("d_x", "d_w", "d_bias")):
        t = torch.empty_like(full[at])
        rrb.expert_linear_backward(d, p.x, p.d_off, p.w, pre=g, activation="silu", **{what: t})
        assert torch.equal(t, full[at])


@pytest.mark.parametrize("sizes,i,o", [([700, 1, 600, 0, 300], 520, 776), ([3, 0, 9], 264, 136), ([60, 90], 99, 77)])
def test_repeats_streams_and_graphs(sizes, i, o):
    """The same bits from call to call, on another stream, and from a captured
    graph replayed among eager work with changed inputs."""
    require_gpu()
    p = Problem(13, sizes, i, o)
    d, ws = p.rows(o), torch.empty(rrb.expert_gated_backward_workspace(p.N, i, o, p.G), dtype=torch.uint8, device=DEV)
    wl = p.put(_bf16(p.rng, (p.G, i, o)))

    def outs():
        return [p.out(*s) for s in ((p.N, o), (p.N, o), (p.N, o), (p.N, i), (p.N, i), (p.G, o, i), (p.G, o, i),
                                    (p.G, i, o), (p.G, i))]

    def run(t, w=None):
        rrb.expert_gated(p.x, p.d_off, p.w, p.w2, t[0], save_gate=t[1], save_up=t[2])
        rrb.expert_linear(t[0], p.d_off, wl, t[3])
        rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, t[1], t[2], d_x=t[4], d_w_gate=t[5], d_w_up=t[6],
                                  workspace=w)
        rrb.expert_linear_backward(t[3], t[0], p.d_off, wl, d_w=t[7], d_bias=t[8])

    a, b, c = outs(), outs(), outs()
    run(a)
    run(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(c)
    torch.cuda.synchronize()
    for q, r, s in zip(a, b, c):
        assert torch.equal(q, r) and torch.equal(q, s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, ws)
    for step in range(3):
        p.x[torch.from_numpy(p.used)] = _bf16(_rng(14, step), (int(p.used.sum()), i)).to(DEV)
        run(a, ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for q, r in zip(a, b):
            assert torch.equal(q, r), step


def test_stream_argument():
    require_gpu()
    p = Problem(15, [90, 40], 72, 56)
    d, g, u = p.rows(p.o), p.rows(p.o), p.rows(p.o)
    want, got = [[p.out(p.N, p.i), p.out(p.G, p.o, p.i), p.out(p.G, p.o, p.i)] for _ in range(2)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for t, stream in ((want, None), (got, s)):
        rrb.expert_gated_backward(d, p.x, p.d_off, p.w, p.w2, g, u, d_x=t[0], d_w_gate=t[1], d_w_up=t[2],
                                  stream=stream)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)


# ---- the gate ------------------------------------------------------------------
#
# Weights are fp32: e^(l - m) is off by at most 2 steps of its argument's error,
# |l - m| 2^-24 + 2^-23, the sum by E 2^-24 relative, the quotient by 2^-23:
# below (E + |l - m| + 8) 2^-23 relative.  bf16 gradients add half a step.

GATES = [(1, 1, 1), (1, 8, 8), (5, 7, 3), (64, 64, 6), (33, 65, 16), (130, 128, 1), (40, 256, 8), (9, 300, 7),
         (17, 1000, 16), (3, 1024, 16), (4099, 96, 4), (5000, 40, 5), (4500, 256, 8), (4200, 130, 16), (4100, 250, 3), (4097, 600, 2)]


def _scores(T, E, kind, dtype):
    rng = _rng(20, T, E)
    l = rng.standard_normal((T, E)).astype(np.float32) * (1 if kind != "wide" else 30)
    if kind == "ties":
        l = np.round(l * 2) / 2
        l[l == 0] *= np.where(rng.random((l == 0).sum()) < 0.5, -1, 1)  # both zeros
    if kind == "masked":
        l[rng.random((T, E)) < 0.7] = -np.inf
        l[0] = -np.inf
    return torch.from_numpy(l.astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, BF])
@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "wide"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gate(dtype, kind, renorm):
    require_gpu()
    for T, E, k in GATES:
        _say(f"gate T={T} E={E} k={k} {kind}")
        logits = _scores(T, E, kind, dtype)
        n = logits.double().numpy()
        d_l = logits.to(DEV)
        idx = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
        w = torch.full((T, k), -1.0, device=DEV)
        rrb.moe_gate(d_l, idx, w, renormalize=renorm)
        want_i, want_w = OE.gate(n, k, renorm)
        assert np.array_equal(idx.cpu().numpy(), want_i), (T, E, k)
        live = np.where(np.isneginf(n), 0, n)
        span = np.abs(live).max(axis=1, keepdims=True) * 2
        rel = (E + span + 8) * 2.0 ** -23
        assert (np.abs(_np(w) - want_w) <= rel * want_w + 1e-37).all(), (T, E, k)
        dw = _rng(21, T, E).standard_normal((T, k)).astype(np.float32)
        d_logits = torch.full_like(d_l, -7.0)
        rrb.moe_gate_backward(d_l, idx, torch.from_numpy(dw).to(DEV), d_logits, renormalize=renorm)
        want = OE.gate_grad(n, want_i, dw.astype(np.float64), renorm)
        scale = OE.softmax(n)
        if renorm:
            sel = np.zeros_like(n)
            np.put_along_axis(sel, want_i, want_w, axis=1)
            scale = sel
        # p (dw - mean): both terms known to rel (the mean to k more additions)
        bound = scale * 3 * (rel + k * 2.0 ** -23) * np.abs(dw).max(axis=1, keepdims=True) * 2
        if dtype == BF:
            bound = bound + HALF * np.abs(want)
        assert (np.abs(_np(d_logits) - want) <= bound + 1e-37).all(), (T, E, k)


def test_gate_special_scores():
    """+inf shares the weight, NaN ranks first and spoils its own row alone."""
    require_gpu()
    inf, nan = float("inf"), float("nan")
    l = torch.tensor([[0, inf, 1, inf], [1, 2, nan, 3], [3, 2, 1, 0], [-inf, -inf, -inf, inf]], device=DEV)
    idx, w = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV)
    rrb.moe_gate(l, idx, w)
    assert idx.tolist() == [[1, 3], [2, 3], [0, 1], [3, 0]]
    assert w[0].tolist() == [0.5, 0.5] and torch.isnan(w[1]).all() and w[3].tolist() == [1.0, 0.0]
    assert torch.isfinite(w[2]).all()
    # a masked expert's dw is not used, an index out of range passed over
    l = torch.tensor([[0.0, -inf, -inf], [1.0, 2.0, 0.5]], device=DEV)
    idx = torch.tensor([[0, 1], [1, 99]], dtype=torch.int32, device=DEV)
    d = torch.tensor([[1.0, nan], [1.0, nan]], device=DEV)
    out = torch.empty_like(l)
    rrb.moe_gate_backward(l, idx, d, out)
    assert torch.isfinite(out).all() and out[0].tolist() == [0.0, 0.0, 0.0]


# ---- the combine's gradient ------------------------------------------------------

def _choices(rng, T, E, k):
    return np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)


def _slots(idx, E):
    T, k = idx.shape
    order = np.argsort((idx.astype(np.int64) * T + np.arange(T)[:, None]).reshape(-1), kind="stable")
    slot = np.empty(T * k, np.int64)
    slot[order] = np.arange(T * k)
    return slot.reshape(T, k)


@pytest.mark.parametrize("T,h,E,k,R", [(8, 8, 4, 1, 1), (16, 13, 8, 2, 2), (64, 136, 16, 3, 4), (40, 7168, 16, 8, 8),
                                       (24, 1032, 32, 16, 8), (512, 4096, 64, 4, 1), (32, 2049, 8, 5, 4)])
@pytest.mark.parametrize("host", [False, True])
def test_combine_backward(T, h, E, k, R, host):
    require_gpu()
    rng = _rng(30, T, h, k)
    idx, w, w2 = _choices(rng, T, E, k), rng.random((T, k)).astype(np.float32), rng.standard_normal((T, k)).astype("f")
    dy, z = _bf16(rng, (T, h)), _bf16(rng, (T * k, h))
    slot = _slots(idx, E)
    dys = [t.contiguous().to(DEV) for t in dy.reshape(R, T // R, h)]
    if host:
        plan = rrb.MoePlan(R, h, E, idx, w, "combine")
        cut = np.cumsum([0] + [c // h for c in plan.in_count])
        zs = [z[a:b].contiguous().to(DEV) for a, b in zip(cut, cut[1:])]
    else:
        plan = rrb.MoeDevicePlan(R, T, h, E, k, "combine")
        plan.route(torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV))
        zs = [z.to(DEV)] + [None] * (R - 1)
    fresh = lambda: [None if t is None else torch.full_like(t, -7.25) for t in zs]
    nz, ny = _np(z), _np(dy)
    for weights in (None, w2):
        used = w if weights is None else weights
        dzs, dw = fresh(), torch.full((T, k), -7.0, device=DEV)
        plan.backward(dys, zs, dzs, d_weights=dw,
                      weights=None if weights is None else torch.from_numpy(weights).to(DEV))
        torch.cuda.synchronize()
        want_z, want_w = OE.combine_grad(ny, nz, slot, used.astype(np.float64))
        got = torch.cat([t for t in dzs if t is not None])
        _check("dz", got, want_z, ADD * np.abs(want_z), HALF * 1.01)
        bound = (h + 2) * ADD * (np.abs(ny)[:, None, :] * np.abs(nz[slot])).sum(axis=2)
        assert (np.abs(_np(dw) - want_w) <= bound).all()
        alone, dw2 = fresh(), torch.full((T, k), -7.0, device=DEV)
        kw = {"weights": None if weights is None else torch.from_numpy(weights).to(DEV)}
        plan.backward(dys, None, alone, **kw)
        plan.backward(dys, zs, None, d_weights=dw2, **kw)
        assert all(a is None or torch.equal(a, b) for a, b in zip(alone, dzs)) and torch.equal(dw, dw2)


def test_combine_backward_misaligned():
    require_gpu()
    T, h, E, k = 32, 64, 8, 2
    rng = _rng(31)
    idx, w = _choices(rng, T, E, k), rng.random((T, k)).astype(np.float32)
    put = Shifted(1)
    dy, z = put(_bf16(rng, (T, h))), put(_bf16(rng, (T * k, h)))
    plan = rrb.MoeDevicePlan(1, T, h, E, k, "combine")
    plan.route(torch.from_numpy(idx).to(DEV), torch.from_numpy(w).to(DEV))
    dz, dw = put(torch.zeros(T * k, h, dtype=BF)), torch.zeros(T, k, device=DEV)
    plan.backward([dy], [z], [dz], d_weights=dw)
    want_z, want_w = OE.combine_grad(_np(dy), _np(z), _slots(idx, E), w.astype(np.float64))
    _check("dz", dz, want_z, ADD * np.abs(want_z))
    assert (np.abs(_np(dw) - want_w) <= h * ADD * 200).all()


def test_combine_backward_many_experts_per_token():
    """A host plan's top-k above 16."""
    require_gpu()
    T, h, E, k = 24, 200, 48, 20
    rng = _rng(32)
    idx, w = _choices(rng, T, E, k), rng.random((T, k)).astype(np.float32)
    dy, z = _bf16(rng, (T, h)), _bf16(rng, (T * k, h))
    plan = rrb.MoePlan(1, h, E, idx, w, "combine")
    dz, dw = torch.zeros(T * k, h, dtype=BF, device=DEV), torch.zeros(T, k, device=DEV)
    plan.backward([dy.to(DEV)], [z.to(DEV)], [dz], d_weights=dw)
    slot = _slots(idx, E)
    want_z, want_w = OE.combine_grad(_np(dy), _np(z), slot, w.astype(np.float64))
    _check("dz", dz, want_z, ADD * np.abs(want_z))
    assert (np.abs(_np(dw) - want_w) <= (h + 2) * ADD * (np.abs(_np(dy))[:, None] * np.abs(_np(z)[slot])).sum(2)).all()


def test_failed_routing_does_no_work():
    """After a routing with a repeated expert every offset is 0, so the
    experts run on no rows, and the combine's gradient writes nothing; a good
    routing on the same plan works again."""
    require_gpu()
    T, h, E, k = 64, 32, 8, 2
    rng = _rng(33)
    idx, w = _choices(rng, T, E, k), torch.rand(T, k, device=DEV)
    bad = idx.copy()
    bad[5] = [3, 3]
    disp = rrb.MoeDevicePlan(1, T, h, E, k, "dispatch")
    comb = rrb.MoeDevicePlan(1, T, h, E, k, "combine", share=disp)
    off = torch.full((E + 1,), 9, dtype=torch.int32, device=DEV)
    x, dy = _bf16(rng, (T * k, h)).to(DEV), _bf16(rng, (T, h)).to(DEV)
    we = _bf16(rng, (E, 16, h)).to(DEV)
    for idx_, ok in ((bad, False), (idx, True)):
        disp.route(torch.from_numpy(idx_).to(DEV), w)
        disp.expert_offsets(off)
        y, dz, dw = (torch.full(s, -7.25, device=DEV, dtype=t) for s, t in
                     (((T * k, 16), BF), ((T * k, h), BF), ((T, k), torch.float32)))
        rrb.expert_gated(x, off, we, we, y)
        comb.backward([dy], [x], [dz], d_weights=dw)
        torch.cuda.synchronize()
        if ok:
            want = np.concatenate([[0], np.cumsum(np.bincount(idx.reshape(-1), minlength=E))])
            assert off.tolist() == want.tolist() and not (y == -7.25).all() and not (dw == -7.25).any()
        else:
            assert not off.any() and (y == -7.25).all() and (dz == -7.25).all() and (dw == -7.25).all()


# ---- the whole step ----------------------------------------------------------------

@pytest.mark.parametrize("T,h,f,E,k,R", [(64, 64, 96, 8, 2, 2), (256, 136, 72, 16, 4, 4), (8, 256, 64, 32, 8, 8),
                                         (1, 48, 40, 16, 4, 1)])
def test_moe_step(T, h, f, E, k, R):
    """Gate, route, dispatch, gated feed-forward, down projection, combine and
    every gradient back to scores, tokens and weights, as a training step runs
    them, against the oracle's step.  Each stage rounds its results once to
    bf16 (relative 2^-8): two before the output's own on the way forward (h,
    z), and up to eight on the way back, so norms of errors of at most 3 and
    9 times 2^-8 (roundings add in squares, so this is loose)."""
    require_gpu()
    _say(f"moe step T={T} h={h} f={f} E={E} k={k} R={R}")
    rng = _rng(40, T, h, f)
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    x, dy = _bf16(rng, (T, h)).to(DEV), _bf16(rng, (T, h)).to(DEV)
    wg, wu = (_bf16(rng, (E, f, h), h ** -0.5).to(DEV) for _ in range(2))
    wd = _bf16(rng, (E, h, f), f ** -0.5).to(DEV)
    n = T * k
    new = lambda *s, dtype=BF: torch.full(s, float("nan"), device=DEV).to(dtype)
    disp = rrb.MoeDevicePlan(R, T, h, E, k, "dispatch")
    comb = rrb.MoeDevicePlan(R, T, h, E, k, "combine", share=disp)
    shards = lambda t: list(t.reshape(R, T // R, h).unbind(0))
    arena = lambda t: [t] + [None] * (R - 1)

    idx, w = torch.zeros(T, k, dtype=torch.int32, device=DEV), new(T, k, dtype=torch.float32)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    xe, g, u, hh, z, y = new(n, h), new(n, f), new(n, f), new(n, f), new(n, h), new(T, h)
    d_z, d_h, d_xe, d_x = new(n, h), new(n, f), new(n, h), new(T, h)
    d_w, d_logits = new(T, k, dtype=torch.float32), new(T, E, dtype=torch.float32)
    d_wg, d_wu, d_wd = new(E, f, h), new(E, f, h), new(E, h, f)
    ones = torch.ones(T, k, device=DEV)

    def step():
        rrb.moe_gate(logits, idx, w, renormalize=True)
        disp.route(idx, w)
        disp.expert_offsets(off)
        disp.run(shards(x), arena(xe))
        rrb.expert_gated(xe, off, wg, wu, hh, save_gate=g, save_up=u)
        rrb.expert_linear(hh, off, wd, z)
        comb.run(arena(z), shards(y))
        comb.backward(shards(dy), arena(z), arena(d_z), d_weights=d_w)
        rrb.expert_linear_backward(d_z, hh, off, wd, d_x=d_h, d_w=d_wd)
        rrb.expert_gated_backward(d_h, xe, off, wg, wu, g, u, d_x=d_xe, d_w_gate=d_wg, d_w_up=d_wu)
        comb.run(arena(d_xe), shards(d_x), weights=ones)
        rrb.moe_gate_backward(logits, idx, d_w, d_logits, renormalize=True)

    step()
    disp.check()
    torch.cuda.synchronize()

    nl, nx, ny = _np(logits), _np(x), _np(dy)
    ng, nu_, nd = _np(wg), _np(wu), _np(wd)
    oi, ow = OE.gate(nl, k, True)
    assert np.array_equal(idx.cpu().numpy(), oi)
    o_off = np.concatenate([[0], np.cumsum(np.bincount(oi.reshape(-1), minlength=E))])
    assert off.tolist() == o_off.tolist()
    slot = _slots(oi, E)
    ox = np.empty((n, h))
    ox[slot.reshape(-1)] = np.repeat(nx, k, axis=0)
    assert np.array_equal(_np(xe), ox)
    oh, og, ou = OE.gated(ox, o_off, ng, nu_, "silu")
    oz = OE.linear(oh, o_off, nd)[0]
    oy = (ow[:, :, None] * oz[slot]).sum(axis=1)
    odz, odw = OE.combine_grad(ny, oz, slot, ow)
    odh, odwd, _ = OE.linear_grad(odz, oh, o_off, nd)
    odxe, odwg, odwu = OE.gated_grad(odh, ox, o_off, ng, nu_, og, ou, "silu")
    odx = odxe[slot].sum(axis=1)
    odl = OE.gate_grad(nl, oi, odw, True)

    def near(what, got, want, steps):
        err = np.sqrt(((_np(got) - want) ** 2).sum())
        assert err <= steps * HALF * np.sqrt((want ** 2).sum()), (what, err / np.sqrt((want ** 2).sum()))

    near("y", y, oy, 3)
    for what, got, want in (("d_w", d_w, odw), ("d_wd", d_wd, odwd), ("d_wg", d_wg, odwg), ("d_wu", d_wu, odwu),
                            ("d_x", d_x, odx), ("d_logits", d_logits, odl)):
        near(what, got, want, 9)

    # the same step captured: three replays among eager steps, other tokens
    # and scores each time
    names = (y, d_w, d_wd, d_wg, d_wu, d_x, d_logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for q in range(3):
        x.copy_(_bf16(_rng(41, q), (T, h)))
        logits.copy_(torch.from_numpy(_rng(42, q).standard_normal((T, E)).astype(np.float32)))
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in names]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, names):
            assert torch.equal(a, b)
