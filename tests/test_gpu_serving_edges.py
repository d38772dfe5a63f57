"""GPU tests of the serving calls at their edges, against the binary64 oracle:
infinite weights, both bf16 parts of h, every kernel of the layer, groups of
very unequal sizes, replays on changed inputs.  Bounds as in
tests/test_gpu_serving.py where a test does not state its own."""

import numpy as np
import pytest
import torch

import reduce_rank_buffers_amd as rrb
from oracle import experts as OE
from tests import test_gpu_serving as S
from tests import test_gpu_experts as X
from tests.gpu_util import DEV, require_gpu

BF = torch.bfloat16


# ---- infinite weights ------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 11, 40])
@pytest.mark.parametrize("f", [48, 47])
def test_decode_infinite_weights(T, f):
    """An infinite weight of the second product gives the infinity that its sign
    and h's make, not a NaN, also where h is a bf16 value (its second part is 0)
    or its two parts differ in sign; results without one are as ever.  One and
    more tokens than four meet an expert, on both forms of the kernels."""
    require_gpu()
    rng = X._rng(41, T, f)
    p = S.Layer(41, T, 2, 3, 64, f, idx=np.stack([rng.permutation(3)[:2] for _ in range(T)]))
    down = p.mats[2].cpu()
    for e in range(3):
        for n in range(0, 64, 3):
            v = float("inf") if (n + e) % 2 else float("-inf")
            down[e, n, (n + 5 * e) % f] = v
            p.wide[2][e, n, (n + 5 * e) % f] = v
    p.mats[2].copy_(down)
    p.run("silu")
    got = X._np(p.y)
    with np.errstate(invalid="ignore"):
        want, parts = OE.decode(p.x.double().numpy(), p.idx, p.nw.astype(np.float64), *p.wide, "silu")
        finite, bound = p.expect("silu")
    assert all((hid != 0).all() for _, hid, _, _ in parts.values())
    known = ~np.isnan(want)  # (two experts' infinities of both signs have no sum)
    assert known[:, ::3].any() and np.isinf(want[known]).any() and np.isfinite(want[:, 1::3]).all()
    assert np.isnan(got[~known]).all() and not np.isnan(got[known]).any()
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])
    X._check("y", p.y[:, 1::3], finite[:, 1::3], bound[:, 1::3])


@pytest.mark.gpu
@pytest.mark.parametrize("width", [8, 7])
@pytest.mark.parametrize("tokens", [1, 6])
def test_decode_infinite_weight_of_a_whole_h(width, tokens):
    """h = 1, which has no second part."""
    require_gpu()
    one = torch.zeros(1, width, width, dtype=BF)
    one[0, 0, 0] = 1
    x = torch.zeros(tokens, width, dtype=BF)
    x[:, 0] = 1
    down = torch.zeros(1, width, width, dtype=BF)
    down[0, 0, 0], down[0, 1, 0], down[0, 2, 0] = float("inf"), float("-inf"), 3
    y = torch.empty(tokens, width, dtype=BF, device=DEV)
    rrb.moe_decode(x.to(DEV), torch.zeros(tokens, 1, dtype=torch.int32, device=DEV), torch.ones(tokens, 1, device=DEV),
                   one.to(DEV), one.to(DEV), down.to(DEV), y, activation="none")
    want = torch.tensor([float("inf"), float("-inf"), 3] + [0.0] * (width - 3)).expand(tokens, width)
    assert torch.equal(y.float().cpu(), want)


# ---- groups of very unequal sizes ----------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("sizes", [[7] * 5 + [500] + [9, 0, 1, 33, 32] + [4] * 20, [0] * 7 + [1024] + [0] * 24,
                                   [65, 0, 1], [64], [33] + [31] * 3], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("i,o", [(208, 264), (2064, 136)])
def test_few_rows_on_average(sizes, i, o):
    """Arenas of at most 32 rows a group on average (and some just above): groups
    of one row tile, whose weights go past the caches, beside groups of many,
    whose tiles share theirs."""
    require_gpu()
    S._linear_int8(S.Integers(42, sizes, i, o), "gelu", True, True)
    S._gated_int8(S.Integers(43, sizes, i, o // 2, 2, 3), "silu")


@pytest.mark.gpu
def test_few_rows_of_an_arena():
    """A slice of the groups over the whole arena: eight times the rows that the
    offsets bound, the other rows left as they were."""
    require_gpu()
    S._linear_int8(S.Integers(44, [5, 0, 40, 1], 272, 200, 300, 20), "none", True, False)
    S._gated_int8(S.Integers(45, [5, 0, 40, 1], 272, 200, 300, 20), "silu")


# ---- both parts of h ---------------------------------------------------------------

class Exact:
    """A layer of whole numbers in which nothing is rounded but the result: x and
    the weights small integers (int8: with scales that are powers of two), g and
    u at most 255, so that h = g u has at most 16 bits and its two bf16 parts
    hold it, and every sum below 2^24 quarters.  Half of the tokens take expert
    0, so that experts have one token and many."""

    def __init__(self, T, k, E, h, f, int8=False):
        rng = X._rng(46, T, k, E, h, f)
        self.shape, self.int8 = (T, k, E, h, f), int8
        self.x = rng.integers(-3, 4, (T, h)).astype(np.float64)
        self.idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        for t in range(0, T, 2):
            if 0 not in self.idx[t]:
                self.idx[t, 0] = 0
        self.w = 2.0 ** rng.integers(-2, 1, (T, k))
        draw = lambda *s: np.clip(np.rint(rng.standard_normal(s) * 17 / h ** 0.5), -9, 9)
        self.m = [draw(E, f, h), draw(E, f, h), rng.integers(-1, 2, (E, h, f)).astype(np.float64)]
        self.s = [2.0 ** rng.integers(-1, 2, m.shape[:2]) if int8 else np.ones(m.shape[:2]) for m in self.m]

    def expect(self, parts=lambda h: h):
        """The result as a float64 array; `parts` is what becomes of a token's h."""
        T, k, E, h, f = self.shape
        y, mass = np.zeros((T, h)), np.zeros((T, h))
        for e in range(E):
            t, j = np.nonzero(self.idx == e)
            g, u = (self.x[t] @ m[e].T for m in self.m[:2])
            assert g.size == 0 or max(np.abs(g).max(), np.abs(u).max()) <= 255
            hid = (g * self.s[0][e]) * (u * self.s[1][e])
            add = self.w[t, j, None] * ((parts(hid) @ self.m[2][e].T) * self.s[2][e])
            np.add.at(y, t, add)
            np.add.at(mass, t, self.w[t, j, None] * ((np.abs(hid) @ np.abs(self.m[2][e]).T) * self.s[2][e]))
        # (quarters of h's scales, 1/4, and of Wd's, 1/2, and weights, 1/4: multiples of 1/32)
        assert mass.max() * 32 * 1.01 < 2 ** 24 or not self.int8
        assert mass.max() * 4 * 1.01 < 2 ** 24
        return y

    def run(self, **kw):
        to = lambda a, t: torch.from_numpy(a).to(t).to(DEV)
        y = torch.full(self.x.shape, -7.25, dtype=BF, device=DEV)
        rrb.moe_decode(to(self.x, BF), to(self.idx, torch.int32), to(self.w, torch.float32),
                       *(to(m, torch.int8 if self.int8 else BF) for m in self.m), y, activation="none",
                       scales=tuple(to(s, torch.float32) for s in self.s) if self.int8 else None, **kw)
        return y


def _round(y):
    return torch.from_numpy(y).float().to(BF)


# T, k, E, h, f, and the kernels they are for: the first kernel's tokens, the second's
# tokens and waves (d: for few experts), or tiles of registers (r).
EXACT = [
    (3, 2, 5, 64, 48),      # 8; 8 with 8 waves, a token's two columns 4 apart
    (8, 2, 3, 64, 48),      # 8; 8 with 8 waves, 8 apart
    (6, 2, 4, 4112, 48),    # 8; 8 with 4 waves
    (16, 2, 4, 64, 48),     # 16; 16 with 8 waves
    (12, 2, 9, 4112, 64),   # 16; 16 with 4 waves
    (40, 2, 32, 128, 64),   # 64; 64 with 8 waves
    (40, 2, 32, 4112, 64),  # 64; 64 with 4 waves
    (64, 8, 64, 4112, 48),  # 64; 64 with 4 waves, an expert with 32 tokens and more beside those of a few
    (64, 4, 8, 128, 48),    # 64; 64 d
    (3, 2, 5, 63, 47), (16, 2, 4, 63, 47), (24, 2, 3, 63, 47), (64, 4, 8, 63, 47),  # r: 1 1, 1 2, 2 4, 4 4
    (9, 2, 600, 64, 32),    # r 1 2: more experts than the tables in LDS hold
    (5, 2, 4, 64, 47), (5, 2, 4, 63, 48),  # bf16: one kernel of each kind
]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", EXACT, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("int8", [False, True])
def test_decode_exact(shape, int8):
    """Bit for bit, with nothing rounded but the result."""
    require_gpu()
    p = Exact(*shape, int8=int8)
    assert torch.equal(p.run().cpu(), _round(p.expect()))


@pytest.mark.parametrize("shape", EXACT, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("int8", [False, True])
def test_exact_layers_tell(shape, int8):
    """What test_decode_exact would see: without h's second part, with that of
    another channel, or with it taken off, more than a third of the results
    differ."""
    p = Exact(*shape, int8=int8)
    want = _round(p.expect())
    one = lambda h: torch.from_numpy(h).float().to(BF).double().numpy()
    wrong = {"no second part": one, "of the next channel": lambda h: one(h) + np.roll(h - one(h), 1, axis=1),
             "subtracted": lambda h: 2 * one(h) - h}
    for what, parts in wrong.items():
        off = (_round(p.expect(parts)) != want).double().mean().item()
        assert off > 0.33, f"{what}: {off}"


@pytest.mark.gpu
@pytest.mark.parametrize("shape", S.LAYERS, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("int8", [False, True])
def test_decode_within_two_parts(shape, int8, monkeypatch):
    """Random layers with h's rounding bounded by what two bf16 parts leave: half a
    step of a remainder that is itself at most half a step of h, 2^-16 of it."""
    require_gpu()
    monkeypatch.setattr(S, "HALF", 2.0 ** -16)
    k = S.LAYERS.index(shape)
    S.Layer(47, *shape[:5], int8=int8, beyond=shape[5]).check(S.ACTS[(k + int8) % 5])


@pytest.mark.gpu
@pytest.mark.parametrize("int8", [False, True])
def test_decode_large_within_two_parts(int8, monkeypatch):
    """The layer's full widths likewise."""
    monkeypatch.setattr(S, "HALF", 2.0 ** -16)
    S.test_decode_large(int8)


# ---- kernels that other sizes do not reach --------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("shape", [
    (12, 2, 9, 4112, 64),   # 9 to 16 tokens, the second kernel with four waves
    (40, 2, 32, 4112, 64),  # 17 to 64, four waves, not so few experts that all columns go at once
    (64, 8, 64, 4112, 48),  # the same with 8 tokens an expert and more
], ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("uneven", [False, True])
def test_decode_wide(shape, int8, uneven):
    """More than 256 tiles of channels, 9 tokens and more; uneven: every token on
    the first expert, half of them on the second, so that these go by turns."""
    require_gpu()
    T, k, E, h, f = shape
    rng = X._rng(48, *shape)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    if uneven:
        for t in range(T):
            rest = 2 + rng.permutation(E - 2)[:k]
            rest[0] = 0
            if t % 2 and k > 1:
                rest[1] = 1
            idx[t] = rest
    S.Layer(48, *shape, int8=int8, idx=idx).check(S.ACTS[(T + int8) % 5])


@pytest.mark.gpu
@pytest.mark.parametrize("n,width", [(4096, 1000), (4097, 2048), (4100, 4090), (4096, 4096), (4099, 515),  # waves
                                     (4096, 4097), (3, 40000), (2, 65536), (2, 70001), (1, 1 << 20)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_quantize_many_and_wide_rows(n, width, dtype):
    """A wave a row in two to eight turns, and workgroups whose rows take eight
    turns and those that are read twice."""
    require_gpu()
    x = S._rows(X._rng(49, n, width), n, width, dtype)
    q, s = S._quantize(S.Put(width & 1), x)
    wq, ws = OE.quantize(x.double().numpy())
    assert np.array_equal(s, ws) and np.array_equal(q, wq)


# ---- replays on changed inputs -------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("sizes,i,o", [([40, 0, 90, 3], 176, 136), ([1, 0, 30, 3], 177, 135)])
def test_products_replay_changed_inputs(sizes, i, o):
    """Quantised rows and both products captured together: each replay, on rows and
    group sizes that changed since the last, over results and intermediates that
    hold junk, gives the bits of an eager step with buffers of its own."""
    require_gpu()
    p = S.Integers(50, sizes, i, o)
    (wg, sg), (wu, su) = ([t.to(DEV) for t in p.weight()] for _ in range(2))
    wd = torch.from_numpy(p.rng.integers(-127, 128, (p.G, i, o)).astype(np.int8)).to(DEV)
    sd = torch.full((p.G, i), 0.01, device=DEV)
    x = X._bf16(p.rng, (p.N, i)).to(DEV)
    off = p.d_off.clone()

    def buffers():
        e = lambda n, t, v: torch.full((p.N, n) if n else (p.N,), v, dtype=t, device=DEV)
        return (e(i, torch.int8, 77), e(0, torch.float32, float("nan")), e(o, BF, 5.0), e(o, torch.int8, 77),
                e(0, torch.float32, float("nan")), e(i, BF, 5.0))

    def step(q, s, h, hq, hs, y):
        rrb.quantize_rows(x, q, s, offsets=off)
        rrb.expert_gated_int8(q, s, off, wg, sg, wu, su, h)
        rrb.quantize_rows(h, hq, hs, offsets=off)
        rrb.expert_linear_int8(hq, hs, off, wd, sd, y, residual=x)

    own = buffers()
    step(*own)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*own)
    seen = []
    for turn in range(4):
        x.copy_(X._bf16(p.rng, (p.N, i), 1 + turn))
        off.copy_(torch.from_numpy(X._offsets(np.roll(sizes, turn))))
        for t, junk in zip(own, buffers()):
            t.copy_(junk)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in own]
        eager = buffers()
        step(*eager)
        for a, b in zip(got, eager):
            assert torch.equal(a, b)
        assert not any(torch.equal(got[-1], y) for y in seen)
        seen.append(got[-1])


# ---- limits of h ------------------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("f", [524280, 524288])
def test_decode_h_of_two_gigabytes(f):
    """64 tokens with 16 choices each and rows of h whose offsets come to the end of
    31 bits (the kernel that reads h through a buffer), and past it (the one that
    does not).  Whole numbers, Wd zero but for some channels of h, the first and
    the last among them."""
    require_gpu()
    T, k, E, h = 64, 16, 16, 8
    rng = X._rng(51, f)
    gen = torch.Generator(device=DEV).manual_seed(6)
    some = np.unique(np.concatenate([[0, 7, 8, f - 1, f - 8, f - 9], rng.integers(0, f, 60)]))
    on = torch.from_numpy(some).to(DEV)
    draw = lambda *s: torch.empty(s, dtype=BF, device=DEV).random_(-3, 4, generator=gen)
    x, wg, wu, wd = draw(T, h), draw(E, f, h), draw(E, f, h), torch.zeros(E, h, f, dtype=BF, device=DEV)
    part = draw(E, h, len(some))
    wd[:, :, on] = part
    idx = torch.from_numpy(np.stack([rng.permutation(E) for _ in range(T)]).astype(np.int32))
    w = torch.full((T, k), 0.5, device=DEV)
    y = torch.empty(T, h, dtype=BF, device=DEV)
    rrb.moe_decode(x, idx.to(DEV), w, wg, wu, wd, y, activation="none")
    nx = X._np(x)
    want, _ = OE.decode(nx, idx.numpy(), X._np(w), X._np(wg[:, on]), X._np(wu[:, on]), X._np(part), "none")
    assert np.abs(want).max() < 2 ** 22
    assert torch.equal(y.cpu(), _round(want))


@pytest.mark.gpu
@pytest.mark.parametrize("f", [48, 47])
@pytest.mark.parametrize("exponent", [-130, -100, 90])
def test_decode_exact_of_any_magnitude(f, exponent):
    """Whole h times a power of two down to bf16's subnormal numbers and up to its
    largest, and Wd times the inverse of one."""
    require_gpu()
    p = Exact(6, 2, 4, 64, f)
    want = p.expect()
    half = exponent // 2
    p.m[0] *= 2.0 ** half
    p.m[1] *= 2.0 ** (exponent - half)
    p.m[2] *= 2.0 ** -(exponent + 10)
    assert torch.equal(p.run().cpu(), _round(want * 2.0 ** -10))
