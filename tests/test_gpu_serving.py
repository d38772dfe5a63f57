"""GPU parity of the serving calls (quantised rows, the experts' products in
8-bit integers, the expert layer of a few tokens) against the binary64 oracle.

Tolerances.  Quantised rows are exact, integers and scales.  An integer
product's sum is exact; its conversion to fp32 and the two scales round it three
times, 3 2^-24 of the value.  The layer's sums are of exact fp32 products (an
8-bit weight is exact in bf16) in some order: K 2^-23 sum |a b| for K terms and
the few joins, which 16 more terms cover.  h is rounded to bf16, 2^-8 of it.
Activations and factors as in tests/test_gpu_experts.py, and one rounding of the
result, 2^-8 of it.
"""

import numpy as np
import pytest
import torch

import reduce_rank_buffers_amd as rrb
from oracle import experts as OE
from tests import test_gpu_experts as X
from tests.gpu_util import DEV, require_gpu
from tests.test_gpu_experts import ACT, ACTS, ADD, BF, HALF, _check, _np, _offsets, _rng, _say

pytestmark = pytest.mark.gpu


class Put:
    """CPU tensors on the GPU, `shift` elements into a larger buffer whose other
    elements are NaN (integers: 127), so that any of them that reached a result
    would show."""

    def __init__(self, shift=0):
        self.shift = shift

    def __call__(self, t):
        if t is None:
            return None
        side = 4096
        fill = float("nan") if t.is_floating_point() else 127
        buf = torch.full((t.numel() + 2 * side,), fill, dtype=t.dtype, device=DEV)
        out = buf[side + self.shift:side + self.shift + t.numel()].reshape(t.shape)
        out.copy_(t)
        return out


# ---- quantised rows ------------------------------------------------------------

def _quantize(put, x, offsets=None):
    d = put(x)
    q, s = put(torch.full(x.shape, 99, dtype=torch.int8)), put(torch.full(x.shape[:-1], -7.0))
    rrb.quantize_rows(d, q, s, offsets=None if offsets is None else torch.from_numpy(offsets).to(DEV))
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


def _rows(rng, n, width, dtype):
    x = rng.standard_normal((n, width)) * np.exp(rng.standard_normal((n, 1)))
    x = torch.from_numpy(x.astype(np.float32)).to(dtype)
    if width > 3 and n > 2:
        # quotients at and beside ties: multiples of half of a row's scale
        m = x[0].abs().max()
        x[0, 1:3] = torch.stack([m / 2, -m / 4]).to(dtype)
        x[1] = 0
    return x


WIDTHS = [1, 2, 7, 8, 9, 64, 250, 512, 1000, 1024, 1031, 2048, 2056, 4096, 7168, 8192, 8200, 20001]


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("shift", [0, 1])
def test_quantize_rows(width, dtype, shift):
    require_gpu()
    for n in (1, 5, 33):
        x = _rows(_rng(1, width, n), n, width, dtype)
        q, s = _quantize(Put(shift), x)
        wq, ws = OE.quantize(x.double().numpy())
        assert np.array_equal(s, ws) and np.array_equal(q, wq), (n, width)


def test_quantize_every_bf16():
    """Every finite bf16 against the largest that is beside it in its row, and
    rows of subnormals and of the largest values."""
    require_gpu()
    bits = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(BF)
    x = torch.cat([bits.reshape(-1, 8), -bits.reshape(-1, 8).flip(0), bits.reshape(8, -1).T.contiguous()])
    q, s = _quantize(Put(), x)
    wq, ws = OE.quantize(x.double().numpy())
    assert np.array_equal(s, ws) and np.array_equal(q, wq)


def test_quantize_ties_and_subnormals():
    """fp32 rows whose quotients lie on a tie or one last place beside it, at
    scales from the smallest subnormal to the largest."""
    require_gpu()
    rows = []
    for e in list(range(-149, -120)) + [-101, -100, -99, -61, -60, -59, 0, 60, 119, 120]:
        s = np.float32(2.0) ** np.float32(e)
        top = np.float32(127.0) * s
        half = (np.arange(-126, 127, dtype=np.float32) + np.float32(0.5)) * s
        for v in (half, np.nextafter(half, np.float32(np.inf)), np.nextafter(half, np.float32(-np.inf))):
            rows.append(np.concatenate([[top], v]))
    rows += [np.float32(1.4e-45) * np.arange(k, k + 254) % 3e-43 for k in range(0, 200, 7)]
    x = torch.from_numpy(np.array(rows, dtype=np.float32))
    q, s = _quantize(Put(), x)
    wq, ws = OE.quantize(x.double().numpy())
    assert np.array_equal(s, ws) and np.array_equal(q, wq)


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("width", [3, 64, 1031, 9000])
def test_quantize_special_rows(dtype, width):
    """A row with an infinity or a NaN has scale NaN and zeros; others do not
    see it."""
    require_gpu()
    x = _rows(_rng(2, width), 9, width, dtype)
    x[2, width // 2] = float("inf")
    x[4, 0] = float("nan")
    x[6, width - 1] = float("-inf")
    q, s = _quantize(Put(), x)
    bad = [2, 4, 6]
    ok = [i for i in range(9) if i not in bad]
    assert np.isnan(s[bad]).all() and (q[bad] == 0).all()
    wq, ws = OE.quantize(x[ok].double().numpy())
    assert np.array_equal(s[ok], ws) and np.array_equal(q[ok], wq)


def test_quantize_offsets_and_dimensions():
    require_gpu()
    x = _rows(_rng(3), 40, 72, BF)
    x[:4] = x[30:] = float("nan")  # never read
    q, s = _quantize(Put(), x, np.array([4, 9, 9, 30], dtype=np.int32))
    wq, ws = OE.quantize(x[4:30].double().numpy())
    assert np.array_equal(q[4:30], wq) and np.array_equal(s[4:30], ws)
    for part in (slice(0, 4), slice(30, 40)):
        assert (q[part] == 99).all() and (s[part] == -7).all()
    # clamped to the arena, and empty
    x = _rows(_rng(4), 6, 16, BF)
    q, s = _quantize(Put(), x, np.array([-3, 900], dtype=np.int32))
    assert np.array_equal(q, OE.quantize(x.double().numpy())[0])
    for off in ([3, 3], [5, 2], [900, 1000]):
        q, s = _quantize(Put(), x, np.array(off, dtype=np.int32))
        assert (q == 99).all() and (s == -7).all()
    w = _rows(_rng(5), 6, 24, torch.float32).reshape(2, 3, 24)
    q, s = _quantize(Put(), w)
    wq, ws = OE.quantize(w.reshape(6, 24).double().numpy())
    assert np.array_equal(q.reshape(6, 24), wq) and np.array_equal(s.reshape(6), ws)
    e = torch.empty(0, 8, dtype=BF, device=DEV)
    rrb.quantize_rows(e, torch.empty(0, 8, dtype=torch.int8, device=DEV), torch.empty(0, device=DEV))


# ---- products in integers ----------------------------------------------------------

class Integers:
    """Rows grouped by `sizes`, `lead` unused rows before and `tail` behind, as
    integers; rows of no group have NaN for their scale."""

    def __init__(self, seed, sizes, i, o, lead=0, tail=0, shift=0):
        self.rng = _rng(seed, i, o, *sizes)
        self.off = _offsets(sizes, lead)
        self.N, self.G, self.i, self.o = int(self.off[-1]) + tail, len(sizes), i, o
        self.put = Put(shift)
        self.used = np.zeros(self.N, bool)
        for _, r in OE.groups(self.off):
            self.used[r] = True
        self.x = torch.from_numpy(self.rng.integers(-128, 128, (self.N, i)).astype(np.int8))
        self.sx = torch.from_numpy(np.exp(self.rng.standard_normal(self.N)).astype(np.float32) / 64)
        self.sx[~torch.from_numpy(self.used)] = float("nan")
        self.d_off = torch.from_numpy(self.off).to(DEV)

    def weight(self):
        w = torch.from_numpy(self.rng.integers(-128, 128, (self.G, self.o, self.i)).astype(np.int8))
        s = torch.from_numpy((np.exp(0.3 * self.rng.standard_normal((self.G, self.o))) / 64 * self.i ** -0.5)
                             .astype(np.float32))
        return w, s

    def out(self):
        return self.put(torch.full((self.N, self.o), -7.25, dtype=BF))

    def product(self, w, s):
        """The product, its sums exact (integers below 2^53) before the scales;
        NaN outside the groups."""
        y = OE.linear(self.x.double().numpy(), self.off, w.double().numpy())[0] * self.sx.double().numpy()[:, None]
        for e, rows in OE.groups(self.off):
            y[rows] *= s[e].double().numpy()
        return y

    def untouched(self, t):
        assert (_np(t)[~self.used] == -7.25).all(), "rows of no group were written"


SCALED = 3 * 2.0 ** -24


def _linear_int8(p, name, bias, residual):
    w, s = p.weight()
    b = X._bf16(p.rng, (p.G, p.o)) if bias else None
    r = X._bf16(p.rng, (p.N, p.o)) if residual else None
    y, put = p.out(), p.put
    rrb.expert_linear_int8(put(p.x), put(p.sx), p.d_off, put(w), put(s), y, bias=put(b), activation=name,
                           residual=put(r))
    torch.cuda.synchronize()
    pre = prod = p.product(w, s)
    if bias:
        pre = pre.copy()
        for e, rows in OE.groups(p.off):
            pre[rows] += b[e].double().numpy()
    want = OE.act(name, pre)
    e = 1.13 * (SCALED * np.abs(prod) + ADD * np.abs(pre)) + (0 if name == "none" else ACT * (1 + np.abs(pre)))
    if residual:
        nr = r.double().numpy()
        want = want + nr
        e = e + ADD * (np.abs(want) + np.abs(nr))
    _check("out", y, want, e)
    p.untouched(y)


def _gated_int8(p, name):
    (wg, sg), (wu, su) = p.weight(), p.weight()
    y, put = p.out(), p.put
    rrb.expert_gated_int8(put(p.x), put(p.sx), p.d_off, put(wg), put(sg), put(wu), put(su), y, activation=name)
    torch.cuda.synchronize()
    g, u = p.product(wg, sg), p.product(wu, su)
    want = OE.act(name, g) * u
    e = np.abs(u) * (1.13 * SCALED * np.abs(g) + ACT * (1 + np.abs(g))) + (SCALED + ADD) * np.abs(want)
    _check("out", y, want, e)
    p.untouched(y)


SHAPES = X.SHAPES + [([40, 3], 16, 32), ([70], 144, 72), ([9, 0, 200], 400, 96), ([3], 131071, 5)]


@pytest.mark.parametrize("shape", SHAPES, ids=X._ids)
@pytest.mark.parametrize("lead,tail,shift", [(0, 0, 0), (3, 5, 0), (0, 2, 1)])
def test_linear_int8(shape, lead, tail, shift):
    require_gpu()
    k = SHAPES.index(shape) + lead + shift
    _linear_int8(Integers(11, *shape, lead=lead, tail=tail, shift=shift), ACTS[k % 5], k % 2 == 0, k % 3 == 0)


@pytest.mark.parametrize("shape", SHAPES, ids=X._ids)
@pytest.mark.parametrize("lead,tail,shift", [(0, 0, 0), (3, 5, 0), (0, 2, 1)])
def test_gated_int8(shape, lead, tail, shift):
    require_gpu()
    k = SHAPES.index(shape) + lead + shift
    _gated_int8(Integers(12, *shape, lead=lead, tail=tail, shift=shift), ACTS[(k + 2) % 5])


@pytest.mark.parametrize("i,o", [(208, 4104), (128, 4104), (2064, 1032), (2061, 2050)])
@pytest.mark.parametrize("lead,tail", [(0, 0), (7, 9)])
def test_large_int8(i, o, lead, tail):
    """Enough tiles for every tile shape."""
    require_gpu()
    _say(f"large int8 {i} -> {o}")
    _linear_int8(Integers(13, X.RAGGED, i, o, lead, tail), ACTS[i % 5], True, True)
    _gated_int8(Integers(14, X.RAGGED, i, o // 2, lead, tail), ACTS[(i + 2) % 5])


@pytest.mark.parametrize("sizes,i,o", [([1500, 0, 300, 1], 2064, 2056), ([700, 129, 64, 1, 0, 300], 1040, 2056),
                                       ([2500, 1, 0, 4000, 77], 528, 4104), ([900, 0, 65, 257], 272, 1032),
                                       ([8000], 272, 4104), ([300, 130, 0, 1, 500], 4112, 520),
                                       ([64, 1, 30, 0] * 8, 1040, 264)], ids=lambda v: str(v)[:24])
def test_int8_tile_shapes(sizes, i, o):
    """Each tile shape that the sizes choose, with partial tiles in both
    directions and a residual in the output's place."""
    require_gpu()
    _say(f"int8 tiles {sizes} {i} {o}")
    _gated_int8(Integers(31, sizes, i, o, 1, 2), "silu")
    _gated_int8(Integers(32, sizes, i, o // 2), "gelu")
    _linear_int8(Integers(33, sizes, i, o, 1, 2), "gelu_tanh", True, True)
    p = Integers(34, sizes, i, o)
    w, s = p.weight()
    r = X._bf16(p.rng, (p.N, p.o))
    y = p.put(r)
    rrb.expert_linear_int8(p.put(p.x), p.put(p.sx), p.d_off, p.put(w), p.put(s), y, residual=y)
    prod, nr = p.product(w, s), r.double().numpy()
    _check("out", y, prod + nr, SCALED * np.abs(prod) + ADD * (np.abs(prod) + np.abs(nr)))


def test_int8_sums_are_exact():
    """The largest sums: all -128 against all -128 at the largest depth."""
    require_gpu()
    K = (1 << 17) - 1
    for k in (K, K - 15):  # a partial and a whole last chunk
        x = torch.full((2, k), -128, dtype=torch.int8, device=DEV)
        w = torch.full((1, 3, k), -128, dtype=torch.int8, device=DEV)
        y = torch.empty(2, 3, dtype=BF, device=DEV)
        rrb.expert_linear_int8(x, torch.ones(2, device=DEV), None, w, torch.full((1, 3), 2.0 ** -20, device=DEV), y)
        want = float(torch.tensor(np.float32(16384 * k) * np.float32(2.0 ** -20)).to(BF))
        assert (y.float() == want).all(), k


def test_int8_scales_of_any_size():
    """Row scales far from the columns': the product is in range where the value
    is.  Zero rows give the epilogue of 0, NaN rows NaN, and no other row sees
    them."""
    require_gpu()
    x = torch.full((6, 32), 64, dtype=torch.int8, device=DEV)
    w = torch.full((1, 8, 32), 2, dtype=torch.int8, device=DEV)
    sx = torch.tensor([1e-30, 1e30, 0.0, float("nan"), 1.0, 1e-38], device=DEV)
    sw = torch.full((1, 8), 1.0, device=DEV)
    y = torch.empty(6, 8, dtype=BF, device=DEV)
    rrb.expert_linear_int8(x, sx, None, w, sw, y)
    want = (4096.0 * sx).to(BF)
    assert torch.equal(y[:3], want[:3, None].expand(3, 8)) and y[3].isnan().all()
    assert torch.equal(y[4:], want[4:, None].expand(2, 8))
    rrb.expert_linear_int8(x, torch.full((6,), 1e-30, device=DEV), None, w, torch.full((1, 8), 1e30, device=DEV), y)
    assert ((y.float() - 4096).abs() <= 4096 * HALF).all()


def test_int8_in_place_residual_and_dense():
    require_gpu()
    p = Integers(15, [150], 80, 200)
    w, s = p.weight()
    r = X._bf16(p.rng, (p.N, p.o))
    y = r.to(DEV)
    rrb.expert_linear_int8(p.x.to(DEV), p.sx.to(DEV), None, w.to(DEV), s.to(DEV), y, residual=y)
    nr = r.double().numpy()
    prod = p.product(w, s)
    _check("out", y, prod + nr, SCALED * np.abs(prod) + ADD * (np.abs(prod) + np.abs(nr)))


def test_int8_arena_past_4_gib():
    """Rows, results and weights whose byte offsets pass 32 bits."""
    require_gpu()
    _say("int8 arena past 4 GiB")
    N, i, o, G = 70000, 65536, 8, 2
    x = torch.empty(N, i, dtype=torch.int8, device=DEV)
    x.random_(-128, 128, generator=torch.Generator(device=DEV).manual_seed(3))
    w = torch.randint(-128, 128, (G, o, i), device=DEV, dtype=torch.int8)
    sx, sw = torch.full((N,), 2.0 ** -10, device=DEV), torch.full((G, o), 2.0 ** -6, device=DEV)
    off = torch.tensor([0, 69000, N], dtype=torch.int32, device=DEV)
    y = torch.empty(N, o, dtype=BF, device=DEV)
    rrb.expert_linear_int8(x, sx, off, w, sw, y)
    for rows, g in ((slice(0, 40), 0), (slice(68990, 69000), 0), (slice(69000, 69010), 1), (slice(N - 40, N), 1)):
        want = (x[rows].double() @ w[g].double().T * 2.0 ** -16).cpu().numpy()
        _check("out", y[rows], want, SCALED * np.abs(want))
    q, s = torch.empty_like(y, dtype=torch.int8), torch.empty(N, device=DEV)
    rrb.quantize_rows(y, q, s)
    wq, ws = OE.quantize(_np(y))
    assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


# ---- the layer of a few tokens --------------------------------------------------------

class Layer:
    """Tokens, choices and an expert layer's weights (bf16, or integers with
    scales).  Experts that no token chose are NaN (integers: their scales)."""

    def __init__(self, seed, T, k, E, h, f, int8=False, shift=0, idx=None, beyond=0):
        rng = self.rng = _rng(seed, T, k, E, h, f)
        self.T, self.k, self.E, self.h, self.f, self.int8 = T, k, E, h, f, int8
        put = self.put = Put(shift)
        if idx is None:
            idx = np.stack([rng.permutation(E + 2 * beyond)[:k] for _ in range(T)]) - beyond
        self.idx = np.asarray(idx, dtype=np.int32).reshape(T, k)
        w = rng.random((T, k)).astype(np.float32)
        self.nw = w / w.sum(axis=1, keepdims=True)
        self.x = X._bf16(rng, (T, h))
        live = np.isin(np.arange(E), self.idx)
        self.mats, self.scales, self.wide = [], [], []
        for o, i in ((f, h), (f, h), (h, f)):
            if int8:
                m = torch.from_numpy(rng.integers(-128, 128, (E, o, i)).astype(np.int8))
                s = torch.from_numpy((np.exp(0.3 * rng.standard_normal((E, o))) / 64 * i ** -0.5).astype(np.float32))
                s[torch.from_numpy(~live)] = float("nan")
                self.scales.append(put(s))
                self.wide.append(m.double().numpy() * s.double().numpy()[:, :, None])
            else:
                m = X._bf16(rng, (E, o, i), i ** -0.5)
                m[torch.from_numpy(~live)] = float("nan")
                self.wide.append(m.double().numpy())
            self.mats.append(put(m))
        self.d_x, self.d_idx, self.d_w = put(self.x), put(torch.from_numpy(self.idx)), put(torch.from_numpy(self.nw))
        self.y = put(torch.full((T, h), -7.25, dtype=BF))
        self.work = torch.full((rrb.moe_decode_workspace(T, k, h, f),), 255, dtype=torch.uint8, device=DEV)

    def run(self, name, **kw):
        return rrb.moe_decode(self.d_x, self.d_idx, self.d_w, *self.mats, self.y, activation=name,
                              scales=tuple(self.scales) if self.int8 else None,
                              workspace=kw.pop("workspace", self.work), **kw)

    def expect(self, name):
        """The result and its bound."""
        x, w = self.x.double().numpy(), self.nw.astype(np.float64)
        wg, wu, wd = self.wide
        want, parts = OE.decode(x, self.idx, w, wg, wu, wd, name)
        bound = np.zeros_like(want)
        sc = SCALED if self.int8 else 0.0
        for (t, j), (z, hid, g, u) in parts.items():
            e = self.idx[t, j]
            eg = (self.h + 16) * ADD * (np.abs(wg[e]) @ np.abs(x[t])) + sc * np.abs(g)
            eu = (self.h + 16) * ADD * (np.abs(wu[e]) @ np.abs(x[t])) + sc * np.abs(u)
            eh = np.abs(u) * (1.13 * eg + ACT * (1 + np.abs(g))) + np.abs(OE.act(name, g)) * eu + 1.13 * eg * eu
            eh = eh + HALF * (np.abs(hid) + eh) + ADD * np.abs(hid)
            az = np.abs(wd[e]) @ (np.abs(hid) + eh)
            ez = np.abs(wd[e]) @ eh + (self.f + 16) * ADD * az + sc * np.abs(z)
            bound[t] += w[t, j] * (ez + (self.k + 16) * ADD * az)
        return want, bound

    def check(self, name, **kw):
        self.run(name, **kw)
        torch.cuda.synchronize()
        _check("y", self.y, *self.expect(name))


LAYERS = [
    (6, 2, 5, 264, 301, 0), (6, 2, 5, 301, 264, 0), (30, 2, 5, 72, 203, 1), (30, 2, 5, 203, 72, 1),
    (64, 4, 8, 256, 144, 0), (20, 6, 6, 4160, 64, 0), (12, 2, 600, 64, 32, 0), (8, 3, 1024, 64, 32, 1),
    (3, 16, 1023, 96, 48, 0), (33, 2, 400, 96, 32, 10), (64, 16, 513, 64, 16, 0),
    # T, k, E, h, f, experts beyond either end
    (1, 1, 1, 8, 8, 0), (1, 1, 1, 1, 1, 0), (1, 8, 64, 512, 256, 0), (2, 2, 3, 7, 5, 0), (3, 1, 4, 64, 48, 1),
    (5, 3, 12, 1001, 333, 6), (16, 4, 8, 256, 128, 0), (17, 2, 3, 136, 72, 0), (16, 16, 40, 72, 200, 0),
    (33, 3, 5, 130, 66, 2), (40, 1, 1, 264, 40, 0), (64, 8, 32, 320, 96, 64), (64, 2, 2, 200, 104, 0),
    (64, 16, 1024, 24, 8, 0), (4, 5, 1000, 16, 24, 0), (48, 4, 7, 2048, 31, 0), (9, 2, 4, 33, 2056, 0),
    (7, 4, 6, 4096, 512, 0),
]


@pytest.mark.parametrize("shape", LAYERS, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("shift", [0, 1])
def test_decode(shape, int8, shift):
    require_gpu()
    k = LAYERS.index(shape)
    _say(f"decode {shape} int8 {int8}")
    p = Layer(21, *shape[:5], int8=int8, shift=shift, beyond=shape[5])
    p.check(ACTS[(k + int8 + shift) % 5])


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("int8", [False, True])
def test_decode_activations(name, int8):
    require_gpu()
    Layer(22, 6, 3, 5, 192, 80, int8=int8).check(name)


@pytest.mark.parametrize("int8", [False, True])
def test_decode_choices(int8):
    """Tokens without choices here, the same expert twice, all tokens on one
    expert, experts of no token."""
    require_gpu()
    low, high = -2 ** 31, 2 ** 31 - 1
    p = Layer(23, 4, 3, 5, 96, 40, int8=int8, idx=[[4, 4, 4], [-1, 5, high], [0, 4, 0], [low, 2, 2]])
    p.check("silu")
    assert (p.y[1] == 0).all()
    Layer(24, 64, 1, 9, 72, 40, int8=int8, idx=[[7]] * 64).check("relu")
    Layer(24, 31, 2, 9, 72, 40, int8=int8, idx=[[7, 7]] * 31).check("gelu")
    p = Layer(25, 20, 2, 4, 72, 40, int8=int8, idx=[[-1, 4]] * 20)
    p.run("silu")
    assert (p.y == 0).all()


@pytest.mark.parametrize("int8", [False, True])
def test_decode_values_do_not_leak(int8):
    """A token with an infinity or a NaN, and experts with them, show in the
    tokens that meet them and in no other, bit for bit."""
    require_gpu()
    for T, f in ((9, 72), (40, 20)):
        idx = np.stack([np.arange(T) % 5, (np.arange(T) + 1) % 5], axis=1)
        p = Layer(26, T, 2, 7, 104, f, int8=int8, idx=idx)
        p.run("silu")
        clean = p.y.clone()
        p.d_x[3, 5] = float("nan")
        p.d_x[7, 100] = float("inf")
        if int8:
            p.scales[0][4, 3] = float("nan")
            p.scales[2][1] = float("inf")
        else:
            p.mats[0][4, 3, 9] = float("nan")
            p.mats[2][1, :, 0] = float("inf")
        p.run("silu")
        hit = np.zeros(T, bool)
        hit[[3, 7]] = True
        hit |= (idx == 4).any(axis=1) | (idx == 1).any(axis=1)
        hit_t = torch.from_numpy(hit).to(DEV)
        assert torch.equal(p.y[~hit_t], clean[~hit_t])
        assert not p.y[3].isfinite().any() and not p.y[torch.from_numpy((idx == 4).any(axis=1)).to(DEV)].isfinite().any()


@pytest.mark.parametrize("width", [8, 7])
def test_decode_hidden_values_that_round_to_infinity(width):
    """h half a step above bf16's largest: finite in fp32, an infinity once
    rounded, and no NaN."""
    require_gpu()
    bf = lambda *s: torch.zeros(s, dtype=BF)
    x, wg, wu, wd = bf(1, width), bf(1, width, width), bf(1, width, width), bf(1, width, width)
    x[0, :2] = 1
    wg[0, 0, 0], wg[0, 0, 1], wu[0, 0, 0] = 1.9921875 * 2.0 ** 63, 2.0 ** 55, 2.0 ** 64
    wd[0, :, 0] = 1
    assert (wg[0, 0, 0].double() + wg[0, 0, 1].double()) * 2.0 ** 64 < torch.finfo(torch.float32).max
    y = torch.empty(1, width, dtype=BF, device=DEV)
    rrb.moe_decode(x.to(DEV), torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.ones(1, 1, device=DEV), wg.to(DEV),
                   wu.to(DEV), wd.to(DEV), y, activation="none")
    assert torch.isposinf(y).all()


def test_decode_zero_weight_of_a_finite_expert():
    require_gpu()
    p = Layer(27, 3, 2, 4, 64, 48)
    p.nw[:, 1] = 0
    p.d_w[:, 1] = 0
    p.check("silu")


@pytest.mark.parametrize("int8", [False, True])
def test_decode_large(int8):
    """Weights whose byte offsets pass 32 bits, and the layer's full widths; a
    sample of tokens against the oracle."""
    require_gpu()
    _say("decode large")
    T, k, E, h, f = 6, 2, 160 if not int8 else 300, 7168, 2048
    gen = torch.Generator(device=DEV).manual_seed(5)
    mats, scales = [], []
    for o, i in ((f, h), (f, h), (h, f)):
        if int8:
            m = torch.empty(E, o, i, dtype=torch.int8, device=DEV)
            m.random_(-127, 128, generator=gen)
            scales.append(torch.full((E, o), i ** -0.5 / 74, device=DEV))
        else:
            m = torch.empty(E, o, i, dtype=BF, device=DEV)
            m.normal_(0, i ** -0.5, generator=gen)
        mats.append(m)
    idx = torch.tensor([[0, E - 1], [E - 1, E - 2], [5, 0], [E - 1, 3], [E // 2, E - 3], [E - 4, 1]], dtype=torch.int32,
                       device=DEV)
    x = torch.empty(T, h, dtype=BF, device=DEV).normal_(0, 1, generator=gen)
    w = torch.full((T, k), 0.5, device=DEV)
    y = torch.empty_like(x)
    rrb.moe_decode(x, idx, w, *mats, y, scales=tuple(scales) if int8 else None)
    for t in range(T):
        want, mass = np.zeros(h), np.zeros(h)
        for j in range(k):
            e = int(idx[t, j])
            full = [m[e].double() * (s[e].double()[:, None] if int8 else 1)
                    for m, s in zip(mats, scales or [None] * 3)]
            g, u = full[0] @ x[t].double(), full[1] @ x[t].double()
            hid = g / (1 + torch.exp(-g)) * u
            want += 0.5 * (full[2] @ hid).cpu().numpy()
            # h is off by its rounding and by its projections' sums, (K + 16) 2^-23
            # of their terms' sizes, with a slope of at most 1.13
            eg, eu = ((h + 16) * ADD * (m.abs() @ x[t].double().abs()) for m in full[:2])
            eh = HALF * hid.abs() + u.abs() * (1.13 * eg + ACT * (1 + g.abs())) + g.abs() * eu + 1.13 * eg * eu
            mass += 0.5 * (full[2].abs() @ (1.01 * eh + (f + 32) * ADD * hid.abs())).cpu().numpy()
        _check("y", y[t], want, mass)


@pytest.mark.parametrize("int8", [False, True])
def test_decode_repeats_streams_and_graphs(int8):
    """The same bits again, on another stream, with a workspace of its own, and
    replayed from two graphs that share a workspace, on changed inputs, with
    eager work between."""
    require_gpu()
    p = Layer(28, 12, 4, 9, 264, 136, int8=int8)
    p.run("silu")
    first = p.y.clone()
    for _ in range(3):
        p.y.fill_(3)
        p.run("silu")
        assert torch.equal(p.y, first)
    p.y.fill_(3)
    p.run("silu", workspace=None)
    assert torch.equal(p.y, first)
    s = torch.cuda.Stream()
    p.y.fill_(3)
    s.wait_stream(torch.cuda.current_stream())
    p.run("silu", stream=s, workspace=None)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(p.y, first)
    with torch.cuda.stream(s):
        p.run("silu")
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graphs = []
    for name in ("silu", "relu"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            p.run(name)
        graphs.append((name, g))
    for turn in range(4):
        p.x = X._bf16(p.rng, (p.T, p.h))
        p.idx = np.roll(p.idx, turn, axis=0)
        p.d_x.copy_(p.x)
        p.d_idx.copy_(torch.from_numpy(p.idx))
        for name, g in graphs:
            p.y.fill_(3)
            p.work.fill_(255)
            g.replay()
            torch.cuda.synchronize()
            got = p.y.clone()
            p.run(name)
            assert torch.equal(p.y, got)
            _check("y", got, *p.expect(name))


def test_decode_scales_off_16_bytes():
    """Weights on 16-byte boundaries, scales and results 4 and 2 bytes off."""
    require_gpu()
    p = Layer(35, 5, 3, 6, 256, 96, int8=True)
    put = Put(1)
    p.scales = [put(s.cpu()) for s in p.scales]
    p.d_w, p.d_idx, p.y = put(p.d_w.cpu()), put(p.d_idx.cpu()), put(p.y.cpu())
    p.check("silu")


def test_calls_refuse_tensors_off_the_gpu():
    """One tensor on the host among those on the GPU, whichever it is."""
    require_gpu()
    p = Layer(36, 3, 2, 4, 32, 16, int8=True)
    args = [p.d_x, p.d_idx, p.d_w, *p.mats, p.y]
    for i in range(len(args)):
        a = list(args)
        a[i] = a[i].cpu()
        with pytest.raises(ValueError, match="not on the current GPU"):
            rrb.moe_decode(*a, scales=tuple(p.scales), workspace=p.work)
    with pytest.raises(ValueError, match="not on the current GPU"):
        rrb.moe_decode(*args, scales=(p.scales[0], p.scales[1].cpu(), p.scales[2]), workspace=p.work)
    with pytest.raises(ValueError, match="not on the current GPU"):
        rrb.moe_decode(*args, scales=tuple(p.scales), workspace=p.work.cpu())
    q = Integers(37, [5, 3], 32, 16)
    (w, s), put = q.weight(), q.put
    args = [put(q.x), put(q.sx), q.d_off, put(w), put(s), q.out()]
    for i in range(len(args)):
        a = list(args)
        a[i] = a[i].cpu()
        with pytest.raises(ValueError, match="not on the current GPU"):
            rrb.expert_linear_int8(*a)
        with pytest.raises(ValueError, match="not on the current GPU"):
            rrb.expert_gated_int8(a[0], a[1], a[2], a[3], a[4], args[3], args[4], a[5])
    x = torch.zeros(4, 8, dtype=BF, device=DEV)
    for a in ((x.cpu(), torch.zeros(4, 8, dtype=torch.int8, device=DEV), torch.zeros(4, device=DEV)),
              (x, torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, device=DEV)),
              (x, torch.zeros(4, 8, dtype=torch.int8, device=DEV), torch.zeros(4))):
        with pytest.raises(ValueError, match="not on the current GPU"):
            rrb.quantize_rows(*a)


def test_decode_refuses_workspaces():
    require_gpu()
    p = Layer(38, 3, 2, 4, 32, 16)
    for bad in (p.work[:-1], torch.empty(p.work.numel() + 16, dtype=torch.uint8, device=DEV)[8:]):
        with pytest.raises(rrb.RrbError):
            p.run("silu", workspace=bad)
    with pytest.raises(ValueError):
        p.run("silu", workspace=p.work.view(torch.int8))
    with pytest.raises(ValueError):
        p.run("silu", workspace=torch.empty(2 * p.work.numel(), dtype=torch.uint8, device=DEV)[::2])


def test_decode_without_tokens():
    require_gpu()
    bf = lambda *s: torch.zeros(s, dtype=BF, device=DEV)
    y = bf(0, 8)
    rrb.moe_decode(bf(0, 8), torch.zeros(0, 2, dtype=torch.int32, device=DEV), torch.zeros(0, 2, device=DEV),
                   bf(3, 4, 8), bf(3, 4, 8), bf(3, 8, 4), y)


def test_products_repeat_and_replay():
    """Quantised rows and both products captured together and replayed."""
    require_gpu()
    p = Integers(29, [40, 0, 90, 3], 176, 136)
    (wg, sg), (wu, su) = ([t.to(DEV) for t in p.weight()] for _ in range(2))
    x = X._bf16(p.rng, (p.N, p.i)).to(DEV)
    wd = torch.from_numpy(p.rng.integers(-127, 128, (p.G, p.i, p.o)).astype(np.int8)).to(DEV)
    sd = torch.full((p.G, p.i), 0.01, device=DEV)
    q, s = torch.empty(p.N, p.i, dtype=torch.int8, device=DEV), torch.empty(p.N, device=DEV)
    h, hq, hs = torch.empty(p.N, p.o, dtype=BF, device=DEV), torch.empty(p.N, p.o, dtype=torch.int8, device=DEV), s.clone()
    y = torch.empty(p.N, p.i, dtype=BF, device=DEV)

    def step():
        rrb.quantize_rows(x, q, s, offsets=p.d_off)
        rrb.expert_gated_int8(q, s, p.d_off, wg, sg, wu, su, h)
        rrb.quantize_rows(h, hq, hs, offsets=p.d_off)
        rrb.expert_linear_int8(hq, hs, p.d_off, wd, sd, y, residual=x)

    step()
    first = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for turn in range(3):
        for t in (y, h):
            t.fill_(5)
        hq.fill_(9)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, first)
        step()
        assert torch.equal(y, first)
        x.mul_(1)
        torch.cuda.synchronize()


# ---- a run of them together --------------------------------------------------------------

@pytest.mark.parametrize("T,h,f,E,k,R", [(64, 256, 96, 8, 2, 2), (40, 512, 128, 16, 4, 4)])
def test_serving_a_layer(T, h, f, E, k, R):
    """A batch through gate, rows quantised before they are dispatched (half of
    the bytes), products in integers and combine; then the same tokens through
    moe_decode with the same weights.  The two differ by what quantising rows
    costs: a row's values are off by half a step, max |x| / 254 each."""
    require_gpu()
    _say(f"serving {T} {h} {f}")
    rng = _rng(30, T, h, f, E)
    x = X._bf16(rng, (T, h))
    dense = [torch.from_numpy((rng.standard_normal(s) * s[2] ** -0.5).astype(np.float32)).to(DEV)
             for s in ((E, f, h), (E, f, h), (E, h, f))]
    mats = []
    for m in dense:
        q, s = torch.empty_like(m, dtype=torch.int8), torch.empty(m.shape[:2], device=DEV)
        rrb.quantize_rows(m, q, s)
        mats.append((q, s))
    (wg, sg), (wu, su), (wd, sd) = mats
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    idx, w = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    rrb.moe_gate(logits, idx, w, renormalize=True)
    d_x = x.to(DEV)
    xq, xs = torch.empty(T, h, dtype=torch.int8, device=DEV), torch.empty(T, device=DEV)
    rrb.quantize_rows(d_x, xq, xs)
    # Rows of h bytes travel as h / 2 elements of 16 bits, scales as rows of two.
    rows = rrb.MoeDevicePlan(R, T, h // 2, E, k, "dispatch")
    scales = rrb.MoeDevicePlan(R, T, 2, E, k, "dispatch")
    comb = rrb.MoeDevicePlan(R, T, h, E, k, "combine")
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    for plan in (rows, scales, comb):
        plan.route(idx, w)
    rows.expert_offsets(off)
    n = T * k
    rq, rs = torch.empty(n, h // 2, dtype=torch.int16, device=DEV), torch.empty(n, 2, dtype=torch.int16, device=DEV)
    none = [None] * (R - 1)
    rows.run([t.contiguous() for t in xq.view(torch.int16).chunk(R)], [rq] + none)
    scales.run([t.contiguous() for t in xs.view(torch.int16).reshape(T, 2).chunk(R)], [rs] + none)
    hh, z = torch.empty(n, f, dtype=BF, device=DEV), torch.empty(n, h, dtype=BF, device=DEV)
    rrb.expert_gated_int8(rq.view(torch.int8), rs.view(torch.float32).reshape(n), off, wg, sg, wu, su, hh)
    hq, hs = torch.empty(n, f, dtype=torch.int8, device=DEV), torch.empty(n, device=DEV)
    rrb.quantize_rows(hh, hq, hs, offsets=off)
    rrb.expert_linear_int8(hq, hs, off, wd, sd, z)
    ys = [torch.empty(T // R, h, dtype=BF, device=DEV) for _ in range(R)]
    comb.run([z] + none, ys)
    got = _np(torch.cat(ys))

    # By the oracle, with the same integers.
    nidx, nw = idx.cpu().numpy(), w.cpu().double().numpy()
    wide = [q.cpu().double().numpy() * s.cpu().double().numpy()[:, :, None] for q, s in mats]
    nq, ns = OE.quantize(x.double().numpy())
    want, parts = OE.decode(nq * ns[:, None].astype(np.float64), nidx, nw, *wide, "silu")
    # h is rounded to bf16 and to integers, z to bf16
    bound = np.zeros_like(want)
    for (t, j), (zz, hid, g, u) in parts.items():
        e = nidx[t, j]
        eh = (2 * ACT * (1 + np.abs(g))) * np.abs(u) + 8 * ADD * np.abs(hid) + HALF * np.abs(hid)
        eh = eh + (np.abs(hid).max() + eh.max()) / 254 * (1 + 1e-4)
        bound[t] += nw[t, j] * (np.abs(wide[2][e]) @ eh + 2 * HALF * np.abs(zz) + 8 * ADD * np.abs(zz))
    err = np.abs(got - want) - bound - HALF * np.abs(want)
    assert err.max() <= 0, f"off by {err.max()} over the bound"

    got_y = torch.empty(64 if T > 64 else T, h, dtype=BF, device=DEV)
    rrb.moe_decode(d_x, idx, w, wg, wu, wd, got_y, scales=(sg, su, sd))
    full, parts = OE.decode(x.double().numpy(), nidx, nw, *wide, "silu")
    err = np.linalg.norm(_np(got_y) - full) / np.linalg.norm(full)
    assert err <= 2 * HALF, err
