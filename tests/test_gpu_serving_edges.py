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
