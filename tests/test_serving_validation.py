"""The serving calls refuse what they cannot run, before any GPU work: the
Python binding and the C ABI itself.  Runs on the CPU."""

import ctypes

import pytest
import torch

import reduce_rank_buffers_amd as rrb
from reduce_rank_buffers_amd import _lib as L

E, U = L.RRB_EINVAL, L.RRB_EUNSUPPORTED


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _i8(*shape):
    return torch.zeros(shape, dtype=torch.int8)


def _f32(*shape):
    return torch.zeros(shape)


def _off(n, G):
    return torch.full((G + 1,), n, dtype=torch.int32)


def _call(fn, defaults, positional):
    def call(**kw):
        a = {**defaults(), **kw}
        return fn(*[a.pop(n) for n in positional], **a)
    return call


_quantize = _call(rrb.quantize_rows, lambda: dict(x=_bf(5, 8), q=_i8(5, 8), scale=_f32(5)), ("x", "q", "scale"))
_linear = _call(rrb.expert_linear_int8,
                lambda: dict(x=_i8(5, 8), x_scale=_f32(5), offsets=_off(5, 2), w=_i8(2, 6, 8), w_scale=_f32(2, 6),
                             out=_bf(5, 6)), ("x", "x_scale", "offsets", "w", "w_scale", "out"))
_gated = _call(rrb.expert_gated_int8,
               lambda: dict(x=_i8(5, 8), x_scale=_f32(5), offsets=_off(5, 2), w_gate=_i8(2, 6, 8), gate_scale=_f32(2, 6),
                            w_up=_i8(2, 6, 8), up_scale=_f32(2, 6), out=_bf(5, 6)),
               ("x", "x_scale", "offsets", "w_gate", "gate_scale", "w_up", "up_scale", "out"))
_decode = _call(rrb.moe_decode,
                lambda: dict(x=_bf(3, 8), topk_idx=torch.zeros(3, 2, dtype=torch.int32), topk_w=_f32(3, 2),
                             w_gate=_bf(4, 6, 8), w_up=_bf(4, 6, 8), w_down=_bf(4, 8, 6), out=_bf(3, 8)),
                ("x", "topk_idx", "topk_w", "w_gate", "w_up", "w_down", "out"))
_INT = dict(w_gate=_i8(4, 6, 8), w_up=_i8(4, 6, 8), w_down=_i8(4, 8, 6))
_SC = (_f32(4, 6), _f32(4, 6), _f32(4, 8))

REFUSED = [
    (_quantize, {}, "not on the current GPU"),
    (_quantize, {"x": _bf(5, 8).half()}, "neither bf16"),
    (_quantize, {"x": _bf(8)}, "x: expected"),
    (_quantize, {"x": None}, "x: expected"),
    (_quantize, {"x": _bf(5, 16)[:, ::2]}, "x: tensor is not contiguous"),
    (_quantize, {"q": _i8(5, 9)}, "q: shape"),
    (_quantize, {"q": torch.zeros(5, 8, dtype=torch.uint8)}, "q: dtype"),
    (_quantize, {"scale": _f32(4)}, "scale: shape"),
    (_quantize, {"scale": _bf(5)}, "scale: dtype"),
    (_quantize, {"offsets": torch.zeros(1, dtype=torch.int32)}, "offsets: expected"),
    (_quantize, {"offsets": torch.zeros(3, dtype=torch.int64)}, "offsets: dtype"),
    (_quantize, {"x": _bf(2, 5, 8), "q": _i8(2, 5, 8), "scale": _f32(2, 5), "offsets": _off(5, 1)},
     "x of two dimensions"),
    (_linear, {}, "not on the current GPU"),
    (_linear, {"x": _bf(5, 8)}, "x: dtype"),
    (_linear, {"w": _bf(2, 6, 8)}, "w: dtype"),
    (_linear, {"x_scale": _f32(6)}, "x_scale: shape"),
    (_linear, {"x_scale": None}, "x_scale is required"),
    (_linear, {"w_scale": _f32(6)}, "w_scale: shape"),
    (_linear, {"w_scale": _f32(2, 6).double()}, "w_scale: dtype"),
    (_linear, {"offsets": None}, "offsets is required with 2 groups"),
    (_linear, {"w": _i8(2, 6, 9)}, "w: 9 columns for rows of 8"),
    (_linear, {"out": _bf(5, 8)}, "out: shape"),
    (_linear, {"out": _f32(5, 6)}, "out: dtype"),
    (_linear, {"bias": _bf(6)}, "bias: shape"),
    (_linear, {"residual": _bf(5, 8)}, "residual: shape"),
    (_linear, {"activation": "tanh"}, "unknown activation"),
    (_gated, {}, "not on the current GPU"),
    (_gated, {"w_up": _i8(2, 7, 8)}, "w_up: shape"),
    (_gated, {"gate_scale": _f32(2, 7)}, "gate_scale: shape"),
    (_gated, {"up_scale": None}, "up_scale is required"),
    (_gated, {"out": _bf(4, 6)}, "out: shape"),
    (_decode, {}, "not on the current GPU"),
    (_decode, {"x": _f32(3, 8)}, "x: dtype"),
    (_decode, {"x": _bf(3, 9)}, "w_gate: 8 columns for rows of 9"),
    (_decode, {"x": _bf(8)}, "x: expected a tensor of 2"),
    (_decode, {"topk_idx": torch.zeros(3, 2, dtype=torch.int64)}, "topk_idx: dtype"),
    (_decode, {"topk_idx": torch.zeros(4, 2, dtype=torch.int32)}, "topk_idx: shape"),
    (_decode, {"topk_w": _f32(3, 3)}, "topk_w: shape"),
    (_decode, {"w_up": _bf(4, 6, 9)}, "w_up: shape"),
    (_decode, {"w_down": _bf(4, 6, 8)}, "w_down: shape"),
    (_decode, {"out": _bf(3, 6)}, "out: shape"),
    (_decode, {"activation": "tanh"}, "unknown activation"),
    (_decode, {"scales": _SC}, "w_gate: dtype"),
    (_decode, {**_INT}, "w_gate: dtype"),
    (_decode, {**_INT, "scales": _SC}, "not on the current GPU"),
    (_decode, {**_INT, "scales": _SC[:2]}, "scales: expected"),
    (_decode, {**_INT, "scales": (_SC[0], _SC[1], None)}, "scales: expected"),
    (_decode, {**_INT, "scales": (_SC[0], _SC[1], _f32(4, 6))}, "scales[2]: shape"),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_binding_refuses(librrb, case):
    call, kw, message = REFUSED[case]
    with pytest.raises(ValueError) as e:
        call(**kw)
    assert message in str(e.value)


# ---- the C ABI ---------------------------------------------------------------

P = 4096  # a non-NULL address that no refused call reads


def at(n):
    """n addresses far apart."""
    return [P + (i << 36) for i in range(n)]


def test_abi_quantize_refuses(librrb):
    f = librrb.rrb_quantize_rows
    for rows, width, dt, want in [(-1, 8, 0, E), (4, 0, 0, E), (4, 8, 2, E), (1 << 31, 8, 0, U),
                                  (4, (1 << 20) + 1, 0, U)]:
        assert f(rows, width, dt, P, None, 0, P, P, None) == want
    for i in (0, 3, 4):
        a = [P, None, 0, P << 8, P << 12]
        a[i] = None
        assert f(4, 8, 0, *a, None) == E
    assert f(4, 8, 0, P, P, 0, P, P, None) == E
    assert f(0, 8, 0, None, None, 0, None, None, None) == L.RRB_OK


def test_abi_quantize_refuses_overlaps(librrb):
    for dt, size in ((L.RRB_BF16, 2), (L.RRB_F32, 4)):
        sizes = [5 * 8 * size, 12, 5 * 8, 5 * 4]
        for o in (2, 3):
            for i in range(4):
                if i != o:
                    for shift in (sizes[i] - 1, 1 - sizes[o]):
                        a = at(4)
                        a[o] = a[i] + shift
                        assert librrb.rrb_quantize_rows(5, 8, dt, a[0], a[1], 2, a[2], a[3], None) == E
                        assert b"overlaps" in librrb.rrb_last_error()


def _spec(rows=4, i=8, o=8, G=1, act=0):
    return ctypes.byref(L.ExpertSpec(rows, i, o, G, act))


SPECS = [(_spec(rows=-1), E), (_spec(i=0), E), (_spec(o=0), E), (_spec(G=0), E), (_spec(act=5), E), (None, E),
         (_spec(rows=1 << 31), U), (_spec(i=1 << 17), U), (_spec(o=(1 << 20) + 1), U), (_spec(G=4097), U)]


@pytest.mark.parametrize("case", range(len(SPECS)))
def test_abi_products_refuse_specs(librrb, case):
    spec, want = SPECS[case]
    assert librrb.rrb_expert_linear_int8(spec, P, P, P, P, P, None, None, P, None) == want
    assert librrb.rrb_expert_gated_int8(spec, P, P, P, P, P, P, P, P, None) == want


def test_abi_products_refuse_pointers(librrb):
    s = _spec()
    for i in (0, 1, 3, 4, 7):
        a = at(5) + [None, None, P << 22]
        a[i] = None
        assert librrb.rrb_expert_linear_int8(s, *a, None) == E
    for i in (0, 1, 3, 4, 5, 6, 7):
        a = at(8)
        a[i] = None
        assert librrb.rrb_expert_gated_int8(s, *a, None) == E
    a = at(8)
    a[2] = None
    assert librrb.rrb_expert_gated_int8(_spec(G=2), *a, None) == E
    assert librrb.rrb_expert_linear_int8(_spec(rows=0), *[None] * 8, None) == L.RRB_OK
    assert librrb.rrb_expert_gated_int8(_spec(rows=0), *[None] * 8, None) == L.RRB_OK


def test_abi_products_refuse_overlaps(librrb):
    s = _spec(rows=4, i=8, o=16, G=2)
    x, xs, off, w, ws, b, y = 32, 16, 12, 256, 128, 64, 128
    for f, sizes, o in ((librrb.rrb_expert_linear_int8, [x, xs, off, w, ws, b, y, y], 7),
                        (librrb.rrb_expert_gated_int8, [x, xs, off, w, ws, w, ws, y], 7)):
        for i in range(o):
            for shift in (sizes[i] - 1, 1 - sizes[o]):
                a = at(8)
                a[o] = a[i] + shift
                assert f(s, *a, None) == E and b"overlaps" in librrb.rrb_last_error()


def _layer(T=3, h=8, f=6, experts=4, k=2, act=1):
    return ctypes.byref(L.DecodeSpec(T, h, f, experts, k, act, 0))


LAYERS = [(_layer(T=-1), E), (_layer(h=0), E), (_layer(f=0), E), (_layer(experts=0), E), (_layer(k=0), E),
          (_layer(act=5), E), (_layer(act=-1), E), (None, E), (_layer(T=65), U), (_layer(h=(1 << 20) + 1), U),
          (_layer(f=(1 << 20) + 1), U), (_layer(experts=1025), U), (_layer(k=17), U)]


@pytest.mark.parametrize("case", range(len(LAYERS)))
def test_abi_decode_refuses_specs(librrb, case):
    spec, want = LAYERS[case]
    n = ctypes.c_size_t(1)
    assert librrb.rrb_moe_decode_workspace(spec, ctypes.byref(n)) == want and n.value == 0
    assert librrb.rrb_moe_decode(spec, *[P] * 11, 1 << 30, None) == want


def test_abi_decode_refuses_pointers(librrb):
    n = ctypes.c_size_t()
    assert librrb.rrb_moe_decode_workspace(_layer(), None) == E
    assert librrb.rrb_moe_decode_workspace(_layer(), ctypes.byref(n)) == L.RRB_OK
    assert n.value == rrb.moe_decode_workspace(3, 2, 8, 6) == 3 * 2 * 2 * 8 * 2
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10):  # (6, 7, 8: one scale without the others)
        a = at(11)
        a[i] = None
        assert librrb.rrb_moe_decode(_layer(), *a, n.value, None) == E
    assert librrb.rrb_moe_decode(_layer(), *at(11), n.value - 1, None) == E
    a = at(11)
    a[10] += 8
    assert librrb.rrb_moe_decode(_layer(), *a, n.value, None) == E and b"aligned" in librrb.rrb_last_error()
    assert librrb.rrb_moe_decode(_layer(T=0), *[None] * 11, 0, None) == L.RRB_OK


def test_abi_decode_refuses_overlaps(librrb):
    n = rrb.moe_decode_workspace(3, 2, 8, 6)
    for integers in (False, True):
        w = 4 * 6 * 8 * (1 if integers else 2)
        sizes = [48, 24, 24, w, w, w, 96, 96, 128, 48, n]
        for o in (9, 10):
            for i in range(11):
                if i == o or (not integers and i in (6, 7, 8)):
                    continue
                for shift in (sizes[i] - 1, 1 - sizes[o]):
                    a = at(11)
                    a[o] = a[i] + shift
                    if o == 10:
                        a[o] &= ~15
                        if shift < 0:
                            a[o] += 16
                    if not integers:
                        a[6] = a[7] = a[8] = None
                    assert librrb.rrb_moe_decode(_layer(), *a, n, None) == E, (o, i, shift)
                    assert b"overlaps" in librrb.rrb_last_error()


def test_decode_workspace_refuses(librrb):
    with pytest.raises(rrb.RrbError) as e:
        rrb.moe_decode_workspace(65, 8, 64, 64)
    assert e.value.status == U
