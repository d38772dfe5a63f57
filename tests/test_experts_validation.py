"""The gate's and the experts' calls refuse what they cannot run, before any GPU
work: the Python binding (shapes, types, strides, missing and overlapping
tensors, tensors off the GPU) and the C ABI itself (sizes, NULL pointers,
limits, workspaces).  Runs on the CPU."""

import ctypes

import pytest
import torch

import reduce_rank_buffers_amd as rrb
from reduce_rank_buffers_amd import _lib as L


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _off(n, G):
    return torch.full((G + 1,), n, dtype=torch.int32)


def _gated(**kw):
    a = dict(x=_bf(5, 8), offsets=_off(5, 2), w_gate=_bf(2, 6, 8), w_up=_bf(2, 6, 8), out=_bf(5, 6))
    a.update(kw)
    return rrb.expert_gated(a.pop("x"), a.pop("offsets"), a.pop("w_gate"), a.pop("w_up"), a.pop("out"), **a)


def _gated_back(**kw):
    a = dict(d_out=_bf(5, 6), x=_bf(5, 8), offsets=_off(5, 2), w_gate=_bf(2, 6, 8), w_up=_bf(2, 6, 8),
             gate=_bf(5, 6), up=_bf(5, 6), d_x=_bf(5, 8), d_w_gate=_bf(2, 6, 8), d_w_up=_bf(2, 6, 8))
    a.update(kw)
    pos = [a.pop(n) for n in ("d_out", "x", "offsets", "w_gate", "w_up", "gate", "up")]
    return rrb.expert_gated_backward(*pos, **a)


def _linear(**kw):
    a = dict(x=_bf(5, 8), offsets=_off(5, 2), w=_bf(2, 6, 8), out=_bf(5, 6))
    a.update(kw)
    return rrb.expert_linear(a.pop("x"), a.pop("offsets"), a.pop("w"), a.pop("out"), **a)


def _linear_back(**kw):
    a = dict(d_out=_bf(5, 6), x=_bf(5, 8), offsets=_off(5, 2), w=_bf(2, 6, 8), d_x=_bf(5, 8))
    a.update(kw)
    return rrb.expert_linear_backward(*[a.pop(n) for n in ("d_out", "x", "offsets", "w")], **a)


def _gate(**kw):
    a = dict(logits=torch.zeros(4, 8), topk_idx=torch.zeros(4, 2, dtype=torch.int32), topk_w=torch.zeros(4, 2))
    a.update(kw)
    return rrb.moe_gate(**a)


def _gate_back(**kw):
    a = dict(logits=torch.zeros(4, 8), topk_idx=torch.zeros(4, 2, dtype=torch.int32), d_topk_w=torch.zeros(4, 2),
             d_logits=torch.zeros(4, 8))
    a.update(kw)
    return rrb.moe_gate_backward(**a)


_SHARED = _bf(5, 8)

REFUSED = [
    (_gated, {}, "not on the current GPU"),
    (_gated, {"x": _bf(5, 8).float()}, "x: dtype"),
    (_gated, {"x": _bf(8)}, "x: expected a tensor of 2"),
    (_gated, {"x": None}, "x: expected a tensor"),
    (_gated, {"x": _bf(5, 9)}, "w_gate: 8 columns for rows of 9"),
    (_gated, {"x": _bf(5, 16)[:, ::2]}, "x: tensor is not contiguous"),
    (_gated, {"w_up": _bf(2, 7, 8)}, "w_up: shape"),
    (_gated, {"w_up": _bf(3, 6, 8)}, "w_up: shape"),
    (_gated, {"w_gate": _bf(6, 8)}, "w_gate: expected a tensor of 3"),
    (_gated, {"out": _bf(4, 6)}, "out: shape"),
    (_gated, {"offsets": None}, "offsets is required with 2 groups"),
    (_gated, {"offsets": torch.zeros(3, dtype=torch.int64)}, "offsets: dtype"),
    (_gated, {"offsets": _off(5, 3)}, "offsets: shape"),
    (_gated, {"activation": "tanh"}, "unknown activation"),
    (_gated, {"save_gate": _bf(5, 6)}, "go together"),
    (_gated, {"save_gate": _bf(5, 6), "save_up": _bf(5, 5)}, "save_up: shape"),
    (_gated_back, {}, "not on the current GPU"),
    (_gated_back, {"d_x": None, "d_w_gate": None, "d_w_up": None}, "no gradient asked for"),
    (_gated_back, {"d_w_up": None}, "go together"),
    (_gated_back, {"gate": _bf(5, 8)}, "gate: shape"),
    (_gated_back, {"d_out": _bf(5, 6).half()}, "d_out: dtype"),
    (_gated_back, {"d_x": _bf(4, 8)}, "d_x: shape"),
    (_linear, {}, "not on the current GPU"),
    (_linear, {"bias": _bf(6)}, "bias: shape"),
    (_linear, {"bias": torch.zeros(2, 6)}, "bias: dtype"),
    (_linear, {"residual": _bf(5, 8)}, "residual: shape"),
    (_linear, {"save_pre": _bf(5, 8)}, "save_pre: shape"),
    (_linear, {"out": None}, "not on the current GPU"),
    (_linear_back, {}, "not on the current GPU"),
    (_linear_back, {"d_x": None}, "no gradient asked for"),
    (_linear_back, {"activation": "silu"}, "pre is required"),
    (_linear_back, {"d_bias": _bf(6)}, "d_bias: shape"),
    (_gate, {}, "not on the current GPU"),
    (_gate, {"logits": torch.zeros(4, 8).half()}, "neither bf16"),
    (_gate, {"logits": torch.zeros(8)}, "logits: expected"),
    (_gate, {"topk_idx": torch.zeros(4, 9, dtype=torch.int32)}, "9 experts per token of 8"),
    (_gate, {"topk_idx": torch.zeros(4, 0, dtype=torch.int32)}, "0 experts per token"),
    (_gate, {"topk_idx": torch.zeros(4, 2, dtype=torch.int64)}, "topk_idx: dtype"),
    (_gate, {"topk_w": torch.zeros(4, 3)}, "topk_w: shape"),
    (_gate_back, {}, "not on the current GPU"),
    (_gate_back, {"d_logits": _bf(4, 8)}, "d_logits: dtype"),
    (_gate_back, {"d_topk_w": torch.zeros(3, 2)}, "d_topk_w: shape"),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_binding_refuses(librrb, case):
    call, kw, message = REFUSED[case]
    with pytest.raises(ValueError) as e:
        call(**kw)
    assert message in str(e.value)


def _bare_plan(tk):
    p = rrb.MoeDevicePlan.__new__(rrb.MoeDevicePlan)
    p.handle = None
    p._lib = None
    p.nranks, p.tk, p.dtype, p.experts = 2, tk, L.RRB_BF16, 4
    p.in_count, p.out_count = [64, 0], [16, 16]
    return p


BACKWARD = {"dispatch": "combine plans only", "none": "no gradient", "dys": "d_ys[1]", "zs": "zs[0]",
            "dzs": "d_zs[0]", "dw": "d_weights", "w": "weights", "device": "not on the current GPU"}


@pytest.mark.parametrize("case", list(BACKWARD))
def test_combine_backward_refuses(case):
    p = _bare_plan(None if case == "dispatch" else 8)
    dys, zs, dzs = [_bf(16), _bf(16)], [_bf(64), None], [_bf(64), None]
    dw, w = torch.zeros(4, 2), torch.zeros(4, 2)
    if case == "none":
        dzs = dw = None
    elif case == "dys":
        dys = dys[:1]
    elif case == "zs":
        zs = [_bf(63)]
    elif case == "dzs":
        dzs = [None]
    elif case == "dw":
        dw = torch.zeros(4, 2).double()
    elif case == "w":
        w = torch.zeros(7)
    with pytest.raises(ValueError) as e:
        p.backward(dys, zs, dzs, d_weights=dw, weights=w)
    assert BACKWARD[case] in str(e.value)


def test_expert_offsets_refuses():
    p = _bare_plan(None)
    for bad in (None, torch.zeros(5), torch.zeros(4, dtype=torch.int32)):
        with pytest.raises(ValueError):
            p.expert_offsets(bad)


# ---- the C ABI ---------------------------------------------------------------

P = 4096  # a non-NULL address that no refused call reads


def at(n):
    """n addresses far apart."""
    return [P + (i << 36) for i in range(n)]


def _spec(rows=4, i=8, o=8, G=1, act=0):
    return ctypes.byref(L.ExpertSpec(rows, i, o, G, act))


SPECS = [(_spec(rows=-1), L.RRB_EINVAL), (_spec(i=0), L.RRB_EINVAL), (_spec(o=0), L.RRB_EINVAL),
         (_spec(G=0), L.RRB_EINVAL), (_spec(act=5), L.RRB_EINVAL), (_spec(act=-1), L.RRB_EINVAL),
         (None, L.RRB_EINVAL), (_spec(rows=1 << 31), L.RRB_EUNSUPPORTED),
         (_spec(i=(1 << 20) + 1), L.RRB_EUNSUPPORTED), (_spec(o=(1 << 20) + 1), L.RRB_EUNSUPPORTED),
         (_spec(G=4097), L.RRB_EUNSUPPORTED)]


@pytest.mark.parametrize("case", range(len(SPECS)))
def test_abi_refuses_specs(librrb, case):
    spec, want = SPECS[case]
    n = ctypes.c_size_t()
    assert librrb.rrb_expert_gated(spec, P, P, P, P, P, None, None, None) == want
    assert librrb.rrb_expert_linear(spec, P, P, P, None, None, P, None, None) == want
    assert librrb.rrb_expert_gated_backward(spec, P, P, P, P, P, P, P, P, P, P, P, 1 << 40, None) == want
    assert librrb.rrb_expert_linear_backward(spec, P, P, P, P, P, P, P, P, P, 1 << 40, None) == want
    for f in (librrb.rrb_expert_gated_backward_workspace, librrb.rrb_expert_linear_backward_workspace):
        assert f(spec, ctypes.byref(n)) == want and n.value == 0


def test_abi_refuses_pointers(librrb):
    s, E = _spec(), L.RRB_EINVAL
    f = librrb.rrb_expert_gated
    for i in (0, 2, 3, 4):
        a = at(5) + [None, None]
        a[i] = None
        assert f(s, *a, None) == E
    assert f(s, *at(6), None, None) == E
    assert f(_spec(G=2), P, None, P, P, P, None, None, None) == E
    f = librrb.rrb_expert_linear
    for i in (0, 2, 5):
        a = at(3) + [None, None, P << 20, None]
        a[i] = None
        assert f(s, *a, None) == E
    f = librrb.rrb_expert_gated_backward
    for i in (0, 1, 3, 4, 5, 6, 8, 10):
        a = at(11)
        a[i] = None
        assert f(s, *a, 1 << 20, None) == E
    a = at(11)
    a[7] = a[8] = a[9] = None
    assert f(s, *a, 1 << 20, None) == E
    assert f(s, *at(11), 4 * 8 * 4 - 1, None) == E
    assert f(s, *at(10), (P << 30) + 8, 1 << 20, None) == E
    f = librrb.rrb_expert_linear_backward
    for i in (0, 1, 3, 8):
        a = at(9)
        a[i] = None
        assert f(s, *a, 1 << 20, None) == E
    a = at(9)
    a[4] = None
    assert f(_spec(act=1), *a, 1 << 20, None) == E
    a = at(9)
    a[5] = a[6] = a[7] = None
    assert f(s, *a, 1 << 20, None) == E
    assert librrb.rrb_expert_gated_backward_workspace(s, None) == E
    assert librrb.rrb_expert_linear_backward_workspace(s, None) == E


def test_abi_refuses_overlaps(librrb):
    """An output that shares its last byte with an input or another output."""
    s, E = _spec(rows=4, i=8, o=16, G=2), L.RRB_EINVAL
    x, y, w, off = 4 * 8 * 2, 4 * 16 * 2, 2 * 8 * 16 * 2, 12

    def refused(f, args, sizes, outs, *more):
        for o in outs:
            for i in range(len(args)):
                if i == o or args[i] is None:
                    continue
                a = list(args)
                a[o] = a[i] + sizes[i] - 1
                a[o] -= a[o] % 16 if o == len(args) - 1 and more else 0
                assert f(s, *a, *more, None) == E
                assert b"overlaps" in librrb.rrb_last_error()

    refused(librrb.rrb_expert_gated, at(7), [x, off, w, w, y, y, y], (4, 5, 6))
    refused(librrb.rrb_expert_linear, at(7), [x, off, w, 2 * 16 * 2, y, y, y], (5, 6))
    ws = 4 * 16 * 2 * 2
    refused(librrb.rrb_expert_gated_backward, at(11), [y, x, off, w, w, y, y, x, w, w, ws], (7, 8, 9, 10), 1 << 20)
    a = at(9)
    a[4] = None
    refused(librrb.rrb_expert_linear_backward, a, [y, x, off, w, y, x, w, 64, ws // 2], (5, 6, 7, 8), 1 << 20)


def test_abi_gate_refuses(librrb):
    g, b = librrb.rrb_moe_gate, librrb.rrb_moe_gate_backward
    E, U = L.RRB_EINVAL, L.RRB_EUNSUPPORTED
    for T, e, k, dt, fl, want in [(-1, 8, 2, 1, 0, E), (4, 0, 1, 1, 0, E), (4, 8, 0, 1, 0, E), (4, 8, 9, 1, 0, E),
                                  (4, 8, 2, 2, 0, E), (4, 8, 2, 1, 2, E), (4, 1025, 2, 1, 0, U),
                                  (4, 64, 17, 1, 0, U), (1 << 40, 8, 2, 1, 0, U)]:
        assert g(T, e, k, dt, fl, P, P, P, None) == want
        assert b(T, e, k, dt, fl, P, P, P, P, None) == want
    for i in range(3):
        a = [P, P, P]
        a[i] = None
        assert g(4, 8, 2, 1, 0, *a, None) == E
    for i in range(4):
        a = [P] * 4
        a[i] = None
        assert b(4, 8, 2, 1, 0, *a, None) == E
    assert g(0, 8, 2, 1, 0, None, None, None, None) == L.RRB_OK
    assert b(0, 8, 2, 1, 0, None, None, None, None, None) == L.RRB_OK


def test_abi_plans_refuse(librrb):
    uni = rrb.Plan(2, 64, "bf16", rrb.PARTIAL, rrb.REPLICATED, "reduce")
    none = L.ptr_array([None, None])
    assert librrb.rrb_moe_expert_offsets(uni.handle, P, None) == L.RRB_EINVAL
    assert librrb.rrb_moe_expert_offsets(None, P, None) == L.RRB_EINVAL
    assert librrb.rrb_moe_combine_backward(uni.handle, none, none, none, None, None, None) == L.RRB_EINVAL
    h = ctypes.c_void_p()
    for d in (L.RRB_MOE_DISPATCH, L.RRB_MOE_COMBINE):
        assert librrb.rrb_plan_create_rows_device(2, 4, 8, 4, 2, d, ctypes.byref(h)) == L.RRB_OK
        # not bound; a dispatch plan has no combine gradient
        assert librrb.rrb_moe_combine_backward(h, none, none, none, None, P, None) == L.RRB_EINVAL
        assert librrb.rrb_moe_expert_offsets(h, P, None) == L.RRB_EINVAL
        librrb.rrb_plan_destroy(h)


def test_workspace_sizes(librrb):
    assert rrb.expert_gated_backward_workspace(10, 4, 13, 2) == 10 * 16 * 2 * 2
    assert rrb.expert_linear_backward_workspace(10, 4, 13, 2) >= 10 * 16 * 2
    assert rrb.expert_gated_backward_workspace(0, 4, 13, 2) == 0


def test_linear_backward_workspace_holds_the_bias_sums(librrb):
    """Where a bias gradient's rows are split, its fp32 sums have room behind
    dZ, and a workspace without it is refused."""
    n = rrb.expert_linear_backward_workspace(32768, 8, 64, 1)
    assert n == 32768 * 64 * 2 + 64 * 64 * 4
    a = at(9)
    assert librrb.rrb_expert_linear_backward(_spec(rows=32768, o=64), *a, n - 1, None) == L.RRB_EINVAL
    assert b"workspace of" in librrb.rrb_last_error()


def test_abi_gate_refuses_overlaps(librrb):
    """An output that shares its last or first byte with an input or the other
    output."""
    T, E, k = 5, 8, 2
    for dt, scores in ((L.RRB_BF16, T * E * 2), (L.RRB_F32, T * E * 4)):
        chosen = T * k * 4
        for call, sizes, outs in ((librrb.rrb_moe_gate, [scores, chosen, chosen], (1, 2)),
                                  (librrb.rrb_moe_gate_backward, [scores, chosen, chosen, scores], (3,))):
            for o in outs:
                for i in range(len(sizes)):
                    if i == o:
                        continue
                    for shift in (sizes[i] - 1, 1 - sizes[o]):
                        a = at(len(sizes))
                        a[o] = a[i] + shift
                        assert call(T, E, k, dt, 0, *a, None) == L.RRB_EINVAL
                        assert b"overlaps" in librrb.rrb_last_error()


def test_abi_takes_empty_arrays_anywhere(librrb):
    """Without rows x, dx and dout are empty: where they lie does not matter."""
    s, w = _spec(rows=0, i=8, o=16, G=2), P + 64
    assert librrb.rrb_expert_linear_backward(s, w, w, P << 20, P, w, w, None, None, None, 0, None) == L.RRB_OK
    assert librrb.rrb_expert_gated_backward(s, w, w, P << 20, P, P << 8, w, w, w, None, None, None, 0, None) == L.RRB_OK


def test_abi_combine_backward_refuses_overlaps(librrb):
    """dz or dw over one byte of dy, z, the weights, each other or another
    rank's dz (host plan of 2 ranks, each with rows; the addresses are compared
    before the plan's maps are asked for)."""
    T, k, E, h = 4, 2, 4, 24
    idx = (ctypes.c_int32 * (T * k))(0, 2, 1, 3, 0, 3, 1, 2)
    w = (ctypes.c_float * (T * k))(*[0.5] * (T * k))
    plan = ctypes.c_void_p()
    assert librrb.rrb_plan_create_rows(2, T, h, E, k, idx, w, L.RRB_MOE_COMBINE, ctypes.byref(plan)) == L.RRB_OK
    rows = T * k // 2 * h * 2  # two tokens of each expert: four rows a rank
    size = [T // 2 * h * 2] * 2 + [rows] * 4 + [T * k * 4] * 2  # dy dy, z z, dz dz, weights, dw

    def call(a):
        return librrb.rrb_moe_combine_backward(plan, L.ptr_array(a[:2]), L.ptr_array(a[2:4]), L.ptr_array(a[4:6]),
                                               a[6], a[7], None)

    assert call(at(8)) == L.RRB_EINVAL and b"not bound" in librrb.rrb_last_error()
    for o in (4, 5, 7):
        for i in range(8):
            if i != o:
                for shift in (size[i] - 1, 0, 1 - size[o]):
                    a = at(8)
                    a[o] = a[i] + shift
                    assert call(a) == L.RRB_EINVAL and b"overlaps" in librrb.rrb_last_error(), (o, i, shift)
    a = at(8)
    a[0] = a[1]  # inputs may share
    assert call(a) == L.RRB_EINVAL and b"not bound" in librrb.rrb_last_error()
    librrb.rrb_plan_destroy(plan)
