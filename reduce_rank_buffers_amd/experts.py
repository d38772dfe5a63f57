"""Torch-facing calls of the MoE gate and the experts' products.

The steps of an MoE layer around dispatch and combine: ``moe_gate`` makes the
routing arrays from scores, the ``expert_*`` calls run on the dispatched rows,
grouped by expert (``MoeDevicePlan.expert_offsets``), and each has its
gradient.  For serving, ``quantize_rows`` and the ``expert_*_int8`` calls run
the products in 8-bit integers, and ``moe_decode`` the whole expert layer of a
few tokens without dispatch and combine; these have none.  Outputs are the
caller's tensors, written in place; argument rules are api.py's (contiguous, on
the current GPU, bf16 as torch.bfloat16 or its int16 / uint16 bit patterns),
and shapes are checked too; the library refuses outputs that overlap what a
call reads.  None of the calls takes part in autograd.
"""

import ctypes

import torch

from . import _lib as L
from .api import _BF16_TYPES, _F32_TYPES, _dtype_of, _on_gpu, _raw_stream

ACTIVATIONS = {"none": L.RRB_ACT_NONE, "silu": L.RRB_ACT_SILU, "gelu": L.RRB_ACT_GELU,
               "gelu_tanh": L.RRB_ACT_GELU_TANH, "relu": L.RRB_ACT_RELU}


def _shaped(t, what, shape, dtypes=_BF16_TYPES):
    """ValueError unless t is None or a contiguous tensor of that shape and
    one of these types; returns (what, t) for _addresses."""
    if t is None:
        return what, None
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise ValueError(f"{what}: dtype {t.dtype} is not {' or '.join(str(d)[6:] for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)} is not {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor is not contiguous")
    return what, t


def _addresses(named, optional=()):
    """Addresses of checked tensors, in order; those not in `optional` must be
    there and every one on the current GPU.  Also its index."""
    out, dev = [], None
    for what, t in named:
        if t is None:
            if what not in optional:
                raise ValueError(f"{what} is required")
            out.append(None)
            continue
        if t.get_device() != dev:
            _on_gpu(t, what)
            dev = t.get_device()
        out.append(t.data_ptr())
    return out, dev


# ---- the gate ----------------------------------------------------------------

def _gate_sizes(logits, topk_idx):
    for t, what in ((logits, "logits"), (topk_idx, "topk_idx")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{what}: expected a tensor of two dimensions")
    (T, E), k = logits.shape, topk_idx.shape[1]
    if not 1 <= k <= E:
        raise ValueError(f"topk_idx: {k} experts per token of {E}")
    return T, E, k


def moe_gate(logits, topk_idx, topk_w, renormalize=False, stream=None):
    """The topk experts of the largest scores (ties to the lower id; -inf
    masks) and their softmax weights: logits [T, E] bf16 or float32 ->
    topk_idx int32 [T, k], topk_w float32 [T, k], as MoeDevicePlan.route takes
    them.  renormalize: weights over the chosen experts alone."""
    T, E, k = _gate_sizes(logits, topk_idx)
    dt = _dtype_of(logits)
    named = [_shaped(logits, "logits", (T, E), (logits.dtype,)),
             _shaped(topk_idx, "topk_idx", (T, k), (torch.int32,)),
             _shaped(topk_w, "topk_w", (T, k), _F32_TYPES)]
    at, dev = _addresses(named)
    L.check(L.lib().rrb_moe_gate(T, E, k, dt, L.RRB_GATE_RENORMALIZE if renormalize else 0, *at, _raw_stream(stream, dev)),
            "rrb_moe_gate")
    return topk_idx, topk_w


def moe_gate_backward(logits, topk_idx, d_topk_w, d_logits, renormalize=False, stream=None):
    """The scores' gradient from the weights': d_topk_w float32 [T, k] ->
    d_logits [T, E] of the scores' type (may be logits itself), for moe_gate's
    logits and topk_idx."""
    T, E, k = _gate_sizes(logits, topk_idx)
    dt = _dtype_of(logits)
    named = [_shaped(logits, "logits", (T, E), (logits.dtype,)),
             _shaped(topk_idx, "topk_idx", (T, k), (torch.int32,)),
             _shaped(d_topk_w, "d_topk_w", (T, k), _F32_TYPES),
             _shaped(d_logits, "d_logits", (T, E), (logits.dtype,))]
    at, dev = _addresses(named)
    L.check(L.lib().rrb_moe_gate_backward(T, E, k, dt, L.RRB_GATE_RENORMALIZE if renormalize else 0, *at,
                                          _raw_stream(stream, dev)), "rrb_moe_gate_backward")
    return d_logits


# ---- the experts' products -----------------------------------------------------

def _spec(x, w, activation, what):
    """The sizes that rows x [N, in] and weights w [G, out, in] name."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    for t, name, dims in ((x, "x", 2), (w, what, 3)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name}: expected a tensor of {dims} dimensions")
    (N, i), (G, o, wi) = x.shape, w.shape
    if wi != i:
        raise ValueError(f"{what}: {wi} columns for rows of {i}")
    return L.ExpertSpec(N, i, o, G, ACTIVATIONS[activation]), N, i, o, G


def _offsets_for(offsets, G):
    if offsets is None and G != 1:
        raise ValueError(f"offsets is required with {G} groups")


def _offsets(offsets, G):
    _offsets_for(offsets, G)
    return _shaped(offsets, "offsets", (G + 1,), (torch.int32,))


def expert_gated(x, offsets, w_gate, w_up, out, activation="silu", save_gate=None, save_up=None, stream=None):
    """out = act(x Wg^T) * (x Wu^T) for rows x [N, in] grouped by offsets
    (int32 [G + 1]; None: one group), w_gate and w_up [G, inner, in], out
    [N, inner].  save_gate, save_up [N, inner] (both or neither) receive the
    projections that expert_gated_backward takes."""
    spec, N, i, o, G = _spec(x, w_gate, activation, "w_gate")
    if (save_gate is None) != (save_up is None):
        raise ValueError("save_gate and save_up go together")
    ins = [_shaped(x, "x", (N, i)), _offsets(offsets, G),
           _shaped(w_gate, "w_gate", (G, o, i)), _shaped(w_up, "w_up", (G, o, i))]
    outs = [_shaped(out, "out", (N, o)), _shaped(save_gate, "save_gate", (N, o)),
            _shaped(save_up, "save_up", (N, o))]
    at, dev = _addresses(ins + outs, ("offsets", "save_gate", "save_up"))
    L.check(L.lib().rrb_expert_gated(ctypes.byref(spec), *at, _raw_stream(stream, dev)), "rrb_expert_gated")
    return out


def expert_linear(x, offsets, w, out, bias=None, activation="none", residual=None, save_pre=None, stream=None):
    """out = act(x W^T + bias) + residual for rows x [N, in] grouped by
    offsets (int32 [G + 1]; None: one group), w [G, out, in], bias [G, out],
    residual [N, out] (may be out itself).  save_pre [N, out] receives the
    pre-activation values that expert_linear_backward takes."""
    spec, N, i, o, G = _spec(x, w, activation, "w")
    ins = [_shaped(x, "x", (N, i)), _offsets(offsets, G), _shaped(w, "w", (G, o, i)),
           _shaped(bias, "bias", (G, o)), _shaped(residual, "residual", (N, o))]
    outs = [_shaped(out, "out", (N, o)), _shaped(save_pre, "save_pre", (N, o))]
    at, dev = _addresses(ins + outs, ("offsets", "bias", "residual", "save_pre"))
    L.check(L.lib().rrb_expert_linear(ctypes.byref(spec), *at, _raw_stream(stream, dev)), "rrb_expert_linear")
    return out


def _workspace_bytes(name, rows, in_width, out_width, groups):
    n = ctypes.c_size_t()
    L.check(getattr(L.lib(), name)(ctypes.byref(L.ExpertSpec(rows, in_width, out_width, groups, 0)), ctypes.byref(n)),
            name)
    return n.value


def expert_gated_backward_workspace(rows, in_width, inner, groups):
    """Bytes of workspace that expert_gated_backward needs."""
    return _workspace_bytes("rrb_expert_gated_backward_workspace", rows, in_width, inner, groups)


def expert_linear_backward_workspace(rows, in_width, out_width, groups):
    """Bytes of workspace that expert_linear_backward needs."""
    return _workspace_bytes("rrb_expert_linear_backward_workspace", rows, in_width, out_width, groups)


def _workspace(workspace, need, like, stream):
    """The caller's workspace (uint8, 16-byte aligned, large enough), or one
    from torch's allocator that belongs to the stream the work runs on."""
    if workspace is None:
        with torch.cuda.stream(stream):
            return torch.empty(need, dtype=torch.uint8, device=like.device)
    if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8:
        raise ValueError("workspace: expected a tensor of torch.uint8")
    if not workspace.is_contiguous() or workspace.numel() < need or workspace.data_ptr() % 16:
        raise ValueError(f"workspace: expected a contiguous, 16-byte aligned tensor of at least {need} bytes")
    _on_gpu(workspace, "workspace")
    return workspace


def expert_gated_backward(d_out, x, offsets, w_gate, w_up, gate, up, activation="silu", d_x=None, d_w_gate=None,
                          d_w_up=None, workspace=None, stream=None):
    """Gradients of expert_gated: from d_out [N, inner], its inputs and the
    projections it saved to d_x [N, in] and (together) d_w_gate and d_w_up
    [G, inner, in]; those left None are not computed.  The weight gradients of
    a group without rows are 0.  workspace: uint8 tensor of
    expert_gated_backward_workspace bytes (allocated per call if None)."""
    spec, N, i, o, G = _spec(x, w_gate, activation, "w_gate")
    if (d_w_gate is None) != (d_w_up is None):
        raise ValueError("d_w_gate and d_w_up go together")
    if d_x is None and d_w_gate is None:
        raise ValueError("no gradient asked for: d_x and d_w_gate are None")
    ins = [_shaped(d_out, "d_out", (N, o)), _shaped(x, "x", (N, i)), _offsets(offsets, G),
           _shaped(w_gate, "w_gate", (G, o, i)), _shaped(w_up, "w_up", (G, o, i)),
           _shaped(gate, "gate", (N, o)), _shaped(up, "up", (N, o))]
    outs = [_shaped(d_x, "d_x", (N, i)), _shaped(d_w_gate, "d_w_gate", (G, o, i)),
            _shaped(d_w_up, "d_w_up", (G, o, i))]
    at, dev = _addresses(ins + outs, ("offsets", "d_x", "d_w_gate", "d_w_up"))
    need = expert_gated_backward_workspace(N, i, o, G)
    ws = _workspace(workspace, need, x, stream)
    L.check(L.lib().rrb_expert_gated_backward(ctypes.byref(spec), *at, ws.data_ptr(), need, _raw_stream(stream, dev)),
            "rrb_expert_gated_backward")
    return d_x, d_w_gate, d_w_up


def expert_linear_backward(d_out, x, offsets, w, pre=None, activation="none", d_x=None, d_w=None, d_bias=None,
                           workspace=None, stream=None):
    """Gradients of expert_linear: from d_out [N, out], its inputs and, with
    an activation, the saved pre [N, out] to d_x [N, in], d_w [G, out, in] and
    d_bias [G, out]; those left None are not computed.  The residual's
    gradient is d_out.  d_w and d_bias of a group without rows are 0.
    workspace: uint8 tensor of expert_linear_backward_workspace bytes
    (allocated per call if None)."""
    spec, N, i, o, G = _spec(x, w, activation, "w")
    if d_x is None and d_w is None and d_bias is None:
        raise ValueError("no gradient asked for: d_x, d_w and d_bias are None")
    if activation != "none" and pre is None:
        raise ValueError(f"pre is required with activation {activation!r}")
    ins = [_shaped(d_out, "d_out", (N, o)), _shaped(x, "x", (N, i)), _offsets(offsets, G),
           _shaped(w, "w", (G, o, i)), _shaped(pre, "pre", (N, o))]
    outs = [_shaped(d_x, "d_x", (N, i)), _shaped(d_w, "d_w", (G, o, i)),
            _shaped(d_bias, "d_bias", (G, o))]
    at, dev = _addresses(ins + outs, ("offsets", "pre", "d_x", "d_w", "d_bias"))
    need = expert_linear_backward_workspace(N, i, o, G)
    ws = _workspace(workspace, need, x, stream)
    L.check(L.lib().rrb_expert_linear_backward(ctypes.byref(spec), *at, ws.data_ptr(), need, _raw_stream(stream, dev)),
            "rrb_expert_linear_backward")
    return d_x, d_w, d_bias


# ---- serving -------------------------------------------------------------------

_INT8 = (torch.int8,)
_INT32 = (torch.int32,)


def _required(**tensors):
    for what, t in tensors.items():
        if t is None:
            raise ValueError(f"{what} is required")


def _checked(named):
    """Addresses of (what, tensor, shape, dtypes), None where there is none,
    and the GPU they are on; as _shaped and _addresses check them, in one pass
    over tensors that are as they should be (a decode step's calls are bound by
    the host)."""
    out, dev, mixed = [], None, False
    for what, t, shape, types in named:
        if t is None:
            out.append(None)
            continue
        if not isinstance(t, torch.Tensor) or t.dtype not in types or t.shape != shape or not t.is_contiguous():
            _shaped(t, what, shape, types)
        at = t.get_device()
        if at != dev:
            mixed = mixed or dev is not None
            dev = at
        out.append(t.data_ptr())
    if mixed or dev < 0 or dev != torch.cuda.current_device():
        for what, t, _, _ in named:
            if t is not None:
                _on_gpu(t, what)
    return out, dev


def quantize_rows(x, q, scale, offsets=None, stream=None):
    """Rows as 8-bit integers: x [..., n] bf16 or float32 -> q int8 of its
    shape and scale float32 of x.shape[:-1], scale = max |x| / 127 of a row
    (float32) and q = x / scale to the nearest integer, ties to even.  A row
    of zeros has scale 0, a row with an infinity or a NaN scale NaN and zeros.
    offsets (int32 [G + 1], x of two dimensions): only rows offsets[0] ..
    offsets[-1] - 1 are read and written."""
    if not isinstance(x, torch.Tensor) or x.dim() < 2:
        raise ValueError("x: expected a tensor of at least two dimensions")
    dt, n = _dtype_of(x), x.shape[-1]
    groups = 0
    if offsets is not None:
        if x.dim() != 2 or not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError("offsets: expected a tensor of one dimension and at least two entries, "
                             "x of two dimensions")
        groups = offsets.numel() - 1
    _required(q=q, scale=scale)
    (xp, qp, sp, op), dev = _checked((("x", x, x.shape, (x.dtype,)), ("q", q, x.shape, _INT8),
                                      ("scale", scale, x.shape[:-1], _F32_TYPES),
                                      ("offsets", offsets, (groups + 1,), _INT32)))
    L.check(L.lib().rrb_quantize_rows(scale.numel(), n, dt, xp, op, groups, qp, sp, _raw_stream(stream, dev)),
            "rrb_quantize_rows")
    return q, scale


def expert_linear_int8(x, x_scale, offsets, w, w_scale, out, bias=None, activation="none", residual=None, stream=None):
    """expert_linear of rows and weights as quantize_rows makes them: x int8
    [N, in], x_scale float32 [N], w int8 [G, out, in], w_scale float32
    [G, out]; out, bias [G, out] and residual [N, out] (may be out itself)
    bf16."""
    spec, N, i, o, G = _spec(x, w, activation, "w")
    _offsets_for(offsets, G)
    _required(x_scale=x_scale, w_scale=w_scale, out=out)
    at, dev = _checked((("x", x, (N, i), _INT8), ("x_scale", x_scale, (N,), _F32_TYPES),
                        ("offsets", offsets, (G + 1,), _INT32), ("w", w, (G, o, i), _INT8),
                        ("w_scale", w_scale, (G, o), _F32_TYPES), ("bias", bias, (G, o), _BF16_TYPES),
                        ("residual", residual, (N, o), _BF16_TYPES), ("out", out, (N, o), _BF16_TYPES)))
    L.check(L.lib().rrb_expert_linear_int8(ctypes.byref(spec), *at, _raw_stream(stream, dev)),
            "rrb_expert_linear_int8")
    return out


def expert_gated_int8(x, x_scale, offsets, w_gate, gate_scale, w_up, up_scale, out, activation="silu", stream=None):
    """expert_gated of rows and weights as quantize_rows makes them: x int8
    [N, in], x_scale float32 [N], w_gate and w_up int8 [G, inner, in] with
    scales float32 [G, inner]; out [N, inner] bf16."""
    spec, N, i, o, G = _spec(x, w_gate, activation, "w_gate")
    _offsets_for(offsets, G)
    _required(x_scale=x_scale, gate_scale=gate_scale, w_up=w_up, up_scale=up_scale, out=out)
    at, dev = _checked((("x", x, (N, i), _INT8), ("x_scale", x_scale, (N,), _F32_TYPES),
                        ("offsets", offsets, (G + 1,), _INT32), ("w_gate", w_gate, (G, o, i), _INT8),
                        ("gate_scale", gate_scale, (G, o), _F32_TYPES), ("w_up", w_up, (G, o, i), _INT8),
                        ("up_scale", up_scale, (G, o), _F32_TYPES), ("out", out, (N, o), _BF16_TYPES)))
    L.check(L.lib().rrb_expert_gated_int8(ctypes.byref(spec), *at, _raw_stream(stream, dev)), "rrb_expert_gated_int8")
    return out


def _decode_workspace(spec):
    n = ctypes.c_size_t()
    L.check(L.lib().rrb_moe_decode_workspace(ctypes.byref(spec), ctypes.byref(n)), "rrb_moe_decode_workspace")
    return n.value


def moe_decode_workspace(tokens, topk, hidden, inner):
    """Bytes of workspace that moe_decode needs."""
    return _decode_workspace(L.DecodeSpec(tokens, hidden, inner, 1, topk, 0, 0))


def moe_decode(x, topk_idx, topk_w, w_gate, w_up, w_down, out, activation="silu", scales=None, workspace=None,
               stream=None):
    """The expert layer of up to 64 tokens in two kernels, without dispatch and
    combine: out[t] = sum over j of topk_w[t, j] Wd[e] (act(Wg[e] x[t]) *
    (Wu[e] x[t])), e = topk_idx[t, j], for x and out [T, h], topk_idx int32
    and topk_w float32 [T, k] (as moe_gate writes them), w_gate and w_up
    [E, f, h], w_down [E, h, f].  Choices outside 0 .. E - 1 take no part.
    scales: (gate, up, down) float32 [E, f], [E, f], [E, h] of weights held in
    int8 (quantize_rows).  workspace: uint8 tensor of moe_decode_workspace
    bytes (allocated per call if None)."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}")
    for t, name, dims in ((x, "x", 2), (topk_idx, "topk_idx", 2), (w_gate, "w_gate", 3)):
        if not isinstance(t, torch.Tensor) or t.dim() != dims:
            raise ValueError(f"{name}: expected a tensor of {dims} dimensions")
    (T, h), (E, f, wh), k = x.shape, w_gate.shape, topk_idx.shape[1]
    if wh != h:
        raise ValueError(f"w_gate: {wh} columns for rows of {h}")
    types = _BF16_TYPES
    sg = su = sd = None
    if scales is not None:
        if not isinstance(scales, (tuple, list)) or len(scales) != 3 or any(s is None for s in scales):
            raise ValueError("scales: expected those of w_gate, w_up and w_down")
        (sg, su, sd), types = scales, _INT8
    _required(topk_w=topk_w, w_up=w_up, w_down=w_down, out=out)
    at, dev = _checked((("x", x, (T, h), _BF16_TYPES), ("topk_idx", topk_idx, (T, k), _INT32),
                        ("topk_w", topk_w, (T, k), _F32_TYPES), ("w_gate", w_gate, (E, f, h), types),
                        ("w_up", w_up, (E, f, h), types), ("w_down", w_down, (E, h, f), types),
                        ("scales[0]", sg, (E, f), _F32_TYPES), ("scales[1]", su, (E, f), _F32_TYPES),
                        ("scales[2]", sd, (E, h), _F32_TYPES), ("out", out, (T, h), _BF16_TYPES)))
    spec = L.DecodeSpec(T, h, f, E, k, ACTIVATIONS[activation], 0)
    if workspace is None:
        workspace = _workspace(None, _decode_workspace(spec), x, stream)
    elif not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor of torch.uint8")
    elif workspace.get_device() != dev:
        _on_gpu(workspace, "workspace")
    ws, size = workspace.data_ptr(), workspace.numel()  # (too small or misaligned: refused by the library)
    L.check(L.lib().rrb_moe_decode(ctypes.byref(spec), *at, ws, size, _raw_stream(stream, dev)), "rrb_moe_decode")
    return out
