"""Torch-facing calls of the MoE gate and the experts' products.

The steps of an MoE layer around dispatch and combine: ``moe_gate`` makes the
routing arrays from scores, the ``expert_*`` calls run on the dispatched rows,
grouped by expert (``MoeDevicePlan.expert_offsets``), and each has its
gradient.  Outputs are the caller's tensors, written in place; argument rules
are api.py's (contiguous, on the current GPU, bf16 as torch.bfloat16 or its
int16 / uint16 bit patterns), and shapes are checked too; the library refuses
outputs that overlap what a call reads.  None of the calls takes part in
autograd.
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


def _offsets(offsets, G):
    if offsets is None and G != 1:
        raise ValueError(f"offsets is required with {G} groups")
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
