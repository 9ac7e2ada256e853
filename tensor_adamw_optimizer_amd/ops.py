"""Operators of a model around the optimizer step, on CUDA (ROCm) tensors.

``gated_ffn``, ``linear_cross_entropy`` and ``qk_norm_rope`` are
differentiable functions; each stands on a ``*_forward`` and a ``*_backward``
that take and return plain tensors, for programs that run their backward
pass themselves (under graph capture, or with gradients written where the
optimizer reads them).  All of it runs in the HIP library on torch's current
stream; torch allocates outputs and workspaces.  Tensors are float32 or
bfloat16, all matrices of a call of one type and on one device.
"""
from __future__ import annotations

import math
from typing import Optional, Tuple

import torch

from . import _lib as L

_DT = {torch.float32: L.APEXW_F32, torch.bfloat16: L.APEXW_BF16}
_LOSS = {"mean": L.APEXW_LOSS_MEAN, "sum": L.APEXW_LOSS_SUM, "none": L.APEXW_LOSS_NONE}
_ACT = {"silu": L.APEXW_ACT_SILU, "gelu_tanh": L.APEXW_ACT_GELU_TANH}

_MAX_STRIDE = 1 << 20

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _queue(call, device: torch.device, *args) -> None:
    """The library's call on torch's current stream of the tensors' device, that
    device made current: a raw stream, and the default one, 0, above all, is one of
    the thread's current device."""
    if _current_device() == device.index:
        call(*args, _stream(device))
    else:
        with torch.cuda.device(device):
            call(*args, _stream(device))


def _sig(t: torch.Tensor):
    return t.shape, t.stride(), t.dtype, t.device


_plans: dict = {}


def _plan(make, *key):
    """What `make` works out of a call's shapes, strides, types and options, and
    its checks of them: once for each such call.  Nothing of the tensors'
    contents or places is in it."""
    p = _plans.get((make, key))
    if p is None:
        if len(_plans) >= 1024:
            _plans.clear()
        p = _plans[make, key] = make(*key)
    return p


def _dtype(where: str, first, *others) -> int:
    """The C code of the element type; `first` and the others (name, signature)
    have to agree."""
    dtype, device = first[2:]
    if dtype not in _DT:
        raise TypeError("%s takes float32 or bfloat16 tensors, not %s" % (where, dtype))
    if device.type != "cuda":
        raise ValueError("%s needs CUDA tensors" % where)
    for name, (_, _, dt, dev) in others:
        if dt != dtype:
            raise TypeError("%s: %s is %s, the first operand %s" % (where, name, dt, dtype))
        if dev != device:
            raise ValueError("%s: %s is on %s, the first operand on %s" % (where, name, dev, device))
    return _DT[dtype]


def _index(where: str, name: str, sig, device) -> None:
    if sig[2] != torch.int64:
        raise TypeError("%s: %s is %s, not int64" % (where, name, sig[2]))
    if sig[3] != device:
        raise ValueError("%s: %s is on %s, the first operand on %s" % (where, name, sig[3], device))


def _row_stride(sig, aligned: bool) -> int:
    """Elements from one row to the next where the tensor can be read as rows of
    adjacent values from an aligned start; 0 where it has to be copied."""
    shape, stride = sig[:2]
    cols = shape[-1]
    if not aligned or (cols > 1 and stride[-1] != 1):
        return 0
    if len(shape) == 2:
        return cols if shape[0] < 2 else stride[0] if cols <= stride[0] <= _MAX_STRIDE else 0
    want = cols
    for n, st in zip(reversed(shape[:-1]), reversed(stride[:-1])):
        if n > 1 and st != want:
            return 0
        want *= n
    return cols


def _aligned(t: torch.Tensor) -> bool:
    return t.data_ptr() % 16 == 0


def _copy(t: torch.Tensor) -> torch.Tensor:
    return t.clone(memory_format=torch.contiguous_format)


def _whole(t: torch.Tensor) -> torch.Tensor:
    """Contiguous and 16-byte aligned (a copy where it is not already)."""
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else _copy(t)


# (empty_like of something at hand takes a third of the time of empty)
def _empty(like: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(like, memory_format=torch.contiguous_format)


_elements: dict = {}


def _like(dtype, device, *shape) -> torch.Tensor:
    """What _empty makes tensors of that shape from: one element, expanded, the same
    one for all plans (one of a plan's own, made under graph capture, would hold on
    to the graph's memory)."""
    e = _elements.get((dtype, device))
    if e is None:
        e = _elements[dtype, device] = torch.empty((), dtype=dtype, device=device)
    return e.expand(shape)


# ------------------------------------------------------ gated feed-forward

def _ffn_plan(x, w_gate, w_up, w_down, dy, activation, kept, x_aligned, dy_aligned):
    where = "gated_ffn"
    if activation not in _ACT:
        raise ValueError("%s: unknown activation %r (one of %s)"
                         % (where, activation, ", ".join(sorted(_ACT))))
    d_ff, d_model = w_gate[0] if len(w_gate[0]) == 2 else (0, 0)
    if x[0][-1:] != (d_model,) or tuple(w_up[0]) != (d_ff, d_model) or \
            tuple(w_down[0]) != (d_model, d_ff):
        raise ValueError("%s: x [..., D], w_gate and w_up [F, D], w_down [D, F] expected, got %s"
                         % (where, [tuple(t[0]) for t in (x, w_gate, w_up, w_down)]))
    dt = _dtype(where, x, ("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down),
                *((("dy", dy),) if dy is not None else ()))
    x_stride = _row_stride(x, x_aligned)
    dy_stride = 0 if dy is None else _row_stride(dy, dy_aligned)
    s = L.apexw_gated_ffn_shape(math.prod(x[0][:-1]), d_model, d_ff, x_stride, dy_stride, dt,
                                _ACT[activation])
    kept_len = L.apexw_gated_ffn_kept_bytes(s) if kept else 0
    n = L.apexw_gated_ffn_workspace_bytes(s, dy is not None, kept)
    dev = x[3]
    return (s, x_stride != 0, dy_stride != 0, kept_len, _like(torch.uint8, dev, kept_len), n,
            _like(torch.uint8, dev, n))


def gated_ffn_forward(x, w_gate, w_up, w_down, activation: str = "silu", keep: bool = False):
    """``(act(x w_gate^T) * (x w_up^T)) w_down^T`` and, with ``keep``, the
    buffer that spares :func:`gated_ffn_backward` the recomputation (else
    None)."""
    s, direct, _, kept_len, kept_like, n, ws_like = _plan(
        _ffn_plan, _sig(x), _sig(w_gate), _sig(w_up), _sig(w_down), None, activation, keep,
        _aligned(x), True)
    w_gate, w_up, w_down = _whole(w_gate), _whole(w_up), _whole(w_down)
    xr = x if direct else _copy(x)
    y = _empty(x)
    kept = _empty(kept_like) if keep else None
    ws = _empty(ws_like)
    _queue(L.apexw_gated_ffn_forward, x.device, s, xr.data_ptr(), w_gate.data_ptr(),
           w_up.data_ptr(), w_down.data_ptr(), y.data_ptr(), kept.data_ptr() if keep else 0,
           kept_len, ws.data_ptr(), n)
    return y, kept


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, kept: Optional[torch.Tensor] = None,
                       activation: str = "silu", needs=(True, True, True, True)):
    """The gradients of x, w_gate, w_up and w_down (None where ``needs`` is
    false) for the gradient ``dy`` of the output."""
    if dy.shape != x.shape:
        raise ValueError("gated_ffn: dy is %s, x %s" % (tuple(dy.shape), tuple(x.shape)))
    s, direct, dy_direct, kept_len, _, n, ws_like = _plan(
        _ffn_plan, _sig(x), _sig(w_gate), _sig(w_up), _sig(w_down), _sig(dy), activation,
        kept is not None, _aligned(x), _aligned(dy))
    if kept is not None and (kept.dtype != torch.uint8 or kept.device != x.device or
                             kept.shape != (kept_len,) or not kept.is_contiguous()):
        raise ValueError("gated_ffn: kept must be the buffer of the forward pass over the same "
                         "inputs, %d contiguous bytes (uint8) on %s" % (kept_len, x.device))
    w_gate, w_up, w_down = _whole(w_gate), _whole(w_up), _whole(w_down)
    xr, dyr = x if direct else _copy(x), dy if dy_direct else _copy(dy)
    outs = [_empty(t) if need else None for t, need in zip((x, w_gate, w_up, w_down), needs)]
    ws = _empty(ws_like)
    _queue(L.apexw_gated_ffn_backward, x.device, s, dyr.data_ptr(), xr.data_ptr(),
           w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(),
           0 if kept is None else kept.data_ptr(), kept_len,
           *(0 if o is None else o.data_ptr() for o in outs), ws.data_ptr(), n)
    return tuple(outs)


class _GatedFFN(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation):
        y, kept = gated_ffn_forward(x, w_gate, w_up, w_down, activation, True)
        ctx.save_for_backward(x, w_gate, w_up, w_down, kept)
        ctx.activation = activation
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        *args, kept = ctx.saved_tensors
        return (*gated_ffn_backward(dy, *args, kept=kept, activation=ctx.activation,
                                    needs=ctx.needs_input_grad[:4]), None)


def gated_ffn(x, w_gate, w_up, w_down, activation: str = "silu") -> torch.Tensor:
    """``(act(x w_gate^T) * (x w_up^T)) w_down^T``, differentiable in all four.

    x [..., D], w_gate and w_up [F, D], w_down [D, F]; ``activation`` is
    "silu" or "gelu_tanh".
    """
    # (a function's forward sees only what requires a gradient, not whether one can
    # be asked for: without this, evaluation would fill a kept buffer too)
    if not torch.is_grad_enabled() or \
            not any(t.requires_grad for t in (x, w_gate, w_up, w_down)):
        return gated_ffn_forward(x, w_gate, w_up, w_down, activation)[0]
    return _GatedFFN.apply(x, w_gate, w_up, w_down, activation)


# --------------------------------------------------- linear cross entropy

def _xent_plan(x, weight, target, reduction, ignore_index, backward, aligned):
    where = "linear_cross_entropy"
    if reduction not in _LOSS:
        raise ValueError("%s: unknown reduction %r (one of %s)"
                         % (where, reduction, ", ".join(sorted(_LOSS))))
    if len(weight[0]) != 2 or x[0][-1:] != weight[0][1:] or target[0] != x[0][:-1]:
        raise ValueError("%s: x [..., D], weight [V, D], target [...] expected, got %s"
                         % (where, [tuple(t[0]) for t in (x, weight, target)]))
    dt = _dtype(where, x, ("weight", weight))
    _index(where, "target", target, x[3])
    stride = _row_stride(x, aligned)
    s = L.apexw_linear_xent_shape(math.prod(x[0][:-1]), weight[0][1], weight[0][0], stride,
                                  ignore_index, dt, _LOSS[reduction])
    n = L.apexw_linear_xent_workspace_bytes(s, backward)
    return (s, stride != 0, n, _like(torch.uint8, x[3], n), _like(torch.float32, x[3]),
            _like(torch.float32, x[3], *target[0]))


def linear_cross_entropy_forward(x, weight, target, reduction: str = "mean",
                                 ignore_index: int = -100):
    """The loss (of ``reduction``; None with "none"), each token's loss, and
    each token's log-sum-exp, which :func:`linear_cross_entropy_backward`
    takes; all float32."""
    s, direct, n, ws_like, loss_like, token_like = _plan(
        _xent_plan, _sig(x), _sig(weight), _sig(target), reduction, ignore_index, False,
        _aligned(x))
    xr, w, tg = x if direct else _copy(x), _whole(weight), target.contiguous()
    loss = None if reduction == "none" else _empty(loss_like)
    token, lse, ws = _empty(token_like), _empty(token_like), _empty(ws_like)
    _queue(L.apexw_linear_xent_forward, x.device, s, xr.data_ptr(), w.data_ptr(), tg.data_ptr(),
           0 if loss is None else loss.data_ptr(), token.data_ptr(), lse.data_ptr(),
           ws.data_ptr(), n)
    return loss, token, lse


def linear_cross_entropy_backward(x, weight, target, lse, dloss, reduction: str = "mean",
                                  ignore_index: int = -100, needs=(True, True)):
    """The gradients of x and weight (None where ``needs`` is false) for the
    gradient ``dloss`` of the loss: float32, a scalar, or one value for each
    token with "none"."""
    s, direct, n, ws_like, _, _ = _plan(
        _xent_plan, _sig(x), _sig(weight), _sig(target), reduction, ignore_index, True,
        _aligned(x))
    dev = x.device
    for name, t, shape in (("lse", lse, target.shape),
                           ("dloss", dloss, target.shape if reduction == "none" else ())):
        if t.dtype != torch.float32 or t.device != dev or t.shape != shape:
            raise ValueError("linear_cross_entropy: %s must be float32 %s on %s"
                             % (name, tuple(shape), dev))
    xr, w, tg = x if direct else _copy(x), _whole(weight), target.contiguous()
    lse, dloss = lse.contiguous(), dloss.contiguous()
    outs = [_empty(t) if need else None for t, need in zip((x, weight), needs)]
    ws = _empty(ws_like)
    _queue(L.apexw_linear_xent_backward, dev, s, dloss.data_ptr(), xr.data_ptr(), w.data_ptr(),
           tg.data_ptr(), lse.data_ptr(), *(0 if o is None else o.data_ptr() for o in outs),
           ws.data_ptr(), n)
    return tuple(outs)


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, target, reduction, ignore_index):
        loss, token, lse = linear_cross_entropy_forward(x, weight, target, reduction, ignore_index)
        if any(ctx.needs_input_grad):
            ctx.save_for_backward(x, weight, target, lse)
        ctx.how = reduction, ignore_index
        return token if loss is None else loss

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss):
        return (*linear_cross_entropy_backward(*ctx.saved_tensors, dloss, *ctx.how,
                                               needs=ctx.needs_input_grad[:2]), None, None, None)


def linear_cross_entropy(x, weight, target, reduction: str = "mean",
                         ignore_index: int = -100) -> torch.Tensor:
    """The softmax cross entropy of the logits ``x weight^T``, differentiable
    in x and weight, without the logits in memory.

    x [..., D], weight [V, D], target int64 [...]; ``reduction`` is "mean"
    (over the tokens whose target is not ``ignore_index``; 0 if there are
    none), "sum" or "none".  The loss is float32.
    """
    return _LinearCrossEntropy.apply(x, weight, target, reduction, ignore_index)


# ------------------------------- norm of queries and keys with the rotation

def _head_strides(sig):
    """Elements from one token and from one head to the next where all tokens
    are one stride apart; None where the tensor has to be copied."""
    shape, stride = sig[:2]
    heads, hd = shape[-2:]
    if hd > 1 and stride[-1] != 1:
        return None
    head = stride[-2] if heads > 1 else hd
    token = want = None
    for n, st in zip(reversed(shape[:-2]), reversed(stride[:-2])):
        if n > 1:
            if token is None:
                token = want = st
            elif st != want:
                return None
        if want is not None:
            want *= n
    if head <= 0 or (token is not None and token <= 0):
        return None
    return heads * hd if token is None else token, head


def _qk_plan(q, k, q_weight, k_weight, positions, dq, dk, theta, rotary_dim, interleaved, eps):
    where = "qk_norm_rope"
    if len(q[0]) < 3 or q[0][:-2] != k[0][:-2] or q[0][-1] != k[0][-1] or \
            positions[0] != q[0][:-2] or any(tuple(w[0]) != (q[0][-1],) for w in (q_weight, k_weight)):
        raise ValueError("%s: q [..., Hq, D], k [..., Hk, D], weights [D], positions [...] "
                         "expected, got %s" % (where, [tuple(t[0]) for t in (
                             q, k, q_weight, k_weight, positions)]))
    dt = _dtype(where, q, ("k", k), ("q_weight", q_weight), ("k_weight", k_weight),
                *((("dq", dq), ("dk", dk)) if dq is not None else ()))
    _index(where, "positions", positions, q[3])
    hd = q[0][-1]
    strides = [(0, 0) if t is None else _head_strides(t) for t in (q, k, dq, dk)]
    s = L.apexw_qk_norm_rope_shape(math.prod(q[0][:-2]), *(st or (0, 0) for st in strides), theta,
                                   eps, q[0][-2], k[0][-2], hd,
                                   hd if rotary_dim is None else rotary_dim, int(interleaved), dt)
    n = L.apexw_qk_norm_rope_workspace_bytes(s)
    return (s, *(st is not None for st in strides), n, _like(torch.uint8, q[3], n))


def qk_norm_rope_forward(q, k, q_weight, k_weight, positions, theta: float = 10000.0,
                         rotary_dim: Optional[int] = None, interleaved: bool = False,
                         eps: float = 1e-6):
    """Queries and keys, each head normed, weighted and turned by its token's
    position; contiguous."""
    s, q_direct, k_direct, _, _, _, _ = _plan(
        _qk_plan, _sig(q), _sig(k), _sig(q_weight), _sig(k_weight), _sig(positions), None, None,
        theta, rotary_dim, interleaved, eps)
    qr, kr = q if q_direct else _copy(q), k if k_direct else _copy(k)
    qw, kw, pos = q_weight.contiguous(), k_weight.contiguous(), positions.contiguous()
    q_out, k_out = _empty(q), _empty(k)
    _queue(L.apexw_qk_norm_rope_forward, q.device, s, qr.data_ptr(), kr.data_ptr(),
           qw.data_ptr(), kw.data_ptr(), pos.data_ptr(), q_out.data_ptr(), k_out.data_ptr())
    return q_out, k_out


def qk_norm_rope_backward(dq, dk, q, k, q_weight, k_weight, positions, theta: float = 10000.0,
                          rotary_dim: Optional[int] = None, interleaved: bool = False,
                          eps: float = 1e-6, needs=(True, True, True, True)):
    """The gradients of q, k, q_weight and k_weight (None where ``needs`` is
    false) for the gradients ``dq`` and ``dk`` of the two outputs."""
    if dq.shape != q.shape or dk.shape != k.shape:
        raise ValueError("qk_norm_rope: dq is %s, q %s, dk %s, k %s"
                         % tuple(tuple(t.shape) for t in (dq, q, dk, k)))
    s, *direct, n, ws_like = _plan(
        _qk_plan, _sig(q), _sig(k), _sig(q_weight), _sig(k_weight), _sig(positions), _sig(dq),
        _sig(dk), theta, rotary_dim, interleaved, eps)
    qr, kr, dqr, dkr = (t if d else _copy(t) for t, d in zip((q, k, dq, dk), direct))
    qw, kw, pos = q_weight.contiguous(), k_weight.contiguous(), positions.contiguous()
    outs = [_empty(t) if need else None for t, need in zip((q, k, q_weight, k_weight), needs)]
    ws = _empty(ws_like)
    _queue(L.apexw_qk_norm_rope_backward, q.device, s, dqr.data_ptr(), dkr.data_ptr(),
           qr.data_ptr(), kr.data_ptr(), qw.data_ptr(), kw.data_ptr(), pos.data_ptr(),
           *(0 if o is None else o.data_ptr() for o in outs), ws.data_ptr(), n)
    return tuple(outs)


class _QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, *how):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions)
        ctx.how = how
        return qk_norm_rope_forward(q, k, q_weight, k_weight, positions, *how)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk):
        return (*qk_norm_rope_backward(dq, dk, *ctx.saved_tensors, *ctx.how,
                                       needs=ctx.needs_input_grad[:4]), *[None] * 5)


def qk_norm_rope(q, k, q_weight, k_weight, positions, theta: float = 10000.0,
                 rotary_dim: Optional[int] = None, interleaved: bool = False, eps: float = 1e-6):
    """The root-mean-square norm of each head of q and k, times its weight,
    with the rotation of the head's first ``rotary_dim`` values (None: all) by
    its token's position; differentiable in q, k and both weights.

    q [..., Hq, D], k [..., Hk, D] (views into a fused projection's output are
    read as they are), weights [D], positions int64 [...].  Pairs that turn
    together are values i and i + rotary_dim / 2 or, with ``interleaved``, 2 i
    and 2 i + 1; pair i turns by position * theta^(-2 i / rotary_dim).
    """
    return _QKNormRope.apply(q, k, q_weight, k_weight, positions, theta, rotary_dim, interleaved,
                             eps)
