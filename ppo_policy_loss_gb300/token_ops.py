"""Token log-probabilities and distillation over torch CUDA tensors: the
log-probabilities of given tokens with entropy and top alternatives, their
gradient, the loss and gradient of distillation from a teacher's top
log-probabilities, and the autograd wrappers around them (include/rltoken.h;
the rollout buffer of the ainews.cool RL.cu article, section "技术深度解析",
holds such log-probabilities).

Outputs are allocated with torch, everything is computed by librlloss's
kernels.  Inputs are checked and never copied: a tensor of another type,
layout or device is refused with a ValueError.  Calls run on the logits'
device, on ``stream`` (a torch.cuda.Stream) or torch's current stream there;
their outputs belong to that stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import (DISTILL_STATS_BYTES, DISTILL_TAILS, DTYPES, _check, distill_stats_from_bytes, load,
               rl_topk_distill_desc, rl_topk_distill_workspace_size)

_DT = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"], torch.float16: DTYPES["f16"]}
_F32, _I64 = torch.float32, torch.int64
_HERE = contextlib.nullcontext()


def _on(device: torch.device, stream, inputs):
    """The context in which a call allocates and launches: the logits' device
    and, if one is given, the caller's stream.  Memory of the inputs is not
    reused before that stream has read them."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the logits are on {device}")
        if stream != torch.cuda.current_stream(device):
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)
        return torch.cuda.stream(stream)
    if device.index != torch._C._cuda_getDevice():
        return torch.cuda.device(device)
    return _HERE


def _raw_stream(device: torch.device) -> int:
    # a decode step's call is host-bound: the raw handle, without a Stream object
    return torch._C._cuda_getCurrentRawStream(device.index)


def _written(*tensors):
    """Count a kernel's writes into the caller's tensors as changes in place, so
    that autograd refuses to use what it has kept of them."""
    for t in tensors:
        if isinstance(t, torch.Tensor) and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _p(t):
    return None if t is None else t.data_ptr()


def _logits(logits: torch.Tensor):
    """(dtype code, rows, columns, row stride) of a [R, V] matrix of logits."""
    dt = _DT.get(logits.dtype)
    if dt is None or logits.dim() != 2 or not logits.is_cuda:
        raise ValueError("logits must be a 2-D float32, bfloat16 or float16 CUDA tensor")
    R, V = logits.shape
    ld = logits.stride(0) if R > 1 else max(V, logits.stride(0))
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("logits must have unit column stride")
    return dt, R, V, ld


def _given(name: str, t: torch.Tensor, dtype, shape, device):
    """Check a dense input tensor: its type, shape and place."""
    if t.dtype != dtype or t.device != device or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    return t


def _mask(mask, R, device):
    if mask is None:
        return None
    if mask.dtype == torch.bool:
        mask = mask.view(torch.uint8)
    return _given("mask", mask.view(-1) if mask.is_contiguous() else mask, torch.uint8, (R,), device)


def _status(status, device):
    if status is not None and (status.dtype not in (torch.int32, torch.uint32) or status.device != device or
                               status.numel() != 1):
        raise ValueError(f"status must be an int32 tensor of one element on {device}")
    return _p(status)


def _n_ids(ids, R):
    if ids is None:
        return 0
    if ids.dim() not in (1, 2):
        raise ValueError("ids must be of shape [R] or [R, n]")
    return 1 if ids.dim() == 1 else ids.shape[1]


def token_logprobs(logits: torch.Tensor, ids: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                   k: int = 0, temperature: float = 1.0, want_entropy: bool = True, want_lse: bool = False,
                   status: torch.Tensor | None = None, stream=None) -> dict:
    """Log-probabilities of given tokens, entropy and the k most likely tokens
    of each row of ``logits`` [R, V] at a sampling temperature.

    ``ids``: int64 [R] or [R, n] (None: no given tokens); ``mask``: uint8 or
    bool [R], masked rows give 0 (and alternatives of id -1); ``status``: int32
    [1], collects RL_DEVERR_* bits.  Returns dict(logp: like ids, entropy and
    lse: [R], topk_ids: int64 [R, k], topk_logp: [R, k]); None for what was not
    asked for."""
    dt, R, V, ld = _logits(logits)
    dev = logits.device
    n = _n_ids(ids, R)
    if ids is not None:
        _given("ids", ids, torch.int64, (R,) if ids.dim() == 1 else (R, n), dev)
    mask = _mask(mask, R, dev)
    status_p = _status(status, dev)
    with _on(dev, stream, (logits, ids, mask, status)):
        logp = torch.empty(ids.shape, dtype=_F32, device=dev) if ids is not None else None
        ent = torch.empty(R, dtype=_F32, device=dev) if want_entropy else None
        lse = torch.empty(R, dtype=_F32, device=dev) if want_lse else None
        top = torch.empty((R, k), dtype=_I64, device=dev) if k > 0 else None
        top_lp = torch.empty((R, k), dtype=_F32, device=dev) if k > 0 else None
        _check(load().rl_token_logprobs(
            logits.data_ptr(), dt, R, V, ld, _p(ids) if n else None, n, _p(mask), temperature, k,
            _p(logp) if n else None, _p(ent), _p(lse), _p(top), _p(top_lp), status_p, _raw_stream(dev)),
            "rl_token_logprobs")
    return dict(logp=logp, entropy=ent, lse=lse, topk_ids=top, topk_logp=top_lp)


def token_logprobs_backward(logits: torch.Tensor, ids: torch.Tensor | None, dlogp: torch.Tensor | None,
                            lse: torch.Tensor, entropy: torch.Tensor | None = None,
                            dentropy: torch.Tensor | None = None, mask: torch.Tensor | None = None,
                            temperature: float = 1.0, dlogits="new", status: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Gradient with respect to ``logits`` of the log-probabilities (``dlogp``,
    like ``ids``) and, with ``entropy`` and ``dentropy`` [R], the entropies that
    token_logprobs gave; ``lse`` [R] is its log-sum-exp.  ``dlogits``: "new"
    allocates it with the logits' row stride, a tensor of that stride is written
    in place (``dlogits=logits`` overwrites the logits).  ids of shape [R, 0]
    without ``dentropy`` give a gradient of zeros."""
    dt, R, V, ld = _logits(logits)
    dev = logits.device
    n = _n_ids(ids, R)
    if ids is not None:
        shape = (R,) if ids.dim() == 1 else (R, n)
        _given("ids", ids, torch.int64, shape, dev)
        if dlogp is None:
            raise ValueError("dlogp must be given with ids")
        _given("dlogp", dlogp, torch.float32, shape, dev)
    elif dlogp is not None:
        raise ValueError("ids must be given with dlogp")
    _given("lse", lse, torch.float32, (R,), dev)
    for name, t in (("entropy", entropy), ("dentropy", dentropy)):
        if t is not None:
            _given(name, t, torch.float32, (R,), dev)
    mask = _mask(mask, R, dev)
    status_p = _status(status, dev)
    given = None if isinstance(dlogits, str) else dlogits
    with _on(dev, stream, (logits, ids, dlogp, lse, entropy, dentropy, mask, status, given)):
        dlogits = _dlogits_like(logits, dlogits, ld)
        if ids is not None and n == 0 and entropy is None and dentropy is None:
            return dlogits.zero_()
        _check(load().rl_token_logprobs_bwd(
            logits.data_ptr(), dt, R, V, ld, _p(ids) if n else None, n, _p(mask), temperature, _p(lse), _p(entropy),
            _p(dlogp) if n else None, _p(dentropy), _p(dlogits), status_p, _raw_stream(dev)),
            "rl_token_logprobs_bwd")
        _written(given)
    return dlogits


def _dlogits_like(logits: torch.Tensor, dlogits, ld: int) -> torch.Tensor:
    """The gradient's tensor: new with the logits' row stride, or the caller's."""
    R, V = logits.shape
    if isinstance(dlogits, str):
        if ld == V:
            return torch.empty((R, V), dtype=logits.dtype, device=logits.device)
        return torch.empty((R, ld), dtype=logits.dtype, device=logits.device)[:, :V]
    if (dlogits.dtype != logits.dtype or dlogits.device != logits.device or dlogits.shape != logits.shape or
            (R > 1 and dlogits.stride(0) != ld) or (V > 1 and dlogits.stride(1) != 1)):
        raise ValueError("dlogits must be like the logits, with the same row stride")
    return dlogits


class TokenLogprobs(torch.autograd.Function):
    """Autograd wrapper: logp, entropy = TokenLogprobs.apply(logits, ids, mask, temperature).

    The backward pass is one launch of rl_token_logprobs_bwd on the incoming
    gradients; it reads no value on the host, so it can be captured.  Capture it
    with torch.autograd.grad, or while no eager graph of the same leaves is
    alive: torch's accumulation into a leaf's .grad belongs to the stream of the
    leaf's first graph, which a capture must not wait for."""

    @staticmethod
    def forward(ctx, logits, ids, mask=None, temperature=1.0):
        out = token_logprobs(logits.detach(), ids, mask=mask, temperature=temperature, want_lse=True)
        ctx.save_for_backward(logits, ids, mask, out["lse"], out["entropy"])
        ctx.temperature = temperature
        ctx.set_materialize_grads(False)
        return out["logp"], out["entropy"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dlogp, dent):
        logits, ids, mask, lse, ent = ctx.saved_tensors
        if dlogp is None and dent is None:
            return None, None, None, None
        return token_logprobs_backward(
            logits.detach(), ids if dlogp is not None else None,
            dlogp.float().contiguous() if dlogp is not None else None, lse,
            entropy=ent if dent is not None else None,
            dentropy=dent.float().contiguous() if dent is not None else None, mask=mask,
            temperature=ctx.temperature), None, None, None


def new_distill_workspace(device) -> torch.Tensor:
    """Zero-filled workspace for topk_distill (every call leaves it ready for the next)."""
    return torch.zeros(rl_topk_distill_workspace_size(), dtype=torch.uint8, device=device)


def read_distill_stats(stats: torch.Tensor) -> dict:
    return distill_stats_from_bytes(stats.cpu().numpy().tobytes())


def topk_distill(logits: torch.Tensor, teacher_ids: torch.Tensor, teacher_logp: torch.Tensor,
                 mask: torch.Tensor | None = None, weight: torch.Tensor | None = None, tail: str = "bucket",
                 reverse: float = 0.0, temperature: float = 1.0, grad_scale: float = 1.0, norm: float = 0.0,
                 dlogits="new", row_loss="new", workspace: torch.Tensor | None = None,
                 stats: torch.Tensor | None = None, stream=None) -> dict:
    """Distillation of the student's ``logits`` [R, V] from a teacher's top
    entries, loss and gradient in one launch (rl_topk_distill_fwd_bwd).

    ``teacher_ids`` int64 and ``teacher_logp`` float32 [R, K]: what
    token_logprobs gives as topk_ids and topk_logp (an id of -1 is an empty
    entry).  ``tail``: "bucket" keeps the rest of the vocabulary as one more
    outcome, "renormalise" normalises the teacher over its entries.
    ``reverse``: the weight of KL(student || teacher) beside KL(teacher ||
    student).  ``mask`` uint8 or bool [R]; ``weight`` float32 [R]; ``norm``: what
    the sum over rows is divided by (0: the number of valid rows).
    ``dlogits`` / ``row_loss``: "new" allocates, None skips, a tensor is written
    (``dlogits=logits`` overwrites the logits).  ``workspace``: one call at a
    time may use it; calls on two streams, or graphs replayed at once, take one
    each (None: a new one).

    Returns dict(loss: float32 scalar, row_loss: [R], dlogits, stats: the device
    record for read_distill_stats, workspace)."""
    dt, R, V, ld = _logits(logits)
    dev = logits.device
    if teacher_ids.dim() != 2:
        raise ValueError("teacher_ids must be of shape [R, K]")
    K = teacher_ids.shape[1]
    _given("teacher_ids", teacher_ids, torch.int64, (R, K), dev)
    _given("teacher_logp", teacher_logp, torch.float32, (R, K), dev)
    mask = _mask(mask, R, dev)
    if weight is not None:
        _given("weight", weight, torch.float32, (R,), dev)
    if tail not in DISTILL_TAILS:
        raise ValueError(f"tail must be one of {sorted(DISTILL_TAILS)}")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous and on the logits' device")
    if stats is not None and (stats.dtype != torch.uint8 or stats.device != dev or
                              stats.numel() < DISTILL_STATS_BYTES or not stats.is_contiguous()):
        raise ValueError(f"stats must be a contiguous uint8 tensor of {DISTILL_STATS_BYTES} bytes on the logits' device")
    given = [None if isinstance(t, str) else t for t in (dlogits, row_loss)]
    with _on(dev, stream, (logits, teacher_ids, teacher_logp, mask, weight, workspace, stats, *given)):
        if dlogits is not None:
            dlogits = _dlogits_like(logits, dlogits, ld)
        if isinstance(row_loss, str):
            row_loss = torch.empty(R, dtype=torch.float32, device=dev)
        elif row_loss is not None:
            _given("row_loss", row_loss, torch.float32, (R,), dev)
        loss = torch.empty((), dtype=torch.float32, device=dev)
        workspace = new_distill_workspace(dev) if workspace is None else workspace
        stats = torch.empty(DISTILL_STATS_BYTES, dtype=torch.uint8, device=dev) if stats is None else stats
        d = rl_topk_distill_desc(
            logits=logits.data_ptr(), dtype=dt, R=R, V=V, ld=ld, teacher_ids=teacher_ids.data_ptr(),
            teacher_logp=teacher_logp.data_ptr(), K=K, mask=_p(mask), weight=_p(weight), tail=DISTILL_TAILS[tail],
            reverse=reverse, temperature=temperature, grad_scale=grad_scale, norm=norm, dlogits=_p(dlogits),
            row_loss_out=_p(row_loss), loss_out=loss.data_ptr(), stats_dev=stats.data_ptr(),
            workspace=workspace.data_ptr(), workspace_bytes=workspace.numel() * workspace.element_size())
        _check(load().rl_topk_distill_fwd_bwd(d, _raw_stream(dev)), "rl_topk_distill_fwd_bwd")
        _written(*given)
    return dict(loss=loss, row_loss=row_loss, dlogits=dlogits, stats=stats, workspace=workspace)


class FusedTopkDistill(torch.autograd.Function):
    """Autograd wrapper: loss = FusedTopkDistill.apply(logits, teacher_ids,
    teacher_logp, mask, options), ``options`` a dict of topk_distill's keyword
    arguments: not dlogits, for every call keeps its own, and not stream, for the
    backward pass runs on the stream that is current here (call it under
    ``torch.cuda.stream`` for another one).

    The forward pass runs the fused kernel and keeps its gradient; the backward
    pass hands it back times the incoming gradient.  That product is skipped
    where the incoming gradient is 1, which is read on the host, except while
    a CUDA graph is being captured, where nothing is read and the product is
    always taken (captured as TokenLogprobs' backward is)."""

    @staticmethod
    def forward(ctx, logits, teacher_ids, teacher_logp, mask=None, options=None):
        options = dict(options or {})
        if "dlogits" in options:
            raise ValueError("the wrapper keeps a gradient of its own: options must not name dlogits")
        if "stream" in options:
            raise ValueError("the backward pass runs on the current stream: options must not name stream")
        out = topk_distill(logits.detach(), teacher_ids, teacher_logp, mask=mask, **options)
        ctx.save_for_backward(out["dlogits"])
        return out["loss"]

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        (dlogits,) = ctx.saved_tensors
        if torch.cuda.is_current_stream_capturing() or float(grad) != 1.0:
            # the product in fp32: a loss scale may not fit the gradient's type
            dlogits = (dlogits.float() * grad).to(dlogits.dtype)
        return dlogits, None, None, None, None
