"""Token log-probabilities over torch CUDA tensors: the log-probabilities of
given tokens with entropy and top alternatives, their gradient, and the
autograd wrapper around both (rl_token_logprobs, rl_token_logprobs_bwd of
include/rltoken.h; the rollout buffer of the ainews.cool RL.cu article,
section "技术深度解析", holds such log-probabilities).

Outputs are allocated with torch, everything is computed by librlloss's
kernels.  Inputs are checked and never copied: a tensor of another type,
layout or device is refused with a ValueError.  Calls run on the logits'
device, on ``stream`` (a torch.cuda.Stream) or torch's current stream there;
their outputs belong to that stream.
"""
from __future__ import annotations

import contextlib

import torch

from . import DTYPES, rl_token_logprobs, rl_token_logprobs_bwd

_DT = {torch.float32: DTYPES["f32"], torch.bfloat16: DTYPES["bf16"], torch.float16: DTYPES["f16"]}
_HERE = contextlib.nullcontext()


def _on(device: torch.device, stream):
    """The context in which a call allocates and launches: the logits' device
    and, if one is given, the caller's stream."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if device.index is not None and device.index != torch.cuda.current_device():
        return torch.cuda.device(device)
    return _HERE


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
    with _on(dev, stream):
        f32 = dict(dtype=torch.float32, device=dev)
        logp = torch.empty(ids.shape, **f32) if ids is not None else None
        ent = torch.empty(R, **f32) if want_entropy else None
        lse = torch.empty(R, **f32) if want_lse else None
        top = torch.empty((R, k), dtype=torch.int64, device=dev) if k > 0 else None
        top_lp = torch.empty((R, k), **f32) if k > 0 else None
        rl_token_logprobs(logits, dt, R, V, ld, ids if n else None, n, mask, temperature, k, logp if n else None, ent,
                          lse, top, top_lp, status)
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
    in place (``dlogits=logits`` overwrites the logits)."""
    dt, R, V, ld = _logits(logits)
    dev = logits.device
    n = _n_ids(ids, R)
    if ids is not None:
        shape = (R,) if ids.dim() == 1 else (R, n)
        _given("ids", ids, torch.int64, shape, dev)
        if dlogp is None:
            raise ValueError("dlogp must be given with ids")
        _given("dlogp", dlogp, torch.float32, shape, dev)
    _given("lse", lse, torch.float32, (R,), dev)
    for name, t in (("entropy", entropy), ("dentropy", dentropy)):
        if t is not None:
            _given(name, t, torch.float32, (R,), dev)
    mask = _mask(mask, R, dev)
    with _on(dev, stream):
        dlogits = _dlogits_like(logits, dlogits, ld)
        rl_token_logprobs_bwd(logits, dt, R, V, ld, ids if n else None, n, mask, temperature, lse, entropy,
                              dlogp if n else None, dentropy, dlogits, status)
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
    gradients; it reads no value on the host, so it can be captured."""

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
