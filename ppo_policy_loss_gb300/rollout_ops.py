"""The rollout's operators over torch CUDA tensors: 8-bit codes of hidden states
and of the LM head, the logits of that 8-bit head, verification of drafted
tokens against those logits, and sampling (include/rlrollout.h; the actions and
log-probabilities that the rollout buffer of the ainews.cool RL.cu article,
section "技术深度解析", holds come from here).

Outputs are allocated with torch, everything is computed by librlloss's
kernels.  Inputs are checked and never copied: a tensor of another type,
layout or device is refused with a ValueError.  Calls run on the inputs'
device, on ``stream`` (a torch.cuda.Stream) or torch's current stream there;
their outputs belong to that stream.
"""
from __future__ import annotations

import torch

from . import _check, load, rl_lmhead_int8_workspace_size, rl_verify_drafts_desc
from .token_ops import _DT, _given, _logits, _on, _p, _raw_stream, _status, _written

_F32, _I64 = torch.float32, torch.int64


def _codes(name: str, t: torch.Tensor) -> int:
    """Row stride of a [rows, D] matrix of 8-bit codes."""
    if t.dtype != torch.int8 or t.dim() != 2 or not t.is_cuda or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D int8 CUDA tensor with unit column stride")
    return -(-t.shape[1] // 16) * 16 if t.shape[0] == 1 else t.stride(0)


def quantize_rows(x: torch.Tensor, codes: torch.Tensor | None = None, scale: torch.Tensor | None = None, stream=None):
    """8-bit codes of each row of ``x`` [R, D] and the scale they stand for, x ~
    scale[:, None] * codes: hidden states token by token, or a weight [V, D]
    channel by channel.  Returns (codes: int8 [R, D], rows a multiple of 16
    bytes apart; scale: float32 [R]); ``codes`` and ``scale`` are written where
    given.  A row with NaN or an infinity has scale NaN and codes 0."""
    dt, R, D, ld = _logits(x, "x")
    dev = x.device
    ld_c = -(-D // 16) * 16
    if codes is not None:
        ld_c = _codes("codes", codes)
        if tuple(codes.shape) != (R, D) or codes.device != dev:
            raise ValueError(f"codes must be of shape {(R, D)} on {dev}")
    if scale is not None:
        _given("scale", scale, _F32, (R,), dev)
    given = (codes, scale)
    with _on(dev, stream, (x, *given)):
        if codes is None:
            codes = torch.empty((R, ld_c), dtype=torch.int8, device=dev)
            codes = codes if ld_c == D else codes[:, :D]
        if scale is None:
            scale = torch.empty(R, dtype=_F32, device=dev)
        _check(load().rl_quantize_rows_int8(x.data_ptr(), dt, R, D, ld, codes.data_ptr(), ld_c, scale.data_ptr(), _raw_stream(dev)),
               "rl_quantize_rows_int8")
        _written(*given)
    return codes, scale


def new_int8_workspace(R: int, D: int, device) -> torch.Tensor:
    """Workspace for lmhead_logits_int8 of at most R tokens (it need not be initialised)."""
    return torch.empty(max(16, rl_lmhead_int8_workspace_size(R, D)), dtype=torch.uint8, device=device)


def lmhead_logits_int8(hidden: torch.Tensor, scale_h: torch.Tensor, weight: torch.Tensor, scale_w: torch.Tensor,
                       dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Logits [R, V] of an 8-bit LM head: scale_h[r] scale_w[v] times the exact
    sum of products of the codes ``hidden`` int8 [R, D] and ``weight`` int8 [V, D]
    (quantize_rows gives both).

    ``out``: [R, V] float32, bfloat16 or float16, written where given (else new, of
    ``dtype``, rows a multiple of 16 bytes apart, as the token operators want
    them).  ``workspace``: new_int8_workspace(R, D); calls on two streams, or
    graphs replayed at once, take one each (None: a new one).  ``status``: int32
    [1], collects RL_DEVERR_* bits."""
    ld_h, ld_w = _codes("hidden", hidden), _codes("weight", weight)
    (R, D), V, dev = hidden.shape, weight.shape[0], hidden.device
    if weight.shape[1] != D or weight.device != dev:
        raise ValueError(f"weight must be of shape [V, {D}] on {dev}")
    _given("scale_h", scale_h, _F32, (R,), dev)
    _given("scale_w", scale_w, _F32, (V,), dev)
    if out is not None:
        dt, _, _, ld = _logits(out, "out")
        if tuple(out.shape) != (R, V) or out.device != dev:
            raise ValueError(f"out must be of shape {(R, V)} on {dev}")
    elif dtype not in _DT:
        raise ValueError("dtype must be float32, bfloat16 or float16")
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError("workspace must be contiguous and on the codes' device")
    status_p = _status(status, dev)
    given = out
    with _on(dev, stream, (hidden, scale_h, weight, scale_w, out, workspace, status)):
        if out is None:
            dt, per = _DT[dtype], 4 if dtype == _F32 else 8
            ld = -(-V // per) * per
            out = torch.empty((R, ld), dtype=dtype, device=dev)
            out = out if ld == V else out[:, :V]
        if workspace is None:
            workspace = new_int8_workspace(R, D, dev)
        _check(load().rl_lmhead_logits_int8(
            hidden.data_ptr(), ld_h, scale_h.data_ptr(), weight.data_ptr(), ld_w, scale_w.data_ptr(), R, D, V, dt, out.data_ptr(),
            ld, status_p, workspace.data_ptr(), workspace.numel() * workspace.element_size(), _raw_stream(dev)),
            "rl_lmhead_logits_int8")
        _written(given)
    return out


def _rows3(name: str, t: torch.Tensor, dtype, B: int, n: int, V: int, device) -> int:
    """Row stride of a [B, n, V] tensor whose rows are all equally far apart."""
    if t.dtype != dtype or t.device != device or t.shape != (B, n, V) or (V > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be a {dtype} tensor of shape {(B, n, V)} on {device} with unit column stride, "
                         f"not {t.dtype} {tuple(t.shape)} on {t.device}")
    ld = t.stride(1) if n > 1 else t.stride(0) if B > 1 else max(V, t.stride(0))
    if n > 1 and B > 1 and t.stride(0) != n * ld:
        raise ValueError(f"the rows of {name} must be equally far apart: stride(0) = {n} * stride(1)")
    return ld


def verify_drafts(target_logits: torch.Tensor, draft_ids: torch.Tensor | None, uniforms: torch.Tensor,
                  draft_logits: torch.Tensor | None = None, draft_lse: torch.Tensor | None = None,
                  n_draft: torch.Tensor | None = None, temperature: float = 1.0, status: torch.Tensor | None = None,
                  stream=None) -> dict:
    """Which of its drafted tokens each sequence keeps, and the token drawn after
    them: tokens come out as drawn from softmax(target_logits / temperature)
    alone (rl_verify_drafts).

    ``target_logits`` [B, G + 1, V] float32, bfloat16 or float16: row i follows
    the first i drafts.  ``draft_ids`` int64 [B, G] (None with G = 0).
    ``uniforms`` float64 [B, G + 1] in [0, 1): one for each draft, the last for
    the drawn token.  ``draft_logits`` [B, G, V] like the target's and
    ``draft_lse`` float32 [B, G] (what sample_tokens gave as lse): the
    distribution the drafts were drawn from; None: they were not drawn (looked
    up, or the most likely).  ``n_draft`` int32 [B]: drafts of each sequence, -1
    leaves a sequence out (None: G).  ``status`` int32 [1] collects RL_DEVERR_* bits.

    Returns dict(tokens: int64 [B, G + 1], -1 behind the drawn one; n_accepted:
    int64 [B]; logp: float32 [B, G + 1], the tokens' log-probabilities under the
    target; lse: float32 [B, G + 1], the target rows' log-sum-exp; both 0 behind)."""
    dt = _DT.get(target_logits.dtype)
    if dt is None or target_logits.dim() != 3 or not target_logits.is_cuda or target_logits.shape[1] < 1:
        raise ValueError("target_logits must be a [B, G + 1, V] float32, bfloat16 or float16 CUDA tensor")
    B, rows, V = target_logits.shape
    G, dev = rows - 1, target_logits.device
    ld = _rows3("target_logits", target_logits, target_logits.dtype, B, rows, V, dev)
    if draft_ids is not None:
        _given("draft_ids", draft_ids, _I64, (B, G), dev)
    elif G:
        raise ValueError("draft_ids must be given")
    _given("uniforms", uniforms, torch.float64, (B, rows), dev)
    if (draft_logits is None) != (draft_lse is None):
        raise ValueError("draft_logits and draft_lse go together")
    ld_draft = 0
    if draft_logits is not None:
        ld_draft = _rows3("draft_logits", draft_logits, target_logits.dtype, B, G, V, dev)
        _given("draft_lse", draft_lse, _F32, (B, G), dev)
    if n_draft is not None:
        _given("n_draft", n_draft, torch.int32, (B,), dev)
    status_p = _status(status, dev)
    with _on(dev, stream, (target_logits, draft_ids, uniforms, draft_logits, draft_lse, n_draft, status)):
        tokens = torch.empty((B, rows), dtype=_I64, device=dev)
        kept = torch.empty(B, dtype=_I64, device=dev)
        logp = torch.empty((B, rows), dtype=_F32, device=dev)
        lse = torch.empty((B, rows), dtype=_F32, device=dev)
        d = rl_verify_drafts_desc(  # in the record's order: by name it takes a microsecond more
            target_logits.data_ptr(), dt, B, G, V, ld, _p(draft_logits) if G else None, ld_draft, _p(draft_lse) if G else None,
            _p(draft_ids) if G else None, _p(n_draft), uniforms.data_ptr(), temperature, tokens.data_ptr(), kept.data_ptr(),
            logp.data_ptr(), lse.data_ptr(), status_p)
        _check(load().rl_verify_drafts(d, _raw_stream(dev)), "rl_verify_drafts")
    return dict(tokens=tokens, n_accepted=kept, logp=logp, lse=lse)


def sample_tokens(logits: torch.Tensor, uniforms: torch.Tensor, temperature: float = 1.0, status: torch.Tensor | None = None,
                  stream=None) -> dict:
    """One token of each row of ``logits`` [B, V], drawn from softmax(logits /
    temperature) with ``uniforms`` float64 [B] in [0, 1): the first token at which
    the running sum of probabilities exceeds it.  Returns dict(tokens: int64 [B],
    logp: float32 [B], lse: float32 [B])."""
    if logits.dim() != 2:
        raise ValueError("logits must be of shape [B, V]")
    if uniforms.dim() != 1:
        raise ValueError("uniforms must be of shape [B]")
    out = verify_drafts(logits.unsqueeze(1), None, uniforms.unsqueeze(1), temperature=temperature, status=status, stream=stream)
    return dict(tokens=out["tokens"].view(-1), logp=out["logp"].view(-1), lse=out["lse"].view(-1))
