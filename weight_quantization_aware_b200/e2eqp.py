"""One E2E-QP training step of a quantized output projection against a full-precision
teacher.

E2E-QP trains the step sizes s of frozen codes end to end (modelfoundations note
"EfficientQAT, low-bit training on a single GPU": Phase 2, "Both phases").  The pages
train on the next token; here the loss is the distillation from a teacher's top
alternatives, which a quantized copy of a model has at hand: its own full-precision
original.  This module strings the library's calls together:

    teacher (once per batch):  ids, tlp = teacher_alternatives(logits of the original)
    per step:   Y = dq_linear_fwd(X, codes, zq, s)              logits [T, V]
                loss, dY = distill_topk_step(Y, ids, tlp, ...)  in place of Y
                dX, ds = dq_linear_bwd_s(X, codes, zq, s, dY)
                adamw_step over s

dX is what the layers below the projection train on.
"""
from __future__ import annotations

from dataclasses import dataclass

import torch

from . import (EQAT_BF16, adamw_step, cosine_lr, distill_topk_step, dq_linear_bwd_s, dq_linear_fwd, load_library,
               token_logprobs, workspace)


@dataclass
class QuantHead:
    """A packed output projection: codes and zq as pack_codes gives them, s trained."""
    codes: torch.Tensor
    zq: torch.Tensor
    s: torch.Tensor
    moments: tuple | None = None
    ws: torch.Tensor | None = None


@dataclass
class E2EQPConfig:
    bits: int = 2
    group: int = 64
    lr: float = 2e-5          # step sizes (2-bit setting of the pages)
    lr_min: float = 0.0
    total_steps: int = 4096
    beta1: float = 0.9
    beta2: float = 0.999
    eps: float = 1e-8
    temperature: float = 1.0
    tail: bool = True         # compare the mass outside the alternatives too


def teacher_alternatives(logits, k, temperature=1.0):
    """(ids, tlp) of a teacher's logits [T, V]: its k alternatives per row and their log
    probabilities at the temperature."""
    skip = torch.full((logits.shape[0],), -1, dtype=torch.int64, device=logits.device)
    _, _, ids, tlp = token_logprobs(logits, skip, top_k=k, temperature=temperature)
    return ids, tlp


def e2eqp_head_step(head: QuantHead, X, ids, tlp, cfg: E2EQPConfig, step: int, weight=None):
    """One step (step >= 1): returns (loss fp32 [T], dX).  X [T, K] bf16; weight fp32 [T]
    (default: 1 / T each, the mean over the tokens).  Without tokens the scales' gradient is 0."""
    T, K = X.shape
    N = head.codes.shape[0]
    need = load_library().eqat_workspace_bytes(T, N, K, cfg.bits, cfg.group, EQAT_BF16)
    if head.ws is None or head.ws.numel() < need:  # few tokens of a narrow layer need more than many
        head.ws = workspace(T, N, K, cfg.bits, cfg.group, X.dtype, X.device)
    if weight is None:
        weight = torch.full((T,), 1.0 / max(T, 1), dtype=torch.float32, device=X.device)
    Y = dq_linear_fwd(X, head.codes, head.zq, head.s, cfg.bits, cfg.group, ws=head.ws)
    loss, dY = distill_topk_step(Y, ids, tlp, weight=weight, temperature=cfg.temperature, tail=cfg.tail, dlogits=Y)
    # a forward at decode sizes leaves no W-hat in the workspace
    dX, ds = dq_linear_bwd_s(X, head.codes, head.zq, head.s, dY, cfg.bits, cfg.group, ws=head.ws, w_hat_in_ws=T > 8)
    if head.moments is None:
        head.moments = (torch.zeros_like(head.s), torch.zeros_like(head.s))
    group = dict(lr=cosine_lr(cfg.lr, cfg.lr_min, step - 1, cfg.total_steps), beta1=cfg.beta1, beta2=cfg.beta2, eps=cfg.eps)
    adamw_step([(head.s, ds, *head.moments, None, 0)], [group], step)
    return loss, dX
