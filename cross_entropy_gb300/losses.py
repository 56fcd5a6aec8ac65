"""The losses of post-training, each with its gradient.

* :func:`distill_fwd`, :func:`distill_bwd`, :func:`distill_fwd_bwd_fused` --
  distillation from a teacher's top logits: KL of the teacher's distribution
  over the tokens it lists, and a bucket for its others where their mass is
  known, against the student's whole softmax.
* :func:`policy_loss_fwd_bwd_fused` -- the clipped policy loss with a KL term,
  from logits; :func:`policy_loss` the same from log-probs.
* :func:`preference_loss_fwd_bwd_fused` -- the preference loss of paired
  sequences, from logits; :func:`preference_loss` the same from log-probs.

The calls from log-probs serve the heads that do not keep their logits: their
``dlogp`` is the ``grad_logp`` of :func:`linear_selective_logsoftmax_bwd`,
:func:`vocab_slice_grad` and :func:`selective_logsoftmax_bwd`.

Everything is checked and marshalled here and computed in the library's
kernels; see ``include/gbce.h`` for the formulas and for what each call does
with rows left out, empty lists and bad indices.  With ``stream`` given,
whatever a call has to convert or allocate is converted and allocated on that
stream.
"""

from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import (GBCE_BF16, GBCE_F32, REDUCTIONS, _check, _check_buffer, _check_dlogits, _check_status,
               _dtype_code, _ptr, load_library)
from .linear import _flat, _floats, _int64, _mask, _matrix, _on, _stream_ptr, _stride

KINDS = {"sigmoid": 0, "squared": 1}


class DistillForward(NamedTuple):
    loss: torch.Tensor              # [rows] for 'none', [] otherwise
    rest_state: torch.Tensor        # [rows, 2] max and sum of exp over the unlisted columns
    n_items: torch.Tensor           # [] int64


class DistillFused(NamedTuple):
    loss: torch.Tensor
    dlogits: torch.Tensor
    n_items: torch.Tensor


class PolicyLoss(NamedTuple):
    loss: torch.Tensor              # [rows] for 'none', [] otherwise
    dlogp: Optional[torch.Tensor]   # logp's shape
    n_items: torch.Tensor           # [] int64


class PolicyFused(NamedTuple):
    loss: torch.Tensor
    dlogits: torch.Tensor
    logp: Optional[torch.Tensor]    # [rows] log p of the label (0 for ignored rows)
    n_items: torch.Tensor


class PreferenceLoss(NamedTuple):
    loss: torch.Tensor              # [pairs] for 'none', [] otherwise
    dlogp: Optional[torch.Tensor]   # logp's shape
    seq_score: torch.Tensor         # [2 pairs] each sequence's sum (or mean) of log p - ref


class PreferenceFused(NamedTuple):
    loss: torch.Tensor
    dlogits: torch.Tensor
    logp: Optional[torch.Tensor]
    seq_score: torch.Tensor


class PolicyOptions(ctypes.Structure):
    """gbce_policy_options."""

    _fields_ = [("clip_low", ctypes.c_float), ("clip_high", ctypes.c_float),
                ("kl_beta", ctypes.c_float)]


class PreferenceOptions(ctypes.Structure):
    """gbce_preference_options."""

    _fields_ = [("beta", ctypes.c_float), ("margin", ctypes.c_float),
                ("label_smoothing", ctypes.c_float), ("kind", ctypes.c_int32),
                ("average", ctypes.c_int32)]


@functools.lru_cache(maxsize=64)
def _policy_options(clip_low: float, clip_high: float, kl_beta: float):
    """The options and their (host) address; by value, so only of plain numbers."""
    opt = PolicyOptions(clip_low, clip_high, kl_beta)
    return opt, ctypes.addressof(opt)


@functools.lru_cache(maxsize=256)
def preference_workspace_size(rows: int, pairs: int) -> int:
    return int(load_library().gbce_preference_workspace_size(int(rows), int(pairs)))


@functools.lru_cache(maxsize=256)
def _row_workspace_size(rows: int) -> int:
    return int(load_library().gbce_workspace_size(rows, 1, 1))


_CODES = {torch.float32: GBCE_F32, torch.bfloat16: GBCE_BF16}


def _logits(logits: torch.Tensor):
    """The [rows, vocab] view (no copy), its type's code, and its row stride."""
    x = _matrix(logits, "logits")
    code = _CODES.get(x.dtype)
    if code is None:
        _dtype_code(x)  # (raises)
    return x, code, _stride(x)


def _per_row(x, lead, what, device):
    """One fp32 value per row: lead's shape, any shape that broadcasts to it, or flat [rows]."""
    if x is None:
        return None
    t = x
    if not (isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.device == device):
        t = torch.as_tensor(t, dtype=torch.float32, device=device)
    rows = 1
    for n in lead:
        rows *= n
    if t.dim() != 1 or t.numel() != rows:
        try:
            t = t.broadcast_to(lead)
        except RuntimeError as exc:
            raise ValueError(f"{what} must have one value per row {tuple(lead)}, or broadcast to "
                             f"that, got {tuple(t.shape)}") from exc
    return _flat(t, rows)


def _upstream(grad_out, n, what, device):
    """[n] for 'none', one value otherwise; ones when not given."""
    if grad_out is None:
        return torch.ones(n, dtype=torch.float32, device=device)
    g = grad_out
    if not (isinstance(g, torch.Tensor) and g.dtype == torch.float32 and g.device == device):
        g = torch.as_tensor(g, dtype=torch.float32, device=device)
    if g.numel() != n:
        raise ValueError(f"grad_out must have one entry per {what} for 'none', one otherwise")
    return _flat(g, n)


def _scratch(ws, need, device):
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    elif ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _row_scratch(ws, rows, device):
    """The workspace, its address and size, and the item count: the workspace's own first element
    where the workspace is this call's (an allocation less), else one of its own."""
    if ws is None and rows > 0:
        need = _row_workspace_size(rows)
        ws = torch.empty((need + 7) // 8, dtype=torch.int64, device=device)
        return ws, ws.data_ptr(), need, ws[0]
    ws, wp, wb = _scratch(ws, 0, device)
    return ws, wp, wb, torch.empty((), dtype=torch.int64, device=device)


def _dlogits(buf, logits, x):
    """The gradient's buffer, its address and its row stride."""
    if buf is None:
        buf = torch.empty(logits.shape, dtype=x.dtype, device=x.device)
        return buf, buf.data_ptr(), x.shape[1]
    d = _matrix(buf, "dlogits")
    _check_dlogits(d, x)
    return buf, d.data_ptr(), _stride(d)


def _teacher(index, teacher_logits, teacher_rest, rows, device):
    idx = _int64(index, device)
    t = teacher_logits
    if t.dtype != torch.float32 or t.device != device:
        t = t.to(device=device, dtype=torch.float32)
    t = t.contiguous()
    shape = idx.shape
    k = shape[-1] if shape else 0
    if t.shape != shape or idx.numel() != rows * k:
        raise ValueError(f"index and teacher_logits must have one shape [..., k] with k entries for "
                         f"each of the {rows} rows, got {tuple(shape)} and {tuple(t.shape)}")
    rest = None if teacher_rest is None else _floats(teacher_rest, (rows,), device)
    return idx, k, t, rest


def distill_fwd(logits: torch.Tensor, index, teacher_logits: torch.Tensor,
                teacher_rest: Optional[torch.Tensor] = None, temperature: float = 1.0,
                row_mask: Optional[torch.Tensor] = None, reduction: str = "mean", *,
                workspace: Optional[torch.Tensor] = None,
                dev_status: Optional[torch.Tensor] = None, stream=None) -> DistillForward:
    """Distillation from a teacher's top logits: the loss, and the state :func:`distill_bwd` takes.

    ``index`` [..., k] holds the teacher's columns of each row (-1: no entry) and
    ``teacher_logits`` [..., k] its logits there; the same temperature softens both
    sides.  ``teacher_rest`` [...] is log-sum-exp of the teacher's other logits /
    T; without it the listed entries are renormalised.  Of a teacher given as
    log-probs lp it is log1p(-sum exp(lp)) at T = 1 only: at another T the listed
    log-probs do not determine it, and it has to come from the teacher's logits.
    """
    lib = load_library()
    x, code, xs = _logits(logits)
    rows, vocab = x.shape
    dev = x.device
    red = REDUCTIONS[reduction]
    with _on(dev, stream):
        idx, k, t, rest = _teacher(index, teacher_logits, teacher_rest, rows, dev)
        mask = _mask(row_mask, rows, dev)
        loss = torch.empty((rows,) if red == 0 else (), dtype=torch.float32, device=dev)
        state = torch.empty((rows, 2), dtype=torch.float32, device=dev)
        _check_status(dev_status, dev)
        ws, wp, wb, n_items = _row_scratch(workspace, rows, dev)
        st = lib.distill_fwd(x.data_ptr(), code, rows, vocab, xs, idx.data_ptr(), k,
                             t.data_ptr(), _ptr(rest), float(temperature), _ptr(mask), red,
                             loss.data_ptr(), state.data_ptr(), n_items.data_ptr(), wp, wb,
                             _ptr(dev_status), _stream_ptr(stream, dev))
    _check(st, "distill_fwd")
    return DistillForward(loss, state, n_items)


def distill_bwd(logits: torch.Tensor, index, teacher_logits: torch.Tensor,
                teacher_rest: Optional[torch.Tensor], grad_out, rest_state: torch.Tensor,
                n_items=None, temperature: float = 1.0, row_mask: Optional[torch.Tensor] = None,
                reduction: str = "mean", *, dlogits: Optional[torch.Tensor] = None,
                dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dL/dlogits of :func:`distill_fwd`, given the same arguments, its ``rest_state`` and (for
    'mean') its ``n_items``."""
    lib = load_library()
    x, code, xs = _logits(logits)
    rows, vocab = x.shape
    dev = x.device
    red = REDUCTIONS[reduction]
    with _on(dev, stream):
        idx, k, t, rest = _teacher(index, teacher_logits, teacher_rest, rows, dev)
        mask = _mask(row_mask, rows, dev)
        g = _upstream(grad_out, rows if red == 0 else 1, "row", dev)
        state = _floats(rest_state, (rows, 2), dev)
        n = None if n_items is None else _int64(n_items, dev).reshape(1)
        dlogits, dp, ds = _dlogits(dlogits, logits, x)
        _check_status(dev_status, dev)
        st = lib.distill_bwd(x.data_ptr(), code, rows, vocab, xs, idx.data_ptr(), k,
                             t.data_ptr(), _ptr(rest), float(temperature), _ptr(mask), red,
                             g.data_ptr(), state.data_ptr(), _ptr(n), dp, ds,
                             _ptr(dev_status), _stream_ptr(stream, dev))
    _check(st, "distill_bwd")
    return dlogits


def distill_fwd_bwd_fused(logits: torch.Tensor, index, teacher_logits: torch.Tensor,
                          teacher_rest: Optional[torch.Tensor] = None, grad_out=None,
                          temperature: float = 1.0, row_mask: Optional[torch.Tensor] = None,
                          reduction: str = "mean", *, dlogits: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None,
                          dev_status: Optional[torch.Tensor] = None, stream=None) -> DistillFused:
    """:func:`distill_fwd` and its gradient in one call (upstream gradient known up front)."""
    lib = load_library()
    x, code, xs = _logits(logits)
    rows, vocab = x.shape
    dev = x.device
    red = REDUCTIONS[reduction]
    with _on(dev, stream):
        idx, k, t, rest = _teacher(index, teacher_logits, teacher_rest, rows, dev)
        mask = _mask(row_mask, rows, dev)
        g = _upstream(grad_out, rows if red == 0 else 1, "row", dev)
        loss = torch.empty((rows,) if red == 0 else (), dtype=torch.float32, device=dev)
        dlogits, dp, ds = _dlogits(dlogits, logits, x)
        _check_status(dev_status, dev)
        ws, wp, wb, n_items = _row_scratch(workspace, rows, dev)
        st = lib.distill_fwd_bwd_fused(x.data_ptr(), code, rows, vocab, xs,
                                       idx.data_ptr(), k, t.data_ptr(), _ptr(rest),
                                       float(temperature), _ptr(mask), red, g.data_ptr(),
                                       loss.data_ptr(), n_items.data_ptr(), dp, ds,
                                       wp, wb, _ptr(dev_status), _stream_ptr(stream, dev))
    _check(st, "distill_fwd_bwd_fused")
    return DistillFused(loss, dlogits, n_items)


def policy_loss(logp: torch.Tensor, advantages, old_logp=None, ref_logp=None, grad_out=None,
                row_mask: Optional[torch.Tensor] = None, *, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_beta: float = 0.0, reduction: str = "mean",
                want_grad: bool = True, dlogp: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, stream=None) -> PolicyLoss:
    """The clipped policy loss with a KL term from log-probs [...] of the sampled tokens.

    ``advantages``, ``old_logp`` (None: the current policy is the old one) and
    ``ref_logp`` have logp's shape or broadcast to it (an advantage per sequence as
    [sequences, 1]).  ``dlogp`` is the derivative by ``logp`` times ``grad_out``.
    """
    lib = load_library()
    if not logp.is_cuda:
        raise ValueError("logp must be a CUDA tensor (no CPU path exists)")
    dev, rows = logp.device, logp.numel()
    red = REDUCTIONS[reduction]
    opt = _policy_options(float(clip_low), float(clip_high), float(kl_beta))
    with _on(dev, stream):
        lp = _floats(logp, (rows,), dev)
        adv = _per_row(advantages, logp.shape, "advantages", dev)
        old = _per_row(old_logp, logp.shape, "old_logp", dev)
        ref = _per_row(ref_logp, logp.shape, "ref_logp", dev)
        mask = _mask(row_mask, rows, dev)
        g = _upstream(grad_out, rows if red == 0 else 1, "row", dev) if want_grad else None
        loss = torch.empty((rows,) if red == 0 else (), dtype=torch.float32, device=dev)
        if want_grad and dlogp is None:
            dlogp = torch.empty(logp.shape, dtype=torch.float32, device=dev)
        _check_buffer(dlogp, "dlogp", torch.float32, rows, dev)
        ws, wp, wb, n_items = _row_scratch(workspace, rows, dev)
        st = lib.policy_loss(lp.data_ptr(), rows, _ptr(mask), adv.data_ptr(), _ptr(old), _ptr(ref),
                             opt[1], red, _ptr(g), loss.data_ptr(),
                             _ptr(dlogp) if want_grad else None, n_items.data_ptr(), wp, wb,
                             _stream_ptr(stream, dev))
    _check(st, "policy_loss")
    return PolicyLoss(loss, dlogp if want_grad else None, n_items)


def policy_loss_fwd_bwd_fused(logits: torch.Tensor, labels, advantages, old_logp=None,
                              ref_logp=None, grad_out=None, ignore_index: int = -100, *,
                              clip_low: float = 0.2, clip_high: float = 0.2, kl_beta: float = 0.0,
                              temperature: float = 1.0, reduction: str = "mean",
                              dlogits: Optional[torch.Tensor] = None, want_logp: bool = True,
                              workspace: Optional[torch.Tensor] = None,
                              dev_status: Optional[torch.Tensor] = None,
                              stream=None) -> PolicyFused:
    """:func:`policy_loss` of log p of the labels, and its gradient with respect to the logits,
    in one sweep; rows with label ``ignore_index`` (prompt, padding) are left out."""
    lib = load_library()
    x, code, xs = _logits(logits)
    rows, vocab = x.shape
    lead, dev = logits.shape[:-1], x.device
    red = REDUCTIONS[reduction]
    opt = _policy_options(float(clip_low), float(clip_high), float(kl_beta))
    with _on(dev, stream):
        lab = _flat(_int64(labels, dev), rows)
        adv = _per_row(advantages, lead, "advantages", dev)
        old = _per_row(old_logp, lead, "old_logp", dev)
        ref = _per_row(ref_logp, lead, "ref_logp", dev)
        g = _upstream(grad_out, rows if red == 0 else 1, "row", dev)
        loss = torch.empty((rows,) if red == 0 else (), dtype=torch.float32, device=dev)
        logp = torch.empty(rows, dtype=torch.float32, device=dev) if want_logp else None
        dlogits, dp, ds = _dlogits(dlogits, logits, x)
        _check_status(dev_status, dev)
        ws, wp, wb, n_items = _row_scratch(workspace, rows, dev)
        st = lib.policy_loss_fwd_bwd_fused(x.data_ptr(), code, rows, vocab, xs,
                                           lab.data_ptr(), int(ignore_index), float(temperature),
                                           adv.data_ptr(), _ptr(old), _ptr(ref),
                                           opt[1], red, g.data_ptr(), loss.data_ptr(),
                                           _ptr(logp), n_items.data_ptr(), dp, ds,
                                           wp, wb, _ptr(dev_status), _stream_ptr(stream, dev))
    _check(st, "policy_loss_fwd_bwd_fused")
    return PolicyFused(loss, dlogits, logp, n_items)


def _sequences(seq_offsets, lead, device):
    """Offsets [2 pairs + 1] and the number of pairs; None: the rows of a [2 pairs, length] batch."""
    if seq_offsets is None:
        if len(lead) != 2 or lead[0] < 2 or lead[0] % 2:
            raise ValueError("without seq_offsets the rows must be a batch [2 pairs, length]")
        off = torch.arange(lead[0] + 1, dtype=torch.int64, device=device) * lead[1]
    else:
        off = _int64(seq_offsets, device)
        if off.dim() != 1 or off.numel() < 3 or off.numel() % 2 == 0:
            raise ValueError("seq_offsets must hold 2 pairs + 1 offsets (chosen sequences, then "
                             "rejected ones)")
    return off, (off.numel() - 1) // 2


@functools.lru_cache(maxsize=64)
def _preference_options(beta: float, margin: float, label_smoothing: float, kind: int,
                        average: bool):
    """The options and their (host) address; by value, so only of plain numbers.  Margin and
    smoothing are the sigmoid's: the library refuses them with the squared kind, so that one set
    of options can serve both kinds they stop here."""
    if kind == KINDS["squared"]:
        margin = label_smoothing = 0.0
    opt = PreferenceOptions(beta, margin, label_smoothing, kind, 1 if average else 0)
    return opt, ctypes.addressof(opt)


def preference_loss(logp: torch.Tensor, seq_offsets=None, ref_logp=None, grad_out=None,
                    row_mask: Optional[torch.Tensor] = None, *, beta: float = 0.1,
                    margin: float = 0.0, label_smoothing: float = 0.0, kind: str = "sigmoid",
                    average: bool = False, reduction: str = "mean", want_grad: bool = True,
                    dlogp: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None,
                    dev_status: Optional[torch.Tensor] = None, stream=None) -> PreferenceLoss:
    """The preference loss of paired sequences from their tokens' log-probs.

    ``seq_offsets`` [2 pairs + 1]: the first row of each sequence, the chosen
    answers before the rejected ones, and the end; None for logp [2 pairs, length].
    ``ref_logp`` is the reference policy's log-probs of the same tokens (None: no
    reference); ``average`` divides each sequence's sum by its live tokens.
    ``margin`` and ``label_smoothing`` are options of the sigmoid kind; the squared
    kind has neither and takes no notice of them.
    """
    lib = load_library()
    if not logp.is_cuda:
        raise ValueError("logp must be a CUDA tensor (no CPU path exists)")
    dev, rows = logp.device, logp.numel()
    red = REDUCTIONS[reduction]
    opt = _preference_options(float(beta), float(margin), float(label_smoothing), KINDS[kind],
                              bool(average))
    with _on(dev, stream):
        off, pairs = _sequences(seq_offsets, logp.shape, dev)
        lp = _floats(logp, (rows,), dev)
        ref = _per_row(ref_logp, logp.shape, "ref_logp", dev)
        mask = _mask(row_mask, rows, dev)
        g = _upstream(grad_out, pairs if red == 0 else 1, "pair", dev) if want_grad else None
        loss = torch.empty((pairs,) if red == 0 else (), dtype=torch.float32, device=dev)
        score = torch.empty(2 * pairs, dtype=torch.float32, device=dev)
        if want_grad and dlogp is None:
            dlogp = torch.empty(logp.shape, dtype=torch.float32, device=dev)
        _check_buffer(dlogp, "dlogp", torch.float32, rows, dev)
        _check_status(dev_status, dev)
        ws, wp, wb = _scratch(workspace, preference_workspace_size(rows, pairs), dev)
        st = lib.preference_loss(lp.data_ptr(), rows, _ptr(mask), off.data_ptr(), pairs, _ptr(ref),
                                 opt[1], red, _ptr(g), loss.data_ptr(),
                                 _ptr(dlogp) if want_grad else None, score.data_ptr(), wp, wb,
                                 _ptr(dev_status), _stream_ptr(stream, dev))
    _check(st, "preference_loss")
    return PreferenceLoss(loss, dlogp if want_grad else None, score)


def preference_loss_fwd_bwd_fused(logits: torch.Tensor, labels, seq_offsets=None, ref_logp=None,
                                  grad_out=None, ignore_index: int = -100, *, beta: float = 0.1,
                                  margin: float = 0.0, label_smoothing: float = 0.0,
                                  kind: str = "sigmoid", average: bool = False,
                                  temperature: float = 1.0, reduction: str = "mean",
                                  dlogits: Optional[torch.Tensor] = None, want_logp: bool = True,
                                  workspace: Optional[torch.Tensor] = None,
                                  dev_status: Optional[torch.Tensor] = None,
                                  stream=None) -> PreferenceFused:
    """:func:`preference_loss` (and its options) of log p of the labels, and its gradient with
    respect to the logits; rows with label ``ignore_index`` are left out of their sequence."""
    lib = load_library()
    x, code, xs = _logits(logits)
    rows, vocab = x.shape
    lead, dev = logits.shape[:-1], x.device
    red = REDUCTIONS[reduction]
    opt = _preference_options(float(beta), float(margin), float(label_smoothing), KINDS[kind],
                              bool(average))
    with _on(dev, stream):
        off, pairs = _sequences(seq_offsets, lead, dev)
        lab = _flat(_int64(labels, dev), rows)
        ref = _per_row(ref_logp, lead, "ref_logp", dev)
        g = _upstream(grad_out, pairs if red == 0 else 1, "pair", dev)
        loss = torch.empty((pairs,) if red == 0 else (), dtype=torch.float32, device=dev)
        score = torch.empty(2 * pairs, dtype=torch.float32, device=dev)
        logp = torch.empty(rows, dtype=torch.float32, device=dev) if want_logp else None
        dlogits, dp, ds = _dlogits(dlogits, logits, x)
        _check_status(dev_status, dev)
        ws, wp, wb = _scratch(workspace, preference_workspace_size(rows, pairs), dev)
        st = lib.preference_loss_fwd_bwd_fused(x.data_ptr(), code, rows, vocab, xs,
                                               lab.data_ptr(), int(ignore_index),
                                               float(temperature), off.data_ptr(), pairs, _ptr(ref),
                                               opt[1], red, g.data_ptr(),
                                               loss.data_ptr(), _ptr(logp), score.data_ptr(),
                                               dp, ds, wp, wb, _ptr(dev_status),
                                               _stream_ptr(stream, dev))
    _check(st, "preference_loss_fwd_bwd_fused")
    return PreferenceFused(loss, dlogits, logp, score)
