"""The calls that start from hidden states, and the table's lookup.

* :func:`linear_selective_logsoftmax`, :func:`linear_selective_logsoftmax_bwd`
  -- :func:`selective_logsoftmax` of ``hidden @ weight.T`` without keeping the
  logits, and its gradient with respect to ``hidden`` and ``weight``.
* :func:`linear_ce_fwd`, :func:`linear_ce_bwd`, :func:`linear_ce_fwd_bwd_fused`
  -- the token cross-entropy of the same logits.
* :func:`embedding_lookup`, :func:`embedding_lookup_bwd` -- rows of a table by
  token with a scale, and the lookup's gradient, which with ``accumulate``
  joins the head's gradient of a tied table.

Everything is checked and marshalled here and computed in the library's
kernels; see ``include/gbce.h`` for what each call does with masked rows, bad
indices and strides.  With ``stream`` given, whatever a call has to convert or
allocate is converted and allocated on that stream.
"""

from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

import torch

from . import REDUCTIONS, _check, _check_buffer, _check_status, _dtype_code, _ptr, load_library


class LinearCeForward(NamedTuple):
    loss: torch.Tensor              # [rows] for 'none', [] otherwise
    logp: torch.Tensor              # [rows] log p of the label (0 for ignored rows)
    row_state: torch.Tensor         # [rows, 2] max and sum of exp over the row's columns
    n_items: torch.Tensor           # [] int64


class LinearCeFused(NamedTuple):
    loss: torch.Tensor
    dhidden: Optional[torch.Tensor]
    dweight: Optional[torch.Tensor]
    logp: Optional[torch.Tensor]
    n_items: torch.Tensor


_HERE = contextlib.nullcontext()


@contextlib.contextmanager
def _elsewhere(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _on(device, stream):
    """The tensors' device, and the stream where one is given."""
    if stream is None and torch.cuda.current_device() == device.index:
        return _HERE
    return _elsewhere(device, stream)


def _stream_ptr(stream, device) -> int:
    if stream is not None:
        return int(stream.cuda_stream)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _int64(x, device) -> torch.Tensor:
    if not (isinstance(x, torch.Tensor) and x.dtype == torch.int64 and x.device == device):
        x = torch.as_tensor(x, dtype=torch.int64, device=device)
    return x.contiguous()


def _matrix(t: torch.Tensor, what: str) -> torch.Tensor:
    """[..., n] with unit stride along n -> [rows, n] view (no copy)."""
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor (no CPU path exists)")
    if t.dim() < 2:
        raise ValueError(f"{what} must have shape [rows, dim] or [..., dim]")
    if t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{what} must have unit stride along its last dimension")
    if t.dim() > 2:
        try:
            t = t.view(-1, t.shape[-1])
        except RuntimeError as exc:
            raise ValueError(f"leading dimensions of {what} must flatten without a copy") from exc
    return t


def _stride(t: torch.Tensor) -> int:
    """Row stride of a [rows, dim] view; that of a single row says nothing."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _operands(hidden, weight):
    h, w = _matrix(hidden, "hidden"), _matrix(weight, "weight")
    if weight.dim() != 2:
        raise ValueError("weight must have shape [vocab, dim]")
    if w.device != h.device or w.dtype != h.dtype or w.shape[1] != h.shape[1]:
        raise ValueError(f"weight must be a {h.dtype} tensor [vocab, {h.shape[1]}] on {h.device}, "
                         f"got {w.dtype} {tuple(w.shape)} on {w.device}")
    _dtype_code(h)
    return h, w


def _flat(x, *shape):
    """x with this shape, contiguous; x itself where it is."""
    return (x if x.shape == shape else x.reshape(shape)).contiguous()


def _mask(row_mask, rows, device):
    if row_mask is None:
        return None
    if row_mask.dtype != torch.uint8 or row_mask.device != device:
        row_mask = row_mask.to(device=device, dtype=torch.uint8)
    return _flat(row_mask, rows)


def _index(index, lead, rows, device):
    idx = _int64(index, device)
    squeeze = idx.dim() == len(lead)
    k = 1 if squeeze else idx.shape[-1]
    return _flat(idx, rows, k), k, squeeze


def _floats(x, shape, device):
    if not (isinstance(x, torch.Tensor) and x.dtype == torch.float32 and x.device == device):
        x = torch.as_tensor(x, dtype=torch.float32, device=device)
    return _flat(x, *shape)


def _gradient(buf, like: torch.Tensor, name: str, want: bool):
    """The caller's gradient buffer, a new one, or None when it is not wanted."""
    if not want:
        if buf is not None:
            raise ValueError(f"{name} was given although it is not wanted")
        return None, None
    if buf is None:
        buf = torch.empty_like(like, memory_format=torch.contiguous_format)
        return buf, buf if buf.dim() == 2 else buf.view(-1, buf.shape[-1])
    d = _matrix(buf, name)
    if d.device != like.device or d.dtype != like.dtype or buf.shape != like.shape:
        raise ValueError(f"{name} must be a {like.dtype} tensor of shape {tuple(like.shape)} on "
                         f"{like.device}")
    return buf, d


def _wanted(d: Optional[torch.Tensor], weight: torch.Tensor) -> Optional[int]:
    """Address of a wanted gradient.  An empty tensor has none, which the library would read as
    not wanted: any address does for it, the weight's for one."""
    return None if d is None else d.data_ptr() or weight.data_ptr()


def linear_workspace_size(rows: int, vocab: int, dim: int, k: int = 1, dtype=torch.bfloat16,
                          backward: bool = True) -> int:
    """Bytes of workspace of a linear_* call of these sizes."""
    code = _dtype_code(torch.empty(0, dtype=dtype))
    return int(load_library().gbce_linear_workspace_size(int(rows), int(vocab), int(dim), int(k),
                                                         code, 1 if backward else 0))


def _workspace(ws, need: int, device):
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
        return ws, ws.data_ptr(), need
    if ws.device != device or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _linear_workspace(ws, lib, h, w, k, backward):
    need = 0
    if ws is None:
        need = lib.gbce_linear_workspace_size(h.shape[0], w.shape[0], h.shape[1], k,
                                              _dtype_code(h), backward)
    return _workspace(ws, need, h.device)


def _accumulates(accumulate, dweight, name="dweight"):
    if accumulate and dweight is None:
        raise ValueError(f"accumulate needs the {name} to add to")
    return 1 if accumulate else 0


def linear_selective_logsoftmax(hidden: torch.Tensor, weight: torch.Tensor, index,
                                temperature: float = 1.0,
                                row_mask: Optional[torch.Tensor] = None, *,
                                out: Optional[torch.Tensor] = None, with_state: bool = False,
                                workspace: Optional[torch.Tensor] = None,
                                dev_status: Optional[torch.Tensor] = None, stream=None):
    """log p_{index[r, k]} of the logits ``hidden @ weight.T`` at temperature T.

    ``hidden`` [..., dim] and ``weight`` [vocab, dim] are both fp32 or both
    bf16; ``index`` is [..., K] (or [...] for K = 1).  fp32, shape
    index.shape; masked-out rows give 0 whatever they hold (a bf16 call of up
    to 128 rows may read them).  ``with_state``: returns ``(logp, row_state)``, row_state [rows, 2] being what the backward
    takes.
    """
    lib = load_library()
    h, w = _operands(hidden, weight)
    rows = h.shape[0]
    lead = hidden.shape[:-1]
    with _on(h.device, stream):
        idx, k, squeeze = _index(index, lead, rows, h.device)
        mask = _mask(row_mask, rows, h.device)
        shape = lead if squeeze else (*lead, k)
        if out is None:
            out = torch.empty(shape, dtype=torch.float32, device=h.device)
        else:
            _check_buffer(out, "out", torch.float32, rows * k, h.device)
        _check_status(dev_status, h.device)
        state = (torch.empty((rows, 2), dtype=torch.float32, device=h.device)
                 if with_state else None)
        ws, ws_ptr, ws_bytes = _linear_workspace(workspace, lib, h, w, k, 0)
        st = lib.linear_selective_logsoftmax(
            h.data_ptr(), _stride(h), w.data_ptr(), _stride(w), _dtype_code(h), rows, w.shape[0],
            h.shape[1], idx.data_ptr(), k, float(temperature), _ptr(mask), out.data_ptr(),
            _ptr(state), ws_ptr, ws_bytes, _ptr(dev_status), _stream_ptr(stream, h.device))
    _check(st, "linear_selective_logsoftmax")
    res = out if out.shape == shape else out.view(shape)
    return (res, state) if with_state else res


def linear_selective_logsoftmax_bwd(hidden: torch.Tensor, weight: torch.Tensor, index, grad_logp,
                                    saved_logp: torch.Tensor, row_state: torch.Tensor,
                                    temperature: float = 1.0,
                                    row_mask: Optional[torch.Tensor] = None, *,
                                    dhidden: Optional[torch.Tensor] = None,
                                    dweight: Optional[torch.Tensor] = None,
                                    want_dhidden: bool = True, want_dweight: bool = True,
                                    accumulate: bool = False,
                                    workspace: Optional[torch.Tensor] = None,
                                    dev_status: Optional[torch.Tensor] = None, stream=None):
    """(dhidden, dweight) for upstream grad_logp = dL/d linear_selective_logsoftmax(...).

    ``saved_logp`` and ``row_state`` are the forward's (with_state=True).
    With ``accumulate`` the gradient is added to the given ``dweight``; a
    gradient that is not wanted is not computed (None).
    """
    lib = load_library()
    acc = _accumulates(accumulate, dweight)
    h, w = _operands(hidden, weight)
    rows = h.shape[0]
    with _on(h.device, stream):
        idx, k, _ = _index(index, hidden.shape[:-1], rows, h.device)
        mask = _mask(row_mask, rows, h.device)
        g = _floats(grad_logp, (rows, k), h.device)
        lp = _floats(saved_logp, (rows, k), h.device)
        rs = _floats(row_state, (rows, 2), h.device)
        dhidden, dh = _gradient(dhidden, hidden, "dhidden", want_dhidden)
        dweight, dw = _gradient(dweight, weight, "dweight", want_dweight)
        _check_status(dev_status, h.device)
        ws, ws_ptr, ws_bytes = _linear_workspace(workspace, lib, h, w, k, 1)
        st = lib.linear_selective_logsoftmax_bwd(
            h.data_ptr(), _stride(h), w.data_ptr(), _stride(w), _dtype_code(h), rows, w.shape[0],
            h.shape[1], idx.data_ptr(), k, float(temperature), _ptr(mask), g.data_ptr(),
            lp.data_ptr(), rs.data_ptr(), _wanted(dh, w), 0 if dh is None else _stride(dh), _ptr(dw),
            0 if dw is None else _stride(dw), acc, ws_ptr, ws_bytes, _ptr(dev_status),
            _stream_ptr(stream, h.device))
    _check(st, "linear_selective_logsoftmax_bwd")
    return dhidden, dweight


def linear_ce_fwd(hidden: torch.Tensor, weight: torch.Tensor, labels, ignore_index: int = -100,
                  temperature: float = 1.0, reduction: str = "mean", *,
                  workspace: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None) -> LinearCeForward:
    """Token cross-entropy of the logits ``hidden @ weight.T``; returns loss, log p of the
    labels, row states and n_items (log p and row states for :func:`linear_ce_bwd`)."""
    lib = load_library()
    h, w = _operands(hidden, weight)
    rows = h.shape[0]
    red = REDUCTIONS[reduction]
    with _on(h.device, stream):
        lab = _flat(_int64(labels, h.device), rows)
        loss = torch.empty((rows,) if red == 0 else (), dtype=torch.float32, device=h.device)
        logp = torch.empty(rows, dtype=torch.float32, device=h.device)
        state = torch.empty((rows, 2), dtype=torch.float32, device=h.device)
        n_items = torch.empty((), dtype=torch.int64, device=h.device)
        _check_status(dev_status, h.device)
        ws, ws_ptr, ws_bytes = _linear_workspace(workspace, lib, h, w, 1, 0)
        st = lib.linear_ce_fwd(
            h.data_ptr(), _stride(h), w.data_ptr(), _stride(w), _dtype_code(h), rows, w.shape[0],
            h.shape[1], lab.data_ptr(), int(ignore_index), float(temperature), red,
            loss.data_ptr(), logp.data_ptr(), state.data_ptr(), n_items.data_ptr(), ws_ptr,
            ws_bytes, _ptr(dev_status), _stream_ptr(stream, h.device))
    _check(st, "linear_ce_fwd")
    return LinearCeForward(loss, logp, state, n_items)


def _upstream(grad_out, rows, red, device):
    n = rows if red == 0 else 1
    if not isinstance(grad_out, torch.Tensor):
        grad_out = torch.as_tensor(grad_out, dtype=torch.float32)
    if grad_out.numel() != n:
        raise ValueError("grad_out must have one entry per row for 'none', one otherwise")
    return _floats(grad_out, (n,), device)


def linear_ce_bwd(hidden: torch.Tensor, weight: torch.Tensor, labels, grad_out,
                  saved_logp: torch.Tensor, row_state: torch.Tensor, n_items=None,
                  ignore_index: int = -100, temperature: float = 1.0, reduction: str = "mean", *,
                  dhidden: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                  want_dhidden: bool = True, want_dweight: bool = True, accumulate: bool = False,
                  workspace: Optional[torch.Tensor] = None,
                  dev_status: Optional[torch.Tensor] = None, stream=None):
    """(dhidden, dweight) from :func:`linear_ce_fwd`'s log p, row states and n_items."""
    lib = load_library()
    acc = _accumulates(accumulate, dweight)
    h, w = _operands(hidden, weight)
    rows = h.shape[0]
    red = REDUCTIONS[reduction]
    with _on(h.device, stream):
        lab = _flat(_int64(labels, h.device), rows)
        g = _upstream(grad_out, rows, red, h.device)
        n = None if n_items is None else _int64(n_items, h.device).reshape(1)
        lp = _floats(saved_logp, (rows,), h.device)
        rs = _floats(row_state, (rows, 2), h.device)
        dhidden, dh = _gradient(dhidden, hidden, "dhidden", want_dhidden)
        dweight, dw = _gradient(dweight, weight, "dweight", want_dweight)
        _check_status(dev_status, h.device)
        ws, ws_ptr, ws_bytes = _linear_workspace(workspace, lib, h, w, 1, 1)
        st = lib.linear_ce_bwd(
            h.data_ptr(), _stride(h), w.data_ptr(), _stride(w), _dtype_code(h), rows, w.shape[0],
            h.shape[1], lab.data_ptr(), int(ignore_index), float(temperature), red, g.data_ptr(),
            lp.data_ptr(), rs.data_ptr(), _ptr(n), _wanted(dh, w), 0 if dh is None else _stride(dh),
            _ptr(dw), 0 if dw is None else _stride(dw), acc, ws_ptr, ws_bytes, _ptr(dev_status),
            _stream_ptr(stream, h.device))
    _check(st, "linear_ce_bwd")
    return dhidden, dweight


def linear_ce_fwd_bwd_fused(hidden: torch.Tensor, weight: torch.Tensor, labels, grad_out=None,
                            ignore_index: int = -100, temperature: float = 1.0,
                            reduction: str = "mean", *, dhidden: Optional[torch.Tensor] = None,
                            dweight: Optional[torch.Tensor] = None, want_dhidden: bool = True,
                            want_dweight: bool = True, accumulate: bool = False,
                            want_logp: bool = False, workspace: Optional[torch.Tensor] = None,
                            dev_status: Optional[torch.Tensor] = None,
                            stream=None) -> LinearCeFused:
    """Token cross-entropy of ``hidden @ weight.T`` with both gradients (upstream
    gradient known up front)."""
    lib = load_library()
    acc = _accumulates(accumulate, dweight)
    h, w = _operands(hidden, weight)
    rows = h.shape[0]
    red = REDUCTIONS[reduction]
    with _on(h.device, stream):
        lab = _flat(_int64(labels, h.device), rows)
        if grad_out is None:
            g = torch.ones(rows if red == 0 else 1, dtype=torch.float32, device=h.device)
        else:
            g = _upstream(grad_out, rows, red, h.device)
        loss = torch.empty((rows,) if red == 0 else (), dtype=torch.float32, device=h.device)
        logp = torch.empty(rows, dtype=torch.float32, device=h.device) if want_logp else None
        n_items = torch.empty((), dtype=torch.int64, device=h.device)
        dhidden, dh = _gradient(dhidden, hidden, "dhidden", want_dhidden)
        dweight, dw = _gradient(dweight, weight, "dweight", want_dweight)
        _check_status(dev_status, h.device)
        ws, ws_ptr, ws_bytes = _linear_workspace(workspace, lib, h, w, 1, 1)
        st = lib.linear_ce_fwd_bwd_fused(
            h.data_ptr(), _stride(h), w.data_ptr(), _stride(w), _dtype_code(h), rows, w.shape[0],
            h.shape[1], lab.data_ptr(), int(ignore_index), float(temperature), red, g.data_ptr(),
            loss.data_ptr(), _ptr(logp), None, n_items.data_ptr(), _wanted(dh, w),
            0 if dh is None else _stride(dh), _ptr(dw), 0 if dw is None else _stride(dw), acc,
            ws_ptr, ws_bytes, _ptr(dev_status), _stream_ptr(stream, h.device))
    _check(st, "linear_ce_fwd_bwd_fused")
    return LinearCeFused(loss, dhidden, dweight, logp, n_items)


# ------------------------------------------------------------ the table's lookup

def embedding_lookup(table: torch.Tensor, tokens, scale: float = 1.0, *, ignore_index: int = -100,
                     out: Optional[torch.Tensor] = None,
                     dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``scale * table[tokens]``, shape [*tokens.shape, dim], in the table's type; rows of
    zeros where a token equals ``ignore_index``."""
    lib = load_library()
    t = _matrix(table, "table")
    if table.dim() != 2:
        raise ValueError("table must have shape [vocab, dim]")
    code = _dtype_code(t)
    with _on(t.device, stream):
        tok = _int64(tokens, t.device)
        rows = tok.numel()
        shape = (*tok.shape, t.shape[1])
        if out is None:
            out = torch.empty(shape, dtype=t.dtype, device=t.device)
        elif out.shape != torch.Size(shape) or out.dtype != t.dtype or out.device != t.device:
            raise ValueError(f"out must be a {t.dtype} tensor of shape {shape} on {t.device}")
        o = _matrix(out.unsqueeze(0) if out.dim() == 1 else out, "out")
        _check_status(dev_status, t.device)
        st = lib.embedding_lookup(t.data_ptr(), _stride(t), code, t.shape[0], t.shape[1],
                                  tok.data_ptr(), rows, int(ignore_index), float(scale),
                                  o.data_ptr(), _stride(o), _ptr(dev_status),
                                  _stream_ptr(stream, t.device))
    _check(st, "embedding_lookup")
    return out


def embedding_lookup_bwd(grad_out: torch.Tensor, tokens, vocab: int, scale: float = 1.0, *,
                         ignore_index: int = -100, dtable: Optional[torch.Tensor] = None,
                         accumulate: bool = False, workspace: Optional[torch.Tensor] = None,
                         dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """dL/dtable [vocab, dim] for upstream ``grad_out`` [*tokens.shape, dim]; with
    ``accumulate`` added to the given ``dtable``."""
    lib = load_library()
    acc = _accumulates(accumulate, dtable, "dtable")
    g = _matrix(grad_out.unsqueeze(0) if grad_out.dim() == 1 else grad_out, "grad_out")
    code = _dtype_code(g)
    rows, dim = g.shape
    with _on(g.device, stream):
        tok = _int64(tokens, g.device)
        if tok.shape != grad_out.shape[:-1]:
            raise ValueError(f"tokens must have shape {tuple(grad_out.shape[:-1])}")
        if dtable is None:
            dtable = torch.empty((int(vocab), dim), dtype=g.dtype, device=g.device)
        d = _matrix(dtable, "dtable")
        if d.device != g.device or d.dtype != g.dtype or tuple(dtable.shape) != (int(vocab), dim):
            raise ValueError(f"dtable must be a {g.dtype} tensor of shape {(int(vocab), dim)} on "
                             f"{g.device}")
        _check_status(dev_status, g.device)
        need = 0
        if workspace is None:
            need = lib.gbce_embedding_workspace_size(rows, int(vocab), dim)
        ws, ws_ptr, ws_bytes = _workspace(workspace, need, g.device)
        st = lib.embedding_lookup_bwd(g.data_ptr(), _stride(g), code, rows, dim, tok.data_ptr(),
                                      int(vocab), int(ignore_index), float(scale), d.data_ptr(),
                                      _stride(d), acc, ws_ptr, ws_bytes, _ptr(dev_status),
                                      _stream_ptr(stream, g.device))
    _check(st, "embedding_lookup_bwd")
    return dtable
