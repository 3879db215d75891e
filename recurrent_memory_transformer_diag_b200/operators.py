"""The operators at the ends of the model, on device tensors: token embedding,
the norm in front of the head and the vocabulary loss, each with its gradients
(``include/armt.h``, "The ends of the model").

Each function checks its tensors (type, shape, dense layout, one device), hands
their addresses to the C ABI on ``stream`` (default: PyTorch's current stream of
the tensors' device) and returns without waiting; results go into the tensors
that the caller passes.  A wrong argument, or an empty one (no rows, no tokens),
raises ``ArmtError`` before anything is launched.  Results carry no autograd
history, but count as written in place: a backward pass that has kept one of
those tensors raises instead of using the new values.  Workspaces come from
PyTorch's allocator on the call's stream, unless the caller passes one (a uint8
tensor of ``workspace_bytes`` bytes).
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional

import torch
from torch.autograd.graph import increment_version as _written

from .armt import ARMT_BF16, ARMT_FP32, ArmtError, _check, lib

_TYPES = {torch.bfloat16: ARMT_BF16, torch.float32: ARMT_FP32}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def torch_type(name: str) -> torch.dtype:
    return torch.bfloat16 if name == "bf16" else torch.float32


def _bad(where: str, what: str):
    raise ArmtError(1, where, what)


def _tensor(where: str, name: str, t, dtype, shape, device):
    """One dense tensor of this type and shape on this device."""
    if not isinstance(t, torch.Tensor):
        _bad(where, f"{name} must be a tensor")
    if t.dtype is not dtype:
        _bad(where, f"{name} must be {dtype}, not {t.dtype}")
    if t.get_device() != device.index:
        _bad(where, f"{name} is on {t.device}, not on {device}")
    if t.shape != shape:
        _bad(where, f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        _bad(where, f"{name} must be contiguous")


def _matrix(where: str, name: str, t):
    """(library type, rows, columns, device) of the tensor the others go by."""
    kind = _TYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if kind is None or t.dim() != 2:
        _bad(where, f"{name} must be a 2-d tensor, bfloat16 or float32")
    if not t.is_cuda:
        _bad(where, f"{name} must be on a CUDA device")
    if not t.is_contiguous():
        _bad(where, f"{name} must be contiguous")
    n, d = t.shape
    return kind, n, d, t.device


def _ids(where: str, name: str, t, n: Optional[int], device) -> int:
    size = _ID_BYTES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if size is None:
        _bad(where, f"{name} must be an int32 or int64 tensor")
    if t.get_device() != device.index:
        _bad(where, f"{name} is on {t.device}, not on {device}")
    if not t.is_contiguous() or t.dim() != 1 or (n is not None and t.shape[0] != n):
        _bad(where, f"{name} must be contiguous, one id per row")
    return size


def _aligned(where: str, name: str, t):
    """On a 16-byte boundary (the operators look at this themselves; for what they look at too late)."""
    if t.data_ptr() % 16:
        _bad(where, f"{name} must start on a 16-byte boundary")


def _finite(where: str, name: str, x):
    if not math.isfinite(ctypes.c_float(x).value):
        _bad(where, f"{name} must be finite")


def _apart(where: str, outputs, others):
    """No output shares memory with an input or another output."""
    spans = [(name, t.data_ptr(), t.nbytes) for name, t in others if isinstance(t, torch.Tensor)]
    for name, t in outputs:
        a, size = t.data_ptr(), t.nbytes
        for other, b, n in spans:
            if a < b + n and b < a + size:
                _bad(where, f"{name} overlaps {other}")
        spans.append((name, a, size))


class _Here:
    """The current device and stream as they are."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE = _Here()


def on_stream(stream, device):
    """Make `device` and `stream` (a PyTorch stream, a raw handle, or None for the
    device's current one) current, so that what is allocated inside belongs to it."""
    if stream is None:
        return _HERE if torch._C._cuda_getDevice() == device.index else torch.cuda.device(device)
    if isinstance(stream, int):
        # 0 is the default stream; PyTorch would take it for "any stream of the pool"
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    if stream.device != device:
        _bad("stream", f"the stream belongs to {stream.device}, the tensors to {device}")
    return torch.cuda.stream(stream)


def _handle(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


@functools.lru_cache(maxsize=256)
def _need(size_fn: str, args) -> int:
    """Bytes of workspace, a function of the sizes alone."""
    need = ctypes.c_size_t()
    _check(getattr(lib(), size_fn)(*args, ctypes.byref(need)), size_fn)
    return need.value


def _space(where: str, size_fn: str, args, workspace, device, inputs):
    """(address, bytes, tensor to keep until the launches are made).  A given workspace
    shares no memory with an input: it is written while the inputs are read."""
    need = _need(size_fn, args)
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    else:
        if not isinstance(workspace, torch.Tensor) or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            _bad(where, "workspace must be a contiguous uint8 tensor")
        if workspace.get_device() != device.index:
            _bad(where, f"workspace is on {workspace.device}, not on {device}")
        if workspace.numel() < need:
            _bad(where, f"workspace holds {workspace.numel()} bytes, {need} are needed")
        _aligned(where, "workspace", workspace)
        _apart(where, [("workspace", workspace.view(-1)[:need])], inputs)   # what is used of it
    return workspace.data_ptr(), workspace.numel(), workspace


def workspace_bytes(op: str, dtype: torch.dtype, n: int, d: int, vocab: int = 1) -> int:
    """Bytes of workspace one call of ``op`` needs ("embed_grad", "rms_norm_grad",
    "token_loss" or "token_loss_grad") for n rows of d columns and this vocabulary."""
    t = _TYPES.get(dtype)
    if t is None:
        _bad("workspace_bytes", f"no operator takes {dtype}")
    calls = {"embed_grad": ("armt_embed_grad_workspace", (t, n, vocab, d)),
             "rms_norm_grad": ("armt_rms_norm_grad_workspace", (t, n, d)),
             "token_loss": ("armt_token_loss_workspace", (t, n, vocab, d, 0)),
             "token_loss_grad": ("armt_token_loss_workspace", (t, n, vocab, d, 1))}
    if op not in calls:
        _bad("workspace_bytes", f"unknown operator {op!r}")
    return _need(*calls[op])


def workspace_status(workspace, stream=None):
    """Wait for the stream; raises if a bounded wait ran out in the last
    ``token_loss`` or ``token_loss_grad`` call that used this workspace."""
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or workspace.nbytes < 4:
        _bad("armt_workspace_status", "workspace must be a tensor on a CUDA device")
    with on_stream(stream, workspace.device):
        _check(lib().armt_workspace_status(workspace.data_ptr(), _handle(workspace.device)), "armt_workspace_status")


def embed(ids, table, out, scale: float = 1.0, stream=None):
    """out[n] = scale * table[ids[n]]; zeros where the id is outside the table."""
    w = "armt_embed"
    t, vocab, d, dev = _matrix(w, "table", table)
    b = _ids(w, "ids", ids, None, dev)
    n = ids.shape[0]
    _tensor(w, "out", out, table.dtype, (n, d), dev)
    _apart(w, [("out", out)], [("table", table), ("ids", ids)])
    with on_stream(stream, dev):
        _check(lib().armt_embed(t, n, vocab, d, ids.data_ptr(), b, table.data_ptr(), scale, out.data_ptr(),
                                _handle(dev)), w)
    _written(out)


def embed_grad(ids, d_out, d_table, scale: float = 1.0, accumulate: bool = False, workspace=None, stream=None):
    """Gradient of ``embed`` to its table: d_table[v] = scale * sum of the d_out rows
    with id v, added to what d_table holds with ``accumulate``."""
    w = "armt_embed_grad"
    t, n, d, dev = _matrix(w, "d_out", d_out)
    b = _ids(w, "ids", ids, n, dev)
    if not isinstance(d_table, torch.Tensor) or d_table.dim() != 2:
        _bad(w, "d_table must be a 2-d tensor")
    vocab = d_table.shape[0]
    _tensor(w, "d_table", d_table, d_out.dtype, (vocab, d), dev)
    inputs = [("d_out", d_out), ("ids", ids)]
    _apart(w, [("d_table", d_table)], inputs + [("workspace", workspace)])
    with on_stream(stream, dev):
        at, size, keep = _space(w, "armt_embed_grad_workspace", (t, n, vocab, d), workspace, dev, inputs)
        _check(lib().armt_embed_grad(t, n, vocab, d, ids.data_ptr(), b, d_out.data_ptr(), scale, d_table.data_ptr(),
                                     int(bool(accumulate)), at, size, _handle(dev)), w)
    _written(d_table)


def rms_norm(x, gain, y, rstd=None, eps: float = 1e-5, stream=None):
    """y = x * rstd * gain with rstd = (mean x^2 + eps)^-1/2 per row; y may be x."""
    w = "armt_rms_norm"
    t, n, d, dev = _matrix(w, "x", x)
    _tensor(w, "gain", gain, x.dtype, (d,), dev)
    _tensor(w, "y", y, x.dtype, (n, d), dev)
    if rstd is not None:
        _tensor(w, "rstd", rstd, torch.float32, (n,), dev)
    _apart(w, [("y", y)], [("gain", gain)] + ([] if y.data_ptr() == x.data_ptr() else [("x", x)]))
    if rstd is not None:
        _apart(w, [("rstd", rstd)], [("x", x), ("gain", gain), ("y", y)])
    with on_stream(stream, dev):
        _check(lib().armt_rms_norm(t, n, d, x.data_ptr(), gain.data_ptr(), eps, y.data_ptr(),
                                   None if rstd is None else rstd.data_ptr(), _handle(dev)), w)
    _written(y if rstd is None else (y, rstd))


def rms_norm_grad(x, gain, rstd, dy, dx, d_gain, workspace=None, stream=None):
    """Gradients of ``rms_norm`` from its x and rstd; dx may be dy or x."""
    w = "armt_rms_norm_grad"
    t, n, d, dev = _matrix(w, "x", x)
    _tensor(w, "gain", gain, x.dtype, (d,), dev)
    _tensor(w, "rstd", rstd, torch.float32, (n,), dev)
    _tensor(w, "dy", dy, x.dtype, (n, d), dev)
    _tensor(w, "dx", dx, x.dtype, (n, d), dev)
    _tensor(w, "d_gain", d_gain, x.dtype, (d,), dev)
    same = [(k, u) for k, u in (("x", x), ("dy", dy)) if u.data_ptr() != dx.data_ptr()]
    _apart(w, [("dx", dx)], same + [("gain", gain), ("rstd", rstd), ("workspace", workspace)])
    _apart(w, [("d_gain", d_gain)], [("x", x), ("gain", gain), ("rstd", rstd), ("dy", dy), ("dx", dx),
                                     ("workspace", workspace)])
    with on_stream(stream, dev):
        at, size, keep = _space(w, "armt_rms_norm_grad_workspace", (t, n, d), workspace, dev,
                                [("x", x), ("gain", gain), ("rstd", rstd), ("dy", dy)])
        _check(lib().armt_rms_norm_grad(t, n, d, x.data_ptr(), gain.data_ptr(), rstd.data_ptr(), dy.data_ptr(),
                                        dx.data_ptr(), d_gain.data_ptr(), at, size, _handle(dev)), w)
    _written((dx, d_gain))


def _loss_args(w, hidden, head, targets):
    t, n, d, dev = _matrix(w, "hidden", hidden)
    if not isinstance(head, torch.Tensor) or head.dim() != 2:
        _bad(w, "head must be a 2-d tensor")
    _tensor(w, "head", head, hidden.dtype, (head.shape[0], d), dev)
    return t, n, head.shape[0], d, dev, _ids(w, "targets", targets, n, dev)


def token_loss(hidden, head, targets, loss, lse, scale: float = 1.0, workspace=None, stream=None):
    """Cross entropy of the logits scale * hidden @ head.T against targets, without
    keeping the logits: loss[i] = lse[i] - logit of the target; rows whose target is
    outside the vocabulary give 0 for both."""
    w = "armt_token_loss"
    t, n, vocab, d, dev, b = _loss_args(w, hidden, head, targets)
    _tensor(w, "loss", loss, torch.float32, (n,), dev)
    _tensor(w, "lse", lse, torch.float32, (n,), dev)
    inputs = [("hidden", hidden), ("head", head), ("targets", targets)]
    _apart(w, [("loss", loss), ("lse", lse)], inputs + [("workspace", workspace)])
    with on_stream(stream, dev):
        at, size, keep = _space(w, "armt_token_loss_workspace", (t, n, vocab, d, 0), workspace, dev, inputs)
        _check(lib().armt_token_loss(t, n, vocab, d, hidden.data_ptr(), head.data_ptr(), targets.data_ptr(), b, scale,
                                     loss.data_ptr(), lse.data_ptr(), at, size, _handle(dev)), w)
    _written((loss, lse))


def token_loss_grad(hidden, head, targets, lse, d_loss, d_hidden=None, d_head=None, scale: float = 1.0,
                    workspace=None, stream=None):
    """Gradients of sum(d_loss * loss) of ``token_loss`` (with its lse) to hidden and
    head; either result may be left out."""
    w = "armt_token_loss_grad"
    t, n, vocab, d, dev, b = _loss_args(w, hidden, head, targets)
    _tensor(w, "lse", lse, torch.float32, (n,), dev)
    _tensor(w, "d_loss", d_loss, torch.float32, (n,), dev)
    outs = []
    if d_hidden is not None:
        _tensor(w, "d_hidden", d_hidden, hidden.dtype, (n, d), dev)
        outs.append(("d_hidden", d_hidden))
    if d_head is not None:
        _tensor(w, "d_head", d_head, hidden.dtype, (vocab, d), dev)
        outs.append(("d_head", d_head))
    if not outs:
        _bad(w, "d_hidden or d_head must be given")
    inputs = [("hidden", hidden), ("head", head), ("targets", targets), ("lse", lse), ("d_loss", d_loss)]
    _apart(w, outs, inputs + [("workspace", workspace)])
    with on_stream(stream, dev):
        at, size, keep = _space(w, "armt_token_loss_workspace", (t, n, vocab, d, 1), workspace, dev, inputs)
        _check(lib().armt_token_loss_grad(t, n, vocab, d, hidden.data_ptr(), head.data_ptr(), targets.data_ptr(), b,
                                          scale, lse.data_ptr(), d_loss.data_ptr(),
                                          None if d_hidden is None else d_hidden.data_ptr(),
                                          None if d_head is None else d_head.data_ptr(), at, size, _handle(dev)), w)
    _written([x for _, x in outs])
