"""Python binding of the operators addressed by token ids: the C entry points
under the same names.

They work at the two ends of a model's arena: ``dp_embed_lookup`` reads the
embedding table in a weight replica, ``dp_embed_grad`` fills its gradient in a
rank's gradient arena, and ``dp_token_logprobs`` / ``dp_distill_loss`` with
their gradients form the loss, whose per-token weights are what the
token-weighted mean (``dp_reduce_scatter_mean(..., token_counts=...)``)
divides by.

A table is a 2-D view of an arena (``arena[off:off + vocab * dim].view(vocab,
dim)``); its rows, like those of every matrix here, may be strided.  As in the
rest of the binding the caller owns every buffer, the work is enqueued on the
current stream of the tensors' device (or ``stream``), and nothing
synchronises the host.
"""

import functools

import torch

from . import _native as N
from ._native import check, lib

_TYPES = {torch.float32: N.GRZ_F32, torch.bfloat16: N.GRZ_BF16}
_IDS = {torch.int32: 32, torch.int64: 64}
_F32, _I32 = torch.float32, torch.int32

# The smallest calls take a few microseconds on the device, about what the host
# needs for one launch, so the checks below use the cheapest accessors: device
# indices (-1 for the host) instead of device objects, and explanations only
# where a check has failed.  A torch without GPU support lacks the accessors of
# _C that _call uses, so they are looked up there.
_C = torch._C


def _device(t, name, dev=None):
    """Index of the tensor's GPU, which must be ``dev`` if that is given."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be on the GPU, not {t.device}")
    if dev is not None and at != dev:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on cuda:{dev}")
    return at


def _rows(t, name, dev, rows=None, cols=None, dtype=None):
    """(pointer, type, rows, columns, row stride) of a row matrix on GPU ``dev``."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _device(t, name, dev)
    shape, own = t.shape, t.dtype
    kind = _TYPES.get(own)
    if kind is None or (dtype is not None and own != dtype):
        raise TypeError(f"{name} has dtype {own}, expected {dtype or 'float32 or bfloat16'}")
    if len(shape) != 2:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected two dimensions")
    r, c = shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError(f"{name} has shape {tuple(shape)}, expected "
                         f"({'any' if rows is None else rows}, {'any' if cols is None else cols})")
    stride, inner = t.stride()
    if inner != 1 and c > 1:
        raise ValueError(f"{name}'s columns must be adjacent in memory (strides {t.stride()})")
    if r <= 1:
        stride = max(c, 1)
    elif stride < c:
        raise ValueError(f"{name}'s rows overlap (strides {t.stride()})")
    return t.data_ptr(), kind, r, c, stride


def _list(t, name, dev, dtype, *shape):
    """Pointer of a contiguous array, None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _device(t, name, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _ids(t, name, dev, *shape):
    """(pointer, bits) of a contiguous id array."""
    if t is None:
        return None, 32
    own = t.dtype if isinstance(t, torch.Tensor) else None
    bits = _IDS.get(own)
    if bits is None:
        raise TypeError(f"{name} must be an int32 or int64 tensor")
    return _list(t, name, dev, own, *shape), bits


def _call(name, dev, stream, *args):
    """Call entry point ``name`` with GPU ``dev`` current, on ``stream`` or its
    current stream."""
    if stream is None:
        handle = _C._cuda_getCurrentRawStream(dev)
    elif stream.device.index != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{dev}")
    else:
        handle = stream.cuda_stream
    fn = getattr(lib(), name)
    if _C._cuda_getDevice() == dev:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, handle)
    if status != N.GRZ_OK:
        check(name, status)


def dp_embed_lookup(table, ids, out, scale=1.0, stream=None):
    """``out[i] = scale * table[ids[i]]``; a row of zeros where the id is outside
    the table."""
    dev = _device(table, "table")
    tp, tt, vocab, dim, ts = _rows(table, "table", dev)
    op, ot, n, _, os_ = _rows(out, "out", dev, None, dim)
    ip, bits = _ids(ids, "ids", dev, n)
    _call("dp_embed_lookup", dev, stream, tp, tt, vocab, dim, ts, ip, bits, n, scale, op, ot,
          os_)


@functools.lru_cache(maxsize=1024)
def dp_embed_grad_workspace(n, vocab, dim):
    """Bytes of workspace ``dp_embed_grad`` needs for ``n`` ids."""
    return int(lib().dp_embed_grad_workspace(int(n), int(vocab), int(dim)))


def dp_embed_grad(dout, ids, dtable, workspace, scale=1.0, accumulate=False, stream=None):
    """``dtable[v] = scale * sum of dout[i] over ids[i] = v``, zeros in the rows no
    id names; with ``accumulate`` added to what the named rows hold
    (``GRZ_ACCUMULATE``).  ``workspace``: ``dp_embed_grad_workspace`` bytes of
    any type, 16-byte aligned."""
    dev = _device(dout, "dout")
    dp, dt, n, dim, ds = _rows(dout, "dout", dev)
    tp, tt, vocab, _, ts = _rows(dtable, "dtable", dev, None, dim)
    ip, bits = _ids(ids, "ids", dev, n)
    need = dp_embed_grad_workspace(n, vocab, dim)
    ws = None
    if need:
        if workspace is None:
            raise ValueError(f"dp_embed_grad needs {need} bytes of workspace")
        _device(workspace, "workspace", dev)
        have = workspace.numel() * workspace.element_size()
        if have < need or not workspace.is_contiguous():
            raise ValueError(f"the workspace must be {need} contiguous bytes; it holds {have}")
        ws = workspace.data_ptr()
    _call("dp_embed_grad", dev, stream, dp, dt, ds, ip, bits, n, vocab, dim, scale,
          N.GRZ_ACCUMULATE if accumulate else 0, ws, tp, tt, ts)


def dp_token_logprobs(logits, targets=None, logprob=None, entropy=None, top_ids=None,
                      top_logprobs=None, stream=None):
    """Log probabilities under ``softmax(logits[i])``: of ``targets[i]`` into
    ``logprob`` (0 where it names no token), the entropy into ``entropy``, and
    the tokens of the largest logits (ties by lower id) with their log
    probabilities into ``top_ids`` (int32) / ``top_logprobs``, both ``n x k``.
    Each output may be None."""
    dev = _device(logits, "logits")
    lp, lt, n, vocab, ls = _rows(logits, "logits", dev)
    ip, bits = _ids(targets, "targets", dev, n)
    top = 0
    if top_ids is not None or top_logprobs is not None:
        if not isinstance(top_ids, torch.Tensor) or top_ids.dim() != 2 or top_logprobs is None:
            raise ValueError("top_ids and top_logprobs come together, two dimensions each")
        top = top_ids.shape[1]
    _call("dp_token_logprobs", dev, stream, lp, lt, n, vocab, ls, ip, bits, top,
          _list(logprob, "logprob", dev, _F32, n), _list(entropy, "entropy", dev, _F32, n),
          _list(top_ids, "top_ids", dev, _I32, n, top),
          _list(top_logprobs, "top_logprobs", dev, _F32, n, top))


def dp_token_logprobs_grad(logits, targets, glogprob, gentropy, dlogits, logprob=None,
                           entropy=None, stream=None):
    """Gradient of ``dp_token_logprobs``' logprob and entropy with respect to the
    logits, for the incoming gradients ``glogprob`` and ``gentropy`` (either may
    be None for 0), optionally with both values from the same pass.
    ``dlogits`` may be ``logits`` itself."""
    dev = _device(logits, "logits")
    lp, lt, n, vocab, ls = _rows(logits, "logits", dev)
    ip, bits = _ids(targets, "targets", dev, n)
    gp, _, _, _, gs = _rows(dlogits, "dlogits", dev, n, vocab, logits.dtype)
    _call("dp_token_logprobs_grad", dev, stream, lp, lt, n, vocab, ls, ip, bits,
          _list(glogprob, "glogprob", dev, _F32, n),
          _list(gentropy, "gentropy", dev, _F32, n), _list(logprob, "logprob", dev, _F32, n),
          _list(entropy, "entropy", dev, _F32, n), gp, gs)


def _teacher(ids, teacher, dev, n):
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("teacher_ids must be a tensor of two dimensions")
    k = ids.shape[1]
    if not isinstance(teacher, torch.Tensor) or teacher.dtype not in _TYPES:
        raise TypeError("teacher_logits must be a float32 or bfloat16 tensor")
    ip, bits = _ids(ids, "teacher_ids", dev, n, k)
    return (ip, bits, _list(teacher, "teacher_logits", dev, teacher.dtype, n, k),
            _TYPES[teacher.dtype], k)


def dp_distill_loss(logits, teacher_ids, teacher_logits, loss, temperature=1.0, weights=None,
                    stream=None):
    """``loss[i] = weights[i] T^2 KL(p || q)``: p the softmax of row i's listed
    ``teacher_logits`` / T, q that of ``logits[i]`` / T over the vocabulary.
    Entries of ``teacher_ids`` that name no token are left out."""
    dev = _device(logits, "logits")
    lp, lt, n, vocab, ls = _rows(logits, "logits", dev)
    _call("dp_distill_loss", dev, stream, lp, lt, n, vocab, ls,
          *_teacher(teacher_ids, teacher_logits, dev, n), temperature,
          _list(weights, "weights", dev, _F32, n), _list(loss, "loss", dev, _F32, n))


def dp_distill_grad(logits, teacher_ids, teacher_logits, dlogits, temperature=1.0, weights=None,
                    grad_scale=1.0, loss=None, stream=None):
    """Gradient of ``grad_scale`` times the sum of ``dp_distill_loss``'s losses
    with respect to the logits, optionally with the losses from the same pass.
    ``dlogits`` may be ``logits`` itself."""
    dev = _device(logits, "logits")
    lp, lt, n, vocab, ls = _rows(logits, "logits", dev)
    gp, _, _, _, gs = _rows(dlogits, "dlogits", dev, n, vocab, logits.dtype)
    _call("dp_distill_grad", dev, stream, lp, lt, n, vocab, ls,
          *_teacher(teacher_ids, teacher_logits, dev, n), temperature,
          _list(weights, "weights", dev, _F32, n), grad_scale,
          _list(loss, "loss", dev, _F32, n), gp, gs)
