"""Python binding of the mixture-of-experts operators: the C entry points under the
same names.

The way of n tokens to k experts each and back::

    dp_expert_route(logits, ids, weights, normalize=True)
    dp_expert_sort(ids, experts, offsets, places, workspace)
    dp_expert_dispatch(x, places, rows)
    # y[r]: expert e's output for rows[r], offsets[e] <= r < offsets[e + 1]
    dp_expert_combine(y, places, out, weights=weights)

and the gradients'::

    dp_expert_combine_grad(dout, y, places, weights, dy=dy, dweights=dweights)
    # drows[r]: the experts' gradient for dy[r]
    dp_expert_combine(drows, places, dx)
    dp_expert_route_grad(logits, ids, dweights, dlogits, normalize=True)

``ids`` and ``places`` are ``n x k``, weights and their gradients float32 of that
shape, all contiguous; matrices may have any row stride.  As in the rest of the
binding the caller owns every buffer, the work is enqueued on the current stream of
the tensors' device (or ``stream``), and nothing synchronises the host.
"""

import functools

import torch

from . import _native as N
from ._native import lib
from .tokens import _F32, _I32, _call, _device, _ids, _list, _rows


def _slots(t, name, dev, dtype, n):
    """(pointer, k) of a contiguous array of ``n`` tokens' slots."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _device(t, name, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[0] != n:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected ({n}, any)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr(), shape[1]


def dp_expert_route(logits, ids, weights, normalize=False, stream=None):
    """The experts with each token's ``k`` largest logits (ties by lower id) into
    ``ids`` (int32, ``n x k``) and their softmax weights into ``weights``; with
    ``normalize`` each token's weights sum to 1 (``GRZ_NORMALIZE``).  Experts whose
    logit is -inf are closed: slots left over have id -1 and weight 0."""
    dev = _device(logits, "logits")
    lp, lt, n, experts, ls = _rows(logits, "logits", dev)
    ip, k = _slots(ids, "ids", dev, _I32, n)
    _call("dp_expert_route", dev, stream, lp, lt, n, experts, ls, k,
          N.GRZ_NORMALIZE if normalize else 0, ip, _list(weights, "weights", dev, _F32, n, k))


def dp_expert_route_grad(logits, ids, dweights, dlogits, normalize=False, stream=None):
    """Gradient of ``dp_expert_route``'s weights with respect to the logits, for the
    listed ``ids``.  ``dlogits`` may be ``logits`` itself."""
    dev = _device(logits, "logits")
    lp, lt, n, experts, ls = _rows(logits, "logits", dev)
    ip, k = _slots(ids, "ids", dev, _I32, n)
    gp, _, _, _, gs = _rows(dlogits, "dlogits", dev, n, experts, logits.dtype)
    _call("dp_expert_route_grad", dev, stream, lp, lt, n, experts, ls, k,
          N.GRZ_NORMALIZE if normalize else 0, ip,
          _list(dweights, "dweights", dev, _F32, n, k), gp, gs)


@functools.lru_cache(maxsize=1024)
def dp_expert_sort_workspace(n, k, experts):
    """Bytes of workspace ``dp_expert_sort`` needs for ``n`` tokens of ``k`` slots."""
    return int(lib().dp_expert_sort_workspace(int(n), int(k), int(experts)))


def dp_expert_sort(ids, experts, offsets, places, workspace=None, stream=None):
    """Rows of the slots sorted by expert, stable, into ``places`` (int32, -1 where
    the id names no expert), and the experts' first rows into ``offsets`` (int32,
    ``experts + 1``).  ``workspace``: ``dp_expert_sort_workspace`` bytes of any type,
    4-byte aligned, or None where it needs none."""
    dev = _device(ids, "ids")
    if ids.dim() != 2:
        raise ValueError(f"ids has shape {tuple(ids.shape)}, expected tokens x slots")
    n, k = ids.shape
    ip, bits = _ids(ids, "ids", dev, n, k)
    need = dp_expert_sort_workspace(n, k, experts)
    ws = None
    if need:
        if workspace is None:
            raise ValueError(f"dp_expert_sort needs {need} bytes of workspace")
        _device(workspace, "workspace", dev)
        have = workspace.numel() * workspace.element_size()
        if have < need or not workspace.is_contiguous():
            raise ValueError(f"the workspace must be {need} contiguous bytes; it holds {have}")
        ws = workspace.data_ptr()
    if offsets is None or places is None:
        raise TypeError("offsets and places must be tensors")
    _call("dp_expert_sort", dev, stream, ip, bits, n, k, experts, ws,
          _list(offsets, "offsets", dev, _I32, experts + 1),
          _list(places, "places", dev, _I32, n, k))


def dp_expert_dispatch(x, places, out, weights=None, stream=None):
    """``out[places[i, j]] = weights[i, j] * x[i]`` (``x[i]`` without weights); rows
    that no place names are left as they were."""
    dev = _device(x, "x")
    xp, xt, n, dim, xs = _rows(x, "x", dev)
    pp, k = _slots(places, "places", dev, _I32, n)
    op, ot, rows, _, os_ = _rows(out, "out", dev, None, dim)
    _call("dp_expert_dispatch", dev, stream, xp, xt, xs, pp,
          _list(weights, "weights", dev, _F32, n, k), n, k, dim, rows, op, ot, os_)


def dp_expert_combine(y, places, out, weights=None, accumulate=False, stream=None):
    """``out[i] = sum over j of weights[i, j] * y[places[i, j]]`` (of the rows without
    weights: the gradient of ``dp_expert_dispatch``); with ``accumulate`` added to
    what ``out`` holds (``GRZ_ACCUMULATE``)."""
    dev = _device(y, "y")
    yp, yt, rows, dim, ys = _rows(y, "y", dev)
    op, ot, n, _, os_ = _rows(out, "out", dev, None, dim)
    pp, k = _slots(places, "places", dev, _I32, n)
    _call("dp_expert_combine", dev, stream, yp, yt, ys, rows, pp,
          _list(weights, "weights", dev, _F32, n, k), n, k, dim,
          N.GRZ_ACCUMULATE if accumulate else 0, op, ot, os_)


def dp_expert_combine_grad(dout, y, places, weights, dy=None, dweights=None, stream=None):
    """Gradient of ``dp_expert_combine``: ``dy[places[i, j]] = weights[i, j] *
    dout[i]`` (1 for ``weights`` None) and ``dweights[i, j] = <dout[i],
    y[places[i, j]]>``.  Either output may be None; ``dy`` may be ``y`` itself, and
    ``y`` None where ``dweights`` is."""
    dev = _device(dout, "dout")
    dp, dt, n, dim, ds = _rows(dout, "dout", dev)
    pp, k = _slots(places, "places", dev, _I32, n)
    if y is not None:
        yp, yt, rows, _, ys = _rows(y, "y", dev, None, dim)
    elif dweights is not None or dy is None:
        raise ValueError("dweights needs y, and the call an output")
    gp = gs = None
    if dy is not None:
        gp, gt, grows, _, gs = _rows(dy, "dy", dev, None if y is None else rows, dim,
                                     None if y is None else y.dtype)
    if y is None:
        yp, yt, rows, ys = None, gt, grows, dim
    _call("dp_expert_combine_grad", dev, stream, dp, dt, ds, yp, yt, ys, rows, pp,
          _list(weights, "weights", dev, _F32, n, k), n, k, dim, gp, gs or 0,
          _list(dweights, "dweights", dev, _F32, n, k))
