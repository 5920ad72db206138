"""Python binding of the norm and the clip over many tensors: the C entry points
under the same names.

For gradients that sit in no arena (an expert-parallel rank's own experts), alone or
beside an arena's: the arena's piece sums stand in front of the workspace (``lead``
of them) and the tensors' join them, so that one clip factor counts both::

    grads = TensorList([p.grad for p in experts])
    ws = torch.empty(dp_grad_sqnorm_tensors_workspace(grads, lead) // 8,
                     dtype=torch.float64, device=dev)
    dp_reduce_scatter_mean(arenas, buckets, chunk, mean, ws[:lead])
    dp_grad_sqnorm_tensors(grads, max_norm, ws, sqnorm, scale, lead=lead)
    zero1_adamw_gather(w, m, v, mean, buckets, nranks, chunk, scale, args, replicas)
    dp_grad_clip_tensors(grads, scale)

The factor has to be there before the arena's update; the step drivers form their
own, of the arena alone.  AdamW applies the factor it is given, so fp32 gradients that go
through ``zero1_adamw_step`` need no clip of their own.

As in the rest of the binding the caller owns every buffer, the work is enqueued on
the current stream of the tensors' device (or ``stream``), and nothing synchronises
the host.
"""

import functools

import torch

from . import _native as N
from ._native import check, lib
from .tokens import _TYPES, _call, _device


class TensorList:
    """A list of bfloat16 and float32 tensors of one GPU as the library takes it, made
    once for tensors that keep their memory (the list holds views of them; a storage
    that is resized under it is an error of the caller): making it takes the host about
    0.85 us a tensor.  Each tensor's elements must fill one run of memory, in any order of
    its dimensions."""

    def __init__(self, tensors):
        tensors = list(tensors)
        self.device = _device(tensors[0], "tensors[0]") if tensors else None
        self.views, entries = [], []
        for i, t in enumerate(tensors):
            if not isinstance(t, torch.Tensor) or t.get_device() != self.device:
                _device(t, f"tensors[{i}]", self.device)
            kind = _TYPES.get(t.dtype)
            if kind is None:
                raise TypeError(f"tensors[{i}] has dtype {t.dtype}, expected float32 or bfloat16")
            if not t.is_contiguous() and not _one_run(t):
                raise ValueError(f"tensors[{i}]'s elements lie apart in memory or over each "
                                 f"other (shape {tuple(t.shape)}, strides {t.stride()})")
            self.views.append(t.detach())
            entries.append((t.data_ptr(), t.numel(), kind))
        self.table = (N.Tensor * max(len(entries), 1))(*entries)
        self.pieces = lib().dp_tensor_pieces(self.table, len(entries))
        if self.pieces < 0:
            check("dp_tensor_pieces", -self.pieces)

    def __len__(self):
        return len(self.views)

    @functools.cached_property
    def layouts(self):
        """(shape, strides) of each tensor."""
        return [(t.shape, t.stride()) for t in self.views]


def _one_run(t):
    """Whether the elements fill one run of memory, each place once."""
    need = 1
    for size, stride in sorted(((s, d) for s, d in zip(t.shape, t.stride()) if s != 1),
                               key=lambda p: p[1]):
        if size and stride != need:
            return False
        need *= size
    return True


def _as_list(tensors):
    return tensors if isinstance(tensors, TensorList) else TensorList(tensors)


def dp_tensor_pieces(tensors):
    """Norm pieces of the tensors: ``GRZ_PIECE`` consecutive elements of one each."""
    return _as_list(tensors).pieces


def dp_grad_sqnorm_tensors_workspace(tensors, lead=0):
    """Bytes of workspace ``dp_grad_sqnorm_tensors`` needs (at least 8)."""
    tensors = _as_list(tensors)
    if lead < 0:
        raise ValueError("lead must not be negative")
    return max(8, int(lib().dp_grad_sqnorm_tensors_workspace(tensors.table, len(tensors),
                                                             int(lead))))


def _scalar(t, name, dev, dtype):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _device(t, name, dev)
    if t.dtype != dtype or t.numel() < 1:
        raise TypeError(f"{name} must hold a {dtype} value")
    return t.data_ptr()


def dp_grad_sqnorm_tensors(tensors, max_norm, workspace, sqnorm_out, clip_scale_out, lead=0,
                           stream=None):
    """Global squared norm (float64) and clip factor (float32) over the ``lead`` piece
    sums in front of the workspace and all elements of ``tensors`` (a ``TensorList``
    or tensors); the tensors' piece sums are left behind the ``lead``.
    ``workspace``: ``dp_grad_sqnorm_tensors_workspace`` bytes of any type, 8-byte
    aligned."""
    tensors = _as_list(tensors)
    dev = tensors.device if tensors.device is not None else _device(workspace, "workspace")
    if not isinstance(workspace, torch.Tensor) or workspace.get_device() != dev:
        _device(workspace, "workspace", dev)
    need = lib().dp_grad_sqnorm_tensors_workspace(tensors.table, len(tensors), lead)
    have = workspace.numel() * workspace.element_size()
    if have < need or not workspace.is_contiguous():
        raise ValueError(f"the workspace must be {need} contiguous bytes; it holds {have}")
    _call("dp_grad_sqnorm_tensors", dev, stream, tensors.table, len(tensors), max_norm, lead,
          workspace.data_ptr(), _scalar(sqnorm_out, "sqnorm_out", dev, torch.float64),
          _scalar(clip_scale_out, "clip_scale_out", dev, torch.float32))


def dp_grad_clip_tensors(tensors, clip_scale, out=None, stream=None):
    """``clip_scale * t`` of each tensor (a ``TensorList`` or tensors), in place or into
    ``out``'s, of the same shapes, strides and order (types may differ).
    ``clip_scale``: a float32 device scalar, or None for 1."""
    tensors = _as_list(tensors)
    table = None
    if out is not None:
        out = _as_list(out)
        if out.layouts != tensors.layouts:
            _check_layouts(tensors, out)
        if out.device != tensors.device:
            raise ValueError("out is on another device than the tensors")
        table = out.table
    if not len(tensors):
        return
    dev = tensors.device
    _call("dp_grad_clip_tensors", dev, stream, tensors.table, len(tensors),
          _scalar(clip_scale, "clip_scale", dev, torch.float32), table)


def _check_layouts(tensors, out):
    if len(tensors) != len(out):
        raise ValueError(f"{len(tensors)} tensors, {len(out)} outputs")
    for i, ((s, d), (so, do)) in enumerate(zip(tensors.layouts, out.layouts)):
        if s != so:
            raise ValueError(f"out[{i}] has shape {tuple(so)}, tensors[{i}] {tuple(s)}")
        # Strides count only where there is more than one element along them.
        if any(a != b for n, a, b in zip(s, d, do) if n > 1) and 0 not in s:
            raise ValueError(f"out[{i}] has strides {do}, tensors[{i}] {d}")
