"""The two ends of a language model and the clip between the reduction and the
optimizer: plumbing over ddp_clip_grads, ddp_embedding_* and ddp_vocab_loss_*.

Each object keeps what a program keeps from step to step (sizes, pointer tables)
and forwards to the library, which does all of the work.  Calls run on `stream`
(default: torch's current stream).  Scratch memory is taken from torch's
allocator for the length of a call, on the stream that the call runs on, and so
are outputs that the caller does not pass.
"""
from __future__ import annotations

import math

import numpy as np

from . import (DDP_BF16, DDP_CLIP_WORKSPACE_BYTES, DDP_F16, DDP_F32, DDP_NORM_INF, DDP_NORM_L2, ddp_clip_grads,
               ddp_embedding_backward, ddp_embedding_forward, ddp_embedding_workspace, ddp_grad_norm,
               ddp_vocab_loss_backward, ddp_vocab_loss_forward, ddp_vocab_loss_workspace)


def _dtype(t) -> int:
    import torch

    try:
        return {torch.float32: DDP_F32, torch.bfloat16: DDP_BF16, torch.float16: DDP_F16}[t]
    except KeyError:
        raise ValueError(f"dtype {t} is not float32, bfloat16 or float16") from None


def _on(stream):
    """Allocations and the call on the same stream."""
    import contextlib

    import torch

    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _raw(stream, device) -> int:
    import torch

    return (torch.cuda.current_stream(device) if stream is None else stream).cuda_stream


def _rows(x, name, rows, dim, dtypes):
    """x as a [rows, dim] matrix with contiguous rows; its row stride."""
    if x.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {x.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if not x.is_cuda:
        raise ValueError(f"{name} is not on the GPU")
    if x.dim() != 2 or x.shape[0] != rows or x.shape[1] != dim or (dim > 1 and x.stride(1) != 1) or \
            (rows > 1 and x.stride(0) < dim):
        raise ValueError(f"{name} must be [{rows}, {dim}] with contiguous rows, got shape {tuple(x.shape)} and "
                         f"strides {x.stride()}")
    return x.stride(0) if rows > 1 else dim


def _ids(x, name):
    import torch

    if x.dtype not in (torch.int64, torch.int32) or not x.is_cuda:
        raise ValueError(f"{name} must be int32 or int64 on the GPU")
    if x.dim() != 1 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector, got shape {tuple(x.shape)}")
    return x.element_size()


class GradClipper:
    """The global norm of a list of gradient tensors, and clipping by it.

    grads      contiguous fp32 / bf16 / fp16 tensors on the GPU (types may be mixed;
               None: the parameter has no gradient).  Their addresses are read once:
               the tensors must keep their storage.
    out        tensors receiving the clipped gradients (None: in place).
    norm_type  2 or inf.
    """

    def __init__(self, grads, out=None, norm_type=2.0):
        import torch

        if norm_type not in (2, 2.0, math.inf):
            raise ValueError(f"norm_type {norm_type} is neither 2 nor inf")
        self.norm_type = DDP_NORM_INF if norm_type == math.inf else DDP_NORM_L2
        if out is not None and len(out) != len(grads):
            raise ValueError(f"{len(out)} outputs for {len(grads)} gradients")
        given = [g for g in grads if g is not None]
        for k, g in enumerate(grads):
            o = None if out is None else out[k]
            if g is None:
                if o is not None:
                    raise ValueError(f"gradient {k} is None and has an output")
                continue
            _dtype(g.dtype)
            if not g.is_cuda or not g.is_contiguous():
                raise ValueError(f"gradient {k} is not a contiguous tensor on the GPU")
            if o is not None and (o.dtype != g.dtype or o.numel() != g.numel() or not o.is_cuda
                                  or not o.is_contiguous()):
                raise ValueError(f"output {k} is not a contiguous {g.dtype} tensor of {g.numel()} elements on the GPU")
        dev = given[0].device if given else torch.device("cuda")
        self._tensors = (grads, out)   # the pointer tables below point into these
        n = [0 if g is None else g.numel() for g in grads]
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
        self.total, self.ntensors = int(off[-1]), len(grads)

        def table(ts):
            return torch.from_numpy(np.array([0 if t is None else t.data_ptr() for t in ts] or [0], np.int64)).to(dev)

        self.grads_tab = table(grads)
        self.out_tab = None if out is None else table(out)
        self.offset = torch.from_numpy(off).to(dev)
        self.dtypes = torch.from_numpy(np.array([DDP_F32 if g is None else _dtype(g.dtype) for g in grads] or [0],
                                                np.int32)).to(dev)
        self.device = dev

    @classmethod
    def of_reducer(cls, reducer, w=0, norm_type=2.0):
        """Over replica w's reduced gradients: the views of a BucketReducer's main_grad."""
        return cls([reducer.view(p, w) for p in range(reducer.plan.nparams)], norm_type=norm_type)

    def _call(self, clip, max_norm, stream):
        import torch

        with _on(stream):
            norm = torch.empty(1, dtype=torch.float32, device=self.device)
            ws = torch.empty(DDP_CLIP_WORKSPACE_BYTES, dtype=torch.uint8, device=self.device)
            if clip:
                ddp_clip_grads(self.grads_tab, self.out_tab, self.offset, self.dtypes, self.ntensors, self.total,
                               self.norm_type, float(max_norm), norm, ws, DDP_CLIP_WORKSPACE_BYTES,
                               _raw(stream, self.device))
            else:
                ddp_grad_norm(self.grads_tab, self.offset, self.dtypes, self.ntensors, self.total, self.norm_type,
                              norm, ws, DDP_CLIP_WORKSPACE_BYTES, _raw(stream, self.device))
        return norm

    def norm(self, stream=None):
        """The global norm, as a one-element tensor."""
        return self._call(False, 0.0, stream)

    def clip(self, max_norm, stream=None):
        """Scale the gradients by min(1, max_norm / (norm + 1e-6)); returns the norm
        before clipping, as a one-element tensor."""
        return self._call(True, max_norm, stream)


class TokenEmbedding:
    """Lookup in a [vocab, dim] table with a scale, and the table's gradient."""

    def __init__(self, vocab, dim, dtype, scale=1.0, padding_idx=None):
        self.vocab, self.dim, self.torch_dtype, self.dtype = int(vocab), int(dim), dtype, _dtype(dtype)
        self.scale = float(scale)
        self.padding_idx = -1 if padding_idx is None else int(padding_idx)

    def forward(self, weight, ids, out=None, stream=None):
        """out[t] = scale * weight[ids[t]], a [tokens, dim] tensor."""
        import torch

        n = ids.numel()
        id_bytes = _ids(ids, "ids")
        ws = _rows(weight, "weight", self.vocab, self.dim, (self.torch_dtype,))
        with _on(stream):
            if out is None:
                out = torch.empty((n, self.dim), dtype=self.torch_dtype, device=weight.device)
            ddp_embedding_forward(weight, ws, self.dtype, self.vocab, self.dim, ids, id_bytes, n, self.scale, out,
                                  _rows(out, "out", n, self.dim, (self.torch_dtype,)), _raw(stream, weight.device))
        return out

    def backward(self, grad_out, ids, grad_weight=None, accumulate=False, stream=None):
        """The gradient of the table, [vocab, dim]; with accumulate it is added to
        grad_weight (of dtype, or float32: a main_grad view)."""
        import torch

        n = ids.numel()
        id_bytes = _ids(ids, "ids")
        gs = _rows(grad_out, "grad_out", n, self.dim, (self.torch_dtype,))
        with _on(stream):
            if grad_weight is None:
                if accumulate:
                    raise ValueError("accumulate needs a grad_weight")
                grad_weight = torch.empty((self.vocab, self.dim), dtype=self.torch_dtype, device=grad_out.device)
            gws = _rows(grad_weight, "grad_weight", self.vocab, self.dim, (self.torch_dtype, torch.float32))
            size = ddp_embedding_workspace(n, self.vocab, self.dim)
            ws = torch.empty(size, dtype=torch.uint8, device=grad_out.device)
            ddp_embedding_backward(grad_out, gs, self.dtype, ids, id_bytes, n, self.scale, self.padding_idx,
                                   self.vocab, self.dim, grad_weight, gws, _dtype(grad_weight.dtype), accumulate, ws,
                                   size, _raw(stream, grad_out.device))
        return grad_weight


class VocabLoss:
    """Softmax cross entropy of hidden states against a [vocab, dim] projection.

    piece  words of the vocabulary whose softmax gradient is held at a time by the
           backward pass (0: the library's choice); its memory is
           2 * piece * tokens bytes.
    """

    def __init__(self, vocab, dim, dtype, ignore_index=-100, piece=0):
        self.vocab, self.dim, self.torch_dtype, self.dtype = int(vocab), int(dim), dtype, _dtype(dtype)
        if self.dtype == DDP_F32:
            raise ValueError("the vocabulary loss takes bfloat16 or float16 inputs")
        self.ignore_index, self.piece = int(ignore_index), int(piece)
        self._sizes = {}

    def _workspace(self, n, weight, ws):
        aligned = weight.data_ptr() % 16 == 0 and ws % 8 == 0
        key = (n, aligned)
        if key not in self._sizes:
            if len(self._sizes) > 64:
                self._sizes.clear()
            self._sizes[key] = ddp_vocab_loss_workspace(n, self.vocab, self.dim, self.piece, aligned)
        return self._sizes[key]

    def _inputs(self, hidden, weight, targets):
        n = targets.numel()
        id_bytes = _ids(targets, "targets")
        hs = _rows(hidden, "hidden", n, self.dim, (self.torch_dtype,))
        ws = _rows(weight, "weight", self.vocab, self.dim, (self.torch_dtype,))
        return n, id_bytes, hs, ws

    def forward(self, hidden, weight, targets, stream=None):
        """(loss, lse) of each token, float32; both 0 where the target is ignore_index."""
        import torch

        n, id_bytes, hs, ws = self._inputs(hidden, weight, targets)
        size = self._workspace(n, weight, ws)[0]
        with _on(stream):
            both = torch.empty((2, n), dtype=torch.float32, device=weight.device)
            scratch = torch.empty(size, dtype=torch.uint8, device=weight.device)
            loss, lse = both[0], both[1]
            ddp_vocab_loss_forward(hidden, hs, weight, ws, self.dtype, n, self.vocab, self.dim, targets, id_bytes,
                                   self.ignore_index, loss, lse, scratch, size, _raw(stream, weight.device))
        return loss, lse

    def backward(self, hidden, weight, targets, lse, grad_loss, grad_hidden=None, grad_weight=None, accumulate=False,
                 need_hidden=True, need_weight=True, stream=None):
        """(grad_hidden, grad_weight) of sum(grad_loss * loss).  grad_loss: float32,
        one value a token, or one value for all of them.  With accumulate the
        weight's gradient is added to grad_weight (of dtype, or float32: a
        main_grad view)."""
        import torch

        n, id_bytes, hs, ws = self._inputs(hidden, weight, targets)
        for x, name in ((lse, "lse"), (grad_loss, "grad_loss")):
            if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
                raise ValueError(f"{name} must be a contiguous float32 tensor on the GPU")
        if lse.numel() != n:
            raise ValueError(f"lse has {lse.numel()} elements for {n} tokens")
        if grad_loss.numel() not in (1, n):
            raise ValueError(f"grad_loss has {grad_loss.numel()} elements for {n} tokens")
        size = self._workspace(n, weight, ws)[1]
        with _on(stream):
            ghs = gws = self.dim
            if need_hidden:
                if grad_hidden is None:
                    grad_hidden = torch.empty((n, self.dim), dtype=self.torch_dtype, device=weight.device)
                ghs = _rows(grad_hidden, "grad_hidden", n, self.dim, (self.torch_dtype,))
            if need_weight:
                if grad_weight is None:
                    if accumulate:
                        raise ValueError("accumulate needs a grad_weight")
                    grad_weight = torch.empty((self.vocab, self.dim), dtype=self.torch_dtype, device=weight.device)
                gws = _rows(grad_weight, "grad_weight", self.vocab, self.dim, (self.torch_dtype, torch.float32))
            scratch = torch.empty(size, dtype=torch.uint8, device=weight.device)
            ddp_vocab_loss_backward(hidden, hs, weight, ws, self.dtype, n, self.vocab, self.dim, targets, id_bytes,
                                    self.ignore_index, lse, grad_loss, int(grad_loss.numel() == n and n != 1),
                                    grad_hidden if need_hidden else None, ghs, grad_weight if need_weight else None,
                                    gws, _dtype(grad_weight.dtype) if need_weight else self.dtype, accumulate,
                                    self.piece, scratch, size, _raw(stream, weight.device))
        return (grad_hidden if need_hidden else None), (grad_weight if need_weight else None)
