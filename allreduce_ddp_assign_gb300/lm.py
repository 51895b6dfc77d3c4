"""The two ends of a language model and the clip between the reduction and the
optimizer: plumbing over ddp_clip_grads, ddp_embedding_* and ddp_vocab_loss_*.

Each object keeps what a program keeps from step to step (sizes, pointer tables)
and forwards to the library, which does all of the work.  Calls run on `stream`
(default: torch's current stream).  Scratch memory is taken from torch's
allocator for the length of a call, on the stream that the call runs on, and so
are outputs that the caller does not pass.  Tensors passed to a call with `stream`
may be dropped when it returns: the allocator is told of their use there.  (As
everywhere in torch, `stream` does not wait for the work that fills them, and
outputs belong to the stream that they were made on.)  Everything lies on the
current device, where the library launches; other tensors are refused.

The smallest calls take a few microseconds on the GPU, so little is done on the
way there: attributes are read once, and addresses go to the library as integers.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import (DDP_ALLREDUCE, DDP_BF16, DDP_CLIP_WORKSPACE_BYTES, DDP_F16, DDP_F32, DDP_NORM_INF, DDP_NORM_L2, _check,
               lib, ddp_embedding_workspace, ddp_vocab_loss_workspace)

try:
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:  # pragma: no cover - another torch
    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream

try:
    from torch._C import _cuda_getDevice as _current_device
except ImportError:  # pragma: no cover - another torch
    from torch.cuda import current_device as _current_device

_DTYPES = {torch.float32: DDP_F32, torch.bfloat16: DDP_BF16, torch.float16: DDP_F16}


def _dtype(t) -> int:
    try:
        return _DTYPES[t]
    except KeyError:
        raise ValueError(f"dtype {t} is not float32, bfloat16 or float16") from None


def _here(x, name) -> None:
    """x lies on the current device, where the library launches."""
    at = x.get_device()   # -1: not on a GPU
    if at < 0:
        raise ValueError(f"{name} is not on the GPU")
    if at != _current_device():
        raise ValueError(f"{name} is on {x.device}, the current device is cuda:{_current_device()}")


def _rows(x, name, rows, dim, dtypes) -> int:
    """x as a [rows, dim] matrix with contiguous rows on the GPU; its row stride."""
    if x.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {x.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    _here(x, name)
    if x.dim() == 2:
        r, c = x.shape
        s, one = x.stride()
        if r == rows and c == dim and (one == 1 or dim == 1) and (s >= dim or rows <= 1):
            return s if rows > 1 else dim
    raise ValueError(f"{name} must be [{rows}, {dim}] with contiguous rows, got shape {tuple(x.shape)} and "
                     f"strides {x.stride()}")


def _ids(x, name) -> int:
    """Bytes of an id."""
    size = {torch.int64: 8, torch.int32: 4}.get(x.dtype)
    if size is None:
        raise ValueError(f"{name} must be int32 or int64 on the GPU")
    _here(x, name)
    if x.dim() != 1 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector, got shape {tuple(x.shape)}")
    return size


def _lend(stream, *tensors) -> None:
    """Memory of these tensors, allocated on other streams, is in use on this one: it is not
    given away before the work queued here, whatever becomes of the tensors."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _floats(x, name) -> None:
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor on the GPU")
    _here(x, name)


class GradClipper:
    """The global norm of a list of gradient tensors, and clipping by it.

    grads      contiguous fp32 / bf16 / fp16 tensors on the GPU (types may be mixed;
               None: the parameter has no gradient).  Their addresses are read once:
               the tensors must keep their storage.
    out        tensors receiving the clipped gradients (None: in place).
    norm_type  2 or inf.

    Making one builds the tables of addresses and copies them to the GPU, which waits for
    the copy: it pays where the gradients keep their storage (main_grad views), once for
    many steps, and costs about as much as a call where they are made anew each step.
    """

    def __init__(self, grads, out=None, norm_type=2.0):
        # (lists of its own: the tables below keep pointing at these tensors whatever becomes of the caller's)
        grads, out = tuple(grads), None if out is None else tuple(out)
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
            _here(g, f"gradient {k}")
            if o is not None and (o.dtype != g.dtype or o.numel() != g.numel() or not o.is_cuda
                                  or not o.is_contiguous()):
                raise ValueError(f"output {k} is not a contiguous {g.dtype} tensor of {g.numel()} elements on the GPU")
            if o is not None:
                _here(o, f"output {k}")
        self.device = given[0].device if given else torch.device("cuda", torch.cuda.current_device())
        self._tensors = (grads, out)   # the pointer tables below point into these
        n = [0 if g is None else g.numel() for g in grads]
        off = np.concatenate([[0], np.cumsum(n)]).astype(np.int64)
        self.total, self.ntensors = int(off[-1]), len(grads)

        def table(ts):
            return np.array([0 if t is None else t.data_ptr() for t in ts], np.int64)

        # one device buffer: offsets, addresses, the outputs' addresses, types
        types = np.array([DDP_F32 if g is None else _dtype(g.dtype) for g in grads] + [0] * (len(grads) & 1), np.int32)
        parts = [off, table(grads), table(out or []), types.view(np.int64)]
        self._tables = torch.from_numpy(np.concatenate(parts)).to(self.device)
        at = self._tables.data_ptr() + 8 * np.cumsum([0] + [len(p) for p in parts])
        self.offset, self.grads_tab, out_tab, self.dtypes = (int(a) for a in at[:4])
        self.out_tab = None if out is None else out_tab
        self._streams = {_raw_stream(self.device.index)}   # those on which the allocator knows the memory in use

    @classmethod
    def of_reducer(cls, reducer, w=0, norm_type=2.0):
        """Over replica w's reduced gradients: the views of an all-reducing BucketReducer's main_grad."""
        if reducer.mode != DDP_ALLREDUCE:
            # the rest of its main_grad is not written by the reduction, and a norm over the shard is not the model's
            raise ValueError("after a reduce-scatter a replica holds only its own shard of the reduced gradients")
        if reducer.main_grad is None:
            raise ValueError("the reducer keeps no main_grad")
        return cls([reducer.view(p, w) for p in range(reducer.plan.nparams)], norm_type=norm_type)

    def _stream(self):
        """The current stream's handle.  The tables were allocated on the stream that was current when they
        were made; on another one the allocator has to learn of their use, or it gives their memory away, while
        the kernels still read it, when the object and its tensors are dropped."""
        if self.device.index != _current_device():
            raise ValueError(f"the gradients are on {self.device}, the current device is cuda:{_current_device()}")
        raw = _raw_stream(self.device.index)
        if raw not in self._streams:
            _lend(torch.cuda.current_stream(self.device), self._tables, *self._tensors[0], *(self._tensors[1] or ()))
            self._streams.add(raw)
        return raw

    def norm(self, stream=None):
        """The global norm, as a one-element tensor."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.norm()
        on = self._stream()
        norm = torch.empty(1, dtype=torch.float32, device=self.device)
        ws = torch.empty(DDP_CLIP_WORKSPACE_BYTES, dtype=torch.uint8, device=self.device)
        _check(lib().ddp_grad_norm(self.grads_tab, self.offset, self.dtypes, self.ntensors, self.total, self.norm_type,
                                   norm.data_ptr(), ws.data_ptr(), DDP_CLIP_WORKSPACE_BYTES, on))
        return norm

    def clip(self, max_norm, stream=None):
        """Scale the gradients by min(1, max_norm / (norm + 1e-6)); returns the norm
        before clipping, as a one-element tensor."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.clip(max_norm)
        on = self._stream()
        norm = torch.empty(1, dtype=torch.float32, device=self.device)
        ws = torch.empty(DDP_CLIP_WORKSPACE_BYTES, dtype=torch.uint8, device=self.device)
        _check(lib().ddp_clip_grads(self.grads_tab, self.out_tab, self.offset, self.dtypes, self.ntensors, self.total,
                                    self.norm_type, max_norm, norm.data_ptr(), ws.data_ptr(),
                                    DDP_CLIP_WORKSPACE_BYTES, on))
        return norm


class TokenEmbedding:
    """Lookup in a [vocab, dim] table with a scale, and the table's gradient.

    padding_idx  the id whose row gets no gradient (None or negative: none).
    """

    def __init__(self, vocab, dim, dtype, scale=1.0, padding_idx=None):
        self.vocab, self.dim, self.torch_dtype, self.dtype = int(vocab), int(dim), dtype, _dtype(dtype)
        self.scale = float(scale)
        self.padding_idx = -1 if padding_idx is None else int(padding_idx)
        self._same = (dtype,)
        self._wide = (dtype, torch.float32)

    def forward(self, weight, ids, out=None, stream=None):
        """out[t] = scale * weight[ids[t]], a [tokens, dim] tensor."""
        if stream is not None:
            with torch.cuda.stream(stream):
                res = self.forward(weight, ids, out)
            _lend(stream, weight, ids, out)
            return res
        n, dim = ids.numel(), self.dim
        id_bytes = _ids(ids, "ids")
        ws = _rows(weight, "weight", self.vocab, dim, self._same)
        if out is None:
            out, stride = torch.empty((n, dim), dtype=self.torch_dtype, device=weight.device), dim
        else:
            stride = _rows(out, "out", n, dim, self._same)
        _check(lib().ddp_embedding_forward(weight.data_ptr(), ws, self.dtype, self.vocab, dim, ids.data_ptr(), id_bytes,
                                           n, self.scale, out.data_ptr(), stride, _raw_stream(weight.get_device())))
        return out

    def backward(self, grad_out, ids, grad_weight=None, accumulate=False, stream=None):
        """The gradient of the table, [vocab, dim]; with accumulate it is added to
        grad_weight (of dtype, or float32: a main_grad view)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                res = self.backward(grad_out, ids, grad_weight, accumulate)
            _lend(stream, grad_out, ids, grad_weight)
            return res
        n, dim = ids.numel(), self.dim
        id_bytes = _ids(ids, "ids")
        gs = _rows(grad_out, "grad_out", n, dim, self._same)
        if grad_weight is None:
            if accumulate:
                raise ValueError("accumulate needs a grad_weight")
            grad_weight = torch.empty((self.vocab, dim), dtype=self.torch_dtype, device=grad_out.device)
            gws = dim
        else:
            gws = _rows(grad_weight, "grad_weight", self.vocab, dim, self._wide)
        size = ddp_embedding_workspace(n, self.vocab, dim)
        ws = torch.empty(size, dtype=torch.uint8, device=grad_out.device)
        _check(lib().ddp_embedding_backward(grad_out.data_ptr(), gs, self.dtype, ids.data_ptr(), id_bytes, n, self.scale,
                                            self.padding_idx, self.vocab, dim, grad_weight.data_ptr(), gws,
                                            _DTYPES[grad_weight.dtype], int(accumulate), ws.data_ptr(), size,
                                            _raw_stream(grad_out.get_device())))
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
        self._same = (dtype,)
        self._wide = (dtype, torch.float32)
        self._sizes = {}

    def _inputs(self, hidden, weight, targets):
        n = targets.numel()
        id_bytes = _ids(targets, "targets")
        hs = _rows(hidden, "hidden", n, self.dim, self._same)
        ws = _rows(weight, "weight", self.vocab, self.dim, self._same)
        at = weight.data_ptr()
        key = n, at % 16 == 0 and ws % 8 == 0
        sizes = self._sizes.get(key)
        if sizes is None:
            if len(self._sizes) >= 64:
                self._sizes.clear()
            sizes = self._sizes[key] = ddp_vocab_loss_workspace(n, self.vocab, self.dim, self.piece, key[1])
        return n, id_bytes, hs, ws, at, sizes

    def forward(self, hidden, weight, targets, stream=None):
        """(loss, lse) of each token, float32; both 0 where the target is ignore_index."""
        if stream is not None:
            with torch.cuda.stream(stream):
                res = self.forward(hidden, weight, targets)
            _lend(stream, hidden, weight, targets)
            return res
        n, id_bytes, hs, ws, at, (size, _) = self._inputs(hidden, weight, targets)
        both = torch.empty((2, n), dtype=torch.float32, device=weight.device)
        scratch = torch.empty(size, dtype=torch.uint8, device=weight.device)
        loss, lse = both[0], both[1]
        _check(lib().ddp_vocab_loss_forward(hidden.data_ptr(), hs, at, ws, self.dtype, n, self.vocab, self.dim,
                                            targets.data_ptr(), id_bytes, self.ignore_index, loss.data_ptr(),
                                            lse.data_ptr(), scratch.data_ptr(), size,
                                            _raw_stream(weight.get_device())))
        return loss, lse

    def backward(self, hidden, weight, targets, lse, grad_loss, grad_hidden=None, grad_weight=None, accumulate=False,
                 need_hidden=True, need_weight=True, stream=None):
        """(grad_hidden, grad_weight) of sum(grad_loss * loss).  grad_loss: float32,
        one value a token, or one value for all of them.  With accumulate the
        weight's gradient is added to grad_weight (of dtype, or float32: a
        main_grad view)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                res = self.backward(hidden, weight, targets, lse, grad_loss, grad_hidden, grad_weight, accumulate,
                                    need_hidden, need_weight)
            _lend(stream, hidden, weight, targets, lse, grad_loss, grad_hidden, grad_weight)
            return res
        n, id_bytes, hs, ws, at, (_, size) = self._inputs(hidden, weight, targets)
        _floats(lse, "lse")
        _floats(grad_loss, "grad_loss")
        if lse.numel() != n:
            raise ValueError(f"lse has {lse.numel()} elements for {n} tokens")
        if grad_loss.numel() not in (1, n):
            raise ValueError(f"grad_loss has {grad_loss.numel()} elements for {n} tokens")
        dim = ghs = gws = self.dim
        if not need_hidden:
            grad_hidden = None
        elif grad_hidden is None:
            grad_hidden = torch.empty((n, dim), dtype=self.torch_dtype, device=weight.device)
        else:
            ghs = _rows(grad_hidden, "grad_hidden", n, dim, self._same)
        if not need_weight:
            grad_weight = None
        elif grad_weight is None:
            if accumulate:
                raise ValueError("accumulate needs a grad_weight")
            grad_weight = torch.empty((self.vocab, dim), dtype=self.torch_dtype, device=weight.device)
        else:
            gws = _rows(grad_weight, "grad_weight", self.vocab, dim, self._wide)
        scratch = torch.empty(size, dtype=torch.uint8, device=weight.device)
        # an empty output has no address; the library takes NULL for "not wanted"
        if grad_hidden is not None and n == 0 and grad_weight is None:
            return grad_hidden, None
        _check(lib().ddp_vocab_loss_backward(hidden.data_ptr(), hs, at, ws, self.dtype, n, self.vocab, dim,
                                             targets.data_ptr(), id_bytes, self.ignore_index, lse.data_ptr(),
                                             grad_loss.data_ptr(), int(grad_loss.numel() == n and n != 1),
                                             None if grad_hidden is None else grad_hidden.data_ptr(), ghs,
                                             None if grad_weight is None else grad_weight.data_ptr(), gws,
                                             self.dtype if grad_weight is None else _DTYPES[grad_weight.dtype],
                                             int(accumulate), self.piece, scratch.data_ptr(), size,
                                             _raw_stream(weight.get_device())))
        return grad_hidden, grad_weight
