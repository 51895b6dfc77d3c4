"""The two ends of a language model, the norms between them, and the clip and the
optimizer's step behind the reduction: plumbing over ddp_clip_grads, ddp_embedding_*,
ddp_vocab_loss_*, ddp_layer_norm_* and ddp_adamw_step.

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
import numbers

import numpy as np
import torch

from . import (DDP_ADAMW_BLOCK, DDP_ALLREDUCE, DDP_BF16, DDP_CLIP_WORKSPACE_BYTES, DDP_F16, DDP_F32, DDP_NORM_INF,
               DDP_NORM_L2, _check, lib, ddp_embedding_workspace, ddp_layer_norm_workspace, ddp_vocab_loss_workspace)

try:
    from torch._C import _cuda_getCurrentRawStream as _raw_stream
except ImportError:  # pragma: no cover - another torch
    def _raw_stream(device):
        return torch.cuda.current_stream(device).cuda_stream

try:
    from torch._C import _cuda_getDevice as _current_device
except ImportError:  # pragma: no cover - another torch
    from torch.cuda import current_device as _current_device

_empty, _empty_like, _F32 = torch.empty, torch.empty_like, torch.float32
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
        self._streams = set()   # those on which the allocator knows all of this memory in use

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
        were made, the caller's tensors on any; on another one the allocator has to learn of their use, or it gives
        their memory away, while the kernels still read it, when the object and its tensors are dropped."""
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


class LayerNorm:
    """Layer norm over the rows of a [tokens, dim] matrix, with the residual addition before it, and its gradients.

    dtype  of the rows.  Weights and biases are of dtype too, or float32.
    """

    def __init__(self, dim, dtype, eps=1e-5):
        self.dim, self.torch_dtype, self.dtype, self.eps = int(dim), dtype, _dtype(dtype), float(eps)
        if self.dim < 1:
            raise ValueError(f"dim = {dim}")
        self._same = (dtype,)
        self._wide = (dtype, torch.float32)
        self._sizes = {}

    def _columns(self, x, name):
        """x as dim contiguous values of dtype or float32 on the GPU; its address."""
        if x.dtype not in self._wide:
            raise ValueError(f"{name} has dtype {x.dtype}, expected {' or '.join(str(d) for d in self._wide)}")
        _here(x, name)
        if x.numel() != self.dim or not x.is_contiguous():
            raise ValueError(f"{name} must be {self.dim} contiguous values, got shape {tuple(x.shape)} and "
                             f"strides {x.stride()}")
        return x.data_ptr()

    def forward(self, x, weight, bias=None, residual=None, out=None, sum_out=None, stream=None):
        """(norm of s, s, stats) with s = x + residual as it is stored (x itself without a residual) and stats
        a float32 [2, tokens] tensor of the rows' means and reciprocal deviations, for backward.
        out and sum_out may be x or the residual."""
        if stream is not None:
            with torch.cuda.stream(stream):
                res = self.forward(x, weight, bias, residual, out, sum_out)
            _lend(stream, x, weight, bias, residual, out, sum_out)
            return res
        dim, same = self.dim, self._same
        n = x.numel() // dim   # (_rows checks the shape)
        os = xs = _rows(x, "x", n, dim, same)
        w, kind = self._columns(weight, "weight"), weight.dtype
        b = None
        if bias is not None:
            b = self._columns(bias, "bias")
            if bias.dtype != kind:
                raise ValueError(f"bias has dtype {bias.dtype}, the weight {kind}")
        dense = xs == dim   # new tensors are made like x, which is the least work where that is what they should be
        if out is not None:
            os = _rows(out, "out", n, dim, same)
        elif dense:
            out = _empty_like(x)
        else:
            out, os = _empty((n, dim), dtype=self.torch_dtype, device=x.device), dim
        r = sp = None
        rs = ss = dim
        s = x
        if residual is not None:
            rs = _rows(residual, "residual", n, dim, same)
            if sum_out is not None:
                s, ss = sum_out, _rows(sum_out, "sum_out", n, dim, same)
            else:
                s = _empty_like(x) if dense else _empty((n, dim), dtype=self.torch_dtype, device=x.device)
            r, sp = residual.data_ptr(), s.data_ptr()
        elif sum_out is not None:
            raise ValueError("a sum_out without a residual")
        stats = _empty((2, n), dtype=_F32, device=x.device)
        if n:   # (an empty tensor has no address)
            at = stats.data_ptr()
            status = lib().ddp_layer_norm_forward(x.data_ptr(), xs, r, rs, self.dtype, n, dim, w, b, _DTYPES[kind], self.eps,
                                                  out.data_ptr(), os, sp, ss, at, at + 4 * n, _raw_stream(x.get_device()))
            if status:
                _check(status)
        return out, s, stats

    def backward(self, grad_out, s, weight, stats, grad_sum=None, grad_x=None, grad_weight=None, grad_bias=None,
                 accumulate=False, need_weight=True, need_bias=True, stream=None):
        """(grad_x, grad_weight, grad_bias).  grad_x is the gradient of x and of the residual alike; grad_sum is added to
        it: the gradient that reaches s past the norm.  With accumulate the weight's and the bias's gradients are added to
        grad_weight and grad_bias (of dtype, or float32: main_grad views).  grad_x may be grad_out, grad_sum or s."""
        if stream is not None:
            with torch.cuda.stream(stream):
                res = self.backward(grad_out, s, weight, stats, grad_sum, grad_x, grad_weight, grad_bias, accumulate,
                                    need_weight, need_bias)
            _lend(stream, grad_out, s, weight, stats, grad_sum, grad_x, grad_weight, grad_bias)
            return res
        dim, same = self.dim, self._same
        n = s.numel() // dim   # (_rows checks the shape)
        gxs = xs = _rows(s, "s", n, dim, same)
        gs = _rows(grad_out, "grad_out", n, dim, same)
        w, kind = self._columns(weight, "weight"), weight.dtype
        w_dtype = _DTYPES[kind]
        _floats(stats, "stats")
        if stats.numel() != 2 * n:
            raise ValueError(f"stats has {stats.numel()} elements for {n} tokens")
        if grad_x is not None:
            gxs = _rows(grad_x, "grad_x", n, dim, same)
        elif xs == dim:
            grad_x = _empty_like(s)
        else:
            grad_x, gxs = _empty((n, dim), dtype=self.torch_dtype, device=s.device), dim
        ds, dss = None, dim
        if grad_sum is not None:
            dss = _rows(grad_sum, "grad_sum", n, dim, same)
            ds = grad_sum.data_ptr()
        if accumulate and (need_weight and grad_weight is None or need_bias and grad_bias is None):
            raise ValueError("accumulate needs a grad_weight and a grad_bias")
        if not need_weight:
            grad_weight = None
        if not need_bias:
            grad_bias = None
        # (what the caller does not pass is made of the type of what he passes)
        if grad_weight is not None:
            kind = grad_weight.dtype
        elif grad_bias is not None:
            kind = grad_bias.dtype
        gw = gb = scratch = None
        if need_weight:
            if grad_weight is None:
                grad_weight = _empty(dim, dtype=kind, device=s.device)
                gw = grad_weight.data_ptr()
            else:
                gw = self._columns(grad_weight, "grad_weight")
        if need_bias:
            if grad_bias is None:
                grad_bias = _empty(dim, dtype=kind, device=s.device)
                gb = grad_bias.data_ptr()
            else:
                gb = self._columns(grad_bias, "grad_bias")
                if grad_bias.dtype != kind:
                    raise ValueError(f"grad_bias has dtype {grad_bias.dtype}, grad_weight {kind}")
        size = 0
        if need_weight or need_bias:
            key = n, s.get_device()   # (it depends on the number of SMs)
            size = self._sizes.get(key)
            if size is None:
                if len(self._sizes) >= 64:
                    self._sizes.clear()
                size = self._sizes[key] = ddp_layer_norm_workspace(n, dim)
            memory = _empty(size, dtype=torch.uint8, device=s.device)
            scratch = memory.data_ptr()
        at = stats.data_ptr()
        status = lib().ddp_layer_norm_backward(grad_out.data_ptr(), gs, s.data_ptr(), xs, at, at + 4 * n, ds, dss, self.dtype,
                                               n, dim, w, w_dtype, grad_x.data_ptr(), gxs, gw, gb, _DTYPES[kind],
                                               accumulate, scratch, size, _raw_stream(s.get_device()))
        if status:
            _check(status)
        return grad_x, grad_weight, grad_bias


def _apart(names, lists) -> None:
    """No tensor of the lists shares memory with another, but those of the last list among themselves."""
    held = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), j, k)
                  for j, ts in enumerate(lists) for k, t in enumerate(ts) if t is not None and t.numel())
    end, of = 0, None        # the furthest end so far of a list's before the last, and of the last's
    read_end, read_of = 0, None
    last = len(lists) - 1
    for a, b, j, k in held:
        for limit, other, only_written in ((end, of, False), (read_end, read_of, True)):
            if a < limit and not (only_written and j == last):
                raise ValueError(f"{names[j]} {k} shares memory with {names[other[0]]} {other[1]}")
        if j == last:
            if b > read_end:
                read_end, read_of = b, (j, k)
        elif b > end:
            end, of = b, (j, k)


_RECORD = np.dtype([("param", np.int64), ("copy", np.int64), ("grad", np.int64), ("numel", np.int64),
                    ("param_dtype", np.int32), ("copy_dtype", np.int32), ("grad_dtype", np.int32),
                    ("weight_decay", np.float32)])   # ddp_adamw_tensor


class AdamW:
    """AdamW over a list of parameters, all in one launch, with moments in 32 or in 8 bits.

    params        contiguous fp32 / bf16 / fp16 tensors on the GPU, stepped in place.
    grads         the gradients, of any of those types (None: that parameter is left as it is): main_grad views, say.
                  Addresses are read once: parameters, gradients and copies must keep their storage.
    copies        tensors that receive the new parameters, rounded to their types (a list with None where there is none):
                  the 16-bit weights that a model computes with.  Parameters and copies share memory with nothing: a
                  tied parameter is given once.
    weight_decay  one value, or one for each parameter.
    state_bits    32: moments in fp32.  8: in e4m3 with a scale for each 256 values, rounded by chances that follow from
                  `seed` and the step's number.

    The moments (exp_avg, exp_avg_sq, in 8 bits with exp_avg_scale and exp_avg_sq_scale) are laid out in blocks of 256
    values, where every parameter starts a new one; in 8 bits exp_avg_sq holds square roots.  The number of steps taken
    is kept on the GPU, so a step that was captured into a graph counts on.
    """

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, copies=None,
                 state_bits=32, seed=0):
        params, grads = tuple(params), tuple(grads)
        copies = (None,) * len(params) if copies is None else tuple(copies)
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits {state_bits} is neither 8 nor 32")
        if len(grads) != len(params) or len(copies) != len(params):
            raise ValueError(f"{len(grads)} gradients and {len(copies)} copies for {len(params)} parameters")
        decays = [float(weight_decay)] * len(params) if isinstance(weight_decay, numbers.Real) else [float(d) for d in weight_decay]
        if len(decays) != len(params):
            raise ValueError(f"{len(decays)} weight decays for {len(params)} parameters")
        if not all(0.0 <= d <= 3e38 for d in decays):   # (fp32)
            raise ValueError("a weight decay is negative or not finite")
        table = np.zeros(len(params), _RECORD)
        for k, (p, g, c) in enumerate(zip(params, grads, copies)):
            if p is None:
                raise ValueError(f"parameter {k} is None")
            for name, t in (("parameter", p), ("gradient", g), ("copy", c)):
                if t is None:
                    continue
                _dtype(t.dtype)
                if not t.is_cuda or not t.is_contiguous() or t.numel() != p.numel():
                    raise ValueError(f"{name} {k} is not a contiguous tensor of {p.numel()} elements on the GPU")
                _here(t, f"{name} {k}")
            table[k] = (p.data_ptr(), 0 if c is None else c.data_ptr(), 0 if g is None else g.data_ptr(), p.numel(),
                        _dtype(p.dtype), DDP_F32 if c is None else _dtype(c.dtype), DDP_F32 if g is None else _dtype(g.dtype),
                        decays[k])
        _apart(("parameter", "copy", "gradient"), (params, copies, grads))
        self.device = params[0].device if params else torch.device("cuda", torch.cuda.current_device())
        self.lr, self.betas, self.eps = float(lr), (float(betas[0]), float(betas[1])), float(eps)
        self.state_bits, self.seed = state_bits, int(seed) % (1 << 64)
        self.ntensors = len(params)
        self._tensors = params, grads, copies   # the table below points into these
        blocks = np.array([-(-p.numel() // DDP_ADAMW_BLOCK) for p in params], np.int64)
        self.first_block = np.concatenate([[0], np.cumsum(blocks)]).astype(np.int64)
        n = self.nblocks = int(self.first_block[-1])
        # one device buffer: the steps taken and a word of the kernel's own, then the blocks, then the records
        words = [np.zeros(2, np.int64), self.first_block, table.view(np.int64).reshape(-1)]
        self._tables = torch.from_numpy(np.concatenate(words)).to(self.device)
        at = self._tables.data_ptr()
        self._state, self._first_at = at, at + 16
        self._records = self._first_at + 8 * len(self.first_block)
        kind = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        self.exp_avg, self.exp_avg_sq = (torch.zeros((n, DDP_ADAMW_BLOCK), dtype=kind, device=self.device) for _ in range(2))
        self.exp_avg_scale = self.exp_avg_sq_scale = None
        if state_bits == 8:
            self.exp_avg_scale, self.exp_avg_sq_scale = (torch.zeros(n, device=self.device) for _ in range(2))
        self._moments = [None if t is None else t.data_ptr() for t in
                         (self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale)]
        self._streams = set()   # those on which the allocator knows all of this memory in use

    @classmethod
    def of_reducer(cls, reducer, params, w=0, **kw):
        """Over replica w's reduced gradients: the views of an all-reducing BucketReducer's main_grad, in the order of
        its parameters."""
        if reducer.mode != DDP_ALLREDUCE:
            raise ValueError("after a reduce-scatter a replica holds only its own shard of the reduced gradients")
        if reducer.main_grad is None:
            raise ValueError("the reducer keeps no main_grad")
        return cls(params, [reducer.view(p, w) for p in range(reducer.plan.nparams)], **kw)

    def step(self, lr=None, norm=None, max_norm=None, grad_scale=1.0, stream=None):
        """One step.  lr: a number, or a float32 tensor of one element on the GPU (None: the object's).
        norm, max_norm: the gradients' global norm (GradClipper.norm()) and what it is clipped to on the way; a norm
        that is not finite leaves everything as it is.  grad_scale: the factor that is in the gradients and the norm."""
        if stream is not None:
            with torch.cuda.stream(stream):
                self.step(lr, norm, max_norm, grad_scale)
            _lend(stream, norm, lr if isinstance(lr, torch.Tensor) else None)
            return
        if self.device.index != _current_device():
            raise ValueError(f"the parameters are on {self.device}, the current device is cuda:{_current_device()}")
        on = self._stream()
        lr_at = norm_at = None
        if lr is None:
            lr = self.lr
        elif isinstance(lr, torch.Tensor):
            lr_at, lr = self._one(lr, "lr"), 0.0
        if (norm is None) != (max_norm is None):
            raise ValueError("norm and max_norm come together")
        if norm is not None:
            norm_at = self._one(norm, "norm")
        m, v, ms, vs = self._moments
        _check(lib().ddp_adamw_step(self._records, self._first_at, self.ntensors, self.nblocks, m, v, ms, vs, self.state_bits,
                                    self._state, lr, lr_at, self.betas[0], self.betas[1], self.eps, self.seed, grad_scale,
                                    norm_at, max_norm or 0.0, on))

    @staticmethod
    def _one(t, name):
        _floats(t, name)
        if t.numel() != 1:
            raise ValueError(f"{name} has {t.numel()} elements")
        return t.data_ptr()

    def _stream(self):
        """The current stream's handle.  Before its first use there the allocator learns that all of the memory is: the
        moments and tables are of the stream that the object was made on, the caller's tensors of any."""
        on = _raw_stream(self.device.index)
        if on not in self._streams:
            _lend(torch.cuda.current_stream(self.device), self._tables, self.exp_avg, self.exp_avg_sq, self.exp_avg_scale,
                  self.exp_avg_sq_scale, *self._tensors[0], *self._tensors[1], *self._tensors[2])
            self._streams.add(on)
        return on

    def steps(self) -> int:
        """The steps taken (waits for the current stream)."""
        return int(self._tables[0])

    def moments(self, k):
        """(m, v) of parameter k in fp32, in its shape: copies."""
        self._stream()
        p = self._tensors[0][k]
        rows = slice(int(self.first_block[k]), int(self.first_block[k + 1]))
        m, v = (x[rows].to(torch.float32, copy=True) for x in (self.exp_avg, self.exp_avg_sq))
        if self.state_bits == 8:
            m, v = m * self.exp_avg_scale[rows, None], (v * self.exp_avg_sq_scale[rows, None]).square()
        return tuple(x.reshape(-1)[:p.numel()].view(p.shape) for x in (m, v))

    def state_dict(self):
        """The steps taken and copies of the moments as they are held."""
        self._stream()
        d = {"step": self.steps(), "exp_avg": self.exp_avg.clone(), "exp_avg_sq": self.exp_avg_sq.clone()}
        if self.state_bits == 8:
            d.update(exp_avg_scale=self.exp_avg_scale.clone(), exp_avg_sq_scale=self.exp_avg_sq_scale.clone())
        return d

    def load_state_dict(self, state):
        """Takes what state_dict of an object over the same parameters, with moments of the same kind, gave."""
        names = ["exp_avg", "exp_avg_sq"] + (["exp_avg_scale", "exp_avg_sq_scale"] if self.state_bits == 8 else [])
        if set(state) != {"step", *names}:
            raise ValueError(f"a state of {sorted(state)}, expected {sorted(['step', *names])}")
        for name in names:
            mine, new = getattr(self, name), state[name]
            if new.shape != mine.shape or new.dtype != mine.dtype:
                raise ValueError(f"{name} is {new.dtype} {tuple(new.shape)}, expected {mine.dtype} {tuple(mine.shape)}")
        if int(state["step"]) < 0:
            raise ValueError(f"{state['step']} steps")
        self._stream()
        for name in names:
            getattr(self, name).copy_(state[name])
        self._tables[0] = int(state["step"])
