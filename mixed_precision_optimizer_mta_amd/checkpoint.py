"""8-bit activation checkpoints over PyTorch tensors: mta_ckpt_* of
include/mta_ops.h.

Marshalling only, like MtaList: it checks types, shapes, strides and devices,
allocates outputs and workspaces from PyTorch's allocator (on the current
stream, so a captured call keeps its own), and passes pointers.  Every call
runs on the current stream of its tensors' device.

``ckpt_pack`` / ``ckpt_unpack`` keep tensors at one byte and 1/32 a value and
bring them back; ``ckpt_act`` computes an activation function and keeps its
input, ``ckpt_act_backward`` is its gradient; ``ckpt_wgrad`` is a linear
layer's weight and bias gradient, straight from the kept input, written to a
new tensor or added into an existing gradient (the float32 ``p.grad`` that an
MtaOptimizer's clip and step read, for one).  ``checkpointed_linear`` and
``checkpointed_act`` are the same as autograd functions.

All of them may be captured into a HIP graph.  As with any autograd function,
a backward pass is captured whole: capture the forward and its backward
together, with no graph of an earlier eager forward over the same parameters
still alive.
"""
import torch

from . import _binding as B
from .torch_list import _G, _raw_stream

BLOCK = B.MTA_CKPT_BLOCK


_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on_stream(index, call, *args):
    """call(*args, stream) on the current stream of device `index`, made the
    current device for the call where it is not."""
    if _device() != index:
        with torch.cuda.device(index):
            return _on_stream(index, call, *args)
    stream = _raw_stream(index) if _raw_stream is not None else \
        torch.cuda.current_stream(index).cuda_stream
    return call(*args, stream)


def _check_type(t, what):
    if t.dtype not in _G:
        raise TypeError(f"{what} is float32, bfloat16 or float16, not "
                        f"{t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} is not on the GPU")


def _as_rows(t, what):
    """(rows, cols, pitch) of a tensor whose last dimension is contiguous and
    whose other dimensions are one run of equally spaced rows."""
    if t.dim() == 0:
        raise ValueError(f"{what} needs at least one dimension")
    cols = t.shape[-1]
    rows = t.numel() // cols if cols else 0
    if rows and t.is_contiguous():
        return rows, cols, cols
    if rows == 0:
        return 0, cols, max(1, cols)
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"the last dimension of {what} is not contiguous")
    if rows == 1:
        return 1, cols, cols
    # the spacing of rows: the innermost dimension of more than one
    pitch, step = None, 0
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if pitch is None:
            pitch, step = stride, stride * size
        elif stride != step:
            raise ValueError(f"the rows of {what} are not equally spaced")
        else:
            step *= size
    if pitch < cols:
        raise ValueError(f"the rows of {what} overlap")
    return rows, cols, pitch


def _same_device(device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("the tensors of a call are on one device")


def _written(*tensors):
    """Tensors of the caller's that a call wrote: an autograd graph that saved
    their old values refuses its backward, as after any in-place operation."""
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


class Checkpoint8:
    """A tensor kept in 8 bits: ``q`` (uint8 [rows, cols rounded up to 32],
    e4m3 codes), ``scale`` (uint8 [rows, blocks of 32], biased exponents),
    the tensor's ``shape`` and ``dtype``."""

    __slots__ = ("_q", "_scale", "shape", "dtype", "rows", "blocks")

    def __init__(self, q, scale, shape, dtype=torch.float32):
        self._q, self._scale, self.dtype = q, scale, dtype
        self.shape = shape = tuple(shape)
        self.rows, self.blocks = rows, blocks = self._layout(shape)
        if q.dtype != torch.uint8 or scale.dtype != torch.uint8:
            raise TypeError("q and scale are uint8")
        if dtype not in _G:
            raise TypeError("a checkpoint's dtype is float32, bfloat16 or "
                            "float16")
        if not q.is_cuda or q.device != scale.device:
            raise ValueError("q and scale are on one GPU")
        if not q.is_contiguous() or not scale.is_contiguous():
            raise ValueError("q and scale are contiguous")
        if q.numel() != rows * blocks * BLOCK or scale.numel() != rows * blocks:
            raise ValueError(f"q and scale do not fit the shape {shape}")

    @staticmethod
    def _layout(shape):
        if not shape:
            raise ValueError("a checkpoint needs at least one dimension")
        rows = 1
        for n in shape[:-1]:
            rows *= n
        return rows, -(-shape[-1] // BLOCK)

    @classmethod
    def empty(cls, shape, dtype, device):
        """A checkpoint with room for a tensor, its contents not set.  One
        allocation holds the codes, then the scales."""
        rows, blocks = cls._layout(shape)
        return cls._of_storage(
            torch.empty(rows * blocks * (BLOCK + 1), dtype=torch.uint8,
                        device=device), tuple(shape), dtype)

    @classmethod
    def _of_storage(cls, storage, shape, dtype):
        """The checkpoint that empty() made over `storage`."""
        self = cls.__new__(cls)
        self.rows, self.blocks = cls._layout(shape)
        self._q, self._scale = storage, None
        self.shape, self.dtype = shape, dtype
        return self

    @property
    def q(self):
        if self._scale is None:
            return self._q[:self.rows * self.blocks * BLOCK]
        return self._q

    @property
    def scale(self):
        if self._scale is None:
            return self._q[self.rows * self.blocks * BLOCK:]
        return self._scale

    @property
    def device(self):
        return self._q.device

    def pointers(self):
        """The addresses of the codes and of the scales."""
        q = self._q.data_ptr()
        return q, (q + self.rows * self.blocks * BLOCK
                   if self._scale is None else self._scale.data_ptr())

    def nbytes(self):
        return self.rows * self.blocks * (BLOCK + 1)

    def unpack(self, dtype=None):
        return ckpt_unpack(self, dtype)


def _act_code(act):
    if act not in B.ACTIVATIONS:
        raise ValueError(f"act is one of {sorted(B.ACTIVATIONS)}, not {act!r}")
    return B.ACTIVATIONS[act]


def _pack(tensors, act):
    if not tensors:
        return [], []
    dt, dev = tensors[0].dtype, tensors[0].device
    code = B.MTA_ACT_NONE if act is None else _act_code(act)
    cks, ys, entries = [], [], []
    for t in tensors:
        _check_type(t, "a kept tensor")
        if t.dtype != dt:
            raise TypeError("the tensors of a call share one dtype")
        _same_device(dev, t)
        rows, cols, ld = _as_rows(t, "a kept tensor")
        ck = Checkpoint8.empty(t.shape, dt, dev)
        y = None if act is None else t.new_empty(t.shape)
        cks.append(ck)
        ys.append(y)
        entries.append((t.data_ptr(), None if y is None else y.data_ptr(),
                        *ck.pointers(), rows, cols, ld, cols))
    _on_stream(dev.index, B.mta_ckpt_pack, entries, _G[dt], code)
    return cks, ys


def ckpt_pack(x):
    """Keep a tensor, or the tensors of a list (of one dtype, one launch for
    32 of them), in 8 bits: a Checkpoint8, or a list of them."""
    if isinstance(x, torch.Tensor):
        return _pack([x], None)[0][0]
    return _pack(list(x), None)[0]


def ckpt_unpack(ck, dtype=None):
    """The kept tensor, or the tensors of a list (then of one dtype), in
    `dtype` (default: the dtype kept)."""
    if isinstance(ck, Checkpoint8):
        return ckpt_unpack([ck], dtype)[0]
    cks = list(ck)
    if not cks:
        return []
    dt = cks[0].dtype if dtype is None else dtype
    if dt not in _G or (dtype is None and any(c.dtype != dt for c in cks)):
        raise TypeError("the tensors of a call share one of float32, bfloat16 "
                        "and float16")
    dev = cks[0].device
    outs, entries = [], []
    for c in cks:
        _same_device(dev, c)
        y = torch.empty(c.shape, dtype=dt, device=dev)
        cols = c.shape[-1]
        outs.append(y)
        entries.append((None, y.data_ptr(), *c.pointers(), c.rows, cols, cols,
                        cols))
    _on_stream(dev.index, B.mta_ckpt_unpack, entries, _G[dt])
    return outs


def ckpt_act(x, act):
    """(act(x), the Checkpoint8 of x) in one pass over x; act is "relu",
    "silu", "gelu" or "gelu_tanh"."""
    _act_code(act)
    cks, ys = _pack([x], act)
    return ys[0], cks[0]


def ckpt_act_backward(ck, dy, act):
    """dy * act'(kept), in dy's dtype."""
    code = _act_code(act)
    _check_type(dy, "dy")
    _same_device(ck.device, dy)
    if tuple(dy.shape) != ck.shape:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, the checkpoint "
                         f"{ck.shape}")
    rows, cols, ld = _as_rows(dy, "dy")
    dx = dy.new_empty(ck.shape)
    _on_stream(dy.device.index, B.mta_ckpt_act_backward,
               [(dy.data_ptr(), dx.data_ptr(), *ck.pointers(), rows, cols, ld,
                 cols)], _G[dy.dtype], code)
    return dx


def ckpt_wgrad(ck, dy, bias=True, out=None, out_bias=None, accumulate=False,
               dtype=torch.float32):
    """(dw, db): the weight gradient sum_t dy[t, o] kept[t, i] as [fout, fin]
    and the bias gradient sum_t dy[t, o] (None with bias=False), from the
    checkpoint of a linear layer's input [..., fin] and its output's gradient
    dy [..., fout].  They are new tensors of `dtype`, or `out` and `out_bias`
    (of one dtype), overwritten or, with accumulate, added to; a missing one
    of the two is new.  out may have padded rows."""
    _check_type(dy, "dy")
    _same_device(ck.device, dy, out, out_bias)
    tokens, fin = ck.rows, ck.shape[-1]
    if tuple(dy.shape[:-1]) != ck.shape[:-1]:
        raise ValueError(f"dy has shape {tuple(dy.shape)}, the checkpoint "
                         f"{ck.shape}")
    rows, fout, lddy = _as_rows(dy, "dy")
    if accumulate and (out is None or (bias and out_bias is None)):
        raise ValueError("accumulate needs out (and out_bias for a bias)")
    if out_bias is not None and not bias:
        raise ValueError("out_bias without a bias")
    for t in (out_bias, out):
        if t is not None:
            dtype = t.dtype
    if dtype not in _G:
        raise TypeError("gradients are float32, bfloat16 or float16")
    dev = dy.device
    given = out, out_bias
    if out is None:
        out = torch.empty(fout, fin, dtype=dtype, device=dev)
    if bias and out_bias is None:
        out_bias = torch.empty(fout, dtype=dtype, device=dev)
    if tuple(out.shape) != (fout, fin) or out.dtype != dtype or (
            fin > 1 and out.stride(1) != 1):
        raise ValueError(f"out is [{fout}, {fin}] with contiguous rows")
    lddw = out.stride(0) if fout > 1 else max(1, fin)
    if bias and (tuple(out_bias.shape) != (fout,) or out_bias.dtype != dtype
                 or not out_bias.is_contiguous()):
        raise ValueError(f"out_bias is [{fout}], contiguous, of out's dtype")
    gt = _G[dy.dtype]
    need = _on_stream(dev.index, lambda *x: B.mta_ckpt_wgrad_workspace(
        *x[:-1]), tokens, fin, fout, gt)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _on_stream(dev.index, B.mta_ckpt_wgrad, B.mta_ckpt_wgrad_args(
        *ck.pointers(), dy.data_ptr(), out.data_ptr(),
        out_bias.data_ptr() if bias else None,
        ws.data_ptr() if need else None, need, tokens, fin, fout, lddy, lddw,
        gt, _G[dtype], 1 if accumulate else 0, 0))
    _written(*given)
    return out, out_bias


# --------------------------------------------------------------------------
# autograd
#
# A checkpoint's storage is kept as a saved tensor, so that autograd frees it
# with the graph's other buffers and saved-tensor hooks see it.
# --------------------------------------------------------------------------

def _product(x, weight, bias):
    b = None if bias is None else bias.to(x.dtype)
    return torch.nn.functional.linear(x, weight.to(x.dtype), b)


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        _, need_w, need_b = ctx.needs_input_grad
        # a bias alone needs no input: a checkpoint of no features
        ck = ckpt_pack(_rows_or_copy(x)) if need_w else \
            Checkpoint8.empty((*x.shape[:-1], 0), x.dtype, x.device)
        ctx.kept = ck.shape, ck.dtype
        ctx.save_for_backward(weight, ck._q)
        ctx.bias_dtype = None if bias is None else bias.dtype
        return _product(x, weight, bias)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        weight, storage = ctx.saved_tensors
        need_x, need_w, need_b = ctx.needs_input_grad
        dx = dy.matmul(weight.to(dy.dtype)) if need_x else None
        dw = db = None
        if need_w or need_b:
            # parameters of two dtypes: each rounded once, from float32
            dtype = weight.dtype
            if need_b and ctx.bias_dtype != dtype:
                dtype = torch.float32
            dw, db = ckpt_wgrad(
                Checkpoint8._of_storage(storage, *ctx.kept),
                _rows_or_copy(dy), bias=need_b, dtype=dtype)
            dw = dw.to(weight.dtype) if need_w else None
            db = db.to(ctx.bias_dtype) if need_b else None
        return dx, dw, db


class _Act(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, act):
        y, ck = ckpt_act(_rows_or_copy(x), act)
        ctx.save_for_backward(ck._q)
        ctx.kept, ctx.act = (ck.shape, ck.dtype), act
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        storage, = ctx.saved_tensors
        return ckpt_act_backward(Checkpoint8._of_storage(storage, *ctx.kept),
                                 _rows_or_copy(dy), ctx.act), None


def _rows_or_copy(t):
    """t, or a contiguous copy where its rows are not equally spaced (an
    expanded gradient, a transposed one)."""
    try:
        _as_rows(t, "a tensor")
        return t
    except ValueError:
        return t.contiguous()


def checkpointed_linear(x, weight, bias=None):
    """x W^T + b whose backward keeps x in 8 bits.  The product and x's
    gradient are PyTorch's, in x's dtype; the weight and bias gradients come
    from the checkpoint, in the parameter's own dtype (float32 parameters under
    a 16-bit x get float32 gradients that were never rounded to 16 bits)."""
    _check_type(x, "x")
    _check_type(weight, "weight")
    if weight.dim() != 2 or x.shape[-1] != weight.shape[1]:
        raise ValueError("weight is [fout, fin] with x's last dimension fin")
    if not torch.is_grad_enabled():  # nothing to keep
        return _product(x, weight, bias)
    return _Linear.apply(x, weight, bias)


def checkpointed_act(x, act):
    """act(x) whose backward keeps x in 8 bits (where gradients are off, the
    checkpoint is made and dropped)."""
    _act_code(act)
    return _Act.apply(x, act)
