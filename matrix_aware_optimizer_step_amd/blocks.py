"""8-bit block codes of libmuon355 for torch: a matrix as e4m3 codes with an
fp32 scale for each block of 128, and the products of such codes.

The operators stand around the optimizer step: ``WeightCodes`` keeps the codes
of the weights that a step has just changed (``OptimizerStep(codes=...)`` writes
them after every step), ``quantize`` makes those of activations and gradients,
``block_matmul`` and ``expert_matmul`` run a layer forward and backward on them,
and ``expert_grad`` (or ``block_matmul`` of two transposed operands) adds the
gradient of the weights to the fp32 buffer that the next step reads.

Every call only enqueues kernels, on the current stream of its tensors' device
or on ``stream``; there is no CPU path.
"""

from __future__ import annotations

import torch

from . import _lib as L
from .multi import _OnDevice
from .muon import _made_on, _record_on, _stream, _stream_object, batch, dtype_code

E4M3 = torch.float8_e4m3fn
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: int(torch.cuda.current_stream(index).cuda_stream))


def _up(n: int, to: int) -> int:
    return -(-n // to) * to


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _same_device(device, t, name) -> None:
    if t is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _enqueue(device, stream, fresh, fn, *args) -> None:
    """fn(*args, raw stream) with ``device`` current.  ``fresh``: tensors that
    the call allocated, of the current stream's memory or of ``stream``'s: they
    are used on both."""
    if device.type != "cuda":
        raise RuntimeError("the tensors are not on a GPU (there is no CPU path)")
    if device.index == torch.cuda.current_device():
        if stream is None:
            fn(*args, _raw_stream(device.index))
        else:
            fn(*args, _stream(stream))
            _use(stream, fresh)
        return
    with torch.cuda.device(device):
        fn(*args, _raw_stream(device.index) if stream is None else _stream(stream))
        _use(stream, fresh)


def _use(stream, tensors) -> None:
    """Tensors of a call on ``stream``: the call's kernels write them there, and
    what follows on the current stream reads them, each longer than the caller
    may hold them.  The device is current."""
    if stream is not None:
        _record_on(_stream_object(stream), tensors)
        _record_on(torch.cuda.current_stream(), tensors)


def _filled(t, value, stream, offsets=None):
    """t, filled on the call's stream (results that no kernel computes); with
    ``offsets`` its rows from the first of them to the last."""
    if t.is_cuda:
        with torch.cuda.device(t.device):
            with torch.cuda.stream(_stream_object(stream)):
                if offsets is None:
                    t.fill_(value)
                else:
                    row = torch.arange(t.shape[0], device=t.device)
                    t.masked_fill_(((row >= offsets[0]) & (row < offsets[-1]))[:, None], value)
            _use(stream, [t])
        return t
    return t.fill_(value)


class BlockCodes:
    """A matrix (or a batch of equal ones) as e4m3 codes with block scales.

    ``codes``: float8_e4m3fn, [rows, cols] or [count, rows, cols], rows padded
    in memory to whole blocks of 128 whose codes behind the last column are
    zero.  ``scales``: float32, [blocks of columns, blocks of rows] with
    ``block_rows`` (1 or 128) rows to a block.  The value of an element is
    ``codes[r, c] * scales[c // 128, r // block_rows]``.

    ``BlockCodes.empty`` makes the buffers; codes of other origin are taken as
    they are: their padding must be zero.
    """

    __slots__ = ("codes", "scales", "block_rows", "shape", "count", "rows", "cols", "device", "desc")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, block_rows: int = 1):
        _need(block_rows in (1, L.CODE_BLOCK), "block_rows must be 1 or 128")
        if codes.dtype != E4M3 or scales.dtype != torch.float32:
            raise TypeError("codes must be float8_e4m3fn and scales float32")
        _need(codes.dim() in (2, 3) and scales.dim() == codes.dim(), "codes and scales must both be 2-D or both 3-D")
        _same_device(codes.device, scales, "scales")
        rows, cols = codes.shape[-2:]
        wide, high = -(-cols // L.CODE_BLOCK), -(-rows // block_rows)
        if tuple(scales.shape) != (*codes.shape[:-2], wide, high):
            raise ValueError(f"scales of {tuple(codes.shape)} codes must be {(*codes.shape[:-2], wide, high)}, "
                             f"not {tuple(scales.shape)}")
        # (a dimension of one element may carry any stride)
        _need(codes.stride(-1) == 1 or cols <= 1, "codes must be row-major (last stride 1)")
        _need(scales.stride(-1) == 1 or high <= 1, "the scales of a block column must be contiguous")
        ld = codes.stride(-2) if rows > 1 else max(codes.stride(-2), wide * L.CODE_BLOCK)
        scale_ld = scales.stride(-2) if wide > 1 else max(scales.stride(-2), high)
        _need(rows == 0 or cols == 0 or (ld >= wide * L.CODE_BLOCK and ld % 16 == 0),
              "rows of codes must be padded to whole blocks of 128 (a row stride that is a multiple of 16)")
        end = codes.storage_offset() + wide * L.CODE_BLOCK
        if rows and cols:
            end += (rows - 1) * ld + (codes.stride(0) * (codes.shape[0] - 1) if codes.dim() == 3 else 0)
            _need(end <= codes.untyped_storage().nbytes(), "the last row's padding lies outside of the codes' memory")
        self._describe(codes, scales, block_rows, codes.shape[0] if codes.dim() == 3 else None, rows, cols, ld, scale_ld)

    def _describe(self, codes, scales, block_rows, count, rows, cols, ld, scale_ld) -> None:
        self.codes, self.scales, self.block_rows = codes, scales, block_rows
        self.shape, self.device = codes.shape, codes.device
        self.rows, self.cols = rows, cols
        self.count = 1 if count is None else count
        self.desc = L.MuonCodes(codes.data_ptr(), scales.data_ptr(), 0 if count is None else codes.stride(0),
                                0 if count is None else scales.stride(0), self.count, rows, cols, ld, scale_ld,
                                block_rows, 0)

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, count: int | None = None, device="cuda") -> "BlockCodes":
        """Buffers for ``quantize(..., out=)`` to fill (whole blocks: it also writes the padding)."""
        _need(block_rows in (1, L.CODE_BLOCK), "block_rows must be 1 or 128")
        ld, high = _up(cols, L.CODE_BLOCK), -(-rows // block_rows)
        wide = ld // L.CODE_BLOCK
        lead = () if count is None else (count,)
        codes = torch.empty((*lead, rows, ld), dtype=E4M3, device=device)
        scales = torch.empty((*lead, wide, high), dtype=torch.float32, device=device)
        self = cls.__new__(cls)
        self._describe(codes if ld == cols else codes[..., :cols], scales, block_rows, count, rows, cols, max(ld, 1),
                       max(high, 1))
        return self

    def __getitem__(self, i: int) -> "BlockCodes":
        """Matrix i of a batch."""
        _need(self.codes.dim() == 3, "only a batch has matrices")
        return BlockCodes(self.codes[i], self.scales[i], self.block_rows)

    def float(self) -> torch.Tensor:
        """The values in fp32 (torch operations, for looking at them)."""
        s = self.scales.transpose(-1, -2)
        s = s.repeat_interleave(self.block_rows, -2)[..., :self.rows, :] if self.block_rows > 1 else s
        return self.codes.float() * s.repeat_interleave(L.CODE_BLOCK, -1)[..., :self.cols]


def quantize(x, *, block_rows: int = 1, order: str = "rows", pairs: torch.Tensor | None = None,
             weights: torch.Tensor | None = None, out=None, stream=None):
    """A matrix, a batch [count, rows, cols] or a list of equal matrices as
    block codes (``muon_block_quantize``).

    ``order``: "rows" gives codes of x, "cols" codes of its transpose, "both"
    (codes, codes of the transpose) from one pass.  Forward and backward
    products by the weights take a weight's two orders with ``block_rows=128``;
    activations and gradients take blocks of one row.

    ``pairs`` (int32 [n], as ``route`` returns them): row i is row
    ``pairs[i] // k`` of x, zeros where pairs[i] < 0; ``weights`` (float32 [rows of
    x, k]) multiplies it by the pair's weight.  Without weights pairs are rows
    of x (k = 1) unless ``weights`` or a tuple ``(pairs, k)`` says otherwise.

    ``out``: the BlockCodes (or the pair of them) to write into.
    """
    _need(order in ("rows", "cols", "both"), 'order must be "rows", "cols" or "both"')
    _need(block_rows in (1, L.CODE_BLOCK), "block_rows must be 1 or 128")
    if isinstance(x, torch.Tensor) and x.dim() == 2:
        desc, owned, count, device = _matrix(x, "x"), [], None, x.device
    else:
        b = batch(x)
        desc, owned, count, device = b.desc, b.owned, b.count, b.keep[-1].device
    k, rows, cols = 1, desc.rows, desc.cols
    if pairs is not None:
        if isinstance(pairs, tuple):
            pairs, k = pairs
        _need(pairs.dtype == torch.int32 and pairs.dim() == 1 and pairs.is_contiguous(),
              "pairs must be a contiguous int32 vector")
        _need(count is None, "pairs take one matrix")
        _need(block_rows == 1, "pairs take blocks of one row")
        _same_device(device, pairs, "pairs")
        if weights is not None:
            _need(weights.dim() == 2 and weights.shape[0] == rows, "weights must be [rows of x, k]")
            _need(weights.dtype == torch.float32 and weights.is_contiguous(), "weights must be contiguous float32")
            _need(k in (1, weights.shape[1]), "weights and k differ")
            _same_device(device, weights, "weights")
            k = weights.shape[1]
        rows = pairs.numel()
    else:
        _need(weights is None, "weights need pairs")
    fresh = []
    if out is None:
        q, qt = _made_on(stream, device, lambda: (
            None if order == "cols" else BlockCodes.empty(rows, cols, block_rows, count, device),
            None if order == "rows" else BlockCodes.empty(cols, rows, block_rows, count, device)))
        fresh = [t for one in (q, qt) if one is not None for t in (one.codes, one.scales)]
    else:
        q, qt = out if order == "both" else (None, out) if order == "cols" else (out, None)
        for one, shape in ((q, (rows, cols)), (qt, (cols, rows))):
            if one is not None:
                _need(isinstance(one, BlockCodes) and (one.rows, one.cols) == shape and one.block_rows == block_rows and
                      one.codes.dim() == (2 if count is None else 3) and one.count == (count or 1),
                      "out must be BlockCodes of the codes' shape (a pair of them for both orders)")
                _same_device(device, one.codes, "out")
    if rows and cols and count != 0:
        _enqueue(device, stream, fresh + owned, L.muon_block_quantize, desc,
                 None if pairs is None else pairs.data_ptr(), None if weights is None else weights.data_ptr(), k,
                 None if q is None else q.desc, None if qt is None else qt.desc)
    return (q, qt) if order == "both" else q if qt is None else qt


class WeightCodes(_OnDevice):
    """The codes of a weight, or of several equal ones (an expert layer's), kept
    in both orders and made anew from the weights by ``refresh()``.

    ``weights``: a matrix, a batch [count, rows, cols], or a list of equal
    matrices, bfloat16 or float32, read from the same storage every time.
    ``codes`` are the weights' (the forward product reads them), ``transposed`` those
    of their transposes (the gradient of a layer's input does), both with blocks of
    128x128.  ``OptimizerStep(codes={...})`` refreshes after each of its steps.
    """

    def __init__(self, weights):
        self.batch = batch(weights)
        first = self.batch.keep[-1]
        _need(self.batch.rows > 0 and self.batch.cols > 0 and self.batch.count > 0, "no weights")
        count = None if isinstance(weights, torch.Tensor) and weights.dim() == 2 else self.batch.count
        device = first.device
        self.codes = BlockCodes.empty(self.batch.rows, self.batch.cols, L.CODE_BLOCK, count, device)
        self.transposed = BlockCodes.empty(self.batch.cols, self.batch.rows, L.CODE_BLOCK, count, device)
        self._own(device, [t for q in (self.codes, self.transposed) for t in (q.codes, q.scales)] + self.batch.owned)
        self.refresh()
        torch.cuda.current_stream(device).synchronize()  # any stream may use them from here on

    def refresh(self, stream=None) -> None:
        """Enqueues ``muon_block_quantize`` of the weights as they are then."""
        raw = self._on(stream)
        self._call(self._here(), L.muon_block_quantize, self.batch.desc, None, None, 1, self.codes.desc,
                   self.transposed.desc, raw)


def _matrix(t, what) -> L.MuonBatch:
    if t.dim() != 2 or not (t.stride(1) == 1 or t.shape[1] <= 1):
        raise ValueError(f"{what} must be a row-major matrix (last stride 1)")
    rows, cols = t.shape
    ld = t.stride(0)
    return L.MuonBatch(None, t.data_ptr(), 0, 1, rows, cols, ld if rows > 1 or ld > cols else max(cols, 1),
                       dtype_code(t), 0)


def _result(out, shape, dtype, accumulate, device, stream):
    """(the result's tensor, whether it was allocated here)."""
    if out is None:
        _need(not accumulate, "accumulate needs out")
        return _made_on(stream, device, lambda: torch.empty(shape, dtype=dtype, device=device)), True
    if tuple(out.shape) != shape:
        raise ValueError(f"out must be {shape}, not {tuple(out.shape)}")
    _need(out.stride(-1) == 1 or out.shape[-1] <= 1, "out must be row-major (last stride 1)")
    _same_device(device, out, "out")
    if accumulate and out.dtype != torch.float32:
        raise TypeError("only a float32 result accumulates")
    return out, False


def _c_desc(t: torch.Tensor) -> L.MuonBatch:
    rows, cols = t.shape[-2:]
    return L.MuonBatch(None, t.data_ptr(), t.stride(0) if t.dim() == 3 else 0, t.shape[0] if t.dim() == 3 else 1, rows,
                       cols, t.stride(-2) if rows > 1 else max(t.stride(-2), cols), dtype_code(t), 0)


def _check_operands(a, b) -> None:
    if not (isinstance(a, BlockCodes) and isinstance(b, BlockCodes)):
        raise TypeError("a and b must be BlockCodes")
    _need(a.block_rows == 1, "a's blocks must have one row")
    _need(a.cols == b.cols, "a and b differ in columns")
    _same_device(a.device, b.codes, "b")


def _check_offsets(offsets, device) -> None:
    _need(offsets.dtype == torch.int32 and offsets.dim() == 1 and offsets.is_contiguous() and offsets.numel() >= 2,
          "offsets must be a contiguous int32 vector of one more than the experts")
    _same_device(device, offsets, "offsets")


def block_matmul(a: BlockCodes, b: BlockCodes, *, out: torch.Tensor | None = None, dtype=torch.bfloat16,
                 accumulate: bool = False, stream=None) -> torch.Tensor:
    """A B^T of two matrices, or of two batches matrix by matrix.

    A's blocks have one row (activations, gradients), B's one or 128 (weights).
    ``dtype`` (bfloat16 or float32) is the result's where ``out`` is None.
    ``accumulate`` adds to a float32 ``out``.  With the codes of the transposes of
    an output's gradient and of the input this is the gradient of a weight.
    """
    _check_operands(a, b)
    _need(a.codes.dim() == b.codes.dim() and a.count == b.count, "a and b must be two matrices or two equal batches")
    shape = (a.rows, b.rows) if a.codes.dim() == 2 else (a.count, a.rows, b.rows)
    c, made = _result(out, shape, dtype, accumulate, a.device, stream)
    if c.numel() == 0:
        return c
    if a.cols == 0:
        return c if accumulate else _filled(c, 0, stream)
    _enqueue(a.device, stream, [c] if made else [], L.muon_block_matmul, a.desc, b.desc, _c_desc(c), None,
             L.PRODUCT_BATCH, int(bool(accumulate)))
    return c


def expert_matmul(a: BlockCodes, b: BlockCodes, offsets: torch.Tensor, *, out: torch.Tensor | None = None,
                  dtype=torch.bfloat16, accumulate: bool = False, stream=None) -> torch.Tensor:
    """Every expert's product with its own rows: rows offsets[e] .. offsets[e+1]
    of the result are those rows of A times B[e]^T.

    ``a`` [rows, cols], ``b`` [experts, outputs, cols], ``offsets`` int32 [experts + 1]
    on the device, ascending (``Routing.offsets``).  Rows behind the last expert's
    are left as they were (unwritten memory where ``out`` is None).
    """
    _check_operands(a, b)
    _need(a.codes.dim() == 2 and b.codes.dim() == 3, "a must be one matrix and b a batch")
    _check_offsets(offsets, a.device)
    _need(offsets.numel() == b.count + 1, "offsets must be one more than the experts")
    c, made = _result(out, (a.rows, b.rows), dtype, accumulate, a.device, stream)
    if c.numel() == 0:
        return c
    if a.cols == 0:
        return c if accumulate else _filled(c, 0, stream, None if made else offsets)
    _enqueue(a.device, stream, [c] if made else [], L.muon_block_matmul, a.desc, b.desc, _c_desc(c),
             offsets.data_ptr(), L.PRODUCT_ROWS, int(bool(accumulate)))
    return c


def expert_grad(a: BlockCodes, b: BlockCodes, offsets: torch.Tensor, *, out: torch.Tensor | None = None,
                dtype=torch.float32, accumulate: bool = False, stream=None) -> torch.Tensor:
    """Every expert's weight gradient: C[e] = A[:, o_e:o_(e+1)] B[:, o_e:o_(e+1)]^T.

    ``a`` [outputs, rows] and ``b`` [inputs, rows] are codes of the transposes (of
    the outputs' gradients and of the inputs, rows as ``offsets`` divides them;
    ``route(align=128)`` starts each expert on a block of its own, otherwise two
    experts may share a block's scales).  The result is
    [experts, outputs, inputs]; ``accumulate`` adds to a float32 ``out``, which may
    be the gradient buffers that an optimizer step reads.  An expert without
    rows gets zeros, or stays as it is.
    """
    _check_operands(a, b)
    _need(a.codes.dim() == 2 and b.codes.dim() == 2, "a and b must be one matrix each")
    _check_offsets(offsets, a.device)
    c, made = _result(out, (offsets.numel() - 1, a.rows, b.rows), dtype, accumulate, a.device, stream)
    if c.numel() == 0:
        return c
    if a.cols == 0:
        return c if accumulate else _filled(c, 0, stream)
    _enqueue(a.device, stream, [c] if made else [], L.muon_block_matmul, a.desc, b.desc, _c_desc(c),
             offsets.data_ptr(), L.PRODUCT_REDUCE, int(bool(accumulate)))
    return c
