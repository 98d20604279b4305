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
from .muon import _record_on, _stream, _stream_object, batch, dtype_code

E4M3 = torch.float8_e4m3fn
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: int(torch.cuda.current_stream(index).cuda_stream))


def _up(n: int, to: int) -> int:
    return -(-n // to) * to


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _same_device(device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _enqueue(device, stream, fresh, fn, *args) -> None:
    """fn(*args, raw stream) with ``device`` current.  ``fresh``: tensors that
    the call allocated, recorded on a stream that is not the current one."""
    if device.type != "cuda":
        raise RuntimeError("the tensors are not on a GPU (there is no CPU path)")
    if device.index == torch.cuda.current_device():
        if stream is None:
            fn(*args, _raw_stream(device.index))
        else:
            fn(*args, _stream(stream))
            _record_on(_stream_object(stream), fresh)
        return
    with torch.cuda.device(device):
        fn(*args, _raw_stream(device.index) if stream is None else _stream(stream))
        _record_on(_stream_object(stream), fresh)


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
        _same_device(codes.device, scales=scales)
        rows, cols = codes.shape[-2:]
        wide, high = -(-cols // L.CODE_BLOCK), -(-rows // block_rows)
        _need(tuple(scales.shape[-2:]) == (wide, high) and codes.shape[:-2] == scales.shape[:-2],
              f"scales of {tuple(codes.shape)} codes must be {(*codes.shape[:-2], wide, high)}, not {tuple(scales.shape)}")
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
        self.codes, self.scales, self.block_rows = codes, scales, block_rows
        self.shape, self.device = codes.shape, codes.device
        self.rows, self.cols = rows, cols
        self.count = codes.shape[0] if codes.dim() == 3 else 1
        many = codes.dim() == 3
        self.desc = L.MuonCodes(codes.data_ptr(), scales.data_ptr(), codes.stride(0) if many else 0,
                                scales.stride(0) if many else 0, self.count, rows, cols, ld, scale_ld, block_rows, 0)

    @classmethod
    def empty(cls, rows: int, cols: int, block_rows: int = 1, count: int | None = None, device="cuda") -> "BlockCodes":
        """Buffers for ``quantize(..., out=)`` to fill (whole blocks: it also writes the padding)."""
        lead = () if count is None else (count,)
        codes = torch.empty(*lead, rows, _up(cols, L.CODE_BLOCK), dtype=E4M3, device=device)
        scales = torch.empty(*lead, -(-cols // L.CODE_BLOCK), -(-rows // block_rows), dtype=torch.float32,
                             device=device)
        return cls(codes[..., :cols], scales, block_rows)

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
    b = batch(x)
    first = b.keep[-1]
    device = first.device
    k = 1
    if isinstance(pairs, tuple):
        pairs, k = pairs
    if weights is not None:
        _need(pairs is not None, "weights need pairs")
        _need(weights.dim() == 2 and weights.shape[0] == b.rows, "weights must be [rows of x, k]")
        _need(weights.dtype == torch.float32 and weights.is_contiguous(), "weights must be contiguous float32")
        _need(k in (1, weights.shape[1]), "weights and k differ")
        k = weights.shape[1]
    rows = b.rows
    if pairs is not None:
        _need(pairs.dtype == torch.int32 and pairs.dim() == 1 and pairs.is_contiguous(),
              "pairs must be a contiguous int32 vector")
        _need(b.count == 1 and first.dim() == 2, "pairs take one matrix")
        _need(block_rows == 1, "pairs take blocks of one row")
        rows = pairs.numel()
    _same_device(device, pairs=pairs, weights=weights)
    many = None if isinstance(first, torch.Tensor) and first.dim() == 2 and not isinstance(x, (list, tuple)) else b.count
    fresh = []
    if out is None:
        shapes = [(rows, b.cols)] * (order != "cols") + [(b.cols, rows)] * (order != "rows")
        got = [BlockCodes.empty(r, c, block_rows, many, device) for r, c in shapes]
        fresh = [t for q in got for t in (q.codes, q.scales)]
    else:
        got = list(out) if order == "both" else [out]
        _need(len(got) == (2 if order == "both" else 1) and all(isinstance(q, BlockCodes) for q in got),
              "out must be a BlockCodes, or two of them for both orders")
        for i, q in enumerate(got):
            turned = order == "cols" or i == 1
            _need((q.rows, q.cols) == ((b.cols, rows) if turned else (rows, b.cols)) and q.count == b.count and
                  q.block_rows == block_rows, "out does not fit the codes")
            _same_device(device, out=q.codes)
    if rows and b.cols and b.count:
        q = got[0].desc if order != "cols" else None
        qt = got[-1].desc if order != "rows" else None
        _enqueue(device, stream, fresh + b.owned, L.muon_block_quantize, b.desc,
                 None if pairs is None else pairs.data_ptr(), None if weights is None else weights.data_ptr(), k, q, qt)
    return tuple(got) if order == "both" else got[0]


def _result(out, shape, dtype, accumulate, device):
    """(the result's tensor, whether it was allocated here)."""
    if out is None:
        _need(not accumulate, "accumulate needs out")
        return torch.empty(shape, dtype=dtype, device=device), True
    _need(tuple(out.shape) == tuple(shape), f"out must be {tuple(shape)}, not {tuple(out.shape)}")
    _need(out.stride(-1) == 1 or out.shape[-1] <= 1, "out must be row-major (last stride 1)")
    _same_device(device, out=out)
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
    _need(a.cols == b.cols, f"a has {a.cols} columns and b {b.cols}")
    _same_device(a.device, b=b.codes)


def _check_offsets(offsets, device) -> None:
    _need(offsets.dtype == torch.int32 and offsets.dim() == 1 and offsets.is_contiguous() and offsets.numel() >= 2,
          "offsets must be a contiguous int32 vector of one more than the experts")
    _same_device(device, offsets=offsets)


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
    c, made = _result(out, shape, dtype, accumulate, a.device)
    if c.numel() == 0:
        return c
    if a.cols == 0:
        return c if accumulate else c.zero_()
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
    c, made = _result(out, (a.rows, b.rows), dtype, accumulate, a.device)
    if c.numel() == 0:
        return c
    _need(a.cols > 0, "no columns")
    _enqueue(a.device, stream, [c] if made else [], L.muon_block_matmul, a.desc, b.desc, _c_desc(c),
             offsets.data_ptr(), L.PRODUCT_ROWS, int(bool(accumulate)))
    return c


def expert_grad(a: BlockCodes, b: BlockCodes, offsets: torch.Tensor, *, out: torch.Tensor | None = None,
                dtype=torch.float32, accumulate: bool = False, stream=None) -> torch.Tensor:
    """Every expert's weight gradient: C[e] = A[:, o_e:o_(e+1)] B[:, o_e:o_(e+1)]^T.

    ``a`` [outputs, rows] and ``b`` [inputs, rows] are codes of the transposes (of
    the outputs' gradients and of the inputs, rows as ``offsets`` divides them,
    each expert starting on a multiple of 128: ``route(align=128)``).  The result is
    [experts, outputs, inputs]; ``accumulate`` adds to a float32 ``out``, which may
    be the gradient buffers that an optimizer step reads.  An expert without
    rows gets zeros, or stays as it is.
    """
    _check_operands(a, b)
    _need(a.codes.dim() == 2 and b.codes.dim() == 2, "a and b must be one matrix each")
    _check_offsets(offsets, a.device)
    c, made = _result(out, (offsets.numel() - 1, a.rows, b.rows), dtype, accumulate, a.device)
    if c.numel() == 0:
        return c
    if a.cols == 0:
        return c if accumulate else c.zero_()
    _enqueue(a.device, stream, [c] if made else [], L.muon_block_matmul, a.desc, b.desc, _c_desc(c),
             offsets.data_ptr(), L.PRODUCT_REDUCE, int(bool(accumulate)))
    return c
