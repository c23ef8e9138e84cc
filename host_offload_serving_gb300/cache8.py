"""8-bit records around RESOLVE: rotary positions, packing and sparse attention.

``Records``       what a record of e4m3 bytes holds (heads, sizes, scale blocks).
``rotary_turns``  the frequency table of ``rotate`` and ``pack`` with the usual
                  scalings for long contexts.
``rotate``        rotary positions of q and k (``hisparse_rotary``).
``pack``          K and V of new tokens into records and their scales
                  (``hisparse_pack``): a decode step's ``new_rows``, or a
                  prompt's rows of a host pool, mirror or resident store.
``attend``        attention over the rows that a slot vector names
                  (``hisparse_attend``).

Each call checks its tensors' types, shapes and places here and everything else in the
C library, launches on the current stream (or ``stream``) and returns at once;
none allocates, so all can be captured in a CUDA graph.  ``status`` (an int32
tensor of one element, optional) collects the ERR_* bits of device-side inputs.
"""
import ctypes
import math

import torch

from . import hisparse as H
from .runtime import _stream

# (a third of the time of torch.cuda.current_device, for tensors that CUDA has already)
_cuda_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)

_DTYPES = {torch.bfloat16: H.BF16, torch.float16: H.F16, torch.float32: H.F32}


def _dtype(t, what):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"{what}: bfloat16, float16 or float32 expected, got {t.dtype}") from None


def _need(ok, message):
    if not ok:
        raise ValueError(message)


def _i32(t, what, numel=None):
    if t is None:
        return 0
    if t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous int32 tensor expected")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{what}: {numel} values expected, got {t.numel()}")
    return t.data_ptr()


def _reach(what, first, *others):
    """Raises unless the current CUDA device reads every tensor (or None) where it lies: on that
    device, or in pinned host memory."""
    dev = first.get_device()
    if dev >= 0 and dev == _cuda_device():
        for t in others:
            if t is not None and t.get_device() != dev:
                break
        else:
            return
    for t in (first, *others):
        if t is None or (t.is_cuda and t.get_device() == torch.cuda.current_device()) \
                or (t.device.type == "cpu" and t.is_pinned()):
            continue
        raise ValueError(f"{what}: a tensor of shape {tuple(t.shape)} is on {t.device}; all are on the "
                         "current CUDA device, or in pinned host memory")


def _turns(turns, what):
    if turns.dtype is not torch.int64 or not turns.is_contiguous():
        raise ValueError(f"{what}: turns is a contiguous int64 tensor")
    return turns.data_ptr()


class Records:
    """Layout of a token's record: ``kv_heads`` K heads of ``k_dim`` e4m3 bytes
    and as many V heads of ``v_dim``, or (``latent``) K heads whose first
    ``v_dim`` values are V too.  One float32 scale for every ``block_tokens``
    positions of each head."""

    def __init__(self, kv_heads, k_dim, v_dim, block_tokens, latent=False):
        self.kv_heads, self.k_dim, self.v_dim = int(kv_heads), int(k_dim), int(v_dim)
        self.block_tokens, self.latent = int(block_tokens), bool(latent)
        self.columns = self.kv_heads * (1 if latent else 2)
        self.row_bytes = self.kv_heads * (self.k_dim + (0 if latent else self.v_dim))
        self.c = (self.kv_heads, self.k_dim, self.v_dim, int(self.latent), self.block_tokens)

    def blocks(self, positions):
        """Scale blocks that ``positions`` positions need."""
        return -(-int(positions) // self.block_tokens)


def rotary_turns(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0,
                 fast_turns=32.0, slow_turns=1.0):
    """(turns, amplitude): pair i of ``rot_dim / 2`` turns by base^(-2i/rot_dim)
    radians per position, as 64-bit binary fractions of a turn (a CPU int64 tensor).

    scaling "none"; "linear": positions interpolated, frequencies / factor;
    "base": the base grows with the factor, so the slowest pair is
    interpolated and the fastest is not; "parts": pairs that make at least
    ``fast_turns`` turns over ``original_len`` positions keep their frequency,
    those that make fewer than ``slow_turns`` are divided by the factor, a linear ramp
    between, and the amplitude is 0.1 ln(factor) + 1."""
    _need(rot_dim >= 2 and rot_dim % 2 == 0, "rotary_turns: rot_dim is even and at least 2")
    _need(factor >= 1.0 and base > 1.0, "rotary_turns: factor >= 1 and base > 1")
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freqs = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    amplitude = 1.0
    if scaling == "linear":
        freqs = [f / factor for f in freqs]
    elif scaling == "parts":
        _need(original_len > 0 and fast_turns > slow_turns,
              "rotary_turns: \"parts\" needs original_len and fast_turns > slow_turns")
        for i, f in enumerate(freqs):
            made = original_len * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (made - slow_turns) / (fast_turns - slow_turns)))
            freqs[i] = f * keep + f / factor * (1.0 - keep)
        amplitude = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "base"):
        raise ValueError(f"rotary_turns: unknown scaling {scaling!r}")
    raw = [int(round(f / (2 * math.pi) * 2.0 ** 64)) & (2 ** 64 - 1) for f in freqs]
    return torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in raw],
                        dtype=torch.int64), amplitude


def _rotary_tensor(x, y, tokens, what):
    """The fields of one rotated tensor."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != tokens or (y is not x and (shape != y.shape or x.dtype is not y.dtype)):
        raise ValueError(f"rotate: {what} and its output are [tokens][heads][dim] of one type")
    xs = x.stride()
    ys = xs if y is x else y.stride()
    if xs[2] != 1 or ys[2] != 1:
        raise ValueError(f"rotate: the values of a head of {what} are contiguous")
    return x.data_ptr(), y.data_ptr(), xs[0], xs[1], ys[0], ys[1], shape[1], shape[2]


_NO_TENSOR = (0,) * 8


def rotate(x, positions, turns, *, k=None, out=None, k_out=None, offset=0, interleaved=False,
           inverse=False, amplitude=1.0, stream=None):
    """Rotary positions of ``x`` [tokens][heads][dim], and of ``k`` in the same
    launch: values [offset, offset + 2 * len(turns)) of each head.  Without
    ``out`` in place.  ``positions`` int32 [tokens]; ``turns`` int64 on the
    device.  ``inverse`` turns back (the gradient of a rotation).  Strided views are taken as they
    are.  Returns (out, k_out)."""
    out = x if out is None else out
    dtype = _dtype(x, "rotate")
    tokens = x.shape[0]
    first, second = _rotary_tensor(x, out, tokens, "x"), _NO_TENSOR
    if k is not None:
        k_out = k if k_out is None else k_out
        _need(k.dtype is x.dtype, "rotate: x and k are of one type")
        second = _rotary_tensor(k, k_out, tokens, "k")
    d_turns, d_pos = _turns(turns, "rotate"), _i32(positions, "rotate: positions", tokens)
    _reach("rotate", x, positions, turns, out, k, k_out)
    flags = (H.ROTARY_INTERLEAVED if interleaved else 0) | (H.ROTARY_INVERSE if inverse else 0)
    a = H.pack_rotary(dtype, 2 * turns.numel(), offset, flags, tokens, amplitude,
                      d_pos, d_turns, *first, *second)
    H.check(H.hisparse_rotary(a, _stream(stream)), "hisparse_rotary")
    return out, k_out


def pack(rec, k, v, dst, scales, start, *, cu_lens=None, reqs=None, max_len=1, headroom=2.0,
         turns=None, rot_offset=0, interleaved=False, amplitude=1.0, blocks=None, page_tokens=0,
         status=None, stream=None):
    """Pack tokens ``k`` [tokens][kv_heads][k_dim] and ``v`` (None when latent)
    into e4m3 rows and their scales [R][blocks][columns] (updated in place).

    Sequence i holds tokens cu_lens[i] .. cu_lens[i+1] - 1 (``max_len`` each
    without ``cu_lens``), begins at position start[i] and belongs to request
    reqs[i] (i).  ``dst`` uint8: [tokens][row_bytes], row t for token t;
    [R][P][row_bytes], by position; or, with the page table ``blocks`` int32
    [R][max_blocks], a store [rows][row_bytes] of pages of ``page_tokens`` rows.  ``turns``:
    K is rotated on the way.  See hisparse_pack for the scales."""
    dtype = _dtype(k, "pack")
    shape, ks = k.shape, k.stride()
    if len(shape) != 3 or shape[1] != rec.kv_heads or shape[2] != rec.k_dim or ks[2] != 1:
        raise ValueError("pack: k is [tokens][kv_heads][k_dim]")
    tokens = shape[0]
    v_ptr, vs = 0, (0, 0)
    if not rec.latent:
        if v is None or v.shape != (tokens, rec.kv_heads, rec.v_dim) or v.dtype is not k.dtype \
                or v.stride(2) != 1:
            raise ValueError("pack: v is [tokens][kv_heads][v_dim] of k's type")
        v_ptr, vs = v.data_ptr(), v.stride()
    elif v is not None:
        raise ValueError("pack: a latent record has no v")
    cs, ss = scales.shape, scales.stride()
    if scales.dtype is not torch.float32 or len(cs) != 3 or cs[2] != rec.columns or ss[2] != 1 \
            or ss[1] != rec.columns:
        raise ValueError("pack: scales are float32 [R][blocks][columns]")
    n, R = start.numel(), cs[0]
    _need(reqs is not None or n <= R, "pack: more sequences than requests")
    rows, ds = dst.shape, dst.stride()
    if dst.dtype is not torch.uint8 or not 2 <= len(rows) <= 3 or rows[-1] != rec.row_bytes or ds[-1] != 1:
        raise ValueError("pack: dst is uint8 [rows][row_bytes] or [R][P][row_bytes]")
    req_stride = table = max_blocks = 0
    if len(rows) == 3:
        if rows[0] != R or blocks is not None:
            raise ValueError("pack: dst by position is [R][P][row_bytes], without a page table")
        if R > 1 and ds[0] == 0:
            raise ValueError("pack: dst by position has rows of its own for each request")
        req_stride = ds[0] if R > 1 else max(16, ds[0])  # (one request goes by position too)
    if blocks is not None:
        table, max_blocks = _i32(blocks, "pack: blocks"), blocks.shape[1]
        _need(blocks.shape[0] == R, "pack: blocks is [R][max_blocks]")
    else:
        page_tokens = 0
    rot = (0, 0, 0, 0.0, 0)
    if turns is not None:
        rot = (2 * turns.numel(), rot_offset, H.ROTARY_INTERLEAVED if interleaved else 0, amplitude,
               _turns(turns, "pack"))
    lists = (_i32(cu_lens, "pack: cu_lens", n + 1), _i32(start, "pack: start"), _i32(reqs, "pack: reqs", n),
             _i32(status, "pack: status"))
    _reach("pack", k, v, dst, scales, start, cu_lens, reqs, blocks, turns, status)
    a = H.pack_pack(*rec.c, dtype, n, max_len, R, cs[1], headroom, *lists[:3], tokens, k.data_ptr(), v_ptr,
                    ks[0], ks[1], vs[0], vs[1], scales.data_ptr(), ss[0], dst.data_ptr(), rows[-2], ds[-2],
                    req_stride, table, max_blocks, page_tokens, *rot, lists[3])
    H.check(H.hisparse_pack(a, _stream(stream)), "hisparse_pack")
    return dst


def attend(rec, q, sel, slots, hot, scales, out, *, softmax_scale=None, lse=None, record_tokens=1,
           sel_block_tokens=1, seq_lens=None, resident=None, num_reqs=None, status=None,
           stream=None):
    """Attention of ``q`` [R][rows][heads][k_dim] over the records that ``slots``
    [R][rows * entries] (RESOLVE's output for ``sel``) names in ``hot``
    [R][B + 1][record_tokens * row_bytes] and ``resident`` [rows][same], into
    ``out`` [R][rows][heads][v_dim]; ``lse`` float32 [R][rows][heads] optional.
    ``scales`` [R][blocks][columns].  See hisparse_attend."""
    dtype = _dtype(q, "attend")
    shape, to = q.shape, out.shape
    if len(shape) != 4 or shape[3] != rec.k_dim or len(to) != 4 or to[:3] != shape[:3] \
            or to[3] != rec.v_dim or out.dtype is not q.dtype:
        raise ValueError("attend: q is [R][rows][heads][k_dim], out [R][rows][heads][v_dim], of one type")
    R, rows, heads, _ = shape
    qs, os = q.stride(), out.stride()
    if qs[3] != 1 or os[3] != 1 or (rows > 1 and R > 1 and (qs[0] != rows * qs[1] or os[0] != rows * os[1])):
        raise ValueError("attend: q and out have one stride from row to row, and contiguous heads")
    by = 0 if rows == 1 else 1
    listed = slots.shape
    if len(listed) != 2 or listed[0] != R or listed[1] % rows:
        raise ValueError("attend: slots is [R][rows * entries]")
    d_slots = _i32(slots, "attend: slots")
    d_sel = _i32(sel, "attend: sel", R * listed[1] // max(1, sel_block_tokens))
    hot_shape, hs = hot.shape, hot.stride()
    if hot.dtype is not torch.uint8 or len(hot_shape) != 3 or hot_shape[0] != R or hs[2] != 1 \
            or hot_shape[2] != record_tokens * rec.row_bytes:
        raise ValueError("attend: hot is uint8 [R][B + 1][record_tokens * row_bytes]")
    store = (0, 0, 0)
    if resident is not None:
        if resident.dtype is not torch.uint8 or resident.dim() != 2 or resident.stride(1) != 1 \
                or resident.shape[1] != hot_shape[2]:
            raise ValueError("attend: resident is uint8 [rows][record_tokens * row_bytes]")
        store = (resident.data_ptr(), resident.shape[0], resident.stride(0))
    cs, ss = scales.shape, scales.stride()
    if scales.dtype is not torch.float32 or len(cs) != 3 or cs[0] != R or cs[2] != rec.columns \
            or ss[2] != 1 or ss[1] != rec.columns:
        raise ValueError("attend: scales are float32 [R][blocks][columns]")
    if lse is not None and (lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.shape != shape[:3]):
        raise ValueError("attend: lse is float32 [R][rows][heads]")
    lists = (_i32(seq_lens, "attend: seq_lens", R), _i32(num_reqs, "attend: num_reqs", 1),
             _i32(status, "attend: status"))
    _reach("attend", q, sel, slots, hot, scales, out, lse, seq_lens, resident, num_reqs, status)
    a = H.pack_attend(*rec.c, dtype, R, rows, listed[1] // rows, heads, hot_shape[1] - 1, record_tokens,
                      sel_block_tokens, rec.k_dim ** -0.5 if softmax_scale is None else softmax_scale,
                      q.data_ptr(), qs[by], qs[2], out.data_ptr(), os[by], os[2],
                      0 if lse is None else lse.data_ptr(), d_sel, d_slots, hot.data_ptr(), hs[0], hs[1],
                      *store, scales.data_ptr(), ss[0], cs[1], *lists)
    H.check(H.hisparse_attend(a, _stream(stream)), "hisparse_attend")
    return out
