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

Each call checks its tensors' types and shapes here and everything else in the
C library, launches on the current stream (or ``stream``) and returns at once;
none allocates, so all can be captured in a CUDA graph.  ``status`` (an int32
tensor of one element, optional) collects the ERR_* bits of device-side inputs.
"""
import ctypes
import math

import torch

from . import hisparse as H
from .runtime import _stream

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
        return None
    if t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{what}: a contiguous int32 tensor expected")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{what}: {numel} values expected, got {t.numel()}")
    return t.data_ptr()


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
        self.c = H.Records(self.kv_heads, self.k_dim, self.v_dim, int(self.latent),
                           self.block_tokens)

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


def _rotary_tensor(t, x, y, tokens, what):
    if x.dim() != 3 or x.shape[0] != tokens or x.shape != y.shape or x.dtype is not y.dtype:
        raise ValueError(f"rotate: {what} and its output are [tokens][heads][dim] of one type")
    xs, ys = x.stride(), y.stride()
    if xs[2] != 1 or ys[2] != 1:
        raise ValueError(f"rotate: the values of a head of {what} are contiguous")
    t.x, t.y = x.data_ptr(), y.data_ptr()
    t.x_token_stride, t.x_head_stride = xs[0], xs[1]
    t.y_token_stride, t.y_head_stride = ys[0], ys[1]
    t.heads, t.dim = x.shape[1], x.shape[2]


def rotate(x, positions, turns, *, k=None, out=None, k_out=None, offset=0, interleaved=False,
           inverse=False, amplitude=1.0, stream=None):
    """Rotary positions of ``x`` [tokens][heads][dim], and of ``k`` in the same
    launch: values [offset, offset + 2 * len(turns)) of each head.  Without
    ``out`` in place.  ``positions`` int32 [tokens]; ``turns`` int64 on the
    device.  ``inverse`` turns back (the gradient of a rotation).  Strided views are taken as they
    are.  Returns (out, k_out)."""
    a = H.RotaryArgs()
    out = x if out is None else out
    a.dtype = _dtype(x, "rotate")
    a.tokens = x.shape[0]
    _rotary_tensor(a.t[0], x, out, a.tokens, "x")
    if k is not None:
        k_out = k if k_out is None else k_out
        _need(k.dtype is x.dtype, "rotate: x and k are of one type")
        _rotary_tensor(a.t[1], k, k_out, a.tokens, "k")
    if turns.dtype is not torch.int64 or not turns.is_contiguous():
        raise ValueError("rotate: turns is a contiguous int64 tensor")
    a.rot_dim, a.offset, a.amplitude = 2 * turns.numel(), offset, amplitude
    a.flags = (H.ROTARY_INTERLEAVED if interleaved else 0) | (H.ROTARY_INVERSE if inverse else 0)
    a.d_positions, a.d_turns = _i32(positions, "rotate: positions", a.tokens), turns.data_ptr()
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
    a = H.PackArgs()
    a.rec = rec.c
    a.dtype = _dtype(k, "pack")
    a.tokens = k.shape[0]
    ks = k.stride()
    if k.dim() != 3 or k.shape[1] != rec.kv_heads or k.shape[2] != rec.k_dim or ks[2] != 1:
        raise ValueError("pack: k is [tokens][kv_heads][k_dim]")
    a.k, a.k_token_stride, a.k_head_stride = k.data_ptr(), ks[0], ks[1]
    if not rec.latent:
        if v is None or v.shape != (a.tokens, rec.kv_heads, rec.v_dim) or v.dtype is not k.dtype \
                or v.stride(2) != 1:
            raise ValueError("pack: v is [tokens][kv_heads][v_dim] of k's type")
        a.v, a.v_token_stride, a.v_head_stride = v.data_ptr(), v.stride(0), v.stride(1)
    elif v is not None:
        raise ValueError("pack: a latent record has no v")
    if scales.dtype is not torch.float32 or scales.dim() != 3 or scales.shape[2] != rec.columns \
            or scales.stride(2) != 1 or scales.stride(1) != rec.columns:
        raise ValueError("pack: scales are float32 [R][blocks][columns]")
    a.n, a.max_len, a.headroom = start.numel(), max_len, headroom
    a.num_requests, a.scale_blocks = scales.shape[0], scales.shape[1]
    a.scales, a.scales_req_stride = scales.data_ptr(), scales.stride(0)
    a.d_start = _i32(start, "pack: start")
    a.d_cu_lens = _i32(cu_lens, "pack: cu_lens", a.n + 1)
    a.d_reqs = _i32(reqs, "pack: reqs", a.n)
    if reqs is None:
        _need(a.n <= a.num_requests, "pack: more sequences than requests")
    ds = dst.stride()
    if dst.dtype is not torch.uint8 or dst.shape[-1] != rec.row_bytes or ds[-1] != 1:
        raise ValueError("pack: dst is uint8 [..][row_bytes]")
    a.dst, a.dst_rows, a.dst_row_stride = dst.data_ptr(), dst.shape[-2], ds[-2]
    if dst.dim() == 3:
        if dst.shape[0] != a.num_requests or blocks is not None:
            raise ValueError("pack: dst by position is [R][P][row_bytes], without a page table")
        # one request, or an expanded one, still goes by position
        a.dst_req_stride = ds[0] if dst.shape[0] > 1 else max(16, ds[0])
    if blocks is not None:
        a.d_blocks = _i32(blocks, "pack: blocks")
        _need(blocks.shape[0] == a.num_requests, "pack: blocks is [R][max_blocks]")
        a.max_blocks, a.page_tokens = blocks.shape[1], page_tokens
    if turns is not None:
        a.rot_dim, a.rot_offset, a.amplitude = 2 * turns.numel(), rot_offset, amplitude
        a.rot_flags = H.ROTARY_INTERLEAVED if interleaved else 0
        a.d_turns = turns.data_ptr()
    a.d_status = _i32(status, "pack: status")
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
    a = H.AttendArgs()
    a.rec = rec.c
    a.dtype = _dtype(q, "attend")
    if q.dim() != 4 or q.shape[3] != rec.k_dim or out.dim() != 4 or out.shape[:3] != q.shape[:3] \
            or out.shape[3] != rec.v_dim or out.dtype is not q.dtype:
        raise ValueError("attend: q is [R][rows][heads][k_dim], out [R][rows][heads][v_dim], of one type")
    R, rows, heads, _ = q.shape
    qs, os = q.stride(), out.stride()
    if qs[3] != 1 or os[3] != 1 or (rows > 1 and R > 1 and (qs[0] != rows * qs[1] or os[0] != rows * os[1])):
        raise ValueError("attend: q and out have one stride from row to row, and contiguous heads")
    a.num_requests, a.rows, a.heads = R, rows, heads
    by = 0 if rows == 1 else 1
    a.q, a.q_row_stride, a.q_head_stride = q.data_ptr(), qs[by], qs[2]
    a.out, a.out_row_stride, a.out_head_stride = out.data_ptr(), os[by], os[2]
    if slots.dim() != 2 or slots.shape[0] != R or slots.shape[1] % rows:
        raise ValueError("attend: slots is [R][rows * entries]")
    a.entries = slots.shape[1] // rows
    a.sel_block_tokens = sel_block_tokens
    a.d_slots = _i32(slots, "attend: slots")
    a.d_sel = _i32(sel, "attend: sel", slots.numel() // max(1, sel_block_tokens))
    hs = hot.stride()
    if hot.dtype is not torch.uint8 or hot.dim() != 3 or hot.shape[0] != R or hs[2] != 1 \
            or hot.shape[2] != record_tokens * rec.row_bytes:
        raise ValueError("attend: hot is uint8 [R][B + 1][record_tokens * row_bytes]")
    a.buffer_slots, a.record_tokens = hot.shape[1] - 1, record_tokens
    a.hot, a.hot_req_stride, a.hot_row_stride = hot.data_ptr(), hs[0], hs[1]
    if resident is not None:
        if resident.dtype is not torch.uint8 or resident.dim() != 2 or resident.stride(1) != 1 \
                or resident.shape[1] != hot.shape[2]:
            raise ValueError("attend: resident is uint8 [rows][record_tokens * row_bytes]")
        a.resident, a.resident_rows = resident.data_ptr(), resident.shape[0]
        a.resident_row_stride = resident.stride(0)
    if scales.dtype is not torch.float32 or scales.dim() != 3 or scales.shape[0] != R \
            or scales.shape[2] != rec.columns or scales.stride(2) != 1 \
            or scales.stride(1) != rec.columns:
        raise ValueError("attend: scales are float32 [R][blocks][columns]")
    a.scales, a.scales_req_stride, a.scale_blocks = scales.data_ptr(), scales.stride(0), scales.shape[1]
    if lse is not None:
        if lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.shape != q.shape[:3]:
            raise ValueError("attend: lse is float32 [R][rows][heads]")
        a.lse = lse.data_ptr()
    a.softmax_scale = rec.k_dim ** -0.5 if softmax_scale is None else softmax_scale
    a.d_seq_lens = _i32(seq_lens, "attend: seq_lens", R)
    a.d_num_reqs = _i32(num_reqs, "attend: num_reqs", 1)
    a.d_status = _i32(status, "attend: status")
    H.check(H.hisparse_attend(a, _stream(stream)), "hisparse_attend")
    return out
