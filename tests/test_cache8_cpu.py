"""The 8-bit record operators on a machine without a GPU: layouts, refusals
before any CUDA call, and the frequency tables."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

from host_offload_serving_gb300 import cache8, pages
from host_offload_serving_gb300 import hisparse as H

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x1000          # an aligned address that no refused call reads


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    pairs = [("hisparse_rotary_tensor", H.RotaryTensor), ("hisparse_rotary_args", H.RotaryArgs),
             ("hisparse_records", H.Records), ("hisparse_pack_args", H.PackArgs),
             ("hisparse_attend_args", H.AttendArgs), ("hisparse_page_pool", H.PagePool)]
    lines, want = [], []
    for name, cls in pairs:
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            cf = "store" if f == "store" else f
            lines.append(f'printf("%zu\\n", offsetof({name}, {cf}));')
            want.append(getattr(cls, f).offset)
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "hisparse.h"\nint main(void) {\n'
                    + "\n".join(lines) + "\nreturn 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.check_call([cc, "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)])
    got = [int(x) for x in subprocess.check_output([str(exe)], text=True).split()]
    assert got == want


# ---- rotary ------------------------------------------------------------------
def _rotary(**kw):
    a = H.RotaryArgs()
    a.dtype, a.rot_dim, a.tokens, a.amplitude = H.BF16, 64, 3, 1.0
    a.d_positions, a.d_turns = P, P
    t = a.t[0]
    t.x, t.y, t.heads, t.dim = P, P, 2, 128
    t.x_token_stride = t.y_token_stride = 256
    t.x_head_stride = t.y_head_stride = 128
    for k, v in kw.items():
        setattr(t if k in dict(H.RotaryTensor._fields_) else a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), H.EINVAL), (dict(rot_dim=0), H.EINVAL), (dict(rot_dim=63), H.EINVAL),
    (dict(rot_dim=130), H.EINVAL), (dict(offset=-2), H.EINVAL), (dict(offset=66), H.EINVAL),
    (dict(flags=4), H.EINVAL), (dict(tokens=-1), H.EINVAL), (dict(x=0), H.EINVAL),
    (dict(y=P + 1), H.EINVAL), (dict(heads=-1), H.EINVAL), (dict(d_positions=0), H.EINVAL),
    (dict(d_turns=0), H.EINVAL), (dict(x_token_stride=512), H.EINVAL),   # in place, two layouts
    (dict(rot_dim=16384, dim=16384), H.EBOUND),
    (dict(tokens=0), H.OK), (dict(heads=0), H.OK),
])
def test_rotary_refusals(kw, code):
    assert H.hisparse_rotary(_rotary(**kw), None) == code


def test_null_arguments_are_refused():
    lib = H.load()
    assert lib.hisparse_rotary(None, None) == H.EINVAL
    assert lib.hisparse_pack(None, None) == H.EINVAL
    assert lib.hisparse_attend(None, None) == H.EINVAL
    assert lib.hisparse_pages_compact(None, None) == H.EINVAL
    assert lib.hisparse_pages_free(None, None, 0, None) == H.EINVAL


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)),
                                        ("base", dict(factor=8.0)),
                                        ("parts", dict(factor=32.0, original_len=4096))])
def test_rotary_turns(scaling, kw):
    """The table's fractions are the frequencies over a turn, and position *
    turns mod 2^64 is the phase at any position."""
    rot = 64
    turns, amp = cache8.rotary_turns(rot, 10000.0, scaling, **kw)
    f = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    got = [(int(t) % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for t in turns]
    if scaling == "none":
        assert amp == 1.0
        assert all(abs(a - b) <= 1e-14 * b + 1e-18 for a, b in zip(got, f))
    if scaling == "linear":
        assert all(abs(a - b / 4) <= 1e-14 * b + 1e-18 for a, b in zip(got, f))
    if scaling == "base":       # the fastest pair stays, the slowest is divided by the factor
        assert abs(got[0] - 1.0) < 1e-14 and abs(got[-1] * 8 / f[-1] - 1) < 1e-9
    if scaling == "parts":
        assert abs(amp - (0.1 * math.log(32.0) + 1)) < 1e-12
        assert abs(got[0] - 1.0) < 1e-14 and abs(got[-1] * 32 / f[-1] - 1) < 1e-9
        mid = [i for i in range(rot // 2) if f[i] / 32 < got[i] * (1 - 1e-9) < f[i] * (1 - 2e-9)]
        assert mid and all(got[i] > got[i + 1] for i in range(rot // 2 - 1))
    p = 1048573
    ph = (p * (int(turns[1]) % 2 ** 64)) % 2 ** 64 / 2.0 ** 64
    exact = (p * got[1] / (2 * math.pi)) % 1.0
    assert min(abs(ph - exact), 1 - abs(ph - exact)) < 1e-8


def test_rotary_turns_refusals():
    for bad in (dict(rot_dim=3), dict(rot_dim=0), dict(rot_dim=8, factor=0.5),
                dict(rot_dim=8, scaling="parts"), dict(rot_dim=8, scaling="other")):
        with pytest.raises(ValueError):
            cache8.rotary_turns(**bad)


# ---- pack --------------------------------------------------------------------
def _pack(**kw):
    a = H.PackArgs()
    a.rec = H.Records(2, 64, 32, 0, 16)
    a.dtype, a.n, a.max_len, a.num_requests, a.scale_blocks = H.BF16, 1, 4, 1, 8
    a.headroom, a.tokens = 2.0, 4
    a.d_start, a.k, a.v, a.scales, a.dst = P, P, P, P, P
    a.k_token_stride, a.k_head_stride, a.v_token_stride, a.v_head_stride = 128, 64, 64, 32
    a.scales_req_stride, a.dst_rows, a.dst_row_stride = 32, 4, 192
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(rec=H.Records(0, 64, 32, 0, 16)), H.EINVAL), (dict(rec=H.Records(2, 60, 32, 0, 16)), H.EINVAL),
    (dict(rec=H.Records(2, 64, 8, 0, 16)), H.EINVAL), (dict(rec=H.Records(1, 64, 80, 1, 16)), H.EINVAL),
    (dict(rec=H.Records(2, 64, 32, 2, 16)), H.EINVAL), (dict(rec=H.Records(2, 64, 32, 0, 0)), H.EINVAL),
    (dict(rec=H.Records(1, 656, 32, 0, 16)), H.EBOUND), (dict(rec=H.Records(1, 64, 528, 0, 16)), H.EBOUND),
    (dict(rec=H.Records(2, 64, 32, 0, 5000)), H.EBOUND),
    (dict(dtype=-1), H.EINVAL), (dict(n=-1), H.EINVAL), (dict(max_len=0), H.EINVAL),
    (dict(headroom=0.5), H.EINVAL), (dict(headroom=float("nan")), H.EINVAL),
    (dict(d_start=0), H.EINVAL), (dict(k=0), H.EINVAL), (dict(v=0), H.EINVAL), (dict(k=P + 2), H.EINVAL),
    (dict(k_token_stride=130), H.EINVAL), (dict(dst=P + 8), H.EINVAL), (dict(dst_row_stride=176), H.EINVAL),
    (dict(tokens=3), H.EINVAL),                         # fewer than n * max_len
    (dict(dst_rows=3), H.EINVAL),                       # by token, too few rows
    (dict(d_blocks=P), H.EINVAL),                       # a page table without sizes
    (dict(rot_dim=8, d_turns=P), H.EINVAL), (dict(rot_dim=64, rot_offset=8, d_turns=P), H.EINVAL),
    (dict(rot_dim=16, rot_offset=4, d_turns=P), H.EINVAL), (dict(rot_dim=16), H.EINVAL),
    (dict(n=70000, d_cu_lens=P), H.EBOUND),
    (dict(n=0), H.OK), (dict(tokens=0), H.OK),
])
def test_pack_refusals(kw, code):
    assert H.hisparse_pack(_pack(**kw), None) == code


# ---- attend ------------------------------------------------------------------
def _attend(**kw):
    a = H.AttendArgs()
    a.rec = H.Records(2, 64, 64, 0, 16)
    a.dtype, a.num_requests, a.rows, a.entries, a.heads = H.BF16, 2, 1, 8, 4
    a.buffer_slots, a.record_tokens, a.softmax_scale, a.scale_blocks = 16, 1, 0.125, 4
    for f in ("q", "out", "d_sel", "d_slots", "hot", "scales"):
        setattr(a, f, P)
    a.q_row_stride, a.q_head_stride, a.out_row_stride, a.out_head_stride = 256, 64, 256, 64
    a.hot_req_stride, a.hot_row_stride, a.scales_req_stride = 17 * 256, 256, 16
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=H.F32), H.EINVAL), (dict(rows=0), H.EINVAL), (dict(entries=-1), H.EINVAL),
    (dict(heads=3), H.EINVAL), (dict(heads=0), H.EINVAL), (dict(record_tokens=0), H.EINVAL),
    (dict(scale_blocks=0), H.EINVAL), (dict(buffer_slots=-1), H.EINVAL),
    (dict(sel_block_tokens=3), H.EINVAL), (dict(sel_block_tokens=-1), H.EINVAL),
    (dict(q=0), H.EINVAL), (dict(out=0), H.EINVAL), (dict(hot=0), H.EINVAL), (dict(scales=0), H.EINVAL),
    (dict(d_slots=0), H.EINVAL), (dict(d_sel=0), H.EINVAL), (dict(q=P + 4), H.EINVAL),
    (dict(q_head_stride=65), H.EINVAL), (dict(hot_row_stride=240), H.EINVAL),
    (dict(hot_row_stride=264), H.EINVAL), (dict(record_tokens=2), H.EINVAL),   # row too short
    (dict(resident=P, resident_rows=3, resident_row_stride=128), H.EINVAL),
    (dict(resident_rows=-1), H.EINVAL), (dict(num_requests=-1), H.EINVAL),
    (dict(rec=H.Records(2, 656, 64, 0, 16)), H.EBOUND), (dict(num_requests=0), H.OK),
])
def test_attend_refusals(kw, code):
    assert H.hisparse_attend(_attend(**kw), None) == code


def test_wrappers_refuse_wrong_tensors():
    rec = cache8.Records(2, 64, 64, 16)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    sel = torch.zeros(2, 8, dtype=torch.int32)
    hot = torch.zeros(2, 17, 256, dtype=torch.uint8)
    sc = torch.zeros(2, 4, 4)
    out = torch.zeros_like(q)
    for bad in (dict(q=q.double()), dict(q=q[..., :32]), dict(sel=sel.long()), dict(slots=sel[:1]),
                dict(hot=hot.float()), dict(hot=hot[..., :128]), dict(scales=sc.double()),
                dict(scales=sc[..., :2]), dict(out=out.half()), dict(lse=torch.zeros(2, 1, 3)),
                dict(seq_lens=torch.zeros(3, dtype=torch.int32)),
                dict(resident=torch.zeros(3, 128, dtype=torch.uint8))):
        kw = dict(dict(q=q, sel=sel, slots=sel, hot=hot, scales=sc, out=out), **bad)
        with pytest.raises(ValueError):
            cache8.attend(rec, kw.pop("q"), kw.pop("sel"), kw.pop("slots"), kw.pop("hot"),
                          kw.pop("scales"), kw.pop("out"), stream=0, **kw)
    x = torch.zeros(3, 2, 64)
    turns = torch.zeros(16, dtype=torch.int64)
    pos = torch.zeros(3, dtype=torch.int32)
    for a, kw in (((x.int(), pos, turns), {}), ((x, pos[:2], turns), {}), ((x, pos.long(), turns), {}),
                  ((x, pos, turns.int()), {}), ((x, pos, turns), dict(out=x[:, :1])),
                  ((x, pos, turns), dict(k=x.half())), ((x.transpose(1, 2), pos, turns), {})):
        with pytest.raises(ValueError):
            cache8.rotate(*a, stream=0, **kw)
    k = torch.zeros(3, 2, 64)
    dst = torch.zeros(3, 256, dtype=torch.uint8)
    st = torch.zeros(1, dtype=torch.int32)
    for kw in (dict(k=k[:, :1]), dict(v=None), dict(v=k.half()), dict(dst=dst[:, :128]),
               dict(dst=dst.int()), dict(scales=sc[..., :2]), dict(start=st.long()),
               dict(start=torch.zeros(3, dtype=torch.int32))):
        kw = dict(dict(k=k, v=k, dst=dst, scales=sc, start=st), **kw)
        with pytest.raises(ValueError):
            cache8.pack(rec, kw["k"], kw["v"], kw["dst"], kw["scales"], kw["start"], max_len=3, stream=0)


# ---- pages -------------------------------------------------------------------
def _pool(**kw):
    p = H.PagePool(8, 2, 4, 16, 1, 64, P, 8 * 1024, 1024, P, P, P, None)
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@pytest.mark.parametrize("kw,code", [
    (dict(num_pages=0), H.EINVAL), (dict(num_requests=0), H.EINVAL), (dict(max_blocks=0), H.EINVAL),
    (dict(page_tokens=0), H.EINVAL), (dict(layers=0), H.EINVAL), (dict(row_bytes=24), H.EINVAL),
    (dict(store=0), H.EINVAL), (dict(store=P + 8), H.EINVAL), (dict(d_tables=0), H.EINVAL),
    (dict(d_refs=0), H.EINVAL), (dict(d_refs=P + 4), H.EINVAL), (dict(d_work=0), H.EINVAL),
    (dict(page_stride=1000), H.EINVAL), (dict(page_stride=512), H.EINVAL),
    (dict(layer_stride=-16), H.EINVAL), (dict(num_requests=9000), H.EBOUND),
])
def test_pages_refusals(kw, code):
    p = _pool(**kw)
    assert H.hisparse_pages_compact(p, None) == code
    assert H.hisparse_pages_grow(p, P, P, 1, None) == code
    assert H.hisparse_pages_fork(p, P, P, P, 1, None) == code
    assert H.hisparse_pages_free(p, P, 1, None) == code


def test_pages_list_refusals():
    p = _pool()
    assert H.hisparse_pages_grow(p, None, P, 1, None) == H.EINVAL
    assert H.hisparse_pages_grow(p, P, P, 3, None) == H.EBOUND          # more than requests
    assert H.hisparse_pages_fork(p, P, None, P, 1, None) == H.EINVAL
    assert H.hisparse_pages_fork(p, P, P, P, -1, None) == H.EINVAL
    assert H.hisparse_pages_free(p, None, 2, None) == H.EINVAL
    assert H.hisparse_pages_grow(p, None, None, 0, None) == H.OK
    assert H.hisparse_pages_work_ints(0, 4) == -1 and H.hisparse_pages_work_ints(8, 9000) == -1
    assert H.hisparse_pages_work_ints(8, 4) > 24
    with pytest.raises(ValueError):
        pages.PagePool(torch.zeros(1, 4, 60, dtype=torch.uint8), requests=2, max_blocks=2, block_tokens=16)
