"""Python binding of the C ABI in ``include/hisparse.h`` (argument marshalling only).

Every function keeps the C name and takes plain integers for pointers and
streams (``tensor.data_ptr()``, ``torch.cuda.Stream.cuda_stream``).  Nothing
here computes any part of RESOLVE: all of it runs in ``libhisparse.so``.  If the
library cannot be built or loaded the import fails -- there is no fallback.
"""
import ctypes
import os
import struct

from . import _build

OK, EINVAL, EBOUND, ENOMEM, ECUDA, EROLE = 0, -1, -2, -3, -4, -5
ERR_RANGE, ERR_DUP, ERR_FULL, ERR_WAIT = 1, 2, 4, 8
RECORD_PLAN, SKIP_IO, FROM_MIRROR, UNION, WITH_SHARED = 1, 2, 4, 8, 16
LOOKUP_PAGE_TABLE, LOOKUP_HASH = 0, 1
HOST_HUGE, HOST_PINNED = 0, 1
BF16, F16, F32 = 0, 1, 2
ROTARY_INTERLEAVED, ROTARY_INVERSE = 1, 2

_i32, _i64, _u32, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p
_f32 = ctypes.c_float


class Config(ctypes.Structure):
    _fields_ = [("num_requests", _i32), ("num_layers", _i32), ("top_k", _i32),
                ("buffer_slots", _i32), ("host_rows", _i64), ("record_bytes", _i32),
                ("ctas_per_request", _i32), ("replay_ctas", _i32), ("lookup", _i32),
                ("anchor_of", _vp)]


class LayerBuffers(ctypes.Structure):
    _fields_ = [("host_pool", _vp), ("host_req_stride", _i64), ("host_row_stride", _i64),
                ("hot", _vp), ("hot_req_stride", _i64), ("hot_row_stride", _i64),
                ("mirror", _vp)]


class Info(ctypes.Structure):
    _fields_ = [("ctas_per_request", _i32), ("threads_per_cta", _i32), ("smem_bytes", _i32),
                ("hash_capacity", _i32), ("replay_ctas", _i32), ("sm_count", _i32),
                ("metadata_bytes", _i64), ("lookup", _i32)]


class RotaryTensor(ctypes.Structure):
    _fields_ = [("x", _vp), ("y", _vp), ("x_token_stride", _i64), ("x_head_stride", _i64),
                ("y_token_stride", _i64), ("y_head_stride", _i64), ("heads", _i32), ("dim", _i32)]


class RotaryArgs(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("rot_dim", _i32), ("offset", _i32), ("flags", _u32),
                ("tokens", _i64), ("amplitude", _f32), ("d_positions", _vp), ("d_turns", _vp),
                ("t", RotaryTensor * 2)]


class Records(ctypes.Structure):
    _fields_ = [("kv_heads", _i32), ("k_dim", _i32), ("v_dim", _i32), ("latent", _i32),
                ("block_tokens", _i32)]


class PackArgs(ctypes.Structure):
    _fields_ = [("rec", Records), ("dtype", _i32), ("n", _i32), ("max_len", _i32),
                ("num_requests", _i32), ("scale_blocks", _i32), ("headroom", _f32),
                ("d_cu_lens", _vp), ("d_start", _vp), ("d_reqs", _vp), ("tokens", _i64),
                ("k", _vp), ("v", _vp), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_token_stride", _i64), ("v_head_stride", _i64), ("scales", _vp),
                ("scales_req_stride", _i64), ("dst", _vp), ("dst_rows", _i64),
                ("dst_row_stride", _i64), ("dst_req_stride", _i64), ("d_blocks", _vp),
                ("max_blocks", _i32), ("page_tokens", _i32), ("rot_dim", _i32),
                ("rot_offset", _i32), ("rot_flags", _u32), ("amplitude", _f32), ("d_turns", _vp),
                ("d_status", _vp)]


class AttendArgs(ctypes.Structure):
    _fields_ = [("rec", Records), ("dtype", _i32), ("num_requests", _i32), ("rows", _i32),
                ("entries", _i32), ("heads", _i32), ("buffer_slots", _i32),
                ("record_tokens", _i32), ("sel_block_tokens", _i32), ("softmax_scale", _f32),
                ("q", _vp), ("q_row_stride", _i64), ("q_head_stride", _i64), ("out", _vp),
                ("out_row_stride", _i64), ("out_head_stride", _i64), ("lse", _vp),
                ("d_sel", _vp), ("d_slots", _vp), ("hot", _vp), ("hot_req_stride", _i64),
                ("hot_row_stride", _i64), ("resident", _vp), ("resident_rows", _i64),
                ("resident_row_stride", _i64), ("scales", _vp), ("scales_req_stride", _i64),
                ("scale_blocks", _i32), ("d_seq_lens", _vp), ("d_num_reqs", _vp),
                ("d_status", _vp)]


class PagePool(ctypes.Structure):
    _fields_ = [("num_pages", _i32), ("num_requests", _i32), ("max_blocks", _i32),
                ("page_tokens", _i32), ("layers", _i32), ("row_bytes", _i64), ("store", _vp),
                ("layer_stride", _i64), ("page_stride", _i64), ("d_tables", _vp),
                ("d_refs", _vp), ("d_work", _vp), ("d_status", _vp)]


def packer(cls):
    """The values of a structure, in the order of its fields and theirs, into its bytes: a quarter of
    the time that setting them one by one takes."""
    codes = {_i32: "i", _u32: "I", _i64: "q", _f32: "f", _vp: "P"}

    def code(t):
        if issubclass(t, ctypes.Array):
            return code(t._type_) * t._length_
        if issubclass(t, ctypes.Structure):
            return "".join(code(f) for _, f in t._fields_)
        return codes[t]
    s = struct.Struct(code(cls) + "0q")
    assert s.size == ctypes.sizeof(cls)
    return s.pack


pack_rotary, pack_pack, pack_attend = packer(RotaryArgs), packer(PackArgs), packer(AttendArgs)

# (name, restype, argtypes) of every exported symbol, in header order
SIGNATURES = [
    ("hisparse_init", _i32, [ctypes.POINTER(Config), ctypes.POINTER(LayerBuffers),
                             ctypes.POINTER(_vp)]),
    ("hisparse_destroy", _i32, [_vp]),
    ("hisparse_resolve", _i32, [_vp, _i32, _vp, _vp, _vp, _vp, _u32, _vp]),
    ("hisparse_resolve_step", _i32, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _u32, _vp]),
    ("hisparse_resolve_resident", _i32, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _vp,
                                         _u32, _vp]),
    ("hisparse_resolve_ex", _i32, [_vp, _i32, _vp, _vp, _vp, _vp, _vp, _u32, _vp]),
    ("hisparse_admit", _i32, [_vp, _i32, _vp, _i32, _vp, _vp]),
    ("hisparse_writeback", _i32, [_vp, _i32, _vp, _vp, _vp, _vp]),
    ("hisparse_prefetch_plan", _i32, [_vp, _i32, _i32, _vp, _vp]),
    ("hisparse_copy", _i32, [_vp, _vp, _i64, _vp]),
    ("hisparse_copy_miss_counts", _i32, [_vp, _i32, _vp, _vp]),
    ("hisparse_get_status", _i32, [_vp, ctypes.POINTER(_u32), _vp]),
    ("hisparse_export_state", _i32, [_vp, _i32, _vp, _vp, _vp, _vp]),
    ("hisparse_import_state", _i32, [_vp, _i32, _vp, _vp, _vp, _vp]),
    ("hisparse_export_plan", _i32, [_vp, _i32, _vp, _vp, _vp]),
    ("hisparse_reset", _i32, [_vp, _i32, _vp]),
    ("hisparse_set_l2_persisting", _i32, [_vp, _i64]),
    ("hisparse_rotary", _i32, [_vp, _vp]),
    ("hisparse_pack", _i32, [_vp, _vp]),
    ("hisparse_attend", _i32, [_vp, _vp]),
    ("hisparse_pages_work_ints", _i64, [_i32, _i32]),
    ("hisparse_pages_grow", _i32, [ctypes.POINTER(PagePool), _vp, _vp, _i32, _vp]),
    ("hisparse_pages_fork", _i32, [ctypes.POINTER(PagePool), _vp, _vp, _vp, _i32, _vp]),
    ("hisparse_pages_free", _i32, [ctypes.POINTER(PagePool), _vp, _i32, _vp]),
    ("hisparse_pages_compact", _i32, [ctypes.POINTER(PagePool), _vp]),
    ("hisparse_get_info", _i32, [_vp, ctypes.POINTER(Info)]),
    ("hisparse_host_alloc", _i32, [ctypes.c_size_t, ctypes.POINTER(_vp)]),
    ("hisparse_host_free", _i32, [_vp]),
    ("hisparse_host_alloc_kind", _i32, [ctypes.c_size_t, _i32, ctypes.POINTER(_vp)]),
    ("hisparse_host_hugepage_bytes", _i32, [_vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t)]),
    ("hisparse_last_cuda_error", _i32, []),
    ("hisparse_strerror", ctypes.c_char_p, [_i32]),
]

_lib = None


def load(path=None):
    """Build (if stale) and load libhisparse.so; raises if that is impossible."""
    global _lib
    if _lib is None:
        path = path or _build.build()
        lib = ctypes.CDLL(path)
        for name, res, args in SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def library_path():
    return os.path.abspath(load()._name)


class HiSparseError(RuntimeError):
    def __init__(self, code, what):
        lib = load()
        msg = lib.hisparse_strerror(code).decode()
        if code == ECUDA:
            msg += f" (cudaError {lib.hisparse_last_cuda_error()})"
        super().__init__(f"{what}: {msg} [{code}]")
        self.code = code


def check(code, what):
    if code != OK:
        raise HiSparseError(code, what)
    return code


# ---- thin same-name wrappers ---------------------------------------------
def hisparse_init(cfg, layers):
    h = _vp()
    arr = (LayerBuffers * len(layers))(*layers)
    rc = load().hisparse_init(ctypes.byref(cfg), arr, ctypes.byref(h))
    return rc, h.value


def hisparse_destroy(h):
    return load().hisparse_destroy(h)


def hisparse_resolve(h, layer, d_sel, d_num_reqs, d_newest, d_out, flags, stream):
    return load().hisparse_resolve(h, layer, d_sel, d_num_reqs, d_newest, d_out, flags, stream)


def hisparse_resolve_step(h, layer, d_sel, d_num_reqs, d_newest, d_prev_pos, d_new_rows, d_out,
                          flags, stream):
    return load().hisparse_resolve_step(h, layer, d_sel, d_num_reqs, d_newest, d_prev_pos,
                                        d_new_rows, d_out, flags, stream)


class ResolveOptions(ctypes.Structure):
    """hisparse_resolve_options."""
    _fields_ = [("d_prev_pos", ctypes.c_void_p), ("d_new_rows", ctypes.c_void_p),
                ("d_res_blocks", ctypes.c_void_p), ("res_max_blocks", ctypes.c_int32),
                ("res_block_tokens", ctypes.c_int32), ("sel_block_tokens", ctypes.c_int32),
                ("d_seq_lens", ctypes.c_void_p)]


def hisparse_resolve_ex(h, layer, d_sel, d_num_reqs, d_newest, opt, d_out, flags, stream):
    return load().hisparse_resolve_ex(h, layer, d_sel, d_num_reqs, d_newest,
                                      ctypes.addressof(opt) if opt is not None else None, d_out,
                                      flags, stream)


def hisparse_resolve_resident(h, layer, d_sel, d_num_reqs, d_newest, d_prev_pos, d_new_rows,
                              d_res_blocks, res_max_blocks, res_block_tokens, d_out, flags,
                              stream):
    return load().hisparse_resolve_resident(h, layer, d_sel, d_num_reqs, d_newest, d_prev_pos,
                                            d_new_rows, d_res_blocks, res_max_blocks,
                                            res_block_tokens, d_out, flags, stream)


def hisparse_writeback(h, layer, d_pos, d_new_rows, d_num_reqs, stream):
    return load().hisparse_writeback(h, layer, d_pos, d_new_rows, d_num_reqs, stream)


def hisparse_prefetch_plan(h, anchor_layer, follower_layer, d_num_reqs, stream):
    return load().hisparse_prefetch_plan(h, anchor_layer, follower_layer, d_num_reqs, stream)


def hisparse_copy(dst, src, nbytes, stream):
    return load().hisparse_copy(dst, src, nbytes, stream)


def hisparse_copy_miss_counts(h, layer, d_dst, stream):
    return load().hisparse_copy_miss_counts(h, layer, d_dst, stream)


def hisparse_get_status(h, unit_err_ptr=None):
    f = _u32()
    rc = load().hisparse_get_status(h, ctypes.byref(f), unit_err_ptr)
    return rc, f.value


def hisparse_export_state(h, layer, slot_pos, lru, page_table, miss_counts):
    return load().hisparse_export_state(h, layer, slot_pos, lru, page_table, miss_counts)


def hisparse_import_state(h, layer, slot_pos, lru, page_table, miss_counts):
    return load().hisparse_import_state(h, layer, slot_pos, lru, page_table, miss_counts)


def hisparse_export_plan(h, layer, count, pos, slot):
    return load().hisparse_export_plan(h, layer, count, pos, slot)


def hisparse_reset(h, layer, stream):
    return load().hisparse_reset(h, layer, stream)


def hisparse_set_l2_persisting(h, nbytes):
    return load().hisparse_set_l2_persisting(h, nbytes)


def hisparse_get_info(h):
    info = Info()
    rc = load().hisparse_get_info(h, ctypes.byref(info))
    return rc, info


def hisparse_host_alloc(nbytes):
    p = _vp()
    rc = load().hisparse_host_alloc(nbytes, ctypes.byref(p))
    return rc, p.value


def hisparse_host_alloc_kind(nbytes, kind):
    p = _vp()
    rc = load().hisparse_host_alloc_kind(nbytes, kind, ctypes.byref(p))
    return rc, p.value


def hisparse_host_free(p):
    return load().hisparse_host_free(p)


def hisparse_host_hugepage_bytes(p, nbytes):
    v = ctypes.c_size_t()
    rc = load().hisparse_host_hugepage_bytes(p, nbytes, ctypes.byref(v))
    return rc, v.value


def hisparse_admit(h, layer, d_reqs, n, d_preload, stream):
    return load().hisparse_admit(h, layer, d_reqs, n, d_preload, stream)


# ---- 8-bit records and resident pages --------------------------------------
# (args: the structure, or its bytes)
def hisparse_rotary(args, stream):
    return load().hisparse_rotary(args if type(args) is bytes else ctypes.byref(args), stream)


def hisparse_pack(args, stream):
    return load().hisparse_pack(args if type(args) is bytes else ctypes.byref(args), stream)


def hisparse_attend(args, stream):
    return load().hisparse_attend(args if type(args) is bytes else ctypes.byref(args), stream)


def hisparse_pages_work_ints(num_pages, num_requests):
    return load().hisparse_pages_work_ints(num_pages, num_requests)


def hisparse_pages_grow(pool, d_reqs, d_blocks, n, stream):
    return load().hisparse_pages_grow(pool, d_reqs, d_blocks, n, stream)


def hisparse_pages_fork(pool, d_src, d_dst, d_tokens, n, stream):
    return load().hisparse_pages_fork(pool, d_src, d_dst, d_tokens, n, stream)


def hisparse_pages_free(pool, d_reqs, n, stream):
    return load().hisparse_pages_free(pool, d_reqs, n, stream)


def hisparse_pages_compact(pool, stream):
    return load().hisparse_pages_compact(pool, stream)
