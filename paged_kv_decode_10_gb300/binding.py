"""ctypes binding of ``libpkv.so`` (the C ABI declared in ``include/pkv.h``).

Argument marshalling only: torch tensors become device pointers, the current
torch CUDA stream becomes the ``cudaStream_t`` argument, numpy arrays hold the
allocator's host outputs.  Every computation runs in the library's CUDA kernels
or in its C++ allocator; if the library has not been built this module raises
instead of falling back to anything else.
"""
import ctypes
import os

import numpy as np

from . import build as _build

OK, ERR_INVALID_ARG, ERR_OUT_OF_BLOCKS, ERR_UNKNOWN_SEQ, ERR_UNSUPPORTED, ERR_CUDA = range(6)
F32, BF16 = 0, 1
BLOCK_SIZE = 16
DEVERR_BAD_BLOCK, DEVERR_BAD_SLOT, DEVERR_BAD_LEN, DEVERR_TIMEOUT = 1, 2, 4, 8
DEVERR_BAD_PLAN = 16
PLAN_INTS = 24
ATTN_SIMT = 1
ATTN_SEPARATE_MERGE = 2
ATTN_SHORT_WAITS = 8
ATTN_CHECK_PLAN = 16
LAYERS_MERGE_HELPERS = 32
STEP_FUSED = 4
ROTARY_HALF, ROTARY_INTERLEAVED = 0, 1
ROTARY_PLAIN, ROTARY_LINEAR, ROTARY_NTK, ROTARY_RAMP, ROTARY_BANDS = range(5)

_c_i32 = ctypes.c_int32
_c_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_p_i32 = ctypes.POINTER(ctypes.c_int32)
_p_i64 = ctypes.POINTER(ctypes.c_int64)
_p_f32 = ctypes.POINTER(ctypes.c_float)
_size_t = ctypes.c_size_t


class PkvError(RuntimeError):
    def __init__(self, code, msg):
        super().__init__(f"pkv error {code}: {msg}")
        self.code = code


class OutOfBlocks(PkvError):
    pass


class UnknownSequence(PkvError):
    pass


class StepArgs(ctypes.Structure):
    _fields_ = [
        ("q", _vp), ("k", _vp), ("v", _vp),
        ("q_rot", _vp), ("k_rot", _vp),
        ("k_cache", _vp), ("v_cache", _vp),
        ("num_blocks", _c_i32),
        ("positions", _vp), ("slot_mapping", _vp), ("seq_lens", _vp),
        ("block_tables", _vp), ("bt_stride", _c_i32),
        ("attn_bias", _vp), ("bias_stride", _c_i32),
        ("B", _c_i32), ("Hq", _c_i32), ("Hkv", _c_i32), ("d", _c_i32),
        ("scale", ctypes.c_float), ("rope_base", ctypes.c_float),
        ("dtype", _c_i32), ("flags", _c_i32), ("num_parts", _c_i32),
        ("workspace", _vp), ("workspace_bytes", _size_t),
        ("out", _vp), ("dev_err_flag", _vp), ("plan", _vp),
    ]


class StepHostIO(ctypes.Structure):
    _fields_ = [
        ("q", _vp), ("k", _vp), ("v", _vp),
        ("positions", _vp), ("slot_mapping", _vp), ("seq_lens", _vp),
        ("block_tables", _vp), ("out", _vp), ("flags", _c_i32), ("plan", _vp),
    ]


class ServerDesc(ctypes.Structure):
    _fields_ = [
        ("step", StepArgs), ("alloc", _vp), ("rows", _vp),
        ("meta_host", _vp * 2), ("prefix_host", _vp * 2), ("max_prefix_tokens", _c_i32),
    ]


class RotarySpec(ctypes.Structure):
    _fields_ = [
        ("rot_dim", _c_i32), ("layout", _c_i32), ("scaling", _c_i32), ("original_len", _c_i32),
        ("base", ctypes.c_double), ("factor", ctypes.c_double), ("low", ctypes.c_double),
        ("high", ctypes.c_double), ("amplitude", ctypes.c_double),
    ]


class RotaryTable(ctypes.Structure):
    _fields_ = [
        ("d", _c_i32), ("rot_dim", _c_i32), ("layout", _c_i32), ("amplitude", ctypes.c_float),
        ("turns", ctypes.c_uint64 * 128), ("check", ctypes.c_uint32),
    ]


class RotaryArgs(ctypes.Structure):
    _fields_ = [
        ("rotary", ctypes.POINTER(RotaryTable)),
        ("q", _vp), ("k", _vp), ("v", _vp),
        ("q_stride", _c_i64), ("k_stride", _c_i64), ("v_stride", _c_i64),
        ("q_out", _vp), ("k_out", _vp), ("q_out_stride", _c_i64), ("k_out_stride", _c_i64),
        ("positions", _vp), ("slot_mapping", _vp), ("k_cache", _vp), ("v_cache", _vp),
        ("num_blocks", _c_i32), ("T", _c_i32), ("Hq", _c_i32), ("Hkv", _c_i32), ("d", _c_i32),
        ("dtype", _c_i32), ("dev_err_flag", _vp),
    ]


class SharedArgs(ctypes.Structure):
    _fields_ = [
        ("q_rot", _vp), ("k_cache", _vp), ("v_cache", _vp),
        ("block_tables", _vp), ("seq_lens", _vp), ("attn_bias", _vp), ("plan", _vp),
        ("prefix_tables", _vp), ("prefix_plan", _vp),
        ("mass", _vp), ("scores", _vp), ("mass_lens", _vp),
        ("workspace", _vp), ("workspace_bytes", _size_t),
        ("out", _vp), ("lse_out", _vp), ("dev_err_flag", _vp),
        ("num_blocks", _c_i32), ("bt_stride", _c_i32), ("bias_stride", _c_i32),
        ("n_prefixes", _c_i32), ("pt_stride", _c_i32), ("plan_ints", _c_i32), ("slots", _c_i32),
        ("B", _c_i32), ("Hq", _c_i32), ("Hkv", _c_i32), ("d", _c_i32), ("dtype", _c_i32),
        ("flags", _c_i32), ("num_parts", _c_i32), ("num_ctas", _c_i32),
        ("scale", ctypes.c_float), ("mass_decay", ctypes.c_float),
    ]


class EvictArgs(ctypes.Structure):
    _fields_ = [
        ("k_cache", _vp), ("v_cache", _vp), ("mass", _vp),
        ("block_tables", _vp), ("seq_lens", _vp), ("keep_lens", _vp), ("kept", _vp),
        ("workspace", _vp), ("workspace_bytes", _size_t), ("dev_err_flag", _vp),
        ("num_blocks", _c_i32), ("bt_stride", _c_i32), ("kept_stride", _c_i32),
        ("sink", _c_i32), ("recent", _c_i32),
        ("B", _c_i32), ("Hkv", _c_i32), ("d", _c_i32), ("dtype", _c_i32),
    ]


# name -> (restype, argtypes); every symbol declared in include/pkv.h
SIGNATURES = {
    "pkv_last_error": (ctypes.c_char_p, []),
    "pkv_abi_version": (ctypes.c_int, []),
    "pkv_alloc_create": (ctypes.c_int, [_c_i32, _c_i32, _c_i32, _c_i32, _p_i32,
                                        ctypes.POINTER(_vp)]),
    "pkv_alloc_destroy": (None, [_vp]),
    "pkv_seq_join": (ctypes.c_int, [_vp, _c_i32, _p_i32]),
    "pkv_seq_leave": (ctypes.c_int, [_vp, _c_i32]),
    "pkv_seqs_join": (ctypes.c_int, [_vp, _p_i32, _c_i32, _p_i32, _p_i32, _p_i64]),
    "pkv_seqs_leave": (ctypes.c_int, [_vp, _p_i32, _c_i32]),
    "pkv_prepare_step": (ctypes.c_int, [_vp, _p_i32, _c_i32, _p_i32, _p_i64, _p_i32, _p_i32,
                                        _c_i32]),
    "pkv_prepare_step_cached": (ctypes.c_int, [_vp, _p_i32, _c_i32, _p_i32, _p_i64, _p_i32,
                                               _p_i32, _c_i32, _p_i32]),
    "pkv_seq_len": (ctypes.c_int, [_vp, _c_i32, _p_i32]),
    "pkv_seq_blocks": (ctypes.c_int, [_vp, _c_i32, _p_i32, _c_i32, _p_i32]),
    "pkv_seq_slots": (ctypes.c_int, [_vp, _c_i32, _c_i32, _c_i32, _p_i32, _p_i64]),
    "pkv_num_free": (ctypes.c_int, [_vp, _p_i32]),
    "pkv_pool_blocks": (ctypes.c_int, [ctypes.c_uint64, _c_i32, _c_i32, _c_i32, _c_i32, _p_i32]),
    "pkv_alloc_dump": (ctypes.c_int, [_vp, _p_i32, _c_i32, _p_i32]),
    "pkv_rope": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _c_i32,
                                ctypes.c_float, _c_i32, _vp]),
    "pkv_rope_append": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_i32,
                                       _c_i32, _c_i32, _c_i32, _c_i32, ctypes.c_float, _c_i32,
                                       _vp, _vp]),
    "pkv_append": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32, _c_i32,
                                  _c_i32, _vp, _vp]),
    "pkv_prefill_kv": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i32, _c_i32, _c_i32,
                                      _c_i32, ctypes.c_float, _c_i32, _vp, _vp]),
    "pkv_attn_default_parts": (ctypes.c_int, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _p_i32]),
    "pkv_attn_workspace_bytes": (ctypes.c_int, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                                ctypes.POINTER(_size_t)]),
    "pkv_decode_attn_split": (ctypes.c_int, [_vp, _vp, _vp, _c_i32, _vp, _c_i32, _vp, _vp,
                                             _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                             ctypes.c_float, _c_i32, _vp, _size_t, _vp, _c_i32,
                                             _c_i32, _vp, _vp]),
    "pkv_decode_attn_static": (ctypes.c_int, [_vp, _vp, _vp, _c_i32, _vp, _c_i32, _vp, _vp,
                                              _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                              ctypes.c_float, _c_i32, _vp, _c_i32, _c_i32, _vp,
                                              _vp]),
    "pkv_plan_parts": (ctypes.c_int, [_p_i32, _c_i32, _c_i32, _c_i32, _p_i32, _c_i32, _c_i32,
                                      _c_i32, _p_i32]),
    "pkv_decode_attn_planned": (ctypes.c_int, [_vp, _vp, _vp, _c_i32, _vp, _c_i32, _vp, _vp,
                                               _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                               ctypes.c_float, _c_i32, _vp, _vp, _size_t, _vp,
                                               _c_i32, _c_i32, _vp, _vp]),
    "pkv_lse_merge": (ctypes.c_int, [_vp, _size_t, _vp, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                     _c_i32, _c_i32, _vp, _c_i32, _vp]),
    "pkv_decode_step": (ctypes.c_int, [ctypes.POINTER(StepArgs), _vp]),
    "pkv_mapped_pointer": (ctypes.c_int, [_vp, ctypes.POINTER(_vp)]),
    "pkv_decode_step_layers": (ctypes.c_int, [ctypes.POINTER(StepArgs), _c_i32, _vp]),
    "pkv_dense_assemble": (ctypes.c_int, [ctypes.POINTER(_vp), ctypes.POINTER(_vp), _p_i32,
                                          _c_i32, _c_i32, _vp, _vp, _c_i32, _c_i32, _c_i32,
                                          _c_i32, _vp]),
    "pkv_dense_extract": (ctypes.c_int, [_vp, _vp, _c_i32, _p_i32, _p_i32, _c_i32, _c_i32,
                                         _c_i32, ctypes.POINTER(_vp), ctypes.POINTER(_vp),
                                         _c_i32, _c_i32, _c_i32, _vp]),
    "pkv_decode_step_host": (ctypes.c_int, [ctypes.POINTER(StepArgs),
                                            ctypes.POINTER(StepHostIO), _vp]),
    "pkv_step_graph_create": (ctypes.c_int, [ctypes.POINTER(StepArgs),
                                             ctypes.POINTER(StepHostIO), ctypes.POINTER(_vp)]),
    "pkv_step_graph_launch": (ctypes.c_int, [_vp, _vp]),
    "pkv_step_graph_enqueue": (ctypes.c_int, [_vp, _vp]),
    "pkv_step_graph_wait": (ctypes.c_int, [_vp]),
    "pkv_step_graph_destroy": (None, [_vp]),
    "pkv_server_meta_bytes": (_size_t, [_c_i32, _c_i32, _c_i32]),
    "pkv_server_prefix_bytes": (_size_t, [_c_i32]),
    "pkv_server_create": (ctypes.c_int, [ctypes.POINTER(ServerDesc), ctypes.POINTER(_vp)]),
    "pkv_server_step": (ctypes.c_int, [_vp, _p_i32, _p_i32, _c_i32, _vp, _vp, _vp, _vp, _vp,
                                       _vp]),
    "pkv_server_rows": (ctypes.c_int, [_vp, _p_i32]),
    "pkv_server_destroy": (None, [_vp]),
    "pkv_seq_set_offset": (ctypes.c_int, [_vp, _c_i32, _c_i32]),
    "pkv_seq_offset": (ctypes.c_int, [_vp, _c_i32, _p_i32]),
    "pkv_seqs_evict": (ctypes.c_int, [_vp, _p_i32, _p_i32, _c_i32]),
    "pkv_rotary_init": (ctypes.c_int, [ctypes.POINTER(RotarySpec), _c_i32,
                                       ctypes.POINTER(RotaryTable)]),
    "pkv_rotary_append": (ctypes.c_int, [ctypes.POINTER(RotaryArgs), _vp]),
    "pkv_shared_plan_cap": (ctypes.c_int, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _p_i32,
                                           _p_i32]),
    "pkv_shared_plan": (ctypes.c_int, [_p_i32, _c_i32, _p_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                       _c_i32, _c_i32, _p_i32, _c_i32, _p_i32, _p_i32]),
    "pkv_shared_default_parts": (ctypes.c_int, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                                _p_i32]),
    "pkv_shared_short": (ctypes.c_int, [_c_i32] * 7 + [_p_i32]),
    "pkv_shared_workspace_bytes": (ctypes.c_int, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                                  ctypes.POINTER(_size_t)]),
    "pkv_decode_attn_shared": (ctypes.c_int, [ctypes.POINTER(SharedArgs), _vp]),
    "pkv_evict_workspace_bytes": (ctypes.c_int, [_c_i32, _c_i32, _c_i32, _c_i32, _c_i32,
                                                 ctypes.POINTER(_size_t)]),
    "pkv_evict": (ctypes.c_int, [ctypes.POINTER(EvictArgs), _vp]),
}

_LIB = None
ABI_VERSION = 5   # pkv_abi_version() of the library this binding describes


def library_path():
    return _build.LIB


def load():
    """Load the built library (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"CUDA library {path} is missing: build it with "
            "`python -m paged_kv_decode_10_gb300.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.pkv_abi_version() != ABI_VERSION:
        raise RuntimeError(f"{path} has ABI version {lib.pkv_abi_version()}, this binding "
                           f"expects {ABI_VERSION}: rebuild it")
    _LIB = lib
    return lib


def _check(rc):
    if rc == OK:
        return
    msg = load().pkv_last_error().decode(errors="replace")
    if rc == ERR_OUT_OF_BLOCKS:
        raise OutOfBlocks(rc, msg)
    if rc == ERR_UNKNOWN_SEQ:
        raise UnknownSequence(rc, msg)
    raise PkvError(rc, msg)


# --------------------------------------------------------------------------
# host allocator
# --------------------------------------------------------------------------
_NP_OF = {ctypes.c_int32: np.int32, ctypes.c_int64: np.int64}


def _np_ptr(a, ctype, min_len=0):
    """Pointer to a numpy array the library reads or fills: the dtype must be
    the C type's, the array C-contiguous and at least ``min_len`` long (the C
    side writes through the pointer without knowing the array)."""
    if not isinstance(a, np.ndarray) or a.dtype != _NP_OF[ctype]:
        raise PkvError(ERR_INVALID_ARG, f"expected a numpy {np.dtype(_NP_OF[ctype])} array, "
                                        f"got {getattr(a, 'dtype', type(a))}")
    if not a.flags.c_contiguous or a.size < min_len:
        raise PkvError(ERR_INVALID_ARG, f"array must be C-contiguous with >= {min_len} entries")
    return a.ctypes.data_as(ctypes.POINTER(ctype))


class BlockAllocator:
    """Host block allocator (C++); policy in ``include/pkv.h``."""

    def __init__(self, num_blocks, max_seqs, max_blocks_per_seq, initial_free=None):
        lib = load()
        handle = _vp()
        init = None
        if initial_free is not None:
            self._init = np.ascontiguousarray(initial_free, dtype=np.int32)
            init = _np_ptr(self._init, ctypes.c_int32)
        _check(lib.pkv_alloc_create(num_blocks, BLOCK_SIZE, max_seqs, max_blocks_per_seq, init,
                                    ctypes.byref(handle)))
        self._h = handle
        self._lib = lib
        self.num_blocks = num_blocks

    def close(self):
        if self._h:
            self._lib.pkv_alloc_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def join(self, prefix_len):
        sid = ctypes.c_int32()
        _check(self._lib.pkv_seq_join(self._h, int(prefix_len), ctypes.byref(sid)))
        return sid.value

    def leave(self, seq_id):
        _check(self._lib.pkv_seq_leave(self._h, int(seq_id)))

    def join_many(self, prefix_lens, slots_out=None):
        """Joins one sequence per prefix length in one call (``pkv_seqs_join``);
        returns their ids.  ``slots_out = (positions, slot_mapping)``, arrays of at
        least sum(prefix_lens) entries, also receives every joiner's prefix
        positions and cache slots, packed in order."""
        lens = np.ascontiguousarray(prefix_lens, dtype=np.int32)
        ids = np.empty(len(lens), np.int32)
        pos = slots = None
        if slots_out is not None:
            n = int(lens.astype(np.int64).sum())
            pos = _np_ptr(slots_out[0], ctypes.c_int32, n)
            slots = _np_ptr(slots_out[1], ctypes.c_int64, n)
        _check(self._lib.pkv_seqs_join(self._h, _np_ptr(lens, ctypes.c_int32), len(lens),
                                       _np_ptr(ids, ctypes.c_int32), pos, slots))
        return ids

    def leave_many(self, seq_ids):
        """Retires the listed sequences in one call (``pkv_seqs_leave``)."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int32)
        _check(self._lib.pkv_seqs_leave(self._h, _np_ptr(ids, ctypes.c_int32), len(ids)))

    def prepare_step(self, seq_ids, bt_stride, out=None):
        """Returns ``positions, slot_mapping, seq_lens, block_tables`` (numpy).
        ``out`` may supply preallocated (e.g. pinned) arrays to fill."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int32)
        B = len(ids)
        if out is None:
            out = (np.empty(B, np.int32), np.empty(B, np.int64), np.empty(B, np.int32),
                   np.empty((B, bt_stride), np.int32))
        pos, slots, lens, tables = out
        _check(self._lib.pkv_prepare_step(self._h, _np_ptr(ids, ctypes.c_int32), B,
                                          _np_ptr(pos, ctypes.c_int32, B),
                                          _np_ptr(slots, ctypes.c_int64, B),
                                          _np_ptr(lens, ctypes.c_int32, B),
                                          _np_ptr(tables, ctypes.c_int32, B * int(bt_stride)),
                                          int(bt_stride)))
        return pos, slots, lens, tables

    def step_runner(self, seq_ids, bt_stride, out, row_state=None):
        """A no-argument callable that runs ``prepare_step`` for these sequence ids
        into the arrays ``out`` (positions, slot_mapping, seq_lens, block_tables),
        with every pointer converted once (a serving loop calls it every step).
        With ``row_state`` (int32 [B*3], -1 before the first call) it runs
        ``prepare_step_cached``: ``out`` must then be the same arrays every call."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int32)
        pos, slots, lens, tables = out
        h, B, bt = self._h, len(ids), int(bt_stride)
        ptrs = (_np_ptr(ids, ctypes.c_int32), _np_ptr(pos, ctypes.c_int32, B),
                _np_ptr(slots, ctypes.c_int64, B), _np_ptr(lens, ctypes.c_int32, B),
                _np_ptr(tables, ctypes.c_int32, B * bt))
        if row_state is None:
            fn, extra = self._lib.pkv_prepare_step, ()
        else:
            fn, extra = self._lib.pkv_prepare_step_cached, (_np_ptr(row_state, ctypes.c_int32,
                                                                    3 * B),)
        keep = (ids, out, row_state)
        args = (h, ptrs[0], B, ptrs[1], ptrs[2], ptrs[3], ptrs[4], bt) + extra

        def run():
            _check(fn(*args))
            return keep[1]
        return run

    def prepare_step_cached(self, seq_ids, bt_stride, out, row_state):
        """``pkv_prepare_step_cached`` into ``out`` (positions, slot_mapping,
        seq_lens, block_tables) with the caller-kept ``row_state`` (int32 [B*3])."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int32)
        B = len(ids)
        pos, slots, lens, tables = out
        _check(self._lib.pkv_prepare_step_cached(
            self._h, _np_ptr(ids, ctypes.c_int32), B, _np_ptr(pos, ctypes.c_int32, B),
            _np_ptr(slots, ctypes.c_int64, B), _np_ptr(lens, ctypes.c_int32, B),
            _np_ptr(tables, ctypes.c_int32, B * int(bt_stride)), int(bt_stride),
            _np_ptr(row_state, ctypes.c_int32, 3 * B)))
        return out

    def seq_len(self, seq_id):
        n = ctypes.c_int32()
        _check(self._lib.pkv_seq_len(self._h, int(seq_id), ctypes.byref(n)))
        return n.value

    def seq_blocks(self, seq_id):
        n = ctypes.c_int32()
        _check(self._lib.pkv_seq_blocks(self._h, int(seq_id), None, 0, ctypes.byref(n)))
        buf = np.empty(n.value, np.int32)
        _check(self._lib.pkv_seq_blocks(self._h, int(seq_id), _np_ptr(buf, ctypes.c_int32),
                                        n.value, ctypes.byref(n)))
        return buf.tolist()

    def seq_slots(self, seq_id, start, count, out=None):
        """Positions and cache slots of tokens [start, start+count) of a live
        sequence (``pkv_seq_slots``); ``out`` may supply the two arrays."""
        if out is None:
            out = (np.empty(count, np.int32), np.empty(count, np.int64))
        pos, slots = out
        _check(self._lib.pkv_seq_slots(self._h, int(seq_id), int(start), int(count),
                                       _np_ptr(pos, ctypes.c_int32, int(count)),
                                       _np_ptr(slots, ctypes.c_int64, int(count))))
        return pos, slots

    def set_offset(self, seq_id, offset):
        """The sequence's next position is its cached length plus ``offset`` from
        now on (``pkv_seq_set_offset``)."""
        _check(self._lib.pkv_seq_set_offset(self._h, int(seq_id), int(offset)))

    def offset(self, seq_id):
        n = ctypes.c_int32()
        _check(self._lib.pkv_seq_offset(self._h, int(seq_id), ctypes.byref(n)))
        return n.value

    def evict_many(self, seq_ids, keep_lens):
        """Shortens the sequences to ``keep_lens`` after ``evict`` (``pkv_seqs_evict``)."""
        ids = np.ascontiguousarray(seq_ids, dtype=np.int32)
        keep = np.ascontiguousarray(keep_lens, dtype=np.int32)
        if len(ids) != len(keep):
            raise PkvError(ERR_INVALID_ARG, "one keep length per sequence")
        _check(self._lib.pkv_seqs_evict(self._h, _np_ptr(ids, ctypes.c_int32),
                                        _np_ptr(keep, ctypes.c_int32), len(ids)))

    def num_free(self):
        n = ctypes.c_int32()
        _check(self._lib.pkv_num_free(self._h, ctypes.byref(n)))
        return n.value

    def free_stack(self):
        n = ctypes.c_int32()
        _check(self._lib.pkv_alloc_dump(self._h, None, 0, ctypes.byref(n)))
        buf = np.empty(n.value, np.int32)
        _check(self._lib.pkv_alloc_dump(self._h, _np_ptr(buf, ctypes.c_int32), n.value,
                                        ctypes.byref(n)))
        return buf.tolist()


# --------------------------------------------------------------------------
# device calls (torch tensors in, torch tensors out)
# --------------------------------------------------------------------------
def _torch():
    import torch
    return torch


def dtype_code(t):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise PkvError(ERR_UNSUPPORTED, f"dtype {t.dtype}")


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise PkvError(ERR_INVALID_ARG, "tensor must be on a CUDA device")
    if not t.is_contiguous():
        raise PkvError(ERR_INVALID_ARG, "tensor must be contiguous")
    return _vp(t.data_ptr())


def mapped_pointer(t):
    """Device-side address of a contiguous pinned CPU tensor (``pkv_mapped_pointer``)."""
    if t.is_cuda or not t.is_pinned():
        raise PkvError(ERR_INVALID_ARG, "tensor must be in pinned host memory")
    if not t.is_contiguous():
        raise PkvError(ERR_INVALID_ARG, "tensor must be contiguous")
    out = _vp()
    _check(load().pkv_mapped_pointer(_vp(t.data_ptr()), ctypes.byref(out)))
    return out


def _meta_ptr(t):
    """Step metadata may be a device tensor or a pinned host tensor the kernels
    read in place."""
    if t is not None and not t.is_cuda:
        return mapped_pointer(t)
    return _ptr(t)


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return _vp(s.cuda_stream)


def rope(q, k, positions, base=10000.0, q_out=None, k_out=None, stream=None):
    """a1: rotate-half RoPE of ``q [B,Hq,d]`` and ``k [B,Hkv,d]`` at ``positions [B]`` (int32)."""
    torch = _torch()
    with torch.cuda.stream(stream):
        q_out = torch.empty_like(q) if q_out is None else q_out
        k_out = torch.empty_like(k) if k_out is None else k_out
    B, Hq, d = q.shape
    _check(load().pkv_rope(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), _meta_ptr(positions), B, Hq,
                           k.shape[1], d, float(base), dtype_code(q), _stream(stream)))
    return q_out, k_out


def rope_append(q, k, v, positions, slot_mapping, k_cache, v_cache, base=10000.0, q_out=None,
                k_out=None, err=None, stream=None):
    """a1 + a2 fused: rotate q/k and write the rotated k and raw v into the cache slots."""
    torch = _torch()
    with torch.cuda.stream(stream):
        q_out = torch.empty_like(q) if q_out is None else q_out
        k_out = torch.empty_like(k) if k_out is None else k_out
    B, Hq, d = q.shape
    _check(load().pkv_rope_append(_ptr(q), _ptr(k), _ptr(v), _ptr(q_out), _ptr(k_out),
                                  _meta_ptr(positions), _meta_ptr(slot_mapping), _ptr(k_cache),
                                  _ptr(v_cache), B, Hq, k.shape[1], d, k_cache.shape[0],
                                  float(base), dtype_code(q), _ptr(err), _stream(stream)))
    return q_out, k_out


def prefill_kv(k, v, positions, slot_mapping, k_cache, v_cache, base=10000.0, err=None,
               stream=None):
    """Prefix KV of joining sequences: rotate ``k [T,Hkv,d]`` at ``positions [T]``
    and write it and ``v`` into ``slot_mapping [T]`` of the caches."""
    T, Hkv, d = k.shape
    _check(load().pkv_prefill_kv(_ptr(k), _ptr(v), _meta_ptr(positions),
                                 _meta_ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache), T, Hkv,
                                 d, k_cache.shape[0], float(base), dtype_code(k), _ptr(err),
                                 _stream(stream)))


def append(k_rot, v, slot_mapping, k_cache, v_cache, err=None, stream=None):
    """a2: write ``k_rot``/``v`` ``[B,Hkv,d]`` into cache slots ``slot_mapping [B]`` (int64)."""
    B, Hkv, d = k_rot.shape
    _check(load().pkv_append(_ptr(k_rot), _ptr(v), _meta_ptr(slot_mapping), _ptr(k_cache),
                             _ptr(v_cache), B, Hkv, d, k_cache.shape[0], dtype_code(k_rot),
                             _ptr(err), _stream(stream)))


def default_parts(d, dtype, flags=0, Hq=32, Hkv=8):
    n = ctypes.c_int32()
    _check(load().pkv_attn_default_parts(d, Hq, Hkv, dtype, flags, ctypes.byref(n)))
    return n.value


def workspace_bytes(B, Hq, Hkv, d, num_parts):
    n = _size_t()
    _check(load().pkv_attn_workspace_bytes(B, Hq, Hkv, d, num_parts, ctypes.byref(n)))
    return n.value


def alloc_workspace(B, Hq, Hkv, d, num_parts, device=None):
    torch = _torch()
    nbytes = workspace_bytes(B, Hq, Hkv, d, num_parts)
    # zero-filled once: the fused merge's counters start (and stay) at zero
    return torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=device or "cuda")


def decode_attn_split(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, num_parts,
                      workspace, out, attn_bias=None, flags=0, err=None, stream=None):
    """a3: split-KV paged GQA attention (fills ``out`` for single-part units and
    the workspace partials for the rest)."""
    B, Hq, d = q_rot.shape
    Hkv = k_cache.shape[1]
    bias_stride = attn_bias.shape[1] if attn_bias is not None else 0
    _check(load().pkv_decode_attn_split(
        _ptr(q_rot), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _meta_ptr(block_tables),
        block_tables.shape[1], _meta_ptr(seq_lens), _ptr(attn_bias), bias_stride, B, Hq, Hkv, d,
        float(scale), int(num_parts), _ptr(workspace), workspace.numel(), _ptr(out),
        dtype_code(q_rot), int(flags), _ptr(err), _stream(stream)))


def plan_parts(seq_lens, Hkv, d, block_tables, num_parts, bias_stride=0, out=None):
    """Host-planned partition (``pkv_plan_parts``) of numpy step metadata:
    ``seq_lens int32 [B]``, ``block_tables int32 [B, bt_stride]``; returns (or
    fills) ``int32 [num_parts, PLAN_INTS]``."""
    lens = np.ascontiguousarray(seq_lens, dtype=np.int32)
    tables = np.ascontiguousarray(block_tables, dtype=np.int32)
    B = len(lens)
    if tables.ndim != 2 or tables.shape[0] != B:
        raise PkvError(ERR_INVALID_ARG, "block_tables must be [B, bt_stride]")
    if out is None:
        out = np.empty((num_parts, PLAN_INTS), np.int32)
    _check(load().pkv_plan_parts(_np_ptr(lens, ctypes.c_int32), B, int(Hkv), int(d),
                                 _np_ptr(tables, ctypes.c_int32), tables.shape[1],
                                 int(bias_stride), int(num_parts),
                                 _np_ptr(out, ctypes.c_int32, num_parts * PLAN_INTS)))
    return out


def plan_runner(seq_lens, block_tables, Hkv, d, num_parts, out, bias_stride=0):
    """A no-argument callable running ``pkv_plan_parts`` on these (fixed)
    numpy arrays into ``out`` with every pointer converted once, for a loop
    that re-plans every step after a0 rewrote the arrays in place."""
    fn = load().pkv_plan_parts
    B, bt = len(seq_lens), block_tables.shape[1]
    ptrs = (_np_ptr(seq_lens, ctypes.c_int32, B), _np_ptr(block_tables, ctypes.c_int32, B * bt),
            _np_ptr(out, ctypes.c_int32, num_parts * PLAN_INTS))
    args = (ptrs[0], B, int(Hkv), int(d), ptrs[1], bt, int(bias_stride), int(num_parts), ptrs[2])
    keep = (seq_lens, block_tables, out)

    def run():
        _check(fn(*args))
        return keep[2]
    return run


def decode_attn_planned(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, num_parts, plan,
                        workspace, out, attn_bias=None, flags=0, err=None, stream=None):
    """a3 with a host-planned partition (``plan``: device or pinned int32
    ``[num_parts, PLAN_INTS]`` tensor from ``plan_parts``)."""
    B, Hq, d = q_rot.shape
    Hkv = k_cache.shape[1]
    bias_stride = attn_bias.shape[1] if attn_bias is not None else 0
    _check(load().pkv_decode_attn_planned(
        _ptr(q_rot), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _meta_ptr(block_tables),
        block_tables.shape[1], _meta_ptr(seq_lens), _ptr(attn_bias), bias_stride, B, Hq, Hkv, d,
        float(scale), int(num_parts), _meta_ptr(plan), _ptr(workspace), workspace.numel(),
        _ptr(out), dtype_code(q_rot), int(flags), _ptr(err), _stream(stream)))


def decode_attention_static(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, out,
                            num_parts=0, attn_bias=None, flags=0, err=None, stream=None):
    """a3 + fused a4 with the library's built-in scratch array instead of a
    workspace, for callers that cannot allocate device memory (see
    ``pkv_decode_attn_static`` in ``include/pkv.h``)."""
    B, Hq, d = q_rot.shape
    Hkv = k_cache.shape[1]
    bias_stride = attn_bias.shape[1] if attn_bias is not None else 0
    _check(load().pkv_decode_attn_static(
        _ptr(q_rot), _ptr(k_cache), _ptr(v_cache), k_cache.shape[0], _meta_ptr(block_tables),
        block_tables.shape[1], _meta_ptr(seq_lens), _ptr(attn_bias), bias_stride, B, Hq, Hkv, d,
        float(scale), int(num_parts), _ptr(out), dtype_code(q_rot), int(flags), _ptr(err),
        _stream(stream)))
    return out


def lse_merge(workspace, seq_lens, bt_stride, B, Hq, Hkv, d, num_parts, out, bias_stride=0,
              stream=None):
    """a4: LSE merge of the split partials into ``out``."""
    _check(load().pkv_lse_merge(_ptr(workspace), workspace.numel(), _meta_ptr(seq_lens),
                                int(bt_stride), int(bias_stride), B, Hq, Hkv, d, int(num_parts),
                                _ptr(out), dtype_code(out), _stream(stream)))


def decode_attention(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, num_parts=None,
                     workspace=None, out=None, attn_bias=None, flags=0, err=None, stream=None,
                     plan=None):
    """a3 + a4: returns ``out [B,Hq,d]`` (with ``plan``, through the host-planned
    partition; ``num_parts`` must then be the plan's)."""
    torch = _torch()
    B, Hq, d = q_rot.shape
    Hkv = k_cache.shape[1]
    if num_parts is None:
        num_parts = default_parts(d, dtype_code(q_rot), flags, Hq, Hkv)
    with torch.cuda.stream(stream):   # (scratch of the stream that the kernels run on)
        if workspace is None:
            workspace = alloc_workspace(B, Hq, Hkv, d, num_parts, q_rot.device)
        if out is None:
            out = torch.empty_like(q_rot)
    if plan is not None:
        decode_attn_planned(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, num_parts,
                            plan, workspace, out, attn_bias, flags, err, stream)
    else:
        decode_attn_split(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, num_parts,
                          workspace, out, attn_bias, flags, err, stream)
    if flags & ATTN_SEPARATE_MERGE:
        lse_merge(workspace, seq_lens, block_tables.shape[1], B, Hq, Hkv, d, num_parts, out,
                  attn_bias.shape[1] if attn_bias is not None else 0, stream)
    return out


def make_step_args(q, k, v, q_rot, k_rot, k_cache, v_cache, positions, slot_mapping, seq_lens,
                   block_tables, scale, rope_base, num_parts, workspace, out, attn_bias=None,
                   flags=0, err=None, plan=None):
    """Fills the ``pkv_step_args`` struct.  All tensors are on the device except
    that q, k, v, positions, slot_mapping, seq_lens and block_tables may be pinned
    host tensors, which the kernels then read in place, and out may be a pinned
    host tensor, which the kernels then write in place."""
    a = StepArgs()
    a.q, a.k, a.v = _meta_ptr(q), _meta_ptr(k), _meta_ptr(v)
    a.q_rot, a.k_rot = _ptr(q_rot), _ptr(k_rot)
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.num_blocks = k_cache.shape[0]
    a.positions, a.slot_mapping = _meta_ptr(positions), _meta_ptr(slot_mapping)
    a.seq_lens = _meta_ptr(seq_lens)
    a.block_tables, a.bt_stride = _meta_ptr(block_tables), block_tables.shape[1]
    a.attn_bias = _ptr(attn_bias)
    a.bias_stride = attn_bias.shape[1] if attn_bias is not None else 0
    a.B, a.Hq, a.d = q.shape
    a.Hkv = k.shape[1]
    a.scale, a.rope_base = float(scale), float(rope_base)
    a.dtype, a.flags, a.num_parts = dtype_code(q), int(flags), int(num_parts)
    a.workspace, a.workspace_bytes = _ptr(workspace), workspace.numel()
    a.out = _meta_ptr(out)
    a.dev_err_flag = _ptr(err)
    a.plan = _meta_ptr(plan)
    return a


def decode_step_args(args, stream=None):
    """Runs a1 -> a4 from a prepared ``StepArgs``."""
    _check(load().pkv_decode_step(ctypes.byref(args), _stream(stream)))


def layer_args_array(layers):
    """A ctypes array of ``StepArgs``, one per layer, for ``decode_step_layers``."""
    arr = (StepArgs * len(layers))()
    for i, a in enumerate(layers):
        arr[i] = a
    return arr


def decode_step_layers(layers, stream=None):
    """One decode step through every layer (``pkv_decode_step_layers``);
    ``layers`` is a list of ``StepArgs`` or an array from ``layer_args_array``."""
    arr = layers if isinstance(layers, ctypes.Array) else layer_args_array(layers)
    _check(load().pkv_decode_step_layers(arr, len(arr), _stream(stream)))


def _ptr_array(tensors):
    arr = (_vp * max(len(tensors), 1))()
    for i, t in enumerate(tensors):
        arr[i] = _ptr(t)
    return arr


def dense_assemble(k_snaps, v_snaps, lens, padded_len, k_dense, v_dense, cap, stream=None):
    """Right-padded dense batch from per-sequence snapshots (``pkv_dense_assemble``).
    Snapshots and the dense caches use the block layout ``[blocks, Hkv, 16, d]``;
    the dense batch has ``cap`` tokens per row."""
    lens = np.ascontiguousarray(lens, dtype=np.int32)
    if not len(k_snaps) == len(v_snaps) == len(lens):
        raise PkvError(ERR_INVALID_ARG, "one K and one V snapshot per length")
    Hkv, d = k_dense.shape[1], k_dense.shape[3]
    _check(load().pkv_dense_assemble(_ptr_array(k_snaps), _ptr_array(v_snaps),
                                     _np_ptr(lens, ctypes.c_int32), len(lens), int(padded_len),
                                     _ptr(k_dense), _ptr(v_dense), int(cap), Hkv, d,
                                     dtype_code(k_dense), _stream(stream)))


def dense_extract(k_dense, v_dense, cap, rows, prefix_lens, padded_len, steps, k_snaps, v_snaps,
                  stream=None):
    """Rows of a dense batch back into snapshots: prefix plus decode columns
    (``pkv_dense_extract``)."""
    rows = np.ascontiguousarray(rows, dtype=np.int32)
    prefix_lens = np.ascontiguousarray(prefix_lens, dtype=np.int32)
    if not len(prefix_lens) == len(k_snaps) == len(v_snaps) == len(rows):
        raise PkvError(ERR_INVALID_ARG, "one prefix length and K/V snapshot per row")
    Hkv, d = k_dense.shape[1], k_dense.shape[3]
    _check(load().pkv_dense_extract(_ptr(k_dense), _ptr(v_dense), int(cap),
                                    _np_ptr(rows, ctypes.c_int32),
                                    _np_ptr(prefix_lens, ctypes.c_int32), len(rows),
                                    int(padded_len), int(steps), _ptr_array(k_snaps),
                                    _ptr_array(v_snaps), Hkv, d, dtype_code(k_dense),
                                    _stream(stream)))


# --------------------------------------------------------------------------
# rotary layouts and scalings, shared-prefix attention, eviction
# --------------------------------------------------------------------------
# These calls take argument structs made once (``make_*_args``: every pointer,
# size and type is checked there) and launched as often as wanted; the struct
# keeps its tensors alive.  What a call makes itself (outputs, workspaces) is made on
# the stream that is current: prepare a struct on the stream that it is launched on, or
# order the two.  The calls that prepare and launch in one do that for their ``stream``.
def _want(t, name, shape=None, dtype=None, device=None, host=False):
    """The checked address of a dense tensor: shape (None: any size there), type
    and device as stated; ``host`` allows pinned host memory read in place."""
    if shape is not None and (t.dim() != len(shape) or any(
            w is not None and w != n for w, n in zip(shape, t.shape))):
        raise PkvError(ERR_INVALID_ARG, f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if dtype is not None and t.dtype != dtype:
        raise PkvError(ERR_INVALID_ARG, f"{name}: {t.dtype}, expected {dtype}")
    if host and not t.is_cuda:
        return mapped_pointer(t)
    if device is not None and t.device != device:
        raise PkvError(ERR_INVALID_ARG, f"{name} is on {t.device}, expected {device}")
    return _ptr(t)


def _heads(t, name, T, d, dtype, device):
    """Address and token stride of ``t [T,H,d]`` whose heads are dense (a slice of
    a wider projection's output has a larger token stride)."""
    if t.dim() != 3 or t.shape[0] != T or t.shape[2] != d:
        raise PkvError(ERR_INVALID_ARG, f"{name}: shape {tuple(t.shape)}, expected [{T}, H, {d}]")
    if t.dtype != dtype or t.device != device or not t.is_cuda:
        raise PkvError(ERR_INVALID_ARG, f"{name}: {t.dtype} on {t.device}, expected {dtype} on "
                                        f"one CUDA device")
    if t.numel() and ((t.stride(2) != 1 and d > 1) or (t.stride(1) != d and t.shape[1] > 1)):
        raise PkvError(ERR_INVALID_ARG, f"{name}: the heads of a token must be dense")
    return _vp(t.data_ptr()), t.stride(0) if T > 1 else t.shape[1] * d


def _overlap(a, b):
    """Whether the memory of two non-empty tensors overlaps (by first and last byte)."""
    def span(t):
        last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
        return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()
    if not a.numel() or not b.numel():
        return False
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def _launch_on(args, stream):
    """The stream of a launch: ``stream`` or the current one, on the tensors' device."""
    device = args.current_device()
    if device != args.index:
        raise PkvError(ERR_INVALID_ARG, f"tensors are on cuda:{args.index}, the current device is "
                                        f"cuda:{device}")
    return args.current_stream(device) if stream is None else stream.cuda_stream


def _finish(args, device, keep):
    """What a launch of the struct needs besides its fields.  (The current device and
    stream as numbers where torch gives them: through its objects they were a quarter of
    a small call's 5.1 us.)"""
    torch = _torch()
    args.index, args.keep = device.index, keep
    args.current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    args.current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda d: torch.cuda.current_stream(d).cuda_stream)
    return args


class Rotary:
    """Rotary frequencies of a head of ``d`` elements (``pkv_rotary_init``): the
    first ``rot_dim`` rotate, in the ``"half"`` or ``"interleaved"`` layout, scaled
    ``"plain"``, ``"linear"``, ``"ntk"``, ``"ramp"`` or ``"bands"`` (include/pkv.h
    states the formulas)."""
    LAYOUTS = {"half": ROTARY_HALF, "interleaved": ROTARY_INTERLEAVED}
    SCALINGS = {"plain": ROTARY_PLAIN, "linear": ROTARY_LINEAR, "ntk": ROTARY_NTK,
                "ramp": ROTARY_RAMP, "bands": ROTARY_BANDS}

    def __init__(self, d, rot_dim=None, layout="half", scaling="plain", base=10000.0, factor=1.0,
                 low=1.0, high=32.0, original_len=0, amplitude=1.0):
        if layout not in self.LAYOUTS or scaling not in self.SCALINGS:
            raise PkvError(ERR_UNSUPPORTED, f"layout {layout!r}, scaling {scaling!r}")
        self.d, self.rot_dim = int(d), int(d if rot_dim is None else rot_dim)
        spec = RotarySpec(self.rot_dim, self.LAYOUTS[layout], self.SCALINGS[scaling],
                          int(original_len), float(base), float(factor), float(low), float(high),
                          float(amplitude))
        self.table = RotaryTable()
        _check(load().pkv_rotary_init(ctypes.byref(spec), self.d, ctypes.byref(self.table)))


def make_rotary_args(rotary, q, k, v, positions, q_out=None, k_out=None, slot_mapping=None,
                     k_cache=None, v_cache=None, err=None):
    """``pkv_rotary_args``: ``q [T,Hq,d]`` and ``k, v [T,Hkv,d]`` may be slices of
    one projection's output (any token stride); without ``slot_mapping`` nothing is
    appended and ``v`` may be None; ``q`` (with ``q_out``) or ``k`` may be None.
    ``q_out``/``k_out`` may be ``q``/``k`` themselves; ``k_out`` None reports no
    rotated keys (they still go to the cache)."""
    torch = _torch()
    first = q if q is not None else k
    if first is None or not first.is_cuda:
        raise PkvError(ERR_INVALID_ARG, "q or k must be a CUDA tensor")
    T, d, dt, dev = first.shape[0], first.shape[-1], first.dtype, first.device
    a = RotaryArgs()
    a.rotary = ctypes.pointer(rotary.table)
    a.T, a.d, a.dtype = T, d, dtype_code(first)
    if q is not None:
        if q_out is None:
            raise PkvError(ERR_INVALID_ARG, "q needs q_out")
        a.Hq = q.shape[1]
        a.q, a.q_stride = _heads(q, "q", T, d, dt, dev)
        a.q_out, a.q_out_stride = _heads(q_out, "q_out", T, d, dt, dev)
        if q_out.shape != q.shape:
            raise PkvError(ERR_INVALID_ARG, "q_out must have q's shape")
    if k is not None:
        a.Hkv = k.shape[1]
        a.k, a.k_stride = _heads(k, "k", T, d, dt, dev)
        if k_out is not None:
            a.k_out, a.k_out_stride = _heads(k_out, "k_out", T, d, dt, dev)
            if k_out.shape != k.shape:
                raise PkvError(ERR_INVALID_ARG, "k_out must have k's shape")
    a.positions = _want(positions, "positions", (T,), torch.int32, dev, host=True)
    if slot_mapping is not None:
        if k is None or v is None or k_cache is None or v_cache is None:
            raise PkvError(ERR_INVALID_ARG, "appending needs k, v and both caches")
        if v.shape != k.shape:
            raise PkvError(ERR_INVALID_ARG, "v must have k's shape")
        a.slot_mapping = _want(slot_mapping, "slot_mapping", (T,), torch.int64, dev, host=True)
        a.v, a.v_stride = _heads(v, "v", T, d, dt, dev)
        shape = (k_cache.shape[0], a.Hkv, BLOCK_SIZE, d)
        a.k_cache = _want(k_cache, "k_cache", shape, dt, dev)
        a.v_cache = _want(v_cache, "v_cache", shape, dt, dev)
        a.num_blocks = k_cache.shape[0]
    if err is not None:
        a.dev_err_flag = _want(err, "err", None, torch.int32, dev)
    return _finish(a, dev, (rotary, q, k, v, q_out, k_out, positions, slot_mapping, k_cache,
                            v_cache, err))


def set_rotary_inputs(layers, q, k, v):
    """Puts ``q [L,T,Hq,d]``, ``k``, ``v [L,T,Hkv,d]`` into prepared ``RotaryArgs``, one per
    layer, made for inputs of the same shapes, type and device (all three of them)."""
    for x, name, at in ((q, "q", 1), (k, "k", 2), (v, "v", 3)):
        old = layers[0].keep[at]
        if x.dim() != 4 or x.shape[0] != len(layers) or x.shape[1:] != old.shape:
            raise PkvError(ERR_INVALID_ARG, f"{name}: shape {tuple(x.shape)}, the calls were made for "
                                            f"{len(layers)} x {tuple(old.shape)}")
        first, stride = _heads(x[0], name, old.shape[0], old.shape[2], old.dtype, old.device)
        addr, step = first.value or 0, x.stride(0) * x.element_size()
        for i, a in enumerate(layers):
            setattr(a, name, addr + i * step)
            setattr(a, name + "_stride", stride)
    for a in layers:
        a.inputs = (q, k, v)


def rotary_append_args(args, stream=None):
    """Runs ``pkv_rotary_append`` from prepared ``RotaryArgs``."""
    _check(load().pkv_rotary_append(ctypes.byref(args), _launch_on(args, stream)))


def rotary_append(rotary, q, k, v, positions, slot_mapping=None, k_cache=None, v_cache=None,
                  q_out=None, k_out=None, err=None, stream=None):
    """Rotates ``q`` and ``k`` at ``positions`` and, with ``slot_mapping``, writes
    the rotated keys and the values into the cache slots; returns ``(q_out, k_out)``."""
    torch = _torch()
    with torch.cuda.stream(stream):
        if q is not None and q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
        rotary_append_args(make_rotary_args(rotary, q, k, v, positions, q_out, k_out, slot_mapping,
                                            k_cache, v_cache, err), stream)
    return q_out, k_out


def shared_plan_cap(B, n_prefixes, Hq, Hkv, num_ctas=0):
    """int32 words and partial slots that serve every plan of these sizes."""
    cap, slots = ctypes.c_int32(), ctypes.c_int32()
    _check(load().pkv_shared_plan_cap(int(B), int(n_prefixes), int(Hq), int(Hkv), int(num_ctas),
                                      ctypes.byref(cap), ctypes.byref(slots)))
    return cap.value, slots.value


def shared_plan(row_prefix, prefix_lens, Hq, Hkv, d, dtype, num_ctas=0, out=None):
    """Host plan of the shared-prefix attention (``pkv_shared_plan``): row b has
    prefix ``row_prefix[b]`` (negative: none) of ``prefix_lens[p]`` tokens.  Returns
    the plan (numpy int32, the used part of ``out`` if given)."""
    rows = np.ascontiguousarray(row_prefix, dtype=np.int32)
    lens = np.ascontiguousarray(prefix_lens, dtype=np.int32)
    if out is None:
        out = np.empty(shared_plan_cap(len(rows), len(lens), Hq, Hkv, num_ctas)[0], np.int32)
    n, slots = ctypes.c_int32(), ctypes.c_int32()
    _check(load().pkv_shared_plan(_np_ptr(rows, ctypes.c_int32), len(rows),
                                  _np_ptr(lens, ctypes.c_int32), len(lens), int(Hq), int(Hkv),
                                  int(d), int(dtype), int(num_ctas), _np_ptr(out, ctypes.c_int32),
                                  out.size, ctypes.byref(n), ctypes.byref(slots)))
    return out[:n.value]


def shared_default_parts(B, Hq, Hkv, d, dtype, bt_stride):
    """Partition of the own tokens that ``make_shared_args`` takes unless told."""
    n = ctypes.c_int32()
    _check(load().pkv_shared_default_parts(int(B), int(Hq), int(Hkv), int(d), int(dtype),
                                           int(bt_stride), ctypes.byref(n)))
    return n.value


def shared_short(B, Hq, Hkv, d, dtype, bt_stride, pt_stride=0):
    """Whether a call without ``num_parts``, ``plan`` and flags takes the one-kernel form for
    short contexts (``pt_stride`` 0: no prefixes)."""
    n = ctypes.c_int32()
    _check(load().pkv_shared_short(int(B), int(Hq), int(Hkv), int(d), int(dtype), int(bt_stride),
                                   int(pt_stride), ctypes.byref(n)))
    return bool(n.value)


def shared_workspace_bytes(B, Hq, Hkv, d, num_parts, slots):
    n = _size_t()
    _check(load().pkv_shared_workspace_bytes(int(B), int(Hq), int(Hkv), int(d), int(num_parts),
                                             int(slots), ctypes.byref(n)))
    return n.value


def alloc_scores(num_blocks, Hq, device=None):
    """Scratch of the weights' accumulation: the scores of every cache slot."""
    torch = _torch()
    return torch.empty((num_blocks, Hq * BLOCK_SIZE), dtype=torch.float32, device=device or "cuda")


def make_shared_args(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, out,
                     prefix_tables=None, prefix_plan=None, slots=None, num_ctas=None, mass=None,
                     scores=None, mass_lens=None, decay=1.0, lse=None, attn_bias=None, plan=None,
                     num_parts=None, workspace=None, flags=0, err=None):
    """``pkv_shared_args``.  ``prefix_plan`` is ``shared_plan``'s output on the
    device (or pinned); ``slots`` and ``num_ctas`` are read from it once unless
    given (give them, with a workspace for ``slots``, when the buffer will later
    hold other plans).  Without ``num_parts`` and ``plan`` short contexts are computed
    by one kernel (``shared_short``), the rest in ``shared_default_parts`` parts."""
    torch = _torch()
    if q_rot.dim() != 3 or k_cache.dim() != 4 or not q_rot.is_cuda:
        raise PkvError(ERR_INVALID_ARG, "q_rot must be [B,Hq,d] and the caches [blocks,Hkv,16,d], "
                                        "on a CUDA device")
    B, Hq, d = q_rot.shape
    nb, Hkv = k_cache.shape[0], k_cache.shape[1]
    dt, dev = q_rot.dtype, q_rot.device
    i32, f32 = torch.int32, torch.float32
    a = SharedArgs()
    a.dtype = dtype_code(q_rot)
    a.q_rot = _want(q_rot, "q_rot", (B, Hq, d), dt, dev)
    a.k_cache = _want(k_cache, "k_cache", (nb, Hkv, BLOCK_SIZE, d), dt, dev)
    a.v_cache = _want(v_cache, "v_cache", (nb, Hkv, BLOCK_SIZE, d), dt, dev)
    a.block_tables = _want(block_tables, "block_tables", (B, None), i32, dev, host=True)
    a.seq_lens = _want(seq_lens, "seq_lens", (B,), i32, dev, host=True)
    a.out = _want(out, "out", (B, Hq, d), dt, dev)
    if _overlap(out, q_rot):
        raise PkvError(ERR_INVALID_ARG, "out must not overlap q_rot")
    a.num_blocks, a.bt_stride = nb, block_tables.shape[1]
    a.B, a.Hq, a.Hkv, a.d = B, Hq, Hkv, d
    a.scale, a.mass_decay, a.flags = float(scale), float(decay), int(flags)
    if attn_bias is not None:
        a.attn_bias = _want(attn_bias, "attn_bias", (B, None), f32, dev)
        a.bias_stride = attn_bias.shape[1]
    if plan is not None:
        if num_parts is None:
            num_parts = plan.shape[0]
        a.plan = _want(plan, "plan", (num_parts, PLAN_INTS), i32, dev, host=True)
    if prefix_tables is not None and prefix_tables.shape[0] > 0:
        if prefix_plan is None:
            raise PkvError(ERR_INVALID_ARG, "prefix_tables need a prefix_plan")
        a.prefix_tables = _want(prefix_tables, "prefix_tables", (None, None), i32, dev, host=True)
        a.n_prefixes, a.pt_stride = prefix_tables.shape
        a.prefix_plan = _want(prefix_plan, "prefix_plan", (None,), i32, dev, host=True)
        a.plan_ints = prefix_plan.numel()
        if slots is None or num_ctas is None:
            head = prefix_plan[:8].cpu().tolist()
            slots = head[3] if slots is None else slots
            num_ctas = head[4] if num_ctas is None else num_ctas
        a.slots, a.num_ctas = int(slots), int(num_ctas)
    if mass is not None:
        if scores is None:
            raise PkvError(ERR_INVALID_ARG, "mass needs scores (alloc_scores)")
        a.mass = _want(mass, "mass", (nb, Hkv, BLOCK_SIZE), f32, dev)
        a.scores = _want(scores, "scores", (nb, Hq * BLOCK_SIZE), f32, dev)
        if mass_lens is not None:
            a.mass_lens = _want(mass_lens, "mass_lens", (B,), i32, dev, host=True)
    if lse is not None:
        a.lse_out = _want(lse, "lse", (B, Hq), f32, dev)
    if err is not None:
        a.dev_err_flag = _want(err, "err", None, i32, dev)
    a.num_parts = int(num_parts or 0)
    if workspace is None and B > 0:
        parts = a.num_parts or shared_default_parts(B, Hq, Hkv, d, a.dtype, block_tables.shape[1])
        nbytes = shared_workspace_bytes(B, Hq, Hkv, d, parts, a.slots)
        workspace = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    if workspace is not None:
        a.workspace = _want(workspace, "workspace", (None,), torch.uint8, dev)
        a.workspace_bytes = workspace.numel()
    return _finish(a, dev, (q_rot, k_cache, v_cache, block_tables, seq_lens, out, prefix_tables,
                            prefix_plan, mass, scores, mass_lens, lse, attn_bias, plan, workspace,
                            err))


def decode_attn_shared_args(args, stream=None):
    """Runs ``pkv_decode_attn_shared`` from prepared ``SharedArgs``."""
    _check(load().pkv_decode_attn_shared(ctypes.byref(args), _launch_on(args, stream)))


def decode_attention_shared(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, out=None,
                            stream=None, **kw):
    """Attention over shared prefixes and own tokens: returns ``out [B,Hq,d]`` (see
    ``make_shared_args`` for the rest)."""
    torch = _torch()
    with torch.cuda.stream(stream):
        out = torch.empty_like(q_rot) if out is None else out
        args = make_shared_args(q_rot, k_cache, v_cache, block_tables, seq_lens, scale, out, **kw)
        decode_attn_shared_args(args, stream)
    return out


def evict_workspace_bytes(B, Hkv, d, dtype, max_keep):
    n = _size_t()
    _check(load().pkv_evict_workspace_bytes(int(B), int(Hkv), int(d), int(dtype), int(max_keep),
                                            ctypes.byref(n)))
    return n.value


def make_evict_args(k_cache, v_cache, mass, block_tables, seq_lens, keep_lens, kept, sink=0,
                    recent=0, workspace=None, err=None):
    """``pkv_evict_args``: ``kept [B,Hkv,>=kept tokens]`` int32 receives the kept
    tokens' indices; ``workspace`` (uint8, ``evict_workspace_bytes``) is made here
    unless given."""
    torch = _torch()
    if k_cache.dim() != 4 or not k_cache.is_cuda:
        raise PkvError(ERR_INVALID_ARG, "caches must be [blocks,Hkv,16,d] on a CUDA device")
    nb, Hkv, _, d = k_cache.shape
    B, dt, dev, i32 = block_tables.shape[0], k_cache.dtype, k_cache.device, torch.int32
    a = EvictArgs()
    a.dtype = dtype_code(k_cache)
    a.k_cache = _want(k_cache, "k_cache", (nb, Hkv, BLOCK_SIZE, d), dt, dev)
    a.v_cache = _want(v_cache, "v_cache", (nb, Hkv, BLOCK_SIZE, d), dt, dev)
    a.mass = _want(mass, "mass", (nb, Hkv, BLOCK_SIZE), torch.float32, dev)
    a.block_tables = _want(block_tables, "block_tables", (B, None), i32, dev, host=True)
    a.seq_lens = _want(seq_lens, "seq_lens", (B,), i32, dev, host=True)
    a.keep_lens = _want(keep_lens, "keep_lens", (B,), i32, dev, host=True)
    a.kept = _want(kept, "kept", (B, Hkv, None), i32, dev)
    if err is not None:
        a.dev_err_flag = _want(err, "err", None, i32, dev)
    a.num_blocks, a.bt_stride, a.kept_stride = nb, block_tables.shape[1], kept.shape[2]
    a.sink, a.recent = int(sink), int(recent)
    a.B, a.Hkv, a.d = B, Hkv, d
    if workspace is None:
        workspace = torch.empty(evict_workspace_bytes(B, Hkv, d, a.dtype, kept.shape[2]),
                                dtype=torch.uint8, device=dev)
    a.workspace = _want(workspace, "workspace", (None,), torch.uint8, dev)
    a.workspace_bytes = workspace.numel()
    return _finish(a, dev, (k_cache, v_cache, mass, block_tables, seq_lens, keep_lens, kept,
                            workspace, err))


def evict_args(args, stream=None):
    """Runs ``pkv_evict`` from prepared ``EvictArgs``."""
    _check(load().pkv_evict(ctypes.byref(args), _launch_on(args, stream)))


def evict(k_cache, v_cache, mass, block_tables, seq_lens, keep_lens, max_keep, sink=0, recent=0,
          kept=None, err=None, stream=None):
    """Evicts rows down to ``keep_lens`` tokens by ``mass``; returns ``kept
    [B,Hkv,max_keep]``, the indices of the tokens kept."""
    torch = _torch()
    with torch.cuda.stream(stream):
        if kept is None:
            kept = torch.empty((block_tables.shape[0], k_cache.shape[1], max(int(max_keep), 1)),
                               dtype=torch.int32, device=k_cache.device)
        evict_args(make_evict_args(k_cache, v_cache, mass, block_tables, seq_lens, keep_lens, kept,
                                   sink, recent, err=err), stream)
    return kept


def pool_blocks(budget_bytes, n_layers, Hkv, d, dtype):
    """Blocks of a K/V pool for ``n_layers`` layers that fit in ``budget_bytes``."""
    n = ctypes.c_int32()
    _check(load().pkv_pool_blocks(int(budget_bytes), int(n_layers), int(Hkv), int(d),
                                  int(dtype), ctypes.byref(n)))
    return n.value


def decode_step_host(args, host_io, stream=None):
    """End-to-end step from host buffers (see ``pkv_decode_step_host``)."""
    _check(load().pkv_decode_step_host(ctypes.byref(args), ctypes.byref(host_io),
                                       _stream(stream)))


HOST_IN_PLACE = 1


class StepGraph:
    """``pkv_step_graph``: the host step for fixed buffers captured once;
    ``launch()`` runs one step and waits for its output in host memory."""

    def __init__(self, args, io):
        self._lib = load()
        self._keep = (args, io)
        h = _vp()
        _check(self._lib.pkv_step_graph_create(ctypes.byref(args), ctypes.byref(io),
                                               ctypes.byref(h)))
        self._h = h

    def launch(self, stream=None):
        _check(self._lib.pkv_step_graph_launch(self._h, _stream(stream)))

    def enqueue(self, stream=None):
        """The launch without the wait (``wait`` waits for the last one)."""
        _check(self._lib.pkv_step_graph_enqueue(self._h, _stream(stream)))

    def wait(self):
        """Waits for this graph's last ``enqueue`` (its output is then set)."""
        _check(self._lib.pkv_step_graph_wait(self._h))

    def close(self):
        if self._h:
            self._lib.pkv_step_graph_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def host_io(q, k, v, positions, slot_mapping, seq_lens, block_tables, out, flags=0, plan=None):
    """``pkv_step_host_io`` over host (CPU, ideally pinned; pinned for
    ``HOST_IN_PLACE``) torch tensors."""
    io = StepHostIO()
    io.flags = int(flags)
    for name, t in (("q", q), ("k", k), ("v", v), ("positions", positions),
                    ("slot_mapping", slot_mapping), ("seq_lens", seq_lens),
                    ("block_tables", block_tables), ("out", out), ("plan", plan)):
        if t is None and name == "plan":
            continue
        if t.is_cuda or not t.is_contiguous():
            raise PkvError(ERR_INVALID_ARG, f"{name} must be a contiguous host tensor")
        setattr(io, name, _vp(t.data_ptr()))
    return io


class Server:
    """The native serving loop (``pkv_server``) over a single-layer
    ``engine.PagedDecoder``'s device buffers for the sequences ``rows`` (one
    per row); joins and leaves then go through ``step``.  Holds the pinned host
    buffers the server needs."""

    def __init__(self, dec, rows, max_prefix_tokens):
        torch = _torch()
        lib = load()
        B = len(rows)
        self.B, self._lib = B, lib
        nb = lib.pkv_server_meta_bytes(B, dec.bt_stride, dec.num_parts)
        pb = lib.pkv_server_prefix_bytes(int(max_prefix_tokens))
        self.meta = [torch.empty(nb, dtype=torch.uint8).pin_memory() for _ in range(2)]
        self.prefix = [torch.empty(max(pb, 16), dtype=torch.uint8).pin_memory() for _ in range(2)]
        self.rows_in = np.ascontiguousarray(rows, dtype=np.int32)
        step = make_step_args(dec.q_in[:B], dec.k_in[:B], dec.v_in[:B], dec.q_rot[:B],
                              dec.k_rot[:B], dec.k_cache, dec.v_cache, dec.positions[:B],
                              dec.slots[:B], dec.seq_lens[:B], dec.tables[:B], dec.scale,
                              dec.rope_base, dec.num_parts, dec.workspace, dec.out[:B],
                              flags=dec.flags, err=dec.err)
        self.desc = ServerDesc()
        self.desc.step = step
        self.desc.alloc = dec.alloc._h
        self.desc.rows = self.rows_in.ctypes.data_as(_vp)
        for t in range(2):
            self.desc.meta_host[t] = _vp(self.meta[t].data_ptr())
            self.desc.prefix_host[t] = _vp(self.prefix[t].data_ptr())
        self.desc.max_prefix_tokens = int(max_prefix_tokens)
        h = _vp()
        _check(lib.pkv_server_create(ctypes.byref(self.desc), ctypes.byref(h)))
        self._h = h

    def step(self, leave_rows, prefix_lens, prefix_k=None, prefix_v=None, q=None, k=None,
             v=None, stream=None):
        """One step (see ``pkv_server_step``); leave_rows and prefix_lens are
        int32 numpy arrays of the same length."""
        lr = np.ascontiguousarray(leave_rows, dtype=np.int32)
        pl = np.ascontiguousarray(prefix_lens, dtype=np.int32)
        if len(lr) != len(pl):
            raise PkvError(ERR_INVALID_ARG, "one prefix length per leaving row")
        _check(self._lib.pkv_server_step(
            self._h, _np_ptr(lr, ctypes.c_int32), _np_ptr(pl, ctypes.c_int32), len(lr),
            _ptr(prefix_k), _ptr(prefix_v), _ptr(q), _ptr(k), _ptr(v), _stream(stream)))

    def step_runner(self, leave_rows, prefix_lens, prefix_k=None, prefix_v=None, q=None, k=None,
                    v=None, stream=None):
        """A no-argument callable running this step with every argument
        converted once (a loop that replays a planned schedule)."""
        lr = np.ascontiguousarray(leave_rows, dtype=np.int32)
        pl = np.ascontiguousarray(prefix_lens, dtype=np.int32)
        if len(lr) != len(pl):
            raise PkvError(ERR_INVALID_ARG, "one prefix length per leaving row")
        args = (self._h, _np_ptr(lr, ctypes.c_int32), _np_ptr(pl, ctypes.c_int32), len(lr),
                _ptr(prefix_k), _ptr(prefix_v), _ptr(q), _ptr(k), _ptr(v), _stream(stream))
        fn, keep = self._lib.pkv_server_step, (lr, pl, prefix_k, prefix_v, q, k, v)

        def run():
            _check(fn(*args))
            return keep
        return run

    def rows(self):
        out = np.empty(self.B, np.int32)
        _check(self._lib.pkv_server_rows(self._h, _np_ptr(out, ctypes.c_int32, self.B)))
        return out

    def close(self):
        if self._h:
            self._lib.pkv_server_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
