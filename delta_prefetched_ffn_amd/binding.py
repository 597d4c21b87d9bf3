"""ctypes binding of libnp.so (include/np.h): argument marshalling only.

Every step of the method runs in the HIP library; this module converts Python
arguments (NumPy arrays on the host, integer device pointers and stream
handles, e.g. torch's `tensor.data_ptr()` and `stream.cuda_stream`) into the
C ABI's plain pointers and sizes, and turns error codes into exceptions. It
raises at import time of the library if libnp.so has not been built; there is
no fallback path.
"""
from __future__ import annotations

import array
import ctypes
import os
from functools import lru_cache

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnp.so")

NP_OK, NP_EINVAL, NP_ECAPACITY, NP_ENOMEM, NP_EHIP, NP_ESTATE, NP_EDEVICE = range(7)
MASK_UNION, MASK_INTERSECT, MASK_SINGLE = 0, 1, 2
MODES = {"union": MASK_UNION, "intersect": MASK_INTERSECT, "single": MASK_SINGLE}
ACT_RELU, ACT_SILU = 0, 1
REDUCE_ATOMIC, REDUCE_ORDERED = 0, 1
REDUCES = {"atomic": REDUCE_ATOMIC, "ordered": REDUCE_ORDERED}
LAYOUTS = {"slots": 0, "compact": 1}
ACTS = {"relu": ACT_RELU, "silu": ACT_SILU}
DTYPES = {"f32": 0, "bf16": 1, "f16": 2}
KV_HOST = -1
KV_MODES = {"share": 0, "copy": 1}
_NAMES = {0: "NP_OK", 1: "NP_EINVAL", 2: "NP_ECAPACITY", 3: "NP_ENOMEM", 4: "NP_EHIP",
          5: "NP_ESTATE", 6: "NP_EDEVICE"}

# every symbol include/np.h declares
EXPORTS = ["np_layer_create", "np_layer_destroy", "np_layer_reset", "np_delta_assign",
           "np_scatter_rows", "np_sparse_ffn", "np_decode_step", "np_layer_read_state",
           "np_layer_read_rows", "np_layer_info", "np_layer_counters", "np_layer_set_ffn_shape", "np_last_error",
           "np_layer_raise_error", "np_probe_read", "np_probe_read_set", "np_probe_copy", "np_decode_use_graphs", "np_layer_set_window",
           "np_sparse_ffn_acc", "np_layer_set_ffn_reduce", "np_layer_set_levels",
           "np_layer_set_layout", "np_layer_read_moves", "np_decode_set_staging",
           "np_layer_set_planar", "np_sparse_ffn_noalloc",
           "np_kv_bytes", "np_kv_create", "np_kv_destroy", "np_kv_reset", "np_kv_extend", "np_kv_append",
           "np_kv_attend", "np_kv_fork", "np_kv_trim", "np_kv_free", "np_kv_adopt", "np_kv_evict",
           "np_kv_compact", "np_kv_read_pages", "np_kv_read_tokens", "np_kv_info"]


class NPError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{_NAMES.get(status, status)}: {msg}")
        self.status = status


class LayerDesc(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("k_max", ctypes.c_int32),
                ("n_rows", ctypes.c_int32), ("n_centroids", ctypes.c_int32),
                ("mask_mode", ctypes.c_int32), ("act", ctypes.c_int32), ("device", ctypes.c_int32),
                ("masks", ctypes.c_void_p), ("row_store", ctypes.c_void_p)]


class KVDesc(ctypes.Structure):
    _fields_ = [(k, ctypes.c_int32) for k in ("n_layers", "n_heads", "n_kv_heads", "head_dim", "page_tokens", "n_pages",
                                              "max_seqs", "max_pages", "device")] + \
               [("codes", ctypes.c_void_p), ("exps", ctypes.c_void_p)]


@lru_cache(maxsize=1)
def lib() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -m delta_prefetched_ffn_amd.build` "
                           "(the HIP library is required; there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    sig = {
        "np_layer_create": [ctypes.POINTER(LayerDesc), ctypes.POINTER(vp)],
        "np_layer_destroy": [vp],
        "np_layer_reset": [vp],
        "np_delta_assign": [vp, i32, i32, vp],
        "np_scatter_rows": [vp, vp],
        "np_sparse_ffn": [vp, vp, vp, vp],
        "np_decode_step": [vp, i32, vp, vp, vp, vp, vp],
        "np_layer_read_state": [vp, vp, vp, vp, vp, vp, vp, vp],
        "np_layer_read_rows": [vp, vp, i32, vp],
        "np_layer_info": [vp, vp],
        "np_layer_counters": [vp, vp],
        "np_layer_set_ffn_shape": [vp, i32, i32, i32],
        "np_layer_raise_error": [vp, i32, vp],
        "np_probe_read": [vp, i64, vp, vp],
        "np_probe_read_set": [vp, i32, i64, i32, vp, vp],
        "np_probe_copy": [vp, vp, i64, vp],
        "np_decode_use_graphs": [i32],
        "np_layer_set_window": [vp, i32],
        "np_sparse_ffn_acc": [vp, vp, vp, vp],
        "np_layer_set_ffn_reduce": [vp, i32],
        "np_layer_set_levels": [vp, i32, vp],
        "np_layer_set_layout": [vp, i32],
        "np_layer_read_moves": [vp, vp, vp, vp],
        "np_decode_set_staging": [i64, i32],
        "np_layer_set_planar": [vp, i32],
        "np_sparse_ffn_noalloc": [vp, vp, vp, vp],
        "np_kv_bytes": [vp, vp],
        "np_kv_create": [vp, vp],
        "np_kv_destroy": [vp],
        "np_kv_reset": [vp],
        "np_kv_extend": [vp, i32, vp, vp, vp],
        "np_kv_append": [vp, i32, vp, vp, i32, vp, vp],
        "np_kv_attend": [vp, i32, vp, vp, vp, i32, vp, ctypes.c_float, i32, i32, vp],
        "np_kv_fork": [vp, i32, i32, i32, i32, vp],
        "np_kv_trim": [vp, i32, i32],
        "np_kv_free": [vp, i32],
        "np_kv_adopt": [vp, i32, vp, i32, i32],
        "np_kv_evict": [vp, i32, i32, i32, vp],
        "np_kv_compact": [vp, vp, vp],
        "np_kv_read_pages": [vp, i32, vp, i32, vp, vp],
        "np_kv_read_tokens": [vp, i32, i32, i32, i32, vp, vp],
        "np_kv_info": [vp, vp],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    L.np_last_error.argtypes = []
    L.np_last_error.restype = ctypes.c_char_p
    return L


def _check(status: int) -> None:
    if status != NP_OK:
        raise NPError(status, lib().np_last_error().decode())


def _ptr(a: np.ndarray | None) -> int | None:
    return None if a is None else a.ctypes.data


def _i32(x: int) -> int:
    """x, if it fits the C ABI's 32 bits (ctypes would cut it)."""
    if not -(1 << 31) <= x < 1 << 31:
        raise OverflowError(f"{x} does not fit in 32 bits")
    return x


class Layer:
    """One sparse FFN layer (np_layer). row_store is a device or pinned-host pointer (int)."""

    def __init__(self, *, d_model: int, d_ff: int, k_max: int, n_rows: int, masks: np.ndarray,
                 mask_mode: int, row_store: int, device: int = 0, act: int = ACT_RELU,
                 keepalive=None):
        masks = np.ascontiguousarray(masks, dtype=np.uint64)
        n_tables = 1 if mask_mode == MASK_SINGLE else 2
        W = (d_ff + 63) // 64
        assert masks.ndim == 3 and masks.shape[0] == n_tables and masks.shape[2] == W, masks.shape
        desc = LayerDesc(d_model, d_ff, k_max, n_rows, masks.shape[1], mask_mode, act, device,
                         masks.ctypes.data, row_store)
        h = ctypes.c_void_p()
        _check(lib().np_layer_create(ctypes.byref(desc), ctypes.byref(h)))
        self.h = h
        self.d_model, self.d_ff, self.k_max, self.n_rows = d_model, d_ff, k_max, n_rows
        self._keepalive = keepalive

    def close(self) -> None:
        if self.h:
            _check(lib().np_layer_destroy(self.h))
            self.h = ctypes.c_void_p()

    def __del__(self):
        try:
            if getattr(self, "h", None):
                lib().np_layer_destroy(self.h)
        except Exception:
            pass

    def reset(self) -> None:
        _check(lib().np_layer_reset(self.h))

    def delta_assign(self, gate_cid: int, up_cid: int, stream: int = 0) -> None:
        _check(lib().np_delta_assign(self.h, gate_cid, up_cid, stream or None))

    def scatter_rows(self, stream: int = 0) -> None:
        _check(lib().np_scatter_rows(self.h, stream or None))

    def sparse_ffn(self, x_ptr: int, y_ptr: int, stream: int = 0) -> None:
        _check(lib().np_sparse_ffn(self.h, x_ptr, y_ptr, stream or None))

    def set_ffn_shape(self, slots_per_wg: int = 0, tile_cols: int = 0, threads: int = 0) -> None:
        _check(lib().np_layer_set_ffn_shape(self.h, slots_per_wg, tile_cols, threads))

    def sparse_ffn_acc(self, x_ptr: int, y_ptr: int, stream: int = 0) -> None:
        """y += FFN(x)."""
        _check(lib().np_sparse_ffn_acc(self.h, x_ptr, y_ptr, stream or None))

    def sparse_ffn_noalloc(self, x_ptr: int, y_ptr: int, stream: int = 0) -> None:
        """np_sparse_ffn_noalloc: the FFN with its exchange words in the library's static scratch."""
        _check(lib().np_sparse_ffn_noalloc(self.h, x_ptr, y_ptr, stream or None))

    def set_ffn_reduce(self, mode: str) -> None:
        """"ordered" (default; atomics-free, fixed order, bit-reproducible) or "atomic" (fp32 atomics, order free)."""
        _check(lib().np_layer_set_ffn_reduce(self.h, REDUCES[mode]))

    def set_window(self, window: int) -> None:
        """Residency window in tokens (1 = the buffer holds exactly the active set)."""
        _check(lib().np_layer_set_window(self.h, window))

    def set_levels(self, levels, n_levels: int) -> None:
        """Retention by frequency level: levels uint8 [d_ff], each < n_levels (0 switches it off)."""
        if n_levels == 0:
            _check(lib().np_layer_set_levels(self.h, 0, None))
            return
        lv = np.ascontiguousarray(levels, dtype=np.uint8)
        assert lv.shape == (self.d_ff,), lv.shape
        _check(lib().np_layer_set_levels(self.h, n_levels, lv.ctypes.data))

    def set_layout(self, layout: str) -> None:
        """"slots" (slot map, the default) or "compact" (active rows at positions 0 .. |S|-1)."""
        _check(lib().np_layer_set_layout(self.h, LAYOUTS[layout]))

    def set_planar(self, planar: bool) -> None:
        """Slot buffer as one plane per row kind (True) or one bundle per slot (False, the default)."""
        _check(lib().np_layer_set_planar(self.h, 1 if planar else 0))

    def raise_error(self, bits: int, stream: int = 0) -> None:
        """Raise device error bits as a failing kernel would (tests of error reporting)."""
        _check(lib().np_layer_raise_error(self.h, bits, stream or None))

    def read_moves(self) -> tuple[np.ndarray, np.ndarray]:
        """(src, dst) positions of the rows the last assignment moved (compact layout)."""
        src = np.empty(self.k_max, dtype=np.int32)
        dst = np.empty(self.k_max, dtype=np.int32)
        n = ctypes.c_int32(0)
        _check(lib().np_layer_read_moves(self.h, src.ctypes.data, dst.ctypes.data, ctypes.byref(n)))
        return src[: n.value].copy(), dst[: n.value].copy()

    def info(self) -> dict:
        out = np.zeros(6, dtype=np.int32)
        _check(lib().np_layer_info(self.h, out.ctypes.data))
        return dict(zip(["d_model", "d_ff", "k_max", "n_rows", "n_active", "n_in"], out.tolist()))

    def counters(self) -> tuple[int, int]:
        """(sum of |S|, sum of |D_in|) over accepted assignments since create/reset."""
        out = np.zeros(2, dtype=np.int64)
        _check(lib().np_layer_counters(self.h, out.ctypes.data))
        return int(out[0]), int(out[1])

    def read_state(self, check: bool = True) -> dict:
        K, M = self.k_max, self.d_ff
        st = {k: np.empty(K, dtype=np.int32) for k in ("owner", "d_in", "slot_in", "d_out", "act")}
        st["slot_map"] = np.empty(M, dtype=np.int32)
        counts = np.empty(4, dtype=np.int32)
        rc = lib().np_layer_read_state(self.h, _ptr(st["slot_map"]), _ptr(st["owner"]), _ptr(st["d_in"]),
                                       _ptr(st["slot_in"]), _ptr(st["d_out"]), _ptr(st["act"]),
                                       counts.ctypes.data)
        if check:
            _check(rc)
        n_in, n_out, n_act, err = counts.tolist()
        st["d_in"] = st["d_in"][:n_in]
        st["slot_in"] = st["slot_in"][:n_in]
        st["d_out"] = st["d_out"][:n_out]
        st["act"] = st["act"][:n_act]
        st["err"] = err
        return st

    def read_rows(self, slots=None) -> np.ndarray:
        """uint16 bf16 bits [n][n_rows][d_model]; slots=None reads the whole buffer."""
        if slots is None:
            out = np.empty((self.k_max, self.n_rows, self.d_model), dtype=np.uint16)
            _check(lib().np_layer_read_rows(self.h, None, self.k_max, out.ctypes.data))
            return out
        s = np.ascontiguousarray(slots, dtype=np.int32)
        out = np.empty((s.size, self.n_rows, self.d_model), dtype=np.uint16)
        _check(lib().np_layer_read_rows(self.h, s.ctypes.data, s.size, out.ctypes.data))
        return out


def kv_bytes(*, n_layers: int, n_heads: int, n_kv_heads: int, head_dim: int, page_tokens: int, n_pages: int,
             max_seqs: int = 1, max_pages: int = 1) -> tuple[int, int]:
    """Bytes of a cache's pool: (codes, exps)."""
    desc = KVDesc(*map(_i32, (n_layers, n_heads, n_kv_heads, head_dim, page_tokens, n_pages, max_seqs, max_pages)), KV_HOST, None, None)
    out = (ctypes.c_int64 * 2)()
    _check(lib().np_kv_bytes(ctypes.byref(desc), out))
    return out[0], out[1]


class KVCache:
    """An 8-bit key/value cache (np_kv). codes and exps are device pointers (ints) to the caller's pool of
    kv_bytes() bytes; device KV_HOST (no pool) keeps the books only."""

    def __init__(self, *, n_layers: int, n_heads: int, n_kv_heads: int, head_dim: int, page_tokens: int, n_pages: int,
                 max_seqs: int, max_pages: int, codes: int = 0, exps: int = 0, device: int = 0, keepalive=None):
        desc = KVDesc(*map(_i32, (n_layers, n_heads, n_kv_heads, head_dim, page_tokens, n_pages, max_seqs, max_pages, device)),
                      codes or None, exps or None)
        h = ctypes.c_void_p()
        _check(lib().np_kv_create(ctypes.byref(desc), ctypes.byref(h)))
        self.h = h
        self.n_layers, self.n_heads, self.n_kv_heads, self.head_dim = n_layers, n_heads, n_kv_heads, head_dim
        self.page_tokens, self.n_pages, self.max_seqs, self.max_pages = page_tokens, n_pages, max_seqs, max_pages
        self._keepalive = keepalive
        # What the page calls hand back, kept: they run between decode steps.
        self._pages = (ctypes.c_int32 * max_pages)()
        self._n = ctypes.c_int32(0)
        self._n_ref, self._pages_at = ctypes.byref(self._n), ctypes.addressof(self._pages)
        # The calls of every layer and token: their functions and the strides in use, looked up once.
        self._append, self._attend, self._strides = lib().np_kv_append, lib().np_kv_attend, {None: None}

    def close(self) -> None:
        if self.h:
            _check(lib().np_kv_destroy(self.h))
            self.h = ctypes.c_void_p()

    def __del__(self):
        try:
            if getattr(self, "h", None):
                lib().np_kv_destroy(self.h)
        except Exception:
            pass

    def reset(self) -> None:
        _check(lib().np_kv_reset(self.h))

    def extend(self, seqs, n_new, stream: int = 0) -> None:
        """seqs[i] gets n_new[i] more tokens; they become the current tokens of append and attend."""
        n = len(seqs)
        if len(n_new) != n:
            raise ValueError(f"extend: {n} sequences and {len(n_new)} counts")
        s, c = array.array("i", seqs), array.array("i", n_new)
        _check(lib().np_kv_extend(self.h, n, s.buffer_info()[0], c.buffer_info()[0], stream or None))

    def append(self, layer: int, k_ptr: int, v_ptr: int, dtype: str, strides=None, stream: int = 0) -> None:
        """Stores the current tokens' k, v [rows][n_kv_heads][head_dim]; strides (elements): k row, k head, v row, v head."""
        if layer >> 31 > 0:
            _i32(layer)
        rc = self._append(self.h, layer, k_ptr, v_ptr, DTYPES[dtype], self._stride_array(strides), stream or None)
        if rc:
            _check(rc)

    def _stride_array(self, strides):
        try:
            return self._strides[strides]
        except (KeyError, TypeError):   # new ones, or a list
            four = array.array("q", strides)
            if len(four) != 4:
                raise ValueError(f"strides: {len(four)} numbers instead of 4")
            if len(self._strides) > 64:
                self._strides = {None: None}
            return self._strides.setdefault(tuple(four), (ctypes.c_int64 * 4)(*four))

    def attend(self, layer: int, q_ptr: int, out_ptr: int, dtype: str, strides=None, *, scale: float, window: int = 0,
               sinks: int = 0, lse_ptr: int = 0, stream: int = 0) -> None:
        """Attention of the current tokens: q, out [rows][n_heads][head_dim]; strides (elements): q row, q head, out row,
        out head; window 0: every earlier token, else the last `window` and the first `sinks`."""
        if (layer | window | sinks) >> 31 > 0:
            for x in (layer, window, sinks):
                _i32(x)
        rc = self._attend(self.h, layer, q_ptr, out_ptr, lse_ptr or None, DTYPES[dtype], self._stride_array(strides), scale,
                          window, sinks, stream or None)
        if rc:
            _check(rc)

    def fork(self, src: int, dst: int, n_tokens: int, mode: str = "share", stream: int = 0) -> None:
        """The empty sequence dst becomes the first n_tokens of src ("share": shared pages, copied on write; "copy")."""
        _check(lib().np_kv_fork(self.h, _i32(src), _i32(dst), _i32(n_tokens), KV_MODES[mode], stream or None))

    def trim(self, seq: int, n_tokens: int) -> None:
        _check(lib().np_kv_trim(self.h, _i32(seq), _i32(n_tokens)))

    def free(self, seq: int) -> None:
        _check(lib().np_kv_free(self.h, _i32(seq)))

    def adopt(self, seq: int, pages, n_tokens: int, stream: int = 0) -> None:
        """The empty sequence seq becomes these pages of the pool, holding n_tokens tokens (nothing is enqueued)."""
        if isinstance(pages, list):
            p = array.array("i", pages)
            at, n = p.buffer_info()
        else:
            given = np.asarray(pages)
            if given.ndim != 1 or (given.size and given.dtype.kind not in "iu"):
                raise TypeError("pages must be a list of whole numbers")
            if given.size:
                _i32(int(given.min()))
                _i32(int(given.max()))
            p = np.ascontiguousarray(given, dtype=np.int32)
            at, n = p.ctypes.data, p.size
        _check(lib().np_kv_adopt(self.h, _i32(seq), at, n, _i32(n_tokens)))

    def evict(self, seq: int, window: int, sinks: int = 0, stream: int = 0) -> int:
        """Drops the pages that no later query of this window sees; how many (nothing is enqueued)."""
        n = ctypes.c_int32(0)
        _check(lib().np_kv_evict(self.h, _i32(seq), _i32(window), _i32(sinks), ctypes.byref(n)))
        return n.value

    def compact(self, stream: int = 0) -> int:
        """Moves the pages in use to the front of the pool; how many moved."""
        n = ctypes.c_int32(0)
        _check(lib().np_kv_compact(self.h, ctypes.byref(n), stream or None))
        return n.value

    def pages(self, seq: int) -> np.ndarray:
        _check(lib().np_kv_read_pages(self.h, _i32(seq), self._pages_at, self.max_pages, self._n_ref, None))
        return np.frombuffer(self._pages, np.int32, self._n.value).copy() if self._n.value else np.empty(0, np.int32)

    def tokens(self, seq: int) -> int:
        t = ctypes.c_int32(0)
        _check(lib().np_kv_read_pages(self.h, _i32(seq), None, 0, self._n_ref, ctypes.byref(t)))
        return t.value

    def read_tokens(self, layer: int, seq: int, first: int = 0, n: int | None = None) -> tuple[np.ndarray, np.ndarray]:
        """Keys and values fp32 [n][n_kv_heads][head_dim] of tokens [first, first + n) (host)."""
        n = self.tokens(seq) - first if n is None else n
        for x in (layer, seq, first, n):
            _i32(x)
        k = np.empty((max(n, 0), self.n_kv_heads, self.head_dim), dtype=np.float32)
        v = np.empty_like(k)
        _check(lib().np_kv_read_tokens(self.h, layer, seq, first, n, k.ctypes.data, v.ctypes.data))
        return k, v

    def info(self) -> dict:
        out = (ctypes.c_int32 * 4)()
        _check(lib().np_kv_info(self.h, out))
        return dict(zip(["n_pages", "free", "shared", "current"], list(out)))


def decode_step(layers, cids: np.ndarray, x_ptr: int, y_ptr: int, compute_stream: int = 0,
                copy_stream: int | None = None) -> None:
    """np_decode_step over `layers` (list of Layer); cids int32 [n_layers][2] (host)."""
    cids = np.ascontiguousarray(cids, dtype=np.int32).reshape(len(layers), 2)
    handles = (ctypes.c_void_p * len(layers))(*[L.h.value for L in layers])
    cs = compute_stream or None
    ps = cs if copy_stream is None else (copy_stream or None)
    _check(lib().np_decode_step(handles, len(layers), cids.ctypes.data, x_ptr, y_ptr, cs, ps))


def decode_set_staging(nbytes: int, threads: int = 0) -> None:
    """Staged delta I/O for pinned host row stores (0 bytes: zero-copy pull, the default)."""
    _check(lib().np_decode_set_staging(nbytes, threads))


def decode_use_graphs(enable: bool) -> None:
    """np_decode_use_graphs: replay decode steps as captured HIP graphs, or launch one by one (default)."""
    _check(lib().np_decode_use_graphs(1 if enable else 0))


def probe_read(src_ptr: int, nbytes: int, sink_ptr: int, stream: int = 0) -> None:
    _check(lib().np_probe_read(src_ptr, nbytes, sink_ptr, stream or None))


def probe_read_set(src_ptrs, nbytes: int, passes: int, sink_ptr: int, stream: int = 0) -> None:
    arr = (ctypes.c_void_p * len(src_ptrs))(*src_ptrs)
    _check(lib().np_probe_read_set(arr, len(src_ptrs), nbytes, passes, sink_ptr, stream or None))


def probe_copy(dst_ptr: int, src_ptr: int, nbytes: int, stream: int = 0) -> None:
    _check(lib().np_probe_copy(dst_ptr, src_ptr, nbytes, stream or None))
