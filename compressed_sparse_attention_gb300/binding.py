"""Thin Python binding of the CSA2 C ABI (include/csa2.h).

Argument marshalling only: every function here checks that its tensors live
on the context's CUDA device with the expected dtype and contiguity, takes
their data pointers and the current CUDA stream, and calls the C entry point
of the same name. All arithmetic happens in the library's CUDA kernels. There
is no fallback: if the shared library is missing or a call fails, an error is
raised.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

from . import build as _build

_LIB = None

CSA2_OK = 0
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported geometry", 3: "CUDA error",
          4: "bad input recorded on the device", 5: "device wait timed out", 6: "workspace too small"}
KV_BF16, KV_FP8, KV_FP4, KV_MXFP4 = 0, 1, 2, 3
CAND_NONE, CAND_SOURCE, CAND_READ = 0, 1, 2  # csa2_kv_format
MODE_FULL, MODE_REINDEX, MODE_REUSE = 0, 1, 2

FLAG_BAD_TOPK_INDEX = 0x01
FLAG_BAD_WINDOW = 0x02
FLAG_BAD_SEGMENT = 0x04
FLAG_NVIS_TOO_LARGE = 0x08
FLAG_WAIT_TIMEOUT = 0x10
FLAG_BAD_QUERY = 0x20
FLAG_BAD_PAGE = 0x40
FLAG_OUT_OF_PAGES = 0x80
FLAG_BAD_SEQ = 0x100
FLAG_BATCH_FULL = 0x200

DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}  # csa2_dtype
ROPE_LAYOUTS = {"interleaved": 0, "half": 1}  # csa2_rope_layout
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}  # csa2_rope_scaling
ROPE_MAX_PAIRS = 256
PAGE_ARRAYS_MAX = 128


class Csa2Error(RuntimeError):
    def __init__(self, status, msg=""):
        super().__init__(f"{STATUS.get(status, status)}: {msg}")
        self.status = status


class HostIO(C.Structure):
    _fields_ = [("q", C.c_void_p), ("raw", C.c_void_p), ("gate", C.c_void_p), ("out", C.c_void_p)]


class Config(C.Structure):
    _fields_ = [("n_heads", C.c_int32), ("head_dim", C.c_int32), ("rope_dim", C.c_int32),
                ("window", C.c_int32), ("compress_ratio", C.c_int32), ("idx_heads", C.c_int32),
                ("idx_dim", C.c_int32), ("topk", C.c_int32), ("kv_format", C.c_int32),
                ("idx_key_format", C.c_int32), ("softmax_scale", C.c_float), ("norm_eps", C.c_float),
                ("rope_theta", C.c_double), ("yarn_factor", C.c_double), ("yarn_orig_len", C.c_double),
                ("yarn_beta_fast", C.c_double), ("yarn_beta_slow", C.c_double),
                ("cand_block", C.c_int32), ("cand_keep", C.c_int32)]


class StepArgs(C.Structure):
    _fields_ = [("mode", C.c_int32), ("n_seq", C.c_int32), ("n_query", C.c_int32), ("max_vis", C.c_int64),
                ("q", C.c_void_p), ("q_pos", C.c_void_p), ("seq_of_q", C.c_void_p), ("n_vis", C.c_void_p),
                ("q_idx", C.c_void_p), ("w_heads", C.c_void_p), ("sink", C.c_void_p),
                ("win_kv", C.c_void_p), ("win_scale", C.c_void_p), ("win_off", C.c_void_p),
                ("win_lo", C.c_void_p),
                ("pool_kv", C.c_void_p), ("pool_scale", C.c_void_p), ("idx_keys", C.c_void_p),
                ("idx_key_scale", C.c_void_p), ("pool_off", C.c_void_p),
                ("n_tokens", C.c_int64), ("raw", C.c_void_p), ("gate", C.c_void_p), ("tok_off", C.c_void_p),
                ("first_pos", C.c_void_p), ("norm_w", C.c_void_p), ("w_idx", C.c_void_p),
                ("k_norm_w", C.c_void_p),
                ("topk_idx", C.c_void_p), ("out", C.c_void_p), ("lse", C.c_void_p),
                ("workspace", C.c_void_p), ("workspace_bytes", C.c_size_t),
                ("append", C.c_int32), ("state_raw", C.c_void_p), ("state_gate", C.c_void_p),
                ("cand_role", C.c_int32), ("cand", C.c_void_p)]


class PagedKVArgs(C.Structure):
    _fields_ = [("pages", C.c_void_p), ("scales", C.c_void_p), ("page_stride", C.c_int64),
                ("scale_stride", C.c_int64), ("table", C.c_void_p), ("table_ld", C.c_int64), ("max_pages", C.c_int32),
                ("n_pages", C.c_int32), ("page_size", C.c_int32), ("n_seq", C.c_int32)]


class PagePoolArgs(C.Structure):
    _fields_ = [("table", C.c_void_p), ("table_ld", C.c_int64), ("seq_len", C.c_void_p), ("ref", C.c_void_p),
                ("max_pages", C.c_int32), ("n_pages", C.c_int32), ("page_size", C.c_int32), ("n_seq", C.c_int32)]


class PageArray(C.Structure):
    _fields_ = [("base", C.c_void_p), ("page_stride", C.c_int64), ("row_bytes", C.c_int32), ("reserved", C.c_int32)]


class BatchArgs(C.Structure):
    _fields_ = [("table", C.c_void_p), ("table_ld", C.c_int64), ("tok_off", C.c_void_p), ("first_pos", C.c_void_p),
                ("req_of_tok", C.c_void_p), ("tok_pos", C.c_void_p), ("tok_slot", C.c_void_p), ("max_tokens", C.c_int64)]


class RopeTable(C.Structure):
    _fields_ = [("rope_dim", C.c_int32), ("offset", C.c_int32), ("layout", C.c_int32), ("reserved", C.c_int32),
                ("amplitude", C.c_double), ("freq", C.c_double * ROPE_MAX_PAIRS)]


# name -> (restype, argtypes); every symbol include/csa2.h declares
SIGNATURES = {
    "csa2_default_config": (None, [C.POINTER(Config)]),
    "csa2_create": (C.c_int, [C.POINTER(Config), C.POINTER(C.c_void_p)]),
    "csa2_destroy": (None, [C.c_void_p]),
    "csa2_last_error": (C.c_char_p, [C.c_void_p]),
    "csa2_status_string": (C.c_char_p, [C.c_int]),
    "csa2_rope_frequencies": (C.c_int, [C.c_void_p, C.POINTER(C.c_double), C.c_int32]),
    "csa2_check": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(C.c_uint32)]),
    "csa2_debug_wait_timeout": (C.c_int, [C.c_void_p, C.c_void_p, C.c_uint64]),
    "csa2_store_rows": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.c_int32, C.c_void_p,
                                  C.c_int32, C.c_void_p, C.c_void_p]),
    "csa2_compress": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int32, C.c_int64,
                                C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "csa2_compress_append": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int32, C.c_int64,
                                       C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                       C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "csa2_index_score": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                                   C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64,
                                   C.c_void_p, C.c_int64]),
    "csa2_topk_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int32, C.c_int64]),
    "csa2_candidate_pool_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int32, C.c_int64]),
    "csa2_candidate_pool": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_int64, C.c_void_p,
                                      C.c_int64, C.c_void_p, C.c_void_p, C.c_size_t]),
    "csa2_index_score_pool": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                                        C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64,
                                        C.c_void_p, C.c_void_p, C.c_void_p]),
    "csa2_topk_pool": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p,
                                 C.c_int32, C.c_void_p, C.c_void_p, C.c_size_t]),
    "csa2_topk": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64,
                            C.c_int32, C.c_void_p, C.c_void_p, C.c_size_t]),
    "csa2_attend_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int32]),
    "csa2_attend": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                              C.c_void_p, C.c_size_t]),
    "csa2_step_host": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "csa2_step_graph_create": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "csa2_step_graph_launch": (C.c_int, [C.c_void_p, C.c_void_p]),
    "csa2_step_graph_destroy": (None, [C.c_void_p]),
    "csa2_step_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int32, C.c_int64]),
    "csa2_step": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(StepArgs)]),
    "csa2_last_launch_count": (C.c_int32, [C.c_void_p]),
    "csa2_shard_visible": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_int64, C.c_int64,
                                     C.c_void_p]),
    "csa2_topk_pairs": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_int64, C.c_void_p, C.c_int32,
                                  C.c_int64, C.c_void_p, C.c_void_p]),
    "csa2_topk_merge": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                                  C.c_int32, C.c_void_p]),
    "csa2_attend_partial": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                                      C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                      C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64,
                                      C.c_void_p, C.c_void_p, C.c_void_p]),
    "csa2_attend_combine": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                                      C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "csa2_attend_paged_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int32]),
    "csa2_attend_paged": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagedKVArgs), C.c_int32, C.c_void_p, C.c_void_p,
                                    C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p,
                                    C.c_void_p, C.c_size_t]),
    "csa2_append_paged": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagedKVArgs), C.c_int32, C.c_void_p, C.c_int64,
                                    C.c_void_p, C.c_void_p]),
    "csa2_append_slots": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagedKVArgs), C.c_int32, C.c_void_p, C.c_int64,
                                    C.c_void_p, C.c_void_p]),
    "csa2_batch_tables": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagePoolArgs), C.c_int32, C.c_void_p, C.c_void_p,
                                    C.POINTER(BatchArgs)]),
    "csa2_query_groups": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int64, C.c_int32, C.c_int32, C.c_int32,
                                    C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                    C.c_void_p, C.c_void_p]),
    "csa2_attend_shared_workspace_size": (C.c_size_t, [C.c_void_p, C.c_int32]),
    "csa2_attend_shared": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagedKVArgs), C.c_int32, C.c_void_p, C.c_void_p,
                                     C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                     C.c_void_p, C.c_size_t]),
    "csa2_pages_workspace_size": (C.c_size_t, [C.c_void_p, C.POINTER(PagePoolArgs)]),
    "csa2_pages_extend": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagePoolArgs), C.c_int32, C.c_void_p, C.c_void_p,
                                    C.c_void_p, C.c_size_t]),
    "csa2_pages_fork": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagePoolArgs), C.c_int32, C.c_void_p, C.c_void_p,
                                  C.c_int32, C.c_int32, C.POINTER(PageArray), C.c_void_p, C.c_size_t]),
    "csa2_pages_free": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagePoolArgs), C.c_int32, C.c_void_p]),
    "csa2_pages_trim": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagePoolArgs), C.c_int32, C.c_void_p, C.c_int64,
                                  C.c_int64, C.c_void_p]),
    "csa2_pages_compact": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(PagePoolArgs), C.c_int32, C.POINTER(PageArray),
                                     C.c_void_p, C.c_void_p, C.c_size_t]),
    "csa2_rope_table_init": (C.c_int, [C.POINTER(RopeTable), C.c_int32, C.c_int32, C.c_int32, C.c_double, C.c_int32,
                                       C.c_double, C.c_double, C.c_double, C.c_double, C.c_double]),
    "csa2_rope": (C.c_int, [C.c_void_p, C.c_void_p, C.POINTER(RopeTable), C.c_int32, C.c_int64, C.c_int32, C.c_int32,
                            C.c_void_p, C.c_int64, C.c_int64, C.c_void_p, C.c_void_p, C.c_int64, C.c_int64, C.c_int32]),
    "csa2_attend_noalloc": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                                      C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                      C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
}


def library_path() -> str:
    return _build.LIB_PATH


def load_library(path: str | None = None):
    """Load libcsa2.so (built by build.build()); raises if it is absent."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"CSA2 CUDA library not built: {path} is missing "
                           "(run compressed_sparse_attention_gb300.build.build())")
    lib = C.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


def default_config(**overrides) -> Config:
    lib = load_library()
    cfg = Config()
    lib.csa2_default_config(C.byref(cfg))
    for k, v in overrides.items():
        if k in ("kv_format", "idx_key_format") and isinstance(v, str):
            v = {"bf16": KV_BF16, "fp8": KV_FP8, "fp4": KV_FP4, "mxfp4": KV_MXFP4}[v]
        setattr(cfg, k, v)
    return cfg


def rope_table(rope_dim, theta=10000.0, layout="interleaved", offset=0, scaling="none", factor=1.0, orig_len=65536.0,
               beta_fast=32.0, beta_slow=1.0, amplitude=1.0) -> RopeTable:
    """The frequencies of csa2_rope (csa2_rope_table_init), made once and kept
    by the caller: `layout` "interleaved" or "half", `scaling` "none",
    "linear", "ntk" or "yarn", on the channels offset .. offset + rope_dim - 1."""
    tab = RopeTable()
    st = load_library().csa2_rope_table_init(C.byref(tab), rope_dim, offset, ROPE_LAYOUTS[layout], theta,
                                             ROPE_SCALINGS[scaling], factor, orig_len, beta_fast, beta_slow, amplitude)
    if st != CSA2_OK:
        raise Csa2Error(st, "csa2_rope_table_init")
    return tab


def _stream() -> int:
    """Handle of the current device's current stream. Asked for by number: a
    torch.cuda.Stream object made for each call costs 2.9 us of host time, more
    than the rest of a call with one launch's arguments."""
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


class Context:
    """Owns one csa2_ctx bound to the current CUDA device."""

    def __init__(self, cfg: Config | None = None, **overrides):
        self.lib = load_library()
        self.cfg = cfg if cfg is not None else default_config(**overrides)
        self.device = torch.device("cuda", torch.cuda.current_device())
        h = C.c_void_p()
        st = self.lib.csa2_create(C.byref(self.cfg), C.byref(h))
        if st != CSA2_OK:
            raise Csa2Error(st, "csa2_create")
        self.h = h

    def close(self):
        if getattr(self, "h", None):
            self.lib.csa2_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- marshalling helpers
    def _p(self, t, dtype=None, name="tensor"):
        if t is None:
            return None
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, is on {t.device}")
        if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
            raise TypeError(f"{name} must be {dtype}, is {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def _ok(self, st, what):
        if st != CSA2_OK:
            raise Csa2Error(st, f"{what}: {self.lib.csa2_last_error(self.h).decode()}")

    @property
    def last_launch_count(self) -> int:
        return int(self.lib.csa2_last_launch_count(self.h))

    def rope_frequencies(self):
        n = max(1, self.cfg.rope_dim // 2)
        buf = (C.c_double * n)()
        self._ok(self.lib.csa2_rope_frequencies(self.h, buf, n), "csa2_rope_frequencies")
        return [buf[i] for i in range(self.cfg.rope_dim // 2)]

    def check(self):
        """Synchronise the current stream; return the device error word (raises on error)."""
        fl = C.c_uint32(0)
        st = self.lib.csa2_check(self.h, C.c_void_p(_stream()), C.byref(fl))
        if st not in (CSA2_OK, 4, 5):
            self._ok(st, "csa2_check")
        return int(fl.value), st

    def debug_wait_timeout(self, limit_ns: int):
        """Enqueue the wait probe (csa2_debug_wait_timeout) on the current stream."""
        self._ok(self.lib.csa2_debug_wait_timeout(self.h, C.c_void_p(_stream()), int(limit_ns)),
                 "csa2_debug_wait_timeout")

    # -- entry points
    def store_rows(self, rows, pos, fmt, out, out_scale=None):
        n, dim = rows.shape
        self._ok(self.lib.csa2_store_rows(self.h, C.c_void_p(_stream()), self._p(rows, torch.float32, "rows"),
                                          n, dim, self._p(pos, torch.int64, "pos"), fmt,
                                          self._p(out, None, "out"), self._p(out_scale, torch.uint8, "out_scale")),
                 "csa2_store_rows")

    def compress(self, raw, gate, n_seq, tok_off, first_pos, pool_off, norm_w, w_idx, k_norm_w,
                 pool_kv, pool_kv_scale, idx_keys, idx_key_scale):
        n_tokens = raw.shape[0]
        self._ok(self.lib.csa2_compress(
            self.h, C.c_void_p(_stream()), self._p(raw, torch.bfloat16, "raw"), self._p(gate, torch.float32, "gate"),
            n_seq, n_tokens, self._p(tok_off, torch.int64, "tok_off"), self._p(first_pos, torch.int64, "first_pos"),
            self._p(pool_off, torch.int64, "pool_off"), self._p(norm_w, torch.float32, "norm_w"),
            self._p(w_idx, torch.bfloat16, "w_idx"), self._p(k_norm_w, torch.float32, "k_norm_w"),
            self._p(pool_kv, None, "pool_kv"), self._p(pool_kv_scale, torch.uint8, "pool_kv_scale"),
            self._p(idx_keys, None, "idx_keys"), self._p(idx_key_scale, torch.uint8, "idx_key_scale")),
            "csa2_compress")

    def compress_append(self, raw, gate, n_seq, tok_off, first_pos, pool_off, norm_w, w_idx, k_norm_w,
                        pool_kv, pool_kv_scale, idx_keys, idx_key_scale, state_raw, state_gate):
        n_tokens = 0 if raw is None else raw.shape[0]
        self._ok(self.lib.csa2_compress_append(
            self.h, C.c_void_p(_stream()), self._p(raw, torch.bfloat16, "raw"), self._p(gate, torch.float32, "gate"),
            n_seq, n_tokens, self._p(tok_off, torch.int64, "tok_off"), self._p(first_pos, torch.int64, "first_pos"),
            self._p(pool_off, torch.int64, "pool_off"), self._p(norm_w, torch.float32, "norm_w"),
            self._p(w_idx, torch.bfloat16, "w_idx"), self._p(k_norm_w, torch.float32, "k_norm_w"),
            self._p(pool_kv, None, "pool_kv"), self._p(pool_kv_scale, torch.uint8, "pool_kv_scale"),
            self._p(idx_keys, None, "idx_keys"), self._p(idx_key_scale, torch.uint8, "idx_key_scale"),
            self._p(state_raw, torch.bfloat16, "state_raw"), self._p(state_gate, torch.float32, "state_gate")),
            "csa2_compress_append")

    def index_score(self, n_seq, q_idx, w_heads, idx_keys, idx_key_scale, pool_off, seq_of_q, n_vis, max_vis,
                    scores):
        self._ok(self.lib.csa2_index_score(
            self.h, C.c_void_p(_stream()), n_seq, q_idx.shape[0], self._p(q_idx, torch.bfloat16, "q_idx"),
            self._p(w_heads, torch.float32, "w_heads"), self._p(idx_keys, None, "idx_keys"),
            self._p(idx_key_scale, torch.uint8, "idx_key_scale"), self._p(pool_off, torch.int64, "pool_off"),
            self._p(seq_of_q, torch.int32, "seq_of_q"), self._p(n_vis, torch.int32, "n_vis"), max_vis,
            self._p(scores, torch.float32, "scores"), scores.shape[1]), "csa2_index_score")

    # -- the hierarchical indexer's pool
    def candidate_pool_workspace_size(self, n_query, max_vis) -> int:
        return int(self.lib.csa2_candidate_pool_workspace_size(self.h, n_query, max_vis))

    def candidate_pool(self, scores, n_vis, max_vis, cand, workspace):
        self._ok(self.lib.csa2_candidate_pool(
            self.h, C.c_void_p(_stream()), n_vis.shape[0], self._p(scores, torch.float32, "scores"), scores.shape[1],
            self._p(n_vis, torch.int32, "n_vis"), max_vis, self._p(cand, torch.int32, "cand"),
            self._p(workspace, None, "workspace"),
            0 if workspace is None else workspace.numel() * workspace.element_size()), "csa2_candidate_pool")

    def index_score_pool(self, n_seq, q_idx, w_heads, idx_keys, idx_key_scale, pool_off, seq_of_q, n_vis, max_vis,
                         cand, scores_pool, n_pool):
        self._ok(self.lib.csa2_index_score_pool(
            self.h, C.c_void_p(_stream()), n_seq, q_idx.shape[0], self._p(q_idx, torch.bfloat16, "q_idx"),
            self._p(w_heads, torch.float32, "w_heads"), self._p(idx_keys, None, "idx_keys"),
            self._p(idx_key_scale, torch.uint8, "idx_key_scale"), self._p(pool_off, torch.int64, "pool_off"),
            self._p(seq_of_q, torch.int32, "seq_of_q"), self._p(n_vis, torch.int32, "n_vis"), max_vis,
            self._p(cand, torch.int32, "cand"), self._p(scores_pool, torch.float32, "scores_pool"),
            self._p(n_pool, torch.int32, "n_pool")), "csa2_index_score_pool")

    def topk_pool(self, scores_pool, n_pool, cand, k, out_idx, workspace):
        self._ok(self.lib.csa2_topk_pool(
            self.h, C.c_void_p(_stream()), n_pool.shape[0], self._p(scores_pool, torch.float32, "scores_pool"),
            self._p(n_pool, torch.int32, "n_pool"), self._p(cand, torch.int32, "cand"), k,
            self._p(out_idx, torch.int32, "out_idx"), self._p(workspace, None, "workspace"),
            0 if workspace is None else workspace.numel() * workspace.element_size()), "csa2_topk_pool")

    def topk_workspace_size(self, n_query, max_vis) -> int:
        return int(self.lib.csa2_topk_workspace_size(self.h, n_query, max_vis))

    def topk(self, scores, n_vis, max_vis, k, out_idx, workspace):
        self._ok(self.lib.csa2_topk(
            self.h, C.c_void_p(_stream()), scores.shape[0], self._p(scores, torch.float32, "scores"),
            scores.shape[1], self._p(n_vis, torch.int32, "n_vis"), max_vis, k,
            self._p(out_idx, torch.int32, "out_idx"), self._p(workspace, None, "workspace"),
            0 if workspace is None else workspace.numel() * workspace.element_size()), "csa2_topk")

    def attend_workspace_size(self, n_query) -> int:
        return int(self.lib.csa2_attend_workspace_size(self.h, n_query))

    def attend(self, n_seq, q, q_pos, seq_of_q, win_kv, win_scale, win_off, win_lo, pool_kv, pool_scale, pool_off,
               topk_idx, sink, out, lse, workspace):
        self._ok(self.lib.csa2_attend(
            self.h, C.c_void_p(_stream()), n_seq, q.shape[0], self._p(q, torch.bfloat16, "q"),
            self._p(q_pos, torch.int64, "q_pos"), self._p(seq_of_q, torch.int32, "seq_of_q"),
            self._p(win_kv, None, "win_kv"), self._p(win_scale, torch.uint8, "win_scale"),
            self._p(win_off, torch.int64, "win_off"), self._p(win_lo, torch.int64, "win_lo"),
            self._p(pool_kv, None, "pool_kv"), self._p(pool_scale, torch.uint8, "pool_scale"),
            self._p(pool_off, torch.int64, "pool_off"), self._p(topk_idx, torch.int32, "topk_idx"),
            self._p(sink, torch.float32, "sink"), self._p(out, torch.bfloat16, "out"),
            self._p(lse, torch.float32, "lse"), self._p(workspace, None, "workspace"),
            0 if workspace is None else workspace.numel() * workspace.element_size()), "csa2_attend")

    # -- pool sharding (csa2_shard_visible .. csa2_attend_combine)
    def shard_visible(self, n_vis, lo, hi, out):
        self._ok(self.lib.csa2_shard_visible(self.h, C.c_void_p(_stream()), n_vis.shape[0],
                                             self._p(n_vis, torch.int32, "n_vis"), int(lo), int(hi),
                                             self._p(out, torch.int32, "n_vis_shard")), "csa2_shard_visible")

    def topk_pairs(self, scores, sel, index_base, pair_score, pair_idx):
        self._ok(self.lib.csa2_topk_pairs(self.h, C.c_void_p(_stream()), sel.shape[0],
                                          self._p(scores, torch.float32, "scores"), scores.shape[1],
                                          self._p(sel, torch.int32, "sel"), sel.shape[1], int(index_base),
                                          self._p(pair_score, torch.float32, "pair_score"),
                                          self._p(pair_idx, torch.int32, "pair_idx")), "csa2_topk_pairs")

    def topk_merge(self, pair_score, pair_idx, k, out_idx):
        """pair_score / pair_idx [n_lists, n_query, list_len] -> out_idx [n_query, k]."""
        n_lists, n_query, list_len = pair_idx.shape
        self._ok(self.lib.csa2_topk_merge(self.h, C.c_void_p(_stream()), n_query, n_lists, list_len,
                                          self._p(pair_score, torch.float32, "pair_score"),
                                          self._p(pair_idx, torch.int32, "pair_idx"), k,
                                          self._p(out_idx, torch.int32, "out_idx")), "csa2_topk_merge")

    def attend_partial(self, n_seq, q, q_pos, seq_of_q, with_window, win_kv, win_scale, win_off, win_lo, pool_kv,
                       pool_scale, pool_off, topk_idx, shard_lo, shard_hi, part_o, part_m, part_l):
        self._ok(self.lib.csa2_attend_partial(
            self.h, C.c_void_p(_stream()), n_seq, q.shape[0], self._p(q, torch.bfloat16, "q"),
            self._p(q_pos, torch.int64, "q_pos"), self._p(seq_of_q, torch.int32, "seq_of_q"), 1 if with_window else 0,
            self._p(win_kv, None, "win_kv"), self._p(win_scale, torch.uint8, "win_scale"),
            self._p(win_off, torch.int64, "win_off"), self._p(win_lo, torch.int64, "win_lo"),
            self._p(pool_kv, None, "pool_kv"), self._p(pool_scale, torch.uint8, "pool_scale"),
            self._p(pool_off, torch.int64, "pool_off"), self._p(topk_idx, torch.int32, "topk_idx"),
            int(shard_lo), int(shard_hi), self._p(part_o, torch.float32, "part_o"),
            self._p(part_m, torch.float32, "part_m"), self._p(part_l, torch.float32, "part_l")),
            "csa2_attend_partial")

    def attend_combine(self, part_o, part_m, part_l, q_pos, sink, out, lse=None):
        """part_o [n_parts, n_query, 64, 512], part_m / part_l [n_parts, n_query, 64]."""
        n_parts, n_query = part_m.shape[0], part_m.shape[1]
        self._ok(self.lib.csa2_attend_combine(
            self.h, C.c_void_p(_stream()), n_query, n_parts, self._p(part_o, torch.float32, "part_o"),
            self._p(part_m, torch.float32, "part_m"), self._p(part_l, torch.float32, "part_l"),
            self._p(q_pos, torch.int64, "q_pos"), self._p(sink, torch.float32, "sink"),
            self._p(out, torch.bfloat16, "out"), self._p(lse, torch.float32, "lse")), "csa2_attend_combine")

    # -- paged caches (csa2_attend_paged .. csa2_pages_compact) and csa2_rope
    #
    # Each has a prepare_ form that checks the tensors and builds the argument
    # block once, for a serving loop that reuses its buffers: every
    # PreparedCall.run() is then a single C call on the current stream. Tensors
    # are the caller's; a PreparedCall keeps them alive.

    def _strided(self, t, dtype, name):
        """Pointer and row stride (elements) of a 2-D tensor whose rows are contiguous."""
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
            raise ValueError(f"{name} must be 2-D with contiguous rows")
        if t.device != self.device or t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype} on {self.device}, is {t.dtype} on {t.device}")
        return t.data_ptr(), (t.stride(0) if t.shape[0] > 1 else t.shape[1])

    def _page_array(self, t, name):
        """(pointer, page stride in bytes, row bytes) of [n_pages, page_size, ...] pages, contiguous inside a page."""
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, is on {t.device}")
        if t.dim() < 2 or not t[:1].is_contiguous():
            raise ValueError(f"{name} must be [n_pages, page_size, ...], contiguous inside a page")
        size = t.element_size()
        inner = t.shape[1:].numel()
        stride = t.stride(0) if t.shape[0] > 1 else inner
        if stride < inner:
            raise ValueError(f"{name}: pages overlap")
        return t.data_ptr(), stride * size, inner // max(1, t.shape[1]) * size

    def paged_kv(self, pages, table=None, scales=None) -> "PagedKV":
        """A cache in pages: `pages` [n_pages, page_size, 512] bf16, or uint8
        codes [.., 512] (fp8) / [.., 256] (fp4) with uint8 `scales` [n_pages,
        page_size, 16 / 32] (the page axis may be strided: pages of several
        layers side by side); `table` int32 [n_seq, max_pages], the page of
        each run of page_size positions, -1 for none (None: a cache for
        append_slots, which reads no table)."""
        fmt = self.cfg.kv_format
        dtype, width, sw = {KV_BF16: (torch.bfloat16, 512, 0), KV_FP8: (torch.uint8, 512, 16),
                            KV_FP4: (torch.uint8, 256, 32)}[fmt]
        if pages.dim() != 3 or pages.shape[2] != width or pages.dtype != dtype:
            raise ValueError(f"pages must be {dtype} [n_pages, page_size, {width}] in this context's format")
        a = PagedKVArgs()
        a.pages, a.page_stride, _ = self._page_array(pages, "pages")
        if sw:
            if scales is None or scales.dtype != torch.uint8 or tuple(scales.shape) != (*pages.shape[:2], sw):
                raise ValueError(f"scales must be uint8 [n_pages, page_size, {sw}]")
            a.scales, a.scale_stride, _ = self._page_array(scales, "scales")
        if table is not None:
            a.table, a.table_ld = self._strided(table, torch.int32, "table")
            a.n_seq, a.max_pages = table.shape
        a.n_pages, a.page_size = pages.shape[:2]
        return PagedKV(a, (pages, scales, table), fmt, self.device)

    def _kv(self, kv: "PagedKV"):
        """The block of a cache whose rows this context reads: of its format and on its device."""
        if kv.fmt != self.cfg.kv_format or kv.device != self.device:
            raise ValueError(f"kv is of format {kv.fmt} on {kv.device}, the context of format {self.cfg.kv_format} on {self.device}")
        return C.byref(kv.args)

    def _pool(self, pool: "PagePool"):
        if pool.device != self.device:
            raise ValueError(f"pool is on {pool.device}, the context on {self.device}")
        return C.byref(pool.args)

    def attend_paged_workspace_size(self, n_query) -> int:
        return int(self.lib.csa2_attend_paged_workspace_size(self.h, n_query))

    def prepare_attend_paged(self, kv: "PagedKV", q, q_pos, seq_of_q, out, workspace, *, sink=None, lse=None, lo=None,
                             window=0, n_first=0) -> "PreparedCall":
        n = q.shape[0]
        self._shape(q, (n, 64, 512), "q")
        self._shape(out, (n, 64, 512), "out")
        self._shape(q_pos, (n,), "q_pos")
        self._shape(seq_of_q, (n,), "seq_of_q")
        self._shape(sink, (64,), "sink")
        self._shape(lse, (n, 64), "lse")
        self._shape(lo, (kv.args.n_seq,), "lo")
        return PreparedCall(self, "csa2_attend_paged", (
            self._kv(kv), n, self._p(q, torch.bfloat16, "q"), self._p(q_pos, torch.int64, "q_pos"),
            self._p(seq_of_q, torch.int32, "seq_of_q"), self._p(lo, torch.int64, "lo"), int(window), int(n_first),
            self._p(sink, torch.float32, "sink"), self._p(out, torch.bfloat16, "out"),
            self._p(lse, torch.float32, "lse"), self._p(workspace, None, "workspace"),
            0 if workspace is None else workspace.numel() * workspace.element_size()),
            (kv, q, q_pos, seq_of_q, out, workspace, sink, lse, lo))

    def attend_paged(self, kv, q, q_pos, seq_of_q, out, workspace, **kw):
        """csa2_attend_paged: every visible row of a paged cache (`window` 0), or
        the last `window` rows and the first `n_first`."""
        self.prepare_attend_paged(kv, q, q_pos, seq_of_q, out, workspace, **kw).run()

    def prepare_append_paged(self, kv: "PagedKV", rows, tok_off, first_pos) -> "PreparedCall":
        self._shape(rows, (rows.shape[0], 512), "rows")
        self._shape(tok_off, (kv.args.n_seq + 1,), "tok_off")
        self._shape(first_pos, (kv.args.n_seq,), "first_pos")
        return PreparedCall(self, "csa2_append_paged", (
            self._kv(kv), DTYPE_CODES.get(rows.dtype, -1), self._p(rows, (torch.bfloat16, torch.float32), "rows"),
            rows.shape[0], self._p(tok_off, torch.int64, "tok_off"), self._p(first_pos, torch.int64, "first_pos")),
            (kv, rows, tok_off, first_pos))

    def append_paged(self, kv, rows, tok_off, first_pos):
        """csa2_append_paged: rows [n, 512] rotated at their positions and stored in their pages."""
        self.prepare_append_paged(kv, rows, tok_off, first_pos).run()

    def prepare_append_slots(self, kv: "PagedKV", rows, pos, slots) -> "PreparedCall":
        n = rows.shape[0]
        self._shape(rows, (n, 512), "rows")
        self._shape(pos, (n,), "pos")
        self._shape(slots, (n,), "slots")
        return PreparedCall(self, "csa2_append_slots", (
            self._kv(kv), DTYPE_CODES.get(rows.dtype, -1), self._p(rows, (torch.bfloat16, torch.float32), "rows"), n,
            self._p(pos, torch.int64, "pos"), self._p(slots, torch.int64, "slots")), (kv, rows, pos, slots))

    def append_slots(self, kv, rows, pos, slots):
        """csa2_append_slots: rows [n, 512] rotated at pos (None: as they are) and stored at their slots (-1: not)."""
        self.prepare_append_slots(kv, rows, pos, slots).run()

    def prepare_batch_tables(self, pool: "PagePool", seqs, n_new, table, tok_off, first_pos, req_of_tok, tok_pos,
                             tok_slot) -> "PreparedCall":
        n = seqs.numel()
        self._shape(seqs, (n,), "seqs")
        self._shape(n_new, (n,), "n_new")
        self._shape(table, (n, pool.args.max_pages), "table")
        self._shape(tok_off, (n + 1,), "tok_off")
        self._shape(first_pos, (n,), "first_pos")
        tokens = req_of_tok.numel()
        for t, name in ((req_of_tok, "req_of_tok"), (tok_pos, "tok_pos"), (tok_slot, "tok_slot")):
            self._shape(t, (tokens,), name)
        a = BatchArgs()
        a.table, a.table_ld = self._strided(table, torch.int32, "table")
        a.tok_off, a.first_pos = self._p(tok_off, torch.int64, "tok_off"), self._p(first_pos, torch.int64, "first_pos")
        a.req_of_tok = self._p(req_of_tok, torch.int32, "req_of_tok")
        a.tok_pos, a.tok_slot = self._p(tok_pos, torch.int64, "tok_pos"), self._p(tok_slot, torch.int64, "tok_slot")
        a.max_tokens = tokens
        return PreparedCall(self, "csa2_batch_tables", (
            self._pool(pool), n, self._p(seqs, torch.int32, "seqs"), self._p(n_new, torch.int64, "n_new"), C.byref(a)),
            (pool, seqs, n_new, a, table, tok_off, first_pos, req_of_tok, tok_pos, tok_slot))

    def batch_tables(self, pool, seqs, n_new, table, tok_off, first_pos, req_of_tok, tok_pos, tok_slot):
        """csa2_batch_tables: of the requests `seqs` of the pool with n_new new
        tokens each, the page table [n, max_pages], the offsets and first
        positions of the new tokens, and each token's request, position and slot
        (their length is the batch's capacity; -1 behind the last token)."""
        self.prepare_batch_tables(pool, seqs, n_new, table, tok_off, first_pos, req_of_tok, tok_pos, tok_slot).run()

    def prepare_query_groups(self, table, page_size, n_pages, q_pos, seq_of_q, min_shared, order, head, shared,
                             n_groups=None) -> "PreparedCall":
        n = q_pos.numel()
        for t, name in ((q_pos, "q_pos"), (seq_of_q, "seq_of_q"), (order, "order"), (head, "head"), (shared, "shared")):
            self._shape(t, (n,), name)
        self._shape(n_groups, (1,), "n_groups")
        ptr, ld = self._strided(table, torch.int32, "table")
        return PreparedCall(self, "csa2_query_groups", (
            ptr, ld, table.shape[1], n_pages, page_size, table.shape[0], n, self._p(q_pos, torch.int64, "q_pos"),
            self._p(seq_of_q, torch.int32, "seq_of_q"), int(min_shared), self._p(order, torch.int32, "order"),
            self._p(head, torch.int32, "head"), self._p(shared, torch.int64, "shared"),
            self._p(n_groups, torch.int32, "n_groups")),
            (table, q_pos, seq_of_q, order, head, shared, n_groups))

    def query_groups(self, table, page_size, n_pages, q_pos, seq_of_q, min_shared, order, head, shared, n_groups=None):
        """csa2_query_groups: queries whose sequences share at least min_shared
        leading positions (whole pages) placed group by group, as attend_shared
        takes them: order, head and shared [n]."""
        self.prepare_query_groups(table, page_size, n_pages, q_pos, seq_of_q, min_shared, order, head, shared,
                                  n_groups).run()

    def attend_shared_workspace_size(self, n_query) -> int:
        return int(self.lib.csa2_attend_shared_workspace_size(self.h, n_query))

    def prepare_attend_shared(self, kv: "PagedKV", q, q_pos, seq_of_q, order, head, shared, out, workspace, *, sink=None,
                              lse=None) -> "PreparedCall":
        n = q.shape[0]
        self._shape(q, (n, 64, 512), "q")
        self._shape(out, (n, 64, 512), "out")
        for t, name in ((q_pos, "q_pos"), (seq_of_q, "seq_of_q"), (order, "order"), (head, "head"), (shared, "shared")):
            self._shape(t, (n,), name)
        self._shape(sink, (64,), "sink")
        self._shape(lse, (n, 64), "lse")
        return PreparedCall(self, "csa2_attend_shared", (
            self._kv(kv), n, self._p(q, torch.bfloat16, "q"), self._p(q_pos, torch.int64, "q_pos"),
            self._p(seq_of_q, torch.int32, "seq_of_q"), self._p(order, torch.int32, "order"),
            self._p(head, torch.int32, "head"), self._p(shared, torch.int64, "shared"),
            self._p(sink, torch.float32, "sink"), self._p(out, torch.bfloat16, "out"), self._p(lse, torch.float32, "lse"),
            *self._ws(workspace)), (kv, q, q_pos, seq_of_q, order, head, shared, sink, out, lse, workspace))

    def attend_shared(self, kv, q, q_pos, seq_of_q, order, head, shared, out, workspace, *, sink=None, lse=None):
        """csa2_attend_shared: q [n, 64, 512] over every row up to q_pos; query
        order[k] at place k, groups of places from head[k] on, the rows below
        shared[head[k]] read (and multiplied) once for two queries."""
        self.prepare_attend_shared(kv, q, q_pos, seq_of_q, order, head, shared, out, workspace, sink=sink, lse=lse).run()

    def page_pool(self, table, seq_len, ref, page_size) -> "PagePool":
        """The state of the page operations: `table` int32 [n_seq, max_pages],
        `seq_len` int64 [n_seq], `ref` int32 [n_pages] (table entries naming
        each page)."""
        a = PagePoolArgs()
        a.table, a.table_ld = self._strided(table, torch.int32, "table")
        a.n_seq, a.max_pages = table.shape
        self._shape(seq_len, (a.n_seq,), "seq_len")
        a.seq_len = self._p(seq_len, torch.int64, "seq_len")
        a.ref = self._p(ref, torch.int32, "ref")
        a.n_pages, a.page_size = ref.numel(), page_size
        return PagePool(a, (table, seq_len, ref), self.device)

    def pages_workspace_size(self, pool: "PagePool") -> int:
        return int(self.lib.csa2_pages_workspace_size(self.h, C.byref(pool.args)))

    def _page_arrays(self, pool, arrays):
        c = (PageArray * max(1, len(arrays)))()
        for i, t in enumerate(arrays):
            if t.dim() < 2 or t.shape[0] != pool.args.n_pages or t.shape[1] != pool.args.page_size:
                raise ValueError(f"arrays[{i}] must be [{pool.args.n_pages}, {pool.args.page_size}, ...]")
            c[i].base, c[i].page_stride, c[i].row_bytes = self._page_array(t, f"arrays[{i}]")
        return c

    def _ws(self, workspace):
        return self._p(workspace, None, "workspace"), (0 if workspace is None else
                                                       workspace.numel() * workspace.element_size())

    def prepare_pages_extend(self, pool, seqs, new_len, workspace) -> "PreparedCall":
        self._shape(seqs, (seqs.numel(),), "seqs")
        self._shape(new_len, (seqs.shape[0],), "new_len")
        return PreparedCall(self, "csa2_pages_extend", (
            self._pool(pool), seqs.shape[0], self._p(seqs, torch.int32, "seqs"),
            self._p(new_len, torch.int64, "new_len"), *self._ws(workspace)), (pool, seqs, new_len, workspace))

    def pages_extend(self, pool, seqs, new_len, workspace):
        """csa2_pages_extend: sequences grow to new_len tokens, fresh pages where they lack them."""
        self.prepare_pages_extend(pool, seqs, new_len, workspace).run()

    def prepare_pages_fork(self, pool, parents, children, arrays, workspace, deep=False) -> "PreparedCall":
        self._shape(parents, (parents.numel(),), "parents")
        self._shape(children, (parents.shape[0],), "children")
        c = self._page_arrays(pool, arrays)
        return PreparedCall(self, "csa2_pages_fork", (
            self._pool(pool), parents.shape[0], self._p(parents, torch.int32, "parents"),
            self._p(children, torch.int32, "children"), 1 if deep else 0, len(arrays), c, *self._ws(workspace)),
            (pool, parents, children, tuple(arrays), c, workspace))

    def pages_fork(self, pool, parents, children, arrays, workspace, deep=False):
        """csa2_pages_fork: children become copies of parents, sharing their full pages (`deep`: none)."""
        self.prepare_pages_fork(pool, parents, children, arrays, workspace, deep).run()

    def prepare_pages_free(self, pool, seqs) -> "PreparedCall":
        self._shape(seqs, (seqs.numel(),), "seqs")
        return PreparedCall(self, "csa2_pages_free", (self._pool(pool), seqs.shape[0],
                                                      self._p(seqs, torch.int32, "seqs")), (pool, seqs))

    def pages_free(self, pool, seqs):
        """csa2_pages_free: every page of the sequences given back."""
        self.prepare_pages_free(pool, seqs).run()

    def prepare_pages_trim(self, pool, seqs, window, n_first=0, lo=None) -> "PreparedCall":
        self._shape(seqs, (seqs.numel(),), "seqs")
        self._shape(lo, (pool.args.n_seq,), "lo")
        return PreparedCall(self, "csa2_pages_trim", (
            self._pool(pool), seqs.shape[0], self._p(seqs, torch.int32, "seqs"), int(window), int(n_first),
            self._p(lo, torch.int64, "lo")), (pool, seqs, lo))

    def pages_trim(self, pool, seqs, window, n_first=0, lo=None):
        """csa2_pages_trim: the pages no later query sees under the window given back."""
        self.prepare_pages_trim(pool, seqs, window, n_first, lo).run()

    def prepare_pages_compact(self, pool, arrays, n_live, workspace) -> "PreparedCall":
        c = self._page_arrays(pool, arrays)
        self._shape(n_live, (1,), "n_live")
        return PreparedCall(self, "csa2_pages_compact", (
            self._pool(pool), len(arrays), c, self._p(n_live, torch.int32, "n_live"), *self._ws(workspace)),
            (pool, tuple(arrays), c, n_live, workspace))

    def pages_compact(self, pool, arrays, n_live, workspace):
        """csa2_pages_compact: the pages in use moved to the lowest indices; n_live (nullable) receives their number."""
        self.prepare_pages_compact(pool, arrays, n_live, workspace).run()

    def prepare_rope(self, table: RopeTable, x, pos, out=None, transpose=False) -> "PreparedCall":
        out = x if out is None else out
        for t, name in ((x, "x"), (out, "out")):
            if t.dim() != 3 or (t.shape[2] > 1 and t.stride(2) != 1):
                raise ValueError(f"{name} must be [n_tokens, n_heads, head_dim] with contiguous channels")
            if t.device != self.device or t.dtype != x.dtype or t.shape != x.shape:
                raise ValueError(f"{name} must be {tuple(x.shape)} {x.dtype} on {self.device}")
        if x.dtype not in DTYPE_CODES:
            raise TypeError(f"x must be bf16, fp16 or fp32, is {x.dtype}")
        self._shape(pos, (x.shape[0],), "pos")
        return PreparedCall(self, "csa2_rope", (
            C.byref(table), DTYPE_CODES[x.dtype], *x.shape, x.data_ptr(), x.stride(0), x.stride(1),
            self._p(pos, torch.int64, "pos"), out.data_ptr(), out.stride(0), out.stride(1), 1 if transpose else 0),
            (table, x, pos, out))

    def rope(self, table, x, pos, out=None, transpose=False):
        """csa2_rope: x [n_tokens, n_heads, head_dim] rotated at pos into out (in
        place without one); `transpose` rotates back (the gradient's direction)."""
        self.prepare_rope(table, x, pos, out, transpose).run()

    @staticmethod
    def _shape(t, shape, name):
        if t is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {tuple(shape)}, is {tuple(t.shape)}")

    def step_workspace_size(self, n_query, max_vis) -> int:
        return int(self.lib.csa2_step_workspace_size(self.h, n_query, max_vis))

    def step(self, mode, n_seq, max_vis, **kw):
        self._ok(self.lib.csa2_step(self.h, C.c_void_p(_stream()), C.byref(self.step_args(mode, n_seq, max_vis, **kw))),
                 "csa2_step")

    def prepare_step(self, mode, n_seq, max_vis, **kw) -> "PreparedStep":
        """The step's argument block built once, for a serving loop that reuses
        its buffers from step to step: each run is then a single C call."""
        return PreparedStep(self, self.step_args(mode, n_seq, max_vis, **kw), kw)

    def step_args(self, mode, n_seq, max_vis, *, q, q_pos, seq_of_q, n_vis, sink, win_kv, win_off, pool_kv,
                  pool_off, topk_idx, out, workspace, q_idx=None, w_heads=None, win_scale=None, win_lo=None,
                  pool_scale=None, idx_keys=None, idx_key_scale=None, raw=None, gate=None, tok_off=None,
                  first_pos=None, norm_w=None, w_idx=None, k_norm_w=None, lse=None, append=False, state_raw=None,
                  state_gate=None, cand_role=0, cand=None) -> StepArgs:
        a = StepArgs()
        a.mode, a.n_seq, a.n_query, a.max_vis = mode, n_seq, q.shape[0], max_vis
        a.q = self._p(q, torch.bfloat16, "q")
        a.q_pos = self._p(q_pos, torch.int64, "q_pos")
        a.seq_of_q = self._p(seq_of_q, torch.int32, "seq_of_q")
        a.n_vis = self._p(n_vis, torch.int32, "n_vis")
        a.q_idx = self._p(q_idx, torch.bfloat16, "q_idx")
        a.w_heads = self._p(w_heads, torch.float32, "w_heads")
        a.sink = self._p(sink, torch.float32, "sink")
        a.win_kv = self._p(win_kv, None, "win_kv")
        a.win_scale = self._p(win_scale, torch.uint8, "win_scale")
        a.win_off = self._p(win_off, torch.int64, "win_off")
        a.win_lo = self._p(win_lo, torch.int64, "win_lo")
        a.pool_kv = self._p(pool_kv, None, "pool_kv")
        a.pool_scale = self._p(pool_scale, torch.uint8, "pool_scale")
        a.idx_keys = self._p(idx_keys, None, "idx_keys")
        a.idx_key_scale = self._p(idx_key_scale, torch.uint8, "idx_key_scale")
        a.pool_off = self._p(pool_off, torch.int64, "pool_off")
        a.n_tokens = 0 if raw is None else raw.shape[0]
        a.raw = self._p(raw, torch.bfloat16, "raw")
        a.gate = self._p(gate, torch.float32, "gate")
        a.tok_off = self._p(tok_off, torch.int64, "tok_off")
        a.first_pos = self._p(first_pos, torch.int64, "first_pos")
        a.norm_w = self._p(norm_w, torch.float32, "norm_w")
        a.w_idx = self._p(w_idx, torch.bfloat16, "w_idx")
        a.k_norm_w = self._p(k_norm_w, torch.float32, "k_norm_w")
        a.topk_idx = self._p(topk_idx, torch.int32, "topk_idx")
        a.out = self._p(out, torch.bfloat16, "out")
        a.lse = self._p(lse, torch.float32, "lse")
        a.workspace = self._p(workspace, None, "workspace")
        a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        a.append = 1 if append else 0
        a.state_raw = self._p(state_raw, torch.bfloat16, "state_raw")
        a.state_gate = self._p(state_gate, torch.float32, "state_gate")
        a.cand_role = cand_role
        a.cand = self._p(cand, torch.int32, "cand")
        return a


class PagedKV:
    """A csa2_paged_kv block kept alive with the tensors it points at, and the
    row format and device that it was made for."""

    def __init__(self, args: PagedKVArgs, tensors, fmt, device):
        self.args, self._keep, self.fmt, self.device = args, tensors, fmt, device


class PagePool:
    """A csa2_page_pool block kept alive with the tensors it points at, and
    their device."""

    def __init__(self, args: PagePoolArgs, tensors, device):
        self.args, self._keep, self.device = args, tensors, device


class PreparedCall:
    """One entry point's arguments, checked and converted once; each run()
    enqueues the call on the current stream."""

    def __init__(self, ctx: Context, name: str, args: tuple, tensors):
        self.ctx, self.name, self._keep = ctx, name, tensors
        self._fn = getattr(ctx.lib, name)
        types = SIGNATURES[name][1]
        conv = [C.c_void_p, C.c_int32, C.c_int64, C.c_size_t]
        self._args = tuple(t(a) if t in conv and not isinstance(a, t) else a for t, a in zip(types[2:], args))

    def run(self):
        st = self._fn(self.ctx.h, _stream(), *self._args)
        if st != CSA2_OK:
            self.ctx._ok(st, self.name)


class PreparedStep:
    """A csa2_step argument block kept alive with the tensors it points at."""

    def __init__(self, ctx: Context, args: StepArgs, tensors: dict):
        self.ctx, self.args, self._keep = ctx, args, tensors
        self.io = HostIO()

    def run(self):
        self.ctx._ok(self.ctx.lib.csa2_step(self.ctx.h, C.c_void_p(_stream()), C.byref(self.args)), "csa2_step")

    def run_host(self, q=None, raw=None, gate=None, out=None):
        """csa2_step_host: the step with its inputs in host tensors (pinned):
        q is copied in beside the scan, the raw tokens and gates before
        compress. A pinned `out` is written by the step directly; any other
        host `out` gets one copy of the prepared device output."""
        io = self.io
        io.q = None if q is None else q.data_ptr()
        io.raw = None if raw is None else raw.data_ptr()
        io.gate = None if gate is None else gate.data_ptr()
        io.out = None if out is None else out.data_ptr()
        self.ctx._ok(self.ctx.lib.csa2_step_host(self.ctx.h, C.c_void_p(_stream()), C.byref(self.args),
                                                 C.byref(io)), "csa2_step_host")

    def host_graph(self, q=None, raw=None, gate=None, out=None) -> "StepGraph":
        """csa2_step_graph_create: this step with these host buffers captured
        once; each StepGraph.launch() repeats the copies and the step."""
        io = HostIO()
        io.q = None if q is None else q.data_ptr()
        io.raw = None if raw is None else raw.data_ptr()
        io.gate = None if gate is None else gate.data_ptr()
        io.out = None if out is None else out.data_ptr()
        h = C.c_void_p()
        self.ctx._ok(self.ctx.lib.csa2_step_graph_create(self.ctx.h, C.byref(self.args), C.byref(io), C.byref(h)),
                     "csa2_step_graph_create")
        return StepGraph(self, h, (q, raw, gate, out))


class StepGraph:
    """A captured host step; holds the prepared step and host tensors it uses."""

    def __init__(self, prep: PreparedStep, handle, host_tensors):
        self.prep, self.h, self._keep = prep, handle, host_tensors

    def launch(self):
        self.prep.ctx._ok(self.prep.ctx.lib.csa2_step_graph_launch(self.h, C.c_void_p(_stream())),
                          "csa2_step_graph_launch")

    def __del__(self):
        if getattr(self, "h", None):
            self.prep.ctx.lib.csa2_step_graph_destroy(self.h)
            self.h = None


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A 256-byte-aligned byte buffer of at least nbytes (caching-allocator memory)."""
    t = torch.empty(max(int(nbytes), 1) + 256, dtype=torch.uint8, device=device or "cuda")
    off = (-t.data_ptr()) % 256
    return t[off:off + max(int(nbytes), 1)]
