"""Thin ctypes binding of libspin.so (include/spin.h).

Argument marshalling only: every step of the SPIN indexer step runs in the library's CUDA
kernels.  Tensors are passed as raw device pointers on torch's current stream.  There is
no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os
import re
from fractions import Fraction
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "libspin.so")
HEADER = os.path.join(ROOT, "include", "spin.h")

DTYPE = {"f32": 0, "bf16": 1, "e4m3": 2, "f16": 3}
TORCH_DTYPE = {0: torch.float32, 1: torch.bfloat16, 3: torch.float16}
COMBINE = {"max": 0, "sum": 1}
POOLING = {"max": 0, "mean": 1, "top4": 2, "slots": 3, "a2": 4}
EXPLORE = {"random": 0, "age": 1}
ROPE_LAYOUT = {"half": 0, "interleaved": 1}
SCORE_PATH = {"auto": 0, "generic": 1, "stream": 2, "tcgen05": 3}

# 2^64 / (2 pi): far enough that a frequency's own rounding to float64 is all that is lost
TURNS = Fraction(1 << 64) / (2 * Fraction("3.14159265358979323846264338327950288419716939937510582097"))

STATUS_BITS = {
    "BAD_N": 0x01, "BAD_QPOS": 0x02, "BAD_LIST": 0x04, "BAD_PAGE": 0x08,
    "BAD_ACCEPTED": 0x10, "TIMEOUT": 0x20, "BAD_RHO": 0x40, "BAD_PARENT": 0x80, "BAD_REF": 0x100,
    "NO_PAGES": 0x200,
}

ERRORS = {0: "SPIN_OK", 1: "SPIN_ERR_INVALID_ARG", 2: "SPIN_ERR_SHAPE", 3: "SPIN_ERR_CAPACITY",
          4: "SPIN_ERR_UNSUPPORTED", 5: "SPIN_ERR_CUDA"}


class SpinError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("%s: %s" % (ERRORS.get(code, code), msg))
        self.code = code


class SpinScoreExtras(ctypes.Structure):
    _fields_ = [("topk_hint", ctypes.c_void_p), ("topk_hint_bytes", ctypes.c_size_t)]


class SpinConfig(ctypes.Structure):
    _fields_ = [
        ("n_req", ctypes.c_int32), ("max_slots", ctypes.c_int32), ("max_rows", ctypes.c_int32),
        ("block", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("kv_heads", ctypes.c_int32), ("q_dtype", ctypes.c_int32), ("k_dtype", ctypes.c_int32),
        ("top_k", ctypes.c_int32), ("rho_bp", ctypes.c_int32), ("gamma_bp", ctypes.c_int32),
        ("alpha", ctypes.c_float), ("combine", ctypes.c_int32), ("seed", ctypes.c_uint64),
        ("score_path", ctypes.c_int32), ("pooling", ctypes.c_int32), ("explore", ctypes.c_int32),
        ("reserved", ctypes.c_int32),
    ]

    @property
    def max_blocks(self) -> int:
        return (self.max_slots + self.block - 1) // self.block

    @property
    def d_len(self) -> int:
        return self.max_slots + self.max_rows


class SpinKvConfig(ctypes.Structure):
    _fields_ = [
        ("n_req", ctypes.c_int32), ("max_slots", ctypes.c_int32), ("max_rows", ctypes.c_int32),
        ("block", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("softmax_scale", ctypes.c_float),
        ("reserved", ctypes.c_int32),
    ]


class SpinRopeConfig(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int32), ("rot_first", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
        ("layout", ctypes.c_int32), ("dtype", ctypes.c_int32), ("magnitude", ctypes.c_float),
    ]


class SpinRopeRows(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("in_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64), ("heads", ctypes.c_int64)]


class SpinPagePool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_bytes", ctypes.c_int64)]


def make_config(n_req, max_slots, max_rows, n_heads, head_dim, kv_heads, q_dtype, k_dtype, top_k,
                rho_bp, gamma_bp, alpha, combine="max", seed=0, block=64, score_path="auto",
                pooling="max", explore="random", **_ignored) -> SpinConfig:
    return SpinConfig(int(n_req), int(max_slots), int(max_rows), int(block), int(n_heads),
                      int(head_dim), int(kv_heads), DTYPE[q_dtype], DTYPE[k_dtype], int(top_k),
                      int(rho_bp), int(gamma_bp), float(alpha), COMBINE[combine],
                      int(seed) & 0xFFFFFFFFFFFFFFFF, SCORE_PATH[score_path], POOLING[pooling],
                      EXPLORE[explore], 0)


def make_kv_config(n_req, max_slots, max_rows, n_heads, kv_heads, head_dim, dtype, softmax_scale=None,
                   block=64) -> SpinKvConfig:
    """softmax_scale: 1 / sqrt(head_dim) by default."""
    if softmax_scale is None:
        softmax_scale = head_dim ** -0.5
    return SpinKvConfig(int(n_req), int(max_slots), int(max_rows), int(block), int(n_heads), int(kv_heads),
                        int(head_dim), DTYPE[dtype], float(softmax_scale), 0)


def make_rope_config(head_dim, dtype, rot_dim=None, rot_first=0, layout="half", magnitude=1.0) -> SpinRopeConfig:
    """rot_dim: the whole head by default."""
    return SpinRopeConfig(int(head_dim), int(rot_first), int(head_dim if rot_dim is None else rot_dim),
                          ROPE_LAYOUT[layout], DTYPE[dtype], float(magnitude))


def ensure_built() -> str:
    """Build the library in-tree if it is missing or stale (needs nvcc; no GPU needed)."""
    from . import build
    return build.build()


_LIB = None


def lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libspin.so is not built (%s); run __graft_entry__.build()" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, u64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64
        C = ctypes.POINTER(SpinConfig)
        K = ctypes.POINTER(SpinKvConfig)
        sig = {
            "spin_init_state": [C, P, P, P, P, i32, P],
            "spin_select_blocks": [C, P, P, P, P, P, P, i32, P, u64, i32, P, P, P, P, P,
                                   ctypes.c_size_t, P, P],
            "spin_select_blocks_noalloc": [C, P, P, P, P, P, P, i32, P, u64, i32, P, P, P, P, P, P],
            "spin_select_blocks_dstep": [C, P, P, P, P, P, P, i32, P, P, i32, P, P, P, P, P,
                                         ctypes.c_size_t, P, P],
            "spin_select_blocks_layers": [C, i32, i32, P, P, P, P, P, P, i32, P, u64, P, P, P, P, P,
                                          P, ctypes.c_size_t, P, P],
            "spin_update_ema_layers": [C, i32, P, P, P, P, P, P, P, P, P, P, P],
            "spin_commit_mtp_layers": [C, i32, P, P, P, P, P, i32, P, P, P, P, P, P, P],
            "spin_indexer_score": [C, P, P, P, P, i64, P, i64, P, P, P, i32, P, P, P],
            "spin_indexer_score_ex": [C, P, P, P, P, i64, P, i64, P, P, P, i32, P,
                                      ctypes.POINTER(SpinScoreExtras), P, P],
            "spin_topk_hint_size": [C, i32, ctypes.POINTER(ctypes.c_size_t)],
            "spin_init_topk_hint": [C, i32, P, ctypes.c_size_t, i32, P],
            "spin_topk_hinted": [C, P, P, P, P, P, i32, P, P, ctypes.c_size_t, P, P],
            "spin_topk": [C, P, P, P, P, i32, P, P, P],
            "spin_update_ema": [C, P, P, P, P, P, P, P, P, P, P, P],
            "spin_select_blocks_age": [C, P, P, P, P, P, P, i32, P, u64, i32, P, P, P, P, P, P,
                                       ctypes.c_size_t, P, P],
            "spin_update_ema_age": [C, P, P, P, P, P, P, P, P, P, P, u64, P, P],
            "spin_commit_mtp": [C, P, P, P, P, P, i32, P, P, P, P, P, P, P],
            "spin_workspace_size": [C, i32, ctypes.POINTER(ctypes.c_size_t)],
            "spin_kv_workspace_size": [K, i32, i32, ctypes.POINTER(ctypes.c_size_t)],
            "spin_kv_attend": [K, P, P, P, P, P, i64, P, i64, P, i32, P, i32, P, P, P, ctypes.c_size_t, P, P],
            "spin_kv_append": [K, P, P, i64, P, i32, P, P, P, P, P, i64, P, i64, P, P],
            "spin_rope": [ctypes.POINTER(SpinRopeConfig), ctypes.POINTER(SpinRopeRows), i32, i64, P, P, P],
            "spin_kv_prefill_workspace_size": [K, i64, i32, ctypes.POINTER(ctypes.c_size_t)],
            "spin_kv_prefill": [K, P, i64, P, i32, P, P, P, P, P, i64, P, i64, P, P, P, ctypes.c_size_t, P, P],
            "spin_kv_weigh_workspace_size": [K, i64, i32, ctypes.POINTER(ctypes.c_size_t)],
            "spin_kv_weigh": [K, P, P, i64, P, i32, P, P, P, i64, P, i64, ctypes.c_float, P, P, ctypes.c_size_t, P, P],
            "spin_pages_evict_workspace_size": [i32, i64, ctypes.POINTER(ctypes.c_size_t)],
            "spin_pages_evict": [i32, i64, P, i64, P, P, P, P, i32, i32, P, P, P, ctypes.c_size_t, P, P],
            "spin_pages_workspace_size": [i32, i64, ctypes.POINTER(ctypes.c_size_t)],
            "spin_pages_fork": [i32, i64, P, i64, P, P, P, P, P],
            "spin_pages_free": [i32, i64, P, i64, P, P, P, P],
            "spin_pages_reserve": [i32, i64, P, i64, P, P, P, P, i32, P, P, ctypes.c_size_t, P, P],
            "spin_pages_copy": [i32, i64, P, i32, P, ctypes.c_size_t, P, P],
            "spin_pages_compact": [i32, i64, P, i64, P, P, i32, P, P, ctypes.c_size_t, P, P],
            "spin_selftest_wait": [i32, u64, P, P, P],
            "spin_selftest_wait_moving": [i32, i32, u64, P, P, P],
            "spin_miss_curve": [P, i32, i64, P, P, i32, i32, P],
            "spin_allocate_budgets": [P, i32, i32, i32, i32, P, P],
        }
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        L.spin_version.restype = ctypes.c_char_p
        L.spin_last_error_string.restype = ctypes.c_char_p
        _LIB = L
    return _LIB


def header_functions():
    """Names of the functions include/spin.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(spin_[a-z_]+)\s*\(", text)))


def _check(rc: int):
    if rc != 0:
        raise SpinError(rc, lib().spin_last_error_string().decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    assert t.is_cuda and t.is_contiguous(), "device tensors must be contiguous CUDA tensors"
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    """The stream's handle (torch's current one by default, read without making a Stream object:
    0.3 us instead of 3)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _host(a, dtype):
    """A C-contiguous numpy array of `dtype` (host functions take host arrays)."""
    import numpy as np
    a = np.ascontiguousarray(a, dtype=dtype)
    return a, ctypes.c_void_p(a.ctypes.data)


def miss_curve(S, nb, topk, n_points=101):
    """One layer's miss curve over a batch (host arrays): S [n_req][stride] predicted block
    scores of a dense probe step, nb [n_req] blocks per context, topk [n_req][K] the probe's
    dense top-K.  Returns float32 [n_points]."""
    import numpy as np
    S, pS = _host(S, np.float32)
    nb, pnb = _host(nb, np.int32)
    topk, pk = _host(topk, np.int32)
    out = np.zeros(n_points, np.float32)
    _check(lib().spin_miss_curve(pS, S.shape[0], S.shape[1], pnb, pk, topk.shape[1], n_points,
                                 ctypes.c_void_p(out.ctypes.data)))
    return out


def allocate_budgets(miss, target_g, g_min=0):
    """Per-layer grid points and sparsities (basis points) from the layers' miss curves
    (host array [n_layers][n_points])."""
    import numpy as np
    miss, pm = _host(miss, np.float32)
    L, n_points = miss.shape
    g = np.zeros(L, np.int32)
    rho = np.zeros(L, np.int32)
    _check(lib().spin_allocate_budgets(pm, L, n_points, int(target_g), int(g_min),
                                       ctypes.c_void_p(g.ctypes.data), ctypes.c_void_p(rho.ctypes.data)))
    return g, rho


def selftest_wait(mode, limit_ns, status, elapsed_ns, stream=None):
    """spin_selftest_wait: the library's bounded barrier wait, with no arrival (mode 0), the
    abort flag raised (1) or an arrival (2)."""
    _check(lib().spin_selftest_wait(int(mode), int(limit_ns), _ptr(status), _ptr(elapsed_ns), _stream(stream)))


def selftest_wait_moving(steps, arrives, limit_ns, status, elapsed_ns, stream=None):
    """spin_selftest_wait_moving: the wait whose limit begins anew while a counter moves; the counter moves `steps` times,
    then the arrival comes (arrives true) or does not."""
    _check(lib().spin_selftest_wait_moving(int(steps), int(arrives), int(limit_ns), _ptr(status), _ptr(elapsed_ns), _stream(stream)))


def version() -> str:
    return lib().spin_version().decode()


def workspace_size(cfg: SpinConfig, rows: int = 1) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().spin_workspace_size(ctypes.byref(cfg), rows, ctypes.byref(out)))
    return int(out.value)


def init_state(cfg, V, D, Vmax, warm, req=-1, stream=None):
    _check(lib().spin_init_state(ctypes.byref(cfg), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm), req,
                                 _stream(stream)))


def select_blocks(cfg, V, D, Vmax, warm, n_slots, q_pos, rows, rho_override, step, layer, blocks,
                  n_blocks, union_blocks, n_union, workspace, status, stream=None):
    """`step` is an int, or a one-element int64 device tensor read by the kernels when they run
    (spin_select_blocks_dstep: a captured graph replays every step)."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if isinstance(step, torch.Tensor):
        assert step.dtype == torch.int64 and step.numel() == 1
        _check(lib().spin_select_blocks_dstep(
            ctypes.byref(cfg), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm), _ptr(n_slots), _ptr(q_pos),
            rows, _ptr(rho_override), _ptr(step), int(layer), _ptr(blocks), _ptr(n_blocks),
            _ptr(union_blocks), _ptr(n_union), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)))
        return
    _check(lib().spin_select_blocks(
        ctypes.byref(cfg), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm), _ptr(n_slots), _ptr(q_pos),
        rows, _ptr(rho_override), int(step), int(layer), _ptr(blocks), _ptr(n_blocks),
        _ptr(union_blocks), _ptr(n_union), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)))


def select_blocks_age(cfg, V, D, Vmax, warm, n_slots, q_pos, rows, rho_override, step, layer, block_age,
                      blocks, n_blocks, union_blocks, n_union, workspace, status, stream=None):
    """spin_select_blocks_age: block-age exploration; block_age is an int32 device tensor
    [R][MB] holding the uint32 ages."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().spin_select_blocks_age(
        ctypes.byref(cfg), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm), _ptr(n_slots), _ptr(q_pos),
        rows, _ptr(rho_override), int(step), int(layer), _ptr(block_age), _ptr(blocks), _ptr(n_blocks),
        _ptr(union_blocks), _ptr(n_union), _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)))


def update_ema_age(cfg, V, D, Vmax, warm, scores, list_, n_list, n_slots, q_pos, block_age, step, status,
                   stream=None):
    """spin_update_ema_age: the EMA update that also records the listed blocks' age."""
    _check(lib().spin_update_ema_age(ctypes.byref(cfg), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm),
                                     _ptr(scores), _ptr(list_), _ptr(n_list), _ptr(n_slots), _ptr(q_pos),
                                     _ptr(block_age), int(step), _ptr(status), _stream(stream)))


def select_blocks_layers(cfg, n_layers, layer0, V, D, Vmax, warm, n_slots, q_pos, rows, rho_table,
                         step, blocks, n_blocks, union_blocks, n_union, workspace, status, stream=None):
    """Selections of n_layers stacked layers (arrays [L][...]) in one launch.  `step` is an int
    or a one-element int64 device tensor read when the kernels run."""
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    step_dev = step if isinstance(step, torch.Tensor) else None
    _check(lib().spin_select_blocks_layers(
        ctypes.byref(cfg), int(n_layers), int(layer0), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm),
        _ptr(n_slots), _ptr(q_pos), rows, _ptr(rho_table), 0 if step_dev is not None else int(step),
        _ptr(step_dev), _ptr(blocks), _ptr(n_blocks), _ptr(union_blocks), _ptr(n_union),
        _ptr(workspace), ws_bytes, _ptr(status), _stream(stream)))


def update_ema_layers(cfg, n_layers, V, D, Vmax, warm, scores, list_, n_list, n_slots, q_pos, status,
                      stream=None):
    _check(lib().spin_update_ema_layers(ctypes.byref(cfg), int(n_layers), _ptr(V), _ptr(D), _ptr(Vmax),
                                        _ptr(warm), _ptr(scores), _ptr(list_), _ptr(n_list),
                                        _ptr(n_slots), _ptr(q_pos), _ptr(status), _stream(stream)))


def commit_mtp_layers(cfg, n_layers, V, D, Vmax, warm, scores, rows, union_blocks, n_union, n_slots,
                      q_pos, accepted, status, stream=None):
    _check(lib().spin_commit_mtp_layers(ctypes.byref(cfg), int(n_layers), _ptr(V), _ptr(D), _ptr(Vmax),
                                        _ptr(warm), _ptr(scores), rows, _ptr(union_blocks),
                                        _ptr(n_union), _ptr(n_slots), _ptr(q_pos), _ptr(accepted),
                                        _ptr(status), _stream(stream)))


def select_blocks_noalloc(cfg, V, D, Vmax, warm, n_slots, q_pos, rows, rho_override, step, layer,
                          blocks, n_blocks, union_blocks, n_union, status, stream=None):
    """spin_select_blocks without a workspace: for callers that cannot allocate device
    memory, the library's own static scratch array is used instead."""
    _check(lib().spin_select_blocks_noalloc(
        ctypes.byref(cfg), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm), _ptr(n_slots), _ptr(q_pos),
        rows, _ptr(rho_override), int(step), int(layer), _ptr(blocks), _ptr(n_blocks),
        _ptr(union_blocks), _ptr(n_union), _ptr(status), _stream(stream)))


def indexer_score(cfg, q, w, k_pool, k_scale, n_pages, block_table, list_, n_list, n_slots, rows,
                  scores, status, stream=None):
    _check(lib().spin_indexer_score(
        ctypes.byref(cfg), _ptr(q), _ptr(w), _ptr(k_pool), _ptr(k_scale), int(n_pages),
        _ptr(block_table), block_table.shape[-1], _ptr(list_), _ptr(n_list), _ptr(n_slots), rows,
        _ptr(scores), _ptr(status), _stream(stream)))


def indexer_score_ex(cfg, q, w, k_pool, k_scale, n_pages, block_table, list_, n_list, n_slots, rows,
                     scores, status, topk_hint=None, stream=None):
    """spin_indexer_score_ex: the score kernel also collects the hinted top-K's candidates
    into `topk_hint` (a TopkHint)."""
    ex = SpinScoreExtras()
    if topk_hint is not None:
        ex.topk_hint = topk_hint.buf.data_ptr()
        ex.topk_hint_bytes = topk_hint.nbytes
    _check(lib().spin_indexer_score_ex(
        ctypes.byref(cfg), _ptr(q), _ptr(w), _ptr(k_pool), _ptr(k_scale), int(n_pages),
        _ptr(block_table), block_table.shape[-1], _ptr(list_), _ptr(n_list), _ptr(n_slots), rows,
        _ptr(scores), ctypes.byref(ex), _ptr(status), _stream(stream)))


def topk_hint_size(cfg: SpinConfig, rows: int = 1) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().spin_topk_hint_size(ctypes.byref(cfg), rows, ctypes.byref(out)))
    return int(out.value)


def init_topk_hint(cfg, rows, hint, req=-1, stream=None):
    _check(lib().spin_init_topk_hint(ctypes.byref(cfg), rows, _ptr(hint.buf), hint.nbytes, int(req),
                                     _stream(stream)))


def topk_hinted(cfg, scores, w, list_, n_list, n_slots, rows, topk_idx, hint, status, stream=None):
    _check(lib().spin_topk_hinted(ctypes.byref(cfg), _ptr(scores), _ptr(w), _ptr(list_), _ptr(n_list),
                                  _ptr(n_slots), rows, _ptr(topk_idx), _ptr(hint.buf), hint.nbytes,
                                  _ptr(status), _stream(stream)))


HINT_WORDS = 16
HINT_FIELDS = ("guess", "count", "extra", "hit", "miss", "overflow", "cold", "exact", "last")


class TopkHint:
    """Device buffer of the temporal top-K hint (allocated by PyTorch), zeroed on creation."""

    def __init__(self, cfg: SpinConfig, rows: int = 1, device="cuda"):
        self.cfg, self.rows = cfg, rows
        self.nbytes = topk_hint_size(cfg, rows)
        self.buf = torch.zeros(((self.nbytes + 255) // 256) * 256, dtype=torch.uint8, device=device)
        assert self.buf.data_ptr() % 256 == 0

    def reset(self, req=-1, stream=None):
        init_topk_hint(self.cfg, self.rows, self, req, stream)

    def records(self):
        """uint32 [n_req * rows][HINT_WORDS] copy of the records (synchronises)."""
        n = self.cfg.n_req * self.rows * HINT_WORDS
        return self.buf[: 4 * n].view(torch.int32).view(-1, HINT_WORDS).cpu().numpy().view("uint32")

    def stats(self):
        """Totals over all rows of the hit / miss / overflow / cold / exact counters."""
        r = self.records().astype("int64")
        return {f: int(r[:, i].sum()) for i, f in enumerate(HINT_FIELDS) if f in
                ("hit", "miss", "overflow", "cold", "exact")}


def topk(cfg, scores, list_, n_list, n_slots, rows, topk_idx, status, stream=None):
    _check(lib().spin_topk(ctypes.byref(cfg), _ptr(scores), _ptr(list_), _ptr(n_list),
                           _ptr(n_slots), rows, _ptr(topk_idx), _ptr(status), _stream(stream)))


def update_ema(cfg, V, D, Vmax, warm, scores, list_, n_list, n_slots, q_pos, status, stream=None):
    _check(lib().spin_update_ema(ctypes.byref(cfg), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm),
                                 _ptr(scores), _ptr(list_), _ptr(n_list), _ptr(n_slots),
                                 _ptr(q_pos), _ptr(status), _stream(stream)))


def commit_mtp(cfg, V, D, Vmax, warm, scores, rows, union_blocks, n_union, n_slots, q_pos,
               accepted, status, stream=None):
    _check(lib().spin_commit_mtp(ctypes.byref(cfg), _ptr(V), _ptr(D), _ptr(Vmax), _ptr(warm),
                                 _ptr(scores), rows, _ptr(union_blocks), _ptr(n_union),
                                 _ptr(n_slots), _ptr(q_pos), _ptr(accepted), _ptr(status),
                                 _stream(stream)))


# --------------------------------------------------------------------------- KV cache
# The calls below check their tensors' types, shapes and device before they pass them on: every
# tensor must be contiguous and on the current device (a wrong shape would be read past its end).

def _arg(name, t, dtype, shape, device):
    """The address of a tensor argument of exactly this type and shape on `device`."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    raise SpinError(1, "%s must be a contiguous %s tensor of shape %s on the current device (cuda:%d); got %s %s "
                    "on %s%s" % (name, dtype, tuple(shape), device, t.dtype, tuple(t.shape), t.device,
                                 "" if t.is_contiguous() else ", not contiguous"))


def _kv_pool_args(cfg, k, v, k_scale, v_scale, block_table, dev):
    n = k.shape[0]
    pool, scale = (n, 64, cfg.kv_heads, cfg.head_dim), (n, cfg.kv_heads)
    bt = block_table.shape[-1]
    return (_arg("k", k, torch.uint8, pool, dev), _arg("v", v, torch.uint8, pool, dev),
            _arg("k_scale", k_scale, torch.float32, scale, dev), _arg("v_scale", v_scale, torch.float32, scale, dev),
            n, _arg("block_table", block_table, torch.int32, (cfg.n_req, bt), dev), bt)


def _status_arg(status, dev):
    return None if status is None else _arg("status", status, torch.int32, (1,), dev)


def _workspace_arg(workspace, dev):
    if workspace.get_device() != dev or not workspace.is_contiguous():
        raise SpinError(1, "workspace must be a contiguous tensor on the current device (cuda:%d)" % dev)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def kv_workspace(cfg: SpinKvConfig, rows: int = 1, top_k: int = 0, device="cuda"):
    """A workspace for kv_attend (spin_kv_workspace_size bytes)."""
    out = ctypes.c_size_t(0)
    _check(lib().spin_kv_workspace_size(ctypes.byref(cfg), rows, top_k, ctypes.byref(out)))
    return torch.empty(int(out.value), dtype=torch.uint8, device=device)


def kv_attend(cfg, q, k, v, k_scale, v_scale, block_table, n_slots, rows, topk_idx, out, lse, workspace, status,
              stream=None):
    """spin_kv_attend: attention of q [R][rows][n_heads][d] over the cache, over every slot
    (topk_idx None) or over the listed ones [R][rows][K].  n_slots int32 [R][rows]; lse fp32
    [R][rows][n_heads] or None."""
    dev = torch._C._cuda_getDevice()
    R, t, shape = cfg.n_req, TORCH_DTYPE.get(cfg.dtype), (cfg.n_req, rows, cfg.n_heads, cfg.head_dim)
    top_k = 0 if topk_idx is None else topk_idx.shape[-1]
    ws, ws_bytes = _workspace_arg(workspace, dev)
    _check(lib().spin_kv_attend(
        cfg, _arg("q", q, t, shape, dev),
        *_kv_pool_args(cfg, k, v, k_scale, v_scale, block_table, dev),
        _arg("n_slots", n_slots, torch.int32, (R, rows), dev), rows,
        None if topk_idx is None else _arg("topk_idx", topk_idx, torch.int32, (R, rows, top_k), dev), top_k,
        _arg("out", out, t, shape, dev),
        None if lse is None else _arg("lse", lse, torch.float32, shape[:3], dev), ws, ws_bytes,
        _status_arg(status, dev), _stream(stream)))


def kv_append(cfg, new_k, new_v, new_start, max_new, n_before, k, v, k_scale, v_scale, block_table, status,
              stream=None):
    """spin_kv_append: new_k, new_v [T][kv_heads][d]; request r's tokens new_start[r] ..
    new_start[r+1]-1 (at most max_new) go to its slots from n_before[r] on."""
    dev = torch._C._cuda_getDevice()
    T, t = new_k.shape[0], TORCH_DTYPE.get(cfg.dtype)
    shape = (T, cfg.kv_heads, cfg.head_dim)
    _check(lib().spin_kv_append(
        cfg, _arg("new_k", new_k, t, shape, dev), _arg("new_v", new_v, t, shape, dev), T,
        _arg("new_start", new_start, torch.int32, (cfg.n_req + 1,), dev), max_new,
        _arg("n_before", n_before, torch.int32, (cfg.n_req,), dev),
        *_kv_pool_args(cfg, k, v, k_scale, v_scale, block_table, dev), _status_arg(status, dev), _stream(stream)))


# --------------------------------------------------------------------- rotary positions
def rope_frequencies(rot_dim, theta=10000.0, scaling=None, factor=1.0, original=None, fast=32.0, slow=1.0):
    """Radians a position of the rot_dim / 2 pairs (float64 tensor on the host) and the magnitude that goes
    with them.  theta^(-2i / rot_dim), for contexts `factor` times as long as the `original` ones:
      None      as they are
      "linear"  positions squeezed together: every frequency divided by factor
      "base"    a larger base, theta factor^(rot_dim / (rot_dim - 2)): the slowest pair is divided by
                factor, the fastest one stays
      "parts"   (YaRN, arXiv 2309.00071) pairs that turn `fast` times or more within the original context
                stay, those that turn `slow` times or less are divided by factor, a linear ramp over
                the pairs between; magnitude 0.1 ln(factor) + 1"""
    if rot_dim < 2 or rot_dim % 2:
        raise SpinError(1, "rot_dim %d must be even and at least 2" % rot_dim)
    if not (0 < theta < math.inf and 1.0 <= factor < math.inf):
        raise SpinError(1, "theta must be positive and factor at least 1, both finite")
    i = torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim
    if scaling is None:
        if factor != 1.0:
            raise SpinError(1, "a factor needs a scaling")
        return theta ** -i, 1.0
    if scaling == "linear":
        return theta ** -i / factor, 1.0
    if scaling == "base":
        return (theta * factor ** (rot_dim / max(1, rot_dim - 2))) ** -i, 1.0
    if scaling == "parts":
        if original is None or not 0 < original < math.inf or not fast > slow > 0 or theta <= 1.0:
            raise SpinError(1, "parts: original > 0, fast > slow > 0 and theta above 1 needed")
        # the pair (a real number) that turns x times within the original context
        pair = lambda x: rot_dim * math.log(original / (2 * math.pi * x)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(0, math.floor(pair(fast))), min(rot_dim - 1, math.ceil(pair(slow)))
        ramp = ((torch.arange(rot_dim // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        ramp[max(0, math.ceil(pair(slow))):] = 1.0     # (the first pair too, where even that turns no more than `slow` times)
        f = theta ** -i
        return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    raise SpinError(1, "scaling must be None, linear, base or parts; got %r" % (scaling,))


def rope_turns(frequencies, device=None):
    """Radians a position (float64, [pairs]) as spin_rope's turns: round(f / (2 pi) 2^64) modulo 2^64, an
    int64 tensor that holds the 64 bits, on `device` (by default where the frequencies are, or cuda).  Set-up, kept for a model:
    exact arithmetic on the host (0.2 ms for 64 pairs), which waits for frequencies that are on the device."""
    f = torch.as_tensor(frequencies)
    if f.dtype is not torch.float64 or f.dim() != 1 or not bool(torch.isfinite(f).all()):
        raise SpinError(1, "frequencies must be a finite float64 tensor of one dimension")
    if device is None:
        device = f.device if f.is_cuda else "cuda"
    bits = [round(Fraction(x) * TURNS) % (1 << 64) for x in f.tolist()]
    return torch.tensor([b - (1 << 64) if b >> 63 else b for b in bits], dtype=torch.int64, device=device)


def _rope_rows(cfg, i, name, x, t, T, dev):
    """The address and token stride of a [T][heads][head_dim] tensor whose heads lie side by side."""
    if x.dtype is not t or x.get_device() != dev or x.dim() != 3 or x.shape[0] != T or x.shape[2] != cfg.head_dim:
        raise SpinError(1, "%s of rows %d must be a %s tensor of shape [%d][heads][%d] on the current device (cuda:%d); "
                        "got %s %s on %s" % (name, i, t, T, cfg.head_dim, dev, x.dtype, tuple(x.shape), x.device))
    heads = x.shape[1]
    if (x.stride(2) != 1 and x.shape[2] > 1) or (heads > 1 and x.stride(1) != cfg.head_dim):
        raise SpinError(1, "%s of rows %d: a token's heads must lie side by side" % (name, i))
    return x.data_ptr(), x.stride(0) if T > 1 else heads * cfg.head_dim


def rope(cfg, tensors, positions, turns, out=None, stream=None):
    """spin_rope: turns the heads of up to four tensors [T][heads][head_dim] (queries, keys; views of a
    fused projection may be given) by positions int32 [T] and turns int64 [rot_dim / 2] (rope_turns), into
    `out` (tensors of the same shapes) or, without it, in place."""
    dev = torch._C._cuda_getDevice()
    outs = tensors if out is None else out
    if len(outs) != len(tensors):
        raise SpinError(1, "as many tensors in out as given")
    T, t = positions.shape[0], TORCH_DTYPE.get(cfg.dtype)
    rows = (SpinRopeRows * max(1, len(tensors)))()
    for i, (x, y) in enumerate(zip(tensors, outs)):
        p, ps = _rope_rows(cfg, i, "in", x, t, T, dev)
        q, qs = _rope_rows(cfg, i, "out", y, t, T, dev)
        if x.shape != y.shape:
            raise SpinError(1, "out of rows %d has another shape" % i)
        rows[i] = SpinRopeRows(p, q, ps, qs, x.shape[1])
    _check(lib().spin_rope(cfg, rows, len(tensors), T, _arg("positions", positions, torch.int32, (T,), dev),
                           _arg("turns", turns, torch.int64, (cfg.rot_dim // 2,), dev), _stream(stream)))


# --------------------------------------------------------------------- chunks of new tokens
def _chunk_workspace(size, cfg, n_tokens, max_new, device):
    out = ctypes.c_size_t(0)
    _check(size(ctypes.byref(cfg), n_tokens, max_new, ctypes.byref(out)))
    return torch.empty(int(out.value), dtype=torch.uint8, device=device)


def kv_prefill_workspace(cfg: SpinKvConfig, n_tokens: int, max_new: int, device="cuda"):
    """A workspace for kv_prefill (spin_kv_prefill_workspace_size bytes)."""
    return _chunk_workspace(lib().spin_kv_prefill_workspace_size, cfg, n_tokens, max_new, device)


def kv_weigh_workspace(cfg: SpinKvConfig, n_tokens: int, max_new: int, device="cuda"):
    """A workspace for kv_weigh (spin_kv_weigh_workspace_size bytes)."""
    return _chunk_workspace(lib().spin_kv_weigh_workspace_size, cfg, n_tokens, max_new, device)


def _chunk_args(cfg, q, new_start, max_new, n_before, dev):
    T = q.shape[0]
    return (_arg("q", q, TORCH_DTYPE.get(cfg.dtype), (T, cfg.n_heads, cfg.head_dim), dev), T,
            _arg("new_start", new_start, torch.int32, (cfg.n_req + 1,), dev), max_new,
            _arg("n_before", n_before, torch.int32, (cfg.n_req,), dev))


def kv_prefill(cfg, q, new_start, max_new, n_before, k, v, k_scale, v_scale, block_table, out, lse, workspace, status,
               stream=None):
    """spin_kv_prefill: causal attention of the new tokens q [T][n_heads][d] over the cache that holds their keys
    and values already; request r's tokens new_start[r] .. new_start[r+1]-1 (at most max_new) are its slots from
    n_before[r] on.  lse fp32 [T][n_heads] or None."""
    dev = torch._C._cuda_getDevice()
    ws, ws_bytes = _workspace_arg(workspace, dev)
    _check(lib().spin_kv_prefill(
        cfg, *_chunk_args(cfg, q, new_start, max_new, n_before, dev),
        *_kv_pool_args(cfg, k, v, k_scale, v_scale, block_table, dev), _arg("out", out, q.dtype, q.shape, dev),
        None if lse is None else _arg("lse", lse, torch.float32, q.shape[:2], dev), ws, ws_bytes,
        _status_arg(status, dev), _stream(stream)))


def kv_weigh(cfg, q, lse, new_start, max_new, n_before, k, k_scale, block_table, decay, weight, workspace, status,
             stream=None):
    """spin_kv_weigh: adds the attention weight that the cached slots get from the tokens q (as in kv_prefill) to
    weight fp32 [R][64 bt] (a layer's own), after multiplying that by decay; lse fp32 [T][n_heads] as the attention over
    whole contexts returned it."""
    dev = torch._C._cuda_getDevice()
    ws, ws_bytes = _workspace_arg(workspace, dev)
    n, bt = k.shape[0], block_table.shape[-1]
    chunk = _chunk_args(cfg, q, new_start, max_new, n_before, dev)
    _check(lib().spin_kv_weigh(
        cfg, chunk[0], _arg("lse", lse, torch.float32, q.shape[:2], dev), *chunk[1:],
        _arg("k", k, torch.uint8, (n, 64, cfg.kv_heads, cfg.head_dim), dev),
        _arg("k_scale", k_scale, torch.float32, (n, cfg.kv_heads), dev), n,
        _arg("block_table", block_table, torch.int32, (cfg.n_req, bt), dev), bt, decay,
        _arg("weight", weight, torch.float32, (cfg.n_req, 64 * bt), dev), ws, ws_bytes, _status_arg(status, dev),
        _stream(stream)))


class KvCache:
    """Device buffers of one layer's 8-bit KV cache (allocated by PyTorch): codes and scales."""

    def __init__(self, n_pages: int, kv_heads: int, head_dim: int, device="cuda"):
        shape = (n_pages, 64, kv_heads, head_dim)
        self.k = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.v = torch.zeros(shape, dtype=torch.uint8, device=device)
        self.k_scale = torch.zeros((n_pages, kv_heads), dtype=torch.float32, device=device)
        self.v_scale = torch.zeros((n_pages, kv_heads), dtype=torch.float32, device=device)

    @property
    def tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale


class CoreAttention:
    """The attention behind the indexer's top-K, with its per-step device buffers: out
    [R][rows][n_heads][d], lse [R][rows][n_heads] and the workspace."""

    def __init__(self, cfg: SpinKvConfig, cache: KvCache, rows: int = 1, top_k: int = 0, device="cuda"):
        self.cfg, self.cache, self.rows = cfg, cache, rows
        shape = (cfg.n_req, rows, cfg.n_heads, cfg.head_dim)
        self.out = torch.zeros(shape, dtype=TORCH_DTYPE[cfg.dtype], device=device)
        self.lse = torch.zeros(shape[:3], dtype=torch.float32, device=device)
        self.row_slots = torch.zeros(shape[:2], dtype=torch.int32, device=device)
        self.workspace = kv_workspace(cfg, rows, top_k, device)

    def check(self, q, block_table, n_slots, topk_idx, status):
        """Refuses arguments that attend() would refuse, without a launch."""
        cfg, dev = self.cfg, torch._C._cuda_getDevice()
        R, shape = cfg.n_req, (cfg.n_req, self.rows, cfg.n_heads, cfg.head_dim)
        if _arg("core_q", q, TORCH_DTYPE[cfg.dtype], shape, dev) % 16:
            raise SpinError(1, "core_q must be 16-byte aligned")
        _kv_pool_args(cfg, *self.cache.tensors, block_table, dev)
        if 64 * block_table.shape[-1] < cfg.max_slots:
            raise SpinError(2, "block_table holds %d slots a request, the core attention's max_slots is %d" % (
                64 * block_table.shape[-1], cfg.max_slots))
        _arg("n_slots", n_slots, torch.int32, (R,), dev)
        if topk_idx is not None:
            _arg("topk_idx", topk_idx, torch.int32, (R, self.rows, topk_idx.shape[-1]), dev)
            if not 1 <= topk_idx.shape[-1] <= 16384:
                raise SpinError(1, "the core attention takes 1 to 16384 listed slots, got %d" % topk_idx.shape[-1])
        _arg("out", self.out, q.dtype, shape, dev)
        _status_arg(status, dev)

    def attend(self, q, block_table, n_slots, topk_idx, status, stream=None):
        """Every row of request r sees its n_slots[r] slots (the indexer's verifier rows do), or the
        listed ones of them."""
        row_slots = n_slots.view(-1, 1)
        if self.rows > 1:
            with torch.cuda.stream(stream):
                self.row_slots.copy_(row_slots.expand(-1, self.rows))
            row_slots = self.row_slots
        kv_attend(self.cfg, q, *self.cache.tensors, block_table, row_slots, self.rows, topk_idx, self.out, self.lse,
                  self.workspace, status, stream)


class PromptAttention:
    """The attention of prompts' chunks, with its buffers for up to n_tokens tokens a call, max_new of one request: rotated
    queries and keys, out [T][n_heads][d], lse [T][n_heads] and the workspaces.  rope: a SpinRopeConfig of the cache's
    head_dim and type, with its turns; None: queries and keys come as they are to be used.  Chunks that may run at the same
    time (on other streams) need one each; the layers of a model, one after the other, can share one by way of `cache` (but
    not a weight array: see kv_weigh)."""

    def __init__(self, cfg: SpinKvConfig, cache: KvCache, n_tokens: int, max_new: int, rope: Optional[SpinRopeConfig] = None,
                 turns=None, device="cuda"):
        if rope is not None and (turns is None or rope.head_dim != cfg.head_dim or rope.dtype != cfg.dtype):
            raise SpinError(1, "rope needs turns, and the cache's head_dim and type")
        self.cfg, self.cache, self.n_tokens, self.max_new, self.rope, self.turns = cfg, cache, n_tokens, max_new, rope, turns
        self.workspace = kv_prefill_workspace(cfg, n_tokens, max_new, device)
        self.weigh_workspace = kv_weigh_workspace(cfg, n_tokens, max_new, device)
        t = TORCH_DTYPE[cfg.dtype]
        self.q, self.out = (torch.empty((n_tokens, cfg.n_heads, cfg.head_dim), dtype=t, device=device) for _ in range(2))
        self.k, self.v = (torch.empty((n_tokens, cfg.kv_heads, cfg.head_dim), dtype=t, device=device) for _ in range(2))
        self.lse = torch.empty((n_tokens, cfg.n_heads), dtype=torch.float32, device=device)

    def check(self, q, k, v, positions, new_start, max_new, n_before, block_table, status, weight, decay=1.0):
        """Refuses arguments that a step of run_prompt would refuse, without a launch."""
        cfg, dev, T = self.cfg, torch._C._cuda_getDevice(), q.shape[0]
        if self.out.get_device() != dev:
            raise SpinError(1, "the buffers are on %s, the current device is cuda:%d" % (self.out.device, dev))
        if T > self.n_tokens or not 0 <= max_new <= min(self.max_new, cfg.max_slots):
            raise SpinError(2, "%d tokens, %d of a request at most; there is room for %d and %d" % (
                T, max_new, self.n_tokens, self.max_new))
        t = TORCH_DTYPE[cfg.dtype]
        for name, x, heads in (("q", q, cfg.n_heads), ("k", k, cfg.kv_heads), ("v", v, cfg.kv_heads)):
            if x.dtype is not t or x.shape != (T, heads, cfg.head_dim) or x.get_device() != dev:
                raise SpinError(1, "%s must be a %s tensor of shape %s on the current device (cuda:%d); got %s %s on %s" % (
                    name, t, (T, heads, cfg.head_dim), dev, x.dtype, tuple(x.shape), x.device))
            if name != "v" and self.rope is not None:
                _rope_rows(self.rope, name == "k", name, x, t, T, dev)
        if (positions is None) != (self.rope is None):
            raise SpinError(1, "positions and a rope go together")
        if positions is not None:
            _arg("positions", positions, torch.int32, (T,), dev)
            _arg("turns", self.turns, torch.int64, (self.rope.rot_dim // 2,), dev)
        _arg("new_start", new_start, torch.int32, (cfg.n_req + 1,), dev)
        _arg("n_before", n_before, torch.int32, (cfg.n_req,), dev)
        _kv_pool_args(cfg, *self.cache.tensors, block_table, dev)
        if 64 * block_table.shape[-1] < cfg.max_slots:
            raise SpinError(2, "block_table holds %d slots a request, max_slots is %d" % (64 * block_table.shape[-1], cfg.max_slots))
        if weight is not None:
            _arg("weight", weight, torch.float32, (cfg.n_req, 64 * block_table.shape[-1]), dev)
            if not math.isfinite(ctypes.c_float(decay).value):
                raise SpinError(1, "decay is not finite")
        _status_arg(status, dev)


POOLS_A_CALL = 16          # page arrays that one C call moves


class PagePools:
    """The arrays indexed by page that move with it: contiguous tensors [n_pages, ...] on one
    device, a page's bytes in each a multiple of 4.  Keeps them alive; a layer stack lists every layer's
    (`groups`: their descriptors, as many as a call takes at a time)."""

    def __init__(self, *tensors):
        if not tensors:
            raise SpinError(1, "at least one pool")
        self.tensors = tensors
        self.n_pages = tensors[0].shape[0]
        self.device = tensors[0].get_device()
        if self.n_pages < 1:
            raise SpinError(1, "pools without pages")
        descriptors = []
        for i, t in enumerate(tensors):
            if t.shape[0] != self.n_pages or t.get_device() != self.device or not t.is_contiguous() or not t.is_cuda:
                raise SpinError(1, "pool %d: contiguous CUDA tensors of as many pages on one device" % i)
            page_bytes = t.numel() // self.n_pages * t.element_size()
            # (all of them before the first call: a later group's refusal would tear the pages apart)
            if not 4 <= page_bytes <= 1 << 30 or page_bytes % 4 or t.data_ptr() % 4:
                raise SpinError(1, "pool %d: a page's bytes must be a multiple of 4 in [4, 2^30], 4-byte aligned" % i)
            descriptors.append(SpinPagePool(t.data_ptr(), page_bytes))
        cut = [descriptors[i:i + POOLS_A_CALL] for i in range(0, len(descriptors), POOLS_A_CALL)]
        self.groups = [(SpinPagePool * len(c))(*c) for c in cut]


def pages_workspace(n_req: int, n_pages: int, device="cuda"):
    """A workspace for pages_reserve and pages_compact (spin_pages_workspace_size bytes)."""
    out = ctypes.c_size_t(0)
    _check(lib().spin_pages_workspace_size(n_req, n_pages, ctypes.byref(out)))
    return torch.empty(int(out.value), dtype=torch.uint8, device=device)


def _table_shape(table, ref):
    if table.dim() != 2 or ref.dim() != 1:
        raise SpinError(2, "a block table has shape [n_req][blocks] and ref [n_pages]; got %s and %s" % (
            tuple(table.shape), tuple(ref.shape)))
    return (*table.shape, ref.shape[0])


def _pools_of(pools, n_pages, dev):
    if pools.n_pages != n_pages or pools.device != dev:
        raise SpinError(1, "the pools must have ref's %d pages and be on the current device" % n_pages)
    return pools.groups[0], len(pools.groups[0])


def _copy_rest(pools, n_req, ws, ws_bytes, status, s):
    """The copies of the call before, in the arrays that it did not take."""
    for g in pools.groups[1:]:
        _check(lib().spin_pages_copy(n_req, pools.n_pages, g, len(g), ws, ws_bytes, status, s))


def pages_fork(table_in, parent, table_out, ref, status, stream=None):
    """spin_pages_fork: row r of table_out becomes row parent[r] of table_in (-1: empty)."""
    R, bt, n_pages = _table_shape(table_out, ref)
    dev = torch._C._cuda_getDevice()
    _check(lib().spin_pages_fork(
        R, n_pages, _arg("table_in", table_in, torch.int32, (R, bt), dev), bt,
        _arg("parent", parent, torch.int32, (R,), dev), _arg("table_out", table_out, torch.int32, (R, bt), dev),
        _arg("ref", ref, torch.int32, (n_pages,), dev), _status_arg(status, dev), _stream(stream)))


def pages_free(block_table, keep_slots, ref, status, stream=None):
    """spin_pages_free: request r keeps the pages of its first keep_slots[r] slots (< 0: all)."""
    R, bt, n_pages = _table_shape(block_table, ref)
    dev = torch._C._cuda_getDevice()
    _check(lib().spin_pages_free(
        R, n_pages, _arg("block_table", block_table, torch.int32, (R, bt), dev), bt,
        _arg("keep_slots", keep_slots, torch.int32, (R,), dev), _arg("ref", ref, torch.int32, (n_pages,), dev),
        _status_arg(status, dev), _stream(stream)))


def pages_reserve(block_table, n_slots, n_new, ref, pools, granted, workspace, status, stream=None):
    """spin_pages_reserve: makes the next n_new[r] slots of every request writable."""
    R, bt, n_pages = _table_shape(block_table, ref)
    dev = torch._C._cuda_getDevice()
    ws, ws_bytes = _workspace_arg(workspace, dev)
    st, s = _status_arg(status, dev), _stream(stream)
    _check(lib().spin_pages_reserve(
        R, n_pages, _arg("block_table", block_table, torch.int32, (R, bt), dev), bt,
        _arg("n_slots", n_slots, torch.int32, (R,), dev), _arg("n_new", n_new, torch.int32, (R,), dev),
        _arg("ref", ref, torch.int32, (n_pages,), dev), *_pools_of(pools, n_pages, dev),
        _arg("granted", granted, torch.int32, (R,), dev), ws, ws_bytes, st, s))
    _copy_rest(pools, R, ws, ws_bytes, st, s)


def pages_compact(block_table, ref, pools, n_live, workspace, status, stream=None):
    """spin_pages_compact: moves the used pages to the lowest ids; n_live int32 [1]."""
    R, bt, n_pages = _table_shape(block_table, ref)
    dev = torch._C._cuda_getDevice()
    ws, ws_bytes = _workspace_arg(workspace, dev)
    st, s = _status_arg(status, dev), _stream(stream)
    _check(lib().spin_pages_compact(
        R, n_pages, _arg("block_table", block_table, torch.int32, (R, bt), dev), bt,
        _arg("ref", ref, torch.int32, (n_pages,), dev), *_pools_of(pools, n_pages, dev),
        _arg("n_live", n_live, torch.int32, (1,), dev), ws, ws_bytes, st, s))
    _copy_rest(pools, R, ws, ws_bytes, st, s)


def pages_evict_workspace(n_req: int, blocks: int, device="cuda"):
    """A workspace for pages_evict on tables of `blocks` entries a request."""
    out = ctypes.c_size_t(0)
    _check(lib().spin_pages_evict_workspace_size(n_req, blocks, ctypes.byref(out)))
    return torch.empty(int(out.value), dtype=torch.uint8, device=device)


def pages_evict(block_table, n_slots, weight, weight_out, keep_blocks, n_first, n_last, ref, kept, workspace, status,
                stream=None):
    """spin_pages_evict: request r is cut down to keep_blocks[r] blocks (< 0: left as it is), the first n_first, the
    newest n_last and the heaviest others by weight fp32 [R][64 bt] (kv_weigh's; of layers on one table, their sum);
    weight_out takes the weights in their new places, kept int32 [R][bt] the blocks that stayed.  A request's other arrays
    by slots or blocks follow that, or are reset: the indexer's by init_state and TopkHint.reset."""
    R, bt, n_pages = _table_shape(block_table, ref)
    dev = torch._C._cuda_getDevice()
    ws, ws_bytes = _workspace_arg(workspace, dev)
    _check(lib().spin_pages_evict(
        R, n_pages, _arg("block_table", block_table, torch.int32, (R, bt), dev), bt,
        _arg("n_slots", n_slots, torch.int32, (R,), dev), _arg("weight", weight, torch.float32, (R, 64 * bt), dev),
        _arg("weight_out", weight_out, torch.float32, (R, 64 * bt), dev),
        _arg("keep_blocks", keep_blocks, torch.int32, (R,), dev), n_first, n_last,
        _arg("ref", ref, torch.int32, (n_pages,), dev), _arg("kept", kept, torch.int32, (R, bt), dev), ws, ws_bytes,
        _status_arg(status, dev), _stream(stream)))


# ------------------------------------------------------------------------ convenience

class LayerState:
    """Device buffers of one layer's SPIN state (allocated by PyTorch)."""

    def __init__(self, cfg: SpinConfig, device="cuda"):
        R, MB = cfg.n_req, cfg.max_blocks
        self.V = torch.zeros((R, cfg.max_slots), dtype=torch.float32, device=device)
        self.D = torch.zeros((R, cfg.d_len), dtype=torch.float32, device=device)
        self.Vmax = torch.zeros((R, MB), dtype=torch.float32, device=device)
        self.warm = torch.zeros((R,), dtype=torch.int32, device=device)


class StepBuffers:
    """Per-step device buffers: selections, union, scores, top-K, workspace, status."""

    def __init__(self, cfg: SpinConfig, rows: int = 1, device="cuda"):
        R, MB = cfg.n_req, cfg.max_blocks
        self.rows = rows
        self.blocks = torch.full((R, rows, MB), -1, dtype=torch.int32, device=device)
        self.n_blocks = torch.zeros((R, rows), dtype=torch.int32, device=device)
        self.union = torch.full((R, MB), -1, dtype=torch.int32, device=device)
        self.n_union = torch.zeros((R,), dtype=torch.int32, device=device)
        self.scores = torch.zeros((R, rows, MB * 64), dtype=torch.float32, device=device)
        self.topk = torch.full((R, rows, cfg.top_k), -1, dtype=torch.int32, device=device)
        ws = workspace_size(cfg, rows)
        self.workspace = torch.zeros((ws + 255) // 256 * 64, dtype=torch.float32, device=device)
        self.status = torch.zeros((1,), dtype=torch.int32, device=device)

    @property
    def blist(self):
        return self.blocks[:, 0, :] if self.rows == 1 else self.union

    @property
    def n_list(self):
        return self.n_blocks[:, 0] if self.rows == 1 else self.n_union


def run_step(cfg, state: LayerState, buf: StepBuffers, q, w, k_pool, k_scale, n_pages,
             block_table, n_slots, q_pos, step=0, layer=0, rho_override=None, accepted=None,
             stream=None, hint: Optional[TopkHint] = None, block_age=None,
             core: Optional[CoreAttention] = None, core_q=None):
    """One decode step of one layer through the C ABI: select -> score -> top-K -> EMA
    (or, with rows > 1, select -> union -> score -> top-K -> deferred commit).  With a
    TopkHint the score kernel collects the temporal top-K's candidates and the hinted top-K
    replaces the plain one.  With a CoreAttention (of top_k = cfg.top_k) its queries core_q then
    attend to the top-K slots of its cache, whose pages block_table names too: core.out, core.lse."""
    rows = buf.rows
    if core is not None:  # before anything is launched: a step is not to stop halfway
        if core_q is None:
            raise SpinError(1, "core needs its queries core_q")
        core.check(core_q, block_table, n_slots, buf.topk, buf.status)
    union = buf.union if rows > 1 else None
    n_union = buf.n_union if rows > 1 else None
    if block_age is None:
        select_blocks(cfg, state.V, state.D, state.Vmax, state.warm, n_slots, q_pos, rows,
                      rho_override, step, layer, buf.blocks, buf.n_blocks, union, n_union,
                      buf.workspace, buf.status, stream)
    else:
        select_blocks_age(cfg, state.V, state.D, state.Vmax, state.warm, n_slots, q_pos, rows,
                          rho_override, step, layer, block_age, buf.blocks, buf.n_blocks, union, n_union,
                          buf.workspace, buf.status, stream)
    if rows == 1:
        blist = buf.blocks            # row 0 list: stride MB per request
        nlist = buf.n_blocks
    else:
        blist, nlist = buf.union, buf.n_union
    if hint is None:
        indexer_score(cfg, q, w, k_pool, k_scale, n_pages, block_table, blist, nlist, n_slots, rows,
                      buf.scores, buf.status, stream)
        topk(cfg, buf.scores, blist, nlist, n_slots, rows, buf.topk, buf.status, stream)
    else:
        indexer_score_ex(cfg, q, w, k_pool, k_scale, n_pages, block_table, blist, nlist, n_slots,
                         rows, buf.scores, buf.status, hint, stream)
        topk_hinted(cfg, buf.scores, w, blist, nlist, n_slots, rows, buf.topk, hint, buf.status, stream)
    if core is not None:
        core.attend(core_q, block_table, n_slots, buf.topk, buf.status, stream)
    if rows == 1 and block_age is not None:
        update_ema_age(cfg, state.V, state.D, state.Vmax, state.warm, buf.scores, blist, nlist,
                       n_slots, q_pos, block_age, step, buf.status, stream)
    elif rows == 1:
        update_ema(cfg, state.V, state.D, state.Vmax, state.warm, buf.scores, blist, nlist,
                   n_slots, q_pos, buf.status, stream)
    elif accepted is not None:
        commit_mtp(cfg, state.V, state.D, state.Vmax, state.warm, buf.scores, rows, blist, nlist,
                   n_slots, q_pos, accepted, buf.status, stream)


def run_prompt(core: PromptAttention, q, k, v, new_start, max_new, n_before, block_table, status, positions=None, weight=None,
               decay=1.0, stream=None):
    """One chunk of new tokens of one layer through the C ABI: rotate -> append -> attend (-> weigh).  q [T][n_heads][d], k and v
    [T][kv_heads][d] (views of a fused projection may be given); request r's tokens new_start[r] .. new_start[r+1]-1 become its
    slots from n_before[r] on, whose pages are there (pages_reserve).  With positions int32 [T] queries and keys are rotated by
    core.rope first; with weight fp32 [R][64 bt] the attention weight that the slots get from these tokens is added to it, after
    its multiplication with decay.  Returns core.out[:T] and core.lse[:T]; the rows of tokens behind the last request stay."""
    core.check(q, k, v, positions, new_start, max_new, n_before, block_table, status, weight, decay)
    cfg, T = core.cfg, q.shape[0]
    out, lse = core.out[:T], core.lse[:T]
    with torch.cuda.stream(stream):
        if positions is not None:
            rope(core.rope, (q, k), positions, core.turns, (core.q[:T], core.k[:T]), stream)
            q, k = core.q[:T], core.k[:T]
        # (views of a fused projection, and vectors at odd addresses, are laid out)
        laid = []
        for x, room in ((q, core.q), (k, core.k), (v, core.v)):
            if not x.is_contiguous() or x.data_ptr() % 16:
                room[:T].copy_(x)
                x = room[:T]
            laid.append(x)
        q, k, v = laid
    kv_append(cfg, k, v, new_start, max_new, n_before, *core.cache.tensors, block_table, status, stream)
    kv_prefill(cfg, q, new_start, max_new, n_before, *core.cache.tensors, block_table, out, lse, core.workspace, status, stream)
    if weight is not None:
        kv_weigh(cfg, q, lse, new_start, max_new, n_before, core.cache.k, core.cache.k_scale, block_table, decay, weight,
                 core.weigh_workspace, status, stream)
    return out, lse
