"""Thin ctypes binding of the C ABI in include/fi.h (argument marshalling only).

Every step of the attention path runs inside the compiled library; this module
only converts numpy / torch arguments into pointers and sizes.  Loading fails
loudly when the library has not been built: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_double, c_float, c_int, c_int32, c_int64, c_void_p

import numpy as np

from . import build as _build

FI_OK = 0
STATUS = {0: "ok", 1: "invalid argument", 2: "capacity", 3: "unsupported", 4: "cuda", 5: "device", 6: "no plan"}
DEVERR_PAGE_OOB = 0x1
DEVERR_WAIT_TIMEOUT = 0x2
DEVERR_TMEM = 0x4
DEVERR_KEPT = 0x8

_LIB = None


class FiError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}" + (f" ({detail})" if detail else ""))


def lib_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load the built library (raises if it is missing; run build() first)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"library not built: {path} is missing (call serving_attention_plan_gb300.build.build())")
    L = ctypes.CDLL(path)
    P32 = POINTER(c_int32)
    L.fi_workspace_create.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int, c_int, POINTER(c_void_p)]
    L.fi_workspace_destroy.argtypes = [c_void_p]
    L.fi_workspace_set_cost_model.argtypes = [c_void_p, c_int64, c_int64, c_int32]
    L.fi_workspace_set_variant.argtypes = [c_void_p, c_int32, ctypes.c_float, c_int32]
    L.fi_workspace_set_kv_dtype.argtypes = [c_void_p, c_int32, ctypes.c_float, ctypes.c_float]
    L.fi_plan.argtypes = [c_void_p, P32, P32, P32, P32, c_int, c_int, c_int, c_int, c_int, c_int, c_void_p]
    L.fi_plan_composable.argtypes = [c_void_p, P32, P32, P32, P32, c_int, P32, P32, P32, P32, c_int, c_int, c_int,
                                     c_int, c_int, c_int, c_void_p]
    L.fi_run.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p]
    L.fi_run_merge.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_void_p, c_void_p, c_void_p,
                               c_void_p]
    L.fi_merge_states.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_int, c_int,
                                  c_void_p]
    L.fi_workspace_set_rope.argtypes = [c_void_p, POINTER(c_double), c_int32, c_int32]
    L.fi_cache_plan_compute.argtypes = [P32, P32, P32, P32, c_int, c_int, P32, P32]
    L.fi_append.argtypes = [c_void_p, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_int64, c_void_p, c_void_p,
                            c_float, c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p]
    L.fi_key_weights.argtypes = [c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_float, c_int32, c_void_p, c_void_p]
    L.fi_select_keys.argtypes = [c_void_p, c_void_p, c_int, c_int32, c_int32, c_int32, c_void_p, c_void_p]
    L.fi_compact.argtypes = [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_int, c_void_p]
    L.fi_tree_run.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_int32, c_void_p, c_void_p, c_void_p]
    L.fi_tree_commit.argtypes = [c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int, c_void_p]
    L.fi_page_bounds.argtypes = [c_void_p, c_void_p, c_int, c_int32, c_void_p, c_void_p]
    L.fi_score_pages.argtypes = [c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_int32, c_void_p]
    L.fi_select_pages.argtypes = [c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p, c_void_p]
    L.fi_run_pages.argtypes = [c_void_p, c_void_p, c_void_p, c_void_p, c_int, c_void_p, c_int32, c_void_p, c_void_p, c_void_p]
    L.fi_get_error.argtypes = [c_void_p, P32]
    L.fi_plan_info.argtypes = [c_void_p, P32]
    L.fi_plan_compute.argtypes = [P32, P32, P32, c_int, c_int, c_int, c_int, c_int, c_int, c_int, c_int64, c_int64,
                                  c_int32, c_int32, P32, c_int64, POINTER(c_int64)]
    L.fi_plan_composable_compute.argtypes = [P32, P32, P32, c_int, P32, P32, P32, c_int, c_int, c_int, c_int, c_int,
                                             c_int, c_int, P32, c_int64, POINTER(c_int64)]
    L.fi_decode_noalloc.argtypes = [P32, P32, P32, P32, c_int, c_int, c_int, c_int, c_int, c_int, c_void_p, c_void_p,
                                    c_void_p, c_int, c_void_p, c_void_p, c_void_p]
    L.fi_decode_noalloc_get_error.argtypes = [P32]
    L.fi_device_sm_count.argtypes = [POINTER(c_int)]
    L.fi_status_string.argtypes = [c_int]
    L.fi_status_string.restype = ctypes.c_char_p
    L.fi_last_error_message.argtypes = []
    L.fi_last_error_message.restype = ctypes.c_char_p
    for name in ("fi_workspace_create", "fi_workspace_destroy", "fi_workspace_set_cost_model",
                 "fi_workspace_set_variant", "fi_workspace_set_kv_dtype", "fi_plan", "fi_run",
                 "fi_run_merge", "fi_merge_states", "fi_get_error", "fi_plan_info", "fi_plan_compute", "fi_device_sm_count",
                 "fi_decode_noalloc", "fi_decode_noalloc_get_error", "fi_plan_composable_compute",
                 "fi_plan_composable", "fi_workspace_set_rope", "fi_append", "fi_key_weights", "fi_select_keys",
                 "fi_compact", "fi_cache_plan_compute", "fi_tree_run", "fi_tree_commit", "fi_page_bounds", "fi_score_pages",
                 "fi_select_pages", "fi_run_pages"):
        getattr(L, name).restype = c_int
    _LIB = L
    return L


def _check(st: int, what: str):
    if st != FI_OK:
        detail = lib().fi_last_error_message().decode() if st == 4 else ""
        raise FiError(st, what, detail)


def _i32(a) -> np.ndarray:
    return np.ascontiguousarray(np.asarray(a, dtype=np.int32))


def _p32(a: np.ndarray):
    return a.ctypes.data_as(POINTER(c_int32))


def _stream_ptr(stream) -> c_void_p:
    if stream is None:
        import torch
        return c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return c_void_p(stream)
    return c_void_p(stream.cuda_stream)


def _dptr(t) -> c_void_p:
    return c_void_p(0 if t is None else t.data_ptr())


def _need(ok, what: str):
    if not ok:
        raise ValueError(what)


def _dense_error(t, name: str, dtypes, shape, device):
    """Says what is wrong with a tensor argument that should be dense, on the workspace's GPU, of a type and shape."""
    _need(t.dtype in dtypes, f"{name}: {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    _need(t.is_cuda, f"{name}: a CUDA tensor is needed")
    _need(t.get_device() == device, f"{name}: on GPU {t.get_device()}, the workspace is on GPU {device}")
    _need(tuple(t.shape) == tuple(shape), f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name}: a contiguous tensor is needed")


def _raw_stream(stream, device) -> int:
    """The stream's handle; the device's current stream for None."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def plan_compute(qo_indptr, kv_indptr, last_page_len, num_qo_heads, num_kv_heads, page_size, causal, num_sms,
                 head_dim=128, alpha=1, beta=1, l_min=256, window_left=-1) -> np.ndarray:
    """The host planner alone (no GPU): returns the flat int32 plan."""
    L = lib()
    qo, kv, last = _i32(qo_indptr), _i32(kv_indptr), _i32(last_page_len)
    batch = qo.shape[0] - 1
    n = c_int64(0)
    st = L.fi_plan_compute(_p32(qo), _p32(kv), _p32(last), batch, num_qo_heads, num_kv_heads, head_dim, page_size,
                           int(causal), num_sms, alpha, beta, l_min, window_left, None, 0, ctypes.byref(n))
    if st not in (FI_OK, 2):
        _check(st, "fi_plan_compute")
    out = np.zeros(max(int(n.value), 1), dtype=np.int32)
    st = L.fi_plan_compute(_p32(qo), _p32(kv), _p32(last), batch, num_qo_heads, num_kv_heads, head_dim, page_size,
                           int(causal), num_sms, alpha, beta, l_min, window_left, _p32(out), out.shape[0],
                           ctypes.byref(n))
    _check(st, "fi_plan_compute")
    return out[: n.value]


def plan_composable_compute(shared, unique, num_qo_heads, num_kv_heads, page_size, causal, num_sms,
                            head_dim=128) -> np.ndarray:
    """The composable planner alone (no GPU): shared and unique are (qo_indptr, kv_indptr, last_page_len)."""
    L = lib()
    sq, sk, sl = (_i32(x) for x in shared)
    uq, uk, ul = (_i32(x) for x in unique)
    n = c_int64(0)
    args = [_p32(sq), _p32(sk), _p32(sl), sq.shape[0] - 1, _p32(uq), _p32(uk), _p32(ul), uq.shape[0] - 1,
            num_qo_heads, num_kv_heads, head_dim, page_size, int(causal), num_sms]
    st = L.fi_plan_composable_compute(*args, None, 0, ctypes.byref(n))
    if st not in (FI_OK, 2):
        _check(st, "fi_plan_composable_compute")
    out = np.zeros(max(int(n.value), 1), dtype=np.int32)
    _check(L.fi_plan_composable_compute(*args, _p32(out), out.shape[0], ctypes.byref(n)), "fi_plan_composable_compute")
    return out[: n.value]


def cache_plan_compute(qo_indptr, kv_indptr, kv_indices, last_page_len, page_size):
    """What the cache operators derive from a batch (no GPU): (geometry [batch + 1, 8], pages twice, tails twice)."""
    qo, kv, idx, last = _i32(qo_indptr), _i32(kv_indptr), _i32(kv_indices), _i32(last_page_len)
    if idx.size == 0:
        idx = np.zeros(1, np.int32)
    geo, twice = np.zeros((qo.shape[0], 8), np.int32), np.zeros(2, np.int32)
    _check(lib().fi_cache_plan_compute(_p32(qo), _p32(kv), _p32(idx), _p32(last), qo.shape[0] - 1, page_size, _p32(geo),
                                       _p32(twice)), "fi_cache_plan_compute")
    return geo, bool(twice[0]), bool(twice[1])


def tree_mask(qo_indptr, parents) -> np.ndarray:
    """tree_run's mask of drafted trees: parents[t] is the place, within its request, of query token t's parent (before t's own), or -1
    for a child of the context.  int32 [total_q, words]: bit u of row t says that t sees its request's token u (ancestors and itself)."""
    qo, parents = _i32(qo_indptr), _i32(parents)
    _need(parents.shape == (int(qo[-1]),), f"parents: shape {parents.shape}, expected {(int(qo[-1]),)}")
    lens = np.diff(qo)
    words = max(1, -(-int(lens.max(initial=0)) // 32))
    mask = np.zeros((parents.shape[0], words), np.uint32)
    for q0, n in zip(qo[:-1], lens):
        for t in range(n):
            up = int(parents[q0 + t])
            _need(-1 <= up < t, f"parents[{q0 + t}] = {up}: a token's parent comes before it")
            if up >= 0:
                mask[q0 + t] = mask[q0 + up]
            mask[q0 + t, t >> 5] |= np.uint32(1 << (t & 31))
    return mask.view(np.int32)


def tree_positions(qo_indptr, parents, first) -> np.ndarray:
    """append's positions of drafted trees: first[i], the position of a child of request i's context (the tokens before the tree), plus a
    token's depth; parents as for tree_mask.  int32 [total_q]."""
    qo, parents, first = _i32(qo_indptr), _i32(parents), _i32(first)
    lens = np.diff(qo)
    _need(parents.shape == (int(qo[-1]),), f"parents: shape {parents.shape}, expected {(int(qo[-1]),)}")
    _need(first.shape == lens.shape, f"first: shape {first.shape}, expected {lens.shape}")
    out = np.zeros(parents.shape[0], np.int32)
    for t in range(int(lens.max(initial=0))):  # token t of all requests that have one
        i = np.flatnonzero(lens > t)
        q0, up = qo[i], parents[qo[i] + t]
        bad = np.flatnonzero((up < -1) | (up >= t))
        _need(len(bad) == 0, f"parents: token {t} of requests {i[bad].tolist()} does not have its parent before it")
        out[q0 + t] = np.where(up < 0, first[i], out[q0 + np.maximum(up, 0)] + 1)
    return out


def device_sm_count() -> int:
    v = c_int(0)
    _check(lib().fi_device_sm_count(ctypes.byref(v)), "fi_device_sm_count")
    return v.value


class Workspace:
    """Owns one fi_workspace (device + pinned buffers) at fixed capacity."""

    def __init__(self, max_batch, max_total_q, max_kv_pages, num_qo_heads, num_kv_heads, head_dim=128, num_sms=0):
        self._h = c_void_p(0)
        _check(lib().fi_workspace_create(max_batch, max_total_q, max_kv_pages, num_qo_heads, num_kv_heads, head_dim,
                                         num_sms, ctypes.byref(self._h)), "fi_workspace_create")
        import torch
        self._device = torch.cuda.current_device()  # where the workspace was just made
        self.num_qo_heads, self.num_kv_heads, self.head_dim = num_qo_heads, num_kv_heads, head_dim
        self._layout, self._kv_dtype = "HND", "bf16"
        self._plan = None  # (total_q, batch, page_size, layout, kv_dtype) of the current plan
        self._shapes_of = None  # the plan whose argument shapes the cache operators hold: _set_plan()

    def close(self):
        if self._h:
            lib().fi_workspace_destroy(self._h)
            self._h = c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def set_cost_model(self, alpha=1, beta=1, l_min=256):
        _check(lib().fi_workspace_set_cost_model(self._h, alpha, beta, l_min), "fi_workspace_set_cost_model")

    def set_variant(self, window_left=-1, logits_soft_cap=0.0, kv_layout="HND"):
        """Sliding window / logit soft-cap / page layout ("HND" or "NHD") for the following plan()."""
        layout = {"HND": 0, "NHD": 1}[kv_layout]
        _check(lib().fi_workspace_set_variant(self._h, int(window_left), float(logits_soft_cap), layout),
               "fi_workspace_set_variant")
        self._layout = kv_layout

    def set_kv_dtype(self, kv_dtype="bf16", k_scale=1.0, v_scale=1.0):
        """KV page element type ("bf16" or "e4m3", with per-tensor scales) for the following plan()."""
        _check(lib().fi_workspace_set_kv_dtype(self._h, {"bf16": 0, "e4m3": 1}[kv_dtype], float(k_scale),
                                               float(v_scale)), "fi_workspace_set_kv_dtype")
        self._kv_dtype = kv_dtype

    def set_rope(self, inv_freq, interleaved=False):
        """Rotary position of the following append() calls: radians per position of each pair (empty: none)."""
        f = np.ascontiguousarray(np.asarray(inv_freq, dtype=np.float64))
        _need(f.ndim == 1, "inv_freq: one value for each rotated pair")
        _check(lib().fi_workspace_set_rope(self._h, f.ctypes.data_as(POINTER(c_double)), 2 * f.shape[0],
                                           int(interleaved)), "fi_workspace_set_rope")

    def plan(self, qo_indptr, kv_indptr, kv_indices, last_page_len, page_size, causal, stream=None):
        qo, kv, idx, last = _i32(qo_indptr), _i32(kv_indptr), _i32(kv_indices), _i32(last_page_len)
        if idx.size == 0:
            idx = np.zeros(1, np.int32)
        _check(lib().fi_plan(self._h, _p32(qo), _p32(kv), _p32(idx), _p32(last), qo.shape[0] - 1, self.num_qo_heads,
                             self.num_kv_heads, self.head_dim, page_size, int(causal), _stream_ptr(stream)), "fi_plan")
        self._plan = (int(qo[-1]), qo.shape[0] - 1, page_size, self._layout, self._kv_dtype)

    def plan_composable(self, shared, unique, page_size, causal, stream=None):
        """Composable plan: shared and unique are (qo_indptr, kv_indptr, kv_indices, last_page_len)."""
        sq, sk, si, sl = (_i32(x) for x in shared)
        uq, uk, ui, ul = (_i32(x) for x in unique)
        si = si if si.size else np.zeros(1, np.int32)
        ui = ui if ui.size else np.zeros(1, np.int32)
        _check(lib().fi_plan_composable(self._h, _p32(sq), _p32(sk), _p32(si), _p32(sl), sq.shape[0] - 1, _p32(uq),
                                        _p32(uk), _p32(ui), _p32(ul), uq.shape[0] - 1, self.num_qo_heads,
                                        self.num_kv_heads, self.head_dim, page_size, int(causal), _stream_ptr(stream)),
               "fi_plan_composable")
        self._plan = (int(uq[-1]), uq.shape[0] - 1, page_size, self._layout, self._kv_dtype)

    def run(self, q, k_pages, v_pages, o, lse, stream=None):
        _check(lib().fi_run(self._h, _dptr(q), _dptr(k_pages), _dptr(v_pages), int(k_pages.shape[0]), _dptr(o),
                            _dptr(lse), _stream_ptr(stream)), "fi_run")

    def run_merge(self, q, k_pages, v_pages, o_prev, lse_prev, o, lse, stream=None):
        """fi_run with each output row merged (⊕) into the state (o_prev, lse_prev); o may be o_prev."""
        _check(lib().fi_run_merge(self._h, _dptr(q), _dptr(k_pages), _dptr(v_pages), int(k_pages.shape[0]),
                                  _dptr(o_prev), _dptr(lse_prev), _dptr(o), _dptr(lse), _stream_ptr(stream)),
               "fi_run_merge")

    def _set_plan(self):
        """The shapes and types that go with the current plan."""
        import torch
        if self._plan is None:
            raise FiError(6, "cache operator")
        total_q, batch, page_size, layout, kv_dtype = self._plan
        h, d = self.num_kv_heads, self.head_dim
        self._bf16, self._f32, self._i32 = (torch.bfloat16,), (torch.float32,), (torch.int32,)
        self._kv_types = self._bf16 if kv_dtype == "bf16" else (torch.float8_e4m3fn, torch.uint8)
        self._page_tail = (h, page_size, d) if layout == "HND" else (page_size, h, d)
        self._q_shape, self._kv_shape = (total_q, self.num_qo_heads, d), (total_q, h, d)
        self._lse_shape, self._kept_rows, self._page_size = (total_q, self.num_qo_heads), (batch, h), page_size
        self._pool, self._shapes_of = -1, self._plan

    def _need_plan(self):
        if self._plan is None or self._plan is not self._shapes_of:
            self._set_plan()

    def _set_pool(self, num_pages: int):
        """Shapes that go with a pool of so many pages."""
        self._need_plan()
        if num_pages != self._pool:
            self._pool = num_pages
            self._pool_shape = (num_pages, *self._page_tail)
            self._weights_shape = (num_pages, self.num_kv_heads, self._page_size)

    # every argument is checked in one expression; the slow path says what is wrong with it
    def _dense(self, t, name, dtypes, shape) -> int:
        if t.dtype in dtypes and t.get_device() == self._device and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
        _dense_error(t, name, dtypes, shape, self._device)

    def _rows(self, t, name, shape):
        """A tensor of shape [total_q, heads, 128] with dense heads: (pointer, token stride in elements)."""
        if t.dtype in self._bf16 and t.get_device() == self._device and t.shape == shape:
            st = t.stride()
            if st[2] == 1 and (st[1] == shape[2] or shape[1] == 1):
                return t.data_ptr(), (st[0] if shape[0] > 1 else max(st[0], shape[1] * shape[2]))
            raise ValueError(f"{name}: the heads of a token must be contiguous")
        _dense_error(t, name, self._bf16, shape, self._device)

    def append(self, q, k, v, k_pages, v_pages, q_out, q_weight=None, k_weight=None, eps=1e-6, positions=None,
               stream=None):
        """Norm (with weights) and rotate q and k of the plan's tokens; write q_out and the K/V page slots."""
        pool = k_pages.shape[0]
        self._set_pool(pool)
        dense = self._dense
        kp, vp = dense(k_pages, "k_pages", self._kv_types, self._pool_shape), dense(v_pages, "v_pages", self._kv_types, self._pool_shape)
        (pq, sq), (pk, sk), (pv, sv) = self._rows(q, "q", self._q_shape), self._rows(k, "k", self._kv_shape), self._rows(v, "v", self._kv_shape)
        out = dense(q_out, "q_out", self._bf16, self._q_shape)
        wq = None if q_weight is None else dense(q_weight, "q_weight", self._bf16, (self.head_dim,))
        wk = None if k_weight is None else dense(k_weight, "k_weight", self._bf16, (self.head_dim,))
        pos = None if positions is None else dense(positions, "positions", self._i32, (self._plan[0],))
        st = lib().fi_append(self._h, pq, sq, pk, sk, pv, sv, wq, wk, float(eps), pos, out, kp, vp, pool,
                             _raw_stream(stream, q.get_device()))
        if st:
            _check(st, "fi_append")

    def key_weights(self, q, k_pages, lse, weights, decay=1.0, new_keys=True, stream=None):
        """Add the attention weight of each cached key (from q, K and run()'s lse) to the decayed sums in weights."""
        pool = k_pages.shape[0]
        self._set_pool(pool)
        dense = self._dense
        st = lib().fi_key_weights(self._h, dense(q, "q", self._bf16, self._q_shape),
                                  dense(k_pages, "k_pages", self._kv_types, self._pool_shape), pool,
                                  dense(lse, "lse", self._f32, self._lse_shape), float(decay), int(new_keys),
                                  dense(weights, "weights", self._f32, self._weights_shape),
                                  _raw_stream(stream, weights.get_device()))
        if st:
            _check(st, "fi_key_weights")

    def select_keys(self, weights, budget, kept, recent=0, sink=0, stream=None):
        """kept[request, KV head] = the positions to keep: the first sink, the last recent, the heaviest of the rest."""
        pool, budget = weights.shape[0], int(budget)
        self._set_pool(pool)
        st = lib().fi_select_keys(self._h, self._dense(weights, "weights", self._f32, self._weights_shape), pool,
                                  int(sink), int(recent), budget, self._dense(kept, "kept", self._i32, (*self._kept_rows, budget)),
                                  _raw_stream(stream, weights.get_device()))
        if st:
            _check(st, "fi_select_keys")

    def compact(self, kept, k_pages, v_pages, weights=None, stream=None):
        """Move the kept K/V rows (and weights) of every request over the budget (kept's last size) to its first slots."""
        pool = k_pages.shape[0]
        self._set_pool(pool)
        dense = self._dense
        budget = kept.shape[-1]
        st = lib().fi_compact(self._h, dense(kept, "kept", self._i32, (*self._kept_rows, budget)), budget,
                              dense(k_pages, "k_pages", self._kv_types, self._pool_shape),
                              dense(v_pages, "v_pages", self._kv_types, self._pool_shape),
                              None if weights is None else dense(weights, "weights", self._f32, self._weights_shape), pool,
                              _raw_stream(stream, k_pages.get_device()))
        if st:
            _check(st, "fi_compact")

    def tree_run(self, q, k_pages, v_pages, mask, o, lse, stream=None):
        """Attention of drafted tokens: each query token sees the context and the drafted tokens of its row of mask (see tree_mask)."""
        pool = k_pages.shape[0]
        self._set_pool(pool)
        dense, n = self._dense, self._plan[0]
        words = mask.shape[-1] if mask.dim() == 2 else -1
        st = lib().fi_tree_run(self._h, dense(q, "q", self._bf16, self._q_shape),
                               dense(k_pages, "k_pages", self._kv_types, self._pool_shape),
                               dense(v_pages, "v_pages", self._kv_types, self._pool_shape), pool,
                               dense(mask, "mask", self._i32, (n, words)), words,
                               dense(o, "o", self._bf16, self._q_shape), dense(lse, "lse", self._f32, self._lse_shape),
                               _raw_stream(stream, q.get_device()))
        if st:
            _check(st, "fi_tree_run")

    def tree_commit(self, path, k_pages, v_pages, stream=None):
        """Move the K/V rows of each request's accepted drafted tokens (path: ascending, then -1) to the first drafted slots."""
        pool = k_pages.shape[0]
        self._set_pool(pool)
        dense, length = self._dense, path.shape[-1]
        st = lib().fi_tree_commit(self._h, dense(path, "path", self._i32, (self._plan[1], length)), length,
                                  dense(k_pages, "k_pages", self._kv_types, self._pool_shape),
                                  dense(v_pages, "v_pages", self._kv_types, self._pool_shape), pool,
                                  _raw_stream(stream, k_pages.get_device()))
        if st:
            _check(st, "fi_tree_commit")

    def page_bounds(self, k_pages, bounds, new_keys=False, stream=None):
        """bounds[page, KV head] = smallest and largest key of the plan's pages (new_keys: of those that hold the new tokens), per dim."""
        pool = k_pages.shape[0]
        self._set_pool(pool)
        st = lib().fi_page_bounds(self._h, self._dense(k_pages, "k_pages", self._kv_types, self._pool_shape), pool, int(new_keys),
                                  self._dense(bounds, "bounds", self._bf16, (pool, self.num_kv_heads, 2, self.head_dim)),
                                  _raw_stream(stream, k_pages.get_device()))
        if st:
            _check(st, "fi_page_bounds")

    def score_pages(self, q, bounds, scores, stream=None):
        """scores[token, KV head, place in the page list] = upper bound of the logits of the page's keys for the token's heads."""
        pool, row = bounds.shape[0], scores.shape[-1]
        self._set_pool(pool)
        st = lib().fi_score_pages(self._h, self._dense(q, "q", self._bf16, self._q_shape),
                                  self._dense(bounds, "bounds", self._bf16, (pool, self.num_kv_heads, 2, self.head_dim)), pool,
                                  self._dense(scores, "scores", self._f32, (self._plan[0], self.num_kv_heads, row)), row,
                                  _raw_stream(stream, q.get_device()))
        if st:
            _check(st, "fi_score_pages")

    def select_pages(self, scores, selected, recent=0, sink=0, stream=None):
        """selected[token, KV head] = the page ids to attend to: the first sink, the last recent, the best of the rest, then -1."""
        self._need_plan()
        row, budget = scores.shape[-1], selected.shape[-1]
        st = lib().fi_select_pages(self._h, self._dense(scores, "scores", self._f32, (self._plan[0], self.num_kv_heads, row)), row,
                                   int(sink), int(recent), budget,
                                   self._dense(selected, "selected", self._i32, (self._plan[0], self.num_kv_heads, budget)),
                                   _raw_stream(stream, scores.get_device()))
        if st:
            _check(st, "fi_select_pages")

    def run_pages(self, q, k_pages, v_pages, selected, o, lse, stream=None):
        """Attention of each query token and KV head over its own list of pages (as select_pages writes it)."""
        pool = k_pages.shape[0]
        self._set_pool(pool)
        dense, budget = self._dense, selected.shape[-1]
        st = lib().fi_run_pages(self._h, dense(q, "q", self._bf16, self._q_shape),
                                dense(k_pages, "k_pages", self._kv_types, self._pool_shape),
                                dense(v_pages, "v_pages", self._kv_types, self._pool_shape), pool,
                                dense(selected, "selected", self._i32, (self._plan[0], self.num_kv_heads, budget)), budget,
                                dense(o, "o", self._bf16, self._q_shape), dense(lse, "lse", self._f32, self._lse_shape),
                                _raw_stream(stream, q.get_device()))
        if st:
            _check(st, "fi_run_pages")

    def info(self) -> np.ndarray:
        h = np.zeros(16, np.int32)
        _check(lib().fi_plan_info(self._h, _p32(h)), "fi_plan_info")
        return h

    def get_error(self) -> int:
        e = np.zeros(1, np.int32)
        _check(lib().fi_get_error(self._h, _p32(e)), "fi_get_error")
        return int(e[0])

    @property
    def handle(self) -> int:
        return self._h.value


def decode_noalloc(qo_indptr, kv_indptr, kv_indices, last_page_len, num_qo_heads, num_kv_heads, page_size, causal,
                   q, k_pages, v_pages, o, lse, stream=None, head_dim=128):
    """Plan and run one decode batch with no workspace (the library's static scratch array)."""
    qo, kv, idx, last = _i32(qo_indptr), _i32(kv_indptr), _i32(kv_indices), _i32(last_page_len)
    if idx.size == 0:
        idx = np.zeros(1, np.int32)
    _check(lib().fi_decode_noalloc(_p32(qo), _p32(kv), _p32(idx), _p32(last), qo.shape[0] - 1, num_qo_heads,
                                   num_kv_heads, head_dim, page_size, int(causal), _dptr(q), _dptr(k_pages),
                                   _dptr(v_pages), int(k_pages.shape[0]), _dptr(o), _dptr(lse), _stream_ptr(stream)),
           "fi_decode_noalloc")


def decode_noalloc_get_error() -> int:
    """Read and clear the device-side error bits of the allocation-free entry point (synchronises)."""
    e = np.zeros(1, np.int32)
    _check(lib().fi_decode_noalloc_get_error(_p32(e)), "fi_decode_noalloc_get_error")
    return int(e[0])


def merge_states(o_a, lse_a, o_b, lse_b, o, lse, stream=None):
    rows, heads, d = o.shape
    _check(lib().fi_merge_states(_dptr(o_a), _dptr(lse_a), _dptr(o_b), _dptr(lse_b), _dptr(o), _dptr(lse), rows, heads,
                                 d, _stream_ptr(stream)), "fi_merge_states")
