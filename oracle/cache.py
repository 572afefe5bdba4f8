"""Float64 oracle of the cache operators: append, accumulated attention weights, selection, compaction.

Test infrastructure only; every step is the definition, on the arrays of a batch:
qo_indptr, kv_indptr, kv_indices, last_page_len, page_size.
"""
from __future__ import annotations

import numpy as np

from .attention import gather_kv, request_lengths


def places(batch, i: int, keys) -> tuple[np.ndarray, np.ndarray]:
    """Pages and slots of the given keys of request i."""
    keys = np.asarray(keys, np.int64)
    page = np.asarray(batch.kv_indices, np.int64)[int(batch.kv_indptr[i]) + keys // batch.page_size]
    return page, keys % batch.page_size


def lengths(batch):
    return request_lengths(batch.qo_indptr, batch.kv_indptr, batch.last_page_len, batch.page_size)


def norm_rotate(x, weight, eps, inv_freq, positions, interleaved):
    """[tokens, heads, D] float64: x w / sqrt(mean x^2 + eps), then each pair turned by position * frequency."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight
    for j, f in enumerate(inv_freq):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + len(inv_freq))
        c, s = np.cos(positions * f)[:, None], np.sin(positions * f)[:, None]
        x[..., a], x[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return x


def append_places(batch):
    """(token, page, slot) of every query token that has a slot, and each token's key index."""
    l_q, l_kv = lengths(batch)
    tok, page, slot, key = [], [], [], np.zeros(int(batch.qo_indptr[-1]), np.int64)
    for i in range(len(l_q)):
        for t in range(int(l_q[i])):
            j = int(l_kv[i] - l_q[i]) + t
            key[int(batch.qo_indptr[i]) + t] = j
            if j >= 0:
                p, s = places(batch, i, [j])
                tok.append(int(batch.qo_indptr[i]) + t)
                page.append(int(p[0]))
                slot.append(int(s[0]))
    return np.array(tok, np.int64), np.array(page, np.int64), np.array(slot, np.int64), key


def key_weights(batch, q, k_pages, lse, weights, decay, new_keys, k_scale=1.0, window=-1, cap=0.0, layout="HND"):
    """The updated weights [pages, H_kv, page_size] and, per entry, a bound of sum |terms of the logit| (for tolerances)."""
    l_q, l_kv = lengths(batch)
    hkv = weights.shape[1]
    g = q.shape[1] // hkv
    out = np.array(weights, np.float64)
    reach = 0.0
    scale = 1.0 / np.sqrt(q.shape[2])
    for i in range(len(l_q)):
        n, t = int(l_kv[i]), int(l_q[i])
        if n == 0:
            continue
        rows = slice(int(batch.qo_indptr[i]), int(batch.qo_indptr[i]) + t)
        pos = n - t + np.arange(t)[:, None]
        j = np.arange(n)[None, :]
        seen = np.ones((t, n), bool)
        if batch.causal:
            seen = j <= pos
            if window >= 0:
                seen &= j >= pos - window
        page, slot = places(batch, i, np.arange(n))
        for h in range(hkv):
            k = gather_kv(k_pages, batch.kv_indptr, batch.kv_indices, n, batch.page_size, i, h, layout) * k_scale
            add = np.zeros(n)
            for hh in range(h * g, (h + 1) * g):
                x = scale * q[rows, hh] @ k.T
                if cap > 0:
                    x = cap * np.tanh(x / cap)
                l = np.asarray(lse, np.float64)[rows, hh][:, None]
                with np.errstate(invalid="ignore", over="ignore"):
                    w = np.where(seen & ~np.isneginf(l), np.exp(np.where(seen, x, 0) - np.where(np.isneginf(l), 0, l)), 0.0)
                add += w.sum(0)
                if t:
                    with np.errstate(invalid="ignore"):
                        r = (np.abs(q[rows, hh]) @ np.abs(k).T * scale)[seen]
                    if r.size and np.isfinite(r).any():
                        reach = max(reach, float(np.nanmax(np.where(np.isfinite(r), r, 0))))
            old = out[page, h, slot] * decay if decay else np.zeros(n)
            if new_keys:
                old[max(0, n - t):] = 0.0
            out[page, h, slot] = old + add
    return out, reach


def select(batch, weights, budget, recent, sink):
    """[batch, H_kv, budget] int32: kept positions, ascending, then -1."""
    _, l_kv = lengths(batch)
    kept = np.full((len(l_kv), weights.shape[1], budget), -1, np.int32)
    for i, n in enumerate(int(x) for x in l_kv):
        for h in range(weights.shape[1]):
            if n <= budget:
                kept[i, h, :n] = np.arange(n)
                continue
            page, slot = places(batch, i, np.arange(n))
            w = weights[page, h, slot].astype(np.float64)
            free = np.arange(sink, n - recent)
            # the largest first (NaN before everything), then the lowest position
            nan = np.isnan(w[free])
            order = np.lexsort((free, np.where(nan, 0.0, -w[free]), ~nan))
            best = free[order[:budget - sink - recent]]
            kept[i, h] = np.sort(np.concatenate([np.arange(sink), best, np.arange(n - recent, n)]))
    return kept


def compact(batch, kept, arrays, layouts):
    """Copies of the page arrays ([pages, H_kv, slot, ...] "HND" or [pages, slot, H_kv, ...] "NHD") with the kept rows in front."""
    _, l_kv = lengths(batch)
    out = [a.copy() for a in arrays]
    budget = kept.shape[2]
    for i, n in enumerate(int(x) for x in l_kv):
        if n <= budget:
            continue
        tp, ts = places(batch, i, np.arange(budget))
        for h in range(kept.shape[1]):
            fp, fs = places(batch, i, kept[i, h])
            for a, o, layout in zip(arrays, out, layouts):
                if layout == "HND":
                    o[tp, h, ts] = a[fp, h, fs]
                else:
                    o[tp, ts, h] = a[fp, fs, h]
    return out
