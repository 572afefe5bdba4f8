"""Float64 oracle of attention over parts of a cache: trees of drafted tokens, and pages chosen by a score.

Test infrastructure only; every step is the definition, on the arrays of a batch:
qo_indptr, kv_indptr, kv_indices, last_page_len, page_size, causal.
"""
from __future__ import annotations

import numpy as np

from .attention import gather_kv
from .cache import lengths, places


def state(q, k, v, seen, cap=0.0, q_floor=0.0):
    """(o, lse, spread, reach) of rows q [m, D] over keys k, v [n, D] under seen [m, n]: softmax(x) v with x = q.k / sqrt(D),
    soft-capped; spread = softmax(x) |v| and reach = the largest sum of |terms| of a seen logit, each |q_d| with q_floor of the
    row's largest added (both for tolerances)."""
    m, n = seen.shape
    o, lse = np.zeros((m, q.shape[1])), np.full(m, -np.inf)
    spread, reach = np.zeros_like(o), np.zeros(m)
    scale = 1.0 / np.sqrt(q.shape[1])
    for r in range(m):
        on = np.nonzero(seen[r])[0]
        if not len(on):
            continue
        x = scale * (k[on] @ q[r])
        if cap > 0:
            x = cap * np.tanh(x / cap)
        top = x.max()
        w = np.exp(x - top)
        lse[r] = top + np.log(w.sum())
        w /= w.sum()
        o[r], spread[r] = w @ v[on], w @ np.abs(v[on])
        reach[r] = scale * (np.abs(k[on]) @ (np.abs(q[r]) + q_floor * np.abs(q[r]).max())).max()
    return o, lse, spread, reach


def tree_seen(mask, q0, l_q, l_kv):
    """[l_q, l_kv] bool of one request: the context, and the drafted keys whose bit is set."""
    seen = np.zeros((l_q, l_kv), bool)
    words = np.asarray(mask).view(np.uint32)
    for t in range(l_q):
        for j in range(l_kv):
            u = j - (l_kv - l_q)
            seen[t, j] = u < 0 or (u >> 5 < words.shape[1] and bool(words[q0 + t, u >> 5] >> np.uint32(u & 31) & 1))
    return seen


def tree_attention(batch, q, k_pages, v_pages, mask, cap=0.0, layout="HND", q_floor=0.0):
    """(o, lse, spread, reach) of every query row: [total_q, H_qo, D] and [total_q, H_qo]."""
    l_q, l_kv = lengths(batch)
    hkv = k_pages.shape[1] if layout == "HND" else k_pages.shape[2]
    g = q.shape[1] // hkv
    out = [np.zeros(q.shape), np.full(q.shape[:2], -np.inf), np.zeros(q.shape), np.zeros(q.shape[:2])]
    for i in range(len(l_q)):
        n, t, q0 = int(l_kv[i]), int(l_q[i]), int(batch.qo_indptr[i])
        if t == 0 or n == 0:
            continue
        seen = tree_seen(mask, q0, t, n)
        for h in range(hkv):
            k, v = (gather_kv(x, batch.kv_indptr, batch.kv_indices, n, batch.page_size, i, h, layout) for x in (k_pages, v_pages))
            for hh in range(h * g, (h + 1) * g):
                for a, b in zip(out, state(q[q0:q0 + t, hh], k, v, seen, cap, q_floor)):
                    a[q0:q0 + t, hh] = b
    return out


def commit(batch, path, arrays, layout="HND"):
    """Copies of the page arrays with the rows of the accepted tokens (ascending places, then -1) at the first drafted slots."""
    l_q, l_kv = lengths(batch)
    out = [a.copy() for a in arrays]
    for i in range(len(l_q)):
        off = int(l_kv[i] - l_q[i])
        for j, e in enumerate(int(x) for x in path[i]):
            if e < 0:
                break
            if off + j < 0:
                continue
            (fp,), (fs,) = places(batch, i, [off + e])
            (tp,), (ts,) = places(batch, i, [off + j])
            for a, o in zip(arrays, out):
                if layout == "HND":
                    o[tp, :, ts] = a[fp, :, fs]
                else:
                    o[tp, ts] = a[fp, fs]
    return out


def page_bounds(batch, k_pages, old, new_keys, layout="HND"):
    """[pages, H_kv, 2, D]: smallest and largest key of each visited page, NaN first; other pages as in old."""
    l_q, l_kv = lengths(batch)
    out = np.array(old, np.float64)
    for i in range(len(l_q)):
        n = int(l_kv[i])
        first = max(0, n - int(l_q[i])) if new_keys else 0
        if new_keys and l_q[i] == 0:
            continue
        for e in range(first // batch.page_size, -(-n // batch.page_size)):
            page = int(batch.kv_indices[int(batch.kv_indptr[i]) + e])
            used = min(batch.page_size, n - e * batch.page_size)
            rows = k_pages[page][:, :used] if layout == "HND" else k_pages[page][:used].transpose(1, 0, 2)
            out[page, :, 0], out[page, :, 1] = rows.min(1), rows.max(1)
    return out


def last_key(batch, i, t):
    """The last key that query token t of request i sees."""
    l_q, l_kv = lengths(batch)
    return int(l_kv[i] - l_q[i]) + t if batch.causal else int(l_kv[i]) - 1


def page_scores(batch, q, bounds, old, k_scale=1.0):
    """(scores [total_q, H_kv, row], the largest sum of |terms| of a row)."""
    l_q, _ = lengths(batch)
    out, reach = np.array(old, np.float64), 0.0
    hkv = bounds.shape[1]
    g = q.shape[1] // hkv
    scale = k_scale / np.sqrt(q.shape[2])
    for i in range(len(l_q)):
        ids = batch.kv_indices[int(batch.kv_indptr[i]):int(batch.kv_indptr[i + 1])]
        for t in range(int(l_q[i])):
            row = int(batch.qo_indptr[i]) + t
            for h in range(hkv):
                x = q[row, h * g:(h + 1) * g]
                lo, hi = bounds[ids, h, 0], bounds[ids, h, 1]
                y = np.minimum(x, 0) @ lo.T + np.maximum(x, 0) @ hi.T
                if len(ids):
                    reach = max(reach, float(scale * (np.abs(x) @ np.maximum(np.abs(lo), np.abs(hi)).T).max()))
                unseen = np.arange(len(ids)) * batch.page_size > last_key(batch, i, t)
                out[row, h, :len(ids)] = np.where(unseen, -np.inf, scale * y.max(0) if len(ids) else 0.0)
    return out, reach


def select_pages(batch, scores, sink, recent, budget):
    """[total_q, H_kv, budget] int32: page ids in list order, then -1."""
    l_q, _ = lengths(batch)
    out = np.full((*scores.shape[:2], budget), -1, np.int32)
    for i in range(len(l_q)):
        ids = batch.kv_indices[int(batch.kv_indptr[i]):int(batch.kv_indptr[i + 1])]
        for t in range(int(l_q[i])):
            row, n = int(batch.qo_indptr[i]) + t, max(0, last_key(batch, i, t) // batch.page_size + 1)
            for h in range(scores.shape[1]):
                if n <= budget:
                    out[row, h, :n] = ids[:n]
                    continue
                free = np.arange(sink, n - recent)
                w = scores[row, h, free].astype(np.float64)
                nan = np.isnan(w)
                best = free[np.lexsort((free, np.where(nan, 0.0, -w), ~nan))[:budget - sink - recent]]
                out[row, h] = ids[np.sort(np.concatenate([np.arange(sink), best, np.arange(n - recent, n)]))]
    return out


def pages_attention(batch, q, k_pages, v_pages, selected, cap=0.0, layout="HND"):
    """(o, lse, spread, reach) of every query row over its own list of pages."""
    l_q, _ = lengths(batch)
    hkv = selected.shape[1]
    g = q.shape[1] // hkv
    out = [np.zeros(q.shape), np.full(q.shape[:2], -np.inf), np.zeros(q.shape), np.zeros(q.shape[:2])]
    for i in range(len(l_q)):
        ids = batch.kv_indices[int(batch.kv_indptr[i]):int(batch.kv_indptr[i + 1])]
        for t in range(int(l_q[i])):
            row, last = int(batch.qo_indptr[i]) + t, last_key(batch, i, t)
            for h in range(hkv):
                k, v = [], []
                for p in selected[row, h]:
                    if p < 0 or last < 0:
                        break
                    used = last % batch.page_size + 1 if p == ids[last // batch.page_size] else batch.page_size
                    for dst, src in ((k, k_pages), (v, v_pages)):
                        dst.append(src[p, h, :used] if layout == "HND" else src[p, :used, h])
                if not k:
                    continue
                k, v = np.concatenate(k), np.concatenate(v)
                for a, b in zip(out, state(q[row, h * g:(h + 1) * g], k, v, np.ones((g, len(k)), bool), cap)):
                    a[row, h * g:(h + 1) * g] = b
    return out
