"""GPU parity of the cache operators (append, key weights, selection, compaction) against the float64 oracle."""
import dataclasses

import numpy as np
import pytest

from oracle import attention as A
from oracle import cache as C
from serving_attention_plan_gb300 import workloads as W

from .gpu_helpers import torch_mod

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from serving_attention_plan_gb300 import build
    build.build()
    assert torch_mod().cuda.is_available()


def bf16(bits):
    torch = torch_mod()
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def dev(a):
    return torch_mod().from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def bits(t):
    return t.view(torch_mod().int16).cpu().numpy().view(np.uint16)


def batch_of(lq, lkv, hq, hk, ps, causal=False, seed=0, extra=3, scale=1.0):
    rng = np.random.default_rng(seed)
    n = sum(-(-x // ps) for x in lkv)
    return W.make_paged_batch(rng, "cache", lq, lkv, hq, hk, ps, causal, pool_pages=n + extra, scale=scale)


def as_layout(a, layout):
    return a if layout == "HND" else np.ascontiguousarray(a.transpose(0, 2, 1, 3))


def workspace(b, window=-1, cap=0.0, layout="HND", dtype="bf16", scales=(1.0, 1.0), num_sms=0):
    from serving_attention_plan_gb300 import binding as B
    ws = B.Workspace(max(b.batch_size, 1), max(b.total_q, 1), max(int(b.kv_indptr[-1]), 1), b.num_qo_heads,
                     b.num_kv_heads, 128, num_sms)
    ws.set_variant(window, cap, layout)
    ws.set_kv_dtype(dtype, *scales)
    ws.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, b.page_size, b.causal)
    return ws


# ---- append ----------------------------------------------------------------------------------------

APPEND = [
    # lq, lkv, hq, hk, page, dtype, layout, rotary, interleaved, norm, fused, first position
    ([1], [1], 1, 1, 1, "bf16", "HND", 128, False, True, False, 0),
    ([1, 1, 1, 1], [37, 128, 255, 512], 8, 2, 16, "bf16", "HND", 128, False, True, True, 0),
    ([1, 0, 2, 1], [5, 9, 2, 300], 4, 4, 5, "bf16", "HND", 64, True, True, True, 1_000_003),
    ([33, 0, 129, 5], [33, 4, 500, 3], 12, 4, 8, "bf16", "NHD", 96, False, False, True, 100_000),
    ([70, 1], [70, 65], 40, 8, 64, "e4m3", "NHD", 32, True, True, False, 7),
    ([17, 40], [20, 41], 16, 1, 32, "e4m3", "HND", 16, False, False, True, 131_071),
    ([9] * 150, [9] * 150, 8, 8, 16, "bf16", "HND", 128, True, False, True, 5),   # four tokens a step, odd batches
    ([300, 961], [300, 1000], 16, 8, 16, "bf16", "HND", 0, False, True, True, 0),
    ([1300, 11], [1300, 11], 2, 2, 128, "e4m3", "NHD", 112, False, True, True, 2_000_000_000),
]


@pytest.mark.parametrize("case", APPEND, ids=range(len(APPEND)))
def test_append(case):
    torch = torch_mod()
    lq, lkv, hq, hk, ps, dtype, layout, rotary, inter, norm, fused, first = case
    b = batch_of(lq, lkv, hq, hk, ps, False, seed=len(lq) + ps)
    rng = np.random.default_rng(11)
    n = b.total_q
    x = rng.standard_normal((n, hq + 2 * hk, 128)).astype(np.float32) * 2
    raw = bf16(W.f32_to_bf16_bits(x))
    x = f64(raw)
    q, k, v = raw[:, :hq], raw[:, hq:hq + hk], raw[:, hq + hk:]
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    wq, wk = (bf16(W.f32_to_bf16_bits(1 + 0.3 * rng.standard_normal(128).astype(np.float32))) for _ in range(2))
    inv_freq = 10000.0 ** (-np.arange(0, rotary, 2) / max(rotary, 1))
    tok, page, slot, key = C.append_places(b)
    positions = key + first
    scales = (0.03125, 0.0625) if dtype == "e4m3" else (1.0, 1.0)
    ws = workspace(b, layout=layout, dtype=dtype, scales=scales)
    ws.set_rope(inv_freq, inter)
    if dtype == "bf16":
        k0, v0 = as_layout(b.k_pages, layout), as_layout(b.v_pages, layout)
        kp, vp = bf16(k0), bf16(v0)
    else:
        k0, v0 = (as_layout(rng.integers(0, 127, size=b.k_pages.shape).astype(np.uint8), layout) for _ in range(2))
        kp, vp = dev(k0), dev(v0)
    out = torch.full((n, hq, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws.append(q, k, v, kp, vp, out, wq if norm else None, wk if norm else None, 1e-5,
              dev(positions.astype(np.int32)) if first else None)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    rq = C.norm_rotate(x[:, :hq], f64(wq) if norm else None, 1e-5, inv_freq, positions.astype(np.float64), inter)
    rk = C.norm_rotate(x[:, hq:hq + hk], f64(wk) if norm else None, 1e-5, inv_freq, positions.astype(np.float64), inter)
    rv = x[:, hq + hk:]
    # fp32 steps before the rounding: a dozen of half a unit each of values up to the row's largest, and the
    # angle (2^-25 turns after the fp32 rounding of the fraction): 2^-19 of the row's largest covers both
    slack = lambda r: np.abs(r).max(-1, keepdims=True) * 2.0 ** -19
    assert (np.abs(f64(out) - rq) <= np.abs(rq) * 2.0 ** -8 + slack(rq)).all()
    for got, before, ref, scale in ((kp, k0, rk, scales[0]), (vp, v0, rv, scales[1])):
        host = bits(got) if dtype == "bf16" else got.cpu().numpy()
        rows = host[page, :, slot] if layout == "HND" else host[page, slot]
        ref = ref[tok]
        if dtype == "bf16":
            assert (np.abs(A.bf16_to_f64(rows) - ref) <= np.abs(ref) * 2.0 ** -8 + slack(ref)).all()
        else:
            lim = np.clip(ref / scale, -448, 448)
            # half a step: 2^-4 of a normal value, 2^-10 below the smallest normal
            assert (np.abs(A.e4m3_to_f64(rows) - lim) <= np.maximum(np.abs(lim) * 2.0 ** -4, 2.0 ** -10) + slack(ref) / scale).all()
        # every other slot is as it was
        rest = np.ones(host.shape[:1] + (ps,), bool)
        rest[page, slot] = False
        a, z = (host.transpose(0, 2, 1, 3), before.transpose(0, 2, 1, 3)) if layout == "HND" else (host, before)
        assert np.array_equal(a[rest], z[rest])


def test_append_in_place_q_and_saturation():
    """q_out is q; e4m3 saturates at +-448 and infinities with it; NaN becomes the NaN code; -0 and denormal inputs pass."""
    torch = torch_mod()
    b = batch_of([1, 1], [4, 7], 2, 1, 4)
    ws = workspace(b, dtype="e4m3", scales=(1.0, 1.0))
    q = torch.randn(2, 2, 128, device="cuda").to(torch.bfloat16)
    want = q.clone()
    k = torch.zeros(2, 1, 128, device="cuda", dtype=torch.bfloat16)
    k[0, 0, :6] = torch.tensor([1e30, -1e30, float("inf"), -float("inf"), float("nan"), -0.0])
    kp, vp = (torch.zeros(b.num_pages, 1, 4, 128, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ws.append(q, k, k, kp, vp, q)
    torch.cuda.synchronize()
    assert torch.equal(q, want)
    _, page, slot, _ = C.append_places(b)
    row = kp[page[0], 0, slot[0]].float().cpu()
    assert row[:4].tolist() == [448, -448, 448, -448] and torch.isnan(row[4]) and row[5] == 0 and torch.signbit(row[5])
    assert torch.equal(kp.view(torch.uint8), vp.view(torch.uint8))


# ---- key weights -----------------------------------------------------------------------------------

WEIGHTS = [
    # lq, lkv, hq, hk, page, causal, dtype, layout, window, cap, decay, new keys, SM budget
    ([1], [1], 1, 1, 1, False, "bf16", "HND", -1, 0.0, 1.0, True, 0),
    ([1] * 4, [37, 128, 255, 512], 8, 2, 16, False, "bf16", "HND", -1, 0.0, 0.9, False, 0),
    ([1, 0, 1, 2], [33, 64, 0, 700], 16, 4, 5, True, "bf16", "HND", -1, 0.0, 0.5, True, 1),
    ([1, 1], [900, 31], 64, 8, 1, False, "e4m3", "HND", -1, 30.0, 0.0, True, 3),
    ([2, 1], [300, 257], 20, 5, 4, True, "bf16", "HND", 40, 0.0, 0.75, True, 0),
    ([1, 1, 1], [32, 63, 65], 6, 2, 8, False, "e4m3", "NHD", -1, 0.0, 1.0, True, 0),
    ([17, 40, 0], [17, 300, 5], 8, 2, 16, True, "bf16", "HND", -1, 0.0, 0.9, True, 0),
    ([130, 1], [130, 700], 32, 8, 16, True, "bf16", "NHD", -1, 0.0, 1.0, False, 5),
    ([257, 9], [513, 9], 10, 2, 32, True, "e4m3", "HND", -1, 20.0, 0.3, True, 0),
    ([200, 64], [600, 64], 12, 4, 8, True, "bf16", "HND", 128, 5.0, 1.0, True, 2),
    ([40, 20], [10, 300], 8, 8, 64, True, "bf16", "HND", -1, 0.0, 0.9, True, 0),   # rows that see no key
    ([66, 3], [200, 129], 16, 16, 128, False, "e4m3", "NHD", -1, 0.0, 0.9, False, 0),
    ([5, 9], [290, 70], 130, 1, 16, True, "bf16", "HND", -1, 0.0, 1.0, True, 0),   # 130 heads a group
    ([520], [1100], 4, 1, 16, True, "bf16", "HND", -1, 0.0, 1.0, True, 0),
    # row counts around the limit between the two kernels, in one batch with long ones and empty ones
    ([8, 9, 1, 0, 300, 7, 2], [700, 70, 513, 40, 400, 7, 1000], 16, 4, 16, True, "bf16", "HND", -1, 0.0, 0.9, True, 0),
    ([16, 17, 1, 0, 90, 33], [700, 70, 513, 40, 400, 290], 16, 4, 16, True, "e4m3", "NHD", 60, 10.0, 0.9, True, 3),
]


def lse_of(b, q, kp, k_scale, window, cap, layout):
    """float32 log-sum-exp per row, from the definition."""
    l_q, l_kv = C.lengths(b)
    g = b.num_qo_heads // b.num_kv_heads
    lse = np.full((b.total_q, b.num_qo_heads), -np.inf)
    for i in range(b.batch_size):
        n, t = int(l_kv[i]), int(l_q[i])
        if n == 0 or t == 0:
            continue
        rows = slice(int(b.qo_indptr[i]), int(b.qo_indptr[i]) + t)
        pos, j = n - t + np.arange(t)[:, None], np.arange(n)[None, :]
        seen = (j <= pos) & ((j >= pos - window) | (window < 0)) if b.causal else np.ones((t, n), bool)
        for h in range(b.num_qo_heads):
            x = q[rows, h] @ (A.gather_kv(kp, b.kv_indptr, b.kv_indices, n, b.page_size, i, h // g, layout) * k_scale).T
            x /= np.sqrt(128)
            x = cap * np.tanh(x / cap) if cap else x
            with np.errstate(divide="ignore"):
                lse[rows, h] = np.log(np.where(seen, np.exp(x), 0).sum(1))
    return lse.astype(np.float32)


def weights_case(case, seed=5):
    lq, lkv, hq, hk, ps, causal, dtype, layout, window, cap, decay, new, sms = case
    b = batch_of(lq, lkv, hq, hk, ps, causal, seed=seed, scale=1.3)
    rng = np.random.default_rng(3)
    k_scale = 0.03125 if dtype == "e4m3" else 1.0
    k = b.k_pages if dtype == "bf16" else W.to_e4m3(A.bf16_to_f64(b.k_pages) / k_scale)
    k = as_layout(k, layout)
    q = A.bf16_to_f64(b.q)
    lse = lse_of(b, q, k, k_scale, window, cap, layout)
    old = rng.random((b.num_pages, hk, ps)).astype(np.float32) * 3
    return b, q, k, k_scale, lse, old


def weights_tol(reach, lse):
    """Relative error of one term: the logit's fp32 sum (128 products, each sum up to a unit in the last place of the
    largest partial sum), the exponent's own roundings and the exponential (2^-21)."""
    big = float(np.abs(np.where(np.isfinite(lse), lse, 0)).max(initial=0.0))
    return reach * 128 * 2.0 ** -23 + (reach + big) * 2.0 ** -21 + 2.0 ** -20


@pytest.mark.parametrize("case", WEIGHTS, ids=range(len(WEIGHTS)))
def test_key_weights(case):
    torch = torch_mod()
    lq, lkv, hq, hk, ps, causal, dtype, layout, window, cap, decay, new, sms = case
    b, q, k, k_scale, lse, old = weights_case(case)
    # what must not be read: new keys' former sums (with new_keys), slots no key has, with NaN in both
    _, l_kv = C.lengths(b)
    l_q, _ = C.lengths(b)
    used = np.zeros((b.num_pages, ps), bool)
    start = old.copy()
    for i in range(b.batch_size):
        p, s = C.places(b, i, np.arange(int(l_kv[i])))
        used[p, s] = True
        if new:
            p, s = C.places(b, i, np.arange(max(0, int(l_kv[i] - l_q[i])), int(l_kv[i])))
            start[p, :, s] = np.nan
    start.transpose(0, 2, 1)[~used] = np.nan
    if decay == 0.0:
        start[:] = np.nan
    k = k.copy()
    nan = 0x7FFF if dtype == "bf16" else 0x7F
    (k.transpose(0, 2, 1, 3) if layout == "HND" else k)[~used] = nan
    ws = workspace(b, window, cap, layout, dtype, (k_scale, 1.0), sms)
    w = dev(start)
    kd = bf16(k) if dtype == "bf16" else dev(k)
    ws.key_weights(bf16(b.q), kd, dev(lse), w, decay, new)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    ref, reach = C.key_weights(b, q, k, lse, old, decay, new, k_scale, window, cap, layout)
    got = w.cpu().numpy()
    assert np.isnan(got.transpose(0, 2, 1)[~used]).all()
    g, r = got.transpose(0, 2, 1)[used].astype(np.float64), ref.transpose(0, 2, 1)[used]
    tol = weights_tol(reach, lse)
    # sums of n terms in fp32: n / 2 half units more at the very worst order
    n = max(lq) * (hq // hk)
    assert (np.abs(g - r) <= r * (tol + n * 2.0 ** -24) + 1e-30).all(), (np.abs(g - r) / np.maximum(r, 1e-30)).max()


def test_key_weights_masked_rows_and_infinities():
    """A row with lse = -inf adds nothing even with NaN in its q; NaN in another request's q or in keys a row does not
    see stays there; a key of infinities poisons only its own sum."""
    torch = torch_mod()
    b = batch_of([20, 20], [40, 90], 8, 2, 16, True, scale=1.0)
    q = A.bf16_to_f64(b.q)
    lse = lse_of(b, q, b.k_pages, 1.0, -1, 0.0, "HND")
    old = np.zeros((b.num_pages, 2, 16), np.float32)
    ref, reach = C.key_weights(b, q, b.k_pages, np.where(np.arange(40)[:, None] == 3, -np.inf, lse), old, 1.0, True)
    bad_q = b.q.copy()
    bad_q[20:] = 0x7FC0  # the second request: NaN
    bad_q[3] = 0x7FC0
    lse_dev = lse.copy()
    lse_dev[3] = -np.inf
    k = b.k_pages.copy()
    p, s = C.places(b, 0, [39])  # the first request's last key: seen by its last token alone
    k[p, :, s] = 0x7F80          # +inf
    ws = workspace(b)
    w = dev(old)
    ws.key_weights(bf16(bad_q), bf16(k), dev(lse_dev), w, 1.0, True)
    torch.cuda.synchronize()
    got = w.cpu().numpy()
    p, s = C.places(b, 0, np.arange(39))
    tol = weights_tol(reach, lse) + 80 * 2.0 ** -24
    assert (np.abs(got[p, :, s] - ref[p, :, s]) <= ref[p, :, s] * tol + 1e-30).all()
    p, s = C.places(b, 1, np.arange(90))
    assert np.isnan(got[p, :, s]).all()



def exact_case(lq, lkv, hq, hk, dtype, gain, seed=7):
    """q and K of few significant bits: multiples of gain / 8 and 1 / 8 up to 15 / 8, so that products and their sums
    (below 2^15 units) are exact in every type and order, and a weight's error is that of its exponential, its tanh and its sum."""
    b = batch_of(lq, lkv, hq, hk, 16, True, seed=seed)
    rng = np.random.default_rng(seed)
    q = rng.integers(-15, 16, size=b.q.shape) * (gain / 8)
    k = rng.integers(-15, 16, size=b.k_pages.shape) / 8
    qb = W.f32_to_bf16_bits(q.astype(np.float32))
    kb = W.f32_to_bf16_bits(k.astype(np.float32)) if dtype == "bf16" else W.to_e4m3(k)
    back = A.bf16_to_f64(kb) if dtype == "bf16" else A.e4m3_to_f64(kb)
    assert np.array_equal(A.bf16_to_f64(qb), q) and np.array_equal(back, k)
    return dataclasses.replace(b, q=qb), q, kb


@pytest.mark.parametrize("cap,gain", [(0.0, 1), (0.0, 8), (2.0, 1), (5.0, 1), (30.0, 1), (30.0, 4), (64.0, 8), (65.0, 8), (100.0, 8), (1e4, 1), (1e4, 8),
                                      (1e6, 1), (1e30, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lq,lkv", [([1, 1, 2], [300, 77, 512]), ([70, 130], [300, 600])], ids=["rows", "tiles"])
def test_key_weights_of_exact_products(lq, lkv, dtype, cap, gain):
    """Soft-caps from saturation to none at all, on both sides of where the tanh changes its form, at a bound that a
    coarser exponential or tanh would miss."""
    torch = torch_mod()
    hq, hk = 8, 2
    b, q, k = exact_case(lq, lkv, hq, hk, dtype, gain)
    lse = lse_of(b, q, k, 1.0, -1, cap, "HND")
    ws = workspace(b, cap=cap, dtype=dtype)
    w = torch.zeros(b.num_pages, hk, 16, device="cuda")
    ws.key_weights(bf16(b.q), bf16(k) if dtype == "bf16" else dev(k), dev(lse), w, 0.0, True)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    ref, _ = C.key_weights(b, q, k, lse, np.zeros(w.shape), 0.0, True, cap=cap)
    # largest |logit| before and after the cap and largest |lse|, in powers of two
    keys = [A.gather_kv(k, b.kv_indptr, b.kv_indices, n, 16, i, h, "HND") for i, n in enumerate(lkv) for h in range(hk)]
    raw = max(float(np.abs(q[int(b.qo_indptr[i // hk]):int(b.qo_indptr[i // hk + 1]), 4 * (i % hk):4 * (i % hk) + 4] @ x.T).max())
              for i, x in enumerate(keys)) / np.sqrt(128)
    x2 = (cap * np.tanh(raw / cap) if cap else raw) / np.log(2)
    l2 = float(np.abs(lse[np.isfinite(lse)]).max()) / np.log(2)
    unit = 2.0 ** -24
    # error of the exponent: -lse in powers of two (constant, product), the last sum, and the logit:
    steps = 2 * l2 + (x2 + l2)
    if not cap:
        steps += 4 * x2  # log2 e, the root, their quotient, the product
    elif cap <= 64:
        # tanh by exponentials: at most 2^-21 (2^-22 of its exponential, 2^-23 of the reciprocal, twice); its argument's eight
        # roundings times y (1 - tanh(y)^2) < 0.45; the cap's own two and the product
        steps += cap / np.log(2) * (8 + 8 * 0.45) + 3 * x2
    else:
        # relative: sixteen roundings through the series; by exponentials 2^-21 of at least 0.244
        steps += x2 * (16 if raw <= cap / 4 else 48)
    n = max(lq) * (hq // hk) + 16  # additions of one sum
    tol = np.log(2) * steps * unit + 2.0 ** -22 + n * unit
    got = w.cpu().numpy().astype(np.float64)
    assert (np.abs(got - ref) <= ref * tol + 1e-30).all(), (float((np.abs(got - ref) / np.maximum(ref, 1e-30)).max()), tol)


# ---- selection -------------------------------------------------------------------------------------

SELECT = [
    # lkv, hk, page, budget, recent, sink, kind, SM budget
    ([1], 1, 1, 1, 0, 0, "random", 0),
    ([5, 0, 8, 9], 3, 4, 8, 2, 1, "random", 0),
    ([100, 33, 700], 2, 16, 32, 32, 0, "random", 0),      # nothing but recent keys
    ([100, 33, 700], 2, 16, 33, 0, 33, "equal", 1),       # nothing but sinks
    ([1000, 513], 8, 5, 257, 31, 4, "ties", 0),
    ([4000], 2, 16, 3999, 0, 0, "equal", 0),              # one key goes
    ([20000], 1, 16, 1, 0, 0, "random", 0),               # a cluster shares the row
    ([40001, 12], 3, 1, 20000, 100, 4, "ties", 0),
    ([300000], 1, 64, 1000, 10, 4, "random", 0),          # slices longer than shared memory at 8 CTAs: 37.5 K each
    ([450000], 1, 128, 400, 0, 0, "ties", 0),             # 56 K keys a slice: read again from memory
    ([60000, 100, 59999] * 4, 8, 64, 9000, 64, 4, "random", 0),  # many rows, each too long for one CTA's shared memory
    ([64] * 40, 8, 16, 20, 5, 2, "signs", 2),
    ([777] * 3, 2, 8, 100, 7, 3, "special", 0),
]


def some_weights(rng, shape, kind):
    if kind == "equal":
        return np.full(shape, 0.25, np.float32)
    if kind == "ties":
        return rng.integers(0, 4, size=shape).astype(np.float32)
    if kind == "signs":
        return rng.standard_normal(shape).astype(np.float32).round(1)
    w = np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    if kind == "special":
        w = np.where(rng.random(shape) < 0.3, rng.choice(np.array([0.0, -0.0, np.inf, -np.inf, np.nan, 1e-45, -1e-45, 3e38], np.float32), shape), w)
    return w.astype(np.float32)


@pytest.mark.parametrize("case", SELECT, ids=range(len(SELECT)))
def test_select_keys(case):
    torch = torch_mod()
    lkv, hk, ps, budget, recent, sink, kind, sms = case
    rng = np.random.default_rng(9)
    b = W.make_paged_batch(rng, "select", [1] * len(lkv), lkv, hk, hk, ps, False, with_data=False)
    w = some_weights(rng, (max(b.num_pages, 1), hk, ps), kind)
    _, l_kv = C.lengths(b)
    used = np.zeros((w.shape[0], ps), bool)
    for i in range(b.batch_size):
        p, s = C.places(b, i, np.arange(int(l_kv[i])))
        used[p, s] = True
    w.transpose(0, 2, 1)[~used] = np.nan  # slots behind the last key are not read
    ws = workspace(b, num_sms=sms)
    kept = torch.full((b.batch_size, hk, budget), -7, dtype=torch.int32, device="cuda")
    ws.select_keys(dev(w), budget, kept, recent=recent, sink=sink)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    assert np.array_equal(kept.cpu().numpy(), C.select(b, w, budget, recent, sink))


# lkv, hk, page, budget, recent, sink, kind, SM budget, share of the free keys' pages that lie outside the pool
OUTSIDE = [
    ([100, 33, 700, 64], 2, 4, 32, 8, 2, "random", 1, 0.95),   # rows one after another in a CTA
    ([1000, 513], 2, 5, 257, 31, 4, "ties", 0, 0.9),           # one weight a load
    ([1000, 900], 2, 16, 500, 0, 0, "random", 0, 1.0),         # nothing left
    ([20000, 18000], 1, 16, 5000, 100, 4, "random", 0, 0.9),   # a cluster shares the row
    ([450000], 1, 128, 4000, 50, 0, "special", 0, 0.995),      # slices that are read again from memory
    ([3000, 2000], 4, 16, 300, 20, 4, "random", 0, 0.3),       # enough keys are left
]


@pytest.mark.parametrize("case", OUTSIDE, ids=range(len(OUTSIDE)))
def test_replayed_selection_with_pages_outside_the_pool(case):
    """A replay whose plan lists pages that the captured pool does not have: their keys are left out, the error bit is set,
    every entry of kept is written and nothing beside it is."""
    from serving_attention_plan_gb300 import binding as B
    torch = torch_mod()
    lkv, hk, ps, budget, recent, sink, kind, sms, share = case
    rng = np.random.default_rng(12)
    b = W.make_paged_batch(rng, "select", [1] * len(lkv), lkv, hk, hk, ps, False, with_data=False)
    w = some_weights(rng, (b.num_pages, hk, ps), kind)
    ws = workspace(b, num_sms=sms)
    guard, n_kept = 256, b.batch_size * hk * budget
    flat = torch.full((n_kept + 2 * guard,), -7, dtype=torch.int32, device="cuda")
    kept = flat[guard:guard + n_kept].view(b.batch_size, hk, budget)
    wd, side = dev(w), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ws.select_keys(wd, budget, kept, recent=recent, sink=sink, stream=side)
    lost = rng.random(b.kv_indices.shape[0]) < share
    idx = np.where(lost, b.kv_indices + b.num_pages, b.kv_indices).astype(np.int32)
    ws.plan(b.qo_indptr, b.kv_indptr, idx, b.last_page_len, ps, False, stream=side)
    for _ in range(2):
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert ws.get_error() == B.DEVERR_PAGE_OOB
    want = np.full((b.batch_size, hk, budget), -1, np.int32)
    for i, n in enumerate(lkv):
        j = np.arange(n)
        gone = lost[int(b.kv_indptr[i]) + j // ps]
        page, slot = C.places(b, i, j)
        for h in range(hk):
            free = np.arange(sink, n - recent)
            free = free[~gone[free]]
            x = w[page[free], h, slot[free]].astype(np.float64)
            order = np.lexsort((free, np.where(np.isnan(x), 0.0, -x), ~np.isnan(x)))[:budget - sink - recent]
            row = np.concatenate([j[:sink], np.sort(free[order]), j[n - recent:]]) if n > budget else j
            want[i, h, :len(row)] = row
    got = flat.cpu().numpy()
    assert np.array_equal(got[guard:guard + n_kept].reshape(want.shape), want)
    assert (got[:guard] == -7).all() and (got[guard + n_kept:] == -7).all()



def test_select_keys_largest_budget():
    """A budget of 2^31 - 1, far beyond the request: the keys, then -1 to the last entry, nothing beside them."""
    torch = torch_mod()
    budget, guard = 2**31 - 1, 1024
    b = batch_of([1], [5], 1, 1, 4)
    ws = workspace(b)
    flat = torch.full((budget + 2 * guard,), -7, dtype=torch.int32, device="cuda")
    kept = flat[guard:guard + budget].view(1, 1, budget)
    ws.select_keys(torch.zeros(b.num_pages, 1, 4, device="cuda"), budget, kept, recent=3, sink=1)
    torch.cuda.synchronize()
    assert ws.get_error() == 0 and kept[0, 0, :5].tolist() == [0, 1, 2, 3, 4]
    assert int(kept.min()) == -1 and int(kept[0, 0, 5:].max()) == -1
    assert (flat[:guard] == -7).all() and (flat[guard + budget:] == -7).all()


# ---- compaction ------------------------------------------------------------------------------------

COMPACT = [
    # lkv, hk, page, budget, dtype, layout, weights, pick
    ([1], 1, 1, 1, "bf16", "HND", True, "random"),
    ([9, 3, 0, 40], 2, 4, 8, "bf16", "HND", True, "random"),
    ([700, 650, 333], 3, 5, 300, "bf16", "HND", False, "random"),
    ([1000, 129], 8, 16, 128, "e4m3", "NHD", True, "random"),
    ([2000], 1, 1, 1999, "bf16", "HND", True, "drop first"),   # every row moves down by one slot
    ([3000, 2999], 2, 16, 2500, "e4m3", "HND", True, "drop first"),
    ([9000], 2, 64, 8000, "bf16", "NHD", True, "random"),
    ([600], 4, 16, 500, "bf16", "HND", True, "front"),         # nothing moves
    ([600], 4, 16, 7, "e4m3", "HND", True, "back"),
]


@pytest.mark.parametrize("case", COMPACT, ids=range(len(COMPACT)))
def test_compact(case):
    torch = torch_mod()
    lkv, hk, ps, budget, dtype, layout, with_w, pick = case
    rng = np.random.default_rng(4)
    b = W.make_paged_batch(rng, "compact", [1] * len(lkv), lkv, hk, hk, ps, False, with_data=False, pool_pages=None)
    shape = (max(b.num_pages, 1), hk, ps, 128)
    kind = np.uint16 if dtype == "bf16" else np.uint8
    k, v = (as_layout(rng.integers(0, np.iinfo(kind).max, size=shape, endpoint=True).astype(kind), layout) for _ in range(2))
    w = rng.random(shape[:3]).astype(np.float32)
    kept = np.full((len(lkv), hk, budget), -1, np.int32)
    for i, n in enumerate(lkv):
        for h in range(hk):
            m = min(n, budget)
            kept[i, h, :m] = {"random": lambda: np.sort(rng.choice(n, m, replace=False)), "front": lambda: np.arange(m),
                              "back": lambda: np.arange(n - m, n), "drop first": lambda: np.arange(n - m, n)}[pick]()
    ws = workspace(b, layout=layout, dtype=dtype)
    kd, vd = (bf16(k), bf16(v)) if dtype == "bf16" else (dev(k), dev(v))
    wd = dev(w)
    ws.compact(dev(kept), kd, vd, wd if with_w else None)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    rk, rv, rw = C.compact(b, kept, [k, v, w], [layout, layout, "HND"])
    host = (lambda t: bits(t)) if dtype == "bf16" else (lambda t: t.cpu().numpy())
    assert np.array_equal(host(kd), rk) and np.array_equal(host(vd), rv)
    assert np.array_equal(wd.cpu().numpy(), rw if with_w else w)


def test_compact_skips_bad_entries():
    """Entries out of range or out of order are skipped and reported; the others move."""
    from serving_attention_plan_gb300 import binding as B
    torch = torch_mod()
    b = batch_of([1], [20], 1, 1, 4)
    ws = workspace(b)
    kept = np.array([[[0, 5, 5, 20, 2**30, 19]]], np.int32)  # ok, ok, not above, out of range (2), ok only if ascending
    k, v = bf16(b.k_pages), bf16(b.v_pages)
    ws.compact(dev(kept), k, v)
    torch.cuda.synchronize()
    assert ws.get_error() == B.DEVERR_KEPT
    want = b.k_pages.copy()
    fp, fs = C.places(b, 0, [5])
    tp, ts = C.places(b, 0, [1])
    want[tp, :, ts] = b.k_pages[fp, :, fs]
    assert np.array_equal(bits(k), want)
    kept = np.array([[[-1, 1, 3, 4, 6, 7]]], np.int32)
    ws.compact(dev(kept), k, v)
    torch.cuda.synchronize()
    assert ws.get_error() == B.DEVERR_KEPT


# ---- together --------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype,layout,causal_chunk", [("bf16", "HND", False), ("e4m3", "NHD", False), ("bf16", "HND", True)])
def test_life_of_a_cache(dtype, layout, causal_chunk):
    """Prompt, decode steps, eviction, more decode steps: the attention over the evicted cache is the oracle's over the
    rows that the oracle's own selection keeps."""
    from serving_attention_plan_gb300 import binding as B
    torch = torch_mod()
    rng = np.random.default_rng(21)
    hq, hk, ps, budget, recent, sink = 8, 2, 16, 48, 8, 2
    prompts = [100, 37, 260]
    n_req, steps, pool = 3, 4, 64
    free = list(rng.permutation(pool))
    lists = [[] for _ in range(n_req)]
    length, position = [0] * n_req, [0] * n_req
    scales = (0.0625, 0.0625) if dtype == "e4m3" else (1.0, 1.0)
    inv_freq = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    ws = B.Workspace(n_req, 1024, pool, hq, hk)
    ws.set_variant(kv_layout=layout)
    ws.set_kv_dtype(dtype, *scales)
    ws.set_rope(inv_freq)
    t = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    shape = (pool, hk, ps, 128) if layout == "HND" else (pool, ps, hk, 128)
    kp, vp = torch.zeros(shape, device="cuda", dtype=t), torch.zeros(shape, device="cuda", dtype=t)
    w = torch.full((pool, hk, ps), float("nan"), device="cuda")
    raw = (lambda x: bits(x)) if dtype == "bf16" else (lambda x: x.view(torch.uint8).cpu().numpy())

    def step(new):
        nonlocal lists
        for i in range(n_req):
            length[i] += new[i]
            while len(lists[i]) * ps < length[i]:
                lists[i].append(free.pop())
        qo = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        kv = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
        last = np.array([length[i] - (len(lists[i]) - 1) * ps for i in range(n_req)], np.int32)
        b = W.PagedBatch("life", hq, hk, 128, ps, True, qo, kv, np.concatenate(lists).astype(np.int32), last, None, None, None)
        ws.plan(qo, kv, b.kv_indices, last, ps, True)
        n = int(qo[-1])
        x = bf16(W.f32_to_bf16_bits(rng.standard_normal((n, hq + 2 * hk, 128), dtype=np.float32)))
        pos = np.concatenate([np.arange(position[i], position[i] + new[i]) for i in range(n_req)])
        for i in range(n_req):
            position[i] += new[i]
        q = torch.empty(n, hq, 128, device="cuda", dtype=torch.bfloat16)
        o, lse = torch.empty_like(q), torch.empty(n, hq, device="cuda")
        ws.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], kp, vp, q, positions=dev(pos.astype(np.int32)))
        ws.run(q, kp, vp, o, lse)
        ws.key_weights(q, kp, lse, w, decay=0.9)
        torch.cuda.synchronize()
        assert ws.get_error() == 0
        b = dataclasses.replace(b, q=bits(q), k_pages=raw(kp), v_pages=raw(vp))
        ro, rl = A.batch_attention(b, layout=layout, k_scale=scales[0], v_scale=scales[1])
        assert np.abs(f64(o) - ro).max() <= 2e-2 and np.abs(f64(lse) - rl).max() <= 1e-3 * max(1, np.abs(rl).max())
        return b, f64(q), lse.cpu().numpy()

    want = np.zeros((pool, hk, ps))
    for k_step in range(steps):
        new = prompts if k_step == 0 else ([20, 1, 33] if causal_chunk else [1] * n_req)
        b, q, lse = step(new)
        want, reach = C.key_weights(b, q, b.k_pages, lse, want, 0.9, True, scales[0], layout=layout)
        got = w.cpu().numpy()
        tol = weights_tol(reach, lse) + 1024 * 2.0 ** -24
        for i in range(n_req):
            p, s = C.places(b, i, np.arange(length[i]))
            assert (np.abs(got[p, :, s] - want[p, :, s]) <= (k_step + 1) * tol * want[p, :, s] + 1e-30).all()
            want[p, :, s] = got[p, :, s]
            # every row spreads a weight of one over its keys
        if k_step % 2 == 1:
            kept = torch.empty(n_req, hk, budget, device="cuda", dtype=torch.int32)
            ws.select_keys(w, budget, kept, recent=recent, sink=sink)
            ws.compact(kept, kp, vp, w)
            torch.cuda.synchronize()
            assert ws.get_error() == 0
            rkept = C.select(b, got, budget, recent, sink)
            assert np.array_equal(kept.cpu().numpy(), rkept)
            rk, rv, rw = C.compact(b, rkept, [b.k_pages, b.v_pages, got], [layout, layout, "HND"])
            assert np.array_equal(raw(kp), rk) and np.array_equal(raw(vp), rv)
            assert np.array_equal(w.cpu().numpy(), rw, equal_nan=True)
            want = rw.astype(np.float64)
            for i in range(n_req):
                length[i] = min(length[i], budget)
                keep = -(-length[i] // ps)
                free.extend(lists[i][keep:])
                lists[i] = lists[i][:keep]


def test_captured_chain_follows_a_new_plan():
    """append, run, key_weights, select and compact captured once: a replay after another plan of the same path does what
    separate calls do, on a side stream, twice over."""
    torch = torch_mod()
    hq, hk, ps, budget = 8, 2, 16, 100

    def one(lkv, seed):
        b = batch_of([1] * len(lkv), lkv, hq, hk, ps, True, seed=seed, extra=60 - sum(-(-x // ps) for x in lkv))
        return b
    first, second = one([130, 90, 20], 1), one([220, 31, 300, 101], 2)
    from serving_attention_plan_gb300 import binding as B
    ws = B.Workspace(4, 4, 60, hq, hk)
    ws.set_rope(10000.0 ** (-np.arange(0, 128, 2) / 128))
    side = torch.cuda.Stream()
    x = torch.randn(4, hq + 2 * hk, 128, device="cuda").to(torch.bfloat16)
    kp0, vp0 = bf16(first.k_pages), bf16(first.v_pages)
    w0 = torch.rand(60, hk, ps, device="cuda")

    def buffers():
        return dict(kp=kp0.clone(), vp=vp0.clone(), w=w0.clone(), q=torch.zeros(4, hq, 128, device="cuda", dtype=torch.bfloat16),
                    o=torch.zeros(4, hq, 128, device="cuda", dtype=torch.bfloat16), lse=torch.zeros(4, hq, device="cuda"),
                    kept=torch.full((4, hk, budget), -9, device="cuda", dtype=torch.int32))

    def plan(b):
        ws.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, ps, True, stream=side)

    def calls(d, n):
        v = lambda t: t[:n]
        ws.append(x[:n, :hq], x[:n, hq:hq + hk], x[:n, hq + hk:], d["kp"], d["vp"], v(d["q"]), stream=side)
        ws.run(v(d["q"]), d["kp"], d["vp"], v(d["o"]), v(d["lse"]), stream=side)
        ws.key_weights(v(d["q"]), d["kp"], v(d["lse"]), d["w"], 0.9, True, stream=side)
        ws.select_keys(d["w"], budget, v(d["kept"]), recent=10, sink=2, stream=side)
        ws.compact(v(d["kept"]), d["kp"], d["vp"], d["w"], stream=side)

    cap = buffers()
    torch.cuda.synchronize()
    plan(first)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(cap, 3)
    for b in (first, second, first):
        for k, val in buffers().items():
            cap[k].copy_(val)
        ref = buffers()
        torch.cuda.synchronize()
        plan(b)
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        calls(ref, b.batch_size)
        side.synchronize()
        assert ws.get_error() == 0
        for k in ref:
            assert torch.equal(ref[k], cap[k]), k



EMPTY_PLANS = {  # what the capture's plan holds: (qo_indptr, kv_indptr, kv_indices, last_page_len), and the later plan's (l_q, l_kv)
    "no requests": (([0], [0], [], []), [1, 1, 1], [130, 90, 20]),
    "no tokens": (([0, 0], [0, 2], [0, 1], [3]), [1, 1, 1], [130, 90, 20]),
    "no keys": (([0, 1, 2, 3], [0, 0, 0, 0], [], [0, 0, 0]), [1, 1, 1], [130, 90, 20]),
    "prompts without keys": (([0, 20, 60], [0, 0, 0], [], [0, 0]), [20, 40], [120, 300]),
}


@pytest.mark.parametrize("which", EMPTY_PLANS)
def test_capture_on_an_empty_plan(which):
    """The operators captured while the plan has no requests, tokens or keys: a replay after a plan that has all of them
    does what direct calls do.  Null pointers are refused then, whatever the plan at hand would excuse."""
    torch = torch_mod()
    from serving_attention_plan_gb300 import binding as B
    L = B.lib()
    empty, lq, lkv = EMPTY_PLANS[which]
    hq, hk, ps, budget = 8, 2, 16, 60
    b = batch_of(lq, lkv, hq, hk, ps, True, seed=3)
    n, rows, pages = b.batch_size, b.total_q, b.num_pages
    ws = B.Workspace(4, 64, 64, hq, hk)
    side = torch.cuda.Stream()
    x = torch.randn(rows, hq + 2 * hk, 128, device="cuda").to(torch.bfloat16)
    lse = dev(lse_of(b, A.bf16_to_f64(b.q), b.k_pages, 1.0, -1, 0.0, "HND"))
    q = bf16(b.q)
    w0 = torch.rand(pages, hk, ps, device="cuda")

    def buffers():
        return dict(kp=bf16(b.k_pages), vp=bf16(b.v_pages), w=w0.clone(), out=torch.zeros(rows, hq, 128, device="cuda", dtype=torch.bfloat16),
                    kept=torch.full((n, hk, budget), -9, device="cuda", dtype=torch.int32))

    cap, ref = buffers(), buffers()
    P = {k: t.data_ptr() for k, t in cap.items()}
    h, s = ws._h, side.cuda_stream
    d, width = x.data_ptr(), (hq + 2 * hk) * 128

    def append(q=d, k=d + 256 * hq, v=d + 256 * (hq + hk), out=P["out"], kp=P["kp"], vp=P["vp"]):
        return L.fi_append(h, q, width, k, width, v, width, None, None, 0.0, None, out, kp, vp, pages, s)

    def weights(q=q.data_ptr(), kp=P["kp"], lse=lse.data_ptr(), w=P["w"]):
        return L.fi_key_weights(h, q, kp, pages, lse, 0.5, 1, w, s)

    def select(w=P["w"], kept=P["kept"]):
        return L.fi_select_keys(h, w, pages, 2, 10, budget, kept, s)

    def compact(kept=P["kept"], kp=P["kp"], vp=P["vp"], w=P["w"]):
        return L.fi_compact(h, kept, budget, kp, vp, w, pages, s)

    torch.cuda.synchronize()
    ws.plan(*empty, ps, True, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        refused = [append(q=None), append(k=None), append(v=None), append(out=None), append(kp=None), append(vp=None), weights(q=None),
                   weights(kp=None), weights(lse=None), weights(w=None), select(w=None), select(kept=None), compact(kept=None),
                   compact(kp=None), compact(vp=None)]
        taken = [weights(), select(), compact(), append()]
    assert refused == [1] * 15 and taken == [0] * 4
    for plan in (empty, (b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len)) * 2:
        for k, t in buffers().items():
            cap[k].copy_(t)
        ws.plan(*plan, ps, True, stream=side)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        assert ws.get_error() == 0
    ws.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, ps, True)
    ws.key_weights(q, ref["kp"], lse, ref["w"], 0.5, True)
    ws.select_keys(ref["w"], budget, ref["kept"], recent=10, sink=2)
    ws.compact(ref["kept"], ref["kp"], ref["vp"], ref["w"])
    ws.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], ref["kp"], ref["vp"], ref["out"])
    torch.cuda.synchronize()
    for k in ref:
        assert torch.equal(ref[k], cap[k]), k
    assert not torch.equal(cap["w"], w0) and (cap["kept"] > budget).any() and cap["out"].any()



@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_captured_small_replayed_large(dtype):
    """The operators captured on one request of one key, replayed on forty of up to 3000: the same as direct calls."""
    torch = torch_mod()
    from serving_attention_plan_gb300 import binding as B
    hq, hk, ps, budget, n = 8, 2, 16, 700, 40
    rng = np.random.default_rng(2)
    lkv = [int(x) for x in rng.integers(1, 3000, n)]
    pages = sum(-(-x // ps) for x in lkv)
    b, one = (batch_of([1] * len(x), x, hq, hk, ps, True, seed=4, extra=0) for x in (lkv, [1]))
    ws = B.Workspace(64, 64, pages, hq, hk)
    ws.set_kv_dtype(dtype, 0.0625, 0.0625)
    scale = 0.0625 if dtype == "e4m3" else 1.0
    k = b.k_pages if dtype == "bf16" else W.to_e4m3(A.bf16_to_f64(b.k_pages) / scale)
    lse = dev(lse_of(b, A.bf16_to_f64(b.q), k, scale, -1, 0.0, "HND"))
    x = torch.randn(n, hq + 2 * hk, 128, device="cuda").to(torch.bfloat16)
    w0, q = torch.rand(pages, hk, ps, device="cuda"), bf16(b.q)

    def buffers():
        pool = bf16(k) if dtype == "bf16" else dev(k)
        return dict(kp=pool, vp=pool.clone(), w=w0.clone(), out=torch.zeros(n, hq, 128, device="cuda", dtype=torch.bfloat16),
                    kept=torch.full((n, hk, budget), -9, device="cuda", dtype=torch.int32))

    def calls(d, m):
        ws.key_weights(q[:m], d["kp"], lse[:m], d["w"], 0.5, True, stream=side)
        ws.select_keys(d["w"], budget, d["kept"][:m], recent=10, sink=2, stream=side)
        ws.compact(d["kept"][:m], d["kp"], d["vp"], d["w"], stream=side)
        ws.append(x[:m, :hq], x[:m, hq:hq + hk], x[:m, hq + hk:], d["kp"], d["vp"], d["out"][:m], stream=side)

    side = torch.cuda.Stream()
    plan = lambda b: ws.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, ps, True, stream=side)
    cap, ref = buffers(), buffers()
    torch.cuda.synchronize()
    plan(one)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls(cap, 1)
    plan(b)
    with torch.cuda.stream(side):
        graph.replay()
    calls(ref, n)
    side.synchronize()
    assert ws.get_error() == 0
    for name in ref:
        assert torch.equal(ref[name].view(torch.uint8), cap[name].view(torch.uint8)), name


def test_composable_plan():
    """With a composable plan the operators work on the per-request part; positions must be given."""
    from serving_attention_plan_gb300 import binding as B
    torch = torch_mod()
    sp = W.shared_prefix_decode(n_req=5, prefix_len=64, lo=20, hi=50)
    s = sp.suffix
    ws = B.Workspace(5, 5, 200, 32, 8)
    idx = lambda b: (b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len)
    ws.plan_composable(idx(sp.prefix), idx(s), 16, False)
    q, kp, vp = bf16(s.q), bf16(s.k_pages), bf16(s.v_pages)
    o, lse = torch.empty_like(q), torch.empty(5, 32, device="cuda")
    ws.run(q, kp, vp, o, lse)
    w = torch.zeros(s.num_pages, 8, 16, device="cuda")
    ws.key_weights(q, kp, lse, w)
    torch.cuda.synchronize()
    lse_h = lse.cpu().numpy()
    ref, reach = C.key_weights(s, A.bf16_to_f64(s.q), s.k_pages, lse_h, np.zeros(w.shape), 1.0, True)
    assert (np.abs(w.cpu().numpy() - ref) <= ref * weights_tol(reach, lse_h) + 1e-30).all()
    x = torch.randn(5, 8, 128, device="cuda").to(torch.bfloat16)
    with pytest.raises(B.FiError) as e:
        ws.append(q, x, x, kp, vp, o)
    assert e.value.status == 1
    ws.append(q, x, x, kp, vp, o, positions=torch.arange(5, device="cuda", dtype=torch.int32))
    torch.cuda.synchronize()
    ws2 = B.Workspace(5, 5, 200, 32, 8)
    shares = s.kv_indices.copy()
    shares[int(s.kv_indptr[1]) - 1] = sp.prefix.kv_indices[0]  # a tail page that is the prefix's too
    ws2.plan_composable(idx(sp.prefix), (s.qo_indptr, s.kv_indptr, shares, s.last_page_len), 16, False)
    for call in (lambda: ws2.append(q, x, x, kp, vp, o, positions=torch.arange(5, device="cuda", dtype=torch.int32)),
                 lambda: ws2.key_weights(q, kp, lse, w)):
        with pytest.raises(B.FiError) as e:
            call()
        assert e.value.status == 3
    _, page, slot, _ = C.append_places(s)
    want = s.k_pages.copy()
    want[page, :, slot] = bits(x)
    assert np.array_equal(bits(kp), want) and ws.get_error() == 0



@pytest.mark.parametrize("lq,lkv,dtype,layout", [([1, 1, 2, 1], [300, 77, 513, 40], "bf16", "HND"), ([1, 1], [200, 900], "e4m3", "NHD"),
                                                 ([130, 1, 40], [300, 500, 40], "bf16", "NHD"), ([200, 9], [700, 130], "e4m3", "HND")])
def test_replays_skip_pages_outside_the_pool(lq, lkv, dtype, layout):
    """Append, weights and compaction replayed after a plan with pages that the captured pool does not have: the error bit is
    set, keys of those pages are left alone, all others get what they should."""
    from serving_attention_plan_gb300 import binding as B
    torch = torch_mod()
    hq, hk, ps, budget, scale = 8, 2, 16, 33, 0.03125 if dtype == "e4m3" else 1.0
    b = batch_of(lq, lkv, hq, hk, ps, True, seed=6, extra=0)
    n, pages = b.batch_size, b.num_pages
    rng = np.random.default_rng(8)
    k = b.k_pages if dtype == "bf16" else W.to_e4m3(A.bf16_to_f64(b.k_pages) / scale)
    k = as_layout(k, layout)
    pool = lambda: bf16(k) if dtype == "bf16" else dev(k)
    host = (lambda t: bits(t)) if dtype == "bf16" else (lambda t: t.cpu().numpy())
    lost = rng.random(b.kv_indices.shape[0]) < 0.4
    lost[0], lost[-1] = True, False
    idx = np.where(lost, b.kv_indices + pages, b.kv_indices).astype(np.int32)
    ws = workspace(b, layout=layout, dtype=dtype, scales=(scale, scale))
    side = torch.cuda.Stream()
    plan = lambda idx: ws.plan(b.qo_indptr, b.kv_indptr, idx, b.last_page_len, ps, True, stream=side)
    x = torch.randn(b.total_q, hk, 128, device="cuda").to(torch.bfloat16)
    q, out = bf16(b.q), torch.zeros(b.total_q, hq, 128, device="cuda", dtype=torch.bfloat16)
    qd = A.bf16_to_f64(b.q)
    lse = lse_of(b, qd, k, scale, -1, 0.0, layout)
    old = rng.random((pages, hk, ps)).astype(np.float32)
    kept = np.full((n, hk, budget), -1, np.int32)
    for i, length in enumerate(lkv):
        for h in range(hk):
            m = min(length, budget)
            kept[i, h, :m] = np.sort(rng.choice(length, m, replace=False))
    kp, vp, w, ck, cv, cw = pool(), pool(), dev(old), pool(), pool(), dev(old)
    lse_d, kept_d = dev(lse), dev(kept)
    torch.cuda.synchronize()
    graphs = []
    for call in (lambda: ws.append(q, x, x, kp, vp, out, stream=side), lambda: ws.key_weights(q, ck, lse_d, w, 0.5, True, stream=side),
                 lambda: ws.compact(kept_d, ck, cv, cw, stream=side)):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            call()
    plan(idx)
    for g in graphs:
        before = [host(kp), host(vp)] if g is graphs[0] else None
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        err = ws.get_error()
        if g is graphs[0]:
            tok, page, slot, key = C.append_places(b)
            entry = np.concatenate([int(b.kv_indptr[i]) + key[int(b.qo_indptr[i]):int(b.qo_indptr[i + 1])] // ps for i in range(n)])
            here = ~lost[entry[tok]]
            assert err == (0 if here.all() else B.DEVERR_PAGE_OOB) and torch.equal(out, q)
            rows = x if dtype == "bf16" else (x.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            rows = bits(rows) if dtype == "bf16" else rows.view(torch.uint8).cpu().numpy()
            for got, want in zip((host(kp), host(vp)), before):
                if layout == "HND":
                    want[page[here], :, slot[here]] = rows[tok[here]]
                else:
                    want[page[here], slot[here]] = rows[tok[here]]
                assert np.array_equal(got, want)
        elif g is graphs[1]:
            assert err == B.DEVERR_PAGE_OOB
            # (the weights read a pool whose pages hold the plan's keys; compaction comes after)
            ref, reach = C.key_weights(b, qd, k, lse, old, 0.5, True, scale, layout=layout)
            got = w.cpu().numpy()
            gone = np.zeros(pages, bool)
            gone[b.kv_indices[lost]] = True
            used = np.zeros((pages, ps), bool)
            for i, length in enumerate(lkv):
                used[C.places(b, i, np.arange(length))] = True
            used[gone] = False
            tol = weights_tol(reach, lse) + 1000 * 2.0 ** -24
            err_w, lim = np.abs(got - ref).transpose(0, 2, 1), (ref * tol + 1e-30).transpose(0, 2, 1)
            assert (err_w[used] <= lim[used]).all()
            assert np.array_equal(got.transpose(0, 2, 1)[~used], old.transpose(0, 2, 1)[~used])
        else:
            assert err == B.DEVERR_PAGE_OOB
            rk, rw = k.copy(), old.copy()
            for i, length in enumerate(lkv):
                if length <= budget:
                    continue
                for h in range(hk):
                    j = np.arange(budget)
                    src = kept[i, h]
                    at = int(b.kv_indptr[i])
                    ok = ~lost[at + j // ps] & ~lost[at + src // ps]
                    tp, ts = C.places(b, i, j[ok])
                    fp, fs = C.places(b, i, src[ok])
                    if layout == "HND":
                        rk[tp, h, ts] = k[fp, h, fs]
                    else:
                        rk[tp, ts, h] = k[fp, fs, h]
                    rw[tp, h, ts] = old[fp, h, fs]
            assert np.array_equal(host(ck), rk) and np.array_equal(host(cv), rk) and np.array_equal(cw.cpu().numpy(), rw)


@pytest.mark.parametrize("lq,lkv,dtype", [([1, 2, 1], [37, 64, 1], "bf16"), ([90, 1, 300], [90, 70, 700], "bf16"), ([90, 200], [400, 200], "e4m3")])
def test_key_weights_window_of_zero(lq, lkv, dtype):
    """A window of zero: every token sees the key of its own position alone."""
    test_key_weights((lq, lkv, 8, 2, 16, True, dtype, "HND", 0, 0.0, 0.5, False, 0))


def test_append_smallest_scales():
    """Scales whose reciprocal is beyond 32 bits: everything saturates, zeros stay zero."""
    torch = torch_mod()
    b = batch_of([1, 1], [4, 7], 2, 1, 4)
    ws = workspace(b, dtype="e4m3", scales=(1e-40, 1e-44))
    q = torch.randn(2, 2, 128, device="cuda").to(torch.bfloat16)
    k = torch.zeros(2, 1, 128, device="cuda", dtype=torch.bfloat16)
    k[:, :, 1], k[:, :, 2] = 0.5, -3.0
    kp, vp = (torch.full((b.num_pages, 1, 4, 128), 1.0, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
    ws.append(q, k, k, kp, vp, torch.empty_like(q))
    torch.cuda.synchronize()
    _, page, slot, _ = C.append_places(b)
    for pool in (kp, vp):
        rows = pool.float().cpu()[page, 0, slot]
        assert (rows[:, 1] == 448).all() and (rows[:, 2] == -448).all() and (rows[:, 0] == 0).all() and (rows[:, 3:] == 0).all()


# ---- refusals --------------------------------------------------------------------------------------


def test_refusals():
    from serving_attention_plan_gb300 import binding as B
    torch = torch_mod()
    b = batch_of([1, 1], [20, 30], 4, 2, 4)
    q, kp, vp = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages)
    n = b.num_pages
    k = torch.zeros(2, 2, 128, device="cuda", dtype=torch.bfloat16)
    o, lse = torch.empty_like(q), torch.zeros(2, 4, device="cuda")
    w = torch.zeros(n, 2, 4, device="cuda")
    kept = torch.zeros(2, 2, 8, device="cuda", dtype=torch.int32)
    fresh = B.Workspace(2, 2, 64, 4, 2)
    for call in (lambda: fresh.append(q, k, k, kp, vp, o), lambda: fresh.key_weights(q, kp, lse, w),
                 lambda: fresh.select_keys(w, 8, kept), lambda: fresh.compact(kept, kp, vp)):
        with pytest.raises(B.FiError) as e:
            call()
        assert e.value.status == 6
    ws = workspace(b)
    used = int(b.kv_indices.max())
    bad = [
        (1, lambda: ws.append(q, k, k, kp[:used], vp[:used], o)),            # a planned page outside the pool
        (1, lambda: ws.key_weights(q, kp[:used], lse, w[:used])),
        (1, lambda: ws.select_keys(w[:used], 8, kept)),
        (1, lambda: ws.compact(kept, kp[:used], vp[:used])),
        (1, lambda: ws.append(q, k, k, kp, vp, o, eps=-1.0)),
        (1, lambda: ws.append(q, k, k, kp, vp, o, eps=float("nan"))),
        (1, lambda: ws.key_weights(q, kp, lse, w, decay=1.5)),
        (1, lambda: ws.key_weights(q, kp, lse, w, decay=float("nan"))),
        (1, lambda: ws.select_keys(w, 8, kept, recent=5, sink=4)),
        (1, lambda: ws.select_keys(w, 8, kept, recent=-1)),
        (1, lambda: ws.set_rope([float("inf")] * 8)),
        (1, lambda: ws.set_rope(np.ones(65))),
        (3, lambda: ws.set_rope(np.ones(9))),
    ]
    for status, call in bad:
        with pytest.raises(B.FiError) as e:
            call()
        assert e.value.status == status
    wrong = [
        lambda: ws.append(q.float(), k, k, kp, vp, o), lambda: ws.append(q[:1], k, k, kp, vp, o),
        lambda: ws.append(q, k.transpose(0, 1), k, kp, vp, o), lambda: ws.append(q, k, k, kp, vp, o[..., :64]),
        lambda: ws.append(q, k, k, kp.view(torch.uint8), vp, o), lambda: ws.append(q, k, k, kp, vp[:-1], o),
        lambda: ws.append(q, k, k, kp, vp, o, positions=torch.zeros(2, device="cuda")),
        lambda: ws.append(q, k, k, kp, vp, o, q_weight=torch.ones(128, device="cuda")),
        lambda: ws.append(q.cpu(), k, k, kp, vp, o),
        lambda: ws.key_weights(q, kp, lse.double(), w), lambda: ws.key_weights(q, kp, lse, w[:, :1]),
        lambda: ws.key_weights(q, kp, lse, w.half()), lambda: ws.select_keys(w, 9, kept),
        lambda: ws.select_keys(w, 8, kept.long()), lambda: ws.compact(kept[:1], kp, vp),
        lambda: ws.compact(kept[0], kp, vp), lambda: ws.compact(kept, kp, vp, w[:-1]),
        lambda: ws.set_rope(np.ones((2, 8))),
    ]
    for call in wrong:
        with pytest.raises(ValueError):
            call()
    # shared pages: one tail for two requests, one prefix for two requests
    ws.plan([0, 1, 2], [0, 2, 4], [0, 1, 2, 1], [2, 3], 4, False)
    for call in (lambda: ws.append(q, k, k, kp, vp, o), lambda: ws.key_weights(q, kp, lse, w), lambda: ws.compact(kept, kp, vp)):
        with pytest.raises(B.FiError) as e:
            call()
        assert e.value.status == 3
    ws.plan([0, 1, 2], [0, 2, 4], [0, 1, 0, 3], [2, 3], 4, False)
    ws.append(q, k, k, kp, vp, o)
    with pytest.raises(B.FiError):
        ws.key_weights(q, kp, lse, w)
    # nothing to do: no requests, no tokens, no keys
    ws.plan([0], [0], [], [], 4, False)
    ws.append(q[:0], k[:0], k[:0], kp, vp, o[:0])
    ws.key_weights(q[:0], kp, lse[:0], w)
    ws.select_keys(w, 8, kept[:0])
    ws.compact(kept[:0], kp, vp, w)
    ws.plan([0, 1], [0, 0], [], [0], 4, False)
    ws.append(q[:1], k[:1], k[:1], kp, vp, o[:1])
    ws.key_weights(q[:1], kp, lse[:1], w)
    ws.select_keys(w, 8, kept[:1])
    ws.compact(kept[:1], kp, vp, w)
    torch.cuda.synchronize()
    assert (kept[0] == -1).all() and torch.equal(o[0], q[0]) and (w == 0).all() and ws.get_error() == 0


def test_captured_prompt_weights_follow_a_new_plan():
    """The tensor-core weights captured once: a replay after a plan of other lengths (the same total of query tokens)."""
    torch = torch_mod()
    from serving_attention_plan_gb300 import binding as B
    first = batch_of([100, 300, 40], [120, 900, 40], 8, 2, 16, True, seed=1, extra=20)
    second = batch_of([440], [1210], 8, 2, 16, True, seed=2, extra=first.num_pages - 76)
    third = batch_of([400, 39, 1], [500, 600, 100], 8, 2, 16, True, seed=4, extra=first.num_pages - 77)  # both kernels
    assert second.num_pages == first.num_pages == third.num_pages and second.total_q == first.total_q == third.total_q
    ws = B.Workspace(4, 500, 200, 8, 2)
    side = torch.cuda.Stream()
    q, k = bf16(first.q), bf16(first.k_pages)
    lse = torch.full((440, 8), 5.0, device="cuda")
    w, want = torch.zeros(first.num_pages, 2, 16, device="cuda"), torch.zeros(first.num_pages, 2, 16, device="cuda")
    plan = lambda b: ws.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, 16, True, stream=side)
    torch.cuda.synchronize()
    plan(first)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ws.key_weights(q, k, lse, w, 1.0, True, stream=side)
    for b in (second, third, first, third, second):
        plan(b)
        w.zero_()
        want.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        ws.key_weights(q, k, lse, want, 1.0, True, stream=side)
        side.synchronize()
        assert ws.get_error() == 0 and torch.equal(w, want) and w.abs().sum() > 0
        ref, reach = C.key_weights(b, f64(q), first.k_pages, lse.cpu().numpy(), np.zeros(w.shape), 1.0, True)
        tol = weights_tol(reach, lse.cpu().numpy()) + 1800 * 2.0 ** -24
        assert (np.abs(w.cpu().numpy() - ref) <= ref * tol + 1e-30).all()


@pytest.mark.parametrize("n_req,lq,causal,window", [(1500, 1, False, -1), (1100, 9, True, 2**31 - 1), (1100, 9, True, 3)])
def test_many_requests(n_req, lq, causal, window):
    """More requests than two rounds of the 32-way search, some of them empty; append and weights."""
    torch = torch_mod()
    rng = np.random.default_rng(6)
    ql = np.where(rng.random(n_req) < 0.2, 0, lq)
    kl = np.where(rng.random(n_req) < 0.1, 0, rng.integers(1, 40, n_req))
    kl = np.where(ql > 0, np.maximum(kl, 1), kl)
    b = batch_of(list(ql), list(kl), 2, 1, 8, causal, seed=3)
    q = A.bf16_to_f64(b.q)
    lse = lse_of(b, q, b.k_pages, 1.0, window, 0.0, "HND")
    old = rng.random((b.num_pages, 1, 8)).astype(np.float32)
    ws = workspace(b, window=window)
    w = dev(old)
    ws.key_weights(bf16(b.q), bf16(b.k_pages), dev(lse), w, 0.5, True)
    torch.cuda.synchronize()
    ref, reach = C.key_weights(b, q, b.k_pages, lse, old, 0.5, True, window=window)
    used = np.zeros((b.num_pages, 8), bool)
    for i in range(n_req):
        p, s = C.places(b, i, np.arange(int(kl[i])))
        used[p, s] = True
    got = w.cpu().numpy()
    tol = weights_tol(reach, lse) + 18 * 2.0 ** -24
    assert (np.abs(got - ref)[:, 0][used] <= (ref * tol + 1e-30)[:, 0][used]).all()
    assert np.array_equal(got[:, 0][~used], old[:, 0][~used])
    k = torch.randn(b.total_q, 1, 128, device="cuda").to(torch.bfloat16)
    kp, vp, out = bf16(b.k_pages), bf16(b.v_pages), torch.zeros(b.total_q, 2, 128, device="cuda", dtype=torch.bfloat16)
    ws.append(bf16(b.q), k, k, kp, vp, out)
    torch.cuda.synchronize()
    tok, page, slot, _ = C.append_places(b)
    want = b.k_pages.copy()
    want[page, :, slot] = bits(k)[tok]
    assert np.array_equal(bits(kp), want) and np.array_equal(bits(out), b.q) and ws.get_error() == 0


@pytest.mark.parametrize("lq,causal", [(1, False), (30, True)])
def test_pool_beyond_32_bit_offsets(lq, causal):
    """Pages at the end of a pool of more than 2^31 elements (and 2^32 bytes): append, weights, selection, compaction."""
    torch = torch_mod()
    pool, hk, ps, hq = (1 << 31) // (8 * 16 * 128) + 50, 8, 16, 16
    b = batch_of([lq, lq], [300, 77], hq, hk, ps, causal, seed=2, extra=0)
    n = b.num_pages
    high = dataclasses.replace(b, kv_indices=(b.kv_indices + pool - n).astype(np.int32))
    kp, vp = (torch.empty(pool, hk, ps, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = torch.empty(pool, hk, ps, device="cuda")
    for t in (kp, vp, w):
        t[-2 * n:] = 0
    kp[-n:], vp[-n:] = bf16(b.k_pages), bf16(b.v_pages)
    rng = np.random.default_rng(1)
    old = rng.random((n, hk, ps)).astype(np.float32)
    w[-n:] = dev(old)
    q = A.bf16_to_f64(b.q)
    lse = lse_of(b, q, b.k_pages, 1.0, -1, 0.0, "HND")
    ws = workspace(high)
    ws.key_weights(bf16(b.q), kp, dev(lse), w, 0.5, True)
    kept = torch.empty(2, hk, 64, dtype=torch.int32, device="cuda")
    ws.select_keys(w, 64, kept, recent=8, sink=4)
    torch.cuda.synchronize()
    ref, reach = C.key_weights(b, q, b.k_pages, lse, old, 0.5, True)
    got = w[-n:].cpu().numpy()
    used = np.zeros((n, ps), bool)
    for i, length in enumerate((300, 77)):
        p, s = C.places(b, i, np.arange(length))
        used[p, s] = True
    err, lim = np.abs(got - ref), ref * (weights_tol(reach, lse) + 60 * 2.0 ** -24) + 1e-30
    assert (err <= lim).transpose(0, 2, 1)[used].all()
    rkept = C.select(b, got, 64, 8, 4)
    assert np.array_equal(kept.cpu().numpy(), rkept)
    ws.compact(kept, kp, vp, w)
    torch.cuda.synchronize()
    rk, rv, rw = C.compact(b, rkept, [b.k_pages, b.v_pages, got], ["HND"] * 3)
    assert np.array_equal(bits(kp[-n:]), rk) and np.array_equal(bits(vp[-n:]), rv) and np.array_equal(w[-n:].cpu().numpy(), rw)
    x = torch.randn(2 * lq, hk, 128, device="cuda").to(torch.bfloat16)
    out = torch.empty(2 * lq, hq, 128, dtype=torch.bfloat16, device="cuda")
    ws.append(bf16(b.q), x, x, kp, vp, out)
    torch.cuda.synchronize()
    tok, page, slot, _ = C.append_places(b)
    rk[page, :, slot], rv[page, :, slot] = bits(x)[tok], bits(x)[tok]
    assert np.array_equal(bits(kp[-n:]), rk) and np.array_equal(bits(vp[-n:]), rv)
    assert not kp[-2 * n:-n].any() and not w[-2 * n:-n].any() and ws.get_error() == 0


def test_c_entry_refusals():
    """Misaligned pointers, narrow or odd strides, null pointers and a workspace of another shape, at the C entry."""
    from serving_attention_plan_gb300 import binding as B
    torch = torch_mod()
    L = B.lib()
    b = batch_of([2, 1], [20, 30], 4, 2, 4)
    ws = workspace(b)
    n = b.num_pages
    q, kp = bf16(b.q), bf16(b.k_pages)
    x = torch.zeros(3, 2, 128, device="cuda", dtype=torch.bfloat16)
    w, lse = torch.zeros(n, 2, 4, device="cuda"), torch.zeros(3, 4, device="cuda")
    kept = torch.zeros(2, 2, 8, device="cuda", dtype=torch.int32)
    h, s = ws._h, torch.cuda.current_stream().cuda_stream
    P = {k: t.data_ptr() for k, t in dict(q=q, x=x, kp=kp, w=w, lse=lse, kept=kept).items()}

    def append(q=P["q"], sq=512, k=P["x"], sk=256, v=P["x"], sv=256, wq=None, wk=None, eps=0.0, pos=None, out=P["q"],
               kp=P["kp"], vp=P["kp"], pages=n):
        return L.fi_append(h, q, sq, k, sk, v, sv, wq, wk, eps, pos, out, kp, vp, pages, s)

    for bad in (dict(q=P["q"] + 2), dict(k=P["x"] + 8), dict(v=None), dict(q=None), dict(out=None), dict(out=P["q"] + 4), dict(kp=None),
                dict(vp=P["kp"] + 2), dict(sq=511), dict(sq=516), dict(sk=128), dict(sv=260), dict(wq=P["x"] + 2), dict(pos=P["lse"] + 1),
                dict(eps=float("inf")), dict(pages=-1), dict(pages=int(b.kv_indices.max()))):
        assert append(**bad) == 1, bad
    weights = lambda q=P["q"], k=P["kp"], pages=n, lse=P["lse"], decay=1.0, new=1, w=P["w"]: L.fi_key_weights(h, q, k, pages, lse, decay, new, w, s)
    for bad in (dict(q=None), dict(q=P["q"] + 2), dict(k=None), dict(k=P["kp"] + 8), dict(lse=None), dict(lse=P["lse"] + 2), dict(w=None),
                dict(w=P["w"] + 1), dict(decay=-0.1), dict(new=2), dict(pages=0)):
        assert weights(**bad) == 1, bad
    select = lambda w=P["w"], pages=n, sink=1, recent=2, budget=8, kept=P["kept"]: L.fi_select_keys(h, w, pages, sink, recent, budget, kept, s)
    for bad in (dict(w=None), dict(w=P["w"] + 2), dict(kept=None), dict(kept=P["kept"] + 2), dict(budget=0), dict(sink=-1), dict(recent=8),
                dict(sink=2**31 - 1, recent=2**31 - 1), dict(pages=1)):
        assert select(**bad) == 1, bad
    compact = lambda kept=P["kept"], budget=8, k=P["kp"], v=P["kp"], w=None, pages=n: L.fi_compact(h, kept, budget, k, v, w, pages, s)
    for bad in (dict(kept=None), dict(kept=P["kept"] + 1), dict(budget=0), dict(k=None), dict(v=None), dict(k=P["kp"] + 4), dict(w=P["w"] + 3), dict(pages=2)):
        assert compact(**bad) == 1, bad
    # more rows than the kernels number in 32 bits
    assert append(pages=2**31 - 1) == 3 and select(pages=2**30) == 3
    torch.cuda.synchronize()
    assert np.array_equal(bits(kp), b.k_pages) and np.array_equal(bits(q), b.q) and ws.get_error() == 0


def test_two_workspaces_at_once():
    """Prompts on one stream and a decode batch on another, each with its own workspace, launched without waiting."""
    torch = torch_mod()
    jobs = []
    for seed, (lq, lkv) in enumerate([([700, 300], [900, 300]), ([1] * 40, list(range(50, 850, 20)))]):
        b = batch_of(lq, lkv, 16, 4, 16, True, seed=seed)
        q = A.bf16_to_f64(b.q)
        lse = lse_of(b, q, b.k_pages, 1.0, -1, 0.0, "HND")
        jobs.append((workspace(b), bf16(b.q), bf16(b.k_pages), dev(lse), b, q, lse, torch.cuda.Stream()))
    alone = []
    for ws, q, k, lse, b, *_ in jobs:
        w = torch.zeros(b.num_pages, 4, 16, device="cuda")
        for _ in range(8):
            ws.key_weights(q, k, lse, w, 1.0, False)
        alone.append(w)
    torch.cuda.synchronize()
    both = [torch.zeros_like(w) for w in alone]
    torch.cuda.synchronize()
    for _ in range(8):
        for (ws, q, k, lse, b, _, _, stream), w in zip(jobs, both):
            ws.key_weights(q, k, lse, w, 1.0, False, stream=stream)
    torch.cuda.synchronize()
    for (ws, *_), w, ref in zip(jobs, both, alone):
        assert torch.equal(w, ref) and ws.get_error() == 0
    for (_, _, _, _, b, q, lse, _), w in zip(jobs, both):
        one, reach = C.key_weights(b, q, b.k_pages, lse, np.zeros(w.shape), 1.0, False)
        tol = weights_tol(reach, lse) + (2800 + 8) * 2.0 ** -24
        assert (np.abs(w.cpu().numpy() - 8 * one) <= 8 * one * tol + 1e-30).all()
