"""GPU parity of attention over parts of a cache (trees of drafted tokens, pages chosen by a score) against the float64 oracle."""
import ctypes
import dataclasses

import numpy as np
import pytest

from oracle import attention as A
from oracle import cache as C
from oracle import parts as P
from serving_attention_plan_gb300 import binding as B
from serving_attention_plan_gb300 import workloads as W

from .gpu_helpers import torch_mod
from .test_gpu_cache import as_layout, batch_of, bf16, bits, dev, f64, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from serving_attention_plan_gb300 import build
    build.build()
    assert torch_mod().cuda.is_available()


def pool(b, side, dtype, layout, scale, spread=1.0):
    """(device pages, their values in 64 bits) of the batch's K or V."""
    torch = torch_mod()
    x = as_layout(getattr(b, side), layout)
    if dtype == "bf16":
        return bf16(x), A.bf16_to_f64(x)
    codes = (torch.from_numpy(A.bf16_to_f64(x).astype(np.float32)) * (spread / scale)).to(torch.float8_e4m3fn)
    return codes.cuda(), A.e4m3_to_f64(codes.view(torch.uint8).numpy()) * scale


def outputs(b):
    torch = torch_mod()
    o = torch.full((b.total_q, b.num_qo_heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    return o, torch.full((b.total_q, b.num_qo_heads), float("nan"), dtype=torch.float32, device="cuda")


def assert_state(o, lse, ref, weight_bits, cap=0.0, cap_rel=0.0):
    """Against the definition.  A logit is off by the fp32 sum of 128 products (each of 128 additions by 2^-24 of the sum of
    |terms|: 2^-17, twice that for products that drop bits below the sum's), by its scaling in the exponent (2^-23 of it), and by the soft-cap's tanh (1.5e-7
    of the cap, or cap_rel of the logit); a weight by e^delta, by the exponential's 2^-22 and by its rounding to 16 bits; the output by its
    own rounding to bf16, 2^-8.  The sums of weights and products are fp32: 2^-15 of the sum of |terms| covers some
    hundred chained tiles."""
    want_o, want_lse, spread, reach = ref
    o, lse = f64(o), lse.cpu().numpy().astype(np.float64)
    none = np.isneginf(want_lse)
    assert not np.isnan(o).any() and not np.isnan(lse).any()
    assert np.array_equal(np.isneginf(lse), none) and (o[none] == 0).all()
    some = ~none
    delta = reach * 2.0 ** -16 + cap * 2e-7 + cap_rel * cap + np.abs(np.where(none, 0, want_lse)) * 2.0 ** -20 + 2.0 ** -18
    assert (np.abs(lse[some] - want_lse[some]) <= delta[some]).all(), np.abs(lse[some] - want_lse[some]).max()
    tol = np.abs(want_o) * 2.0 ** -8 + spread * (weight_bits + 2 * delta[..., None] + 2.0 ** -15) + 1e-30
    assert (np.abs(o - want_o) <= tol).all(), (np.abs(o - want_o) / tol).max()


BF16_WEIGHTS = 2.0 ** -8
# f16 weights: half a step of 2^-11; those below 2^-14 lose at most 2^-25 each, and a row's weights are relative to its largest
F16_WEIGHTS = 2.0 ** -11 + 2.0 ** -14


# e4m3 trees: an element of q below 2^-9 of its row's largest may be off by 2^-10 where the largest is 128 or more, 2^-17 of the
# largest, in place of nothing: half of that of the largest, on top of each |q_d|, in units of the 2^-16 that a logit's terms get
Q_FLOOR = 0.5


# ---- trees -------------------------------------------------------------------------------------------


def random_mask(rng, b, kind):
    """int32 [total_q, words] masks."""
    lens = np.diff(b.qo_indptr)
    if kind == "tree":
        parents = np.concatenate([[rng.integers(-1, t) if t else -1 for t in range(n)] for n in lens] + [[]]).astype(np.int32)
        return B.tree_mask(b.qo_indptr, parents)
    words = max(1, -(-int(lens.max(initial=0)) // 32)) + (kind == "wide")
    m = rng.integers(0, 2 ** 32, size=(b.total_q, words), dtype=np.uint64).astype(np.uint32)
    if kind == "sparse":  # most rows see few drafted tokens, some none
        m &= rng.integers(0, 2 ** 32, size=m.shape, dtype=np.uint64).astype(np.uint32) & rng.integers(0, 2 ** 32, size=m.shape, dtype=np.uint64).astype(np.uint32)
        m[::3] = 0
    return m.view(np.int32)


TREES = [
    # l_q, l_kv, query heads, KV heads, page, dtype, layout, cap, masks, SMs
    ([1], [1], 1, 1, 16, "bf16", "HND", 0.0, "tree", 0),
    ([1, 1, 1], [1, 129, 640], 8, 2, 16, "bf16", "HND", 0.0, "tree", 0),
    ([16, 0, 11, 13], [316, 40, 11, 583], 8, 2, 16, "bf16", "HND", 0.0, "tree", 0),
    ([5, 33, 64], [133, 33, 700], 12, 4, 8, "bf16", "NHD", 0.0, "tree", 4),
    ([64, 100], [1500, 131], 8, 1, 32, "bf16", "HND", 0.0, "wide", 0),            # 512 and 800 rows: several row tiles
    ([7, 9], [7, 260], 16, 2, 128, "bf16", "HND", 0.0, "sparse", 3),             # rows that see nothing
    ([20, 3], [12, 0], 4, 2, 16, "bf16", "HND", 0.0, "sparse", 0),               # more tokens than keys, no keys
    ([3, 2], [300, 65], 128, 1, 64, "bf16", "HND", 0.0, "tree", 0),              # one token a row tile
    ([3, 40], [200, 999], 10, 2, 16, "bf16", "HND", 30.0, "tree", 7),            # five heads a group
    ([17, 2], [1030, 90], 8, 2, 16, "bf16", "NHD", 200.0, "wide", 0),
    ([1], [5000], 1, 1, 16, "bf16", "HND", 0.0, "tree", 0),                     # one row over many CTAs
    ([2] * 70, list(range(1, 211, 3)), 4, 2, 8, "bf16", "HND", 0.0, "tree", 0),  # many short requests
    ([1], [1], 1, 1, 16, "e4m3", "HND", 0.0, "tree", 0),
    ([16, 0, 11, 13], [316, 40, 11, 583], 8, 2, 16, "e4m3", "HND", 0.0, "tree", 0),
    ([5, 33, 64], [133, 33, 700], 12, 4, 8, "e4m3", "NHD", 0.0, "wide", 4),
    ([20, 3], [12, 0], 4, 2, 128, "e4m3", "HND", 0.0, "sparse", 0),
    ([25, 30], [1300, 777], 64, 8, 64, "e4m3", "NHD", 30.0, "tree", 0),
    ([30], [4000], 4, 1, 32, "e4m3", "HND", 100.0, "tree", 0),
]


@pytest.mark.parametrize("case", TREES, ids=range(len(TREES)))
def test_tree(case):
    lq, lkv, hq, hk, ps, dtype, layout, cap, kind, sms = case
    b = batch_of(lq, lkv, hq, hk, ps, False, seed=len(lq) + ps + hq, scale=1.3)
    scales = (0.0625, 0.03125) if dtype == "e4m3" else (1.0, 1.0)
    (k, kv), (v, vv) = pool(b, "k_pages", dtype, layout, scales[0]), pool(b, "v_pages", dtype, layout, scales[1])
    mask = random_mask(np.random.default_rng(hq + ps), b, kind)
    ws = workspace(b, cap=cap, layout=layout, dtype=dtype, scales=scales, num_sms=sms)
    q, (o, lse) = bf16(b.q), outputs(b)
    ws.tree_run(q, k, v, dev(mask), o, lse)
    torch_mod().cuda.synchronize()
    assert ws.get_error() == 0
    ref = P.tree_attention(b, f64(q), kv, vv, mask, cap, layout, Q_FLOOR if dtype == "e4m3" else 0.0)
    assert_state(o, lse, ref, F16_WEIGHTS if dtype == "e4m3" else BF16_WEIGHTS, cap, 4e-6 if cap > 64 else 0.0)
    again = outputs(b)
    ws.tree_run(q, k, v, dev(mask), *again)
    assert np.array_equal(bits(again[0]), bits(o)) and torch_mod().equal(again[1], lse)


@pytest.mark.parametrize("dtype,ps", [("bf16", 16), ("bf16", 128), ("e4m3", 32)])
def test_tree_unseen_values_and_unused_slots(dtype, ps):
    """NaN and infinities in the page slots behind the last key, and in K rows that no token sees, reach no output."""
    torch = torch_mod()
    b = batch_of([4, 6], [ps + 9, 70], 8, 2, ps, False, seed=3)
    (k, kv), (v, vv) = pool(b, "k_pages", dtype, "HND", 1.0), pool(b, "v_pages", dtype, "HND", 1.0)
    mask = np.zeros((10, 1), np.int32)
    mask[:4, 0] = [0b1, 0b11, 0b1, 0b1001]      # nobody sees drafted token 2 of request 0
    mask[4:, 0] = [0b1, 0b10, 0b101, 0b1001, 0b10001, 0b100001]
    codes_k, codes_v = (x.view(torch.uint8 if dtype == "e4m3" else torch.int16) for x in (k, v))
    nan, inf = (0x7F, 0x7E) if dtype == "e4m3" else (0x7FC0, 0x7F80)
    for i, n in enumerate((ps + 9, 70)):
        page = int(b.kv_indices[b.kv_indptr[i + 1] - 1])
        codes_k[page, :, (n - 1) % ps + 1:] = nan
        codes_v[page, :, (n - 1) % ps + 1:] = nan
    j = ps + 9 - 4 + 2
    codes_k[int(b.kv_indices[j // ps]), 0, j % ps] = nan
    codes_k[int(b.kv_indices[j // ps]), 1, j % ps] = inf
    ws = workspace(b, dtype=dtype)
    q, (o, lse) = bf16(b.q), outputs(b)
    ws.tree_run(q, k, v, dev(mask), o, lse)
    torch.cuda.synchronize()
    assert_state(o, lse, P.tree_attention(b, f64(q), kv, vv, mask, q_floor=Q_FLOOR if dtype == "e4m3" else 0.0), F16_WEIGHTS if dtype == "e4m3" else BF16_WEIGHTS)


def test_tree_of_a_chain_is_causal_attention():
    """A chain's mask is the causal one: the same rows as fi_run's on a causal plan, within both kernels' roundings."""
    torch = torch_mod()
    b = batch_of([40, 7, 1], [900, 7, 300], 8, 2, 16, True, seed=9)
    ws = workspace(b)
    q, k, v = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages)
    mask = B.tree_mask(b.qo_indptr, np.concatenate([np.arange(n) - 1 for n in (40, 7, 1)]))
    (o, lse), (ro, rl) = outputs(b), outputs(b)
    ws.tree_run(q, k, v, dev(mask), o, lse)
    ws.run(q, k, v, ro, rl)
    torch.cuda.synchronize()
    assert (lse - rl).abs().max() <= 2.0 ** -12 and (o.float() - ro.float()).abs().max() <= 0.04


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_tree_rows_that_are_not_finite(dtype):
    """A NaN or infinity in q shows in its own row alone."""
    torch = torch_mod()
    b = batch_of([5, 40], [300, 700], 8, 2, 16, False, seed=12)
    k, v = (pool(b, x, dtype, "HND", 1.0)[0] for x in ("k_pages", "v_pages"))
    ws = workspace(b, dtype=dtype)
    q, (o, lse), (ro, rl) = bf16(b.q), outputs(b), outputs(b)
    mask = dev(random_mask(np.random.default_rng(0), b, "tree"))
    ws.tree_run(q, k, v, mask, ro, rl)
    bad = q.clone()
    bad[3, 1, 7], bad[20, 6, 100] = float("nan"), float("inf")
    ws.tree_run(bad, k, v, mask, o, lse)
    torch.cuda.synchronize()
    assert torch.isnan(lse[3, 1]) and torch.isnan(o[3, 1]).all()
    assert not torch.isfinite(lse[20, 6]) and not torch.isfinite(o[20, 6]).any()
    rest = torch.ones(45, 8, dtype=torch.bool, device="cuda")
    rest[3, 1] = rest[20, 6] = False
    assert torch.equal(lse[rest], rl[rest]) and torch.equal(o[rest], ro[rest])


def test_tree_then_a_launch_that_reads_its_output():
    """Back to back, the second call on the first's output: where no unit is cut (the joining launch has nothing to do), where some are."""
    torch = torch_mod()
    for lq, lkv, sms in (([20] * 300, [256] * 300, 0), ([30, 60, 9] * 30, [5000, 900, 70] * 30, 0)):
        b = W.make_paged_batch(np.random.default_rng(3), "chain", lq, lkv, 8, 2, 16, False)
        ws, ws2 = workspace(b, num_sms=sms), workspace(b, num_sms=sms)
        q, k, v = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages)
        mask = dev(random_mask(np.random.default_rng(1), b, "tree"))
        (o1, l1), (o2, l2), (r1, s1), (r2, s2) = (outputs(b) for _ in range(4))
        for turn in range(5):
            ws.tree_run(q, k, v, mask, r1, s1)
            torch.cuda.synchronize()
            ws.tree_run(r1, k, v, mask, r2, s2)
            torch.cuda.synchronize()
            o1.fill_(float("nan"))
            ws.tree_run(q, k, v, mask, o1, l1)
            ws2.tree_run(o1, k, v, mask, o2, l2)
            torch.cuda.synchronize()
            assert torch.equal(o1, r1) and torch.equal(o2, r2) and torch.equal(l2, s2)
        assert ws.get_error() == 0 and ws2.get_error() == 0


def capture(call):
    torch = torch_mod()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    torch.cuda.synchronize()
    return g


def plan(ws, b):
    ws.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, b.page_size, b.causal)


def test_tree_replayed():
    """A captured call follows later plans of as many tokens: other lengths, page lists and masks."""
    torch = torch_mod()
    a = batch_of([20, 12], [60, 30], 8, 2, 16, False, seed=1, extra=200)
    b = batch_of([1, 29, 2], [900, 1500, 2], 8, 2, 16, False, seed=2, extra=a.num_pages - 153)
    assert a.num_pages >= int(b.kv_indptr[-1])
    ws = B.Workspace(4, 32, 300, 8, 2)
    pages = max(a.num_pages, b.num_pages)
    rng = np.random.default_rng(0)
    k, v = (bf16(W.f32_to_bf16_bits(rng.standard_normal((pages, 2, 16, 128)).astype(np.float32))) for _ in range(2))
    q, (o, lse) = bf16(a.q), outputs(a)
    mask = torch.zeros(32, 2, dtype=torch.int32, device="cuda")
    plan(ws, a)
    g = capture(lambda: ws.tree_run(q, k, v, mask, o, lse))
    for x in (b, a):
        plan(ws, x)
        m = random_mask(rng, x, "wide")[:, :2]
        mask.copy_(dev(np.ascontiguousarray(m)))
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert ws.get_error() == 0
        assert_state(o, lse, P.tree_attention(x, f64(q), A.bf16_to_f64(bits(k)), A.bf16_to_f64(bits(v)), m), BF16_WEIGHTS)


def test_tree_refusals():
    torch = torch_mod()
    b = batch_of([40, 1], [100, 20], 8, 2, 16, False)
    ws = workspace(b)
    q, k, v, (o, lse) = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages), outputs(b)
    ones = torch.ones(41, 2, dtype=torch.int32, device="cuda")
    for args in ((q[1:], k, v, ones, o, lse), (q, k[:, :1], v, ones, o, lse), (q, k, v, ones[:40], o, lse), (q, k, v, ones.long(), o, lse),
                 (q, k, v, ones, o.float(), lse), (q, k, v, ones, o, lse[:, :7]), (q, k, v, ones.cpu(), o, lse), (q, k, v, ones[:, 0], o, lse),
                 (q, k, v, ones.t().contiguous().t(), o, lse)):
        with pytest.raises(ValueError):
            ws.tree_run(*args)
    with pytest.raises(B.FiError) as e:  # one word for 40 tokens
        ws.tree_run(q, k, v, ones[:, :1].contiguous(), o, lse)
    assert e.value.status == 1
    for change, status in (({"window": 5, "causal": True}, 3),):
        w = workspace(dataclasses.replace(b, causal=True), window=5)
        with pytest.raises(B.FiError) as e:
            w.tree_run(q, k, v, ones, o, lse)
        assert e.value.status == status
    small = batch_of([1, 1], [9, 20], 8, 2, 4, False)
    w = workspace(small)
    with pytest.raises(B.FiError) as e:  # a page size that the tiles do not take
        w.tree_run(bf16(small.q), bf16(small.k_pages), bf16(small.v_pages), ones[:2], *outputs(small))
    assert e.value.status == 3
    many = batch_of([1], [9], 129, 1, 16, False)
    w = workspace(many)
    with pytest.raises(B.FiError) as e:
        w.tree_run(bf16(many.q), bf16(many.k_pages), bf16(many.v_pages), ones[:1], *outputs(many))
    assert e.value.status == 3
    with pytest.raises(B.FiError) as e:
        B.Workspace(2, 41, 20, 8, 2).tree_run(q, k, v, ones, o, lse)
    assert e.value.status == 6
    assert ws.get_error() == 0


# ---- the accepted path ---------------------------------------------------------------------------------

COMMITS = [
    # l_q, l_kv, KV heads, page, dtype, layout, path length
    ([1], [1], 1, 1, "bf16", "HND", 1),
    ([16, 9, 0, 30], [116, 9, 40, 333], 2, 16, "bf16", "HND", 7),
    ([64, 50], [80, 700], 8, 32, "bf16", "NHD", 64),          # paths over several groups of rows
    ([5, 8], [3, 8], 2, 5, "bf16", "HND", 6),                 # a token without a slot, an odd page size
    ([16, 9, 0, 30], [116, 9, 40, 333], 3, 8, "e4m3", "HND", 7),
    ([60] * 40, [60 + 3 * i for i in range(40)], 4, 16, "e4m3", "NHD", 33),
]


@pytest.mark.parametrize("case", COMMITS, ids=range(len(COMMITS)))
def test_commit(case):
    torch = torch_mod()
    lq, lkv, hk, ps, dtype, layout, length = case
    b = batch_of(lq, lkv, hk, hk, ps, False, seed=ps + hk)
    rng = np.random.default_rng(ps)
    path = np.full((len(lq), length), -1, np.int32)
    for i, n in enumerate(lq):
        first = max(0, n - lkv[i])  # tokens before the first key have no slot
        m = min(length, n - first, int(rng.integers(0, n + 1)) + (i % 2))
        path[i, :m] = np.sort(rng.permutation(np.arange(first, n))[:m])
        path[i, m + 1:] = 7  # behind the path's end
    ws = workspace(b, layout=layout, dtype=dtype)
    if dtype == "bf16":
        k0, v0 = as_layout(b.k_pages, layout), as_layout(b.v_pages, layout)
        k, v = bf16(k0), bf16(v0)
    else:
        k0, v0 = (as_layout(rng.integers(0, 256, size=b.k_pages.shape).astype(np.uint8), layout) for _ in range(2))
        k, v = dev(k0), dev(v0)
    ws.tree_commit(dev(path), k, v)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    ended = np.where(np.cumsum(path < 0, 1) > 0, -1, path)
    for got, want in zip((k, v), P.commit(b, ended, [k0, v0], layout)):
        assert np.array_equal(bits(got) if dtype == "bf16" else got.cpu().numpy(), want)


def test_commit_skips_bad_entries():
    """Entries that do not ascend or lie outside the request are skipped and reported; no other slot is touched."""
    torch = torch_mod()
    b = batch_of([8, 8], [20, 50], 2, 2, 4, False, seed=4)
    ws = workspace(b)
    k0, v0 = b.k_pages, b.v_pages
    k, v = bf16(k0), bf16(v0)
    path = np.array([[2, 2, 5, 8, 2 ** 31 - 1], [1, 0, 7, -1, 3]], np.int32)
    ws.tree_commit(dev(path), k, v)
    torch.cuda.synchronize()
    assert ws.get_error() == B.DEVERR_KEPT and ws.get_error() == 0
    want_k, want_v = k0.copy(), v0.copy()
    for i, j, e in ((0, 0, 2), (0, 2, 5), (1, 0, 1), (1, 2, 7)):
        (fp,), (fs,) = P.places(b, i, [(12, 42)[i] + e])
        (tp,), (ts,) = P.places(b, i, [(12, 42)[i] + j])
        want_k[tp, :, ts], want_v[tp, :, ts] = k0[fp, :, fs], v0[fp, :, fs]
    assert np.array_equal(bits(k), want_k) and np.array_equal(bits(v), want_v)


def test_commit_refusals():
    torch = torch_mod()
    b = batch_of([3, 3], [9, 20], 2, 2, 16, False)
    ws = workspace(b)
    k, v = bf16(b.k_pages), bf16(b.v_pages)
    path = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    for args in ((path[:1], k, v), (path.long(), k, v), (path, k[:, :1], v), (path, k, v.float()), (path.cpu(), k, v)):
        with pytest.raises(ValueError):
            ws.tree_commit(*args)
    with pytest.raises(B.FiError) as e:
        ws.tree_commit(path[:, :0], k, v)
    assert e.value.status == 1
    same = b.kv_indices.copy()
    same[-1] = same[0]  # the page of request 0's tokens takes request 1's, too
    ws.plan(b.qo_indptr, b.kv_indptr, same, b.last_page_len, 16, False)
    with pytest.raises(B.FiError) as e:
        ws.tree_commit(path, k, v)
    assert e.value.status == 3
    assert np.array_equal(bits(k), b.k_pages) and np.array_equal(bits(v), b.v_pages)


# ---- bounds, scores, choice ------------------------------------------------------------------------------

BOUNDS = [
    # l_q, l_kv, KV heads, page, dtype, layout
    ([1], [1], 1, 1, "bf16", "HND"),
    ([1, 0, 17, 300], [40, 33, 17, 900], 2, 16, "bf16", "HND"),
    ([2, 1, 1], [7, 64, 129], 8, 64, "bf16", "NHD"),
    ([9, 3], [5, 0], 3, 8, "bf16", "HND"),                        # more tokens than keys, no keys
    ([1, 2], [30, 11], 1, 5, "bf16", "HND"),
    ([130, 1], [1000, 300], 4, 128, "bf16", "HND"),
    ([1, 0, 17, 300], [40, 33, 17, 900], 2, 16, "e4m3", "NHD"),
    ([1, 1], [500, 3], 4, 128, "e4m3", "HND"),
    ([1, 1, 1], [5, 4, 1], 2, 4, "e4m3", "HND"),
    ([1] * 200, [2 * i + 1 for i in range(200)], 8, 8, "e4m3", "HND"),
]


@pytest.mark.parametrize("new_keys", [False, True])
@pytest.mark.parametrize("case", BOUNDS, ids=range(len(BOUNDS)))
def test_bounds(case, new_keys):
    torch = torch_mod()
    lq, lkv, hk, ps, dtype, layout = case
    b = batch_of(lq, lkv, hk, hk, ps, False, seed=ps + hk)
    k, kv = pool(b, "k_pages", dtype, layout, 1.0, spread=3.0)
    # slots behind the last key hold NaN: they are not looked at
    raw = k.view(torch.uint8 if dtype == "e4m3" else torch.int16)
    for i, n in enumerate(lkv):
        if n % ps:
            page = int(b.kv_indices[b.kv_indptr[i + 1] - 1])
            (raw[page][:, n % ps:] if layout == "HND" else raw[page][n % ps:]).fill_(0x7F if dtype == "e4m3" else 0x7FC0)
    ws = workspace(b, layout=layout, dtype=dtype, scales=(0.5, 1.0))
    old = torch.full((b.num_pages, hk, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = old.clone()
    ws.page_bounds(k, got, new_keys=new_keys)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    assert np.array_equal(f64(got), P.page_bounds(b, kv, f64(old), new_keys, layout))


def test_bounds_of_nan_infinite_and_signed_zero_keys():
    torch = torch_mod()
    b = batch_of([1], [16], 1, 1, 16, False)
    k = bf16(b.k_pages)
    page = int(b.kv_indices[0])
    k[page, 0, 3, 0] = float("nan")
    k[page, 0, 4, 1], k[page, 0, 5, 1] = float("inf"), -float("inf")
    k[page, 0, :, 2] = -0.0
    got = torch.zeros(b.num_pages, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    ws = workspace(b)
    ws.page_bounds(k, got)
    lo, hi = f64(got)[page, 0]
    assert np.isnan(lo[0]) and np.isnan(hi[0]) and lo[1] == -np.inf and hi[1] == np.inf and lo[2] == 0 and hi[2] == 0
    assert np.array_equal(lo[3:], f64(k)[page, 0].min(0)[3:]) and np.array_equal(hi[3:], f64(k)[page, 0].max(0)[3:])


SCORES = [
    # l_q, l_kv, query heads, KV heads, page, causal, row slack
    ([1], [1], 1, 1, 16, False, 0),
    ([1, 1, 0, 1], [500, 17, 60, 1024], 8, 2, 16, False, 3),
    ([4, 3, 1], [600, 2, 40], 12, 4, 8, True, 0),                  # three heads a group, more tokens than keys
    ([2, 5], [300, 299], 10, 2, 16, True, 1),                      # five
    ([1, 2], [900, 64], 7, 1, 32, False, 0),
    ([3, 1], [500, 129], 24, 2, 8, True, 0),                       # twelve: two sets of columns
    ([2], [333], 33, 1, 16, False, 0),
    ([40, 20], [700, 20], 8, 8, 16, True, 0),                      # a prompt's tokens
    ([1, 1], [40, 0], 4, 2, 1, True, 0),
    ([2, 1] * 40, [3 + 7 * (i % 40) for i in range(80)], 4, 2, 4, False, 0),
    ([7, 0, 2, 1], [900, 40, 2, 333], 16, 2, 16, True, 2),         # more than eight columns, eight heads a group
    ([13, 1], [413, 20], 8, 2, 16, False, 0),                      # four
    ([9, 17], [109, 700], 4, 2, 8, True, 0),                       # two
    ([6, 3], [777, 3], 18, 3, 32, True, 1),                        # six
    ([1, 3], [600, 90], 64, 4, 16, True, 0),                       # sixteen
    ([2, 1], [520, 33], 40, 2, 16, False, 0),                      # twenty
    ([70, 3, 0, 33], [500, 90, 50, 1033], 16, 2, 16, True, 0),     # a block's tokens in sixteen parts
]


@pytest.mark.parametrize("case", SCORES, ids=range(len(SCORES)))
def test_scores(case):
    torch = torch_mod()
    lq, lkv, hq, hk, ps, causal, slack = case
    b = batch_of(lq, lkv, hq, hk, ps, causal, seed=ps + hq, scale=1.5)
    rng = np.random.default_rng(hq)
    lo = rng.standard_normal((b.num_pages, hk, 128)).astype(np.float32)
    both = np.stack([lo, lo + np.abs(rng.standard_normal(lo.shape).astype(np.float32)) * 2], 2)
    bounds = bf16(W.f32_to_bf16_bits(both))
    row = max(1, int(np.diff(b.kv_indptr).max()) + slack)
    scores = torch.full((b.total_q, hk, row), 5.0, device="cuda")
    q = bf16(b.q)
    ws = workspace(b, dtype="e4m3", scales=(0.25, 1.0)) if ps in (8, 16) else workspace(b)
    ws.score_pages(q, bounds, scores)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    want, reach = P.page_scores(b, f64(q), f64(bounds), np.full(scores.shape, 5.0), 0.25 if ps in (8, 16) else 1.0)
    got = scores.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isneginf(got), np.isneginf(want))
    fin = np.isfinite(want)
    # 256 exact products summed in fp32, 2^-24 of the sum of |terms| each, twice that for products that drop bits
    assert (np.abs(got[fin] - want[fin]) <= reach * 2.0 ** -15).all()


def test_scores_show_nan_and_infinite_bounds():
    torch = torch_mod()
    b = batch_of([1], [48], 4, 1, 16, False)
    bounds = torch.zeros(b.num_pages, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    p0, p1, p2 = (int(x) for x in b.kv_indices)
    bounds[p0, 0, 0, 3] = float("nan")
    bounds[p1, 0, 1, 7] = float("inf")
    bounds[p2, 0, 1] = 1.0
    scores = torch.zeros(1, 1, 3, device="cuda")
    q = torch.ones(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    workspace(b).score_pages(q, bounds, scores)
    s = scores.cpu().numpy()[0, 0]
    assert np.isnan(s[0]) and s[1] == np.inf and abs(s[2] - 128 ** 0.5) < 1e-4


SELECT = [
    # l_q, l_kv, KV heads, page, causal, sink, recent, budget, kind
    ([1], [1], 1, 16, False, 0, 0, 1, "normal"),
    ([1, 1, 0, 1], [500, 17, 60, 4097], 2, 16, False, 1, 2, 9, "normal"),
    ([4, 3, 2], [600, 2, 40], 4, 8, True, 1, 1, 5, "normal"),
    ([1, 1], [3000, 2999], 2, 4, False, 0, 0, 300, "ties"),
    ([1, 1], [3000, 2999], 2, 4, False, 2, 3, 700, "ties"),
    ([1], [5000], 1, 1, False, 4, 100, 1000, "equal"),
    ([1], [5000], 1, 1, False, 0, 0, 4999, "special"),
    ([1], [700], 2, 1, False, 3, 4, 7, "special"),              # nothing but sink and recent
    ([2, 1], [700, 9], 2, 1, True, 0, 5, 2 ** 20, "normal"),     # all pages
    ([1], [40_000], 1, 1, False, 4, 16, 10_000, "ties"),         # longer than the threads hold
    ([3], [20_000], 2, 1, True, 1, 0, 64, "special"),
    ([3], [16_000], 2, 1, True, 1, 0, 64, "special"),            # several warps: the last bits' few to one of them
    ([1, 2], [9000, 300], 2, 1, False, 0, 0, 1, "normal"),
    ([1], [6000], 1, 1, False, 2, 8, 2500, "near"),
    ([1, 1], [900, 513], 1, 1, False, 0, 0, 512, "near"),
]


@pytest.mark.parametrize("case", SELECT, ids=range(len(SELECT)))
def test_select(case):
    torch = torch_mod()
    lq, lkv, hk, ps, causal, sink, recent, budget, kind = case
    n = sum(-(-x // ps) for x in lkv)
    b = W.make_paged_batch(np.random.default_rng(5), "select", lq, lkv, hk, hk, ps, causal, pool_pages=n + 3, with_data=False)
    total_q = int(b.qo_indptr[-1])
    rng = np.random.default_rng(budget)
    row = int(np.diff(b.kv_indptr).max()) + 2
    x = rng.standard_normal((total_q, hk, row)).astype(np.float32) * 8
    if kind == "ties":
        x = np.round(x)
    elif kind == "equal":
        x[:] = -3.5
    elif kind == "near":
        x = 1 + np.round(x) * np.float32(2.0 ** -23)
    elif kind == "special":
        x[rng.random(x.shape) < 0.3] = -np.inf
        x[rng.random(x.shape) < 0.01] = np.nan
        x[rng.random(x.shape) < 0.01] = np.inf
        x[rng.random(x.shape) < 0.05] = -0.0
        x[rng.random(x.shape) < 0.05] = 0.0
    ws = B.Workspace(len(lq), max(total_q, 1), n, hk, hk)
    plan(ws, b)
    selected = torch.full((total_q, hk, budget), 77, dtype=torch.int32, device="cuda")
    ws.select_pages(dev(x), selected, recent=recent, sink=sink)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    assert np.array_equal(selected.cpu().numpy(), P.select_pages(b, x, sink, recent, budget))


# ---- attention over the chosen pages -----------------------------------------------------------------------

PAGES = [
    # l_q, l_kv, query heads, KV heads, page, dtype, layout, causal, cap, budget, SMs
    ([1], [1], 1, 1, 16, "bf16", "HND", False, 0.0, 1, 0),
    ([1, 1, 0, 1], [500, 17, 60, 1500], 8, 2, 16, "bf16", "HND", False, 0.0, 20, 0),
    ([4, 3, 2], [600, 2, 40], 8, 2, 8, "bf16", "HND", True, 0.0, 7, 3),
    ([1, 1], [900, 800], 16, 2, 32, "bf16", "HND", False, 0.0, 10, 0),
    ([1, 1], [300, 77], 5, 1, 5, "bf16", "HND", True, 0.0, 30, 0),        # the loader of odd page sizes
    ([1, 1], [64, 129], 4, 4, 64, "bf16", "NHD", False, 30.0, 2, 0),
    ([1] * 9, [10, 0, 2000, 64, 31, 32, 33, 1000, 1], 10, 2, 1, "bf16", "HND", False, 0.0, 400, 0),
    ([2, 3], [1000, 700], 40, 2, 16, "bf16", "HND", True, 0.0, 12, 0),     # 20 heads a group: tensor-core tiles
    ([1], [3000], 64, 1, 8, "bf16", "NHD", False, 0.0, 200, 0),            # cut over many CTAs
    ([1, 1, 0, 1], [500, 17, 60, 1500], 8, 2, 16, "e4m3", "HND", False, 0.0, 20, 0),
    ([1, 4], [400, 260], 16, 2, 64, "e4m3", "NHD", True, 30.0, 3, 5),
    ([2], [300], 2, 2, 4, "e4m3", "HND", True, 0.0, 60, 0),
    ([2, 3], [1000, 700], 24, 2, 128, "e4m3", "HND", True, 0.0, 4, 0),
    ([1] * 152, [40] * 152, 2, 1, 32, "bf16", "HND", False, 0.0, 2, 0),     # a CTA's piece ends where a unit does
    ([1] * 3, [128] * 3, 8, 1, 128, "bf16", "HND", False, 0.0, 1, 2),
]


@pytest.mark.parametrize("case", PAGES, ids=range(len(PAGES)))
def test_pages(case):
    torch = torch_mod()
    lq, lkv, hq, hk, ps, dtype, layout, causal, cap, budget, sms = case
    b = batch_of(lq, lkv, hq, hk, ps, causal, seed=ps + hq, scale=1.3)
    scales = (0.0625, 0.03125) if dtype == "e4m3" else (1.0, 1.0)
    (k, kv), (v, vv) = pool(b, "k_pages", dtype, layout, scales[0]), pool(b, "v_pages", dtype, layout, scales[1])
    rng = np.random.default_rng(budget)
    row = max(1, int(np.diff(b.kv_indptr).max()))
    selected = P.select_pages(b, rng.standard_normal((b.total_q, hk, row)), 0, 1 if budget > 1 else 0, budget)
    selected[0, 0] = -1  # a list without pages
    if b.total_q > 2:  # a list that ends before its room does
        some = selected[2, 0][selected[2, 0] >= 0]
        selected[2, 0] = -1
        selected[2, 0, :len(some) // 2] = some[:len(some) // 2]
    ws = workspace(b, cap=cap, layout=layout, dtype=dtype, scales=scales, num_sms=sms)
    q, (o, lse) = bf16(b.q), outputs(b)
    ws.run_pages(q, k, v, dev(selected), o, lse)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    ref = P.pages_attention(b, f64(q), kv, vv, selected, cap, layout)
    assert_state(o, lse, ref, F16_WEIGHTS if dtype == "e4m3" else BF16_WEIGHTS, cap)
    again = outputs(b)
    ws.run_pages(q, k, v, dev(selected), *again)
    assert np.array_equal(bits(again[0]), bits(o)) and torch.equal(again[1], lse)
    # fi_run of the same workspace has its own plan still
    (ro, rl), ref = outputs(b), A.batch_attention(b) if dtype == "bf16" and layout == "HND" and cap == 0 else None
    if ref is not None:
        ws.run(q, k, v, ro, rl)
        torch.cuda.synchronize()
        assert np.abs(f64(ro) - ref[0]).max(initial=0) <= 2e-2


def test_pages_list_with_the_end_page_elsewhere():
    """The page that is not full counts as a list's last alone: elsewhere the list is empty and reported."""
    torch = torch_mod()
    b = batch_of([1, 1], [40, 48], 4, 1, 16, False, seed=6)
    ws = workspace(b)
    q, k, v, (o, lse) = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages), outputs(b)
    first, second = b.kv_indices[:3], b.kv_indices[3:]
    selected = np.array([[first[[0, 2, 1]]], [second[[2, 0, 1]]]], np.int32)  # request 1's pages are full: any order
    ws.run_pages(q, k, v, dev(selected), o, lse)
    torch.cuda.synchronize()
    assert ws.get_error() == B.DEVERR_KEPT
    assert torch.isneginf(lse[0]).all() and (o[0] == 0).all()
    selected[0] = -1
    assert_state(o, lse, P.pages_attention(b, f64(q), f64(k), f64(v), selected), BF16_WEIGHTS)


def test_choice_replayed():
    """Bounds, scores, choice and attention captured in one graph on a small batch and replayed on a larger one, and on none."""
    torch = torch_mod()
    small = batch_of([1], [20], 8, 2, 16, True, seed=1)
    large = batch_of([2, 1, 3], [900, 1500, 64], 8, 2, 16, True, seed=2)
    none = batch_of([], [], 8, 2, 16, True, seed=3)
    pages = large.num_pages + 40
    rng = np.random.default_rng(1)
    k, v = (bf16(W.f32_to_bf16_bits(rng.standard_normal((pages, 2, 16, 128)).astype(np.float32))) for _ in range(2))
    q = bf16(W.f32_to_bf16_bits(rng.standard_normal((6, 8, 128)).astype(np.float32)))
    ws = B.Workspace(4, 6, 200, 8, 2)
    L = B.lib()
    bounds = torch.zeros(pages, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros(6, 2, 100, device="cuda")
    selected = torch.zeros(6, 2, 8, dtype=torch.int32, device="cuda")
    o, lse = torch.zeros(6, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(6, 8, device="cuda")

    def step():
        s = torch.cuda.current_stream().cuda_stream
        h = ws.handle
        assert L.fi_page_bounds(h, k.data_ptr(), pages, 0, bounds.data_ptr(), s) == 0
        assert L.fi_score_pages(h, q.data_ptr(), bounds.data_ptr(), pages, scores.data_ptr(), 100, s) == 0
        assert L.fi_select_pages(h, scores.data_ptr(), 100, 1, 1, 8, selected.data_ptr(), s) == 0
        assert L.fi_run_pages(h, q.data_ptr(), k.data_ptr(), v.data_ptr(), pages, selected.data_ptr(), 8, o.data_ptr(), lse.data_ptr(), s) == 0

    plan(ws, small)
    g = capture(step)
    for b in (large, none, small):
        n = b.total_q
        plan(ws, b)
        o.fill_(9.0)
        g.replay()
        torch.cuda.synchronize()
        assert ws.get_error() == 0
        assert (o[n:] == 9.0).all()  # rows behind the last token are as they were
        if n == 0:
            continue
        kv, vv = A.bf16_to_f64(bits(k)), A.bf16_to_f64(bits(v))
        want = P.page_bounds(b, kv, np.zeros(bounds.shape), False)
        used = b.kv_indices[:int(b.kv_indptr[-1])]
        assert np.array_equal(f64(bounds)[used], want[used])
        sc = scores[:n].cpu().numpy()
        sel = P.select_pages(b, sc, 1, 1, 8)
        assert np.array_equal(selected[:n].cpu().numpy(), sel)
        assert_state(o[:n], lse[:n], P.pages_attention(b, f64(q)[:n], kv, vv, sel), BF16_WEIGHTS)


def test_choice_refusals():
    torch = torch_mod()
    b = batch_of([1, 1], [40, 20], 8, 2, 16, False)
    ws = workspace(b)
    q, k, v, (o, lse) = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages), outputs(b)
    bounds = torch.zeros(b.num_pages, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    scores = torch.zeros(2, 2, 3, device="cuda")
    sel = torch.full((2, 2, 2), -1, dtype=torch.int32, device="cuda")
    for call in (lambda: ws.page_bounds(k, bounds[1:]), lambda: ws.page_bounds(k, bounds.float()), lambda: ws.page_bounds(k[:, :, :8], bounds),
                 lambda: ws.score_pages(q[:1], bounds, scores), lambda: ws.score_pages(q, bounds, scores[:, :1]),
                 lambda: ws.score_pages(q, bounds, scores.double()), lambda: ws.select_pages(scores, sel.long()),
                 lambda: ws.select_pages(scores, sel[:1]), lambda: ws.run_pages(q, k, v, sel.long(), o, lse),
                 lambda: ws.run_pages(q, k, v, sel, o[:, :4], lse), lambda: ws.run_pages(q, k, v, sel.cpu(), o, lse)):
        with pytest.raises(ValueError):
            call()

    def refused(status, call):
        with pytest.raises(B.FiError) as e:
            call()
        assert e.value.status == status

    refused(1, lambda: ws.score_pages(q, bounds, scores[..., :2].contiguous()))  # a request has three pages
    refused(1, lambda: ws.select_pages(scores[..., :2].contiguous(), sel))
    refused(1, lambda: ws.select_pages(scores, sel, recent=2, sink=1))
    refused(1, lambda: ws.select_pages(scores, sel, recent=-1))
    refused(1, lambda: ws.select_pages(scores, sel[..., :0]))
    refused(1, lambda: ws.run_pages(q, k, v, sel[..., :0], o, lse))
    L, s, h = B.lib(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), ws.handle
    ptr = lambda t, off=0: t.data_ptr() + off
    assert L.fi_run_pages(h, ptr(q), ptr(k), ptr(v), b.num_pages, ptr(sel), 2, ptr(o, 8), ptr(lse), s) == 1
    assert L.fi_run_pages(h, ptr(q), ptr(k), 0, b.num_pages, ptr(sel), 2, ptr(o), ptr(lse), s) == 1
    assert L.fi_run_pages(h, ptr(q), ptr(k), ptr(v), b.num_pages, ptr(sel), 2 ** 30, ptr(o), ptr(lse), s) == 3
    assert L.fi_page_bounds(h, ptr(k), b.num_pages, 2, ptr(bounds), s) == 1
    assert L.fi_page_bounds(h, ptr(k), 1, 0, ptr(bounds), s) == 1  # pages outside the pool
    w = workspace(dataclasses.replace(b, causal=True), window=5)
    for call in (lambda: w.score_pages(q, bounds, scores), lambda: w.select_pages(scores, sel), lambda: w.run_pages(q, k, v, sel, o, lse)):
        refused(3, call)
    empty = B.Workspace(2, 2, 20, 8, 2)
    for call in (lambda: empty.page_bounds(k, bounds), lambda: empty.score_pages(q, bounds, scores), lambda: empty.select_pages(scores, sel),
                 lambda: empty.run_pages(q, k, v, sel, o, lse), lambda: empty.tree_commit(sel[0], k, v)):
        refused(6, call)
    three = batch_of([1], [40], 3, 3, 16, False)  # three KV heads, token-major
    t = workspace(three)
    t.set_variant(kv_layout="NHD")
    refused(3, lambda: plan(t, three))
    assert ws.get_error() == 0


# ---- together ----------------------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_speculative_steps(dtype):
    """Two rounds of drafting over chosen pages, verifying the tree, and committing the path, against a cache kept on the host."""
    torch = torch_mod()
    rng = np.random.default_rng(8)
    hq, hk, ps = 8, 2, 16
    scales = (0.0625, 0.03125) if dtype == "e4m3" else (1.0, 1.0)
    lens, pages = np.array([500, 77]), 64
    lists = [rng.permutation(pages)[:40], None]
    lists[1] = np.setdiff1d(np.arange(pages), lists[0])[:20]
    ws = B.Workspace(2, 32, 64, hq, hk)
    ws.set_kv_dtype(dtype, *scales)
    kind = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    k, v = ((torch.randn(pages, hk, ps, 128, device="cuda") / s).to(kind) for s in scales)
    bounds = torch.zeros(pages, hk, 2, 128, dtype=torch.bfloat16, device="cuda")
    weights = F16_WEIGHTS if dtype == "e4m3" else BF16_WEIGHTS

    def batch(lq, lkv):
        kv = np.concatenate([x[:-(-n // ps)] for x, n in zip(lists, lkv)]).astype(np.int32)
        n = [-(-x // ps) for x in lkv]
        return W.PagedBatch(name="step", num_qo_heads=hq, num_kv_heads=hk, head_dim=128, page_size=ps, causal=True,
                            qo_indptr=np.concatenate([[0], np.cumsum(lq)]).astype(np.int32), kv_indptr=np.concatenate([[0], np.cumsum(n)]).astype(np.int32),
                            kv_indices=kv, last_page_len=np.array([x - (m - 1) * ps for x, m in zip(lkv, n)], np.int32), q=None, k_pages=None, v_pages=None)

    def values(x, s):
        return f64(x) * s

    def rows(n):
        return torch.randn(n, hq + 2 * hk, 128, device="cuda").to(torch.bfloat16)

    for turn in range(2):
        # a draft token over eight pages of each request
        b = batch([1, 1], lens + 1)
        plan(ws, b)
        x = rows(2)
        q = torch.empty(2, hq, 128, dtype=torch.bfloat16, device="cuda")
        ws.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], k, v, q)
        ws.page_bounds(k, bounds, new_keys=turn > 0)
        scores, sel = torch.zeros(2, hk, 40, device="cuda"), torch.zeros(2, hk, 8, dtype=torch.int32, device="cuda")
        ws.score_pages(q, bounds, scores)
        ws.select_pages(scores, sel, recent=1, sink=1)
        o, lse = torch.empty_like(q), torch.empty(2, hq, device="cuda")
        ws.run_pages(q, k, v, sel, o, lse)
        host = P.select_pages(b, scores.cpu().numpy(), 1, 1, 8)
        assert np.array_equal(sel.cpu().numpy(), host)
        want, reach = P.page_scores(b, f64(q), P.page_bounds(b, f64(k), f64(bounds), False), np.zeros(scores.shape), scales[0])
        assert np.abs(scores.cpu().numpy() - want).max() <= reach * 2.0 ** -15  # the bounds are those of the whole cache
        assert_state(o, lse, P.pages_attention(b, f64(q), values(k, scales[0]), values(v, scales[1]), host), weights)
        # a tree behind the context, verified, one path of it kept
        lq = [9, 14]
        b = batch(lq, lens + lq)
        plan(ws, b)
        x = rows(23)
        q = torch.empty(23, hq, 128, dtype=torch.bfloat16, device="cuda")
        ws.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], k, v, q)
        parents = np.concatenate([[rng.integers(-1, t) if t else -1 for t in range(n)] for n in lq])
        mask = B.tree_mask(b.qo_indptr, parents)
        o, lse = torch.empty_like(q), torch.empty(23, hq, device="cuda")
        ws.tree_run(q, k, v, dev(mask), o, lse)
        torch.cuda.synchronize()
        assert_state(o, lse, P.tree_attention(b, f64(q), values(k, scales[0]), values(v, scales[1]), mask, q_floor=Q_FLOOR if dtype == "e4m3" else 0.0), weights)
        path = np.full((2, 5), -1, np.int32)
        for i, n in enumerate(lq):
            up, leaf = [], int(rng.integers(0, n))
            while leaf >= 0:
                up.append(leaf)
                leaf = int(parents[b.qo_indptr[i] + leaf])
            up = up[::-1][:5]
            path[i, :len(up)] = up
        raw = lambda t: t.view(torch.int16 if dtype == "bf16" else torch.uint8).cpu().numpy()
        want = P.commit(b, path, [raw(k), raw(v)])
        ws.tree_commit(dev(path), k, v)
        torch.cuda.synchronize()
        assert np.array_equal(raw(k), want[0]) and np.array_equal(raw(v), want[1])
        ws.page_bounds(k, bounds, new_keys=True)  # of what the tree's slots hold now, the refused tokens' too
        lens = lens + (path >= 0).sum(1)
        plan(ws, batch((path >= 0).sum(1), lens))
        ws.page_bounds(k, bounds, new_keys=True)
        assert ws.get_error() == 0


# ---- where calls can get in each other's way -----------------------------------------------------------


def every_call(b, ws, q, k, v, mask, path, stream=None):
    """The outputs of each operator on the batch, the pools' changes last (k and v are the call's own)."""
    torch = torch_mod()
    hk, row = b.num_kv_heads, int(np.diff(b.kv_indptr).max())
    (o, lse), (po, plse) = outputs(b), outputs(b)
    bounds = torch.empty(k.shape[0], hk, 2, 128, dtype=torch.bfloat16, device="cuda")
    scores = torch.full((b.total_q, hk, row), 3.0, device="cuda")
    sel = torch.empty(b.total_q, hk, 5, dtype=torch.int32, device="cuda")
    ws.tree_run(q, k, v, mask, o, lse, stream=stream)
    ws.page_bounds(k, bounds, stream=stream)
    ws.score_pages(q, bounds, scores, stream=stream)
    ws.select_pages(scores, sel, recent=1, stream=stream)
    ws.run_pages(q, k, v, sel, po, plse, stream=stream)
    ws.tree_commit(path, k, v, stream=stream)
    return o, lse, scores, sel, po, plse, bounds


def case_of(seed, lq, lkv, dtype="bf16"):
    b = batch_of(lq, lkv, 8, 2, 16, False, seed=seed)
    mask = dev(random_mask(np.random.default_rng(seed), b, "tree"))
    path = dev(np.array([[i for i in range(1, n, 2)][:6] + [-1] * (6 - len(range(1, n, 2)[:6])) for n in lq], np.int32))
    return b, bf16(b.q), bf16(b.k_pages), bf16(b.v_pages), mask, path


def same(x, y):
    return all(torch_mod().equal(a, c) for a, c in zip(x, y))


def test_far_pages():
    """Pages behind 2^32 bytes and 2^31 elements of a pool: bit for bit what the same pages give at its beginning."""
    torch = torch_mod()
    b = batch_of([20, 1, 40], [400, 33, 900], 32, 8, 16, False, seed=4)
    far = 140_000
    mask = dev(random_mask(np.random.default_rng(1), b, "tree"))
    path = dev(np.array([[3, 7, 19, -1], [-1, -1, -1, -1], [1, 2, 30, 39]], np.int32))
    q, k, v = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages)
    big = [torch.empty(far + x.shape[0], *x.shape[1:], dtype=x.dtype, device="cuda") for x in (k, v)]
    for x, near in zip(big, (k, v)):
        x[far:] = near
    c = dataclasses.replace(b, kv_indices=(b.kv_indices + far).astype(np.int32))
    near = every_call(b, workspace(b), q, k, v, mask, path)
    ws = workspace(c)
    got = every_call(c, ws, q, *big, mask, path)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    used = dev(np.unique(b.kv_indices)).long()
    assert same(near[:3], got[:3]) and same(near[4:6], got[4:6])
    assert torch.equal(torch.where(near[3] >= 0, near[3] + far, near[3]), got[3])
    assert torch.equal(near[6][used], got[6][used + far])
    assert torch.equal(big[0][far:], k) and torch.equal(big[1][far:], v)


def test_two_streams_at_once():
    """Two workspaces on two streams, their launches side by side, against the same calls alone."""
    torch = torch_mod()
    cases = [case_of(5, [30, 9, 16] * 20, [3000, 90, 800] * 20), case_of(6, [12] * 90, [333] * 90)]
    want, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for b, q, k, v, mask, path in cases:
        kc, vc = k.clone(), v.clone()
        want.append((every_call(b, workspace(b), q, kc, vc, mask, path), kc, vc))
    spaces = [workspace(c[0]) for c in cases]
    torch.cuda.synchronize()
    for turn in range(4):
        got = []
        for ws, s, (b, q, k, v, mask, path) in zip(spaces, streams, cases):
            with torch.cuda.stream(s):  # the outputs are made there, too
                kc, vc = k.clone(), v.clone()
                got.append((every_call(b, ws, q, kc, vc, mask, path, stream=s if turn % 2 else None), kc, vc))
        torch.cuda.synchronize()
        for (x, xk, xv), (y, yk, yv), (b, *_) in zip(got, want, cases):
            used = dev(np.unique(b.kv_indices)).long()
            assert same(x[:6], y[:6]) and torch.equal(x[6][used], y[6][used]) and torch.equal(xk, yk) and torch.equal(xv, yv)


@pytest.mark.parametrize("apart", [False, True], ids=["one stream", "plans on another stream"])
def test_plans_and_calls_in_turn(apart):
    """New plans between calls of one workspace, nothing waited for on the host: each call sees its own plan."""
    torch = torch_mod()
    plans, calls = (torch.cuda.Stream(), torch.cuda.Stream()) if apart else (None, torch.cuda.current_stream())
    cases = [case_of(7, [30, 9, 16] * 20, [3000, 90, 800] * 20), case_of(8, [12, 1] * 30, [333, 20] * 30), case_of(9, [5], [16_000])]
    ws = B.Workspace(60, 1100, 14_000, 8, 2)
    want = []
    for b, q, k, v, mask, path in cases:
        kc, vc = k.clone(), v.clone()
        want.append((every_call(b, workspace(b), q, kc, vc, mask, path), kc, vc))
        torch.cuda.synchronize()
    got = []
    for turn in range(12):
        b, q, k, v, mask, path = cases[turn % 3]
        with torch.cuda.stream(calls):
            kc, vc = k.clone(), v.clone()
            if apart:
                plans.wait_stream(calls)
            ws.plan(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, b.page_size, b.causal, stream=plans if apart else calls)
            kc.add_(0)  # a kernel between the plan's copy and the calls, or beside it
            if apart:
                calls.wait_stream(plans)
            got.append((every_call(b, ws, q, kc, vc, mask, path), kc, vc))
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    for turn, (x, xk, xv) in enumerate(got):
        y, yk, yv = want[turn % 3]
        used = dev(np.unique(cases[turn % 3][0].kv_indices)).long()
        assert same(x[:6], y[:6]) and torch.equal(x[6][used], y[6][used]) and torch.equal(xk, yk) and torch.equal(xv, yv)


# ---- where tensors may lie ------------------------------------------------------------------------------


def moved(t):
    """A copy of t whose data begin at the smallest offset that the calls allow behind an allocation's own alignment: 16 bytes
    for rows of 128 elements, 4 for the others."""
    torch = torch_mod()
    off = (16 if t.shape[-1] == 128 else 4) // t.element_size()
    flat = torch.empty(t.numel() + off, dtype=t.dtype, device="cuda")
    out = flat[off:].view(t.shape)
    out.copy_(t)
    assert out.is_contiguous() and out.data_ptr() % 32 == off * t.element_size()
    return out


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq", [8, 24], ids=["4 heads a group", "12"])
def test_tensors_at_the_smallest_alignment(hq, dtype):
    """Every operator on tensors that begin 16 bytes (rows of a head) or 4 bytes (all else) behind a multiple of 32: bit for bit as on
    tensors of their own.  Trees with whole units and with cut ones, lists on both kinds of tiles."""
    torch = torch_mod()
    for lq, lkv in (([30, 4, 64], [2000, 4, 900]), ([3] * 200, [60] * 200)):
        b = batch_of(lq, lkv, hq, 2, 16, False, seed=hq)
        q, k, v = bf16(b.q), pool(b, "k_pages", dtype, "HND", 1.0)[0], pool(b, "v_pages", dtype, "HND", 1.0)[0]
        mask = dev(random_mask(np.random.default_rng(1), b, "tree"))
        path = dev(np.array([[0, 2, -1]] * len(lq), np.int32))
        ws = workspace(b, dtype=dtype)
        row = int(np.diff(b.kv_indptr).max())

        def calls(at):
            kc, vc, qc = at(k.clone()), at(v.clone()), at(q)
            (o, lse), (po, plse) = (tuple(at(x) for x in outputs(b)) for _ in range(2))
            bounds = at(torch.zeros(b.num_pages, 2, 2, 128, dtype=torch.bfloat16, device="cuda"))
            scores = at(torch.full((b.total_q, 2, row), 3.0, device="cuda"))
            sel = at(torch.zeros(b.total_q, 2, 5, dtype=torch.int32, device="cuda"))
            ws.tree_run(qc, kc, vc, at(mask), o, lse)
            ws.page_bounds(kc, bounds)
            ws.score_pages(qc, bounds, scores)
            ws.select_pages(scores, sel, recent=1)
            ws.run_pages(qc, kc, vc, sel, po, plse)
            ws.tree_commit(at(path), kc, vc)
            torch.cuda.synchronize()
            return o, lse, bounds, scores, sel, po, plse, kc.view(torch.uint8), vc.view(torch.uint8)

        want, got = calls(lambda t: t), calls(moved)
        assert ws.get_error() == 0
        assert same(want, got)


def record(call):
    """The call in a graph, with no call before it."""
    torch = torch_mod()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        call()
    torch.cuda.synchronize()
    return g


@pytest.mark.parametrize("hq,most", [(16, 64), (16, 4), (4, 64)], ids=["few of many tokens", "all tokens", "decode tiles"])
def test_lists_of_a_workspace_whose_first_call_is_captured(hq, most):
    """Lists cut over many CTAs, replayed from a capture with no call before it, the grid made for more tokens than the plan has."""
    torch = torch_mod()
    b = batch_of([2, 1, 1], [3000, 900, 40], hq, 1, 16, True, seed=4)
    ws = B.Workspace(8, most, 400, hq, 1)
    plan(ws, b)
    q, k, v, (o, lse) = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages), outputs(b)
    row = int(np.diff(b.kv_indptr).max())
    selected = P.select_pages(b, np.random.default_rng(0).standard_normal((4, 1, row)), 0, 1, 150)
    sel = dev(selected)
    g = record(lambda: ws.run_pages(q, k, v, sel, o, lse))
    for _ in range(2):
        o.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert ws.get_error() == 0
        assert_state(o, lse, P.pages_attention(b, f64(q), f64(k), f64(v), selected), BF16_WEIGHTS)


@pytest.mark.parametrize("hq", [8, 24], ids=["decode tiles", "tensor-core tiles"])
def test_capture_of_calls_on_a_plan_without_tokens(hq):
    """Every call of a step is accepted, and the graph does nothing on a plan without tokens.  What was captured on decode tiles follows
    a later plan; trees and lists on tensor-core tiles hold the capture's tokens and are left out."""
    torch = torch_mod()
    none, b = batch_of([], [], hq, 2, 16, True, seed=3), batch_of([2, 1], [90, 40], hq, 2, 16, True, seed=4)
    ws = B.Workspace(2, 3, 40, hq, 2)
    q, k, v = bf16(b.q), bf16(b.k_pages), bf16(b.v_pages)
    o, lse, to, tl = (torch.full(s, 9.0, dtype=t, device="cuda") for s, t in
                      (((3, hq, 128), torch.bfloat16), ((3, hq), torch.float32), ((3, hq, 128), torch.bfloat16), ((3, hq), torch.float32)))
    mask, path = torch.ones(3, 1, dtype=torch.int32, device="cuda"), torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    bounds, scores = torch.zeros(b.num_pages, 2, 2, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 2, 6, device="cuda")
    sel = torch.full((3, 2, 6), 7, dtype=torch.int32, device="cuda")
    L, h, n = B.lib(), ws.handle, b.num_pages

    def step():
        s = torch.cuda.current_stream().cuda_stream
        x = lambda t: t.data_ptr()
        assert L.fi_page_bounds(h, x(k), n, 0, x(bounds), s) == 0
        assert L.fi_score_pages(h, x(q), x(bounds), n, x(scores), 6, s) == 0
        assert L.fi_select_pages(h, x(scores), 6, 0, 0, 6, x(sel), s) == 0
        assert L.fi_run_pages(h, x(q), x(k), x(v), n, x(sel), 6, x(o), x(lse), s) == 0
        assert L.fi_tree_run(h, x(q), x(k), x(v), n, x(mask), 1, x(to), x(tl), s) == 0
        assert L.fi_tree_commit(h, x(path), 1, x(k), x(v), n, s) == 0

    plan(ws, none)
    g = record(step)
    g.replay()
    torch.cuda.synchronize()
    assert ws.get_error() == 0 and (o == 9).all() and (lse == 9).all() and (sel == 7).all() and (scores == 0).all() and (bounds == 0).all()
    plan(ws, b)
    g.replay()
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    host = P.select_pages(b, scores.cpu().numpy(), 0, 0, 6)
    assert np.array_equal(sel.cpu().numpy(), host) and (to == 9).all()
    if hq == 24:
        assert (o == 9).all()
    else:
        assert_state(o, lse, P.pages_attention(b, f64(q), f64(k), f64(v), host), BF16_WEIGHTS)


@pytest.mark.parametrize("dtype,inter", [("bf16", False), ("bf16", True), ("e4m3", False)])
def test_tree_with_rotary_positions(dtype, inter):
    """Trees appended at their depths: q and the tree's keys against a rotation by depth, the attention against the oracle on them, and the
    committed path bit for bit as an append of its tokens alone."""
    torch = torch_mod()
    rng = np.random.default_rng(21)
    hq, hk, ps, lq, ctx = 8, 2, 16, [13, 30, 1], [300, 47, 16]
    scales = (0.0625, 0.03125) if dtype == "e4m3" else (1.0, 1.0)
    b = batch_of(lq, [c + n for c, n in zip(ctx, lq)], hq, hk, ps, True, seed=2)
    inv_freq = 10000.0 ** (-np.arange(0, 128, 2) / 128)
    kind = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    k, v = ((torch.randn(b.num_pages, hk, ps, 128, device="cuda") / s).to(kind) for s in scales)
    k0, v0 = k.clone(), v.clone()
    x = torch.randn(b.total_q, hq + 2 * hk, 128, device="cuda").to(torch.bfloat16)
    parents = np.concatenate([[rng.integers(max(-1, t - 4), t) if t else -1 for t in range(n)] for n in lq])
    depth = np.zeros(b.total_q, np.int64)  # by walking up, one token at a time
    for i, n in enumerate(lq):
        for t in range(n):
            up = parents[b.qo_indptr[i] + t]
            while up >= 0:
                depth[b.qo_indptr[i] + t] += 1
                up = parents[b.qo_indptr[i] + up]
    positions = np.repeat(ctx, lq) + depth
    given = B.tree_positions(b.qo_indptr, parents, ctx)
    assert np.array_equal(given, positions)

    ws = workspace(b, dtype=dtype, scales=scales)
    ws.set_rope(inv_freq, inter)
    q, (o, lse) = torch.empty(b.total_q, hq, 128, dtype=torch.bfloat16, device="cuda"), outputs(b)
    ws.append(x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:], k, v, q, positions=dev(given))
    mask = B.tree_mask(b.qo_indptr, parents)
    ws.tree_run(q, k, v, dev(mask), o, lse)
    torch.cuda.synchronize()
    # the rotation by depth: rounded once, 2^-19 of the row's largest for the fp32 steps and the angle before that
    rq, rk = (C.norm_rotate(f64(x[:, s]), None, 0.0, inv_freq, positions.astype(np.float64), inter) for s in (slice(0, hq), slice(hq, hq + hk)))
    slack = lambda r: np.abs(r).max(-1, keepdims=True) * 2.0 ** -19
    assert (np.abs(f64(q) - rq) <= np.abs(rq) * 2.0 ** -8 + slack(rq)).all()
    tok, page, slot, _ = C.append_places(b)
    rows = f64(k)[page, :, slot] * scales[0]
    step = np.abs(rk[tok]) * 2.0 ** -8 if dtype == "bf16" else np.maximum(np.abs(rk[tok]) * 2.0 ** -4, scales[0] * 2.0 ** -10)
    assert (np.abs(rows - rk[tok]) <= step + slack(rk[tok])).all()
    assert_state(o, lse, P.tree_attention(b, f64(q), f64(k) * scales[0], f64(v) * scales[1], mask, q_floor=Q_FLOOR if dtype == "e4m3" else 0.0),
                 F16_WEIGHTS if dtype == "e4m3" else BF16_WEIGHTS)

    # the path to a leaf, committed; beside it the same tokens appended as a chain
    path = np.full((3, 30), -1, np.int32)
    for i, n in enumerate(lq):
        up, at = [], n - 1
        while at >= 0:
            up.append(at)
            at = int(parents[b.qo_indptr[i] + at])
        path[i, :len(up)] = up[::-1]
    taken = (path >= 0).sum(1)
    assert taken.max() > 3 and (depth[b.qo_indptr[1:] - 1] == taken - 1).all()
    ws.tree_commit(dev(path), k, v)
    keep = dev(np.concatenate([b.qo_indptr[i] + path[i, :n] for i, n in enumerate(taken)])).long()
    lkv = np.array(ctx) + taken
    n = -(-lkv // ps)
    lists = np.concatenate([b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i] + m] for i, m in enumerate(n)])
    ws2 = B.Workspace(3, 44, 64, hq, hk)
    ws2.set_kv_dtype(dtype, *scales)
    ws2.set_rope(inv_freq, inter)
    ws2.plan(np.concatenate([[0], np.cumsum(taken)]), np.concatenate([[0], np.cumsum(n)]), lists, lkv - (n - 1) * ps, ps, True)
    y = x[keep]
    ws2.append(y[:, :hq], y[:, hq:hq + hk], y[:, hq + hk:], k0, v0, torch.empty(len(keep), hq, 128, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    assert ws.get_error() == 0 and ws2.get_error() == 0
    for i in range(3):
        for j in range(ctx[i], int(lkv[i])):
            p, s = int(b.kv_indices[b.kv_indptr[i] + j // ps]), j % ps
            assert torch.equal(k[p, :, s].view(torch.uint8), k0[p, :, s].view(torch.uint8)) and torch.equal(v[p, :, s].view(torch.uint8), v0[p, :, s].view(torch.uint8))


@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("k_scale", [1.0, 2.0 ** -24, 2.0 ** -149])
def test_tree_rows_of_the_smallest_numbers(k_scale, cap):
    """e4m3 pages: rows of q down to bf16's smallest number, under scales whose product with a row's own leaves fp32's range."""
    torch = torch_mod()
    b = batch_of([5, 40], [300, 700], 8, 2, 16, False, seed=12)
    (k, kv), (v, vv) = pool(b, "k_pages", "e4m3", "HND", 1.0), pool(b, "v_pages", "e4m3", "HND", 1.0)
    q, (o, lse) = bf16(b.q), outputs(b)
    q[::2] = (q[::2].double() * 2.0 ** -126).to(torch.bfloat16)
    q[4], q[6] = 2.0 ** -133, -(2.0 ** -126)
    mask = random_mask(np.random.default_rng(0), b, "tree")
    ws = workspace(b, dtype="e4m3", scales=(k_scale, 1.0), cap=cap)
    ws.tree_run(q, k, v, dev(mask), o, lse)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    assert_state(o, lse, P.tree_attention(b, f64(q), kv * k_scale, vv, mask, cap, q_floor=Q_FLOOR), F16_WEIGHTS, cap)


@pytest.mark.parametrize("big", [2.0 ** 4, 2.0 ** 9, 2.0 ** 20])
def test_tree_rows_with_one_large_element(big):
    """e4m3 pages: a dim of q far above the others, whose elements fall below 2^-9 of it and are rounded to 2^-17 of it."""
    torch = torch_mod()
    b = batch_of([5, 40], [300, 700], 8, 2, 16, False, seed=13)
    (k, kv), (v, vv) = pool(b, "k_pages", "e4m3", "HND", 1.0), pool(b, "v_pages", "e4m3", "HND", 1.0)
    raw = k.view(torch.uint8)
    raw[..., 7] = 0  # where the large element meets zeros the others decide
    kv = A.e4m3_to_f64(raw.cpu().numpy())
    q, (o, lse) = bf16(b.q), outputs(b)
    q[:, :, 7] = big
    mask = random_mask(np.random.default_rng(0), b, "tree")
    ws = workspace(b, dtype="e4m3")
    ws.tree_run(q, k, v, dev(mask), o, lse)
    torch.cuda.synchronize()
    assert ws.get_error() == 0
    # an element is off by half of the second term's smallest step, 2^-10 where the row's largest is 128 or more: 2^-17 of the largest at most
    ref = P.tree_attention(b, f64(q), kv, vv, mask)
    off = big * 2.0 ** -17 / np.sqrt(128)
    for i, (q0, q1) in enumerate(zip(b.qo_indptr[:-1], b.qo_indptr[1:])):
        ids = b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i + 1]]
        for h in range(8):
            ref[3][q0:q1, h] += off * np.abs(kv[ids, h // 4]).sum(-1).max() * 2.0 ** 16
    assert_state(o, lse, ref, F16_WEIGHTS)


@pytest.mark.parametrize("tokens", [1, 5], ids=["eight columns", "sixteen"])
def test_scores_of_infinite_bounds_against_either_sign(tokens):
    """An infinite bound: infinity where q takes it, NaN by 0 * infinity where q takes the other one, in the kernel as in the formula; the
    choice ranks both before every number."""
    torch = torch_mod()
    b = batch_of([tokens], [96], 4, 1, 16, False)
    bounds = torch.ones(b.num_pages, 1, 2, 128, dtype=torch.bfloat16, device="cuda")
    bounds[:, :, 0] = -1.0
    p = [int(x) for x in b.kv_indices]
    inf = float("inf")
    bounds[p[0], 0, 1, 3] = inf     # against q > 0
    bounds[p[1], 0, 1, 4] = inf     # against q < 0
    bounds[p[2], 0, 0, 3] = -inf    # against q > 0
    bounds[p[3], 0, 0, 4] = -inf    # against q < 0
    bounds[p[4], 0, 1, 5] = inf     # against 0
    q = torch.full((tokens, 4, 128), 0.5, dtype=torch.bfloat16, device="cuda")
    q[..., 4], q[..., 5] = -0.5, 0.0
    scores = torch.zeros(tokens, 1, 6, device="cuda")
    ws = workspace(b)
    ws.score_pages(q, bounds, scores)
    got = scores.cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, _ = P.page_scores(b, f64(q), f64(bounds), np.zeros(scores.shape))
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got == inf, want == inf)
    assert np.isnan(got[0, 0]).tolist() == [False, True, True, False, True, False] and got[0, 0, 0] == got[0, 0, 3] == inf
    assert np.allclose(got[:, 0, 5], 127 * 0.5 / np.sqrt(128))
    sel = torch.zeros(tokens, 1, 5, dtype=torch.int32, device="cuda")
    ws.select_pages(scores, sel)
    assert (sel.cpu().numpy()[:, 0] == p[:5]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("hq", [8, 24], ids=["4 heads a group", "12"])
def test_replays_on_pages_outside_the_pool(hq, dtype):
    """A replay whose plan lists pages outside the pool: reported; a tree takes their keys as zeros, scores leave them out, bounds and commits
    skip them, and what other requests get is right."""
    torch = torch_mod()
    hk, ps, lq, lkv = 2, 16, [5, 3, 7], [200, 90, 45]
    a = batch_of(lq, lkv, hq, hk, ps, False, seed=5)
    pages = a.num_pages  # the pools hold eight more, which the calls are not told of
    ids = a.kv_indices.copy()
    first, third = int(a.kv_indptr[0]), int(a.kv_indptr[2])
    ids[first + 4], ids[first + 9], ids[third + 2] = pages, pages + 7, pages + 3  # within a context, and where drafted tokens lie
    b = dataclasses.replace(a, kv_indices=ids)
    inside = ids < pages
    kind = torch.bfloat16 if dtype == "bf16" else torch.float8_e4m3fn
    k, v = (torch.randn(pages + 8, hk, ps, 128, device="cuda").to(kind) for _ in range(2))
    q, (o, lse), (po, plse) = bf16(a.q), outputs(a), outputs(a)
    mask = random_mask(np.random.default_rng(2), a, "tree")
    path = np.array([[1, 3, -1], [0, 2, -1], [2, 4, 6]], np.int32)
    dmask, dpath = dev(mask), dev(path)
    bounds = torch.full((pages + 8, hk, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    scores, sel = torch.zeros(15, hk, 13, device="cuda"), torch.zeros(15, hk, 4, dtype=torch.int32, device="cuda")
    ws = workspace(a, dtype=dtype)
    L, h, x = B.lib(), ws.handle, lambda t: t.data_ptr()

    def graph(call):
        return record(lambda: call(torch.cuda.current_stream().cuda_stream))

    def ok(st):
        assert st == 0

    tree = graph(lambda s: ok(L.fi_tree_run(h, x(q), x(k), x(v), pages, x(dmask), mask.shape[1], x(o), x(lse), s)))
    bound = graph(lambda s: ok(L.fi_page_bounds(h, x(k), pages, 0, x(bounds), s)))
    score = graph(lambda s: ok(L.fi_score_pages(h, x(q), x(bounds), pages, x(scores), 13, s)))
    pick = graph(lambda s: ok(L.fi_select_pages(h, x(scores), 13, 0, 0, 4, x(sel), s)))
    lists = graph(lambda s: ok(L.fi_run_pages(h, x(q), x(k), x(v), pages, x(sel), 4, x(po), x(plse), s)))
    commit = graph(lambda s: ok(L.fi_tree_commit(h, x(dpath), 3, x(k), x(v), pages, s)))
    plan(ws, b)

    def replay(g, bits):
        g.replay()
        torch.cuda.synchronize()
        assert ws.get_error() == bits

    kv, vv = f64(k), f64(v)
    kz, vz = kv.copy(), vv.copy()
    kz[pages:], vz[pages:] = 0, 0
    replay(tree, B.DEVERR_PAGE_OOB)
    assert_state(o, lse, P.tree_attention(b, f64(q), kz, vz, mask, q_floor=Q_FLOOR if dtype == "e4m3" else 0.0), F16_WEIGHTS if dtype == "e4m3" else BF16_WEIGHTS)
    replay(bound, B.DEVERR_PAGE_OOB)
    want = P.page_bounds(a, kv, np.full(bounds.shape, 7.0), False)
    assert np.array_equal(f64(bounds)[ids[inside]], want[ids[inside]]) and (f64(bounds)[pages:] == 7.0).all()
    replay(score, B.DEVERR_PAGE_OOB)
    want, reach = P.page_scores(b, f64(q), f64(bounds), np.zeros(scores.shape))
    for i in range(3):
        at = inside[b.kv_indptr[i]:b.kv_indptr[i + 1]]
        got = scores[b.qo_indptr[i]:b.qo_indptr[i + 1], :, :len(at)].cpu().numpy().astype(np.float64)
        assert np.isneginf(got[:, :, ~at]).all()
        assert np.abs(got - want[b.qo_indptr[i]:b.qo_indptr[i + 1], :, :len(at)])[:, :, at].max() <= reach * 2.0 ** -15
    replay(pick, 0)
    host = P.select_pages(b, scores.cpu().numpy(), 0, 0, 4)
    assert np.array_equal(sel.cpu().numpy(), host)
    outside = (host >= pages).any((1, 2))
    assert outside[8:].all() and not outside[:8].any()  # the last request has three pages in all
    replay(lists, B.DEVERR_PAGE_OOB)
    ref = P.pages_attention(b, f64(q), kv, vv, host)
    assert_state(po[:8], plse[:8], [r[:8] for r in ref], F16_WEIGHTS if dtype == "e4m3" else BF16_WEIGHTS)
    raw = lambda t: t.view(torch.int16 if dtype == "bf16" else torch.uint8).cpu().numpy()
    k0, v0 = raw(k), raw(v)
    replay(commit, B.DEVERR_PAGE_OOB)
    want_k, want_v = k0.copy(), v0.copy()
    for i in range(3):
        for j, e in enumerate(path[i]):
            if e < 0:
                break
            off = lkv[i] - lq[i]
            (fp,), (fs,) = P.places(b, i, [off + int(e)])
            (tp,), (ts,) = P.places(b, i, [off + j])
            if fp < pages and tp < pages:
                want_k[tp, :, ts], want_v[tp, :, ts] = k0[fp, :, fs], v0[fp, :, fs]
    assert np.array_equal(raw(k), want_k) and np.array_equal(raw(v), want_v)


def test_lists_at_their_limits():
    """A budget of 2^30 keys is the last that is taken: the next is refused before a pointer is looked at."""
    b = batch_of([1], [40], 4, 1, 16, False)
    ws = workspace(b)
    L, s = B.lib(), ctypes.c_void_p(torch_mod().cuda.current_stream().cuda_stream)
    for budget, status in ((2 ** 26, 1), (2 ** 26 + 1, 3), (2 ** 31 - 1, 3)):
        assert L.fi_run_pages(ws.handle, None, None, None, b.num_pages, None, budget, None, None, s) == status
    for row, status in ((0, 1), (2, 1), (3, 1)):  # three pages: the pointers are what is wrong with the last
        assert L.fi_score_pages(ws.handle, None, None, b.num_pages, None, row, s) == status
        assert L.fi_select_pages(ws.handle, None, row, 0, 0, 1, None, s) == status
    assert ws.get_error() == 0
