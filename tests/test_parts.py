"""Attention over parts of a cache, what needs no GPU: the oracle against brute force, masks of trees, null handles."""
import numpy as np
import pytest

from oracle import attention as A
from oracle import parts as P
from serving_attention_plan_gb300 import binding as B
from serving_attention_plan_gb300 import build as BLD
from serving_attention_plan_gb300 import workloads as W


@pytest.fixture(scope="module", autouse=True)
def built():
    BLD.build()
    B.lib()


def test_tree_mask():
    # request 0: 0 and 1 under the context, 2 under 0, 3 under 2; request 1: none; request 2: a chain of 40
    parents = np.concatenate([[-1, -1, 0, 2], np.arange(40) - 1])
    m = B.tree_mask([0, 4, 4, 44], parents).view(np.uint32)
    assert m.shape == (44, 2)
    assert [int(x) for x in m[:4, 0]] == [0b1, 0b10, 0b101, 0b1101] and not m[:4, 1].any()
    for t in range(40):
        assert int(m[4 + t, 0]) | int(m[4 + t, 1]) << 32 == (1 << (t + 1)) - 1
    assert B.tree_mask([0], []).shape == (0, 1)
    for bad in ([-1, 1], [-2, -1], [-1, 5]):
        with pytest.raises(ValueError):
            B.tree_mask([0, 2], bad)
    with pytest.raises(ValueError):
        B.tree_mask([0, 3], [-1, 0])


def test_tree_oracle():
    """A chain's mask gives causal attention; a row's keys by hand."""
    assert np.array_equal(P.tree_seen(B.tree_mask([0, 3], [-1, 0, 1]), 0, 3, 5), np.arange(5)[None, :] <= 2 + np.arange(3)[:, None])
    seen = P.tree_seen(np.array([[0b100], [0], [0b1011]], np.int32), 0, 3, 4)
    assert seen.tolist() == [[True, False, False, True], [True, False, False, False], [True, True, True, False]]
    # more tokens than keys: token u's key is l_kv - l_q + u
    assert P.tree_seen(np.array([[0b11], [0b10], [0b111]], np.int32), 0, 3, 2).tolist() == [[True, False], [True, False], [True, True]]


def test_state_oracle():
    """Two keys of logits 0 and log 3; a row that sees none."""
    q, k = np.zeros((2, 4)), np.zeros((2, 4))
    q[0, 0], k[1, 0] = 2.0, np.log(3.0)
    v = np.array([[0.0, 0, 0, 4.0], [4.0, 0, 0, 0]])
    o, lse, spread, reach = P.state(q, k, v, np.array([[True, True], [False, False]]))
    assert np.allclose(o[0], [3, 0, 0, 1]) and np.isclose(lse[0], np.log(4)) and np.isneginf(lse[1]) and not o[1].any()
    assert np.isclose(reach[0], np.log(3)) and np.allclose(spread[0], [3, 0, 0, 1])


def test_choice_oracle():
    """A page's score is no less than the logit of any of its keys; the choice by sorting."""
    b = W.random_small_batch(4, 3, 4, 2, 8, True, (1, 3), (20, 90))
    q, k = A.bf16_to_f64(b.q), A.bf16_to_f64(b.k_pages)
    bounds = P.page_bounds(b, k, np.zeros((k.shape[0], 2, 2, 128)), False)
    row = int(np.diff(b.kv_indptr).max())
    scores, _ = P.page_scores(b, q, bounds, np.zeros((b.total_q, 2, row)))
    lq, lkv = P.lengths(b)
    for i in range(3):
        for t in range(int(lq[i])):
            r = int(b.qo_indptr[i]) + t
            for j in range(P.last_key(b, i, t) + 1):
                (p,), (s,) = P.places(b, i, [j])
                for h in range(4):
                    assert scores[r, h // 2, j // 8] >= q[r, h] @ k[p, h // 2, s] / np.sqrt(128) - 1e-9
    chosen = P.select_pages(b, scores, 1, 1, 4)
    for i in range(3):
        ids = list(b.kv_indices[b.kv_indptr[i]:b.kv_indptr[i + 1]])
        for r in range(int(b.qo_indptr[i]), int(b.qo_indptr[i + 1])):
            for h in range(2):
                at = [ids.index(p) for p in chosen[r, h] if p >= 0]
                n = P.last_key(b, i, r - int(b.qo_indptr[i])) // 8 + 1
                assert at == sorted(at) and len(at) == min(n, 4)
                if n > 4:
                    assert 0 in at and n - 1 in at
                    rest = [x for x in range(1, n - 1) if x not in at]
                    assert max(scores[r, h, rest], default=-np.inf) <= min(scores[r, h, x] for x in at if 0 < x < n - 1)


def test_null_workspace():
    L = B.lib()
    assert L.fi_tree_run(None, None, None, None, 1, None, 1, None, None, None) == 1
    assert L.fi_tree_commit(None, None, 1, None, None, 1, None) == 1
    assert L.fi_page_bounds(None, None, 1, 0, None, None) == 1
    assert L.fi_score_pages(None, None, None, 1, None, 1, None) == 1
    assert L.fi_select_pages(None, None, 1, 0, 0, 1, None, None) == 1
    assert L.fi_run_pages(None, None, None, None, 1, None, 1, None, None, None) == 1


def test_tree_positions():
    # request 0: 0 and 1 under the context, 2 under 0, 3 under 2; request 1: none; request 2: a chain of 40
    parents = np.concatenate([[-1, -1, 0, 2], np.arange(40) - 1])
    p = B.tree_positions([0, 4, 4, 44], parents, [100, 7, 2 ** 30])
    assert p.dtype == np.int32 and p[:4].tolist() == [100, 100, 101, 102] and p[4:].tolist() == [2 ** 30 + t for t in range(40)]
    # the depth is the number of a row's mask bits but for its own
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 70, size=30)
    qo = np.concatenate([[0], np.cumsum(lens)])
    parents = np.concatenate([[rng.integers(-1, t) if t else -1 for t in range(n)] for n in lens])
    sees = np.unpackbits(B.tree_mask(qo, parents).view(np.uint8), axis=1).sum(1)
    assert np.array_equal(B.tree_positions(qo, parents, np.arange(30) * 11), np.repeat(np.arange(30) * 11, lens) + sees - 1)
    assert B.tree_positions([0], [], []).shape == (0,)
    for qo, parents, first in (([0, 2], [-1, 1], [5]), ([0, 2], [-2, -1], [5]), ([0, 2], [-1, 5], [5]), ([0, 3], [-1, 0], [5]), ([0, 2], [-1, 0], [5, 6])):
        with pytest.raises(ValueError):
            B.tree_positions(qo, parents, first)
