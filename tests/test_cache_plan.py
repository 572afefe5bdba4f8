"""Host side of the cache operators (no GPU): request geometry, page conditions, refusals of the binding."""
import ctypes

import numpy as np
import pytest

from oracle import cache as C
from serving_attention_plan_gb300 import binding as B
from serving_attention_plan_gb300 import build as BLD
from serving_attention_plan_gb300 import workloads as W


@pytest.fixture(scope="module", autouse=True)
def built():
    BLD.build()
    B.lib()


@pytest.mark.parametrize("seed,batch,ps,ql,kl", [(0, 1, 16, (1, 1), (1, 1)), (1, 7, 16, (0, 40), (0, 700)),
                                                 (2, 130, 1, (1, 1), (0, 90)), (3, 3, 5, (2, 9), (0, 31))])
def test_geometry(seed, batch, ps, ql, kl):
    b = W.random_small_batch(seed, batch, 4, 2, ps, False, ql, kl)
    geo, pages_twice, tails_twice = B.cache_plan_compute(b.qo_indptr, b.kv_indptr, b.kv_indices, b.last_page_len, ps)
    l_q, l_kv = C.lengths(b)
    assert np.array_equal(geo[:, 0], b.qo_indptr) and np.array_equal(geo[:, 2], b.kv_indptr)
    assert np.array_equal(geo[:-1, 1], l_q) and np.array_equal(geo[:-1, 3], l_kv)
    assert np.array_equal(geo[:, 4], np.concatenate([[0], np.cumsum(-(-l_kv // 32))]))
    assert np.array_equal(geo[:, 5], np.concatenate([[0], np.cumsum(-(-l_kv // 256))]))
    assert not pages_twice and not tails_twice


@pytest.mark.parametrize("lists,q,last,pages,tails", [
    ([[0, 1], [0, 2]], [1, 1], [3, 4], True, False),      # a shared full prefix page, own tails
    ([[0, 1], [2, 1]], [1, 1], [3, 4], True, True),       # a shared tail
    ([[0, 1], [2, 1]], [1, 0], [3, 4], True, False),      # a shared tail that only one request writes
    ([[0, 0]], [1], [2], True, False),                    # the same page twice, one token
    ([[0, 0]], [5], [2], True, True),                     # the same page twice, both written
    ([[], [3]], [2, 1], [0, 1], False, False),            # a request without pages
])
def test_page_conditions(lists, q, last, pages, tails):
    kv = np.concatenate([[0], np.cumsum([len(x) for x in lists])])
    got = B.cache_plan_compute(np.concatenate([[0], np.cumsum(q)]), kv, [p for x in lists for p in x], last, 4)
    assert got[1:] == (pages, tails)


@pytest.mark.parametrize("q,last", [([], []), ([0], [0]), ([1], [0]), ([3, 0, 2], [0, 0, 0])])
def test_batches_without_pages(q, last):
    """No request, or requests that have no page: a geometry of no keys, and no page listed twice."""
    geo, pages_twice, tails_twice = B.cache_plan_compute(np.concatenate([[0], np.cumsum(q)]), [0] * (len(q) + 1), [], last, 16)
    assert np.array_equal(geo[:, 0], np.concatenate([[0], np.cumsum(q)])) and np.array_equal(geo[:-1, 1], q)
    assert not geo[:, 2:].any() and not pages_twice and not tails_twice


def test_bad_batches_are_refused():
    for args in (([0, 1], [0, 1], [-1], [1]), ([0, 1], [0, 1], [0], [5]), ([0, 1], [0, 1], [0], [0]),
                 ([1, 1], [0, 1], [0], [1]), ([0, 1], [1, 0], [0], [1])):
        with pytest.raises(B.FiError) as e:
            B.cache_plan_compute(*args, 4)
        assert e.value.status == 1
    with pytest.raises(B.FiError) as e:  # a key position above 2^30
        B.cache_plan_compute([0, 1], [0, 3], [0, 1, 2], [1], 1 << 30)
    assert e.value.status == 3


def test_null_workspace_and_pointers():
    L = B.lib()
    z = ctypes.c_void_p(0)
    assert L.fi_workspace_set_rope(z, None, 0, 0) == 1
    assert L.fi_append(z, z, 0, z, 0, z, 0, z, z, 0.0, z, z, z, z, 0, z) == 1
    assert L.fi_key_weights(z, z, z, 0, z, 1.0, 0, z, z) == 1
    assert L.fi_select_keys(z, z, 0, 0, 0, 1, z, z) == 1
    assert L.fi_compact(z, z, 1, z, z, z, 0, z) == 1
    assert L.fi_cache_plan_compute(None, None, None, None, 0, 1, None, None) == 1


class OnGpu:
    """Stands for a dense CUDA tensor of a GPU (there is none here): what the binding asks of a tensor, and no memory."""

    def __init__(self, shape, dtype, gpu):
        self.shape, self.dtype, self.gpu, self.is_cuda = shape, dtype, gpu, True

    def get_device(self):
        return self.gpu

    def stride(self):
        return tuple(int(np.prod(self.shape[i + 1:])) for i in range(len(self.shape)))

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0


@pytest.mark.parametrize("which", range(13))
def test_tensors_of_another_gpu_are_refused(which):
    """Each tensor of each cache operator on GPU 1, the others and the workspace on GPU 0."""
    torch = pytest.importorskip("torch")
    ws = B.Workspace.__new__(B.Workspace)
    ws._h, ws._device = ctypes.c_void_p(0), 0
    ws.num_qo_heads, ws.num_kv_heads, ws.head_dim = 4, 2, 128
    ws._plan, ws._shapes_of = (3, 3, 16, "HND", "bf16"), None
    made = 0

    def t(shape, dtype=torch.bfloat16):
        nonlocal made
        made += 1
        return OnGpu(shape, dtype, int(made - 1 == which))

    q, k, v, out = t((3, 4, 128)), t((3, 2, 128)), t((3, 2, 128)), t((3, 4, 128))
    kp, vp = t((9, 2, 16, 128)), t((9, 2, 16, 128))
    wq, wk, pos = t((128,)), t((128,)), t((3,), torch.int32)
    lse, w, kept, none = t((3, 4), torch.float32), t((9, 2, 16), torch.float32), t((3, 2, 8), torch.int32), t((1,))
    assert made == 13
    uses = {ws.append: (q, k, v, kp, vp, out, wq, wk, 1e-6, pos), ws.key_weights: (q, kp, lse, w), ws.select_keys: (w, 8, kept),
            ws.compact: (kept, kp, vp, w)}
    for call, args in uses.items():
        away = any(getattr(a, "gpu", 0) for a in args)
        with pytest.raises(ValueError if away else B.FiError) as e:
            call(*args, stream=0)
        assert "on GPU 1, the workspace is on GPU 0" in str(e.value) if away else e.value.status == 1  # no workspace behind it
