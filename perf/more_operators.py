"""Attention over parts of a paged KV-cache, in plain form and as the framework's calls.

One step of speculative decoding over long contexts: drafts attend to a few pages of the cache that a cheap score selects for
each query (bounds of the pages' keys, scores, selection, attention over the selected pages); the tree of drafted tokens is
verified with attention over the whole cache (tree), and the accepted path's keys move to their places (commit).  `own`
chooses between elementary torch operations and the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

D = 128
DEV = "cuda"


# ---- cases -----------------------------------------------------------------------------------------


def listed():
    return [
        # a few short requests with small trees, where the launches count: 8/2 heads
        _case("tree_small", "tree", 4, 300, 600, 8, 2, 16, qlo=11, qhi=16),
        # a verification step of long contexts: uneven trees of two row tiles a KV head, e4m3 pages
        _case("tree_long_e4m3", "tree", 12, 8000, 24_000, 64, 8, 16, qlo=17, qhi=30, dtype="e4m3"),
        # what the verification of an ordinary batch leaves to move
        _case("commit_b32", "commit", 32, 40, 200, 32, 8, 16, qlo=16, qhi=32, depth=6),
        # many requests with large trees, e4m3, token-major
        _case("commit_b512", "commit", 512, 10, 90, 64, 8, 32, qlo=40, qhi=64, depth=17, dtype="e4m3", layout="NHD"),
        # after a decode step: the page that took each request's new token
        _case("bounds_step", "bounds", 128, 500, 4096, 64, 8, 32, dtype="e4m3", layout="NHD", new_keys=True),
        # after the prompts: every page
        _case("bounds_prompts", "bounds", 13, 4000, 32_000, 32, 8, 16, qlo=4000, qhi=4000),
        # the pages' scores for a decode batch of the 8B shape
        _case("scores_b128", "scores", 128, 1000, 8192, 32, 8, 16),
        # two long contexts, four tokens each, 64/8 heads
        _case("scores_long", "scores", 2, 100_000, 131_072, 64, 8, 16, qlo=4, qhi=4, causal=True),
        # the choice of 64 pages among up to 512
        _case("select_b64", "select", 64, 2049, 8192, 32, 8, 16, budget=64, recent=4),
        # 512 of the 8192 pages of a long context, four tokens
        _case("select_long", "select", 1, 131_071, 131_071, 64, 8, 16, qlo=4, qhi=4, budget=512, recent=16, causal=True),
        # one draft step of a few requests over 32 pages each
        _case("pages_small", "pages", 3, 700, 3000, 32, 8, 16, budget=32, recent=2),
        # a large batch of long contexts, 2048 keys of each
        _case("pages_b128", "pages", 128, 2500, 6000, 32, 8, 16, budget=128, recent=4),
    ]


def _case(name, op, batch, lo, hi, hq, hkv, page, qlo=1, qhi=1, dtype="bf16", layout="HND", cap=0.0, depth=0, new_keys=False, causal=False, budget=0, recent=0, sink=1):
    """lo .. hi keys before the qlo .. qhi new tokens of a request; depth: longest accepted path."""
    return {"name": name, "op": op, "batch": batch, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "page": page, "qlo": qlo, "qhi": qhi, "dtype": dtype, "layout": layout,
            "cap": cap, "depth": depth, "new_keys": new_keys, "causal": causal, "budget": budget, "recent": recent, "sink": sink}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tree", "tree", "tree", "commit", "bounds", "scores", "scores", "select", "pages", "pages"])
    hkv = rng.choice([1, 2, 4, 8])
    g = rng.choice([1, 2, 4, 5, 8])
    more = {"dtype": rng.choice(["bf16", "bf16", "e4m3"]), "layout": rng.choice(["HND", "HND", "NHD"])}
    qhi = log(1, 64) if op in ("tree", "commit") else rng.choice([1, 3, log(1, 500)]) if op == "bounds" else rng.choice([1, 1, 2, 4])
    # page sizes that a plan takes: 8 to 128 tokens for requests of more than 8 query rows, else powers of two, and any for bf16 head-major pages
    page = rng.choice([8, 16, 16, 32, 64, 128])
    if qhi * g <= 8 and op != "tree" and rng.random() < 0.4:
        page = rng.choice([1, 4, 5, 24] if more == {"dtype": "bf16", "layout": "HND"} else [1, 2, 4])
    more.update(qlo=max(1, qhi // 2), qhi=qhi, cap=rng.choice([0.0, 0.0, 30.0]) if op in ("tree", "pages") else 0.0)
    if op == "commit":
        hi = log(1, 90)
        return _unnamed(_case("", op, log(1, 512), hi // 3, hi, hkv * g, hkv, page, depth=rng.randint(1, 17), **more))
    keys = log(500, 250_000)
    batch = min(log(1, 64 if op == "tree" else 128), max(1, keys // 100))
    hi = max(2, keys // batch)
    if op == "tree":
        return _unnamed(_case("", op, batch, hi // 3, hi, hkv * g, hkv, page, **more))
    if op == "bounds":
        return _unnamed(_case("", op, batch, hi // 3, hi, hkv * g, hkv, page, new_keys=rng.random() < 0.5, **more))
    more["causal"] = rng.random() < 0.7
    if op == "scores":
        return _unnamed(_case("", op, batch, hi // 3, hi, hkv * g, hkv, page, **more))
    budget = max(1, int(hi / page * rng.uniform(0.05, 0.8)))
    if op == "pages":
        budget = max(1, min(budget, 270_000 // (batch * qhi * page)))
    return _unnamed(_case("", op, batch, hi // 3, hi, hkv * g, hkv, page, budget=budget, recent=int(budget * rng.uniform(0, 0.5)), sink=rng.choice([0, min(1, budget - budget // 2)]), **more))


def _unnamed(case):
    del case["name"]
    return case


def _lengths(case):
    """(query tokens, keys) of each request: from the case alone."""
    r = np.random.RandomState((case["batch"] * 7919 + case["lo"] * 31 + case["hi"]) % (1 << 31))
    lq = r.randint(case["qlo"], case["qhi"] + 1, size=case["batch"]).astype(np.int64)
    ctx = r.randint(case["lo"], case["hi"] + 1, size=case["batch"]).astype(np.int64)
    return lq, lq + ctx


def _accepted(case):
    """Tokens on each request's accepted path: from the case alone."""
    lq, _ = _lengths(case)
    r = np.random.RandomState(case["batch"] + case["depth"])
    return np.minimum(r.randint(0, case["depth"] + 1, size=case["batch"]), lq)


def _ptr(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


# ---- inputs ----------------------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    c = case
    lq, lk = _lengths(c)
    page, hkv, hq = c["page"], c["hkv"], c["hq"]
    n_pages = (lk + page - 1) // page
    pool = int(n_pages.sum())
    order = torch.randperm(pool, generator=gen, device=DEV)
    s = {"case": c, "lq": lq, "lk": lk, "n_pool": pool, "n_q": int(lq.sum()), "order": order}
    s["qo"], s["kv"] = _ptr(lq), _ptr(n_pages)
    s["last"] = (lk - (n_pages - 1) * page).astype(np.int32)
    s["scales"] = (0.0625, 0.03125) if c["dtype"] == "e4m3" else (1.0, 1.0)
    # the requests' page lists side by side, page 0 behind the last; the query tokens side by side, token 0 behind the last
    e = np.arange(int(n_pages.max()))[None, :]
    s["has_page"] = _dev(e < n_pages[:, None])
    s["table"] = torch.where(s["has_page"], order[_dev(np.minimum(s["kv"][:-1, None] + e, pool - 1))], 0)
    t = np.arange(int(lq.max()))[None, :]
    s["padded"] = _dev(np.where(t < lq[:, None], s["qo"][:-1, None] + t, 0))  # [batch, tokens] -> query token
    req = np.repeat(np.arange(c["batch"]), lq)
    at = np.arange(s["n_q"]) - s["qo"][req]
    s["flat"] = _dev(req * t.shape[1] + at)  # query token -> [batch, tokens]
    s["req"], s["tokens"], s["keys"] = _dev(req), _dev(lq), _dev(lk)
    # the keys that each query token may see at most
    s["visible"] = _dev((lk - lq)[req] + at + 1 if c["causal"] else lk[req])
    {"tree": _prepare_tree, "commit": _prepare_commit, "bounds": _prepare_bounds, "scores": _prepare_scores, "select": _prepare_select, "pages": _prepare_pages}[c["op"]](s, gen)
    if own:
        from serving_attention_plan_gb300 import binding

        ws = binding.Workspace(c["batch"], s["n_q"], pool, hq, hkv)
        ws.set_variant(logits_soft_cap=c["cap"], kv_layout=c["layout"])
        ws.set_kv_dtype(c["dtype"], *s["scales"])
        ws.plan(s["qo"], s["kv"], order.cpu().numpy(), s["last"], page, c["causal"])
        s["ws"] = ws
    return s


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _pool(s, gen, scale):
    """A pool of K or V pages in the case's layout and type: standard normal values."""
    c = s["case"]
    shape = (s["n_pool"], c["hkv"], c["page"], D) if c["layout"] == "HND" else (s["n_pool"], c["page"], c["hkv"], D)
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return x.to(torch.bfloat16) if c["dtype"] == "bf16" else (x / scale).to(torch.float8_e4m3fn)


def _outputs(s, gen):
    s["q"] = (1.5 * torch.randn(s["n_q"], s["case"]["hq"], D, generator=gen, device=DEV)).to(torch.bfloat16)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["n_q"], s["case"]["hq"], device=DEV)


def _prepare_tree(s, gen):
    s["k_pages"], s["v_pages"] = _pool(s, gen, s["scales"][0]), _pool(s, gen, s["scales"][1])
    _outputs(s, gen)
    # random trees: each token's parent is one of those before it, or the context; a token sees its ancestors and itself
    r = np.random.RandomState(int(torch.randint(1 << 30, (1,), generator=gen, device=DEV)))
    t = int(s["lq"].max())
    sees = np.zeros((s["case"]["batch"], t + 1, (t + 31) // 32 * 32), bool)  # the last row: the context's
    for u in range(t):
        parent = r.randint(-1, u, size=s["case"]["batch"])
        sees[:, u] = sees[np.arange(s["case"]["batch"]), parent]
        sees[:, u, u] = True
    words = np.packbits(sees, axis=-1, bitorder="little").view(np.int32)
    rows = np.arange(t)[None, :] < s["lq"][:, None]
    s["mask"] = _dev(words[:, :t][rows])


def _prepare_commit(s, gen):
    s["k_pages"], s["v_pages"] = _pool(s, gen, s["scales"][0]), _pool(s, gen, s["scales"][1])
    r = np.random.RandomState(int(torch.randint(1 << 30, (1,), generator=gen, device=DEV)))
    path = np.full((s["case"]["batch"], max(1, s["case"]["depth"])), -1, np.int32)
    for i, n in enumerate(_accepted(s["case"])):
        path[i, :n] = np.sort(r.permutation(s["lq"][i])[:n])
    s["path"] = _dev(path)


def _prepare_bounds(s, gen):
    s["k_pages"] = _pool(s, gen, s["scales"][0])
    s["bounds"] = torch.zeros(s["n_pool"], s["case"]["hkv"], 2, D, dtype=torch.bfloat16, device=DEV)


def _prepare_scores(s, gen):
    _outputs(s, gen)
    # bounds as a page of 16 normal keys leaves them, around a value of the page's own
    mid = 0.5 * torch.randn(s["n_pool"], s["case"]["hkv"], 1, D, generator=gen, device=DEV)
    half = 1.7 + 0.4 * torch.randn(s["n_pool"], s["case"]["hkv"], 2, D, generator=gen, device=DEV)
    sign = torch.tensor([-1.0, 1.0], device=DEV)[:, None]
    s["bounds"] = ((mid + half.abs() * sign) / s["scales"][0]).to(torch.bfloat16)
    s["scores"] = torch.zeros(s["n_q"], s["case"]["hkv"], s["table"].shape[1], device=DEV)


def _prepare_select(s, gen):
    # scores with a few equal ones among them; what lies behind a request's pages is left from earlier steps
    x = 8 * torch.randn(s["n_q"], s["case"]["hkv"], s["table"].shape[1], generator=gen, device=DEV)
    s["scores"] = torch.where(torch.rand(x.shape, generator=gen, device=DEV) < 0.1, x.round(), x)
    s["selected"] = torch.empty(s["n_q"], s["case"]["hkv"], s["case"]["budget"], dtype=torch.int32, device=DEV)


def _prepare_pages(s, gen):
    _prepare_select(s, gen)
    s["k_pages"], s["v_pages"] = _pool(s, gen, s["scales"][0]), _pool(s, gen, s["scales"][1])
    _outputs(s, gen)
    s["selected"] = _plain_select(s)


# ---- one pass --------------------------------------------------------------------------------------


def run(state):
    return {"tree": _run_tree, "commit": _run_commit, "bounds": _run_bounds, "scores": _run_scores, "select": _run_select, "pages": _run_pages}[state["case"]["op"]](state)


def _by_key(s, pages):
    """[pages, hkv, slot, D], as raw codes where the pages hold e4m3."""
    x = pages.view(torch.uint8) if s["case"]["dtype"] == "e4m3" else pages
    return x if s["case"]["layout"] == "HND" else x.transpose(1, 2)


def _values(s, x, scale):
    return x.view(torch.float8_e4m3fn).float() * scale if s["case"]["dtype"] == "e4m3" else x.float()


def _padded_rows(s, pages, scale):
    """[batch, hkv, keys, D] in 32 bits: the keys of each request's page list in order."""
    return _values(s, _by_key(s, pages)[s["table"]], scale).transpose(1, 2).flatten(2, 3)


def _softmax(x, seen, v):
    """(softmax(x) v, log sum exp x) over the seen keys: zeros and -inf where there are none."""
    x = x.masked_fill_(~seen, -math.inf)
    m = x.amax(-1, keepdim=True)
    w = (x - torch.where(m == -math.inf, 0.0, m)).exp_()
    total = w.sum(-1, keepdim=True)
    return torch.matmul(w, v) / torch.where(total == 0, 1.0, total), (m + total.log()).squeeze(-1)


def _capped(s, x):
    x = x.mul_(1 / math.sqrt(D))
    return x.div_(s["case"]["cap"]).tanh_().mul_(s["case"]["cap"]) if s["case"]["cap"] else x


def _run_tree(s):
    c = s["case"]
    if own:
        s["ws"].tree_run(s["q"], s["k_pages"], s["v_pages"], s["mask"], s["o"], s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    b, t = s["padded"].shape
    g = c["hq"] // c["hkv"]
    q = s["q"].float()[s["padded"]].view(b, t, c["hkv"], g, D).transpose(1, 2).reshape(b, c["hkv"], t * g, D)
    x = _capped(s, torch.matmul(q, _padded_rows(s, s["k_pages"], s["scales"][0]).transpose(2, 3)))
    # what each token sees: the context, and the drafted tokens of its mask
    bits = (s["mask"][s["padded"]][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1
    bits = bits.flatten(2).bool()
    u = torch.arange(x.shape[-1], device=DEV) - (s["keys"] - s["tokens"])[:, None]
    drafted = torch.gather(bits, 2, u.clamp(0, bits.shape[2] - 1)[:, None, :].expand(b, t, -1))
    seen = (u < 0)[:, None, :] | (drafted & (u < s["tokens"][:, None])[:, None, :])
    o, lse = _softmax(x.view(b, c["hkv"], t, g, -1), seen[:, None, :, None, :], _padded_rows(s, s["v_pages"], s["scales"][1])[:, :, None])
    s["o"] = o.transpose(1, 2).reshape(b * t, c["hq"], D)[s["flat"]].to(torch.bfloat16)
    s["lse"] = lse.transpose(1, 2).reshape(b * t, c["hq"])[s["flat"]]
    return {"o": s["o"], "lse": s["lse"]}


def _run_commit(s):
    if own:
        s["ws"].tree_commit(s["path"], s["k_pages"], s["v_pages"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    page = s["case"]["page"]
    first = (s["keys"] - s["tokens"])[:, None]
    j = torch.arange(s["path"].shape[1], device=DEV)[None, :]
    on = s["path"] >= 0
    src = torch.where(on, first + s["path"], 0)
    # an entry that is not there writes the request's first key to itself
    dst = torch.where(on, first + j, 0)
    fp, tp = torch.gather(s["table"], 1, src // page), torch.gather(s["table"], 1, dst // page)
    for pages in (_by_key(s, s["k_pages"]), _by_key(s, s["v_pages"])):
        pages[tp, :, dst % page] = pages[fp, :, src % page]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _run_bounds(s):
    c = s["case"]
    if own:
        s["ws"].page_bounds(s["k_pages"], s["bounds"], new_keys=c["new_keys"])
        return s["bounds"]
    if c["new_keys"]:  # the pages that hold the last tokens of a request: at most so many
        n = (c["qhi"] - 1 + c["page"] - 1) // c["page"] + 1
        e = torch.clamp((s["keys"] - s["tokens"]) // c["page"], max=s["table"].shape[1])[:, None] + torch.arange(n, device=DEV)
        e = torch.minimum(e, ((s["keys"] - 1) // c["page"])[:, None])  # the last one again, behind it
    else:
        e = torch.minimum(torch.arange(s["table"].shape[1], device=DEV)[None, :], ((s["keys"] - 1) // c["page"])[:, None])
    p = torch.gather(s["table"], 1, e)
    k = _values(s, _by_key(s, s["k_pages"])[p], 1.0)  # [batch, pages, hkv, slot, D]
    there = (e[:, :, None] * c["page"] + torch.arange(c["page"], device=DEV) < s["keys"][:, None, None])[:, :, None, :, None]
    s["bounds"][p, :, 0] = torch.where(there, k, math.inf).amin(3).to(torch.bfloat16)
    s["bounds"][p, :, 1] = torch.where(there, k, -math.inf).amax(3).to(torch.bfloat16)
    return s["bounds"]


def _run_scores(s):
    c = s["case"]
    if own:
        s["ws"].score_pages(s["q"], s["bounds"], s["scores"])
        return s["scores"]
    b, t = s["padded"].shape
    g, n = c["hq"] // c["hkv"], s["table"].shape[1]
    q = s["q"].float()[s["padded"]].view(b, t, c["hkv"], g, D).transpose(1, 2).reshape(b, c["hkv"], t * g, D)
    q = torch.cat([q.clamp(max=0), q.clamp(min=0)], -1)
    x = torch.matmul(q, s["bounds"][s["table"]].float().flatten(3).permute(0, 2, 3, 1))  # [batch, hkv, tokens * g, pages]
    x = x.view(b, c["hkv"], t, g, n).amax(3).mul_(s["scales"][0] / math.sqrt(D)).transpose(1, 2).reshape(b * t, c["hkv"], n)[s["flat"]]
    seen = torch.arange(n, device=DEV) * c["page"] < s["visible"][:, None]
    x = x.masked_fill_(~seen[:, None, :], -math.inf)
    s["scores"] = torch.where(s["has_page"][s["req"]][:, None, :], x, s["scores"])
    return s["scores"]


def _run_select(s):
    c = s["case"]
    if own:
        s["ws"].select_pages(s["scores"], s["selected"], recent=c["recent"], sink=c["sink"])
    else:
        s["selected"] = _plain_select(s)
    return s["selected"]


def _plain_select(s):
    c = s["case"]
    n, budget = s["table"].shape[1], c["budget"]
    e = torch.arange(n, device=DEV)[None, :]
    count = ((s["visible"] + c["page"] - 1) // c["page"])[:, None]  # pages that the token sees
    always = ((e < c["sink"]) | (e >= count - c["recent"]))[:, None, :]
    there = (e < count)[:, None, :]
    rank = torch.sort(s["scores"], dim=-1, descending=True, stable=True).indices
    kind = torch.where(there, torch.where(always, 0, 1), 2).expand_as(rank)
    rank = torch.gather(rank, 2, torch.sort(torch.gather(kind, 2, rank), dim=-1, stable=True).indices)[..., :budget]
    rank = torch.nn.functional.pad(rank, (0, budget - rank.shape[-1]), value=n)
    gone = (torch.arange(budget, device=DEV)[None, :] >= count.clamp(max=budget))[:, None, :]
    rank = torch.where(gone, n, rank).sort(-1).values
    ids = torch.gather(s["table"][s["req"]][:, None, :].expand(-1, rank.shape[1], -1), 2, rank.clamp(max=n - 1))
    return torch.where(gone, -1, ids).to(torch.int32)


def _run_pages(s):
    c = s["case"]
    if own:
        s["ws"].run_pages(s["q"], s["k_pages"], s["v_pages"], s["selected"], s["o"], s["lse"])
        return {"o": s["o"], "lse": s["lse"]}
    g, ids = c["hq"] // c["hkv"], s["selected"].long()
    h = torch.arange(c["hkv"], device=DEV)[None, :, None]
    k = _values(s, _by_key(s, s["k_pages"])[ids.clamp(min=0), h], s["scales"][0]).flatten(2, 3)  # [tokens, hkv, keys, D]
    v = _values(s, _by_key(s, s["v_pages"])[ids.clamp(min=0), h], s["scales"][1]).flatten(2, 3)
    x = _capped(s, torch.matmul(s["q"].float().view(-1, c["hkv"], g, D), k.transpose(2, 3)))
    # the page of the last key that a token sees ends there
    end = torch.gather(s["table"][s["req"]], 1, (s["visible"] - 1)[:, None] // c["page"])[:, :, None]
    slots = torch.where(ids == end, ((s["visible"] - 1) % c["page"] + 1)[:, None, None], c["page"])
    seen = (ids >= 0)[..., None] & (torch.arange(c["page"], device=DEV) < slots[..., None])
    o, lse = _softmax(x, seen.flatten(2)[:, :, None, :], v)
    s["o"], s["lse"] = o.reshape(-1, c["hq"], D).to(torch.bfloat16), lse.reshape(-1, c["hq"])
    return {"o": s["o"], "lse": s["lse"]}


# ---- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    lq, lk = (x.astype(np.float64) for x in _lengths(case))
    c, e = case, 1 if case["dtype"] == "e4m3" else 2
    hq, hkv = c["hq"], c["hkv"]
    rows = lq.sum() * hq
    pages = np.ceil(lk / c["page"])
    if c["op"] == "tree":
        seen = lq * (lk - lq) + lq * np.log2(lq + 1)  # a token of a random tree has about log(tokens) ancestors
        return {"bytes": lk.sum() * hkv * 2 * D * e + rows * (4 * D + 4) + (lq * np.ceil(lq / 32) * 4).sum(), "flops": seen.sum() * hq * 4 * D}
    if c["op"] == "commit":
        n = float(_accepted(c).sum())
        return {"bytes": n * (4 + 2 * 2 * hkv * D * e), "flops": n}
    if c["op"] == "bounds":
        first = np.floor((lk - lq) / c["page"]) if c["new_keys"] else 0 * lk
        return {"bytes": hkv * ((lk - first * c["page"]).sum() * D * e + (pages - first).sum() * 4 * D), "flops": hkv * (lk - first * c["page"]).sum() * 2 * D}
    if c["op"] == "scores":
        return {"bytes": hkv * (pages.sum() * 4 * D + (lq * pages).sum() * 4) + rows * 2 * D, "flops": (lq * pages).sum() * hq * 4 * D}
    chosen = (lq * np.minimum(pages, c["budget"])).sum() * hkv
    if c["op"] == "select":
        return {"bytes": (lq * pages).sum() * hkv * 4 + chosen * 4, "flops": (lq * pages).sum() * hkv}
    keys = chosen * c["page"]
    return {"bytes": chosen * 4 + keys * 2 * D * e + rows * (4 * D + 4), "flops": keys * (hq / hkv) * 4 * D}


# ---- the definitions in 64 bits ------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    lists = [torch.from_numpy(x).to(DEV) for x in np.split(s["order"].cpu().numpy(), s["kv"][1:-1])]
    return {"tree": _exact_tree, "commit": _exact_commit, "bounds": _exact_bounds, "scores": _exact_scores, "select": _exact_select, "pages": _exact_pages}[case["op"]](s, lists)


def _head_rows(s, pages, pl, h):
    """Rows of KV head h of the pages in a list, [len * page, D], as they are stored."""
    x = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = x[pl, h] if s["case"]["layout"] == "HND" else x[pl][:, :, h]
    return x.reshape(-1, D).view(pages.dtype)


def _attend(s, q, k, v, see):
    """Rows q [m, D] over keys k, v [n, D]; see: [m, n] or None."""
    x = q.double() @ k.t() / D**0.5
    if s["case"]["cap"]:
        x = s["case"]["cap"] * torch.tanh(x / s["case"]["cap"])
    if see is not None:
        x = torch.where(see, x, -math.inf)
    lse = torch.logsumexp(x, -1)
    return torch.exp(x - lse[:, None]).nan_to_num(0.0) @ v, lse


def _exact_tree(s, lists):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    if (s["lq"] * s["lk"]).sum() * c["hq"] > 4e9:
        return None
    o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    mask = s["mask"].cpu().numpy().view(np.uint32)
    for i, pl in enumerate(lists):
        n, t, q0 = int(s["lk"][i]), int(s["lq"][i]), int(s["qo"][i])
        see = np.ones((t, n), bool)
        u = np.arange(t)
        see[:, n - t :] = (mask[q0 : q0 + t][:, u >> 5] >> (u & 31).astype(np.uint32)) & 1
        see = _dev(see).repeat_interleave(g, 0)
        for h in range(c["hkv"]):
            k = _head_rows(s, s["k_pages"], pl, h)[:n].double() * s["scales"][0]
            v = _head_rows(s, s["v_pages"], pl, h)[:n].double() * s["scales"][1]
            a, b = _attend(s, s["q"][q0 : q0 + t, h * g : (h + 1) * g].reshape(-1, D), k, v, see)
            o[q0 : q0 + t, h * g : (h + 1) * g], lse[q0 : q0 + t, h * g : (h + 1) * g] = a.view(t, g, D), b.view(t, g)
    return {"o": o, "lse": lse}


def _exact_commit(s, lists):
    c = s["case"]
    out = {"k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double()}
    path = s["path"].cpu().numpy()
    for name in ("k_pages", "v_pages"):
        old = out[name].clone()
        for i, pl in enumerate(lists):
            src = path[i][path[i] >= 0].astype(np.int64) + s["lk"][i] - s["lq"][i]
            dst = np.arange(len(src)) + s["lk"][i] - s["lq"][i]
            fp, tp, fs, ts = pl[_dev(src // c["page"])], pl[_dev(dst // c["page"])], _dev(src % c["page"]), _dev(dst % c["page"])
            if c["layout"] == "HND":
                out[name][tp, :, ts] = old[fp, :, fs]
            else:
                out[name][tp, ts] = old[fp, fs]
    return out


def _exact_bounds(s, lists):
    c = s["case"]
    out = s["bounds"].double()
    for i, pl in enumerate(lists):
        n, page = int(s["lk"][i]), c["page"]
        first = (n - int(s["lq"][i])) // page if c["new_keys"] else 0
        for h in range(c["hkv"]):
            k = _head_rows(s, s["k_pages"], pl, h)[:n].double()
            whole = n // page
            if whole > first:
                x = k[first * page : whole * page].view(-1, page, D)
                out[pl[first:whole], h, 0], out[pl[first:whole], h, 1] = x.min(1).values, x.max(1).values
            if n % page:
                out[pl[whole], h, 0], out[pl[whole], h, 1] = k[whole * page :].min(0).values, k[whole * page :].max(0).values
    return out


def _exact_scores(s, lists):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = s["scores"].double()
    q = s["q"].double()
    for i, pl in enumerate(lists):
        for t in range(int(s["qo"][i]), int(s["qo"][i + 1])):
            see = torch.arange(len(pl), device=DEV) * c["page"] < s["visible"][t]
            b = s["bounds"][pl].double()  # [pages, hkv, 2, D]
            x = q[t].view(c["hkv"], g, D)[None]
            x = torch.where(x > 0, x * b[:, :, 1:2], x * b[:, :, 0:1]).sum(-1).amax(-1) * (s["scales"][0] / D**0.5)
            out[t, :, : len(pl)] = torch.where(see[:, None], x, -math.inf).t()
    return out


def _exact_select(s, lists):
    c = s["case"]
    out = np.full(tuple(s["selected"].shape), -1, np.int32)
    score, visible, req = s["scores"].cpu().numpy().astype(np.float64), s["visible"].cpu().numpy(), s["req"].cpu().numpy()
    for t in range(s["n_q"]):
        pl = lists[req[t]].cpu().numpy()
        n = int(-(-visible[t] // c["page"]))
        m = min(n, c["budget"])
        lo, hi = (min(c["sink"], n), max(n - c["recent"], c["sink"])) if n > m else (0, n)
        for h in range(c["hkv"]):
            best = lo + np.argsort(-score[t, h, lo:hi], kind="stable")[: m - (n - (hi - lo))]
            out[t, h, :m] = pl[np.sort(np.concatenate([np.arange(lo), best, np.arange(hi, n)]))]
    return out


def _exact_pages(s, lists):
    c = s["case"]
    g, page = c["hq"] // c["hkv"], c["page"]
    o, lse = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV), torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    ids, visible, req = s["selected"].cpu().numpy(), s["visible"].cpu().numpy(), s["req"].cpu().numpy()
    tails = [x.cpu().numpy() for x in lists]
    for t in range(s["n_q"]):
        last = int(visible[t]) - 1
        for h in range(c["hkv"]):
            pl = ids[t, h][ids[t, h] >= 0]
            n = len(pl) * page
            if len(pl) and pl[-1] == tails[req[t]][last // page]:
                n -= page - 1 - last % page
            on = torch.from_numpy(pl.astype(np.int64)).to(DEV)
            k = _head_rows(s, s["k_pages"], on, h)[:n].double() * s["scales"][0]
            v = _head_rows(s, s["v_pages"], on, h)[:n].double() * s["scales"][1]
            o[t, h * g : (h + 1) * g], lse[t, h * g : (h + 1) * g] = _attend(s, s["q"][t, h * g : (h + 1) * g], k, v, None)
    return {"o": o, "lse": lse}
