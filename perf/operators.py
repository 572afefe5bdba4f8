"""The cache operators of the serving path, in plain form and as the framework's calls.

One life cycle of a paged KV-cache: new tokens are normed, rotated and written into pages (append), the attention weight
of every cached key is accumulated (weights), the keys worth keeping are chosen (select), and they are moved to the front
of each request's pages (compact).  `own` chooses between elementary torch operations and the framework's kernels.
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
        # one decode step early in generation: 128 requests, one token each, 32/8 heads
        _append("append_decode_b128", 128, 1, 1, 64, 32, 8, 16),
        # ragged prompts of 128..4096 tokens, continued far into a long context
        _append("append_prefill_ragged", 16, 128, 4096, 0, 32, 8, 16, first=100_000),
        # chunks of an uneven length into e4m3 token-major pages: no norm, half of the dims rotated in adjacent pairs
        _append("append_chunk_e4m3", 7, 997, 997, 0, 64, 8, 64, dtype="e4m3", layout="NHD", rotary=64, interleaved=True, norm=False),
        # a tiny decode batch, where the launch counts: 8/2 heads
        _weights("weights_decode_tiny", 4, 1, 37, 512, 8, 2, 16),
        # an ordinary decode batch of the 8B shape
        _weights("weights_decode_b128", 128, 1, 1, 4096, 32, 8, 16),
        # two long contexts in e4m3 pages of one token, 64/8 heads
        _weights("weights_decode_long", 2, 1, 100_000, 131_072, 64, 8, 1, dtype="e4m3"),
        # causal prompts: every key's weight over all the tokens after it
        _weights("weights_prefill", 4, 0, 1024, 4096, 32, 8, 16, causal=True),
        # a chunk of new tokens over a cache, soft-capped logits, e4m3 pages
        _weights("weights_chunk", 2, 509, 8192, 16_384, 64, 8, 16, causal=True, dtype="e4m3", cap=30.0),
        # a batch over its budget: half of each cache stays
        _select("select_b64", 64, 2049, 4096, 8, 16, 2048, 128),
        # one long context cut to an eighth
        _select("select_long", 1, 131_071, 131_071, 8, 16, 16_384, 1024),
        # the batch's pages after the choice
        _compact("compact_b64", 64, 2049, 4096, 8, 16, 2048, 128),
        # the long context's pages, e4m3, token-major
        _compact("compact_long", 1, 131_071, 131_071, 8, 16, 32_768, 1024, dtype="e4m3", layout="NHD"),
    ]


def _append(name, batch, lo, hi, ctx, hq, hkv, page, dtype="bf16", layout="HND", rotary=128, interleaved=False, norm=True, first=0):
    return {"name": name, "op": "append", "batch": batch, "lo": lo, "hi": hi, "ctx": ctx, "hq": hq, "hkv": hkv, "page": page, "dtype": dtype,
            "layout": layout, "rotary": rotary, "interleaved": interleaved, "norm": norm, "first": first}


def _weights(name, batch, q_len, lo, hi, hq, hkv, page, causal=False, dtype="bf16", layout="HND", cap=0.0, decay=0.95):
    return {"name": name, "op": "weights", "batch": batch, "q_len": q_len, "lo": lo, "hi": hi, "hq": hq, "hkv": hkv, "page": page, "causal": causal,
            "dtype": dtype, "layout": layout, "cap": cap, "decay": decay}


def _select(name, batch, lo, hi, hkv, page, budget, recent, sink=4):
    return {"name": name, "op": "select", "batch": batch, "lo": lo, "hi": hi, "hkv": hkv, "page": page, "budget": budget, "recent": recent, "sink": sink}


def _compact(name, batch, lo, hi, hkv, page, budget, recent, dtype="bf16", layout="HND"):
    return {"name": name, "op": "compact", "batch": batch, "lo": lo, "hi": hi, "hkv": hkv, "page": page, "budget": budget, "recent": recent, "sink": 4,
            "dtype": dtype, "layout": layout}


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    page = rng.choice([1, 2, 4, 5, 8, 16, 16, 32, 64])
    dtype = rng.choice(["bf16", "bf16", "e4m3"])
    if dtype == "e4m3" and page == 5:
        page = 4
    layout = rng.choice(["HND", "HND", "NHD"]) if page != 5 else "HND"
    op = rng.choice(["append", "append", "weights", "weights", "weights", "select", "compact"])
    if op == "append":
        hkv = rng.choice([1, 2, 8])
        g = rng.choice([1, 2, 4, 5, 8])
        if rng.random() < 0.5:
            case = _append("", log(1, 128), 1, 1, log(1, 64), hkv * g, hkv, page)
        else:
            tokens = log(200, 30_000)
            batch = min(log(1, 16), max(1, tokens // 2))
            page = page if page >= 8 else 16  # more than 8 rows a request: pages of 8 to 128 tokens
            case = _append("", batch, max(1, tokens // batch // 3), max(1, tokens // batch), log(1, 64), hkv * min(g, 4), hkv, page)
        case.update(dtype=dtype, layout=layout, rotary=rng.choice([0, 32, 64, 128, 128]), interleaved=rng.random() < 0.4, norm=rng.random() < 0.7, first=rng.choice([0, log(1, 1_000_000)]))
    elif op == "weights":
        hkv = rng.choice([1, 2, 4, 8])
        g = rng.choice([1, 2, 4, 5, 8])
        kind = rng.random()
        if kind < 0.4:
            keys = log(32, 250_000)
            batch = min(log(1, 128), max(1, keys // 8))
            case = _weights("", batch, 1, max(1, keys // batch // 4), max(1, keys // batch), hkv * g, hkv, page)
            case["layout"] = layout if page & (page - 1) == 0 else "HND"
        elif kind < 0.7:
            hi = log(64, 4096)
            case = _weights("", rng.randint(1, 4), 0, max(1, hi // 4), hi, hkv * min(g, 4), hkv, page if page >= 8 else 16, causal=True)
        else:
            hi = log(600, 16_384)
            case = _weights("", rng.randint(1, 2), log(2, 500), max(500, hi // 2), hi, hkv * g, hkv, 16, causal=True, cap=rng.choice([0.0, 20.0, 50.0]))
        case.update(dtype=dtype if case["page"] != 5 else "bf16", decay=rng.choice([1.0, 0.9, 0.5, 0.0]))
    else:
        keys = log(512, 200_000)
        batch = min(log(1, 64), max(1, keys // 64))
        hi = max(8, keys // batch)
        budget = max(4, int(hi * rng.uniform(0.1, 0.9)))
        recent = int(budget * rng.uniform(0, 0.6))
        hkv = rng.choice([1, 2, 4, 8])
        if op == "select":
            case = _select("", batch, max(1, hi // 3), hi, hkv, page, budget, recent)
        else:
            case = _compact("", batch, max(1, hi // 3), hi, hkv, page, budget, recent, dtype, layout)
        case["sink"] = rng.choice([0, 1, 4]) if budget - recent >= 4 else 0
    del case["name"]
    return case


def _lengths(case):
    """(query tokens, keys) of each request: from the case alone."""
    r = np.random.RandomState((case["batch"] * 7919 + case["lo"] * 31 + case["hi"]) % (1 << 31))
    n = r.randint(case["lo"], case["hi"] + 1, size=case["batch"]).astype(np.int64)
    if case["op"] == "append":  # n new tokens behind 0 to ctx - 1 earlier ones
        return n, n + (r.randint(0, case["ctx"], size=case["batch"]) if case["ctx"] else 0)
    if case["op"] == "weights":
        return (np.minimum(n, case["q_len"]) if case["q_len"] else n), n
    return np.ones_like(n), n


def _ptr(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


# ---- inputs ----------------------------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    lq, lk = _lengths(case)
    page, hkv = case["page"], case["hkv"]
    hq = case.get("hq", hkv)
    pages = (lk + page - 1) // page
    pool = int(pages.sum())
    order = torch.randperm(pool, generator=gen, device=DEV)
    s = {"case": case, "lq": lq, "lk": lk, "n_pool": pool}
    s["qo"], s["kv"] = _ptr(lq), _ptr(pages)
    s["last"] = np.where(pages > 0, lk - (pages - 1) * page, 0).astype(np.int32)
    s["order"] = order
    # where key j of request i lies: page * page_size + slot; invalid places (j >= length) point at slot 0
    j = torch.arange(int(lk.max()), device=DEV)
    klen = torch.from_numpy(lk).to(DEV)
    s["valid"] = j[None, :] < klen[:, None]
    entry = torch.from_numpy(s["kv"][:-1].astype(np.int64)).to(DEV)[:, None] + j[None, :] // page
    s["slot"] = torch.where(s["valid"], order[torch.where(s["valid"], entry, 0)] * page + j[None, :] % page, 0)
    {"append": _prepare_append, "weights": _prepare_weights, "select": _prepare_select, "compact": _prepare_compact}[case["op"]](s, gen, hq)
    if own:
        from serving_attention_plan_gb300 import binding

        ws = binding.Workspace(case["batch"], int(lq.sum()), pool, hq, hkv)
        ws.set_variant(logits_soft_cap=case.get("cap", 0.0), kv_layout=case.get("layout", "HND"))
        ws.set_kv_dtype(case.get("dtype", "bf16"), *s.get("scales", (1.0, 1.0)))
        if case["op"] == "append":
            ws.set_rope(s["inv_freq"].cpu().numpy(), case["interleaved"])
        ws.plan(s["qo"], s["kv"], order.cpu().numpy(), s["last"], page, case.get("causal", False))
        s["ws"] = ws
        if case["op"] == "compact":
            s["kept"] = s["kept"].contiguous()  # the calls take dense tensors
    return s


def _randn(gen, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _pages(s, gen, scale):
    """A pool of K or V pages in the case's layout and type: standard normal values."""
    c = s["case"]
    shape = (s["n_pool"], c["hkv"], c["page"], D) if c["layout"] == "HND" else (s["n_pool"], c["page"], c["hkv"], D)
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    return x.to(torch.bfloat16) if c["dtype"] == "bf16" else (x / scale).to(torch.float8_e4m3fn)


def _prepare_append(s, gen, hq):
    c = s["case"]
    hkv, n = c["hkv"], int(s["lq"].sum())
    s["scales"] = (0.0625, 0.03125) if c["dtype"] == "e4m3" else (1.0, 1.0)
    # q, k and v of a token lie in one row, as a fused projection writes them
    s["qkv"] = _randn(gen, n, (hq + 2 * hkv) * D)
    s["q"] = s["qkv"][:, : hq * D].view(n, hq, D)
    s["k"] = s["qkv"][:, hq * D : (hq + hkv) * D].view(n, hkv, D)
    s["v"] = s["qkv"][:, (hq + hkv) * D :].view(n, hkv, D)
    s["wq"] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(torch.bfloat16) if c["norm"] else None
    s["wk"] = (1 + 0.2 * torch.randn(D, generator=gen, device=DEV)).to(torch.bfloat16) if c["norm"] else None
    s["inv_freq"] = 500_000.0 ** (-torch.arange(0, c["rotary"], 2, dtype=torch.float64, device=DEV) / max(1, c["rotary"]))
    req = np.repeat(np.arange(c["batch"]), s["lq"])
    at = np.arange(n) - s["qo"][req] + (s["lk"] - s["lq"])[req]
    s["positions"] = torch.from_numpy((at + c["first"]).astype(np.int32)).to(DEV)
    where = s["slot"][torch.from_numpy(req).to(DEV), torch.from_numpy(at).to(DEV)]
    s["to_page"], s["to_slot"] = where // c["page"], where % c["page"]
    s["k_pages"], s["v_pages"] = _pages(s, gen, s["scales"][0]), _pages(s, gen, s["scales"][1])
    s["q_out"] = torch.empty(n, hq, D, dtype=torch.bfloat16, device=DEV)


def _prepare_weights(s, gen, hq):
    c = s["case"]
    n = int(s["lq"].sum())
    s["scales"] = (0.0625, 0.03125) if c["dtype"] == "e4m3" else (1.0, 1.0)
    s["q"] = (2 * torch.randn(n, hq, D, generator=gen, device=DEV)).to(torch.bfloat16)
    s["k_pages"] = _pages(s, gen, s["scales"][0])
    # the running sums of earlier steps: what a page's former owner left in the new keys' slots is still there
    s["weights"] = torch.rand(s["n_pool"], c["hkv"], c["page"], generator=gen, device=DEV) ** 4 * 8
    b, t = np.nonzero(np.arange(int(s["lq"].max()))[None, :] < s["lq"][:, None])
    s["row_b"], s["row_t"] = torch.from_numpy(b).to(DEV), torch.from_numpy(t).to(DEV)
    s["off"] = torch.from_numpy(s["lk"] - s["lq"]).to(DEV)
    s["tokens"] = torch.from_numpy(s["lq"]).to(DEV)
    # the log-sum-exp that the attention of these rows left: [tokens, heads], natural log
    x = _masked_logits(s)
    m = x.amax(-1, keepdim=True)
    lse = (m + (x - m).exp_().sum(-1, keepdim=True).log()).squeeze(-1)  # [batch, hkv, tokens, g]
    s["lse"] = lse[s["row_b"], :, s["row_t"]].reshape(n, hq).contiguous()


def _prepare_select(s, gen, hq):
    c = s["case"]
    # accumulated weights: a few heavy keys, a long tail, and keys that never got any
    w = torch.exp(2 * torch.randn(s["n_pool"], c["hkv"], c["page"], generator=gen, device=DEV))
    s["weights"] = torch.where(torch.rand(w.shape, generator=gen, device=DEV) < 0.1, torch.zeros_like(w), w)
    s["kept"] = torch.empty(c["batch"], c["hkv"], c["budget"], dtype=torch.int32, device=DEV)


def _prepare_compact(s, gen, hq):
    _prepare_select(s, gen, hq)
    s["scales"] = (0.0625, 0.03125) if s["case"]["dtype"] == "e4m3" else (1.0, 1.0)
    s["k_pages"], s["v_pages"] = _pages(s, gen, s["scales"][0]), _pages(s, gen, s["scales"][1])
    s["kept"] = _plain_select(s)


# ---- one pass --------------------------------------------------------------------------------------


def run(state):
    return {"append": _run_append, "weights": _run_weights, "select": _run_select, "compact": _run_compact}[state["case"]["op"]](state)


def _run_append(s):
    if own:
        s["ws"].append(s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"], s["q_out"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, positions=s["positions"])
        return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    s["q_out"] = _normed_and_rotated(s, s["q"], s["wq"]).to(torch.bfloat16)
    _write_rows(s, s["k_pages"], _normed_and_rotated(s, s["k"], s["wk"]), s["scales"][0])
    _write_rows(s, s["v_pages"], s["v"].float(), s["scales"][1])
    return {"q": s["q_out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _normed_and_rotated(s, x, w):
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    if not c["rotary"]:
        return x
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]  # far positions: in 64 bits
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    r, half = c["rotary"], c["rotary"] // 2
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :half], x[..., half:r])
    if c["interleaved"]:
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    else:
        y[..., :half], y[..., half:r] = a * cos - b * sin, a * sin + b * cos
    return y


def _write_rows(s, pages, x, scale):
    if s["case"]["dtype"] == "e4m3":
        x = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        pages = pages.view(torch.uint8)
    else:
        x = x.to(torch.bfloat16)
    if s["case"]["layout"] == "HND":
        pages[s["to_page"], :, s["to_slot"]] = x
    else:
        pages[s["to_page"], s["to_slot"]] = x


def _padded_keys(s):
    """[batch, hkv, keys, D] in 32 bits: each request's keys in order, zeros behind its last."""
    c = s["case"]
    pages = s["k_pages"].view(torch.uint8) if c["dtype"] == "e4m3" else s["k_pages"]
    pages = pages.transpose(1, 2) if c["layout"] == "HND" else pages  # [pool, page, hkv, D]
    k = pages[s["slot"] // c["page"], s["slot"] % c["page"]]
    k = k.view(torch.float8_e4m3fn).float() * s["scales"][0] if c["dtype"] == "e4m3" else k.float()
    return (k * s["valid"][:, :, None, None]).transpose(1, 2)


def _masked_logits(s):
    """[batch, hkv, tokens, g, keys]: the scaled (and capped) logits, -inf where a token does not see a key."""
    c = s["case"]
    g, t = c["hq"] // c["hkv"], int(s["lq"].max())
    q = torch.zeros(c["batch"], t, c["hkv"], g, D, device=DEV)
    q[s["row_b"], s["row_t"]] = s["q"].float().view(-1, c["hkv"], g, D)
    q = q.permute(0, 2, 1, 3, 4).reshape(c["batch"], c["hkv"], t * g, D)
    x = torch.matmul(q, _padded_keys(s).transpose(2, 3)).mul_(1 / math.sqrt(D)).view(c["batch"], c["hkv"], t, g, -1)
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    ti, j = torch.arange(t, device=DEV), torch.arange(x.shape[-1], device=DEV)
    seen = s["valid"][:, None, :] & (ti[None, :, None] < s["tokens"][:, None, None])
    if c["causal"]:
        seen = seen & (j[None, None, :] <= ti[None, :, None] + s["off"][:, None, None])
    return x.masked_fill_(~seen[:, None, :, None, :], -math.inf)


def _run_weights(s):
    c = s["case"]
    if own:
        s["ws"].key_weights(s["q"], s["k_pages"], s["lse"], s["weights"], decay=c["decay"], new_keys=True)
        return s["weights"]
    g, t = c["hq"] // c["hkv"], int(s["lq"].max())
    x = _masked_logits(s)
    lse = torch.zeros(c["batch"], t, c["hkv"], g, device=DEV)
    lse[s["row_b"], s["row_t"]] = s["lse"].view(-1, c["hkv"], g)
    w = x.sub_(lse.permute(0, 2, 1, 3)[..., None]).exp_().sum((2, 3))  # [batch, hkv, keys]
    b, j = s["valid"].nonzero(as_tuple=True)
    page, slot = s["slot"][b, j] // c["page"], s["slot"][b, j] % c["page"]
    old = torch.where((j < s["off"][b])[:, None], c["decay"] * s["weights"][page, :, slot], 0.0)
    s["weights"][page, :, slot] = old + w[b, :, j]
    return s["weights"]


def _run_select(s):
    c = s["case"]
    if own:
        s["ws"].select_keys(s["weights"], c["budget"], s["kept"], recent=c["recent"], sink=c["sink"])
    else:
        s["kept"] = _plain_select(s)
    return s["kept"]


def _plain_select(s):
    c = s["case"]
    n = s["valid"].shape[1]
    j = torch.arange(n, device=DEV)
    klen = s["valid"].sum(1)
    w = s["weights"][s["slot"] // c["page"], :, s["slot"] % c["page"]].transpose(1, 2)  # [batch, hkv, keys]
    always = (j[None, :] < c["sink"]) | (j[None, :] >= klen[:, None] - c["recent"])
    w = torch.where(always[:, None, :], math.inf, w)
    w = torch.where(s["valid"][:, None, :], w, -math.inf)
    first = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., : c["budget"]]
    first = torch.nn.functional.pad(first, (0, c["budget"] - first.shape[-1]), value=n)
    rank = torch.arange(c["budget"], device=DEV)
    gone = rank[None, :] >= torch.clamp(klen, max=c["budget"])[:, None]
    kept = torch.where(gone[:, None, :], n, first).sort(-1).values
    return torch.where(gone[:, None, :], -1, kept).to(torch.int32)


def _run_compact(s):
    c = s["case"]
    if own:
        s["ws"].compact(s["kept"], s["k_pages"], s["v_pages"], s["weights"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights"]}
    b, h, j = (s["kept"] >= 0).nonzero(as_tuple=True)
    src, dst = s["slot"][b, s["kept"][b, h, j].long()], s["slot"][b, j]
    fp, fs, tp, ts = src // c["page"], src % c["page"], dst // c["page"], dst % c["page"]
    _move(s, s["k_pages"], h, fp, fs, tp, ts)
    _move(s, s["v_pages"], h, fp, fs, tp, ts)
    s["weights"][tp, h, ts] = s["weights"][fp, h, fs]
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"], "weights": s["weights"]}


def _move(s, pages, h, fp, fs, tp, ts):
    pages = pages.view(torch.uint8) if s["case"]["dtype"] == "e4m3" else pages
    if s["case"]["layout"] == "HND":
        pages[tp, h, ts] = pages[fp, h, fs]
    else:
        pages[tp, ts, h] = pages[fp, fs, h]


# ---- what a pass cannot do without -------------------------------------------------------------------


def work(case):
    lq, lk = (x.astype(np.float64) for x in _lengths(case))
    hkv, e = case["hkv"], 1 if case.get("dtype") == "e4m3" else 2
    hq = case.get("hq", hkv)
    if case["op"] == "append":
        n = lq.sum()
        return {"bytes": n * D * ((hq + 2 * hkv) * 2 + hq * 2 + 2 * hkv * e), "flops": n * D * (hq + hkv) * 8.0}
    if case["op"] == "weights":
        pairs = (lq * lk - (lq * (lq - 1) / 2 if case["causal"] else 0)).sum()
        return {"bytes": lk.sum() * hkv * (D * e + 8) + lq.sum() * hq * (D * 2 + 4), "flops": pairs * hq * (2 * D + 4)}
    kept = np.minimum(lk, case["budget"]).sum()
    if case["op"] == "select":
        return {"bytes": hkv * (lk.sum() * 4 + kept * 4), "flops": hkv * lk.sum()}
    moved = np.where(lk > case["budget"], np.minimum(lk, case["budget"]) - case["sink"], 0).sum()
    return {"bytes": hkv * (kept * 4 + moved * 2 * (2 * D * e + 4)), "flops": hkv * moved}


# ---- the definitions in 64 bits ------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    lists = np.split(s["order"].cpu().numpy(), s["kv"][1:-1])
    return {"append": _exact_append, "weights": _exact_weights, "select": _exact_select, "compact": _exact_compact}[case["op"]](s, lists)


def _rows(case, pages, pl, h, n):
    """Rows 0 .. n - 1 of a request's list of pages, KV head h."""
    p = torch.from_numpy(pl).to(DEV)
    x = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    x = x[p, h] if case["layout"] == "HND" else x[p][:, :, h]
    return x.reshape(-1, x.shape[-1])[:n].view(pages.dtype)


def _exact_append(s, lists):
    c = s["case"]
    f = s["inv_freq"].cpu().numpy()
    half = len(f)
    phase = np.outer(s["positions"].cpu().numpy().astype(np.float64), f)
    turn = torch.from_numpy(np.exp(1j * phase)).to(DEV)[:, None, :]

    def full(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        if not half:
            return x
        head, rest = x[..., : 2 * half], x[..., 2 * half :]
        z = torch.view_as_complex(head.unflatten(-1, (half, 2)).contiguous()) if c["interleaved"] else torch.complex(head[..., :half], head[..., half:])
        z = z * turn
        return torch.cat([torch.view_as_real(z).flatten(-2) if c["interleaved"] else torch.cat([z.real, z.imag], -1), rest], -1)

    out = {"q": full(s["q"], s["wq"])}
    for name, x, scale in (("k_pages", full(s["k"], s["wk"]), s["scales"][0]), ("v_pages", s["v"].double(), s["scales"][1])):
        pages = s[name].double()
        x = (x / scale).clamp(-448, 448) if c["dtype"] == "e4m3" else x
        for i, pl in enumerate(lists):
            at = np.arange(s["lk"][i] - s["lq"][i], s["lk"][i])
            p, t = torch.from_numpy(pl[at // c["page"]]).to(DEV), torch.from_numpy(at % c["page"]).to(DEV)
            new = x[int(s["qo"][i]) : int(s["qo"][i + 1])]
            if c["layout"] == "HND":
                pages[p, :, t] = new
            else:
                pages[p, t] = new
        out[name] = pages
    return out


def _exact_weights(s, lists):
    c = s["case"]
    g = c["hq"] // c["hkv"]
    out = s["weights"].double()
    for i, pl in enumerate(lists):
        n, t = int(s["lk"][i]), int(s["lq"][i])
        rows = slice(int(s["qo"][i]), int(s["qo"][i + 1]))
        p, at = torch.from_numpy(pl[np.arange(n) // c["page"]]).to(DEV), torch.arange(n, device=DEV) % c["page"]
        late = torch.arange(n, device=DEV)[None, :] > torch.arange(n - t, n, device=DEV)[:, None]
        for h in range(c["hkv"]):
            k = _rows(c, s["k_pages"], pl, h, n).double() * s["scales"][0]
            z = torch.einsum("tgd,nd->gtn", s["q"][rows, h * g : (h + 1) * g].double(), k) / D**0.5
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            z = torch.exp(z - s["lse"][rows, h * g : (h + 1) * g].double().t()[:, :, None])
            if c["causal"]:
                z = z.masked_fill(late, 0.0)
            before = out[p, h, at] * c["decay"]
            before[n - t :] = 0
            out[p, h, at] = before + z.sum((0, 1))
    return out


def _exact_select(s, lists):
    c = s["case"]
    kept = np.full((c["batch"], c["hkv"], c["budget"]), -1, np.int32)
    w = s["weights"].cpu().numpy()
    for i, pl in enumerate(lists):
        n = int(s["lk"][i])
        m = min(n, c["budget"])
        for h in range(c["hkv"]):
            x = w[pl, h].reshape(-1)[:n].astype(np.float64)
            free = np.arange(c["sink"], n - c["recent"]) if n > m else np.arange(n)
            take = m - (n - len(free))
            best = free[np.argsort(-x[free], kind="stable")[:take]]
            kept[i, h, :m] = np.sort(np.concatenate([best, np.setdiff1d(np.arange(n), free)]))
    return kept


def _exact_compact(s, lists):
    c = s["case"]
    out = {"k_pages": s["k_pages"].double(), "v_pages": s["v_pages"].double(), "weights": s["weights"].double()}
    kept = s["kept"].cpu().numpy()
    for i, pl in enumerate(lists):
        for h in range(c["hkv"]):
            src = kept[i, h][kept[i, h] >= 0]
            dst = np.arange(len(src))
            p, t = torch.from_numpy(pl[dst // c["page"]]).to(DEV), torch.from_numpy(dst % c["page"]).to(DEV)
            pick = torch.from_numpy(src.astype(np.int64)).to(DEV)
            for name in ("k_pages", "v_pages"):
                new = _rows(c, s[name], pl, h, int(s["lk"][i]))
                new = (new.view(torch.uint8)[pick].view(new.dtype) if c["dtype"] == "e4m3" else new[pick]).double()
                if c["layout"] == "HND":
                    out[name][p, h, t] = new
                else:
                    out[name][p, t, h] = new
            flat = torch.from_numpy(pl).to(DEV)
            out["weights"][p, h, t] = s["weights"][flat, h].reshape(-1)[pick].double()
    return out
