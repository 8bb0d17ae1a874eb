"""The paged decode operators as they are measured: their cases, their inputs and their plain forms.

Three operators carry one decode step over a paged key/value cache:

  assign   pages, slots, positions and block tables of a step's new rows, from the requests' lengths;
  append   RMS norm of every query and key head, rotary positions, and the new K / V rows written into the cache;
  attend   attention of one new query row per head over a request's cached rows, read through its block table.

``own`` chooses between the plain form (elementary torch operations in 32 bits) and the library's kernels.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "e4m3": 1}


# ------------------------------------------------------------------------------------------- cases
def _assign(name, batch, len_min, len_max, new_min, new_max, page, pad):
    return {"name": name, "op": "assign", "batch": batch, "len_min": len_min, "len_max": len_max, "new_min": new_min,
            "new_max": new_max, "page": page, "pad": pad}


def _append(name, tokens, pad, h_q, h_kv, d, page, dtype, cache, order, norm, rot, layout, scaling, pos_max, run):
    return {"name": name, "op": "append", "tokens": tokens, "pad": pad, "h_q": h_q, "h_kv": h_kv, "d": d, "page": page,
            "dtype": dtype, "cache": cache, "order": order, "norm": norm, "rot": rot, "layout": layout,
            "scaling": scaling, "pos_max": pos_max, "run": run}


def _attend(name, batch, len_min, len_max, h_q, h_kv, d, page, dtype, cache, order, softcap, window, slopes):
    return {"name": name, "op": "attend", "batch": batch, "len_min": len_min, "len_max": len_max, "h_q": h_q,
            "h_kv": h_kv, "d": d, "page": page, "dtype": dtype, "cache": cache, "order": order, "softcap": softcap,
            "window": window, "slopes": slopes}


def listed():
    return [
        # a small decode batch: the ragged batch of 8 prompts, one new row each
        _assign("assign decode 8", 8, 8192, 32768, 1, 1, 16, 0),
        # a full decode batch padded to a captured step's size; some requests are idle (no new row)
        _assign("assign decode 1024", 1024, 1, 8191, 0, 1, 16, 37),
        # chunked prefill of 64 requests at any depth, the step's token budget not quite filled
        _assign("assign chunks 64", 64, 0, 24571, 0, 8191, 16, 129),
        # one request decoding: 8B-shaped heads, normed queries and keys
        _append("append decode 1", 1, 0, 32, 8, 128, 16, "bf16", "bf16", "head", True, 128, "half", "plain", 131072, 1),
        # a decode batch padded for a captured step: 70B-shaped heads, half of each head rotated in pairs
        _append("append decode 200", 200, 56, 64, 8, 128, 16, "f16", "f16", "row", False, 64, "interleaved", "linear",
                32768, 1),
        # a prefill chunk deep in a long prompt whose last page is not full
        _append("append prefill 8200", 8200, 0, 32, 8, 128, 16, "bf16", "bf16", "head", True, 128, "half", "banded",
                131072, 8200),
        # several prompts' chunks at once into an 8-bit cache, 70B-shaped heads
        _append("append prefill 32768", 32768, 0, 64, 8, 128, 64, "bf16", "e4m3", "head", True, 128, "half", "ramp",
                131072, 4096),
        # a tiny model's short prompt: latency alone
        _attend("attend 1 x 517", 1, 517, 517, 4, 2, 64, 16, "bf16", "bf16", "head", 0.0, 0, False),
        # one request at the benchmark's 128K context, 8B-shaped
        _attend("attend 1 x 131072", 1, 131072, 131072, 32, 8, 128, 16, "bf16", "bf16", "head", 0.0, 0, False),
        # the ragged batch of 8
        _attend("attend 8 ragged", 8, 8192, 32768, 32, 8, 128, 16, "bf16", "bf16", "head", 0.0, 0, False),
        # a full decode batch over an 8-bit cache: short and long requests, capped scores and a sliding window
        _attend("attend 256 short", 256, 1, 4095, 64, 8, 128, 32, "f16", "e4m3", "row", 50.0, 2048, False),
        # the largest: 32 long requests, 70B-shaped, scores with a distance bias
        _attend("attend 32 long", 32, 2048, 65536, 64, 8, 128, 64, "bf16", "bf16", "head", 0.0, 0, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["assign", "append", "append", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    order = rng.choice(["head", "row"])
    d = rng.choice([64, 128, 128])
    h_kv = rng.choice([1, 2, 4, 8, 8])
    h_q = h_kv * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
    page = rng.choice([8, 16, 16, 32, 64, 128, rng.randint(1, 256)])
    if op == "assign":
        batch = _log_int(rng, 1, 1024)
        budget = _log_int(rng, 1, 262144)
        new_max = max(1, min(8191, budget // batch)) if rng.random() < 0.6 else 1
        len_min = rng.choice([0, 0, 1, rng.randint(0, 4000)])
        c = _assign("", batch, len_min, len_min + _log_int(rng, 1, 30000), rng.choice([0, 1]), new_max, page,
                    rng.randint(0, 256))
    elif op == "append":
        # no more values than the largest listed case; one row a page only for decode batches
        tokens = _log_int(rng, 1, min(32768, 32768 * 80 * 128 // ((h_q + 2 * h_kv) * d)))
        runs = [1, tokens] if tokens <= 1024 else [1000, tokens]
        c = _append("", tokens, rng.choice([0, rng.randint(0, 64)]), h_q, h_kv, d, page, dtype, cache, order,
                    rng.random() < 0.6, rng.choice([d, d, d // 2, d // 4]), rng.choice(["half", "half", "interleaved"]),
                    rng.choice(["plain", "linear", "banded", "ramp"]), rng.choice([32768, 131072, 1048576]),
                    rng.choice(runs))
    else:
        batch = _log_int(rng, 1, 256)
        # no more rows than the largest listed case
        most = min(131072, 1048576 // batch)
        len_max = _log_int(rng, 1, most)
        len_min = rng.choice([0, 1, len_max, rng.randint(0, len_max)])
        c = _attend("", batch, min(len_min, len_max), len_max, h_q, h_kv, d, page, dtype, cache, order,
                    rng.choice([0.0, 0.0, 30.0, 50.0]), rng.choice([0, 0, rng.randint(1, len_max)]),
                    rng.random() < 0.3)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------ inputs
def _spread(lo, hi, n, g):
    """n whole numbers spread evenly over lo .. hi, in an order of the seed's."""
    x = torch.tensor([hi] if n == 1 else [lo + round((hi - lo) * i / (n - 1)) for i in range(n)], device="cuda")
    return x[torch.randperm(n, generator=g, device="cuda")]


def _tables(lens, page, max_blocks, ids):
    """Block tables [batch, max_blocks] that give each request its pages from `ids` in order, and how many were given."""
    n = (lens + page - 1) // page
    first = torch.cumsum(n, 0) - n
    col = torch.arange(max_blocks, device="cuda")
    at = first[:, None] + col
    held = col < n[:, None]
    return torch.where(held, ids[at.clamp(max=ids.numel() - 1)], 0).to(torch.int32), int(n.sum())


def _pages(lo, hi, n, page):
    return sum(-(-x // page) for x in ([hi] if n == 1 else [lo + round((hi - lo) * i / (n - 1)) for i in range(n)]))


def _pool_shape(c, n_pages):
    return (n_pages, c["h_kv"], c["page"], c["d"]) if c["order"] == "head" else (n_pages, c["page"], c["h_kv"], c["d"])


def _rotation(c):
    """Angles per position [rot / 2] in 64 bits and the factor on cos and sin, with the long-context scalings."""
    rot, base, factor, original = c["rot"], 500000.0, 8.0, 8192
    f = base ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    if c["scaling"] == "linear":
        return f / factor, 1.0
    if c["scaling"] == "banded":      # long waves are stretched, short ones kept, those between blended
        low, high = 1.0, 4.0
        s = ((original * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        return (1 - s) * f / factor + s * f, 1.0
    if c["scaling"] == "ramp":        # by the number of turns over the original context, linear in the index
        def index(turns):
            return rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(index(32.0))), min(rot - 1, math.ceil(index(1.0)))
        r = ((torch.arange(rot // 2, device="cuda", dtype=torch.float64) - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return r * f / factor + (1 - r) * f, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"assign": _prepare_assign, "append": _prepare_append, "attend": _prepare_attend}[case["op"]](case, g)


def _prepare_assign(c, g):
    batch, page = c["batch"], c["page"]
    lens, n_new = _spread(c["len_min"], c["len_max"], batch, g), _spread(c["new_min"], c["new_max"], batch, g)
    max_blocks = -(-(c["len_max"] + c["new_max"]) // page)
    n_pages = _pages(c["len_min"], c["len_max"], batch, page) + batch + -(-int(n_new.sum()) // page) + 5
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    tables, used = _tables(lens, page, max_blocks, ids)
    max_tokens = int(n_new.sum()) + c["pad"]
    long = dict(dtype=torch.int64, device="cuda")
    return {"case": c, "lens": lens, "n_new": n_new, "free_pages": ids[used:].contiguous(), "n_pages": n_pages,
            "free_head": torch.full((1,), 3, **long), "block_tables": tables, "max_tokens": max_tokens,
            "lens_out": torch.empty(batch, **long), "free_head_out": torch.empty(1, **long),
            "indptr": torch.empty(batch + 1, **long), "slots": torch.empty(max_tokens, **long),
            "positions": torch.empty(max_tokens, **long),
            "seq_ids": torch.empty(max_tokens, dtype=torch.int32, device="cuda")}


def _prepare_append(c, g):
    n, page, d = c["tokens"] + c["pad"], c["page"], c["d"]
    dtype, cache = DTYPES[c["dtype"]], DTYPES[c["cache"]]
    heads = c["h_q"] + 2 * c["h_kv"]
    qkv = torch.randn((n, heads, d), generator=g, device="cuda", dtype=dtype)      # a fused projection's rows
    t = torch.arange(n, device="cuda")
    if c["run"] == 1:                                                              # one row of each request
        n_pages = n + 3
        pages = torch.randperm(n_pages, generator=g, device="cuda")
        slots = pages[t] * page + torch.randint(0, page, (n,), generator=g, device="cuda")
        positions = torch.randint(0, c["pos_max"], (n,), generator=g, device="cuda")
    else:                                                                          # runs of `run` rows of one request
        per_run = -(-c["run"] // page)
        n_pages = -(-n // c["run"]) * per_run + 3
        pages = torch.randperm(n_pages, generator=g, device="cuda")
        seq, row = t // c["run"], t % c["run"]
        slots = pages[seq * per_run + row // page] * page + row % page
        first = torch.randint(0, max(1, c["pos_max"] - c["run"]), (n,), generator=g, device="cuda")
        positions = first[seq] + row
    slots = torch.where(t < c["tokens"], slots, -1)
    # one page behind the pool takes the plain form's writes of the padding rows
    store = torch.zeros((2, *_pool_shape(c, n_pages + 1)), device="cuda", dtype=dtype).to(cache)
    weights = [1 + 0.1 * torch.randn(d, generator=g, device="cuda") if c["norm"] else None for _ in range(2)]
    scales = [0.01 + 0.01 * torch.rand(c["h_kv"], generator=g, device="cuda") if c["cache"] == "e4m3" else None
              for _ in range(2)]
    inv_freq, factor = _rotation(c)
    return {"case": c, "q": qkv[:, :c["h_q"]], "k": qkv[:, c["h_q"]:c["h_q"] + c["h_kv"]],
            "v": qkv[:, c["h_q"] + c["h_kv"]:], "positions": positions, "slots": slots, "n_pages": n_pages,
            "store": store, "k_cache": store[0][:n_pages], "v_cache": store[1][:n_pages],
            "q_weight": None if weights[0] is None else weights[0].to(dtype),
            "k_weight": None if weights[1] is None else weights[1].to(dtype), "k_scale": scales[0],
            "v_scale": scales[1], "inv_freq": inv_freq, "factor": factor,
            "q_out": torch.zeros((n, c["h_q"], d), dtype=dtype, device="cuda")}


def _prepare_attend(c, g):
    batch, page, d = c["batch"], c["page"], c["d"]
    dtype, cache = DTYPES[c["dtype"]], DTYPES[c["cache"]]
    lens = _spread(c["len_min"], c["len_max"], batch, g)
    n_pages = _pages(c["len_min"], c["len_max"], batch, page) + 3
    ids = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    tables, _ = _tables(lens, page, -(-c["len_max"] // page), ids)
    shape = _pool_shape(c, n_pages)
    scales = [None, None]
    pools = [torch.randn(shape, generator=g, device="cuda", dtype=dtype) for _ in range(2)]
    if c["cache"] == "e4m3":
        scales = [0.01 + 0.01 * torch.rand(c["h_kv"], generator=g, device="cuda") for _ in range(2)]
        pools = [(x * 64).clamp(-E4M3_MAX, E4M3_MAX).to(cache) for x in pools]
    q = 1.5 * torch.randn((batch, c["h_q"], d), generator=g, device="cuda")
    slopes = 2.0 ** (-8.0 * torch.arange(1, c["h_q"] + 1, device="cuda", dtype=torch.float32) / c["h_q"])
    return {"case": c, "q": q.to(dtype), "k_cache": pools[0], "v_cache": pools[1], "block_tables": tables, "lens": lens,
            "n_pages": n_pages, "k_scale": scales[0], "v_scale": scales[1], "slopes": slopes if c["slopes"] else None,
            "o": torch.empty((batch, c["h_q"], d), dtype=dtype, device="cuda"),
            "lse": torch.empty((batch, c["h_q"]), device="cuda")}


# ------------------------------------------------------------------------------------- plain forms
def _assign_plain(s):
    page, table, lens = s["case"]["page"], s["block_tables"].long(), s["lens"]
    after = lens + s["n_new"]
    held = (lens + page - 1) // page
    need = (after + page - 1) // page - held
    first = s["free_head"] + torch.cumsum(need, 0) - need          # of each request's new pages in the queue
    ends = torch.cumsum(s["n_new"], 0)
    last = s["free_pages"].numel() - 1
    col = torch.arange(table.shape[1], device="cuda")
    is_new = (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(is_new, s["free_pages"][(first[:, None] + col - held[:, None]).clamp(0, last)].long(), table)
    t = torch.arange(s["max_tokens"], device="cuda")
    seq = torch.searchsorted(ends, t, right=True)
    real = seq < lens.numel()
    at = seq.clamp(max=lens.numel() - 1)
    pos = torch.where(real, lens[at] + t - (ends - s["n_new"])[at], 0)
    slots = table[at, pos // page] * page + pos % page
    return {"slots": torch.where(real, slots, -1), "positions": pos,
            "seq_ids": torch.where(real, seq, -1).to(torch.int32), "lens": after,
            "indptr": torch.cat([ends.new_zeros(1), ends]), "free_head": s["free_head"] + need.sum(),
            "block_tables": table.to(torch.int32)}


def _to_cache(x, scale, cache):
    if cache != "e4m3":
        return x.to(DTYPES[cache])
    return (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(DTYPES[cache])


def _write(store, order, page, off, rows):
    """rows [n, h_kv, d] into the pool at (page, off); 8-bit values are moved as bytes."""
    if rows.element_size() == 1:
        store, rows = store.view(torch.uint8), rows.view(torch.uint8)
    if order == "head":
        store[page, :, off] = rows
    else:
        store[page, off] = rows


def _append_plain(s):
    c = s["case"]
    rot, d = c["rot"], c["d"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    cos, sin = (torch.cos(angle) * s["factor"]).float()[:, None], (torch.sin(angle) * s["factor"]).float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
        if c["layout"] == "half":
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        return torch.cat([y, x[..., rot:]], -1) if rot < d else y

    real = s["slots"] >= 0
    q_out = torch.where(real[:, None, None], turned(s["q"], s["q_weight"]).to(DTYPES[c["dtype"]]), s["q_out"])
    slots = torch.where(real, s["slots"], s["n_pages"] * c["page"])
    page, off = slots // c["page"], slots % c["page"]
    _write(s["store"][0], c["order"], page, off, _to_cache(turned(s["k"], s["k_weight"]), s["k_scale"], c["cache"]))
    _write(s["store"][1], c["order"], page, off, _to_cache(s["v"].float(), s["v_scale"], c["cache"]))
    return {"q": q_out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _rows(pool, order, table):
    """The rows of every table's pages [batch, h_kv, blocks * page, d] in 32 bits."""
    kind = pool.dtype
    x = (pool.view(torch.uint8) if pool.element_size() == 1 else pool)[table].view(kind)
    x = x.permute(0, 2, 1, 3, 4) if order == "head" else x.permute(0, 3, 1, 2, 4)
    return x.float().reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _attend_plain(s):
    c, lens = s["case"], s["lens"][:, None, None, None]
    batch, h_kv, d = c["batch"], c["h_kv"], c["d"]
    group = c["h_q"] // h_kv
    table = s["block_tables"].long()
    q = s["q"].float().view(batch, h_kv, group, d)
    z = q @ _rows(s["k_cache"], c["order"], table).transpose(-1, -2) / math.sqrt(d)
    if s["k_scale"] is not None:
        z = z * s["k_scale"][:, None, None]
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    t = torch.arange(z.shape[-1], device="cuda")
    if s["slopes"] is not None:
        z = z + s["slopes"].view(h_kv, group, 1) * (t - (lens - 1))
    seen = t < lens
    if c["window"]:
        seen = seen & (t >= lens - c["window"])
    z = torch.where(seen, z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(z - torch.where(m == -math.inf, 0.0, m)), 0.0)
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, 0, :, None], _rows(s["v_cache"], c["order"], table), 0.0)
    o = p @ v / torch.where(total == 0, 1.0, total)
    if s["v_scale"] is not None:
        o = o * s["v_scale"][:, None, None]
    return {"o": o.view(batch, c["h_q"], d).to(DTYPES[c["dtype"]]),
            "lse": (m + torch.log(total)).view(batch, c["h_q"])}


# --------------------------------------------------------------------------------- the library's own
def _workspace(K, n):
    ws = torch.zeros(n + K.WS_ALIGN, dtype=torch.uint8, device="cuda")
    off = (-ws.data_ptr()) % K.WS_ALIGN
    return ws[off:off + n]


def _plan(s):
    """What a serving program keeps next to its buffers: descriptors and a workspace."""
    from attention_kv_cache_gb300 import kvsel as K
    c = s["case"]
    kinds = {"bf16": K.DTYPE_BF16, "f16": K.DTYPE_F16, "e4m3": K.DTYPE_E4M3}
    if c["op"] == "assign":
        return {"K": K, "ws": _workspace(K, K.kvsel_page_assign_workspace_size(c["batch"]))}
    cache = K.make_cache_desc(h_q=c["h_q"], h_kv=c["h_kv"], head_dim=c["d"], page_size=c["page"], n_pages=s["n_pages"],
                              dtype=kinds[c["dtype"]], cache_dtype=kinds[c["cache"]],
                              order=K.ORDER_HEAD if c["order"] == "head" else K.ORDER_ROW)
    if c["op"] == "append":
        rope = K.make_rope_desc(rot_dim=c["rot"],
                                layout=K.ROPE_HALF if c["layout"] == "half" else K.ROPE_INTERLEAVED,
                                factor=s["factor"], norm_eps=1e-6, q=s["q"], k=s["k"], v=s["v"])
        return {"K": K, "cache": cache, "rope": rope, "ws": _workspace(K, K.WS_ALIGN)}
    attend = K.make_paged_attend_desc(batch=c["batch"], max_blocks=s["block_tables"].shape[1], softcap=c["softcap"],
                                      window=c["window"])
    return {"K": K, "cache": cache, "attend": attend,
            "ws": _workspace(K, K.kvsel_paged_attend_workspace_size(cache, attend))}


def _own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    p, op = s["plan"], s["case"]["op"]
    K = p["K"]
    if op == "assign":
        K.kvsel_page_assign(s["case"]["page"], s["n_pages"], s["lens"], s["n_new"], s["free_pages"], s["free_head"],
                            s["block_tables"], s["lens_out"], s["free_head_out"], s["indptr"], s["slots"],
                            s["positions"], s["seq_ids"], p["ws"])
        return {"slots": s["slots"], "positions": s["positions"], "seq_ids": s["seq_ids"], "lens": s["lens_out"],
                "indptr": s["indptr"], "free_head": s["free_head_out"], "block_tables": s["block_tables"]}
    if op == "append":
        K.kvsel_rope_append(p["cache"], p["rope"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["q_weight"],
                            s["k_weight"], s["inv_freq"], s["q_out"], s["k_cache"], s["v_cache"], s["k_scale"],
                            s["v_scale"], p["ws"])
        return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    K.kvsel_paged_attend(p["cache"], p["attend"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["lens"],
                         s["slopes"], s["k_scale"], s["v_scale"], s["o"], s["lse"], p["ws"])
    return {"o": s["o"], "lse": s["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"assign": _assign_plain, "append": _append_plain, "attend": _attend_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------- work
def _values(lo, hi, n):
    return [hi] if n == 1 else [lo + round((hi - lo) * i / (n - 1)) for i in range(n)]


def work(case):
    c = case
    if c["op"] == "assign":
        rows = sum(_values(c["new_min"], c["new_max"], c["batch"]))
        pages = rows / c["page"]
        # per request: two lengths read, the new length, the offset and the page of its first row; per new page: its
        # id read and written; per row: slot, position and request
        return {"bytes": c["batch"] * (3 * 8 + 8 + 4) + pages * 8 + (rows + c["pad"]) * 20, "flops": 0}
    if c["op"] == "append":
        n, row = c["tokens"], c["d"] * BYTES[c["dtype"]]
        read = n * ((c["h_q"] + 2 * c["h_kv"]) * row + 16)
        write = n * (c["h_q"] * row + 2 * c["h_kv"] * c["d"] * BYTES[c["cache"]])
        turned = n * (c["h_q"] + c["h_kv"])
        return {"bytes": read + write, "flops": turned * (3 * c["rot"] + (4 * c["d"] if c["norm"] else 0))}
    lens = _values(c["len_min"], c["len_max"], c["batch"])
    seen = sum(min(x, c["window"]) if c["window"] else x for x in lens)
    kv = 2 * c["h_kv"] * c["d"] * BYTES[c["cache"]]
    io = c["batch"] * c["h_q"] * (2 * c["d"] * BYTES[c["dtype"]] + 4)
    return {"bytes": seen * kv + io + seen / c["page"] * 4, "flops": seen * c["h_q"] * 4 * c["d"]}


# --------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"assign": _assign_exact, "append": _append_exact, "attend": _attend_exact}[case["op"]](s)


def _assign_exact(s):
    """Request by request, as a host scheduler would: rows take the pages they have, then the queue's next ones."""
    page = s["case"]["page"]
    lens, n_new, free = s["lens"].tolist(), s["n_new"].tolist(), s["free_pages"].cpu()
    tables, head = s["block_tables"].cpu().clone(), int(s["free_head"])
    slots = torch.full((s["max_tokens"],), -1, dtype=torch.int64)
    positions = torch.zeros(s["max_tokens"], dtype=torch.int64)
    seq_ids = torch.full((s["max_tokens"],), -1, dtype=torch.int32)
    indptr = [0]
    for b, (n, new) in enumerate(zip(lens, n_new)):
        have, want = -(-n // page), -(-(n + new) // page)
        tables[b, have:want] = free[head:head + want - have]
        head += want - have
        at = indptr[-1]
        pos = torch.arange(n, n + new)
        slots[at:at + new] = tables[b, pos // page].long() * page + pos % page
        positions[at:at + new] = pos
        seq_ids[at:at + new] = b
        indptr.append(at + new)
    return {"slots": slots, "positions": positions, "seq_ids": seq_ids, "lens": torch.tensor(lens) + torch.tensor(n_new),
            "indptr": torch.tensor(indptr), "free_head": torch.tensor([head]), "block_tables": tables}


def _append_exact(s):
    """Each head row as complex numbers turned by exp(i angle), in 64 bits."""
    c = s["case"]
    rot, page = c["rot"], c["page"]
    real = (s["slots"] >= 0).nonzero()[:, 0]
    slots = s["slots"][real]
    turn = torch.polar(torch.full((), float(s["factor"]), dtype=torch.float64, device="cuda"),
                       s["positions"][real, None].double() * s["inv_freq"])[:, None]

    def head(x, weight):
        x = x[real].double()
        if weight is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6) * weight.double()
        y = x.clone()
        pair = (slice(0, rot // 2), slice(rot // 2, rot)) if c["layout"] == "half" else \
            (slice(0, rot, 2), slice(1, rot, 2))
        w = torch.complex(x[..., pair[0]], x[..., pair[1]]) * turn
        y[..., pair[0]], y[..., pair[1]] = w.real, w.imag
        return y

    q = s["q_out"].double()
    q[real] = head(s["q"], s["q_weight"])
    out = {"q": q}
    for name, rows, scale in (("k_cache", head(s["k"], s["k_weight"]), s["k_scale"]),
                              ("v_cache", s["v"][real].double(), s["v_scale"])):
        if scale is not None:
            rows = (rows / scale.double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        pool = s[name].double()
        view = pool if c["order"] == "row" else pool.transpose(1, 2)      # [page, row, head, d]
        view[slots // page, slots % page] = rows
        out[name] = pool
    return out


def _attend_exact(s):
    """One request at a time: softmax of its visible rows' scores, in 64 bits."""
    c = s["case"]
    group, d, page = c["h_q"] // c["h_kv"], c["d"], c["page"]
    o = torch.zeros((c["batch"], c["h_q"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        t = torch.arange(first, n, device="cuda")
        ids = s["block_tables"][b, t // page].long()
        k, v = (x[ids, :, t % page] if c["order"] == "head" else x[ids, t % page]
                for x in (s["k_cache"].view(torch.uint8), s["v_cache"].view(torch.uint8)))
        k, v = (x.contiguous().view(s["k_cache"].dtype).double().transpose(0, 1) for x in (k, v))   # [h_kv, rows, d]
        z = torch.einsum("hgd,htd->hgt", s["q"][b].double().view(c["h_kv"], group, d), k) * d ** -0.5
        if s["k_scale"] is not None:
            z = z * s["k_scale"].double()[:, None, None]
        if c["softcap"]:
            z = torch.tanh(z / c["softcap"]) * c["softcap"]
        if s["slopes"] is not None:
            z = z - s["slopes"].double().view(c["h_kv"], group, 1) * (n - 1 - t).double()
        r = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), v)
        if s["v_scale"] is not None:
            r = r * s["v_scale"].double()[:, None, None]
        o[b], lse[b] = r.reshape(c["h_q"], d), torch.logsumexp(z, -1).reshape(-1)
    return {"o": o, "lse": lse}
