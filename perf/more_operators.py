"""The operators of prompts and beams over a paged cache as they are measured: their cases, inputs and plain forms.

Four operators join the paged decode:

  chunk    attention of many new tokens of each request (a prompt's chunk, the tokens of a draft) over its cached rows;
  prefix   attention of one new token per request, where groups of requests share the pages of a long prefix;
  select   the best continuations of every beam set: log-softmax over the vocabulary, the beams' sums, the first n;
  reorder  the beams' block tables after a selection: pages shared, freed, and the last page of a twin copied.

``own`` chooses between the plain form (elementary torch operations) and the library's kernels.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
MOST_SCORES = 4096 * 32 * 16384          # scores of a drawn attention case: those of the largest listed one
MOST_VALUES = 2 ** 31                    # of a drawn case's gathered keys, as the plain form holds them
MOST_COPIED = 64 * 3 * 16 * 32 * 8 * 128   # of a drawn case's copied pages, K alone


# ------------------------------------------------------------------------------------------- cases
def _chunk(name, batch, len_min, len_max, new_min, new_max, pad, h_q, h_kv, d, page, dtype, cache, order, softcap, window,
           slopes):
    return {"name": name, "op": "chunk", "batch": batch, "len_min": len_min, "len_max": len_max, "new_min": new_min,
            "new_max": new_max, "pad": pad, "h_q": h_q, "h_kv": h_kv, "d": d, "page": page, "dtype": dtype, "cache": cache,
            "order": order, "softcap": softcap, "window": window, "slopes": slopes}


def _prefix(name, groups, each, shared_min, shared_max, own_min, own_max, h_q, h_kv, d, page, dtype, cache, order, softcap,
            window, slopes):
    return {"name": name, "op": "prefix", "groups": groups, "each": each, "shared_min": shared_min,
            "shared_max": shared_max, "own_min": own_min, "own_max": own_max, "h_q": h_q, "h_kv": h_kv, "d": d,
            "page": page, "dtype": dtype, "cache": cache, "order": order, "softcap": softcap, "window": window,
            "slopes": slopes}


def _select(name, batch, beams, n_out, vocab, dtype, pad, ended, banned, first):
    return {"name": name, "op": "select", "batch": batch, "beams": beams, "n_out": n_out, "vocab": vocab, "dtype": dtype,
            "pad": pad, "ended": ended, "banned": banned, "first": first}


def _reorder(name, batch, beams, kept, prompt_min, prompt_max, grown, layers, h_kv, d, page, cache, order):
    return {"name": name, "op": "reorder", "batch": batch, "beams": beams, "kept": kept, "prompt_min": prompt_min,
            "prompt_max": prompt_max, "grown": grown, "layers": layers, "h_kv": h_kv, "d": d, "page": page,
            "cache": cache, "order": order}


def listed():
    return [
        # a decode batch that checks a draft of five tokens for every request
        _chunk("chunk draft 16 x 5", 16, 500, 8191, 5, 5, 3, 32, 8, 128, 16, "bf16", "bf16", "head", 0.0, 0, False),
        # chunks of a ragged batch of 8 prompts at any depth, an 8-bit cache, capped scores and a sliding window
        _chunk("chunk ragged 8", 8, 0, 7000, 1, 1023, 129, 32, 8, 64, 32, "f16", "e4m3", "row", 50.0, 4096, False),
        # a large chunk that ends a 16K prompt, 8B-shaped heads
        _chunk("chunk 4096 of 16384", 1, 12288, 12288, 4096, 4096, 0, 32, 8, 128, 16, "bf16", "bf16", "head", 0.0, 0, False),
        # one prompt's beams: 8B-shaped heads, a short tail of their own
        _prefix("prefix 1 x 8 of 8192", 1, 8, 8192, 8192, 33, 33, 32, 8, 128, 16, "bf16", "bf16", "head", 0.0, 0, False),
        # beams of a ragged batch of prompts, with a distance bias
        _prefix("prefix 24 x 4 ragged", 24, 4, 500, 8191, 1, 200, 32, 4, 64, 24, "f16", "f16", "row", 0.0, 0, True),
        # a serving batch behind one long system prompt, 70B-shaped heads, an 8-bit cache
        _prefix("prefix 64 of 32768", 1, 64, 32768, 32768, 1, 2047, 64, 8, 128, 64, "bf16", "e4m3", "head", 0.0, 0, False),
        # a single prompt's first step: every beam but the first is empty
        _select("select 1 x 4 first", 1, 4, 8, 32000, "f32", 2, False, False, True),
        # an odd vocabulary, some beams ended, some tokens not allowed
        _select("select 8 x 5 odd", 8, 5, 10, 50003, "bf16", 0, True, True, False),
        # a full batch of wide beams over a large vocabulary
        _select("select 64 x 16 wide", 64, 16, 32, 128256, "bf16", 1, True, False, False),
        # a single prompt's beams: latency alone
        _reorder("reorder 1 x 4", 1, 4, 3, 517, 517, 9, 2, 2, 64, 16, "bf16", "head"),
        # a ragged batch of prompts, an 8-bit cache whose pages hold rows outside heads
        _reorder("reorder 24 x 5 ragged", 24, 5, 3, 500, 8191, 117, 8, 4, 128, 24, "e4m3", "row"),
        # a full batch of wide beams: every layer of an 8B-shaped model's cache
        _reorder("reorder 64 x 8 deep", 64, 8, 5, 300, 363, 200, 32, 8, 128, 16, "bf16", "head"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _too_large(layers, rows, copied, width):
    return layers * rows * width > 2 ** 32 or layers * copied * width > MOST_COPIED


def draw(rng):
    op = rng.choice(["chunk", "prefix", "select", "reorder"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([dtype, dtype, "e4m3"])
    order = rng.choice(["head", "row"])
    d = rng.choice([64, 128, 128])
    h_kv = rng.choice([1, 2, 4, 8, 8])
    h_q = h_kv * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
    page = rng.choice([8, 16, 16, 32, 64, 128, rng.randint(1, 256)])
    softcap = rng.choice([0.0, 0.0, 0.0, 30.0])
    if op == "chunk":
        batch = _log_int(rng, 1, 64)
        new_max = _log_int(rng, 1, max(1, 4096 // batch))
        # no more scores, and no more gathered values, than the plain form of the largest listed case
        most = min(16384, MOST_SCORES // (batch * new_max * h_q), MOST_VALUES // (batch * h_kv * d))
        held = _log_int(rng, 1, max(1, most - new_max)) - 1
        c = _chunk("", batch, rng.choice([0, held, held // 2]), held, rng.choice([0, 1, new_max]), new_max,
                   rng.choice([0, rng.randint(0, 64)]), h_q, h_kv, d, page, dtype, cache, order, softcap,
                   rng.choice([0, 0, rng.randint(1, held + new_max)]), rng.random() < 0.25)
    elif op == "prefix":
        groups = rng.choice([1, 1, _log_int(rng, 1, 32)])
        each = _log_int(rng, 1, 128 // groups if groups > 1 else 128)
        batch = groups * each
        most = min(32768, MOST_SCORES // (batch * h_q), MOST_VALUES // (batch * h_kv * d))
        own_max = _log_int(rng, 1, max(1, min(2047, most // 4)))
        shared = _log_int(rng, 1, max(1, most - own_max))
        c = _prefix("", groups, each, rng.choice([0, shared, shared // 3]), shared, rng.choice([0, 1, own_max]), own_max,
                    h_q, h_kv, d, page, dtype, cache, order, softcap, rng.choice([0, 0, 0, rng.randint(1, shared)]),
                    rng.random() < 0.25)
    elif op == "select":
        beams = _log_int(rng, 1, 32)
        batch = _log_int(rng, 1, max(1, min(256, 1024 // beams)))
        vocab = rng.choice([_log_int(rng, 100, 128256), rng.choice([32000, 50003, 65536, 128256])])
        n_out = min(beams * rng.choice([1, 2, 2]), 64)
        c = _select("", batch, beams, n_out, vocab, rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([0, 0, 1, 7, 64]),
                    rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.15)
        if c["dtype"] == "f32" and batch * beams * vocab > 2 ** 26:
            c["dtype"] = "bf16"
    else:
        beams = _log_int(rng, 1, 32)
        batch = _log_int(rng, 1, max(1, 512 // beams))
        prompt = _log_int(rng, 1, 8191)
        grown = _log_int(rng, 1, 400)
        # no more values in the cache, and in the pages copied, than in the largest listed case
        layers = _log_int(rng, 1, 32)
        kept = rng.randint(1, beams)
        rows = batch * (prompt + beams * (grown + 4 * page))
        while layers > 1 and _too_large(layers, rows, batch * (beams - kept) * page, h_kv * d):
            layers //= 2
        while batch > 1 and _too_large(layers, rows, batch * (beams - kept) * page, h_kv * d):
            batch, rows = batch // 2, rows // 2
        c = _reorder("", batch, beams, kept, rng.choice([1, prompt, (prompt + 1) // 2]), prompt, grown, layers, h_kv, d, page,
                     cache, order)
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------ inputs
def _values(lo, hi, n):
    """n whole numbers spread evenly over lo .. hi (hi alone for one)."""
    return [hi] if n == 1 else [lo + round((hi - lo) * i / (n - 1)) for i in range(n)]


def _turned(values, by):
    """The same numbers from place `by` on: two spreads of one case are paired neither rising nor falling together."""
    by = by % len(values)
    return values[by:] + values[:by]


def _requests(c):
    """Rows held before the step and new rows of a chunk case's requests."""
    return _values(c["len_min"], c["len_max"], c["batch"]), _turned(_values(c["new_min"], c["new_max"], c["batch"]),
                                                                    c["batch"] // 3)


def _sharers(c):
    """Per group of a prefix case: its shared rows (whole pages) and its members' own rows."""
    shared = [x // c["page"] * c["page"] for x in _values(c["shared_min"], c["shared_max"], c["groups"])]
    own_rows = _turned(_values(c["own_min"], c["own_max"], c["groups"] * c["each"]), c["groups"] * c["each"] // 3)
    return shared, [own_rows[i * c["each"]:(i + 1) * c["each"]] for i in range(c["groups"])]


def _pool_shape(c, n_pages):
    return (n_pages, c["h_kv"], c["page"], c["d"]) if c["order"] == "head" else (n_pages, c["page"], c["h_kv"], c["d"])


def _pools(c, n_pages, g):
    """K and V pools and their scales: normal rows, as normed projections leave them."""
    pools = [torch.randn(_pool_shape(c, n_pages), generator=g, device="cuda", dtype=DTYPES[c["dtype"]]) for _ in range(2)]
    if c["cache"] != "e4m3":
        return pools, [None, None]
    scales = [0.01 + 0.01 * torch.rand(c["h_kv"], generator=g, device="cuda") for _ in range(2)]
    return [(x * 64).clamp(-E4M3_MAX, E4M3_MAX).to(DTYPES["e4m3"]) for x in pools], scales


def _slopes(c):
    return 2.0 ** (-8.0 * torch.arange(1, c["h_q"] + 1, device="cuda", dtype=torch.float32) / c["h_q"])


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"chunk": _prepare_chunk, "prefix": _prepare_prefix, "select": _prepare_select,
            "reorder": _prepare_reorder}[case["op"]](case, g)


def _prepare_chunk(c, g):
    page, dtype = c["page"], DTYPES[c["dtype"]]
    held, new = (torch.tensor(x, device="cuda") for x in _requests(c))
    lens = held + new
    n_blocks = (lens + page - 1) // page
    max_blocks = max(1, int(n_blocks.max()))
    n_pages = int(n_blocks.sum()) + 3
    ids = torch.randperm(n_pages, generator=g, device="cuda")
    first = torch.cumsum(n_blocks, 0) - n_blocks
    col = torch.arange(max_blocks, device="cuda")
    tables = torch.where(col < n_blocks[:, None], ids[(first[:, None] + col).clamp(max=n_pages - 1)], 0)
    pools, scales = _pools(c, n_pages, g)
    ends = torch.cumsum(new, 0)
    tokens = int(ends[-1]) + c["pad"]
    heads = c["h_q"] + 2 * c["h_kv"]
    qkv = (1.5 * torch.randn((max(1, tokens), heads, c["d"]), generator=g, device="cuda")).to(dtype)   # a projection's rows
    return {"case": c, "q": qkv[:tokens, :c["h_q"]], "k_cache": pools[0], "v_cache": pools[1], "k_scale": scales[0],
            "v_scale": scales[1], "block_tables": tables.to(torch.int32), "lens": lens, "new_max": c["new_max"],
            "indptr": torch.cat([ends.new_zeros(1), ends]), "slopes": _slopes(c) if c["slopes"] else None,
            "n_pages": n_pages, "o": torch.zeros((tokens, c["h_q"], c["d"]), dtype=dtype, device="cuda"),
            "lse": torch.zeros((tokens, c["h_q"]), device="cuda")}


def _prepare_prefix(c, g):
    page, dtype = c["page"], DTYPES[c["dtype"]]
    shared, own_rows = _sharers(c)
    batch = c["groups"] * c["each"]
    shared_blocks = torch.tensor(shared, device="cuda") // page
    lens = torch.tensor([s + x for s, xs in zip(shared, own_rows) for x in xs], device="cuda")
    n_blocks = (lens + page - 1) // page
    max_blocks = max(1, int(n_blocks.max()))
    by_request = shared_blocks.repeat_interleave(c["each"])
    tail = n_blocks - by_request
    n_pages = int(shared_blocks.sum() + tail.sum()) + 3
    ids = torch.randperm(n_pages, generator=g, device="cuda")
    first_shared = (torch.cumsum(shared_blocks, 0) - shared_blocks).repeat_interleave(c["each"])
    first_tail = shared_blocks.sum() + torch.cumsum(tail, 0) - tail
    col = torch.arange(max_blocks, device="cuda")
    at = torch.where(col < by_request[:, None], first_shared[:, None] + col, first_tail[:, None] + col - by_request[:, None])
    tables = torch.where(col < n_blocks[:, None], ids[at.clamp(0, n_pages - 1)], 0)
    pools, scales = _pools(c, n_pages, g)
    q = 1.5 * torch.randn((batch, c["h_q"], c["d"]), generator=g, device="cuda")
    return {"case": c, "q": q.to(dtype), "k_cache": pools[0], "v_cache": pools[1], "k_scale": scales[0],
            "v_scale": scales[1], "block_tables": tables.to(torch.int32), "lens": lens,
            "group_indptr": torch.arange(0, batch + 1, c["each"], device="cuda"),
            "shared_lens": torch.tensor(shared, device="cuda"), "slopes": _slopes(c) if c["slopes"] else None,
            "n_pages": n_pages, "o": torch.zeros((batch, c["h_q"], c["d"]), dtype=dtype, device="cuda"),
            "lse": torch.zeros((batch, c["h_q"]), device="cuda")}


def _prepare_select(c, g):
    batch, beams, vocab = c["batch"], c["beams"], c["vocab"]
    rows = batch * beams
    # a head's logits: a broad spread, the same few likely tokens for the beams of a set with some of each beam's own
    store = torch.randn((rows, vocab + c["pad"]), generator=g, device="cuda")
    store *= 2.0
    likely = torch.randint(0, vocab, (batch, 40), generator=g, device="cuda").repeat_interleave(beams, 0)
    store.scatter_add_(1, likely, 3.0 + 6.0 * torch.rand((rows, 40), generator=g, device="cuda"))
    if c["banned"]:
        store[:, torch.randint(0, vocab, (max(1, vocab // 50),), generator=g, device="cuda")] = -math.inf
    scores = -20.0 - 3.0 * torch.rand((batch, beams), generator=g, device="cuda")
    if c["first"]:
        scores = torch.full((batch, beams), -math.inf, device="cuda")
        scores[:, 0] = 0.0
    ended = torch.rand((batch, beams), generator=g, device="cuda") < (0.2 if c["ended"] else 0.0)
    return {"case": c, "logits": store.to(DTYPES[c["dtype"]])[:, :vocab], "scores": scores,
            "ended": ended.to(torch.uint8) if c["ended"] else None, "pad_token": min(2, vocab - 1),
            "scores_out": torch.empty((batch, c["n_out"]), device="cuda"),
            "parents": torch.empty((batch, c["n_out"]), dtype=torch.int32, device="cuda"),
            "tokens": torch.empty((batch, c["n_out"]), dtype=torch.int32, device="cuda"),
            "lse": torch.empty((batch, beams), device="cuda")}


def _prompts(c):
    return _values(c["prompt_min"], c["prompt_max"], c["batch"])


def _prepare_reorder(c, g):
    batch, beams, page = c["batch"], c["beams"], c["page"]
    lens = torch.tensor([x + c["grown"] for x in _prompts(c)], device="cuda")[:, None].expand(batch, beams)
    prompt_blocks = torch.tensor(_prompts(c), device="cuda") // page
    n_blocks = (lens + page - 1) // page
    max_blocks = int(n_blocks.max()) + 1
    # The page of beam k in column i is its set's in the prompt; behind it beams share the more the older the page is.
    col = torch.arange(max_blocks, device="cuda")
    age = (n_blocks[:, :, None] - 1 - col).clamp(0, 6)
    k = torch.arange(beams, device="cuda")[None, :, None]
    owner = torch.where(col < prompt_blocks[:, None, None], 0, (k >> age) << age)
    held = col < n_blocks[:, :, None]
    fresh = (held & (owner == k)).flatten()
    order = torch.cumsum(fresh, 0) - 1
    used = int(fresh.sum())
    spare = batch * beams + 5
    n_pages = used + spare
    ids = torch.randperm(n_pages, generator=g, device="cuda")
    own_page = ids[order.clamp(min=0)].view(batch, beams, max_blocks)
    tables = torch.where(held, own_page.gather(1, owner), 0)
    # `kept` beams of every set go on, each at least once; which ones, and in what order, is the seed's
    chosen = torch.rand((batch, beams), generator=g, device="cuda").argsort(1)[:, :c["kept"]]
    more = chosen.gather(1, torch.randint(0, c["kept"], (batch, beams - c["kept"]), generator=g, device="cuda"))
    parents = torch.cat([chosen, more], 1)
    parents = parents.gather(1, torch.rand((batch, beams), generator=g, device="cuda").argsort(1))
    # the queue: entries taken so far (as many as there are pages in use), then the free ones
    queue = torch.cat([torch.full((used,), -1, device="cuda"), ids[used:]]).to(torch.int32)
    # one page behind the pool takes the plain form's writes where nothing is copied
    shape = _pool_shape(c, n_pages + 1)
    store = torch.empty((2, c["layers"], *shape), dtype=torch.uint8 if c["cache"] == "e4m3" else DTYPES[c["cache"]],
                        device="cuda")
    if c["cache"] == "e4m3":
        store = store.random_(0, 0x7f, generator=g).view(DTYPES["e4m3"])
    else:
        store.view(torch.int16).random_(0, 0x3c00, generator=g)      # any finite values: they are copied, not computed
    return {"case": c, "parents": parents.to(torch.int32).contiguous(), "lens": lens.flatten().contiguous(),
            "block_tables": tables.view(batch * beams, max_blocks).to(torch.int32).contiguous(), "free_pages": queue,
            "free_head": torch.tensor([used], device="cuda"), "n_pages": n_pages, "store": store,
            "k_cache": store[0][:, :n_pages], "v_cache": store[1][:, :n_pages],
            "tables_out": torch.zeros((batch * beams, max_blocks), dtype=torch.int32, device="cuda"),
            "lens_out": torch.zeros(batch * beams, dtype=torch.int64, device="cuda"),
            "head_out": torch.zeros(1, dtype=torch.int64, device="cuda")}


# ------------------------------------------------------------------------------------- plain forms
def _rows(pool, order, table):
    """The rows of every table's pages [batch, h_kv, blocks * page, d] in 32 bits."""
    kind = pool.dtype
    x = (pool.view(torch.uint8) if pool.element_size() == 1 else pool)[table].view(kind)
    x = x.permute(0, 2, 1, 3, 4) if order == "head" else x.permute(0, 3, 1, 2, 4)
    return x.float().reshape(x.shape[0], x.shape[1], -1, x.shape[-1])


def _softmax_rows(s, q, pos, real):
    """Attention of q [batch, n, h_q, d] at row numbers pos [batch, n] (real: there is such a token) over the requests'
    rows, in 32 bits: o [batch, n, h_q, d] and lse [batch, n, h_q]."""
    c = s["case"]
    batch, n, h_kv, d = q.shape[0], q.shape[1], c["h_kv"], c["d"]
    group = c["h_q"] // h_kv
    table = s["block_tables"].long()
    q = q.float().view(batch, n, h_kv, group, d).permute(0, 2, 3, 1, 4).reshape(batch, h_kv, group * n, d)
    z = (q @ _rows(s["k_cache"], c["order"], table).transpose(-1, -2)).view(batch, h_kv, group, n, -1)
    z /= math.sqrt(d)
    if s["k_scale"] is not None:
        z *= s["k_scale"][:, None, None, None]
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    t = torch.arange(z.shape[-1], device="cuda")
    far = t - pos[:, :, None]                                           # 0 at the token's own row
    if s["slopes"] is not None:
        z = z + s["slopes"].view(h_kv, group, 1, 1) * far[:, None, None]
    seen = (far <= 0) & real[:, :, None]
    if c["window"]:
        seen = seen & (far > -c["window"])
    z = torch.where(seen[:, None, None], z, -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - torch.where(m == -math.inf, 0.0, m))              # (0 where nothing is seen)
    total = p.sum(-1, keepdim=True)
    v = _rows(s["v_cache"], c["order"], table)
    o = (p.view(batch, h_kv, group * n, -1) @ v).view(batch, h_kv, group, n, d) / torch.where(total == 0, 1.0, total)
    if s["v_scale"] is not None:
        o = o * s["v_scale"][:, None, None, None]
    lse = (m + torch.log(total))[..., 0]
    return (o.permute(0, 3, 1, 2, 4).reshape(batch, n, c["h_q"], d), lse.permute(0, 3, 1, 2).reshape(batch, n, c["h_q"]))


def _chunk_plain(s):
    c = s["case"]
    first, n_new = s["indptr"][:-1], s["indptr"].diff()
    i = torch.arange(s["new_max"], device="cuda")
    real = i < n_new[:, None]
    tokens = s["q"].shape[0]
    token = torch.where(real, first[:, None] + i, tokens)               # [batch, n]; one more row takes the others' writes
    q = s["q"][token.clamp(max=tokens - 1)]
    o, lse = _softmax_rows(s, q, (s["lens"] - n_new)[:, None] + i, real)
    o_out = torch.cat([s["o"], s["o"].new_zeros((1, c["h_q"], c["d"]))])
    lse_out = torch.cat([s["lse"], s["lse"].new_zeros((1, c["h_q"]))])
    o_out[token] = o.to(o_out.dtype)
    lse_out[token] = lse
    return {"o": o_out[:tokens], "lse": lse_out[:tokens]}


def _prefix_plain(s):
    pos = (s["lens"] - 1)[:, None]
    o, lse = _softmax_rows(s, s["q"][:, None], pos, pos >= 0)
    return {"o": o[:, 0].to(s["o"].dtype), "lse": lse[:, 0]}


def _select_plain(s):
    c = s["case"]
    batch, beams, vocab = c["batch"], c["beams"], c["vocab"]
    # in 64 bits: scores of different beams that lie next to each other decide the order
    x = s["logits"].double().view(batch, beams, vocab)
    top = x.amax(-1, keepdim=True)
    lse = top + torch.log(torch.exp(x - top).sum(-1, keepdim=True))
    score = s["scores"].double()[..., None] + (x - lse)
    if s["ended"] is not None:
        stays = torch.where(torch.arange(vocab, device="cuda") == s["pad_token"], s["scores"].double()[..., None], -math.inf)
        score = torch.where(s["ended"].bool()[..., None], stays, score)
    score = torch.where(torch.isnan(score), -math.inf, score).view(batch, beams * vocab)
    best, at = torch.sort(score, dim=-1, descending=True, stable=True)
    best, at = best[:, :c["n_out"]], at[:, :c["n_out"]]
    return {"scores": best.float(), "parents": (at // vocab).int(), "tokens": (at % vocab).int(), "lse": lse[..., 0].float()}


def _reorder_plain(s):
    c = s["case"]
    batch, beams, page = c["batch"], c["beams"], c["page"]
    parents = s["parents"].long()
    table = s["block_tables"].long().view(batch, beams, -1)
    lens = s["lens"].view(batch, beams)
    n_blocks = (lens + page - 1) // page
    col = torch.arange(table.shape[-1], device="cuda")
    held = col < n_blocks[:, :, None]
    k = torch.arange(beams, device="cuda")
    goes_on = (parents[:, None, :] == k[:, None]).any(-1)               # beam k has a child
    same = (table[:, :, None] == table[:, None]) & held[:, :, None] & held[:, None]       # [batch, k, other, column]
    kept = (same & goes_on[:, None, :, None]).any(2)
    named_before = (same & (k < k[:, None])[None, :, :, None]).any(2)
    dies = (held & ~kept & ~named_before).permute(0, 2, 1).flatten()    # set, column, beam
    n_freed = dies.sum()
    head, n = s["free_head"], s["free_pages"].numel()
    place = torch.where(dies, head - n_freed + torch.cumsum(dies, 0) - 1, n)
    queue = torch.cat([s["free_pages"], s["free_pages"].new_zeros(1)])
    queue[place] = table.permute(0, 2, 1).flatten().int()
    queue = queue[:n]
    # the children: the first of a beam goes on in its pages, the others get a copy of its last page if that is not full
    len_out = lens.gather(1, parents)
    rest = len_out % page
    twin = ((parents[:, :, None] == parents[:, None]) & (k < k[:, None])).any(2)
    copied = (twin & (rest > 0)).flatten()
    last = n_blocks.gather(1, parents) - 1
    to = queue[torch.where(copied, head - n_freed + torch.cumsum(copied, 0) - 1, 0)].long()
    out = table.gather(1, parents[:, :, None].expand(-1, -1, table.shape[-1]))
    source = out.gather(2, last.clamp(min=0)[:, :, None]).flatten()
    out = torch.where((col == last[:, :, None]) & copied.view(batch, beams, 1), to.view(batch, beams, 1), out)
    out = torch.where(held.gather(1, parents[:, :, None].expand_as(held)), out, s["tables_out"].view_as(out))
    dump = torch.where(copied, to, s["n_pages"])
    rows = torch.arange(page, device="cuda") < rest.view(-1, 1)
    rows = rows[:, None, :, None] if c["order"] == "head" else rows[:, :, None, None]
    store = s["store"].view(torch.uint8) if c["cache"] == "e4m3" else s["store"]
    store[:, :, dump] = torch.where(rows, store[:, :, source], store[:, :, dump])
    return {"block_tables": out.view(batch * beams, -1).int(), "lens": len_out.flatten(), "free_pages": queue,
            "free_head": head - n_freed + copied.sum(), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# --------------------------------------------------------------------------------- the library's own
def _workspace(K, n):
    ws = torch.zeros(n + K.WS_ALIGN, dtype=torch.uint8, device="cuda")
    off = (-ws.data_ptr()) % K.WS_ALIGN
    return ws[off:off + n]


def _plan(s):
    """What a serving program keeps next to its buffers: descriptors and a workspace."""
    from attention_kv_cache_gb300 import kvsel as K
    c = s["case"]
    kinds = {"bf16": K.DTYPE_BF16, "f16": K.DTYPE_F16, "f32": K.DTYPE_F32, "e4m3": K.DTYPE_E4M3}
    if c["op"] == "select":
        desc = K.make_beam_select_desc(batch=c["batch"], beams=c["beams"], n_out=c["n_out"], vocab=c["vocab"],
                                       dtype=kinds[c["dtype"]], row_stride=s["logits"].stride(0), pad_token=s["pad_token"])
        return {"K": K, "desc": desc, "ws": _workspace(K, K.kvsel_beam_select_workspace_size(desc))}
    dtype = c["cache"] if c["op"] == "reorder" else c["dtype"]
    cache = K.make_cache_desc(h_q=c.get("h_q", c["h_kv"]), h_kv=c["h_kv"], head_dim=c["d"], page_size=c["page"],
                              n_pages=s["n_pages"], dtype=kinds["bf16" if dtype == "e4m3" else dtype],
                              cache_dtype=kinds[c["cache"]], order=K.ORDER_HEAD if c["order"] == "head" else K.ORDER_ROW)
    max_blocks = s["block_tables"].shape[1]
    if c["op"] == "reorder":
        desc = K.make_beam_reorder_desc(batch=c["batch"], beams=c["beams"], max_blocks=max_blocks, n_layers=c["layers"],
                                        layer_stride=s["k_cache"].stride(0))
        return {"K": K, "cache": cache, "desc": desc, "ws": _workspace(K, K.kvsel_beam_reorder_workspace_size(desc))}
    if c["op"] == "chunk":
        desc = K.make_chunk_attend_desc(batch=c["batch"], max_blocks=max_blocks, max_tokens=s["q"].shape[0],
                                        q_stride=s["q"].stride(0), softcap=c["softcap"], window=c["window"])
        return {"K": K, "cache": cache, "desc": desc,
                "ws": _workspace(K, K.kvsel_chunk_attend_workspace_size(cache, desc))}
    desc = K.make_paged_attend_desc(batch=s["lens"].numel(), max_blocks=max_blocks, softcap=c["softcap"],
                                    window=c["window"])
    return {"K": K, "cache": cache, "desc": desc,
            "ws": _workspace(K, K.kvsel_prefix_attend_workspace_size(cache, desc, c["groups"]))}


def _own(s):
    if "plan" not in s:
        s["plan"] = _plan(s)
    p, op = s["plan"], s["case"]["op"]
    K = p["K"]
    if op == "chunk":
        K.kvsel_chunk_attend(p["cache"], p["desc"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["lens"],
                             s["indptr"], s["slopes"], s["k_scale"], s["v_scale"], s["o"], s["lse"], p["ws"])
        return {"o": s["o"], "lse": s["lse"]}
    if op == "prefix":
        K.kvsel_prefix_attend(p["cache"], p["desc"], s["q"], s["k_cache"], s["v_cache"], s["block_tables"], s["lens"],
                              s["group_indptr"], s["shared_lens"], s["slopes"], s["k_scale"], s["v_scale"], s["o"],
                              s["lse"], p["ws"])
        return {"o": s["o"], "lse": s["lse"]}
    if op == "select":
        K.kvsel_beam_select(p["desc"], s["logits"], s["scores"], s["ended"], s["scores_out"], s["parents"], s["tokens"],
                            s["lse"], p["ws"])
        return {"scores": s["scores_out"], "parents": s["parents"], "tokens": s["tokens"], "lse": s["lse"]}
    K.kvsel_beam_reorder(p["cache"], p["desc"], s["parents"], s["lens"], s["block_tables"], s["free_pages"],
                         s["free_head"], s["tables_out"], s["lens_out"], s["head_out"], s["k_cache"], s["v_cache"], p["ws"])
    return {"block_tables": s["tables_out"], "lens": s["lens_out"], "free_pages": s["free_pages"],
            "free_head": s["head_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    if own:
        return _own(state)
    return {"chunk": _chunk_plain, "prefix": _prefix_plain, "select": _select_plain,
            "reorder": _reorder_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------- work
def _seen(n, window):
    return min(n, window) if window else n


def work(case):
    c = case
    if c["op"] == "chunk":
        held, new = _requests(c)
        kv = 2 * c["h_kv"] * c["d"] * BYTES[c["cache"]]
        rows = sum(min(h + n, _seen(h + 1, c["window"]) + n - 1) if n else 0 for h, n in zip(held, new))
        pairs = sum(_seen(h + i + 1, c["window"]) for h, n in zip(held, new) for i in range(n))
        io = sum(new) * c["h_q"] * (2 * c["d"] * BYTES[c["dtype"]] + 4)
        return {"bytes": rows * kv + io + rows / c["page"] * 4, "flops": pairs * c["h_q"] * 4 * c["d"]}
    if c["op"] == "prefix":
        shared, own_rows = _sharers(c)
        kv = 2 * c["h_kv"] * c["d"] * BYTES[c["cache"]]
        rows = pairs = 0
        for s, xs in zip(shared, own_rows):
            # of the shared rows what the shortest member's window reaches
            rows += max(0, s - max(0, s + min(xs) - c["window"])) if c["window"] else s
            rows += sum(_seen(x, c["window"]) for x in xs)
            pairs += sum(_seen(s + x, c["window"]) for x in xs)
        io = c["groups"] * c["each"] * c["h_q"] * (2 * c["d"] * BYTES[c["dtype"]] + 4)
        return {"bytes": rows * kv + io + rows / c["page"] * 4, "flops": pairs * c["h_q"] * 4 * c["d"]}
    if c["op"] == "select":
        values = c["batch"] * c["beams"] * c["vocab"]
        return {"bytes": values * BYTES[c["dtype"]] + c["batch"] * (c["beams"] * 9 + c["n_out"] * 12), "flops": 3 * values}
    copies = c["beams"] - c["kept"]
    lens = [x + c["grown"] for x in _prompts(c)]
    row = c["layers"] * 2 * c["h_kv"] * c["d"] * BYTES[c["cache"]]
    moved = sum(copies * (n % c["page"]) * row * 2 for n in lens)                # read and written
    tables = sum(c["beams"] * (-(-n // c["page"]) * 8 + 20) for n in lens)
    return {"bytes": moved + tables, "flops": 0}


# --------------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"chunk": _chunk_exact, "prefix": _prefix_exact, "select": _select_exact, "reorder": _reorder_exact}[case["op"]](s)


def _attended(s, q, b, first):
    """q [n, h_q, d] as request b's rows from `first` on, head by head in 64 bits: o [n, h_q, d], lse [n, h_q]."""
    c = s["case"]
    group, page, n = c["h_q"] // c["h_kv"], c["page"], q.shape[0]
    o = torch.zeros((n, c["h_q"], c["d"]), dtype=torch.float64, device="cuda")
    lse = torch.full((n, c["h_q"]), -math.inf, dtype=torch.float64, device="cuda")
    low = max(0, first + 1 - c["window"]) if c["window"] else 0
    t = torch.arange(low, first + n, device="cuda")
    if n == 0 or t.numel() == 0:
        return o, lse
    ids = s["block_tables"][b, t // page].long()
    behind = (first + torch.arange(n, device="cuda"))[:, None] - t                # rows between a row and the token's own
    hidden = behind < 0
    if c["window"]:
        hidden |= behind >= c["window"]
    for h in range(c["h_q"]):
        g = h // group
        k, v = (x.view(torch.uint8)[ids, g, t % page] if c["order"] == "head" else x.view(torch.uint8)[ids, t % page, g]
                for x in (s["k_cache"], s["v_cache"]))
        k, v = (x.contiguous().view(s["k_cache"].dtype).double() for x in (k, v))
        z = q[:, h].double() @ k.T * c["d"] ** -0.5
        if s["k_scale"] is not None:
            z = z * s["k_scale"][g].double()
        if c["softcap"]:
            z = torch.tanh(z / c["softcap"]) * c["softcap"]
        if s["slopes"] is not None:
            z = z - s["slopes"][h].double() * behind.double()
        z.masked_fill_(hidden, -math.inf)
        lse[:, h] = torch.logsumexp(z, -1)
        o[:, h] = torch.softmax(z, -1) @ v
        if s["v_scale"] is not None:
            o[:, h] *= s["v_scale"][g].double()
    return o, lse


def _chunk_exact(s):
    o, lse = s["o"].double(), s["lse"].double()
    ends = s["indptr"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        x, y = ends[b], ends[b + 1]
        o[x:y], lse[x:y] = _attended(s, s["q"][x:y], b, n - (y - x))
    return {"o": o, "lse": lse}


def _prefix_exact(s):
    o, lse = s["o"].double(), s["lse"].double()
    for b, n in enumerate(s["lens"].tolist()):
        x, y = _attended(s, s["q"][b:b + 1] if n else s["q"][:0], b, n - 1)
        o[b] = x[0] if n else 0.0
        lse[b] = y[0] if n else -math.inf
    return {"o": o, "lse": lse}


def _select_exact(s):
    """Set by set: each beam's n best tokens, then the best of all of them, with Python's own sort."""
    c = s["case"]
    if c["batch"] * c["beams"] > 2048:
        return None
    scores, ended = s["scores"].double().tolist(), None if s["ended"] is None else s["ended"].tolist()
    logs = torch.logsumexp(s["logits"].double(), -1).view(c["batch"], c["beams"])
    out = {"scores": [], "parents": [], "tokens": []}
    for b in range(c["batch"]):
        found = []
        for k in range(c["beams"]):
            x = s["logits"][b * c["beams"] + k].double()
            if ended is not None and ended[b][k]:
                x = torch.full_like(x, -math.inf)
                x[s["pad_token"]] = logs[b, k] if math.isfinite(logs[b, k]) else 0.0
            # the n best of the row, the earlier token first among equals: of those at or above the n-th value
            n = min(c["n_out"], c["vocab"])
            edge = torch.topk(x, n).values[-1]
            over = (x > edge).nonzero()[:, 0].tolist()
            at = sorted(over + (x == edge).nonzero()[:n - len(over), 0].tolist())
            for v, y in zip(at, (x - logs[b, k])[at].tolist()):
                if ended is not None and ended[b][k]:
                    y = 0.0 if v == s["pad_token"] else -math.inf
                z = scores[b][k] + y
                found.append((z if z == z else -math.inf, k, v))
        found.sort(key=lambda f: (-f[0], f[1], f[2]))
        for name, i in (("scores", 0), ("parents", 1), ("tokens", 2)):
            out[name].append([f[i] for f in found[:c["n_out"]]])
    return {"scores": torch.tensor(out["scores"], dtype=torch.float64),
            "parents": torch.tensor(out["parents"], dtype=torch.int32),
            "tokens": torch.tensor(out["tokens"], dtype=torch.int32), "lse": logs}


def _reorder_exact(s):
    """Set by set with lists, as a host scheduler keeps its pages: those that no beam names any more are freed."""
    c = s["case"]
    page, beams = c["page"], c["beams"]
    parents, lens = s["parents"].tolist(), s["lens"].tolist()
    tables, out = s["block_tables"].cpu(), s["tables_out"].cpu().clone()
    queue, head = s["free_pages"].cpu().clone(), int(s["free_head"])
    len_out, freed, twins = [], [], []
    for b in range(c["batch"]):
        rows = [tables[b * beams + k, :-(-lens[b * beams + k] // page)].tolist() for k in range(beams)]
        living = {x for p in set(parents[b]) for x in rows[p]}
        for i in range(max(len(r) for r in rows)):
            for r in rows:
                if i < len(r) and r[i] not in living:
                    living.add(r[i])                                     # (freed once)
                    freed.append(r[i])
        taken = set()
        for j, p in enumerate(parents[b]):
            n = lens[b * beams + p]
            len_out.append(n)
            out[b * beams + j, :len(rows[p])] = torch.tensor(rows[p], dtype=torch.int32)
            if p in taken and n % page:
                twins.append((b * beams + j, rows[p][-1], n % page))
            taken.add(p)
    queue[head - len(freed):head] = torch.tensor(freed, dtype=torch.int32)
    head -= len(freed)
    k_cache, v_cache = s["k_cache"].clone(), s["v_cache"].clone()
    for i, (row, source, n) in enumerate(twins):
        to = int(queue[head + i])
        out[row, -(-len_out[row] // page) - 1] = to
        for x in (k_cache, v_cache):
            y = x.view(torch.uint8)
            y = y if c["order"] == "row" else y.transpose(2, 3)          # [layer, page, row, head, bytes]
            y[:, to, :n] = y[:, source, :n]
    return {"block_tables": out, "lens": torch.tensor(len_out), "free_pages": queue,
            "free_head": torch.tensor([head + len(twins)]), "k_cache": k_cache, "v_cache": v_cache}
