"""Long contexts over the paged key-value cache, case by case: attention for
sequences that share a prefix, sparse attention over pages that a cheap score
selects, attention that adds up the weight of every cached token, and the
eviction of the tokens with the least of it.

Every case is a dict of plain values; ``prepare`` makes its inputs on the
GPU, ``run`` is one pass -- in plain 32-bit torch operations, or with the
framework's kernels when ``own`` is true -- and ``exact`` the same results in
64 bits from the definitions.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _cache_case(name, op, seqs, length, heads, group, dim, page, order, dtype,
                store, **more):
    return dict({"name": name, "op": op, "seqs": seqs, "length": length,
                 "heads": heads, "group": group, "dim": dim, "page": page,
                 "order": order, "dtype": dtype, "store": store}, **more)


def _shared(name, seqs, groups, shared, *rest):
    return _cache_case(name, "shared", seqs, *rest, groups=groups,
                       shared=shared)


def _sparse(name, seqs, length, heads, group, dim, page, order, dtype, store,
            keep):
    return _cache_case(name, "sparse", seqs, length, heads, group, dim, page,
                       order, dtype, store, keep=keep)


def _evict(name, seqs, length, heads, dim, page, order, dtype, store, keep,
           recent):
    return _cache_case(name, "evict", seqs, length, heads, 1, dim, page,
                       order, dtype, store, keep=keep, recent=recent)


def listed():
    return [
        # two users of one short instruction, a few tokens in: latency counts
        _shared("shared_pair", 2, 1, 600, 40, 8, 4, 128, 16, "nhd", "bf16",
                "same"),
        # a serving batch behind one long document
        _shared("shared_batch", 64, 1, 16384, 1024, 8, 4, 128, 16, "nhd",
                "bf16", "same"),
        # the largest: three documents, 128 sequences, an 8-bit cache
        _shared("shared_e4m3", 128, 3, 32768, 512, 8, 8, 128, 64, "hnd",
                "bf16", "e4m3"),
        # uneven groups, odd heads, rows of 80, pages of 24
        _shared("shared_odd_f16", 21, 4, 5003, 700, 5, 7, 80, 24, "nhd",
                "f16", "same"),
        # the bounds of a prefill batch's pages
        _cache_case("bound_prefill", "bound", 8, 8192, 8, 1, 128, 16, "nhd",
                    "bf16", "same"),
        # one user far into a long context: 4096 of 131072 tokens are read
        _sparse("sparse_one", 1, 131072, 8, 4, 128, 16, "nhd", "bf16", "same",
                256),
        # a batch of long contexts, 2048 tokens each
        _sparse("sparse_batch", 32, 32768, 8, 4, 128, 32, "nhd", "bf16",
                "same", 64),
        # whole numbers, an odd group, pages of 40
        _sparse("sparse_int8", 13, 20011, 4, 5, 64, 40, "nhd", "f16", "int8",
                50),
        # a decoding step that also adds up each cached token's weight
        _cache_case("weigh_batch", "weigh", 32, 8192, 8, 4, 128, 16, "nhd",
                    "bf16", "same"),
        # the same over whole numbers, an odd group
        _cache_case("weigh_int8", "weigh", 5, 30011, 4, 5, 64, 40, "nhd",
                    "f16", "int8"),
        # a batch's caches brought back to half, the last tokens kept
        _evict("evict_batch", 64, 4096, 8, 128, 16, "nhd", "bf16", "same",
               2048, 256),
        # two very long ones brought back to a quarter
        _evict("evict_long_int8", 2, 100003, 4, 64, 40, "hnd", "f16", "int8",
               25000, 1000),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["shared", "shared", "bound", "sparse", "sparse", "weigh",
                     "evict"])
    heads = rng.choice([1, 2, 4, 5, 8, 16])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    dim = rng.choice([64, 80, 112, 128, 128, 256])
    rest = (heads, group, dim, rng.choice([8, 16, 20, 32, 40, 64, 128]),
            rng.choice(["nhd", "hnd"]), rng.choice(["bf16", "f16"]),
            rng.choice(["same", "e4m3", "int8"]))
    page = rest[3]
    # no more cached elements, and no more products, than the largest listed
    room = 16 * 8192 * 8 * 128 // (heads * dim)
    if op == "shared":
        seqs = _log(rng, 1, 160)
        groups = min(seqs, rng.choice([1, 1, 2, 3, 5, 8]))
        most = 128 * 8 * 8 * 128 * 32768 // (seqs * group * heads * dim)
        shared = _log(rng, 1, max(1, min(40000, room // groups, most)))
        length = _log(rng, 1, max(1, min(2048, room // seqs)))
        c = _shared("", seqs, groups, shared, length, *rest)
    else:
        seqs = _log(rng, 1, 64)
        length = _log(rng, 1, max(1, min(131072, room // seqs)))
        if op == "bound":
            c = _cache_case("", op, seqs, length, heads, 1, *rest[2:])
        elif op == "weigh":
            c = _cache_case("", op, seqs, length, *rest)
        elif op == "sparse":
            keep = _log(rng, 2, max(2, min(512, length // page)))
            c = _sparse("", seqs, length, *rest, keep)
        else:
            keep = _log(rng, 1, max(1, length))
            c = _evict("", seqs, length, heads, *rest[2:], keep,
                       rng.randint(0, keep // 2))
    del c["name"]
    return c


def _lens(case, top=None, n=None):
    """The lengths of a case's sequences: the longest as given, the others
    spread below it; in a larger batch one row is empty and one holds a
    single token.  The case alone decides them."""
    n, top = n or case["seqs"], top or case["length"]
    r = np.random.RandomState(n * 7919 + top * 31 + case["heads"])
    lens = r.randint(max(1, top // 2), top + 1, n)
    lens[0] = top
    if n >= 8 and top > 1:
        lens[n // 2] = 0
        lens[n // 3] = 1
    return [int(v) for v in lens]


def _group_starts(case):
    """Where each group's sequences start: uneven runs of at least one."""
    n, g = case["seqs"], case["groups"]
    r = np.random.RandomState(n * 131 + g)
    cuts = np.sort(r.permutation(n - 1)[:g - 1] + 1) if g > 1 else []
    return [0] + [int(c) for c in cuts] + [n]


def _row_bytes(case):
    """Bytes of a held row: its elements and its scale."""
    return case["dim"] * 2 if case["store"] == "same" else case["dim"] + 4


def work(case):
    heads, dim, page = case["heads"], case["dim"], case["page"]
    row = _row_bytes(case)
    lens = _lens(case)
    total = sum(lens)
    if case["op"] == "bound":
        pages = sum(-(-n // page) for n in lens)
        return {"bytes": heads * (total * row + pages * (2 * dim + 4)) +
                8 * pages, "flops": 2 * total * heads * dim}
    if case["op"] == "evict":
        kept = sum(min(n, case["keep"]) for n in lens)
        return {"bytes": heads * (4 * total + kept * 2 * (2 * row + 4)),
                "flops": total * heads}
    heads_q = heads * case["group"]
    ends = case["seqs"] * heads_q * (dim * 4 + 4)
    if case["op"] == "weigh":
        return {"bytes": heads * total * (2 * row + 8) + ends,
                "flops": 4 * total * heads_q * dim}
    if case["op"] == "shared":
        shared = _lens(case, case["shared"], case["groups"])
        starts = _group_starts(case)
        seen = sum(n * (starts[g + 1] - starts[g])
                   for g, n in enumerate(shared))
        return {"bytes": heads * (total + sum(shared)) * 2 * row + ends,
                "flops": 4 * (total + seen) * heads_q * dim}
    pages = [-(-n // page) for n in lens]
    kept = [min(m, case["keep"]) for m in pages]
    tokens = sum(k * page - (m * page - n)
                 for k, m, n in zip(kept, pages, lens))
    return {"bytes": heads * (sum(pages) * (2 * dim + 4) +
                              tokens * 2 * row + sum(kept) * 4) +
            4 * sum(pages) + ends,
            "flops": 2 * heads_q * dim * (2 * sum(pages) + 2 * tokens)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _tables(case, gen, *lengths):
    """A page table [sequences, most] for each list of lengths, their pages
    scattered over one pool a little larger than they need; and its size."""
    p = case["page"]
    used = sum(-(-n // p) for lens in lengths for n in lens)
    pool = used + max(1, used // 16)
    ids = torch.randperm(pool, generator=gen, device="cuda")[:used].cpu()
    tables, at = [], 0
    for lens in lengths:
        most = max(1, max(-(-n // p) for n in lens))
        table = torch.full((len(lens), most), -1, dtype=torch.int32)
        for b, n in enumerate(lens):
            m = -(-n // p)
            table[b, :m] = ids[at:at + m].int()
            at += m
        tables.append(table.cuda())
    return tables, pool


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _page_shape(case, pool):
    p, h, d = case["page"], case["heads"], case["dim"]
    return (pool, p, h, d) if case["order"] == "nhd" else (pool, h, p, d)


def _by_token(case, pages):
    """Pages as [page, token, head, ...] whatever their order."""
    return pages if case["order"] == "nhd" else pages.transpose(1, 2)


def _by_head(case, pages):
    """Pages as [page, head, token, ...] whatever their order."""
    return pages.transpose(1, 2) if case["order"] == "nhd" else pages


def _store_dtype(case):
    return {"same": DTYPES[case["dtype"]], "e4m3": torch.float8_e4m3fn,
            "int8": torch.int8}[case["store"]]


def _pow2(e):
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x, store):
    """(codes, scale) of 32-bit rows: e4m3 codes under the smallest power of
    two that brings the row's largest magnitude to 448 or less, or whole
    numbers under a 127th of that magnitude.  A row of zeros has scale 1."""
    top = x.abs().amax(-1)
    if store == "e4m3":
        f, n = torch.frexp(top)
        e = torch.where(f <= 0.875, n - 9, n - 8).clamp(min=-126)
        e = torch.where(top == 0, torch.zeros_like(e), e)
        return (x * _pow2(-e)[..., None]).to(torch.float8_e4m3fn), _pow2(e)
    scale = torch.where(top == 0, torch.ones_like(top),
                        (top / 127.0).clamp(min=2.0 ** -126))
    return (x / scale[..., None]).round().clamp(-127, 127).to(torch.int8), \
        scale


def _filled(case, pool, gen, drift=0.0):
    """A cache's pages and scales with the rows of random keys (or values);
    with ``drift`` a page's rows have something in common."""
    rows = torch.empty(_page_shape(case, pool), dtype=_store_dtype(case),
                       device="cuda")
    scales = torch.ones((pool, case["heads"], case["page"]), device="cuda") \
        if case["store"] != "same" else None
    step = max(1, (1 << 28) // (rows[0].numel() * 4))
    for at in range(0, pool, step):
        part = rows[at:at + step]
        x = _randn(part.shape, torch.float32, gen)
        # rows of different magnitude, as a model's tokens have
        x *= torch.exp(_randn(part.shape[:-1] + (1,), torch.float32, gen)
                       * 0.3)
        if drift:
            x += drift * _common(case, part.shape, gen)
        if scales is None:
            part.copy_(x)
        else:
            x = x.to(DTYPES[case["dtype"]]).float()
            codes, scale = _quantise(x, case["store"])
            part.copy_(codes) if case["store"] == "int8" else \
                part.view(torch.uint8).copy_(codes.view(torch.uint8))
            scales[at:at + step] = scale.transpose(1, 2) \
                if case["order"] == "nhd" else scale
    return rows, scales


def _common(case, shape, gen):
    """One random row a page and head."""
    shape = list(shape)
    shape[1 if case["order"] == "nhd" else 2] = 1
    return _randn(shape, torch.float32, gen)


def _queries(case, s, gen):
    b, heads, d = case["seqs"], case["heads"] * case["group"], case["dim"]
    s["q"] = _randn((b, heads, d), DTYPES[case["dtype"]], gen)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((b, heads), device="cuda")
    s["scale"] = d ** -0.5


def _kv_cache(case, s):
    """The framework's plan and cache over the state's buffers."""
    import layout_driven_movement_gb300 as lm
    p, h, d = case["page"], case["heads"], case["dim"]
    page = lm.Layout.make([p, h, d], [h * d, d, 1] if case["order"] == "nhd"
                          else [d, p * d, 1], [1, 1, 1])
    store = None if case["store"] == "same" else case["store"]
    plan = lm.KVPlan(page, DTYPES[case["dtype"]], store)
    return lm.KVCache(plan, s["k_pages"], s["v_pages"], s["k_scale"],
                      s["v_scale"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "v_scale": None}
    lens, op = _lens(case), case["op"]
    p, h, d = case["page"], case["heads"], case["dim"]
    s["lens"] = _ints(lens)
    if op == "shared":
        shared, starts = _lens(case, case["shared"], case["groups"]), \
            _group_starts(case)
        (s["page_table"], s["shared_table"]), pool = \
            _tables(case, gen, lens, shared)
        s["shared_lens"], s["starts"] = _ints(shared), _ints(starts)
        # which sequences a group has (for the plain form: padded to the
        # largest), each one's group and place there
        most = max(b - a for a, b in zip(starts, starts[1:]))
        of = np.searchsorted(starts, np.arange(case["seqs"]), "right") - 1
        place = np.arange(case["seqs"]) - np.array(starts)[of]
        members = np.zeros((case["groups"], most), np.int64)
        members[of, place] = np.arange(case["seqs"])
        s["group_of"], s["place"], s["members"] = (
            torch.from_numpy(x).cuda() for x in (of, place, members))
    elif op == "evict":
        # the kept rows go to pages of their own behind the pool
        (s["page_table"],), pool = _tables(case, gen, lens)
        most = -(-case["keep"] // p)
        s["kept_table"] = (pool + torch.arange(
            case["seqs"] * most, dtype=torch.int32, device="cuda")).view(
                case["seqs"], most)
        s["kept_from"], pool = pool, pool + case["seqs"] * most
        s["kept_lens"] = torch.empty_like(s["lens"])
    else:
        (s["page_table"],), pool = _tables(case, gen, lens)
    s["k_pages"], s["k_scale"] = _filled(case, pool, gen,
                                         1.0 if op == "sparse" else 0.0)
    if op == "bound":
        s["v_pages"], s["v_scale"] = torch.empty_like(s["k_pages"]), \
            s["k_scale"] if s["k_scale"] is None else \
            torch.ones_like(s["k_scale"])
    else:
        s["v_pages"], s["v_scale"] = _filled(case, pool, gen)
    if op in ("bound", "sparse"):
        s["bounds"] = torch.zeros((pool, h, 2, d), dtype=torch.int8,
                                  device="cuda")
        s["bound_scale"] = torch.ones((pool, h), device="cuda")
        at = torch.arange(s["page_table"].shape[1], device="cuda") * p
        left = s["lens"][:, None] - at
        s["pages"] = s["page_table"][left > 0].contiguous()
        s["counts"] = left[left > 0].clamp(max=p).int()
    if op == "sparse":
        step = max(1, (1 << 28) // (p * h * d * 4))
        for i in range(0, s["pages"].numel(), step):
            ids = s["pages"][i:i + step].long()
            s["bounds"][ids], s["bound_scale"][ids] = \
                _bounds(case, s, ids, s["counts"][i:i + step])
        b = case["seqs"]
        s["selected"] = torch.empty((b, h, case["keep"]), dtype=torch.int32,
                                    device="cuda")
        s["selected_lens"] = torch.empty((b,), dtype=torch.int32,
                                         device="cuda")
    if op in ("weigh", "evict"):
        # what earlier steps have added up, most of it on few tokens
        s["weights"] = torch.exp(2 * torch.randn(
            (pool, h, p), generator=gen, device="cuda"))
    if op in ("shared", "sparse", "weigh"):
        _queries(case, s, gen)
    if own:
        _own_prepare(case, s)
    return s


def _own_prepare(case, s):
    import layout_driven_movement_gb300 as lm
    s["cache"] = _kv_cache(case, s)
    plan, b, op = s["cache"].plan, case["seqs"], case["op"]
    heads_q = case["heads"] * case["group"]
    width = s["page_table"].shape[1]

    def space(n):
        return torch.zeros(n, dtype=torch.uint8, device="cuda")
    if op == "shared":
        s["workspace"] = space(lm.kv_attend_shared_workspace(
            plan, b, heads_q))
    elif op == "weigh":
        s["workspace"] = space(lm.kv_attend_workspace(
            plan, b, heads_q, max_pages=width))
    elif op == "sparse":
        s["workspace"] = space(lm.kv_attend_workspace(plan, b, heads_q))
        s["select_space"] = space(lm.kv_select_workspace(plan, b, width))
    elif op == "evict":
        s["workspace"] = space(lm.kv_evict_workspace(plan, b, case["keep"]))


# ---------------------------------------------------------------------------
# One pass: the plain forms
# ---------------------------------------------------------------------------

def _rows(case, s, name, table):
    """The rows of the pages of `table`, in 32 bits: [..., page, head, dim]
    for every entry."""
    pages = s[name + "_pages"]
    x = _by_token(case, pages.view(torch.uint8) if case["store"] == "e4m3"
                  else pages)[table]
    if case["store"] == "e4m3":
        x = x.view(torch.float8_e4m3fn)
    x = x.float()
    if s[name + "_scale"] is not None:
        x = x * s[name + "_scale"].transpose(1, 2)[table][..., None]
    return x


def _softmax(q, k, v, seen, scale):
    """(largest score, sum, unnormalised output) of queries [.., head, rows,
    dim] over keys and values [.., token, head, dim], those that are seen
    [.., token]."""
    score = torch.matmul(q, k.transpose(-3, -2).transpose(-2, -1)) * scale
    score = torch.where(seen[..., None, None, :], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    v = torch.where(seen[..., None, None], v, torch.zeros_like(v))
    return top, p.sum(-1, keepdim=True), torch.matmul(
        p, v.transpose(-3, -2)), p


def _finish(s, top, total, out):
    b, heads, d = s["q"].shape
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.reshape(b, heads, d).to(s["q"].dtype),
            "lse": lse.reshape(b, heads)}


def _own_state(s):
    """The attention of each sequence's query over its own pages."""
    c = s["case"]
    q = s["q"].float().view(c["seqs"], c["heads"], c["group"], c["dim"])
    table = s["page_table"].long().clamp(min=0)
    k = _rows(c, s, "k", table).flatten(1, 2)
    v = _rows(c, s, "v", table).flatten(1, 2)
    seen = torch.arange(k.shape[1], device="cuda") < s["lens"][:, None]
    return _softmax(q, k, v, seen, s["scale"])


def _run_shared(s):
    c = s["case"]
    top, total, out, _ = _own_state(s)
    # the shared keys once for all queries of a group
    q = s["q"].float().view(c["seqs"], c["heads"], c["group"], c["dim"])
    q = q[s["members"]].transpose(1, 2)           # [group, head, seq, ..]
    table = s["shared_table"].long().clamp(min=0)
    k = _rows(c, s, "k", table).flatten(1, 2)
    v = _rows(c, s, "v", table).flatten(1, 2)
    seen = torch.arange(k.shape[1], device="cuda") < \
        s["shared_lens"][:, None]
    state = _softmax(q.flatten(2, 3), k, v, seen, s["scale"])[:3]
    at = (s["group_of"], slice(None), s["place"])
    top2, total2, out2 = (
        x.unflatten(2, (q.shape[2], c["group"]))[at] for x in state)
    top1 = torch.where(total > 0, top, -math.inf)
    top2 = torch.where(total2 > 0, top2, -math.inf)
    both = torch.maximum(top1, top2)
    both = torch.where(both == -math.inf, torch.zeros_like(both), both)
    a, b = torch.exp(top1 - both), torch.exp(top2 - both)
    return _finish(s, both, a * total + b * total2, a * out + b * out2)


def _power(top):
    """The smallest power of two's exponent, -126 or more, that brings a
    magnitude to 127 or less; 0 for 0."""
    f, n = torch.frexp(top)
    e = torch.where(f <= 127 / 128, n - 7, n - 6).clamp(min=-126)
    return torch.where(top == 0, torch.zeros_like(e), e)


def _bounds(case, s, pages, counts):
    """The bounds of pages' first tokens: (whole numbers [pages, heads, 2,
    dim], a power of two [pages, heads])."""
    x = _rows(case, s, "k", pages)                # [page, token, head, dim]
    held = torch.arange(case["page"], device="cuda") < counts[:, None]
    held = held[..., None, None]
    low = torch.where(held, x, math.inf).amin(1)
    high = torch.where(held, x, -math.inf).amax(1)
    e = _power(torch.maximum(low.abs(), high.abs()).amax(-1))
    by = _pow2(-e)[..., None]
    return torch.stack([torch.floor(low * by), torch.ceil(high * by)],
                       2).to(torch.int8), _pow2(e)


def _run_bound(s):
    ids = s["pages"].long()
    s["bounds"][ids], s["bound_scale"][ids] = \
        _bounds(s["case"], s, ids, s["counts"])
    return {"bounds": s["bounds"], "bound_scale": s["bound_scale"]}


def _run_sparse(s):
    c = s["case"]
    b, h, g, d, p = (c[x] for x in ("seqs", "heads", "group", "dim", "page"))
    q = s["q"].float().view(b, h, g, d)
    e = _power(q.abs().amax(-1))
    code = (q * _pow2(-e)[..., None]).round()
    table = s["page_table"].long().clamp(min=0)
    bound = s["bounds"][table].float()            # [b, page, h, 2, d]
    low, high = bound.permute(3, 0, 2, 4, 1)      # [b, h, d, page]
    score = torch.matmul(code.clamp(min=0), high) + \
        torch.matmul(code.clamp(max=0), low)      # whole numbers below 2^24
    score = (score * _pow2(e)[..., None]).amax(2) * \
        s["bound_scale"][table].transpose(1, 2)
    lens = s["lens"].long()
    n = (lens + p - 1) // p
    at = torch.arange(table.shape[1], device="cuda")[None, None]
    n3 = n[:, None, None]
    # the first and the last page are always among them
    score = torch.where((at == 0) | (at == n3 - 1), math.inf, score)
    score = torch.where(at < n3, score, -math.inf)
    keep = min(c["keep"], table.shape[1])
    best = score.sort(dim=-1, descending=True, stable=True)[1][..., :keep]
    count = n.clamp(max=c["keep"])
    live = torch.arange(keep, device="cuda") < count[:, None, None]
    best = torch.where(live, best, table.shape[1]).sort(-1)[0]
    pages = torch.where(live, table[:, None].expand(-1, h, -1).gather(
        2, best.clamp(max=table.shape[1] - 1)), -1)
    s["selected"].fill_(-1)
    s["selected"][..., :keep] = pages.int()
    s["selected_lens"].copy_(lens - (n - count) * p)
    # each head's own pages
    head = torch.arange(h, device="cuda")[None, :, None]
    rows = []
    for name in ("k", "v"):
        x = s[name + "_pages"]
        x = _by_head(c, x.view(torch.uint8) if c["store"] == "e4m3" else x)[
            pages.clamp(min=0), head]             # [b, h, page, token, dim]
        x = (x.view(torch.float8_e4m3fn) if c["store"] == "e4m3"
             else x).float()
        if c["store"] != "same":
            x = x * s[name + "_scale"][pages.clamp(min=0), head][..., None]
        rows.append(x.flatten(2, 3).transpose(1, 2))
    seen = torch.arange(rows[0].shape[1], device="cuda") < \
        s["selected_lens"][:, None]
    out = _finish(s, *_softmax(q, *rows, seen, s["scale"])[:3])
    return dict(out, selected=s["selected"],
                selected_lens=s["selected_lens"])


def _run_weigh(s):
    c = s["case"]
    top, total, out, p = _own_state(s)
    share = torch.where(total > 0, p / total, torch.zeros_like(p)).sum(2)
    # to the weights of the tokens' places: [page, token, head]
    place = s["weights"].transpose(1, 2)
    at = torch.arange(share.shape[-1], device="cuda")[None]
    b, j = torch.nonzero(at < s["lens"][:, None], as_tuple=True)
    page, off = s["page_table"].long()[b, j // c["page"]], j % c["page"]
    place[page, off] = place[page, off] + share.transpose(1, 2)[b, j]
    return dict(_finish(s, top, total, out), weights=s["weights"])


def _run_evict(s):
    c = s["case"]
    p, keep, recent = c["page"], c["keep"], c["recent"]
    table, lens = s["page_table"].long().clamp(min=0), s["lens"].long()
    w = s["weights"][table].transpose(1, 2).flatten(2)    # [b, h, token]
    at = torch.arange(w.shape[-1], device="cuda")[None, None]
    n = lens[:, None, None]
    w = torch.where(at >= n - recent, math.inf, w)
    w = torch.where(at < n, w, -math.inf)
    most = min(keep, w.shape[-1])
    best = w.sort(dim=-1, descending=True, stable=True)[1][..., :most]
    count = lens.clamp(max=keep)
    live = torch.arange(most, device="cuda") < count[:, None, None]
    best = torch.where(live, best, w.shape[-1]).sort(-1)[0]
    b, h, i = torch.nonzero(live.expand_as(best), as_tuple=True)
    j = best[b, h, i]
    src, dst = (table[b, j // p], h, j % p), \
        (s["kept_table"].long()[b, i // p], h, i % p)
    out = {}
    for name in ("k_pages", "v_pages"):
        x = _by_head(c, s[name].view(torch.uint8) if c["store"] == "e4m3"
                     else s[name])
        x[dst] = x[src]
        out[name] = s[name][s["kept_from"]:]
    for name in ("k_scale", "v_scale", "weights"):
        if s[name] is not None:
            s[name][dst] = s[name][src]
            out[name] = s[name][s["kept_from"]:]
    s["kept_lens"].copy_(count)
    return dict(out, kept_lens=s["kept_lens"])


# ---------------------------------------------------------------------------
# One pass: the framework's kernels
# ---------------------------------------------------------------------------

def _own_shared(s):
    import layout_driven_movement_gb300 as lm
    lm.kv_attend_shared(s["cache"], s["q"], s["shared_table"],
                        s["shared_lens"], s["starts"], s["page_table"],
                        s["lens"], s["out"], s["workspace"], lse=s["lse"],
                        scale=s["scale"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_bound(s):
    import layout_driven_movement_gb300 as lm
    lm.kv_bound(s["cache"], s["pages"], s["counts"], s["bounds"],
                s["bound_scale"])
    return {"bounds": s["bounds"], "bound_scale": s["bound_scale"]}


def _own_sparse(s):
    import layout_driven_movement_gb300 as lm
    lm.kv_select(s["cache"], s["q"], s["bounds"], s["bound_scale"],
                 s["page_table"], s["lens"], s["selected"],
                 s["selected_lens"], s["select_space"], first=1, last=1)
    lm.kv_attend(s["cache"], s["q"], s["selected"], s["selected_lens"],
                 s["out"], s["workspace"], lse=s["lse"], scale=s["scale"])
    return {"out": s["out"], "lse": s["lse"], "selected": s["selected"],
            "selected_lens": s["selected_lens"]}


def _own_weigh(s):
    import layout_driven_movement_gb300 as lm
    lm.kv_attend(s["cache"], s["q"], s["page_table"], s["lens"], s["out"],
                 s["workspace"], lse=s["lse"], scale=s["scale"],
                 weights=s["weights"])
    return {"out": s["out"], "lse": s["lse"], "weights": s["weights"]}


def _own_evict(s):
    import layout_driven_movement_gb300 as lm
    c = s["case"]
    lm.kv_evict(s["cache"], s["weights"], s["page_table"], s["lens"],
                s["kept_table"], s["kept_lens"], c["keep"], s["workspace"],
                recent=c["recent"])
    out = {name: s[name][s["kept_from"]:] for name in
           ("k_pages", "v_pages", "k_scale", "v_scale", "weights")
           if s[name] is not None}
    return dict(out, kept_lens=s["kept_lens"])


PLAIN = {"shared": _run_shared, "bound": _run_bound, "sparse": _run_sparse,
         "weigh": _run_weigh, "evict": _run_evict}
OWN = {"shared": _own_shared, "bound": _own_bound, "sparse": _own_sparse,
       "weigh": _own_weigh, "evict": _own_evict}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _rows64(case, s, name, ids, n, h=None):
    """The first n rows that a list of pages holds: [n, heads, dim], or one
    head's [n, dim]."""
    ids = ids[:-(-n // case["page"])].long()
    pages = s[name + "_pages"]
    if case["store"] == "e4m3":
        pages = pages.view(torch.uint8)
    pages = pages if case["order"] == "hnd" else pages.permute(0, 2, 1, 3)
    x = pages[ids] if h is None else pages[ids, h]
    if case["store"] == "e4m3":
        x = x.view(torch.float8_e4m3fn)
    x = x.double()
    if case["store"] != "same":
        scale = s[name + "_scale"]
        x = x * (scale[ids] if h is None else scale[ids, h]).double()[..., None]
    if h is not None:
        return x.reshape(-1, case["dim"])[:n]
    return x.permute(0, 2, 1, 3).reshape(-1, case["heads"], case["dim"])[:n]


def _attend64(case, s, keys_of):
    """Outputs and lse a sequence and key head at a time; `keys_of(b, h)`:
    its keys and values."""
    b, heads, d = s["q"].shape
    out = torch.zeros((b, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, heads), -math.inf, dtype=torch.float64,
                     device="cuda")
    for i in range(b):
        for h in range(case["heads"]):
            k, v = keys_of(i, h)
            if len(k) == 0:
                continue
            g = slice(h * case["group"], (h + 1) * case["group"])
            z = s["q"][i, g].double() @ k.T * s["scale"]
            lse[i, g] = torch.logsumexp(z, -1)
            out[i, g] = torch.softmax(z, -1) @ v
    return out, lse


def _exact_shared(case, s):
    lens, shared = _lens(case), _lens(case, case["shared"], case["groups"])
    of = s["group_of"].tolist()
    held = {}

    def of_group(g):
        if g not in held:
            held.clear()                          # (sequences come in order)
            held[g] = [_rows64(case, s, x, s["shared_table"][g], shared[g])
                       for x in "kv"]
        return held[g]

    def keys(b, h):
        own_rows = [_rows64(case, s, x, s["page_table"][b], lens[b], h)
                    for x in "kv"]
        return [torch.cat([x[:, h], y])
                for x, y in zip(of_group(of[b]), own_rows)]
    out, lse = _attend64(case, s, keys)
    return {"out": out, "lse": lse}


def _exact_bound(case, s):
    bounds, scale = s["bounds"].clone(), s["bound_scale"].clone()
    x = s["k_pages"]
    # a row's values are those that a read back in 32 bits gives
    x = x.float() if case["store"] == "same" else x.float() * (
        s["k_scale"].transpose(1, 2) if case["order"] == "nhd"
        else s["k_scale"])[..., None]
    x = x.double() if case["order"] == "nhd" else x.double().transpose(1, 2)
    for count in sorted(set(s["counts"].tolist())):
        ids = s["pages"][s["counts"] == count].long()
        part = x[ids, :count]
        lo, hi = part.min(1)[0], part.max(1)[0]
        most = torch.maximum(-lo, hi).amax(-1)
        by = torch.exp2(torch.ceil(torch.log2(most / 127)))
        by = torch.where(most > 0, by, 1.0)[..., None]
        bounds[ids, :, 0] = torch.floor(lo / by).to(torch.int8)
        bounds[ids, :, 1] = torch.ceil(hi / by).to(torch.int8)
        scale[ids] = by[..., 0].float()
    return {"bounds": bounds, "bound_scale": scale.double()}


def _exact_sparse(case, s):
    h, g, keep, p = (case[x] for x in ("heads", "group", "keep", "page"))
    selected = torch.full((case["seqs"], h, keep), -1, dtype=torch.int32)
    lens = []
    table = s["page_table"].cpu()
    bounds, scale = s["bounds"].cpu().numpy(), s["bound_scale"].cpu().numpy()
    q = s["q"].double().cpu().numpy()
    for b, n in enumerate(_lens(case)):
        pages = table[b, :-(-n // p)].numpy()
        m = len(pages)
        lens.append(n - max(0, m - keep) * p)
        for i in range(h):
            chosen = np.arange(m)
            if m > keep:
                best = np.full(m, -np.inf)
                lo, hi = (bounds[pages, i, j].astype(np.float64)
                          for j in (0, 1))
                for row in q[b, i * g:(i + 1) * g]:
                    top = np.abs(row).max()
                    by = 2.0 ** np.ceil(np.log2(top / 127)) if top else 1.0
                    code = np.rint(row / by)
                    each = np.maximum(lo * code, hi * code).sum(1)
                    best = np.maximum(best, each * by)
                best = best * scale[pages, i]
                best[0] = best[-1] = np.inf
                order = np.lexsort((np.arange(m), -best))
                chosen = np.sort(order[:keep])
            selected[b, i, :len(chosen)] = torch.from_numpy(pages[chosen])

    def keys(b, i):
        return [_rows64(case, s, x, selected[b, i].cuda(), lens[b], i)
                for x in "kv"]
    out, lse = _attend64(case, s, keys)
    return {"out": out, "lse": lse, "selected": selected,
            "selected_lens": torch.tensor(lens, dtype=torch.int32)}


def _exact_weigh(case, s):
    lens, p, g = _lens(case), case["page"], case["group"]
    out, lse = _attend64(case, s, lambda b, h: [
        _rows64(case, s, x, s["page_table"][b], lens[b], h) for x in "kv"])
    weights = s["weights"].double()
    for b, n in enumerate(lens):
        if n == 0:
            continue
        k = _rows64(case, s, "k", s["page_table"][b], n)
        q = s["q"][b].double().view(case["heads"], g, -1)
        z = torch.einsum("nhd,hgd->hgn", k, q) * s["scale"]
        share = torch.exp(z - lse[b].view(-1, g, 1)).sum(1)
        m = -(-n // p)
        wide = torch.zeros((case["heads"], m * p), dtype=torch.float64,
                           device="cuda")
        wide[:, :n] = share
        weights[s["page_table"][b, :m].long()] += \
            wide.view(-1, m, p).transpose(0, 1)
    return {"out": out, "lse": lse, "weights": weights}


def _exact_evict(case, s):
    p, keep, recent = case["page"], case["keep"], case["recent"]
    lens = _lens(case)
    names = [x for x in ("k_pages", "v_pages", "k_scale", "v_scale",
                         "weights") if s[x] is not None]
    bits = {x: s[x].view(torch.uint8) if s[x].dtype == torch.float8_e4m3fn
            else s[x] for x in names}
    full = {x: v[s["kept_from"]:].clone() for x, v in bits.items()}
    by_head = {x: _by_head(case, full[x]) if x[1:] == "_pages" else full[x]
               for x in names}
    for b, n in enumerate(lens):
        w = s["weights"][s["page_table"][b].long().clamp(min=0)]
        w = w.transpose(0, 1).flatten(1)[:, :n].double().cpu().numpy()
        for h in range(case["heads"]):
            old = max(0, n - recent)
            order = np.lexsort((np.arange(old), -w[h, :old]))
            kept = np.concatenate([
                np.sort(order[:max(0, keep - min(n, recent))]),
                np.arange(old, n)]) if n > keep else np.arange(n)
            j = torch.from_numpy(kept).cuda()
            i = torch.arange(len(kept), device="cuda")
            src = s["page_table"][b].long()[j // p]
            dst = s["kept_table"][b].long()[i // p] - s["kept_from"]
            for x in names:
                v = _by_head(case, bits[x]) if x[1:] == "_pages" else bits[x]
                by_head[x][dst, h, i % p] = v[src, h, j % p]
    out = {x: v.view(torch.float8_e4m3fn) if s[x].dtype ==
           torch.float8_e4m3fn else v for x, v in full.items()}
    return dict({x: v.double() if "float" in str(v.dtype) else v
                 for x, v in out.items()},
                kept_lens=torch.tensor([min(n, keep) for n in lens],
                                       dtype=torch.int32))


EXACT = {"shared": _exact_shared, "bound": _exact_bound,
         "sparse": _exact_sparse, "weigh": _exact_weigh,
         "evict": _exact_evict}


def exact(case, seed):
    return EXACT[case["op"]](case, prepare(case, seed))
