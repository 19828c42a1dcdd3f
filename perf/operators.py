"""The paged key-value cache's operators, case by case: rotary positions, the
cache's (quantising) write and its read back, and the attention of one new
token over it.

Every case is a dict of plain values; ``prepare`` makes its inputs on the
GPU, ``run`` is one pass -- in plain 32-bit torch operations, or with the
framework's kernels when ``own`` is true -- and ``exact`` the same results in
64 bits from the definitions.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _rope(name, tokens, heads, dim, rot, dtype, interleaved, backward, gap):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads,
            "dim": dim, "rot": rot, "dtype": dtype,
            "interleaved": interleaved, "backward": backward, "gap": gap}


def _cache(name, seqs, length, heads, dim, page, order, dtype, store, rope,
           readback):
    return {"name": name, "op": "cache", "seqs": seqs, "length": length,
            "heads": heads, "dim": dim, "page": page, "order": order,
            "dtype": dtype, "store": store, "rope": rope,
            "readback": readback}


def _read(name, seqs, length, heads, dim, page, order, dtype, store):
    return {"name": name, "op": "read", "seqs": seqs, "length": length,
            "heads": heads, "dim": dim, "page": page, "order": order,
            "dtype": dtype, "store": store}


def _attend(name, seqs, length, heads, group, dim, page, order, dtype, store,
            window):
    return {"name": name, "op": "attend", "seqs": seqs, "length": length,
            "heads": heads, "group": group, "dim": dim, "page": page,
            "order": order, "dtype": dtype, "store": store, "window": window}


def listed():
    return [
        # the queries and keys of one decoding step of 32 sequences, sliced
        # out of a fused projection's rows: latency counts
        _rope("rope_step", 32, 40, 128, 128, "bf16", False, False, 8),
        # a training step's queries and their gradient
        _rope("rope_train", 16384, 32, 128, 128, "bf16", False, True, 0),
        # interleaved pairs over part of an odd head, odd counts, 32 bits
        _rope("rope_part_f32", 4099, 7, 96, 64, "f32", True, False, 3),
        # the new keys and values of a decoding step of 128 sequences,
        # rotated and written unquantised
        _cache("write_step", 128, 1, 8, 128, 16, "nhd", "bf16", "same", True,
               False),
        # one short prompt: written in 8 bits and read back
        _cache("prompt_e4m3", 1, 37, 8, 128, 16, "nhd", "bf16", "e4m3", True,
               True),
        # a long prefill batch, rotated, quantised and read back
        _cache("prefill_e4m3", 8, 8192, 8, 128, 64, "hnd", "bf16", "e4m3",
               True, True),
        # ragged prompts, five heads of 80, pages of 24, whole numbers
        _cache("ragged_int8", 13, 1531, 5, 80, 24, "nhd", "f16", "int8",
               False, True),
        # the cached prefixes of a batch, brought back for a chunk's prefill
        _read("prefix_e4m3", 16, 16384, 8, 128, 32, "nhd", "bf16", "e4m3"),
        # one sequence, a few hundred tokens: the latency of a lone user
        _attend("attend_one", 1, 500, 8, 4, 128, 16, "nhd", "bf16", "same",
                0),
        # a serving batch of ragged lengths, some rows empty
        _attend("attend_batch", 64, 8192, 8, 4, 128, 16, "nhd", "bf16",
                "same", 0),
        # the largest: many sequences over an 8-bit cache
        _attend("attend_e4m3", 128, 12288, 8, 8, 128, 64, "hnd", "bf16",
                "e4m3", 0),
        # few sequences with very long caches of whole numbers, an odd group
        _attend("attend_long_int8", 3, 131072, 4, 5, 64, 40, "nhd", "f16",
                "int8", 0),
    ]


def _log(rng, low, high):
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n - 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["rope", "cache", "read", "attend", "attend"])
    dim = rng.choice([64, 80, 112, 128, 128, 256])
    page = rng.choice([8, 16, 20, 32, 40, 64, 128])
    order = rng.choice(["nhd", "hnd"])
    dtype = rng.choice(["bf16", "f16"])
    store = rng.choice(["same", "e4m3", "int8"])
    heads = rng.choice([1, 2, 4, 5, 8, 16])
    if op == "rope":
        heads = rng.choice([1, 5, 8, 20, 28, 40])
        tokens = _log(rng, 1, 65536 * 32 * 128 // (heads * dim * 4))
        rot = dim if rng.random() < 0.6 else dim // 2
        c = _rope("", tokens, heads, dim, rot,
                  rng.choice(["bf16", "f16", "f32"]), rng.random() < 0.5,
                  rng.random() < 0.5, rng.choice([0, 1, 3]))
    else:
        total = 128 * 12288 * 8 * 128 // (8 if op != "attend" else 1)
        room = total // (2 * heads * dim)
        seqs = min(_log(rng, 1, 256), room)
        length = _log(rng, 1, max(1, min(131072, room // seqs)))
        if op == "cache":
            c = _cache("", seqs, length, heads, dim, page, order, dtype,
                       store, rng.random() < 0.5, True)
        elif op == "read":
            c = _read("", seqs, length, heads, dim, page, order, dtype, store)
        else:
            window = 0 if rng.random() < 0.75 else _log(rng, 1, length)
            c = _attend("", seqs, length, heads,
                        rng.choice([1, 2, 4, 5, 7, 8, 16]), dim, page, order,
                        dtype, store, window)
    del c["name"]
    return c


def _lens(case):
    """The lengths of a case's sequences: the longest as given, the others
    spread below it; in a larger batch one row is empty and one holds a
    single token.  The case alone decides them."""
    n, top = case["seqs"], case["length"]
    r = np.random.RandomState(n * 7919 + top * 31 + case["heads"])
    lens = r.randint(max(1, top // 2), top + 1, n)
    lens[0] = top
    if n >= 8 and top > 1:
        lens[n // 2] = 0
        lens[n // 3] = 1
    return [int(v) for v in lens]


def _spans(case):
    """How many keys each sequence's new token sees."""
    w = case["window"]
    return [min(n, w) if w else n for n in _lens(case)]


def work(case):
    if case["op"] == "rope":
        es = 4 if case["dtype"] == "f32" else 2
        n = case["tokens"] * case["heads"] * case["dim"]
        passes = 2 if case["backward"] else 1
        return {"bytes": passes * (2 * n * es) + case["tokens"] *
                (8 + 4 * case["rot"]), "flops": passes * 3 * n}
    es = 1 if case["store"] != "same" else 2
    scale = 0 if case["store"] == "same" else 4
    rows = sum(_lens(case)) * case["heads"]
    stored = 2 * rows * (case["dim"] * es + scale)   # keys and values
    dense = 2 * rows * case["dim"] * 2
    if case["op"] == "cache":
        bytes_ = dense + stored + 8 * sum(_lens(case))
        if case["rope"]:
            bytes_ += sum(_lens(case)) * (8 + 4 * case["dim"])
        if case["readback"]:
            bytes_ += stored + dense
        return {"bytes": bytes_, "flops": 8 * rows * case["dim"]}
    if case["op"] == "read":
        return {"bytes": stored + dense, "flops": 2 * rows * case["dim"]}
    rows = sum(_spans(case)) * case["heads"]
    heads_q = case["heads"] * case["group"]
    return {"bytes": 2 * rows * (case["dim"] * es + scale) +
            case["seqs"] * heads_q * (case["dim"] * 4 + 4),
            "flops": 4 * rows * case["group"] * case["dim"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _angles(rot):
    """Rotations a position: base 10000 over the rotated part's pairs."""
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return 10000.0 ** (-2.0 * i / rot)


def _table(rows, rot):
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * \
        _angles(rot)
    return torch.stack([a.cos(), a.sin()], 1).float()    # [rows, 2, rot / 2]


def _randn(shape, dtype, gen):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _pages(case, lens, gen):
    """(page table [seqs, most], pages): every sequence's pages, scattered
    over a pool a little larger than they need."""
    p = case["page"]
    most = max(1, max(-(-n // p) for n in lens))
    used = sum(-(-n // p) for n in lens)
    pool = used + max(1, used // 16)
    ids = torch.randperm(pool, generator=gen, device="cuda")[:used].cpu()
    table = torch.full((len(lens), most), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // p)
        table[b, :m] = ids[at:at + m].int()
        at += m
    return table.cuda(), pool


def _page_shape(case, pool):
    p, h, d = case["page"], case["heads"], case["dim"]
    return (pool, p, h, d) if case["order"] == "nhd" else (pool, h, p, d)


def _by_token(case, pages):
    """Pages as [page, token, head, ...] whatever their order."""
    return pages if case["order"] == "nhd" else pages.transpose(1, 2)


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
    inv = torch.where(top == 0, torch.zeros_like(top), 127.0 / top)
    inv = inv.clamp(max=2.0 ** 126)
    return (x * inv[..., None]).round().to(torch.int8), scale


def _filled(case, pool, gen):
    """A cache's pages and scales with the rows of random keys (or values)."""
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
    s = {"case": case}
    if case["op"] == "rope":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        dtype = DTYPES[case["dtype"]]
        rows = max(4096, t // 4)
        s["x"] = _randn((t, h + case["gap"], d), dtype, gen)[:, :h]
        s["pos"] = torch.randint(0, rows, (t,), generator=gen, device="cuda")
        s["table"] = _table(rows, case["rot"])
        s["out"] = torch.empty((t, h, d), dtype=dtype, device="cuda")
        if case["backward"]:
            s["dy"] = _randn((t, h, d), dtype, gen)
            s["dx"] = torch.empty_like(s["out"])
        if own:
            import layout_driven_movement_gb300 as lm
            s["plan"] = lm.RopePlan(d, case["rot"],
                                    interleaved=case["interleaved"])
        return s
    lens = _lens(case)
    s["page_table"], pool = _pages(case, lens, gen)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    starts = np.concatenate([[0], np.cumsum(lens)])
    s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    total = int(starts[-1])
    dtype, h, d = DTYPES[case["dtype"]], case["heads"], case["dim"]
    if case["op"] == "cache":
        shape, kind = _page_shape(case, pool), _store_dtype(case)
        s["k_pages"] = torch.zeros(shape, device="cuda").to(kind)
        s["v_pages"] = torch.zeros(shape, device="cuda").to(kind)
        s["k_scale"] = s["v_scale"] = None
        if case["store"] != "same":
            s["k_scale"] = torch.ones((pool, h, case["page"]), device="cuda")
            s["v_scale"] = torch.ones_like(s["k_scale"])
        kv = _randn((total, 2, h, d), dtype, gen)
        s["k"], s["v"] = kv[:, 0], kv[:, 1]
        seq = torch.repeat_interleave(
            torch.arange(len(lens), device="cuda"), s["lens"].long())
        pos = torch.arange(total, device="cuda") - s["starts"].long()[seq]
        s["slots"] = s["page_table"].long()[seq, pos // case["page"]] * \
            case["page"] + pos % case["page"]
        s["pos"] = pos
        if case["rope"]:
            s["table"] = _table(max(lens), d)
            s["rope"] = None
            if own:
                import layout_driven_movement_gb300 as lm
                s["rope"] = lm.RopePlan(d)
        s["seq"], s["total"] = seq, total
    else:
        s["k_pages"], s["k_scale"] = _filled(case, pool, gen)
        s["v_pages"], s["v_scale"] = _filled(case, pool, gen)
    if case["op"] != "attend":
        s["total"] = total
        s["k_out"] = torch.empty((total, h, d), dtype=dtype, device="cuda")
        s["v_out"] = torch.empty_like(s["k_out"])
    else:
        b, heads = len(lens), h * case["group"]
        s["q"] = _randn((b, heads, d), dtype, gen)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((b, heads), device="cuda")
        s["scale"] = d ** -0.5
    if own:
        s["cache"] = _kv_cache(case, s)
        if case["op"] == "attend":
            import layout_driven_movement_gb300 as lm
            s["workspace"] = torch.zeros(
                lm.kv_attend_workspace(s["cache"].plan, *s["q"].shape[:2]),
                dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass: the plain forms
# ---------------------------------------------------------------------------

def _rotate(x, pos, table, rot, interleaved, inverse):
    """Rotary positions of rows [tokens, heads, dim], in 32 bits."""
    x = x.float()
    cos, sin = table[pos][:, None].unbind(2)          # [tokens, 1, rot / 2]
    if inverse:
        sin = -sin
    part, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else \
        torch.cat([c, d], -1)
    return torch.cat([turned, rest], -1)


def _run_rope(s):
    c = s["case"]
    dtype = DTYPES[c["dtype"]]
    out = {"y": _rotate(s["x"], s["pos"], s["table"], c["rot"],
                        c["interleaved"], False).to(dtype)}
    if c["backward"]:
        out["dx"] = _rotate(s["dy"], s["pos"], s["table"], c["rot"],
                            c["interleaved"], True).to(dtype)
    return out


def _values(case, pages, scales, table):
    """The rows of the pages of `table`, in 32 bits: [..., page, head, dim]
    for every entry."""
    x = _by_token(case, pages.view(torch.uint8) if case["store"] == "e4m3"
                  else pages)[table]
    if case["store"] == "e4m3":
        x = x.view(torch.float8_e4m3fn)
    x = x.float()
    if scales is not None:
        x = x * scales.transpose(1, 2)[table][..., None]
    return x


def _run_cache(s):
    c = s["case"]
    p = c["page"]
    page, at = s["slots"] // p, s["slots"] % p
    for name in ("k", "v"):
        x = s[name].float()
        if c["rope"] and name == "k":
            x = _rotate(x, s["pos"], s["table"], c["dim"], False, False)
        pages = _by_token(c, s[name + "_pages"])
        if c["store"] == "same":
            pages[page, at] = x.to(pages.dtype)
            continue
        codes, scale = _quantise(x, c["store"])
        if c["store"] == "e4m3":
            _by_token(c, s[name + "_pages"].view(torch.uint8))[page, at] = \
                codes.view(torch.uint8)
        else:
            pages[page, at] = codes
        s[name + "_scale"].transpose(1, 2)[page, at] = scale
    out = {}
    if c["store"] != "same":
        out = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if not c["readback"]:
        return dict(out, k_pages=s["k_pages"], v_pages=s["v_pages"])
    return dict(out, **_run_read(s))


def _run_read(s):
    c = s["case"]
    out = {}
    every = torch.arange(s["page_table"].shape[1] * c["page"], device="cuda")
    seen = every[None] < s["lens"][:, None]
    for name in ("k", "v"):
        x = _values(c, s[name + "_pages"], s[name + "_scale"],
                    s["page_table"].long().clamp(min=0))
        x = x.flatten(1, 2)[seen]                     # the rows, in order
        out[name] = x.to(DTYPES[c["dtype"]])
    return out


def _run_attend(s):
    c = s["case"]
    b, heads, d = s["q"].shape
    table = s["page_table"].long().clamp(min=0)
    k = _values(c, s["k_pages"], s["k_scale"], table).flatten(1, 2)
    q = s["q"].float().view(b, c["heads"], c["group"], d)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]
    at = torch.arange(k.shape[1], device="cuda")[None]
    n = s["lens"].long()[:, None]
    seen = at < n
    if c["window"]:
        seen &= at >= n - c["window"]
    score = torch.where(seen[:, None, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    v = _values(c, s["v_pages"], s["v_scale"], table).flatten(1, 2)
    v = torch.where(seen[:, :, None, None], v, torch.zeros_like(v))
    out = torch.matmul(p, v.transpose(1, 2))
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + torch.log(total))[..., 0]
    return {"out": out.view(b, heads, d).to(s["q"].dtype),
            "lse": lse.view(b, heads)}


# ---------------------------------------------------------------------------
# One pass: the framework's kernels
# ---------------------------------------------------------------------------

def _own_rope(s):
    import layout_driven_movement_gb300 as lm
    lm.rope(s["plan"], s["x"], s["pos"], s["table"], s["out"])
    out = {"y": s["out"]}
    if s["case"]["backward"]:
        lm.rope(s["plan"], s["dy"], s["pos"], s["table"], s["dx"],
                inverse=True)
        out["dx"] = s["dx"]
    return out


def _own_cache(s):
    import layout_driven_movement_gb300 as lm
    c = s["case"]
    if c["rope"]:
        lm.kv_write(s["cache"], s["k"], s["v"], s["slots"], rope=s["rope"],
                    positions=s["pos"], table=s["table"])
    else:
        lm.kv_write(s["cache"], s["k"], s["v"], s["slots"])
    out = {}
    if c["store"] != "same":
        out = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if not c["readback"]:
        return dict(out, k_pages=s["k_pages"], v_pages=s["v_pages"])
    return dict(out, **_own_read(s))


def _own_read(s):
    import layout_driven_movement_gb300 as lm
    lm.kv_read(s["cache"], s["page_table"], s["lens"], s["starts"],
               s["k_out"], s["v_out"])
    return {"k": s["k_out"], "v": s["v_out"]}


def _own_attend(s):
    import layout_driven_movement_gb300 as lm
    lm.kv_attend(s["cache"], s["q"], s["page_table"], s["lens"], s["out"],
                 s["workspace"], lse=s["lse"], scale=s["scale"],
                 window=s["case"]["window"])
    return {"out": s["out"], "lse": s["lse"]}


PLAIN = {"rope": _run_rope, "cache": _run_cache, "read": _run_read,
         "attend": _run_attend}
OWN = {"rope": _own_rope, "cache": _own_cache, "read": _own_read,
       "attend": _own_attend}


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _turn64(x, pos, table, rot, interleaved, sign):
    """Each pair as a complex number times cos + i sin."""
    x = x.double()
    t = table.double()[pos]
    w = torch.complex(t[:, 0], sign * t[:, 1])[:, None]
    half = rot // 2
    first = torch.arange(half, device=x.device)
    lo, hi = (2 * first, 2 * first + 1) if interleaved else \
        (first, first + half)
    z = torch.complex(x[..., lo], x[..., hi]) * w
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _e4m3_64(x):
    """The nearest e4m3 value, ties to the even one."""
    e = torch.frexp(x.abs())[1] - 1
    step = torch.exp2(e.clamp(min=-6).double() - 3)
    return torch.round(x / step) * step


def _held64(x, store):
    """(the values that a row is held as, its scale)."""
    top = x.abs().amax(-1, keepdim=True)
    if store == "e4m3":
        scale = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX)))
        scale = torch.where(top > 0, scale, 1.0)
        return _e4m3_64(x / scale) * scale, scale[..., 0]
    scale = torch.where(top > 0, top / 127, 1.0)
    return torch.round(x / scale) * scale, scale[..., 0]


def _rows64(case, s, name, b, n):
    """The first n rows that sequence b holds: [n, heads, dim]."""
    p = case["page"]
    ids = s["page_table"][b, :-(-n // p)].long()
    pages = s[name + "_pages"]
    x = pages.view(torch.uint8)[ids].view(torch.float8_e4m3fn) \
        if case["store"] == "e4m3" else pages[ids]
    x = x.double()
    if case["order"] == "hnd":
        x = x.permute(0, 2, 1, 3)
    if case["store"] != "same":
        x = x * s[name + "_scale"][ids].double().permute(0, 2, 1)[..., None]
    return x.reshape(-1, case["heads"], case["dim"])[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        turn = (s["pos"], s["table"], case["rot"], case["interleaved"])
        out = {"y": _turn64(s["x"], *turn, 1.0)}
        if case["backward"]:
            out["dx"] = _turn64(s["dy"], *turn, -1.0)
        return out
    lens = _lens(case)
    if case["op"] == "cache":
        out = {}
        for name in ("k", "v"):
            x = s[name].double()
            if case["rope"] and name == "k":
                x = _turn64(x, s["pos"], s["table"], case["dim"], False, 1.0)
            if case["store"] != "same":
                x, scale = _held64(x, case["store"])
                place = torch.ones(s[name + "_scale"].shape, device="cuda",
                                   dtype=torch.float64)
                place.permute(0, 2, 1)[s["slots"] // case["page"],
                                       s["slots"] % case["page"]] = scale
                out[name + "_scale"] = place
            if case["readback"]:
                out[name] = x
            else:
                place = s[name + "_pages"].double()
                by = place if case["order"] == "nhd" else \
                    place.permute(0, 2, 1, 3)
                by[s["slots"] // case["page"],
                   s["slots"] % case["page"]] = x
                out[name + "_pages"] = place
        return out
    if case["op"] == "read":
        return {name: torch.cat([_rows64(case, s, name, b, n)
                                 for b, n in enumerate(lens)])
                for name in ("k", "v")}
    # attention, a sequence at a time
    b, heads, d = s["q"].shape
    out = torch.zeros((b, heads, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, heads), -math.inf, dtype=torch.float64,
                     device="cuda")
    for i, n in enumerate(lens):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        k = _rows64(case, s, "k", i, n)[lo:]
        v = _rows64(case, s, "v", i, n)[lo:]
        for h in range(case["heads"]):
            g = slice(h * case["group"], (h + 1) * case["group"])
            z = s["q"][i, g].double() @ k[:, h].T * s["scale"]
            lse[i, g] = torch.logsumexp(z, -1)
            out[i, g] = torch.softmax(z, -1) @ v[:, h]
    return {"out": out, "lse": lse}
