"""Random caches and the long-context operators in 64 bits, from their
definitions.  Shares no code with the library."""

import math

import torch

from kv_reference import e4m3_values


class Held:
    """A cache on the GPU with random rows in every page, and the 64-bit rows
    that they stand for; what the first `lens` tokens of its sequences do not
    name holds NaN (or, as codes, scales that are NaN)."""

    def __init__(self, lens, heads, dim, page, order, dtype, store, seed=0,
                 spare=3, drift=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.heads, self.dim, self.page = lens, heads, dim, page
        self.order, self.dtype, self.store = order, dtype, store
        need = [-(-n // page) for n in lens]
        self.pool = sum(need) + spare
        self.most = max(1, max(need, default=1))
        ids = torch.randperm(self.pool, generator=g, device="cuda").cpu()
        self.table = torch.full((len(lens), self.most), -7, dtype=torch.int32)
        live = torch.zeros(self.pool, page, dtype=torch.bool)
        at = 0
        for b, (n, m) in enumerate(zip(lens, need)):
            self.table[b, :m] = ids[at:at + m].int()
            full = torch.zeros(m * page, dtype=torch.bool)
            full[:n] = True
            live[ids[at:at + m]] = full.view(m, page)
            at += m
        self.spare = ids[at:]
        live = live.cuda()[:, :, None, None]
        shape = (self.pool, page, heads, dim)
        self.held, self.scales, self.rows = [], [], []
        for kv in range(2):
            x = torch.randn(shape, generator=g, device="cuda")
            x *= torch.exp(0.5 * torch.randn(shape[:3] + (1,), generator=g,
                                             device="cuda"))
            if drift:
                x += drift * torch.randn((self.pool, 1, heads, dim),
                                         generator=g, device="cuda")
            scale = None
            if store is None:
                x = torch.where(live, x, math.nan).to(dtype)
                row = x.double()
            else:
                scale = torch.exp(torch.randn(shape[:3], generator=g,
                                              device="cuda")) * 2.0 ** -7
                scale = torch.where(live[..., 0], scale, math.nan)
                if store == "int8":
                    x = (x * 40).round().clamp(-128, 127).to(torch.int8)
                    row = x.double() * scale.double()[..., None]
                else:
                    # any code but the ones that are no number
                    c = torch.randint(0, 127, shape, generator=g,
                                      device="cuda")
                    c += 128 * torch.randint(0, 2, shape, generator=g,
                                             device="cuda")
                    row = e4m3_values().cuda()[c] * scale.double()[..., None]
                    x = c.to(torch.uint8)
            if order == "hnd":
                x = x.transpose(1, 2)
            self.held.append(x.contiguous())
            self.scales.append(None if scale is None else
                               scale.transpose(1, 2).contiguous())
            self.rows.append(row)

    def cache(self, lm):
        p, h, d = self.page, self.heads, self.dim
        page = lm.Layout.make([p, h, d], [h * d, d, 1] if self.order == "nhd"
                              else [d, p * d, 1], [1, 1, 1])
        plan = lm.KVPlan(page, self.dtype, self.store)
        return lm.KVCache(plan, *self.held, *self.scales), plan

    def of(self, kv, pages, n):
        """The first n rows of a list of pages: [n, heads, dim] in 64 bits."""
        pages = pages[:-(-n // self.page)].long().cuda()
        return self.rows[kv][pages].reshape(-1, self.heads, self.dim)[:n]

    def seq(self, kv, b):
        return self.of(kv, self.table[b], self.lens[b])

    def values32(self):
        """The keys as a read back into 32 bits gives them (a row's code times
        its scale, rounded once): [page, token, head, dim]."""
        return self.rows[0].float()


def attend(q, keys, values, group, scale):
    """q [heads_q, dim], keys and values [n, heads, dim] in 64 bits: (out, lse,
    p [heads_q, n], sum p |v|, largest sum |q||k| scale)."""
    hq, d = q.shape
    n, heads = keys.shape[:2]
    if n == 0:
        z = torch.zeros(hq, dtype=torch.float64, device=q.device)
        return z[:, None].expand(hq, d), z - math.inf, z[:, None][:, :0], \
            z[:, None].expand(hq, d), z
    qg = q.view(heads, group, d)
    s = torch.einsum("hgd,nhd->hgn", qg, keys) * scale
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    lse = (top + torch.log(total)).reshape(hq)
    p = torch.where(total > 0, p / total, 0.0)
    out = torch.einsum("hgn,nhd->hgd", p, values).reshape(hq, d)
    mag = torch.einsum("hgn,nhd->hgd", p, values.abs()).reshape(hq, d)
    dot = torch.einsum("hgd,nhd->hgn", qg.abs(), keys.abs()).amax(-1) \
        * abs(scale)
    return out, lse, p.reshape(hq, n), mag, dot.reshape(hq)


def power(top):
    """The smallest power of two 2^e, e >= -126, with top <= 127 * 2^e."""
    if top == 0:
        return 1.0
    e = max(-126, math.frexp(top / 127)[1] - 1)
    while top > math.ldexp(127.0, e):
        e += 1
    return math.ldexp(1.0, e)


def bounds(rows):
    """rows [tokens, dim] (values of 32 bits): (lo, hi, scale) as whole
    numbers."""
    d = rows.shape[1]
    if rows.shape[0] == 0:
        return torch.zeros(d), torch.zeros(d), 1.0
    rows = rows.double().cpu()
    if not torch.isfinite(rows).all():
        return torch.zeros(d), torch.zeros(d), math.nan
    by = power(rows.abs().max().item())
    return torch.floor(rows.amin(0) / by), torch.ceil(rows.amax(0) / by), by


def choose(score, keep, first, last):
    """Which of the pages a choice by score takes, in order."""
    n = len(score)
    if n <= keep:
        return list(range(n))
    middle = list(range(first, n - last))
    rank = sorted(middle, key=lambda i: (
        -math.inf if math.isnan(score[i]) else -score[i], i))
    if any(math.isnan(score[i]) for i in middle):
        rank = sorted(middle, key=lambda i: (not math.isnan(score[i]),
                                             0 if math.isnan(score[i])
                                             else -score[i], i))
    return sorted(list(range(first)) + rank[:keep - first - last] +
                  list(range(n - last, n)))


def scores(q, lo, hi, scale, group):
    """q [heads_q, dim]; lo, hi [pages, heads, dim] and scale [pages, heads]
    of one sequence's pages: [heads, pages] in 64 bits."""
    heads = lo.shape[1]
    out = torch.full((heads, lo.shape[0]), -math.inf, dtype=torch.float64)
    for h in range(heads):
        for g in range(group):
            x = q[h * group + g].double().cpu()
            if not torch.isfinite(x).all():
                out[h] = math.nan
                continue
            by = power(x.abs().max().item())
            c = torch.round(x / by)
            s = torch.where(c > 0, c * hi[:, h].double(),
                            c * lo[:, h].double()).sum(-1) * by
            out[h] = torch.where(out[h].isnan(), out[h],
                                 torch.maximum(out[h], s))
    return out * scale.T.double()
