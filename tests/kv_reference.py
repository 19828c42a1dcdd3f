"""The paged key-value cache in 64 bits, by loops over tokens and sequences,
and the inputs of its tests.  Shares no code with the library."""

import math

import torch

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11,
         torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25,
        torch.float32: 2.0 ** -150}


def e4m3_values():
    """The 256 codes' values from the format: 4 exponent bits (bias 7), 3
    mantissa bits, code 127 is not a number."""
    out = []
    for c in range(256):
        s, e, m = (-1.0 if c & 128 else 1.0), (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out.append(math.nan if c & 127 == 127 else s * v)
    return torch.tensor(out, dtype=torch.float64)


def e4m3_nearest(x):
    """The codes of 64-bit values of magnitude 448 at most: nearest, ties to
    the even code."""
    grid = e4m3_values()[:127]
    a = x.abs().unsqueeze(-1)
    d = (a - grid).abs()
    best = d.argmin(-1)                      # the lower of two equal ones
    up = (best + 1).clamp(max=126)
    tie = d.gather(-1, up.unsqueeze(-1))[..., 0] == \
        d.gather(-1, best.unsqueeze(-1))[..., 0]
    best = torch.where(tie & (best % 2 == 1), up, best)
    return best + 128 * torch.signbit(x).long()


def e4m3_scale(top):
    """The smallest power of two 2^e, e >= -126, with top <= 448 * 2^e."""
    if top == 0:
        return 1.0
    e = -126
    while top > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


def turn(x, pos, freqs, rot, interleaved, sign=1.0, amplitude=1.0):
    """x [tokens, heads, dim] in 64 bits; pair by pair."""
    x = x.double()
    y = x.clone()
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        # the angle's cosine and sine as the 32-bit table holds them
        ang = pos.double() * f
        c = (ang.cos() * amplitude).float().double()[:, None]
        s = sign * (ang.sin() * amplitude).float().double()[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def turn_bound(x, rot, interleaved, dtype, y, amplitude=1.0):
    """Elementwise bound of a 32-bit turn: three roundings of terms no larger
    than the pair's magnitudes, then the rounding to dtype; the table's sines
    may differ from the reference's by a rounding of 2^-24."""
    x = x.double().abs()
    pair = x.clone()
    half = rot // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        pair[..., a] = pair[..., b] = x[..., a] + x[..., b]
    t = 4 * 2.0 ** -24 * amplitude * pair
    t[..., rot:] = 0
    return t * (1 + ROUND[dtype]) + y.abs() * ROUND[dtype] + TINY[dtype]


def attend(q, keys, values, group, scale, window=0):
    """One sequence: q [heads_q, dim], keys and values [n, heads, dim], all in
    64 bits.  Returns (out, lse, sum p |v|, largest sum |q||k| scale)."""
    hq, d = q.shape
    n = keys.shape[0]
    lo = max(0, n - window) if window else 0
    out = torch.zeros(hq, d, dtype=torch.float64)
    lse = torch.full((hq,), -math.inf, dtype=torch.float64)
    mag = torch.zeros(hq, d, dtype=torch.float64)
    dot = torch.zeros(hq, dtype=torch.float64)
    if n == lo:
        return out, lse, mag, dot
    for h in range(hq):
        k, v = keys[lo:, h // group], values[lo:, h // group]
        s = (k @ q[h]) * scale
        top = s.max()
        if top == -math.inf:
            continue
        p = torch.exp(s - top)
        lse[h] = top + torch.log(p.sum())
        p = p / p.sum()
        out[h] = p @ v
        mag[h] = p @ v.abs()
        dot[h] = (k.abs() @ q[h].abs()).max() * abs(scale)
    return out, lse, mag, dot


def attend_bounds(dtype, dim, out, lse, mag, dot):
    """(bound of out, bound of lse).  A score of dim products in 32 bits is
    off by e = (dim + 4) 2^-24 sum |q||k| scale at most, a weight then by the
    factor 1 + 2e, one rounding of a weight to 16 bits (2^-11 for the 8-bit
    caches) and 2^-20 of its exponential; 2^-10 covers the last two and the
    sums.  The result is rounded once to dtype."""
    e = ((dim + 4) * 2.0 ** -24 * dot)
    b = (2 * e[..., None] + 2.0 ** -10) * mag + \
        out.abs() * ROUND[dtype] * 1.01 + TINY[dtype]
    return b, 2 * e + 2.0 ** -18 + 2.0 ** -23 * lse.abs().nan_to_num(0, 0, 0)


class Pages:
    """A cache on the CPU: held codes and scales, and the 64-bit rows that
    they stand for, filled for `lens` tokens of random sequences.  What no
    token names holds garbage (NaN where the type has one)."""

    def __init__(self, lens, heads, dim, page, order, dtype, store, seed=0,
                 spare=3, mult=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.dim, self.page = lens, heads, dim, page
        self.order, self.dtype, self.store = order, dtype, store
        need = [-(-n // page) for n in lens]
        self.pool = sum(need) + spare
        self.most = max(1, max(need, default=1))
        ids = torch.randperm(self.pool, generator=g)[:sum(need)].tolist()
        self.table = torch.full((len(lens), self.most), -7, dtype=torch.int32)
        shape = (self.pool, page, heads, dim)
        self.rows, self.codes, self.scales = [], [], []
        at = 0
        where = []
        for b, m in enumerate(need):
            self.table[b, :m] = torch.tensor(ids[at:at + m],
                                             dtype=torch.int32)
            where.append(ids[at:at + m])
            at += m
        for kv in range(2):
            if store is None:
                held = torch.full(shape, math.nan, dtype=dtype)
                scale = None
            else:
                held = torch.full(shape, 127, dtype=torch.uint8)
                scale = torch.full((self.pool, page, heads), math.nan)
            rows = []
            for b, n in enumerate(lens):
                x = torch.randn(n, heads, dim, generator=g) * mult
                x = x * torch.exp(0.5 * torch.randn(n, heads, 1, generator=g))
                if store is None:
                    code, sc = x.to(dtype), None
                    row = code.double()
                elif store == "e4m3":
                    sc = torch.exp2(torch.ceil(torch.log2(
                        x.abs().amax(-1) / 448)))
                    code = e4m3_nearest(x.double() / sc[..., None].double())
                    row = e4m3_values()[code] * sc[..., None].double()
                    code = code.to(torch.uint8)
                else:
                    sc = x.abs().amax(-1) / 127
                    code = torch.round(x / sc[..., None])
                    row = code.double() * sc[..., None].double()
                    code = code.to(torch.int8).view(torch.uint8)
                rows.append(row)
                for j in range(n):
                    p, o = where[b][j // page], j % page
                    held[p, o] = code[j]
                    if sc is not None:
                        scale[p, o] = sc[j]
            self.rows.append(rows)
            self.codes.append(held)
            self.scales.append(scale)

    def page_layout(self):
        h, d, p = self.heads, self.dim, self.page
        return ([p, h, d], [h * d, d, 1] if self.order == "nhd"
                else [d, p * d, 1], [1, 1, 1])

    def device(self, kv):
        """The held pages, in the cache's order, flat, on the GPU."""
        x = self.codes[kv]
        if self.order == "hnd":
            x = x.transpose(1, 2)
        return x.contiguous().cuda()

    def device_scale(self, kv):
        if self.scales[kv] is None:
            return None
        return self.scales[kv].transpose(1, 2).contiguous().cuda()
