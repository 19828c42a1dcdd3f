// Argument checks that the calls of the paged key-value cache share: dense rows,
// tables, overlaps, a cache against its plan.
#pragma once

#include <cmath>
#include <cstring>
#include <new>

#include "lm_kv.h"

namespace lm {

template <class F>
int guarded(F&& f) {
  try {
    f();
    return LM_OK;
  } catch (const Error& e) {
    return e.status;
  } catch (const std::bad_alloc&) {
    return LM_E_NOMEM;
  } catch (...) {
    return LM_E_INVALID;
  }
}

inline void need(bool ok, int status = LM_E_INVALID) {
  if (!ok) fail(status);
}

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

struct Range {
  uintptr_t lo = 0, hi = 0;
  bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
};

// Checks a dense tensor of `tokens` x `heads` rows of dim elements and gives
// the bytes it spans.  Rows of an output must not share elements.
inline Range check_rows(const lm_rows* r, int64_t tokens, int64_t heads, int64_t dim,
                 int es, bool output) {
  need(r && r->data && r->token_stride >= 0 && r->head_stride >= 0 &&
       r->capacity >= 0 && addr(r->data) % uintptr_t(es) == 0);
  const int64_t last =
      add_chk(add_chk(mul_chk(tokens - 1, r->token_stride),
                      mul_chk(heads - 1, r->head_stride)),
              dim);
  need(last <= r->capacity, LM_E_CAPACITY);
  if (output) {
    const int64_t t = tokens > 1 ? r->token_stride : INT64_MAX;
    const int64_t h = heads > 1 ? r->head_stride : INT64_MAX;
    const int64_t small = t < h ? t : h;
    const int64_t n_small = t < h ? tokens : heads;
    need(small >= dim);
    if (t != INT64_MAX && h != INT64_MAX)
      need((t < h ? h : t) >= add_chk(mul_chk(n_small - 1, small), dim));
  }
  return {addr(r->data), addr(r->data) + uintptr_t(mul_chk(last, es))};
}

typedef __int128 wide;

// Whether |r + i big + j small| < w for an i in [i0, i1] and a j in [j0, j1].
// Few i come near where a span of j's is no longer than big, as the rows of an
// output are.
inline bool near_zero(wide r, wide big, wide i0, wide i1, wide small, wide j0,
               wide j1, wide w) {
  auto down = [](wide a, wide b) { return a / b - (a % b < 0); };
  if (big == 0) i0 = i1 = 0;
  if (small == 0) j0 = j1 = 0;
  if (big > 0) {
    const wide lo = down(-w - j1 * small - r, big);
    const wide hi = down(w - j0 * small - r, big) + 1;
    if (i0 < lo) i0 = lo;
    if (i1 > hi) i1 = hi;
  }
  for (wide i = i0; i <= i1; ++i) {
    const wide rest = r + i * big;
    const wide at = small == 0 ? 0 : down(-rest, small);
    for (wide j = at; j <= at + 1; ++j) {
      const wide k = j < j0 ? j0 : j > j1 ? j1 : j;
      const wide d = rest + k * small;
      if (d < w && d > -w) return true;
    }
  }
  return false;
}

// Whether two outputs of one shape share elements.  Each one's own rows are
// apart.  Tokens a different distance apart in the two: taken as shared.
inline bool rows_meet(const lm_rows& a, const lm_rows& b, int64_t tokens,
               int64_t heads, int64_t dim, int es) {
  const wide w = wide(dim) * es;
  const wide r = wide(addr(b.data)) - wide(addr(a.data));
  const wide ts = tokens > 1 ? wide(b.token_stride) * es : 0;
  const wide ah = heads > 1 ? wide(a.head_stride) * es : 0;
  const wide bh = heads > 1 ? wide(b.head_stride) * es : 0;
  if (tokens > 1 && a.token_stride != b.token_stride) return true;
  const wide t = tokens - 1;
  auto meet = [&](wide from, wide h0, wide h1) {
    return ts >= bh ? near_zero(from, ts, -t, t, bh, h0, h1, w)
                    : near_zero(from, bh, h0, h1, ts, -t, t, w);
  };
  if (ah == bh) return meet(r, 1 - heads, heads - 1);
  for (int64_t h = 0; h < heads; ++h)
    if (meet(r - h * ah, 0, heads - 1)) return true;
  return false;
}

inline bool vector_rows(const lm_rows& r, int es) {
  const int64_t v = 16 / es;
  return addr(r.data) % 16 == 0 && r.token_stride % v == 0 &&
         r.head_stride % v == 0;
}

inline Rows rows_of(const lm_rows& r) {
  Rows o;
  o.p = static_cast<char*>(r.data);
  o.ts = r.token_stride;
  o.hs = r.head_stride;
  return o;
}

inline Turn check_turn(const lm_rope_plan& rope, const void* positions,
                int position_bytes, const float* table, int64_t table_rows,
                int inverse) {
  need(positions && table && (position_bytes == 4 || position_bytes == 8) &&
       table_rows >= 0 && addr(table) % 4 == 0 &&
       addr(positions) % uintptr_t(position_bytes) == 0);
  Turn t;
  t.table = table;
  t.pos = positions;
  t.rows = table_rows;
  t.pos64 = position_bytes == 8;
  t.rot = rope.rotary;
  t.inter = rope.inter;
  t.inverse = inverse != 0;
  return t;
}

// Whether a range meets one of the pages that lie in `all` (not the room
// between them).
inline bool pages_meet(const lm_kv_plan& p, const lm_kv_cache* c, const Range& all,
                const Range& o) {
  if (!o.meets(all)) return false;
  const uintptr_t stride = uintptr_t(p.page_stride) * uintptr_t(p.held);
  const uintptr_t page = uintptr_t(p.page_cosize) * uintptr_t(p.held);
  const uintptr_t lo = o.lo > all.lo ? o.lo - all.lo : 0, hi = o.hi - all.lo;
  const uintptr_t n = lo / stride;      // the last page that starts at or below
  return lo - n * stride < page ||
         (n + 1 < uintptr_t(c->pages) && (n + 1) * stride < hi);
}

// The bytes that a cache's keys, values and scales (empty for SAME) span.
struct CacheRanges {
  Range k, v, ks, vs;
  bool meet(const Range& o) const {
    return o.meets(k) || o.meets(v) || o.meets(ks) || o.meets(vs);
  }
};

// Checks a cache against its plan.
inline CacheArgs check_cache(const lm_kv_plan& p, const lm_kv_cache* c,
                      CacheRanges* r) {
  need(c && c->k && c->v && c->pages >= 1 && c->k_capacity >= 0 &&
       c->v_capacity >= 0);
  need(addr(c->k) % 16 == 0 && addr(c->v) % 16 == 0);
  need(c->k != c->v, LM_E_OVERLAP);
  const int64_t span =
      add_chk(mul_chk(c->pages - 1, p.page_stride), p.page_cosize);
  need(span <= c->k_capacity && span <= c->v_capacity, LM_E_CAPACITY);
  mul_chk(c->pages, p.page_tokens);  // every slot number fits 64 bits
  CacheArgs a;
  if (p.store != LM_KV_SAME) {
    need(c->k_scale && c->v_scale && addr(c->k_scale) % 4 == 0 &&
         addr(c->v_scale) % 4 == 0);
    const int64_t scales = mul_chk(c->pages, mul_chk(p.heads, p.page_tokens));
    need(scales <= c->scale_capacity, LM_E_CAPACITY);
    const uintptr_t bytes = uintptr_t(mul_chk(scales, 4));
    r->ks = {addr(c->k_scale), addr(c->k_scale) + bytes};
    r->vs = {addr(c->v_scale), addr(c->v_scale) + bytes};
    need(!r->ks.meets(r->vs), LM_E_OVERLAP);
    a.ks = c->k_scale;
    a.vs = c->v_scale;
  }
  a.k = static_cast<char*>(c->k);
  a.v = static_cast<char*>(c->v);
  a.page_b = mul_chk(p.page_stride, p.held);
  a.token_b = mul_chk(p.token_stride, p.held);
  a.head_b = mul_chk(p.head_stride, p.held);
  a.pages = c->pages;
  a.page_tokens = uint32_t(p.page_tokens);
  a.heads = uint32_t(p.heads);
  a.page_div = make_fastdiv(uint32_t(p.page_tokens));
  a.dim = int32_t(p.dim);
  const uintptr_t bytes = uintptr_t(mul_chk(span, p.held));
  r->k = {addr(c->k), addr(c->k) + bytes};
  r->v = {addr(c->v), addr(c->v) + bytes};
  for (const Range& scale : {r->ks, r->vs})
    need(!pages_meet(p, c, r->k, scale) && !pages_meet(p, c, r->v, scale),
         LM_E_OVERLAP);
  return a;
}

// Checks the bounds of a plan's pages and gives the bytes that they span.
struct BoundRanges {
  Range data, scale;
};
inline BoundRanges check_bounds(const lm_kv_plan& p, int64_t pages,
                                const lm_kv_bounds* b) {
  need(b && b->data && b->scale && b->capacity >= 0 &&
       b->scale_capacity >= 0 && addr(b->data) % 16 == 0 &&
       addr(b->scale) % 4 == 0);
  const int64_t scales = mul_chk(pages, p.heads);
  const int64_t bytes = mul_chk(scales, 2 * p.dim);
  need(bytes <= b->capacity && scales <= b->scale_capacity, LM_E_CAPACITY);
  BoundRanges r;
  r.data = {addr(b->data), addr(b->data) + uintptr_t(bytes)};
  r.scale = {addr(b->scale), addr(b->scale) + uintptr_t(mul_chk(scales, 4))};
  need(!r.data.meets(r.scale), LM_E_OVERLAP);
  return r;
}

// Pages, tokens and sequences as the kernels count them.
inline void check_table(const lm_kv_plan& p, const int32_t* table, int64_t stride,
                 int seqs, int64_t max_pages, const int32_t* lens) {
  need((table || max_pages == 0) && lens && seqs >= 0 && max_pages >= 0 &&
       stride >= 0 && addr(table) % 4 == 0 && addr(lens) % 4 == 0);
  need(seqs <= 1 || stride >= max_pages);
  // key numbers, rounded up to whole tiles, fit 32 bits
  need(mul_chk(max_pages, p.page_tokens) < (int64_t(1) << 31) - 4096,
       LM_E_OVERFLOW);
}

}  // namespace lm
