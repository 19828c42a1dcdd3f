// The paged key-value cache and rotary positions, host side: plans, argument
// checks and the hand-over to the kernels' launchers.
#include <cmath>
#include <cstring>
#include <new>

#include "lm_kv.h"

namespace lm {
namespace {

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

void need(bool ok, int status = LM_E_INVALID) {
  if (!ok) fail(status);
}

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

struct Range {
  uintptr_t lo = 0, hi = 0;
  bool meets(const Range& o) const { return lo < o.hi && o.lo < hi; }
};

// Checks a dense tensor of `tokens` x `heads` rows of dim elements and gives
// the bytes it spans.  Rows of an output must not share elements.
Range check_rows(const lm_rows* r, int64_t tokens, int64_t heads, int64_t dim,
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
bool near_zero(wide r, wide big, wide i0, wide i1, wide small, wide j0,
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
bool rows_meet(const lm_rows& a, const lm_rows& b, int64_t tokens,
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

bool vector_rows(const lm_rows& r, int es) {
  const int64_t v = 16 / es;
  return addr(r.data) % 16 == 0 && r.token_stride % v == 0 &&
         r.head_stride % v == 0;
}

Rows rows_of(const lm_rows& r) {
  Rows o;
  o.p = static_cast<char*>(r.data);
  o.ts = r.token_stride;
  o.hs = r.head_stride;
  return o;
}

Turn check_turn(const lm_rope_plan& rope, const void* positions,
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
bool pages_meet(const lm_kv_plan& p, const lm_kv_cache* c, const Range& all,
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
CacheArgs check_cache(const lm_kv_plan& p, const lm_kv_cache* c,
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

// Pages, tokens and sequences as the kernels count them.
void check_table(const lm_kv_plan& p, const int32_t* table, int64_t stride,
                 int seqs, int64_t max_pages, const int32_t* lens) {
  need((table || max_pages == 0) && lens && seqs >= 0 && max_pages >= 0 &&
       stride >= 0 && addr(table) % 4 == 0 && addr(lens) % 4 == 0);
  need(seqs <= 1 || stride >= max_pages);
  // key numbers, rounded up to whole tiles, fit 32 bits
  need(mul_chk(max_pages, p.page_tokens) < (int64_t(1) << 31) - 4096,
       LM_E_OVERFLOW);
}

}  // namespace
}  // namespace lm

using lm::need;

extern "C" {

int lm_rope_plan_create(int head_dim, int rotary_dim, int interleaved,
                        double base, int scaling, double factor,
                        int64_t original_positions, double beta_fast,
                        double beta_slow, lm_rope_plan** out) {
  if (out) *out = nullptr;
  return lm::guarded([&] {
    need(out && head_dim >= 2 && head_dim <= lm::kRopeMaxDim &&
         rotary_dim >= 2 && rotary_dim <= head_dim && rotary_dim % 2 == 0);
    need(std::isfinite(base) && base > 1 && std::isfinite(factor) &&
         factor >= 1);
    need(scaling >= LM_ROPE_NONE && scaling <= LM_ROPE_YARN);
    lm_rope_plan p;
    p.head_dim = head_dim;
    p.rotary = rotary_dim;
    p.inter = interleaved != 0;
    double b = base;
    if (scaling == LM_ROPE_NTK) {
      need(rotary_dim > 2);
      b = base * std::pow(factor, double(rotary_dim) / (rotary_dim - 2));
      need(std::isfinite(b));
    }
    if (scaling == LM_ROPE_YARN) {
      need(original_positions >= 1 && std::isfinite(beta_fast) &&
           std::isfinite(beta_slow) && beta_slow >= 0 &&
           beta_fast > beta_slow);
      p.amplitude = 0.1 * std::log(factor) + 1;
    }
    const double two_pi = 2 * std::acos(-1.0);
    for (int i = 0; i < rotary_dim / 2; ++i) {
      double f = std::pow(b, -2.0 * i / rotary_dim);
      if (scaling == LM_ROPE_LINEAR) f /= factor;
      if (scaling == LM_ROPE_YARN) {
        const double turns = double(original_positions) * f / two_pi;
        double g = (turns - beta_slow) / (beta_fast - beta_slow);
        g = g < 0 ? 0 : g > 1 ? 1 : g;
        f = (1 - g) * f / factor + g * f;
      }
      p.freq.push_back(f);
    }
    *out = new lm_rope_plan(std::move(p));
  });
}

int lm_rope_plan_frequencies(const lm_rope_plan* plan, double* freqs, int cap,
                             double* amplitude) {
  return lm::guarded([&] {
    need(plan);
    if (freqs) {
      need(cap >= int(plan->freq.size()), LM_E_BUFFER);
      std::memcpy(freqs, plan->freq.data(), plan->freq.size() * 8);
    }
    if (amplitude) *amplitude = plan->amplitude;
  });
}

int lm_rope_table(const lm_rope_plan* plan, float* table, int64_t rows,
                  int64_t capacity, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && rows >= 0);
    if (rows == 0) return;
    need(table && lm::addr(table) % 4 == 0);
    need(lm::mul_chk(rows, plan->rotary) <= capacity, LM_E_CAPACITY);
    lm::RopeTableArgs a;
    a.table = table;
    a.rows = rows;
    a.half = plan->rotary / 2;
    a.amplitude = plan->amplitude;
    std::memcpy(a.freq, plan->freq.data(), plan->freq.size() * 8);
    rc = lm::launch_rope_table(a, cuda_stream);
  });
  return checked != LM_OK ? checked : rc;
}

int lm_rope(const lm_rope_plan* plan, int elem, const lm_rows* x,
            const lm_rows* out, int64_t tokens, int heads,
            const void* positions, int position_bytes, const float* table,
            int64_t table_rows, int inverse, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && elem >= LM_BF16 && elem <= LM_F32 && tokens >= 0 &&
         heads >= 0);
    if (tokens == 0 || heads == 0) return;
    const int es = lm::elem_size(elem);
    const lm::Range rx =
        lm::check_rows(x, tokens, heads, plan->head_dim, es, false);
    const lm::Range ro =
        lm::check_rows(out, tokens, heads, plan->head_dim, es, true);
    const bool in_place = x->data == out->data &&
                          (tokens == 1 || x->token_stride == out->token_stride) &&
                          (heads == 1 || x->head_stride == out->head_stride);
    need(in_place || !rx.meets(ro), LM_E_OVERLAP);
    lm::RopeArgs a;
    a.turn = lm::check_turn(*plan, positions, position_bytes, table,
                            table_rows, inverse);
    a.x = lm::rows_of(*x);
    a.out = lm::rows_of(*out);
    a.heads = uint32_t(heads);
    a.dim = plan->head_dim;
    a.copy_rest = !in_place;
    // 16-byte accesses: the chunks of both tensors and of the table's rows
    // (cosines and sines each) are aligned, and no chunk straddles the
    // rotated part's halves or its end
    const int v = 16 / es;
    a.vec = lm::vector_rows(*x, es) && lm::vector_rows(*out, es) &&
            lm::addr(table) % 16 == 0 && plan->head_dim % v == 0 &&
            plan->rotary % 8 == 0 &&
            (plan->inter ? plan->rotary : plan->rotary / 2) % v == 0;
    a.status = lm::device_status_word();
    // 32-bit unit numbers: at most head_dim units a row
    const int64_t unit_rows = (int64_t(1) << 31) / plan->head_dim;
    const int64_t most = unit_rows / heads > 0 ? unit_rows / heads : 0;
    need(most > 0, LM_E_OVERFLOW);
    const lm::RopeArgs whole = a;
    for (int64_t t = 0; t < tokens && rc == LM_OK; t += most) {
      a = whole;
      a.tokens = uint32_t(tokens - t < most ? tokens - t : most);
      a.x.p += t * a.x.ts * es;
      a.out.p += t * a.out.ts * es;
      a.turn.pos = static_cast<const char*>(positions) + t * position_bytes;
      rc = lm::launch_rope(a, elem, cuda_stream);
    }
  });
  return checked != LM_OK ? checked : rc;
}

void lm_rope_plan_destroy(lm_rope_plan* plan) { delete plan; }

int lm_kv_plan_create(const lm_layout* page, int64_t page_stride, int elem,
                      int store, lm_kv_plan** out) {
  if (out) *out = nullptr;
  return lm::guarded([&] {
    need(page && out && (elem == LM_BF16 || elem == LM_F16) &&
         store >= LM_KV_SAME && store <= LM_KV_INT8 && page_stride >= 0);
    need(!page->swz.on(), LM_E_NOT_REPRESENTABLE);
    need(page->leaves.size() == 3 && page->mode_leaves.size() == 3 &&
         page->size > 0);
    const lm::Leaf t = page->leaves[0], h = page->leaves[1],
                   d = page->leaves[2];
    need(t.e < (int64_t(1) << 24) && h.e < (int64_t(1) << 16) &&
         d.e <= lm::kKvMaxDim);
    need(d.d == 1, LM_E_NOT_REPRESENTABLE);
    need(lm::affine_injective(page->leaves), LM_E_NOT_INJECTIVE);
    lm_kv_plan p;
    p.held = store == LM_KV_SAME ? 2 : 1;
    const int64_t v = 16 / p.held;
    need(d.e % v == 0 && (t.e == 1 || t.d % v == 0) &&
             (h.e == 1 || h.d % v == 0) && page_stride % v == 0,
         LM_E_NOT_REPRESENTABLE);
    p.page_tokens = t.e;
    p.heads = h.e;
    p.dim = d.e;
    p.token_stride = t.e > 1 ? t.d : 0;
    p.head_stride = h.e > 1 ? h.d : 0;
    p.page_cosize = page->cosize;
    p.page_stride = page_stride
                        ? page_stride
                        : lm::add_chk(page->cosize, v - 1) / v * v;
    need(p.page_stride >= page->cosize);
    p.elem = elem;
    p.store = store;
    static const char* const stores[] = {"same", "e4m3", "int8"};
    p.describe = std::string("{\"page_tokens\": ") +
                 std::to_string(p.page_tokens) +
                 ", \"heads\": " + std::to_string(p.heads) +
                 ", \"dim\": " + std::to_string(p.dim) + ", \"page\": \"" +
                 lm::to_string(*page) +
                 "\", \"page_stride\": " + std::to_string(p.page_stride) +
                 ", \"elem\": \"" + (elem == LM_BF16 ? "bf16" : "f16") +
                 "\", \"store\": \"" + stores[store] +
                 "\", \"held_bytes\": " + std::to_string(p.held) + "}";
    *out = new lm_kv_plan(std::move(p));
  });
}

int lm_kv_plan_describe(const lm_kv_plan* plan, char* buf, size_t cap) {
  if (!plan || (!buf && cap)) return LM_E_INVALID;
  if (cap == 0) return LM_E_BUFFER;
  const std::string& s = plan->describe;
  const size_t n = s.size() < cap - 1 ? s.size() : cap - 1;
  std::memcpy(buf, s.data(), n);
  buf[n] = '\0';
  return s.size() + 1 > cap ? LM_E_BUFFER : LM_OK;
}

int lm_kv_write(const lm_kv_plan* plan, const lm_kv_cache* cache,
                const lm_rows* k, const lm_rows* v, int64_t tokens,
                const int64_t* slots, const lm_rope_plan* rope,
                const void* positions, int position_bytes, const float* table,
                int64_t table_rows, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && tokens >= 0);
    lm::CacheRanges held;
    lm::KvWriteArgs a;
    a.c = lm::check_cache(*plan, cache, &held);
    if (tokens == 0) return;
    need(slots && lm::addr(slots) % 8 == 0);
    for (const lm_rows* r : {k, v}) {
      const lm::Range ri =
          lm::check_rows(r, tokens, plan->heads, plan->dim, 2, false);
      need(!held.meet(ri), LM_E_OVERLAP);
    }
    if (rope) {
      need(rope->head_dim == plan->dim);
      a.turn = lm::check_turn(*rope, positions, position_bytes, table,
                              table_rows, 0);
      a.table16 = lm::addr(table) % 16 == 0 && rope->rotary % 8 == 0;
    }
    a.k = lm::rows_of(*k);
    a.v = lm::rows_of(*v);
    a.heads_div = lm::make_fastdiv(uint32_t(plan->heads));
    a.vec = lm::vector_rows(*k, 2) && lm::vector_rows(*v, 2);
    a.status = lm::device_status_word();
    const int64_t most = (int64_t(1) << 26) / plan->heads;
    const lm::KvWriteArgs whole = a;
    for (int64_t t = 0; t < tokens && rc == LM_OK; t += most) {
      a = whole;
      a.tokens = uint32_t(tokens - t < most ? tokens - t : most);
      a.k.p += t * a.k.ts * 2;
      a.v.p += t * a.v.ts * 2;
      a.slots = slots + t;
      if (rope)
        a.turn.pos = static_cast<const char*>(positions) + t * position_bytes;
      rc = lm::launch_kv_write(a, plan->elem, plan->store, cuda_stream);
    }
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_read(const lm_kv_plan* plan, const lm_kv_cache* cache,
               const int32_t* page_table, int64_t table_stride, int seqs,
               int64_t max_pages, const int32_t* lens, const int32_t* starts,
               int out_elem, const lm_rows* k_out, const lm_rows* v_out,
               int64_t rows, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && rows >= 0 && out_elem >= LM_BF16 && out_elem <= LM_F32);
    lm::CacheRanges held;
    lm::KvReadArgs a;
    a.c = lm::check_cache(*plan, cache, &held);
    if (rows == 0 || seqs == 0 || max_pages == 0) return;
    lm::check_table(*plan, page_table, table_stride, seqs, max_pages, lens);
    need(starts && lm::addr(starts) % 4 == 0);
    need(rows < (int64_t(1) << 31), LM_E_OVERFLOW);
    const int es = lm::elem_size(out_elem);
    lm::Range o[2];
    const lm_rows* outs[2] = {k_out, v_out};
    for (int i = 0; i < 2; ++i) {
      o[i] = lm::check_rows(outs[i], rows, plan->heads, plan->dim, es, true);
      need(!held.meet(o[i]), LM_E_OVERLAP);
    }
    need(!o[0].meets(o[1]) ||
             !lm::rows_meet(*k_out, *v_out, rows, plan->heads, plan->dim, es),
         LM_E_OVERLAP);
    a.k = lm::rows_of(*k_out);
    a.v = lm::rows_of(*v_out);
    a.table = page_table;
    a.table_stride = table_stride;
    a.max_tokens = max_pages * plan->page_tokens;
    a.lens = lens;
    a.starts = starts;
    a.seqs = seqs;
    a.rows = rows;
    a.vec = lm::vector_rows(*k_out, es) && lm::vector_rows(*v_out, es);
    a.status = lm::device_status_word();
    rc = lm::launch_kv_read(a, plan->elem, plan->store, out_elem,
                            cuda_stream);
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_attend_workspace(const lm_kv_plan* plan, int seqs, int heads_q,
                           int64_t* bytes) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && bytes && seqs >= 0 && heads_q >= 1 &&
         heads_q <= (1 << 20) && heads_q % plan->heads == 0);
    rc = lm::attend_workspace(plan->store, int(plan->dim),
                              int(heads_q / plan->heads), bytes);
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_attend(const lm_kv_plan* plan, const lm_kv_cache* cache,
                 const lm_rows* q, const lm_rows* out, int seqs, int heads_q,
                 const int32_t* page_table, int64_t table_stride,
                 int64_t max_pages, const int32_t* lens, int64_t window,
                 float scale, float* lse, void* workspace,
                 int64_t workspace_bytes, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && seqs >= 0 && heads_q >= 1 && heads_q % plan->heads == 0 &&
         heads_q <= (1 << 20) && std::isfinite(scale) && window >= 0);
    lm::CacheRanges held;
    lm::KvAttendArgs a;
    a.c = lm::check_cache(*plan, cache, &held);
    if (seqs == 0) return;
    lm::check_table(*plan, page_table, table_stride, seqs, max_pages, lens);
    const lm::Range rq =
        lm::check_rows(q, seqs, heads_q, plan->dim, 2, false);
    const lm::Range ro =
        lm::check_rows(out, seqs, heads_q, plan->dim, 2, true);
    const bool in_place =
        q->data == out->data &&
        (seqs == 1 || q->token_stride == out->token_stride) &&
        (heads_q == 1 || q->head_stride == out->head_stride);
    need(in_place || !rq.meets(ro), LM_E_OVERLAP);
    need(!held.meet(ro), LM_E_OVERLAP);
    need(lse == nullptr || lm::addr(lse) % 4 == 0);
    lm::Range rl;
    if (lse) {
      rl = {lm::addr(lse),
            lm::addr(lse) + uintptr_t(int64_t(seqs) * heads_q * 4)};
      need(!held.meet(rl) && !rl.meets(rq) && !rl.meets(ro), LM_E_OVERLAP);
    }
    a.q = lm::rows_of(*q);
    a.out = lm::rows_of(*out);
    a.table = page_table;
    a.table_stride = table_stride;
    a.max_tokens = max_pages * plan->page_tokens;
    a.lens = lens;
    a.seqs = seqs;
    a.heads_q = heads_q;
    a.group = int(heads_q / plan->heads);
    a.elem = plan->elem;
    a.window = window;
    a.scale = scale;
    a.lse = lse;
    a.ws = workspace;
    a.status = lm::device_status_word();
    int64_t want = 0;
    rc = lm::attend_workspace(plan->store, int(plan->dim), a.group, &want);
    if (rc != LM_OK) return;
    need(want == 0 || (workspace && lm::addr(workspace) % 16 == 0));
    need(workspace_bytes >= want, LM_E_CAPACITY);
    const lm::Range rw = {lm::addr(workspace),
                          lm::addr(workspace) + uintptr_t(want)};
    need(!held.meet(rw) && !rw.meets(rq) && !rw.meets(ro) && !rw.meets(rl),
         LM_E_OVERLAP);
    rc = lm::launch_kv_attend(a, plan->store, cuda_stream);
  });
  return checked != LM_OK ? checked : rc;
}

void lm_kv_plan_destroy(lm_kv_plan* plan) { delete plan; }

}  // extern "C"
