// The cache's attention and its operators for long contexts, host side:
// argument checks and the hand-over to the kernels' launchers.
#include "lm_kv_long.h"

#include "lm_kv_check.h"

using lm::need;

namespace lm {
namespace {

int64_t whole(int64_t bytes) { return add_chk(bytes, 255) / 256 * 256; }

// What an attention that weighs keeps in its workspace, behind the plain
// attention's: references and sums of all rows, then the scores.
struct WeighSpace {
  int64_t norms = 0, scores = 0, bytes = 0;
};
WeighSpace weigh_space(int64_t plain, int64_t rows, int64_t max_tokens) {
  WeighSpace s;
  s.norms = whole(plain);
  s.scores = add_chk(s.norms, whole(mul_chk(rows, 8)));
  s.bytes = add_chk(s.scores, mul_chk(mul_chk(rows, max_tokens), 4));
  return s;
}

// What an attention over shared prefixes keeps behind the plain attention's:
// each row's state over its own pages, up to two over its group's, and the
// parts of rows that several blocks share.
struct SharedSpace {
  int64_t state = 0, mean = 0, shared_state = 0, shared_mean = 0, pieces = 0,
          parts = 0, bytes = 0;
};
SharedSpace shared_space(int64_t plain, int64_t rows, int dim, int sms) {
  const int64_t states = whole(mul_chk(rows, 8));
  const int64_t means = whole(mul_chk(rows, int64_t(dim) * 4));
  SharedSpace s;
  s.state = whole(plain);
  s.mean = add_chk(s.state, states);
  s.shared_state = add_chk(s.mean, means);
  s.shared_mean = add_chk(s.shared_state, 2 * states);
  s.pieces = add_chk(s.shared_mean, mul_chk(means, 2));
  s.parts = add_chk(s.pieces, 2 * states);
  s.bytes = add_chk(s.parts, 2 * int64_t(sms) * shared_part(dim) * 4);
  return s;
}

Range range_of(const void* p, int64_t bytes) {
  return {addr(p), addr(p) + uintptr_t(bytes)};
}

void check_workspace(const void* ws, int64_t have, int64_t want) {
  need(want == 0 || (ws && addr(ws) % 16 == 0));
  need(have >= want, LM_E_CAPACITY);
}

void check_queries(const lm_kv_plan& p, int seqs, int heads_q) {
  need(seqs >= 0 && heads_q >= 1 && heads_q <= (1 << 20) &&
       heads_q % p.heads == 0);
}

// The bytes that an attention's queries, outputs and lse (empty: none) span.
struct AttendRanges {
  Range q, out, lse;
  bool meet(const Range& o) const {
    return o.meets(q) || o.meets(out) || o.meets(lse);
  }
};
AttendRanges check_attend(const lm_kv_plan& p, const CacheRanges& held,
                          const lm_rows* q, const lm_rows* out, int seqs,
                          int heads_q, const float* lse) {
  AttendRanges r;
  r.q = check_rows(q, seqs, heads_q, p.dim, 2, false);
  r.out = check_rows(out, seqs, heads_q, p.dim, 2, true);
  const bool in_place = q->data == out->data &&
                        (seqs == 1 || q->token_stride == out->token_stride) &&
                        (heads_q == 1 || q->head_stride == out->head_stride);
  need(in_place || !r.q.meets(r.out), LM_E_OVERLAP);
  need(!held.meet(r.out), LM_E_OVERLAP);
  need(lse == nullptr || addr(lse) % 4 == 0);
  if (lse) {
    r.lse = range_of(lse, int64_t(seqs) * heads_q * 4);
    need(!held.meet(r.lse) && !r.lse.meets(r.q) && !r.lse.meets(r.out),
         LM_E_OVERLAP);
  }
  return r;
}

}  // namespace
}  // namespace lm

extern "C" {

int lm_kv_attend_workspace(const lm_kv_plan* plan, int seqs, int heads_q,
                           int64_t* bytes) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && bytes);
    lm::check_queries(*plan, seqs, heads_q);
    rc = lm::attend_workspace(plan->store, int(plan->dim),
                              int(heads_q / plan->heads), bytes);
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_attend_weigh_workspace(const lm_kv_plan* plan, int seqs,
                                 int heads_q, int64_t max_pages,
                                 int64_t* bytes) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && bytes && max_pages >= 0);
    lm::check_queries(*plan, seqs, heads_q);
    int64_t plain = 0;
    rc = lm::attend_workspace(plan->store, int(plan->dim),
                              int(heads_q / plan->heads), &plain);
    if (rc != LM_OK) return;
    *bytes = lm::weigh_space(plain, int64_t(seqs) * heads_q,
                             lm::mul_chk(max_pages, plan->page_tokens))
                 .bytes;
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_attend(const lm_kv_plan* plan, const lm_kv_cache* cache,
                 const lm_rows* q, const lm_rows* out, int seqs, int heads_q,
                 const int32_t* page_table, int64_t table_stride,
                 int64_t max_pages, const int32_t* lens, int64_t window,
                 float scale, float* lse, void* workspace,
                 int64_t workspace_bytes, void* cuda_stream) {
  return lm_kv_attend_weigh(plan, cache, q, out, seqs, heads_q, page_table,
                            table_stride, 0, max_pages, lens, window, scale,
                            lse, nullptr, 0, workspace, workspace_bytes,
                            cuda_stream);
}

int lm_kv_attend_weigh(const lm_kv_plan* plan, const lm_kv_cache* cache,
                       const lm_rows* q, const lm_rows* out, int seqs,
                       int heads_q, const int32_t* page_table,
                       int64_t table_stride, int64_t head_stride,
                       int64_t max_pages, const int32_t* lens, int64_t window,
                       float scale, float* lse, float* weights,
                       int64_t weights_capacity, void* workspace,
                       int64_t workspace_bytes, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && std::isfinite(scale) && window >= 0 && head_stride >= 0);
    lm::check_queries(*plan, seqs, heads_q);
    lm::CacheRanges held;
    lm::KvAttendArgs a;
    a.c = lm::check_cache(*plan, cache, &held);
    if (seqs == 0) return;
    lm::check_table(*plan, page_table, table_stride, seqs, max_pages, lens);
    const int64_t rows = int64_t(seqs) * heads_q;
    const lm::AttendRanges r =
        lm::check_attend(*plan, held, q, out, seqs, heads_q, lse);
    lm::Range rw;
    if (weights) {
      need(lm::addr(weights) % 4 == 0);
      const int64_t n = lm::mul_chk(
          cache->pages, lm::mul_chk(plan->heads, plan->page_tokens));
      need(n <= weights_capacity, LM_E_CAPACITY);
      rw = lm::range_of(weights, lm::mul_chk(n, 4));
      need(!held.meet(rw) && !r.meet(rw), LM_E_OVERLAP);
    }
    a.q = lm::rows_of(*q);
    a.out = lm::rows_of(*out);
    a.table = page_table;
    a.table_stride = table_stride;
    a.table_head = plan->heads > 1 ? head_stride : 0;
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
    lm::WeighSpace space;
    if (weights) {
      space = lm::weigh_space(want, rows, a.max_tokens);
      want = space.bytes;
    }
    lm::check_workspace(workspace, workspace_bytes, want);
    const lm::Range rs = lm::range_of(workspace, want);
    need(!held.meet(rs) && !r.meet(rs) && !rs.meets(rw), LM_E_OVERLAP);
    if (weights) {
      char* const ws = static_cast<char*>(workspace);
      a.norms = reinterpret_cast<float*>(ws + space.norms);
      a.scores = reinterpret_cast<float*>(ws + space.scores);
    }
    rc = lm::launch_kv_attend(a, plan->store, cuda_stream);
    if (rc != LM_OK || !weights) return;
    lm::KvWeighArgs w;
    w.c = a.c;
    w.table = a.table;
    w.table_stride = a.table_stride;
    w.table_head = a.table_head;
    w.max_tokens = a.max_tokens;
    w.window = window;
    w.lens = lens;
    w.seqs = seqs;
    w.group = a.group;
    w.scores = a.scores;
    w.norms = a.norms;
    w.weights = weights;
    rc = lm::launch_kv_weigh(w, cuda_stream);
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_attend_shared_workspace(const lm_kv_plan* plan, int seqs,
                                  int heads_q, int64_t* bytes) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && bytes);
    lm::check_queries(*plan, seqs, heads_q);
    int64_t plain = 0;
    rc = lm::attend_workspace(plan->store, int(plan->dim),
                              int(heads_q / plan->heads), &plain);
    int dev = 0, sms = 0;
    if (rc == LM_OK) rc = lm::kv_device(&dev, &sms);
    if (rc != LM_OK) return;
    *bytes = lm::shared_space(plain, int64_t(seqs) * heads_q, int(plan->dim),
                              sms)
                 .bytes;
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_attend_shared(
    const lm_kv_plan* plan, const lm_kv_cache* cache, const lm_rows* q,
    const lm_rows* out, int seqs, int heads_q, const int32_t* shared_table,
    int64_t shared_stride, int groups, int64_t max_shared_pages,
    const int32_t* shared_lens, const int32_t* starts,
    const int32_t* page_table, int64_t table_stride, int64_t max_pages,
    const int32_t* lens, float scale, float* lse, void* workspace,
    int64_t workspace_bytes, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && std::isfinite(scale));
    lm::check_queries(*plan, seqs, heads_q);
    lm::CacheRanges held;
    lm::KvAttendArgs a;
    a.c = lm::check_cache(*plan, cache, &held);
    if (seqs == 0) return;
    lm::check_table(*plan, page_table, table_stride, seqs, max_pages, lens);
    need(groups >= 0);
    if (groups > 0) {
      lm::check_table(*plan, shared_table, shared_stride, groups,
                      max_shared_pages, shared_lens);
      need(starts && lm::addr(starts) % 4 == 0);
    }
    const int64_t rows = lm::mul_chk(seqs, heads_q);
    need(rows < (int64_t(1) << 31) - 4096, LM_E_OVERFLOW);
    const lm::AttendRanges r =
        lm::check_attend(*plan, held, q, out, seqs, heads_q, lse);
    // rows of codes are counted in 16 bytes, in 32 bits
    need(plan->store == LM_KV_SAME ||
             lm::mul_chk(cache->pages, plan->page_stride) <
                 (int64_t(1) << 36) - 4096,
         LM_E_OVERFLOW);
    const int group = int(heads_q / plan->heads);
    int64_t plain = 0;
    int dev = 0, sms = 0;
    rc = lm::attend_workspace(plan->store, int(plan->dim), group, &plain);
    if (rc == LM_OK) rc = lm::kv_device(&dev, &sms);
    if (rc != LM_OK) return;
    const lm::SharedSpace space =
        lm::shared_space(plain, rows, int(plan->dim), sms);
    lm::check_workspace(workspace, workspace_bytes, space.bytes);
    const lm::Range rs = lm::range_of(workspace, space.bytes);
    need(!held.meet(rs) && !r.meet(rs), LM_E_OVERLAP);
    char* const ws = static_cast<char*>(workspace);
    auto floats = [&](int64_t at) { return reinterpret_cast<float*>(ws + at); };
    a.q = lm::rows_of(*q);
    a.out = lm::rows_of(*out);
    a.table = page_table;
    a.table_stride = table_stride;
    a.max_tokens = max_pages * plan->page_tokens;
    a.lens = lens;
    a.seqs = seqs;
    a.heads_q = heads_q;
    a.group = group;
    a.elem = plan->elem;
    a.scale = scale;
    a.ws = workspace;
    a.status = lm::device_status_word();
    if (groups == 0 || max_shared_pages == 0) {
      a.lse = lse;
      rc = lm::launch_kv_attend(a, plan->store, cuda_stream);
      return;
    }
    lm::KvJoinArgs j;
    lm::KvSharedArgs& s = j.s;
    s.c = a.c;
    s.q = a.q;
    s.table = shared_table;
    s.table_stride = shared_stride;
    s.max_tokens = max_shared_pages * plan->page_tokens;
    s.lens = shared_lens;
    s.starts = starts;
    s.groups = groups;
    s.seqs = seqs;
    s.group = group;
    s.heads_q = heads_q;
    s.q16 = lm::vector_rows(*q, 2);
    s.elem = plan->elem;
    s.scale = scale;
    s.state = floats(space.shared_state);
    s.mean = floats(space.shared_mean);
    s.parts = floats(space.parts);
    s.status = a.status;
    s.pieces = reinterpret_cast<int32_t*>(ws + space.pieces);
    a.state = floats(space.state);
    a.mean = floats(space.mean);
    a.pieces = s.pieces;
    // (this one first: it writes that rows have no pieces)
    rc = lm::launch_kv_attend(a, plan->store, cuda_stream);
    if (rc == LM_OK) rc = lm::launch_kv_shared(s, plan->store, cuda_stream);
    if (rc != LM_OK) return;
    j.out = a.out;
    j.state = a.state;
    j.mean = a.mean;
    j.lse = lse;
    rc = lm::launch_kv_join(j, cuda_stream);
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_bound(const lm_kv_plan* plan, const lm_kv_cache* cache,
                const int32_t* pages, const int32_t* counts, int64_t n,
                const lm_kv_bounds* bounds, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && n >= 0);
    lm::CacheRanges held;
    lm::KvBoundArgs a;
    a.c = lm::check_cache(*plan, cache, &held);
    const lm::BoundRanges r = lm::check_bounds(*plan, cache->pages, bounds);
    need(!held.meet(r.data) && !held.meet(r.scale), LM_E_OVERLAP);
    if (n == 0) return;
    need(pages && counts && lm::addr(pages) % 4 == 0 &&
         lm::addr(counts) % 4 == 0);
    const lm::Range rp = lm::range_of(pages, lm::mul_chk(n, 4));
    const lm::Range rc_ = lm::range_of(counts, n * 4);
    need(!r.data.meets(rp) && !r.data.meets(rc_) && !r.scale.meets(rp) &&
             !r.scale.meets(rc_),
         LM_E_OVERLAP);
    a.bounds = bounds->data;
    a.scale = bounds->scale;
    a.heads_div = lm::make_fastdiv(uint32_t(plan->heads));
    a.status = lm::device_status_word();
    const int64_t most = (int64_t(1) << 30) / plan->heads;
    for (int64_t i = 0; i < n && rc == LM_OK; i += most) {
      a.pages = pages + i;
      a.counts = counts + i;
      a.n = n - i < most ? n - i : most;
      rc = lm::launch_kv_bound(a, plan->elem, plan->store, cuda_stream);
    }
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_select_workspace(const lm_kv_plan* plan, int seqs,
                           int64_t max_pages, int64_t* bytes) {
  return lm::guarded([&] {
    need(plan && bytes && seqs >= 0 && max_pages >= 0);
    *bytes = lm::mul_chk(
        lm::mul_chk(lm::mul_chk(seqs, plan->heads), max_pages), 4);
  });
}

int lm_kv_select(const lm_kv_plan* plan, int64_t pages,
                 const lm_kv_bounds* bounds, const lm_rows* q, int seqs,
                 int heads_q, const int32_t* page_table, int64_t table_stride,
                 int64_t max_pages, const int32_t* lens, int keep, int first,
                 int last, int32_t* selected, int32_t* selected_lens,
                 void* workspace, int64_t workspace_bytes,
                 void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && pages >= 1 && first >= 0 && last >= 1 && keep >= 1 &&
         int64_t(first) + last <= keep);
    lm::check_queries(*plan, seqs, heads_q);
    const lm::BoundRanges r = lm::check_bounds(*plan, pages, bounds);
    if (seqs == 0) return;
    lm::check_table(*plan, page_table, table_stride, seqs, max_pages, lens);
    need(selected && selected_lens && lm::addr(selected) % 4 == 0 &&
         lm::addr(selected_lens) % 4 == 0);
    const lm::Range rq =
        lm::check_rows(q, seqs, heads_q, plan->dim, 2, false);
    const int64_t units = lm::mul_chk(seqs, plan->heads);
    need(units < (int64_t(1) << 30), LM_E_OVERFLOW);
    const lm::Range out[2] = {
        lm::range_of(selected, lm::mul_chk(lm::mul_chk(units, keep), 4)),
        lm::range_of(selected_lens, int64_t(seqs) * 4)};
    const int64_t table =
        lm::add_chk(lm::mul_chk(seqs - 1, table_stride), max_pages);
    const lm::Range in[5] = {rq, r.data, r.scale,
                             lm::range_of(page_table, lm::mul_chk(table, 4)),
                             lm::range_of(lens, int64_t(seqs) * 4)};
    const int64_t want = lm::mul_chk(lm::mul_chk(units, max_pages), 4);
    lm::check_workspace(workspace, workspace_bytes, want);
    const lm::Range rs = lm::range_of(workspace, want);
    need(!out[0].meets(out[1]) && !rs.meets(out[0]) && !rs.meets(out[1]),
         LM_E_OVERLAP);
    for (const lm::Range& i : in)
      need(!i.meets(out[0]) && !i.meets(out[1]) && !i.meets(rs),
           LM_E_OVERLAP);
    lm::KvSelectArgs a;
    a.q = lm::rows_of(*q);
    a.q16 = lm::vector_rows(*q, 2);
    a.pages = pages;
    a.heads = uint32_t(plan->heads);
    a.page_tokens = int32_t(plan->page_tokens);
    a.dim = int32_t(plan->dim);
    a.group = int(heads_q / plan->heads);
    a.seqs = seqs;
    a.bounds = bounds->data;
    a.bound_scale = bounds->scale;
    a.table = page_table;
    a.table_stride = table_stride;
    a.max_pages = max_pages;
    a.lens = lens;
    a.keep = keep;
    a.first = first;
    a.last = last;
    a.selected = selected;
    a.selected_lens = selected_lens;
    a.scores = static_cast<float*>(workspace);
    a.status = lm::device_status_word();
    rc = lm::launch_kv_select(a, plan->elem, cuda_stream);
  });
  return checked != LM_OK ? checked : rc;
}

int lm_kv_evict_workspace(const lm_kv_plan* plan, int seqs, int keep,
                          int64_t* bytes) {
  return lm::guarded([&] {
    need(plan && bytes && seqs >= 0 && keep >= 1);
    *bytes = lm::mul_chk(lm::mul_chk(lm::mul_chk(seqs, plan->heads), keep), 4);
  });
}

int lm_kv_evict(const lm_kv_plan* plan, const lm_kv_cache* cache,
                float* weights, int64_t weights_capacity,
                const int32_t* page_table, int64_t table_stride, int seqs,
                int64_t max_pages, const int32_t* lens,
                const int32_t* kept_table, int64_t kept_stride,
                int64_t kept_pages, int32_t* kept_lens, int keep, int recent,
                void* workspace, int64_t workspace_bytes, void* cuda_stream) {
  int rc = LM_OK;
  const int checked = lm::guarded([&] {
    need(plan && keep >= 1 && recent >= 0 && recent <= keep);
    lm::CacheRanges held;
    lm::KvEvictArgs a;
    a.c = lm::check_cache(*plan, cache, &held);
    if (seqs == 0) return;
    lm::check_table(*plan, page_table, table_stride, seqs, max_pages, lens);
    lm::check_table(*plan, kept_table, kept_stride, seqs, kept_pages, lens);
    need(weights && lm::addr(weights) % 4 == 0 && kept_lens &&
         lm::addr(kept_lens) % 4 == 0);
    a.max_tokens = max_pages * plan->page_tokens;
    need(kept_pages * plan->page_tokens >=
             (keep < a.max_tokens ? keep : a.max_tokens),
         LM_E_CAPACITY);
    const int64_t n = lm::mul_chk(
        cache->pages, lm::mul_chk(plan->heads, plan->page_tokens));
    need(n <= weights_capacity, LM_E_CAPACITY);
    const int64_t units = lm::mul_chk(seqs, plan->heads);
    need(units < (int64_t(1) << 29), LM_E_OVERFLOW);
    const int64_t want = lm::mul_chk(lm::mul_chk(units, keep), 4);
    lm::check_workspace(workspace, workspace_bytes, want);
    // what is written: rows and scales, weights, lengths and the workspace
    const lm::Range out[3] = {lm::range_of(weights, lm::mul_chk(n, 4)),
                              lm::range_of(kept_lens, int64_t(seqs) * 4),
                              lm::range_of(workspace, want)};
    for (int i = 0; i < 3; ++i) {
      need(!held.meet(out[i]), LM_E_OVERLAP);
      for (int j = 0; j < i; ++j) need(!out[i].meets(out[j]), LM_E_OVERLAP);
    }
    const lm::Range in[3] = {
        lm::range_of(page_table,
                     lm::mul_chk(lm::add_chk(lm::mul_chk(seqs - 1, table_stride),
                                             max_pages),
                                 4)),
        lm::range_of(kept_table,
                     lm::mul_chk(lm::add_chk(lm::mul_chk(seqs - 1, kept_stride),
                                             kept_pages),
                                 4)),
        lm::range_of(lens, int64_t(seqs) * 4)};
    for (int i = 0; i < 3; ++i)
      for (int j = 0; j < 3; ++j)
        need(!in[i].meets(out[j]) ||
                 (i == 2 && j == 1 && lens == kept_lens),
             LM_E_OVERLAP);
    a.weights = weights;
    a.table = page_table;
    a.table_stride = table_stride;
    a.lens = lens;
    a.kept_table = kept_table;
    a.kept_stride = kept_stride;
    a.kept_lens = kept_lens;
    a.seqs = seqs;
    a.keep = keep;
    a.recent = recent;
    a.list = static_cast<int32_t*>(workspace);
    a.chunks = uint32_t(plan->dim * plan->held / 16);
    a.chunk_div = lm::make_fastdiv(a.chunks);
    a.status = lm::device_status_word();
    rc = lm::launch_kv_evict(a, cuda_stream);
  });
  return checked != LM_OK ? checked : rc;
}

}  // extern "C"
