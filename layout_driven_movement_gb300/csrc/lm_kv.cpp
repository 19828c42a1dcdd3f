// The paged key-value cache and rotary positions, host side: plans, argument
// checks and the hand-over to the kernels' launchers.
#include "lm_kv_check.h"

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

void lm_kv_plan_destroy(lm_kv_plan* plan) { delete plan; }

}  // extern "C"
