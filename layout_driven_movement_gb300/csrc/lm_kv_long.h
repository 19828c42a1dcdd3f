// Argument blocks of the cache's operators for long contexts: accumulated
// weights, page bounds, the choice of pages, eviction, shared prefixes.
#pragma once

#include "lm_kv.h"

namespace lm {

// Scores into weights: the second launch of an attention that weighs.
struct KvWeighArgs {
  CacheArgs c;
  const int32_t* table = nullptr;
  int64_t table_stride = 0, table_head = 0, max_tokens = 0, window = 0;
  const int32_t* lens = nullptr;
  int32_t seqs = 0, group = 1;
  const float *scores = nullptr, *norms = nullptr;  // of KvAttendArgs
  float* weights = nullptr;
};

struct KvBoundArgs {
  CacheArgs c;
  const int32_t *pages = nullptr, *counts = nullptr;
  int64_t n = 0;
  int8_t* bounds = nullptr;       // [pages, heads, 2, dim]
  float* scale = nullptr;         // [pages, heads]
  FastDiv heads_div;
  unsigned int* status = nullptr;
};

struct KvSelectArgs {
  Rows q;
  int64_t pages = 0;
  uint32_t heads = 1;
  int32_t page_tokens = 1;
  int32_t dim = 0, group = 1, seqs = 0;
  int32_t q16 = 0;                // the queries allow 16-byte loads
  const int8_t* bounds = nullptr;
  const float* bound_scale = nullptr;
  const int32_t* table = nullptr;
  int64_t table_stride = 0, max_pages = 0;
  const int32_t* lens = nullptr;
  int32_t keep = 1, first = 0, last = 1;
  int32_t *selected = nullptr, *selected_lens = nullptr;
  float* scores = nullptr;        // [seqs, heads, max_pages]
  unsigned int* status = nullptr;
};

struct KvEvictArgs {
  CacheArgs c;
  float* weights = nullptr;       // [pages, heads, page_tokens]
  const int32_t* table = nullptr;
  int64_t table_stride = 0, max_tokens = 0;
  const int32_t* lens = nullptr;
  const int32_t* kept_table = nullptr;
  int64_t kept_stride = 0;
  int32_t* kept_lens = nullptr;
  int32_t seqs = 0, keep = 1, recent = 0;
  int32_t* list = nullptr;        // [seqs, heads, keep]
  uint32_t chunks = 1;            // 16-byte units of a held row
  FastDiv chunk_div;
  unsigned int* status = nullptr;
};

// Attention of groups of sequences over the pages that each group shares, and
// its join with that over each sequence's own.
struct KvSharedArgs {
  CacheArgs c;
  Rows q;
  const int32_t* table = nullptr;         // [groups, pages]
  int64_t table_stride = 0, max_tokens = 0;
  const int32_t *lens = nullptr, *starts = nullptr;
  int32_t groups = 0, seqs = 0, group = 1, heads_q = 1;
  int32_t q16 = 0;                        // the queries allow 16-byte loads
  int32_t elem = LM_BF16;
  float scale = 1;
  // rows that one block finishes: up to two states (m, l) and means each, [2,
  // seqs, heads_q] and [2, seqs, heads_q, dim]
  float *state = nullptr, *mean = nullptr;
  float* parts = nullptr;                 // two for each block
  // Where each row's pieces are, [seqs, heads_q] of 4: how many blocks have one
  // (0: none), the part that the first of them wrote, the second's (the others'
  // two on each), and the row's place there, + 65536 where a second state of
  // the row lies 128 places behind.  One block: its pieces are in `state`.
  int32_t* pieces = nullptr;
  unsigned int* status = nullptr;
};

struct KvJoinArgs {
  KvSharedArgs s;
  Rows out;
  const float *state = nullptr, *mean = nullptr;    // of each one's own pages
  float* lse = nullptr;
};

// The tiles of a shared-prefix kernel for rows of `dim` elements.
LM_HD int shared_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }
LM_HD int shared_keys(int dim) { return dim > 128 ? 64 : 128; }
LM_HD int shared_rows(int dim) { return dim > 128 ? 128 : 256; }
// Floats of a part: (m, l) of its rows, then their means.
LM_HD int64_t shared_part(int dim) {
  return int64_t(shared_rows(dim)) * (shared_dim(dim) + 2);
}

int launch_kv_shared(const KvSharedArgs& a, int store, void* stream);
int launch_kv_join(const KvJoinArgs& a, void* stream);
int launch_shared_same(const KvSharedArgs& a, void* stream);
int launch_shared_e4m3(const KvSharedArgs& a, void* stream);
int launch_shared_int8(const KvSharedArgs& a, void* stream);
int launch_kv_weigh(const KvWeighArgs& a, void* stream);
int launch_kv_bound(const KvBoundArgs& a, int elem, int store, void* stream);
int launch_kv_select(const KvSelectArgs& a, int elem, void* stream);
int launch_kv_evict(const KvEvictArgs& a, void* stream);

}  // namespace lm
