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
  const float *scores = nullptr, *lse2 = nullptr;
  float* weights = nullptr;
  unsigned int* status = nullptr;
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
  FastDiv page_div;               // division by page_tokens
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

int launch_kv_weigh(const KvWeighArgs& a, void* stream);
int launch_kv_bound(const KvBoundArgs& a, int elem, int store, void* stream);
int launch_kv_select(const KvSelectArgs& a, int elem, void* stream);
int launch_kv_evict(const KvEvictArgs& a, void* stream);

}  // namespace lm
