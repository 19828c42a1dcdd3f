// Internal structures of the paged key-value cache and of rotary positions:
// the plans and the argument blocks handed to their kernels.
#pragma once

#include "lm_internal.h"

namespace lm {

constexpr int kKvMaxDim = 256;     // elements of a cached row at most
constexpr int kRopeMaxDim = 1024;  // elements of a rotated row at most

inline int elem_size(int elem) { return elem == LM_F32 ? 4 : 2; }

// A dense tensor of rows: strides in elements.
struct Rows {
  char* p = nullptr;
  int64_t ts = 0, hs = 0;
};

// What turns a row: the table and the positions (pos == nullptr: nothing).
struct Turn {
  const float* table = nullptr;
  const void* pos = nullptr;
  int64_t rows = 0;      // of the table
  int32_t pos64 = 0;     // positions are 64-bit
  int32_t rot = 0;       // rotated elements
  int32_t inter = 0;     // pairs (2i, 2i+1)
  int32_t inverse = 0;
};

struct RopeArgs {
  Rows x, out;
  Turn turn;
  uint32_t tokens = 0, heads = 0;
  int32_t dim = 0;
  int32_t vec = 0;       // 16-byte accesses
  int32_t copy_rest = 0; // the unrotated part is copied
  unsigned int* status = nullptr;
};

struct RopeTableArgs {
  float* table = nullptr;
  int64_t rows = 0;
  int32_t half = 0;
  float pad = 0;
  double amplitude = 1;
  double freq[kRopeMaxDim / 2];
};

// The cache as the kernels see it: strides in BYTES of the held elements,
// scales in floats at (page * heads + head) * page_tokens + token.
struct CacheArgs {
  char *k = nullptr, *v = nullptr;
  float *ks = nullptr, *vs = nullptr;
  int64_t page_b = 0, token_b = 0, head_b = 0;
  int64_t pages = 0;
  uint32_t page_tokens = 1, heads = 1;
  FastDiv page_div;      // division by page_tokens
  int32_t dim = 0;
};

struct KvWriteArgs {
  CacheArgs c;
  Rows k, v;
  Turn turn;
  const int64_t* slots = nullptr;
  uint32_t tokens = 0;
  FastDiv heads_div;
  int32_t vec = 0;       // the inputs allow 16-byte loads
  int32_t table16 = 0;   // and so does the rotary table
  unsigned int* status = nullptr;
};

struct KvReadArgs {
  CacheArgs c;
  Rows k, v;             // outputs
  const int32_t* table = nullptr;
  int64_t table_stride = 0, max_tokens = 0;
  const int32_t *lens = nullptr, *starts = nullptr;
  int32_t seqs = 0;
  int64_t rows = 0;
  int32_t vec = 0;       // the outputs allow 16-byte stores
  unsigned int* status = nullptr;
};

struct KvAttendArgs {
  CacheArgs c;
  Rows q, out;           // token = sequence
  const int32_t* table = nullptr;
  int64_t table_stride = 0, max_tokens = 0;
  const int32_t* lens = nullptr;
  int32_t seqs = 0, group = 1, heads_q = 1;
  int32_t elem = LM_BF16;
  int64_t window = 0;
  float scale = 1;
  float* lse = nullptr;
  void* ws = nullptr;
  unsigned int* status = nullptr;
  // elements of the page table from one key head's pages to the next one's
  // (0: the heads share them)
  int64_t table_head = 0;
  // where set: the scores s in units of ln 2, [seqs, key heads, max_tokens,
  // group], and of each row a reference t and 1 / sum 2^(s - t) (0 and 0: no
  // weights), [seqs, heads_q, 2]
  float *scores = nullptr, *norms = nullptr;
  // where set: the state (m, l) and the mean of each row in 32 bits, [seqs,
  // heads_q] and [seqs, heads_q, dim], in the output's place
  float *state = nullptr, *mean = nullptr;
  // and no pieces (see KvSharedArgs) of the rows
  int32_t* pieces = nullptr;
};

int launch_rope(const RopeArgs& a, int elem, void* stream);
int launch_rope_table(const RopeTableArgs& a, void* stream);
int launch_kv_write(const KvWriteArgs& a, int elem, int store, void* stream);
int launch_kv_read(const KvReadArgs& a, int elem, int store, int out_elem,
                   void* stream);
int launch_kv_attend(const KvAttendArgs& a, int store, void* stream);
// The current device (below 64) and its SMs.
int kv_device(int* dev, int* sms);
// Bytes of the attention's workspace on the current device.
int attend_workspace(int store, int dim, int group, int64_t* bytes);

}  // namespace lm

struct lm_rope_plan {
  int head_dim = 0, rotary = 0, inter = 0;
  double amplitude = 1;
  std::vector<double> freq;
};

struct lm_kv_plan {
  int64_t page_tokens = 0, heads = 0, dim = 0;
  int64_t token_stride = 0, head_stride = 0, page_stride = 0;  // elements
  int64_t page_cosize = 0;
  int elem = LM_BF16, store = LM_KV_SAME;
  int held = 2;  // bytes of a held element
  std::string describe;
};
