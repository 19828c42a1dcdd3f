// Attention of many queries over keys and values that they share: the new
// tokens of a group of sequences, all of their query heads of one key head,
// against the pages of the group's common prefix.
//
// With R = sequences x queries a key head, S = Q K^T and O = P V are products
// of R rows, 4 R dim operations for every 4 dim bytes of a key and its value
// (16 bits): from R of some 280 on the tensor cores bound it and not memory,
// and below that it is one pass over the prefix where R / group passes, one a
// sequence, would each read all of it.  So here the products are the 128-row
// ones of tcgen05, whose sums stay in tensor memory.
//
// A block has two tiles of 128 queries (one where rows are longer than 128
// elements) and streams tiles of 128 (64) keys past them:
//   warps 8-11  bring keys and values from their pages into shared memory, as
//               they are or widened from codes, in the 128-byte swizzle
//   warp 12     one lane issues S_q = Q_q K^T and O_q += P_q V, in turn for the
//               two q (a warp for each let the two fall into step, so that
//               nothing overlapped: 4.6 against 3.8 thousand cycles a tile)
//   warp 13     passes on what copies have brought: a fence between the copies'
//               writes and the products' reads, which would hold warp 12 up
//   warps 0-3   and 4-7, one for each tile of queries: Q into shared memory, a
//               row a thread; then S from tensor memory, 16 rows at a time and
//               four threads a row, its exponentials, and P back in S's place.
//               (A row a thread would be one exchange less, but every thread
//               then reads every key's scales: 4000 of 9500 cycles a tile.)
// While one tile's exponentials are taken the tensor cores have the other's
// products.  Where there are no more than 128 queries, the two take every
// second tile of keys instead, with states of their own that are joined later.
//
// What bounds it is how long one tile of queries takes: its exponentials, 2300
// cycles (4100 for codes, whose every score meets three numbers of its key),
// and then its two products, 1050, one after the other, while the tensor cores
// are 23-26% busy.  (The way out to rare tiles, see SharedRare, came after those
// counts and takes 5 to 8% more.)  Measured: 31 us for 256 queries of 8 key heads
// over 16384 tokens of 128 bf16 elements (the bytes 10, the products 9), 287 us
// for 128 sequences x 8 queries of 8 key heads in e4m3, 360, 112 and 552 rows a
// head over 32768, 19371 and 28126 tokens, 0.42 PFLOP/s.  552 rows are two full
// tiles and one of 40, whose empty rows take as long as full ones and which reads
// the prefix a third time.  Giving uneven tiles of rows more tiles of keys by
// weight made the line's end even but its time no shorter (349 us for the whole
// call against 344 then), nor did three more loading warps for the values, or one
// pass for largest and weights that is taken again when a reference moves (367).
//
// Work is one line of key tiles over all groups, key heads and tiles of rows,
// cut evenly over the resident blocks; what one block holds of rows that others
// share goes to the workspace, and the launch that joins it with the attention
// over each sequence's own pages reads it in the order of the line.
//
// Weights are one 16-bit part each (bf16's rounding of a weight costs a result
// about as much as its own): a second part would be half as many products
// again.  Codes become f16, whose 11 bits hold them, for f16 queries (bf16 ones
// times a power of two a row) and f16 weights.  A value's scale v_j is folded
// into its weight's exponent, 2^(s_j - m + log2 v_j - L), with the row's
// reference m the largest s_j + log2 v_j - L: what a weight loses is relative to
// the largest contribution of its row, whatever the scales.  L, a multiple of
// 32, is the end of the band that the logarithms of a run's scales lie in.  The
// sum of the weights alone, relative to m too, adds 2^L / v_j of each.  Where a
// run's scales lie in several bands (those of a model do not), a score may
// exceed m by more than 32 bits' range has room for: from there on the weights
// are summed for themselves, relative to a largest score of their own (see
// SharedRare).
#pragma once

#include "lm_attend.cuh"
#include "lm_kv_long.h"
#include "lm_line.cuh"
#include "lm_mbar.cuh"
#include "lm_tcgen05.cuh"

namespace lm {

// Four warpgroups, whose threads' registers are as many as their work wants;
// together those of 512 threads of 128.
constexpr int kSharedThreads = 512;
constexpr int kRegsExp = 160, kRegsLoad = 136, kRegsProducts = 56;
static_assert(128 * (2 * kRegsExp + kRegsLoad + kRegsProducts) <= 512 * 128,
              "no more registers than the block has");

template <int D>
struct SharedShape {
  static constexpr int QT = D == 256 ? 1 : 2;          // tiles of queries
  static constexpr int NK = D == 256 ? 64 : 128;       // keys of a tile
  static constexpr int kRows = QT * 128;
  static constexpr int kTile = NK * D * 2;             // bytes of K or of V
  static constexpr int kQ = 128 * D * 2;               // and of a tile of Q
  static constexpr int NS = D == 64 ? 3 : 2;           // stages of K, of V
  // What goes with a tile's keys (scales and which are seen) is read until
  // its weights are written.  When a tile's turn comes the values NS + 1 tiles
  // before it are done with, so that many hold: for each key of a cache of
  // codes its scale times log2(e) and the softmax's, its value's scale's
  // logarithm to base 2 and the scale's inverse; then the masks, and each
  // loading warp's least and largest logarithm.
  static constexpr int NM = NS + 1;
  static constexpr int kMeta = NK * 12 + 48;
  static constexpr uint32_t kOut = 256;                // O's first column
  static constexpr int kBars = 6 * NS + 12;
  static constexpr int kSmem =
      1024 + QT * kQ + 2 * NS * kTile + NM * kMeta + kBars * 8 + 16;
};

// A wait on an mbarrier that ends: after about a second, or when another of
// the block's waits has, it gives up.
__device__ __forceinline__ bool gate(uint32_t bar, uint32_t parity,
                                     volatile int* dead) {
  if (mbar_try(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try(bar, parity)) {
    if (*dead) return false;
    if (clock64() - t0 > kWaitCycles) {
      *dead = 1;
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool warp_gate(uint32_t bar, uint32_t parity,
                                          volatile int* dead) {
  return __all_sync(0xffffffffu, gate(bar, parity, dead));
}

struct SharedSpan {
  int start, n;        // the group's sequences
  int len, tiles;      // its tokens and tiles of keys
  int row_tiles;
};
__device__ __forceinline__ SharedSpan shared_span(const KvSharedArgs& a, int g,
                                                  int keys, int rows) {
  SharedSpan s;
  const int end = min(max(a.starts[g + 1], 0), a.seqs);
  s.start = min(max(a.starts[g], 0), a.seqs);
  s.n = max(end - s.start, 0);
  const int64_t len = a.lens[g];
  s.len = int(len < 0 ? 0 : len > a.max_tokens ? a.max_tokens : len);
  s.tiles = s.n ? (s.len + keys - 1) / keys : 0;
  s.row_tiles = (s.n * a.group + rows - 1) / rows;
  return s;
}

// A run of key tiles of one group, key head and tile of rows.
struct SharedSeg {
  SharedSpan s;
  int g, h, rt;
  int t0, steps;       // tiles t0 .. t0 + steps - 1
  int rows;            // valid ones of the tile of rows
  int64_t item_at;     // where the item's tiles start on the line
};

// The segments of a block's share, one after the other.
template <int NK, int ROWS>
struct SharedWalk {
  int64_t left, in, line;      // tiles left; the next one's number in group g,
  int g;                       // whose tiles start at `line`
  __device__ __forceinline__ bool next(const KvSharedArgs& a, SharedSeg* seg) {
    if (left <= 0) return false;
    seg->s = shared_span(a, g, NK, ROWS);
    int64_t units = int64_t(seg->s.tiles) * seg->s.row_tiles * a.c.heads;
    while (in >= units) {
      // (never, unless the lengths change while the kernel runs)
      if (g + 1 >= a.groups) return false;
      in -= units;
      line += units;
      seg->s = shared_span(a, ++g, NK, ROWS);
      units = int64_t(seg->s.tiles) * seg->s.row_tiles * a.c.heads;
    }
    const int64_t item = small_div(in, seg->s.tiles);
    seg->g = g;
    seg->t0 = int(in - item * seg->s.tiles);
    seg->h = int(small_div(item, seg->s.row_tiles));
    seg->rt = int(item - int64_t(seg->h) * seg->s.row_tiles);
    const int64_t rest = seg->s.tiles - seg->t0;
    seg->steps = int(left < rest ? left : rest);
    seg->rows = min(ROWS, seg->s.n * a.group - seg->rt * ROWS);
    seg->item_at = line + item * seg->s.tiles;
    in += seg->steps;
    left -= seg->steps;
    return true;
  }
};

// 16 codes as f16, in order.
template <int STORE>
__device__ __forceinline__ void widen16(const uint4& w, uint32_t* y) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (STORE == LM_KV_E4M3) {
      Codes<KIND_E4M3>::keys(r[i], y + 2 * i);
    } else {
      uint32_t p[2];
      Codes<KIND_INT8>::keys(r[i], p);
      y[2 * i] = __byte_perm(p[0], p[1], 0x5410);
      y[2 * i + 1] = __byte_perm(p[0], p[1], 0x7632);
    }
  }
}

// Two numbers at a time: the pair forms of a multiplication, an addition and
// both take one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long y;
  asm("mul.rn.f32x2 %0, %1, %2;\n"
      : "=l"(y)
      : "l"(reinterpret_cast<unsigned long long&>(a)),
        "l"(reinterpret_cast<unsigned long long&>(b)));
  return reinterpret_cast<float2&>(y);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long y;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(y)
      : "l"(reinterpret_cast<unsigned long long&>(a)),
        "l"(reinterpret_cast<unsigned long long&>(b)));
  return reinterpret_cast<float2&>(y);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long y;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(y)
      : "l"(reinterpret_cast<unsigned long long&>(a)),
        "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return reinterpret_cast<float2&>(y);
}

// The band that the logarithm of a scale lies in, (end - 32, end]: its end.
__device__ __forceinline__ float scale_band(float x) {
  return 32.f * ceilf(x * (1.f / 32));
}

__device__ __forceinline__ void st_smem16(uint32_t to, uint32_t a, uint32_t b,
                                          uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(to), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ float over_quad(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
// The means of 16 rows times keep[0] (rows t / 4 of thread t) and keep[1].
__device__ __forceinline__ void scale_means(uint32_t at, int dim,
                                            const float* keep) {
#pragma unroll 1
  for (int c = 0; c < dim; c += 32) {
    uint32_t o[16];
    tmem_ld<4>(o, at + c);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i)
      o[i] = __float_as_uint(__uint_as_float(o[i]) * keep[i / 2 % 2]);
    tmem_st4(at + c, o);
  }
}

// A row's reference moves when a score passes it by SLACK (in units of ln
// 2).  f16 weights lie below 2^15, the reference's at 2^12.  bf16 values
// reach the end of 32 bits' range, so their weights' sum stays below 1.
template <bool BF>
constexpr float kSharedSlack = BF ? 8.f : 3.f;

// What a warp of the exponentials does with a tile of keys where their values'
// scales lie in several bands, or in another than those before, or where a
// row's reference is large; and with the segment's tiles from there on.  Apart
// from the kernel's own way for all others, and with few instructions rather than
// fast.  What is rounded with a score here is its difference from a number near
// it: beside a score of 2^20 the logarithm of a scale would lose all but four of
// its bits.
struct SharedRare {
  uint32_t s_at, o_at;         // the warp's scores and means in tensor memory
  const char* meta;            // what goes with the tile's keys
  // of rows t / 4 of thread t and 8 on, of the warp's first 16 and its others.
  // Sums are relative to references of their own, largest scores: one may exceed
  // m by what scales differ by.
  float m[4], ref[4], l[4], down[4];
  float band, off, unit;
  int dim, half;               // from which half of the rows on
  bool first;
};
template <bool BF, bool CODES, int NK>
__device__ __forceinline__ void shared_rare(SharedRare* const io) {
  constexpr float SLACK = kSharedSlack<BF>;
  SharedRare r = *io;
  const int lane = threadIdx.x % 32;
  const float2* const ku = reinterpret_cast<const float2*>(r.meta) + lane % 4;
  const uint32_t* const words =
      reinterpret_cast<const uint32_t*>(r.meta + NK * 12);
  float band = 0, up = 0;        // a higher band than before, by so much
  if (CODES) {
    const float4 tops = reinterpret_cast<const float4*>(words)[2];
    band = fmaxf(r.band, scale_band(fmaxf(fmaxf(tops.x, tops.y),
                                          fmaxf(tops.z, tops.w))));
    if (!r.first) up = band - r.band;
    r.band = band;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (half < r.half) continue;
    const uint32_t lanes = uint32_t(half * 16) << 16;
    float* const m = r.m + 2 * half;
    float* const ref = r.ref + 2 * half;
    float* const l = r.l + 2 * half;
    const float* const down = r.down + 2 * half;
    // the scores of columns 32c .. 32c + 31
    auto scores = [&](int c, float2 (&x)[4][2]) {
      uint32_t w[16];
      tmem_ld<4>(w, r.s_at + lanes + c * 32);
      tmem_wait_ld();
      const uint32_t seen =
          (NK == 128 ? words[c] : words[2 * c] | words[2 * c + 1] << 16) >>
          (lane % 4 * 2);
#pragma unroll
      for (int g = 0; g < 4; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float2 y = make_float2(__uint_as_float(w[4 * g + 2 * i]),
                                 __uint_as_float(w[4 * g + 2 * i + 1]));
          y = CODES ? mul2(mul2(y, ku[16 * c + 4 * g]),
                           make_float2(down[i], down[i]))
                    : mul2(y, make_float2(r.unit, r.unit));
          x[g][i] = make_float2(seen >> 8 * g & 1 ? y.x : -INFINITY,
                                seen >> (8 * g + 1) & 1 ? y.y : -INFINITY);
        }
    };
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
    for (int c = 0; c < NK / 32; ++c) {
      float2 x[4][2];
      scores(c, x);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        best[e % 2] = fmaxf(best[e % 2],
                            fmaxf(x[e / 2][e % 2].x, x[e / 2][e % 2].y));
    }
    float base[2], from[2], top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      best[i] = over_quad(best[i]);
      if (best[i] - ref[i] > SLACK) {
        l[i] *= ex2(ref[i] - best[i]);
        ref[i] = best[i];
      }
      // (a row that has seen no key yet, or only ones of -infinity)
      from[i] = ref[i] == -INFINITY ? 0.f : ref[i];
      base[i] = fabsf(m[i]) < INFINITY      ? m[i]
                : fabsf(best[i]) < INFINITY ? best[i]
                                            : 0.f;
    }
    // the largest score with its value's scale, relative to the base
#pragma unroll 1
    for (int c = 0; c < NK / 32; ++c) {
      float2 x[4][2];
      scores(c, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int g = e / 2, i = e % 2;
        float2 y = make_float2(x[g][i].x - base[i], x[g][i].y - base[i]);
        if (CODES) y = add2(y, ku[NK / 2 + 16 * c + 4 * g]);
        top[i] = fmaxf(top[i], fmaxf(y.x, y.y));
      }
    }
    float keep[2] = {1, 1}, sub[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[i] = over_quad(top[i]) - band;
      const float was = m[i] - base[i] - up;
      float to = base[i] + (top[i] - was > SLACK ? top[i] : was);
      // (A sum that is rounded down.  No weight lies above the largest score's,
      // whose scale's logarithm is no more than the band's end.)
      if (top[i] - (to - base[i]) > SLACK) to = best[i];
      // (nor is what a sum that is rounded differs by lost)
      const float at = to - base[i];
      if (at != was) keep[i] = ex2(was - at);
      m[i] = to;
      sub[i] = r.off - band - (at == -INFINITY ? 0.f : at);
    }
    if (!r.first) scale_means(r.o_at + lanes, r.dim, keep);
#pragma unroll 1
    for (int c = 0; c < NK / 32; ++c) {
      float2 x[4][2];
      scores(c, x);
      uint32_t p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int g = e / 2, i = e % 2;
        const float2 y = x[g][i];
        float2 lv = make_float2(0, 0);
        if (CODES) lv = ku[NK / 2 + 16 * c + 4 * g];
        l[i] += ex2(y.x - from[i]) + ex2(y.y - from[i]);
        p[e] = pair16<BF>(ex2((y.x - base[i]) + (lv.x + sub[i])),
                          ex2((y.y - base[i]) + (lv.y + sub[i])));
      }
      // (over scores that have been read)
      tmem_st_pairs<4>(r.s_at + lanes + c * 16, p);
    }
  }
  r.first = false;
  r.half = 0;
  *io = r;
}
// As a call for 16-bit rows, in line for codes: the other way round 64 sequences
// of bf16 behind 16384 tokens take 94.2 us for 93.2, 128 in e4m3 370 for 365.
// (What it costs either way is registers of the loops that never come here, 346
// and 91.4 us without.)
template <bool BF, int NK>
__device__ __noinline__ void shared_rare_rows(SharedRare* const io) {
  shared_rare<BF, false, NK>(io);
}

// BF: the cache holds bf16 rows (and the products are bf16's).  At 128 registers
// a thread the forms for up to 128 elements spill: 144 bytes those for codes, up
// to 52 the others; rows of 256 elements 24 and none.
template <bool BF, int STORE, int D>
__global__ void __launch_bounds__(kSharedThreads, 1)
    lm_kv_shared_kernel(const __grid_constant__ KvSharedArgs a) {
  using S = SharedShape<D>;
  constexpr int NK = S::NK, QT = S::QT, NS = S::NS, NM = S::NM;
  constexpr bool CODES = STORE != LM_KV_SAME;
  constexpr float SLACK = kSharedSlack<BF>;
  // A reference is the largest score, so that the heaviest key's weight is a
  // power of two and loses nothing to its rounding (the next whole number in its
  // place: errors of 0.0022 for 0.0018 of a few hundred tokens of bf16).  Beyond
  // LARGE what a logarithm or the sum of `off` and a reference lose beside one
  // (2^-15 there), or what a fused multiplication leaves of a score's rounding,
  // would matter: see SharedRare.
  constexpr float LARGE = 0x1p10f;
  constexpr int KPW = NK / 4;                   // keys of a loading warp
  extern __shared__ char smem_raw[];
  __shared__ volatile int dead;
  __shared__ uint32_t tmem_at;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x / 32, 0);
  const int lane = threadIdx.x % 32;
  const int dim = a.c.dim;
  const int dim16 = (dim + 15) / 16 * 16;

  char* const base = smem_raw + ((1024 - (uint32_t(__cvta_generic_to_shared(
                                             smem_raw)) &
                                         1023)) &
                                 1023);
  const uint32_t base_s = uint32_t(__cvta_generic_to_shared(base));
  const uint32_t q_s = base_s, k_s = q_s + QT * S::kQ,
                 v_s = k_s + NS * S::kTile, meta_s = v_s + NS * S::kTile;
  char* const metas = base + (meta_s - base_s);
  const uint32_t bars = meta_s + NM * S::kMeta;
  auto k_full = [&](int i) { return bars + 8 * i; };
  auto k_empty = [&](int i) { return bars + 8 * (NS + i); };
  auto v_full = [&](int i) { return bars + 8 * (2 * NS + i); };
  auto v_empty = [&](int i) { return bars + 8 * (3 * NS + i); };
  auto s_full = [&](int q) { return bars + 8 * (4 * NS + q); };
  auto p_full = [&](int q) { return bars + 8 * (4 * NS + 2 + q); };
  auto o_full = [&](int q) { return bars + 8 * (4 * NS + 4 + q); };
  auto o_empty = [&](int q) { return bars + 8 * (4 * NS + 6 + q); };
  const uint32_t q_full = bars + 8 * (4 * NS + 8);
  const uint32_t q_empty = bars + 8 * (4 * NS + 9);
  const uint32_t drain = bars + 8 * (4 * NS + 10);
  // what the products wait for
  auto k_ready = [&](int i) {
    return CODES ? k_full(i) : bars + 8 * (4 * NS + 12 + i);
  };
  auto v_ready = [&](int i) {
    return CODES ? v_full(i) : bars + 8 * (5 * NS + 12 + i);
  };

  // (none of this touches global memory)
  if (threadIdx.x == 0) {
    dead = 0;
    // a loading thread's copies arrive by themselves, and a warp's scales and
    // masks with one lane
    const uint32_t come = CODES ? 128 : 132;
    for (int i = 0; i < NS; ++i) {
      mbar_init(k_full(i), come);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), 128);
      mbar_init(v_empty(i), 1);
      if (!CODES) {
        mbar_init(k_ready(i), 1);
        mbar_init(v_ready(i), 1);
      }
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(s_full(q), 1);
      mbar_init(p_full(q), 128);
      mbar_init(o_full(q), 1);
      mbar_init(o_empty(q), 128);
    }
    mbar_init(q_full, 256);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 12)
    tmem_alloc(uint32_t(__cvta_generic_to_shared(&tmem_at)), 512);
  stream_order();
  tmem_before_sync();
  const LineShare share = line_share<kSharedThreads>(
      a.groups, blockIdx.x, gridDim.x, [&](int g) {
        const SharedSpan s = shared_span(a, g, NK, S::kRows);
        return int64_t(s.tiles) * s.row_tiles * a.c.heads;
      });
  __syncthreads();
  tmem_after_sync();
  const uint32_t tmem = tmem_at;
  SharedWalk<NK, S::kRows> walk;
  walk.left = share.left;
  walk.in = share.in;
  walk.line = share.begin - share.in;
  walk.g = share.b;
  SharedSeg seg;
  // no more than 128 rows: each half of the exponential warps has every second
  // tile of keys
  auto split_of = [&](const SharedSeg& s) { return QT == 2 && s.rows <= 128; };

  if (warp >= 8 && warp < 12) {
    // --- keys and values ---
    if (CODES) registers_up<kRegsLoad>();
    const int lw = warp - 8;
    constexpr int EB = CODES ? 1 : 2;
    constexpr int CPR = D * EB / 16;            // 16-byte chunks of a row
    constexpr int RPI = 32 / CPR;               // rows an instruction
    constexpr int IT = KPW / RPI;
    const int c = lane % CPR, r0 = lane / CPR;
    const bool held = c * 16 < dim * EB;
    const bool used = c * 16 < dim16 * EB;
    int tile = 0;
    bool alive = true;
    auto acquire = [&](uint32_t bar, uint32_t parity) {
      if (!warp_gate(bar, parity, &dead)) alive = false;
    };
    const float unit =
        a.scale == 0 ? 1.f : fabsf(a.scale) * 1.44269504088896341f;
    const bool mine = KPW == 32 || lane < KPW;       // a key of this lane's
    const uint32_t to = lw * KPW * 128;
    float last = 1;                 // the largest scale of the tile before
    while (alive && walk.next(a, &seg)) {
      const int32_t* const table = a.table + seg.g * a.table_stride;
      const int t1 = seg.t0 + seg.steps;
      auto look = [&](int t) {
        const int key = t * NK + lw * KPW + lane;
        return mine && t < t1 && key < seg.s.len
                   ? table[fdiv(uint32_t(key), a.c.page_div)]
                   : -1;
      };
      int page = look(seg.t0);
      // the lane's key of tile t, whose page has been looked up: where its row
      // lies (-1: not seen), and the next tile's page on its way
      int64_t from, scale_at;
      uint32_t seen, off16[IT];      // of codes: the lane's chunks, in 16 bytes
      auto find = [&](int t) {
        const int key = t * NK + lw * KPW + lane;
        const bool in = mine && t < t1 && key < seg.s.len;
        const bool ok = in && page >= 0 && page < a.c.pages;
        if (in && !ok && a.status) atomicOr(a.status, kStatusRange);
        const uint32_t off =
            uint32_t(key) - fdiv(uint32_t(key), a.c.page_div) * a.c.page_tokens;
        from = ok ? int64_t(page) * a.c.page_b + int64_t(off) * a.c.token_b +
                        int64_t(seg.h) * a.c.head_b
                  : -1;
        if (CODES) {
          scale_at = ok ? (int64_t(page) * a.c.heads + seg.h) *
                                  a.c.page_tokens +
                              off
                        : -1;
          // A cache of 2^36 bytes or more is refused.  A key that is not seen,
          // and a chunk past the row's end, has any other's codes: the mask
          // hides the key, `widen` clears its values, and the chunk stays in
          // its registers.
          const uint32_t row = ok ? uint32_t(from >> 4) : 0;
#pragma unroll
          for (int i = 0; i < IT; ++i)
            off16[i] = __shfl_sync(0xffffffffu, row, i * RPI + r0) +
                       (held ? c : 0);
        }
        seen = __ballot_sync(0xffffffffu, ok);
        page = look(t + 1);
      };
      if constexpr (CODES) {
        // Codes pass through registers.  The next tile's keys are asked for
        // while this one's values are widened, its values while the next one's
        // keys are.
        uint4 kr[IT], vr[IT];
        float ks, vs;
        auto ask = [&](uint4* w, const char* rows) {
#pragma unroll
          for (int i = 0; i < IT; ++i)
            w[i] = *(reinterpret_cast<const uint4*>(rows) + off16[i]);
        };
        auto ask_keys = [&](int t) {
          find(t);
          ks = vs = 0;
          if (scale_at >= 0) {
            ks = a.c.ks[scale_at];
            vs = a.c.vs[scale_at];
          }
          ask(kr, a.c.k);
        };
        // Widened to f16.  What the logarithm of a value's scale says nothing of
        // goes to the widened values (of the codes -128 has no opposite):
        // `turned` where a row of the warp's is to be.  Its factor is the scale
        // for its sign, 0 or NaN, and infinite for a key that is not seen, whose
        // values become 0 whatever they are.
        auto widen = [&](uint32_t tile_s, const uint4* w, auto turned,
                         float factor) {
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            const int r = i * RPI + r0;
            uint32_t y[8];
            widen16<STORE>(w[i], y);
            if constexpr (decltype(turned)::value) {
              const float f = __shfl_sync(0xffffffffu, factor, r);
              const __half2 by =
                  __float2half2_rn(f > 0 ? 1.f : f < 0 ? -1.f : f);
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const __half2 v =
                    __hmul2(*reinterpret_cast<const __half2*>(&y[e]), by);
                y[e] = f == INFINITY ? 0u : *reinterpret_cast<const uint32_t*>(&v);
              }
            }
            if (!held) continue;
            // (four lanes begin with their first chunk and four with their
            // second, so that eight lanes' stores lie in all banks)
            const bool odd = c / 4 & 1;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int ch = 2 * c + (j ^ int(odd));
              uint32_t x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[e] = odd ? y[4 * (1 - j) + e] : y[4 * j + e];
              st_smem16(tile_s + ch / 8 * (NK * 128) + r * 128 +
                            ((ch ^ r) & 7) * 16,
                        x[0], x[1], x[2], x[3]);
            }
          }
          smem_to_products();
        };
        ask_keys(seg.t0);
        ask(vr, a.c.v);
        for (int t = seg.t0; t < t1 && alive; ++t, ++tile) {
          const int slot = tile % NS;
          const uint32_t turn = tile / NS & 1;
          if (tile >= NS) acquire(k_empty(slot), turn ^ 1);
          if (!alive) break;
          // (see NM: nothing reads these any more)
          char* const m = metas + tile % NM * S::kMeta;
          // a scale of 0, or that is no number or infinite, counts as the largest
          // about: its key has a weight like any other, and its values are 0 or
          // no numbers
          // (magnitudes in the order of their bits)
          const bool usable = fabsf(vs) > 0 && fabsf(vs) < INFINITY;
          const uint32_t top = __reduce_max_sync(
              0xffffffffu, usable ? __float_as_uint(fabsf(vs)) : 0u);
          if (top) last = __uint_as_float(top);
          const float size = usable ? fabsf(vs) : last;
          const uint32_t bits = __float_as_uint(size);
          const uint32_t least = __reduce_min_sync(0xffffffffu, bits);
          const uint32_t most = __reduce_max_sync(0xffffffffu, bits);
          const float end = log2f(__uint_as_float(lane ? most : least));
          const float band =
              scale_band(__shfl_sync(0xffffffffu, end, 1));
          if (mine) {
            float* f = reinterpret_cast<float*>(m) + lw * KPW + lane;
            f[0] = scale_at >= 0 ? ks * unit : 1.f;
            const float log = log2f(size);
            f[NK] = log;
            // (of the rounded logarithm, so that a weight's two factors cancel)
            f[2 * NK] = ex2(band - log);
          }
          if (lane == 0)
            reinterpret_cast<uint32_t*>(m + NK * 12)[lw] = seen;
          if (lane < 2)
            reinterpret_cast<float*>(m + NK * 12 + 16)[lane * 4 + lw] = end;
          widen(k_s + slot * S::kTile + to, kr, std::false_type{}, 0.f);
          mbar_arrive(k_full(slot));
          const float factor = scale_at < 0          ? INFINITY
                               : usable || vs == 0 ? vs
                                                   : NAN;
          ask_keys(t + 1);
          if (tile >= NS) acquire(v_empty(slot), turn ^ 1);
          if (!alive) break;
          if (__any_sync(0xffffffffu, mine && !(factor > 0 && factor < INFINITY)))
            widen(v_s + slot * S::kTile + to, vr, std::true_type{}, factor);
          else
            widen(v_s + slot * S::kTile + to, vr, std::false_type{}, 0.f);
          mbar_arrive(v_full(slot));
          ask(vr, a.c.v);
        }
      } else {
        for (int t = seg.t0; t < t1 && alive; ++t, ++tile) {
          find(t);
          const int slot = tile % NS;
          const uint32_t turn = tile / NS & 1;
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (tile >= NS)
              acquire(kv ? v_empty(slot) : k_empty(slot), turn ^ 1);
            if (!alive) break;
            // (see NM: nothing reads the mask there any more)
            if (kv == 0 && lane == 0) {
              reinterpret_cast<uint32_t*>(metas + tile % NM * S::kMeta +
                                          NK * 12)[lw] = seen;
              mbar_arrive(k_full(slot));
            }
            const uint32_t tile_s = (kv ? v_s : k_s) + slot * S::kTile + to;
            const char* const src = kv ? a.c.v : a.c.k;
#pragma unroll
            for (int i = 0; i < IT; ++i) {
              const int r = i * RPI + r0;
              const int64_t o = __shfl_sync(0xffffffffu, from, r);
              const uint32_t bytes = o >= 0 && held ? 16 : 0;
              if (used)
                cp16(tile_s + c / 8 * (NK * 128) + r * 128 +
                         ((c ^ r) & 7) * 16,
                     src + (bytes ? o + c * 16 : 0), bytes);
            }
            cp_async_arrive_noinc(kv ? v_full(slot) : k_full(slot));
          }
        }
      }
    }
    cp_commit();
    cp_wait<0>();
  } else if (warp >= 12) {
    if (CODES) registers_down<kRegsProducts>();
    if (!CODES && warp == 13) {
      // --- copies passed on ---
      for (int64_t tile = 0; tile < share.left; ++tile) {
        const int slot = int(tile % NS);
        const uint32_t turn = tile / NS & 1;
        if (!warp_gate(k_full(slot), turn, &dead)) break;
        smem_to_products();
        if (lane == 0) mbar_arrive(k_ready(slot));
        if (!warp_gate(v_full(slot), turn, &dead)) break;
        smem_to_products();
        if (lane == 0) mbar_arrive(v_ready(slot));
      }
    }
    // --- products: the warp together, one lane issues ---
    const uint32_t kind_s = mma_kind(BF, false, 128, NK);
    const uint32_t kind_o = mma_kind(BF, true, 128, dim16);
    const int ks = dim16 / 16;
    const uint64_t q_op = smem_operand(q_s, 16, 1024);
    const uint64_t k_op = smem_operand(k_s, 16, 1024);
    const uint64_t v_op = smem_operand(v_s, NK * 128, 1024);
    int tile = 0, nth = 0;
    // the phases of p_full and o_empty, a bit a tile of queries, and whether a
    // tile's O was ever read
    uint32_t p_phase = 0, o_phase = 0, o_read = 0;
    bool alive = warp == 12;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (alive && !warp_gate(bar, parity, &dead)) alive = false;
      return alive;
    };
    while (alive && walk.next(a, &seg)) {
      const bool split = split_of(seg);
      const int per = split || QT == 1 ? 1 : (seg.rows + 127) / 128;
      const int units = seg.steps * per;
      // unit u: key tile u / per, and which half of the exponential warps has
      // it
      const bool two = split || per == 2;
      const int ahead = two ? 2 : 1;
      // (by one lane)
      auto score = [&](int u, int slot) {
        const int q = two ? u & 1 : 0;
        const uint64_t qa = q_op + (split ? 0 : q) * (S::kQ / 16);
        const uint64_t ka = k_op + slot * (S::kTile / 16);
        const uint32_t to = tmem + q * NK;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          if (k >= ks) break;
          mma_ss(to, qa + (k / 4 * (128 * 128) + k % 4 * 32) / 16,
                 ka + (k / 4 * (NK * 128) + k % 4 * 32) / 16, kind_s, k > 0);
        }
        mma_commit(s_full(q));
        if (per == 1 || q == 1) mma_commit(k_empty(slot));
        if (u == units - 1) mma_commit(q_empty);
      };
      auto tile_of = [&](int u) { return tile + (per == 2 ? u / 2 : u); };
      if (!wait(q_full, nth & 1)) break;
      ++nth;
      for (int u = 0; u < ahead && u < units; ++u) {
        const int t = tile_of(u), slot = t % NS;
        if ((per == 1 || u == 0) && !wait(k_ready(slot), t / NS & 1)) break;
        tmem_after_sync();
        if (one_lane()) score(u, slot);
        __syncwarp();
      }
      for (int u = 0; u < units && alive; ++u) {
        const int t = tile_of(u), slot = t % NS;
        const int q = two ? u & 1 : 0;
        const bool opens = per == 1 || q == 0;     // a tile's first unit
        // The values, and whether the next scores' keys are there already,
        // before the weights, which are waited for longest.
        if (opens && !wait(v_ready(slot), t / NS & 1)) break;
        const bool more = u + ahead < units;
        const int t2 = tile_of(u + ahead), slot2 = t2 % NS;
        bool keys = more;
        if (more && opens)
          keys = __all_sync(0xffffffffu, mbar_try(k_ready(slot2), t2 / NS & 1));
        const bool first = split ? u < 2 : t == tile;
        if (first && (o_read >> q & 1)) {
          if (!wait(o_empty(q), o_phase >> q & 1)) break;
          o_phase ^= 1u << q;
        }
        const bool last = u + (split ? 2 : per) >= units;
        if (!wait(p_full(q), p_phase >> q & 1)) break;
        p_phase ^= 1u << q;
        tmem_after_sync();
        if (one_lane()) {
          const uint64_t va = v_op + slot * (S::kTile / 16);
          const uint32_t o = tmem + S::kOut + q * D;
          const uint32_t p = tmem + q * NK;
#pragma unroll
          for (int i = 0; i < NK / 16; ++i)
            mma_ts(o, p + i * 8, va + i * (2048 / 16), kind_o,
                   !(first && i == 0));
          if (keys) score(u + ahead, slot2);
          if (per == 1 || q == 1) mma_commit(v_empty(slot));
          if (last) mma_commit(o_full(q));
        }
        __syncwarp();
        if (last) o_read |= 1u << q;
        if (more && !keys) {
          if (!wait(k_ready(slot2), t2 / NS & 1)) break;
          tmem_after_sync();
          if (one_lane()) score(u + ahead, slot2);
          __syncwarp();
        }
      }
      tile += seg.steps;
    }
    if (dead && warp == 12) {
      // products may still read shared memory and write tensor memory
      if (one_lane()) mma_commit(drain);
      warp_wait(drain, 0, kDrainCycles);
    }
  } else {
    // --- exponentials ---
    if (CODES) registers_up<kRegsExp>();
    const int q = warp / 4;
    const int row = warp % 4 * 32 + lane;
    const uint32_t quarter = uint32_t(warp % 4 * 32) << 16;
    const uint32_t s_at = tmem + q * NK + quarter;
    const uint32_t o_at = tmem + S::kOut + q * D + quarter;
    // (with a scale of 0 the queries are taken as 0)
    const float unit =
        a.scale == 0 ? 1.f : fabsf(a.scale) * 1.44269504088896341f;
    const uint32_t flip = a.scale < 0 ? 0x80008000u : 0;
    int tile = 0, nth = 0, n_s = 0, n_o = 0;
    bool alive = true;
    while (alive && walk.next(a, &seg)) {
      const bool split = split_of(seg);
      const int t_first = tile;
      tile += seg.steps;
      const int r = split ? row : q * 128 + row;
      const int rg = seg.rt * S::kRows + r;
      const int si = rg / a.group;
      const bool valid = r < seg.rows;
      const uint16_t* const query =
          reinterpret_cast<const uint16_t*>(a.q.p) +
          int64_t(seg.s.start + si) * a.q.ts +
          int64_t(seg.h * a.group + (rg - si * a.group)) * a.q.hs;
      if (nth == 0 && valid)
        for (int c = 0; c < dim; c += 64)
          asm volatile("prefetch.global.L1 [%0];\n" ::"l"(query + c));
      const int step = split ? 2 : 1;
      const bool active = split || q * 128 < seg.rows;
      // The thread's share of four rows: t / 4 and 8 on of a warp's first 16,
      // then of its other 16.  The pairs change places after each 16.
      float m[2], l[2], m2[2], l2[2];
      // of codes: what the rows' queries were held times, the band that scales
      // lie in
      float down[2] = {1, 1}, down2[2] = {1, 1}, band = -INFINITY;
      auto clear = [&] {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[i] = m2[i] = -INFINITY;
          l[i] = l2[i] = 0;
        }
        band = -INFINITY;
      };
      clear();
      // the reference's weight, as a power of two
      const float off = BF ? -float(8 + 32 - __clz(seg.steps * NK)) : 12.f;
      bool first = true, rare = false;       // (see SharedRare)
      int from_half = 0;                     // of its first tile
      float ref[2], ref2[2];                 // and so what sums are relative to
      int j = -1;
      // Tile -1 stands for the row's query, which goes to shared memory.  In
      // the block's first one the weights are formed once of whatever tensor
      // memory holds and thrown away: so that their instructions, which come
      // from memory the first time (some 5000 cycles), are there when the first
      // scores are.
      for (;;) {
        if (j >= 0) {
          if (!warp_gate(s_full(q), n_s & 1, &dead)) {
            alive = false;
            break;
          }
          ++n_s;
          tmem_after_sync();
        }
        if (j >= 0 || nth == 0) {
          const char* const meta = metas + (t_first + max(j, 0)) % NM * S::kMeta;
          // (from the thread's first pair of columns on)
          const float2* const ku =
              reinterpret_cast<const float2*>(meta) + lane % 4;
          const uint32_t* const words =
              reinterpret_cast<const uint32_t*>(meta + NK * 12);
          // which of 32 keys are seen
          auto seen = [&](int c) {
            return KPW == 32 ? words[c]
                             : words[2 * c] | words[2 * c + 1] << 16;
          };
          // (Tile -1 takes no way that hangs on what is there: the masks of tile
          // 0 may just be written, and a warp whose lanes read them before and
          // after would come apart.)
          bool part = false;
#pragma unroll
          for (int c = 0; c < NK / 32; ++c) part |= seen(c) != 0xffffffffu;
          part = __any_sync(0xffffffffu, part && j >= 0);
          // Where scales of values lie within a few powers of two of each other,
          // their largest is taken for all of them in a row's reference.
          float most_of = 0;
          bool near = true;
          if (CODES) {
            const float4 lows =
                *reinterpret_cast<const float4*>(meta + NK * 12 + 16);
            const float4 tops =
                *reinterpret_cast<const float4*>(meta + NK * 12 + 32);
            const float least =
                fminf(fminf(lows.x, lows.y), fminf(lows.z, lows.w));
            most_of = fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w));
            near = !__any_sync(0xffffffffu, !(most_of - least < 4) && j >= 0);
            // (the loading warps' inverses are relative to their own keys'
            // bands, and good to 2^64)
            const float low =
                fminf(fminf(tops.x, tops.y), fminf(tops.z, tops.w));
            const float of = first ? scale_band(most_of) : band;
            if (__any_sync(0xffffffffu, !(most_of <= of && low > of - 32 &&
                                          least > of - 64) &&
                                            j >= 0)) {
              rare = true;
              break;
            }
            band = of;
          }
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            const uint32_t lanes = uint32_t(half * 16) << 16;
            uint32_t s[NK / 2];
            tmem_ld<NK / 8>(s, s_at + lanes);
            tmem_wait_ld();
            // columns 8g + 2 (t % 4) and the next of row i
            auto pair = [&](int g, int i) {
              return make_float2(__uint_as_float(s[4 * g + 2 * i]),
                                 __uint_as_float(s[4 * g + 2 * i + 1]));
            };
            if (part) {
              // -infinity where a key is not seen
#pragma unroll
              for (int g = 0; g < NK / 8; ++g) {
                const uint32_t mask =
                    seen(g / 4) >> (g % 4 * 8 + lane % 4 * 2);
#pragma unroll
                for (int k = 0; k < 2; ++k)
                  if (!(mask >> k & 1))
                    s[4 * g + k] = s[4 * g + 2 + k] = 0xff800000u;
              }
            }
            // the largest exponent, in units of ln 2
            float tops[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
#pragma unroll
            for (int g = 0; g < NK / 8; ++g) {
              float2 f = make_float2(1, 1);
              if (CODES) f = ku[4 * g];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float2 x = pair(g, i);
                if (CODES) x = mul2(x, f);
                if (CODES && !near)
                  x = fma2(x, make_float2(down[i], down[i]),
                           ku[NK / 2 + 4 * g]);
                tops[i][0] = fmaxf(tops[i][0], x.x);
                tops[i][1] = fmaxf(tops[i][1], x.y);
              }
            }
            float to[2];
            bool move = false, large = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float top = over_quad(fmaxf(tops[i][0], tops[i][1]));
              if (!CODES) top *= unit;
              if (CODES && near) top = __fmaf_rn(top, down[i], most_of);
              if (CODES) top -= band;
              // (by the difference: of numbers from 2^24 on the sum may be
              // rounded to more than the bound, and an f16 weight be infinite)
              to[i] = m[i];
              if (top - m[i] > SLACK) {
                to[i] = top;
                move = true;
                large |= fabsf(to[i]) > LARGE && fabsf(to[i]) < INFINITY;
              }
            }
            if (__any_sync(0xffffffffu, move)) {
              if (__any_sync(0xffffffffu, large && j >= 0)) {
                rare = true;
                from_half = half;
                break;
              }
              float keep[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                keep[i] = 1;
                if (to[i] != m[i]) {
                  // (in two halves: the whole may be below 2^-126 and, with
                  // small scales of values, the sum large)
                  keep[i] = ex2(0.5f * (m[i] - to[i]));
                  l[i] = l[i] * keep[i] * keep[i];
                  keep[i] *= keep[i];
                  m[i] = to[i];
                }
              }
              if (!first) scale_means(o_at + lanes, dim, keep);
            }
            float2 sub[2], by[2], sums[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float ref = m[i] == -INFINITY ? 0.f : m[i];
              const float x = CODES ? off - ref - band : off - ref;
              sub[i] = make_float2(x, x);
              by[i] = make_float2(down[i], down[i]);
              sums[i] = make_float2(0, 0);
            }
            uint32_t p[NK / 4];
#pragma unroll
            for (int g = 0; g < NK / 8; ++g) {
              float2 f, lv, inv;
              if (CODES) {
                f = ku[4 * g];
                lv = ku[NK / 2 + 4 * g];
                inv = ku[NK + 4 * g];
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float2 x = pair(g, i);
                if (CODES)
                  x = fma2(mul2(x, f), by[i], add2(lv, sub[i]));
                else
                  x = fma2(x, make_float2(unit, unit), sub[i]);
                x = make_float2(ex2(x.x), ex2(x.y));
                sums[i] = CODES ? fma2(x, inv, sums[i]) : add2(x, sums[i]);
                p[2 * g + i] = pair16<BF>(x.x, x.y);
              }
            }
            tmem_st_pairs<NK / 8>(s_at + lanes, p);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              l[i] += sums[i].x + sums[i].y;
              float t = m[i];
              m[i] = m2[i];
              m2[i] = t;
              t = l[i];
              l[i] = l2[i];
              l2[i] = t;
              t = down[i];
              down[i] = down2[i];
              down2[i] = t;
            }
          }
          if (rare) break;
          first = false;
          tmem_wait_st();
        }
        if (j >= 0) {
          tmem_before_sync();
          mbar_arrive(p_full(q));
          j += step;
        } else {
          clear();
          first = true;
          // the row's query, turned round where the scale is negative
          if (nth > 0 && !warp_gate(q_empty, (nth - 1) & 1, &dead)) {
            alive = false;
            break;
          }
          ++nth;
          const bool row_in = valid && a.scale != 0;
          auto load = [&](int c) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (row_in && c * 8 < dim)
              w = *reinterpret_cast<const uint4*>(query + c * 8);
            return w;
          };
          auto narrow = [&](int c) {       // of a row that allows no wide loads
            uint32_t x[4] = {0, 0, 0, 0};
            if (row_in && c * 8 < dim)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[i] = query[c * 8 + 2 * i] |
                       uint32_t(query[c * 8 + 2 * i + 1]) << 16;
            return make_uint4(x[0], x[1], x[2], x[3]);
          };
          // Codes are met by f16 queries, scaled by a power of two so that the
          // largest element lies in [2^14, 2^15): exact for bf16 elements down
          // to 2^-31 of it and f16 ones down to 2^-28, below that within 2^-39
          // of it.
          float up = 1;
          const bool in_bf = a.elem == LM_BF16;
          if (CODES) {
            float top = 0;
#pragma unroll 1
            for (int c = 0; c < dim16 / 8; ++c) {
              const uint4 w = a.q16 ? load(c) : narrow(c);
              const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = in_bf ? unpair16<true>(x[i])
                                       : unpair16<false>(x[i]);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            }
            int e = 14 + 127 - int(__float_as_uint(top) >> 23);
            if (top == 0 || top == INFINITY) e = 0;
            e = min(120, max(-120, e));
            up = __int_as_float((127 + e) << 23);
            const float back = __int_as_float((127 - e) << 23);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              down[i] = __shfl_sync(0xffffffffu, back, lane / 4 + 8 * i);
              down2[i] = __shfl_sync(0xffffffffu, back, 16 + lane / 4 + 8 * i);
            }
          }
          if (q * 128 < (split ? 128 : seg.rows)) {
            const uint32_t to = q_s + q * S::kQ + row * 128;
            auto store = [&](int c, const uint4& w) {
              uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (CODES) {
                  const float2 f = in_bf ? unpair16<true>(x[i])
                                         : unpair16<false>(x[i]);
                  x[i] = pair16<false>(f.x * up, f.y * up);
                }
                x[i] ^= flip;
              }
              if (c * 8 < dim16)
                st_smem16(to + c / 8 * (128 * 128) + ((c ^ row) & 7) * 16,
                          x[0], x[1], x[2], x[3]);
            };
            if (a.q16) {
#pragma unroll 1
              for (int c0 = 0; c0 < dim16 / 8; c0 += 16) {
                uint4 w[16];
#pragma unroll
                for (int c = 0; c < 16; ++c) w[c] = load(c0 + c);
#pragma unroll
                for (int c = 0; c < 16; ++c) store(c0 + c, w[c]);
              }
            } else {
#pragma unroll 1
              for (int c = 0; c < dim16 / 8; ++c) store(c, narrow(c));
            }
          }
          smem_to_products();
          tmem_before_sync();
          mbar_arrive(q_full);
          if (!active) break;
          j = split ? q : 0;
        }
        if (j >= seg.steps) break;
      }
      if (rare) {
        SharedRare r;
        r.s_at = s_at;
        r.o_at = o_at;
        r.dim = dim;
        r.off = off;
        r.unit = unit;
        r.band = band;
        r.first = first;
        r.half = from_half;
        const float low = __int_as_float((127 - int(off)) << 23);  // 2^-off
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          // (the pairs change places after each half)
          r.m[i] = from_half ? m2[i] : m[i];
          r.m[2 + i] = from_half ? m[i] : m2[i];
          r.l[i] = (from_half ? l2[i] : l[i]) * low;
          r.l[2 + i] = (from_half ? l[i] : l2[i]) * low;
          r.down[i] = from_half ? down2[i] : down[i];
          r.down[2 + i] = from_half ? down[i] : down2[i];
          r.ref[i] = r.m[i];
          r.ref[2 + i] = r.m[2 + i];
        }
        for (;;) {
          r.meta = metas + (t_first + j) % NM * S::kMeta;
          if constexpr (CODES)
            shared_rare<BF, true, NK>(&r);
          else
            shared_rare_rows<BF, NK>(&r);
          tmem_wait_st();
          tmem_before_sync();
          mbar_arrive(p_full(q));
          j += step;
          if (j >= seg.steps) break;
          if (!warp_gate(s_full(q), n_s & 1, &dead)) {
            alive = false;
            break;
          }
          ++n_s;
          tmem_after_sync();
        }
        first = false;
        band = r.band;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          m[i] = r.m[i];
          m2[i] = r.m[2 + i];
          l[i] = r.l[i];
          l2[i] = r.l[2 + i];
          ref[i] = r.ref[i];
          ref2[i] = r.ref[2 + i];
        }
      }
      if (!alive) break;
      // --- the rows' states ---
      if (!active) continue;
      const bool none = first;                   // no tile of keys
      if (!none) {
        if (!warp_gate(o_full(q), n_o & 1, &dead)) break;
        ++n_o;
        tmem_after_sync();
      }
      const bool whole = seg.steps == seg.s.tiles;
      const int sub = split ? q : 0;
      float* const part =
          a.parts + (2 * int64_t(blockIdx.x) +
                     (share.begin < seg.item_at ? 1 : 0)) *
                        (int64_t(S::kRows) * (D + 2));
      // where the rows' pieces will be: the block of tile i of the line is
      // ((i + 1) parts - 1) / total, and none of them is without any
      const int pieces =
          seg.t0 == 0 && sub == 0
              ? int(small_div((seg.item_at + seg.s.tiles) * share.parts - 1,
                              share.total) -
                    blockIdx.x) +
                    1
              : 0;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const uint32_t lanes = uint32_t(half * 16) << 16;
        float f[2], f2[2] = {1, 1};
        float* to[2];                // a row's mean, NULL where there is none
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int in = warp % 4 * 32 + half * 16 + lane / 4 + 8 * i;
          const int r = split ? in : q * 128 + in;
          const int rg = seg.rt * S::kRows + r, si = rg / a.group;
          const int64_t out_row =
              int64_t(sub) * a.seqs * a.heads_q +
              int64_t(seg.s.start + si) * a.heads_q + seg.h * a.group +
              (rg - si * a.group);
          const int part_row = q * 128 + in;
          float sum = l[i];
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          // weights were taken times 2^off, and relative to m and the band; the
          // sum is relative to m, or to a reference of its own and without 2^off
          const float low = __int_as_float((127 - int(off)) << 23);
          float from = m[i];
          if (rare)
            from = ref[i];
          else
            sum *= low;
          f[i] = sum == 0 ? 0.f : __fdividef(low, sum);
          if (CODES || rare) {
            // (in two halves: the whole may be past 32 bits' range)
            f2[i] = ex2(0.5f * ((CODES ? band : 0.f) + (m[i] - from)));
            f[i] = sum == 0 ? 0.f : f[i] * f2[i];
          }
          to[i] = nullptr;
          if (r < seg.rows) {
            to[i] = whole ? a.mean + out_row * dim
                          : part + 2 * S::kRows + part_row * D;
            if (lane % 4 == 0) {
              // (the sum's exponent goes to the reference, where that holds it:
              // next to scales of values the sum may be of any size, and
              // references far apart then say nothing about weights)
              const int e = int(__float_as_uint(sum) >> 23) - 127;
              float2 ml = make_float2(from, sum);
              if (CODES && sum > 0x1p-120f && sum < INFINITY &&
                  fabsf(from) < 0x1p14f) {
                ml.x += float(e);
                ml.y *= __int_as_float((127 - e) << 23);
              }
              if (whole)
                reinterpret_cast<float2*>(a.state)[out_row] = ml;
              else
                reinterpret_cast<float2*>(part)[part_row] = ml;
              if (pieces > 0)
                reinterpret_cast<int4*>(a.pieces)[out_row] = make_int4(
                    pieces,
                    2 * int(blockIdx.x) + (share.begin < seg.item_at ? 1 : 0),
                    2 * int(blockIdx.x) + 2, part_row | (split ? 65536 : 0));
            }
          }
        }
        if (!none) {
#pragma unroll 1
          for (int c = 0; c < dim; c += 32) {
            uint32_t x[16];
            __syncwarp();
            tmem_ld<4>(x, o_at + lanes + c);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                const int d = c + g * 8 + lane % 4 * 2;
                if (to[i] && d < dim)
                  *reinterpret_cast<float2*>(to[i] + d) = make_float2(
                      __uint_as_float(x[4 * g + 2 * i]) * f[i] * f2[i],
                      __uint_as_float(x[4 * g + 2 * i + 1]) * f[i] * f2[i]);
              }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float t = m[i];
          m[i] = m2[i];
          m2[i] = t;
          t = l[i];
          l[i] = l2[i];
          l2[i] = t;
          ref[i] = ref2[i];
        }
      }
      if (!none) {
        __syncwarp();
        tmem_before_sync();
        mbar_arrive(o_empty(q));
      }
    }
  }

  __syncthreads();
  if (warp == 12) {
    tmem_after_sync();
    tmem_free(tmem, 512);
  }
  if (threadIdx.x == 0 && dead && a.status) atomicOr(a.status, kStatusTimeout);
}

template <bool BF, int STORE, int D>
int launch_shared_d(const KvSharedArgs& a, cudaStream_t st) {
  using S = SharedShape<D>;
  int sms = 0, dev = 0;
  const int rc = kv_device(&dev, &sms);
  if (rc != LM_OK) return rc;
  auto* kernel = lm_kv_shared_kernel<BF, STORE, D>;
  static std::atomic<uint64_t> allowed{0};    // a bit per device
  if (!(allowed.load() >> dev & 1)) {
    const cudaError_t e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) {
      set_cuda_error(int(e));
      return LM_E_CUDA;
    }
    allowed.fetch_or(uint64_t(1) << dev);
  }
  return launch(kernel, sms, kSharedThreads, S::kSmem, st, a);
}

template <bool BF, int STORE>
int launch_shared_store(const KvSharedArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int d = shared_dim(a.c.dim);
  return d == 64    ? launch_shared_d<BF, STORE, 64>(a, st)
         : d == 128 ? launch_shared_d<BF, STORE, 128>(a, st)
                    : launch_shared_d<BF, STORE, 256>(a, st);
}

}  // namespace lm
