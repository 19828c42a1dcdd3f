// Which pages a sparse attention reads: the bounds of a page's keys, and the
// choice of the pages whose bounds promise the largest products.
//
// For a page and key head, lo_d and hi_d are the least and the largest element
// d of its keys.  sum_d (c_d > 0 ? c_d hi_d : c_d lo_d) is no less than the
// product of c with any of them, so it ranks pages without their keys: 2 dim
// bytes for a page of P keys of 2 dim bytes each.  Bounds are held as whole
// numbers, lo rounded down and hi up, under a power of two, and the query as
// whole numbers under one of its own: products and their sums are whole numbers below 2^24,
// the same in any order and in 32-bit floats, so that ties are ties and the
// choice depends on nothing but the inputs.
#include <type_traits>

#include "lm_kv_long.h"
#include "lm_kv_top.cuh"
#include "lm_line.cuh"

namespace lm {
namespace {

// The exponent e >= -126 of the smallest power of two with top / 2^e <= 127 =
// 1.984375 * 2^6, from the bits of a finite top > 0.
__device__ __forceinline__ int power_of(uint32_t top) {
  const int e =
      int(top >> 23) - 127 - ((top & 0x7fffffu) <= 0x7e0000u ? 6 : 5);
  return max(e, -126);
}
__device__ __forceinline__ float pow2f(int e) {
  return __int_as_float((127 + e) << 23);
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;\n" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Of two pairs of 16-bit elements.
template <class T>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  uint32_t y;
  if (std::is_same<T, bf16>::value)
    asm("min.NaN.bf16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
template <class T>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t y;
  if (std::is_same<T, bf16>::value)
    asm("max.NaN.bf16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;\n" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// --- bounds ----------------------------------------------------------------

constexpr int kBoundThreads = 128;

// A warp has one page and head: L lanes hold a row in 16-byte chunks, 32 / L
// of them take turns with the tokens, kAhead loads each in flight.  It is one
// pass over the keys: 8 x 8192 tokens x 8 x 128 bf16 (81 MB) 17 us, 4.8 TB/s or
// 71% of a copy's rate, 20 us with elements widened to 32 bits one by one.  A
// page of 16 tokens is one batch of loads behind two that wait for each other
// (its number and count), and the warp ends: its loads fly for a part of its life.
template <class T, int STORE, int L>
__global__ void __launch_bounds__(kBoundThreads, STORE == LM_KV_SAME ? 8 : 4)
    lm_kv_bound_kernel(const __grid_constant__ KvBoundArgs a) {
  constexpr int N = STORE == LM_KV_SAME ? 8 : 16;   // elements of a chunk
  constexpr int TL = 32 / L;                        // tokens at once
  constexpr int kAhead = 8;
  stream_order();
  const int lane = threadIdx.x % 32, c = lane % L, t0 = lane / L;
  const uint32_t unit =
      blockIdx.x * (kBoundThreads / 32) + threadIdx.x / 32;
  const uint32_t i = fdiv(unit, a.heads_div), h = unit - i * a.c.heads;
  if (i >= a.n) return;
  const int64_t page = a.pages[i];
  if (page < 0 || page >= a.c.pages) {
    if (page >= 0 && lane == 0 && a.status) atomicOr(a.status, kStatusRange);
    return;
  }
  const int count = min(max(a.counts[i], 0), int(a.c.page_tokens));
  const bool has = c * N < a.c.dim;
  const char* src = a.c.k + page * a.c.page_b + int64_t(h) * a.c.head_b +
                    int64_t(t0) * a.c.token_b + c * 16;
  const float* scales =
      a.c.ks + (page * a.c.heads + h) * a.c.page_tokens + t0;
  float lo[N], hi[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    lo[e] = INFINITY;
    hi[e] = -INFINITY;
  }
  // (16-bit rows two elements at a time, as they are)
  uint32_t lo2[4], hi2[4];
  if (STORE == LM_KV_SAME) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float inf[2] = {INFINITY, INFINITY};
      const float minus[2] = {-INFINITY, -INFINITY};
      lo2[e] = Word<T>::put(inf);
      hi2[e] = Word<T>::put(minus);
    }
  }
  if (has)
    for (int t = t0; t < count; t += TL * kAhead) {
      uint4 w[kAhead];
      float scale[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        scale[k] = 1;
        if (t + k * TL >= count) continue;
        w[k] = *reinterpret_cast<const uint4*>(
            src + int64_t(t - t0 + k * TL) * a.c.token_b);
        if (STORE != LM_KV_SAME) scale[k] = scales[t - t0 + k * TL];
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (t + k * TL >= count) continue;
        if (STORE == LM_KV_SAME) {
          const uint32_t r[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            lo2[e] = min2_nan<T>(lo2[e], r[e]);
            hi2[e] = max2_nan<T>(hi2[e], r[e]);
          }
        } else {
          float x[N];
          held_values<T, STORE>(w[k], scale[k], x);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            lo[e] = min_nan(lo[e], x[e]);
            hi[e] = max_nan(hi[e], x[e]);
          }
        }
      }
    }
  if (STORE == LM_KV_SAME) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int k = L; k < 32; k *= 2) {
        lo2[e] = min2_nan<T>(lo2[e], __shfl_xor_sync(0xffffffffu, lo2[e], k));
        hi2[e] = max2_nan<T>(hi2[e], __shfl_xor_sync(0xffffffffu, hi2[e], k));
      }
      Word<T>::get(lo2[e], lo + 2 * e);
      Word<T>::get(hi2[e], hi + 2 * e);
    }
  }
  float top = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
#pragma unroll
    for (int k = STORE == LM_KV_SAME ? 32 : L; k < 32; k *= 2) {
      lo[e] = min_nan(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], k));
      hi[e] = max_nan(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], k));
    }
    if (has) top = max_nan(top, max_nan(fabsf(lo[e]), fabsf(hi[e])));
  }
#pragma unroll
  for (int k = 1; k < L; k *= 2)
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, k));
  // no tokens, or nothing but zeros; a key that is no number, or infinite
  float scale = 1, by = 0;
  if (count == 0) {
    top = 0;
  } else if (!(top < INFINITY)) {
    scale = __int_as_float(0x7fc00000);
  } else if (top > 0) {
    const int e = power_of(__float_as_uint(top));
    scale = pow2f(e);
    by = pow2f(-e);
  }
  if (!has || t0 > 0) return;
  const bool zero = by == 0;
  int8_t* to = a.bounds + (page * a.c.heads + h) * 2 * a.c.dim + c * N;
  uint32_t y[2][N / 4];
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    uint32_t l = 0, u = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // (outwards twice: beside a large key a small one's product lies below
      // 2^-150, and to the nearest number of 32 bits it would be 0)
      const int f = zero ? 0 : __float2int_rd(__fmul_rd(lo[e + k], by));
      const int g = zero ? 0 : __float2int_ru(__fmul_ru(hi[e + k], by));
      l |= uint32_t(f & 0xff) << (8 * k);
      u |= uint32_t(g & 0xff) << (8 * k);
    }
    y[0][e / 4] = l;
    y[1][e / 4] = u;
  }
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int e = 0; e < N / 4; e += 2)
      *reinterpret_cast<uint2*>(to + side * a.c.dim + e * 4) =
          make_uint2(y[side][e], y[side][e + 1]);
  if (c == 0) a.scale[page * a.c.heads + h] = scale;
}

// --- scores ----------------------------------------------------------------

constexpr int kScoreThreads = 256;
constexpr int kScorePages = 32;      // of a warp's unit

// D += A B: 16 rows by 32 whole numbers of 8 bits, those by 8 columns.
__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4],
                                       uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A unit is kScorePages pages of one sequence and head, two products of 16
// pages by 8 queries: hi meets the queries' positive parts and lo their
// negative ones, in KS steps of 32 elements each.  A sum has no order, so that
// of a step's elements lane t % 4 takes 8 side by side, 32 bytes of a row a
// quad.  What bounds it are the loads, one after the other, of a unit's pages,
// bounds and queries: 32 sequences x up to 1024 pages x 8 heads x 4 queries of
// 128 elements (47 MB of bounds) 20 us, 13 sequences x 500 pages x 4 x 5 x 64
// 7.8.  Three blocks an SM with one product's rows on their way, or two with
// both: 20 against 23 us for the first, 8.4 against 7.8 for the second; three
// spill 88 bytes, the form for 256 elements at two blocks 184.  (Byte products on
// the vector units, sums exchanged between lanes: 24 and 11.)
template <class T, int KS>
__global__ void __launch_bounds__(kScoreThreads, KS == 4 ? 3 : 2)
    lm_kv_score_kernel(const __grid_constant__ KvSelectArgs a) {
  constexpr int kRounds = KS == 2 ? 2 : 1;  // of 16 pages, loaded together
  stream_order();
  auto pages_of = [&](int b) {
    const int64_t most = a.max_pages * a.page_tokens;
    int64_t n = a.lens[b];
    n = n < 0 ? 0 : n > most ? most : n;
    return int((n + a.page_tokens - 1) / a.page_tokens);
  };
  // a sequence that keeps all of its pages needs no scores
  auto tiles_of = [&](int b) {
    const int n = pages_of(b);
    return n <= a.keep ? 0 : (n + kScorePages - 1) / kScorePages;
  };
  LineShare at = line_share<kScoreThreads>(
      a.seqs, blockIdx.x, gridDim.x,
      [&](int b) { return int64_t(tiles_of(b)) * a.heads; });
  if (at.left <= 0) return;
  const int lane = threadIdx.x % 32, c = lane % 4, r = lane / 4;
  const int warp = threadIdx.x / 32;
  // this warp's units: every eighth of the block's
  int tiles = tiles_of(at.b);
  at.in += warp;
  at.left -= warp;
  for (; at.left > 0; at.left -= kScoreThreads / 32) {
    while (at.in >= int64_t(tiles) * a.heads) {
      // (never, unless the lengths change while the kernel runs)
      if (at.b + 1 >= a.seqs) return;
      at.in -= int64_t(tiles) * a.heads;
      tiles = tiles_of(++at.b);
    }
    // the heads of a tile of pages one after the other: their bounds are
    const int tile = int(small_div(at.in, a.heads));
    const uint32_t h = uint32_t(at.in - int64_t(tile) * a.heads);
    at.in += kScoreThreads / 32;
    const int p0 = tile * kScorePages, pages = pages_of(at.b);
    const int p1 = min(pages, p0 + kScorePages);
    const int mine = p0 + lane < p1
                         ? a.table[at.b * a.table_stride + p0 + lane]
                         : -1;
    const bool there = mine >= 0 && mine < a.pages;
    // (a power of two or NaN: it multiplies the largest of the queries' as well
    // as each)
    const float scale =
        there ? a.bound_scale[int64_t(mine) * a.heads + h] : 0.f;
    float best = -INFINITY;            // of page p0 + lane
    for (int g0 = 0; g0 < a.group; g0 += 8) {
      // query g0 + r as whole numbers
      uint32_t qp[KS][2], qn[KS][2], raw[KS][4];
      float top = 0;
      const bool is = g0 + r < a.group;
      const T* const q = reinterpret_cast<const T*>(a.q.p) +
                         int64_t(at.b) * a.q.ts +
                         int64_t(h * a.group + g0 + (is ? r : 0)) * a.q.hs;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const int d = (4 * k + c) * 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) raw[k][e] = 0;
        if (is && d < a.dim) {
          if (a.q16) {
            const uint4 w = *reinterpret_cast<const uint4*>(q + d);
            raw[k][0] = w.x;
            raw[k][1] = w.y;
            raw[k][2] = w.z;
            raw[k][3] = w.w;
          } else {
            const uint16_t* const y = reinterpret_cast<const uint16_t*>(q + d);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              raw[k][e] = y[2 * e] | uint32_t(y[2 * e + 1]) << 16;
          }
        }
        float x[8];
        get_words<T, 4>(raw[k], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max_nan(top, fabsf(x[e]));
      }
      top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float by = 0, unit = 1;
      if (!(top < INFINITY)) {
        unit = __int_as_float(0x7fc00000);
      } else if (top > 0) {
        const int e = power_of(__float_as_uint(top));
        unit = pow2f(e);
        by = pow2f(-e);
      }
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        float x[8];
        get_words<T, 4>(raw[k], x);
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          qp[k][w] = qn[k][w] = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int v = by == 0 ? 0 : __float2int_rn(x[4 * w + e] * by);
            qp[k][w] |= uint32_t(max(v, 0)) << (8 * e);
            qn[k][w] |= uint32_t(min(v, 0) & 0xff) << (8 * e);
          }
        }
      }
      // those of a product's columns that this lane has
      const bool is0 = g0 + 2 * c < a.group, is1 = g0 + 2 * c + 1 < a.group;
      const float unit0 = __shfl_sync(0xffffffffu, unit, 8 * c);
      const float unit1 = __shfl_sync(0xffffffffu, unit, 8 * c + 4);
#pragma unroll 1
      for (int p = 0; p < p1 - p0; p += 16 * kRounds) {
        uint2 lo[kRounds][2][KS], hi[kRounds][2][KS];
#pragma unroll
        for (int n = 0; n < kRounds; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int64_t page =
                __shfl_sync(0xffffffffu, mine, p + 16 * n + 8 * i + r);
            const bool ok = page >= 0 && page < a.pages;
            const int8_t* const from =
                a.bounds + ((ok ? page : 0) * a.heads + h) * 2 * a.dim;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              const int d = (4 * k + c) * 8;
              lo[n][i][k] = hi[n][i][k] = make_uint2(0, 0);
              if (ok && d < a.dim) {
                lo[n][i][k] = *reinterpret_cast<const uint2*>(from + d);
                hi[n][i][k] = *reinterpret_cast<const uint2*>(from + a.dim + d);
              }
            }
          }
#pragma unroll
        for (int n = 0; n < kRounds; ++n) {
          int s[4] = {0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            const uint32_t up[4] = {hi[n][0][k].x, hi[n][1][k].x,
                                    hi[n][0][k].y, hi[n][1][k].y};
            const uint32_t down[4] = {lo[n][0][k].x, lo[n][1][k].x,
                                      lo[n][0][k].y, lo[n][1][k].y};
            mma_s8(s, up, qp[k][0], qp[k][1]);
            mma_s8(s, down, qn[k][0], qn[k][1]);
          }
          // of rows r and r + 8 the largest over the queries
          float y[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            y[i] = is0 ? float(s[2 * i]) * unit0 : -INFINITY;
            if (is1) y[i] = max_nan(y[i], float(s[2 * i + 1]) * unit1);
            y[i] = max_nan(y[i], __shfl_xor_sync(0xffffffffu, y[i], 1));
            y[i] = max_nan(y[i], __shfl_xor_sync(0xffffffffu, y[i], 2));
          }
          // to the lane that has the page
          const float y0 = __shfl_sync(0xffffffffu, y[0], lane % 8 * 4);
          const float y1 = __shfl_sync(0xffffffffu, y[1], lane % 8 * 4);
          if (lane / 16 == p / 16 + n)
            best = max_nan(best, lane & 8 ? y1 : y0);
        }
      }
    }
    if (p0 + lane < p1) {
      if (!there && h == 0 && a.status) atomicOr(a.status, kStatusRange);
      a.scores[(int64_t(at.b) * a.heads + h) * a.max_pages + p0 + lane] =
          there ? best * scale : -INFINITY;
    }
  }
}

// --- the choice --------------------------------------------------------------

// A cluster of C blocks has one sequence and head.  Its steps wait for one
// another: 256 lists of 1024 pages 11 us, 8 lists of 8192 17.5.
template <int T, int C>
__global__ void __launch_bounds__(T)
    lm_kv_select_kernel(const __grid_constant__ KvSelectArgs a, int cap) {
  extern __shared__ uint32_t cache[];
  __shared__ TopSpace<T> sh;
  stream_order();
  const int unit = blockIdx.x / C, rank = blockIdx.x % C;
  const int b = unit / int(a.heads), h = unit - b * int(a.heads);
  const int64_t most = a.max_pages * a.page_tokens;
  int64_t len = a.lens[b];
  len = len < 0 ? 0 : len > most ? most : len;
  const int n = int((len + a.page_tokens - 1) / a.page_tokens);
  const int count = min(n, a.keep);
  const int32_t* table = a.table + b * a.table_stride;
  int32_t* to = a.selected + int64_t(unit) * a.keep;
  if (h == 0 && rank == 0 && threadIdx.x == 0)
    a.selected_lens[b] =
        int32_t(len - int64_t(n - count) * a.page_tokens);
  // (numbers without a sign: one past a list of 2^31 - 1 is still one)
  const uint32_t threads = T * C, me = rank * T + threadIdx.x;
  for (uint32_t i = count + me; i < uint32_t(a.keep); i += threads) to[i] = -1;
  if (n <= a.keep) {
    for (uint32_t i = me; i < uint32_t(n); i += threads) to[i] = table[i];
    return;
  }
  for (uint32_t i = me; i < uint32_t(a.first); i += threads) to[i] = table[i];
  for (uint32_t i = me; i < uint32_t(a.last); i += threads)
    to[uint32_t(a.keep - a.last) + i] = table[uint32_t(n - a.last) + i];
  const int need = a.keep - a.first - a.last;
  if (need == 0) return;
  const float* scores =
      a.scores + (int64_t(b) * a.heads + h) * a.max_pages + a.first;
  take_top<T, C>(
      n - a.first - a.last, need, cache, cap, &sh,
      [&](int i) { return order_of(scores[i]); },
      [&](int place, int i) {
        to[a.first + place] = table[a.first + i];
      });
}

template <class T>
int launch_score(const KvSelectArgs& a, int sms, cudaStream_t st) {
  auto run = [&](auto* kernel, int blocks) {
    return launch(kernel, uint64_t(sms) * blocks, kScoreThreads, 0, st, a);
  };
  return a.dim <= 64    ? run(lm_kv_score_kernel<T, 2>, 2)
         : a.dim <= 128 ? run(lm_kv_score_kernel<T, 4>, 3)
                        : run(lm_kv_score_kernel<T, 8>, 2);
}

template <class T, int STORE>
int launch_bound_s(const KvBoundArgs& a, cudaStream_t st) {
  const uint64_t units = uint64_t(a.n) * a.c.heads;
  const uint64_t grid = (units + kBoundThreads / 32 - 1) / (kBoundThreads / 32);
  const int bytes = a.c.dim * (STORE == LM_KV_SAME ? 2 : 1);
  if (bytes <= 128)
    return launch(lm_kv_bound_kernel<T, STORE, 8>, grid, kBoundThreads, 0, st, a);
  if (bytes <= 256)
    return launch(lm_kv_bound_kernel<T, STORE, 16>, grid, kBoundThreads, 0, st, a);
  return launch(lm_kv_bound_kernel<T, STORE, 32>, grid, kBoundThreads, 0, st, a);
}

}  // namespace

int launch_kv_bound(const KvBoundArgs& a, int elem, int store, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (store == LM_KV_E4M3) return launch_bound_s<bf16, LM_KV_E4M3>(a, st);
  if (store == LM_KV_INT8) return launch_bound_s<bf16, LM_KV_INT8>(a, st);
  return elem == LM_BF16 ? launch_bound_s<bf16, LM_KV_SAME>(a, st)
                         : launch_bound_s<__half, LM_KV_SAME>(a, st);
}

int launch_kv_select(const KvSelectArgs& a, int elem, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0, sms = 0;
  int rc = kv_device(&dev, &sms);
  if (rc != LM_OK) return rc;
  if (a.max_pages > a.keep) {
    rc = elem == LM_BF16 ? launch_score<bf16>(a, sms, st)
                         : launch_score<__half>(a, sms, st);
    if (rc != LM_OK) return rc;
  }
  const uint64_t lists = uint64_t(a.seqs) * a.heads;
  static std::atomic<uint64_t> allowed{0};    // a bit per device
  return launch_top(lm_kv_select_kernel<kTopThreads, 1>,
                    lm_kv_select_kernel<kTopMore, 1>,
                    lm_kv_select_kernel<kTopMore, kTopCluster>, &allowed, dev,
                    top_plan(int64_t(lists), a.max_pages, sms), lists, st, a);
}

}  // namespace lm
