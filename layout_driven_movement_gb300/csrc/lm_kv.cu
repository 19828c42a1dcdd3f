// The paged cache's write (rotating and quantising) and its read back.
#include "lm_kv_device.cuh"

namespace lm {
namespace {

// --- write -----------------------------------------------------------------

// The scale of a row from the bits of its largest magnitude, and what its
// elements are multiplied by (INT8: the last 32-bit number up to 127 / max|x|,
// the one above it is the next).  E4M3: 448 = 1.75 * 2^8, so with max|x| =
// m * 2^E, 1 <= m < 2, the smallest e with max|x| <= 448 * 2^e is E - 8 for
// m <= 1.75 and E - 7 above; 2^-e multiplies exactly.
template <int STORE>
__device__ __forceinline__ float row_scale(uint32_t top, float* by) {
  if (top >= 0x7f800000u) {
    *by = 0;
    return __int_as_float(0x7fc00000);
  }
  if (top == 0) {
    *by = 0;
    return 1.f;
  }
  if (STORE == LM_KV_E4M3) {
    int e = int(top >> 23) - 127 - ((top & 0x7fffffu) <= 0x600000u ? 8 : 7);
    if (e < -126) e = -126;
    *by = __int_as_float((127 - e) << 23);
    return __int_as_float((127 + e) << 23);
  }
  const float m = __uint_as_float(top);
  *by = fminf(__fdiv_rn(127.f, m), 0x1p126f);
  if (__fmaf_rn(-*by, m, 127.f) < 0)
    *by = __int_as_float(__float_as_int(*by) - 1);
  return fmaxf(__fdiv_rn(m, 127.f), 0x1p-126f);
}

// 8 elements' codes.  Whole numbers: with 1.5 * 2^23 added a product's last bit
// is 1, so it is rounded to a whole one, once, whose low byte is the sum's.  An
// element exactly between two codes (x = max / 2 is one) gets the lower one
// from the factor up to 127 / max|x| and the upper one from the next, any other
// the same from both: the even one of the two is the formula's.
template <int STORE>
__device__ __forceinline__ uint2 row_codes(const float* x, float by) {
  uint32_t w[2];
  const float next = __int_as_float(__float_as_int(by) + 1);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (STORE == LM_KV_E4M3) {
      const uint32_t a = __nv_cvt_float2_to_fp8x2(
          make_float2(x[4 * i] * by, x[4 * i + 1] * by), __NV_SATFINITE,
          __NV_E4M3);
      const uint32_t b = __nv_cvt_float2_to_fp8x2(
          make_float2(x[4 * i + 2] * by, x[4 * i + 3] * by), __NV_SATFINITE,
          __NV_E4M3);
      w[i] = a | b << 16;
    } else {
      auto codes = [&](float f) {
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r[j] = __float_as_uint(__fmaf_rn(x[4 * i + j], f, 12582912.f));
        return __byte_perm(__byte_perm(r[0], r[1], 0x0040),
                           __byte_perm(r[2], r[3], 0x0040), 0x5410);
      };
      const uint32_t lower = codes(by), upper = codes(next);
      const uint32_t odd = (upper & 0x01010101u) * 0xffu;
      w[i] = (lower & odd) | (upper & ~odd);
    }
  }
  return make_uint2(w[0], w[1]);
}

// The largest magnitude of 8, NaN above all, as bits.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;\n" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ uint32_t top_of(const float* x) {
  const float a = max3(x[0], x[1], x[2]), b = max3(x[3], x[4], x[5]);
  return __float_as_uint(max3(max3(x[6], x[7], a), b, 0.f));
}

// A row's 8 elements at `at`, as words; one 16-byte load when the rows allow
// it.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int at) {
  if (VEC) return *reinterpret_cast<const uint4*>(row + at);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = row[at + 2 * i] | uint32_t(row[at + 2 * i + 1]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <class T>
__device__ __forceinline__ void get8(const uint4& u, float* x) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  get_words<T, 4>(w, x);
}

// L lanes hold a row in chunks of 8 elements, lane c the chunks c and c + L of
// a key and of its value: four 16-byte loads are in flight before the first is
// used, a row's largest magnitude is log2 L shuffles away, its codes leave as
// 8-byte stores of adjacent lanes, and the turn of a whole row of 16 L
// elements (partners 8 L apart) stays inside a thread, one cosine and sine
// for both partners.  Bound by memory: inputs read once, codes written once (8
// sequences of up to 8192 tokens of 8 x 128 into e4m3, 234 MB: 35 us, 6.6
// TB/s).  With the turn, 49 us, the angles' loads (a quarter of the rows' bytes
// again, from L2) and the turn's instructions show: a third of the issue slots
// go to the roundings as it is.
//
// TURN: 0 no turn, 1 partners 8 L apart, 2 any other.  Two heads a thread, to
// share a token's slot and angles, leave fewer warps resident and gain 3% (8 x
// 8192 tokens of 8 x 128 turned into e4m3: 47.7 us against 49.2): not kept.
template <class T, int STORE, int L, bool VEC, int TURN>
__global__ void __launch_bounds__(256, TURN == 0 ? 6 : 4) lm_kv_write_kernel(
    const __grid_constant__ KvWriteArgs a) {
  stream_order();
  const uint32_t row = (blockIdx.x * 256 + threadIdx.x) / L;
  const int c = int(threadIdx.x % L);
  const bool live = row < a.tokens * a.c.heads;
  const uint32_t t = live ? fdiv(row, a.heads_div) : 0;
  const uint32_t h = live ? row - t * a.c.heads : 0;
  const int at[2] = {c * 8, (c + L) * 8};
  const bool has[2] = {at[0] < a.c.dim, at[1] < a.c.dim};
  const uint16_t* k = reinterpret_cast<const uint16_t*>(a.k.p) +
                      int64_t(t) * a.k.ts + int64_t(h) * a.k.hs;
  const uint16_t* v = reinterpret_cast<const uint16_t*>(a.v.p) +
                      int64_t(t) * a.v.ts + int64_t(h) * a.v.hs;
  uint4 xr[2][2];                            // key or value, chunk
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    xr[0][p] = xr[1][p] = make_uint4(0, 0, 0, 0);
    if (live && has[p]) {
      xr[0][p] = load8<VEC>(k, at[p]);
      xr[1][p] = load8<VEC>(v, at[p]);
    }
  }
  const int64_t slot = live ? a.slots[t] : -1;
  const int half = a.turn.rot / 2;
  const float* tr = nullptr;
  float cs[8], sn[8];
  const float nan = __int_as_float(0x7fc00000);
  if (TURN && live && a.turn.pos) {
    // (a skipped token's position may be anything)
    tr = turn_row(a.turn, t, c == 0 && slot >= 0 ? a.status : nullptr);
    if (TURN == 1) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(cs + i) =
            tr ? *reinterpret_cast<const float4*>(tr + at[0] + i)
               : make_float4(nan, nan, nan, nan);
        *reinterpret_cast<float4*>(sn + i) =
            tr ? *reinterpret_cast<const float4*>(tr + half + at[0] + i)
               : make_float4(nan, nan, nan, nan);
      }
    }
  }
  const int64_t tokens = a.c.pages * int64_t(a.c.page_tokens);
  if (slot >= tokens && c == 0 && a.status) atomicOr(a.status, kStatusRange);
  const bool to = slot >= 0 && slot < tokens;
  int64_t page = 0;
  if (to)
    page = tokens <= INT32_MAX ? int64_t(fdiv(uint32_t(slot), a.c.page_div))
                               : slot / a.c.page_tokens;
  const uint32_t off = to ? uint32_t(slot - page * a.c.page_tokens) : 0;
  const int64_t base = page * a.c.page_b + int64_t(off) * a.c.token_b +
                       int64_t(h) * a.c.head_b;

#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float x[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p) get8<T>(xr[kv][p], x[p]);
    if (TURN == 1 && kv == 0 && live) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = x[0][i], w = x[1][i];
        x[0][i] = turn_lo(u, w, cs[i], sn[i]);
        x[1][i] = turn_hi(u, w, cs[i], sn[i]);
      }
    }
    if (TURN == 2 && kv == 0 && live) {
      // part of a row, odd halves or interleaved pairs: an element's partner
      // and angle one by one (their lines are at hand)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float own[8];
        get8<T>(xr[0][p], own);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = at[p] + i;
          if (e >= a.turn.rot) continue;
          const bool first = a.turn.inter ? i % 2 == 0 : e < half;
          const int n = a.turn.inter ? e / 2 : first ? e : e - half;
          const float o =
              a.turn.inter
                  ? own[i ^ 1]
                  : to_f32(reinterpret_cast<const T*>(
                        k)[first ? e + half : e - half]);
          const float cn = tr ? tr[n] : nan, s = tr ? tr[half + n] : nan;
          x[p][i] = first ? turn_lo(own[i], o, cn, s)
                          : turn_hi(o, own[i], cn, s);
        }
      }
    }
    char* dst = (kv ? a.c.v : a.c.k) + base;
    if (STORE == LM_KV_SAME) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint4 y = xr[kv][p];
        if (kv == 0 && TURN && at[p] < a.turn.rot) {
          // what is not turned keeps its bits
          const uint32_t* raw = reinterpret_cast<const uint32_t*>(&xr[0][p]);
          uint32_t w[4];
          put_words<T, 4>(x[p], w);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (at[p] + 2 * i >= a.turn.rot) w[i] = raw[i];
          y = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (to && has[p]) *reinterpret_cast<uint4*>(dst + at[p] * 2) = y;
      }
      continue;
    }
    uint32_t top = max(top_of(x[0]), top_of(x[1]));
#pragma unroll
    for (int m = L / 2; m; m /= 2)
      top = max(top, __shfl_xor_sync(0xffffffffu, top, m, L));
    float by;
    const float scale = row_scale<STORE>(top, &by);
    if (to) {
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (has[p])
          *reinterpret_cast<uint2*>(dst + at[p]) =
              top < 0x7f800000u ? row_codes<STORE>(x[p], by)
                                : make_uint2(0, 0);
      if (c == 0)
        (kv ? a.c.vs : a.c.ks)[(page * a.c.heads + h) * a.c.page_tokens +
                               off] = scale;
    }
  }
}

template <class T, int STORE, int L>
int launch_write_l(const KvWriteArgs& a, cudaStream_t st) {
  const uint64_t threads = uint64_t(a.tokens) * a.c.heads * L;
  const uint64_t grid = (threads + 255) / 256;
  auto run = [&](auto* kernel) { return launch(kernel, grid, 256, 0, st, a); };
  // (dim == 16 L: whole chunks, every lane has both)
  const bool own = a.table16 && !a.turn.inter && a.turn.rot == 16 * L;
  if (!a.vec) return run(lm_kv_write_kernel<T, STORE, L, false, 2>);
  if (!a.turn.pos) return run(lm_kv_write_kernel<T, STORE, L, true, 0>);
  if (own) return run(lm_kv_write_kernel<T, STORE, L, true, 1>);
  return run(lm_kv_write_kernel<T, STORE, L, true, 2>);
}

template <class T, int STORE>
int launch_write_s(const KvWriteArgs& a, cudaStream_t st) {
  if (a.c.dim <= 64) return launch_write_l<T, STORE, 4>(a, st);
  if (a.c.dim <= 128) return launch_write_l<T, STORE, 8>(a, st);
  return launch_write_l<T, STORE, 16>(a, st);
}

template <class T>
int launch_write_t(const KvWriteArgs& a, int store, cudaStream_t st) {
  if (store == LM_KV_E4M3) return launch_write_s<T, LM_KV_E4M3>(a, st);
  if (store == LM_KV_INT8) return launch_write_s<T, LM_KV_INT8>(a, st);
  return launch_write_s<T, LM_KV_SAME>(a, st);
}

// --- read ------------------------------------------------------------------

// 16 held bytes as 32-bit values: 16 codes times their scale, or 8 elements.
template <class T, int STORE>
__device__ __forceinline__ void held_values(const uint4& w, float scale,
                                            float* x) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
  if (STORE == LM_KV_SAME) {
    get_words<T, 4>(r, x);
  } else if (STORE == LM_KV_E4M3) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
          __nv_fp8x2_storage_t(r[i / 2] >> (16 * (i & 1))), __NV_E4M3));
      const float2 f = __half22float2(h);
      x[2 * i] = f.x * scale;
      x[2 * i + 1] = f.y * scale;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      x[i] = float(int8_t(r[i / 4] >> (8 * (i & 3)))) * scale;
  }
}

constexpr int kReadTokens = 32;   // tokens of a block at most
constexpr int kReadThreads = 128;
constexpr int kReadUnits = 2;     // 16-byte loads of a thread in flight

struct ReadGrid {
  int32_t tokens = 1;        // of a block
  uint32_t chunks = 1;       // 16-byte units of a row
  uint32_t row_units = 1;    // of a token: keys and values of all heads
  FastDiv chunk_div, row_div;
};

// A block takes a few output rows (tokens).  It finds the first one's sequence
// by counting the starts at or below it, all at once; the threads of the rows
// go on from there to their page and offset.  Then all threads move 16 held
// bytes at a time, heads and dim fastest, so that a token's rows leave as one
// run.  Bound by memory: codes and scales read once, rows written once.
// Small blocks in many waves measured best (16 x 16384 tokens of 8 x 128 e4m3,
// 1.02 GB: 161 us, 6.4 TB/s; 166 and 176 with 256 and 512 threads, 174 with
// four loads a thread, 206 with resident blocks that look the next rows up
// while they move these).
template <class T, int STORE, class TO, bool VEC>
__global__ void __launch_bounds__(kReadThreads) lm_kv_read_kernel(
    const __grid_constant__ KvReadArgs a, const __grid_constant__ ReadGrid g) {
  __shared__ int64_t s_page[kReadTokens];   // -1: no token, -2: zeros
  __shared__ uint32_t s_off[kReadTokens];
  stream_order();
  const int64_t t0 = int64_t(blockIdx.x) * g.tokens;
  int below = 0;                             // starts[0 .. seqs) <= t0
  for (int b = 0; b < a.seqs; b += kReadThreads)
    below += __syncthreads_count(b + int(threadIdx.x) < a.seqs &&
                                 a.starts[b + threadIdx.x] <= t0);
  if (threadIdx.x < g.tokens) {
    const int64_t r = t0 + threadIdx.x;
    int64_t page = -1;
    uint32_t off = 0;
    int b = max(below - 1, 0);
    while (b + 1 < a.seqs && a.starts[b + 1] <= r) ++b;
    if (r < a.rows) {
      const int64_t j = r - a.starts[b];
      const int64_t n = a.lens[b] < a.max_tokens ? a.lens[b] : a.max_tokens;
      if (j >= 0 && j < n && r < a.starts[b + 1]) {
        const uint32_t p = fdiv(uint32_t(j), a.c.page_div);
        off = uint32_t(j) - p * a.c.page_tokens;
        page = a.table[int64_t(b) * a.table_stride + p];
        if (page < 0 || page >= a.c.pages) {
          if (a.status) atomicOr(a.status, kStatusRange);
          page = -2;
        }
      }
    }
    s_page[threadIdx.x] = page;
    s_off[threadIdx.x] = off;
  }
  __syncthreads();
  constexpr int N = STORE == LM_KV_SAME ? 8 : 16;   // elements of a unit
  const uint32_t units = g.tokens * g.row_units;
  for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kReadThreads * kReadUnits) {
    uint4 held[kReadUnits];
    float scale[kReadUnits];
    TO* dst[kReadUnits];
#pragma unroll
    for (int k = 0; k < kReadUnits; ++k) {
      const uint32_t u = u0 + kReadThreads * k;
      dst[k] = nullptr;
      if (u >= units) continue;
      const uint32_t i = fdiv(u, g.row_div);
      const uint32_t w = u - i * g.row_units;
      const int64_t page = s_page[i];
      if (page == -1) continue;
      const uint32_t hk = fdiv(w, g.chunk_div);     // kv * heads + head
      const int at = int(w - hk * g.chunks) * N;
      const bool kv = hk >= a.c.heads;
      const uint32_t h = kv ? hk - a.c.heads : hk;
      held[k] = make_uint4(0, 0, 0, 0);
      scale[k] = 1.f;
      if (page >= 0) {
        const char* src = (kv ? a.c.v : a.c.k) + page * a.c.page_b +
                          int64_t(s_off[i]) * a.c.token_b +
                          int64_t(h) * a.c.head_b;
        held[k] = *reinterpret_cast<const uint4*>(
            src + at * (STORE == LM_KV_SAME ? 2 : 1));
        if (STORE != LM_KV_SAME)
          scale[k] = (kv ? a.c.vs : a.c.ks)[(page * a.c.heads + h) *
                                                a.c.page_tokens + s_off[i]];
      }
      const Rows& out = kv ? a.v : a.k;
      dst[k] = reinterpret_cast<TO*>(out.p) + (t0 + i) * out.ts +
               int64_t(h) * out.hs + at;
    }
#pragma unroll
    for (int k = 0; k < kReadUnits; ++k) {
      if (!dst[k]) continue;
      float x[N];
      held_values<T, STORE>(held[k], scale[k], x);
      if (VEC) {
        constexpr int V = 16 / int(sizeof(TO));
#pragma unroll
        for (int e = 0; e < N; e += V) {
          Words<4> y;
          put_words<TO, 4>(x + e, y.w);
          *reinterpret_cast<Words<4>*>(dst[k] + e) = y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) dst[k][e] = from_f32<TO>(x[e]);
      }
    }
  }
}

template <class T, int STORE, class TO>
int launch_read_o(const KvReadArgs& a, cudaStream_t st) {
  ReadGrid g;
  g.chunks = uint32_t(a.c.dim) / (STORE == LM_KV_SAME ? 8 : 16);
  g.row_units = 2 * a.c.heads * g.chunks;
  g.chunk_div = make_fastdiv(g.chunks);
  g.row_div = make_fastdiv(g.row_units);
  // a round of the block's loads, or less where that leaves SMs idle
  const uint32_t most = kReadThreads * kReadUnits / g.row_units;
  const int64_t spread = a.rows / 608;
  int64_t tokens = most < kReadTokens ? most : kReadTokens;
  if (tokens > spread) tokens = spread;
  g.tokens = int(tokens < 1 ? 1 : tokens);
  const uint64_t grid = uint64_t((a.rows + g.tokens - 1) / g.tokens);
  return a.vec ? launch(lm_kv_read_kernel<T, STORE, TO, true>, grid, kReadThreads, 0,
                        st, a, g)
               : launch(lm_kv_read_kernel<T, STORE, TO, false>, grid, kReadThreads, 0,
                        st, a, g);
}

template <class TO>
int launch_read_e(const KvReadArgs& a, int elem, int store, cudaStream_t st) {
  if (store == LM_KV_E4M3) return launch_read_o<bf16, LM_KV_E4M3, TO>(a, st);
  if (store == LM_KV_INT8) return launch_read_o<bf16, LM_KV_INT8, TO>(a, st);
  return elem == LM_BF16 ? launch_read_o<bf16, LM_KV_SAME, TO>(a, st)
                         : launch_read_o<__half, LM_KV_SAME, TO>(a, st);
}

}  // namespace

int launch_kv_write(const KvWriteArgs& a, int elem, int store, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return elem == LM_BF16 ? launch_write_t<bf16>(a, store, st)
                         : launch_write_t<__half>(a, store, st);
}

int launch_kv_read(const KvReadArgs& a, int elem, int store, int out_elem,
                   void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (out_elem == LM_F32) return launch_read_e<float>(a, elem, store, st);
  if (out_elem == LM_F16) return launch_read_e<__half>(a, elem, store, st);
  return launch_read_e<bf16>(a, elem, store, st);
}

}  // namespace lm
