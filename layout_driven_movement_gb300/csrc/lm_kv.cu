// The paged cache's write (rotating and quantising) and its read back.
#include "lm_kv_device.cuh"

namespace lm {
namespace {

// --- write -----------------------------------------------------------------

// The scale of a row from the bits of its largest magnitude, and what its
// elements are multiplied by.  E4M3: 448 = 1.75 * 2^8, so with max|x| =
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
  return fmaxf(__fdiv_rn(m, 127.f), 0x1p-126f);
}

// 8 elements' codes.  A row that is not finite has by == 0: its codes are 0.
template <int STORE>
__device__ __forceinline__ uint2 row_codes(const float* x, float by,
                                           bool finite) {
  uint32_t w[2];
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
      w[i] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[i] |= uint32_t(__float2int_rn(x[4 * i + j] * by) & 255) << (8 * j);
    }
    if (!finite) w[i] = 0;
  }
  return make_uint2(w[0], w[1]);
}

// A row's 8 elements at `at`; one 16-byte load when the rows allow it.
template <class T, bool VEC>
__device__ __forceinline__ void load8(const T* row, int at, T* x) {
  if (VEC) {
    *reinterpret_cast<Pack<T, 8>*>(x) =
        *reinterpret_cast<const Pack<T, 8>*>(row + at);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = row[at + i];
  }
}

// L lanes hold a token-head's rows, 8 elements a lane of its key and its
// value: the row's largest magnitude is then a few shuffles away, and its
// codes leave as 8-byte stores of adjacent lanes.  Bound by memory: each
// input element is read once (the turn's partner elements come from the
// cache lines that the same lanes just read), each code written once.
template <class T, int STORE, int L, bool VEC>
__global__ void __launch_bounds__(256) lm_kv_write_kernel(
    const __grid_constant__ KvWriteArgs a) {
  const uint32_t row = (blockIdx.x * 256 + threadIdx.x) / L;
  const int at = int(threadIdx.x % L) * 8;
  const uint32_t rows = a.tokens * a.c.heads;
  const uint32_t t = row < rows ? fdiv(row, a.heads_div) : 0;
  const uint32_t h = row < rows ? row - t * a.c.heads : 0;
  const bool in = row < rows && at < a.c.dim;
  alignas(16) T xr[2][8];
  const T* src[2] = {
      reinterpret_cast<const T*>(a.k.p) + int64_t(t) * a.k.ts +
          int64_t(h) * a.k.hs,
      reinterpret_cast<const T*>(a.v.p) + int64_t(t) * a.v.ts +
          int64_t(h) * a.v.hs};
  if (in) {
    load8<T, VEC>(src[0], at, xr[0]);
    load8<T, VEC>(src[1], at, xr[1]);
  }
  const int64_t slot = row < rows ? a.slots[t] : -1;
  const bool turned = a.turn.pos != nullptr;
  float x[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[0][i] = in ? to_f32(xr[0][i]) : 0.f;
    x[1][i] = in ? to_f32(xr[1][i]) : 0.f;
  }
  if (turned && in && at < a.turn.rot) {
    const float* tr = turn_row(a.turn, t, at == 0 ? a.status : nullptr);
    const int half = a.turn.rot / 2;
    const float nan = __int_as_float(0x7fc00000);
    if (a.turn.inter) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const int p = (at + i) / 2;
        if (at + i < a.turn.rot) {
          const float c = tr ? tr[p] : nan, s = tr ? tr[half + p] : nan;
          const float u = x[0][i], w = x[0][i + 1];
          x[0][i] = turn_lo(u, w, c, s);
          x[0][i + 1] = turn_hi(u, w, c, s);
        }
      }
    } else {
      // the partner of element i is half a rotated part away; when halves
      // are whole chunks it is one more aligned load
      alignas(16) T pr[8];
      if (half % 8 == 0) {
        load8<T, VEC>(src[0], at < half ? at + half : at - half, pr);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = at + i;
          pr[i] = e < a.turn.rot ? src[0][e < half ? e + half : e - half]
                                 : xr[0][i];
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int e = at + i;
        if (e < a.turn.rot) {
          const int p = e < half ? e : e - half;
          const float c = tr ? tr[p] : nan, s = tr ? tr[half + p] : nan;
          const float o = to_f32(pr[i]);
          x[0][i] = e < half ? turn_lo(x[0][i], o, c, s)
                             : turn_hi(o, x[0][i], c, s);
        }
      }
    }
  }
  const int64_t tokens = a.c.pages * int64_t(a.c.page_tokens);
  if (slot >= tokens && at == 0 && a.status) atomicOr(a.status, kStatusRange);
  const bool to = in && slot >= 0 && slot < tokens;
  const int64_t page = to ? slot / a.c.page_tokens : 0;
  const uint32_t off = to ? uint32_t(slot - page * a.c.page_tokens) : 0;
  const int64_t base = page * a.c.page_b + int64_t(off) * a.c.token_b +
                       int64_t(h) * a.c.head_b;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    char* dst = (kv ? a.c.v : a.c.k) + base;
    if (STORE == LM_KV_SAME) {
      if (kv == 0 && turned && at < a.turn.rot) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (at + i < a.turn.rot) xr[0][i] = from_f32<T>(x[0][i]);
      }
      if (to)
        *reinterpret_cast<Pack<T, 8>*>(dst + at * 2) =
            *reinterpret_cast<const Pack<T, 8>*>(xr[kv]);
      continue;
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      top = max(top, __float_as_uint(x[kv][i]) & 0x7fffffffu);
#pragma unroll
    for (int m = L / 2; m; m /= 2)
      top = max(top, __shfl_xor_sync(0xffffffffu, top, m, L));
    float by;
    const float scale = row_scale<STORE>(top, &by);
    if (to) {
      *reinterpret_cast<uint2*>(dst + at) =
          row_codes<STORE>(x[kv], by, top < 0x7f800000u);
      if (at == 0)
        (kv ? a.c.vs : a.c.ks)[(page * a.c.heads + h) * a.c.page_tokens +
                               off] = scale;
    }
  }
}

template <class T, int STORE, int L>
int launch_write_l(const KvWriteArgs& a, cudaStream_t st) {
  const uint64_t threads = uint64_t(a.tokens) * a.c.heads * L;
  const unsigned grid = unsigned((threads + 255) / 256);
  if (a.vec)
    lm_kv_write_kernel<T, STORE, L, true><<<grid, 256, 0, st>>>(a);
  else
    lm_kv_write_kernel<T, STORE, L, false><<<grid, 256, 0, st>>>(a);
  return launch_status();
}

template <class T, int STORE>
int launch_write_s(const KvWriteArgs& a, cudaStream_t st) {
  if (a.c.dim <= 64) return launch_write_l<T, STORE, 8>(a, st);
  if (a.c.dim <= 128) return launch_write_l<T, STORE, 16>(a, st);
  return launch_write_l<T, STORE, 32>(a, st);
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
    const T* e = reinterpret_cast<const T*>(r);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
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

constexpr int kReadTokens = 32;

// A block takes 32 output rows (tokens): its first threads find each row's
// sequence (a binary search of starts), page and offset, then all threads
// move 16 held bytes at a time, heads and dim fastest, so that a token's rows
// leave as one run.  Bound by memory: codes and scales read once, rows
// written once.
template <class T, int STORE, class TO, bool VEC>
__global__ void __launch_bounds__(256) lm_kv_read_kernel(
    const __grid_constant__ KvReadArgs a, const FastDiv chunk_div,
    const uint32_t chunks, const FastDiv row_div, const uint32_t row_units) {
  __shared__ int64_t s_page[kReadTokens];   // -1: no token, -2: zeros
  __shared__ uint32_t s_off[kReadTokens];
  const int64_t t0 = int64_t(blockIdx.x) * kReadTokens;
  if (threadIdx.x < kReadTokens) {
    const int64_t r = t0 + threadIdx.x;
    int64_t page = -1;
    uint32_t off = 0;
    if (r < a.rows) {
      int lo = 0, hi = a.seqs;             // the last b with starts[b] <= r
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.starts[mid] <= r)
          lo = mid;
        else
          hi = mid;
      }
      const int64_t j = r - a.starts[lo];
      const int64_t n = a.lens[lo] < a.max_tokens ? a.lens[lo] : a.max_tokens;
      if (j >= 0 && j < n && r < a.starts[lo + 1]) {
        const uint32_t p = fdiv(uint32_t(j), a.c.page_div);
        off = uint32_t(j) - p * a.c.page_tokens;
        page = a.table[int64_t(lo) * a.table_stride + p];
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
  const uint32_t units = kReadTokens * row_units;   // keys and values
  for (uint32_t u = threadIdx.x; u < units; u += 256) {
    const uint32_t i = fdiv(u, row_div);
    const uint32_t w = u - i * row_units;
    const int64_t page = s_page[i];
    if (page == -1) continue;
    const uint32_t hk = fdiv(w, chunk_div);         // kv * heads + head
    const int at = int(w - hk * chunks) * N;
    const bool kv = hk >= a.c.heads;
    const uint32_t h = kv ? hk - a.c.heads : hk;
    uint4 held = make_uint4(0, 0, 0, 0);
    float scale = 1.f;
    if (page >= 0) {
      const char* src = (kv ? a.c.v : a.c.k) + page * a.c.page_b +
                        int64_t(s_off[i]) * a.c.token_b +
                        int64_t(h) * a.c.head_b;
      held = *reinterpret_cast<const uint4*>(
          src + at * (STORE == LM_KV_SAME ? 2 : 1));
      if (STORE != LM_KV_SAME)
        scale = (kv ? a.c.vs : a.c.ks)[(page * a.c.heads + h) *
                                           a.c.page_tokens +
                                       s_off[i]];
    }
    const Rows& out = kv ? a.v : a.k;
    TO* dst = reinterpret_cast<TO*>(out.p) + (t0 + i) * out.ts +
              int64_t(h) * out.hs + at;
    float x[N];
    held_values<T, STORE>(held, scale, x);
    alignas(16) TO y[N];
#pragma unroll
    for (int k = 0; k < N; ++k) y[k] = from_f32<TO>(x[k]);
    if (VEC) {
      constexpr int V = 16 / int(sizeof(TO));
#pragma unroll
      for (int k = 0; k < N; k += V)
        *reinterpret_cast<Pack<TO, V>*>(dst + k) =
            *reinterpret_cast<const Pack<TO, V>*>(y + k);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) dst[k] = y[k];
    }
  }
}

template <class T, int STORE, class TO>
int launch_read_o(const KvReadArgs& a, cudaStream_t st) {
  const uint32_t chunks = uint32_t(a.c.dim) / (STORE == LM_KV_SAME ? 8 : 16);
  const uint32_t row_units = 2 * a.c.heads * chunks;
  const unsigned grid = unsigned((a.rows + kReadTokens - 1) / kReadTokens);
  const FastDiv cd = make_fastdiv(chunks), rd = make_fastdiv(row_units);
  if (a.vec)
    lm_kv_read_kernel<T, STORE, TO, true><<<grid, 256, 0, st>>>(
        a, cd, chunks, rd, row_units);
  else
    lm_kv_read_kernel<T, STORE, TO, false><<<grid, 256, 0, st>>>(
        a, cd, chunks, rd, row_units);
  return launch_status();
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
