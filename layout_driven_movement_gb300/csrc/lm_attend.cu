// Attention of one new token per sequence over the paged cache.
#include "lm_kv_device.cuh"

namespace lm {
namespace {

constexpr int kWarps = 4;

template <class T, int STORE>
__device__ __forceinline__ float held_value(const char* row, int d,
                                            float scale) {
  if (STORE == LM_KV_SAME)
    return to_f32(reinterpret_cast<const T*>(row)[d]);
  if (STORE == LM_KV_INT8)
    return float(reinterpret_cast<const int8_t*>(row)[d]) * scale;
  const __half h = __half(__nv_cvt_fp8_to_halfraw(
      reinterpret_cast<const __nv_fp8_storage_t*>(row)[d], __NV_E4M3));
  return __half2float(h) * scale;
}

// A block per (sequence, query head).  Each warp takes every fourth key with
// a running maximum m, sum l and output o: a key of score s turns (m, l, o)
// into (m', l e^(m-m') + e^(s-m'), o e^(m-m') + e^(s-m') v), m' = max(m, s);
// the warps' states join by the same rule.
template <class T, int STORE>
__global__ void __launch_bounds__(32 * kWarps) lm_kv_attend_kernel(
    const __grid_constant__ KvAttendArgs a) {
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][kKvMaxDim];
  const int b = blockIdx.x / a.heads_q, hq = blockIdx.x % a.heads_q;
  const int h = hq / a.group;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int dim = a.c.dim;
  int64_t n = a.lens[b];
  n = n < 0 ? 0 : n > a.max_tokens ? a.max_tokens : n;
  const int64_t first = a.window && n > a.window ? n - a.window : 0;
  const T* q = reinterpret_cast<const T*>(a.q.p) + int64_t(b) * a.q.ts +
               int64_t(hq) * a.q.hs;
  float qr[8], o[8], m = -INFINITY, l = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int d = lane + 32 * i;
    qr[i] = d < dim ? to_f32(q[d]) : 0.f;
    o[i] = 0;
  }
  for (int64_t j = first + warp; j < n; j += kWarps) {
    const uint32_t p = fdiv(uint32_t(j), a.c.page_div);
    const uint32_t off = uint32_t(j) - p * a.c.page_tokens;
    const int64_t page = a.table[int64_t(b) * a.table_stride + p];
    if (page < 0 || page >= a.c.pages) {
      if (lane == 0 && a.status) atomicOr(a.status, kStatusRange);
      continue;
    }
    const int64_t at = page * a.c.page_b + int64_t(off) * a.c.token_b +
                       int64_t(h) * a.c.head_b;
    const int64_t sat = (page * a.c.heads + h) * a.c.page_tokens + off;
    const float ks = STORE == LM_KV_SAME ? 1.f : a.c.ks[sat];
    const float vs = STORE == LM_KV_SAME ? 1.f : a.c.vs[sat];
    float s = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      if (d < dim) s += qr[i] * held_value<T, STORE>(a.c.k + at, d, ks);
    }
#pragma unroll
    for (int k = 16; k; k /= 2) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= a.scale;
    const float top = fmaxf(m, s);
    const float keep = m == top ? 1.f : expf(m - top);
    // -infinity weighs nothing even alone; a NaN stays a NaN
    const float w = s == -INFINITY ? 0.f : expf(s - top);
    l = l * keep + w;
    m = top;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = lane + 32 * i;
      if (d < dim)
        o[i] = o[i] * keep + w * held_value<T, STORE>(a.c.v + at, d, vs);
    }
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < 8; ++i) so[warp][lane + 32 * i] = o[i];
  __syncthreads();
  float top = -INFINITY, total = 0, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = sl[w] == 0 ? 0.f : expf(sm[w] - top);
    total += sl[w] * f[w];
  }
  T* out = reinterpret_cast<T*>(a.out.p) + int64_t(b) * a.out.ts +
           int64_t(hq) * a.out.hs;
  for (int d = threadIdx.x; d < dim; d += 32 * kWarps) {
    float x = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
      x += so[w][d] * f[w];
    out[d] = from_f32<T>(total == 0 ? 0.f : x / total);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[int64_t(b) * a.heads_q + hq] =
        total == 0 ? -INFINITY : top + logf(total);
}

template <class T>
int launch_t(const KvAttendArgs& a, int store, cudaStream_t st) {
  const unsigned grid = unsigned(a.seqs) * unsigned(a.heads_q);
  if (store == LM_KV_E4M3)
    lm_kv_attend_kernel<T, LM_KV_E4M3><<<grid, 32 * kWarps, 0, st>>>(a);
  else if (store == LM_KV_INT8)
    lm_kv_attend_kernel<T, LM_KV_INT8><<<grid, 32 * kWarps, 0, st>>>(a);
  else
    lm_kv_attend_kernel<T, LM_KV_SAME><<<grid, 32 * kWarps, 0, st>>>(a);
  return launch_status();
}

}  // namespace

int attend_workspace(int, int, int, int64_t* bytes) {
  *bytes = 0;
  return LM_OK;
}

int launch_kv_attend(const KvAttendArgs& a, int store, void* stream) {
  if (int64_t(a.seqs) * a.heads_q >= (int64_t(1) << 31)) return LM_E_OVERFLOW;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.elem == LM_BF16 ? launch_t<bf16>(a, store, st)
                           : launch_t<__half>(a, store, st);
}

}  // namespace lm
