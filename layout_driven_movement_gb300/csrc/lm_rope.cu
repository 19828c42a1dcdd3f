// Rotary positions: the table of cosines and sines, and the turn of dense
// rows.
#include "lm_kv_device.cuh"

namespace lm {
namespace {

// One angle per thread: position * f_i in 64 bits (at position 131072 a
// 32-bit product would be off by 2^-8 of a turn's radian), then one rounding.
// Run once per plan; bound by the 64-bit sine and cosine.
__global__ void __launch_bounds__(256) lm_rope_table_kernel(
    const __grid_constant__ RopeTableArgs a) {
  const int64_t n = a.rows * a.half;
  for (int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x; at < n;
       at += int64_t(gridDim.x) * 256) {
    const int64_t p = at / a.half;
    const int i = int(at - p * a.half);
    double s, c;
    sincos(double(p) * a.freq[i], &s, &c);
    float* row = a.table + p * 2 * a.half;
    row[i] = float(c * a.amplitude);
    row[a.half + i] = float(s * a.amplitude);
  }
}

// A unit is one (token, group of H heads, chunk): V pairs of the rotated
// part -- two chunks of V elements rot/2 apart, or with INTER one chunk of V
// elements holding V/2 pairs -- or one chunk of the rest.  The unit's cosines
// and sines serve all H heads of the group, which lie HG heads apart, so that
// a warp's accesses stay whole rows.
struct RopeGrid {
  uint32_t units = 0;      // of all tokens
  uint32_t chunks = 0;     // units of one head
  uint32_t turned = 0;     // of which rotated
  uint32_t groups = 0;     // head groups (HG)
  FastDiv chunk_div, group_div;
};

template <class T, int V, bool INTER, int H>
__global__ void __launch_bounds__(256) lm_rope_kernel(
    const __grid_constant__ RopeArgs a, const __grid_constant__ RopeGrid g) {
  const uint32_t u = blockIdx.x * 256 + threadIdx.x;
  if (u >= g.units) return;
  const uint32_t th = fdiv(u, g.chunk_div);
  const uint32_t c = u - th * g.chunks;
  const uint32_t t = fdiv(th, g.group_div);
  const uint32_t h0 = th - t * g.groups;
  const T* x = reinterpret_cast<const T*>(a.x.p) + int64_t(t) * a.x.ts;
  T* o = reinterpret_cast<T*>(a.out.p) + int64_t(t) * a.out.ts;
  constexpr int E = INTER && V == 1 ? 2 : V;   // elements of a chunk
  typedef Pack<T, V> P;
  if (c >= g.turned) {
    const int at = a.turn.rot + int(c - g.turned) * V;
#pragma unroll
    for (int k = 0; k < H; ++k) {
      const uint32_t h = h0 + k * g.groups;
      if (h < a.heads)
        *reinterpret_cast<P*>(o + int64_t(h) * a.out.hs + at) =
            *reinterpret_cast<const P*>(x + int64_t(h) * a.x.hs + at);
    }
    return;
  }
  const int half = a.turn.rot / 2;
  constexpr int N = INTER ? E / 2 : V;         // pairs of a unit
  const int lo = int(c) * E, hi = INTER ? lo + V : lo + half;
  // the rows first, then the position and its table row: their latencies
  // overlap
  P xl[H], xh[H];
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const uint32_t h = h0 + k * g.groups;
    if (h < a.heads) {
      const T* r = x + int64_t(h) * a.x.hs;
      xl[k] = *reinterpret_cast<const P*>(r + lo);
      if (!INTER || V == 1) xh[k] = *reinterpret_cast<const P*>(r + hi);
    }
  }
  const float* row = turn_row(a.turn, t, a.status);
  const int i0 = int(c) * N;
  float cs[N], sn[N];
  if (row) {
    constexpr int W = N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 1;
    typedef Pack<float, W> F;
#pragma unroll
    for (int i = 0; i < N; i += W) {
      *reinterpret_cast<F*>(cs + i) =
          *reinterpret_cast<const F*>(row + i0 + i);
      *reinterpret_cast<F*>(sn + i) =
          *reinterpret_cast<const F*>(row + half + i0 + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) cs[i] = sn[i] = __int_as_float(0x7fc00000);
  }
  if (a.turn.inverse) {
#pragma unroll
    for (int i = 0; i < N; ++i) sn[i] = -sn[i];
  }
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const uint32_t h = h0 + k * g.groups;
    if (h >= a.heads) break;
    T* r = o + int64_t(h) * a.out.hs;
    if (INTER && V > 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float p = to_f32(xl[k].v[2 * i]), q = to_f32(xl[k].v[2 * i + 1]);
        xl[k].v[2 * i] = from_f32<T>(turn_lo(p, q, cs[i], sn[i]));
        xl[k].v[2 * i + 1] = from_f32<T>(turn_hi(p, q, cs[i], sn[i]));
      }
      *reinterpret_cast<P*>(r + lo) = xl[k];
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float p = to_f32(xl[k].v[i]), q = to_f32(xh[k].v[i]);
        xl[k].v[i] = from_f32<T>(turn_lo(p, q, cs[i], sn[i]));
        xh[k].v[i] = from_f32<T>(turn_hi(p, q, cs[i], sn[i]));
      }
      *reinterpret_cast<P*>(r + lo) = xl[k];
      *reinterpret_cast<P*>(r + hi) = xh[k];
    }
  }
}

template <class T, int V, bool INTER, int H>
int launch_h(const RopeArgs& a, cudaStream_t st) {
  RopeGrid g;
  constexpr int E = INTER && V == 1 ? 2 : V;
  g.turned = uint32_t(INTER ? a.turn.rot / E : a.turn.rot / 2 / V);
  g.chunks = g.turned;
  if (a.copy_rest) g.chunks += uint32_t(a.dim - a.turn.rot) / V;
  g.groups = (a.heads + H - 1) / H;
  g.chunk_div = make_fastdiv(g.chunks);
  g.group_div = make_fastdiv(g.groups);
  g.units = a.tokens * g.groups * g.chunks;
  lm_rope_kernel<T, V, INTER, H><<<(g.units + 255) / 256, 256, 0, st>>>(a, g);
  return launch_status();
}

template <class T, int V, bool INTER>
int launch_v(const RopeArgs& a, cudaStream_t st) {
  return launch_h<T, V, INTER, 1>(a, st);
}

template <class T>
int launch_t(const RopeArgs& a, cudaStream_t st) {
  constexpr int V = 16 / int(sizeof(T));
  if (a.vec)
    return a.turn.inter ? launch_v<T, V, true>(a, st)
                        : launch_v<T, V, false>(a, st);
  return a.turn.inter ? launch_v<T, 1, true>(a, st)
                      : launch_v<T, 1, false>(a, st);
}

}  // namespace

int launch_rope(const RopeArgs& a, int elem, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (elem == LM_F32) return launch_t<float>(a, st);
  if (elem == LM_F16) return launch_t<__half>(a, st);
  return launch_t<bf16>(a, st);
}

int launch_rope_table(const RopeTableArgs& a, void* stream) {
  const int64_t blocks = (a.rows * a.half + 255) / 256;
  lm_rope_table_kernel<<<unsigned(blocks < (1 << 20) ? blocks : (1 << 20)),
                         256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return launch_status();
}

}  // namespace lm
