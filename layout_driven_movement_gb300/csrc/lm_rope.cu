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
  stream_order();
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
// a warp's accesses stay whole rows.  Bound by memory: x read once, out
// written once (16384 x 32 x 128 bf16, 268 MB: 40 us, 6.7 TB/s; 45 us with one
// head a thread, 42 with four).
struct RopeGrid {
  uint32_t units = 0;      // of all tokens
  uint32_t chunks = 0;     // units of one head
  uint32_t turned = 0;     // of which rotated
  uint32_t groups = 0;     // head groups (HG)
  FastDiv chunk_div, group_div;
};

// The unit `u`: token, first head and chunk.
struct RopeUnit {
  uint32_t t, h0, c;
  __device__ __forceinline__ RopeUnit(const RopeGrid& g, uint32_t u) {
    const uint32_t th = fdiv(u, g.chunk_div);
    c = u - th * g.chunks;
    t = fdiv(th, g.group_div);
    h0 = th - t * g.groups;
  }
};

// N cosines and as many sines from pair i0 on; NaN without a table row.
template <int N>
__device__ __forceinline__ void angles(const Turn& turn, const float* row,
                                       int i0, float* cs, float* sn) {
  if (row) {
    constexpr int W = N % 4 == 0 ? 4 : N % 2 == 0 ? 2 : 1;
    typedef Pack<float, W> F;
    const float* sines = row + turn.rot / 2;
#pragma unroll
    for (int i = 0; i < N; i += W) {
      *reinterpret_cast<F*>(cs + i) =
          *reinterpret_cast<const F*>(row + i0 + i);
      *reinterpret_cast<F*>(sn + i) =
          *reinterpret_cast<const F*>(sines + i0 + i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) cs[i] = sn[i] = __int_as_float(0x7fc00000);
  }
  if (turn.inverse) {
#pragma unroll
    for (int i = 0; i < N; ++i) sn[i] = -sn[i];
  }
}

template <class T, bool INTER, int H>
__global__ void __launch_bounds__(256) lm_rope_kernel(
    const __grid_constant__ RopeArgs a, const __grid_constant__ RopeGrid g) {
  stream_order();
  const uint32_t u = blockIdx.x * 256 + threadIdx.x;
  if (u >= g.units) return;
  const RopeUnit at(g, u);
  constexpr int V = 16 / int(sizeof(T));       // elements of a chunk
  constexpr int N = INTER ? V / 2 : V;         // pairs of a unit
  typedef Words<4> P;
  const T* x = reinterpret_cast<const T*>(a.x.p) + int64_t(at.t) * a.x.ts;
  T* o = reinterpret_cast<T*>(a.out.p) + int64_t(at.t) * a.out.ts;
  const bool rest = at.c >= g.turned;
  const int lo = rest ? a.turn.rot + int(at.c - g.turned) * V : int(at.c) * V;
  const int hi = lo + a.turn.rot / 2;
  // the rows first, then the position and its table row: their latencies
  // overlap
  P xl[H], xh[H];
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const uint32_t h = at.h0 + k * g.groups;
    if (h < a.heads) {
      const T* r = x + int64_t(h) * a.x.hs;
      xl[k] = *reinterpret_cast<const P*>(r + lo);
      if (!INTER && !rest) xh[k] = *reinterpret_cast<const P*>(r + hi);
    }
  }
  if (!rest) {
    float cs[N], sn[N];
    angles<N>(a.turn, turn_row(a.turn, at.t, a.status), int(at.c) * N, cs,
              sn);
#pragma unroll
    for (int k = 0; k < H; ++k) {
      float p[V], q[V];
      get_words<T, 4>(xl[k].w, p);
      if (INTER) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          q[2 * i] = turn_lo(p[2 * i], p[2 * i + 1], cs[i], sn[i]);
          q[2 * i + 1] = turn_hi(p[2 * i], p[2 * i + 1], cs[i], sn[i]);
        }
        put_words<T, 4>(q, xl[k].w);
      } else {
        float y[V], z[V];
        get_words<T, 4>(xh[k].w, q);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          y[i] = turn_lo(p[i], q[i], cs[i], sn[i]);
          z[i] = turn_hi(p[i], q[i], cs[i], sn[i]);
        }
        put_words<T, 4>(y, xl[k].w);
        put_words<T, 4>(z, xh[k].w);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < H; ++k) {
    const uint32_t h = at.h0 + k * g.groups;
    if (h < a.heads) {
      T* r = o + int64_t(h) * a.out.hs;
      *reinterpret_cast<P*>(r + lo) = xl[k];
      if (!INTER && !rest) *reinterpret_cast<P*>(r + hi) = xh[k];
    }
  }
}

// The same for rows that allow no 16-byte accesses: a pair or an element of
// the rest a unit.
template <class T>
__global__ void __launch_bounds__(256) lm_rope_single_kernel(
    const __grid_constant__ RopeArgs a, const __grid_constant__ RopeGrid g) {
  stream_order();
  const uint32_t u = blockIdx.x * 256 + threadIdx.x;
  if (u >= g.units) return;
  const RopeUnit at(g, u);
  const T* x = reinterpret_cast<const T*>(a.x.p) + int64_t(at.t) * a.x.ts +
               int64_t(at.h0) * a.x.hs;
  T* o = reinterpret_cast<T*>(a.out.p) + int64_t(at.t) * a.out.ts +
         int64_t(at.h0) * a.out.hs;
  if (at.c >= g.turned) {
    const int e = a.turn.rot + int(at.c - g.turned);
    o[e] = x[e];
    return;
  }
  const int lo = a.turn.inter ? 2 * int(at.c) : int(at.c);
  const int hi = a.turn.inter ? lo + 1 : lo + a.turn.rot / 2;
  const float p = to_f32(x[lo]), q = to_f32(x[hi]);
  float cs, sn;
  angles<1>(a.turn, turn_row(a.turn, at.t, a.status), int(at.c), &cs, &sn);
  o[lo] = from_f32<T>(turn_lo(p, q, cs, sn));
  o[hi] = from_f32<T>(turn_hi(p, q, cs, sn));
}

// Chunks of V elements (1: single elements, a pair a unit), H heads a thread.
RopeGrid rope_grid(const RopeArgs& a, int v, int h) {
  RopeGrid g;
  g.turned = uint32_t(v > 1 && a.turn.inter ? a.turn.rot / v
                                            : a.turn.rot / 2 / v);
  g.chunks = g.turned;
  if (a.copy_rest) g.chunks += uint32_t((a.dim - a.turn.rot) / v);
  g.groups = (a.heads + h - 1) / h;
  g.chunk_div = make_fastdiv(g.chunks);
  g.group_div = make_fastdiv(g.groups);
  g.units = a.tokens * g.groups * g.chunks;
  return g;
}

template <class T, bool INTER, int H>
int launch_h(const RopeArgs& a, cudaStream_t st) {
  const RopeGrid g = rope_grid(a, 16 / int(sizeof(T)), H);
  return launch(lm_rope_kernel<T, INTER, H>, (uint64_t(g.units) + 255) / 256,
                256, 0, st, a, g);
}

constexpr uint64_t kRopeShare = 152 * 2048;

template <class T, bool INTER>
int launch_v(const RopeArgs& a, cudaStream_t st) {
  // few rows spread over as many threads as they can; many share a token's
  // angles between two heads
  constexpr int V = 16 / int(sizeof(T));
  if (a.heads > 1 &&
      uint64_t(a.tokens) * a.heads * uint32_t(a.dim / V) >= 2 * kRopeShare)
    return launch_h<T, INTER, 2>(a, st);
  return launch_h<T, INTER, 1>(a, st);
}

template <class T>
int launch_t(const RopeArgs& a, cudaStream_t st) {
  if (a.vec)
    return a.turn.inter ? launch_v<T, true>(a, st) : launch_v<T, false>(a, st);
  const RopeGrid g = rope_grid(a, 1, 1);
  return launch(lm_rope_single_kernel<T>, (uint64_t(g.units) + 255) / 256, 256,
                0, st, a, g);
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
  return launch(lm_rope_table_kernel, blocks < (1 << 20) ? blocks : (1 << 20),
                256, 0, static_cast<cudaStream_t>(stream), a);
}

}  // namespace lm
