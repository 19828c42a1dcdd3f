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
//   warp 12     one thread issues S_q = Q_q K^T and O_q += P_q V
//   warps 0-3   and 4-7, one for each tile of queries, a row a thread: S from
//               tensor memory, its exponentials, and P back in S's place
// While one tile's exponentials are taken the tensor cores have the other's
// products.  Where there are no more than 128 queries, the two take every
// second tile of keys instead, with states of their own that are joined later.
//
// Work is one line of key tiles over all groups, key heads and tiles of rows,
// cut evenly over the resident blocks; what one block holds of rows that others
// share goes to the workspace, and the launch that joins it with the attention
// over each sequence's own pages reads it in the order of the line.
//
// Weights are one 16-bit part each (bf16's rounding of a weight costs a result
// about as much as its own): a second part would be half as many products
// again.  Float16 queries of 8-bit caches get the second part, since their
// values are met by bf16 weights (of any size, as their scales are).
#pragma once

#include "lm_attend.cuh"
#include "lm_kv_long.h"
#include "lm_line.cuh"
#include "lm_mbar.cuh"
#include "lm_tcgen05.cuh"

namespace lm {

constexpr int kSharedThreads = 13 * 32;

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
  // before it are done with, so that many hold.
  static constexpr int NM = NS + 1;
  static constexpr int kMeta = NK * 8 + 32;
  static constexpr uint32_t kOut = 256;                // O's first column
  static constexpr int kBars = 4 * NS + 12;
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

// 16 codes as 16-bit floats, in order.
template <int STORE, bool BF>
__device__ __forceinline__ void widen16(const uint4& w, uint32_t* y) {
  const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t p[2];
    if (STORE == LM_KV_E4M3) {
      Codes<KIND_E4M3>::keys(r[i], p);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (BF) {
          const float2 f = unpair16<false>(p[j]);
          p[j] = pair16<true>(f.x, f.y);
        }
        y[2 * i + j] = p[j];
      }
    } else {
      if (BF)
        Codes<KIND_INT8>::values(r[i], p, nullptr);
      else
        Codes<KIND_INT8>::keys(r[i], p);
      y[2 * i] = __byte_perm(p[0], p[1], 0x5410);
      y[2 * i + 1] = __byte_perm(p[0], p[1], 0x7632);
    }
  }
}

__device__ __forceinline__ void st_smem16(uint32_t to, uint32_t a, uint32_t b,
                                          uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(to), "r"(a),
               "r"(b), "r"(c), "r"(d)
               : "memory");
}

template <int ELEM, int STORE, int D>
__global__ void __launch_bounds__(kSharedThreads, 1)
    lm_kv_shared_kernel(const __grid_constant__ KvSharedArgs a) {
  using S = SharedShape<D>;
  constexpr int NK = S::NK, QT = S::QT, NS = S::NS, NM = S::NM;
  constexpr bool CODES = STORE != LM_KV_SAME;
  constexpr bool QBF = ELEM == LM_BF16;         // queries and keys are bf16
  constexpr bool VBF = QBF || CODES;            // values and weights are
  constexpr int PARTS = CODES && !QBF ? 2 : 1;  // 16-bit parts of a weight
  // A row's reference moves when a score passes it by SLACK (in units of ln
  // 2).  f16 weights lie below 2^15, the reference's at 2^12.  bf16 values
  // reach the end of 32 bits' range, so their weights' sum stays below 1.
  constexpr float SLACK = VBF ? 8.f : 3.f;
  constexpr int KPW = NK / 4;                   // keys of a loading warp
  extern __shared__ char smem_raw[];
  __shared__ volatile int dead;
  __shared__ uint32_t tmem_at;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
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

  stream_order();
  const LineShare share = line_share<kSharedThreads>(
      a.groups, blockIdx.x, gridDim.x, [&](int g) {
        const SharedSpan s = shared_span(a, g, NK, S::kRows);
        return int64_t(s.tiles) * s.row_tiles * a.c.heads;
      });
  if (share.left <= 0) return;

  if (threadIdx.x == 0) {
    dead = 0;
    for (int i = 0; i < NS; ++i) {
      mbar_init(k_full(i), 128);
      mbar_init(k_empty(i), 1);
      mbar_init(v_full(i), 128);
      mbar_init(v_empty(i), 1);
    }
    for (int q = 0; q < 2; ++q) {
      mbar_init(s_full(q), 1);
      mbar_init(p_full(q), 128);
      mbar_init(o_full(q), 1);
      mbar_init(o_empty(q), 128);
    }
    mbar_init(q_full, 128);
    mbar_init(q_empty, 1);
    mbar_init(drain, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 12)
    tmem_alloc(uint32_t(__cvta_generic_to_shared(&tmem_at)), 512);
  tmem_before_sync();
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
    const int lw = warp - 8;
    constexpr int EB = CODES ? 1 : 2;
    constexpr int CPR = D * EB / 16;            // 16-byte chunks of a row
    constexpr int RPI = 32 / CPR;               // rows an instruction
    constexpr int IT = KPW / RPI;
    const int c = lane % CPR, r0 = lane / CPR;
    const bool held = c * 16 < dim * EB;
    const bool used = c * 16 < dim16 * EB;
    int tile = 0, nth = 0;
    int pending = 0;                            // copies not yet announced
    uint32_t announce[2] = {0, 0};
    bool alive = true;
    auto announce_all = [&] {
      cp_wait<0>();
      smem_to_products();
      for (; pending > 0; --pending) {
        mbar_arrive(announce[0]);
        announce[0] = announce[1];
      }
    };
    // waits for a stage, with nothing held back meanwhile
    auto acquire = [&](uint32_t bar, uint32_t parity) {
      if (!__all_sync(0xffffffffu, mbar_try(bar, parity))) {
        if (!CODES) announce_all();
        if (!warp_gate(bar, parity, &dead)) alive = false;
      }
    };
    const float unit = fabsf(a.scale) * 1.44269504088896341f;
    while (alive && walk.next(a, &seg)) {
      const int32_t* const table = a.table + seg.g * a.table_stride;
      auto look = [&](int t) {
        const int key = t * NK + lw * KPW + lane;
        return (KPW == 32 || lane < KPW) && t < seg.t0 + seg.steps &&
                       key < seg.s.len
                   ? table[fdiv(uint32_t(key), a.c.page_div)]
                   : -1;
      };
      int page = look(seg.t0);
      // the queries, turned round where the scale is negative
      if (nth > 0) {
        if (!CODES) announce_all();
        if (!warp_gate(q_empty, (nth - 1) & 1, &dead)) break;
      }
      {
        const int tiles = split_of(seg) ? 1 : (seg.rows + 127) / 128;
        const uint16_t flip = a.scale < 0 ? 0x8000 : 0;
        const uint32_t flip2 = flip * 0x10001u;
        const int chunks = dim16 / 8;
        for (int u = threadIdx.x - 256; u < tiles * 128 * chunks; u += 128) {
          const int row = u / chunks, ch = u - row * chunks;
          uint4 w = make_uint4(0, 0, 0, 0);
          if (row < seg.rows && ch * 8 < dim) {
            const int rg = seg.rt * S::kRows + row;
            const int si = rg / a.group;
            const uint16_t* q =
                reinterpret_cast<const uint16_t*>(a.q.p) +
                int64_t(seg.s.start + si) * a.q.ts +
                int64_t(seg.h * a.group + (rg - si * a.group)) * a.q.hs +
                ch * 8;
            if (a.q16) {
              w = *reinterpret_cast<const uint4*>(q);
            } else {
              uint32_t r[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                r[i] = q[2 * i] | uint32_t(q[2 * i + 1]) << 16;
              w = make_uint4(r[0], r[1], r[2], r[3]);
            }
          }
          const uint32_t to = q_s + row / 128 * S::kQ + ch / 8 * (128 * 128) +
                              row % 128 * 128 + ((ch ^ row) & 7) * 16;
          st_smem16(to, w.x ^ flip2, w.y ^ flip2, w.z ^ flip2, w.w ^ flip2);
        }
        smem_to_products();
        mbar_arrive(q_full);
      }
      ++nth;
      for (int t = seg.t0; t < seg.t0 + seg.steps && alive; ++t, ++tile) {
        const int key = t * NK + lw * KPW + lane;
        const bool in = (KPW == 32 || lane < KPW) && key < seg.s.len;
        const bool ok = in && page >= 0 && page < a.c.pages;
        if (in && !ok && a.status) atomicOr(a.status, kStatusRange);
        const uint32_t off =
            uint32_t(key) - fdiv(uint32_t(key), a.c.page_div) * a.c.page_tokens;
        const int64_t from =
            ok ? int64_t(page) * a.c.page_b + int64_t(off) * a.c.token_b +
                     int64_t(seg.h) * a.c.head_b
               : -1;
        float ku = 0, vs = 0;
        if (CODES && ok) {
          const int64_t so = (int64_t(page) * a.c.heads + seg.h) *
                                 a.c.page_tokens + off;
          ku = a.c.ks[so] * unit;
          vs = a.c.vs[so];
        }
        const uint32_t seen = __ballot_sync(0xffffffffu, ok);
        page = look(t + 1);
        const int slot = tile % NS;
        const uint32_t turn = tile / NS & 1;
        const uint32_t to = lw * KPW * 128;
        if constexpr (CODES) {
          uint4 kr[IT], vr[IT];
#pragma unroll
          for (int i = 0; i < IT; ++i) {
            const int64_t o = __shfl_sync(0xffffffffu, from, i * RPI + r0);
            kr[i] = vr[i] = make_uint4(0, 0, 0, 0);
            if (o >= 0 && held) {
              kr[i] = *reinterpret_cast<const uint4*>(a.c.k + o + c * 16);
              vr[i] = *reinterpret_cast<const uint4*>(a.c.v + o + c * 16);
            }
          }
          float top = fabsf(vs);
#pragma unroll
          for (int k = 16; k; k /= 2)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (tile >= NS)
              acquire(kv ? v_empty(slot) : k_empty(slot), turn ^ 1);
            if (!alive) break;
            if (kv == 0) {
              // (see NM: nothing reads these any more)
              char* const m = metas + tile % NM * S::kMeta;
              if (KPW == 32 || lane < KPW) {
                float* f = reinterpret_cast<float*>(m) + lw * KPW + lane;
                f[0] = ku;
                f[NK] = vs;
              }
              if (lane == 0) {
                uint32_t* w = reinterpret_cast<uint32_t*>(m + NK * 8);
                w[lw] = seen;
                w[4 + lw] = __float_as_uint(top);
              }
            }
            const uint32_t tile_s = (kv ? v_s : k_s) + slot * S::kTile + to;
            if (held) {
#pragma unroll
              for (int i = 0; i < IT; ++i) {
                const int r = i * RPI + r0;
                uint32_t y[8];
                if (kv)
                  widen16<STORE, true>(vr[i], y);
                else
                  widen16<STORE, QBF>(kr[i], y);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const int ch = 2 * c + j;
                  st_smem16(tile_s + ch / 8 * (NK * 128) + r * 128 +
                                ((ch ^ r) & 7) * 16,
                            y[4 * j], y[4 * j + 1], y[4 * j + 2],
                            y[4 * j + 3]);
                }
              }
            }
            smem_to_products();
            mbar_arrive(kv ? v_full(slot) : k_full(slot));
          }
        } else {
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            if (tile >= NS)
              acquire(kv ? v_empty(slot) : k_empty(slot), turn ^ 1);
            if (!alive) break;
            if (kv == 0 && lane == 0)
              reinterpret_cast<uint32_t*>(metas + tile % NM * S::kMeta +
                                          NK * 8)[lw] = seen;
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
            cp_commit();
            // two copies stay in flight; the one before them has come
            const uint32_t bar = kv ? v_full(slot) : k_full(slot);
            if (pending == 2) {
              cp_wait<2>();
              smem_to_products();
              mbar_arrive(announce[0]);
              announce[0] = announce[1];
              announce[1] = bar;
            } else {
              announce[pending++] = bar;
            }
          }
        }
      }
    }
    if (!CODES) announce_all();
  } else if (warp == 12) {
    // --- products: one thread ---
    if (lane == 0) {
      const uint32_t kind_s = mma_kind(QBF, false, 128, NK);
      const uint32_t kind_o = mma_kind(VBF, true, 128, dim16);
      const int ks = dim16 / 16;
      int tile = 0, nth = 0;
      int n_p[2] = {0, 0}, n_o[2] = {0, 0};
      bool alive = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (alive && !gate(bar, parity, &dead)) alive = false;
        tmem_after_sync();
        return alive;
      };
      while (alive && walk.next(a, &seg)) {
        const bool split = split_of(seg);
        const int per = split || QT == 1 ? 1 : (seg.rows + 127) / 128;
        const int units = seg.steps * per;
        // unit u: key tile u / per, and which half of the exponential warps
        // has it
        auto q_of = [&](int u) {
          return split ? u & 1 : per == 2 ? u & 1 : 0;
        };
        const int ahead = split || per == 2 ? 2 : 1;
        auto score = [&](int u) {
          const int j = u / per, t = tile + j, slot = t % NS, q = q_of(u);
          if (u % per == 0 && !wait(k_full(slot), t / NS & 1)) return;
          const uint32_t qa = q_s + (split ? 0 : q) * S::kQ;
          const uint32_t ka = k_s + slot * S::kTile;
          for (int k = 0; k < ks; ++k)
            mma_ss(tmem + q * NK,
                   smem_operand(qa + k / 4 * (128 * 128) + k % 4 * 32, 16, 1024),
                   smem_operand(ka + k / 4 * (NK * 128) + k % 4 * 32, 16, 1024),
                   kind_s, k > 0);
          mma_commit(s_full(q));
          if (u % per == per - 1) mma_commit(k_empty(slot));
          if (u == units - 1) mma_commit(q_empty);
        };
        if (!wait(q_full, nth & 1)) break;
        ++nth;
        for (int u = 0; u < ahead && u < units; ++u) score(u);
        for (int u = 0; u < units && alive; ++u) {
          const int j = u / per, t = tile + j, slot = t % NS, q = q_of(u);
          if (!wait(p_full(q), n_p[q]++ & 1)) break;
          if (u % per == 0 && !wait(v_full(slot), t / NS & 1)) break;
          const bool first = split ? u < 2 : j == 0;
          if (first && n_o[q] > 0 && !wait(o_empty(q), (n_o[q] - 1) & 1)) break;
          const uint32_t va = v_s + slot * S::kTile;
          const uint32_t o = tmem + S::kOut + q * D;
#pragma unroll
          for (int part = 0; part < PARTS; ++part)
            for (int i = 0; i < NK / 16; ++i)
              mma_ts(o,
                     tmem + q * NK + i / 2 * 32 + part * 16 + i % 2 * 8,
                     smem_operand(va + i * 2048, NK * 128, 1024), kind_o,
                     !(first && part == 0 && i == 0));
          if (u % per == per - 1) mma_commit(v_empty(slot));
          if (u + (split ? 2 : per) >= units) {
            mma_commit(o_full(q));
            ++n_o[q];
          }
          if (u + ahead < units) score(u + ahead);
        }
        tile += seg.steps;
      }
      if (dead) {
        // products may still read shared memory and write tensor memory
        mma_commit(drain);
        mbar_wait(drain, 0, kDrainCycles);
      }
    }
    __syncwarp();
  } else {
    // --- exponentials: a row a thread ---
    const int q = warp / 4;
    const int row = warp % 4 * 32 + lane;
    const uint32_t quarter = uint32_t(warp % 4 * 32) << 16;
    const uint32_t s_at = tmem + q * NK + quarter;
    const uint32_t o_at = tmem + S::kOut + q * D + quarter;
    const float unit = fabsf(a.scale) * 1.44269504088896341f;
    int tile = 0, n_s = 0, n_o = 0;
    bool alive = true;
    while (alive && walk.next(a, &seg)) {
      const bool split = split_of(seg);
      const int t_first = tile;
      tile += seg.steps;
      if (!split && q * 128 >= seg.rows) continue;
      float m = -INFINITY, l = 0, gain = 1;
      bool gained = false;
      // the reference's weight, as a power of two
      const float off =
          VBF ? -float(8 + 32 - __clz(seg.steps * NK)) : 12.f;
      bool first = true;
      for (int j = split ? q : 0; j < seg.steps; j += split ? 2 : 1) {
        if (!warp_gate(s_full(q), n_s++ & 1, &dead)) {
          alive = false;
          break;
        }
        tmem_after_sync();
        const char* const meta = metas + (t_first + j) % NM * S::kMeta;
        const float* const ku = reinterpret_cast<const float*>(meta);
        const uint32_t* const words =
            reinterpret_cast<const uint32_t*>(meta + NK * 8);
        uint32_t seen[NK / 32];
        bool part = false;
#pragma unroll
        for (int i = 0; i < NK / 32; ++i) {
          seen[i] = KPW == 32 ? words[i] : words[2 * i] | words[2 * i + 1] << 16;
          part |= seen[i] != 0xffffffffu;
        }
        // the largest score
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < NK / 32; ++c) {
          uint32_t r[32];
          tmem_ld32(r, s_at + c * 32);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x = __uint_as_float(r[i]);
            if (CODES) x *= ku[c * 32 + i];
            if (part && !(seen[c] >> i & 1)) x = -INFINITY;
            top = fmaxf(top, x);
          }
        }
        if (!CODES) top *= unit;
        const bool move = top > m + SLACK;
        // values' scales are met times `gain`, a power of two: the largest of
        // the first tile lies at 1, and one that passes 2^40 sets it again
        float scale_o = 1;
        bool change = move;
        if (CODES) {
          float big = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            big = fmaxf(big, __uint_as_float(words[4 + i]));
          if (big > 0 && (!gained || big * gain > 0x1p40f)) {
            const int e = min(max(127 - int(__float_as_uint(big) >> 23), -120),
                              120);
            const float next = __int_as_float((127 + e) << 23);
            scale_o = next / gain;
            gain = next;
            gained = change = true;
          }
        }
        if (__any_sync(0xffffffffu, change)) {
          if (move) {
            const float keep = ex2(m - top);
            l *= keep;
            scale_o *= keep;
            m = top;
          }
          __syncwarp();
          if (!first) {
#pragma unroll 1
            for (int c = 0; c < dim; c += 32) {
              uint32_t r[32];
              tmem_ld32(r, o_at + c);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i)
                r[i] = __float_as_uint(__uint_as_float(r[i]) * scale_o);
              tmem_st32(o_at + c, r);
            }
          }
        }
        first = false;
        const float sub = (m == -INFINITY ? 0.f : m) - off;
#pragma unroll
        for (int c = 0; c < NK / 32; ++c) {
          uint32_t r[32], hi[16], lo[16];
          tmem_ld32(r, s_at + c * 32);
          tmem_wait_ld();
          float sum = 0;
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float w[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float x = __fmaf_rn(__uint_as_float(r[i + k]),
                                  CODES ? ku[c * 32 + i + k] : unit, -sub);
              if (part && !(seen[c] >> (i + k) & 1)) x = -INFINITY;
              w[k] = ex2(x);
              sum += w[k];
              if (CODES) w[k] *= ku[NK + c * 32 + i + k] * gain;
            }
            hi[i / 2] = pair16<VBF>(w[0], w[1]);
            if (PARTS == 2) {
              const float2 f = unpair16<VBF>(hi[i / 2]);
              lo[i / 2] = pair16<VBF>(w[0] - f.x, w[1] - f.y);
            }
          }
          l += sum;
          tmem_st16(s_at + c * 32, hi);
          if (PARTS == 2) tmem_st16(s_at + c * 32 + 16, lo);
        }
        tmem_wait_st();
        tmem_before_sync();
        mbar_arrive(p_full(q));
      }
      if (!alive) break;
      // --- the rows' states ---
      const bool none = first;                   // no tile of keys
      if (!none) {
        if (!warp_gate(o_full(q), n_o & 1, &dead)) break;
        ++n_o;
        tmem_after_sync();
      }
      const bool whole = seg.steps == seg.s.tiles;
      const int r = split ? row : q * 128 + row;
      const bool valid = r < seg.rows;
      const int rg = seg.rt * S::kRows + r;
      const int si = rg / a.group;
      const int sub = split ? q : 0;
      const int64_t out_row =
          int64_t(sub) * a.seqs * a.heads_q +
          int64_t(seg.s.start + si) * a.heads_q + seg.h * a.group +
          (rg - si * a.group);
      const int part_row = q * 128 + row;
      float* const part =
          a.parts + (2 * int64_t(blockIdx.x) +
                     (share.begin < seg.item_at ? 1 : 0)) *
                        (int64_t(S::kRows) * (D + 2));
      // weights were taken times 2^off (and the values' gain)
      const float f = l == 0 ? 0.f : __fdividef(1.f, l);
      if (valid) {
        const float2 ml = make_float2(none ? -INFINITY : m - off, l);
        if (whole)
          reinterpret_cast<float2*>(a.state)[out_row] = ml;
        else
          reinterpret_cast<float2*>(part)[part_row] = ml;
      }
      if (!none) {
        const int ge = 127 - (__float_as_int(gain) >> 23);
        const float g1 = __int_as_float((127 + ge / 2) << 23);
        const float g2 = __int_as_float((127 + ge - ge / 2) << 23);
#pragma unroll 1
        for (int c = 0; c < dim; c += 32) {
          uint32_t x[32];
          __syncwarp();
          tmem_ld32(x, o_at + c);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            if (!valid || c + i >= dim) break;
            float4 y;
            float* const ys = &y.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              ys[k] = __uint_as_float(x[i + k]) * f;
              if (CODES) ys[k] = ys[k] * g1 * g2;
            }
            float* to = whole ? a.mean + out_row * dim + c + i
                              : part + 2 * S::kRows +
                                    (int64_t((c + i) / 4) * S::kRows +
                                     part_row) * 4;
            *reinterpret_cast<float4*>(to) = y;
          }
        }
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

template <int ELEM, int STORE, int D>
int launch_shared_d(const KvSharedArgs& a, cudaStream_t st) {
  using S = SharedShape<D>;
  int sms = 0, dev = 0;
  const int rc = kv_device(&dev, &sms);
  if (rc != LM_OK) return rc;
  auto* kernel = lm_kv_shared_kernel<ELEM, STORE, D>;
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

template <int STORE>
int launch_shared_store(const KvSharedArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int d = shared_dim(a.c.dim);
  if (a.elem == LM_BF16)
    return d == 64    ? launch_shared_d<LM_BF16, STORE, 64>(a, st)
           : d == 128 ? launch_shared_d<LM_BF16, STORE, 128>(a, st)
                      : launch_shared_d<LM_BF16, STORE, 256>(a, st);
  return d == 64    ? launch_shared_d<LM_F16, STORE, 64>(a, st)
         : d == 128 ? launch_shared_d<LM_F16, STORE, 128>(a, st)
                    : launch_shared_d<LM_F16, STORE, 256>(a, st);
}

}  // namespace lm
