// The largest numbers of a list, in the order of the list: which pages an
// attention reads, which tokens an eviction keeps.
#pragma once

#include <atomic>

#include "lm_kv_device.cuh"

namespace lm {

// A number's place in the order of numbers, as a whole one: -0 and 0 are the
// same, and a NaN is above all.
__device__ __forceinline__ uint32_t order_of(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ (u >> 31 ? 0xffffffffu : 0x80000000u);
}

constexpr int kTopBins = 2048;

template <int T>
struct TopSpace {
  uint32_t bins[kTopBins];
  uint32_t warp_a[T / 32], warp_b[T / 32];
  uint32_t found[3];                 // a bin, how many lie above it, and in it
  uint32_t rank_a, rank_b;           // the block's counts
};

template <int C>
__device__ __forceinline__ void cluster_sync() {
  if (C == 1) {
    __syncthreads();
  } else {
    asm volatile("barrier.cluster.arrive.aligned;\n" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
  }
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
// A word of the same variable in block `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_word(const uint32_t* p,
                                                 uint32_t rank) {
  uint32_t at, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n"
               : "=r"(at)
               : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n"
               : "=r"(v)
               : "r"(at)
               : "memory");
  return v;
}

__device__ __forceinline__ void cluster_put(uint32_t* p, uint32_t rank,
                                            uint32_t v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n"
               : "=r"(at)
               : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(at), "r"(v)
               : "memory");
}

// Of numbers i in [0, m) the `need` (0 < need <= m) that are largest by
// key(i), the lowest i where they are equal, to put(place, i) with places
// rising with i, by the T threads of each of a cluster's C blocks: every block
// has a part of the list, held in `cache` where its `cap` words suffice.
//
// A key's 32 bits in three steps (11, 11 and 10 from the top): the counts of
// each value of a step's bits among the keys that agree with the threshold so
// far give the threshold's own.  Then places: counts of what is taken before
// each warp's part of the list.
template <int T, int C, class Key, class Put>
__device__ __forceinline__ void take_top(int m, int need, uint32_t* cache,
                                         int cap, TopSpace<T>* sh, Key&& key,
                                         Put&& put) {
  constexpr int W = T / 32;
  // a block has kTopBins / C of the bins to add up and look through, PER a
  // thread
  constexpr int PER = (kTopBins / C + T - 1) / T;
  static_assert(kTopBins / C % PER == 0, "whole threads");
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int rank = C == 1 ? 0 : int(cluster_rank());
  const int i0 = int(int64_t(m) * rank / C);
  const int n = int(int64_t(m) * (rank + 1) / C) - i0;
  const bool held = n <= cap;
  if (held)
    for (int at = threadIdx.x; at < n; at += 4 * T) {
      uint32_t k[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at + e * T < n) k[e] = key(i0 + at + e * T);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at + e * T < n) cache[at + e * T] = k[e];
    }
  auto at = [&](int i) { return held ? cache[i] : key(i0 + i); };

  uint32_t prefix = 0;
  uint32_t left = uint32_t(need);    // to take among the keys that agree
  uint64_t floor = 0;                // every key from here on is taken
  uint32_t tie = 0;                  // and `left` of those that are this
  bool whole = false;
#pragma unroll
  for (int step = 0; step < 3; ++step) {
    const int bits = step == 2 ? 10 : 11;
    const int shift = step == 0 ? 21 : step == 1 ? 10 : 0;
    for (int i = threadIdx.x; i < kTopBins; i += T) sh->bins[i] = 0;
    __syncthreads();
    if (!whole)
      for (int i = threadIdx.x; i < n; i += T) {
        const uint32_t k = at(i);
        if (step == 0 || k >> (shift + bits) == prefix)
          atomicAdd(&sh->bins[(k >> shift) & ((1u << bits) - 1)], 1u);
      }
    cluster_sync<C>();
    // The bins from the top: the first block has the first of them, thread t
    // PER of its own.
    uint32_t mine[PER], sum = 0;
    const int first = rank * (kTopBins / C) + int(threadIdx.x) * PER;
    const bool has = int(threadIdx.x) * PER < kTopBins / C;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      mine[i] = 0;
      if (has) {
        const int bin = kTopBins - 1 - (first + i);
        if (C == 1) {
          mine[i] = sh->bins[bin];
        } else {
          uint32_t v[C];
#pragma unroll
          for (int r = 0; r < C; ++r) v[r] = cluster_word(&sh->bins[bin], r);
#pragma unroll
          for (int r = 0; r < C; ++r) mine[i] += v[r];
        }
      }
      sum += mine[i];
    }
    uint32_t upto = sum;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += v;
    }
    if (lane == 31) sh->warp_a[warp] = upto;
    __syncthreads();
    uint32_t above = upto - sum, all = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (w < warp) above += sh->warp_a[w];
      all += sh->warp_a[w];
    }
    if (C > 1) {
      if (threadIdx.x == 0) sh->rank_a = all;
      cluster_sync<C>();
      uint32_t v = lane < rank ? cluster_word(&sh->rank_a, lane) : 0;
      above += __reduce_add_sync(0xffffffffu, v);
    }
    if (!whole && above < left && left <= above + sum) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (above < left && left <= above + mine[i]) {
          const uint32_t f[3] = {uint32_t(kTopBins - 1 - (first + i)), above,
                                 mine[i]};
#pragma unroll
          for (int e = 0; e < 3; ++e) {
            if (C == 1) {
              sh->found[e] = f[e];
            } else {
#pragma unroll
              for (int r = 0; r < C; ++r) cluster_put(&sh->found[e], r, f[e]);
            }
          }
        }
        above += mine[i];
      }
    }
    // (the cluster's: no block clears its bins before all have read them)
    cluster_sync<C>();
    if (!whole) {
      prefix = prefix << bits | sh->found[0];
      left -= sh->found[1];
      if (sh->found[2] == left) {    // all that agree are taken
        whole = true;
        floor = uint64_t(prefix) << shift;
      } else if (step == 2) {
        floor = uint64_t(prefix) + 1;
        tie = prefix;
      }
    }
    __syncthreads();
  }
  if (whole) left = 0;

  // what each warp's part of the list has of those above and at the threshold
  const int w0 = int(int64_t(n) * warp / W), w1 = int(int64_t(n) * (warp + 1) / W);
  uint32_t above = 0, equal = 0;
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = at(i);
    above += k >= floor;
    equal += left && k == tie;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    sh->warp_a[warp] = above;
    sh->warp_b[warp] = equal;
  }
  __syncthreads();
  uint32_t a0 = 0, e0 = 0, a1 = 0, e1 = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < warp) {
      a0 += sh->warp_a[w];
      e0 += sh->warp_b[w];
    }
    a1 += sh->warp_a[w];
    e1 += sh->warp_b[w];
  }
  if (C > 1) {
    if (threadIdx.x == 0) {
      sh->rank_a = a1;
      sh->rank_b = e1;
    }
    cluster_sync<C>();
    for (int r = 0; r < rank; ++r) {
      a0 += cluster_word(&sh->rank_a, r);
      e0 += cluster_word(&sh->rank_b, r);
    }
  }
  for (int i = w0; i < w1; i += 32) {
    const bool in = i + lane < w1;
    const uint32_t k = in ? at(i + lane) : 0;
    const uint32_t ma = __ballot_sync(0xffffffffu, in && k >= floor);
    const uint32_t me = __ballot_sync(0xffffffffu, in && left && k == tie);
    const uint32_t low = (1u << lane) - 1;
    const uint32_t ra = a0 + __popc(ma & low), re = e0 + __popc(me & low);
    const bool is_e = me >> lane & 1;
    if ((ma >> lane & 1) || (is_e && re < left))
      put(int(ra + min(re, left)), i0 + i + lane);
    a0 += __popc(ma);
    e0 += __popc(me);
  }
  if (C > 1) cluster_sync<C>();      // nothing of this block is read from now
}

// The blocks of a list and their threads: a small block (256 lists of 1024: 9 us,
// 18 with large ones), a large one for a list that a small one does not hold or a
// few long ones, and eight where no block holds the list (its numbers would be
// read again in every step: 8 lists of 100003, 703 us against 31).
constexpr int kTopCluster = 8, kTopThreads = 256, kTopMore = 1024;
constexpr int kTopHeld = 8192, kTopHeldMore = 40960;
struct TopPlan {
  bool clusters, more;
  int held;                          // numbers that a block holds
};
inline TopPlan top_plan(int64_t lists, int64_t longest, int sms) {
  TopPlan p;
  p.more = longest > kTopHeld || (longest > 4096 && lists <= int64_t(sms));
  p.clusters = longest > kTopHeldMore;
  const int64_t n =
      p.clusters ? (longest + kTopCluster - 1) / kTopCluster : longest;
  const int most = p.more ? kTopHeldMore : kTopHeld;
  p.held = int(n < most ? n : most);
  return p;
}
// Launches the form of a kernel that a plan asks for; `small`, `large` and
// `eight` are its forms <kTopThreads, 1>, <kTopMore, 1> and <kTopMore, 8>.
template <class... P, class A>
int launch_top(void (*small)(P...), void (*large)(P...), void (*eight)(P...),
               std::atomic<uint64_t>* allowed, int dev, const TopPlan& plan,
               uint64_t lists, cudaStream_t st, const A& a) {
  if (!(allowed->load() >> dev & 1)) {
    for (auto* kernel : {large, eight}) {
      const cudaError_t e = cudaFuncSetAttribute(
          kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
          kTopHeldMore * 4);
      if (e != cudaSuccess) {
        set_cuda_error(int(e));
        return LM_E_CUDA;
      }
    }
    allowed->fetch_or(uint64_t(1) << dev);
  }
  if (plan.clusters)
    return launch_clusters(eight, kTopCluster, lists * kTopCluster, kTopMore,
                           plan.held * 4, st, a, plan.held);
  return plan.more
             ? launch(large, lists, kTopMore, plan.held * 4, st, a, plan.held)
             : launch(small, lists, kTopThreads, plan.held * 4, st, a,
                      plan.held);
}

}  // namespace lm
