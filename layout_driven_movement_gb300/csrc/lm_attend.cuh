// Attention of one new token per sequence over the paged cache: the kernel.
// Each of the four lm_attend_*.cu files compiles it for one kind of cache.
//
// For one key head of one sequence, its G query heads q_g and its keys and
// values k_j, v_j:  s_gj = scale q_g . k_j,  o_g = sum_j e^{s_gj} v_j / sum_j
// e^{s_gj}.  One pass over the cache with a running maximum m, sum l and
// unnormalised output o: a block of keys turns (m, l, o) into
// (m', l 2^(m-m') + sum 2^(s-m'), o 2^(m-m') + sum 2^(s-m') v), scores in
// units of ln 2.  Where two states join they hold the weighted mean o / l in
// o's place, (m, l, a): with c = l 2^(m-t) for each, t the larger m, the joined
// mean is sum (c / sum c) a, which is finite where the values are, however
// large they and their number.
//
// The cache is read once and nothing else matters: 4 G D operations per key
// head and token against 4 D (2 D at 8 bits) bytes.  At 6.8 TB/s an SM gets
// some 24 bytes a cycle, that is 16 keys and values of 128 16-bit elements in
// 340 cycles, and their two products with up to 8 queries are 16 warp-level
// 16x8x16 matrix instructions, a tenth of what the SM does in that time.  So
// the warp-level instruction is used and not the one that takes whole 128-row
// tiles: keys are its 16 rows and queries its 8 columns (S^T = K Q^T, O^T =
// V^T P^T), so that no row is wasted on a group of 8 or fewer, no barrier
// stands between a key's arrival and its use, and 8-bit codes can be widened
// on their way from shared memory to registers.
//
// Work.  Each warp of a block streams keys of its own: KW keys and their
// values a step, through a ring of kS stages filled by 16-byte asynchronous
// copies (a page table lookup per key, one step ahead, so any page size and
// any strides do), consumed with no barrier but the warp's own.  The grid is
// the resident blocks; the tiles (4 KW keys of one sequence and head) of all
// sequences are one line cut into equal parts, so ragged batches and single
// long sequences load all SMs alike.  A block's ring runs on across the
// borders of sequences.  HP adjacent heads share a block (its warps take them
// in turn) where their rows share memory lines.  What one block holds of a head that others share
// goes to the workspace as (m, l, a); the block that comes last by a counter
// joins the parts, in the order of the line, so results do not depend on
// which came last.
//
// Measured (bytes that cannot be done without / time): 64 sequences of up to
// 8192 tokens, 8 key heads x 4 queries x 128 bf16, pages of 16: 248 us, 6.4
// TB/s; 128 of up to 12288, 8 x 8 x 128 e4m3, pages of 64: 405 us, 6.1 TB/s; 3
// of up to 131072, 4 x 5 x 64 int8, pages of 40: 52 us, 2.8 TB/s (its step's
// instructions are as many for rows half as long); one of 500 tokens: 8.4 us
// of latency.
#pragma once

#include <atomic>
#include <type_traits>

#include "lm_kv_device.cuh"

namespace lm {

// Kinds of cache: the type of the matrix instructions' operands and how the
// held bytes become it.
enum AttendKind { KIND_BF16, KIND_F16, KIND_E4M3, KIND_INT8 };

constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = 32 * kAttendWarps;
constexpr int kAttendRun = 16;   // parts of a head joined at once, at most

template <int KIND, int D, int NT, int HP>
struct AttendShape {
  static constexpr bool kCodes = KIND == KIND_E4M3 || KIND == KIND_INT8;
  static constexpr int kHeld = kCodes ? 1 : 2;           // bytes an element
  // keys of a warp's step
  static constexpr int KW = kCodes ? (D == 64 ? 64 : D == 128 ? 32 : 16) : 16;
  static constexpr int KL = (KW + 31) / 32;              // keys a lane
  static constexpr int WK = kAttendWarps / HP;           // warps a head
  static constexpr int TK = KW * WK;                     // keys of a tile
  static constexpr int MT = KW / 16;                     // row tiles of S^T
  static constexpr int Q = 8 * NT;                       // queries
  static constexpr int kRow = D * kHeld;                 // bytes of a row
  static constexpr int kPart = KW * kRow;                // a warp's K or V
  static constexpr int kStage = kAttendWarps * 2 * kPart;
  // blocks per SM and stages: what shared memory holds.  Widening codes is
  // latency that only more warps hide: 128 sequences of 12288 tokens, 8 x 8 x
  // 128 e4m3, take 390 us with three blocks of two stages an SM, 481 with two
  // of three.  16 queries of 128 elements do not fit a third block's
  // registers: 64 sequences of 8192 tokens, 8 x 16, take 256 us (80 elements,
  // e4m3) and 327 (128, int8) with two blocks, 263 and 330 with three.
  static constexpr bool kTwo = D == 256 || (D == 128 && NT == 2);
  static constexpr int kBlocks = kCodes ? (kTwo ? 2 : 3) : D == 256 ? 1 : 2;
  static constexpr int kS = D == 256  ? 3
                            : kCodes ? (kTwo ? 3 : 2)
                                     : (D == 64 ? 6 : 3);
  static constexpr int kScales = kCodes ? kAttendWarps * 2 * KW * 4 : 0;
  static constexpr int kMasks = kAttendWarps * KL * 4;
  static constexpr int kState = kAttendWarps * Q * 2 * 4;
  static constexpr int kSmem =
      kS * (kStage + kScales + kMasks) + kState + 64;
  // workspace: a part is, for each head, (m, l) per query, then its mean
  static constexpr int kHeadFloats = Q * (D + 2);
  static constexpr int kPartFloats = HP * kHeadFloats;
  static_assert(Q * D * 4 <= 2 * kPart, "a warp's output fits its stage");
};

// --- instructions ------------------------------------------------------------

__device__ __forceinline__ void cp16(uint32_t dst, const void* src,
                                     uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src,
                                    uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;\n" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldm(uint32_t* r, uint32_t addr) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void ldm_t(uint32_t* r, uint32_t addr) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(addr)
      : "memory");
}
// The transpose of an 8x8 matrix of 16-bit elements held across the warp.
__device__ __forceinline__ uint32_t mov_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n"
               : "=r"(y)
               : "r"(x));
  return y;
}
template <bool BF>
__device__ __forceinline__ void mma(float* c, const uint32_t* a,
                                    const uint32_t* b) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// 2^x; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// Two 32-bit numbers as a pair of 16-bit ones, the first in the low half.
template <bool BF>
__device__ __forceinline__ uint32_t pair16(float lo, float hi) {
  if (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool BF>
__device__ __forceinline__ float2 unpair16(uint32_t x) {
  if (BF)
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&x));
  return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// --- 8-bit codes as 16-bit floats -------------------------------------------
//
// Keys become f16, whose 11 bits hold any scaled query (bf16 or f16) they
// meet; values become bf16, so that weights of nearly any size meet them.

// Logic and byte moves run at half the rate of the rest and are what an 8-bit
// cache spends most of its instructions on, so each form below is the
// cheapest known for its bytes; "2 of 4" names the ones a pair is taken from
// (any pairing does for keys: the queries are laid out to match).

// One word by masks: where p is 0, the bits of q; where p is 1, those of r,
// turned where q is 1.
__device__ __forceinline__ uint32_t masked(uint32_t r, uint32_t p,
                                           uint32_t q) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;\n" : "=r"(y) : "r"(r), "r"(p), "r"(q));
  return y;
}
template <int KIND>
struct Codes;

// e4m3: keys by the conversion instruction (bytes 0 1 and 2 3).  Values:
// sign, 4 exponent bits (bias 7) and 3 mantissa bits moved onto the sign, the
// low exponent bits (bias 127) and the high mantissa bits of a bf16, the same
// number, subnormals included, times 2^-120, which is put back where the
// means are formed (bytes 0 2 and 1 3).
template <>
struct Codes<KIND_E4M3> {
  static __device__ __forceinline__ void keys(uint32_t r, uint32_t* y) {
    asm("{.reg .b16 a, b;\n mov.b32 {a, b}, %2;\n"
        " cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(y[0]), "=r"(y[1])
        : "r"(r));
  }
  static __device__ __forceinline__ void values(uint32_t r, uint32_t* y,
                                                uint32_t* top) {
    const uint32_t a = (r << 4) & 0x07f007f0u, b = (r >> 4) & 0x07f007f0u;
    *top = __vimax3_u16x2(*top, a, b);
    y[0] = a | ((r << 8) & 0x80008000u);
    y[1] = b | (r & 0x80008000u);
  }
  // Codes 0x7f and 0xff are not numbers, but become 480 * 2^-120 here, 0x07f0
  // above all others.  So the largest magnitudes' bits of a step are kept,
  // and where one is that, `nans` gives the step's elements again: NaN for
  // such a code and 0 for any other.  (128 sequences of up to 12288 tokens, 8
  // x 8 x 128: 389 us without the look, 405 with it; 411 and 425 where twice
  // the codes as bf16, or their product with 0, show that one is no number.)
  static __device__ __forceinline__ uint32_t nans(uint32_t y) {
    return ((((y & 0x07f007f0u) + 0x00100010u) >> 11) & 0x00010001u) * 0x7fc0u;
  }
  static __device__ __forceinline__ void values_nan(uint32_t r, uint32_t* y) {
    uint32_t top = 0;
    values(r, y, &top);
    y[0] = nans(y[0]);
    y[1] = nans(y[1]);
  }
};

// Whole numbers -128..127 (bytes 0 2 and 1 3).  Keys: with its sign bit
// turned the byte u = code + 128 under the high byte 0x64 is the f16 1024 + u;
// less 1152 it is the code.  Values: bf16 has 8 bits; the low 7 bits w under
// 0x43 are 128 + w, the sign bit alone under 0x43 is 128 or 256, and the
// difference is the code.
template <>
struct Codes<KIND_INT8> {
  static __device__ __forceinline__ void keys(uint32_t r, uint32_t* y) {
    const uint32_t m = 0x64806480u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = masked(i ? r >> 8 : r, 0x00ff00ffu, 0x64806480u);
      const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u),
                                *reinterpret_cast<const __half2*>(&m));
      y[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  static __device__ __forceinline__ void values(uint32_t r, uint32_t* y,
                                                uint32_t*) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t t = i ? r >> 8 : r;
      const uint32_t a = (t & 0x007f007fu) | 0x43004300u;
      const uint32_t b = (t & 0x00800080u) | 0x43004300u;
      const __nv_bfloat162 v =
          __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a),
                  *reinterpret_cast<const __nv_bfloat162*>(&b));
      y[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};
template <>
struct Codes<KIND_BF16> {
  static __device__ __forceinline__ void keys(uint32_t, uint32_t*) {}
  static __device__ __forceinline__ void values(uint32_t, uint32_t*,
                                                uint32_t*) {}
};
template <>
struct Codes<KIND_F16> : Codes<KIND_BF16> {};

// --- where in the line of work -----------------------------------------------

struct AttendGrid {
  int items = 1;        // (HP key heads) x (groups of Q queries)
  int groups = 1;       // groups of Q queries of a key head
  int shared_page = 0;  // the keys of a warp's step share a page
  int q_pairs = 0;      // the queries allow 4-byte loads
  // workspace: see attend_space
  unsigned int *counters = nullptr, *run_counters = nullptr;
  float *parts = nullptr, *runs = nullptr;
};

// a / b of numbers that are not negative; most are small, and a 64-bit
// division takes several times a 32-bit one's time.
__device__ __forceinline__ int64_t line_div(int64_t a, int64_t b) {
  if ((a | b) >> 31 == 0) return uint32_t(a) / uint32_t(b);
  return a / b;
}

struct AttendAt {
  int b, item, tile, lo, hi, first, n;
  int64_t left;         // tiles of the block's share from here on
};

template <int TK>
__device__ __forceinline__ void attend_span(const KvAttendArgs& a, int b,
                                            AttendAt* at) {
  int64_t n = a.lens[b];
  n = n < 0 ? 0 : n > a.max_tokens ? a.max_tokens : n;
  const int64_t first = a.window && n > a.window ? n - a.window : 0;
  at->n = int(n);
  at->first = int(first);
  at->lo = int(first / TK);
  at->hi = int((n + TK - 1) / TK);
}

// One tile on; past a head the next head, past a sequence the next one that
// has keys.
template <int TK>
__device__ __forceinline__ void attend_next(const KvAttendArgs& a, int items,
                                            AttendAt* at) {
  --at->left;
  if (++at->tile < at->hi || at->left <= 0) return;
  if (++at->item == items) {
    at->item = 0;
    do {
      attend_span<TK>(a, ++at->b, at);
    } while (at->hi <= at->lo);
  }
  at->tile = at->lo;
}

// --- the kernel ----------------------------------------------------------------

template <int KIND, int D, int NT, int HP>
__global__ void
__launch_bounds__(kAttendThreads, AttendShape<KIND, D, NT, HP>::kBlocks)
    lm_kv_attend_kernel(const __grid_constant__ KvAttendArgs a,
                        const __grid_constant__ AttendGrid g) {
  using S = AttendShape<KIND, D, NT, HP>;
  constexpr bool CODES = S::kCodes;
  constexpr bool KBF = KIND == KIND_BF16;    // bf16 keys in the products
  constexpr bool VBF = KIND != KIND_F16;     // bf16 values and weights
  // f16 weights are held times UP, see the weights below; the largest passes
  // 1 by up to 2^SLACK
  constexpr float UP = KIND == KIND_F16 ? 0x1p12f : 1.f;
  constexpr float DOWN = 1 / UP;
  constexpr float SLACK = KIND == KIND_F16 ? 3.f : 8.f;
  // Scales of 8-bit values may be any; a head's are taken times `gain`, a
  // power of two that the largest so far decides: it lies at 2^TOP when the
  // gain is set and passes MOST before it is set again, smaller ones are not
  // raised by more than 2^120.  With weights up to 2^8 and sums of 2^31 of
  // them the products stay finite (e4m3's are 2^-120 of themselves), and
  // values beside scales 2^95 (e4m3) or 2^170 (int8) times their own keep
  // their bits.
  constexpr int TOP = KIND == KIND_E4M3 ? 106 : 60;
  constexpr float MOST = KIND == KIND_E4M3 ? 0x1p118f : 0x1p76f;
  // bf16 values reach the end of 32 bits' range, so their weights' sum stays
  // below 1: a weight's reference lies ROOM above the largest score
  constexpr bool LOW = KIND == KIND_BF16;
  constexpr float ROOM = LOW ? 13.f : 0.f;
  constexpr int KW = S::KW, KL = S::KL, TK = S::TK, MT = S::MT, NS = S::kS;
  constexpr int Q = S::Q;
  constexpr int KS = D / 16;                 // 16-element steps along dim
  extern __shared__ __align__(1024) char smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int row8 = lane / 4, col2 = (lane % 4) * 2;
  const int sub = warp % HP, wk = warp / HP;   // the warp's head and keys
  const int dim = a.c.dim;

  char* const ring = smem;
  char* const scale_ring = ring + NS * S::kStage;
  uint32_t* const masks =
      reinterpret_cast<uint32_t*>(scale_ring + NS * S::kScales);
  float* const state = reinterpret_cast<float*>(masks + NS * kAttendWarps * KL);
  int64_t* const share = reinterpret_cast<int64_t*>(
      (reinterpret_cast<uintptr_t>(state + kAttendWarps * Q * 2) + 7) & ~7ull);
  const uint32_t ring_s = uint32_t(__cvta_generic_to_shared(ring));
  const uint32_t scale_s = uint32_t(__cvta_generic_to_shared(scale_ring));

  // A row's 16-byte chunks are permuted by an exclusive or with its number,
  // so that the 8 rows of a matrix load lie in different banks.  Rows and
  // stages are aligned to the row's size: the chunk of a step is then one
  // exclusive or away from the lane's first.
  auto turned = [](int r) { return S::kRow == 64 ? (r >> 1) & 3 : r & 7; };
  const uint32_t k_lane =
      lane % 16 * S::kRow + ((lane / 16) ^ turned(lane % 16)) * 16;
  // values: 16 keys by two chunks, or codes of 32 keys by one
  constexpr bool LONG = CODES && KW >= 32;
  const int v_row = LONG    ? lane
                    : CODES ? lane % 16
                            : lane % 8 + lane / 16 * 8;
  const int v_chunk = LONG ? 0 : CODES ? lane / 16 : lane / 8 & 1;
  const uint32_t v_lane = v_row * S::kRow + (v_chunk ^ turned(v_row)) * 16;

  // The line of work: every thread counts the tiles of a run of sequences;
  // a scan over the block gives the line's length and where this block's
  // share starts.
  stream_order();
  AttendAt at;
  int64_t total, begin;
  int64_t line_b;        // where sequence at.b starts on the line
  {
    const int per = (a.seqs + kAttendThreads - 1) / kAttendThreads;
    const int b0 = min(a.seqs, int(threadIdx.x) * per);
    const int b1 = min(a.seqs, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) {
      AttendAt s;
      attend_span<TK>(a, b, &s);
      mine += int64_t(s.hi - s.lo) * g.items;
    }
    int64_t sum = mine;
#pragma unroll
    for (int k = 1; k < 32; k *= 2) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sum, k);
      if (lane >= k) sum += v;
    }
    if (lane == 31) share[warp] = sum;
    __syncthreads();
    int64_t before = sum - mine;
    total = 0;
#pragma unroll
    for (int w = 0; w < kAttendWarps; ++w) {
      if (w < warp) before += share[w];
      total += share[w];
    }
    if (total == 0) {
      at.left = 0;
    } else {
      // as many blocks as the line feeds (at least two or four tiles for each
      // measured no faster, and slower from eight on)
      const int64_t blocks = min(total, int64_t(gridDim.x));
      const int64_t c = blockIdx.x;
      begin = line_div(c * total, blocks);
      at.left = c < blocks ? line_div((c + 1) * total, blocks) - begin : 0;
      if (at.left > 0 && begin >= before && begin < before + mine) {
        int b = b0;
        AttendAt s;
        for (;; ++b) {
          attend_span<TK>(a, b, &s);
          const int64_t k = int64_t(s.hi - s.lo) * g.items;
          if (begin < before + k) break;
          before += k;
        }
        share[4] = b;
        share[5] = before;
      }
      total = total * 65536 + blocks;      // both, for the join
    }
    __syncthreads();
  }
  const int64_t blocks = total & 65535;
  total >>= 16;

  if (at.left > 0) {
    at.b = int(share[4]);
    line_b = share[5];
    attend_span<TK>(a, at.b, &at);
    const int tiles = at.hi - at.lo;
    const int64_t in = begin - line_b;
    at.item = int(line_div(in, tiles));
    at.tile = at.lo + int(in - int64_t(at.item) * tiles);
  }

  // --- the ring's filling side ---
  AttendAt ld = at;
  struct Pages {
    // of this lane's keys of a tile or, where a step's keys share a page, of
    // all of them
    int of[KL];
  };
  constexpr int LPR = S::kRow / 16;            // lanes a row
  constexpr int RPI = 32 / LPR;                // rows an instruction
  const int c = lane % LPR, r0 = lane / LPR;
  // the products take 32 bytes of a row at a time; past dim they are 0
  const bool held = c * 16 < dim * S::kHeld;
  const bool used = c * 16 < (dim * S::kHeld + 31) / 32 * 32;
  const uint32_t to_lane = r0 * S::kRow;
  const int64_t from_lane = r0 * a.c.token_b + c * 16;
  const int64_t v_from_k = a.c.v - a.c.k;
  constexpr uint32_t full = KW >= 32 ? 0xffffffffu : (1u << KW % 32) - 1;
  auto fetch = [&](Pages* pg) {
    const int key0 = ld.tile * TK + wk * KW;
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      const int key = key0 + (g.shared_page ? 0 : lane + 32 * i);
      const int reach = g.shared_page ? KW : 1;
      pg->of[i] = -1;
      if (ld.left > 0 && (g.shared_page || KW >= 32 || lane < KW) &&
          key + reach > ld.first && key < ld.n && (i == 0 || !g.shared_page))
        pg->of[i] = a.table[int64_t(ld.b) * a.table_stride +
                            fdiv(uint32_t(key), a.c.page_div)];
      if (i && g.shared_page) pg->of[i] = pg->of[0];
    }
  };
  auto fill = [&](int stage, const Pages& pg) {
    const int key0 = ld.tile * TK + wk * KW;
    const uint32_t h = uint32_t(ld.item / g.groups * HP + sub);
    const uint32_t k_s = ring_s + stage * S::kStage + warp * 2 * S::kPart;
    uint32_t mask[KL], off[KL];
    int64_t from[KL];
    bool all = g.shared_page;
#pragma unroll
    for (int i = 0; i < KL; ++i) {
      const int at_key = key0 + lane + 32 * i;
      const bool in = (KW >= 32 || lane < KW) && at_key >= ld.first &&
                      at_key < ld.n;
      const bool ok = in && pg.of[i] >= 0 && pg.of[i] < a.c.pages;
      if (in && !ok && a.status) atomicOr(a.status, kStatusRange);
      mask[i] = __ballot_sync(0xffffffffu, ok);
      if (lane == 0) masks[(stage * kAttendWarps + warp) * KL + i] = mask[i];
      all = all && mask[i] == full;
      // (of a shared page, the step's first key)
      const uint32_t key = uint32_t(g.shared_page ? key0 : at_key);
      off[i] = key - fdiv(key, a.c.page_div) * a.c.page_tokens;
      from[i] = int64_t(pg.of[i]) * a.c.page_b +
                int64_t(off[i]) * a.c.token_b + int64_t(h) * a.c.head_b;
      if (CODES && (KW >= 32 || lane < KW)) {
        const int64_t so =
            ok ? (int64_t(pg.of[i]) * a.c.heads + h) * a.c.page_tokens +
                     off[i] + (g.shared_page ? lane + 32 * i : 0)
               : 0;
        const uint32_t to = scale_s + stage * S::kScales +
                            (warp * 2 * KW + lane + 32 * i) * 4;
        cp4(to, a.c.ks + so, ok ? 4 : 0);
        cp4(to + KW * 4, a.c.vs + so, ok ? 4 : 0);
      }
    }
    if (all) {
      const char* src = a.c.k + (from[0] + from_lane);
      if (used) {
        const uint32_t bytes = held ? 16 : 0;
        if (!held) src = a.c.k;
#pragma unroll
        for (int i = 0; i < KW / RPI; ++i) {
          const int r = i * RPI;
          const uint32_t to =
              k_s + to_lane + r * S::kRow + ((c ^ turned(r + r0)) * 16);
          cp16(to, src, bytes);
          cp16(to + S::kPart, src + v_from_k, bytes);
          if (held) src += RPI * a.c.token_b;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < KW / RPI; ++i) {
        const int r = i * RPI + r0, kl = i * RPI / 32;
        const int64_t o =
            (g.shared_page ? from[0] + r * a.c.token_b
                           : __shfl_sync(0xffffffffu, from[kl], r % 32)) +
            c * 16;
        const uint32_t bytes = held && (mask[kl] >> r % 32 & 1) ? 16 : 0;
        const uint32_t to = k_s + r * S::kRow + ((c ^ turned(r)) * 16);
        if (used) {
          cp16(to, a.c.k + (bytes ? o : 0), bytes);
          cp16(to + S::kPart, a.c.v + (bytes ? o : 0), bytes);
        }
      }
    }
  };

  // --- the queries, as they lie ---
  // as the second operand's fragments: lane row8 of a column tile holds
  // query row8's elements
  uint32_t qf[KS][NT][2];
  const bool q_pairs = g.q_pairs;
  auto load_q = [&](const AttendAt& p) {
    const int hp = p.item / g.groups, q0 = (p.item - hp * g.groups) * Q;
    const int h = hp * HP + sub;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int qi = nt * 8 + row8;
      const uint16_t* q = reinterpret_cast<const uint16_t*>(a.q.p) +
                          int64_t(p.b) * a.q.ts +
                          int64_t(h * a.group + q0 + qi) * a.q.hs;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        // as the keys' elements lie: codes come by the 4 of a lane
        const int d = k * 16 + (CODES ? 2 * col2 : col2);
        const int d2 = d + (CODES ? 2 : 8);
        uint32_t x = 0, y = 0;
        if (qi < a.group - q0 && d < dim) {
          if (q_pairs) {
            x = *reinterpret_cast<const uint32_t*>(q + d);
            if (d2 < dim) y = *reinterpret_cast<const uint32_t*>(q + d2);
          } else {
            x = q[d] | uint32_t(q[d + 1]) << 16;
            if (d2 < dim) y = q[d2] | uint32_t(q[d2 + 1]) << 16;
          }
        }
        // int8 pairs are elements 0 2 and 1 3
        qf[k][nt][0] = KIND == KIND_INT8 ? __byte_perm(x, y, 0x5410) : x;
        qf[k][nt][1] = KIND == KIND_INT8 ? __byte_perm(x, y, 0x7632) : y;
      }
    }
  };

  // the first steps' pages all at once, then their fills
  Pages next;
  if (at.left > 0) {
    Pages pg[NS - 1];
    AttendAt to[NS - 1];
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      to[s] = ld;
      fetch(&pg[s]);
      if (ld.left > 0) attend_next<TK>(a, g.items, &ld);
    }
    fetch(&next);
    load_q(at);
    const AttendAt on = ld;
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      ld = to[s];
      if (ld.left > 0) fill(s, pg[s]);
      cp_commit();
    }
    ld = on;
  }
  // sequences without keys
  for (int b = blockIdx.x; b < a.seqs; b += gridDim.x) {
    AttendAt s;
    attend_span<TK>(a, b, &s);
    if (s.hi > s.lo) continue;
    for (int e = threadIdx.x; e < a.heads_q * dim; e += kAttendThreads) {
      const int qi = e / dim, d = e - qi * dim;
      reinterpret_cast<uint16_t*>(a.out.p)[int64_t(b) * a.out.ts +
                                           int64_t(qi) * a.out.hs + d] = 0;
    }
    if (a.lse)
      for (int qi = threadIdx.x; qi < a.heads_q; qi += kAttendThreads)
        a.lse[int64_t(b) * a.heads_q + qi] = -INFINITY;
  }

  int stage = 0;
  while (at.left > 0) {
    // --- one head of one sequence: `steps` tiles of it ---
    const int hp = at.item / g.groups;
    const int q0 = (at.item - hp * g.groups) * Q;    // of a key head's
    const int nq = min(Q, a.group - q0);
    const int steps = int(min(at.left, int64_t(at.hi - at.tile)));

    // Codes are met by f16 queries, scaled by a power of two so that the
    // largest element lies in [2^14, 2^15): exact for bf16 elements down to
    // 2^-31 of it and f16 ones down to 2^-28, below that within 2^-39 of it.
    float fac[NT][2];
    const float unit = a.scale * 1.44269504088896341f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      fac[nt][0] = fac[nt][1] = unit;
      if (CODES) {
        const bool in_bf = a.elem == LM_BF16;
        float top = 0;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 v = in_bf ? unpair16<true>(qf[k][nt][j])
                                   : unpair16<false>(qf[k][nt][j]);
            top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e, e = 14 - floor(log2 top) within +-120
        int e = 14 + 127 - int(__float_as_uint(top) >> 23);
        if (top == 0 || top == INFINITY) e = 0;
        e = min(120, max(-120, e));
        const float up = __int_as_float((127 + e) << 23);
        const float down = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 v = in_bf ? unpair16<true>(qf[k][nt][j])
                                   : unpair16<false>(qf[k][nt][j]);
            qf[k][nt][j] = pair16<false>(v.x * up, v.y * up);
          }
        // the factor belongs to query row8; the scores' columns are
        // queries col2 and col2 + 1
        fac[nt][0] *= __shfl_sync(0xffffffffu, down, col2 * 4);
        fac[nt][1] *= __shfl_sync(0xffffffffu, down, col2 * 4 + 4);
      }
    }

    float m[NT][2], l[NT][2], o[KS][NT][4], gain = 0x1p120f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nt][j] = -INFINITY;
        l[nt][j] = 0;
      }
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[k][nt][i] = 0;

    for (int step = 0; step < steps; ++step) {
      __syncwarp();
      if (ld.left > 0) {
        fill(stage == 0 ? NS - 1 : stage - 1, next);
        attend_next<TK>(a, g.items, &ld);
        fetch(&next);
      }
      cp_commit();
      cp_wait<NS - 1>();
      __syncwarp();
      const uint32_t k_s = ring_s + stage * S::kStage + warp * 2 * S::kPart;
      const uint32_t v_s = k_s + S::kPart;
      uint32_t mask[KL];
      bool part = false;
#pragma unroll
      for (int i = 0; i < KL; ++i) {
        mask[i] = masks[(stage * kAttendWarps + warp) * KL + i];
        part |= mask[i] != full;
      }

      // S^T = K Q^T
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[mt][nt][i] = 0;
#pragma unroll
      for (int k = 0; k < KS; k += CODES ? 2 : 1) {
        if (k * 16 >= dim) break;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          // 16 bits: 16 rows by 16 elements; codes: by 32
          uint32_t x[4];
          ldm(x, (k_s + k_lane + mt * 16 * S::kRow) ^ (k * (CODES ? 16 : 32)));
          if (CODES) {
            uint32_t f[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t y[2];
              Codes<KIND>::keys(x[i], y);
              f[i / 2][i % 2] = y[0];
              f[i / 2][i % 2 + 2] = y[1];
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<false>(s[mt][nt], f[e], qf[k + e][nt]);
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<KBF>(s[mt][nt], x, qf[k][nt]);
          }
        }
      }

      // scores in units of ln 2; -infinity where no key is seen
      float ks[MT][2], vs[MT][2];
      const float* const sc = reinterpret_cast<const float*>(
                                  scale_ring + stage * S::kScales) +
                              warp * 2 * KW + row8;
      bool above = false;
      if (CODES) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ks[mt][i] = sc[mt * 16 + 8 * i];
            vs[mt][i] = sc[KW + mt * 16 + 8 * i] * gain;
            above |= fabsf(vs[mt][i]) > MOST;
          }
      }
      // A head's reference m moves only when a score passes the largest one
      // that it was set for by SLACK, that is when a weight would pass 2^SLACK
      // (LOW: 2^-5): one vote a step instead of the maximum over the lanes and the
      // products' rescaling.  LOW: and when a lane's sum passes 2^-4, so that
      // the 8 lanes' sums, with the step's 2 weights each, stay below 1 and
      // the products below the largest value.
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = s[mt][nt][i] * fac[nt][i & 1];
            if (CODES) x *= ks[mt][i >> 1];
            s[mt][nt][i] = x;
          }
      if (part) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (!(mask[mt / 2] >> (mt % 2 * 16 + 8 * r + row8) & 1)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                s[mt][nt][2 * r] = s[mt][nt][2 * r + 1] = -INFINITY;
            }
      }
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float t = s[0][nt][j];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            t = fmaxf(t, mt ? fmaxf(s[mt][nt][j], s[mt][nt][2 + j])
                            : s[mt][nt][2 + j]);
          top[nt][j] = t;
          above |= t > m[nt][j] + (SLACK - ROOM);
          if (LOW) above |= l[nt][j] > 0x1p-4f;
        }
      if (__any_sync(0xffffffffu, above)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            // over the 8 lanes that hold the column's keys
            float t = fmaxf(top[nt][j] + ROOM, m[nt][j]);
#pragma unroll
            for (int k = 4; k < 32; k *= 2)
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, k));
            if (LOW) {
              float sum = l[nt][j];
#pragma unroll
              for (int k = 4; k < 32; k *= 2)
                sum += __shfl_xor_sync(0xffffffffu, sum, k);
              // 2^e or more: down to 2^-9
              const int e = int(__float_as_uint(sum) >> 23) - 127;
              if (sum > 0x1p-5f) t = fmaxf(t, m[nt][j] + float(e + 9));
            }
            const float keep = ex2(m[nt][j] - (t == -INFINITY ? 0.f : t));
            m[nt][j] = t;
            l[nt][j] *= keep;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              o[k][nt][j] *= keep;
              o[k][nt][2 + j] *= keep;
            }
          }
        if (CODES) {
          float big = 0;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              big = fmaxf(big, fabsf(sc[KW + mt * 16 + 8 * i]));
#pragma unroll
          for (int k = 4; k < 32; k *= 2)
            big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, k));
          const int up =
              min(120, TOP + 127 - int(__float_as_uint(big) >> 23));
          const float next = fminf(gain, __int_as_float((127 + up) << 23));
          if (next != gain) {
            // (in two halves: the whole may be below 2^-126)
            const int by =
                (__float_as_int(next) >> 23) - (__float_as_int(gain) >> 23);
            const float by1 = __int_as_float((127 + by / 2) << 23);
            const float by2 = __int_as_float((127 + by - by / 2) << 23);
            gain = next;
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  o[k][nt][i] = o[k][nt][i] * by1 * by2;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 2; ++i)
                vs[mt][i] = sc[KW + mt * 16 + 8 * i] * gain;
          }
        }
      }
      // nothing seen yet: relative to 0, every weight is 0
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          top[nt][j] = m[nt][j] == -INFINITY ? 0.f : m[nt][j];

      // weights, and their transposes as the second operand.  A weight's 8
      // (bf16) or 11 (f16) bits alone would cost the result about as much as
      // its own rounding does, so what the rounding of a weight leaves goes
      // through the products too.  A value's scale is folded into its weight.
      //
      // f16 weights, held times UP, run up to 2^15.  Two f16 parts of one
      // below WEAK leave more than 2^-14 of it, and nothing at all of one
      // below 2^-26.  Such weak ones wait for products of their own; below
      // 2^-71 of the largest they add less than f16 holds, whatever their
      // number.
      constexpr float WEAK = 0x1p-11f;
      float weak[MT][NT][4];
      bool some_weak = false;
      uint32_t p[MT][NT][2], p2[MT][NT][2];
      auto operand = [&](int mt, int nt, int r, const float* w) {
        const uint32_t hi = pair16<VBF>(w[0], w[1]);
        const float2 f = unpair16<VBF>(hi);
        p[mt][nt][r] = mov_t(hi);
        p2[mt][nt][r] = mov_t(pair16<VBF>(w[0] - f.x, w[1] - f.y));
      };
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            float w[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              w[j] = ex2(s[mt][nt][2 * r + j] - top[nt][j]);
              l[nt][j] += w[j];
              if (CODES) w[j] *= vs[mt][r];
              if (UP != 1.f) w[j] *= UP;
              if (KIND == KIND_F16) {
                const bool is = w[j] < WEAK;
                float& x = weak[mt][nt][2 * r + j];
                x = is && w[j] >= WEAK * 0x1p-48f ? w[j] : 0.f;
                some_weak |= x > 0;
                if (is) w[j] = 0;
              }
            }
            operand(mt, nt, r, w);
          }

      // O^T += V^T P^T
      // codes: widened by `widen`, met by both parts of the weights or one
      auto code_products = [&](auto&& widen, auto both) {
#pragma unroll
        for (int k = 0; k < KS; k += CODES && !LONG ? 2 : 1) {
          if (k * 16 >= dim) break;
          uint32_t x[4];
          if constexpr (LONG) {                       // 32 keys, 16 elements
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              if (mt % 2 == 0)
                ldm_t(x, (v_s + v_lane + mt * 16 * S::kRow) ^ (k * 16));
              // elements 2i are the tile's rows 0-7, elements 2i + 1 its
              // rows 8-15
              uint32_t f[4];
              widen(x[mt % 2 * 2], f);
              widen(x[mt % 2 * 2 + 1], f + 2);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma<true>(o[k][nt], f, p[mt][nt]);
                if constexpr (decltype(both)::value) mma<true>(o[k][nt], f, p2[mt][nt]);
              }
            }
          } else {                                    // 16 keys, 32 elements
            ldm_t(x, (v_s + v_lane) ^ (k * 16));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t f[4];
              widen(x[2 * e], f);
              widen(x[2 * e + 1], f + 2);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma<true>(o[k + e][nt], f, p[0][nt]);
                if constexpr (decltype(both)::value) mma<true>(o[k + e][nt], f, p2[0][nt]);
              }
            }
          }
        }
      };
      auto products = [&] {
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          if (k * 16 >= dim) break;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            uint32_t x[4];
            ldm_t(x, (v_s + v_lane + mt * 16 * S::kRow) ^ (k * 32));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<VBF>(o[k][nt], x, p[mt][nt]);
              mma<VBF>(o[k][nt], x, p2[mt][nt]);
            }
          }
        }
      };
      if constexpr (CODES) {
        uint32_t code_top = 0;
        code_products(
            [&](uint32_t r, uint32_t* y) {
              Codes<KIND>::values(r, y, &code_top);
            },
            std::true_type{});
        if constexpr (KIND == KIND_E4M3) {
          if (__any_sync(0xffffffffu, (code_top + 0x00100010u) & 0x08000800u))
            code_products(Codes<KIND>::values_nan, std::false_type{});
        }
      } else {
        products();
      }
      if constexpr (KIND == KIND_F16) {
        // Weak weights 2^24 up, those that are still weak 2^48; the sums go
        // up with them and down again.  A step with a round of it takes about
        // half as long again: 64 sequences of 8192 tokens, 8 x 4 x 128, 325 us
        // where scores lie within some 15 of each other, 356 where they
        // deviate by 4 and 432 where by 12 (4 x 16 x 256, 32 sequences: 267,
        // 367 and 458).
        auto scale = [&](float by) {
#pragma unroll
          for (int k = 0; k < KS; ++k)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[k][nt][i] *= by;
        };
        float down = 1;
        while (__any_sync(0xffffffffu, some_weak)) {
          some_weak = false;
          down *= 0x1p-24f;
          scale(0x1p24f);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                float w[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  float& x = weak[mt][nt][2 * r + j];
                  x *= 0x1p24f;
                  const bool now = x >= WEAK;
                  w[j] = now ? x : 0;
                  if (now) x = 0;
                  some_weak |= x > 0;
                }
                operand(mt, nt, r, w);
              }
          products();
        }
        if (down != 1) scale(down);
      }
      if (++stage == NS) stage = 0;
    }

    // the warp's state: the sums over its lanes, and the means.  (Formed before
    // the next queries take registers: 32 sequences of 8192 tokens, 4 x 16 x
    // 256 bf16, 247 us so and 260 where the means are written.)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2], f2 = 1;
      if (CODES) {
        // 1 / gain, and the 2^120 of e4m3 values, in two halves
        const int e = (KIND == KIND_E4M3 ? 120 : 0) + 127 -
                      (__float_as_int(gain) >> 23);
        f[0] = f[1] = __int_as_float((127 + e / 2) << 23);
        f2 = __int_as_float((127 + e - e / 2) << 23);
      } else {
        f[0] = f[1] = DOWN;
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int k = 4; k < 32; k *= 2)
          l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], k);
        f[j] = l[nt][j] == 0 ? 0.f : __fdividef(f[j], l[nt][j]);
        if (row8 == 0) {
          float* st = state + (warp * Q + nt * 8 + col2 + j) * 2;
          st[0] = m[nt][j];
          st[1] = l[nt][j];
        }
      }
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          o[k][nt][i] = o[k][nt][i] * f[i & 1] * f2;
    }

    // the next head's queries are on their way while this one's parts join
    const AttendAt done = at;
    const int tiles = at.hi - at.lo;
    const int64_t item_at = line_b + int64_t(at.item) * tiles;
    at.left -= steps;
    at.tile += steps;
    if (at.left > 0) {
      if (++at.item == g.items) {
        line_b += int64_t(tiles) * g.items;
        at.item = 0;
        do {
          attend_span<TK>(a, ++at.b, &at);
        } while (at.hi <= at.lo);
      }
      at.tile = at.lo;
      load_q(at);
    }

    // --- the warps' states join; each warp's means lie in the stage that
    // it used last, which nothing fills before the next step ---
    const int used = stage == 0 ? NS - 1 : stage - 1;
    float* const mine = reinterpret_cast<float*>(
        ring + used * S::kStage + warp * 2 * S::kPart);
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // column col2 + j of the products is a query: its elements, the
          // words turned so that the warp's lanes hit all banks
          float* to = mine + (nt * 8 + col2 + j) * D;
          const int turn = col2 * 4;
          if (CODES) {
            const int d = (k * 16 + 2 * row8) ^ turn;
            *reinterpret_cast<float2*>(to + d) =
                make_float2(o[k][nt][j], o[k][nt][2 + j]);
          } else {
            to[(k * 16 + row8) ^ turn] = o[k][nt][j];
            to[(k * 16 + 8 + row8) ^ turn] = o[k][nt][2 + j];
          }
        }
    }
    __syncthreads();
    const bool whole = steps == tiles;
    const int64_t c0 = whole ? 0 : line_div((item_at + 1) * blocks - 1, total);
    const int64_t c1 =
        whole ? 0 : line_div((item_at + tiles) * blocks - 1, total);
    float* part = nullptr;
    if (!whole)
      part = g.parts +
             (2 * int64_t(blockIdx.x) + (begin < item_at ? 1 : 0)) *
                 S::kPartFloats;
    const bool out_bf = a.elem == LM_BF16;
    // query qi of the block's head i: its row, its outputs and its lse
    auto row_of = [&](int i, int qi) {
      return (hp * HP + i) * a.group + q0 + qi;
    };
    auto put = [&](int i, int qi, int d, float x) {
      char* to = a.out.p + (int64_t(done.b) * a.out.ts +
                            int64_t(row_of(i, qi)) * a.out.hs + d) * 2;
      if (out_bf)
        *reinterpret_cast<bf16*>(to) = from_f32<bf16>(x);
      else
        *reinterpret_cast<__half*>(to) = from_f32<__half>(x);
    };
    auto put_lse = [&](int i, int qi, float t, float sum) {
      if (a.lse)
        a.lse[int64_t(done.b) * a.heads_q + row_of(i, qi)] =
            sum == 0 ? -INFINITY
                     : (t + log2f(sum)) * 0.693147180559945309f;
    };
    for (int i = 0; i < HP; ++i)
      for (int e = threadIdx.x; e < nq * D; e += kAttendThreads) {
        const int qi = e / D, d = e % D;
        float t = -INFINITY, x = 0, sum = 0, c[S::WK];
#pragma unroll
        for (int w = 0; w < S::WK; ++w)
          t = fmaxf(t, state[((w * HP + i) * Q + qi) * 2]);
        const float t0 = t == -INFINITY ? 0.f : t;
#pragma unroll
        for (int w = 0; w < S::WK; ++w) {
          const float* st = state + ((w * HP + i) * Q + qi) * 2;
          c[w] = st[1] * ex2(st[0] - t0);
          sum += c[w];
        }
        const float part_of = sum == 0 ? 0.f : __fdividef(1.f, sum);
#pragma unroll
        for (int w = 0; w < S::WK; ++w)
          x += c[w] * part_of *
               reinterpret_cast<const float*>(
                   ring + used * S::kStage + (w * HP + i) * 2 * S::kPart)
                   [qi * D + (d ^ ((qi & 6) * 4))];
        if (whole) {
          if (d < dim) put(i, qi, d, sum == 0 ? 0.f : x);
          if (d == 0) put_lse(i, qi, t, sum);
        } else {
          float* to = part + i * S::kHeadFloats;
          to[2 * Q + qi * D + d] = x;
          if (d == 0) {
            to[2 * qi] = t;
            to[2 * qi + 1] = sum;
          }
        }
      }
    __syncthreads();
    if (!whole) {
      // The block that comes last joins the parts c0 .. c1.  Where they are
      // more than 16, even runs of up to 16 are joined first, each by the
      // last of its own blocks, and then the runs: no block reads more than a
      // few rounds of parts, 8 at once.
      const int n = int(c1 - c0) + 1;
      const int runs = (n + kAttendRun - 1) / kAttendRun;
      const int run = ((int(blockIdx.x) - int(c0) + 1) * runs - 1) / n;
      const int from = run * n / runs;
      const int size = (run + 1) * n / runs - from;
      // whether this block is the last of `count` to come by a counter, which
      // it then leaves at zero
      auto last_of = [&](unsigned int* counter, int count) {
        if (threadIdx.x == 0) {
          __threadfence();
          const unsigned before = atomicAdd(counter, 1u);
          __threadfence();
          share[6] = before == unsigned(count - 1);
          if (share[6]) *counter = 0;
        }
        __syncthreads();
        const bool last = share[6];
        __syncthreads();
        return last;
      };
      // the mean over parts 0 .. m - 1, 4 elements a thread at a time
      auto join = [&](int m, auto&& part_of, auto&& emit) {
        for (int i = 0; i < HP; ++i)
          for (int e = threadIdx.x * 4; e < nq * D; e += kAttendThreads * 4) {
            float t = -INFINITY, sum = 0, x[4] = {0, 0, 0, 0};
            for (int k0 = 0; k0 < m; k0 += 8) {
              float2 ml[8];
              float4 v[8];
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                ml[k] = make_float2(-INFINITY, 0);
                v[k] = make_float4(0, 0, 0, 0);
                if (k0 + k < m) {
                  const float* pk = part_of(k0 + k) + i * S::kHeadFloats;
                  ml[k] = __ldcg(reinterpret_cast<const float2*>(pk) + e / D);
                  v[k] = __ldcg(
                      reinterpret_cast<const float4*>(pk + 2 * Q + e));
                }
              }
              float top = t;
#pragma unroll
              for (int k = 0; k < 8; ++k) top = fmaxf(top, ml[k].x);
              const float t0 = top == -INFINITY ? 0.f : top;
              const float kept = sum * ex2(t - t0);
              sum = kept;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                ml[k].y *= ex2(ml[k].x - t0);
                sum += ml[k].y;
              }
              const float share_of = sum == 0 ? 0.f : __fdividef(1.f, sum);
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] *= kept * share_of;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float f = ml[k].y * share_of;
                x[0] += v[k].x * f;
                x[1] += v[k].y * f;
                x[2] += v[k].z * f;
                x[3] += v[k].w * f;
              }
              t = top;
            }
            emit(i, e, t, sum, x);
          }
      };
      auto finish = [&](int i, int e, float t, float sum, const float* x) {
        const int qi = e / D, d = e % D;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (d + k < dim) put(i, qi, d + k, sum == 0 ? 0.f : x[k]);
        if (d == 0) put_lse(i, qi, t, sum);
      };
      const int64_t p0 = 2 * c0 + (line_div(c0 * total, blocks) < item_at ? 1 : 0);
      auto block_part = [&](int k) -> const float* {
        const int c = from + k;
        return g.parts + (c == 0 ? p0 : 2 * (c0 + c)) * S::kPartFloats;
      };
      // Runs of a head that has several hold 8 parts or more, so that their
      // first blocks lie 7 or more apart (neighbouring heads share a block).
      auto run_slot = [&](int r) {
        return (int(c0) + r * n / runs) / (kAttendRun / 2 - 1);
      };
      auto run_part = [&](int r) {
        return g.runs + run_slot(r) * int64_t(S::kPartFloats);
      };
      if (runs == 1) {
        if (last_of(g.counters + c0, n)) join(n, block_part, finish);
      } else if (last_of(g.run_counters + run_slot(run), size)) {
        join(size, block_part,
             [&](int i, int e, float t, float sum, const float* x) {
               float* to = run_part(run) + i * S::kHeadFloats;
               *reinterpret_cast<float4*>(to + 2 * Q + e) =
                   make_float4(x[0], x[1], x[2], x[3]);
               if (e % D == 0) {
                 to[2 * (e / D)] = t;
                 to[2 * (e / D) + 1] = sum;
               }
             });
        __syncthreads();
        if (last_of(g.counters + c0, runs))
          join(runs, [&](int r) -> const float* { return run_part(r); },
               finish);
      }
    }
    __syncthreads();
  }
  cp_wait<0>();
}

// --- launch --------------------------------------------------------------------

inline int attend_dim(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// Queries a block holds at once: 8 when a key head has no more, else 16; a
// larger group reads its keys again per 16.  Codes of 256 elements: always 8,
// with steps of 16 keys and two blocks an SM, as shared memory then allows (32
// sequences of up to 8192 tokens, 4 key heads: 113 us for 8 queries each in
// e4m3, 233 for 16 in int8; 159 and 273 with steps of 32 keys, 16 queries at
// once and one block).
inline int attend_tiles(bool codes, int dim, int group) {
  return group <= 8 || (codes && attend_dim(dim) == 256) ? 1 : 2;
}

// The workspace: a counter per block and one per run of parts, as many as the
// largest grid has whatever the kernel (so that one buffer serves them all),
// then two parts of `floats` per block and one per run.
constexpr int kAttendBlocks = 3;      // blocks an SM at most
struct AttendSpace {
  int64_t run_counters, parts, runs, bytes;
};
inline AttendSpace attend_space(int64_t sms, int64_t blocks, int64_t floats) {
  auto runs_of = [](int64_t n) { return n / (kAttendRun / 2 - 1) + 1; };
  const int64_t most = sms * kAttendBlocks;
  AttendSpace s;
  s.run_counters = most * 4;
  s.parts = (s.run_counters + runs_of(most) * 4 + 255) / 256 * 256;
  s.runs = s.parts + 2 * blocks * floats * 4;
  s.bytes = s.runs + runs_of(blocks) * floats * 4;
  return s;
}

template <int KIND, int D, int NT, int HP>
int launch_attend(const KvAttendArgs& a, cudaStream_t st) {
  using S = AttendShape<KIND, D, NT, HP>;
  int sms = 0, dev = 0;
  const int rc = kv_device(&dev, &sms);
  if (rc != LM_OK) return rc;
  auto* kernel = lm_kv_attend_kernel<KIND, D, NT, HP>;
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
  const int blocks = sms * S::kBlocks;
  AttendGrid g;
  g.groups = (a.group + S::Q - 1) / S::Q;
  g.items = int(a.c.heads) / HP * g.groups;
  g.shared_page = a.c.page_tokens % S::KW == 0;
  g.q_pairs = reinterpret_cast<uintptr_t>(a.q.p) % 4 == 0 &&
              a.q.ts % 2 == 0 && a.q.hs % 2 == 0;
  char* const ws = static_cast<char*>(a.ws);
  static_assert(S::kBlocks <= kAttendBlocks, "the counters suffice");
  const AttendSpace at = attend_space(sms, blocks, S::kPartFloats);
  g.counters = reinterpret_cast<unsigned int*>(ws);
  g.run_counters = reinterpret_cast<unsigned int*>(ws + at.run_counters);
  g.parts = reinterpret_cast<float*>(ws + at.parts);
  g.runs = reinterpret_cast<float*>(ws + at.runs);
  return launch(kernel, blocks, kAttendThreads, S::kSmem, st, a, g);
}

template <int KIND, int D>
int launch_attend_dim(const KvAttendArgs& a, cudaStream_t st) {
  constexpr bool kCodes = KIND == KIND_E4M3 || KIND == KIND_INT8;
  const bool few = attend_tiles(kCodes, D, a.group) == 1;
  if constexpr (kCodes && D == 256) return launch_attend<KIND, D, 1, 1>(a, st);
  if constexpr (kCodes && D <= 128) {
    // Rows that are no whole 128-byte lines, heads side by side: lines that
    // two heads share come in once when one block takes both (3 x 131072
    // tokens of 4 x 64 int8, 145 MB: 220 MB read in 55 us a head at a time,
    // 146 MB in 52 us in pairs).
    if (a.c.dim % 128 != 0 && a.c.heads % 2 == 0 &&
        a.c.head_b < a.c.token_b)
      return few ? launch_attend<KIND, D, 1, 2>(a, st)
                 : launch_attend<KIND, D, 2, 2>(a, st);
  }
  if constexpr (!(kCodes && D == 256))
    return few ? launch_attend<KIND, D, 1, 1>(a, st)
               : launch_attend<KIND, D, 2, 1>(a, st);
}

template <int KIND>
int launch_attend_kind(const KvAttendArgs& a, cudaStream_t st) {
  const int d = attend_dim(a.c.dim);
  return d == 64    ? launch_attend_dim<KIND, 64>(a, st)
         : d == 128 ? launch_attend_dim<KIND, 128>(a, st)
                    : launch_attend_dim<KIND, 256>(a, st);
}

int launch_attend_bf16(const KvAttendArgs& a, cudaStream_t st);
int launch_attend_f16(const KvAttendArgs& a, cudaStream_t st);
int launch_attend_e4m3(const KvAttendArgs& a, cudaStream_t st);
int launch_attend_int8(const KvAttendArgs& a, cudaStream_t st);

}  // namespace lm
