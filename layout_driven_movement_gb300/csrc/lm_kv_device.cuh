// Device helpers of the key-value cache's kernels: element conversions,
// aligned packs and the lookup of a position's row in the rotary table.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "lm_kv.h"

namespace lm {

typedef __nv_bfloat16 bf16;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) {
  return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) {
  return __float2half_rn(x);
}

// V elements moved as one access (V * sizeof(T) bytes, aligned to that).
template <class T, int V>
struct alignas(sizeof(T) * V) Pack {
  T v[V];
};

// The elements of a word: two of 16 bits (the first in the low half), or one.
// Pairs convert in one or two instructions; element by element a 16-bit
// element takes a register and its moves.
template <class T>
struct Word;
template <>
struct Word<float> {
  static constexpr int N = 1;
  static __device__ __forceinline__ void get(uint32_t w, float* x) {
    x[0] = __uint_as_float(w);
  }
  static __device__ __forceinline__ uint32_t put(const float* x) {
    return __float_as_uint(x[0]);
  }
};
template <>
struct Word<bf16> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void get(uint32_t w, float* x) {
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ uint32_t put(const float* x) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x[0], x[1]);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct Word<__half> {
  static constexpr int N = 2;
  static __device__ __forceinline__ void get(uint32_t w, float* x) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    x[0] = f.x;
    x[1] = f.y;
  }
  static __device__ __forceinline__ uint32_t put(const float* x) {
    const __half2 v = __floats2half2_rn(x[0], x[1]);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// N words, moved as one access.
template <int N>
struct alignas(4 * N) Words {
  uint32_t w[N];
};
template <class T, int N>
__device__ __forceinline__ void get_words(const uint32_t* w, float* x) {
#pragma unroll
  for (int i = 0; i < N; ++i) Word<T>::get(w[i], x + i * Word<T>::N);
}
template <class T, int N>
__device__ __forceinline__ void put_words(const float* x, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < N; ++i) w[i] = Word<T>::put(x + i * Word<T>::N);
}

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

// Row `position` of the rotary table, or nullptr (and the status bit) when
// the position lies outside it.
__device__ __forceinline__ const float* turn_row(const Turn& t, uint32_t token,
                                                 unsigned int* status) {
  const int64_t p = t.pos64
                        ? static_cast<const int64_t*>(t.pos)[token]
                        : int64_t(static_cast<const int32_t*>(t.pos)[token]);
  if (p < 0 || p >= t.rows) {
    if (status) atomicOr(status, kStatusRange);
    return nullptr;
  }
  return t.table + p * t.rot;
}

// a*c - b*s and its partner, each product and the sum rounded on its own, so
// that the result does not depend on which of them a compiler fuses.
__device__ __forceinline__ float turn_lo(float a, float b, float c, float s) {
  return __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
}
__device__ __forceinline__ float turn_hi(float a, float b, float c, float s) {
  return __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// First in every kernel of this section, before it touches global memory: the
// next kernel on the stream may take the room that this one leaves, and this
// one goes on when all before it are done and their writes visible.
__device__ __forceinline__ void stream_order() {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

// Launches a kernel that begins with stream_order(): its launch overlaps the
// end of the kernel before it.
// In clusters of `cluster` blocks, which `grid` is a multiple of.
template <class... P, class... A>
int launch_clusters(void (*kernel)(P...), int cluster, uint64_t grid, int block,
                    int smem, cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(unsigned(block));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e == cudaSuccess) return LM_OK;
  cudaGetLastError();                      // not left for a later call
  set_cuda_error(int(e));
  return LM_E_CUDA;
}

template <class... P, class... A>
int launch(void (*kernel)(P...), uint64_t grid, int block, int smem,
           cudaStream_t st, const A&... args) {
  return launch_clusters(kernel, 1, grid, block, smem, st, args...);
}

}  // namespace lm
