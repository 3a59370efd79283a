// block.cuh -- internal interface of the 4-bit weights (int4.cu) and the block norms (norm.cu):
// what their entry points (api_block.cu) hand to the kernels' launches.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "int8mm.h"
#include "ptx.cuh"

namespace i8mm {

// ---------------------------------------------------------------- 16-bit types

template <typename T>
struct Half2Of;
template <>
struct Half2Of<__half> {
  using type = __half2;
};
template <>
struct Half2Of<__nv_bfloat16> {
  using type = __nv_bfloat162;
};

__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Two neighbours in one 32-bit word, low half first.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------- waits
//
// mbar_wait_bounded (ptx.cuh) for a role that waits long and has time: it sleeps between its polls,
// which otherwise take issue slots from the warps it waits for.
__device__ __forceinline__ bool wait_asleep(uint64_t* bar, uint32_t parity, volatile int* abort,
                                            uint32_t ns) {
#pragma unroll 1
  for (int i = 0; i < 20000; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    __nanosleep(ns);
  }
  return mbar_wait_bounded(bar, parity, abort);
}

// ---------------------------------------------------------------- ahead of a wait

// The box of a 2-D tiled load, brought as far as L2: no value of it reaches the SM.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int32_t x, int32_t y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}

// ---------------------------------------------------------------- 4-bit weights
//
// Of the 8 neighbours k = 8j .. 8j+7 in a 32-bit word, nibble i (from the low end) holds
// k = 8j + 0, 2, 4, 6, 1, 3, 5, 7.  One AND with 0x000F000F (of the word shifted
// right by 0, 4, 8, 12) leaves the neighbours (0,1), (2,3), (4,5), (6,7) in the two halves of a
// register, the order in which a 16-byte load of X holds their factors.
// The nibble that holds neighbour j of its word.
__host__ __device__ constexpr int int4_nibble(int j) { return (j & 1) * 4 + (j >> 1); }

constexpr int kInt4Zero = 8;  // the zero point where none is given

// (w & mask) | ones in one instruction: left to itself the compiler spends two and more on it.
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t mask, uint32_t ones) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(ones));
  return r;
}

// W_hat of 4-bit words: the group's constants, and 8 values of a word.  A nibble set into the low
// mantissa bits of 1024 (fp16) or 128 (bf16) reads as that number plus the code (Kim, Henry, Fahim and
// Awadalla, "Who Says Elephants Can't Run", 2022, for fp16).  LOP3: masks and
// sets a nibble by the one instruction; the tensor-core kernel, bound by its instructions, gains
// by it (107 us against 119 for 16 tokens of 12288 x 49152), the inverse quantizer, bound by
// memory, does better with what the compiler chooses (273 us against 299 for the same weights).
template <bool LOP3>
__device__ __forceinline__ uint32_t nibbles(uint32_t w, uint32_t mask, uint32_t base) {
  return LOP3 ? and_or(w, mask, base) : ((w & mask) | base);
}
template <typename T>
struct Int4Values;
template <>
struct Int4Values<__half> {
  uint32_t s, z0, z1;
  // the scale in both halves, and the zero point (below 64)
  __device__ __forceinline__ void set(uint32_t s2, uint32_t z) {
    s = s2;
    z0 = 0x64006400u + z * 0x00010001u;  // 1024 + z
    z1 = 0xD400D400u + z * 0x00100010u;  // -64 - z, of a code in bits 4..7: (1024 + 16 u) / 16
  }
  static __device__ __forceinline__ __half2 of(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
  // u - z, exact; word: times the scale, rounded
  template <bool LOP3>
  __device__ __forceinline__ void offsets(uint32_t w, uint32_t* out) const {
    constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u, k1024 = 0x64006400u;
    const uint32_t w8 = w >> 8;
    const uint32_t a[4] = {nibbles<LOP3>(w, kLow, k1024), nibbles<LOP3>(w, kHigh, k1024),
                           nibbles<LOP3>(w8, kLow, k1024), nibbles<LOP3>(w8, kHigh, k1024)};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 d = (i & 1) ? __hfma2(of(a[i]), __float2half2_rn(0.0625f), of(z1))
                                : __hsub2(of(a[i]), of(z0));
      out[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
  }
  template <bool LOP3>
  __device__ __forceinline__ void word(uint32_t w, uint32_t* out) const {
    offsets<LOP3>(w, out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __hmul2(of(out[i]), of(s));
      out[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};
template <>
struct Int4Values<__nv_bfloat16> {
  uint32_t s, z0;
  __device__ __forceinline__ void set(uint32_t s2, uint32_t z) {
    s = s2;
    z0 = 0x43004300u + z * 0x00010001u;  // 128 + z
  }
  static __device__ __forceinline__ __nv_bfloat162 of(uint32_t v) {
    return *reinterpret_cast<__nv_bfloat162*>(&v);
  }
  template <bool LOP3>
  __device__ __forceinline__ void offsets(uint32_t w, uint32_t* out) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 d =
          __hsub2(of(nibbles<LOP3>(w >> (4 * i), 0x000F000Fu, 0x43004300u)), of(z0));
      out[i] = *reinterpret_cast<const uint32_t*>(&d);
    }
  }
  template <bool LOP3>
  __device__ __forceinline__ void word(uint32_t w, uint32_t* out) const {
    offsets<LOP3>(w, out);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __hmul2(of(out[i]), of(s));
      out[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
};

struct Int4Weight {
  const uint8_t* codes;
  const void* scales;    // T [N, groups]
  const uint8_t* zeros;  // [N, groups] or null
  int N, K, group, groups;
  bool bf16;
};
inline int int4_groups(int K, int group) { return (K + group - 1) / group; }

struct Int4LinearArgs {
  Int4Weight w;
  const void* X;     // T [M, K]
  const void* bias;  // T [N] or null
  void* Y;           // T [M, N]
  int M;
  int32_t* status;   // nullable
};

cudaError_t launch_int4_quant(const void* W, int N, int K, int group, bool bf16, uint8_t* codes,
                              void* scales, uint8_t* zeros, int num_sms, cudaStream_t stream);
cudaError_t launch_int4_dequant(const Int4Weight& w, void* W_hat, int num_sms,
                                cudaStream_t stream);
cudaError_t launch_int4_linear(const Int4LinearArgs& a, int num_sms, cudaStream_t stream);
// few tokens (int4_stream.cu): up to 8 whose activations fit into shared memory, where it is faster
bool int4_stream_suits(int M, int N, int K, int group, int num_sms);
cudaError_t launch_int4_stream(const Int4LinearArgs& a, int num_sms, cudaStream_t stream);
// all others (int4_tile.cu): tcgen05
cudaError_t launch_int4_tile(const Int4LinearArgs& a, int num_sms, cudaStream_t stream);

// ---------------------------------------------------------------- launches

// Lets `kernel` use `bytes` of dynamic shared memory, once on each device (`done`: of this kernel, a bit
// for each device).
inline cudaError_t allow_smem(const void* kernel, size_t bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---------------------------------------------------------------- block norms

struct BlockNormArgs {
  const void* f;            // T [M, D], or null: the norm before a block alone
  const void* x;            // R [M, D]
  const void *post_w, *post_b, *gate, *next_w, *next_b;  // nullable
  void* y;                  // R [M, D] or null
  void* h;                  // T [M, D] or null
  int M, D;
  int rows_per_gate;        // rows that share a gate row
  float x_scale, f_scale, eps;
  bool bf16, layer_norm, f32_residual, post_norm;
};
cudaError_t launch_block_norm(const BlockNormArgs& a, int num_sms, cudaStream_t stream);

}  // namespace i8mm
