// int4.cu -- 4-bit weights with group scales: the quantizer, its inverse, and which kernel multiplies.
#include "block.cuh"

namespace i8mm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The maximum over the `width` lanes of a warp segment (a power of two up to 32).
__device__ __forceinline__ float seg_max(float v, int width) {
  for (int o = width / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
  return v;
}

// The largest w and -w of 8 neighbours (at least 0), and whether any is NaN or infinite.
template <typename T>
__device__ __forceinline__ void extremes8(const uint4& v, float& hi, float& nlo, bool& bad) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<T>(r[i]);
    hi = fmaxf(hi, fmaxf(p.x, p.y));
    nlo = fmaxf(nlo, fmaxf(-p.x, -p.y));
    bad |= !(fabsf(p.x) <= 3.4028235e38f) || !(fabsf(p.y) <= 3.4028235e38f);
  }
}

// Scale and zero point of a group from its extremes (hi = max(w, 0), nlo = max(-w, 0)).
template <typename T>
__device__ __forceinline__ void group_params(float hi, float nlo, bool bad, bool affine, T& s,
                                             float& z) {
  if (bad) {
    s = from_f32<T>(__int_as_float(0x7FC00000));
    z = kInt4Zero;
    return;
  }
  if (!affine) {
    s = from_f32<T>(__fdiv_rn(fmaxf(hi, nlo), 7.0f));
    z = kInt4Zero;
    return;
  }
  s = from_f32<T>(__fadd_rn(__fdiv_rn(hi, 15.0f), __fdiv_rn(nlo, 15.0f)));
  const float sf = to_f32(s);
  z = sf > 0.0f ? fminf(rintf(__fdiv_rn(nlo, sf)), 15.0f) : 0.0f;
}

template <typename T>
__device__ __forceinline__ uint32_t encode8(const uint4& v, float s, float z, bool affine) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
  const float lo = affine ? 0.0f : 1.0f;
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 p = unpack2<T>(r[j / 2]);
    const float w = (j & 1) ? p.y : p.x;
    float u = z;
    if (s > 0.0f) u = fminf(fmaxf(__fadd_rn(rintf(__fdiv_rn(w, s)), z), lo), 15.0f);
    word |= static_cast<uint32_t>(u) << (4 * int4_nibble(j));
  }
  return word;
}

}  // namespace

// One warp per span of `span` columns of a row (256, or the whole group where a group is longer
// or no power of two); a group of up to 256 columns is a segment of span lanes.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    int4_quant_kernel(const T* __restrict__ W, int N, int K, int group, int groups, int span,
                      uint8_t* __restrict__ codes, T* __restrict__ scales,
                      uint8_t* __restrict__ zeros) {
  const int lane = threadIdx.x & 31;
  const int spans = (K + span - 1) / span;
  const long long total = static_cast<long long>(N) * spans;
  const int width = group <= 256 ? group / 8 : 32;  // lanes of a group
  const bool affine = zeros != nullptr;
  for (long long i = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32; i < total;
       i += static_cast<long long>(gridDim.x) * kWarps) {
    const long long n = i / spans;
    const int k0 = static_cast<int>(i % spans) * span;
    const int k1 = min(K, k0 + span);
    const uint4* row = reinterpret_cast<const uint4*>(W + n * K);
    float hi = 0.0f, nlo = 0.0f;
    bool bad = false;
    for (int k = k0 + lane * 8; k < k1; k += 256) extremes8<T>(row[k / 8], hi, nlo, bad);
    hi = seg_max(hi, width);
    nlo = seg_max(nlo, width);
    bad = seg_max(bad ? 1.0f : 0.0f, width) > 0.0f;
    T s;
    float z;
    group_params<T>(hi, nlo, bad, affine, s, z);
    const float sf = to_f32(s);
    const int k = k0 + lane * 8;
    if (k < k1 && lane % width == 0) {
      scales[n * groups + k / group] = s;
      if (affine) zeros[n * groups + k / group] = static_cast<uint8_t>(z);
    }
    uint32_t* out = reinterpret_cast<uint32_t*>(codes + n * (K / 2));
    for (int c = k; c < k1; c += 256) out[c / 8] = encode8<T>(row[c / 8], sf, z, affine);
  }
}

// One thread per word.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    int4_dequant_kernel(const uint32_t* __restrict__ codes, const T* __restrict__ scales,
                        const uint8_t* __restrict__ zeros, int N, int K, int group, int groups,
                        uint4* __restrict__ W_hat) {
  const int words = K / 8;
  const long long total = static_cast<long long>(N) * words;
  for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * kThreads) {
    const long long n = i / words;
    const int k = static_cast<int>(i % words) * 8;
    const long long c = n * groups + k / group;
    const float s = to_f32(scales[c]);
    const float z = zeros ? static_cast<float>(zeros[c]) : static_cast<float>(kInt4Zero);
    const uint32_t w = codes[i];
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = static_cast<float>((w >> (4 * j)) & 15u) - z;
      const float b = static_cast<float>((w >> (4 * j + 16)) & 15u) - z;
      r[j] = pack2<T>(a * s, b * s);
    }
    W_hat[i] = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

namespace {

int blocks_for(long long work, int per_block, int num_sms) {
  const long long want = (work + per_block - 1) / per_block;
  const long long most = static_cast<long long>(num_sms) * 8;
  return static_cast<int>(want < most ? want : most);
}

}  // namespace

cudaError_t launch_int4_quant(const void* W, int N, int K, int group, bool bf16, uint8_t* codes,
                              void* scales, uint8_t* zeros, int num_sms, cudaStream_t stream) {
  const int groups = int4_groups(K, group);
  const int span = (group == 32 || group == 64 || group == 128 || group == 256) ? 256 : group;
  const long long total = static_cast<long long>(N) * ((K + span - 1) / span);
  const int grid = blocks_for(total, kWarps, num_sms);
  if (bf16)
    int4_quant_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(W), N, K, group, groups, span, codes,
        static_cast<__nv_bfloat16*>(scales), zeros);
  else
    int4_quant_kernel<__half><<<grid, kThreads, 0, stream>>>(static_cast<const __half*>(W), N, K,
                                                             group, groups, span, codes,
                                                             static_cast<__half*>(scales), zeros);
  return cudaGetLastError();
}

cudaError_t launch_int4_dequant(const Int4Weight& w, void* W_hat, int num_sms,
                                cudaStream_t stream) {
  const int grid = blocks_for(static_cast<long long>(w.N) * (w.K / 8), kThreads, num_sms);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(w.codes);
  uint4* out = static_cast<uint4*>(W_hat);
  if (w.bf16)
    int4_dequant_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(
        codes, static_cast<const __nv_bfloat16*>(w.scales), w.zeros, w.N, w.K, w.group, w.groups,
        out);
  else
    int4_dequant_kernel<__half><<<grid, kThreads, 0, stream>>>(
        codes, static_cast<const __half*>(w.scales), w.zeros, w.N, w.K, w.group, w.groups, out);
  return cudaGetLastError();
}

cudaError_t launch_int4_linear(const Int4LinearArgs& a, int num_sms, cudaStream_t stream) {
  return int4_stream_fits(a.M, a.w.K, a.w.group) ? launch_int4_stream(a, num_sms, stream)
                                      : launch_int4_tile(a, num_sms, stream);
}

}  // namespace i8mm
