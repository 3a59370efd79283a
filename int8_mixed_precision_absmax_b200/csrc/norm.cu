// norm.cu -- the row passes around a block: norm, and output norm + gate + residual + next norm.
#include "block.cuh"

namespace i8mm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float block_sum(float v, float* red) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();  // red may still be read from the sum before
  if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) v += red[i];
  return v;
}

}  // namespace

// One block per row; the row is read again for each step.
template <typename T, typename R>
__global__ void __launch_bounds__(kThreads) block_norm_kernel(const BlockNormArgs a) {
  __shared__ float red[kWarps];
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const T *pw = static_cast<const T*>(a.post_w), *pb = static_cast<const T*>(a.post_b);
  const T *nw = static_cast<const T*>(a.next_w), *nb = static_cast<const T*>(a.next_b);
  for (long long m = blockIdx.x; m < a.M; m += gridDim.x) {
    const T* f = a.f ? static_cast<const T*>(a.f) + m * a.D : nullptr;
    const R* x = static_cast<const R*>(a.x) + m * a.D;
    const T* gate = a.gate ? static_cast<const T*>(a.gate) + m / (a.M / a.gate_rows) * a.D : nullptr;
    R* y = a.y ? static_cast<R*>(a.y) + m * a.D : nullptr;
    T* h = a.h ? static_cast<T*>(a.h) + m * a.D : nullptr;
    float fm = 0.0f, fr = 1.0f;  // the output norm's mean and reciprocal deviation
    if (a.post_norm) {
      if (a.layer_norm) {
        float s = 0.0f;
        for (int j = threadIdx.x; j < a.D; j += kThreads) s += to_f32(f[j]);
        fm = block_sum(s, red) * inv_d;
      }
      float q = 0.0f;
      for (int j = threadIdx.x; j < a.D; j += kThreads) {
        const float d = to_f32(f[j]) - fm;
        q = fmaf(d, d, q);
      }
      fr = 1.0f / sqrtf(block_sum(q, red) * inv_d + a.eps);
    }
    // the residual sum's element j, rounded as it is stored
    auto value = [&](int j) {
      const float xv = to_f32(x[j]);
      if (!f) return xv;
      float p = (to_f32(f[j]) - fm) * fr;
      if (pw) p *= to_f32(pw[j]);
      if (pb) p += to_f32(pb[j]);
      if (gate) p *= to_f32(gate[j]);
      return to_f32(from_f32<R>(fmaf(a.f_scale, p, a.x_scale * xv)));
    };
    float ym = 0.0f, yr = 1.0f;
    if (h) {
      if (a.layer_norm) {
        float s = 0.0f;
        for (int j = threadIdx.x; j < a.D; j += kThreads) s += value(j);
        ym = block_sum(s, red) * inv_d;
      }
      float q = 0.0f;
      for (int j = threadIdx.x; j < a.D; j += kThreads) {
        const float d = value(j) - ym;
        q = fmaf(d, d, q);
      }
      yr = 1.0f / sqrtf(block_sum(q, red) * inv_d + a.eps);
    }
    for (int j = threadIdx.x; j < a.D; j += kThreads) {
      const float v = value(j);
      if (y) y[j] = from_f32<R>(v);
      if (h) {
        float n = (v - ym) * yr;
        if (nw) n *= to_f32(nw[j]);
        if (nb) n += to_f32(nb[j]);
        h[j] = from_f32<T>(n);
      }
    }
  }
}

cudaError_t launch_block_norm(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
  const int grid = a.M < num_sms * 8 ? a.M : num_sms * 8;
  if (a.bf16 && a.f32_residual)
    block_norm_kernel<__nv_bfloat16, float><<<grid, kThreads, 0, stream>>>(a);
  else if (a.bf16)
    block_norm_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kThreads, 0, stream>>>(a);
  else if (a.f32_residual)
    block_norm_kernel<__half, float><<<grid, kThreads, 0, stream>>>(a);
  else
    block_norm_kernel<__half, __half><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace i8mm
