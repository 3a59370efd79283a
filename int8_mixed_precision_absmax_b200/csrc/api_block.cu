// api_block.cu -- the extern "C" entry points of the 4-bit weights and the block norms (declared
// in include/int8mm.h): argument checks and launches.  Nothing here allocates or synchronizes.
#include <atomic>
#include <cmath>
#include <cstdint>

#include "block.cuh"
#include "kernels.cuh"

using namespace i8mm;

namespace {

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

int on_sm100() {
  static std::atomic<int> known{-1};  // the last device found to be one
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return INT8MM_ERR_CUDA;
  if (known.load(std::memory_order_relaxed) == dev) return INT8MM_OK;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return INT8MM_ERR_CUDA;
  if (major != 10 || minor != 0) return INT8MM_ERR_DEVICE;
  known.store(dev, std::memory_order_relaxed);
  return INT8MM_OK;
}

int launched(cudaError_t e) {
  if (e == cudaSuccess) return INT8MM_OK;
  (void)cudaGetLastError();  // reported here, not by the caller's next CUDA call
  return INT8MM_ERR_CUDA;
}

int check_int4(int N, int K, int group, unsigned flags) {
  if (flags & ~INT8MM_BFLOAT16) return INT8MM_ERR_FLAGS;
  if (N <= 0 || N > INT8MM_MAX_ROWS || K <= 0 || K > INT8MM_MAX_K) return INT8MM_ERR_SHAPE;
  if (K % 32 != 0) return INT8MM_ERR_ALIGN;
  if (group <= 0 || (group != 32 && group != 64 && group % 128 != 0)) return INT8MM_ERR_GROUP;
  return INT8MM_OK;
}

Int4Weight weight_of(const uint8_t* codes, const void* scales, const uint8_t* zeros, int N, int K,
                     int group, unsigned flags) {
  Int4Weight w;
  w.codes = codes;
  w.scales = scales;
  w.zeros = zeros;
  w.N = N;
  w.K = K;
  w.group = group < K ? group : (K + 127) / 128 * 128;  // one group: its length does not matter
  w.groups = int4_groups(K, w.group);
  w.bf16 = (flags & INT8MM_BFLOAT16) != 0;
  return w;
}

int check_norm(int M, int D, float eps, unsigned flags, unsigned allowed) {
  if (flags & ~allowed) return INT8MM_ERR_FLAGS;
  if (M <= 0 || M > INT8MM_MAX_ROWS || D <= 0 || D > INT8MM_MAX_K) return INT8MM_ERR_SHAPE;
  if (D % 16 != 0) return INT8MM_ERR_ALIGN;
  if (!(eps >= 0.0f) || std::isinf(eps)) return INT8MM_ERR_VALUE;
  return INT8MM_OK;
}

}  // namespace

extern "C" {

int int4_quant_weight(const void* W, int N, int K, int group, unsigned flags, uint8_t* codes,
                      void* scales, uint8_t* zeros, int8mm_stream_t stream) {
  if (!W || !codes || !scales) return INT8MM_ERR_NULL;
  int rc = check_int4(N, K, group, flags);
  if (rc) return rc;
  if (off16(W) || off16(codes) || off16(scales) || off16(zeros)) return INT8MM_ERR_ALIGN;
  if ((rc = on_sm100())) return rc;
  const Int4Weight w = weight_of(codes, scales, zeros, N, K, group, flags);
  return launched(launch_int4_quant(W, N, K, w.group, w.bf16, codes, scales, zeros,
                                    device_sm_count(), reinterpret_cast<cudaStream_t>(stream)));
}

int int4_dequant_weight(const uint8_t* codes, const void* scales, const uint8_t* zeros, int N,
                        int K, int group, unsigned flags, void* W_hat, int8mm_stream_t stream) {
  if (!codes || !scales || !W_hat) return INT8MM_ERR_NULL;
  int rc = check_int4(N, K, group, flags);
  if (rc) return rc;
  if (off16(W_hat) || off16(codes) || off16(scales) || off16(zeros)) return INT8MM_ERR_ALIGN;
  if ((rc = on_sm100())) return rc;
  return launched(launch_int4_dequant(weight_of(codes, scales, zeros, N, K, group, flags), W_hat,
                                      device_sm_count(), reinterpret_cast<cudaStream_t>(stream)));
}

int int4_linear_forward(const void* X, int M, int K, const uint8_t* codes, const void* scales,
                        const uint8_t* zeros, const void* bias, int N, int group, unsigned flags,
                        void* Y, int32_t* dev_status, int8mm_stream_t stream) {
  if (!X || !codes || !scales || !Y) return INT8MM_ERR_NULL;
  int rc = check_int4(N, K, group, flags);
  if (rc) return rc;
  if (M <= 0 || M > INT8MM_MAX_ROWS) return INT8MM_ERR_SHAPE;
  if (off16(X) || off16(codes) || off16(scales) || off16(zeros) || off16(bias) || off16(Y) ||
      (reinterpret_cast<uintptr_t>(dev_status) & 3u))
    return INT8MM_ERR_ALIGN;
  if ((rc = on_sm100())) return rc;
  Int4LinearArgs a;
  a.w = weight_of(codes, scales, zeros, N, K, group, flags);
  a.X = X;
  a.bias = bias;
  a.Y = Y;
  a.M = M;
  a.status = dev_status;
  return launched(
      launch_int4_linear(a, device_sm_count(), reinterpret_cast<cudaStream_t>(stream)));
}

int int8_block_norm(const void* x, int M, int D, const void* weight, const void* bias, float eps,
                    unsigned flags, void* h, int8mm_stream_t stream) {
  if (!x || !h) return INT8MM_ERR_NULL;
  int rc = check_norm(M, D, eps, flags,
                      INT8MM_BFLOAT16 | INT8MM_LAYER_NORM | INT8MM_F32_RESIDUAL);
  if (rc) return rc;
  if (off16(x) || off16(weight) || off16(bias) || off16(h)) return INT8MM_ERR_ALIGN;
  if ((rc = on_sm100())) return rc;
  BlockNormArgs a = {};
  a.x = x;
  a.next_w = weight;
  a.next_b = bias;
  a.h = h;
  a.M = M;
  a.D = D;
  a.x_scale = 1.0f;
  a.eps = eps;
  a.bf16 = (flags & INT8MM_BFLOAT16) != 0;
  a.layer_norm = (flags & INT8MM_LAYER_NORM) != 0;
  a.f32_residual = (flags & INT8MM_F32_RESIDUAL) != 0;
  return launched(launch_block_norm(a, device_sm_count(), reinterpret_cast<cudaStream_t>(stream)));
}

int int8_block_residual(const void* f, const void* x, int M, int D, const void* post_weight,
                        const void* post_bias, const void* gate, int gate_rows, float x_scale,
                        float f_scale, const void* next_weight, const void* next_bias, float eps,
                        unsigned flags, void* y, void* h, int8mm_stream_t stream) {
  if (!f || !x || (!y && !h)) return INT8MM_ERR_NULL;
  int rc = check_norm(
      M, D, eps, flags,
      INT8MM_BFLOAT16 | INT8MM_LAYER_NORM | INT8MM_F32_RESIDUAL | INT8MM_POST_NORM);
  if (rc) return rc;
  if (!(flags & INT8MM_POST_NORM) && (post_weight || post_bias)) return INT8MM_ERR_FLAGS;
  if (!h && (next_weight || next_bias)) return INT8MM_ERR_NULL;
  if (gate ? (gate_rows <= 0 || gate_rows > M || M % gate_rows != 0) : gate_rows != 0)
    return INT8MM_ERR_SHAPE;
  if (!std::isfinite(x_scale) || !std::isfinite(f_scale)) return INT8MM_ERR_VALUE;
  if (off16(f) || off16(x) || off16(post_weight) || off16(post_bias) || off16(gate) ||
      off16(next_weight) || off16(next_bias) || off16(y) || off16(h))
    return INT8MM_ERR_ALIGN;
  if ((rc = on_sm100())) return rc;
  BlockNormArgs a;
  a.f = f;
  a.x = x;
  a.post_w = post_weight;
  a.post_b = post_bias;
  a.gate = gate;
  a.next_w = next_weight;
  a.next_b = next_bias;
  a.y = y;
  a.h = h;
  a.M = M;
  a.D = D;
  a.rows_per_gate = gate ? M / gate_rows : 1;
  a.x_scale = x_scale;
  a.f_scale = f_scale;
  a.eps = eps;
  a.bf16 = (flags & INT8MM_BFLOAT16) != 0;
  a.layer_norm = (flags & INT8MM_LAYER_NORM) != 0;
  a.f32_residual = (flags & INT8MM_F32_RESIDUAL) != 0;
  a.post_norm = (flags & INT8MM_POST_NORM) != 0;
  return launched(launch_block_norm(a, device_sm_count(), reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
