// norm.cu -- the row passes around a block of layers.
//
//   before:  h = norm(x; w, b)
//   after:   y = x_scale x + f_scale gate norm(f; w, b),  h = norm(y; w', b')
//   norm(v; w, b) = (v - mean) / sqrt(mean((v - mean)^2) + eps) w + b   (mean 0 for the RMS norm)
//
// One pass over memory: a row lives in the registers of its threads between its loads and its
// stores, both norms' sums are taken there (deviations about the mean, not differences of squares),
// and h is made of y as it was rounded for storing.  What bounds it is the bytes of f, x, y and h; the
// weights and gates stay in cache.  With many rows a thread takes 2 pieces of 8 elements (blocks
// small enough that an SM has several rows in flight); with few rows 1, for latency.
#include "block.cuh"
#include "ptx.cuh"

namespace i8mm {

namespace {

constexpr int kMaxRowThreads = 512, kMaxPieces = 4;  // rows of up to 16384 elements in registers
constexpr int kLongThreads = 1024;

// 8 neighbours.
template <typename V>
struct Piece {
  uint4 q[sizeof(V) / 2];
};
template <typename V>
__device__ __forceinline__ Piece<V> load8(const V* p) {
  Piece<V> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(V)) / 2; ++i) r.q[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename V>
__device__ __forceinline__ void floats8(const Piece<V>& r, float (&v)[8]) {
  if constexpr (sizeof(V) == 4) {
    const uint32_t w[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = unpack2<V>(w[i]);
      v[2 * i] = p.x;
      v[2 * i + 1] = p.y;
    }
  }
}
// Stores 8 neighbours and leaves in v what was stored.
template <typename V>
__device__ __forceinline__ void round8(Piece<V>& r, float (&v)[8]) {
  if constexpr (sizeof(V) == 4) {
    r.q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    r.q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    r.q[0] = make_uint4(pack2<V>(v[0], v[1]), pack2<V>(v[2], v[3]), pack2<V>(v[4], v[5]), pack2<V>(v[6], v[7]));
    floats8<V>(r, v);
  }
}
template <typename V>
__device__ __forceinline__ void store8(V* p, const Piece<V>& r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(V)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.q[i];
}

// v = v * s [+ b], elementwise over 8 neighbours; null pointers stand for ones and zeros.
template <typename T>
__device__ __forceinline__ void scale8(float (&v)[8], const T* w, const T* b) {
  float t[8];
  if (w) {
    floats8<T>(load8<T>(w), t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= t[i];
  }
  if (b) {
    floats8<T>(load8<T>(b), t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += t[i];
  }
}

__device__ __forceinline__ float warp_sum(float v) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

// The sum over a row's `warps` warps, in the same order for each of its threads.  red: a place of
// its own for each sum, so that one barrier is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int first_warp, int warps) {
  v = warp_sum(v);
  if (warps == 1) return v;  // the same for the whole block
  if ((threadIdx.x & 31) == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.0f;
  for (int i = 0; i < warps; ++i) v += red[first_warp + i];
  return v;
}

}  // namespace

// One row for every `width` threads (whole warps), NV pieces of 8 elements a thread.
template <typename T, typename R, int NV, bool AFTER>
__global__ void __launch_bounds__(kMaxRowThreads)
    block_norm_kernel(const BlockNormArgs a, int width) {
  __shared__ float red[4][kMaxRowThreads / 32];
  grid_launch_dependents();
  const int warps = width / 32, in_block = threadIdx.x / width, tid = threadIdx.x % width;
  const int first_warp = in_block * warps;
  const long long m = static_cast<long long>(blockIdx.x) * (blockDim.x / width) + in_block;
  const int pieces = a.D / 8;
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const bool row_ok = m < a.M;
  const long long at = (row_ok ? m : 0) * a.D;
  const T* f = static_cast<const T*>(a.f) + at;
  const R* x = static_cast<const R*>(a.x) + at;
  grid_dependency_wait();

  Piece<R> xp[NV];
  Piece<T> fp[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * width;
    if (row_ok && c < pieces) {
      if (AFTER) fp[i] = load8<T>(f + 8 * c);
      xp[i] = load8<R>(x + 8 * c);
    }
  }
  float v[NV][8];  // the residual sum, or x
  if constexpr (AFTER) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool ok = row_ok && tid + i * width < pieces;
      if (ok) floats8<T>(fp[i], v[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = ok ? v[i][e] : 0.0f;
    }
    if (a.post_norm) {
      float mean = 0.0f, s = 0.0f;
      if (a.layer_norm) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) s += v[i][e];
        }
        mean = row_sum(s, red[0], first_warp, warps) * inv_d;
        s = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool ok = tid + i * width < pieces;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[i][e] = ok ? v[i][e] - mean : 0.0f;
          s = fmaf(v[i][e], v[i][e], s);
        }
      }
      const float r = 1.0f / sqrtf(row_sum(s, red[1], first_warp, warps) * inv_d + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = tid + i * width;
        if (c < pieces) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] *= r;
          scale8<T>(v[i], a.post_w ? static_cast<const T*>(a.post_w) + 8 * c : nullptr,
                    a.post_b ? static_cast<const T*>(a.post_b) + 8 * c : nullptr);
        }
      }
    }
    const T* gate = a.gate ? static_cast<const T*>(a.gate) + (row_ok ? m : 0) / (a.M / a.gate_rows) * a.D
                           : nullptr;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * width;
      if (row_ok && c < pieces) {
        if (gate) scale8<T>(v[i], gate + 8 * c, nullptr);
        float xv[8];
        floats8<R>(xp[i], xv);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = fmaf(a.f_scale, v[i][e], a.x_scale * xv[e]);
        round8<R>(xp[i], v[i]);
        if (a.y) store8<R>(static_cast<R*>(a.y) + at + 8 * c, xp[i]);
      }
    }
    if (!a.h) return;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool ok = row_ok && tid + i * width < pieces;
      if (ok) floats8<R>(xp[i], v[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] = ok ? v[i][e] : 0.0f;
    }
  }
  float mean = 0.0f, s = 0.0f;
  if (a.layer_norm) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[i][e];
    }
    mean = row_sum(s, red[2], first_warp, warps) * inv_d;
    s = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool ok = tid + i * width < pieces;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[i][e] = ok ? v[i][e] - mean : 0.0f;
      s = fmaf(v[i][e], v[i][e], s);
    }
  }
  const float r = 1.0f / sqrtf(row_sum(s, red[3], first_warp, warps) * inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * width;
    if (row_ok && c < pieces) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[i][e] *= r;
      scale8<T>(v[i], a.next_w ? static_cast<const T*>(a.next_w) + 8 * c : nullptr,
                a.next_b ? static_cast<const T*>(a.next_b) + 8 * c : nullptr);
      Piece<T> out;
      round8<T>(out, v[i]);
      store8<T>(static_cast<T*>(a.h) + at + 8 * c, out);
    }
  }
}

// Longer rows: one block a row, which is read again (from L2) for each of the sums and written in
// the last pass, every element by the thread that read it.
template <typename T, typename R>
__global__ void __launch_bounds__(kLongThreads) block_norm_long_kernel(const BlockNormArgs a) {
  __shared__ float red[4][kLongThreads / 32];
  constexpr int kWarps = kLongThreads / 32;
  grid_launch_dependents();
  const long long m = blockIdx.x, at = m * a.D;
  const int pieces = a.D / 8;
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const T* f = a.f ? static_cast<const T*>(a.f) + at : nullptr;
  const R* x = static_cast<const R*>(a.x) + at;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + m / (a.M / a.gate_rows) * a.D : nullptr;
  grid_dependency_wait();

  float fm = 0.0f, fr = 1.0f;
  if (a.post_norm) {
    float s = 0.0f, v[8];
    if (a.layer_norm) {
      for (int c = threadIdx.x; c < pieces; c += kLongThreads) {
        floats8<T>(load8<T>(f + 8 * c), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];
      }
      fm = row_sum(s, red[0], 0, kWarps) * inv_d;
      s = 0.0f;
    }
    for (int c = threadIdx.x; c < pieces; c += kLongThreads) {
      floats8<T>(load8<T>(f + 8 * c), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[e] - fm, v[e] - fm, s);
    }
    fr = 1.0f / sqrtf(row_sum(s, red[1], 0, kWarps) * inv_d + a.eps);
  }
  // the residual sum's piece c, as it is stored
  auto value = [&](int c, float (&v)[8], Piece<R>& piece) {
    piece = load8<R>(x + 8 * c);
    if (!f) {
      floats8<R>(piece, v);
      return;
    }
    floats8<T>(load8<T>(f + 8 * c), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (v[e] - fm) * fr;
    scale8<T>(v, a.post_w ? static_cast<const T*>(a.post_w) + 8 * c : nullptr,
              a.post_b ? static_cast<const T*>(a.post_b) + 8 * c : nullptr);
    if (gate) scale8<T>(v, gate + 8 * c, nullptr);
    float xv[8];
    floats8<R>(piece, xv);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(a.f_scale, v[e], a.x_scale * xv[e]);
    round8<R>(piece, v);
  };
  float ym = 0.0f, yr = 1.0f, v[8];
  Piece<R> piece;
  if (a.h) {
    float s = 0.0f;
    if (a.layer_norm) {
      for (int c = threadIdx.x; c < pieces; c += kLongThreads) {
        value(c, v, piece);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];
      }
      ym = row_sum(s, red[2], 0, kWarps) * inv_d;
      s = 0.0f;
    }
    for (int c = threadIdx.x; c < pieces; c += kLongThreads) {
      value(c, v, piece);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[e] - ym, v[e] - ym, s);
    }
    yr = 1.0f / sqrtf(row_sum(s, red[3], 0, kWarps) * inv_d + a.eps);
  }
  for (int c = threadIdx.x; c < pieces; c += kLongThreads) {
    value(c, v, piece);
    if (a.y) store8<R>(static_cast<R*>(a.y) + at + 8 * c, piece);
    if (a.h) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (v[e] - ym) * yr;
      scale8<T>(v, a.next_w ? static_cast<const T*>(a.next_w) + 8 * c : nullptr,
                a.next_b ? static_cast<const T*>(a.next_b) + 8 * c : nullptr);
      Piece<T> out;
      round8<T>(out, v);
      store8<T>(static_cast<T*>(a.h) + at + 8 * c, out);
    }
  }
}

namespace {

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), long long grid, int threads, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, typename R, bool AFTER>
cudaError_t launch_rows(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
  const int pieces = a.D / 8;
  if (pieces > kMaxRowThreads * kMaxPieces)
    return launch(block_norm_long_kernel<T, R>, a.M, kLongThreads, stream, a);
  int nv = a.M >= num_sms * 4 ? 2 : 1;
  while ((pieces + nv - 1) / nv > kMaxRowThreads) nv *= 2;
  const int width = ((pieces + nv - 1) / nv + 31) / 32 * 32;
  const int rows = width >= 128 ? 1 : 128 / width;  // of a block
  const long long grid = (static_cast<long long>(a.M) + rows - 1) / rows;
  switch (nv) {
    case 1: return launch(block_norm_kernel<T, R, 1, AFTER>, grid, width * rows, stream, a, width);
    case 2: return launch(block_norm_kernel<T, R, 2, AFTER>, grid, width * rows, stream, a, width);
    default: return launch(block_norm_kernel<T, R, 4, AFTER>, grid, width * rows, stream, a, width);
  }
}

template <typename T, typename R>
cudaError_t launch_typed(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
  return a.f ? launch_rows<T, R, true>(a, num_sms, stream) : launch_rows<T, R, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_block_norm(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
  if (a.bf16)
    return a.f32_residual ? launch_typed<__nv_bfloat16, float>(a, num_sms, stream)
                          : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, num_sms, stream);
  return a.f32_residual ? launch_typed<__half, float>(a, num_sms, stream)
                        : launch_typed<__half, __half>(a, num_sms, stream);
}

}  // namespace i8mm
