// norm.cu -- the row passes around a block of layers.
//
//   before:  h = norm(x; w, b)
//   after:   y = x_scale x + f_scale gate norm(f; w, b),  h = norm(y; w', b')
//   norm(v; w, b) = (v - mean) / sqrt(mean((v - mean)^2) + eps) w + b   (mean 0 for the RMS norm)
//
// One pass over memory: a row lives in the registers of its threads between its loads and its
// stores, both norms' sums are taken there (deviations about the mean, not differences of squares),
// and h is made of y as it was rounded for storing.  What bounds it is the bytes of f, x, y and h; the
// weights and gates stay in cache (rows do not allocate in L1).  With many rows a thread takes 4 pieces
// of 8 elements (blocks small enough that an SM has several rows in flight); with few rows 1, for
// latency.  A ring of rows copied ahead by each thread was slower (2048 x 12288 after a block: 75 us
// against 48): it leaves fewer threads, and instructions, about 290 for 8 elements there, bound it.
#include "block.cuh"
#include "ptx.cuh"

namespace i8mm {

namespace {

constexpr int kMaxPieces = 4;
// threads of a block whose threads hold nv pieces in registers
template <typename R>
__host__ __device__ constexpr int max_threads(int nv) {
  return nv * static_cast<int>(sizeof(R)) > 8 ? 512 : 1024;
}
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
// The same of a row, which is read once: it does not push the weights out of L1.
template <typename V>
__device__ __forceinline__ Piece<V> load8_once(const V* p) {
  Piece<V> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(V)) / 2; ++i)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.q[i].x), "=r"(r.q[i].y), "=r"(r.q[i].z), "=r"(r.q[i].w)
                 : "l"(reinterpret_cast<const uint4*>(p) + i));
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
template <typename V>
__device__ __forceinline__ Piece<V> round8(const float (&v)[8]) {
  Piece<V> r;
  if constexpr (sizeof(V) == 4) {
    r.q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    r.q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    r.q[0] = make_uint4(pack2<V>(v[0], v[1]), pack2<V>(v[2], v[3]), pack2<V>(v[4], v[5]), pack2<V>(v[6], v[7]));
  }
  return r;
}
template <typename V>
__device__ __forceinline__ void store8(V* p, const Piece<V>& r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(V)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.q[i];
}

// v = v w + b over 8 neighbours; null pointers stand for ones and zeros.
template <typename T>
__device__ __forceinline__ void affine8(float (&v)[8], const T* w, const T* b) {
  float t[8], u[8];
  if (w && b) {
    floats8<T>(load8<T>(w), t);
    floats8<T>(load8<T>(b), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], t[i], u[i]);
  } else if (w) {
    floats8<T>(load8<T>(w), t);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= t[i];
  } else if (b) {
    floats8<T>(load8<T>(b), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] += u[i];
  }
}
template <typename T>
__device__ __forceinline__ const T* piece_of(const void* p, int c) {
  return p ? static_cast<const T*>(p) + 8 * c : nullptr;
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
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[first_warp + lane] : 0.0f);
}

}  // namespace

// One row for every `width` threads (whole warps), NV pieces of 8 elements a thread.
template <typename T, typename R, int NV, bool AFTER, bool LAYER>
__global__ void __launch_bounds__(max_threads<R>(NV)) block_norm_kernel(const BlockNormArgs a, int width) {
  __shared__ float red[4][32];
  grid_launch_dependents();
  const int warps = width / 32, in_block = threadIdx.x / width, tid = threadIdx.x % width;
  const int first_warp = in_block * warps;
  const int m = blockIdx.x * (blockDim.x / width) + in_block;
  const int pieces = a.D / 8;
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const bool row_ok = m < a.M;
  const long long at = static_cast<long long>(row_ok ? m : 0) * a.D;
  bool ok[NV];  // this thread's pieces that there are
#pragma unroll
  for (int i = 0; i < NV; ++i) ok[i] = row_ok && tid + i * width < pieces;
  grid_dependency_wait();

  // The row stays packed between its passes: f and x, then y in x's place.
  Piece<R> xp[NV];
  Piece<T> fp[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (ok[i]) {
      if (AFTER) fp[i] = load8_once<T>(static_cast<const T*>(a.f) + at + 8 * (tid + i * width));
      xp[i] = load8_once<R>(static_cast<const R*>(a.x) + at + 8 * (tid + i * width));
    }
  }
  // sum of the squares of p about `mean`, and of p
  auto squares = [&](auto& p, float mean) {
    float s = 0.0f, v[8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (ok[i]) {
        floats8(p[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (LAYER) v[e] -= mean;
          s = fmaf(v[e], v[e], s);
        }
      }
    }
    return s;
  };
  auto total = [&](auto& p) {
    float s = 0.0f, v[8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (ok[i]) {
        floats8(p[i], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[e];
      }
    }
    return s;
  };
  float mean = 0.0f, s = 0.0f;  // s: of y, its sum for the layer norm, otherwise of its squares
  if constexpr (AFTER) {
    float r = 1.0f;
    if (a.post_norm) {
      if (LAYER) mean = row_sum(total(fp), red[0], first_warp, warps) * inv_d;
      r = rsqrtf(row_sum(squares(fp, mean), red[1], first_warp, warps) * inv_d + a.eps);
    }
    const T* gate = nullptr;
    if (a.gate)
      gate = static_cast<const T*>(a.gate) +
             static_cast<long long>(static_cast<unsigned>(row_ok ? m : 0) / static_cast<unsigned>(a.rows_per_gate)) * a.D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * width;
      if (ok[i]) {
        float v[8], t[8];
        floats8(fp[i], v);
        if (a.post_norm) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = (LAYER ? v[e] - mean : v[e]) * r;
          affine8<T>(v, piece_of<T>(a.post_w, c), piece_of<T>(a.post_b, c));
        }
        if (gate) affine8<T>(v, gate + 8 * c, nullptr);
        floats8(xp[i], t);
        if (a.x_scale != 1.0f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] *= a.x_scale;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(a.f_scale, v[e], t[e]);
        xp[i] = round8<R>(v);
        if (a.y) store8<R>(static_cast<R*>(a.y) + at + 8 * c, xp[i]);
        floats8(xp[i], v);  // as it is stored
#pragma unroll
        for (int e = 0; e < 8; ++e) s = LAYER ? s + v[e] : fmaf(v[e], v[e], s);
      }
    }
    if (!a.h) return;
  } else {
    s = LAYER ? total(xp) : squares(xp, 0.0f);
  }
  s = row_sum(s, red[2], first_warp, warps);
  if (LAYER) {
    mean = s * inv_d;
    s = row_sum(squares(xp, mean), red[3], first_warp, warps);
  }
  const float r = rsqrtf(s * inv_d + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = tid + i * width;
    if (ok[i]) {
      float v[8];
      floats8(xp[i], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (LAYER ? v[e] - mean : v[e]) * r;
      affine8<T>(v, piece_of<T>(a.next_w, c), piece_of<T>(a.next_b, c));
      store8<T>(static_cast<T*>(a.h) + at + 8 * c, round8<T>(v));
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
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + m / a.rows_per_gate * a.D : nullptr;
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
    fr = rsqrtf(row_sum(s, red[1], 0, kWarps) * inv_d + a.eps);
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
    affine8<T>(v, piece_of<T>(a.post_w, c), piece_of<T>(a.post_b, c));
    if (gate) affine8<T>(v, gate + 8 * c, nullptr);
    float xv[8];
    floats8<R>(piece, xv);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(a.f_scale, v[e], a.x_scale * xv[e]);
    piece = round8<R>(v);
    floats8<R>(piece, v);
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
    yr = rsqrtf(row_sum(s, red[3], 0, kWarps) * inv_d + a.eps);
  }
  for (int c = threadIdx.x; c < pieces; c += kLongThreads) {
    value(c, v, piece);
    if (a.y) store8<R>(static_cast<R*>(a.y) + at + 8 * c, piece);
    if (a.h) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (v[e] - ym) * yr;
      affine8<T>(v, piece_of<T>(a.next_w, c), piece_of<T>(a.next_b, c));
      store8<T>(static_cast<T*>(a.h) + at + 8 * c, round8<T>(v));
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

template <typename T, typename R, bool AFTER, bool LAYER>
cudaError_t launch_rows(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
  const int pieces = a.D / 8;
  if (pieces > max_threads<R>(kMaxPieces) * kMaxPieces)
    return launch(block_norm_long_kernel<T, R>, a.M, kLongThreads, stream, a);
  // 1 / 2 / 4 pieces a thread, us: 2048 x 12288 after 65 / 65 / 48, 4096 x 4096 before 18.8 / 14.5 /
  // 13.7, 128 x 4096 after 4.2 / 4.1 / 5.3, 1 x 4096 after 2.8 / 3.3 / 4.7
  int nv = a.M >= num_sms * 4 ? 4 : 1;
  while ((pieces + nv - 1) / nv > max_threads<R>(nv)) nv *= 2;
  const int width = ((pieces + nv - 1) / nv + 31) / 32 * 32;
  const int rows = width >= 128 ? 1 : 128 / width;  // of a block
  const long long grid = (static_cast<long long>(a.M) + rows - 1) / rows;
  switch (nv) {
    case 1: return launch(block_norm_kernel<T, R, 1, AFTER, LAYER>, grid, width * rows, stream, a, width);
    case 2: return launch(block_norm_kernel<T, R, 2, AFTER, LAYER>, grid, width * rows, stream, a, width);
    default: return launch(block_norm_kernel<T, R, 4, AFTER, LAYER>, grid, width * rows, stream, a, width);
  }
}

template <typename T, typename R>
cudaError_t launch_typed(const BlockNormArgs& a, int num_sms, cudaStream_t stream) {
  if (a.layer_norm)
    return a.f ? launch_rows<T, R, true, true>(a, num_sms, stream)
               : launch_rows<T, R, false, true>(a, num_sms, stream);
  return a.f ? launch_rows<T, R, true, false>(a, num_sms, stream)
             : launch_rows<T, R, false, false>(a, num_sms, stream);
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
