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
// against 48 then): it leaves fewer threads, and instructions were what bound it; packed float32
// halves the arithmetic.
//
// Measured, us: 2048 x 12288 after a block, norm of f, gate of every channel, 39 (5.2 TB/s, 79 % of
// the measured copy rate; 43 with a gate row for each of 4 sequences), 4096 x 5120 layer norm of float32
// rows 25 (5.1 TB/s), 8 x 4096 1.9 before and 2.7 after a block (latency: one trip to memory, 1 to 4
// block-wide sums, one store).
#include "block.cuh"
#include "codes.cuh"
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
// Blocks of 384 threads and a little less: with 56 registers a thread (80 with float32 rows), 3 of them
// fit on an SM (2), not 2 (1).  2048 x 12288 after a block, 16-bit rows 45.0 -> 42.7 us, float32 rows
// 71.7 -> 67.7; other widths gain no block, or lose by it (4096 x 4096 26.9 -> 27.4).
constexpr int kTight = 8;  // of KIND
constexpr int kTightThreads = 384;
inline bool tight_width(int width) { return width > 341 && width <= kTightThreads; }
template <typename R>
__host__ __device__ constexpr int threads_bound(int nv, int kind) {
  return kind & kTight ? kTightThreads : max_threads<R>(nv);
}
template <typename R>
__host__ __device__ constexpr int blocks_bound(int kind) {
  return kind & kTight ? (sizeof(R) == 4 ? 2 : 3) : 0;  // 0: no bound
}

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
// 8 neighbours as float32, two to a register pair: the arithmetic is in packed float32, half as many
// instructions.
struct Floats {
  uint64_t p[4];
};
template <typename V>
__device__ __forceinline__ Floats floats8(const Piece<V>& r) {
  Floats f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(V) == 4) {
      const uint4& q = r.q[i / 2];
      f.p[i] = (i & 1) ? f32x2_pack(__uint_as_float(q.z), __uint_as_float(q.w))
                       : f32x2_pack(__uint_as_float(q.x), __uint_as_float(q.y));
    } else {
      const uint32_t w = i == 0 ? r.q[0].x : i == 1 ? r.q[0].y : i == 2 ? r.q[0].z : r.q[0].w;
      const float2 v = unpack2<V>(w);
      f.p[i] = f32x2_pack(v.x, v.y);
    }
  }
  return f;
}
template <typename V>
__device__ __forceinline__ Piece<V> round8(const Floats& f) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f32x2_unpack(f.p[i], w[2 * i], w[2 * i + 1]);
  Piece<V> r;
  if constexpr (sizeof(V) == 4) {
    r.q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    r.q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack2<V>(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    r.q[0] = make_uint4(h[0], h[1], h[2], h[3]);
  }
  return r;
}
__device__ __forceinline__ uint64_t twice(float v) { return f32x2_pack(v, v); }
__device__ __forceinline__ void scale(Floats& f, uint64_t s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = f32x2_mul(f.p[i], s);
}
__device__ __forceinline__ void shift(Floats& f, uint64_t s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f.p[i] = f32x2_add(f.p[i], s);
}
__device__ __forceinline__ void add_squares(uint64_t& s, const Floats& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s = f32x2_fma(f.p[i], f.p[i], s);
}
__device__ __forceinline__ void add_all(uint64_t& s, const Floats& f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) s = f32x2_add(s, f.p[i]);
}
__device__ __forceinline__ float halves(uint64_t s) {
  uint32_t x, y;
  f32x2_unpack(s, x, y);
  return __uint_as_float(x) + __uint_as_float(y);
}
template <typename V>
__device__ __forceinline__ void store8(V* p, const Piece<V>& r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(V)) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = r.q[i];
}

// f = f w + b over piece c; null pointers stand for ones and zeros.  Where STD, w is there, and b just
// for the layer norm.
template <typename T, bool STD, bool LAYER>
__device__ __forceinline__ void affine8(Floats& f, const void* w, const void* b, int c) {
  const bool has_w = STD || w, has_b = STD ? LAYER : b != nullptr;
  Floats t, u;
  if (has_w) t = floats8<T>(load8<T>(static_cast<const T*>(w) + 8 * c));
  if (has_b) u = floats8<T>(load8<T>(static_cast<const T*>(b) + 8 * c));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (has_w && has_b) f.p[i] = f32x2_fma(f.p[i], t.p[i], u.p[i]);
    else if (has_w) f.p[i] = f32x2_mul(f.p[i], t.p[i]);
    else if (has_b) f.p[i] = f32x2_add(f.p[i], u.p[i]);
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
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  return warp_sum(lane < warps ? red[first_warp + lane] : 0.0f);
}

}  // namespace

// One row for every `width` threads (whole warps), NV pieces of 8 elements a thread.
// KIND: 0 any call; otherwise the usual one, whose norms have weights (and biases just if they are
// layer norms), whose x_scale is 1 and whose results are all wanted: 1, and 2 more with a norm of f,
// and 4 more with a gate; kTight more in blocks of that width.
template <typename T, typename R, int NV, bool AFTER, bool LAYER, int KIND>
__global__ void __launch_bounds__(threads_bound<R>(NV, KIND), blocks_bound<R>(KIND))
    block_norm_kernel(const BlockNormArgs a, int width) {
  constexpr bool STD = KIND != 0;
  __shared__ float red[4][32];
  const bool post = STD ? (KIND & 2) != 0 : a.post_norm, gated = STD ? (KIND & 4) != 0 : a.gate != nullptr;
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
  grid_launch_dependents();  // not before the wait: the launch after this one would reach back past it

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
    uint64_t s = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (ok[i]) {
        Floats v = floats8(p[i]);
        if (LAYER) shift(v, twice(-mean));
        add_squares(s, v);
      }
    }
    return halves(s);
  };
  auto total = [&](auto& p) {
    uint64_t s = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (ok[i]) add_all(s, floats8(p[i]));
    return halves(s);
  };
  float mean = 0.0f, s;  // s: of y, its sum for the layer norm, otherwise of its squares
  if constexpr (AFTER) {
    float r = 1.0f;
    if (post) {
      if (LAYER) mean = row_sum(total(fp), red[0], first_warp, warps) * inv_d;
      r = rsqrtf(row_sum(squares(fp, mean), red[1], first_warp, warps) * inv_d + a.eps);
    }
    const T* gate = nullptr;
    if (gated)
      gate = static_cast<const T*>(a.gate) +
             static_cast<long long>(static_cast<unsigned>(row_ok ? m : 0) / static_cast<unsigned>(a.rows_per_gate)) * a.D;
    const uint64_t f_scale = twice(a.f_scale);
    uint64_t sums = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = tid + i * width;
      if (ok[i]) {
        Floats v = floats8(fp[i]);
        if (post) {
          if (LAYER) shift(v, twice(-mean));
          scale(v, twice(r));
          affine8<T, STD, LAYER>(v, a.post_w, a.post_b, c);
        }
        if (gated) affine8<T, true, false>(v, gate, nullptr, c);
        Floats x = floats8(xp[i]);
        if (!STD && a.x_scale != 1.0f) scale(x, twice(a.x_scale));
#pragma unroll
        for (int e = 0; e < 4; ++e) v.p[e] = f32x2_fma(f_scale, v.p[e], x.p[e]);
        xp[i] = round8<R>(v);
        if (STD || a.y) store8<R>(static_cast<R*>(a.y) + at + 8 * c, xp[i]);
        v = floats8(xp[i]);  // as it is stored
        if (LAYER) add_all(sums, v);
        else add_squares(sums, v);
      }
    }
    if (!STD && !a.h) return;
    s = halves(sums);
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
      Floats v = floats8(xp[i]);
      if (LAYER) shift(v, twice(-mean));
      scale(v, twice(r));
      affine8<T, STD, LAYER>(v, a.next_w, a.next_b, c);
      store8<T>(static_cast<T*>(a.h) + at + 8 * c, round8<T>(v));
    }
  }
}

// Longer rows: one block a row, which is read again (from L2) for each of the sums and written in
// the last pass, every element by the thread that read it.  2048 rows, us: 18432 in float32 76 before and
// 156 after a block (35 and 69 of bytes), 40960 in 16 bits 109 and 207 (51 and 102).
template <typename T, typename R>
__global__ void __launch_bounds__(kLongThreads) block_norm_long_kernel(const BlockNormArgs a) {
  __shared__ float red[4][kLongThreads / 32];
  constexpr int kWarps = kLongThreads / 32;
  const long long m = blockIdx.x, at = m * a.D;
  const int pieces = a.D / 8;
  const float inv_d = 1.0f / static_cast<float>(a.D);
  const T* f = a.f ? static_cast<const T*>(a.f) + at : nullptr;
  const R* x = static_cast<const R*>(a.x) + at;
  const T* gate = a.gate ? static_cast<const T*>(a.gate) + m / a.rows_per_gate * a.D : nullptr;
  grid_dependency_wait();
  grid_launch_dependents();

  // mean and reciprocal deviation of the row whose piece c is piece(c)
  auto statistics = [&](auto piece, float* red0, float* red1, float& mean, float& r) {
    uint64_t s = 0;
    mean = 0.0f;
    if (a.layer_norm) {
      for (int c = threadIdx.x; c < pieces; c += kLongThreads) add_all(s, piece(c));
      mean = row_sum(halves(s), red0, 0, kWarps) * inv_d;
      s = 0;
    }
    for (int c = threadIdx.x; c < pieces; c += kLongThreads) {
      Floats v = piece(c);
      shift(v, twice(-mean));
      add_squares(s, v);
    }
    r = rsqrtf(row_sum(halves(s), red1, 0, kWarps) * inv_d + a.eps);
  };
  float fm = 0.0f, fr = 1.0f, ym = 0.0f, yr = 1.0f;
  if (a.post_norm)
    statistics([&](int c) { return floats8(load8<T>(f + 8 * c)); }, red[0], red[1], fm, fr);
  // the residual sum's piece c, as it is stored
  auto value = [&](int c) {
    const Piece<R> xp = load8<R>(x + 8 * c);
    if (!f) return xp;
    Floats v = floats8(load8<T>(f + 8 * c)), t = floats8(xp);
    shift(v, twice(-fm));
    scale(v, twice(fr));
    affine8<T, false, false>(v, a.post_w, a.post_b, c);
    affine8<T, false, false>(v, gate, nullptr, c);
    scale(t, twice(a.x_scale));
#pragma unroll
    for (int e = 0; e < 4; ++e) v.p[e] = f32x2_fma(twice(a.f_scale), v.p[e], t.p[e]);
    return round8<R>(v);
  };
  if (a.h) statistics([&](int c) { return floats8(value(c)); }, red[2], red[3], ym, yr);
  for (int c = threadIdx.x; c < pieces; c += kLongThreads) {
    const Piece<R> y = value(c);
    if (a.y) store8<R>(static_cast<R*>(a.y) + at + 8 * c, y);
    if (a.h) {
      Floats v = floats8(y);
      shift(v, twice(-ym));
      scale(v, twice(yr));
      affine8<T, false, false>(v, a.next_w, a.next_b, c);
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
  // 1 / 2 / 4 pieces a thread, us: 2048 x 12288 after 68 / 68 / 42, 4096 x 4096 before 19.1 / 16.0 /
  // 13.2, 592 x 4096 after 7.0 / 5.5 / 5.3, 128 x 4096 3.7 / 4.3 / 4.2, 1 x 4096 3.1 / 3.7 / 3.9
  int nv = a.M >= num_sms * 4 ? 4 : 1;
  while ((pieces + nv - 1) / nv > max_threads<R>(nv)) nv *= 2;
  const int width = ((pieces + nv - 1) / nv + 31) / 32 * 32;
  const int rows = width >= 128 ? 1 : 128 / width;  // of a block
  const long long grid = (static_cast<long long>(a.M) + rows - 1) / rows;
  auto run = [&](auto kernel) { return launch(kernel, grid, width * rows, stream, a, width); };
  if (nv == 1) return run(block_norm_kernel<T, R, 1, AFTER, LAYER, 0>);
  if (nv == 2) return run(block_norm_kernel<T, R, 2, AFTER, LAYER, 0>);
  // many rows: the usual calls without the tests of each option (2048 x 12288 after: 48 -> 42 us)
  auto usual = [](const void* w, const void* b) { return w && (b != nullptr) == LAYER; };
  if (a.h && usual(a.next_w, a.next_b) && a.x_scale == 1.0f) {
    if constexpr (!AFTER) {
      return run(block_norm_kernel<T, R, 4, AFTER, LAYER, 1>);
    } else if (a.y && (!a.post_norm || usual(a.post_w, a.post_b))) {
      auto kind = [&](auto plain, auto tight) { return run(tight_width(width) ? tight : plain); };
      if (a.post_norm)
        return a.gate ? kind(block_norm_kernel<T, R, 4, AFTER, LAYER, 7>,
                             block_norm_kernel<T, R, 4, AFTER, LAYER, 7 + kTight>)
                      : kind(block_norm_kernel<T, R, 4, AFTER, LAYER, 3>,
                             block_norm_kernel<T, R, 4, AFTER, LAYER, 3 + kTight>);
      return a.gate ? kind(block_norm_kernel<T, R, 4, AFTER, LAYER, 5>,
                           block_norm_kernel<T, R, 4, AFTER, LAYER, 5 + kTight>)
                    : kind(block_norm_kernel<T, R, 4, AFTER, LAYER, 1>,
                           block_norm_kernel<T, R, 4, AFTER, LAYER, 1 + kTight>);
    }
  }
  return run(block_norm_kernel<T, R, 4, AFTER, LAYER, 0>);
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
