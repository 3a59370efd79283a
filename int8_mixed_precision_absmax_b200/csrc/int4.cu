// int4.cu -- 4-bit weights with group scales: the quantizer, its inverse, and which kernel multiplies.
//
// Both passes are bound by the bytes of the 16-bit weights (one read or one write, and a quarter of
// that for the codes).  A lane takes 16 neighbouring columns at a time, so a group's scale is found
// once for 16 values, and asks for its next ones before it works on those it has.  Measured, us, fp16
// 49152 x 12288, groups of 128: quantizer 276 (5.5 TB/s, 84 % of the measured copy rate), its inverse 269
// (5.6 TB/s); 4096 x 4096, groups of 64 with zero points: 11.3 and 8.6.
#include <type_traits>

#include "block.cuh"
#include "codes.cuh"

namespace i8mm {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The extremes of values of type T, two at a time: the largest and, where AFFINE, the smallest, or
// else the largest magnitude; a NaN wherever one of the values is.
template <typename T, bool AFFINE>
struct Extremes {
  using T2 = typename Half2Of<T>::type;
  T2 hi, lo;
  static __device__ __forceinline__ T2 of(uint32_t w) { return *reinterpret_cast<T2*>(&w); }
  static __device__ __forceinline__ T2 from(T2 v, int o) {
    return of(__shfl_xor_sync(~0u, *reinterpret_cast<uint32_t*>(&v), o));
  }
  __device__ __forceinline__ void start() { hi = lo = of(0u); }
  __device__ __forceinline__ void add(uint32_t w) {
    hi = __hmax2_nan(hi, AFFINE ? of(w) : __habs2(of(w)));
    if (AFFINE) lo = __hmin2_nan(lo, of(w));
  }
  // over the lanes of a segment of `width`
  __device__ __forceinline__ void join(int width) {
    for (int o = width / 2; o > 0; o >>= 1) {
      hi = __hmax2_nan(hi, from(hi, o));
      if (AFFINE) lo = __hmin2_nan(lo, from(lo, o));
    }
  }
};

// a / D correctly rounded: a (1/D) put right by its remainder (Markstein), above float32's smallest
// numbers.
template <int D>
__device__ __forceinline__ float divide(float a) {
  constexpr float kD = static_cast<float>(D), kInv = 1.0f / kD;
  if (a < 1e-30f) return __fdiv_rn(a, kD);
  const float q = a * kInv;
  return fmaf(fmaf(-q, kD, a), kInv, q);
}

// Whole numbers rne(w / s), as float32, for w and s of a 16-bit type: kSnap makes w (1/s) a multiple
// of 2^-14.  The true quotient (|w / s| < 16) is half-way between two whole numbers, and then comes
// out so, or 2^-13 and more away from that, since w and s have at most 11 bits; so the second
// rounding, to a whole number, goes as that of the float32 quotient.
constexpr float kSnap = 768.0f, kWhole = 12582912.0f;  // 1.5 * 2^9, 1.5 * 2^23

// Whether the reciprocal of s is a normal number, and s is rounded to T finely enough (half a step
// of 2^-8) that |w / s| stays below 7.5.
template <typename T>
__device__ __forceinline__ bool plain_scale(float s) {
  return std::is_same<T, __half>::value ? s >= 6.2e-5f : s >= 1e-30f && s <= 1e30f;
}
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
}

// Scale and zero point of a group from its extremes.
template <typename T, bool AFFINE>
__device__ __forceinline__ void group_params(const Extremes<T, AFFINE>& e, T& s, float& z) {
  const float hi = to_f32(__hmax_nan(e.hi.x, e.hi.y));
  const float nlo = AFFINE ? -to_f32(__hmin_nan(e.lo.x, e.lo.y)) : 0.0f;
  z = kInt4Zero;
  if (!(hi <= 3.4028235e38f && nlo <= 3.4028235e38f)) {
    s = from_f32<T>(__int_as_float(0x7FC00000));
    return;
  }
  if (!AFFINE) {
    s = from_f32<T>(divide<7>(hi));
    return;
  }
  s = from_f32<T>(__fadd_rn(divide<15>(hi), divide<15>(nlo)));
  const float sf = to_f32(s);
  z = 0.0f;
  if (plain_scale<T>(sf))
    z = (fmaf(nlo, reciprocal(sf), kSnap) + (kWhole - kSnap)) - kWhole;
  else if (sf > 0.0f)
    z = rintf(__fdiv_rn(nlo, sf));
  z = fminf(z, 15.0f);
}

// The word of 8 neighbours, two at a time in the order of the word's halves.  Four codes of a half
// are one number below 2^16.
template <typename T, bool AFFINE>
__device__ __forceinline__ uint32_t encode8(const uint4& v, float inv, float z) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
  const uint64_t inv2 = f32x2_pack(inv, inv), k16 = f32x2_pack(16.0f, 16.0f);
  const uint64_t snap = f32x2_pack(kSnap, kSnap), up = f32x2_pack(kWhole - kSnap, kWhole - kSnap);
  const uint64_t down = f32x2_pack(z - kWhole, z - kWhole);
  uint64_t acc = 0;
#pragma unroll
  for (int j = 3; j >= 0; --j) {
    const float2 f = unpack2<T>(r[j]);
    uint64_t u = f32x2_add(f32x2_add(f32x2_fma(f32x2_pack(f.x, f.y), inv2, snap), up), down);
    if (AFFINE) {  // both extremes may have been rounded away from the zero point
      uint32_t x, y;
      f32x2_unpack(u, x, y);
      u = f32x2_pack(fminf(__uint_as_float(x), 15.0f), fminf(__uint_as_float(y), 15.0f));
    }
    acc = j == 3 ? u : f32x2_fma(acc, k16, u);
  }
  uint32_t even, odd;
  f32x2_unpack(f32x2_add(acc, f32x2_pack(8388608.0f, 8388608.0f)), even, odd);
  return __byte_perm(even, odd, 0x5410);
}

// The same by the definition, for any scale.
template <typename T, bool AFFINE>
__device__ __noinline__ uint32_t encode8_any(uint4 v, float s, float z) {
  const uint32_t r[4] = {v.x, v.y, v.z, v.w};
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 p = unpack2<T>(r[j / 2]);
    const float w = (j & 1) ? p.y : p.x;
    float u = z;
    if (s > 0.0f) u = fminf(fmaxf(__fadd_rn(rintf(__fdiv_rn(w, s)), z), AFFINE ? 0.0f : 1.0f), 15.0f);
    word |= static_cast<uint32_t>(u) << (4 * int4_nibble(j));
  }
  return word;
}

// Goes through the spans of `n` rows in steps of all warps of the grid, without divisions.
struct SpanWalk {
  long long row;
  int span, d_span;
  long long d_row;
  int spans;
  __device__ __forceinline__ SpanWalk(int spans_) : spans(spans_) {
    const long long i = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
    const long long step = static_cast<long long>(gridDim.x) * kWarps;
    row = i / spans;
    span = static_cast<int>(i % spans);
    d_row = step / spans;
    d_span = static_cast<int>(step % spans);
  }
  __device__ __forceinline__ void next() {
    row += d_row;
    span += d_span;
    if (span >= spans) {
      span -= spans;
      ++row;
    }
  }
};

}  // namespace

// Groups of 32, 64, 128 or 256 columns: `width` lanes of 16 columns each; a warp takes 512 columns.
template <typename T, bool AFFINE>
__global__ void __launch_bounds__(kThreads)
    int4_quant_kernel(const T* __restrict__ W, int N, int K, int width, int groups,
                      uint8_t* __restrict__ codes, T* __restrict__ scales,
                      uint8_t* __restrict__ zeros) {
  const int lane = threadIdx.x & 31;
  const int group_shift = 4 + __ffs(width) - 1;
  SpanWalk at((K + 511) / 512);
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 v0 = none, v1 = none;
  auto fetch = [&]() {
    const int k = at.span * 512 + lane * 16;
    v0 = v1 = none;
    if (at.row < N && k < K) {
      const uint4* p = reinterpret_cast<const uint4*>(W + at.row * K + k);
      v0 = __ldcs(p);
      v1 = __ldcs(p + 1);
    }
  };
  fetch();
  while (at.row < N) {
    const uint4 a = v0, b = v1;
    const long long row = at.row;
    const int k = at.span * 512 + lane * 16;
    at.next();
    fetch();
    Extremes<T, AFFINE> e;
    e.start();
    e.add(a.x), e.add(a.y), e.add(a.z), e.add(a.w);
    e.add(b.x), e.add(b.y), e.add(b.z), e.add(b.w);
    e.join(width);
    T s;
    float z;
    group_params<T, AFFINE>(e, s, z);
    const float sf = to_f32(s);
    uint32_t w0, w1;
    if (plain_scale<T>(sf)) {
      const float inv = reciprocal(sf);
      w0 = encode8<T, AFFINE>(a, inv, z);
      w1 = encode8<T, AFFINE>(b, inv, z);
    } else {
      w0 = encode8_any<T, AFFINE>(a, sf, z);
      w1 = encode8_any<T, AFFINE>(b, sf, z);
    }
    if (k < K) {
      __stcs(reinterpret_cast<uint2*>(codes + row * (K / 2) + k / 2), make_uint2(w0, w1));
      if ((lane & (width - 1)) == 0) {
        scales[row * groups + (k >> group_shift)] = s;
        if (AFFINE) zeros[row * groups + (k >> group_shift)] = static_cast<uint8_t>(z);
      }
    }
  }
}

// Other groups (multiples of 128, or a whole row): one warp per group, which it reads twice, with nothing
// asked for ahead: 49152 x 12288, groups of 512 492 us, of 1024 310, one for each row 459 (231 of bytes).
template <typename T, bool AFFINE>
__global__ void __launch_bounds__(kThreads)
    int4_quant_long_kernel(const T* __restrict__ W, int N, int K, int group, int groups,
                           uint8_t* __restrict__ codes, T* __restrict__ scales,
                           uint8_t* __restrict__ zeros) {
  const int lane = threadIdx.x & 31;
  for (SpanWalk at(groups); at.row < N; at.next()) {
    const int k0 = at.span * group, k1 = static_cast<int>(min(static_cast<long long>(K), static_cast<long long>(k0) + group));
    const uint4* row = reinterpret_cast<const uint4*>(W + at.row * K);
    Extremes<T, AFFINE> e;
    e.start();
    for (int k = k0 + lane * 8; k < k1; k += 256) {
      const uint4 a = row[k / 8];
      e.add(a.x), e.add(a.y), e.add(a.z), e.add(a.w);
    }
    e.join(32);
    T s;
    float z;
    group_params<T, AFFINE>(e, s, z);
    const float sf = to_f32(s);
    const bool plain = plain_scale<T>(sf);
    const float inv = plain ? reciprocal(sf) : 0.0f;
    uint32_t* out = reinterpret_cast<uint32_t*>(codes + at.row * (K / 2));
    for (int k = k0 + lane * 8; k < k1; k += 256)
      out[k / 8] = plain ? encode8<T, AFFINE>(row[k / 8], inv, z)
                         : encode8_any<T, AFFINE>(row[k / 8], sf, z);
    if (lane == 0) {
      scales[at.row * groups + at.span] = s;
      if (AFFINE) zeros[at.row * groups + at.span] = static_cast<uint8_t>(z);
    }
  }
}

// A warp takes 512 columns: each lane the words lane and lane + 32 of them.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    int4_dequant_kernel(const uint32_t* __restrict__ codes, const T* __restrict__ scales,
                        const uint8_t* __restrict__ zeros, int N, int K, unsigned group, int groups,
                        uint4* __restrict__ W_hat) {
  const int lane = threadIdx.x & 31;
  const int words = K / 8;
  SpanWalk at((K + 511) / 512);
  const uint16_t* s16 = reinterpret_cast<const uint16_t*>(scales);
  grid_dependency_wait();
  uint32_t word[2], scale[2], zero[2];
  auto fetch = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = at.span * 64 + i * 32 + lane;
      if (at.row < N && j < words) {
        const long long c = at.row * groups + static_cast<unsigned>(j * 8) / group;
        word[i] = __ldcs(codes + at.row * words + j);
        scale[i] = s16[c];
        zero[i] = zeros ? zeros[c] : kInt4Zero;
      }
    }
  };
  fetch();
  while (at.row < N) {
    const uint32_t w[2] = {word[0], word[1]}, s[2] = {scale[0], scale[1]}, z[2] = {zero[0], zero[1]};
    const long long row = at.row;
    const int j0 = at.span * 64 + lane;
    at.next();
    fetch();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (j0 + i * 32 < words) {
        Int4Values<T> q;
        uint32_t r[4];
        q.set(s[i] * 0x10001u, z[i]);
        q.template word<false>(w[i], r);
        __stcs(W_hat + row * words + j0 + i * 32, make_uint4(r[0], r[1], r[2], r[3]));
      }
    }
  }
  grid_launch_dependents();
}

namespace {

int blocks_for(long long work, int per_block, int num_sms) {
  const long long want = (work + per_block - 1) / per_block;
  const long long most = static_cast<long long>(num_sms) * 8;
  return static_cast<int>(want < most ? want : most);
}

template <typename T, bool AFFINE>
cudaError_t quant_typed(const void* W, int N, int K, int group, uint8_t* codes, void* scales,
                        uint8_t* zeros, int num_sms, cudaStream_t stream) {
  const int groups = int4_groups(K, group);
  const bool short_groups = group == 32 || group == 64 || group == 128 || group == 256;
  const long long spans = short_groups ? (K + 511) / 512 : groups;
  const int grid = blocks_for(spans * N, kWarps, num_sms);
  if (short_groups)
    int4_quant_kernel<T, AFFINE><<<grid, kThreads, 0, stream>>>(
        static_cast<const T*>(W), N, K, group / 16, groups, codes, static_cast<T*>(scales), zeros);
  else
    int4_quant_long_kernel<T, AFFINE><<<grid, kThreads, 0, stream>>>(
        static_cast<const T*>(W), N, K, group, groups, codes, static_cast<T*>(scales), zeros);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_int4_quant(const void* W, int N, int K, int group, bool bf16, uint8_t* codes,
                              void* scales, uint8_t* zeros, int num_sms, cudaStream_t stream) {
  if (bf16)
    return zeros ? quant_typed<__nv_bfloat16, true>(W, N, K, group, codes, scales, zeros, num_sms, stream)
                 : quant_typed<__nv_bfloat16, false>(W, N, K, group, codes, scales, zeros, num_sms, stream);
  return zeros ? quant_typed<__half, true>(W, N, K, group, codes, scales, zeros, num_sms, stream)
               : quant_typed<__half, false>(W, N, K, group, codes, scales, zeros, num_sms, stream);
}

cudaError_t launch_int4_dequant(const Int4Weight& w, void* W_hat, int num_sms,
                                cudaStream_t stream) {
  const int grid = blocks_for(static_cast<long long>(w.N) * ((w.K + 511) / 512), kWarps, num_sms);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(w.codes);
  uint4* out = static_cast<uint4*>(W_hat);
  // launched while the kernel before drains: it waits for that one's results itself
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const unsigned group = static_cast<unsigned>(w.group);
  return w.bf16 ? cudaLaunchKernelEx(&cfg, int4_dequant_kernel<__nv_bfloat16>, codes,
                                     static_cast<const __nv_bfloat16*>(w.scales), w.zeros, w.N, w.K, group,
                                     w.groups, out)
                : cudaLaunchKernelEx(&cfg, int4_dequant_kernel<__half>, codes,
                                     static_cast<const __half*>(w.scales), w.zeros, w.N, w.K, group,
                                     w.groups, out);
}

cudaError_t launch_int4_linear(const Int4LinearArgs& a, int num_sms, cudaStream_t stream) {
  return int4_stream_suits(a.M, a.w.N, a.w.K, a.w.group, num_sms) ? launch_int4_stream(a, num_sms, stream)
                                                                  : launch_int4_tile(a, num_sms, stream);
}

}  // namespace i8mm
