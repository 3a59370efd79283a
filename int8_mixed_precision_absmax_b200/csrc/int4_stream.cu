// int4_stream.cu -- the product on 4-bit weights for up to 8 tokens: every byte of the weights is
// read once, at the rate of HBM.
//
//   Y[m,n] = T( sum_c s[n,c] ( sum_{k in c} u[n,k] X[m,k] - z[n,c] sum_{k in c} X[m,k] ) + bias[n] )
//
// Instructions, not bytes, are what such a kernel runs out of first: one SM must take in 56 weights
// a cycle to keep up with HBM, and its logic unit gives 64 results a cycle.  So the codes go into
// mma.sync almost as they lie in memory, the weights as the 16-row operand and the activations as
// the 8 columns, in one of two ways.
//
// One token (DIGITS): u8 x s8 MMAs.  One AND makes 4 operands of a word's low nibbles, another 4 of
// its high nibbles (16 u; two accumulators keep the two apart and meet when a group is scaled:
// 16 lo + hi).  The activations of a chunk of 256 columns are written in five digits,
//   X = 2^e (256^4 d4 + 256^3 d3 + 256^2 d2 + 256 d1 + d0),  d in -128..127,
// 2^(e+38) near the chunk's largest |X|: whole numbers of 40 bits.  Five of the MMA's eight columns are
// the token, so all sums of a group are whole numbers and exact; scaled, they are summed in float32
// column by column, and at a pair's end over the columns.  The zero point is taken out with the sum of
// the group's digits, which one more MMA against ones gives in every row; where u = z a column adds
// exactly 0, however large.  Only exact digits are used: a chunk that has none (fp16: its largest
// value is 32640 or more and another has bits below 2^e; bf16: one is below about 2^-31 of the
// largest; a NaN or an infinity) keeps its activations in 16 bits and is multiplied like a chunk of
// two tokens.  (Three digits, rounded, took 5.3 us for 4096 x 4096 and 51 for 12288 x 49152, against 5.9
// and 53, but were wrong: where the largest column has the weight 0, all others had lost what is below
// 2^-22 of it.)
//
// Two to 8 tokens: 16-bit MMAs on u - z, which is exact: a code set into the mantissa of 1024 (bf16:
// 128) by one logic instruction, less that number and the zero point, for two weights at a time.  (MMAs
// on the codes alone, the zero point by a sum of the activations, saved the subtractions but took
// half as many MMAs again: 8 tokens of 4096 x 4096 6.9 us, against 6.2; 3 tokens of 13824 x 5120 18.3,
// 17.1.  One token, us in digits / this way: N = 49152, K = 12288 53 / 74, N = 32768, K = 4096 15.9 /
// 20.9, N = 4096, K = 8192 8.0 / 8.5, K = 4096 5.9 / 5.7.  The digits of two tokens are more columns than
// an MMA has.)
//
// Either way the group's scale meets the float32 sum of the group: the weights are never rounded.
// Which k a lane takes is free as long as both operands agree: lane t of a quad takes neighbouring
// words of its row.
//
// A block owns a range of 16-row units and takes them in pairs; its warps share the K axis in
// chunks of 256 columns, each warp with a ring of its own that TMA fills (boxes of 16 or 32 rows x
// 128 bytes, 128-byte swizzle).  Before the wait for the previous launch, which may have made the
// weights, the first chunks are brought as far as L2.  The warp that takes a chunk of the first pair brings that chunk's activations into shared
// memory for all pairs, so nothing waits for the whole of X.  Partial sums meet in shared memory
// every `batch` pairs, in an order that does not change.  (K split over the blocks of a cluster, to
// even out few units, cost more in joining than it gave.)
//
// Measured, us: one token of 12288 x 49152, groups of 128, 53 (5.9 TB/s, 90 % of the measured copy
// rate); one of 4096 x 4096 5.9 and 8 of 4096 x 4096, groups of 64 with zero points, 6.4 (1.5 TB/s: two
// trips to memory, X and then the rest, and the launch); 3 of 13824 x 5120 18.6 (2.0 TB/s: 320 units
// are 2 or 3 to a block, and with 4 warps a scheduler the latencies of a chunk's steps, loads to
// operands to MMAs to scales, are not covered).
#include <type_traits>

#include "block.cuh"
#include "codes.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace i8mm {

namespace {

constexpr int kMaxTok = 8;
constexpr int kDigits = 5;
constexpr int kUnitRows = 16;
constexpr int kChunkK = 256;                        // columns of a chunk: 128 bytes of a row
constexpr int kUnitBytes = kUnitRows * kChunkK / 2;
constexpr int kStageBytes = 2 * kUnitBytes;         // a pair of units
constexpr int kMaxWarps = 16, kMaxStages = 4;
constexpr size_t kSmemMost = 226 * 1024;  // of an SM, for one block or for two

struct StreamArgs {
  const void* X;
  const void* scales;
  const uint8_t* zeros;
  const void* bias;
  void* Y;
  int32_t* status;
  int M, N, K, group, groups;
  int units, chunks, stages, xstride, batch;
  bool vector_groups;  // load_groups: a chunk's groups of a row are one aligned vector
};

struct StreamShared {
  uint64_t full[kMaxWarps][kMaxStages];
  uint64_t x_full;                           // 16-bit operands: the activations are there
  uint64_t x_ready[INT8MM_MAX_K / kChunkK];  // a chunk's activations are operands
  int abort;
};

// d = a b + (first ? c : d): unsigned by signed bytes, 32-bit sums.
__device__ __forceinline__ void mma_u8s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, bool first, int c) {
  const int c0 = first ? c : d[0], c1 = first ? c : d[1], c2 = first ? c : d[2], c3 = first ? c : d[3];
  asm("mma.sync.aligned.m16n8k32.row.col.s32.u8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(c0), "r"(c1), "r"(c2), "r"(c3));
}

// d = a b + (first ? 0 : d)
template <typename T>
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1, bool first) {
  const float c0 = first ? 0.0f : d[0], c1 = first ? 0.0f : d[1];
  const float c2 = first ? 0.0f : d[2], c3 = first ? 0.0f : d[3];
  if constexpr (std::is_same<T, __half>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// W consecutive 32-bit words of shared memory.
template <int W>
__device__ __forceinline__ void lds(uint32_t (&v)[W], uint32_t a) {
  if constexpr (W == 1)
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a));
  else if constexpr (W == 2)
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a));
  else
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(a));
}

// An untiled copy of `bytes` (a multiple of 16) into shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// The scales and zero points of one row over a chunk, one for each of its 8 / SUB blocks of
// 32 SUB columns (all of a block's columns are of one group).
template <int SUB>
struct RowGroups {
  static constexpr int kBlocks = 8 / SUB;
  uint32_t s[(kBlocks + 1) / 2];  // two to a word
  uint32_t z[(kBlocks + 3) / 4];  // four to a word
};

template <int SUB, bool ZP>
__device__ __forceinline__ void load_groups(RowGroups<SUB>& r, const StreamArgs& p, int row, int k0) {
  constexpr int kBlocks = RowGroups<SUB>::kBlocks;
  const long long base = static_cast<long long>(min(row, p.N - 1)) * p.groups;
  const uint16_t* s = static_cast<const uint16_t*>(p.scales) + base;
  const uint8_t* z = ZP ? p.zeros + base : nullptr;
  // groups of one block's width lie side by side: one vector load where every row is aligned to it
  if (kBlocks > 1 && p.vector_groups) {
    const int g = k0 / (32 * SUB);
    if constexpr (kBlocks == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(s + g);
      r.s[0] = v.x, r.s[1] = v.y, r.s[2] = v.z, r.s[3] = v.w;
      if (ZP) {
        const uint2 w = *reinterpret_cast<const uint2*>(z + g);
        r.z[0] = w.x, r.z[1] = w.y;
      }
    } else if constexpr (kBlocks == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(s + g);
      r.s[0] = v.x, r.s[1] = v.y;
      if (ZP) r.z[0] = *reinterpret_cast<const uint32_t*>(z + g);
    } else {
      r.s[0] = *reinterpret_cast<const uint32_t*>(s + g);
      if (ZP) r.z[0] = *reinterpret_cast<const uint16_t*>(z + g);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < (kBlocks + 1) / 2; ++i) r.s[i] = 0;
#pragma unroll
  for (int i = 0; i < (kBlocks + 3) / 4; ++i) r.z[i] = 0;
#pragma unroll
  for (int j = 0; j < kBlocks; ++j) {
    const int g = min((k0 + 32 * SUB * j) / p.group, p.groups - 1);
    r.s[j / 2] |= static_cast<uint32_t>(s[g]) << (16 * (j & 1));
    if (ZP) r.z[j / 4] |= static_cast<uint32_t>(z[g]) << (8 * (j & 3));
  }
}

template <typename T>
__device__ __forceinline__ float scale_value(uint32_t word, int high) {
  const float2 v = unpack2<T>(word);
  return high ? v.y : v.x;
}

// A whole number below 2^22 added to these bits reads as the float kMagic plus that number.
constexpr int kMagicBits = 0x4B400000;
constexpr float kMagic = 12582912.0f;

// A whole number below 2^23, off the slow conversion pipe.
__device__ __forceinline__ float small_float(uint32_t v) {
  return __uint_as_float(v | 0x4B000000u) - 8388608.0f;
}

// One chunk of a pair of units (or of one, where not TWO) added to acc.  row: this lane's row of the
// first unit in the stage, swz its swizzle (the row's number << 4) and x its column's digits at the
// chunk's start; src: the lane that holds the row's scales.
//
// SUB words a lane takes at once: of 32 SUB columns (of one group), lane t of a quad takes those
// from 8 SUB t on.  Two words and their digits are two MMAs, for the low and the high nibbles;
// the digits lie in that order.  A single word is one MMA, low and high nibbles its two halves of k.
template <typename T, int SUB, bool ZP, bool TWO>
__device__ __forceinline__ void add_chunk_digits(float (&acc)[2][4], const RowGroups<SUB>& rg,
                                                 uint32_t row, uint32_t swz, uint32_t x, int t,
                                                 int src) {
  constexpr uint32_t kOnes = 0x01010101u, kLow = 0x0F0F0F0Fu, kHigh = 0xF0F0F0F0u;
  constexpr int U = TWO ? 2 : 1;
#pragma unroll
  for (int j = 0; j < 8 / SUB; ++j) {
    int lo[2][4], hi[2][4], sum[4];
    // columns 32 SUB j + 8 SUB t on: bytes 16 SUB j + 4 SUB t of the row, 16-byte pieces swizzled
    const uint32_t at = row + ((16u * SUB * j + 4u * SUB * t) ^ swz);
    const uint32_t xj = x + 32u * SUB * j + 8u * SUB * t;
    uint32_t wa[2][SUB], wb[2][SUB];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      lds<SUB>(wa[i], at + i * kUnitBytes);
      lds<SUB>(wb[i], at + i * kUnitBytes + 1024);
    }
    if constexpr (SUB == 1) {
      uint32_t xr[2];
      lds<2>(xr, xj);
#pragma unroll
      for (int i = 0; i < U; ++i)
        mma_u8s8(hi[i], wa[i][0] & kLow, wb[i][0] & kLow, wa[i][0] >> 4 & kLow, wb[i][0] >> 4 & kLow,
                 xr[0], xr[1], true, kMagicBits);
      mma_u8s8(sum, kOnes, kOnes, kOnes, kOnes, xr[0], xr[1], true, kMagicBits);
    } else {
#pragma unroll
      for (int w = 0; w < SUB; w += 2) {
        uint32_t xr[4];
        lds<4>(xr, xj + 8u * w);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          mma_u8s8(lo[i], wa[i][w] & kLow, wb[i][w] & kLow, wa[i][w + 1] & kLow, wb[i][w + 1] & kLow,
                   xr[0], xr[1], w == 0, 0);
          mma_u8s8(hi[i], wa[i][w] & kHigh, wb[i][w] & kHigh, wa[i][w + 1] & kHigh,
                   wb[i][w + 1] & kHigh, xr[2], xr[3], w == 0, kMagicBits);
        }
        mma_u8s8(sum, kOnes, kOnes, kOnes, kOnes, xr[0], xr[1], w == 0, kMagicBits);
        mma_u8s8(sum, kOnes, kOnes, kOnes, kOnes, xr[2], xr[3], false, 0);
      }
    }
    // The block's scales: rows of number src and src + 8 of each unit.  16 times the sums of up to
    // 128 columns stay below 2^22, and the float32 steps before the scale are exact.
    const float S[2] = {__int_as_float(sum[0]) - kMagic, __int_as_float(sum[1]) - kMagic};
#pragma unroll
    for (int r = 0; r < 2 * U; ++r) {
      const uint32_t sw = __shfl_sync(~0u, rg.s[j / 2], src + 8 * r);
      const float s = scale_value<T>(sw, j & 1);
      float z = kInt4Zero;
      if (ZP)
        z = small_float(__shfl_sync(~0u, rg.z[j / 4], src + 8 * r) >> (8 * (j & 3)) & 0xFFu);
      if (SUB > 1) z *= 16.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = r / 2, d = 2 * (r & 1) + h;
        const int v = SUB > 1 ? lo[i][d] * 16 + hi[i][d] : hi[i][d];
        acc[i][d] = fmaf(s, fmaf(-z, S[h], __int_as_float(v) - kMagic), acc[i][d]);
      }
    }
  }
}

// The same with 16-bit operands; x: the lane's token's activations at the chunk's start, those from
// byte 256 on `gap` bytes further.
template <typename T, int SUB, bool ZP, bool TWO>
__device__ __forceinline__ void add_chunk_16(float (&acc)[2][4], const RowGroups<SUB>& rg, uint32_t row,
                                          uint32_t swz, uint32_t x, uint32_t gap, int t, int src) {
  constexpr int U = TWO ? 2 : 1;
  const uint32_t x_t = x + 16u * SUB * t;
#pragma unroll
  for (int j = 0; j < 8 / SUB; ++j) {
    // the block's zero points: rows g and g + 8 of each unit
    Int4Values<T> q[4];
#pragma unroll
    for (int r = 0; r < 2 * U; ++r)
      q[r].set(0, ZP ? __shfl_sync(~0u, rg.z[j / 4], src + 8 * r) >> (8 * (j & 3)) & 0xFFu
                     : static_cast<uint32_t>(kInt4Zero));
    float sum[2][2][4];  // of each unit, two for the MMAs to take in turn
    const uint32_t at = row + ((16u * SUB * j + 4u * SUB * t) ^ swz);
    uint32_t wa[2][SUB], wb[2][SUB];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      lds<SUB>(wa[i], at + i * kUnitBytes);
      lds<SUB>(wb[i], at + i * kUnitBytes + 1024);
    }
#pragma unroll
    for (int w = 0; w < SUB; ++w) {
      uint32_t xr[4];
      lds<4>(xr, x_t + 64u * SUB * j + (64 * SUB * j >= 256 ? gap : 0u) + 16u * w);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint32_t a[4], b[4];
        q[2 * i].template offsets<true>(wa[i][w], a);
        q[2 * i + 1].template offsets<true>(wb[i][w], b);
        mma_16x8x16<T>(sum[i][0], a[0], b[0], a[1], b[1], xr[0], xr[1], w == 0);
        mma_16x8x16<T>(sum[i][1], a[2], b[2], a[3], b[3], xr[2], xr[3], w == 0);
      }
    }
#pragma unroll
    for (int r = 0; r < 2 * U; ++r) {
      const float s = scale_value<T>(__shfl_sync(~0u, rg.s[j / 2], src + 8 * r), j & 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = r / 2, d = 2 * (r & 1) + h;
        acc[i][d] = fmaf(s, sum[i][0][d] + sum[i][1][d], acc[i][d]);
      }
    }
  }
}

__device__ __forceinline__ float power_of_2(int e) {  // of a normal number
  return __int_as_float((127 + e) << 23);
}

// The digits' unit 2^e of a chunk from its largest magnitude `most` and its smallest but 0, 0x8000 -
// `least` (their bits in T): most becomes 1 .. 1.992 * 2^38, since digits of -128..127 reach
// 0x7F7F7F7F7F = 1.992 * 2^38.  exact: no value has bits below the unit.
template <typename T>
__device__ __forceinline__ int digit_exponent(uint32_t most, uint32_t least, bool& exact) {
  const uint32_t f = __float_as_uint(unpack2<T>(most).x);
  const int e = max(static_cast<int>((f + 0x10000u) >> 23) - 127 - 38, -126);
  if (std::is_same<T, __half>::value)  // 2^-24 is the type's own unit
    exact = e <= -24;
  else  // the last of the smallest one's 7 bits; 0 alone: least = 0, which is 2^128
    exact = e <= max(static_cast<int>((0x8000u - least) >> 7), 1) - 127 - 7;
  return e;
}

// The digits of 4 activations with the unit 2^e, one word for each digit: with 128 added to each digit,
// they are the bytes of a whole number h 2^20 + l.  Rounded into the mantissa of kMagic, h and l are
// whole numbers below 2^20.
__device__ __forceinline__ void digits4(const uint64_t (&f)[2], int e, uint32_t (&d)[kDigits]) {
  constexpr long long kBias = 0x8080808080ll - (static_cast<long long>(kMagicBits) << 20) - kMagicBits;
  const float h1 = power_of_2(-e - 20), h0 = -power_of_2(e + 20), l1 = power_of_2(-e);
  const uint64_t magic = f32x2_pack(kMagic, kMagic), minus = f32x2_pack(-kMagic, -kMagic);
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t h = f32x2_fma(f[i], f32x2_pack(h1, h1), magic);
    const uint64_t rest = f32x2_fma(f32x2_add(h, minus), f32x2_pack(h0, h0), f[i]);
    const uint64_t l = f32x2_fma(rest, f32x2_pack(l1, l1), magic);
    uint32_t hb[2], lb[2];
    f32x2_unpack(h, hb[0], hb[1]);
    f32x2_unpack(l, lb[0], lb[1]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const unsigned long long b =
          static_cast<unsigned long long>(kBias + static_cast<long long>(static_cast<int>(hb[k])) * (1 << 20)) + lb[k];
      lo[2 * i + k] = static_cast<uint32_t>(b);
      hi[2 * i + k] = static_cast<uint32_t>(b >> 32);
    }
  }
  const uint32_t a0 = __byte_perm(lo[0], lo[1], 0x5140), a1 = __byte_perm(lo[2], lo[3], 0x5140);
  const uint32_t b0 = __byte_perm(lo[0], lo[1], 0x7362), b1 = __byte_perm(lo[2], lo[3], 0x7362);
  d[0] = __byte_perm(a0, a1, 0x5410) ^ 0x80808080u;
  d[1] = __byte_perm(a0, a1, 0x7632) ^ 0x80808080u;
  d[2] = __byte_perm(b0, b1, 0x5410) ^ 0x80808080u;
  d[3] = __byte_perm(b0, b1, 0x7632) ^ 0x80808080u;
  d[4] = __byte_perm(__byte_perm(hi[0], hi[1], 0x0040), __byte_perm(hi[2], hi[3], 0x0040), 0x5410) ^
         0x80808080u;
}

}  // namespace

template <typename T, int SUB, bool ZP, bool DIGITS>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    int4_stream_kernel(const __grid_constant__ CUtensorMap map_unit,
                       const __grid_constant__ CUtensorMap map_pair, const StreamArgs p) {
  extern __shared__ uint8_t stream_smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(stream_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warps = blockDim.x / 32;
  const int cols = DIGITS ? kDigits : p.M;  // of the activations' operand: digits or tokens
  const int part_floats = 32 * p.M;         // a warp's partial sums of a pair
  uint8_t* xs = ring + static_cast<size_t>(warps) * p.stages * kStageBytes;
  StreamShared& S = *reinterpret_cast<StreamShared*>(xs + static_cast<size_t>(cols) * p.xstride);
  float* xscale = reinterpret_cast<float*>(&S + 1);  // DIGITS: of each chunk, of the highest digit; 0: 16 bits
  float* part = xscale + (DIGITS ? p.chunks : 0);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  volatile int* abort = &S.abort;

  if (threadIdx.x == 0) {
    for (int w = 0; w < warps; ++w)
      for (int s = 0; s < p.stages; ++s) mbar_init(&S.full[w][s], 1);
    mbar_init(&S.x_full, 1);
    S.abort = 0;
    prefetch_tmap(&map_unit);
    prefetch_tmap(&map_pair);
  }
  for (int i = threadIdx.x; i < p.chunks; i += blockDim.x) mbar_init(&S.x_ready[i], 1);
  fence_mbarrier_init();
  __syncthreads();

  const int u0 = static_cast<int>(static_cast<long long>(p.units) * blockIdx.x / gridDim.x);
  const int u1 = static_cast<int>(static_cast<long long>(p.units) * (blockIdx.x + 1) / gridDim.x);
  const int pairs = (u1 - u0 + 1) / 2;
  // Chunks go round the warps, on from pair to pair: warp, warp + warps, ... of all in a row.
  uint8_t* my_ring = ring + static_cast<size_t>(warp) * p.stages * kStageBytes;
  uint64_t* my_full = S.full[warp];

  int fp = 0, fc = warp, f_stage = 0, issued = 0;  // the next chunk to request
  auto settle = [&](int& q, int& c) {  // past the pair's last chunk: into the next pair
    while (c >= p.chunks) {
      c -= p.chunks;
      ++q;
    }
  };
  auto request = [&]() {
    if (fp >= pairs) return;
    if (lane == 0) {
      const int u = u0 + 2 * fp;
      const bool two = u + 1 < u1;
      uint8_t* dst = my_ring + f_stage * kStageBytes;
      mbar_arrive_expect_tx(&my_full[f_stage], two ? kStageBytes : kUnitBytes);
      tma_load_2d(two ? &map_pair : &map_unit, dst, &my_full[f_stage], fc * (kChunkK / 2),
                  u * kUnitRows);
    }
    ++issued;
    if (++f_stage == p.stages) f_stage = 0;
    fc += warps;
    settle(fp, fc);
  };
  settle(fp, fc);
  int q = fp, c = fc;  // the next chunk to multiply
  // The weights may be the launch before's, so only L2, which sees its writes, gets them early.
  for (int s = 0, eq = q, ec = c; s < p.stages && eq < pairs; ++s) {
    const int u = u0 + 2 * eq;
    if (lane == 0)
      tma_prefetch_2d(u + 1 < u1 ? &map_pair : &map_unit, ec * (kChunkK / 2), u * kUnitRows);
    ec += warps;
    settle(eq, ec);
  }
  RowGroups<SUB> cur, nxt;
  if (q < pairs) {
    const long long at = static_cast<long long>(min((u0 + 2 * q) * kUnitRows + lane, p.N - 1)) * p.groups +
                         c * kChunkK / p.group;
    prefetch_l2(static_cast<const uint16_t*>(p.scales) + at);
    if (ZP) prefetch_l2(p.zeros + at);
  }

  grid_dependency_wait();
  grid_launch_dependents();  // not before the wait: the launch after this one would reach back past it
  const int pieces = p.K / 8;  // 16 bytes, 8 columns; a lane takes one of each chunk and token
  uint4 xv;                    // DIGITS: of the next chunk of the first pair
  auto load_x = [&](int chunk) {
    const int i = chunk * 32 + lane;
    xv = i < pieces ? static_cast<const uint4*>(p.X)[i] : make_uint4(0, 0, 0, 0);
  };
  if constexpr (DIGITS) {
    if (q == 0) load_x(c);
  } else if (threadIdx.x == 0) {
    const uint32_t bytes = static_cast<uint32_t>(p.K) * 2;
    mbar_arrive_expect_tx(&S.x_full, bytes * p.M);
    for (int m = 0; m < p.M; ++m)
      bulk_load(xs + static_cast<size_t>(m) * p.xstride,
                static_cast<const T*>(p.X) + static_cast<size_t>(m) * p.K, bytes, &S.x_full);
  }
  for (int s = 0; s < p.stages; ++s) request();
  if (q < pairs) load_groups<SUB, ZP>(nxt, p, (u0 + 2 * q) * kUnitRows + lane, c * kChunkK);

  // Row g of an MMA is row `gr` of the unit, the bits of g reversed: the rows that read shared
  // memory together then differ in the swizzle's high bits (conflict-free for 4, 8 and 16 bytes).
  const int gr = (g & 1) << 2 | (g & 2) | g >> 2;
  // columns past the last repeat it: their results are not kept
  const uint32_t x_lane = smem_addr(xs) + static_cast<uint32_t>(min(g, cols - 1)) * p.xstride;
  const uint32_t w_lane = smem_addr(my_ring) + static_cast<uint32_t>(gr) * 128;
  constexpr uint32_t kXChunk = kChunkK * (DIGITS ? 1 : 2);
  // DIGITS: what a digit in this lane's two columns counts, next to the highest; columns past it, 0
  const float weight0 = t <= (kDigits - 1) / 2 ? power_of_2(8 * (2 * t - (kDigits - 1))) : 0.0f;
  const float weight1 = t < (kDigits - 1) / 2 ? power_of_2(8 * (2 * t + 1 - (kDigits - 1))) : 0.0f;
  bool ok = true;
  int stage = 0, done = 0;  // pairs before `done` are stored
  uint32_t phase = 0;
  for (int pair = 0; pair < pairs; ++pair) {
    float acc[2][4] = {};
    while (q == pair) {
      cur = nxt;
      int nq = q, nc = c + warps;
      settle(nq, nc);
      if (nq < pairs) load_groups<SUB, ZP>(nxt, p, (u0 + 2 * nq) * kUnitRows + lane, nc * kChunkK);
      if (pair == 0) {
        // this chunk's activations, for every pair
        if constexpr (DIGITS) {
          const uint4 v = xv;
          // magnitudes of a 16-bit type compare as whole numbers
          const uint32_t m[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
          const uint32_t two = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
          const uint32_t most = __reduce_max_sync(~0u, max(two & 0xFFFFu, two >> 16));
          uint32_t least = 0;
          if (std::is_same<T, __nv_bfloat16>::value) {
            uint32_t l[4];  // 0x8000 less the magnitude, and 0 for 0
#pragma unroll
            for (int i = 0; i < 4; ++i) l[i] = (0x80008000u - m[i]) & 0x7FFF7FFFu;
            const uint32_t both = __vmaxu2(__vmaxu2(l[0], l[1]), __vmaxu2(l[2], l[3]));
            least = __reduce_max_sync(~0u, max(both & 0xFFFFu, both >> 16));
          }
          constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7C00u : 0x7F80u;
          bool exact;
          const int e = digit_exponent<T>(most, least, exact);
          exact = exact && most < kInf;
          uint8_t* out = xs + c * kChunkK;
          if (exact) {
            const float2 p01 = unpack2<T>(v.x), p23 = unpack2<T>(v.y), p45 = unpack2<T>(v.z),
                         p67 = unpack2<T>(v.w);
            // bytes of a word's low nibbles: columns 0, 4, 1, 5; of its high ones: 2, 6, 3, 7
            const uint64_t low[2] = {f32x2_pack(p01.x, p45.x), f32x2_pack(p01.y, p45.y)};
            const uint64_t high[2] = {f32x2_pack(p23.x, p67.x), f32x2_pack(p23.y, p67.y)};
            uint32_t dl[kDigits], dh[kDigits];
            digits4(low, e, dl);
            digits4(high, e, dh);
            // one word: its low nibbles' digits, then its high ones'; two words: both low, then both high
            const int at = SUB == 1 ? 2 * lane : (lane & ~1) * 2 + (lane & 1);
#pragma unroll
            for (int d = 0; d < kDigits; ++d) {
              uint32_t* words = reinterpret_cast<uint32_t*>(out + static_cast<size_t>(d) * p.xstride);
              words[at] = dl[d];
              words[at + (SUB == 1 ? 1 : 2)] = dh[d];
            }
          } else {  // 512 bytes in the places of the first two digits
            *reinterpret_cast<uint4*>(out + lane / 16 * p.xstride + lane % 16 * 16) = v;
          }
          // 16 lo + hi is 16 times the sum
          if (lane == 0)
            xscale[c] = exact ? power_of_2(e + 8 * (kDigits - 1) - (SUB > 1 ? 4 : 0)) : 0.0f;
          if (nq == 0) load_x(nc);
        } else {
          if (ok) ok = __all_sync(~0u, mbar_wait_bounded(&S.x_full, 0, abort));
          const int i = c * 32 + lane;
          if (i >= pieces) {  // zeros up to the chunk's end
            for (int m = 0; m < p.M; ++m)
              reinterpret_cast<uint4*>(xs + static_cast<size_t>(m) * p.xstride)[i] = make_uint4(0, 0, 0, 0);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.x_ready[c]);
      } else if (ok) {
        ok = __all_sync(~0u, mbar_wait_bounded(&S.x_ready[c], 0, abort));
      }
      if (ok) ok = __all_sync(~0u, mbar_wait_bounded(&my_full[stage], phase, abort));
      if (ok) {
        const uint32_t w = w_lane + static_cast<uint32_t>(stage) * kStageBytes;
        const uint32_t x = x_lane + kXChunk * c;
        const bool two = u0 + 2 * pair + 1 < u1;
        if constexpr (DIGITS) {
          float chunk[2][4] = {};
          const float f = xscale[c];
          float w0 = weight0, w1 = weight1;
          if (f != 0.0f) {
            if (two) add_chunk_digits<T, SUB, ZP, true>(chunk, cur, w, 16u * gr, x, t, gr);
            else add_chunk_digits<T, SUB, ZP, false>(chunk, cur, w, 16u * gr, x, t, gr);
            w0 *= f;
            w1 *= f;
          } else {  // every column is the token: the highest digit's place takes it
            const uint32_t x16 = smem_addr(xs) + kXChunk * c, gap = p.xstride - 256;
            if (two) add_chunk_16<T, SUB, ZP, true>(chunk, cur, w, 16u * gr, x16, gap, t, gr);
            else add_chunk_16<T, SUB, ZP, false>(chunk, cur, w, 16u * gr, x16, gap, t, gr);
            w0 = t == (kDigits - 1) / 2 ? 1.0f : 0.0f;
            w1 = 0.0f;
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float* a = &acc[r / 2][2 * (r & 1)];
            const float* v = &chunk[r / 2][2 * (r & 1)];
            a[0] = fmaf(w0, v[0], a[0]);
            a[1] = fmaf(w1, v[1], a[1]);
          }
        } else {
          if (two) add_chunk_16<T, SUB, ZP, true>(acc, cur, w, 16u * gr, x, 0, t, gr);
          else add_chunk_16<T, SUB, ZP, false>(acc, cur, w, 16u * gr, x, 0, t, gr);
        }
      }
      __syncwarp();
      if (ok) request();
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      q = nq;
      c = nc;
    }
    // the pair's partial sums, [token][row] of each warp, in the last 2 batch pairs' places
    float* mine = part + (pair % (2 * p.batch) * warps + warp) * part_floats;
    if constexpr (DIGITS) {  // the columns, all of one token, are added up over the quad
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[r] = acc[r / 2][2 * (r & 1)] + acc[r / 2][2 * (r & 1) + 1];
        v[r] += __shfl_xor_sync(~0u, v[r], 1);
        v[r] += __shfl_xor_sync(~0u, v[r], 2);
      }
      mine[gr + 8 * t] = t == 0 ? v[0] : t == 1 ? v[1] : t == 2 ? v[2] : v[3];
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = 2 * t + h;
        if (m < cols) {
#pragma unroll
          for (int r = 0; r < 4; ++r) mine[m * 32 + gr + 8 * r] = acc[r / 2][2 * (r & 1) + h];
        }
      }
    }
    if ((pair + 1) % p.batch != 0 && pair + 1 < pairs) continue;
    __syncthreads();
    // a warp adds up 32 rows of one token: the first warps after the batch's last pair's number
    for (int o = (warp + pair) % warps; o < (pair + 1 - done) * p.M; o += warps) {
      const int from = done + o / p.M, m = o % p.M;
      const float* sums = part + from % (2 * p.batch) * warps * part_floats + lane;
      float v = 0.0f;
#pragma unroll 8
      for (int w = 0; w < warps; ++w) v += sums[w * part_floats + m * 32];
      const int n = (u0 + 2 * from) * kUnitRows + lane;
      if (n < min(p.N, u1 * kUnitRows)) {
        if (p.bias) v += to_f32(static_cast<const T*>(p.bias)[n]);
        static_cast<T*>(p.Y)[static_cast<size_t>(m) * p.N + n] = from_f32<T>(v);
      }
    }
    done = pair + 1;
  }
  if (!ok) {
    if (lane == 0 && p.status)
      atomicCAS(reinterpret_cast<int*>(p.status), 0, INT8MM_ERR_TIMEOUT);
    // what was requested lands before the block's shared memory is given back
    int dummy = 0;
    for (int j = issued > p.stages ? issued - p.stages : 0; j < issued; ++j)
      mbar_wait_bounded(&my_full[j % p.stages], static_cast<uint32_t>(j / p.stages) & 1u, &dummy);
    if (!DIGITS) mbar_wait_bounded(&S.x_full, 0, &dummy);
  }
}

namespace {

struct StreamPlan {
  int warps, per_sm, stages, xstride, batch;
  bool digits;
  size_t smem;
};

// Columns of 32 SUB are one load of a lane and lie in one group.
int sub_of(int group) { return group == 32 ? 1 : group == 64 ? 2 : 4; }

// The block's shape, the first of an order that fits, at least two stages for each warp.  One block of
// 16 warps brings the activations into shared memory once an SM and lets all warps share the chunks,
// but with few of them a warp has one in a pair, and waits; two blocks of 8 also fill each other's
// pauses.  (us of two blocks of 8 / one of 16 / one of 8; K = 4096: one token, N 4096 6.0 / 6.0 / 5.6,
// N 32768 15.9 / 20.9 / 19.5, 3 tokens 5.9 / 6.3 / 5.7, 18.6 / 20.9 / 22.9, 6 tokens, N 4096 - / 6.5 /
// 5.8; K = 8192: one token, N 4096 - / 8.0 / 8.6, 3 tokens, N 32768 - / 35.5 / 40.0; K = 12288: one
// token, N 49152 - / 53.3 / 68.3, 3 tokens, N 32768 - / 48.5 / 55.9.)
struct Shape { int warps, per_sm; };
constexpr Shape kFewChunks[] = {{8, 2}, {8, 1}, {16, 1}}, kManyChunks[] = {{16, 1}, {8, 1}};
constexpr int kMany = 32;

bool plan_shapes(int M, int K, int group, bool digits, const Shape* shapes, int n, StreamPlan& s) {
  const int sub = sub_of(group), cols = digits ? kDigits : M;
  const int chunks = (K + kChunkK - 1) / kChunkK;
  s.digits = digits;
  // a column's activations up to the last chunk's end, and a pad that sets the quads of two columns
  // apart: 8, 16 or 32 bytes a lane of digits, twice that in 16 bits
  s.xstride = chunks * kChunkK * (digits ? 1 : 2) +
              (digits ? (sub == 1 ? 32 : sub == 2 ? 64 : 16) : (sub == 1 ? 64 : 16));
  for (int i = 0; i < n; ++i) {
    const Shape& shape = shapes[i];
    s.warps = shape.warps;
    s.per_sm = shape.per_sm;
    const size_t most = shape.per_sm == 2 ? kSmemMost / 2 : kSmemMost;
    const size_t pair_bytes = static_cast<size_t>(s.warps) * 32 * M * sizeof(float);
    const size_t fixed = 1024 + static_cast<size_t>(cols) * s.xstride + sizeof(StreamShared) +
                         (digits ? chunks * sizeof(float) : 0);
    for (s.stages = kMaxStages; s.stages >= 2; --s.stages) {
      const size_t ring = static_cast<size_t>(s.warps) * s.stages * kStageBytes;
      for (s.batch = 4; s.batch >= 1; s.batch /= 2) {
        s.smem = fixed + ring + 2 * s.batch * pair_bytes;
        if (s.smem <= most) return true;
      }
    }
  }
  return false;
}

bool plan_stream(int M, int K, int group, StreamPlan& s) {
  if (M > kMaxTok) return false;
  const bool many = K > (kMany - 1) * kChunkK;
  const Shape* shapes = many ? kManyChunks : kFewChunks;
  // one token: digits where the first of the shapes holds them, 5 bytes a column, and 16 bits beyond (K
  // = 18432, N = 16384: 33 us in digits; K = 24576: 45 us in 16 bits)
  return (M == 1 && plan_shapes(M, K, group, true, shapes, 1, s)) ||
         plan_shapes(M, K, group, false, shapes, many ? 2 : 3, s);
}

template <typename T, int SUB, bool ZP, bool DIGITS>
cudaError_t launch_variant(const CUtensorMap (&map)[2], const StreamArgs& p, const StreamPlan& s,
                           int grid, cudaStream_t stream) {
  static std::atomic<unsigned long long> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(int4_stream_kernel<T, SUB, ZP, DIGITS>),
                                   kSmemMost, allowed);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(s.warps * 32);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int4_stream_kernel<T, SUB, ZP, DIGITS>, map[0], map[1], p);
}

template <typename T, bool ZP, bool DIGITS>
cudaError_t launch_sub(const CUtensorMap (&map)[2], const StreamArgs& p, const StreamPlan& s,
                       int grid, cudaStream_t stream) {
  switch (sub_of(p.group)) {
    case 1: return launch_variant<T, 1, ZP, DIGITS>(map, p, s, grid, stream);
    case 2: return launch_variant<T, 2, ZP, DIGITS>(map, p, s, grid, stream);
    default: return launch_variant<T, 4, ZP, DIGITS>(map, p, s, grid, stream);
  }
}

template <typename T>
cudaError_t launch_typed(const CUtensorMap (&map)[2], const StreamArgs& p, const StreamPlan& s,
                         int grid, cudaStream_t stream) {
  if (s.digits)
    return p.zeros ? launch_sub<T, true, true>(map, p, s, grid, stream)
                   : launch_sub<T, false, true>(map, p, s, grid, stream);
  return p.zeros ? launch_sub<T, true, false>(map, p, s, grid, stream)
                 : launch_sub<T, false, false>(map, p, s, grid, stream);
}

}  // namespace

// Where the activations leave room for one block of 8 warps only, though they are of few columns (8
// tokens), instructions bound the kernel, and many units to a block are better off with the tensor
// cores.  (us of this / of int4_tile.cu, N = 11008, 32768; 8 tokens, K = 2048 8.2 / 9.2, 16.7 / 14.2,
// K = 4096 12.3 / 12.4, 25.9 / 23.8, K = 8192 19.0 / 19.0, 43.0 / 43.1; 6 tokens, K = 4096 11.5 / 12.4,
// 24.0 / 23.8; 4 tokens, K = 12288 24.4 / 25.1, 56.0 / 63.1.)
bool int4_stream_suits(int M, int N, int K, int group, int num_sms) {
  StreamPlan s;
  if (!plan_stream(M, K, group, s)) return false;
  return s.warps * s.per_sm > 8 || K / kChunkK >= kMany || N <= 8 * kUnitRows * num_sms;
}

cudaError_t launch_int4_stream(const Int4LinearArgs& a, int num_sms, cudaStream_t stream) {
  const Int4Weight& w = a.w;
  StreamPlan s;
  CUtensorMap map[2];  // boxes of a unit and of a pair
  if (!plan_stream(a.M, w.K, w.group, s) ||
      !encode_tmap_2d(&map[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K / 2, w.N, w.K / 2,
                      kChunkK / 2, kUnitRows) ||
      !encode_tmap_2d(&map[1], CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K / 2, w.N, w.K / 2,
                      kChunkK / 2, 2 * kUnitRows))
    return cudaErrorInvalidValue;
  StreamArgs p;
  p.X = a.X;
  p.scales = w.scales;
  p.zeros = w.zeros;
  p.bias = a.bias;
  p.Y = a.Y;
  p.status = a.status;
  p.M = a.M;
  p.N = w.N;
  p.K = w.K;
  p.group = w.group;
  p.groups = w.groups;
  p.units = static_cast<int>((static_cast<long long>(w.N) + kUnitRows - 1) / kUnitRows);
  p.chunks = (w.K + kChunkK - 1) / kChunkK;
  p.stages = s.stages;
  p.xstride = s.xstride;
  p.batch = s.batch;
  const int grid = p.units < num_sms * s.per_sm ? p.units : num_sms * s.per_sm;
  const int blocks = w.group == 32 ? 8 : w.group == 64 ? 4 : 2;  // groups in a chunk
  p.vector_groups = w.group <= 128 && w.groups % blocks == 0;
  return w.bf16 ? launch_typed<__nv_bfloat16>(map, p, s, grid, stream)
                : launch_typed<__half>(map, p, s, grid, stream);
}

}  // namespace i8mm
