// int4_stream.cu -- the product on 4-bit weights for up to 8 tokens: every byte of the weights is
// read once, at the rate of HBM.
//
//   Y[m,n] = T( sum_c s[n,c] ( sum_{k in c} u[n,k] X[m,k] - z[n,c] sum_{k in c} X[m,k] ) + bias[n] )
//
// Instructions, not bytes, are what such a kernel runs out of first (one SM must take in 56 weights
// a cycle to keep up with HBM), so the unpacking is what everything is arranged around:
//   - fp16: a code in the low bits of a 16-bit half is a subnormal, u 2^-24 (bits 0-3) or u 2^-20
//     (bits 4-7), which the tensor core multiplies exactly.  One AND gives two of them, so 8
//     weights cost 4 ANDs and a shift, and no conversion.  Two accumulators keep the two powers
//     apart and meet when a group is scaled: t = 16 lo + hi.
//   - bf16 has no subnormals to spare (their products would be below float32's range): a code set
//     into the mantissa of 128 reads as 128 + u, one AND-OR and a shift for two.
//   - The zero point (and the 128) is taken out afterwards, with the sum of the group's activations
//     that one more MMA against a constant gives in every row.
//   - m16n8k16 with the weights as the 16-row operand: the 8 tokens are its columns.  The packing
//     order puts neighbours into the two halves of a register, as X has them in memory; which k a
//     lane takes is free as long as both operands agree: lane t of a quad takes the words 4q + t.
// The group's scale meets the float32 sum of the group: the weights are never rounded.
//
// A block owns a range of 16-row units and takes them in pairs; its warps share the K axis in
// chunks of 256 columns, each warp with a ring of its own that TMA fills (boxes of 16 rows x 128
// bytes, 128-byte swizzle: the 32-bit reads of a quad's words hit 32 banks).  The first chunks are
// requested before the wait for the previous launch.  Partial sums of a pair meet in shared
// memory, in the order of the warps.
#include <type_traits>

#include "block.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace i8mm {

namespace {

constexpr int kMaxTok = 8;
constexpr int kUnitRows = 16;
constexpr int kChunkK = 256;                        // columns of a chunk: 128 bytes of a row
constexpr int kUnitBytes = kUnitRows * kChunkK / 2;
constexpr int kStageBytes = 2 * kUnitBytes;         // a pair of units
constexpr int kMaxWarps = 16, kMaxStages = 4;
constexpr size_t kSmemMost = 227 * 1024;

struct StreamArgs {
  const void* X;
  const void* scales;
  const uint8_t* zeros;
  const void* bias;
  void* Y;
  int32_t* status;
  int M, N, K, group, groups;
  int units, chunks, stages, xstride;
  bool vector_groups;  // load_groups: a chunk's groups of a row are one aligned vector
};

struct StreamShared {
  uint64_t full[kMaxWarps][kMaxStages];
  uint64_t x_full;
  int abort;
};

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

// Words a lane takes at once: of 32 kWords<SUB> columns, lane t of a quad takes those from
// 8 kWords t on (columns of one group only).
template <int SUB>
constexpr int kWords = SUB < 4 ? SUB : 4;

// One chunk of a pair of units (or of one, where not TWO) added to acc.  row: this lane's row g of
// the first unit in the stage, swz its swizzle (the row's number << 4) and x its activations at the
// chunk's start; src: the lane that holds row g's scales.
template <typename T, int SUB, bool ZP, bool TWO>
__device__ __forceinline__ void add_chunk(float (&acc)[2][4], const RowGroups<SUB>& rg, uint32_t row,
                                          uint32_t swz, uint32_t x, int t, int src) {
  constexpr bool kHalf = std::is_same<T, __half>::value;
  constexpr uint32_t kOne = kHalf ? 0x00100010u : 0x3F803F80u;  // 2^-20 or 1, twice
  constexpr int W = kWords<SUB>;
  const uint32_t x_t = x + 16u * W * t;
#pragma unroll
  for (int j = 0; j < 8 / SUB; ++j) {
    float lo[2][4], hi[2][4], sum[4];
#pragma unroll
    for (int e = 0; e < SUB / W; ++e) {
      const int k = (j * SUB + e * W) * 32;  // first column
      // bytes k/2 + 4 W t of the row, 16-byte pieces swizzled
      const uint32_t at = row + ((static_cast<uint32_t>(k / 2) + 4u * W * t) ^ swz);
      uint32_t wa[2][W], wb[2][W];
#pragma unroll
      for (int i = 0; i < (TWO ? 2 : 1); ++i) {
        lds<W>(wa[i], at + i * kUnitBytes);
        lds<W>(wb[i], at + i * kUnitBytes + 1024);
      }
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const bool first = e == 0 && w == 0;
        uint32_t xr[4];
        lds<4>(xr, x_t + 2u * k + 16u * w);
#pragma unroll
        for (int i = 0; i < (TWO ? 2 : 1); ++i) {
          const uint32_t a = wa[i][w], b = wb[i][w];
          if constexpr (kHalf) {
            // the activations' words lie in the order 0, 2, 1, 3
            const uint32_t a8 = a >> 8, b8 = b >> 8;
            mma_16x8x16<T>(lo[i], a & 0x000F000Fu, b & 0x000F000Fu, a8 & 0x000F000Fu,
                           b8 & 0x000F000Fu, xr[0], xr[1], first);
            mma_16x8x16<T>(hi[i], a & 0x00F000F0u, b & 0x00F000F0u, a8 & 0x00F000F0u,
                           b8 & 0x00F000F0u, xr[2], xr[3], first);
          } else {
            constexpr uint32_t k128 = 0x43004300u;
            mma_16x8x16<T>(lo[i], (a & 0x000F000Fu) | k128, (b & 0x000F000Fu) | k128,
                           (a >> 4 & 0x000F000Fu) | k128, (b >> 4 & 0x000F000Fu) | k128, xr[0],
                           xr[1], first);
            mma_16x8x16<T>(lo[i], (a >> 8 & 0x000F000Fu) | k128, (b >> 8 & 0x000F000Fu) | k128,
                           (a >> 12 & 0x000F000Fu) | k128, (b >> 12 & 0x000F000Fu) | k128, xr[2],
                           xr[3], false);
          }
        }
        mma_16x8x16<T>(sum, kOne, kOne, kOne, kOne, xr[0], xr[1], first);
        mma_16x8x16<T>(sum, kOne, kOne, kOne, kOne, xr[2], xr[3], false);
      }
    }
    // the block's scales: rows g and g + 8 of each unit
#pragma unroll
    for (int r = 0; r < (TWO ? 4 : 2); ++r) {
      const uint32_t sw = __shfl_sync(~0u, rg.s[j / 2], src + 8 * r);
      const float s = scale_value<T>(sw, j & 1);
      float z = kInt4Zero;
      if (ZP)
        z = static_cast<float>(__shfl_sync(~0u, rg.z[j / 4], src + 8 * r) >> (8 * (j & 3)) & 0xFFu);
      if (!kHalf) z += 128.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = r / 2, d = 2 * (r & 1) + h;
        const float v = kHalf ? fmaf(lo[i][d], 16.0f, hi[i][d]) : lo[i][d];
        acc[i][d] = fmaf(s, fmaf(-z, sum[h], v), acc[i][d]);
      }
    }
  }
}

}  // namespace

template <typename T, int SUB, bool ZP>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    int4_stream_kernel(const __grid_constant__ CUtensorMap map_w, const StreamArgs p) {
  extern __shared__ uint8_t stream_smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(stream_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warps = blockDim.x / 32;
  uint8_t* xs = ring + static_cast<size_t>(warps) * p.stages * kStageBytes;
  float* part = reinterpret_cast<float*>(xs + static_cast<size_t>(p.M) * p.xstride);
  StreamShared& S = *reinterpret_cast<StreamShared*>(part + 2 * warps * 32 * p.M);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int g = lane / 4, t = lane % 4;
  volatile int* abort = &S.abort;

  if (threadIdx.x == 0) {
    for (int w = 0; w < warps; ++w)
      for (int s = 0; s < p.stages; ++s) mbar_init(&S.full[w][s], 1);
    mbar_init(&S.x_full, 1);
    S.abort = 0;
    fence_mbarrier_init();
    prefetch_tmap(&map_w);
  }
  __syncthreads();
  grid_launch_dependents();

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
      tma_load_2d(&map_w, dst, &my_full[f_stage], fc * (kChunkK / 2), u * kUnitRows);
      if (two)
        tma_load_2d(&map_w, dst + kUnitBytes, &my_full[f_stage], fc * (kChunkK / 2),
                    (u + 1) * kUnitRows);
    }
    ++issued;
    if (++f_stage == p.stages) f_stage = 0;
    fc += warps;
    settle(fp, fc);
  };
  settle(fp, fc);
  int q = fp, c = fc;  // the next chunk to multiply
  for (int s = 0; s < p.stages; ++s) request();
  RowGroups<SUB> cur, nxt;
  if (q < pairs) load_groups<SUB, ZP>(nxt, p, (u0 + 2 * q) * kUnitRows + lane, c * kChunkK);

  grid_dependency_wait();
  if (threadIdx.x == 0) {
    const uint32_t row_bytes = static_cast<uint32_t>(p.K) * 2;
    mbar_arrive_expect_tx(&S.x_full, row_bytes * p.M);
    for (int m = 0; m < p.M; ++m)
      bulk_load(xs + static_cast<size_t>(m) * p.xstride,
                static_cast<const T*>(p.X) + static_cast<size_t>(m) * p.K, row_bytes, &S.x_full);
  }
  // zeros behind the rows, up to the end of the last chunk
  const int pad = p.chunks * kChunkK / 8 - p.K / 8;  // 16-byte pieces
  for (int i = threadIdx.x; i < pad * p.M; i += blockDim.x)
    *reinterpret_cast<uint4*>(xs + static_cast<size_t>(i / pad) * p.xstride + 2 * p.K + i % pad * 16) =
        make_uint4(0, 0, 0, 0);
  bool ok = __all_sync(~0u, mbar_wait_bounded(&S.x_full, 0, abort));
  if constexpr (std::is_same<T, __half>::value) {
    // The two operand words of an MMA are a register pair: the words 0 and 2 of 16 bytes (the low
    // nibbles' columns), then 1 and 3.
    for (int m = 0; m < p.M; ++m) {
      for (int i = threadIdx.x; i < p.K / 8; i += blockDim.x) {
        uint32_t* v = reinterpret_cast<uint32_t*>(xs + static_cast<size_t>(m) * p.xstride) + 4 * i;
        const uint32_t one = v[1], two = v[2];
        v[1] = two;
        v[2] = one;
      }
    }
  }
  __syncthreads();

  // Row g of an MMA is row `gr` of the unit, the bits of g reversed: the rows that read shared
  // memory together then differ in the swizzle's high bits (conflict-free for 4, 8 and 16 bytes).
  const int gr = (g & 1) << 2 | (g & 2) | g >> 2;
  // columns past the last token repeat it: their results are not kept
  const uint32_t x_lane = smem_addr(xs) + static_cast<uint32_t>(min(g, p.M - 1)) * p.xstride;
  const uint32_t w_lane = smem_addr(my_ring) + static_cast<uint32_t>(gr) * 128;
  int stage = 0;
  uint32_t phase = 0;
  for (int pair = 0; pair < pairs; ++pair) {
    float acc[2][4] = {};
    while (q == pair) {
      cur = nxt;
      int nq = q, nc = c + warps;
      settle(nq, nc);
      if (nq < pairs) load_groups<SUB, ZP>(nxt, p, (u0 + 2 * nq) * kUnitRows + lane, nc * kChunkK);
      if (ok) ok = __all_sync(~0u, mbar_wait_bounded(&my_full[stage], phase, abort));
      if (ok) {
        const uint32_t w = w_lane + static_cast<uint32_t>(stage) * kStageBytes;
        const uint32_t x = x_lane + 2u * kChunkK * c;
        if (u0 + 2 * pair + 1 < u1)
          add_chunk<T, SUB, ZP, true>(acc, cur, w, 16u * gr, x, t, gr);
        else
          add_chunk<T, SUB, ZP, false>(acc, cur, w, 16u * gr, x, t, gr);
      }
      __syncwarp();
      if (ok) request();
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      q = nq;
      c = nc;
    }
    // the pair's partial sums: [token][row] of each warp
    float* mine = part + ((pair & 1) * warps + warp) * 32 * p.M;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = 2 * t + h;
      if (m < p.M) {
#pragma unroll
        for (int r = 0; r < 4; ++r) mine[m * 32 + gr + 8 * r] = acc[r / 2][2 * (r & 1) + h];
      }
    }
    __syncthreads();
    const int row0 = (u0 + 2 * pair) * kUnitRows;
    const int row_end = min(p.N, u1 * kUnitRows);
    const float* all = part + (pair & 1) * warps * 32 * p.M;
    for (int i = threadIdx.x; i < 32 * p.M; i += blockDim.x) {
      const int n = row0 + (i & 31), m = i >> 5;
      if (n >= row_end) continue;
      float v = 0.0f;
      for (int w = 0; w < warps; ++w) v += all[w * 32 * p.M + i];
      if (std::is_same<T, __half>::value) v *= 1048576.0f;  // the sums are of 2^-20 u X
      if (p.bias) v += to_f32(static_cast<const T*>(p.bias)[n]);
      static_cast<T*>(p.Y)[static_cast<size_t>(m) * p.N + n] = from_f32<T>(v);
    }
  }
  if (!ok) {
    if (lane == 0 && p.status)
      atomicCAS(reinterpret_cast<int*>(p.status), 0, INT8MM_ERR_TIMEOUT);
    // what was requested lands before the block's shared memory is given back
    int dummy = 0;
    for (int j = issued > p.stages ? issued - p.stages : 0; j < issued; ++j)
      mbar_wait_bounded(&my_full[j % p.stages], static_cast<uint32_t>(j / p.stages) & 1u, &dummy);
  }
}

namespace {

struct StreamPlan {
  int warps, stages, xstride;
  size_t smem;
};

// Fits where the activations of all tokens leave room for two stages of 8 warps.
bool plan_stream(int M, int K, int group, StreamPlan& s) {
  if (M > kMaxTok) return false;
  // a row up to its last chunk's end, and a pad that sets the quads of two tokens apart (64 bytes
  // where a lane reads every fourth 16 bytes, otherwise 16)
  s.xstride = (K + kChunkK - 1) / kChunkK * kChunkK * 2 + (group == 32 ? 64 : 16);
  for (int warps = kMaxWarps; warps >= 8; warps /= 2) {
    const size_t fixed = 1024 + sizeof(StreamShared) + static_cast<size_t>(M) * s.xstride +
                         static_cast<size_t>(2) * warps * 32 * M * sizeof(float);
    for (int stages = kMaxStages; stages >= 2; --stages) {
      s.smem = fixed + static_cast<size_t>(warps) * stages * kStageBytes;
      if (s.smem <= kSmemMost) {
        s.warps = warps;
        s.stages = stages;
        return true;
      }
    }
  }
  return false;
}

template <typename T, int SUB, bool ZP>
cudaError_t launch_variant(const CUtensorMap& map, const StreamArgs& p, const StreamPlan& s,
                           int grid, cudaStream_t stream) {
  cudaError_t e = cudaFuncSetAttribute(int4_stream_kernel<T, SUB, ZP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemMost));
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
  return cudaLaunchKernelEx(&cfg, int4_stream_kernel<T, SUB, ZP>, map, p);
}

template <typename T, bool ZP>
cudaError_t launch_sub(const CUtensorMap& map, const StreamArgs& p, const StreamPlan& s, int grid,
                       cudaStream_t stream) {
  if (p.group == 32) return launch_variant<T, 1, ZP>(map, p, s, grid, stream);
  if (p.group == 64) return launch_variant<T, 2, ZP>(map, p, s, grid, stream);
  if (p.group % 256 == 0) return launch_variant<T, 8, ZP>(map, p, s, grid, stream);
  return launch_variant<T, 4, ZP>(map, p, s, grid, stream);
}

}  // namespace

bool int4_stream_fits(int M, int K, int group) {
  StreamPlan s;
  return plan_stream(M, K, group, s);
}

cudaError_t launch_int4_stream(const Int4LinearArgs& a, int num_sms, cudaStream_t stream) {
  const Int4Weight& w = a.w;
  StreamPlan s;
  CUtensorMap map;
  if (!plan_stream(a.M, w.K, w.group, s) ||
      !encode_tmap_2d(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K / 2, w.N, w.K / 2,
                      kChunkK / 2, kUnitRows))
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
  const int blocks = w.group == 32 ? 8 : w.group == 64 ? 4 : 2;  // groups in a chunk
  p.vector_groups = w.group <= 128 && w.groups % blocks == 0;
  const int grid = p.units < num_sms ? p.units : num_sms;
  if (w.bf16)
    return w.zeros ? launch_sub<__nv_bfloat16, true>(map, p, s, grid, stream)
                   : launch_sub<__nv_bfloat16, false>(map, p, s, grid, stream);
  return w.zeros ? launch_sub<__half, true>(map, p, s, grid, stream)
                 : launch_sub<__half, false>(map, p, s, grid, stream);
}

}  // namespace i8mm
