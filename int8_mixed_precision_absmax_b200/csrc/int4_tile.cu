// int4_tile.cu -- the product on 4-bit weights for more than a few tokens, on the tensor cores.
//
//   D[n, m] = sum_k W_hat[n,k] X[m,k],   Y[m,n] = T(D[n,m] + bias[n])
//
// One tile is 128 output channels (the MMA's rows) by `tn` tokens (its columns).  The weights never
// exist in 16 bits outside the SM: the dequantizing warps read the packed codes that TMA put into
// shared memory, make W_hat = T(s (u - z)) in registers (u - z is exact, so one rounding to T: the
// tensor core's operand type) and store it to tensor memory, from where tcgen05.mma takes its A
// operand; X comes through TMA as the B operand.  Sums are float32 in tensor memory.
//
// Roles: two teams of warps dequantize the steps of 128 k in turn and, after a tile's last, store its
// results; one warp issues TMA, one allocates tensor memory and issues the MMAs.  (Warps of their own
// for the results cost the dequantizing ones registers, whose lack made a third of their
// instructions moves of constants.)  Rings: `stages` steps of codes and X in shared memory,
// `a_stages` steps of W_hat in tensor memory.
//
// Few tiles: the K axis is split over the CTAs of a cluster, which leave their partial sums in
// shared memory; each CTA then adds up a slice of the tokens from all of them, in rank order.
//
// Measured, us: 2048 tokens of 4096 x 11008, groups of 128, 144 (1280 TFLOP/s, 77 % of the measured
// bf16 rate of the tensor cores alone; 165 in a long run under the power cap); 77 tokens of the same
// 15.0 (1.8 TB/s), 16 tokens 12.5, and of 12288 x 49152 107 (2.9 TB/s).  With many tokens the MMAs bound
// it, which read A from tensor memory while the dequantizing warps write it.  With few no pipe does: 16
// tokens of 12288 x 8192 issue an instruction in 54 % of a scheduler's active cycles, none of its pipes
// is above 40 %, and of 1830 instructions a step the dequantizing arithmetic (13 for 8 weights) is 832;
// what is left are the waits between the roles, once a step, with two or three steps of W_hat in tensor
// memory to cover them, and the start and joining of a cluster.
//
// Every wait on a barrier is bounded (ptx.cuh); a wait that gives up reports INT8MM_ERR_TIMEOUT, and the
// block drains its copies and MMAs, frees its tensor memory and exits.  The allocation of tensor memory
// waits without a bound; plan_tile sizes shared memory so that it need not wait for a kernel here.
#include <type_traits>

#include "block.cuh"
#include "kernels.cuh"
#include "ptx.cuh"

namespace i8mm {

namespace {

constexpr int kTileN = 128;   // channels per tile
constexpr int kStepK = 128;   // k per step
constexpr int kCodeBytes = kTileN * kStepK / 2;
constexpr int kTeams = 2;
__host__ __device__ constexpr int threads_of(int team_warps) { return (kTeams * team_warps + 2) * 32; }
constexpr int kMaxStages = 10, kMaxA = 4;
constexpr size_t kSmemMost = 226 * 1024;  // of an SM, for one block or for two
constexpr int kACols = kStepK / 2;  // tensor-memory columns of a step of W_hat

struct TileArgs {
  const void* scales;
  const uint8_t* zeros;
  const void* bias;
  void* Y;
  int32_t* status;
  int M, N, K, group, groups;
  int tn, stages, a_stages, tmem_cols, splits;
  int m_tiles, tiles, steps;
};

struct TileShared {  // behind the ring
  uint4 turn[kTeams * 8][8 * 32 * 2 / 16];  // of each dequantizing warp: 8 tokens x 32 channels
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t a_full[kMaxA], a_empty[kMaxA];
  uint64_t d_full, d_empty;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};

// tensor-memory columns of the accumulator
__host__ __device__ constexpr int acc_cols(int tn) { return (tn + 31) / 32 * 32; }
__host__ __device__ constexpr int stage_bytes(int tn) { return kCodeBytes + tn * kStepK * 2; }

// One lane of a converged warp, the same each time.  Where the rest of a step's code is the whole
// warp's, the MMAs' descriptors stay in uniform registers; issued from a branch on the lane's number
// the 8 of a step took 500 to 800 cycles, more than their 256 columns take to multiply.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(p));
  return p != 0;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, 16-bit operands, float32 sums.  Issued by one thread.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate ? 1u : 0u)
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ void report(int32_t* status) {
  if (status) atomicCAS(reinterpret_cast<int*>(status), 0, INT8MM_ERR_TIMEOUT);
}

// Every lane waits; the warp goes on together or gives up together (the tensor-memory accesses
// that follow are warp-wide).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(~0u, mbar_wait_bounded(bar, parity, abort));
}

// The scales and zero points of NG consecutive groups of a row, from group g (a multiple of NG) on.
// Groups past the row's end repeat the last one (their weights are not used).
template <int NG>
struct RowGroups {
  uint32_t s[(NG + 1) / 2], z;  // two scales, four zero points to a word
  __device__ __forceinline__ uint32_t scale2(int i) const {  // in both halves
    return __byte_perm(s[i / 2], s[i / 2], (i & 1) ? 0x3232 : 0x1010);
  }
  template <bool ZP>
  __device__ __forceinline__ uint32_t zero(int i) const {
    return ZP ? z >> (8 * i) & 0xFFu : static_cast<uint32_t>(kInt4Zero);
  }
};
template <int NG, bool ZP>
__device__ __forceinline__ void load_groups(RowGroups<NG>& r, const uint16_t* s, const uint8_t* z, int g,
                                            int groups) {
  if constexpr (NG == 1) {
    g = min(g, groups - 1);
    r.s[0] = s[g];
    r.z = ZP ? z[g] : 0;
  } else {
    if (groups % NG == 0) {  // every row starts on a whole vector
      g = min(g, groups - NG);
      if constexpr (NG == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(s + g);
        r.s[0] = v.x, r.s[1] = v.y;
        if (ZP) r.z = *reinterpret_cast<const uint32_t*>(z + g);
      } else {
        r.s[0] = *reinterpret_cast<const uint32_t*>(s + g);
        if (ZP) r.z = *reinterpret_cast<const uint16_t*>(z + g);
      }
      return;
    }
    r.s[0] = r.s[NG / 4] = r.z = 0;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int at = min(g + i, groups - 1);
      r.s[i / 2] |= static_cast<uint32_t>(s[at]) << (16 * (i & 1));
      if (ZP) r.z |= static_cast<uint32_t>(z[at]) << (8 * i);
    }
  }
}

template <typename T>
__host__ __device__ constexpr uint32_t tile_idesc(int n) {
  return idesc_f16_f32(kTileN, n) | (sizeof(T) && std::is_same<T, __nv_bfloat16>::value
                                         ? (1u << 7) | (1u << 10)
                                         : 0u);
}

}  // namespace

// TW warps dequantize a step: 4 where two blocks share an SM, each warp all of a step's k for its 32
// channels; 8 where a block has the SM to itself, each half of them.
// GROUP: 32, 64, or 128 for all multiples of 128; ZP: zero points are given.
template <typename T, int TW, int GROUP, bool ZP>
__global__ void __launch_bounds__(threads_of(TW), TW == 4 ? 2 : 1)
    int4_tile_kernel(const __grid_constant__ CUtensorMap map_x,
                     const __grid_constant__ CUtensorMap map_w, const TileArgs p) {
  extern __shared__ uint8_t tile_smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(tile_smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int sbytes = stage_bytes(p.tn);
  TileShared& S = *reinterpret_cast<TileShared*>(ring + p.stages * sbytes);
  constexpr int kDequantWarps = kTeams * TW;
  constexpr int kTmaWarp = kDequantWarps, kMmaWarp = kTmaWarp + 1;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&S.full[s], 1);
      mbar_init(&S.empty[s], 1);
    }
    for (int s = 0; s < p.a_stages; ++s) {
      mbar_init(&S.a_full[s], TW);
      mbar_init(&S.a_empty[s], 1);
    }
    mbar_init(&S.d_full, 1);
    mbar_init(&S.d_empty, kDequantWarps);
    mbar_init(&S.drain, 1);
    S.abort = 0;
    fence_mbarrier_init();
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&map_x);
    prefetch_tmap(&map_w);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&S.tmem_base, static_cast<uint32_t>(p.tmem_cols));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_launch_dependents();

  const uint32_t tmem = S.tmem_base;
  const uint32_t a_base = tmem + static_cast<uint32_t>(acc_cols(p.tn));
  volatile int* abort = &S.abort;
  // tiles t0, t0 + dt, ...; this CTA's part of the steps of each
  const int split = p.splits > 1 ? static_cast<int>(blockIdx.x) % p.splits : 0;
  const int t0 = static_cast<int>(blockIdx.x) / p.splits, dt = static_cast<int>(gridDim.x) / p.splits;
  const int k_begin = static_cast<int>(static_cast<long long>(p.steps) * split / p.splits);
  const int k_end = static_cast<int>(static_cast<long long>(p.steps) * (split + 1) / p.splits);
  bool ok = true;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int t = t0; ok && t < p.tiles; t += dt) {
        const int m0 = t % p.m_tiles * p.tn, n0 = t / p.m_tiles * kTileN;
        for (int k = k_begin; k < k_end; ++k) {
          if (!wait_asleep(&S.empty[stage], phase ^ 1u, abort, 20)) { ok = false; break; }
          uint8_t* dst = ring + stage * sbytes;
          mbar_arrive_expect_tx(&S.full[stage], static_cast<uint32_t>(sbytes));
          tma_load_2d(&map_w, dst, &S.full[stage], k * (kStepK / 2), n0);
          tma_load_2d(&map_x, dst + kCodeBytes, &S.full[stage], k * kStepK, m0);
          tma_load_2d(&map_x, dst + kCodeBytes + p.tn * 128, &S.full[stage], k * kStepK + 64, m0);
          ++issued;
          if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        }
      }
      int dummy = 0;  // every copy lands before the block can exit
      for (int j = issued > p.stages ? issued - p.stages : 0; j < issued; ++j)
        mbar_wait_bounded(&S.full[j % p.stages], static_cast<uint32_t>(j / p.stages) & 1u, &dummy);
      if (!ok) report(p.status);
    }
  } else if (warp == kMmaWarp) {
    const uint32_t idesc = tile_idesc<T>(p.tn);
    const uint64_t b0 = sw128_kmajor_desc(smem_addr(ring + kCodeBytes));  // of stage 0; in 16 bytes:
    const uint32_t b_stage = static_cast<uint32_t>(sbytes) >> 4, b_half = static_cast<uint32_t>(p.tn) * 8;
    int stage = 0, as = 0;
    uint32_t phase = 0, a_phase = 0, d_phase = 0;
    for (int t = t0; ok && t < p.tiles; t += dt) {
      if (!warp_wait(&S.d_empty, d_phase ^ 1u, abort)) { ok = false; break; }
      d_phase ^= 1u;
      tc_fence_after();
      for (int k = k_begin; k < k_end; ++k) {
        if (!warp_wait(&S.full[stage], phase, abort) || !warp_wait(&S.a_full[as], a_phase, abort)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a = a_base + static_cast<uint32_t>(as * kACols);
        const uint64_t b = b0 + static_cast<uint32_t>(stage) * b_stage;
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < kStepK / 16; ++j)
            mma_ts(tmem, a + 8u * j, b + (j / 4) * b_half + (j % 4) * 2, idesc, k > k_begin || j > 0);
          mma_commit(&S.empty[stage]);
          mma_commit(&S.a_empty[as]);
        }
        __syncwarp();
        if (++stage == p.stages) { stage = 0; phase ^= 1u; }
        if (++as == p.a_stages) { as = 0; a_phase ^= 1u; }
      }
      if (!ok) break;
      if (elect_one()) mma_commit(&S.d_full);
      __syncwarp();
    }
    if (elect_one()) mma_commit(&S.drain);  // every MMA is done before tensor memory is freed
    __syncwarp();
    int dummy = 0;
    mbar_wait_bounded(&S.drain, 0, &dummy);
    if (!ok && lane == 0) report(p.status);
  } else if (warp < kDequantWarps) {
    constexpr int kChunks = TW == 4 ? 4 : 2;  // of 32 k: 16 bytes of a row's codes
    const int quad = warp & 3, first = TW == 4 ? 0 : (warp >> 2 & 1) * kChunks, team = warp / TW;
    const int row = quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t swz = static_cast<uint32_t>((row >> 1) & 3);  // of the 64-byte swizzle
    constexpr int NG = GROUP / 32 < kChunks ? kChunks * 32 / GROUP : 1;  // groups of a warp's part
    const int g_steps = GROUP == 128 ? p.group / kStepK : 1;
    const bool odd_stages = p.stages % kTeams != 0;
    // the teams take the steps in turn, on from tile to tile; the rings' places of this team's next
    int stage = team, as = team, skip = team;  // skip: of a tile's steps before it
    uint32_t phase = 0, a_phase = 0, d_phase = 0;
    for (int t = t0; ok && t < p.tiles; t += dt) {
      const long long n = min(t / p.m_tiles * kTileN + row, p.N - 1);
      const uint16_t* srow = static_cast<const uint16_t*>(p.scales) + n * p.groups;
      const uint8_t* zrow = ZP ? p.zeros + n * p.groups : nullptr;
      int k = k_begin + skip;
      // groups of this part of step k; long ones last g_steps steps, g_left more from step k on
      int g = GROUP == 128 ? k / g_steps : k * (kStepK / GROUP) + first * 32 / GROUP;
      int g_left = g_steps - k % g_steps;
      RowGroups<NG> next;
      load_groups<NG, ZP>(next, srow, zrow, g, p.groups);
      for (; k < k_end; k += kTeams) {
        const int s_now = stage, a_now = as;
        const uint32_t ph_now = phase, a_ph_now = a_phase;
        if ((stage += kTeams) >= p.stages) { stage -= p.stages; phase ^= 1u; }
        if ((as += kTeams) >= p.a_stages) { as -= p.a_stages; a_phase ^= 1u; }
        const RowGroups<NG> now = next;
        if (GROUP == 128) {
          for (g_left -= kTeams; g_left <= 0; g_left += g_steps) ++g;
        } else {
          g += kTeams * (kStepK / GROUP);
        }
        if (k + kTeams < k_end) load_groups<NG, ZP>(next, srow, zrow, g, p.groups);
        // Where the stage's last step was the other team's: only once that has been multiplied is the
        // barrier's phase the one before this step's.
        if (odd_stages && !warp_wait(&S.empty[s_now], ph_now ^ 1u, abort)) { ok = false; break; }
        if (!warp_wait(&S.full[s_now], ph_now, abort)) { ok = false; break; }
        const uint8_t* codes = ring + s_now * sbytes;
        const uint32_t to = a_base + static_cast<uint32_t>(a_now * kACols + first * 16) + lane_base;
        Int4Values<T> q;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (c * 32 % GROUP == 0) q.set(now.scale2(c * 32 / GROUP), now.template zero<ZP>(c * 32 / GROUP));
          const uint4 w = *reinterpret_cast<const uint4*>(codes + row * 64 + ((first + c) ^ swz) * 16);
          uint32_t out[16];
          q.template word<true>(w.x, out);
          q.template word<true>(w.y, out + 4);
          q.template word<true>(w.z, out + 8);
          q.template word<true>(w.w, out + 12);
          if (c == 0) {
            if (!warp_wait(&S.a_empty[a_now], a_ph_now ^ 1u, abort)) { ok = false; break; }
            tc_fence_after();
          }
          tmem_st16(to + 16 * c, out);
        }
        if (!ok) break;
        // Past the row's end, where the codes' place is filled with zeros, (0 - z) times the scale may be
        // an infinity, and X's 0 times that a NaN: zeros in its place.  (16 tokens of 12288 x 49152, us:
        // 109 without, 110 so, 115 with a test of each chunk, 120 where the MMAs stopped at the row's end.)
        const int chunks = p.K / 32 - k * (kStepK / 32) - first;
        if (chunks < kChunks) {
          const uint32_t none[16] = {};
          tmem_st_wait();
          for (int c = max(chunks, 0); c < kChunks; ++c) tmem_st16(to + 16 * c, none);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.a_full[a_now]);
      }
      if (!ok) break;
      skip = k - k_end;

      // The tile's results: this warp's 32 channels, every (warps / 4)th 16 of the tokens.
      if (!__all_sync(~0u, wait_asleep(&S.d_full, d_phase, abort, 20))) { ok = false; break; }
      d_phase ^= 1u;
      tc_fence_after();
      const int m0 = t % p.m_tiles * p.tn, n_lane = t / p.m_tiles * kTileN + row;
      const bool n_ok = n_lane < p.N, vectors = p.N % 8 == 0;
      const float b = (p.bias && n_ok) ? to_f32(static_cast<const T*>(p.bias)[n_lane]) : 0.0f;
      float* part = reinterpret_cast<float*>(ring);  // splits > 1: the ring is drained
      T* Y = static_cast<T*>(p.Y);
      T* turned = reinterpret_cast<T*>(S.turn[warp]);
      for (int c = warp / 4 * 16; c < p.tn; c += kDequantWarps / 4 * 16) {
        uint32_t r[16];
        __syncwarp();
        tmem_ld16(tmem + static_cast<uint32_t>(c) + lane_base, r);
        tmem_ld_wait();
        if (p.splits > 1) {
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(c + j) * kTileN + row] = __uint_as_float(r[j]);
        } else if (vectors) {
          // a lane has one channel of 16 tokens: through shared memory to 8 channels of one token
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              turned[j * 32 + lane] = from_f32<T>(__uint_as_float(r[8 * i + j]) + b);
            __syncwarp();
            const long long m = m0 + c + 8 * i + lane / 4;
            const int n8 = n_lane - lane + lane % 4 * 8;
            if (m < p.M && n8 < p.N)
              *reinterpret_cast<uint4*>(Y + m * p.N + n8) =
                  *reinterpret_cast<const uint4*>(turned + lane / 4 * 32 + lane % 4 * 8);
          }
        } else if (n_ok) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const long long m = m0 + c + j;
            if (m < p.M) Y[m * p.N + n_lane] = from_f32<T>(__uint_as_float(r[j]) + b);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.d_empty);
    }
    if (!ok) report(p.status);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, static_cast<uint32_t>(p.tmem_cols));
  }
  if (p.splits > 1) {
    // one tile per cluster: every CTA's partial sums are in its shared memory
    __syncwarp();
    cluster_barrier_sync();
    if (!S.abort) {
      const int m0 = t0 % p.m_tiles * p.tn, n0 = t0 / p.m_tiles * kTileN;
      // 4 channels of a token at a time
      const int c_begin = p.tn * split / p.splits, c_end = p.tn * (split + 1) / p.splits;
      constexpr int kRow = kTileN / 4;
      uint32_t base[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) base[r] = r < p.splits ? mapa_shared(smem_addr(ring), r) : 0;
      for (int i = c_begin * kRow + static_cast<int>(threadIdx.x); i < c_end * kRow; i += threads_of(TW)) {
        const long long m = m0 + i / kRow;
        const int n = n0 + i % kRow * 4;
        if (m >= p.M || n >= p.N) continue;
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < p.splits) v[r] = ld_cluster_f32x4(base[r] + 16u * i);
#pragma unroll
        for (int r = 1; r < 8; ++r) {
          if (r < p.splits) {
            v[0].x += v[r].x;
            v[0].y += v[r].y;
            v[0].z += v[r].z;
            v[0].w += v[r].w;
          }
        }
        const float f[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
        T* y = static_cast<T*>(p.Y) + m * p.N + n;
        const T* bias = static_cast<const T*>(p.bias) + n;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < p.N) y[e] = from_f32<T>(f[e] + (p.bias ? to_f32(bias[e]) : 0.0f));
      }
    }
    __syncwarp();
    cluster_barrier_sync();  // no CTA leaves while its sums are read
  }
}

namespace {

struct TilePlan {
  int tn, stages, a_stages, tmem_cols, splits, team_warps, grid;
  size_t smem;
};

TilePlan plan_tile(int M, int N, int K, int num_sms) {
  TilePlan t;
  const int n_tiles = (N + kTileN - 1) / kTileN;
  const int steps = (K + kStepK - 1) / kStepK;
  if (M <= 128) {
    t.tn = (M + 15) / 16 * 16;
  } else {
    // The width that needs the least time: waves of one tile per SM, each of a time that grows with
    // tn + 90 (2048 x 11008 x 4096: 146 us in 5 waves of 256, 167 in 7 of 192, 169 in tiles of 128, two to an SM).
    t.tn = 256;
    long long best = -1;
    for (int tn = 256; tn > 128; tn -= 16) {
      const long long tiles = static_cast<long long>((M + tn - 1) / tn) * n_tiles;
      const long long cost = (tiles + num_sms - 1) / num_sms * (tn + 90);
      if (best < 0 || cost < best) best = cost, t.tn = tn;
    }
  }
  const long long tiles = static_cast<long long>((M + t.tn - 1) / t.tn) * n_tiles;
  const int per_sm = t.tn <= 128 ? 2 : 1;
  const int capacity = num_sms * per_sm;
  t.splits = 1;
  if (tiles < capacity) {
    const int want = static_cast<int>(capacity / tiles);
    const int most = steps / 2 > 1 ? steps / 2 : 1;  // two steps or more each
    t.splits = want < 8 ? want : 8;
    if (t.splits > most) t.splits = most;
    if (t.splits < 1) t.splits = 1;
  }
  t.tmem_cols = per_sm == 2 ? 256 : 512;
  t.team_warps = per_sm == 2 ? 4 : 8;
  t.a_stages = (t.tmem_cols - acc_cols(t.tn)) / kACols;
  if (t.a_stages > kMaxA) t.a_stages = kMaxA;
  const size_t budget = kSmemMost / per_sm - 1024 - sizeof(TileShared);
  t.stages = static_cast<int>(budget / stage_bytes(t.tn));
  if (t.stages > kMaxStages) t.stages = kMaxStages;
  t.smem = static_cast<size_t>(t.stages) * stage_bytes(t.tn) + sizeof(TileShared) + 1024;
  // Where these blocks hold all of an SM's tensor memory, they leave less shared memory than any other
  // kernel with tensor memory needs (33 KB): none waits on the SM for tensor memory that a cluster here
  // will not give back before its blocks elsewhere have got theirs.
  const size_t least = static_cast<size_t>(200 * 1024 / per_sm);
  if (t.smem < least) t.smem = least;
  t.grid = t.splits > 1 ? static_cast<int>(tiles) * t.splits
                        : static_cast<int>(tiles < capacity ? tiles : capacity);
  return t;
}

using TileKernel = void (*)(const CUtensorMap, const CUtensorMap, const TileArgs);

template <typename T, int TW, int GROUP, bool ZP>
cudaError_t ready(TileKernel& kernel) {
  static std::atomic<unsigned long long> allowed{0};
  kernel = int4_tile_kernel<T, TW, GROUP, ZP>;
  return allow_smem(reinterpret_cast<const void*>(kernel), kSmemMost, allowed);
}
template <typename T, int TW, bool ZP>
cudaError_t kernel_of_group(int group, TileKernel& kernel) {
  return group == 32 ? ready<T, TW, 32, ZP>(kernel)
                     : group == 64 ? ready<T, TW, 64, ZP>(kernel) : ready<T, TW, 128, ZP>(kernel);
}
template <typename T>
cudaError_t kernel_of(int team_warps, int group, bool zeros, TileKernel& kernel) {
  if (team_warps == 8)
    return zeros ? kernel_of_group<T, 8, true>(group, kernel) : kernel_of_group<T, 8, false>(group, kernel);
  return zeros ? kernel_of_group<T, 4, true>(group, kernel) : kernel_of_group<T, 4, false>(group, kernel);
}

template <typename T>
cudaError_t launch_typed(const Int4LinearArgs& a, int num_sms, cudaStream_t stream) {
  const Int4Weight& w = a.w;
  const TilePlan t = plan_tile(a.M, w.N, w.K, num_sms);
  CUtensorMap map_x, map_w;
  if (!encode_tmap_2d(&map_x,
                      w.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      a.X, w.K, a.M, static_cast<uint64_t>(w.K) * 2, 64,
                      static_cast<uint32_t>(t.tn)) ||
      !encode_tmap_2d(&map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K / 2, w.N, w.K / 2,
                      kStepK / 2, kTileN, CU_TENSOR_MAP_SWIZZLE_64B))
    return cudaErrorInvalidValue;
  TileArgs p;
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
  p.tn = t.tn;
  p.stages = t.stages;
  p.a_stages = t.a_stages;
  p.tmem_cols = t.tmem_cols;
  p.splits = t.splits;
  p.m_tiles = (a.M + t.tn - 1) / t.tn;
  const long long tiles = static_cast<long long>(p.m_tiles) * ((w.N + kTileN - 1) / kTileN);
  if (tiles > 0x7FFFFFFF / 8) return cudaErrorInvalidValue;
  p.tiles = static_cast<int>(tiles);
  p.steps = (w.K + kStepK - 1) / kStepK;
  TileKernel kernel = nullptr;
  const cudaError_t e = kernel_of<T>(t.team_warps, w.group, w.zeros != nullptr, kernel);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(t.grid);
  cfg.blockDim = dim3(threads_of(t.team_warps));
  cfg.dynamicSmemBytes = t.smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = t.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = t.splits > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, map_x, map_w, p);
}

}  // namespace

cudaError_t launch_int4_tile(const Int4LinearArgs& a, int num_sms, cudaStream_t stream) {
  return a.w.bf16 ? launch_typed<__nv_bfloat16>(a, num_sms, stream)
                  : launch_typed<__half>(a, num_sms, stream);
}

}  // namespace i8mm
