// bsgg_linear_kernel.cuh -- the dense products of the layer and its gradient on
// tcgen05 (bf16 or f16 operands, fp32 accumulators in tensor memory).
//
//   C[j, i] = sum_r P(i, r) Q(j, r),   out[j * ld + i] = act(C + bias_i) + residual
//
// P is the operand whose index i is the output's contiguous one; it takes the
// matrix instruction's M side, so that a tensor-memory lane is an output column
// and a warp writes 32 consecutive values of one output row.  That holds for all
// three products, and for few output rows (decode) the instruction's short side
// N is theirs:
//   forward  y  (m, n): P = W (n, k),         Q = x (m, k)
//   gradient dx (m, k): P = W^T (k, n),       Q = dz (m, n)
//            dw (n, k): P = x^T (k, m),       Q = dz^T (n, m)
// An operand whose reduction index r is its contiguous one is K-major, the
// others are MN-major: both are 64 x 64 boxes under the 128-byte swizzle, only
// the descriptor and the box's sides differ.
#pragma once

#include "bsgg_ops.cuh"

namespace bsgg {

constexpr int kLinDepth = 64;                 // reduction length of a stage: 128 bytes
constexpr int kLinEpiWarps = 8;
constexpr int kLinChunk = 16;                 // output rows an epilogue warp finishes at a time
constexpr int kLinThreads = 32 * (2 + kLinEpiWarps);

struct LinParams {
  int32_t cols, rows;         // i < cols, j < rows
  int32_t k_blocks;           // ceil(depth / 64)
  int32_t p_tiles, q_tiles;
  int32_t p_mn, q_mn;         // MN-major operands
  uint32_t idesc;
  int32_t act, in_kind, out_kind, bias_kind, residual_kind;
  const void* bias;
  const void* residual;
  void* out;
  void* z;
  int64_t ld_residual, ld_out, ldz;
  uint32_t* status;
  uint64_t wait_limit_ns;
};

// act(z).  silu = z / (1 + e^-z); gelu = z Phi(z) with Phi from normcdff,
// which keeps its relative accuracy in the lower tail where 1 + erf cancels.
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == BSGG_ACT_RELU) return z <= 0.0f ? 0.0f : z;               // a NaN stays
  if (ACT == BSGG_ACT_SRELU) return z <= 0.0f ? 0.0f : z * z;
  if (ACT == BSGG_ACT_SILU) return z / (1.0f + expf(-z));
  if (ACT == BSGG_ACT_GELU) return z * normcdff(z);
  return z;
}

// 128-byte-swizzled MN-major operand tile: 64-element (128-byte) rows, one per
// reduction index, groups of 8 of them 1024 bytes apart (stride offset), blocks
// of 64 elements along the tile's rows 8192 bytes apart (leading offset).
__device__ __forceinline__ uint64_t sdesc_mnmajor_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// CH values of output column i, rows j0 .. j0 + CH - 1.
template <int CH, int ACT>
__device__ __forceinline__ void lin_finish_act(const LinParams& p, float (&v)[CH], int i, int j0, int nj, float bias) {
  float r[CH];
  if (p.residual != nullptr) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      r[c] = c < nj ? load1(p.residual_kind, p.residual, (j0 + c) * p.ld_residual + i) : 0.0f;
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) v[c] += bias;
  if (p.z != nullptr) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (c < nj) store1(p.in_kind, p.z, (j0 + c) * p.ldz + i, v[c]);
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    v[c] = act_value<ACT>(v[c]);
    if (p.residual != nullptr) v[c] += r[c];
  }
#pragma unroll
  for (int c = 0; c < CH; ++c)
    if (c < nj) store1(p.out_kind, p.out, (j0 + c) * p.ld_out + i, v[c]);
}
template <int CH>
__device__ __forceinline__ void lin_finish(const LinParams& p, float (&v)[CH], int i, int j0, float bias) {
  const int nj = p.rows - j0;
  if (i >= p.cols || nj <= 0) return;
  switch (p.act) {
    case BSGG_ACT_RELU: lin_finish_act<CH, BSGG_ACT_RELU>(p, v, i, j0, nj, bias); break;
    case BSGG_ACT_SRELU: lin_finish_act<CH, BSGG_ACT_SRELU>(p, v, i, j0, nj, bias); break;
    case BSGG_ACT_SILU: lin_finish_act<CH, BSGG_ACT_SILU>(p, v, i, j0, nj, bias); break;
    case BSGG_ACT_GELU: lin_finish_act<CH, BSGG_ACT_GELU>(p, v, i, j0, nj, bias); break;
    default: lin_finish_act<CH, BSGG_ACT_NONE>(p, v, i, j0, nj, bias); break;
  }
}
__device__ __forceinline__ float lin_bias(const LinParams& p, int i) {
  return p.bias != nullptr && i < p.cols ? load1(p.bias_kind, p.bias, i) : 0.0f;
}

// One stage's box loads of an operand tile of ROWS rows from row r0 at
// reduction block kb.
template <int ROWS, bool PAIR>
__device__ __forceinline__ void lin_load(uint32_t dst, const CUtensorMap* map, uint32_t bar, bool mn, int r0, int kb) {
  if (!mn) {
    if (PAIR) tma_load_2d_pair(dst, map, bar, kb * kLinDepth, r0);
    else tma_load_2d(dst, map, bar, kb * kLinDepth, r0);
  } else {
#pragma unroll
    for (int b = 0; b < ROWS / 64; ++b) {
      if (PAIR) tma_load_2d_pair(dst + 8192 * b, map, bar, r0 + 64 * b, kb * kLinDepth);
      else tma_load_2d(dst + 8192 * b, map, bar, r0 + 64 * b, kb * kLinDepth);
    }
  }
}

// ---------------------------------------------------------------- CTA pairs
// 256 x 256 tiles, persistent, two accumulators: the epilogue of one tile runs
// under the products of the next.
struct LinPair {
  static constexpr int kStages = 6;
  static constexpr int kOpBytes = 128 * 128;               // this CTA's 128 rows of either operand
  static constexpr int kOffP = 0, kOffQ = kStages * kOpBytes;
  static constexpr int kOffBars = 2 * kStages * kOpBytes;
  static constexpr int kNumBars = 2 * kStages + 4 + 1;
  static constexpr int kOffHolder = kOffBars + 8 * kNumBars;
  static constexpr int kOffAbort = kOffHolder + 4;
  static constexpr int kSmem = kOffAbort + 4 + 1024;
};

// Tile order: bands of 8 tiles along q, every p of a band before the next, so
// that the pairs at work share operands in L2.
__device__ __forceinline__ void lin_tile(int t, int p_tiles, int q_tiles, int& tp, int& tq) {
  constexpr int kBand = 8;
  const int per = kBand * p_tiles;
  const int band = t / per, in = t % per;
  const int w = min(kBand, q_tiles - band * kBand);
  tp = in / w;
  tq = band * kBand + in % w;
}

static __global__ void __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ LinParams p) {
  using Ly = LinPair;
  constexpr int S = Ly::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Ly::kOffBars;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto accf_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto acce_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + Ly::kOffHolder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly::kOffAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int unit = blockIdx.x >> 1, units = gridDim.x >> 1;
  const int tiles = p.p_tiles * p.q_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full_bar(s), 1); mbar_init(empty_bar(s), 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(accf_bar(a), 1); mbar_init(acce_bar(a), 2 * kLinEpiWarps); }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
    prefetch_tmap(&tmP);
    prefetch_tmap(&tmQ);
  }
  if (warp == 1) { tmem_alloc_pair(smem_u32(holder), 512); tmem_relinquish_pair(); }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *holder;

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      bool ok = true, any = false;
      for (int t = unit; t < tiles && ok; t += units) {
        int tp, tq;
        lin_tile(t, p.p_tiles, p.q_tiles, tp, tq);
        const int p0 = tp * 256 + static_cast<int>(rank) * 128, q0 = tq * 256 + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(empty_bar(st), phase ^ 1u, abort_flag, p.wait_limit_ns)) { ok = false; break; }
          // both CTAs' bytes complete the even CTA's barrier
          const uint32_t fb = full_bar(st), fbl = mapa_shared(fb, 0);
          if (leader) mbar_expect_tx(fb, 4u * Ly::kOpBytes);
          lin_load<128, true>(sbase + Ly::kOffP + st * Ly::kOpBytes, &tmP, fbl, p.p_mn, p0, kb);
          lin_load<128, true>(sbase + Ly::kOffQ + st * Ly::kOpBytes, &tmQ, fbl, p.q_mn, q0, kb);
          any = true;
          if (++st == S) { st = 0; phase ^= 1u; }
        }
      }
      // the last use of every stage was released: nothing still targets this
      // CTA's shared memory when the CTAs part
      for (int i = 0; i < S && ok; ++i) {
        if (!mbar_wait(empty_bar(st), phase ^ 1u, abort_flag, p.wait_limit_ns)) { ok = false; break; }
        if (++st == S) { st = 0; phase ^= 1u; }
      }
      if (!ok) {
        if (p.status != nullptr) atomicOr(p.status, kStatusTimeout);
        // loads in flight complete barriers of the even CTA: wait out the drain bound
        const uint64_t t0 = globaltimer_ns();
        while (any && globaltimer_ns() - t0 < kDrainLimitNs) {}
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (lane == 0 && leader) {
      int st = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t pd0 = p.p_mn ? sdesc_mnmajor_sw128(sbase + Ly::kOffP) : sdesc_kmajor_sw128(sbase + Ly::kOffP);
      const uint64_t qd0 = p.q_mn ? sdesc_mnmajor_sw128(sbase + Ly::kOffQ) : sdesc_kmajor_sw128(sbase + Ly::kOffQ);
      // 16 reduction indices: 32 bytes inside a K-major row, 16 rows of 128 bytes MN-major
      const uint64_t pstep = p.p_mn ? 2048 >> 4 : 32 >> 4, qstep = p.q_mn ? 2048 >> 4 : 32 >> 4;
      for (int t = unit; t < tiles && ok; t += units) {
        if (!mbar_wait(acce_bar(acc), acc_phase ^ 1u, abort_flag, p.wait_limit_ns)) { ok = false; break; }
        tc_fence_after();
        const uint32_t d = tmem + acc * 256;
        for (int kb = 0; kb < p.k_blocks; ++kb) {
          if (!mbar_wait(full_bar(st), phase, abort_flag, p.wait_limit_ns)) { ok = false; break; }
          tc_fence_after();
          const uint64_t pd = pd0 + static_cast<uint64_t>((st * Ly::kOpBytes) >> 4);
          const uint64_t qd = qd0 + static_cast<uint64_t>((st * Ly::kOpBytes) >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_bf16_pair(d, pd + kk * pstep, qd + kk * qstep, p.idesc, (kb | kk) != 0 ? 1u : 0u);
          tc_commit_pair(empty_bar(st), 3);
          if (++st == S) { st = 0; phase ^= 1u; }
        }
        if (!ok) break;
        tc_commit_pair(accf_bar(acc), 3);
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
      }
      if (!ok) {
        if (p.status != nullptr) atomicOr(p.status, kStatusTimeout);
        tc_commit_pair(drain_bar, 1);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < kDrainLimitNs) {}
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;         // lane quadrant, columns [128 half, + 128)
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = unit; t < tiles; t += units) {
      int tp, tq;
      lin_tile(t, p.p_tiles, p.q_tiles, tp, tq);
      const int i = tp * 256 + static_cast<int>(rank) * 128 + q * 32 + lane;
      const float bias = lin_bias(p, i);
      if (!__all_sync(0xffffffffu, mbar_wait(accf_bar(acc), acc_phase, abort_flag, p.wait_limit_ns))) {
        if (lane == 0 && p.status != nullptr) atomicOr(p.status, kStatusTimeout);
        break;
      }
      tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + acc * 256 + half * 128;
#pragma unroll 1
      for (int c = 0; c < 128; c += kLinChunk) {
        float v[kLinChunk];
        tmem_ld16(ta + c, reinterpret_cast<uint32_t*>(v));
        tmem_wait_ld();
        if (c == 128 - kLinChunk) {
          // every column is in registers or stored: hand the accumulator back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(acce_bar(acc), 0));
        }
        lin_finish<kLinChunk>(p, v, i, tq * 256 + half * 128 + c, bias);
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------- single CTAs
// One 128 x BN tile per CTA, two CTAs per SM; with a cluster of S CTAs the
// reduction is split into S runs of blocks, whose partial tiles are added in
// order of rank through distributed shared memory, every CTA finishing BN / S of
// the output rows.
template <int BN>
struct LinTile {
  static constexpr int kPBytes = 128 * 128, kQBytes = BN * 128;
  static constexpr int kStageBytes = kPBytes + kQBytes;
  static constexpr int kStages = 110 * 1024 / kStageBytes;
  static constexpr int kOffP = 0, kOffQ = kStages * kPBytes;
  static constexpr int kOffBars = kStages * kStageBytes;
  static constexpr int kOffHolder = kOffBars + 8 * (2 * kStages + 1);
  static constexpr int kOffAbort = kOffHolder + 4;
  static constexpr int kSmem = kOffAbort + 4 + 1024;
  static_assert(kStages * kStageBytes >= 128 * BN * 4, "the partial tile reuses the stages");
};

template <int BN>
__global__ void __launch_bounds__(kLinThreads, 2)
    linear_tile_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ LinParams p, int split) {
  using Ly = LinTile<BN>;
  constexpr int S = Ly::kStages;
  constexpr uint32_t kCols = BN;                     // tensor-memory columns, a power of two >= 32
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + Ly::kOffBars;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  const uint32_t accf_bar = bar0 + 8u * (2 * S);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + Ly::kOffHolder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Ly::kOffAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / split;
  const int tp = tile % p.p_tiles, tq = tile / p.p_tiles;
  // this CTA's run of reduction blocks (the host gives every rank at least one)
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full_bar(s), 1); mbar_init(empty_bar(s), 1); }
    mbar_init(accf_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
    prefetch_tmap(&tmP);
    prefetch_tmap(&tmQ);
  }
  if (warp == 1) { tmem_alloc(smem_u32(holder), kCols); tmem_relinquish(); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;

  if (warp == 0) {
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      bool ok = true;
      int kb = kb0;
      for (; kb < kb1; ++kb) {
        if (!mbar_wait(empty_bar(st), phase ^ 1u, abort_flag, p.wait_limit_ns)) { ok = false; break; }
        const uint32_t fb = full_bar(st);
        mbar_expect_tx(fb, Ly::kStageBytes);
        lin_load<128, false>(sbase + Ly::kOffP + st * Ly::kPBytes, &tmP, fb, p.p_mn, tp * 128, kb);
        lin_load<BN, false>(sbase + Ly::kOffQ + st * Ly::kQBytes, &tmQ, fb, p.q_mn, tq * BN, kb);
        if (++st == S) { st = 0; phase ^= 1u; }
      }
      if (!ok) {
        if (p.status != nullptr) atomicOr(p.status, kStatusTimeout);
        // the loads in flight, one per stage at most: wait (bounded) for each
        const int issued = kb - kb0;
        for (int u = max(0, issued - S); u < issued; ++u) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(full_bar(u % S), (u / S) & 1) && globaltimer_ns() - t0 < kDrainLimitNs) {}
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint64_t pd0 = p.p_mn ? sdesc_mnmajor_sw128(sbase + Ly::kOffP) : sdesc_kmajor_sw128(sbase + Ly::kOffP);
      const uint64_t qd0 = p.q_mn ? sdesc_mnmajor_sw128(sbase + Ly::kOffQ) : sdesc_kmajor_sw128(sbase + Ly::kOffQ);
      const uint64_t pstep = p.p_mn ? 2048 >> 4 : 32 >> 4, qstep = p.q_mn ? 2048 >> 4 : 32 >> 4;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(full_bar(st), phase, abort_flag, p.wait_limit_ns)) { ok = false; break; }
        tc_fence_after();
        const uint64_t pd = pd0 + static_cast<uint64_t>((st * Ly::kPBytes) >> 4);
        const uint64_t qd = qd0 + static_cast<uint64_t>((st * Ly::kQBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_bf16(tmem, pd + kk * pstep, qd + kk * qstep, p.idesc, (kb > kb0 || kk > 0) ? 1u : 0u);
        tc_commit(empty_bar(st));
        if (++st == S) { st = 0; phase ^= 1u; }
      }
      // also the drain when a wait ran out: every issued MMA has completed
      tc_commit(accf_bar);
      if (!ok) {
        if (p.status != nullptr) atomicOr(p.status, kStatusTimeout);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(accf_bar, 0) && globaltimer_ns() - t0 < kDrainLimitNs) {}
      }
    }
  }
  __syncwarp();
  const int q = warp & 3, half = (warp - 2) >> 2;
  constexpr int kHalf = BN / 2;
  const int i = tp * 128 + q * 32 + lane;
  if (warp >= 2) {
    const float bias = lin_bias(p, i);
    const bool got = __all_sync(0xffffffffu, mbar_wait(accf_bar, 0, abort_flag, p.wait_limit_ns));
    if (!got) {
      if (lane == 0 && p.status != nullptr) atomicOr(p.status, kStatusTimeout);
    } else {
      tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * kHalf;
#pragma unroll 1
      for (int c = 0; c < kHalf; c += kLinChunk) {
        float v[kLinChunk];
        tmem_ld16(ta + c, reinterpret_cast<uint32_t*>(v));
        tmem_wait_ld();
        if (split == 1) {
          lin_finish<kLinChunk>(p, v, i, tq * BN + half * kHalf + c, bias);
        } else {
          // every load has landed and every MMA has completed: the stages' memory
          // takes the partial tile, a row of 128 columns per output row
          float* part = reinterpret_cast<float*>(smem) + (half * kHalf + c) * 128 + q * 32 + lane;
#pragma unroll
          for (int k = 0; k < kLinChunk; ++k) part[k * 128] = v[k];
        }
      }
    }
  }
  if (split > 1) {
    cluster_sync();
    if (warp >= 2) {
      // this CTA's BN / split rows, shared between the two halves of the warps
      const float bias = lin_bias(p, i);
      const int per = BN / split, r0 = rank * per;
      for (int r = r0 + half; r < r0 + per; r += 2) {
        const uint32_t at = sbase + static_cast<uint32_t>((r * 128 + q * 32 + lane) * 4);
        float v[1] = {0.0f};
        for (int s = 0; s < split; ++s) v[0] += ld_shared_cluster(mapa_shared(at, s));
        lin_finish<1>(p, v, i, tq * BN + r, bias);
      }
    }
  }
  tc_fence_before();
  if (split > 1) cluster_sync();          // the partial tiles stay until every CTA has read them
  else __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

}  // namespace bsgg
