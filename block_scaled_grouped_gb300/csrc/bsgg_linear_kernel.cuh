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
constexpr int kLinMaxSplit = 8;                // CTAs (or with pairs, twice the pairs) that share a tile's reduction
constexpr int kLinChunk = 16;                 // output rows an epilogue warp finishes at a time
constexpr int kLinThreads = 32 * (2 + kLinEpiWarps);

// The tensor core cuts what an addition to the accumulator drops instead of rounding
// it, so a long sum comes out small: by 1.05e-9 of it per element of the reduction,
// measured from 512 to 28672 (normal operands; 1.7e-5 at 14336, where a rounded sum
// in float32 is off by 2e-6).  Kernels with RUNS sum runs of kLinRun blocks apiece
// (512 elements: 6.5e-7) in the two accumulators in turn; the epilogue's warps add
// each to float32 registers, rounding, while the next is multiplied.  float32
// outputs take them for every reduction over one run, 16-bit ones, whose own rounding
// is 2e-4 or more, over kLinWholeHalf blocks (32768: 3.8e-5).
// 2048 x 14336 -> 4096 into float32: 139 us, 136 in one sum; added to a float32 dw,
// where the finish reads as much as it writes, 4096 x 14336 x 4096 336 us against 280.
constexpr int kLinRun = 8;
constexpr int kLinWholeHalf = 512;

struct LinParams {
  int32_t cols, rows;         // i < cols, j < rows
  int32_t k_blocks;           // ceil(depth / 64)
  int32_t p_tiles, q_tiles;
  int32_t tile0, tile1;       // the tiles of this launch (pairs)
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

// Phi(z) = erfc(-z / sqrt 2) / 2: unlike 1 + erf it keeps its relative accuracy in
// the lower tail, up to the argument's rounding, z^2 units of 2^-24.  (normcdff, which
// corrects that rounding too, is more instructions: 333 x 4104 -> 2049 with gelu
// takes 20.4 us with it and 19.8 with this.)
__device__ __forceinline__ float normal_cdf(float z) { return 0.5f * erfcf(-0.707106781f * z); }

// act(z).  silu = z / (1 + e^-z), below 0 as z e^z / (1 + e^z), so that the divisor
// stays between 1 and 2 (the hardware's quotient is 0 from a divisor of 2^126, z = -87.3,
// on), with the hardware's exponential and quotient (off by up to 5 + 1.2 |z| units of
// 2^-23; a quarter of the instructions of expf and an IEEE division); gelu = z Phi(z).
template <int ACT>
__device__ __forceinline__ float act_value(float z) {
  if (ACT == BSGG_ACT_RELU) return z <= 0.0f ? 0.0f : z;               // a NaN stays
  if (ACT == BSGG_ACT_SRELU) return z <= 0.0f ? 0.0f : z * z;
  if (ACT == BSGG_ACT_SILU) {
    const float e = __expf(-fabsf(z));
    return __fdividef(z >= 0.0f ? z : z * e, 1.0f + e);
  }
  if (ACT == BSGG_ACT_GELU) return z * normal_cdf(z);
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

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32"
      " [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      :
      : "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}

// sum += the N columns at ta, and the sum back into them.
template <int N>
__device__ __forceinline__ void lin_add_run(uint32_t ta, float (&sum)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += kLinChunk) {
    float v[kLinChunk];
    tmem_ld16(ta + c, reinterpret_cast<uint32_t*>(v));
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < kLinChunk; ++k) sum[c + k] += v[k];
  }
}
template <int N>
__device__ __forceinline__ void lin_put_sum(uint32_t ta, const float (&sum)[N]) {
#pragma unroll
  for (int c = 0; c < N; c += kLinChunk) {
    uint32_t v[kLinChunk];
#pragma unroll
    for (int k = 0; k < kLinChunk; ++k) v[k] = __float_as_uint(sum[c + k]);
    tmem_st16(ta + c, v);
  }
  tmem_wait_st();
}

// CH values of output column i, rows j0 .. j0 + CH - 1 (FULL: all of them exist).
// Every choice of type and function is made once for the chunk, around a loop
// whose accesses step by the row pitch: with the choices inside the loop the
// epilogue took 72 thousand cycles per 256 x 256 tile, twice the products of a
// reduction of 4096.
template <int KIND, int CH, bool FULL>
__device__ __forceinline__ void lin_load_rows(const void* base, int64_t at, int64_t ld, int nj, float (&r)[CH]) {
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    r[c] = (FULL || c < nj) ? load1<KIND>(base, at) : 0.0f;
    at += ld;
  }
}
template <int KIND, int CH, bool FULL>
__device__ __forceinline__ void lin_store_rows(void* base, int64_t at, int64_t ld, int nj, const float (&v)[CH]) {
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    if (FULL || c < nj) store1<KIND>(base, at, v[c]);
    at += ld;
  }
}
template <int ACT, int CH>
__device__ __forceinline__ void lin_act(float (&v)[CH]) {
#pragma unroll
  for (int c = 0; c < CH; ++c) v[c] = act_value<ACT>(v[c]);
}
template <int CH, bool FULL>
__device__ __forceinline__ void lin_finish_rows(const LinParams& p, float (&v)[CH], int i, int j0, int nj, float bias,
                                                bool residual) {
  float r[CH];
  if (residual) {
    const int64_t at = static_cast<int64_t>(j0) * p.ld_residual + i;
    if (p.residual_kind == OK_BF16) lin_load_rows<OK_BF16, CH, FULL>(p.residual, at, p.ld_residual, nj, r);
    else if (p.residual_kind == OK_F16) lin_load_rows<OK_F16, CH, FULL>(p.residual, at, p.ld_residual, nj, r);
    else lin_load_rows<OK_F32, CH, FULL>(p.residual, at, p.ld_residual, nj, r);
  }
  if (p.bias != nullptr) {
#pragma unroll
    for (int c = 0; c < CH; ++c) v[c] += bias;
  }
  if (p.z != nullptr) {
    const int64_t at = static_cast<int64_t>(j0) * p.ldz + i;
    if (p.in_kind == OK_BF16) lin_store_rows<OK_BF16, CH, FULL>(p.z, at, p.ldz, nj, v);
    else lin_store_rows<OK_F16, CH, FULL>(p.z, at, p.ldz, nj, v);
  }
  switch (p.act) {
    case BSGG_ACT_RELU: lin_act<BSGG_ACT_RELU>(v); break;
    case BSGG_ACT_SRELU: lin_act<BSGG_ACT_SRELU>(v); break;
    case BSGG_ACT_SILU: lin_act<BSGG_ACT_SILU>(v); break;
    case BSGG_ACT_GELU: lin_act<BSGG_ACT_GELU>(v); break;
  }
  if (residual) {
#pragma unroll
    for (int c = 0; c < CH; ++c) v[c] += r[c];
  }
  const int64_t at = static_cast<int64_t>(j0) * p.ld_out + i;
  if (p.out_kind == OK_BF16) lin_store_rows<OK_BF16, CH, FULL>(p.out, at, p.ld_out, nj, v);
  else if (p.out_kind == OK_F16) lin_store_rows<OK_F16, CH, FULL>(p.out, at, p.ld_out, nj, v);
  else lin_store_rows<OK_F32, CH, FULL>(p.out, at, p.ld_out, nj, v);
}
template <int CH>
__device__ __forceinline__ void lin_finish(const LinParams& p, float (&v)[CH], int i, int j0, float bias, bool residual) {
  const int nj = p.rows - j0;
  if (i >= p.cols || nj <= 0) return;
  if (nj >= CH) lin_finish_rows<CH, true>(p, v, i, j0, nj, bias, residual);
  else lin_finish_rows<CH, false>(p, v, i, j0, nj, bias, residual);
}
__device__ __forceinline__ float lin_bias(const LinParams& p, int i) {
  return p.bias != nullptr && i < p.cols ? load1(p.bias_kind, p.bias, i) : 0.0f;
}

// The residual of `rows` output rows from j0 and of the warp's 32 columns from i0, into L2.
__device__ __forceinline__ void lin_fetch_residual(const LinParams& p, int i0, int j0, int rows) {
  if (p.residual == nullptr || i0 >= p.cols) return;
  const int size = p.residual_kind == OK_F32 ? 4 : 2, last = min(i0 + 31, p.cols - 1);
  const int end = min(j0 + rows, p.rows);
  for (int j = j0 + (threadIdx.x & 31); j < end; j += 32) {
    const char* row = static_cast<const char*>(p.residual) + static_cast<int64_t>(j) * p.ld_residual * size;
    prefetch_l2(row + static_cast<int64_t>(i0) * size);
    prefetch_l2(row + static_cast<int64_t>(last) * size);       // a row that is off the lines has a second one
  }
}

// Partial tiles of a split reduction: CH output rows from row r of the tile, this
// lane's column, 128 columns per row; the stages' memory takes them, once every
// load has landed and every MMA completed.
template <int CH>
__device__ __forceinline__ void lin_put_part(uint8_t* smem, const float (&v)[CH], int r, int col) {
  float* at = reinterpret_cast<float*>(smem) + r * 128 + col;
#pragma unroll
  for (int k = 0; k < CH; ++k) at[k * 128] = v[k];
}

// Adds the partial tiles of SPLIT CTAs (ranks first, first + stride, ...) in
// order of rank, so the sum does not depend on timing, into this CTA's own tile:
// part p takes rows [p BN / SPLIT, ...), which nobody else reads here.  A warp
// reads a whole row of 128 columns per load, 16 bytes a lane, and has eight such
// loads in flight: distributed shared memory answers in about a microsecond, and
// 4-byte loads moved 2.2 MB/us over the whole chip, more time than the products.
template <int SPLIT>
__device__ __forceinline__ void lin_sum_parts(uint32_t part_base, int r0, int r1, uint32_t stride, uint32_t first) {
  constexpr int kRows = 8 / SPLIT;
  const int warp = (threadIdx.x >> 5) - 2, lane = threadIdx.x & 31;
  for (int r = r0 + warp * kRows; r < r1; r += kLinEpiWarps * kRows) {
    const uint32_t at = part_base + static_cast<uint32_t>((r * 128 + lane * 4) * 4);
    float4 u[SPLIT][kRows];
#pragma unroll
    for (int s = 0; s < SPLIT; ++s) {
      const uint32_t from = mapa_shared(at, first + stride * s);
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (r + k < r1) u[s][k] = ld_shared_cluster4(from + 512u * k);
    }
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      if (r + k >= r1) break;
      float4 v = u[0][k];
#pragma unroll
      for (int s = 1; s < SPLIT; ++s) { v.x += u[s][k].x; v.y += u[s][k].y; v.z += u[s][k].z; v.w += u[s][k].w; }
      st_shared_v4(at + 512u * k, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z), __float_as_uint(v.w));
    }
  }
}
// Then this part's rows go out, lanes along the columns as everywhere else.
template <int RUN>
__device__ __forceinline__ void lin_finish_part(const LinParams& p, const uint8_t* smem, int r0, int r1, int i0, int j0) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int q = warp & 3, half = (warp - 2) >> 2, i = i0 + q * 32 + lane;
  const float bias = lin_bias(p, i);
  for (int r = r0 + half * RUN; r < r1; r += 2 * RUN) {
    const float* at = reinterpret_cast<const float*>(smem) + r * 128 + q * 32 + lane;
    float v[RUN];
#pragma unroll
    for (int k = 0; k < RUN; ++k) v[k] = at[k * 128];
    lin_finish<RUN>(p, v, i, j0 + r, bias, p.residual != nullptr);
  }
}
// Only the epilogue's warps come here.
template <int BN>
__device__ __forceinline__ void lin_join(const LinParams& p, uint8_t* smem, int split, int part, uint32_t stride,
                                         uint32_t first, int i0, int j0) {
  const int per = BN / split, r0 = part * per;
  const uint32_t base = smem_u32(smem);
  if (split == 2) lin_sum_parts<2>(base, r0, r0 + per, stride, first);
  else if (split == 4) lin_sum_parts<4>(base, r0, r0 + per, stride, first);
  else lin_sum_parts<8>(base, r0, r0 + per, stride, first);
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kLinEpiWarps) : "memory");
  if (per >= 32) lin_finish_part<16>(p, smem, r0, r0 + per, i0, j0);
  else lin_finish_part<4>(p, smem, r0, r0 + per, i0, j0);
}

// True in one lane of a converged warp.  The matrix instructions are issued
// under it by a warp whose every lane runs the loop: issued by a lane chosen with
// an ordinary branch, each cost about 85 cycles of the issuing thread (a 128 x 32
// block of 64 took 0.22 us whatever its width), under elect.sync about 33.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
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
// 256 x BN tiles (BN 256 or 128), persistent, two accumulators: the epilogue of one
// tile runs under the products of the next.  A pair's instruction takes 128 rows of
// either operand from each CTA, 32 KB a block of 64 for 512 cycles of products, which
// is what shared memory and L2 can feed; single CTAs of 128 x 128 need twice that
// (2048 x 4096 x 4096: 60 us against 45).  Where there are too few tiles for the SMs,
// clusters of `split` pairs share a tile's reduction instead, one tile each.
//   4096 x 14336 x 4096, bf16, bias, silu, z kept: 249 us, 1930 TFLOP/s (the library's
//     product of the shape alone: 229); 8192 cubed 592 us, 1858.  Bound by the tensor
//     pipe (80 % of the elapsed cycles by counter) and by power: with operands of
//     zeros, at full clocks, the first takes 209 us.
//   4096 x 14336 x 64: 44 us for 117 MB written, 2.7 TB/s: bound by the epilogue, whose
//     lanes store 2 bytes at a time (a plain fill of as much takes 30 us).
template <int BN>
struct LinPair {
  // 64-blocks of the reduction per stage.  Handing a stage over costs its threads
  // about 230 cycles; a block's products take 512 at BN = 256, where they hide it,
  // and 256 at BN = 128
  static constexpr int kBlocks = BN == 256 ? 1 : 2;
  static constexpr int kPBlock = 128 * 128, kQBlock = BN / 2 * 128;   // this CTA's 128 and BN / 2 rows
  static constexpr int kPBytes = kBlocks * kPBlock, kQBytes = kBlocks * kQBlock;
  static constexpr int kStageBytes = kPBytes + kQBytes;
  static constexpr int kStages = 196608 / kStageBytes;
  static constexpr int kOffP = 0, kOffQ = kStages * kPBytes;
  static constexpr int kOffBars = kStages * kStageBytes;
  static constexpr int kNumBars = 2 * kStages + 4 + 1;
  static constexpr int kOffHolder = kOffBars + 8 * kNumBars;
  static constexpr int kOffAbort = kOffHolder + 4;
  static constexpr int kSmem = kOffAbort + 4 + 1024;
  static constexpr uint32_t kCols = 2 * BN;                           // two accumulators
  static_assert(kOffBars >= 128 * BN * 4, "the partial tile reuses the stages");
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

template <int BN, bool RUNS>
__global__ void __launch_bounds__(kLinThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ LinParams p, int split) {
  using Ly = LinPair<BN>;
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
  // ranks 2 s and 2 s + 1 are the pair that sums run s of the reduction
  const uint32_t rank = cluster_ctarank(), prank = rank & 1u, even = rank & ~1u;
  const uint16_t pair_mask = static_cast<uint16_t>(3u << even);
  const int part = static_cast<int>(rank >> 1);
  const bool leader = prank == 0;
  const int unit = blockIdx.x / (2 * split), units = gridDim.x / (2 * split);
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * part / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (part + 1) / split);
  const int run = RUNS ? kLinRun : kb1 - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full_bar(s), 1); mbar_init(empty_bar(s), 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(accf_bar(a), 1); mbar_init(acce_bar(a), 2 * kLinEpiWarps); }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    mbar_fence_init();
    prefetch_tmap(&tmP);
    prefetch_tmap(&tmQ);
  }
  if (warp == 1) { tmem_alloc_pair(smem_u32(holder), Ly::kCols); tmem_relinquish_pair(); }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *holder;
  let_next_kernel_start();
  wait_for_previous_kernel();

  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      bool ok = true, any = false;
      for (int t = p.tile0 + unit; t < p.tile1 && ok; t += units) {
        int tp, tq;
        lin_tile(t, p.p_tiles, p.q_tiles, tp, tq);
        const int p0 = tp * 256 + static_cast<int>(prank) * 128, q0 = tq * BN + static_cast<int>(prank) * (BN / 2);
        for (int kb = kb0; kb < kb1; kb += Ly::kBlocks) {
          if (!mbar_wait(empty_bar(st), phase ^ 1u, abort_flag, p.wait_limit_ns)) { ok = false; break; }
          // both CTAs' bytes complete the even CTA's barrier
          const uint32_t fb = full_bar(st), fbl = mapa_shared(fb, even);
          const int nb = min(Ly::kBlocks, kb1 - kb);
          if (leader) mbar_expect_tx(fb, 2u * nb * (Ly::kPBlock + Ly::kQBlock));
          for (int b = 0; b < nb; ++b) {
            lin_load<128, true>(sbase + Ly::kOffP + st * Ly::kPBytes + b * Ly::kPBlock, &tmP, fbl, p.p_mn, p0, kb + b);
            lin_load<BN / 2, true>(sbase + Ly::kOffQ + st * Ly::kQBytes + b * Ly::kQBlock, &tmQ, fbl, p.q_mn, q0, kb + b);
          }
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
    if (leader) {
      int st = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      const uint64_t pd0 = p.p_mn ? sdesc_mnmajor_sw128(sbase + Ly::kOffP) : sdesc_kmajor_sw128(sbase + Ly::kOffP);
      const uint64_t qd0 = p.q_mn ? sdesc_mnmajor_sw128(sbase + Ly::kOffQ) : sdesc_kmajor_sw128(sbase + Ly::kOffQ);
      // 16 reduction indices: 32 bytes inside a K-major row, 16 rows of 128 bytes MN-major
      const uint64_t pstep = p.p_mn ? 2048 >> 4 : 32 >> 4, qstep = p.q_mn ? 2048 >> 4 : 32 >> 4;
      for (int t = p.tile0 + unit; t < p.tile1 && ok; t += units) {
        for (int kr = kb0; kr < kb1; kr += run) {
          if (!__all_sync(0xffffffffu, mbar_wait(acce_bar(acc), acc_phase ^ 1u, abort_flag, p.wait_limit_ns))) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem + acc * BN;
          const int kend = min(kb1, kr + run);
          for (int kb = kr; kb < kend; kb += Ly::kBlocks) {
            if (!__all_sync(0xffffffffu, mbar_wait(full_bar(st), phase, abort_flag, p.wait_limit_ns))) { ok = false; break; }
            tc_fence_after();
            const uint64_t pd = pd0 + static_cast<uint64_t>((st * Ly::kPBytes) >> 4);
            const uint64_t qd = qd0 + static_cast<uint64_t>((st * Ly::kQBytes) >> 4);
            const bool whole = Ly::kBlocks == 1 || kb + 1 < kb1;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < 4 * Ly::kBlocks; ++kk) {
                if (kk >= 4 && !whole) break;
                tc_mma_bf16_pair(d, pd + (kk / 4) * (Ly::kPBlock >> 4) + (kk % 4) * pstep,
                                 qd + (kk / 4) * (Ly::kQBlock >> 4) + (kk % 4) * qstep, p.idesc, (kb > kr || kk > 0) ? 1u : 0u);
              }
              tc_commit_pair(empty_bar(st), pair_mask);
            }
            __syncwarp();
            if (++st == S) { st = 0; phase ^= 1u; }
          }
          if (!ok) break;
          if (elect_one()) tc_commit_pair(accf_bar(acc), pair_mask);
          __syncwarp();
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
      }
      if (!ok && elect_one()) {
        if (p.status != nullptr) atomicOr(p.status, kStatusTimeout);
        tc_commit_pair(drain_bar, static_cast<uint16_t>(1u << even));
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < kDrainLimitNs) {}
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;         // lane quadrant, half of the columns
    constexpr int kHalf = BN / 2;
    // With runs only one of them hides what finishing a tile takes, and the products
    // wait for the rest: the tile is finished in half the steps, its residual is fetched
    // at its start, and one in float32 that no function of the sum precedes (a gradient
    // being added to) is summed in while the last run is multiplied.
    constexpr int kFinish = RUNS ? 2 * kLinChunk : kLinChunk;
    const bool add_early = RUNS && split == 1 && p.residual != nullptr && p.residual_kind == OK_F32 &&
                           p.act == BSGG_ACT_NONE && p.z == nullptr && kb1 - kb0 > run;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int t = p.tile0 + unit; t < p.tile1; t += units) {
      int tp, tq;
      lin_tile(t, p.p_tiles, p.q_tiles, tp, tq);
      const int i = tp * 256 + static_cast<int>(prank) * 128 + q * 32 + lane;
      const float bias = lin_bias(p, i);
      const uint32_t ta0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * kHalf;
      const bool early = add_early && tq * BN + (half + 1) * kHalf <= p.rows;     // every row exists
      if (RUNS && split == 1) lin_fetch_residual(p, i - lane, tq * BN + half * kHalf, kHalf);
      bool got = __all_sync(0xffffffffu, mbar_wait(accf_bar(acc), acc_phase, abort_flag, p.wait_limit_ns));
      if (RUNS && got) {
        float sum[kHalf];
#pragma unroll
        for (int c = 0; c < kHalf; ++c) sum[c] = 0.0f;
#pragma unroll 1
        for (int kr = kb0 + run;; kr += run) {
          tc_fence_after();
          lin_add_run(ta0 + acc * BN, sum);
          if (kr >= kb1) break;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(acce_bar(acc), even));
          if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
          if (early && kr + run >= kb1) {
            // a lane past the last column reads that one: its sums go nowhere
            const float* from = static_cast<const float*>(p.residual) +
                                static_cast<int64_t>(tq * BN + half * kHalf) * p.ld_residual + min(i, p.cols - 1);
#pragma unroll
            for (int c = 0; c < kHalf; c += kLinChunk) {
              float r[kLinChunk];
#pragma unroll
              for (int k = 0; k < kLinChunk; ++k) { r[k] = *from; from += p.ld_residual; }
#pragma unroll
              for (int k = 0; k < kLinChunk; ++k) sum[c + k] += r[k];
              asm volatile("" : "+l"(from) :: "memory");   // sixteen addresses at a time, not all of them
            }
          }
          got = __all_sync(0xffffffffu, mbar_wait(accf_bar(acc), acc_phase, abort_flag, p.wait_limit_ns));
          if (!got) break;
        }
        if (got) lin_put_sum(ta0 + acc * BN, sum);
      }
      if (!got) {
        if (lane == 0 && p.status != nullptr) atomicOr(p.status, kStatusTimeout);
        break;
      }
      tc_fence_after();
      const uint32_t ta = ta0 + acc * BN;
#pragma unroll 1
      for (int c = 0; c < kHalf; c += kFinish) {
        float v[kFinish];
#pragma unroll
        for (int k = 0; k < kFinish; k += 16) tmem_ld16(ta + c + k, reinterpret_cast<uint32_t*>(v) + k);
        tmem_wait_ld();
        if (c == kHalf - kFinish) {
          // every column is in registers or stored: hand the accumulator back
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(acce_bar(acc), even));
        }
        if (split == 1) lin_finish<kFinish>(p, v, i, tq * BN + half * kHalf + c, bias, p.residual != nullptr && !early);
        else lin_put_part(smem, v, half * kHalf + c, q * 32 + lane);
      }
      if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
  }
  __syncwarp();
  if (split > 1) {
    cluster_sync();
    if (warp >= 2) {
      // the pairs' CTAs of this half of p
      int tp, tq;
      lin_tile(p.tile0 + unit, p.p_tiles, p.q_tiles, tp, tq);
      lin_join<BN>(p, smem, split, part, 2, prank, tp * 256 + static_cast<int>(prank) * 128, tq * BN);
    }
  }
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem, Ly::kCols);
  }
}

// ---------------------------------------------------------------- single CTAs
// One 128 x BN tile per CTA; with a cluster of S CTAs the reduction is split into
// S runs of blocks, whose partial tiles are added in order of rank through
// distributed shared memory, every CTA finishing BN / S of the output rows.
// Where every CTA has an SM to itself (ALONE) the ring takes the whole of its shared
// memory in stages of two 64-blocks: operands that come from DRAM want the depth
// (three 32 KB stages: 0.36 us a block, six: 0.22), and handing a stage over costs
// its threads about 230 cycles, which the products of one block do not hide
// (BN = 32: 0.19 us a block with one block per stage, 0.146 with two).  Two CTAs
// on an SM hide each other's.
//   one row x 14336 -> 4096: 21.2 us for 117 MB of weights, 5.5 TB/s; bound by memory,
//     with 4 us of start, join and end;
//   128 x 4096 x 7168: 16.2 us; 16 x 7168 x 2048: 8.6 us, half of it fixed.
template <int BN, bool ALONE>
struct LinTile {
  static constexpr int kBlocks = ALONE ? 2 : 1;            // 64-blocks of the reduction per stage
  static constexpr int kPBlock = 128 * 128, kQBlock = BN * 128;
  static constexpr int kPBytes = kBlocks * kPBlock, kQBytes = kBlocks * kQBlock;
  static constexpr int kStageBytes = kPBytes + kQBytes;
  static constexpr int kStages = (ALONE ? 220 : 110) * 1024 / kStageBytes;
  static constexpr int kHead = 1024;                       // barriers, holder, flag; the ring follows
  static_assert(8 * (2 * kStages + 5) + 8 <= kHead, "barriers");
  static_assert(kStages * kStageBytes >= 128 * BN * 4, "the partial tile reuses the stages");
  static constexpr int kSmem = kStages * kStageBytes + kHead + 1024;
};

template <int BN, bool ALONE, bool RUNS>
__global__ void __launch_bounds__(kLinThreads, ALONE ? 1 : 2)
    linear_tile_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ LinParams p, int split) {
  using Ly = LinTile<BN, ALONE>;
  constexpr int S = Ly::kStages;
  constexpr uint32_t kCols = RUNS ? 2 * BN : BN;     // tensor-memory columns, a power of two >= 32
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t bar0 = smem_u32(smem);
  const uint32_t ring = bar0 + Ly::kHead;                  // stages of P, then of Q
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto accf_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto acce_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + 8 * (2 * S + 5));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 8 * (2 * S + 5) + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / split;
  const int tp = tile % p.p_tiles, tq = tile / p.p_tiles;
  // this CTA's run of reduction blocks (the host gives every rank at least one)
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * rank / split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.k_blocks) * (rank + 1) / split);
  const int run = RUNS ? kLinRun : kb1 - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) { mbar_init(full_bar(s), 1); mbar_init(empty_bar(s), 1); }
    for (int a = 0; a < 2; ++a) { mbar_init(accf_bar(a), 1); mbar_init(acce_bar(a), kLinEpiWarps); }
    mbar_init(drain_bar, 1);
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
  let_next_kernel_start();
  wait_for_previous_kernel();

  if (warp == 0) {
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      bool ok = true;
      int kb = kb0;
      for (; kb < kb1; kb += Ly::kBlocks) {
        if (!mbar_wait(empty_bar(st), phase ^ 1u, abort_flag, p.wait_limit_ns)) { ok = false; break; }
        const uint32_t fb = full_bar(st);
        const int nb = min(Ly::kBlocks, kb1 - kb);
        mbar_expect_tx(fb, nb * (Ly::kPBlock + Ly::kQBlock));
        for (int b = 0; b < nb; ++b) {
          lin_load<128, false>(ring + st * Ly::kPBytes + b * Ly::kPBlock, &tmP, fb, p.p_mn, tp * 128, kb + b);
          lin_load<BN, false>(ring + S * Ly::kPBytes + st * Ly::kQBytes + b * Ly::kQBlock, &tmQ, fb, p.q_mn, tq * BN, kb + b);
        }
        if (++st == S) { st = 0; phase ^= 1u; }
      }
      if (!ok) {
        if (p.status != nullptr) atomicOr(p.status, kStatusTimeout);
        // the loads in flight, one per stage at most: wait (bounded) for each
        const int issued = (kb - kb0 + Ly::kBlocks - 1) / Ly::kBlocks;
        for (int u = max(0, issued - S); u < issued; ++u) {
          const uint64_t t0 = globaltimer_ns();
          while (!mbar_try_wait(full_bar(u % S), (u / S) & 1) && globaltimer_ns() - t0 < kDrainLimitNs) {}
        }
      }
    }
  } else if (warp == 1) {
    int st = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t ring_q = ring + S * Ly::kPBytes;
    const uint64_t pd0 = p.p_mn ? sdesc_mnmajor_sw128(ring) : sdesc_kmajor_sw128(ring);
    const uint64_t qd0 = p.q_mn ? sdesc_mnmajor_sw128(ring_q) : sdesc_kmajor_sw128(ring_q);
    const uint64_t pstep = p.p_mn ? 2048 >> 4 : 32 >> 4, qstep = p.q_mn ? 2048 >> 4 : 32 >> 4;
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int kr = kb0; kr < kb1; kr += run) {
      if (RUNS && !__all_sync(0xffffffffu, mbar_wait(acce_bar(acc), acc_phase ^ 1u, abort_flag, p.wait_limit_ns))) { ok = false; break; }
      if (RUNS) tc_fence_after();
      const uint32_t d = tmem + acc * BN;
      const int kend = min(kb1, kr + run);
      for (int kb = kr; kb < kend; kb += Ly::kBlocks) {
        if (!__all_sync(0xffffffffu, mbar_wait(full_bar(st), phase, abort_flag, p.wait_limit_ns))) { ok = false; break; }
        tc_fence_after();
        const uint64_t pd = pd0 + static_cast<uint64_t>((st * Ly::kPBytes) >> 4);
        const uint64_t qd = qd0 + static_cast<uint64_t>((st * Ly::kQBytes) >> 4);
        const bool whole = Ly::kBlocks == 1 || kb + 1 < kb1;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4 * Ly::kBlocks; ++kk) {
            if (kk >= 4 && !whole) break;
            tc_mma_bf16(d, pd + (kk / 4) * (Ly::kPBlock >> 4) + (kk % 4) * pstep,
                        qd + (kk / 4) * (Ly::kQBlock >> 4) + (kk % 4) * qstep, p.idesc, (kb > kr || kk > 0) ? 1u : 0u);
          }
          tc_commit(empty_bar(st));
        }
        __syncwarp();
        if (++st == S) { st = 0; phase ^= 1u; }
      }
      if (!ok) break;
      if (elect_one()) tc_commit(accf_bar(acc));
      __syncwarp();
      if (RUNS && ++acc == 2) { acc = 0; acc_phase ^= 1u; }
    }
    if (!ok && elect_one()) {
      if (p.status != nullptr) atomicOr(p.status, kStatusTimeout);
      tc_commit(drain_bar);                         // every issued MMA has completed
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(drain_bar, 0) && globaltimer_ns() - t0 < kDrainLimitNs) {}
    }
  }
  __syncwarp();
  const int q = warp & 3, half = (warp - 2) >> 2;
  constexpr int kHalf = BN / 2;
  const int i = tp * 128 + q * 32 + lane;
  if (warp >= 2) {
    const float bias = lin_bias(p, i);
    const uint32_t ta0 = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * kHalf;
    int acc = 0;
    bool got = __all_sync(0xffffffffu, mbar_wait(accf_bar(0), 0, abort_flag, p.wait_limit_ns));
    if (RUNS && got) {
      uint32_t acc_phase = 0;
      float sum[kHalf];
#pragma unroll
      for (int c = 0; c < kHalf; ++c) sum[c] = 0.0f;
#pragma unroll 1
      for (int kr = kb0 + run;; kr += run) {
        tc_fence_after();
        lin_add_run(ta0 + acc * BN, sum);
        if (kr >= kb1) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce_bar(acc));
        if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        got = __all_sync(0xffffffffu, mbar_wait(accf_bar(acc), acc_phase, abort_flag, p.wait_limit_ns));
        if (!got) break;
      }
      if (got) lin_put_sum(ta0 + acc * BN, sum);
    }
    if (!got) {
      if (lane == 0 && p.status != nullptr) atomicOr(p.status, kStatusTimeout);
    } else {
      tc_fence_after();
      const uint32_t ta = ta0 + acc * BN;
#pragma unroll 1
      for (int c = 0; c < kHalf; c += kLinChunk) {
        float v[kLinChunk];
        tmem_ld16(ta + c, reinterpret_cast<uint32_t*>(v));
        tmem_wait_ld();
        if (split == 1) {
          lin_finish<kLinChunk>(p, v, i, tq * BN + half * kHalf + c, bias, p.residual != nullptr);
        } else {
          lin_put_part(smem + Ly::kHead, v, half * kHalf + c, q * 32 + lane);
        }
      }
    }
  }
  if (split > 1) {
    cluster_sync();
    if (warp >= 2) lin_join<BN>(p, smem + Ly::kHead, split, rank, 1, 0, tp * 128, tq * BN);
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
