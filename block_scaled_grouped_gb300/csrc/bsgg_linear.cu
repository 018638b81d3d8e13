// bsgg_linear.cu -- the dense layer act(x W^T + bias) + residual and its
// gradient.
#include <cudaTypedefs.h>

#include <mutex>

#include "bsgg_linear_kernel.cuh"

namespace {

using namespace bsgg;

// act'(z).  silu: s (1 + z (1 - s)) with e = e^-z, s = 1 / (1 + e), 1 - s = e s: no
// cancellation, one exponential and one reciprocal (the argument is held below 87,
// where s is 1e-38, so that e s stays a number: below z = -87 the slope, which falls
// under 1e-36 there, stays near -2e-36; with e^-|z| it would follow it to 0, and this
// pass take 64 us for 62); gelu: Phi(z) + z phi(z).
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
  if (ACT == BSGG_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if (ACT == BSGG_ACT_SRELU) return z > 0.0f ? 2.0f * z : 0.0f;
  if (ACT == BSGG_ACT_SILU) {
    const float e = __expf(fminf(-z, 87.0f)), s = __fdividef(1.0f, 1.0f + e);
    return s * fmaf(z, e * s, 1.0f);
  }
  if (ACT == BSGG_ACT_GELU) return normal_cdf(z) + z * 0.398942280401432678f * __expf(-0.5f * z * z);
  return 1.0f;
}

// dz = dy act'(z) and dbias.  dz is rounded to the operands' 16 bits, which is what the
// products take (dx and dw come out 2.3e-3 off in norm where a dz in 32 bits would leave
// their own rounding's 1.7e-3; into float32 about 1e-3 of it remains); dbias sums the
// values before that.  A block owns 64 columns (a lane eight of them, so
// that a warp reads four 128-byte pieces of rows at a time) and one of the
// cluster's runs of rows; its sums join through shared memory and, between the
// cluster's blocks, through distributed shared memory, in a fixed order.  Bound by
// the loads' latency, so the rows are split no further than fills the chip twice
// (what a block pays once, its joins above all, cost 4096 x 14336 in eight runs a
// quarter of its time): 352 MB in 62 us, 5.7 TB/s; in eight runs 83.
constexpr int kDzThreads = 512, kDzSplit = 8, kDzRows = 3, kDzLanes = 8;

template <int KIND, int ACT>
__global__ void __launch_bounds__(kDzThreads, 2) dz_kernel(int64_t m, int64_t n, int64_t ld_dy, int64_t ldz, int64_t ld_dz,
                                                        const void* dy, const void* z, void* dz, float* dbias, int runs) {
  constexpr int kCols = kDzLanes * 8, kWarps = kDzThreads / 32, kStep = kDzThreads / kDzLanes;
  __shared__ float part[kWarps][kCols];
  __shared__ float block_sum[kCols];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the runs of a group of columns are neighbours along x, which alone holds 2^24 / 64 groups
  const int group = static_cast<int>(blockIdx.x) / runs, run = static_cast<int>(blockIdx.x) - group * runs;
  const int64_t j = static_cast<int64_t>(group) * kCols + (threadIdx.x % kDzLanes) * 8;
  const int64_t i0 = m * run / runs, i1 = m * (run + 1) / runs;
  float sum[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (j + 8 <= n) {
    for (int64_t i = i0 + threadIdx.x / kDzLanes; i < i1; i += kStep * kDzRows) {
      Raw8<KIND, false> g[kDzRows], v[kDzRows];
#pragma unroll
      for (int u = 0; u < kDzRows; ++u) {
        const int64_t r = i + u * kStep;
        g[u].load(dy, r * ld_dy + j, r < i1);
        if (ACT != BSGG_ACT_NONE) v[u].load(z, r * ldz + j, r < i1);
      }
#pragma unroll
      for (int u = 0; u < kDzRows; ++u) {
        const int64_t r = i + u * kStep;
        if (r >= i1) break;
        float f[8];
        g[u].values(f);
        if (ACT != BSGG_ACT_NONE) {
          float w[8];
          v[u].values(w);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] *= act_slope<ACT>(w[k]);
          store8<KIND>(dz, r * ld_dz + j, f);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += f[k];
      }
    }
  } else if (j < n) {
    // the last lane of a width that is no multiple of 8 takes its columns one by one:
    // what lies past them need not be the caller's to read or write (4096 x 2049
    // 9.7 us, as with whole pieces; 4096 x 33, where this lane's rows are the longest
    // chain, 7.8 against 5.7)
    const int cols = static_cast<int>(n - j);
    for (int64_t r = i0 + threadIdx.x / kDzLanes; r < i1; r += kStep) {
#pragma unroll
      for (int k = 0; k < 7; ++k) {
        if (k >= cols) break;
        float f = load1<KIND>(dy, r * ld_dy + j + k);
        if (ACT != BSGG_ACT_NONE) {
          f *= act_slope<ACT>(load1<KIND>(z, r * ldz + j + k));
          store1<KIND>(dz, r * ld_dz + j + k, f);
        }
        sum[k] += f;
      }
    }
  }
  if (dbias == nullptr) return;
#pragma unroll
  for (int o = kDzLanes; o < 32; o <<= 1)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[k] += __shfl_xor_sync(0xFFFFFFFFu, sum[k], o);
  if (lane < kDzLanes) {
#pragma unroll
    for (int k = 0; k < 8; ++k) part[warp][lane * 8 + k] = sum[k];
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += part[w][threadIdx.x];
    block_sum[threadIdx.x] = s;
  }
  if (runs > 1) cluster_sync(); else __syncthreads();
  const int64_t c = static_cast<int64_t>(group) * kCols + threadIdx.x;
  if (run == 0 && threadIdx.x < kCols && c < n) {
    float s = 0.0f;
    for (int r = 0; r < runs; ++r) s += ld_shared_cluster(mapa_shared(smem_u32(&block_sum[threadIdx.x]), r));
    dbias[c] = s;
  }
  if (runs > 1) cluster_sync();               // the sums stay until block 0 has read them
}

__global__ void clear_bits_kernel(uint32_t* word, uint32_t bits) {
  let_next_kernel_start();
  wait_for_previous_kernel();
  atomicAnd(word, ~bits);
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (succeeded(cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q)) &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return nullptr;
  }();
  return fn;
}

// An operand of a product: `rows` indices and `depth` reduction indices; mn: the
// row index is the contiguous one.
struct Operand {
  const void* base;
  int64_t rows, depth, ld;
  bool mn;
};

// Boxes of 64 reduction indices: (64, tile_rows) K-major, (64, 64) MN-major.
bool encode_operand(CUtensorMap* map, const Operand& o, int tile_rows) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {cuuint64_t(o.mn ? o.rows : o.depth), cuuint64_t(o.mn ? o.depth : o.rows)};
  const cuuint64_t strides[1] = {cuuint64_t(2 * o.ld)};
  const cuuint32_t box[2] = {64, cuuint32_t(o.mn ? 64 : tile_rows)};
  const cuuint32_t es[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void*>(o.base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

uint32_t lin_idesc(int in_format, bool p_mn, bool q_mn, int m, int n) {
  // kind::f16: F32 accumulator (bits 4-5 = 1), F16 (0) or BF16 (1) operands, majorness (1 = MN)
  const uint32_t fmt = in_format == BSGG_OUT_BF16 ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (p_mn ? 1u << 15 : 0u) | (q_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// What a device holds of the products' kernels: SMs, and for each kernel and
// cluster size the clusters resident at once (a GPC's SMs are shared out in whole
// clusters, so that 16 clusters of 8 CTAs with an SM each do not fit 152 SMs).
struct Device {
  bool ok = false;
  int sms = 0;
  int pair_clusters[2][3];        // [bn 256, 128][split 1, 2, 4]
  int tile_clusters[3][2][4];     // [bn 32, 64, 128][shared, alone][split 1, 2, 4, 8]
};

// The kernel that sums in runs is launched like the other: its own shared-memory
// limit is raised, and the other's residency holds for both (launch bounds and shared
// memory are the same, and two blocks' accumulators fit an SM's tensor memory).
template <typename K>
bool prepare_kernel(K kern, K with_runs, int smem, int ctas, int clusters, int* resident) {
  for (const K k : {kern, with_runs})
    if (!succeeded(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return false;
  for (int i = 0; i < clusters; ++i) {
    const int cluster = ctas << i;
    const LaunchConfig c(dim3(static_cast<unsigned>(cluster)), kLinThreads, static_cast<size_t>(smem), nullptr, cluster);
    if (cluster == 1) {
      int blocks = 0, sms = 0, dev = 0;
      if (!succeeded(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kern, kLinThreads, static_cast<size_t>(smem))) ||
          !succeeded(cudaGetDevice(&dev)) || !succeeded(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)))
        return false;
      resident[i] = blocks * sms;
    } else if (!succeeded(cudaOccupancyMaxActiveClusters(&resident[i], kern, &c.cfg))) {
      return false;
    }
    if (resident[i] < 1) return false;
  }
  return true;
}
template <int BN>
bool prepare_tile(int (*resident)[4]) {
  return prepare_kernel(linear_tile_kernel<BN, false, false>, linear_tile_kernel<BN, false, true>, LinTile<BN, false>::kSmem, 1, 4, resident[0]) &&
         prepare_kernel(linear_tile_kernel<BN, true, false>, linear_tile_kernel<BN, true, true>, LinTile<BN, true>::kSmem, 1, 4, resident[1]);
}

// The current device's state, set up at its first call.
const Device* device_state() {
  static Device state[64];
  static std::mutex mu;
  int dev = 0;
  if (!succeeded(cudaGetDevice(&dev)) || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lk(mu);
  Device& d = state[dev];
  if (!d.ok) {
    if (!succeeded(cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev))) return nullptr;
    if (!prepare_kernel(linear_pair_kernel<256, false>, linear_pair_kernel<256, true>, LinPair<256>::kSmem, 2, 3, d.pair_clusters[0]) ||
        !prepare_kernel(linear_pair_kernel<128, false>, linear_pair_kernel<128, true>, LinPair<128>::kSmem, 2, 3, d.pair_clusters[1]) ||
        !prepare_tile<32>(d.tile_clusters[0]) || !prepare_tile<64>(d.tile_clusters[1]) ||
        !prepare_tile<128>(d.tile_clusters[2]))
      return nullptr;
    d.ok = true;
  }
  return &d;
}

// Whether a part of the reduction is summed in runs (see kLinRun).
bool in_runs(const LinParams& p, int split) {
  return ceil_div(p.k_blocks, split) > (p.out_kind == OK_F32 ? kLinRun : kLinWholeHalf);
}

template <int BN, bool ALONE>
bsgg_status launch_tile_as(const CUtensorMap& tp, const CUtensorMap& tq, const LinParams& p, int64_t ctas, int split,
                           cudaStream_t s) {
  const LaunchConfig c(dim3(static_cast<unsigned>(ctas)), kLinThreads, LinTile<BN, ALONE>::kSmem, s, split);
  return launch_kernel(c, in_runs(p, split) ? linear_tile_kernel<BN, ALONE, true> : linear_tile_kernel<BN, ALONE, false>, tp,
                       tq, p, split);
}
template <int BN>
bsgg_status launch_tile(const CUtensorMap& tp, const CUtensorMap& tq, const LinParams& p, int split, int sms, cudaStream_t s) {
  const int64_t ctas = int64_t(p.p_tiles) * p.q_tiles * split;
  return ctas <= sms ? launch_tile_as<BN, true>(tp, tq, p, ctas, split, s) : launch_tile_as<BN, false>(tp, tq, p, ctas, split, s);
}
// Tiles [tile0, tile1), a cluster of `split` pairs each, or the resident pairs
// walking them.
template <int BN>
bsgg_status launch_pairs(const CUtensorMap& tp, const CUtensorMap& tq, LinParams p, int64_t tile0, int64_t tile1, int split,
                         const Device& dev, cudaStream_t s) {
  p.tile0 = static_cast<int32_t>(tile0);
  p.tile1 = static_cast<int32_t>(tile1);
  const int64_t tiles = tile1 - tile0, resident = dev.pair_clusters[BN == 256 ? 0 : 1][0];
  const int64_t units = split > 1 || tiles < resident ? tiles : resident;
  const LaunchConfig c(dim3(static_cast<unsigned>(2 * split * units)), kLinThreads, LinPair<BN>::kSmem, s, 2 * split);
  return launch_kernel(c, in_runs(p, split) ? linear_pair_kernel<BN, true> : linear_pair_kernel<BN, false>, tp, tq, p, split);
}

// All tiles.  Where the last round of the pairs would be less than half full and
// long, its tiles get a launch of their own, their reduction split over the idle
// pairs: the gradient dx of 4096 x 14336 x 4096 has 256 tiles for 76 pairs, and takes
// 273 us in 4 rounds of 224 blocks, 263 in 3 and a split remainder.  (8192 cubed, 36
// tiles of 128 blocks left after 13 rounds, gains nothing: 12 us have to be in it.)
template <int BN>
bsgg_status launch_pair(const CUtensorMap& tp, const CUtensorMap& tq, const LinParams& p, int split, const Device& dev,
                        cudaStream_t s) {
  const int64_t tiles = int64_t(p.p_tiles) * p.q_tiles, resident = dev.pair_clusters[BN == 256 ? 0 : 1][0];
  const int64_t rest = tiles % resident;
  if (split > 1 || tiles < resident || rest == 0) return launch_pairs<BN>(tp, tq, p, 0, tiles, split, dev, s);
  int best = 1;
  double most = 12.0;                                  // microseconds saved, by cost_us's figures
  for (int log2 = 1; log2 <= 2; ++log2) {
    const int parts = 1 << log2;
    if (rest > dev.pair_clusters[BN == 256 ? 0 : 1][log2] || p.k_blocks < 2 * parts) continue;
    const double saved = p.k_blocks * (BN == 256 ? 0.33 : 0.21) * (1.0 - 1.0 / parts) - 8.0 -
                         double(rest) * parts * 256 * BN * 4.0 / 4e6;
    if (saved > most) { most = saved; best = parts; }
  }
  if (best == 1) return launch_pairs<BN>(tp, tq, p, 0, tiles, 1, dev, s);
  const bsgg_status st = launch_pairs<BN>(tp, tq, p, 0, tiles - rest, 1, dev, s);
  return st == BSGG_OK ? launch_pairs<BN>(tp, tq, p, tiles - rest, tiles, best, dev, s) : st;
}

// How a product is tiled: 256 x bn on CTA pairs, or 128 x bn on single CTAs, with
// the reduction in `split` parts.
struct Choice {
  bool pair;
  int bn, split;
};

// Microseconds of a choice, from what a block of 64 of the reduction took on GB300
// (bf16 operands out of DRAM) and what is paid once:
//   start, tensor-memory allocation, first load, epilogue      5, pairs of 256 6.5
//   256 x 256 pair block 0.33, 256 x 128 pair block 0.21
//   128 x 32 / 64 / 128 block, a CTA per SM   0.155 / 0.165 / 0.24
//   the same, several CTAs per SM, per block of each SM   0.15 / 0.173 / 0.256
//   joining a split reduction                 1.5 and 4 MB of partial tiles per us
// Measured both ways: 512 x 4096 x 4096 takes 19.8 us on 64 pairs of 256 x 128 and
// 27.3 on 32 of 256 x 256; 2048 x 4096 x 4096 45.3 on 256 x 256, 56.2 on 256 x 128,
// 60.5 on 128 x 128; 128 x 4096 x 7168 17.5 on 64-wide tiles in two parts, 24.0 whole;
// one row x 14336 -> 4096 22.2 in four parts, 40.0 whole.
// Clusters beyond those resident at once wait for a second round.
double cost_us(const Choice& c, int64_t p_rows, int64_t q_rows, int64_t k_blocks, const Device& dev) {
  const int side = c.pair ? 256 : 128, log2 = c.split == 1 ? 0 : c.split == 2 ? 1 : c.split == 4 ? 2 : 3;
  const int64_t tiles = ceil_div(p_rows, side) * ceil_div(q_rows, c.bn);
  const double blocks = double(ceil_div(k_blocks, c.split));
  double run, fixed = 5.0;
  if (c.pair) {
    run = double(ceil_div(tiles, dev.pair_clusters[c.bn == 256 ? 0 : 1][log2])) * blocks * (c.bn == 256 ? 0.33 : 0.21);
    if (c.bn == 256) fixed = 6.5;
  } else {
    const int w = c.bn == 32 ? 0 : c.bn == 64 ? 1 : 2;
    const double alone[3] = {0.155, 0.165, 0.24}, shared[3] = {0.15, 0.173, 0.256};
    const int64_t ctas = tiles * c.split;
    if (ctas <= dev.sms) {
      run = double(ceil_div(tiles, dev.tile_clusters[w][1][log2])) * blocks * alone[w];
    } else {
      const double rounds = double(tiles) / dev.tile_clusters[w][0][log2];
      run = blocks * shared[w] * (rounds > 1.0 ? 2.0 * rounds : double(ctas) / dev.sms);
    }
  }
  const double join = c.split > 1 ? 1.5 + double(tiles) * c.split * side * c.bn * 4.0 / 4e6 : 0.0;
  return fixed + run + join;
}

Choice choose(const Operand& P, const Operand& Q, int k_blocks, const Device& dev) {
  Choice best = {true, 256, 1};
  double least = cost_us(best, P.rows, Q.rows, k_blocks, dev);
  for (const int pair : {1, 0})
    for (const int bn : {256, 128, 64, 32}) {
      if (pair ? bn < 128 : bn > 128) continue;
      if (bn == 32 && Q.mn) continue;                        // MN-major boxes are 64 wide
      for (int split = 1; split <= (pair ? kLinMaxSplit / 2 : kLinMaxSplit) && k_blocks >= 2 * split; split *= 2) {
        const Choice c = {pair != 0, bn, split};
        const double t = cost_us(c, P.rows, Q.rows, k_blocks, dev);
        if (t < least) { least = t; best = c; }
      }
    }
  return best;
}

bsgg_status launch_product(const Operand& P, const Operand& Q, int in_format, LinParams p, cudaStream_t s) {
  const Device* dev = device_state();
  if (!dev) return BSGG_ERR_CUDA;
  p.cols = static_cast<int32_t>(P.rows);
  p.rows = static_cast<int32_t>(Q.rows);
  p.k_blocks = static_cast<int32_t>(ceil_div(P.depth, kLinDepth));
  p.p_mn = P.mn;
  p.q_mn = Q.mn;
  p.in_kind = in_format;
  p.wait_limit_ns = kWaitLimitNs;
  CUtensorMap tp, tq;
  const Choice c = choose(P, Q, p.k_blocks, *dev);
  const int side = c.pair ? 256 : 128;
  p.p_tiles = static_cast<int32_t>(ceil_div(P.rows, side));
  p.q_tiles = static_cast<int32_t>(ceil_div(Q.rows, c.bn));
  p.idesc = lin_idesc(in_format, P.mn, Q.mn, side, c.bn);
  if (!encode_operand(&tp, P, 128) || !encode_operand(&tq, Q, c.pair ? c.bn / 2 : c.bn)) return BSGG_ERR_CUDA;
  if (c.pair) return c.bn == 256 ? launch_pair<256>(tp, tq, p, c.split, *dev, s) : launch_pair<128>(tp, tq, p, c.split, *dev, s);
  if (c.bn == 128) return launch_tile<128>(tp, tq, p, c.split, dev->sms, s);
  return c.bn == 64 ? launch_tile<64>(tp, tq, p, c.split, dev->sms, s) : launch_tile<32>(tp, tq, p, c.split, dev->sms, s);
}

template <int KIND, int ACT>
bsgg_status launch_dz_one(const bsgg_linear_bwd_desc* d, const void* dy, const void* z, void* dz, float* dbias,
                          int sms, cudaStream_t s) {
  // two blocks an SM, runs of at least one step of rows, the portable cluster's eight at most
  const int64_t groups = ceil_div(d->n, kDzLanes * 8), steps = ceil_div(d->m, kDzThreads / kDzLanes);
  int64_t runs = 2 * sms / groups;
  runs = runs < 1 ? 1 : runs > kDzSplit ? kDzSplit : runs;
  if (runs > steps) runs = steps;
  const LaunchConfig c(dim3(static_cast<unsigned>(runs * groups)), kDzThreads, 0, s, static_cast<int>(runs));
  return launch_kernel(c, dz_kernel<KIND, ACT>, d->m, d->n, d->ld_dy, d->ldz, d->ld_dz, dy, z, dz, dbias,
                       static_cast<int>(runs));
}
template <int KIND>
bsgg_status launch_dz_kind(const bsgg_linear_bwd_desc* d, const void* dy, const void* z, void* dz, float* dbias,
                           int sms, cudaStream_t s) {
  switch (d->activation) {
    case BSGG_ACT_RELU: return launch_dz_one<KIND, BSGG_ACT_RELU>(d, dy, z, dz, dbias, sms, s);
    case BSGG_ACT_SRELU: return launch_dz_one<KIND, BSGG_ACT_SRELU>(d, dy, z, dz, dbias, sms, s);
    case BSGG_ACT_SILU: return launch_dz_one<KIND, BSGG_ACT_SILU>(d, dy, z, dz, dbias, sms, s);
    case BSGG_ACT_GELU: return launch_dz_one<KIND, BSGG_ACT_GELU>(d, dy, z, dz, dbias, sms, s);
    default: return launch_dz_one<KIND, BSGG_ACT_NONE>(d, dy, z, dz, dbias, sms, s);
  }
}
bsgg_status launch_dz(const bsgg_linear_bwd_desc* d, const void* dy, const void* z, void* dz, float* dbias, cudaStream_t s) {
  const Device* dev = device_state();
  if (!dev) return BSGG_ERR_CUDA;
  const int sms = dev->sms;
  return d->in_format == BSGG_OUT_BF16 ? launch_dz_kind<OK_BF16>(d, dy, z, dz, dbias, sms, s)
                                       : launch_dz_kind<OK_F16>(d, dy, z, dz, dbias, sms, s);
}

bool is_half_format(int f) { return f == BSGG_OUT_BF16 || f == BSGG_OUT_F16; }
bool good_extent(int64_t v) { return v >= 1 && v <= (int64_t(1) << 24); }
bool good_pitch(int64_t ld, int64_t cols, int64_t multiple) {
  return ld >= cols && ld <= (int64_t(1) << 30) && ld % multiple == 0;
}
bool good_act(int a) { return a >= BSGG_ACT_NONE && a <= BSGG_ACT_GELU; }

}  // namespace

extern "C" {

bsgg_status bsgg_linear(const bsgg_linear_desc* d, const void* x, const void* w, const void* bias, const void* residual,
                        void* y, void* z, uint32_t* status, void* stream) {
  if (!d || d->m < 0 || d->m > (int64_t(1) << 24) || !good_extent(d->n) || !good_extent(d->k)) return BSGG_ERR_INVALID_ARG;
  if (!is_half_format(d->in_format) || !is_float_format(d->out_format) || !good_act(d->activation))
    return BSGG_ERR_INVALID_ARG;
  if (!good_pitch(d->ldx, d->k, 8) || !good_pitch(d->ldw, d->k, 8) || !good_pitch(d->ldy, d->n, 1)) return BSGG_ERR_INVALID_ARG;
  if ((residual && !good_pitch(d->ld_residual, d->n, 1)) || (z && !good_pitch(d->ldz, d->n, 1))) return BSGG_ERR_INVALID_ARG;
  if (bias && !is_float_format(d->bias_format)) return BSGG_ERR_INVALID_ARG;
  if (d->m == 0) return BSGG_OK;
  if (!x || !w || !y || !aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(y, float_bytes(d->out_format)) ||
      !aligned_to(residual, 2) || !aligned_to(z, 2) || (bias && !aligned_to(bias, float_bytes(d->bias_format))) ||
      !aligned_to(status, 4))
    return BSGG_ERR_INVALID_ARG;
  LinParams p = {};
  p.act = d->activation; p.out_kind = d->out_format; p.bias_kind = d->bias_format; p.residual_kind = d->in_format;
  p.bias = bias; p.residual = residual; p.ld_residual = d->ld_residual;
  p.out = y; p.ld_out = d->ldy; p.z = z; p.ldz = d->ldz; p.status = status;
  return launch_product({w, d->n, d->k, d->ldw, false}, {x, d->m, d->k, d->ldx, false}, d->in_format, p,
                        static_cast<cudaStream_t>(stream));
}

bsgg_status bsgg_linear_backward(const bsgg_linear_bwd_desc* d, const void* dy, const void* x, const void* w,
                                 const void* z, void* dz, void* dx, void* dw, float* dbias, uint32_t* status,
                                 void* stream) {
  if (!d || d->m < 0 || d->m > (int64_t(1) << 24) || !good_extent(d->n) || !good_extent(d->k)) return BSGG_ERR_INVALID_ARG;
  if (!is_half_format(d->in_format) || !good_act(d->activation) || (d->accumulate_dw != 0 && d->accumulate_dw != 1))
    return BSGG_ERR_INVALID_ARG;
  if ((dx && !is_float_format(d->dx_format)) || (dw && !is_float_format(d->dw_format)) ||
      (!dx && !dw && !dbias && d->m > 0))                    // no rows: an empty dx may be NULL
    return BSGG_ERR_INVALID_ARG;
  const bool has_act = d->activation != BSGG_ACT_NONE;
  if (has_act ? (d->m > 0 && (!z || !dz)) : (z || dz)) return BSGG_ERR_INVALID_ARG;
  if (!good_pitch(d->ld_dy, d->n, 8) || (has_act && (!good_pitch(d->ldz, d->n, 8) || !good_pitch(d->ld_dz, d->n, 8))))
    return BSGG_ERR_INVALID_ARG;
  if ((dx && (!good_pitch(d->ldw, d->k, 8) || !good_pitch(d->ld_dx, d->k, 1))) ||
      (dw && (!good_pitch(d->ldx, d->k, 8) || !good_pitch(d->ld_dw, d->k, 1))))
    return BSGG_ERR_INVALID_ARG;
  if (d->m > 0 && (!dy || (dx && !w) || (dw && !x))) return BSGG_ERR_INVALID_ARG;
  if (!aligned_to(dy, 16) || !aligned_to(z, 16) || !aligned_to(dz, 16) || (dw && !aligned_to(x, 16)) ||
      (dx && !aligned_to(w, 16)) || (dx && !aligned_to(dx, float_bytes(d->dx_format))) ||
      (dw && !aligned_to(dw, float_bytes(d->dw_format))) || !aligned_to(dbias, 4) || !aligned_to(status, 4))
    return BSGG_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->m == 0) {
    // empty sums
    if (dbias && !succeeded(cudaMemsetAsync(dbias, 0, sizeof(float) * d->n, s))) return BSGG_ERR_CUDA;
    const size_t es = float_bytes(d->dw_format);
    if (dw && !d->accumulate_dw && !succeeded(cudaMemset2DAsync(dw, es * d->ld_dw, 0, es * d->k, d->n, s)))
      return BSGG_ERR_CUDA;
    return BSGG_OK;
  }
  if (has_act || dbias) {
    const bsgg_status st = launch_dz(d, dy, z, dz, dbias, s);
    if (st != BSGG_OK) return st;
  }
  const void* g = has_act ? dz : dy;
  const int64_t ldg = has_act ? d->ld_dz : d->ld_dy;
  if (dx) {
    LinParams p = {};
    p.out_kind = d->dx_format; p.out = dx; p.ld_out = d->ld_dx; p.status = status;
    const bsgg_status st = launch_product({w, d->k, d->n, d->ldw, true}, {g, d->m, d->n, ldg, false}, d->in_format, p, s);
    if (st != BSGG_OK) return st;
  }
  if (dw) {
    LinParams p = {};
    p.out_kind = d->dw_format; p.out = dw; p.ld_out = d->ld_dw; p.status = status;
    if (d->accumulate_dw) { p.residual = dw; p.residual_kind = d->dw_format; p.ld_residual = d->ld_dw; }
    const bsgg_status st = launch_product({x, d->k, d->m, d->ldx, true}, {g, d->n, d->m, ldg, true}, d->in_format, p, s);
    if (st != BSGG_OK) return st;
  }
  return BSGG_OK;
}

bsgg_status bsgg_query_status_word(uint32_t* status, void* stream) {
  if (!status) return BSGG_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t w = 0;
  if (!succeeded(cudaMemcpyAsync(&w, status, sizeof(w), cudaMemcpyDeviceToHost, s)) || !succeeded(cudaStreamSynchronize(s)))
    return BSGG_ERR_CUDA;
  if (w != 0) {
    // the bits that were read, no others: another stream's kernel may have set one since
    const LaunchConfig c(dim3(1), 1, 0, s);
    if (launch_kernel(c, clear_bits_kernel, status, w) != BSGG_OK || !succeeded(cudaStreamSynchronize(s))) return BSGG_ERR_CUDA;
  }
  if (w & kStatusTimeout) return BSGG_ERR_DEVICE_TIMEOUT;
  if (w & kStatusBadOffsets) return BSGG_ERR_BAD_OFFSETS;
  return w == 0 ? BSGG_OK : BSGG_ERR_CUDA;
}

}  // extern "C"
