// bsgg_linear.cu -- the dense layer act(x W^T + bias) + residual and its
// gradient.
#include <cudaTypedefs.h>

#include <mutex>

#include "bsgg_linear_kernel.cuh"

namespace {

using namespace bsgg;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// act'(z).  silu: s + z s (1 - s) with 1 - s = s(-z), no cancellation;
// gelu: Phi(z) + z phi(z).
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case BSGG_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case BSGG_ACT_SRELU: return 2.0f * fmaxf(z, 0.0f);
    case BSGG_ACT_SILU: {
      const float s = 1.0f / (1.0f + expf(-z)), c = 1.0f / (1.0f + expf(z));
      return s * (1.0f + z * c);
    }
    case BSGG_ACT_GELU: return normcdff(z) + z * 0.398942280401432678f * expf(-0.5f * z * z);
    default: return 1.0f;
  }
}

// dz = dy act'(z) and dbias, a warp's lanes over 32 columns, the block's 8
// warps over the rows; the 8 partial sums are added in order.
__global__ void __launch_bounds__(256) dz_kernel(int64_t m, int64_t n, int64_t ld_dy, int64_t ldz, int64_t ld_dz, int kind,
                                                 int act, const void* dy, const void* z, void* dz, float* dbias) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float sum = 0.0f;
  if (j < n)
    for (int64_t i = warp; i < m; i += 8) {
      float v = load1(kind, dy, i * ld_dy + j);
      if (z != nullptr) {
        v *= act_slope(act, load1(kind, z, i * ldz + j));
        store1(kind, dz, i * ld_dz + j, v);
      }
      sum += v;
    }
  part[warp][lane] = sum;
  __syncthreads();
  if (dbias != nullptr && warp == 0 && j < n) {
    float s = 0.0f;
    for (int w = 0; w < 8; ++w) s += part[w][lane];
    dbias[j] = s;
  }
}

bsgg_status launch_status() { return cudaGetLastError() == cudaSuccess ? BSGG_OK : BSGG_ERR_CUDA; }

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
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

struct Device {
  int sms = 0;
  bool ok = false;
};

template <typename K>
bool allow_smem(K kern, int bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

// SM count and the kernels' shared-memory limits, once per device.
const Device* device_state() {
  static Device state[64];
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
  std::lock_guard<std::mutex> lk(mu);
  Device& d = state[dev];
  if (!d.ok) {
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return nullptr;
    if (!allow_smem(linear_pair_kernel, LinPair::kSmem) || !allow_smem(linear_tile_kernel<32>, LinTile<32>::kSmem) ||
        !allow_smem(linear_tile_kernel<64>, LinTile<64>::kSmem) || !allow_smem(linear_tile_kernel<128>, LinTile<128>::kSmem))
      return nullptr;
    d.ok = true;
  }
  return &d;
}

uint32_t lin_idesc(int in_format, bool p_mn, bool q_mn, int m, int n) {
  // kind::f16: F32 accumulator (bits 4-5 = 1), F16 (0) or BF16 (1) operands, majorness (1 = MN)
  const uint32_t fmt = in_format == BSGG_OUT_BF16 ? 1u : 0u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | (p_mn ? 1u << 15 : 0u) | (q_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

template <int BN>
cudaError_t launch_tile(const CUtensorMap& tp, const CUtensorMap& tq, const LinParams& p, int split, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(int64_t(p.p_tiles) * p.q_tiles * split), 1, 1);
  cfg.blockDim = dim3(kLinThreads, 1, 1);
  cfg.dynamicSmemBytes = LinTile<BN>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_tile_kernel<BN>, tp, tq, p, split);
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
  const int64_t pair_tiles = ceil_div(P.rows, 256) * ceil_div(Q.rows, 256);
  cudaError_t e;
  if (pair_tiles >= dev->sms / 2 && Q.rows > 128) {
    p.p_tiles = static_cast<int32_t>(ceil_div(P.rows, 256));
    p.q_tiles = static_cast<int32_t>(ceil_div(Q.rows, 256));
    p.idesc = lin_idesc(in_format, P.mn, Q.mn, 256, 256);
    if (!encode_operand(&tp, P, 128) || !encode_operand(&tq, Q, 128)) return BSGG_ERR_CUDA;
    const int64_t units = pair_tiles < dev->sms / 2 ? pair_tiles : dev->sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * units), 1, 1);
    cfg.blockDim = dim3(kLinThreads, 1, 1);
    cfg.dynamicSmemBytes = LinPair::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, linear_pair_kernel, tp, tq, p);
  } else {
    // the instruction's N: the least that holds the output rows (MN-major boxes are 64 wide)
    const int bn = Q.rows <= 32 && !Q.mn ? 32 : Q.rows <= 64 ? 64 : 128;
    p.p_tiles = static_cast<int32_t>(ceil_div(P.rows, 128));
    p.q_tiles = static_cast<int32_t>(ceil_div(Q.rows, bn));
    p.idesc = lin_idesc(in_format, P.mn, Q.mn, 128, bn);
    // split the reduction while the tiles leave SMs idle and every part keeps four blocks
    const int64_t tiles = int64_t(p.p_tiles) * p.q_tiles;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 2 * dev->sms && p.k_blocks >= 8 * split) split *= 2;
    if (!encode_operand(&tp, P, 128) || !encode_operand(&tq, Q, bn)) return BSGG_ERR_CUDA;
    e = bn == 32   ? launch_tile<32>(tp, tq, p, split, s)
        : bn == 64 ? launch_tile<64>(tp, tq, p, split, s)
                   : launch_tile<128>(tp, tq, p, split, s);
  }
  return e == cudaSuccess ? BSGG_OK : BSGG_ERR_CUDA;
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
  if ((dx && !is_float_format(d->dx_format)) || (dw && !is_float_format(d->dw_format)) || (!dx && !dw && !dbias))
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
    if (dbias && cudaMemsetAsync(dbias, 0, sizeof(float) * d->n, s) != cudaSuccess) return BSGG_ERR_CUDA;
    const size_t es = float_bytes(d->dw_format);
    if (dw && !d->accumulate_dw && cudaMemset2DAsync(dw, es * d->ld_dw, 0, es * d->k, d->n, s) != cudaSuccess)
      return BSGG_ERR_CUDA;
    return BSGG_OK;
  }
  if (has_act || dbias) {
    dz_kernel<<<static_cast<unsigned>(ceil_div(d->n, 32)), 256, 0, s>>>(d->m, d->n, d->ld_dy, d->ldz, d->ld_dz, d->in_format,
                                                                       d->activation, dy, z, dz, dbias);
    if (launch_status() != BSGG_OK) return BSGG_ERR_CUDA;
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
  if (cudaMemcpyAsync(&w, status, sizeof(w), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaMemsetAsync(status, 0, sizeof(w), s) != cudaSuccess || cudaStreamSynchronize(s) != cudaSuccess)
    return BSGG_ERR_CUDA;
  if (w & kStatusTimeout) return BSGG_ERR_DEVICE_TIMEOUT;
  if (w & kStatusBadOffsets) return BSGG_ERR_BAD_OFFSETS;
  return w == 0 ? BSGG_OK : BSGG_ERR_CUDA;
}

}  // extern "C"
