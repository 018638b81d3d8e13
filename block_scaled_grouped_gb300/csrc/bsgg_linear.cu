// bsgg_linear.cu -- the dense layer act(x W^T + bias) + residual and its
// gradient.
#include "bsgg_ops.cuh"

namespace {

using namespace bsgg;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// act(z).  silu = z / (1 + e^-z); gelu = z Phi(z) with Phi from normcdff,
// which keeps its relative accuracy in the lower tail where 1 + erf cancels.
__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case BSGG_ACT_RELU: return z <= 0.0f ? 0.0f : z;               // a NaN stays
    case BSGG_ACT_SRELU: return z <= 0.0f ? 0.0f : z * z;
    case BSGG_ACT_SILU: return z / (1.0f + expf(-z));
    case BSGG_ACT_GELU: return z * normcdff(z);
    default: return z;
  }
}
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

// C[i, j] = sum_r A(i, r) B(j, r): operand elements at i * s_i + r * s_r.
struct MatParams {
  int64_t rows, cols, depth;
  const void *a, *b;
  int64_t a_i, a_r, b_j, b_r;
  int in_kind, out_kind, bias_kind, act;
  const void* bias;          // by column
  const void* residual;
  int residual_kind;
  int64_t ld_residual;
  void* out;
  int64_t ld_out;
  void* z;
  int64_t ldz;
};

__device__ __forceinline__ void finish(const MatParams& p, int64_t i, int64_t j, float v) {
  if (p.bias != nullptr) v += load1(p.bias_kind, p.bias, j);
  if (p.z != nullptr) store1(p.in_kind, p.z, i * p.ldz + j, v);
  v = act_value(p.act, v);
  if (p.residual != nullptr) v += load1(p.residual_kind, p.residual, i * p.ld_residual + j);
  store1(p.out_kind, p.out, i * p.ld_out + j, v);
}

constexpr int kTile = 64, kDepth = 16;

// A 64 x 64 tile per block of 256 threads, 4 x 4 values each, over depth 16
// slices in shared memory.
__global__ void __launch_bounds__(256) mat_kernel(MatParams p) {
  __shared__ float sa[kDepth][kTile + 1], sb[kDepth][kTile + 1];
  const int64_t i0 = static_cast<int64_t>(blockIdx.y) * kTile, j0 = static_cast<int64_t>(blockIdx.x) * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int64_t r0 = 0; r0 < p.depth; r0 += kDepth) {
    for (int e = threadIdx.x; e < kTile * kDepth; e += 256) {
      const int i = e / kDepth, r = e % kDepth;
      const bool in = r0 + r < p.depth;
      sa[r][i] = in && i0 + i < p.rows ? load1(p.in_kind, p.a, (i0 + i) * p.a_i + (r0 + r) * p.a_r) : 0.0f;
      sb[r][i] = in && j0 + i < p.cols ? load1(p.in_kind, p.b, (j0 + i) * p.b_j + (r0 + r) * p.b_r) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kDepth; ++r)
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[u][v] = fmaf(sa[r][ty + 16 * u], sb[r][tx + 16 * v], acc[u][v]);
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t i = i0 + ty + 16 * u, j = j0 + tx + 16 * v;
      if (i < p.rows && j < p.cols) finish(p, i, j, acc[u][v]);
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

bsgg_status launch_mat(const MatParams& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(p.cols, kTile)), static_cast<unsigned>(ceil_div(p.rows, kTile)));
  mat_kernel<<<grid, 256, 0, s>>>(p);
  return launch_status();
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
  MatParams p = {};
  p.rows = d->m; p.cols = d->n; p.depth = d->k;
  p.a = x; p.a_i = d->ldx; p.a_r = 1;
  p.b = w; p.b_j = d->ldw; p.b_r = 1;
  p.in_kind = d->in_format; p.out_kind = d->out_format; p.bias_kind = d->bias_format; p.act = d->activation;
  p.bias = bias; p.residual = residual; p.residual_kind = d->in_format; p.ld_residual = d->ld_residual;
  p.out = y; p.ld_out = d->ldy; p.z = z; p.ldz = d->ldz;
  return launch_mat(p, static_cast<cudaStream_t>(stream));
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
    MatParams p = {};
    p.rows = d->m; p.cols = d->k; p.depth = d->n;
    p.a = g; p.a_i = ldg; p.a_r = 1;
    p.b = w; p.b_j = 1; p.b_r = d->ldw;
    p.in_kind = d->in_format; p.out_kind = d->dx_format;
    p.out = dx; p.ld_out = d->ld_dx;
    if (launch_mat(p, s) != BSGG_OK) return BSGG_ERR_CUDA;
  }
  if (dw) {
    MatParams p = {};
    p.rows = d->n; p.cols = d->k; p.depth = d->m;
    p.a = g; p.a_i = 1; p.a_r = ldg;
    p.b = x; p.b_j = 1; p.b_r = d->ldx;
    p.in_kind = d->in_format; p.out_kind = d->dw_format;
    p.out = dw; p.ld_out = d->ld_dw;
    if (d->accumulate_dw) { p.residual = dw; p.residual_kind = d->dw_format; p.ld_residual = d->ld_dw; }
    if (launch_mat(p, s) != BSGG_OK) return BSGG_ERR_CUDA;
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
