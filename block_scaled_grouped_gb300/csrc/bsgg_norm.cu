// bsgg_norm.cu -- root-mean-square norm with the residual's addition, out in 16 or 32
// bits and as quantized rows of the grouped GEMM's A; and its gradient.
#include <cmath>

#include "bsgg_ops.cuh"

namespace {

using namespace bsgg;

// Values of a row that a thread holds at a time, in two runs of eight, as the block
// quantizer takes them.
constexpr int kNormValues = 16;
constexpr int kNormMaxThreads = 512, kNormWarpRows = 4, kNormPadRows = 8;

struct NormParams {
  int64_t tokens, m_pad;
  int64_t ld_x, ld_residual, ld_h, ld_y;
  int hidden, kq;             // kq: scale words of a row
  int weight_kind, y_kind;
  float eps, inv_hidden;
  const void *x, *residual, *weight;
  void *h, *y;
  float* rstd;
  uint8_t *a, *sfa;
};

// The sum over the threads of a row: a warp's, or (WARP = false) the block's, every
// thread's in the same order.
template <bool WARP>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = warp_sum(v);
  if (WARP) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0f;
  const int warps = blockDim.x >> 5;
  for (int w = 0; w < warps; ++w) v += part[w];
  return v;
}

template <int KIND>
__device__ __forceinline__ float round_to(float v) {
  if (KIND == OK_F32) return v;
  if (KIND == OK_F16) return __half2float(__float2half_rn(v));
  return __bfloat162float(__float2bfloat16_rn(v));
}

// Eight values of a tensor whose type is known at run time only.
__device__ __forceinline__ void load8_as(int kind, const void* base, int64_t i, float* v) {
  float(&r)[8] = *reinterpret_cast<float(*)[8]>(v);
  if (kind == OK_F32) load8<OK_F32>(base, i, r);
  else if (kind == OK_F16) load8<OK_F16>(base, i, r);
  else load8<OK_BF16>(base, i, r);
}
__device__ __forceinline__ void store8_as(int kind, void* base, int64_t i, const float* v) {
  const float(&r)[8] = *reinterpret_cast<const float(*)[8]>(v);
  if (kind == OK_F32) store8<OK_F32>(base, i, r);
  else if (kind == OK_F16) store8<OK_F16>(base, i, r);
  else store8<OK_BF16>(base, i, r);
}

// One row per warp (WARP) or per block; a thread holds NV runs of 16 values from the
// first load to the last store, so that every tensor is passed over once.  FMT: the
// quantized rows' format, BSGG_IN_BF16 for none.  The blocks past the tokens write A's
// padding rows.
//   8192 x 7168 bfloat16 with a residual, into h, y and E4M3 rows: 530 MB in 89 to 91 us, 5.8
//     TB/s, 85 % of the copy rate, bound by the loads' latency and the mix of three writes to
//     two reads (marked as read once 97 us; six blocks an SM with 40 registers 100);
//   128 x 7168: 4.7 us, 333 x 4104 float16: 4.9, of which the launch and two trips to memory
//     are most;
//   8192 x 7168 into y and MXFP4 92 us, NVFP4 105 (4.8 TB/s; without y 95): a division a value.
template <int KIND, int FMT, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kNormWarpRows : kNormMaxThreads)
    rms_norm_kernel(const __grid_constant__ NormParams p) {
  constexpr int V = kNormValues;
  constexpr bool kRows = rf_scaled(FMT);
  constexpr int kLanes = kRows ? rf_vec(FMT) / 16 : 1;
  __shared__ float part[kNormMaxThreads / 32];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int row_bytes = p.hidden / 8 * rf_bits(FMT);
  const int64_t blocks = WARP ? (p.tokens + kNormWarpRows - 1) / kNormWarpRows : p.tokens;
  if (kRows && blockIdx.x >= blocks) {
    const int64_t r0 = p.tokens + (static_cast<int64_t>(blockIdx.x) - blocks) * kNormPadRows;
    constexpr uint32_t one = rf_one(FMT) * 0x01010101u;
    for (int64_t r = r0; r < min(r0 + kNormPadRows, p.m_pad); ++r) {
      uint8_t* row = p.a + r * row_bytes;                // row_bytes is a multiple of 16
      for (int c = threadIdx.x * 16; c < row_bytes; c += blockDim.x * 16) *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
      const int kb = (p.hidden + rf_vec(FMT) - 1) / rf_vec(FMT);
      uint8_t* sf = p.sfa + sf_off(r, 0, p.kq);
      for (int q = threadIdx.x; q < p.kq; q += blockDim.x) {
        const int left = kb - 4 * q;                     // blocks of this word inside hidden
        *reinterpret_cast<uint32_t*>(sf + static_cast<int64_t>(q) * 512) = left >= 4 ? one : one & ((1u << (8 * left)) - 1u);
      }
    }
    return;
  }
  const int lane = threadIdx.x & 31, first = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const int64_t t = WARP ? static_cast<int64_t>(blockIdx.x) * kNormWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && t >= p.tokens) return;
  const bool added = p.residual != nullptr;
  float v[NV][V];
  // all loads before the first use
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (first + i * step) * V;
#pragma unroll
    for (int h = 0; h < V; h += 8) {
      float(&r)[8] = reinterpret_cast<float(&)[8]>(v[i][h]);
      if (c + h < p.hidden) {
        load8<KIND>(p.x, t * p.ld_x + c + h, r);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) r[k] = 0.0f;
      }
    }
  }
  if (added) {
    Raw8<KIND, false> raw[NV][V / 8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int h = 0; h < V / 8; ++h) {
        const int c = (first + i * step) * V + 8 * h;
        raw[i][h].load(p.residual, t * p.ld_residual + c, c < p.hidden);
      }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int h = 0; h < V / 8; ++h) {
        float r[8];
        raw[i][h].values(r);
        // what is normed is what is kept: the backward sees the same h
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][8 * h + k] = round_to<KIND>(v[i][8 * h + k] + r[k]);
      }
  }
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) s = fmaf(v[i][k], v[i][k], s);
    sum += s;
  }
  if (p.h != nullptr) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int h = 0; h < V; h += 8) {
        const int c = (first + i * step) * V + h;
        if (c < p.hidden) store8<KIND>(p.h, t * p.ld_h + c, reinterpret_cast<float(&)[8]>(v[i][h]));
      }
  }
  sum = row_sum<WARP>(sum, part);
  const float rstd = 1.0f / sqrtf(fmaf(sum, p.inv_hidden, p.eps));
  if (p.rstd != nullptr && first == 0) p.rstd[t] = rstd;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (first + i * step) * V;
#pragma unroll
    for (int h = 0; h < V; h += 8) {
      if (c + h >= p.hidden) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][h + k] *= rstd;
      if (p.weight != nullptr) {
        float w[8];
        load8_as(p.weight_kind, p.weight, c + h, w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][h + k] *= w[k];
      }
      if (p.y != nullptr) store8_as(p.y_kind, p.y, t * p.ld_y + c + h, &v[i][h]);
    }
    if constexpr (kRows) {
      const bool in = c < p.hidden;
      uint32_t word = 0, packed[rf_words(FMT)];
      const uint32_t code = block_code<FMT>(v[i], in, word);
      quantize16<FMT>(v[i], code, packed);
      if (lane % (4 * kLanes) == 0 && c < p.kq * 4 * rf_vec(FMT))
        *reinterpret_cast<uint32_t*>(p.sfa + sf_off(t, 0, p.kq) + static_cast<int64_t>(c / (4 * rf_vec(FMT))) * 512) = word;
      if (in) store_codes16<FMT>(p.a + t * row_bytes + c / 8 * rf_bits(FMT), packed, true);
    }
  }
}

struct NormBwdParams {
  int64_t tokens;
  int64_t ld_dy, ld_h, ld_dh, ld_dx;
  int hidden, weight_kind;
  float inv_hidden;
  const void *dy, *h, *weight, *dh;
  const float* rstd;
  void* dx;
  float* part;                // (blocks, hidden) sums of dy * n, with a dweight
};

// A row's dy, h and dh in the registers of their stored form.
template <int KIND, int YKIND, int NV>
struct NormRow {
  Raw8<YKIND, false> dy[NV][2];
  Raw8<KIND, false> h[NV][2], dh[NV][2];
  float rstd;
  __device__ __forceinline__ void load(const NormBwdParams& p, int64_t t, int first, int step) {
    const bool on = t < p.tokens;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = (first + i * step) * kNormValues + 8 * j;
        const bool in = on && c < p.hidden;
        dy[i][j].load(p.dy, t * p.ld_dy + c, in);
        h[i][j].load(p.h, t * p.ld_h + c, in);
        dh[i][j].load(p.dh, t * p.ld_dh + c, in && p.dh != nullptr);
      }
    rstd = on ? p.rstd[t] : 0.0f;
  }
};

// With n = h rstd and g = dy w:  dx = rstd (g - n mean(g n)) + dh,  dweight = sum dy n.
// A block (or each of its warps) walks rows, gridDim apart, its threads holding the
// same columns of each, so that the weight's gradient stays in registers until the
// block's rows are done; the blocks' sums meet in a second launch, in order.  The next
// row is on its way while this one is reduced and written (where registers hold two).
//   8192 x 4096 bfloat16 with dh: 268 MB in 47 to 51 us with that launch, 5.3 TB/s, bound by
//     the loads' latency (without the next row ahead 71, with its loads after the first half
//     of the row's arithmetic 56); float32 99, with 36 to 96 bytes of spills a thread.
//   Above 4096 columns registers hold no row ahead: 8192 x 7168 129 us, 3.6 TB/s, 8192 x 8192 136,
//     float32 7168 228 (up to 116 bytes of spills).  Above 8192 four runs a thread spill up to 600
//     bytes: 4096 x 12288 296 us, 1.4 TB/s, 2048 x 32768 359.
template <int KIND, int YKIND, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kNormWarpRows : NV <= 2 ? 256 : kNormMaxThreads, WARP ? 1 : NV <= 2 ? 2 : 1)
    rms_norm_backward_kernel(const __grid_constant__ NormBwdParams p) {
  constexpr int V = kNormValues;
  constexpr bool kAhead = NV == 1, kKeepWeight = NV == 1;
  // rows too wide for that keep the weight's gradient in shared memory, a thread its own values
  constexpr bool kShared = NV == 4;
  extern __shared__ float4 wide[];
  __shared__ float part[2][kNormMaxThreads / 32];
  __shared__ float warp_sums[WARP ? kNormWarpRows : 1][WARP ? 32 * V * NV : 1];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, first = WARP ? lane : threadIdx.x, step = WARP ? 32 : blockDim.x;
  const int64_t rows = WARP ? kNormWarpRows : 1, row0 = blockIdx.x * rows + (WARP ? threadIdx.x >> 5 : 0);
  auto weight = [&](int i, int j, float (&w)[8]) {
    const int c = (first + i * step) * V + 8 * j;
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = 1.0f;
    if (p.weight != nullptr && c < p.hidden) load8_as(p.weight_kind, p.weight, c, w);
  };
  float acc[kShared ? 1 : NV][V], keep[kKeepWeight ? NV : 1][V];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (kShared) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) wide[(i * 4 + q) * blockDim.x + threadIdx.x] = make_float4(0, 0, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) acc[kShared ? 0 : i][k] = 0.0f;
    }
    if (kKeepWeight) {
#pragma unroll
      for (int j = 0; j < 2; ++j) weight(i, j, reinterpret_cast<float(&)[8]>(keep[i][8 * j]));
    }
  }
  int turn = 0;
  NormRow<KIND, YKIND, NV> row, next;
  if (kAhead) row.load(p, row0, first, step);
  for (int64_t t = row0; t < p.tokens; t += gridDim.x * rows, turn ^= 1) {
    if (!kAhead) row.load(p, t, first, step);
    if (kAhead) next.load(p, t + gridDim.x * rows, first, step);
    const float2 rstd = make_float2(row.rstd, row.rstd);
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float g[8], n[8], w[8];
        row.dy[i][j].values(g);
        row.h[i][j].values(n);
        if (!kKeepWeight) weight(i, j, w);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float* ww = kKeepWeight ? &keep[kKeepWeight ? i : 0][8 * j + k] : &w[k];
          const float2 q = __fmul2_rn(make_float2(g[k], g[k + 1]), __fmul2_rn(make_float2(n[k], n[k + 1]), rstd));
          if (kShared) {
            float2* at = reinterpret_cast<float2*>(&wide[(i * 4 + 2 * j + k / 4) * blockDim.x + threadIdx.x]) + (k & 2) / 2;
            *at = __fadd2_rn(*at, q);
          } else {
            float* at = &acc[kShared ? 0 : i][8 * j + k];
            const float2 a = __fadd2_rn(make_float2(at[0], at[1]), q);
            at[0] = a.x;
            at[1] = a.y;
          }
          sum = __ffma2_rn(q, make_float2(ww[0], ww[1]), sum);
        }
      }
    // two buffers: the next row's sums are written while this row's may still be read
    const float mean = row_sum<WARP>(sum.x + sum.y, part[turn]) * p.inv_hidden;
    const float2 minus = make_float2(-mean, -mean);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int c = (first + i * step) * V + 8 * j;
        if (c >= p.hidden) continue;
        float g[8], n[8], d[8], w[8];
        row.dy[i][j].values(g);
        row.h[i][j].values(n);
        row.dh[i][j].values(d);
        if (!kKeepWeight) weight(i, j, w);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float* ww = kKeepWeight ? &keep[kKeepWeight ? i : 0][8 * j + k] : &w[k];
          const float2 m = __fmul2_rn(make_float2(n[k], n[k + 1]), rstd);
          const float2 u = __ffma2_rn(m, minus, __fmul2_rn(make_float2(g[k], g[k + 1]), make_float2(ww[0], ww[1])));
          const float2 v = __ffma2_rn(u, rstd, make_float2(d[k], d[k + 1]));
          d[k] = v.x;
          d[k + 1] = v.y;
        }
        store8<KIND>(p.dx, t * p.ld_dx + c, d);
      }
    if (kAhead) row = next;
  }
  if (p.part == nullptr) return;
  float* out = p.part + static_cast<int64_t>(blockIdx.x) * p.hidden;
  if constexpr (WARP) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) warp_sums[threadIdx.x >> 5][(lane + 32 * i) * V + k] = acc[kShared ? 0 : i][k];
    __syncthreads();
    for (int c = threadIdx.x; c < p.hidden; c += blockDim.x) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kNormWarpRows; ++w) s += warp_sums[w][c];
      out[c] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; j += 8) {
        const int c = (first + i * step) * V + j;
        if (c >= p.hidden) continue;
        if (kShared) {
#pragma unroll
          for (int q = 0; q < 2; ++q) reinterpret_cast<float4*>(out + c)[q] = wide[(i * 4 + j / 4 + q) * blockDim.x + threadIdx.x];
        } else {
          store8<OK_F32>(out, c, reinterpret_cast<float(&)[8]>(acc[kShared ? 0 : i][j]));
        }
      }
  }
}

// dweight[c] = the sum of the blocks' parts: 32 columns a block, 32 warps that take
// every 32nd part, joined in order: a chain of ten loads (304 parts of 4096: 6 us alone; eight
// warps 8).
constexpr int kNormJoinWarps = 32;
__global__ void __launch_bounds__(32 * kNormJoinWarps) norm_join_kernel(const float* part, int64_t parts, int hidden, float* dweight) {
  __shared__ float sums[kNormJoinWarps][32];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < hidden) {
#pragma unroll 8
    for (int64_t b = warp; b < parts; b += kNormJoinWarps) s += part[b * hidden + c];
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < hidden) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kNormJoinWarps; ++w) s += sums[w][lane];
    dweight[c] = s;
  }
}

// ---------------------------------------------------------------- host
constexpr int64_t kNormMaxHidden = 32768;
// Blocks of the gradient on each of the 152 SMs: two, or as many of fewer threads as 512 hold
// (at 128 registers a thread no more are there at once).  They walk the rows until there are
// none, so that a few more blocks than fit would wait for the first to end and double the time:
// 8192 rows of 7168 took 194 us in 347 blocks and take 129 in 304, 16384 of 1536 55 in 810 and
// 40 in 760.
constexpr int64_t kNormSms = 152, kNormSmThreads = 512;

// How rows of `cols` columns lie: a warp each up to 512, a run of 16 a lane (16384 rows of
// 512, forward 18 us and back 23; in blocks 22 and 62); wider ones a block each, with the
// fewest runs a thread that 256 threads (512 at the most) hold: 16384 rows of 1024 take 29
// and 33 us so, in warps of two runs 31 and 39; 8192 of 7168, forward, 91 us in two runs and
// 96 in one of 512 threads.
struct RowShape {
  bool warp;
  int values, threads;
};
RowShape row_shape(int64_t cols) {
  const int64_t runs = ceil_div(cols, kNormValues);
  if (runs <= 32) return {true, 1, 32 * kNormWarpRows};
  const int nv = runs <= 256 ? 1 : runs <= 512 ? 2 : 4;
  return {false, nv, static_cast<int>(ceil_div(ceil_div(runs, nv), 32) * 32)};
}
template <typename F>
bsgg_status with_shape(const RowShape& s, F&& f) {
  using std::integral_constant;
  if (s.warp) return f(integral_constant<int, 1>(), std::true_type());
  if (s.values == 1) return f(integral_constant<int, 1>(), std::false_type());
  if (s.values == 2) return f(integral_constant<int, 2>(), std::false_type());
  return f(integral_constant<int, 4>(), std::false_type());
}

bool good_rows(int64_t ld, int64_t hidden, int format) {
  return ld >= hidden && ld <= (int64_t(1) << 30) && ld * float_bytes(format) % 16 == 0;
}

bsgg_status check_norm(int64_t tokens, int64_t hidden, int token_format, int weight_format, int y_format) {
  if (tokens < 0 || tokens > (int64_t(1) << 30) || hidden < 8 || hidden % 8 != 0) return BSGG_ERR_INVALID_ARG;
  if (!is_float_format(token_format) || !is_float_format(weight_format) || !is_float_format(y_format))
    return BSGG_ERR_INVALID_ARG;
  return hidden > kNormMaxHidden ? BSGG_ERR_UNSUPPORTED : BSGG_OK;
}

// Calls f with the row format as a constant, BSGG_IN_BF16 standing for none.
template <typename F>
bsgg_status with_quantized(int fmt, F&& f) {
  switch (fmt) {
    case BSGG_IN_MXFP8_E4M3: return f(std::integral_constant<int, BSGG_IN_MXFP8_E4M3>());
    case BSGG_IN_MXFP8_E5M2: return f(std::integral_constant<int, BSGG_IN_MXFP8_E5M2>());
    case BSGG_IN_NVFP4: return f(std::integral_constant<int, BSGG_IN_NVFP4>());
    case BSGG_IN_FP4_UE8M0_16: return f(std::integral_constant<int, BSGG_IN_FP4_UE8M0_16>());
    case BSGG_IN_MXFP4: return f(std::integral_constant<int, BSGG_IN_MXFP4>());
    default: return f(std::integral_constant<int, BSGG_IN_BF16>());
  }
}

int64_t norm_bwd_blocks(int64_t tokens, int64_t hidden) {
  const RowShape shape = row_shape(hidden);
  const int64_t rows = shape.warp ? ceil_div(tokens, kNormWarpRows) : tokens;
  const int64_t each = kNormSmThreads / shape.threads, most = kNormSms * (each < 2 ? 2 : each);
  return rows < most ? rows : most;
}

}  // namespace

extern "C" {

bsgg_status bsgg_rms_norm(const bsgg_norm_desc* d, const void* x, const void* residual, const void* weight, void* h,
                          void* y, float* rstd, void* a, void* sfa, void* stream) {
  if (!d) return BSGG_ERR_INVALID_ARG;
  const bsgg_status st = check_norm(d->tokens, d->hidden, d->token_format, d->weight_format, d->y_format);
  if (st == BSGG_ERR_INVALID_ARG || !std::isfinite(d->eps) || !(d->eps >= 0.0f)) return BSGG_ERR_INVALID_ARG;
  const int tf = d->token_format;
  if (!good_rows(d->ld_x, d->hidden, tf) || (residual && !good_rows(d->ld_residual, d->hidden, tf)) ||
      (h && (!residual || !good_rows(d->ld_h, d->hidden, tf))) || (y && !good_rows(d->ld_y, d->hidden, d->y_format)))
    return BSGG_ERR_INVALID_ARG;
  if (a ? !sfa : sfa != nullptr) return BSGG_ERR_INVALID_ARG;
  if (a) {
    if (d->row_format < BSGG_IN_MXFP8_E4M3 || d->row_format > BSGG_IN_MXFP4 ||
        d->hidden % (rf_fp4(d->row_format) ? 32 : 16) != 0 || d->m_pad <= 0 || d->m_pad % 128 != 0 || d->m_pad < d->tokens ||
        d->m_pad > (int64_t(1) << 30))
      return BSGG_ERR_INVALID_ARG;
  }
  if (d->tokens > 0 && (!x || (!y && !a))) return BSGG_ERR_INVALID_ARG;
  if (!aligned_to(x, 16) || !aligned_to(residual, 16) || !aligned_to(weight, 16) || !aligned_to(h, 16) || !aligned_to(y, 16) ||
      !aligned_to(rstd, 4) || !aligned_to(a, 16) || !aligned_to(sfa, 16))
    return BSGG_ERR_INVALID_ARG;
  if (st != BSGG_OK) return st;
  const RowShape shape = row_shape(d->hidden);
  const int64_t blocks = shape.warp ? ceil_div(d->tokens, kNormWarpRows) : d->tokens;
  const int64_t pads = a ? ceil_div(d->m_pad - d->tokens, kNormPadRows) : 0;
  if (blocks + pads == 0) return BSGG_OK;
  NormParams p = {};
  p.tokens = d->tokens; p.m_pad = d->m_pad; p.ld_x = d->ld_x; p.ld_residual = d->ld_residual; p.ld_h = d->ld_h; p.ld_y = d->ld_y;
  p.hidden = static_cast<int>(d->hidden); p.weight_kind = d->weight_format; p.y_kind = d->y_format;
  p.eps = d->eps; p.inv_hidden = 1.0f / static_cast<float>(d->hidden);
  p.x = x; p.residual = residual; p.weight = weight; p.h = h; p.y = y; p.rstd = rstd;
  p.a = static_cast<uint8_t*>(a); p.sfa = static_cast<uint8_t*>(sfa);
  const LaunchConfig c(dim3(static_cast<unsigned>(blocks + pads)), shape.threads, 0, static_cast<cudaStream_t>(stream));
  return with_float(tf, [&](auto kind) {
    return with_quantized(a ? d->row_format : BSGG_IN_BF16, [&](auto fmt) {
      return with_shape(shape, [&](auto nv, auto warp) {
        constexpr int K = decltype(kind)::value, F = decltype(fmt)::value, N = decltype(nv)::value;
        p.kq = rf_scaled(F) ? static_cast<int>(ceil_div(ceil_div(d->hidden, rf_vec(F)), 4)) : 0;
        return launch_kernel(c, rms_norm_kernel<K, F, N, decltype(warp)::value>, p);
      });
    });
  });
}

uint64_t bsgg_rms_norm_workspace_bytes(int64_t tokens, int64_t hidden) {
  if (check_norm(tokens, hidden, 0, 0, 0) != BSGG_OK) return 0;
  return uint64_t(4) * norm_bwd_blocks(tokens, hidden) * hidden;
}

bsgg_status bsgg_rms_norm_backward(const bsgg_norm_bwd_desc* d, const void* dy, const void* h, const void* weight,
                                   const float* rstd, const void* dh, void* dx, float* dweight, void* workspace,
                                   void* stream) {
  if (!d || d->reserved != 0) return BSGG_ERR_INVALID_ARG;
  const bsgg_status st = check_norm(d->tokens, d->hidden, d->token_format, d->weight_format, d->y_format);
  if (st == BSGG_ERR_INVALID_ARG) return st;
  const int tf = d->token_format;
  if (!good_rows(d->ld_dy, d->hidden, d->y_format) || !good_rows(d->ld_h, d->hidden, tf) ||
      (dh && !good_rows(d->ld_dh, d->hidden, tf)) || !good_rows(d->ld_dx, d->hidden, tf))
    return BSGG_ERR_INVALID_ARG;
  if (d->tokens > 0 && (!dy || !h || !rstd || !dx || (dweight && !workspace))) return BSGG_ERR_INVALID_ARG;
  if (!aligned_to(dy, 16) || !aligned_to(h, 16) || !aligned_to(weight, 16) || !aligned_to(rstd, 4) || !aligned_to(dh, 16) ||
      !aligned_to(dx, 16) || !aligned_to(dweight, 4) || !aligned_to(workspace, 16))
    return BSGG_ERR_INVALID_ARG;
  if (st != BSGG_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int hidden = static_cast<int>(d->hidden);
  if (d->tokens == 0) {
    // an empty sum
    return !dweight || succeeded(cudaMemsetAsync(dweight, 0, sizeof(float) * hidden, s)) ? BSGG_OK : BSGG_ERR_CUDA;
  }
  NormBwdParams p = {};
  p.tokens = d->tokens; p.ld_dy = d->ld_dy; p.ld_h = d->ld_h; p.ld_dh = d->ld_dh; p.ld_dx = d->ld_dx;
  p.hidden = hidden; p.weight_kind = d->weight_format; p.inv_hidden = 1.0f / static_cast<float>(hidden);
  p.dy = dy; p.h = h; p.weight = weight; p.dh = dh; p.rstd = rstd; p.dx = dx;
  p.part = dweight ? static_cast<float*>(workspace) : nullptr;
  const RowShape shape = row_shape(d->hidden);
  const int64_t blocks = norm_bwd_blocks(d->tokens, d->hidden);
  const bsgg_status ran = with_float(tf, [&](auto kind) {
    return with_float(d->y_format, [&](auto ykind) {
      return with_shape(shape, [&](auto nv, auto warp) {
        constexpr int K = decltype(kind)::value, Y = decltype(ykind)::value, N = decltype(nv)::value;
        constexpr auto kernel = rms_norm_backward_kernel<K, Y, N, decltype(warp)::value>;
        const size_t smem = N == 4 ? sizeof(float) * kNormValues * N * shape.threads : 0;       // 128 KB at the most
        if (N == 4 && !allowed<kernel>(static_cast<int>(sizeof(float)) * kNormValues * N * kNormMaxThreads)) return BSGG_ERR_CUDA;
        const LaunchConfig c(dim3(static_cast<unsigned>(blocks)), shape.threads, smem, s);
        return launch_kernel(c, kernel, p);
      });
    });
  });
  if (ran != BSGG_OK || !dweight) return ran;
  const LaunchConfig j(dim3(static_cast<unsigned>(ceil_div(hidden, 32))), 32 * kNormJoinWarps, 0, s);
  return launch_kernel(j, norm_join_kernel, static_cast<const float*>(workspace), blocks, hidden, dweight);
}

}  // extern "C"
