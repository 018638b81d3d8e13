// bsgg_tokens.cu -- the operators that lead tokens into the grouped GEMM and
// back: softmax top-k routing, the sort by expert, dispatch (with the block
// quantization of A), combine, and their gradients.
#include "bsgg_ops.cuh"

namespace {

using namespace bsgg;

// ---------------------------------------------------------------- routing
// Order-preserving key of a logit: larger float, larger key; NaN above all;
// -0 = +0.  -inf and below it is kMaskedKey.
constexpr uint32_t kMaskedKey = 0x007FFFFFu;
__device__ __forceinline__ uint32_t logit_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

constexpr int kRouteWarps = 4;

// One warp per token; lane i holds logits i, i + 32, ... in registers.  Each of
// the topk rounds is two warp reductions: the largest key, then the lowest index
// that has it.  NI: registers of logits per lane, ceil(L / 32) rounded up.
template <int NI>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(int64_t tokens, int64_t ld, int L, int topk, int kind,
                                                                 int normalize, const void* logits, int32_t* ids,
                                                                 float* weights) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  uint32_t key[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 32 * i;
    key[i] = e < L ? logit_key(load1(kind, logits, t * ld + e)) : 0u;
  }
  float top = 0.0f, total = 0.0f, mine = 0.0f;   // largest logit; denominator; this lane's choice
  int32_t my_id = -1;
  if (!normalize) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) m = max(m, key[i]);
    const float mx = key_logit(__reduce_max_sync(0xFFFFFFFFu, m));
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (key[i] > kMaskedKey) total += expf(key_logit(key[i]) - mx);
    total = warp_sum(total);
  }
  for (int j = 0; j < topk; ++j) {
    uint32_t m = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < NI; ++i)
      if (key[i] > m) { m = key[i]; at = i; }
    const uint32_t best = __reduce_max_sync(0xFFFFFFFFu, m);
    if (best <= kMaskedKey) break;                 // only masked experts are left
    const uint32_t e = __reduce_min_sync(0xFFFFFFFFu, m == best ? static_cast<uint32_t>(lane + 32 * at) : 0xFFFFFFFFu);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (e == static_cast<uint32_t>(lane + 32 * i)) key[i] = 0u;
    const float v = key_logit(best);
    if (j == 0) top = v;
    const float ev = expf(v - top);
    if (normalize) total += ev;
    if (lane == j) { mine = ev; my_id = static_cast<int32_t>(e); }
  }
  if (lane < topk) {
    ids[t * topk + lane] = my_id;
    weights[t * topk + lane] = my_id < 0 ? 0.0f : mine / total;
  }
}

// One warp per token; lane j < topk holds choice j's id, weight and gradient.
template <int NI>
__global__ void __launch_bounds__(32 * kRouteWarps) route_backward_kernel(
    int64_t tokens, int64_t ld, int L, int topk, int kind, int normalize, const void* logits, const int32_t* ids,
    const float* weights, const float* dweights, const int32_t* row_of_slot, int64_t m_pad, void* dlogits) {
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
  if (t >= tokens) return;
  int32_t id = -1;
  float w = 0.0f, g = 0.0f;
  if (lane < topk) {
    const int64_t s = t * topk + lane;
    id = ids[s];
    if (id >= L) id = -1;
    if (id >= 0) {
      w = weights[s];
      if (row_of_slot != nullptr) {
        const int32_t r = row_of_slot[s];
        g = (r >= 0 && r < m_pad) ? dweights[r] : 0.0f;
      } else {
        g = dweights[s];
      }
    }
  }
  const float inner = warp_sum(w * g);
  float p[NI];
  if (!normalize) {
    float l[NI], mx = -INFINITY, total = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < L ? load1(kind, logits, t * ld + e) : -INFINITY;
      mx = fmaxf(mx, l[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      p[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - mx);
      total += p[i];
    }
    total = warp_sum(total);
    const float r = total > 0.0f ? 1.0f / total : total;    // a row of -inf: every p is 0 (NaN stays)
#pragma unroll
    for (int i = 0; i < NI; ++i) p[i] *= r;
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 32 * i;
    float gi = 0.0f, wi = 0.0f;
    bool chosen = false;
    for (int j = 0; j < topk; ++j) {
      const int32_t idj = __shfl_sync(0xFFFFFFFFu, id, j);
      const float gj = __shfl_sync(0xFFFFFFFFu, g, j), wj = __shfl_sync(0xFFFFFFFFu, w, j);
      if (idj == e) { gi = gj; wi = wj; chosen = true; }
    }
    if (e < L) {
      const float d = normalize ? (chosen ? wi * (gi - inner) : 0.0f) : p[i] * (gi - inner);
      store1(kind, dlogits, t * ld + e, d);
    }
  }
}

// ---------------------------------------------------------------- sort by expert
// A stable counting sort.  Each warp owns a contiguous run of slots, each block
// the runs of its warps in order.  A warp finds the slots of its 32 that name the
// same expert with one match instruction, so a slot's rank is the count before
// its run plus the run's own before it: no order depends on timing.
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32;

struct SortParams {
  int64_t slots, m_pad;
  int L, steps, blocks;          // 32-slot steps per warp
  const int32_t* ids;
  const float* weights;
  int32_t *offsets, *row_of_slot, *slot_of_row, *rows_used;
  float* prob;
  int32_t* counts;               // (blocks, L)
  uint32_t* status;
};

__device__ __forceinline__ int sort_id(const SortParams& p, int64_t s) {
  const int32_t e = s < p.slots ? p.ids[s] : -1;
  return (e >= 0 && e < p.L) ? e : -1;
}

// Per-warp counts of this block's slots into cnt[warp][L] (cleared here).
__device__ __forceinline__ void sort_count(const SortParams& p, int32_t* cnt, int block) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * p.L; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t s0 = (static_cast<int64_t>(block) * kSortWarps + warp) * p.steps * 32;
  for (int k = 0; k < p.steps; ++k) {
    const int e = sort_id(p, s0 + 32 * k + lane);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    if (e >= 0 && lane == __ffs(same) - 1) cnt[warp * p.L + e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortParams p) {
  extern __shared__ int32_t sm[];
  sort_count(p, sm, blockIdx.x);
  for (int e = threadIdx.x; e < p.L; e += kSortThreads) {
    int32_t c = 0;
    for (int w = 0; w < kSortWarps; ++w) c += sm[w * p.L + e];
    p.counts[static_cast<int64_t>(blockIdx.x) * p.L + e] = c;
  }
}

// Rows of every slot: shared memory holds cnt[warps][L], then total[L] and
// first[L + 1] (an expert's first row).
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortParams p) {
  extern __shared__ int32_t sm[];
  int32_t* cnt = sm;
  int32_t* total = sm + kSortWarps * p.L;
  int32_t* first = total + p.L;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  sort_count(p, cnt, blockIdx.x);
  for (int e = threadIdx.x; e < p.L; e += kSortThreads) {
    int32_t all = 0, before = 0;
    if (p.blocks == 1) {
      for (int w = 0; w < kSortWarps; ++w) all += cnt[w * p.L + e];
    } else {
      for (int b = 0; b < p.blocks; ++b) {
        const int32_t c = p.counts[static_cast<int64_t>(b) * p.L + e];
        all += c;
        before += b < static_cast<int>(blockIdx.x) ? c : 0;
      }
    }
    total[e] = all;
    // per-warp starts inside the expert
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t c = cnt[w * p.L + e];
      cnt[w * p.L + e] = before;
      before += c;
    }
  }
  __syncthreads();
  if (warp == 0) {
    // exclusive prefix of the padded sizes, one contiguous chunk per lane
    const int chunk = (p.L + 31) / 32, e0 = min(lane * chunk, p.L), e1 = min(e0 + chunk, p.L);
    int32_t local = 0;
    for (int e = e0; e < e1; ++e) local += (total[e] + 127) / 128 * 128;
    int32_t incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += y;
    }
    int32_t run = incl - local;
    for (int e = e0; e < e1; ++e) {
      first[e] = run;
      run += (total[e] + 127) / 128 * 128;
    }
    if (lane == 31) first[p.L] = incl;
  }
  __syncthreads();
  const int32_t m_pad = static_cast<int32_t>(p.m_pad);
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e < p.L; e += kSortThreads)
      p.offsets[e] = e + 1 == p.L ? m_pad : min(first[e + 1], m_pad);
    if (threadIdx.x == 0) {
      if (p.rows_used != nullptr) *p.rows_used = first[p.L];
      if (first[p.L] > m_pad && p.status != nullptr) atomicOr(p.status, kStatusBadOffsets);
    }
  }
  // padding rows: between an expert's last slot and the next expert, and after
  // the last expert up to m_pad; a warp per expert, the tail over all threads
  for (int e = blockIdx.x * kSortWarps + warp; e < p.L; e += gridDim.x * kSortWarps) {
    for (int32_t r = first[e] + total[e] + lane; r < min(first[e + 1], m_pad); r += 32) {
      p.slot_of_row[r] = -1;
      if (p.prob != nullptr) p.prob[r] = 0.0f;
    }
  }
  for (int64_t r = first[p.L] + static_cast<int64_t>(blockIdx.x) * kSortThreads + threadIdx.x; r < m_pad;
       r += static_cast<int64_t>(gridDim.x) * kSortThreads) {
    p.slot_of_row[r] = -1;
    if (p.prob != nullptr) p.prob[r] = 0.0f;
  }
  // the slots
  const int64_t s0 = (static_cast<int64_t>(blockIdx.x) * kSortWarps + warp) * p.steps * 32;
  for (int k = 0; k < p.steps; ++k) {
    const int64_t s = s0 + 32 * k + lane;
    const int e = sort_id(p, s);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    int32_t r = -1;
    if (e >= 0) {
      r = first[e] + cnt[warp * p.L + e] + __popc(same & ((1u << lane) - 1u));
      if (r >= m_pad) r = -1;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) cnt[warp * p.L + e] += __popc(same);
    __syncwarp();
    if (s < p.slots) {
      p.row_of_slot[s] = r;
      if (r >= 0) {
        p.slot_of_row[r] = static_cast<int32_t>(s);
        if (p.prob != nullptr) p.prob[r] = p.weights != nullptr ? p.weights[s] : 1.0f;
      }
    }
  }
}

// ---------------------------------------------------------------- dispatch
struct RowsParams {
  int64_t tokens, hidden, m_pad, ld_token, ld_residual;
  int topk;
  int64_t kq;                       // scale atoms per 128 rows
  const void* x;                    // x or dy
  const int32_t *row_of_slot, *slot_of_row;
  const float* weights;
  void* a;
  uint8_t* sfa;
};

constexpr int kRowThreads = 256;

// One block per row of A: gather, scale by the slot's weight, quantize.  Lanes
// hold eight values each, so a block of v values is v / 8 neighbouring lanes.
template <int KIND, int FMT>
__global__ void __launch_bounds__(kRowThreads) dispatch_row_kernel(RowsParams p) {
  const int64_t r = blockIdx.x;
  const int32_t s = p.slot_of_row[r];
  const bool real = s >= 0 && s < p.tokens * p.topk;
  const int64_t t = real ? s / p.topk : 0;
  const float w = real && p.weights != nullptr ? p.weights[s] : 1.0f;
  constexpr int kLanes = rf_vec(FMT) / 8;
  const int64_t cols = rf_scaled(FMT) ? p.kq * 4 * rf_vec(FMT) : p.hidden;
  for (int64_t c = threadIdx.x * 8; c < (cols + 255) / 256 * 256; c += kRowThreads * 8) {
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (real && c < p.hidden) load8<KIND>(p.x, t * p.ld_token + c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = p.weights != nullptr ? v[k] * w : v[k];
    uint32_t code = 0;
    if (rf_scaled(FMT)) {
      uint32_t m = max_abs_bits8(v);
#pragma unroll
      for (int o = 1; o < kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      code = scale_code<FMT>(m);
      if (threadIdx.x % kLanes == 0 && c < cols)
        p.sfa[sf_off(r, c / rf_vec(FMT), p.kq)] = static_cast<uint8_t>(c < p.hidden ? code : 0u);
    }
    if (c < p.hidden) {
      uint32_t out[4];
      quantize8<FMT>(v, code, out);
      store_codes8<FMT>(p.a, r * p.hidden + c, out);
    }
  }
}

// ---------------------------------------------------------------- combine
struct CombineParams {
  int64_t tokens, hidden, m_pad, ld_token, ld_residual;
  int topk;
  const void* d;
  const int32_t* row_of_slot;
  const float* weights;
  const void* residual;
  void* y;
};

template <int DK, int KIND>
__global__ void __launch_bounds__(kRowThreads) combine_kernel(CombineParams p) {
  const int64_t t = blockIdx.x;
  for (int64_t c = threadIdx.x * 8; c < p.hidden; c += kRowThreads * 8) {
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (p.residual != nullptr) load8<KIND>(p.residual, t * p.ld_residual + c, acc);
    for (int j = 0; j < p.topk; ++j) {
      const int64_t s = t * p.topk + j;
      const int32_t r = p.row_of_slot[s];
      if (r < 0 || r >= p.m_pad) continue;
      const float w = p.weights != nullptr ? p.weights[s] : 1.0f;
      float v[8];
      load8<DK>(p.d, r * p.hidden + c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, v[k], acc[k]);
    }
    store8<KIND>(p.y, t * p.ld_token + c, acc);
  }
}

// dweights: one warp per slot.
template <int DK, int KIND>
__global__ void __launch_bounds__(kRowThreads) dweights_kernel(int64_t tokens, int64_t hidden, int64_t m_pad,
                                                               int64_t ld_token, int topk, const void* dy,
                                                               const void* d, const int32_t* row_of_slot,
                                                               float* dweights) {
  const int lane = threadIdx.x & 31;
  const int64_t s = static_cast<int64_t>(blockIdx.x) * (kRowThreads / 32) + (threadIdx.x >> 5);
  if (s >= tokens * topk) return;
  const int64_t t = s / topk;
  const int32_t r = row_of_slot[s];
  float acc = 0.0f;
  if (r >= 0 && r < m_pad) {
    for (int64_t c = lane * 8; c < hidden; c += 256) {
      float u[8], v[8];
      load8<KIND>(dy, t * ld_token + c, u);
      load8<DK>(d, r * hidden + c, v);
#pragma unroll
      for (int k = 0; k < 8; ++k) acc = fmaf(u[k], v[k], acc);
    }
  }
  acc = warp_sum(acc);
  if (lane == 0) dweights[s] = acc;
}

// ---------------------------------------------------------------- host
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bsgg_status launch_status() { return cudaGetLastError() == cudaSuccess ? BSGG_OK : BSGG_ERR_CUDA; }

bsgg_status check_route(const bsgg_route_desc* d) {
  if (!d || d->tokens < 0 || d->tokens > (int64_t(1) << 30) || d->num_experts < 1 || d->num_experts > 1024)
    return BSGG_ERR_INVALID_ARG;
  if (d->topk < 1 || d->topk > 32 || d->topk > d->num_experts || d->ld < d->num_experts || d->ld > (int64_t(1) << 30))
    return BSGG_ERR_INVALID_ARG;
  if (!is_float_format(d->logit_format) || (d->normalize != 0 && d->normalize != 1)) return BSGG_ERR_INVALID_ARG;
  return BSGG_OK;
}

// Registers of logits per lane: the least power of two times 32 that holds L.
template <typename F>
void with_route_regs(int L, F&& f) {
  if (L <= 32) f(std::integral_constant<int, 1>());
  else if (L <= 64) f(std::integral_constant<int, 2>());
  else if (L <= 128) f(std::integral_constant<int, 4>());
  else if (L <= 256) f(std::integral_constant<int, 8>());
  else if (L <= 512) f(std::integral_constant<int, 16>());
  else f(std::integral_constant<int, 32>());
}

// Calls f with the format (f: bf16, f16, f32) as a constant.
template <typename F>
bsgg_status with_float(int fmt, F&& f) {
  switch (fmt) {
    case BSGG_OUT_BF16: return f(std::integral_constant<int, OK_BF16>());
    case BSGG_OUT_F16: return f(std::integral_constant<int, OK_F16>());
    default: return f(std::integral_constant<int, OK_F32>());
  }
}
template <typename F>
bsgg_status with_rows(int fmt, F&& f) {
  switch (fmt) {
    case BSGG_IN_MXFP8_E4M3: return f(std::integral_constant<int, BSGG_IN_MXFP8_E4M3>());
    case BSGG_IN_MXFP8_E5M2: return f(std::integral_constant<int, BSGG_IN_MXFP8_E5M2>());
    case BSGG_IN_NVFP4: return f(std::integral_constant<int, BSGG_IN_NVFP4>());
    case BSGG_IN_FP4_UE8M0_16: return f(std::integral_constant<int, BSGG_IN_FP4_UE8M0_16>());
    case BSGG_IN_MXFP4: return f(std::integral_constant<int, BSGG_IN_MXFP4>());
    case BSGG_ROW_F16: return f(std::integral_constant<int, BSGG_ROW_F16>());
    default: return f(std::integral_constant<int, BSGG_IN_BF16>());
  }
}

// What dispatch, combine and combine_backward share.
bsgg_status check_tokens(const bsgg_tokens_desc* d, bool quantizes, bool reads_d) {
  if (!d || d->tokens < 0 || d->tokens > (int64_t(1) << 30) || d->hidden < 8 || d->hidden % 8 != 0 ||
      d->hidden > (int64_t(1) << 24) || d->topk < 1 || d->tokens * d->topk >= (int64_t(1) << 31))
    return BSGG_ERR_INVALID_ARG;
  if (d->m_pad <= 0 || d->m_pad % 128 != 0 || d->m_pad > (int64_t(1) << 30)) return BSGG_ERR_INVALID_ARG;
  if (!is_float_format(d->token_format)) return BSGG_ERR_INVALID_ARG;
  if (d->ld_token < d->hidden || d->ld_token > (int64_t(1) << 30) || d->ld_token * float_bytes(d->token_format) % 16 != 0)
    return BSGG_ERR_INVALID_ARG;
  if (quantizes) {
    if (d->row_format < BSGG_IN_MXFP8_E4M3 || d->row_format > BSGG_ROW_F16) return BSGG_ERR_INVALID_ARG;
    if (d->hidden % (rf_fp4(d->row_format) ? 32 : rf_scaled(d->row_format) ? 16 : 8) != 0) return BSGG_ERR_INVALID_ARG;
  }
  if (reads_d && !is_float_format(d->d_format)) return BSGG_ERR_INVALID_ARG;
  return BSGG_OK;
}

bsgg_status launch_rows(const bsgg_tokens_desc* d, const void* x, const int32_t* row_of_slot, const int32_t* slot_of_row,
                        const float* weights, void* a, void* sfa, cudaStream_t s) {
  RowsParams p = {};
  p.tokens = d->tokens; p.hidden = d->hidden; p.m_pad = d->m_pad; p.ld_token = d->ld_token; p.topk = d->topk;
  p.x = x; p.row_of_slot = row_of_slot; p.slot_of_row = slot_of_row; p.weights = weights;
  p.a = a; p.sfa = static_cast<uint8_t*>(sfa);
  return with_float(d->token_format, [&](auto kind) {
    return with_rows(d->row_format, [&](auto fmt) {
      constexpr int K = decltype(kind)::value, F = decltype(fmt)::value;
      p.kq = rf_scaled(F) ? ceil_div(ceil_div(d->hidden, rf_vec(F)), 4) : 0;
      dispatch_row_kernel<K, F><<<static_cast<unsigned>(d->m_pad), kRowThreads, 0, s>>>(p);
      return launch_status();
    });
  });
}

}  // namespace

extern "C" {

bsgg_status bsgg_route(const bsgg_route_desc* d, const void* logits, int32_t* ids, float* weights, void* stream) {
  const bsgg_status st = check_route(d);
  if (st != BSGG_OK) return st;
  if (d->tokens == 0) return BSGG_OK;
  if (!logits || !ids || !weights || !aligned_to(logits, float_bytes(d->logit_format)) || !aligned_to(ids, 4) ||
      !aligned_to(weights, 4))
    return BSGG_ERR_INVALID_ARG;
  const unsigned grid = static_cast<unsigned>(ceil_div(d->tokens, kRouteWarps));
  with_route_regs(d->num_experts, [&](auto ni) {
    route_kernel<decltype(ni)::value><<<grid, 32 * kRouteWarps, 0, static_cast<cudaStream_t>(stream)>>>(
        d->tokens, d->ld, d->num_experts, d->topk, d->logit_format, d->normalize, logits, ids, weights);
  });
  return launch_status();
}

bsgg_status bsgg_route_backward(const bsgg_route_desc* d, const void* logits, const int32_t* ids, const float* weights,
                                const float* dweights, const int32_t* row_of_slot, int64_t m_pad, void* dlogits,
                                void* stream) {
  const bsgg_status st = check_route(d);
  if (st != BSGG_OK) return st;
  if (row_of_slot && (m_pad <= 0 || m_pad > (int64_t(1) << 30))) return BSGG_ERR_INVALID_ARG;
  if (d->tokens == 0) return BSGG_OK;
  const uintptr_t es = float_bytes(d->logit_format);
  if (!logits || !ids || !weights || !dweights || !dlogits || !aligned_to(logits, es) || !aligned_to(dlogits, es) ||
      !aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4) || !aligned_to(row_of_slot, 4))
    return BSGG_ERR_INVALID_ARG;
  const unsigned grid = static_cast<unsigned>(ceil_div(d->tokens, kRouteWarps));
  with_route_regs(d->num_experts, [&](auto ni) {
    route_backward_kernel<decltype(ni)::value><<<grid, 32 * kRouteWarps, 0, static_cast<cudaStream_t>(stream)>>>(
        d->tokens, d->ld, d->num_experts, d->topk, d->logit_format, d->normalize, logits, ids, weights, dweights,
        row_of_slot, m_pad, dlogits);
  });
  return launch_status();
}

int64_t bsgg_sort_rows(int64_t slots, int32_t num_experts) {
  if (slots < 0 || slots >= (int64_t(1) << 31) || num_experts < 1 || num_experts > 1024) return -1;
  // the most that sizes adding up to `slots` can need: as many experts as can
  // be, each one slot past a multiple of 128 (one block of rows for no slots)
  const int64_t some = slots < num_experts ? slots : num_experts;
  const int64_t blocks = some + (slots - some) / 128;
  return 128 * (blocks > 0 ? blocks : 1);
}

// Blocks of the sort: one while a block's warps hold the slots in a few steps,
// else as many as give every warp the same run, at most kSortBlocks.
static int64_t sort_steps(int64_t slots) {
  constexpr int64_t kOneBlock = 8, kSortBlocks = 148;
  const int64_t per_step = 32 * kSortWarps;
  const int64_t steps = ceil_div(slots, per_step);
  return steps <= kOneBlock ? (steps > 0 ? steps : 1) : (ceil_div(steps, kSortBlocks) > 4 ? ceil_div(steps, kSortBlocks) : 4);
}
static int64_t sort_blocks(int64_t slots) {
  const int64_t b = ceil_div(slots, sort_steps(slots) * 32 * kSortWarps);
  return b > 0 ? b : 1;
}

uint64_t bsgg_sort_workspace_bytes(int64_t slots, int32_t num_experts) {
  if (bsgg_sort_rows(slots, num_experts) < 0) return 0;
  const int64_t b = sort_blocks(slots);
  return b > 1 ? uint64_t(4) * b * num_experts : 0;
}

bsgg_status bsgg_sort_tokens(int64_t slots, int32_t num_experts, int64_t m_pad, const int32_t* ids, const float* weights,
                             int32_t* padded_offsets, int32_t* row_of_slot, int32_t* slot_of_row, float* prob,
                             int32_t* rows_used, void* workspace, uint32_t* status, void* stream) {
  if (bsgg_sort_rows(slots, num_experts) < 0) return BSGG_ERR_INVALID_ARG;
  if (m_pad <= 0 || m_pad % 128 != 0 || m_pad > (int64_t(1) << 30)) return BSGG_ERR_INVALID_ARG;
  if ((slots > 0 && (!ids || !row_of_slot)) || !padded_offsets || !slot_of_row) return BSGG_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(ids), static_cast<const void*>(weights),
                        static_cast<const void*>(padded_offsets), static_cast<const void*>(row_of_slot),
                        static_cast<const void*>(slot_of_row), static_cast<const void*>(prob),
                        static_cast<const void*>(rows_used), static_cast<const void*>(workspace),
                        static_cast<const void*>(status)})
    if (!aligned_to(q, 4)) return BSGG_ERR_INVALID_ARG;
  SortParams p = {};
  p.slots = slots; p.m_pad = m_pad; p.L = num_experts;
  p.steps = static_cast<int>(sort_steps(slots));
  p.blocks = static_cast<int>(sort_blocks(slots));
  if (p.blocks > 1 && !workspace) return BSGG_ERR_INVALID_ARG;
  p.ids = ids; p.weights = weights; p.offsets = padded_offsets; p.row_of_slot = row_of_slot; p.slot_of_row = slot_of_row;
  p.rows_used = rows_used; p.prob = prob; p.counts = static_cast<int32_t*>(workspace); p.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.blocks > 1) {
    sort_count_kernel<<<p.blocks, kSortThreads, sizeof(int32_t) * kSortWarps * p.L, s>>>(p);
    if (launch_status() != BSGG_OK) return BSGG_ERR_CUDA;
  }
  sort_place_kernel<<<p.blocks, kSortThreads, sizeof(int32_t) * ((kSortWarps + 2) * p.L + 1), s>>>(p);
  return launch_status();
}

bsgg_status bsgg_dispatch(const bsgg_tokens_desc* d, const void* x, const int32_t* row_of_slot,
                          const int32_t* slot_of_row, void* a, void* sfa, void* stream) {
  const bsgg_status st = check_tokens(d, true, false);
  if (st != BSGG_OK) return st;
  if ((d->tokens > 0 && (!x || !row_of_slot)) || !slot_of_row || !a || (rf_scaled(d->row_format) ? !sfa : sfa != nullptr))
    return BSGG_ERR_INVALID_ARG;
  if (!aligned_to(x, 16) || !aligned_to(a, 16) || !aligned_to(sfa, 16) || !aligned_to(row_of_slot, 4) ||
      !aligned_to(slot_of_row, 4))
    return BSGG_ERR_INVALID_ARG;
  return launch_rows(d, x, row_of_slot, slot_of_row, nullptr, a, sfa, static_cast<cudaStream_t>(stream));
}

bsgg_status bsgg_combine(const bsgg_tokens_desc* d, const void* dd, const int32_t* row_of_slot, const float* weights,
                         const void* residual, void* y, void* stream) {
  const bsgg_status st = check_tokens(d, false, true);
  if (st != BSGG_OK) return st;
  if (residual && (d->ld_residual < d->hidden || d->ld_residual > (int64_t(1) << 30) ||
                   d->ld_residual * float_bytes(d->token_format) % 16 != 0))
    return BSGG_ERR_INVALID_ARG;
  if (d->tokens == 0) return BSGG_OK;
  if (!dd || !row_of_slot || !y || !aligned_to(dd, 16) || !aligned_to(residual, 16) || !aligned_to(y, 16) ||
      !aligned_to(row_of_slot, 4) || !aligned_to(weights, 4))
    return BSGG_ERR_INVALID_ARG;
  CombineParams p = {d->tokens, d->hidden, d->m_pad, d->ld_token, d->ld_residual, d->topk, dd, row_of_slot, weights,
                     residual, y};
  return with_float(d->d_format, [&](auto dk) {
    return with_float(d->token_format, [&](auto kind) {
      combine_kernel<decltype(dk)::value, decltype(kind)::value>
          <<<static_cast<unsigned>(d->tokens), kRowThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
      return launch_status();
    });
  });
}

bsgg_status bsgg_combine_backward(const bsgg_tokens_desc* d, const void* dy, const void* rows,
                                  const int32_t* row_of_slot, const int32_t* slot_of_row, const float* weights, void* dd,
                                  void* sfd, float* dweights, void* stream) {
  const bsgg_status st = check_tokens(d, dd != nullptr, dweights != nullptr);
  if (st != BSGG_OK) return st;
  if (!dd && !dweights) return BSGG_ERR_INVALID_ARG;
  if (d->tokens > 0 && (!dy || !row_of_slot || (dweights && !rows))) return BSGG_ERR_INVALID_ARG;
  if (dd ? (!slot_of_row || (rf_scaled(d->row_format) ? !sfd : sfd != nullptr)) : sfd != nullptr)
    return BSGG_ERR_INVALID_ARG;
  if (!aligned_to(dy, 16) || !aligned_to(rows, 16) || !aligned_to(dd, 16) || !aligned_to(sfd, 16) ||
      !aligned_to(row_of_slot, 4) || !aligned_to(slot_of_row, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4))
    return BSGG_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dd) {
    const bsgg_status r = launch_rows(d, dy, row_of_slot, slot_of_row, weights, dd, sfd, s);
    if (r != BSGG_OK) return r;
  }
  if (!dweights || d->tokens == 0) return BSGG_OK;
  return with_float(d->d_format, [&](auto dk) {
    return with_float(d->token_format, [&](auto kind) {
      dweights_kernel<decltype(dk)::value, decltype(kind)::value>
          <<<static_cast<unsigned>(ceil_div(d->tokens * d->topk, kRowThreads / 32)), kRowThreads, 0, s>>>(
              d->tokens, d->hidden, d->m_pad, d->ld_token, d->topk, dy, rows, row_of_slot, dweights);
      return launch_status();
    });
  });
}

}  // extern "C"
