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
// the topk rounds is two warp reductions (single instructions on integers, hence the
// keys): the largest key, then the lowest index that has it.  The weights need no
// second pass: the first choice is the maximum, and every lane sees each chosen
// logit.  NI: registers of logits per lane, ceil(L / 32) rounded up.
// What takes the time is this loop's issue (56 % of the slots) and the first load's
// latency, not the bytes: 16384 x 128 float32, top-4 (8.4 MB, 1.2 us of them) takes
// 6 us, 128 x 64 top-8 2 us.
template <int NI>
__global__ void __launch_bounds__(32 * kRouteWarps) route_kernel(int64_t tokens, int64_t ld, int L, int topk, int kind,
                                                                 int normalize, const void* logits, int32_t* ids,
                                                                 float* weights) {
  let_next_kernel_start();
  wait_for_previous_kernel();
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

// One warp per token; lane j < topk holds choice j's id, weight and gradient, which
// go round one by one, every lane looking for the expert among its own.  Logits are
// read only where the softmax runs over all of them.  16384 x 128, top-4: 6 us,
// bound as the forward is.
template <int NI>
__global__ void __launch_bounds__(32 * kRouteWarps) route_backward_kernel(
    int64_t tokens, int64_t ld, int L, int topk, int kind, int normalize, const void* logits, const int32_t* ids,
    const float* weights, const float* dweights, const int32_t* row_of_slot, int64_t m_pad, void* dlogits) {
  let_next_kernel_start();
  wait_for_previous_kernel();
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
  // each expert's gradient: choice by choice, every lane looking for it among its own
  float gi[NI], wi[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) gi[i] = wi[i] = 0.0f;
  uint32_t chosen = 0;
  for (int j = 0; j < topk; ++j) {
    const int32_t at = __shfl_sync(0xFFFFFFFFu, id, j) - lane;
    const float gj = __shfl_sync(0xFFFFFFFFu, g, j), wj = __shfl_sync(0xFFFFFFFFu, w, j);
#pragma unroll
    for (int i = 0; i < NI; ++i)
      if (at == 32 * i) { gi[i] = gj; wi[i] = wj; chosen |= 1u << i; }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int e = lane + 32 * i;
    if (e < L) {
      const float d = normalize ? ((chosen >> i) & 1u ? wi[i] * (gi[i] - inner) : 0.0f) : p[i] * (gi[i] - inner);
      store1(kind, dlogits, t * ld + e, d);
    }
  }
}

// ---------------------------------------------------------------- sort by expert
// A stable counting sort.  Each warp owns a contiguous run of slots, each block
// the runs of its warps in order.  A warp finds the slots of its 32 that name the
// same expert with one match instruction, so a slot's rank is the count before
// its run plus the run's own before it: no order depends on timing.
//
// Up to kSortClusterSlots slots one cluster does it all in one launch, its blocks'
// totals meeting in distributed shared memory; more slots take a launch that
// counts and one that places, since scattered 4-byte stores want many SMs.
// Either way the bytes (16 a slot) are nothing and what is left is a chain of
// latencies: load, match, prefix, exchange, scatter.  One after the other in a graph,
// 1024 slots over 64 experts and 8192 over 8 take 5.0 us (1024 in one block of 256
// threads: 11), 65536 over 64 10.2 (in one cluster the scatter alone would take 8) and
// over 1024 29.7.
constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kSortMaxCluster = 8;
constexpr int64_t kSortClusterSlots = 2 * kSortThreads * kSortMaxCluster;

struct SortParams {
  int64_t slots, m_pad;
  int L, steps, blocks;          // steps: of 32 slots, per warp
  const int32_t* ids;
  const float* weights;
  int32_t *offsets, *row_of_slot, *slot_of_row, *rows_used;
  float* prob;
  int32_t* counts;               // (blocks, L), two launches only
  uint32_t* status;
};

// Shared memory of L experts: total and before (this block's first rank) of each,
// first row of each and one past the last; a scratch word per warp and expert
// group; the warps' counts, then their ranks inside the block (a block's slots may
// all name one expert and are 512 a step: 16 bits would hold the ranks of 128 steps,
// 9.7 million slots in all).
struct SortShared {
  int32_t *mine, *total, *before, *first, *scan;
  int32_t* warp_count;
  __device__ SortShared(int32_t* sm, int L)
      : mine(sm), total(sm + L), before(sm + 2 * L), first(sm + 3 * L), scan(sm + 4 * L + 1),
        warp_count(sm + 4 * L + 1 + kSortWarps) {}
};
constexpr size_t sort_shared_bytes(int L) { return 4 * (4 * size_t(L) + 1 + kSortWarps + size_t(L) * kSortWarps); }

__device__ __forceinline__ int sort_id(const SortParams& p, int64_t s) {
  const int32_t e = s < p.slots ? p.ids[s] : -1;
  return (e >= 0 && e < p.L) ? e : -1;
}

// Counts of this block's slots: per warp (as ranks inside the block) and in all.
__device__ __forceinline__ void sort_count(const SortParams& p, const SortShared& sh, int block) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < kSortWarps * p.L; i += kSortThreads) sh.warp_count[i] = 0;
  __syncthreads();
  const int64_t s0 = (static_cast<int64_t>(block) * kSortWarps + warp) * p.steps * 32;
  for (int k = 0; k < p.steps; ++k) {
    const int e = sort_id(p, s0 + 32 * k + lane);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    if (e >= 0 && lane == __ffs(same) - 1) sh.warp_count[warp * p.L + e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.L; e += kSortThreads) {
    int32_t run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const int32_t c = sh.warp_count[w * p.L + e];
      sh.warp_count[w * p.L + e] = run;
      run += c;
    }
    sh.mine[e] = run;
  }
}

// first[e] from total[e]: exclusive prefix of the padded sizes (L <= 1024: two
// experts a thread).
__device__ __forceinline__ void sort_first(const SortParams& p, const SortShared& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, e = 2 * threadIdx.x;
  auto padded = [&](int i) { return i < p.L ? (sh.total[i] + 127) / 128 * 128 : 0; };
  const int32_t a = padded(e), both = a + padded(e + 1);
  int32_t incl = both;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int32_t y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) sh.scan[warp] = incl;
  __syncthreads();
  int32_t base = 0;
  for (int w = 0; w < warp; ++w) base += sh.scan[w];
  const int32_t at = base + incl - both;
  if (e < p.L) sh.first[e] = at;
  if (e + 1 < p.L) sh.first[e + 1] = at + a;
  if (e == ((p.L - 1) & ~1)) sh.first[p.L] = at + both;
  __syncthreads();
}

// Offsets, padding rows and this block's slots; block of `blocks`.
__device__ __forceinline__ void sort_place(const SortParams& p, const SortShared& sh, int block, int blocks) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t m_pad = static_cast<int32_t>(p.m_pad);
  const int64_t s0 = (static_cast<int64_t>(block) * kSortWarps + warp) * p.steps * 32;
  for (int k = 0; k < p.steps; ++k) {
    const int64_t s = s0 + 32 * k + lane;
    const int e = sort_id(p, s);
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
    int32_t r = -1;
    if (e >= 0) {
      r = sh.first[e] + sh.before[e] + sh.warp_count[warp * p.L + e] + __popc(same & ((1u << lane) - 1u));
      if (r >= m_pad) r = -1;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) sh.warp_count[warp * p.L + e] += __popc(same);
    __syncwarp();
    if (s < p.slots) {
      p.row_of_slot[s] = r;
      if (r >= 0) {
        p.slot_of_row[r] = static_cast<int32_t>(s);
        if (p.prob != nullptr) p.prob[r] = p.weights != nullptr ? p.weights[s] : 1.0f;
      }
    }
  }
  if (block == 0) {
    for (int e = threadIdx.x; e < p.L; e += kSortThreads)
      p.offsets[e] = e + 1 == p.L ? m_pad : min(sh.first[e + 1], m_pad);
    if (threadIdx.x == 0) {
      if (p.rows_used != nullptr) *p.rows_used = sh.first[p.L];
      if (sh.first[p.L] > m_pad && p.status != nullptr) atomicOr(p.status, kStatusBadOffsets);
    }
  }
  // padding rows: between an expert's last slot and the next expert, a warp per
  // expert; after the last expert up to m_pad, over all threads
  for (int e = block * kSortWarps + warp; e < p.L; e += blocks * kSortWarps) {
    for (int32_t r = sh.first[e] + sh.total[e] + lane; r < min(sh.first[e + 1], m_pad); r += 32) {
      p.slot_of_row[r] = -1;
      if (p.prob != nullptr) p.prob[r] = 0.0f;
    }
  }
  for (int64_t r = sh.first[p.L] + static_cast<int64_t>(block) * kSortThreads + threadIdx.x; r < m_pad;
       r += static_cast<int64_t>(blocks) * kSortThreads) {
    p.slot_of_row[r] = -1;
    if (p.prob != nullptr) p.prob[r] = 0.0f;
  }
}

__global__ void __launch_bounds__(kSortThreads) sort_cluster_kernel(SortParams p) {
  extern __shared__ int32_t sm[];
  const SortShared sh(sm, p.L);
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int rank = blockIdx.x, blocks = p.blocks;
  sort_count(p, sh, rank);
  if (blocks > 1) cluster_sync(); else __syncthreads();
  for (int e = threadIdx.x; e < p.L; e += kSortThreads) {
    int32_t all = 0, before = 0;
    for (int r = 0; r < blocks; ++r) {
      int32_t c;
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(c) : "r"(mapa_shared(smem_u32(&sh.mine[e]), r)) : "memory");
      all += c;
      before += r < rank ? c : 0;
    }
    sh.total[e] = all;
    sh.before[e] = before;
  }
  __syncthreads();
  sort_first(p, sh);
  sort_place(p, sh, rank, blocks);
  if (blocks > 1) cluster_sync();          // the totals stay until every block has read them
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortParams p) {
  extern __shared__ int32_t sm[];
  const SortShared sh(sm, p.L);
  let_next_kernel_start();
  wait_for_previous_kernel();
  sort_count(p, sh, blockIdx.x);
  for (int e = threadIdx.x; e < p.L; e += kSortThreads) p.counts[static_cast<int64_t>(blockIdx.x) * p.L + e] = sh.mine[e];
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortParams p) {
  extern __shared__ int32_t sm[];
  const SortShared sh(sm, p.L);
  let_next_kernel_start();
  wait_for_previous_kernel();
  for (int e = threadIdx.x; e < p.L; e += kSortThreads) sh.total[e] = sh.before[e] = 0;
  sort_count(p, sh, blockIdx.x);
  // the blocks' counts of an expert: shared out over as many threads as there are
  // (integer sums: the order of the atomics does not matter)
  const int per = (p.L + 31) / 32 * 32, groups = max(1, kSortThreads / per);
  for (int i = threadIdx.x; i < per * groups; i += kSortThreads) {
    const int e = i % per, g = i / per;
    if (e >= p.L) continue;
    int32_t all = 0, before = 0;
#pragma unroll 4
    for (int b = g; b < p.blocks; b += groups) {
      const int32_t c = p.counts[static_cast<int64_t>(b) * p.L + e];
      all += c;
      before += b < static_cast<int>(blockIdx.x) ? c : 0;
    }
    atomicAdd(&sh.total[e], all);
    atomicAdd(&sh.before[e], before);
  }
  __syncthreads();
  sort_first(p, sh);
  sort_place(p, sh, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- dispatch
struct RowsParams {
  int64_t tokens, m_pad, ld_token;
  int hidden, topk;
  int kq;                           // scale atoms per 128 rows
  const void* x;                    // x or dy
  const int32_t *row_of_slot, *slot_of_row;
  void* a;
  uint8_t* sfa;
  // the gradient of combine
  const float* weights;
  const void* d;
  int d_kind;
  float* dweights;
};

// What a kernel of the rows does: dispatch; the gradient of combine, rows (and
// dweights); dweights alone.
enum : int { ROWS_DISPATCH = 0, ROWS_GRAD = 1, ROWS_DOT = 2 };

constexpr int kRowThreads = 512, kMaxTopk = 32, kPadRows = 8;

// Values a thread holds, in two runs of eight (hidden is a multiple of 8, for rows
// with scales of 16): with D's two rows of a top-2 token that is 96 bytes a thread
// in flight.
constexpr int kRowValues = 16;

// The scale code of this thread's block (shared by rf_vec / 16 lanes), and the
// word of the four blocks it lies in, complete in every lane: their bytes are
// neighbours in the scale factors' layout.
template <int FMT>
__device__ __forceinline__ uint32_t block_code(const float (&v)[16], bool in, uint32_t& word) {
  constexpr int kLanes = rf_vec(FMT) / 16;
  uint32_t m = max_abs_bits16(v);
  if (kLanes == 2) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  const uint32_t code = scale_code<FMT>(m);
  word = in ? code << (8 * ((threadIdx.x / kLanes) & 3)) : 0u;
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, kLanes);
  word |= __shfl_xor_sync(0xFFFFFFFFu, word, 2 * kLanes);
  return code;
}

// Blocks [0, tokens): one token each.  Its values are read once, and (without
// weights) quantized once, for all of its rows: x is T H elements where the rows
// are topk times that, and reading and quantizing per row took 276 us for 8192
// tokens of 7168, top-8.  The blocks after them write the padding rows, kPadRows
// each.  A lane holds 16 values: half a block of 32, whose other half is one
// exchange away, and a whole 16-byte store of FP8 codes.
//   8192 x 7168 float16, top-8 of 64 into E5M2: 117 MB read, 546 written, 126 us,
//     5.3 TB/s, bound by writing (a plain fill of 554 MB takes 139 us);
//   4096 x 4096 bfloat16, top-2 of 8 into E4M3: 72 MB, 15 us, bound by issue (two
//     thirds of the slots) and the loads' latency;
//   128 x 7168, top-8 of 64: 59 MB, nearly all of it padding rows, 13 us.
// The gradient of combine also takes the products <dy, D[row]>, with D's rows in
// flight while dy is in registers: 4096 x 4096, top-2, 175 MB in 30 us, 5.8 TB/s,
// bound by the loads' latency (as two launches 42 us, reading dy twice).
template <int KIND, int FMT, int MODE>
__global__ void __launch_bounds__(kRowThreads, MODE == ROWS_DISPATCH ? 3 : 2) rows_kernel(RowsParams p) {
  constexpr int V = kRowValues, kLanes = rf_scaled(FMT) ? rf_vec(FMT) / 16 : 1;
  constexpr int kBatch = 2;                           // rows of D in flight
  __shared__ float part[MODE == ROWS_DISPATCH ? 1 : kMaxTopk][kRowThreads / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  let_next_kernel_start();
  wait_for_previous_kernel();
  // columns in whole warps, up to the end of the last scale atom.  A column and a
  // row's bytes fit 32 bits (hidden is at most 2^24); a row's offset does not
  const int cols = rf_scaled(FMT) ? p.kq * 4 * rf_vec(FMT) : p.hidden;
  const int end = (cols + 32 * V - 1) / (32 * V) * (32 * V);
  const int row_bytes = p.hidden / 8 * rf_bits(FMT), atoms_bytes = p.kq * 512;   // of a row; of 128 rows' scales
  uint8_t* const a = static_cast<uint8_t*>(p.a);
  if (blockIdx.x >= p.tokens) {
    const int64_t r0 = (static_cast<int64_t>(blockIdx.x) - p.tokens) * kPadRows;
    constexpr uint32_t one = rf_one(FMT) * 0x01010101u;
    for (int64_t r = r0; r < min(r0 + kPadRows, p.m_pad); ++r) {
      const int32_t s = p.slot_of_row[r];
      if (s >= 0 && s < p.tokens * p.topk) continue;
      uint8_t* row = a + r * row_bytes;                  // row_bytes is a multiple of 16
      for (int c = threadIdx.x * 16; c < row_bytes; c += blockDim.x * 16) *reinterpret_cast<uint4*>(row + c) = make_uint4(0, 0, 0, 0);
      if (rf_scaled(FMT)) {
        const int kb = (p.hidden + rf_vec(FMT) - 1) / rf_vec(FMT);
        uint8_t* sf = p.sfa + sf_off(r, 0, p.kq);
        for (int q = threadIdx.x; q < p.kq; q += blockDim.x) {
          const int left = kb - 4 * q;                   // blocks of this word inside hidden
          *reinterpret_cast<uint32_t*>(sf + static_cast<int64_t>(q) * 512) = left >= 4 ? one : one & ((1u << (8 * left)) - 1u);
        }
      }
    }
    return;
  }
  const int64_t t = blockIdx.x;
  // lane j holds choice j's row and weight, fetched beside the token's values
  int32_t my_row = lane < p.topk ? p.row_of_slot[t * p.topk + lane] : -1;
  if (my_row >= p.m_pad) my_row = -1;
  const bool weighted = MODE == ROWS_GRAD && p.weights != nullptr;
  const float my_weight = weighted && lane < p.topk ? p.weights[t * p.topk + lane] : 1.0f;
  const bool dot = MODE != ROWS_DISPATCH && p.dweights != nullptr;
  for (int c = threadIdx.x * V; c < end; c += blockDim.x * V) {
    const bool in = c < p.hidden, both = c + 8 < p.hidden;
    float v[V];
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = 0.0f;
    if (in) {
#pragma unroll
      for (int h = 0; h < V; h += 8)
        if (h == 0 || both) load8<KIND>(p.x, t * p.ld_token + c + h, reinterpret_cast<float(&)[8]>(v[h]));
    }
    if (dot) {
      // D's rows stay packed until they are used: a batch of 16-bit rows in flight
      // costs half the registers of its values
      const bool first = c == static_cast<int>(threadIdx.x) * V;
      for (int j0 = 0; j0 < p.topk; j0 += kBatch) {
        int32_t r[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          r[b] = j0 + b < p.topk ? __shfl_sync(0xFFFFFFFFu, my_row, j0 + b) : -1;
        }
        float acc[kBatch];
        if (p.d_kind == OK_F32) {
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            acc[b] = 0.0f;
#pragma unroll
            for (int h = 0; h < V; h += 8) {
              float w[8] = {0, 0, 0, 0, 0, 0, 0, 0};
              if ((h == 0 ? in : both) && r[b] >= 0) load8<OK_F32>(p.d, static_cast<int64_t>(r[b]) * p.hidden + c + h, w);
#pragma unroll
              for (int k = 0; k < 8; ++k) acc[b] = fmaf(v[h + k], w[k], acc[b]);
            }
          }
        } else {
          uint4 u[kBatch][V / 8];
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int h = 0; h < V / 8; ++h) {
              u[b][h] = make_uint4(0, 0, 0, 0);
              if ((h == 0 ? in : both) && r[b] >= 0)
                u[b][h] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.d) + static_cast<int64_t>(r[b]) * p.hidden + c + 8 * h);
            }
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            acc[b] = 0.0f;
#pragma unroll
            for (int h = 0; h < V / 8; ++h) {
              const uint32_t q[4] = {u[b][h].x, u[b][h].y, u[b][h].z, u[b][h].w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = p.d_kind == OK_F16 ? unpack2<OK_F16>(q[k]) : unpack2<OK_BF16>(q[k]);
                acc[b] = fmaf(v[8 * h + 2 * k], f.x, acc[b]);
                acc[b] = fmaf(v[8 * h + 2 * k + 1], f.y, acc[b]);
              }
            }
          }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (j0 + b >= p.topk) break;
          // a slot without a row has the gradient 0 whatever dy holds
          const float sum = warp_sum(r[b] >= 0 ? acc[b] : 0.0f);
          if (lane == 0) part[j0 + b][warp] = first ? sum : part[j0 + b][warp] + sum;
        }
      }
    }
    if (MODE == ROWS_DOT) continue;
    // quantized once for all rows; with weights, once per row
    uint32_t word = 0, packed[rf_words(FMT)];
    if (!weighted) {
      uint32_t code = 0;
      if constexpr (rf_scaled(FMT)) code = block_code<FMT>(v, in, word);
      quantize16<FMT>(v, code, packed);
    }
    uint8_t* const a_col = a + c / 8 * rf_bits(FMT);
    uint8_t* const sf_col = rf_scaled(FMT) ? p.sfa + static_cast<int64_t>(c / (4 * rf_vec(FMT))) * 512 : nullptr;
    const bool writes_word = rf_scaled(FMT) && lane % (4 * kLanes) == 0 && c < cols;
    for (int j = 0; j < p.topk; ++j) {
      const int32_t r = __shfl_sync(0xFFFFFFFFu, my_row, j);
      if (r < 0) continue;                              // the same for the whole block
      if (weighted) {
        const float f = __shfl_sync(0xFFFFFFFFu, my_weight, j);
        float w[V];
#pragma unroll
        for (int k = 0; k < V; ++k) w[k] = v[k] * f;
        uint32_t code = 0;
        if constexpr (rf_scaled(FMT)) code = block_code<FMT>(w, in, word);
        quantize16<FMT>(w, code, packed);
      }
      if (writes_word)
        *reinterpret_cast<uint32_t*>(sf_col + static_cast<int64_t>(r >> 7) * atoms_bytes + (r & 31) * 16 + ((r >> 5) & 3) * 4) = word;
      if (in) store_codes16<FMT>(a_col + static_cast<int64_t>(r) * row_bytes, packed, both);
    }
  }
  if (dot) {
    __syncthreads();
    for (int j = warp; j < p.topk; j += warps) {
      const float s = warp_sum(lane < warps ? part[j][lane] : 0.0f);
      if (lane == 0) p.dweights[t * p.topk + j] = s;
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

// One token per block of x, a run of columns per block of y; four rows of D are
// loaded before any is added (64 bytes a thread in flight; eight rows are no
// faster).  8192 tokens, top-8, 7168 wide: 1.17 GB in 186 us, 6.3 TB/s, 93 % of the
// measured copy rate, bound by memory.
// Rows that L2 cannot hold are marked as read once (8192 tokens, top-8, 7168 wide:
// 206 us without the mark, 198 with it); smaller ones are where the product that
// wrote them left them (128 tokens: 3.7 us without, 7.2 with).
// Small blocks, since a block's first load waits for its token's row numbers: 197 us
// with 512 threads, 190 with 256, 186 with 128.
constexpr int kCombineThreads = 128;

template <int DK, int KIND, bool STREAM>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(CombineParams p) {
  constexpr int kBatch = 4;
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int64_t t = blockIdx.x;
  const int32_t* rows = p.row_of_slot + t * p.topk;
  const float* weights = p.weights != nullptr ? p.weights + t * p.topk : nullptr;
  for (int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * 8; c < p.hidden;
       c += static_cast<int64_t>(gridDim.y) * blockDim.x * 8) {
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (p.residual != nullptr) load8<KIND>(p.residual, t * p.ld_residual + c, acc);
    for (int j0 = 0; j0 < p.topk; j0 += kBatch) {
      Raw8<DK, STREAM> v[kBatch];
      float w[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int32_t r = j0 + b < p.topk ? rows[j0 + b] : -1;
        const bool real = r >= 0 && r < p.m_pad;
        w[b] = !real ? 0.0f : weights != nullptr ? weights[j0 + b] : 1.0f;
        v[b].load(p.d, r * p.hidden + c, real);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        float f[8];
        v[b].values(f);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = fmaf(w[b], f[k], acc[k]);
      }
    }
    store8<KIND>(p.y, t * p.ld_token + c, acc);
  }
}

// ---------------------------------------------------------------- host
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

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
bsgg_status with_route_regs(int L, F&& f) {
  if (L <= 32) return f(std::integral_constant<int, 1>());
  if (L <= 64) return f(std::integral_constant<int, 2>());
  if (L <= 128) return f(std::integral_constant<int, 4>());
  if (L <= 256) return f(std::integral_constant<int, 8>());
  if (L <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
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
      d->hidden > (int64_t(1) << 24) || d->topk < 1 || d->topk > kMaxTopk || d->tokens * d->topk >= (int64_t(1) << 31))
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

// Threads of a block whose threads take `values` of `cols` columns: whole warps.
int row_threads(int64_t cols, int values) {
  const int64_t t = ceil_div(ceil_div(cols, values), 32) * 32;
  return static_cast<int>(t < kRowThreads ? t : kRowThreads);
}

// Threads of a token's block of rows_kernel.  With the products <dy, D[row]> four
// warps, in several passes: loads, reductions and barrier follow one another, and
// many small blocks overlap them (4096 x 4096, top-2: 256 threads 34.6 us, 128 30.3, 64
// 29.6).  Without them one pass (128 threads: 3 % slower).
int rows_threads(int64_t hidden, bool dot) {
  const int t = row_threads(hidden, kRowValues);
  return dot && t > 128 ? 128 : t;
}

template <int MODE>
bsgg_status launch_rows(const bsgg_tokens_desc* d, RowsParams p, cudaStream_t s) {
  p.tokens = d->tokens; p.hidden = static_cast<int>(d->hidden); p.m_pad = d->m_pad; p.ld_token = d->ld_token; p.topk = d->topk;
  return with_float(d->token_format, [&](auto kind) {
    return with_rows(d->row_format, [&](auto fmt) {
      constexpr int K = decltype(kind)::value, F = decltype(fmt)::value;
      p.kq = rf_scaled(F) ? static_cast<int>(ceil_div(ceil_div(d->hidden, rf_vec(F)), 4)) : 0;
      const int64_t grid = d->tokens + ceil_div(d->m_pad, kPadRows);
      const LaunchConfig c(dim3(static_cast<unsigned>(grid)), rows_threads(d->hidden, p.dweights != nullptr), 0, s);
      return launch_kernel(c, rows_kernel<K, F, MODE>, p);
    });
  });
}

// Blocks of the sort and 32-slot steps of their warps.
void sort_shape(int64_t slots, int64_t* blocks, int64_t* steps) {
  if (slots <= kSortClusterSlots) {
    // one cluster: one step while its blocks suffice, then two; powers of two
    *blocks = 1;
    while (*blocks < kSortMaxCluster && *blocks * kSortThreads < slots) *blocks *= 2;
    *steps = slots > *blocks * kSortThreads ? 2 : 1;
  } else {
    // two steps while the blocks are at most about one an SM (152 here), then more steps
    constexpr int64_t kBlocks = 148;
    *steps = ceil_div(slots, kBlocks * kSortThreads);
    if (*steps < 2) *steps = 2;
    *blocks = ceil_div(slots, *steps * kSortThreads);
  }
}

// Shared memory beyond the default 48 KB has to be asked for.
template <typename K>
bool sort_allowed(K kern, size_t smem) {
  return smem <= 48 * 1024 ||
         succeeded(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)));
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
  const LaunchConfig c(dim3(grid), 32 * kRouteWarps, 0, static_cast<cudaStream_t>(stream));
  return with_route_regs(d->num_experts, [&](auto ni) {
    return launch_kernel(c, route_kernel<decltype(ni)::value>, d->tokens, d->ld, d->num_experts, d->topk, d->logit_format,
                         d->normalize, logits, ids, weights);
  });
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
  const LaunchConfig c(dim3(grid), 32 * kRouteWarps, 0, static_cast<cudaStream_t>(stream));
  return with_route_regs(d->num_experts, [&](auto ni) {
    return launch_kernel(c, route_backward_kernel<decltype(ni)::value>, d->tokens, d->ld, d->num_experts, d->topk,
                         d->logit_format, d->normalize, logits, ids, weights, dweights, row_of_slot, m_pad, dlogits);
  });
}

int64_t bsgg_sort_rows(int64_t slots, int32_t num_experts) {
  if (slots < 0 || slots >= (int64_t(1) << 31) || num_experts < 1 || num_experts > 1024) return -1;
  // the most that sizes adding up to `slots` can need: as many experts as can
  // be, each one slot past a multiple of 128 (one block of rows for no slots)
  const int64_t some = slots < num_experts ? slots : num_experts;
  const int64_t blocks = some + (slots - some) / 128;
  return 128 * (blocks > 0 ? blocks : 1);
}

uint64_t bsgg_sort_workspace_bytes(int64_t slots, int32_t num_experts) {
  if (bsgg_sort_rows(slots, num_experts) < 0) return 0;
  if (slots <= kSortClusterSlots) return 0;
  int64_t blocks, steps;
  sort_shape(slots, &blocks, &steps);
  return uint64_t(4) * blocks * num_experts;
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
  if (slots > (int64_t(1) << 30)) return BSGG_ERR_UNSUPPORTED;   // the padded sizes' sum stays below 2^31
  int64_t blocks, steps;
  sort_shape(slots, &blocks, &steps);
  p.steps = static_cast<int>(steps);
  p.blocks = static_cast<int>(blocks);
  const bool one_cluster = slots <= kSortClusterSlots;
  if (!one_cluster && !workspace) return BSGG_ERR_INVALID_ARG;
  p.ids = ids; p.weights = weights; p.offsets = padded_offsets; p.row_of_slot = row_of_slot; p.slot_of_row = slot_of_row;
  p.rows_used = rows_used; p.prob = prob; p.counts = static_cast<int32_t*>(workspace); p.status = status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t smem = sort_shared_bytes(p.L);                // 82 KB at the most: 1024 experts
  if (one_cluster) {
    if (!sort_allowed(sort_cluster_kernel, smem)) return BSGG_ERR_CUDA;
    const LaunchConfig c(dim3(static_cast<unsigned>(p.blocks)), kSortThreads, smem, s, p.blocks);
    return launch_kernel(c, sort_cluster_kernel, p);
  }
  if (!sort_allowed(sort_count_kernel, smem) || !sort_allowed(sort_place_kernel, smem)) return BSGG_ERR_CUDA;
  const LaunchConfig c(dim3(static_cast<unsigned>(p.blocks)), kSortThreads, smem, s);
  const bsgg_status st = launch_kernel(c, sort_count_kernel, p);
  return st == BSGG_OK ? launch_kernel(c, sort_place_kernel, p) : st;
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
  RowsParams p = {};
  p.x = x; p.row_of_slot = row_of_slot; p.slot_of_row = slot_of_row; p.a = a; p.sfa = static_cast<uint8_t*>(sfa);
  return launch_rows<ROWS_DISPATCH>(d, p, static_cast<cudaStream_t>(stream));
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
  // half of L2's 126 MB
  const bool large = d->tokens * d->topk * d->hidden * float_bytes(d->d_format) > (int64_t(64) << 20);
  CombineParams p = {d->tokens, d->hidden, d->m_pad, d->ld_token, d->ld_residual, d->topk, dd, row_of_slot, weights,
                     residual, y};
  return with_float(d->d_format, [&](auto dk) {
    return with_float(d->token_format, [&](auto kind) {
      // a token's columns over blocks of four warps; over blocks of two where there
      // are so few that the chip would have less than four blocks an SM
      int threads = row_threads(d->hidden, 8);
      if (threads > kCombineThreads) threads = kCombineThreads;
      if (threads > 64 && d->tokens * ceil_div(d->hidden, threads * 8) < 608) threads = 64;
      const dim3 grid(static_cast<unsigned>(d->tokens), static_cast<unsigned>(ceil_div(d->hidden, threads * 8)));
      constexpr int D = decltype(dk)::value, K = decltype(kind)::value;
      const LaunchConfig c(grid, threads, 0, static_cast<cudaStream_t>(stream));
      return large ? launch_kernel(c, combine_kernel<D, K, true>, p) : launch_kernel(c, combine_kernel<D, K, false>, p);
    });
  });
}

bsgg_status bsgg_combine_backward(const bsgg_tokens_desc* d, const void* dy, const void* rows,
                                  const int32_t* row_of_slot, const int32_t* slot_of_row, const float* weights, void* dd,
                                  void* sfd, float* dweights, void* stream) {
  const bsgg_status st = check_tokens(d, dd != nullptr, dweights != nullptr);
  if (st != BSGG_OK) return st;
  if (!dd && !dweights) return d->tokens == 0 ? BSGG_OK : BSGG_ERR_INVALID_ARG;   // no tokens: an empty dweights may be NULL
  if (d->tokens > 0 && (!dy || !row_of_slot || (dweights && !rows))) return BSGG_ERR_INVALID_ARG;
  if (dd ? (!slot_of_row || (rf_scaled(d->row_format) ? !sfd : sfd != nullptr)) : sfd != nullptr)
    return BSGG_ERR_INVALID_ARG;
  if (!aligned_to(dy, 16) || !aligned_to(rows, 16) || !aligned_to(dd, 16) || !aligned_to(sfd, 16) ||
      !aligned_to(row_of_slot, 4) || !aligned_to(slot_of_row, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4))
    return BSGG_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowsParams p = {};
  p.x = dy; p.row_of_slot = row_of_slot; p.slot_of_row = slot_of_row; p.a = dd; p.sfa = static_cast<uint8_t*>(sfd);
  p.weights = weights; p.d = rows; p.d_kind = d->d_format; p.dweights = dweights;
  if (dd) return launch_rows<ROWS_GRAD>(d, p, s);
  if (d->tokens == 0) return BSGG_OK;
  p.tokens = d->tokens; p.hidden = static_cast<int>(d->hidden); p.m_pad = d->m_pad; p.ld_token = d->ld_token; p.topk = d->topk;
  return with_float(d->token_format, [&](auto kind) {
    constexpr int F = BSGG_IN_BF16;
    const LaunchConfig c(dim3(static_cast<unsigned>(d->tokens)), rows_threads(d->hidden, true), 0, s);
    return launch_kernel(c, rows_kernel<decltype(kind)::value, F, ROWS_DOT>, p);
  });
}

}  // extern "C"
