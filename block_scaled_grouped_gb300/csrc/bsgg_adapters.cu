// bsgg_adapters.cu -- low-rank adapters of many requests at once beside a dense layer,
// and their gradient.
//
// Three products cover both directions, since A (rank, k) and B (rank, n) both have
// their rows along the wide dimension.  W is either, i the adapter of a token:
//   shrink  u[t]  = f_i X[t] W_i^T        forward u = x A^T; backward du = s dy B^T
//   expand  Y[t]  = base[t] + f_i u[t] W_i  forward y (B); backward dx (A)
//   outer   dW_i  = f_i sum_t g[t]^T X[t]   dA from du and x, dB from u and dy
// Each reads its wide operand once, 2 rank products per value of two bytes: 435 TFLOP/s at a
// rank of 64 and the memory's rate.  That is within mma.sync's 620 (1024 products a cycle
// and SM), whose tiles of 16 x 8 fit what a batch holds, from one token of an adapter up,
// where tcgen05's are 128 rows.  What they cost was looked at: expand of 4096 tokens, rank
// 64, 4096 to 14336, takes as long with half of its products left out, and 11 us less of 87
// without any.
#include "bsgg_ops.cuh"

namespace {

using namespace bsgg;

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Sums of more than this many products are added up in registers in runs of this length: the
// matrix instruction cuts what an addition drops, and a sum of one sign comes out small by
// 3.5e-9 of it per product (float16, 32768 rows in two terms 2.3e-4; in runs of 512 3.1e-6).
constexpr int kRun = 512;
constexpr int kMaxCluster = 8;

struct AdapterMap {
  int64_t tokens, m_pad;
  int adapters;
  const int32_t *offsets, *row_of_slot, *slot_of_row;
};

// ---------------------------------------------------------------- pieces
// `bytes` (16 or 0) from global to shared memory, zeros behind them; with 0 the source is
// not read.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 get_shared4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float4 get_shared4f(uint32_t at) {
  const uint4 v = get_shared4(at);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void load_matrices_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void store_matrices(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// c (16 x 8) += a (16 x 16) b (16 x 8)
template <int KIND>
__device__ __forceinline__ void multiply(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (KIND == OK_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The place of 16-byte piece `piece` of a 128-byte row: eight rows' pieces of one
// column lie in different banks.
__device__ __forceinline__ uint32_t swizzled(int row, int piece) {
  return static_cast<uint32_t>(row * 128 + ((piece ^ (row & 7)) << 4));
}

// A pair of 32-bit values as a sum of TERMS pairs of 16-bit ones: the products take them one
// after the other, so that u and du enter nearly as they are (two terms: to 2^-17 of the value in
// bfloat16, to 2^-22 in float16; three of bfloat16: 2^-24).
template <int KIND, int TERMS>
__device__ __forceinline__ void split_terms(float x, float y, uint32_t (&t)[TERMS]) {
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    t[i] = pack2<KIND>(x, y);
    const float2 f = unpack2<KIND>(t[i]);
    // nothing is left of an infinity
    x = fabsf(f.x) < INFINITY ? x - f.x : 0.0f;
    y = fabsf(f.y) < INFINITY ? y - f.y : 0.0f;
  }
}
// 2^-e for a value whose largest magnitude is 2^e to 2^(e+1): float16 has to be kept
// inside its range, bfloat16 has float's.
__device__ __forceinline__ float unit_of(float largest) {
  const uint32_t e = __float_as_uint(largest) >> 23;
  return e >= 1u && e <= 253u ? __uint_as_float((254u - e) << 23) : 1.0f;
}

__device__ __forceinline__ int32_t token_at(const AdapterMap& m, int64_t row) {
  const int32_t t = row < m.m_pad ? m.slot_of_row[row] : -1;
  return t >= 0 && t < m.tokens ? t : -1;
}
// ROWS rows from row0: their tokens into shared memory, one past the last row that has one,
// and the adapter whose rows they are.  All threads call it: the map and the offsets are
// read at once.
struct Tile {
  int n, adapter;
};
template <int ROWS>
__device__ __forceinline__ Tile tile_at(const AdapterMap& m, int64_t row0, int32_t* token) {
  __shared__ uint32_t mask[ROWS / 32];
  __shared__ int ends[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t t = threadIdx.x < ROWS ? token_at(m, row0 + threadIdx.x) : -1;
  int before = 0;                                      // adapters whose rows end before these
  for (int i = threadIdx.x; i < m.adapters; i += kThreads) before += m.offsets[i] <= row0;
  const uint32_t b = __ballot_sync(0xFFFFFFFFu, t >= 0);
  before = __reduce_add_sync(0xFFFFFFFFu, before);
  if (threadIdx.x < ROWS) token[threadIdx.x] = t;
  if (lane == 0) {
    ends[warp] = before;
    if (warp < ROWS / 32) mask[warp] = b;
  }
  __syncthreads();
  Tile tile = {0, 0};
#pragma unroll
  for (int i = 0; i < ROWS / 32; ++i)
    if (mask[i] != 0) tile.n = 32 * i + 32 - __clz(mask[i]);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) tile.adapter += ends[w];
  tile.adapter = min(tile.adapter, m.adapters - 1);
  return tile;
}
// Groups of 16 rows, as a power of two, that hold n rows.
__device__ __forceinline__ int row_groups(int n) { return n <= 16 ? 1 : n <= 32 ? 2 : n <= 64 ? 4 : 8; }

// ---------------------------------------------------------------- shrink
// A block takes 64 rows of one adapter and one of `split` parts of the reduction; the
// cluster's blocks join through distributed shared memory, in order.  Its warps are as
// many groups of 16 rows as there are tokens, and share the reduction's steps of 16 beyond
// that: a decoding batch has a token or two per adapter, and is then a stream of A.
//   4096 tokens, rank 64, from 4096: 19 us for 34 MB of x, 1.8 TB/s; rank 32, from 14336: 31 us
//   for 117 MB, 3.8 TB/s: bound by the chain from stage to stage (barrier, matrix loads,
//   products) and the cluster's join; with one block of 64 of the reduction between barriers
//   35.  128 tokens of 64 adapters, rank 16, from 4096: 11 us alone, 7.3 MB of A.
template <int R>
struct Shrink {
  static constexpr int kRows = 64, kStages = R == 128 ? 4 : 3;
  // rows of 128 bytes in a stage: 64 of X and R of W twice (two blocks of 64 of the reduction
  // between barriers), once at a rank of 128; with few tokens up to four
  static constexpr int kStageRows = R == 128 ? 192 : 2 * (64 + R);
  static constexpr int kStageBytes = kStageRows * 128;
  // 8 rows more: of an odd number of eights of ranks the last matrix load reads 16 rows
  static constexpr int kSmem = kStages * kStageBytes + 8 * 128 + 128;
};

struct ShrinkParams {
  AdapterMap map;
  const void* x;
  const void* w;
  const float* scales;
  float* u;
  int64_t ldx;
  int depth, rank, split;
};

template <int KIND, int R, bool FULL, bool RUNS>
__global__ void __launch_bounds__(kThreads, R <= 32 ? 3 : R == 64 || !RUNS ? 2 : 1) shrink_kernel(const __grid_constant__ ShrinkParams p) {
  using S = Shrink<R>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int32_t token[S::kRows];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tile = blockIdx.x / p.split;
  const int part = static_cast<int>(blockIdx.x - tile * p.split);
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int64_t row0 = tile * S::kRows;
  const Tile at_tile = tile_at<S::kRows>(p.map, row0, token);
  const int n = at_tile.n, adapter = at_tile.adapter;
  if (n == 0) return;                                  // for the whole cluster
  const int groups = row_groups(n), rows = 16 * groups, shares = kWarps / groups;
  const int mw = warp % groups, kw = warp / groups;
  const int blocks = max(1, min(4, S::kStageRows / (rows + p.rank)));   // of 64, a stage
  const int64_t nb = (p.depth + 63) / 64;
  const int b0 = static_cast<int>(nb * part / p.split), b1 = static_cast<int>(nb * (part + 1) / p.split);
  const int steps = (b1 - b0 + blocks - 1) / blocks;
  const int rank = FULL ? R : p.rank;
  const uint32_t block_bytes = static_cast<uint32_t>(rows + rank) * 128;
  // a thread copies one 16-byte piece of every 32nd row; its sources move on by a block of 64
  // with each block loaded
  const int piece = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const uint16_t* xp[S::kRows / 32];
  int xb[S::kRows / 32];
#pragma unroll
  for (int i = 0; i < S::kRows / 32; ++i) {
    const int32_t t = r0 + 32 * i < n ? token[r0 + 32 * i] : -1;
    xb[i] = t >= 0 ? 16 : 0;
    xp[i] = static_cast<const uint16_t*>(p.x) + (t >= 0 ? t * p.ldx + b0 * 64 + piece * 8 : 0);
  }
  const uint16_t* wp = static_cast<const uint16_t*>(p.w) + (static_cast<int64_t>(adapter) * rank + r0) * p.depth + b0 * 64 + piece * 8;
  const uint32_t to0 = base + swizzled(r0, piece);
  int left = p.depth - b0 * 64 - piece * 8;            // of the reduction from this thread's piece on
  int next = b0;                                       // the next block to load

  auto load = [&](int step) {
    uint32_t to = to0 + (step % S::kStages) * S::kStageBytes;
    for (int j = 0; j < blocks && next < b1; ++j, ++next, to += block_bytes, left -= 64, wp += 64) {
#pragma unroll
      for (int i = 0; i < S::kRows / 32; ++i) {
        if (r0 + 32 * i < rows) copy16(to + 4096 * i, xp[i], left > 0 ? xb[i] : 0);
        xp[i] += 64;
      }
#pragma unroll
      for (int i = 0; i < (R + 31) / 32; ++i)
        if (r0 + 32 * i < rank) copy16(to + rows * 128 + 4096 * i, wp + 32 * i * static_cast<int64_t>(p.depth), left > 0 ? 16 : 0);
    }
    copies_commit();
  };
  const int ar = mw * 16 + (lane & 15), br = (lane & 7) + ((lane >> 4) << 3);

  float acc[R / 8][4], sum[RUNS ? R / 8 : 1][4];
#pragma unroll
  for (int i = 0; i < (RUNS ? R / 8 : 1); ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[i][k] = 0.0f;
  for (int s = 0; s < S::kStages - 1; ++s) load(s);
  const int run = RUNS ? kRun / 64 * shares / blocks : steps;   // stages until a warp has summed kRun products
  for (int s0 = 0; s0 < steps; s0 += run) {
#pragma unroll
    for (int i = 0; i < R / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
    const int s1 = min(s0 + run, steps);
    for (int s = s0; s < s1; ++s) {
      copies_wait<S::kStages - 2>();
      __syncthreads();                                 // stage s is there, and s - 1 is read
      load(s + S::kStages - 1);
      const uint32_t stage = base + (s % S::kStages) * S::kStageBytes;
      const int end = 4 * min(blocks, b1 - b0 - s * blocks);
      for (int q = kw; q < end; q += shares) {         // steps of 16
        const uint32_t xs = stage + (q >> 2) * block_bytes;
        const int kk = (q & 3) * 2;
        uint32_t a[4];
        load_matrices(a, xs + swizzled(ar, kk + (lane >> 4)));
        const uint32_t bs = xs + rows * 128 + swizzled(br, kk + ((lane >> 3) & 1));
        uint32_t b[R / 16][4];
#pragma unroll
        for (int i = 0; i < R / 16; ++i)
          // of an odd number of eights the last pair's second half is what lies behind, and unused
          if (FULL || i * 16 < rank) load_matrices(b[i], bs + i * 2048);
#pragma unroll
        for (int i = 0; i < R / 16; ++i) {
          if (FULL || i * 16 < rank) multiply<KIND>(acc[2 * i], a, b[i][0], b[i][1]);
          if (FULL || i * 16 + 8 < rank) multiply<KIND>(acc[2 * i + 1], a, b[i][2], b[i][3]);
        }
      }
    }
    if (RUNS) {
#pragma unroll
      for (int i = 0; i < R / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[i][k] = sum[RUNS ? i : 0][k] += acc[i][k];
    }
  }
  copies_wait<0>();
  __syncthreads();
  // the warps' shares, then the cluster's parts, in order
  float* sums = reinterpret_cast<float*>(smem);
  {
    const int row = mw * 16 + (lane >> 2);
    float* at = sums + (static_cast<int64_t>(kw) * rows + row) * rank + 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < R / 8; ++i) {
      if (i * 8 >= rank) break;
      *reinterpret_cast<float2*>(at + i * 8) = make_float2(acc[i][0], acc[i][1]);
      *reinterpret_cast<float2*>(at + 8 * rank + i * 8) = make_float2(acc[i][2], acc[i][3]);
    }
  }
  __syncthreads();
  const int quads = rows * rank / 4;
  for (int e = threadIdx.x; e < quads; e += kThreads) {
    float4* at = reinterpret_cast<float4*>(sums) + e;
    float4 v = *at;
    for (int k = 1; k < shares; ++k) {
      const float4 o = at[k * quads];
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
    *at = v;
  }
  if (p.split > 1) cluster_sync(); else __syncthreads();
  const float f = p.scales != nullptr ? p.scales[adapter] : 1.0f;
  const int e0 = quads * part / p.split, e1 = quads * (part + 1) / p.split;
  for (int e = e0 + threadIdx.x; e < e1; e += kThreads) {
    const uint32_t at = smem_u32(sums) + e * 16;
    float4 v = make_float4(0, 0, 0, 0);
    for (int k = 0; k < p.split; ++k) {
      const float4 o = ld_shared_cluster4(mapa_shared(at, k));
      v.x += o.x; v.y += o.y; v.z += o.z; v.w += o.w;
    }
    const int row = e * 4 / rank, col = e * 4 - row * rank;
    const int32_t t = row < n ? token[row] : -1;
    if (t >= 0) *reinterpret_cast<float4*>(p.u + static_cast<int64_t>(t) * rank + col) = make_float4(f * v.x, f * v.y, f * v.z, f * v.w);
  }
  if (p.split > 1) cluster_sync();                     // the sums stay until every block has read them
}

// ---------------------------------------------------------------- expand
// A block takes 128 rows of one adapter and kCols columns.  W's columns come in at once;
// behind that one barrier the warps go their own ways: each fetches the base of its 16 rows
// and 64 columns by asynchronous copies, kBuffers passes ahead, starts its sums from it,
// multiplies, and stores rows of 128 bytes.  Eight groups of 16 rows are eight warps that
// walk the same columns; with fewer tokens the warps lie along the columns too.  The blocks
// behind the tiles see to the tokens without an adapter.
//   4096 tokens, rank 64, to 14336: 57 us for 235 MB, 4.1 TB/s: shared memory is busy 60 % of
//   the time (every warp reads all of W for its 16 rows) and the matrix pipe 45 %; rank 32, to
//   4096: 19 us for 67 MB with the dx of a fifth of the tokens copied.  128 tokens of 64
//   adapters, rank 16, to 14336: 15 us for 36 MB (in blocks of 512 columns 22).  Base and W of
//   128 rows in passes behind a barrier each: 76 us; neighbouring blocks on other rows of the
//   same columns: 7 more.
template <int R>
struct Expand {
  static constexpr int kRows = 128, kCols = R == 16 ? 1024 : R == 128 ? 256 : 512, kBuffers = 2;
  static constexpr int kTileBytes = 16 * 128;             // a warp's rows of 64 columns
  static constexpr int kWBytes = kCols * R * 2;
  static constexpr int kSmem = kWBytes + kWarps * kBuffers * kTileBytes + 128;
};

struct ExpandParams {
  AdapterMap map;
  const float* u;
  const void* w;
  const float* scales;
  const void* base;
  void* y;
  float* zero_u;              // u's rows of tokens without an adapter, where wanted
  int64_t tiles;
  int ld_base, ldy, width, rank, cols, col_blocks, rest_parts;   // cols: of a block, a multiple of 64
};

// Tokens without an adapter: y = base, u = 0.  A block has 32 tokens and one of `rest_parts`
// parts of the columns.
constexpr int kRestTokens = 32;
__device__ __noinline__ void expand_rest(const ExpandParams& p, int64_t number, uint8_t* smem) {
  int32_t* list = reinterpret_cast<int32_t*>(smem);
  int* count = list + kRestTokens;
  const int64_t block = number / p.rest_parts;
  const int part = static_cast<int>(number - block * p.rest_parts);
  if (threadIdx.x < kRestTokens) {
    const int64_t t = block * kRestTokens + threadIdx.x;
    bool none = false;
    if (t < p.map.tokens) {
      const int32_t r = p.map.row_of_slot[t];
      none = r < 0 || r >= p.map.m_pad;
    }
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, none);
    if (none) list[__popc(b & ((1u << threadIdx.x) - 1u))] = static_cast<int32_t>(t);
    if (threadIdx.x == 0) *count = __popc(b);
  }
  __syncthreads();
  const int all = *count, eights = p.width / 8;
  if (p.base != p.y) {
    // four pieces a thread in flight
    const int c0 = static_cast<int>(static_cast<int64_t>(eights) * part / p.rest_parts);
    const int pieces = static_cast<int>(static_cast<int64_t>(eights) * (part + 1) / p.rest_parts) - c0;
    for (int e0 = threadIdx.x; e0 < all * pieces; e0 += 4 * kThreads) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = e0 + k * kThreads;
        v[k] = make_uint4(0, 0, 0, 0);
        if (p.base != nullptr && e < all * pieces)
          v[k] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.base) +
                                                 list[e / pieces] * static_cast<int64_t>(p.ld_base) + (c0 + e % pieces) * 8);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int e = e0 + k * kThreads;
        if (e < all * pieces)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + list[e / pieces] * static_cast<int64_t>(p.ldy) +
                                    (c0 + e % pieces) * 8) = v[k];
      }
    }
  }
  if (p.zero_u != nullptr && part == 0) {
    const int pieces = p.rank / 4;
    for (int e = threadIdx.x; e < all * pieces; e += kThreads)
      *reinterpret_cast<float4*>(p.zero_u + static_cast<int64_t>(list[e / pieces]) * p.rank + (e % pieces) * 4) = make_float4(0, 0, 0, 0);
  }
}

template <int KIND, int R, bool FULL>
__global__ void __launch_bounds__(kThreads, R == 16 ? 3 : 2) expand_kernel(const __grid_constant__ ExpandParams p) {
  using E = Expand<R>;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ int32_t token[E::kRows];
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int64_t number = blockIdx.x / p.col_blocks;
  const int col_at = static_cast<int>(blockIdx.x - number * p.col_blocks);
  if (number >= p.tiles) {
    expand_rest(p, blockIdx.x - p.tiles * p.col_blocks, smem_raw);
    return;
  }
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row0 = number * E::kRows, col0 = static_cast<int64_t>(col_at) * p.cols;
  const Tile at_rows = tile_at<E::kRows>(p.map, row0, token);
  const int n = at_rows.n, adapter = at_rows.adapter;
  if (n == 0) return;
  const int groups = row_groups(n), across = min(kWarps / groups, p.cols / 64);
  const int mw = warp % groups, cw = warp / groups;
  const int rank = FULL ? R : p.rank, ranks = FULL ? R : (rank + 15) & ~15;   // whole steps of 16, zeros behind the rank
  const int cols = static_cast<int>(min(int64_t(p.cols), p.width - col0));
  const int passes = (cols + 64 * across - 1) / (64 * across);
  const uint32_t w_bytes = ranks * 128;                 // of 64 columns

  // this lane's pieces of the warp's rows, of base and y alike
  const uint16_t* from = static_cast<const uint16_t*>(p.base);
  const uint32_t tile = base + E::kWBytes + warp * E::kBuffers * E::kTileBytes;
  const int at_row = lane >> 3, at_col = static_cast<int>(cw * 64 + (lane & 7) * 8);
  int32_t at_token[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = mw * 16 + e * 4 + at_row;
    at_token[e] = r < n ? token[r] : -1;
  }
  // rows e * 4 + at_row of the tile: the swizzle of row 4 + r is that of r with its piece moved by 4
  const uint32_t at0 = swizzled(at_row, lane & 7), at1 = swizzled(4 + at_row, lane & 7);
  const int stride = across * 64;
  int load_col = at_col;
  const uint16_t* load_from = from + col0 + at_col;
  auto load = [&](int pass) {
    if (from != nullptr && cw < across && load_col < cols) {
      const uint32_t to = tile + (pass % E::kBuffers) * E::kTileBytes;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        copy16(to + ((e & 1) ? at1 : at0) + (e >> 1) * 1024, load_from + static_cast<int64_t>(max(at_token[e], 0)) * p.ld_base,
               at_token[e] >= 0 ? 16 : 0);
    }
    load_col += stride;
    load_from += stride;
    copies_commit();
  };
  uint16_t* store_to = static_cast<uint16_t*>(p.y) + col0 + at_col;
  uint32_t w_at[4];                                    // pieces 2 i of the products' rows of W
#pragma unroll
  for (int i = 0; i < 4; ++i) w_at[i] = base + swizzled(lane & 15, 2 * i + (lane >> 4));
  uint32_t y_at[4];                                    // pieces 2 i of the tile's rows: the same places
#pragma unroll
  for (int i = 0; i < 4; ++i) y_at[i] = w_at[i] - base;
#pragma unroll
  for (int i = 0; i < E::kBuffers; ++i) load(i);
  // W: a thread copies one 16-byte piece of every 32nd row of each 64 columns
  {
    const int piece = threadIdx.x & 7, r0 = threadIdx.x >> 3;
    const uint16_t* w = static_cast<const uint16_t*>(p.w) + (static_cast<int64_t>(adapter) * rank + r0) * p.width + col0 + piece * 8;
    uint32_t to = base + swizzled(r0, piece);
    for (int c = piece * 8; c - piece * 8 < cols; c += 64, to += w_bytes, w += 64) {
#pragma unroll
      for (int i = 0; i < (R + 31) / 32; ++i) {
        const int k = r0 + 32 * i;
        if (k < ranks) copy16(to + 4096 * i, w + 32 * i * static_cast<int64_t>(p.width), c < cols && (FULL || k < rank) ? 16 : 0);
      }
    }
  }
  copies_commit();

  // this warp's rows of u, as the products take them
  constexpr int kTerms = 2;
  uint32_t a[kTerms][R / 16][4];
  float unit[2] = {1.0f, 1.0f}, back[2] = {1.0f, 1.0f};
  const float f = p.scales != nullptr ? p.scales[adapter] : 1.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = mw * 16 + (lane >> 2) + 8 * h;
    const int32_t t = r < n ? token[r] : -1;
    const float* u = p.u + static_cast<int64_t>(t < 0 ? 0 : t) * rank + 2 * (lane & 3);
    float2 v[R / 8];
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < R / 8; ++i) {
      v[i] = t >= 0 && (FULL || i * 8 < rank) ? *reinterpret_cast<const float2*>(u + i * 8) : make_float2(0.0f, 0.0f);
      most = fmaxf(most, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
    }
    if (KIND == OK_F16) {
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      // bounded, so that the base times it stays a number of full precision
      unit[h] = fminf(fmaxf(unit_of(most * fabsf(f)), 0x1p-90f), 0x1p40f);
      back[h] = 1.0f / unit[h];
    }
#pragma unroll
    for (int i = 0; i < R / 8; ++i) {
      uint32_t term[kTerms];
      split_terms<KIND, kTerms>(v[i].x * f * unit[h], v[i].y * f * unit[h], term);
#pragma unroll
      for (int k = 0; k < kTerms; ++k) a[k][i / 2][2 * (i & 1) + h] = term[k];
    }
  }
  copies_wait<0>();
  __syncthreads();                                     // W is there

  for (int pass = 0; pass < passes; ++pass) {
    copies_wait<E::kBuffers - 1>();
    __syncwarp();                                      // and this pass's base
    const int c0 = (pass * across + cw) * 64;
    if (cw < across && c0 < cols) {
      const uint32_t ys = tile + (pass % E::kBuffers) * E::kTileBytes, ws = (c0 >> 6) * w_bytes;
      // the sums start from the base, whose 8 x 8 matrices lie in the lanes as the sums do
      float acc[8][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v[4] = {0, 0, 0, 0};
        if (from != nullptr) load_matrices(v, ys + y_at[i]);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f2 = unpack2<KIND>(v[k]);
          acc[2 * i + k / 2][2 * (k & 1)] = KIND == OK_F16 ? f2.x * unit[k & 1] : f2.x;
          acc[2 * i + k / 2][2 * (k & 1) + 1] = KIND == OK_F16 ? f2.y * unit[k & 1] : f2.y;
        }
      }
#pragma unroll
      for (int s = 0; s < R / 16; ++s) {
        if (!FULL && s * 16 >= rank) break;
        uint32_t b[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) load_matrices_t(b[i], w_at[i] + ws + s * 2048);
#pragma unroll
        for (int k = 0; k < kTerms; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            multiply<KIND>(acc[2 * i], a[k][s], b[i][0], b[i][1]);
            multiply<KIND>(acc[2 * i + 1], a[k][s], b[i][2], b[i][3]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* at = &acc[2 * i + k / 2][2 * (k & 1)];
          v[k] = KIND == OK_F16 ? pack2<KIND>(at[0] * back[k & 1], at[1] * back[k & 1]) : pack2<KIND>(at[0], at[1]);
        }
        store_matrices(ys + y_at[i], v[0], v[1], v[2], v[3]);
      }
      __syncwarp();
      const int c = pass * across * 64 + at_col;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 v = get_shared4(ys + ((e & 1) ? at1 : at0) + (e >> 1) * 1024);
        if (at_token[e] >= 0 && c < cols) *reinterpret_cast<uint4*>(store_to + static_cast<int64_t>(at_token[e]) * p.ldy) = v;
      }
      __syncwarp();                                    // the buffer is read
    }
    store_to += stride;
    load(pass + E::kBuffers);
  }
  copies_wait<0>();
}

// ---------------------------------------------------------------- outer
// dA and dB together.  u and du are first written as terms of 16 bits, row by row of the map
// (every block of columns would do it again).  Then a block takes one segment of an
// adapter's rows (`segment` of them, so that blocks are alike however the tokens are shared
// out) and kCols columns of x or dy.  An adapter of one segment is finished there; the
// segments' sums of the others meet in another launch, in order.  The products are
// (rank x 64 tokens) (64 tokens x columns), both read across their rows.
//   4096 tokens of 4 adapters, rank 32, 4096 and 14336: 47 us for 151 MB, 3.2 TB/s, after 8 us
//   of terms and before 10 of join (both less behind one another): shared memory is busy half
//   of the time, the matrix pipe as long, in turns.  With the reduction split over clusters
//   by adapter, whose shares are unlike, the two took 65 and 37 us.
template <int R, int TERMS, bool RUNS>
struct Outer {
  // the room that a single run leaves goes to a second block on an SM
  static constexpr int kCols = R == 128 ? 128 : 256, kTokens = 64, kStages = R > 32 && RUNS ? 3 : 2;
  static constexpr int kTermPitch = 2 * R + 16;         // bytes of a token's ranks: eight rows in different banks
  static constexpr int kXBytes = kTokens * kCols * 2, kTermBytes = kTokens * kTermPitch;
  static constexpr int kStageBytes = kXBytes + TERMS * kTermBytes;
  static constexpr int kSmem = kStages * kStageBytes;
  static_assert(R * kCols * 4 <= kSmem, "the sums reuse the stages");
};

// One of the two gradients: sum over an adapter's tokens of g[t]^T X[t], times f_i.
struct OuterSide {
  const float* g;
  const void* x;
  const float* scales;
  void* out;
  float* part;                    // (slots, rank, width) sums of segments
  uint16_t* terms;                // (TERMS, m_pad, ranks) of g
  float* units;                   // of each segment's terms
  float* most;                    // the largest |g| of every 64 rows (float16)
  int64_t ldx;
  int width, blocks;              // blocks of columns; 0: not wanted
};
struct OuterParams {
  AdapterMap map;
  const int32_t* rows_used;       // where the last adapter's rows end
  OuterSide side[2];
  int rank, segment, slots, out_kind;
};

// Where an adapter's segments are.
struct Segment {
  int adapter;                    // -1: there is no such segment
  int index, count;               // of the adapter's segments
  int slot;                       // of the first one's sums, if there are several
};
__device__ __forceinline__ int64_t adapter_end(const OuterParams& p, int i) {
  int64_t end = p.map.offsets[i];
  if (i + 1 == p.map.adapters) end = min(end, static_cast<int64_t>(*p.rows_used));
  return max(int64_t(0), min(end, p.map.m_pad));
}
// (rounded down to what the sort writes: chunks of 64 rows of terms end inside m_pad)
__device__ __forceinline__ int64_t adapter_begin(const OuterParams& p, int i) {
  return i > 0 ? max(int64_t(0), min(static_cast<int64_t>(p.map.offsets[i - 1]), p.map.m_pad)) & ~int64_t(127) : 0;
}
// The segment with this number (wanted >= 0), or those of an adapter (index 0).  All
// threads call it: four adapters each, their counts summed over the block.  Where no adapter
// can have two (slots = 0), the number is the adapter's.
__device__ __forceinline__ Segment find_segment(const OuterParams& p, int64_t wanted, int of_adapter) {
  if (p.slots == 0) {
    const int i = static_cast<int>(wanted);
    return {i, 0, adapter_end(p, i) > adapter_begin(p, i) ? 1 : 0, 0};
  }
  __shared__ int sums[2][kWarps];
  __shared__ Segment found;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int count[4], all = 0, slots = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = 4 * threadIdx.x + k;
    count[k] = 0;
    if (i < p.map.adapters) {
      const int64_t rows = adapter_end(p, i) - adapter_begin(p, i);
      // (bounded, so that no offsets make the sums overflow: a sorted map has some hundreds)
      count[k] = rows > 0 ? static_cast<int>(min((rows + p.segment - 1) / p.segment, int64_t(1) << 20)) : 0;
    }
    all += count[k];
    slots += count[k] > 1 ? count[k] : 0;
  }
  int before = all, slot = slots;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, before, o), y = __shfl_up_sync(0xFFFFFFFFu, slot, o);
    if (lane >= o) { before += x; slot += y; }
  }
  if (lane == 31) { sums[0][warp] = before; sums[1][warp] = slot; }
  if (threadIdx.x == 0) found.adapter = -1;
  __syncthreads();
  before -= all;
  slot -= slots;
  for (int w = 0; w < warp; ++w) { before += sums[0][w]; slot += sums[1][w]; }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int i = 4 * threadIdx.x + k;
    if (i < p.map.adapters && (wanted >= 0 ? wanted >= before && wanted < before + count[k] : i == of_adapter))
      found = {i, wanted >= 0 ? static_cast<int>(wanted - before) : 0, count[k], slot};
    before += count[k];
    slot += count[k] > 1 ? count[k] : 0;
  }
  __syncthreads();
  return found;
}

// The largest of the threads' values, in all of them.
__device__ __forceinline__ float block_max(float v) {
  __shared__ float of_warp[kWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) v = fmaxf(v, of_warp[w]);
  return v;
}

// The largest |g| of 64 rows of the map, for float16's powers of two (4096 tokens, rank 32, all
// of the gradient 111 us; with the terms' blocks going through their segments by themselves
// 139).
constexpr int kTermRows = 64;
__global__ void __launch_bounds__(kThreads) outer_most_kernel(const __grid_constant__ OuterParams p) {
  let_next_kernel_start();
  wait_for_previous_kernel();
  const OuterSide& side = p.side[blockIdx.y];
  if (side.blocks == 0) return;
  const int quads = p.rank / 4;
  float most = 0.0f;
#pragma unroll 4
  for (int e = threadIdx.x; e < kTermRows * quads; e += kThreads) {
    const int i = e / quads;
    const int32_t t = token_at(p.map, static_cast<int64_t>(blockIdx.x) * kTermRows + i);
    float4 v = make_float4(0, 0, 0, 0);
    if (t >= 0) v = *reinterpret_cast<const float4*>(side.g + static_cast<int64_t>(t) * p.rank + (e - i * quads) * 4);
    most = fmaxf(fmaxf(most, fmaxf(fabsf(v.x), fabsf(v.y))), fmaxf(fabsf(v.z), fabsf(v.w)));
  }
  most = block_max(most);
  if (threadIdx.x == 0) side.most[blockIdx.x] = most;
}

// g of a segment's rows as terms of 16 bits, zeros for padding rows (up to a multiple of 64)
// and behind the rank (to a multiple of 16).  float16 keeps them inside its range by the
// segment's own power of two; its sums are scaled back before they are joined.
template <int KIND, int TERMS>
__global__ void __launch_bounds__(kThreads) outer_terms_kernel(const __grid_constant__ OuterParams p) {
  let_next_kernel_start();
  wait_for_previous_kernel();
  const OuterSide& side = p.side[blockIdx.y];
  const int chunks = p.segment / kTermRows;
  const int64_t number = blockIdx.x / chunks;
  const int chunk = static_cast<int>(blockIdx.x - number * chunks);
  const Segment seg = find_segment(p, number, 0);
  if (seg.adapter < 0 || side.blocks == 0) return;
  const int64_t row0 = adapter_begin(p, seg.adapter) + static_cast<int64_t>(seg.index) * p.segment;
  const int64_t row1 = min(row0 + p.segment, adapter_end(p, seg.adapter));
  const int quads = p.rank / 4;
  float unit = 1.0f;
  if (KIND == OK_F16) {
    float most = 0.0f;
    for (int64_t r = row0 + threadIdx.x * kTermRows; r < row1; r += kThreads * kTermRows) most = fmaxf(most, side.most[r / kTermRows]);
    unit = unit_of(block_max(most));
    if (threadIdx.x == 0) side.units[number] = unit;             // the same from each of them
  }
  const int ranks = (p.rank + 15) & ~15, all = ranks / 4;
  const int64_t from = row0 + static_cast<int64_t>(chunk) * kTermRows;
  if (from >= row1) return;
  for (int e = threadIdx.x; e < kTermRows * all; e += kThreads) {
    const int i = e / all, q = e - i * all;
    const int64_t r = from + i;
    if (r >= p.map.m_pad) break;
    const int32_t t = r < row1 ? token_at(p.map, r) : -1;
    float4 v = make_float4(0, 0, 0, 0);
    if (t >= 0 && q < quads) v = *reinterpret_cast<const float4*>(side.g + static_cast<int64_t>(t) * p.rank + q * 4);
    uint32_t lo[TERMS], hi[TERMS];
    split_terms<KIND, TERMS>(v.x * unit, v.y * unit, lo);
    split_terms<KIND, TERMS>(v.z * unit, v.w * unit, hi);
#pragma unroll
    for (int k = 0; k < TERMS; ++k)
      *reinterpret_cast<uint2*>(side.terms + (k * p.map.m_pad + r) * ranks + q * 4) = make_uint2(lo[k], hi[k]);
  }
}

template <int KIND, int R, int TERMS, bool FULL, bool RUNS>
__global__ void __launch_bounds__(kThreads, R <= 32 || !RUNS ? 2 : 1) outer_kernel(const __grid_constant__ OuterParams p) {
  using O = Outer<R, TERMS, RUNS>;
  constexpr int kTiles = O::kCols / 8 / kWarps;         // of 8 columns, a warp
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t token[O::kStages + 1][O::kTokens];
  const int rank = FULL ? R : p.rank, ranks = FULL ? R : (rank + 15) & ~15;
  const uint32_t base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_segment = p.side[0].blocks + p.side[1].blocks;
  const int64_t number = blockIdx.x / per_segment;
  int block = static_cast<int>(blockIdx.x - number * per_segment);
  const bool second = block >= p.side[0].blocks;
  const OuterSide& side = p.side[second ? 1 : 0];
  if (second) block -= p.side[0].blocks;
  const int64_t col0 = static_cast<int64_t>(block) * O::kCols;
  let_next_kernel_start();
  wait_for_previous_kernel();
  const Segment seg = find_segment(p, number, 0);
  // more sums than there is room for come of no map that the sort writes
  if (seg.adapter < 0 || (seg.count > 1 && seg.slot + seg.index >= p.slots)) return;
  // (without tokens, which only a numbering by adapters asks for, the sums are zeros)
  const int64_t row0 = adapter_begin(p, seg.adapter) + static_cast<int64_t>(seg.index) * p.segment;
  const int64_t row1 = min(row0 + p.segment, adapter_end(p, seg.adapter));
  const int chunks = static_cast<int>((row1 - row0 + O::kTokens - 1) / O::kTokens);
  auto token_of = [&](int c, int i) {
    const int64_t r = row0 + static_cast<int64_t>(c) * O::kTokens + i;
    return r < row1 ? token_at(p.map, r) : -1;
  };

  // a thread copies one piece of every kStep-th token's columns, and one of every kGStep-th
  // row of terms
  constexpr int kPieces = O::kCols / 8, kStep = kThreads / kPieces, kTermPieces = R / 8, kGStep = kThreads / kTermPieces;
  static_assert(kStep % 8 == 0, "a thread's rows have one swizzle");
  const int piece = threadIdx.x % kPieces, r0 = threadIdx.x / kPieces;
  const int g_piece = threadIdx.x % kTermPieces, g0 = threadIdx.x / kTermPieces;
  const bool in_cols = col0 + piece * 8 < side.width;
  const int64_t ldx = side.ldx, term_size = p.map.m_pad * ranks;
  const uint16_t* xp = static_cast<const uint16_t*>(side.x) + (in_cols ? col0 + piece * 8 : 0);
  const uint16_t* gp = side.terms + (row0 + g0) * ranks + g_piece * 8;
  const uint32_t x_to = base + (piece >> 3) * (O::kTokens * 128) + swizzled(r0, piece & 7);
  const uint32_t g_to = base + O::kXBytes + g0 * O::kTermPitch + g_piece * 16;
  auto load = [&](int c) {
    if (c < chunks) {
      const int32_t* tok = token[c % (O::kStages + 1)];
      const uint32_t stage = (c % O::kStages) * O::kStageBytes;
#pragma unroll
      for (int i = 0; i < O::kTokens / kStep; ++i) {
        const int32_t t = tok[r0 + i * kStep];
        copy16(x_to + stage + i * kStep * 128, xp + (t >= 0 ? t * ldx : 0), t >= 0 && in_cols ? 16 : 0);
      }
      if (FULL || g_piece * 8 < ranks) {
#pragma unroll
        for (int k = 0; k < TERMS; ++k)
#pragma unroll
          for (int i = 0; i < O::kTokens; i += kGStep)
            if (kGStep <= O::kTokens || g0 < O::kTokens)
              copy16(g_to + stage + k * O::kTermBytes + i * O::kTermPitch, gp + k * term_size + i * ranks, 16);
      }
      gp += O::kTokens * ranks;
    }
    copies_commit();
  };

  float acc[R / 16][kTiles][4], sum[RUNS ? R / 16 : 1][kTiles][4];
#pragma unroll
  for (int m = 0; m < R / 16; ++m)
#pragma unroll
    for (int i = 0; i < kTiles; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[m][i][k] = sum[RUNS ? m : 0][i][k] = 0.0f;
  for (int c = 0; c < O::kStages - 1; ++c)
    if (threadIdx.x < O::kTokens) token[c][threadIdx.x] = token_of(c, threadIdx.x);
  __syncthreads();
  for (int c = 0; c < O::kStages - 1; ++c) load(c);
  // a chunk's tokens are fetched two rounds before their rows are
  int32_t next = threadIdx.x < O::kTokens ? token_of(O::kStages - 1, threadIdx.x) : -1;
  const int run = RUNS ? kRun / O::kTokens : chunks;
  for (int c0 = 0; c0 < chunks; c0 += run) {
    if (RUNS) {
#pragma unroll
      for (int m = 0; m < R / 16; ++m)
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[m][i][k] = 0.0f;
    }
    const int c1 = min(c0 + run, chunks);
    for (int c = c0; c < c1; ++c) {
      const int ahead = c + O::kStages - 1;
      copies_wait<O::kStages - 2>();
      if (threadIdx.x < O::kTokens) token[ahead % (O::kStages + 1)][threadIdx.x] = next;
      __syncthreads();                                 // chunk c is there, c - 1 is read, the next one's tokens are known
      load(ahead);
      if (threadIdx.x < O::kTokens) next = token_of(ahead + 1, threadIdx.x);
      const uint32_t stage = base + (c % O::kStages) * O::kStageBytes;
#pragma unroll
      for (int s = 0; s < O::kTokens / 16; ++s) {
        uint32_t b[kTiles / 2][4];
#pragma unroll
        for (int i = 0; i < kTiles; i += 2) {
          const int tile = warp * kTiles + i;          // of 8 columns; 8 of them share 128 bytes
          load_matrices_t(b[i / 2], stage + (tile >> 3) * (O::kTokens * 128) + swizzled(s * 16 + (lane & 15), (tile & 7) + (lane >> 4)));
        }
        const uint32_t as = stage + O::kXBytes + (s * 16 + (lane & 7) + ((lane >> 4) << 3)) * O::kTermPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
        for (int k = 0; k < TERMS; ++k) {
          uint32_t a[R / 16][4];
#pragma unroll
          for (int m = 0; m < R / 16; ++m)
            if (FULL || m * 16 < rank) load_matrices_t(a[m], as + k * O::kTermBytes + m * 32);
#pragma unroll
          for (int m = 0; m < R / 16; ++m) {
            if (!FULL && m * 16 >= rank) break;
#pragma unroll
            for (int i = 0; i < kTiles; i += 2) {
              multiply<KIND>(acc[m][i], a[m], b[i / 2][0], b[i / 2][1]);
              multiply<KIND>(acc[m][i + 1], a[m], b[i / 2][2], b[i / 2][3]);
            }
          }
        }
      }
    }
    if (RUNS) {
#pragma unroll
      for (int m = 0; m < R / 16; ++m)
#pragma unroll
        for (int i = 0; i < kTiles; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[m][i][k] = sum[RUNS ? m : 0][i][k] += acc[m][i][k];
    }
  }
  copies_wait<0>();
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);
  const bool alone = seg.count <= 1;
  const float f = alone && chunks > 0 && side.scales != nullptr ? side.scales[seg.adapter] : 1.0f,
              back = KIND == OK_F16 && chunks > 0 ? 1.0f / side.units[number] : 1.0f;
#pragma unroll
  for (int m = 0; m < R / 16; ++m) {
    if (!FULL && m * 16 >= rank) break;
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
      float* at = sums + (m * 16 + (lane >> 2)) * O::kCols + (warp * kTiles + i) * 8 + 2 * (lane & 3);
      *reinterpret_cast<float2*>(at) = make_float2(acc[m][i][0] * back * f, acc[m][i][1] * back * f);
      *reinterpret_cast<float2*>(at + 8 * O::kCols) = make_float2(acc[m][i][2] * back * f, acc[m][i][3] * back * f);
    }
  }
  __syncthreads();
  const int64_t to = (alone ? static_cast<int64_t>(seg.adapter) : seg.slot + seg.index) * rank * side.width + col0 + piece * 8;
  for (int r = r0; r < rank; r += kStep) {
    if (!in_cols) break;
    const uint32_t at = base + (r * O::kCols + piece * 8) * 4;
    const float4 lo = get_shared4f(at), hi = get_shared4f(at + 16);
    const float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    const int64_t e = to + static_cast<int64_t>(r) * side.width;
    if (!alone) store8<OK_F32>(side.part, e, v);
    else if (p.out_kind == OK_F32) store8<OK_F32>(side.out, e, v);
    else if (p.out_kind == OK_F16) store8<OK_F16>(side.out, e, v);
    else store8<OK_BF16>(side.out, e, v);
  }
}

// The adapters of several segments (their sums in order, times f_i) and those of none
// (zeros): blockIdx.y is the adapter, a thread has eight values of either gradient.
__global__ void __launch_bounds__(kThreads) outer_join_kernel(const __grid_constant__ OuterParams p) {
  let_next_kernel_start();
  wait_for_previous_kernel();
  const Segment seg = find_segment(p, -1, blockIdx.y);
  if (seg.count == 1) return;
  const int64_t size0 = p.side[0].blocks > 0 ? static_cast<int64_t>(p.rank) * p.side[0].width : 0;
  const int64_t size1 = p.side[1].blocks > 0 ? static_cast<int64_t>(p.rank) * p.side[1].width : 0;
  for (int64_t e = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * 8; e < size0 + size1;
       e += static_cast<int64_t>(gridDim.x) * kThreads * 8) {
    const bool second = e >= size0;
    const OuterSide& side = p.side[second ? 1 : 0];
    const int64_t at = second ? e - size0 : e, size = second ? size1 : size0;
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll 4
    for (int k = 0; k < min(seg.count, p.slots - seg.slot); ++k) {
      float w[8];
      load8<OK_F32>(side.part, (seg.slot + k) * size + at, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += w[i];
    }
    if (side.scales != nullptr && seg.count > 0) {
      const float f = side.scales[seg.adapter];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= f;
    }
    const int64_t to = seg.adapter * size + at;
    if (p.out_kind == OK_F32) store8<OK_F32>(side.out, to, v);
    else if (p.out_kind == OK_F16) store8<OK_F16>(side.out, to, v);
    else store8<OK_BF16>(side.out, to, v);
  }
}

// ---------------------------------------------------------------- host
// Calls f with the least of 16, 32, 64, 128 that holds the rank, and whether it is the rank.
template <typename F>
bsgg_status with_rank(int rank, F&& f) {
  auto at = [&](auto r) {
    return rank == decltype(r)::value ? f(r, std::true_type()) : f(r, std::false_type());
  };
  if (rank <= 16) return at(std::integral_constant<int, 16>());
  if (rank <= 32) return at(std::integral_constant<int, 32>());
  if (rank <= 64) return at(std::integral_constant<int, 64>());
  return at(std::integral_constant<int, 128>());
}
template <typename F>
bsgg_status with_half(int format, F&& f) {
  return format == BSGG_OUT_BF16 ? f(std::integral_constant<int, OK_BF16>()) : f(std::integral_constant<int, OK_F16>());
}
// Tiles of `rows` rows that can hold tokens, at the most.
int64_t busy_tiles(const AdapterMap& m, int rows) {
  const int64_t most = (m.tokens < m.adapters ? m.tokens : m.adapters) + m.tokens / rows;
  const int64_t all = m.m_pad / rows;
  return most < all ? most : all;
}

bsgg_status launch_shrink(int format, ShrinkParams p, cudaStream_t s) {
  const int64_t tiles = p.map.m_pad / 64, busy = busy_tiles(p.map, 64), nb = ceil_div(p.depth, 64);
  p.split = 1;
  while (p.split < kMaxCluster && busy * p.split < 228 && nb >= 4 * p.split) p.split *= 2;
  return with_half(format, [&](auto kind) {
    return with_rank(p.rank, [&](auto r, auto full) {
      constexpr int K = decltype(kind)::value, R = decltype(r)::value;
      constexpr bool E = decltype(full)::value;
      auto launch = [&](auto runs) {
        constexpr bool N = decltype(runs)::value;
        if (!allowed<shrink_kernel<K, R, E, N>>(Shrink<R>::kSmem)) return BSGG_ERR_CUDA;
        const LaunchConfig c(dim3(static_cast<unsigned>(tiles * p.split)), kThreads, Shrink<R>::kSmem, s, p.split);
        return launch_kernel(c, shrink_kernel<K, R, E, N>, p);
      };
      // two warps at least share a part: of up to 1024 each sums a run.  At a rank of 128 the
      // registers for more leave room for one block on an SM: 3362 tokens, 1952 wide, rank 88,
      // take 46 us with their expand and 32 without; 904 tokens, 7152 wide, whose blocks have
      // an SM each anyway, 30 with and 37 without
      if constexpr (R == 128) {
        if (ceil_div(nb, p.split) * 64 <= 2 * kRun && busy * p.split > 228) return launch(std::false_type());
      }
      return launch(std::true_type());
    });
  });
}

// A launch has less than 2^31 blocks; the calls refuse sizes that want more before anything runs.
bool fits_grid(int64_t blocks) { return blocks < (int64_t(1) << 31); }

// Sets how the tiles and columns are shared out; the number of blocks.
int64_t plan_expand(ExpandParams& p) {
  p.tiles = p.map.m_pad / 128;
  const int64_t rest = ceil_div(p.map.tokens, kRestTokens);
  int most = 0;
  with_rank(p.rank, [&](auto r, auto) {
    most = Expand<decltype(r)::value>::kCols;
    return BSGG_OK;
  });
  // the fewer tiles hold tokens, the fewer columns a block takes, down to a warp's 64: 109
  // tokens of 13 adapters, 3688 wide, took 14 us in blocks of 1024 columns
  const int64_t each = ceil_div(p.width, ceil_div(304, busy_tiles(p.map, 128)));
  p.cols = static_cast<int>(ceil_div(each, 64) * 64);
  if (p.cols > most) p.cols = most;
  p.col_blocks = static_cast<int>(ceil_div(p.width, p.cols));
  // six blocks an SM for the tokens without an adapter, whose number only the map knows (4096
  // tokens, 14336 wide, a fifth of them without: 91 us with two, 79 with six, 81 with sixteen)
  const int64_t parts = ceil_div(912, rest);
  p.rest_parts = static_cast<int>(parts < p.col_blocks ? parts : p.col_blocks);
  return p.tiles * p.col_blocks + rest * p.rest_parts;
}

bsgg_status launch_expand(int format, const ExpandParams& p, int64_t grid, cudaStream_t s) {
  return with_half(format, [&](auto kind) {
    return with_rank(p.rank, [&](auto r, auto full) {
      constexpr int K = decltype(kind)::value, R = decltype(r)::value;
      constexpr bool E = decltype(full)::value;
      if (!allowed<expand_kernel<K, R, E>>(Expand<R>::kSmem)) return BSGG_ERR_CUDA;
      const LaunchConfig c(dim3(static_cast<unsigned>(grid)), kThreads, Expand<R>::kSmem, s);
      return launch_kernel(c, expand_kernel<K, R, E>, p);
    });
  });
}

// Rows of a segment: 128, or as many more as make the blocks one or two rounds of two an SM.
// 4096 tokens of 4 adapters, rank 32, 4096 and 14336, all of the gradient: 107 us (1024 rows; with
// half as many 112, twice as many 114); rank 128 268 (286); 8192 tokens, rank 64, 1024 wide, 75
// (92); 16384 tokens of 8 adapters, rank 16, 4096 wide, 158 (157, and 181 with twice as many).
// Layers so wide that one segment of all tokens has more blocks than that stay with one.
int64_t outer_segment(int64_t tokens, int64_t k, int64_t n) {
  const int64_t blocks = ceil_div(k, 256) + ceil_div(n, 256);
  int64_t rows = 128;
  while (rows < tokens && ceil_div(tokens, rows) * blocks > 456) rows *= 2;
  return rows;
}
// Sums of segments that can be needed at once: only adapters of several segments have any.
int64_t outer_slots(int64_t tokens, int64_t k, int64_t n) {
  const int64_t rows = outer_segment(tokens, k, n);
  return tokens > rows ? 2 * ceil_div(tokens, rows) : 0;
}

// Segments of a map, at the most; where a segment holds all tokens, one for each adapter.
int64_t outer_segments(int64_t tokens, int64_t m_pad, int64_t adapters, int64_t rows) {
  if (tokens <= rows) return adapters;
  // an adapter's rows are its tokens rounded up to 128
  const int64_t used = tokens < adapters ? tokens : adapters, all = tokens + 128 * used;
  return used + (all < m_pad ? all : m_pad) / rows;
}

// What lies where in the workspace, in bytes: both sides' terms (three at the most), their
// units and largest values, and the segments' sums.
struct OuterSpace {
  uint64_t terms[2], units[2], most[2], part[2], bytes;
  OuterSpace(int64_t tokens, int64_t k, int64_t n, int64_t m_pad, int64_t adapters, int64_t rank) {
    uint64_t at = 0;
    auto take = [&](uint64_t size) {
      const uint64_t from = at;
      at += (size + 15) / 16 * 16;
      return from;
    };
    const int64_t segments = outer_segments(tokens, m_pad, adapters, outer_segment(tokens, k, n)), slots = outer_slots(tokens, k, n);
    for (uint64_t& t : terms) t = take(uint64_t(6) * m_pad * ((rank + 15) / 16 * 16));
    for (uint64_t& u : units) u = take(uint64_t(4) * segments);
    for (uint64_t& v : most) v = take(uint64_t(4) * (m_pad / kTermRows));
    part[0] = take(uint64_t(4) * slots * rank * n);
    part[1] = take(uint64_t(4) * slots * rank * k);
    bytes = at;
  }
};

// Sets the blocks of columns; the most blocks that a launch of the gradient has.
int64_t plan_outer(OuterParams& p) {
  with_rank(p.rank, [&](auto r, auto) {
    for (OuterSide& side : p.side)
      side.blocks = side.out != nullptr ? static_cast<int>(ceil_div(side.width, Outer<decltype(r)::value, 2, true>::kCols)) : 0;
    return BSGG_OK;
  });
  const int64_t segments = outer_segments(p.map.tokens, p.map.m_pad, p.map.adapters, p.segment);
  const int64_t products = segments * (p.side[0].blocks + p.side[1].blocks), terms = segments * (p.segment / kTermRows);
  return products > terms ? products : terms;
}

bsgg_status launch_outer(int format, const OuterParams& p, cudaStream_t s) {
  return with_half(format, [&](auto kind) {
    return with_rank(p.rank, [&](auto r, auto full) {
      constexpr int K = decltype(kind)::value, R = decltype(r)::value;
      constexpr bool E = decltype(full)::value;
      int64_t most = 0;
      for (const OuterSide& side : p.side) most += side.out != nullptr ? ceil_div(int64_t(p.rank) * side.width, 8 * kThreads) : 0;
      const int64_t segments = outer_segments(p.map.tokens, p.map.m_pad, p.map.adapters, p.segment), grid = segments * (p.side[0].blocks + p.side[1].blocks);
      auto launch = [&](auto terms, auto runs) {
        constexpr int N = decltype(terms)::value;
        constexpr bool U = decltype(runs)::value;
        constexpr int kSmem = Outer<R, N, U>::kSmem;
        if (!allowed<outer_kernel<K, R, N, E, U>>(kSmem)) return BSGG_ERR_CUDA;
        bsgg_status st = BSGG_OK;
        if (K == OK_F16) {
          const LaunchConfig v(dim3(static_cast<unsigned>(p.map.m_pad / kTermRows), 2), kThreads, 0, s);
          st = launch_kernel(v, outer_most_kernel, p);
          if (st != BSGG_OK) return st;
        }
        const LaunchConfig t(dim3(static_cast<unsigned>(segments * (p.segment / kTermRows)), 2), kThreads, 0, s);
        st = launch_kernel(t, outer_terms_kernel<K, N>, p);
        if (st != BSGG_OK) return st;
        const LaunchConfig c(dim3(static_cast<unsigned>(grid)), kThreads, kSmem, s);
        st = launch_kernel(c, outer_kernel<K, R, N, E, U>, p);
        if (st != BSGG_OK || p.slots == 0) return st;
        // two rounds of blocks over all adapters
        const int64_t each = 2432 / p.map.adapters < 1 ? 1 : 2432 / p.map.adapters;
        const LaunchConfig j(dim3(static_cast<unsigned>(most < each ? most : each), static_cast<unsigned>(p.map.adapters)), kThreads, 0, s);
        return launch_kernel(j, outer_join_kernel, p);
      };
      // What is rounded to 16 bits is summed whole at ranks over 32, as long as what the additions
      // drop is under an eighth of the rounding where all products have one sign: into bfloat16
      // up to 32768 rows (2.3e-4 of 3.9e-3), into float16 up to 8192 (5.9e-5 of 4.9e-4).  Without
      // registers for runs two blocks fit an SM (4096 tokens in segments of 512, rank 64, all of the
      // gradient 150 us for 167, rank 128 284 for 320; db alone of 8192 tokens in one segment, 45056
      // wide, rank 64, 377 for 445; at ranks 16 and 32 no change)
      if (R > 32 && p.out_kind != OK_F32 && p.segment <= (p.out_kind == OK_F16 ? 8192 : 32768)) {
        if constexpr (R > 32) return launch(std::integral_constant<int, 2>(), std::false_type());
      }
      if constexpr (K == OK_BF16) {
        if (p.out_kind == OK_F32) return launch(std::integral_constant<int, 3>(), std::true_type());
      }
      return launch(std::integral_constant<int, 2>(), std::true_type());
    });
  });
}

bool good_width(int64_t v) { return v >= 8 && v <= (int64_t(1) << 24) && v % 8 == 0; }
bool good_pitch(int64_t ld, int64_t cols) { return ld >= cols && ld <= (int64_t(1) << 30) && ld % 8 == 0; }

bsgg_status check_adapters(int64_t tokens, int64_t k, int64_t n, int64_t m_pad, int adapters, int rank, int format) {
  if (tokens < 0 || tokens > (int64_t(1) << 30) || !good_width(k) || !good_width(n) || m_pad <= 0 || m_pad % 128 != 0 ||
      m_pad > (int64_t(1) << 30) || adapters < 1 || adapters > 1024 || rank < 8 || rank > 128 || rank % 8 != 0 ||
      (format != BSGG_OUT_BF16 && format != BSGG_OUT_F16))
    return BSGG_ERR_INVALID_ARG;
  return BSGG_OK;
}

}  // namespace

extern "C" {

bsgg_status bsgg_adapters(const bsgg_adapters_desc* d, const void* x, const void* a, const void* b, const float* scales,
                          const int32_t* padded_offsets, const int32_t* row_of_slot, const int32_t* slot_of_row,
                          const void* base, float* u, void* y, void* stream) {
  if (!d || d->reserved != 0) return BSGG_ERR_INVALID_ARG;
  const bsgg_status st = check_adapters(d->tokens, d->k, d->n, d->m_pad, d->adapters, d->rank, d->format);
  if (st != BSGG_OK) return st;
  if (!good_pitch(d->ldx, d->k) || !good_pitch(d->ldy, d->n) || (base && !good_pitch(d->ld_base, d->n)) ||
      (base && base == y && d->ld_base != d->ldy))
    return BSGG_ERR_INVALID_ARG;
  if (d->tokens == 0) return BSGG_OK;
  if (!x || !a || !b || !padded_offsets || !row_of_slot || !slot_of_row || !u || !y) return BSGG_ERR_INVALID_ARG;
  for (const void* q : {x, a, b, base, static_cast<const void*>(u), static_cast<const void*>(y)})
    if (!aligned_to(q, 16)) return BSGG_ERR_INVALID_ARG;
  if (!aligned_to(scales, 4) || !aligned_to(padded_offsets, 4) || !aligned_to(row_of_slot, 4) || !aligned_to(slot_of_row, 4))
    return BSGG_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const AdapterMap map = {d->tokens, d->m_pad, d->adapters, padded_offsets, row_of_slot, slot_of_row};
  ExpandParams e = {map, u, b, scales, base, y, u, 0, base ? static_cast<int>(d->ld_base) : 0, static_cast<int>(d->ldy),
                    static_cast<int>(d->n), d->rank};
  const int64_t grid = plan_expand(e);
  if (!fits_grid(grid)) return BSGG_ERR_UNSUPPORTED;
  const bsgg_status ran = launch_shrink(d->format, {map, x, a, nullptr, u, d->ldx, static_cast<int>(d->k), d->rank, 1}, s);
  return ran == BSGG_OK ? launch_expand(d->format, e, grid, s) : ran;
}

uint64_t bsgg_adapters_workspace_bytes(int64_t tokens, int64_t k, int64_t n, int64_t m_pad, int32_t adapters, int32_t rank) {
  if (check_adapters(tokens, k, n, m_pad, adapters, rank, BSGG_OUT_BF16) != BSGG_OK || tokens == 0) return 0;
  return OuterSpace(tokens, k, n, m_pad, adapters, rank).bytes;
}

bsgg_status bsgg_adapters_backward(const bsgg_adapters_bwd_desc* d, const void* dy, const void* x, const float* u,
                                   const void* a, const void* b, const float* scales, const int32_t* padded_offsets,
                                   const int32_t* row_of_slot, const int32_t* slot_of_row, const int32_t* rows_used,
                                   const void* base, float* du, void* dx, void* da, void* db, void* workspace, void* stream) {
  if (!d) return BSGG_ERR_INVALID_ARG;
  const bsgg_status st = check_adapters(d->tokens, d->k, d->n, d->m_pad, d->adapters, d->rank, d->format);
  if (st != BSGG_OK) return st;
  if (!good_pitch(d->ld_dy, d->n) || (da && !good_pitch(d->ldx, d->k)) || (dx && !good_pitch(d->ld_dx, d->k)) ||
      (dx && base && !good_pitch(d->ld_base, d->k)) || (dx && base && base == dx && d->ld_base != d->ld_dx))
    return BSGG_ERR_INVALID_ARG;
  if ((da || db) && !is_float_format(d->grad_format)) return BSGG_ERR_INVALID_ARG;
  for (const void* q : {dy, x, a, b, base, static_cast<const void*>(u), static_cast<const void*>(du),
                        static_cast<const void*>(dx), static_cast<const void*>(da), static_cast<const void*>(db),
                        static_cast<const void*>(workspace)})
    if (!aligned_to(q, 16)) return BSGG_ERR_INVALID_ARG;
  if (!aligned_to(scales, 4) || !aligned_to(padded_offsets, 4) || !aligned_to(row_of_slot, 4) || !aligned_to(slot_of_row, 4) ||
      !aligned_to(rows_used, 4))
    return BSGG_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->tokens == 0) {
    // empty sums
    const size_t es = static_cast<size_t>(float_bytes(d->grad_format)) * d->adapters * d->rank;
    if ((da && !succeeded(cudaMemsetAsync(da, 0, es * d->k, s))) || (db && !succeeded(cudaMemsetAsync(db, 0, es * d->n, s))))
      return BSGG_ERR_CUDA;
    return BSGG_OK;
  }
  if (!dx && !da && !db) return BSGG_ERR_INVALID_ARG;
  const bool wants_du = dx || da;
  if (!dy || !padded_offsets || !slot_of_row || (wants_du && (!b || !du)) || (dx && (!a || !row_of_slot)) || (da && !x) ||
      (db && !u) || ((da || db) && !rows_used) || ((da || db) && !workspace))
    return BSGG_ERR_INVALID_ARG;
  const AdapterMap map = {d->tokens, d->m_pad, d->adapters, padded_offsets, row_of_slot, slot_of_row};
  ExpandParams e = {map, du, a, nullptr, base, dx, nullptr, 0, base ? static_cast<int>(d->ld_base) : 0, static_cast<int>(d->ld_dx),
                    static_cast<int>(d->k), d->rank};
  const int64_t grid = dx ? plan_expand(e) : 0;
  if (!fits_grid(grid)) return BSGG_ERR_UNSUPPORTED;
  OuterParams p = {};
  if (da || db) {
    p.map = map; p.rows_used = rows_used; p.rank = d->rank; p.out_kind = d->grad_format;
    p.segment = static_cast<int>(outer_segment(d->tokens, d->k, d->n));
    p.slots = static_cast<int>(outer_slots(d->tokens, d->k, d->n));
    const OuterSpace space(d->tokens, d->k, d->n, d->m_pad, d->adapters, d->rank);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    auto side = [&](int i, const float* g, const void* in, const float* f, void* out, int64_t ld, int64_t width) {
      p.side[i] = {g, in, f, out, reinterpret_cast<float*>(ws + space.part[i]), reinterpret_cast<uint16_t*>(ws + space.terms[i]),
                   reinterpret_cast<float*>(ws + space.units[i]), reinterpret_cast<float*>(ws + space.most[i]), ld, static_cast<int>(width), 0};
    };
    side(0, u, dy, scales, db, d->ld_dy, d->n);
    side(1, du, x, nullptr, da, d->ldx, d->k);
    if (!fits_grid(plan_outer(p))) return BSGG_ERR_UNSUPPORTED;
  }
  bsgg_status ran = BSGG_OK;
  if (wants_du) ran = launch_shrink(d->format, {map, dy, b, scales, du, d->ld_dy, static_cast<int>(d->n), d->rank, 1}, s);
  if (ran == BSGG_OK && (da || db)) ran = launch_outer(d->format, p, s);
  if (ran == BSGG_OK && dx) ran = launch_expand(d->format, e, grid, s);
  return ran;
}

}  // extern "C"
