// bsgg_router.cu -- routing with softmax or sigmoid scores, a bias that steers the
// choice, and experts in groups; and its gradient.
#include <cmath>

#include "bsgg_ops.cuh"

namespace {

using namespace bsgg;

constexpr int kRouterWarps = 4;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct RouterParams {
  int64_t tokens, ld;
  int L, groups, size, topk, topk_groups, group_top;   // size: experts of a group
  int per;                    // lanes of a group: the largest power of two with groups * per <= 32
  int kind, sigmoid, normalize;
  float scale;
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
};

// 1 / (1 + e^-l), with e^-|l| on either side: as exact near 0 as near 1.
__device__ __forceinline__ float sigmoid32(float l) {
  const float e = expf(-fabsf(l));
  return (l >= 0.0f ? 1.0f : e) / (1.0f + e);
}
// The same for the choice, with the hardware's exponential and quotient: off by 2^-21 at most
// (e^-l by (2 + 1.2 |l|) 2^-23 of itself, which moves the score by its slope, the quotient by
// 2^-22), and by 2^-15 of itself down to l = -87.3.  There the denominator passes 2^126 and the
// quotient is 0: off by 2^-126, which is less than the least that two scores have to differ.
__device__ __forceinline__ float sigmoid_choice(float l) { return __fdividef(1.0f, 1.0f + __expf(-l)); }
__device__ __forceinline__ double sigmoid64(double l) {
  const double e = exp(-fabs(l));
  return (l >= 0.0 ? 1.0 : e) / (1.0 + e);
}

// Order-preserving key of a double, as logit_key.
__device__ __forceinline__ uint64_t key64(double x) {
  if (x != x) return ~0ull;
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(x + 0.0));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}
// The largest over the warp.
__device__ __forceinline__ uint64_t warp_max64(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
  const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// Where a warp's lanes have a token's experts, and how these score.  Lane g * per + q
// holds experts q, q + per, ... of group g (of the whole row without groups, `per` = 32).
struct Row {
  int64_t at;                 // of the row's logits
  int first, own;             // this lane's first expert; how many it has
  float m;                    // largest logit (softmax)
};
__device__ __forceinline__ float row_logit(const RouterParams& p, const Row& r, int i) {
  return load1(p.kind, p.logits, r.at + r.first + p.per * i);
}
// The sum of e^(l - m) in 64 bits, 1 where it is not needed.  Called by all lanes together.
__device__ __forceinline__ double row_sum64(const RouterParams& p, const Row& r) {
  if (p.sigmoid || p.bias == nullptr) return 1.0;        // without a bias only ratios matter
  double sum = 0.0;
#pragma unroll 1
  for (int i = 0; i < r.own; ++i) {
    const float l = row_logit(p, r, i);
    if (!(l == -INFINITY)) sum += exp(static_cast<double>(l) - static_cast<double>(r.m));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  return sum;
}
// The key of expert i's c in 64 bits, 0 for a masked one.
__device__ __forceinline__ uint64_t row_choice64(const RouterParams& p, const Row& r, double sum, int i) {
  const float l = row_logit(p, r, i);
  const float b = p.bias != nullptr ? p.bias[r.first + p.per * i] : 0.0f;
  if (l == -INFINITY || b == -INFINITY) return 0;
  const double s = p.sigmoid ? sigmoid64(l) : exp(static_cast<double>(l) - static_cast<double>(r.m)) / sum;
  return key64(s + static_cast<double>(b));
}

// The top two of two pairs' (a >= b, x >= y).
template <typename T>
__device__ __forceinline__ void top_two(T& a, T& b, T x, T y) {
  const T low = a < x ? a : x;
  a = a < x ? x : a;
  b = b < y ? y : b;
  b = b < low ? low : b;
}

// A group's score in 64 bits, as a key, the same in all of its lanes, from those of this
// lane's experts that are in `open` (bits: the ones that may be among its best two); called
// by all lanes of the warp.
__device__ __noinline__ uint64_t group64(const RouterParams& p, Row r, uint64_t open) {
  const double sum = row_sum64(p, r);
  uint64_t a = 0, b = 0;
#pragma unroll 1
  while (open != 0) {
    const int i = __ffsll(static_cast<long long>(open)) - 1;
    open &= open - 1;
    top_two(a, b, row_choice64(p, r, sum, i), uint64_t(0));
  }
  __syncwarp();
  for (int o = 1; o < p.per; o <<= 1) {
    const uint64_t x = __shfl_xor_sync(kAll, a, o), y = __shfl_xor_sync(kAll, b, o);
    top_two(a, b, x, y);
  }
  auto value = [](uint64_t k) { return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & ~(1ull << 63)) : ~k)); };
  return p.group_top == 1 || b == 0 ? a : key64(value(a) + value(b));
}

// Whether the experts in `open` (bits of this lane's, of the groups in doubt) all have one
// logit and one bias, and each such group two of them: then the groups are equal.  A router
// that starts from zeros has such rows.  Called by all lanes of the warp.
__device__ __noinline__ bool all_alike(const RouterParams& p, Row r, uint64_t open) {
  int count = __popcll(open);
  for (int o = 1; o < p.per; o <<= 1) count += __shfl_xor_sync(kAll, count, o);
  uint32_t low[2] = {kAll, kAll}, high[2] = {0, 0};
  const bool some = open != 0;
#pragma unroll 1
  while (open != 0) {
    const int i = __ffsll(static_cast<long long>(open)) - 1;
    open &= open - 1;
    const uint32_t k[2] = {logit_key(row_logit(p, r, i)), logit_key(p.bias[r.first + p.per * i])};
    for (int j = 0; j < 2; ++j) { low[j] = min(low[j], k[j]); high[j] = max(high[j], k[j]); }
  }
  __syncwarp();
  bool alike = !__any_sync(kAll, some && count < 2);
  for (int j = 0; j < 2; ++j) {
    const uint32_t least = __reduce_min_sync(kAll, low[j]), most = __reduce_max_sync(kAll, high[j]);
    alike = alike && least == most;
  }
  return alike;
}

// Of the experts in `near` (bits of this lane's) the best by c in 64 bits: its index in
// the lane that has it, kAll in the others.  Called by all lanes of the warp.
__device__ __noinline__ uint32_t expert64(const RouterParams& p, Row r, uint64_t near) {
  const double sum = row_sum64(p, r);
  uint64_t k = 0;
  uint32_t best = kAll;
#pragma unroll 1
  while (near != 0) {                              // ascending: the lowest of equals stays
    const int i = __ffsll(static_cast<long long>(near)) - 1;
    near &= near - 1;
    const uint64_t c = row_choice64(p, r, sum, i);
    if (c > k) { k = c; best = static_cast<uint32_t>(r.first + p.per * i); }
  }
  __syncwarp();
  return k == warp_max64(k) ? best : kAll;
}

template <int KIND, int NI>
__device__ __forceinline__ void load_logits(const RouterParams& p, const Row& r, float (&l)[NI]) {
#pragma unroll
  for (int i = 0; i < NI; ++i) l[i] = i < r.own ? load1<KIND>(p.logits, r.at + r.first + p.per * i) : -INFINITY;
}

// The experts left with a key of at least `least`, as bits of this lane's.
template <int NI>
__device__ __forceinline__ uint64_t keys_from(const uint32_t (&key)[NI], uint32_t least) {
  uint64_t bits = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (key[i] >= least && key[i] > kMaskedKey) bits |= 1ull << i;
  return bits;
}
// The best expert left: its key, and its index (the lowest of equals).
template <int NI>
__device__ __forceinline__ uint32_t best_left(const uint32_t (&key)[NI], const Row& row, int per, uint32_t& e) {
  uint32_t m = key[0];
  int at = 0;
#pragma unroll
  for (int i = 1; i < NI; ++i)
    if (key[i] > m) { m = key[i]; at = i; }
  const uint32_t best = __reduce_max_sync(kAll, m);
  e = __reduce_min_sync(kAll, m == best ? static_cast<uint32_t>(row.first + per * at) : kAll);
  return best;
}
template <int NI>
__device__ __forceinline__ void set_key(uint32_t (&key)[NI], const Row& row, int per, uint32_t e, uint32_t to) {
#pragma unroll
  for (int i = 0; i < NI; ++i)
    if (e == static_cast<uint32_t>(row.first + per * i) && i < row.own) key[i] = to;
}

// One warp per token.  Its experts go by 32-bit keys (logits themselves without a bias,
// where they are exact): each round takes a warp's maximum and the lowest index that has
// it.  With a bias a choice is certain only where it leads the next one by more than
// what 32-bit scores may be off; that is looked at once for all rounds, a lane per choice,
// one round more than there are choices.  Where it fails, in some hundredths of a per
// cent of the rows, the rounds are gone through again, and those of each round that are
// that near are compared in 64 bits.  Equal logits under equal biases are equal, and
// need none of it.  Groups likewise, but there only the last one kept has to lead.
//   8192 x 256 bfloat16, top-8 of the best 4 of 8 groups, sigmoid and bias: 20 us (4.2 MB: 0.6
//   of them the bytes'; the plain softmax router 12.5); 16384 x 128 float32, top-4 of 3 of 8: 21; 128
//   x 64 top-8: 4.2.  8192 x 256 whose every row is in doubt to the last choice: 1150.  Without a
//   bias 16; normal logits times 8, groups of two large scores: softmax 19, sigmoid 41 (sums near 2
//   that 32 bits do not tell apart), times 16 softmax 34.  Bound by
//   issue (58 to 67 % of the slots; 1350 instructions a token of 256 experts, half of them the
//   rounds).  With the near ones looked for in every round 25 and 23 us.
template <int NI>
__global__ void __launch_bounds__(32 * kRouterWarps) route_groups_kernel(const __grid_constant__ RouterParams p) {
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const int group = lane / p.per, q = lane - group * p.per;
  Row row = {t * p.ld, group * p.size + q, 0, 0.0f};
  row.own = group < p.groups && q < p.size ? (p.size - q + p.per - 1) / p.per : 0;
  uint32_t key[NI];
  float l[NI];
  if (p.kind == OK_F32) load_logits<OK_F32>(p, row, l);
  else if (p.kind == OK_F16) load_logits<OK_F16>(p, row, l);
  else load_logits<OK_BF16>(p, row, l);
  const bool biased = p.bias != nullptr;
  float total = 0.0f, off = 0.0f;            // softmax's denominator; the most a 32-bit score is off
  if (!p.sigmoid) {
    row.m = l[0];
#pragma unroll
    for (int i = 1; i < NI; ++i) row.m = fmaxf(row.m, l[i]);
    row.m = warp_max(row.m);
    if (biased || !p.normalize) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (!(l[i] == -INFINITY)) total += expf(l[i] - row.m);
      total = warp_sum(total);
    }
  }
  if (biased) {
    // a softmax's score, 1 / total at most, is off by 2^-17 of that (64 + 5 roundings of the sum)
    const float inv = p.sigmoid ? 0.0f : 1.0f / total;
    off = p.sigmoid ? 0x1p-21f : 0x1p-17f * fminf(inv, 1.0f);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float c = -INFINITY;
      if (!(l[i] == -INFINITY)) c = (p.sigmoid ? sigmoid_choice(l[i]) : expf(l[i] - row.m) * inv) + p.bias[row.first + p.per * i];
      key[i] = logit_key(c);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NI; ++i) key[i] = logit_key(l[i]);
  }

  // ---- groups
  if (p.topk_groups < p.groups) {
    uint32_t a = 0, b = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) top_two(a, b, key[i], 0u);
    for (int o = 1; o < p.per; o <<= 1) {
      const uint32_t x = __shfl_xor_sync(kAll, a, o), y = __shfl_xor_sync(kAll, b, o);
      top_two(a, b, x, y);
    }
    uint32_t g = a;
    float size = 0.0f;                             // of the sum's terms
    if (a <= kMaskedKey || group >= p.groups) {
      g = 0;
    } else {
      auto value = [&](uint32_t k) {
        const float v = key_logit(k);
        return biased ? v : p.sigmoid ? sigmoid_choice(v) : expf(v - row.m);
      };
      size = fabsf(key_logit(a));
      if (p.group_top == 2) {
        const float x = value(a), y = b > kMaskedKey ? value(b) : 0.0f;
        g = logit_key(x + y);
        size = fabsf(x) + fabsf(y);
      }
    }
    const uint32_t g0 = g;
    bool kept = false;
    uint32_t last = 0;                             // the last group kept
    int who = 0;
    for (int j = 0; j < p.topk_groups; ++j) {
      const uint32_t best = __reduce_max_sync(kAll, g);
      if (best == 0) { last = 0; break; }
      last = best;
      who = __ffs(__ballot_sync(kAll, g == best)) - 1;             // the lowest of equals
      if (group == who / p.per) { kept = true; g = 0; }
    }
    const uint32_t rest = __reduce_max_sync(kAll, g);
    if ((biased || p.group_top == 2) && last != 0 && rest != 0) {
      // with a bias two scores of `off` each and roundings; without one each is positive and off
      // by 2^-15 of itself at most, or by 2^-126.  (Of the largest group: more than the last one
      // kept needs, so that rows of a few large scores are compared in 64 bits oftener than they
      // have to be.)
      const float most = warp_max(size);
      const float slack = biased ? 4.0f * off + 0x1p-20f * most : 0x1p-13f * most + 0x1p-120f;
      const uint32_t last_a = __shfl_sync(kAll, a, who), last_b = __shfl_sync(kAll, b, who);
      const bool near = g0 != 0 && (g0 == last || fabsf(key_logit(g0) - key_logit(last)) <= slack);
      // groups with the same two logits are equal, and in order of index: common where logits
      // have few bits
      const bool same = !biased && a == last_a && b == last_b;
      const bool left_out = __any_sync(kAll, near && g != 0), unlike = __any_sync(kAll, near && !same);
      // the experts that may be a group's best two
      const float least = b > kMaskedKey ? key_logit(b) : -INFINITY;
      const float under = least - (2.0f * off + 0x1p-21f * fabsf(least));
      const bool doubt = left_out && unlike;
      const uint64_t open = doubt ? keys_from(key, biased && b != kAll ? logit_key(under) : biased ? 0u : p.group_top == 2 ? b : a) : 0;
      if (doubt && !(biased && all_alike(p, row, near ? open : 0))) {
        // all of the groups in 64 bits
        uint64_t k = group64(p, row, g0 != 0 ? open : 0);
        if (g0 == 0) k = 0;
        kept = false;
        for (int j = 0; j < p.topk_groups; ++j) {
          const uint64_t best = warp_max64(k);
          if (best == 0) break;
          const int winner = (__ffs(__ballot_sync(kAll, k == best)) - 1) / p.per;
          if (group == winner) { kept = true; k = 0; }
        }
      }
    }
    if (!kept) {
#pragma unroll
      for (int i = 0; i < NI; ++i) key[i] = 0u;
    }
  }

  // ---- experts: lane j has choice j, its key and (with a bias) its logit and bias
  int32_t my_id = -1;
  uint32_t my_key = 0;
  for (int j = 0; j < p.topk; ++j) {
    uint32_t e;
    const uint32_t best = best_left(key, row, p.per, e);
    if (best <= kMaskedKey) break;                 // only masked experts are left
    set_key(key, row, p.per, e, 0u);
    if (lane == j) { my_id = static_cast<int32_t>(e); my_key = best; }
  }
  float mine = my_id >= 0 ? load1(p.kind, p.logits, row.at + my_id) : -INFINITY;
  if (biased) {
    uint32_t rest_id;
    const uint32_t rest = best_left(key, row, p.per, rest_id);
    const float my_bias = my_id >= 0 ? p.bias[my_id] : 0.0f;
    uint32_t next = __shfl_down_sync(kAll, my_key, 1);
    float next_logit = __shfl_down_sync(kAll, mine, 1), next_bias = __shfl_down_sync(kAll, my_bias, 1);
    if (lane == p.topk - 1) {
      next = rest;
      if (rest > kMaskedKey) {
        next_logit = load1(p.kind, p.logits, row.at + rest_id);
        next_bias = p.bias[rest_id];
      }
    }
    const float v = key_logit(my_key);
    const bool tie = my_key == next && mine == next_logit && my_bias == next_bias;     // in order of index already
    const bool open = lane < p.topk && my_id >= 0 && next > kMaskedKey && !tie &&
                      !(key_logit(next) < v - (2.0f * off + 0x1p-22f * fabsf(v))) && v < INFINITY;
    // equal infinities, and NaN, are in order of index
    if (__any_sync(kAll, open && v == v)) {
      for (int j = 0; j < p.topk; ++j) {
        const uint32_t e = static_cast<uint32_t>(__shfl_sync(kAll, my_id, j)), k = __shfl_sync(kAll, my_key, j);
        set_key(key, row, p.per, e, k);
      }
      my_id = -1;
      for (int j = 0; j < p.topk; ++j) {
        uint32_t e;
        const uint32_t best = best_left(key, row, p.per, e);
        if (best <= kMaskedKey) break;
        const float lead = key_logit(best);
        const uint64_t near = keys_from(key, best == kAll ? kAll : logit_key(lead - (2.0f * off + 0x1p-22f * fabsf(lead))));
        const uint32_t some = __ballot_sync(kAll, near != 0);
        const bool several = __any_sync(kAll, (near & (near - 1)) != 0);
        if (__popc(some) > 1 || several) e = __reduce_min_sync(kAll, expert64(p, row, near));
        set_key(key, row, p.per, e, 0u);
        if (lane == j) my_id = static_cast<int32_t>(e);
      }
      mine = my_id >= 0 ? load1(p.kind, p.logits, row.at + my_id) : -INFINITY;
    }
  }

  // ---- weights, lane j's for choice j
  float w = 0.0f;
  if (!p.normalize) {
    if (my_id >= 0) w = p.scale * (p.sigmoid ? sigmoid32(mine) : expf(mine - row.m) / total);
  } else {
    // scores over their sum, both over e^top where all logits are negative, so that
    // scores below the smallest number keep their ratios
    const float top = warp_max(mine);
    float s = 0.0f;
    if (my_id >= 0) {
      if (!p.sigmoid) s = expf(mine - top);
      else s = top >= 0.0f ? sigmoid32(mine) : expf(mine - top) / (1.0f + expf(mine));
    }
    const float sum = warp_sum(s);
    if (my_id >= 0) w = p.scale * (s / sum);
  }
  if (lane < p.topk) {
    p.ids[t * p.topk + lane] = my_id;
    p.weights[t * p.topk + lane] = w;
  }
}

struct RouterBwdParams {
  int64_t tokens, ld, m_pad;
  int L, topk, kind, sigmoid, normalize;
  float scale;
  const void* logits;
  const int32_t* ids;
  const float *weights, *dweights;
  const int32_t* row_of_slot;
  void* dlogits;
};

// One warp per token; lane j < topk has choice j.  Where only the chosen logits have a
// gradient (NI = 0) the row is filled with zeros and the lanes place theirs; softmax
// without renormalising reaches every logit (NI registers of them a lane).  16384 x 128
// float32, top-4: 8 us, bound by the latency of ids, logits and stores one after the other.
template <int NI>
__global__ void __launch_bounds__(32 * kRouterWarps) route_groups_backward_kernel(const __grid_constant__ RouterBwdParams p) {
  let_next_kernel_start();
  wait_for_previous_kernel();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouterWarps + (threadIdx.x >> 5);
  if (t >= p.tokens) return;
  const int64_t at = t * p.ld;
  int32_t id = -1;
  float w = 0.0f, g = 0.0f;
  if (lane < p.topk) {
    const int64_t s = t * p.topk + lane;
    id = p.ids[s];
    if (id >= p.L || id < 0) id = -1;
    if (id >= 0) {
      w = p.weights[s];
      if (p.row_of_slot != nullptr) {
        const int32_t r = p.row_of_slot[s];
        g = (r >= 0 && r < p.m_pad) ? p.dweights[r] : 0.0f;
      } else {
        g = p.dweights[s];
      }
    }
  }
  if constexpr (NI == 0) {
    // 1 - s = 1 / (1 + e^l), before the row is filled: dlogits may be the logits
    const float rest = p.sigmoid && id >= 0 ? sigmoid32(-load1(p.kind, p.logits, at + id)) : 1.0f;
    const float inner = p.normalize ? warp_sum(w * g) / p.scale : 0.0f;
    const float d = w * (g - inner) * rest;
    __syncwarp();
    for (int e = lane; e < p.L; e += 32) store1(p.kind, p.dlogits, at + e, 0.0f);
    __syncwarp();
    if (id >= 0) store1(p.kind, p.dlogits, at + id, d);
  } else {
    const float inner = warp_sum(w * g);
    float l[NI], mx = -INFINITY, total = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = lane + 32 * i;
      l[i] = e < p.L ? load1(p.kind, p.logits, at + e) : -INFINITY;
      mx = fmaxf(mx, l[i]);
    }
    mx = warp_max(mx);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      l[i] = l[i] == -INFINITY ? 0.0f : expf(l[i] - mx);
      total += l[i];
    }
    total = warp_sum(total);
    const float r = total > 0.0f ? 1.0f / total : total;    // a row of -inf: every score is 0 (NaN stays)
    float gi[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) gi[i] = 0.0f;
    for (int j = 0; j < p.topk; ++j) {
      const int32_t e = __shfl_sync(kAll, id, j) - lane;
      const float gj = p.scale * __shfl_sync(kAll, g, j);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (e == 32 * i) gi[i] = gj;
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int e = lane + 32 * i;
      if (e < p.L) store1(p.kind, p.dlogits, at + e, l[i] * r * (gi[i] - inner));
    }
  }
}

// ---------------------------------------------------------------- host
bsgg_status check_router(const bsgg_route_groups_desc* d, bool forward) {
  if (!d || d->tokens < 0 || d->tokens > (int64_t(1) << 30) || d->num_experts < 1 || d->num_experts > 1024)
    return BSGG_ERR_INVALID_ARG;
  if (d->topk < 1 || d->topk > 32 || d->topk > d->num_experts || d->ld < d->num_experts || d->ld > (int64_t(1) << 30))
    return BSGG_ERR_INVALID_ARG;
  if (!is_float_format(d->logit_format) || (d->normalize != 0 && d->normalize != 1) ||
      (d->score != BSGG_SCORE_SOFTMAX && d->score != BSGG_SCORE_SIGMOID) || !std::isfinite(d->scale) || !(d->scale > 0.0f))
    return BSGG_ERR_INVALID_ARG;
  if (!forward) return BSGG_OK;
  if (d->groups < 1 || d->groups > 32 || d->num_experts % d->groups != 0 || d->topk_groups < 1 || d->topk_groups > d->groups ||
      (d->group_top != 1 && d->group_top != 2) || d->topk > d->num_experts / d->groups * d->topk_groups)
    return BSGG_ERR_INVALID_ARG;
  return BSGG_OK;
}

// Calls f with the least power of two that holds n registers, as a constant.
template <typename F>
bsgg_status with_registers(int n, F&& f) {
  if (n <= 1) return f(std::integral_constant<int, 1>());
  if (n <= 2) return f(std::integral_constant<int, 2>());
  if (n <= 4) return f(std::integral_constant<int, 4>());
  if (n <= 8) return f(std::integral_constant<int, 8>());
  if (n <= 16) return f(std::integral_constant<int, 16>());
  if (n <= 32) return f(std::integral_constant<int, 32>());
  return f(std::integral_constant<int, 64>());
}

}  // namespace

extern "C" {

bsgg_status bsgg_route_groups(const bsgg_route_groups_desc* d, const void* logits, const float* bias, int32_t* ids,
                              float* weights, void* stream) {
  const bsgg_status st = check_router(d, true);
  if (st != BSGG_OK) return st;
  if (d->tokens == 0) return BSGG_OK;
  if (!logits || !ids || !weights || !aligned_to(logits, float_bytes(d->logit_format)) || !aligned_to(bias, 4) ||
      !aligned_to(ids, 4) || !aligned_to(weights, 4))
    return BSGG_ERR_INVALID_ARG;
  RouterParams p = {};
  p.tokens = d->tokens; p.ld = d->ld; p.L = d->num_experts; p.topk = d->topk; p.group_top = d->group_top;
  p.kind = d->logit_format; p.sigmoid = d->score == BSGG_SCORE_SIGMOID; p.normalize = d->normalize; p.scale = d->scale;
  p.logits = logits; p.bias = bias; p.ids = ids; p.weights = weights;
  // all groups stay: as good as one
  p.groups = d->topk_groups < d->groups ? d->groups : 1;
  p.topk_groups = d->topk_groups < d->groups ? d->topk_groups : 1;
  p.size = p.L / p.groups;
  p.per = 32;
  while (p.per * p.groups > 32) p.per /= 2;
  const LaunchConfig c(dim3(static_cast<unsigned>(ceil_div(d->tokens, kRouterWarps))), 32 * kRouterWarps, 0,
                       static_cast<cudaStream_t>(stream));
  return with_registers(static_cast<int>(ceil_div(p.size, p.per)),
                        [&](auto ni) { return launch_kernel(c, route_groups_kernel<decltype(ni)::value>, p); });
}

bsgg_status bsgg_route_groups_backward(const bsgg_route_groups_desc* d, const void* logits, const int32_t* ids,
                                       const float* weights, const float* dweights, const int32_t* row_of_slot,
                                       int64_t m_pad, void* dlogits, void* stream) {
  const bsgg_status st = check_router(d, false);
  if (st != BSGG_OK) return st;
  if (row_of_slot && (m_pad <= 0 || m_pad > (int64_t(1) << 30))) return BSGG_ERR_INVALID_ARG;
  if (d->tokens == 0) return BSGG_OK;
  const uintptr_t es = float_bytes(d->logit_format);
  if (!logits || !ids || !weights || !dweights || !dlogits || !aligned_to(logits, es) || !aligned_to(dlogits, es) ||
      !aligned_to(ids, 4) || !aligned_to(weights, 4) || !aligned_to(dweights, 4) || !aligned_to(row_of_slot, 4))
    return BSGG_ERR_INVALID_ARG;
  const RouterBwdParams p = {d->tokens, d->ld, m_pad, d->num_experts, d->topk, d->logit_format,
                             d->score == BSGG_SCORE_SIGMOID, d->normalize, d->scale, logits, ids, weights, dweights,
                             row_of_slot, dlogits};
  const LaunchConfig c(dim3(static_cast<unsigned>(ceil_div(d->tokens, kRouterWarps))), 32 * kRouterWarps, 0,
                       static_cast<cudaStream_t>(stream));
  if (p.sigmoid || p.normalize) return launch_kernel(c, route_groups_backward_kernel<0>, p);
  return with_registers(static_cast<int>(ceil_div(p.L, 32)), [&](auto ni) {
    constexpr int N = decltype(ni)::value;
    return launch_kernel(c, route_groups_backward_kernel<(N > 32 ? 32 : N)>, p);
  });
}

}  // extern "C"
