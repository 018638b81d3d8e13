// bsgg_ops.cuh -- what the operators around the grouped GEMM share: formats,
// 8-value vector loads and stores, and the block quantizer.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bsgg.h"
#include "bsgg_kernel.cuh"

namespace bsgg {

// Programmatic dependent launch: every kernel of the operators is set up while the
// kernel before it on the stream still runs, waits here before it touches any
// memory that kernel may read or write, and lets the one after it be set up.  A
// chain of launches saves 1.2 us each.
__device__ __forceinline__ void wait_for_previous_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A launch's configuration: clusters of `cluster` blocks along x (1: none).
struct LaunchConfig {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  LaunchConfig(dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster = 1) {
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
  }
  LaunchConfig(const LaunchConfig&) = delete;
};
// Whether a call of the runtime succeeded.  The runtime keeps an error until it is
// read; one left there would be reported by the next launch that asks for it, as the
// grouped GEMM's do.
inline bool succeeded(cudaError_t e) {
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e == cudaSuccess;
}
template <typename... P, typename... A>
bsgg_status launch_kernel(const LaunchConfig& c, void (*kern)(P...), A... args) {
  return succeeded(cudaLaunchKernelEx(&c.cfg, kern, P(args)...)) ? BSGG_OK : BSGG_ERR_CUDA;
}

inline bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool is_float_format(int f) { return f == BSGG_OUT_BF16 || f == BSGG_OUT_F16 || f == BSGG_OUT_F32; }
inline int float_bytes(int f) { return f == BSGG_OUT_F32 ? 4 : 2; }

// One element of a bf16, f16 or f32 tensor (KIND: OK_BF16, OK_F16, OK_F32).
template <int KIND>
__device__ __forceinline__ float load1(const void* base, int64_t i) {
  if (KIND == OK_F32) return static_cast<const float*>(base)[i];
  if (KIND == OK_F16) return __half2float(static_cast<const __half*>(base)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i]);
}
__device__ __forceinline__ float load1(int kind, const void* base, int64_t i) {
  if (kind == OK_F32) return load1<OK_F32>(base, i);
  return kind == OK_F16 ? load1<OK_F16>(base, i) : load1<OK_BF16>(base, i);
}
template <int KIND>
__device__ __forceinline__ void store1(void* base, int64_t i, float v) {
  if (KIND == OK_F32) static_cast<float*>(base)[i] = v;
  else if (KIND == OK_F16) static_cast<__half*>(base)[i] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ void store1(int kind, void* base, int64_t i, float v) {
  if (kind == OK_F32) store1<OK_F32>(base, i, v);
  else if (kind == OK_F16) store1<OK_F16>(base, i, v);
  else store1<OK_BF16>(base, i, v);
}

template <int KIND>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if (KIND == OK_F16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
template <int KIND>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (KIND == OK_F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight consecutive values from element i (16-byte aligned pieces).
template <int KIND>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&v)[8]) {
  if constexpr (KIND == OK_F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = unpack2<KIND>(w[k]);
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
    }
  }
}
// Eight values in the registers of their stored form (zeros where absent).
// STREAM: they are read once and do not fit L2 anyway, so evict them first.
template <int KIND, bool STREAM>
struct Raw8 {
  uint4 q[KIND == OK_F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t i, bool present) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + i * (KIND == OK_F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (KIND == OK_F32 ? 2 : 1); ++k) q[k] = !present ? make_uint4(0, 0, 0, 0) : STREAM ? __ldcs(p + k) : p[k];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (KIND == OK_F32) {
      const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(w[k]);
    } else {
      const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = unpack2<KIND>(w[k]);
        v[2 * k] = f.x;
        v[2 * k + 1] = f.y;
      }
    }
  }
};
template <int KIND>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&v)[8]) {
  if constexpr (KIND == OK_F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + i) =
        make_uint4(pack2<KIND>(v[0], v[1]), pack2<KIND>(v[2], v[3]), pack2<KIND>(v[4], v[5]), pack2<KIND>(v[6], v[7]));
  }
}

// ---------------------------------------------------------------- quantizer
// Row formats by their bsgg_in_format: bits per value, values per scale.
__host__ __device__ constexpr bool rf_scaled(int f) { return f != BSGG_IN_BF16 && f != BSGG_ROW_F16; }
__host__ __device__ constexpr bool rf_fp4(int f) {
  return f == BSGG_IN_NVFP4 || f == BSGG_IN_FP4_UE8M0_16 || f == BSGG_IN_MXFP4;
}
__host__ __device__ constexpr int rf_vec(int f) { return f == BSGG_IN_NVFP4 || f == BSGG_IN_FP4_UE8M0_16 ? 16 : 32; }
__host__ __device__ constexpr int rf_bits(int f) { return !rf_scaled(f) ? 16 : rf_fp4(f) ? 4 : 8; }
// the code of scale 1
__host__ __device__ constexpr uint32_t rf_one(int f) { return f == BSGG_IN_NVFP4 ? 0x38u : 127u; }

// The scale code of a block whose largest magnitude has the bits `amax`.
// UE8M0: e = ceil(log2(amax / q_max)) read off the bits: q_max = m_q 2^p with
// m_q = 1.75 (E4M3, E5M2) or 1.5 (E2M1), so e is amax's exponent - p, and one
// more when its significand is above m_q.  No quotient is formed, so no rounding
// can move a block's exponent.
template <int FMT>
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  if (FMT == BSGG_IN_NVFP4) {
    if (amax >= 0x7F800000u) return 0x7Fu;
    const uint32_t c = cvt_e4m3x2(__fdiv_rn(__uint_as_float(amax), 6.0f), 0.0f) & 0xFFu;
    return c == 0u ? rf_one(FMT) : c;
  }
  if (amax >= 0x7F800000u) return 0xFFu;
  if (amax == 0u) return rf_one(FMT);
  constexpr int p = FMT == BSGG_IN_MXFP8_E4M3 ? 8 : FMT == BSGG_IN_MXFP8_E5M2 ? 15 : 2;
  constexpr uint32_t mq = rf_fp4(FMT) ? 0x400000u : 0x600000u;
  const int e = static_cast<int>(amax >> 23) - p + ((amax & 0x7FFFFFu) > mq ? 1 : 0);
  return static_cast<uint32_t>(e < 0 ? 0 : e);   // biased by 127; 2^-127 at the least
}

// Sixteen values over the scale of `code`, packed as the rows hold them: 4 words of
// FP8, 2 of FP4, 8 of 16-bit values (no scale).  UE8M0: times 2^-e, exact.  E4M3
// scales: the correctly rounded quotient, whose comparison with E2M1's thresholds is
// that of the exact one (a value off a tie differs from it by more than a rounding).
// A block with the NaN scale has zero codes.
__host__ __device__ constexpr int rf_words(int f) { return rf_bits(f) / 2; }
template <int FMT>
__device__ __forceinline__ void quantize16(const float (&v)[16], uint32_t code, uint32_t (&out)[rf_words(FMT)]) {
  if constexpr (!rf_scaled(FMT)) {
#pragma unroll
    for (int k = 0; k < 8; ++k) out[k] = pack2<FMT == BSGG_ROW_F16 ? OK_F16 : OK_BF16>(v[2 * k], v[2 * k + 1]);
  } else {
    float q[16];
    if (FMT == BSGG_IN_NVFP4) {
      const float s = e4m3_to_float(code);
#pragma unroll
      for (int k = 0; k < 16; ++k) q[k] = __fdiv_rn(v[k], s);
    } else {
      // 2^(127 - code): exponent field 254 - code, at code 254 the subnormal 2^-127
      const float r = code >= 254u ? __uint_as_float(0x400000u) : __uint_as_float((254u - code) << 23);
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        const float2 f = __fmul2_rn(make_float2(v[k], v[k + 1]), make_float2(r, r));
        q[k] = f.x;
        q[k + 1] = f.y;
      }
    }
    const bool nan_block = code == (FMT == BSGG_IN_NVFP4 ? 0x7Fu : 0xFFu);
#pragma unroll
    for (int k = 0; k < rf_words(FMT); ++k) {
      if (FMT == BSGG_IN_MXFP8_E4M3)
        out[k] = cvt_e4m3x2(q[4 * k], q[4 * k + 1]) | (cvt_e4m3x2(q[4 * k + 2], q[4 * k + 3]) << 16);
      else if (FMT == BSGG_IN_MXFP8_E5M2)
        out[k] = cvt_e5m2x2(q[4 * k], q[4 * k + 1]) | (cvt_e5m2x2(q[4 * k + 2], q[4 * k + 3]) << 16);
      else
        out[k] = cvt_e2m1x2(q[8 * k], q[8 * k + 1]) | (cvt_e2m1x2(q[8 * k + 2], q[8 * k + 3]) << 8) |
                 (cvt_e2m1x2(q[8 * k + 4], q[8 * k + 5]) << 16) | (cvt_e2m1x2(q[8 * k + 6], q[8 * k + 7]) << 24);
      if (nan_block) out[k] = 0u;
    }
  }
}

// Stores them; without scales the second eight only if `both`.
template <int FMT>
__device__ __forceinline__ void store_codes16(uint8_t* p, const uint32_t (&w)[rf_words(FMT)], bool both) {
  if constexpr (rf_fp4(FMT)) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    if constexpr (!rf_scaled(FMT)) {
      if (both) *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// The bits of the largest magnitude (a NaN's are above an infinity's).
__device__ __forceinline__ uint32_t max_abs_bits16(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 16; ++k) m = max(m, __float_as_uint(v[k]) & 0x7FFFFFFFu);
  return m;
}

}  // namespace bsgg
