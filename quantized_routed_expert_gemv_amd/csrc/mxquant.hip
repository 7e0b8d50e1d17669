// Microscaled formats: rows of values <-> codes of 4 (E2M1) or 6 (E2M3) bits, each block of
// 32 sharing a power-of-two scale 2^(s - 127) held as its byte s.
//   s      = max(1, floor(log2 a) - 2 + 127), a the block's largest magnitude: both element
//            formats have 2 as their largest exponent, so a lands in [4, 8)
//   code   = the element format's value nearest to v * 2^(127 - s), halves to the even code,
//            saturated at 6 (E2M1) or 7.5 (E2M3)
// A block with an infinity or NaN has s = 255 and codes 0 and stands for NaNs: the products'
// matrix instruction turns that scale into NaN in the rows that it belongs to, and only there.
// Blocks lie flat in both planes (a row is a whole number of them), so rows do not matter.
// Copy rate bounds these kernels; see each for its split.
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

constexpr int kTh = 256;

// 8 consecutive values as fp32
template <typename S> struct Src;
template <> struct Src<float> {
  static __device__ __forceinline__ void load8(const void* p, int64_t i, float* v) {
    const f32x4 a = ((const f32x4*)p)[2 * i], b = ((const f32x4*)p)[2 * i + 1];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = a[q], v[4 + q] = b[q];
  }
};
template <> struct Src<__bf16> {
  static __device__ __forceinline__ void load8(const void* p, int64_t i, float* v) {
    const u32x4 a = ((const u32x4*)p)[i];
#pragma unroll
    for (int q = 0; q < 4; ++q) v[2 * q] = bf16_lo(a[q]), v[2 * q + 1] = bf16_hi(a[q]);
  }
};
template <> struct Src<_Float16> {
  static __device__ __forceinline__ void load8(const void* p, int64_t i, float* v) {
    const u32x4 a = ((const u32x4*)p)[i];
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[2 * q] = fp16_to_f32(a[q] & 0xFFFF), v[2 * q + 1] = fp16_to_f32(a[q] >> 16);
  }
};

__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The scale byte of a block whose largest magnitude has these fp32 bits (sign cleared).
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e == 255 ? 255u : e < 3 ? 1u : e - 2;
}

// E2M3 code of t, |t| < 8: magnitudes from 1 up are the fp32 bits rounded to three mantissa
// bits, below it whole eighths. Both tend to the even code on halves.
__device__ __forceinline__ uint32_t e2m3(float t) {
  const uint32_t u = __float_as_uint(t), a = u & 0x7FFFFFFFu;
  const uint32_t hi = ((a + 0x7FFFFu + ((a >> 20) & 1u)) >> 20) - (126u << 3);
  const uint32_t lo = (uint32_t)__float2int_rn(__uint_as_float(a) * 8.f);
  uint32_t c = a >= 0x3F800000u ? hi : lo;
  c = c > 31u ? 31u : c;
  return c | (u >> 31) << 5;
}

// 4 threads a block of 32, 8 values a thread: one 16-byte load of a 16-bit type (two of
// fp32) and the block's maximum by two lane exchanges.
template <int FMT, typename S>
__global__ __launch_bounds__(kTh) void k_quantize(const void* __restrict__ src, int64_t n8,
                                                  uint8_t* __restrict__ q,
                                                  uint8_t* __restrict__ s) {
  const int64_t i = (int64_t)blockIdx.x * kTh + threadIdx.x;   // group of 8 values
  if (i >= n8) return;   // n8 is a multiple of 4: a block's threads go together
  float v[8];
  Src<S>::load8(src, i, v);
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max_u(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  m = max_u(m, __shfl_xor(m, 1, kWave));
  m = max_u(m, __shfl_xor(m, 2, kWave));
  const uint32_t sb = scale_byte(m);
  const bool bad = sb == 255;
  if ((i & 3) == 0) s[i >> 2] = (uint8_t)sb;
  if constexpr (FMT == kMxFp4) {
    const float sc = __uint_as_float(sb << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], sc, 3);
    ((uint32_t*)q)[i] = bad ? 0u : c;
  } else {
    const float inv = __uint_as_float((254u - (bad ? 127u : sb)) << 23);   // 2^(127 - s), exact
    uint64_t c = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) c |= (uint64_t)e2m3(v[j] * inv) << (6 * j);
    if (bad) c = 0;
    uint16_t* o = (uint16_t*)(q + i * 6);
    o[0] = (uint16_t)c;
    o[1] = (uint16_t)(c >> 16);
    o[2] = (uint16_t)(c >> 32);
  }
}

// code -> value: with exponent field f and mantissa m of B bits, m / 2^B for f = 0, else
// (1 + m / 2^B) 2^(f - 1)
template <int B>
__device__ __forceinline__ float code_value(uint32_t c) {
  const uint32_t a = c & ((4u << B) - 1);
  const float lo = (float)a * (1.f / (1 << B));
  const float hi = __uint_as_float((126u << 23) + (a << (23 - B)));
  const float v = a < (1u << B) ? lo : hi;
  return (c >> (B + 2)) & 1u ? -v : v;
}

// 8 values a thread: one 4- (E2M1) or 6-byte read, one 16-byte store of a 16-bit type. A
// value is code * 2^(s - 127), rounded to the output's type where it is too fine for it.
template <int FMT, typename D>
__global__ __launch_bounds__(kTh) void k_dequantize(const uint8_t* __restrict__ q,
                                                    const uint8_t* __restrict__ s, int64_t n8,
                                                    void* __restrict__ dst) {
  const int64_t i = (int64_t)blockIdx.x * kTh + threadIdx.x;
  if (i >= n8) return;
  const uint32_t sb = s[i >> 2];
  // 2^(s - 127) in two factors, so that s = 0 needs no subnormal constant
  const float f0 = __uint_as_float((sb == 255 ? 255u : sb / 2 + 64) << 23);
  const float f1 = __uint_as_float((sb == 255 ? 127u : sb - sb / 2 + 63) << 23);
  float v[8];
  uint64_t c;
  if constexpr (FMT == kMxFp4) {
    c = ((const uint32_t*)q)[i];
  } else {
    const uint16_t* p = (const uint16_t*)(q + i * 6);
    c = p[0] | (uint64_t)p[1] << 16 | (uint64_t)p[2] << 32;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    constexpr int kBits = FMT == kMxFp4 ? 4 : 6;
    v[j] = code_value<kBits - 3>((uint32_t)(c >> (kBits * j)) & ((1u << kBits) - 1)) * f0 * f1;
    if (sb == 255) v[j] = __builtin_nanf("");
  }
  if constexpr (sizeof(D) == 4) {
    ((f32x4*)dst)[2 * i] = f32x4{v[0], v[1], v[2], v[3]};
    ((f32x4*)dst)[2 * i + 1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    typedef D d8 __attribute__((__vector_size__(16)));
    ((d8*)dst)[i] = d8{(D)v[0], (D)v[1], (D)v[2], (D)v[3], (D)v[4], (D)v[5], (D)v[6], (D)v[7]};
  }
}

template <int FMT>
hipError_t quantize_f(const void* src, int type, int64_t n8, uint8_t* q, uint8_t* s,
                      hipStream_t st) {
  const dim3 grid((unsigned)((n8 + kTh - 1) / kTh));
  if (type == kBF16) hipLaunchKernelGGL((k_quantize<FMT, __bf16>), grid, dim3(kTh), 0, st, src, n8, q, s);
  else if (type == kFP16) hipLaunchKernelGGL((k_quantize<FMT, _Float16>), grid, dim3(kTh), 0, st, src, n8, q, s);
  else hipLaunchKernelGGL((k_quantize<FMT, float>), grid, dim3(kTh), 0, st, src, n8, q, s);
  return hipGetLastError();
}

template <int FMT>
hipError_t dequantize_f(const uint8_t* q, const uint8_t* s, int64_t n8, void* dst, int type,
                        hipStream_t st) {
  const dim3 grid((unsigned)((n8 + kTh - 1) / kTh));
  if (type == kBF16) hipLaunchKernelGGL((k_dequantize<FMT, __bf16>), grid, dim3(kTh), 0, st, q, s, n8, dst);
  else if (type == kFP16) hipLaunchKernelGGL((k_dequantize<FMT, _Float16>), grid, dim3(kTh), 0, st, q, s, n8, dst);
  else hipLaunchKernelGGL((k_dequantize<FMT, float>), grid, dim3(kTh), 0, st, q, s, n8, dst);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void* src, int type, int64_t n, int fmt, uint8_t* q,
                              uint8_t* s, hipStream_t st) {
  return fmt == kMxFp4 ? quantize_f<kMxFp4>(src, type, n / 8, q, s, st)
                       : quantize_f<kMxFp6>(src, type, n / 8, q, s, st);
}

hipError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t n, int fmt, void* dst,
                                int type, hipStream_t st) {
  return fmt == kMxFp4 ? dequantize_f<kMxFp4>(q, s, n / 8, dst, type, st)
                       : dequantize_f<kMxFp6>(q, s, n / 8, dst, type, st);
}

}  // namespace moe
