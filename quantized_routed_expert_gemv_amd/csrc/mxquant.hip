// Microscaled formats: rows of values <-> codes of 4 (E2M1) or 6 (E2M3) bits, each block of
// 32 sharing a power-of-two scale 2^(s - 127) held as its byte s.
//   s      = max(1, floor(log2 a) - 2 + 127), a the block's largest magnitude: both element
//            formats have 2 as their largest exponent, so a lands in [4, 8)
//   code   = the element format's value nearest to v * 2^(127 - s), halves to the even code,
//            saturated at 6 (E2M1) or 7.5 (E2M3)
// A block with an infinity or NaN has s = 255 and codes 0 and stands for NaNs: the products'
// matrix instruction turns that scale into NaN in the rows that it belongs to, and only there.
// Blocks lie flat in both planes (a row is a whole number of them), so rows do not matter.
// Copy rate bounds these kernels; see each for its split. Measured on 92160 x 2880 values,
// MXFP4 / MXFP6, in a kernel trace, three sets of inputs in turn: quantise from bf16 133 / 153 us
// (5.1 / 4.8 TB/s), from fp32 244 / 259 us (4.9); dequantise to bf16 149 / 147 us (4.5 / 5.0), to
// fp32 232 / 247 us (5.2 / 5.1).
#include <algorithm>

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

// A thread takes V values, a block's threads exchange their maxima. V is 8 for E2M1 (one
// 16-byte load of a 16-bit type, a dword of codes) and 16 for E2M3, whose 16 codes are three
// whole dwords.
template <int FMT, typename S, int V>
__global__ __launch_bounds__(kTh) void k_quantize(const void* __restrict__ src, int64_t n,
                                                  uint8_t* __restrict__ q,
                                                  uint8_t* __restrict__ s) {
  constexpr int kPer = 32 / V;   // threads a block
  const int64_t i = (int64_t)blockIdx.x * kTh + threadIdx.x;   // group of V values
  if (i >= n) return;   // n is a multiple of kPer: a block's threads go together
  float v[V];
#pragma unroll
  for (int h = 0; h < V / 8; ++h) Src<S>::load8(src, i * (V / 8) + h, v + 8 * h);
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) m = max_u(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
  for (int x = 1; x < kPer; x <<= 1) m = max_u(m, __shfl_xor(m, x, kWave));
  const uint32_t sb = scale_byte(m);
  const bool bad = sb == 255;
  if (i % kPer == 0) s[i / kPer] = (uint8_t)sb;
  if constexpr (FMT == kMxFp4) {
    static_assert(V == 8, "a dword of codes");
    const float sc = __uint_as_float(sb << 23);
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], sc, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], sc, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], sc, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], sc, 3);
    ((uint32_t*)q)[i] = bad ? 0u : c;
  } else {
    static_assert(V == 16, "three dwords of codes");
    const float inv = __uint_as_float((254u - (bad ? 127u : sb)) << 23);   // 2^(127 - s), exact
    uint32_t c[3] = {0, 0, 0};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t code = bad ? 0u : e2m3(v[j] * inv);
      c[6 * j / 32] |= code << (6 * j % 32);
      if (6 * j % 32 > 26) c[6 * j / 32 + 1] |= code >> (32 - 6 * j % 32);
    }
    uint32_t* o = (uint32_t*)(q + i * 12);
#pragma unroll
    for (int d = 0; d < 3; ++d) o[d] = c[d];
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

// V values a thread, 32 bytes stored: 16 of a 16-bit type (an 8- or 12-byte read of codes), 8
// of fp32 (wider strides between the lanes' stores cost a quarter of the rate). A value is
// code * 2^(s - 127), rounded to the output's type where it is too fine for it.
template <int FMT, typename D>
__global__ __launch_bounds__(kTh) void k_dequantize(const uint8_t* __restrict__ q,
                                                    const uint8_t* __restrict__ s, int64_t n,
                                                    void* __restrict__ dst) {
  constexpr int kBits = FMT == kMxFp4 ? 4 : 6, V = 32 / sizeof(D), kHalves = kBits * V / 16;
  const int64_t i = (int64_t)blockIdx.x * kTh + threadIdx.x;
  if (i >= n) return;
  const uint32_t sb = s[i / (32 / V)];
  // 2^(s - 127) in two factors, so that s = 0 needs no subnormal constant
  const float f0 = __uint_as_float((sb == 255 ? 255u : sb / 2 + 64) << 23);
  const float f1 = __uint_as_float((sb == 255 ? 127u : sb - sb / 2 + 63) << 23);
  uint32_t c[(kHalves + 1) / 2] = {};
  if constexpr (kHalves % 2 == 0) {
#pragma unroll
    for (int d = 0; d < kHalves / 2; ++d) c[d] = ((const uint32_t*)q)[i * (kHalves / 2) + d];
  } else {   // 6 bytes, 2-byte aligned
#pragma unroll
    for (int d = 0; d < kHalves; ++d)
      c[d / 2] |= (uint32_t)((const uint16_t*)q)[i * kHalves + d] << (16 * (d % 2));
  }
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = kBits * j;
    uint32_t code = c[at / 32] >> (at % 32);
    if (at % 32 > 32 - kBits) code |= c[at / 32 + 1] << (32 - at % 32);
    v[j] = code_value<kBits - 3>(code & ((1u << kBits) - 1)) * f0 * f1;
    if (sb == 255) v[j] = __builtin_nanf("");
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float* u = v + V / 2 * h;
    if constexpr (sizeof(D) == 4) {
      ((f32x4*)dst)[2 * i + h] = f32x4{u[0], u[1], u[2], u[3]};
    } else {
      typedef D d8 __attribute__((__vector_size__(16)));
      ((d8*)dst)[2 * i + h] = d8{(D)u[0], (D)u[1], (D)u[2], (D)u[3], (D)u[4], (D)u[5], (D)u[6], (D)u[7]};
    }
  }
}

template <int FMT>
hipError_t quantize_f(const void* src, int type, int64_t n, uint8_t* q, uint8_t* s,
                      hipStream_t st) {
  constexpr int V = FMT == kMxFp4 ? 8 : 16;
  n /= V;
  const dim3 grid((unsigned)((n + kTh - 1) / kTh));
  if (type == kBF16)
    hipLaunchKernelGGL((k_quantize<FMT, __bf16, V>), grid, dim3(kTh), 0, st, src, n, q, s);
  else if (type == kFP16)
    hipLaunchKernelGGL((k_quantize<FMT, _Float16, V>), grid, dim3(kTh), 0, st, src, n, q, s);
  else
    hipLaunchKernelGGL((k_quantize<FMT, float, V>), grid, dim3(kTh), 0, st, src, n, q, s);
  return hipGetLastError();
}

template <int FMT>
hipError_t dequantize_f(const uint8_t* q, const uint8_t* s, int64_t n, void* dst, int type,
                        hipStream_t st) {
  n /= type == kFP32 ? 8 : 16;
  const dim3 grid((unsigned)((n + kTh - 1) / kTh));
  if (type == kBF16)
    hipLaunchKernelGGL((k_dequantize<FMT, __bf16>), grid, dim3(kTh), 0, st, q, s, n, dst);
  else if (type == kFP16)
    hipLaunchKernelGGL((k_dequantize<FMT, _Float16>), grid, dim3(kTh), 0, st, q, s, n, dst);
  else
    hipLaunchKernelGGL((k_dequantize<FMT, float>), grid, dim3(kTh), 0, st, q, s, n, dst);
  return hipGetLastError();
}

// A launch holds fewer than 2^32 threads, of 8 values or 16: values go 2^34 at a time.
constexpr int64_t kMaxValues = int64_t(1) << 34;

}  // namespace

hipError_t launch_mx_quantize(const void* src, int type, int64_t n, int fmt, uint8_t* q,
                              uint8_t* s, hipStream_t st) {
  for (int64_t at = 0; at < n; at += kMaxValues) {
    const void* from = (const uint8_t*)src + at * (type == kFP32 ? 4 : 2);
    uint8_t* to = q + at / 32 * mx_block_bytes(fmt);
    const int64_t m = std::min(n - at, kMaxValues);   // HIP has its own min for int alone
    const hipError_t e = fmt == kMxFp4 ? quantize_f<kMxFp4>(from, type, m, to, s + at / 32, st)
                                       : quantize_f<kMxFp6>(from, type, m, to, s + at / 32, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_mx_dequantize(const uint8_t* q, const uint8_t* s, int64_t n, int fmt, void* dst,
                                int type, hipStream_t st) {
  for (int64_t at = 0; at < n; at += kMaxValues) {
    const uint8_t* from = q + at / 32 * mx_block_bytes(fmt);
    void* to = (uint8_t*)dst + at * (type == kFP32 ? 4 : 2);
    const int64_t m = std::min(n - at, kMaxValues);   // HIP has its own min for int alone
    const hipError_t e = fmt == kMxFp4 ? dequantize_f<kMxFp4>(from, s + at / 32, m, to, type, st)
                                       : dequantize_f<kMxFp6>(from, s + at / 32, m, to, type, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
