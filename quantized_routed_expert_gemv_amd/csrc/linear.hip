// Dense products: out = resid + act(x w^T + bias), x [M][K], w [N][K], 16-bit operands, fp32 sums.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

typedef _Float16 f16x8 __attribute__((__vector_size__(8 * sizeof(_Float16))));

template <bool F16>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float load1(const void* p, int64_t i, int type) {
  if (type == kFP32) return ((const float*)p)[i];
  const uint16_t v = ((const uint16_t*)p)[i];
  return type == kFP16 ? fp16_to_f32(v) : bf16_to_f32(v);
}
__device__ __forceinline__ void store1(void* p, int64_t i, int type, float v) {
  if (type == kFP32) ((float*)p)[i] = v;
  else ((uint16_t*)p)[i] = type == kFP16 ? __builtin_bit_cast(uint16_t, (_Float16)v)
                                         : __builtin_bit_cast(uint16_t, (__bf16)v);
}

// act of the header's moe_act.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case 1: return v < 0.f ? 0.f : v;   // NaN stays NaN
    case 2: return 0.5f * v * erfcf(v * -0.70710678118654752440f);
    case 3: {   // 0.5 v (1 + tanh z) = v / (1 + e^{-2z})
      const float z = 0.79788456080286535588f * (v + 0.044715f * v * v * v);
      return v / (1.f + __expf(-2.f * z));
    }
    case 4: return v / (1.f + __expf(-v));
    default: return v;
  }
}

__device__ __forceinline__ void finish(const LinearCall& a, int64_t m, int64_t n, float v) {
  if (a.bias) v += load1(a.bias, n, a.bias_type);
  v = activate(v, a.act);
  if (a.resid) v += load1(a.resid, m * a.resid_stride + n, a.out_type);
  store1(a.out, m * a.out_stride + n, a.out_type, v);
}

// Few rows: one workgroup 16 rows of w; its four waves share K, 64 values at a time, and add
// their sums in LDS. Up to 16 MT rows of x ride along as the instruction's columns.
constexpr int kThreads = 256;
template <bool F16, int MT>
__global__ __launch_bounds__(kThreads) void k_linear_rows(LinearCall a) {
  constexpr int NW = kThreads / kWave;
  __shared__ f32x4 red[NW][MT][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int r = lane & 15, g = lane >> 4;
  const int64_t tile = a.tile0 + blockIdx.x, ntiles = ((int64_t)a.N + 15) / 16;
  const int64_t n0 = tile % ntiles * 16, m0 = tile / ntiles * (16 * MT);
  const uint16_t* w = a.w + min(n0 + r, (int64_t)a.N - 1) * a.w_stride;
  const uint16_t* x[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) x[i] = a.x + min(m0 + 16 * i + r, (int64_t)a.M - 1) * a.x_stride;
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
  for (int k0 = 64 * wave; k0 < a.K; k0 += 64 * NW) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = k0 + 32 * u + 8 * g;
      const bool in = k < a.K;
      const u32x4 zero = {0, 0, 0, 0};
      const u32x4 wf = in ? *(const u32x4*)(w + k) : zero;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x4 xf = in ? *(const u32x4*)(x[i] + k) : zero;
        acc[i] = mma16<F16>(wf, xf, acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  // lane: rows n0 + 4 g .. + 3 of w, row m0 + 16 i + r of x
  for (int i = wave; i < MT; i += NW) {
    f32x4 v = red[0][i][lane];
#pragma unroll
    for (int q = 1; q < NW; ++q) v += red[q][i][lane];
    const int64_t m = m0 + 16 * i + r;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (m < a.M && n0 + 4 * g + e < a.N) finish(a, m, n0 + 4 * g + e, v[e]);
  }
}

constexpr int64_t kMaxTiles = 1 << 22;   // a launch holds fewer than 2^32 threads

template <typename K>
hipError_t launch_tiles(LinearCall a, int64_t tiles, K kernel, hipStream_t stream) {
  for (int64_t t = 0; t < tiles; t += kMaxTiles) {
    a.tile0 = t;
    hipLaunchKernelGGL(kernel, dim3((unsigned)min(tiles - t, kMaxTiles)), dim3(kThreads), 0, stream,
                       a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool F16>
hipError_t launch_t(const LinearCall& a, hipStream_t stream) {
  const int64_t n = ((int64_t)a.N + 15) / 16;
  if (a.M <= 16) return launch_tiles(a, n, k_linear_rows<F16, 1>, stream);
  if (a.M <= 32) return launch_tiles(a, n, k_linear_rows<F16, 2>, stream);
  return launch_tiles(a, n * (((int64_t)a.M + 63) / 64), k_linear_rows<F16, 4>, stream);
}

}  // namespace

hipError_t launch_linear(const LinearCall& a, hipStream_t stream) {
  return a.type == kFP16 ? launch_t<true>(a, stream) : launch_t<false>(a, stream);
}

}  // namespace moe
