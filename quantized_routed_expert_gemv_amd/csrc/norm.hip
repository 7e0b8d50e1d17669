// The two ends of a block around the routed layer, on the residual stream r [T x H]:
//   entry  s = r + scale * delta;  r' = s;  x = s / sqrt(mean(s^2) + eps) * w
//   exit   c = sum_j w_j y[inv_perm[t*k + j]];  n = c, or c / sqrt(mean(c^2) + eps) * w_post;
//          s = r + scale * gate * n;  r' = s;  x = s / sqrt(mean(s^2) + eps) * w_next
// The arithmetic is fp32 throughout: r' and x are each rounded once, on their store, and x
// comes from the unrounded s, so the stream's storage type costs the norm nothing.
//
// About ten flops a value: copy rate bounds them (latency for a few rows), so a row is
// read once and held in registers between its sums and its stores, up to 16384 values; longer
// rows are recomputed from the inputs for each sum. r' may be r itself: a thread stores a
// value only after every read of it. Measured, in a kernel trace: entry, 16384 x 2880, all bf16:
// 75 us (5.0 TB/s, a copy's rate); exit, 8192 x 2048, k = 8, fp32 stream, post-norm, gate and
// next norm: 119 us (5.9 TB/s, reads for the most part; 130 us a call in a row of calls); one row
// of 2880: 3 us.
// A row's mean square is an fp32 number: past 3.4e38 in the sum x is 0.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

__device__ __forceinline__ f32x4 load4(const float* p) { return *(const f32x4*)p; }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
  const u32x2 v = *(const u32x2*)p;
  return f32x4{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])};
}
// a row of a parameter or stream of either type, by a flag that is uniform over the launch
__device__ __forceinline__ f32x4 load4(const void* p, bool f32, int64_t i) {
  return f32 ? load4((const float*)p + i) : load4((const uint16_t*)p + i);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});   // RNE, NaN kept
}
__device__ __forceinline__ void store4(float* p, f32x4 v) { *(f32x4*)p = v; }
__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  *(u32x2*)p = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// Sum over the workgroup of NW waves; every thread gets it. `red` is reused by each call.
template <int NW>
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
  for (int m = kWave / 2; m; m >>= 1) v += wave_xor(v, m);
  if constexpr (NW > 1) {
    __syncthreads();   // the previous sum has been read
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[w];
  }
  return v;
}

__device__ __forceinline__ float dot4(f32x4 v, float s) {
#pragma unroll
  for (int q = 0; q < 4; ++q) s = fmaf(v[q], v[q], s);
  return s;
}

// A row's choices: positions in y, -1 for one outside [0, T*k), which adds nothing.
struct Choices {
  int pos[kMaxK];
  float w[kMaxK];
};
__device__ __forceinline__ Choices read_choices(const BlockNorm& a, int64_t t) {
  Choices c;
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    const int64_t p = t * a.k + (j < a.k ? j : 0);
    const int q = a.inv_perm[p];
    c.pos[j] = (unsigned)q < (unsigned)(a.T * a.k) ? q : -1;
    c.w[j] = a.w[p];
  }
  return c;
}

// sum_{j < K} w_j y[pos_j][c..c+3] in increasing j. Every load is unconditional (a choice that
// adds nothing reads row 0 and is dropped), so all of a row's are in flight at once. y is read
// once where a row stays in registers: nontemporal.
template <int K, bool NT>
__device__ __forceinline__ f32x4 combine4(const BlockNorm& a, const Choices& ch, int c) {
  f32x4 v[K], acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const f32x4* p = (const f32x4*)(a.y + (int64_t)max(ch.pos[j], 0) * a.H + c);
    v[j] = NT ? __builtin_nontemporal_load(p) : *p;
  }
#pragma unroll
  for (int j = 0; j < K; ++j) {
    const bool in = ch.pos[j] >= 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = in ? fmaf(ch.w[j], v[j][q], acc[q]) : acc[q];
  }
  return acc;
}

// Calls f with k as a constant.
template <typename F>
__device__ __forceinline__ void with_k(int k, F f) {
  switch (k) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 5: f(std::integral_constant<int, 5>{}); break;
    case 6: f(std::integral_constant<int, 6>{}); break;
    case 7: f(std::integral_constant<int, 7>{}); break;
    default: f(std::integral_constant<int, 8>{});
  }
}

// One row a workgroup of TH threads, 4 neighbouring values a thread and chunk, NCH chunks.
template <int TH, int NCH, bool EXIT, typename R>
__global__ __launch_bounds__(TH) void k_block_norm(BlockNorm a) {
  constexpr int NW = TH / kWave;
  __shared__ float red[NW];
  const int64_t t = (int64_t)a.t0 + blockIdx.x;
  const R* rin = (const R*)a.resid + t * a.H;
  f32x4 s[NCH], v[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * TH + threadIdx.x) * 4;
    s[i] = v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (c < a.H) {
      s[i] = load4(rin + c);
      if (!EXIT && a.delta) v[i] = load4(a.delta, a.delta_f32, t * a.H + c);
    }
  }
  if constexpr (EXIT) {
    const Choices ch = read_choices(a, t);
    with_k(a.k, [&](auto k) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = (i * TH + threadIdx.x) * 4;
        if (c < a.H) v[i] = combine4<decltype(k)::value, true>(a, ch, c);
      }
    });
  }
  if (EXIT && a.post) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) ss = dot4(v[i], ss);
    const float rs = rsqrtf(group_sum<NW>(ss, red) / a.H + a.eps);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (i * TH + threadIdx.x) * 4;
      if (c < a.H) v[i] = v[i] * rs * load4(a.post, a.par_f32, c);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * TH + threadIdx.x) * 4;
    if (c < a.H) {
      if (EXIT && a.gate) v[i] *= load4(a.gate, a.par_f32, t * a.gate_stride + c);
#pragma unroll
      for (int q = 0; q < 4; ++q) s[i][q] = fmaf(a.scale, v[i][q], s[i][q]);
      if (a.resid_out) store4((R*)a.resid_out + t * a.H + c, s[i]);
      ss = dot4(s[i], ss);
    }
  }
  if (EXIT && !a.x) return;
  const float rs = rsqrtf(group_sum<NW>(ss, red) / a.H + a.eps);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (i * TH + threadIdx.x) * 4;
    if (c < a.H) store4(a.x + t * a.H + c, s[i] * rs * load4(a.weight, a.par_f32, c));
  }
}

// Rows of any length: each sum recomputes the row's values from the inputs, and r' is
// stored in the last pass. A thread adds its chunks' sums in 64 bits: their number grows with
// the row, and in 32 bits 2^20 squares of 25 came out 1.4% low.
template <bool EXIT, typename R>
__global__ __launch_bounds__(1024) void k_block_norm_long(BlockNorm a) {
  constexpr int TH = 1024, NW = TH / kWave;
  __shared__ float red[NW];
  const int64_t t = (int64_t)a.t0 + blockIdx.x;
  const uint32_t H = a.H;   // a column past the last, up to 2^31 + 4095, has to compare as such
  Choices ch;
  if constexpr (EXIT) ch = read_choices(a, t);
  auto combined = [&](int c) {
    f32x4 v;
    with_k(a.k, [&](auto k) { v = combine4<decltype(k)::value, false>(a, ch, c); });
    return v;
  };
  float rs_post = 1.f;
  if (EXIT && a.post) {
    double ss = 0.;
    for (uint32_t c = threadIdx.x * 4; c < H; c += TH * 4) ss += dot4(combined(c), 0.f);
    rs_post = rsqrtf(group_sum<NW>((float)ss, red) / a.H + a.eps);
  }
  auto value = [&](int c) {
    f32x4 s = load4((const R*)a.resid + t * a.H + c), v = {0.f, 0.f, 0.f, 0.f};
    if (EXIT) {
      v = combined(c);
      if (a.post) v = v * rs_post * load4(a.post, a.par_f32, c);
      if (a.gate) v *= load4(a.gate, a.par_f32, t * a.gate_stride + c);
    } else if (a.delta) {
      v = load4(a.delta, a.delta_f32, t * a.H + c);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] = fmaf(a.scale, v[q], s[q]);
    return s;
  };
  float rs = 1.f;
  if (a.x) {
    double ss = 0.;
    for (uint32_t c = threadIdx.x * 4; c < H; c += TH * 4) ss += dot4(value(c), 0.f);
    rs = rsqrtf(group_sum<NW>((float)ss, red) / a.H + a.eps);
  }
  for (uint32_t c = threadIdx.x * 4; c < H; c += TH * 4) {
    const f32x4 s = value(c);
    if (a.resid_out) store4((R*)a.resid_out + t * a.H + c, s);
    if (a.x) store4(a.x + t * a.H + c, s * rs * load4(a.weight, a.par_f32, c));
  }
}

// A launch holds fewer than 2^32 threads: rows go 2^21 at a time, of 1024 threads at most.
constexpr int kMaxRows = 1 << 21;

template <bool EXIT, typename R>
hipError_t launch_t(BlockNorm a, hipStream_t stream) {
  for (; a.t0 < a.T; a.t0 += kMaxRows) {
    const dim3 grid((unsigned)min(a.T - a.t0, kMaxRows));
#define MOE_NORM(TH, NCH)                                                                  \
  hipLaunchKernelGGL((k_block_norm<TH, NCH, EXIT, R>), grid, dim3(TH), 0, stream, a)
    if (a.H <= 256) MOE_NORM(64, 1);
    else if (a.H <= 512) MOE_NORM(64, 2);
    else if (a.H <= 1024) MOE_NORM(64, 4);
    else switch ((a.H - 1) / 1024 + 1) {   // chunks of 256 threads x 4 values
      case 2: MOE_NORM(256, 2); break;
      case 3: MOE_NORM(256, 3); break;
      case 4: MOE_NORM(256, 4); break;
      case 5: case 6: MOE_NORM(256, 6); break;
      case 7: case 8: MOE_NORM(256, 8); break;
      case 9: case 10: case 11: case 12: MOE_NORM(1024, 3); break;
      case 13: case 14: case 15: case 16: MOE_NORM(1024, 4); break;
      default: hipLaunchKernelGGL((k_block_norm_long<EXIT, R>), grid, dim3(1024), 0, stream, a);
    }
#undef MOE_NORM
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_block_norm(const BlockNorm& a, bool exit, bool resid_f32, hipStream_t stream) {
  if (exit) return resid_f32 ? launch_t<true, float>(a, stream) : launch_t<true, uint16_t>(a, stream);
  return resid_f32 ? launch_t<false, float>(a, stream) : launch_t<false, uint16_t>(a, stream);
}

}  // namespace moe
