// Expert products on microscaled rows: y[pos] = W[slot(e)] a[pos] for every bucket position
// pos of expert e, W in MXFP4 (the pool's tiled layout), a in MXFP4 or MXFP6:
//   y[n] = sum_b 2^(sw[n,b] - 127) 2^(sa[b] - 127) sum_{i < 32} w[n,b,i] a[b,i]
// which is one scaled matrix instruction's arithmetic: it takes both operands' codes and
// scale bytes as they lie in memory and accumulates in fp32, so nothing is widened. A lane
// holds one block of 32 of one row; the pool's unit order is that of a wave's lanes.
// E2M1 and E2M3 operands run at the same rate, twice E4M3's.
#include "common.hpp"
#include "kernels.hpp"

namespace moe {

namespace {

typedef int v8i __attribute__((__vector_size__(32)));

constexpr uint32_t kOne = 127;   // scale byte of 1.0

// A block's codes as a matrix operand; zeros where !ok (p is then any readable block).
template <int FMT>
__device__ __forceinline__ v8i load_block(const uint8_t* p, bool ok) {
  v8i v = {0, 0, 0, 0, 0, 0, 0, 0};
  if constexpr (FMT == kMxFp4) {
    const u32x4 a = *(const u32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = ok ? (int)a[i] : 0;
  } else {   // 24 bytes, 8-byte aligned
    const u32x2* s = (const u32x2*)p;
    const u32x2 a = s[0], b = s[1], c = s[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i] = ok ? (int)a[i] : 0;
      v[2 + i] = ok ? (int)b[i] : 0;
      v[4 + i] = ok ? (int)c[i] : 0;
    }
  }
  return v;
}

// Matrix-instruction format codes of the row operand.
template <int FMT> constexpr int kOperand = FMT == kMxFp4 ? 4 : 2;

// 16 weight rows x 128 K  times  128 K x 16 columns. Lane l holds block l / 16 of weight row
// and of column l % 16, and rows 4 (l / 16) .. + 3 of column l % 16 of the result.
template <int FMT>
__device__ __forceinline__ f32x4 mma16(v8i w, uint32_t ws, v8i a, uint32_t as, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, kOperand<FMT>, 0, (int)ws, 0,
                                                          (int)as);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});   // RNE, NaN kept
}

// First and last bucket position of expert e, inside [0, n_pairs] whatever offsets holds.
__device__ __forceinline__ void bucket_range(const int32_t* offsets, int e, int n_pairs, int* lo,
                                             int* hi) {
  *lo = min(max(offsets[e], 0), n_pairs);
  *hi = min(max(offsets[e + 1], *lo), n_pairs);
}

// The row that bucket position pos reads.
template <bool GATED>
__device__ __forceinline__ int source_row(const MxProduct& p, int pos) {
  if (!GATED) return pos;
  const int t = p.perm[pos] / p.k;
  return (unsigned)t < (unsigned)p.T ? t : 0;
}

constexpr int kGemvThreads = 256;

// Few rows: the weights' bytes bound it. One workgroup a 16-row group of one active expert;
// its 4 waves share the row group's blocks, 4 at a time (one coalesced KiB), and add their
// sums in LDS in wave order. Up to 16 rows of the expert ride along as the instruction's
// columns; more are taken 16 at a time.
template <int FMT, bool GATED>
__global__ __launch_bounds__(kGemvThreads) void k_mx_gemv(MxProduct p) {
  constexpr int NM = GATED ? 2 : 1;
  constexpr int kBytes = mx_block_bytes(FMT);
  __shared__ int cnt[kGemvThreads / kWave];
  __shared__ int found[3];
  __shared__ f32x4 red[3][NM][kWave];
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = threadIdx.x / kWave;
  const int n_pairs = p.T * p.k;
  // the blockIdx.y-th expert that has rows
  int lo = 0, hi = 0;
  if ((int)threadIdx.x < p.E) bucket_range(p.offsets, threadIdx.x, n_pairs, &lo, &hi);
  const uint64_t has = __ballot(hi > lo);
  if (lane == 0) cnt[wave] = __popcll(has);
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  int at = __popcll(has & ((1ull << lane) - 1));
  for (int w = 0; w < wave; ++w) at += cnt[w];
  if (hi > lo && at == (int)blockIdx.y) {
    found[0] = threadIdx.x;
    found[1] = lo;
    found[2] = hi;
  }
  __syncthreads();
  const int e = found[0];
  if (e < 0) return;
  lo = found[1];
  hi = found[2];
  const int n0 = blockIdx.x * kRowGroup;
  const int slot = p.slot_map[e];
  if (slot < 0 || slot >= p.n_slots) {
    for (int t = threadIdx.x; t < (hi - lo) * kRowGroup; t += kGemvThreads) {
      const int64_t o = (int64_t)(lo + t / kRowGroup) * p.N + n0 + t % kRowGroup;
      if (GATED) p.h[o] = 0;
      else p.y[o] = 0.f;
    }
    if (threadIdx.x == 0 && p.err && slot != kSlotMiss) atomicOr(p.err, 1u);
    return;
  }
  const int nb = p.K / kBlock;
  const int nsteps = (nb + 3) / 4;
  const uint8_t* wq[2] = {p.a.q + slot * p.a.q_slot, p.b.q + slot * p.b.q_slot};
  const uint8_t* ws[2] = {p.a.s + slot * p.a.s_slot, p.b.s + slot * p.b.s_slot};
  const int64_t u0 = (int64_t)blockIdx.x * nb * kRowGroup + (lane & 15);
  for (int m0 = lo; m0 < hi; m0 += 16) {
    const int pos = m0 + (lane & 15);
    const int64_t row = source_row<GATED>(p, min(pos, hi - 1));
    const uint8_t* aq = p.q + row * nb * kBytes;
    const uint8_t* as = p.s + row * nb;
    f32x4 acc[NM];
#pragma unroll
    for (int i = 0; i < NM; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int c = wave; c < nsteps; c += kGemvThreads / kWave) {
      const int b = 4 * c + (lane >> 4);
      const bool ok = b < nb;               // past the row: zero codes, scales of one
      const int bb = ok ? b : nb - 1;
      const v8i a = load_block<FMT>(aq + (int64_t)bb * kBytes, ok);
      const uint32_t sa = ok ? as[bb] : kOne;
      const int64_t u = u0 + (int64_t)bb * kRowGroup;
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        const v8i w = load_block<kMxFp4>(wq[i] + u * 16, ok);
        const uint32_t sw = ok ? ws[i][u] : kOne;
        acc[i] = mma16<FMT>(w, sw, a, sa, acc[i]);
      }
    }
    __syncthreads();   // the previous tile's sums have been read
    if (wave) {
#pragma unroll
      for (int i = 0; i < NM; ++i) red[wave - 1][i][lane] = acc[i];
    }
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int w = 0; w < 3; ++w)
#pragma unroll
        for (int i = 0; i < NM; ++i) acc[i] += red[w][i][lane];
      if (pos < hi) {
        const int64_t o = (int64_t)pos * p.N + n0 + 4 * (lane >> 4);
        if constexpr (GATED) {
          float v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = silu_mul(acc[0][q], acc[NM - 1][q]);
          *(u32x2*)(p.h + o) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
        } else {
          *(f32x4*)(p.y + o) = acc[0];
        }
      }
    }
  }
}

template <int FMT, bool GATED>
hipError_t launch_gemv_t(const MxProduct& p, hipStream_t st) {
  const dim3 grid(p.N / kRowGroup, min(p.E, p.T * p.k));
  hipLaunchKernelGGL((k_mx_gemv<FMT, GATED>), grid, dim3(kGemvThreads), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_product(const MxProduct& p, int fmt, bool gated, bool gemv, hipStream_t st) {
  (void)gemv;
  if (fmt == kMxFp4) return gated ? launch_gemv_t<kMxFp4, true>(p, st) : launch_gemv_t<kMxFp4, false>(p, st);
  return gated ? launch_gemv_t<kMxFp6, true>(p, st) : launch_gemv_t<kMxFp6, false>(p, st);
}

}  // namespace moe
