// Dense products: out = resid + act(x w^T + bias), x [M][K], w [N][K], 16-bit operands, fp32 sums.
// Few rows are bound by w's bytes, many by the matrix instructions. One kernel, whose tile, steps under
// way and groups follow the sizes (launch_t).
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

// Four neighbouring outputs of row m, n on: whole vectors where the caller's rows allow it.
__device__ __forceinline__ void finish4(const LinearCall& a, int64_t m, int64_t n, f32x4 v) {
  if (!a.vec4 || n + 4 > a.N) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N) finish(a, m, n + e, v[e]);
    return;
  }
  if (a.bias) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += load1(a.bias, n + e, a.bias_type);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = activate(v[e], a.act);
  if (a.resid) {
    const int64_t at = m * a.resid_stride + n;
    if (a.out_type == kFP32) {
      v += *(const f32x4*)((const float*)a.resid + at);
    } else {
      const u32x2 r = *(const u32x2*)((const uint16_t*)a.resid + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint16_t h = uint16_t(r[e / 2] >> 16 * (e & 1));
        v[e] += a.out_type == kFP16 ? fp16_to_f32(h) : bf16_to_f32(h);
      }
    }
  }
  const int64_t at = m * a.out_stride + n;
  if (a.out_type == kFP32) {
    *(f32x4*)((float*)a.out + at) = v;
  } else {
    u32x2 w;
    if (a.out_type == kFP16) {
      typedef _Float16 f16x2 __attribute__((__vector_size__(4)));
      w = u32x2{__builtin_bit_cast(uint32_t, f16x2{(_Float16)v[0], (_Float16)v[1]}),
                __builtin_bit_cast(uint32_t, f16x2{(_Float16)v[2], (_Float16)v[3]})};
    } else {
      w = u32x2{__builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[0], (__bf16)v[1]}),
                __builtin_bit_cast(uint32_t, bf16x2{(__bf16)v[2], (__bf16)v[3]})};
    }
    *(u32x2*)((uint16_t*)a.out + at) = w;
  }
}

// A wave's 16 TM x 16 TN outputs: 32 rows at a time through LDS of its own, so that rows leave in
// whole lines, and so that what is done to an output stands once in the code: unrolled over all
// products of a tile it came to more than the instruction cache holds, and took as long as the tile.
constexpr int kOutRows = 32;
template <int TN> constexpr int kOutStride = 16 * TN + 4;
template <int TM, int TN>
__device__ __forceinline__ void store_tile(const LinearCall& a, const f32x4 (&acc)[TN][TM], float* out,
                                           int64_t m0, int64_t n0) {
  constexpr int ST = kOutStride<TN>, JR = TM < 2 ? TM : kOutRows / 16, OR = 16 * JR;
  const int lane = threadIdx.x & (kWave - 1), r = lane & 15, g = lane >> 4;
#pragma unroll 1
  for (int c = 0; c < TM / JR; ++c) {
    if (m0 + OR * c >= a.M) return;
#pragma unroll
    for (int q = 0; q < TM / JR; ++q)
      if (q == c) {
#pragma unroll
        for (int j = 0; j < JR; ++j)
#pragma unroll
          for (int i = 0; i < TN; ++i)
            *(f32x4*)(out + (16 * j + r) * ST + 16 * i + 4 * g) = acc[i][JR * q + j];
      }
    __builtin_amdgcn_wave_barrier();
    constexpr int RL = kWave / (4 * TN);   // rows at once, of four values a lane
    const int row = lane / (4 * TN), col = lane % (4 * TN) * 4;
#pragma unroll 1
    for (int k = 0; k < OR; k += RL) {
      const int64_t m = m0 + OR * c + k + row;
      const f32x4 v = *(const f32x4*)(out + (k + row) * ST + col);
      if (m < a.M && n0 + col < a.N) finish4(a, m, n0 + col, v);
    }
    __builtin_amdgcn_wave_barrier();
  }
}

typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(1))) const void* global_ptr;

__device__ __align__(16) const uint32_t g_zero[4] = {0, 0, 0, 0};   // read in place of what is behind K

// The waves meet: their LDS accesses are done, and of their loads into LDS all but the newest N. A
// fence would wait for all of them.
template <int N>
__device__ __forceinline__ void meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// The workgroup's tile: an eighth of them to each XCD (workgroups go round the XCDs), and there 8
// tiles of rows of x side by side, column by column.
template <int BM, int BN>
__device__ __forceinline__ void find_tile(const LinearCall& a, int64_t* m0, int64_t* n0) {
  // M * N is below 2^40, and tiles of fewer than 64 x 64 are few: their number fits 32 bits
  const uint32_t tm = (uint32_t)(a.M + BM - 1) / BM, tn = (uint32_t)(a.N + BN - 1) / BN;
  uint32_t id = (uint32_t)a.tile0 + blockIdx.x;
  const uint32_t all = tm * tn, per = (all + 7) / 8, x = id % 8, full = all - 8 * (per - 1);
  id = id / 8 + (x < full ? x * per : full * per + (x - full) * (per - 1));
  const uint32_t band = id / (8 * tn), left = id - band * (8 * tn), high = min(tm - 8 * band, 8u);
  const uint32_t col = high == 8 ? left / 8 : left / high;
  *m0 = (int64_t)(8 * band + left - col * high) * BM;
  *n0 = (int64_t)col * BN;
}

// A workgroup of KG groups of WM x WN waves makes a tile of BM rows of x and BN of w; each group takes a
// part of K, BK values a step, and the groups' sums meet in LDS, in their order. Steps land in LDS straight
// from memory, S - 1 of them under way. A row's 16-byte pieces lie there in the order piece ^ row (BK
// 64) or piece ^ row / 2 (BK 32), so that eight neighbouring rows of a read fall on different banks
// (piece ^ row / 4 had 23 conflict cycles in 100).
// w is the matrix instruction's row operand, so that a lane's four sums are neighbours of one row of out.
// Measured: 4 x 5120 x 2880 8.4 us, 3.5 TB/s of w (a copy here: 4.85); 333 x 2880 x 4096 28 us, bound by
// the tiles' way from the L2s (290 MB); 16384 x 5120 x 2880 with bias and SiLU 508-534 us a call in a row of
// calls, 0.90-0.95 PFLOP/s, and 574-638 after idle time, the matrix pipes busy in 44 cycles of 100, at the
// clock that power leaves (without bias and SiLU 483-506; a library's product 325-415). Products with few
// tiles and a deep K leave most CUs idle, since K is shared inside a workgroup alone: 16 x 512 x 14336 in 32
// of them 19.7 us, where its bytes are 3.1; 1 x 64 x 14336 11.0 (a library's products 19 and 18).
template <bool F16, int BM, int BN, int BK, int WM, int WN, int S, int KG>
__global__ __launch_bounds__(WM * WN * KG * kWave) void k_linear_tile(LinearCall a) {
  constexpr int NW = WM * WN, PR = BK / 8;                 // waves of a group; pieces of a row
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;      // 16 x 16 products of a wave
  constexpr int RL = kWave / PR;                           // rows of a load
  constexpr int LM = BM / RL / NW, LN = BN / RL / NW;      // loads of a wave and step
  static_assert(BK == 64 || BK == 32, "swizzle");
  static_assert(LM * RL * NW == BM && LN * RL * NW == BN, "rows share out among the waves");
  constexpr int kStage = (BM + BN) * BK * 2;
  // the steps, then the other groups' sums, then outputs
  constexpr int kSums = (KG - 1) * NW * TM * TN * 1024, kOut = NW * kOutRows * kOutStride<TN> * 4;
  constexpr int kSteps = KG * S * kStage, kMost = kSums > kOut ? kSums : kOut;
  __shared__ __align__(16) uint8_t lds[kSteps > kMost ? kSteps : kMost];
  const int lane = threadIdx.x & (kWave - 1);
  const int all = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int group = all / NW, wave = all % NW;
  const int r = lane & 15, g = lane >> 4;
  int64_t m0, n0;
  find_tile<BM, BN>(a, &m0, &n0);

  // this wave's rows to load, RL at a time: the lane's row and piece
  auto swizzle = [](int row) { return BK == 64 ? row & 7 : row >> 1 & 3; };
  const int lrow = lane / PR, piece = (lane % PR) ^ swizzle(lrow);
  const int steps = ((a.K + BK - 1) / BK + KG - 1) / KG, k0 = group * steps * BK + 8 * piece;
  const uint16_t* src[LM + LN];
#pragma unroll
  for (int i = 0; i < LM + LN; ++i) {
    const int row = RL * ((i < LM ? i : i - LM) * NW + wave) + lrow;
    src[i] = (i < LM ? a.x + min(m0 + row, (int64_t)a.M - 1) * a.x_stride
                     : a.w + min(n0 + row, (int64_t)a.N - 1) * a.w_stride) + k0;
  }
  uint8_t* const mine = lds + group * S * kStage;
  auto load = [&](int c, int stage) {   // behind K: zeros
    const bool in = k0 + c * BK < a.K;
#pragma unroll
    for (int i = 0; i < LM + LN; ++i)
      __builtin_amdgcn_global_load_lds(
          in ? (global_ptr)(src[i] + (int64_t)c * BK) : (global_ptr)g_zero,
          (lds_ptr)(mine + stage * kStage + (i < LM ? 0 : BM * BK * 2) +
                    ((i < LM ? i : i - LM) * NW + wave) * 1024), 16, 0, 0);
  };
  f32x4 acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wm = wave / WN, wn = wave % WN;
  auto compute = [&](int stage) {
    const uint8_t* xs = mine + stage * kStage + wm * (BM / WM) * BK * 2;
    const uint8_t* ws = mine + stage * kStage + (BM + wn * (BN / WN)) * BK * 2;
#pragma unroll
    for (int k = 0; k < BK / 32; ++k) {
      const int at = r * BK * 2 + (((4 * k + g) ^ swizzle(r)) * 16);
      u32x4 xf[TM], wf[TN];
#pragma unroll
      for (int j = 0; j < TM; ++j) xf[j] = *(const u32x4*)(xs + j * 16 * BK * 2 + at);
#pragma unroll
      for (int i = 0; i < TN; ++i) wf[i] = *(const u32x4*)(ws + i * 16 * BK * 2 + at);
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = mma16<F16>(wf[i], xf[j], acc[i][j]);
    }
  };
#pragma unroll
  for (int c = 0; c < S - 1; ++c) load(c, c);
  int stage = 0, over = S - 1;   // of step c, and of step c - 1
  for (int c = 0; c < steps; ++c) {
    meet<(S - 2) * (LM + LN)>();   // step c is there; the loads of the S - 2 steps behind it may not be
    load(c + S - 1, over);
    compute(stage);
    over = stage;
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  meet<0>();   // the operands' places are free
  if constexpr (KG > 1) {
    f32x4* sums = (f32x4*)lds + wave * TM * TN * kWave + lane;
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) sums[((group - 1) * NW * TM * TN + i * TM + j) * kWave] = acc[i][j];
    }
    meet<0>();
    if (group > 0) return;
#pragma unroll
    for (int q = 0; q < KG - 1; ++q)
#pragma unroll
      for (int i = 0; i < TN; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] += sums[(q * NW * TM * TN + i * TM + j) * kWave];
    // a wave's outputs go where another's sums may still be read: not before it has them
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
  }
  store_tile<TM, TN>(a, acc, (float*)lds + wave * kOutRows * kOutStride<TN>, m0 + wm * (BM / WM),
                     n0 + wn * (BN / WN));
}

constexpr int64_t kMaxTiles = 1 << 22;   // a launch holds fewer than 2^32 threads

template <typename K>
hipError_t launch_tiles(LinearCall a, int64_t tiles, K kernel, int threads,
                        hipStream_t stream) {
  for (int64_t t = 0; t < tiles; t += kMaxTiles) {
    a.tile0 = t;
    hipLaunchKernelGGL(kernel, dim3((unsigned)min(tiles - t, kMaxTiles)), dim3(threads), 0, stream,
                       a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

int64_t tiles_of(const LinearCall& a, int bm, int bn) {
  return (((int64_t)a.M + bm - 1) / bm) * (((int64_t)a.N + bn - 1) / bn);
}

template <bool F16, int BM, int BN, int BK, int WM, int WN, int S, int KG>
hipError_t launch_tile(const LinearCall& a, hipStream_t stream) {
  return launch_tiles(a, tiles_of(a, BM, BN), k_linear_tile<F16, BM, BN, BK, WM, WN, S, KG>,
                      WM * WN * KG * kWave, stream);
}

// The tile, by how many there are of it. Up to 256: the smallest of which every CU has one at most, with
// as many groups and steps under way as LDS holds, for such products are bound by the bytes' way to the
// CUs (16 x 5120 x 2880, us: 16 x 32 tiles 7.3, 32 x 32 8.0, 64 x 32 10.9, 64 x 64 13.5; 64 rows: 32 x 32
// 14.0, 64 x 32 11.6, 64 x 64 14.8). Then 64 x 64 in two groups, two workgroups a CU (333 x 2880 x 4096:
// 26.7 against 29.4 for three of one group; 512 x 5120 x 2880: 40.7 against 31.8), in one group, 128 x 128
// (2048 x 5120 x 2880: 83 against 100, and 87 for 128 x 256), and 128 x 256 once they fill one and a half
// rounds of two a CU (16384 x 5120 x 2880: 526 against 581; 256 x 256, one a CU: 554).
template <bool F16>
hipError_t launch_t(LinearCall a, hipStream_t stream) {
  const int bytes = a.out_type == kFP32 ? 4 : 2;
  a.vec4 = ((uintptr_t)a.out & (4 * bytes - 1)) == 0 && a.out_stride % 4 == 0 &&
           (!a.resid || (((uintptr_t)a.resid & (4 * bytes - 1)) == 0 && a.resid_stride % 4 == 0));
  auto one_each = [&](int bm, int bn) { return tiles_of(a, bm, bn) <= 256; };
  if (one_each(16, 16)) return launch_tile<F16, 16, 16, 64, 1, 1, 4, 8>(a, stream);
  if (one_each(16, 32)) return launch_tile<F16, 16, 32, 64, 1, 2, 4, 4>(a, stream);
  if (a.M <= 16) return launch_tile<F16, 16, 64, 64, 1, 2, 4, 4>(a, stream);
  if (one_each(32, 32)) return launch_tile<F16, 32, 32, 64, 2, 2, 4, 4>(a, stream);
  if (one_each(64, 32)) return launch_tile<F16, 64, 32, 64, 2, 2, 4, 2>(a, stream);
  if (one_each(64, 64)) return launch_tile<F16, 64, 64, 64, 2, 2, 4, 2>(a, stream);
  if (tiles_of(a, 64, 64) <= 400) return launch_tile<F16, 64, 64, 64, 2, 2, 2, 2>(a, stream);
  if (tiles_of(a, 128, 128) < 300) return launch_tile<F16, 64, 64, 64, 2, 2, 3, 1>(a, stream);
  if (tiles_of(a, 128, 256) < 768) return launch_tile<F16, 128, 128, 64, 2, 2, 2, 1>(a, stream);
  return launch_tile<F16, 128, 256, 32, 2, 4, 3, 1>(a, stream);
}

}  // namespace

hipError_t launch_linear(const LinearCall& a, hipStream_t stream) {
  return a.type == kFP16 ? launch_t<true>(a, stream) : launch_t<false>(a, stream);
}

}  // namespace moe
