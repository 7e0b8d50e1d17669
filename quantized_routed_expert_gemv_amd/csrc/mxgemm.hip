// Expert products on microscaled rows: y[pos] = W[slot(e)] a[pos] for every bucket position
// pos of expert e, W in MXFP4 (the pool's tiled layout), a in MXFP4 or MXFP6:
//   y[n] = sum_b 2^(sw[n,b] - 127) 2^(sa[b] - 127) sum_{i < 32} w[n,b,i] a[b,i]
// which is one scaled matrix instruction's arithmetic: it takes both operands' codes and
// scale bytes as they lie in memory and accumulates in fp32, so nothing is widened. A lane
// holds one block of 32 of one row; the pool's unit order is that of a wave's lanes.
// E2M1 and E2M3 row operands run at the same rate (6.4 PFLOP/s measured with random operands)
// and their sums are exact in fp32; E4M3 ones at 4.4, with partial sums held shorter.
#include <type_traits>

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
// columns; more are taken 16 at a time. Measured, in rows of calls: gate/up of one token, H = I =
// 2880, 4 experts: 8.7 us for 35 MB (4.0 TB/s; 9.3 us in a kernel trace); down of four tokens, H
// 4096, I 14336: 33 us for about 5 experts' 156 MB.
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
    // 64 bits: an expert of 2^27 rows has 2^31 values here
    for (int64_t t = threadIdx.x; t < (int64_t)(hi - lo) * kRowGroup; t += kGemvThreads) {
      const int64_t o = (lo + t / kRowGroup) * p.N + n0 + t % kRowGroup;
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

constexpr int kStepBlocks = 8;    // blocks of K a step: four matrix instructions deep
constexpr int kSlices = kStepBlocks / 2;
constexpr int kSuperRows = 16, kSuperCols = 4;   // tiles of a run, by rows and columns
constexpr int kScaleBlocks = 128;              // blocks of K whose row scales lie in LDS at once
constexpr int kScaleRow = kScaleBlocks + 8;    // bytes between rows: 34 dwords, bank by bank

typedef float v16f __attribute__((__vector_size__(64)));

// 32 weight rows x 64 K  times  64 K x 32 columns. Lane l holds block l / 32 of weight row and
// of column l % 32; element v of the result is row 8 (v / 4) + 4 (l / 32) + v % 4 of column
// l % 32. AB: byte of `as` that holds the column's scale.
template <int FMT, int AB>
__device__ __forceinline__ v16f mma32(v8i w, uint32_t ws, v8i a, uint32_t as, v16f c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, a, c, 4, kOperand<FMT>, 0, (int)ws, AB,
                                                         (int)as);
}

// A step's rows in LDS: the first 16 bytes of each block, row by row, then (MXFP6) the last 8
// of each. Block b of tile row r lies in place b ^ (r / 2 % 8) of the row's eight, and in the
// second part b ^ (r / 4 % 8), to spread the lanes of each pass of a 64-lane read (one block of
// 32 rows and the next of the same) over the banks: 128-byte rows repeat their banks every 2
// rows, 64-byte rows every 4. In the whole kernel, conflicts take 13% of LDS's busy cycles on
// MXFP4 rows and 33% on MXFP6 rows (H 4096, I 14336, gate/up). Read whole, MXFP6's 24-byte blocks would take three
// 8-byte reads, at half the rate of 16-byte ones. Rows 32 apart lie at one distance.
__device__ __forceinline__ int lds_place(int r, int b) {
  return (r * kStepBlocks + (b ^ ((r >> 1) & 7))) * 16;
}
__device__ __forceinline__ int lds_place_tail(int r, int b) {
  return (r * kStepBlocks + (b ^ ((r >> 2) & 7))) * 8;
}

// A block's codes as they travel from memory to LDS.
template <int FMT> struct Codes {
  u32x4 v;
  u32x2 t;   // MXFP6
  __device__ __forceinline__ void load(const uint8_t* p) {
    typedef u32x4 __attribute__((aligned(8))) u32x4_8;   // MXFP6 blocks: every 24 bytes
    if constexpr (FMT == kMxFp4) {
      v = *(const u32x4*)p;
    } else {
      v = *(const u32x4_8*)p;
      t = *(const u32x2*)(p + 16);
    }
  }
  __device__ __forceinline__ void store(uint8_t* p, uint8_t* tail, bool ok) const {   // or zeros
    *(u32x4*)p = ok ? v : u32x4{0, 0, 0, 0};
    if constexpr (FMT == kMxFp6) *(u32x2*)tail = ok ? t : u32x2{0, 0};
  }
};

// Orders the LDS accesses of a wave's lanes against each other (the wave runs them in order).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The expert and first bucket position of row tile mt (tiles of bm rows, expert by expert);
// false past the last one.
__device__ bool find_tile(const MxProduct& p, int bm, int mt, int* e, int* m0, int* mend,
                          int* part, int* found) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  int lo = 0, hi = 0;
  if ((int)threadIdx.x < p.E) bucket_range(p.offsets, threadIdx.x, p.T * p.k, &lo, &hi);
  const int nt = (hi - lo + bm - 1) / bm;
  int end = nt;   // inclusive scan of nt
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) {
    const int o = __shfl_up(end, m, kWave);
    if (lane >= m) end += o;
  }
  if (lane == kWave - 1) part[wave] = end;
  if (threadIdx.x == 0) found[0] = -1;
  __syncthreads();
  for (int w = 0; w < wave; ++w) end += part[w];
  if (mt < end && mt >= end - nt) {
    found[0] = threadIdx.x;
    found[1] = lo + (mt - (end - nt)) * bm;
    found[2] = hi;
  }
  __syncthreads();
  *e = found[0];
  *m0 = found[1];
  *mend = found[2];
  return *e >= 0;
}

// Many rows: tiles of 32 MF bucket rows x 64 NW weight rows; NW waves, each all rows by 64
// weight rows (gated: 32 gate and the same 32 up, so SwiGLU stays in registers). Weight blocks
// go from the pool straight to the registers of the one wave that uses them (the pool's unit
// order is the operand's); the gathered rows are shared by the waves and pass through
// registers to one of two LDS buffers. Both are loaded one step of 256 K ahead: a row's 128
// bytes of MXFP4 codes are then one whole cache line, where half steps asked L2 for every
// line twice. Row scales, one byte a block, come 128 blocks at a time for the same reason.
// Measured, 16384 tokens, H = I = 2880, 4 of 32 experts, skewed, in rows of calls: gate/up MXFP4
// 0.70 ms (3.1 PFLOP/s), MXFP6 0.84 ms; down 0.43 and 0.48 ms. Over a longer K a tile gains 4.0
// (MXFP4) and 3.3 PFLOP/s; what it costs before its first and after its last step is the rest,
// 70 us over 32768 x 4096 fp32 outputs. The matrix pipes are busy 48-51% (MXFP6 37-39%) of the
// cycles over K = 16384 and 41-44% (33-35%) of gate/up's over 2880, at a clock that the chip's
// power takes from 2.4 down to 1.4-2.0 GHz; with the loads left out an earlier form reached 5.3
// PFLOP/s, so the operands' way into registers costs as much as the clock.
template <int FMT, bool GATED, int MF, int NW>
__global__ __launch_bounds__(kWave * NW, MF == 4 ? 2 : MF == 2 ? 3 : 4) void k_mx_gemm(
    MxProduct p, int n_mtiles, int n_ntiles, int first) {
  constexpr int kThreads = kWave * NW, kCols = 64 * NW;   // weight rows a tile
  constexpr int BM = 32 * MF;
  constexpr int TN = GATED ? kCols / 2 : kCols;   // output columns a tile
  constexpr int kBytes = mx_block_bytes(FMT);
  constexpr int NB = BM * kStepBlocks / kThreads;   // row blocks a thread loads a step
  static_assert(NB >= 1, "a thread loads whole blocks");
  // two buffers of rows; the epilogue's fragments take their place
  constexpr int kBuf = BM * kStepBlocks * kBytes;
  constexpr int kPiece = GATED ? 2 : 4;                    // bytes of an output
  constexpr int kOutRow = 32 * kPiece + 16;                // padded against bank conflicts
  constexpr int kTurn = kThreads / kWave * 32 * kOutRow;
  __shared__ __attribute__((aligned(16))) uint8_t lds_q[2 * kBuf > kTurn ? 2 * kBuf : kTurn];
  __shared__ __attribute__((aligned(16))) uint8_t lds_s[BM * kScaleRow];
  __shared__ int part[kThreads / kWave];
  __shared__ int found[3];
  // XCD-aware tile order: workgroups go to the 8 XCDs in turn, and each XCD gets runs of 64
  // tiles that share their rows and weights in its L2; first: 512s of tiles of earlier launches
  const int xcd = blockIdx.x & 7, local = blockIdx.x >> 3;
  const int64_t i = (int64_t)(first + (local >> 6)) * 512 + xcd * 64 + (local & 63);
  if (i >= (int64_t)n_mtiles * n_ntiles) return;
  const int sr = (int)(i / ((int64_t)kSuperRows * n_ntiles));
  const int sh = min(kSuperRows, n_mtiles - kSuperRows * sr);
  const int sj = (int)(i - (int64_t)kSuperRows * n_ntiles * sr);
  const int sc = sj / (kSuperCols * sh);
  const int sw = min(kSuperCols, n_ntiles - kSuperCols * sc);
  const int sk = sj - kSuperCols * sh * sc;
  const int mt = kSuperRows * sr + sk / sw, nt = kSuperCols * sc + sk % sw;
  int e, m0, mend;
  if (!find_tile(p, BM, mt, &e, &m0, &mend, part, found)) return;
  const int n0 = nt * TN;
  const int slot = p.slot_map[e];
  if (slot < 0 || slot >= p.n_slots) {
    for (int t = threadIdx.x; t < BM * TN; t += kThreads) {
      const int pos = m0 + t / TN, n = n0 + t % TN;
      if (pos < mend && n < p.N) {
        if (GATED) p.h[(int64_t)pos * p.N + n] = 0;
        else p.y[(int64_t)pos * p.N + n] = 0.f;
      }
    }
    if (threadIdx.x == 0 && p.err && slot != kSlotMiss) atomicOr(p.err, 1u);
    return;
  }
  const int nb = p.K / kBlock;
  const int nsteps = (nb + kStepBlocks - 1) / kStepBlocks;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int half = lane >> 5;

  // ---- rows: thread t carries block t % 8 of tile rows t / 8 + kThreads / 8 j
  const int rb = threadIdx.x & (kStepBlocks - 1);
  const uint8_t* rq[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int r = threadIdx.x / kStepBlocks + kThreads / kStepBlocks * j;
    const int64_t row = source_row<GATED>(p, min(m0 + r, mend - 1));   // past the end: the last
    rq[j] = p.q + row * nb * kBytes;
  }
  // ---- weights: fragment f is 32 rows from col[f] on; lane l holds row l % 32
  int col[2];
  const uint8_t* wq[2];
  const uint8_t* ws[2];
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    col[f] = GATED ? n0 + 32 * wave : n0 + 64 * wave + 32 * f;
    const int c0 = col[f] < p.N ? col[f] : 0;   // never stored past N
    const PoolView& m = GATED && f ? p.b : p.a;
    const int64_t u = pool_unit(c0, 0, nb);
    wq[f] = m.q + slot * m.q_slot + u * 16;
    ws[f] = m.s + slot * m.s_slot + u;
  }
  const uint32_t wlane = (uint32_t)((lane & 31) >> 4) * nb * kRowGroup + (lane & 15);   // unit
  // Loads: nothing here may wait for them. A block past the row reads the row's last; its
  // codes are replaced by zeros when they are put in LDS, which is enough on one side.
  constexpr int kRows32 = 32 * kStepBlocks;      // blocks from one row to that 32 further on
  constexpr int kTail = BM * kStepBlocks * 16;   // MXFP6: where a buffer's second part begins
  const int place = lds_place(threadIdx.x / kStepBlocks, rb);
  const int place_tail = kTail + lds_place_tail(threadIdx.x / kStepBlocks, rb);
  Codes<FMT> rows[NB];
  auto load_rows = [&](int c) {
    const int b = min(kStepBlocks * c + rb, nb - 1);
#pragma unroll
    for (int j = 0; j < NB; ++j) rows[j].load(rq[j] + (uint32_t)b * kBytes);
  };
  auto put = [&](int c) {
    uint8_t* to = lds_q + (c & 1) * kBuf;
    auto all = [&](bool ok) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
        rows[j].store(to + place + j * kThreads * 16, to + place_tail + j * kThreads * 8, ok);
    };
    if (kStepBlocks * (c + 1) <= nb) all(true);   // only a row's last step can be short
    else all(kStepBlocks * c + rb < nb);
  };
  u32x4 wgt[2][kSlices];
  uint32_t wsc[2][kSlices];
  auto load_weights = [&](int c, int s) {
    const uint32_t u = wlane + (uint32_t)min(kStepBlocks * c + 2 * s + half, nb - 1) * kRowGroup;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      wgt[f][s] = *(const u32x4*)(wq[f] + u * 16);
      wsc[f][s] = *(const uint32_t*)(ws[f] + (u & ~3u));   // the scales of 4 rows
    }
  };
  // Row scales of blocks b0 .. b0 + kScaleBlocks - 1, and ones past the row: a thread takes
  // every kParts-th 8 blocks of its row and stores the even ones' bytes, then the odd ones',
  // so that a lane's four of a step are one dword. The rows lie at any byte, so a row's last
  // dwords are gathered byte by byte.
  auto load_scales = [&](int b0) {
    constexpr int kParts = kThreads / BM;
    const int r = threadIdx.x / kParts;
    const uint8_t* src = p.s + (int64_t)source_row<GATED>(p, min(m0 + r, mend - 1)) * nb + b0;
    const int n = min(nb - b0, kScaleBlocks);
    u32x2* dst = (u32x2*)(lds_s + r * kScaleRow);
#pragma unroll 4
    for (int d = threadIdx.x % kParts; d < kScaleBlocks / 8; d += kParts) {
      uint32_t v[2] = {kOne * 0x01010101u, kOne * 0x01010101u};
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const int at = 8 * d + 4 * w;
        if (at + 4 <= n) {
          __builtin_memcpy(&v[w], src + at, 4);
        } else {
          for (int i = 0; at + i < n; ++i)
            v[w] = (v[w] & ~(0xFFu << (8 * i))) | (uint32_t)src[at + i] << (8 * i);
        }
      }
      dst[d] = u32x2{__builtin_amdgcn_perm(v[1], v[0], 0x06040200u),
                     __builtin_amdgcn_perm(v[1], v[0], 0x07050301u)};
    }
  };
  // where the lane reads block `half` of the first 32 rows; block 2 s + half lies at an
  // exclusive or of that
  const int from = lds_place(lane & 31, half);
  const int from_tail = lds_place_tail(lane & 31, half);
  auto read_block = [&](int buf, int s, int m) {
    const u32x4 v = *(const u32x4*)(lds_q + buf + (from ^ (2 * s * 16)) + m * kRows32 * 16);
    v8i a = {(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
    if constexpr (FMT == kMxFp6) {
      const u32x2 t =
          *(const u32x2*)(lds_q + buf + kTail + (from_tail ^ (2 * s * 8)) + m * kRows32 * 8);
      a[4] = (int)t[0];
      a[5] = (int)t[1];
    }
    return a;
  };
  v16f acc[MF][2];
#pragma unroll
  for (int m = 0; m < MF; ++m)
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[m][f][v] = 0.f;
  load_rows(0);
#pragma unroll
  for (int s = 0; s < kSlices; ++s) load_weights(0, s);
  put(0);
  // put(0) is seen behind the barrier that the first scales bring
  uint32_t as[MF];
  auto read_scales = [&](int c) {   // those of 128 blocks on are loaded where their first is due
    const int sb = kStepBlocks * c % kScaleBlocks;
    if (sb == 0) {
      int b0 = kStepBlocks * c;
      asm volatile("" : "+s"(b0));   // no addresses kept and stepped along for this
      load_scales(b0);
      __syncthreads();
    }
#pragma unroll
    for (int m = 0; m < MF; ++m)
      as[m] = *(const uint32_t*)(lds_s + (32 * m + (lane & 31)) * kScaleRow + sb + 4 * half);
  };
  auto products = [&](int c, auto sl) {   // of one slice, a pair of blocks
    constexpr int s = decltype(sl)::value;
    uint32_t wscale[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      asm volatile("" : "+v"(wsc[f][s]));   // waited for here, not where the step begins
      wscale[f] = wsc[f][s] >> (8 * (lane & 3));
    }
#pragma unroll
    for (int m = 0; m < MF; ++m) {
      const v8i a = read_block((c & 1) * kBuf, s, m);
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        const v8i w = {(int)wgt[f][s][0], (int)wgt[f][s][1], (int)wgt[f][s][2],
                       (int)wgt[f][s][3], 0, 0, 0, 0};
        acc[m][f] = mma32<FMT, s>(w, wscale[f], a, as[m], acc[m][f]);
      }
    }
    // the products stay in their slice, and one slice's operands at a time in registers:
    // without this the compiler reads every slice's first and spills
#pragma unroll
    for (int m = 0; m < MF; ++m) asm volatile("" : "+v"(acc[m][0]), "+v"(acc[m][1]));
  };
  typedef std::integral_constant<int, 0> S0;
  typedef std::integral_constant<int, 1> S1;
  typedef std::integral_constant<int, 2> S2;
  typedef std::integral_constant<int, 3> S3;
  const int last = nsteps - 1;
  for (int c = 0; c < last; ++c) {
    read_scales(c);
    load_rows(c + 1);
    __builtin_amdgcn_sched_barrier(0);   // the loads go first, what waits for them last
    products(c, S0{});
    load_weights(c + 1, 0);
    products(c, S1{});
    load_weights(c + 1, 1);
    products(c, S2{});
    load_weights(c + 1, 2);
    products(c, S3{});
    load_weights(c + 1, 3);
    put(c + 1);
    __syncthreads();
  }
  // the last step, of 1 to kStepBlocks blocks
  const int left = nb - kStepBlocks * last;
  read_scales(last);
  products(last, S0{});
  if (left > 2) products(last, S1{});
  if (left > 4) products(last, S2{});
  if (left > 6) products(last, S3{});
  __syncthreads();   // the rows' buffers have been read
  // ---- a lane holds, of one bucket row, 4 groups of 4 neighbouring columns a fragment; each
  // wave turns its fragments round in LDS of its own (the rows' buffers, no longer read), so
  // that the stores are whole cache lines of a row (gated: halves) and not 16-byte pieces
  constexpr int kLanesRow = 32 * kPiece / 16;              // lanes that store one row
  uint8_t* turn = lds_q + wave * 32 * kOutRow;
  uint8_t* out = GATED ? (uint8_t*)p.h : (uint8_t*)p.y;
#pragma unroll
  for (int m = 0; m < MF; ++m) {
#pragma unroll
    for (int f = 0; f < (GATED ? 1 : 2); ++f) {
      if (col[f] >= p.N) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f32x4 v;
#pragma unroll
        for (int t = 0; t < 4; ++t) v[t] = acc[m][f][4 * q + t];
        uint8_t* to = turn + (lane & 31) * kOutRow + (8 * q + 4 * half) * kPiece;
        if constexpr (GATED) {
          float z[4];
#pragma unroll
          for (int t = 0; t < 4; ++t) z[t] = silu_mul(v[t], acc[m][1][4 * q + t]);
          *(u32x2*)to = u32x2{pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3])};
        } else {
          *(f32x4*)to = v;
        }
      }
      wave_sync();
#pragma unroll
      for (int j = 0; j < kLanesRow / 2; ++j) {
        const int r = j * (kWave / kLanesRow) + lane / kLanesRow;
        const int pos = m0 + 32 * m + r;
        const u32x4 v = *(const u32x4*)(turn + r * kOutRow + lane % kLanesRow * 16);
        if (pos < mend)
          __builtin_nontemporal_store(
              v, (u32x4*)(out + ((int64_t)pos * p.N + col[f]) * kPiece + lane % kLanesRow * 16));
      }
      wave_sync();
    }
  }
}

template <int FMT, bool GATED, int MF, int NW>
hipError_t launch_gemm_t(const MxProduct& p, hipStream_t st) {
  constexpr int BM = 32 * MF, kCols = 64 * NW, TN = GATED ? kCols / 2 : kCols;
  const int pairs = p.T * p.k;
  const int n_mtiles = (pairs + BM - 1) / BM + min(p.E, pairs);   // most that can be
  const int n_ntiles = (p.N + TN - 1) / TN;
  // a launch holds fewer than 2^32 threads: 2^22 workgroups of at most 512 at a time. T*k*N below
  // 2^38 fills at most 2^25 tiles, and 256 experts' last ones 2^28 of N below 2^27
  constexpr int kMax = (1 << 22) / 512;
  const int n = (int)(((int64_t)n_mtiles * n_ntiles + 511) / 512);   // below 2^21
  for (int first = 0; first < n; first += kMax) {
    const dim3 grid(512 * (n - first < kMax ? n - first : kMax));
    hipLaunchKernelGGL((k_mx_gemm<FMT, GATED, MF, NW>), grid, dim3(kWave * NW), 0, st, p, n_mtiles,
                       n_ntiles, first);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Rows a tile. A tall tile reads the weights less often and feeds more products per operand
// read; a low one leaves fewer of its rows empty, and there are more of them to fill the CUs.
// So by the mean rows of an expert: gate/up, us with 32 / 64 / 128 rows, H = I = 2880, 32
// experts, MXFP6, mean 41: 74 / 73 / 76; 62: 87 / 90 / 78; 125: 127 / 104 / 136; 250: 204 / 163
// / 146; where the r-th expert is wanted r^-1.1 times as often: 74 / 86 / 76, 93 / 87 / 108, 127
// / 111 / 133, 198 / 160 / 166; H 2048, I 768, 128 experts, MXFP4, mean 62: 62 / 56 / 61; 125: 87
// / 68 / 72. And by the tiles that there are (256 CUs hold 512 of 128 rows at once): MXFP4, down,
// 184 tiles of 128 rows, H 1024, I 1536: 18 / 15 / 22; 60 tiles, H = I = 1024: 9.7 / 12 / 17;
// gate/up, 552 tiles: 31 / 27 / 30; 1000 tiles, H 256, I 512: 25 / 22 / 20. Where it loses: down,
// H = I = 2880, mean 200 to 250, whose 600 to 744 tiles of 128 rows take 73-82 us (MXFP6 68-95)
// against the 76-94 (83-102) of 64 rows. The height is the same for every expert of a launch.
// MXFP6 rows take eight waves a tile of 128 x 512: half the row bytes and registers a wave
// (four waves spill): 16384 tokens, H = I = 2880, gate/up 819 against 817 us, down 485 against
// 466; 4096 tokens, H 4096, I 14336, 681 against 638 and 361 against 359. MXFP4, in the same
// order: 705 against 724, 421 against 417, 572 against 568, 295 against 306, so four.
template <int FMT, bool GATED>
hipError_t launch_t(const MxProduct& p, bool gemv, hipStream_t st) {
  if (gemv) return launch_gemv_t<FMT, GATED>(p, st);
  const int pairs = p.T * p.k, mean = pairs / p.E;
  const int64_t n_ntiles = (p.N + (GATED ? 127 : 255)) / (GATED ? 128 : 256);
  if (mean > 200 && pairs / 128 * n_ntiles >= 768)
    return launch_gemm_t<FMT, GATED, 4, FMT == kMxFp6 ? 8 : 4>(p, st);
  if (mean > 64 && pairs / 64 * n_ntiles >= 300) return launch_gemm_t<FMT, GATED, 2, 4>(p, st);
  return launch_gemm_t<FMT, GATED, 1, 4>(p, st);
}

}  // namespace

hipError_t launch_mx_product(const MxProduct& p, int fmt, bool gated, bool gemv, hipStream_t st) {
  if (fmt == kMxFp4) return gated ? launch_t<kMxFp4, true>(p, gemv, st) : launch_t<kMxFp4, false>(p, gemv, st);
  return gated ? launch_t<kMxFp6, true>(p, gemv, st) : launch_t<kMxFp6, false>(p, gemv, st);
}

}  // namespace moe
