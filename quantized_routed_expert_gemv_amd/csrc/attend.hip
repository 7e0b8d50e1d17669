// Attention of new tokens over a paged cache: with s_j = scale <q, k_j> over the keys in sight,
//   out = sum_j e^{s_j} v_j / (sum_j e^{s_j} + e^{sink})
// in one pass over the keys with a running reference m and sum l: weights are 2^{s'_j - m} with
// s' = s log2 e. m is a whole number, so that rescaling is exact, and is raised only where a score is
// more than 8 above the one that m was set by: the sums seldom have to be rescaled.
// m, l and the weighted sum are fp32; a weight is rounded to the queries' 16-bit type where it
// meets the values in a matrix instruction, or to two numbers of it (few rows, see kMost). With one number
// (many rows) l adds up the rounded weights, so that half a step of each counts by how far its value is
// from the row's output: with few keys, or one that has most of the weight, by little. In fp16 half a
// step is 2^-25 for weights below 2^-14. So m is set 7 below the highest score there, which leaves
// a row's largest weight between 2^6 and 2^15 (fp16 ends at 65504): weights down to 2^-20 of the
// largest have all of their bits, and smaller ones lose at most 2^-31 of it each. With m at the highest
// score, 131068 keys 23 binary orders below four others, 0.5 per cent of a row, came to a fifth less.
// (Scores past 2^28 in s' are too far apart in fp32 for fp16 weights.)
//
// The query heads of a KV head are rows of one tile, so its keys and values are read once. Both
// products have keys as the matrix rows: S^T = K Q^T leaves a lane the scores of one query, in
// the order in which P^T is an operand of O^T = V^T P^T, so weights never leave their lane.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"
#include "kv.hpp"

namespace moe {

namespace {

typedef _Float16 f16x8 __attribute__((__vector_size__(8 * sizeof(_Float16))));
typedef _Float16 f16x2 __attribute__((__vector_size__(2 * sizeof(_Float16))));

typedef float f32x16 __attribute__((__vector_size__(16 * sizeof(float))));
typedef short i16x4 __attribute__((__vector_size__(4 * sizeof(short))));

constexpr float kLog2e = 1.44269504088896340736f;
// How far below the highest score m is set, and how far above m a score has to be to raise it.
template <bool F16> constexpr float kBelow = F16 ? 7.f : 0.f;
template <bool F16> constexpr float kRaise = kBelow<F16> + 8.f;

template <bool F16>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // RNE, NaN kept
  if constexpr (F16) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  else return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
template <bool F16>
__device__ __forceinline__ float value(uint32_t bits) {
  return F16 ? fp16_to_f32(uint16_t(bits)) : bf16_lo(bits);
}
template <bool F16>
__device__ __forceinline__ float value_hi(uint32_t bits) {
  return F16 ? fp16_to_f32(uint16_t(bits >> 16)) : bf16_hi(bits);
}
// sum and both 16-bit values. The instruction's own sum of three is not always to nearest in fp16.
template <bool F16>
__device__ __forceinline__ float add2(uint32_t w, float sum) {
  if constexpr (F16)
    return sum + __builtin_amdgcn_fdot2(__builtin_bit_cast(f16x2, w), f16x2{1, 1}, 0.f, false);
  else
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), bf16x2{1, 1}, sum, false);
}
// Two E4M3 codes (the low or the high half of v) as two values of the 16-bit type, exactly.
template <bool F16, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t v) {
  if constexpr (F16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.f, HI));
}
// N values of a cache's row as they lie there: N / 2 dwords of a 16-bit cache, N / 4 of an 8-bit one.
template <int N, bool FP8>
__device__ __forceinline__ void load_raw(const uint8_t* plane, int64_t at, uint32_t* w) {
  constexpr int DW = FP8 ? N / 4 : N / 2;
  const uint8_t* p = plane + at * (FP8 ? 1 : 2);
  if constexpr (DW == 4) {
    const u32x4 v = *(const u32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = v[i];
  } else if constexpr (DW == 2) {
    const u32x2 v = *(const u32x2*)p;
    w[0] = v[0], w[1] = v[1];
  } else {
    w[0] = *(const uint32_t*)p;
  }
}
// The same as values of the 16-bit type, two a dword.
template <int N, bool F16, bool FP8>
__device__ __forceinline__ void widen(const uint32_t* raw, uint32_t* w) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    if constexpr (!FP8) w[i] = raw[i];
    else w[i] = i & 1 ? widen2<F16, true>(raw[i / 2]) : widen2<F16, false>(raw[i / 2]);
  }
}

__device__ __forceinline__ float plane_value(const uint8_t* plane, int64_t at, int type) {
  if (type == kE4M3) return __builtin_amdgcn_cvt_f32_fp8((int)plane[at], 0);
  const uint16_t v = ((const uint16_t*)plane)[at];
  return type == kFP16 ? fp16_to_f32(v) : bf16_to_f32(v);
}

// What a tile of query rows is, the same for the whole workgroup. Row r of the tile is query head
// r % group of the KV head, of new token r / group counted from the sequence's first.
struct Tile {
  int seq, head;
  int row0, rows;      // the tile's first row in its sequence, and how many it has
  int token0;          // row of the sequence's first new token in q and out
  int pos0;            // that token's position
  int end;             // keys that can be seen: [0, end)
  int first, kept;     // of them [0, kept) and [first, end) are in sight of some row
  int last_of_first;   // the last key that the first row sees, and the first one in the window of
  int first_of_last;   // the last row: between them every row sees every key
};

// The new token of a row.
__device__ __forceinline__ int token_of(const AttendCall& a, int row) {
  return div_by(row, a.group, a.group_inv);
}

// The first key in the window of position pos.
__device__ __forceinline__ int window_start(const AttendCall& a, int pos) {
  return a.window ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
}

// Sequences of up to this many rows (new tokens * group) go to the kernel for few rows. Alone behind 16384
// keys (32 over 4 heads of 128, us): 32 rows 24 against 29 with the one for many, 48 rows 26 against 29, 64
// rows 32 against 29; 16 sequences of up to 40 rows, where the keys are read again for each 16 of them:
// 269 for all, 237 for those of up to 32.
constexpr int kFewRows = 32;

// The tile that stands at place x of the launch, of R rows; false: none.
// FEW: of the sequences with few rows; else of the others, or of all where no second launch takes them.
// Sequence b's begin at floor(q_start[b] * group / R) + b, which leaves each sequence as many places
// as it can need. Beside the launch for many rows, each has as many as few rows need.
template <int R, bool FEW>
__device__ __forceinline__ bool find_tile(const AttendCall& a, int64_t x, int head, Tile* t) {
  constexpr int kFewTiles = kFewRows / R;
  const KvBatchView& b = a.batch;
  int seq;
  int64_t row0;
  if (FEW && a.both) {
    seq = (int)(x / max(kFewTiles, 1));
    row0 = (x - (int64_t)seq * kFewTiles) * R;
  } else if (!FEW && b.n_seq <= kWave) {
    // The longest context's tiles first, and of a sequence those of its last rows, which see most: a
    // batch ends with short tiles. A lane counts the tiles in front of its sequence's.
    const int lane = threadIdx.x & (kWave - 1);
    int tiles = 0, len = 0, before = 0;
    if (lane < b.n_seq) {
      const int64_t rows = (int64_t)(first_row(b, lane + 1) - first_row(b, lane)) * a.group;
      if (rows > (a.both ? kFewRows : 0)) tiles = (int)((rows + R - 1) / R);
      len = b.seq_len[lane];
    }
    for (int i = 0; i < b.n_seq; ++i) {
      const int other = __builtin_amdgcn_readlane(len, i), n = __builtin_amdgcn_readlane(tiles, i);
      before += other > len || (other == len && i < lane) ? n : 0;
    }
    const uint64_t here = __ballot(before <= x && x < (int64_t)before + tiles);
    if (here == 0) return false;
    seq = __builtin_ctzll(here);
    row0 = ((int64_t)__builtin_amdgcn_readlane(before, seq) + __builtin_amdgcn_readlane(tiles, seq) - 1 -
            x) * R;
  } else {
    if (!FEW) x = a.tiles - 1 - x;   // later tiles first
    seq = wave_find(b.n_seq, x, [&](int i) {
      return (int64_t)first_row(b, i) * a.group / R + i;
    });
    row0 = (x - (int64_t)first_row(b, seq) * a.group / R - seq) * R;
  }
  const int lo = first_row(b, seq), n = first_row(b, seq + 1) - lo;
  const int64_t rows = (int64_t)n * a.group - row0;
  if (n <= 0 || row0 < 0 || rows <= 0) return false;
  if (a.both && ((int64_t)n * a.group <= kFewRows) != FEW) return false;
  const int64_t cap = (int64_t)b.max_pages * a.cache.page_size;
  const int len = max(b.seq_len[seq], 0);
  t->seq = seq;
  t->head = head;
  t->row0 = (int)row0;
  t->rows = (int)min(rows, (int64_t)R);
  t->token0 = lo;
  t->pos0 = len - n;
  const int first_tok = token_of(a, t->row0), last_tok = token_of(a, t->row0 + t->rows - 1);
  const int end = (int)min((int64_t)len, cap);
  t->end = a.causal ? max(min(end, t->pos0 + last_tok + 1), 0) : end;
  t->last_of_first = a.causal ? min(t->pos0 + first_tok, t->end - 1) : t->end - 1;
  t->first = window_start(a, t->pos0 + first_tok);
  t->first_of_last = window_start(a, t->pos0 + last_tok);
  t->first = min(t->first, t->end);
  t->kept = min(min(a.keep_first, t->first), t->end);
  if (a.err && threadIdx.x == 0 && (t->pos0 < 0 || len > cap)) atomicOr(a.err, 1u);
  return true;
}

// Keys go in blocks of 32 (B): those that hold kept ones, then those of the window.
template <int B>
struct Blocks {
  int kept, first, count;
  __device__ explicit Blocks(const Tile& t) {
    kept = (t.kept + B - 1) / B;
    first = t.first / B;
    if (first <= kept) first = kept = 0;
    count = kept + max((t.end + B - 1) / B - first, 0);
  }
  __device__ int key(int i) const { return (i < kept ? i : i - kept + first) * B; }
};

// Element offsets of a key's rows in the cache. A key out of sight, or on no page, has ok false
// and the offsets of some readable row.
struct KeyRow {
  int64_t k, v;
  bool ok;
};
// RUN keys from pos on are on one page; the first key's row is returned.
template <int RUN>
__device__ __forceinline__ KeyRow key_row(const AttendCall& a, const Tile& t, int pos) {
  KeyRow r;
  r.ok = pos < t.end && (pos + RUN > t.first || pos < t.kept);
  int row = 0, page = 0;
  if (r.ok) {
    const int p = page_of((uint32_t)pos, a.cache.page_size, a.cache.page_inv, &row);
    page = a.batch.table[t.seq * a.batch.table_stride + p];
    if ((unsigned)page >= (unsigned)a.cache.n_pages) {
      if (a.err) atomicOr(a.err, 1u);
      r.ok = false;
      page = row = 0;
    }
  }
  r.k = page * a.cache.k_page + row * a.cache.k_token + t.head * a.cache.k_head;
  r.v = page * a.cache.v_page + row * a.cache.v_token + t.head * a.cache.v_head;
  return r;
}

// The row of a split's parts that holds row r of a tile. Beside a launch for many rows, each sequence's few
// rows have kFewRows places for every KV head, so that the room that they need does not grow with the
// others' rows.
template <bool FEW>
__device__ __forceinline__ int64_t part_row(const AttendCall& a, const Tile& t, int split, int r,
                                            int64_t token, int head) {
  if (FEW && a.both)
    return split * a.parts_few.rows + ((int64_t)t.seq * a.cache.n_heads + t.head) * kFewRows + t.row0 + r;
  return split * (FEW ? a.parts_few.rows : a.parts.rows) + token * a.n_q_heads + head;
}

// Where a tile's sums go: out, or a split's part.
template <bool F16, bool FEW, int N>
__device__ __forceinline__ void store_row(const AttendCall& a, const Tile& t, int split, int r, int d,
                                          float m, float l, const float* o) {
  const int tok = token_of(a, t.row0 + r), g = t.row0 + r - tok * a.group;
  const int64_t token = t.token0 + tok;
  const int head = t.head * a.group + g;
  if ((FEW ? a.splits_few : a.splits) > 1) {
    const AttendParts& parts = FEW ? a.parts_few : a.parts;
    const int64_t at = part_row<FEW>(a, t, split, r, token, head);
    if (d == 0) {
      parts.stats[2 * at] = m;
      parts.stats[2 * at + 1] = l;
    }
#pragma unroll
    for (int i = 0; i < N; i += 4) *(f32x4*)(parts.sums + at * a.cache.D + d + i) = f32x4{
        o[i], o[i + 1], o[i + 2], o[i + 3]};
    return;
  }
  float w = 1.f;
  if (a.sinks) {
    const float s = a.sinks[head] * kLog2e, top = fmaxf(m, s);
    w = exp2f(m - top);
    l = l * w + exp2f(s - top);
  }
  w = m == -INFINITY ? 0.f : w / l;
  uint16_t* p = (uint16_t*)a.out.p + token * a.out.token + head * a.out.head + d;
#pragma unroll
  for (int i = 0; i < N; i += 4)
    *(u32x2*)(p + i) = u32x2{pack2<F16>(w == 0.f ? 0.f : o[i] * w, w == 0.f ? 0.f : o[i + 1] * w),
                             pack2<F16>(w == 0.f ? 0.f : o[i + 2] * w, w == 0.f ? 0.f : o[i + 3] * w)};
}

// Whether every row of the tile sees every key of key0 .. key0 + B - 1 (that is on a page).
template <int B>
__device__ __forceinline__ bool whole_block(const AttendCall& a, const Tile& t, int key0) {
  return key0 + B - 1 <= t.last_of_first &&
         (key0 >= t.first_of_last || (a.window && key0 + B - 1 < a.keep_first));
}

// A matrix instruction would multiply a weight of 0, of a row that does not see a key, by that key's
// values. Where not every row sees a block, values that are infinite or NaN go into the product as 0,
// and a workgroup that met one comes here when its rows are stored: each row takes the odd values of
// the keys that it sees, times a weight that is not 0, which is adding them.
template <bool F16, bool FEW, int B>
__device__ void add_odd_values(const AttendCall& a, const Tile& t, const Blocks<B>& blocks, int b0,
                               int b1, int split) {
  __threadfence_block();
  __syncthreads();   // the rows are stored
  const int d = threadIdx.x;
  if (d >= a.cache.D) return;
  const float vs = a.cache.type == kE4M3 && a.cache.v_scale ? a.cache.v_scale[t.head] : 1.f;
  for (int b = b0; b < b1; ++b) {
    const int key0 = blocks.key(b);
    if (whole_block<B>(a, t, key0)) continue;
    for (int key = key0; key < key0 + B; ++key) {
      const KeyRow kv = key_row<1>(a, t, key);
      if (!kv.ok) continue;
      const float v = plane_value(a.cache.v, kv.v + d, a.cache.type) * vs;
      if (fabsf(v) < INFINITY) continue;
      for (int r = 0; r < t.rows; ++r) {
        const int tok = token_of(a, t.row0 + r), pos = t.pos0 + tok;
        if (a.causal && key > pos) continue;
        if (key < window_start(a, pos) && key >= a.keep_first) continue;
        const int64_t token = t.token0 + tok;
        const int head = t.head * a.group + t.row0 + r - tok * a.group;
        if ((FEW ? a.splits_few : a.splits) > 1) {
          (FEW ? a.parts_few : a.parts).sums[part_row<FEW>(a, t, split, r, token, head) * a.cache.D + d] += v;
        } else {
          uint16_t* p = (uint16_t*)a.out.p + token * a.out.token + head * a.out.head + d;
          *p = (uint16_t)pack2<F16>(value<F16>(*p) + v, 0.f);
        }
      }
    }
  }
}

// Takes infinities and NaN out of a pair of 16-bit values; whether there were any.
template <bool F16>
__device__ __forceinline__ bool take_odd(uint32_t& v, bool take = true) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  const bool lo = take & ((v & e) == e), hi = take & ((v >> 16 & e) == e);
  v = (lo ? 0u : v & 0xFFFFu) | (hi ? 0u : v & 0xFFFF0000u);
  return lo || hi;
}

constexpr int kRowTile = 16;
constexpr int kRowThreads = 256;

// The part of a weight that is rounded to its first operand; its second one is what is left. Together
// they have 14 bits (bf16) or 13 (fp16), where one has 8 or 11. Both are positive, so that an infinite value
// stays one: a rest of 0 or less, as beside the rounded weight itself, would make it NaN. (Of fp16 a quarter
// is left, a number down to weights of 2^-22.)
template <bool F16> constexpr float kMost = F16 ? 0.75f : 0.984375f;

// Few rows a sequence: the cache's bytes bound it. A tile is 16 rows, the columns of 16x16x32
// instructions, so nothing goes through LDS but the end: a lane's 16-byte loads of K rows are
// operands as they are, and its loads of eight V rows become V^T operands by 16-bit picks (one a
// dword). The four waves take every fourth block of 32 keys and join in LDS.
// Key of matrix row m of the block's product u: 8 (m / 4) + 4 u + m % 4, so that a lane's eight
// scores are those of eight neighbouring keys, 8 (lane / 16) on.
// The matrix pipes have time, so a weight is two operands: rounded to one, it added as much error to the
// outputs as their own rounding (0.0024 in place of 0.0017 of bf16). It added 2 us to the 555 below, and 1 to 42.
// Blocks are loaded one ahead, into registers. 64 sequences of up to 16384 keys, 32 heads over 8 of 128:
// 557-562 us, 4.9 TB/s; 131072 keys of an 8-bit cache, 32 over 4 heads, in 128 splits: 38 us, 3.5 TB/s.
// P8: pages hold a multiple of 8 tokens, so such a run of keys is on one page.
template <bool F16, bool FP8, int DV, bool P8>
__global__ __launch_bounds__(kRowThreads, DV > 128 ? 1 : 2) void k_attend_rows(AttendCall a) {
  constexpr int NW = kRowThreads / kWave;
  constexpr int E = DV >= 128 ? 8 : DV / 16, NH = DV / (16 * E), NK = DV / 32;
  constexpr int OS = DV + 4;
  __shared__ float so[NW][kRowTile][OS];
  __shared__ float sm[NW][kRowTile], sl[NW][kRowTile];
  __shared__ int s_odd;
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int n = lane & 15, g = lane >> 4;
  // workgroups go KV head by KV head (an XCD's stay on few of them), then split by split
  const int split = (int)(blockIdx.x / (unsigned)a.cache.n_heads);
  const int head = (int)blockIdx.x - split * a.cache.n_heads;
  Tile t;
  if (!find_tile<kRowTile, true>(a, a.block0 + blockIdx.y, head, &t)) return;
  const Blocks<32> blocks(t);
  const int b0 = (int)((int64_t)blocks.count * split / a.splits_few);
  const int b1 = (int)((int64_t)blocks.count * (split + 1) / a.splits_few);
  const int D = a.cache.D;
  if (threadIdx.x == 0) s_odd = 0;
  __syncthreads();

  // this lane's query: the keys that it sees, and its row of q as an operand
  const int tok = token_of(a, t.row0 + n);
  const bool row_ok = n < t.rows;
  const int pos = t.pos0 + tok;
  const int see_last = !row_ok ? -1 : a.causal ? min(pos, t.end - 1) : t.end - 1;
  const int see_first = window_start(a, pos);
  const int keep = a.window ? a.keep_first : 0;
  float c = a.scale * kLog2e;
  if (FP8 && a.cache.k_scale) c *= a.cache.k_scale[t.head];
  const uint32_t flip = c < 0.f ? 0x80008000u : 0u;   // scores are scaled by a positive number
  c = fabsf(c) < 1e-37f ? 1e-37f : fabsf(c);
  // Where in a row a lane's operand of k-step k begins: any order serves that is the same for
  // queries and keys, and an 8-bit cache's lane takes 16 bytes, two steps, at once.
  auto depth = [&](int k) { return FP8 ? 64 * (k / 2) + 16 * g + 8 * (k & 1) : 32 * k + 8 * g; };
  u32x4 q[NK];
  {
    const uint16_t* p = (const uint16_t*)a.q.p + (int64_t)(t.token0 + tok) * a.q.token +
                        (int64_t)(t.head * a.group + t.row0 + n - tok * a.group) * a.q.head;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      q[k] = u32x4{0, 0, 0, 0};
      if (row_ok && depth(k) < D) q[k] = *(const u32x4*)(p + depth(k)) ^ flip;
    }
  }
  f32x4 o[NH][E];
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int i = 0; i < E; ++i) o[h][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  // A block's loads, as they lie in the cache; those of the next block are under way while one is
  // computed. ok: of this lane's eight keys, those on a page and in sight.
  constexpr int KS = FP8 ? 16 : 8, NL = DV / (4 * KS), KW = 4, VW = FP8 ? E / 4 : E / 2;
  struct Raw {
    uint32_t k[2][NL][KW], v[8][NH][VW], ok;
  };
  auto load_k = [&](Raw& raw, int u, int64_t at) {
#pragma unroll
    for (int k = 0; k < NL; ++k) {
      const int d = 4 * KS * k + KS * g;
      load_raw<KS, FP8>(a.cache.k, at + (d < D ? d : 0), raw.k[u][k]);
    }
  };
  auto load_v = [&](Raw& raw, int j, int64_t at) {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const int d = 16 * E * h + E * n;
      load_raw<E, FP8>(a.cache.v, at + (d < D ? d : 0), raw.v[j][h]);
    }
  };
  auto load = [&](Raw& raw, int b) {
    const int key0 = blocks.key(b);
    if constexpr (P8) {
      const KeyRow rk = key_row<8>(a, t, key0 + 8 * (n >> 2));
#pragma unroll
      for (int u = 0; u < 2; ++u)
        load_k(raw, u, rk.k + (rk.ok ? (4 * u + (n & 3)) * a.cache.k_token : 0));
      const KeyRow rv = key_row<8>(a, t, key0 + 8 * g);
#pragma unroll
      for (int j = 0; j < 8; ++j) load_v(raw, j, rv.v + (rv.ok ? j * a.cache.v_token : 0));
      raw.ok = rv.ok ? 0xFFu : 0u;
    } else {
      raw.ok = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u)
        load_k(raw, u, key_row<1>(a, t, key0 + 8 * (n >> 2) + 4 * u + (n & 3)).k);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const KeyRow rv = key_row<1>(a, t, key0 + 8 * g + j);
        load_v(raw, j, rv.v);
        raw.ok |= (uint32_t)rv.ok << j;
      }
    }
  };

  Raw raw;
  if (b0 + wave < b1) load(raw, b0 + wave);
  for (int b = b0 + wave; b < b1; b += NW) {
    const int key0 = blocks.key(b);
    Raw next;
    if (b + NW < b1) load(next, b + NW);
    u32x4 kf[2][NK];
    uint32_t vf[8][NH][E / 2];
    const uint32_t v_ok = raw.ok;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < NL; ++k) {
        widen<KS, F16, FP8>(raw.k[u][k], (uint32_t*)&kf[u][k * NK / NL]);
        if (4 * KS * k + KS * g >= D)
#pragma unroll
          for (int i = 0; i < NK / NL; ++i) kf[u][k * NK / NL + i] = u32x4{0, 0, 0, 0};
      }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int h = 0; h < NH; ++h) widen<E, F16, FP8>(raw.v[j][h], vf[j][h]);
    f32x4 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NK; ++k) s[u] = mma16<F16>(kf[u][k], q[k], s[u]);
    }
    // lane (n, g): s[u][i] is the score of query n and key key0 + 8 g + 4 u + i
    float x[8];   // scores, then weights
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = s[j / 4][j % 4];
    const bool seen = whole_block<32>(a, t, key0);
    if (!seen || !__all(v_ok == 0xFFu)) {
      bool odd = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = key0 + 8 * g + j;
        const bool ok = v_ok >> j & 1;
        // selects of scalars, no branches (see k_attend_tiles)
        const bool out = (key > see_last) | ((key < see_first) & (key >= keep)) | !ok;
        x[j] = out ? -INFINITY : x[j];
        // values behind the end, before the window, or on no page: anything may stand there
        const bool some = ok & (key < t.end) & ((key >= t.first) | (key < t.kept));
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int i = 0; i < E / 2; ++i) {
            vf[j][h][i] = some ? vf[j][h][i] : 0;
            if (!seen) odd |= take_odd<F16>(vf[j][h][i]);
          }
      }
      if (odd) s_odd = 1;
    }
    float top = x[0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, x[j]);
    top *= c;
    if (__any(top - m > kRaise<F16>)) {   // (m + kRaise would be rounded, past 2^27 by 8)
      top = fmaxf(top, wave_xor(top, 16));
      top = fmaxf(top, wave_xor(top, 32));
      const float to = top - m > kRaise<F16> ? ceilf(top) - kBelow<F16> : m;   // by a row's own scores alone
      const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int i = 0; i < E; ++i) o[h][i] *= f;
    }
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = __builtin_amdgcn_exp2f(fmaf(x[j], c, -base));
      l += x[j];
    }
    u32x4 most, rest;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      most[j] = pack2<F16>(kMost<F16> * x[2 * j], kMost<F16> * x[2 * j + 1]);
      rest[j] = pack2<F16>(x[2 * j] - value<F16>(most[j]), x[2 * j + 1] - value_hi<F16>(most[j]));
    }
#pragma unroll
    for (int h = 0; h < NH; ++h)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        u32x4 vt;
        const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          vt[j] = __builtin_amdgcn_perm(vf[2 * j + 1][h][i / 2], vf[2 * j][h][i / 2], sel);
        o[h][i] = mma16<F16>(vt, most, o[h][i]);
        o[h][i] = mma16<F16>(vt, rest, o[h][i]);
      }
    raw = next;
  }

  l += wave_xor(l, 16);
  l += wave_xor(l, 32);
  if (g == 0) {
    sm[wave][n] = m;
    sl[wave][n] = l;
  }
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) so[wave][n][16 * E * h + E * (4 * g + e) + i] = o[h][i][e];
  __syncthreads();
  const int r = threadIdx.x / 16, col = threadIdx.x % 16;
  float top = sm[0][r];
#pragma unroll
  for (int w = 1; w < NW; ++w) top = fmaxf(top, sm[w][r]);
  float f[NW], sum = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    f[w] = sm[w][r] == -INFINITY ? 0.f : exp2f(sm[w][r] - top);
    // scores of NaN alone leave the maximum where it was, and a sum that is NaN
    sum = sl[w][r] == 0.f ? sum : fmaf(sm[w][r] == -INFINITY ? 1.f : f[w], sl[w][r], sum);
  }
  const float vs = FP8 && a.cache.v_scale ? a.cache.v_scale[t.head] : 1.f;
#pragma unroll
  for (int h = 0; h < NH; ++h) {
    const int d = 16 * E * h + E * col;
    if (d >= D || r >= t.rows) continue;
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v[i] = fmaf(f[w], so[w][r][d + i], v[i]);
      v[i] *= vs;
    }
    store_row<F16, true, E>(a, t, split, r, d, sum != sum ? fmaxf(top, 0.f) : top, sum, v);
  }
  if (s_odd) add_odd_values<F16, true>(a, t, blocks, b0, b1, split);
}

constexpr int kTileThreads = 256;
constexpr int kTileRows = 128;   // 32 a wave
constexpr int kTileKeys = 64;

// A row of keys or values in LDS is DV values in 16-byte pieces, in the order piece ^ key_order(row) or
// piece ^ value_order(row). Keys are read a piece a lane over 16 rows, values through the transposing
// read, four pieces of four rows at once: either way on all banks.
template <int DV> __device__ __forceinline__ int key_order(int row) {
  return row & (DV >= 128 ? 15 : 7);
}
template <int DV> __device__ __forceinline__ int value_order(int row) {
  return DV >= 128 ? 4 * (row & 3) : 4 * (row >> 1 & 1);
}

__device__ __align__(16) const uint32_t g_zero[4] = {0, 0, 0, 0};   // read in place of what is behind D

// The transposing LDS read: of 16 lanes, lane i reads 8 bytes (its address) of row i / 4, columns
// 4 (i % 4) on, and is left with column i of the four rows. (The compiler waits in front of it for
// every load into LDS that is under way. Reads in inline assembly, which carry their own wait, gained
// 2.3-3.9 per cent over staging through registers, these 3.4-4.7.)
__device__ __forceinline__ u32x2 read_columns(const uint8_t* p) {
  typedef __attribute__((address_space(3))) i16x4* lds_p;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)p));
}

// Many rows a sequence: the matrix instructions bound it. Four waves of 32 rows (columns of
// 32x32x16 instructions) share tiles of 64 keys and values in two LDS buffers, the next tile's loads in
// flight behind the products of this one: of a 16-bit cache straight into LDS, of an 8-bit one through
// registers, where they are widened. Values reach the second product through the transposing LDS read,
// in the order of keys in which the first left the weights: 16 s + {4 h .. + 3, 8 + 4 h .. + 3} for
// k-step s and lane half h.
// 8192 tokens behind 8192 others, 32 heads over 8 of 128: 1.78-1.85 ms, 0.89-0.92 PFLOP/s, 2.04 where 16-bit
// keys and values were staged through registers. The matrix pipes are busy in 40 cycles of 100 and the
// vector ones in 52: the scores' exponentials, sums and roundings are as long as the products, and run
// beside them by halves of a block, but not all of the way; without any loads it would take 1.50. LDS
// reads have no conflicts. 128 rows: at 2 waves a SIMD the sums and operands just fit the registers.
// The same over an 8-bit cache 1.79-1.80; as many operations in 64 heads over 8 of 64 2.09-2.15 on either
// cache, in 16 over 8 of 256 2.50 (8-bit 2.44), one workgroup a CU; in a window of 4096 keys 0.65-0.69.
// U16: pages hold a multiple of 16 tokens, so the 16 rows of a tile that a wave loads are on one.
template <bool F16, bool FP8, int DV, bool U16>
__global__ __launch_bounds__(kTileThreads, DV > 128 ? 1 : 2) void k_attend_tiles(AttendCall a) {
  constexpr int NK = DV / 16, ND = DV / 32;
  constexpr int CH = DV * (FP8 ? 1 : 2) / 16;          // 16-byte chunks of a row
  constexpr int RP = kWave / CH, NP = 16 / RP;         // rows a wave loads at once; passes
  constexpr int CV = FP8 ? 16 : 8;                     // values of a chunk
  constexpr int kRow = 2 * DV;                         // bytes of a row in LDS
  __shared__ __align__(16) uint8_t s_k[2][kTileKeys * kRow], s_v[2][kTileKeys * kRow];
  __shared__ uint64_t s_ok[2];                         // rows of the tile that are on a page
  __shared__ int s_odd;
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int n = lane & 31, hf = lane >> 5;
  const int split = (int)(blockIdx.x / (unsigned)a.cache.n_heads);
  const int head = (int)blockIdx.x - split * a.cache.n_heads;
  Tile t;
  if (!find_tile<kTileRows, false>(a, a.block0 + blockIdx.y, head, &t)) return;
  const Blocks<kTileKeys> blocks(t);
  const int b0 = (int)((int64_t)blocks.count * split / a.splits);
  const int b1 = (int)((int64_t)blocks.count * (split + 1) / a.splits);
  const int D = a.cache.D;
  if (threadIdx.x == 0) s_odd = 0;
  __syncthreads();

  const int r = 32 * wave + n;
  const int tok = token_of(a, t.row0 + r);
  const bool row_ok = r < t.rows;
  const int pos = t.pos0 + tok;
  const int see_last = !row_ok ? -1 : a.causal ? min(pos, t.end - 1) : t.end - 1;
  const int see_first = window_start(a, pos);
  const int keep = a.window ? a.keep_first : 0;
  // what all of the wave's rows see last, and first
  const int w_rows = min(max(t.rows - 32 * wave, 0), 32);
  const int w_first = t.pos0 + token_of(a, t.row0 + 32 * wave);
  const int w_last = t.pos0 + token_of(a, t.row0 + 32 * wave + max(w_rows, 1) - 1);
  const int w_all = a.causal ? min(w_first, t.end - 1) : t.end - 1;
  const int w_from = window_start(a, w_last);
  float c = a.scale * kLog2e;
  if (FP8 && a.cache.k_scale) c *= a.cache.k_scale[t.head];
  const uint32_t flip = c < 0.f ? 0x80008000u : 0u;
  c = fabsf(c) < 1e-37f ? 1e-37f : fabsf(c);
  u32x4 q[NK];
  {
    const uint16_t* p = (const uint16_t*)a.q.p + (int64_t)(t.token0 + tok) * a.q.token +
                        (int64_t)(t.head * a.group + t.row0 + r - tok * a.group) * a.q.head;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const int d = 16 * k + 8 * hf;
      q[k] = u32x4{0, 0, 0, 0};
      if (row_ok && d < D) q[k] = *(const u32x4*)(p + d) ^ flip;
    }
  }
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
  float m = -INFINITY, l = 0.f;

  // Loads: the rows of each pass, j RP + rsub, and this lane's chunk of them. Straight into LDS lane l's
  // piece lands at place l, so the chunk is the one whose place that is.
  typedef __attribute__((address_space(3))) void* lds_ptr;
  typedef __attribute__((address_space(1))) const void* global_ptr;
  constexpr int kSize = FP8 ? 1 : 2;
  const int rsub = lane / CH;
  int k_chunk[NP], v_chunk[NP];
  uint32_t k_off[NP], v_off[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    k_chunk[j] = FP8 ? lane % CH : (lane % CH) ^ key_order<DV>(j * RP + rsub);
    v_chunk[j] = FP8 ? lane % CH : (lane % CH) ^ value_order<DV>(j * RP + rsub);
    k_off[j] = (uint32_t)(rsub * a.cache.k_token + (k_chunk[j] * CV < D ? k_chunk[j] * CV : 0)) * kSize;
    v_off[j] = (uint32_t)(rsub * a.cache.v_token + (v_chunk[j] * CV < D ? v_chunk[j] * CV : 0)) * kSize;
  }
  u32x4 kr[NP], vr[NP];   // of an 8-bit cache
  auto fetch = [&](const uint8_t* p, bool in, uint8_t* to, u32x4& reg) {
    if constexpr (FP8)
      reg = *(const u32x4*)p;
    else if (D == DV)
      __builtin_amdgcn_global_load_lds((global_ptr)p, (lds_ptr)to, 16, 0, 0);
    else
      __builtin_amdgcn_global_load_lds(in ? (global_ptr)p : (global_ptr)g_zero, (lds_ptr)to, 16, 0, 0);
  };
  // Of this wave's 16 rows of a block: U16, their page (asked for a block ahead of its use) and the
  // row of it, and which are on a page and in sight.
  struct Rows {
    int page, row;
    uint32_t ok;
  };
  auto lookup = [&](int b) {
    Rows r = {0, 0, 0};
    if constexpr (U16) {
      const int p = blocks.key(b) + 16 * wave;
      if (b < b1 && p < t.end && (p + 16 > t.first || p < t.kept)) {
        const int e = page_of((uint32_t)p, a.cache.page_size, a.cache.page_inv, &r.row);
        r.page = a.batch.table[t.seq * a.batch.table_stride + e];
        const uint32_t below = t.end - p >= 16 ? 0xFFFFu : (1u << (t.end - p)) - 1;
        const uint32_t from = p >= t.first ? 0xFFFFu : (0xFFFFu << min(t.first - p, 16)) & 0xFFFFu;
        const uint32_t kept = p >= t.kept ? 0u
                              : t.kept - p >= 16 ? 0xFFFFu : (1u << (t.kept - p)) - 1;
        r.ok = below & (from | kept);
      }
    }
    return r;
  };
  auto checked = [&](Rows r) {   // U16: a page outside the cache is page 0, with no row in sight
    if constexpr (U16) {
      r.page = __builtin_amdgcn_readfirstlane(r.page);
      if ((unsigned)r.page >= (unsigned)a.cache.n_pages) {
        if (a.err && lane == 0) atomicOr(a.err, 1u);
        r = {0, 0, 0};
      }
    }
    return r;
  };
  auto load_k = [&](int b, int to, Rows& r) {
    uint8_t* lds = s_k[to] + 16 * wave * kRow;
    if constexpr (U16) {
      const uint8_t* base = a.cache.k + (r.page * a.cache.k_page + r.row * a.cache.k_token +
                                         t.head * a.cache.k_head) * kSize;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        fetch(base + j * RP * a.cache.k_token * kSize + k_off[j], k_chunk[j] * CV < D, lds + 1024 * j,
              kr[j]);
    } else {
      r.ok = 0;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const KeyRow kv = key_row<1>(a, t, blocks.key(b) + 16 * wave + j * RP + rsub);
        const bool in = k_chunk[j] * CV < D;
        fetch(a.cache.k + (kv.k + (in ? k_chunk[j] * CV : 0)) * kSize, in, lds + 1024 * j, kr[j]);
        const uint64_t rows = __ballot(kv.ok);
#pragma unroll
        for (int i = 0; i < RP; ++i) r.ok |= (uint32_t)(rows >> (i * CH) & 1) << (j * RP + i);
      }
      r.ok = __builtin_amdgcn_readfirstlane(r.ok);
    }
  };
  auto load_v = [&](int b, int to, const Rows& r) {
    uint8_t* lds = s_v[to] + 16 * wave * kRow;
    if constexpr (U16) {
      const uint8_t* base = a.cache.v + (r.page * a.cache.v_page + r.row * a.cache.v_token +
                                         t.head * a.cache.v_head) * kSize;
#pragma unroll
      for (int j = 0; j < NP; ++j)
        fetch(base + j * RP * a.cache.v_token * kSize + v_off[j], v_chunk[j] * CV < D, lds + 1024 * j,
              vr[j]);
    } else {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const KeyRow kv = key_row<1>(a, t, blocks.key(b) + 16 * wave + j * RP + rsub);
        const bool in = v_chunk[j] * CV < D;
        fetch(a.cache.v + (kv.v + (in ? v_chunk[j] * CV : 0)) * kSize, in, lds + 1024 * j, vr[j]);
      }
    }
  };
  // What lies in registers goes to LDS, widened; values as `finish` says.
  auto store_k = [&](int to) {
    if constexpr (FP8) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int row = 16 * wave + j * RP + rsub;
        uint32_t w[8];
        widen<16, F16, true>((const uint32_t*)&kr[j], w);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          u32x4 v = {w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
          if (D != DV && k_chunk[j] * CV >= D) v = u32x4{0, 0, 0, 0};
          *(u32x4*)(s_k[to] + row * kRow + ((2 * k_chunk[j] + i) ^ key_order<DV>(row)) * 16) = v;
        }
      }
    }
  };
  // The block's values are in LDS, those out of sight as zeros. In sight of some rows only: an infinity
  // or NaN is 0 here, and given to the rows that see it at the end (add_odd_values).
  auto finish_v = [&](int b, int to, const Rows& r) {
    const bool seen = whole_block<kTileKeys>(a, t, blocks.key(b));
    const bool plain = seen && r.ok == 0xFFFFu;
    bool odd = false;
    if (FP8 || !plain) {
      if (!FP8) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wave's loads are in LDS
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int row = j * RP + rsub;
        const bool some = r.ok >> row & 1;
        uint32_t w[8];
        uint8_t* at[2];
        if constexpr (FP8) {
          widen<16, F16, true>((const uint32_t*)&vr[j], w);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            at[i] = s_v[to] + (16 * wave + row) * kRow + ((2 * v_chunk[j] + i) ^ value_order<DV>(row)) * 16;
        } else {
          at[0] = s_v[to] + 16 * wave * kRow + 1024 * j + 16 * lane;
          const u32x4 v = *(const u32x4*)at[0];
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] = v[i];
        }
        if (!plain) {
#pragma unroll
          for (int i = 0; i < CV / 2; ++i) {
            w[i] = some ? w[i] : 0;
            odd |= take_odd<F16>(w[i], !seen);
          }
        }
#pragma unroll
        for (int i = 0; i < CV / 8; ++i)
          *(u32x4*)at[i] = u32x4{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
      }
    }
    if (odd) s_odd = 1;
    if (lane == 0) ((uint16_t*)&s_ok[to])[wave] = (uint16_t)r.ok;
  };
  auto meet = [] {   // loads into LDS and stores to it are done, of all waves
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };

  // Whether all rows of this wave see all of a block. (A wave none of whose rows sees any of it goes
  // through it with the others: leaving the products out cost more registers than it saved time.)
  auto whole = [&](int key0) {
    return key0 + kTileKeys - 1 <= w_all && (key0 >= w_from || key0 + kTileKeys - 1 < keep);
  };
  auto key_frag = [&](int at, int u, int k) {   // operand of k-step k of the scores of half u
    return *(const u32x4*)(s_k[at] + (32 * u + n) * kRow + ((2 * k + hf) ^ key_order<DV>(n)) * 16);
  };
  const int v_row = (lane & 15) / 4, v_piece = 2 * (n / 16) + (lane & 3) / 2;
  auto value_frag = [&](int at, int k, int d) {   // of keys 16 k on, values 32 d on
    const uint8_t* v = s_v[at] + (16 * k + 4 * hf + v_row) * kRow +
                       ((4 * d + v_piece) ^ value_order<DV>(v_row)) * 16 + 8 * (lane & 1);
    const u32x2 lo = read_columns(v), hi = read_columns(v + 8 * kRow);
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  };
  auto raise = [&](float top) {
    top *= c;
    if (__any(top - m > kRaise<F16>)) {   // (m + kRaise would be rounded, past 2^27 by 8)
      top = fmaxf(top, wave_xor(top, 32));
      const float to = top - m > kRaise<F16> ? ceilf(top) - kBelow<F16> : m;   // by a row's own scores alone
      const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
    }
    return m == -INFINITY ? 0.f : -m;
  };

  // A step takes 32 keys, half a block: the next half's scores beside this one's weights, then the
  // weighted values. So the second half's keys are wanted with a block's values and the first half's
  // a step before them: of two buffers, block b writes the second half of b + 1 and the first half of
  // b + 2, which `low` waves load, over keys that were last read before the barrier.
  const bool low = wave < 2;
  Rows now = {0, 0, 0}, next = {0, 0, 0}, far = {0, 0, 0};
  if (b0 < b1) {
    now = checked(lookup(b0));
    load_k(b0, 0, now);
    load_v(b0, 0, now);
    next = lookup(b0 + 1);
    store_k(0);
    finish_v(b0, 0, now);
    next = checked(next);
    if (low && b0 + 1 < b1) {
      load_k(b0 + 1, 1, next);
      store_k(1);
    }
    far = lookup(b0 + 2);
  }
  meet();
  // Scores of the blocks' first and second halves: [i] of key 8 (i / 4) + 4 hf + i % 4 of the half.
  f32x16 s0, s1;
#pragma unroll
  for (int i = 0; i < 16; ++i) s0[i] = 0.f;
#pragma unroll
  for (int k = 0; k < NK; ++k) s0 = mma32<F16>(key_frag(0, 0, k), q[k], s0);
  meet();   // the first step loads over these keys
  auto step = [&](auto half, int key0, uint32_t ok, bool all, int at, const f32x16& in, f32x16& out) {
    constexpr int U = decltype(half)::value;
    float x[16];   // scores, then weights
    u32x4 p[2];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = in[i];
    // Selects of scalars, no branches: with a branch a mask, or a store into an element of a
    // vector, was compiled to code that left the first element as it was.
    if (!all) {
      const int key_l = key0 + 32 * U + 4 * hf;
      const int to_last = see_last - key_l, to_first = see_first - key_l, to_keep = keep - key_l;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = 8 * (i / 4) + i % 4;   // of key key_l + k
        const bool no = (k > to_last) | ((k < to_first) & (k >= to_keep));
        x[i] = no ? -INFINITY : x[i];
      }
    }
    if (ok != ~0u) {
      const uint32_t ok_l = ok >> 4 * hf;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = ok_l >> (8 * (i / 4) + i % 4) & 1 ? x[i] : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, x[i]);
    const float base = raise(top);
    auto weights = [&](int i) {   // of two keys
      x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], c, base));
      x[i + 1] = __builtin_amdgcn_exp2f(fmaf(x[i + 1], c, base));
      const uint32_t w = pack2<F16>(x[i], x[i + 1]);
      l = add2<F16>(w, l);
      asm("" : "+v"(l));   // here, not behind the loop's end: the weights would stay in registers
      p[i / 8][i % 8 / 2] = w;
    };
    // Each matrix instruction has weights to run beside it. (Behind the last block the scores are of
    // what lies in LDS, and are dropped.)
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = 0.f;
    constexpr int NV = 2 * ND, AHEAD = 2;
    u32x4 kf[AHEAD + 1], vf[AHEAD + 1];
    const int k_at = U ? at ^ 1 : at;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) kf[i] = key_frag(k_at, 1 - U, i);
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      if (i + AHEAD < NK) kf[(i + AHEAD) % (AHEAD + 1)] = key_frag(k_at, 1 - U, i + AHEAD);
      out = mma32<F16>(kf[i % (AHEAD + 1)], q[i], out);
      if constexpr (NK <= 8) {
#pragma unroll
        for (int e = 0; e < 8 / NK; ++e) weights(2 * (i * (8 / NK) + e));
      } else if (i % (NK / 8) == 0) {
        weights(2 * (i / (NK / 8)));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) vf[i] = value_frag(at, 2 * U + i / ND, i % ND);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int f = i + AHEAD;
      if (f < NV) vf[f % (AHEAD + 1)] = value_frag(at, 2 * U + f / ND, f % ND);
      o[i % ND] = mma32<F16>(vf[i % (AHEAD + 1)], p[i / ND], o[i % ND]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int b = b0; b < b1; ++b) {
    const int at = (b - b0) & 1;
    Rows last = checked(far);
    far = lookup(b + 3);
    const int kb = low ? b + 2 : b + 1;   // whose keys this wave loads
    if (kb < b1) {
      if (low) load_k(kb, at, last);
      else load_k(kb, at ^ 1, next);
    }
    if (b + 1 < b1) load_v(b + 1, at ^ 1, next);
    const int key0 = blocks.key(b);
    const uint64_t ok = s_ok[at];
    const bool all = whole(key0);
    step(std::integral_constant<int, 0>{}, key0, (uint32_t)ok, all, at, s0, s1);
    step(std::integral_constant<int, 1>{}, key0, (uint32_t)(ok >> 32), all, at, s1, s0);
    if (kb < b1) store_k(low ? at : at ^ 1);
    if (b + 1 < b1) finish_v(b + 1, at ^ 1, next);
    next = last;
    meet();
  }

  l += wave_xor(l, 32);
  const float vs = FP8 && a.cache.v_scale ? a.cache.v_scale[t.head] : 1.f;
  const float top = l != l ? fmaxf(m, 0.f) : m;   // scores of NaN alone leave m where it was
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int at_d = 32 * d + 8 * (i / 4) + 4 * hf;
      if (at_d >= D || !row_ok) continue;
      const float v[4] = {o[d][i] * vs, o[d][i + 1] * vs, o[d][i + 2] * vs, o[d][i + 3] * vs};
      store_row<F16, false, 4>(a, t, split, r, at_d, top, l, v);
    }
  if (s_odd) add_odd_values<F16, false>(a, t, blocks, b0, b1, split);
}

// The splits of a row meet: one workgroup a row. Each wave adds every fourth split's sums, several of
// them in flight at once, and the four meet in LDS; the order depends on the sizes alone.
// 32 heads of 128, 128 splits: 5.5 us (with a wave a row, one split after the other, the call took 239 us
// in place of 82).
constexpr int kMaxSplits = 256;
template <bool F16>
__global__ __launch_bounds__(kRowThreads) void k_attend_join(AttendCall a) {
  constexpr int NW = kRowThreads / kWave;
  __shared__ float weight[kMaxSplits];
  __shared__ f32x4 sums[NW][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  bool few = a.few;
  int head;
  int64_t token = a.block0 + blockIdx.y, row;
  if (a.both && a.splits == 1) {   // of the sequences with few rows alone: row r of one and a KV head
    const int r = blockIdx.x, kv = (int)(token % a.cache.n_heads), seq = (int)(token / a.cache.n_heads);
    few = true;
    row = token * kFewRows + r;
    const int lo = first_row(a.batch, seq), n = first_row(a.batch, seq + 1) - lo;
    if (n <= 0 || (int64_t)n * a.group > kFewRows || r >= n * a.group) return;
    token = lo + r / a.group;
    head = kv * a.group + r % a.group;
  } else {
    head = blockIdx.x;
    if (token < first_row(a.batch, 0) || token >= first_row(a.batch, a.batch.n_seq)) return;
    row = token * a.n_q_heads + head;
    if (a.both) {
      const int seq = wave_find(a.batch.n_seq, token, [&](int i) { return first_row(a.batch, i); });
      const int lo = first_row(a.batch, seq), hi = first_row(a.batch, seq + 1), kv = head / a.group;
      if (token < lo || token >= hi) return;
      few = (int64_t)(hi - lo) * a.group <= kFewRows;
      if (few) {
        if (a.splits_few == 1) return;   // written already
        row = ((int64_t)seq * a.cache.n_heads + kv) * kFewRows + (token - lo) * a.group + head - kv * a.group;
      }
    }
  }
  const int splits = few ? a.splits_few : a.splits;
  const AttendParts parts = few ? a.parts_few : a.parts;
  const int64_t all = parts.rows;
  typedef float f32x2 __attribute__((__vector_size__(8)));
  f32x2 st[kMaxSplits / kWave];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kWave; ++i) {
    const int s = i * kWave + lane;
    st[i] = s < splits ? *(const f32x2*)(parts.stats + 2 * (s * all + row)) : f32x2{-INFINITY, 0.f};
    top = fmaxf(top, st[i][0]);
  }
#pragma unroll
  for (int x = kWave / 2; x; x >>= 1) top = fmaxf(top, wave_xor(top, x));
  const float sink = a.sinks ? a.sinks[head] * kLog2e : -INFINITY;
  const float high = fmaxf(top, sink);
  float l = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / kWave; ++i) {
    const int s = i * kWave + lane;
    // a split with nothing in sight has m = -infinity, l = 0
    const float f = st[i][0] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(st[i][0] - high);
    l = fmaf(f, st[i][1], l);
    if (wave == 0 && s < splits) weight[s] = f;
  }
#pragma unroll
  for (int x = kWave / 2; x; x >>= 1) l += wave_xor(l, x);
  if (a.sinks) l += __builtin_amdgcn_exp2f(sink - high);
  __syncthreads();
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  const int d = 4 * lane;
  if (d < a.cache.D) {
    const float* part = parts.sums + row * a.cache.D + d;
#pragma unroll 8
    for (int s = wave; s < splits; s += NW) {
      const f32x4 v = *(const f32x4*)(part + s * all * a.cache.D);
      const float f = weight[s];
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(f, v[i], o[i]);
    }
  }
  sums[wave][lane] = o;
  __syncthreads();
  if (wave || d >= a.cache.D) return;
#pragma unroll
  for (int w = 1; w < NW; ++w) o += sums[w][lane];
  const bool none = top == -INFINITY;
  uint16_t* p = (uint16_t*)a.out.p + token * a.out.token + head * a.out.head + d;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = none ? 0.f : o[i] / l;
  *(u32x2*)p = u32x2{pack2<F16>(o[0], o[1]), pack2<F16>(o[2], o[3])};
}

// across workgroups for each of `count` tiles or rows, as many of these at a time as a launch takes.
template <typename K>
hipError_t launch_blocks(AttendCall a, int64_t across, int64_t count, K kernel, int threads,
                         hipStream_t stream) {
  // a launch holds fewer than 2^32 threads, a grid's second dimension fewer than 2^16 workgroups
  const int64_t most = min(max((int64_t(1) << 22) / across, (int64_t)1), (int64_t)kMaxGridY);
  for (int64_t b = 0; b < count; b += most) {
    a.block0 = b;
    hipLaunchKernelGGL(kernel, dim3((unsigned)across, (unsigned)min(count - b, most)), dim3(threads),
                       0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool F16, bool FP8, int DV>
hipError_t launch_depth(AttendCall a, hipStream_t stream) {
  hipError_t e = hipSuccess;
  const bool tiles = a.both || !a.few, rows = a.both || a.few;
  if (tiles) {
    a.tiles = (int64_t)a.batch.T * a.group / kTileRows + a.batch.n_seq;
    const int64_t across = (int64_t)a.cache.n_heads * a.splits;
    // a page's 16 rows have to be within 32-bit offsets of the first
    const bool near = max(a.cache.k_token, a.cache.v_token) < (int64_t(1) << 26);
    e = a.cache.page_size % 16 == 0 && near
            ? launch_blocks(a, across, a.tiles, k_attend_tiles<F16, FP8, DV, true>, kTileThreads, stream)
            : launch_blocks(a, across, a.tiles, k_attend_tiles<F16, FP8, DV, false>, kTileThreads, stream);
  }
  if (rows && e == hipSuccess) {
    a.tiles = a.both ? (int64_t)a.batch.n_seq * (kFewRows / kRowTile)
                     : (int64_t)a.batch.T * a.group / kRowTile + a.batch.n_seq;
    const int64_t across = (int64_t)a.cache.n_heads * a.splits_few;
    e = a.cache.page_size % 8 == 0
            ? launch_blocks(a, across, a.tiles, k_attend_rows<F16, FP8, DV, true>, kRowThreads, stream)
            : launch_blocks(a, across, a.tiles, k_attend_rows<F16, FP8, DV, false>, kRowThreads, stream);
  }
  const bool join = (tiles && a.splits > 1) || (rows && a.splits_few > 1);
  if (!join || e != hipSuccess) return e;
  if (a.both && a.splits == 1)
    return launch_blocks(a, kFewRows, (int64_t)a.batch.n_seq * a.cache.n_heads, k_attend_join<F16>,
                         kRowThreads, stream);
  return launch_blocks(a, a.n_q_heads, a.batch.T, k_attend_join<F16>, kRowThreads, stream);
}

template <bool F16, bool FP8>
hipError_t launch_type(const AttendCall& a, hipStream_t stream) {
  if (a.cache.D <= 64) return launch_depth<F16, FP8, 64>(a, stream);
  if (a.cache.D <= 128) return launch_depth<F16, FP8, 128>(a, stream);
  return launch_depth<F16, FP8, 256>(a, stream);
}

}  // namespace

AttendPlan attend_plan(const KvCacheView& c, const KvBatchView& b, int n_q_heads, int window,
                       int keep_first, int max_q, int max_len) {
  AttendPlan p;
  const int64_t group = n_q_heads / c.n_heads;
  // new tokens of the longest chunk; where that is not known, as if all rows were one's
  const int64_t chunk = max_q > 0 ? min(max_q, b.T) : b.T;
  p.few = chunk * group <= kFewRows;
  p.both = !p.few && b.n_seq > 1 && group <= kFewRows;   // one token's rows may be more than few
  int64_t keys = (int64_t)b.max_pages * c.page_size;
  if (max_len > 0) keys = min(keys, (int64_t)max_len);
  if (window) keys = min(keys, (int64_t)window + keep_first + chunk);
  const int64_t few_tiles = (p.both ? b.n_seq : (b.T * group / kRowTile + b.n_seq)) * c.n_heads;
  const int64_t tiles = (b.T * group / kTileRows + 1) * c.n_heads;
  // Workgroups for the CUs, with enough keys each: two blocks a wave, or eight tiles.
  // Few rows: two a CU (131072 keys of one sequence, 32 over 4 heads, us: 43 for 256, 36 for 512, 40 for
  // 1024; 2 sequences 27 for 512, 32 for 1024), and four where sequences of different lengths would leave
  // some CUs the long ones (8 over 8 heads 112 for 512, 100 for 1024; 32 of them 483, 330, 310 for 2048; 64
  // of them 635, 591, 592).
  // Many rows: the sums' way through memory costs more than a last round of tiles that is not full (2048
  // tokens behind 8192, 516 tiles: 386; in two splits 446).
  const int64_t few_groups = b.n_seq >= 8 ? 1024 : 512;
  p.splits_few = (int)max(min(min(few_groups / max(few_tiles, (int64_t)1), keys / 256),
                              (int64_t)kMaxSplits), (int64_t)1);
  p.splits = (int)max(min(min(1024 / max(tiles, (int64_t)1), keys / 512), (int64_t)kMaxSplits),
                      (int64_t)1);
  p.rows = (int64_t)b.T * n_q_heads;
  p.rows_few = p.both ? (int64_t)b.n_seq * c.n_heads * kFewRows : p.rows;
  return p;
}

hipError_t launch_attend(const AttendCall& a, hipStream_t stream) {
  const bool f16 = a.type == kFP16, fp8 = a.cache.type == kE4M3;
  if (f16) return fp8 ? launch_type<true, true>(a, stream) : launch_type<true, false>(a, stream);
  return fp8 ? launch_type<false, true>(a, stream) : launch_type<false, false>(a, stream);
}

}  // namespace moe
