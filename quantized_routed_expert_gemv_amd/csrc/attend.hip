// Attention of new tokens over a paged cache: with s_j = scale <q, k_j> over the keys in sight,
//   out = sum_j e^{s_j} v_j / (sum_j e^{s_j} + e^{sink})
// in one pass over the keys with a running maximum m and sum l: weights are 2^{s'_j - m} with
// s' = s log2 e, and m is raised only where a score passes it by 8, so weights stay below 2^8
// (exact scaling by a power of two changes no rounding) and the sums seldom have to be rescaled.
// m, l and the weighted sum are fp32; a weight is rounded to the queries' 16-bit type where it
// meets the values in a matrix instruction, which adds half a step of that type to each term.
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

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kRaise = 8.f;   // by how much a score passes the running maximum before it moves

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
__device__ __forceinline__ uint32_t pack2(float a, float b) {   // RNE, NaN kept
  if constexpr (F16) return __builtin_bit_cast(uint32_t, f16x2{(_Float16)a, (_Float16)b});
  else return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
template <bool F16>
__device__ __forceinline__ float value(uint32_t bits) {
  return F16 ? fp16_to_f32(uint16_t(bits)) : bf16_lo(bits);
}
// Two E4M3 codes (the low or the high half of v) as two values of the 16-bit type, exactly.
template <bool F16, bool HI>
__device__ __forceinline__ uint32_t widen2(uint32_t v) {
  if constexpr (F16)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(v, 1.f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.f, HI));
}
// Whether either half of a dword of 16-bit values is an infinity or NaN.
template <bool F16>
__device__ __forceinline__ bool not_finite(uint32_t v) {
  constexpr uint32_t e = F16 ? 0x7C00u : 0x7F80u;
  return (v & e) == e || (v >> 16 & e) == e;
}

// 2N bytes of a 16-bit cache, or N of an 8-bit one, as N values of the 16-bit type.
template <int N, bool F16, bool FP8>
__device__ __forceinline__ void load_row(const uint8_t* plane, int64_t at, uint32_t* w) {
  if constexpr (!FP8) {
    if constexpr (N == 8) {
      const u32x4 v = *(const u32x4*)(plane + 2 * at);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = v[i];
    } else {
      const u32x2 v = *(const u32x2*)(plane + 2 * at);
      w[0] = v[0], w[1] = v[1];
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint32_t v = ((const uint32_t*)(plane + at))[i];
      w[2 * i] = widen2<F16, false>(v);
      w[2 * i + 1] = widen2<F16, true>(v);
    }
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

// The first key in the window of position pos.
__device__ __forceinline__ int window_start(const AttendCall& a, int pos) {
  return a.window ? (int)max((int64_t)pos - a.window + 1, (int64_t)0) : 0;
}

// The x-th tile of R rows: sequence b's begin at floor(q_start[b] * group / R) + b, which leaves
// each sequence as many places as it can need.
template <int R>
__device__ __forceinline__ bool find_tile(const AttendCall& a, int64_t x, int head, Tile* t) {
  const KvBatchView& b = a.batch;
  const int seq = wave_find(b.n_seq, x, [&](int i) {
    return (int64_t)first_row(b, i) * a.group / R + i;
  });
  const int lo = first_row(b, seq), n = first_row(b, seq + 1) - lo;
  const int64_t row0 = (x - (int64_t)lo * a.group / R - seq) * R;
  const int64_t rows = (int64_t)n * a.group - row0;
  if (n <= 0 || row0 < 0 || rows <= 0) return false;
  const int64_t cap = (int64_t)b.max_pages * a.cache.page_size;
  const int len = max(b.seq_len[seq], 0);
  t->seq = seq;
  t->head = head;
  t->row0 = (int)row0;
  t->rows = (int)min(rows, (int64_t)R);
  t->token0 = lo;
  t->pos0 = len - n;
  const int first_tok = t->row0 / a.group, last_tok = (t->row0 + t->rows - 1) / a.group;
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

// Where a tile's sums go: out, or a split's part.
template <bool F16, int N>
__device__ __forceinline__ void store_row(const AttendCall& a, const Tile& t, int split, int r,
                                          int d, float m, float l, const float* o) {
  const int tok = (t.row0 + r) / a.group, g = t.row0 + r - tok * a.group;
  const int64_t token = t.token0 + tok;
  const int head = t.head * a.group + g;
  if (a.splits > 1) {
    const int64_t at = ((int64_t)split * a.batch.T + token) * a.n_q_heads + head;
    if (d == 0) {
      a.stats[2 * at] = m;
      a.stats[2 * at + 1] = l;
    }
#pragma unroll
    for (int i = 0; i < N; i += 4) *(f32x4*)(a.part + at * a.cache.D + d + i) = f32x4{
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

constexpr int kRowTile = 16;
constexpr int kRowThreads = 256;

// Few rows a sequence: the cache's bytes bound it. A tile is 16 rows, the columns of 16x16x32
// instructions, so nothing goes through LDS but the end: a lane's 16-byte loads of K rows are
// operands as they are, and its loads of eight V rows become V^T operands by 16-bit picks (one a
// dword). The four waves take every fourth block of 32 keys and join in LDS.
// Key of matrix row m of the block's product u: 8 (m / 4) + 4 u + m % 4, so that a lane's eight
// scores are those of eight neighbouring keys, 8 (lane / 16) on.
// P8: pages hold a multiple of 8 tokens, so such a run of keys is on one page.
template <bool F16, bool FP8, int DV, bool P8>
__global__ __launch_bounds__(kRowThreads) void k_attend_rows(AttendCall a) {
  constexpr int NW = kRowThreads / kWave;
  constexpr int E = DV >= 128 ? 8 : DV / 16, NH = DV / (16 * E), NK = DV / 32;
  constexpr int OS = DV + 4;
  __shared__ float so[NW][kRowTile][OS];
  __shared__ float sm[NW][kRowTile], sl[NW][kRowTile];
  __shared__ float sp[NW][kRowTile][33];
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const int n = lane & 15, g = lane >> 4;
  const int64_t id = a.block0 + blockIdx.x;
  const int split = (int)(id % a.splits);
  const int64_t th = id / a.splits;
  Tile t;
  if (!find_tile<kRowTile>(a, th / a.cache.n_heads, (int)(th % a.cache.n_heads), &t)) return;
  const Blocks<32> blocks(t);
  const int b0 = (int)((int64_t)blocks.count * split / a.splits);
  const int b1 = (int)((int64_t)blocks.count * (split + 1) / a.splits);
  const int D = a.cache.D;

  // this lane's query: the keys that it sees, and its row of q as an operand
  const int tok = (t.row0 + n) / a.group;
  const bool row_ok = n < t.rows;
  const int pos = t.pos0 + tok;
  const int see_last = !row_ok ? -1 : a.causal ? min(pos, t.end - 1) : t.end - 1;
  const int see_first = window_start(a, pos);
  const int keep = a.window ? a.keep_first : 0;
  float c = a.scale * kLog2e;
  if (FP8 && a.cache.k_scale) c *= a.cache.k_scale[t.head];
  const uint32_t flip = c < 0.f ? 0x80008000u : 0u;   // scores are scaled by a positive number
  c = fabsf(c) < 1e-37f ? 1e-37f : fabsf(c);
  u32x4 q[NK];
  {
    const uint16_t* p = (const uint16_t*)a.q.p + (t.token0 + tok) * a.q.token +
                        (t.head * a.group + t.row0 + n - tok * a.group) * a.q.head;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const int d = 32 * k + 8 * g;
      q[k] = u32x4{0, 0, 0, 0};
      if (row_ok && d < D) q[k] = *(const u32x4*)(p + d) ^ flip;
    }
  }
  f32x4 o[NH][E];
#pragma unroll
  for (int h = 0; h < NH; ++h)
#pragma unroll
    for (int i = 0; i < E; ++i) o[h][i] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, l = 0.f;

  for (int b = b0 + wave; b < b1; b += NW) {
    const int key0 = blocks.key(b);
    u32x4 kf[2][NK];
    uint32_t vf[8][NH][E / 2];
    uint32_t v_ok = 0;   // of this lane's eight keys, those whose values are read
    auto load_k = [&](int u, const KeyRow& r) {
#pragma unroll
      for (int k = 0; k < NK; ++k) {
        const int d = 32 * k + 8 * g;
        load_row<8, F16, FP8>(a.cache.k, r.k + (d < D ? d : 0), (uint32_t*)&kf[u][k]);
        if (d >= D) kf[u][k] = u32x4{0, 0, 0, 0};
      }
    };
    auto load_v = [&](int j, int64_t at) {
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const int d = 16 * E * h + E * n;
        load_row<E, F16, FP8>(a.cache.v, at + (d < D ? d : 0), vf[j][h]);
      }
    };
    if constexpr (P8) {
      const KeyRow rk = key_row<8>(a, t, key0 + 8 * (n >> 2));
#pragma unroll
      for (int u = 0; u < 2; ++u)
        load_k(u, {rk.k + (rk.ok ? (4 * u + (n & 3)) * a.cache.k_token : 0), 0, rk.ok});
      const KeyRow rv = key_row<8>(a, t, key0 + 8 * g);
#pragma unroll
      for (int j = 0; j < 8; ++j) load_v(j, rv.v + (rv.ok ? j * a.cache.v_token : 0));
      v_ok = rv.ok ? 0xFFu : 0u;
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) load_k(u, key_row<1>(a, t, key0 + 8 * (n >> 2) + 4 * u + (n & 3)));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const KeyRow rv = key_row<1>(a, t, key0 + 8 * g + j);
        load_v(j, rv.v);
        v_ok |= (uint32_t)rv.ok << j;
      }
    }
    f32x4 s[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s[u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < NK; ++k) s[u] = mma16<F16>(kf[u][k], q[k], s[u]);
    }
    // lane (n, g): s[u][i] is the score of query n and key key0 + 8 g + 4 u + i
    const bool whole = key0 + 31 <= t.last_of_first &&
                       (key0 >= t.first_of_last || key0 + 31 < keep) && __all(v_ok == 0xFFu);
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int key = key0 + 8 * g + j;
        const bool in = key <= see_last && (key >= see_first || key < keep) && (v_ok >> j & 1);
        if (!in) s[j / 4][j % 4] = -INFINITY;
        // values behind the end, before the window, or on no page: anything may stand there
        if (!(key < t.end && (key >= t.first || key < t.kept) && (v_ok >> j & 1)))
#pragma unroll
          for (int h = 0; h < NH; ++h)
#pragma unroll
            for (int i = 0; i < E / 2; ++i) vf[j][h][i] = 0;
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int j = 1; j < 8; ++j) top = fmaxf(top, s[j / 4][j % 4]);
    top *= c;
    if (__any(top > m + kRaise)) {
      top = fmaxf(top, wave_xor(top, 16));
      top = fmaxf(top, wave_xor(top, 32));
      const float to = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.f : exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int i = 0; i < E; ++i) o[h][i] *= f;
    }
    const float base = m == -INFINITY ? 0.f : m;
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      p[j] = exp2f(fmaf(s[j / 4][j % 4], c, -base));
      l += p[j];
    }
    const u32x4 pf = {pack2<F16>(p[0], p[1]), pack2<F16>(p[2], p[3]), pack2<F16>(p[4], p[5]),
                      pack2<F16>(p[6], p[7])};
    bool odd = false;
    if (!whole) {   // a value that some rows see and others do not must not be 0 * infinity there
      bool bad = false;
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int i = 0; i < E / 2; ++i) bad |= not_finite<F16>(vf[j][h][i]);
      odd = __any(bad);
    }
    if (!odd) {
#pragma unroll
      for (int h = 0; h < NH; ++h)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          u32x4 vt;
          const uint32_t sel = i & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            vt[j] = __builtin_amdgcn_perm(vf[2 * j + 1][h][i / 2], vf[2 * j][h][i / 2], sel);
          o[h][i] = mma16<F16>(vt, pf, o[h][i]);
        }
    } else {   // key by key, each row with the keys that it sees
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float r = value<F16>(pf[j / 2] >> 16 * (j & 1));
        sp[wave][n][8 * g + j] = s[j / 4][j % 4] == -INFINITY ? -1.f : r;
      }
      __builtin_amdgcn_wave_barrier();
      for (int k = 0; k < 32; ++k) {
        const KeyRow r = key_row<1>(a, t, key0 + k);
        const float w = sp[wave][n][k];
#pragma unroll
        for (int h = 0; h < NH; ++h)
#pragma unroll
          for (int i = 0; i < E; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int d = 16 * E * h + E * (4 * g + e) + i;
              const float v = plane_value(a.cache.v, r.v + (d < D ? d : 0), a.cache.type);
              if (!(w < 0.f) && r.ok) o[h][i][e] = fmaf(w, v, o[h][i][e]);
            }
      }
    }
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
  if (r >= t.rows) return;
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
    if (d >= D) continue;
    float v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      v[i] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v[i] = fmaf(f[w], so[w][r][d + i], v[i]);
      v[i] *= vs;
    }
    store_row<F16, E>(a, t, split, r, d, sum != sum ? fmaxf(top, 0.f) : top, sum, v);
  }
}

// The splits of a row meet: one wave a row, in the splits' order.
template <bool F16>
__global__ __launch_bounds__(kRowThreads) void k_attend_join(AttendCall a) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t row = (a.block0 + blockIdx.x) * (kRowThreads / kWave) + threadIdx.x / kWave;
  const int64_t token = row / a.n_q_heads;
  if (token < first_row(a.batch, 0) || token >= first_row(a.batch, a.batch.n_seq)) return;
  const int head = (int)(row - token * a.n_q_heads);
  const int64_t all = (int64_t)a.batch.T * a.n_q_heads;
  float top = -INFINITY;
  for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.stats[2 * (s * all + row)]);
  const float sink = a.sinks ? a.sinks[head] * kLog2e : -INFINITY;
  const float high = fmaxf(top, sink);
  float l = a.sinks ? exp2f(sink - high) : 0.f;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  const int d = 4 * lane;
  for (int s = 0; s < a.splits; ++s) {
    const float m = a.stats[2 * (s * all + row)];
    if (m == -INFINITY) continue;   // nothing in sight there
    const float f = exp2f(m - high);
    l = fmaf(f, a.stats[2 * (s * all + row) + 1], l);
    if (d < a.cache.D) {
      const f32x4 v = *(const f32x4*)(a.part + (s * all + row) * a.cache.D + d);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = fmaf(f, v[i], o[i]);
    }
  }
  if (d >= a.cache.D) return;
  const bool none = top == -INFINITY;
  uint16_t* p = (uint16_t*)a.out.p + token * a.out.token + head * a.out.head + d;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = none ? 0.f : o[i] / l;
  *(u32x2*)p = u32x2{pack2<F16>(o[0], o[1]), pack2<F16>(o[2], o[3])};
}

constexpr int64_t kMaxBlocks = 1 << 22;   // a launch holds fewer than 2^32 threads

template <typename K>
hipError_t launch_blocks(AttendCall a, int64_t blocks, K kernel, int threads, hipStream_t stream) {
  for (int64_t b = 0; b < blocks; b += kMaxBlocks) {
    a.block0 = b;
    hipLaunchKernelGGL(kernel, dim3((unsigned)min(blocks - b, kMaxBlocks)), dim3(threads), 0,
                       stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <bool F16, bool FP8, int DV>
hipError_t launch_rows(const AttendCall& a, hipStream_t stream) {
  const int64_t tiles = (int64_t)a.batch.T * a.group / kRowTile + a.batch.n_seq;
  const int64_t blocks = tiles * a.cache.n_heads * a.splits;
  if (a.cache.page_size % 8 == 0)
    return launch_blocks(a, blocks, k_attend_rows<F16, FP8, DV, true>, kRowThreads, stream);
  return launch_blocks(a, blocks, k_attend_rows<F16, FP8, DV, false>, kRowThreads, stream);
}

template <bool F16, bool FP8>
hipError_t launch_depth(const AttendCall& a, hipStream_t stream) {
  if (a.cache.D <= 64) return launch_rows<F16, FP8, 64>(a, stream);
  if (a.cache.D <= 128) return launch_rows<F16, FP8, 128>(a, stream);
  return launch_rows<F16, FP8, 256>(a, stream);
}

}  // namespace

int attend_splits(const KvCacheView& c, const KvBatchView& b, int n_q_heads, int window,
                  int keep_first, int max_q, int max_len) {
  const int64_t group = n_q_heads / c.n_heads;
  const int64_t tiles = ((int64_t)b.T * group / kRowTile + b.n_seq) * c.n_heads;
  int64_t keys = (int64_t)b.max_pages * c.page_size;
  if (max_len > 0) keys = min(keys, (int64_t)max_len);
  if (window) keys = min(keys, (int64_t)window + keep_first + max(max_q, 1));
  const int64_t want = 1024 / max(tiles, (int64_t)1);   // four workgroups a CU
  return (int)max(min(want, keys / 256), (int64_t)1);   // of two blocks a wave at least
}

hipError_t launch_attend(const AttendCall& a, hipStream_t stream) {
  const bool f16 = a.type == kFP16, fp8 = a.cache.type == kE4M3;
  const hipError_t e = f16 ? (fp8 ? launch_depth<true, true>(a, stream) : launch_depth<true, false>(a, stream))
                           : (fp8 ? launch_depth<false, true>(a, stream)
                                  : launch_depth<false, false>(a, stream));
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t rows = (int64_t)a.batch.T * a.n_q_heads, per = kRowThreads / kWave;
  return f16 ? launch_blocks(a, (rows + per - 1) / per, k_attend_join<true>, kRowThreads, stream)
             : launch_blocks(a, (rows + per - 1) / per, k_attend_join<false>, kRowThreads, stream);
}

}  // namespace moe
