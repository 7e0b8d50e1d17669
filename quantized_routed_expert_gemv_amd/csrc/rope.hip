// Rotary positions, and the append of keys and values to a paged cache with the rotation on the
// way. Pair i of a head turns by a = position * freq[i]:
//   (u, v) -> scale * (u cos a - v sin a, u sin a + v cos a)
// a is formed in fp64 and reduced to within half a turn there (at position 10^6 an fp32 angle is
// off by 0.03), then its sine and cosine are fp32. A token's angles are formed once, in LDS, and
// serve all of its heads. About three flops a value: copy rate bounds it, and latency for a few
// tokens. Rotation of 16384 rows of 40 heads of 128: 77 us, 4.4 TB/s (a copy here: 4.85); one row
// 2.5 us. Append of 8192 tokens, 32 + 2 * 4 heads of 128, into an 8-bit cache: 44 us, 3.6 TB/s; of four
// tokens, 64 + 2 * 8 heads of 64: 4.9 us.
#include "common.hpp"
#include "kernels.hpp"
#include "kv.hpp"

namespace moe {

namespace {

constexpr int kThreads = 256;

template <int N> struct Vals { float v[N]; };

__device__ __forceinline__ float to_f32(uint16_t v, int type) {
  return type == kFP16 ? fp16_to_f32(v) : bf16_to_f32(v);
}
__device__ __forceinline__ uint16_t from_f32(float v, int type) {
  return type == kFP16 ? __builtin_bit_cast(uint16_t, (_Float16)v)
                          : __builtin_bit_cast(uint16_t, (__bf16)v);   // RNE, NaN kept
}

template <int V, typename T>
__device__ __forceinline__ Vals<V> load(const T* p, int type) {
  Vals<V> r;
  if constexpr (sizeof(T) == 4) {
    if constexpr (V == 8) {
      const f32x4 a = *(const f32x4*)p, b = *(const f32x4*)(p + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[i] = a[i], r.v[4 + i] = b[i];
    } else {
      r.v[0] = *(const float*)p;
    }
  } else if constexpr (V == 8) {
    const u32x4 a = *(const u32x4*)p;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[2 * i] = to_f32(uint16_t(a[i]), type);
      r.v[2 * i + 1] = to_f32(uint16_t(a[i] >> 16), type);
    }
  } else {
    r.v[0] = to_f32(*p, type);
  }
  return r;
}

template <int V, typename T>
__device__ __forceinline__ void store(T* p, const Vals<V>& r, int type) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (V == 8) {
      *(f32x4*)p = f32x4{r.v[0], r.v[1], r.v[2], r.v[3]};
      *(f32x4*)(p + 4) = f32x4{r.v[4], r.v[5], r.v[6], r.v[7]};
    } else {
      *(float*)p = r.v[0];
    }
  } else if constexpr (V == 8) {
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a[i] = from_f32(r.v[2 * i], type) | (uint32_t)from_f32(r.v[2 * i + 1], type) << 16;
    *(u32x4*)p = a;
  } else {
    *p = from_f32(r.v[0], type);
  }
}

// The E4M3 code nearest to x / scale; past 448 it is 448, and NaN stays NaN.
__device__ __forceinline__ float over_scale(float x, float scale) {
  x /= scale;
  return x > 448.f ? 448.f : x < -448.f ? -448.f : x;
}

// V values to element `at` of a cache's plane.
template <int V>
__device__ __forceinline__ void store_cache(uint8_t* plane, int64_t at, const Vals<V>& r, int type,
                                            float scale) {
  if (type != kE4M3) {
    store<V>((uint16_t*)plane + at, r, type);
    return;
  }
  if constexpr (V == 8) {
    u32x2 q;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int w = 0;
      w = __builtin_amdgcn_cvt_pk_fp8_f32(over_scale(r.v[4 * i], scale),
                                          over_scale(r.v[4 * i + 1], scale), w, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(over_scale(r.v[4 * i + 2], scale),
                                          over_scale(r.v[4 * i + 3], scale), w, true);
      q[i] = (uint32_t)w;
    }
    *(u32x2*)(plane + at) = q;
  } else {
    plane[at] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(over_scale(r.v[0], scale), 0.f, 0, false);
  }
}

// Cosine and sine of position * freq.
__device__ __forceinline__ void angle(double freq, int position, float scale, float* c, float* s) {
  const double turns = (double)position * freq * 0.15915494309189533577;
  const float half_turns = 2.f * (float)(turns - rint(turns));
  sincospif(half_turns, s, c);
  *c *= scale;
  *s *= scale;
}

// Units of one head: pairs of V values and V values each for the turned part, then V values each.
template <int V>
__device__ __forceinline__ int units(int D, int dim) { return dim / (2 * V) + (D - dim) / V; }

// Loads unit u of a head, turns it where it is of the turned part, and hands it to `put` as
// (first value, values) once or twice.
template <int V, typename T, typename F>
__device__ __forceinline__ void unit(const T* x, int u, int type, const RopeView& r,
                                     const float* cs, F put) {
  const int n = r.dim / 2, turned = n / V;
  if (u >= turned) {
    const int d = r.dim + (u - turned) * V;
    put(d, load<V>(x + d, type));
    return;
  }
  const float* c = cs;
  const float* s = cs + n;
  if (r.interleaved) {
    const int d = 2 * u * V;
    Vals<V> a = load<V>(x + d, type), b = load<V>(x + d + V, type);
    auto turn = [&](float& p, float& q, int i) {
      const float t = p * c[i] - q * s[i];
      q = p * s[i] + q * c[i];
      p = t;
    };
    if constexpr (V == 1) {
      turn(a.v[0], b.v[0], u);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        turn(a.v[2 * i], a.v[2 * i + 1], u * V + i);
        turn(b.v[2 * i], b.v[2 * i + 1], u * V + V / 2 + i);
      }
    }
    put(d, a);
    put(d + V, b);
  } else {
    const int d = u * V;
    const Vals<V> a = load<V>(x + d, type), b = load<V>(x + n + d, type);
    Vals<V> p, q;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p.v[i] = a.v[i] * c[d + i] - b.v[i] * s[d + i];
      q.v[i] = a.v[i] * s[d + i] + b.v[i] * c[d + i];
    }
    put(d, p);
    put(n + d, q);
  }
}

// TK tokens a workgroup; T is the rows' element (uint16_t or float), V the values a thread moves at
// once: 8, or 1 where sizes, strides or addresses are not of 16 bytes. The units of a token's heads
// are shared out among the workgroups of the grid's second dimension, each of which forms the angles.
template <typename T, int V, int TK>
__global__ __launch_bounds__(kThreads) void k_rope(RopeCall a) {
  constexpr int kTokens = TK;
  extern __shared__ float cs[];   // [kTokens][2][dim / 2]
  const int64_t t0 = ((int64_t)a.block0 + blockIdx.x) * kTokens;
  const int nt = (int)min((int64_t)kTokens, a.T - t0);
  const int n = a.rope.dim / 2;
  for (int i = threadIdx.x; i < nt * n; i += kThreads) {
    const int t = i / n, j = i - t * n;
    angle(a.rope.freq[j], a.positions[t0 + t], a.rope.scale, &cs[2 * t * n + j],
          &cs[(2 * t + 1) * n + j]);
    if (a.inverse) cs[(2 * t + 1) * n + j] *= -1.f;
  }
  __syncthreads();
  const int per_head = units<V>(a.D, a.rope.dim), per_token = a.n_heads * per_head;
  const int first = blockIdx.y * kThreads + threadIdx.x, stride = gridDim.y * kThreads;
  for (int t = 0; t < nt; ++t) {
    const T* x = (const T*)a.x.p + (t0 + t) * a.x.token;
    T* out = (T*)a.out.p + (t0 + t) * a.out.token;
    for (int i = first; i < per_token; i += stride) {
      const int h = i / per_head;
      unit<V>(x + h * a.x.head, i - h * per_head, a.type, a.rope, cs + 2 * t * n,
              [&](int d, const Vals<V>& r) { store<V>(out + h * a.out.head + d, r, a.type); });
    }
  }
}

template <typename T, int V, int TK>
__global__ __launch_bounds__(kThreads) void k_append(AppendCall a) {
  constexpr int kTokens = TK;
  extern __shared__ float cs[];   // [kTokens][2][dim / 2]
  __shared__ int64_t place[kTokens][2];   // of the token's row in the k and v planes; < 0: none
  __shared__ int turn_by[kTokens];
  const int64_t t0 = ((int64_t)a.block0 + blockIdx.x) * kTokens;
  const int end = first_row(a.batch, a.batch.n_seq);
  const int nt = (int)min((int64_t)kTokens, end - t0);
  if (nt <= 0) return;
  const int wave = threadIdx.x / kWave;
  for (int t = wave; t < nt; t += kThreads / kWave) {   // one token a wave
    const int row = (int)t0 + t;
    const int b = wave_find(a.batch.n_seq, row, [&](int i) { return first_row(a.batch, i); });
    const int lo = first_row(a.batch, b), hi = first_row(a.batch, b + 1);
    const int64_t pos = (int64_t)a.batch.seq_len[b] - hi + row;
    int64_t kp = -1, vp = -1;
    if (row >= lo && row < hi && pos >= 0) {
      int in_page;
      const int p = page_of((uint32_t)pos, a.cache.page_size, a.cache.page_inv, &in_page);
      const int page = p < a.batch.max_pages ? a.batch.table[b * a.batch.table_stride + p] : -1;
      if (page >= 0 && page < a.cache.n_pages) {
        kp = page * a.cache.k_page + in_page * a.cache.k_token;
        vp = page * a.cache.v_page + in_page * a.cache.v_token;
      }
    }
    if ((threadIdx.x & (kWave - 1)) == 0) {
      place[t][0] = kp;
      place[t][1] = vp;
      turn_by[t] = a.positions ? a.positions[row] : (int)pos;
      if (kp < 0 && a.err) atomicOr(a.err, 1u);
    }
  }
  __syncthreads();
  const int n = a.rope.dim / 2;
  for (int i = threadIdx.x; i < nt * n; i += kThreads) {
    const int t = i / n, j = i - t * n;
    angle(a.rope.freq[j], turn_by[t], a.rope.scale, &cs[2 * t * n + j], &cs[(2 * t + 1) * n + j]);
  }
  __syncthreads();
  const int first = blockIdx.y * kThreads + threadIdx.x, stride = gridDim.y * kThreads;
  const int D = a.cache.D, Hkv = a.cache.n_heads;
  const int per_head = units<V>(D, a.rope.dim);
  const int n_q = a.q.p ? a.n_q_heads * per_head : 0, n_k = Hkv * per_head, n_v = Hkv * (D / V);
  for (int t = 0; t < nt; ++t) {
    const int64_t row = t0 + t;
    const int64_t kp = place[t][0], vp = place[t][1];
    const float* angles = cs + 2 * t * n;
    for (int i = first; i < n_q + n_k + n_v; i += stride) {
      if (i < n_q) {
        const int h = i / per_head;
        T* out = (T*)a.q_out.p + row * a.q_out.token + h * a.q_out.head;
        unit<V>((const T*)a.q.p + row * a.q.token + h * a.q.head, i - h * per_head, a.type, a.rope,
                angles, [&](int d, const Vals<V>& r) { store<V>(out + d, r, a.type); });
      } else if (kp < 0) {
        continue;
      } else if (i < n_q + n_k) {
        const int h = (i - n_q) / per_head;
        const float scale = a.cache.k_scale ? a.cache.k_scale[h] : 1.f;
        const int64_t at = kp + h * a.cache.k_head;
        unit<V>((const T*)a.k.p + row * a.k.token + h * a.k.head, i - n_q - h * per_head, a.type,
                a.rope, angles, [&](int d, const Vals<V>& r) {
                  store_cache<V>(a.cache.k, at + d, r, a.cache.type, scale);
                });
      } else {
        const int u = i - n_q - n_k, h = u / (D / V), d = (u - h * (D / V)) * V;
        const float scale = a.cache.v_scale ? a.cache.v_scale[h] : 1.f;
        store_cache<V>(a.cache.v, vp + h * a.cache.v_head + d,
                       load<V>((const T*)a.v.p + row * a.v.token + h * a.v.head + d, a.type),
                       a.cache.type, scale);
      }
    }
  }
}

bool vector_rows(const HeadsView& h, int size) {
  const int64_t mask = 16 / size - 1;
  return ((uintptr_t)h.p & 15) == 0 && (h.token & mask) == 0 && (h.head & mask) == 0;
}

// A launch holds fewer than 2^32 threads.
constexpr int kMaxBlocks = 1 << 21;

// `units`: of a token's heads. For up to 2048 tokens one a workgroup, and one unit a thread as far as
// eight workgroups go; else four a workgroup, one after the other, whose angles fill its threads. Rotation
// of 40 heads of 128, us: 64 tokens 3.3 against 7.1, 1024 6.4 against 8.3, 2048 9.9 against 11.4, 4096 16.7
// against 16.3; append to an 8-bit cache, 32 + 2 * 4 heads: 2048 tokens 17.0 against 19.1, 4096 28.8 against
// 22.8.
template <typename Call, typename K>
hipError_t launch_blocks(Call a, int64_t T, int64_t units, K few, K many, hipStream_t stream) {
  const bool small = T <= 2048;
  const int tokens = small ? 1 : 4;
  const int64_t blocks = (T + tokens - 1) / tokens;
  const unsigned across = small ? (unsigned)min((units + kThreads - 1) / kThreads, (int64_t)8) : 1u;
  const size_t lds = (size_t)tokens * a.rope.dim * sizeof(float);
  for (int64_t b = 0; b < blocks; b += kMaxBlocks) {
    a.block0 = (int)b;
    hipLaunchKernelGGL(small ? few : many, dim3((unsigned)min(blocks - b, (int64_t)kMaxBlocks), across),
                       dim3(kThreads), lds, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T, int V>
hipError_t launch_rope_t(const RopeCall& a, hipStream_t stream) {
  const int64_t per_head = a.rope.dim / (2 * V) + (a.D - a.rope.dim) / V;
  return launch_blocks(a, a.T, a.n_heads * per_head, k_rope<T, V, 1>, k_rope<T, V, 4>, stream);
}
template <typename T, int V>
hipError_t launch_append_t(const AppendCall& a, hipStream_t stream) {
  const int64_t per_head = a.rope.dim / (2 * V) + (a.cache.D - a.rope.dim) / V;
  const int64_t heads = (a.q.p ? a.n_q_heads : 0) + a.cache.n_heads;
  return launch_blocks(a, a.batch.T, heads * per_head + a.cache.n_heads * (a.cache.D / V),
                       k_append<T, V, 1>, k_append<T, V, 4>, stream);
}

}  // namespace

hipError_t launch_rope(const RopeCall& a, hipStream_t stream) {
  const bool f32 = a.type == kFP32;
  const int size = f32 ? 4 : 2;
  const bool wide = a.rope.dim % 16 == 0 && a.D % 8 == 0 && vector_rows(a.x, size) &&
                    vector_rows(a.out, size);
  if (f32) return wide ? launch_rope_t<float, 8>(a, stream) : launch_rope_t<float, 1>(a, stream);
  return wide ? launch_rope_t<uint16_t, 8>(a, stream) : launch_rope_t<uint16_t, 1>(a, stream);
}

hipError_t launch_append(const AppendCall& a, hipStream_t stream) {
  const bool f32 = a.type == kFP32;
  const int size = f32 ? 4 : 2;
  const bool wide = a.rope.dim % 16 == 0 && vector_rows(a.k, size) && vector_rows(a.v, size) &&
                    (!a.q.p || (vector_rows(a.q, size) && vector_rows(a.q_out, size)));
  if (f32) return wide ? launch_append_t<float, 8>(a, stream) : launch_append_t<float, 1>(a, stream);
  return wide ? launch_append_t<uint16_t, 8>(a, stream) : launch_append_t<uint16_t, 1>(a, stream);
}

}  // namespace moe
