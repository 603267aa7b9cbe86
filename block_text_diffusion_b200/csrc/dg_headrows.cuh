// RMSNorm of query and key heads with the position rotation, into token
// buffers or straight into the pages of a cache.
//
//   y = x / sqrt(mean(x^2) + eps) * gain            (each head, if the norm is on)
//   (a, b) = pair j of y  ->  amplitude (a cos t - b sin t, b cos t + a sin t),
//   t = position * inv_freq[j]                       (the first rot_dim components)
//
// Angles: position * inv_freq reaches 1e5 radians and more in a long context,
// where binary32 has lost the phase.  The product is formed in fp64 in units
// of a turn, its whole turns are dropped there, and sincospi takes the
// remainder in [-1/2, 1/2] turns in fp32: the sine and cosine are good to
// fp32 rounding at every position.
//
// Everything is read once and written once, in fp32 between; one rounding.
#pragma once
#include "dg_paged.cuh"

struct HeadRows {
  void* data;
  long long ts, hs;   // token and head strides, elements
};

struct HeadRowsArgs {
  int n_tokens, n_q, n_k, n_v, head_dim;   // heads of each kind (n_v: copied values, append only)
  HeadRows q, qo, k, ko, v;
  const int* positions;
  // rotation
  const double* inv_freq;
  int rot_dim, interleaved;
  float amplitude;
  // norm
  int norm;
  float eps;
  const void* q_gain;
  const void* k_gain;
  // append: the pages take the keys and values instead of ko
  int paged;
  void *k_pages, *v_pages;   // [n_pages][n_k][page_size][head_dim]
  PagedBatch b;
};

// Where token t goes: its position, and for an append its slot.
struct TokenSpot {
  int pos;
  long long page;   // page id, -1: not stored
  int off;          // offset in the page
  bool live;        // false: the row belongs to no sequence
};

// The sequence of row t: the number of entries cu_q[1 ..] that are <= t.  The
// whole warp searches, 32 pivots a step, so 1024 sequences take two dependent
// reads where a binary search takes ten.
__device__ __forceinline__ int seq_of_row(const int* __restrict__ cu, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seqs;   // the answer is lo + (entries of cu[1 + lo .. 1 + lo + n) that are <= t)
  while (n > 32) {
    const int step = (n + 31) / 32;
    const int i = min((lane + 1) * step, n);   // last entry of the lane's part
    const unsigned le = __ballot_sync(0xffffffffu, cu[lo + i] <= t);
    const int full = __popc(le);               // parts that lie wholly at or before t
    const int done = min(full * step, n);
    lo += done;
    n = min(step, n - done);
  }
  const unsigned le = __ballot_sync(0xffffffffu, lane < n && cu[1 + lo + min(lane, n - 1)] <= t);
  return lo + __popc(le);
}

__device__ __forceinline__ TokenSpot token_spot(const HeadRowsArgs& a, int t) {
  TokenSpot s;
  s.page = -1;
  s.off = 0;
  s.live = true;
  if (!a.paged) {
    s.pos = a.positions ? a.positions[t] : 0;
    return s;
  }
  s.pos = 0;
  const PagedBatch& b = a.b;
  const int i = b.n_seqs > 0 ? seq_of_row(b.cu_q, b.n_seqs, t) : 0;
  if (i >= b.n_seqs || t < b.cu_q[0]) {
    s.live = false;
    return s;
  }
  const PagedSeq q = paged_seq(b, i);
  const int own = q.kv - q.nq + (t - q.q0);
  s.pos = b.prefix_len + own;
  // own < kv <= max_pages * page_size, so the table entry exists
  if (own >= 0 && own < q.kv) {
    const int page = b.table[(long long)i * b.table_stride + (own >> b.page_shift)];
    if (page >= 0 && page < b.n_pages) {
      s.page = page;
      s.off = own & ((1 << b.page_shift) - 1);
    }
  }
  if (s.page < 0) dev_error(b.status, kStatusState);
  return s;
}

__device__ __forceinline__ void turn_sincos(int pos, double inv_freq, float amplitude, float& c, float& s) {
  const double turns = (double)pos * (inv_freq * 0.15915494309189533577);   // 1 / (2 pi)
  const float r = (float)(turns - rint(turns));
  sincospif(2.0f * r, &s, &c);
  c *= amplitude;
  s *= amplitude;
}

// Any head_dim, stride and alignment: one warp per head, a lane takes the
// pairs lane, lane + 32, ...
constexpr int kHeadPairs = 4;   // head_dim <= 256: at most 4 pairs a lane

template <typename T>
__global__ void __launch_bounds__(256) k_head_rows_any(HeadRowsArgs a) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int heads = a.n_q + a.n_k + a.n_v;
  const long long n = (long long)a.n_tokens * heads;
  const int hd = a.head_dim, half = hd / 2, rp = a.rot_dim / 2;
  for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < n; w += (long long)gridDim.x * 8) {
    const int t = (int)(w / heads);
    int h = (int)(w % heads);
    const TokenSpot spot = token_spot(a, t);
    if (!spot.live) continue;
    const int kind = h < a.n_q ? 0 : h < a.n_q + a.n_k ? 1 : 2;
    h -= kind == 0 ? 0 : kind == 1 ? a.n_q : a.n_q + a.n_k;
    const HeadRows in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    const HeadRows out = kind == 0 ? a.qo : a.ko;
    const T* src = (const T*)in.data + (long long)t * in.ts + (long long)h * in.hs;
    T* dst;
    if (kind == 0 || !a.paged) {
      dst = (T*)out.data + (long long)t * out.ts + (long long)h * out.hs;
    } else {
      if (spot.page < 0) continue;
      dst = (T*)(kind == 1 ? a.k_pages : a.v_pages) +
            (((spot.page * a.n_k + h) << a.b.page_shift) + spot.off) * hd;
    }
    int e0[kHeadPairs], e1[kHeadPairs];
    float x[kHeadPairs], y[kHeadPairs];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kHeadPairs; ++i) {
      const int p = lane + 32 * i;
      const bool turn = p < rp;
      e0[i] = !turn || a.interleaved ? 2 * p : p;   // past the rotated part the pairs are neighbours
      e1[i] = !turn || a.interleaved ? 2 * p + 1 : p + rp;
      x[i] = p < half ? to_f(src[e0[i]]) : 0.0f;
      y[i] = p < half ? to_f(src[e1[i]]) : 0.0f;
      ss += x[i] * x[i] + y[i] * y[i];
    }
    const bool work = kind < 2;
    const T* gain = (const T*)(kind == 0 ? a.q_gain : a.k_gain);
    float r = 1.0f;
    if (a.norm && work) r = rsqrtf(warp_sum(ss) / (float)hd + a.eps);
#pragma unroll
    for (int i = 0; i < kHeadPairs; ++i) {
      const int p = lane + 32 * i;
      if (p >= half) continue;
      if (!work) {   // values move as they are
        dst[e0[i]] = src[e0[i]];
        dst[e1[i]] = src[e1[i]];
        continue;
      }
      if (a.norm) {
        x[i] *= r * (gain ? to_f(gain[e0[i]]) : 1.0f);
        y[i] *= r * (gain ? to_f(gain[e1[i]]) : 1.0f);
      }
      if (p < rp) {
        float c, s;
        turn_sincos(spot.pos, a.inv_freq[p], a.amplitude, c, s);
        const float u = x[i] * c - y[i] * s, v = y[i] * c + x[i] * s;
        x[i] = u;
        y[i] = v;
      }
      dst[e0[i]] = from_f<T>(x[i]);
      dst[e1[i]] = from_f<T>(y[i]);
    }
  }
}

// Eight bf16 or four fp32 values of a 16-byte chunk, as floats and back.
template <typename T> struct Chunk;
template <> struct Chunk<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};
template <> struct Chunk<bf16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Whole 16-byte chunks: a lane holds two chunks of a head, and in the half
// layout the second one holds the partners of the first, so a rotation needs
// no exchange between lanes.  head_dim / (2 * chunk) lanes (a power of two)
// share a head; a warp takes `kGroups` groups of 32 / lanes heads of one token,
// computes the token's sines and cosines once and has every load of its heads
// in flight before it needs the first.
template <typename T, int kGroups>
__global__ void __launch_bounds__(256) k_head_rows(HeadRowsArgs a, int lph_shift, int warps_per_token) {
  constexpr int N = Chunk<T>::kN;
  __shared__ __align__(16) float s_cos[8][128], s_sin[8][128];
  pdl_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 8 + warp;
  const int t = (int)(w / warps_per_token);
  if (t >= a.n_tokens) return;
  const int lph = 1 << lph_shift, hpw = 32 >> lph_shift;   // lanes a head, heads a group
  const int j = lane & (lph - 1), sub = lane >> lph_shift;
  const int gq = (a.n_q + hpw - 1) / hpw, gk = (a.n_k + hpw - 1) / hpw, gv = (a.n_v + hpw - 1) / hpw;
  const int g0 = (int)(w % warps_per_token) * kGroups;

  // chunks of the lane; rotated chunks and their partners first
  const int rp = a.rot_dim / 2, rc = rp / N;          // rotated pairs, chunks of them (half layout)
  int ca = j, cb = j + lph;
  bool turn_a, turn_b;
  if (a.interleaved) {
    turn_a = ca * N < a.rot_dim;
    turn_b = cb * N < a.rot_dim;
  } else {
    turn_a = turn_b = j < rc;
    cb = j + rc;
    if (!turn_a) {
      ca = j + rc;
      cb = ca + (lph - rc);
    }
  }

  uint4 xa[kGroups] = {}, xb[kGroups] = {};
  int kind[kGroups], head[kGroups];
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int g = g0 + i;
    kind[i] = g < gq ? 0 : g < gq + gk ? 1 : g < gq + gk + gv ? 2 : 3;
    head[i] = (g - (kind[i] == 0 ? 0 : kind[i] == 1 ? gq : gq + gk)) * hpw + sub;
    if (kind[i] == 3 || head[i] >= (kind[i] == 0 ? a.n_q : a.n_k)) head[i] = -1;
    if (head[i] >= 0) {
      const HeadRows in = kind[i] == 0 ? a.q : kind[i] == 1 ? a.k : a.v;
      const uint4* src = reinterpret_cast<const uint4*>((const T*)in.data + (long long)t * in.ts +
                                                        (long long)head[i] * in.hs);
      xa[i] = src[ca];
      xb[i] = src[cb];
    }
  }
  const TokenSpot spot = token_spot(a, t);
  if (!spot.live) return;
  float c[N], s[N];
  if (rp > 0 && g0 < gq + gk) {
    for (int p = lane; p < rp; p += 32)
      turn_sincos(spot.pos, a.inv_freq[p], a.amplitude, s_cos[warp][p], s_sin[warp][p]);
    __syncwarp();
    const int pa = a.interleaved ? ca * (N / 2) : j * N, pb = a.interleaved ? cb * (N / 2) : j * N + N / 2;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool on = i < N / 2 ? turn_a : turn_b;
      const int p = i < N / 2 ? pa + i : pb + i - N / 2;
      c[i] = on ? s_cos[warp][p] : 1.0f;
      s[i] = on ? s_sin[warp][p] : 0.0f;
    }
  }
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    if (kind[i] == 3) break;
    T* dst = nullptr;
    if (head[i] >= 0) {
      if (kind[i] == 0 || !a.paged) {
        const HeadRows out = kind[i] == 0 ? a.qo : a.ko;
        dst = (T*)out.data + (long long)t * out.ts + (long long)head[i] * out.hs;
      } else if (spot.page >= 0) {
        dst = (T*)(kind[i] == 1 ? a.k_pages : a.v_pages) +
              (((spot.page * a.n_k + head[i]) << a.b.page_shift) + spot.off) * a.head_dim;
      }
    }
    uint4 oa = xa[i], ob = xb[i];
    if (kind[i] < 2) {
      float x[N], y[N];
      Chunk<T>::unpack(xa[i], x);
      Chunk<T>::unpack(xb[i], y);
      if (a.norm) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < N; ++e) ss += x[e] * x[e] + y[e] * y[e];
        for (int o = lph >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss / (float)a.head_dim + a.eps);
        const uint4* gain = reinterpret_cast<const uint4*>(kind[i] == 0 ? a.q_gain : a.k_gain);
        if (gain) {
          float ga[N], gb[N];
          Chunk<T>::unpack(gain[ca], ga);
          Chunk<T>::unpack(gain[cb], gb);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            x[e] *= r * ga[e];
            y[e] *= r * gb[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            x[e] *= r;
            y[e] *= r;
          }
        }
      }
      if (rp > 0) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            if (turn_a) {
              const float u = x[2 * e], v = x[2 * e + 1];
              x[2 * e] = u * c[e] - v * s[e];
              x[2 * e + 1] = v * c[e] + u * s[e];
            }
            if (turn_b) {
              const float u = y[2 * e], v = y[2 * e + 1];
              y[2 * e] = u * c[N / 2 + e] - v * s[N / 2 + e];
              y[2 * e + 1] = v * c[N / 2 + e] + u * s[N / 2 + e];
            }
          }
        } else if (turn_a) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float u = x[e], v = y[e];
            x[e] = u * c[e] - v * s[e];
            y[e] = v * c[e] + u * s[e];
          }
        }
      }
      oa = Chunk<T>::pack(x);
      ob = Chunk<T>::pack(y);
    }
    if (dst) {
      reinterpret_cast<uint4*>(dst)[ca] = oa;
      reinterpret_cast<uint4*>(dst)[cb] = ob;
    }
  }
}
