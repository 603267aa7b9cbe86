// RMSNorm of query and key heads with the position rotation, into token
// buffers or straight into the pages of a cache.
//
//   y = x / sqrt(mean(x^2) + eps) * gain            (each head, if the norm is on)
//   (a, b) = pair j of y  ->  amplitude (a cos t - b sin t, b cos t + a sin t),
//   t = position * inv_freq[j]                       (the first rot_dim components)
//
// Angles: position * inv_freq reaches 1e5 radians and more in a long context,
// where binary32 has lost the phase, and at the ends of int32 a product rounded
// to fp64 is off by 5e-7.  So the product is formed in units of a turn as a sum
// of two fp64 values (the rounding of 1 / (2 pi), of the frequency and of the
// product are kept), its whole turns are dropped, and sincospi takes the
// remainder in [-1/2, 1/2] turns in fp32: the sine and cosine are good to fp32
// rounding (4 units of 2^-24) at every position.
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
  float inv_dim;                           // 1 / head_dim
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
  const int end = b.cu_q[i + 1], kv = b.kv_lens[i];
  paged_seq(b, b.cu_q[i], end, kv);   // (reports lengths and offsets out of range)
  // The token's place by the lengths as they are, not brought into range: one
  // that lies past the table has no slot, and must not take an earlier token's.
  const long long own = (long long)kv - end + t;
  s.pos = (int)(b.prefix_len + own);
  // (a row past its sequence's end, by offsets that decrease, has none either)
  if (own >= 0 && own < lmin(kv, (long long)b.max_pages << b.page_shift)) {
    const int page = b.table[(long long)i * b.table_stride + (own >> b.page_shift)];
    if (page >= 0 && page < b.n_pages) {
      s.page = page;
      s.off = (int)own & ((1 << b.page_shift) - 1);
    }
  }
  if (s.page < 0) paged_error(b, kStatusState);
  return s;
}

__device__ __forceinline__ void turn_sincos(int pos, double inv_freq, float amplitude, float& c, float& s) {
  constexpr double kTurn = 0.15915494309189533577, kTurnLo = -9.839338337591243e-18;   // 1 / (2 pi), and what that leaves
  // (products by name: one that the compiler fused into the difference below
  // would count its low part twice)
  const double f = __dmul_rn(inv_freq, kTurn), f_lo = fma(inv_freq, kTurn, -f) + inv_freq * kTurnLo;
  const double turns = __dmul_rn(pos, f), turns_lo = fma((double)pos, f, -turns) + pos * f_lo;
  const float r = (float)((turns - rint(turns)) + turns_lo);
  sincospif(2.0f * r, &s, &c);
  c *= amplitude;
  s *= amplitude;
}

// Any head_dim, stride and alignment: one warp per head, a lane takes the
// pairs lane, lane + 32, ...  One value a load, and the angles of a token once
// for every head: 8192 tokens of 24 bf16 heads of 96 take 93 us, of 128 with 24
// components turned 87, where the kernel of whole chunks takes 20 for 128.
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

// Two binary32 operations in one instruction (sm_100).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
      "mov.b64 {%0, %1}, z;\n\t}" : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

// Whole 16-byte chunks: a lane holds two chunks of a head, and in the half
// layout the second one holds the partners of the first, so a rotation needs
// no exchange between lanes.  head_dim / (2 * chunk) lanes (a power of two)
// share a head, a warp takes 32 / lanes heads (a group) at once and kGroups
// groups of one kind (a batch) with all their loads in flight.
//
// With u, v a pair, gains gu, gv and r = 1 / rms:
//   u' = r (u gu c - v gv s),   v' = r (v gv c + u gu s);
// the four products of gain and sine or cosine belong to the lane and the
// token, not to the head, so they are formed once a batch, and two pairs go
// through one packed instruction.
//
// A block is one warp: nothing is shared between warps, and a slot is free as
// soon as its warp ends, where the block of 8 waited for its last one (26B
// heads: 32 canvases of 256 tokens 28.7 to 26.6 us, an append of 16384 prompt
// tokens 61.4 to 55.3, of 64 single tokens 8.2 to 6.7; blocks of 4 and 2 lie
// between).  What comes from memory without the position (frequencies, gains)
// is asked for before the sequence is looked up, so the chain of dependent
// loads is the batch's alone.
//
// Many tokens: 4.6 TB/s (101 MB, 22.0 us among others) and 5.3 (268 MB, 50.7 us),
// bound by the latency of the loads: 114 registers leave 16 to 17 warps an SM,
// and their 1300 or so instructions fill under half of the issue slots.  Few: the
// launch and two dependent reads (3.1 to 3.6 us).
template <typename T, int kGroups, bool kInter>
__global__ void __launch_bounds__(32, 16) k_head_rows(const __grid_constant__ HeadRowsArgs a, int lph_shift,
                                                      unsigned warps_per_token, int batches_per_warp) {
  constexpr int N = Chunk<T>::kN;
  __shared__ __align__(16) float s_cos[128], s_sin[128];
  pdl_enter();
  const int lane = threadIdx.x;
  const unsigned w = blockIdx.x;
  const int t = (int)(warps_per_token == 1 ? w : w / warps_per_token);
  if (t >= a.n_tokens) return;
  const int lph = 1 << lph_shift, hpw = 32 >> lph_shift;   // lanes a head, heads a group
  const int j = lane & (lph - 1), sub = lane >> lph_shift;
  const int batch_shift = 5 - lph_shift + (kGroups == 4 ? 2 : 0), per_batch = 1 << batch_shift;   // heads
  const int bq = (a.n_q + per_batch - 1) >> batch_shift, bk = (a.n_k + per_batch - 1) >> batch_shift,
            bv = (a.n_v + per_batch - 1) >> batch_shift;
  const int b0 = (int)(warps_per_token == 1 ? 0 : w - t * warps_per_token) * batches_per_warp,
            b1 = min(b0 + batches_per_warp, bq + bk + bv);

  // chunks of the lane; in the half layout rotated chunks and their partners first
  const int rp = a.rot_dim / 2, rc = rp / N;          // rotated pairs, chunks of them (half layout)
  int ca = j, cb = j + lph;
  bool turn_a, turn_b;
  if (kInter) {
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

  const bool all_turn = __all_sync(0xffffffffu, turn_a && turn_b);

  if (kGroups == 4 && b1 - b0 > 2) {
    // the warp has the whole token: the lines of its later batches start for L2
    // while the first is worked on (three batches, an append of 16384 prompt
    // tokens: 51.2 to 48.4 us; two batches, 8192 tokens without values: 22.1
    // without and 22.6 with it; a batch ahead in registers: a third slower)
    const int first = min(per_batch, a.n_q ? a.n_q : a.n_k);
    const int lines = max(1, a.head_dim * (int)sizeof(T) / 128), n = (a.n_q + a.n_k + a.n_v - first) * lines;
#pragma unroll 1
    for (int i = lane; i < n; i += 32) {
      const int head = i / lines, line = i - head * lines;
      int h = first + head;
      const int kind = h < a.n_q ? 0 : h < a.n_q + a.n_k ? 1 : 2;
      h -= kind == 0 ? 0 : kind == 1 ? a.n_q : a.n_q + a.n_k;
      const HeadRows& in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
      const T* at = (const T*)in.data + (long long)t * in.ts + (long long)h * in.hs + line * (128 / (int)sizeof(T));
      asm volatile("prefetch.global.L2 [%0];" :: "l"(at));
    }
  }
  TokenSpot spot;
  bool have_spot = false;
  float c[N], s[N];
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int kind = b < bq ? 0 : b < bq + bk ? 1 : 2;
    const int n = kind == 0 ? a.n_q : a.n_k;
    const int h0 = (b - (kind == 0 ? 0 : kind == 1 ? bq : bq + bk)) * per_batch + sub;
    const HeadRows in = kind == 0 ? a.q : kind == 1 ? a.k : a.v;
    // (heads past n read the last one: no branches)
    const T* src = (const T*)in.data + (long long)t * in.ts;
    uint4 xa[kGroups], xb[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const uint4* at = reinterpret_cast<const uint4*>(src + (long long)min(h0 + i * hpw, n - 1) * in.hs);
      xa[i] = at[ca];
      xb[i] = at[cb];
    }
    const uint4* gain = reinterpret_cast<const uint4*>(kind == 0 ? a.q_gain : a.k_gain);
    const bool gained = kind < 2 && a.norm && gain;
    uint4 gain_a = {}, gain_b = {};
    if (gained) {
      gain_a = gain[ca];
      gain_b = gain[cb];
    }
    if (!have_spot) {
      have_spot = true;
      double freq[4];                                  // (rp <= 128)
#pragma unroll
      for (int i = 0; i < 4; ++i) freq[i] = lane + 32 * i < rp ? a.inv_freq[lane + 32 * i] : 0.0;
      spot = token_spot(a, t);
      if (!spot.live) return;
      if (rp > 0 && kind < 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = lane + 32 * i;
          if (p < rp) turn_sincos(spot.pos, freq[i], a.amplitude, s_cos[p], s_sin[p]);
        }
        __syncwarp();
        const int pa = kInter ? ca * (N / 2) : j * N, pb = kInter ? cb * (N / 2) : j * N + N / 2;
#pragma unroll
        for (int e = 0; e < N / 2; e += 2) {
          const float2 c0 = *reinterpret_cast<const float2*>(&s_cos[pa + e]),
                       c1 = *reinterpret_cast<const float2*>(&s_cos[pb + e]),
                       s0 = *reinterpret_cast<const float2*>(&s_sin[pa + e]),
                       s1 = *reinterpret_cast<const float2*>(&s_sin[pb + e]);
          c[e] = c0.x; c[e + 1] = c0.y; c[N / 2 + e] = c1.x; c[N / 2 + e + 1] = c1.y;
          s[e] = s0.x; s[e + 1] = s0.y; s[N / 2 + e] = s1.x; s[N / 2 + e + 1] = s1.y;
        }
      }
      // parts that do not turn keep their gain alone
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (!(e < N / 2 ? turn_a : turn_b)) { c[e] = 1.0f; s[e] = 0.0f; }
    }
    T* dst;
    long long out_hs;
    if (kind == 0 || !a.paged) {
      const HeadRows out = kind == 0 ? a.qo : a.ko;
      dst = (T*)out.data + (long long)t * out.ts;
      out_hs = out.hs;
    } else {
      if (spot.page < 0) continue;
      dst = (T*)(kind == 1 ? a.k_pages : a.v_pages) + (((spot.page * a.n_k) << a.b.page_shift) + spot.off) * a.head_dim;
      out_hs = (long long)a.head_dim << a.b.page_shift;
    }
    dst += h0 * out_hs;
    const long long out_step = out_hs << (5 - lph_shift);
    if (kind == 2) {
#pragma unroll
      for (int i = 0; i < kGroups; ++i, dst += out_step)
        if (h0 + i * hpw < n) {
          reinterpret_cast<uint4*>(dst)[ca] = xa[i];
          reinterpret_cast<uint4*>(dst)[cb] = xb[i];
        }
      continue;
    }
    // the lane's pair e is (u, v): half layout elements e of both chunks,
    // interleaved neighbours of chunk a (e < N / 2) or b
    float2 uc[N / 2], vs[N / 2], vc[N / 2], us[N / 2];
    {
      float ga[N], gb[N];
      if (gained) {
        Chunk<T>::unpack(gain_a, ga);
        Chunk<T>::unpack(gain_b, gb);
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) ga[e] = gb[e] = 1.0f;
      }
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float2 u = kInter ? (e < N / 2 ? make_float2(ga[2 * e], ga[2 * e + 2])
                                             : make_float2(gb[2 * e - N], gb[2 * e - N + 2]))
                                : make_float2(ga[e], ga[e + 1]);
        const float2 v = kInter ? (e < N / 2 ? make_float2(ga[2 * e + 1], ga[2 * e + 3])
                                             : make_float2(gb[2 * e - N + 1], gb[2 * e - N + 3]))
                                : make_float2(gb[e], gb[e + 1]);
        uc[e / 2] = mul2(u, make_float2(c[e], c[e + 1]));
        us[e / 2] = mul2(u, make_float2(s[e], s[e + 1]));
        vc[e / 2] = mul2(v, make_float2(c[e], c[e + 1]));
        vs[e / 2] = mul2(v, make_float2(-s[e], -s[e + 1]));
      }
    }
#pragma unroll
    for (int i = 0; i < kGroups; ++i, dst += out_step) {
      if (h0 - sub + i * hpw >= n) break;
      float x[N], y[N];
      Chunk<T>::unpack(xa[i], x);
      Chunk<T>::unpack(xb[i], y);
      float r = 1.0f;
      if (a.norm) {
        float2 ss = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int e = 0; e < N; e += 2) {
          ss = fma2(make_float2(x[e], x[e + 1]), make_float2(x[e], x[e + 1]), ss);
          ss = fma2(make_float2(y[e], y[e + 1]), make_float2(y[e], y[e + 1]), ss);
        }
        float z = ss.x + ss.y;
        for (int o = lph >> 1; o; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        r = rsqrtf(fmaf(z, a.inv_dim, a.eps));
      }
      const float2 rr = make_float2(r, r);
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        float2 u, v;
        if (kInter) {
          const int k = e < N / 2 ? 2 * e : 2 * e - N;
          u = e < N / 2 ? make_float2(x[k], x[k + 2]) : make_float2(y[k], y[k + 2]);
          v = e < N / 2 ? make_float2(x[k + 1], x[k + 3]) : make_float2(y[k + 1], y[k + 3]);
        } else {
          u = make_float2(x[e], x[e + 1]);
          v = make_float2(y[e], y[e + 1]);
        }
        float2 un = mul2(u, uc[e / 2]), vn = mul2(v, vc[e / 2]);
        // (a part that does not turn takes nothing from its partner, not even 0 times an infinity)
        if (all_turn || (e < N / 2 ? turn_a : turn_b)) {
          un = fma2(v, vs[e / 2], un);
          vn = fma2(u, us[e / 2], vn);
        }
        un = mul2(un, rr);
        vn = mul2(vn, rr);
        if (kInter) {
          const int k = e < N / 2 ? 2 * e : 2 * e - N;
          float(&z)[N] = e < N / 2 ? x : y;
          z[k] = un.x; z[k + 2] = un.y; z[k + 1] = vn.x; z[k + 3] = vn.y;
        } else {
          x[e] = un.x; x[e + 1] = un.y; y[e] = vn.x; y[e + 1] = vn.y;
        }
      }
      if (h0 + i * hpw < n) {
        reinterpret_cast<uint4*>(dst)[ca] = Chunk<T>::pack(x);
        reinterpret_cast<uint4*>(dst)[cb] = Chunk<T>::pack(y);
      }
    }
  }
}
