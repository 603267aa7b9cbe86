// Attention of ragged queries over a paged cache with a prefix the whole
// batch shares:
//
//   out_r = sum_j softmax_j(scale q_r.k_j) v_j,   lse_r = ln sum_j exp(scale q_r.k_j)
//
// over the prefix's keys and the sequence's own.  Softmax over a union of key
// sets splits exactly: with per-set lse_i and normalised out_i,
// lse = ln sum_i exp(lse_i) and out = sum_i exp(lse_i - lse) out_i.  So the
// prefix is one attention problem whose query rows are the whole batch's (its
// keys are read once, and 64 single tokens fill a matrix tile together), every
// sequence's own keys are another, and any tile may be cut along its keys.
//
// Work.  For one key head, the rows (token, query head of the group) of a
// sequence are cut into tiles of kRows rows, and each tile has the key blocks
// its rows can see.  All (part, sequence, key head, tile, key block) units lie
// on one line, every tile preceded by a few units for what a tile costs
// besides its blocks; CTA c takes the c-th of equal intervals of it.  A CTA so gets
// the end of one tile, whole tiles, and the start of another, whatever the
// lengths are, and no length has to be known on the host.  A tile that lies in
// one interval goes straight to the output; of a cut tile the CTA holding its
// first block keeps its result by row, the others in a slot of their own, and
// a second kernel joins them in order (the sums never depend on timing).
#pragma once
#include "dg_paged.cuh"

// n / d for n < 65536 and 1 <= d <= 32768 by one multiplication: with
// m = ceil(2^32 / d), m d - 2^32 < d, so n (m d - 2^32) < 2^32 and
// floor(n m / 2^32) = floor(n / d).  (d = 1: m would be 2^32.)
struct SmallDiv {
  uint32_t m;
  static uint32_t magic(uint32_t d) { return d == 1 ? 0u : (uint32_t)(((1ull << 32) + d - 1) / d); }
  DG_HD int div(int n) const {
#ifdef __CUDA_ARCH__
    return m ? (int)__umulhi((uint32_t)n, m) : n;
#else
    return m ? (int)(((uint64_t)(uint32_t)n * m) >> 32) : n;
#endif
  }
};

struct PagedAttnArgs {
  PagedBatch b;
  const void* q;
  void* out;
  long long q_ts, q_hs, o_ts, o_hs;   // token and head strides, elements
  int n_heads, n_kv_heads, G;         // G = n_heads / n_kv_heads
  SmallDiv by_g;
  int causal;
  float scale_log2;                   // scale * log2(e)
  const void *k_pages, *v_pages;
  float* lse;                         // natural, [n_tokens][n_heads], or null
  // workspace (rows = n_tokens * n_heads; parts: 0 own keys, 1 the prefix)
  int2* meta;                         // [parts][rows]: see PagedFrag::meta
  float* part_lse;                    // [parts][rows] log2-sum-exp of a cut tile's first piece
  float* slot_lse;                    // [grid][kRows]
  float* part_o;                      // [parts][rows][hd] normalised
  float* slot_o;                      // [grid][kRows][hd]
};

// One piece of work of a CTA: key blocks [kb0, kb1) of a tile.
struct PagedFrag {
  int nblk;        // key blocks; 0: no more work
  int part;        // 0: own keys, 1: the prefix
  int q0;          // first token of the sequence (part 1: of the batch)
  int row0, rows;  // the tile's first row of the sequence (row = token * G + head in group), its rows
  int tok0, rem0;  // row0 / G, row0 % G: row r of the tile is token tok0 + (rem0 + r) / G
  int kvh;         // key head
  int kb0;
  int limit;       // keys the tile's last row can see
  int vis0;        // row r sees the keys below min(vis_max, vis0 + (row0 + r) / G)
  int vis_max;
  int pages;       // needed entries of the page list
  int first;       // the piece starts its tile
  int whole;       // the piece is the whole tile
  int n_cont;      // later CTAs that hold pieces of this tile (valid where first)
  const int* page_list;
};

// Starting and ending a tile (query rows in, first scores, output) in units of
// a key block.  Measured on 8 canvases behind a 32768-token prefix (256-row
// tiles): 2 units 285 us, 3 to 5 263 us; ragged causal prompts 129, 128.5,
// 125 and 123 us for 2, 3, 4 and 5; 64 single tokens (128-row tiles, bound by
// memory, which a tile's start and end hardly hold up): 4 units 90.0 us,
// 3 86.7, 2 85.1, 1 84.9.  Twice or three times as many 256-row tiles of 1 to 16
// blocks on every CTA cost 10 to 14 us a tile beside 2.2 us a block, which is
// the 5.  The fp32 tiles of 64 rows took the 2 over from the 128-row ones, where
// a tile costs 7 us beside 5.5 us a block of 64 keys of 64: four causal prompts of
// 512 tokens (8 heads of 128) take 94 us with 0, 98 with 1, 107 with 2 and 3,
// 125 with 5; a canvas of 256 tokens 14 with 0 to 3, 18.5 with 5.
constexpr int paged_tile_cost(int rows) { return rows == 256 ? 5 : 2; }

template <int kRows, int kBlk>
struct PagedWalk {
  static constexpr int kTileCost = paged_tile_cost(kRows);
  const PagedAttnArgs& a;
  // (the host refuses batches whose line could reach 2^31 units)
  int x, x1;          // interval left: [x, x1)
  int per;            // interval length
  // current tile
  int part, seq, kvh, tile, n_tiles;
  int tile_x0;        // where the current tile starts on the line
  PagedSeq s;         // the sequence (part 1: the whole batch over the prefix)

  DG_HD PagedWalk(const PagedAttnArgs& a_) : a(a_) {}

  // (rows of a sequence are at most n_tokens * n_heads < 2^31)
  DG_HD int tiles_of(const PagedSeq& q) const { return (int)(((unsigned)(q.nq * a.G) + kRows - 1) / kRows); }
  // keys visible to the last row of a tile
  DG_HD int tile_limit(const PagedSeq& q, int part_, int tl) const {
    if (part_ == 1 || !a.causal) return q.kv;
    const unsigned rows = (unsigned)(q.nq * a.G), end = (unsigned)(tl + 1) * kRows;
    return imax(0, q.kv - q.nq + (int)(((end < rows ? end : rows) - 1) / (unsigned)a.G) + 1);
  }
  // A tile whose rows see nothing keeps one (masked) block: it writes its zeros.
  DG_HD int tile_blocks(const PagedSeq& q, int part_, int tl) const {
    return imax(1, (int)(((unsigned)tile_limit(q, part_, tl) + kBlk - 1) / kBlk));
  }
  DG_HD int tile_units(const PagedSeq& q, int part_, int tl) const { return kTileCost + tile_blocks(q, part_, tl); }
  DG_HD PagedSeq whole_batch() const {
    const PagedBatch& b = a.b;
    PagedSeq p;
    const int lo = b.cu_q[0], hi = b.cu_q[b.n_seqs];
    p.q0 = imin(imax(lo, 0), b.n_tokens);
    p.nq = imin(imax(hi, p.q0), b.n_tokens) - p.q0;
    p.kv = b.prefix_len;
    return p;
  }
  // Units of the tiles of one sequence for one key head (a whole warp asks for
  // one sequence).  Unsigned and without a check: a batch that passes the
  // host's bound fits, and offsets that overlap (reported by paged_seq) only
  // leave rows uncovered, whatever the sums wrap to.
  DG_HD unsigned units_of(const PagedSeq& q, int part_) const {
    const int n = tiles_of(q);
    if (part_ == 1 || !a.causal || n < 2) return n == 0 ? 0 : (unsigned)n * tile_units(q, part_, 0);
    unsigned sum = 0;
#ifdef __CUDA_ARCH__
    for (int i = threadIdx.x & 31; i < n; i += 32) sum += tile_units(q, 0, i);
    sum = __reduce_add_sync(0xffffffffu, sum);
#else
    for (int i = 0; i < n; ++i) sum += tile_units(q, 0, i);
#endif
    return sum;
  }
  // Interval `cta` of kSMs equal ones of a line of `total` units; false if it is empty.
  DG_HD bool take_interval(unsigned total, int cta) {
    total &= 0x7fffffffu;
    per = imax(1, (int)((total + kSMs - 1u) / kSMs));
    x = (int)lmin(total, (long long)cta * per);
    x1 = (int)lmin(total, (long long)x + per);
    return x < x1;
  }
  DG_HD void enter_prefix(int each) {
    part = 1;
    seq = -1;
    s = whole_batch();
    n_tiles = tiles_of(s);
    const int len = tile_units(s, 1, 0);
    kvh = x / each;
    tile = (x - kvh * each) / len;
    tile_x0 = kvh * each + tile * len;
  }
  // x lies in sequence i = q, which starts at x0 on the line (a whole warp)
  DG_HD void enter_sequence(int i, const PagedSeq& q, int x0) {
    part = 0;
    seq = i;
    s = q;
    n_tiles = tiles_of(s);
    tile = 0;
    const unsigned each = units_of(s, 0);
    kvh = each ? imin(a.n_kv_heads - 1, (int)((unsigned)(x - x0) / each)) : 0;
    tile_x0 = x0 + kvh * (int)each;
    if (n_tiles < 2) return;
    if (!a.causal) {   // tiles of one length
      const int len = tile_units(s, 0, 0);
      tile = imin(n_tiles - 1, (x - tile_x0) / len);
      tile_x0 += tile * len;
      return;
    }
#ifdef __CUDA_ARCH__
    const int lane = threadIdx.x & 31;
    for (int t0 = 0; t0 < n_tiles; t0 += 32) {   // 32 tiles at a time
      const int len = t0 + lane < n_tiles ? tile_units(s, 0, t0 + lane) : 0;
      int incl = len;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, x < tile_x0 + incl);   // the tile of x or a later one
      const int k = past ? __ffs(past) - 1 : 31;
      const int before = __shfl_sync(0xffffffffu, incl - len, k), all = __shfl_sync(0xffffffffu, incl, 31);
      if (past || t0 + 32 >= n_tiles) {
        tile = imin(t0 + k, n_tiles - 1);
        tile_x0 += before;
        break;
      }
      tile_x0 += all;
    }
#else
    for (int len; tile + 1 < n_tiles && x >= tile_x0 + (len = tile_units(s, 0, tile)); ++tile) tile_x0 += len;
#endif
  }

#ifdef __CUDACC__
  // Sequence base + lane and its units for all key heads (0 past the last).
  __device__ __noinline__ unsigned lane_units(int base, PagedSeq& q) const {
    const int lane = threadIdx.x & 31;
    q = PagedSeq{0, 0, 0};
    if (base + lane < a.b.n_seqs) q = paged_seq(a.b, base + lane);
    // one tile, or tiles of one length: by the lane; the others by the warp
    const int n = tiles_of(q);
    const bool many = a.causal && n > 1;
    unsigned u = n == 0 || many ? 0 : (unsigned)n * tile_units(q, 0, 0);
    for (unsigned m = __ballot_sync(0xffffffffu, many); m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const unsigned v = units_of(PagedSeq{0, __shfl_sync(0xffffffffu, q.nq, l), __shfl_sync(0xffffffffu, q.kv, l)}, 0);
      if (lane == l) u = v;
    }
    return u * a.n_kv_heads;
  }

  // Finds the CTA's interval and where it starts, by one warp; false if there
  // is nothing to do.  Up to 32 sequences are read once.
  __device__ bool begin() {
    const int lane = threadIdx.x & 31, n = a.b.n_seqs;
    PagedSeq q;
    unsigned u = lane_units(0, q), mine = u;
    unsigned each = 0;
    if (a.b.prefix_len > 0) each = units_of(whole_batch(), 1);
#pragma unroll 1
    for (int base = 32; base < n; base += 32) mine += lane_units(base, q);
    const unsigned pre = each * a.n_kv_heads;
    if (!take_interval(__reduce_add_sync(0xffffffffu, mine) + pre, blockIdx.x)) return false;
    if ((unsigned)x < pre) {
      enter_prefix((int)each);
      return true;
    }
    int at = (int)pre;
#pragma unroll 1
    for (int base = 0; base < n; base += 32) {
      if (n > 32) u = lane_units(base, q);
      int incl = (int)u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, x < at + incl);
      if (past) {
        const int k = __ffs(past) - 1;
        const PagedSeq f{__shfl_sync(0xffffffffu, q.q0, k), __shfl_sync(0xffffffffu, q.nq, k),
                         __shfl_sync(0xffffffffu, q.kv, k)};
        enter_sequence(base + k, f, at + __shfl_sync(0xffffffffu, incl - (int)u, k));
        return true;
      }
      at += __shfl_sync(0xffffffffu, incl, 31);
    }
    return false;   // (lengths that change while the kernel runs)
  }
#endif

  // The same on the host, for a batch in host memory.
  bool begin_host(int cta) {
    const unsigned each = a.b.prefix_len > 0 && a.b.n_seqs > 0 ? units_of(whole_batch(), 1) : 0;
    const unsigned pre = each * a.n_kv_heads;
    unsigned total = pre;
    for (int i = 0; i < a.b.n_seqs; ++i) total += units_of(paged_seq(a.b, i), 0) * a.n_kv_heads;
    if (!take_interval(total, cta)) return false;
    if ((unsigned)x < pre) {
      enter_prefix((int)each);
      return true;
    }
    int at = (int)pre;
    for (int i = 0; i < a.b.n_seqs; ++i) {
      const PagedSeq q = paged_seq(a.b, i);
      const int n = (int)(units_of(q, 0) * a.n_kv_heads);
      if (x < at + n) {
        enter_sequence(i, q, at);
        return true;
      }
      at += n;
    }
    return false;
  }

  // The next piece of the interval (nblk 0 at its end).
  DG_HD PagedFrag next() {
    PagedFrag f;
    f.nblk = 0;
    while (x < x1) {
      f.limit = tile_limit(s, part, tile);
      const int nb = imax(1, (int)(((unsigned)f.limit + kBlk - 1) / kBlk));
      const int b0 = tile_x0 + kTileCost;   // where block 0 lies
      x = imax(x, b0);
      if (x < x1) {
        f.part = part;
        f.q0 = s.q0;
        f.row0 = tile * kRows;
        f.rows = imin(kRows, s.nq * a.G - f.row0);
        f.tok0 = (int)((unsigned)f.row0 / (unsigned)a.G);
        f.rem0 = f.row0 - f.tok0 * a.G;
        f.kvh = kvh;
        f.kb0 = imin(nb - 1, x - b0);
        f.nblk = imax(1, imin(nb - f.kb0, x1 - x));
        f.vis_max = s.kv;
        f.vis0 = part == 1 || !a.causal ? s.kv : s.kv - s.nq + 1;
        f.first = f.kb0 == 0;
        f.whole = f.first && f.nblk == nb;
        // (the CTA of the last block is this one unless the interval ends before it)
        f.n_cont = b0 + nb <= x1 ? 0 : (b0 + nb - 1 - x1) / per + 1;
        f.pages = (int)(((unsigned)f.limit + (1u << a.b.page_shift) - 1) >> a.b.page_shift);
        f.page_list = part == 1 ? a.b.prefix_pages : a.b.table + (long long)seq * a.b.table_stride;
        x += f.nblk;
      }
      if (x < x1) {   // on to the next tile
        tile_x0 = b0 + nb;
        if (++tile >= n_tiles) {
          tile = 0;
          if (++kvh >= a.n_kv_heads) {
            kvh = 0;
            part = 0;
            do {
              if (++seq >= a.b.n_seqs) {
                x = x1;   // (lengths that change while the kernel runs)
                break;
              }
              s = paged_seq(a.b, seq);
            } while (s.nq == 0);
            n_tiles = tiles_of(s);
          }
        }
      }
      if (f.nblk) break;
    }
    return f;
  }
};

// Where a row's piece goes.  meta of a row of a cut tile: {first CTA,
// later CTAs * kRows + row in the tile}; of a finished row: {-1, 0}.
struct PagedDest {
  float* o;       // fp32 destination, or null
  float* lse;
  bool final;     // straight to the output
};

template <int kRows>
__device__ __forceinline__ PagedDest paged_dest(const PagedAttnArgs& a, const PagedFrag& f, int r, int hd,
                                                long long row) {
  PagedDest d;
  const long long rows = (long long)a.b.n_tokens * a.n_heads;
  d.final = f.whole && a.b.prefix_len == 0;
  d.o = nullptr;
  d.lse = nullptr;
  if (f.first) a.meta[f.part * rows + row] = d.final ? make_int2(-1, 0)
                                                     : make_int2((int)blockIdx.x, f.n_cont * kRows + r);
  if (d.final) return d;
  if (f.first) {
    d.o = a.part_o + (f.part * rows + row) * hd;
    d.lse = a.part_lse + f.part * rows + row;
  } else {
    d.o = a.slot_o + ((long long)blockIdx.x * kRows + r) * hd;
    d.lse = a.slot_lse + (long long)blockIdx.x * kRows + r;
  }
  return d;
}

constexpr float kLn2 = 0.69314718055994530942f;

// Joins the pieces of every row: own keys first, then the prefix, each in key
// order.  A block looks at `per_block` rows (at most 64), lists those the main
// kernel did not finish (without a prefix most are), and its 16 groups of 16
// lanes take them in turn, kBatch pieces at a time.  With few rows a block has
// one, and its groups (kShare = 16) share the pieces: a long context may have
// cut it into 148.
//
// Bound by the chain batch -> meta -> pieces and its instructions (41 % of the
// issue slots, 33 % of the memory rate).  Listing the open rows for the whole
// block, dividing and clamping once a row in the listing, and one reference for
// a batch of pieces took ragged causal prompts from 18.5 to 11.4 us (a sixth of
// their rows is cut), 8 canvases behind a shared prompt from 16.5 to 14.4.
// Blocks an SM x pieces in flight: 4 x 4 as good as 5 x 2 and 3 x 4; with one or
// two pieces at 8 blocks the registers spill (91 and 105 us for the whole call
// against 85).
constexpr int kJoinRows = 64;

template <typename T, int kHd, int kShare>
__global__ void __launch_bounds__(256, kShare > 1 ? 1 : 4)
k_paged_join(const __grid_constant__ PagedAttnArgs a, int row_shift, int grid_main, int per_block) {
  constexpr int kPer = kHd / 16, kBatch = kShare > 1 ? 8 : 4;   // columns a lane, pieces in flight
  __shared__ float s_acc[kShare > 1 ? 16 : 1][kHd], s_ref[16], s_sum[16];
  __shared__ int4 s_job[kJoinRows];       // row, first slot of each part, pieces of part 0 and (from bit 16) 1
  __shared__ long long s_dst[kJoinRows];
  __shared__ int s_n;
  pdl_wait();
  const int grp = threadIdx.x >> 4, lane = threadIdx.x & 15;
  const int share = kShare > 1 ? grp : 0;
  const long long rows = (long long)a.b.n_tokens * a.n_heads;
  const int parts = a.b.prefix_len > 0 ? 2 : 1;
  if (threadIdx.x < 32) {
    const int lo = a.b.n_seqs > 0 ? a.b.cu_q[0] : 0, hi = a.b.n_seqs > 0 ? a.b.cu_q[a.b.n_seqs] : 0;
    const long long row_lo = (long long)lo * a.n_heads, row_hi = lmin((long long)hi * a.n_heads, rows);
    int2 m0[kJoinRows / 32], m1[kJoinRows / 32];
#pragma unroll
    for (int h = 0; h < kJoinRows / 32; ++h) {
      const int i = 32 * h + threadIdx.x;
      const long long row = (long long)blockIdx.x * per_block + i;
      const bool in = i < per_block && row >= row_lo && row < row_hi;
      m0[h] = in ? a.meta[row] : make_int2(-1, 0);       // (-1: written by the main kernel)
      m1[h] = in && parts == 2 ? a.meta[rows + row] : make_int2(0, 0);
    }
    int n = 0;
#pragma unroll
    for (int h = 0; h < kJoinRows / 32; ++h) {
      const unsigned open = __ballot_sync(0xffffffffu, m0[h].x >= 0);
      const int at = n + __popc(open & ((1u << threadIdx.x) - 1));
      if (m0[h].x >= 0) {
        // first CTA, row in the tile, later CTAs of each part (what a row no
        // tile covered finds here still stays in the workspace)
        const int cta0 = min(m0[h].x, grid_main - 1), cta1 = min(max(m1[h].x, 0), grid_main - 1);
        const int n0 = 1 + min(max(m0[h].y >> row_shift, 0), grid_main - 1 - cta0);
        const int n1 = parts == 1 ? 0 : 1 + min(max(m1[h].y >> row_shift, 0), grid_main - 1 - cta1);
        const int i = 32 * h + threadIdx.x, mask = (1 << row_shift) - 1;
        s_job[at] = make_int4(i, (cta0 << row_shift) + (m0[h].y & mask), (cta1 << row_shift) + (m1[h].y & mask),
                              n0 | n1 << 16);
        const unsigned row = (unsigned)blockIdx.x * per_block + i, tok = row / (unsigned)a.n_heads;
        s_dst[at] = tok * a.o_ts + (row - tok * a.n_heads) * a.o_hs;
      }
      n += __popc(open);
    }
    if (threadIdx.x == 0) s_n = n;
  }
  __syncthreads();
  for (int k = kShare > 1 ? 0 : grp; k < s_n; k += kShare > 1 ? 1 : 16) {
    const int4 job = s_job[k];
    const long long row = (long long)blockIdx.x * per_block + job.x;
    const int n0 = job.w & 0xffff, n = n0 + (job.w >> 16);
    float acc[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.0f;
    float top = -INFINITY, sum = 0.0f;   // reference and sum of 2^(lse - top)
    for (int i0 = share; i0 < n; i0 += kShare * kBatch) {
      float4 v[kBatch][kPer / 4];
      float lse[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int i = i0 + u * kShare;
        lse[u] = -INFINITY;
        if (i >= n) continue;
        // a part's first piece lies in the row's place, the others in their CTA's slot
        const bool p = i >= n0, slot = i != 0 && i != n0;
        const long long at = slot ? (p ? job.z : job.y) + ((p ? i - n0 : i) << row_shift) : p ? rows + row : row;
        const float* o = (slot ? a.slot_o : a.part_o) + at * kHd;
        lse[u] = (slot ? a.slot_lse : a.part_lse)[at];
#pragma unroll
        for (int c = 0; c < kPer / 4; ++c) v[u][c] = *reinterpret_cast<const float4*>(o + c * 64 + lane * 4);
      }
      float up = top;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) up = fmaxf(up, lse[u]);
      const float ref = up == -INFINITY ? 0.0f : up, w0 = exp2f(top - ref);
      top = up;
      sum *= w0;
#pragma unroll
      for (int c = 0; c < kPer; ++c) acc[c] *= w0;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (lse[u] == -INFINITY) continue;    // (no piece, or no visible key)
        const float w = exp2f(lse[u] - ref);
        sum += w;
#pragma unroll
        for (int c = 0; c < kPer / 4; ++c) {
          acc[c * 4] += v[u][c].x * w;
          acc[c * 4 + 1] += v[u][c].y * w;
          acc[c * 4 + 2] += v[u][c].z * w;
          acc[c * 4 + 3] += v[u][c].w * w;
        }
      }
    }
    T* dst = (T*)a.out + s_dst[k];
    if (kShare == 1) {
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
      for (int c = 0; c < kPer / 4; ++c)
        store4<T>(dst + c * 64 + lane * 4, acc[c * 4] * inv, acc[c * 4 + 1] * inv, acc[c * 4 + 2] * inv,
                  acc[c * 4 + 3] * inv);
      if (a.lse && lane == 0) a.lse[row] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
    } else {
      // (the whole block is on its one row: the branches above were uniform)
      __syncthreads();
#pragma unroll
      for (int c = 0; c < kPer / 4; ++c)
        *reinterpret_cast<float4*>(&s_acc[grp % (kShare > 1 ? 16 : 1)][c * 64 + lane * 4]) =
            make_float4(acc[c * 4], acc[c * 4 + 1], acc[c * 4 + 2], acc[c * 4 + 3]);
      if (lane == 0) {
        s_ref[grp] = top;
        s_sum[grp] = sum;
      }
      __syncthreads();
      if (threadIdx.x < kHd) {
        float ref = -INFINITY, x = 0.0f, z = 0.0f;
#pragma unroll
        for (int g = 0; g < 16; ++g) ref = fmaxf(ref, s_ref[g]);
#pragma unroll
        for (int g = 0; g < 16; ++g) {
          const float w = s_ref[g] == -INFINITY ? 0.0f : exp2f(s_ref[g] - ref);
          x += s_acc[g % (kShare > 1 ? 16 : 1)][threadIdx.x] * w;
          z += s_sum[g] * w;
        }
        dst[threadIdx.x] = from_f<T>(z == 0.0f ? 0.0f : x / z);
        if (a.lse && threadIdx.x == 0) a.lse[row] = z == 0.0f ? -INFINITY : (ref + log2f(z)) * kLn2;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// fp32: CUDA cores (the tensor cores have no fp32 product).  A CTA of 256
// threads holds a tile of 64 rows and takes 64 keys at a time, the next block
// on its way into the other half of a double buffer (asynchronous copies that
// write zeros for keys past the last visible one, so what the cache holds
// there never enters a sum).
//
// More than 8 rows: thread (ty, tx) owns the scores of rows 4 ty .. 4 ty + 3
// and keys tx + 16 c, and of the output the same rows with columns 4 tx + 64 c;
// warps whose rows lie past the piece's end only load.  Bound by the FMA pipe.
// At most 8 rows (single tokens): that mapping would leave seven of eight
// warps without a row, so a thread takes the scores of one key for two rows,
// and warp r then has row r for the softmax and the product with V.  Bound by
// memory: 16 tokens over 2000 keys of 128, 1 to 8 rows a key head, 28 to 40 us,
// with the other mapping 55 to 57.
//
// Measured, with the join: a canvas of 256 tokens (4 heads of 64, 64 keys
// before it, 84 MFLOP) 14.3 us, of which the loads that depend on one another
// (lengths, pages, keys) and the second launch are most; the single mapping
// without the double buffer took 16.7.  Four causal prompts of 512 tokens (8
// heads of 128) 107 us, 8 canvases of 256 behind a shared 1024-token prompt (8
// heads of 128 over 2) 371: 20 and 29 TFLOP/s of a nominal 74, the FMA pipe busy
// for 48 % of the former; a thread's 4 x 4 scores read 8 values for 16 products.
// ---------------------------------------------------------------------------
constexpr int kPaF32Rows = 64, kPaF32Blk = 64, kPaF32Few = 8;
template <int kHd>
struct PaF32 {
  static constexpr int kLd = kHd + 4;                                   // padded rows of Q and K
  static constexpr int kKv = kPaF32Blk * (kLd + kHd);                   // floats of a block's K and V
  static constexpr int kLdP = kPaF32Blk + 4;
  static constexpr int kSmem = (kPaF32Rows * kLd + 2 * kKv + kPaF32Rows * kLdP) * 4;
};

// 16 bytes, zeros where not `ok`.
__device__ __forceinline__ void cp_async_16z(float* dst, const float* src, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0)
               : "memory");
}

// Where the output of a row of a piece goes, and its log-sum-exp (l2: base 2).
__device__ __forceinline__ float* paged_f32_dest(const PagedAttnArgs& a, const PagedFrag& f, int r, int hd, float l2,
                                                 bool writer) {
  const int t = a.by_g.div(f.rem0 + r), tok = f.q0 + f.tok0 + t, head = f.kvh * a.G + f.rem0 + r - t * a.G;
  const long long row = (long long)tok * a.n_heads + head;
  const PagedDest d = paged_dest<kPaF32Rows>(a, f, r, hd, row);   // (every thread of the row stores the same meta)
  if (writer) {
    if (!d.final) *d.lse = l2;
    else if (a.lse) a.lse[row] = l2 * kLn2;
  }
  return d.final ? (float*)a.out + (long long)tok * a.o_ts + (long long)head * a.o_hs : d.o;
}

template <int kHd>
__global__ void __launch_bounds__(256, 1) k_paged_attn_f32(const __grid_constant__ PagedAttnArgs a) {
  using C = PaF32<kHd>;
  constexpr int R = kPaF32Rows, B = kPaF32Blk, kLd = C::kLd, kLdP = C::kLdP, kOc = kHd / 64, kCh = kHd / 4;
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;
  float* sKV = sQ + R * kLd;
  float* sP = sKV + 2 * C::kKv;
  pdl_enter();
  PagedWalk<R, B> walk(a);
  if (!walk.begin()) return;   // (each warp finds the same)
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, warp = tid >> 5, lane = tid & 31;
  const int page_mask = (1 << a.b.page_shift) - 1;
  for (;;) {
    const PagedFrag f = walk.next();
    if (f.nblk == 0) break;
    auto issue = [&](int kb, int buf) {
      float* sK = sKV + buf * C::kKv;
      float* sV = sK + B * kLd;
      for (int i = tid; i < B * kCh; i += 256) {
        const int r = i / kCh, c = i % kCh * 4, key = kb * B + r;
        bool ok = key < f.limit;
        long long off = 0;
        if (ok) {
          const int page = f.page_list[key >> a.b.page_shift];
          ok = page >= 0 && page < a.b.n_pages;
          if (ok) off = ((((long long)page * a.n_kv_heads + f.kvh) << a.b.page_shift) + (key & page_mask)) * kHd + c;
          else paged_error(a.b, kStatusState);
        }
        cp_async_16z(sK + r * kLd + c, (const float*)a.k_pages + off, ok);
        cp_async_16z(sV + r * kHd + c, (const float*)a.v_pages + off, ok);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();   // the previous piece is done with shared memory
    for (int i = tid; i < R * kCh; i += 256) {
      const int r = i / kCh, c = i % kCh * 4;
      const bool ok = r < f.rows;
      const int t = ok ? a.by_g.div(f.rem0 + r) : 0;
      const float* src = (const float*)a.q;
      if (ok)
        src += (long long)(f.q0 + f.tok0 + t) * a.q_ts + (long long)(f.kvh * a.G + f.rem0 + r - t * a.G) * a.q_hs + c;
      cp_async_16z(sQ + r * kLd + c, src, ok);
    }
    issue(f.kb0, 0);
    const bool few = f.rows <= kPaF32Few;
    const bool on = few ? warp < f.rows : warp * 8 < f.rows;
    int vis[4];
    float top[4], sum[4], o[4][4 * kOc];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      vis[i] = min(f.vis_max, f.vis0 + f.tok0 + a.by_g.div(f.rem0 + (few ? warp : ty * 4 + i)));
      top[i] = -INFINITY;
      sum[i] = 0.0f;
#pragma unroll
      for (int c = 0; c < 4 * kOc; ++c) o[i][c] = 0.0f;
    }
    for (int j = 0; j < f.nblk; ++j) {
      const int key0 = (f.kb0 + j) * B;
      const float* sK = sKV + (j & 1) * C::kKv;
      const float* sV = sK + B * kLd;
      if (j + 1 < f.nblk) {
        issue(f.kb0 + j + 1, (j + 1) & 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      if (few) {
        // scores of key tid % 64 for rows 2 (tid / 64) and the next
        const int key = tid & 63, r0 = tid >> 6 << 1;
        if (r0 < f.rows) {
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 8
          for (int d = 0; d < kHd; d += 4) {
            const float4 k = *reinterpret_cast<const float4*>(sK + key * kLd + d);
            const float4 q0 = *reinterpret_cast<const float4*>(sQ + r0 * kLd + d);
            const float4 q1 = *reinterpret_cast<const float4*>(sQ + (r0 + 1) * kLd + d);
            s0 += q0.x * k.x + q0.y * k.y + q0.z * k.z + q0.w * k.w;
            s1 += q1.x * k.x + q1.y * k.y + q1.z * k.z + q1.w * k.w;
          }
          sP[r0 * kLdP + key] = s0 * a.scale_log2;
          sP[(r0 + 1) * kLdP + key] = s1 * a.scale_log2;
        }
        __syncthreads();
        if (on) {
          float x[2], mx = -INFINITY;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            x[u] = key0 + lane + 32 * u < vis[0] ? sP[warp * kLdP + lane + 32 * u] : -INFINITY;
            mx = fmaxf(mx, x[u]);
          }
#pragma unroll
          for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float up = fmaxf(top[0], mx), old = top[0] == -INFINITY ? 0.0f : exp2f(top[0] - up);
          float add = 0.0f;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float p = x[u] == -INFINITY ? 0.0f : exp2f(x[u] - up);
            add += p;
            sP[warp * kLdP + lane + 32 * u] = p;
          }
          sum[0] = sum[0] * old + warp_sum(add);
          top[0] = up;
          __syncwarp();
          // columns 2 lane + 64 c and the next
#pragma unroll
          for (int c = 0; c < 2 * kOc; ++c) o[0][c] *= old;
#pragma unroll 4
          for (int k = 0; k < B; k += 4) {
            const float4 p = *reinterpret_cast<const float4*>(sP + warp * kLdP + k);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
#pragma unroll
              for (int c = 0; c < kOc; ++c) {
                const float2 v = *reinterpret_cast<const float2*>(sV + (k + kk) * kHd + c * 64 + lane * 2);
                const float pp = kk == 0 ? p.x : kk == 1 ? p.y : kk == 2 ? p.z : p.w;
                o[0][2 * c] += pp * v.x;
                o[0][2 * c + 1] += pp * v.y;
              }
          }
        }
      } else if (on) {
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[i][k] = 0.0f;
#pragma unroll 4
        for (int d = 0; d < kHd; d += 4) {
          float4 qv[4], kv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4*>(sQ + (ty * 4 + i) * kLd + d);
#pragma unroll
          for (int k = 0; k < 4; ++k) kv[k] = *reinterpret_cast<const float4*>(sK + (tx + 16 * k) * kLd + d);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              s[i][k] += qv[i].x * kv[k].x + qv[i].y * kv[k].y + qv[i].z * kv[k].z + qv[i].w * kv[k].w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float mx = -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[i][k] = key0 + tx + 16 * k < vis[i] ? s[i][k] * a.scale_log2 : -INFINITY;
            mx = fmaxf(mx, s[i][k]);
          }
#pragma unroll
          for (int w = 8; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          const float up = fmaxf(top[i], mx);
          const float old = top[i] == -INFINITY ? 0.0f : exp2f(top[i] - up);
          float add = 0.0f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float p = s[i][k] == -INFINITY ? 0.0f : exp2f(s[i][k] - up);
            add += p;
            sP[(ty * 4 + i) * kLdP + tx + 16 * k] = p;
          }
#pragma unroll
          for (int w = 8; w; w >>= 1) add += __shfl_xor_sync(0xffffffffu, add, w);
          sum[i] = sum[i] * old + add;
          top[i] = up;
#pragma unroll
          for (int c = 0; c < 4 * kOc; ++c) o[i][c] *= old;
        }
        __syncwarp();   // rows 4 ty .. belong to one half warp
#pragma unroll 2
        for (int k = 0; k < B; k += 4) {
          float4 p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(sP + (ty * 4 + i) * kLdP + k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
#pragma unroll
            for (int c = 0; c < kOc; ++c) {
              const float4 v = *reinterpret_cast<const float4*>(sV + (k + kk) * kHd + c * 64 + tx * 4);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float pp = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
                o[i][c * 4] += pp * v.x;
                o[i][c * 4 + 1] += pp * v.y;
                o[i][c * 4 + 2] += pp * v.z;
                o[i][c * 4 + 3] += pp * v.w;
              }
            }
        }
      }
      __syncthreads();   // the block's buffer is free
    }
    if (few) {
      if (on) {
        const float inv = sum[0] == 0.0f ? 0.0f : 1.0f / sum[0];
        float* dst = paged_f32_dest(a, f, warp, kHd, sum[0] == 0.0f ? -INFINITY : top[0] + log2f(sum[0]), lane == 0);
#pragma unroll
        for (int c = 0; c < kOc; ++c)
          *reinterpret_cast<float2*>(dst + c * 64 + lane * 2) = make_float2(o[0][2 * c] * inv, o[0][2 * c + 1] * inv);
      }
      continue;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= f.rows) continue;
      const float inv = sum[i] == 0.0f ? 0.0f : 1.0f / sum[i];
      float* dst = paged_f32_dest(a, f, r, kHd, sum[i] == 0.0f ? -INFINITY : top[i] + log2f(sum[i]), tx == 0);
#pragma unroll
      for (int c = 0; c < kOc; ++c)
        *reinterpret_cast<float4*>(dst + c * 64 + tx * 4) =
            make_float4(o[i][c * 4] * inv, o[i][c * 4 + 1] * inv, o[i][c * 4 + 2] * inv, o[i][c * 4 + 3] * inv);
    }
  }
}
