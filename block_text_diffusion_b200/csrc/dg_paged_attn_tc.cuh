// The paged attention of dg_paged_attn.cuh on the tensor cores (bf16).
//
// One CTA per SM, 384 threads:
//   warps 0-3, 4-7  softmax of the accumulators A and B (thread = query row =
//                   TMEM lane) and epilogue;
//   warp 8          walks the CTA's interval and loads K and V blocks of 128
//                   keys by TMA, page by page;
//   warps 9, 11     issue the MMAs of A and B;
//   warp 10         loads the query rows and clears the rows of V past the last
//                   visible key.
// A piece of more than 128 rows runs wide: A holds its first 128 rows, B the
// rest, and both use every K/V block.  A piece of at most 128 rows (single
// tokens, the end of a ragged sequence) runs split: A and B hold the same rows
// and take every other key block, so two softmaxes run side by side; A joins
// the two halves at the end.
//
// S = Q K^T goes to TMEM; the softmax thread reads its row, writes P back over
// it as bf16, and O += P V takes P from TMEM, so P never crosses shared
// memory.  V stays as the cache holds it ([key][component]): the MMA reads it
// as an MN-major operand.  TMEM columns: S_A/P_A [0,128), S_B/P_B [128,256),
// O_A [256,256+hd), O_B [384,384+hd).
//
// The loads of the next piece (K and V as the ring empties, the query rows
// after the last Q K^T) run under the end of the current one.  Each role's
// code is written once, in a loop over both modes: with the roles unrolled
// per mode the kernel was 150 KB and spent its time fetching instructions.
//
// Measured, with the join: 8 canvases of 256 tokens behind 32768 + 256 keys
// (8 heads of 128 over 2 key heads) 288 us, 0.97 PFLOP/s of
// 1.62: a step of 2 x 128 rows x 128 keys takes 3770 clocks, its MMAs 2560 (the
// products with Q and K from shared memory run at 80 clocks for 64), its
// exponentials 2048; what is left is the way from S to P and back.  64 single
// tokens behind a shared 2048-token prompt 75 to 79 us, 3.9 to 4.1 TB/s of keys
// and values.  All 12 warps have the 168 registers of an even share, and 40
// bytes are spilled; nothing moves registers from the four loading and issuing
// warps to the softmax's eight.
#pragma once
#include "dg_paged_attn.cuh"

constexpr int kPaThreads = 384;
constexpr int kPaBlk = 128;
constexpr int kPaFrags = 4;       // pieces announced ahead
constexpr int kPaPart = 96;       // keys of a block whose probabilities go to the MMA before the rest
constexpr int kPaStage = 4096;    // epilogue staging of a softmax warp: 32 rows x 128 bytes

// kNarrow: tiles of 128 rows, every piece split.  Without the second query
// tile and the epilogue staging the ring has half as many blocks again, which
// is what single tokens over long contexts are bound by: the bytes in flight.
template <int kHd, bool kNarrow>
struct PaTc {
  static constexpr int kRows = kNarrow ? 128 : 256;  // of a tile
  static constexpr int kHalves = kHd / 64;           // 128-byte column groups of a row
  static constexpr int kBytes = 128 * kHd * 2;       // 128 rows of Q, K or V
  static constexpr int kStages = (kNarrow ? 6 : 4) * (kHd == 128 ? 1 : 2);
  static constexpr int kStageBytes = kNarrow ? 0 : 8 * kPaStage;
  static constexpr int kSmem = (kRows / 128 + kStages) * kBytes + kStageBytes + 1024;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc], A bf16 pairs in 32-bit columns.
__device__ __forceinline__ void tc_mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  const uint32_t z = 0;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, {%5, %6, %7, %8}, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(z), "r"(z), "r"(z), "r"(z)
      : "memory");
}

// MN-major operand, 128-byte swizzle: 64 components (128 B) x 8 keys an atom,
// atoms 1024 B apart along the keys (stride offset), column groups of 64
// components 128 rows = 16 KB apart (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(16384 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32_nw(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// A wait of the whole warp, agreed on by its lanes (what follows is often
// warp-collective).  Reading the wall clock takes longer than most waits, so
// it starts after a number of failed tries (each suspends for a while itself).
__device__ __noinline__ bool pa_wait_slow(uint64_t* bar, uint32_t parity, int* err) {
  for (int i = 0; i < 64; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait(bar, parity, err ? err : &g_serving_status, kStatusTimeout);
}
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, int* err) {
  bool ok = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) ok = __all_sync(0xffffffffu, pa_wait_slow(bar, parity, err));
  else ok = true;
  tc_fence_after();
  return ok;
}
__device__ __forceinline__ bool pa_wait_one(uint64_t* bar, uint32_t parity, int* err) {   // one thread
  return mbar_try_wait(bar, parity) || pa_wait_slow(bar, parity, err);
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The last block of a piece.  Its keys past the last visible one are masked in
// S, so P is 0 there, but 0 times whatever their values hold (the cache may
// hold anything) is not 0 for an infinity or a NaN: the product with V stops
// after the last 16 keys that hold a visible one, and the rows of V past it in
// those 16 become zeros.
struct PaTail {
  int valid, steps;   // visible keys of the block, MMAs of 16 keys (one at least)
  bool clear;
  __device__ __forceinline__ PaTail(const PagedFrag& f) {
    valid = max(0, min(kPaBlk, f.limit - (f.kb0 + f.nblk - 1) * kPaBlk));
    steps = max(1, (valid + 15) >> 4);
    clear = steps * 16 != valid;
  }
};

template <int kHd, bool kNarrow>
__global__ void __launch_bounds__(kPaThreads, 1)
k_paged_attn_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ PagedAttnArgs a) {
  using C = PaTc<kHd, kNarrow>;
  constexpr int ST = C::kStages, kRows = C::kRows;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;                             // A, B
  uint8_t* sKV = smem + kRows / 128 * C::kBytes;  // ring of K and V blocks
  uint8_t* sStage = sKV + ST * C::kBytes;         // epilogue staging
  __shared__ __align__(8) uint64_t kv_full[ST], kv_empty[ST], frag_full[kPaFrags], frag_empty[kPaFrags];
  __shared__ __align__(8) uint64_t q_full[2], q_empty[2], s_full[2], p_part[2], p_full[2], o_done[2];
  __shared__ __align__(8) uint64_t half_full, half_empty, v_last, v_tail[2], turn[2][4], mma_end[2];
  __shared__ PagedFrag s_frag[kPaFrags];
  __shared__ float s_half[128][2];                // split: maximum and sum of B's half, per row
  __shared__ uint32_t tmem_base;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const err = a.b.status;
  pdl_launch();
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 2); }
    for (int s = 0; s < kPaFrags; ++s) { mbar_init(&frag_full[s], 1); mbar_init(&frag_empty[s], 11); }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1);
      mbar_init(&q_empty[t], 2 - t);   // A's rows serve both accumulators of a split piece
      mbar_init(&v_tail[t], 1);
      for (int w = 0; w < 4; ++w) mbar_init(&turn[t][w], 1);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_part[t], 4);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_done[t], 1);
      mbar_init(&mma_end[t], 1);
    }
    mbar_init(&v_last, 2);
    mbar_init(&half_full, 4);
    mbar_init(&half_empty, 4);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&tmem_base, 512);
  if (warp == 8 && lane == 0) { prefetch_tmap(&tmK); prefetch_tmap(&tmV); }
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  bool ok = true;

  if (warp == 8) {
    // ---------------- walk and TMA ----------------
    const int page_shift = a.b.page_shift, page = 1 << page_shift;
    const int per_blk = page >= kPaBlk ? 1 : kPaBlk >> page_shift;   // pages a block
    int cnt = 0;
    PagedWalk<kRows, kPaBlk> walk(a);
    if (!walk.begin()) walk.x = walk.x1 = 0;
#pragma unroll 1
    for (int fi = 0; ok; ++fi) {
      const PagedFrag f = walk.next();
      const int slot = fi % kPaFrags;
      if (fi >= kPaFrags) ok = pa_wait(&frag_empty[slot], ((fi / kPaFrags) & 1) ^ 1, err);
      if (!ok) break;
      if (lane == 0) {
        s_frag[slot] = f;
        mbar_arrive(&frag_full[slot]);
      }
      if (f.nblk == 0) break;
      const bool split = kNarrow || f.rows <= 128;
      // The page ids of 32 pages are held by the 32 lanes, for K and for V apart
      // (in a split piece V trails K by two blocks).
      int base_k = -64, base_v = -64, id_k = 0, id_v = 0;
      // Blocks in the order the MMAs use them.  Wide: K0 V0 K1 V1 ...; split:
      // K0 K1 V0 K2 V1 ... (each accumulator one block ahead).
      const int n2 = 2 * f.nblk;
#pragma unroll 1
      for (int i = 0; i < n2; ++i) {
        const bool is_v = split ? (i > 0 && (i & 1) == 0) || i == n2 - 1 : (i & 1);
        const int j = !split ? i >> 1 : i == n2 - 1 ? f.nblk - 1 : is_v ? i / 2 - 1 : (i + 1) / 2;
        const int s = cnt % ST;
        if (cnt >= ST) ok = pa_wait(&kv_empty[s], ((cnt / ST) & 1) ^ 1, err);
        if (!ok) break;
        ++cnt;
        const int key0 = (f.kb0 + j) * kPaBlk, pg0 = key0 >> page_shift;
        // pages of the block that hold a visible key (none in a block that is there for its zeros)
        const int n_pg = max(0, min(per_blk, f.pages - pg0));
        int base = is_v ? base_v : base_k, id = is_v ? id_v : id_k;
        if (pg0 < base || pg0 + per_blk > base + 32) {
          base = pg0;
          id = -1;
          if (pg0 + lane < f.pages) {
            id = f.page_list[pg0 + lane];
            if (id < 0 || id >= a.b.n_pages) {
              paged_error(a.b, kStatusState);
              id = a.b.n_pages;   // past the tensor's end: reads as zeros
            }
          }
          if (is_v) { base_v = base; id_v = id; } else { base_k = base; id_k = id; }
        }
        if (lane == 0) mbar_expect_tx(&kv_full[s], page >= kPaBlk ? (n_pg ? C::kBytes : 0) : n_pg * page * kHd * 2);
        __syncwarp();
        // a page of 128 keys or more: one box for all; smaller: one box per page and column group
        const int pi = page >= kPaBlk ? lane : lane / C::kHalves, half = page >= kPaBlk ? 0 : lane % C::kHalves;
        const int my = __shfl_sync(0xffffffffu, id, (pg0 - base + pi) & 31);
        if (pi < n_pg)
          tma_load_4d(smem_u32(sKV + s * C::kBytes) + half * 16384 + pi * page * 128, is_v ? &tmV : &tmK, 0,
                      key0 & (page - 1), half, my * a.n_kv_heads + f.kvh, &kv_full[s]);
        __syncwarp();
      }
    }
    // The ring's last loads have landed before the block gives its memory up.
    // (They have long been used, unless a wait ran out somewhere.)
#pragma unroll 1
    for (int c = max(0, cnt - ST); c < cnt; ++c)
      if (!pa_wait(&kv_full[c % ST], (c / ST) & 1, err)) break;
  } else if (warp == 9 || warp == 11) {
    // ---------------- MMA issue: warp 9 for A, warp 11 for B ----------------
    // One thread for each accumulator: what a thread does between two products
    // (bookkeeping, waits, commits: a few hundred cycles) the tensor core
    // spends on the other's.
    constexpr uint32_t kIdS = idesc_bf16(128, kPaBlk);
    constexpr uint32_t kIdO = idesc_bf16(128, kHd) | (1u << 16);   // B is MN-major
    if (lane == 0) {
      const int t = warp == 9 ? 0 : 1;
      const uint32_t dS = tmem + t * 128, dO = tmem + 256 + t * 128;
      const uint64_t q_base = sdesc_sw128(smem_u32(sQ)), k_base = sdesc_sw128(smem_u32(sKV)),
                     v_base = sdesc_mn_sw128(smem_u32(sKV));
      int slot = 0, q_cnt = 0;                      // next block of the ring; wide pieces
      uint32_t phase = 0, p_phase = 0, tail_phase = 0;
      for (int fi = 0; ok; ++fi) {
        ok = pa_wait_one(&frag_full[fi % kPaFrags], (fi / kPaFrags) & 1, err);
        if (!ok) break;
        const PagedFrag& sf = s_frag[fi % kPaFrags];
        const int n = sf.nblk;
        const bool wide = !kNarrow && sf.rows > 128;
        const PaTail tail(sf);
        mbar_arrive(&frag_empty[fi % kPaFrags]);
        if (n == 0) break;
        // (both threads follow every phase of q_full[0], needed or not: a parity
        // tells neighbouring phases apart, no more)
        ok = pa_wait_one(&q_full[0], fi & 1, err);
        if (ok && wide && t) ok = pa_wait_one(&q_full[1], q_cnt++ & 1, err);
        const int stride = wide ? 1 : 2, j_first = wide ? 0 : t;   // split: A the even blocks, B the odd ones
        const uint64_t qd = q_base + (wide && t ? C::kBytes >> 4 : 0);
        if (t && (wide || n == 1)) mbar_arrive(&q_empty[0]);       // B does not read A's rows
        // Block `at` of the piece, in ring order; those before it that only the
        // other accumulator uses are handed on.
        int i = 0;
        auto step = [&]() {
          ok = pa_wait_one(&kv_full[slot], phase, err);
          const int s = slot;
          if (++slot == ST) { slot = 0; phase ^= 1; }
          ++i;
          return s;
        };
        auto take = [&](int at) {
          while (ok && i < at) mbar_arrive(&kv_empty[step()]);
          return ok ? step() : 0;
        };
#pragma unroll 1
        for (int j = j_first - stride; j < n && ok; j += stride) {
          // the product with V of block j, then the scores of block jn
          const int jn = j + stride;
          const bool do_v = j >= 0, do_k = jn < n;
          int v_slot = 0, k_slot = 0;
          if (do_v) v_slot = take(wide ? 2 * j + 1 : j == n - 1 ? 2 * n - 1 : 2 * j + 2);
          if (do_k && ok) k_slot = take(wide ? 2 * jn : jn == 0 ? 0 : 2 * jn - 1);
          if (do_v && ok) {
            if (tail.clear && j == n - 1) {
              // warp 10 clears the rows past the last key once every user of the
              // block is here (the softmax still runs)
              mbar_arrive(&v_last);
              if (!wide) mbar_arrive(&v_last);
              ok = pa_wait_one(&v_tail[t], tail_phase, err);
              tail_phase ^= 1;
            }
          }
          if (!ok) break;
          tc_fence_after();
          if (do_v) {
            // P comes in two parts (see kPaPart), so most of the product runs
            // under the exponentials of the rest
            const uint64_t vd = v_base + v_slot * (C::kBytes >> 4);
            const uint32_t acc = j > j_first ? 1u : 0u;
            const int steps = j == n - 1 ? tail.steps : kPaBlk / 16;
            ok = pa_wait_one(&p_part[t], p_phase, err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kPaPart / 16; ++kk)
              if (kk < steps) tc_mma_bf16_ta(dO, dS + kk * 8, vd + kk * (2048 >> 4), kIdO, kk > 0 ? 1u : acc);
            ok = pa_wait_one(&p_full[t], p_phase, err);
            p_phase ^= 1;
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int kk = kPaPart / 16; kk < kPaBlk / 16; ++kk)
              if (kk < steps) tc_mma_bf16_ta(dO, dS + kk * 8, vd + kk * (2048 >> 4), kIdO, 1u);
          }
          if (do_k) {
            const uint64_t kd = k_base + k_slot * (C::kBytes >> 4);
#pragma unroll
            for (int kk = 0; kk < kHd / 16; ++kk)
              tc_mma_bf16(dS, qd + (kk >> 2) * (16384 >> 4) + 2 * (kk & 3), kd + (kk >> 2) * (16384 >> 4) + 2 * (kk & 3),
                          kIdS, kk > 0 ? 1u : 0u);
            tc_commit(&s_full[t]);
            tc_commit(&kv_empty[k_slot]);
            if (jn + stride >= n) tc_commit(&q_empty[wide ? t : 0]);   // the query rows' space is free
          } else if (do_v) {
            tc_commit(&o_done[t]);
          }
          if (do_v) tc_commit(&kv_empty[v_slot]);
        }
        while (ok && i < 2 * n) mbar_arrive(&kv_empty[step()]);
      }
      // and so have this thread's products
      tc_commit(&mma_end[t]);
      pa_wait_one(&mma_end[t], 0, err);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---------------- query rows ----------------
    // 16 bytes at a time, asynchronously, in the layout the MMA reads.  Rows
    // past the piece's end keep what is there: no row of the products mixes
    // with another.
    constexpr int kPer = kHd / 8, kAt = 32 / kPer;   // chunks a row, rows a pass of the warp
    const int c = lane % kPer;
    const uint32_t dst = smem_u32(sQ) + (c >> 3) * 16384;
    int used_a = 0, used_b = 0, blocks = 0, tails = 0;   // pieces loaded for; K and V blocks up to this piece; tails cleared
    for (int fi = 0; ok; ++fi) {
      ok = pa_wait(&frag_full[fi % kPaFrags], (fi / kPaFrags) & 1, err);
      if (!ok) break;
      const PagedFrag& sf = s_frag[fi % kPaFrags];
      const int n = sf.nblk, rows = sf.rows, rem0 = sf.rem0;
      const PaTail tail(sf);
      const bf16* src = (const bf16*)a.q + (long long)(sf.q0 + sf.tok0) * a.q_ts +
                        (long long)(sf.kvh * a.G + rem0) * a.q_hs + c * 8;
      warp_arrive(&frag_empty[fi % kPaFrags]);
      if (n == 0) break;
      blocks += 2 * n;
#pragma unroll 1
      for (int t = 0; t < kRows / 128 && t * 128 < rows && ok; ++t) {   // (no B in a split piece)
        int& used = t ? used_b : used_a;
        if (used > 0) ok = pa_wait(&q_empty[t], (used - 1) & 1, err);
        if (!ok) break;
        ++used;
        const int last = min(rows, t * 128 + 128);
#pragma unroll 4
        for (int row = t * 128 + lane / kPer; row < last; row += kAt) {
          const int tk = a.by_g.div(rem0 + row);
          cp_async_16(dst + row * 128 + t * (C::kBytes - 16384) + (((c & 7) ^ (row & 7)) << 4),
                      src + (long long)tk * a.q_ts + (long long)(row - tk * a.G) * a.q_hs);
        }
        cp_async_wait_all();
        fence_async_smem();
        warp_arrive(&q_full[t]);
      }
      if (ok && tail.clear) {
        const int s = (blocks - 1) % ST;
        ok = pa_wait(&v_last, tails++ & 1, err);
        if (!ok) break;
        const int n16 = (tail.steps * 16 - tail.valid) * 8;
#pragma unroll
        for (int g = 0; g < C::kHalves; ++g)
#pragma unroll 1
          for (int i = lane; i < n16; i += 32)
            *reinterpret_cast<uint4*>(sKV + s * C::kBytes + g * 16384 + tail.valid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
        const bool wide = !kNarrow && rows > 128;
        if (lane == 0) {
          if (wide || ((n - 1) & 1) == 0) mbar_arrive(&v_tail[0]);
          if (wide || ((n - 1) & 1) == 1) mbar_arrive(&v_tail[1]);
        }
      }
    }
  } else {
    // ---------------- softmax ----------------
    const int t = warp >> 2, wt = warp & 3;
    const int r = threadIdx.x & 127;               // TMEM lane, row of the accumulator
    const uint32_t lane_off = (uint32_t)(wt * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lane_off, tO = tmem + 256 + t * 128 + lane_off;
    int s_cnt = 0, done_cnt = 0, half_cnt = 0;
    uint32_t turn_phase = t ? 0 : 1;               // (A's first turn is free)
    for (int fi = 0; ok; ++fi) {
      ok = pa_wait(&frag_full[fi % kPaFrags], (fi / kPaFrags) & 1, err);
      if (!ok) break;
      const PagedFrag& sf = s_frag[fi % kPaFrags];
      const int nblk = sf.nblk, kb0 = sf.kb0, part = sf.part;
      const bool split = kNarrow || sf.rows <= 128, first = sf.first, whole = sf.whole;
      const int row_t = split ? r : t * 128 + r;     // row of the tile
      const int n_rows = min(128, sf.rows - (split ? 0 : t * 128));
      const int n_cont = sf.n_cont, rem0 = sf.rem0;
      const int tk = a.by_g.div(rem0 + row_t);
      const int tok = sf.q0 + sf.tok0 + tk, head = sf.kvh * a.G + rem0 + row_t - tk * a.G;
      const int vis = min(sf.vis_max, sf.vis0 + sf.tok0 + tk);
      warp_arrive(&frag_empty[fi % kPaFrags]);
      if (nblk == 0) break;
      const bool turns = !split;                      // (a split piece waits for memory, not for exponentials)
      const bool warp_on = wt * 32 < n_rows;         // rows past the piece's end do no work
      float m_run = -INFINITY, l_run = 0.0f;
      const int step = split ? 2 : 1, j0 = split ? t : 0;
#pragma unroll 1
      for (int j = j0; j < nblk; j += step) {
        ok = pa_wait(&s_full[t], s_cnt++ & 1, err);
        if (!ok) break;
        if (warp_on) {
          const int key0 = (kb0 + j) * kPaBlk;
          uint32_t w[kPaBlk];
#pragma unroll
          for (int q = 0; q < kPaBlk; q += 32) tmem_ld32_nw(tS + q, w + q);
          tmem_wait_ld();
          if (__any_sync(0xffffffffu, key0 + kPaBlk > vis)) {
#pragma unroll
            for (int c = 0; c < kPaBlk; ++c)
              if (key0 + c >= vis) w[c] = 0xFF800000u;   // -inf
          }
          float mt[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) mt[u] = __uint_as_float(w[u]);
#pragma unroll
          for (int c = 4; c < kPaBlk - 4; c += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u) mt[u] = max3(mt[u], __uint_as_float(w[c + u]), __uint_as_float(w[c + u + 4]));
#pragma unroll
          for (int u = 0; u < 4; ++u) mt[u] = fmaxf(mt[u], __uint_as_float(w[kPaBlk - 4 + u]));
          const float mx = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3])) * a.scale_log2;
          // The reference moves only when the block's maximum passes it by more
          // than 8 (P stays below 256), so O is rarely rescaled; the sum uses
          // the same reference, so the quotient does not change.
          const float m_new = (m_run == -INFINITY || mx > m_run + 8.0f) ? mx : m_run;
          const float alpha = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - m_new);
          const float nm = m_new == -INFINITY ? 0.0f : -m_new;
          // S(j) was complete, so the PV before it, issued earlier, was too: O is ours
          if (j > j0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll 1
            for (int q = 0; q < kHd; q += 16) {
              uint32_t o[16];
              tmem_ld16_nw(tO + q, o);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u) o[u] = __float_as_uint(__uint_as_float(o[u]) * alpha);
              tmem_st16_nw(tO + q, o);
            }
          }
          // The exponential unit is what both softmaxes need most; the warps of A
          // and B on it take turns, so one exponentiates while the other's MMAs run.
          if (turns) {
            ok = pa_wait(&turn[t][wt], turn_phase, err);
            turn_phase ^= 1;
            if (!ok) break;
          }
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
          // P is rounded to bf16 for the MMA (its operands are 16-bit); the row
          // sum adds the fp32 values.  By itself this puts the output off by
          // 0.0013 of its size (root mean square), the rounding of the output to
          // bf16 by 0.0017, both together by 0.0021.
#pragma unroll
          for (int ch = 0; ch < kPaBlk; ch += 32) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float p0 = ex2_approx(fmaf(__uint_as_float(w[ch + 2 * q]), a.scale_log2, nm));
              const float p1 = ex2_approx(fmaf(__uint_as_float(w[ch + 2 * q + 1]), a.scale_log2, nm));
              ls[q & 3] += p0 + p1;
              const __nv_bfloat162 pr = __floats2bfloat162_rn(p0, p1);
              pk[q] = *reinterpret_cast<const uint32_t*>(&pr);
            }
            tmem_st16_nw(tS + ch / 2, pk);
            if (ch + 32 == kPaPart) {
              tmem_wait_st();
              tc_fence_before();
              warp_arrive(&p_part[t]);
            }
          }
          if (turns && lane == 0) mbar_arrive(&turn[1 - t][wt]);
          l_run = l_run * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
          m_run = m_new;
          tmem_wait_st();
        } else {
          if (turns) {
            ok = pa_wait(&turn[t][wt], turn_phase, err);
            turn_phase ^= 1;
            if (!ok) break;
            warp_arrive(&turn[1 - t][wt]);
          }
          warp_arrive(&p_part[t]);
        }
        tc_fence_before();
        warp_arrive(&p_full[t]);
      }
      // ---------------- epilogue ----------------
      const bool both = split && nblk > 1;           // B has a half to join
      if (ok && (t == 0 || !split || both)) ok = pa_wait(&o_done[t], done_cnt++ & 1, err);
      if (!ok) break;
      if (split && t == 1) {
        if (both) {
          // A reads O_B from tensor memory (its lanes are the same rows)
          s_half[r][0] = m_run;
          s_half[r][1] = l_run;
          tc_fence_before();
          warp_arrive(&half_full);
          ok = pa_wait(&half_empty, half_cnt++ & 1, err);
        }
        continue;
      }
      float w0 = 1.0f, w1 = 0.0f;
      if (both) {
        ok = pa_wait(&half_full, half_cnt++ & 1, err);
        if (!ok) break;
        const float m1 = s_half[r][0], l1 = s_half[r][1];
        const float m = fmaxf(m_run, m1);
        w0 = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - m);
        w1 = m1 == -INFINITY ? 0.0f : ex2_approx(m1 - m);
        l_run = l_run * w0 + l1 * w1;
        m_run = m;
      }
      if (warp_on) {
        const long long rows_all = (long long)a.b.n_tokens * a.n_heads, row = (long long)tok * a.n_heads + head;
        const bool final = whole && a.b.prefix_len == 0;
        // (a sum of 0: no visible key; not a number stays that)
        const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
        const float l2 = l_run == 0.0f ? -INFINITY : m_run + log2f(l_run);
        w0 *= inv;
        w1 = both ? w1 * inv : 0.0f;
        // where the row goes, as bytes
        char* dst = nullptr;
        if (r < n_rows) {
          if (first)
            a.meta[part * rows_all + row] = final ? make_int2(-1, 0) : make_int2((int)blockIdx.x, n_cont * kRows + row_t);
          const long long at = first ? part * rows_all + row : (long long)blockIdx.x * kRows + row_t;
          if (final) {
            dst = (char*)((bf16*)a.out + (long long)tok * a.o_ts + (long long)head * a.o_hs);
            if (a.lse) a.lse[row] = l2 * kLn2;
          } else {
            dst = (char*)((first ? a.part_o : a.slot_o) + at * kHd);
            (first ? a.part_lse : a.slot_lse)[at] = l2;
          }
        }
        uint8_t* stage = sStage + warp * kPaStage;
        const int cols = final ? 64 : 32;            // columns of 128 bytes
        const int live = min(32, n_rows - wt * 32);
        // (by the piece, never by values: rows past the end may hold anything, and
        // past B's columns there is no tensor memory)
        const bool add_b = both;
#pragma unroll 1
        for (int q = 0; q < kHd; q += 16) {
          uint32_t o[16];
          tmem_ld16_nw(tO + q, o);
          if (add_b) {
            uint32_t ob[16];
            tmem_ld16_nw(tO + 128 + q, ob);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 16; ++u) {
              const float x = w0 == 0.0f ? 0.0f : __uint_as_float(o[u]) * w0;
              o[u] = __float_as_uint(w1 == 0.0f ? x : fmaf(__uint_as_float(ob[u]), w1, x));
            }
          } else {
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 16; ++u) o[u] = w0 == 0.0f ? 0u : __float_as_uint(__uint_as_float(o[u]) * w0);
          }
          if (final) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const __nv_bfloat162 pr = __floats2bfloat162_rn(__uint_as_float(o[2 * u]), __uint_as_float(o[2 * u + 1]));
              o[u] = *reinterpret_cast<const uint32_t*>(&pr);
            }
          }
          const int chunks = final ? 2 : 4;          // of 16 bytes
          if (kNarrow) {                             // few rows: each lane stores its own
#pragma unroll
            for (int u = 0; u < 4; ++u)
              if (u < chunks && dst)
                *reinterpret_cast<uint4*>(dst + q * (128 / cols) + u * 16) =
                    make_uint4(o[u * 4], o[u * 4 + 1], o[u * 4 + 2], o[u * 4 + 3]);
            continue;
          }
          // 32 rows x 128 bytes through shared memory, chunk c of row r at
          // c ^ (r & 7): a warp then stores whole 128-byte lines, four rows an
          // instruction (a thread storing its own row touches 32 lines)
          const int c0 = final ? (q & 48) / 8 : (q & 16) / 4;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (u < chunks)
              *reinterpret_cast<uint4*>(stage + lane * 128 + (((c0 + u) ^ (lane & 7)) << 4)) =
                  make_uint4(o[u * 4], o[u * 4 + 1], o[u * 4 + 2], o[u * 4 + 3]);
          if ((q + 16) % cols) continue;             // the rest of the 128 bytes follows
          const int at = (q + 16 - cols) * (128 / cols);
          __syncwarp();
#pragma unroll 4
          for (int i = 0; i < 32; i += 4) {
            if (i >= live) break;
            const int rr = i + (lane >> 3), c = lane & 7;
            char* to = (char*)__shfl_sync(0xffffffffu, (unsigned long long)dst, rr);
            if (to)
              *reinterpret_cast<uint4*>(to + at + c * 16) =
                  *reinterpret_cast<const uint4*>(stage + rr * 128 + ((c ^ (rr & 7)) << 4));
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      if (both) warp_arrive(&half_empty);
    }
    tmem_wait_st();   // (a wait that ran out leaves the loop between a store and its end)
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}
