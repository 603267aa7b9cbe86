// The paged attention of dg_paged_attn.cuh on the tensor cores (bf16).
//
// One CTA per SM, 320 threads:
//   warps 0-3, 4-7  softmax of the accumulators A and B (thread = query row =
//                   TMEM lane), the query rows into shared memory, epilogue;
//   warp 8          walks the CTA's interval and loads K and V blocks of 128
//                   keys by TMA, page by page;
//   warp 9          issues the MMAs.
// A piece of more than 128 rows runs wide: A holds its first 128 rows, B the
// rest, and both use every K/V block.  A piece of at most 128 rows (single
// tokens, the end of a ragged sequence) runs split: A and B hold the same rows
// and take every other key block, so twice the bytes are in flight and two
// softmaxes run side by side; the two halves join at the end.
//
// S = Q K^T goes to TMEM; the softmax thread reads its row, writes P back over
// it as bf16, and O += P V takes P from TMEM, so P never crosses shared
// memory.  V stays as the cache holds it ([key][component]): the MMA reads it
// as an MN-major operand.  TMEM columns: S_A/P_A [0,128), S_B/P_B [128,256),
// O_A [256,256+hd), O_B [384,384+hd).
#pragma once
#include "dg_paged_attn.cuh"

constexpr int kPaThreads = 320;
constexpr int kPaRows = 256, kPaBlk = 128;
constexpr int kPaFrags = 4;   // pieces announced ahead

template <int kHd>
struct PaTc {
  static constexpr int kHalves = kHd / 64;           // 128-byte column groups of a row
  static constexpr int kBytes = 128 * kHd * 2;       // 128 rows of Q, K or V
  static constexpr int kStages = kHd == 128 ? 5 : 10;
  static constexpr int kSmem = (2 + kStages) * kBytes + 1024;
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

template <int kHd>
__global__ void __launch_bounds__(kPaThreads, 1)
k_paged_attn_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ PagedAttnArgs a) {
  using C = PaTc<kHd>;
  constexpr int ST = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;                       // A, B
  uint8_t* sKV = smem + 2 * C::kBytes;      // ring of K and V blocks
  __shared__ __align__(8) uint64_t kv_full[ST], kv_empty[ST], frag_full[kPaFrags], frag_empty[kPaFrags];
  __shared__ __align__(8) uint64_t q_full[2], s_full[2], p_full[2], o_done[2], half_full, half_empty;
  __shared__ PagedFrag s_frag[kPaFrags];
  __shared__ float s_half[128][2];          // split: maximum and sum of B's half, per row
  __shared__ long long s_tmp[kPaThreads / 32 + 1];
  __shared__ int s_found;
  __shared__ uint32_t tmem_base;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int* const err = a.b.status;
  pdl_launch();
  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) { mbar_init(&kv_full[s], 1); mbar_init(&kv_empty[s], 1); }
    for (int s = 0; s < kPaFrags; ++s) { mbar_init(&frag_full[s], 1); mbar_init(&frag_empty[s], 9); }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 128);
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[t], 128);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(&half_full, 128);
    mbar_init(&half_empty, 128);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&tmem_base, 512);
  if (warp == 8 && lane == 0) { prefetch_tmap(&tmK); prefetch_tmap(&tmV); }
  pdl_wait();
  PagedWalk<kPaRows, kPaBlk> walk(a);
  const bool any = walk.template begin<kPaThreads>(s_tmp, s_found);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;

  if (!any) {
  } else if (warp == 8) {
    // ---------------- walk and TMA ----------------
    const int page_shift = a.b.page_shift, page = 1 << page_shift;
    int cnt = 0;
    bool ok = true;
    for (int fi = 0; ok; ++fi) {
      const PagedFrag f = walk.next();
      const int slot = fi % kPaFrags;
      if (fi >= kPaFrags)
        ok = __all_sync(0xffffffffu, mbar_wait(&frag_empty[slot], ((fi / kPaFrags) & 1) ^ 1, err, kStatusTimeout));
      if (!ok) break;
      if (lane == 0) {
        s_frag[slot] = f;
        mbar_arrive(&frag_full[slot]);
      }
      if (f.nblk == 0) break;
      // The page ids of 32 pages are held by the 32 lanes, for K and for V apart
      // (in a split piece V trails K by two blocks).
      int base[2] = {-64, -64}, ids[2] = {0, 0};
      auto load = [&](int which, int j) {
        const int s = cnt % ST;
        if (cnt >= ST) {
          ok = __all_sync(0xffffffffu, mbar_wait(&kv_empty[s], ((cnt / ST) & 1) ^ 1, err, kStatusTimeout));
          if (!ok) return;
        }
        ++cnt;
        const int key0 = (f.kb0 + j) * kPaBlk, pg0 = key0 >> page_shift;
        // pages of the block that hold a visible key (none in a block that is there for its zeros)
        const int per_blk = page >= kPaBlk ? 1 : kPaBlk >> page_shift;
        const int n_pg = max(0, min(per_blk, f.pages - pg0));
        const int w = which;
        if (pg0 < base[w] || pg0 + per_blk > base[w] + 32) {
          base[w] = pg0;
          int id = -1;
          if (pg0 + lane < f.pages) {
            id = f.page_list[pg0 + lane];
            if (id < 0 || id >= a.b.n_pages) {
              dev_error(err, kStatusState);
              id = a.b.n_pages;   // past the tensor's end: reads as zeros
            }
          }
          ids[w] = id;
        }
        const CUtensorMap* map = which ? &tmV : &tmK;
        const uint32_t dst = smem_u32(sKV + s * C::kBytes);
        if (page >= kPaBlk) {
          const int id = __shfl_sync(0xffffffffu, ids[w], pg0 - base[w]);
          if (lane == 0) {
            mbar_expect_tx(&kv_full[s], n_pg ? C::kBytes : 0);
            if (n_pg) tma_load_4d(dst, map, 0, key0 & (page - 1), 0, id * a.n_kv_heads + f.kvh, &kv_full[s]);
          }
        } else {
          if (lane == 0) mbar_expect_tx(&kv_full[s], n_pg * page * kHd * 2);
          __syncwarp();
          const int pi = lane / C::kHalves, half = lane % C::kHalves;
          const int id = __shfl_sync(0xffffffffu, ids[w], (pg0 - base[w] + pi) & 31);
          if (pi < n_pg)
            tma_load_4d(dst + half * 16384 + pi * page * 128, map, 0, 0, half, id * a.n_kv_heads + f.kvh,
                        &kv_full[s]);
        }
        __syncwarp();
      };
      // in the order the MMAs use them
      load(0, 0);
      if (f.rows > 128) {
        for (int j = 0; j < f.nblk && ok; ++j) {
          load(1, j);
          if (ok && j + 1 < f.nblk) load(0, j + 1);
        }
      } else {
        if (ok && f.nblk > 1) load(0, 1);
        for (int j = 0; j < f.nblk && ok; ++j) {
          load(1, j);
          if (ok && j + 2 < f.nblk) load(0, j + 2);
        }
      }
    }
  } else if (warp == 9) {
    // ---------------- MMA issue ----------------
    constexpr uint32_t kIdS = idesc_bf16(128, kPaBlk);
    constexpr uint32_t kIdO = idesc_bf16(128, kHd) | (1u << 16);   // B is MN-major
    int cnt = 0, p_cnt[2] = {0, 0}, q_cnt = 0;   // q_cnt: wide pieces
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, err, kStatusTimeout));
      tc_fence_after();
    };
    auto take = [&]() {
      const int s = cnt % ST;
      wait(&kv_full[s], (cnt / ST) & 1);
      ++cnt;
      return s;
    };
    auto qk = [&](int t, int q, int s) {
      if (!ok || lane != 0) return;
      const uint32_t qa = smem_u32(sQ + q * C::kBytes), ka = smem_u32(sKV + s * C::kBytes);
#pragma unroll
      for (int kk = 0; kk < kHd / 16; ++kk)
        tc_mma_bf16(tmem + t * 128, sdesc_sw128(qa + (kk >> 2) * 16384) + 2 * (kk & 3),
                    sdesc_sw128(ka + (kk >> 2) * 16384) + 2 * (kk & 3), kIdS, kk > 0 ? 1u : 0u);
      tc_commit(&s_full[t]);
    };
    auto pv = [&](int t, int s, bool acc) {
      wait(&p_full[t], p_cnt[t]++ & 1);
      if (!ok || lane != 0) return;
      const uint32_t va = smem_u32(sKV + s * C::kBytes);
#pragma unroll
      for (int kk = 0; kk < kPaBlk / 16; ++kk)
        tc_mma_bf16_ta(tmem + 256 + t * 128, tmem + t * 128 + kk * 8, sdesc_mn_sw128(va + kk * 2048), kIdO,
                       acc || kk > 0 ? 1u : 0u);
    };
    auto free_kv = [&](int s) {
      if (ok && lane == 0) tc_commit(&kv_empty[s]);
    };
    // Keys past the last visible one are masked in S, but 0 times whatever
    // their values hold (the cache may hold anything there) is not 0 for an
    // infinity or a NaN: their rows of V become zeros.
    auto clear_tail = [&](const PagedFrag& f, int j, int s) {
      const int valid = f.limit - (f.kb0 + j) * kPaBlk;
      if (valid >= kPaBlk) return;
      const int n = (kPaBlk - max(valid, 0)) * 8;
      for (int h = 0; h < C::kHalves; ++h)
        for (int i = lane; i < n; i += 32)
          *reinterpret_cast<uint4*>(sKV + s * C::kBytes + h * 16384 + max(valid, 0) * 128 + i * 16) =
              make_uint4(0, 0, 0, 0);
      fence_async_smem();
      __syncwarp();
    };
    for (int fi = 0; ok; ++fi) {
      wait(&frag_full[fi % kPaFrags], (fi / kPaFrags) & 1);
      if (!ok) break;
      const PagedFrag f = s_frag[fi % kPaFrags];
      __syncwarp();
      if (lane == 0) mbar_arrive(&frag_empty[fi % kPaFrags]);
      if (f.nblk == 0) break;
      wait(&q_full[0], fi & 1);
      if (f.rows > 128) {
        wait(&q_full[1], q_cnt++ & 1);
        int k = take();
        qk(0, 0, k);
        qk(1, 1, k);
        free_kv(k);
        for (int j = 0; j < f.nblk && ok; ++j) {
          const int v = take();
          clear_tail(f, j, v);
          const bool more = j + 1 < f.nblk;
          pv(0, v, j > 0);
          if (more) {
            k = take();
            qk(0, 0, k);
          } else if (ok && lane == 0) {
            tc_commit(&o_done[0]);
          }
          pv(1, v, j > 0);
          free_kv(v);
          if (more) {
            qk(1, 1, k);
            free_kv(k);
          } else if (ok && lane == 0) {
            tc_commit(&o_done[1]);
          }
        }
      } else {
        for (int t = 0; t < 2 && t < f.nblk; ++t) {
          const int k = take();
          qk(t, 0, k);
          free_kv(k);
        }
        for (int j = 0; j < f.nblk && ok; ++j) {
          const int t = j & 1, v = take();
          clear_tail(f, j, v);
          pv(t, v, j > 1);
          free_kv(v);
          if (j + 2 < f.nblk) {
            const int k = take();
            qk(t, 0, k);
            free_kv(k);
          } else if (ok && lane == 0) {
            tc_commit(&o_done[t]);
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ---------------- softmax ----------------
    const int t = warp >> 2, wt = warp & 3;
    const int r = threadIdx.x & 127;               // TMEM lane, row of the accumulator
    const uint32_t lane_off = (uint32_t)(wt * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lane_off, tO = tmem + 256 + t * 128 + lane_off;
    int s_cnt = 0, done_cnt[2] = {0, 0}, half_cnt = 0;
    bool ok = true;
    // tcgen05 loads and stores are warp-collective: outcomes are agreed on
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity, err, kStatusTimeout));
      tc_fence_after();
    };
    for (int fi = 0; ok; ++fi) {
      wait(&frag_full[fi % kPaFrags], (fi / kPaFrags) & 1);
      if (!ok) break;
      const PagedFrag f = s_frag[fi % kPaFrags];
      __syncwarp();
      if (lane == 0) mbar_arrive(&frag_empty[fi % kPaFrags]);
      if (f.nblk == 0) break;
      const bool split = f.rows <= 128;
      const int first_row = split ? 0 : t * 128;       // of the tile
      const int n_rows = min(128, f.rows - first_row);
      // query rows, 16 bytes at a time, in the layout the MMA reads
      if (!split || t == 0) {
        uint8_t* dst = sQ + t * C::kBytes;
        for (int i = r; i < n_rows * (kHd / 8); i += 128) {
          const int row = i / (kHd / 8), c = i % (kHd / 8), gr = f.row0 + first_row + row;
          const uint4 v = *reinterpret_cast<const uint4*>((const bf16*)a.q + (long long)(f.q0 + gr / a.G) * a.q_ts +
                                                          (long long)(f.kvh * a.G + gr % a.G) * a.q_hs + c * 8);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v;
        }
        fence_async_smem();
        mbar_arrive(&q_full[t]);
      }

      const int gr = f.row0 + first_row + r;
      const int vis = min(f.vis_max, f.vis0 + gr / a.G);
      const bool warp_on = wt * 32 < n_rows;           // rows past the piece's end do no work
      float m_run = -INFINITY, l_run = 0.0f;
      const int step = split ? 2 : 1, j0 = split ? t : 0;
      for (int j = j0; j < f.nblk && ok; j += step) {
        wait(&s_full[t], s_cnt++ & 1);
        if (!ok) break;
        if (warp_on) {
          const int key0 = (f.kb0 + j) * kPaBlk;
          float v[kPaBlk];
          {
            uint32_t w[kPaBlk / 16][16];
#pragma unroll
            for (int q = 0; q < kPaBlk / 16; ++q) tmem_ld16_nw(tS + q * 16, w[q]);
            tmem_wait_ld();
#pragma unroll
            for (int q = 0; q < kPaBlk / 16; ++q)
#pragma unroll
              for (int u = 0; u < 16; ++u) v[q * 16 + u] = __uint_as_float(w[q][u]);
          }
          if (__any_sync(0xffffffffu, key0 + kPaBlk > vis)) {
#pragma unroll
            for (int c = 0; c < kPaBlk; ++c)
              if (key0 + c >= vis) v[c] = -INFINITY;
          }
          float mt[8];
#pragma unroll
          for (int c = 0; c < 8; ++c) mt[c] = fmaxf(v[c], v[c + 8]);
#pragma unroll
          for (int c = 16; c < kPaBlk; ++c) mt[c & 7] = fmaxf(mt[c & 7], v[c]);
          const float mx = fmaxf(fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3])),
                                 fmaxf(fmaxf(mt[4], mt[5]), fmaxf(mt[6], mt[7]))) * a.scale_log2;
          // The reference moves only when the block's maximum passes it by more
          // than 8 (P stays below 256), so O is rarely rescaled; the sum uses
          // the same reference, so the quotient does not change.
          const float m_new = (m_run == -INFINITY || mx > m_run + 8.0f) ? mx : m_run;
          const float alpha = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - m_new);
          const float nm = m_new == -INFINITY ? 0.0f : -m_new;
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
          // P is rounded to bf16 for the MMA (its operands are 16-bit); the row
          // sum adds the fp32 values
#pragma unroll
          for (int ch = 0; ch < kPaBlk / 32; ++ch) {
            uint32_t pk[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const float p0 = ex2_approx(fmaf(v[ch * 32 + 2 * q], a.scale_log2, nm));
              const float p1 = ex2_approx(fmaf(v[ch * 32 + 2 * q + 1], a.scale_log2, nm));
              ls[q & 3] += p0 + p1;
              const __nv_bfloat162 pr = __floats2bfloat162_rn(p0, p1);
              pk[q] = *reinterpret_cast<const uint32_t*>(&pr);
            }
            tmem_st16_nw(tS + ch * 16, pk);
          }
          // S(j) was complete, so the PV before it, issued earlier, was too: O is ours
          if (j > j0 && __any_sync(0xffffffffu, alpha != 1.0f)) {
#pragma unroll
            for (int q = 0; q < kHd / 32; ++q) {
              uint32_t o[2][16];
              tmem_ld16_nw(tO + q * 32, o[0]);
              tmem_ld16_nw(tO + q * 32 + 16, o[1]);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                o[0][u] = __float_as_uint(__uint_as_float(o[0][u]) * alpha);
                o[1][u] = __float_as_uint(__uint_as_float(o[1][u]) * alpha);
              }
              tmem_st16_nw(tO + q * 32, o[0]);
              tmem_st16_nw(tO + q * 32 + 16, o[1]);
            }
          }
          l_run = l_run * alpha + ((ls[0] + ls[1]) + (ls[2] + ls[3]));
          m_run = m_new;
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&p_full[t]);
      }
      // ---------------- epilogue ----------------
      if (!ok) break;
      const bool both = split && f.nblk > 1;           // B has a half to join
      if (t == 0 || !split || both) wait(&o_done[t], done_cnt[t]++ & 1);
      if (split && t == 1) {
        if (both) {
          // A's MMAs no longer read Q: its space takes B's half, float4 c of
          // row r at c ^ (r & 15)
          wait(&o_done[0], done_cnt[0] & 1);
          float4* stage = reinterpret_cast<float4*>(sQ);
          if (ok && warp_on) {
#pragma unroll
            for (int q = 0; q < kHd / 16; ++q) {
              uint32_t o[16];
              tmem_ld16_nw(tO + q * 16, o);
              tmem_wait_ld();
#pragma unroll
              for (int u = 0; u < 4; ++u)
                stage[r * (kHd / 4) + ((q * 4 + u) ^ (r & 15))] =
                    make_float4(__uint_as_float(o[u * 4]), __uint_as_float(o[u * 4 + 1]),
                                __uint_as_float(o[u * 4 + 2]), __uint_as_float(o[u * 4 + 3]));
            }
            s_half[r][0] = m_run;
            s_half[r][1] = l_run;
          }
          tc_fence_before();
          mbar_arrive(&half_full);
          wait(&half_empty, half_cnt++ & 1);
        }
        ++done_cnt[0];
        continue;
      }
      float w0 = 1.0f, w1 = 0.0f;
      if (both) {
        wait(&half_full, half_cnt++ & 1);
        if (ok && warp_on) {
          const float m1 = s_half[r][0], l1 = s_half[r][1];
          const float m = fmaxf(m_run, m1);
          w0 = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - m);
          w1 = m1 == -INFINITY ? 0.0f : ex2_approx(m1 - m);
          l_run = l_run * w0 + l1 * w1;
          m_run = m;
        }
      }
      if (ok && warp_on) {
        const bool valid = r < n_rows;
        const int tok = f.q0 + gr / a.G, head = f.kvh * a.G + gr % a.G;
        const long long row = (long long)tok * a.n_heads + head;
        const float inv = l_run > 0.0f ? 1.0f / l_run : 0.0f;
        const float l2 = l_run > 0.0f ? m_run + log2f(l_run) : -INFINITY;
        w0 = l_run > 0.0f ? w0 * inv : 0.0f;
        w1 *= inv;
        PagedDest d;
        d.o = nullptr;
        d.final = false;
        if (valid) {
          d = paged_dest<kPaRows>(a, f, first_row + r, kHd, row);
          if (!d.final) *d.lse = l2;
          else if (a.lse) a.lse[row] = l2 * kLn2;
        }
        const float4* stage = reinterpret_cast<const float4*>(sQ);
        bf16* dst = (bf16*)a.out + (long long)tok * a.o_ts + (long long)head * a.o_hs;
#pragma unroll
        for (int q = 0; q < kHd / 16; ++q) {
          uint32_t o[16];
          tmem_ld16_nw(tO + q * 16, o);
          tmem_wait_ld();
          float x[16];
#pragma unroll
          for (int u = 0; u < 16; ++u) x[u] = w0 == 0.0f ? 0.0f : __uint_as_float(o[u]) * w0;
          if (both && w1 != 0.0f) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float4 s4 = stage[r * (kHd / 4) + ((q * 4 + u) ^ (r & 15))];
              x[u * 4] += s4.x * w1;
              x[u * 4 + 1] += s4.y * w1;
              x[u * 4 + 2] += s4.z * w1;
              x[u * 4 + 3] += s4.w * w1;
            }
          }
          if (!valid) continue;
          if (d.final) {
            uint32_t w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const __nv_bfloat162 p = __floats2bfloat162_rn(x[2 * u], x[2 * u + 1]);
              w[u] = *reinterpret_cast<const uint32_t*>(&p);
            }
            reinterpret_cast<uint4*>(dst + q * 16)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst + q * 16)[1] = make_uint4(w[4], w[5], w[6], w[7]);
          } else {
#pragma unroll
            for (int u = 0; u < 4; ++u)
              reinterpret_cast<float4*>(d.o + q * 16)[u] =
                  make_float4(x[u * 4], x[u * 4 + 1], x[u * 4 + 2], x[u * 4 + 3]);
          }
        }
      }
      tc_fence_before();
      if (both) {
        // the next piece's query rows, which each warp loads for all of them,
        // take the space the other warps may still be reading
        mbar_arrive(&half_empty);
        wait(&half_empty, (half_cnt - 1) & 1);
      }
      if (t == 1) ++done_cnt[0];   // B follows A's count of finished pieces
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}
