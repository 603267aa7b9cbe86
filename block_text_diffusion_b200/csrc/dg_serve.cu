// Serving operators over a paged key/value cache (include/dg.h): argument
// checks, launch choices and launches.  Nothing is kept between calls but an
// error that a call without a status word met.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <utility>

#include "../../include/dg.h"
#include "../../include/dg_test.h"
#include "dg_headrows.cuh"
#include "dg_paged_attn.cuh"
#include "dg_paged_attn_tc.cuh"

namespace {

typedef CUresult (*PFN_encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                               const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                               CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

PFN_encode lookup_encode() {
  cudaDriverEntryPointQueryResult q;
  void* p = nullptr;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return (PFN_encode)p;
}

// Pages [n_pages * heads][page][hd] of bf16 as {64 components, rows of a page,
// groups of 64 components, pages x heads}: a box is one page's (or 128) rows of
// one group, or of every group when a block of 128 keys lies in one page.
bool page_map(CUtensorMap* m, const void* base, long long outer, int page, int hd) {
  static const PFN_encode fn = lookup_encode();
  if (!fn) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)page, (cuuint64_t)(hd / 64), (cuuint64_t)outer};
  cuuint64_t strides[3] = {(cuuint64_t)hd * 2, 128, (cuuint64_t)page * hd * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)std::min(page, 128), page >= 128 ? (cuuint32_t)(hd / 64) : 1u, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Programmatic launch: the kernels wait (griddepcontrol.wait) before they touch
// global memory, so only their launch and prologue overlap what runs before.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), unsigned grid, unsigned block, size_t smem, cudaStream_t s,
                   Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// The dynamic shared memory of a kernel, raised once on each device (the
// attribute stays; two threads that raise it at once set the same value).
template <typename K>
cudaError_t raise_smem(K kernel, int bytes, std::atomic<uint64_t>& done_on) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done_on.load(std::memory_order_acquire) & bit) return cudaSuccess;
  const cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (r == cudaSuccess) done_on.fetch_or(bit, std::memory_order_release);
  return r;
}

dg_status done(cudaError_t e) {
  if (e == cudaSuccess) return DG_OK;
  cudaGetLastError();   // the error is returned here, not left for the next call
  return DG_ERR_CUDA;
}

int elem_size(int dtype) { return dtype == DG_BF16 ? 2 : 4; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// Largest |offset| a row of heads reaches stays far inside 64 bits.  Buffers of
// no rows may have no address.
bool heads_ok(const dg_heads* h, int dtype, int64_t n_tokens) {
  const int64_t lim = (int64_t)1 << 40;
  return h && (h->data || n_tokens == 0) && aligned(h->data, elem_size(dtype)) && h->token_stride >= 0 &&
         h->head_stride >= 0 && h->token_stride < lim && h->head_stride < lim;
}

bool rope_ok(const dg_rope* r, int head_dim) {
  if (!r) return true;
  if (r->rot_dim < 0 || r->rot_dim > head_dim || r->rot_dim % 2) return false;
  return r->rot_dim == 0 || (r->inv_freq && aligned(r->inv_freq, 8));
}

bool norm_ok(const dg_head_norm* n, int dtype) {
  return !n || !n->enabled ||
         (n->eps >= 0.0f && aligned(n->q_gain, elem_size(dtype)) && aligned(n->k_gain, elem_size(dtype)));
}

bool cache_ok(const dg_paged_kv* c) {
  if (!c || !c->k || !c->v || (c->dtype != DG_FP32 && c->dtype != DG_BF16)) return false;
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->head_dim < 2 || c->head_dim > 256 || c->head_dim % 2) return false;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1))) return false;
  if ((int64_t)c->n_pages * c->n_kv_heads >= (int64_t)1 << 31) return false;
  return aligned(c->k, 16) && aligned(c->v, 16);
}

bool batch_ok(const dg_paged_kv* c, const dg_paged_batch* b) {
  if (!b || b->n_seqs < 0 || b->n_tokens < 0 || b->max_pages < 0 || b->prefix_len < 0) return false;
  if (b->n_seqs > 0 && (!b->cu_q || !b->kv_lens)) return false;
  for (const int32_t* p : {b->cu_q, b->kv_lens, b->page_table, b->prefix_pages})
    if (!aligned(p, 4)) return false;
  if (b->n_seqs > 0 && b->max_pages > 0 && (!b->page_table || b->table_stride < b->max_pages)) return false;
  // positions are int32
  if ((int64_t)b->prefix_len + (int64_t)b->max_pages * c->page_size >= (int64_t)1 << 31) return false;
  return b->prefix_len == 0 || b->prefix_pages;
}

PagedBatch device_batch(const dg_paged_kv* c, const dg_paged_batch* b, int32_t* status_word) {
  PagedBatch d{};
  d.n_seqs = b->n_seqs;
  d.n_tokens = b->n_tokens;
  d.cu_q = b->cu_q;
  d.kv_lens = b->kv_lens;
  d.table = b->page_table;
  d.table_stride = b->table_stride;
  d.max_pages = b->max_pages;
  d.prefix_pages = b->prefix_pages;
  d.prefix_len = b->prefix_len;
  d.n_pages = c->n_pages;
  while ((1 << d.page_shift) < c->page_size) ++d.page_shift;
  d.status = status_word;
  return d;
}

HeadRows head_rows(const dg_heads* h) { return HeadRows{h->data, h->token_stride, h->head_stride}; }

void set_steps(HeadRowsArgs& a, const dg_rope* rope, const dg_head_norm* norm) {
  if (rope && rope->rot_dim > 0) {
    a.inv_freq = rope->inv_freq;
    a.rot_dim = rope->rot_dim;
    a.interleaved = rope->interleaved != 0;
    a.amplitude = rope->amplitude;
  }
  if (norm && norm->enabled) {
    a.norm = 1;
    a.eps = norm->eps;
    a.q_gain = norm->q_gain;
    a.k_gain = norm->k_gain;
  }
}

template <typename T>
dg_status run_head_rows(const HeadRowsArgs& a, cudaStream_t s) {
  if (a.n_tokens == 0 || a.n_q + a.n_k == 0) return DG_OK;
  constexpr int N = Chunk<T>::kN;
  // whole chunks: every row 16-byte aligned, head_dim a power of two of chunk
  // pairs, the rotated halves whole chunks
  auto rows_ok = [](const HeadRows& h) { return aligned(h.data, 16) && h.ts % N == 0 && h.hs % N == 0; };
  const int lph = a.head_dim / (2 * N);
  bool chunks = a.head_dim % (2 * N) == 0 && (lph & (lph - 1)) == 0 && lph <= 32 && (a.rot_dim / 2) % N == 0;
  if (a.n_q) chunks = chunks && rows_ok(a.q) && rows_ok(a.qo);
  if (a.n_k) chunks = chunks && rows_ok(a.k) && (a.paged ? rows_ok(a.v) : rows_ok(a.ko));
  chunks = chunks && aligned(a.q_gain, 16) && aligned(a.k_gain, 16);
  if (!chunks) {
    const long long warps = (long long)a.n_tokens * (a.n_q + a.n_k + a.n_v);
    return done(launch(k_head_rows_any<T>, (unsigned)std::min<long long>((warps + 7) / 8, kSMs * 16), 256, 0, s, a));
  }
  int shift = 0;
  while ((1 << shift) < lph) ++shift;
  // Batches of `groups` x 32 / lph heads of one kind; a warp takes one batch
  // while the batches do not fill the SMs, all of its token's when they do
  // (its sines and cosines then serve every head).  One batch against all, us
  // (bf16, 16 + 8 heads of 128, 6 batches a token): 128 tokens 2.4 and 3.4, 256
  // 2.8 and 3.4, 400 4.2 and 3.7, 789 5.6 and 3.9, 8192 53 and 20; (fp32, 4 + 4
  // of 64, 2 batches) 1001 tokens 3.0 and 3.2, 1500 3.6 and 3.4, 2300 5.2 and
  // 4.2.  The sides meet between 1500 and 3000 batches, where the warps no
  // longer fit at once; from there to the 4736 of this rule one batch a warp
  // costs up to 1.7 us more.
  const int hpw = 32 / lph;
  auto batches = [&](int groups) {
    auto of = [&](int n) { return (n + hpw * groups - 1) / (hpw * groups); };
    return of(a.n_q) + of(a.n_k) + of(a.n_v);
  };
  const bool many = (long long)a.n_tokens * batches(1) > kSMs * 32;
  const int nb = batches(many ? 4 : 1), per = many ? nb : 1;
  const int wpt = (nb + per - 1) / per;
  const long long blocks = (long long)a.n_tokens * wpt;
  if (blocks >= (1ll << 31)) return DG_ERR_INVALID_ARG;   // (blocks of one warp, counted in 32 bits)
  const unsigned g = (unsigned)blocks;
  if (a.interleaved)
    return done(many ? launch(k_head_rows<T, 4, true>, g, 32, 0, s, a, shift, (unsigned)wpt, per)
                     : launch(k_head_rows<T, 1, true>, g, 32, 0, s, a, shift, (unsigned)wpt, per));
  return done(many ? launch(k_head_rows<T, 4, false>, g, 32, 0, s, a, shift, (unsigned)wpt, per)
                   : launch(k_head_rows<T, 1, false>, g, 32, 0, s, a, shift, (unsigned)wpt, per));
}

dg_status run_head_rows(int dtype, HeadRowsArgs& a, cudaStream_t s) {
  a.inv_dim = 1.0f / (float)a.head_dim;
  return dtype == DG_BF16 ? run_head_rows<bf16>(a, s) : run_head_rows<float>(a, s);
}

// Workspace of the paged attention; every part starts on 256 bytes.
constexpr int kPaMaxRows = 256;   // rows of the largest tile
struct PagedSpace {
  size_t meta, part_lse, slot_lse, part_o, slot_o, total;
};
PagedSpace paged_space(int64_t n_tokens, int64_t n_heads, int64_t head_dim, bool prefix) {
  const size_t rows = (size_t)(n_tokens * n_heads) * (prefix ? 2 : 1);
  PagedSpace p;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return here;
  };
  p.meta = take(rows * sizeof(int2));
  p.part_lse = take(rows * 4);
  p.slot_lse = take((size_t)kSMs * kPaMaxRows * 4);
  p.part_o = take(rows * head_dim * 4);
  p.slot_o = take((size_t)kSMs * kPaMaxRows * head_dim * 4);
  p.total = at;
  return p;
}

template <typename T, int kHd>
dg_status run_join(const PagedAttnArgs& a, int tile, cudaStream_t s) {
  const long long rows = (long long)a.b.n_tokens * a.n_heads;
  int shift = 0;   // (tiles have 2^shift rows)
  while ((1 << shift) < tile) ++shift;
  // A block per row while the rows do not fill the SMs: one token over 32768 keys
  // with 8 to 128 heads 16.8 to 18.5 us for the call, 27.9 to 43.3 without; up to
  // four rows an SM neither side wins (8 to 16 tokens of 16 heads: within 3 %).
  if (rows <= kSMs) return done(launch(k_paged_join<T, kHd, 16>, (unsigned)rows, 256, 0, s, a, shift, (int)kSMs, 1));
  const int per_block = (int)std::min<long long>(kJoinRows, (rows / (kSMs * 5) + 16) / 16 * 16);
  return done(launch(k_paged_join<T, kHd, 1>, (unsigned)((rows + per_block - 1) / per_block), 256, 0, s, a, shift,
                     (int)kSMs, per_block));
}

template <int kHd, bool kNarrow>
cudaError_t launch_tc(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, cudaStream_t s) {
  using C = PaTc<kHd, kNarrow>;
  static std::atomic<uint64_t> raised{0};
  const cudaError_t e = raise_smem(k_paged_attn_tc<kHd, kNarrow>, C::kSmem, raised);
  return e != cudaSuccess ? e : launch(k_paged_attn_tc<kHd, kNarrow>, kSMs, kPaThreads, C::kSmem, s, tk, tv, a);
}

template <int kHd>
dg_status run_paged_attention(const dg_paged_kv* c, PagedAttnArgs& a, cudaStream_t s) {
  cudaError_t e;
  // Tiles of 128 rows where the average sequence has no more (single tokens);
  // the lengths themselves are on the device.  128-row against 256-row tiles, us
  // (16 heads of 128 over 8): 16 sequences of 16 rows a key head after 1000 keys
  // 24.7 and 28.9, of 128 rows 32.9 and 36.4, of 256 rows 55.4 and 52.6.  Uneven
  // batches: 63 single tokens after 1500 keys beside a prompt of 700 tokens 102
  // and 128, of 4000 184 and 223 (128-row by this rule); 7 of them beside a
  // prompt of 2048 57.1 and 63.3, and there the rule takes the slower 256.
  const bool narrow = (long long)a.b.n_tokens * a.G <= 128ll * a.b.n_seqs;
  if (c->dtype == DG_BF16) {
    CUtensorMap tk, tv;
    const long long outer = (long long)c->n_pages * c->n_kv_heads;
    if (!page_map(&tk, c->k, outer, c->page_size, kHd) || !page_map(&tv, c->v, outer, c->page_size, kHd))
      return DG_ERR_CUDA;
    e = narrow ? launch_tc<kHd, true>(tk, tv, a, s) : launch_tc<kHd, false>(tk, tv, a, s);
  } else {
    static std::atomic<uint64_t> raised{0};
    e = raise_smem(k_paged_attn_f32<kHd>, PaF32<kHd>::kSmem, raised);
    if (e == cudaSuccess) e = launch(k_paged_attn_f32<kHd>, kSMs, 256, PaF32<kHd>::kSmem, s, a);
  }
  if (e != cudaSuccess) return done(e);
  return c->dtype == DG_BF16 ? run_join<bf16, kHd>(a, narrow ? 128 : 256, s) : run_join<float, kHd>(a, kPaF32Rows, s);
}

}  // namespace

extern "C" dg_status dg_qk_norm_rope(int32_t dtype, int32_t n_tokens, int32_t n_heads, int32_t n_kv_heads,
                                     int32_t head_dim, const dg_heads* q, const dg_heads* q_out, const dg_heads* k,
                                     const dg_heads* k_out, const int32_t* positions, const dg_rope* rope,
                                     const dg_head_norm* norm, void* stream) {
  if ((dtype != DG_FP32 && dtype != DG_BF16) || n_tokens < 0 || n_heads < 0 || n_kv_heads < 0) return DG_ERR_INVALID_ARG;
  if (head_dim < 2 || head_dim > 256 || head_dim % 2) return DG_ERR_INVALID_ARG;
  if (n_heads > 0 && (!heads_ok(q, dtype, n_tokens) || !heads_ok(q_out, dtype, n_tokens))) return DG_ERR_INVALID_ARG;
  if (n_kv_heads > 0 && (!heads_ok(k, dtype, n_tokens) || !heads_ok(k_out, dtype, n_tokens))) return DG_ERR_INVALID_ARG;
  if ((int64_t)n_heads + n_kv_heads > 65536) return DG_ERR_INVALID_ARG;
  if (!rope_ok(rope, head_dim) || !norm_ok(norm, dtype) || !aligned(positions, 4)) return DG_ERR_INVALID_ARG;
  if (rope && rope->rot_dim > 0 && !positions && n_tokens > 0) return DG_ERR_INVALID_ARG;
  HeadRowsArgs a{};
  a.n_tokens = n_tokens;
  a.n_q = n_heads;
  a.n_k = n_kv_heads;
  a.head_dim = head_dim;
  if (n_heads) { a.q = head_rows(q); a.qo = head_rows(q_out); }
  if (n_kv_heads) { a.k = head_rows(k); a.ko = head_rows(k_out); }
  a.positions = positions;
  set_steps(a, rope, norm);
  return run_head_rows(dtype, a, (cudaStream_t)stream);
}

extern "C" dg_status dg_paged_append(const dg_paged_kv* cache, const dg_paged_batch* batch, const dg_heads* k,
                                     const dg_heads* v, const dg_rope* rope, const dg_head_norm* norm,
                                     int32_t n_heads, const dg_heads* q, const dg_heads* q_out,
                                     int32_t* status_word, void* stream) {
  if (!cache_ok(cache) || !batch_ok(cache, batch)) return DG_ERR_INVALID_ARG;
  const int64_t rows = batch->n_tokens;
  const int dtype = cache->dtype;
  if (!heads_ok(k, dtype, rows) || !heads_ok(v, dtype, rows) || !aligned(status_word, 4)) return DG_ERR_INVALID_ARG;
  if (n_heads < 0 || (n_heads > 0 && (!heads_ok(q, dtype, rows) || !heads_ok(q_out, dtype, rows)))) return DG_ERR_INVALID_ARG;
  if ((int64_t)n_heads + 2ll * cache->n_kv_heads > 65536) return DG_ERR_INVALID_ARG;
  if (!rope_ok(rope, cache->head_dim) || !norm_ok(norm, dtype)) return DG_ERR_INVALID_ARG;
  HeadRowsArgs a{};
  a.n_tokens = batch->n_seqs > 0 ? batch->n_tokens : 0;
  a.n_q = n_heads;
  a.n_k = a.n_v = cache->n_kv_heads;
  a.head_dim = cache->head_dim;
  if (n_heads) { a.q = head_rows(q); a.qo = head_rows(q_out); }
  a.k = head_rows(k);
  a.v = head_rows(v);
  set_steps(a, rope, norm);
  a.paged = 1;
  a.k_pages = cache->k;
  a.v_pages = cache->v;
  a.b = device_batch(cache, batch, status_word);
  return run_head_rows(cache->dtype, a, (cudaStream_t)stream);
}

extern "C" size_t dg_paged_attention_workspace(int32_t n_tokens, int32_t n_heads, int32_t head_dim,
                                               int32_t with_prefix) {
  if (n_tokens < 0 || n_heads < 1 || n_heads > 32768 || (head_dim != 64 && head_dim != 128)) return 0;
  if ((int64_t)n_tokens * n_heads >= (int64_t)1 << 31) return 0;
  return paged_space(n_tokens, n_heads, head_dim, with_prefix != 0).total;
}

extern "C" dg_status dg_paged_attention(const dg_paged_kv* cache, const dg_paged_batch* batch, int32_t n_heads,
                                        const dg_heads* q, float scale, int32_t causal, const dg_heads* out,
                                        float* lse, void* workspace, size_t workspace_bytes, int32_t* status_word,
                                        void* stream) {
  if (!cache_ok(cache) || !batch_ok(cache, batch)) return DG_ERR_INVALID_ARG;
  const int hd = cache->head_dim;
  if (hd != 64 && hd != 128) return DG_ERR_UNSUPPORTED;
  if (n_heads < 1 || n_heads > 32768 || n_heads % cache->n_kv_heads || !(scale > 0.0f) || scale > 1e30f) return DG_ERR_INVALID_ARG;
  const size_t need = dg_paged_attention_workspace(batch->n_tokens, n_heads, hd, batch->prefix_len > 0);
  if (need == 0 || !workspace || workspace_bytes < need || !aligned(workspace, 256) || !aligned(lse, 4) ||
      !aligned(status_word, 4))
    return DG_ERR_INVALID_ARG;
  if (batch->n_seqs == 0 || batch->n_tokens == 0) return DG_OK;
  const int per16 = 16 / elem_size(cache->dtype);
  for (const dg_heads* h : {q, out})
    if (!heads_ok(h, cache->dtype, batch->n_tokens) || !aligned(h->data, 16) || h->token_stride % per16 || h->head_stride % per16)
      return DG_ERR_INVALID_ARG;
  // The line of work units (see dg_paged_attn.cuh) is counted in 32 bits: at
  // most this many tiles of 64 rows, each with every block of 64 keys.
  const int64_t rows = (int64_t)batch->n_tokens * (n_heads / cache->n_kv_heads);
  const int64_t keys = (int64_t)batch->max_pages * cache->page_size;
  if (((rows / 64 + batch->n_seqs) * (keys / 64 + 4) + (rows / 64 + 1) * ((int64_t)batch->prefix_len / 64 + 4)) *
          cache->n_kv_heads >= (int64_t)1 << 31)
    return DG_ERR_UNSUPPORTED;
  const PagedSpace sp = paged_space(batch->n_tokens, n_heads, hd, batch->prefix_len > 0);
  char* ws = (char*)workspace;
  PagedAttnArgs a{};
  a.b = device_batch(cache, batch, status_word);
  a.q = q->data;
  a.q_ts = q->token_stride;
  a.q_hs = q->head_stride;
  a.out = out->data;
  a.o_ts = out->token_stride;
  a.o_hs = out->head_stride;
  a.n_heads = n_heads;
  a.n_kv_heads = cache->n_kv_heads;
  a.G = n_heads / cache->n_kv_heads;
  a.by_g.m = SmallDiv::magic((uint32_t)a.G);
  a.causal = causal != 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.k_pages = cache->k;
  a.v_pages = cache->v;
  a.lse = lse;
  a.meta = (int2*)(ws + sp.meta);
  a.part_lse = (float*)(ws + sp.part_lse);
  a.slot_lse = (float*)(ws + sp.slot_lse);
  a.part_o = (float*)(ws + sp.part_o);
  a.slot_o = (float*)(ws + sp.slot_o);
  return hd == 64 ? run_paged_attention<64>(cache, a, (cudaStream_t)stream)
                  : run_paged_attention<128>(cache, a, (cudaStream_t)stream);
}

extern "C" dg_status dg_serving_status(void* stream) {
  const cudaStream_t s = (cudaStream_t)stream;
  int code = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&code, g_serving_status, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && code) {
    const int none = 0;
    e = cudaMemcpyToSymbolAsync(g_serving_status, &none, sizeof(int), 0, cudaMemcpyHostToDevice, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  return e == cudaSuccess ? (dg_status)code : done(e);
}

extern "C" dg_status dg_test_paged_walk(const dg_paged_kv* cache, const dg_paged_batch* batch, int32_t n_heads,
                                        int32_t causal, int32_t tile_rows, int32_t* status_word, int32_t* out,
                                        int32_t cap, int32_t* n_out) {
  if (!cache_ok(cache) || !batch_ok(cache, batch) || n_heads < 1 || n_heads > 32768 || n_heads % cache->n_kv_heads) return DG_ERR_INVALID_ARG;
  if ((tile_rows != 256 && tile_rows != 128 && tile_rows != kPaF32Rows) || !out || !n_out) return DG_ERR_INVALID_ARG;
  PagedAttnArgs a{};
  a.b = device_batch(cache, batch, status_word);
  a.n_heads = n_heads;
  a.n_kv_heads = cache->n_kv_heads;
  a.G = n_heads / cache->n_kv_heads;
  a.by_g.m = SmallDiv::magic((uint32_t)a.G);
  a.causal = causal != 0;
  int n = 0;
  auto walk = [&](auto w) {
    for (int cta = 0; cta < kSMs; ++cta) {
      if (!w.begin_host(cta)) continue;
      for (PagedFrag f = w.next(); f.nblk; f = w.next(), ++n) {
        if (n >= cap) return false;
        const int seq = f.part ? -1 : (int)((f.page_list - a.b.table) / std::max<int64_t>(1, a.b.table_stride));
        const int v[16] = {cta, f.part, seq, f.q0, f.row0, f.rows, f.kvh, f.kb0, f.nblk, f.limit, f.vis0, f.vis_max,
                           f.pages, f.first, f.whole, f.n_cont};
        for (int i = 0; i < 16; ++i) out[16 * (int64_t)n + i] = v[i];
      }
    }
    return true;
  };
  const bool ok = tile_rows == 256   ? walk(PagedWalk<256, kPaBlk>(a))
                  : tile_rows == 128 ? walk(PagedWalk<128, kPaBlk>(a))
                                     : walk(PagedWalk<kPaF32Rows, kPaF32Blk>(a));
  *n_out = n;
  return ok ? DG_OK : DG_ERR_INVALID_ARG;
}
