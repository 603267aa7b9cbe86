// What the paged serving operators share: the ragged batch as kernels see it.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "dg_device.cuh"

// The caller's arrays are device memory the host never looks at, so every
// value read from them is brought into range before it is used as an index
// and reported through the status word when it was out of range.

// The word of calls that were given none: one on each device, zero until an
// error, read and cleared by dg_serving_status.
__device__ int g_serving_status;

struct PagedBatch {
  int n_seqs, n_tokens;
  const int* cu_q;
  const int* kv_lens;
  const int* table;
  long long table_stride;
  int max_pages;
  const int* prefix_pages;
  int prefix_len;
  int n_pages, page_shift;   // page size = 1 << page_shift
  int* status;               // null: the device's own word
};

struct PagedSeq {
  int q0, nq;   // rows of the token buffers
  int kv;       // own tokens in the cache, the new ones included
};

// status word values: dg_status codes of include/dg.h
constexpr int kStatusTimeout = 4;   // DG_ERR_TIMEOUT
constexpr int kStatusState = 5;     // DG_ERR_STATE

#define DG_HD __host__ __device__ __forceinline__

DG_HD int imin(int a, int b) { return a < b ? a : b; }
DG_HD int imax(int a, int b) { return a > b ? a : b; }
DG_HD long long lmin(long long a, long long b) { return a < b ? a : b; }

DG_HD void paged_error(const PagedBatch& b, int code) {
#ifdef __CUDA_ARCH__
  dev_error(b.status ? b.status : &g_serving_status, code);
#else
  if (b.status && *b.status == 0) *b.status = code;
#endif
}

// Sequence of the rows a0 .. a1 - 1 and kv tokens, as read.
DG_HD PagedSeq paged_seq(const PagedBatch& b, int a0, int a1, int kv) {
  PagedSeq s;
  s.q0 = imin(imax(a0, 0), b.n_tokens);
  const int q1 = imin(imax(a1, s.q0), b.n_tokens);
  s.nq = q1 - s.q0;
  const long long room = (long long)b.max_pages << b.page_shift;
  s.kv = (int)lmin(imax(kv, 0), room);
  if (s.q0 != a0 || q1 != a1 || s.kv != kv) paged_error(b, kStatusState);
  return s;
}
DG_HD PagedSeq paged_seq(const PagedBatch& b, int i) { return paged_seq(b, b.cu_q[i], b.cu_q[i + 1], b.kv_lens[i]); }
