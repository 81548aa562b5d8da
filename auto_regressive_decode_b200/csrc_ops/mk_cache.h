// The cache handle of mk_cache_* and what its kernels share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/mk.h"

struct mk_cache;

namespace mk {

constexpr int kCacheMaxBatch = 1024;  // sequences of a cache handle
constexpr int kCacheMaxGroup = 64;    // query heads per KV head
constexpr int kCachePageUnit = 16;    // page_size is a multiple of this
constexpr float kLog2e = 1.44269504088896341f;  // scores are in units of log2
constexpr int kWholeRows = 64;        // cache rows of a whole box of the tensor maps: an attention tile

// What a kernel needs to find a row of the cache: contiguous
// [L][B][nkv][T][hd], or pages [L][n_pages][nkv][page][hd] through bt[B][bt_stride].
struct CacheView {
  int B, nq, nkv, T;
  const int32_t* bt;
  int bt_stride, page, n_pages;
  int* status;  // [0] code, [1] detail

#ifdef __CUDACC__
  // Row index of (layer, sequence, KV head 0, position); a KV head adds head_pitch() rows.
  // A page outside the pool is recorded and read as page 0 (*ok = false).
  __device__ __forceinline__ int64_t row(int layer, int b, int pos, bool* ok) const {
    if (bt) {
      int pg = bt[(int64_t)b * bt_stride + pos / page];
      *ok = pg >= 0 && pg < n_pages;
      if (!*ok) pg = 0;
      return ((int64_t)layer * n_pages + pg) * nkv * page + pos % page;
    }
    *ok = true;
    return ((int64_t)layer * B + b) * nkv * T + pos;
  }
  __device__ __forceinline__ int64_t head_pitch() const { return bt ? page : T; }
#endif
};

// Rows of a TMA box of the cache, at most `most` (a power of two): it lies in one page.
inline int cache_box_rows(int page, int most) {
  int r = most;
  while (page % r) r /= 2;  // a contiguous cache (page 0): the most
  return r;
}

cudaError_t append(const mk_cache& c, int layer, const mk_append_args& a, cudaStream_t stream);
size_t attend_workspace(const mk_cache_desc& d, int n_sm);
cudaError_t attend_prepare();
cudaError_t attend(const mk_cache& c, int layer, const void* q, const int32_t* seq_lens, int prefix_len, float scale,
                   void* out, float* lse, void* workspace, cudaStream_t stream);

// Makes `device` (-1: as it is) the current one of this thread for a scope.
struct OnDevice {
  int before = -1;
  bool ok = true;
  explicit OnDevice(int device) {
    int now = -1;
    if (device < 0) return;
    ok = cudaGetDevice(&now) == cudaSuccess;
    if (ok && now != device) {
      ok = cudaSetDevice(device) == cudaSuccess;
      if (ok) before = now;
    }
    if (!ok) cudaGetLastError();
  }
  ~OnDevice() {
    if (before >= 0) cudaSetDevice(before);
  }
  OnDevice(const OnDevice&) = delete;
};

// Streaming multiprocessors of the current device; 0 when it cannot be asked.
int current_sms();

}  // namespace mk

struct mk_cache {
  mk_cache_desc d;
  mk::CacheView view;
  uint16_t *k, *v;
  int device, n_sm, box, tall;
  float2* rope;  // [max_ctx][hd/2] (cos, sin)
  CUtensorMap kmap, vmap;      // boxes of 64 columns x box rows
  CUtensorMap kwhole, vwhole;  // boxes of all columns x kWholeRows rows
  CUtensorMap ktall, vtall;    // boxes of 64 columns x tall rows
  void* region;
};
