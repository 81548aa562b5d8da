// The cache handle: validation, rotation table, tensor maps, status word, and
// the C entry points of the operators that work on it (include/mk.h).
#include <math.h>
#include <string.h>

#include <atomic>
#include <mutex>
#include <new>

#include "mk_cache.h"

namespace mk {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Maps of a cache or pool (rows of head_dim elements), 128-byte swizzle
// (16-byte chunk c of row r at c ^ (r & 7)).  Small and tall boxes: 64 columns
// x so many rows.  Whole boxes: all columns x kWholeRows rows, which land as
// [64-column block][row].
cudaError_t encode_maps(const void* base, int64_t rows, int hd, int small_rows, int tall_rows, CUtensorMap* small,
                        CUtensorMap* tall, CUtensorMap* whole) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return cudaErrorNotSupported;
  const auto encode = reinterpret_cast<EncodeTiledFn>(p);
  const cuuint64_t dims2[2] = {(cuuint64_t)hd, (cuuint64_t)rows};
  const cuuint64_t strides2[1] = {(cuuint64_t)hd * 2};
  cuuint32_t box2[2] = {64, (cuuint32_t)small_rows};
  const cuuint64_t dims3[3] = {64, (cuuint64_t)rows, (cuuint64_t)(hd / 64)};
  const cuuint64_t strides3[2] = {(cuuint64_t)hd * 2, 128};
  const cuuint32_t box3[3] = {64, (cuuint32_t)kWholeRows, (cuuint32_t)(hd / 64)};
  const cuuint32_t ones[3] = {1, 1, 1};
  CUresult r = encode(small, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims2, strides2, box2, ones,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  box2[1] = (cuuint32_t)tall_rows;
  if (r == CUDA_SUCCESS)
    r = encode(tall, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims2, strides2, box2, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS)
    r = encode(whole, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims3, strides3, box3, ones,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// (cos, sin) of pos * theta^(-2i/hd), angles and functions in double: an angle
// of a far position has no fraction left in fp32.  A thread keeps its i.
__global__ void rope_table(float2* out, int T, int half, double theta) {
  const int i = threadIdx.x % half, rows = blockDim.x / half;
  const double freq = pow(theta, -(double)i / half);
  for (int pos = blockIdx.x * rows + threadIdx.x / half; pos < T; pos += gridDim.x * rows) {
    double s, c;
    sincos(pos * freq, &s, &c);
    out[(int64_t)pos * half + i] = make_float2((float)c, (float)s);
  }
}

// Device memory of the handles, from a pool of the library that keeps some of what is
// freed: cudaMalloc and cudaFree take milliseconds next to live work.  More goes back
// to the device when a handle is destroyed (a table of 131072 positions of 128 is 64 MB).
constexpr uint64_t kKeptBytes = 64ull << 20;
cudaError_t pool_of(int dev, cudaMemPool_t* out) {
  static std::mutex lock;
  static cudaMemPool_t pools[64];
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> hold(lock);
  if (!pools[dev]) {
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    cudaMemPool_t p;
    cudaError_t e = cudaMemPoolCreate(&p, &props);
    if (e != cudaSuccess) return e;
    uint64_t keep = kKeptBytes;
    e = cudaMemPoolSetAttribute(p, cudaMemPoolAttrReleaseThreshold, &keep);
    if (e != cudaSuccess) {
      cudaMemPoolDestroy(p);
      return e;
    }
    pools[dev] = p;
  }
  *out = pools[dev];
  return cudaSuccess;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int launched(cudaError_t e) {
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  return MK_ERR_CUDA;
}

}  // namespace

int current_sms() {
  static std::atomic<int> known[64];  // an attribute of the device: the same for good
  int dev = -1, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace mk

extern "C" int mk_cache_create(const mk_cache_desc* desc, const mk_kv* kv, mk_cache** out) {
  if (!out) return MK_ERR_INVALID_ARG;
  *out = nullptr;
  if (!desc || !kv || !kv->k || !kv->v) return MK_ERR_INVALID_ARG;
  const mk_cache_desc& d = *desc;
  if (d.n_layers <= 0 || d.batch <= 0 || d.n_q_heads <= 0 || d.n_kv_heads <= 0 || d.head_dim <= 0 || d.max_ctx <= 0 ||
      !(d.rms_eps >= 0) || !(d.rope_theta > 0))
    return MK_ERR_INVALID_ARG;
  if (kv->block_table && (kv->page_size <= 0 || kv->n_pages <= 0)) return MK_ERR_INVALID_ARG;
  if ((d.head_dim != 64 && d.head_dim != 128) || d.n_q_heads % d.n_kv_heads ||
      d.n_q_heads / d.n_kv_heads > mk::kCacheMaxGroup || d.batch > mk::kCacheMaxBatch ||
      !mk::aligned(kv->k, 16) || !mk::aligned(kv->v, 16) || !mk::aligned(kv->block_table, 4) ||
      (kv->block_table && kv->page_size % mk::kCachePageUnit) || d.max_ctx > (1 << 30) || d.n_q_heads > (1 << 16))
    return MK_ERR_UNSUPPORTED;
  // rows of the cache, each factor below 2^31: compare step by step
  const int64_t limit = (int64_t)1 << 31;
  const int64_t factors[4] = {d.n_layers, kv->block_table ? kv->n_pages : d.batch, d.n_kv_heads,
                              kv->block_table ? kv->page_size : d.max_ctx};
  int64_t rows = 1;
  for (int64_t f : factors) {
    rows *= f;
    if (rows >= limit) return MK_ERR_UNSUPPORTED;
  }

  // the attention's schedule counts tiles of 64 positions, for every sequence and KV head, in 32 bits
  if (((int64_t)d.max_ctx / 64 + 4) * d.n_kv_heads * d.batch >= limit) return MK_ERR_UNSUPPORTED;

  int dev = 0, n_sm = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  if (major != 10 || minor != 0) return MK_ERR_UNSUPPORTED;
  if (mk::attend_prepare() != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  mk_cache* c = new (std::nothrow) mk_cache();
  if (!c) return MK_ERR_CUDA;
  c->d = d;
  c->device = dev;
  c->n_sm = n_sm;
  c->k = (uint16_t*)kv->k;
  c->v = (uint16_t*)kv->v;
  c->box = mk::cache_box_rows(kv->block_table ? kv->page_size : 0, 32);
  c->tall = mk::cache_box_rows(kv->block_table ? kv->page_size : 0, 128);
  cudaError_t e = mk::encode_maps(kv->k, rows, d.head_dim, c->box, c->tall, &c->kmap, &c->ktall, &c->kwhole);
  if (e == cudaSuccess) e = mk::encode_maps(kv->v, rows, d.head_dim, c->box, c->tall, &c->vmap, &c->vtall, &c->vwhole);
  if (e != cudaSuccess) {
    delete c;
    return e == cudaErrorInvalidValue ? MK_ERR_UNSUPPORTED : MK_ERR_CUDA;
  }
  const size_t table = sizeof(float2) * (size_t)d.max_ctx * (d.head_dim / 2);
  cudaMemPool_t pool;
  if (mk::pool_of(dev, &pool) != cudaSuccess ||
      cudaMallocFromPoolAsync(&c->region, 256 + table, pool, cudaStreamPerThread) != cudaSuccess) {
    cudaGetLastError();
    delete c;
    return MK_ERR_CUDA;
  }
  mk::CacheView& w = c->view;
  w.B = d.batch;
  w.nq = d.n_q_heads;
  w.nkv = d.n_kv_heads;
  w.T = d.max_ctx;
  w.bt = kv->block_table;
  if (w.bt) {
    w.page = kv->page_size;
    w.n_pages = kv->n_pages;
    w.bt_stride = (int)(((int64_t)d.max_ctx + kv->page_size - 1) / kv->page_size);
  }
  w.status = (int*)c->region;
  c->rope = (float2*)((uint8_t*)c->region + 256);
  mk::rope_table<<<n_sm * 4, 256, 0, cudaStreamPerThread>>>(c->rope, d.max_ctx, d.head_dim / 2, (double)d.rope_theta);
  // the table is ready when this returns: calls may come on any stream
  if (cudaGetLastError() != cudaSuccess || cudaMemsetAsync(c->region, 0, 256, cudaStreamPerThread) != cudaSuccess ||
      cudaStreamSynchronize(cudaStreamPerThread) != cudaSuccess) {
    cudaGetLastError();
    cudaFreeAsync(c->region, cudaStreamPerThread);
    delete c;
    return MK_ERR_CUDA;
  }
  *out = c;
  return MK_OK;
}

extern "C" int mk_cache_destroy(mk_cache* c) {
  if (!c) return MK_OK;
  cudaError_t e;
  {
    mk::OnDevice here(c->device);
    e = cudaDeviceSynchronize();  // calls on any stream may still read the table
    if (e == cudaSuccess) e = cudaFreeAsync(c->region, cudaStreamPerThread);  // else it stays: better lost than read after
    if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamPerThread);     // what the pool holds above its limit is released
  }
  delete c;
  return mk::launched(e);
}

extern "C" int mk_cache_get_status(mk_cache* c, void* stream) {
  if (!c) return MK_ERR_INVALID_ARG;
  mk::OnDevice here(c->device);
  if (!here.ok) return MK_ERR_CUDA;
  int st[2] = {0, 0};
  cudaStream_t s = (cudaStream_t)stream;
  if (cudaMemcpyAsync(st, c->view.status, sizeof(st), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess ||
      (st[0] && (cudaMemsetAsync(c->view.status, 0, sizeof(st), s) != cudaSuccess ||
                 cudaStreamSynchronize(s) != cudaSuccess))) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  return st[0];
}

extern "C" int mk_cache_append(mk_cache* c, int layer, const mk_append_args* a, void* stream) {
  if (!c || !a || layer < 0 || layer >= c->d.n_layers || a->n_tokens < 0 ||
      (!a->starts && a->n_tokens != c->d.batch) || (a->dtype != MK_DTYPE_BF16 && a->dtype != MK_DTYPE_FP32))
    return MK_ERR_INVALID_ARG;
  if (a->n_tokens == 0) return MK_OK;
  if (!a->k || !a->v || !a->seq_lens || !a->q != !a->q_out) return MK_ERR_INVALID_ARG;
  const int64_t es = a->dtype == MK_DTYPE_BF16 ? 2 : 4;
  if ((a->q && (!mk::aligned(a->q, 16) || !mk::aligned(a->q_out, 16) || (a->q_stride * es) % 16)) ||
      !mk::aligned(a->k, 16) || !mk::aligned(a->v, 16) || (a->k_stride * es) % 16 || (a->v_stride * es) % 16 ||
      !mk::aligned(a->q_norm, 16) || !mk::aligned(a->k_norm, 16) || !mk::aligned(a->starts, 4) ||
      !mk::aligned(a->seq_lens, 4) || !mk::aligned(a->positions, 4))
    return MK_ERR_UNSUPPORTED;
  mk::OnDevice here(c->device);
  if (!here.ok) return MK_ERR_CUDA;
  return mk::launched(mk::append(*c, layer, *a, (cudaStream_t)stream));
}

extern "C" size_t mk_cache_attend_bytes(const mk_cache* c) { return c ? mk::attend_workspace(c->d, c->n_sm) : 0; }

extern "C" int mk_cache_attend(mk_cache* c, int layer, const void* q, const int32_t* seq_lens, int prefix_len,
                               float scale, void* out, float* lse, void* workspace, size_t workspace_bytes,
                               void* stream) {
  if (!c || !q || !seq_lens || !out || !workspace) return MK_ERR_INVALID_ARG;
  if (layer < 0 || layer >= c->d.n_layers || prefix_len < 0 || prefix_len > c->d.max_ctx || !isfinite(scale * mk::kLog2e) ||
      workspace_bytes < mk::attend_workspace(c->d, c->n_sm))
    return MK_ERR_INVALID_ARG;
  if (!mk::aligned(q, 16) || !mk::aligned(out, 16) || !mk::aligned(seq_lens, 4) || !mk::aligned(lse, 4) ||
      !mk::aligned(workspace, 256))
    return MK_ERR_UNSUPPORTED;
  mk::OnDevice here(c->device);
  if (!here.ok) return MK_ERR_CUDA;
  return mk::launched(mk::attend(*c, layer, q, seq_lens, prefix_len, scale, out, lse, workspace, (cudaStream_t)stream));
}
