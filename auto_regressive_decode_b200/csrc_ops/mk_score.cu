// Log probabilities of given tokens, entropy and the most likely alternatives.
//
// One pass over a row of logits x.  Every thread keeps its maximum m and, in
// units of log2 (d = (x - m) log2 e), z = sum 2^d and s = sum 2^d d, moved to a
// new m when it grows; the threads' (m, z, s) join at the end:
//   logprob(t) = x_t - m - ln z,   entropy = ln z - ln 2 * s / z
// (every term of the entropy is >= 0: nothing cancels).
//
// Alternatives: a key packs the order-preserving map of the logit over the
// inverted index, so that the largest key is the largest logit, of the lowest
// index among equals, and no two keys are equal.  A threshold below at least
// top_k keys seen so far lets few keys through into a buffer; the first chunk's
// thread maxima give the first threshold, a full buffer the next ones.  The result does not depend on the order of arrival.
//
// Bound: memory for many rows (one read of the logits).  Few rows: each is
// cut over the blocks of a cluster, which join through distributed shared memory:
// no workspace, one launch.
#include <cooperative_groups.h>
#include <math.h>

#include "mk_cache.h"
#include "mk_ptx.h"

namespace mk {
namespace {

using namespace ptx;
namespace cg = cooperative_groups;

constexpr int kMaxTop = 32;
constexpr int kCap = 1024;    // candidate buffer
constexpr int kChunk = 16;    // logits a thread holds at once
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
typedef unsigned long long Key;

struct ScoreParams {
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float *logprob, *entropy;
  int32_t* ids;
  float* tops;
  int vocab, top_k;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // -0 becomes +0: they are equal logits
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7fffffffu) : ~u);
}
__device__ __forceinline__ Key make_key(float x, int i) { return ((Key)ordered(x) << 32) | (uint32_t)~i; }

// Running maximum, sum and weighted sum (log2 units).
struct Sum {
  float m, z, s;
  __device__ __forceinline__ void join(const Sum& o) {
    const float M = fmaxf(m, o.m), ref = M == -INFINITY ? 0.f : M;
    auto part = [&](const Sum& x, float& zz, float& ss) {
      if (x.z == 0.f) return;  // nothing but -infinity (a NaN sum is passed on)
      const float dm = (x.m - ref) * kLog2e, f = ex2(dm);
      zz += f * x.z;
      if (f > 0.f) ss += f * (x.s + x.z * dm);
    };
    float zz = 0.f, ss = 0.f;
    part(*this, zz, ss);
    part(o, zz, ss);
    m = M;
    z = zz;
    s = ss;
  }
};

template <typename T>
struct Load;  // 16 consecutive logits a thread, in 16-byte vectors a warp apart
template <>
struct Load<float> {
  static constexpr int kVec = 4;
};
template <>
struct Load<uint16_t> {
  static constexpr int kVec = 8;
};

template <int NT>
struct Shared {
  Key buf[kCap];
  Key best[kMaxTop];
  Key limit;  // keys below it are not among the best
  int count;
  Sum part[NT / 32];
  Sum sum;    // this block's
  int n_best;
};

// The n keys of buf: the k largest to best[], in order.  Returns how many.
template <int NT>
__device__ __forceinline__ int select_best(Shared<NT>& sh, int n, int k) {
  for (int e = threadIdx.x; e < n; e += NT) {
    const Key x = sh.buf[e];
    int rank = 0;
    for (int i = 0; i < n; ++i) rank += sh.buf[i] > x;
    if (rank < k) sh.best[rank] = x;
  }
  __syncthreads();
  return min(n, k);
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT) score_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int VEC = Load<T>::kVec, U = kChunk / VEC;
  __shared__ Shared<NT> sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  const int tid = threadIdx.x, k = p.top_k;
  const int64_t row = blockIdx.x / parts;
  const T* x = reinterpret_cast<const T*>(p.logits) + row * p.stride;

  // this block's logits [c0, c1), walked in aligned vectors: vector v covers
  // [v * VEC - skew, ...) where skew is the row's offset from alignment
  const int skew = (int)(((uintptr_t)x & 15) / sizeof(T));
  const int vecs = (p.vocab + skew + VEC - 1) / VEC;
  const int v0 = (int)((int64_t)vecs * part / parts), v1 = (int)((int64_t)vecs * (part + 1) / parts);

  if (tid == 0) {
    sh.limit = 0;
    sh.count = 0;
  }
  Sum a{-INFINITY, 0.f, 0.f};

  uint4 raw[U];
  auto fetch = [&](int base) {  // vectors base + tid, base + NT + tid, ...
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = base + u * NT + tid;
      const int i0 = v * VEC - skew;
      if (v < v1 && i0 >= 0 && i0 + VEC <= p.vocab) {
        raw[u] = __ldcs(reinterpret_cast<const uint4*>(x + i0));
      } else {  // the ends of the row: nothing outside of it is read
        T e[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const bool in = v < v1 && i0 + i >= 0 && i0 + i < p.vocab;
          if constexpr (sizeof(T) == 4) e[i] = in ? x[i0 + i] : -INFINITY;
          else e[i] = in ? x[i0 + i] : (T)0xff80;
        }
        memcpy(&raw[u], e, 16);
      }
    }
  };
  fetch(v0);
  __syncthreads();
  for (int base = v0; base < v1; base += NT * U) {
    float f[kChunk];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          f[u * 4 + i] = __uint_as_float(w[i]);
        } else {
          f[u * 8 + 2 * i] = bf16_lo(w[i]);
          f[u * 8 + 2 * i + 1] = bf16_hi(w[i]);
        }
      }
    }
    if (base + NT * U < v1) fetch(base + NT * U);
    float top = f[0];
#pragma unroll
    for (int i = 1; i < kChunk; ++i) top = fmaxf(top, f[i]);
    if (top > a.m) {
      if (a.m > -INFINITY) {
        const float dm = (a.m - top) * kLog2e, g = ex2(dm);
        a.s = g > 0.f ? g * (a.s + a.z * dm) : 0.f;
        a.z *= g;
      }
      a.m = top;
    }
    const float ref = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      // far below the maximum 2^d is 0: the bound keeps 0 * -infinity out of s
      const float d = max_nan((f[i] - ref) * kLog2e, -150.f), e = ex2(d);
      a.z += e;
      a.s = fmaf(e, d, a.s);
    }
    if (k > 0) {
      const uint32_t lim = (uint32_t)(sh.limit >> 32);
      const uint32_t mine = ordered(top);
      const bool cand = top > -INFINITY && mine >= lim;
      const int n = __syncthreads_count(cand);
      if (n) {
        if (n > 2 * k) {  // raise the threshold: the largest 16-bit prefix that k thread maxima reach
          uint32_t t = 0;
          for (int bit = 15; bit >= 0; --bit) {
            const uint32_t want = t | (1u << bit);
            if (__syncthreads_count(cand && (mine >> 16) >= want) >= k) t = want;
          }
          if (tid == 0 && ((Key)t << 48) > sh.limit) sh.limit = (Key)t << 48;
          __syncthreads();
        }
        uint32_t todo = cand ? 0xffffu : 0u;
        while (true) {
          const Key limit = sh.limit;
          if (todo) {
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
              if (todo >> i & 1) {
                const int idx = (base + (i / VEC) * NT + tid) * VEC - skew + i % VEC;
                const Key key = make_key(f[i], idx);
                bool left = false;
                if (f[i] > -INFINITY && key >= limit) {
                  const int at = atomicAdd(&sh.count, 1);
                  if (at < kCap) sh.buf[at] = key;
                  else left = true;
                }
                if (!left) todo &= ~(1u << i);
              }
            }
          }
          __syncthreads();
          const bool full = sh.count > kCap;
          if (!full) break;
          select_best<NT>(sh, kCap, k);
          if (tid < k) sh.buf[tid] = sh.best[tid];
          if (tid == 0) {
            sh.count = k;
            sh.limit = sh.best[k - 1] + 1;
          }
          __syncthreads();
        }
      }
    }
  }

  // join the threads' sums
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Sum b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.z = __shfl_xor_sync(0xffffffffu, a.z, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    a.join(b);
  }
  if (tid % 32 == 0) sh.part[tid / 32] = a;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < NT / 32; ++w) a.join(sh.part[w]);
    sh.sum = a;
  }
  const int got = k > 0 ? select_best<NT>(sh, sh.count, k) : 0;
  if (tid == 0) sh.n_best = got;
  __syncthreads();

  if (parts > 1) {
    cluster.sync();
    if (part == 0) {
      if (tid == 0)
        for (int r = 1; r < parts; ++r) a.join(cluster.map_shared_rank(&sh, r)->sum);
      // the blocks' best keys, one after another
      int n = got;
      if (tid < got) sh.buf[tid] = sh.best[tid];
      for (int r = 1; r < parts; ++r) {
        const Shared<NT>* o = cluster.map_shared_rank(&sh, r);
        const int m = o->n_best;
        if (tid < m) sh.buf[n + tid] = o->best[tid];
        n += m;
      }
      __syncthreads();
      if (tid == 0) sh.sum = a;
      if (k > 0) {
        const int m = select_best<NT>(sh, n, k);
        if (tid == 0) sh.n_best = m;
      }
      __syncthreads();
    }
    cluster.sync();  // a block's shared memory stays until it has been read
    if (part) return;
  }
  const Sum r = sh.sum;
  const float lnz = logf(r.z);
  const bool none = !(r.z > 0.f) || isinf(r.m);  // NaN, infinities, or nothing allowed
  if (tid == 0) {
    const int t = p.tokens[row];
    float v = NAN;
    if (t >= 0 && t < p.vocab && !none) {
      const float xt = sizeof(T) == 4 ? reinterpret_cast<const float*>(x)[t]
                                      : __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(x)[t] << 16);
      v = xt - r.m - lnz;
    }
    p.logprob[row] = v;
    if (p.entropy) p.entropy[row] = none ? NAN : lnz - kLn2 * r.s / r.z;
  }
  if (tid < k) {
    const bool has = !none && tid < sh.n_best;
    const Key key = has ? sh.best[tid] : 0;
    p.ids[row * k + tid] = has ? (int32_t)~(uint32_t)key : -1;
    p.tops[row * k + tid] = none ? NAN : (has ? from_ordered((uint32_t)(key >> 32)) - r.m - lnz : -INFINITY);
  }
}

template <typename T, int NT>
cudaError_t launch(const ScoreParams& p, int rows, int parts, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * parts);
  cfg.blockDim = dim3(NT);
  cfg.stream = stream;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = parts;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, score_kernel<T, NT>, p);
}

template <typename T>
cudaError_t score(const ScoreParams& p, int rows, int n_sm, cudaStream_t stream) {
  if (p.vocab <= 4096) return launch<T, 128>(p, rows, 1, stream);
  // Few rows: as many blocks a row as fill the SMs, 4096 logits a block at least.
  int parts = 1;
  while (parts < 8 && rows * parts < n_sm && p.vocab / (2 * parts) >= 4096) parts *= 2;
  return launch<T, 512>(p, rows, parts, stream);
}

__global__ void advance_lens(int32_t* lens, int n) {
  for (int b = threadIdx.x; b < n; b += blockDim.x) lens[b] += 1;
}

}  // namespace
}  // namespace mk

extern "C" int mk_token_logprobs(const void* logits, int dtype, int64_t row_stride, int n_rows, int vocab,
                                 const int32_t* tokens, float* out_logprob, float* out_entropy, int top_k,
                                 int32_t* out_top_ids, float* out_top_logprobs, int device, void* stream) {
  if (n_rows < 0 || vocab <= 0 || top_k < 0 || (dtype != MK_DTYPE_BF16 && dtype != MK_DTYPE_FP32))
    return MK_ERR_INVALID_ARG;
  if (n_rows == 0) return MK_OK;
  if (!logits || !tokens || !out_logprob || (top_k > 0 && (!out_top_ids || !out_top_logprobs)) || row_stride < 0)
    return MK_ERR_INVALID_ARG;
  const int es = dtype == MK_DTYPE_BF16 ? 2 : 4;
  if (top_k > mk::kMaxTop || vocab > (1 << 30) || n_rows > (1 << 27) || ((uintptr_t)logits & (es - 1)) ||
      ((uintptr_t)tokens & 3) || ((uintptr_t)out_logprob & 3) || ((uintptr_t)out_entropy & 3) ||
      ((uintptr_t)out_top_ids & 3) || ((uintptr_t)out_top_logprobs & 3))
    return MK_ERR_UNSUPPORTED;
  mk::OnDevice here(device);
  const int n_sm = here.ok ? mk::current_sms() : 0;
  if (!n_sm) return MK_ERR_CUDA;
  const mk::ScoreParams p{logits, row_stride, tokens, out_logprob, out_entropy, out_top_ids, out_top_logprobs, vocab, top_k};
  const cudaError_t e = es == 2 ? mk::score<uint16_t>(p, n_rows, n_sm, (cudaStream_t)stream)
                                : mk::score<float>(p, n_rows, n_sm, (cudaStream_t)stream);
  if (e == cudaSuccess) return MK_OK;
  cudaGetLastError();
  return MK_ERR_CUDA;
}

extern "C" int mk_decode_greedy_scored(mk_handle* h, const mk_model_desc* desc, int n_steps, const int32_t* tokens,
                                       const int32_t* seq_lens, void* stream, int32_t* out_tokens, int32_t* out_lens,
                                       float* logits, float* out_logprob, float* out_entropy, int top_k,
                                       int32_t* out_top_ids, float* out_top_logprobs) {
  if (!h || !desc || n_steps < 0 || !tokens || !seq_lens || !out_lens || out_lens == seq_lens || desc->batch <= 0 ||
      desc->vocab <= 0 || top_k < 0 ||
      (n_steps > 0 && (!out_tokens || !logits || !out_logprob || (top_k > 0 && (!out_top_ids || !out_top_logprobs)))))
    return MK_ERR_INVALID_ARG;
  if (top_k > mk::kMaxTop) return MK_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  const int B = desc->batch;
  if (cudaMemcpyAsync(out_lens, seq_lens, sizeof(int32_t) * B, cudaMemcpyDeviceToDevice, s) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  for (int t = 0; t < n_steps; ++t) {
    int32_t* picks = out_tokens + (size_t)t * B;
    int rc = mk_decode_greedy(h, 1, t ? picks - B : tokens, out_lens, stream, picks, logits);
    if (rc == MK_OK)
      rc = mk_token_logprobs(logits, MK_DTYPE_FP32, desc->vocab, B, desc->vocab, picks, out_logprob + (size_t)t * B,
                             out_entropy ? out_entropy + (size_t)t * B : nullptr, top_k,
                             top_k ? out_top_ids + (size_t)t * B * top_k : nullptr,
                             top_k ? out_top_logprobs + (size_t)t * B * top_k : nullptr, -1, stream);
    if (rc != MK_OK) return rc;
    mk::advance_lens<<<1, 32, 0, s>>>(out_lens, B);
    if (cudaGetLastError() != cudaSuccess) return MK_ERR_CUDA;
  }
  return MK_OK;
}
