// Appending keys and values to the cache, rotated on the way.
//
// A token's rows (query heads, key heads, value heads) are independent; each
// is read once, normalised (optional), rotated and written once:
//   y = x / sqrt(mean(x^2) + eps) * gain
//   out[i]     = y[i] cos a_i - y[i + hd/2] sin a_i
//   out[i + h] = y[i + hd/2] cos a_i + y[i] sin a_i,   a_i = pos theta^(-2i/hd)
// Bound: memory (3 flops a value): 16384 tokens of 120 fp32 rows of 128 (1.5 GB) take 232 to 236 us, 6.4
// to 6.5 TB/s; 4100 of 48 bf16 rows 19.6 us, 5.1 TB/s (the latency of finding a token's place; 18.5 with the
// rows in the L2 cache); one token of each of 8 sequences 2.1 us, a launch.
// hd/16 neighbouring lanes hold a row, each 8 values of its first half and the 8
// they pair with, so that loads and stores are 16 bytes and a lane's cos/sin (8
// pairs) serve all its rows of the token.
#include "mk_cache.h"
#include "mk_ptx.h"

namespace mk {
namespace {

using namespace ptx;

struct AppendParams {
  CacheView c;
  int layer, n_tokens;
  const void *q, *k, *v;
  int64_t qs, ks, vs;  // bytes from a token to the next
  const int32_t *starts, *seq_lens, *positions;
  const uint16_t *q_norm, *k_norm;
  uint16_t *q_out, *kc, *vc;
  const float2* rope;
  float eps;
};

template <typename T>
struct Vec8;  // 8 consecutive values as loaded
template <>
struct Vec8<uint16_t> {
  uint4 a;
  __device__ __forceinline__ void load(const uint16_t* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float f[8]) const {
    f[0] = bf16_lo(a.x); f[1] = bf16_hi(a.x); f[2] = bf16_lo(a.y); f[3] = bf16_hi(a.y);
    f[4] = bf16_lo(a.z); f[5] = bf16_hi(a.z); f[6] = bf16_lo(a.w); f[7] = bf16_hi(a.w);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void get(float f[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

__device__ __forceinline__ uint4 pack8(const float f[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Block (t, y): token t, rows y * kSlots + slot, stepping by all slots of the
// token.  kSlots rows at once, R of them in a lane's registers before it uses
// the first.  A token's place takes two loads that wait for each other (its sequence's numbers,
// then its page beside its rotations; one after the other, four loads, 16000 tokens of 32 rows of 64
// took 29 us instead of 26).  What hides them is the number of resident blocks, hence few threads
// and registers a block: the same tokens took 43 us with 32 slots and R = 4, 25 with 16 and 2 (rows in L2).
// Tokens of many rows want the larger block: 16384 of 120 fp32 rows of 128 245 us with 16 slots, 230 with 32
// (at 128 registers: two blocks an SM; the compiler's own choice, 140, took 144 us instead of 101 for 6000 with norms).
template <typename T, int HD, int kSlots, int R>
__global__ void __launch_bounds__(kSlots * HD / 16, kSlots == 32 ? 512 / (kSlots * HD / 16) : 0) append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = HD / 16;              // lanes of a row
  constexpr int kThreadsA = kSlots * kLanes;
  const CacheView& c = p.c;
  const int t = blockIdx.x, lane = threadIdx.x % kLanes, slot = blockIdx.y * kSlots + threadIdx.x / kLanes;
  const int step = gridDim.y * kSlots;
  const int nq = p.q ? c.nq : 0, nh = nq + 2 * c.nkv;

  // rows h, h + step, ...: queries, keys, values in this order
  auto source = [&](int h) -> const T* {
    const char* base = h < nq ? (const char*)p.q + t * p.qs
                              : (h < nq + c.nkv ? (const char*)p.k + t * p.ks : (const char*)p.v + t * p.vs);
    const int head = h < nq ? h : (h < nq + c.nkv ? h - nq : h - nq - c.nkv);
    return reinterpret_cast<const T*>(base) + (int64_t)head * HD + lane * 8;
  };
  Vec8<T> x[R][2];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = h0 + r * step;
      if (h < nh) {
        const T* s = source(h);
        x[r][0].load(s);
        x[r][1].load(s + HD / 2);
      }
    }
  };
  // Launched while the kernel ahead is under way; nothing of its is read before.  Nor is anything that it may write read as
  // constant (__ldg): only the rotations are.
  grid_wait();
  grid_launch_next();
  fetch(slot);  // in flight while the token finds its place

  // The token's sequence, its first token and the rows held before: a thread a sequence, all its loads at once.
  int b = t, first = t, held;
  if (p.starts) {
    __shared__ int owner[3];
    bool bad = false, mine = false;
#pragma unroll 4
    for (int i = threadIdx.x; i < c.B; i += kThreadsA) {
      const int lo = p.starts[i], hi = p.starts[i + 1], n = p.seq_lens[i];
      bad |= lo > hi || lo < 0 || hi > p.n_tokens;
      if (lo <= t && t < hi) {
        owner[0] = i;
        owner[1] = lo;
        owner[2] = n;
        mine = true;
      }
    }
    if (bad) set_status(c.status, MK_ERR_RANGE, t);
    if (!__syncthreads_or(mine)) return;  // before the first sequence or behind the last
    b = owner[0];
    first = owner[1];
    held = owner[2];
  } else {
    held = p.seq_lens[t];
  }
  const int64_t row = (int64_t)held + (t - first);
  const int pos = p.positions ? p.positions[t] : (int)row;
  const bool ok = row >= 0 && row < c.T && pos >= 0 && pos < c.T;
  bool in_pool = true;
  int64_t at = 0;
  float cs[8], sn[8];
  if (ok) {  // the page's entry and the rotations: neither waits for the other
    const float4* r4 = reinterpret_cast<const float4*>(p.rope + (int64_t)pos * (HD / 2) + lane * 8);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(r4 + i);
      cs[2 * i] = f.x; sn[2 * i] = f.y; cs[2 * i + 1] = f.z; sn[2 * i + 1] = f.w;
    }
    at = c.row(p.layer, b, (int)row, &in_pool);
  }
  if (!ok || !in_pool) {
    if (threadIdx.x == 0) set_status(c.status, MK_ERR_RANGE, t);
    return;
  }
  // Whole warps walk the rows together (the norm's sums are warp shuffles).
  const int warp_slot = blockIdx.y * kSlots + (threadIdx.x & ~31) / kLanes;
  for (int h0 = warp_slot, mine = slot; h0 < nh; h0 += R * step, mine += R * step) {
    if (h0 != warp_slot) fetch(mine);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int h = mine + r * step;
      float lo[8], hi[8];
      if (h < nh) {
        x[r][0].get(lo);
        x[r][1].get(hi);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) lo[i] = hi[i] = 0.f;
      }
      if (p.q_norm || p.k_norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(lo[i], lo[i], fmaf(hi[i], hi[i], ss));
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const uint16_t* gain = h < nq ? p.q_norm : (h < nq + c.nkv ? p.k_norm : nullptr);
        if (gain && h < nh) {
          const float inv = rsqrtf(ss * (1.0f / HD) + p.eps);  // off by 2^-22 at most: a root and a division took 5 to 10 % of the call
          Vec8<uint16_t> ga, gb;
          ga.a = *reinterpret_cast<const uint4*>(gain + lane * 8);
          gb.a = *reinterpret_cast<const uint4*>(gain + HD / 2 + lane * 8);
          float g[8];
          ga.get(g);
#pragma unroll
          for (int i = 0; i < 8; ++i) lo[i] *= inv * g[i];
          gb.get(g);
#pragma unroll
          for (int i = 0; i < 8; ++i) hi[i] *= inv * g[i];
        }
      }
      if (h >= nh) continue;
      uint16_t* dst;
      if (h < nq + c.nkv) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = lo[i] * cs[i] - hi[i] * sn[i], d = hi[i] * cs[i] + lo[i] * sn[i];
          lo[i] = a;
          hi[i] = d;
        }
        dst = h < nq ? p.q_out + ((int64_t)t * c.nq + h) * HD : p.kc + (at + (h - nq) * c.head_pitch()) * HD;
      } else {
        dst = p.vc + (at + (h - nq - c.nkv) * c.head_pitch()) * HD;
      }
      *reinterpret_cast<uint4*>(dst + lane * 8) = pack8(lo);
      *reinterpret_cast<uint4*>(dst + HD / 2 + lane * 8) = pack8(hi);
    }
  }
}

typedef void (*Kernel)(AppendParams);
template <typename T, int HD, int kSlots>
Kernel pick(int rows) {
  return rows <= 1 ? append_kernel<T, HD, kSlots, 1>
                   : (rows == 2 ? append_kernel<T, HD, kSlots, 2> : (rows == 3 ? append_kernel<T, HD, kSlots, 3> : append_kernel<T, HD, kSlots, 4>));
}
template <typename T, int HD>
Kernel pick(int slots, int rows) {
  return slots == 16 ? pick<T, HD, 16>(rows) : pick<T, HD, 32>(rows);
}

}  // namespace

cudaError_t append(const mk_cache& c, int layer, const mk_append_args& a, cudaStream_t stream) {
  const int es = a.dtype == MK_DTYPE_BF16 ? 2 : 4;
  AppendParams p{c.view, layer, a.n_tokens, a.q, a.k, a.v, a.q_stride * es, a.k_stride * es, a.v_stride * es,
                 a.starts, a.seq_lens, a.positions, (const uint16_t*)a.q_norm, (const uint16_t*)a.k_norm,
                 (uint16_t*)a.q_out, c.k, c.v, c.rope, c.d.rms_eps};
  const int nh = (a.q ? c.d.n_q_heads : 0) + 2 * c.d.n_kv_heads;
  const int slots = nh <= 64 ? 16 : 32;  // four rows a lane, or more
  // Few tokens: their rows are spread over more blocks, until the SMs have two each.
  const int most = (nh + slots - 1) / slots, want = (2 * c.n_sm + a.n_tokens - 1) / a.n_tokens;
  const dim3 grid(a.n_tokens, want < most ? want : most);
  const int rows = (most + (int)grid.y - 1) / (int)grid.y;  // a lane's
  const auto kernel = c.d.head_dim == 128 ? (es == 2 ? pick<uint16_t, 128>(slots, rows) : pick<float, 128>(slots, rows))
                                          : (es == 2 ? pick<uint16_t, 64>(slots, rows) : pick<float, 64>(slots, rows));
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(slots * (c.d.head_dim / 16));
  cfg.stream = stream;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace mk
