// Log probabilities of given tokens, entropy and the most likely alternatives.
//
// One pass over a row of logits x.  Every warp keeps its maximum m so far, every
// thread, in units of log2 (d = (x - m) log2 e), z = sum 2^d and s = sum 2^d d;
// the warps' (m, z, s) move to the row's maximum at the end:
//   logprob(t) = x_t - m - ln z,   entropy = ln z - ln 2 * s / z
// With the true maximum z is 1 at least and s 0 at most: nothing cancels, and a token that is all but
// certain keeps its small log probability (references up to 16 below the maximum left 1e-6 of both logarithms).
//
// Alternatives: a key packs the order-preserving map of the logit over the
// inverted index, so that the largest key is the largest logit, of the lowest
// index among equals, and no two keys are equal.  On the way a thread keeps only its
// largest maxima of a chunk and where they were.  At the row's end the k-th largest of
// the thread groups' maxima is a limit that k keys reach; the few chunk shares that
// reach it are read once more and their keys ranked.  (Candidates collected on the
// way, against a limit raised after chunks 1, 2, 4, ..., cost two barriers a raise and the slower
// the later the best ones came: 137 us instead of 117 for the 2047 rows below, 310 instead of 38 for 444 ascending ones.)
// The result does not depend on the order of arrival.
//
// Bound: memory for many rows (one read of the logits), at half of the issue slots and of the
// exponentials' rate: 2047 rows of 128256 bf16 logits take 88 us without alternatives (5.9
// TB/s) and 104 with 20 (5.1 TB/s); short rows, the latency of a row's join: 2000 of 32000 bf16 29 and 44 us.
// Few rows: each is cut over the blocks of a cluster, which join through distributed
// shared memory: no workspace, one launch.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "mk_cache.h"
#include "mk_ptx.h"

namespace mk {
namespace {

using namespace ptx;
namespace cg = cooperative_groups;

constexpr int kMaxTop = 32;
constexpr int kVecs = 4;      // 16-byte vectors of logits a thread holds at once
constexpr float kLn2 = 0.693147180559945309f;
typedef unsigned long long Key;

struct ScoreParams {
  const void* logits;
  int64_t stride;
  const int32_t* tokens;
  float *logprob, *entropy;
  int32_t* ids;
  float* tops;
  int vocab, top_k, rows;
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// Largest of the warp's 32 values, none of them NaN.
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
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
};

// The logits of one 16-byte vector, and their maximum (NaN ignored).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int kLen = 4;
  static __device__ __forceinline__ uint4 none() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
  static __device__ __forceinline__ float one(float x) { return x; }
  static __device__ __forceinline__ void get(const uint4& r, float f[4]) {
    f[0] = __uint_as_float(r.x); f[1] = __uint_as_float(r.y); f[2] = __uint_as_float(r.z); f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float top(const uint4 (&r)[kVecs]) {
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      float f[4];
      get(r[u], f);
      m = fmaxf(fmaxf(m, fmaxf(f[0], f[1])), fmaxf(f[2], f[3]));
    }
    return m;
  }
};
template <>
struct Vec<uint16_t> {
  static constexpr int kLen = 8;
  static __device__ __forceinline__ uint4 none() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
  static __device__ __forceinline__ float one(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
  static __device__ __forceinline__ void get(const uint4& r, float f[8]) {
    f[0] = bf16_lo(r.x); f[1] = bf16_hi(r.x); f[2] = bf16_lo(r.y); f[3] = bf16_hi(r.y);
    f[4] = bf16_lo(r.z); f[5] = bf16_hi(r.z); f[6] = bf16_lo(r.w); f[7] = bf16_hi(r.w);
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of bf16 pairs
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ float top(const uint4 (&r)[kVecs]) {
    uint32_t m = 0xff80ff80u;  // -infinity twice
#pragma unroll
    for (int u = 0; u < kVecs; ++u) m = max2(max2(m, max2(r[u].x, r[u].y)), max2(r[u].z, r[u].w));
    return fmaxf(bf16_lo(m), bf16_hi(m));
  }
};

constexpr int kStagesS = 4;   // chunks in flight, each NT * kVecs vectors
constexpr int kGroups = 64;   // thread groups whose maxima raise the limit
constexpr int kRoom = 64;     // keys a warp holds
constexpr int kMaxParts = 8;  // blocks of a cluster

// NT compute threads and a producer warp.
template <int NT>
struct Shared {
  static constexpr int kWarps = NT / 32, kStageBytes = NT * kVecs * 16;
  uint8_t ring[kStagesS][kStageBytes];
  unsigned long long full[kStagesS], empty[kStagesS];
  alignas(16) Key keys[kWarps * kRoom];  // each warp's, then all of them side by side
  Key best[kMaxTop];
  alignas(16) uint32_t tops[NT];  // the threads' maxima
  uint32_t raised;          // upper word of the limit
  int held[kWarps];
  int n_best, dead;
  float given;              // the given token's logit
  Sum part[kWarps];
  Sum sum;                  // this block's
};

// The NT compute threads.
template <int NT>
__device__ __forceinline__ void compute_bar() {
  asm volatile("bar.sync 1, %0;" ::"n"(NT) : "memory");
}

// Largest k of the n keys at `keys`, sorted, to `best` (not `keys` itself), by
// comparison with all; threads t of nt (whole warps), n <= 2 nt.  Few keys: a key's
// comparisons are shared by four threads.
__device__ __forceinline__ void rank_keys(const Key* keys, int n, int k, Key* best, int t, int nt) {
  if (n <= nt / 4) {
    const int e = t / 4;
    if ((t & ~31) / 4 >= n) return;
    const Key a = e < n ? keys[e] : 0;
    int rank = 0;
#pragma unroll 4
    for (int i = t % 4; i < n; i += 4) rank += keys[i] > a;
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if (e < n && t % 4 == 0 && rank < k) best[rank] = a;
    return;
  }
  for (; (t & ~31) < n; t += nt) {
    const Key a = t < n ? keys[t] : 0;
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i + 1 < n; i += 2) {
      const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(keys + i);
      rank += (q.x > a) + (q.y > a);
    }
    if (n & 1) rank += keys[n - 1] > a;
    if (t < n && rank < k) best[rank] = a;
  }
}

// Largest k of the keys of `parts` sorted lists of k, side by side at `keys`, sorted, to `best` (not `keys`
// itself): a key's rank is the number of larger ones in every list, found by halving in all lists at once.
__device__ __forceinline__ void merge_keys(const Key* keys, int parts, int k, Key* best, int t, int nt) {
  for (; t < parts * k; t += nt) {
    const Key a = keys[t];
    int larger[kMaxParts] = {};
#pragma unroll 1
    for (int step = 1 << (31 - __clz(k)); step; step >>= 1) {  // the first `larger` keys of a list are known to be larger
#pragma unroll
      for (int l = 0; l < kMaxParts; ++l) {
        const int at = larger[l] + step;
        if (l < parts && at <= k && keys[l * k + at - 1] > a) larger[l] = at;
      }
    }
    int rank = 0;
#pragma unroll
    for (int l = 0; l < kMaxParts; ++l) rank += larger[l];
    if (a && rank < k) best[rank] = a;
  }
}

// The block's part of a row, walked in aligned vectors: vector v covers logits
// from v * VEC - skew on, where skew is the row's offset from alignment.  Whole
// vectors [v0, v1) come through the ring in chunks; the partial ones at the
// row's ends are read by themselves (nothing outside the row is read).
template <typename T>
struct Part {
  const T* x;
  int skew, v0, v1;
  __device__ __forceinline__ Part(const ScoreParams& p, int row, int part, int parts) {
    constexpr int VEC = Vec<T>::kLen;
    x = reinterpret_cast<const T*>(p.logits) + (int64_t)row * p.stride;
    skew = (int)(((uintptr_t)x & 15) / sizeof(T));
    v0 = skew ? 1 : 0;
    v1 = max((p.vocab + skew) / VEC, v0);
    if (parts > 1) {
      const int n = v1 - v0, first = v0;
      v0 = first + (int)((int64_t)n * part / parts);
      v1 = first + (int)((int64_t)n * (part + 1) / parts);
    }
  }
};

// The given token's logit; NaN for a token that is none.
template <typename T>
__device__ __forceinline__ float given_logit(const ScoreParams& p, const T* x, int row) {
  const int t = __ldg(p.tokens + row);
  return t >= 0 && t < p.vocab ? Vec<T>::one(x[t]) : NAN;
}

// A thread's sums, m the maximum of its warp so far.  d = x log2 e - c is one fma, c = m log2 e rounded;
// what the rounding left (res) is put right when the sums move to another maximum.
struct Acc {
  float m = -INFINITY, c = 0.f, res = 0.f, z = 0.f, s = 0.f;
  bool huge = false;  // m log2 e overflows, or its rounding is no small part of a power of two
  // Sums to the reference whose c is `dm` below this one's.
  __device__ __forceinline__ void move(float dm) {
    if (z == 0.f) return;  // nothing but -infinity so far (a NaN sum is passed on)
    const float f = ex2(dm);
    s = f > 0.f ? f * (s + z * dm) : 0.f;
    z *= f;
  }
  // The warp's maximum has grown: `top` is this thread's largest logit, above it in some thread.
  __device__ __forceinline__ void lift(float top) {
    const float m0 = m, res0 = res;
    top = warp_max(top);
    m = top;
    huge = fabsf(top) > 1e6f;
    c = huge ? 0.f : top * kLog2e;
    res = huge ? 0.f : fmaf(top, kLog2e, -c);
    move(m0 == -INFINITY ? 0.f : (m0 - top) * kLog2e - res0 + res);
  }
  // d, bounded where 2^d is 0: 0 * -infinity is NaN
  __device__ __forceinline__ float bounded(float x) const { return max_nan(huge ? (x - m) * kLog2e : fmaf(x, kLog2e, -c), -150.f); }
  __device__ __forceinline__ Sum sum() {
    move(-res);
    return Sum{m, z, s};
  }
};

// Sum of the 32 lanes, in every lane.
__device__ __forceinline__ Sum warp_join(Sum a) {
  const float m = warp_max(a.m);
  Sum r{m, 0.f, 0.f};
  if (a.z != 0.f) {  // else nothing but -infinity (a NaN sum is passed on)
    const float dm = (a.m - (m == -INFINITY ? 0.f : m)) * kLog2e, f = ex2(dm);
    r.z = f * a.z;
    r.s = f > 0.f ? f * (a.s + a.z * dm) : 0.f;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    r.z += __shfl_xor_sync(0xffffffffu, r.z, o);
    r.s += __shfl_xor_sync(0xffffffffu, r.s, o);
  }
  return r;
}

// Rows of a cluster of `parts` blocks; with one block a row, blocks step over the rows.
template <typename T, int NT>
__global__ void __launch_bounds__(NT + 32, NT == 256 ? 3 : 6) score_kernel(const __grid_constant__ ScoreParams p) {
  constexpr int VEC = Vec<T>::kLen, U = kVecs, CH = NT * U;
  using S = Shared<NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  S& sh = *reinterpret_cast<S*>(smem);
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, k = p.top_k;
  const int row0 = blockIdx.x / parts, row_step = gridDim.x / parts;
  volatile int* dead = &sh.dead;

  if (tid == 0) {
    for (int i = 0; i < kStagesS; ++i) {
      mbar_init(smem_addr(&sh.full[i]), 1);
      mbar_init(smem_addr(&sh.empty[i]), S::kWarps);
    }
    sh.dead = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == S::kWarps) {  // ---- producer: the chunks of all rows, as far ahead as the ring goes
    if (lane == 0) {
      int slot = 0;
      uint32_t phase = 0;
      for (int row = row0; row < p.rows; row += row_step) {
        const Part<T> r(p, row, part, parts);
        const uint8_t* src = reinterpret_cast<const uint8_t*>(r.x - r.skew);
        for (int v = r.v0; v < r.v1; v += CH) {
          const uint32_t bytes = min(CH, r.v1 - v) * 16;
          mbar_wait(smem_addr(&sh.empty[slot]), phase ^ 1, dead);
          if (!*dead) {
            mbar_expect_tx(smem_addr(&sh.full[slot]), bytes);
            bulk_load(smem_addr(sh.ring[slot]), src + (int64_t)v * 16, bytes, smem_addr(&sh.full[slot]));
          }
          if (++slot == kStagesS) slot = 0, phase ^= 1;
        }
      }
      if (*dead) {  // copies still in flight land before the block's shared memory is given back
        const uint64_t t0 = globaltimer();
        for (int i = 0; i < kStagesS; ++i)
          while (!mbar_try(smem_addr(&sh.full[i]), i < slot ? phase : phase ^ 1) && globaltimer() - t0 < 10000000ull) {
          }
      }
    }
    if (parts > 1) {  // one row, on which the compute warps have no time to wait for a word
      if (lane == 0 && part == 0) sh.given = given_logit<T>(p, reinterpret_cast<const T*>(p.logits) + (int64_t)row0 * p.stride, row0);
      __syncwarp();
      cluster.sync();
      cluster.sync();
    }
    return;
  }

  Key* mine = sh.keys + warp * kRoom;
  int slot = 0;
  uint32_t phase = 0;
  for (int row = row0; row < p.rows; row += row_step) {
    const Part<T> r(p, row, part, parts);
    Acc acc;
    // The thread's largest chunk maximum and the two next ones, each the first of equal ones; their chunks (as first
    // vectors; -1: none, or the row's partial vectors, whose keys are already among the warp's).
    float most = -INFINITY, second = -INFINITY, third = -INFINITY;
    int where = -1, where2 = -1, where3 = -1;
    Key limit = 0;             // keys below it are not among the best,
    float least = -3.402823466e38f;  // nor are logits below this one
    auto set_limit = [&](Key to) {
      if (to > limit) {
        limit = to;
        least = from_ordered((uint32_t)(to >> 32));
      }
    };
    int held = 0;   // keys of this warp
    float given = NAN;
    if (tid == 0 && parts == 1) given = given_logit<T>(p, r.x, row);
    // the keys of a warp, a lane each (0: none), into its room; a full room is cut to its k best
    auto push = [&](Key key) {
      const bool pass = key != 0 && key >= limit;
      const uint32_t who = __ballot_sync(0xffffffffu, pass);
      const int n = __popc(who);
      if (held + n > kRoom) {
        __syncwarp();
        const Key x = lane < held ? mine[lane] : 0, y = lane + 32 < held ? mine[lane + 32] : 0;
        int rx = 0, ry = 0;
        for (int i = 0; i < held; ++i) {
          const Key q = mine[i];
          rx += q > x;
          ry += q > y;
        }
        __syncwarp();
        if (lane < held && rx < k) mine[rx] = x;
        if (lane + 32 < held && ry < k) mine[ry] = y;
        __syncwarp();
        held = k;  // more than 32 keys were held
        set_limit(mine[k - 1] + 1);
      }
      if (pass) mine[held + __popc(who & ((1u << lane) - 1))] = key;
      held += n;
    };

    // the partial vectors: at the row's start this side of alignment, and behind its last whole one
    if (part == 0 && warp == 0) {
      const int tail = max((p.vocab + r.skew) / VEC, r.skew ? 1 : 0) * VEC - r.skew;
      const int i = lane < VEC ? lane : tail + lane - VEC;
      const bool in = lane < VEC ? r.skew && i < VEC - r.skew && i < p.vocab : lane < 2 * VEC && i < p.vocab;
      const float f = in ? Vec<T>::one(r.x[i]) : -INFINITY;
      most = fmaxf(f, -INFINITY);
      if (__any_sync(0xffffffffu, most > -INFINITY)) acc.lift(most);
      const float d = acc.bounded(f);
      acc.z = ex2(d);
      acc.s = acc.z * d;
      if (k > 0) push(f > -INFINITY ? make_key(f, i) : 0);
    }

    for (int v0 = r.v0; v0 < r.v1; v0 += CH) {
      mbar_wait(smem_addr(&sh.full[slot]), phase, dead);
      const T* here = reinterpret_cast<const T*>(sh.ring[slot]);
      uint4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u] = reinterpret_cast<const uint4*>(here)[u * NT + tid];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&sh.empty[slot]));
      if (++slot == kStagesS) slot = 0, phase ^= 1;
      if (v0 + CH > r.v1) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v0 + u * NT + tid >= r.v1) raw[u] = Vec<T>::none();
      }
      const float top = Vec<T>::top(raw);
      if (k > 0) {
        const bool first = top > most, next = top > second;
        const bool last = next ? second >= third : top > third;  // what is second now came before an equal third
        where3 = last ? (next ? where2 : v0) : where3;
        third = last ? (next ? second : top) : third;
        second = first ? most : (next ? top : second);
        where2 = first ? where : (next ? v0 : where2);
        most = first ? top : most;
        where = first ? v0 : where;
      }
      if (__any_sync(0xffffffffu, top > acc.m)) acc.lift(top);
      F2 z2 = pack2(0.f, 0.f), s2 = z2;
      const F2 back = pack2(-acc.c, -acc.c), scale = pack2(kLog2e, kLog2e);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float f[VEC];
        Vec<T>::get(raw[u], f);
#pragma unroll
        for (int i = 0; i < VEC; i += 2) {
          const F2 d = fma2(pack2(f[i], f[i + 1]), scale, back);
          float d0, d1;
          unpack2(d, d0, d1);
          const F2 e = pack2(ex2(d0), ex2(d1));
          z2 = add2(z2, e);
          s2 = fma2(e, d, s2);
        }
      }
      float z0, z1, s0, s1;
      unpack2(z2, z0, z1);
      unpack2(s2, s0, s1);
      float z = z0 + z1, s = s0 + s1;
      if (!(s == s) || acc.huge) {
        // 0 * -infinity (masked logits), a real NaN, or a maximum too large for the fma: again, bounded
        z = s = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[VEC];
          Vec<T>::get(raw[u], f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float d = acc.bounded(f[i]), e = ex2(d);
            z += e;
            s = fmaf(e, d, s);
          }
        }
      }
      acc.z += z;
      acc.s += s;
    }

    // the warps' sums; a limit of the keys: the k-th largest maximum of the thread groups, which k keys reach
    Sum a = warp_join(acc.sum());
    if (lane == 0) sh.part[warp] = a;
    constexpr int GT = NT / kGroups;
    // Thread t is of group t % kGroups: the threads that have a part of a short row are in different ones (300 bf16 logits,
    // 20 alternatives: neighbours in one group left fewer than 20 groups and no limit, 12 us against 8).  No two
    // groups' values are equal; a limit that is too low by less than kGroups steps is still one.
    sh.tops[tid] = (most > -INFINITY ? ordered(most) & ~(kGroups - 1u) : 0u) | tid % kGroups;
    compute_bar<NT>();
    if (warp == 0) {
      a = warp_join(lane < S::kWarps ? sh.part[lane] : Sum{-INFINITY, 0.f, 0.f});
      if (*dead) a.z = NAN;  // a copy never came: the block's share, and with it the row, has no scores
      if (lane == 0) sh.sum = a;
    }
    int n = 0, got = 0;
    if (k > 0) {
      // GT threads share the comparisons of a group's maximum with the others (each from another bank on)
      uint32_t g = 0;
#pragma unroll
      for (int q = 0; q < GT; ++q) g = max(g, sh.tops[q * kGroups + tid / GT]);
      int rank = 0;
#pragma unroll
      for (int i = 0; i < kGroups / GT; i += 4) {
        uint4 w = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < GT; ++q) {
          const uint4 x = *reinterpret_cast<const uint4*>(sh.tops + q * kGroups + tid % GT * (kGroups / GT) + ((i + tid % GT * 4) & (kGroups / GT - 1)));
          w = make_uint4(max(w.x, x.x), max(w.y, x.y), max(w.z, x.z), max(w.w, x.w));
        }
        rank += (w.x > g) + (w.y > g) + (w.z > g) + (w.w > g);
      }
#pragma unroll
      for (int o = GT / 2; o; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (rank == k - 1 && tid % GT == 0) sh.raised = g & ~(kGroups - 1u);
      compute_bar<NT>();
      set_limit((Key)sh.raised << 32);
      // The warp looks through the chunks whose maxima reach the limit, read once more: a lane a logit of one thread's
      // share, or of two whose 16 logits fill a half warp each; several shares' loads under way at once.
      constexpr int kMine = U * VEC, kAtOnce = 32 / kMine, kAhead = 4;
      const int at = lane % kMine, u = at / VEC, i = at % VEC;
      auto look = [&](uint32_t todo, int from) {
        while (todo) {
          float f[kAhead];
          int index[kAhead];
#pragma unroll
          for (int q = 0; q < kAhead; ++q) {
            int t = __ffs(todo) - 1;
            todo &= todo - 1;
            if (kAtOnce == 2) {
              const int t2 = __ffs(todo) - 1;
              todo &= todo - 1;
              if (lane >= kMine) t = t2;
            }
            const int v = __shfl_sync(0xffffffffu, from, t & 31) + u * NT + (tid & ~31) + t;
            f[q] = -INFINITY;
            index[q] = v * VEC - r.skew + i;
            if (t >= 0 && v < r.v1) f[q] = Vec<T>::one(r.x[index[q]]);
          }
#pragma unroll
          for (int q = 0; q < kAhead; ++q) push(f[q] > -INFINITY ? make_key(f[q], index[q]) : 0);
        }
      };
      // whether this thread's share of a chunk, or of a later one of no larger maximum, can hold a key to be kept
      auto reaches = [&](float top, int v0) {
        return top >= least && make_key(top, max((v0 + tid) * VEC - r.skew, 0)) >= limit;
      };
      look(__ballot_sync(0xffffffffu, where >= 0 && reaches(most, where)), where);
      look(__ballot_sync(0xffffffffu, where2 >= 0 && reaches(second, where2)), where2);
      // a thread with more than two such chunks (one row of 20 has one): its others are looked for, a lane a chunk
      for (uint32_t more = __ballot_sync(0xffffffffu, reaches(third, where3)); more; more &= more - 1) {
        const int t = __ffs(more) - 1, known = __shfl_sync(0xffffffffu, where, t), known2 = __shfl_sync(0xffffffffu, where2, t);
        for (int v0 = r.v0; v0 < r.v1; v0 += 32 * CH) {
          const int mine0 = v0 + lane * CH, v = mine0 + (tid & ~31) + t;
          uint4 raw[U];
#pragma unroll
          for (int w = 0; w < U; ++w)
            raw[w] = v + w * NT < r.v1 ? __ldg(reinterpret_cast<const uint4*>(r.x - r.skew) + v + w * NT) : Vec<T>::none();
          const float top = Vec<T>::top(raw);
          uint32_t hit = __ballot_sync(0xffffffffu, top >= least && mine0 != known && mine0 != known2);
          for (; hit; hit &= hit - 1) look(1u << t, v0 + (__ffs(hit) - 1) * CH);
        }
      }
      if (lane == 0) sh.held[warp] = held;
      const Key ka = lane < held ? mine[lane] : 0, kb = lane + 32 < held ? mine[lane + 32] : 0;
      compute_bar<NT>();
      int before = 0;
#pragma unroll
      for (int w = 0; w < S::kWarps; ++w) {
        if (w == warp) before = n;
        n += sh.held[w];
      }
      if (lane < held) sh.keys[before + lane] = ka;
      if (lane + 32 < held) sh.keys[before + lane + 32] = kb;
      compute_bar<NT>();
      got = min(n, k);
      rank_keys(sh.keys, n, k, sh.best, tid, NT);
      if (tid >= n && tid < k) sh.best[tid] = 0;
      if (tid == 0) sh.n_best = got;
    }
    compute_bar<NT>();

    if (parts > 1) {  // one row a cluster
      cluster.sync();
      if (part == 0) {
        if (warp == 0) {
          a = warp_join(lane < parts ? cluster.map_shared_rank(&sh, lane)->sum : Sum{-INFINITY, 0.f, 0.f});
          if (lane == 0) sh.sum = a;
        }
        // the blocks' best keys side by side (0 where one has fewer), one remote read a thread
        n = parts * k;
        for (int i = tid; i < n; i += NT) sh.keys[i] = cluster.map_shared_rank(&sh, i / k)->best[i % k];
        got = lane < parts ? cluster.map_shared_rank(&sh, lane)->n_best : 0;
        got = min(__reduce_add_sync(0xffffffffu, got), k);
        compute_bar<NT>();
        merge_keys(sh.keys, parts, k, sh.best, tid, NT);
        compute_bar<NT>();
      }
      cluster.sync();  // a block's shared memory stays until it has been read
    }
    if (part == 0) {
      Sum q = sh.sum;
      if (q.z < 1.f) q.z = 1.f;  // less, or s above 0, is rounding: no log probability above 0, no entropy below
      if (q.s > 0.f) q.s = 0.f;
      const float lnz = logf(q.z);
      const bool none = !(q.z == q.z) || isinf(q.m);  // NaN (a copy that never came, too), infinities, nothing allowed
      if (tid == 0) {
        if (parts > 1) given = sh.given;
        p.logprob[row] = none ? NAN : given - q.m - lnz;
        if (p.entropy) p.entropy[row] = none ? NAN : lnz - kLn2 * q.s / q.z;
      }
      if (tid < k) {
        const bool has = !none && tid < got;
        const Key key = has ? sh.best[tid] : 0;
        p.ids[(int64_t)row * k + tid] = has ? (int32_t)~(uint32_t)key : -1;
        p.tops[(int64_t)row * k + tid] = none ? NAN : (has ? from_ordered((uint32_t)(key >> 32)) - q.m - lnz : -INFINITY);
      }
    }
  }
}

template <typename T, int NT>
cudaError_t launch(const ScoreParams& p, int parts, int n_sm, cudaStream_t stream) {
  // per device and process, not per call: the limit is an attribute of the function
  static std::atomic<uint64_t> prepared;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(prepared.load(std::memory_order_relaxed) >> (dev & 63) & 1)) {
    e = cudaFuncSetAttribute(score_kernel<T, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared<NT>));
    if (e != cudaSuccess) return e;
    prepared.fetch_or(1ull << (dev & 63), std::memory_order_relaxed);
  }
  const int resident = parts > 1 ? p.rows : n_sm * (NT == 256 ? 3 : 6);  // rows at once
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min(p.rows, resident) * parts);
  cfg.blockDim = dim3(NT + 32);
  cfg.dynamicSmemBytes = sizeof(Shared<NT>);
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
cudaError_t score(const ScoreParams& p, int n_sm, cudaStream_t stream) {
  // More rows than large blocks fit the SMs, and not long: small blocks, twice as many (20 alternatives of bf16
  // rows: 500 of 4096 7.4 us against 11.6, 2000 of 16000 30.5 against 33.7, of 32000 43.7 against 44.6, 1000 of 32000 24.7
  // against 24.1, 200 of 32000 11.6 against 9.9; of fp32 rows of 50257 79 both; 2000 bf16 rows of 50257 would gain, 58 against 62).
  if (p.rows > 3 * n_sm && p.vocab <= 32768) return launch<T, 128>(p, 1, n_sm, stream);
  // Few rows: as many blocks a row as fill the SMs, 4096 logits a block at least (20 alternatives of fp32 rows: one of
  // 128256 9.1 us, 15.9 as one block; 64 of 151936 13.8 with 4 blocks each, 19.3 with one, 21.3 with 8).
  int parts = 1;
  while (parts < kMaxParts && p.rows * parts < n_sm && p.vocab / (2 * parts) >= 4096) parts *= 2;
  return launch<T, 256>(p, parts, n_sm, stream);
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
  const mk::ScoreParams p{logits, row_stride, tokens, out_logprob, out_entropy, out_top_ids, out_top_logprobs, vocab, top_k, n_rows};
  const cudaError_t e = es == 2 ? mk::score<uint16_t>(p, n_sm, (cudaStream_t)stream)
                                : mk::score<float>(p, n_sm, (cudaStream_t)stream);
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
  // The handle's own description is its first member (csrc/mk_api.cu): the buffers are of its sizes.
  const mk_model_desc& own = *reinterpret_cast<const mk_model_desc*>(h);
  if (own.n_layers != desc->n_layers || own.batch != desc->batch || own.hidden != desc->hidden || own.vocab != desc->vocab)
    return MK_ERR_INVALID_ARG;
  if (top_k > mk::kMaxTop) return MK_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  // a step's launch carries the step's number: replayed, its waits would find the counters of the steps before
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &capture) != cudaSuccess) {
    cudaGetLastError();
    return MK_ERR_CUDA;
  }
  if (capture != cudaStreamCaptureStatusNone) return MK_ERR_UNSUPPORTED;
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
