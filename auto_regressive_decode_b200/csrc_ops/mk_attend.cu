// Attention of one query token a sequence over a cache whose first positions
// all sequences share.
//
// Query heads that read the same cache rows are the rows of one product: for a
// KV head, the prefix serves batch x group rows at once (group = query heads
// per KV head), a sequence's own positions serve its group rows.  Both are cut
// into tiles of kTile positions; a "group" is the tiles of one set of rows
// (prefix: KV head x row tile; own: sequence x KV head).  The tiles of all groups, in
// order, are dealt to the blocks as equal contiguous runs; a block's run within
// a group is a piece, which keeps the running maximum m and sum l of every row
// (softmax in one pass) and its unnormalised output o, and leaves them in the
// workspace.  A second kernel joins the pieces of a row:
//   M = max m,  o = sum 2^(m - M) o / sum 2^(m - M) l,  lse = ln 2 (M + log2 sum 2^(m - M) l)
// with scores in units of log2 (scale * log2 e folded into one factor).
//
// Bound: memory, 4 head_dim bytes of cache a position and KV head against
// 4 head_dim flops a row; a producer warp keeps a ring of TMA boxes in flight.
#include <algorithm>

#include "mk_cache.h"
#include "mk_ptx.h"

namespace mk {
namespace {

using namespace ptx;

constexpr int kWarps = 8;                        // compute warps; warp 8 is the producer
constexpr int kAttThreads = kWarps * 32 + 32;
constexpr int kMaxRows = 64;                     // rows of a prefix row tile
constexpr int kRedPitch = 64 + 4;                // floats a row of the joining buffer (64 columns at a time)

template <int HD>
struct Layout {
  static constexpr int kSlotBytes = kTile * HD * 2;         // one tile of K or of V: [HD/64][128 rows][128 B], swizzled
  static constexpr int kSlots = 160 * 1024 / kSlotBytes;
  static constexpr int kRed = kSlots * kSlotBytes;          // float[kWarps][16][kRedPitch]
  static constexpr int kMl = kRed + kWarps * 16 * kRedPitch * 4;  // float2[kWarps][16]
  static constexpr int kCum = kMl + kWarps * 16 * 8;        // int[kCacheMaxBatch + 1]: own tiles of the sequences before
  static constexpr int kLen = kCum + (kCacheMaxBatch + 4) * 4;    // int[kCacheMaxBatch]
  static constexpr int kCtl = kLen + kCacheMaxBatch * 4;
  static constexpr int kTotal = kCtl + 512 + 1024;          // 1024: the ring is aligned by hand
};

struct Ctl {
  unsigned long long full[20], empty[20];
  int dead, max_len;
};
static_assert(sizeof(Ctl) <= 512, "control block");

struct AttendParams {
  CacheView c;
  int layer, group, box;
  int prefix, base;        // own tiles start at base: prefix rounded down to a whole box of a paged cache
  int row_tile, row_tiles; // prefix rows per group, row tiles per KV head
  float scale;             // scale * log2 e
  const uint16_t* q;
  const int32_t* seq_lens;
  uint16_t* out;
  float* lse;
  // workspace
  float *pre_o, *own_o;    // [piece][row_tile | group][hd]
  float2 *pre_ml, *own_ml; // [piece][rows]
  int* sched;              // [0] prefix tiles a group, [2, 3] tiles (int64), [4...] own tiles of the sequences before (batch + 1)
};

// Blocks that work: a block has at least one tile.
__device__ __forceinline__ int active_blocks(int64_t tiles, int grid) { return (int)min(tiles, (int64_t)grid); }
// First tile of block i of G, and the block that holds tile u.
__device__ __forceinline__ int64_t first_tile(int64_t tiles, int i, int G) { return tiles * i / G; }
__device__ __forceinline__ int block_of(int64_t u, int64_t tiles, int G) { return (int)(((u + 1) * G - 1) / tiles); }

__device__ __forceinline__ int own_tiles(const AttendParams& p, int len) {
  return len > p.prefix ? (len - p.base + kTile - 1) / kTile : 0;
}

// A piece: tiles [i0, i1) of a group.
struct Piece {
  bool shared;
  int b, kvh, tile0;  // own: the sequence; shared: first row of the row tile
  int i0, i1, gidx;
};

struct Walk {
  const AttendParams& p;
  const int* cum;
  int pre_tiles, pre_groups;
  int64_t u, end;
  __device__ Walk(const AttendParams& prm, const int* cumulative, int pre, int64_t u0, int64_t u1)
      : p(prm), cum(cumulative), pre_tiles(pre), pre_groups(pre ? prm.c.nkv * prm.row_tiles : 0), u(u0), end(u1) {}
  __device__ __forceinline__ bool next(Piece& a) {
    if (u >= end) return false;
    const int64_t shared_tiles = (int64_t)pre_groups * pre_tiles;
    int n;
    if (u < shared_tiles) {
      a.shared = true;
      a.gidx = (int)(u / pre_tiles);
      a.i0 = (int)(u % pre_tiles);
      a.kvh = a.gidx / p.row_tiles;
      a.tile0 = a.gidx % p.row_tiles * p.row_tile;
      a.b = 0;
      n = pre_tiles;
    } else {
      const int64_t v = u - shared_tiles;
      const int w = (int)(v / p.c.nkv);
      int lo = 0, hi = p.c.B;  // the sequence with cum[b] <= w < cum[b + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cum[mid] <= w) lo = mid; else hi = mid;
      }
      n = cum[lo + 1] - cum[lo];
      const int r = (int)(v - (int64_t)cum[lo] * p.c.nkv);
      a.shared = false;
      a.b = lo;
      a.kvh = r / n;
      a.i0 = r % n;
      a.tile0 = 0;
      a.gidx = lo * p.c.nkv + a.kvh;
    }
    a.i1 = (int)min((int64_t)n, a.i0 + (end - u));
    u += a.i1 - a.i0;
    return true;
  }
};

template <int HD>
__global__ void __launch_bounds__(kAttThreads, 1)
    attend_tiles(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  using S = Layout<HD>;
  constexpr int KS = HD / 16;  // k-steps of the score product
  constexpr int NT = HD / 8;   // column tiles of the output
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const uint32_t ring = smem_addr(smem);
  float* red = reinterpret_cast<float*>(smem + S::kRed);
  float2* sml = reinterpret_cast<float2*>(smem + S::kMl);
  int* cum = reinterpret_cast<int*>(smem + S::kCum);
  int* lens = reinterpret_cast<int*>(smem + S::kLen);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + S::kCtl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const CacheView& c = p.c;
  volatile int* dead = &ctl->dead;

  if (tid == 0) {
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 1);
      mbar_init(smem_addr(&ctl->empty[s]), kWarps);
    }
    ctl->dead = 0;
    ctl->max_len = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // lengths, and the tiles of the sequences before each
  int longest = 0;
  for (int b = tid; b < c.B; b += kAttThreads) {
    int n = __ldg(p.seq_lens + b);
    if (n < 0 || n > c.T) {
      if (blockIdx.x == 0) set_status(c.status, MK_ERR_RANGE, b);
      n = n < 0 ? 0 : c.T;
    }
    lens[b] = n;
    longest = max(longest, n);
  }
  if (longest) atomicMax(&ctl->max_len, longest);
  __syncthreads();
  if (warp == 0) {
    int sum = 0;
    for (int b0 = 0; b0 < c.B; b0 += 32) {
      const int b = b0 + lane;
      const int n = b < c.B ? own_tiles(p, lens[b]) : 0;
      int x = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < c.B) cum[b] = sum + x - n;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) cum[c.B] = sum;
  }
  __syncthreads();
  // No sequence attends behind the longest: what lies there is not read.
  const int prefix_end = min(p.prefix, ctl->max_len);
  const int pre_tiles = (prefix_end + kTile - 1) / kTile;
  const int64_t tiles = (int64_t)pre_tiles * p.row_tiles * c.nkv + (int64_t)cum[c.B] * c.nkv;
  if (blockIdx.x == 0) {
    for (int b = tid; b <= c.B; b += kAttThreads) p.sched[4 + b] = cum[b];
    if (tid == 0) {
      p.sched[0] = pre_tiles;
      *reinterpret_cast<int64_t*>(p.sched + 2) = tiles;
    }
  }
  const int G = active_blocks(tiles, gridDim.x), cta = blockIdx.x;
  if (cta >= G) return;
  Walk walk(p, cum, pre_tiles, first_tile(tiles, cta, G), first_tile(tiles, cta + 1, G));
  Piece a;

  if (warp == kWarps) {  // ---- producer: K tile, V tile, K tile, ... into the ring
    uint32_t slot = 0, phase = 0;
    const int boxes = kTile / p.box;               // boxes of one 64-column block
    const int cb = lane / boxes, j = lane % boxes; // this lane's box
    const bool mine = cb < HD / 64;
    while (walk.next(a)) {
      const int start = a.shared ? 0 : p.base, lo = a.shared ? 0 : p.prefix, hi = a.shared ? prefix_end : lens[a.b];
      for (int i = a.i0; i < a.i1; ++i) {
        const int t0 = start + i * kTile, at = t0 + j * p.box;
        const bool wanted = mine && at < hi && at + p.box > lo;
        bool ok = true;
        int row = 0;
        if (wanted) row = (int)(c.row(p.layer, a.b, at, &ok) + a.kvh * c.head_pitch());
        if (!ok) set_status(c.status, MK_ERR_RANGE, a.b);
        const int n = __popc(__ballot_sync(0xffffffffu, wanted));
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t full = smem_addr(&ctl->full[slot]);
          mbar_wait(smem_addr(&ctl->empty[slot]), phase ^ 1, dead);
          if (!__any_sync(0xffffffffu, *dead)) {
            if (lane == 0) mbar_expect_tx(full, n * p.box * 128);
            __syncwarp();
            if (wanted)
              tma_box2(ring + slot * S::kSlotBytes + cb * (kTile * 128) + j * p.box * 128, kv ? (const void*)&vmap : (const void*)&kmap,
                       cb * 64, row, full);
          }
          __syncwarp();
          if (++slot == S::kSlots) slot = 0, phase ^= 1;
        }
      }
    }
    // a block that gave up waits for its own copies in flight before it ends
    if (__any_sync(0xffffffffu, *dead)) {
      for (int s = 0; s < S::kSlots; ++s) {
        const uint64_t t0 = globaltimer();
        const uint32_t full = smem_addr(&ctl->full[s]);
        // the slot's latest fill: the phase before the producer's next one
        const uint32_t last = (uint32_t)s < slot ? phase : phase ^ 1;
        while (!mbar_try(full, last) && globaltimer() - t0 < 10000000ull) {
        }
      }
      if (lane == 0) set_status(c.status, MK_ERR_DEVICE_TIMEOUT, cta);
    }
    return;
  }

  // ---- compute warps: rows as the mma's M (16 a row block), warps = row blocks x position splits
  uint32_t slot = 0, phase = 0;
  const int gq = lane / 4, cq = lane % 4;
  while (walk.next(a)) {
    const int rows = a.shared ? min(p.row_tile, c.B * p.group - a.tile0) : p.group;
    const int R = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);  // row blocks
    const int rb = warp % R, sp = warp / R;
    const int lo = a.shared ? 0 : p.prefix, start = a.shared ? 0 : p.base;
    const int hi = a.shared ? prefix_end : lens[a.b];
    // this lane's two rows: their positions end at lim
    int lim[2];
    const uint16_t* qp[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = rb * 16 + gq + 8 * h;
      const int b = a.shared ? (a.tile0 + r) / p.group : a.b, jh = a.shared ? (a.tile0 + r) % p.group : r;
      lim[h] = r < rows ? min(lens[b], hi) : 0;
      qp[h] = r < rows ? p.q + ((int64_t)b * c.nq + a.kvh * p.group + jh) * HD + cq * 2 : nullptr;
    }
    uint32_t qf[KS][4];
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        qf[k][e] = qp[e & 1] ? __ldg(reinterpret_cast<const uint32_t*>(qp[e & 1] + k * 16 + (e >> 1) * 8)) : 0u;

    float o[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int i = a.i0; i < a.i1; ++i) {
      const uint32_t kslot = ring + slot * S::kSlotBytes, kfull = smem_addr(&ctl->full[slot]), kphase = phase;
      const uint32_t kempty = smem_addr(&ctl->empty[slot]);
      if (++slot == S::kSlots) slot = 0, phase ^= 1;
      const uint32_t vslot = ring + slot * S::kSlotBytes, vfull = smem_addr(&ctl->full[slot]), vphase = phase;
      const uint32_t vempty = smem_addr(&ctl->empty[slot]);
      if (++slot == S::kSlots) slot = 0, phase ^= 1;
      const int t0 = start + i * kTile;
      mbar_wait(kfull, kphase, dead);
      bool have_v = false;
      for (int js = 0; js < R; ++js) {  // 16-position slices of this warp: sp * R + js
        const int s0 = (sp * R + js) * 16, p0 = t0 + s0;
        if (p0 < hi && p0 + 16 > lo) {
          float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
          {
            const int mi = lane >> 3, row = s0 + (mi >> 1) * 8 + (lane & 7);
#pragma unroll
            for (int k = 0; k < KS; ++k) {
              const int ch = k * 2 + (mi & 1);
              uint32_t f[4];
              ldmatrix_x4(f, kslot + (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
              mma16816(s[0], qf[k], f[0], f[1]);
              mma16816(s[1], qf[k], f[2], f[3]);
            }
          }
          // mask, maximum
          float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int pos = p0 + n * 8 + cq * 2 + (e & 1);
              s[n][e] = pos >= lo && pos < lim[e >> 1] ? s[n][e] * p.scale : -INFINITY;
              mx[e >> 1] = fmaxf(mx[e >> 1], s[n][e]);
            }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            mx[h] = fmaxf(mx[h], m[h]);
          }
          const bool grew = mx[0] > m[0] || mx[1] > m[1];
          float ref[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) ref[h] = mx[h] == -INFINITY ? 0.f : mx[h];
          if (__any_sync(0xffffffffu, grew)) {
            const float f0 = ex2(m[0] - ref[0]), f1 = ex2(m[1] - ref[1]);
            l[0] *= f0;
            l[1] *= f1;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              o[n][0] *= f0;
              o[n][1] *= f0;
              o[n][2] *= f1;
              o[n][3] *= f1;
            }
            m[0] = mx[0];
            m[1] = mx[1];
          }
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              s[n][e] = ex2(s[n][e] - ref[e >> 1]);
              l[e >> 1] += s[n][e];
            }
          // probabilities as the A operand of the second product: rounded to bf16, as the cache is
          const uint32_t pf[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                                  pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
          if (!have_v) {
            mbar_wait(vfull, vphase, dead);
            have_v = true;
          }
          // rows outside [lo, hi) hold anything, and 0 x NaN is NaN: clear them in the fragment
          uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
          if (p0 < lo || p0 + 16 > hi) {
            const int q0 = p0 + cq * 2;
            keep0 = (q0 >= lo && q0 < hi ? 0xffffu : 0u) | (q0 + 1 >= lo && q0 + 1 < hi ? 0xffff0000u : 0u);
            keep1 = (q0 + 8 >= lo && q0 + 8 < hi ? 0xffffu : 0u) | (q0 + 9 >= lo && q0 + 9 < hi ? 0xffff0000u : 0u);
          }
          const int mi = lane >> 3, row = s0 + (mi & 1) * 8 + (lane & 7);
#pragma unroll
          for (int n = 0; n < NT; n += 2) {
            const int ch = n + (mi >> 1);
            uint32_t f[4];
            ldmatrix_x4_trans(f, vslot + (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
            mma16816(o[n], pf, f[0] & keep0, f[1] & keep1);
            mma16816(o[n + 1], pf, f[2] & keep0, f[3] & keep1);
          }
        }
      }
      if (!have_v) mbar_wait(vfull, vphase, dead);  // nothing of it is this warp's: still seen before it is given back
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(kempty);
        mbar_arrive(vempty);
      }
    }

    // ---- join the position splits of each row block and leave the piece in the workspace
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (cq == 0) sml[warp * 16 + gq + 8 * h] = make_float2(m[h], l[h]);
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float M = -INFINITY;
      for (int w = rb; w < kWarps; w += R) M = fmaxf(M, sml[w * 16 + gq + 8 * h].x);
      f[h] = M == -INFINITY ? 0.f : ex2(m[h] - M);
    }
    const int64_t pid = (int64_t)cta + a.gidx;
    const int stride = a.shared ? p.row_tile : p.group;
    float* po = (a.shared ? p.pre_o : p.own_o) + pid * stride * HD;
    float2* pml = (a.shared ? p.pre_ml : p.own_ml) + pid * stride;
    if (tid < rows) {
      const int blk = tid / 16, r = tid % 16;
      float M = -INFINITY, L = 0.f;
      for (int w = blk; w < kWarps; w += R) M = fmaxf(M, sml[w * 16 + r].x);
      for (int w = blk; w < kWarps; w += R) {
        const float2 x = sml[w * 16 + r];
        if (x.y != 0.f) L += x.y * ex2(x.x - M);
      }
      pml[tid] = make_float2(M, L);
    }
#pragma unroll
    for (int half = 0; half < HD / 64; ++half) {
      if (half) asm volatile("bar.sync 1, 256;" ::: "memory");
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float* v = o[half * 8 + n];
        float* d = red + (warp * 16 + gq) * kRedPitch + n * 8 + cq * 2;
        *reinterpret_cast<float2*>(d) = make_float2(v[0] * f[0], v[1] * f[0]);
        *reinterpret_cast<float2*>(d + 8 * kRedPitch) = make_float2(v[2] * f[1], v[3] * f[1]);
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      for (int e = tid; e < rows * 16; e += kWarps * 32) {
        const int r = e / 16, col = e % 16 * 4;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = r / 16; w < kWarps; w += R) {
          const float4 x = *reinterpret_cast<const float4*>(red + (w * 16 + r % 16) * kRedPitch + col);
          sum.x += x.x; sum.y += x.y; sum.z += x.z; sum.w += x.w;
        }
        *reinterpret_cast<float4*>(po + (int64_t)r * HD + half * 64 + col) = sum;
      }
    }
    asm volatile("bar.sync 1, 256;" ::: "memory");  // sml and red are free for the next piece
  }
}

// Joins the pieces of every row: a warp a row, block (b) x row group.
template <int HD>
__global__ void __launch_bounds__(256) attend_join(const __grid_constant__ AttendParams p, int grid) {
  constexpr int V = HD / 32;
  const CacheView& c = p.c;
  const int b = blockIdx.x, head = blockIdx.y * 8 + threadIdx.x / 32, lane = threadIdx.x % 32;
  if (head >= c.nq) return;
  const int kvh = head / p.group, j = head % p.group;
  const int pre_tiles = p.sched[0], cum0 = p.sched[4 + b], own = p.sched[5 + b] - cum0;
  const int64_t tiles = *reinterpret_cast<const int64_t*>(p.sched + 2);
  const int G = active_blocks(tiles, grid);
  const int64_t shared_tiles = (int64_t)pre_tiles * p.row_tiles * c.nkv;

  float M = -INFINITY, L = 0.f, o[V] = {};
  auto take = [&](const float2* ml, const float* po) {
    const float2 x = *ml;
    if (x.y == 0.f) return;  // every position masked (a NaN sum is passed on)
    const float m = fmaxf(M, x.x), fa = M == -INFINITY ? 0.f : ex2(M - m), fb = ex2(x.x - m);
    L = L * fa + x.y * fb;
#pragma unroll
    for (int i = 0; i < V; ++i) o[i] = o[i] * fa + po[lane * V + i] * fb;
    M = m;
  };
  if (pre_tiles) {
    const int row = b * p.group + j, gidx = kvh * p.row_tiles + row / p.row_tile, r = row % p.row_tile;
    const int64_t u0 = (int64_t)gidx * pre_tiles;
    const int last = block_of(u0 + pre_tiles - 1, tiles, G);
    for (int i = block_of(u0, tiles, G); i <= last; ++i) {
      const int64_t at = (int64_t)(i + gidx) * p.row_tile + r;
      take(p.pre_ml + at, p.pre_o + at * HD);
    }
  }
  if (own) {
    const int gidx = b * c.nkv + kvh;
    const int64_t u0 = shared_tiles + (int64_t)cum0 * c.nkv + (int64_t)kvh * own;
    const int last = block_of(u0 + own - 1, tiles, G);
    for (int i = block_of(u0, tiles, G); i <= last; ++i) {
      const int64_t at = (int64_t)(i + gidx) * p.group + j;
      take(p.own_ml + at, p.own_o + at * HD);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;  // a row without positions: zeros
  const int64_t at = (int64_t)b * c.nq + head;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + at * HD + lane * V);
#pragma unroll
  for (int i = 0; i < V; i += 2) out[i / 2] = pack_bf16x2(o[i] * inv, o[i + 1] * inv);
  if (p.lse && lane == 0) p.lse[at] = M == -INFINITY ? -INFINITY : (M + log2f(L)) * 0.693147180559945309f;
}

// Workspace: schedule, then the pieces of the prefix and of the own positions.
struct Carve {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off += (bytes + 255) / 256 * 256;
    return o;
  }
};
struct Plan {
  int row_tile, row_tiles;
  size_t sched, pre_o, pre_ml, own_o, own_ml, total;
};

Plan plan(const mk_cache_desc& d, int n_sm) {
  Plan w;
  const int group = d.n_q_heads / d.n_kv_heads, rows = d.batch * group;
  w.row_tile = std::min((rows + 15) / 16 * 16, kMaxRows);
  w.row_tiles = (rows + w.row_tile - 1) / w.row_tile;
  // a piece more than its predecessor starts a block or a group: at most blocks + groups of them
  const size_t pre = ((size_t)n_sm + (size_t)d.n_kv_heads * w.row_tiles) * w.row_tile;
  const size_t own = ((size_t)n_sm + (size_t)d.n_kv_heads * d.batch) * group;
  Carve cv;
  w.sched = cv.take(sizeof(int) * (d.batch + 5));
  w.pre_o = cv.take(pre * d.head_dim * sizeof(float));
  w.pre_ml = cv.take(pre * sizeof(float2));
  w.own_o = cv.take(own * d.head_dim * sizeof(float));
  w.own_ml = cv.take(own * sizeof(float2));
  w.total = cv.off;
  return w;
}

template <int HD>
cudaError_t run(const AttendParams& p, const mk_cache& c, cudaStream_t stream) {
  attend_tiles<HD><<<c.n_sm, kAttThreads, Layout<HD>::kTotal, stream>>>(p, c.kmap, c.vmap);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  attend_join<HD><<<dim3(c.d.batch, (c.d.n_q_heads + 7) / 8), 256, 0, stream>>>(p, c.n_sm);
  return cudaGetLastError();
}

}  // namespace

size_t attend_workspace(const mk_cache_desc& d, int n_sm) { return plan(d, n_sm).total; }

cudaError_t attend_prepare() {
  static_assert(Layout<64>::kSlots <= 20 && Layout<128>::kSlots <= 20, "barriers of the ring");
  cudaError_t e = cudaFuncSetAttribute(attend_tiles<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<64>::kTotal);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attend_tiles<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<128>::kTotal);
}

cudaError_t attend(const mk_cache& c, int layer, const void* q, const int32_t* seq_lens, int prefix_len, float scale,
                   void* out, float* lse, void* workspace, cudaStream_t stream) {
  const Plan w = plan(c.d, c.n_sm);
  uint8_t* ws = (uint8_t*)workspace;
  AttendParams p;
  p.c = c.view;
  p.layer = layer;
  p.group = c.d.n_q_heads / c.d.n_kv_heads;
  p.box = c.box;
  p.prefix = prefix_len;
  p.base = c.view.bt ? prefix_len / c.box * c.box : prefix_len;
  p.row_tile = w.row_tile;
  p.row_tiles = w.row_tiles;
  p.scale = (scale == 0.f ? 1.f / sqrtf((float)c.d.head_dim) : scale) * 1.44269504088896341f;
  p.q = (const uint16_t*)q;
  p.seq_lens = seq_lens;
  p.out = (uint16_t*)out;
  p.lse = lse;
  p.sched = (int*)(ws + w.sched);
  p.pre_o = (float*)(ws + w.pre_o);
  p.pre_ml = (float2*)(ws + w.pre_ml);
  p.own_o = (float*)(ws + w.own_o);
  p.own_ml = (float2*)(ws + w.own_ml);
  return c.d.head_dim == 128 ? run<128>(p, c, stream) : run<64>(p, c, stream);
}

}  // namespace mk
