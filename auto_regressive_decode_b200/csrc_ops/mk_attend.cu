// Attention of one query token a sequence over a cache whose first positions
// all sequences share.
//
// Query heads that read the same cache rows are the rows of one product: for a
// KV head, the prefix serves batch x group rows at once (group = query heads
// per KV head), a sequence's own positions serve its group rows.  Both are cut
// into tiles of kTile positions; a "group" is the tiles of one set of rows
// (prefix: KV head; own: sequence x KV head).  The tiles of all
// groups, in order, are dealt to the blocks as equal contiguous runs (a group
// counts kHead tiles more: what starting and ending it costs); a block's run
// within a group is a piece, which keeps the running maximum m and sum l of
// every row (softmax in one pass) and its unnormalised output o, and leaves
// them in the workspace.  A second kernel joins the pieces of a row:
//   M = max m,  o = sum 2^(m - M) o / sum 2^(m - M) l,  lse = ln 2 (M + log2 sum 2^(m - M) l)
// with scores in units of log2 (scale * log2 e folded into one factor).
//
// Bound: memory, 4 head_dim bytes of cache a position and KV head against
// 4 head_dim flops a row, and for short sequences the latency of a piece's start
// and end.  A producer warp keeps a ring of TMA boxes in flight; two or three small
// blocks an SM, so that one streams while the others start or end a piece.
// Measured with the join, heads of 128: 32 sequences of 4000 to 4096 positions, 8 KV heads,
// 87 us, 6.1 TB/s; 8 sequences of 40 heads over 2048 shared and up to 2048 own positions
// 42 us, 5.2 TB/s; 512 sequences of 64 positions 42 us, 3.4 TB/s (starting and ending a
// piece takes 2600 of its 5000 clocks); one sequence over 1024 7.4 us, two launches' latency.
//
// Up to 8 rows (NARROW) are the N of the products, S^T = K Q^T and O^T = V^T P^T;
// more are their M, 16 at a time.  As M, 8 rows would take twice the products and
// registers, and two blocks an SM instead of three: 50 us for the 8 sequences above.
#include <algorithm>

#include "mk_attend.h"
#include "mk_ptx.h"

namespace mk {
namespace {

using namespace ptx;

constexpr int kTile = 64;                        // cache positions a tile
constexpr int kWarps = 4;                        // compute warps; the next one is the producer
constexpr int kComputeThreads = kWarps * 32;
constexpr int kAttThreads = kComputeThreads + 32;
constexpr int kHead = 2;                         // tiles that a group's start and end count as
// Rows of a KV head that share a prefix: more go to the tensor-core kernel, which does 128 in the time of one.
// 32 rows over 2500 positions (8 KV heads) take 16.5 us here and 18.4 there, 64 rows 21.0 and 20.3; over 16000 27.5 and
// 26.4, 39.9 and 28.3 (by rows alone; the length would move the limit a little).
constexpr int kTcFrom = 32;

template <int HD, bool NARROW>
struct Layout {
  static constexpr int kBlocksPerSm = NARROW ? 3 : 2;
  static constexpr int kSlotBytes = kTile * HD * 2;         // one tile of K or of V: [HD/64][kTile rows][128 B], swizzled
  static constexpr int kSlots = (NARROW ? 48 : 64) * 1024 / kSlotBytes;
  static constexpr int kCols = NARROW ? HD : 64;            // columns joined at a time
  static constexpr int kRedRows = NARROW ? 8 : 16;
  static constexpr int kRedPitch = kCols + 4;               // floats a row of the joining buffer
  static constexpr int kRed = kSlots * kSlotBytes;          // float[kWarps][kRedRows][kRedPitch]
  static constexpr int kQRows = NARROW ? 8 : 32;            // rows of a query buffer; there are two
  static constexpr int kQPitch = HD * 2 + 16;               // bytes a query row: ldmatrix rows in different banks
  static constexpr int kQ = kRed + kWarps * kRedRows * kRedPitch * 4;
  static constexpr int kMl = kQ + 2 * kQRows * kQPitch;     // float2[kWarps][16]
  static constexpr int kCtl = kMl + kWarps * 16 * 8;
  static constexpr int kLens = kCtl + 256;                  // int[batch], then int[batch + 1]: cost of the sequences before
  static constexpr int total(int batch) { return kLens + (2 * batch + 1) * 4 + 1024; }  // 1024: the ring is aligned by hand
  static_assert(NARROW || kTcFrom <= kQRows, "the rows over a prefix");
  static_assert(kLens + 2048 + 1024 <= 227 * 1024 / kBlocksPerSm - 1024, "blocks an SM");
};

struct Ctl {
  unsigned long long full[8], empty[8], qfull[2], qempty[2];
  int dead, max_len;
};
static_assert(sizeof(Ctl) <= 256, "control block");

__device__ __forceinline__ int own_tiles(const AttendParams& p, int len) {
  return len > p.prefix ? (len - p.base + kTile - 1) / kTile : 0;
}

__device__ __forceinline__ void compute_bar() { asm volatile("bar.sync 1, %0;" ::"n"(kComputeThreads) : "memory"); }

// A piece: tiles [i0, i1) of a group.
struct Piece {
  bool shared;
  int b, kvh;         // the sequence (shared: 0)
  int i0, i1, gidx;
  bool last;          // it ends its group
};

// The pieces of a block's run [u, end) of the groups' costs: found once, then
// group after group (a division is slow next to a short piece).
struct Walk {
  const AttendParams& p;
  const int* cum;
  int pre_tiles, u, end;
  bool shared;
  int g, kvh, b, n, r;  // the group: prefix group or sequence and KV head; its cost, the run's place in it
  __device__ Walk(const AttendParams& prm, const int* cumulative, int pre, int u0, int u1)
      : p(prm), cum(cumulative), pre_tiles(pre), u(u0), end(u1) {
    const int pre_cost = pre ? pre + kHead : 0, shared_cost = p.c.nkv * pre_cost;
    shared = u < shared_cost;
    if (shared) {
      g = u / pre_cost;
      r = u - g * pre_cost;
      n = pre_cost;
      kvh = g;
      b = 0;
    } else {
      const int v = u - shared_cost, w = v / p.c.nkv;
      int lo = 0, hi = p.c.B;  // the sequence with cum[b] <= w < cum[b + 1]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cum[mid] <= w) lo = mid; else hi = mid;
      }
      b = lo;
      n = max(cum[b + 1] - cum[b], 1);
      const int at = v - cum[b] * p.c.nkv;
      kvh = at / n;
      r = at - kvh * n;
      g = b * p.c.nkv + kvh;
    }
  }
  __device__ __forceinline__ bool next(Piece& a) {
    while (u < end) {
      if (r == n) {  // the next group
        r = 0;
        ++g;
        if (++kvh == p.c.nkv) {
          kvh = 0;
          if (shared) {
            shared = false;
            g = 0;
            n = cum[1];
          } else {
            ++b;
          }
        }
        while (!shared && (n = cum[b + 1] - cum[b]) == 0) {  // sequences without tiles; u < end: one follows
          ++b;
          g += p.c.nkv;
        }
      }
      const int take = min(n - r, end - u);
      a.shared = shared;
      a.gidx = g;
      a.kvh = kvh;
      a.b = b;
      a.i0 = max(r - kHead, 0);
      a.i1 = r + take - kHead;
      u += take;
      r += take;
      a.last = r == n;
      if (a.i1 > a.i0) return true;
    }
    return false;
  }
};

__device__ __forceinline__ int piece_rows(const AttendParams& p, const Piece& a) {
  return a.shared ? p.rows : p.group;
}

template <int HD, bool NARROW>
__global__ void __launch_bounds__(kAttThreads, Layout<HD, NARROW>::kBlocksPerSm)
    attend_tiles(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap kwhole,
                 const __grid_constant__ CUtensorMap vwhole) {
  using S = Layout<HD, NARROW>;
  constexpr int KS = HD / 16;  // k-steps of the score product
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const uint32_t ring = smem_addr(smem);
  float* red = reinterpret_cast<float*>(smem + S::kRed);
  float2* sml = reinterpret_cast<float2*>(smem + S::kMl);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + S::kCtl);
  int* lens = reinterpret_cast<int*>(smem + S::kLens);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const CacheView& c = p.c;
  int* cum = lens + c.B;
  volatile int* dead = &ctl->dead;

  if (tid == kAttThreads - 1) {
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 1);
      mbar_init(smem_addr(&ctl->empty[s]), kWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl->qfull[s]), 1);
      mbar_init(smem_addr(&ctl->qempty[s]), kWarps);
    }
    ctl->dead = 0;
    fence_mbar_init();
  }
  if (tid == kComputeThreads) {
    prefetch_map(&kwhole);
    prefetch_map(&vwhole);
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  // Nothing is read or written before the kernel ahead is done (after attend_prefix_tc: the one ahead of
  // that, whose own wait precedes this launch; their workspaces are apart.  The fence: no line of the first cache from before).
  if (p.tc) fence_gpu();
  else grid_wait();
  grid_launch_next();
  for (int b = tid; b < c.B; b += kAttThreads) {
    const int n = p.seq_lens[b], m = n < 0 ? 0 : min(n, c.T);
    if (n != m && blockIdx.x == 0) set_status(c.status, MK_ERR_RANGE, b);
    lens[b] = m;
  }
  __syncthreads();
  if (warp == 0) {  // the cost of the sequences before each, and the longest
    int sum = 0, longest = 0;
    for (int b0 = 0; b0 < c.B; b0 += 32) {
      const int b = b0 + lane, m = b < c.B ? lens[b] : 0, t = own_tiles(p, m), cost = t ? t + kHead : 0;
      longest = max(longest, m);
      int x = cost;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (b < c.B) cum[b + 1] = sum + x;
      sum += __shfl_sync(0xffffffffu, x, 31);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 0) {
      cum[0] = 0;
      ctl->max_len = longest;
    }
  }
  __syncthreads();
  // No sequence attends behind the longest: what lies there is not read.
  const int prefix_end = min(p.prefix, ctl->max_len);
  const int pre_tiles = p.tc ? 0 : (prefix_end + kTile - 1) / kTile;
  const int cost = (pre_tiles ? (pre_tiles + kHead) * c.nkv : 0) + cum[c.B] * c.nkv;
  if (blockIdx.x == 0) {
    for (int b = tid; b < c.B; b += kAttThreads) p.sched[1 + b] = cum[b + 1] - cum[b];
    if (tid == 0) p.sched[0] = prefix_end;
  }
  const int G = active_blocks(cost, gridDim.x), cta = blockIdx.x;
  if (cta >= G) {
    grid_wait();
    return;
  }
  Walk walk(p, cum, pre_tiles, first_unit(cost, cta, G), first_unit(cost, cta + 1, G));
  Piece a;

  if (warp == kWarps) {  // ---- producer: the pieces' query rows; K tile, V tile, K tile, ... into the ring
    uint32_t slot = 0, phase = 0, qbuf = 0, qphase = 0;
    const int boxes = kTile / p.box;               // boxes of one 64-column block of a tile that is no single box
    const int cb = lane / boxes, j = lane % boxes; // this lane's box
    const bool boxed = cb < HD / 64;
    int lo = 0, hi = 0, start = 0, i = 0;
    // Tiles in order; the place of the next one is looked up while this one's copies are under way.
    int i1 = 0;  // end of the open piece
    bool have = false, one_now = false, wanted_now = false;
    int row_now = 0;
    uint32_t bytes = 0;
    while (true) {
      bool more = true;
      if (i == i1) {  // the next piece: its tiles, its query rows
        more = walk.next(a);
        if (more) {
          i = a.i0;
          i1 = a.i1;
          start = a.shared ? 0 : p.base;
          lo = a.shared ? 0 : p.prefix;
          hi = a.shared ? prefix_end : lens[a.b];
          const int rows = piece_rows(p, a);
          const uint32_t full = smem_addr(&ctl->qfull[qbuf]), dst = ring + S::kQ + qbuf * S::kQRows * S::kQPitch;
          mbar_wait(smem_addr(&ctl->qempty[qbuf]), qphase ^ 1, dead);
          if (!__any_sync(0xffffffffu, *dead)) {
            if (lane == 0) mbar_expect_tx(full, rows * HD * 2);
            __syncwarp();
            for (int r = lane; r < rows; r += 32) {
              const int b = a.shared ? r / p.group : a.b, jh = a.shared ? r % p.group : r;
              bulk_load(dst + r * S::kQPitch, p.q + ((int64_t)b * c.nq + a.kvh * p.group + jh) * HD, HD * 2, full);
            }
          }
          if (p.wide || qbuf) qphase ^= 1;
          qbuf = p.wide ? 0 : qbuf ^ 1;
        }
      }
      bool one = false, wanted = false;
      int row = 0;
      if (more) {  // this lane's box of tile i
        const int t0 = start + i * kTile;
        one = p.whole && t0 >= lo && t0 + kTile <= hi;
        const int at = one ? t0 : t0 + j * p.box;
        wanted = one ? lane == 0 : boxed && at < hi && at + p.box > lo;
        bool ok = true;
        if (wanted) row = (int)(c.row(p.layer, a.b, at, &ok) + a.kvh * c.head_pitch());
        if (!ok) set_status(c.status, MK_ERR_RANGE, a.b);
        ++i;
      }
      for (int kv = 0; kv < 2 && have; ++kv) {  // the tile looked up before
        const uint32_t full = smem_addr(&ctl->full[slot]), dst = ring + slot * S::kSlotBytes;
        mbar_wait(smem_addr(&ctl->empty[slot]), phase ^ 1, dead);
        if (!__any_sync(0xffffffffu, *dead)) {
          if (lane == 0) mbar_expect_tx(full, bytes);
          __syncwarp();
          if (wanted_now) {
            if (one_now) tma_box3(dst, kv ? &vwhole : &kwhole, 0, row_now, 0, full);
            else tma_box2(dst + cb * (kTile * 128) + j * p.box * 128, kv ? &vmap : &kmap, cb * 64, row_now, full);
          }
        }
        __syncwarp();
        if (++slot == S::kSlots) slot = 0, phase ^= 1;
      }
      if (!more) break;
      have = true;
      one_now = one;
      wanted_now = wanted;
      row_now = row;
      bytes = one ? S::kSlotBytes : __popc(__ballot_sync(0xffffffffu, wanted)) * p.box * 128;
    }
    // a block that gave up waits for its own copies in flight before it ends
    if (__any_sync(0xffffffffu, *dead)) {
      const uint64_t t0 = globaltimer();
      for (int s = 0; s < S::kSlots + 2; ++s) {
        // the latest fill: the phase before the producer's next one
        const bool ring_slot = s < S::kSlots;
        const uint32_t full = smem_addr(ring_slot ? &ctl->full[s] : &ctl->qfull[s - S::kSlots]);
        const uint32_t last = ring_slot ? ((uint32_t)s < slot ? phase : phase ^ 1)
                                        : ((uint32_t)(s - S::kSlots) < qbuf ? qphase : qphase ^ 1);
        while (!mbar_try(full, last) && globaltimer() - t0 < 20000000ull) {
        }
      }
      if (lane == 0) set_status(c.status, MK_ERR_DEVICE_TIMEOUT, cta);
    }
    grid_wait();
    return;
  }

  // ---- compute warps
  uint32_t slot = 0, phase = 0, qbuf = 0, qphase = 0;
  const int gq = lane / 4, cq = lane % 4, mi = lane >> 3;
  while (walk.next(a)) {
    const int rows = piece_rows(p, a);
    const int lo = a.shared ? 0 : p.prefix, start = a.shared ? 0 : p.base;
    const int hi = a.shared ? prefix_end : lens[a.b];
    // row blocks of 16 (or the one of 8); a warp has row block rb and of every tile the 16-position slices sp * R + ...
    const int R = NARROW || rows <= 16 ? 1 : (rows <= 32 ? 2 : 4), rb = warp % R, sp = warp / R;
    // this lane's two rows: columns of S^T, or rows of S; their positions end at lim
    const int row0 = NARROW ? 2 * cq : rb * 16 + gq, row1 = NARROW ? 2 * cq + 1 : rb * 16 + gq + 8;
    int lim[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = h ? row1 : row0;
      lim[h] = r >= rows ? 0 : (a.shared ? min(lens[r / p.group], hi) : hi);
    }
    constexpr int kQRegs = NARROW ? 2 : 4;
    uint32_t qf[KS][kQRegs];
    mbar_wait(smem_addr(&ctl->qfull[qbuf]), qphase, dead);
    {
      const uint32_t buf = ring + S::kQ + qbuf * S::kQRows * S::kQPitch;
      if constexpr (NARROW) {  // B fragments: rows 0-7, 32 columns at a time
        const uint32_t at = buf + (lane & 7) * S::kQPitch + mi * 16;
#pragma unroll
        for (int k = 0; k < KS; k += 2) {
          uint32_t f[4];
          ldmatrix_x4(f, at + k * 32);
          qf[k][0] = f[0]; qf[k][1] = f[1]; qf[k + 1][0] = f[2]; qf[k + 1][1] = f[3];
        }
      } else {  // A fragments
        const uint32_t at = buf + (rb * 16 + (lane & 15)) * S::kQPitch + (lane >> 4) * 16;
#pragma unroll
        for (int k = 0; k < KS; ++k) ldmatrix_x4(qf[k], at + k * 32);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_addr(&ctl->qempty[qbuf]));
    if (p.wide || qbuf) qphase ^= 1;
    qbuf = p.wide ? 0 : qbuf ^ 1;

    // the output: HD columns of this lane's two rows (S::kTiles fragments of 4)
    constexpr int kTiles = NARROW ? HD / 16 : HD / 8;
    float o[kTiles][4];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
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
      for (int js = 0; js < R; ++js) {
        const int s0 = (sp * R + js) * 16, p0 = t0 + s0;
        if (p0 >= hi || p0 + 16 <= lo) continue;
        // scores, e = 0..3 of two 8-wide parts: value [part][e], its position and row
        constexpr int kParts = NARROW ? 1 : 2;
        float s[kParts][4], u[kParts][4];  // u: odd k-steps (shorter chains)
#pragma unroll
        for (int n = 0; n < kParts; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = u[n][e] = 0.f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int ch = k * 2 + (NARROW ? lane >> 4 : mi & 1), row = s0 + (NARROW ? lane & 15 : (mi >> 1) * 8 + (lane & 7));
          uint32_t f[4];
          ldmatrix_x4(f, kslot + (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
          if constexpr (NARROW) {
            mma16816(k & 1 ? u[0] : s[0], f, qf[k][0], qf[k][1]);
          } else {
            mma16816(k & 1 ? u[0] : s[0], qf[k], f[0], f[1]);
            mma16816(k & 1 ? u[1] : s[1], qf[k], f[2], f[3]);
          }
        }
        // mask, maximum of the lane's two rows
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < kParts; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int pos = NARROW ? p0 + gq + (e >> 1) * 8 : p0 + n * 8 + cq * 2 + (e & 1), h = NARROW ? e & 1 : e >> 1;
            s[n][e] = pos >= lo && pos < lim[h] ? (s[n][e] + u[n][e]) * p.scale : -INFINITY;
            mx[h] = fmaxf(mx[h], s[n][e]);
          }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int x = NARROW ? 4 : 1; x < (NARROW ? 32 : 4); x <<= 1) mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], x));
          mx[h] = fmaxf(mx[h], m[h]);
        }
        const bool grew = mx[0] > m[0] || mx[1] > m[1];
        float ref[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) ref[h] = mx[h] == -INFINITY ? 0.f : mx[h];
        if (__any_sync(0xffffffffu, grew)) {
          const float f[2] = {ex2(m[0] - ref[0]), ex2(m[1] - ref[1])};
          l[0] *= f[0];
          l[1] *= f[1];
#pragma unroll
          for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= f[NARROW ? e & 1 : e >> 1];
          m[0] = mx[0];
          m[1] = mx[1];
        }
#pragma unroll
        for (int n = 0; n < kParts; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = NARROW ? e & 1 : e >> 1;
            s[n][e] = ex2(s[n][e] - ref[h]);
            l[h] += s[n][e];
          }
        // probabilities as an operand of the second product: rounded to bf16, as the cache is
        uint32_t pf[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]), 0, 0};
        if constexpr (NARROW) {  // [position][row] to B's [row][position]
          pf[0] = movmatrix(pf[0]);
          pf[1] = movmatrix(pf[1]);
        } else {
          pf[2] = pack_bf16x2(s[1][0], s[1][1]);
          pf[3] = pack_bf16x2(s[1][2], s[1][3]);
        }
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
        const int row = s0 + (NARROW ? mi >> 1 : mi & 1) * 8 + (lane & 7);
#pragma unroll
        for (int n = 0; n < HD / 16; ++n) {  // 16 columns at a time
          const int ch = 2 * n + (NARROW ? mi & 1 : mi >> 1);
          uint32_t f[4];
          ldmatrix_x4_trans(f, vslot + (ch >> 3) * (kTile * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
          if constexpr (NARROW) {
            f[0] &= keep0;
            f[1] &= keep0;
            f[2] &= keep1;
            f[3] &= keep1;
            mma16816(o[n], f, pf[0], pf[1]);
          } else {
            mma16816(o[2 * n], pf, f[0] & keep0, f[1] & keep1);
            mma16816(o[2 * n + 1], pf, f[2] & keep0, f[3] & keep1);
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
#pragma unroll
      for (int x = NARROW ? 4 : 1; x < (NARROW ? 32 : 4); x <<= 1) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
      if ((NARROW ? gq : cq) == 0) sml[warp * 16 + (h ? row1 : row0) % 16] = make_float2(m[h], l[h]);
    }
    const int64_t pid = (int64_t)cta + a.gidx;
    float* po = (a.shared ? p.pre_o : p.own_o) + pid * rows * HD;
    float2* pml = (a.shared ? p.pre_ml : p.own_ml) + pid * rows;
    if (tid == 0) {
      int2* at = (a.shared ? p.pre_blocks : p.own_blocks) + a.gidx;
      if (a.i0 == 0) at->x = cta;
      if (a.last) at->y = cta;
    }
#pragma unroll
    for (int part = 0; part < HD / S::kCols; ++part) {
      if (part) compute_bar();
      if constexpr (NARROW) {
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          float* d = red + (warp * 8 + 2 * cq) * S::kRedPitch + n * 16 + gq;
          if (row0 < rows) d[0] = o[n][0], d[8] = o[n][2];
          if (row1 < rows) d[S::kRedPitch] = o[n][1], d[S::kRedPitch + 8] = o[n][3];
        }
      } else {
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const float* v = o[part * 8 + n];
          float* d = red + (warp * 16 + gq) * S::kRedPitch + n * 8 + cq * 2;
          if (row0 < rows) *reinterpret_cast<float2*>(d) = make_float2(v[0], v[1]);
          if (row1 < rows) *reinterpret_cast<float2*>(d + 8 * S::kRedPitch) = make_float2(v[2], v[3]);
        }
      }
      compute_bar();
      constexpr int kQuads = S::kCols / 4;
      for (int e = tid; e < rows * kQuads; e += kComputeThreads) {
        const int r = e / kQuads, col = e % kQuads * 4, w0 = NARROW ? 0 : r / 16;
        float M = -INFINITY, L = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        auto ml_of = [&](int w) { return sml[w * 16 + r % 16]; };
        auto add = [&](int w, float to) {
          const float2 ml = ml_of(w);
          const float4 x = *reinterpret_cast<const float4*>(red + (w * S::kRedRows + r % 16) * S::kRedPitch + col);
          if (ml.y == 0.f) return;  // every position masked (a NaN sum is passed on)
          const float f = ex2(ml.x - to);
          L += f * ml.y;
          sum.x += f * x.x; sum.y += f * x.y; sum.z += f * x.z; sum.w += f * x.w;
        };
        if constexpr (NARROW) {  // every warp has the row
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ml_of(w).x);
          const float to = M == -INFINITY ? 0.f : M;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) add(w, to);
        } else {
          for (int w = w0; w < kWarps; w += R) M = fmaxf(M, ml_of(w).x);
          const float to = M == -INFINITY ? 0.f : M;
          for (int w = w0; w < kWarps; w += R) add(w, to);
        }
        *reinterpret_cast<float4*>(po + (int64_t)r * HD + part * S::kCols + col) = sum;
        if (part == 0 && col == 0) pml[r] = make_float2(M, L);
      }
    }
    compute_bar();  // sml and red are free for the next piece
  }
  // launched while attend_prefix_tc runs, this grid ends after it: the join waits for this one alone
  grid_wait();
}

// Joins the pieces of every row: W warps a row take them in turn.  Bound: the latency of three
// loads that wait for each other (four, with the first outputs behind their weights: 0.5 us more); for thousands of rows the pieces' bytes (8192 rows, 24 MB: 8 us).
template <int HD, int W>
__global__ void __launch_bounds__(128) attend_join(const __grid_constant__ AttendParams p) {
  constexpr int V = HD / 32, kEarly = 4;
  __shared__ float so[4][HD];
  __shared__ float2 sml[4];
  const CacheView& c = p.c;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, sub = warp % W;
  const int64_t task = (int64_t)blockIdx.x * (4 / W) + warp / W;
  const int b = (int)(task / c.nq), head = (int)(task % c.nq);
  const int kvh = head / p.group, j = head % p.group;
  const int row = b * p.group + j, g1 = b * c.nkv + kvh;
  // the prefix's pieces are entries of some rows: one a piece, or of kTcRows rows, two a piece: for
  // two row tiles, or, with one row tile in the group, for its even and odd tiles
  const int entry = p.tc ? kTcRows : p.rows, per = p.tc ? 2 * kTcRows : entry;
  const int g0 = p.tc ? kvh * p.tc_groups + row / per : kvh;
  const bool both = p.tc && p.rows - row / per * per <= kTcRows;
  grid_wait();
  const bool have = b < c.B;
  // the row's pieces: blocks [x, y] of its prefix group and of its own
  int2 r0 = make_int2(0, -1), r1 = r0;
  if (have && p.prefix) r0 = p.pre_blocks[g0];
  if (have) r1 = p.own_blocks[g1];
  if (p.prefix && p.sched[0] == 0) r0 = make_int2(0, -1);  // no sequence reaches into the prefix: its groups have no pieces
  if (have && p.sched[1 + b] == 0) r1 = make_int2(0, -1);  // nor this sequence beyond it
  const int n0 = (r0.y - r0.x + 1) * (both ? 2 : 1), n = n0 + r1.y - r1.x + 1, step = both ? entry : per;
  const int first = p.tc ? tc_entry(p, p.tc_lanes > 1 ? row / per : 0, r0.x, p.tc_lanes > 1 ? kvh : g0) : r0.x + g0;
  const int64_t at0 = (int64_t)first * per + (both ? row % entry : row % per), at1 = (int64_t)(r1.x + g1) * p.group + j;

  // piece i of the row: its (m, l), and its output from this lane's columns on
  const float2* ml0 = p.pre_ml + at0;
  const float2* ml1 = p.own_ml + (at1 - (int64_t)n0 * p.group);
  const int r0c = row % kTcRows;
  const float* o0 = p.pre_o + (p.tc ? (at0 - r0c) * HD + TcOut<HD>::chunk(r0c, lane * V / 4) + lane * V % 4 : at0 * HD + lane * V);
  const float* o1 = p.own_o + (at1 - (int64_t)n0 * p.group) * HD + lane * V;
  float M = -INFINITY, L = 0.f, o[V] = {};
  for (int i0 = sub; i0 < n; i0 += 32 * W) {  // 32 pieces at a time: a lane's weight, then the weighted sum
    const int i = i0 + lane * W, k = min(32, (n - i0 + W - 1) / W);
    auto piece = [&](int q, float* v) {
      const int iq = i0 + q * W;
      const float* po = iq < n0 ? o0 + (int64_t)iq * (step * HD) : o1 + (int64_t)iq * (p.group * HD);
      if constexpr (V == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(po);
      else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(po);
    };
    float early[kEarly][V];  // the first outputs come while the weights do
#pragma unroll
    for (int q = 0; q < kEarly; ++q)
      if (q < k) piece(q, early[q]);
    float2 x = make_float2(-INFINITY, 0.f);
    if (i < n) x = i < n0 ? ml0[(int64_t)i * step] : ml1[(int64_t)i * p.group];
    float m = x.x;
#pragma unroll
    for (int s = 16; s; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    m = fmaxf(m, M);
    const float ref = m == -INFINITY ? 0.f : m, back = ex2(M - ref);
    const float w = x.y == 0.f ? 0.f : ex2(x.x - ref);  // a piece without positions has no part (a NaN sum is passed on)
    float l = w * x.y;
#pragma unroll
    for (int s = 16; s; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
    L = L * back + l;
    M = m;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] *= back;
    auto add = [&](int q, const float* v) {
      const float wq = __shfl_sync(0xffffffffu, w, q);
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = wq == 0.f ? o[e] : fmaf(v[e], wq, o[e]);
    };
#pragma unroll
    for (int q = 0; q < kEarly; ++q)
      if (q < k) add(q, early[q]);
#pragma unroll 4
    for (int q = kEarly; q < k; ++q) {
      float v[V];
      piece(q, v);
      add(q, v);
    }
  }
  if (W > 1) {  // the warps' parts
#pragma unroll
    for (int e = 0; e < V; ++e) so[warp][lane * V + e] = o[e];
    if (lane == 0) sml[warp] = make_float2(M, L);
    __syncthreads();
    if (sub) return;
    const float mine = M;
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, sml[warp + w].x);
    const float ref = M == -INFINITY ? 0.f : M, f = ex2(mine - ref);
    L *= f;
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] *= f;
#pragma unroll
    for (int w = 1; w < W; ++w) {
      const float2 x = sml[warp + w];
      const float g = x.y == 0.f ? 0.f : ex2(x.x - ref);
      L += g * x.y;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = g == 0.f ? o[e] : fmaf(so[warp + w][lane * V + e], g, o[e]);
    }
  }
  if (!have) return;
  const float inv = L == 0.f ? 0.f : 1.f / L;  // a row without positions: zeros
  const int64_t at = (int64_t)b * c.nq + head;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + at * HD + lane * V);
#pragma unroll
  for (int e = 0; e < V; e += 2) out[e / 2] = pack_bf16x2(o[e] * inv, o[e + 1] * inv);
  // by the sum: maxima drop NaN, so that M alone cannot tell a row of NaN scores from one without positions
  if (p.lse && lane == 0) p.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.693147180559945309f;
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
  int tc_groups;
  size_t sched, pre_blocks, own_blocks, pre_o, pre_ml, own_o, own_ml, total;
};

Plan plan(const mk_cache_desc& d, int n_sm) {
  Plan w;
  const int group = d.n_q_heads / d.n_kv_heads, rows = d.batch * group;
  // a piece more than its predecessor starts a block or a group: at most blocks + groups of them
  const size_t blocks = (size_t)n_sm * 3;
  w.tc_groups = (rows + 2 * kTcRows - 1) / (2 * kTcRows);
  const size_t pre = rows > kTcFrom ? ((size_t)n_sm + (size_t)d.n_kv_heads * w.tc_groups) * 2 * kTcRows
                                    : (blocks + (size_t)d.n_kv_heads) * rows;
  const size_t own = (blocks + (size_t)d.n_kv_heads * d.batch) * group;
  Carve cv;
  w.sched = cv.take(sizeof(int) * (d.batch + 1));
  w.pre_blocks = cv.take(sizeof(int2) * d.n_kv_heads * w.tc_groups);
  w.own_blocks = cv.take(sizeof(int2) * d.n_kv_heads * d.batch);
  w.pre_o = cv.take(pre * d.head_dim * sizeof(float));
  w.pre_ml = cv.take(pre * sizeof(float2));
  w.own_o = cv.take(own * d.head_dim * sizeof(float));
  w.own_ml = cv.take(own * sizeof(float2));
  w.total = cv.off;
  return w;
}

template <int HD, bool NARROW>
cudaError_t run(const AttendParams& p, const mk_cache& c, cudaStream_t stream) {
  using S = Layout<HD, NARROW>;
  const int smem = S::total(c.d.batch);
  const int grid = c.n_sm * std::min(S::kBlocksPerSm, 228 * 1024 / (smem + 1024));  // all of them resident
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.stream = stream;
  cudaError_t e;
  if (p.tc) {
    e = attend_prefix_tc(p, c, stream);
    if (e != cudaSuccess) return e;
  }
  // blocks of the next kernel are set up while this one's are still under way
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kAttThreads);
  cfg.dynamicSmemBytes = smem;
  e = cudaLaunchKernelEx(&cfg, attend_tiles<HD, NARROW>, p, c.kmap, c.vmap, c.kwhole, c.vwhole);
  if (e != cudaSuccess) return e;
  // Few rows: four warps each, since a row then has many pieces; else the SMs are busy with a warp a row.
  const int64_t rows = (int64_t)c.d.batch * c.d.n_q_heads;
  const bool few = rows <= 8 * c.n_sm;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(few ? rows : (rows + 3) / 4));
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return few ? cudaLaunchKernelEx(&cfg, attend_join<HD, 4>, p) : cudaLaunchKernelEx(&cfg, attend_join<HD, 1>, p);
}

}  // namespace

size_t attend_workspace(const mk_cache_desc& d, int n_sm) { return plan(d, n_sm).total; }

template <int HD, bool NARROW>
cudaError_t allow_smem() {
  static_assert(Layout<HD, NARROW>::kSlots <= 8, "barriers of the ring");
  return cudaFuncSetAttribute(attend_tiles<HD, NARROW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Layout<HD, NARROW>::total(kCacheMaxBatch));
}

cudaError_t attend_prepare() {
  cudaError_t e = attend_prefix_tc_prepare();
  if (e == cudaSuccess) e = allow_smem<64, false>();
  if (e == cudaSuccess) e = allow_smem<64, true>();
  if (e == cudaSuccess) e = allow_smem<128, false>();
  if (e == cudaSuccess) e = allow_smem<128, true>();
  return e;
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
  p.whole = !c.view.bt || c.view.page % kTile == 0;
  p.prefix = prefix_len;
  p.base = !c.view.bt ? prefix_len : prefix_len / (p.whole ? kTile : c.box) * (p.whole ? kTile : c.box);
  p.rows = c.d.batch * p.group;
  p.tc = prefix_len > 0 && p.rows > kTcFrom;
  p.tc_groups = w.tc_groups;
  p.tc_lanes = c.n_sm % w.tc_groups * 16 <= c.n_sm ? w.tc_groups : 1;  // where at most 1 SM of 16 is left without work
  p.tc_blocks = c.n_sm / p.tc_lanes;
  p.wide = p.group > 32;
  p.scale = (scale == 0.f ? 1.f / sqrtf((float)c.d.head_dim) : scale) * kLog2e;
  p.q = (const uint16_t*)q;
  p.seq_lens = seq_lens;
  p.out = (uint16_t*)out;
  p.lse = lse;
  p.sched = (int*)(ws + w.sched);
  p.pre_blocks = (int2*)(ws + w.pre_blocks);
  p.own_blocks = (int2*)(ws + w.own_blocks);
  p.pre_o = (float*)(ws + w.pre_o);
  p.pre_ml = (float2*)(ws + w.pre_ml);
  p.own_o = (float*)(ws + w.own_o);
  p.own_ml = (float2*)(ws + w.own_ml);
  const bool narrow = std::max(p.group, prefix_len && !p.tc ? p.rows : 0) <= 8;
  if (c.d.head_dim == 128) return narrow ? run<128, true>(p, c, stream) : run<128, false>(p, c, stream);
  return narrow ? run<64, true>(p, c, stream) : run<64, false>(p, c, stream);
}

}  // namespace mk
