// Attention over a shared prefix on the tensor cores (tcgen05), for many rows.
//
// For a KV head, the batch's queries are the rows of S = Q K^T and O += P V
// (M = 128 rows, tiles of 128 positions).  A block holds two streams, each with
// its scores S and its output O in tensor memory and a warpgroup for its
// softmax, a thread a row; while the matrix unit works for one stream, the
// other's warpgroup computes.  More than 128 rows: the streams are two row tiles that read
// the same K and V tiles.  Fewer: they are the even and the odd tiles of the same rows.
//
//   warps 0-7, 8-15 softmax of stream 0, 1, two threads a row (half the columns
//                   each): S from tensor memory, maximum and sum of the row, P =
//                   2^(s - m) as bf16 over S's columns
//   warps 16, 18    one thread each issues the products of stream 0, 1, in turns
//   warp 17         TMA of K and V tiles into a ring
//   warp 19         nothing: it fills the warpgroup that gives its registers to the softmax
//
// A row's reference m is raised, and its output scaled, only when a score
// exceeds it by kSlack (log2): p stays below 2^kSlack, far inside fp32 and
// bf16, and after the first tiles the output is hardly ever touched.
//
// The tiles of all groups (KV head x 256 rows) are dealt to the blocks as equal
// contiguous runs; a piece leaves m, l and o of its rows for the join (mk_attend.cu).
// Where the row groups of a KV head divide the SMs almost evenly, each has its own
// blocks (a lane), so that all row groups pass over the same tiles at the same time
// and a tile is read from memory once (65536 positions of 8 KV heads, 268 MB, for
// 1024 rows each: 274 us to 242).
//
// Bound: the tensor cores (4 head_dim flops a row and position) and, nearly as
// much, the exponentials (16 a clock and SM: 128 x 128 of them last as long as the
// tile's two products); with up to about 128 rows, the cache's bytes.  1024 rows of 8
// KV heads over 65536 positions: 235 to 255 us with the join (by the machine), 1080 to 1170 TFLOP/s; 128 rows: 62 us,
// 4.3 TB/s.  A stream's products and softmax alternate, about 1300 and 2000 clocks a
// tile of 128 x 128; for heads of 128 a third stream has no room in tensor memory.
#include <type_traits>

#include "mk_attend.h"
#include "mk_ptx.h"

namespace mk {
namespace {

using namespace ptx;

constexpr int kSoftmaxThreads = 512;  // two a row of each stream
constexpr int kTcThreads = kSoftmaxThreads + 128;
// Registers a thread: the compiler's share of the launch (96 at 640 threads), then split.
constexpr int kRegsFew = 64, kRegsMany = 104;
static_assert(kRegsFew * 128 + kRegsMany * kSoftmaxThreads <= 96 * kTcThreads, "the launch's registers");
constexpr int kHalf = kTcTile / 2;  // positions of a thread's half row
constexpr float kSlack = 8.f;
// References above it: a reference is a rounded product, and the exponent's fused product less the reference is then off
// by more than 2^-4, without bound; product and difference are rounded one after the other instead.
constexpr float kFar = 1 << 20;
constexpr int kTcHead = 1;  // tiles that a group's start and end count as

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int HD>
struct TcLayout {
  static constexpr int kSlotBytes = kTcTile * HD * 2;       // K or V tile: [HD/64][128 rows][128 B], swizzled
  static constexpr int kSlots = 128 * 1024 / kSlotBytes;
  static constexpr int kQ = kSlots * kSlotBytes;            // two query tiles, laid out the same
  static constexpr int kQBytes = kTcRows * HD * 2;
  static constexpr int kSwap = kQ + 2 * kQBytes;             // float[stream][turn][half][128]
  static constexpr int kCtl = kSwap + 2 * 2 * 2 * 128 * 4;
  static constexpr int kTotal = kCtl + 512 + 1024;          // 1024: aligned by hand
};

struct TcCtl {
  // tail[slot]: what lies behind the prefix in the slot's V tile is cleared.  One a slot, so that its phase cannot
  // run ahead of those who wait for it: the slot is filled again only after its tile has been read.
  unsigned long long full[8], empty[8], tail[8];
  unsigned long long q_full, s_full[2], p_half[2], p_full[2], o_done[2];  // [stream]
  uint32_t tmem;
  int dead, max_len;
};
static_assert(sizeof(TcCtl) <= 512, "control block");

// One block's run within a group.
struct Piece {
  int kvh, row0, rows, n, t0;  // rows of the group from row0 on, tiles t0 ... t0 + n
  int k, gidx;                 // the group in its lane, among all
  bool first, last, pair;
};

struct Walk {
  int tiles, groups, total_rows, lane;  // lane -1: there is one
  int u, end;
  __device__ __forceinline__ bool next(Piece& a) {
    while (u < end) {
      const int n = tiles + kTcHead;
      a.k = u / n;
      const int r = u - a.k * n, take = min(n - r, end - u);
      u += take;
      a.kvh = lane < 0 ? a.k / groups : a.k;
      const int row_group = lane < 0 ? a.k - a.kvh * groups : lane;
      a.gidx = a.kvh * groups + row_group;
      a.row0 = row_group * 2 * kTcRows;
      a.rows = min(2 * kTcRows, total_rows - a.row0);
      a.pair = a.rows > kTcRows;
      a.t0 = max(r - kTcHead, 0);
      a.n = r + take - kTcHead - a.t0;
      a.first = a.t0 == 0;
      a.last = r + take == n;
      if (a.n > 0) return true;
    }
    return false;
  }
};

// The order in which a piece's 2 n tiles of K and V pass through the ring: as
// the products want them.  Pair: K0 V0 K1 V1 ...; else K0 K1 V0 K2 V1 K3 V2 ...
__device__ __forceinline__ int k_place(bool pair, int t) { return pair ? 2 * t : (t ? 2 * t - 1 : 0); }
__device__ __forceinline__ int v_place(bool pair, int t, int n) { return pair ? 2 * t + 1 : min(2 * t + 2, 2 * n - 1); }

template <int HD>
__global__ void __launch_bounds__(kTcThreads, 1)
    attend_prefix_kernel(const __grid_constant__ AttendParams p, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, int tall) {
  using S = TcLayout<HD>;
  constexpr int CB = HD / 64;  // 64-column blocks of a row
  constexpr uint32_t kS = 0, kO = 256;  // columns of tensor memory: S0 S1 (P over them), O0 O1
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const uint32_t base = smem_addr(smem);
  TcCtl* ctl = reinterpret_cast<TcCtl*>(smem + S::kCtl);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const CacheView& cv = p.c;
  volatile int* dead = &ctl->dead;

  if (tid == 0) {
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 1);
      mbar_init(smem_addr(&ctl->empty[s]), 2);
      mbar_init(smem_addr(&ctl->tail[s]), 1);
    }
    mbar_init(smem_addr(&ctl->q_full), kSoftmaxThreads);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl->s_full[s]), 1);
      mbar_init(smem_addr(&ctl->p_half[s]), kSoftmaxThreads / 2);
      mbar_init(smem_addr(&ctl->p_full[s]), kSoftmaxThreads / 2);
      mbar_init(smem_addr(&ctl->o_done[s]), 1);
    }
    ctl->dead = 0;
    ctl->max_len = 0;
    fence_mbar_init();
  }
  if (warp == 16) tmem_alloc(smem_addr(&ctl->tmem), 512);
  if (tid == 0) {
    prefetch_map(&kmap);
    prefetch_map(&vmap);
  }
  __syncthreads();
  grid_wait();  // nothing is read or written before the kernel ahead is done
  grid_launch_next();
  int longest = 0;
  for (int b = tid; b < cv.B; b += kTcThreads) longest = max(longest, min(p.seq_lens[b], cv.T));
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) atomicMax(&ctl->max_len, longest);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  // No sequence attends behind the longest: what lies there is not read.
  const int prefix_end = min(p.prefix, ctl->max_len);
  const int tiles = (prefix_end + kTcTile - 1) / kTcTile;
  const int cost = tiles ? (tiles + kTcHead) * (p.tc_groups / p.tc_lanes) * cv.nkv : 0;
  const int G = active_blocks(cost, p.tc_blocks), cta = blockIdx.x / p.tc_lanes, row_lane = blockIdx.x % p.tc_lanes;
  Walk walk{tiles, p.tc_groups, p.rows, p.tc_lanes > 1 ? row_lane : -1, 0, 0};
  if (cta < G) walk.u = first_unit(cost, cta, G), walk.end = first_unit(cost, cta + 1, G);
  Piece a;

  const int whole_tiles = prefix_end / kTcTile;
  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsFew));
    if (warp == 17) {  // ---- TMA: K and V tiles in the order of k_place, v_place
    uint32_t slot = 0, phase = 0;
    const int boxes = kTcTile / tall, cb = lane / boxes, j = lane % boxes;  // this lane's box of a tile
    while (walk.next(a)) {
      for (int i = 0; i < 2 * a.n; ++i) {
        bool is_k;
        int t;
        if (a.pair) {
          is_k = !(i & 1);
          t = i >> 1;
        } else {
          is_k = i == 0 || ((i & 1) && (i + 1) / 2 < a.n);
          t = is_k ? (i + 1) / 2 : (i == 2 * a.n - 1 ? a.n - 1 : (i - 2) / 2);
        }
        const int at = (a.t0 + t) * kTcTile + j * tall;
        const bool wanted = cb < CB && at < prefix_end;
        bool ok = true;
        int row = 0;
        if (wanted) row = (int)(cv.row(p.layer, 0, at, &ok) + a.kvh * cv.head_pitch());
        if (!ok) set_status(cv.status, MK_ERR_RANGE, 0);
        const uint32_t full = smem_addr(&ctl->full[slot]);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, wanted)) * tall * 128;
        mbar_wait(smem_addr(&ctl->empty[slot]), phase ^ 1, dead);
        if (!__any_sync(0xffffffffu, *dead)) {
          if (lane == 0) mbar_expect_tx(full, bytes);
          __syncwarp();
          if (wanted)
            tma_box2(base + slot * S::kSlotBytes + cb * (kTcTile * 128) + j * tall * 128, is_k ? &kmap : &vmap, cb * 64, row, full);
        }
        __syncwarp();
        if (!is_k && a.t0 + t == whole_tiles) {
          // the prefix ends in this tile: what lies behind is anything, and 0 x NaN is NaN
          const int have = prefix_end - whole_tiles * kTcTile;
          const uint32_t v = base + slot * S::kSlotBytes;
          mbar_wait(full, phase, dead);
          for (int e = lane; e < (kTcTile - have) * 8 * CB; e += 32) {
            const int chunk = e % 8, block = e / 8 % CB, r = have + e / (8 * CB);
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + block * (kTcTile * 128) + r * 128 + chunk * 16), "r"(0) : "memory");
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&ctl->tail[slot]));
        }
        if (++slot == S::kSlots) slot = 0, phase ^= 1;
      }
    }
    if (__any_sync(0xffffffffu, *dead)) {  // copies still in flight land before the block ends
      const uint64_t t0 = globaltimer();
      for (int s = 0; s < S::kSlots; ++s)
        while (!mbar_try(smem_addr(&ctl->full[s]), (uint32_t)s < slot ? phase : phase ^ 1) && globaltimer() - t0 < 20000000ull) {
        }
      if (lane == 0) set_status(cv.status, MK_ERR_DEVICE_TIMEOUT, cta);
    }
  } else if (warp == 16 || warp == 18) {  // ---- products of stream s
    const int s = (warp - 16) / 2;
    constexpr uint32_t kQk = mma_desc(kTcRows, kTcTile, false), kPv = mma_desc(kTcRows, HD, true);
    const uint32_t leader = lane == 0;
    const uint64_t q_desc = smem_desc(base + S::kQ, 16, 1024), k_desc = smem_desc(base, 16, 1024),
                   v_desc = smem_desc(base, kTcTile * 128, 1024);
    uint32_t at = 0;  // tiles that passed through the ring in earlier pieces
    uint32_t q_phase = 0, tail_phase = 0 /* a bit a slot */, p_phase = 0;
    const uint32_t s_full = smem_addr(&ctl->s_full[s]), p_half = smem_addr(&ctl->p_half[s]), p_full = smem_addr(&ctl->p_full[s]), o_done = smem_addr(&ctl->o_done[s]);
    const uint32_t s_col = tmem + kS + s * 128, o_col = tmem + kO + s * 128;
    // The streams' warps take turns.  A product is issued as the matrix unit takes it (65 to
    // 71 clocks each, a commit 40 to 75), so that whatever stands between two runs of them is
    // time lost: one warp waits for its operands while the other issues.
    auto take_turn = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(9 + s) : "memory"); };
    auto pass_turn = [&]() { asm volatile("bar.arrive %0, 64;" ::"r"(10 - s) : "memory"); };
    if (s == 1) pass_turn();
    while (walk.next(a)) {
      const int turns = a.pair ? a.n : (a.n + 1) / 2, n = a.pair ? a.n : (a.n + 1 - s) / 2;
      const uint64_t q = q_desc + (a.pair ? s : 0) * (S::kQBytes >> 4);
      mbar_wait(smem_addr(&ctl->q_full), q_phase, dead);
      q_phase ^= 1;
      auto k_tile = [&](int i) {  // the descriptor of the stream's K tile i, once it is there
        const uint32_t place = at + k_place(a.pair, a.pair ? i : 2 * i + s), slot = place % S::kSlots;
        mbar_wait(smem_addr(&ctl->full[slot]), place / S::kSlots & 1, dead);
        return k_desc + slot * (S::kSlotBytes >> 4);
      };
      auto qk = [&](uint64_t k) {  // scores
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {  // 16 columns are 32 bytes of a swizzled line; 4 k-steps a 64-column block
          constexpr uint32_t kBlock = kTcRows * 128 >> 4;
          const uint32_t off = ks / 4 * kBlock + ks % 4 * 2;
          tc_mma_ss(s_col, q + off, k + off, kQk, ks > 0, leader);
        }
        // tells the softmax that the scores are there, that the product before is done (in order of
        // issue) and, through the softmax, the ring that both tiles have been read
        tc_commit(s_full, leader);
      };
      uint64_t k = n ? k_tile(0) : 0;
      take_turn();
      if (n) qk(k);
      pass_turn();
      for (int i = 0; i < turns; ++i) {
        uint64_t v = 0;
        if (i < n) {
          const int t = a.pair ? i : 2 * i + s;
          const uint32_t place = at + v_place(a.pair, t, a.n), slot = place % S::kSlots;
          mbar_wait(smem_addr(&ctl->full[slot]), place / S::kSlots & 1, dead);
          if (a.t0 + t == whole_tiles) mbar_wait(smem_addr(&ctl->tail[slot]), tail_phase >> slot & 1, dead);
          v = v_desc + slot * (S::kSlotBytes >> 4);
          if (i + 1 < n) k = k_tile(i + 1);
          mbar_wait(p_half, p_phase, dead);
        }
        take_turn();
        tc_fence_after();
        if (i < n) {
          // k-steps of 16 positions, 16 lines on.  The probabilities come in two parts, the first 32
          // positions of each half and the rest, so that half of the product runs under the
          // other half's exponentials (242 us to 235 for 65536 positions, 1024 rows of 8 KV heads).
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            if (q) {
              mbar_wait(p_full, p_phase, dead);
              tc_fence_after();
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int ks = q * 2 + e / 2 * 4 + e % 2;
              tc_mma_ts(o_col, s_col + ks * 8, v + ks * (16 * 128 >> 4), kPv, q + e > 0 || i > 0, leader);
            }
          }
          p_phase ^= 1;
          // The next scores overwrite the probabilities: after the product that reads them, in order of issue.
          if (i + 1 < n) qk(k);
          else tc_commit(o_done, leader);
        }
        pass_turn();
      }
      if (a.t0 + a.n > whole_tiles) tail_phase ^= 1u << (at + 2 * a.n - 1) % S::kSlots;  // the piece's last tile was the cleared one
      at += 2 * a.n;
    }
    if (s == 0) take_turn();  // the last one passed
  }
  } else {  // ---- softmax of stream s
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMany));
    const int s = warp / 8, c = warp / 4 % 2, r = tid % 128;  // half c of row r of the stream's tile
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    const uint32_t s_at = tmem + lanes + kS + s * 128, o_at = tmem + lanes + kO + s * 128 + c * (HD / 2);
    const float scale = fabsf(p.scale);
    const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;  // a negative scale goes into the query's signs
    float* swap = reinterpret_cast<float*>(smem + S::kSwap) + s * 512;  // [turn][half][row]
    auto stream_bar = [&]() { asm volatile("bar.sync %0, 256;" ::"r"(11 + s) : "memory"); };
    auto pair_bar = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + s * 4 + warp % 4) : "memory"); };
    uint32_t q_phase = 0, s_phase = 0, o_phase = 0, other_phase = 0, at = 0, turn = 0;
    // The other half's value for this row.
    auto other = [&](float mine) {
      float* w = swap + turn * 256;
      turn ^= 1;
      w[c * 128 + r] = mine;
      pair_bar();
      return w[(c ^ 1) * 128 + r];
    };
    while (walk.next(a)) {
      const int n = a.pair ? a.n : (a.n + 1 - s) / 2;
      const int row = (a.pair ? s * kTcRows : 0) + r;
      const bool valid = row < a.rows;
      const int b = (a.row0 + row) / p.group;
      const int lim = valid ? min(p.seq_lens[b], prefix_end) : 0;
      if (a.pair || s == 0) {  // the query tile, a thread a 16-byte chunk of every kStep-th row, swizzled as TMA would
        constexpr int kChunks = HD / 8, kStep = 256 / kChunks;
        const int ch = tid % kChunks, first = tid % 256 / kChunks, row0 = a.pair ? s * kTcRows : 0;
        const int step_b = kStep / p.group, step_j = kStep % p.group;
        int qb = (a.row0 + row0 + first) / p.group, qj = (a.row0 + row0 + first) % p.group;
        uint4 x[kTcRows / kStep];
#pragma unroll
        for (int i = 0; i < kTcRows / kStep; ++i) {
          x[i] = make_uint4(0, 0, 0, 0);
          if (row0 + first + i * kStep < a.rows)
            x[i] = reinterpret_cast<const uint4*>(p.q + ((int64_t)qb * cv.nq + a.kvh * p.group + qj) * HD)[ch];
          qb += step_b;
          qj += step_j;
          if (qj >= p.group) qj -= p.group, ++qb;
        }
        uint8_t* to = smem + S::kQ + (a.pair ? s : 0) * S::kQBytes + ch / 8 * (kTcRows * 128);
#pragma unroll
        for (int i = 0; i < kTcRows / kStep; ++i) {
          const int to_row = first + i * kStep;
          x[i].x ^= flip; x[i].y ^= flip; x[i].z ^= flip; x[i].w ^= flip;
          *reinterpret_cast<uint4*>(to + to_row * 128 + (((ch % 8) ^ (to_row & 7)) << 4)) = x[i];
        }
        fence_async_shared();
      }
      tc_fence_before();
      mbar_arrive(smem_addr(&ctl->q_full));
      // a stream without tiles waits for nothing else: it must not arrive for the next piece before the other has for this
      if (n == 0) mbar_wait(smem_addr(&ctl->q_full), q_phase, dead);
      q_phase ^= 1;

      float m = -INFINITY, l = 0.f;
      bool far = false;  // of a row of the warp
      for (int i = 0; i < n; ++i) {
        const int t = a.pair ? i : 2 * i + s, t0 = (a.t0 + t) * kTcTile + c * kHalf;
        mbar_wait(smem_addr(&ctl->s_full[s]), s_phase, dead);
        s_phase ^= 1;
        tc_fence_after();
        if (r == 0 && c == 0) {  // the scores' K tile has been read, and the V tile of the product before
          const uint32_t uses = a.pair ? 1 : 2;
          mbar_arrive(smem_addr(&ctl->empty[(at + k_place(a.pair, t)) % S::kSlots]), uses);
          if (i) mbar_arrive(smem_addr(&ctl->empty[(at + v_place(a.pair, a.pair ? t - 1 : t - 2, a.n)) % S::kSlots]), uses);
        }
        uint32_t x[kHalf];
        tmem_ld32(s_at + c * kHalf, x);
        tmem_ld32(s_at + c * kHalf + 32, x + 32);
        tmem_wait_ld();
        if (__any_sync(0xffffffffu, t0 + kHalf > lim)) {
#pragma unroll
          for (int e = 0; e < kHalf; ++e)
            if (t0 + e >= lim) x[e] = 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < kHalf; e += 8) {
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = max3_nan(mx[q], __uint_as_float(x[e + q]), __uint_as_float(x[e + q + 4]));
        }
        float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * scale;
        const float twin = other(top);  // also: both halves have read their scores before probabilities cover them
        top = max3_nan(top, twin, twin);
        if (top == INFINITY) top = NAN;  // a NaN or an infinite score leaves nothing but NaN of the row
        const bool raise = !(top <= m + kSlack);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2(m - top) : 1.f;
          if (raise) m = top;
          far = __any_sync(0xffffffffu, m != -INFINITY && fabsf(m) > kFar);
          l *= f;
          if (i > 0) {  // half of the stream's output so far: its last product was done before these scores
#pragma unroll 1
            for (int q = 0; q < HD / 32; ++q) {
              uint32_t y[16];
              tmem_ld16(o_at + q * 16, y);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
              tmem_st16(o_at + q * 16, y);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float by = scale, back = -ref;
        if (far) {
#pragma unroll
          for (int e = 0; e < kHalf; ++e) x[e] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(x[e]), scale), ref));
          by = 1.f;
          back = 0.f;
        }
        const F2 scale2 = pack2(by, by), back2 = pack2(back, back);
        F2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const F2 d = fma2(pack2(__uint_as_float(x[q * 32 + 2 * e]), __uint_as_float(x[q * 32 + 2 * e + 1])), scale2, back2);
            float d0, d1;
            unpack2(d, d0, d1);
            const float p0 = ex2(d0), p1 = ex2(d1);
            sum[e & 1] = add2(sum[e & 1], pack2(p0, p1));
            y[e] = pack_bf16x2(p0, p1);  // the operand of the second product, as the cache is
          }
          tmem_st16(s_at + c * (kHalf / 2) + q * 16, y);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(smem_addr(q ? &ctl->p_full[s] : &ctl->p_half[s]));
        }
        float u0, u1;
        unpack2(add2(sum[0], sum[1]), u0, u1);
        l += u0 + u1;
      }
      // leave the piece
      const int64_t entry = (int64_t)tc_entry(p, row_lane, cta, a.k) * 2 + s;
      if (tid == 0) {
        if (a.first) p.pre_blocks[a.gidx].x = cta;
        if (a.last) p.pre_blocks[a.gidx].y = cta;
      }
      l += other(l);
      if (valid && c == 0) p.pre_ml[entry * kTcRows + r] = make_float2(m, l);
      if (n) {
        mbar_wait(smem_addr(&ctl->o_done[s]), o_phase, dead);
        o_phase ^= 1;
        tc_fence_after();
        if (r == 0 && c == 0)
          mbar_arrive(smem_addr(&ctl->empty[(at + v_place(a.pair, a.pair ? n - 1 : 2 * n - 2 + s, a.n)) % S::kSlots]), a.pair ? 1 : 2);
        // The outputs leave through the query tile's memory, half of them at a time, as copies
        // of whole blocks (from each thread's row directly, 32 lanes' 16 bytes went to 32 lines: a clock
        // a lane, 7000 a piece).  The tile is free once the stream's products are done (with one row
        // tile, once the other stream's are too).
        if (s == 0 && !a.pair && a.n > 1) mbar_wait(smem_addr(&ctl->o_done[1]), other_phase, dead);
        using Out = TcOut<HD>;
        constexpr uint32_t kBytes = Out::kFloats * 4;
        static_assert(2 * kBytes <= S::kQBytes, "two parts at a time");
        float* out = p.pre_o + entry * kTcRows * HD;
#pragma unroll 1
        for (int part = 0; part < kTcParts; ++part) {
          uint32_t y[4 * Out::kMine];
          if constexpr (HD == 128) tmem_ld16(o_at + part * 16, y);
          else tmem_ld8(o_at + part * 8, y);
          tmem_wait_ld();
          const uint32_t at_part = S::kQ + s * S::kQBytes + part % 2 * kBytes;
          if (part >= 2) {  // this memory's part before has been read
            if (tid % 256 == 0) bulk_stores_read<1>();
            stream_bar();
          }
          float4* stage = reinterpret_cast<float4*>(smem + at_part) + r * Out::kRow;
#pragma unroll
          for (int e = 0; e < Out::kMine; ++e)
            stage[Out::swizzle(r, c * Out::kMine + e)] =
                make_float4(__uint_as_float(y[4 * e]), __uint_as_float(y[4 * e + 1]), __uint_as_float(y[4 * e + 2]), __uint_as_float(y[4 * e + 3]));
          fence_async_shared();
          stream_bar();
          if (tid % 256 == 0) bulk_store(out + part * Out::kFloats, base + at_part, kBytes);
        }
        if (tid % 256 == 0) bulk_stores_read<0>();
        stream_bar();  // the memory is free for the next piece's queries
      }
      if (a.pair || a.n > 1) other_phase ^= 1;  // stream 1 had products in this piece
      at += 2 * a.n;
    }
    if (tid % 256 == 0) bulk_stores_done();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

}  // namespace

cudaError_t attend_prefix_tc_prepare() {
  cudaError_t e = cudaFuncSetAttribute(attend_prefix_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcLayout<64>::kTotal);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(attend_prefix_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, TcLayout<128>::kTotal);
}

cudaError_t attend_prefix_tc(const AttendParams& p, const mk_cache& c, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // set up while the kernel ahead is under way
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(c.n_sm);
  cfg.blockDim = dim3(kTcThreads);
  cfg.stream = stream;
  if (c.d.head_dim == 128) {
    cfg.dynamicSmemBytes = TcLayout<128>::kTotal;
    return cudaLaunchKernelEx(&cfg, attend_prefix_kernel<128>, p, c.ktall, c.vtall, c.tall);
  }
  cfg.dynamicSmemBytes = TcLayout<64>::kTotal;
  return cudaLaunchKernelEx(&cfg, attend_prefix_kernel<64>, p, c.ktall, c.vtall, c.tall);
}

}  // namespace mk
