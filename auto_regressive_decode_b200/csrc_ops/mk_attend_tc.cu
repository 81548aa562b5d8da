// Attention over a shared prefix on the tensor cores (tcgen05), for many rows.
//
// For a KV head, the batch's queries are the rows of S = Q K^T and O += P V
// (M = 128 rows, tiles of 128 positions).  A block holds two streams, each with
// its scores S and its output O in tensor memory and a warpgroup for its
// softmax, a thread a row; while the matrix unit works for one stream, the
// other's warpgroup computes.  More than 128 rows: the streams are two row tiles that read
// the same K and V tiles.  Fewer: they are the even and the odd tiles of the same rows.
//
//   warps 0-3, 4-7  softmax of stream 0, 1: S from tensor memory, maximum and
//                   sum of the row, P = 2^(s - m) as bf16 over S's columns
//   warp 8          one thread issues the products
//   warp 9          TMA of K and V tiles into a ring
//
// A row's reference m is raised, and its output scaled, only when a score
// exceeds it by kSlack (log2): p stays below 2^kSlack, far inside fp32 and
// bf16, and after the first tiles the output is hardly ever touched.
//
// The tiles of all groups (KV head x 256 rows) are dealt to the blocks as equal
// contiguous runs; a piece leaves m, l and o of its rows for the join (mk_attend.cu).
//
// Bound: the tensor cores (4 head_dim flops a row and position) and, nearly as
// much, the exponentials (16 a clock and SM: 128 x 128 of them last as long as the
// tile's two products); with up to about 128 rows, the cache's bytes.
#include "mk_attend.h"
#include "mk_ptx.h"

namespace mk {
namespace {

using namespace ptx;

constexpr int kSoftmaxThreads = 256;
constexpr int kTcThreads = kSoftmaxThreads + 64;
constexpr float kSlack = 8.f;
constexpr int kTcHead = 1;  // tiles that a group's start and end count as

template <int HD>
struct TcLayout {
  static constexpr int kSlotBytes = kTcTile * HD * 2;       // K or V tile: [HD/64][128 rows][128 B], swizzled
  static constexpr int kSlots = 128 * 1024 / kSlotBytes;
  static constexpr int kQ = kSlots * kSlotBytes;            // two query tiles, laid out the same
  static constexpr int kQBytes = kTcRows * HD * 2;
  static constexpr int kCtl = kQ + 2 * kQBytes;
  static constexpr int kTotal = kCtl + 512 + 1024;          // 1024: aligned by hand
};

struct TcCtl {
  unsigned long long full[8], empty[8];
  unsigned long long q_full, s_full[2], p_full[2], o_done[2];
  uint32_t tmem;
  int dead, max_len;
};
static_assert(sizeof(TcCtl) <= 512, "control block");

// One block's run within a group.
struct Piece {
  int kvh, row0, rows, n, t0;  // rows of the group from row0 on, tiles t0 ... t0 + n
  int gidx;
  bool first, last, pair;
};

struct Walk {
  int tiles, groups, total_rows;
  int64_t u, end;
  __device__ __forceinline__ bool next(Piece& a) {
    while (u < end) {
      const int n = tiles + kTcHead;
      a.gidx = (int)(u / n);
      const int r = (int)(u % n), take = (int)min((int64_t)(n - r), end - u);
      u += take;
      a.kvh = a.gidx / groups;
      a.row0 = a.gidx % groups * 2 * kTcRows;
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
__device__ __forceinline__ int k_place(const Piece& a, int t) { return a.pair ? 2 * t : (t ? 2 * t - 1 : 0); }
__device__ __forceinline__ int v_place(const Piece& a, int t) { return a.pair ? 2 * t + 1 : min(2 * t + 2, 2 * a.n - 1); }

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
  const CacheView& c = p.c;
  volatile int* dead = &ctl->dead;

  if (tid == 0) {
    for (int s = 0; s < S::kSlots; ++s) {
      mbar_init(smem_addr(&ctl->full[s]), 1);
      mbar_init(smem_addr(&ctl->empty[s]), 1);
    }
    mbar_init(smem_addr(&ctl->q_full), kSoftmaxThreads);
    for (int s = 0; s < 2; ++s) {
      mbar_init(smem_addr(&ctl->s_full[s]), 1);
      mbar_init(smem_addr(&ctl->p_full[s]), kSoftmaxThreads / 2);
      mbar_init(smem_addr(&ctl->o_done[s]), 1);
    }
    ctl->dead = 0;
    ctl->max_len = 0;
    fence_mbar_init();
  }
  if (warp == 8) tmem_alloc(smem_addr(&ctl->tmem), 512);
  __syncthreads();
  grid_launch_next();
  int longest = 0;
  for (int b = tid; b < c.B; b += kTcThreads) longest = max(longest, min(__ldg(p.seq_lens + b), c.T));
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) atomicMax(&ctl->max_len, longest);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  // No sequence attends behind the longest: what lies there is not read.
  const int prefix_end = min(p.prefix, ctl->max_len);
  const int tiles = (prefix_end + kTcTile - 1) / kTcTile;
  const int64_t cost = tiles ? (int64_t)(tiles + kTcHead) * p.tc_groups * c.nkv : 0;
  const int G = active_blocks(cost, gridDim.x), cta = blockIdx.x;
  Walk walk{tiles, p.tc_groups, c.B * p.group, 0, 0};
  if (cta < G) walk.u = first_unit(cost, cta, G), walk.end = first_unit(cost, cta + 1, G);
  Piece a;

  if (warp == 9) {  // ---- TMA: K and V tiles in the order of k_place, v_place
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
        if (wanted) row = (int)(c.row(p.layer, 0, at, &ok) + a.kvh * c.head_pitch());
        if (!ok) set_status(c.status, MK_ERR_RANGE, 0);
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
        if (++slot == S::kSlots) slot = 0, phase ^= 1;
      }
    }
    if (__any_sync(0xffffffffu, *dead)) {  // copies still in flight land before the block ends
      const uint64_t t0 = globaltimer();
      for (int s = 0; s < S::kSlots; ++s)
        while (!mbar_try(smem_addr(&ctl->full[s]), (uint32_t)s < slot ? phase : phase ^ 1) && globaltimer() - t0 < 20000000ull) {
        }
      if (lane == 0) set_status(c.status, MK_ERR_DEVICE_TIMEOUT, cta);
    }
  } else if (warp == 8) {  // ---- products
    constexpr uint32_t kQk = mma_desc(kTcRows, kTcTile, false), kPv = mma_desc(kTcRows, HD, true);
    uint32_t at = 0;  // tiles that passed through the ring in earlier pieces
    uint32_t q_phase = 0, p_phase[2] = {0, 0};
    while (walk.next(a)) {
      const int n0 = a.pair ? a.n : (a.n + 1) / 2, n1 = a.pair ? a.n : a.n / 2;
      mbar_wait(smem_addr(&ctl->q_full), q_phase, dead);
      q_phase ^= 1;
      tc_fence_after();
      auto slot_of = [&](int place) { return (at + place) % S::kSlots; };
      auto wait_full = [&](int place) { mbar_wait(smem_addr(&ctl->full[slot_of(place)]), (at + place) / S::kSlots & 1, dead); };
      auto qk = [&](int s, int i) {  // scores of the stream's tile i
        const int place = k_place(a, a.pair ? i : 2 * i + s);
        wait_full(place);
        tc_fence_after();
        if (lane == 0) {
          const uint32_t q = base + S::kQ + (a.pair ? s : 0) * S::kQBytes, k = base + slot_of(place) * S::kSlotBytes;
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            const uint32_t off = ks / 4 * (128 * 128) + ks % 4 * 32;
            tc_mma_ss(tmem + kS + s * 128, smem_desc(q + off, 16, 1024), smem_desc(k + off, 16, 1024), kQk, ks > 0);
          }
          tc_commit(smem_addr(&ctl->s_full[s]));
          if (!a.pair || s == 1) tc_commit(smem_addr(&ctl->empty[slot_of(place)]));
        }
        __syncwarp();
      };
      auto pv = [&](int s, int i) {
        const int t = a.pair ? i : 2 * i + s, place = v_place(a, t);
        mbar_wait(smem_addr(&ctl->p_full[s]), p_phase[s], dead);
        p_phase[s] ^= 1;
        wait_full(place);
        const uint32_t v = base + slot_of(place) * S::kSlotBytes;
        const int have = prefix_end - (a.t0 + t) * kTcTile;
        if (have < kTcTile && (!a.pair || s == 0)) {
          // the prefix ends in this tile: what lies behind is anything, and 0 x NaN is NaN
          for (int e = lane; e < (kTcTile - have) * 8 * CB; e += 32) {
            const int chunk = e % 8, cb = e / 8 % CB, r = have + e / (8 * CB);
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v + cb * (kTcTile * 128) + r * 128 + chunk * 16), "r"(0) : "memory");
          }
          fence_async_shared();
          __syncwarp();
        }
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int ks = 0; ks < kTcTile / 16; ++ks)
            tc_mma_ts(tmem + kO + s * 128, tmem + kS + s * 128 + ks * 8, smem_desc(v + ks * 2048, kTcTile * 128, 1024), kPv, i > 0 || ks > 0);
          tc_commit(smem_addr(&ctl->o_done[s]));
          if (!a.pair || s == 1) tc_commit(smem_addr(&ctl->empty[slot_of(place)]));
        }
        __syncwarp();
      };
      qk(0, 0);
      if (n1) qk(1, 0);
      for (int i = 0; i < n0; ++i) {
        pv(0, i);
        if (i + 1 < n0) qk(0, i + 1);
        if (i < n1) pv(1, i);
        if (i + 1 < n1) qk(1, i + 1);
      }
      at += 2 * a.n;
    }
  } else {  // ---- softmax of stream s
    const int s = warp / 4, r = tid % 128;  // row of the stream's tile
    const uint32_t lanes = (uint32_t)(warp % 4) << 21;
    const uint32_t s_at = tmem + lanes + kS + s * 128, o_at = tmem + lanes + kO + s * 128;
    const float scale = fabsf(p.scale);
    const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;  // a negative scale goes into the query's signs
    uint32_t q_phase = 0, s_phase = 0, o_phase = 0;
    while (walk.next(a)) {
      const int n = a.pair ? a.n : (a.n + 1 - s) / 2;
      const int row = (a.pair ? s * kTcRows : 0) + r;
      const bool valid = row < a.rows;
      const int b = (a.row0 + row) / p.group, head = a.kvh * p.group + (a.row0 + row) % p.group;
      const int lim = valid ? min(__ldg(p.seq_lens + b), prefix_end) : 0;
      if (a.pair || s == 0) {  // the row's query, swizzled as TMA would
        const uint4* q = reinterpret_cast<const uint4*>(p.q + ((int64_t)b * c.nq + head) * HD);
        uint4 x[HD / 8];
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) x[i] = valid ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
        uint8_t* at = smem + S::kQ + (a.pair ? s : 0) * S::kQBytes + r * 128;
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) {
          x[i].x ^= flip; x[i].y ^= flip; x[i].z ^= flip; x[i].w ^= flip;
          *reinterpret_cast<uint4*>(at + i / 8 * (kTcRows * 128) + (((i % 8) ^ (r & 7)) << 4)) = x[i];
        }
        fence_async_shared();
      }
      tc_fence_before();
      mbar_arrive(smem_addr(&ctl->q_full));
      // a stream without tiles waits for nothing else: it must not arrive for the next piece before the other has for this
      if (n == 0) mbar_wait(smem_addr(&ctl->q_full), q_phase, dead);
      q_phase ^= 1;

      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i) {
        const int t0 = (a.t0 + (a.pair ? i : 2 * i + s)) * kTcTile;
        mbar_wait(smem_addr(&ctl->s_full[s]), s_phase, dead);
        s_phase ^= 1;
        tc_fence_after();
        uint32_t x[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(s_at + q * 32, x + q * 32);
        tmem_wait_ld();
        if (__any_sync(0xffffffffu, t0 + kTcTile > lim)) {
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (t0 + e >= lim) x[e] = 0xff800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 4) {
#pragma unroll
          for (int q = 0; q < 4; ++q) mx[q] = fmaxf(mx[q], __uint_as_float(x[e + q]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale;
        const bool raise = top > m + kSlack || (m == -INFINITY && top > m);
        if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? ex2(m - top) : 1.f;
          if (raise) m = top;
          l *= f;
          if (i > 0) {  // the stream's output so far, once its last product is done
            mbar_wait(smem_addr(&ctl->o_done[s]), o_phase ^ 1, dead);
            tc_fence_after();
#pragma unroll 1
            for (int q = 0; q < HD / 32; ++q) {
              uint32_t y[32];
              tmem_ld32(o_at + q * 32, y);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
              tmem_st32(o_at + q * 32, y);
            }
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p0 = ex2(fmaf(__uint_as_float(x[q * 32 + 2 * e]), scale, -ref));
            const float p1 = ex2(fmaf(__uint_as_float(x[q * 32 + 2 * e + 1]), scale, -ref));
            sum[e & 1] += p0;
            sum[2 + (e & 1)] += p1;
            y[e] = pack_bf16x2(p0, p1);  // the operand of the second product, as the cache is
          }
          tmem_st16(s_at + q * 16, y);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_addr(&ctl->p_full[s]));
        o_phase ^= 1;
      }
      // leave the piece
      const int64_t entry = ((int64_t)cta + a.gidx) * 2 + s;
      if (tid == 0) {
        if (a.first) p.pre_blocks[a.gidx].x = cta;
        if (a.last) p.pre_blocks[a.gidx].y = cta;
      }
      if (valid) p.pre_ml[entry * kTcRows + r] = make_float2(m, l);
      if (n) {
        mbar_wait(smem_addr(&ctl->o_done[s]), o_phase ^ 1, dead);
        tc_fence_after();
        float* out = p.pre_o + (entry * kTcRows + r) * HD;
#pragma unroll 1
        for (int q = 0; q < HD / 32; ++q) {
          uint32_t y[32];
          tmem_ld32(o_at + q * 32, y);
          tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) *reinterpret_cast<uint4*>(out + q * 32 + e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
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
  if (c.d.head_dim == 128)
    attend_prefix_kernel<128><<<c.n_sm, kTcThreads, TcLayout<128>::kTotal, stream>>>(p, c.ktall, c.vtall, c.tall);
  else
    attend_prefix_kernel<64><<<c.n_sm, kTcThreads, TcLayout<64>::kTotal, stream>>>(p, c.ktall, c.vtall, c.tall);
  return cudaGetLastError();
}

}  // namespace mk
