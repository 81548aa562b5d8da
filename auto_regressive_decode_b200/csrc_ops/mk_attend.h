// What the attention kernels share: parameters, workspace layout.
#pragma once

#include "mk_cache.h"

namespace mk {

constexpr int kTcRows = 128;    // rows of a tensor-core row tile (the M of its products)
constexpr int kTcTile = 128;    // cache positions of its tiles

struct AttendParams {
  CacheView c;
  int layer, group, box;
  int whole;               // a tile that starts at a multiple of kTile (contiguous: anywhere) is one TMA box
  int prefix, base;        // own tiles start at base: prefix rounded down so that no box crosses a page
  int rows;                // batch * group: rows of a KV head over the prefix
  int wide;                // some piece has more than 32 rows: one query buffer
  float scale;             // scale * log2 e
  const uint16_t* q;
  const int32_t* seq_lens;
  uint16_t* out;
  float* lse;
  int tc, tc_groups;       // the prefix runs in attend_prefix_tc: row groups of two row tiles per KV head
  int tc_lanes;            // tc_groups: every row group has blocks of its own; 1: they follow one another
  int tc_blocks;           // blocks of a lane
  // workspace
  float *pre_o, *own_o;    // [piece][rows of the piece][hd]
  float2 *pre_ml, *own_ml; // [piece][rows]
  int2 *pre_blocks, *own_blocks;  // [group] first and last block with a piece of it
  int* sched;              // [0] whether prefix groups have pieces, [1...] own tiles of each sequence
};

// Blocks that work, and the first unit of cost of block i of G (G is below 2^15).
__device__ __forceinline__ int active_blocks(int cost, int grid) { return min(cost, grid); }
__device__ __forceinline__ int first_unit(int cost, int i, int G) {
  const int q = cost / G;
  return q * i + (cost - q * G) * i / G;
}

// A lane of attend_prefix_tc goes through its groups in order; the entry of the workspace that block i
// of the lane leaves its piece of the lane's group k at (a piece is one more than its predecessor's).
__device__ __forceinline__ int tc_entry(const AttendParams& p, int lane, int i, int k) {
  return lane * (p.tc_blocks + p.c.nkv * (p.tc_groups / p.tc_lanes)) + i + k;
}

// Where attend_prefix_tc leaves an output: float offset, within an entry of kTcRows rows, of the
// 16-byte chunk `ch` of row r.  kTcParts blocks, [row][chunk]: of each half of the row's columns the
// first part, the second, ...; chunks swizzled, as they lay in shared memory.
constexpr int kTcParts = 4;
template <int HD>
struct TcOut {
  static constexpr int kHalf = HD / 8, kMine = kHalf / kTcParts, kRow = 2 * kMine;  // chunks of half a row, of its part, of a row there
  static constexpr int kFloats = kTcRows * kRow * 4;                                // a block
  // rows r ... r + 7 of one chunk lie in different banks
  static __device__ __forceinline__ int swizzle(int r, int ch) { return ch ^ (kRow == 8 ? r & 7 : r >> 1 & 3); }
  static __device__ __forceinline__ int chunk(int r, int ch) {
    const int half = ch / kHalf, part = ch % kHalf / kMine, e = ch % kMine;
    return part * kFloats + (r * kRow + swizzle(r, half * kMine + e)) * 4;
  }
};

// Attention over the prefix with tcgen05 (mk_attend_tc.cu): leaves its pieces
// in pre_o / pre_ml as entries of kTcRows rows, two a piece, and the blocks of
// every group in pre_blocks.
cudaError_t attend_prefix_tc_prepare();
cudaError_t attend_prefix_tc(const AttendParams& p, const mk_cache& c, cudaStream_t stream);

}  // namespace mk
