// What the attention kernels share: which row, head and tokens a unit of work
// has, which keys its tokens see, and the status words.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "attn.h"
#include "dl_device.cuh"

namespace dl {
namespace at {

// A translation unit's own status word (a static __device__ variable): wait, read, clear.
inline cudaError_t take_status(int32_t& word, cudaStream_t s, int32_t* code) {
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, word, sizeof *code);
  if (e == cudaSuccess && *code != 0) {
    const int32_t zero = 0;
    e = cudaMemcpyToSymbol(word, &zero, sizeof zero);
  }
  return e;
}

// One tile of a row: tokens [t0, t0 + nt) of it, at positions pos0 ...
struct Tile {
  int row, slot, t0, nt, pos0, begin;  // begin: the row's first token in a packed tensor
};
// Tile numbers.  Token-major: ceil(T / tpt) a row.  Packed: row i has the numbers from starts[i] / tpt + i on, at
// least ceil(its tokens / tpt) of them before the next row's, since floor((s + t) / p) - floor(s / p) + 1 >= ceil(t / p);
// so a tile's row is found without sums over the rows.  One warp calls; false: the tile has no tokens.
__device__ __forceinline__ int packed_tile0(const AttnArgs& a, int i, int tpt) { return a.starts[i] / tpt + i; }
// The tokens of a row, and where they begin in a packed tensor.  A number of tokens below zero or above T is held to
// that and reported to *status, if that is given; starts are held to [0, T].
__device__ __forceinline__ int row_tokens(const AttnArgs& a, int row, int& begin, int32_t* status) {
  begin = 0;
  if (!a.starts) {
    if (!a.tokens) return a.T;
    const int t = a.tokens[row];
    if ((unsigned)t > (unsigned)a.T && status) atomicCAS(status, 0, DEV_BAD_LENGTH);
    return min(max(t, 0), a.T);
  }
  begin = min(max(a.starts[row], 0), a.T);
  return min(max(a.starts[row + 1], begin), a.T) - begin;
}
// The length of a row's slot, at most what its table holds; negative: there is no such slot.  What is out of range is
// reported to *status, if that is given.
__device__ __forceinline__ int row_length(const AttnArgs& a, int row, int& slot, int32_t* status) {
  slot = a.slots[row];
  if (slot < 0 || slot >= a.num_slots) {
    if (status) atomicCAS(status, 0, DEV_BAD_SLOT);
    return -1;
  }
  const int len = a.lengths[slot], cap = a.max_pages << a.page_shift;
  if ((len < 0 || len > cap) && status) atomicCAS(status, 0, DEV_BAD_LENGTH);
  return min(max(len, 0), cap);
}
// Tile `tile` of a row; false: it has no tokens.  (One lane reports.)
__device__ __forceinline__ bool make_tile(const AttnArgs& a, int row, int tile, int tpt, Tile& w, int32_t* status) {
  w.row = row;
  if ((threadIdx.x & 31) != 0) status = nullptr;
  const int t = row_tokens(a, row, w.begin, status);
  if (tile < 0 || (int64_t)tile * tpt >= t) return false;
  w.t0 = tile * tpt;
  w.nt = min(tpt, t - w.t0);
  const int len = row_length(a, row, w.slot, status);
  if (len < 0) return false;
  w.pos0 = len - t + w.t0;             // the new tokens are the slot's last; negative positions see nothing
  return true;
}
__device__ __forceinline__ bool find_tile(const AttnArgs& a, int x, int tpt, Tile& w, int32_t* status) {
  int row, tile;
  if (a.starts) {
    // the last row that starts at or before x: every 32nd row, then the 32 from there on
    const int lane = threadIdx.x & 31, i = 32 * lane;
    const unsigned m = __ballot_sync(0xffffffffu, i < a.n && packed_tile0(a, i, tpt) <= x);
    if (m == 0) return false;
    const int i0 = 32 * (31 - __clz(m)) + lane;
    const unsigned r = __ballot_sync(0xffffffffu, i0 < a.n && packed_tile0(a, i0, tpt) <= x);
    if (r == 0) return false;
    row = i0 - lane + 31 - __clz(r);
    tile = x - packed_tile0(a, row, tpt);
  } else {
    const int per = (a.T + tpt - 1) / tpt;
    row = x / per;
    if (row >= a.n) return false;
    tile = x - row * per;
  }
  return make_tile(a, row, tile, tpt, w, status);
}
// Tiles that a call may have.
inline int64_t tiles_of(int n, int T, bool packed, int tpt) {
  return packed ? (int64_t)T / tpt + n : (int64_t)n * ((T + tpt - 1) / tpt);
}

// The keys that tokens at positions p0 .. p1 see, in blocks of BK: the blocks of the sinks that lie before the window,
// then those of the window.  Numbered 0 .. count - 1.
struct Blocks {
  int sink_blocks, first, count;       // block b: b < sink_blocks ? b : first + b - sink_blocks
  __device__ __forceinline__ int at(int b) const { return b < sink_blocks ? b : first + b - sink_blocks; }
};
template <int BK>
__device__ __forceinline__ Blocks blocks_of(const AttnArgs& a, int p0, int p1) {
  Blocks w;
  const int lo = a.window ? max(0, p0 - a.window + 1) : 0;
  w.sink_blocks = (min(a.sinks, lo) + BK - 1) / BK;
  w.first = max(lo / BK, w.sink_blocks);
  w.count = p1 < 0 ? 0 : w.sink_blocks + max(0, p1 / BK + 1 - w.first);
  if (p1 < 0) w.sink_blocks = 0;
  return w;
}
// Whether position p sees key j.
__device__ __forceinline__ bool sees(const AttnArgs& a, int p, int j) {
  return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
}
// Whether every token at p0 .. p1 sees all keys [j0, j1), and whether none sees key j.
__device__ __forceinline__ bool all_see(const AttnArgs& a, int p0, int p1, int j0, int j1) {
  return j1 - 1 <= p0 && (a.window == 0 || j0 > p1 - a.window || j1 <= a.sinks);
}
__device__ __forceinline__ bool none_sees(const AttnArgs& a, int p0, int p1, int j) {
  return j > p1 || (a.window != 0 && j <= p0 - a.window && j >= a.sinks);
}

// The page of key j of a slot; ids out of range are reported and read as page 0.
__device__ __forceinline__ int page_of(const AttnArgs& a, int slot, int j, int32_t* status) {
  const int id = a.table[(int64_t)slot * a.table_stride + (j >> a.page_shift)];
  if ((unsigned)id < (unsigned)a.num_pages) return id;
  atomicCAS(status, 0, DEV_BAD_PAGE);
  return 0;
}

// A running maximum that is -inf (nothing seen, or every score is -inf) counts as zero where it is subtracted.
__device__ __forceinline__ float held(float m) { return m == -INFINITY ? 0.f : m; }

}  // namespace at
}  // namespace dl
