// Kernel arguments and launch entry points of the mixer operators: short
// causal convolution, state space scan, gated and residual norms (internal).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace dl {
namespace mx {

constexpr int MX_ROWS = 1024;          // rows of one call
// Rows of one launch: their plan travels as a launch parameter, which costs
// about 0.2 us of host time a KiB, so it is kept to 2 KiB.
constexpr int MX_GROUP = 128;          // prompts
constexpr int MX_STEP = 512;           // one token a row: only slots
enum { T_F32 = 0, T_BF16 = 1, T_F16 = 2 };
enum { ACT_NONE = 0, ACT_SILU = 1, ACT_SIGMOID = 2 };
enum { NORM_RMS = 0, NORM_LAYER = 1 };

// One row (a sequence) of a call.  Its token t sits at tensor offset
// (begin + t) * stride_t + row * stride_n (packed tokens have stride_n = 0,
// token-major ones begin = 0).  tile0: the row's first work tile.
struct RowItem {
  int32_t slot, begin, len, tile0;
};
// A row's length and whether it starts from an empty state share one word.
constexpr int32_t FRESH_BIT = (int32_t)0x80000000u;
__host__ __device__ inline int32_t row_len(const RowItem& r) { return r.len & 0x7fffffff; }
__host__ __device__ inline bool row_fresh(const RowItem& r) { return r.len < 0; }

// A per-token tensor: element strides between tokens and between rows.
struct TokView {
  const void* p;
  int64_t st, sn;
};

// The row that tile `tile` belongs to: tiles are numbered row by row, with
// `per_row` of them in every row when that is not zero.
__device__ __forceinline__ int find_row(const RowItem* items, int rows, int tile, int per_row) {
  if (per_row) return tile / per_row;
  int lo = 0, hi = rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (items[mid].tile0 <= tile) lo = mid; else hi = mid - 1;
  }
  return lo;
}

constexpr int CONV_PARTS = 4;
struct ConvArgs {
  TokView x;
  const void* w;            // [C, W]
  const void* b;            // [C] or null
  void* state;              // [num_slots, W - 1, C] or null
  TokView y[CONV_PARTS];    // outputs: consecutive channel ranges
  int32_t c0[CONV_PARTS + 1];   // first channel of each range; unused ranges start at C
  int32_t C, W, act, l2c, hd, w_f32;
  int32_t rows, tiles, per_row, TT;   // TT: tokens of one tile (step: rows)
  float eps;
};
struct ConvPrompt : ConvArgs {
  RowItem items[MX_GROUP];
};
struct ConvStep : ConvArgs {
  int32_t slot[MX_STEP];    // ~slot for a fresh row
};
// Tokens of a tile for this much work (a step: rows, one token each).
int conv_tile(int64_t tokens, int C, int sms);
cudaError_t launch_conv(int dtype, bool vec, const ConvPrompt& a, cudaStream_t s);
// One token a row, tiles of TT rows.
cudaError_t launch_conv_step(int dtype, bool vec, const ConvStep& a, cudaStream_t s);

struct SsmBase {
  TokView x, dt, B, C, y;
  const float* A;           // [H]
  const float* D;           // [H] or null
  const float* dt_bias;     // [H] or null
  float* state;             // [num_slots, H, P, N] or null
  int32_t H, G, P, N, softplus, dt_f32;
  int32_t rows;
};
struct SsmArgs : SsmBase {
  RowItem items[MX_GROUP];
};
struct SsmStep : SsmBase {
  int32_t slot[MX_STEP];    // ~slot for a fresh row
};
cudaError_t launch_ssm_step(int dtype, const SsmStep& a, cudaStream_t s);

// How a scan splits a call: `units` units of work a segment of seg_tokens
// tokens (ptiles a head); split: a row may have several segments, joined
// through a workspace of tiles * H * (P * N + 1) floats.
struct SsmPlan {
  int32_t ptiles, units, seg_tokens, sms;
  bool split;
};
SsmPlan ssm_scan_plan(int H, int P, int N, int rows, const int32_t* lens, int64_t T, int sms);
// vec: x, B, C and y are 16-byte aligned, in their strides and widths too.
cudaError_t launch_ssm_scan(int dtype, bool vec, const SsmArgs& a, const SsmPlan& p, int tiles, int per_row, float* ws,
                            cudaStream_t s);
// The states at the segments' starts from each segment's own end state and decay (in place).
cudaError_t launch_ssm_join(const SsmArgs& a, int seg_tokens, int tiles, int per_row, float* ws, cudaStream_t s);
SsmPlan ssm_tc_plan(int H, int P, int rows, const int32_t* lens, int64_t T, int sms);
// bf16, N <= 128.  tokens: extent of the token axis (packed: all rows').
cudaError_t launch_ssm_tc(bool vec, int64_t tokens, const SsmArgs& a, const SsmPlan& p, int tiles, int per_row,
                          float* ws, cudaStream_t s);
// Wait for the stream, then read and clear the kernels' status word.
cudaError_t read_mixer_status(cudaStream_t s, int32_t* code);

struct GatedNormArgs {
  const void *x, *gate, *w, *b;
  void* y;
  int64_t xs, gs, ys;       // row strides; heads and channels are contiguous
  int64_t rows;
  int32_t H, d, kind, act, gate_first, w_f32, w_heads;   // w_heads: w, b are [H, d]
  float eps;
};
cudaError_t launch_gated_norm(int dtype, bool vec, const GatedNormArgs& a, cudaStream_t s);

struct AddNormArgs {
  const void *x, *res, *w, *b, *scale, *post;
  void *y, *h;
  int64_t xs, rs, ys, hs;
  int64_t rows;
  int32_t D, kind, w_f32;
  float eps, alpha;
};
cudaError_t launch_add_norm(int dtype, bool res_f32, bool vec, const AddNormArgs& a, cudaStream_t s);

}  // namespace mx
}  // namespace dl
