// Kernel arguments and launch entry points of the attention operators: block
// tables and slot maps, keys and values into pages, attention over the pages
// (internal).
#pragma once
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace dl {
namespace at {

constexpr int AT_ROWS = 1024;          // rows (requests) of one call
constexpr int AT_DIM = 256;            // head dimension at most

// Block tables: row i of a call is slot slots[i]; token p of a slot lies in
// page table[slot][p / page] at place p % page.
struct PagesArgs {
  const int32_t* slots;      // [n]
  const int32_t* tokens;     // [n] new tokens (extend; null: one each) or lengths to keep (truncate; null: 0)
  int32_t* table;            // [num_slots][max_pages], rows table_stride apart
  int32_t* lengths;          // [num_slots]
  int32_t* free;             // [1 + num_pages]: how many pages are free, then a stack of them
  int32_t* starts;           // [n + 1]
  int32_t* where;            // [size], or [T][n] when T > 0
  int32_t* positions;        // as where, or null
  int32_t* work;             // [2 n + 2] scratch: every row's old length and first page on the stack; its height; error
  int64_t table_stride, size;
  int32_t n, T, num_slots, max_pages, num_pages, page_shift;
};
cudaError_t launch_extend(const PagesArgs& a, int sms, cudaStream_t s);
cudaError_t launch_truncate(const PagesArgs& a, cudaStream_t s);

// A pool of pages: element strides between pages, heads and tokens.
struct PoolView {
  void* p;
  int64_t sp, sg, st;
};

struct AppendArgs {
  const void *k, *v;         // token t of row i at t * st + i * sn, [G][d] contiguous
  int64_t k_st, k_sn, v_st, v_sn;
  PoolView kp, vp;
  const int32_t* where;      // [T][n] places (page * page_size + token); negative: left out
  int64_t T;
  int32_t n, G, d, page_shift, num_pages;
};
cudaError_t launch_append(int elem, bool vec, const AppendArgs& a, cudaStream_t s);

struct AttnArgs {
  const void* q;             // token t of row i: packed (starts[i] + t) * st, else t * st + i * sn; [H][d] contiguous
  void* o;
  int64_t q_st, q_sn, o_st, o_sn;
  PoolView kp, vp;
  const int32_t *table, *lengths, *slots;
  const int32_t* starts;     // [n + 1], packed rows; else null
  const int32_t* tokens;     // [n] or null: T each (not packed)
  int64_t table_stride;
  int32_t n, T, H, G, d;     // T: tokens a row at most (packed: of all rows together)
  int32_t page_shift, max_pages, num_slots, num_pages;
  int32_t window, sinks;     // window 0: none
  float scale_log2;          // scale * log2 e
  float* ws;                 // partial results
};

// A tile is `rows` consecutive rows of (token, head of the group) of one row of the call and one head of keys: tpt tokens,
// and hgroups tiles for the heads of a group.  `tiles`: as many as the call may have of a head.  A tile's keys are split
// over `splits` units whose results are joined (the tensor-core kernels: more than 1 says that they may be).
struct AttnPlan {
  int32_t rows, tpt, hgroups, tiles, splits, grid;
  int64_t ws_bytes;
};
// Prompts of every type, head dimension, stride and alignment.
AttnPlan simt_plan(int n, int T, bool packed, int H, int G, int d, int sms);
cudaError_t launch_simt(int dtype, bool vec, const AttnArgs& a, const AttnPlan& p, cudaStream_t s);
// The parts of a split call's tiles become one.
cudaError_t launch_simt_join(int dtype, const AttnArgs& a, const AttnPlan& p, cudaStream_t s);

// One token a row (T = 1, not packed), any type and layout.
AttnPlan simt_step_plan(int n, int H, int G, int d, int sms);
cudaError_t launch_simt_step(int dtype, bool vec, const AttnArgs& a, const AttnPlan& p, cudaStream_t s);
cudaError_t read_simt_step_status(cudaStream_t s, int32_t* code);

// The same for 16-bit types and aligned tensors, on the tensor cores.
bool step_fits(int dtype, bool vec, const AttnArgs& a);
AttnPlan step_plan(int n, int H, int G, int d, int sms);
cudaError_t launch_step(int dtype, const AttnArgs& a, const AttnPlan& p, cudaStream_t s);

// Prompts of 16-bit types with 16-byte aligned tensors and strides, on the tensor cores.
bool tc_fits(int dtype, bool vec, const AttnArgs& a);
AttnPlan tc_plan(int n, int T, bool packed, int H, int G, int d, int sms);
cudaError_t launch_tc(int dtype, const AttnArgs& a, const AttnPlan& p, cudaStream_t s);

// Wait for the stream, then read and clear the kernels' status words.
cudaError_t read_pages_status(cudaStream_t s, int32_t* code);
cudaError_t read_simt_status(cudaStream_t s, int32_t* code);
cudaError_t read_step_status(cudaStream_t s, int32_t* code);
cudaError_t read_tc_status(cudaStream_t s, int32_t* code);

}  // namespace at
}  // namespace dl
