// Block tables and slot maps from request lengths, and the new tokens' keys and
// values into their pages.
//   extend    row i gets t_i new tokens: with L_i its length and p the page size, f_i = ceil((L_i + t_i) / p) -
//             ceil(L_i / p) pages come off the free stack, rows in order (b_i: pages of the rows before it):
//             table[s_i][ceil(L_i / p) + j] = free[top - 1 - b_i - j]; its token at position P goes to place
//             table[s_i][P / p] p + P % p
//   truncate  row i keeps its first K_i tokens; the pages behind them go back, in the order that undoes an extend
//   append    [G][d] values of a token to the place that extend gave it
// Sums over the rows are exclusive prefix sums in one block (one row a thread), so the result depends on nothing but
// the inputs.  Slots and lengths live on the device: everything is checked here before anything is changed, and a call
// that cannot be done (a slot that is out of range or comes twice, no pages left, a table row that is full, a page
// number out of range among those it would hand out or give back) changes nothing, hands out no places (-1) and leaves
// its code in the status word.  A page number is checked before it becomes a place: id * page_size would wrap in 32 bits.
//
// The tokens' places are independent of one another: each finds its row and takes its page from the old table or the
// old stack, so a second launch over as many blocks as there is work writes them.
//
// Measured on a GB300: extend and truncate of 256 rows of one token 7.0 us (two
// launches of one block; their checks, sums and two trips to memory), of 64
// prompts of up to 2048 tokens in pages of 16 11.5 us (three launches).  Without
// the checks of page numbers 6.5 and 10.2 us.  append of
// 16 x 512 tokens of 8 heads of 128 bf16 12.3 us (5.5 TB/s of the 6.8 of a copy;
// 18.2 us with a place looked up before each load), of 256 tokens 2.6 us.
#include "attn.h"
#include "attn_device.cuh"

namespace dl {
namespace at {

static __device__ int32_t g_pages_status;

namespace {

constexpr int PT = AT_ROWS;            // threads of the block that sums over the rows

// Exclusive prefix sums of two numbers over the block; the totals as well.
__device__ __forceinline__ void scan2(long long& a, long long& b, long long& ta, long long& tb, long long* sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  if (lane == 31) {
    sm[warp] = x;
    sm[32 + warp] = y;
  }
  __syncthreads();
  if (warp == 0) {
    const int nw = blockDim.x >> 5;
    long long p = lane < nw ? sm[lane] : 0, r = lane < nw ? sm[32 + lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, p, o), v = __shfl_up_sync(0xffffffffu, r, o);
      if (lane >= o) {
        p += u;
        r += v;
      }
    }
    sm[lane] = p;
    sm[32 + lane] = r;
  }
  __syncthreads();
  const long long pa = warp ? sm[warp - 1] : 0, pb = warp ? sm[32 + warp - 1] : 0;
  ta = sm[(blockDim.x >> 5) - 1];
  tb = sm[32 + (blockDim.x >> 5) - 1];
  a = pa + x - a;
  b = pb + y - b;
  __syncthreads();
}

// Whether this thread's slot (one a thread, negative: none) was named by another thread as well: a table of 4 n places.
__device__ __forceinline__ bool named_twice(int slot, int32_t* seen) {
  for (int k = threadIdx.x; k < 4 * PT; k += blockDim.x) seen[k] = -1;
  __syncthreads();
  bool twice = false;
  if (slot >= 0) {
    uint32_t k = ((uint32_t)slot * 2654435761u >> 12) & (4 * PT - 1);
    for (;;) {                         // PT names in 4 PT places: there is an empty one
      const int was = atomicCAS(&seen[k], -1, slot);
      if (was == -1) break;
      if (was == slot) {
        twice = true;
        break;
      }
      k = (k + 1) & (4 * PT - 1);
    }
  }
  __syncthreads();
  return twice;
}

// One entry of the maps: token t of row `row`, whose length was `old` and whose new pages start at `base` from the
// top of a stack of `height`.
__device__ __forceinline__ void place(const PagesArgs& a, int64_t e, int slot, int old, int base, int height, int t) {
  const int pos = old + t, page = 1 << a.page_shift, col = pos >> a.page_shift, have = (old + page - 1) >> a.page_shift;
  int id;
  if (col >= have) {
    id = a.free[1 + height - 1 - base - (col - have)];
    if ((pos & (page - 1)) == 0) a.table[(int64_t)slot * a.table_stride + col] = id;
  } else {
    id = a.table[(int64_t)slot * a.table_stride + col];
  }
  a.where[e] = (int32_t)(((uint32_t)id << a.page_shift) + (uint32_t)(pos & (page - 1)));
  if (a.positions) a.positions[e] = pos;
}
__device__ __forceinline__ void no_place(const PagesArgs& a, int64_t e) {
  a.where[e] = -1;
  if (a.positions) a.positions[e] = -1;
}

// Checks, sums, and what changes a row: its length and the stack's height.  One block.  FILL: the maps as well.
template <bool FILL>
__global__ void __launch_bounds__(PT) extend_kernel(const PagesArgs a) {
  __shared__ long long sm[64];
  __shared__ int32_t seen[4 * PT];     // the names, then (FILL) the rows' slots, lengths, bases and starts
  const int i = threadIdx.x, page = 1 << a.page_shift;
  const bool row = i < a.n;
  int slot = -1, tok = 0, old = 0, err = 0;
  if (row) {
    slot = a.slots[i];
    tok = a.tokens ? a.tokens[i] : 1;
  }
  const int height = a.free[0];
  const bool stack = height >= 0 && height <= a.num_pages;
  // The i-th page from the top and the row's half-filled one: asked for early, looked at behind the sums.
  const int top = stack && i < height ? a.free[height - i] : 0;
  int half = 0;
  auto out_of_range = [&](int id) { return (unsigned)id >= (unsigned)a.num_pages; };
  if (row) {
    if (slot < 0 || slot >= a.num_slots) {
      err = DEV_BAD_SLOT;
      slot = -1;
    } else {
      old = a.lengths[slot];
      const int cap = a.max_pages << a.page_shift;
      if (tok < 0 || old < 0 || old > cap || (a.T > 0 && tok > a.T)) err = DEV_BAD_LENGTH;
      else if (tok > cap - old) err = DEV_ROW_FULL;
      else if (tok > 0 && (old & (page - 1))) half = a.table[(int64_t)slot * a.table_stride + (old >> a.page_shift)];
    }
    if (err) tok = 0;
  }
  if (named_twice(slot, seen)) err = DEV_BAD_SLOT;
  const int fresh = err ? 0 : ((old + tok + page - 1) >> a.page_shift) - ((old + page - 1) >> a.page_shift);
  long long start = tok, base = fresh, tokens, pages;
  scan2(start, base, tokens, pages, sm);
  if (i == 0) {
    if (a.T == 0 && tokens > a.size) err = DEV_BAD_LENGTH;
    if (!stack) err = DEV_BAD_PAGE;
    else if (pages > height) err = DEV_NO_PAGES;
  }
  if (stack && pages <= height) {
    bool odd = i < pages && out_of_range(top);
#pragma unroll 4
    for (int k = i + PT; k < (int)pages; k += PT) odd |= out_of_range(a.free[height - k]);
    if (odd) err = DEV_BAD_PAGE;
  }
  if (out_of_range(half)) err = DEV_BAD_PAGE;
  if (err) atomicCAS(&g_pages_status, 0, err);
  int32_t *slots = seen, *olds = seen + PT, *bases = seen + 2 * PT, *starts = seen + 3 * PT;
  __shared__ int32_t toks[PT];
  if (FILL) {
    slots[i] = slot;
    olds[i] = old;
    bases[i] = (int32_t)base;
    starts[i] = row ? (int32_t)start : 0x7fffffff;
    toks[i] = tok;
  }
  const bool bad = __syncthreads_or(err != 0);
  if (row) {
    a.starts[i] = bad ? 0 : (int32_t)start;
    if (!bad) a.lengths[slot] = old + tok;
  }
  if (i == 0) {
    a.starts[a.n] = bad ? 0 : (int32_t)tokens;
    if (!bad) a.free[0] = height - (int32_t)pages;
  }
  if (!FILL) {
    if (row) {
      a.work[2 * i] = old;
      a.work[2 * i + 1] = (int32_t)base;
    }
    if (i == 0) {
      a.work[2 * a.n] = height;
      a.work[2 * a.n + 1] = bad;
    }
    return;
  }
  if (a.T > 0) {
    for (int e = i; e < (int)a.size; e += PT) {
      const int t = e / a.n, r = e - t * a.n;
      if (!bad && t < toks[r]) place(a, e, slots[r], olds[r], bases[r], height, t);
      else no_place(a, e);
    }
  } else {
    for (int e = i; e < (int)a.size; e += PT) {
      if (bad || e >= tokens) {
        no_place(a, e);
        continue;
      }
      int lo = 0, hi = a.n - 1;
      while (lo < hi) {                // the last row that starts at or before e
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= e) lo = mid; else hi = mid - 1;
      }
      place(a, e, slots[lo], olds[lo], bases[lo], height, e - starts[lo]);
    }
  }
}

constexpr int FT = 256;                // threads of a block that writes places
__global__ void __launch_bounds__(FT) fill_kernel(const PagesArgs a) {
  __shared__ int32_t starts[AT_ROWS + 1];
  pdl_wait_primary();
  const int height = a.work[2 * a.n];
  const bool bad = a.work[2 * a.n + 1] != 0;
  for (int i = threadIdx.x; i <= a.n; i += FT) starts[i] = a.starts[i];
  __syncthreads();
  const int64_t tokens = starts[a.n];
  for (int64_t e = (int64_t)blockIdx.x * FT + threadIdx.x; e < a.size; e += (int64_t)gridDim.x * FT) {
    int r, t;
    bool live;
    if (a.T > 0) {
      t = (int)(e / a.n);
      r = (int)(e - (int64_t)t * a.n);
      live = !bad && t < starts[r + 1] - starts[r];
    } else {
      live = !bad && e < tokens;
      int lo = 0, hi = a.n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (starts[mid] <= e) lo = mid; else hi = mid - 1;
      }
      r = lo;
      t = (int)(e - starts[r]);
    }
    if (live) place(a, e, a.slots[r], a.work[2 * r], a.work[2 * r + 1], height, t);
    else no_place(a, e);
  }
}

// Pages that a thread gives back and keeps in registers between their check and the stack; further ones are read again.
constexpr int BACK = 4;
__global__ void __launch_bounds__(PT) truncate_kernel(const PagesArgs a) {
  __shared__ long long sm[64];
  __shared__ int32_t seen[4 * PT];
  const int i = threadIdx.x, page = 1 << a.page_shift;
  const bool row = i < a.n;
  int slot = -1, keep = 0, old = 0, err = 0;
  if (row) {
    slot = a.slots[i];
    keep = a.tokens ? a.tokens[i] : 0;
  }
  const int height = a.free[0];
  if (row) {
    if (slot < 0 || slot >= a.num_slots) {
      err = DEV_BAD_SLOT;
      slot = -1;
    } else {
      old = a.lengths[slot];
      if (old < 0 || old > (a.max_pages << a.page_shift) || keep < 0 || keep > old) err = DEV_BAD_LENGTH;
    }
  }
  if (named_twice(slot, seen)) err = DEV_BAD_SLOT;
  const int first = err ? 0 : (keep + page - 1) >> a.page_shift;
  const int back = err ? 0 : ((old + page - 1) >> a.page_shift) - first;
  long long none = 0, base = back, zero, pages;
  scan2(none, base, zero, pages, sm);
  if (i == 0 && (height < 0 || height > a.num_pages || pages > a.num_pages - height)) err = DEV_BAD_PAGE;
  if (err) atomicCAS(&g_pages_status, 0, err);
  int32_t *slots = seen, *firsts = seen + PT, *bases = seen + 2 * PT;
  slots[i] = slot;
  firsts[i] = first;
  bases[i] = row ? (int32_t)base : 0x7fffffff;
  if (__syncthreads_or(err != 0)) return;
  const int most = (int)pages;
  auto page_at = [&](int k) {          // the k-th page that goes back
    int lo = 0, hi = a.n - 1;
    while (lo < hi) {                  // the last row whose pages start at or before k
      const int mid = (lo + hi + 1) >> 1;
      if (bases[mid] <= k) lo = mid; else hi = mid - 1;
    }
    return a.table[(int64_t)slots[lo] * a.table_stride + firsts[lo] + k - bases[lo]];
  };
  int ids[BACK];
  bool odd = false;
#pragma unroll
  for (int u = 0; u < BACK; ++u) {
    ids[u] = i + u * PT < most ? page_at(i + u * PT) : 0;
    odd |= (unsigned)ids[u] >= (unsigned)a.num_pages;
  }
  for (int k = i + BACK * PT; k < most; k += PT) odd |= (unsigned)page_at(k) >= (unsigned)a.num_pages;
  if (odd) atomicCAS(&g_pages_status, 0, DEV_BAD_PAGE);
  if (__syncthreads_or(odd)) return;
  if (row) a.lengths[slot] = keep;
  if (i == 0) a.free[0] = height + most;
  int32_t* const to = a.free + 1 + height + most - 1;
#pragma unroll
  for (int u = 0; u < BACK; ++u)
    if (i + u * PT < most) to[-(i + u * PT)] = ids[u];
  for (int k = i + BACK * PT; k < most; k += PT) to[-k] = page_at(k);
}

// Values of V bytes (16: vectors; else one element), [G][d] of a token in E of them.
template <int V> struct Piece;
template <> struct Piece<16> { using T = uint4; };
template <> struct Piece<4> { using T = uint32_t; };
template <> struct Piece<2> { using T = uint16_t; };

// A block moves AT_U * AT_T consecutive pieces of k and of v, every load of a thread before its first store.
constexpr int AT_U = 4, AT_T = 256;
template <int V, int EL>
__global__ void __launch_bounds__(AT_T) append_kernel(const AppendArgs a) {
  using P = typename Piece<V>::T;
  constexpr int PE = V / EL;           // elements of a piece
  const uint32_t per_head = (uint32_t)a.d / PE, per = (uint32_t)a.G * per_head;
  const int64_t total = a.T * a.n * per, e0 = (int64_t)blockIdx.x * (AT_U * AT_T) + threadIdx.x;
  P kv[AT_U], vv[AT_U];
  int at[AT_U];
  uint32_t c[AT_U];
#pragma unroll
  for (int u = 0; u < AT_U; ++u) {
    const int64_t e = e0 + u * AT_T;
    at[u] = -1;
    if (e >= total) continue;
    const int64_t tok = total <= 0xffffffffll ? (int64_t)((uint32_t)e / per) : e / per;
    c[u] = (uint32_t)(e - tok * per);
    const int64_t t = a.n == 1 ? tok : (int64_t)((uint32_t)tok / (uint32_t)a.n), r = tok - t * a.n;
    at[u] = a.where[tok];
    kv[u] = *reinterpret_cast<const P*>(static_cast<const char*>(a.k) + EL * (t * a.k_st + r * a.k_sn + (int64_t)c[u] * PE));
    vv[u] = *reinterpret_cast<const P*>(static_cast<const char*>(a.v) + EL * (t * a.v_st + r * a.v_sn + (int64_t)c[u] * PE));
  }
#pragma unroll
  for (int u = 0; u < AT_U; ++u) {
    if (at[u] < 0) continue;
    const int id = at[u] >> a.page_shift, off = at[u] & ((1 << a.page_shift) - 1);
    if (id >= a.num_pages) {
      atomicCAS(&g_pages_status, 0, DEV_BAD_PAGE);
      continue;
    }
    const uint32_t g = c[u] / per_head, x = (c[u] - g * per_head) * PE;
    *reinterpret_cast<P*>(static_cast<char*>(a.kp.p) + EL * (id * a.kp.sp + g * a.kp.sg + off * a.kp.st + x)) = kv[u];
    *reinterpret_cast<P*>(static_cast<char*>(a.vp.p) + EL * (id * a.vp.sp + g * a.vp.sg + off * a.vp.st + x)) = vv[u];
  }
}

}  // namespace

// Up to this many entries the block that sums over the rows writes the maps itself.  256 rows, with the truncate that
// follows: 2048 entries 7.5 us, 8.0 in two launches; 4096 entries 8.8 and 7.9.
constexpr int64_t FILL_ONE = 2048;

cudaError_t launch_extend(const PagesArgs& a, int sms, cudaStream_t s) {
  if (a.size <= FILL_ONE) {
    extend_kernel<true><<<1, PT, 0, s>>>(a);
    return cudaGetLastError();
  }
  extend_kernel<false><<<1, PT, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t want = (a.size + FT - 1) / FT, most = 8 * (int64_t)sms;
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.gridDim = dim3((unsigned)(want < most ? want : most));
  c.blockDim = dim3(FT);
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, fill_kernel, a);
}

cudaError_t launch_truncate(const PagesArgs& a, cudaStream_t s) {
  truncate_kernel<<<1, PT, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_append(int elem, bool vec, const AppendArgs& a, cudaStream_t s) {
  const int64_t pieces = a.T * a.n * (int64_t)a.G * a.d / (vec ? 16 / elem : 1);
  const int64_t blocks = (pieces + AT_U * AT_T - 1) / (AT_U * AT_T);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)blocks;
  if (vec && elem == 4) append_kernel<16, 4><<<grid, AT_T, 0, s>>>(a);
  else if (vec) append_kernel<16, 2><<<grid, AT_T, 0, s>>>(a);
  else if (elem == 4) append_kernel<4, 4><<<grid, AT_T, 0, s>>>(a);
  else append_kernel<2, 2><<<grid, AT_T, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t read_pages_status(cudaStream_t s, int32_t* code) { return take_status(g_pages_status, s, code); }

}  // namespace at
}  // namespace dl
