// Attention of one token a row over pages, 16-bit types: split over the keys of
// all rows and heads alike, and joined.
//
// A row's H / G query heads that share a head of keys are the 16 rows of
// mma.sync products (scores = q k^T, o += p v; fp32 accumulators), so every key
// and value is read from memory once: per = H / G multiply-adds a 16-bit value,
// HBM-bound up to per = 16 and beyond.  What counts is bytes on their way, not
// the products' rate: with 16 rows the 128-row tcgen05 products would be mostly
// padding and their scores would pass through tensor memory; a warp's own
// products keep everything in registers.  Running softmax as in attn_simt.cu,
// in fp32; the reference that scores are taken against moves only when one
// passes it by more than 2^8, so a step needs no maximum over lanes.  Weights
// are rounded to the type for the second product: half a step of the output's
// own type each.
//
// Work is the list of all blocks of 64 keys: rows, then heads, then the blocks
// of a row that its token sees.  Every CTA takes an equal, contiguous part of
// it, whatever the rows' lengths; the lengths are on the device, so each CTA
// sums them itself (a few loads and one scan).  A CTA that has all blocks of a
// head writes its output; a head that several CTAs share leaves (reference, sum,
// o) in the workspace, two parts a CTA at most, and a second launch joins them in
// order.
//
// A warp takes 16 keys of a block: they lie in one page (pages have 16 tokens or
// more), so it looks up one page a block, 32 blocks at a time, and copies 16 rows
// of K and of V asynchronously into its own ring of stages, which no other warp
// reads: no barriers but where a head ends.
//
// Measured on a GB300 (copy: 6.8 TB/s), bf16, 8 heads of keys of 128: 256 x 2048
// tokens 318 us (6.76 TB/s), one row of 131072 87 us (6.2 TB/s), one of 512 9 us
// (two launches, the lengths, the table and the keys one after the other).  A
// head's start and end cost about two blocks: the 37 ragged rows of five heads of
// 64 under a window of 1000 keys take 25 us (2.7 TB/s), 256 rows of 100 tokens of
// 16 heads over each of 4 35 us. 
#include <cmath>

#include "attn_device.cuh"
#include "mixer_device.cuh"

namespace dl {
namespace at {

static __device__ int32_t g_step_status;

namespace {

using mx::from_f;
using mx::pack2;

constexpr int NW = 4, THREADS = 32 * NW, KT = 16, BK = KT * NW;   // warps, keys of a warp's step and of a block
constexpr int ROWS = 16;               // query heads of a product
constexpr int RED = 2 * (NW + 1) * ROWS;   // the warps' references and sums of a segment, and the segment's own
// A head's start and end cost about as much as this many blocks; they count where the list is long enough for every
// CTA to get a block all the same.  37 ragged rows under a window 25 us, 34 with 0 and 26 with 4; 256 rows of 100 tokens
// 37, 33 and 37; 100 ragged rows of up to 300 26, 32 and 28.
constexpr int HEAD_COST = 2;

template <class T> __device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
}
// 16 bytes to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

struct StepKernelArgs {
  AttnArgs a;
  int32_t ctas, hgroups, orows;        // orows: query heads of a product that exist, at most
  int32_t* desc;                       // [ctas][4] per CTA: the head it is the first of several for
  float* parts;                        // [2 ctas]: o [orows][D], then reference and sum [orows][2]
};
// Floats of a part: its vectors stay aligned.
__host__ __device__ inline int part_size(int orows, int D) { return orows * D + ((2 * orows + 3) & ~3); }

// Ring of stages: 16 rows of K, 16 of V, of D values.  As many as keep some 128 KB on their way on an SM, with CTAS of them
// there.  Fewer fit where the rest of a CTA's memory grows: 12 bytes a row of the call and 4 (D + 8) a query head.  With
// 4 query heads a head of keys that begins behind 306 rows (heads of 64: three CTAs instead of four) and 818 rows (heads of
// 128: one instead of two), with 16 behind 18 and 274.  The parts then run in two waves: 512 rows of 2048 tokens over 2
// heads of 128 take 166 us with 4 query heads each, 251 with 16; over 4 of 64 235 and 252; 1024 rows over 2 of 128 459.
template <int D> struct Cfg {
  static constexpr int STAGES = 3, CTAS = D == 64 ? 4 : D == 128 ? 2 : 1;
  static constexpr uint32_t HALF = KT * D * 2, STAGE = 2 * HALF;
  static constexpr uint32_t RING = NW * STAGES * STAGE;
  // Heads of 256: the queries wait in shared memory (in registers they would spill), where o is summed later.
  static constexpr bool Q_SHARED = D == 256;
  static constexpr int OS = D + 8;     // its rows: eight of them share no banks
  __host__ __device__ static constexpr int obuf(int orows) {
    return Q_SHARED && orows * OS < ROWS * D / 2 ? ROWS * D / 2 : orows * OS;
  }
  static constexpr int QBUF = Q_SHARED ? 0 : ROWS * D / 2;   // the queries on their way to registers
  static size_t smem(int n, int orows) { return RING + 4 * ((size_t)QBUF + obuf(orows) + 2 * RED + 3 * (size_t)n); }
};

// The block list, walked: block b of the `count` of a head (row, gh), which starts at x of the list.
struct Walk {
  int row, gh, b, count;
  Blocks bl;
  int slot, pos;
  int64_t x;
};

// The reference that weights are taken against: fp16 weights are kept 2^7 up, so that those of 2^-21 are still normal
// numbers (at most 2^15: in range).
template <class T> constexpr float LIFT = 0.f;
template <> constexpr float LIFT<__half> = 7.f;

template <class T, int D>
__global__ void __launch_bounds__(THREADS, Cfg<D>::CTAS) step_kernel(const __grid_constant__ StepKernelArgs g) {
  extern __shared__ __align__(128) unsigned char sm[];
  using C = Cfg<D>;
  const AttnArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, n = a.n, per = a.H / a.G, units = a.G * g.hgroups;
  float* obuf = reinterpret_cast<float*>(sm + C::RING) + C::QBUF;   // [orows][OS]
  float* red = obuf + C::obuf(g.orows);                             // two of [NW + 1][ROWS][2], in turns
  int32_t* slots = reinterpret_cast<int32_t*>(red + 2 * RED);       // [n]
  int32_t* lens = slots + n;                                        // [n]
  int32_t* pre = lens + n;                                          // [n]: blocks of a head of the rows before
  __shared__ int32_t wsum[2 * NW];
  pdl_launch_dependents();

  // ---- sums of the rows' blocks: rows tid * each ... of this thread
  const int each = (n + THREADS - 1) / THREADS;
  int sum = 0, live = 0;
  for (int k = 0; k < each; ++k) {
    const int i = tid * each + k;
    if (i >= n) break;
    int s = a.slots[i], len = 0;
    if (s < 0 || s >= a.num_slots) {
      if (blockIdx.x == 0) atomicCAS(&g_step_status, 0, DEV_BAD_SLOT);
      s = -1;
    } else {
      len = a.lengths[s];
      if (len < 0 || len > (a.max_pages << a.page_shift)) {
        if (blockIdx.x == 0) atomicCAS(&g_step_status, 0, DEV_BAD_LENGTH);
        len = min(max(len, 0), a.max_pages << a.page_shift);
      }
    }
    slots[i] = s;
    lens[i] = len;
    sum += blocks_of<BK>(a, len - 1, len - 1).count;
    live += len > 0;
  }
  int run = sum, rows = live;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, o), w = __shfl_up_sync(0xffffffffu, rows, o);
    if (lane >= o) {
      run += v;
      rows += w;
    }
  }
  if (lane == 31) {
    wsum[warp] = run;
    wsum[NW + warp] = rows;
  }
  __syncthreads();
  int before = run - sum, rows_before = rows - live, all = 0, all_rows = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) {
      before += wsum[w];
      rows_before += wsum[NW + w];
    }
    all += wsum[w];
    all_rows += wsum[NW + w];
  }
  const int cost = (int64_t)all * units >= (int64_t)(HEAD_COST + 2) * g.ctas ? HEAD_COST : 0;
  before += cost * rows_before;
  for (int k = 0; k < each && tid * each + k < n; ++k) {
    const int len = lens[tid * each + k];
    pre[tid * each + k] = before;
    if (len > 0) before += blocks_of<BK>(a, len - 1, len - 1).count + cost;
  }
  __syncthreads();

  // Rows of length zero give zero.
  auto out_at = [&](int row, int gh, int h) {
    return static_cast<T*>(a.o) + (int64_t)row * a.o_sn + ((int64_t)(gh / g.hgroups) * per + (gh % g.hgroups) * ROWS + h) * a.d;
  };
  if (all_rows < n)
    for (int i = blockIdx.x; i < n; i += g.ctas)
      if (lens[i] == 0 && slots[i] >= 0)
        for (int e = tid; e < a.H * a.d; e += THREADS) static_cast<T*>(a.o)[(int64_t)i * a.o_sn + e] = from_f<T>(0.f);

  // The CTA's part [w0, w1) of the list.  Block 0 of a head takes 1 + cost of it, the others 1; a block is the CTA's in
  // whose part it starts.  Parts are longer than cost, so every CTA has a block.
  const int64_t total = ((int64_t)all + (int64_t)cost * all_rows) * units;
  const int ctas = (int)min((int64_t)g.ctas, total);
  if (tid == 0) g.desc[4 * blockIdx.x] = -1;
  if ((int)blockIdx.x >= ctas) return;
  const int64_t w0 = total * blockIdx.x / ctas, w1 = total * (blockIdx.x + 1) / ctas;

  auto enter = [&](Walk& w) {           // the head's row is set: what its token sees
    w.slot = slots[w.row];
    w.pos = lens[w.row] - 1;
    w.bl = blocks_of<BK>(a, w.pos, w.pos);
    w.count = w.bl.count;
  };
  auto next = [&](Walk& w) {
    w.x += w.b == 0 ? 1 + cost : 1;
    if (++w.b < w.count) return;
    w.b = 0;
    if (++w.gh == units) {
      w.gh = 0;
      do ++w.row; while (w.row < n && lens[w.row] == 0);
      if (w.row < n) enter(w);
    }
  };
  Walk c;                               // where the products are
  {
    int lo = 0, hi = n - 1;             // the last row that starts at or before w0: one that has blocks
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)pre[mid] * units <= w0) lo = mid; else hi = mid - 1;
    }
    c.row = lo;
    enter(c);
    const int64_t start = (int64_t)pre[lo] * units;
    c.gh = (int)((w0 - start) / (c.count + cost));
    const int off = (int)(w0 - start - (int64_t)c.gh * (c.count + cost));
    c.b = off == 0 ? 0 : max(1, off - cost);
    const bool past = c.b >= c.count;   // block 0 of the head before is all that is left of it
    if (past) c.b = c.count - 1;
    c.x = start + (int64_t)c.gh * (c.count + cost) + (c.b == 0 ? 0 : cost + c.b);
    if (past) next(c);
  }
  Walk ld = c;                          // where the loads are

  // ---- loads: this warp's 16 keys of block ld.b; lane: pieces lane % CH ... of rows lane / CH ...
  constexpr int CH = D / 8 < 32 ? D / 8 : 32, RP = 32 / CH, NC = D / 8 / CH;   // pieces and rows a pass, passes a row
  const uint32_t ring = smem_u32(sm) + warp * C::STAGES * C::STAGE;
  const int d8 = a.d >> 3, lr = lane / CH, lc = lane % CH;
  auto key0 = [&](const Walk& w, int b) { return w.bl.at(b) * BK + warp * KT; };
  auto any_seen = [&](const Walk& w, int j0) {
    return j0 <= w.pos && (a.window == 0 || j0 + KT - 1 > w.pos - a.window || j0 < a.sinks);
  };
  auto all_seen = [&](const Walk& w, int j0) {
    return j0 + KT - 1 <= w.pos && (a.window == 0 || j0 > w.pos - a.window || j0 + KT <= a.sinks);
  };
  // The pages of this warp's keys in up to 32 blocks from ld's on, a lane each.
  int ids = 0, ids_b = 0;
  auto look_up = [&]() {
    ids_b = ld.b;
    const int b = ld.b + lane, j0 = key0(ld, b);
    ids = b < ld.count && any_seen(ld, j0) ? a.table[(int64_t)ld.slot * a.table_stride + (j0 >> a.page_shift)] : 0;
  };
  auto load = [&](int stage) {
    const int j0 = key0(ld, ld.b);
    int id = __shfl_sync(0xffffffffu, ids, ld.b - ids_b);
    if (!any_seen(ld, j0)) return;
    if ((unsigned)id >= (unsigned)a.num_pages) {
      if (lane == 0) atomicCAS(&g_step_status, 0, DEV_BAD_PAGE);
      id = 0;
    }
    const int off = j0 & ((1 << a.page_shift) - 1), gk = g.hgroups == 1 ? ld.gh : ld.gh / g.hgroups;
    const T* k = static_cast<const T*>(a.kp.p) + (id * a.kp.sp + gk * a.kp.sg + (off + lr) * a.kp.st);
    const T* v = static_cast<const T*>(a.vp.p) + (id * a.vp.sp + gk * a.vp.sg + (off + lr) * a.vp.st);
    const uint32_t dst = ring + stage * C::STAGE;
    const bool whole = all_seen(ld, j0) && d8 == D / 8;
#pragma unroll
    for (int r0 = 0; r0 < KT; r0 += RP) {
      const int r = r0 + lr;
#pragma unroll
      for (int p = 0; p < NC; ++p) {
        const int ch = p * CH + lc;
        const uint32_t to = dst + r * (D * 2) + ((ch ^ (r & 7)) << 4);
        const bool got = whole || (sees(a, ld.pos, j0 + r) && ch < d8);
        copy16(to, got ? k + ch * 8 : static_cast<const T*>(a.kp.p), got);
        copy16(to + C::HALF, got ? v + ch * 8 : static_cast<const T*>(a.vp.p), got);
      }
      k += RP * a.kp.st;
      v += RP * a.vp.st;
    }
  };
  auto advance = [&]() {                // the loads' walk; the pages of what comes are looked up a step ahead
    const int row = ld.row, gh = ld.gh;
    next(ld);
    if (ld.x < w1 && (ld.gh != gh || ld.row != row || ld.b - ids_b == 32)) look_up();
  };
  // ---- this thread's part of the products: rows lane / 4 and 8 more, pairs of columns lane % 4
  uint32_t q[C::Q_SHARED ? 1 : D / 16][4];
  unsigned char* const qs = C::Q_SHARED ? reinterpret_cast<unsigned char*>(obuf) : sm + C::RING;
  const uint32_t qb = smem_u32(qs);
  constexpr int QP = ROWS * D / 8 / THREADS;        // 16-byte pieces of the queries a thread
  uint4 qv[QP];
  auto ask = [&](const Walk& w) {       // a head's queries, zeros where there are none
    const int hg = g.hgroups == 1 ? 0 : w.gh % g.hgroups, heads = per - hg * ROWS;
    const int gk = g.hgroups == 1 ? w.gh : w.gh / g.hgroups;
    const T* base = static_cast<const T*>(a.q) + (int64_t)w.row * a.q_sn + ((int64_t)gk * per + hg * ROWS) * a.d;
#pragma unroll
    for (int p = 0; p < QP; ++p) {
      const int e = tid + p * THREADS, h = e / (D / 8), ch = e % (D / 8);
      qv[p] = make_uint4(0u, 0u, 0u, 0u);
      if (h < heads && ch < d8) qv[p] = *reinterpret_cast<const uint4*>(base + h * a.d + 8 * ch);
    }
  };
  auto put = [&]() {
#pragma unroll
    for (int p = 0; p < QP; ++p) {
      const int e = tid + p * THREADS, h = e / (D / 8), ch = e % (D / 8);
      *reinterpret_cast<uint4*>(qs + h * (D * 2) + ((ch ^ (h & 7)) << 4)) = qv[p];
    }
  };
  auto take = [&]() {                   // (after a barrier)
    if constexpr (!C::Q_SHARED) {
#pragma unroll
      for (int k = 0; k < D / 16; ++k) ldsm4(q[k], qb + (lane & 15) * (D * 2) + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
    }
  };
  float m[2], l[2], o[D / 8][4];
  auto empty = [&]() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 8; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
  };

  look_up();
  ask(c);
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) {
    if (ld.x < w1) {
      load(s);
      advance();
    }
    copy_commit();
  }
  empty();
  put();
  __syncthreads();
  take();
  int first = c.b, seg = 0;             // the segment's first block; segments before it
  int at = 0;                           // c's stage
  for (;;) {
    copy_wait<C::STAGES - 2>();
    __syncwarp();                       // the stage has landed for every lane, and the one before is read
    if (ld.x < w1) {
      load(at == 0 ? C::STAGES - 1 : at - 1);
      advance();
    }
    copy_commit();

    const int j0 = key0(c, c.b);
    if (any_seen(c, j0)) {
      const uint32_t kb = ring + at * C::STAGE;
      float s[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[0][e] = s[1][e] = 0.f;
      const int kr = (lane & 7) + ((lane >> 4) << 3), kc = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm4(b, kb + kr * (D * 2) + (((2 * k + kc) ^ (kr & 7)) << 4));
        if constexpr (C::Q_SHARED) ldsm4(q[0], qb + (lane & 15) * (D * 2) + (((2 * k + (lane >> 4)) ^ (lane & 7)) << 4));
        mma16816<T>(s[0], q[C::Q_SHARED ? 0 : k], b[0], b[1]);
        mma16816<T>(s[1], q[C::Q_SHARED ? 0 : k], b[2], b[3]);
      }
      const bool whole = all_seen(c, j0);
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[t][e] *= a.scale_log2;
          if (!whole && !sees(a, c.pos, j0 + 8 * t + 2 * (lane & 3) + (e & 1))) s[t][e] = -INFINITY;
          top[e >> 1] = fmaxf(top[e >> 1], s[t][e]);
        }
      // a new reference where a score passes the old one by more than 2^8
      if (__any_sync(0xffffffffu, top[0] > m[0] + 8.f + LIFT<T> || top[1] > m[1] + 8.f + LIFT<T>)) {
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
          top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
          const float was = m[r];
          m[r] = fmaxf(was, top[r] - LIFT<T>);
          f[r] = mx::ex2_f(was - held(m[r]));
          l[r] *= f[r];
        }
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[k][e] *= f[e >> 1];
      }
      const float base[2] = {held(m[0]), held(m[1])};
      uint32_t p[4];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[t][e] = mx::ex2_f(s[t][e] - base[e >> 1]);
          l[e >> 1] += s[t][e];
        }
        p[2 * t] = pack2<T>(s[t][0], s[t][1]);
        p[2 * t + 1] = pack2<T>(s[t][2], s[t][3]);
      }
      const int vr = lane & 15, vc = lane >> 4;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        uint32_t b[4];
        ldsm4t(b, kb + C::HALF + vr * (D * 2) + (((2 * k + vc) ^ (vr & 7)) << 4));
        mma16816<T>(o[2 * k], p, b[0], b[1]);
        mma16816<T>(o[2 * k + 1], p, b[2], b[3]);
      }
    }
    at = at == C::STAGES - 1 ? 0 : at + 1;
    Walk cn = c;
    next(cn);
    const bool unit_ends = c.b + 1 == c.count, more = cn.x < w1;
    if (!unit_ends && more) {
      c.b = cn.b;
      c.x = cn.x;
      continue;
    }

    // ---- the segment ends: the four warps' parts become one, a quarter of the columns at a time and warp
    const bool whole_unit = first == 0 && unit_ends;
    const int heads = min(g.orows, per - (c.gh % g.hgroups) * ROWS);
    float* rd = red + (seg & 1) * RED;
    if (more) ask(cn);                  // on their way meanwhile
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if ((lane & 3) == 0) {
        float* to = rd + 2 * (warp * ROWS + lane / 4 + 8 * r);
        to[0] = m[r];
        to[1] = l[r];
      }
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float* from = rd + 2 * (lane / 4 + 8 * r);
      float ref = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) ref = fmaxf(ref, from[2 * ROWS * w]);
      f[r] = mx::ex2_f(m[r] - held(ref));
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float lw = from[2 * ROWS * w + 1];
        if (lw != 0.f) L = fmaf(lw, mx::ex2_f(from[2 * ROWS * w] - held(ref)), L);
      }
      if (warp == 0 && (lane & 3) == 0) {
        rd[2 * (NW * ROWS + lane / 4 + 8 * r)] = ref;
        rd[2 * (NW * ROWS + lane / 4 + 8 * r) + 1] = L;
      }
    }
    if (!C::Q_SHARED && more) put();    // (the barrier above is behind this head's own)
#pragma unroll 1
    for (int w = 0; w < NW; ++w) {
      const int part = (warp + w) & (NW - 1);
#pragma unroll
      for (int k = 0; k < D / 8; ++k) {
        if (k / (D / 8 / NW) != part) continue;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int h = lane / 4 + 8 * r;
          if (h < heads) {
            float2* to = reinterpret_cast<float2*>(obuf + h * C::OS + 8 * k + 2 * (lane & 3));
            float2 v = make_float2(o[k][2 * r] * f[r], o[k][2 * r + 1] * f[r]);
            if (w > 0) {
              const float2 u = *to;
              v.x += u.x;
              v.y += u.y;
            }
            *to = v;
          }
        }
      }
      __syncthreads();
    }
    rd += 2 * NW * ROWS;
    const int slot_no = 2 * blockIdx.x + (seg == 0 ? 0 : 1);   // the CTA's first segment, or its last
    float* part = g.parts + (int64_t)slot_no * part_size(g.orows, D);
    for (int e = tid; e < heads * (D / 4); e += THREADS) {
      const int h = e / (D / 4), x = 4 * (e - h * (D / 4));
      const float4 v = *reinterpret_cast<const float4*>(obuf + h * C::OS + x);
      if (whole_unit) {
        const float sum_l = rd[2 * h + 1], inv = 1.f / sum_l;
        if (x < a.d) {
          uint2 w = make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
          if (sum_l == 0.f) w = make_uint2(0u, 0u);
          *reinterpret_cast<uint2*>(out_at(c.row, c.gh, h) + x) = w;
        }
      } else {
        *reinterpret_cast<float4*>(part + h * D + x) = v;
      }
    }
    if (!whole_unit && tid < heads) {
      part[g.orows * D + 2 * tid] = rd[2 * tid];
      part[g.orows * D + 2 * tid + 1] = rd[2 * tid + 1];
    }
    if (tid == 0 && first == 0 && !unit_ends) {      // the first of several CTAs: the last one has the last block
      const int64_t last = c.x + (c.b == 0 ? cost : 0) + (c.count - 1 - c.b);
      int32_t* to = g.desc + 4 * blockIdx.x;
      to[1] = c.gh;
      to[2] = (int32_t)(((last + 1) * ctas - 1) / total);
      to[3] = slot_no;
      to[0] = c.row;
    }
    if (!more) return;
    if (C::Q_SHARED) {
      __syncthreads();                  // o is read from where the queries go
      put();
      __syncthreads();
    }
    take();
    c = cn;
    first = c.b;
    ++seg;
    empty();
  }
}

// The heads that several CTAs share, from the first of those CTAs: block (first CTA, query head).  Up to JOIN_FEW parts
// one block does all query heads, a warp each; more are taken by the 16 warps of a block a query head in turns, and
// their sums added in order.
constexpr int JOIN_FEW = 4, JW = ROWS;      // 1 x 512 tokens (8 parts a head): 8.5 us, 10.2 with 8
template <class T, int D>
__global__ void __launch_bounds__(32 * JW) step_join(const __grid_constant__ StepKernelArgs g) {
  __shared__ float4 o_of[JW][D / 4];
  __shared__ float l_of[JW];
  const AttnArgs& a = g.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait_primary();
  const int4 d = *reinterpret_cast<const int4*>(g.desc + 4 * blockIdx.x);
  if (d.x < 0) return;
  const int per = a.H / a.G, h0 = (d.y % g.hgroups) * ROWS, parts = d.z - (int)blockIdx.x + 1;
  const bool few = parts <= JOIN_FEW;
  const int h = few ? warp : blockIdx.y, step = few ? 1 : JW;
  if (few ? blockIdx.y > 0 : h0 + h >= per) return;
  const bool mine = h < g.orows && h0 + h < per;
  auto part_at = [&](int k) {           // the first CTA's part, then the first parts of those after it
    return g.parts + (int64_t)(k == 0 ? d.w : 2 * ((int)blockIdx.x + k)) * part_size(g.orows, D);
  };
  constexpr int V = D / 4 < 32 ? 1 : D / 128;       // float4 pieces of a lane
  float4 o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  if (mine) {
    float top = -INFINITY;
    for (int k = lane; k < parts; k += 32) top = fmaxf(top, part_at(k)[g.orows * D + 2 * h]);
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float base = held(top);
#pragma unroll 4
    for (int k = few ? 0 : warp; k < parts; k += step) {
      const float* p = part_at(k);
      const float2 ml = *reinterpret_cast<const float2*>(p + g.orows * D + 2 * h);
      const float f = ml.y == 0.f ? 0.f : mx::ex2_f(ml.x - base);
      l = fmaf(ml.y, f, l);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (4 * (32 * v + lane) < D) {
          const float4 x = *reinterpret_cast<const float4*>(p + h * D + 4 * (32 * v + lane));
          o[v].x = fmaf(x.x, f, o[v].x);
          o[v].y = fmaf(x.y, f, o[v].y);
          o[v].z = fmaf(x.z, f, o[v].z);
          o[v].w = fmaf(x.w, f, o[v].w);
        }
    }
  }
  if (!few) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (4 * (32 * v + lane) < D) o_of[warp][32 * v + lane] = o[v];
    if (lane == 0) l_of[warp] = l;
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < JW; ++w) l += l_of[w];
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (4 * (32 * v + lane) < D)
#pragma unroll
        for (int w = 1; w < JW; ++w) {
          const float4 x = o_of[w][32 * v + lane];
          o[v].x += x.x;
          o[v].y += x.y;
          o[v].z += x.z;
          o[v].w += x.w;
        }
  }
  if (!mine) return;
  const float inv = 1.f / l;
  T* out = static_cast<T*>(a.o) + (int64_t)d.x * a.o_sn + ((int64_t)(d.y / g.hgroups) * per + h0 + h) * a.d;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int x = 4 * (32 * v + lane);
    if (x >= a.d) continue;
    uint2 w = make_uint2(pack2<T>(o[v].x * inv, o[v].y * inv), pack2<T>(o[v].z * inv, o[v].w * inv));
    if (l == 0.f) w = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(out + x) = w;
  }
}

template <class T, int D>
cudaError_t go(StepKernelArgs& g, const AttnPlan& p, cudaStream_t s) {
  static thread_local int ready = -1;  // the device whose limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready != dev) {
    e = cudaFuncSetAttribute(step_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)Cfg<D>::smem(AT_ROWS, ROWS));
    if (e != cudaSuccess) return e;
    ready = dev;
  }
  step_kernel<T, D><<<g.ctas, THREADS, Cfg<D>::smem(g.a.n, g.orows), s>>>(g);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.gridDim = dim3((unsigned)g.ctas, (unsigned)g.orows);
  c.blockDim = dim3(32 * JW);
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, step_join<T, D>, g);
}
int width_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

}  // namespace

// 16-bit types with 16-byte aligned tensors and strides, while the blocks of all rows are counted in 32 bits.
bool step_fits(int dtype, bool vec, const AttnArgs& a) {
  const int64_t blocks = ((int64_t)a.max_pages << a.page_shift) / BK + 2;
  return dtype != mx::T_F32 && vec && (int64_t)a.n * blocks < 0x7fffffff;
}

AttnPlan step_plan(int n, int H, int G, int d, int sms) {
  AttnPlan p{};
  const int per = H / G, D = width_of(d);
  p.rows = per < ROWS ? per : ROWS;
  p.hgroups = (per + ROWS - 1) / ROWS;
  p.grid = sms * (D == 64 ? Cfg<64>::CTAS : D == 128 ? Cfg<128>::CTAS : Cfg<256>::CTAS);
  p.ws_bytes = 16 * (int64_t)p.grid + 2 * (int64_t)p.grid * part_size(p.rows, D) * 4;
  return p;
}

cudaError_t launch_step(int dtype, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  StepKernelArgs g{a, p.grid, p.hgroups, p.rows, reinterpret_cast<int32_t*>(a.ws), a.ws + 4 * (int64_t)p.grid};
  const int D = width_of(a.d);
  if (dtype == mx::T_BF16)
    return D == 64 ? go<__nv_bfloat16, 64>(g, p, s) : D == 128 ? go<__nv_bfloat16, 128>(g, p, s) : go<__nv_bfloat16, 256>(g, p, s);
  return D == 64 ? go<__half, 64>(g, p, s) : D == 128 ? go<__half, 128>(g, p, s) : go<__half, 256>(g, p, s);
}

cudaError_t read_step_status(cudaStream_t s, int32_t* code) { return take_status(g_step_status, s, code); }

}  // namespace at
}  // namespace dl
