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
// more), so it looks up one page, a step ahead, and copies 16 rows of K and of V
// asynchronously into its own ring of stages, which no other warp reads: no
// barriers but where a head ends.
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

// Ring of stages: 16 rows of K, 16 of V, of D values.  As many as keep some 128 KB on their way on an SM.
template <int D> struct Cfg {
  static constexpr int STAGES = D == 64 ? 6 : 3, CTAS = D == 256 ? 1 : 2;
  static constexpr uint32_t HALF = KT * D * 2, STAGE = 2 * HALF;
  static constexpr uint32_t RING = NW * STAGES * STAGE;
  // Heads of 256: the queries wait in shared memory (in registers they would spill), where o is summed later.
  static constexpr bool Q_SHARED = D == 256;
  __host__ __device__ static constexpr int obuf(int orows) {
    return Q_SHARED && orows * D < ROWS * D / 2 ? ROWS * D / 2 : orows * D;
  }
  static size_t smem(int n, int orows) { return RING + 4 * ((size_t)obuf(orows) + 2 * NW * ROWS + 3 * (size_t)n); }
};

// The block list, walked.
struct Walk {
  int row, gh, b, count;               // unit: row and group of heads; its block b of count
  Blocks bl;
  int slot, pos;
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
  float* obuf = reinterpret_cast<float*>(sm + C::RING);             // [orows][D]
  float* red = obuf + C::obuf(g.orows);                             // [NW][ROWS][2]
  int32_t* slots = reinterpret_cast<int32_t*>(red + 2 * NW * ROWS); // [n]
  int32_t* lens = slots + n;                                        // [n]
  int32_t* pre = lens + n;                                          // [n]: blocks of a head of the rows before, and of row n
  __shared__ int32_t wsum[NW + 1];
  pdl_launch_dependents();

  // ---- sums of the rows' blocks: rows tid * each ... of this thread
  const int each = (n + THREADS - 1) / THREADS;
  int sum = 0;
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
    pre[i] = sum;
    sum += blocks_of<BK>(a, len - 1, len - 1).count;
  }
  int run = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += v;
  }
  if (lane == 31) wsum[warp] = run;
  __syncthreads();
  int before = run - sum, all = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += wsum[w];
    all += wsum[w];
  }
  for (int k = 0; k < each && tid * each + k < n; ++k) pre[tid * each + k] += before;
  __syncthreads();

  // Rows of length zero (and of a slot out of range) give zero.
  auto out_at = [&](int row, int gh, int h) {
    return static_cast<T*>(a.o) + (int64_t)row * a.o_sn + ((int64_t)(gh / g.hgroups) * per + (gh % g.hgroups) * ROWS + h) * a.d;
  };
  for (int i = blockIdx.x; i < n; i += g.ctas)
    if ((i + 1 < n ? pre[i + 1] : all) == pre[i] && slots[i] >= 0)
      for (int e = tid; e < a.H * a.d; e += THREADS)
        static_cast<T*>(a.o)[(int64_t)i * a.o_sn + e] = from_f<T>(0.f);

  const int64_t total = (int64_t)all * units;
  const int ctas = (int)min((int64_t)g.ctas, total);                // each has a block at least
  if (tid == 0) g.desc[4 * blockIdx.x] = -1;
  if ((int)blockIdx.x >= ctas) return;
  const int64_t w0 = total * blockIdx.x / ctas, w1 = total * (blockIdx.x + 1) / ctas;
  const int count = (int)(w1 - w0);

  auto enter = [&](Walk& w) {           // the unit's row is set: what its token sees
    w.slot = slots[w.row];
    w.pos = lens[w.row] - 1;
    w.bl = blocks_of<BK>(a, w.pos, w.pos);
    w.count = w.bl.count;
  };
  auto next = [&](Walk& w) {
    if (++w.b < w.count) return;
    w.b = 0;
    if (++w.gh == units) {
      w.gh = 0;
      do ++w.row; while (w.row + 1 < n && pre[w.row + 1] == pre[w.row]);
      if (w.row < n) enter(w);
    }
  };
  Walk c;                               // where the products are
  {
    int lo = 0, hi = n - 1;             // the last row whose blocks start at or before w0
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((int64_t)pre[mid] * units <= w0) lo = mid; else hi = mid - 1;
    }
    c.row = lo;
    enter(c);
    const int64_t off = w0 - (int64_t)pre[lo] * units;
    c.gh = (int)(off / c.count);
    c.b = (int)(off - (int64_t)c.gh * c.count);
  }
  Walk ld = c;                          // where the loads are

  // ---- loads: this warp's 16 keys of block ld.b; lane: pieces lane % CH ... of rows lane / CH ...
  constexpr int CH = D / 8 < 32 ? D / 8 : 32, RP = 32 / CH, NC = D / 8 / CH;   // pieces and rows a pass, passes a row
  const uint32_t ring = smem_u32(sm) + warp * C::STAGES * C::STAGE;
  const int d8 = a.d >> 3;
  auto key0 = [&](const Walk& w) { return w.bl.at(w.b) * BK + warp * KT; };
  auto any_seen = [&](const Walk& w, int j0) {
    return j0 <= w.pos && (a.window == 0 || j0 + KT - 1 > w.pos - a.window || j0 < a.sinks);
  };
  int id = 0;                           // the page of ld's keys
  auto look_up = [&]() {
    const int j0 = key0(ld);
    if (any_seen(ld, j0)) id = a.table[(int64_t)ld.slot * a.table_stride + (j0 >> a.page_shift)];
  };
  auto load = [&](int stage) {
    const int j0 = key0(ld);
    if (!any_seen(ld, j0)) return;
    if ((unsigned)id >= (unsigned)a.num_pages) {
      if (lane == 0) atomicCAS(&g_step_status, 0, DEV_BAD_PAGE);
      id = 0;
    }
    const int off = j0 & ((1 << a.page_shift) - 1), gk = ld.gh / g.hgroups;
    const T* k = static_cast<const T*>(a.kp.p) + id * a.kp.sp + gk * a.kp.sg + off * a.kp.st;
    const T* v = static_cast<const T*>(a.vp.p) + id * a.vp.sp + gk * a.vp.sg + off * a.vp.st;
    const bool whole = j0 + KT - 1 <= ld.pos && (a.window == 0 || j0 > ld.pos - a.window || j0 + KT <= a.sinks);
    const uint32_t dst = ring + stage * C::STAGE;
#pragma unroll
    for (int r0 = 0; r0 < KT; r0 += RP) {
      const int r = r0 + lane / CH;
      const bool seen = whole || sees(a, ld.pos, j0 + r);
#pragma unroll
      for (int p = 0; p < NC; ++p) {
        const int ch = p * CH + lane % CH;
        const bool live = seen && ch < d8;
        const uint32_t to = dst + r * (D * 2) + ((ch ^ (r & 7)) << 4);
        copy16(to, live ? k + r * a.kp.st + ch * 8 : k, live);
        copy16(to + C::HALF, live ? v + r * a.vp.st + ch * 8 : v, live);
      }
    }
  };
  // ---- this thread's part of the products: rows lane / 4 and 8 more, pairs of columns lane % 4
  uint32_t q[C::Q_SHARED ? 1 : D / 16][4];
  const uint32_t qb = smem_u32(obuf);
  float m[2], l[2], o[D / 8][4];
  auto begin = [&]() {                  // the unit's queries (zeros where there are none), an empty softmax
    const T* base = static_cast<const T*>(a.q) + (int64_t)c.row * a.q_sn + ((int64_t)(c.gh / g.hgroups) * per + (c.gh % g.hgroups) * ROWS) * a.d;
    const int heads = per - (c.gh % g.hgroups) * ROWS;
    if constexpr (C::Q_SHARED) {
      for (int e = tid; e < ROWS * D / 8; e += THREADS) {
        const int h = e / (D / 8), ch = e - h * (D / 8);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (h < heads && ch < d8) v = *reinterpret_cast<const uint4*>(base + h * a.d + 8 * ch);
        *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(obuf) + h * (D * 2) + ((ch ^ (h & 7)) << 4)) = v;
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = lane / 4 + 8 * (e & 1), x = 16 * k + 8 * (e >> 1) + 2 * (lane & 3);
          q[k][e] = h < heads && x < a.d ? *reinterpret_cast<const uint32_t*>(base + h * a.d + x) : 0u;
        }
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int k = 0; k < D / 8; ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[k][e] = 0.f;
  };

  look_up();
#pragma unroll
  for (int s = 0; s < C::STAGES - 1; ++s) {
    if (s < count) {
      load(s);
      next(ld);
      if (s + 1 < count) look_up();
    }
    copy_commit();
  }
  begin();
  int first = c.b;                      // the segment's first block
  for (int i = 0; i < count; ++i) {
    copy_wait<C::STAGES - 2>();
    __syncwarp();                       // stage i has landed for every lane, and stage i - 1 is read
    if (i + C::STAGES - 1 < count) {
      load((i + C::STAGES - 1) % C::STAGES);
      next(ld);
      if (i + C::STAGES < count) look_up();
    }
    copy_commit();

    const int j0 = key0(c);
    if (any_seen(c, j0)) {
      const uint32_t kb = ring + (i % C::STAGES) * C::STAGE;
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
      const bool whole = j0 + KT - 1 <= c.pos && (a.window == 0 || j0 > c.pos - a.window || j0 + KT <= a.sinks);
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
    const bool unit_ends = c.b + 1 == c.count;
    if (!unit_ends && i + 1 < count) {
      ++c.b;
      continue;
    }

    // ---- the segment ends: the four warps' parts become one
    const bool whole_unit = first == 0 && unit_ends;
    const int heads = min(g.orows, per - (c.gh % g.hgroups) * ROWS);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if ((lane & 3) == 0) {
        float* to = red + 2 * (warp * ROWS + lane / 4 + 8 * r);
        to[0] = m[r];
        to[1] = l[r];
      }
    }
    __syncthreads();
    float f[2], ref[2], L[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float* from = red + 2 * (lane / 4 + 8 * r);
      ref[r] = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) ref[r] = fmaxf(ref[r], from[2 * ROWS * w]);
      f[r] = mx::ex2_f(m[r] - held(ref[r]));
      L[r] = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float lw = from[2 * ROWS * w + 1];
        if (lw != 0.f) L[r] = fmaf(lw, mx::ex2_f(from[2 * ROWS * w] - held(ref[r])), L[r]);
      }
    }
#pragma unroll 1
    for (int w = 0; w < NW; ++w) {
      if (warp == w) {
#pragma unroll
        for (int k = 0; k < D / 8; ++k)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int h = lane / 4 + 8 * r;
            if (h < heads) {
              float2* to = reinterpret_cast<float2*>(obuf + h * D + 8 * k + 2 * (lane & 3));
              float2 v = make_float2(o[k][2 * r] * f[r], o[k][2 * r + 1] * f[r]);
              if (w > 0) {
                v.x += to->x;
                v.y += to->y;
              }
              *to = v;
            }
          }
      }
      __syncthreads();
    }
    if (warp == 0 && (lane & 3) == 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        red[2 * (lane / 4 + 8 * r)] = ref[r];
        red[2 * (lane / 4 + 8 * r) + 1] = L[r];
      }
    }
    __syncthreads();
    const int slot_no = 2 * blockIdx.x + (i + 1 - (c.b + 1 - first) == 0 ? 0 : 1);   // the CTA's first segment, or its last
    float* part = g.parts + (int64_t)slot_no * part_size(g.orows, D);
    for (int e = tid; e < heads * (D / 4); e += THREADS) {
      const int h = e / (D / 4), x = 4 * (e - h * (D / 4));
      float4 v = *reinterpret_cast<const float4*>(obuf + h * D + x);
      if (whole_unit) {
        const float sum_l = red[2 * h + 1], inv = sum_l == 0.f ? 0.f : 1.f / sum_l;
        if (x < a.d) {
          uint2 w;
          w.x = sum_l == 0.f ? 0u : pack2<T>(v.x * inv, v.y * inv);
          w.y = sum_l == 0.f ? 0u : pack2<T>(v.z * inv, v.w * inv);
          *reinterpret_cast<uint2*>(out_at(c.row, c.gh, h) + x) = w;
        }
      } else {
        *reinterpret_cast<float4*>(part + h * D + x) = v;
      }
    }
    if (!whole_unit && tid < heads) {
      part[g.orows * D + 2 * tid] = red[2 * tid];
      part[g.orows * D + 2 * tid + 1] = red[2 * tid + 1];
    }
    if (tid == 0 && first == 0 && !unit_ends) {      // the first of several CTAs: the last one has block `end`
      const int64_t end = ((int64_t)pre[c.row] * units + (int64_t)(c.gh + 1) * c.count);
      int32_t* to = g.desc + 4 * blockIdx.x;
      to[1] = c.gh;
      to[2] = (int32_t)((end * ctas - 1) / total);
      to[3] = slot_no;
      to[0] = c.row;
    }
    __syncthreads();                    // obuf and red are read
    if (i + 1 < count) {
      next(c);
      first = c.b;
      begin();
    }
  }
}

// A head that several CTAs share: block (first CTA, query head); warps take its parts in turns, then the four sums are
// added in order.
template <class T, int D>
__global__ void __launch_bounds__(THREADS) step_join(const __grid_constant__ StepKernelArgs g) {
  __shared__ float4 o_of[NW][D / 4];
  __shared__ float l_of[NW];
  const AttnArgs& a = g.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  pdl_wait_primary();
  const int4 d = *reinterpret_cast<const int4*>(g.desc + 4 * blockIdx.x);
  if (d.x < 0) return;
  const int per = a.H / a.G, h0 = (d.y % g.hgroups) * ROWS;
  if (h0 + h >= per) return;
  const int parts = d.z - (int)blockIdx.x + 1;
  auto part_at = [&](int k) {           // the first CTA's part, then the first parts of those after it
    return g.parts + (int64_t)(k == 0 ? d.w : 2 * ((int)blockIdx.x + k)) * part_size(g.orows, D);
  };
  float top = -INFINITY;
  for (int k = lane; k < parts; k += 32) top = fmaxf(top, part_at(k)[g.orows * D + 2 * h]);
#pragma unroll
  for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float base = held(top);
  constexpr int V = D / 4 < 32 ? 1 : D / 128;       // float4 pieces of a lane
  float4 o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) o[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int k = warp; k < parts; k += NW) {
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
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (4 * (32 * v + lane) < D) o_of[warp][32 * v + lane] = o[v];
  if (lane == 0) l_of[warp] = l;
  __syncthreads();
  const float sum = l_of[0] + l_of[1] + l_of[2] + l_of[3];
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  T* out = static_cast<T*>(a.o) + (int64_t)d.x * a.o_sn + ((int64_t)(d.y / g.hgroups) * per + h0 + h) * a.d;
  for (int x = threadIdx.x; x < D / 4; x += THREADS) {
    if (4 * x >= a.d) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      v.x += o_of[w][x].x;
      v.y += o_of[w][x].y;
      v.z += o_of[w][x].z;
      v.w += o_of[w][x].w;
    }
    uint2 w = make_uint2(pack2<T>(v.x * inv, v.y * inv), pack2<T>(v.z * inv, v.w * inv));
    if (sum == 0.f) w = make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(out + 4 * x) = w;
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
  c.blockDim = dim3(THREADS);
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
  p.grid = sms * (D == 256 ? Cfg<256>::CTAS : Cfg<128>::CTAS);
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
