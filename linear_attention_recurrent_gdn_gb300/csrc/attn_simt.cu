// Attention of prompts over pages on the FP32 cores: every type, head dimension
// (up to 256), stride and alignment.
//
// A block takes R rows (tokens times the heads that share a head of keys) and
// walks over the keys they see, 32 at a time.  With m the running maximum of a
// row's scores s = scale log2(e) q . k, l the sum of 2^(s - m) and o the sum of
// 2^(s - m) v,
//   m' = max(m, s),  l' = l 2^(m - m') + sum 2^(s - m'),  o' = o 2^(m - m') + sum 2^(s - m') v
// all in fp32; o / l at the end is rounded once.  A row that sees nothing gives zero.
//
// A key that a row does not see has weight zero; where its value is an
// infinity or a NaN the product would still be a NaN, so a block of keys with
// such a value takes the sums that leave masked keys out (MASK_P marks them).
//
// Few tiles: their keys are split over several blocks of the grid, which leave
// (m, l, o) in the workspace, and a second launch joins them.
//
// R = 64: 16 x 16 threads with four rows and two keys (four rows and 4 d / 64
// columns) each, 2 wavefronts of shared memory for 8 multiply-adds of a warp; R =
// 16 where a tile of 64 would be mostly empty.  Bound by shared memory and
// instructions, 16 to 20 TFLOP/s: 4 x 512 tokens of 32 heads of 128 over 8 fp32
// 537 us, one prompt of 2048 1.77 ms (bf16 heads of 100: 551 us, 1.81 ms).  The
// 16-bit types of head dimensions that eight divides run on the tensor cores
// instead.
#include <cmath>

#include "attn_device.cuh"
#include "mixer_device.cuh"

namespace dl {
namespace at {

static __device__ int32_t g_simt_status;

namespace {

using mx::load8;
using mx::unpack8;
using mx::to_f;
using mx::from_f;
using mx::Vec8;

constexpr int BK = 32, THREADS = 256;
constexpr float MASK_P = -1.f;
constexpr int MIN_BLOCKS = 4;          // blocks of keys that a split is worth

struct SimtArgs {
  AttnArgs a;
  AttnPlan p;
};

__host__ __device__ inline int padded(int d) { return ((d + 3) & ~3) + 4; }
inline size_t smem_bytes(int R, int d) { return sizeof(float) * ((size_t)(R + 2 * BK) * padded(d) + (size_t)R * (BK + 4)); }

template <class T, int R, bool VEC>
__global__ void __launch_bounds__(THREADS) simt_kernel(const __grid_constant__ SimtArgs g) {
  extern __shared__ __align__(16) float sm[];
  constexpr int RPT = R / 16;
  const AttnArgs& a = g.a;
  const int per = a.H / a.G, hpt = min(per, R), tid = threadIdx.x, d = a.d, dp = padded(d), pp = BK + 4;
  const int gh = blockIdx.y / g.p.hgroups, h0 = (blockIdx.y - gh * g.p.hgroups) * R;
  Tile w;
  if (!find_tile(a, gridDim.x - 1 - blockIdx.x, g.p.tpt, w, &g_simt_status)) return;
  const int p1 = w.pos0 + w.nt - 1;
  const Blocks bl = blocks_of<BK>(a, w.pos0, p1);
  const int each = max(MIN_BLOCKS, (bl.count + g.p.splits - 1) / g.p.splits);
  const int b0 = blockIdx.z * each, b1 = min(bl.count, b0 + each);

  float *Q = sm, *K = Q + R * dp, *V = K + BK * dp, *P = V + BK * dp;
  const int rows = w.nt * hpt, heads = min(hpt, per - h0);
  auto token_off = [&](int64_t st, int64_t sn, int t) { return (int64_t)(w.begin + w.t0 + t) * st + (int64_t)w.row * sn; };
  // rows of [valid] values into fp32 rows of dp, zero behind the values
  auto put = [&](float* dst, const T* src, int c, bool live) {
    float f[8];
    unpack8<T>(load8<T, VEC>(src + c, live ? d - c : 0), f);
#pragma unroll
    for (int k = 0; k < 8; k += 4)
      if (c + k < dp) *reinterpret_cast<float4*>(dst + c + k) = make_float4(f[k], f[k + 1], f[k + 2], f[k + 3]);
  };
  const int d8 = (d + 7) / 8;
  for (int e = tid; e < R * d8; e += THREADS) {
    const int r = e / d8, c = 8 * (e - r * d8), t = r / hpt, h = r - t * hpt;
    const bool live = r < rows && h < heads;
    put(Q + r * dp, static_cast<const T*>(a.q) + (live ? token_off(a.q_st, a.q_sn, t) + (int64_t)(gh * per + h0 + h) * d : 0), c, live);
  }

  const int rg = tid >> 4, kg = tid & 15;
  float m[RPT], l[RPT], o[RPT][4][4];
  int pos[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
    pos[r] = w.pos0 + (rg * RPT + r) / hpt;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[r][c][k] = 0.f;
  }

  for (int b = b0; b < b1; ++b) {
    const int j0 = bl.at(b) * BK;
    __syncthreads();                   // the last block's keys are read
    bool odd = false;
    for (int e = tid; e < BK * d8; e += THREADS) {
      const int j = e / d8, c = 8 * (e - j * d8);
      const bool live = !none_sees(a, w.pos0, p1, j0 + j);
      int64_t ko = 0, vo = 0;
      if (live) {
        const int id = page_of(a, w.slot, j0 + j, &g_simt_status), off = (j0 + j) & ((1 << a.page_shift) - 1);
        ko = id * a.kp.sp + gh * a.kp.sg + off * a.kp.st;
        vo = id * a.vp.sp + gh * a.vp.sg + off * a.vp.st;
      }
      put(K + j * dp, static_cast<const T*>(a.kp.p) + ko, c, live);
      put(V + j * dp, static_cast<const T*>(a.vp.p) + vo, c, live);
#pragma unroll
      for (int k = 0; k < 8; ++k) odd |= c + k < d && !(fabsf(V[j * dp + c + k]) < INFINITY);
    }
    const bool full = all_see(a, w.pos0, p1, j0, j0 + BK);
    const bool careful = __syncthreads_or(odd) && !full;

    float s[RPT][2];
#pragma unroll
    for (int r = 0; r < RPT; ++r) s[r][0] = s[r][1] = 0.f;
    for (int c = 0; c < d; c += 4) {
      const float4 k0 = *reinterpret_cast<const float4*>(K + kg * dp + c);
      const float4 k1 = *reinterpret_cast<const float4*>(K + (kg + 16) * dp + c);
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const float4 q = *reinterpret_cast<const float4*>(Q + (rg * RPT + r) * dp + c);
        s[r][0] = fmaf(q.x, k0.x, fmaf(q.y, k0.y, fmaf(q.z, k0.z, fmaf(q.w, k0.w, s[r][0]))));
        s[r][1] = fmaf(q.x, k1.x, fmaf(q.y, k1.y, fmaf(q.z, k1.z, fmaf(q.w, k1.w, s[r][1]))));
      }
    }
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      bool see[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        see[k] = full || sees(a, pos[r], j0 + kg + 16 * k);
        s[r][k] = see[k] ? s[r][k] * a.scale_log2 : -INFINITY;
      }
      float top = fmaxf(m[r], fmaxf(s[r][0], s[r][1]));
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float base = held(top), shrink = exp2f(m[r] - base);
      m[r] = top;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float p = see[k] ? exp2f(s[r][k] - base) : 0.f;
        sum += p;
        P[(rg * RPT + r) * pp + kg + 16 * k] = careful && !see[k] ? MASK_P : p;
      }
#pragma unroll
      for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l[r] = fmaf(l[r], shrink, sum);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[r][c][k] *= shrink;
    }
    __syncwarp();                      // a row's weights are written and read by one half of a warp
    for (int j = 0; j < BK; j += 4) {
      float4 p[RPT];
#pragma unroll
      for (int r = 0; r < RPT; ++r) p[r] = *reinterpret_cast<const float4*>(P + (rg * RPT + r) * pp + j);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int col = 64 * c + 4 * kg;
        if (col >= d) break;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 v = *reinterpret_cast<const float4*>(V + (j + k) * dp + col);
#pragma unroll
          for (int r = 0; r < RPT; ++r) {
            const float x = k == 0 ? p[r].x : k == 1 ? p[r].y : k == 2 ? p[r].z : p[r].w;
            if (careful && x == MASK_P) continue;
            o[r][c][0] = fmaf(x, v.x, o[r][c][0]);
            o[r][c][1] = fmaf(x, v.y, o[r][c][1]);
            o[r][c][2] = fmaf(x, v.z, o[r][c][2]);
            o[r][c][3] = fmaf(x, v.w, o[r][c][3]);
          }
        }
      }
    }
    __syncwarp();
  }

#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const int rr = rg * RPT + r, t = rr / hpt, h = rr - t * hpt;
    if (rr >= rows || h >= heads) continue;
    if (g.p.splits == 1) {
      T* out = static_cast<T*>(a.o) + token_off(a.o_st, a.o_sn, t) + (int64_t)(gh * per + h0 + h) * d;
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (64 * c + 4 * kg + k < d) out[64 * c + 4 * kg + k] = from_f<T>(l[r] == 0.f ? 0.f : o[r][c][k] / l[r]);
    } else {
      const int64_t u = (((int64_t)(gridDim.x - 1 - blockIdx.x) * gridDim.y + blockIdx.y) * g.p.splits + blockIdx.z) * R + rr;
      float* part = a.ws + u * (d + 2);
      if (kg == 0) {
        part[0] = m[r];
        part[1] = l[r];
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (64 * c + 4 * kg + k < d) part[2 + 64 * c + 4 * kg + k] = o[r][c][k];
    }
  }
}

// The splits of a tile's rows, four parts at a time: a warp a row, or, where that is less to do one after the other (few
// rows, many parts), all warps a row, parts in turns and their sums in order.  One part after the other took 0.55 us each.
constexpr int WARPS = THREADS / 32, JOIN_Z = 4;
template <class T>
__global__ void __launch_bounds__(THREADS) simt_join(const __grid_constant__ SimtArgs g) {
  constexpr int C = AT_DIM / 32;
  __shared__ float o_of[WARPS][AT_DIM];
  __shared__ float2 ml_of[WARPS];
  const AttnArgs& a = g.a;
  const int R = g.p.rows, per = a.H / a.G, hpt = min(per, R), d = a.d, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gh = blockIdx.y / g.p.hgroups, h0 = (blockIdx.y - gh * g.p.hgroups) * R;
  pdl_wait_primary();
  Tile w;
  if (!find_tile(a, blockIdx.x, g.p.tpt, w, &g_simt_status)) return;
  const int heads = min(hpt, per - h0), rows = w.nt * heads, parts = g.p.splits, z = gridDim.z;
  const bool share = (rows + z - 1) / z * (parts / WARPS + 4) < (rows + WARPS * z - 1) / (WARPS * z) * parts;
  const int by = share ? WARPS : 1;
  const int64_t next = (int64_t)R * (d + 2);
  for (int e = share ? blockIdx.z : WARPS * blockIdx.z + warp; e < rows; e += share ? z : WARPS * z) {
    const int t = e / heads, h = e - t * heads;
    const float* part = a.ws + (((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * parts * R + t * hpt + h) * (d + 2);
    float m = -INFINITY, l = 0.f, o[C];
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = 0.f;
    for (int k0 = share ? warp : 0; k0 < parts; k0 += 4 * by) {
      float mk[4], lk[4], x[4][C];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = k0 + u * by < parts;
        const float* q = part + (in ? k0 + u * by : 0) * next;
        mk[u] = in ? q[0] : -INFINITY;
        lk[u] = in ? q[1] : 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) x[u][c] = 32 * c + lane < d ? q[2 + 32 * c + lane] : 0.f;
      }
      const float was = m;
      m = fmaxf(fmaxf(m, fmaxf(mk[0], mk[1])), fmaxf(mk[2], mk[3]));
      const float base = held(m), f0 = exp2f(was - base);
      l *= f0;
#pragma unroll
      for (int c = 0; c < C; ++c) o[c] *= f0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (lk[u] == 0.f) continue;      // nothing seen
        const float f = exp2f(mk[u] - base);
        l = fmaf(lk[u], f, l);
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] = fmaf(x[u][c], f, o[c]);
      }
    }
    if (share) {
#pragma unroll
      for (int c = 0; c < C; ++c) o_of[warp][32 * c + lane] = o[c];
      if (lane == 0) ml_of[warp] = make_float2(m, l);
      __syncthreads();
      if (warp == 0) {
        float top = m;
        for (int x = 1; x < WARPS; ++x) top = fmaxf(top, ml_of[x].x);
        const float base = held(top), f0 = exp2f(m - base);
        l *= f0;
#pragma unroll
        for (int c = 0; c < C; ++c) o[c] *= f0;
        for (int x = 1; x < WARPS; ++x) {
          if (ml_of[x].y == 0.f) continue;
          const float f = exp2f(ml_of[x].x - base);
          l = fmaf(ml_of[x].y, f, l);
#pragma unroll
          for (int c = 0; c < C; ++c) o[c] = fmaf(o_of[x][32 * c + lane], f, o[c]);
        }
      }
    }
    if (!share || warp == 0) {
      T* out = static_cast<T*>(a.o) + (int64_t)(w.begin + w.t0 + t) * a.o_st + (int64_t)w.row * a.o_sn + (int64_t)(gh * per + h0 + h) * d;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (32 * c + lane < d) out[32 * c + lane] = from_f<T>(l == 0.f ? 0.f : o[c] / l);
    }
    if (share) __syncthreads();          // the sums are read
  }
}

template <class T>
cudaError_t join(const SimtArgs& g, cudaStream_t s) {
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.gridDim = dim3((unsigned)g.p.tiles, (unsigned)(g.a.G * g.p.hgroups), JOIN_Z);
  c.blockDim = dim3(THREADS);
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, simt_join<T>, g);
}
template <class T, int R, bool VEC>
cudaError_t go(const SimtArgs& g, cudaStream_t s) {
  static thread_local int ready = -1;  // the device whose limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready != dev) {
    e = cudaFuncSetAttribute(simt_kernel<T, R, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes(R, AT_DIM));
    if (e != cudaSuccess) return e;
    ready = dev;
  }
  const dim3 grid((unsigned)g.p.tiles, (unsigned)(g.a.G * g.p.hgroups), (unsigned)g.p.splits);
  simt_kernel<T, R, VEC><<<grid, THREADS, smem_bytes(R, g.a.d), s>>>(g);
  e = cudaGetLastError();
  return e != cudaSuccess || g.p.splits == 1 ? e : join<T>(g, s);
}
template <class T>
cudaError_t pick(bool vec, const SimtArgs& g, cudaStream_t s) {
  if (g.p.rows == 16) return vec ? go<T, 16, true>(g, s) : go<T, 16, false>(g, s);
  return vec ? go<T, 64, true>(g, s) : go<T, 64, false>(g, s);
}

}  // namespace

AttnPlan simt_plan(int n, int T, bool packed, int H, int G, int d, int sms) {
  AttnPlan p{};
  const int per = H / G;
  // Tiles of 16 rows where a tile of 64 would be mostly empty.  fp32, 64 rows of some tokens behind 2048, 8 heads of keys:
  // 4 rows a tile 0.99 ms, 1.77 in 64; 32 rows 1.94 ms, 1.79 in 64; 64 rows 3.2 ms, 1.81 in 64.
  p.rows = (int64_t)T * per <= 16 ? 16 : 64;
  p.tpt = per < p.rows ? p.rows / per : 1;
  p.hgroups = per > p.rows ? (per + p.rows - 1) / p.rows : 1;
  p.tiles = (int32_t)tiles_of(n, T, packed, p.tpt);
  // Splits for about four blocks an SM, at most 128.  fp32, 64 rows of 4 tokens behind 2048, 8 heads: 0.99 ms, 1.30 with
  // three a SM, 0.88 with eight; one prompt of 300 behind 3000, 8 heads over 2: 216 us, 210 and 238.
  const int64_t units = (int64_t)p.tiles * G * p.hgroups, want = 4 * (int64_t)sms;
  const int64_t s = units > 0 ? (want + units - 1) / units : 1;
  p.splits = (int32_t)(s < 1 ? 1 : s > 128 ? 128 : s);
  p.ws_bytes = p.splits > 1 ? units * p.splits * p.rows * (int64_t)(d + 2) * 4 : 0;
  return p;
}

cudaError_t launch_simt(int dtype, bool vec, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  const SimtArgs g{a, p};
  if (dtype == mx::T_F32) return pick<float>(vec, g, s);
  return dtype == mx::T_BF16 ? pick<__nv_bfloat16>(vec, g, s) : pick<__half>(vec, g, s);
}

cudaError_t launch_simt_join(int dtype, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  const SimtArgs g{a, p};
  return dtype == mx::T_F32 ? join<float>(g, s) : dtype == mx::T_BF16 ? join<__nv_bfloat16>(g, s) : join<__half>(g, s);
}

cudaError_t read_simt_status(cudaStream_t s, int32_t* code) { return take_status(g_simt_status, s, code); }

}  // namespace at
}  // namespace dl
