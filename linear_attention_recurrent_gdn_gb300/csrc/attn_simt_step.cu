// Attention of one token a row over pages on the FP32 cores: fp32, and what the
// tensor-core kernel does not take (odd head dimensions, strides, alignment).
//
// Only the keys that the token sees are visited: the sinks before its window,
// then the window (or all keys up to its own).  A warp takes eight of them at a
// time; a lane holds DV consecutive dimensions of HB query heads that share the
// keys, of the eight keys and of their values, straight from memory.  The
// products' partial sums of the eight keys and HB heads are added up over the
// lanes together (halving exchanges: about one shuffle a sum), and every weight
// is handed to all lanes for its value: some 12 instructions a key and head.
// Running softmax in fp32 as in attn_simt.cu; its reference moves when a score
// passes it by more than 2^8.
//
// HBM-bound for few heads a group, bound by instructions from eight on: fp32, 64
// x 2048 tokens of 128, 166 us for one head over each of 8 (6.5 TB/s), 216 us for
// 4 (5.0 TB/s; 979 us with the tiles of attn_simt.cu), 363 us for 16 over each of
// 4.  bf16 heads of 100, which no vector divides, 790 us for 4 over each of 8.  A
// block's four warps take the keys of a row (or of a part of it: few rows are
// split, and joined by attn_simt.cu's second launch) in turns.
#include <cmath>

#include "attn_device.cuh"
#include "mixer_device.cuh"

namespace dl {
namespace at {

static __device__ int32_t g_simt_step_status;

namespace {

using mx::from_f;
using mx::to_f;

constexpr int WARPS = 4, THREADS = 32 * WARPS;

struct Args {
  AttnArgs a;
  AttnPlan p;
};

// DV consecutive values at p (vec: as one or two vectors), zero from `valid` on.
template <class T, int DV>
__device__ __forceinline__ void load(const T* p, int valid, bool vec, float (&f)[DV]) {
  if (vec && valid >= DV) {
    if constexpr (sizeof(T) == 4) {
      if constexpr (DV >= 4) {
#pragma unroll
        for (int k = 0; k < DV; k += 4) {
          const float4 v = *reinterpret_cast<const float4*>(p + k);
          f[k] = v.x, f[k + 1] = v.y, f[k + 2] = v.z, f[k + 3] = v.w;
        }
      } else if constexpr (DV == 2) {
        const float2 v = *reinterpret_cast<const float2*>(p);
        f[0] = v.x, f[1] = v.y;
      } else {
        f[0] = to_f(*p);
      }
    } else if constexpr (DV == 1) {
      f[0] = to_f(*p);
    } else {
      uint32_t w[DV / 2];
      if constexpr (DV == 8) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else if constexpr (DV == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x, w[1] = v.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
      }
#pragma unroll
      for (int k = 0; k < DV / 2; ++k) mx::unpack2<T>(w[k], f[2 * k], f[2 * k + 1]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < DV; ++k) f[k] = k < valid ? to_f(p[k]) : 0.f;
  }
}

template <class T, int DV, int HB>
__global__ void __launch_bounds__(THREADS) simt_step_kernel(const __grid_constant__ Args g, bool vec) {
  constexpr int KEYS = DV == 8 ? 4 : 8, NE = KEYS * HB, SHIFT = NE == 32 ? 0 : NE == 16 ? 1 : NE == 8 ? 2 : 3;
  static_assert(NE << SHIFT == 32, "entries and lanes");
  __shared__ float ml[WARPS][HB][2];
  __shared__ float os[WARPS][HB][32 * DV];
  const AttnArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, per = a.H / a.G, d = a.d, row = blockIdx.x;
  const int gh = blockIdx.y / g.p.hgroups, h0 = (blockIdx.y - gh * g.p.hgroups) * HB, heads = min(HB, per - h0);
  int slot;
  const int len = row_length(a, row, slot, tid == 0 ? &g_simt_step_status : nullptr);
  if (len < 0) return;
  // the keys that the token sees, numbered: [0, sk), then [lo, len)
  const int lo = a.window ? max(0, len - a.window) : 0, sk = min(a.sinks, lo), seen = sk + len - lo;
  const int step = KEYS * WARPS, each = ((seen + g.p.splits - 1) / g.p.splits + step - 1) / step * step;
  const int u0 = min(seen, (int)blockIdx.z * each), u1 = min(seen, u0 + each);
  const int c0 = lane * DV, valid = min(DV, d - c0);

  float q[HB][DV], o[HB][DV], m = -INFINITY, l = 0.f;      // m, l: of this lane's entry's head
#pragma unroll
  for (int h = 0; h < HB; ++h) {
    load<T, DV>(static_cast<const T*>(a.q) + (int64_t)row * a.q_sn + ((int64_t)gh * per + h0 + (h < heads ? h : 0)) * d + c0, valid, vec, q[h]);
#pragma unroll
    for (int k = 0; k < DV; ++k) o[h][k] = 0.f;
  }
  const int entry = lane >> SHIFT, ek = entry / HB;        // entry = key * HB + head
  auto look_up = [&](int u) {          // the page of key u + lane
    u += lane;
    if (lane >= KEYS || u >= u1) return 0;
    return page_of(a, slot, u < sk ? u : lo + u - sk, &g_simt_step_status);
  };
  int ids = look_up(u0 + warp * KEYS);
  for (int u = u0 + warp * KEYS; u < u1; u += step) {
    float k[KEYS][DV], v[KEYS][DV];
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      const int id = __shfl_sync(0xffffffffu, ids, i), j = u + i < sk ? u + i : lo + u + i - sk;
      const int off = j & ((1 << a.page_shift) - 1), n = u + i < u1 ? valid : 0;
      load<T, DV>(static_cast<const T*>(a.kp.p) + (id * a.kp.sp + gh * a.kp.sg + off * a.kp.st + c0), n, vec, k[i]);
      load<T, DV>(static_cast<const T*>(a.vp.p) + (id * a.vp.sp + gh * a.vp.sg + off * a.vp.st + c0), n, vec, v[i]);
    }
    ids = look_up(u + step);
    float s[NE];
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        float x = 0.f;
#pragma unroll
        for (int c = 0; c < DV; ++c) x = fmaf(q[h][c], k[i][c], x);
        s[i * HB + h] = x;
      }
    const bool live = u + ek < u1;
    float z = reduce_entries<NE>(s, lane) * a.scale_log2;
    if (!live) z = -INFINITY;
    if (__any_sync(0xffffffffu, z > m + 8.f)) {
      float top = fmaxf(m, z);
#pragma unroll
      for (int x = HB << SHIFT; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float f = exp2f(m - held(top));
      m = top;
      l *= f;
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        const float fh = __shfl_sync(0xffffffffu, f, h << SHIFT);
#pragma unroll
        for (int c = 0; c < DV; ++c) o[h][c] *= fh;
      }
    }
    const float p = live ? exp2f(z - held(m)) : 0.f;
    l += p;
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
#pragma unroll
      for (int h = 0; h < HB; ++h) {
        const float w = __shfl_sync(0xffffffffu, p, (i * HB + h) << SHIFT);
#pragma unroll
        for (int c = 0; c < DV; ++c) o[h][c] = fmaf(w, v[i][c], o[h][c]);
      }
  }

  // ---- the warps' parts become one
#pragma unroll
  for (int x = HB << SHIFT; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
  if (ek == 0 && (lane & ((1 << SHIFT) - 1)) == 0) {
    ml[warp][entry][0] = m;
    ml[warp][entry][1] = l;
  }
#pragma unroll
  for (int h = 0; h < HB; ++h)
#pragma unroll
    for (int c = 0; c < DV; ++c) os[warp][h][c0 + c] = o[h][c];
  __syncthreads();
  for (int e = tid; e < heads * d; e += THREADS) {
    const int h = e / d, c = e - h * d;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, ml[w][h][0]);
    const float base = held(top);
    float sum = 0.f, x = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (ml[w][h][1] == 0.f) continue;                    // saw nothing
      const float f = exp2f(ml[w][h][0] - base);
      sum = fmaf(ml[w][h][1], f, sum);
      x = fmaf(os[w][h][c], f, x);
    }
    if (g.p.splits == 1) {
      static_cast<T*>(a.o)[(int64_t)row * a.o_sn + ((int64_t)gh * per + h0 + h) * d + c] = from_f<T>(sum == 0.f ? 0.f : x / sum);
    } else {
      float* part = a.ws + (((int64_t)row * gridDim.y + blockIdx.y) * g.p.splits + blockIdx.z) * HB * (d + 2) + (int64_t)h * (d + 2);
      if (c == 0) {
        part[0] = top;
        part[1] = sum;
      }
      part[2 + c] = x;
    }
  }
}

template <class T, int DV>
cudaError_t heads(const Args& g, bool vec, cudaStream_t s) {
  const dim3 grid((unsigned)g.a.n, (unsigned)(g.a.G * g.p.hgroups), (unsigned)g.p.splits);
  if (g.p.rows == 1) simt_step_kernel<T, DV, 1><<<grid, THREADS, 0, s>>>(g, vec);
  else simt_step_kernel<T, DV, 4><<<grid, THREADS, 0, s>>>(g, vec);
  return cudaGetLastError();
}
template <class T>
cudaError_t width(const Args& g, bool vec, cudaStream_t s) {
  const int d = g.a.d;
  return d <= 32 ? heads<T, 1>(g, vec, s) : d <= 64 ? heads<T, 2>(g, vec, s) : d <= 128 ? heads<T, 4>(g, vec, s) : heads<T, 8>(g, vec, s);
}

}  // namespace

AttnPlan simt_step_plan(int n, int H, int G, int d, int sms) {
  AttnPlan p{};
  const int per = H / G;
  // Query heads of a block: four of them where there are two or more, although keys are loaded again for the next four.
  // fp32, 64 x 2048 tokens over 8: 8 heads 168 us, 211 in fours; 16 heads 212 us, 245 one by one; 32 heads 215, 425.
  p.rows = per == 1 ? 1 : 4;
  p.tpt = 1;
  p.hgroups = (per + p.rows - 1) / p.rows;
  p.tiles = n;
  // Splits for about eight blocks an SM, at most 128.  fp32, 64 x 2048 tokens of 16 heads over 8: 212 us, 230 with four
  // a SM, 203 with 16 (but 173 and 168 for 8 over 8); one row of 131072 over 8: 230 us, 280 with at most 64, 205 with 256,
  // where one of 8000 over 2 takes 17.3 us instead of 12.2.
  const int64_t units = (int64_t)n * G * p.hgroups, s = units > 0 ? (8 * (int64_t)sms + units - 1) / units : 1;
  p.splits = (int32_t)(s > 128 ? 128 : s);
  p.ws_bytes = p.splits > 1 ? units * p.splits * p.rows * (int64_t)(d + 2) * 4 : 0;
  return p;
}

cudaError_t launch_simt_step(int dtype, bool vec, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  const Args g{a, p};
  const cudaError_t e = dtype == mx::T_F32 ? width<float>(g, vec, s)
                        : dtype == mx::T_BF16 ? width<__nv_bfloat16>(g, vec, s) : width<__half>(g, vec, s);
  return e != cudaSuccess || p.splits == 1 ? e : launch_simt_join(dtype, a, p, s);
}

cudaError_t read_simt_step_status(cudaStream_t s, int32_t* code) { return take_status(g_simt_step_status, s, code); }

}  // namespace at
}  // namespace dl
