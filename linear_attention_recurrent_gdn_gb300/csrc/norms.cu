// The norms on both sides of a mixer.
//   gated_norm   per head of d values:  y = norm(x) w (+ b), times act(gate); or the gate first,
//                y = norm(x act(gate)) w (+ b)
//   add_norm     per row of D values:   h = residual + alpha scale (norm(x) post | x),
//                y = norm(h) w (+ b)
// norm is x / sqrt(mean x^2 + eps) (RMS) or the same of x - mean x (layer).
//
// A group of threads holds a row in registers, eight values a thread and piece,
// so every input is read and every output written once; sums are in 32 bits,
// the variance from the centred values.  About ten operations a value: HBM
// bound, so what counts is bytes on their way.  A row of up to 256 values takes
// a part of a warp (gt threads, a power of two), four rows a thread where there
// are many; one of up to 1024 a warp with up to four pieces a thread; a wider
// one a block of a quarter of its pieces' threads.
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

// Sums of U values over the group's threads (a part of a warp, or the whole block).
template <bool BLOCK, int U>
__device__ __forceinline__ void group_sum(float (&v)[U], int gt, float* sm) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = __shfl_xor_sync(0xffffffffu, v[u], o);
      v[u] += BLOCK || o < gt ? w : 0.f;
    }
  }
  if (BLOCK) {
    __syncthreads();                     // the sums of the call before are read
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v[0];
    __syncthreads();
    v[0] = 0.f;
    for (int k = 0; k < (int)(blockDim.x >> 5); ++k) v[0] += sm[k];
  }
}

// v <- norm(v) for U rows of n values each; `valid` of a piece's eight values
// exist, the others are zero and do not count.
template <bool BLOCK, int U, int VPT>
__device__ __forceinline__ void norm_regs(float (&v)[U][VPT][8], const int (&valid)[VPT], int n, int kind, float eps,
                                          int gt, float* sm) {
  const float inv = 1.f / (float)n;
  float s[U];
  if (kind == NORM_LAYER) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) s[u] += v[u][i][k];
    }
    group_sum<BLOCK, U>(s, gt, sm);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float mean = s[u] * inv;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][i][k] = k < valid[i] ? v[u][i][k] - mean : 0.f;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    s[u] = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) s[u] = fmaf(v[u][i][k], v[u][i][k], s[u]);
  }
  group_sum<BLOCK, U>(s, gt, sm);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float r = rsqrtf(fmaf(s[u], inv, eps));
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][i][k] *= r;
  }
}

constexpr int NT = 128;                  // threads of a block of small rows

// U rows a group of gt threads (neighbouring groups' rows in between), VPT pieces a thread.
template <class T, bool VEC, int U, int VPT, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : NT)
gated_norm_kernel(const __grid_constant__ GatedNormArgs a, int gt) {
  __shared__ float sm[32];
  const int per = BLOCK ? 1 : NT / gt, G = BLOCK ? blockDim.x : gt;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x % gt;
  const int64_t u0 = (int64_t)blockIdx.x * per * U + (BLOCK ? 0 : threadIdx.x / gt);
  const int64_t units = a.rows * a.H;
  int valid[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) valid[i] = min(8, a.d - 8 * (lane + G * i));

  Vec8<T> xv[U][VPT], gv[U][VPT];
  int64_t row[U];
  int h[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t at = u0 + (int64_t)u * per;
    const bool on = at < units;          // idle groups still take part in the shuffles
    row[u] = on ? (int64_t)((uint32_t)at / (uint32_t)a.H) : -1;
    h[u] = on ? (int)((uint32_t)at - (uint32_t)row[u] * (uint32_t)a.H) : 0;
    const T* x = static_cast<const T*>(a.x) + row[u] * a.xs + (int64_t)h[u] * a.d;
    const T* g = static_cast<const T*>(a.gate) + row[u] * a.gs + (int64_t)h[u] * a.d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      xv[u][i] = load8<T, VEC>(x + 8 * (lane + G * i), on ? valid[i] : 0);
      if (a.gate) gv[u][i] = load8<T, VEC>(g + 8 * (lane + G * i), on ? valid[i] : 0);
    }
  }
  float v[U][VPT][8];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      unpack8<T>(xv[u][i], v[u][i]);
      if (a.gate && a.gate_first) {
        float g[8];
        unpack8<T>(gv[u][i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][i][k] = k < valid[i] ? v[u][i][k] * act_f<T>(g[k], a.act) : 0.f;
      }
    }
  norm_regs<BLOCK, U, VPT>(v, valid, a.d, a.kind, a.eps, gt, sm);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    T* y = static_cast<T*>(a.y) + row[u] * a.ys + (int64_t)h[u] * a.d;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (lane + G * i), on = row[u] >= 0 ? valid[i] : 0;
      float w[8], b[8];
      weights8<T, VEC>(a.w, (a.w_heads ? (int64_t)h[u] * a.d : 0) + c, valid[i], a.w_f32, w);
      if (a.b) weights8<T, VEC>(a.b, (a.w_heads ? (int64_t)h[u] * a.d : 0) + c, valid[i], a.w_f32, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][i][k] = a.b ? fmaf(v[u][i][k], w[k], b[k]) : v[u][i][k] * w[k];
      if (a.gate && !a.gate_first) {
        float g[8];
        unpack8<T>(gv[u][i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[u][i][k] *= act_f<T>(g[k], a.act);
      }
      store8<T, VEC>(y + c, pack8<T>(v[u][i]), on);
    }
  }
}

template <class T, class R, bool VEC, int U, int VPT, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : NT)
add_norm_kernel(const __grid_constant__ AddNormArgs a, int gt) {
  __shared__ float sm[32];
  const int per = BLOCK ? 1 : NT / gt, G = BLOCK ? blockDim.x : gt;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x % gt;
  const int64_t u0 = (int64_t)blockIdx.x * per * U + (BLOCK ? 0 : threadIdx.x / gt);
  int valid[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) valid[i] = min(8, a.D - 8 * (lane + G * i));

  Vec8<T> xv[U][VPT];
  Vec8<R> rv[U][VPT];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = u0 + (int64_t)u * per;
    const bool on = row < a.rows;
    const T* x = static_cast<const T*>(a.x) + row * a.xs;
    const R* res = static_cast<const R*>(a.res) + row * a.rs;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      xv[u][i] = load8<T, VEC>(x + 8 * (lane + G * i), on ? valid[i] : 0);
      rv[u][i] = load8<R, VEC>(res + 8 * (lane + G * i), on && a.res ? valid[i] : 0);
    }
  }
  float v[U][VPT][8];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VPT; ++i) unpack8<T>(xv[u][i], v[u][i]);
  if (a.post) norm_regs<BLOCK, U, VPT>(v, valid, a.D, a.kind, a.eps, gt, sm);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (lane + G * i);
    float sc[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) sc[k] = a.alpha;
    if (a.post) {
      float w[8];
      weights8<T, VEC>(a.post, c, valid[i], a.w_f32, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) sc[k] *= w[k];
    }
    if (a.scale) {
      float w[8];
      weights8<T, VEC>(a.scale, c, valid[i], a.w_f32, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) sc[k] *= w[k];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = u0 + (int64_t)u * per;
      float f[8];
      unpack8<R>(rv[u][i], f);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][i][k] = k < valid[i] ? fmaf(v[u][i][k], sc[k], f[k]) : 0.f;
      if (a.h)
        store8<R, VEC>(static_cast<R*>(a.h) + row * a.hs + c, pack8<R>(v[u][i]), row < a.rows ? valid[i] : 0);
    }
  }
  // the norm takes h as it is in 32 bits, before its rounding
  norm_regs<BLOCK, U, VPT>(v, valid, a.D, a.kind, a.eps, gt, sm);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (lane + G * i);
    float w[8], b[8];
    weights8<T, VEC>(a.w, c, valid[i], a.w_f32, w);
    if (a.b) weights8<T, VEC>(a.b, c, valid[i], a.w_f32, b);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = u0 + (int64_t)u * per;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[u][i][k] = a.b ? fmaf(v[u][i][k], w[k], b[k]) : v[u][i][k] * w[k];
      store8<T, VEC>(static_cast<T*>(a.y) + row * a.ys + c, pack8<T>(v[u][i]), row < a.rows ? valid[i] : 0);
    }
  }
}

// How `units` rows of n values run: mode 0: a part of a warp, four rows a
// thread; 1: the same, one row (fewer rows than fill the GPU four times over);
// 2, 3: a warp, two or four pieces a thread; 4: a block.
struct Shape { int mode, gt, threads; unsigned grid; };
Shape shape_of(int n, int64_t units) {
  const int vecs = (n + 7) / 8;
  if (vecs > 128) return {4, 0, (vecs + 127) / 128 * 32, (unsigned)units};
  int gt = 1;
  while (gt < vecs && gt < 32) gt <<= 1;
  const int mode = vecs > 64 ? 3 : vecs > 32 ? 2 : units * gt >= 4 * 152 * 2048 ? 0 : 1;
  const int64_t per = (int64_t)NT / gt * (mode == 0 ? 4 : 1);
  return {mode, gt, NT, (unsigned)((units + per - 1) / per)};
}

template <class T, bool VEC>
cudaError_t go_gated(const GatedNormArgs& a, cudaStream_t s) {
  const Shape k = shape_of(a.d, a.rows * a.H);
  switch (k.mode) {
    case 0: gated_norm_kernel<T, VEC, 4, 1, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 1: gated_norm_kernel<T, VEC, 1, 1, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 2: gated_norm_kernel<T, VEC, 1, 2, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 3: gated_norm_kernel<T, VEC, 1, 4, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    default: gated_norm_kernel<T, VEC, 1, 4, true><<<k.grid, k.threads, 0, s>>>(a, 0);
  }
  return cudaGetLastError();
}
template <class T, class R, bool VEC>
cudaError_t go_add(const AddNormArgs& a, cudaStream_t s) {
  const Shape k = shape_of(a.D, a.rows);
  switch (k.mode) {
    case 0: add_norm_kernel<T, R, VEC, 4, 1, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 1: add_norm_kernel<T, R, VEC, 1, 1, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 2: add_norm_kernel<T, R, VEC, 1, 2, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 3: add_norm_kernel<T, R, VEC, 1, 4, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    default: add_norm_kernel<T, R, VEC, 1, 4, true><<<k.grid, k.threads, 0, s>>>(a, 0);
  }
  return cudaGetLastError();
}
template <class T, class R>
cudaError_t go_add_v(bool vec, const AddNormArgs& a, cudaStream_t s) {
  return vec ? go_add<T, R, true>(a, s) : go_add<T, R, false>(a, s);
}

}  // namespace

cudaError_t launch_gated_norm(int dtype, bool vec, const GatedNormArgs& a, cudaStream_t s) {
  if (dtype == T_F32) return vec ? go_gated<float, true>(a, s) : go_gated<float, false>(a, s);
  if (dtype == T_BF16) return vec ? go_gated<__nv_bfloat16, true>(a, s) : go_gated<__nv_bfloat16, false>(a, s);
  return vec ? go_gated<__half, true>(a, s) : go_gated<__half, false>(a, s);
}
cudaError_t launch_add_norm(int dtype, bool res_f32, bool vec, const AddNormArgs& a, cudaStream_t s) {
  if (dtype == T_F32) return go_add_v<float, float>(vec, a, s);
  if (dtype == T_BF16)
    return res_f32 ? go_add_v<__nv_bfloat16, float>(vec, a, s) : go_add_v<__nv_bfloat16, __nv_bfloat16>(vec, a, s);
  return res_f32 ? go_add_v<__half, float>(vec, a, s) : go_add_v<__half, __half>(vec, a, s);
}

}  // namespace mx
}  // namespace dl
