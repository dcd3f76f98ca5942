// The norms on both sides of a mixer.
//   gated_norm   per head of d values:  y = norm(x) w (+ b), times act(gate); or the gate first,
//                y = norm(x act(gate)) w (+ b)
//   add_norm     per row of D values:   h = residual + alpha scale (norm(x) post | x),
//                y = norm(h) w (+ b)
// norm is x / sqrt(mean x^2 + eps) (RMS) or the same of x - mean x (layer).
//
// A group of threads holds one row in registers, eight values a thread and
// pass, so every input is read and every output written once; sums are in 32
// bits, the variance from the centred values.  HBM bound: about ten operations
// a value.  A row of up to 256 values takes a part of a warp (gt threads, a
// power of two); a wider one a whole block.
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

// Sum over the group's threads (a part of a warp, or the whole block).
template <bool BLOCK>
__device__ __forceinline__ float group_sum(float v, int gt, float* sm) {
  const int lim = BLOCK ? 32 : gt;
  for (int o = 1; o < lim; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (BLOCK) {
    __syncthreads();                     // the sums of the call before are read
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int k = 0; k < (int)(blockDim.x >> 5); ++k) v += sm[k];
  }
  return v;
}

// v <- norm(v), over n values of the group; values past n are zero and stay so
// where `live` says so.
template <bool BLOCK, int VPT>
__device__ __forceinline__ void norm_regs(float (&v)[VPT][8], const int (&valid)[VPT], int n, int kind, float eps,
                                          int gt, float* sm) {
  if (kind == NORM_LAYER) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[i][k];
    const float mean = group_sum<BLOCK>(s, gt, sm) / (float)n;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = k < valid[i] ? v[i][k] - mean : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s = fmaf(v[i][k], v[i][k], s);
  const float r = rsqrtf(group_sum<BLOCK>(s, gt, sm) / (float)n + eps);
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] *= r;
}

template <class T, bool VEC, int VPT, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 128)
gated_norm_kernel(const __grid_constant__ GatedNormArgs a, int gt) {
  __shared__ float sm[32];
  const int per = BLOCK ? 1 : blockDim.x / gt;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x % gt;
  const int64_t u = (int64_t)blockIdx.x * per + (BLOCK ? 0 : threadIdx.x / gt);
  const bool on = u < a.rows * a.H;      // idle groups still take part in the shuffles
  const int64_t row = on ? u / a.H : 0;
  const int h = on ? (int)(u - row * a.H) : 0;
  const int G = BLOCK ? blockDim.x : gt;
  const T* x = static_cast<const T*>(a.x) + row * a.xs + (int64_t)h * a.d;
  const T* gp = a.gate ? static_cast<const T*>(a.gate) + row * a.gs + (int64_t)h * a.d : nullptr;
  T* y = static_cast<T*>(a.y) + row * a.ys + (int64_t)h * a.d;
  const int64_t w0 = a.w_heads ? (int64_t)h * a.d : 0;

  float v[VPT][8], g[VPT][8];
  int valid[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (lane + G * i);
    valid[i] = on ? min(8, a.d - c) : 0;
    unpack8<T>(load8<T, VEC>(x + c, valid[i]), v[i]);
    if (gp) unpack8<T>(load8<T, VEC>(gp + c, valid[i]), g[i]);
  }
  if (gp) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        g[i][k] = act_f<T>(g[i][k], a.act);
        if (a.gate_first) v[i][k] = k < valid[i] ? v[i][k] * g[i][k] : 0.f;
      }
  }
  norm_regs<BLOCK, VPT>(v, valid, a.d, a.kind, a.eps, gt, sm);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (lane + G * i);
    float w[8], b[8];
    weights8<T, VEC>(a.w, w0 + c, valid[i], a.w_f32, w);
    if (a.b) weights8<T, VEC>(a.b, w0 + c, valid[i], a.w_f32, b);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      v[i][k] = a.b ? fmaf(v[i][k], w[k], b[k]) : v[i][k] * w[k];
      if (gp && !a.gate_first) v[i][k] *= g[i][k];
    }
    store8<T, VEC>(y + c, pack8<T>(v[i]), valid[i]);
  }
}

template <class T, class R, bool VEC, int VPT, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 128)
add_norm_kernel(const __grid_constant__ AddNormArgs a, int gt) {
  __shared__ float sm[32];
  const int per = BLOCK ? 1 : blockDim.x / gt;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x % gt;
  const int64_t u = (int64_t)blockIdx.x * per + (BLOCK ? 0 : threadIdx.x / gt);
  const bool on = u < a.rows;
  const int64_t row = on ? u : 0;
  const int G = BLOCK ? blockDim.x : gt;
  const T* x = static_cast<const T*>(a.x) + row * a.xs;
  const R* res = a.res ? static_cast<const R*>(a.res) + row * a.rs : nullptr;
  T* y = static_cast<T*>(a.y) + row * a.ys;
  R* hp = static_cast<R*>(a.h) + row * a.hs;

  float v[VPT][8];
  Vec8<R> rv[VPT];
  int valid[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (lane + G * i);
    valid[i] = on ? min(8, a.D - c) : 0;
    unpack8<T>(load8<T, VEC>(x + c, valid[i]), v[i]);
    rv[i] = load8<R, VEC>(res + c, res ? valid[i] : 0);
  }
  if (a.post) {
    norm_regs<BLOCK, VPT>(v, valid, a.D, a.kind, a.eps, gt, sm);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float w[8];
      weights8<T, VEC>(a.post, 8 * (lane + G * i), valid[i], a.w_f32, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] *= w[k];
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float f[8], sc[8];
    unpack8<R>(rv[i], f);
    if (a.scale) weights8<T, VEC>(a.scale, 8 * (lane + G * i), valid[i], a.w_f32, sc);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float s = a.scale ? a.alpha * sc[k] : a.alpha;
      v[i][k] = k < valid[i] ? fmaf(v[i][k], s, f[k]) : 0.f;
    }
    if (a.h) store8<R, VEC>(hp + 8 * (lane + G * i), pack8<R>(v[i]), valid[i]);
  }
  // the norm takes h as it is in 32 bits, before its rounding
  norm_regs<BLOCK, VPT>(v, valid, a.D, a.kind, a.eps, gt, sm);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (lane + G * i);
    float w[8], b[8];
    weights8<T, VEC>(a.w, c, valid[i], a.w_f32, w);
    if (a.b) weights8<T, VEC>(a.b, c, valid[i], a.w_f32, b);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[i][k] = a.b ? fmaf(v[i][k], w[k], b[k]) : v[i][k] * w[k];
    store8<T, VEC>(y + c, pack8<T>(v[i]), valid[i]);
  }
}

// Threads of a group: the row's vectors, up to a power of two in a warp, or
// whole warps of a block.  A row of 8 * 32 values or less is one vector a
// thread of a part of a warp; more is a block, with up to 1024 threads of up
// to two vectors (16384 values).
struct Shape { int gt, vpt, threads; bool block; };
Shape shape_of(int n) {
  const int vecs = (n + 7) / 8;
  if (vecs <= 32) {
    int gt = 1;
    while (gt < vecs) gt <<= 1;
    return {gt, 1, 128, false};
  }
  const int vpt = vecs <= 512 ? 1 : 2;
  return {0, vpt, ((vecs + vpt - 1) / vpt + 31) / 32 * 32, true};
}

template <class T, bool VEC>
cudaError_t go_gated(const GatedNormArgs& a, cudaStream_t s) {
  const Shape k = shape_of(a.d);
  const int64_t units = a.rows * a.H;
  const int64_t per = k.block ? 1 : k.threads / k.gt;
  const unsigned grid = (unsigned)((units + per - 1) / per);
  if (!k.block) gated_norm_kernel<T, VEC, 1, false><<<grid, k.threads, 0, s>>>(a, k.gt);
  else if (k.vpt == 1) gated_norm_kernel<T, VEC, 1, true><<<grid, k.threads, 0, s>>>(a, 0);
  else gated_norm_kernel<T, VEC, 2, true><<<grid, k.threads, 0, s>>>(a, 0);
  return cudaGetLastError();
}
template <class T, class R, bool VEC>
cudaError_t go_add(const AddNormArgs& a, cudaStream_t s) {
  const Shape k = shape_of(a.D);
  const int64_t per = k.block ? 1 : k.threads / k.gt;
  const unsigned grid = (unsigned)((a.rows + per - 1) / per);
  if (!k.block) add_norm_kernel<T, R, VEC, 1, false><<<grid, k.threads, 0, s>>>(a, k.gt);
  else if (k.vpt == 1) add_norm_kernel<T, R, VEC, 1, true><<<grid, k.threads, 0, s>>>(a, 0);
  else add_norm_kernel<T, R, VEC, 2, true><<<grid, k.threads, 0, s>>>(a, 0);
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
