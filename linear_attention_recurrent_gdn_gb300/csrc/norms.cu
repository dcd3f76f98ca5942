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
// are many (of the same head, so that its weights are loaded once); one of up to 1024 a warp with up to four pieces a thread; a wider
// one a block of a quarter of its pieces' threads.
//
// Measured on a GB300 (copy: 6.7 TB/s): residual sum and norm of 8192 x 4096
// bf16 42 us, 6.4 TB/s, with an fp32 stream and both norms 67 us, 6.0 TB/s;
// gated RMS norm of 8192 x 32 heads of 128 35 us, 5.8 TB/s; layer norm with bias
// and gate of 8192 x 40 heads of 64 24 us, 5.2 TB/s (short rows: a warp's sums,
// weights and gates are some 200 instructions for 32 x 8 values, and the
// schedulers issue 63% of the time); one token 2.4 us, the launch.
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

// Sums of U values over the group's threads (a part of a warp, or the whole block).
template <bool BLOCK, int U>
__device__ __forceinline__ void group_sum(float (&v)[U], int gt, float* sm) {
  const int lim = BLOCK ? 32 : gt;
#pragma unroll 1
  for (int o = 1; o < lim; o <<= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
  if (BLOCK) {
    __syncthreads();                     // the sums of the call before are read
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v[0];
    __syncthreads();
    v[0] = 0.f;
    for (int k = 0; k < (int)(blockDim.x >> 5); ++k) v[0] += sm[k];
  }
}

// A piece that ends inside its eight values: what is past the end is zero.
__device__ __forceinline__ f2 mask2(f2 v, int k, int valid) {
  float a, b;
  un2(v, a, b);
  return mk2(2 * k < valid ? a : 0.f, 2 * k + 1 < valid ? b : 0.f);
}

// v <- norm(v) for U rows of n values each; `valid` of a piece's eight values
// exist (FULL: all), the others are zero and do not count.
template <bool BLOCK, bool FULL, int U, int VPT>
__device__ __forceinline__ void norm_regs(f2 (&v)[U][VPT][4], const int (&valid)[VPT], int n, int kind, float eps,
                                          int gt, float* sm) {
  const float inv = 1.f / (float)n;
  float s[U];
  if (kind == NORM_LAYER) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f2 t = mk2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) t = add2(t, v[u][i][k]);
      float p, q;
      un2(t, p, q);
      s[u] = p + q;
    }
    group_sum<BLOCK, U>(s, gt, sm);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float mean = -s[u] * inv;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[u][i][k] = add2(v[u][i][k], mk2(mean, mean));
          if (!FULL) v[u][i][k] = mask2(v[u][i][k], k, valid[i]);
        }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    f2 t = mk2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) t = fma2(v[u][i][k], v[u][i][k], t);
    float p, q;
    un2(t, p, q);
    s[u] = p + q;
  }
  group_sum<BLOCK, U>(s, gt, sm);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const float r = rsqrtf(fmaf(s[u], inv, eps));
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) v[u][i][k] = mul2(v[u][i][k], mk2(r, r));
  }
}

template <class T>
__device__ __forceinline__ f2 gate2(f2 g, int act) {
  return act == ACT_NONE ? g : act == ACT_SILU ? act2<T, true>(g) : act2<T, false>(g);
}
// Eight weights (fp32 or T) as pairs.
template <class T, bool VEC>
__device__ __forceinline__ void wpairs(const void* base, int64_t i, int valid, int f32, f2 (&f)[4]) {
  float t[8];
  weights8<T, VEC>(base, i, valid, f32, t);
#pragma unroll
  for (int k = 0; k < 4; ++k) f[k] = mk2(t[2 * k], t[2 * k + 1]);
}
template <class T>
__device__ __forceinline__ Vec8<T> pack_pairs(const f2 (&v)[4]) {
  float t[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) un2(v[k], t[2 * k], t[2 * k + 1]);
  return pack8<T>(t);
}

constexpr int NT = 128;                  // threads of a block of small rows

// The same head of U following rows a group of gt threads (one load of its
// weights), VPT pieces a thread; FULL: the group's threads have eight values in
// every piece.
template <class T, bool VEC, bool FULL, int U, int VPT, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : NT)
gated_norm_kernel(const __grid_constant__ GatedNormArgs a, int gt) {
  __shared__ float sm[32];
  const int per = BLOCK ? 1 : NT / gt, G = BLOCK ? blockDim.x : gt;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (gt - 1);
  const uint32_t u0 = blockIdx.x * (uint32_t)per + (BLOCK ? 0 : threadIdx.x / gt);
  const int row0 = (int)(u0 / (uint32_t)a.H) * U, h = (int)(u0 % (uint32_t)a.H);
  int valid[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) valid[i] = FULL ? 8 : min(8, a.d - 8 * (lane + G * i));

  Vec8<T> xv[U][VPT], gv[U][VPT];
  const int64_t in = (int64_t)h * a.d + 8 * lane;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool on = row0 + u < a.rows;              // idle groups still take part in the shuffles
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      xv[u][i] = load8<T, VEC>(static_cast<const T*>(a.x) + (int64_t)(row0 + u) * a.xs + in + 8 * G * i, on ? valid[i] : 0);
      if (a.gate)
        gv[u][i] =
            load8<T, VEC>(static_cast<const T*>(a.gate) + (int64_t)(row0 + u) * a.gs + in + 8 * G * i, on ? valid[i] : 0);
    }
  }
  f2 v[U][VPT][4];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VPT; ++i) pairs8<T>(xv[u][i], v[u][i]);
  if (a.gate && a.gate_first) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        f2 g[4];
        pairs8<T>(gv[u][i], g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[u][i][k] = mul2(v[u][i][k], gate2<T>(g[k], a.act));
          if (!FULL) v[u][i][k] = mask2(v[u][i][k], k, valid[i]);
        }
      }
  }
  norm_regs<BLOCK, FULL, U, VPT>(v, valid, a.d, a.kind, a.eps, gt, sm);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int64_t wo = (a.w_heads ? (int64_t)h * a.d : 0) + 8 * (lane + G * i);
    f2 w[4], b[4];
    wpairs<T, VEC>(a.w, wo, valid[i], a.w_f32, w);
    if (a.b) {
      wpairs<T, VEC>(a.b, wo, valid[i], a.w_f32, b);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][i][k] = fma2(v[u][i][k], w[k], b[k]);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][i][k] = mul2(v[u][i][k], w[k]);
    }
  }
  if (a.gate && !a.gate_first) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        f2 g[4];
        pairs8<T>(gv[u][i], g);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[u][i][k] = mul2(v[u][i][k], gate2<T>(g[k], a.act));
      }
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      store8<T, VEC>(static_cast<T*>(a.y) + (int64_t)(row0 + u) * a.ys + in + 8 * G * i, pack_pairs<T>(v[u][i]),
                     row0 + u < a.rows ? valid[i] : 0);
}

template <class T, class R, bool VEC, bool FULL, int U, int VPT, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : NT)
add_norm_kernel(const __grid_constant__ AddNormArgs a, int gt) {
  __shared__ float sm[32];
  const int per = BLOCK ? 1 : NT / gt, G = BLOCK ? blockDim.x : gt;
  const int lane = BLOCK ? threadIdx.x : threadIdx.x & (gt - 1);
  const int64_t u0 = (int64_t)blockIdx.x * (per * U) + (BLOCK ? 0 : threadIdx.x / gt);
  int valid[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) valid[i] = FULL ? 8 : min(8, a.D - 8 * (lane + G * i));

  Vec8<T> xv[U][VPT];
  Vec8<R> rv[U][VPT];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = u0 + u * per;
    const bool on = row < a.rows;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = 8 * (lane + G * i);
      xv[u][i] = load8<T, VEC>(static_cast<const T*>(a.x) + row * a.xs + c, on ? valid[i] : 0);
      rv[u][i] = load8<R, VEC>(static_cast<const R*>(a.res) + row * a.rs + c, on && a.res ? valid[i] : 0);
    }
  }
  f2 v[U][VPT][4];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < VPT; ++i) pairs8<T>(xv[u][i], v[u][i]);
  if (a.post) norm_regs<BLOCK, FULL, U, VPT>(v, valid, a.D, a.kind, a.eps, gt, sm);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (lane + G * i);
    f2 sc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sc[k] = mk2(a.alpha, a.alpha);
    if (a.post) {
      f2 w[4];
      wpairs<T, VEC>(a.post, c, valid[i], a.w_f32, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) sc[k] = mul2(sc[k], w[k]);
    }
    if (a.scale) {
      f2 w[4];
      wpairs<T, VEC>(a.scale, c, valid[i], a.w_f32, w);
#pragma unroll
      for (int k = 0; k < 4; ++k) sc[k] = mul2(sc[k], w[k]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = u0 + u * per;
      f2 f[4];
      pairs8<R>(rv[u][i], f);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[u][i][k] = fma2(v[u][i][k], sc[k], f[k]);
        if (!FULL) v[u][i][k] = mask2(v[u][i][k], k, valid[i]);
      }
      if (a.h)
        store8<R, VEC>(static_cast<R*>(a.h) + row * a.hs + c, pack_pairs<R>(v[u][i]), row < a.rows ? valid[i] : 0);
    }
  }
  // the norm takes h as it is in 32 bits, before its rounding
  norm_regs<BLOCK, FULL, U, VPT>(v, valid, a.D, a.kind, a.eps, gt, sm);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = 8 * (lane + G * i);
    f2 w[4], b[4];
    wpairs<T, VEC>(a.w, c, valid[i], a.w_f32, w);
    if (a.b) wpairs<T, VEC>(a.b, c, valid[i], a.w_f32, b);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t row = u0 + u * per;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[u][i][k] = a.b ? fma2(v[u][i][k], w[k], b[k]) : mul2(v[u][i][k], w[k]);
      store8<T, VEC>(static_cast<T*>(a.y) + row * a.ys + c, pack_pairs<T>(v[u][i]), row < a.rows ? valid[i] : 0);
    }
  }
}

// How rows of `heads` times n values run.  Mode 0: a part of a warp and four rows
// a thread (8192 x 40 heads of 64: 24 us, 31 with one row); 1: the same with one
// row where there are fewer, or where four leave the SMs with less than four times
// their threads (256 x 32 heads of 128: 2.7 us, 2.9 with four); 2, 3: a warp with two or four pieces a
// thread; 4, 5: a block with one piece a thread for a few rows (one of 4096: 2.4
// us, 3.2 with four pieces) or four (8192 rows: 67 us, 85 with one).
struct Shape { int mode, gt, threads; bool full; unsigned grid; };
Shape shape_of(int n, int64_t rows, int64_t heads) {
  const int64_t units = rows * heads;
  const int vecs = (n + 7) / 8;
  const bool few = units < 2 * 152;
  if (vecs > 128 || (vecs > 32 && few)) {
    const int vpt = few && vecs <= 512 ? 1 : 4, threads = ((vecs + vpt - 1) / vpt + 31) / 32 * 32;
    return {vpt == 1 ? 4 : 5, 0, threads, n == 8 * threads * vpt, (unsigned)units};
  }
  int gt = 1;
  while (gt < vecs && gt < 32) gt <<= 1;
  const int mode = vecs > 64 ? 3 : vecs > 32 ? 2 : rows >= 4 && units * gt >= 4 * 152 * 2048 ? 0 : 1;
  const int64_t groups = (mode == 0 ? (rows + 3) / 4 : rows) * heads, per = NT / gt;
  return {mode, gt, NT, n == 8 * gt * (mode == 3 ? 4 : mode == 2 ? 2 : 1), (unsigned)((groups + per - 1) / per)};
}

template <class T, bool VEC, bool FULL>
cudaError_t go_gated(const Shape& k, const GatedNormArgs& a, cudaStream_t s) {
  switch (k.mode) {
    case 0: gated_norm_kernel<T, VEC, FULL, 4, 1, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 1: gated_norm_kernel<T, VEC, FULL, 1, 1, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 2: gated_norm_kernel<T, VEC, FULL, 1, 2, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 3: gated_norm_kernel<T, VEC, FULL, 1, 4, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 4: gated_norm_kernel<T, VEC, FULL, 1, 1, true><<<k.grid, k.threads, 0, s>>>(a, 0); break;
    default: gated_norm_kernel<T, VEC, FULL, 1, 4, true><<<k.grid, k.threads, 0, s>>>(a, 0);
  }
  return cudaGetLastError();
}
template <class T>
cudaError_t go_gated_v(bool vec, const GatedNormArgs& a, cudaStream_t s) {
  const Shape k = shape_of(a.d, a.rows, a.H);
  return !vec ? go_gated<T, false, false>(k, a, s) : k.full ? go_gated<T, true, true>(k, a, s) : go_gated<T, true, false>(k, a, s);
}
template <class T, class R, bool VEC, bool FULL>
cudaError_t go_add(const Shape& k, const AddNormArgs& a, cudaStream_t s) {
  switch (k.mode) {
    case 0: add_norm_kernel<T, R, VEC, FULL, 4, 1, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 1: add_norm_kernel<T, R, VEC, FULL, 1, 1, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 2: add_norm_kernel<T, R, VEC, FULL, 1, 2, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 3: add_norm_kernel<T, R, VEC, FULL, 1, 4, false><<<k.grid, k.threads, 0, s>>>(a, k.gt); break;
    case 4: add_norm_kernel<T, R, VEC, FULL, 1, 1, true><<<k.grid, k.threads, 0, s>>>(a, 0); break;
    default: add_norm_kernel<T, R, VEC, FULL, 1, 4, true><<<k.grid, k.threads, 0, s>>>(a, 0);
  }
  return cudaGetLastError();
}
template <class T, class R>
cudaError_t go_add_v(bool vec, const AddNormArgs& a, cudaStream_t s) {
  const Shape k = shape_of(a.D, a.rows, 1);
  return !vec     ? go_add<T, R, false, false>(k, a, s)
         : k.full ? go_add<T, R, true, true>(k, a, s)
                  : go_add<T, R, true, false>(k, a, s);
}

}  // namespace

cudaError_t launch_gated_norm(int dtype, bool vec, const GatedNormArgs& a, cudaStream_t s) {
  return dtype == T_F32    ? go_gated_v<float>(vec, a, s)
         : dtype == T_BF16 ? go_gated_v<__nv_bfloat16>(vec, a, s)
                           : go_gated_v<__half>(vec, a, s);
}
cudaError_t launch_add_norm(int dtype, bool res_f32, bool vec, const AddNormArgs& a, cudaStream_t s) {
  if (dtype == T_F32) return go_add_v<float, float>(vec, a, s);
  if (dtype == T_BF16)
    return res_f32 ? go_add_v<__nv_bfloat16, float>(vec, a, s) : go_add_v<__nv_bfloat16, __nv_bfloat16>(vec, a, s);
  return res_f32 ? go_add_v<__half, float>(vec, a, s) : go_add_v<__half, __half>(vec, a, s);
}

}  // namespace mx
}  // namespace dl
