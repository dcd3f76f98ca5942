// Short causal convolution over time, with its activation, the L2 norm of the
// leading heads and the carried inputs of every slot:
//   z[t, c] = b[c] + sum_j w[c, j] x[t - W + 1 + j, c],   y = act(z)
//   heads below channel l2c:  y / sqrt(sum over the head of y^2 + eps)
// where x at a negative t is the slot's carried input (its last W - 1, oldest
// first) or zero for a fresh row.
//
// A thread takes eight channels (one 16-byte vector of a 16-bit type) and
// walks the tokens of its tile with the last W - 1 of them in registers, so a
// value is read once a tile plus W - 1 of every TT tokens again.  Sums, the
// activation and the norm are in 32 bits, rounded once.  About 2 W + 4
// operations a value: HBM bound.
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

constexpr int CONV_THREADS = 128;

template <class T, int W, bool VEC>
__global__ void __launch_bounds__(CONV_THREADS)
conv_kernel(const __grid_constant__ ConvArgs a) {
  const int tile = blockIdx.x;
  const int row = find_row(a.items, a.rows, tile, a.per_row);
  const RowItem it = a.items[row];
  const int len = row_len(it);
  const int ti = tile - (a.per_row ? row * a.per_row : it.tile0);
  const int t0 = ti * a.TT, t1 = min(len, t0 + a.TT);
  const int c = (blockIdx.y * CONV_THREADS + threadIdx.x) * 8;
  const int valid = min(8, a.C - c);     // <= 0: only takes part in the shuffles
  const T* x = static_cast<const T*>(a.x.p) + (int64_t)it.begin * a.x.st + (int64_t)row * a.x.sn + c;
  const bool normed = c < a.l2c;

  float w[W][8], bias[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
#pragma unroll
    for (int j = 0; j < W; ++j)
      w[j][k] = k >= valid ? 0.f
                : a.w_f32  ? static_cast<const float*>(a.w)[(int64_t)(c + k) * W + j]
                           : to_f(static_cast<const T*>(a.w)[(int64_t)(c + k) * W + j]);
    bias[k] = k >= valid || !a.b ? 0.f
              : a.w_f32          ? static_cast<const float*>(a.b)[c + k]
                                 : to_f(static_cast<const T*>(a.b)[c + k]);
  }

  // the W - 1 inputs before t0
  Vec8<T> hist[W - 1];
  T* st = a.state ? static_cast<T*>(a.state) + (int64_t)it.slot * (W - 1) * a.C + c : nullptr;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    if (t0 > 0)
      hist[j] = load8<T, VEC>(x + (int64_t)(t0 - (W - 1) + j) * a.x.st, valid);   // TT >= W - 1
    else
      hist[j] = load8<T, VEC>(st + (int64_t)j * a.C, st && !row_fresh(it) ? valid : 0);
  }

  // Carried inputs after the call: the last W - 1 of (old ones, x).  Only the
  // row's first tile reads and writes them, so no other block can see them change.
  if (ti == 0 && st) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int p = len - (W - 1) + j;
      Vec8<T> v;
      if (p >= 0) {
        v = load8<T, VEC>(x + (int64_t)p * a.x.st, valid);
      } else {
        v = hist[0];
#pragma unroll
        for (int i = 1; i < W - 1; ++i)
          if (W - 1 + p == i) v = hist[i];
      }
      store8<T, VEC>(st + (int64_t)j * a.C, v, valid);
    }
  }
  if (t1 <= t0) return;

  float win[W - 1][8];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) unpack8<T>(hist[j], win[j]);

  int part = 0;
#pragma unroll
  for (int k = 1; k < CONV_PARTS; ++k) part += c >= a.c0[k];
  T* y = static_cast<T*>(const_cast<void*>(a.y[part].p)) + (int64_t)it.begin * a.y[part].st +
         (int64_t)row * a.y[part].sn + (c - a.c0[part]);
  const int64_t yst = a.y[part].st;

  for (int t = t0; t < t1; ++t) {
    float cur[8], z[8];
    unpack8<T>(load8<T, VEC>(x + (int64_t)t * a.x.st, valid), cur);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float s = bias[k];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][k], win[j][k], s);
      s = fmaf(w[W - 1][k], cur[k], s);
      z[k] = act_f<T>(s, a.act);
#pragma unroll
      for (int j = 0; j + 2 < W; ++j) win[j][k] = win[j + 1][k];
      win[W - 2][k] = cur[k];
    }
    if (a.l2c) {
      float ss = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(z[k], z[k], ss);
      for (int o = 1; o < (a.hd >> 3); o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = normed ? rsqrtf(ss + a.eps) : 1.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) z[k] *= r;
    }
    const Vec8<T> o = pack8<T>(z);
    if (VEC) {
      store8<T, true>(y + (int64_t)t * yst, o, valid);
    } else {
      // a vector may straddle two ranges
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < valid) {
          int q = 0;
#pragma unroll
          for (int e = 1; e < CONV_PARTS; ++e) q += c + k >= a.c0[e];
          static_cast<T*>(const_cast<void*>(a.y[q].p))[(int64_t)(it.begin + t) * a.y[q].st +
                                                       (int64_t)row * a.y[q].sn + (c + k - a.c0[q])] =
              from_f<T>(z[k]);
        }
    }
  }
}

template <class T, int W>
cudaError_t go(bool vec, const ConvArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.tiles, (unsigned)((a.C + 8 * CONV_THREADS - 1) / (8 * CONV_THREADS)));
  if (vec) conv_kernel<T, W, true><<<grid, CONV_THREADS, 0, s>>>(a);
  else conv_kernel<T, W, false><<<grid, CONV_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}
template <class T>
cudaError_t go_w(bool vec, const ConvArgs& a, cudaStream_t s) {
  return a.W == 2 ? go<T, 2>(vec, a, s) : a.W == 3 ? go<T, 3>(vec, a, s) : go<T, 4>(vec, a, s);
}

}  // namespace

cudaError_t launch_conv(int dtype, bool vec, const ConvArgs& a, cudaStream_t s) {
  return dtype == T_F32    ? go_w<float>(vec, a, s)
         : dtype == T_BF16 ? go_w<__nv_bfloat16>(vec, a, s)
                           : go_w<__half>(vec, a, s);
}

}  // namespace mx
}  // namespace dl
