// One token of the state space scan for every listed slot:
//   dt = softplus(raw + bias_h),  S <- e^{dt A_h} S + (dt x) B^T,  y = S C + D_h x
// It reads and writes every state element once (8 P N bytes a head against
// 2 (2 P + 1) + 4 N of inputs and outputs), with five operations an element:
// HBM bound.  A warp takes ROWS loads of a head's state, lpr lanes to a row with
// a 16-byte vector each, all in flight before the first is used.
//
// Measured on a GB300 (copy: 6.7 TB/s): 256 slots of 32 heads of 128 x 128 159
// us, 6.8 TB/s; 64 slots of 32 heads of 64 x 64 13 us; one slot of 4 heads of
// 64 x 64 2.3 us, the launch and one trip to memory.
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

constexpr int ST_THREADS = 128;

// The state passes through once: streaming loads and stores.
template <bool VEC>
__device__ __forceinline__ float4 ld4(const float* p, int valid) {
  if (VEC) return valid > 0 ? __ldcs(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(valid > 0 ? p[0] : 0.f, valid > 1 ? p[1] : 0.f, valid > 2 ? p[2] : 0.f, valid > 3 ? p[3] : 0.f);
}
template <bool VEC>
__device__ __forceinline__ void st4(float* p, float4 v, int valid) {
  if (VEC) {
    if (valid > 0) __stcs(reinterpret_cast<float4*>(p), v);
  } else {
    if (valid > 0) p[0] = v.x;
    if (valid > 1) p[1] = v.y;
    if (valid > 2) p[2] = v.z;
    if (valid > 3) p[3] = v.w;
  }
}

// IT vectors a lane and row (N <= 128 IT); lpr lanes a row, 32 / lpr rows a
// load, ROWS loads a warp.
template <class T, bool VEC, int IT, int ROWS>
__global__ void __launch_bounds__(ST_THREADS)
ssm_step_kernel(const __grid_constant__ SsmStep a, int lpr, int tiles) {
  const int lane = threadIdx.x & 31, per = 32 / lpr, ln = lane % lpr, sub = lane / lpr;
  const uint32_t w = blockIdx.x * (ST_THREADS / 32) + (threadIdx.x >> 5);
  const uint32_t rh = w / tiles;
  const int tile = (int)(w - rh * tiles);
  if (rh >= (uint32_t)(a.rows * a.H)) return;      // whole warps
  const int row = rh / a.H, h = rh - row * a.H, g = h / (a.H / a.G);
  const bool fresh = a.slot[row] < 0;
  const int slot = fresh ? ~a.slot[row] : a.slot[row];
  const int p0 = tile * ROWS * per + sub;
  float* st = a.state + (((int64_t)slot * a.H + h) * a.P + p0) * a.N + 4 * ln;
  auto off = [&](const TokView& v) { return (int64_t)row * v.sn; };

  // every load before the first use
  float4 S[ROWS][IT];
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
#pragma unroll
    for (int i = 0; i < IT; ++i)
      S[r][i] = ld4<VEC>(st + (int64_t)r * per * a.N + 4 * lpr * i,
                         p0 + r * per < a.P && !fresh ? a.N - 4 * (ln + lpr * i) : 0);
  const int64_t od = off(a.dt) + h;
  float dt = a.dt_f32 ? static_cast<const float*>(a.dt.p)[od] : to_f(static_cast<const T*>(a.dt.p)[od]);
  const float bias = a.dt_bias ? a.dt_bias[h] : 0.f, Ah = a.A[h], Dh = a.D ? a.D[h] : 0.f;
  const T* Bp = static_cast<const T*>(a.B.p) + off(a.B) + (int64_t)g * a.N;
  const T* Cp = static_cast<const T*>(a.C.p) + off(a.C) + (int64_t)g * a.N;
  T braw[IT][4], craw[IT][4], xraw[ROWS];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = 4 * (ln + lpr * i) + e;
      braw[i][e] = n < a.N ? Bp[n] : from_f<T>(0.f);
      craw[i][e] = n < a.N ? Cp[n] : from_f<T>(0.f);
    }
  const T* xp = static_cast<const T*>(a.x.p) + off(a.x) + (int64_t)h * a.P;
  T* yp = static_cast<T*>(const_cast<void*>(a.y.p)) + off(a.y) + (int64_t)h * a.P;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) xraw[r] = p0 + r * per < a.P ? xp[p0 + r * per] : from_f<T>(0.f);

  dt = a.softplus ? softplus_f(dt + bias) : dt + bias;
  const float dec = expf(dt * Ah);
  float B[IT][4], C[IT][4], y[ROWS];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      B[i][e] = dt * to_f(braw[i][e]);
      C[i][e] = to_f(craw[i][e]);
    }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const float x = to_f(xraw[r]);
    y[r] = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      float4& v = S[r][i];
      v.x = fmaf(v.x, dec, x * B[i][0]);
      v.y = fmaf(v.y, dec, x * B[i][1]);
      v.z = fmaf(v.z, dec, x * B[i][2]);
      v.w = fmaf(v.w, dec, x * B[i][3]);
      y[r] = fmaf(v.x, C[i][0], y[r]);
      y[r] = fmaf(v.y, C[i][1], y[r]);
      y[r] = fmaf(v.z, C[i][2], y[r]);
      y[r] = fmaf(v.w, C[i][3], y[r]);
      st4<VEC>(st + (int64_t)r * per * a.N + 4 * lpr * i, v, p0 + r * per < a.P ? a.N - 4 * (ln + lpr * i) : 0);
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    for (int o = 1; o < lpr; o <<= 1) y[r] += __shfl_xor_sync(0xffffffffu, y[r], o);
    if (ln == 0 && p0 + r * per < a.P) yp[p0 + r * per] = from_f<T>(fmaf(Dh, to_f(xraw[r]), y[r]));
  }
}

template <class T, bool VEC, int ROWS>
cudaError_t go_rows(const SsmStep& a, int lpr, cudaStream_t s) {
  const int rows = ROWS * (32 / lpr), tiles = (a.P + rows - 1) / rows;
  const int64_t warps = (int64_t)a.rows * a.H * tiles, wpb = ST_THREADS / 32;
  const unsigned grid = (unsigned)((warps + wpb - 1) / wpb);
  if (a.N <= 128) ssm_step_kernel<T, VEC, 1, ROWS><<<grid, ST_THREADS, 0, s>>>(a, lpr, tiles);
  else ssm_step_kernel<T, VEC, 2, ROWS><<<grid, ST_THREADS, 0, s>>>(a, lpr, tiles);
  return cudaGetLastError();
}
template <class T, bool VEC>
cudaError_t go(const SsmStep& a, cudaStream_t s) {
  int lpr = 1;
  while (lpr < 32 && 4 * lpr < a.N) lpr <<= 1;
  // Eight rows a warp amortise its inputs (the 256 slots: 159 us, 242 with two
  // rows); two where eight leave the GPU's SMs with less than four warps each (a
  // few slots, where latency counts: 2.3 us, 3.4 with eight).
  const int64_t warps8 = (int64_t)a.rows * a.H * a.P / (8 * (32 / lpr));
  return warps8 >= 4 * 152 ? go_rows<T, VEC, 8>(a, lpr, s) : go_rows<T, VEC, 2>(a, lpr, s);
}

}  // namespace

cudaError_t launch_ssm_step(int dtype, const SsmStep& a, cudaStream_t s) {
  const bool vec = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
  if (dtype == T_F32) return vec ? go<float, true>(a, s) : go<float, false>(a, s);
  if (dtype == T_BF16) return vec ? go<__nv_bfloat16, true>(a, s) : go<__nv_bfloat16, false>(a, s);
  return vec ? go<__half, true>(a, s) : go<__half, false>(a, s);
}

}  // namespace mx
}  // namespace dl
