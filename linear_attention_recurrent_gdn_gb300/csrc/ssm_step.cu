// One token of the state space scan for every listed slot:
//   dt = softplus(raw + bias_h),  S <- e^{dt A_h} S + (dt x) B^T,  y = S C + D_h x
// It reads and writes every state element once (8 P N bytes a head against
// 2 (2 P + 1) + 4 N of inputs and outputs), with five operations an element:
// HBM bound.  A warp takes ROWS rows of a head's state at a time, LPR lanes to
// a row with a 16-byte vector each, all ROWS loads in flight before the first
// is used.
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

constexpr int ST_THREADS = 128, ST_ROWS = 8;

template <bool VEC>
__device__ __forceinline__ float4 ld4(const float* p, int valid) {
  if (VEC) return valid > 0 ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(valid > 0 ? p[0] : 0.f, valid > 1 ? p[1] : 0.f, valid > 2 ? p[2] : 0.f, valid > 3 ? p[3] : 0.f);
}
template <bool VEC>
__device__ __forceinline__ void st4(float* p, float4 v, int valid) {
  if (VEC) {
    if (valid > 0) *reinterpret_cast<float4*>(p) = v;
  } else {
    if (valid > 0) p[0] = v.x;
    if (valid > 1) p[1] = v.y;
    if (valid > 2) p[2] = v.z;
    if (valid > 3) p[3] = v.w;
  }
}

// IT vectors a lane and row (N <= 128 IT); lpr lanes a row, 32 / lpr rows a load.
template <class T, bool VEC, int IT>
__global__ void __launch_bounds__(ST_THREADS)
ssm_step_kernel(const __grid_constant__ SsmArgs a, int lpr, int tiles) {
  const int lane = threadIdx.x & 31, per = 32 / lpr, ln = lane % lpr, sub = lane / lpr;
  const int64_t w = (int64_t)blockIdx.x * (ST_THREADS / 32) + (threadIdx.x >> 5);
  const int64_t rh = w / tiles;
  const int tile = (int)(w - rh * tiles);
  if (rh >= (int64_t)a.rows * a.H) return;      // whole warps
  const int row = (int)(rh / a.H), h = (int)(rh - (int64_t)row * a.H), g = h / (a.H / a.G);
  const RowItem it = a.items[row];
  float* st = a.state + ((int64_t)it.slot * a.H + h) * a.P * a.N;
  const int p0 = tile * ST_ROWS * per;
  auto off = [&](const TokView& v) { return (int64_t)it.begin * v.st + (int64_t)row * v.sn; };

  float4 S[ST_ROWS][IT];
#pragma unroll
  for (int r = 0; r < ST_ROWS; ++r) {
    const int p = p0 + r * per + sub;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int n = 4 * (ln + lpr * i);
      S[r][i] = ld4<VEC>(st + (int64_t)p * a.N + n, p < a.P && !row_fresh(it) ? a.N - n : 0);
    }
  }
  const int64_t od = off(a.dt) + h;
  float dt = (a.dt_f32 ? static_cast<const float*>(a.dt.p)[od] : to_f(static_cast<const T*>(a.dt.p)[od])) +
             (a.dt_bias ? a.dt_bias[h] : 0.f);
  dt = a.softplus ? softplus_f(dt) : dt;
  const float dec = expf(dt * a.A[h]), Dh = a.D ? a.D[h] : 0.f;
  float B[IT][4], C[IT][4];
  const T* Bp = static_cast<const T*>(a.B.p) + off(a.B) + (int64_t)g * a.N;
  const T* Cp = static_cast<const T*>(a.C.p) + off(a.C) + (int64_t)g * a.N;
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int n = 4 * (ln + lpr * i) + e;
      B[i][e] = n < a.N ? dt * to_f(Bp[n]) : 0.f;
      C[i][e] = n < a.N ? to_f(Cp[n]) : 0.f;
    }
  const T* xp = static_cast<const T*>(a.x.p) + off(a.x) + (int64_t)h * a.P;
  T* yp = static_cast<T*>(const_cast<void*>(a.y.p)) + off(a.y) + (int64_t)h * a.P;
#pragma unroll
  for (int r = 0; r < ST_ROWS; ++r) {
    const int p = p0 + r * per + sub;
    const float x = p < a.P ? to_f(xp[p]) : 0.f;
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      float4& v = S[r][i];
      v.x = fmaf(v.x, dec, x * B[i][0]);
      v.y = fmaf(v.y, dec, x * B[i][1]);
      v.z = fmaf(v.z, dec, x * B[i][2]);
      v.w = fmaf(v.w, dec, x * B[i][3]);
      y = fmaf(v.x, C[i][0], y);
      y = fmaf(v.y, C[i][1], y);
      y = fmaf(v.z, C[i][2], y);
      y = fmaf(v.w, C[i][3], y);
      const int n = 4 * (ln + lpr * i);
      st4<VEC>(st + (int64_t)p * a.N + n, v, p < a.P ? a.N - n : 0);
    }
    for (int o = 1; o < lpr; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (ln == 0 && p < a.P) yp[p] = from_f<T>(fmaf(Dh, x, y));
  }
}

template <class T, bool VEC>
cudaError_t go(const SsmArgs& a, cudaStream_t s) {
  int lpr = 1;
  while (lpr < 32 && 4 * lpr < a.N) lpr <<= 1;
  const int rows = ST_ROWS * (32 / lpr), tiles = (a.P + rows - 1) / rows;
  const int64_t warps = (int64_t)a.rows * a.H * tiles, wpb = ST_THREADS / 32;
  const unsigned grid = (unsigned)((warps + wpb - 1) / wpb);
  if (a.N <= 128) ssm_step_kernel<T, VEC, 1><<<grid, ST_THREADS, 0, s>>>(a, lpr, tiles);
  else ssm_step_kernel<T, VEC, 2><<<grid, ST_THREADS, 0, s>>>(a, lpr, tiles);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_ssm_step(int dtype, const SsmArgs& a, cudaStream_t s) {
  const bool vec = a.N % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state) & 15) == 0;
  if (dtype == T_F32) return vec ? go<float, true>(a, s) : go<float, false>(a, s);
  if (dtype == T_BF16) return vec ? go<__nv_bfloat16, true>(a, s) : go<__nv_bfloat16, false>(a, s);
  return vec ? go<__half, true>(a, s) : go<__half, false>(a, s);
}

}  // namespace mx
}  // namespace dl
