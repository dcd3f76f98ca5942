// Selective state space scan on the FP32 cores, token after token:
//   dt = softplus(raw + bias_h),  S <- e^{dt A_h} S + (dt x) B^T,  y = S C + D_h x
// with S [P, N] per (row, head) in fp32 and B, C shared by the heads of a group.
//
// One CTA per (row, head, tile of state rows).  A thread keeps PR state rows
// times 16 state columns in registers for the whole row; NL threads share a
// state row and add up their parts of y by shuffles.  Tokens come in chunks of
// TC, staged in shared memory in 32 bits.  Three operations per state element
// and token, so the FP32 cores bound it.  Every size and type runs here.
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

constexpr int SC_THREADS = 128, SC_PR = 2, SC_TC = 16;

// Columns of the thread: 4 (ln + NL i) + e, i, e = 0..3, so that the NL threads
// of a row read consecutive 16-byte vectors of a staged B or C.
template <class T, int NL>
__global__ void __launch_bounds__(SC_THREADS)
ssm_scan_kernel(const __grid_constant__ SsmArgs a) {
  constexpr int NP = 16 * NL;                       // padded state columns
  constexpr int PB = SC_THREADS / NL * SC_PR;       // state rows of the CTA
  __shared__ __align__(16) float sB[SC_TC][NP], sC[SC_TC][NP];
  __shared__ float sx[SC_TC][PB], sy[SC_TC][PB], sdt[SC_TC], sdec[SC_TC];
  const int pt = (a.P + PB - 1) / PB;
  const int tile = blockIdx.x % pt, rh = blockIdx.x / pt;
  const int row = rh / a.H, h = rh - row * a.H, g = h / (a.H / a.G);
  const RowItem it = a.items[row];
  const int len = row_len(it), p0 = tile * PB;
  const int ln = threadIdx.x % NL, pl = threadIdx.x / NL * SC_PR;

  auto at = [&](const TokView& v, int t) {
    return (int64_t)(it.begin + t) * v.st + (int64_t)row * v.sn;
  };
  float* st = a.state ? a.state + ((int64_t)it.slot * a.H + h) * a.P * a.N : nullptr;
  float S[SC_PR][16];
#pragma unroll
  for (int r = 0; r < SC_PR; ++r)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int p = p0 + pl + r, n = 4 * (ln + NL * (i >> 2)) + (i & 3);
      S[r][i] = st && !row_fresh(it) && p < a.P && n < a.N ? st[(int64_t)p * a.N + n] : 0.f;
    }
  const float Ah = a.A[h], Dh = a.D ? a.D[h] : 0.f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;

  for (int t0 = 0; t0 < len; t0 += SC_TC) {
    const int nt = min(SC_TC, len - t0);
    for (int i = threadIdx.x; i < nt * NP; i += SC_THREADS) {
      const int t = i / NP, n = i - t * NP;
      sB[t][n] = n < a.N ? to_f(static_cast<const T*>(a.B.p)[at(a.B, t0 + t) + (int64_t)g * a.N + n]) : 0.f;
      sC[t][n] = n < a.N ? to_f(static_cast<const T*>(a.C.p)[at(a.C, t0 + t) + (int64_t)g * a.N + n]) : 0.f;
    }
    for (int i = threadIdx.x; i < nt * PB; i += SC_THREADS) {
      const int t = i / PB, p = p0 + i - t * PB;
      sx[t][p - p0] = p < a.P ? to_f(static_cast<const T*>(a.x.p)[at(a.x, t0 + t) + (int64_t)h * a.P + p]) : 0.f;
    }
    if (threadIdx.x < nt) {
      const int64_t o = at(a.dt, t0 + threadIdx.x) + h;
      float d = (a.dt_f32 ? static_cast<const float*>(a.dt.p)[o] : to_f(static_cast<const T*>(a.dt.p)[o])) + bias;
      d = a.softplus ? softplus_f(d) : d;
      sdt[threadIdx.x] = d;
      sdec[threadIdx.x] = expf(d * Ah);
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const float dec = sdec[t], dt = sdt[t];
      float xd[SC_PR], acc[SC_PR];
#pragma unroll
      for (int r = 0; r < SC_PR; ++r) {
        xd[r] = sx[t][pl + r] * dt;
        acc[r] = 0.f;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 b4 = *reinterpret_cast<const float4*>(&sB[t][4 * (ln + NL * q)]);
        const float4 c4 = *reinterpret_cast<const float4*>(&sC[t][4 * (ln + NL * q)]);
        const float bb[4] = {b4.x, b4.y, b4.z, b4.w}, cc[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int r = 0; r < SC_PR; ++r) {
            S[r][4 * q + e] = fmaf(S[r][4 * q + e], dec, xd[r] * bb[e]);
            acc[r] = fmaf(S[r][4 * q + e], cc[e], acc[r]);
          }
      }
#pragma unroll
      for (int r = 0; r < SC_PR; ++r) {
#pragma unroll
        for (int o = 1; o < NL; o <<= 1) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
        if (ln == 0) sy[t][pl + r] = fmaf(Dh, sx[t][pl + r], acc[r]);
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nt * PB; i += SC_THREADS) {
      const int t = i / PB, p = p0 + i - t * PB;
      if (p < a.P)
        static_cast<T*>(const_cast<void*>(a.y.p))[at(a.y, t0 + t) + (int64_t)h * a.P + p] = from_f<T>(sy[t][p - p0]);
    }
  }
  if (!st) return;
#pragma unroll
  for (int r = 0; r < SC_PR; ++r)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int p = p0 + pl + r, n = 4 * (ln + NL * (i >> 2)) + (i & 3);
      if (p < a.P && n < a.N) st[(int64_t)p * a.N + n] = S[r][i];
    }
}

template <class T, int NL>
cudaError_t go(const SsmArgs& a, cudaStream_t s) {
  constexpr int PB = SC_THREADS / NL * SC_PR;
  const unsigned grid = (unsigned)((int64_t)a.rows * a.H * ((a.P + PB - 1) / PB));
  ssm_scan_kernel<T, NL><<<grid, SC_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}
template <class T>
cudaError_t go_n(const SsmArgs& a, cudaStream_t s) {
  return a.N <= 16    ? go<T, 1>(a, s)
         : a.N <= 32  ? go<T, 2>(a, s)
         : a.N <= 64  ? go<T, 4>(a, s)
         : a.N <= 128 ? go<T, 8>(a, s)
                      : go<T, 16>(a, s);
}

}  // namespace

cudaError_t launch_ssm_scan(int dtype, const SsmArgs& a, cudaStream_t s) {
  return dtype == T_F32    ? go_n<float>(a, s)
         : dtype == T_BF16 ? go_n<__nv_bfloat16>(a, s)
                           : go_n<__half>(a, s);
}

}  // namespace mx
}  // namespace dl
