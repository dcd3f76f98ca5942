// Selective state space scan on the FP32 cores, token after token:
//   dt = softplus(raw + bias_h),  S <- e^{dt A_h} S + (dt x) B^T,  y = S C + D_h x
// with S [P, N] per (row, head) in fp32 and B, C shared by the heads of a group.
//
// One CTA per (row, head, tile of state rows), and per segment of the row
// where rows are few and long.  A thread keeps PR state rows times 16 state
// columns in registers; NL threads share a state row and add up their parts of
// y.  Tokens come in chunks of TC, fetched a chunk ahead (eight values a piece)
// and staged in shared memory in 32 bits.  Three operations per state element
// and token, two elements an instruction (packed fp32), so the FP32 cores bound
// it: 16 x 512 tokens of 32 heads of 64 x 128 take 360 us in fp16 on a GB300, 174
// of them at the cores' full rate; 4 x 512 in fp32 163.  Every size and type runs
// here.
//
// Segments: a first launch (STATE) runs each but the last from zero (the first
// from the row's state) and leaves its end state and decay in the workspace; a
// second joins them to the states at the segments' starts; the full launch
// goes on from those.
#include "dl_device.cuh"
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

constexpr int SC_THREADS = 128;
constexpr float LOG2E = 1.4426950408889634f;

// State rows of a thread: as many as leave a CTA 64 rows or so, so that a value
// of B or C that was read from shared memory serves several (16 x 512 tokens of
// 32 heads of 64 x 128: 374 us with four, 399 with two, 722 with one, before the
// steps below).
__host__ __device__ constexpr int rows_of(int nl) { return nl == 8 ? 4 : nl >= 4 ? 2 : 1; }

struct ScanArgs {
  SsmArgs a;
  float* ws;                 // segment states [tiles][H][P][N], then log2 decays [tiles][H]
  int32_t seg_tokens, tiles, per_row;
};

// Columns of the thread: 4 (ln + NL i) + e, i, e = 0..3, so that the NL threads
// of a row read consecutive 16-byte vectors of a staged B or C.
template <class T, int NL, bool STATE, bool VEC>
__global__ void __launch_bounds__(SC_THREADS, 4)
ssm_scan_kernel(const __grid_constant__ ScanArgs sa) {
  // Chunks of eight tokens leave eight threads a row the shared memory for their
  // parts of y; UN tokens overlap.
  constexpr int TC = NL == 8 ? 8 : 16, UN = NL <= 2 ? 4 : NL == 8 ? 2 : 1;
  constexpr int PR = rows_of(NL), NP = 16 * NL, PB = SC_THREADS / NL * PR;
  const SsmArgs& a = sa.a;
  __shared__ __align__(16) float sB[TC][NP], sC[STATE ? 1 : TC][NP];
  // The NL parts of a value of y: with four or eight threads a row they wait in
  // shared memory for the chunk's end (16-byte pieces in an order that spares
  // both sides bank conflicts), else shuffles add them at once (4 x 512 tokens of 32 heads in fp32: 64 x 64
  // 74 us, 95 with shuffles; 64 x 128 163 us, 202).
  constexpr bool PARTS = NL == 4 || NL == 8;
  __shared__ __align__(16) float sx[TC][PB], sy[STATE ? 1 : TC][PARTS ? PR * SC_THREADS : PB];
  __shared__ float sdt[TC], sdec[TC];
  const int pt = (a.P + PB - 1) / PB, ph = pt * a.H;
  const int tile = blockIdx.x / ph, rest = blockIdx.x - tile * ph, h = rest / pt, g = h / (a.H / a.G);
  const int row = find_row(a.items, a.rows, tile, sa.per_row);
  const RowItem it = a.items[row];
  const int len = row_len(it), p0 = (rest - h * pt) * PB;
  const int seg = tile - (sa.per_row ? row * sa.per_row : it.tile0);
  const int nseg = len > sa.seg_tokens ? (len + sa.seg_tokens - 1) / sa.seg_tokens : 1;
  if (STATE && seg == nseg - 1) return;              // nothing follows the last segment
  const int s0 = seg * sa.seg_tokens, s1 = min(len, s0 + sa.seg_tokens);
  const int ln = threadIdx.x % NL, pl = threadIdx.x / NL * PR;
  auto place = [](int i) { return ((i >> 2) ^ (i >> 5)) << 2 | (i & 3); };   // of thread i's part
  const int mine = place(threadIdx.x);

  auto at = [&](const TokView& v, int t) {
    return (int64_t)(it.begin + t) * v.st + (int64_t)row * v.sn;
  };
  const int64_t per_tile = (int64_t)a.H * a.P * a.N, e0 = ((int64_t)h * a.P + p0 + pl) * a.N;
  float* pool = a.state ? a.state + (int64_t)it.slot * per_tile : nullptr;
  auto col = [&](int i) { return 4 * (ln + NL * (i >> 2)) + (i & 3); };
  auto on = [&](int r, int i) { return p0 + pl + r < a.P && col(i) < a.N; };
  float S[PR][16];
  {
    const float* from;
    if (STATE || nseg == 1) from = seg == 0 && pool && !row_fresh(it) ? pool : nullptr;
    else from = seg == 0 && row_fresh(it) ? nullptr : sa.ws + (int64_t)tile * per_tile;
#pragma unroll
    for (int r = 0; r < PR; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i) S[r][i] = from && on(r, i) ? from[e0 + (int64_t)r * a.N + col(i)] : 0.f;
    if (STATE && seg == 0 && from) {
      // the last segment's CTA overwrites the pool's entry in the full launch
#pragma unroll
      for (int r = 0; r < PR; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (on(r, i)) sa.ws[(int64_t)tile * per_tile + e0 + (int64_t)r * a.N + col(i)] = S[r][i];
    }
  }
  f2 S2[PR][8];
#pragma unroll
  for (int r = 0; r < PR; ++r)
#pragma unroll
    for (int i = 0; i < 8; ++i) S2[r][i] = mk2(S[r][2 * i], S[r][2 * i + 1]);
  const float Ah = a.A[h], Dh = a.D ? a.D[h] : 0.f, bias = a.dt_bias ? a.dt_bias[h] : 0.f;
  float ltot = 0.f;

  // The next chunk's pieces of eight values of B, C and x on their way: in registers, or where the state takes
  // most of those (eight threads a row), aligned ones to a place of the thread's own in shared memory (64 x 128
  // in fp32 163 us, 173 in registers; with four threads a row 99 us for 74).
  constexpr int NB = TC * NP / 8, NX = TC * PB / 8;      // pieces of a chunk
  constexpr int KB = (NB + SC_THREADS - 1) / SC_THREADS, KX = (NX + SC_THREADS - 1) / SC_THREADS;
  constexpr int KC = STATE ? 0 : KB, V16 = sizeof(T) / 2;
  constexpr bool RAW = VEC && NL == 8;
  __shared__ __align__(16) uint4 raw[RAW ? (KB + KC + KX) * V16 : 1][SC_THREADS];
  Vec8<T> vb[KB], vc[STATE ? 1 : KB], vx[KX];
  float vd = 0.f;
  auto bring = [&](Vec8<T>& v, int k, const T* p, int valid) {
    if constexpr (RAW) {
      if (valid > 0)
#pragma unroll
        for (int e = 0; e < V16; ++e)
          cp_async16(smem_u32(&raw[k * V16 + e][threadIdx.x]), reinterpret_cast<const uint4*>(p) + e);
    } else {
      v = load8<T, VEC>(p, valid);
    }
  };
  auto take = [&](const Vec8<T>& v, int k, bool valid) {
    if constexpr (RAW) {
      Vec8<T> r;
#pragma unroll
      for (int e = 0; e < V16; ++e) {
        const uint4 q = valid ? raw[k * V16 + e][threadIdx.x] : make_uint4(0, 0, 0, 0);
        r.w[4 * e] = q.x;
        r.w[4 * e + 1] = q.y;
        r.w[4 * e + 2] = q.z;
        r.w[4 * e + 3] = q.w;
      }
      return r;
    } else {
      return v;
    }
  };
  auto fetch = [&](int t0) {
    const int nt = s1 - t0;
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int i = threadIdx.x + k * SC_THREADS, t = i / (NP / 8), n = i % (NP / 8) * 8;
      const int valid = i < NB && t < nt ? min(8, a.N - n) : 0;
      bring(vb[k], k, static_cast<const T*>(a.B.p) + at(a.B, t0 + t) + (int64_t)g * a.N + n, valid);
      if constexpr (!STATE)
        bring(vc[k], KB + k, static_cast<const T*>(a.C.p) + at(a.C, t0 + t) + (int64_t)g * a.N + n, valid);
    }
#pragma unroll
    for (int k = 0; k < KX; ++k) {
      const int i = threadIdx.x + k * SC_THREADS, t = i / (PB / 8), p = p0 + i % (PB / 8) * 8;
      bring(vx[k], KB + KC + k, static_cast<const T*>(a.x.p) + at(a.x, t0 + t) + (int64_t)h * a.P + p,
            i < NX && t < nt ? min(8, a.P - p) : 0);
    }
    if constexpr (RAW) asm volatile("cp.async.commit_group;" ::: "memory");
    if (threadIdx.x < TC && (int)threadIdx.x < nt) {
      const int64_t o = at(a.dt, t0 + threadIdx.x) + h;
      vd = a.dt_f32 ? static_cast<const float*>(a.dt.p)[o] : to_f(static_cast<const T*>(a.dt.p)[o]);
    }
  };
  auto put8 = [&](float* to, const Vec8<T>& v) {
    float f[8];
    unpack8<T>(v, f);
    *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(to + 4) = make_float4(f[4], f[5], f[6], f[7]);
  };
  if (s0 < s1) fetch(s0);
  for (int t0 = s0; t0 < s1; t0 += TC) {
    const int nt = min(TC, s1 - t0);
    if constexpr (RAW) asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int k = 0; k < KB; ++k) {
      const int i = threadIdx.x + k * SC_THREADS;
      const bool valid = i / (NP / 8) < nt && i % (NP / 8) * 8 < a.N;
      if (i < NB) {
        put8(&sB[0][0] + 8 * i, take(vb[k], k, valid));
        if constexpr (!STATE) put8(&sC[0][0] + 8 * i, take(vc[k], KB + k, valid));
      }
    }
#pragma unroll
    for (int k = 0; k < KX; ++k) {
      const int i = threadIdx.x + k * SC_THREADS;
      const bool valid = i / (PB / 8) < nt && p0 + i % (PB / 8) * 8 < a.P;
      if (i < NX) put8(&sx[0][0] + 8 * i, take(vx[k], KB + KC + k, valid));
    }
    if (threadIdx.x < TC) {
      const float d = a.softplus ? softplus_f(vd + bias) : vd + bias;
      sdt[threadIdx.x] = d;
      sdec[threadIdx.x] = expf(d * Ah);
    }
    if (t0 + TC < s1) fetch(t0 + TC);
    __syncthreads();
#pragma unroll UN
    for (int t = 0; t < nt; ++t) {
      const float dec = sdec[t], dt = sdt[t];
      const f2 dec2 = mk2(dec, dec);
      if (STATE) ltot = fmaf(dt, Ah, ltot);
      f2 xd[PR], acc[PR];
#pragma unroll
      for (int r = 0; r < PR; ++r) {
        const float v = sx[t][pl + r] * dt;
        xd[r] = mk2(v, v);
        acc[r] = mk2(0.f, 0.f);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 b4 = *reinterpret_cast<const float4*>(&sB[t][4 * (ln + NL * q)]);
        const f2 bb[2] = {mk2(b4.x, b4.y), mk2(b4.z, b4.w)};
        f2 cc[2];
        if (!STATE) {
          const float4 c4 = *reinterpret_cast<const float4*>(&sC[t][4 * (ln + NL * q)]);
          cc[0] = mk2(c4.x, c4.y);
          cc[1] = mk2(c4.z, c4.w);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int r = 0; r < PR; ++r) {
            S2[r][2 * q + e] = fma2(S2[r][2 * q + e], dec2, mul2(xd[r], bb[e]));
            if (!STATE) acc[r] = fma2(S2[r][2 * q + e], cc[e], acc[r]);
          }
      }
      if (!STATE)
#pragma unroll
        for (int r = 0; r < PR; ++r) {
          float u, v;
          un2(acc[r], u, v);
          u += v;
          if constexpr (PARTS) {
            sy[t][r * SC_THREADS + mine] = ln == 0 ? fmaf(Dh, sx[t][pl + r], u) : u;
          } else {
#pragma unroll
            for (int o = 1; o < NL; o <<= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
            if (ln == 0) sy[t][pl + r] = fmaf(Dh, sx[t][pl + r], u);
          }
        }
    }
    __syncthreads();
    if (!STATE)
#pragma unroll
      for (int k = 0; k < KX; ++k) {
        const int i = threadIdx.x + k * SC_THREADS, t = i / (PB / 8), p = p0 + i % (PB / 8) * 8;
        if (i >= NX || t >= nt) continue;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (PARTS) {
            const int q = i % (PB / 8) * 8 + e;
            f[e] = 0.f;
#pragma unroll
            for (int n = 0; n < NL; n += 4) {
              const float4 v = *reinterpret_cast<const float4*>(&sy[t][q % PR * SC_THREADS + place(q / PR * NL + n)]);
              f[e] += (v.x + v.y) + (v.z + v.w);
            }
          } else {
            f[e] = (&sy[0][0])[8 * i + e];
          }
        }
        store8<T, VEC>(static_cast<T*>(const_cast<void*>(a.y.p)) + at(a.y, t0 + t) + (int64_t)h * a.P + p, pack8<T>(f),
                       min(8, a.P - p));
      }
  }
  float* to = STATE ? sa.ws + (int64_t)(tile + 1) * per_tile : seg == nseg - 1 ? pool : nullptr;
  if (to) {
#pragma unroll
    for (int r = 0; r < PR; ++r)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float u, v;
        un2(S2[r][i], u, v);
        if (on(r, 2 * i)) to[e0 + (int64_t)r * a.N + col(2 * i)] = u;
        if (on(r, 2 * i + 1)) to[e0 + (int64_t)r * a.N + col(2 * i + 1)] = v;
      }
  }
  if (STATE && p0 == 0 && threadIdx.x == 0)
    sa.ws[(int64_t)sa.tiles * per_tile + (int64_t)tile * a.H + h] = ltot * LOG2E;
}

// Workspace entry tile0 + k of a row holds the state that segment k - 1 ended
// with, having started from zero (segment 0: from the row's state).  Turns the
// entries into the states that the segments start with:
//   s_1 = e_1,  s_k = decay_{k-1} s_{k-1} + e_k
// An element a thread; a few entries on their way at a time.
__global__ void __launch_bounds__(256)
ssm_join_kernel(const __grid_constant__ ScanArgs sa) {
  const SsmArgs& a = sa.a;
  const int row = blockIdx.y, len = row_len(a.items[row]);
  const int tile0 = sa.per_row ? row * sa.per_row : a.items[row].tile0;
  const int nseg = len > sa.seg_tokens ? (len + sa.seg_tokens - 1) / sa.seg_tokens : 1;
  const int64_t per_tile = (int64_t)a.H * a.P * a.N, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= per_tile || nseg < 3) return;
  const float* dl = sa.ws + (int64_t)sa.tiles * per_tile + (int64_t)tile0 * a.H + e / (a.P * a.N);
  float* at = sa.ws + (int64_t)(tile0 + 1) * per_tile + e;
  float s = *at;
  constexpr int U = 5;
  for (int k = 2; k < nseg; k += U) {
    float v[U], d[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool on = k + i < nseg;
      v[i] = on ? at[(int64_t)(k + i - 1) * per_tile] : 0.f;
      d[i] = on ? dl[(int64_t)(k + i - 1) * a.H] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (k + i < nseg) {
        s = fmaf(s, exp2f(d[i]), v[i]);
        at[(int64_t)(k + i - 1) * per_tile] = s;
      }
  }
}

thread_local ScanArgs t_scan, t_join;

template <class T, int NL, bool VEC>
cudaError_t go_vec(const ScanArgs& k, bool split, cudaStream_t s) {
  constexpr int PB = SC_THREADS / NL * rows_of(NL);
  const unsigned grid = (unsigned)((int64_t)k.tiles * k.a.H * ((k.a.P + PB - 1) / PB));
  if (split) {
    ssm_scan_kernel<T, NL, true, VEC><<<grid, SC_THREADS, 0, s>>>(k);
    const cudaError_t e = launch_ssm_join(k.a, k.seg_tokens, k.tiles, k.per_row, k.ws, s);
    if (e != cudaSuccess) return e;
  }
  ssm_scan_kernel<T, NL, false, VEC><<<grid, SC_THREADS, 0, s>>>(k);
  return cudaGetLastError();
}
template <class T, int NL>
cudaError_t go(const ScanArgs& k, bool vec, bool split, cudaStream_t s) {
  return vec ? go_vec<T, NL, true>(k, split, s) : go_vec<T, NL, false>(k, split, s);
}
int lanes_of(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : N <= 64 ? 4 : N <= 128 ? 8 : 16; }
template <class T>
cudaError_t go_n(const ScanArgs& k, bool vec, bool split, cudaStream_t s) {
  switch (lanes_of(k.a.N)) {
    case 1: return go<T, 1>(k, vec, split, s);
    case 2: return go<T, 2>(k, vec, split, s);
    case 4: return go<T, 4>(k, vec, split, s);
    case 8: return go<T, 8>(k, vec, split, s);
    default: return go<T, 16>(k, vec, split, s);
  }
}

}  // namespace

cudaError_t launch_ssm_join(const SsmArgs& a, int seg_tokens, int tiles, int per_row, float* ws, cudaStream_t s) {
  ScanArgs& k = t_join;
  k.a = a;
  k.ws = ws;
  k.seg_tokens = seg_tokens;
  k.tiles = tiles;
  k.per_row = per_row;
  const int64_t n = (int64_t)a.H * a.P * a.N;
  ssm_join_kernel<<<dim3((unsigned)((n + 255) / 256), (unsigned)a.rows), 256, 0, s>>>(k);
  return cudaGetLastError();
}

SsmPlan ssm_scan_plan(int H, int P, int N, int rows, const int32_t* lens, int64_t T, int sms) {
  SsmPlan p{};
  const int nl = lanes_of(N), pb = SC_THREADS / nl * rows_of(nl);
  p.units = H * ((P + pb - 1) / pb);
  int64_t longest = 0;
  for (int i = 0; i < rows; ++i) longest = (lens ? lens[i] : T) > longest ? (lens ? lens[i] : T) : longest;
  p.seg_tokens = (int)(longest > 0 ? longest : 1);
  // Segments for a call that would leave most SMs with less than one CTA: two
  // more launches and half the work again, so at least four segments in the
  // longest row, at most 16, of 32 tokens or more.  One row of 4096 tokens of 8
  // heads of 64 x 128: 132 us, 844 whole (125 since chunks have eight tokens); 11 rows of up to 203 tokens of 6 heads
  // of 40 x 72: 33 us, 41 whole.
  for (int64_t seg = (longest + 15) / 16 < 32 ? 32 : (longest + 15) / 16; 4 * seg <= longest; seg += (seg + 3) / 4) {
    int64_t tiles = 0;
    for (int i = 0; i < rows; ++i) {
      const int64_t c = lens ? lens[i] : T;
      tiles += c > seg ? (c + seg - 1) / seg : 1;
    }
    if (tiles * p.units <= 4 * (int64_t)sms) {
      p.seg_tokens = (int)seg;
      p.split = true;
      break;
    }
  }
  return p;
}

cudaError_t launch_ssm_scan(int dtype, bool vec, const SsmArgs& a, const SsmPlan& p, int tiles, int per_row, float* ws,
                            cudaStream_t s) {
  ScanArgs& k = t_scan;
  k.a = a;
  k.ws = ws;
  k.seg_tokens = p.seg_tokens;
  k.tiles = tiles;
  k.per_row = per_row;
  return dtype == T_F32    ? go_n<float>(k, vec, p.split, s)
         : dtype == T_BF16 ? go_n<__nv_bfloat16>(k, vec, p.split, s)
                           : go_n<__half>(k, vec, p.split, s);
}

}  // namespace mx
}  // namespace dl
