// Selective state space scan of bf16 prompts on the 5th-generation tensor cores.
//
// A chunk is Q = 128 tokens.  With S the state at its start, L_i the sum of
// dt_k A over tokens k <= i of the chunk and T_j the sum over tokens k > j,
//   y_i = sum_{j <= i} (C_i . B_j) e^{L_i - L_j} dt_j x_j  +  e^{L_i} S C_i  +  D x_i
//   S'  = e^{L_Q} S + sum_j (e^{T_j} dt_j x_j) B_j^T
// Every factor is at most one for A < 0.  Per chunk, rows being tokens (or
// state columns n for the last), tcgen05 MMAs with fp32 accumulators in TMEM:
//   G  [128 x 128] = C B^T                     exact products of the inputs
//   Y2 [128 x PC]  = C S^T                     S rounded to bf16
//   Y1 [128 x PH]  = W X, per head             W_ij = G_ij e^{L_i - L_j} dt_j rounded to bf16, A in TMEM
//   dS [128 x PC]  = B^T (X1 + X2 + X3)        e^{T_j} dt_j x_j as three bf16 terms (2^-25 of it is left)
// W and the S of Y2 are rounded once, like the output itself (half a step of
// bf16 each); the state keeps 32 bits: it lives in registers in fp32 and its
// increments are formed from all 24 bits.  e^{L_i - L_j} outside the diagonal
// 32 x 32 blocks is the product of a row and a column factor, both at most
// one: e^{L_i - L_b} e^{L_b - L_j}, b the last token of j's block, so only the
// diagonal blocks take an exponential a pair.
//
// One CTA of 256 threads for PC = NH * PH columns: one head of up to 128, or
// NH = 2 heads of up to 64 of one group, over a segment of a row.  B and C of
// the group, X, its terms and S sit in shared memory as 8 x 16-byte core
// matrices (no swizzle), read K-major or MN-major as a product needs, so
// nothing is transposed.  Warps 0-3 form W and write y; warps 4-7 form X's
// terms and carry S.  Rows with few heads are split into segments: a first
// launch (STATE) runs each segment from zero and leaves its end state and
// decay in the workspace, and the full launch joins those before its segment.
#include <cuda_bf16.h>

#include "dl_device.cuh"
#include "mixer_device.cuh"
#include "tc_device.cuh"

namespace dl {
namespace mx {

static __device__ int32_t g_mixer_status;

namespace {

constexpr int Q = 128, TCT = 256;
constexpr uint32_t COL_G = 0, COL_Y1 = 128, COL_Y2 = 256, COL_DS = 384;
constexpr float LOG2E = 1.4426950408889634f;

template <int PC>
struct Smem {
  static constexpr uint32_t TILE = Q * 128 * 2;      // B or C: 128 tokens x 128 state columns
  static constexpr uint32_t XT = Q * PC * 2;         // X, one of its terms, or S (128 state columns x PC)
  static constexpr uint32_t B = 0, C = TILE, X = 2 * TILE, X1 = X + 2 * XT, X2 = X1 + XT,
                            X3 = X2 + XT;            // X doubled; S shares X3's place
  static constexpr uint32_t F = X3 + XT;             // per head [2]: L, column factor
  static constexpr uint32_t FB = 2 * Q * 4;
  static constexpr uint32_t BLK = F + 2 * FB;        // per head and block of 32 tokens: L at its end [8],
                                                     // e^{T} of its last token [8]; per head: T of all tokens [2]
  static constexpr uint32_t BAR = BLK + 80;          // four mbarriers, TMEM address
  static constexpr uint32_t BYTES = BAR + 48;
};
static_assert(Smem<128>::BYTES <= 232448, "shared memory");

__device__ __forceinline__ void cp16z(uint32_t dst, const void* src, bool on) {
  const int n = on ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bar_named(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }

// A token tile [128][CW] of core matrices: byte of (token t, 16-byte piece cv).
template <int CW>
__device__ __forceinline__ uint32_t piece_off(int t, int cv) {
  return (uint32_t)(((t >> 3) * (CW / 8) + cv) * 128 + (t & 7) * 16);
}

// Rows [t0, t0 + nt) x `width` values at src (row stride st) into a tile of
// 128 tokens x CW values from column c0 on, zero where there is no such token
// or value; `n` threads take part.
template <int CW, bool VEC>
__device__ __forceinline__ void load_tile(uint32_t sdst, unsigned char* gdst, const uint16_t* src, int64_t st, int nt,
                                          int width, int c0, int cols, int tid, int n) {
  const int pieces = cols / 8;
#pragma unroll 4
  for (int i = tid; i < Q * pieces; i += n) {
    const int r = i >> 5;                           // a warp: 8 tokens x 4 pieces
    const int per = pieces / 4;
    const int t = (i & 7) + 8 * (r / per), cv = ((i >> 3) & 3) + 4 * (r % per);
    const uint32_t off = piece_off<CW>(t, c0 / 8 + cv);
    const uint16_t* p = src + (int64_t)t * st + cv * 8;
    if (VEC) {
      const bool on = t < nt && cv * 8 < width;
      cp16z(sdst + off, on ? p : src, on);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = cv * 8 + 2 * k;
        const uint32_t lo = t < nt && c < width ? p[2 * k] : 0u, hi = t < nt && c + 1 < width ? p[2 * k + 1] : 0u;
        w[k] = lo | (hi << 16);
      }
      *reinterpret_cast<uint4*>(gdst + off) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

struct TcArgs {
  SsmArgs a;
  float* ws;          // segment states [tiles][H][P][N], then log2 decays [tiles][H]
  int32_t seg_tokens, tiles, per_row, units, ptiles;
};

template <int NH, int PH, bool STATE, bool VEC>
__global__ void __launch_bounds__(TCT, 1)
ssm_tc_kernel(const __grid_constant__ TcArgs ta) {
  constexpr int PC = NH * PH;
  using L = Smem<PC>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const SsmArgs& a = ta.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = warp & 3;
  const bool wg1 = warp >= 4;
  const int tile = blockIdx.x / ta.units, unit = blockIdx.x - tile * ta.units;
  const int row = find_row(a.items, a.rows, tile, ta.per_row);
  const RowItem it = a.items[row];
  const int len = row_len(it);
  const int tile0 = ta.per_row ? row * ta.per_row : it.tile0, seg = tile - tile0;
  const int nseg = len > ta.seg_tokens ? (len + ta.seg_tokens - 1) / ta.seg_tokens : 1;
  if (STATE && seg == nseg - 1) return;             // nothing follows the last segment
  const int hu = unit / ta.ptiles, p0 = (unit - hu * ta.ptiles) * PH;
  const int h0 = hu * NH, g = h0 / (a.H / a.G);
  const int s0 = seg * ta.seg_tokens, s1 = min(len, s0 + ta.seg_tokens);
  const int pw = min(PH, a.P - p0);                 // state rows of a head here
  const int nch = (s1 - s0 + Q - 1) / Q;
  const int nk = (a.N + 15) / 16;                   // K steps over the state columns

  const uint32_t sb = smem_u32(sm);
  float* F = reinterpret_cast<float*>(sm + L::F);
  float* blk = reinterpret_cast<float*>(sm + L::BLK);
  const uint32_t barG = sb + L::BAR, barC = barG + 8, barS = barG + 16, barY = barG + 24;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::BAR + 32);

  if (warp == 0) tc::tmem_alloc(sb + L::BAR + 32, 512);
  if (tid == 0) {
    mbar_init(barG, 1);
    mbar_init(barC, 1);
    mbar_init(barS, 1);
    mbar_init(barY, 1);
    fence_mbar_init();
  }

  auto tok = [&](const TokView& v, int t) { return (int64_t)(it.begin + t) * v.st + (int64_t)row * v.sn; };
  const uint16_t* xg = static_cast<const uint16_t*>(a.x.p) + (int64_t)h0 * a.P + p0;
  const uint16_t* bg = static_cast<const uint16_t*>(a.B.p) + (int64_t)g * a.N;
  const uint16_t* cg = static_cast<const uint16_t*>(a.C.p) + (int64_t)g * a.N;
  auto load_x = [&](int c, int t, int n) {
    const int t0 = s0 + c * Q, nt = min(Q, s1 - t0);
#pragma unroll
    for (int hh = 0; hh < NH; ++hh)
      load_tile<PC, VEC>(sb + L::X + (c & 1) * L::XT, sm + L::X + (c & 1) * L::XT, xg + hh * a.P + tok(a.x, t0), a.x.st,
                         nt, pw, hh * PH, PH, t, n);
  };
  auto load_bc = [&](int c, int t, int n) {
    const int t0 = s0 + c * Q, nt = min(Q, s1 - t0);
    load_tile<128, VEC>(sb + L::B, sm + L::B, bg + tok(a.B, t0), a.B.st, nt, a.N, 0, 128, t, n);
    if (!STATE) load_tile<128, VEC>(sb + L::C, sm + L::C, cg + tok(a.C, t0), a.C.st, nt, a.N, 0, 128, t, n);
  };
  // raw dt of token t (of the segment's row) for head hh of the unit, zero past the segment
  auto raw_dt = [&](int t, int hh) {
    if (t >= s1) return 0.f;
    const int64_t o = tok(a.dt, t) + h0 + hh;
    return a.dt_f32 ? static_cast<const float*>(a.dt.p)[o] : to_f(static_cast<const __nv_bfloat16*>(a.dt.p)[o]);
  };
  // Warps 4, 5 scan head warp - 4 of the unit, four tokens a lane; warps 0-3
  // hold their own token's dt of every head.
  const int sh = warp - 4;
  float raw[4];
  auto load_dt = [&](int c) {
    if (sh >= 0 && sh < NH) {
#pragma unroll
      for (int k = 0; k < 4; ++k) raw[k] = raw_dt(s0 + c * Q + 4 * lane + k, sh);
    } else if (!wg1 && !STATE) {
#pragma unroll
      for (int hh = 0; hh < NH; ++hh) raw[hh] = raw_dt(s0 + c * Q + tid, hh);
    }
  };

  if (nch > 0) {
    load_bc(0, tid, TCT);
    load_x(0, tid, TCT);
    load_dt(0);
  }

  // ---- the state at the segment's start: thread n of warps 4-7 holds S[.][n] of every column
  const int n = tid - 128;
  float S[PC];
  const int64_t per_tile = (int64_t)a.H * a.P * a.N;
  const float* wl = ta.ws + (int64_t)ta.tiles * per_tile;      // log2 decays of the segments
  float* pool = a.state ? a.state + (int64_t)it.slot * per_tile : nullptr;
  auto elem = [&](int col) { return ((int64_t)(h0 + col / PH) * a.P + p0 + col % PH) * a.N + n; };
  if (wg1) {
    const bool mine = n < a.N;
    const float* from = nullptr;
    if (STATE || nseg == 1) from = seg == 0 && pool && !row_fresh(it) ? pool : nullptr;
    else if (seg == 0) from = row_fresh(it) ? nullptr : ta.ws + (int64_t)tile * per_tile;
    else from = ta.ws + (int64_t)(tile0 + 1) * per_tile;
#pragma unroll
    for (int c = 0; c < PC; ++c) S[c] = from && mine && c % PH < pw ? from[elem(c)] : 0.f;
    if (STATE && seg == 0 && from) {
      // the last segment's CTA overwrites the pool's entry in the full launch
#pragma unroll
      for (int c = 0; c < PC; ++c)
        if (mine && c % PH < pw) ta.ws[(int64_t)tile * per_tile + elem(c)] = S[c];
    }
    if (!STATE)
      for (int k = 2; k <= seg; ++k) {
        const float* add = ta.ws + (int64_t)(tile0 + k) * per_tile;
        float d[NH];
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) d[hh] = ex2(wl[(int64_t)(tile0 + k - 1) * a.H + h0 + hh]);
#pragma unroll
        for (int c = 0; c < PC; ++c) S[c] = fmaf(S[c], d[c / PH], mine && c % PH < pw ? add[elem(c)] : 0.f);
      }
  }
  auto store_s = [&]() {          // S as a bf16 operand: K = n, columns contiguous
#pragma unroll
    for (int c8 = 0; c8 < PC / 8; ++c8) {
      const float* s = S + 8 * c8;
      *reinterpret_cast<uint4*>(sm + L::X3 + piece_off<PC>(n, c8)) =
          make_uint4(pack2<__nv_bfloat16>(s[0], s[1]), pack2<__nv_bfloat16>(s[2], s[3]),
                     pack2<__nv_bfloat16>(s[4], s[5]), pack2<__nv_bfloat16>(s[6], s[7]));
    }
  };
  if (!STATE && wg1) store_s();
  float Ah[NH], bias[NH], Dh[NH], ltot[NH];
#pragma unroll
  for (int hh = 0; hh < NH; ++hh) {
    Ah[hh] = a.A[h0 + hh] * LOG2E;
    bias[hh] = a.dt_bias ? a.dt_bias[h0 + hh] : 0.f;
    Dh[hh] = a.D ? a.D[h0 + hh] : 0.f;
    ltot[hh] = 0.f;
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = *tslot;
  const uint32_t tl = tm + ((uint32_t)(32 * q4) << 16);
  bool ok = true;                 // a wait that ran out: no further waits, no results

  // The two groups of warps run loops of their own; the barriers at a chunk's
  // start (operands landed) and end (operands and accumulators free) join them.
  auto chunk_begin = [&]() {
    cp_async_wait_all();
    tc::fence_smem_to_async();    // B, C, X and S for the tensor cores
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  };
  auto chunk_end = [&]() {
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  };
  if (wg1) {
    for (int c = 0; c < nch; ++c) {
      const uint32_t par = (uint32_t)c & 1u;
      const uint32_t xs = L::X + par * L::XT;
      const int nt = min(Q, s1 - s0 - c * Q);
      // ---- decays of the chunk
      if (sh >= 0 && sh < NH) {
        float dt[4], l[4], suf[4];
  #pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float d = raw[k] + bias[sh];
          dt[k] = 4 * lane + k < nt ? (a.softplus ? softplus_f(d) : d) : 0.f;
          l[k] = dt[k] * Ah[sh];
        }
        // tokens after j in its block of 32, summed from the end: no cancellation in the sums that matter
        suf[3] = 0.f;
        suf[2] = l[3];
        suf[1] = suf[2] + l[2];
        suf[0] = suf[1] + l[1];
        float post = suf[0] + l[0];
  #pragma unroll
        for (int k = 1; k < 4; ++k) l[k] += l[k - 1];
        float pre = l[3];
  #pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          const float d = __shfl_down_sync(0xffffffffu, post, o, 8);
          if ((lane & 7) + o < 8) post += d;
        }
  #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float u = __shfl_up_sync(0xffffffffu, pre, o);
          if (lane >= o) pre += u;
        }
        const float before = pre - l[3];
        const float nxt = __shfl_down_sync(0xffffffffu, post, 1, 8);
        const float after = (lane & 7) < 7 ? nxt : 0.f;
        const float t1 = __shfl_sync(0xffffffffu, post, 8), t2 = __shfl_sync(0xffffffffu, post, 16),
                    t3 = __shfl_sync(0xffffffffu, post, 24), t0b = __shfl_sync(0xffffffffu, post, 0);
        float* f = F + sh * 2 * Q;
  #pragma unroll
        for (int k = 0; k < 4; ++k) {
          f[4 * lane + k] = before + l[k];
          f[Q + 4 * lane + k] = ex2(after + suf[k]) * dt[k];
        }
        if ((lane & 7) == 7) blk[sh * 4 + (lane >> 3)] = pre;
        if (lane < 4) blk[8 + sh * 4 + lane] = ex2(lane == 0 ? t3 + t2 + t1 : lane == 1 ? t3 + t2 : lane == 2 ? t3 : 0.f);
        if (lane == 0) blk[16 + sh] = t3 + t2 + t1 + t0b;
      }
      if (c + 1 < nch) load_dt(c + 1);
      chunk_begin();
      // ---- X's three terms, then S' = e^{L_Q} S + dS
      auto terms = [&](int pass) {
#pragma unroll 4
        for (int e = 0; e < PC / 8; ++e) {
          const int i = n + e * 128, r = i >> 5, per = PC / 32;
          const int t = (i & 7) + 8 * (r / per), cv = ((i >> 3) & 3) + 4 * (r % per);
          const uint32_t off = piece_off<PC>(t, cv);
          const uint4 xv = *reinterpret_cast<const uint4*>(sm + xs + off);
          const float f = F[(cv * 8 / PH) * 2 * Q + Q + t] * blk[8 + (cv * 8 / PH) * 4 + (t >> 5)];
          const uint32_t w[4] = {xv.x, xv.y, xv.z, xv.w};
          uint32_t o1[4], o2[4], o3[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float u = __uint_as_float(w[k] << 16) * f, v = __uint_as_float(w[k] & 0xffff0000u) * f;
            o1[k] = pack2<__nv_bfloat16>(u, v);
            u -= __uint_as_float(o1[k] << 16);
            v -= __uint_as_float(o1[k] & 0xffff0000u);
            o2[k] = pack2<__nv_bfloat16>(u, v);
            u -= __uint_as_float(o2[k] << 16);
            v -= __uint_as_float(o2[k] & 0xffff0000u);
            o3[k] = pack2<__nv_bfloat16>(u, v);
          }
          if (pass == 0) {
            *reinterpret_cast<uint4*>(sm + L::X1 + off) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
            *reinterpret_cast<uint4*>(sm + L::X2 + off) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
          } else {
            *reinterpret_cast<uint4*>(sm + L::X3 + off) = make_uint4(o3[0], o3[1], o3[2], o3[3]);
          }
        }
      };
      terms(0);
      if (!STATE) ok = ok && mbar_wait(barC, par, &g_mixer_status, DEV_TIMEOUT_MMA);   // Y2 has read S
      terms(1);
      tc::fence_smem_to_async();
      tc::fence_before_sync();
      bar_named(2);
      if (n == 0) {
        tc::fence_after_sync();
        constexpr uint32_t idS = tc::idesc_bf16_f32(128, PC, true, true);
#pragma unroll 1
        for (int term = 0; term < 3; ++term)
          for (int k = 0; k < Q / 16; ++k)
            tc::mma_bf16(tm + COL_DS, tc::sdesc(sb + L::B + k * 4096u, 2048u, 128u),
                         tc::sdesc(sb + L::X1 + term * L::XT + (uint32_t)k * (2 * PC * 16), PC * 16, 128u), idS,
                         term + k > 0);
        tc::mma_commit(barS);
      }
      ok = ok && mbar_wait(barS, par, &g_mixer_status, DEV_TIMEOUT_MMA);
      tc::fence_after_sync();
      if (c + 1 < nch) load_bc(c + 1, n, 128);      // dS (and G, Y2 before it) have read B and C
      float dec[NH];
#pragma unroll
      for (int hh = 0; hh < NH; ++hh) {
        dec[hh] = ex2(blk[16 + hh]);
        ltot[hh] += blk[16 + hh];
      }
#pragma unroll
      for (int c32 = 0; c32 < PC / 32; ++c32) {
        uint32_t r[32];
        tc::tmem_ld32(tl + COL_DS + 32 * c32, r);
        tc::tmem_wait_ld(r);
#pragma unroll
        for (int e = 0; e < 32; ++e)
          S[32 * c32 + e] = fmaf(S[32 * c32 + e], dec[32 * c32 / PH], __uint_as_float(r[e]));
      }
      if (!STATE && c + 1 < nch) store_s();
      chunk_end();
    }
    if (ok) {
      float* to = STATE ? ta.ws + (int64_t)(tile + 1) * per_tile : seg == nseg - 1 ? pool : nullptr;
      if (to) {
  #pragma unroll
        for (int c = 0; c < PC; ++c)
          if (n < a.N && c % PH < pw) to[elem(c)] = S[c];
      }
      if (STATE && n == 0 && p0 == 0) {
        float* out = ta.ws + (int64_t)ta.tiles * per_tile + (int64_t)tile * a.H + h0;
  #pragma unroll
        for (int hh = 0; hh < NH; ++hh) out[hh] = ltot[hh];
      }
    }
  } else {
    for (int c = 0; c < nch; ++c) {
      const uint32_t par = (uint32_t)c & 1u;
      const uint32_t xs = L::X + par * L::XT;
      const int t0 = s0 + c * Q, nt = min(Q, s1 - t0);
      float own[NH];                // warps 0-3: dt of token i = tid
  #pragma unroll
      for (int hh = 0; hh < NH; ++hh) {
        const float d = raw[hh] + bias[hh];
        own[hh] = tid < nt ? (a.softplus ? softplus_f(d) : d) : 0.f;
      }
      if (c + 1 < nch) load_dt(c + 1);
      chunk_begin();
      if (!STATE && tid == 0) {
        constexpr uint32_t idG = tc::idesc_bf16_f32(128, 128), idY = tc::idesc_bf16_f32(128, PC, false, true);
        for (int k = 0; k < nk; ++k)
          tc::mma_bf16(tm + COL_G, tc::sdesc(sb + L::C + k * 256u, 128u, 2048u),
                       tc::sdesc(sb + L::B + k * 256u, 128u, 2048u), idG, k > 0);
        tc::mma_commit(barG);
        for (int k = 0; k < nk; ++k)
          tc::mma_bf16(tm + COL_Y2, tc::sdesc(sb + L::C + k * 256u, 128u, 2048u),
                       tc::sdesc(sb + L::X3 + (uint32_t)k * (2 * PC * 16), PC * 16, 128u), idY, k > 0);
        tc::mma_commit(barC);
      }
      if (c + 1 < nch) load_x(c + 1, tid, 128);
      if (!STATE) {
        // ---- W from G, in place of G
        const int i = tid;
        ok = ok && mbar_wait(barG, par, &g_mixer_status, DEV_TIMEOUT_MMA);
        tc::fence_after_sync();
        float G[Q];
  #pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b <= q4) {
            uint32_t r[32];
            tc::tmem_ld32(tl + COL_G + 32 * b, r);
            tc::tmem_wait_ld(r);
  #pragma unroll
            for (int e = 0; e < 32; ++e) G[32 * b + e] = __uint_as_float(r[e]);
          }
  #pragma unroll
        for (int hh = 0; hh < NH; ++hh) {
          const float* f = F + hh * 2 * Q;
          const float li = f[i];
  #pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t w[16];
            if (b < q4) {
              const float rf = ex2(li - blk[hh * 4 + b]);
  #pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 cf = *reinterpret_cast<const float4*>(f + Q + 32 * b + 4 * e);
                w[2 * e] = pack2<__nv_bfloat16>(G[32 * b + 4 * e] * (rf * cf.x), G[32 * b + 4 * e + 1] * (rf * cf.y));
                w[2 * e + 1] =
                    pack2<__nv_bfloat16>(G[32 * b + 4 * e + 2] * (rf * cf.z), G[32 * b + 4 * e + 3] * (rf * cf.w));
              }
            } else if (b == q4) {
  #pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int j = 32 * b + 2 * e;
                const float2 lj = *reinterpret_cast<const float2*>(f + j);
                const float d0 = __shfl_sync(0xffffffffu, own[hh], 2 * e), d1 = __shfl_sync(0xffffffffu, own[hh], 2 * e + 1);
                w[e] = pack2<__nv_bfloat16>(j <= i ? G[j] * (ex2(li - lj.x) * d0) : 0.f,
                                            j + 1 <= i ? G[j + 1] * (ex2(li - lj.y) * d1) : 0.f);
              }
            } else {
  #pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = 0u;
            }
            tc::tmem_st16(tl + COL_G + 64 * hh + 16 * b, w);
          }
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        bar_named(1);
        if (tid == 0) {
          tc::fence_after_sync();
          constexpr uint32_t id1 = tc::idesc_bf16_f32(128, PH, false, true);
  #pragma unroll
          for (int hh = 0; hh < NH; ++hh)
  #pragma unroll
            for (int k = 0; k < Q / 16; ++k)
              tc::mma_bf16_ta(tm + COL_Y1 + hh * PH, tm + COL_G + 64 * hh + 8 * k,
                              tc::sdesc(sb + xs + (uint32_t)hh * (PH * 16) + (uint32_t)k * (2 * PC * 16), PC * 16, 128u), id1,
                              k > 0);
          tc::mma_commit(barY);
        }
        // ---- y = Y1 + e^{L_i} Y2 + D x
        ok = ok && mbar_wait(barC, par, &g_mixer_status, DEV_TIMEOUT_MMA);
        ok = ok && mbar_wait(barY, par, &g_mixer_status, DEV_TIMEOUT_MMA);
        tc::fence_after_sync();
        uint16_t* yr = static_cast<uint16_t*>(const_cast<void*>(a.y.p)) + tok(a.y, t0 + i) + (int64_t)h0 * a.P + p0;
  #pragma unroll
        for (int c32 = 0; c32 < PC / 32; ++c32) {
          constexpr int per = PH / 32;
          const int hh = c32 / per, pc = 32 * (c32 % per);
          uint32_t r1[32], r2[32];
          tc::tmem_ld32(tl + COL_Y1 + 32 * c32, r1);
          tc::tmem_ld32(tl + COL_Y2 + 32 * c32, r2);
          tc::tmem_wait_ld(r1);
          tc::tmem_wait_ld(r2);
          const float el = ex2(F[hh * 2 * Q + i]);
  #pragma unroll
          for (int e8 = 0; e8 < 4; ++e8) {
            const uint4 xv = *reinterpret_cast<const uint4*>(sm + xs + piece_off<PC>(i, 4 * c32 + e8));
            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
            uint32_t o[4];
  #pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 8 * e8 + 2 * k;
              o[k] = pack2<__nv_bfloat16>(
                  fmaf(Dh[hh], __uint_as_float(xw[k] << 16), fmaf(el, __uint_as_float(r2[e]), __uint_as_float(r1[e]))),
                  fmaf(Dh[hh], __uint_as_float(xw[k] & 0xffff0000u),
                       fmaf(el, __uint_as_float(r2[e + 1]), __uint_as_float(r1[e + 1]))));
            }
            if (i < nt && ok) {
              uint16_t* p = yr + (int64_t)hh * a.P + pc + 8 * e8;
              const int left = pw - (pc + 8 * e8);
              if (VEC) {
                if (left > 0) *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
              } else {
  #pragma unroll
                for (int k = 0; k < 8; ++k)
                  if (k < left) p[k] = (uint16_t)(o[k >> 1] >> (16 * (k & 1)));
              }
            }
          }
        }
      }
      chunk_end();
    }
  }

  if (!__syncthreads_and(ok)) {    // let what was issued land before the memory is given back
    if (tid == 0 && nch > 0) {
      mbar_drain(barS, (uint32_t)(nch - 1) & 1u);
      if (!STATE) mbar_drain(barY, (uint32_t)(nch - 1) & 1u);
    }
    __syncthreads();
  }
  if (warp == 0) tc::tmem_dealloc(tm, 512);
}

thread_local TcArgs t_tc;

template <int NH, int PH, bool STATE, bool VEC>
cudaError_t go(const TcArgs& t, cudaStream_t s) {
  constexpr int BYTES = (int)Smem<NH * PH>::BYTES;
  static thread_local int ready = -1;              // the device whose limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready != dev) {
    e = cudaFuncSetAttribute(ssm_tc_kernel<NH, PH, STATE, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
    if (e != cudaSuccess) return e;
    ready = dev;
  }
  ssm_tc_kernel<NH, PH, STATE, VEC><<<(unsigned)t.tiles * (unsigned)t.units, TCT, BYTES, s>>>(t);
  return cudaGetLastError();
}
template <int NH, int PH, bool VEC>
cudaError_t both(const TcArgs& t, bool split, cudaStream_t s) {
  if (split) {
    const cudaError_t e = go<NH, PH, true, VEC>(t, s);
    if (e != cudaSuccess) return e;
  }
  return go<NH, PH, false, VEC>(t, s);
}

}  // namespace

SsmPlan ssm_tc_plan(int H, int G, int P, int N, int rows, const int32_t* lens, int64_t T, int sms) {
  SsmPlan p{};
  (void)N;
  p.ph = P > 64 ? 128 : 64;
  p.ptiles = (P + p.ph - 1) / p.ph;
  int64_t chunks = 0, longest = 0;
  for (int i = 0; i < rows; ++i) {
    const int64_t c = ((lens ? lens[i] : T) + Q - 1) / Q;
    chunks += c > 0 ? c : 1;
    longest = c > longest ? c : longest;
  }
  const int64_t base = (int64_t)rows * H * p.ptiles;
  p.nh = p.ph == 64 && (H / G) % 2 == 0 && base >= 2 * (int64_t)sms ? 2 : 1;
  p.units = H / p.nh * p.ptiles;
  p.seg_tokens = Q * (int)(longest > 0 ? longest : 1);
  // Segments as short as still fill the GPU once: each runs two launches, so
  // at least three of them in the longest row are wanted, and at most 16,
  // since the last of a row joins the states of all before it.
  for (int64_t seg = (longest + 15) / 16; seg > 0 && 3 * seg <= longest; ++seg) {
    int64_t tiles = 0;
    for (int i = 0; i < rows; ++i) {
      const int64_t c = ((lens ? lens[i] : T) + Q - 1) / Q;
      tiles += c > seg ? (c + seg - 1) / seg : 1;
    }
    if (tiles * p.units <= sms) {
      p.seg_tokens = (int)(Q * seg);
      p.split = true;
      break;
    }
  }
  return p;
}

cudaError_t launch_ssm_tc(bool vec, const SsmArgs& a, const SsmPlan& p, int tiles, int per_row, float* ws,
                          cudaStream_t s) {
  TcArgs& t = t_tc;
  t.a = a;
  t.ws = ws;
  t.seg_tokens = p.seg_tokens;
  t.tiles = tiles;
  t.per_row = per_row;
  t.units = p.units;
  t.ptiles = p.ptiles;
  if (p.ph == 128) return vec ? both<1, 128, true>(t, p.split, s) : both<1, 128, false>(t, p.split, s);
  if (p.nh == 2) return vec ? both<2, 64, true>(t, p.split, s) : both<2, 64, false>(t, p.split, s);
  return vec ? both<1, 64, true>(t, p.split, s) : both<1, 64, false>(t, p.split, s);
}

cudaError_t read_mixer_status(cudaStream_t s, int32_t* code) {
  cudaError_t e = cudaStreamSynchronize(s);
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(code, g_mixer_status, sizeof *code);
  if (e == cudaSuccess && *code != 0) {
    const int32_t zero = 0;
    e = cudaMemcpyToSymbol(g_mixer_status, &zero, sizeof zero);
  }
  return e;
}

}  // namespace mx
}  // namespace dl
