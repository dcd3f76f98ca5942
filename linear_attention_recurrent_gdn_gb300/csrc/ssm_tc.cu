// Selective state space scan of bf16 prompts on the 5th-generation tensor cores.
//
// A chunk is Q = 128 tokens.  With S the state at its start, L_i the sum of
// dt_k A over tokens k <= i of the chunk and T_j the sum over tokens k > j,
//   y_i = sum_{j <= i} (C_i . B_j) e^{L_i - L_j} dt_j x_j  +  e^{L_i} S C_i  +  D x_i
//   S'  = e^{L_Q} S + sum_j (e^{T_j} dt_j x_j) B_j^T
// Every factor is at most one for A < 0.  Per chunk and PC = 64 rows p of the
// state, rows of a product being tokens (state columns n for the last), tcgen05
// MMAs with fp32 accumulators in TMEM:
//   G  [128 x 128] = C B^T               exact products of the inputs
//   Y2 [128 x 64]  = C S^T               S rounded to bf16
//   Y1 [128 x 64]  = W X                 W_ij = G_ij e^{L_i - L_j} dt_j rounded to bf16, A in TMEM
//   dS [128 x 192] = B^T [X1 X2 X3]      e^{T_j} dt_j x_j as three bf16 terms (2^-25 of it is left)
// W and the S of Y2 are rounded once, like the output itself (half a step of
// bf16 each); the state keeps 32 bits: it lives in registers in fp32 and its
// increments are formed from all 24 bits, the terms' sums side by side in one
// product: fewer and wider MMAs.  e^{L_i - L_j} outside
// the diagonal 32 x 32 blocks is the product of a row and a column factor, both
// at most one: e^{L_i - L_b} e^{L_b - L_j}, b the last token of j's block, so
// only the diagonal blocks take an exponential a pair.
//
// A persistent CTA of 16 warps takes units: one head's 64 state rows over a
// segment of a row.  B and C of the group, X, its terms and S sit in shared
// memory as rows of 64 values in the 128-byte swizzle, read K-major or MN-major
// as a product needs, so nothing is transposed; tensor copies bring B, C and X a
// chunk ahead, across units too (and, but for a row's ragged last chunk, take y
// away).  Warps 0-7 form W and y, warps 8-15 X's terms; all of them hold the
// state, a quarter of the columns each.  With nearly all of the SM's memory
// used as shared memory there is next to no L1 cache, so nothing may spill: 128
// rows a unit, or two heads, measured slower for that.
//
// Rows with few heads are split into segments: a first launch (STATE) runs
// each segment from zero and leaves its end state and decay in the workspace,
// and the full launch joins those before its segment.
#include <cuda.h>
#include <cuda_bf16.h>

#include "dl_device.cuh"
#include "mixer_device.cuh"
#include "tc_device.cuh"

namespace dl {
namespace mx {

static __device__ int32_t g_mixer_status;

namespace {

constexpr int Q = 128, PC = 64, TCT = 512;
constexpr int HC = PC / 2;        // columns of one of the two warps of a lane quarter in a group of warps
constexpr int SC = PC / 4;        // state columns of one of the four warps of a lane quarter
constexpr uint32_t COL_G = 0, COL_W = 128, COL_Y1 = 192, COL_Y2 = 256, COL_DS = 320;
constexpr uint32_t BLK64 = Q * 128;                  // bytes of 128 rows of 64 values
constexpr float LOG2E = 1.4426950408889634f;

// Shared memory; B, C, X and the decays are doubled (even and odd chunks).
struct Sm {
  static constexpr uint32_t TILE = 2 * BLK64;        // B or C: 128 tokens x 128 state columns
  static constexpr uint32_t B = 0, C = 2 * TILE, X = 4 * TILE, X1 = X + 2 * BLK64, S = X1 + 3 * BLK64;
  static constexpr uint32_t F = S + BLK64;           // L [128], column factors [128], L at the blocks' ends [4],
  static constexpr uint32_t FB = (2 * Q + 12) * 4;   // e^{T} of the blocks' last tokens [4], log2 of the chunk's decay
  static constexpr uint32_t BAR = F + 2 * FB;        // twelve mbarriers, TMEM address
  static constexpr uint32_t BYTES = BAR + 112;
};
static_assert(Sm::BYTES <= 232448, "shared memory");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bar_named(int id) { asm volatile("bar.sync %0, 256;" ::"r"(id) : "memory"); }
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_store(const CUtensorMap* m, int c0, int c1, int c2, int c3, uint32_t src) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(m),
               "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(src)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// Byte of (row r, 16-byte piece cv) of a tile of 128 rows.
__device__ __forceinline__ uint32_t piece_off(int r, int cv) {
  return (uint32_t)(cv >> 3) * BLK64 + (uint32_t)(r * 128 + (((cv & 7) ^ (r & 7)) << 4));
}
// Descriptors of K step k (16 values of K): rows are K (MN-major), or K runs along the rows (K-major).
__device__ __forceinline__ uint64_t k_rows(uint32_t base, int k) { return tc::sdesc128(base + k * 2048u, BLK64, 1024u); }
__device__ __forceinline__ uint64_t k_cols(uint32_t base, int k) {
  return tc::sdesc128(base + (uint32_t)(k >> 2) * BLK64 + (uint32_t)(k & 3) * 32u, 16u, 1024u);
}

struct TcArgs {
  CUtensorMap mx, mb, mc, my;   // x, B, C, y: [64 values][head or group][128 tokens][row] boxes
  SsmArgs a;
  float* ws;                    // segment states [tiles][H][P][N], then log2 decays [tiles][H]
  int32_t seg_tokens, tiles, per_row, units, ptiles, total, empty_rows;
};

// One unit of work: tokens [s0, s1) of a row (a segment) for 64 state rows from p0 of head h.
struct Unit {
  int tile, row, begin, h, p0, s0, s1, chunks;
};
__device__ __forceinline__ Unit unit_at(const TcArgs& ta, int u) {
  const SsmArgs& a = ta.a;
  Unit w;
  w.tile = u / ta.units;
  const int k = u - w.tile * ta.units;
  w.row = find_row(a.items, a.rows, w.tile, ta.per_row);
  const RowItem it = a.items[w.row];
  const int len = row_len(it), seg = w.tile - (ta.per_row ? w.row * ta.per_row : it.tile0);
  w.begin = it.begin;
  w.h = k / ta.ptiles;
  w.p0 = (k - w.h * ta.ptiles) * PC;
  w.s0 = seg * ta.seg_tokens;
  w.s1 = min(len, w.s0 + ta.seg_tokens);
  w.chunks = (w.s1 - w.s0 + Q - 1) / Q;
  return w;
}
// Segments of the unit's row before it and in all.
__device__ __forceinline__ void segments(const TcArgs& ta, const Unit& w, int& seg, int& nseg) {
  const RowItem it = ta.a.items[w.row];
  const int len = row_len(it);
  seg = w.tile - (ta.per_row ? w.row * ta.per_row : it.tile0);
  nseg = len > ta.seg_tokens ? (len + ta.seg_tokens - 1) / ta.seg_tokens : 1;
}
// Whether a launch leaves a unit out: STATE leaves out last segments, which nothing follows.
template <bool STATE>
__device__ __forceinline__ bool skipped(const TcArgs& ta, const Unit& w) {
  if (!STATE) return w.chunks == 0;
  int seg, nseg;
  segments(ta, w, seg, nseg);
  return seg == nseg - 1;
}
// The first unit from u on (in steps of the grid) that has work; u moves there, or past the last.
template <bool STATE>
__device__ __forceinline__ Unit next_unit(const TcArgs& ta, int& u) {
  Unit w{};
  for (; u < ta.total; u += gridDim.x) {
    w = unit_at(ta, u);
    if (!skipped<STATE>(ta, w)) break;
  }
  return w;
}
// (Not inlined: the loops below have to stay in the instruction cache.)
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t par) {
  return mbar_wait(bar, par, &g_mixer_status, DEV_TIMEOUT_MMA);
}

// TMA: tensor copies (16-byte aligned tensors, widths and strides); else
// threads copy value by value.
template <bool STATE, bool TMA>
__global__ void __launch_bounds__(TCT, 1)
ssm_tc_kernel(const __grid_constant__ TcArgs ta) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const SsmArgs& a = ta.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = warp & 3, hf = (warp >> 2) & 1, cg = warp >> 2;
  const bool wgb = warp >= 8;
  const int i = 32 * q4 + lane;                     // this thread's token row; its state column n
  const int nk = (a.N + 15) / 16;                   // K steps over the state columns

  const uint32_t sb = smem_u32(sm);
  auto decays = [&](uint32_t k) { return reinterpret_cast<float*>(sm + Sm::F + (k & 1) * Sm::FB); };
  const uint32_t barG = sb + Sm::BAR, barC = barG + 8, barS = barG + 16, barY = barG + 24, fullB = barG + 32,
                 fullC = barG + 48, fullX = barG + 64, readyS = barG + 80, readyF = barG + 88;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + Sm::BAR + 96);

  if (warp == 0) tc::tmem_alloc(sb + Sm::BAR + 96, 512);
  if (tid == 0) {
    // products: one commit; loads: one thread's tensor copies, or the eight warps that copy; S: every warp;
    // the decays: one warp
    for (int k = 0; k < 4; ++k) mbar_init(barG + 8 * k, 1);
    for (int k = 4; k < 10; ++k) mbar_init(barG + 8 * k, TMA ? 1 : 8);
    mbar_init(readyS, TCT / 32);
    mbar_init(readyF, 1);
    fence_mbar_init();
  }

  auto tok = [&](const Unit& w, const TokView& v, int t) { return (int64_t)(w.begin + t) * v.st + (int64_t)w.row * v.sn; };
  auto arrive_warp = [&](uint32_t bar) {            // this warp's writes to shared memory are done
    tc::fence_smem_to_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  auto copy_rows = [&](uint32_t dst, const uint16_t* src, int64_t st, int nt, int width, int cols) {
#pragma unroll 1
    for (int e = tid - 256; e < Q * cols / 8; e += 256) {
      const int r = e & (Q - 1), cv = e / Q;
      const uint16_t* p = src + (int64_t)r * st + cv * 8;
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = cv * 8 + 2 * k;
        const uint32_t lo = r < nt && c < width ? p[2 * k] : 0u, hi = r < nt && c + 1 < width ? p[2 * k + 1] : 0u;
        v[k] = lo | (hi << 16);
      }
      *reinterpret_cast<uint4*>(sm + dst + piece_off(r, cv)) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  };
  // Chunk c of unit w, number k of all, into its buffers.  TMA: one thread calls; else warps 8-15 copy.
  auto load = [&](const Unit& w, int c, uint32_t k) {
    const uint32_t b = k & 1;
    const int t0 = w.s0 + c * Q, g = w.h / (a.H / a.G);
    const uint32_t xd = Sm::X + b * BLK64, bd = Sm::B + b * Sm::TILE, cd = Sm::C + b * Sm::TILE;
    const uint32_t fx = fullX + 8 * b, fb = fullB + 8 * b, fc = fullC + 8 * b;
    if (TMA) {
      mbar_arrive_expect_tx(fx, BLK64);
      tma_load(sb + xd, &ta.mx, w.p0, w.h, w.begin + t0, a.x.sn ? w.row : 0, fx);
      const int nb = a.N > 64 ? 2 : 1;
      mbar_arrive_expect_tx(fb, nb * BLK64);
      for (int e = 0; e < nb; ++e) tma_load(sb + bd + e * BLK64, &ta.mb, 64 * e, g, w.begin + t0, a.B.sn ? w.row : 0, fb);
      if (!STATE) {
        mbar_arrive_expect_tx(fc, nb * BLK64);
        for (int e = 0; e < nb; ++e) tma_load(sb + cd + e * BLK64, &ta.mc, 64 * e, g, w.begin + t0, a.C.sn ? w.row : 0, fc);
      }
    } else {
      const int nt = min(Q, w.s1 - t0);
      const uint16_t* xp = static_cast<const uint16_t*>(a.x.p) + (int64_t)w.h * a.P + w.p0;
      copy_rows(xd, xp + tok(w, a.x, t0), a.x.st, nt, min(PC, a.P - w.p0), PC);
      arrive_warp(fx);
      copy_rows(bd, static_cast<const uint16_t*>(a.B.p) + (int64_t)g * a.N + tok(w, a.B, t0), a.B.st, nt, a.N, 128);
      arrive_warp(fb);
      if (!STATE) {
        copy_rows(cd, static_cast<const uint16_t*>(a.C.p) + (int64_t)g * a.N + tok(w, a.C, t0), a.C.st, nt, a.N, 128);
        arrive_warp(fc);
      }
    }
  };
  // dt of token t (past the segment: its last one), as it sits in memory: the conversion waits for the load,
  // so it is left to the use
  auto raw_dt = [&](const Unit& w, int t) -> uint32_t {
    const int64_t o = tok(w, a.dt, min(t, w.s1 - 1)) + w.h;
    return a.dt_f32 ? static_cast<const uint32_t*>(a.dt.p)[o] : static_cast<const uint16_t*>(a.dt.p)[o];
  };
  auto dt_of = [&](uint32_t raw, float bias) {
    const float d = __uint_as_float(a.dt_f32 ? raw : raw << 16) + bias;
    return a.softplus ? softplus_f(d) : d;
  };

  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = *tslot;
  const uint32_t tl = tm + ((uint32_t)(32 * q4) << 16);
  bool ok = true;                 // a wait that ran out: no further waits, no results
  auto wait = [&](uint32_t bar, uint32_t par) {
    if (ok && !mbar_try_wait(bar, par & 1u)) ok = wait_long(bar, par & 1u);
  };
  auto wait2 = [&](uint32_t bar, uint32_t k) { wait(bar + 8 * (k & 1), k >> 1); };   // one of a pair
  const int64_t per_tile = (int64_t)a.H * a.P * a.N;

  // ---- the state: this thread holds S[column cg * SC + .][n = i] of the unit
  float S[SC];
  auto elem0 = [&](const Unit& w) { return ((int64_t)w.h * a.P + w.p0 + cg * SC) * a.N + i; };
  auto live_of = [&](const Unit& w) { return i < a.N ? a.P - w.p0 - cg * SC : 0; };
  auto pool_of = [&](const Unit& w) { return a.state ? a.state + (int64_t)a.items[w.row].slot * per_tile : nullptr; };
  auto load_state = [&](const Unit& w) {
    int seg, nseg;
    segments(ta, w, seg, nseg);
    const bool fresh = row_fresh(a.items[w.row]);
    const int64_t e0 = elem0(w);
    const int live = live_of(w);
    const float* from;
    if (STATE || nseg == 1) from = seg == 0 && !fresh ? pool_of(w) : nullptr;
    else if (seg == 0) from = fresh ? nullptr : ta.ws + (int64_t)w.tile * per_tile;
    else from = ta.ws + (int64_t)(w.tile - seg + 1) * per_tile;
#pragma unroll
    for (int c = 0; c < SC; ++c) S[c] = from && c < live ? from[e0 + (int64_t)c * a.N] : 0.f;
    if (STATE && seg == 0 && from) {
      // the last segment's CTA overwrites the pool's entry in the full launch
      float* to = ta.ws + (int64_t)w.tile * per_tile + e0;
#pragma unroll
      for (int c = 0; c < SC; ++c)
        if (c < live) to[(int64_t)c * a.N] = S[c];
    }
    if (!STATE)
#pragma unroll 1
      for (int k = 2; k <= seg; ++k) {
        const float* add = ta.ws + (int64_t)(w.tile - seg + k) * per_tile + e0;
        const float d = ex2(ta.ws[(int64_t)ta.tiles * per_tile + (int64_t)(w.tile - seg + k - 1) * a.H + w.h]);
#pragma unroll
        for (int c = 0; c < SC; ++c) S[c] = fmaf(S[c], d, c < live ? add[(int64_t)c * a.N] : 0.f);
      }
  };
  auto leave_state = [&](const Unit& w, float ltot) {
    int seg, nseg;
    segments(ta, w, seg, nseg);
    const int64_t e0 = elem0(w);
    const int live = live_of(w);
    float* to = STATE ? ta.ws + (int64_t)(w.tile + 1) * per_tile : seg == nseg - 1 ? pool_of(w) : nullptr;
    if (!ok) return;
    if (to) {
#pragma unroll
      for (int c = 0; c < SC; ++c)
        if (c < live) to[e0 + (int64_t)c * a.N] = S[c];
    }
    if (STATE && tid == 0 && w.p0 == 0)
      ta.ws[(int64_t)ta.tiles * per_tile + (int64_t)w.tile * a.H + w.h] = ltot;
  };
  auto share_state = [&]() {      // S as a bf16 operand (rows n, columns contiguous), and its TMEM place is read
    if (!STATE) {
#pragma unroll
      for (int c8 = 0; c8 < SC / 8; ++c8) {
        const float* s = S + 8 * c8;
        *reinterpret_cast<uint4*>(sm + Sm::S + piece_off(i, cg * (SC / 8) + c8)) =
            make_uint4(pack2<__nv_bfloat16>(s[0], s[1]), pack2<__nv_bfloat16>(s[2], s[3]),
                       pack2<__nv_bfloat16>(s[4], s[5]), pack2<__nv_bfloat16>(s[6], s[7]));
      }
    }
    tc::fence_before_sync();
    arrive_warp(readyS);
  };
  auto update_state = [&](float decl) {             // S' = e^{L_Q} S + dS, the small terms first
    const float dec = ex2(decl);
    uint32_t r1[16], r2[16], r3[16];
    tc::tmem_ld16(tl + COL_DS + cg * SC, r1);
    tc::tmem_ld16(tl + COL_DS + PC + cg * SC, r2);
    tc::tmem_ld16(tl + COL_DS + 2 * PC + cg * SC, r3);
    tc::tmem_wait_ld16(r1);
    tc::tmem_wait_ld16(r2);
    tc::tmem_wait_ld16(r3);
#pragma unroll
    for (int e = 0; e < 16; ++e)
      S[e] = fmaf(S[e], dec, (__uint_as_float(r3[e]) + __uint_as_float(r2[e])) + __uint_as_float(r1[e]));
  };

  // Rows without tokens: a fresh one's state is zero.
  if (!STATE && ta.empty_rows)
#pragma unroll 1
    for (int e = blockIdx.x; e < ta.total; e += gridDim.x) {
      const Unit v = unit_at(ta, e);
      float* to = pool_of(v);
      if (v.chunks == 0 && to && row_fresh(a.items[v.row]))
#pragma unroll 1
        for (int c = 0; c < SC && c < live_of(v); ++c) to[elem0(v) + (int64_t)c * a.N] = 0.f;
    }

  int u = blockIdx.x;
  Unit w = next_unit<STATE>(ta, u);
  bool any = u < ta.total;
  if (any && (TMA ? tid == 32 : wgb)) load(w, 0, 0);
  uint32_t gc = 0;                // chunks done, over all units

  // The two groups of warps run loops of their own, joined by barriers in
  // shared memory, so that one chunk's y is written while the next one's terms
  // are formed.  Each barrier's phase is a chunk (gc counts them; the pairs' a
  // chunk of their parity).  A parity tells two phases apart, so nothing may
  // complete two phases while somebody still waits for the first:
  //   products  a chunk's dS, Y2 (and with it Y1 and the next G) need the S that
  //             every warp shares, after its waits for the chunk before
  //   decays    of chunk k + 1 are published after Y2 (STATE: dS) of chunk k,
  //             which needs warps 0-7 to have seen those of chunk k
  //   loads     of chunk k + 2 follow warps 0-7's (STATE: 8-15's) chunk k
  const int bt = tid - 256;
  const bool scans = warp == 8;                     // four tokens a lane
  // dt of the next chunk: the scanning warp's four tokens, the others' own token
  uint32_t raw[4];
  float bias = 0.f, Ah = 0.f;
  auto load_dt = [&](const Unit& v, int c) {
    if (wgb && !scans) return;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (scans || (k == 0 && !STATE)) raw[k] = raw_dt(v, v.s0 + c * Q + (scans ? 4 * lane + k : i));
    Ah = a.A[v.h];
    bias = a.dt_bias ? a.dt_bias[v.h] : 0.f;
  };
  // decays of chunk number k with nt tokens, from raw
  auto scan = [&](uint32_t k2, int nt) {
    float dt[4], l[4], suf[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dt[k] = 4 * lane + k < nt ? dt_of(raw[k], bias) : 0.f;
      l[k] = dt[k] * (Ah * LOG2E);
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
      const float v = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += v;
    }
    const float before = pre - l[3];
    const float nxt = __shfl_down_sync(0xffffffffu, post, 1, 8);
    const float after = (lane & 7) < 7 ? nxt : 0.f;
    float bs[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) bs[b] = __shfl_sync(0xffffffffu, post, 8 * b);
    float* f = decays(k2);
    *reinterpret_cast<float4*>(f + 4 * lane) = make_float4(before + l[0], before + l[1], before + l[2], pre);
    *reinterpret_cast<float4*>(f + Q + 4 * lane) =
        make_float4(ex2(after + suf[0]) * dt[0], ex2(after + suf[1]) * dt[1], ex2(after + suf[2]) * dt[2],
                    ex2(after + suf[3]) * dt[3]);
    if ((lane & 7) == 7) f[2 * Q + (lane >> 3)] = pre;
    if (lane < 4)
      f[2 * Q + 4 + lane] = ex2(lane == 0 ? bs[3] + bs[2] + bs[1] : lane == 1 ? bs[3] + bs[2] : lane == 2 ? bs[3] : 0.f);
    if (lane == 0) f[2 * Q + 8] = bs[3] + bs[2] + bs[1] + bs[0];
    __syncwarp();
    if (lane == 0) mbar_arrive(readyF);
  };
  // G and Y2 of chunk number k, once their operands are there.
  auto issue_g = [&](uint32_t k) {
    wait2(fullB, k);
    wait2(fullC, k);
    tc::fence_after_sync();
    constexpr uint32_t idG = tc::idesc_bf16_f32(128, 128);
    const uint32_t bo = sb + Sm::B + (k & 1) * Sm::TILE, co = sb + Sm::C + (k & 1) * Sm::TILE;
#pragma unroll 1
    for (int j = 0; j < nk; ++j) tc::mma_bf16(tm + COL_G, k_cols(co, j), k_cols(bo, j), idG, j > 0);
    tc::mma_commit(barG);
  };
  auto issue_y2 = [&](uint32_t k) {
    wait(readyS, k);
    tc::fence_after_sync();
    constexpr uint32_t idY = tc::idesc_bf16_f32(128, PC, false, true);
    const uint32_t co = sb + Sm::C + (k & 1) * Sm::TILE;
#pragma unroll 1
    for (int j = 0; j < nk; ++j) tc::mma_bf16(tm + COL_Y2, k_cols(co, j), k_rows(sb + Sm::S, j), idY, j > 0);
    tc::mma_commit(barC);
  };
  // A ragged chunk (number k, nt tokens) brought by tensor copies: what lies behind its last token is cleared
  // in B and X by the `n` threads from t on.  (C's rows there give rows of y that are not kept.)
  auto clear_tail = [&](uint32_t k, int nt, int t) {
    wait2(fullB, k);
    if (!STATE) wait2(fullX, k);
#pragma unroll 1
    for (int e = t; e < (Q - nt) * (STATE ? 16 : 24); e += 256) {
      const int r = nt + e % (Q - nt), cv = e / (Q - nt);
      const uint32_t off = cv < 16 ? Sm::B + (k & 1) * Sm::TILE + piece_off(r, cv)
                                   : Sm::X + (k & 1) * BLK64 + piece_off(r, cv - 16);
      *reinterpret_cast<uint4*>(sm + off) = make_uint4(0u, 0u, 0u, 0u);
    }
    tc::fence_smem_to_async();
  };
  if (any) {
    load_dt(w, 0);
    if (scans) scan(0, w.s1 - w.s0);
    wait(readyF, 0);
    __syncthreads();
  }
  bool early = false;             // this chunk's G was issued in the chunk before
#pragma unroll 1
  while (any) {
    int un = u + gridDim.x;
    const Unit wn = next_unit<STATE>(ta, un);
    const bool another = un < ta.total;
    load_state(w);
    share_state();
    float ltot = 0.f;
    if (wgb) {
#pragma unroll 1
      for (int c = 0; c < w.chunks; ++c, ++gc) {
        const int nt = min(Q, w.s1 - w.s0 - c * Q);
        const bool last = c + 1 == w.chunks, more = !last || another;
        const Unit wf = last ? wn : w;              // the chunk after this one
        const int cf = last ? 0 : c + 1;
        if (TMA && STATE && more && bt == 0) load(wf, cf, gc + 1);   // the chunk before is done with the buffers
        if (more) load_dt(wf, cf);
        const float* f = decays(gc);
        const uint32_t xs = Sm::X + (gc & 1) * BLK64;
        wait(readyF, gc);
        wait2(fullX, gc);
        // ---- X's three terms, then dS
        const float decl = f[2 * Q + 8];
#pragma unroll
        for (int e = 0; e < Q * PC / 8 / 256; ++e) {
          const int idx = bt + e * 256, t = idx >> 3, cv = idx & 7;
          const uint32_t off = piece_off(t, cv);
          uint4 xv = *reinterpret_cast<const uint4*>(sm + xs + off);
          if (t >= nt) xv = make_uint4(0u, 0u, 0u, 0u);     // a tensor copy brings what lies behind the row
          const float g = f[Q + t] * f[2 * Q + 4 + (t >> 5)];
          const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
          uint32_t o1[4], o2[4], o3[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float p = __uint_as_float(xw[k] << 16) * g, q = __uint_as_float(xw[k] & 0xffff0000u) * g;
            o1[k] = pack2<__nv_bfloat16>(p, q);
            p -= __uint_as_float(o1[k] << 16);
            q -= __uint_as_float(o1[k] & 0xffff0000u);
            o2[k] = pack2<__nv_bfloat16>(p, q);
            p -= __uint_as_float(o2[k] << 16);
            q -= __uint_as_float(o2[k] & 0xffff0000u);
            o3[k] = pack2<__nv_bfloat16>(p, q);
          }
          *reinterpret_cast<uint4*>(sm + Sm::X1 + off) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
          *reinterpret_cast<uint4*>(sm + Sm::X1 + BLK64 + off) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
          *reinterpret_cast<uint4*>(sm + Sm::X1 + 2 * BLK64 + off) = make_uint4(o3[0], o3[1], o3[2], o3[3]);
        }
        if (STATE && TMA && nt < Q) clear_tail(gc, nt, bt);
        tc::fence_smem_to_async();
        bar_named(2);
        if (bt == 0) {
          wait(readyS, gc);                         // every warp has read the dS before
          if (STATE || nt == Q) wait2(fullB, gc);
          else wait(barC, gc);                      // ragged: cleared before G and Y2
          tc::fence_after_sync();
          constexpr uint32_t idS = tc::idesc_bf16_f32(128, 3 * PC, true, true);
          const uint32_t bo = sb + Sm::B + (gc & 1) * Sm::TILE;
#pragma unroll 1
          for (int k = 0; k < Q / 16; ++k) tc::mma_bf16(tm + COL_DS, k_rows(bo, k), k_rows(sb + Sm::X1, k), idS, k > 0);
          tc::mma_commit(barS);
        }
        // Y2 done: S may be overwritten.  It was issued after warps 0-7 were done with the chunk before, whose
        // decays and buffers are free
        if (!STATE) wait(barC, gc);
        else wait(barS, gc);
        if (!TMA && more) load(wf, cf, gc + 1);
        if (more && scans) scan(gc + 1, wf.s1 - wf.s0 - cf * Q);
        wait(barS, gc);
        tc::fence_after_sync();
        ltot += decl;
        update_state(decl);
        if (!last) share_state();
      }
    } else {
#pragma unroll 1
      for (int c = 0; c < w.chunks; ++c, ++gc) {
        const int t0 = w.s0 + c * Q, nt = min(Q, w.s1 - t0);
        const bool last = c + 1 == w.chunks, more = !last || another;
        const Unit wf = last ? wn : w;              // the chunk after this one
        const int cf = last ? 0 : c + 1;
        const float* f = decays(gc);
        if (STATE) {
          const float decl = f[2 * Q + 8];
          wait(barS, gc);
          tc::fence_after_sync();
          ltot += decl;
          update_state(decl);
          if (more) wait(readyF, gc + 1);
          if (!last) share_state();
          continue;
        }
        const uint32_t xs = Sm::X + (gc & 1) * BLK64;
        // ---- this chunk's G and Y2, and the next one's operands
        if (TMA && more && tid == 32) {
          bulk_wait_read();                         // y of the chunk before has left its buffer
          load(wf, cf, gc + 1);
        }
        if (TMA && nt < Q) {
          clear_tail(gc, nt, tid);
          bar_named(1);
        }
        if (tid == 0) {
          if (!early) issue_g(gc);
          issue_y2(gc);
        }
        early = false;
        const float own = i < nt ? dt_of(raw[0], bias) : 0.f;     // dt of token i
        if (more) load_dt(wf, cf);
        // ---- W from G: columns 32 b + 16 hf .. + 15 of every block b
        wait2(fullX, gc);
        wait(barG, gc);
        tc::fence_after_sync();
        const float decl = f[2 * Q + 8], li = f[i];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int j0 = 32 * b + 16 * hf;
          uint32_t v[8], G[16];
          if (b <= q4) {
            tc::tmem_ld16(tl + COL_G + j0, G);
            tc::tmem_wait_ld16(G);
          }
          if (b < q4) {
            const float rf = ex2(li - f[2 * Q + b]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 cf4 = *reinterpret_cast<const float4*>(f + Q + j0 + 4 * e);
              v[2 * e] = pack2<__nv_bfloat16>(__uint_as_float(G[4 * e]) * (rf * cf4.x),
                                              __uint_as_float(G[4 * e + 1]) * (rf * cf4.y));
              v[2 * e + 1] = pack2<__nv_bfloat16>(__uint_as_float(G[4 * e + 2]) * (rf * cf4.z),
                                                  __uint_as_float(G[4 * e + 3]) * (rf * cf4.w));
            }
          } else if (b == q4) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int j = j0 + 2 * e;
              const float2 lj = *reinterpret_cast<const float2*>(f + j);
              const float d0 = __shfl_sync(0xffffffffu, own, 16 * hf + 2 * e),
                          d1 = __shfl_sync(0xffffffffu, own, 16 * hf + 2 * e + 1);
              v[e] = pack2<__nv_bfloat16>(j <= i ? __uint_as_float(G[2 * e]) * (ex2(li - lj.x) * d0) : 0.f,
                                          j + 1 <= i ? __uint_as_float(G[2 * e + 1]) * (ex2(li - lj.y) * d1) : 0.f);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0u;
          }
          tc::tmem_st8(tl + COL_W + 16 * b + 8 * hf, v);
        }
        tc::tmem_wait_st();
        tc::fence_before_sync();
        bar_named(1);             // W is formed, G has been read
        if (tid == 0) {
          tc::fence_after_sync();
          constexpr uint32_t id1 = tc::idesc_bf16_f32(128, PC, false, true);
#pragma unroll 1
          for (int k = 0; k < Q / 16; ++k)
            tc::mma_bf16_ta(tm + COL_Y1, tm + COL_W + 8 * k, k_rows(sb + xs, k), id1, k > 0);
          tc::mma_commit(barY);
          // the next chunk's G, if its operands are there
          if (more && wf.s1 - wf.s0 - cf * Q >= Q && mbar_try_wait(fullB + 8 * ((gc + 1) & 1), ((gc + 1) >> 1) & 1u) &&
              mbar_try_wait(fullC + 8 * ((gc + 1) & 1), ((gc + 1) >> 1) & 1u)) {
            issue_g(gc + 1);
            early = true;
          }
        }
        wait(barC, gc);
        wait(barS, gc);
        tc::fence_after_sync();
        update_state(decl);
        if (!last) share_state();
        wait(barY, gc);
        tc::fence_after_sync();
        // ---- y = Y1 + e^{L_i} Y2 + D x, over x in shared memory (its terms are formed)
        const float ei = ex2(li), Dh = a.D ? a.D[w.h] : 0.f;
        const bool direct = !TMA || nt < Q;
#pragma unroll
        for (int c16 = 0; c16 < HC / 16; ++c16) {
          uint32_t r1[16], r2[16];
          tc::tmem_ld16(tl + COL_Y1 + hf * HC + 16 * c16, r1);
          tc::tmem_ld16(tl + COL_Y2 + hf * HC + 16 * c16, r2);
          tc::tmem_wait_ld16(r1);
          tc::tmem_wait_ld16(r2);
#pragma unroll
          for (int e8 = 0; e8 < 2; ++e8) {
            uint4* xp = reinterpret_cast<uint4*>(sm + xs + piece_off(i, hf * (HC / 8) + 2 * c16 + e8));
            const uint4 xv = *xp;
            const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int e = 8 * e8 + 2 * k;
              o[k] = pack2<__nv_bfloat16>(
                  fmaf(Dh, __uint_as_float(xw[k] << 16), fmaf(ei, __uint_as_float(r2[e]), __uint_as_float(r1[e]))),
                  fmaf(Dh, __uint_as_float(xw[k] & 0xffff0000u),
                       fmaf(ei, __uint_as_float(r2[e + 1]), __uint_as_float(r1[e + 1]))));
            }
            *xp = make_uint4(o[0], o[1], o[2], o[3]);
          }
        }
        if (more) wait(readyF, gc + 1);             // before the next Y2, after which the decays after those come
        tc::fence_smem_to_async();
        tc::fence_before_sync();
        bar_named(1);             // y is in shared memory, and its accumulators are free
        if (!direct) {
          if (tid == 32 && ok) {
            tma_store(&ta.my, w.p0, w.h, w.begin + t0, a.y.sn ? w.row : 0, sb + xs);
            bulk_commit();
          }
        } else {
          // a ragged chunk's rows (or unaligned ones), value by value
          uint16_t* yr = static_cast<uint16_t*>(const_cast<void*>(a.y.p)) + tok(w, a.y, t0) + (int64_t)w.h * a.P + w.p0;
          const int pw = min(PC, a.P - w.p0);
          if (ok)
#pragma unroll 1
            for (int e = tid; e < nt * PC; e += 256) {
              const int t = e / PC, p = e % PC;
              if (p < pw)
                yr[(int64_t)t * a.y.st + p] =
                    *reinterpret_cast<const uint16_t*>(sm + xs + piece_off(t, p >> 3) + 2 * (p & 7));
            }
          bar_named(1);           // read before the buffer is filled again
        }
      }
    }
    leave_state(w, ltot);
    u = un;
    w = wn;
    any = another;
  }
  if (TMA && !STATE && tid == 32) bulk_wait();
  if (!__syncthreads_and(ok)) {    // let what was issued land before the memory is given back
    if (tid == 0 && gc > 0) {
      mbar_drain(barS, (gc - 1) & 1u);
      if (!STATE) mbar_drain(barY, (gc - 1) & 1u);
    }
    __syncthreads();
  }
  if (warp == 0) tc::tmem_dealloc(tm, 512);
}

thread_local TcArgs t_tc;

template <bool STATE, bool TMA>
cudaError_t go(const TcArgs& t, int sms, cudaStream_t s) {
  static thread_local int ready = -1;              // the device whose limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready != dev) {
    e = cudaFuncSetAttribute(ssm_tc_kernel<STATE, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Sm::BYTES);
    if (e != cudaSuccess) return e;
    ready = dev;
  }
  ssm_tc_kernel<STATE, TMA><<<(unsigned)(t.total < sms ? t.total : sms), TCT, Sm::BYTES, s>>>(t);
  return cudaGetLastError();
}
template <bool TMA>
cudaError_t both(const TcArgs& t, bool split, int sms, cudaStream_t s) {
  if (split) {
    const cudaError_t e = go<true, TMA>(t, sms, s);
    if (e != cudaSuccess) return e;
  }
  return go<false, TMA>(t, sms, s);
}

using EncodeFn = decltype(&cuTensorMapEncodeTiled);
EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return (EncodeFn) nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}
// A bf16 token tensor [row][token][head][width] as boxes of 64 values x 128 tokens in the 128-byte swizzle.
bool encode(CUtensorMap* m, const TokView& v, int width, int heads, int64_t tokens, int rows) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)(v.sn ? rows : 1)};
  const cuuint64_t strides[3] = {(cuuint64_t)width * 2, (cuuint64_t)v.st * 2, (cuuint64_t)(v.sn ? v.sn : v.st) * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)Q, 1}, one[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(v.p), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

SsmPlan ssm_tc_plan(int H, int P, int rows, const int32_t* lens, int64_t T, int sms) {
  SsmPlan p{};
  p.sms = sms;
  p.ptiles = (P + PC - 1) / PC;
  int64_t longest = 0;
  for (int i = 0; i < rows; ++i) {
    const int64_t c = ((lens ? lens[i] : T) + Q - 1) / Q;
    longest = c > longest ? c : longest;
  }
  p.units = H * p.ptiles;
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

cudaError_t launch_ssm_tc(bool vec, int64_t tokens, const SsmArgs& a, const SsmPlan& p, int tiles, int per_row,
                          float* ws, cudaStream_t s) {
  TcArgs& t = t_tc;
  t.a = a;
  t.ws = ws;
  t.seg_tokens = p.seg_tokens;
  t.tiles = tiles;
  t.per_row = per_row;
  t.units = p.units;
  t.ptiles = p.ptiles;
  t.total = tiles * p.units;
  t.empty_rows = 0;
  for (int i = 0; i < a.rows; ++i) t.empty_rows |= row_len(a.items[i]) == 0;
  const bool tma = vec && encode(&t.mx, a.x, a.P, a.H, tokens, a.rows) && encode(&t.mb, a.B, a.N, a.G, tokens, a.rows) &&
                   encode(&t.mc, a.C, a.N, a.G, tokens, a.rows) && encode(&t.my, a.y, a.P, a.H, tokens, a.rows);
  return tma ? both<true>(t, p.split, p.sms, s) : both<false>(t, p.split, p.sms, s);
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
