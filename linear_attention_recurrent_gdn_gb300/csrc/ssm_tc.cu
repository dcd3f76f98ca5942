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
// A persistent CTA of 512 threads takes units of PC = NH * PH columns: one
// head of up to 128, or NH = 2 heads of up to 64 of one group, over a segment
// of a row.  B and C of the group, X, its terms and S sit in shared memory as
// rows of 64 values in the 128-byte swizzle, read K-major or MN-major as a
// product needs, so nothing is transposed; tensor copies bring them (and, but
// for a row's ragged last chunk, take y away), the next chunk's as soon as a
// buffer is free, across units too.  Warps 0-7 form W and y, warps 8-15 X's
// terms and the state, two warps to a lane quarter in each, half of the
// columns each.
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

constexpr int Q = 128, TCT = 512;
constexpr uint32_t COL_G = 0, COL_Y1 = 128, COL_Y2 = 256, COL_DS = 384;
constexpr uint32_t BLK64 = Q * 128;                  // bytes of 128 rows of 64 values
constexpr float LOG2E = 1.4426950408889634f;

template <int PC>
struct Smem {
  static constexpr uint32_t TILE = 2 * BLK64;        // B or C: 128 tokens x 128 state columns
  static constexpr uint32_t XT = PC / 64 * BLK64;    // X, one of its terms, or S (128 state columns x PC)
  static constexpr uint32_t B = 0, C = TILE, X = 2 * TILE, X1 = X + 2 * XT, X2 = X1 + XT,
                            X3 = X2 + XT;            // X doubled; S shares X3's place
  static constexpr uint32_t F = X3 + XT;             // per head [2]: L, column factor
  static constexpr uint32_t FB = 2 * Q * 4;
  static constexpr uint32_t BLK = F + 2 * FB;        // per head and block of 32 tokens: L at its end [8],
                                                     // e^{T} of its last token [8]; per head: T of all tokens [2]
  static constexpr uint32_t BAR = BLK + 80;          // eight mbarriers, TMEM address
  static constexpr uint32_t BYTES = BAR + 80;
};
static_assert(Smem<128>::BYTES <= 232448, "shared memory");

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

struct TcArgs {
  CUtensorMap mx, mb, mc, my;   // x, B, C, y: [64 values][head or group][128 tokens][row] boxes
  SsmArgs a;
  float* ws;                    // segment states [tiles][H][P][N], then log2 decays [tiles][H]
  int32_t seg_tokens, tiles, per_row, units, ptiles, total;
};

// One unit of work: a segment of a row for one or two heads.
struct Unit {
  int row, tile, tile0, seg, nseg, h0, p0, g, s0, s1, nch;
  RowItem it;
};
template <int NH, int PH, bool STATE>
__device__ __forceinline__ Unit unit_at(const TcArgs& ta, int u) {
  const SsmArgs& a = ta.a;
  Unit w;
  w.tile = u / ta.units;
  const int k = u - w.tile * ta.units, hu = k / ta.ptiles;
  w.row = find_row(a.items, a.rows, w.tile, ta.per_row);
  w.it = a.items[w.row];
  const int len = row_len(w.it);
  w.tile0 = ta.per_row ? w.row * ta.per_row : w.it.tile0;
  w.seg = w.tile - w.tile0;
  w.nseg = len > ta.seg_tokens ? (len + ta.seg_tokens - 1) / ta.seg_tokens : 1;
  w.h0 = hu * NH;
  w.p0 = (k - hu * ta.ptiles) * PH;
  w.g = w.h0 / (a.H / a.G);
  w.s0 = w.seg * ta.seg_tokens;
  w.s1 = min(len, w.s0 + ta.seg_tokens);
  w.nch = STATE && w.seg == w.nseg - 1 ? 0 : (w.s1 - w.s0 + Q - 1) / Q;   // nothing follows the last segment
  return w;
}
// The first unit from u on that has tokens, or one past the last.
template <int NH, int PH, bool STATE>
__device__ __forceinline__ int next_unit(const TcArgs& ta, int u, int step) {
  while (u < ta.total && unit_at<NH, PH, STATE>(ta, u).nch == 0) u += step;
  return u;
}

// TMA: tensor copies (16-byte aligned tensors, widths and strides); else
// threads copy value by value.
template <int NH, int PH, bool STATE, bool TMA>
__global__ void __launch_bounds__(TCT, 1)
ssm_tc_kernel(const __grid_constant__ TcArgs ta) {
  constexpr int PC = NH * PH, HC = PC / 2;          // columns of a unit, and of one of two warps of a lane quarter
  using L = Smem<PC>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const SsmArgs& a = ta.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = warp & 3, hf = (warp >> 2) & 1;
  const bool wgb = warp >= 8;
  const int i = 32 * q4 + lane;                     // token row (warps 0-7), state column n (warps 8-15)
  const int nk = (a.N + 15) / 16;                   // K steps over the state columns

  const uint32_t sb = smem_u32(sm);
  float* F = reinterpret_cast<float*>(sm + L::F);
  float* blk = reinterpret_cast<float*>(sm + L::BLK);
  const uint32_t barG = sb + L::BAR, barC = barG + 8, barS = barG + 16, barY = barG + 24, fullB = barG + 32,
                 fullC = barG + 40, fullX = barG + 48;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + L::BAR + 64);

  if (warp == 0) tc::tmem_alloc(sb + L::BAR + 64, 512);
  if (tid == 0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) mbar_init(barG + 8 * k, 1);
    fence_mbar_init();
  }

  auto tok = [&](const Unit& w, const TokView& v, int t) {
    return (int64_t)(w.it.begin + t) * v.st + (int64_t)w.row * v.sn;
  };
  // Chunk c of unit w into the buffers.  TMA: one thread issues; else `n` threads copy.
  auto copy_rows = [&](uint32_t dst, const uint16_t* src, int64_t st, int nt, int width, int cols, int t, int n) {
    for (int e = t; e < Q * cols / 8; e += n) {
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
  auto load_x = [&](const Unit& w, int c, uint32_t buf, int t, int n) {
    const int t0 = w.s0 + c * Q;
    if (TMA) {
      const uint32_t bar = fullX + 8 * buf;
      mbar_arrive_expect_tx(bar, L::XT);
#pragma unroll
      for (int b = 0; b < PC / 64; ++b)
        tma_load(sb + L::X + buf * L::XT + b * BLK64, &ta.mx, w.p0 + (NH == 1 ? 64 * b : 0), w.h0 + (NH == 1 ? 0 : b),
                 w.it.begin + t0, a.x.sn ? w.row : 0, bar);
    } else {
#pragma unroll
      for (int hh = 0; hh < NH; ++hh)
        copy_rows(L::X + buf * L::XT + hh * BLK64,
                  static_cast<const uint16_t*>(a.x.p) + (int64_t)(w.h0 + hh) * a.P + w.p0 + tok(w, a.x, t0), a.x.st,
                  min(Q, w.s1 - t0), min(PH, a.P - w.p0), PH, t, n);
    }
  };
  auto load_bc = [&](const Unit& w, int c, bool isb, int t, int n) {
    const int t0 = w.s0 + c * Q;
    const TokView& v = isb ? a.B : a.C;
    const uint32_t dst = isb ? L::B : L::C;
    if (TMA) {
      const uint32_t bar = isb ? fullB : fullC;
      const int nb = a.N > 64 ? 2 : 1;
      mbar_arrive_expect_tx(bar, nb * BLK64);
      for (int b = 0; b < nb; ++b)
        tma_load(sb + dst + b * BLK64, isb ? &ta.mb : &ta.mc, 64 * b, w.g, w.it.begin + t0, v.sn ? w.row : 0, bar);
    } else {
      copy_rows(dst, static_cast<const uint16_t*>(v.p) + (int64_t)w.g * a.N + tok(w, v, t0), v.st,
                min(Q, w.s1 - t0), a.N, 128, t, n);
    }
  };
  // raw dt of token t for head hh of the unit, zero past its segment
  auto raw_dt = [&](const Unit& w, int t, int hh) {
    if (t >= w.s1) return 0.f;
    const int64_t o = tok(w, a.dt, t) + w.h0 + hh;
    return a.dt_f32 ? static_cast<const float*>(a.dt.p)[o] : to_f(static_cast<const __nv_bfloat16*>(a.dt.p)[o]);
  };
  auto step_of = [&](float raw, int h) {
    const float d = raw + (a.dt_bias ? a.dt_bias[h] : 0.f);
    return a.softplus ? softplus_f(d) : d;
  };

  int u = blockIdx.x, cur = next_unit<NH, PH, STATE>(ta, u, gridDim.x);
  if (cur < ta.total) {
    const Unit w = unit_at<NH, PH, STATE>(ta, cur);
    if (!TMA) {
      load_bc(w, 0, true, tid, TCT);
      if (!STATE) load_bc(w, 0, false, tid, TCT);
      load_x(w, 0, 0, tid, TCT);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (TMA && tid == 0 && cur < ta.total) {
    const Unit w = unit_at<NH, PH, STATE>(ta, cur);
    load_bc(w, 0, true, 0, 1);
    if (!STATE) load_bc(w, 0, false, 0, 1);
    load_x(w, 0, 0, 0, 1);
  }
  const uint32_t tm = *tslot;
  const uint32_t tl = tm + ((uint32_t)(32 * q4) << 16);
  bool ok = true;                 // a wait that ran out: no further waits, no results
  auto wait = [&](uint32_t bar, uint32_t par) {
    ok = ok && mbar_wait(bar, par, &g_mixer_status, DEV_TIMEOUT_MMA);
  };
  uint32_t gc = 0;                // chunks done, over all units
  const int64_t per_tile = (int64_t)a.H * a.P * a.N;

  // The two groups of warps run loops of their own; the barriers at a chunk's
  // start (operands landed) and end (operands and accumulators free) join them.
  auto chunk_begin = [&](int nt) {
    if (TMA) {
      wait(fullB, gc & 1);
      if (!STATE) wait(fullC, gc & 1);
      wait(fullX + 8 * (gc & 1), (gc >> 1) & 1);
      if (nt < Q) {
        // what lies behind the row's last token is not zero: clear it (C's rows give y rows that are not kept)
        for (int e = tid; e < (Q - nt) * (16 + PC / 8); e += TCT) {
          const int r = nt + e % (Q - nt), cv = e / (Q - nt);
          const uint32_t off = cv < 16 ? L::B + piece_off(r, cv) : L::X + (gc & 1) * L::XT + piece_off(r, cv - 16);
          *reinterpret_cast<uint4*>(sm + off) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    tc::fence_smem_to_async();    // what threads wrote of B, C, X and S, for the tensor cores
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
  };
  auto chunk_end = [&]() {
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    ++gc;
  };

  if (wgb) {
    const int bt = tid - 256;
    const bool scans = warp - 8 < NH;               // warps 8, 9 scan head warp - 8, four tokens a lane
    const int sh = warp - 8;
    float raw[4];
    auto load_dt = [&](const Unit& w, int c) {
      if (scans) {
#pragma unroll
        for (int k = 0; k < 4; ++k) raw[k] = raw_dt(w, w.s0 + c * Q + 4 * lane + k, sh);
      }
    };
    // decays of chunk c, from raw
    auto scan = [&](const Unit& w, int c) {
      if (!scans) return;
      const int nt = w.s1 - w.s0 - c * Q;
      const float Ah = a.A[w.h0 + sh] * LOG2E;
      float dt[4], l[4], suf[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        dt[k] = 4 * lane + k < nt ? step_of(raw[k], w.h0 + sh) : 0.f;
        l[k] = dt[k] * Ah;
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
      float* f = F + sh * 2 * Q;
      *reinterpret_cast<float4*>(f + 4 * lane) = make_float4(before + l[0], before + l[1], before + l[2], pre);
      *reinterpret_cast<float4*>(f + Q + 4 * lane) =
          make_float4(ex2(after + suf[0]) * dt[0], ex2(after + suf[1]) * dt[1], ex2(after + suf[2]) * dt[2],
                      ex2(after + suf[3]) * dt[3]);
      if ((lane & 7) == 7) blk[sh * 4 + (lane >> 3)] = pre;
      if (lane < 4)
        blk[8 + sh * 4 + lane] = ex2(lane == 0 ? bs[3] + bs[2] + bs[1] : lane == 1 ? bs[3] + bs[2] : lane == 2 ? bs[3] : 0.f);
      if (lane == 0) blk[16 + sh] = bs[3] + bs[2] + bs[1] + bs[0];
    };
    float S[HC];                                    // S[column hf * HC + .][n = i]
    auto store_s = [&]() {                          // as a bf16 operand: rows n, columns contiguous
#pragma unroll
      for (int c8 = 0; c8 < HC / 8; ++c8) {
        const float* s = S + 8 * c8;
        *reinterpret_cast<uint4*>(sm + L::X3 + piece_off(i, hf * (HC / 8) + c8)) =
            make_uint4(pack2<__nv_bfloat16>(s[0], s[1]), pack2<__nv_bfloat16>(s[2], s[3]),
                       pack2<__nv_bfloat16>(s[4], s[5]), pack2<__nv_bfloat16>(s[6], s[7]));
      }
    };
    if (cur < ta.total) {
      const Unit w = unit_at<NH, PH, STATE>(ta, cur);
      load_dt(w, 0);
      scan(w, 0);
    }
    for (; u < ta.total; u += gridDim.x) {
      const Unit w = unit_at<NH, PH, STATE>(ta, u);
      if (STATE && w.seg == w.nseg - 1) continue;
      const int nxt = w.nch ? next_unit<NH, PH, STATE>(ta, u + gridDim.x, gridDim.x) : 0;
      const Unit wn = w.nch && nxt < ta.total ? unit_at<NH, PH, STATE>(ta, nxt) : w;
      // ---- the state at the segment's start
      const float* wl = ta.ws + (int64_t)ta.tiles * per_tile;      // log2 decays of the segments
      float* pool = a.state ? a.state + (int64_t)w.it.slot * per_tile : nullptr;
      // columns [hf * HC, + HC): offset of the first one's element n = i, and how many there are
      const int hcol = NH == 2 ? hf : 0, pcol = w.p0 + (NH == 2 ? 0 : hf * HC);
      const int64_t e0 = ((int64_t)(w.h0 + hcol) * a.P + pcol) * a.N + i;
      const int live = i < a.N ? a.P - pcol : 0;
      {
        const float* from;
        if (STATE || w.nseg == 1) from = w.seg == 0 && pool && !row_fresh(w.it) ? pool : nullptr;
        else if (w.seg == 0) from = row_fresh(w.it) ? nullptr : ta.ws + (int64_t)w.tile * per_tile;
        else from = ta.ws + (int64_t)(w.tile0 + 1) * per_tile;
#pragma unroll
        for (int c = 0; c < HC; ++c) S[c] = from && c < live ? from[e0 + (int64_t)c * a.N] : 0.f;
        if (STATE && w.seg == 0 && from) {
          // the last segment's CTA overwrites the pool's entry in the full launch
#pragma unroll
          for (int c = 0; c < HC; ++c)
            if (c < live) ta.ws[(int64_t)w.tile * per_tile + e0 + (int64_t)c * a.N] = S[c];
        }
        if (!STATE)
          for (int k = 2; k <= w.seg; ++k) {
            const float* add = ta.ws + (int64_t)(w.tile0 + k) * per_tile + e0;
            const float d = ex2(wl[(int64_t)(w.tile0 + k - 1) * a.H + w.h0 + hcol]);
#pragma unroll
            for (int c = 0; c < HC; ++c) S[c] = fmaf(S[c], d, c < live ? add[(int64_t)c * a.N] : 0.f);
          }
      }
      if (!STATE && w.nch) store_s();
      float ltot = 0.f;
      for (int c = 0; c < w.nch; ++c) {
        const uint32_t par = gc & 1u;
        const uint32_t xs = L::X + par * L::XT;
        const bool last = c + 1 == w.nch, more = !last || nxt < ta.total;
        const Unit& wf = last ? wn : w;             // the chunk after this one
        const int cf = last ? 0 : c + 1;
        if (more) load_dt(wf, cf);
        chunk_begin(min(Q, w.s1 - w.s0 - c * Q));
        // ---- X's three terms, then S' = e^{L_Q} S + dS
        const float decl = blk[16 + hcol];
        constexpr int PIECES = Q * PC / 8 / 256;
        uint32_t o3[PIECES][4];
#pragma unroll
        for (int e = 0; e < PIECES; ++e) {
          const int idx = bt + e * 256, t = (idx >> 3) & (Q - 1), cv = (idx & 7) + 8 * (idx >> 10);
          const uint32_t off = piece_off(t, cv);
          const uint4 xv = *reinterpret_cast<const uint4*>(sm + xs + off);
          const int hh = NH == 2 ? cv >> 3 : 0;
          const float f = F[hh * 2 * Q + Q + t] * blk[8 + hh * 4 + (t >> 5)];
          const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
          uint32_t o1[4], o2[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float p = __uint_as_float(xw[k] << 16) * f, q = __uint_as_float(xw[k] & 0xffff0000u) * f;
            o1[k] = pack2<__nv_bfloat16>(p, q);
            p -= __uint_as_float(o1[k] << 16);
            q -= __uint_as_float(o1[k] & 0xffff0000u);
            o2[k] = pack2<__nv_bfloat16>(p, q);
            p -= __uint_as_float(o2[k] << 16);
            q -= __uint_as_float(o2[k] & 0xffff0000u);
            o3[e][k] = pack2<__nv_bfloat16>(p, q);
          }
          *reinterpret_cast<uint4*>(sm + L::X1 + off) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
          *reinterpret_cast<uint4*>(sm + L::X2 + off) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
        }
        if (!STATE) {
          wait(barC, par);        // Y2 has read S and C
          if (more && TMA && bt == 0) load_bc(wf, cf, false, 0, 1);
        }
#pragma unroll
        for (int e = 0; e < PIECES; ++e) {
          const int idx = bt + e * 256, t = (idx >> 3) & (Q - 1), cv = (idx & 7) + 8 * (idx >> 10);
          *reinterpret_cast<uint4*>(sm + L::X3 + piece_off(t, cv)) = make_uint4(o3[e][0], o3[e][1], o3[e][2], o3[e][3]);
        }
        tc::fence_smem_to_async();
        tc::fence_before_sync();
        bar_named(2);
        if (bt == 0) {
          tc::fence_after_sync();
          constexpr uint32_t idS = tc::idesc_bf16_f32(128, PC, true, true);
#pragma unroll 1
          for (int term = 0; term < 3; ++term)
#pragma unroll
            for (int k = 0; k < Q / 16; ++k)
              tc::mma_bf16(tm + COL_DS, tc::sdesc128(sb + L::B + k * 2048u, BLK64, 1024u),
                           tc::sdesc128(sb + L::X1 + term * L::XT + k * 2048u, BLK64, 1024u), idS, term + k > 0);
          tc::mma_commit(barS);
        }
        wait(barS, par);
        tc::fence_after_sync();
        if (more) {               // dS (and G before it) have read B
          if (TMA) {
            if (bt == 0) load_bc(wf, cf, true, 0, 1);
          } else {
            load_bc(wf, cf, true, bt, 256);
            if (!STATE) load_bc(wf, cf, false, bt, 256);
          }
        }
        const float dec = ex2(decl);
        ltot += decl;
#pragma unroll
        for (int c32 = 0; c32 < HC / 32; ++c32) {
          uint32_t r[32];
          tc::tmem_ld32(tl + COL_DS + hf * HC + 32 * c32, r);
          tc::tmem_wait_ld(r);
#pragma unroll
          for (int e = 0; e < 32; ++e) S[32 * c32 + e] = fmaf(S[32 * c32 + e], dec, __uint_as_float(r[e]));
        }
        if (!STATE && !last) store_s();
        if (more && scans) {
          if (!STATE) wait(barY, par);   // W has been formed: the decays' arrays are free
          scan(wf, cf);
        }
        chunk_end();
      }
      if (ok) {
        float* to = STATE ? ta.ws + (int64_t)(w.tile + 1) * per_tile : w.seg == w.nseg - 1 ? pool : nullptr;
        if (to) {
#pragma unroll
          for (int c = 0; c < HC; ++c)
            if (c < live) to[e0 + (int64_t)c * a.N] = S[c];
        }
        if (STATE && i == 0 && w.p0 == 0 && (NH == 2 || hf == 0))
          ta.ws[(int64_t)ta.tiles * per_tile + (int64_t)w.tile * a.H + w.h0 + hcol] = ltot;
      }
    }
  } else {
    float raw[NH];
    auto load_dt = [&](const Unit& w, int c) {
      if (!STATE) {
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) raw[hh] = raw_dt(w, w.s0 + c * Q + i, hh);
      }
    };
    if (cur < ta.total) load_dt(unit_at<NH, PH, STATE>(ta, cur), 0);
    for (u = cur; u < ta.total;) {
      const Unit w = unit_at<NH, PH, STATE>(ta, u);
      const int nxt = next_unit<NH, PH, STATE>(ta, u + gridDim.x, gridDim.x);
      const Unit wn = nxt < ta.total ? unit_at<NH, PH, STATE>(ta, nxt) : w;
      for (int c = 0; c < w.nch; ++c) {
        const uint32_t par = gc & 1u;
        const uint32_t xs = L::X + par * L::XT;
        const int t0 = w.s0 + c * Q, nt = min(Q, w.s1 - t0);
        const bool last = c + 1 == w.nch, more = !last || nxt < ta.total;
        const Unit& wf = last ? wn : w;
        const int cf = last ? 0 : c + 1;
        float own[NH];            // dt of token i
#pragma unroll
        for (int hh = 0; hh < NH; ++hh) own[hh] = !STATE && i < nt ? step_of(raw[hh], w.h0 + hh) : 0.f;
        if (more) load_dt(wf, cf);
        chunk_begin(nt);
        if (!STATE && tid == 0) {
          constexpr uint32_t idG = tc::idesc_bf16_f32(128, 128), idY = tc::idesc_bf16_f32(128, PC, false, true);
          for (int k = 0; k < nk; ++k) {
            const uint32_t o = (uint32_t)(k >> 2) * BLK64 + (uint32_t)(k & 3) * 32u;
            tc::mma_bf16(tm + COL_G, tc::sdesc128(sb + L::C + o, 16u, 1024u), tc::sdesc128(sb + L::B + o, 16u, 1024u),
                         idG, k > 0);
          }
          tc::mma_commit(barG);
          for (int k = 0; k < nk; ++k) {
            const uint32_t o = (uint32_t)(k >> 2) * BLK64 + (uint32_t)(k & 3) * 32u;
            tc::mma_bf16(tm + COL_Y2, tc::sdesc128(sb + L::C + o, 16u, 1024u),
                         tc::sdesc128(sb + L::X3 + k * 2048u, BLK64, 1024u), idY, k > 0);
          }
          tc::mma_commit(barC);
        }
        if (more) {
          if (TMA) {
            if (tid == 0) {
              if (!STATE) bulk_wait_read();     // y of the chunk before has left the buffer
              load_x(wf, cf, par ^ 1u, 0, 1);
            }
          } else {
            load_x(wf, cf, par ^ 1u, tid, 256);
          }
        }
        if (!STATE) {
          // ---- W from G, in place of G: columns 32 b + 16 hf .. + 15 of every block b
          wait(barG, par);
          tc::fence_after_sync();
          float G[64];
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (b <= q4) {
              uint32_t r[16];
              tc::tmem_ld16(tl + COL_G + 32 * b + 16 * hf, r);
              tc::tmem_wait_ld16(r);
#pragma unroll
              for (int e = 0; e < 16; ++e) G[16 * b + e] = __uint_as_float(r[e]);
            }
          tc::fence_before_sync();
          bar_named(1);           // the other warp of these lanes has its values too
          float li[NH];
#pragma unroll
          for (int hh = 0; hh < NH; ++hh) {
            const float* f = F + hh * 2 * Q;
            li[hh] = f[i];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const int j0 = 32 * b + 16 * hf;
              uint32_t v[8];
              if (b < q4) {
                const float rf = ex2(li[hh] - blk[hh * 4 + b]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float4 cf4 = *reinterpret_cast<const float4*>(f + Q + j0 + 4 * e);
                  const float* Gp = G + 16 * b + 4 * e;
                  v[2 * e] = pack2<__nv_bfloat16>(Gp[0] * (rf * cf4.x), Gp[1] * (rf * cf4.y));
                  v[2 * e + 1] = pack2<__nv_bfloat16>(Gp[2] * (rf * cf4.z), Gp[3] * (rf * cf4.w));
                }
              } else if (b == q4) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int j = j0 + 2 * e;
                  const float2 lj = *reinterpret_cast<const float2*>(f + j);
                  const float d0 = __shfl_sync(0xffffffffu, own[hh], 16 * hf + 2 * e),
                              d1 = __shfl_sync(0xffffffffu, own[hh], 16 * hf + 2 * e + 1);
                  v[e] = pack2<__nv_bfloat16>(j <= i ? G[16 * b + 2 * e] * (ex2(li[hh] - lj.x) * d0) : 0.f,
                                              j + 1 <= i ? G[16 * b + 2 * e + 1] * (ex2(li[hh] - lj.y) * d1) : 0.f);
                }
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = 0u;
              }
              tc::tmem_st8(tl + COL_G + 64 * hh + 16 * b + 8 * hf, v);
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
                                tc::sdesc128(sb + xs + hh * (PH / 64 * BLK64) + k * 2048u, BLK64, 1024u), id1, k > 0);
            tc::mma_commit(barY);
          }
          // ---- y = Y1 + e^{L_i} Y2 + D x, over x in shared memory once its terms are formed
          wait(barC, par);
          wait(barY, par);
          wait(barS, par);
          tc::fence_after_sync();
          const int hh = NH == 2 ? hf : 0, pc0 = NH == 2 ? 0 : hf * HC;
          const float el = ex2(NH == 2 ? li[hf ? NH - 1 : 0] : li[0]);
          const float Dh = a.D ? a.D[w.h0 + hh] : 0.f;
          const bool direct = !TMA || nt < Q;
          uint16_t* yr = static_cast<uint16_t*>(const_cast<void*>(a.y.p)) + tok(w, a.y, t0 + i) +
                         (int64_t)(w.h0 + hh) * a.P + w.p0 + pc0;
#pragma unroll
          for (int c32 = 0; c32 < HC / 32; ++c32) {
            uint32_t r1[32], r2[32];
            tc::tmem_ld32(tl + COL_Y1 + hf * HC + 32 * c32, r1);
            tc::tmem_ld32(tl + COL_Y2 + hf * HC + 32 * c32, r2);
            tc::tmem_wait_ld(r1);
            tc::tmem_wait_ld(r2);
#pragma unroll
            for (int e8 = 0; e8 < 4; ++e8) {
              uint4* xp = reinterpret_cast<uint4*>(sm + xs + piece_off(i, hf * (HC / 8) + 4 * c32 + e8));
              const uint4 xv = *xp;
              const uint32_t xw[4] = {xv.x, xv.y, xv.z, xv.w};
              uint32_t o[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int e = 8 * e8 + 2 * k;
                o[k] = pack2<__nv_bfloat16>(
                    fmaf(Dh, __uint_as_float(xw[k] << 16), fmaf(el, __uint_as_float(r2[e]), __uint_as_float(r1[e]))),
                    fmaf(Dh, __uint_as_float(xw[k] & 0xffff0000u),
                         fmaf(el, __uint_as_float(r2[e + 1]), __uint_as_float(r1[e + 1]))));
              }
              if (!direct) {
                *xp = make_uint4(o[0], o[1], o[2], o[3]);
              } else if (i < nt && ok) {
                uint16_t* p = yr + 32 * c32 + 8 * e8;
                const int left = a.P - w.p0 - pc0 - (32 * c32 + 8 * e8);
                if (TMA) {
                  if (left > 0) *reinterpret_cast<uint4*>(p) = make_uint4(o[0], o[1], o[2], o[3]);
                } else {
#pragma unroll
                  for (int k = 0; k < 8; ++k)
                    if (k < left) p[k] = (uint16_t)(o[k >> 1] >> (16 * (k & 1)));
                }
              }
            }
          }
          if (!direct) {
            tc::fence_smem_to_async();
            bar_named(1);
            if (tid == 0 && ok) {
#pragma unroll
              for (int b = 0; b < PC / 64; ++b) {
                const int p = w.p0 + (NH == 1 ? 64 * b : 0);
                if (p < a.P)
                  tma_store(&ta.my, p, w.h0 + (NH == 1 ? 0 : b), w.it.begin + t0, a.y.sn ? w.row : 0,
                            sb + xs + b * BLK64);
              }
              bulk_commit();
            }
          }
        }
        chunk_end();
      }
      u = nxt;
    }
    if (TMA && !STATE && tid == 0) bulk_wait();
  }
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

template <int NH, int PH, bool STATE, bool TMA>
cudaError_t go(const TcArgs& t, int sms, cudaStream_t s) {
  constexpr int BYTES = (int)Smem<NH * PH>::BYTES;
  static thread_local int ready = -1;              // the device whose limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready != dev) {
    e = cudaFuncSetAttribute(ssm_tc_kernel<NH, PH, STATE, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
    if (e != cudaSuccess) return e;
    ready = dev;
  }
  ssm_tc_kernel<NH, PH, STATE, TMA><<<(unsigned)(t.total < sms ? t.total : sms), TCT, BYTES, s>>>(t);
  return cudaGetLastError();
}
template <int NH, int PH, bool TMA>
cudaError_t both(const TcArgs& t, bool split, int sms, cudaStream_t s) {
  if (split) {
    const cudaError_t e = go<NH, PH, true, TMA>(t, sms, s);
    if (e != cudaSuccess) return e;
  }
  return go<NH, PH, false, TMA>(t, sms, s);
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

SsmPlan ssm_tc_plan(int H, int G, int P, int rows, const int32_t* lens, int64_t T, int sms) {
  SsmPlan p{};
  p.sms = sms;
  p.ph = P > 64 ? 128 : 64;
  p.ptiles = (P + p.ph - 1) / p.ph;
  int64_t longest = 0;
  for (int i = 0; i < rows; ++i) {
    const int64_t c = ((lens ? lens[i] : T) + Q - 1) / Q;
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
  const bool tma = vec && encode(&t.mx, a.x, a.P, a.H, tokens, a.rows) && encode(&t.mb, a.B, a.N, a.G, tokens, a.rows) &&
                   encode(&t.mc, a.C, a.N, a.G, tokens, a.rows) && encode(&t.my, a.y, a.P, a.H, tokens, a.rows);
  if (p.ph == 128) return tma ? both<1, 128, true>(t, p.split, p.sms, s) : both<1, 128, false>(t, p.split, p.sms, s);
  if (p.nh == 2) return tma ? both<2, 64, true>(t, p.split, p.sms, s) : both<2, 64, false>(t, p.split, p.sms, s);
  return tma ? both<1, 64, true>(t, p.split, p.sms, s) : both<1, 64, false>(t, p.split, p.sms, s);
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
