// Selective state space scan of bf16 prompts on the 5th-generation tensor cores.
//
// A chunk is Q = 128 tokens.  With S the state at its start, L_i the sum of
// dt_k A over tokens k <= i of the chunk, L_ij over j < k <= i and T_j over k > j,
//   y_i = sum_{j <= i} (C_i . B_j) e^{L_ij} dt_j x_j  +  e^{L_i} S C_i  +  D x_i
//   S'  = e^{L_Q} S + sum_j (e^{T_j} dt_j x_j) B_j^T
// Every factor is at most one for A < 0.  Per chunk and PC = 64 rows p of the
// state, rows of a product being tokens (state columns n for the last), tcgen05
// MMAs with fp32 accumulators in TMEM:
//   G  [128 x 128] = C B^T               exact products of the inputs
//   Y2 [128 x 64]  = C S^T               S rounded to bf16
//   Y1 [128 x 64]  = W X                 W_ij = G_ij e^{L_ij} dt_j rounded to bf16, A in TMEM
//   dS [128 x 64]  = B^T (X3 + X2 + X1)  e^{T_j} dt_j x_j as three bf16 terms (2^-25 of it is left)
// W and the S of Y2 are rounded once, like the output itself (half a step of
// bf16 each); the state keeps 32 bits: it lives in registers in fp32 and its
// increments are formed from all 24 bits.  e^{L_ij} outside the diagonal 32 x 32
// blocks is the product of a row and a column factor, both at most one, with b
// the last token of j's block: e^{L_ib} e^{L_bj}, so only the diagonal blocks
// take an exponential a pair.  Their exponents are summed token by token from i
// downwards: as differences of sums from the chunk's start they would be off by
// a rounding of the whole chunk's decay (one token of dt A = -1.6e5 left
// weights after it 17% off).
//
// A persistent CTA of eight warps takes units: one head's 64 state rows over a
// segment of a row.  B and C of the group, X, its terms and S sit in shared
// memory as rows of 64 values in the 128-byte swizzle, read K-major or MN-major
// as a product needs, so nothing is transposed; tensor copies bring B, C and X
// (and, but for a row's ragged last chunk, take y away).  A chunk's phases
// depend on one another, so the latency of each counts; two CTAs on an SM fill
// each other's waits.  For that a CTA keeps to half of the shared memory and of
// TMEM: the terms take the places of C and S once Y2 has read them, W and dS
// those of G.  With nearly all of the SM's memory used as shared memory there
// is next to no L1 cache, so nothing may spill (300 bytes a thread cost 15%, 20
// bytes 6%), and no form does: the next unit, for one, waits in shared memory.
//
// Measured on a GB300: 16 x 512 tokens of 32 heads of 128 x 128 107 us (1.7
// TB/s of the 6.7 of a copy; a first kernel on the FP32 cores 1.1 ms), of 64 x
// 128 58 us; one row of 2048 tokens of 16 heads of 64 x 128 24 us in three
// launches.  In the first the tensor cores are busy 26% of the time, shared
// memory 53% (the products' operands 28, the threads' accesses 25), the
// schedulers issue 39%, and 11% of the SMs' time passes without work: 1024
// units are four for some of the 304 CTAs and three for others.  One CTA of 16
// warps with everything doubled and the warps specialised took 138 us, 128
// state rows a unit 127 us (spilling), two heads a unit 87 us for 59.
//
// A chunk with an infinity or a NaN in x, B, C or dt is run token by token
// instead, by a function of its own: in the products such a value would meet
// the zero weights of earlier tokens.  x shows in its terms, B, C and dt in the
// pairs of a token with itself, a packed multiply-add for two values; the
// check and what it branches around cost 5% (16 x 512 tokens of 32 heads of
// 128 x 128: 106.9 us, 101.5 without).
//
// Rows with few heads are split into segments: a first launch (STATE) runs
// each segment from zero and leaves its end state and decay in the workspace, a
// second joins them to the states at the segments' starts, and the full launch
// goes on from those.
#include <cstdlib>

#include <cuda.h>
#include <cuda_bf16.h>

#include "dl_device.cuh"
#include "mixer_device.cuh"
#include "tc_device.cuh"

namespace dl {
namespace mx {

static __device__ int32_t g_mixer_status;

namespace {

constexpr int Q = 128, PC = 64, TCT = 256;
constexpr int HC = PC / 2;        // columns of one of the two warps of a lane quarter
constexpr uint32_t COL_G = 0, COL_DS = 0, COL_W = 64, COL_Y1 = 128, COL_Y2 = 192, COLS = 256;
constexpr uint32_t BLK64 = Q * 128;                  // bytes of 128 rows of 64 values
constexpr float LOG2E = 1.4426950408889634f;

struct Sm {
  static constexpr uint32_t TILE = 2 * BLK64;        // B or C: 128 tokens x 128 state columns
  static constexpr uint32_t B = 0, C = TILE, X = 2 * TILE, S = X + BLK64;
  static constexpr uint32_t X1 = C, X2 = C + BLK64, X3 = S;
  static constexpr uint32_t F = S + BLK64;           // the chunk's decays, see F_* below
  static constexpr uint32_t FB = (4 * Q + 16) * 4;
  static constexpr uint32_t BAR = F + FB;            // eight mbarriers
  static constexpr uint32_t TSLOT = BAR + 64;        // TMEM address
  static constexpr uint32_t NEXT = TSLOT + 16;       // the unit after the current one, in turns
  static constexpr uint32_t NOW = NEXT + 2 * 48;     // and that one, where a function wants it
  static constexpr uint32_t BYTES = NOW + 48;
};
// dt, log2 of the tokens' decays, their sums from every 16th token on, the pair weights' column factors (128 of each);
// sums over the blocks of 32 and over their first halves, e^{T} of the blocks' last tokens (4 of each); the whole sum.
constexpr int F_DT = 0, F_L = Q, F_H = 2 * Q, F_COL = 3 * Q, F_BLK = 4 * Q, F_HALF = F_BLK + 4, F_ET = F_BLK + 8,
              F_SUM = F_BLK + 12;
static_assert(2 * (Sm::BYTES + 1024) <= 228 * 1024, "two CTAs an SM");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void bar_pair(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }
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
// Descriptors of an operand whose rows are K (MN-major), or along whose rows K runs (K-major), and what K step k
// (16 values of K) adds to them, in 16 bytes.  With the steps as constants an MMA costs its thread a few
// instructions; formed one by one, the 48 of a chunk took 6% of the time.
__device__ __forceinline__ uint64_t by_rows(uint32_t base) { return tc::sdesc128(base, BLK64, 1024u); }
__device__ __forceinline__ uint64_t by_cols(uint32_t base) { return tc::sdesc128(base, 16u, 1024u); }
__device__ constexpr uint32_t row_step(int k) { return k * (2048u >> 4); }
__device__ constexpr uint32_t col_step(int k) { return (k >> 2) * (BLK64 >> 4) + (k & 3) * 2u; }

struct TcArgs {
  CUtensorMap mx, mb, mc, my;   // x, B, C, y: [64 values][head or group][128 tokens][row] boxes
  SsmArgs a;
  float* ws;                    // segment states [tiles][H][P][N], then log2 decays [tiles][H]
  int32_t seg_tokens, tiles, per_row, units, ptiles, total, empty_rows;
  // Test only (0 in normal use): a thread of CTA 0 also waits, for wait_ns / 2, on a barrier that nothing arrives on.
  int32_t test_stall;
  unsigned long long wait_ns;   // how long a wait spins before it gives up (WAIT_LIMIT_NS but in tests)
};

// One unit of work: tokens [s0, s1) of a row (a segment) for 64 state rows from p0 of head h.
struct Unit {
  int tile, row, begin, h, p0, s0, s1, chunks;
  int u;                        // its number; from TcArgs::total on: none
};
static_assert(sizeof(Unit) <= 48, "its place in shared memory");
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
// The first unit from u on (in steps of the grid) that has work.
template <bool STATE>
__device__ __forceinline__ Unit next_unit(const TcArgs& ta, int u) {
  Unit w{};
  for (; u < ta.total; u += gridDim.x) {
    w = unit_at(ta, u);
    if (!skipped<STATE>(ta, w)) break;
  }
  w.u = u;
  return w;
}
// (Not inlined: the loops below have to stay in the instruction cache.)
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t par, int32_t code, unsigned long long ns) {
  return mbar_wait(bar, par, &g_mixer_status, code, ns);
}
__device__ __noinline__ void drain_long(uint32_t bar, uint32_t par) { mbar_drain(bar, par); }

// acc + 0 x for two bf16 values: whatever is not finite leaves a NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t acc, uint32_t x) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  return acc;
}
// Tokens [t0, t0 + nt) of unit w as they are defined, one after the other, with everything read from where the caller
// left it: for a chunk whose products are not finite.  In those an infinity or a NaN of x, B, C or dt meets the zero
// weights of earlier tokens and the terms that were split off, and 0 inf is a NaN; here it reaches what follows from
// it.  The state is in fp32 [64][128] in C's place, y goes to x's.  0.6 ms a chunk of 64 x 128.
template <bool STATE>
__device__ __noinline__ void chunk_by_tokens(const TcArgs& ta, unsigned char* sm, const Unit* at, int t0, int nt) {
  const SsmArgs& a = ta.a;
  const Unit w = *at;
  float* S = reinterpret_cast<float*>(sm + Sm::C);
  const int tid = threadIdx.x, n = tid & 127, pw = min(PC, a.P - w.p0), g = w.h / (a.H / a.G);
  auto token = [&](const TokView& v, int t) {
    return static_cast<const uint16_t*>(v.p) + (int64_t)(w.begin + t) * v.st + (int64_t)w.row * v.sn;
  };
  auto value = [](const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); };
  const float A = a.A[w.h], D = a.D ? a.D[w.h] : 0.f, bias = a.dt_bias ? a.dt_bias[w.h] : 0.f;
#pragma unroll 1
  for (int t = t0; t < t0 + nt; ++t) {
    const int64_t od = (int64_t)(w.begin + t) * a.dt.st + (int64_t)w.row * a.dt.sn + w.h;
    float dt = (a.dt_f32 ? static_cast<const float*>(a.dt.p)[od] : value(static_cast<const uint16_t*>(a.dt.p) + od)) + bias;
    if (a.softplus) dt = softplus_f(dt);
    const float dec = expf(dt * A);
    const uint16_t* x = token(a.x, t) + (int64_t)w.h * a.P + w.p0;
    if (n < a.N) {
      const float b = value(token(a.B, t) + (int64_t)g * a.N + n);
#pragma unroll 1
      for (int p = tid >> 7; p < pw; p += 2) S[p * 128 + n] = fmaf(S[p * 128 + n], dec, value(x + p) * dt * b);
    }
    __syncthreads();
    if (!STATE) {
      const uint16_t* c = token(a.C, t) + (int64_t)g * a.N;
      const int p = tid >> 2;
      float y = 0.f;
#pragma unroll 1
      for (int k = tid & 3; k < a.N; k += 4) y = fmaf(S[p * 128 + k], value(c + k), y);
      y += __shfl_xor_sync(0xffffffffu, y, 1);
      y += __shfl_xor_sync(0xffffffffu, y, 2);
      if ((tid & 3) == 0 && p < pw)
        *reinterpret_cast<__nv_bfloat16*>(sm + Sm::X + piece_off(t - t0, p >> 3) + 2 * (p & 7)) =
            __float2bfloat16_rn(fmaf(D, value(x + p), y));
      __syncthreads();
    }
  }
}

// TMA: tensor copies (16-byte aligned tensors, widths and strides); else
// threads copy value by value.
template <bool STATE, bool TMA>
__global__ void __launch_bounds__(TCT, 2)
ssm_tc_kernel(const __grid_constant__ TcArgs ta) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const SsmArgs& a = ta.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, q4 = warp & 3, hf = warp >> 2;
  const int i = 32 * q4 + lane;                     // this thread's token row; its state column n
  const int nk = (a.N + 15) / 16;                   // K steps over the state columns
  const bool scans = warp == 7;                     // this warp forms the decays, four tokens a lane

  const uint32_t sb = smem_u32(sm);
  float* f = reinterpret_cast<float*>(sm + Sm::F);
  const uint32_t barG = sb + Sm::BAR, barC = barG + 8, barS = barG + 16, barY = barG + 24, fullB = barG + 32,
                 fullC = barG + 40, fullX = barG + 48, never = barG + 56;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + Sm::TSLOT);

  if (warp == 0) tc::tmem_alloc(sb + Sm::TSLOT, COLS);
  if (tid == 0) {
    for (int k = 0; k < 8; ++k) mbar_init(barG + 8 * k, 1);
    fence_mbar_init();
  }

  auto tok = [&](const Unit& w, const TokView& v, int t) { return (int64_t)(w.begin + t) * v.st + (int64_t)w.row * v.sn; };
  auto copy_rows = [&](uint32_t dst, const uint16_t* src, int64_t st, int nt, int width, int cols) {
#pragma unroll 1
    for (int e = tid; e < Q * cols / 8; e += TCT) {
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
  // Chunk c of unit w into its places.  TMA: one thread calls; else all copy.
  auto load_bc = [&](const Unit& w, int c) {
    const int t0 = w.s0 + c * Q, g = w.h / (a.H / a.G);
    if (TMA) {
      const int nb = a.N > 64 ? 2 : 1;
      mbar_arrive_expect_tx(fullB, nb * BLK64);
      for (int e = 0; e < nb; ++e)
        tma_load(sb + Sm::B + e * BLK64, &ta.mb, 64 * e, g, w.begin + t0, a.B.sn ? w.row : 0, fullB);
      if (!STATE) {
        mbar_arrive_expect_tx(fullC, nb * BLK64);
        for (int e = 0; e < nb; ++e)
          tma_load(sb + Sm::C + e * BLK64, &ta.mc, 64 * e, g, w.begin + t0, a.C.sn ? w.row : 0, fullC);
      }
    } else {
      const int nt = min(Q, w.s1 - t0);
      copy_rows(Sm::B, static_cast<const uint16_t*>(a.B.p) + (int64_t)g * a.N + tok(w, a.B, t0), a.B.st, nt, a.N, 128);
      if (!STATE)
        copy_rows(Sm::C, static_cast<const uint16_t*>(a.C.p) + (int64_t)g * a.N + tok(w, a.C, t0), a.C.st, nt, a.N, 128);
    }
  };
  auto load_x = [&](const Unit& w, int c) {
    const int t0 = w.s0 + c * Q;
    if (TMA) {
      mbar_arrive_expect_tx(fullX, BLK64);
      tma_load(sb + Sm::X, &ta.mx, w.p0, w.h, w.begin + t0, a.x.sn ? w.row : 0, fullX);
    } else {
      copy_rows(Sm::X, static_cast<const uint16_t*>(a.x.p) + (int64_t)w.h * a.P + w.p0 + tok(w, a.x, t0), a.x.st,
                min(Q, w.s1 - t0), min(PC, a.P - w.p0), PC);
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
  // A wait that ran out: this thread waits no more, and at the chunk's end the CTA leaves: no results, and nothing is
  // started over what may still be on its way.
  bool ok = true;
  auto wait = [&](uint32_t bar, uint32_t k) {       // for phase number k
    if (ok && !mbar_try_wait(bar, k & 1u)) ok = wait_long(bar, k & 1u, DEV_TIMEOUT_MMA, ta.wait_ns);
  };
  // After a wait that ran out in chunk number k: let its products and copies land before the memory is given back.
  // ahead: B and C of the next chunk are on their way as well.
  auto drain = [&](uint32_t k, bool ahead) {
    if (tid == 0) {
      if (!STATE) {
        drain_long(barG, k & 1u);
        drain_long(barC, k & 1u);
        drain_long(barY, k & 1u);
      }
      drain_long(barS, k & 1u);
    }
    if (TMA && tid == 32) {
      drain_long(fullX, k & 1u);
      if (ahead) ++k;
      drain_long(fullB, k & 1u);
      if (!STATE) drain_long(fullC, k & 1u);
    }
  };
  const int64_t per_tile = (int64_t)a.H * a.P * a.N;

  // ---- the state: this thread holds S[column hf * HC + .][n = i] of the unit
  float S[HC];
  auto elem0 = [&](const Unit& w) { return ((int64_t)w.h * a.P + w.p0 + hf * HC) * a.N + i; };
  auto live_of = [&](const Unit& w) { return i < a.N ? a.P - w.p0 - hf * HC : 0; };
  auto pool_of = [&](const Unit& w) { return a.state ? a.state + (int64_t)a.items[w.row].slot * per_tile : nullptr; };
  auto load_state = [&](const Unit& w) {
    int seg, nseg;
    segments(ta, w, seg, nseg);
    const bool fresh = row_fresh(a.items[w.row]);
    const int64_t e0 = elem0(w);
    const int live = live_of(w);
    const float* from;
    if (STATE || nseg == 1) from = seg == 0 && !fresh ? pool_of(w) : nullptr;
    else from = seg == 0 && fresh ? nullptr : ta.ws + (int64_t)w.tile * per_tile;
#pragma unroll
    for (int c = 0; c < HC; ++c) S[c] = from && c < live ? from[e0 + (int64_t)c * a.N] : 0.f;
    if (STATE && seg == 0 && from) {
      // the last segment's CTA overwrites the pool's entry in the full launch
      float* to = ta.ws + (int64_t)w.tile * per_tile + e0;
#pragma unroll
      for (int c = 0; c < HC; ++c)
        if (c < live) to[(int64_t)c * a.N] = S[c];
    }
  };
  auto leave_state = [&](const Unit& w, float ltot) {
    int seg, nseg;
    segments(ta, w, seg, nseg);
    const int64_t e0 = elem0(w);
    const int live = live_of(w);
    float* to = STATE ? ta.ws + (int64_t)(w.tile + 1) * per_tile : seg == nseg - 1 ? pool_of(w) : nullptr;
    if (to) {
#pragma unroll
      for (int c = 0; c < HC; ++c)
        if (c < live) to[e0 + (int64_t)c * a.N] = S[c];
    }
    if (STATE && tid == 0 && w.p0 == 0)
      ta.ws[(int64_t)ta.tiles * per_tile + (int64_t)w.tile * a.H + w.h] = ltot;
  };
  auto share_state = [&]() {      // S as a bf16 operand: rows n, columns contiguous
    if (STATE) return;
#pragma unroll
    for (int c8 = 0; c8 < HC / 8; ++c8) {
      const float* s = S + 8 * c8;
      *reinterpret_cast<uint4*>(sm + Sm::S + piece_off(i, hf * (HC / 8) + c8)) =
          make_uint4(pack2<__nv_bfloat16>(s[0], s[1]), pack2<__nv_bfloat16>(s[2], s[3]),
                     pack2<__nv_bfloat16>(s[4], s[5]), pack2<__nv_bfloat16>(s[6], s[7]));
    }
  };

  // Rows without tokens: a fresh one's state is zero.
  if (!STATE && ta.empty_rows)
#pragma unroll 1
    for (int e = blockIdx.x; e < ta.total; e += gridDim.x) {
      const Unit v = unit_at(ta, e);
      float* to = pool_of(v);
      if (v.chunks == 0 && to && row_fresh(a.items[v.row]))
#pragma unroll 1
        for (int c = 0; c < HC && c < live_of(v); ++c) to[elem0(v) + (int64_t)c * a.N] = 0.f;
    }

  // dt of the next chunk: the scanning warp's four tokens
  uint32_t raw[4];
  float bias = 0.f, Ah = 0.f;
  auto load_dt = [&](const Unit& v, int c) {
#pragma unroll
    for (int k = 0; k < 4; ++k) raw[k] = raw_dt(v, v.s0 + c * Q + 4 * lane + k);
    Ah = a.A[v.h];
    bias = a.dt_bias ? a.dt_bias[v.h] : 0.f;
  };
  // Decays of a chunk of nt tokens, from raw.  Every exponent that is used is a sum of the logs it spans and never a
  // difference of longer sums: of one sign for A < 0, such a sum is off by a few steps of its own size, however
  // strong the decays around it are, and one that overflows is -inf (a factor of zero).
  auto scan = [&](int nt) {
    float dt[4], l[4], suf[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      dt[k] = 4 * lane + k < nt ? dt_of(raw[k], bias) : 0.f;
      l[k] = dt[k] * (Ah * LOG2E);
    }
    *reinterpret_cast<float4*>(f + F_DT + 4 * lane) = make_float4(dt[0], dt[1], dt[2], dt[3]);
    *reinterpret_cast<float4*>(f + F_L + 4 * lane) = make_float4(l[0], l[1], l[2], l[3]);
    // over the tokens after one in its block of 32
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
    // up to a token from the first of its 16
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      const float v = __shfl_up_sync(0xffffffffu, pre, o, 4);
      if ((lane & 3) >= o) pre += v;
    }
    const float prv = __shfl_up_sync(0xffffffffu, pre, 1, 4), nxt = __shfl_down_sync(0xffffffffu, post, 1, 8);
    const float before = (lane & 3) > 0 ? prv : 0.f, after = (lane & 7) < 7 ? nxt : 0.f;
    float bs[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) bs[b] = __shfl_sync(0xffffffffu, post, 8 * b);
    *reinterpret_cast<float4*>(f + F_H + 4 * lane) = make_float4(before + l[0], before + l[1], before + l[2], pre);
    *reinterpret_cast<float4*>(f + F_COL + 4 * lane) =
        make_float4(ex2(after + suf[0]) * dt[0], ex2(after + suf[1]) * dt[1], ex2(after + suf[2]) * dt[2],
                    ex2(after + suf[3]) * dt[3]);
    if ((lane & 7) == 3) f[F_HALF + (lane >> 3)] = pre;
    if (lane < 4) {
      f[F_BLK + lane] = lane == 0 ? bs[0] : lane == 1 ? bs[1] : lane == 2 ? bs[2] : bs[3];
      f[F_ET + lane] = ex2(lane == 0 ? bs[3] + bs[2] + bs[1] : lane == 1 ? bs[3] + bs[2] : lane == 2 ? bs[3] : 0.f);
    }
    if (lane == 0) f[F_SUM] = bs[3] + bs[2] + bs[1] + bs[0];
  };

  Unit w = next_unit<STATE>(ta, blockIdx.x);
  if (w.u < ta.total) {
    if (!TMA || tid == 32) {
      load_x(w, 0);
      load_bc(w, 0);
    }
    if (scans) {
      load_dt(w, 0);
      scan(w.s1 - w.s0);
    }
  }
  if (ta.test_stall && blockIdx.x == 0 && tid == 64) ok = wait_long(never, 0, DEV_TEST_STALL, ta.wait_ns / 2);
  uint32_t gc = 0;                // chunks done, over all units: every barrier's phase

  uint32_t place = Sm::NEXT;      // of the next unit; one thread looks it up, and few of them want it, so that it costs
                                  // no registers
#pragma unroll 1
  while (w.u < ta.total) {
    if (tid == 64) *reinterpret_cast<Unit*>(sm + place) = next_unit<STATE>(ta, w.u + gridDim.x);
    load_state(w);
    share_state();
    tc::fence_smem_to_async();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const volatile Unit* wn = reinterpret_cast<const volatile Unit*>(sm + place);
    const bool another = wn->u < ta.total;
    float ltot = 0.f;
#pragma unroll 1
    for (int c = 0; c < w.chunks; ++c, ++gc) {
      const int t0 = w.s0 + c * Q, nt = min(Q, w.s1 - t0);
      const bool last = c + 1 == w.chunks, more = !last || another;
      const int cf = last ? 0 : c + 1;              // the chunk after this one, of this unit or the next
      auto after = [&]() -> Unit {
        if (!last) return w;
        return Unit{wn->tile, wn->row, wn->begin, wn->h, wn->p0, wn->s0, wn->s1, wn->chunks, wn->u};
      };
      const float decl = f[F_SUM];
      // the sums up to token i from the first of its 16, of its block, of the chunk
      const float4 blk = *reinterpret_cast<const float4*>(f + F_BLK);
      const float hi = f[F_H + i], ri = lane >= 16 ? hi + f[F_HALF + q4] : hi;
      const float li = q4 == 0 ? ri : q4 == 1 ? ri + blk.x : q4 == 2 ? ri + (blk.x + blk.y) : ri + (blk.x + blk.y + blk.z);
      if (TMA && nt < Q) {
        // a ragged chunk: what lies behind its last token is cleared in B and X (C's rows there give rows of y
        // that are not kept)
        wait(fullB, gc);
        wait(fullX, gc);
#pragma unroll 1
        for (int e = tid; e < (Q - nt) * 24; e += TCT) {
          const int r = nt + e % (Q - nt), cv = e / (Q - nt);
          const uint32_t off = cv < 16 ? Sm::B + piece_off(r, cv) : Sm::X + piece_off(r, cv - 16);
          *reinterpret_cast<uint4*>(sm + off) = make_uint4(0u, 0u, 0u, 0u);
        }
        tc::fence_smem_to_async();
        __syncthreads();
      }
      uint32_t odd2 = 0u;                           // whether something of the chunk is not finite
      if (!STATE) {
        if (tid == 0) {
          if (TMA) {
            wait(fullB, gc);
            wait(fullC, gc);
          }
          tc::fence_after_sync();
          constexpr uint32_t idG = tc::idesc_bf16_f32(128, 128), idY = tc::idesc_bf16_f32(128, PC, false, true);
          const uint64_t dc = by_cols(sb + Sm::C), db = by_cols(sb + Sm::B), ds = by_rows(sb + Sm::S);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < nk) tc::mma_bf16(tm + COL_G, dc + col_step(k), db + col_step(k), idG, k > 0);
          tc::mma_commit(barG);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < nk) tc::mma_bf16(tm + COL_Y2, dc + col_step(k), ds + row_step(k), idY, k > 0);
          tc::mma_commit(barC);
        }
        if (more && scans) load_dt(after(), cf);
        // ---- W from G: columns 32 b + 16 hf .. + 15 of every block b, in place of blocks 2 and 3 of G once both
        // warps of the lanes have read them
        if (TMA) wait(fullX, gc);
        wait(barG, gc);
        tc::fence_after_sync();
        auto form = [&](int b, uint32_t (&v)[8]) {
          const int j0 = 32 * b + 16 * hf;
          uint32_t G[16];
          if (b <= q4) {
            tc::tmem_ld16(tl + COL_G + j0, G);
            tc::tmem_wait_ld16(G);
          }
          if (b < q4) {
            // from the end of block b to token i
            const float rf = ex2(b == 0 ? (q4 == 1 ? ri : q4 == 2 ? ri + blk.y : ri + (blk.y + blk.z))
                                        : b == 1 && q4 == 3 ? ri + blk.z : ri);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float4 cf4 = *reinterpret_cast<const float4*>(f + F_COL + j0 + 4 * e);
              v[2 * e] = pack2<__nv_bfloat16>(__uint_as_float(G[4 * e]) * (rf * cf4.x),
                                              __uint_as_float(G[4 * e + 1]) * (rf * cf4.y));
              v[2 * e + 1] = pack2<__nv_bfloat16>(__uint_as_float(G[4 * e + 2]) * (rf * cf4.z),
                                                  __uint_as_float(G[4 * e + 3]) * (rf * cf4.w));
            }
          } else if (b == q4) {
            // from the last column down, a token's log at a time
            float sum = hf == 0 && lane >= 16 ? hi : 0.f;
#pragma unroll
            for (int e4 = 3; e4 >= 0; --e4) {
              const float4 l4 = *reinterpret_cast<const float4*>(f + F_L + j0 + 4 * e4);
              const float4 d4 = *reinterpret_cast<const float4*>(f + F_DT + j0 + 4 * e4);
              const float l[4] = {l4.x, l4.y, l4.z, l4.w}, d[4] = {d4.x, d4.y, d4.z, d4.w};
              float w[4];
#pragma unroll
              for (int k = 3; k >= 0; --k) {
                const int e = 4 * e4 + k;             // column j0 + e
                const bool in = 16 * hf + e <= lane;
                w[k] = in ? __uint_as_float(G[e]) * (ex2(sum) * d[k]) : 0.f;
                if (in) sum += l[k];
              }
              v[2 * e4] = pack2<__nv_bfloat16>(w[0], w[1]);
              v[2 * e4 + 1] = pack2<__nv_bfloat16>(w[2], w[3]);
            }
            // B, C and dt that are not finite show in the pairs of a token with itself (C's rows past the last token
            // are not looked at)
            if (i < nt)
#pragma unroll
              for (int e = 0; e < 8; ++e) odd2 = not_finite(odd2, v[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0u;
          }
        };
        uint32_t v2[8], v3[8];
        form(2, v2);
        form(3, v3);
        tc::fence_before_sync();
        bar_pair(1 + q4);
        tc::tmem_st8(tl + COL_W + 32 + 8 * hf, v2);
        tc::tmem_st8(tl + COL_W + 48 + 8 * hf, v3);
        form(0, v2);
        tc::tmem_st8(tl + COL_W + 8 * hf, v2);
        form(1, v3);
        tc::tmem_st8(tl + COL_W + 16 + 8 * hf, v3);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncthreads();
        if (tid == 0) {
          tc::fence_after_sync();
          constexpr uint32_t id1 = tc::idesc_bf16_f32(128, PC, false, true);
          const uint64_t dx = by_rows(sb + Sm::X);
#pragma unroll
          for (int k = 0; k < Q / 16; ++k) tc::mma_bf16_ta(tm + COL_Y1, tm + COL_W + 8 * k, dx + row_step(k), id1, k > 0);
          tc::mma_commit(barY);
        }
        wait(barC, gc);           // G and Y2 have read C and S: the terms take their places
      } else {
        if (more && scans) load_dt(after(), cf);
        if (TMA) {
          wait(fullX, gc);
          wait(fullB, gc);
        }
#pragma unroll
        for (int e = 0; e < Q * 128 / 8 / TCT; ++e) {
          const int idx = tid + e * TCT, t = idx & (Q - 1), cv = idx / Q;
          if (cv * 8 >= a.N) break;
          const uint4 bv = *reinterpret_cast<const uint4*>(sm + Sm::B + piece_off(t, cv));
          odd2 = not_finite(not_finite(not_finite(not_finite(odd2, bv.x), bv.y), bv.z), bv.w);
        }
      }
      // ---- X's three terms, then dS
#pragma unroll
      for (int e = 0; e < Q * PC / 8 / TCT; ++e) {
        const int idx = tid + e * TCT, t = idx >> 3, cv = idx & 7;
        const uint32_t off = piece_off(t, cv);
        const uint4 xv = *reinterpret_cast<const uint4*>(sm + Sm::X + off);
        const float g = f[F_COL + t] * f[F_ET + (t >> 5)];
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
          odd2 = not_finite(odd2, o1[k]);
        }
        *reinterpret_cast<uint4*>(sm + Sm::X1 + off) = make_uint4(o1[0], o1[1], o1[2], o1[3]);
        *reinterpret_cast<uint4*>(sm + Sm::X2 + off) = make_uint4(o2[0], o2[1], o2[2], o2[3]);
        *reinterpret_cast<uint4*>(sm + Sm::X3 + off) = make_uint4(o3[0], o3[1], o3[2], o3[3]);
      }
      tc::fence_smem_to_async();
      const bool odd = __syncthreads_or((odd2 & 0x7fff7fffu) != 0u);      // the decays are free too
      if (tid == 0) {
        tc::fence_after_sync();
        constexpr uint32_t idS = tc::idesc_bf16_f32(128, PC, true, true);
        const uint64_t db = by_rows(sb + Sm::B), dx[3] = {by_rows(sb + Sm::X3), by_rows(sb + Sm::X2), by_rows(sb + Sm::X1)};
#pragma unroll
        for (int k = 0; k < 3 * Q / 16; ++k)        // the small terms first
          tc::mma_bf16(tm + COL_DS, db + row_step(k & 7), dx[k >> 3] + row_step(k & 7), idS, k > 0);
        tc::mma_commit(barS);
      }
      if (more && scans) scan(last ? wn->s1 - wn->s0 : w.s1 - w.s0 - cf * Q);
      if (!STATE) {
        // ---- y = Y1 + e^{L_i} Y2 + D x, over x in shared memory
        const float ei = ex2(li), Dh = a.D ? a.D[w.h] : 0.f;
        wait(barY, gc);
        tc::fence_after_sync();
#pragma unroll
        for (int c16 = 0; c16 < HC / 16; ++c16) {         // (not finite: overwritten below)
          uint32_t r1[16], r2[16];
          tc::tmem_ld16(tl + COL_Y1 + hf * HC + 16 * c16, r1);
          tc::tmem_ld16(tl + COL_Y2 + hf * HC + 16 * c16, r2);
          tc::tmem_wait_ld16(r1);
          tc::tmem_wait_ld16(r2);
#pragma unroll
          for (int e8 = 0; e8 < 2; ++e8) {
            uint4* xp = reinterpret_cast<uint4*>(sm + Sm::X + piece_off(i, hf * (HC / 8) + 2 * c16 + e8));
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
      }
      // ---- S' = e^{L_Q} S + dS
      wait(barS, gc);
      tc::fence_after_sync();
      if (odd) {                  // the chunk again from what was given, with the state as it was before
        float* Sf = reinterpret_cast<float*>(sm + Sm::C) + hf * HC * 128 + i;
#pragma unroll
        for (int c = 0; c < HC; ++c) Sf[c * 128] = S[c];
        if (tid == 0) *reinterpret_cast<Unit*>(sm + Sm::NOW) = w;
        __syncthreads();
        chunk_by_tokens<STATE>(ta, sm, reinterpret_cast<const Unit*>(sm + Sm::NOW), t0, nt);
#pragma unroll
        for (int c = 0; c < HC; ++c) S[c] = Sf[c * 128];
        tc::fence_smem_to_async();
        __syncthreads();
      }
      if (TMA && more && tid == 32) {
        wait(fullB, gc);          // landed long ago, unless a wait ran out
        if (!STATE) wait(fullC, gc);
        if (ok) load_bc(after(), cf);
      }
      ltot += decl;
      if (!odd) {
        const float dec = ex2(decl);
#pragma unroll
        for (int c16 = 0; c16 < HC / 16; ++c16) {
          uint32_t r[16];
          tc::tmem_ld16(tl + COL_DS + hf * HC + 16 * c16, r);
          tc::tmem_wait_ld16(r);
#pragma unroll
          for (int e = 0; e < 16; ++e) S[16 * c16 + e] = fmaf(S[16 * c16 + e], dec, __uint_as_float(r[e]));
        }
      }
      if (!last) share_state();
      tc::fence_smem_to_async();
      tc::fence_before_sync();
      const bool mine = ok;
      ok = __syncthreads_and(ok);  // y and S are in shared memory, TMEM and the next decays are read and written
      tc::fence_after_sync();
      if (!ok) {
        drain(gc, more && mine);
        break;
      }
      if (!STATE && TMA && nt == Q) {
        if (tid == 32) {
          tma_store(&ta.my, w.p0, w.h, w.begin + t0, a.y.sn ? w.row : 0, sb + Sm::X);
          bulk_commit();
          bulk_wait_read();
        }
      } else if (!STATE) {
        // a ragged chunk's rows (or unaligned ones), value by value
        uint16_t* yr = static_cast<uint16_t*>(const_cast<void*>(a.y.p)) + tok(w, a.y, t0) + (int64_t)w.h * a.P + w.p0;
        const int pw = min(PC, a.P - w.p0);
#pragma unroll 1
        for (int e = tid; e < nt * PC; e += TCT) {
          const int t = e / PC, p = e % PC;
          if (p < pw)
            yr[(int64_t)t * a.y.st + p] =
                *reinterpret_cast<const uint16_t*>(sm + Sm::X + piece_off(t, p >> 3) + 2 * (p & 7));
        }
        __syncthreads();          // read before the place is filled again
      }
      if (more) {
        if (TMA) {
          if (tid == 32) load_x(after(), cf);
        } else {
          const Unit wf = after();
          load_x(wf, cf);
          load_bc(wf, cf);
          tc::fence_smem_to_async();
          __syncthreads();
        }
      }
    }
    if (!ok) break;               // every thread's since the vote: the only way out of the loops
    leave_state(w, ltot);
    w = Unit{wn->tile, wn->row, wn->begin, wn->h, wn->p0, wn->s0, wn->s1, wn->chunks, wn->u};
    place ^= Sm::NEXT ^ (Sm::NEXT + 48);
  }
  if (TMA && !STATE && tid == 32) bulk_wait();
  __syncthreads();
  if (warp == 0) tc::tmem_dealloc(tm, COLS);
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
  ssm_tc_kernel<STATE, TMA><<<(unsigned)(t.total < 2 * sms ? t.total : 2 * sms), TCT, Sm::BYTES, s>>>(t);
  return cudaGetLastError();
}
template <bool TMA>
cudaError_t both(const TcArgs& t, bool split, int sms, cudaStream_t s) {
  if (split) {
    cudaError_t e = go<true, TMA>(t, sms, s);
    if (e != cudaSuccess) return e;
    e = launch_ssm_join(t.a, t.seg_tokens, t.tiles, t.per_row, t.ws, s);
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
  // Segments as short as still fill the GPU once (two CTAs an SM): they take
  // three launches and half the work again, so at least three of them in the
  // longest row are wanted, and at most 16.  One row of 2048 tokens of 16 heads
  // of 64 x 128: 24 us, 70 whole.
  for (int64_t seg = (longest + 15) / 16; seg > 0 && 3 * seg <= longest; ++seg) {
    int64_t tiles = 0;
    for (int i = 0; i < rows; ++i) {
      const int64_t c = ((lens ? lens[i] : T) + Q - 1) / Q;
      tiles += c > seg ? (c + seg - 1) / seg : 1;
    }
    if (tiles * p.units <= 2 * (int64_t)sms) {
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
  t.wait_ns = WAIT_LIMIT_NS;
  if (const char* e = getenv("DL_TEST_WAIT_MS")) {
    const long ms = atol(e);
    if (ms > 0 && ms < 2000) t.wait_ns = (unsigned long long)ms * 1000000ull;
  }
  const char* stall = getenv("DL_TEST_STALL");
  t.test_stall = stall && atoi(stall) == 1;
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
