// Attention of prompts over pages on the 5th-generation tensor cores, 16-bit types.
//
// A tile is 128 rows: consecutive tokens times the query heads that share a head of keys.  Against a block of BK keys
//   S [128 x BK] = Q K^T           exact products of the inputs, fp32 sums in TMEM
//   P = 2^(S scale log2(e) - r)    rounded to the type, back to TMEM in the place of S
//   O [128 x D] += P V             A from TMEM, fp32 sums in TMEM
// with r a reference: the maximum of the row's first block, and of all so far whenever the weights of a block get too
// large for the type.  So most blocks take no maximum, and O stays where it is; it is read back and scaled when r moves.
// Sums of P are formed from its 32-bit values.
//
// Per block the products of a tile take about as long as its softmax, and they wait for one another: S of a block for
// its products, P for the softmax.  So a tile has two places for S, and S of the next block is there when the softmax
// of this one ends (blocks of 128 keys in one place each took 1.4 times as long).  A CTA has two tiles of one item for D
// <= 128 (for D = 256 one, whose O takes half of TMEM): they use the same keys, 256 rows a block that is read from L2.
//
// A product that writes over P has to wait for the products that read it: products of different shapes need not run in
// the order of their issue.
//
// Roles: warp 0 copies (queries and pages, tensor copies into the 128-byte swizzle), a warp a tile issues Q K^T and one
// P V, a warp a tile looks blocks over that not every token of the tiles sees, one finds the next items, and a warp
// group a tile does the softmax, a row a thread.  CTAs are persistent and each role goes on to the next item by itself,
// so an item's end overlaps the next one's beginning.  The issuing warps are split because what surrounds a product
// costs more than the product: one warp for both tiles' scores took 1850 cycles a block, now 1450 are the softmax's.
// They are elected threads with operands in uniform registers; from a branch on the lane a product took 80 cycles.
//
// What a token does not see has weight zero, and zero times an infinity or a NaN is a NaN: keys that no token of the
// item sees (behind the row's last, unwritten places) are zeroed in the copy of V, and a block some of whose tokens do
// not see a value that is not finite is added up by the softmax threads, key by key, instead.
//
// Few tiles (and at most 64 rows): their keys are split into items of about the same number of blocks, of the size that
// lets the busiest CTA finish first; the lengths are on the device, so every CTA forms that plan itself and the first
// leaves it for the second launch, which joins the parts (reference, sum, O in the workspace) in order.  A plan formed
// again by each of the join's blocks cost 5 to 20 us a call (32 rows of 4 tokens behind 8192: 63 us, now 42).
//
// Measured on a GB300, bf16, 32 heads of 128 over 8: one prompt of 8192 tokens 356 to 366 us on different machines (1.5
// PFLOP/s, 0.78 of a library product of the same type; 391 after some 0.3 s, when the power limit holds the SMs at 1890
// MHz instead of 2070), of 2048 44.5 us, 16 of 512 50.5 us; pieces of 371 tokens in all behind 30000 150 us; 16 heads of
// 256 over 2, 8192 tokens 422 us; 40 heads of 64 under a window of 1000 399 us (0.58 PFLOP/s).  Heads of 128 are bound by
// the products (without the softmax 340 us of 355) and nearly as much by the softmax (without products 305); heads of 64
// by the softmax: of 324 us 49 are the exponentials, 20 the products, the rest its other instructions and their latency
// (issue 49%, exponentials' units 38%, tensor cores 38%).
//
// Measured and left: four softmax groups with half a row a thread (the two have to agree on every reference; 1.1 to 1.5
// times as long); for heads of 64 a group for each chain with an O of its own (1.03 to 1.4; too few registers) or eight
// stages of keys (0.99); the next block's scores asked for ahead (1.01 to 1.05); the reference folded into one
// multiply-add (2% less, but a score of 2^24 or more loses its differences); tiles half a period apart.
#include <cmath>
#include <cstdlib>

#include <cuda.h>

#include "attn_device.cuh"
#include "mixer_device.cuh"
#include "tc_device.cuh"

namespace dl {
namespace at {

static __device__ int32_t g_tc_status;     // what was out of range
static __device__ int32_t g_tc_waits;      // waits that gave up

namespace {

using mx::add2;
using mx::ex2_f;
using mx::f2;
using mx::fma2;
using mx::from_f;
using mx::mk2;
using mx::pack2;
using mx::un2;

constexpr int R = 128;                     // rows of a tile
constexpr int ITEMS = 4;                   // items that are found ahead
constexpr int BK = 64;                     // keys of a block
constexpr int MIN_BLOCKS = 4;              // blocks that an item is worth
// A split call has at most ITEMS_A_CTA items a CTA and one a tile more, and at most SPLIT_ROWS rows: 64 of up to 40
// tokens behind 2000 take 39 us split, 55 whole (and 15.5, 14.5 behind none); 100 of 2 behind 4096 44 and 53, but 100 of
// 4 behind 200 21.7 and 17.9.  An item's start, its end and its part in the join cost about as much as ITEM_COST blocks,
// a join as JOIN_COST and one for every JOIN_PARTS parts of full tiles (half of that for heads of 64), JOIN_MOST at most.
// 4 tokens of 32 heads over 8 behind 300 keys take 14.8 us whole, 17.2 split; behind 1000 21.8 and 18.3; 64 tokens behind
// 300 16.3 and 19.9, behind 1000 23.3 and 21.1; one prompt of 1000 tokens of 16 heads over 2 22.7 and 28.7.  (And 64
// tokens of 32 heads behind 3000, split into items of 4 blocks, 23.3; 24.3 into 8.)
constexpr int ITEMS_A_CTA = 4, SPLIT_ROWS = 64, ITEM_COST = 10;
constexpr float JOIN_COST = 4.f, JOIN_PARTS = 14.f, JOIN_MOST = 16.f;
constexpr int PLAN = 4 * SPLIT_ROWS;       // words of the plan, before the parts in the workspace

template <int D> struct Cfg {
  static constexpr int QT = D == 256 ? 1 : 2, STAGES = D == 256 ? 2 : 4;   // tiles; a tile has two chains of blocks
  static constexpr int THREADS = 512;
  // Registers of a thread that is not, and that is, of the softmax; a block is launched with LAUNCH_REGS each.  A block's
  // 64 scores and its weights stay in registers that way: 16 x 512 tokens 49.5 us, 53.5 read in halves with 128 for all.
  static constexpr int AUX_REGS = QT == 2 ? 72 : 96, ROW_REGS = QT == 2 ? 184 : 224, LAUNCH_REGS = 128;
  static_assert((THREADS - 128 * QT) * AUX_REGS + 128 * QT * ROW_REGS <= THREADS * LAUNCH_REGS, "what the block has");
  static constexpr uint32_t QBLK = R * 128, KBLK = BK * 128;            // 64 columns of a tile, of a block
  static constexpr uint32_t QTILE = QBLK * (D / 64), KTILE = KBLK * (D / 64);
  static constexpr uint32_t Q = 0, K = QT * QTILE, V = K + STAGES * KTILE, MISC = V + STAGES * KTILE;
  static constexpr uint32_t S_COL = 0, O_COL = 256;                     // chain c's S at c * BK, tile t's O at 256 + t * D
  // barriers, eight bytes each
  enum { QFULL = 0, QEMPTY = 2, KFULL = 4, KEMPTY = 8, VFULL = 12, VEMPTY = 16, VOK = 20, SFULL = 24, PREADY = 28, PVDONE = 32,
         IFULL = 36, IEMPTY = 40, DRAIN = 44, NEVER = 48, BARS = 49 };
  static constexpr uint32_t BAR = MISC, FLAGS = BAR + 8 * (BARS + 1), TSLOT = FLAGS + 32, ITEM = TSLOT + 16;
  static constexpr uint32_t OUT = (ITEM + ITEMS * 64 + 127) & ~127u;    // 32 rows of 128 bytes of every softmax warp
  static constexpr uint32_t ROWS = OUT + 4 * QT * 4096, BYTES = ROWS + 8 * SPLIT_ROWS;          // the plan of a split call
  static_assert(BYTES <= 232448, "of a CTA");
};

struct Item {
  int32_t x, row, slot, begin, t0, nt, pos0, gh, h0;   // x < 0: no more items
  int32_t part, b0, b1, sink_blocks, first, whole;     // blocks [b0, b1); whole: all of the tile's; part: else its number
  int32_t pad;
};
static_assert(sizeof(Item) == 64, "its place in shared memory");

struct TcArgs {
  CUtensorMap mq, mk, mv;
  AttnArgs a;
  int32_t tpt, hpt, hgroups, tiles, split, total, per_row, ctas;   // per_row: tiles of a row (token-major), else 0
  float join;                          // what a part costs in the join, in blocks
  int32_t test_stall;                  // test only: see below
  unsigned long long wait_ns;
};

__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(dst), "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma5(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3, int c4, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(dst), "l"(m), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar) : "memory");
}
// One thread of the warp, the same one every time.
__device__ __forceinline__ bool elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.b32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t par, unsigned long long ns) {
  return mbar_wait(bar, par, &g_tc_waits, DEV_TIMEOUT_MMA, ns);
}

// acc + 0 x for two values: whatever is not finite leaves a NaN.
template <class T> __device__ __forceinline__ uint32_t not_finite(uint32_t acc, uint32_t x) {
  if constexpr (std::is_same<T, __half>::value) asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  else asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0u));
  return acc;
}
// Bits 0 .. n of a word.
__device__ __forceinline__ uint32_t bits_to(int n) { return n < 0 ? 0u : n >= 31 ? 0xffffffffu : (2u << n) - 1u; }
template <class T> __host__ __device__ constexpr uint32_t idesc(int N, bool b_mn) {
  return tc::idesc_bf16_f32(R, N, false, b_mn) & ~(std::is_same<T, __half>::value ? (1u << 7) | (1u << 10) : 0u);
}
// The reference is the row's maximum when it is set, and stays while the weights of a block add up to at most LIMIT:
// bf16 weights keep their precision and sums of 2^20 their range; fp16 ones must stay below 2^16, and are kept 2^7 up,
// so that those of 2^-21 are still normal numbers (a block of them at the maximum adds up to 2^14).
template <class T> constexpr float LIFT = 0.f;
template <> constexpr float LIFT<__half> = 7.f;
template <class T> constexpr float LIMIT = 0x1p20f;
template <> constexpr float LIMIT<__half> = 0x1p15f;

// O += P V for a block with values that are not finite, key by key; a row takes the keys that it sees.  P is in TMEM at
// p_col, O at o_col (first: not yet anything).
template <class T, int D>
__device__ __forceinline__ void by_keys(const AttnArgs& a, const unsigned char* v, uint32_t p_col, uint32_t o_col, int pos,
                                     int j0, bool first) {
  using C = Cfg<D>;
#pragma unroll 1
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    tc::tmem_ld32(o_col + 32 * c, o);
    tc::tmem_wait_ld(o);
    if (first)
#pragma unroll
      for (int k = 0; k < 32; ++k) o[k] = 0u;
#pragma unroll 1
    for (int j = 0; j < BK; ++j) {
      uint32_t w;
      asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(w) : "r"(p_col + (uint32_t)(j >> 1)));
      asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(w)::"memory");
      float lo, hi;
      mx::unpack2<T>(w, lo, hi);
      const float p = j & 1 ? hi : lo;
      const bool see = sees(a, pos, j0 + j);
      const unsigned char* row = v + (c >> 1) * C::KBLK + j * 128;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint4 x = *reinterpret_cast<const uint4*>(row + ((((c & 1) * 4 + k) ^ (j & 7)) << 4));
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          mx::unpack2<T>(xs[e], lo, hi);
          if (see) {
            o[8 * k + 2 * e] = __float_as_uint(fmaf(p, lo, __uint_as_float(o[8 * k + 2 * e])));
            o[8 * k + 2 * e + 1] = __float_as_uint(fmaf(p, hi, __uint_as_float(o[8 * k + 2 * e + 1])));
          }
        }
      }
    }
    tc::tmem_st32(o_col + 32 * c, o);
  }
  tc::tmem_wait_st();
}

// The plan of a split call: of every row the blocks that its last tile's keys make (x), its tiles (the low half of y) and
// the items of a head of the rows before (the high half; less than 2^10 in all).  One warp; a tile has items_of items of
// `each` blocks at most.  Returns the items of a head.  Rows that have more tiles than the call may (starts that go back
// and forth) have none here: the workspace holds the parts of g.tiles.
__device__ __forceinline__ int items_of(int count, int each) { return count > each ? (count + each - 1) / each : 1; }
__device__ __forceinline__ int plan_split(const TcArgs& g, int tpt, uint2* rows, int& each, int32_t* status) {
  const AttnArgs& a = g.a;
  const int lane = threadIdx.x & 31;
  long long work = 0, tiles = 0;
  // every load before what is made of it
  int t[SPLIT_ROWS / 32], slot[SPLIT_ROWS / 32], len[SPLIT_ROWS / 32];
#pragma unroll
  for (int k = 0; k < SPLIT_ROWS / 32; ++k) {
    const int i = lane + 32 * k;
    int begin;
    slot[k] = i < a.n ? a.slots[i] : 0;
    t[k] = i < a.n ? row_tokens(a, i, begin, status) : 0;
  }
  auto there = [&](int k) { return (unsigned)slot[k] < (unsigned)a.num_slots; };
#pragma unroll
  for (int k = 0; k < SPLIT_ROWS / 32; ++k) len[k] = lane + 32 * k < a.n && there(k) ? a.lengths[slot[k]] : 0;
#pragma unroll
  for (int k = 0; k < SPLIT_ROWS / 32; ++k) {
    if (lane + 32 * k >= a.n) break;
    const int cap = a.max_pages << a.page_shift, n = min(max(len[k], 0), cap);      // (as in row_length)
    if (t[k] > 0) {                       // (a row without tokens is not looked at, here as in make_tile)
      if (!there(k)) atomicCAS(status, 0, DEV_BAD_SLOT);
      else if (n != len[k]) atomicCAS(status, 0, DEV_BAD_LENGTH);
    }
    int count = 0, own = 0;
    if (there(k) && t[k] > 0) {
      own = (t[k] + tpt - 1) / tpt;
      count = blocks_of<BK>(a, n - t[k] + (own - 1) * tpt, n - 1).count;
    }
    rows[lane + 32 * k] = make_uint2((uint32_t)count, (uint32_t)own);
    work += (long long)count * own;
    tiles += own;
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    work += __shfl_xor_sync(0xffffffffu, work, o);
    tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
  }
  each = 0x7fffffff;
  if (tiles > g.tiles) {
    if (lane == 0) atomicCAS(status, 0, DEV_BAD_LENGTH);
    for (int i = lane; i < a.n; i += 32) rows[i] = make_uint2(0, 0);
    __syncwarp();
    return 0;
  }
  // The first lane tries whole tiles, the others of `sizes` lanes the sizes that would give 2, 3 ... sizes parts in
  // `sizes` of ITEMS_A_CTA items a CTA, more than 32 rows with half as many sizes and half of the rows each; the CTA that
  // gets the most sets the time.  (An estimate: what is chosen is counted in integers below, and other CTAs choose the
  // same.)  Without whole tiles among them short calls were split whatever that cost.
  static_assert(SPLIT_ROWS <= 64, "groups of rows");
  const int groups = a.n <= 32 ? 1 : 2, sizes = 32 / groups;
  const long long heads = (long long)a.G * g.hgroups, want = (long long)ITEMS_A_CTA * g.ctas * (lane % sizes + 1);
  const int mine = lane % sizes == 0 ? 0x7fffffff : (int)max((long long)MIN_BLOCKS, (sizes * work * heads + want - 1) / want);
  const float inv = 1.f / (float)mine;
  float items = 0.f, most = 0.f;
  __syncwarp();
  for (int i = lane / sizes; i < a.n; i += groups) {
    const uint2 row = rows[i];
    const float c = (float)row.x, p = fmaxf(1.f, ceilf(fmaf(c, inv, -1e-3f)));
    items = fmaf((float)row.y, p, items);
    most = fmaxf(most, ceilf(__fdividef(c, p) - 1e-3f));
  }
  for (int o = sizes; o < 32; o <<= 1) {
    items += __shfl_xor_sync(0xffffffffu, items, o);
    most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  }
  const float rounds = fabsf(ceilf(items * (float)heads / (float)g.ctas - 1e-3f));
  const float join = items > (float)tiles + 0.5f ? JOIN_COST + fminf(items * (float)heads * g.join, JOIN_MOST) : 0.f;
  const uint32_t cost = __float_as_uint(rounds * (most + (float)ITEM_COST) + join);
  const uint32_t least = __reduce_min_sync(0xffffffffu, cost);          // (positive: ordered like its bits)
  each = __shfl_sync(0xffffffffu, mine, __ffs(__ballot_sync(0xffffffffu, cost == least)) - 1);
  int before = 0;
  for (int i0 = 0; i0 < a.n; i0 += 32) {
    const uint2 row = i0 + lane < a.n ? rows[i0 + lane] : make_uint2(0, 0);
    const int own = (int)row.y * items_of((int)row.x, each);
    int run = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += v;
    }
    if (i0 + lane < a.n) rows[i0 + lane].y = row.y | (uint32_t)(before + run - own) << 16;
    before += __shfl_sync(0xffffffffu, run, 31);
  }
  __syncwarp();
  return before;
}

template <class T, int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1) tc_kernel(const __grid_constant__ TcArgs g) {
  extern __shared__ __align__(1024) unsigned char sm[];
  using C = Cfg<D>;
  constexpr int QT = C::QT, ST = C::STAGES;
  const AttnArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)uniform(tid >> 5);
  const uint32_t sb = smem_u32(sm);
  auto bar = [&](int k) { return sb + C::BAR + 8u * (uint32_t)k; };
  volatile int32_t* flags = reinterpret_cast<int32_t*>(sm + C::FLAGS);   // [stage][checker] the block is added up key by key
  Item* const items = reinterpret_cast<Item*>(sm + C::ITEM);

  pdl_launch_dependents();
  if (tid >= 64 && tid < 67) {            // the tensor maps, into their cache
    const CUtensorMap* m = tid == 64 ? &g.mq : tid == 65 ? &g.mk : &g.mv;
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
  }
  if (warp == 0) tc::tmem_alloc(sb + C::TSLOT, 512);
  if (tid == 32) {
    for (int k = 0; k < C::BARS; ++k) {
      auto of = [&](int first) { return k >= first && k < first + 4; };
      // a tile's four softmax warps; everyone who reads an item; a warp a tile
      mbar_init(bar(k), of(C::PREADY) ? 4 : of(C::IEMPTY) ? 1 + 7 * QT : of(C::KEMPTY) || of(C::VEMPTY) || of(C::VOK) ? QT : 1);
    }
    fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tm = uniform(*reinterpret_cast<volatile uint32_t*>(sm + C::TSLOT));

  // A wait (of a whole warp) that ran out: the warp waits no more and leaves, and so does every warp that waits for it.
  bool ok = true;
  auto wait = [&](int k, uint32_t phase) {
    if (!ok) return false;
    bool in = mbar_try_wait(bar(k), phase & 1u);
    if (!__all_sync(0xffffffffu, in)) {
      if (!in) in = wait_long(bar(k), phase & 1u, g.wait_ns);
      ok = __all_sync(0xffffffffu, in);
    }
    return ok;
  };
  // The next item (number `no` of this CTA's), for whole warps.
  auto peek = [&](uint32_t no, Item& it) {
    if (!wait(C::IFULL + no % ITEMS, no / ITEMS)) return false;
    it = items[no % ITEMS];
    return it.x >= 0;
  };
  auto release = [&](uint32_t no) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::IEMPTY + no % ITEMS));
  };
  auto block_at = [&](const Item& it, int b) { return b < it.sink_blocks ? b : it.first + b - it.sink_blocks; };
  auto masked = [&](const Item& it, int j0) { return !all_see(a, it.pos0, it.pos0 + it.nt - 1, j0, j0 + BK); };

  constexpr int SW = 4 + 4 * QT;           // the first warp behind those of the softmax
  if (warp < 4 || warp >= SW) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::AUX_REGS));
    if (warp == 0) {
      // ---- copies.  Pages are looked up for 32 pages at a time, a batch ahead.
      uint32_t no = 0, blocks = 0, filled = 0;
      const int box = min(1 << a.page_shift, BK), pages = BK / box, ahead = 32 / pages;
      const uint32_t qbytes = 128u * (uint32_t)(g.hpt * g.tpt) * (D / 64), pbytes = 128u * (uint32_t)box * (D / 64);
      Item it;
      for (; ok && peek(no, it); ++no) {
        release(no);
        if (it.b0 == it.b1) continue;
        const int p1 = it.pos0 + it.nt - 1;
        const int32_t* const row = a.table + (int64_t)it.slot * a.table_stride;
        // this lane's page of the batch from block b on: its id, and whether some token sees a key of it
        auto look_up = [&](int b, uint32_t& mask) {
          b += lane / pages;
          const int jp = block_at(it, b) * BK + (lane % pages) * box, lo = it.pos0 - a.window + 1;
          const bool got = b < it.b1 && jp <= p1 && (a.window == 0 || jp + box > lo || jp < a.sinks);
          mask = __ballot_sync(0xffffffffu, got);
          return got ? row[jp >> a.page_shift] : 0;
        };
        uint32_t mask, mask_next = 0;
        int ids = look_up(it.b0, mask), ids_next = 0, used = 0;
        for (int t = 0; t < QT && ok; ++t) {
          if (!wait(C::QEMPTY + t, filled + 1)) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(C::QFULL + t), qbytes);
            for (int e = 0; e < D / 64; ++e)
              tma5(sb + C::Q + t * C::QTILE + e * C::QBLK, &g.mq, 64 * e, it.h0, it.gh, it.begin + it.t0 + t * g.tpt,
                   a.starts ? 0 : it.row, bar(C::QFULL + t));
          }
          __syncwarp();
        }
        ++filled;
        for (int b = it.b0; b < it.b1 && ok; ++b, ++blocks) {
          if (used == 0 && b + ahead < it.b1) ids_next = look_up(b + ahead, mask_next);
          const bool got = lane < pages && (mask >> (used * pages + lane) & 1u);
          int id = __shfl_sync(0xffffffffu, ids, used * pages + lane);
          if (got && (unsigned)id >= (unsigned)a.num_pages) {
            atomicCAS(&g_tc_status, 0, DEV_BAD_PAGE);
            id = 0;
          }
          const uint32_t bytes = pbytes * __popc(__ballot_sync(0xffffffffu, got));
          const uint32_t s = blocks % ST, ph = blocks / ST;
          const int off = (block_at(it, b) * BK + lane * box) & ((1 << a.page_shift) - 1);
          if (!wait(C::KEMPTY + s, ph + 1)) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(C::KFULL + s), bytes);
          __syncwarp();
          if (got)
#pragma unroll
            for (int e = 0; e < D / 64; ++e)
              tma4(sb + C::K + s * C::KTILE + e * C::KBLK + lane * box * 128, &g.mk, 64 * e, off, it.gh, id, bar(C::KFULL + s));
          __syncwarp();
          if (!wait(C::VEMPTY + s, ph + 1)) {
            ++blocks;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(C::VFULL + s), bytes);
          __syncwarp();
          if (got)
#pragma unroll
            for (int e = 0; e < D / 64; ++e)
              tma4(sb + C::V + s * C::KTILE + e * C::KBLK + lane * box * 128, &g.mv, 64 * e, off, it.gh, id, bar(C::VFULL + s));
          __syncwarp();
          if (++used == ahead) {
            used = 0;
            ids = ids_next;
            mask = mask_next;
          }
        }
      }
      if (lane == 0) {
        // what is on its way lands before the memory is given back (other roles may have given up waiting for it): the
        // last copy into each place
        for (int t = 0; t < QT; ++t)
          if (filled) mbar_drain(bar(C::QFULL + t), (filled - 1) & 1u);
        for (uint32_t k = 0; k < ST && k < blocks; ++k) {
          const uint32_t b = blocks - 1 - k;
          mbar_drain(bar(C::KFULL + b % ST), (b / ST) & 1u);
          mbar_drain(bar(C::VFULL + b % ST), (b / ST) & 1u);
        }
      }
    } else if (warp == 1 || (QT == 2 && warp == SW + 1)) {
      // ---- S = Q K^T of a tile, block by block, as soon as its place in TMEM is free: P of the step before on the chain
      // has been used
      const uint32_t t = warp == 1 ? 0 : 1;
      const uint64_t qd = tc::sdesc128(sb + C::Q + t * C::QTILE, 16u, 1024u), kd = tc::sdesc128(sb + C::K, 16u, 1024u);
      uint32_t no = 0, s = 0, sp = 0, step = 0, done = 0;      // stage and its phase; steps; items with blocks
      Item it;
      for (; ok && peek(no, it); ++no) {
        const uint32_t nb = uniform((uint32_t)(it.b1 - it.b0));
        release(no);
        if (nb > 0) wait(C::QFULL + t, done++);
        for (uint32_t b = 0; b < nb && ok; ++b, ++step) {
          const uint32_t chain = (step & 1u) * QT + t;
          const uint64_t k0 = kd + s * (C::KTILE >> 4);
          wait(C::PVDONE + chain, (step >> 1) + 1);
          if (!wait(C::KFULL + s, sp)) break;
          tc::fence_after_sync();
          if (elect()) {
#pragma unroll
            for (uint32_t k = 0; k < D / 16; ++k)
              tc::mma_bf16(tm + C::S_COL + chain * BK, qd + ((k >> 2) * (C::QBLK >> 4) + (k & 3) * 2u),
                           k0 + ((k >> 2) * (C::KBLK >> 4) + (k & 3) * 2u), idesc<T>(BK, false), k > 0);
            tc::mma_commit(bar(C::SFULL + chain));
            tc::mma_commit(bar(C::KEMPTY + s));
            if (b == nb - 1) tc::mma_commit(bar(C::QEMPTY + t));
          }
          __syncwarp();
          if (++s == ST) {
            s = 0;
            ++sp;
          }
        }
      }
      if (elect()) {                       // products on their way end before the memory is given back
        tc::mma_commit(bar(C::DRAIN + t));
        mbar_drain(bar(C::DRAIN + t), 0);
      }
    } else if (warp == 3 || (QT == 2 && warp == SW + 3)) {
      // ---- O += P V of a tile
      const uint32_t t = warp == 3 ? 0 : 1;
      const uint64_t vd = tc::sdesc128(sb + C::V, C::KBLK, 1024u);
      uint32_t no = 0, s = 0, sp = 0, step = 0;
      Item it;
      for (; ok && peek(no, it); ++no) {
        const uint32_t nb = uniform((uint32_t)(it.b1 - it.b0));
        release(no);
        for (uint32_t b = 0; b < nb && ok; ++b, ++step) {
          const uint32_t chain = (step & 1u) * QT + t;
          const uint64_t v0 = vd + s * (C::KTILE >> 4);
          wait(C::VFULL + s, sp);
          wait(C::VOK + s, sp);
          const uint32_t skip = uniform((uint32_t)(flags[QT * s] | flags[QT * s + QT - 1]));
          if (!wait(C::PREADY + chain, step >> 1)) break;
          tc::fence_after_sync();
          if (elect()) {
            if (!skip) {
              // 128 columns a product: one of 256 with A in TMEM ended in an illegal access
              constexpr uint32_t N = D < 128 ? D : 128;
#pragma unroll
              for (uint32_t c = 0; c < D / N; ++c)
#pragma unroll
                for (uint32_t k = 0; k < BK / 16; ++k)
                  tc::mma_bf16_ta(tm + C::O_COL + t * D + c * N, tm + C::S_COL + chain * BK + 8 * k,
                                  v0 + c * (2 * C::KBLK >> 4) + k * (2048u >> 4), idesc<T>(N, true), b > 0 || k > 0);
            }
            tc::mma_commit(bar(C::PVDONE + chain));
            tc::mma_commit(bar(C::VEMPTY + s));
          }
          __syncwarp();
          if (++s == ST) {
            s = 0;
            ++sp;
          }
        }
      }
      if (elect()) {
        tc::mma_commit(bar(C::DRAIN + 2 + t));
        mbar_drain(bar(C::DRAIN + 2 + t), 0);
      }
    } else if (warp == SW) {
      // ---- items: every CTA takes each grid'th of the list, longest first as far as that is known
      uint32_t no = 0;
      const int heads = a.G * g.hgroups;
      auto publish = [&](const Item& it) {
        if (!wait(C::IEMPTY + no % ITEMS, no / ITEMS + 1)) return;
        if (lane == 0) {
          items[no % ITEMS] = it;
          mbar_arrive(bar(C::IFULL + no % ITEMS));
        }
        __syncwarp();
        ++no;
      };
      Item it{};
      uint2* const rows = reinterpret_cast<uint2*>(sm + C::ROWS);
      int total = g.total, most = 0;       // most: blocks of an item
      if (g.split) {
        total = plan_split(g, QT * g.tpt, rows, most, &g_tc_status) * heads;
        if (blockIdx.x == 0)               // for the join: tiles, items of each, items before
          for (int i = lane; i < a.n; i += 32) {
            const uint2 v = rows[i];
            reinterpret_cast<int4*>(a.ws)[i] = make_int4(v.y & 0xffff, items_of((int)v.x, most), v.y >> 16, 0);
          }
      }
      for (int k = blockIdx.x; k < total && ok; k += gridDim.x) {
        const int kx = k / heads, h = k - kx * heads;
        Tile w;
        int pieces = 1, piece = 0;
        if (g.split) {
          int row = 0;                     // the last that starts at or before item kx
          for (int i0 = 0; i0 < a.n; i0 += 32) {
            const uint32_t m = __ballot_sync(0xffffffffu, i0 + lane < a.n && (int)(rows[min(i0 + lane, a.n - 1)].y >> 16) <= kx);
            if (m == 0) break;
            row = i0 + 31 - __clz(m);
          }
          const uint2 v = rows[row];
          const int off = kx - (int)(v.y >> 16);
          pieces = items_of((int)v.x, most);
          piece = off % pieces;
          if (!make_tile(a, row, (int)(v.y & 0xffff) - 1 - off / pieces, QT * g.tpt, w, &g_tc_status)) continue;
        } else {
          // token-major: the last tiles of all rows first
          const int x = g.per_row ? (kx % a.n) * g.per_row + g.per_row - 1 - kx / a.n : g.tiles - 1 - kx;
          if (!find_tile(a, x, QT * g.tpt, w, &g_tc_status)) continue;
        }
        const Blocks bl = blocks_of<BK>(a, w.pos0, w.pos0 + w.nt - 1);
        const int each = (bl.count + pieces - 1) / pieces;
        it.b0 = min(bl.count, piece * each);
        it.b1 = min(bl.count, it.b0 + each);
        it.whole = pieces == 1;
        if (piece > 0 && it.b0 == it.b1) continue;
        it.part = k;
        it.sink_blocks = bl.sink_blocks;
        it.first = bl.first;
        it.x = 0;
        it.row = w.row;
        it.slot = w.slot;
        it.begin = w.begin;
        it.t0 = w.t0;
        it.nt = w.nt;
        it.pos0 = w.pos0;
        it.gh = h / g.hgroups;
        it.h0 = (h - it.gh * g.hgroups) * R;
        publish(it);
      }
      it.x = -1;
      publish(it);
    } else if (warp == 2 || (QT == 2 && warp == SW + 2)) {
      // ---- blocks that not every token sees, half of the columns a warp: unseen keys' values become zero, values that
      // are not finite are found
      const int half = warp == 2 ? 0 : 1;
      uint32_t no = 0, blocks = 0;
      Item it;
      if (g.test_stall && blockIdx.x == 0 && half == 0) {
        // Test only: a barrier that nothing arrives on, at half the limit, so that this warp's wait is the first to run out.
        mbar_wait(bar(C::NEVER), 0, &g_tc_waits, DEV_TEST_STALL, g.wait_ns / 2);
        ok = false;
      }
      for (; ok && peek(no, it); ++no) {
        release(no);
        const int p1 = it.pos0 + it.nt - 1;
        for (int b = it.b0; b < it.b1 && ok; ++b, ++blocks) {
          const uint32_t s = blocks % ST;
          if (!wait(C::VFULL + s, blocks / ST)) break;
          const int j0 = block_at(it, b) * BK;
          bool odd = false;
          if (masked(it, j0)) {
            const uint32_t dead[2] = {__ballot_sync(0xffffffffu, none_sees(a, it.pos0, p1, j0 + lane)),
                                      __ballot_sync(0xffffffffu, none_sees(a, it.pos0, p1, j0 + 32 + lane))};
            constexpr int PIECES = BK * D / 8 / QT;
            uint4* const v = reinterpret_cast<uint4*>(sm + C::V + s * C::KTILE) + half * PIECES;
            uint32_t acc = 0;
#pragma unroll 8
            for (int e = lane; e < PIECES; e += 32) {
              const int row = ((e + half * PIECES) >> 3) & (BK - 1);
              if ((row < 32 ? dead[0] : dead[1]) >> (row & 31) & 1u) {
                v[e] = make_uint4(0u, 0u, 0u, 0u);
              } else {
                const uint4 x = v[e];
                acc = not_finite<T>(not_finite<T>(not_finite<T>(not_finite<T>(acc, x.x), x.y), x.z), x.w);
              }
            }
            tc::fence_smem_to_async();
            odd = __any_sync(0xffffffffu, (acc & 0x7fff7fffu) != 0);
          }
          if (lane == 0) flags[QT * s + half] = odd;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::VOK + s));
        }
      }
    }
  } else {
    // ---- softmax: thread = row of tile t; QT = 1: of the only tile
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::ROW_REGS));
    const int t = (warp >> 2) - 1, q4 = warp & 3, r = 32 * q4 + lane, per = a.H / a.G;
    const uint32_t tl = tm + ((uint32_t)(32 * q4) << 16), o_col = tl + C::O_COL + t * D;
    const int tok = r / g.hpt, hd = r - tok * g.hpt;
    const f2 scale2 = mk2(a.scale_log2, a.scale_log2), lift2 = mk2(LIFT<T>, LIFT<T>);
    uint32_t no = 0, steps = 0, blocks = 0;
    Item it;
    for (; ok && peek(no, it); ++no) {
      release(no);
      const int tk = t * g.tpt + tok, pos = it.pos0 + tk;
      const bool mine = tok < g.tpt && tk < it.nt && it.h0 + hd < per;   // other rows hold anything
      float m = -INFINITY, l = 0.f;       // the reference is m scale log2(e) - LIFT
      // blocks that every token of the item sees whole: [full0, full1) of the window's, those before full2 of the sinks'
      const int shift = it.sink_blocks - it.first, p1 = it.pos0 + it.nt - 1;
      const int full0 = a.window ? max(it.sink_blocks, shift + (max(0, p1 - a.window + 1) + BK - 1) / BK) : 0;
      const int full1 = shift + (it.pos0 + 1) / BK, full2 = a.window ? min(min(it.sink_blocks, a.sinks / BK), (it.pos0 + 1) / BK) : 0;
      for (int b = it.b0; b < it.b1 && ok; ++b, ++steps, ++blocks) {
        const uint32_t chain = (steps & 1u) * QT + t, before = ((steps & 1u) ^ 1u) * QT + t, ph = steps >> 1;
        const uint32_t s_col = tl + C::S_COL + chain * BK;
        const int j0 = block_at(it, b) * BK;
        const bool part = !((b >= full0 && b < full1) || b < full2);
        if (!wait(C::SFULL + chain, ph)) break;
        tc::fence_after_sync();
        uint32_t seen[BK / 32];           // keys of the block that the row sees
        if (part) {
          const int hi = pos - j0, lo = a.window ? hi - a.window : -1, sk = a.window ? a.sinks - j0 : 0;
#pragma unroll
          for (int c = 0; c < BK / 32; ++c)
            seen[c] = bits_to(hi - 32 * c) & (~bits_to(lo - 32 * c) | bits_to(sk - 1 - 32 * c));
        }
        uint32_t s[BK / 32][32], p[BK / 2];
#pragma unroll
        for (int c = 0; c < BK / 32; ++c) tc::tmem_ld32(s_col + 32 * c, s[c]);
#pragma unroll
        for (int c = 0; c < BK / 32; ++c) tc::tmem_wait_ld(s[c]);
        if (part)
#pragma unroll
          for (int c = 0; c < BK / 32; ++c)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!(seen[c] >> k & 1u)) s[c][k] = 0xff800000u;
        bool lift = __any_sync(0xffffffffu, mine && m == -INFINITY);     // nothing seen so far
        for (bool again = false;; again = true) {
          if (lift) {                    // a new reference: the row's maximum so far
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < BK / 32; ++c) {
#pragma unroll
              for (int k = 0; k < 32; ++k) top[k & 3] = fmaxf(top[k & 3], __uint_as_float(s[c][k]));
            }
            const float was = m;
            m = fmaxf(was, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
            const float f = ex2_f((was - held(m)) * a.scale_log2);
            l *= f;
            if (b > it.b0) {
              if (!wait(C::PVDONE + before, (steps - 1) >> 1)) break;
              tc::fence_after_sync();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tc::tmem_ld32(o_col + 32 * c, o);
                tc::tmem_wait_ld(o);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                tc::tmem_st32(o_col + 32 * c, o);
              }
            }
          }
          const float base = -held(m);
          const f2 base2 = mk2(base, base);
          f2 sum[2] = {mk2(0.f, 0.f), mk2(0.f, 0.f)};
#pragma unroll
          for (int c = 0; c < BK / 32; ++c) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float x, y;
              // differences first: scores as large as the type goes keep theirs
              un2(fma2(add2(mk2(__uint_as_float(s[c][2 * k]), __uint_as_float(s[c][2 * k + 1])), base2), scale2, lift2), x, y);
              x = ex2_f(x);
              y = ex2_f(y);
              sum[k & 1] = add2(sum[k & 1], mk2(x, y));
              p[16 * c + k] = pack2<T>(x, y);
            }
          }
          float x, y, z, w;
          un2(sum[0], x, y);
          un2(sum[1], z, w);
          x = (x + y) + (z + w);
          lift = !again && __any_sync(0xffffffffu, mine && !(x <= LIMIT<T>));
          if (lift) continue;
          l += x;
          break;
        }
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < BK / 64; ++c) tc::tmem_st32(s_col + 32 * c, *reinterpret_cast<uint32_t (*)[32]>(p + 32 * c));
        tc::tmem_wait_st();
        if (part) {
          const uint32_t st = blocks % ST;
          if (!wait(C::VOK + st, blocks / ST)) break;
          if (flags[QT * st] | flags[QT * st + QT - 1]) {
            if (!wait(C::VFULL + st, blocks / ST)) break;
            if (b > it.b0 && !wait(C::PVDONE + before, (steps - 1) >> 1)) break;
            tc::fence_after_sync();
            by_keys<T, D>(a, sm + C::V + st * C::KTILE, s_col, o_col, pos, j0, b == it.b0);
          }
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::PREADY + chain));
      }
      if (!ok) break;
      const bool any = it.b1 > it.b0;
      if (any) {
        if (!wait(C::PVDONE + ((steps - 1) & 1u) * QT + t, (steps - 1) >> 1)) break;
        tc::fence_after_sync();
      }
      // ---- the row's result
      // Through shared memory, 128 bytes of every row at a time, so that eight lanes write a row's together: a row a lane
      // took 5100 cycles a tile of 128 x 128.
      const float inv = l == 0.f ? 0.f : 1.f / l;
      unsigned char* const stage = sm + C::OUT + (warp - 4) * 4096;
      unsigned char* to = nullptr;         // this lane's row
      if (mine && it.whole) {
        to = reinterpret_cast<unsigned char*>(static_cast<T*>(a.o) + (int64_t)(it.begin + it.t0 + tk) * a.o_st +
                                              (int64_t)it.row * a.o_sn + ((int64_t)it.gh * per + it.h0 + hd) * a.d);
      } else if (mine) {
        float* part = a.ws + PLAN + ((int64_t)it.part * (QT * R) + t * R + r) * (D + 4);
        *reinterpret_cast<float2*>(part) = make_float2(m * a.scale_log2, l);   // (the same LIFT in every part)
        to = reinterpret_cast<unsigned char*>(part + 4);
      }
      const int bytes = it.whole ? 2 * a.d : 4 * D, chunks = it.whole ? D / 64 : D / 32;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t o[32];
          if (it.whole || half == 0) {
            if (any) {
              tc::tmem_ld32(o_col + (it.whole ? 64 * c + 32 * half : 32 * c), o);
              tc::tmem_wait_ld(o);
            }
            if (it.whole) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int i = 8 * k + 2 * e;
                  w[e] = l == 0.f ? 0u : pack2<T>(__uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv);
                }
                *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * half + k) ^ (lane & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
                    make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
          }
        }
        __syncwarp();
        const int piece = lane & 7, at = 128 * c + 16 * piece;
        uint4 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + (lane >> 3);
          v[i] = *reinterpret_cast<const uint4*>(stage + row * 128 + ((piece ^ (row & 7)) << 4));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          unsigned char* const dst = reinterpret_cast<unsigned char*>(
              __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), 4 * i + (lane >> 3)));
          if (dst && at < bytes) *reinterpret_cast<uint4*>(dst + at) = v[i];
        }
        __syncwarp();
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    tc::fence_after_sync();
    tc::tmem_dealloc(tm, 512);
  }
}

// The parts of split items.  Block (tile, head, part of the rows): a warp a row, its parts in order; or, where that is
// less to do one after the other (few rows, many parts), all warps a row, parts in turns and their sums in order: 4
// tokens of 8 heads over one behind 131072 take 33 us, 106 with a warp a row.
constexpr int JOIN_WARPS = 8;
template <class T, int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS) tc_join(const __grid_constant__ TcArgs g) {
  using C = Cfg<D>;
  constexpr int QT = C::QT, V = D / 32 < 4 ? 2 : 4, P = D / 32 / V;     // columns of a lane: P pieces of V
  __shared__ float o_of[JOIN_WARPS][D];
  __shared__ float2 ml_of[JOIN_WARPS];
  const AttnArgs& a = g.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, per = a.H / a.G, gh = blockIdx.y / g.hgroups;
  const int h0 = (blockIdx.y % g.hgroups) * R;
  Tile w;
  const bool tile = find_tile(a, blockIdx.x, QT * g.tpt, w, &g_tc_status);   // (what it reads was there before the first launch)
  pdl_wait_primary();                   // (also by blocks without work: this launch must not end before the first)
  if (!tile) return;
  const int4 plan = reinterpret_cast<const int4*>(a.ws)[w.row];              // tiles, items of each, items before
  if (plan.y == 1) return;
  const Blocks bl = blocks_of<BK>(a, w.pos0, w.pos0 + w.nt - 1);
  const int each = (bl.count + plan.y - 1) / plan.y, parts = bl.count > 0 ? (bl.count + each - 1) / each : 1;
  const int first = plan.z + (plan.x - 1 - w.t0 / (QT * g.tpt)) * plan.y;
  const int64_t item = (int64_t)first * gridDim.y + blockIdx.y, next = (int64_t)gridDim.y * QT * R * (D + 4);
  const int heads = min(g.hpt, per - h0), rows = w.nt * heads, z = gridDim.z;
  const bool share = (rows + z - 1) / z * (parts / JOIN_WARPS + 4) < (rows + JOIN_WARPS * z - 1) / (JOIN_WARPS * z) * parts;
  for (int e = share ? blockIdx.z : JOIN_WARPS * blockIdx.z + warp; e < rows; e += share ? z : JOIN_WARPS * z) {
    const int t = e / heads, h = e - t * heads, sub = t / g.tpt;
    const float* part = a.ws + PLAN + (item * (QT * R) + sub * R + (t - sub * g.tpt) * g.hpt + h) * (D + 4);
    float m = -INFINITY, l = 0.f, o[P][V];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int v = 0; v < V; ++v) o[p][v] = 0.f;
    // four parts at a time: all of their loads, then the sums against the largest reference so far
    const int by = share ? JOIN_WARPS : 1;
    for (int k0 = share ? warp : 0; k0 < parts; k0 += 4 * by) {
      float2 ml[4];
      float x[4][P][V];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool in = k0 + u * by < parts;
        const float* q = part + (in ? k0 + u * by : 0) * next;
        ml[u] = *reinterpret_cast<const float2*>(q);
        if (!in) ml[u] = make_float2(-INFINITY, 0.f);
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const float* from = q + 4 + (32 * p + lane) * V;
          if constexpr (V == 4) {
            const float4 w4 = *reinterpret_cast<const float4*>(from);
            x[u][p][0] = w4.x, x[u][p][1] = w4.y, x[u][p][2] = w4.z, x[u][p][3] = w4.w;
          } else {
            const float2 w2 = *reinterpret_cast<const float2*>(from);
            x[u][p][0] = w2.x, x[u][p][1] = w2.y;
          }
        }
      }
      const float was = m;
      m = fmaxf(fmaxf(m, fmaxf(ml[0].x, ml[1].x)), fmaxf(ml[2].x, ml[3].x));
      const float base = held(m), f0 = ex2_f(was - base);
      l *= f0;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int v = 0; v < V; ++v) o[p][v] *= f0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (ml[u].y == 0.f) continue;   // saw nothing
        const float f = ex2_f(ml[u].x - base);
        l = fmaf(ml[u].y, f, l);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int v = 0; v < V; ++v) o[p][v] = fmaf(x[u][p][v], f, o[p][v]);
      }
    }
    if (share) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int v = 0; v < V; ++v) o_of[warp][(32 * p + lane) * V + v] = o[p][v];
      if (lane == 0) ml_of[warp] = make_float2(m, l);
      __syncthreads();
      if (warp == 0) {
        float top = m;
        for (int x = 1; x < JOIN_WARPS; ++x) top = fmaxf(top, ml_of[x].x);
        const float base = held(top), f0 = ex2_f(m - base);
        l *= f0;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int v = 0; v < V; ++v) o[p][v] *= f0;
        for (int x = 1; x < JOIN_WARPS; ++x) {
          if (ml_of[x].y == 0.f) continue;
          const float f = ex2_f(ml_of[x].x - base);
          l = fmaf(ml_of[x].y, f, l);
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int v = 0; v < V; ++v) o[p][v] = fmaf(o_of[x][(32 * p + lane) * V + v], f, o[p][v]);
        }
      }
    }
    if (!share || warp == 0) {
      T* out = static_cast<T*>(a.o) + (int64_t)(w.begin + w.t0 + t) * a.o_st + (int64_t)w.row * a.o_sn + ((int64_t)gh * per + h0 + h) * a.d;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int v = 0; v < V; ++v)
          if ((32 * p + lane) * V + v < a.d) out[(32 * p + lane) * V + v] = from_f<T>(l == 0.f ? 0.f : o[p][v] / l);
    }
    if (share) __syncthreads();         // the sums are read
  }
}

thread_local TcArgs t_tc;

template <class T, int D>
cudaError_t go(const TcArgs& g, int grid, cudaStream_t s) {
  static thread_local int ready = -1;  // the device whose limit is raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (ready != dev) {
    e = cudaFuncSetAttribute(tc_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<D>::BYTES);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, tc_kernel<T, D>);
    if (e != cudaSuccess) return e;
    if ((fa.numRegs + 7) / 8 * 8 < Cfg<D>::LAUNCH_REGS) return cudaErrorInvalidConfiguration;   // the softmax would wait for its share
    ready = dev;
  }
  tc_kernel<T, D><<<grid, Cfg<D>::THREADS, Cfg<D>::BYTES, s>>>(g);
  e = cudaGetLastError();
  if (e != cudaSuccess || !g.split) return e;
  cudaLaunchConfig_t c{};
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  const int heads = g.a.G * g.hgroups, z = 4 * g.ctas / (g.tiles * heads);        // some four blocks an SM
  c.gridDim = dim3((unsigned)g.tiles, (unsigned)heads, (unsigned)(z < 2 ? 2 : z > 32 ? 32 : z));
  c.blockDim = dim3(32 * JOIN_WARPS);
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, tc_join<T, D>, g);
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
bool encode(CUtensorMap* m, int dtype, int rank, void* p, const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return fn(m, dtype == mx::T_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank, p, dims,
            strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
int width_of(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }
int tiles_a_cta(int d) { return d > 128 ? 1 : 2; }

}  // namespace

// 16-bit types, tensors that tensor maps can describe (16-byte aligned, strides above zero and below 2^40 bytes), and
// items that are counted in 32 bits, a step of the grid behind the last one included.
bool tc_fits(int dtype, bool vec, const AttnArgs& a) {
  auto ok = [](int64_t stride, int64_t extent) { return extent == 1 || (stride > 0 && stride < (int64_t)1 << 39); };
  for (const PoolView& v : {a.kp, a.vp})
    if (!ok(v.st, 2) || !ok(v.sg, a.G) || !ok(v.sp, a.num_pages)) return false;
  const int per = a.H / a.G, tpt = tiles_a_cta(a.d) * (R / (per < R ? per : R));
  const int64_t items = tiles_of(a.n, a.T, a.starts != nullptr, tpt) * a.G * ((per + R - 1) / R);
  return dtype != mx::T_F32 && vec && ok(a.q_st, a.T) && ok(a.q_sn, a.starts ? 1 : a.n) && items < 0x7fffffff - (1 << 16);
}

AttnPlan tc_plan(int n, int T, bool packed, int H, int G, int d, int sms) {
  AttnPlan p{};
  const int per = H / G, hpt = per < R ? per : R, qt = tiles_a_cta(d);
  p.rows = qt * R;
  p.tpt = R / hpt;
  p.hgroups = (per + R - 1) / R;
  const int64_t tiles = tiles_of(n, T, packed, qt * p.tpt);
  p.tiles = (int32_t)tiles;
  const int64_t units = tiles * G * p.hgroups;
  // Split where there are fewer than two tiles and heads for an SM.
  const bool split = units < 2 * (int64_t)sms && n <= SPLIT_ROWS;
  p.splits = split ? 2 : 1;
  p.grid = (int32_t)(split || units > sms ? sms : units);
  p.ws_bytes = split ? 4 * (PLAN + (ITEMS_A_CTA * (int64_t)sms + units) * p.rows * (width_of(d) + 4)) : 0;
  return p;
}

cudaError_t launch_tc(int dtype, const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  TcArgs& g = t_tc;
  const int per = a.H / a.G, page = 1 << a.page_shift;
  g.a = a;
  g.hpt = per < R ? per : R;
  g.tpt = p.tpt;
  g.hgroups = p.hgroups;
  g.tiles = p.tiles;
  g.split = p.splits > 1;
  g.ctas = p.grid;
  g.total = p.tiles * a.G * p.hgroups;
  g.per_row = a.starts ? 0 : p.tiles / a.n;
  // (tiles as full as those of rows of the average length)
  const float fill = (float)a.T / ((float)(a.starts ? a.n : 1) * (float)(tiles_a_cta(a.d) * p.tpt));
  g.join = (a.d <= 64 ? 0.5f : 1.f) * (fill < 1.f ? fill : 1.f) / JOIN_PARTS;
  g.wait_ns = WAIT_LIMIT_NS;
  if (const char* e = getenv("DL_TEST_WAIT_MS")) {
    const long ms = atol(e);
    if (ms > 0 && ms < 2000) g.wait_ns = (unsigned long long)ms * 1000000ull;
  }
  const char* stall = getenv("DL_TEST_STALL");
  g.test_stall = stall && atoi(stall) == 1;
  const cuuint64_t d = (cuuint64_t)a.d;
  const cuuint64_t qdims[5] = {d, (cuuint64_t)per, (cuuint64_t)a.G, (cuuint64_t)a.T, (cuuint64_t)(a.starts ? 1 : a.n)};
  const auto bytes = [](int64_t stride, int64_t extent) { return (cuuint64_t)(extent == 1 ? 16 : 2 * stride); };   // (any, of one)
  const cuuint64_t qst[4] = {2 * d, 2 * d * per, bytes(a.q_st, a.T), bytes(a.q_sn, a.starts ? 1 : a.n)};
  const cuuint32_t qbox[5] = {64, (cuuint32_t)g.hpt, 1, (cuuint32_t)g.tpt, 1};
  const cuuint32_t pbox[4] = {64, (cuuint32_t)(page < BK ? page : BK), 1, 1};
  bool ok = encode(&g.mq, dtype, 5, const_cast<void*>(a.q), qdims, qst, qbox);
  for (int k = 0; k < 2; ++k) {
    const PoolView& v = k ? a.vp : a.kp;
    const cuuint64_t dims[4] = {d, (cuuint64_t)page, (cuuint64_t)a.G, (cuuint64_t)a.num_pages};
    const cuuint64_t st[3] = {bytes(v.st, 2), bytes(v.sg, a.G), bytes(v.sp, a.num_pages)};
    ok = ok && encode(k ? &g.mv : &g.mk, dtype, 4, v.p, dims, st, pbox);
  }
  if (!ok) return cudaErrorInvalidValue;
  const int D = width_of(a.d);
  if (dtype == mx::T_BF16)
    return D == 64 ? go<__nv_bfloat16, 64>(g, p.grid, s) : D == 128 ? go<__nv_bfloat16, 128>(g, p.grid, s)
                                                                    : go<__nv_bfloat16, 256>(g, p.grid, s);
  return D == 64 ? go<__half, 64>(g, p.grid, s) : D == 128 ? go<__half, 128>(g, p.grid, s) : go<__half, 256>(g, p.grid, s);
}

cudaError_t read_tc_status(cudaStream_t s, int32_t* code) {
  int32_t waits = 0;
  cudaError_t e = take_status(g_tc_status, s, code);
  if (e == cudaSuccess) e = take_status(g_tc_waits, s, &waits);
  if (waits) *code = waits;
  return e;
}

}  // namespace at
}  // namespace dl
