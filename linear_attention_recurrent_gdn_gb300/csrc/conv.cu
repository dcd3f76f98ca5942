// Short causal convolution over time, with its activation, the L2 norm of the
// leading heads and the carried inputs of every slot:
//   z[t, c] = b[c] + sum_j w[c, j] x[t - W + 1 + j, c],   y = act(z)
//   heads below channel l2c:  y / sqrt(sum over the head of y^2 + eps)
// where x at a negative t is the slot's carried input (its last W - 1, oldest
// first) or zero for a fresh row.
//
// A thread takes eight channels and walks the tokens of its tile with the last
// W - 1 of them in registers, the next few on their way from memory, so a value is read once a tile plus W - 1 of every TT tokens
// again.  Aligned tensors: the eight channels are one 16-byte vector of a
// 16-bit type.  Others: eight channels 32 apart, so that a warp's loads of one
// value a lane are still contiguous.  Sums, the activation and the norm are in
// 32 bits, rounded once; pairs of channels share a packed fp32 multiply-add,
// and pairs of sigmoids a reciprocal.  About 2 W + 8 operations a value: HBM
// bound, with the instructions not far behind.
//
// Measured on a GB300 (copy: 6.7 TB/s): prompts of 16 x 512 tokens of 12288
// bf16 channels with the L2 norm of two thirds of them 74 us, 5.5 TB/s (with
// tokens fetched into registers instead of shared memory 110 us: 16 warps an SM
// hold too few loads), fp32 of 4 x 512 x 12288 46 us, 4.4 TB/s; one token of 256 x 12288 10 us, 5.0 TB/s; of 1 x 768 2.1
// us, the launch; 3100 packed tokens of 5123 fp16 channels 33 us, 2.0 TB/s,
// bound by loads and stores of two bytes a lane.
#include <type_traits>

#include "dl_device.cuh"
#include "mixer_device.cuh"

namespace dl {
namespace mx {

namespace {

constexpr int CONV_THREADS = 128;

// Eight values of a thread as they sit in memory: VEC: consecutive; else one
// every 32 channels.
template <class T, bool VEC>
struct Eight {
  static constexpr int NW = VEC && sizeof(T) == 2 ? 4 : 8;
  uint32_t w[NW];

  // p: the thread's first value; valid: how many of the channels from it on exist
  __device__ __forceinline__ void load(const T* p, int valid) {
    if constexpr (VEC) {
      const Vec8<T> v = load8<T, true>(p, valid);
#pragma unroll
      for (int k = 0; k < NW; ++k) w[k] = v.w[k];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (sizeof(T) == 4) w[k] = 32 * k < valid ? __float_as_uint(p[32 * k]) : 0u;
        else w[k] = 32 * k < valid ? reinterpret_cast<const uint16_t*>(p)[32 * k] : 0u;
      }
    }
  }
  __device__ __forceinline__ void store(T* p, int valid) const {
    if constexpr (VEC) {
      Vec8<T> v;
#pragma unroll
      for (int k = 0; k < NW; ++k) v.w[k] = w[k];
      store8<T, true>(p, v, valid);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (32 * k < valid) {
          if constexpr (sizeof(T) == 4) p[32 * k] = __uint_as_float(w[k]);
          else reinterpret_cast<uint16_t*>(p)[32 * k] = (uint16_t)w[k];
        }
    }
  }
  // the value pair 2 k, 2 k + 1 in 32 bits
  __device__ __forceinline__ void pair(int k, float& a, float& b) const {
    if constexpr (sizeof(T) == 4) {
      a = __uint_as_float(w[2 * k]);
      b = __uint_as_float(w[2 * k + 1]);
    } else if constexpr (VEC) {
      unpack2<T>(w[k], a, b);
    } else {
      unpack2<T>(w[2 * k] | (w[2 * k + 1] << 16), a, b);
    }
  }
  __device__ __forceinline__ void set(int k, float a, float b) {
    if constexpr (sizeof(T) == 4) {
      w[2 * k] = __float_as_uint(a);
      w[2 * k + 1] = __float_as_uint(b);
    } else {
      const uint32_t v = pack2<T>(a, b);
      if constexpr (VEC) {
        w[k] = v;
      } else {
        w[2 * k] = v & 0xffffu;
        w[2 * k + 1] = v >> 16;
      }
    }
  }
};

// A thread's channels, weights and outputs.
template <class T, int W, bool VEC>
struct Lane {
  int c, valid;              // first channel, and how many from it on exist
  bool normed;               // this warp has channels of normalised heads
  f2 w[W][4], bias[4];

  __device__ __forceinline__ int chan(int k) const { return VEC ? c + k : c + 32 * k; }

  __device__ __forceinline__ void init(const ConvArgs& a) {
    const int lane = threadIdx.x & 31, base = blockIdx.y * CONV_THREADS * 8 + (threadIdx.x >> 5) * 256;
    c = VEC ? base + 8 * lane : base + lane;
    valid = a.C - c;
    normed = base < a.l2c;
    float wf[W][8], bf[8];
    if (VEC && valid > 0 && (reinterpret_cast<uintptr_t>(a.w) & 15) == 0) {
      // the W weights of eight channels follow one another
      float v[W * 8];
#pragma unroll
      for (int j = 0; j < W; ++j) {
        float t[8];
        weights8<T, true>(a.w, (int64_t)c * W + 8 * j, 8, a.w_f32, t);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[8 * j + k] = t[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < W; ++j) wf[j][k] = v[k * W + j];
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int j = 0; j < W; ++j)
          wf[j][k] = chan(k) >= a.C ? 0.f
                     : a.w_f32      ? static_cast<const float*>(a.w)[(int64_t)chan(k) * W + j]
                                    : to_f(static_cast<const T*>(a.w)[(int64_t)chan(k) * W + j]);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      bf[k] = !a.b || chan(k) >= a.C ? 0.f
              : a.w_f32              ? static_cast<const float*>(a.b)[chan(k)]
                                     : to_f(static_cast<const T*>(a.b)[chan(k)]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      bias[k] = mk2(bf[2 * k], bf[2 * k + 1]);
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][k] = mk2(wf[j][2 * k], wf[j][2 * k + 1]);
    }
  }

  // One token: the window moves on by `cur`; returns y in `out`.  All lanes of the warp take part.  ACT, NORM:
  // whether there is an activation, and normalised heads in this warp; without branches inside, the tokens of
  // a group overlap.
  template <bool ACT, bool NORM>
  __device__ __forceinline__ void token(const ConvArgs& a, const Eight<T, VEC>& cur, f2 (&win)[W - 1][4],
                                        Eight<T, VEC>& out) const {
    f2 z[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float p, q;
      cur.pair(k, p, q);
      const f2 x = mk2(p, q);
      f2 s = bias[k];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s = fma2(w[j][k], win[j][k], s);
      s = fma2(w[W - 1][k], x, s);
#pragma unroll
      for (int j = 0; j + 2 < W; ++j) win[j][k] = win[j + 1][k];
      win[W - 2][k] = x;
      z[k] = ACT ? act2<T, true>(s) : s;
    }
    if constexpr (NORM) {
      if constexpr (VEC) {
        // a head is hd / 8 neighbouring lanes
        f2 s2 = mul2(z[0], z[0]);
#pragma unroll
        for (int k = 1; k < 4; ++k) s2 = fma2(z[k], z[k], s2);
        float ss, s1;
        un2(s2, ss, s1);
        ss += s1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float v = __shfl_xor_sync(0xffffffffu, ss, o);
          ss += 8 * o < a.hd ? v : 0.f;
        }
        const float r = c < a.l2c ? rsqrtf(ss + a.eps) : 1.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = mul2(z[k], mk2(r, r));
      } else {
        // a head is hd lanes of one value, or hd / 32 values of every lane
        float v[8], ss[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) un2(z[k], v[2 * k], v[2 * k + 1]);
#pragma unroll
        for (int k = 0; k < 8; ++k) ss[k] = v[k] * v[k];
        const int g = a.hd >> 5;
#pragma unroll
        for (int s = 1; s < 8; s <<= 1)
          if (g > s) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (!(k & s)) ss[k] = ss[k + s] = ss[k] + ss[k + s];
          }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const float u = __shfl_xor_sync(0xffffffffu, ss[k], o);
            ss[k] += o < a.hd ? u : 0.f;
          }
          v[k] *= chan(k) < a.l2c ? rsqrtf(ss[k] + a.eps) : 1.f;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) z[k] = mk2(v[2 * k], v[2 * k + 1]);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float p, q;
      un2(z[k], p, q);
      out.set(k, p, q);
    }
  }
};

// Where a thread's outputs of token t of a row go.
template <class T, bool VEC>
struct Out {
  T* p;                      // token 0, or null: channels of several ranges
  int64_t st;
  __device__ __forceinline__ void init(const ConvArgs& a, int begin, int row, int c) {
    int part = 0, end = 0;
#pragma unroll
    for (int k = 1; k < CONV_PARTS; ++k) {
      part += c >= a.c0[k];
      end += c + 224 >= a.c0[k];
    }
    st = a.y[part].st;
    p = !VEC && part != end ? nullptr
                            : static_cast<T*>(const_cast<void*>(a.y[part].p)) + (int64_t)begin * st +
                                  (int64_t)row * a.y[part].sn + (c - a.c0[part]);
  }
  __device__ __forceinline__ void put(const ConvArgs& a, const Eight<T, VEC>& v, int begin, int row, int t, int c,
                                      int valid) const {
    if (VEC || p) {
      v.store(p + (int64_t)t * st, valid);
      return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int ch = c + 32 * k;
      if (32 * k >= valid) continue;
      int q = 0;
#pragma unroll
      for (int e = 1; e < CONV_PARTS; ++e) q += ch >= a.c0[e];
      T* o = static_cast<T*>(const_cast<void*>(a.y[q].p)) + (int64_t)(begin + t) * a.y[q].st + (int64_t)row * a.y[q].sn +
             (ch - a.c0[q]);
      if constexpr (sizeof(T) == 4) *o = __uint_as_float(v.w[VEC ? 0 : k]);
      else *reinterpret_cast<uint16_t*>(o) = (uint16_t)v.w[VEC ? 0 : k];
    }
  }
};

template <class T, int W, bool VEC>
__global__ void __launch_bounds__(CONV_THREADS, VEC ? 4 : 3)
conv_kernel(const __grid_constant__ ConvPrompt a) {
  const int tile = blockIdx.x;
  const int row = find_row(a.items, a.rows, tile, a.per_row);
  const RowItem it = a.items[row];
  const int len = row_len(it);
  const int ti = tile - (a.per_row ? row * a.per_row : it.tile0);
  const int t0 = ti * a.TT, t1 = min(len, t0 + a.TT);
  Lane<T, W, VEC> ln;
  ln.init(a);
  const T* x = static_cast<const T*>(a.x.p) + (int64_t)it.begin * a.x.st + (int64_t)row * a.x.sn + ln.c;

  // Tokens come in groups of PF.  Aligned ones take the way through shared memory, two groups ahead, each
  // thread its own 16-byte places (no barrier, and no registers held by loads on their way).  Eight fp32 values
  // are two such pieces: two neighbouring lanes move the pieces of the one, then of the other, so that every
  // access takes whole 32-byte sectors (4 x 512 x 12288: 46 us, 65 with two pieces of its own a lane), and groups are two
  // tokens (89 us with four: registers spill), three groups ahead (five: 47 us).
  constexpr int V16 = sizeof(T) == 4 ? 2 : 1;        // 16-byte pieces of eight values
  constexpr int PF = VEC && V16 == 1 ? 4 : 2, RING = V16 == 1 ? 3 : 4;
  __shared__ __align__(16) uint4 ring[VEC ? RING * PF * V16 : 1][CONV_THREADS];
  const T* ahead = x + (int64_t)t0 * a.x.st;         // the next group to fetch, from token tf on
  int tf = t0, slot = 0;
  const int odd = threadIdx.x & 1;
  Eight<T, VEC> buf[PF];
  auto fetch = [&](int place) {
#pragma unroll
    for (int e = 0; e < PF; ++e) {
      if constexpr (VEC) {
        if constexpr (V16 == 1) {
          if (tf + e < t1 && ln.valid > 0)
            cp_async16(smem_u32(&ring[place * PF + e][threadIdx.x]), ahead + (int64_t)e * a.x.st);
        } else {
#pragma unroll
          for (int v = 0; v < V16; ++v)
            if (tf + e < t1 && ln.valid > 8 * (v - odd))
              cp_async16(smem_u32(&ring[(place * PF + e) * V16 + v][threadIdx.x]),
                         ahead + (int64_t)e * a.x.st + 8 * (v - odd) + 4 * odd);
        }
      } else {
        buf[e].load(ahead + (int64_t)e * a.x.st, tf + e < t1 ? ln.valid : 0);
      }
    }
    if constexpr (VEC) asm volatile("cp.async.commit_group;" ::: "memory");
    ahead += (int64_t)PF * a.x.st;
    tf += PF;
  };
  if constexpr (VEC) {
#pragma unroll
    for (int g = 0; g + 1 < RING; ++g) fetch(g);
  } else {
    fetch(0);
  }

  // the W - 1 inputs before t0
  Eight<T, VEC> hist[W - 1];
  T* st = a.state ? static_cast<T*>(a.state) + (int64_t)it.slot * (W - 1) * a.C + ln.c : nullptr;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    if (t0 > 0) hist[j].load(x + (int64_t)(t0 - (W - 1) + j) * a.x.st, ln.valid);   // TT >= W - 1
    else hist[j].load(st + (int64_t)j * a.C, st && !row_fresh(it) ? ln.valid : 0);
  }
  // Carried inputs after the call: the last W - 1 of (old ones, x).  Only the
  // row's first tile reads and writes them, so no other block can see them change.
  if (ti == 0 && st) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int p = len - (W - 1) + j;
      Eight<T, VEC> v;
      if (p >= 0) {
        v.load(x + (int64_t)p * a.x.st, ln.valid);
      } else {
        v = hist[0];
#pragma unroll
        for (int e = 1; e < W - 1; ++e)
          if (W - 1 + p == e) v = hist[e];
      }
      v.store(st + (int64_t)j * a.C, ln.valid);
    }
  }
  if (t1 <= t0) return;

  f2 win[W - 1][4];
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float p, q;
      hist[j].pair(k, p, q);
      win[j][k] = mk2(p, q);
    }
  Out<T, VEC> out;
  out.init(a, it.begin, row, ln.c);
  Out<T, VEC> first, second;                           // of this pair of lanes
  if constexpr (VEC && V16 == 2) {
    first.init(a, it.begin, row, ln.c - 8 * odd);
    second.init(a, it.begin, row, ln.c + 8 - 8 * odd);
  }

  auto walk = [&](auto act, auto norm) {
#pragma unroll 1
    for (int t = t0; t < t1; t += PF) {
      Eight<T, VEC> cur[PF], y[PF];
      if constexpr (VEC) {
        if constexpr (V16 == 2) __syncwarp();          // the neighbour has read what is overwritten
        fetch(slot == 0 ? RING - 1 : slot - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(RING - 1) : "memory");
        if constexpr (V16 == 2) __syncwarp();          // the neighbour's pieces
#pragma unroll
        for (int e = 0; e < PF; ++e)
#pragma unroll
          for (int v = 0; v < V16; ++v) {
            const uint4 r = V16 == 1 ? ring[slot * PF + e][threadIdx.x]
                                     : ring[(slot * PF + e) * V16 + odd][(threadIdx.x & ~1) + v];
            cur[e].w[4 * v] = r.x;
            cur[e].w[4 * v + 1] = r.y;
            cur[e].w[4 * v + 2] = r.z;
            cur[e].w[4 * v + 3] = r.w;
          }
        slot = slot == RING - 1 ? 0 : slot + 1;
      } else {
#pragma unroll
        for (int e = 0; e < PF; ++e) cur[e] = buf[e];
        fetch(0);
      }
#pragma unroll
      for (int e = 0; e < PF; ++e) ln.template token<act.value, norm.value>(a, cur[e], win, y[e]);
      // tokens past the last were whatever the places held; their window is not used again
#pragma unroll
      for (int e = 0; e < PF; ++e) {
        if constexpr (VEC && V16 == 2) {
          uint32_t other[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) other[k] = __shfl_xor_sync(0xffffffffu, odd ? y[e].w[k] : y[e].w[4 + k], 1);
          if (t + e < t1) {
            // the even lane's values, then the odd lane's; half `odd` of each
            if (ln.valid > -8 * odd)
              *reinterpret_cast<uint4*>(first.p + (int64_t)(t + e) * first.st + 4 * odd) =
                  odd ? make_uint4(other[0], other[1], other[2], other[3])
                      : make_uint4(y[e].w[0], y[e].w[1], y[e].w[2], y[e].w[3]);
            if (ln.valid > 8 - 8 * odd)
              *reinterpret_cast<uint4*>(second.p + (int64_t)(t + e) * second.st + 4 * odd) =
                  odd ? make_uint4(y[e].w[4], y[e].w[5], y[e].w[6], y[e].w[7])
                      : make_uint4(other[0], other[1], other[2], other[3]);
          }
        } else {
          out.put(a, y[e], it.begin, row, t + e, ln.c, t + e < t1 ? ln.valid : 0);
        }
      }
    }
  };
  if (a.act) {
    if (ln.normed) walk(std::true_type{}, std::true_type{});
    else walk(std::true_type{}, std::false_type{});
  } else {
    if (ln.normed) walk(std::false_type{}, std::true_type{});
    else walk(std::false_type{}, std::false_type{});
  }
}

// One token of every row: a block takes TT rows, so that the weights are read
// once for all of them.  Six blocks an SM suit 16-bit vectors; at W = 4 other
// forms keep 160 (fp32 vectors) to 310 bytes a thread in memory.
template <class T, int W, bool VEC>
__global__ void __launch_bounds__(CONV_THREADS, 6)
conv_step_kernel(const __grid_constant__ ConvStep a) {
  Lane<T, W, VEC> ln;
  ln.init(a);
  const int r1 = min(a.rows, (int)(blockIdx.x + 1) * a.TT);
#pragma unroll 2
  for (int row = blockIdx.x * a.TT; row < r1; ++row) {
    const int slot = a.slot[row];
    const bool fresh = slot < 0;
    Eight<T, VEC> cur, hist[W - 1], y;
    T* st = a.state ? static_cast<T*>(a.state) + (int64_t)(fresh ? ~slot : slot) * (W - 1) * a.C + ln.c : nullptr;
    cur.load(static_cast<const T*>(a.x.p) + (int64_t)row * a.x.sn + ln.c, ln.valid);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) hist[j].load(st + (int64_t)j * a.C, st && !fresh ? ln.valid : 0);
    if (st) {
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j) hist[j + 1].store(st + (int64_t)j * a.C, ln.valid);
      cur.store(st + (int64_t)(W - 2) * a.C, ln.valid);
    }
    f2 win[W - 1][4];
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float p, q;
        hist[j].pair(k, p, q);
        win[j][k] = mk2(p, q);
      }
    if (a.act) {
      if (ln.normed) ln.template token<true, true>(a, cur, win, y);
      else ln.template token<true, false>(a, cur, win, y);
    } else {
      if (ln.normed) ln.template token<false, true>(a, cur, win, y);
      else ln.template token<false, false>(a, cur, win, y);
    }
    Out<T, VEC> out;
    out.init(a, 0, row, ln.c);
    out.put(a, y, 0, row, 0, ln.c, ln.valid);
  }
}

template <class T, int W, bool VEC, class Args>
cudaError_t go(const Args& a, cudaStream_t s) {
  const dim3 grid((unsigned)a.tiles, (unsigned)((a.C + 8 * CONV_THREADS - 1) / (8 * CONV_THREADS)));
  if constexpr (std::is_same<Args, ConvStep>::value) conv_step_kernel<T, W, VEC><<<grid, CONV_THREADS, 0, s>>>(a);
  else conv_kernel<T, W, VEC><<<grid, CONV_THREADS, 0, s>>>(a);
  return cudaGetLastError();
}
template <class T, int W, class Args>
cudaError_t go_v(bool vec, const Args& a, cudaStream_t s) {
  return vec ? go<T, W, true>(a, s) : go<T, W, false>(a, s);
}
template <class T, class Args>
cudaError_t go_w(bool vec, const Args& a, cudaStream_t s) {
  return a.W == 2 ? go_v<T, 2>(vec, a, s) : a.W == 3 ? go_v<T, 3>(vec, a, s) : go_v<T, 4>(vec, a, s);
}
template <class Args>
cudaError_t go_t(int dtype, bool vec, const Args& a, cudaStream_t s) {
  return dtype == T_F32    ? go_w<float>(vec, a, s)
         : dtype == T_BF16 ? go_w<__nv_bfloat16>(vec, a, s)
                           : go_w<__half>(vec, a, s);
}

}  // namespace

int conv_tile(int64_t tokens, int C, int sms) {
  // As many tokens (rows, for a step) a tile as still give every SM its four blocks: longer tiles read fewer
  // tokens twice and the weights less often (16 x 512 x 12288: 74 us at 64 tokens, 86 at 16), shorter ones fill
  // the GPU (a step of 256 x 12288: 10 us at 4 rows, 60 at 64).
  const int64_t blocks_c = (C + 8 * CONV_THREADS - 1) / (8 * CONV_THREADS);
  int tt = 64;
  while (tt > 4 && (tokens + tt - 1) / tt * blocks_c < 4 * (int64_t)sms) tt >>= 1;
  return tt;
}

cudaError_t launch_conv(int dtype, bool vec, const ConvPrompt& a, cudaStream_t s) { return go_t(dtype, vec, a, s); }
cudaError_t launch_conv_step(int dtype, bool vec, const ConvStep& a, cudaStream_t s) { return go_t(dtype, vec, a, s); }

}  // namespace mx
}  // namespace dl
