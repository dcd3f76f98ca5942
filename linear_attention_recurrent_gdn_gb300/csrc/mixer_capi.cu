// C entry points of the mixer operators: argument checks, tile planning and
// launches.  Everything is checked before the first CUDA call; nothing is
// allocated and nothing kept.  A call's rows and the launch arguments are built
// in a thread's own storage; calls of many rows take several launches.
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include <cuda_runtime.h>

#include "../../include/deltalog.h"
#include "dl_device.cuh"
#include "mixer.h"

namespace {

using namespace dl::mx;

struct ErrOut {
  char* buf;
  int32_t len;
  dl_status operator()(dl_status s, const char* fmt, ...) const {
    if (buf && len > 0) {
      va_list ap;
      va_start(ap, fmt);
      vsnprintf(buf, (size_t)len, fmt, ap);
      va_end(ap);
    }
    return s;
  }
};

// Every row of a call, and the arguments of a launch.
thread_local RowItem t_items[MX_ROWS];
thread_local ConvPrompt t_conv;
thread_local ConvStep t_conv_step;
thread_local SsmArgs t_ssm;
thread_local SsmStep t_ssm_step;

constexpr int64_t MAX_DIM = (int64_t)1 << 30;   // sizes that the kernels hold in 32 bits

int64_t elem(int64_t dtype) { return dtype == DL_F32 ? 4 : 2; }
bool al(const void* p, int64_t b) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(b - 1)) == 0; }

// Every launch: CUDA's sticky state is left clean for the caller's next call.
dl_status done(const ErrOut& fail, cudaError_t e) {
  if (e == cudaSuccess) return DL_OK;
  (void)cudaGetLastError();
  return fail(DL_ECUDA, "launch failed: %s", cudaGetErrorString(e));
}

// Distinct ids in [0, num_slots): an open-addressing table on the stack.
dl_status check_slots(const ErrOut& fail, const int32_t* slots, int64_t n, int64_t num_slots) {
  constexpr uint32_t SIZE = 4096;
  int32_t seen[SIZE];
  uint32_t mask = 15;
  while (mask + 1 < 4 * (uint32_t)n) mask = 2 * mask + 1;
  memset(seen, 0xff, (size_t)(mask + 1) * 4);
  for (int64_t i = 0; i < n; ++i) {
    const int32_t s = slots[i];
    if (s < 0 || s >= num_slots)
      return fail(DL_EINVAL, "slot %d of row %lld is not in [0, %lld)", s, (long long)i, (long long)num_slots);
    uint32_t k = ((uint32_t)s * 2654435761u >> 12) & mask;
    while (seen[k] != -1) {
      if (seen[k] == s) return fail(DL_EINVAL, "slot %d appears twice", s);
      k = (k + 1) & mask;
    }
    seen[k] = s;
  }
  return DL_OK;
}

// The rows' plan.  tt: tokens of a tile (every row has at least one tile, for
// its state); returns the number of tiles, in per_row the tiles of every row
// when all rows have the same number (else 0), and whether there is any token.
dl_status plan_rows(const ErrOut& fail, const dl_tokens& k, bool state, int64_t tt, RowItem* items,
                    int64_t& tiles, int32_t& per_row, bool& any) {
  if (k.n < 0 || k.n > MX_ROWS) return fail(DL_EINVAL, "%lld rows: at most %d a call", (long long)k.n, MX_ROWS);
  if (k.T < 0 || k.T > MAX_DIM) return fail(DL_EINVAL, "%lld tokens a row", (long long)k.T);
  if (k.packed && !k.lengths && k.n > 0) return fail(DL_EINVAL, "packed tokens need lengths");
  if (state) {
    if (!k.slots && k.n > 0) return fail(DL_EINVAL, "a state pool needs slots");
    if (k.num_slots < 1 || k.num_slots > 0x7fffffff) return fail(DL_EINVAL, "%lld slots", (long long)k.num_slots);
    const dl_status s = check_slots(fail, k.slots, k.n, k.num_slots);
    if (s != DL_OK) return s;
  }
  int64_t begin = 0;
  tiles = 0;
  any = false;
  bool same = true;
  for (int64_t i = 0; i < k.n; ++i) {
    const int64_t len = k.lengths ? k.lengths[i] : k.T;
    if (len < 0 || len > k.T) return fail(DL_EINVAL, "row %lld has %lld tokens, T is %lld", (long long)i, (long long)len, (long long)k.T);
    const bool fresh = k.fresh ? k.fresh[i] != 0 : k.fresh_all != 0;
    items[i] = RowItem{state ? k.slots[i] : 0, (int32_t)begin, (int32_t)len | (fresh || !state ? FRESH_BIT : 0),
                       (int32_t)tiles};
    const int64_t nt = len > tt ? (len + tt - 1) / tt : 1;
    if (i == 0) per_row = (int32_t)nt;
    same = same && nt == per_row;
    any = any || len > 0;
    tiles += nt;
    if (k.packed) begin += len;
    if (tiles > MAX_DIM || begin > MAX_DIM) return fail(DL_EINVAL, "too many tokens in one call");
  }
  if (!same) per_row = 0;
  return DL_OK;
}

// Rows [r0, r0 + n) of a call as a launch's own: tiles numbered from zero.
void group_rows(const RowItem* all, int64_t r0, int64_t n, RowItem* items) {
  for (int64_t i = 0; i < n; ++i) {
    items[i] = all[r0 + i];
    items[i].tile0 -= all[r0].tile0;
  }
}
void group_slots(const RowItem* all, int64_t r0, int64_t n, int32_t* slot) {
  for (int64_t i = 0; i < n; ++i) slot[i] = row_fresh(all[r0 + i]) ? ~all[r0 + i].slot : all[r0 + i].slot;
}
// A tensor as rows from r0 on see it.
TokView from_row(const TokView& v, int64_t r0, int64_t elem) {
  return TokView{static_cast<const char*>(v.p) + (v.p ? r0 * v.sn * elem : 0), v.st, v.sn};
}

TokView view(const dl_view& v, bool packed) { return TokView{v.data, v.stride_t, packed ? 0 : v.stride_n}; }

bool view_vec(const dl_view& v, int64_t dtype, bool packed) {
  const int64_t per = 16 / elem(dtype);
  return al(v.data, 16) && v.stride_t % per == 0 && (packed || v.stride_n % per == 0);
}

// Multiprocessors of the current device (a GB300's where there is none to ask).
int num_sms() {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    (void)cudaGetLastError();
    return 152;
  }
  n = known[dev].load(std::memory_order_relaxed);
  if (n) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    return 152;
  }
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

bool bad_type(int64_t t) { return t < DL_F32 || t > DL_F16; }

}  // namespace

extern "C" dl_status dl_conv(const dl_conv_args* p, void* stream, char* errbuf, int32_t errlen) {
  const ErrOut fail{errbuf, errlen};
  if (errbuf && errlen > 0) errbuf[0] = 0;
  if (!p) return fail(DL_EINVAL, "NULL argument");
  const dl_conv_args& q = *p;
  const bool packed = q.tokens.packed != 0;
  if (bad_type(q.dtype)) return fail(DL_EINVAL, "unknown dtype %lld", (long long)q.dtype);
  if (q.C < 1 || q.C > MAX_DIM) return fail(DL_EINVAL, "%lld channels", (long long)q.C);
  if (q.W < 2 || q.W > 4) return fail(DL_EUNSUPPORTED, "width %lld: 2 to 4 are supported", (long long)q.W);
  if (q.act != DL_ACT_NONE && q.act != DL_ACT_SILU) return fail(DL_EINVAL, "activation %lld: none or silu", (long long)q.act);
  if (q.n_parts < 1 || q.n_parts > CONV_PARTS) return fail(DL_EINVAL, "%lld output ranges: 1 to 4", (long long)q.n_parts);
  if (q.l2_channels < 0 || q.l2_channels > q.C) return fail(DL_EINVAL, "%lld normalised channels of %lld", (long long)q.l2_channels, (long long)q.C);
  if (q.l2_channels) {
    const int64_t d = q.head_dim;
    if (d < 8 || d > 256 || (d & (d - 1))) return fail(DL_EUNSUPPORTED, "head_dim %lld: a power of two from 8 to 256", (long long)d);
    if (q.l2_channels % d) return fail(DL_EINVAL, "%lld normalised channels are not whole heads of %lld", (long long)q.l2_channels, (long long)d);
    if (!(q.eps >= 0)) return fail(DL_EINVAL, "eps is negative");
  }
  ConvArgs a{};
  int64_t c = 0;
  bool vec = q.C % 8 == 0;
  for (int k = 0; k < CONV_PARTS; ++k) {
    a.c0[k] = (int32_t)c;
    a.y[k] = TokView{nullptr, 0, 0};
    if (k >= q.n_parts) continue;
    const int64_t ch = q.part_channels[k];
    if (ch < 1 || c + ch > q.C) return fail(DL_EINVAL, "output ranges do not add up to %lld channels", (long long)q.C);
    a.y[k] = view(q.y[k], packed);
    vec = vec && ch % 8 == 0 && view_vec(q.y[k], q.dtype, packed);
    c += ch;
  }
  if (c != q.C) return fail(DL_EINVAL, "output ranges do not add up to %lld channels", (long long)q.C);
  a.c0[CONV_PARTS] = (int32_t)q.C;
  for (int k = (int)q.n_parts; k < CONV_PARTS; ++k) a.c0[k] = (int32_t)q.C;
  const bool step = q.tokens.T == 1 && !q.tokens.lengths && !packed;
  int64_t total = q.tokens.n > 0 ? q.tokens.n * q.tokens.T : 0;
  if (q.tokens.lengths) {
    total = 0;
    for (int64_t i = 0; i < q.tokens.n && i < MX_ROWS; ++i) total += q.tokens.lengths[i];
  }
  a.TT = conv_tile(total, (int)q.C, num_sms());
  int64_t tiles;
  bool any;
  const dl_status s = plan_rows(fail, q.tokens, q.state != nullptr, a.TT, t_items, tiles, a.per_row, any);
  if (s != DL_OK) return s;
  if (q.tokens.n == 0) return DL_OK;
  const int64_t e = elem(q.dtype);
  if ((!q.x.data && any) || !q.weight) return fail(DL_EINVAL, "NULL tensor pointer");
  const int64_t we = q.weight_f32 ? 4 : e;
  bool ok = al(q.x.data, e) && al(q.weight, we) && al(q.bias, we) && al(q.state, e);
  for (int k = 0; k < q.n_parts; ++k) {
    if (!q.y[k].data && any) return fail(DL_EINVAL, "NULL tensor pointer");
    ok = ok && al(q.y[k].data, e);
  }
  if (!ok) return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  vec = vec && view_vec(q.x, q.dtype, packed) && al(q.state, 16);
  a.x = view(q.x, packed);
  a.w = q.weight;
  a.b = q.bias;
  a.state = q.state;
  a.C = (int32_t)q.C;
  a.W = (int32_t)q.W;
  a.act = (int32_t)q.act;
  a.l2c = (int32_t)q.l2_channels;
  a.hd = (int32_t)q.head_dim;
  a.w_f32 = q.weight_f32 ? 1 : 0;
  a.eps = (float)q.eps;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t n = q.tokens.n, most = step ? MX_STEP : MX_GROUP;
  for (int64_t r0 = 0; r0 < n; r0 += most) {
    const int64_t m = n - r0 < most ? n - r0 : most;
    ConvArgs& g = step ? static_cast<ConvArgs&>(t_conv_step) : t_conv;
    g = a;
    g.rows = (int32_t)m;
    g.x = from_row(a.x, r0, e);
    for (int k = 0; k < q.n_parts; ++k) g.y[k] = from_row(a.y[k], r0, e);
    cudaError_t err;
    if (step) {
      g.tiles = (int32_t)((m + a.TT - 1) / a.TT);
      group_slots(t_items, r0, m, t_conv_step.slot);
      err = launch_conv_step((int)q.dtype, vec, t_conv_step, st);
    } else {
      g.tiles = (int32_t)((r0 + m < n ? t_items[r0 + m].tile0 : tiles) - t_items[r0].tile0);
      group_rows(t_items, r0, m, t_conv.items);
      err = launch_conv((int)q.dtype, vec, t_conv, st);
    }
    if (err != cudaSuccess) return done(fail, err);
  }
  return DL_OK;
}

namespace {

dl_status ssm_sizes(const ErrOut& fail, const dl_ssm_args& q) {
  if (bad_type(q.dtype)) return fail(DL_EINVAL, "unknown dtype %lld", (long long)q.dtype);
  if (q.H < 1 || q.H > 65536 || q.G < 1 || q.H % q.G)
    return fail(DL_EINVAL, "%lld heads in %lld groups", (long long)q.H, (long long)q.G);
  if (q.P < 1 || q.P > 65536 || q.N < 1) return fail(DL_EINVAL, "state of %lld x %lld", (long long)q.P, (long long)q.N);
  if (q.N > 256) return fail(DL_EUNSUPPORTED, "N = %lld: at most 256 is supported", (long long)q.N);
  return DL_OK;
}

dl_status ssm_args(const ErrOut& fail, const dl_ssm_args& q, SsmBase& a) {
  dl_status s = ssm_sizes(fail, q);
  if (s != DL_OK) return s;
  int64_t tiles;
  int32_t per_row;
  bool any;
  const bool packed = q.tokens.packed != 0;
  s = plan_rows(fail, q.tokens, q.state != nullptr, MAX_DIM, t_items, tiles, per_row, any);
  if (s != DL_OK || q.tokens.n == 0) return s;
  const int64_t e = elem(q.dtype);
  for (const dl_view* v : {&q.x, &q.B, &q.C, &q.y}) {
    if (!v->data && any) return fail(DL_EINVAL, "NULL tensor pointer");
    if (!al(v->data, e)) return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  }
  if ((!q.dt.data && any) || !q.A) return fail(DL_EINVAL, "NULL tensor pointer");
  if (!al(q.dt.data, q.dt_f32 ? 4 : e) || !al(q.A, 4) || !al(q.D, 4) || !al(q.dt_bias, 4) || !al(q.state, 4))
    return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  a.x = view(q.x, packed);
  a.dt = view(q.dt, packed);
  a.B = view(q.B, packed);
  a.C = view(q.C, packed);
  a.y = view(q.y, packed);
  a.A = q.A;
  a.D = q.D;
  a.dt_bias = q.dt_bias;
  a.state = q.state;
  a.H = (int32_t)q.H;
  a.G = (int32_t)q.G;
  a.P = (int32_t)q.P;
  a.N = (int32_t)q.N;
  a.softplus = q.softplus ? 1 : 0;
  a.dt_f32 = q.dt_f32 ? 1 : 0;
  a.rows = (int32_t)q.tokens.n;
  if ((int64_t)a.rows * q.H * q.P > (int64_t)1 << 31) return fail(DL_EINVAL, "too many state rows in one call");
  return DL_OK;
}

}  // namespace

namespace {

// The tensor cores take bf16 rows of at least TC_TOKENS tokens (the longest
// row's): below that the chunk of 128 is mostly padding.  Heads of 64 x 128 at
// 32 tokens: 16 rows of 32 heads 23 us, 28 on the FP32 cores; one row of 8
// heads 10 us, 13 there; both grow with the tokens there and not here.
constexpr int64_t TC_TOKENS = 32;

bool on_tensor_cores(const dl_ssm_args& q) {
  int64_t longest = q.tokens.lengths ? 0 : q.tokens.T;
  if (q.tokens.lengths)
    for (int64_t i = 0; i < q.tokens.n; ++i) longest = q.tokens.lengths[i] > longest ? q.tokens.lengths[i] : longest;
  return q.dtype == DL_BF16 && q.N <= 128 && longest >= TC_TOKENS;
}

SsmPlan plan_of(const dl_ssm_args& q) {
  const int H = (int)q.H, P = (int)q.P, N = (int)q.N, n = (int)q.tokens.n;
  return on_tensor_cores(q) ? ssm_tc_plan(H, P, n, q.tokens.lengths, q.tokens.T, num_sms())
                            : ssm_scan_plan(H, P, N, n, q.tokens.lengths, q.tokens.T, num_sms());
}

int64_t workspace_of(const dl_ssm_args& q, const SsmPlan& p, int64_t tiles) {
  return p.split ? 4 * tiles * q.H * (q.P * q.N + 1) : 0;
}

}  // namespace

extern "C" int64_t dl_ssm_workspace(const dl_ssm_args* p) {
  const ErrOut quiet{nullptr, 0};
  if (!p || ssm_sizes(quiet, *p) != DL_OK || p->tokens.n < 0 || p->tokens.n > MX_ROWS) return -1;
  if (p->tokens.n == 0) return 0;
  const SsmPlan k = plan_of(*p);
  if (!k.split) return 0;
  int64_t tiles = 0;
  for (int64_t i = 0; i < p->tokens.n; ++i) {
    const int64_t len = p->tokens.lengths ? p->tokens.lengths[i] : p->tokens.T;
    tiles += len > k.seg_tokens ? (len + k.seg_tokens - 1) / k.seg_tokens : 1;
  }
  return workspace_of(*p, k, tiles);
}

extern "C" dl_status dl_ssm(const dl_ssm_args* p, void* stream, char* errbuf, int32_t errlen) {
  const ErrOut fail{errbuf, errlen};
  if (errbuf && errlen > 0) errbuf[0] = 0;
  if (!p) return fail(DL_EINVAL, "NULL argument");
  const dl_ssm_args& q = *p;
  SsmBase a{};
  dl_status s = ssm_args(fail, q, a);
  if (s != DL_OK || q.tokens.n == 0) return s;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const SsmPlan k = plan_of(q);
  int64_t tiles;
  int32_t per_row;
  bool any;
  s = plan_rows(fail, q.tokens, q.state != nullptr, k.seg_tokens, t_items, tiles, per_row, any);
  if (s != DL_OK) return s;
  const int64_t need = workspace_of(q, k, tiles);
  if (need && (!q.workspace || q.workspace_bytes < need || !al(q.workspace, 16)))
    return fail(DL_EINVAL, "the workspace needs %lld bytes, 16-byte aligned (dl_ssm_workspace)", (long long)need);
  if (tiles * k.units > 0x7fffffff) return fail(DL_EINVAL, "too many tokens in one call");
  const bool packed = q.tokens.packed != 0;
  const bool vec = q.P % 8 == 0 && q.N % 8 == 0 && view_vec(q.x, q.dtype, packed) && view_vec(q.B, q.dtype, packed) &&
                   view_vec(q.C, q.dtype, packed) && view_vec(q.y, q.dtype, packed);
  int64_t tokens = q.tokens.T;
  if (packed) tokens = (int64_t)t_items[q.tokens.n - 1].begin + row_len(t_items[q.tokens.n - 1]);
  const bool tc = on_tensor_cores(q);
  const int64_t n = q.tokens.n, e = elem(q.dtype);
  float* ws = static_cast<float*>(q.workspace);
  for (int64_t r0 = 0; r0 < n; r0 += MX_GROUP) {
    const int64_t m = n - r0 < MX_GROUP ? n - r0 : MX_GROUP;
    SsmArgs& g = t_ssm;
    static_cast<SsmBase&>(g) = a;
    g.rows = (int32_t)m;
    g.x = from_row(a.x, r0, e);
    g.B = from_row(a.B, r0, e);
    g.C = from_row(a.C, r0, e);
    g.y = from_row(a.y, r0, e);
    g.dt = from_row(a.dt, r0, q.dt_f32 ? 4 : e);
    group_rows(t_items, r0, m, g.items);
    const int gt = (int)((r0 + m < n ? t_items[r0 + m].tile0 : tiles) - t_items[r0].tile0);
    const cudaError_t err = tc ? launch_ssm_tc(vec, tokens, g, k, gt, per_row, ws, st)
                               : launch_ssm_scan((int)q.dtype, vec, g, k, gt, per_row, ws, st);
    if (err != cudaSuccess) return done(fail, err);
  }
  return DL_OK;
}

extern "C" dl_status dl_mixer_sync(void* stream, int32_t* device_code, char* errbuf, int32_t errlen) {
  const ErrOut fail{errbuf, errlen};
  if (errbuf && errlen > 0) errbuf[0] = 0;
  int32_t code = 0;
  const cudaError_t e = read_mixer_status(static_cast<cudaStream_t>(stream), &code);
  if (device_code) *device_code = code;
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(DL_ECUDA, "status read failed: %s", cudaGetErrorString(e));
  }
  return code ? fail(DL_EDEVICE, "kernel reported device status %d (%s)", code, dl::device_status_str(code)) : DL_OK;
}

extern "C" dl_status dl_ssm_step(const dl_ssm_args* p, void* stream, char* errbuf, int32_t errlen) {
  const ErrOut fail{errbuf, errlen};
  if (errbuf && errlen > 0) errbuf[0] = 0;
  if (!p) return fail(DL_EINVAL, "NULL argument");
  if (!p->state) return fail(DL_EINVAL, "a step needs a state pool");
  if (p->tokens.T != 1 || p->tokens.lengths) return fail(DL_EINVAL, "a step takes one token a row");
  SsmBase a{};
  const dl_status s = ssm_args(fail, *p, a);
  if (s != DL_OK || p->tokens.n == 0) return s;
  const int64_t n = p->tokens.n, e = elem(p->dtype);
  for (int64_t r0 = 0; r0 < n; r0 += MX_STEP) {
    const int64_t m = n - r0 < MX_STEP ? n - r0 : MX_STEP;
    SsmStep& g = t_ssm_step;
    static_cast<SsmBase&>(g) = a;
    g.rows = (int32_t)m;
    g.x = from_row(a.x, r0, e);
    g.B = from_row(a.B, r0, e);
    g.C = from_row(a.C, r0, e);
    g.y = from_row(a.y, r0, e);
    g.dt = from_row(a.dt, r0, p->dt_f32 ? 4 : e);
    group_slots(t_items, r0, m, g.slot);
    const cudaError_t err = launch_ssm_step((int)p->dtype, g, static_cast<cudaStream_t>(stream));
    if (err != cudaSuccess) return done(fail, err);
  }
  return DL_OK;
}

extern "C" dl_status dl_gated_norm(const dl_gated_norm_args* p, void* stream, char* errbuf, int32_t errlen) {
  const ErrOut fail{errbuf, errlen};
  if (errbuf && errlen > 0) errbuf[0] = 0;
  if (!p) return fail(DL_EINVAL, "NULL argument");
  const dl_gated_norm_args& q = *p;
  if (bad_type(q.dtype)) return fail(DL_EINVAL, "unknown dtype %lld", (long long)q.dtype);
  if (q.kind != DL_NORM_RMS && q.kind != DL_NORM_LAYER) return fail(DL_EINVAL, "unknown norm %lld", (long long)q.kind);
  if (q.act < DL_ACT_NONE || q.act > DL_ACT_SIGMOID) return fail(DL_EINVAL, "unknown activation %lld", (long long)q.act);
  if (q.rows < 0 || q.H < 1 || q.d < 1 || q.rows > MAX_DIM || q.H > MAX_DIM || q.rows * q.H > MAX_DIM)
    return fail(DL_EINVAL, "%lld rows of %lld heads of %lld", (long long)q.rows, (long long)q.H, (long long)q.d);
  if (q.d > 16384) return fail(DL_EUNSUPPORTED, "heads of %lld: at most 16384 is supported", (long long)q.d);
  if (!(q.eps >= 0)) return fail(DL_EINVAL, "eps is negative");
  if (q.rows == 0) return DL_OK;
  if (!q.x || !q.y || !q.weight) return fail(DL_EINVAL, "NULL tensor pointer");
  const int64_t e = elem(q.dtype), we = q.weight_f32 ? 4 : e, per = 16 / e;
  if (!al(q.x, e) || !al(q.gate, e) || !al(q.y, e) || !al(q.weight, we) || !al(q.bias, we))
    return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  const bool vec = q.d % 8 == 0 && al(q.x, 16) && al(q.gate, 16) && al(q.y, 16) && al(q.weight, 16) && al(q.bias, 16) &&
                   q.x_stride % per == 0 && q.y_stride % per == 0 && (!q.gate || q.gate_stride % per == 0);
  const GatedNormArgs a{q.x, q.gate, q.weight, q.bias, q.y, q.x_stride, q.gate_stride, q.y_stride, q.rows,
                        (int32_t)q.H, (int32_t)q.d, (int32_t)q.kind, (int32_t)q.act, q.gate_first ? 1 : 0,
                        q.weight_f32 ? 1 : 0, q.weight_heads ? 1 : 0, (float)q.eps};
  return done(fail, launch_gated_norm((int)q.dtype, vec, a, static_cast<cudaStream_t>(stream)));
}

extern "C" dl_status dl_add_norm(const dl_add_norm_args* p, void* stream, char* errbuf, int32_t errlen) {
  const ErrOut fail{errbuf, errlen};
  if (errbuf && errlen > 0) errbuf[0] = 0;
  if (!p) return fail(DL_EINVAL, "NULL argument");
  const dl_add_norm_args& q = *p;
  if (bad_type(q.dtype)) return fail(DL_EINVAL, "unknown dtype %lld", (long long)q.dtype);
  if (q.kind != DL_NORM_RMS && q.kind != DL_NORM_LAYER) return fail(DL_EINVAL, "unknown norm %lld", (long long)q.kind);
  if (q.rows < 0 || q.rows > MAX_DIM || q.D < 1) return fail(DL_EINVAL, "%lld rows of %lld", (long long)q.rows, (long long)q.D);
  if (q.D > 16384) return fail(DL_EUNSUPPORTED, "rows of %lld: at most 16384 is supported", (long long)q.D);
  if (!(q.eps >= 0)) return fail(DL_EINVAL, "eps is negative");
  if (q.rows == 0) return DL_OK;
  if (!q.x || !q.y || !q.weight) return fail(DL_EINVAL, "NULL tensor pointer");
  const bool r32 = q.residual_f32 || q.dtype == DL_F32;
  const int64_t e = elem(q.dtype), re = r32 ? 4 : 2, we = q.weight_f32 ? 4 : e, per = 16 / e, rper = 16 / re;
  if (!al(q.x, e) || !al(q.y, e) || !al(q.residual, re) || !al(q.h, re) || !al(q.weight, we) || !al(q.bias, we) ||
      !al(q.scale, we) || !al(q.post, we))
    return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  bool vec = q.D % 8 == 0 && q.x_stride % per == 0 && q.y_stride % per == 0 &&
             (!q.residual || q.residual_stride % rper == 0) && (!q.h || q.h_stride % rper == 0);
  for (const void* t : {q.x, q.residual, q.weight, q.bias, q.scale, q.post, (const void*)q.y, (const void*)q.h})
    vec = vec && al(t, 16);
  const AddNormArgs a{q.x, q.residual, q.weight, q.bias, q.scale, q.post, q.y, q.h, q.x_stride, q.residual_stride,
                      q.y_stride, q.h_stride, q.rows, (int32_t)q.D, (int32_t)q.kind, q.weight_f32 ? 1 : 0,
                      (float)q.eps, (float)q.alpha};
  return done(fail, launch_add_norm((int)q.dtype, r32, vec, a, static_cast<cudaStream_t>(stream)));
}
