// C entry points of the attention operators: argument checks and the choice of
// a kernel.  Nothing is allocated and nothing kept; what lives on the device
// (slots, lengths, tables) is checked by the kernels.
#include <cmath>
#include <initializer_list>
#include <limits>

#include <cuda_runtime.h>

#include "../../include/deltalog.h"
#include "attn.h"
#include "dl_device.cuh"
#include "host_util.h"

namespace {

using namespace dl::at;
using dl::ErrOut;
using dl::al;
using dl::bad_type;
using dl::done;
using dl::elem;
using dl::num_sms;

constexpr int64_t MAX_DIM = (int64_t)1 << 30;   // sizes that the kernels hold in 32 bits

int shift_of(int64_t page) {
  int s = 0;
  while (((int64_t)1 << s) < page) ++s;
  return s;
}

dl_status page_sizes(const ErrOut& fail, int64_t page, int64_t num_pages) {
  if (page < 16 || page > 256 || (page & (page - 1)))
    return fail(DL_EUNSUPPORTED, "pages of %lld tokens: a power of two from 16 to 256", (long long)page);
  if (num_pages < 1 || num_pages > 0x7fffffff / page)
    return fail(DL_EINVAL, "%lld pages of %lld tokens", (long long)num_pages, (long long)page);
  return DL_OK;
}
dl_status table_sizes(const ErrOut& fail, int64_t n, int64_t page, int64_t num_slots, int64_t max_pages, int64_t stride) {
  if (n < 0 || n > AT_ROWS) return fail(DL_EINVAL, "%lld rows: at most %d a call", (long long)n, AT_ROWS);
  if (num_slots < 1 || num_slots > 0x7fffffff) return fail(DL_EINVAL, "%lld slots", (long long)num_slots);
  if (max_pages < 1 || max_pages > MAX_DIM / page) return fail(DL_EINVAL, "%lld pages a slot", (long long)max_pages);
  if (stride < max_pages && num_slots > 1) return fail(DL_EINVAL, "table rows of %lld entries overlap", (long long)max_pages);
  return DL_OK;
}
bool words(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!al(p, 4)) return false;
  return true;
}

dl_status pages_args(const ErrOut& fail, const dl_pages_args& q, PagesArgs& a) {
  dl_status s = page_sizes(fail, q.page_size, q.num_pages);
  if (s == DL_OK) s = table_sizes(fail, q.n, q.page_size, q.num_slots, q.max_pages, q.table_stride);
  if (s != DL_OK) return s;
  if (q.n > 0 && (!q.slots || !q.table || !q.lengths || !q.free)) return fail(DL_EINVAL, "NULL tensor pointer");
  if (!words({q.slots, q.tokens, q.table, q.lengths, q.free, q.starts, q.where, q.positions, q.work}))
    return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  a = PagesArgs{q.slots, q.tokens, q.table, q.lengths, q.free, q.starts, q.where, q.positions, q.work, q.table_stride,
                q.size, (int32_t)q.n, (int32_t)q.T, (int32_t)q.num_slots, (int32_t)q.max_pages, (int32_t)q.num_pages,
                shift_of(q.page_size)};
  return DL_OK;
}

PoolView pool(const dl_pool& p) { return PoolView{p.data, p.stride_page, p.stride_head, p.stride_token}; }
bool pool_vec(const dl_pool& p, int64_t per) {
  return al(p.data, 16) && p.stride_page % per == 0 && p.stride_head % per == 0 && p.stride_token % per == 0;
}
bool view_vec(const dl_view& v, int64_t per) { return al(v.data, 16) && v.stride_t % per == 0 && v.stride_n % per == 0; }

// Whether two tokens of an output share elements: `w` of them each, token t of row i at t * st + i * sn.  Where the longer
// stride does not span the other dimension, every distance between rows is held against its nearest multiples of st (n
// rows are at most AT_ROWS).
bool tokens_share(int64_t w, int64_t T, int64_t st, int64_t n, int64_t sn) {
  using wide = __int128;
  const wide t = st < 0 ? -(wide)st : st, r = sn < 0 ? -(wide)sn : sn;
  if ((T > 1 && t < w) || (n > 1 && r < w)) return true;
  if (T <= 1 || n <= 1) return false;
  if (t >= r ? t >= (n - 1) * r + w : r >= (T - 1) * t + w) return false;
  for (int64_t i = 1; i < n; ++i) {
    const wide x = i * r, m = x / t;
    if ((m < T && x - m * t < w) || (m + 1 < T && (m + 1) * t - x < w)) return true;
  }
  return false;
}

dl_status head_sizes(const ErrOut& fail, int64_t dtype, int64_t G, int64_t d) {
  if (bad_type(dtype)) return fail(DL_EINVAL, "unknown dtype %lld", (long long)dtype);
  if (G < 1 || G > 4096) return fail(DL_EINVAL, "%lld heads of keys", (long long)G);
  if (d < 1) return fail(DL_EINVAL, "heads of %lld", (long long)d);
  if (d > AT_DIM) return fail(DL_EUNSUPPORTED, "heads of %lld: at most %d is supported", (long long)d, AT_DIM);
  return DL_OK;
}

dl_status attend_sizes(const ErrOut& fail, const dl_attend_args& q) {
  dl_status s = head_sizes(fail, q.dtype, q.G, q.d);
  if (s == DL_OK) s = page_sizes(fail, q.page_size, q.num_pages);
  if (s == DL_OK) s = table_sizes(fail, q.n, q.page_size, q.num_slots, q.max_pages, q.table_stride);
  if (s != DL_OK) return s;
  if (q.H < 1 || q.H > 16384 || q.H % q.G) return fail(DL_EINVAL, "%lld heads over %lld heads of keys", (long long)q.H, (long long)q.G);
  if (q.T < 0 || q.T > MAX_DIM || (!q.packed && q.n * q.T > MAX_DIM)) return fail(DL_EINVAL, "%lld tokens", (long long)q.T);
  if (q.window < 0 || q.sinks < 0 || q.sinks > MAX_DIM)
    return fail(DL_EINVAL, "a window of %lld with %lld first tokens", (long long)q.window, (long long)q.sinks);
  if (!(q.scale > 0) || !std::isfinite((float)(q.scale * 1.4426950408889634)))
    return fail(DL_EINVAL, "the scale must be positive and finite");
  return DL_OK;
}

AttnArgs attn_args(const dl_attend_args& q) {
  AttnArgs a{};
  a.q = q.q.data;
  a.o = q.o.data;
  a.q_st = q.q.stride_t;
  a.q_sn = q.packed ? 0 : q.q.stride_n;
  a.o_st = q.o.stride_t;
  a.o_sn = q.packed ? 0 : q.o.stride_n;
  a.kp = pool(q.k_pages);
  a.vp = pool(q.v_pages);
  a.table = q.table;
  a.lengths = q.lengths;
  a.slots = q.slots;
  a.starts = q.packed ? q.starts : nullptr;
  a.tokens = q.packed ? nullptr : q.tokens;
  a.table_stride = q.table_stride;
  a.n = (int32_t)q.n;
  a.T = (int32_t)q.T;
  a.H = (int32_t)q.H;
  a.G = (int32_t)q.G;
  a.d = (int32_t)q.d;
  a.page_shift = shift_of(q.page_size);
  a.max_pages = (int32_t)q.max_pages;
  a.num_slots = (int32_t)q.num_slots;
  a.num_pages = (int32_t)q.num_pages;
  a.window = (int32_t)(q.window < MAX_DIM ? q.window : MAX_DIM);   // positions are below 2^30: as far as any
  a.sinks = (int32_t)q.sinks;
  // Not zero: the prompts' kernel scales behind the mask, and a masked score of -inf times zero would be a NaN.  The
  // smallest number moves no finite score by more than 2^-21.
  a.scale_log2 = std::fmax((float)(q.scale * 1.4426950408889634), std::numeric_limits<float>::denorm_min());
  a.ws = static_cast<float*>(q.workspace);
  return a;
}

// Which kernel a call runs in, and its workspace.
enum class Kernel { SIMT, SIMT_STEP, STEP, TC };
struct Choice {
  Kernel kernel;
  bool vec;
  AttnPlan plan;
};
Choice choose(const dl_attend_args& q, const AttnArgs& a) {
  Choice c{};
  const int64_t per = 16 / elem(q.dtype);
  c.vec = q.d % 8 == 0 && view_vec(q.q, per) && view_vec(q.o, per) && pool_vec(q.k_pages, per) && pool_vec(q.v_pages, per);
  if (q.T == 1 && !q.packed && !q.tokens) {
    if (step_fits((int)q.dtype, c.vec, a)) {
      c.kernel = Kernel::STEP;
      c.plan = step_plan(a.n, a.H, a.G, a.d, num_sms());
    } else {
      c.kernel = Kernel::SIMT_STEP;
      c.plan = simt_step_plan(a.n, a.H, a.G, a.d, num_sms());
    }
    return c;
  }
  if (tc_fits((int)q.dtype, c.vec, a)) {
    c.kernel = Kernel::TC;
    c.plan = tc_plan(a.n, a.T, q.packed != 0, a.H, a.G, a.d, num_sms());
    return c;
  }
  c.kernel = Kernel::SIMT;
  c.plan = simt_plan(a.n, a.T, q.packed != 0, a.H, a.G, a.d, num_sms());
  return c;
}

dl_status attend(const dl_attend_args* p, void* stream, const ErrOut& fail, bool step) {
  if (!p) return fail(DL_EINVAL, "NULL argument");
  const dl_attend_args& q = *p;
  const dl_status s = attend_sizes(fail, q);
  if (s != DL_OK) return s;
  if (step && (q.T != 1 || q.packed || q.tokens)) return fail(DL_EINVAL, "a step takes one token a row");
  if (q.n == 0 || q.T == 0) return DL_OK;
  if (q.packed && !q.starts) return fail(DL_EINVAL, "packed tokens need starts");
  const int64_t e = elem(q.dtype);
  for (const void* t : {(const void*)q.q.data, (const void*)q.o.data, (const void*)q.k_pages.data, (const void*)q.v_pages.data}) {
    if (!t) return fail(DL_EINVAL, "NULL tensor pointer");
    if (!al(t, e)) return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  }
  if (tokens_share(q.H * q.d, q.T, q.o.stride_t, q.packed ? 1 : q.n, q.packed ? 0 : q.o.stride_n))
    return fail(DL_EINVAL, "out: tokens share elements (strides %lld and %lld)", (long long)q.o.stride_t, (long long)q.o.stride_n);
  if (!q.table || !q.lengths || !q.slots) return fail(DL_EINVAL, "NULL tensor pointer");
  if (!words({q.table, q.lengths, q.slots, q.starts, q.tokens}))
    return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  const AttnArgs a = attn_args(q);
  const Choice c = choose(q, a);
  if (c.plan.ws_bytes && (!q.workspace || q.workspace_bytes < c.plan.ws_bytes || !al(q.workspace, 16)))
    return fail(DL_EINVAL, "the workspace needs %lld bytes, 16-byte aligned (dl_attend_workspace)", (long long)c.plan.ws_bytes);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (c.kernel == Kernel::STEP) return done(fail, launch_step((int)q.dtype, a, c.plan, st));
  if (c.kernel == Kernel::SIMT_STEP) return done(fail, launch_simt_step((int)q.dtype, c.vec, a, c.plan, st));
  if (c.kernel == Kernel::TC) return done(fail, launch_tc((int)q.dtype, a, c.plan, st));
  return done(fail, launch_simt((int)q.dtype, c.vec, a, c.plan, st));
}

}  // namespace

extern "C" dl_status dl_pages_extend(const dl_pages_args* p, void* stream, char* errbuf, int32_t errlen) {
  const ErrOut fail(errbuf, errlen);
  if (!p) return fail(DL_EINVAL, "NULL argument");
  PagesArgs a;
  const dl_status s = pages_args(fail, *p, a);
  if (s != DL_OK) return s;
  if (p->T < 0 || p->T > MAX_DIM || p->size < 0 || p->size > MAX_DIM || (p->T > 0 && p->size != p->T * p->n))
    return fail(DL_EINVAL, "maps of %lld entries for %lld tokens a row", (long long)p->size, (long long)p->T);
  if (!p->starts || !p->work || (p->size > 0 && !p->where)) return fail(DL_EINVAL, "NULL tensor pointer");
  if (p->n == 0) return fail(DL_EINVAL, "no rows");
  return done(fail, launch_extend(a, num_sms(), static_cast<cudaStream_t>(stream)));
}

extern "C" dl_status dl_pages_truncate(const dl_pages_args* p, void* stream, char* errbuf, int32_t errlen) {
  const ErrOut fail(errbuf, errlen);
  if (!p) return fail(DL_EINVAL, "NULL argument");
  PagesArgs a;
  const dl_status s = pages_args(fail, *p, a);
  if (s != DL_OK || p->n == 0) return s;
  return done(fail, launch_truncate(a, static_cast<cudaStream_t>(stream)));
}

extern "C" dl_status dl_kv_append(const dl_kv_append_args* p, void* stream, char* errbuf, int32_t errlen) {
  const ErrOut fail(errbuf, errlen);
  if (!p) return fail(DL_EINVAL, "NULL argument");
  const dl_kv_append_args& q = *p;
  dl_status s = head_sizes(fail, q.dtype, q.G, q.d);
  if (s == DL_OK) s = page_sizes(fail, q.page_size, q.num_pages);
  if (s != DL_OK) return s;
  if (q.n < 0 || q.T < 0 || q.n > MAX_DIM || q.T > MAX_DIM || q.n * q.T > MAX_DIM)
    return fail(DL_EINVAL, "%lld tokens of %lld rows", (long long)q.T, (long long)q.n);
  if (q.n == 0 || q.T == 0) return DL_OK;
  const int64_t e = elem(q.dtype), per = 16 / e;
  for (const void* t : {(const void*)q.k.data, (const void*)q.v.data, (const void*)q.k_pages.data, (const void*)q.v_pages.data}) {
    if (!t) return fail(DL_EINVAL, "NULL tensor pointer");
    if (!al(t, e)) return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  }
  if (!q.where) return fail(DL_EINVAL, "NULL tensor pointer");
  if (!al(q.where, 4)) return fail(DL_EINVAL, "misaligned tensor: every tensor needs its element's alignment");
  const bool vec = q.d % per == 0 && view_vec(q.k, per) && view_vec(q.v, per) && pool_vec(q.k_pages, per) && pool_vec(q.v_pages, per);
  const AppendArgs a{q.k.data, q.v.data, q.k.stride_t, q.k.stride_n, q.v.stride_t, q.v.stride_n, pool(q.k_pages),
                     pool(q.v_pages), q.where, q.T, (int32_t)q.n, (int32_t)q.G, (int32_t)q.d, shift_of(q.page_size),
                     (int32_t)q.num_pages};
  return done(fail, launch_append((int)e, vec, a, static_cast<cudaStream_t>(stream)));
}

extern "C" int64_t dl_attend_workspace(const dl_attend_args* p) {
  const ErrOut quiet(nullptr, 0);
  if (!p || attend_sizes(quiet, *p) != DL_OK) return -1;
  if (p->n == 0 || p->T == 0) return 0;
  return choose(*p, attn_args(*p)).plan.ws_bytes;
}

extern "C" dl_status dl_attend(const dl_attend_args* p, void* stream, char* errbuf, int32_t errlen) {
  return attend(p, stream, ErrOut(errbuf, errlen), false);
}

extern "C" dl_status dl_attend_step(const dl_attend_args* p, void* stream, char* errbuf, int32_t errlen) {
  return attend(p, stream, ErrOut(errbuf, errlen), true);
}

extern "C" dl_status dl_attend_sync(void* stream, int32_t* device_code, char* errbuf, int32_t errlen) {
  const ErrOut fail(errbuf, errlen);
  int32_t code = 0;
  cudaError_t e = cudaSuccess;
  for (const auto read : {read_pages_status, read_simt_status, read_simt_step_status, read_step_status, read_tc_status}) {
    int32_t c = 0;
    e = read(static_cast<cudaStream_t>(stream), &c);
    if (e != cudaSuccess) break;
    code = code ? code : c;
  }
  if (device_code) *device_code = code;
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(DL_ECUDA, "status read failed: %s", cudaGetErrorString(e));
  }
  return code ? fail(DL_EDEVICE, "kernel reported device status %d (%s)", code, dl::device_status_str(code)) : DL_OK;
}
