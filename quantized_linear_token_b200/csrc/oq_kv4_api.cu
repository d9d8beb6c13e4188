// C-ABI entry points of the operators around attention (declared in
// include/orbitquant.h): argument checks, the handle and dispatch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>
#include <string>

#include "oq_kv4.cuh"

namespace oq {
namespace {

oq_status fail(oq_status st, const std::string& msg) {
  set_error(msg);
  return st;
}
oq_status invalid(const char* who, const char* what) { return fail(OQ_ERR_INVALID_ARG, std::string(who) + ": " + what); }
oq_status unsupported(const char* who, const char* what) {
  return fail(OQ_ERR_UNSUPPORTED, std::string(who) + ": " + what);
}
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
constexpr int64_t MOST_BYTES = (int64_t)1 << 60;   // of an array: sums and products of addresses stay within 64 bits
size_t size_of(int32_t dtype) { return dtype == OQ_DTYPE_F32 ? 4 : 2; }
bool known(int32_t dtype) { return dtype == OQ_DTYPE_F32 || dtype == OQ_DTYPE_BF16; }

// Rows of bytes at equal distances; one row where an array is contiguous (its stride is its length).
struct Rows {
  const void* p;
  size_t row, stride;
  int64_t n;
  size_t extent() const { return n > 0 ? (size_t)(n - 1) * stride + row : 0; }
};
Rows flat(const void* p, size_t bytes) { return {p, bytes, bytes, 1}; }
Rows heads_of(const void* p, int64_t T, int32_t heads, int32_t D, int64_t stride, int32_t dtype) {
  const size_t e = size_of(dtype);
  return {p, (size_t)heads * D * e, T > 1 ? (size_t)stride * e : (size_t)heads * D * e, T};   // (one token: any stride)
}
// whether they share a byte; rows with equal strides may lie in each other's gaps
bool overlap(const Rows& a, const Rows& b) {
  if (!a.p || !b.p || !a.extent() || !b.extent()) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (x >= y + b.extent() || y >= x + a.extent()) return false;
  if (a.stride != b.stride) return true;
  const size_t d = y >= x ? (y - x) % a.stride : (a.stride - (x - y) % a.stride) % a.stride;
  return d < a.row || d + b.row > a.stride;
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.row == b.row && a.stride == b.stride; }

struct QkIn {
  const char* who;
  int64_t T;
  int32_t D, dtype, gain_dtype, rot, flags;
  float eps;
  const void *q_gain, *k_gain, *table, *positions;
  int64_t table_rows;
};

// what norm and rotation need, for rows of D channels
oq_status check_qk(const QkIn& a) {
  if (a.T < 0) return invalid(a.who, "T must not be negative");
  if (!known(a.dtype) || !known(a.gain_dtype)) return invalid(a.who, "dtype must be OQ_DTYPE_F32 or OQ_DTYPE_BF16");
  if (a.flags & ~(OQ_QK_INTERLEAVED | OQ_QK_NO_NORM)) return invalid(a.who, "unknown flags");
  if (!(a.eps >= 0.f) || std::isinf(a.eps)) return invalid(a.who, "eps must be finite and not negative");
  if ((a.flags & OQ_QK_NO_NORM) && (a.q_gain || a.k_gain)) return invalid(a.who, "gains without a norm");
  if (!aligned(a.q_gain, 16) || !aligned(a.k_gain, 16) || !aligned(a.table, 16) || !aligned(a.positions, 4))
    return invalid(a.who, "gains and table must be 16-byte aligned, positions 4-byte");
  if (a.table) {
    if (a.table_rows < 1) return invalid(a.who, "the table must have a row");
    if (a.table_rows > MOST_BYTES / 4 / std::max(a.rot, 1)) return unsupported(a.who, "the table is too large");
    if (a.rot <= 0 || a.rot > a.D || a.rot % (a.flags & OQ_QK_INTERLEAVED ? 8 : 16))
      return unsupported(a.who, "rotated channels must be a multiple of 8 (interleaved) or 16, up to the head's");
  }
  if (a.T > 0x7FFFFFFF) return unsupported(a.who, "at most 2^31 - 1 tokens per call");
  return OQ_OK;
}
oq_status check_heads(const char* who, const char* name, const void* p, int32_t heads, int32_t D, int64_t stride,
                      int64_t T, int32_t dtype) {
  if (!p || !aligned(p, 16)) return invalid(who, (std::string(name) + " must be a 16-byte aligned pointer").c_str());
  if ((T > 1 && stride < (int64_t)heads * D) || (T > 1 && (stride * (int64_t)size_of(dtype)) % 16) ||
      stride > ((int64_t)1 << 40) || (T > 1 && stride > MOST_BYTES / (int64_t)size_of(dtype) / (T - 1)))
    return invalid(who, (std::string(name) + "'s token stride must cover its heads and be a multiple of 16 bytes").c_str());
  return OQ_OK;
}
RopeArgs rope_args(const QkIn& a) {
  RopeArgs r = {};
  r.gain[0] = a.q_gain;
  r.gain[1] = a.k_gain;
  r.gain_bf16 = a.gain_dtype == OQ_DTYPE_BF16;
  r.table = static_cast<const float*>(a.table);
  r.table_rows = a.table_rows;
  r.positions = static_cast<const int*>(a.positions);
  r.T = a.T;
  r.eps = a.eps;
  r.D = a.D;
  r.rot = a.table ? a.rot : 0;
  r.dtype = a.dtype;
  r.norm = !(a.flags & OQ_QK_NO_NORM);
  r.interleaved = (a.flags & OQ_QK_INTERLEAVED) != 0;
  return r;
}
Rows table_of(const QkIn& a) { return flat(a.table, a.table ? (size_t)a.table_rows * a.rot * 4 : 0); }
Rows positions_of(const QkIn& a) { return flat(a.positions, a.positions ? (size_t)a.T * 4 : 0); }
Rows gain_of(const QkIn& a, const void* g) { return flat(g, g ? (size_t)a.D * size_of(a.gain_dtype) : 0); }

bool on_device(const oq_kv4* kv) {
  int dev = -1;
  cudaGetDevice(&dev);
  return dev == kv->device;
}
oq_status check_cache(const char* who, const oq_kv4* kv, const void* cache, int64_t pages, const int32_t* table,
                      int32_t width, const int32_t* cu, const int32_t* lens, int32_t B, KvView* view) {
  if (!kv) return invalid(who, "the handle is null");
  if (pages < 0 || width < 0 || B < 0) return invalid(who, "pages, table_width and B must not be negative");
  if (!cache || !aligned(cache, 32)) return invalid(who, "the cache must be a 32-byte aligned pointer");
  if ((!table && B * (int64_t)width > 0) || (B > 0 && (!cu || !lens)) || !aligned(table, 4) || !aligned(cu, 4) || !aligned(lens, 4))
    return invalid(who, "page_table, cu and lens must be 4-byte aligned pointers");
  if (pages == 0 || pages > 0x7FFFFFFF / KV_ROWS / kv->groups)
    return unsupported(who, "the cache must have a page and at most 2^31 / 272 groups of 128 channels in its pages");
  // (attention marks tokens that are not there by a place of 2^30)
  if (width > (1 << 30) / KV_PAGE || B > 65535) return unsupported(who, "at most 2^23 pages a sequence and 65535 sequences");
  if (!on_device(kv)) return invalid(who, "the handle was created on another device than the current one");
  view->cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  view->pages = pages;
  view->table = table;
  view->cu = cu;
  view->lens = lens;
  view->B = B;
  view->width = width;
  view->groups = kv->groups;
  return OQ_OK;
}
Rows cache_of(const oq_kv4* kv, const void* cache, int64_t pages) {
  return flat(cache, (size_t)pages * kv->groups * KV_GROUP_BYTES);
}

oq_status check_overlap(const char* who, std::initializer_list<Rows> written, std::initializer_list<Rows> read) {
  for (const Rows* w = written.begin(); w != written.end(); ++w) {
    for (const Rows* o = w + 1; o != written.end(); ++o)
      if (overlap(*w, *o)) return invalid(who, "two outputs overlap");
    for (const Rows& r : read)
      if (overlap(*w, r)) return invalid(who, "an output overlaps another argument");
  }
  return OQ_OK;
}
oq_status done(oq_status st, const char* who) {
  return st == OQ_ERR_UNSUPPORTED ? unsupported(who, "too much work for one call") : st;
}

}  // namespace
}  // namespace oq

using namespace oq;

extern "C" {

oq_status oq_qk_norm_rope(const void* q, int64_t q_stride, int32_t q_heads, const void* k, int64_t k_stride, int32_t k_heads,
                          int32_t dtype, int64_t T, int32_t head_dim, const void* q_gain, const void* k_gain,
                          int32_t gain_dtype, float eps, const float* table, int64_t table_rows, int32_t rot,
                          const int32_t* positions, int32_t flags, void* q_out, int64_t q_out_stride, void* k_out,
                          int64_t k_out_stride, void* stream) {
  const char* who = "oq_qk_norm_rope";
  if (head_dim <= 0 || q_heads < 0 || k_heads < 0 || q_heads + (int64_t)k_heads < 1)
    return invalid(who, "head_dim must be positive and there must be a head");
  if (head_dim % 8 || head_dim > 256 || q_heads > 65536 || k_heads > 65536)
    return unsupported(who, "head_dim must be a multiple of 8 up to 256, heads at most 65536");
  const QkIn in{who, T, head_dim, dtype, gain_dtype, rot, flags, eps, q_gain, k_gain, table, positions, table_rows};
  oq_status st = check_qk(in);
  if (st != OQ_OK || T == 0) return st;
  if (q_heads && ((st = check_heads(who, "q", q, q_heads, head_dim, q_stride, T, dtype)) != OQ_OK ||
                  (st = check_heads(who, "q_out", q_out, q_heads, head_dim, q_out_stride, T, dtype)) != OQ_OK))
    return st;
  if (k_heads && ((st = check_heads(who, "k", k, k_heads, head_dim, k_stride, T, dtype)) != OQ_OK ||
                  (st = check_heads(who, "k_out", k_out, k_heads, head_dim, k_out_stride, T, dtype)) != OQ_OK))
    return st;
  const Rows none = flat(nullptr, 0);
  const Rows qi = q_heads ? heads_of(q, T, q_heads, head_dim, q_stride, dtype) : none;
  const Rows ki = k_heads ? heads_of(k, T, k_heads, head_dim, k_stride, dtype) : none;
  const Rows qo = q_heads ? heads_of(q_out, T, q_heads, head_dim, q_out_stride, dtype) : none;
  const Rows ko = k_heads ? heads_of(k_out, T, k_heads, head_dim, k_out_stride, dtype) : none;
  if ((st = check_overlap(who, {qo, ko},
                          {same(qo, qi) ? none : qi, none, gain_of(in, q_gain), gain_of(in, k_gain), table_of(in),
                           positions_of(in)})) != OQ_OK ||
      (st = check_overlap(who, {ko}, {same(ko, ki) ? none : ki, qi})) != OQ_OK ||
      (st = check_overlap(who, {qo}, {ki})) != OQ_OK)
    return st;
  RopeArgs r = rope_args(in);
  r.x[0] = q, r.x[1] = k;
  r.out[0] = q_out, r.out[1] = k_out;
  r.in_stride[0] = q_stride, r.in_stride[1] = k_stride;
  r.out_stride[0] = q_out_stride, r.out_stride[1] = k_out_stride;
  r.heads[0] = q_heads, r.heads[1] = k_heads;
  return done(rope_launch(r, stream), who);
}

oq_status oq_kv4_create(int32_t heads, int32_t kv_heads, int32_t head_dim, oq_kv4** out) {
  const char* who = "oq_kv4_create";
  if (!out) return invalid(who, "out is null");
  *out = nullptr;
  if (heads <= 0 || kv_heads <= 0) return invalid(who, "heads must be positive");
  if ((head_dim != 64 && head_dim != 128) || heads % kv_heads || heads > 65536)
    return unsupported(who, "head_dim must be 64 or 128, heads a multiple of kv_heads, at most 65536");
  oq_kv4* kv = new (std::nothrow) oq_kv4();
  if (!kv) return fail(OQ_ERR_NOMEM, "host allocation failed");
  kv->heads = heads;
  kv->kv_heads = kv_heads;
  kv->head_dim = head_dim;
  kv->groups = (kv_heads * head_dim + 127) / 128;
  cudaGetDevice(&kv->device);
  cudaError_t e = cudaMalloc(&kv->d_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(kv->d_error, 0, sizeof(int));
  if (e != cudaSuccess) {
    oq_kv4_destroy(kv);
    return fail(e == cudaErrorMemoryAllocation ? OQ_ERR_NOMEM : OQ_ERR_CUDA,
                std::string("error word: ") + cudaGetErrorString(e));
  }
  *out = kv;
  return OQ_OK;
}

void oq_kv4_destroy(oq_kv4* kv) {
  if (!kv) return;
  if (kv->d_error) cudaFree(kv->d_error);
  delete kv;
}

oq_status oq_kv4_poll_error(const oq_kv4* kv) {
  const char* who = "oq_kv4_poll_error";
  if (!kv) return invalid(who, "the handle is null");
  // (on another device the calls whose word this is would not be waited for)
  if (!on_device(kv)) return invalid(who, "the handle was created on another device than the current one");
  int word = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&word, kv->d_error, sizeof(int), cudaMemcpyDeviceToHost);
  if (e == cudaSuccess && word) e = cudaMemset(kv->d_error, 0, sizeof(int));
  if (e != cudaSuccess) return fail(OQ_ERR_CUDA, std::string(who) + ": " + cudaGetErrorString(e));
  if (word & OQ_DEVERR_TIMEOUT) return fail(OQ_ERR_TIMEOUT, "a kernel's bounded wait ran out");
  return word ? fail(OQ_ERR_DEVICE, "unknown bits in the device error word") : OQ_OK;
}

size_t oq_kv4_cache_size(const oq_kv4* kv, int64_t pages) {
  if (!kv || pages <= 0 || pages > 0x7FFFFFFF / KV_ROWS / kv->groups) return 0;
  return (size_t)pages * kv->groups * KV_GROUP_BYTES;
}

oq_status oq_kv4_append(const oq_kv4* kv, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, int32_t dtype, int64_t T, const void* q_gain, const void* k_gain,
                        int32_t gain_dtype, float eps, const float* table, int64_t table_rows, int32_t rot,
                        const int32_t* positions, int32_t flags, void* q_out, uint8_t* cache, int64_t pages,
                        const int32_t* page_table, int32_t table_width, const int32_t* cu, const int32_t* lens, int32_t B,
                        void* stream) {
  const char* who = "oq_kv4_append";
  AppendArgs a = {};
  oq_status st = check_cache(who, kv, cache, pages, page_table, table_width, cu, lens, B, &a.kv);
  if (st != OQ_OK) return st;
  const int D = kv->head_dim;
  const QkIn in{who, T, D, dtype, gain_dtype, rot, flags, eps, q_gain, k_gain, table, positions, table_rows};
  if ((st = check_qk(in)) != OQ_OK || T == 0 || B == 0) return st;
  if (!q != !q_out) return invalid(who, "q and q_out go together");
  if ((q && ((st = check_heads(who, "q", q, kv->heads, D, q_stride, T, dtype)) != OQ_OK ||
             (st = check_heads(who, "q_out", q_out, kv->heads, D, (int64_t)kv->heads * D, T, OQ_DTYPE_BF16)) != OQ_OK)) ||
      (st = check_heads(who, "k", k, kv->kv_heads, D, k_stride, T, dtype)) != OQ_OK ||
      (st = check_heads(who, "v", v, kv->kv_heads, D, v_stride, T, dtype)) != OQ_OK)
    return st;
  const Rows none = flat(nullptr, 0);
  const Rows qi = q ? heads_of(q, T, kv->heads, D, q_stride, dtype) : none;
  const Rows qo = q ? flat(q_out, (size_t)T * kv->heads * D * 2) : none;
  const bool in_place = q && q == q_out && dtype == OQ_DTYPE_BF16 && (q_stride == (int64_t)kv->heads * D || T == 1);
  const Rows ki = heads_of(k, T, kv->kv_heads, D, k_stride, dtype), vi = heads_of(v, T, kv->kv_heads, D, v_stride, dtype);
  const Rows c = cache_of(kv, cache, pages);
  const Rows tb = flat(page_table, (size_t)B * table_width * 4), cb = flat(cu, (size_t)(B + 1) * 4), lb = flat(lens, (size_t)B * 4);
  if ((st = check_overlap(who, {qo, c},
                          {in_place ? none : qi, ki, vi, tb, cb, lb, gain_of(in, q_gain), gain_of(in, k_gain), table_of(in),
                           positions_of(in)})) != OQ_OK ||
      (st = check_overlap(who, {c}, {qi})) != OQ_OK)
    return st;
  a.rope = rope_args(in);
  a.rope.x[0] = q, a.rope.x[1] = k;
  a.rope.out[0] = q_out;
  a.rope.in_stride[0] = q_stride, a.rope.in_stride[1] = k_stride;
  a.rope.out_stride[0] = (int64_t)kv->heads * D;
  a.rope.heads[0] = q ? kv->heads : 0, a.rope.heads[1] = kv->kv_heads;
  a.v = v;
  a.v_stride = v_stride;
  a.err = kv->d_error;
  return done(kv4_append_launch(a, stream), who);
}

oq_status oq_kv4_read(const oq_kv4* kv, const uint8_t* cache, int64_t pages, const int32_t* page_table, int32_t table_width,
                      const int32_t* cu, const int32_t* lens, int32_t B, int64_t T, void* k, void* v, int32_t dtype,
                      void* stream) {
  const char* who = "oq_kv4_read";
  ReadArgs a = {};
  oq_status st = check_cache(who, kv, cache, pages, page_table, table_width, cu, lens, B, &a.kv);
  if (st != OQ_OK) return st;
  if (T < 0) return invalid(who, "T must not be negative");
  if (!known(dtype)) return invalid(who, "dtype must be OQ_DTYPE_F32 or OQ_DTYPE_BF16");
  if (T > 0x7FFFFFFF) return unsupported(who, "at most 2^31 - 1 tokens per call");
  if (T == 0 || B == 0) return OQ_OK;
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return invalid(who, "k and v must be 16-byte aligned pointers");
  const size_t bytes = (size_t)T * kv->kv_heads * kv->head_dim * size_of(dtype);
  if ((st = check_overlap(who, {flat(k, bytes), flat(v, bytes)},
                          {cache_of(kv, cache, pages), flat(page_table, (size_t)B * table_width * 4),
                           flat(cu, (size_t)(B + 1) * 4), flat(lens, (size_t)B * 4)})) != OQ_OK)
    return st;
  a.k = k;
  a.v = v;
  a.T = T;
  a.kv_heads = kv->kv_heads;
  a.D = kv->head_dim;
  a.dtype = dtype;
  return done(kv4_read_launch(a, stream), who);
}

size_t oq_kv4_attention_workspace_size(const oq_kv4* kv, int64_t T, int32_t B, int32_t max_q, int32_t max_len) {
  if (!kv || T <= 0 || T > 0x7FFFFFFF / kv->heads || B <= 0 || max_q <= 0 || max_len < 0) return 0;   // (such calls are refused or empty)
  return kv4_attention_workspace(kv, T, B, max_q, max_len);
}

oq_status oq_kv4_attention(const oq_kv4* kv, const void* q, int64_t q_stride, int64_t T, const uint8_t* cache, int64_t pages,
                           const int32_t* page_table, int32_t table_width, const int32_t* cu, const int32_t* lens, int32_t B,
                           int32_t max_q, int32_t max_len, float scale, int32_t flags, int32_t window, void* y,
                           void* workspace, size_t workspace_bytes, void* stream) {
  const char* who = "oq_kv4_attention";
  AttentionArgs a = {};
  oq_status st = check_cache(who, kv, cache, pages, page_table, table_width, cu, lens, B, &a.kv);
  if (st != OQ_OK) return st;
  if (T < 0 || max_q < 0 || max_len < 0 || window < 0)
    return invalid(who, "T, max_q, max_len and window must not be negative");
  if (!(scale > 0.f) || std::isinf(scale * 1.4426950408889634f))
    return invalid(who, "scale must be positive, and scale log2(e) finite");
  if (flags & ~OQ_ATTN_CAUSAL) return invalid(who, "unknown flags");
  const int group = kv->heads / kv->kv_heads;
  if (T > 0x7FFFFFFF / kv->heads || (int64_t)max_q * group > 0x7FFFFFFF - 64 || kv->kv_heads > 1023)
    return unsupported(who, "at most 2^31 rows of queries per call and 1023 key heads");
  if (T == 0 || B == 0 || max_q == 0) return OQ_OK;
  if ((st = check_heads(who, "q", q, kv->heads, kv->head_dim, q_stride, T, OQ_DTYPE_BF16)) != OQ_OK) return st;
  if (!y || !aligned(y, 16)) return invalid(who, "y must be a 16-byte aligned pointer");
  if (workspace_bytes && (!workspace || !aligned(workspace, 256)))
    return invalid(who, "the workspace must be a 256-byte aligned pointer");
  const Rows yr = flat(y, (size_t)T * kv->heads * kv->head_dim * 2), ws = flat(workspace, workspace_bytes);
  const Rows qr = heads_of(q, T, kv->heads, kv->head_dim, q_stride, OQ_DTYPE_BF16);
  const Rows tb = flat(page_table, (size_t)B * table_width * 4), cb = flat(cu, (size_t)(B + 1) * 4), lb = flat(lens, (size_t)B * 4);
  if ((st = check_overlap(who, {yr, ws}, {qr, cache_of(kv, cache, pages), tb, cb, lb})) != OQ_OK) return st;
  a.q = q;
  a.q_stride = q_stride;
  a.T = T;
  a.y = y;
  a.scale = scale;
  a.heads = kv->heads;
  a.kv_heads = kv->kv_heads;
  a.D = kv->head_dim;
  a.max_q = max_q;
  a.max_len = max_len;
  a.window = window < (1 << 30) ? window : 0;   // (a sequence has no more tokens: everything is within it)
  a.causal = (flags & OQ_ATTN_CAUSAL) != 0;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.err = kv->d_error;
  return done(kv4_attention_launch(a, stream), who);
}

static oq_status check_w4g(const char* who, int32_t d_out, int32_t d_in, int32_t group, const uint8_t* codes,
                           const void* scales) {
  if (d_out <= 0 || d_in <= 0) return invalid(who, "dimensions must be positive");
  if (group != 32 && group != 64 && group != 128) return unsupported(who, "group must be 32, 64 or 128");
  if (d_in % group || d_in > (1 << 24) || d_out > (1 << 28))
    return unsupported(who, "d_in must be a multiple of group up to 2^24, d_out at most 2^28");
  if (!codes || !scales || !aligned(codes, 16) || !aligned(scales, 16))
    return invalid(who, "codes and scales must be 16-byte aligned pointers");
  return OQ_OK;
}
static Rows w4g_codes(const void* p, int32_t d_out, int32_t d_in) {
  return flat(p, (size_t)d_out * (((size_t)d_in + 127) / 128 * 64));
}
static Rows w4g_groups(const void* p, int32_t d_out, int32_t d_in, int32_t group, size_t e) {
  return flat(p, p ? (size_t)d_out * (d_in / group) * e : 0);
}

oq_status oq_w4g_prepare(const void* W, int32_t W_dtype, int32_t d_out, int32_t d_in, int32_t group, uint8_t* codes,
                         void* scales, uint8_t* zeros, void* stream) {
  const char* who = "oq_w4g_prepare";
  oq_status st = check_w4g(who, d_out, d_in, group, codes, scales);
  if (st != OQ_OK) return st;
  if (!known(W_dtype)) return invalid(who, "dtype must be OQ_DTYPE_F32 or OQ_DTYPE_BF16");
  if (!W || !aligned(W, 16)) return invalid(who, "W must be a 16-byte aligned pointer");
  if ((st = check_overlap(who, {w4g_codes(codes, d_out, d_in), w4g_groups(scales, d_out, d_in, group, 2),
                                w4g_groups(zeros, d_out, d_in, group, 1)},
                          {flat(W, (size_t)d_out * d_in * size_of(W_dtype))})) != OQ_OK)
    return st;
  return done(w4g_prepare_launch(W, W_dtype, d_out, d_in, group, codes, scales, zeros, stream), who);
}

oq_status oq_linear_w4g(const void* x, int32_t x_dtype, int64_t T, int32_t d_in, int32_t d_out, int32_t group,
                        const uint8_t* codes, const void* scales, const uint8_t* zeros, void* y, int32_t y_dtype,
                        void* stream) {
  const char* who = "oq_linear_w4g";
  oq_status st = check_w4g(who, d_out, d_in, group, codes, scales);
  if (st != OQ_OK) return st;
  if (!known(x_dtype) || !known(y_dtype)) return invalid(who, "dtype must be OQ_DTYPE_F32 or OQ_DTYPE_BF16");
  if (T < 0) return invalid(who, "T must not be negative");
  if (T > 65535 * 10) return unsupported(who, "at most 655350 tokens per call");
  if (T == 0) return OQ_OK;
  if (!x || !y || !aligned(x, 16) || !aligned(y, 16)) return invalid(who, "x and y must be 16-byte aligned pointers");
  if ((st = check_overlap(who, {flat(y, (size_t)T * d_out * size_of(y_dtype))},
                          {flat(x, (size_t)T * d_in * size_of(x_dtype)), w4g_codes(codes, d_out, d_in),
                           w4g_groups(scales, d_out, d_in, group, 2), w4g_groups(zeros, d_out, d_in, group, 1)})) != OQ_OK)
    return st;
  W4gArgs a;
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  a.zeros = zeros;
  a.y = y;
  a.T = T;
  a.N = d_out;
  a.K = d_in;
  a.group = group;
  a.x_dtype = x_dtype;
  a.y_dtype = y_dtype;
  return done(w4g_linear_launch(a, stream), who);
}

}  // extern "C"
