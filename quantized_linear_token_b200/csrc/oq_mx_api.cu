// C-ABI entry points of the microscaled operators (declared in
// include/orbitquant.h): argument checks, the microscaled layer and dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <initializer_list>
#include <new>
#include <string>

#include "oq_mx.cuh"

namespace oq {
namespace {

oq_status fail(oq_status st, const std::string& msg) {
  set_error(msg);
  return st;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// row and column coordinates of the kernels' tiles and grids are 32-bit, also
// those behind the end of the last tile
constexpr int64_t MAX_ROWS = ((int64_t)1 << 31) - 1024;

oq_status check_shape(const std::string& who, int64_t rows, int32_t d, int32_t bits) {
  if (rows < 0 || d <= 0) return fail(OQ_ERR_INVALID_ARG, who + ": rows must not be negative, d must be positive");
  if (d % MX_BLOCK || d > 65535) return fail(OQ_ERR_UNSUPPORTED, who + ": d must be a multiple of 32 below 65536");
  if (bits != 4 && bits != 8) return fail(OQ_ERR_UNSUPPORTED, who + ": bits must be 4 or 8");
  if (rows > MAX_ROWS) return fail(OQ_ERR_UNSUPPORTED, who + ": at most 2^31 - 1024 rows per call");
  return OQ_OK;
}

oq_status check_dtype(const std::string& who, int32_t dtype) {
  if (dtype == OQ_DTYPE_F32 || dtype == OQ_DTYPE_BF16) return OQ_OK;
  return fail(OQ_ERR_INVALID_ARG, who + ": dtype must be OQ_DTYPE_F32 or OQ_DTYPE_BF16");
}

oq_status check_codes(const std::string& who, const void* codes, const void* scales) {
  if (!codes || !scales || !aligned(codes, 32) || !aligned(scales, 16))
    return fail(OQ_ERR_INVALID_ARG, who + ": codes (32-byte) / scales (16-byte) pointers invalid");
  return OQ_OK;
}

// A written range against the call's others: any overlap is refused, but for
// the same array given twice where `same` allows it.
struct Range {
  const void* p;
  size_t bytes;
};
bool overlap(const Range& a, const Range& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + b.bytes && y < x + a.bytes;
}
oq_status check_overlap(const char* who, const Range& written, std::initializer_list<Range> others, bool same = false) {
  for (const Range& r : others)
    if (overlap(written, r) && !(same && written.p == r.p))
      return fail(OQ_ERR_INVALID_ARG, std::string(who) + ": an output overlaps another argument");
  return OQ_OK;
}
size_t row_array(int64_t rows, int32_t d, int32_t dtype) {
  return (size_t)rows * (size_t)d * (dtype == OQ_DTYPE_F32 ? 4 : 2);
}

oq_status unsupported(oq_status st, const char* who) {
  return st == OQ_ERR_UNSUPPORTED ? fail(st, std::string(who) + ": too many elements for one call") : st;
}

}  // namespace

int mx_sm_count(int* device) {
  static std::atomic<int> known[64];
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  *device = dev;
  if (dev >= 0 && dev < 64 && (sms = known[dev].load(std::memory_order_relaxed))) return sms;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (dev >= 0 && dev < 64) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

oq_status mx_allow_smem(const void* kernel, size_t bytes, int device, std::atomic<uint64_t>* done) {
  const uint64_t bit = device >= 0 && device < 64 ? (uint64_t)1 << device : 0;
  if (done->load(std::memory_order_relaxed) & bit) return OQ_OK;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess)
    return fail(OQ_ERR_CUDA, std::string("cudaFuncSetAttribute(microscaled product): ") + cudaGetErrorString(e));
  done->fetch_or(bit, std::memory_order_relaxed);
  return OQ_OK;
}

oq_status create_mx_layer(int32_t d_in, int32_t d_out, uint64_t seed, int32_t a_bits, int32_t w_bits, int32_t flags,
                          oq_layer** out) {
  if (flags != OQ_FLAG_MICROSCALED) return fail(OQ_ERR_INVALID_ARG, "OQ_FLAG_MICROSCALED takes no other flag");
  if ((a_bits != 4 && a_bits != 8) || w_bits != 4)
    return fail(OQ_ERR_UNSUPPORTED, "the microscaled layer takes a_bits = 4 or 8 and w_bits = 4");
  if (d_in <= 0 || d_out <= 0) return fail(OQ_ERR_INVALID_ARG, "dimensions must be positive");
  if (d_in % MX_BLOCK || d_in > 65535 || d_out % 16)
    return fail(OQ_ERR_UNSUPPORTED, "the microscaled layer needs d_in % 32 == 0, d_in < 65536 and d_out % 16 == 0");
  if (d_out > MAX_ROWS) return fail(OQ_ERR_UNSUPPORTED, "the microscaled layer takes d_out up to 2^31 - 1024");
  oq_layer* L = new (std::nothrow) oq_layer();
  if (!L) return fail(OQ_ERR_NOMEM, "host allocation failed");
  L->mx = true;
  L->d_in = d_in;
  L->d_out = d_out;
  L->h = d_in & -d_in;
  L->k = d_in / L->h;
  L->a_bits = a_bits;
  L->w_bits = w_bits;
  L->flags = flags;
  L->seed = seed;
  L->a_scale = L->w_scale = 1.0;
  cudaGetDevice(&L->device);
  cudaError_t e = cudaMalloc(&L->d_error, sizeof(int));
  if (e == cudaSuccess) e = cudaMemset(L->d_error, 0, sizeof(int));
  if (e != cudaSuccess) {
    oq_layer_destroy(L);
    return fail(e == cudaErrorMemoryAllocation ? OQ_ERR_NOMEM : OQ_ERR_CUDA,
                std::string("error word: ") + cudaGetErrorString(e));
  }
  *out = L;
  return OQ_OK;
}

}  // namespace oq

using namespace oq;

extern "C" {

size_t oq_mx_codes_size(int64_t rows, int32_t d, int32_t bits) {
  if (rows <= 0 || d <= 0 || d % MX_BLOCK || d > 65535 || (bits != 4 && bits != 8)) return 0;
  return (size_t)rows * (size_t)mx_row_bytes(d, bits);
}

size_t oq_mx_scales_size(int64_t rows, int32_t d) {
  if (rows <= 0 || d <= 0 || d % MX_BLOCK || d > 65535) return 0;
  return (size_t)mx_row_tiles(rows) * (size_t)mx_col_tiles(d) * MX_TILE_BYTES;
}

oq_status oq_mx_quantize(const void* x, int32_t x_dtype, int64_t rows, int32_t d, int32_t bits, uint8_t* codes,
                         uint8_t* scales, void* stream) {
  const char* who = "oq_mx_quantize";
  oq_status st = check_shape(who, rows, d, bits);
  if (st != OQ_OK || (st = check_dtype(who, x_dtype)) != OQ_OK || rows == 0) return st;
  if (!x || !aligned(x, 16)) return fail(OQ_ERR_INVALID_ARG, "oq_mx_quantize: x must be a 16-byte aligned pointer");
  if ((st = check_codes(who, codes, scales)) != OQ_OK) return st;
  const Range in{x, row_array(rows, d, x_dtype)};
  const Range c{codes, oq_mx_codes_size(rows, d, bits)}, s{scales, oq_mx_scales_size(rows, d)};
  if ((st = check_overlap(who, c, {in, s})) != OQ_OK || (st = check_overlap(who, s, {in})) != OQ_OK) return st;
  return unsupported(mx_quantize_launch(x, x_dtype, rows, d, bits, codes, scales, stream), who);
}

oq_status oq_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t d, int32_t bits, void* x,
                           int32_t x_dtype, void* stream) {
  const char* who = "oq_mx_dequantize";
  oq_status st = check_shape(who, rows, d, bits);
  if (st != OQ_OK || (st = check_dtype(who, x_dtype)) != OQ_OK || rows == 0) return st;
  if (!x || !aligned(x, 16)) return fail(OQ_ERR_INVALID_ARG, "oq_mx_dequantize: x must be a 16-byte aligned pointer");
  if ((st = check_codes(who, codes, scales)) != OQ_OK) return st;
  if ((st = check_overlap(who, {x, row_array(rows, d, x_dtype)},
                          {{codes, oq_mx_codes_size(rows, d, bits)}, {scales, oq_mx_scales_size(rows, d)}})) != OQ_OK)
    return st;
  return unsupported(mx_dequantize_launch(codes, scales, rows, d, bits, x, x_dtype, stream), who);
}

oq_status oq_rms_norm_mx(const void* x, const void* residual, int32_t x_dtype, const void* gain, int32_t gain_dtype,
                         float eps, int64_t rows, int32_t d, int32_t bits, void* residual_out, uint8_t* codes,
                         uint8_t* scales, void* stream) {
  const char* who = "oq_rms_norm_mx";
  oq_status st = check_shape(who, rows, d, bits);
  if (st != OQ_OK || (st = check_dtype(who, x_dtype)) != OQ_OK || (st = check_dtype(who, gain_dtype)) != OQ_OK) return st;
  if (!(eps >= 0.f) || std::isinf(eps))
    return fail(OQ_ERR_INVALID_ARG, "oq_rms_norm_mx: eps must be finite and not negative");
  if (rows == 0) return OQ_OK;
  if (!x || !aligned(x, 16) || !aligned(residual, 16) || !aligned(gain, 16) || !aligned(residual_out, 16))
    return fail(OQ_ERR_INVALID_ARG, "oq_rms_norm_mx: x, residual, gain and residual_out must be 16-byte aligned");
  if (residual_out && !residual)
    return fail(OQ_ERR_INVALID_ARG, "oq_rms_norm_mx: residual_out without a residual");
  if ((st = check_codes(who, codes, scales)) != OQ_OK) return st;
  const size_t n = row_array(rows, d, x_dtype);
  const Range in{x, n}, res{residual, n}, kept{residual_out, n}, g{gain, row_array(1, d, gain_dtype)};
  const Range c{codes, oq_mx_codes_size(rows, d, bits)}, s{scales, oq_mx_scales_size(rows, d)};
  if ((st = check_overlap(who, c, {in, res, kept, g, s})) != OQ_OK ||
      (st = check_overlap(who, s, {in, res, kept, g})) != OQ_OK || (st = check_overlap(who, kept, {g})) != OQ_OK ||
      (st = check_overlap(who, kept, {in, res}, true)) != OQ_OK)
    return st;
  MxNormArgs a;
  a.x = x;
  a.residual = residual;
  a.x_dtype = x_dtype;
  a.gain = gain;
  a.gain_dtype = gain_dtype;
  a.eps = eps;
  a.rows = rows;
  a.d = d;
  a.bits = bits;
  a.residual_out = residual_out;
  a.codes = codes;
  a.scales = scales;
  return unsupported(mx_norm_launch(a, stream), who);
}

oq_status oq_linear_mx(const oq_layer* L, const uint8_t* codes, const uint8_t* scales, int64_t T,
                       const uint8_t* Wcodes, const uint8_t* Wscales, void* y, int32_t y_dtype, void* stream) {
  const char* who = "oq_linear_mx";
  if (!L) return fail(OQ_ERR_INVALID_ARG, "oq_linear_mx: layer is null");
  if (!L->mx) return fail(OQ_ERR_UNSUPPORTED, "oq_linear_mx: the layer was not created with OQ_FLAG_MICROSCALED");
  oq_status st = check_shape(who, T, L->d_in, L->a_bits);
  if (st != OQ_OK || (st = check_dtype(who, y_dtype)) != OQ_OK || T == 0) return st;
  if ((st = check_codes(who, codes, scales)) != OQ_OK || (st = check_codes(who, Wcodes, Wscales)) != OQ_OK) return st;
  if (!y || !aligned(y, 16)) return fail(OQ_ERR_INVALID_ARG, "oq_linear_mx: y must be a 16-byte aligned pointer");
  if ((st = check_overlap(who, {y, row_array(T, L->d_out, y_dtype)},
                          {{codes, oq_mx_codes_size(T, L->d_in, L->a_bits)},
                           {scales, oq_mx_scales_size(T, L->d_in)},
                           {Wcodes, oq_mx_codes_size(L->d_out, L->d_in, 4)},
                           {Wscales, oq_mx_scales_size(L->d_out, L->d_in)}})) != OQ_OK)
    return st;
  int dev = -1;
  cudaGetDevice(&dev);
  if (dev != L->device)
    return fail(OQ_ERR_INVALID_ARG, "oq_linear_mx: the layer was created on another device than the current one");
  MxGemmArgs g;
  g.a_codes = codes;
  g.a_scales = scales;
  g.w_codes = Wcodes;
  g.w_scales = Wscales;
  g.y = y;
  g.y_bf16 = y_dtype == OQ_DTYPE_BF16;
  g.T = T;
  g.N = L->d_out;
  g.K = L->d_in;
  g.a_bits = L->a_bits;
  g.err = L->d_error;
  return unsupported(mx_small_batch(T, g.K, g.a_bits) ? mx_small_launch(g, stream) : mx_gemm_launch(g, stream), who);
}

}  // extern "C"
