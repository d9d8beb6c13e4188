// Microscaled quantisation of rows, its read-back, and the root-mean-square
// norm with the residual's addition whose output is quantised (formats and
// layouts: oq_mx.cuh).  All three are bound by HBM.
#include <cuda_bf16.h>

#include <algorithm>
#include <string>

#include "oq_internal.h"
#include "oq_mx.cuh"

namespace oq {
namespace {

oq_status launch_status(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return OQ_OK;
  set_error(std::string(what) + " launch: " + cudaGetErrorString(e));
  return OQ_ERR_CUDA;
}

// ------------------------------------------------------------------ quantise
// A CTA owns one scale tile: 128 rows x 128 elements.  Sixteen lanes take a
// row of the tile, eight elements each, so a warp's loads cover two rows'
// 256-byte (bf16) segments; a thread loads its eight rows' vectors before it
// uses the first.  The tile's 512 scale bytes are gathered in shared memory
// and leave as whole sectors.  Rows past the end read as zeros and get scale
// code 0; columns past d get zero codes and scale code 0.
constexpr int QT = 256;
constexpr int QSTEP = QT / 16;                // rows between a thread's rows
constexpr int QROWS = MX_ROWS / QSTEP;        // rows per thread

// the tile of this CTA: row tile, column tile, and how many of this thread's rows exist
struct TileSpan {
  int64_t row0;
  int ct, sub, col, live;   // live: rows of the tile from this thread's first on
};
__device__ __forceinline__ TileSpan tile_span(int64_t rows, int col_tiles) {
  TileSpan t;
  const unsigned rt = blockIdx.x / (unsigned)col_tiles;
  t.ct = (int)(blockIdx.x - rt * (unsigned)col_tiles);
  t.sub = threadIdx.x >> 4;
  t.col = t.ct * MX_COLS + (threadIdx.x & 15) * 8;
  t.row0 = (int64_t)rt * MX_ROWS + t.sub;
  t.live = (int)(rows - t.row0 < MX_ROWS ? rows - t.row0 : MX_ROWS);
  return t;
}

template <typename T, int BITS>
__global__ void __launch_bounds__(QT) mx_quantize_kernel(const T* __restrict__ x, int64_t rows, int d, int col_tiles,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ uint32_t tile[MX_TILE_BYTES / 4];
  const TileSpan t = tile_span(rows, col_tiles);
  const bool in_cols = t.col < d;
  const T* src = x + t.row0 * d + t.col;
  Vec8<T> in[QROWS];
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    if (in_cols && i * QSTEP < t.live) in[i].load(src + (int64_t)i * QSTEP * d);
    else in[i].zero();
  }
  const int pitch = col_tiles * (MX_COLS * BITS / 8);
  uint8_t* dst = codes + t.row0 * pitch + t.col * BITS / 8;
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    float v[8];
    in[i].get(v);
    const uint32_t code = mx_scale_code<BITS>(mx_block_max(v));
    const float inv = mx_inverse_scale(code);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= inv;
    uint32_t out[BITS / 4];
    mx_element_codes<BITS>(v, code, out);
    const uint32_t word = mx_scale_word(code);
    if (i * QSTEP < t.live) {
      uint8_t* q = dst + (int64_t)i * QSTEP * pitch;
      if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(q) = out[0];
      else *reinterpret_cast<uint2*>(q) = make_uint2(out[0], out[1]);
    }
    if ((threadIdx.x & 15) == 0) tile[mx_tile_word(t.sub + i * QSTEP)] = word;
  }
  __syncthreads();
  if (threadIdx.x < MX_TILE_BYTES / 16)
    reinterpret_cast<uint4*>(scales + (int64_t)blockIdx.x * MX_TILE_BYTES)[threadIdx.x] =
        reinterpret_cast<const uint4*>(tile)[threadIdx.x];
}

// ------------------------------------------------------------------ read-back
// The same tiles: value = element * 2^(scale code - 127).  Scale code 0 is
// 2^-127, a subnormal; code 255 is NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t code) {
  return code == 255u ? __uint_as_float(0x7FFFFFFFu) : code == 0u ? __uint_as_float(1u << 22) : __uint_as_float(code << 23);
}

// Eight e2m1 codes as bf16 pairs: the magnitudes' high and low bytes come from
// two byte tables, four codes a lookup, and the sign bits are moved in.
__device__ __forceinline__ void e2m1_bf16(uint32_t w, uint32_t (&o)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t u = w >> (16 * h), sel = u & 0x7777u;
    // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 as bf16
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel), lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    o[2 * h] = __byte_perm(lo, hi, 0x5140) | ((u << 12) & 0x8000u) | ((u << 24) & 0x80000000u);
    o[2 * h + 1] = __byte_perm(lo, hi, 0x7362) | ((u << 4) & 0x8000u) | ((u << 16) & 0x80000000u);
  }
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// four e4m3 codes to fp32 (exact by way of fp16; 0x7F and 0xFF are NaN)
__device__ __forceinline__ void e4m3_f32(uint32_t w, float* v) {
  uint32_t a, b;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(v[0]), "=f"(v[1])
      : "r"(a));
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(v[2]), "=f"(v[3])
      : "r"(b));
}

// one thread's eight values
template <int BITS>
__device__ __forceinline__ void mx_values(const uint32_t (&in)[BITS / 4], uint32_t code, float* p) {
  const float s = mx_scale_value(code);
  float v[8];
  if constexpr (BITS == 4) {
    uint32_t o[4];
    e2m1_bf16(in[0], o);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(o[k] << 16);
      v[2 * k + 1] = __uint_as_float(o[k] & 0xFFFF0000u);
    }
  } else {
    e4m3_f32(in[0], v);
    e4m3_f32(in[1], v + 4);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= s;
  store8(p, v);
}
template <int BITS>
__device__ __forceinline__ void mx_values(const uint32_t (&in)[BITS / 4], uint32_t code, __nv_bfloat16* p) {
  if constexpr (BITS == 4) {
    // products of bf16 pairs: exact, but for results below bf16's normal range, rounded once
    uint32_t o[4];
    e2m1_bf16(in[0], o);
    const uint32_t s = mx_pack_bf16(mx_scale_value(code), mx_scale_value(code));
    *reinterpret_cast<uint4*>(p) =
        make_uint4(mul_bf16x2(o[0], s), mul_bf16x2(o[1], s), mul_bf16x2(o[2], s), mul_bf16x2(o[3], s));
  } else {
    const float s = mx_scale_value(code);
    float v[8];
    e4m3_f32(in[0], v);
    e4m3_f32(in[1], v + 4);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= s;
    store8(p, v);
  }
}

template <typename T, int BITS>
__global__ void __launch_bounds__(QT) mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t rows, int d,
                                                           int col_tiles, T* __restrict__ x) {
  const TileSpan t = tile_span(rows, col_tiles);
  if (t.col >= d) return;
  const int pitch = col_tiles * (MX_COLS * BITS / 8);
  const uint8_t* src = codes + t.row0 * pitch + t.col * BITS / 8;
  const uint8_t* tile = scales + (int64_t)blockIdx.x * MX_TILE_BYTES + ((threadIdx.x >> 2) & 3);
  uint32_t in[QROWS][BITS / 4], sc[QROWS];
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    if (i * QSTEP >= t.live) continue;
    const uint8_t* q = src + (int64_t)i * QSTEP * pitch;
    if constexpr (BITS == 4) {
      in[i][0] = *reinterpret_cast<const uint32_t*>(q);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(q);
      in[i][0] = u.x;
      in[i][1] = u.y;
    }
    sc[i] = tile[4 * mx_tile_word(t.sub + i * QSTEP)];
  }
  T* dst = x + t.row0 * d + t.col;
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    if (i * QSTEP >= t.live) break;
    mx_values<BITS>(in[i], sc[i], dst + (int64_t)i * QSTEP * d);
  }
}

// ------------------------------------------------------------------ norm
// h = x + r, the kept residual is h rounded to the input's type, and
// n = h * (1 / sqrt(mean(h^2) + eps)) * g from the unrounded h.
//
// tpr threads own a row, each NCH vectors of eight neighbouring elements that
// stay in registers between the sum and the quantisation (one pass over x and
// r).  NCH = 0 reads x and r a second time instead (rows too long for the
// registers): each thread re-reads only elements that it alone writes, so the
// kept residual may overwrite either input in both forms.
//
// Precision: a thread adds its own squares in fp32, the row's sum is fp64, and
// so is 1 / sqrt (an fp32 estimate, two Newton steps).  n is formed in fp32; it
// may be four ulps off, which matters only where an element lies that close to
// the border between two codes (or the block's largest to a power of two).  A
// warp that meets such an element (0.2 % of its steps) forms its elements
// again in fp64, rounded to fp32 towards the odd neighbour, from which the
// rounding to the element type is that of the fp64 value.
struct NormParams {
  const void* x;
  const void* r;
  const void* g;
  bool g_bf16;
  float eps;
  double inv_d;
  int64_t rows;
  int d, col_tiles, tpr, row_ctas;
  void* r_out;
  uint8_t* codes;
  uint8_t* scales;
};

template <typename T>
__device__ __forceinline__ void load_h(const T* x, const T* r, float (&h)[8]) {
  Vec8<T> a;
  a.load(x);
  a.get(h);
  if (r) {
    float b[8];
    Vec8<T> c;
    c.load(r);
    c.get(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += b[i];
  }
}

__device__ __forceinline__ void load_gain(const NormParams& p, int col, float (&g)[8]) {
  if (!p.g) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.f;
  } else if (p.g_bf16) {
    Vec8<__nv_bfloat16> q;
    q.load(static_cast<const __nv_bfloat16*>(p.g) + col);
    q.get(g);
  } else {
    Vec8<float> q;
    q.load(static_cast<const float*>(p.g) + col);
    q.get(g);
  }
}

// an fp64 value as fp32: exact, or the neighbour with an odd last bit
__device__ __forceinline__ float to_odd(double v) {
  const float f = __double2float_rz(v);
  return (double)f == v || !isfinite(f) ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

// 1 / sqrt(v) to 1e-13: an fp32 estimate and one Newton step
__device__ __forceinline__ double rsqrt64(double v) {
  if (!(v > 1e-36 && v < 1e36)) return 1.0 / sqrt(v);
  const double y = (double)rsqrtf((float)v);
  return y * (1.5 - 0.5 * v * y * y);
}

template <typename T, int BITS, int NCH>
__global__ void __launch_bounds__(NCH == 1 || NCH == 2 ? 1024 : 512) mx_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ double part[32];
  if ((int)blockIdx.x >= p.row_ctas) {
    // scales of the rows behind the last one, to the end of its tile: code 0
    const int r = threadIdx.x & (MX_ROWS - 1);
    if (r < (int)(p.rows & (MX_ROWS - 1))) return;
    uint32_t* w = reinterpret_cast<uint32_t*>(p.scales + (p.rows / MX_ROWS) * p.col_tiles * MX_TILE_BYTES) + mx_tile_word(r);
    const int step = blockDim.x / MX_ROWS;   // a CTA has at least 128 threads
    for (int c = threadIdx.x / MX_ROWS; c < p.col_tiles && (int)threadIdx.x < step * MX_ROWS; c += step)
      w[c * (MX_TILE_BYTES / 4)] = 0u;
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rpb = blockDim.x / p.tpr;                       // rows per CTA
  const int sub = threadIdx.x / p.tpr, t = threadIdx.x - sub * p.tpr;
  const int64_t row = (int64_t)blockIdx.x * rpb + sub;
  const bool live = row < p.rows;
  const int64_t base = live ? row * p.d : 0;
  const T* x = static_cast<const T*>(p.x) + base;
  const T* r = p.r ? static_cast<const T*>(p.r) + base : nullptr;
  const int steps = NCH ? NCH : (p.col_tiles * 16 + p.tpr - 1) / p.tpr;
  float h[NCH ? NCH : 1][8];
  double total = 0.0;
#pragma unroll
  for (int k = 0; k < (NCH ? NCH : steps); ++k) {
    const int col = (k * p.tpr + t) * 8;
    float(&v)[8] = h[NCH ? k : 0];
    if (live && col < p.d) {
      load_h(x + col, r ? r + col : r, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
    const float a = fmaf(v[1], v[1], v[0] * v[0]), b = fmaf(v[3], v[3], v[2] * v[2]);
    const float c = fmaf(v[5], v[5], v[4] * v[4]), e = fmaf(v[7], v[7], v[6] * v[6]);
    total += (double)((a + b) + (c + e));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (p.tpr > 32) {
    if (lane == 0) part[warp] = total;
    __syncthreads();
    const int w0 = sub * (p.tpr >> 5);
    total = 0.0;
    for (int w = 0; w < (p.tpr >> 5); ++w) total += part[w0 + w];
  }
  const double rs64 = rsqrt64(total * p.inv_d + (double)p.eps);
  const float rs = (float)rs64;

  T* r_out = p.r_out ? static_cast<T*>(p.r_out) + base : nullptr;
  uint8_t* codes = p.codes + (live ? row : 0) * p.col_tiles * (MX_COLS * BITS / 8);
  uint8_t* scales = p.scales + (live ? row / MX_ROWS : 0) * p.col_tiles * MX_TILE_BYTES + 4 * mx_tile_word((int)(row % MX_ROWS));
#pragma unroll
  for (int k = 0; k < (NCH ? NCH : steps); ++k) {
    const int col = (k * p.tpr + t) * 8;
    float(&v)[8] = h[NCH ? k : 0];
    const bool in = live && col < p.d;
    float g[8], n[8], w[8];
    if constexpr (NCH == 0) {
      if (in) {
        load_h(x + col, r ? r + col : r, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      }
    }
    if (in) {
      load_gain(p, col, g);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = v[i] * rs * g[i];
    uint32_t top = mx_block_max(n);
    uint32_t code = mx_scale_code<BITS>(top);
    float inv = mx_inverse_scale(code);
    // Borders between codes, in the bits of w = n / scale: for e4m3 the middle
    // of the low 20 mantissa bits; for e2m1 the zero of the low 21 (the borders
    // of its least steps among them).  e4m3's subnormals, 2^-15 of the block's
    // largest and less, are left out.
    constexpr int SHIFT = BITS == 4 ? 11 : 12;
    constexpr uint32_t OFFSET = (BITS == 4 ? 4u : 4u - 0x80000u) << SHIFT;
    uint32_t near = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] = n[i] * inv;
      const uint32_t at = (__float_as_uint(w[i]) << SHIFT) + OFFSET;
      near = min(near, BITS == 4 && fabsf(w[i]) < 0.2f ? near : at);
    }
    const bool border = near <= (8u << SHIFT) || ((top + 4u) & 0x7FFFFFu) <= 8u;
    if (__any_sync(0xFFFFFFFFu, in && border && top != 0u)) {
      if (in) {
        double b[8];
        if (r) {   // the sum in fp64: this step's elements are not written yet
          float a[8];
          Vec8<T> q;
          q.load(x + col);
          q.get(a);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] = (double)a[i];
          q.load(r + col);
          q.get(a);
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] += (double)a[i];
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) b[i] = (double)v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) n[i] = to_odd(b[i] * rs64 * (double)g[i]);
      }
      top = mx_block_max(n);
      code = mx_scale_code<BITS>(top);
      inv = mx_inverse_scale(code);
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = n[i] * inv;
    }
    uint32_t out[BITS / 4];
    mx_element_codes<BITS>(w, code, out);
    const uint32_t word = mx_scale_word(code);
    if (in && r_out) store8(r_out + col, v);
    if (live && col < p.col_tiles * MX_COLS) {
      uint8_t* q = codes + col * BITS / 8;
      if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(q) = out[0];
      else *reinterpret_cast<uint2*>(q) = make_uint2(out[0], out[1]);
      if ((threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(scales + (col / MX_COLS) * MX_TILE_BYTES) = word;
    }
  }
}

template <typename T, int BITS>
oq_status norm_launch(const NormParams& p0, cudaStream_t st) {
  NormParams p = p0;
  int device = 0;
  const int sms = mx_sm_count(&device);
  const int chunks = p.col_tiles * 16;   // vectors of eight, padding included
  auto threads_for = [&](int n) { return ((chunks + n - 1) / n + 31) / 32 * 32; };
  // Vectors a thread holds.  Few rows: as many threads as a CTA takes, for the
  // least latency.  Otherwise the count of 2 to 8 that leaves the fewest idle
  // places, four at a tie (loads in flight against registers).
  int nch = 0;
  if (p.rows <= sms) {
    for (const int n : {1, 2, 3, 4, 5, 6, 7, 8})
      if (!nch && threads_for(n) <= (n <= 2 ? 1024 : 512)) nch = n;
  } else {
    for (const int n : {4, 3, 5, 2, 6, 7, 8})
      if (threads_for(n) <= 512 && (!nch || threads_for(n) * n < threads_for(nch) * nch)) nch = n;
  }
  p.tpr = nch ? threads_for(nch) : 512;
  const int rpb = (127 + p.tpr) / p.tpr, threads = p.tpr * rpb;
  const int64_t grid = (p.rows + rpb - 1) / rpb;
  p.row_ctas = (int)grid;
  const unsigned ctas = (unsigned)grid + (p.rows % MX_ROWS ? 1u : 0u);
#define OQ_NORM(N)                                                        \
  case N:                                                                 \
    mx_norm_kernel<T, BITS, N><<<ctas, threads, 0, st>>>(p);              \
    break
  switch (nch) {
    OQ_NORM(1);
    OQ_NORM(2);
    OQ_NORM(3);
    OQ_NORM(4);
    OQ_NORM(5);
    OQ_NORM(6);
    OQ_NORM(7);
    OQ_NORM(8);
    default:
      mx_norm_kernel<T, BITS, 0><<<ctas, threads, 0, st>>>(p);
  }
#undef OQ_NORM
  return launch_status("oq_rms_norm_mx");
}

}  // namespace

oq_status mx_quantize_launch(const void* x, int x_dtype, int64_t rows, int d, int bits, uint8_t* codes,
                             uint8_t* scales, void* stream) {
  const int ct = mx_col_tiles(d);
  const int64_t grid = mx_row_tiles(rows) * ct;
  if (grid > 0x7FFFFFFF) return OQ_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (x_dtype == OQ_DTYPE_BF16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(x);
    if (bits == 4) mx_quantize_kernel<__nv_bfloat16, 4><<<(unsigned)grid, QT, 0, st>>>(p, rows, d, ct, codes, scales);
    else mx_quantize_kernel<__nv_bfloat16, 8><<<(unsigned)grid, QT, 0, st>>>(p, rows, d, ct, codes, scales);
  } else {
    const float* p = static_cast<const float*>(x);
    if (bits == 4) mx_quantize_kernel<float, 4><<<(unsigned)grid, QT, 0, st>>>(p, rows, d, ct, codes, scales);
    else mx_quantize_kernel<float, 8><<<(unsigned)grid, QT, 0, st>>>(p, rows, d, ct, codes, scales);
  }
  return launch_status("oq_mx_quantize");
}

oq_status mx_dequantize_launch(const uint8_t* codes, const uint8_t* scales, int64_t rows, int d, int bits, void* x,
                               int x_dtype, void* stream) {
  const int ct = mx_col_tiles(d);
  const int64_t grid = mx_row_tiles(rows) * ct;
  if (grid > 0x7FFFFFFF) return OQ_ERR_UNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (x_dtype == OQ_DTYPE_BF16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(x);
    if (bits == 4) mx_dequantize_kernel<__nv_bfloat16, 4><<<(unsigned)grid, QT, 0, st>>>(codes, scales, rows, d, ct, p);
    else mx_dequantize_kernel<__nv_bfloat16, 8><<<(unsigned)grid, QT, 0, st>>>(codes, scales, rows, d, ct, p);
  } else {
    float* p = static_cast<float*>(x);
    if (bits == 4) mx_dequantize_kernel<float, 4><<<(unsigned)grid, QT, 0, st>>>(codes, scales, rows, d, ct, p);
    else mx_dequantize_kernel<float, 8><<<(unsigned)grid, QT, 0, st>>>(codes, scales, rows, d, ct, p);
  }
  return launch_status("oq_mx_dequantize");
}

oq_status mx_norm_launch(const MxNormArgs& a, void* stream) {
  NormParams p;
  p.x = a.x;
  p.r = a.residual;
  p.g = a.gain;
  p.g_bf16 = a.gain_dtype == OQ_DTYPE_BF16;
  p.eps = a.eps;
  p.inv_d = 1.0 / (double)a.d;
  p.rows = a.rows;
  p.d = a.d;
  p.col_tiles = mx_col_tiles(a.d);
  p.tpr = p.row_ctas = 0;
  p.r_out = a.residual_out;
  p.codes = a.codes;
  p.scales = a.scales;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.x_dtype == OQ_DTYPE_BF16)
    return a.bits == 4 ? norm_launch<__nv_bfloat16, 4>(p, st) : norm_launch<__nv_bfloat16, 8>(p, st);
  return a.bits == 4 ? norm_launch<float, 4>(p, st) : norm_launch<float, 8>(p, st);
}

}  // namespace oq
