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
constexpr int QROWS = MX_ROWS * 16 / QT;   // rows per thread

template <typename T, int BITS>
__global__ void __launch_bounds__(QT) mx_quantize_kernel(const T* __restrict__ x, int64_t rows, int d, int col_tiles,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  __shared__ uint32_t tile[MX_TILE_BYTES / 4];
  const int64_t rt = blockIdx.x / col_tiles;
  const int ct = (int)(blockIdx.x - rt * col_tiles);
  const int sub = threadIdx.x >> 4, col = ct * MX_COLS + (threadIdx.x & 15) * 8;
  const int64_t row0 = rt * MX_ROWS + sub;
  constexpr int STEP = QT / 16;
  Vec8<T> in[QROWS];
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    const int64_t row = row0 + i * STEP;
    if (row < rows && col < d) in[i].load(x + row * d + col);
    else in[i].zero();
  }
  const int64_t pitch = (int64_t)col_tiles * (MX_COLS * BITS / 8);
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    float v[8];
    in[i].get(v);
    uint32_t out[BITS / 4];
    const uint32_t word = mx_scale_word(mx_quantize8<BITS>(v, out));
    const int64_t row = row0 + i * STEP;
    if (row < rows) {
      uint32_t* dst = reinterpret_cast<uint32_t*>(codes + row * pitch + (int64_t)col * BITS / 8);
      if constexpr (BITS == 4) *dst = out[0];
      else *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    }
    if ((threadIdx.x & 15) == 0) tile[mx_tile_word(sub + i * STEP)] = word;
  }
  __syncthreads();
  if (threadIdx.x < MX_TILE_BYTES / 16)
    reinterpret_cast<uint4*>(scales + (int64_t)blockIdx.x * MX_TILE_BYTES)[threadIdx.x] =
        reinterpret_cast<const uint4*>(tile)[threadIdx.x];
}

// ------------------------------------------------------------------ read-back
// The same tiles: value = element * 2^(scale code - 127).  Scale code 0 is
// 2^-127, a subnormal fp32; code 255 is NaN.
__device__ __forceinline__ float mx_scale_value(uint32_t code) {
  return code == 255u ? __uint_as_float(0x7FFFFFFFu) : code == 0u ? __uint_as_float(1u << 22) : __uint_as_float(code << 23);
}

// the eight e2m1 values of a word of codes
__device__ __forceinline__ void e2m1_values(uint32_t w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t c = (w >> (4 * i)) & 15u;
    // magnitudes 0..7 in eighths of 0.5 steps: a byte table of 2 |value|
    const uint32_t twice = (uint32_t)(0x0C08060403020100ull >> (8 * (c & 7u))) & 0xFFu;
    const float m = 0.5f * (float)twice;
    v[i] = (c & 8u) ? -m : m;
  }
}
__device__ __forceinline__ float e4m3_value(uint32_t c) {
  // exponent 0: m 2^-9; else (8 + m) 2^(e - 10); 0x7F is NaN
  const uint32_t e = (c >> 3) & 15u, m = c & 7u;
  float v = e == 0u ? (float)m * 0x1p-9f : __uint_as_float(((e + 120u) << 23) | (m << 20));
  if ((c & 0x7Fu) == 0x7Fu) v = __uint_as_float(0x7FFFFFFFu);
  return (c & 0x80u) ? -v : v;
}

template <typename T, int BITS>
__global__ void __launch_bounds__(QT) mx_dequantize_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t rows, int d,
                                                           int col_tiles, T* __restrict__ x) {
  const int64_t rt = blockIdx.x / col_tiles;
  const int ct = (int)(blockIdx.x - rt * col_tiles);
  const int sub = threadIdx.x >> 4, col = ct * MX_COLS + (threadIdx.x & 15) * 8;
  if (col >= d) return;
  const int64_t row0 = rt * MX_ROWS + sub;
  constexpr int STEP = QT / 16;
  const int64_t pitch = (int64_t)col_tiles * (MX_COLS * BITS / 8);
  uint32_t in[QROWS][BITS / 4], sc[QROWS];
  const uint8_t* tile = scales + (int64_t)blockIdx.x * MX_TILE_BYTES + ((threadIdx.x >> 2) & 3);
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    const int64_t row = row0 + i * STEP;
    if (row < rows) {
      const uint32_t* src = reinterpret_cast<const uint32_t*>(codes + row * pitch + (int64_t)col * BITS / 8);
      if constexpr (BITS == 4) {
        in[i][0] = *src;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(src);
        in[i][0] = u.x;
        in[i][1] = u.y;
      }
      sc[i] = tile[4 * mx_tile_word(sub + i * STEP)];
    }
  }
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    const int64_t row = row0 + i * STEP;
    if (row >= rows) break;
    float v[8];
    if constexpr (BITS == 4) {
      e2m1_values(in[i][0], v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = e4m3_value((in[i][k >> 2] >> (8 * (k & 3))) & 0xFFu);
    }
    const float s = mx_scale_value(sc[i]);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= s;
    store8(x + row * d + col, v);
  }
}

// ------------------------------------------------------------------ norm
// h = x + r in fp32; the kept residual is h rounded to the input's type;
// n = h * (1 / sqrt(mean(h^2) + eps)) * g from the unrounded h, in fp32.
// TPR threads own a row, each NCH vectors of eight neighbouring elements that
// stay in registers between the sum and the quantisation (one pass over x and
// r).  NCH = 0 reads x and r a second time instead (rows too long for the
// registers): each thread re-reads only elements that it alone writes, so the
// kept residual may overwrite either input in both forms.
struct NormParams {
  const void* x;
  const void* r;
  const void* g;
  bool g_bf16;
  float eps, inv_d;
  int64_t rows;
  int d, col_tiles, tpr;
  void* r_out;
  uint8_t* codes;
  uint8_t* scales;
};

template <typename T>
__device__ __forceinline__ void load_h(const NormParams& p, int64_t off, float (&h)[8]) {
  Vec8<T> a;
  a.load(static_cast<const T*>(p.x) + off);
  a.get(h);
  if (p.r) {
    float b[8];
    Vec8<T> c;
    c.load(static_cast<const T*>(p.r) + off);
    c.get(b);
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] += b[i];
  }
}

template <typename T, int BITS>
__device__ __forceinline__ void norm_emit(const NormParams& p, int64_t row, int col, float rs, float (&h)[8], bool in) {
  if (in) {
    if (p.r_out) store8(static_cast<T*>(p.r_out) + row * p.d + col, h);
    float g[8];
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
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = h[i] * rs * g[i];
  }
  uint32_t out[BITS / 4];
  const uint32_t word = mx_scale_word(mx_quantize8<BITS>(h, out));
  if (row < p.rows && col < p.col_tiles * MX_COLS) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.codes + (row * p.col_tiles * MX_COLS + col) * BITS / 8);
    if constexpr (BITS == 4) *dst = out[0];
    else *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
    if ((threadIdx.x & 15) == 0)
      reinterpret_cast<uint32_t*>(p.scales + ((row / MX_ROWS) * p.col_tiles + col / MX_COLS) * MX_TILE_BYTES)
          [mx_tile_word((int)(row % MX_ROWS))] = word;
  }
}

template <typename T, int BITS, int NCH>
__global__ void __launch_bounds__(512) mx_norm_kernel(const NormParams p) {
  __shared__ float part[16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rpb = blockDim.x / p.tpr;                       // rows per CTA
  const int sub = threadIdx.x / p.tpr, t = threadIdx.x - sub * p.tpr;
  const int64_t row = (int64_t)blockIdx.x * rpb + sub;
  const bool live = row < p.rows;
  const int steps = NCH ? NCH : (p.col_tiles * 16 + p.tpr - 1) / p.tpr;
  float h[NCH ? NCH : 1][8];
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < (NCH ? NCH : steps); ++k) {
    const int col = (k * p.tpr + t) * 8;
    float(&v)[8] = h[NCH ? k : 0];
    if (live && col < p.d) {
      load_h<T>(p, row * p.d + col, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(v[i], v[i], sum);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (p.tpr > 32) {
    if (lane == 0) part[warp] = sum;
    __syncthreads();
    const int w0 = sub * (p.tpr >> 5);
    sum = 0.f;
    for (int w = 0; w < (p.tpr >> 5); ++w) sum += part[w0 + w];
  }
  const float rs = 1.f / sqrtf(fmaf(sum, p.inv_d, p.eps));
#pragma unroll
  for (int k = 0; k < (NCH ? NCH : steps); ++k) {
    const int col = (k * p.tpr + t) * 8;
    float(&v)[8] = h[NCH ? k : 0];
    const bool in = live && col < p.d;
    if constexpr (NCH == 0) {
      if (in) {
        load_h<T>(p, row * p.d + col, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
      }
    }
    norm_emit<T, BITS>(p, row, col, rs, v, in);
  }
  // scales of the rows behind the last one, to the end of its tile: code 0
  if (blockIdx.x == gridDim.x - 1) {
    const int64_t end = mx_row_tiles(p.rows) * MX_ROWS;
    for (int64_t i = threadIdx.x; i < (end - p.rows) * p.col_tiles; i += blockDim.x) {
      const int64_t r = p.rows + i / p.col_tiles;
      const int c = (int)(i % p.col_tiles);
      reinterpret_cast<uint32_t*>(p.scales + ((r / MX_ROWS) * p.col_tiles + c) * MX_TILE_BYTES)
          [mx_tile_word((int)(r % MX_ROWS))] = 0u;
    }
  }
}

template <typename T, int BITS>
oq_status norm_launch(const NormParams& p0, cudaStream_t st) {
  NormParams p = p0;
  const int chunks = p.col_tiles * 16;   // vectors of eight, padding included
  // threads per row: at most four vectors a thread up to 128 threads, then
  // eight (registers), then the re-reading form
  p.tpr = 32;
  while (p.tpr < 512 && p.tpr * 4 < chunks) p.tpr *= 2;
  const int nch = (chunks + p.tpr - 1) / p.tpr;
  const int threads = std::max(p.tpr, 128), rpb = threads / p.tpr;
  const int64_t grid = (p.rows + rpb - 1) / rpb;
#define OQ_NORM(N)                                                            \
  case N:                                                                     \
    mx_norm_kernel<T, BITS, N><<<(unsigned)grid, threads, 0, st>>>(p);        \
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
      mx_norm_kernel<T, BITS, 0><<<(unsigned)grid, threads, 0, st>>>(p);
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
  p.inv_d = 1.f / (float)a.d;
  p.rows = a.rows;
  p.d = a.d;
  p.col_tiles = mx_col_tiles(a.d);
  p.tpr = 0;
  p.r_out = a.residual_out;
  p.codes = a.codes;
  p.scales = a.scales;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (a.x_dtype == OQ_DTYPE_BF16)
    return a.bits == 4 ? norm_launch<__nv_bfloat16, 4>(p, st) : norm_launch<__nv_bfloat16, 8>(p, st);
  return a.bits == 4 ? norm_launch<float, 4>(p, st) : norm_launch<float, 8>(p, st);
}

}  // namespace oq
