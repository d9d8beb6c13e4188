// Microscaled quantisation of rows, its read-back, and the root-mean-square
// norm with the residual's addition whose output is quantised (formats and
// layouts: oq_mx.cuh).  All three are bound by HBM.
#include <cuda_bf16.h>

#include <algorithm>
#include <string>
#include <type_traits>

#include "oq_internal.h"
#include "oq_mx.cuh"

namespace oq {
namespace {

oq_status launch_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return OQ_OK;
  set_error(std::string(what) + " launch: " + cudaGetErrorString(e));
  return OQ_ERR_CUDA;
}

// ------------------------------------------------------------------ quantise
// A CTA owns one scale tile: 128 rows x 128 elements.  Sixteen lanes take a
// row of the tile, eight elements each, so a warp's loads cover two rows'
// 256-byte (bf16) segments; a thread loads its rows' vectors before it uses the
// first.  The tile's 512 scale bytes are gathered in shared memory
// and leave as whole sectors.  Rows past the end read as zeros and get scale
// code 0; columns past d get zero codes and scale code 0.  Bound by HBM: 32760 x
// 5120 bf16 in 4 bits 67 us, 6.4 TB/s (98 % of a copy's rate); a few tiles 2 us.
//
// 256 threads, or 512 with half as many rows each: where there are only a few
// tiles for an SM (bf16 in 4 bits, quantise / read back, 256 -> 512 threads: 200
// tiles 4.3 -> 3.7 / 3.4 -> 3.2 us, 600 tiles 7.0 -> 6.2 / 7.0 -> 6.2, 1200 tiles
// 10.8 -> 10.4 / 9.9 -> 10.3, 10240 tiles 66.4 -> 67.9 / 66.5 -> 68.1), and for
// quantising bf16 rows to 8 bits (5000 tiles 38.2 -> 37.4, 10240 75.0 -> 73.8).
constexpr int QT_WIDE = 512, QT_DEEP = 256;

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

// quantise: x -> codes, scales; read back: codes, scales -> x
struct QuantParams {
  void* x;
  int64_t rows;
  int d, col_tiles;
  uint8_t* codes;
  uint8_t* scales;
};

template <typename T, int BITS, int QT>
__global__ void __launch_bounds__(QT) mx_quantize_kernel(const __grid_constant__ QuantParams p) {
  constexpr int QSTEP = QT / 16, QROWS = MX_ROWS / QSTEP;   // rows between a thread's rows, and their number
  __shared__ uint32_t tile[MX_TILE_BYTES / 4];
  const int d = p.d, col_tiles = p.col_tiles;
  uint8_t* __restrict__ const codes = p.codes;
  uint8_t* __restrict__ const scales = p.scales;
  const TileSpan t = tile_span(p.rows, col_tiles);
  const bool in_cols = t.col < d;
  const T* __restrict__ const src = static_cast<const T*>(p.x) + t.row0 * d + t.col;
  dependency_wait();
  Vec8<T> in[QROWS];
  if (t.live >= MX_ROWS - t.sub && (t.ct + 1) * MX_COLS <= d) {   // a whole tile
#pragma unroll
    for (int i = 0; i < QROWS; ++i) in[i].load(src + (int64_t)i * QSTEP * d);
  } else {
#pragma unroll
    for (int i = 0; i < QROWS; ++i) {
      if (in_cols && i * QSTEP < t.live) in[i].load(src + (int64_t)i * QSTEP * d);
      else in[i].zero();
    }
  }
  const int pitch = col_tiles * (MX_COLS * BITS / 8);
  uint8_t* dst = codes + t.row0 * pitch + t.col * BITS / 8;
#pragma unroll
  for (int i = 0; i < QROWS; ++i) {
    f32x2 v2[4];
    float v[8];
    in[i].get(v2);
    unpack8(v2, v);
    const uint32_t code = mx_scale_code<BITS>(mx_block_max(v));
    const f32x2 inv = pack2(mx_inverse_scale(code), mx_inverse_scale(code));
#pragma unroll
    for (int k = 0; k < 4; ++k) v2[k] = mul2(v2[k], inv);
    unpack8(v2, v);
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
// 2^-127, a subnormal; code 255 is NaN.  Bound by HBM: 32760 x 5120 to bf16 66 us
// from 4 bits, 79 from 8 (6.4, 6.5 TB/s).
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

template <typename T, int BITS, int QT>
__global__ void __launch_bounds__(QT) mx_dequantize_kernel(const __grid_constant__ QuantParams p) {
  constexpr int QSTEP = QT / 16, QROWS = MX_ROWS / QSTEP;
  const int d = p.d, col_tiles = p.col_tiles;
  const uint8_t* __restrict__ const codes = p.codes;
  const uint8_t* __restrict__ const scales = p.scales;
  const TileSpan t = tile_span(p.rows, col_tiles);
  dependency_wait();
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
  T* __restrict__ const dst = static_cast<T*>(p.x) + t.row0 * d + t.col;
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
// r).  Two kernels:
//   - many rows (more than two an SM) of more than 1536 columns (which make a
//     CTA of 128 threads): CTAs stay and walk over rows, and every thread copies
//     its vectors of the next row into its own places in shared memory
//     (cp.async) while it works on this one.  Loads are then in flight all the
//     time without holding registers, and no barrier is about the data (32760 x
//     5120 bf16, residual kept: 195 us, 6.1 TB/s; 552 us with a CTA a row).
//   - other rows (few, narrow, or too long for two stages of shared memory): a
//     CTA a row, or as many as make 128 threads, straight from global memory
//     (32760 rows of 768 columns 61 us, 2.9 TB/s; of 1664, walked over, 73 us,
//     5.2).  NCH = 0 reads x and r a second time instead of keeping them (rows
//     too long for the registers).
// A thread re-reads only elements that it alone writes, so the kept residual may
// overwrite either input everywhere.
//
// Precision: eight squares are added in fp32 (four roundings deep), their sums
// and 1 / sqrt in fp64, so the factor is within 2^-23 of exact.  n is formed in
// fp32; it may be four ulps off, which matters only where an element lies that
// close to the border between two codes (or the block's largest to a power of
// two).  A warp that meets such an element (0.2 % of its steps) forms its
// elements again in fp64, rounded to fp32 towards the odd neighbour, from which
// the rounding to the element type is that of the fp64 value.
//
// All this holds while eps is at least NORM_EPS: then squares below 2^-126, and
// what they round off (2^-150 each), do not count beside it.  A smaller eps
// does not hide rows whose squares leave fp32's range; they are formed in fp64
// throughout (norm_row_far).  The walking kernel has a form of its own for that
// (FAR), because the looking costs every row: 195 us become 212, and a call
// in the loop would make them 254 by its registers.  So it marks such rows, by
// the scale code of their first block, and does them behind the loop.
constexpr size_t NORM_SMEM = 224 * 1024;   // stages of the streaming kernel
constexpr float NORM_EPS = 1e-35f;

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
__device__ __forceinline__ void load_h(const T* x, const T* r, f32x2 (&h)[4]) {
  Vec8<T> a;
  a.load(x);
  a.get(h);
  if (r) {
    f32x2 b[4];
    Vec8<T> c;
    c.load(r);
    c.get(b);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = add2(h[i], b[i]);
  }
}

__device__ __forceinline__ void load_gain(const NormParams& p, int col, f32x2 (&g)[4]) {
  if (!p.g) {
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = pack2(1.f, 1.f);
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
__device__ __forceinline__ bool near_rsqrt64(double v) { return v > 1e-36 && v < 1e36; }
__device__ __noinline__ double rsqrt64_far(double v) { return 1.0 / sqrt(v); }
__device__ __forceinline__ double rsqrt64(double v) {
  if (!near_rsqrt64(v)) return rsqrt64_far(v);
  float e;
  asm("rsqrt.approx.f32 %0, %1;" : "=f"(e) : "f"((float)v));   // 2 ulps: squared by the step
  const double y = (double)e, h = 0.5 * v;
  return y * fma(-h * y, y, 1.5);
}

// squares of one vector, added four roundings deep
__device__ __forceinline__ float sum_squares(const f32x2 (&v)[4]) {
  const f32x2 q = add2(fma2(v[1], v[1], mul2(v[0], v[0])), fma2(v[3], v[3], mul2(v[2], v[2])));
  float lo, hi;
  unpack2(q, lo, hi);
  return lo + hi;
}

// the row's sum over its `warps` warps (at most 32, w0 the first), in every thread of them
__device__ __forceinline__ double row_sum(double v, double* part, int warps, int w0) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (warps > 1) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < warps ? part[w0 + lane] : 0.0;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
      if (o < warps) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (warps > 1) v = __shfl_sync(0xFFFFFFFFu, v, 0);
  }
  return v;
}

// codes and scale of one vector from w = n / scale
template <int BITS>
__device__ __forceinline__ void norm_store(const float (&w)[8], uint32_t code, int col, bool in, bool own, uint8_t* codes,
                                           uint8_t* scales) {
  uint32_t out[BITS / 4];
  mx_element_codes<BITS>(w, in ? code : 255u, out);   // (255: zero elements)
  const uint32_t word = mx_scale_word(code);
  if (own) {
    uint8_t* q = codes + col * BITS / 8;
    if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(q) = out[0];
    else *reinterpret_cast<uint2*>(q) = make_uint2(out[0], out[1]);
    if ((threadIdx.x & 15) == 0) *reinterpret_cast<uint32_t*>(scales + (col >> 7) * MX_TILE_BYTES) = word;
  }
}

// The vector's codes formed in fp64 from x and r; every lane of the warp takes part.
template <typename T, int BITS>
__device__ __forceinline__ void norm_vector_exact(const NormParams& p, const T* x, const T* r, int col, bool in, bool own,
                                                  double rs64, uint8_t* codes, uint8_t* scales) {
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 0.f;
  if (in) {
    float a[8], c[8], g[8];
    f32x2 g2[4];
    Vec8<T> q;
    q.load(x);
    q.get(a);
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 0.f;
    if (r) {
      q.load(r);
      q.get(c);
    }
    load_gain(p, col, g2);
    unpack8(g2, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = to_odd(((double)a[i] + (double)c[i]) * rs64 * (double)g[i]);
  }
  const uint32_t code = mx_scale_code<BITS>(mx_block_max(w));
  const float inv = mx_inverse_scale(code);
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] *= inv;
  norm_store<BITS>(w, code, col, in, own, codes, scales);
}

// One vector of a row: its codes, its scale and the kept residual.  Every lane
// of the warp takes part.  `in`: the vector holds elements (v and g are
// anything, finite or not, where it does not: a block of 32 lies in or out as a
// whole, so nothing of it reaches another); `own`: it lies in the row's padded
// length.  True (in all lanes) where the warp met a border between codes and
// norm_vector_exact has to follow; with REDO it has, from x and r, before the
// kept residual is written, which may lie over them.
template <typename T, int BITS, bool REDO>
__device__ __forceinline__ bool norm_vector(const NormParams& p, const f32x2 (&v)[4], const f32x2 (&g)[4], const T* x,
                                            const T* r, int col, bool in, bool own, f32x2 rs2, double rs64, T* r_out,
                                            uint8_t* codes, uint8_t* scales) {
  f32x2 n[4];
  float w[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) n[i] = mul2(mul2(v[i], rs2), g[i]);
  unpack8(n, w);
  uint32_t top = mx_block_max(w);
  top = in ? top : 0u;
  const uint32_t code = mx_scale_code<BITS>(top);
  // where there are no elements everything becomes 0 * finite: w is masked below
  const float inv = in ? mx_inverse_scale(code) : 0.f;
  const f32x2 inv2 = pack2(inv, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) n[i] = mul2(n[i], inv2);
  unpack8(n, w);
  // Borders between codes, in the bits of w = n / scale: for e4m3 the middle of
  // the low 20 mantissa bits; for e2m1 the zero of the low 21 (the borders of
  // its least steps among them).  e4m3's subnormals, below 2^-14 of the block's
  // largest, are left out: they keep the codes of the fp32 n.
  constexpr int SHIFT = BITS == 4 ? 11 : 12;
  constexpr uint32_t OFFSET = (BITS == 4 ? 4u : 4u - 0x80000u) << SHIFT;
  uint32_t near = 0xFFFFFFFFu;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    uint32_t at[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      at[j] = (__float_as_uint(w[i + j]) << SHIFT) + OFFSET;
      if (BITS == 4 && fabsf(w[i + j]) < 0.2f) at[j] = 0xFFFFFFFFu;
    }
    near = __vimin3_u32(near, at[0], at[1]);
  }
  const bool border = top != 0u && (near <= (8u << SHIFT) || ((top + 4u) & 0x7FFFFFu) <= 8u);
  const bool any = __any_sync(0xFFFFFFFFu, border);
  if (REDO && any) norm_vector_exact<T, BITS>(p, x, r, col, in, own, rs64, codes, scales);
  else norm_store<BITS>(w, code, col, in, own, codes, scales);
  if (in && r_out) {
    float f[8];
    unpack8(v, f);
    store8(r_out + col, f);
  }
  return any;
}

// A row whose mean square is far (a root mean square below 1e-18 under an eps as
// small, or above 1e18), all of it in fp64.  A thread reads and writes its own
// vectors (t, t + tpr, ...).  All threads of the row call it; they meet at
// barrier `bar`, because other rows of the CTA may not come this way.  Out of
// line: it is rare, and its registers would be every row's.
template <typename T, int BITS>
__device__ __noinline__ void norm_row_far(const NormParams& p, const T* x, const T* r, T* r_out, uint8_t* codes,
                                          uint8_t* scales, int t, int tpr, double* part, int w0, int bar) {
  double v = 0.0;
  for (int col = t * 8; col < p.d; col += tpr * 8) {
    for (int i = 0; i < 8; ++i) {
      double h = (double)(float)x[col + i];
      if (r) h += (double)(float)r[col + i];
      v += h * h;
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = tpr >> 5, lane = threadIdx.x & 31;
  if (warps > 1) {
    // (once all have read what part held)
    asm volatile("barrier.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
    if (lane == 0) part[threadIdx.x >> 5] = v;
    asm volatile("barrier.sync %0, %1;" ::"r"(bar), "r"(tpr) : "memory");
    v = 0.0;
    for (int w = 0; w < warps; ++w) v += part[w0 + w];
  }
  const double rs64 = 1.0 / sqrt(v * p.inv_d + (double)p.eps);
  const int cols = p.col_tiles * MX_COLS;
  for (int c0 = (t - lane) * 8; c0 < cols; c0 += tpr * 8) {   // a warp's vectors together
    const int col = c0 + lane * 8;
    const bool in = col < p.d;
    norm_vector_exact<T, BITS>(p, x + col, r ? r + col : r, col, in, col < cols, rs64, codes, scales);
    if (in && r_out) {
      f32x2 h[4];
      float f[8];
      load_h(x + col, r ? r + col : r, h);
      unpack8(h, f);
      store8(r_out + col, f);
    }
  }
}

// scales of the rows behind the last one, to the end of its tile: code 0 (one
// CTA of at least 128 threads)
__device__ __forceinline__ void norm_clear_padding(const NormParams& p) {
  const int r = threadIdx.x & (MX_ROWS - 1), step = blockDim.x / MX_ROWS;
  if (r < (int)(p.rows & (MX_ROWS - 1))) return;
  uint32_t* w = reinterpret_cast<uint32_t*>(p.scales + (p.rows / MX_ROWS) * p.col_tiles * MX_TILE_BYTES) + mx_tile_word(r);
  for (int c = threadIdx.x / MX_ROWS; c < p.col_tiles && (int)threadIdx.x < step * MX_ROWS; c += step)
    w[c * (MX_TILE_BYTES / 4)] = 0u;
}

template <typename T, int BITS, int NCH>
__global__ void __launch_bounds__(NCH == 1 || NCH == 2 ? 1024 : 512) mx_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ double part[32];
  dependency_wait();
  if ((int)blockIdx.x >= p.row_ctas) {
    norm_clear_padding(p);
    return;
  }
  const int rpb = blockDim.x / p.tpr;                       // rows per CTA
  const int sub = threadIdx.x / p.tpr, t = threadIdx.x - sub * p.tpr;
  const int64_t row = (int64_t)blockIdx.x * rpb + sub;
  const bool live = row < p.rows;
  const int64_t base = live ? row * p.d : 0;
  const T* x = static_cast<const T*>(p.x) + base;
  const T* r = p.r ? static_cast<const T*>(p.r) + base : nullptr;
  const int steps = NCH ? NCH : (p.col_tiles * 16 + p.tpr - 1) / p.tpr;
  f32x2 h[NCH ? NCH : 1][4];
  double total = 0.0;
  auto load = [&](int col, f32x2(&v)[4]) {
    if (live && col < p.d) {
      load_h(x + col, r ? r + col : r, v);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = 0ull;
    }
  };
#pragma unroll
  for (int k = 0; k < (NCH ? NCH : steps); ++k) {
    load((k * p.tpr + t) * 8, h[NCH ? k : 0]);
    total += (double)sum_squares(h[NCH ? k : 0]);
  }
  const double mean = row_sum(total, part, p.tpr >> 5, sub * (p.tpr >> 5)) * p.inv_d + (double)p.eps;
  T* r_out = p.r_out ? static_cast<T*>(p.r_out) + base : nullptr;
  uint8_t* codes = p.codes + (live ? row : 0) * p.col_tiles * (MX_COLS * BITS / 8);
  uint8_t* scales = p.scales + (live ? row / MX_ROWS : 0) * p.col_tiles * MX_TILE_BYTES + 4 * mx_tile_word((int)(row % MX_ROWS));
  if (!near_rsqrt64(mean)) {   // the same in all threads of a row
    if (live) norm_row_far<T, BITS>(p, x, r, r_out, codes, scales, t, p.tpr, part, sub * (p.tpr >> 5), 1 + sub);
    return;
  }
  const double rs64 = rsqrt64(mean);
  const f32x2 rs2 = pack2((float)rs64, (float)rs64);
#pragma unroll
  for (int k = 0; k < (NCH ? NCH : steps); ++k) {
    const int col = (k * p.tpr + t) * 8;
    if constexpr (NCH == 0) load(col, h[0]);
    f32x2 g[4];
    load_gain(p, col < p.d ? col : 0, g);
    norm_vector<T, BITS, true>(p, h[NCH ? k : 0], g, x + col, r ? r + col : r, col, live && col < p.d,
                         live && col < p.col_tiles * MX_COLS, rs2, rs64, r_out, codes, scales);
  }
}

__device__ __forceinline__ void copy_async16(void* dst_smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst_smem)), "l"(src)
               : "memory");
}

constexpr uint8_t FAR_ROW = 254;   // no block has it: scale codes end at 252

template <typename T, int BITS, int NCH, bool RES, bool FAR>
__global__ void __launch_bounds__(1024, 1) mx_norm_stream_kernel(const __grid_constant__ NormParams p) {
  __shared__ double part[2][32];
  __shared__ int far_rows;   // FAR: this CTA has marked some (written before a barrier of the first row, and after)
  extern __shared__ __align__(16) unsigned char stage_mem[];
  dependency_wait();
  if ((int)blockIdx.x >= p.row_ctas) {
    norm_clear_padding(p);
    return;
  }
  constexpr int VB = 8 * (int)sizeof(T);   // bytes of a vector
  const int t = threadIdx.x, tpr = blockDim.x;
  // a stage: the row's vectors of x, then of r; a thread uses its own places only
  const int plane = p.d * (int)sizeof(T), stage = RES ? 2 * plane : plane;
  const int cols = p.col_tiles * MX_COLS;
  const int64_t step = (int64_t)p.row_ctas * p.d;
  // this thread's columns; one without elements reads the row's first vector and drops it
  int at[NCH];
  bool in[NCH];
  f32x2 gain[NCH == 2 ? 2 : 1][4];   // its gain, kept where the registers allow it
#pragma unroll
  for (int k = 0; k < NCH; ++k) {
    const int col = (k * tpr + t) * 8;
    in[k] = col < p.d;
    at[k] = in[k] ? col : 0;
    if constexpr (NCH == 2) load_gain(p, at[k], gain[k]);
  }
  const T* x_next = static_cast<const T*>(p.x) + (int64_t)blockIdx.x * p.d;   // the next row to fetch
  const T* r_next = RES ? static_cast<const T*>(p.r) + (int64_t)blockIdx.x * p.d : nullptr;
  auto fetch = [&](bool there, unsigned char* to) {
    if (there) {
#pragma unroll
      for (int k = 0; k < NCH; ++k) {
        if (in[k]) {
          unsigned char* q = to + at[k] * (int)sizeof(T);
#pragma unroll
          for (int b = 0; b < VB; b += 16) {
            copy_async16(q + b, reinterpret_cast<const unsigned char*>(x_next + at[k]) + b);
            if constexpr (RES) copy_async16(q + plane + b, reinterpret_cast<const unsigned char*>(r_next + at[k]) + b);
          }
        }
      }
      x_next += step;
      if constexpr (RES) r_next += step;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (FAR && t == 0) far_rows = 0;
  int s = 0;
  fetch(true, stage_mem);
  T* r_out = RES && p.r_out ? static_cast<T*>(p.r_out) + (int64_t)blockIdx.x * p.d : nullptr;
  for (int64_t row = blockIdx.x; row < p.rows; row += p.row_ctas, s ^= 1) {
    fetch(row + p.row_ctas < p.rows, stage_mem + (s ^ 1) * stage);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const T* q = reinterpret_cast<const T*>(stage_mem + s * stage);
    const T* qr = RES ? reinterpret_cast<const T*>(stage_mem + s * stage + plane) : nullptr;
    f32x2 h[NCH][4];
    double total = 0.0;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      load_h(q + at[k], RES ? qr + at[k] : nullptr, h[k]);
      const float sq = sum_squares(h[k]);
      total += in[k] ? (double)sq : 0.0;
    }
    const double mean = row_sum(total, part[s], tpr >> 5, 0) * p.inv_d + (double)p.eps;
    const bool far = FAR && !near_rsqrt64(mean);   // the same in all threads
    const double rs64 = rsqrt64(mean);
    const f32x2 rs2 = pack2((float)rs64, (float)rs64);
    uint8_t* codes = p.codes + row * (cols * BITS / 8);
    uint8_t* scales = p.scales + (row >> 7) * (p.col_tiles * MX_TILE_BYTES) + 4 * mx_tile_word((int)row & (MX_ROWS - 1));
    uint32_t redo = 0u;
#pragma unroll
    for (int k = 0; k < NCH; ++k) {
      const int col = (k * tpr + t) * 8;
      f32x2 g[4];
      if constexpr (NCH != 2) load_gain(p, at[k], g);
      if (norm_vector<T, BITS, false>(p, h[k], NCH == 2 ? gain[k % 2] : g, nullptr, nullptr, col, in[k], col < cols, rs2, rs64,
                                      far ? nullptr : r_out, codes, scales))
        redo |= 1u << k;
    }
    // the warp's vectors next to a border, again from the stage, which nothing
    // has overwritten (apart from the loop above: its registers are the speed)
    if (redo) {
#pragma unroll 1
      for (int k = 0; k < NCH; ++k) {
        const int col = (k * tpr + t) * 8;
        if (redo >> k & 1u)
          norm_vector_exact<T, BITS>(p, q + col, RES ? qr + col : nullptr, col, col < p.d, col < cols, rs64, codes, scales);
      }
    }
    if (r_out) r_out += step;
    if (far && t == 0) {   // (what the loop made of the row is overwritten)
      *scales = FAR_ROW;
      far_rows = 1;
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if constexpr (FAR) {
    __syncthreads();   // far_rows and the marks
    if (!far_rows) return;
    for (int64_t row = blockIdx.x; row < p.rows; row += p.row_ctas) {
      uint8_t* scales = p.scales + (row >> 7) * (p.col_tiles * MX_TILE_BYTES) + 4 * mx_tile_word((int)row & (MX_ROWS - 1));
      const bool marked = *scales == FAR_ROW;
      __syncthreads();   // read by all before it is overwritten; part is free again
      if (marked)
        norm_row_far<T, BITS>(p, static_cast<const T*>(p.x) + row * p.d, RES ? static_cast<const T*>(p.r) + row * p.d : nullptr,
                              RES && p.r_out ? static_cast<T*>(p.r_out) + row * p.d : nullptr,
                              p.codes + row * (cols * BITS / 8), scales, t, tpr, part[0], 0, 1);
    }
  }
}

template <typename T, int BITS, int NCH, bool RES>
oq_status norm_stream_launch(NormParams& p, int threads, int sms, int device, size_t smem, cudaStream_t st) {
  static std::atomic<uint64_t> smem_set[2] = {};
  const bool far = p.eps < NORM_EPS;
  auto kernel = far ? mx_norm_stream_kernel<T, BITS, NCH, RES, true> : mx_norm_stream_kernel<T, BITS, NCH, RES, false>;
  const oq_status ok = mx_allow_smem(reinterpret_cast<const void*>(kernel), NORM_SMEM, device, &smem_set[far]);
  if (ok != OQ_OK) return ok;
  // CTAs an SM holds: 64 registers a thread, 228 KB of shared memory with 1 KB a CTA of the system's and 512 bytes of sums
  const int resident = std::max(1, std::min(1024 / threads, (int)(228 * 1024 / (smem + 1024 + 512))));
  p.row_ctas = (int)std::min<int64_t>(p.rows, (int64_t)sms * resident);
  const unsigned grid = (unsigned)p.row_ctas + (p.rows % MX_ROWS ? 1u : 0u);
  return launch_status(mx_launch(kernel, dim3(grid), threads, smem, 0, st, p), "oq_rms_norm_mx");
}

template <typename T, int BITS>
oq_status norm_launch(const NormParams& p0, cudaStream_t st) {
  NormParams p = p0;
  int device = 0;
  const int sms = mx_sm_count(&device);
  const int chunks = p.col_tiles * 16;   // vectors of eight, padding included
  auto threads_for = [&](int n) { return ((chunks + n - 1) / n + 31) / 32 * 32; };
  // the streaming kernel, where there are rows enough to walk over
  if (p.rows > 2 * sms) {
    // Two vectors a thread, whose gains then stay in registers, where a CTA's
    // threads allow it; four for longer rows (12288 wide: 72.5 us with two, 76
    // with four).
    const int nch = threads_for(2) <= 1024 ? 2 : 4;
    const int threads = threads_for(nch);
    const size_t smem = (size_t)2 * p.d * sizeof(T) * (p.r ? 2 : 1);
    if (threads >= 128 && threads <= 1024 && smem <= NORM_SMEM) {
      if (nch == 2)
        return p.r ? norm_stream_launch<T, BITS, 2, true>(p, threads, sms, device, smem, st)
                   : norm_stream_launch<T, BITS, 2, false>(p, threads, sms, device, smem, st);
      if (!p.r) return norm_stream_launch<T, BITS, 4, false>(p, threads, sms, device, smem, st);
      // (fp32 rows that long have no room for two stages of x and r)
      if constexpr (sizeof(T) == 2) return norm_stream_launch<T, BITS, 4, true>(p, threads, sms, device, smem, st);
    }
  }
  // A CTA a row: as many threads as fit, for the least latency
  const int nch = threads_for(1) <= 1024 ? 1 : threads_for(2) <= 1024 ? 2 : threads_for(8) <= 512 ? 8 : 0;
  p.tpr = nch ? threads_for(nch) : 512;
  const int rpb = (127 + p.tpr) / p.tpr, threads = p.tpr * rpb;
  const int64_t grid = (p.rows + rpb - 1) / rpb;
  p.row_ctas = (int)grid;
  const unsigned ctas = (unsigned)grid + (p.rows % MX_ROWS ? 1u : 0u);
  auto kernel = nch == 1   ? mx_norm_kernel<T, BITS, 1>
                : nch == 2 ? mx_norm_kernel<T, BITS, 2>
                : nch == 8 ? mx_norm_kernel<T, BITS, 8>
                           : mx_norm_kernel<T, BITS, 0>;
  return launch_status(mx_launch(kernel, dim3(ctas), threads, 0, 0, st, p), "oq_rms_norm_mx");
}

bool few_tiles(int64_t tiles) {
  int device = 0;
  return tiles <= 4 * mx_sm_count(&device);
}

}  // namespace

oq_status mx_quantize_launch(const void* x, int x_dtype, int64_t rows, int d, int bits, uint8_t* codes,
                             uint8_t* scales, void* stream) {
  const QuantParams p{const_cast<void*>(x), rows, d, mx_col_tiles(d), codes, scales};
  const int64_t grid = mx_row_tiles(rows) * p.col_tiles;
  if (grid > 0x7FFFFFFF) return OQ_ERR_UNSUPPORTED;
  const bool bf16 = x_dtype == OQ_DTYPE_BF16, wide = few_tiles(grid) || (bf16 && bits == 8);
  auto pick = [&](auto threads) {
    constexpr int QT = decltype(threads)::value;
    return bf16 ? (bits == 4 ? mx_quantize_kernel<__nv_bfloat16, 4, QT> : mx_quantize_kernel<__nv_bfloat16, 8, QT_WIDE>)
                : (bits == 4 ? mx_quantize_kernel<float, 4, QT> : mx_quantize_kernel<float, 8, QT>);
  };
  auto kernel = wide ? pick(std::integral_constant<int, QT_WIDE>()) : pick(std::integral_constant<int, QT_DEEP>());
  return launch_status(mx_launch(kernel, dim3((unsigned)grid), wide ? QT_WIDE : QT_DEEP, 0, 0, static_cast<cudaStream_t>(stream), p),
                       "oq_mx_quantize");
}

oq_status mx_dequantize_launch(const uint8_t* codes, const uint8_t* scales, int64_t rows, int d, int bits, void* x,
                               int x_dtype, void* stream) {
  const QuantParams p{x, rows, d, mx_col_tiles(d), const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales)};
  const int64_t grid = mx_row_tiles(rows) * p.col_tiles;
  if (grid > 0x7FFFFFFF) return OQ_ERR_UNSUPPORTED;
  const bool bf16 = x_dtype == OQ_DTYPE_BF16, wide = few_tiles(grid);
  auto pick = [&](auto threads) {
    constexpr int QT = decltype(threads)::value;
    return bf16 ? (bits == 4 ? mx_dequantize_kernel<__nv_bfloat16, 4, QT> : mx_dequantize_kernel<__nv_bfloat16, 8, QT>)
                : (bits == 4 ? mx_dequantize_kernel<float, 4, QT> : mx_dequantize_kernel<float, 8, QT>);
  };
  auto kernel = wide ? pick(std::integral_constant<int, QT_WIDE>()) : pick(std::integral_constant<int, QT_DEEP>());
  return launch_status(mx_launch(kernel, dim3((unsigned)grid), wide ? QT_WIDE : QT_DEEP, 0, 0, static_cast<cudaStream_t>(stream), p),
                       "oq_mx_dequantize");
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
