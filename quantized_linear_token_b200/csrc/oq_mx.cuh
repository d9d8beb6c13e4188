// Microscaled formats (OCP Microscaling Formats v1.0): blocks of 32 elements
// along a row share one power-of-two scale.
//   element  e2m1 (4 bits: +-{0, .5, 1, 1.5, 2, 3, 4, 6}) or e4m3 (8 bits, to 448)
//   scale    E8M0: code c stands for 2^(c - 127), 255 for NaN
// Rows are padded with zero codes to a multiple of 128 elements.  Scales are
// stored in tiles of 128 rows x 4 blocks (512 bytes), the order in which the
// tensor cores take them: byte [row / 128][block / 4][row % 32][row / 32 % 4][block % 4].
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "oq_internal.h"

namespace oq {

constexpr int MX_BLOCK = 32;       // elements per scale
constexpr int MX_COLS = 128;       // elements per scale tile and row padding
constexpr int MX_ROWS = 128;       // rows per scale tile
constexpr int MX_TILE_BYTES = 512;

__host__ __device__ inline int mx_col_tiles(int d) { return (d + MX_COLS - 1) / MX_COLS; }
__host__ __device__ inline int64_t mx_row_tiles(int64_t rows) { return (rows + MX_ROWS - 1) / MX_ROWS; }
__host__ __device__ inline int64_t mx_row_bytes(int d, int bits) { return (int64_t)mx_col_tiles(d) * (MX_COLS * bits / 8); }

// 32-bit word of a scale tile that holds row r's four block scales
__device__ __forceinline__ int mx_tile_word(int r) { return (r & 31) * 4 + ((r >> 5) & 3); }

// Pairs of fp32 in one 64-bit register: one instruction does both
// (round to nearest, as the scalar forms).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void unpack8(const f32x2 (&a)[4], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(a[i], v[2 * i], v[2 * i + 1]);
}

// Eight consecutive row elements in fp32: one 16-byte load of bf16, two of fp32.
template <typename T>
struct Vec8;
template <>
struct Vec8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ void get(f32x2 (&v)[4]) const {
    float f[8];
    get(f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void get(f32x2 (&v)[4]) const {
    v[0] = pack2(a.x, a.y), v[1] = pack2(a.z, a.w);
    v[2] = pack2(b.x, b.y), v[3] = pack2(b.z, b.w);
  }
};

__device__ __forceinline__ uint32_t mx_pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(mx_pack_bf16(v[0], v[1]), mx_pack_bf16(v[2], v[3]),
                                            mx_pack_bf16(v[4], v[5]), mx_pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// eight fp32 -> eight e2m1 codes (round to nearest even, saturating at 6), element 0 in the low nibble
__device__ __forceinline__ uint32_t cvt8_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}
// four fp32 -> four e4m3 codes (round to nearest even, saturating at 448)
__device__ __forceinline__ uint32_t cvt4_e4m3(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// |a|, |b|, |c|: the largest, NaN if one of them is
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Largest magnitude of a block of 32 elements, eight in each of four
// neighbouring lanes, as fp32 bits (a NaN or an infinity on top); every lane of
// the warp takes part.
__device__ __forceinline__ uint32_t mx_block_max(const float (&v)[8]) {
  const float m8 = max3_abs_nan(max3_abs_nan(v[0], v[1], v[2]), max3_abs_nan(v[3], v[4], v[5]), max3_abs_nan(v[6], v[7], 0.f));
  uint32_t m = __float_as_uint(m8);   // not negative: ordered as integers
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
}

// Its scale code: scale = 2^(floor(log2 max) - emax), emax 2 (e2m1) or 8
// (e4m3), is the biased exponent of the largest magnitude less emax, not below
// 0; 255 for a block with an infinity or a NaN.
template <int BITS>
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t block_max) {
  const int e = (int)(block_max >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - (BITS == 4 ? 2 : 8), 0);
}

// 1 / scale = 2^(127 - code), a normal number for every code below 255
__device__ __forceinline__ float mx_inverse_scale(uint32_t code) { return __uint_as_float((254u - min(code, 254u)) << 23); }

// Element codes of w = v / scale.  The products are exact except below 2^-126,
// where the elements round to zero either way, so the only rounding is the one
// to the element type.  A NaN block gets zero elements (its scale says NaN).
template <int BITS>
__device__ __forceinline__ void mx_element_codes(const float (&w)[8], uint32_t code, uint32_t (&out)[BITS / 4]) {
  if constexpr (BITS == 4) {
    out[0] = cvt8_e2m1(w);
  } else {
    out[0] = cvt4_e4m3(w[0], w[1], w[2], w[3]);
    out[1] = cvt4_e4m3(w[4], w[5], w[6], w[7]);
  }
  if (code == 255u) {
#pragma unroll
    for (int i = 0; i < BITS / 4; ++i) out[i] = 0u;
  }
}

// the four block codes of 16 neighbouring lanes as one word (in every lane)
__device__ __forceinline__ uint32_t mx_scale_word(uint32_t code) {
  uint32_t w = code << ((threadIdx.x & 12) << 1);
  w |= __shfl_xor_sync(0xFFFFFFFFu, w, 4);
  return w | __shfl_xor_sync(0xFFFFFFFFu, w, 8);
}

// Multiprocessors of the current device, asked for once per device, and the
// opt-in to a kernel's shared memory, once per kernel and device (`done`: a bit
// per device): both cost a small call as much as its other host work.
int mx_sm_count(int* device);
oq_status mx_allow_smem(const void* kernel, size_t bytes, int device, std::atomic<uint64_t>* done);

// The microscaled kernels follow one another in a stream (norm, product, norm),
// so each is launched as a programmatic dependent: it may be set up on the SMs
// while the kernel before it ends.  It reads and writes global memory only after
// dependency_wait, which returns when that kernel is complete, and lets the next
// one begin its set-up from there.  (After a kernel that announces nothing the
// launch is an ordinary one.)
__device__ __forceinline__ void dependency_wait() {
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
}
// launch with that attribute; cluster: CTAs of a cluster along x, or 0 for the kernel's own
template <typename P>
cudaError_t mx_launch(void (*kernel)(P), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream, const P& p) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// launches (oq_mx_quant.cu, oq_mx_gemm.cu, oq_mx_small.cu); arguments checked by the entry points
oq_status mx_quantize_launch(const void* x, int x_dtype, int64_t rows, int d, int bits, uint8_t* codes,
                             uint8_t* scales, void* stream);
oq_status mx_dequantize_launch(const uint8_t* codes, const uint8_t* scales, int64_t rows, int d, int bits, void* x,
                               int x_dtype, void* stream);
struct MxNormArgs {
  const void* x;
  const void* residual;   // or null: no addition
  int x_dtype;
  const void* gain;       // or null: ones
  int gain_dtype;
  float eps;
  int64_t rows;
  int d, bits;
  void* residual_out;     // or null: not kept
  uint8_t* codes;
  uint8_t* scales;
};
oq_status mx_norm_launch(const MxNormArgs& a, void* stream);
struct MxGemmArgs {
  const uint8_t* a_codes;   // [T, row bytes] of a_bits
  const uint8_t* a_scales;
  const uint8_t* w_codes;   // [N, row bytes] of 4 bits
  const uint8_t* w_scales;
  void* y;                  // [T, N]
  bool y_bf16;
  int64_t T;
  int N, K, a_bits;
  int* err;
};
oq_status mx_gemm_launch(const MxGemmArgs& g, void* stream);
oq_status mx_small_launch(const MxGemmArgs& g, void* stream);
// Batches that take the small-batch kernel: up to 128 tokens, and up to 256
// where K runs over more than 24 stages (of 256 4-bit or 128 8-bit elements), so
// that splitting K pays for the exchange of 256 tokens' sums.  Measured at 256
// tokens (us, small / pairs): 13824 -> 5120 18.8 / 21.4 (4 bits, 54 stages), 25.0
// / 38.5 (8 bits, 108); 5120 -> 5120 13.5 / 10.3 (20), 15.5 / 16.6 (40); 2048 ->
// 1040 9.6 / 6.0 (8), 10.5 / 8.3 (16).  The rule does not look at the outputs'
// width, which fills the pairs by itself: 5120 -> 13824 25.0 / 18.0 (8 bits, 40).
// At 129 tokens the two are even where the rule takes pairs (5120 -> 5120, 4 bits
// 9.7 / 10.2; 2048 -> 1040, 8 bits 7.8 / 8.2).
inline bool mx_small_batch(int64_t T, int K, int a_bits) {
  return T <= 128 || (T <= 256 && mx_col_tiles(K) * a_bits / 8 > 24);
}

}  // namespace oq
