// Product with 4-bit weights that have a scale (and a zero) for each group of
// 32, 64 or 128 neighbours of a row, for few tokens, and the weights' coding:
//   y[t, o] = sum_g s[o, g] sum_{i in g} (c[o, i] - z[o, g]) x[t, i]
//
// The weights' stream decides the time.  A CTA owns 16 weight rows; its warps
// split K in runs of 128.  A run's sixteen words are stored so that a lane of a
// quad finds its four words side by side, one in each block of 32: one 16-byte
// load a row and run, and every MMA (m16n8k16, M = 16 weight rows, N = 8 tokens)
// stays within a block, so a group's sum can be scaled in fp32 when it ends.
// Codes become bf16 exactly, without conversions: 0x4300 | c is 128 + c, less
// 128 + z.  fp32 tokens are split into three bf16 terms (8 + 8 + 8 bits, exact),
// one MMA column each.  The warps' sums meet in shared memory in a fixed order.
#include <cuda_bf16.h>

#include <algorithm>

#include "oq_kv4.cuh"

namespace oq {
namespace {

constexpr int ROWS = 16;      // weight rows per CTA
constexpr int NWARP = 8;      // warps per CTA, splitting K
constexpr int RUN = 128;      // codes of a row that a warp takes at once

struct W4gParams {
  W4gArgs a;
  int per_cta;                // tokens per CTA
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// elements 2 j, 2 j + 1 of a word's eight, less the zero (both bf16 pairs, exact)
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j, __nv_bfloat162 zero) {
  const uint32_t u = ((w >> (4 * j)) & 0x000F000Fu) | 0x43004300u;
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), zero);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t z) {
  const uint32_t u = 0x43004300u | z | z << 16;
  return *reinterpret_cast<const __nv_bfloat162*>(&u);
}

// Eight neighbouring elements of one MMA column: a token (bf16), or one of the
// three terms of a token (fp32).
template <typename X>
__device__ __forceinline__ uint4 load_column(const X* p, int term) {
  if constexpr (sizeof(X) == 2) {
    return __ldg(reinterpret_cast<const uint4*>(p));
  } else {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t bits = __float_as_uint(v[i]);
      const float h = __uint_as_float(bits & 0xFFFF0000u), r = v[i] - h;
      const float m = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
      u[i] = __float_as_uint(term == 0 ? h : term == 1 ? m : r - m);
      if ((bits & 0x7F800000u) == 0x7F800000u)   // an infinity or a NaN (kept one) in the first term
        u[i] = term ? 0u : bits | (bits & 0x007FFFFFu ? 0x00400000u : 0u);
    }
    return make_uint4(__byte_perm(u[0], u[1], 0x7632), __byte_perm(u[2], u[3], 0x7632), __byte_perm(u[4], u[5], 0x7632),
                      __byte_perm(u[6], u[7], 0x7632));
  }
}

template <typename X, int GROUP, bool ZEROS, int NT>
__global__ void __launch_bounds__(NWARP * 32, NT == 1 ? 3 : 2) w4g_kernel(const __grid_constant__ W4gParams p) {
  constexpr int TERMS = sizeof(X) == 2 ? 1 : 3, SUB = RUN / GROUP;   // groups in a run
  constexpr int PF = 3;                                              // runs in flight
  __shared__ __align__(16) float part[NWARP][NT][32][4];
  const W4gArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int o0 = (int)blockIdx.x * ROWS;
  const int64_t t0 = (int64_t)blockIdx.y * p.per_cta;
  const int tokens = (int)(a.T - t0 < p.per_cta ? a.T - t0 : p.per_cta);
  dependency_wait();
  const int runs = (a.K + RUN - 1) / RUN, groups = a.K / GROUP;
  const bool in_lo = o0 + g < a.N, in_hi = o0 + g + 8 < a.N;
  const int64_t row_lo = in_lo ? o0 + g : 0, row_hi = in_hi ? o0 + g + 8 : 0;
  const uint4* wl = reinterpret_cast<const uint4*>(a.codes + row_lo * runs * (RUN / 2)) + q;
  const uint4* wh = reinterpret_cast<const uint4*>(a.codes + row_hi * runs * (RUN / 2)) + q;
  const uint16_t* sl = static_cast<const uint16_t*>(a.scales) + row_lo * groups;
  const uint16_t* sh = static_cast<const uint16_t*>(a.scales) + row_hi * groups;
  const uint8_t* zl = ZEROS ? a.zeros + row_lo * groups : nullptr;
  const uint8_t* zh = ZEROS ? a.zeros + row_hi * groups : nullptr;

  struct Run {
    uint4 lo, hi;
    uint32_t s[SUB];   // bf16 scales of both rows
    uint32_t z[ZEROS ? SUB : 1];
  };
  Run buf[PF];
  auto fetch = [&](Run& r, int i) {
    if (i < runs) {
      r.lo = __ldg(wl + i * 4);
      r.hi = __ldg(wh + i * 4);
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        const int grp = i * SUB + k;
        const bool in = grp < groups;
        r.s[k] = in ? (uint32_t)__ldg(sl + grp) | (uint32_t)__ldg(sh + grp) << 16 : 0u;
        if constexpr (ZEROS) r.z[k] = in ? (uint32_t)__ldg(zl + grp) | (uint32_t)__ldg(zh + grp) << 16 : 0u;
      }
    }
  };
#pragma unroll
  for (int u = 0; u < PF; ++u) fetch(buf[u], warp + u * NWARP);

  // this lane's MMA columns
  const X* col[NT];
  int term[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int c = 8 * n + g, t = c / TERMS;
    term[n] = c - t * TERMS;
    col[n] = t < tokens ? static_cast<const X*>(a.x) + (t0 + t) * a.K + 8 * q : nullptr;
  }
  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[n][i] = 0.f;

#pragma unroll 1
  for (int i0 = warp; i0 < runs; i0 += PF * NWARP) {
#pragma unroll
    for (int u = 0; u < PF; ++u) {
      const int i = i0 + u * NWARP;
      if (i >= runs) break;   // warp-uniform
      const Run r = buf[u];
      fetch(buf[u], i + PF * NWARP);
      const uint32_t lo[4] = {r.lo.x, r.lo.y, r.lo.z, r.lo.w}, hi[4] = {r.hi.x, r.hi.y, r.hi.z, r.hi.w};
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        const __nv_bfloat162 z_lo = zero_pair(ZEROS ? r.z[k] & 0xFFFFu : 8u), z_hi = zero_pair(ZEROS ? r.z[k] >> 16 : 8u);
        float sum[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[n][e] = 0.f;
#pragma unroll
        for (int s = k * (4 / SUB); s < (k + 1) * (4 / SUB); ++s) {
          const int pos = i * RUN + 32 * s;
          uint32_t dl[4], dh[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            dl[j] = code_pair(lo[s], j, z_lo);
            dh[j] = code_pair(hi[s], j, z_hi);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 x = col[n] && pos < a.K ? load_column<X>(col[n] + pos, term[n]) : make_uint4(0u, 0u, 0u, 0u);
            mma_bf16(sum[n], dl[0], dh[0], dl[1], dh[1], x.x, x.y);
            mma_bf16(sum[n], dl[2], dh[2], dl[3], dh[3], x.z, x.w);
          }
        }
        const float s_lo = __uint_as_float(r.s[k] << 16), s_hi = __uint_as_float(r.s[k] & 0xFFFF0000u);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n][0] = fmaf(sum[n][0], s_lo, acc[n][0]);
          acc[n][1] = fmaf(sum[n][1], s_lo, acc[n][1]);
          acc[n][2] = fmaf(sum[n][2], s_hi, acc[n][2]);
          acc[n][3] = fmaf(sum[n][3], s_hi, acc[n][3]);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
    *reinterpret_cast<float4*>(part[warp][n][lane]) = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
  __syncthreads();
  for (int idx = threadIdx.x; idx < tokens * ROWS; idx += NWARP * 32) {
    const int t = idx / ROWS, m = idx % ROWS;
    if (o0 + m >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int e = TERMS - 1; e >= 0; --e) {
      const int c = t * TERMS + e;   // MMA column
#pragma unroll
      for (int w = 0; w < NWARP; ++w) v += part[w][c >> 3][(m & 7) * 4 + ((c & 7) >> 1)][(m >> 3) * 2 + (c & 1)];
    }
    const int64_t at = (t0 + t) * a.N + o0 + m;
    if (a.y_dtype == OQ_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(a.y)[at] = v;
  }
}

// ------------------------------------------------------------------ coding
struct PrepareParams {
  const void* W;
  int dtype, N, K, group;
  uint8_t* codes;
  uint16_t* scales;
  uint8_t* zeros;
};

// A warp codes a run of 128 elements of a row, four neighbours a lane.  All
// decisions are fp32 with IEEE division, on the scale as it is stored.
__global__ void __launch_bounds__(256) w4g_prepare_kernel(const __grid_constant__ PrepareParams p) {
  dependency_wait();
  const int lane = threadIdx.x & 31;
  const int runs = (p.K + RUN - 1) / RUN, groups = p.K / p.group;
  const int64_t total = (int64_t)p.N * runs;
  for (int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += (int64_t)gridDim.x * 8) {
    const int64_t row = i / runs;
    const int pos = (int)(i % runs) * RUN + 4 * lane;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    if (pos < p.K) {
      const int64_t at = row * p.K + pos;
      if (p.dtype == OQ_DTYPE_BF16) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.W) + at);
        w[0] = __uint_as_float(v.x << 16), w[1] = __uint_as_float(v.x & 0xFFFF0000u);
        w[2] = __uint_as_float(v.y << 16), w[3] = __uint_as_float(v.y & 0xFFFF0000u);
      } else {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p.W) + at);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      }
    }
    float lo = 0.f, hi = 0.f;
    int bad = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo = fminf(lo, w[j]);
      hi = fmaxf(hi, w[j]);
      bad |= !(fabsf(w[j]) <= 3.402823466e38f);
    }
    for (int o = 1; o < p.group / 4; o <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
      hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
      bad |= __shfl_xor_sync(0xFFFFFFFFu, bad, o);
    }
    __nv_bfloat16 sb = __float2bfloat16_rn(p.zeros ? __fdiv_rn(hi - lo, 15.f) : __fdiv_rn(fmaxf(hi, -lo), 7.f));
    float s = __bfloat162float(sb);
    if (bad || !(s <= 3.402823466e38f)) {   // such a group reads as NaN
      sb = __ushort_as_bfloat16(0x7FC0);
      s = 0.f;
    }
    const float z = !p.zeros ? 8.f : s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(-lo, s)), 0.f), 15.f) : 0.f;
    uint32_t word = 0u;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float c = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(w[j], s)) + z, 0.f), 15.f) : z;
      const int e = 4 * (lane & 1) + j;   // element of the word's eight
      word |= (uint32_t)c << (4 * (e / 2 + 4 * (e % 2)));
    }
    word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
    if (!(lane & 1)) {
      const int blk = lane >> 3, q = (lane & 7) >> 1;
      reinterpret_cast<uint32_t*>(p.codes)[i * 16 + 4 * q + blk] = word;
    }
    if (pos < p.K && (4 * lane) % p.group == 0) {
      const int64_t at = row * groups + pos / p.group;
      p.scales[at] = __bfloat16_as_ushort(sb);
      if (p.zeros) p.zeros[at] = (uint8_t)z;
    }
  }
}

oq_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return OQ_OK;
  set_error(std::string(what) + " launch: " + cudaGetErrorString(e));
  return OQ_ERR_CUDA;
}

template <typename X, int GROUP, bool ZEROS>
cudaError_t launch_tiles(W4gParams& p, cudaStream_t st) {
  constexpr int TERMS = sizeof(X) == 2 ? 1 : 3;
  // 32 columns a CTA at most; more tokens read the weights again (from L2)
  const int columns = (int)std::min<int64_t>(p.a.T * TERMS, 32);
  p.per_cta = p.a.T * TERMS <= 32 ? (int)p.a.T : 32 / TERMS;
  const dim3 grid((unsigned)((p.a.N + ROWS - 1) / ROWS), (unsigned)((p.a.T + p.per_cta - 1) / p.per_cta));
  if (columns <= 8) return mx_launch(w4g_kernel<X, GROUP, ZEROS, 1>, grid, NWARP * 32, 0, 0, st, p);
  if (columns <= 16) return mx_launch(w4g_kernel<X, GROUP, ZEROS, 2>, grid, NWARP * 32, 0, 0, st, p);
  return mx_launch(w4g_kernel<X, GROUP, ZEROS, 4>, grid, NWARP * 32, 0, 0, st, p);
}
template <typename X, int GROUP>
cudaError_t launch_zeros(W4gParams& p, cudaStream_t st) {
  return p.a.zeros ? launch_tiles<X, GROUP, true>(p, st) : launch_tiles<X, GROUP, false>(p, st);
}
template <typename X>
cudaError_t launch_group(W4gParams& p, cudaStream_t st) {
  return p.a.group == 32 ? launch_zeros<X, 32>(p, st) : p.a.group == 64 ? launch_zeros<X, 64>(p, st) : launch_zeros<X, 128>(p, st);
}

}  // namespace

oq_status w4g_linear_launch(const W4gArgs& a, void* stream) {
  W4gParams p;
  p.a = a;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return launched(a.x_dtype == OQ_DTYPE_BF16 ? launch_group<__nv_bfloat16>(p, st) : launch_group<float>(p, st),
                  "group-scaled product");
}

oq_status w4g_prepare_launch(const void* W, int dtype, int N, int K, int group, uint8_t* codes, void* scales,
                             uint8_t* zeros, void* stream) {
  PrepareParams p;
  p.W = W;
  p.dtype = dtype;
  p.N = N;
  p.K = K;
  p.group = group;
  p.codes = codes;
  p.scales = static_cast<uint16_t*>(scales);
  p.zeros = zeros;
  int dev = 0;
  const int64_t warps = (int64_t)N * ((K + RUN - 1) / RUN);
  const int64_t ctas = std::min<int64_t>((warps + 7) / 8, 16 * (int64_t)mx_sm_count(&dev));
  return launched(mx_launch(w4g_prepare_kernel, dim3((unsigned)ctas), 256, 0, 0, static_cast<cudaStream_t>(stream), p),
                  "group-scaled weight coding");
}

}  // namespace oq
