// Product with 4-bit weights that have a scale (and a zero) for each group of
// 32, 64 or 128 neighbours of a row, for few tokens, and the weights' coding:
//   y[t, o] = sum_g s[o, g] sum_{i in g} (c[o, i] - z[o, g]) x[t, i]
//
// The weights' stream decides the time.  A CTA owns 16 or 32 weight rows and a part
// of K; its warps take runs of 128 in turn, each through its own ring in
// shared memory (it copies what it alone reads: no barrier).  A run's sixteen words
// are stored so that a lane of a quad finds its four words side by side, one in each
// block of 32: one 16-byte load a row and run, and every MMA (m16n8k16, M = 16
// weight rows, N = 8 tokens) stays within a block, so a group's sum can be scaled
// in fp32 when it ends.  Codes become bf16 exactly, without conversions: 0x4300 | c
// is 128 + c, less 128 + z.  fp32 tokens are split into three bf16 terms (8 + 8 + 8
// bits, exact), one MMA column each.  K is split over the CTAs of a cluster, so
// that small CTAs fill all SMs evenly; warps' and CTAs' sums are added in a fixed
// order through shared memory.
//
// Bound: latency that 12 to 24 warps an SM leave exposed (issue slots 46 to 48 % active, the
// integer pipe half busy; scales, zeros and tokens are awaited before a chunk's first MMA),
// and the launch.  Measured, bf16 tokens: one token x 13824 inputs x 5120 outputs, groups of 128,
// 13.3 us (the bytes alone 5.6); 13 tokens x 5120 x 13824, groups of 32 with zeros, 23.5 us
// (6.5).  A form on the tensor cores that read shared memory (codes as e4m3 subnormals,
// tokens in two e4m3 terms, 128 rows a CTA) took 19.5 and 52: tiles of 128 rows read 128
// bytes of a row at a time, and each group's accumulators pass through tensor memory.
#include <cuda_bf16.h>

#include <algorithm>

#include "oq_kv4.cuh"
#include "oq_ptx.cuh"

namespace oq {
namespace {

constexpr int ROWS = 16;      // weight rows per CTA
constexpr int RUN = 128;      // codes of a row that a warp takes at once

struct W4gParams {
  W4gArgs a;
  int per_cta;                // tokens per CTA
  int split;                  // CTAs of a cluster, splitting K
  int chunk;                  // runs whose tokens' elements lie in shared memory at once
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Elements 2 j, 2 j + 1 of a word's eight, less the zero (both bf16 pairs, exact).
// Mask and exponent come in registers: as immediates they took two instructions a
// pair, and the integer pipe decides the kernel's rate.
struct Decode {
  uint32_t mask, one;
  __device__ __forceinline__ Decode() {
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(mask));
    asm volatile("mov.b32 %0, 0x43004300;" : "=r"(one));
  }
  __device__ __forceinline__ uint32_t pair(uint32_t w, int j, __nv_bfloat162 zero) const {
    uint32_t u;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(u) : "r"(w >> (4 * j)), "r"(mask), "r"(one));   // (a & b) | c
    const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), zero);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
__device__ __forceinline__ __nv_bfloat162 zero_pair(uint32_t z) {
  const uint32_t u = 0x43004300u | z | z << 16;
  return *reinterpret_cast<const __nv_bfloat162*>(&u);
}

// Eight neighbouring elements of a token in shared memory as one MMA column's
// operand: the token (bf16), or one of its three terms (fp32).
template <typename X>
__device__ __forceinline__ uint4 load_column(const unsigned char* p, int term) {
  const uint4 a = reinterpret_cast<const uint4*>(p)[0];
  if constexpr (sizeof(X) == 2) {
    return a;
  } else {
    const uint4 b = reinterpret_cast<const uint4*>(p)[1];
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float h = __uint_as_float(v[i] & 0xFFFF0000u), r = __uint_as_float(v[i]) - h;
      const float m = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
      u[i] = __float_as_uint(term == 0 ? h : term == 1 ? m : r - m);
      if ((v[i] & 0x7F800000u) == 0x7F800000u)   // an infinity or a NaN (kept one) in the first term
        u[i] = term ? 0u : v[i] | (v[i] & 0x007FFFFFu ? 0x00400000u : 0u);
    }
    return make_uint4(__byte_perm(u[0], u[1], 0x7632), __byte_perm(u[2], u[3], 0x7632), __byte_perm(u[4], u[5], 0x7632),
                      __byte_perm(u[6], u[7], 0x7632));
  }
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_or_zero(uint32_t dst, const void* src, bool copy) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(copy ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// NW warps, which split K
template <int NT, int MT, int NW>
struct Cfg {
  // CTAs an SM and stages of a warp's ring; what the rings leave of an SM's shared memory
  // decides how many runs' tokens are brought in at once.  Measured (us): 13 tokens
  // 5120 -> 13824, 4 warps, 3 CTAs and 4 stages 23.5, 2 stages 23.7, 6 stages 27.6, 5 or 3
  // (the remainders cost more) 28.4, 8 warps and 2 CTAs 27.8 to 31; 32 tokens, 3 CTAs and
  // 4 stages 38.4, 2 CTAs 41.6, with 6 stages 60.
  static constexpr int NWARP = NW, MIN_CTAS = NT == 1 && NW == 4 ? 5 : 3;
  static constexpr int STAGE = MT * 1024, STAGES = NT == 1 && MT == 2 ? 2 : 4;   // MT tiles of 16 rows x 64 bytes
  static constexpr int RING = NWARP * STAGES * STAGE;
  static constexpr int PART = NWARP * MT * NT * 512;            // the warps' sums, in the ring's place
  static constexpr int BYTES = RING > PART ? RING : PART;
};

// bytes of a token's elements of a chunk: two neighbouring tokens share no bank
__host__ __device__ inline int x_pitch(int chunk, int size) { return chunk * RUN * size + 64; }

// MT tiles of 16 weight rows a CTA, NT tiles of 8 MMA columns.
template <typename X, int GROUP, bool ZEROS, int NT, int MT, int NW>
__global__ void __launch_bounds__(Cfg<NT, MT, NW>::NWARP * 32, Cfg<NT, MT, NW>::MIN_CTAS) w4g_kernel(const __grid_constant__ W4gParams p) {
  using C = Cfg<NT, MT, NW>;
  constexpr int TERMS = sizeof(X) == 2 ? 1 : 3, SUB = RUN / GROUP;   // groups in a run
  constexpr int NWARP = C::NWARP, TILE = ROWS * MT, NTHR = NWARP * 32;
  extern __shared__ __align__(128) unsigned char smem[];
  const W4gArgs& a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int rank = (int)blockIdx.x % p.split, o0 = (int)blockIdx.x / p.split * TILE;
  const int64_t t0 = (int64_t)blockIdx.y * p.per_cta;
  const int tokens = (int)(a.T - t0 < p.per_cta ? a.T - t0 : p.per_cta);
  const int all = (a.K + RUN - 1) / RUN, groups = a.K / GROUP;
  const int r0 = (int)((int64_t)all * rank / p.split), r1 = (int)((int64_t)all * (rank + 1) / p.split);
  dependency_wait();
  // lane l copies 16 bytes of row l / 4 (and + 8) of each tile, which are what lane l reads
  const uint8_t* src[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)   // (rows behind the last repeat it and are not stored)
      src[m][h] = a.codes + ((int64_t)min(o0 + 16 * m + 8 * h + g, a.N - 1) * all + r0 + warp) * (RUN / 2) + q * 16;
  unsigned char* ring = smem + warp * C::STAGES * C::STAGE + lane * 16;
  int ahead = r0 + warp;   // the next run to copy
  auto fetch = [&](int st) {
    if (ahead < r1) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          copy16((uint32_t)__cvta_generic_to_shared(ring + st * C::STAGE + m * 1024 + h * 512), src[m][h]);
          src[m][h] += NWARP * (RUN / 2);
        }
    }
    ahead += NWARP;
    copy_commit();
  };
#pragma unroll
  for (int u = 0; u < C::STAGES - 1; ++u) fetch(u);

  const int pitch = x_pitch(p.chunk, (int)sizeof(X));
  unsigned char* xs = smem + C::BYTES;
  uint16_t* scales = reinterpret_cast<uint16_t*>(xs + p.per_cta * pitch);            // [group of the chunk][row]
  uint8_t* zeros = reinterpret_cast<uint8_t*>(scales + p.chunk * SUB * TILE);
  const unsigned char* xcol[NT];   // this lane's MMA columns (those of no token repeat the last one's and are not stored)
  int term[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int c = 8 * n + g, t = c / TERMS;
    term[n] = c - t * TERMS;
    xcol[n] = xs + min(t, tokens - 1) * pitch + 8 * q * (int)sizeof(X);
  }
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
  const Decode decode;
  int st = 0;
#pragma unroll 1
  for (int c0 = r0; c0 < r1; c0 += p.chunk) {
    const int c1 = min(c0 + p.chunk, r1);
    if (c0 > r0) __syncthreads();
    // the tokens' elements of these runs, zeros behind the last, and the rows' scales
    const int words = (c1 - c0) * RUN * (int)sizeof(X) / 16, valid = (a.K - c0 * RUN) * (int)sizeof(X) / 16;
    for (int t = warp; t < tokens; t += NWARP) {
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const X*>(a.x) + (t0 + t) * a.K + (int64_t)c0 * RUN);
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(xs + t * pitch);
      for (int w = lane; w < words; w += 32) copy16_or_zero(to + 16 * w, w < valid ? from + w : from, w < valid);
    }
    copy_commit();
    {
      constexpr int PER = NTHR / TILE;   // threads of a row
      const int m = threadIdx.x / PER, n = (c1 - c0) * SUB, left = groups - c0 * SUB;
      const int64_t at = (int64_t)min(o0 + m, a.N - 1) * groups + c0 * SUB;
#pragma unroll 4
      for (int k = threadIdx.x % PER; k < n; k += PER) {
        scales[k * TILE + m] = k < left ? __ldcg(static_cast<const uint16_t*>(a.scales) + at + k) : (uint16_t)0;
        if constexpr (ZEROS) zeros[k * TILE + m] = k < left ? __ldcg(a.zeros + at + k) : (uint8_t)0;
      }
    }
    copy_wait<0>();
    __syncthreads();
#pragma unroll 1
    for (int i = c0 + warp; i < c1; i += NWARP) {
      copy_wait<C::STAGES - 2>();
      uint4 w[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) w[m][h] = *reinterpret_cast<const uint4*>(ring + st * C::STAGE + m * 1024 + h * 512);
      fetch((st + C::STAGES - 1) % C::STAGES);   // (this lane read that stage's words itself, a run ago)
      st = (st + 1) % C::STAGES;
      const int at = (i - c0) * RUN * (int)sizeof(X);
#pragma unroll
      for (int k = 0; k < SUB; ++k) {
        float sum[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[m][n][e] = 0.f;
        const int row = ((i - c0) * SUB + k) * TILE + g;
#pragma unroll
        for (int s = k * (4 / SUB); s < (k + 1) * (4 / SUB); ++s) {
          uint4 x[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) x[n] = load_column<X>(xcol[n] + at + 32 * s * (int)sizeof(X), term[n]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            uint32_t d[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4& c = w[m][h];
              const uint32_t word = s == 0 ? c.x : s == 1 ? c.y : s == 2 ? c.z : c.w;
              const __nv_bfloat162 z = zero_pair(ZEROS ? (uint32_t)zeros[row + 16 * m + 8 * h] : 8u);
#pragma unroll
              for (int j = 0; j < 4; ++j) d[h][j] = decode.pair(word, j, z);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mma_bf16(sum[m][n], d[0][0], d[1][0], d[0][1], d[1][1], x[n].x, x[n].y);
              mma_bf16(sum[m][n], d[0][2], d[1][2], d[0][3], d[1][3], x[n].z, x[n].w);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const float s_lo = __uint_as_float((uint32_t)scales[row + 16 * m] << 16);
          const float s_hi = __uint_as_float((uint32_t)scales[row + 16 * m + 8] << 16);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[m][n][0] = fmaf(sum[m][n][0], s_lo, acc[m][n][0]);
            acc[m][n][1] = fmaf(sum[m][n][1], s_lo, acc[m][n][1]);
            acc[m][n][2] = fmaf(sum[m][n][2], s_hi, acc[m][n][2]);
            acc[m][n][3] = fmaf(sum[m][n][3], s_hi, acc[m][n][3]);
          }
        }
      }
    }
  }
  copy_wait<0>();
  __syncthreads();   // the ring's place is the sums': [warp][MT][NT][lane][4]
  float* part = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<float4*>(part + (((warp * MT + m) * NT + n) * 32 + lane) * 4) =
          make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
  if (p.split > 1) cluster_sync_all();
  else __syncthreads();
  // outputs in turn over the cluster's CTAs; sums over terms, CTAs and warps in order
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(part);
  for (int idx = rank * NTHR + (int)threadIdx.x; idx < tokens * TILE; idx += p.split * NTHR) {
    const int t = idx / TILE, r = idx % TILE, o = o0 + r;
    if (o >= a.N) continue;
    float v = 0.f;
#pragma unroll
    for (int e = TERMS - 1; e >= 0; --e) {
      const int c = t * TERMS + e;   // MMA column
      const int at = ((r / 16 * NT + (c >> 3)) * 32 + (r & 7) * 4 + ((c & 7) >> 1)) * 4 + ((r >> 3) & 1) * 2 + (c & 1);
      for (int k = 0; k < p.split; ++k) {
        const uint32_t from = p.split > 1 ? mapa_shared(base + 4 * at, (uint32_t)k) : base + 4 * at;
#pragma unroll
        for (int w = 0; w < NWARP; ++w) v += ld_cluster(from + (uint32_t)(w * MT * NT * 512));
      }
    }
    const int64_t at = (t0 + t) * a.N + o;
    if (a.y_dtype == OQ_DTYPE_BF16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(a.y)[at] = v;
  }
  if (p.split > 1) cluster_sync_all();   // no CTA leaves before its sums are read
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

template <typename X, int GROUP, bool ZEROS, int NT, int MT, int NW>
cudaError_t launch_one(W4gParams& p, cudaStream_t st) {
  using C = Cfg<NT, MT, NW>;
  constexpr int NWARP = C::NWARP;
  int dev = 0;
  const int sms = mx_sm_count(&dev);
  const int64_t tiles = (p.a.N + ROWS * MT - 1) / (ROWS * MT), blocks = (p.a.T + p.per_cta - 1) / p.per_cta;
  const int runs = (p.a.K + RUN - 1) / RUN;
  // a cluster of 2, 4 or 8 CTAs while all are resident at once, each warp of them with two runs
  p.split = 1;
  while (p.split < 8 && 2 * p.split * NWARP <= runs && 2 * tiles * blocks * p.split <= (int64_t)C::MIN_CTAS * sms) p.split *= 2;
  // the tokens' elements of as many runs as leave room for MIN_CTAS CTAs on an SM
  const int mine = (runs + p.split - 1) / p.split, budget = 226 * 1024 / C::MIN_CTAS - 1024 - C::BYTES - 64 * p.per_cta;
  const int per_run = p.per_cta * RUN * (int)sizeof(X) + RUN / GROUP * ROWS * MT * (ZEROS ? 3 : 2);
  const int fit = std::max(budget / per_run, 1);
  p.chunk = mine <= fit ? mine : std::max(fit / NWARP * NWARP, NWARP);
  const size_t smem = (size_t)C::BYTES + (size_t)p.per_cta * x_pitch(p.chunk, (int)sizeof(X)) +
                      (size_t)p.chunk * (RUN / GROUP) * ROWS * MT * (ZEROS ? 3 : 2);
  static std::atomic<uint64_t> smem_set{0};
  if (mx_allow_smem(reinterpret_cast<const void*>(w4g_kernel<X, GROUP, ZEROS, NT, MT, NW>), 227 * 1024, dev, &smem_set) != OQ_OK)
    return cudaErrorInvalidConfiguration;
  return mx_launch(w4g_kernel<X, GROUP, ZEROS, NT, MT, NW>, dim3((unsigned)(tiles * p.split), (unsigned)blocks), NWARP * 32, smem,
                   p.split, st, p);
}
template <typename X, int GROUP, bool ZEROS>
cudaError_t launch_tiles(W4gParams& p, cudaStream_t st) {
  constexpr int TERMS = sizeof(X) == 2 ? 1 : 3;
  // 32 columns a CTA at most; more tokens read the weights again (from L2)
  const int columns = (int)std::min<int64_t>(p.a.T * TERMS, 32);
  p.per_cta = p.a.T * TERMS <= 32 ? (int)p.a.T : 32 / TERMS;
  int dev = 0;
  const int sms = mx_sm_count(&dev);
  // Up to eight columns.  Where CTAs of 16 rows need more than one round, 32 rows and 8 warps:
  // one token 5120 -> 13824, groups of 128, 10.7 us, with 16 rows 13.4, eight tokens, groups
  // of 64, 15.3 and 18.6; 8192 -> 28672 31.8 and 33.3, 45.0 and 51.4.  Otherwise 16 rows,
  // whose CTAs read a row to its end: 4096 -> 6144 6.6 us and 7.1, 8.7 and 11.0; but long rows
  // are split, over CTAs of 32 rows and 4 warps: 13824 -> 5120 13.3 and, with 16 rows, 14.0,
  // 18.9 and 21.9; 4096 -> 4096 6.1 and 5.9, 9.9 and 7.7.  Between (to 5120, groups of 128, one
  // token and eight): 6144 7.9 and 8.1, 11.8 and 10.4; 8192 9.0 and 9.2, 13.7 and 12.7; 10240
  // 10.3 and 10.9, 15.2 and 15.2.
  if (columns <= 8) {
    const int64_t ctas = (p.a.N + ROWS - 1) / ROWS * ((p.a.T + p.per_cta - 1) / p.per_cta);
    if (ctas > Cfg<1, 1, 8>::MIN_CTAS * (int64_t)sms) return launch_one<X, GROUP, ZEROS, 1, 2, 8>(p, st);
    if (2 * ctas > Cfg<1, 1, 8>::MIN_CTAS * (int64_t)sms && p.a.K >= 64 * RUN) return launch_one<X, GROUP, ZEROS, 1, 2, 4>(p, st);
    return launch_one<X, GROUP, ZEROS, 1, 1, 8>(p, st);
  }
  // more: 32 weight rows a CTA share what is loaded of the tokens, where they still fill the
  // SMs (13 tokens 5120 -> 13824 23.5 us, with 16 rows 29.0; 13824 -> 5120 32.6, 35.4)
  const bool two = p.a.N >= 32 * sms;
  if (columns <= 16) return two ? launch_one<X, GROUP, ZEROS, 2, 2, 4>(p, st) : launch_one<X, GROUP, ZEROS, 2, 1, 4>(p, st);
  return two ? launch_one<X, GROUP, ZEROS, 4, 2, 4>(p, st) : launch_one<X, GROUP, ZEROS, 4, 1, 4>(p, st);
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
