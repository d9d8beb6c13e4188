// Attention over the 4-bit paged cache, for one query token or many:
//   y = softmax(scale q K^T + mask) V
// on the block-scaled tensor cores, which read the cache's codes as they lie.
//
// The keys are the MMA's M: a CTA takes up to COLS queries (a key head's query
// heads, of one token or several) and walks over tiles of 128 tokens, a page.
//   S^T [128 tokens x queries]  = K [tokens x 128 channels] q^T      (K's scales: A's)
//   O^T [128 channels x queries] += V^T [channels x 128 tokens] P    (V's scales: in P)
// A query in bf16 is split into two e4m3 terms (4 + 4 bits, two MMA columns that are
// added up): exactly, but for elements below 2^-14 of their 32 channels' largest, which
// are off by up to 2^-22 of that.  P is split into two e4m3 terms as well, 8 bits
// as in bf16.  V's scales belong to a token and 32 channels, along M and K both,
// which no operand scale can say; so P takes them up: four copies of P, each
// times V's scales of one block of 32 channels, of which only the block's own 32
// rows of the product are used.  The wasted products cost less than decoding V
// would: the cores are idle most of the time otherwise.
//
// Softmax without a pass for the maximum: a thread has one token.  Each warp's 32
// tokens are one scale block of the second product, so the warp takes a power of
// two at or above its own tokens' largest weight as the block's scale, and
// P / scale fills e4m3's range; the running sums O and l stay relative to one
// power of two a query, which moves (and rescales O in tensor memory) only when
// a weight exceeds it by 2^8: in the first tile, and rarely after.
//
// Long caches are split over CTAs; a second kernel joins the parts in a fixed
// order, so results repeat bit for bit.
//
// Bound: a tile's chain of load, first product, softmax, second product, which the CTAs
// of an SM overlap.  Measured, one token over 32760 x 40 heads of 128: 38 us for 178 MB
// (27 us at the copy's rate); the loads alone took 33, the MMAs alone 34, the softmax
// alone 34.  64 streams of 4096 to 8192 tokens x 8 heads with 4 queries each: 91 us
// for 64; alone 74, 81, 79.
//
// Warps: 0-3 softmax and epilogue, 4 TMA producer, 5 tensor memory and MMAs.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "oq_kv4.cuh"
#include "oq_mx_ptx.cuh"

namespace oq {
namespace {

constexpr int TMA_WARP = 4, MMA_WARP = 5, NTHREADS = 6 * 32;
constexpr int UNIT = 16 * 1024;        // a tile of K or of V, spread to 8-bit containers
constexpr float LAZY = 8.f;            // log2 of the largest weight relative to the running reference
constexpr float NONE = -3.4028234e38f; // reference of a query that has seen no token: below every score's
constexpr float FAR = 4194304.f;       // 2^22: the last bit of a reference is half a unit of log2

// COLS queries; HP heads share a group of 128 channels
template <int COLS, int HP>
struct Cfg {
  static constexpr int HC = HP * COLS;                       // queries with their head of the group
  static constexpr int CTAS = COLS <= 4 ? 3 : 2, UNITS = COLS > 4 ? 5 : HP == 2 ? 3 : 4;   // CTAs an SM; units in the ring
  // columns of S, for each head: first terms, second terms.  Heads are multiplied
  // apart: a NaN among one's keys is nothing to the other.
  static constexpr int N1H = 2 * COLS < 16 ? 16 : 2 * COLS, N1 = HP * N1H;
  static constexpr int N2 = 8 * COLS;                        // of O: [block of 32 channels][term][query]
  // scale columns: K (two sets in turn), q of each head, V's ones, P
  static constexpr int SF_K = 0, SF_Q = 8, SF_ONE = 16, SF_P = 20, SF = 24;
  static constexpr int SB = N2 + 2 * N1 + SF <= 256 ? 2 : 1; // S buffers
  static constexpr uint32_t TMEM = N2 + SB * N1 + SF <= 128 ? 128 : 256;
  static_assert(N2 + SB * N1 + SF <= TMEM && CTAS * TMEM <= 512 && N2 <= 128 && HC <= 32, "tensor memory of an SM's CTAs");
  static constexpr int PITCH = N2 < 32 ? 32 : N2;            // bytes of a token in P: a swizzle's row
  static constexpr int P = UNITS * UNIT, Q = P + 128 * PITCH, KS = Q + N1 * 128, SFQ = KS + UNITS * 512;
  static constexpr int SFP = SFQ + HP * 512;
  static constexpr int RED = SFP + 512, ONES = RED;          // [4][32] floats; before the first tile V's ones
  static constexpr int BAR = RED + 512;
  static constexpr size_t SMEM = 1024 + BAR + 8 * (2 * UNITS + 2 * SB + 3) + 64;
  static_assert((SMEM + 1024) * CTAS <= 228 * 1024, "CTAs an SM");
};

struct AttnParams : AttnSplit {
  CUtensorMap map;
};

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, float* v) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
  if constexpr (N == 2) {
    uint32_t r[2];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr) : "memory");
    v[0] = __uint_as_float(r[0]), v[1] = __uint_as_float(r[1]);
  } else if constexpr (N >= 8) {
#pragma unroll
    for (int i = 0; i < N; i += 8) tmem_ld8(taddr + i, v + i);
  } else {
    tmem_ld4(taddr, v);
  }
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(__float_as_uint(v[0])),
               "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3]))
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// P as the second product's B operand, columns contiguous: [token][PITCH bytes] in
// the swizzle of that row length, groups of eight tokens 8 PITCH apart
template <int PITCH>
__device__ __forceinline__ uint64_t smem_desc_p(uint32_t addr) {
  return (smem_desc_sw128(addr) & ~((uint64_t)0x3FFF << 32) & ~((uint64_t)7 << 61)) | (uint64_t)(8 * PITCH >> 4) << 32 |
         (uint64_t)(PITCH == 128 ? 2 : PITCH == 64 ? 4 : 6) << 61;
}
// place of 16-byte chunk c of a token's columns
template <int PITCH>
__device__ __forceinline__ uint32_t p_at(int token, int c) {
  const int turn = PITCH == 128 ? token & 7 : PITCH == 64 ? token >> 1 & 3 : token >> 2 & 1;
  return (uint32_t)(token * PITCH + ((c ^ turn) << 4));
}

__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// pairs: fp32 -> e4m3 (a low), fp16 -> e4m3, e4m3 -> fp16
__device__ __forceinline__ uint16_t cvt_e4m3(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t cvt_e4m3_h2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t cvt_h2_e4m3(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t h) {
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(v);
}

template <int COLS, int HP>
__global__ void __launch_bounds__(NTHREADS, (Cfg<COLS, HP>::CTAS)) attention_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<COLS, HP>;
  constexpr int HC = C::HC, N1 = C::N1, N2 = C::N2, SB = C::SB, UNITS = C::UNITS;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR);
  uint64_t* empty = full + UNITS;
  uint64_t* s_full = empty + UNITS;
  uint64_t* s_free = s_full + SB;
  uint64_t* p_full = s_free + SB;
  uint64_t* p_free = p_full + 1;
  uint64_t* q_full = p_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 1);
  int* failed = reinterpret_cast<int*>(tmem_slot + 1);
  float* red = reinterpret_cast<float*>(smem + C::RED);

  const AttentionArgs& a = p.a;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < UNITS; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
    for (int i = 0; i < SB; ++i) mbar_init(&s_full[i], 1), mbar_init(&s_free[i], 4);
    mbar_init(p_full, 4);
    mbar_init(p_free, 1);
    mbar_init(q_full, 4);
    *failed = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_slot, C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (a kernel that may start from here finds this CTA's tensor memory allocated)
  dependency_wait();
  const int hg = (int)blockIdx.y / p.splits, split = (int)blockIdx.y % p.splits, b = (int)blockIdx.z;
  const int tok0 = a.kv.cu[b], end = a.kv.cu[b + 1], len = min(a.kv.lens[b], a.kv.width * KV_PAGE);
  // a sequence that the call's arrays do not hold has no queries
  const int n = tok0 < 0 || end > a.T || end < tok0 ? 0 : end - tok0;
  const int past = a.kv.lens[b] - n;                   // place of the first query token
  const int c0 = (int)blockIdx.x * COLS, columns = min(n, a.max_q) * p.group;
  const bool work = c0 < columns;
  const int i_first = c0 / p.group, i_last = (min(c0 + COLS, columns) - 1) / p.group;
  // tokens [lo, hi) that any of these queries sees; this CTA's share of their tiles
  int hi = a.causal ? min(len, past + i_last + 1) : len, lo = 0;
  if (a.window > 0) lo = max(0, past + i_first - a.window + 1);
  const int tile_lo = lo / KV_PAGE, tiles = work && hi > lo ? (hi + KV_PAGE - 1) / KV_PAGE - tile_lo : 0;
  const int first = tile_lo + (int)((int64_t)tiles * split / p.splits);
  const int nt = tile_lo + (int)((int64_t)tiles * (split + 1) / p.splits) - first;
  const int* table = a.kv.table + (int64_t)b * a.kv.width + first;
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t t_o = tmem, t_s = tmem + N2, t_sf = tmem + N2 + SB * N1;

  // units in the order the MMAs use them: K0, K1, V0, K2, V1, .., V(nt - 1)
  auto unit_k = [&](int t) { return t == 0 ? 0 : 2 * t - 1; };
  auto unit_v = [&](int t) { return t < nt - 1 ? 2 * t + 2 : 2 * nt - 1; };

  if (warp == TMA_WARP) {
    if (lane == 0) {
      int u = 0;
      for (; u < 2 * nt; ++u) {
        const int s = u % UNITS;
        const bool is_k = u == 0 || ((u & 1) && u != 2 * nt - 1);
        const int t = u == 0 ? 0 : u == 2 * nt - 1 ? nt - 1 : is_k ? (u + 1) / 2 : u / 2 - 1;
        if (u >= UNITS && !mbar_wait(&empty[s], (uint32_t)(u / UNITS - 1) & 1u, a.err)) break;
        const int page = table[t];
        unsigned char* dst = smem + s * UNIT;
        if (page < 0 || page >= a.kv.pages) {   // not there: its tokens are not seen
          mbar_arrive(&full[s]);
          continue;
        }
        const int64_t row = ((int64_t)page * a.kv.groups + hg) * KV_ROWS;
        mbar_arrive_expect_tx(&full[s], is_k ? 8192 + 512 : 8192);
        tma_load_2d(dst, &p.map, 0, (int32_t)(row + (is_k ? 0 : KV_V_ROW)), &full[s]);
        if (is_k) bulk_g2s(smem + C::KS + s * 512, a.kv.cache + (row + KV_KS_ROW) * 64, 512, &full[s]);
      }
      // no copy may be in flight when the CTA leaves
      for (int g = u > UNITS ? u - UNITS : 0; g < u; ++g) mbar_wait(&full[g % UNITS], (uint32_t)(g / UNITS) & 1u, a.err);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    constexpr uint32_t idesc1 = idesc_mx(128, C::N1H, 5, 0), idesc2 = idesc_mx(128, N2, 5, 0) | (1u << 16);
    const uint32_t lead = elect_one();
    const uint64_t unit0 = smem_desc_sw128(smem_base), q0 = smem_desc_sw128(smem_base + C::Q);
    const uint64_t p0 = smem_desc_p<C::PITCH>(smem_base + C::P), ks0 = smem_desc_scales(smem_base + C::KS);
    bool ok = nt > 0 && __all_sync(0xFFFFFFFFu, mbar_wait(q_full, 0u, a.err));
    if (ok) {
      tc_fence_after();
      if (lead) {
#pragma unroll
        for (int h = 0; h < HP; ++h) tc_copy_scales<1>(t_sf + C::SF_Q + 4 * h, smem_desc_scales(smem_base + C::SFQ + 512 * h));
        tc_copy_scales<1>(t_sf + C::SF_ONE, smem_desc_scales(smem_base + C::ONES));
      }
      __syncwarp();
    }
    for (int t = 0; ok && t <= nt; ++t) {
      if (t < nt) {   // S of tile t
        const int u = unit_k(t), s = u % UNITS, sb = t % SB;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[s], (uint32_t)(u / UNITS) & 1u, a.err));
        if (ok && t >= SB) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_free[sb], (uint32_t)(t / SB - 1) & 1u, a.err));
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          const uint64_t off = (uint64_t)s * (UNIT >> 4);
          const uint32_t sfk = t_sf + C::SF_K + 4 * (t & 1);
          tc_copy_scales<1>(sfk, ks0 + (uint64_t)(s * 512 >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int h = k * HP / 4;
            tc_mma_mx<false>(t_s + sb * N1 + h * C::N1H, unit0 + off + 2 * k, q0 + (h * C::N1H * 128 >> 4) + 2 * k,
                             idesc1 | idesc_mx_sf(k), sfk, t_sf + C::SF_Q + 4 * h, k % (4 / HP) > 0);
          }
          tc_commit(&empty[s]);
          tc_commit(&s_full[sb]);
        }
        __syncwarp();
      }
      if (t > 0) {    // O += V^T P of tile t - 1
        const int u = unit_v(t - 1), s = u % UNITS;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[s], (uint32_t)(u / UNITS) & 1u, a.err)) &&
             __all_sync(0xFFFFFFFFu, mbar_wait(p_full, (uint32_t)(t - 1) & 1u, a.err));
        if (!ok) break;
        tc_fence_after();
        if (lead) {
          const uint64_t off = (uint64_t)s * (UNIT >> 4);
          tc_copy_scales<1>(t_sf + C::SF_P, smem_desc_scales(smem_base + C::SFP));
#pragma unroll
          for (int k = 0; k < 4; ++k)   // 32 tokens: 32 bytes of V's rows, 32 rows of P
            tc_mma_mx<false>(t_o, unit0 + off + 2 * k, p0 + (uint64_t)(k * 32 * C::PITCH >> 4), idesc2 | idesc_mx_sf(k),
                             t_sf + C::SF_ONE, t_sf + C::SF_P, t > 1 || k > 0);
          tc_commit(&empty[s]);
          tc_commit(p_free);
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else if (warp < 4 && work) {
    const int key = (int)threadIdx.x;   // this thread's token of a tile, and its lane of tensor memory
    const uint32_t my = (uint32_t)(warp * 32) << 16;
    // ---- the queries as two e4m3 terms, scales of V's operand
    reinterpret_cast<uint32_t*>(smem + C::ONES)[key] = 0x7F7F7F7Fu;
#pragma unroll 1
    for (int r = warp; r < HC; r += 4) {
      const int hp = r / COLS, col = c0 + r % COLS, ch = lane * 4;
      const int head = (hg * HP + hp) * p.group + col % p.group;
      float x[4] = {0.f, 0.f, 0.f, 0.f};
      if (col < columns && hg * HP + hp < a.kv_heads && (HP == 1 || lane / 16 == hp)) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                        (int64_t)(tok0 + col / p.group) * a.q_stride + head * a.D +
                                                        ch - hp * 64);
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
      }
      uint32_t m = __float_as_uint(max3_abs_nan(max3_abs_nan(x[0], x[1], x[2]), x[3], 0.f));
#pragma unroll
      for (int o = 1; o <= 4; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      // largest magnitude in [128, 256): its first term's rounding leaves at most
      // 8, which the second term holds times 32 to the last bit, of elements down to
      // 2^-7; below, its step is 2^-14
      const int e = (int)(m >> 23);
      const uint32_t sc = e == 255 ? 255u : (uint32_t)max(e - 7, 5);
      const float inv = mx_inverse_scale(sc);
      uint32_t w1 = 0u, w2 = 0u;
      if (sc != 255u) {
        float y[4], z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = x[i] * inv;
        w1 = cvt4_e4m3(y[0], y[1], y[2], y[3]);
        const float2 f0 = unpack_h2(cvt_h2_e4m3((uint16_t)w1)), f1 = unpack_h2(cvt_h2_e4m3((uint16_t)(w1 >> 16)));
        z[0] = (y[0] - f0.x) * 32.f, z[1] = (y[1] - f0.y) * 32.f, z[2] = (y[2] - f1.x) * 32.f, z[3] = (y[3] - f1.y) * 32.f;
        w2 = cvt4_e4m3(z[0], z[1], z[2], z[3]);
      }
      auto put = [&](int row, uint32_t w, uint32_t s) {   // row of its head
        *reinterpret_cast<uint32_t*>(smem + C::Q + (hp * C::N1H + row) * 128 + (((lane >> 2) ^ (row & 7)) << 4) +
                                     (lane & 3) * 4) = w;
        if ((lane & 7) == 0) smem[C::SFQ + hp * 512 + (row & 31) * 16 + (lane >> 3)] = (unsigned char)s;
      };
      put(r % COLS, w1, sc);
      put(COLS + r % COLS, w2, sc == 255u ? 255u : sc - 5u);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);

    // ---- running reference (log2) and sum of each query, the same reference in every thread
    float M[HC], l[HC];
    float M_own = NONE;   // of query `lane`
    bool far = false;     // some query's reference (a block's power, with up to four queries) is beyond FAR
#pragma unroll
    for (int c = 0; c < HC; ++c) M[c] = NONE, l[c] = 0.f;
    const float sl2 = a.scale * 1.4426950408889634f;
    const bool steps = a.causal || a.window > 0;
    // bits of the columns that are queries: a token that only the others would see is hidden
    uint32_t exist = 0u;
#pragma unroll
    for (int h = 0; h < HP; ++h) exist |= (0xFFFFFFFFu >> (32 - min(COLS, columns - c0))) << (h * COLS);
    const int vs_at = (hg * KV_ROWS + KV_VS_ROW) * 64 + key * 4;
    const int64_t page_bytes = a.kv.groups * KV_GROUP_BYTES;
    int page = 0, next_page = nt > 0 ? table[0] : -1;
    uint32_t vs = 0u, next_vs = 0u;
    if (next_page >= 0 && next_page < a.kv.pages)
      next_vs = *reinterpret_cast<const uint32_t*>(a.kv.cache + next_page * page_bytes + vs_at);
    int t = 0;
#pragma unroll 1
    for (; t < nt; ++t) {
      page = next_page, vs = next_vs;
      next_page = t + 1 < nt ? table[t + 1] : -1;
      if (next_page >= 0 && next_page < a.kv.pages)
        next_vs = *reinterpret_cast<const uint32_t*>(a.kv.cache + next_page * page_bytes + vs_at);
      const int j0 = (first + t) * KV_PAGE, j = j0 + key;
      const int sb = t % SB;
      // ---- what is hidden
      const bool there = page >= 0 && page < a.kv.pages && j < len;
      uint32_t seen = there ? exist : 0u;   // bit c: query c sees this token
      if (steps && ((a.causal && j0 + KV_PAGE - 1 > past + i_first) || (a.window > 0 && j0 <= past + i_last - a.window))) {
#pragma unroll
        for (int c = 0; c < COLS; ++c) {
          const int at = past + (c0 + c) / p.group;
          if ((a.causal && j > at) || (a.window > 0 && j <= at - a.window)) {
#pragma unroll
            for (int h = 0; h < HP; ++h) seen &= ~(1u << (h * COLS + c));
          }
        }
      }
      // V's scales relative to the largest among the warp's seen tokens
      // NaN codes apart: they are rare and dealt with where P is written
      const uint32_t bad = seen ? __vcmpeq4(vs, 0xFFFFFFFFu) : 0u, codes = seen ? vs & ~bad : 0u;
      const bool any_nan = __any_sync(0xFFFFFFFFu, bad != 0u);
      uint32_t ref[4], fac[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t code = codes >> (8 * g) & 255u;
        ref[g] = __reduce_max_sync(0xFFFFFFFFu, code);
        // 2^(code - reference) in fp16, twice; nothing below 2^-30
        const float f = __uint_as_float((uint32_t)(max((int)code - (int)ref[g], -30) + 127) << 23);
        fac[g] = pack_h2(f, f);
      }
      bool ok = mbar_wait(&s_full[sb], (uint32_t)(t / SB) & 1u, a.err);
      tc_fence_after();
      float s[HC];
      {
        float u[HC];
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          tmem_ld<COLS>(t_s + my + sb * N1 + h * C::N1H, s + h * COLS);
          tmem_ld<COLS>(t_s + my + sb * N1 + h * C::N1H + COLS, u + h * COLS);
        }
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < HC; ++c) s[c] += u[c];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[sb]);
      float m_own = -INFINITY, bias[HC];
      bool beyond = false;
#pragma unroll
      for (int c = 0; c < HC; ++c) {
        if (!(seen >> c & 1u)) s[c] = -INFINITY;
        const float m = ceilf(warp_max_nan(s[c]) * sl2);
        bias[c] = m;
        beyond |= m > M[c] + LAZY;
        if (lane == c) m_own = m;
      }
      if (!ok) *failed = 1;
      if (named_bar_or(1, 128, beyond || !ok)) {
        // a weight beyond the reference (or a wait that ran out): all warps agree on a new one
        if (lane < HC) red[warp * 32 + lane] = m_own;
        if (named_bar_or(1, 128, !ok || *failed)) {
          ok = false;
          break;
        }
        if (t > 0) {
          if (!mbar_wait(p_free, (uint32_t)(t - 1) & 1u, a.err)) *failed = 1;
          tc_fence_after();
        }
        float keep[HC];
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          // (fmaxf passes over NaNs; a query that has seen nothing keeps NONE)
          const float m = fmaxf(fmaxf(red[c], red[32 + c]), fmaxf(red[64 + c], red[96 + c]));
          const float to = m > M[c] ? m : M[c];
          keep[c] = ex2(M[c] - to);
          M[c] = to;
          l[c] *= keep[c];
          if (lane == c) M_own = to;
        }
        if (t > 0) {
#pragma unroll
          for (int n = 0; n < N2; n += 4) {
            float o[4];
            tmem_ld4(t_o + my + n, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] *= keep[(HP == 2 ? ((n + i) / COLS >> 2) * COLS : 0) + (n + i) % COLS];
            tmem_st4(t_o + my + n, o);
          }
          tmem_wait_st();
        }
        if (COLS > 4) far = __any_sync(0xFFFFFFFFu, fabsf(M_own) > FAR && M_own != NONE);
        named_bar_sync(1, 128);   // `red` is read
      }
      // ---- weights, times 2^8 / the block's power of two
      // From references of FAR on the product s * sl2 is rounded by itself, as the block's power
      // was: rounded once with the difference it exceeds the power by up to half the last
      // bit, and P / scale e4m3's range.  (A block whose power is FAR from the reference adds
      // nothing.)  The difference takes the score's place, and the factor and the power's
      // are 1 and 0.  With up to four queries a tile's votes and a question for each weight
      // cost less: 64 streams of 4096 to 8192 tokens 91 us for 93; with 16 queries 46 for 39
      // (16 sequences of 2048 tokens x 8 heads of 64 channels).
      constexpr bool ASK = COLS <= 4;
      if (ASK) far = __any_sync(0xFFFFFFFFu, fabsf(m_own) > FAR && m_own != -INFINITY);
      const bool swapped = !ASK && far;
      const float mul = swapped ? 1.f : sl2, less = swapped ? 0.f : -1.f;
      if (swapped) {
#pragma unroll
        for (int c = 0; c < HC; ++c) {
          const float m = bias[c] == -INFINITY ? 0.f : bias[c];   // (all hidden: the scores stay -inf)
          s[c] = fabsf(m) > FAR ? __fadd_rn(__fmul_rn(s[c], sl2), -m) : fmaf(s[c], sl2, -m);
        }
      }
      uint32_t hi2[HC / 2], lo2[HC / 2];
#pragma unroll
      for (int c = 0; c < HC; c += 2) {
        float w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float m = bias[c + i], d = m - M[c + i];
          // below 2^-60 of the reference a block adds nothing
          float x = fmaf(s[c + i], mul, d >= -60.f ? fmaf(m, less, 8.f) : NONE);
          if (ASK && far && fabsf(m) > FAR) x = d >= -60.f ? __fadd_rn(__fmul_rn(s[c + i], sl2), -m) + 8.f : NONE;
          w[i] = ex2(x);
          l[c + i] = fmaf(w[i], ex2(d), l[c + i]);
        }
        const uint32_t h = cvt_h2_e4m3(cvt_e4m3(w[0], w[1]));
        const float2 f = unpack_h2(h);
        hi2[c / 2] = h;
        lo2[c / 2] = pack_h2((w[0] - f.x) * 32.f, (w[1] - f.y) * 32.f);
      }
      if (t > 0 && !mbar_wait(p_free, (uint32_t)(t - 1) & 1u, a.err)) *failed = 1;
      uint32_t word[4];   // two queries: all of a token's columns
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int h0 = HP == 2 ? (g >> 1) * COLS : 0;
        constexpr int W = COLS < 4 ? 1 : COLS / 4;
        uint32_t w1[W], w2[W];
        if constexpr (COLS == 2) {
          w1[0] = cvt_e4m3_h2(mul_h2(hi2[h0 / 2], fac[g]));
          w2[0] = cvt_e4m3_h2(mul_h2(lo2[h0 / 2], fac[g]));
        } else {
#pragma unroll
          for (int c = 0; c < COLS; c += 4) {
            const int at = (h0 + c) / 2;
            w1[c / 4] = cvt_e4m3_h2(mul_h2(hi2[at], fac[g])) | cvt_e4m3_h2(mul_h2(hi2[at + 1], fac[g])) << 16;
            w2[c / 4] = cvt_e4m3_h2(mul_h2(lo2[at], fac[g])) | cvt_e4m3_h2(mul_h2(lo2[at + 1], fac[g])) << 16;
          }
        }
        if (any_nan && (vs >> (8 * g) & 255u) == 255u) {   // a NaN among V: in every query that sees it
#pragma unroll
          for (int c = 0; c < COLS; ++c) {
            const uint32_t nan = 0x7Fu << (8 * (c & 3)), clear = ~(0xFFu << (8 * (c & 3)));
            w1[c / 4] = (w1[c / 4] & clear) | (seen >> (h0 + c) & 1u ? nan : 0u);
            w2[c / 4] &= clear;
          }
        }
        if constexpr (COLS == 16) {
          *reinterpret_cast<uint4*>(smem + C::P + p_at<C::PITCH>(key, 2 * g)) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
          *reinterpret_cast<uint4*>(smem + C::P + p_at<C::PITCH>(key, 2 * g + 1)) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
        } else if constexpr (COLS == 8) {
          *reinterpret_cast<uint4*>(smem + C::P + p_at<C::PITCH>(key, g)) = make_uint4(w1[0], w1[1], w2[0], w2[1]);
        } else if constexpr (COLS == 4) {
          *reinterpret_cast<uint2*>(smem + C::P + p_at<C::PITCH>(key, g >> 1) + (g & 1) * 8) = make_uint2(w1[0], w2[0]);
        } else {
          word[g] = w1[0] | w2[0] << 16;
        }
      }
      if constexpr (COLS == 2)
        *reinterpret_cast<uint4*>(smem + C::P + p_at<C::PITCH>(key, 0)) = make_uint4(word[0], word[1], word[2], word[3]);
      // the block's scales: 2^(V's reference + the block's power of two - the query's reference), 2^-5 for second terms
#pragma unroll
      for (int i = 0; i < (N2 + 31) / 32; ++i) {
        const int at = i * 32 + lane, g = at / COLS;   // (with two queries the upper lanes write places of no column)
        const float d = __shfl_sync(0xFFFFFFFFu, m_own - M_own, (HP == 2 ? (g >> 2) * COLS : 0) + at % COLS);
        uint32_t r = ref[0];
#pragma unroll
        for (int k = 1; k < 4; ++k) r = (g >> 1) == k ? ref[k] : r;
        const int e = (int)r + (int)fminf(fmaxf(d, -60.f), LAZY) - 5 * (g & 1);
        smem[C::SFP + (at & 31) * 16 + (at >> 5) * 4 + warp] = (unsigned char)min(max(e, 0), 254);
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
    // ---- epilogue
    bool ok = t == nt;
    if (nt > 0 && ok && !mbar_wait(p_free, (uint32_t)(nt - 1) & 1u, a.err)) *failed = 1;
    tc_fence_after();
#pragma unroll
    for (int c = 0; c < HC; ++c) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) l[c] += __shfl_xor_sync(0xFFFFFFFFu, l[c], o);
      if (lane == c) red[warp * 32 + c] = l[c];
    }
    named_bar_sync(1, 128);
    if (*failed == 0) {
      const int hp = HP == 2 ? warp >> 1 : 0, head0 = (hg * HP + hp) * p.group;
      const int ch = HP == 2 ? (warp & 1) * 32 + lane : warp * 32 + lane;
      float o[COLS], u[COLS];
      if (nt > 0) {
        tmem_ld<COLS>(t_o + my + 2 * warp * COLS, o);
        tmem_ld<COLS>(t_o + my + (2 * warp + 1) * COLS, u);
        tmem_wait_ld();
      }
#pragma unroll
      for (int c = 0; c < COLS; ++c) {
        const int col = c0 + c;
        if (col >= columns || hg * HP + hp >= a.kv_heads) continue;
        const int64_t at = (int64_t)(tok0 + col / p.group) * a.heads + head0 + col % p.group;
        const float* r = red + hp * COLS + c;
        const float sum = (r[0] + r[32]) + (r[64] + r[96]);
        const float v = nt > 0 ? o[c] + u[c] : 0.f;
        if (p.splits == 1) {
          static_cast<__nv_bfloat16*>(a.y)[at * a.D + ch] = __float2bfloat16_rn(sum == 0.f ? 0.f : v / sum);
        } else {
          const int64_t part = (int64_t)split * a.T * a.heads + at;
          p.part_o[part * a.D + ch] = sum == 0.f ? 0.f : v;
          if (lane == 0 && (HP == 1 ? warp == 0 : (warp & 1) == 0)) {
            float m = M[0];
#pragma unroll
            for (int k = 1; k < HC; ++k) m = k == hp * COLS + c ? M[k] : m;
            p.part_ml[part] = make_float2(m, sum);
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
}

// ------------------------------------------------------------------ joining the parts
struct JoinParams {
  const float* part_o;
  const float2* part_ml;
  __nv_bfloat16* y;
  const int* cu;
  int64_t rows, T;     // rows = T heads
  int splits, D, B, heads, max_q;
};
// A warp a row (a token's head): the parts relative to the largest reference, in order.
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ JoinParams p) {
  dependency_wait();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= p.rows) return;
  // tokens of no sequence (before the first, behind the last, past max_q) have no parts, nor
  // have those of a sequence that reaches behind the call's arrays
  const int t = (int)(row / p.heads);
  int start = -1;
  for (int b0 = 0; b0 < p.B && start < 0; b0 += 32) {
    const int b = b0 + lane;
    int at = -1;
    if (b < p.B && p.cu[b] <= t && t < p.cu[b + 1] && p.cu[b + 1] <= p.T) at = p.cu[b];
    start = __reduce_max_sync(0xFFFFFFFFu, at);
  }
  if (start < 0 || t - start >= p.max_q) return;
  // the parts' factors: lane s has parts s and 32 + s (64 at most)
  float2 ml[2];
  float top = NONE;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 32 * i + lane;
    ml[i] = s < p.splits ? p.part_ml[s * p.rows + row] : make_float2(NONE, 0.f);
    top = fmaxf(top, ml[i].x);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  float f[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) f[i] = ml[i].y == 0.f ? 0.f : ex2(ml[i].x - top);   // (0: it saw nothing)
  // sums in the parts' order; a lane has four (or two) channels, eight loads in flight
  float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const bool wide = p.D == 128;
#pragma unroll 8
  for (int s = 0; s < p.splits; ++s) {
    const float l = __shfl_sync(0xFFFFFFFFu, s < 32 ? ml[0].y : ml[1].y, s & 31);
    const float w = __shfl_sync(0xFFFFFFFFu, s < 32 ? f[0] : f[1], s & 31);
    const float* src = p.part_o + (s * p.rows + row) * p.D;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if (wide) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(src) + lane);
      v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    } else {
      const float2 u = __ldcg(reinterpret_cast<const float2*>(src) + lane);
      v[0] = u.x, v[1] = u.y;
    }
    sum = fmaf(l, w, sum);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = l == 0.f ? o[k] : fmaf(v[k], w, o[k]);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = sum == 0.f ? 0.f : o[k] / sum;
  if (wide) *reinterpret_cast<uint2*>(p.y + row * 128 + lane * 4) = make_uint2(mx_pack_bf16(o[0], o[1]), mx_pack_bf16(o[2], o[3]));
  else *reinterpret_cast<uint32_t*>(p.y + row * 64 + lane * 2) = mx_pack_bf16(o[0], o[1]);
}

// ------------------------------------------------------------------ host
int pick_cols(int64_t columns) { return columns <= 2 ? 2 : columns <= 4 ? 4 : columns <= 8 ? 8 : 16; }

// From this many queries a key head on keys and values are decoded (oq_kv4_chunk.cu).
// Measured (us), this form and that one at 32, 48 and 64 queries: one sequence of 8192 x 40
// heads 52 and 76, 67 and 77, 92 and 78; 8 of 4096 x 8 heads 40 and 61, 63 and 61, 63 and
// 61; 16 of 2048 x 8 heads 37 and 56, 64 and 56, 71 and 57; 32 of 300 x 8 heads 30 and 40,
// 44 and 40, 58 and 41; 4 of 4096 x 16 heads of 64 channels 50 and 43, 61 and 43, 75 and 43.
constexpr int64_t CHUNK = 48;

// Parts of a cache.  A CTA costs what seven tiles do besides its tiles (its chain of
// first loads, the first reference, the epilogue: 8 us at three CTAs an SM), joining
// parts about three; the number of parts with the shortest sum of rounds is taken.
// Measured (us): one token over 32760 x 40 heads 11 parts (one round) 37.7, 22 46.0, 32
// 53.7; 64 streams of 4096 to 8192 tokens x 8 heads 1 part 103.5, 3 91.5, 4 90.5.
int splits_of(int groups, int kv_heads, int B, int group, int max_q, int max_len, int window, int sms) {
  const int64_t columns = (int64_t)max_q * group;
  const int64_t seen = window > 0 ? std::min<int64_t>(max_len, (int64_t)window + max_q) : max_len;
  const int64_t tiles = std::max<int64_t>((seen + KV_PAGE - 1) / KV_PAGE, 1);
  if (columns >= CHUNK) return kv4_chunk_splits(kv_heads, B, group, max_q, tiles, sms);
  const int cols = pick_cols(columns);
  const int64_t ctas = (columns + cols - 1) / cols * groups * B, slots = (cols <= 4 ? 3 : 2) * (int64_t)sms;
  int best = 1;
  int64_t least = 0;
  for (int s = 1; s <= 64 && s <= tiles; ++s) {
    const int64_t cost = (ctas * s + slots - 1) / slots * (7 + (tiles + s - 1) / s) + (s > 1 ? 3 : 0);
    if (s == 1 || cost < least) best = s, least = cost;
  }
  return best;
}

size_t part_bytes(int splits, int64_t T, int heads, int D) {
  if (splits == 1) return 0;
  return (size_t)splits * (size_t)T * heads * ((size_t)D * 4 + 8) + 256;
}

template <int COLS, int HP>
oq_status launch(AttnParams& p, cudaStream_t st, int device) {
  using C = Cfg<COLS, HP>;
  static std::atomic<uint64_t> smem_set{0};
  const oq_status r = mx_allow_smem(reinterpret_cast<const void*>(attention_kernel<COLS, HP>), C::SMEM, device, &smem_set);
  if (r != OQ_OK) return r;
  const int64_t columns = (int64_t)p.a.max_q * p.group;
  const dim3 grid((unsigned)((columns + COLS - 1) / COLS), (unsigned)(p.a.kv.groups * p.splits), (unsigned)p.a.kv.B);
  const cudaError_t e = mx_launch(attention_kernel<COLS, HP>, grid, NTHREADS, C::SMEM, 0, st, p);
  if (e != cudaSuccess) {
    set_error(std::string("attention launch: ") + cudaGetErrorString(e));
    return OQ_ERR_CUDA;
  }
  return OQ_OK;
}

template <int HP>
oq_status launch_cols(AttnParams& p, int cols, cudaStream_t st, int device) {
  switch (cols) {
    case 2: return launch<2, HP>(p, st, device);
    case 4: return launch<4, HP>(p, st, device);
    case 8: return launch<8, HP>(p, st, device);
    default: return launch<16, HP>(p, st, device);
  }
}

}  // namespace

size_t kv4_attention_workspace(const oq_kv4* kv, int64_t T, int B, int max_q, int max_len) {
  // (a window only lowers the number of parts: the call takes no more than without one)
  int dev = 0;
  return part_bytes(splits_of(kv->groups, kv->kv_heads, B, kv->heads / kv->kv_heads, max_q, max_len, 0, mx_sm_count(&dev)), T,
                    kv->heads, kv->head_dim);
}

oq_status kv4_attention_launch(const AttentionArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  AttnParams p;
  std::memset(&p.map, 0, sizeof(p.map));
  p.a = a;
  p.group = a.heads / a.kv_heads;
  int dev = 0;
  const int sms = mx_sm_count(&dev);
  p.splits = splits_of(a.kv.groups, a.kv_heads, a.kv.B, p.group, a.max_q, a.max_len, 0, sms);
  if (a.window > 0)
    p.splits = std::min(p.splits, splits_of(a.kv.groups, a.kv_heads, a.kv.B, p.group, a.max_q, a.max_len, a.window, sms));
  if (a.workspace_bytes < part_bytes(p.splits, a.T, a.heads, a.D)) {
    set_error("oq_kv4_attention: the workspace is too small");
    return OQ_ERR_INVALID_ARG;
  }
  const int64_t rows = a.T * a.heads;
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + (size_t)p.splits * rows * a.D);
  oq_status r;
  if ((int64_t)a.max_q * p.group >= CHUNK) {
    r = kv4_chunk_launch(p, st, dev);
  } else {
    const cuuint64_t dims[2] = {128, (cuuint64_t)(a.kv.pages * a.kv.groups * KV_ROWS)};
    const cuuint64_t strides[1] = {64};
    const cuuint32_t box[2] = {128, 128};
    r = mx_encode(&p.map, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 2, a.kv.cache, dims, strides, box,
                  CU_TENSOR_MAP_SWIZZLE_128B, "the cache");
    if (r != OQ_OK) return r;
    const int cols = pick_cols((int64_t)a.max_q * p.group);
    r = a.D == 128 ? launch_cols<1>(p, cols, st, dev) : launch_cols<2>(p, cols, st, dev);
  }
  if (r != OQ_OK || p.splits == 1) return r;
  JoinParams j;
  j.part_o = p.part_o;
  j.part_ml = p.part_ml;
  j.y = static_cast<__nv_bfloat16*>(a.y);
  j.cu = a.kv.cu;
  j.rows = rows;
  j.T = a.T;
  j.splits = p.splits;
  j.D = a.D;
  j.B = a.kv.B;
  j.heads = a.heads;
  j.max_q = a.max_q;
  const cudaError_t e = mx_launch(join_kernel, dim3((unsigned)((rows + 3) / 4)), 128, 0, 0, st, j);
  if (e != cudaSuccess) {
    set_error(std::string("attention join launch: ") + cudaGetErrorString(e));
    return OQ_ERR_CUDA;
  }
  return OQ_OK;
}

}  // namespace oq
