// Attention over the 4-bit paged cache for many query tokens (chunks): the form of
// oq_kv4_attention.cu, whose products read the codes as they lie, spends five times
// the products' work on the scales; from some dozens of queries a key head on it
// pays to decode a tile of keys and values once, to bf16 in shared memory, for 256
// queries.
//   S [128 queries x 128 tokens] = q K^T,  P = 2^(S - reference),  O += P V
// kind::f16 MMAs on bf16 (q and K enter exactly, P rounded to bf16).  Two tiles of 128
// queries take turns: while the tensor cores do one's P V and next S, the other's
// four warps form P, a thread a query, no shuffles.  P takes S's place in tensor
// memory and is the second product's A operand from there.  The reference is moved
// (and O rescaled) only when a weight exceeds it by 2^8, once a tile at most.
//
// Decoding: e2m1's bits s e e m shifted into a bf16's sign, exponent and mantissa are
// its value times 2^-126, exactly (subnormals too); two products bring in 2^126 and
// the scale.  Two elements four apart in a word are done at once; so channels (of
// keys) and tokens (of values) lie permuted within each eight, and q's channels and
// P's tokens are taken in the same order.
//
// Bound: a query tile's softmax and the MMAs in turn (S of the next tile waits for P V of this
// one, since P lies in S's place), with the decoding beside them; no unit is full: issue
// slots 52 % active, the tensor pipe and the exponential unit 35 %.  Measured, 1560 queries over
// 7800 tokens x 40 heads of 128: 381 us, 654 TFLOP/s (154 us at the rate of a large
// library product).  Four decoding warps and two passes over S took 448.
//
// Warps: 0-3 and 4-7 the two query tiles, 8-15 decoding, 16 tensor memory and MMAs
// (17-19 only give up registers).
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "oq_kv4.cuh"
#include "oq_mx_ptx.cuh"

namespace oq {
namespace {

constexpr int QT = 128;                       // queries of a tile
constexpr int DEC_WARP = 8, MMA_WARP = 16, NTHREADS = 20 * 32, DEC_THREADS = 256;
// registers of a thread of each four warps; together the launch's 640 x 96
constexpr int SOFTMAX_REGS = 136, DECODE_REGS = 80, MMA_REGS = 48;
static_assert(2 * SOFTMAX_REGS + 2 * DECODE_REGS + MMA_REGS == 5 * 96, "more would wait for good");
constexpr float LAZY = 8.f, NONE = -3.4028234e38f;   // as in oq_kv4_attention.cu
constexpr float FAR = 4194304.f;              // 2^22: the last bit of a reference is half a unit of log2

template <int D>
struct Cfg {
  static constexpr int Q = QT * D * 2, KT = KV_PAGE * D * 2;        // a tile of queries; of keys or values
  static constexpr int K0 = 2 * Q, V0 = K0 + 2 * KT;
  static constexpr int VS = V0 + 2 * KT;                            // V's scales: [2][D / 32][128] bf16
  static constexpr int NANS = VS + 2 * (D / 32) * 256;              // [4][2 x 128] bits of NaN blocks
  static constexpr int BAR = NANS + 1024;
  static constexpr size_t SMEM = 1024 + BAR + 8 * 18 + 64;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr uint32_t S = 0, O = 2 * 128;                     // tensor memory columns: S of both tiles, O
};

__device__ __forceinline__ float ex2(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// elements j and j + 4 of a word of eight codes, times 2^-126, as bf16
template <int J>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  const uint32_t sign = J == 3 ? w : w << (12 - 4 * J);
  const uint32_t mag = J == 0 ? w << 6 : J == 1 ? w << 2 : J == 2 ? w >> 2 : w >> 6;
  return (sign & 0x80008000u) | (mag & 0x01C001C0u);
}
constexpr uint32_t BIG = 0x7E807E80u;   // 2^126, twice
// a scale code as bf16 bits (255, NaN, included)
__device__ __forceinline__ uint32_t scale_bits(uint32_t code) {
  return code == 0u ? 0x0040u : code == 255u ? 0x7FC0u : code << 7;
}

// 16 tensor-memory columns of a warp's 32 lanes
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// D += A B^T with A (bf16 pairs) in tensor memory
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// byte offset of 16-byte chunk c (of a row's elements) in K-major tiles of 128 rows x 128 bytes
__device__ __forceinline__ uint32_t tile_at(int row, int c) {
  return (uint32_t)((c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}
// the same for D = 64 values, whose tiles have 64 rows
template <int ROWS>
__device__ __forceinline__ uint32_t rows_at(int row, int c) {
  return (uint32_t)((c >> 3) * (ROWS * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1) chunk_kernel(const __grid_constant__ AttnSplit p) {
  using C = Cfg<D>;
  constexpr int BLK = D / 32;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::BAR);
  uint64_t* k_free = k_full + 2;
  uint64_t* v_full = k_free + 2;
  uint64_t* v_free = v_full + 2;
  uint64_t* s_full = v_free + 2;    // of each query tile
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 2;
  uint64_t* q_full = pv_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 1);
  int* any_nan = reinterpret_cast<int*>(tmem_slot + 1);   // [4] the last tile (from 1) with a NaN block among its values

  const AttentionArgs& a = p.a;
  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 8), mbar_init(&k_free[i], 1), mbar_init(&v_full[i], 8), mbar_init(&v_free[i], 1);
      mbar_init(&s_full[i], 1), mbar_init(&p_full[i], 4), mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, 8);
    any_nan[0] = any_nan[1] = any_nan[2] = any_nan[3] = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // (a kernel that may start from here finds this CTA's tensor memory allocated)
  dependency_wait();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0), smem_base = smem_u32(smem);
  const int head = (int)blockIdx.y / p.splits, split = (int)blockIdx.y % p.splits, b = (int)blockIdx.z;   // key head
  const int hg = head * D / 128, half = D == 64 ? head & 1 : 0;
  const int tok0 = a.kv.cu[b], end = a.kv.cu[b + 1], len = min(a.kv.lens[b], a.kv.width * KV_PAGE);
  // a sequence that the call's arrays do not hold has no queries
  const int n = tok0 < 0 || end > a.T || end < tok0 ? 0 : end - tok0;
  const int past = a.kv.lens[b] - n;                   // place of the first query token
  const int c0 = (int)blockIdx.x * 2 * QT, columns = min(n, a.max_q) * p.group;
  const bool work = c0 < columns;
  const int qtiles = c0 + QT < columns ? 2 : 1;
  const int i_first = c0 / p.group, i_last = (min(c0 + 2 * QT, columns) - 1) / p.group;
  // tokens [lo, hi) that any of these queries sees; this CTA's share of their tiles
  int hi = a.causal ? min(len, past + i_last + 1) : len, lo = 0;
  if (a.window > 0) lo = max(0, past + i_first - a.window + 1);
  const int tile_lo = lo / KV_PAGE, tiles = work && hi > lo ? (hi + KV_PAGE - 1) / KV_PAGE - tile_lo : 0;
  const int first = tile_lo + (int)((int64_t)tiles * split / p.splits);
  const int nt = tile_lo + (int)((int64_t)tiles * (split + 1) / p.splits) - first;
  const int* table = a.kv.table + (int64_t)b * a.kv.width + first;

  if (warp >= MMA_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(MMA_REGS));
    if (warp == MMA_WARP) {
    constexpr uint32_t idesc1 = idesc_bf16_f32(QT, KV_PAGE), idesc2 = idesc_bf16_f32(QT, D);
    const uint32_t lead = elect_one();
    const uint64_t base = smem_desc_sw128(smem_base);
    bool ok = nt > 0 && __all_sync(0xFFFFFFFFu, mbar_wait(q_full, 0u, a.err));
    auto wait = [&](uint64_t* bar, int phase) {
      ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(bar, (uint32_t)phase & 1u, a.err));
      tc_fence_after();
    };
    auto mma_s = [&](int q, int t) {
      if (lead) {
        const uint64_t qd = base + (q * C::Q >> 4), kd = base + ((C::K0 + (t & 1) * C::KT) >> 4);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t at = (uint32_t)((k >> 2) * (128 * 128) + (k & 3) * 32) >> 4;
          tc_mma_f16_ss(tmem + C::S + q * 128, qd + at, kd + at, idesc1, k > 0);
        }
        tc_commit(&s_full[q]);
      }
      __syncwarp();
    };
    auto mma_o = [&](int q, int t) {
      if (lead) {
        const uint64_t vd = base + ((C::V0 + (t & 1) * C::KT) >> 4);
#pragma unroll
        for (int k = 0; k < KV_PAGE / 16; ++k)
          tc_mma_f16_ts(tmem + C::O + q * 128, tmem + C::S + q * 128 + k * 8,
                        vd + ((uint32_t)((k >> 2) * (D * 128) + (k & 3) * 32) >> 4), idesc2, t > 0 || k > 0);
        tc_commit(&pv_done[q]);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (lead) tc_commit(bar);
      __syncwarp();
    };
    if (ok) wait(&k_full[0], 0);
    if (ok) {
      mma_s(0, 0);
      if (qtiles == 2) mma_s(1, 0);
      commit(&k_free[0]);
    }
    for (int t = 0; ok && t < nt; ++t) {
      wait(&v_full[t & 1], t >> 1);
      if (ok) wait(&p_full[0], t);
      if (!ok) break;
      mma_o(0, t);
      if (t + 1 < nt) {
        wait(&k_full[(t + 1) & 1], (t + 1) >> 1);
        if (!ok) break;
        mma_s(0, t + 1);
      }
      if (qtiles == 2) {
        wait(&p_full[1], t);
        if (!ok) break;
        mma_o(1, t);
      }
      commit(&v_free[t & 1]);
      if (t + 1 < nt) {
        if (qtiles == 2) mma_s(1, t + 1);
        commit(&k_free[(t + 1) & 1]);
      }
    }
    __syncwarp();
    }
  } else if (warp >= DEC_WARP) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(DECODE_REGS));
    if (nt > 0) {
    // ---- decoding: a thread has half of a token's keys, and a channel's values of 64 or 32 tokens
    const int th = (int)threadIdx.x - DEC_WARP * 32;
    constexpr int NW = D / 16;                 // words of a thread, of keys and of values
    const int key = th & 127, kpart = th >> 7, ch = th % D, vpart = th / D;
    const int64_t page_bytes = a.kv.groups * KV_GROUP_BYTES, group_at = hg * KV_GROUP_BYTES;
    uint4 kr[NW / 4], vr[NW / 4];
    uint32_t ksr = 0u, vsr = 0u;
    const uint8_t* page_k = nullptr;           // the fetched tile's group, or null: not there
    auto find = [&](int t) -> const uint8_t* {
      const int page = t < nt ? table[t] : -1;
      return page >= 0 && page < a.kv.pages ? a.kv.cache + page * page_bytes + group_at : nullptr;
    };
    auto fetch_k = [&](const uint8_t* g) {
      ksr = vsr = 0u;
#pragma unroll
      for (int i = 0; i < NW / 4; ++i) kr[i] = make_uint4(0u, 0u, 0u, 0u);
      if (g) {
#pragma unroll
        for (int i = 0; i < NW / 4; ++i) kr[i] = __ldcg(reinterpret_cast<const uint4*>(g + key * 64 + half * 32 + kpart * (NW * 4)) + i);
        ksr = __ldcg(reinterpret_cast<const uint32_t*>(g + KV_KS_ROW * 64) + mx_tile_word(key));
        vsr = __ldcg(reinterpret_cast<const uint32_t*>(g + KV_VS_ROW * 64) + key);
      }
    };
    auto fetch_v = [&](const uint8_t* g) {
#pragma unroll
      for (int i = 0; i < NW / 4; ++i) vr[i] = make_uint4(0u, 0u, 0u, 0u);
      if (g) {
#pragma unroll
        for (int i = 0; i < NW / 4; ++i)
          vr[i] = __ldcg(reinterpret_cast<const uint4*>(g + (KV_V_ROW + half * 64 + ch) * 64 + vpart * (NW * 4)) + i);
      }
    };
    page_k = find(0);
    const uint8_t* page_next = find(1);
    fetch_k(page_k);
    fetch_v(page_k);
    for (int t = 0; t < nt; ++t) {
      const int buf = t & 1;
      const uint8_t* page_after = find(t + 2);
      bool ok = t < 2 || mbar_wait(&k_free[buf], (uint32_t)(t / 2 - 1) & 1u, a.err);
      // V's scales of this thread's token (0 where nobody sees it), NaN blocks apart
      const bool seen = page_k && (first + t) * KV_PAGE + key < len;
      uint32_t nans = 0u;
      {
        uint16_t* vs = reinterpret_cast<uint16_t*>(smem + C::VS) + buf * BLK * 128;
        const int at = (key & ~7) | (key & 3) << 1 | (key >> 2 & 1);   // tokens j, j + 4 side by side
        for (int g = kpart * (BLK / 2); g < (kpart + 1) * (BLK / 2); ++g) {
          const uint32_t code = vsr >> (8 * (g + 2 * half)) & 255u;
          if (seen && code == 255u) nans |= 1u << g;
          vs[g * 128 + at] = (uint16_t)(seen && code != 255u ? scale_bits(code) : 0u);
        }
      }
      // The marks of four tiles are kept: S of tile t - 2 is done, so P of tile t - 3 is.
      if (nans) any_nan[t & 3] = t + 1;        // (the tile's number, so that it need not be cleared)
      smem[C::NANS + (t & 3) * 256 + th] = (unsigned char)nans;
      unsigned char* kt = smem + C::K0 + buf * C::KT;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const uint4& v = kr[i / 4];
        const uint32_t w = i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w;
        const uint32_t s1 = scale_bits(ksr >> (8 * ((kpart * NW + i) / 4 + 2 * half)) & 255u), s = s1 | s1 << 16;
        if (ok)
          *reinterpret_cast<uint4*>(kt + tile_at(key, kpart * NW + i)) =
              make_uint4(mul_bf2(mul_bf2(code_pair<0>(w), BIG), s), mul_bf2(mul_bf2(code_pair<1>(w), BIG), s),
                         mul_bf2(mul_bf2(code_pair<2>(w), BIG), s), mul_bf2(mul_bf2(code_pair<3>(w), BIG), s));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&k_full[buf]);
      fetch_k(page_next);
      ok = ok && (t < 2 || mbar_wait(&v_free[buf], (uint32_t)(t / 2 - 1) & 1u, a.err));
      if (named_bar_or(2, DEC_THREADS, !ok)) break;   // (all of them, or none)
      unsigned char* vt = smem + C::V0 + buf * C::KT;
      const uint4* sc = reinterpret_cast<const uint4*>(smem + C::VS + (buf * BLK + ch / 32) * 256) + vpart * NW;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const uint4& v = vr[i / 4];
        const uint32_t w = i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w;
        const uint4 s = sc[i];
        *reinterpret_cast<uint4*>(vt + rows_at<D>(ch, vpart * NW + i)) =
            make_uint4(mul_bf2(mul_bf2(code_pair<0>(w), BIG), s.x), mul_bf2(mul_bf2(code_pair<1>(w), BIG), s.y),
                       mul_bf2(mul_bf2(code_pair<2>(w), BIG), s.z), mul_bf2(mul_bf2(code_pair<3>(w), BIG), s.w));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&v_full[buf]);
      fetch_v(page_next);
      page_k = page_next;
      page_next = page_after;
    }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(SOFTMAX_REGS));
    if (work) {
    // ---- a query a thread
    const int q = warp >> 2, r = (warp & 3) * 32 + lane, col = c0 + q * QT + r;
    const bool mine = col < columns;
    const int token = mine ? col / p.group : 0;
    const int64_t row = (int64_t)(tok0 + token) * a.heads + head * p.group + col % p.group;
    if (nt > 0) {
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(a.q) + (int64_t)(tok0 + token) * a.q_stride +
                                 (head * p.group + col % p.group) * D;
      unsigned char* dst = smem + q * C::Q;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (mine) v = *reinterpret_cast<const uint4*>(src + 8 * i);
        uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {   // an infinity makes the row NaN, as its differences would
          if ((u[k] & 0x7F80u) == 0x7F80u) u[k] |= 0x40u;
          if ((u[k] & 0x7F800000u) == 0x7F800000u) u[k] |= 0x400000u;
        }
        // channels j, j + 4 side by side
        *reinterpret_cast<uint4*>(dst + tile_at(r, i)) =
            make_uint4(__byte_perm(u[0], u[2], 0x5410), __byte_perm(u[0], u[2], 0x7632), __byte_perm(u[1], u[3], 0x5410),
                       __byte_perm(u[1], u[3], 0x7632));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
    }
    const float sl2 = a.scale * 1.4426950408889634f;
    const int at = past + token;
    const int see_hi = !mine ? 0 : a.causal ? min(len, at + 1) : len, see_lo = a.window > 0 ? max(0, at - a.window + 1) : 0;
    // all queries of the tile see tokens [all_lo, all_hi)
    const int i0 = (c0 + q * QT) / p.group, i1 = (min(c0 + (q + 1) * QT, columns) - 1) / p.group;
    const int all_hi = a.causal ? min(len, past + i0 + 1) : len, all_lo = a.window > 0 ? past + i1 - a.window + 1 : 0;
    const uint32_t t_s = tmem + C::S + q * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t t_o = tmem + C::O + q * 128 + ((uint32_t)((warp & 3) * 32) << 16);
    float M = NONE, l = 0.f;
    bool far = false;   // a reference of the warp's is beyond FAR
    uint32_t nan_blocks = 0u;
    bool ok = true;
    int next_page = nt > 0 ? table[0] : -1;
#pragma unroll 1
    for (int t = 0; t < nt && q < qtiles; ++t) {
      const int j0 = (first + t) * KV_PAGE;
      const int page = next_page;
      next_page = t + 1 < nt ? table[t + 1] : -1;
      const bool there = page >= 0 && page < a.kv.pages;
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[q], (uint32_t)t & 1u, a.err));
      if (!ok) break;
      tc_fence_after();
      const bool whole = there && j0 >= all_lo && j0 + KV_PAGE <= all_hi;
      const int lo_j = (there ? see_lo : 1 << 30) - j0, hi_j = see_hi - j0;
      // 16 scores from column 16 c on, hidden ones -inf
      auto hide = [&](uint32_t (&v)[16], int c) {
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (!(16 * c + i >= lo_j && 16 * c + i < hi_j)) v[i] = 0xFF800000u;
        }
      };
      // P and its sum relative to M, all of it in registers: S is still there if a
      // weight turns out to exceed the reference
      uint32_t w[64];
      float most = 0.f, part_sum = 0.f;
      auto weigh_as = [&](auto apart) {
        f32x2 sum[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
        const f32x2 c2 = pack2(sl2, sl2), m2 = pack2(-M, -M);
        float top[2] = {0.f, 0.f};
        uint32_t v[2][16];
        tmem_ld16(t_s, v[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_wait_ld();
          if (c < 7) tmem_ld16(t_s + 16 * (c + 1), v[(c + 1) & 1]);
          hide(v[c & 1], c);
#pragma unroll
          for (int g = 0; g < 2; ++g)   // tokens j, j + 4 of eight side by side
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float x, y;
              x = __uint_as_float(v[c & 1][8 * g + j]), y = __uint_as_float(v[c & 1][8 * g + j + 4]);
              // (packed products and sums may be fused again; these are not)
              if constexpr (decltype(apart)::value) x = __fadd_rn(__fmul_rn(x, sl2), -M), y = __fadd_rn(__fmul_rn(y, sl2), -M);
              else unpack2(fma2(pack2(x, y), c2, m2), x, y);
              x = ex2(x), y = ex2(y);
              top[j & 1] = fmaxf(fmaxf(top[j & 1], x), y);
              sum[j & 1] = add2(sum[j & 1], pack2(x, y));
              w[8 * c + 4 * g + j] = mx_pack_bf16(x, y);
            }
        }
        float sx, sy;
        unpack2(add2(sum[0], sum[1]), sx, sy);
        part_sum = sx + sy;
        most = fmaxf(top[0], top[1]);
      };
      // From references of FAR on the product s * sl2 is rounded by itself, as the reference
      // was: in one step with the difference its error of half the reference's last bit
      // would be the exponent (weights of 2^128 and 0 from 2^31 on).  Two forms: one that asks
      // for every 16 scores took 408 us where these take 381 (1560 queries over 7800 tokens x
      // 40 heads).
      auto weigh = [&]() {
        if (far) weigh_as(std::true_type());
        else weigh_as(std::false_type());
      };
      bool move = M == NONE && max(lo_j, 0) < min(hi_j, KV_PAGE);   // the first token it sees
      // Weights are formed twice at most: what they are relative to a reference that has
      // moved is taken as it is.  (The new reference comes from top * sl2 rounded, a weight
      // from s * sl2 - M rounded once: at M + 8 one may see 2^8 exceeded and the other not,
      // so that asking again could go on for ever.)
      bool moved = false;
      while (ok) {
        if (moved || !__any_sync(0xFFFFFFFFu, move)) {
          weigh();
          move = most > 256.f;   // 2^LAZY
          if (moved || !__any_sync(0xFFFFFFFFu, move)) break;
        }
        moved = true;
        // the reference moves, and with it what is summed so far
        float top = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          uint32_t v[16];
          tmem_ld16(t_s + 16 * c, v);
          tmem_wait_ld();
          hide(v, c);
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, __uint_as_float(v[i]));
        }
        const float m = top * sl2, to = m > M + LAZY ? ceilf(m) : M, keep = ex2(M - to);
        if (t > 0) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pv_done[q], (uint32_t)(t - 1) & 1u, a.err));
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(t_o + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * keep);
            tmem_st16(t_o + c, o);
          }
        }
        l *= keep;
        M = to;
        far = __any_sync(0xFFFFFFFFu, fabsf(M) > FAR && M != NONE);
      }
      if (!ok) break;
      l += part_sum;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t u[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) u[i] = w[16 * c + i];
        tmem_st16(t_s + 16 * c, u);
      }
      // NaN blocks of values are noted for the queries that see them
      if (any_nan[t & 3] == t + 1) {
        for (int i = max(lo_j, 0); i < min(hi_j, KV_PAGE); ++i) nan_blocks |= smem[C::NANS + (t & 3) * 256 + i] | smem[C::NANS + (t & 3) * 256 + 128 + i];
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[q]);
    }
    if (q < qtiles) {
      if (nt > 0 && ok) ok = __all_sync(0xFFFFFFFFu, mbar_wait(&pv_done[q], (uint32_t)(nt - 1) & 1u, a.err));
      tc_fence_after();
      if (ok) {
        const float inv = p.splits > 1 ? 1.f : l == 0.f ? 0.f : 1.f / l;
        const int64_t part = (int64_t)split * a.T * a.heads + row;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          if (nt > 0) {
            tmem_ld16(t_o + c, o);
            tmem_wait_ld();
          }
          float f[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            f[i] = nan_blocks >> (c / 32) & 1u ? __int_as_float(0x7FC00000) : l == 0.f ? 0.f : __uint_as_float(o[i]) * inv;
          if (mine && p.splits == 1) {
            uint4* y = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.y) + row * D + c);
            y[0] = make_uint4(mx_pack_bf16(f[0], f[1]), mx_pack_bf16(f[2], f[3]), mx_pack_bf16(f[4], f[5]), mx_pack_bf16(f[6], f[7]));
            y[1] = make_uint4(mx_pack_bf16(f[8], f[9]), mx_pack_bf16(f[10], f[11]), mx_pack_bf16(f[12], f[13]),
                              mx_pack_bf16(f[14], f[15]));
          } else if (mine) {
            float4* y = reinterpret_cast<float4*>(p.part_o + part * D + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
          }
        }
        if (mine && p.splits > 1) p.part_ml[part] = make_float2(M, l);
      }
      tc_fence_before();
    }
    }
  }
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D>
oq_status launch(const AttnSplit& p, cudaStream_t st, int device) {
  using C = Cfg<D>;
  static std::atomic<uint64_t> smem_set{0};
  const oq_status r = mx_allow_smem(reinterpret_cast<const void*>(chunk_kernel<D>), C::SMEM, device, &smem_set);
  if (r != OQ_OK) return r;
  const int64_t columns = (int64_t)p.a.max_q * p.group;
  const dim3 grid((unsigned)((columns + 2 * QT - 1) / (2 * QT)), (unsigned)(p.a.kv_heads * p.splits), (unsigned)p.a.kv.B);
  const cudaError_t e = mx_launch(chunk_kernel<D>, grid, NTHREADS, C::SMEM, 0, st, p);
  if (e != cudaSuccess) {
    set_error(std::string("attention launch: ") + cudaGetErrorString(e));
    return OQ_ERR_CUDA;
  }
  return OQ_OK;
}

}  // namespace

int kv4_chunk_splits(int kv_heads, int B, int group, int max_q, int64_t tiles, int sms) {
  const int64_t ctas = ((int64_t)max_q * group + 2 * QT - 1) / (2 * QT) * kv_heads * B;
  return (int)std::max<int64_t>(1, std::min<int64_t>({sms / std::max<int64_t>(ctas, 1), tiles / 4, 64}));
}

oq_status kv4_chunk_launch(const AttnSplit& p, cudaStream_t st, int device) {
  return p.a.D == 128 ? launch<128>(p, st, device) : launch<64>(p, st, device);
}

}  // namespace oq
