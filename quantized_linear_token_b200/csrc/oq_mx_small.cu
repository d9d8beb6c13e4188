// Product of microscaled operands for small batches (one token to a few
// hundred): the weights' stream decides the time, so the weight rows are the
// MMA's M and the batch, padded to BN tokens, its N:
//   y[t, o] = sum_k w[o, k] a[t, k]
// A CTA takes 128 weight rows, and the K range is split over the CTAs of a
// cluster, so that enough CTAs stream weights at once.  Each CTA owns a share of
// the tokens; all send it their fp32 partial sums by bulk copies from shared
// memory to shared memory, and it adds them in rank order: no workspace, no
// atomics, one launch, and the same bits on every call.  (At 256 tokens, 13824
// deep, loading the peers' sums instead took a third of the kernel.)  4-bit activations use kind::mxf4, 8-bit ones
// kind::mxf8f6f4 with the weights' codes spread to 8-bit containers by TMA.
//
// Measured back to back, weights from HBM (600 MB of them in turn): one token
// 13824 -> 5120 (4 bits) 11.9 us, 3.2 TB/s of weights (5.7 us at the copy
// bandwidth; the rest is launch, first loads, the 570 cycles that a stage's four
// scale copies and MMAs take to issue, and the cluster's two barriers); 16 tokens
// 5120 -> 5120 8.7 us (6.9 with the weights in L2); 256 tokens 13824 -> 5120 with
// 8-bit activations 25 us.  Each of its 40 weight tiles brings in the whole batch:
// 36 stages of 41.5 KB a CTA, 15 us at the 99 bytes a nanosecond that an SM takes
// from L2, beside 10 us of MMAs on 120 SMs and 6 us of exchange and sums.
//
// Warps: 0-3 epilogue, 4 TMA producer, 5 tensor memory and MMAs.
#include <algorithm>
#include <cstring>

#include "oq_epilogue.cuh"
#include "oq_mx_ptx.cuh"

namespace oq {
namespace {

constexpr int SM_ROWS = 128;                 // weight rows per CTA
constexpr int W_TILE = SM_ROWS * 128;
constexpr int TMA_WARP = 4, MMA_WARP = 5, NTHREADS = 6 * 32;

template <bool F4, int BN>
struct Cfg {
  static constexpr int CT = F4 ? 2 : 1;                       // scale column tiles per stage
  static constexpr int RT = (BN + MX_ROWS - 1) / MX_ROWS;     // scale row tiles of the batch
  static constexpr int X_TILE = BN * 128;
  static constexpr int SX = (RT * CT * MX_TILE_BYTES + 1023) / 1024 * 1024;
  static constexpr int STAGE = W_TILE + (X_TILE + 1023) / 1024 * 1024 + 1024 + SX;
  // a load that spreads 4-bit codes counts the packed bytes, half of what it writes
  static constexpr uint32_t TX = (F4 ? W_TILE : W_TILE / 2) + X_TILE + (1 + RT) * CT * MX_TILE_BYTES;
  static constexpr int SF_SET = CT * 4 * (1 + RT), SF_SETS = 4;   // scale columns of a stage; sets used in turn
  static constexpr int SF_COLS = SF_SET * SF_SETS;
  static constexpr uint32_t TMEM = BN + SF_COLS <= 32 ? 32 : BN + SF_COLS <= 64 ? 64 : BN + SF_COLS <= 128 ? 128
                                   : BN + SF_COLS <= 256 ? 256 : 512;
  // up to 64 tokens two CTAs share an SM
  static constexpr int BUDGET = BN <= 64 ? 108 * 1024 : 216 * 1024;
  static constexpr int OS = BUDGET / STAGE < 8 ? BUDGET / STAGE : 8;
  static_assert(OS >= 3, "the checks cover three stages");
  // CTAs that may split the K range: what is received must fit behind the CTA's
  // own partial sums, both in the stages' place once all products are done
  static constexpr int SPLIT = BN <= 128 ? 8 : 3;
  static constexpr int PART = BN * SM_ROWS * 4;               // [token][128 rows]
  static constexpr int RECV = (BN <= 128 ? BN + SPLIT : 2 * ((BN + 2) / 3)) * SM_ROWS * 4;
  static constexpr int RING = OS * STAGE > PART + RECV ? OS * STAGE : PART + RECV;
  static constexpr size_t SMEM = 1024 + (size_t)RING + 8 * (2 * OS + 2) + 16;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  // CTAs of a cluster wait for one another, so none may wait for tensor memory
  // that another cluster's CTA holds: two CTAs of these kernels fit an SM only
  // where their columns do too.
  static_assert(SMEM > 76 * 1024 && (SMEM > 114 * 1024 || 2 * TMEM <= 512), "tensor memory of the CTAs an SM holds");
};

struct SmallParams {
  CUtensorMap w_map, x_map, sw_map, sx_map;
  void* y;
  bool y_bf16;
  int64_t T;
  int N, nkb, split;
  int* err;
};

// bulk copy of this CTA's shared memory into a peer's, counted on the peer's barrier (cluster addresses)
__device__ __forceinline__ void bulk_s2peer(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "r"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// The two halves of a cluster barrier.  The arrival is relaxed: what it tells is
// that this CTA's asynchronous reads and writes of its shared memory are done,
// each of them seen complete on an mbarrier; no ordinary store goes with it (a
// release would wait for those, some 1200 cycles).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

template <bool F4, int BN>
__global__ void __launch_bounds__(NTHREADS, BN <= 64 ? 2 : 1) mx_small_kernel(const __grid_constant__ SmallParams p) {
  using C = Cfg<F4, BN>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t* op_full = reinterpret_cast<uint64_t*>(smem + C::RING);
  uint64_t* op_empty = op_full + C::OS;
  uint64_t* acc_full = op_empty + C::OS;
  uint64_t* received = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(received + 1);
  float* partial = reinterpret_cast<float*>(smem);   // [token][128 rows], then the peers' [source][owned token][128 rows]

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int split = p.split;
  const int rank = split > 1 ? (int)cluster_ctarank() : 0;
  const int n0 = (int)(blockIdx.x / split) * SM_ROWS;
  const int64_t t0 = (int64_t)blockIdx.y * BN;
  // this CTA's share of the stages
  const int kb0 = (int)((int64_t)p.nkb * rank / split), kb1 = (int)((int64_t)p.nkb * (rank + 1) / split);
  const int count = kb1 - kb0;

  // stage i of this CTA's share
  auto fetch = [&](int i) {
    const int s = i % C::OS, kb = kb0 + i;
    mbar_arrive_expect_tx(&op_full[s], C::TX);
    unsigned char* st = smem + s * C::STAGE;
    unsigned char* sw = st + C::STAGE - 1024 - C::SX;
    tma_load_2d(st, &p.w_map, kb * 128, n0, &op_full[s]);
    tma_load_2d(st + W_TILE, &p.x_map, kb * 128, (int32_t)t0, &op_full[s]);
    tma_load_3d(sw, &p.sw_map, 0, kb * C::CT, n0 / MX_ROWS, &op_full[s]);
    tma_load_3d(sw + 1024, &p.sx_map, 0, kb * C::CT, (int32_t)(t0 / MX_ROWS), &op_full[s]);
  };
  // the first two stages' loads leave before tensor memory is there
  if (warp == TMA_WARP && lane == 0) {
    for (int s = 0; s < C::OS; ++s) {
      mbar_init(&op_full[s], 1);
      mbar_init(&op_empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(received, 1);
    fence_mbar_init();
    dependency_wait();
    for (int i = 0; i < count && i < 2; ++i) fetch(i);
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_slot, C::TMEM);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  dependency_wait();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  const uint32_t smem_base = smem_u32(smem);

  if (warp == TMA_WARP) {
    if (lane == 0) {
      int issued = count < 2 ? count : 2;
      for (; issued < count; ++issued) {
        if (issued >= C::OS && !mbar_wait(&op_empty[issued % C::OS], (uint32_t)(issued / C::OS - 1) & 1u, p.err)) break;
        fetch(issued);
      }
      // no copy may be in flight when the stages are reused or the CTA leaves
      for (int g = issued > C::OS ? issued - C::OS : 0; g < issued; ++g)
        mbar_wait(&op_full[g % C::OS], (uint32_t)(g / C::OS) & 1u, p.err);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // The whole warp runs the loop, one elected lane issues: uniform values
    // keep the descriptors in uniform registers (see oq_mx_gemm.cu).
    constexpr uint32_t idesc = F4 ? idesc_mx(SM_ROWS, BN, 1, 1) : idesc_mx(SM_ROWS, BN, 5, 0);
    const uint32_t lead = elect_one();
    const uint64_t desc0 = smem_desc_sw128(smem_base);
    const uint64_t sdesc0 = smem_desc_scales(smem_base + C::STAGE - 1024 - C::SX);
    int s = 0, ahead = 0;
    uint32_t parity = 0, acc = 0, set = 0;
    bool ok = true;
    for (int i = 0; i < count; ++i) {
      if (ahead == 0) {   // this stage and the next two, in one check
        const int s1 = s + 1 == C::OS ? 0 : s + 1, s2 = s1 + 1 == C::OS ? 0 : s1 + 1;
        const uint32_t f = smem_u32(op_full), left = (uint32_t)(count - i);
        const uint32_t flip = (s1 == 0 ? 6u : 0u) | (s2 == 0 ? 4u : 0u);
        const uint32_t full = mbar_test3(f + 8u * s, f + 8u * s1, f + 8u * s2, (parity ? 7u : 0u) ^ flip,
                                         left > 2 ? 7u : left > 1 ? 3u : 1u);
        ahead = !__all_sync(0xFFFFFFFFu, full & 1u)   ? 0
                : !__all_sync(0xFFFFFFFFu, full & 2u) ? 1
                : !__all_sync(0xFFFFFFFFu, full & 4u) ? 2
                                                      : 3;
        if (ahead == 0) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&op_full[s], parity, p.err))) {
            ok = false;
            break;
          }
          ahead = 1;
        }
        tc_fence_after();
      }
      --ahead;
      const uint32_t off = (uint32_t)s * (uint32_t)(C::STAGE >> 4);
      const uint64_t wd = desc0 + off, xd = wd + (W_TILE >> 4), sd = sdesc0 + off;
      const uint32_t sfw = tmem + BN + set * C::SF_SET, sfx = sfw + 4 * C::CT;
      set = (set + 1) % C::SF_SETS;
      if (lead) {
#pragma unroll
        for (int c = 0; c < C::CT; ++c) {
          tc_copy_scales<1>(sfw + 4 * c, sd + (c * MX_TILE_BYTES >> 4));
#pragma unroll
          for (int r = 0; r < C::RT; ++r)
            tc_copy_scales<1>(sfx + 4 * (c * C::RT + r), sd + ((1024 + (r * C::CT + c) * MX_TILE_BYTES) >> 4));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = F4 ? k / 2 : 0;
          tc_mma_mx<F4>(tmem, wd + 2 * k, xd + 2 * k, idesc | idesc_mx_sf(F4 ? 2u * (k & 1) : (uint32_t)k), sfw + 4 * c,
                           sfx + 4 * c * C::RT, k > 0 ? 1u : acc);
        }
        tc_commit(&op_empty[s]);
      }
      __syncwarp();
      acc = 1u;
      if (++s == C::OS) {
        s = 0;
        parity ^= 1u;
      }
    }
    if (ok && lead) tc_commit(acc_full);
    __syncwarp();
  }
  const bool ok = mbar_wait(acc_full, 0u, p.err);
  tc_fence_after();
  __syncthreads();   // the producer's copies have landed too: the stages are free
  const int tokens = (int)(p.T - t0 < BN ? p.T - t0 : BN);
  const int c0 = tokens * rank / split, owned = tokens * (rank + 1) / split - c0;
  if (split > 1) {
    if (threadIdx.x == 0) mbar_arrive_expect_tx(received, (uint32_t)((split - 1) * owned * SM_ROWS * 4));
    cluster_arrive();
  }
  // the partial tile: a lane holds one weight row, neighbouring lanes write neighbouring words
  if (warp < 4) {
    if constexpr (BN >= 32) {
#pragma unroll 1
      for (int cc = 0; cc * 32 < tokens; ++cc) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(warp * 32) << 16) + (uint32_t)(cc * 32), v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; ++j)
          partial[(cc * 32 + j) * SM_ROWS + warp * 32 + lane] = ok ? __uint_as_float(v[j]) : 0.f;
      }
    } else {
      // 16 tokens; the 16 columns behind them are scales and not used
      uint32_t v[32];
      tmem_ld_32x32b_x32(tmem + ((uint32_t)(warp * 32) << 16), v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < BN; ++j) partial[j * SM_ROWS + warp * 32 + lane] = ok ? __uint_as_float(v[j]) : 0.f;
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM);
  }
  if (split > 1) {
    cluster_wait();   // every CTA's stages are free and its barrier armed
    const int r = (int)threadIdx.x;
    if (r < split && r != rank) {
      const int first = tokens * r / split, theirs = tokens * (r + 1) / split - first;
      // in the peer: the sources before and after it, without a place of its own
      const int slot = rank < r ? rank : rank - 1;
      if (theirs > 0)
        bulk_s2peer(mapa_shared(smem_base + (uint32_t)((BN + slot * theirs) * SM_ROWS * 4), (uint32_t)r),
                    smem_base + (uint32_t)(first * SM_ROWS * 4), (uint32_t)(theirs * SM_ROWS * 4),
                    mapa_shared(smem_u32(received), (uint32_t)r));
    }
    __syncwarp();
    mbar_wait(received, 0u, p.err);
    cluster_arrive();   // what was sent here has arrived
  }

  // The owned tokens, four outputs a thread: sums in rank order.  The sources
  // are loaded before the first is used.
  const int quad = threadIdx.x & 31, o = n0 + 4 * quad;
  if (o < p.N) {
    constexpr int QUADS = SM_ROWS / 4;
    const float4* mine = reinterpret_cast<const float4*>(partial + c0 * SM_ROWS) + quad;
    const float4* recv = reinterpret_cast<const float4*>(partial + BN * SM_ROWS) + quad;
#pragma unroll 2
    for (int c = threadIdx.x >> 5; c < owned; c += NTHREADS / 32) {
      float4 v[C::SPLIT];
#pragma unroll
      for (int r = 0; r < C::SPLIT; ++r)
        if (r < split) v[r] = r == rank ? mine[c * QUADS] : recv[((r < rank ? r : r - 1) * owned + c) * QUADS];
      float4 sum = v[0];
#pragma unroll
      for (int r = 1; r < C::SPLIT; ++r) {
        if (r < split) {
          sum.x += v[r].x;
          sum.y += v[r].y;
          sum.z += v[r].z;
          sum.w += v[r].w;
        }
      }
      const int64_t at = (t0 + c0 + c) * p.N + o;
      if (p.y_bf16)
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.y) + at) =
            make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(p.y) + at) = sum;
    }
  }
  if (split > 1) cluster_wait();   // no CTA leaves before its sums have been copied out
}

// CTAs that split a weight tile's K range: as many as the SMs' slots hold, each
// with at least two stages.  (Slots are counted, not clusters: whether all
// clusters are resident at once also depends on how their CTAs fit the GPCs.
// They need not be; clusters do not wait for one another.)
int choose_split(int m_tiles, int64_t t_tiles, int nkb, int slots, int most) {
  int best = 1;
  for (int s = 2; s <= most; ++s)
    if ((int64_t)m_tiles * t_tiles * s <= slots && nkb >= 2 * s) best = s;
  return best;
}

template <bool F4, int BN>
oq_status launch(const MxGemmArgs& g, cudaStream_t stream) {
  using C = Cfg<F4, BN>;
  SmallParams kp;
  std::memset(&kp, 0, sizeof(kp));
  oq_status st = mx_encode_codes(&kp.w_map, g.w_codes, g.N, g.K, 4, !F4, SM_ROWS, "the weight codes");
  if (st == OQ_OK) st = mx_encode_codes(&kp.x_map, g.a_codes, g.T, g.K, g.a_bits, false, BN, "the activation codes");
  if (st == OQ_OK) st = mx_encode_scales(&kp.sw_map, g.w_scales, g.N, g.K, 1, C::CT, "the weight scales");
  if (st == OQ_OK) st = mx_encode_scales(&kp.sx_map, g.a_scales, g.T, g.K, C::RT, C::CT, "the activation scales");
  if (st != OQ_OK) return st;
  kp.y = g.y;
  kp.y_bf16 = g.y_bf16;
  kp.T = g.T;
  kp.N = g.N;
  kp.nkb = (mx_col_tiles(g.K) + C::CT - 1) / C::CT;
  kp.err = g.err;
  const int m_tiles = (g.N + SM_ROWS - 1) / SM_ROWS;
  const int64_t t_tiles = (g.T + BN - 1) / BN;
  int device = 0;
  const int sms = mx_sm_count(&device);
  kp.split = choose_split(m_tiles, t_tiles, kp.nkb, sms * (BN <= 64 ? 2 : 1), C::SPLIT);

  static std::atomic<uint64_t> smem_set{0};
  if ((st = mx_allow_smem(reinterpret_cast<const void*>(mx_small_kernel<F4, BN>), C::SMEM, device, &smem_set)) != OQ_OK)
    return st;
  const cudaError_t e = mx_launch(mx_small_kernel<F4, BN>, dim3((unsigned)(m_tiles * kp.split), (unsigned)t_tiles), NTHREADS,
                                  C::SMEM, kp.split, stream, kp);
  if (e != cudaSuccess) {
    set_error(std::string("microscaled small-batch product launch: ") + cudaGetErrorString(e));
    return OQ_ERR_CUDA;
  }
  return OQ_OK;
}

template <bool F4>
oq_status launch_bn(const MxGemmArgs& g, cudaStream_t st) {
  if (g.T <= 16) return launch<F4, 16>(g, st);
  if (g.T <= 32) return launch<F4, 32>(g, st);
  if (g.T <= 64) return launch<F4, 64>(g, st);
  if (g.T <= 128) return launch<F4, 128>(g, st);
  return launch<F4, 256>(g, st);
}

}  // namespace

oq_status mx_small_launch(const MxGemmArgs& g, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return g.a_bits == 4 ? launch_bn<true>(g, st) : launch_bn<false>(g, st);
}

}  // namespace oq
