// Product of microscaled operands for large batches, on CTA pairs:
//   y[t, o] = sum_k a[t, k] w[o, k],  a in e2m1 or e4m3, w in e2m1, one E8M0
//   scale per 32 elements of a row, fp32 sums in tensor memory.
// The tensor cores apply the scales (tcgen05.mma block_scale), so codes and
// scales go from HBM to the MMA as they are stored: 4-bit activations use
// kind::mxf4 (K 64 an MMA), 8-bit activations kind::mxf8f6f4 (K 32), for which
// TMA spreads the weights' 4-bit codes to 8-bit containers on the way.
//
// Tiles: 256 tokens x 192 outputs a pair (each CTA 128 tokens, and half of the
// weight rows in shared memory).  192 columns and not 256, because two
// accumulators of 256 would fill tensor memory and leave no columns for the
// scales; with two of 192 the epilogue of a tile overlaps the next tile's
// products.  A stage is 128 bytes of every row: 256 elements of 4 bits or 128
// of 8.  Scales of the pair's weight rows start at a multiple of 64 rows, so
// the MMA's scale address may begin two columns into a tile's four.
//
// Warps: 0-3 epilogue, 4 TMA producer, 5 tensor memory and (even CTA) MMAs.
#include <algorithm>
#include <cstring>

#include "oq_epilogue.cuh"
#include "oq_mx_ptx.cuh"

namespace oq {
namespace {

constexpr int RM = 128, PN = 192, RN = PN / 2;
constexpr int A_TILE = RM * 128, B_TILE = RN * 128;
constexpr int OS = 6;
constexpr int TMA_WARP = 4, MMA_WARP = 5, NTHREADS = 6 * 32;
constexpr uint32_t TMEM_COLS = 512, SF_COL = 2 * PN;
constexpr uint32_t ACC_EMPTY_COUNT = 2 * 4;
constexpr int EPI_BYTES = 4 * 2 * 32 * 32 * 4;

// column tiles of scales a stage covers (128 elements each)
__host__ __device__ constexpr int stage_ct(bool f4) { return f4 ? 2 : 1; }
__host__ __device__ constexpr int stage_bytes(bool f4) { return A_TILE + B_TILE + 1024 + 1024 * stage_ct(f4); }
// a load that spreads 4-bit codes counts the packed bytes, half of what it writes
__host__ __device__ constexpr uint32_t stage_tx(bool f4) {
  return A_TILE + (f4 ? B_TILE : B_TILE / 2) + 3 * MX_TILE_BYTES * stage_ct(f4);
}

struct MxParams {
  CUtensorMap a_map, w_map, sa_map, sw_map, y_map;
  bool y_bf16;
  int N, n_tiles, nkb;
  int64_t tiles;
  int* err;
};

// one 32 x 32 chunk of the accumulator (this lane's row in v) staged for a TMA
// store box: fp32 rows in the 128-byte swizzle, bf16 rows in the 64-byte one
__device__ __forceinline__ void stage_chunk(const uint32_t (&v)[32], uint32_t buf, int lane, bool bf16) {
  if (!bf16) {
    const uint32_t rb = buf + (uint32_t)lane * 128u;
#pragma unroll
    for (int k = 0; k < 8; ++k)
      st_shared_v4(rb + ((uint32_t)(k ^ (lane & 7)) << 4), make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
  } else {
    const uint32_t rb = buf + (uint32_t)lane * 64u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack_bf16x2(__uint_as_float(v[8 * k + 2 * j]), __uint_as_float(v[8 * k + 2 * j + 1]));
      st_shared_v4(rb + ((uint32_t)(k ^ ((lane >> 1) & 3)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
}

template <bool F4>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    mx_gemm_kernel(const __grid_constant__ MxParams p) {
  constexpr int CT = stage_ct(F4), STAGE = stage_bytes(F4);
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* epi = smem + OS * STAGE;
  uint64_t* op_full = reinterpret_cast<uint64_t*>(epi + EPI_BYTES);
  uint64_t* op_empty = op_full + OS;
  uint64_t* acc_full = op_empty + OS;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int nkb = p.nkb;
  const int my_tiles = (p.tiles > pair) ? (int)((p.tiles - 1 - pair) / npairs + 1) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < OS; ++s) {
      mbar_init(&op_full[s], 1);    // the even CTA's producer: arrive + expect both CTAs' bytes
      mbar_init(&op_empty[s], 1);   // the MMA commit
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&acc_full[a], 1);
      mbar_init(&acc_empty[a], ACC_EMPTY_COUNT);
    }
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();   // barriers of both CTAs initialised before any remote arrival or load
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t smem_base = smem_u32(smem);
  const int total = my_tiles * nkb;

  if (warp == TMA_WARP) {
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(&op_full[0]), 0);
      int s = 0, kb = 0, tile = 0, issued = 0;
      uint32_t n = 0;
      int32_t m0 = 0, n0 = 0;
      auto origin = [&](int tile_i) {
        const int64_t tt = pair + (int64_t)tile_i * npairs;
        m0 = (int32_t)((tt / p.n_tiles) * (2 * RM) + rank * RM);
        n0 = (int32_t)((tt % p.n_tiles) * PN);
      };
      origin(0);
      for (int g = 0; g < total; ++g) {
        if (n > 0 && !mbar_wait(&op_empty[s], (n - 1) & 1u, p.err)) break;
        if (rank == 0) mbar_arrive_expect_tx(&op_full[s], 2 * stage_tx(F4));
        unsigned char* st = smem + s * STAGE;
        const uint32_t bar = full0 + 8u * (uint32_t)s;
        tma_load_2d_pair(st, &p.a_map, kb * 128, m0, bar);
        tma_load_2d_pair(st + A_TILE, &p.w_map, kb * 128, n0 + (int32_t)rank * RN, bar);
        tma_load_3d_pair(st + A_TILE + B_TILE, &p.sa_map, 0, kb * CT, m0 / MX_ROWS, bar);
        tma_load_3d_pair(st + A_TILE + B_TILE + 1024, &p.sw_map, 0, kb * CT, n0 / MX_ROWS, bar);
        ++issued;
        if (++s == OS) {
          s = 0;
          ++n;
        }
        if (++kb == nkb) {
          kb = 0;
          origin(++tile);
        }
      }
      // no copy of either CTA may be in flight when the pair leaves (they all
      // count on the even CTA's barriers; bounded as every wait)
      if (rank == 0)
        for (int g = issued > OS ? issued - OS : 0; g < issued; ++g) mbar_wait(&op_full[g % OS], (uint32_t)(g / OS) & 1u, p.err);
    }
    __syncwarp();
  } else if (warp < 4) {
    const int q = warp;
    unsigned char* ebuf = epi + q * (2 * 32 * 32 * 4);
    for (int64_t i = 0; i < my_tiles; ++i) {
      const int a = (int)(i & 1);
      if (!mbar_wait(&acc_full[a], (uint32_t)(i >> 1) & 1u, p.err)) break;
      tc_fence_after();
      const int64_t tt = pair + i * npairs;
      const int64_t row0 = (tt / p.n_tiles) * (2 * RM) + rank * RM + q * 32;
      const int n0 = (int)(tt % p.n_tiles) * PN;
#pragma unroll 1
      for (int cc = 0; cc < PN / 32; ++cc) {
        const int nb = n0 + cc * 32;
        if (nb >= p.N) break;
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(a * PN + cc * 32), v);
        tmem_wait_ld();
        unsigned char* buf = ebuf + (cc & 1) * (32 * 32 * 4);
        if (lane == 0) bulk_wait_read<1>();   // the store that last read this buffer
        __syncwarp();
        stage_chunk(v, smem_u32(buf), lane, p.y_bf16);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&p.y_map, nb, (int32_t)row0, buf);
          bulk_commit();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[a]), 0));
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  } else if (warp == MMA_WARP && rank == 0) {
    if (lane == 0) {
      constexpr uint32_t idesc = F4 ? idesc_mx(2 * RM, PN, 1, 1) : idesc_mx(2 * RM, PN, 0, 5);
      int s = 0;
      uint32_t n = 0, slot = 0;
      bool ok = true;
      for (int64_t i = 0; i < my_tiles && ok; ++i) {
        const int a = (int)(i & 1);
        const uint32_t u = (uint32_t)(i >> 1);
        if (u > 0 && !mbar_wait_cluster(&acc_empty[a], (u - 1) & 1u, p.err)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + (uint32_t)(a * PN);
        const uint32_t sf_shift = (uint32_t)(((pair + i * npairs) % p.n_tiles) * PN % MX_ROWS) / 32;   // 0 or 2
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait_cluster(&op_full[s], n & 1u, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_base + (uint32_t)s * STAGE;
          // scale columns, two sets in turn: [4 CT of A][8 CT of W]
          const uint32_t sfa = tmem + SF_COL + slot * (12 * CT), sfw = sfa + 4 * CT;
          slot ^= 1u;
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            tc_copy_scales<2>(sfa + 4 * c, smem_desc_scales(st + A_TILE + B_TILE + c * MX_TILE_BYTES));
#pragma unroll
            for (int r = 0; r < 2; ++r)
              tc_copy_scales<2>(sfw + 8 * c + 4 * r,
                                smem_desc_scales(st + A_TILE + B_TILE + 1024 + (r * CT + c) * MX_TILE_BYTES));
          }
          const uint64_t ad = smem_desc_sw128(st), bd = smem_desc_sw128(st + A_TILE);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int c = F4 ? k / 2 : 0;
            const uint32_t id = idesc | idesc_mx_sf(F4 ? 2u * (k & 1) : (uint32_t)k);
            tc_mma_mx<2, F4>(d_tmem, ad + 2 * k, bd + 2 * k, id, sfa + 4 * c, sfw + 8 * c + sf_shift,
                             kb > 0 || k > 0 ? 1u : 0u);
          }
          tc_commit_pair_mc(&op_empty[s], (uint16_t)0x3);
          if (++s == OS) {
            s = 0;
            ++n;
          }
        }
        if (ok) tc_commit_pair_mc(&acc_full[a], (uint16_t)0x3);
      }
    }
    __syncwarp();
  }

  // neither CTA may leave while its peer can still read its tiles or arrive on its barriers
  tc_fence_before();
  cluster_sync_all();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

template <bool F4>
oq_status launch(MxParams& kp, const MxGemmArgs& g, cudaStream_t stream) {
  constexpr int CT = stage_ct(F4);
  oq_status st = mx_encode_codes(&kp.a_map, g.a_codes, g.T, g.K, g.a_bits, false, RM, "the activation codes");
  if (st == OQ_OK) st = mx_encode_codes(&kp.w_map, g.w_codes, g.N, g.K, 4, !F4, RN, "the weight codes");
  if (st == OQ_OK) st = mx_encode_scales(&kp.sa_map, g.a_scales, g.T, g.K, 1, CT, "the activation scales");
  if (st == OQ_OK) st = mx_encode_scales(&kp.sw_map, g.w_scales, g.N, g.K, 2, CT, "the weight scales");
  if (st == OQ_OK) st = encode_y_map(&kp.y_map, g.y, g.T, g.N, g.y_bf16);
  if (st != OQ_OK) return st;
  kp.nkb = (mx_col_tiles(g.K) + CT - 1) / CT;

  const size_t smem = 1024 + (size_t)OS * stage_bytes(F4) + EPI_BYTES + 8 * (2 * OS + 4) + 16;
  cudaError_t e = cudaFuncSetAttribute(mx_gemm_kernel<F4>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) {
    set_error(std::string("cudaFuncSetAttribute(microscaled product): ") + cudaGetErrorString(e));
    return OQ_ERR_CUDA;
  }
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t grid = std::min<int64_t>(2 * kp.tiles, (int64_t)(sms & ~1));
  // stage counters are 32-bit
  if (((kp.tiles + grid / 2 - 1) / (grid / 2)) * (int64_t)kp.nkb >= (int64_t)1 << 31) return OQ_ERR_UNSUPPORTED;
  mx_gemm_kernel<F4><<<(unsigned)grid, NTHREADS, smem, stream>>>(kp);
  e = cudaGetLastError();
  if (e != cudaSuccess) {
    set_error(std::string("microscaled product launch: ") + cudaGetErrorString(e));
    return OQ_ERR_CUDA;
  }
  return OQ_OK;
}

}  // namespace

oq_status mx_gemm_launch(const MxGemmArgs& g, void* stream) {
  MxParams kp;
  std::memset(&kp, 0, sizeof(kp));
  kp.y_bf16 = g.y_bf16;
  kp.N = g.N;
  kp.err = g.err;
  kp.n_tiles = (g.N + PN - 1) / PN;
  kp.tiles = ((g.T + 2 * RM - 1) / (2 * RM)) * (int64_t)kp.n_tiles;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return g.a_bits == 4 ? launch<true>(kp, g, st) : launch<false>(kp, g, st);
}

}  // namespace oq
