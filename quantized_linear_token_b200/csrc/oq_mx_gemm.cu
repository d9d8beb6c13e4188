// Product of microscaled operands for large batches, on CTA pairs:
//   y[t, o] = sum_k a[t, k] w[o, k],  a in e2m1 or e4m3, w in e2m1, one E8M0
//   scale per 32 elements of a row, fp32 sums in tensor memory.
// The tensor cores apply the scales (tcgen05.mma block_scale), so codes and
// scales go from HBM to the MMA as they are stored: 4-bit activations use
// kind::mxf4 (K 64 an MMA), 8-bit activations kind::mxf8f6f4 (K 32), for which
// TMA spreads the weights' 4-bit codes to 8-bit containers on the way.
//
// A pair's tile is 256 tokens (128 a CTA) by PN outputs, in one part of up to
// 256 columns or two, and a stage is 128 bytes of every row: 256 elements of 4
// bits or 128 of 8.  What bounds a narrow tile is the feed: from L2 an SM takes
// about 99 bytes a nanosecond (measured, copies alone), while a stage of 256 x
// 192 wants 31 KB per 384 cycles of MMAs (145 bytes a nanosecond).  Wider tiles
// reuse the activations' bytes: 256 x 448 wants 49 KB per 896 cycles, as much as
// the feed gives.  448 columns and the scales' 64 fill tensor memory, so there is
// one accumulator; it is drained to registers and handed back to the MMAs before
// the first store.  Narrower tiles are for batches that would leave pairs idle.
//
// The other bound is the thread that issues: per stage and 10 scale copies it
// has 896 cycles.  So the loop runs warp-uniform (1555 cycles a stage otherwise),
// scale copies stand between MMAs that do not need them, and barriers are asked
// for three stages at a time (about 230 cycles a check).  Measured: 881 cycles a
// stage, and 2100 from one tile's last MMA issued to the next one's first.
//
// 32760 x 5120 -> 5120 with 4-bit activations: 291 us alone (5.9 PFLOP/s), 339 us
// in a stream of such calls, where the 1000 W limit holds the clock at 1.46 GHz;
// 4096 x 13824 -> 5120 with 8-bit activations: 210 us with cold caches and 228 in
// a stream (2.8, 2.5).  K is not split: between 257 and some 2000 tokens one tile
// a pair leaves fill, mainloop and drain in series and pairs idle (512 x 5120 ->
// 5120: 11.2 us at 4 bits, 17.4 at 8, on 54 of 74 pairs).
//
// Scales: a 512-byte tile (128 rows x 4 blocks) is one tcgen05.cp into four
// tensor-memory columns.  The pair's weight rows start at a multiple of 64, so
// an MMA's scale address may begin two columns into a tile's four.
//
// Warps: 0-7 epilogue (two per lane quarter), 8 TMA producer, 9 tensor memory
// and (even CTA) MMAs.
#include <algorithm>
#include <cstring>

#include "oq_epilogue.cuh"
#include "oq_mx_ptx.cuh"

namespace oq {
namespace {

constexpr int RM = 128;
constexpr int EPI_WARPS = 8, TMA_WARP = 8, MMA_WARP = 9, NTHREADS = 10 * 32;
constexpr uint32_t TMEM_COLS = 512, SF_COL = 448;
constexpr uint32_t ACC_EMPTY_COUNT = 2 * EPI_WARPS;
constexpr int EPI_BOX = 2048;             // a staging box: 32 rows of 64 bytes
constexpr int SMEM_LIMIT = 227 * 1024;

template <bool F4, int N0, int N1>
struct Cfg {
  static constexpr int PN = N0 + N1;
  static constexpr int CT = F4 ? 2 : 1;                           // column tiles of scales a stage covers
  static constexpr int RT = (PN + (PN % MX_ROWS)) / MX_ROWS;      // row tiles the weight rows can touch
  static constexpr int A_TILE = RM * 128, B0_TILE = N0 / 2 * 128, B1_TILE = N1 / 2 * 128;
  static constexpr int SW = (RT * CT * MX_TILE_BYTES + 1023) / 1024 * 1024;
  static constexpr int B0 = A_TILE, B1 = B0 + B0_TILE, SA_OFF = B1 + B1_TILE, SW_OFF = SA_OFF + 1024;
  static constexpr int STAGE = SW_OFF + SW;
  // a load that spreads 4-bit codes counts the packed bytes, half of what it writes
  static constexpr uint32_t TX = A_TILE + (B0_TILE + B1_TILE) / (F4 ? 1 : 2) + (1 + RT) * CT * MX_TILE_BYTES;
  static constexpr int FIXED = 1024 + EPI_WARPS * EPI_BOX + 256;
  static constexpr int OS = (SMEM_LIMIT - FIXED) / STAGE < 8 ? (SMEM_LIMIT - FIXED) / STAGE : 8;
  static constexpr size_t SMEM = FIXED + (size_t)OS * STAGE;
  static constexpr int SF_SET = 4 + 4 * RT;                       // scale columns of one column tile
  static constexpr int SF_SETS = 64 / SF_SET < 4 ? 64 / SF_SET : 4;   // sets used in turn
  static_assert(OS >= 4, "the checks look three stages ahead");
  static_assert(N0 % 64 == 0 && N1 % 64 == 0 && N0 <= 256 && N1 <= N0 && PN <= (int)SF_COL && SF_SETS >= 3, "tile");
};

struct MxParams {
  CUtensorMap a_map, w0_map, w1_map, sa_map, sw_map, y_map;
  bool y_bf16;
  int N, n_tiles, nkb;
  int64_t tiles;
  int* err;
};

// One 32 x 64-byte box of y through shared memory (64-byte swizzle): this
// lane's row in w.
__device__ __forceinline__ void store_box(const MxParams& p, const uint32_t* w, int lane, int col, int32_t row0,
                                          unsigned char* box) {
  if (lane == 0) bulk_wait_read<0>();   // the store that last read the box
  __syncwarp();
  const uint32_t rb = smem_u32(box) + (uint32_t)lane * 64u, sw = (uint32_t)(lane >> 1) & 3u;
#pragma unroll
  for (int k = 0; k < 4; ++k) st_shared_v4(rb + (((uint32_t)k ^ sw) << 4), make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(&p.y_map, col, row0, box);
    bulk_commit();
  }
}

// The accumulator's columns that this warp drains: chunks of 32, alternating
// between the two warps of a lane quarter.  bf16 y: all of them go to
// registers, packed, and the accumulator is handed back to the MMAs before the
// first store.  fp32 y has no room for that and goes in steps.
template <int PN>
__device__ __forceinline__ void drain_bf16(const MxParams& p, uint32_t tmem_q, int e, int lane, int n0, int32_t row0,
                                           unsigned char* box, uint32_t empty_bar) {
  constexpr int NC = PN / 64;
  uint32_t v[NC][16];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    uint32_t w[32];
    tmem_ld_32x32b_x32(tmem_q + (uint32_t)((2 * c + e) * 32), w);
    tmem_wait_ld();
#pragma unroll
    for (int j = 0; j < 16; ++j) v[c][j] = pack_bf16x2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive_tmem(empty_bar);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int col = n0 + (2 * c + e) * 32;
    if (col < p.N) store_box(p, v[c], lane, col, row0, box);
  }
}

template <int PN>
__device__ __forceinline__ void drain_f32(const MxParams& p, uint32_t tmem_q, int e, int lane, int n0, int32_t row0,
                                          unsigned char* box, uint32_t empty_bar) {
  constexpr int NC = PN / 64, STEP = 3;
#pragma unroll
  for (int c0 = 0; c0 < NC; c0 += STEP) {
    uint32_t v[STEP][32];
#pragma unroll
    for (int c = 0; c < STEP && c0 + c < NC; ++c) tmem_ld_32x32b_x32(tmem_q + (uint32_t)((2 * (c0 + c) + e) * 32), v[c]);
    tmem_wait_ld();
    if (c0 + STEP >= NC) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_tmem(empty_bar);
    }
#pragma unroll
    for (int c = 0; c < STEP && c0 + c < NC; ++c) {
      const int col = n0 + (2 * (c0 + c) + e) * 32;
      if (col < p.N) store_box(p, v[c], lane, col, row0, box);
      if (col + 16 < p.N) store_box(p, v[c] + 16, lane, col + 16, row0, box);
    }
  }
}

template <bool F4, int N0, int N1>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NTHREADS, 1)
    mx_gemm_kernel(const __grid_constant__ MxParams p) {
  using C = Cfg<F4, N0, N1>;
  constexpr int OS = C::OS, CT = C::CT;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  unsigned char* epi = smem + OS * C::STAGE;
  uint64_t* op_full = reinterpret_cast<uint64_t*>(epi + EPI_WARPS * EPI_BOX);
  uint64_t* op_empty = op_full + OS;
  uint64_t* acc_full = op_empty + OS;
  uint64_t* acc_empty = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 1);

  const int warp = __shfl_sync(0xFFFFFFFFu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int64_t pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int nkb = p.nkb;
  const int my_tiles = (p.tiles > pair) ? (int)((p.tiles - 1 - pair) / npairs + 1) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < OS; ++s) {
      mbar_init(&op_full[s], 1);    // the even CTA's producer: arrive + expect both CTAs' bytes
      mbar_init(&op_empty[s], 1);   // the MMA commit
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, ACC_EMPTY_COUNT);
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc_pair(tmem_slot, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();   // barriers of both CTAs initialised before any remote arrival or load
  tc_fence_after();
  dependency_wait();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
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
        n0 = (int32_t)((tt % p.n_tiles) * C::PN);
      };
      origin(0);
      for (int g = 0; g < total; ++g) {
        if (n > 0 && !mbar_wait(&op_empty[s], (n - 1) & 1u, p.err)) break;
        if (rank == 0) mbar_arrive_expect_tx(&op_full[s], 2 * C::TX);
        unsigned char* st = smem + s * C::STAGE;
        const uint32_t bar = full0 + 8u * (uint32_t)s;
        tma_load_2d_pair(st, &p.a_map, kb * 128, m0, bar);
        tma_load_2d_pair(st + C::B0, &p.w0_map, kb * 128, n0 + (int32_t)rank * (N0 / 2), bar);
        if constexpr (N1 > 0) tma_load_2d_pair(st + C::B1, &p.w1_map, kb * 128, n0 + N0 + (int32_t)rank * (N1 / 2), bar);
        tma_load_3d_pair(st + C::SA_OFF, &p.sa_map, 0, kb * CT, m0 / MX_ROWS, bar);
        tma_load_3d_pair(st + C::SW_OFF, &p.sw_map, 0, kb * CT, n0 / MX_ROWS, bar);
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
        for (int g = issued > OS ? issued - OS : 0; g < issued; ++g)
          mbar_wait(&op_full[g % OS], (uint32_t)(g / OS) & 1u, p.err);
    }
    __syncwarp();
  } else if (warp < EPI_WARPS) {
    const int q = warp & 3, e = warp >> 2;
    unsigned char* box = epi + warp * EPI_BOX;
    const uint32_t empty0 = mapa_shared(smem_u32(acc_empty), 0);
    for (int64_t i = 0; i < my_tiles; ++i) {
      if (!mbar_wait(acc_full, (uint32_t)i & 1u, p.err)) break;
      tc_fence_after();
      const int64_t tt = pair + i * npairs;
      const int32_t row0 = (int32_t)((tt / p.n_tiles) * (2 * RM) + rank * RM + q * 32);
      const int n0 = (int)(tt % p.n_tiles) * C::PN;
      const uint32_t tmem_q = tmem + ((uint32_t)(q * 32) << 16);
      if (p.y_bf16) drain_bf16<C::PN>(p, tmem_q, e, lane, n0, row0, box, empty0);
      else drain_f32<C::PN>(p, tmem_q, e, lane, n0, row0, box, empty0);
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  } else if (warp == MMA_WARP && rank == 0) {
    // The whole warp runs this loop and one elected lane issues: with every
    // value uniform over the warp the descriptors stay in uniform registers,
    // where the tensor instructions take them (from one lane's own registers
    // each is moved there first).
    {
      constexpr uint32_t AF = F4 ? 1 : 0, BF = F4 ? 1 : 5;
      constexpr uint32_t id0 = idesc_mx(2 * RM, N0, AF, BF), id1 = idesc_mx(2 * RM, N1 ? N1 : N0, AF, BF);
      constexpr int STRIDE = CT * MX_TILE_BYTES >> 4;
      // the stages' descriptors share their high words
      const uint64_t desc0 = smem_desc_sw128(smem_base), sdesc0 = smem_desc_scales(smem_base + C::SA_OFF);
      const uint32_t d_lo = (uint32_t)desc0, s_lo = (uint32_t)sdesc0;
      constexpr uint32_t SW = (C::SW_OFF - C::SA_OFF) >> 4;
      uint32_t n = 0, set = 0;          // n: parity of the ring's current round
      int s = 0, ahead = 0, left = total;   // stages known to be full after this one; stages left with this one
      auto columns = [&](uint32_t st) { return tmem + SF_COL + st * C::SF_SET; };
      auto next_set = [&]() { return set + 1 == C::SF_SETS ? 0u : set + 1; };
      MxHalf h;
      h.lead = elect_one();
      h.d0 = tmem;
      h.d1 = tmem + N0;
      h.hi = (uint32_t)(desc0 >> 32);
      h.c_hi = (uint32_t)(sdesc0 >> 32);
      bool ok = total > 0 && __all_sync(0xFFFFFFFFu, mbar_wait(&op_full[0], 0u, p.err));
      tc_fence_after();
      if (ok && h.lead) {   // the first half's scales
        tc_copy_scales<2>(columns(0), sdesc0);
#pragma unroll
        for (int r = 0; r < C::RT; ++r) tc_copy_scales<2>(columns(0) + 4 + 4 * r, sdesc0 + SW + r * STRIDE);
      }
      __syncwarp();
      for (int64_t i = 0; i < my_tiles && ok; ++i) {
        const uint32_t free_parity = ((uint32_t)i - 1u) & 1u;
        if (i > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(acc_empty, free_parity, p.err))) break;
        tc_fence_after();
        const uint32_t shift = (uint32_t)(((pair + i * npairs) % p.n_tiles) * C::PN % MX_ROWS) / 32;   // 0 or 2
        for (int kb = 0; kb < nkb; ++kb) {
          // stage s is full and the scales of its first half are in (or on their way to) set `set`
          const int s1 = s + 1 == OS ? 0 : s + 1;
          const bool more = left > 1;
          const uint32_t off = (uint32_t)s * (uint32_t)(C::STAGE >> 4), off1 = (uint32_t)s1 * (uint32_t)(C::STAGE >> 4);
          h.a = d_lo + off;
          h.b0 = h.a + (C::B0 >> 4);
          h.b1 = h.a + (C::B1 >> 4);
          h.sf = columns(set);
          h.w0 = h.sf + 4 + shift;
          h.w1 = h.w0 + N0 / 32;
          h.i0a = id0;
          h.i1a = id1;
          h.i0b = id0 | idesc_mx_sf(F4 ? 2 : 1);
          h.i1b = id1 | idesc_mx_sf(F4 ? 2 : 1);
          h.accumulate = kb > 0 ? 1u : 0u;
          // 4 bits: the second column tile of this stage is copied meanwhile
          h.copy = F4 ? 1u : 0u;
          h.sf_next = columns(next_set());
          h.ca = s_lo + off + (MX_TILE_BYTES >> 4);
          h.cw = h.ca + SW;
          h.commit = 0u;
          h.commit_bar = &op_empty[s];
          tc_half_stage_pair<F4, (N1 > 0), C::RT, STRIDE>(h);
          // The next stage's operands.  A check costs this thread some 230
          // cycles (it queues behind the issued tensor work), and issuing a
          // stage takes about 45 a copy and 53 an MMA of the 896 that its MMAs
          // run, so the next three stages are asked for at once.
          if (more && ahead == 0) {
            const int s2 = s1 + 1 == OS ? 0 : s1 + 1, s3 = s2 + 1 == OS ? 0 : s2 + 1;
            const uint32_t f = smem_u32(op_full);
            const uint32_t flip = (s1 == 0 ? 7u : 0u) | (s2 == 0 ? 6u : 0u) | (s3 == 0 ? 4u : 0u);
            const uint32_t full = mbar_test3(f + 8u * s1, f + 8u * s2, f + 8u * s3, (n & 1u ? 7u : 0u) ^ flip,
                                                     left > 3 ? 7u : left > 2 ? 3u : 1u);
            ahead = !__all_sync(0xFFFFFFFFu, full & 1u)   ? 0
                    : !__all_sync(0xFFFFFFFFu, full & 2u) ? 1
                    : !__all_sync(0xFFFFFFFFu, full & 4u) ? 2
                                                          : 3;
            if (ahead == 0) {
              if (!__all_sync(0xFFFFFFFFu, mbar_wait(&op_full[s1], (n & 1u) ^ (s1 == 0 ? 1u : 0u), p.err))) {
                ok = false;
                break;
              }
              ahead = 1;
            }
            tc_fence_after();
          }
          --ahead;
          --left;
          h.a += 4;
          h.b0 += 4;
          h.b1 += 4;
          if constexpr (F4) {
            set = next_set();
            h.sf = columns(set);
            h.w0 = h.sf + 4 + shift;
            h.w1 = h.w0 + N0 / 32;
          } else {
            h.i0a = id0 | idesc_mx_sf(2);
            h.i1a = id1 | idesc_mx_sf(2);
            h.i0b = id0 | idesc_mx_sf(3);
            h.i1b = id1 | idesc_mx_sf(3);
          }
          h.accumulate = 1u;
          h.copy = more ? 1u : 0u;   // the next stage's first column tile
          set = next_set();
          h.sf_next = columns(set);
          h.ca = s_lo + off1;
          h.cw = h.ca + SW;
          h.commit = 1u;
          tc_half_stage_pair<F4, (N1 > 0), C::RT, STRIDE>(h);
          s = s1;
          if (s1 == 0) n ^= 1u;
        }
        if (ok && h.lead) tc_commit_pair_mc(acc_full, (uint16_t)0x3);
        __syncwarp();
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

// y [M, N] in boxes of 32 rows x 64 bytes, 64-byte swizzle; stores clip rows and columns past the end
oq_status encode_y(CUtensorMap* map, void* y, int64_t M, int N, bool bf16) {
  const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)M};
  const cuuint64_t strides[1] = {(cuuint64_t)N * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {bf16 ? 32u : 16u, 32};
  return mx_encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, y, dims, strides,
                   box, CU_TENSOR_MAP_SWIZZLE_64B, "y");
}

template <bool F4, int N0, int N1>
oq_status launch(const MxGemmArgs& g, int sms, int device, cudaStream_t stream) {
  using C = Cfg<F4, N0, N1>;
  MxParams kp;
  std::memset(&kp, 0, sizeof(kp));
  kp.y_bf16 = g.y_bf16;
  kp.N = g.N;
  kp.err = g.err;
  kp.n_tiles = (g.N + C::PN - 1) / C::PN;
  kp.tiles = ((g.T + 2 * RM - 1) / (2 * RM)) * (int64_t)kp.n_tiles;
  kp.nkb = (mx_col_tiles(g.K) + C::CT - 1) / C::CT;
  oq_status st = mx_encode_codes(&kp.a_map, g.a_codes, g.T, g.K, g.a_bits, false, RM, "the activation codes");
  if (st == OQ_OK) st = mx_encode_codes(&kp.w0_map, g.w_codes, g.N, g.K, 4, !F4, N0 / 2, "the weight codes");
  if (st == OQ_OK && N1 > 0) st = mx_encode_codes(&kp.w1_map, g.w_codes, g.N, g.K, 4, !F4, N1 / 2, "the weight codes");
  if (st == OQ_OK) st = mx_encode_scales(&kp.sa_map, g.a_scales, g.T, g.K, 1, C::CT, "the activation scales");
  if (st == OQ_OK) st = mx_encode_scales(&kp.sw_map, g.w_scales, g.N, g.K, C::RT, C::CT, "the weight scales");
  if (st == OQ_OK) st = encode_y(&kp.y_map, g.y, g.T, g.N, g.y_bf16);
  if (st != OQ_OK) return st;

  static std::atomic<uint64_t> smem_set{0};
  if ((st = mx_allow_smem(reinterpret_cast<const void*>(mx_gemm_kernel<F4, N0, N1>), C::SMEM, device, &smem_set)) != OQ_OK)
    return st;
  const int64_t grid = std::min<int64_t>(2 * kp.tiles, (int64_t)(sms & ~1));
  // stage counters are 32-bit
  if (((kp.tiles + grid / 2 - 1) / (grid / 2)) * (int64_t)kp.nkb >= (int64_t)1 << 31) return OQ_ERR_UNSUPPORTED;
  const cudaError_t e = mx_launch(mx_gemm_kernel<F4, N0, N1>, dim3((unsigned)grid), NTHREADS, C::SMEM, 0, stream, kp);
  if (e != cudaSuccess) {
    set_error(std::string("microscaled product launch: ") + cudaGetErrorString(e));
    return OQ_ERR_CUDA;
  }
  return OQ_OK;
}

// The tile's width: the one whose waves over the pairs cost least, a stage
// costing its feed (16 KB of activations, 64 bytes a column and the scales; the
// MMAs of every width take less or as much).
template <bool F4>
oq_status launch_width(const MxGemmArgs& g, cudaStream_t st) {
  int device = 0;
  const int sms = mx_sm_count(&device);
  const int64_t m_tiles = (g.T + 2 * RM - 1) / (2 * RM), pairs = sms / 2;
  int best = 0;
  int64_t cost = 0;
  for (const int pn : {448, 320, 256, 192, 128}) {
    const int64_t waves = (m_tiles * ((g.N + pn - 1) / pn) + pairs - 1) / pairs;
    const int64_t c = waves * (16384 + 1024 + 72 * pn);
    if (!best || c < cost) {
      best = pn;
      cost = c;
    }
  }
  switch (best) {
    case 448: return launch<F4, 256, 192>(g, sms, device, st);
    case 320: return launch<F4, 192, 128>(g, sms, device, st);
    case 256: return launch<F4, 256, 0>(g, sms, device, st);
    case 192: return launch<F4, 192, 0>(g, sms, device, st);
    default: return launch<F4, 128, 0>(g, sms, device, st);
  }
}

}  // namespace

oq_status mx_gemm_launch(const MxGemmArgs& g, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return g.a_bits == 4 ? launch_width<true>(g, st) : launch_width<false>(g, st);
}

}  // namespace oq
