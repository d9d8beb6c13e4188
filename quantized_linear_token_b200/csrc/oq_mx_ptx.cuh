// Inline PTX of the block-scaled tensor-core path (sm_100a): three-dimensional
// TMA loads of scale tiles, the copy of scales from shared to tensor memory,
// and tcgen05.mma with block scales, one CTA or a CTA pair.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <string>

#include "oq_mx.cuh"
#include "oq_ptx.cuh"
#include "oq_tmap.cuh"

namespace oq {

__device__ __forceinline__ void tma_load_3d(void* dst_smem, const void* tmap, int32_t x, int32_t y, int32_t z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(smem_u32(dst_smem)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}
// the form for CTA pairs: bytes counted on a barrier that may lie in the peer CTA (no multicast)
__device__ __forceinline__ void tma_load_3d_pair(void* dst_smem, const void* tmap, int32_t x, int32_t y, int32_t z,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
      "%4}], [%5];" ::"r"(smem_u32(dst_smem)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(bar_cluster)
      : "memory");
}

// Descriptor of a 512-byte scale tile for tcgen05.cp.32x128b: 32 rows of 16
// bytes, unswizzled, groups of eight rows 128 bytes apart.
__device__ __forceinline__ uint64_t smem_desc_scales(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)(128 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  return d;
}

// One scale tile into four tensor-memory columns: column c, lane l gets the
// 32-bit word of row 32 c + l (its four block scales), repeated in the four
// lane quarters.  With CG = 2 each CTA of the pair copies from its own shared
// memory, at the same offset, into its own tensor memory.  Copies and MMAs
// issued by one thread run in issue order.
template <int CG>
__device__ __forceinline__ void tc_copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

// one lane of a converged warp
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r;
}

// Block-scaled MMA of one CTA, K of 32 bytes per row: F4 multiplies 64 e2m1 by
// 64 e2m1 with two scales a row, otherwise 32 elements in 8-bit containers (e4m3,
// or e2m1 as TMA spreads it: 8 bytes of codes in every 16) with one.
template <bool F4>
__device__ __forceinline__ void tc_mma_mx(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
#define OQ_MX_MMA(KIND, VEC)                                                                             \
  asm volatile(                                                                                          \
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                   \
      "tcgen05.mma.cta_group::1.kind::" KIND ".block_scale.scale_vec::" VEC                              \
      " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),                                            \
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                           \
      : "memory")
  if constexpr (F4) OQ_MX_MMA("mxf4", "2X");
  else OQ_MX_MMA("mxf8f6f4", "1X");
#undef OQ_MX_MMA
}

// Instruction descriptor of the block-scaled kinds: K-major operands, E8M0
// scales; a_fmt / b_fmt 1 for e2m1 in kind::mxf4, and 0 for e4m3, 5 for e2m1
// in kind::mxf8f6f4.
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N, uint32_t a_fmt, uint32_t b_fmt) {
  return (a_fmt << 7) | (b_fmt << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 7) << 27);
}
// the scale's place in its 32-bit column: byte 0..3 (one scale per MMA), or 0 / 2 (two)
__host__ __device__ constexpr uint32_t idesc_mx_sf(uint32_t id) { return (id << 4) | (id << 29); }

// Arrival on a barrier of the cluster that hands over tensor memory only: the
// caller's tcgen05 loads are complete and fenced (before_thread_sync), and no
// ordinary memory goes with it, so the default scope does; a release at cluster
// scope would wait some 1000 cycles for the thread's stores.
__device__ __forceinline__ void mbar_arrive_tmem(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// Which of the phases `parity` (bit j) of the barriers bar[slot[j]] have
// completed: three non-blocking checks whose latencies overlap.  Bit j is only
// asked for where `want` has it.
__device__ __forceinline__ uint32_t mbar_test3(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t parity,
                                                       uint32_t want) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p0, p1, p2, q0, q1, q2;\n\t.reg .b32 t0, t1, t2, u;\n\t"
      "and.b32 u, %5, 1;\n\tsetp.ne.b32 q0, u, 0;\n\tand.b32 u, %5, 2;\n\tsetp.ne.b32 q1, u, 0;\n\t"
      "and.b32 u, %5, 4;\n\tsetp.ne.b32 q2, u, 0;\n\t"
      "and.b32 t0, %4, 1;\n\tshr.u32 t1, %4, 1;\n\tand.b32 t1, t1, 1;\n\tshr.u32 t2, %4, 2;\n\tand.b32 t2, t2, 1;\n\t"
      "setp.ne.b32 p0, 0, 0;\n\tsetp.ne.b32 p1, 0, 0;\n\tsetp.ne.b32 p2, 0, 0;\n\t"
      "@q0 mbarrier.test_wait.parity.shared::cta.b64 p0, [%1], t0;\n\t"
      "@q1 mbarrier.test_wait.parity.shared::cta.b64 p1, [%2], t1;\n\t"
      "@q2 mbarrier.test_wait.parity.shared::cta.b64 p2, [%3], t2;\n\t"
      "selp.u32 t0, 1, 0, p0;\n\tselp.u32 t1, 2, 0, p1;\n\tselp.u32 t2, 4, 0, p2;\n\t"
      "or.b32 t0, t0, t1;\n\tor.b32 %0, t0, t2;\n\t}"
      : "=r"(r)
      : "r"(b0), "r"(b1), "r"(b2), "r"(parity), "r"(want)
      : "memory");
  return r;
}

// Half a stage of a CTA pair: two K steps of the tile's column parts (one, or
// two with TWO: two or four MMAs) with the scale copies of the NEXT half between them, so that no MMA
// waits for a copy just issued.  `commit` reports everything issued so far to
// `commit_bar` in both CTAs.
//   a, b0, b1     low descriptor words of the operand tiles at the first K step (+2: the second)
//   i0a .. i1b    instruction descriptors of part 0 / 1 at the two K steps
//   sf, w0, w1    scale columns of A and of the two parts' weight rows
//   sf_next       columns of the copies: 4 of A, then 4 of each of RT weight row tiles
//   ca, cw        low descriptor words of their shared-memory tiles (weights' row tiles STRIDE apart)
struct MxHalf {
  uint32_t lead;   // this lane issues
  uint32_t d0, d1, a, b0, b1, hi, i0a, i0b, i1a, i1b, sf, w0, w1, accumulate;
  uint32_t sf_next, ca, cw, c_hi, copy;
  uint64_t* commit_bar;
  uint32_t commit;
};
template <bool F4, bool TWO, int RT, int STRIDE>
__device__ __forceinline__ void tc_half_stage_pair(const MxHalf& h) {
#define OQ_DESC(R, LO, OFF, HI) "add.u32 lo, " LO ", " OFF ";\n\tmov.b64 " R ", {lo, " HI "};\n\t"
#define OQ_MMA(KIND, VEC, D, ID, W, P)                                                                      \
  "@pl tcgen05.mma.cta_group::2.kind::" KIND ".block_scale.scale_vec::" VEC " [" D "], da, db, " ID ", [%11], [" W "], " P \
  ";\n\t"
#define OQ_CP(P, COL, LO, OFF)                                                                              \
  "add.u32 t, %15, " COL ";\n\t" OQ_DESC("ds", LO, OFF, "%18")                                              \
  "@" P " tcgen05.cp.cta_group::2.32x128b.warpx4 [t], ds;\n\t"
#define OQ_HALF(KIND, VEC, PART1)                                                                              \
  "{\n\t.reg .pred pl, pa, pt, pc, c0, c1, c2, c3, c4;\n\t.reg .b64 da, db, ds;\n\t.reg .b32 lo, t;\n\t"    \
  "setp.ne.b32 pl, %0, 0;\n\tsetp.ne.b32 pa, %14, 0;\n\tsetp.eq.b32 pt, 0, 0;\n\t"                                  \
  "setp.ne.and.b32 pc, %21, 0, pl;\n\tsetp.ne.and.b32 c0, %19, 0, pl;\n\tsetp.gt.and.s32 c1, %23, 0, c0;\n\t"                \
  "setp.gt.and.s32 c2, %23, 1, c0;\n\tsetp.gt.and.s32 c3, %23, 2, c0;\n\tsetp.gt.and.s32 c4, %23, 3, c0;\n\t" \
  OQ_DESC("da", "%3", "0", "%6") OQ_DESC("db", "%4", "0", "%6") OQ_MMA(KIND, VEC, "%1", "%7", "%12", "pa")  \
  OQ_CP("c0", "0", "%16", "0")                                                                              \
  OQ_DESC("da", "%3", "2", "%6") OQ_DESC("db", "%4", "2", "%6") OQ_MMA(KIND, VEC, "%1", "%8", "%12", "pt")  \
  OQ_CP("c1", "4", "%17", "0") OQ_CP("c2", "8", "%17", "%24") PART1                                         \
  "@pc tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%20], %22;\n\t" \
  "}"
#define OQ_PART1(KIND, VEC)                                                                                 \
  OQ_DESC("da", "%3", "0", "%6") OQ_DESC("db", "%5", "0", "%6") OQ_MMA(KIND, VEC, "%2", "%9", "%13", "pa")  \
  OQ_CP("c3", "12", "%17", "%25") OQ_CP("c4", "16", "%17", "%26")                                           \
  OQ_DESC("da", "%3", "2", "%6") OQ_DESC("db", "%5", "2", "%6") OQ_MMA(KIND, VEC, "%2", "%10", "%13", "pt")
#define OQ_ARGS                                                                                             \
  :                                                                                                         \
  : "r"(h.lead), "r"(h.d0), "r"(h.d1), "r"(h.a), "r"(h.b0), "r"(h.b1), "r"(h.hi), "r"(h.i0a), "r"(h.i0b), "r"(h.i1a),     \
    "r"(h.i1b), "r"(h.sf), "r"(h.w0), "r"(h.w1), "r"(h.accumulate), "r"(h.sf_next), "r"(h.ca), "r"(h.cw),    \
    "r"(h.c_hi), "r"(h.copy), "r"(smem_u32(h.commit_bar)), "r"(h.commit),                                    \
    "h"((uint16_t)0x3), "n"(RT), "n"(STRIDE), "n"(2 * STRIDE),            \
    "n"(3 * STRIDE)                                                                                         \
  : "memory"
  static_assert(TWO || RT <= 2, "one part's copies follow its two MMAs");
  if constexpr (F4 && TWO) asm volatile(OQ_HALF("mxf4", "2X", OQ_PART1("mxf4", "2X")) OQ_ARGS);
  else if constexpr (F4) asm volatile(OQ_HALF("mxf4", "2X", "") OQ_ARGS);
  else if constexpr (TWO) asm volatile(OQ_HALF("mxf8f6f4", "1X", OQ_PART1("mxf8f6f4", "1X")) OQ_ARGS);
  else asm volatile(OQ_HALF("mxf8f6f4", "1X", "") OQ_ARGS);
#undef OQ_ARGS
#undef OQ_PART1
#undef OQ_HALF
#undef OQ_CP
#undef OQ_MMA
#undef OQ_DESC
}

// ------------------------------------------------------------------ tensor maps
inline oq_status mx_encode(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base, const cuuint64_t* dims,
                           const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle sw, const char* what) {
  EncodeTiledFn fn = nullptr;
  const oq_status st = tmap_encode_fn(&fn);
  if (st != OQ_OK) return st;
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, dt, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error(std::string("cuTensorMapEncodeTiled failed for ") + what + " (code " + std::to_string((int)r) + ")");
    return OQ_ERR_CUDA;
  }
  return OQ_OK;
}

// Code rows in boxes of box_rows x 128 shared-memory bytes (one row of the
// 128-byte swizzle).  Codes of 8 bits, and 4-bit codes for the 4-bit MMA,
// travel as bytes; `expand` spreads 4-bit codes to the 8-bit containers of
// kind::mxf8f6f4 on the way (128 codes a box row).  Rows and columns past the
// end read as zeros.  The x coordinate is in bytes, or in codes with `expand`;
// both step by 128.
inline oq_status mx_encode_codes(CUtensorMap* map, const uint8_t* base, int64_t rows, int K, int bits, bool expand,
                                 int box_rows, const char* what) {
  const cuuint64_t row_bytes = (cuuint64_t)mx_row_bytes(K, bits);
  const cuuint64_t dims[2] = {expand ? 2 * row_bytes : row_bytes, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {128, (cuuint32_t)box_rows};
  return mx_encode(map, expand ? CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims,
                   strides, box, CU_TENSOR_MAP_SWIZZLE_128B, what);
}

// Scale tiles [row tile][column tile][512 bytes] in boxes of row_tiles x
// col_tiles tiles; tiles past the end read as zeros (scale code 0).
inline oq_status mx_encode_scales(CUtensorMap* map, const uint8_t* base, int64_t rows, int K, int box_row_tiles,
                                  int box_col_tiles, const char* what) {
  const cuuint64_t ct = (cuuint64_t)mx_col_tiles(K);
  const cuuint64_t dims[3] = {MX_TILE_BYTES / 4, ct, (cuuint64_t)mx_row_tiles(rows)};
  const cuuint64_t strides[2] = {MX_TILE_BYTES, MX_TILE_BYTES * ct};
  const cuuint32_t box[3] = {MX_TILE_BYTES / 4, (cuuint32_t)box_col_tiles, (cuuint32_t)box_row_tiles};
  return mx_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE, what);
}

}  // namespace oq
