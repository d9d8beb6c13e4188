// A paged cache of keys and values in microscaled e2m1 (4 bits, one E8M0 scale
// for 32 channels of a token), and the launches of the operators around it.
//
// Pages hold 128 tokens.  Heads lie side by side in groups of 128 channels (one
// head of 128, two of 64), and a page has for each group 272 rows of 64 bytes:
//   0-127    K codes: a token's 128 channels a row, the even channel in the low half
//   128-255  V codes transposed: a channel's 128 tokens a row, the even token low
//   256-263  K scales in the order the tensor cores take (mx_tile_word)
//   264-271  V scales, four bytes a token
// Both products of attention contract along a row (K over channels, V over
// tokens), so the tensor cores read the codes as they lie here.
#pragma once

#include "oq_mx.cuh"

struct oq_kv4 {
  int heads, kv_heads, head_dim;
  int groups;        // groups of 128 channels a token's keys fill
  int device;
  int* d_error;      // device error word
};

namespace oq {

constexpr int KV_PAGE = 128;                       // tokens of a page
constexpr int KV_ROWS = 272;                       // 64-byte rows of a page's group
constexpr int KV_V_ROW = 128, KV_KS_ROW = 256, KV_VS_ROW = 264;
constexpr int64_t KV_GROUP_BYTES = KV_ROWS * 64;

// Norm and rotation of heads: rows of D channels, heads[0] of x[0] and heads[1]
// of x[1] a token.  strides: elements from one token to the next.
struct RopeArgs {
  const void* x[2];
  void* out[2];
  int64_t in_stride[2], out_stride[2];
  int heads[2];
  const void* gain[2];       // or null: ones
  const float* table;        // [table_rows, rot / 2, 2] cos, sin, or null: no rotation
  const int* positions;      // [T], or null: the token's index (append: its place in the sequence)
  int64_t T, table_rows;
  float eps;
  int D, rot, dtype;
  bool gain_bf16, norm, interleaved;
};
oq_status rope_launch(const RopeArgs& a, void* stream);

// The cache as a call sees it: sequence b has lens[b] tokens, the last
// cu[b + 1] - cu[b] of them are the call's tokens cu[b] .. cu[b + 1] - 1.
struct KvView {
  uint8_t* cache;
  int64_t pages;             // of the cache
  const int* table;          // [B, width] page of a sequence's tokens 128 i ..
  const int* cu;             // [B + 1]
  const int* lens;           // [B]
  int B, width, groups;
};
struct AppendArgs {
  RopeArgs rope;             // x[0] = q (or null), x[1] = k; out[0] bf16
  const void* v;
  int64_t v_stride;
  KvView kv;
  int* err;
};
oq_status kv4_append_launch(const AppendArgs& a, void* stream);
struct ReadArgs {
  KvView kv;
  void* k;                   // [T, kv_heads, D] of dtype
  void* v;
  int64_t T;
  int kv_heads, D, dtype;
};
oq_status kv4_read_launch(const ReadArgs& a, void* stream);

struct AttentionArgs {
  KvView kv;
  const void* q;             // bf16, tokens q_stride elements apart
  int64_t q_stride, T;
  void* y;                   // bf16 [T, heads, D]
  float scale;
  int heads, kv_heads, D, max_q, max_len, window;
  bool causal;
  void* workspace;
  size_t workspace_bytes;
  int* err;
};
// a call's split over parts of the cache, which a second kernel joins
struct AttnSplit {
  AttentionArgs a;
  int splits, group;       // query heads per key head
  float* part_o;           // [splits][T][heads][D], relative to the reference
  float2* part_ml;         // [splits][T][heads]: log2 of the reference, sum
};
int kv4_chunk_splits(int kv_heads, int B, int group, int max_q, int64_t tiles, int sms);
oq_status kv4_chunk_launch(const AttnSplit& p, cudaStream_t st, int device);
size_t kv4_attention_workspace(const oq_kv4* kv, int64_t T, int B, int max_q, int max_len);
oq_status kv4_attention_launch(const AttentionArgs& a, void* stream);

// 4-bit weights with group scales (oq_w4g.cu)
struct W4gArgs {
  const void* x;             // [T, K]
  const uint8_t* codes;      // [N, K rounded up to 128, / 2]
  const void* scales;        // bf16 [N, K / group]
  const uint8_t* zeros;      // [N, K / group] or null
  void* y;                   // [T, N]
  int64_t T;
  int N, K, group, x_dtype, y_dtype;
};
oq_status w4g_linear_launch(const W4gArgs& a, void* stream);
oq_status w4g_prepare_launch(const void* W, int dtype, int N, int K, int group, uint8_t* codes, void* scales,
                             uint8_t* zeros, void* stream);

// The sequence and the range of a call's tokens that this CTA's index `i` stands
// for, when every sequence has as many units as its tokens' places in it touch
// aligned windows of W tokens.  All threads of the CTA get the same answer; `shared`
// is three ints.  False: there are fewer units.
template <int W>
__device__ __forceinline__ bool kv_window(const KvView& kv, int64_t T, int i, int* shared, int& b, int& first, int& count,
                                          int& place) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int before = 0, found = -1, win = 0;
    for (int b0 = 0; b0 < kv.B; b0 += 32) {
      const int bb = b0 + lane;
      int units = 0;
      if (bb < kv.B) {
        const int n = kv.cu[bb + 1] - kv.cu[bb], p0 = kv.lens[bb] - n;
        if (n > 0 && p0 >= 0) units = (p0 + n - 1) / W - p0 / W + 1;
      }
      int sum = units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += u;
      }
      const unsigned hit = __ballot_sync(0xFFFFFFFFu, before + sum > i);
      if (hit) {
        const int l = __ffs(hit) - 1;
        found = b0 + l;
        win = i - before - __shfl_sync(0xFFFFFFFFu, sum - units, l);
        break;
      }
      before += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) shared[0] = found, shared[1] = win;
  }
  __syncthreads();
  b = shared[0];
  if (b < 0) return false;
  const int c0 = kv.cu[b], n = kv.cu[b + 1] - c0, p0 = kv.lens[b] - n;
  const int w0 = (p0 / W + shared[1]) * W;           // the window's first place
  const int lo = w0 > p0 ? w0 : p0, hi = w0 + W < p0 + n ? w0 + W : p0 + n;
  place = lo;
  first = c0 + (lo - p0);
  count = hi - lo;
  // tokens that the arrays do not have, places that the table does not have
  if (c0 < 0 || first + count > T || (lo >> 7) >= kv.width) return false;
  return true;
}

}  // namespace oq
