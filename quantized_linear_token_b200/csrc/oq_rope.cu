// Norms of queries and keys for each head with the position rotation in the
// same pass, and the same pass with keys and values going to the 4-bit cache.
//
//   n_i = x_i g_i / sqrt(mean(x^2) + eps)                 over a head's D channels
//   (a, b) -> (a cos - b sin, b cos + a sin)              for the first `rot` channels,
//   pairs (2 i, 2 i + 1) or (i, i + rot / 2), cos and sin from a table row.
//
// A row (a token's head) is held by 4 to 32 neighbouring lanes, eight channels
// each, so the mean is a few shuffles and nothing is read twice.  A lane keeps
// its place in the row for all heads of a token: gains and the token's cos and
// sin are loaded once.  Bound: HBM for many tokens, the latency of one dependent
// load and of the launch for one.
#include <cuda_bf16.h>

#include <algorithm>

#include "oq_kv4.cuh"

namespace oq {
namespace {

constexpr int NT = 256;   // threads of a CTA

// cos and sin of this lane's channels.  Interleaved pairs: c[j], s[j] for pair j
// of the four; halves: for each of the eight channels, s negated in the first half.
template <bool INTER>
struct Turn {
  float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
  bool on;        // these channels are rotated
  int partner;    // halves: lane distance of the other half (signed)
};

template <bool INTER>
__device__ __forceinline__ Turn<INTER> load_turn(const float* table, int64_t rows, int64_t pos, int rot, int ch) {
  Turn<INTER> t;
  t.on = table != nullptr && ch < rot;
  t.partner = 0;
  if (!t.on) return t;
  const bool ok = pos >= 0 && pos < rows;   // a place outside the table makes the channels NaN
  const float* row = table + (ok ? pos : 0) * rot;
  const int half = rot >> 1;
  if constexpr (INTER) {
    const float4* p = reinterpret_cast<const float4*>(row + ch);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    t.c[0] = a.x, t.s[0] = a.y, t.c[1] = a.z, t.s[1] = a.w;
    t.c[2] = b.x, t.s[2] = b.y, t.c[3] = b.z, t.s[3] = b.w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!ok) t.c[i] = t.s[i] = __int_as_float(0x7FC00000);
  } else {
    const bool second = ch >= half;
    const float4* p = reinterpret_cast<const float4*>(row + 2 * (second ? ch - half : ch));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = __ldg(p + i);
      t.c[2 * i] = a.x, t.s[2 * i] = second ? a.y : -a.y, t.c[2 * i + 1] = a.z, t.s[2 * i + 1] = second ? a.w : -a.w;
    }
    t.partner = second ? -(half >> 3) : half >> 3;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!ok) t.c[i] = t.s[i] = __int_as_float(0x7FC00000);
  }
  return t;
}

template <typename F>
__device__ __forceinline__ F group_sum(F v, int lanes) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// the rotation in F (fp32 or fp64) of this lane's eight channels, in place
template <bool INTER, typename F>
__device__ __forceinline__ void rotate(F (&n)[8], const Turn<INTER>& t) {
  if constexpr (INTER) {
    if (t.on) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const F a = n[2 * j], b = n[2 * j + 1], c = (F)t.c[j], s = (F)t.s[j];
        n[2 * j] = a * c - b * s;
        n[2 * j + 1] = b * c + a * s;
      }
    }
  } else {
    const int lane = threadIdx.x & 31, from = lane + t.partner;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const F o = __shfl_sync(0xFFFFFFFFu, n[j], from);
      if (t.on) n[j] = n[j] * (F)t.c[j] + o * (F)t.s[j];
    }
  }
}

// Whether the sum of squares in fp32 is good to fp32's precision: it neither
// overflowed nor lost squares that eps does not hide.
__device__ __forceinline__ bool plain_range(float ss, float eps) { return ss < 3e38f && (ss > 1e-30f || eps > 1e-24f); }

// n = x g inv of a row held by `lanes` lanes; rows out of fp32's range in fp64
__device__ __forceinline__ void head_norm(float (&n)[8], const float (&g)[8], float eps, float inv_d, int lanes, bool norm) {
  if (!norm) return;
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(n[j], n[j], ss);
  ss = group_sum(ss, lanes);
  if (__all_sync(0xFFFFFFFFu, plain_range(ss, eps))) {
    const float inv = 1.0f / sqrtf(fmaf(ss, inv_d, eps));
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = n[j] * inv * g[j];
  } else {
    double sd = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) sd += (double)n[j] * (double)n[j];
    sd = group_sum(sd, lanes);
    const double inv = 1.0 / sqrt(sd * (double)inv_d + (double)eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = (float)((double)n[j] * inv * (double)g[j]);
  }
}

__device__ __forceinline__ void load_gain(float (&g)[8], const void* gain, bool bf16, int ch, bool in) {
  if (gain && in && bf16) {
    Vec8<__nv_bfloat16> v;
    v.load(static_cast<const __nv_bfloat16*>(gain) + ch);
    v.get(g);
  } else if (gain && in) {
    Vec8<float> v;
    v.load(static_cast<const float*>(gain) + ch);
    v.get(g);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 1.f;
  }
}

// Heads sub, sub + step, .. of a token: first those of x[0], then those of x[1].
// All lanes of a warp make the same number of turns.
template <typename T, typename OUT, bool INTER>
__device__ __forceinline__ void rope_token(const RopeArgs& p, int64_t t, bool token, int sub, int step, int lanes, int rows,
                                           int64_t pos) {
  const int vec = (int)threadIdx.x & (lanes - 1), ch = vec * 8;
  const bool in = token && ch < p.D;
  const Turn<INTER> turn = load_turn<INTER>(in ? p.table : nullptr, p.table_rows, pos, p.rot, ch);
  float g0[8], g1[8];
  load_gain(g0, p.gain[0], p.gain_bf16, ch, in);
  load_gain(g1, p.gain[1], p.gain_bf16, ch, in);
  const float inv_d = 1.0f / (float)p.D;
  auto at = [&](int r, int& which) -> int64_t {
    which = r >= p.heads[0];
    return t * p.in_stride[which] + (int64_t)(which ? r - p.heads[0] : r) * p.D + ch;
  };
  Vec8<T> next;
  next.zero();
  int which = 0;
  if (in && sub < rows) {
    const int64_t a = at(sub, which);
    next.load(static_cast<const T*>(p.x[which]) + a);
  }
  const int turns = (rows + step - 1) / step;
#pragma unroll 1
  for (int i = 0; i < turns; ++i) {
    const int r = sub + i * step;
    float n[8];
    next.get(n);
    const int w = which;
    if (in && r + step < rows) {
      const int64_t a = at(r + step, which);
      next.load(static_cast<const T*>(p.x[which]) + a);
    } else {
      next.zero();
    }
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = w ? g1[j] : g0[j];
    head_norm(n, g, p.eps, inv_d, lanes, p.norm);
    rotate<INTER, float>(n, turn);
    if (in && r < rows)
      store8(static_cast<OUT*>(p.out[w]) + t * p.out_stride[w] + (int64_t)(w ? r - p.heads[0] : r) * p.D + ch, n);
  }
}

struct RopeGrid {
  int lanes;      // lanes of a row
  int per_token;  // rows of a token that a CTA does at once
  int tokens;     // tokens of a CTA
  int split;      // CTAs that share a token's rows
};
struct RopeParams {
  RopeArgs a;
  RopeGrid g;
};

template <typename T, bool INTER>
__global__ void __launch_bounds__(NT) rope_kernel(const __grid_constant__ RopeParams p) {
  dependency_wait();
  const int grp = (int)threadIdx.x / p.g.lanes;
  const int64_t t = (int64_t)blockIdx.x * p.g.tokens + grp / p.g.per_token;
  const bool token = t < p.a.T;
  const int64_t pos = !token ? 0 : p.a.positions ? (int64_t)p.a.positions[t] : t;
  rope_token<T, T, INTER>(p.a, t, token, (int)blockIdx.y * p.g.per_token + grp % p.g.per_token, p.g.split * p.g.per_token,
                          p.g.lanes, p.a.heads[0] + p.a.heads[1], pos);
}

int row_lanes(int D) {
  int l = 4;
  while (l * 8 < D) l *= 2;
  return l;
}

// A CTA takes one token (several where a token has few heads); few tokens are
// shared by several CTAs, up to two for each SM.
RopeGrid rope_grid(int64_t T, int rows, int D, int sms) {
  RopeGrid g;
  g.lanes = row_lanes(D);
  const int groups = NT / g.lanes;
  g.per_token = 1;
  while (g.per_token < groups && g.per_token < rows) g.per_token *= 2;
  g.tokens = groups / g.per_token;
  const int64_t ctas = (T + g.tokens - 1) / g.tokens;
  const int turns = (rows + g.per_token - 1) / g.per_token;
  g.split = (int)std::max<int64_t>(1, std::min<int64_t>(turns, 2 * (int64_t)sms / ctas));
  return g;
}

oq_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return OQ_OK;
  set_error(std::string(what) + " launch: " + cudaGetErrorString(e));
  return OQ_ERR_CUDA;
}

// ------------------------------------------------------------------ append
// A CTA of the cache's part takes one group of 128 channels of up to 32 tokens
// whose places share an aligned window of 32, so that no byte of V (two tokens)
// and no sector of its transposed rows is written by two CTAs.  Keys go the way
// of the queries and are then quantised; values are quantised as they are and
// transposed through shared memory.
//
// A key's codes are those of the value in exact arithmetic: its fp32 value is
// off by less than DELTA of |a| + |b| (the pair it was turned from), and where
// that could change a code or the block's scale, the row is formed again in fp64
// and rounded once.  (The sum of squares takes 8 + 4 roundings, halved by the
// root; the mean, the root, the quotient, two products and the rotation's three
// operations add at most 9 half-ulps: below 16 * 2^-24, taken as 32 * 2^-24.)
constexpr float DELTA = 32.f / 16777216.f;

struct AppendParams {
  AppendArgs a;
  RopeGrid g;
  int q_ctas, kv_units, kv_heads, D;
};

__device__ __forceinline__ float round_odd(double w) {
  float f = __double2float_rz(w);
  if ((double)f != w) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

// largest of four neighbouring lanes
__device__ __forceinline__ float max4(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}

// Eight channels of a key (norm, rotation) -> codes and the block's scale code.
template <typename T, bool INTER>
__device__ __forceinline__ uint32_t key_codes(const Vec8<T>& raw, const RopeArgs& p, const float (&g)[8],
                                              const Turn<INTER>& turn, int lanes, float inv_d, uint32_t& scale) {
  float n[8], mag[8], w[8];
  raw.get(n);
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss = fmaf(n[j], n[j], ss);
  ss = group_sum(ss, lanes);
  bool doubt = p.norm && !plain_range(ss, p.eps);
  if (p.norm) {
    const float inv = 1.0f / sqrtf(fmaf(ss, inv_d, p.eps));
#pragma unroll
    for (int j = 0; j < 8; ++j) n[j] = n[j] * inv * g[j];
  }
  const float delta = p.norm || p.table ? DELTA : 0.f;
  // |a| + |b|, scaled to the possible error
  float most = 0.f;
  if constexpr (INTER) {
#pragma unroll
    for (int j = 0; j < 8; ++j) mag[j] = delta * (fabsf(n[j]) + (turn.on ? fabsf(n[j ^ 1]) : 0.f));
  } else {
    const int from = ((int)threadIdx.x & 31) + turn.partner;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float o = __shfl_sync(0xFFFFFFFFu, n[j], from);
      mag[j] = delta * (fabsf(n[j]) + (turn.on ? fabsf(o) : 0.f));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) most = fmaxf(most, mag[j]);
  most = max4(most);
  rotate<INTER, float>(n, turn);
  const uint32_t block = mx_block_max(n);
  scale = mx_scale_code<4>(block);
  const float top = __uint_as_float(block);
  doubt |= scale != 255u && (__float_as_uint(top + most) >> 23) != (__float_as_uint(fmaxf(top - most, 0.f)) >> 23);
  const float inv_s = mx_inverse_scale(scale);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = n[j] * inv_s;
  uint32_t out[1];
  mx_element_codes<4>(w, scale, out);
  if (delta > 0.f) {
    doubt |= top > 0.f && top < 1e-30f;   // products below fp32's normal numbers are off by more
    float lo[8], hi[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lo[j] = fmaxf(fabsf(w[j]) - mag[j] * inv_s, 0.f);
      hi[j] = fabsf(w[j]) + mag[j] * inv_s;
    }
    doubt |= scale != 255u && cvt8_e2m1(lo) != cvt8_e2m1(hi);
    if (__any_sync(0xFFFFFFFFu, doubt)) {
      double d[8], top_d = 0.0;
      raw.get(n);
      double sd = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[j] = (double)n[j];
        sd += d[j] * d[j];
      }
      sd = group_sum(sd, lanes);
      if (p.norm) {
        const double root = sqrt(sd / (double)p.D + (double)p.eps);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = d[j] / root * (double)g[j];
      }
      rotate<INTER, double>(d, turn);
      bool bad = false;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        bad |= !(fabs(d[j]) <= 3.4028234663852886e38);
        top_d = fmax(top_d, fabs(d[j]));
      }
      float f = bad ? __int_as_float(0x7F800000) : __double2float_rz(top_d);
      f = max4(f);
      scale = mx_scale_code<4>(__float_as_uint(f));
      const double s = (double)mx_inverse_scale(scale);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = round_odd(d[j] * s);
      mx_element_codes<4>(w, scale, out);
    }
  }
  return out[0];
}

template <typename T, bool INTER>
__global__ void __launch_bounds__(NT) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int found[4];
  __shared__ __align__(16) uint8_t tile[128 * 36];   // V codes, one a byte: [channel][token], rows 36 bytes apart
  const RopeArgs& r = p.a.rope;
  const KvView& kv = p.a.kv;
  dependency_wait();
  if ((int)blockIdx.x < p.q_ctas) {
    // the queries of one token
    const int64_t t = blockIdx.x / p.g.split;
    const int part = (int)(blockIdx.x % p.g.split);
    int64_t pos = 0;
    if (r.positions) {
      pos = r.positions[t];
    } else {
      // the token's sequence: how many of them end at or before it
      int ends = 0;
      for (int b = threadIdx.x; b < kv.B; b += NT) ends += kv.cu[b + 1] <= t;
      if (threadIdx.x == 0) found[0] = 0;
      __syncthreads();
      if (ends) atomicAdd(&found[0], ends);
      __syncthreads();
      const int b = min(found[0], kv.B - 1);
      pos = (int64_t)kv.lens[b] - kv.cu[b + 1] + t;
    }
    const int grp = (int)threadIdx.x / p.g.lanes, groups = NT / p.g.lanes;
    rope_token<T, __nv_bfloat16, INTER>(r, t, true, part * groups + grp, p.g.split * groups, p.g.lanes, r.heads[0], pos);
    return;
  }
  const int unit = ((int)blockIdx.x - p.q_ctas) / kv.groups, hg = ((int)blockIdx.x - p.q_ctas) % kv.groups;
  int b, first, count, place;
  if (!kv_window(kv, r.T, unit, found, b, first, count, place)) return;
  const int64_t page = kv.table[(int64_t)b * kv.width + (place >> 7)];
  if (page < 0 || page >= kv.pages) return;
  uint8_t* base = kv.cache + (page * kv.groups + hg) * KV_GROUP_BYTES;
  const int lanes = p.D / 8, sub = (int)threadIdx.x & 15, head = hg * (128 / p.D) + sub / lanes;
  const int vec = sub & (lanes - 1), ch = vec * 8;   // 16 lanes hold the group's 128 channels of a token
  const bool has = head < p.kv_heads;
  float g[8];
  load_gain(g, r.gain[1], r.gain_bf16, ch, has);
  const float inv_d = 1.0f / (float)p.D;
  const int w0 = place & 127 & ~31;                  // the window's first row in its page
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = half * 16 + ((int)threadIdx.x >> 4);   // of the window
    const int i = row - (place & 31);
    const bool token = i >= 0 && i < count;
    const int64_t t = first + i;
    Vec8<T> k, v;
    k.zero();
    v.zero();
    if (token && has) {
      k.load(static_cast<const T*>(r.x[1]) + t * r.in_stride[1] + (int64_t)head * p.D + ch);
      v.load(static_cast<const T*>(p.a.v) + t * p.a.v_stride + (int64_t)head * p.D + ch);
    }
    const int64_t pos = !token ? 0 : r.positions ? (int64_t)r.positions[t] : (int64_t)(place + i);
    const Turn<INTER> turn = load_turn<INTER>(token && has ? r.table : nullptr, r.table_rows, pos, r.rot, ch);
    uint32_t ks, vs, kc, vc[1];
    kc = key_codes<T, INTER>(k, r, g, turn, lanes, inv_d, ks);
    if (!has) kc = 0u, ks = 0u;
    float x[8];
    v.get(x);
    vs = mx_scale_code<4>(mx_block_max(x));
    const float inv_s = mx_inverse_scale(vs);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] *= inv_s;
    mx_element_codes<4>(x, vs, vc);
    const uint32_t kw = mx_scale_word(ks), vw = mx_scale_word(vs);
    if (token) {
      const int at = w0 + row;
      *reinterpret_cast<uint32_t*>(base + at * 64 + sub * 4) = kc;
      if (sub == 0) {
        *reinterpret_cast<uint32_t*>(base + KV_KS_ROW * 64 + mx_tile_word(at) * 4) = kw;
        *reinterpret_cast<uint32_t*>(base + KV_VS_ROW * 64 + at * 4) = vw;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) tile[(sub * 8 + j) * 36 + row] = (uint8_t)((vc[0] >> (4 * j)) & 15u);
  }
  __syncthreads();
  // a thread packs a channel's 32 tokens; tokens that are not the call's keep their codes
  if (threadIdx.x < 128) {
    const uint32_t* src = reinterpret_cast<const uint32_t*>(tile + threadIdx.x * 36);
    uint4* dst = reinterpret_cast<uint4*>(base + (KV_V_ROW + threadIdx.x) * 64 + (w0 >> 5) * 16);
    uint32_t out[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t x = src[2 * q], y = src[2 * q + 1];
      x |= x >> 4;
      y |= y >> 4;
      out[q] = __byte_perm(x, y, 0x6420);
    }
    if (count != 32) {
      const uint4 old = *dst;
      const uint32_t o[4] = {old.x, old.y, old.z, old.w};
      const int lo = place & 31, hi = lo + count;   // nibbles [lo, hi) of the 32 are new
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int a = min(max(lo - 8 * q, 0), 8), e = min(max(hi - 8 * q, 0), 8);
        const uint32_t below_e = e == 8 ? 0xFFFFFFFFu : (1u << (4 * e)) - 1u;
        const uint32_t below_a = a == 8 ? 0xFFFFFFFFu : (1u << (4 * a)) - 1u;
        const uint32_t mask = below_e & ~below_a;
        out[q] = (out[q] & mask) | (o[q] & ~mask);
      }
    }
    *dst = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// ------------------------------------------------------------------ read back
// e2m1 of the low nibble
__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const uint32_t m = c & 7u;
  const float v = m < 2u ? 0.5f * (float)m : __uint_as_float(((m >> 1) + 126u) << 23 | (m & 1u) << 22);
  return c & 8u ? -v : v;
}
__device__ __forceinline__ float scale_value(uint32_t code) {
  return code == 255u ? __int_as_float(0x7FC00000) : code == 0u ? __uint_as_float(1u << 22) : __uint_as_float(code << 23);
}

template <typename T>
__global__ void __launch_bounds__(NT) read_kernel(const __grid_constant__ ReadArgs p) {
  __shared__ int found[4];
  __shared__ __align__(16) uint32_t rows[128 * 5];   // V: a channel's 32 tokens, rows 20 bytes apart
  const KvView& kv = p.kv;
  dependency_wait();
  const int unit = (int)blockIdx.x / kv.groups, hg = (int)blockIdx.x % kv.groups;
  int b, first, count, place;
  if (!kv_window(kv, p.T, unit, found, b, first, count, place)) return;
  const int64_t page = kv.table[(int64_t)b * kv.width + (place >> 7)];
  const bool ok = page >= 0 && page < kv.pages;   // a page that is not there reads as NaN
  const uint8_t* base = kv.cache + ((ok ? page : 0) * kv.groups + hg) * KV_GROUP_BYTES;
  const int w0 = place & 127 & ~31;
  if (threadIdx.x < 128) {
    const uint4 v = *reinterpret_cast<const uint4*>(base + (KV_V_ROW + threadIdx.x) * 64 + (w0 >> 5) * 16);
    uint32_t* d = rows + threadIdx.x * 5;
    d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
  }
  __syncthreads();
  const int sub = (int)threadIdx.x & 15, c0 = hg * 128 + sub * 8, blk = sub >> 2;
  if (c0 >= p.kv_heads * p.D) return;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = half * 16 + ((int)threadIdx.x >> 4), i = row - (place & 31), at = w0 + row;
    if (i < 0 || i >= count) continue;
    const uint32_t kc = *reinterpret_cast<const uint32_t*>(base + at * 64 + sub * 4);
    const float ks = scale_value(ok ? base[KV_KS_ROW * 64 + mx_tile_word(at) * 4 + blk] : 255u);
    const float vs = scale_value(ok ? base[KV_VS_ROW * 64 + at * 4 + blk] : 255u);
    float k[8], v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      k[j] = e2m1_value(kc >> (4 * j)) * ks;
      v[j] = e2m1_value(rows[(sub * 8 + j) * 5 + (row >> 3)] >> (4 * (row & 7))) * vs;
    }
    const int64_t o = (int64_t)(first + i) * p.kv_heads * p.D + c0;
    store8(static_cast<T*>(p.k) + o, k);
    store8(static_cast<T*>(p.v) + o, v);
  }
}

// units of kv_window that B sequences with T tokens may have
int64_t window_units(int64_t T, int B) { return std::min<int64_t>(T, T / 32 + 2 * (int64_t)B); }

}  // namespace

oq_status rope_launch(const RopeArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  RopeParams p;
  p.a = a;
  p.g = rope_grid(a.T, a.heads[0] + a.heads[1], a.D, mx_sm_count(&dev));
  const int64_t ctas = (a.T + p.g.tokens - 1) / p.g.tokens;
  if (ctas > 0x7FFFFFFF) return OQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas, (unsigned)p.g.split);
  cudaError_t e;
  if (a.dtype == OQ_DTYPE_BF16)
    e = a.interleaved ? mx_launch(rope_kernel<__nv_bfloat16, true>, grid, NT, 0, 0, st, p)
                      : mx_launch(rope_kernel<__nv_bfloat16, false>, grid, NT, 0, 0, st, p);
  else
    e = a.interleaved ? mx_launch(rope_kernel<float, true>, grid, NT, 0, 0, st, p)
                      : mx_launch(rope_kernel<float, false>, grid, NT, 0, 0, st, p);
  return launched(e, "norm and rotation");
}

oq_status kv4_append_launch(const AppendArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  AppendParams p;
  p.a = a;
  p.D = a.rope.D;
  p.kv_heads = a.rope.heads[1];
  p.g = rope_grid(a.rope.T, std::max(a.rope.heads[0], NT / row_lanes(p.D)), p.D, mx_sm_count(&dev));
  const int64_t q = a.rope.x[0] ? a.rope.T * p.g.split : 0, units = window_units(a.rope.T, a.kv.B);
  if (q + units * a.kv.groups > 0x7FFFFFFF) return OQ_ERR_UNSUPPORTED;
  p.q_ctas = (int)q;
  p.kv_units = (int)units;
  const dim3 grid((unsigned)(q + units * a.kv.groups));
  cudaError_t e;
  if (a.rope.dtype == OQ_DTYPE_BF16)
    e = a.rope.interleaved ? mx_launch(append_kernel<__nv_bfloat16, true>, grid, NT, 0, 0, st, p)
                           : mx_launch(append_kernel<__nv_bfloat16, false>, grid, NT, 0, 0, st, p);
  else
    e = a.rope.interleaved ? mx_launch(append_kernel<float, true>, grid, NT, 0, 0, st, p)
                           : mx_launch(append_kernel<float, false>, grid, NT, 0, 0, st, p);
  return launched(e, "cache append");
}

oq_status kv4_read_launch(const ReadArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t ctas = window_units(a.T, a.kv.B) * a.kv.groups;
  if (ctas > 0x7FFFFFFF) return OQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas);
  const cudaError_t e = a.dtype == OQ_DTYPE_BF16 ? mx_launch(read_kernel<__nv_bfloat16>, grid, NT, 0, 0, st, a)
                                                 : mx_launch(read_kernel<float>, grid, NT, 0, 0, st, a);
  return launched(e, "cache read-back");
}

}  // namespace oq
