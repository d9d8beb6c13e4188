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

// What a lane multiplies its eight channels x and their partners xp in the
// rotation by, gains included:  n sqrt(mean + eps) = x c + xp s.
template <bool INTER>
struct Coef {
  f32x2 c[4], s[4];
  bool on;        // these channels are rotated
  int from;       // halves: the lane that holds the partners
};

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

// cos and sin of the lane's channels in a table row; s as it multiplies the partner
template <bool INTER>
__device__ __forceinline__ void load_turn(float (&c)[8], float (&s)[8], const float* row, int half, int ch) {
  if constexpr (INTER) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row + ch)), b = __ldg(reinterpret_cast<const float4*>(row + ch) + 1);
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      c[j] = c[j + 1] = v[j];
      s[j] = -v[j + 1], s[j + 1] = v[j + 1];
    }
  } else {
    const bool second = ch >= half;
    const float4* p = reinterpret_cast<const float4*>(row + 2 * (second ? ch - half : ch));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 a = __ldg(p + i);
      c[2 * i] = a.x, s[2 * i] = second ? a.y : -a.y;
      c[2 * i + 1] = a.z, s[2 * i + 1] = second ? a.w : -a.w;
    }
  }
}

template <bool INTER>
__device__ __forceinline__ Coef<INTER> make_coef(const RopeArgs& p, const void* gain, int64_t pos, int ch, bool in) {
  Coef<INTER> k;
  float g[8];
  load_gain(g, gain, p.gain_bf16, ch, in);
  k.on = in && p.table != nullptr && ch < p.rot;
  k.from = (int)threadIdx.x & 31;
  if (!k.on) {
#pragma unroll
    for (int i = 0; i < 4; ++i) k.c[i] = pack2(g[2 * i], g[2 * i + 1]), k.s[i] = pack2(0.f, 0.f);
    return k;
  }
  const int half = p.rot >> 1;
  float c[8], s[8], o[8];
  const bool ok = pos >= 0 && pos < p.table_rows;   // a place outside the table makes the channels NaN
  load_turn<INTER>(c, s, p.table + (ok ? pos : 0) * p.rot, half, ch);
  if constexpr (INTER) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = g[j ^ 1];
  } else {
    const int d = ch >= half ? -half : half;
    load_gain(o, gain, p.gain_bf16, ch + d, true);
    k.from += d / 8;
  }
  const float nan = ok ? 1.f : __int_as_float(0x7FC00000);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    k.c[i] = pack2(g[2 * i] * c[2 * i] * nan, g[2 * i + 1] * c[2 * i + 1] * nan);
    k.s[i] = pack2(o[2 * i] * s[2 * i], o[2 * i + 1] * s[2 * i + 1]);
  }
  return k;
}

template <int LANES, typename F>
__device__ __forceinline__ F group_sum(F v) {
#pragma unroll
  for (int o = LANES / 2; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ uint32_t shfl_word(uint32_t v, int from) { return __shfl_sync(0xFFFFFFFFu, v, from); }
__device__ __forceinline__ void shfl_vec(Vec8<__nv_bfloat16>& v, int from) {
  v.w = make_uint4(shfl_word(v.w.x, from), shfl_word(v.w.y, from), shfl_word(v.w.z, from), shfl_word(v.w.w, from));
}
__device__ __forceinline__ void shfl_vec(Vec8<float>& v, int from) {
  float* f = &v.a.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __shfl_sync(0xFFFFFFFFu, f[i], from);
  f = &v.b.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __shfl_sync(0xFFFFFFFFu, f[i], from);
}

// the partners of this lane's channels, 0 where they are not rotated
template <bool INTER, typename T>
__device__ __forceinline__ void partners(f32x2 (&xp)[4], const f32x2 (&x)[4], Vec8<T> raw, const Coef<INTER>& k) {
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      unpack2(x[i], lo, hi);
      xp[i] = pack2(k.on ? hi : 0.f, k.on ? lo : 0.f);
    }
  } else {
    shfl_vec(raw, k.from);
    if (!k.on) raw.zero();
    raw.get(xp);
  }
}

__device__ __forceinline__ float square_sum(const f32x2 (&x)[4]) {
  f32x2 s = mul2(x[0], x[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(x[i], x[i], s);
  float lo, hi;
  unpack2(s, lo, hi);
  return lo + hi;
}

// Whether the sum of squares in fp32 is good to fp32's precision: it neither
// overflowed nor lost squares that eps does not hide (a NaN is not).
__device__ __forceinline__ bool plain_range(float ss, float eps) { return ss < 3e38f && (ss > 1e-30f || eps > 1e-24f); }

// A row's eight channels in fp64, from the inputs: norm, gains and rotation.
// Every lane of the warp takes part.
template <bool INTER, int LANES>
__device__ __forceinline__ void exact_row(double (&d)[8], const RopeArgs& p, const void* gain, int64_t pos, int ch, bool in) {
  float g[8];
  load_gain(g, gain, p.gain_bf16, ch, in);
  if (p.norm) {
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += d[j] * d[j];
    ss = group_sum<LANES>(ss);
    const double root = sqrt(ss / (double)p.D + (double)p.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = d[j] / root * (double)g[j];
  }
  const bool on = in && p.table != nullptr && ch < p.rot, ok = pos >= 0 && pos < p.table_rows;
  const int half = p.rot >> 1;
  float c[8], s[8];
  if (on) load_turn<INTER>(c, s, p.table + (ok ? pos : 0) * p.rot, half, ch);
  double o[8];
  const int from = ((int)threadIdx.x & 31) + (INTER || !on ? 0 : (ch >= half ? -half : half) / 8);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = INTER ? d[j ^ 1] : __shfl_sync(0xFFFFFFFFu, d[j], from);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (on) d[j] = ok ? d[j] * (double)c[j] + o[j] * (double)s[j] : nan("");
}

// How the rows of one tensor (queries or keys) go to CTAs.
struct RopeGrid {
  int per_token;  // rows of a token that a CTA does at once
  int tokens;     // tokens of a CTA
  int split;      // CTAs that share a token's rows
  int ctas;
};

// Rows of x[which] by CTA `cta` of grid g.  All lanes of a warp make the same
// number of turns, two at a time without a branch between them (their latencies
// overlap; one at a time took 306 us for 237 at 32760 tokens of 40 + 40 heads).  The
// first rows' loads leave before the token's place and its table row are known,
// and PF rows stay in flight.  Rows out of fp32's range are
// marked and done in fp64 behind each 32 turns (inside the loop they would cost
// all rows registers).  place: a token's row of the table, and whether it has one: the
// rows of a token that has none stay as they are.
template <typename T, typename OUT, bool INTER, int LANES, typename POS>
__device__ __forceinline__ void rope_rows(const RopeArgs& p, const RopeGrid& g, int which, int cta, POS&& place) {
  constexpr int PF = sizeof(T) == 2 ? 4 : 2, PAIR = 2, MARKS = 32;
  const int grp = (int)threadIdx.x / LANES, ch = ((int)threadIdx.x & (LANES - 1)) * 8;
  const int64_t t = (int64_t)(cta / g.split) * g.tokens + grp / g.per_token;
  const int sub = cta % g.split * g.per_token + grp % g.per_token, step = g.split * g.per_token;
  const bool in = t < p.T && ch < p.D;
  const int rows = p.heads[which], turns = (rows + step - 1) / step, hop = step * p.D;
  int mine = in && sub < rows ? (rows - sub + step - 1) / step : 0;   // this lane's rows
  const T* x0 = static_cast<const T*>(p.x[which]) + t * p.in_stride[which] + sub * p.D + ch;
  OUT* y0 = static_cast<OUT*>(p.out[which]) + t * p.out_stride[which] + sub * p.D + ch;
  Vec8<T> raw[PF];
  const T* xn = x0;   // the next row to load
  int loaded = 0;
  auto fetch = [&](Vec8<T>& v) {
    if (loaded < mine) v.load(xn);
    else v.zero();
    ++loaded;
    xn += hop;
  };
#pragma unroll
  for (int u = 0; u < PF; ++u) fetch(raw[u]);
  bool held = true;
  const int64_t pos = place(t, held);
  if (!held) mine = 0;
  const Coef<INTER> k = make_coef<INTER>(p, p.gain[which], pos, ch, in);
  const float inv_d = 1.0f / (float)p.D;
  OUT* y = y0;
#pragma unroll 1
  for (int i0 = 0; i0 < turns; i0 += MARKS) {
    uint32_t marks = 0u;
#pragma unroll 1
    for (int i1 = 0; i1 < MARKS && i0 + i1 < turns; i1 += PF) {
#pragma unroll
      for (int u = 0; u < PF; ++u) {
        const int i = i0 + i1 + u;
        if (u % PAIR == 0 && u > 0 && i >= turns) break;   // the same in all lanes
        const Vec8<T> now = raw[u];
        fetch(raw[u]);
        f32x2 x[4], xp[4];
        now.get(x);
        partners<INTER, T>(xp, x, now, k);
        float inv = 1.f, n[8];
        bool good = true;
        if (p.norm) {
          const float ss = group_sum<LANES>(square_sum(x));
          good = plain_range(ss, p.eps) || i >= turns;
          inv = rsqrtf(fmaf(ss, inv_d, p.eps));
        }
        if (!good) marks |= 1u << (i1 + u);
        const f32x2 i2 = pack2(inv, inv);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = mul2(fma2(xp[j], k.s[j], mul2(x[j], k.c[j])), i2);
        unpack8(x, n);
        if (i < mine && good) store8(y, n);
        y += hop;
      }
    }
    const uint32_t all = __reduce_or_sync(0xFFFFFFFFu, marks);
#pragma unroll 1
    for (int j = 0; all >> j != 0u; ++j) {
      if (!(all >> j & 1u)) {
        if (j == MARKS - 1) break;
        continue;
      }
      const int i = i0 + j;
      const bool have = i < mine;
      Vec8<T> now;
      now.zero();
      if (have) now.load(x0 + (int64_t)i * hop);
      float n[8];
      double d[8];
      now.get(n);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = (double)n[e];
      exact_row<INTER, LANES>(d, p, p.gain[which], pos, ch, in);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] = (float)d[e];
      if (have && (marks >> j & 1u)) store8(y0 + (int64_t)i * hop, n);
      if (j == MARKS - 1) break;
    }
  }
}

struct RopeParams {
  RopeArgs a;
  RopeGrid g[2];
  bool both;      // a CTA does its tokens' queries, then their keys (the grids are alike); else CTAs of each
};

template <typename T, bool INTER, int LANES>
__global__ void __launch_bounds__(NT, 3) rope_kernel(const __grid_constant__ RopeParams p) {
  dependency_wait();
  int which = !p.both && (int)blockIdx.x >= p.g[0].ctas;
  const int last = p.both ? 1 : which, cta = (int)blockIdx.x - (which ? p.g[0].ctas : 0);
#pragma unroll 1
  for (; which <= last; ++which)
    rope_rows<T, T, INTER, LANES>(p.a, p.g[which], which, cta, [&](int64_t t, bool&) {
      return t >= p.a.T ? (int64_t)0 : p.a.positions ? (int64_t)p.a.positions[t] : t;
    });
}

int row_lanes(int D) {
  int l = 4;
  while (l * 8 < D) l *= 2;
  return l;
}

// Lane groups of a token: as few as still make two CTAs for each SM (what a token's
// table row and gains cost is spent once for all its rows); few tokens are shared
// by as many CTAs.  Measured: 1001 tokens of 24 + 8 fp32 rows of 96 channels, two
// CTAs an SM 9.7 us, three 14.2, four 17.1; 32760 tokens of 80 bf16 rows of 128, one
// group a token 237 us, two 237, four 248, sixteen 477.
// False: more CTAs than a grid takes.
bool rope_grid(int64_t T, int rows, int D, int sms, int threads, RopeGrid* out) {
  RopeGrid g;
  const int groups = threads / row_lanes(D);
  const int64_t want = 2 * (int64_t)sms * groups / T;
  g.per_token = 1;
  while (g.per_token < groups && g.per_token < rows && g.per_token < want) g.per_token *= 2;
  g.tokens = groups / g.per_token;
  const int64_t ctas = (T + g.tokens - 1) / g.tokens;
  const int turns = (rows + g.per_token - 1) / g.per_token;
  g.split = (int)std::max<int64_t>(1, std::min<int64_t>(turns, 2 * (int64_t)sms / ctas));
  if (ctas * g.split > 0x3FFFFFFF) return false;
  g.ctas = rows > 0 ? (int)(ctas * g.split) : 0;
  *out = g;
  return true;
}

oq_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return OQ_OK;
  set_error(std::string(what) + " launch: " + cudaGetErrorString(e));
  return OQ_ERR_CUDA;
}

// ------------------------------------------------------------------ append
// A CTA of the cache's part takes up to AWIN tokens whose places share an aligned
// window, so that no word of V's transposed rows (eight tokens) is written by two
// CTAs, and walks over groups of 128 channels.  Keys go the way
// of the queries and are then quantised; values are quantised as they are and
// transposed through shared memory.
//
// A key's codes are those of the value in exact arithmetic: its fp32 value is
// off by less than DELTA of |a| + |b| (the pair it was turned from), and where
// that could change a code or the block's scale, the row is formed again in fp64
// and rounded once.  (The sum of squares takes 8 + 4 roundings, halved by the
// root; the mean, halved too, the reciprocal root's two ulps, two products and the
// rotation's three operations add at most 10: 16 * 2^-24, taken as 32 * 2^-24.)
constexpr float DELTA = 32.f / 16777216.f;

struct AppendParams {
  AppendArgs a;
  RopeGrid g;
  int kv_heads, parts;    // CTAs that share a window's groups of 128 channels
};
constexpr int AWIN = 16, ANT = AWIN * 16;   // tokens of a window, 16 lanes each

__device__ __forceinline__ float round_odd(double w) {
  float f = __double2float_rz(w);
  if ((double)f != w) f = __uint_as_float(__float_as_uint(f) | 1u);
  return f;
}

// the low four nibbles, one a byte
__device__ __forceinline__ uint32_t spread_nibbles(uint32_t v) {
  v &= 0xFFFFu;
  v = (v | v << 8) & 0x00FF00FFu;
  return (v | v << 4) & 0x0F0F0F0Fu;
}

// largest of four neighbouring lanes
__device__ __forceinline__ float max4(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 2));
}

// The same in fp64: codes, and the block's scale code above them.
template <typename T, bool INTER, int LANES>
__device__ __forceinline__ uint64_t exact_codes(Vec8<T> raw, const RopeArgs* p, int64_t pos, int ch, bool in) {
  float w[8];
  double d[8], top = 0.0;
  raw.get(w);
#pragma unroll
  for (int j = 0; j < 8; ++j) d[j] = (double)w[j];
  exact_row<INTER, LANES>(d, *p, p->gain[1], pos, ch, in);
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bad |= !(fabs(d[j]) <= 3.4028234663852886e38);
    top = fmax(top, fabs(d[j]));
  }
  const float f = max4(bad ? __int_as_float(0x7F800000) : __double2float_rz(top));
  const uint32_t scale = mx_scale_code<4>(__float_as_uint(f));
  const double s = (double)mx_inverse_scale(scale);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = round_odd(d[j] * s);
  uint32_t out[1];
  mx_element_codes<4>(w, scale, out);
  return (uint64_t)scale << 32 | out[0];
}

// Eight channels of a key (norm, rotation) -> codes and the block's scale code.
template <typename T, bool INTER, int LANES>
__device__ __forceinline__ uint32_t key_codes(const Vec8<T>& raw, const RopeArgs& p, const Coef<INTER>& k, int64_t pos, int ch,
                                              bool in, float inv_d, uint32_t& scale) {
  f32x2 x[4], xp[4];
  raw.get(x);
  partners<INTER, T>(xp, x, raw, k);
  bool doubt = false;
  float inv = 1.f;
  if (p.norm) {
    const float ss = group_sum<LANES>(square_sum(x));
    doubt = !plain_range(ss, p.eps);
    inv = rsqrtf(fmaf(ss, inv_d, p.eps));
  }
  const f32x2 i2 = pack2(inv, inv);
  float n[8], a[8], b[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = mul2(mul2(x[i], k.c[i]), i2);
    xp[i] = mul2(mul2(xp[i], k.s[i]), i2);
  }
  unpack8(x, a);
  unpack8(xp, b);
#pragma unroll
  for (int j = 0; j < 8; ++j) n[j] = a[j] + b[j];
  const uint32_t block = mx_block_max(n);
  scale = mx_scale_code<4>(block);
  const float inv_s = mx_inverse_scale(scale);
  float w[8];
  uint32_t out[1];
  if (!p.norm && !p.table) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = n[j] * inv_s;
    mx_element_codes<4>(w, scale, out);
  } else {
    // what |a| + |b| lets the fp32 value be off: where the codes of both ends are
    // one, it is the value's (ends around zero differ in its sign: looked at too)
    const float top = __uint_as_float(block);
    const f32x2 is2 = pack2(inv_s, inv_s), off = pack2(DELTA * inv_s, DELTA * inv_s);
    const f32x2 noff = pack2(-DELTA * inv_s, -DELTA * inv_s);
    float m[8], lo[8], hi[8];
    f32x2 l2[4], h2[4];
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = fabsf(a[j]) + fabsf(b[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 wi = mul2(pack2(n[2 * i], n[2 * i + 1]), is2), mi = pack2(m[2 * i], m[2 * i + 1]);
      l2[i] = fma2(mi, noff, wi);
      h2[i] = fma2(mi, off, wi);
    }
    unpack8(l2, lo);
    unpack8(h2, hi);
    mx_element_codes<4>(lo, scale, out);
    float most = fmaxf(fmaxf(m[0], m[1]), m[2]);
    most = fmaxf(fmaxf(most, m[3]), m[4]);
    most = max4(fmaxf(fmaxf(fmaxf(most, m[5]), m[6]), m[7])) * DELTA;
    doubt |= top > 0.f && top < 1e-30f;   // products below fp32's normal numbers are off by more
    doubt |= scale != 255u && ((__float_as_uint(top + most) >> 23) != (__float_as_uint(fmaxf(top - most, 0.f)) >> 23) ||
                               out[0] != cvt8_e2m1(hi));
    if (__any_sync(0xFFFFFFFFu, doubt)) {
      const uint64_t r = exact_codes<T, INTER, LANES>(raw, &p, pos, ch, in);
      out[0] = (uint32_t)r;
      scale = (uint32_t)(r >> 32);
    }
  }
  return out[0];
}

template <typename T, bool INTER, int LANES>
__global__ void __launch_bounds__(ANT, 3) append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int found[2];
  constexpr int TP = AWIN / 2 + 4;                     // (rows' distance: no bank twice)
  __shared__ __align__(16) uint8_t tile[2][128 * TP];  // V codes, two tokens a byte: channel 8 s + j in row 16 j + s
  const RopeArgs& r = p.a.rope;
  const KvView& kv = p.a.kv;
  dependency_wait();
  if ((int)blockIdx.x < p.g.ctas) {
    rope_rows<T, __nv_bfloat16, INTER, LANES>(r, p.g, 0, (int)blockIdx.x, [&](int64_t t, bool& held) {
      held = t >= kv.cu[0] && t < kv.cu[kv.B];   // a token of no sequence has no place
      if (!r.table) return (int64_t)0;
      if (r.positions) return t < r.T ? (int64_t)r.positions[t] : (int64_t)0;
      // the token's sequence: how many of them end at or before it
      int ends = 0;
      for (int b = (int)threadIdx.x & (LANES - 1); b < kv.B; b += LANES) ends += kv.cu[b + 1] <= t;
      const int b = min(group_sum<LANES>(ends), kv.B - 1);
      return (int64_t)kv.lens[b] - kv.cu[b + 1] + t;
    });
    return;
  }
  const int unit = ((int)blockIdx.x - p.g.ctas) / p.parts, part = ((int)blockIdx.x - p.g.ctas) % p.parts;
  int b, first, count, place;
  if (!kv_window<AWIN>(kv, r.T, unit, found, b, first, count, place)) return;
  const int64_t page = kv.table[(int64_t)b * kv.width + (place >> 7)];
  if (page < 0 || page >= kv.pages) return;
  constexpr int D = LANES * 8;
  const int sub = (int)threadIdx.x & 15, ch = (sub & (LANES - 1)) * 8;   // 16 lanes hold a group's channels of a token
  const int w0 = place & 127 & ~(AWIN - 1);                              // the window's first row in its page
  const int row = (int)threadIdx.x >> 4, at = w0 + row, i = row - (place & (AWIN - 1));
  const bool token = i >= 0 && i < count;
  const int64_t t = first + i;
  int hg = (int)((int64_t)kv.groups * part / p.parts);
  const int hg_end = (int)((int64_t)kv.groups * (part + 1) / p.parts);
  uint8_t* base = kv.cache + (page * kv.groups + hg) * KV_GROUP_BYTES;
  int head = hg * (128 / D) + sub / LANES;
  const T* kp = static_cast<const T*>(r.x[1]) + t * r.in_stride[1] + head * D + ch;
  const T* vp = static_cast<const T*>(p.a.v) + t * p.a.v_stride + head * D + ch;
  Vec8<T> kn, vn;   // the next group's
  auto fetch = [&]() {
    if (token && head < p.kv_heads) kn.load(kp), vn.load(vp);
    else kn.zero(), vn.zero();
  };
  fetch();
  const int64_t pos = !token ? 0 : r.positions ? (int64_t)r.positions[t] : (int64_t)(place + i);
  const Coef<INTER> coef = make_coef<INTER>(r, r.gain[1], pos, ch, token);
#pragma unroll 1
  for (int buf = 0; hg < hg_end; ++hg, buf ^= 1, base += KV_GROUP_BYTES) {
    const Vec8<T> k = kn, v = vn;
    const bool has = head < p.kv_heads;
    head += 128 / D;
    kp += 128;
    vp += 128;
    if (hg + 1 < hg_end) fetch();
    uint32_t ks, vs, kc, vc[1];
    kc = key_codes<T, INTER, LANES>(k, r, coef, pos, ch, token, 1.0f / D, ks);
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
      *reinterpret_cast<uint32_t*>(base + at * 64 + sub * 4) = kc;
      if (sub == 0) {
        *reinterpret_cast<uint32_t*>(base + KV_KS_ROW * 64 + mx_tile_word(at) * 4) = kw;
        *reinterpret_cast<uint32_t*>(base + KV_VS_ROW * 64 + at * 4) = vw;
      }
    }
    // two tokens a byte: the lanes of a pair of rows take four channels each
    const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, vc[0], 16);
    const bool odd = (row & 1) != 0;
    const uint32_t even_row = spread_nibbles(odd ? other >> 16 : vc[0]), odd_row = spread_nibbles(odd ? vc[0] >> 16 : other);
    const uint32_t pairs = even_row | odd_row << 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) tile[buf][((j + (odd ? 4 : 0)) * 16 + sub) * TP + (row >> 1)] = (uint8_t)(pairs >> (8 * j));
    __syncthreads();   // (the other tile's readers are past the barrier before)
    // AWIN / 8 threads write a channel's tokens; tokens that are not the call's keep their codes
    {
      constexpr int PER = AWIN / 8;
      const int c = (int)threadIdx.x / PER, q = (int)threadIdx.x % PER;
      uint32_t out = reinterpret_cast<const uint32_t*>(tile[buf] + ((c & 7) * 16 + (c >> 3)) * TP)[q];
      uint32_t* dst = reinterpret_cast<uint32_t*>(base + (KV_V_ROW + c) * 64 + w0 / 2) + q;
      if (count != AWIN) {
        const int lo = min(max((place & (AWIN - 1)) - 8 * q, 0), 8), hi = min(max((place & (AWIN - 1)) + count - 8 * q, 0), 8);
        const uint32_t below_hi = hi == 8 ? 0xFFFFFFFFu : (1u << (4 * hi)) - 1u;
        const uint32_t below_lo = lo == 8 ? 0xFFFFFFFFu : (1u << (4 * lo)) - 1u;
        const uint32_t mask = below_hi & ~below_lo;   // nibbles [lo, hi) are new
        if (mask != 0xFFFFFFFFu && mask != 0u) out = (out & mask) | (*dst & ~mask);
        if (mask != 0u) *dst = out;
      } else {
        *dst = out;
      }
    }
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
  if (!kv_window<32>(kv, p.T, unit, found, b, first, count, place)) return;
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

template <typename T, bool INTER>
cudaError_t rope_launch_lanes(const RopeParams& p, dim3 grid, cudaStream_t st) {
  switch (row_lanes(p.a.D)) {
    case 4: return mx_launch(rope_kernel<T, INTER, 4>, grid, NT, 0, 0, st, p);
    case 8: return mx_launch(rope_kernel<T, INTER, 8>, grid, NT, 0, 0, st, p);
    case 16: return mx_launch(rope_kernel<T, INTER, 16>, grid, NT, 0, 0, st, p);
    default: return mx_launch(rope_kernel<T, INTER, 32>, grid, NT, 0, 0, st, p);
  }
}
template <typename T, bool INTER>
cudaError_t append_launch_lanes(const AppendParams& p, dim3 grid, cudaStream_t st) {
  return p.a.rope.D == 64 ? mx_launch(append_kernel<T, INTER, 8>, grid, ANT, 0, 0, st, p)
                          : mx_launch(append_kernel<T, INTER, 16>, grid, ANT, 0, 0, st, p);
}

// units of kv_window<W> that B sequences with T tokens may have
int64_t window_units(int64_t T, int B, int W) { return std::min<int64_t>(T, T / W + 2 * (int64_t)B); }

}  // namespace

oq_status rope_launch(const RopeArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  RopeParams p;
  p.a = a;
  const int sms = mx_sm_count(&dev), most = std::max(a.heads[0], a.heads[1]);
  if (!rope_grid(a.T, most, a.D, sms, NT, &p.g[0])) return OQ_ERR_UNSUPPORTED;
  // Many tokens: a token's queries and keys, which lie side by side in a
  // projection's output, are read by one CTA.  Few: a CTA has one or the other.
  p.both = a.heads[0] > 0 && a.heads[1] > 0 && p.g[0].ctas >= 8 * sms;
  p.g[1] = p.g[0];
  if (!p.both)
    for (int i = 0; i < 2; ++i)
      if (!rope_grid(a.T, a.heads[i], a.D, sms, NT, &p.g[i])) return OQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(p.both ? p.g[0].ctas : p.g[0].ctas + p.g[1].ctas));
  cudaError_t e;
  if (a.dtype == OQ_DTYPE_BF16)
    e = a.interleaved ? rope_launch_lanes<__nv_bfloat16, true>(p, grid, st) : rope_launch_lanes<__nv_bfloat16, false>(p, grid, st);
  else
    e = a.interleaved ? rope_launch_lanes<float, true>(p, grid, st) : rope_launch_lanes<float, false>(p, grid, st);
  return launched(e, "norm and rotation");
}

oq_status kv4_append_launch(const AppendArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int dev = 0;
  AppendParams p;
  p.a = a;
  p.kv_heads = a.rope.heads[1];
  const int D = a.rope.D;
  const int64_t units = window_units(a.rope.T, a.kv.B, AWIN);
  const int sms = mx_sm_count(&dev);
  // a window's groups: in one CTA (what a token's table row costs is spent once)
  // where there are windows for four CTAs an SM, else shared
  p.parts = (int)std::max<int64_t>(1, std::min<int64_t>(a.kv.groups, 4 * (int64_t)sms / units));
  if (!rope_grid(a.rope.T, a.rope.heads[0], D, sms, ANT, &p.g) || p.g.ctas + units * p.parts > 0x7FFFFFFF)
    return OQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)(p.g.ctas + units * p.parts));
  cudaError_t e;
  if (a.rope.dtype == OQ_DTYPE_BF16)
    e = a.rope.interleaved ? append_launch_lanes<__nv_bfloat16, true>(p, grid, st)
                           : append_launch_lanes<__nv_bfloat16, false>(p, grid, st);
  else
    e = a.rope.interleaved ? append_launch_lanes<float, true>(p, grid, st) : append_launch_lanes<float, false>(p, grid, st);
  return launched(e, "cache append");
}

oq_status kv4_read_launch(const ReadArgs& a, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t ctas = window_units(a.T, a.kv.B, 32) * a.kv.groups;
  if (ctas > 0x7FFFFFFF) return OQ_ERR_UNSUPPORTED;
  const dim3 grid((unsigned)ctas);
  const cudaError_t e = a.dtype == OQ_DTYPE_BF16 ? mx_launch(read_kernel<__nv_bfloat16>, grid, NT, 0, 0, st, a)
                                                 : mx_launch(read_kernel<float>, grid, NT, 0, 0, st, a);
  return launched(e, "cache read-back");
}

}  // namespace oq
