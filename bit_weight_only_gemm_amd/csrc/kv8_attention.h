// kv8_attention.h -- attention of 16-bit queries over the paged 8-bit cache:
//
//   O[t, h] = sum_l softmax_l(scale q[t, h] . k_l) v_l  over the visible l.
//
// Mathematics.  One pass over the keys with the running maximum m and sum of
// the softmax (fp32, base 2).  A code c enters the matrix instructions as the
// fp16 value c - 128, which is exact; the queries enter as fp16, a bf16 row
// after an exact power of two that brings its largest magnitude to 2^14 (what
// that loses lies 2^-39 below the row's largest).  The scales of a page are
// applied in fp32: the keys' to the scores, the values' to the sum over 64
// tokens.  Probabilities are rounded to fp16 (to nearest) for the second
// product, their sum is taken before that rounding.
#pragma once
#include <algorithm>
#include <type_traits>

#include "kv8.h"
#include "launch.h"

namespace w4a16 {

// What the scored form puts on the scores before the softmax, and which keys a
// query sees:
//   s <- cap tanh(s / cap) (cap > 0),  s <- s - slope[head] |position - l|,
//   first[token] <= l < its limit, and below prefix[sequence] both ways; but
//   never from end[token] on.
// Scores are in base 2 here (cap is times log2 e).  They are brought to their
// final value before the maximum is taken, but for the cap itself (or 1), by which
// everything after it multiplies.
struct Scoring {
  float cap, per_cap;     // and 1 / cap
  const float* slopes;    // [H] or null
  const int32_t* first;   // [tokens] or null
  const int32_t* prefix;  // [B] or null
  const int32_t* end;     // [tokens] or null
};

// What a kernel is built to do to scores.
enum { kPlain = 0, kMasks = 1, kCap = 2, kBias = 4 };

// A call is split into this many workgroups or more, so one that is split has
// fewer row tiles, each of which has a counter.
constexpr int64_t kWanted = 512, kCounters = kWanted;

// waves: of the prompt kernel's workgroups (32 rows each); 0: the decode kernel.
struct Plan {
  int waves, rows, row_tiles, splits, units;
};

// Launches a call's kernels for one dtype, head size and mode.
typedef hipError_t AttentionLaunch(const Kv8& c, const Plan& p, const void* q, int64_t q_stride,
                                   float scale, int causal, void* out, int64_t out_stride,
                                   float* lse, int64_t max_new, void* ws, const Scoring& sc,
                                   hipStream_t st);
// The scored modes' launchers, each compiled in its own file.
AttentionLaunch* scored_launch(int mode, int32_t D, int32_t dtype);
AttentionLaunch* capped_launch(int mode, int32_t D, int32_t dtype);

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kUnit = 64;  // tokens a wave takes at a time

// The running maximum m of a row (of its scores s in base 2) moves only when a
// score passes it by kLag, and the reference u that the values' page scales are
// taken relative to only when one passes twice u.  A probability enters the
// second product as w = 2^kLift exp2(s - m) (vs / u), at most 2^15 and so in
// fp16's range, and exact to 2^-11 down to 2^-25 of the largest (2^-36 of it
// absolutely below that); the sum takes w (u / vs).  vs / u is held to kLeast and
// up, where every w is 0 in fp16, so that a page of zeros divides nothing by 0.
// u is at least kRef, the least that has a reciprocal; pages of subnormal scales
// below it lose part of the lift instead.
// Sums of both products carry the factor 2^kLift, which their quotient drops.
//
// m is the rounded product of a sum and its factor, and one fma forms a score's
// distance from it: exact but for m's own rounding, 2^-24 |m|, which all of a
// row's probabilities share.  From |m| = 2^24 on that is a factor fp16 cannot
// hold, and kLift is lost beside m; so where m of a row passes kFar, scores are
// rounded as m was and m is subtracted first.  (kFar is low so that the factor,
// 2^-14 there, does not tell keys seen before the change from those after.)  A
// row's m before its first key is kNone, the least of fp32.
constexpr float kFar = 0x1p10f, kNone = -0x1.fffffep127f;
constexpr float kLift = 11.0f, kLag = 3.0f, kLeast = 0x1p-45f, kRef = 0x1p-126f;

// Results that are still to be joined are o u and l, both times 2^-kShrink: an o
// of up to 2^38 (codes, weights and tokens) would leave fp32 at values of 1e28,
// and l, 2^8 and more where it counts, keeps the products of bf16's least values
// above fp32's.
constexpr float kShrink = 20.0f, kPart = 0x1p-20f;

// log(sum exp) of a row, natural, from its maximum and its sum times 2^-shrunk.
__device__ __forceinline__ float lse_of(float m, float l, float shrunk) {
  return l == 0.0f ? -INFINITY : (m + (__log2f(l) + (shrunk - kLift))) * kLn2;
}

typedef float float16_t __attribute__((ext_vector_type(16)));

// 8 codes of two dwords as an fp16 operand: 0x6400 | c is 1024 + c.
__device__ __forceinline__ half8_t codes_f16(uint32_t a, uint32_t b) {
  const half2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = __builtin_amdgcn_perm(0x64646464u, i < 2 ? a : b,
                                               (i & 1) ? 0x04030402u : 0x04010400u);
    r[i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(half2_t, two) - off);
  }
  return __builtin_bit_cast(half8_t, r);
}

// A row of queries as fp16 operands: N pieces of 8 channels in each of the
// lanes l, l ^ FIRST, .. that hold the row (FIRST = 16: four lanes, 32: two).
// fp16 rows as they are; bf16 rows times a power of two that brings the row's
// largest magnitude to [2^14, 2^15), held to fp32's normal range.  What the
// scores have to be multiplied by.
template <int DT, int N, int FIRST>
__device__ __forceinline__ float queries_f16(const u32x4_t (&w)[N], half8_t (&out)[N]) {
  if constexpr (DT == DT_F16) {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = __builtin_bit_cast(half8_t, w[i]);
    return 1.0f;
  } else {
    uint32_t mag = 0;
    float f[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      widen8<DT>(w[i], f[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(f[i][j]));
    }
#pragma unroll
    for (int o = FIRST; o < 64; o <<= 1) mag = max(mag, (uint32_t)__shfl_xor((int)mag, o, 64));
    const int e2 = clamp_int((int)(mag >> 23) - 127, -100, 126);
    const float up = __builtin_bit_cast(float, (uint32_t)(127 + 14 - e2) << 23);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) out[i][j] = (_Float16)(f[i][j] * up);
    return __builtin_bit_cast(float, (uint32_t)(127 - 14 + e2) << 23);
  }
}

// Query rows of a (sequence, kv head): row i is token i / G, head i % G.  A
// row tile is `rows` of them; it sees keys up to the largest limit of its rows.
// (prefix: keys below it are seen by every token that has a position)
__device__ __forceinline__ int row_limit(const Kv8Seq& s, int causal, int j, int prefix = 0) {
  const int p = s.first + j;
  return causal ? clamp_int(p < 0 ? 0 : max(p + 1, prefix), 0, s.len) : s.len;
}
__device__ __forceinline__ int tile_limit(const Kv8Seq& s, int causal, int rt, int rows, int G,
                                          int prefix = 0) {
  return row_limit(s, causal, min((rt * rows + rows - 1) / G, s.n - 1), prefix);
}

// Kernels are built for what they do to scores: kMasks nothing, else kCap and
// kBias.  (As branches at run time these cost the prompt kernel more registers than
// it has: 30 ms instead of 1.6.)
//
// tanh(x) = 1 - 2 / (1 + exp(2 x)), an exponential and a reciprocal of 1 ulp and
// three roundings, is 2^-20 off at most, which the cap multiplies: 5e-5 of a
// probability under a cap of 50, where its rounding to fp16 is 5e-4.  x P(x^2), P a
// fit of degree 4 to tanh(x) / x over |x| < 3 / 4, is 9.1e-7 of itself off (2^-20) and
// costs 28 cycles a wave and score instead of 44: a unit whose scores are all that
// small under their cap takes it (MI355X, chunks of 2048 over 8192, 40 / 8 heads,
// under a cap of 50: 1383 us, 1559 with the exponential alone; without a cap 1112).
// Under caps beyond kWideCap every small score does, so that the error stays a part
// of the score.  (Keys that a row does not see count as 0 in this choice: what an
// unused row of a page holds does not show in a result.)
constexpr float kWideCap = 512.0f, kBend = 0.75f;

__device__ __forceinline__ float tanh_near(float x) {
  const float y = x * x;
  float p = __builtin_fmaf(y, 0.012918088f, -0.050102882f);
  p = __builtin_fmaf(y, p, 0.132636398f);
  p = __builtin_fmaf(y, p, -0.333293557f);
  return x * __builtin_fmaf(y, p, 0.99999994f);
}
__device__ __forceinline__ float tanh_any(float twice_x_log2e) {
  const float r = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(twice_x_log2e));
  return __builtin_fmaf(-2.0f, r, 1.0f);
}

// The scores of N groups of 16 tokens from products that are to be multiplied by
// f[a]; back[a]: the query's position less the group's first token.  Afterwards f[a]
// is what they are still to be multiplied by: the cap, or 1 where a bias came on.
template <int MODE, int N>
__device__ __forceinline__ void put_on(float (&s)[N][16], float (&f)[N], const Scoring& sc,
                                       float slope, const float (&back)[N]) {
  constexpr bool CAPPED = (MODE & kCap) != 0, BIAS = (MODE & kBias) != 0;
  if constexpr (CAPPED) {
    float to_x[N];
#pragma unroll
    for (int a = 0; a < N; ++a) to_x[a] = f[a] * sc.per_cap;
    float most = 0.0f;
#pragma unroll
    for (int a = 0; a < N; ++a) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; i += 2) t = fmaxf(fmaxf(t, fabsf(s[a][i])), fabsf(s[a][i + 1]));
      most = fmaxf(most, t * to_x[a]);
    }
    if (__all(most < kBend)) {
#pragma unroll
      for (int a = 0; a < N; ++a)
#pragma unroll
        for (int i = 0; i < 16; ++i) s[a][i] = tanh_near(s[a][i] * to_x[a]);
    } else if (sc.cap <= kWideCap) {
#pragma unroll
      for (int a = 0; a < N; ++a) {
        const float z = to_x[a] * (2.0f * kLog2e);
#pragma unroll
        for (int i = 0; i < 16; ++i) s[a][i] = tanh_any(s[a][i] * z);
      }
    } else {
#pragma unroll
      for (int a = 0; a < N; ++a)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float x = s[a][i] * to_x[a];
          s[a][i] = fabsf(x) < kBend ? tanh_near(x) : tanh_any(x * (2.0f * kLog2e));
        }
    }
#pragma unroll
    for (int a = 0; a < N; ++a) f[a] = sc.cap;
  }
  if constexpr (BIAS) {
#pragma unroll
    for (int a = 0; a < N; ++a) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        s[a][i] = __builtin_fmaf(s[a][i], f[a], -(slope * fabsf(back[a] - (float)i)));
      f[a] = 1.0f;
    }
  }
}

// Units of a split: this sequence's in equal shares, none below the planned.
__device__ __forceinline__ int split_units(int nu, int splits, int units) {
  return max(units, (nu + splits - 1) / splits);
}

// Partial results of a split: O [row][split][D], then (m, l) [row][split],
// row = token * H + head; and one counter for each (sequence, kv head, row
// tile) of the decode kernel, 0 between calls.
struct Parts {
  float* o;
  float* ml;
  uint32_t* count;
};

// Two floats past the caches of one die, for a workgroup on another.
__device__ __forceinline__ void send2(float* to, float a, float b) {
  const uint64_t v = (uint64_t)__builtin_bit_cast(uint32_t, a) |
                     (uint64_t)__builtin_bit_cast(uint32_t, b) << 32;
  __hip_atomic_store((uint64_t*)to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 fetch2(const float* from) {
  const uint64_t v =
      __hip_atomic_load((const uint64_t*)from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__builtin_bit_cast(float, (uint32_t)v),
                     __builtin_bit_cast(float, (uint32_t)(v >> 32)));
}

// The larger of the values that lanes l and l ^ 32 (HALF), or l and l ^ 16
// hold.  (The swap's results are copied out of their vector before they are
// reinterpreted: a reinterpreted vector element reads element 0.)
template <bool HALF>
__device__ __forceinline__ float swapped_max(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x);
  const auto r = HALF ? __builtin_amdgcn_permlane32_swap(b, b, false, false)
                      : __builtin_amdgcn_permlane16_swap(b, b, false, false);
  const uint32_t u = r[0], v = r[1];
  return fmaxf(__builtin_bit_cast(float, u), __builtin_bit_cast(float, v));
}
__device__ __forceinline__ float both_halves_max(float x) { return swapped_max<true>(x); }
// The largest of the values that the lanes l, l ^ 16, l ^ 32 and l ^ 48 hold.
__device__ __forceinline__ float four_rows_max(float x) {
  return swapped_max<true>(swapped_max<false>(x));
}

// One workgroup of 4 waves per (sequence, kv head, row tile, split of the
// keys); its waves take units of 64 tokens in turn and are joined in LDS.
// Scores come out as S^T (16 tokens x 16 rows): lane l holds row l & 15 and
// tokens 16 g + 4 a + i (g = l >> 4) of the unit in register i of product a,
// which is the operand layout of the second product: neither keys, values
// nor probabilities pass through LDS.
//
// The cache's bytes bound it where there are many: 64 ragged sequences of up to
// 8192 tokens, 40 / 8 heads of 128, 139 us, 5.0 TB/s of codes (MI355X; a plain
// read gets 5.7); 3 of up to 131001, 113 us.  Few tokens are a chain of waits
// (length, table, keys, values, join): one sequence of 777, 32 heads, 10.3 us.
// With 16 rows to a wave and not more, three waves share a SIMD and cover each
// other's waits: 32 or 48 rows a wave read the codes less often, and took 27 us
// against 21 for 24 sequences of 4001, 40 rows of 64 channels a kv head.
template <int DT, int D, int MODE>
__global__ void __launch_bounds__(256)
kv8_decode_kernel(Kv8 c, const uint16_t* __restrict__ q, int64_t q_stride, float scale, int causal,
                  uint16_t* __restrict__ out, int64_t out_stride, float* __restrict__ lse,
                  Parts parts, int row_tiles, int splits, int units, Scoring sc) {
  constexpr int DC = D / 64, DN = D / 16;
  constexpr bool SCORED = MODE != kPlain;
  __shared__ float joined[4][16][D + 4];
  __shared__ float stat[4][2][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;
  // workgroups go to the 8 XCDs in turn: the row tiles of one (split, kv head,
  // sequence) follow one another on one of them and share its cache
  const int at_xcd = (int)(blockIdx.x >> 3);
  int id = at_xcd / row_tiles * 8 + (int)(blockIdx.x & 7);
  const int rt = at_xcd % row_tiles;
  const int split = id % splits;
  id /= splits;
  const int hk = id % c.Hkv, b = id / c.Hkv;
  if (b >= c.B) return;
  const int G = c.H / c.Hkv;
  const Kv8Seq seq = kv8_seq(c, b);
  if (rt * 16 >= seq.n * G) return;
  const int ridx = rt * 16 + col;
  const bool rv = ridx < seq.n * G;
  const int tok = seq.tok + (rv ? ridx / G : 0), head = hk * G + (rv ? ridx % G : 0);
  const int prefix = SCORED && sc.prefix ? sc.prefix[b] : 0;
  int lim = rv ? row_limit(seq, causal, ridx / G, prefix) : 0;
  // rows with ends: the largest limit, the least, and where tokens begin that hold
  // nothing which some row sees
  int lim_most = 0, lim_least = 0, held_to = seq.len;
  if (SCORED && sc.end) {
    const int end = rv ? clamp_int(sc.end[tok], 0, seq.len) : 0;
    lim = min(lim, end);
    lim_most = lim;
    lim_least = rv ? lim : INT32_MAX;
    held_to = end;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      lim_most = max(lim_most, __shfl_xor(lim_most, o, 64));
      lim_least = min(lim_least, __shfl_xor(lim_least, o, 64));
      held_to = max(held_to, __shfl_xor(held_to, o, 64));
    }
    lim_most = __builtin_amdgcn_readfirstlane(lim_most);
    lim_least = __builtin_amdgcn_readfirstlane(lim_least);
    held_to = __builtin_amdgcn_readfirstlane(held_to);
  }
  // first key that this row sees, that some row and that every row does
  int low = 0, low_min = 0, low_max = 0;
  if (SCORED && sc.first) {
    low = rv ? max(sc.first[tok], 0) : 0;
    low_max = low;
    low_min = rv ? low : INT32_MAX;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
      low_max = max(low_max, __shfl_xor(low_max, o, 64));
      low_min = min(low_min, __shfl_xor(low_min, o, 64));
    }
    low_max = __builtin_amdgcn_readfirstlane(low_max);
    low_min = __builtin_amdgcn_readfirstlane(low_min);
  }
  const float slope = (MODE & kBias) != 0 ? sc.slopes[head] * kLog2e : 0.0f;

  // units nu0 .. nu - 1, this split's u0 .. u1 - 1
  const int top = SCORED && sc.end ? lim_most : tile_limit(seq, causal, rt, 16, G, prefix);
  const int nu = (top + kUnit - 1) / kUnit, nu0 = min(low_min / kUnit, nu);
  const int share = split_units(nu - nu0, splits, units);
  const int u0 = nu0 + split * share, u1 = min(u0 + share, nu);
  if (split > 0 && u0 >= nu) return;

  // ---- queries: channels 64 c + 16 g + 8 e .. + 7 of this lane's row
  half8_t qf[DC][2];
  float f_row = fabsf(scale) * kLog2e;
  {
    const uint16_t* qp = q + (int64_t)tok * q_stride + head * D + 16 * g;
    u32x4_t w[2 * DC];
#pragma unroll
    for (int i = 0; i < 2 * DC; ++i) {
      w[i] = u32x4_t{0, 0, 0, 0};
      if (rv) w[i] = *(const u32x4_t*)(qp + 64 * (i >> 1) + 8 * (i & 1));
      if (scale < 0.0f) w[i] ^= 0x80008000u;  // the scores' factor is kept positive
    }
    half8_t f[2 * DC];
    f_row *= queries_f16<DT, 2 * DC, 16>(w, f);
#pragma unroll
    for (int i = 0; i < 2 * DC; ++i) qf[i >> 1][i & 1] = f[i];
  }

  float m = kNone, l = 0.0f, ref = 0.0f;
  bool far = false;  // m of some row of the wave has passed kFar
  float4_t o[DN];
#pragma unroll
  for (int i = 0; i < DN; ++i) o[i] = float4_t{};

  // ---- a unit's loads: its keys go out as soon as the products have taken the
  // unit's before, its values likewise, the pages of the unit after ahead of
  // both.  Lane: keys of the 16 tokens at 16 (col >> 2), values and scales of
  // those at 16 g.  Units past the last repeat it.
  const int64_t page_bytes = (int64_t)D << c.lgT;
  const int32_t* table = c.table + (int64_t)b * c.width;
  const int last = max(u1 - 1, 0), mask = (1 << c.lgT) - 1;
  int k_page, v_page;
  auto turn_pages = [&](int u) {
    const int t0 = min(u, last) * kUnit;
    k_page = table[min((t0 + 16 * (col >> 2)) >> c.lgT, c.width - 1)];
    v_page = table[min((t0 + 16 * g) >> c.lgT, c.width - 1)];
  };
  u32x4_t kw[4][DC], vw[DN];
  float ks, vs;
  auto load_keys = [&](int u) {
    const int t = min(u, last) * kUnit + 16 * (col >> 2);
    const uint8_t* from = c.k + ((int64_t)clamp_int(k_page, 0, c.pages - 1) * c.Hkv + hk) * page_bytes +
                          (t & mask) * D + (col & 3) * D + 16 * g;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < DC; ++i) kw[a][i] = *(const u32x4_t*)(from + a * 4 * D + 64 * i);
  };
  auto load_values = [&](int u) {
    const int t = min(u, last) * kUnit + 16 * g;
    const int64_t slot = (int64_t)clamp_int(v_page, 0, c.pages - 1) * c.Hkv + hk;
    const uint8_t* from = c.v + slot * page_bytes + (t & mask) * D + col * 16;
    ks = c.ks[slot];
    vs = c.vs[slot];
#pragma unroll
    for (int i = 0; i < DN; ++i) vw[i] = *(const u32x4_t*)(from + i * 256);
  };
  if (u0 + wave < u1) {
    turn_pages(u0 + wave);
    load_keys(u0 + wave);
    load_values(u0 + wave);
    turn_pages(u0 + wave + 4);
  }
  // keys that every row of the tile sees
  const int lim_all = SCORED && sc.end ? lim_least : row_limit(seq, causal, rt * 16 / G, prefix);
  const bool whole = c.lgT >= 6;  // a unit lies in one page
  for (int u = u0 + wave; u < u1; u += 4) {
    const int t0 = u * kUnit;
    float4_t s[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      s[a] = float4_t{};
#pragma unroll
      for (int i = 0; i < DC; ++i) {
        s[a] = mfma16x16x32<DT_F16>(codes_f16(kw[a][i][0], kw[a][i][1]), qf[i][0], s[a]);
        s[a] = mfma16x16x32<DT_F16>(codes_f16(kw[a][i][2], kw[a][i][3]), qf[i][1], s[a]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    load_keys(u + 4);
    __builtin_amdgcn_sched_barrier(0);
    // past the sequence's end it may be no page of this sequence
    // (scored: nor does the scale matter of tokens that no row sees)
    const bool held = (whole || t0 + 16 * g < held_to) &&
                      (!SCORED || t0 + (whole ? 63 : 16 * g + 15) >= low_min);
    float f = held ? f_row * ks : 0.0f;
    // rows past the tile's last see what the others do; they are not written
    const bool edge = t0 + kUnit > lim_all || (SCORED && t0 < low_max);
    auto hidden = [&](int l) { return l >= lim || (SCORED && l < low); };
    if constexpr ((MODE & ~kMasks) != 0) {
      float t[1][16], factor[1] = {f};
#pragma unroll
      for (int i = 0; i < 16; ++i) t[0][i] = s[i >> 2][i & 3];
      if ((MODE & kCap) && edge) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (hidden(t0 + 16 * g + i)) t[0][i] = 0.0f;
      }
      put_on<MODE>(t, factor, sc, slope, {(float)(seq.first + ridx / G - t0 - 16 * g)});
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i >> 2][i & 3] = t[0][i];
      f = factor[0];
    }
    if (f == 0.0f) f = 1e-37f;  // a hidden key stays at -inf
    const float v_scale = held ? vs : 0.0f;
    const float vs_top = whole ? v_scale : four_rows_max(v_scale);
    if (edge) {
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (hidden(t0 + 16 * g + 4 * a + i)) s[a][i] = -INFINITY;
    }
    float mx = fmaxf(s[0][0], s[0][1]);
#pragma unroll
    for (int i = 2; i < 16; i += 2) mx = fmaxf(fmaxf(mx, s[i >> 2][i & 3]), s[i >> 2][(i & 3) + 1]);
    mx = four_rows_max(mx * f);
    float back = 1.0f;
    if (vs_top > 2.0f * ref) {
      const float to = fmaxf(vs_top, kRef);
      back = ref * __builtin_amdgcn_rcpf(to);
      ref = to;
    }
    if (__any(mx > m + kLag) || back != 1.0f) {
      const float mn = fmaxf(m, mx), alpha = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= alpha;
      const float both = alpha * back;
#pragma unroll
      for (int i = 0; i < DN; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][j] *= both;
      far = far || __any(fabsf(m) > kFar && m != kNone);
    }
    float off = m;
    if (__builtin_expect(far, false)) {
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[a][i] = s[a][i] * f - m;
      f = 1.0f;
      off = 0.0f;
    }
    const float q_v = v_scale * (ref > 0.0f ? __builtin_amdgcn_rcpf(ref) : 0.0f);
    const float ratio = q_v < kLeast ? kLeast : q_v;
    const float shift = __builtin_amdgcn_logf(ratio) + kLift - off;
    half8_t pf[2];
    float sum = 0.0f;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[a][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[a][i], f, shift));
    if (edge) {
      // exactly 0 where hidden, whatever the page's scales are
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (hidden(t0 + 16 * g + 4 * a + i)) s[a][i] = 0.0f;
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum += s[a][i];
        pf[a >> 1][4 * (a & 1) + i] = (_Float16)s[a][i];
      }
    l = sum != 0.0f ? __builtin_fmaf(sum, __builtin_amdgcn_rcpf(ratio), l) : l;
#pragma unroll
    for (int i = 0; i < DN; ++i) {
      o[i] = mfma16x16x32<DT_F16>(codes_f16(vw[i][0], vw[i][1]), pf[0], o[i]);
      o[i] = mfma16x16x32<DT_F16>(codes_f16(vw[i][2], vw[i][3]), pf[1], o[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    load_values(u + 4);
    turn_pages(u + 8);
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // ---- join the waves: lane holds channels 16 i + 4 g + j of row col
#pragma unroll
  for (int i = 0; i < DN; ++i) *(float4_t*)&joined[wave][col][16 * i + 4 * g] = o[i] * kPart * ref;
  if (g == 0) {
    stat[wave][0][col] = m;
    stat[wave][1][col] = l * kPart;
  }
  __syncthreads();
  // 16 lanes per row
  const int row = tid >> 4, part = tid & 15;
  const int rr = rt * 16 + row;
  float mm = -INFINITY, ll = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) mm = fmaxf(mm, stat[w][0][row]);
  const float base = mm == -INFINITY ? 0.0f : mm;
  float wt[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    wt[w] = __builtin_amdgcn_exp2f(stat[w][0][row] - base);
    ll += wt[w] * stat[w][1][row];
  }
  // channels of this lane: pairs 32 apart, so that 16 lanes hold 32 in a row
  constexpr int E = D / 16;
  auto channel = [&](int j) { return 32 * (j >> 1) + 2 * part + (j & 1); };
  float r[E];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    r[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) r[j] += wt[w] * joined[w][row][channel(j)];
  }
  const int64_t tk = seq.tok + min(rr / G, seq.n - 1);
  const int hd = hk * G + rr % G;
  const int mine = max(1, (nu - nu0 + share - 1) / share);  // splits with a unit
  if (mine > 1) {
    // ---- the last workgroup of the tile to arrive joins the splits, in order.
    // The partials go through the point where the GPU's caches meet (agent-scope
    // accesses) and have arrived there before the count does: a fence instead
    // would write back and empty a whole L2 for each workgroup (MI355X, 64
    // sequences of 8192 tokens: 490 us with fences).
    const int64_t at = (tk * c.H + hd) * splits;
    if (rr < seq.n * G) {
#pragma unroll
      for (int j = 0; j < E; j += 2) send2(parts.o + (at + split) * D + channel(j), r[j], r[j + 1]);
      if (part == 0) send2(parts.ml + (at + split) * 2, mm, ll);
    }
    __shared__ uint32_t arrived;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0) {
      uint32_t* count = parts.count + ((int64_t)b * c.Hkv + hk) * row_tiles + rt;
      arrived = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      if (arrived == (uint32_t)mine - 1)  // the last: ready for the next call
        __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (arrived != (uint32_t)mine - 1 || rr >= seq.n * G) return;
    mm = -INFINITY;
#pragma unroll 8
    for (int i = 0; i < mine; ++i) mm = fmaxf(mm, fetch2(parts.ml + (at + i) * 2).x);
    const float from = mm == -INFINITY ? 0.0f : mm;
    ll = 0.0f;
#pragma unroll
    for (int j = 0; j < E; ++j) r[j] = 0.0f;
#pragma unroll 4
    for (int i = 0; i < mine; ++i) {
      const float2 s = fetch2(parts.ml + (at + i) * 2);
      const float w = __builtin_amdgcn_exp2f(s.x - from);
      ll += w * s.y;
#pragma unroll
      for (int j = 0; j < E; j += 2) {
        const float2 v = fetch2(parts.o + (at + i) * D + channel(j));
        r[j] += w * v.x;
        r[j + 1] += w * v.y;
      }
    }
  }
  if (rr >= seq.n * G) return;
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;  // a row that sees nothing is 0
#pragma unroll
  for (int j = 0; j < E; j += 2)
    *(uint32_t*)(out + tk * out_stride + hd * D + channel(j)) =
        (uint32_t)round16<DT>(r[j] * inv) | (uint32_t)round16<DT>(r[j + 1] * inv) << 16;
  if (lse && part == 0)
    lse[tk * c.H + hd] = lse_of(mm, ll, kShrink);
}

// Position of a key row's 16-byte chunks in LDS (rows of 2 D bytes): 16 lanes
// that read one chunk of 16 rows meet all banks.
template <int D>
__device__ __forceinline__ int swizzle(int row) {
  return D == 128 ? row & 15 : (row >> 1) & 7;
}

// The products of many rows: W waves, each 32 rows, share the conversion of
// the keys and values of a unit of 64 tokens to fp16 in LDS.
//
//  * v_mfma_f32_32x32x16_f16.  Scores come out as S^T; the keys' rows are
//    permuted so that lane l (half h = l >> 5) holds tokens 16 h + i of each 32
//    in register i, the operand layout of the second product, O^T += V^T P^T.
//  * The scores of the next unit are formed while this one's become
//    probabilities, and later units' codes are staged while the second product
//    runs: a wave's matrix and vector instructions alternate.
//  * A unit's codes are loaded into registers a unit before they are turned to
//    fp16 and written to LDS, its scales and page numbers ahead of those.
//    Keys: rows of 2 D bytes, their 16-byte chunks permuted by row; values:
//    [16 tokens][8 of them][channel] pieces of 16 bytes.  Reads and writes meet
//    all banks.
//
// The matrix and the vector unit share the time: a unit of 64 tokens costs a
// wave 2 D / 16 products of 32 cycles, and some 600 vector operations for its
// probabilities.  MI355X, 4 sequences of 2048 new over 8192, D = 128: 40 / 8 heads
// 1247 us (965 TFLOP/s), 32 / 32 heads 953 TFLOP/s, D = 64: 694 TFLOP/s (random
// codes).  Ragged chunks of up to 2048 over up to 8192 (normal keys and values) take
// 1076 us, matrix units busy 46 %, and 2161 in the decode kernel's form.
//
// WHOLE: pages of 64 tokens and more, a unit lies in one page.
template <int D>
constexpr int kPromptWaves = D / 16;

template <int DT, int D, bool WHOLE, int MODE>
__global__ void __launch_bounds__(64 * kPromptWaves<D>) __attribute__((amdgpu_waves_per_eu(1, 2)))
kv8_prompt_kernel(Kv8 c, const uint16_t* __restrict__ q, int64_t q_stride, float scale, int causal,
                  uint16_t* __restrict__ out, int64_t out_stride, float* __restrict__ lse,
                  Parts parts, int row_tiles, int splits, int units, Scoring sc) {
  // in iteration u the keys of u + 1 and the values of u are read, and both of
  // u + 2 written
  constexpr int NBK = 2, NBV = 3, W = kPromptWaves<D>;
  constexpr bool SCORED = MODE != kPlain;
  constexpr int KS = D / 16, DN = D / 32, ROWS = 32 * W;
  constexpr int BUF = kUnit * D * 2;                // fp16 keys (or values) of a unit
  static_assert(kUnit * D == 64 * W * 16, "a 16-byte piece of each for every lane");
  // two waves to a SIMD: 256 registers each, the queries wait in LDS
  constexpr bool Q_LDS = W == 8;
  __shared__ __attribute__((aligned(16))) uint8_t lds[(NBK + NBV) * BUF + (Q_LDS ? ROWS * D * 2 : 0)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, h = lane >> 5;
  // workgroups go to the 8 XCDs in turn: all row tiles of one (split, sequence,
  // kv head) go to one of them and share their keys in its cache; those of the
  // groups that are left when each has as many go to all of them, so that none
  // waits for the others (12 groups of 251 tiles, packed documents: 600 us -> 472);
  // the last tiles, which see the most, first
  const int groups = c.B * c.Hkv * splits, per_xcd = groups >> 3, rest = groups & 7;
  const int shared = (rest * row_tiles + 7) >> 3;  // workgroups of an XCD for those
  int at = (int)(blockIdx.x >> 3), grp, rt;
  if (at < shared) {
    const int i = at * 8 + (int)(blockIdx.x & 7);
    if (i >= rest * row_tiles) return;
    grp = per_xcd * 8 + i % rest;
    rt = row_tiles - 1 - i / rest;
  } else {
    at -= shared;
    grp = at % per_xcd * 8 + (int)(blockIdx.x & 7);
    rt = row_tiles - 1 - at / per_xcd;
  }
  // (but where there are documents and a prefix the first ones do, which see the
  // prefix to its end: packed documents, half of them prefix, 472 us -> 425)
  if (SCORED && sc.first && sc.prefix) rt = row_tiles - 1 - rt;
  const int hk = grp % c.Hkv, b = grp / c.Hkv % c.B, split = grp / c.Hkv / c.B;
  const int G = c.H / c.Hkv;
  const Kv8Seq seq = kv8_seq(c, b);
  if (rt * ROWS >= seq.n * G) return;
  const int row0 = rt * ROWS + wave * 32, ridx = row0 + col;
  const bool rv = ridx < seq.n * G;
  const int tok = seq.tok + (rv ? ridx / G : 0), head = hk * G + (rv ? ridx % G : 0);
  const int prefix = SCORED && sc.prefix ? sc.prefix[b] : 0;
  int lim = rv ? row_limit(seq, causal, ridx / G, prefix) : 0;
  // keys that every row of this wave sees
  int lim_all = row0 + 31 < seq.n * G ? row_limit(seq, causal, row0 / G, prefix) : 0;
  // rows with ends: the largest limit of the workgroup; and where tokens begin that
  // hold nothing which some row of this wave sees
  int lim_most = 0, held_to = WHOLE ? INT32_MAX : seq.len;
  // first key that this row sees, that some row of the workgroup and that every
  // row of this wave does
  int low = 0, low_min = 0, low_max = 0, low_wave = 0;
  if constexpr (SCORED) {
    __shared__ int lows[W], tops[W];
    if (sc.end) {
      const int end = rv ? clamp_int(sc.end[tok], 0, seq.len) : 0;
      lim = min(lim, end);
      lim_most = lim_all = lim;
      held_to = end;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        lim_most = max(lim_most, __shfl_xor(lim_most, o, 64));
        lim_all = min(lim_all, __shfl_xor(lim_all, o, 64));
        held_to = max(held_to, __shfl_xor(held_to, o, 64));
      }
      lim_all = __builtin_amdgcn_readfirstlane(lim_all);
      held_to = __builtin_amdgcn_readfirstlane(held_to);
      if (lane == 0) tops[wave] = lim_most;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) lim_most = max(lim_most, tops[w]);
      lim_most = __builtin_amdgcn_readfirstlane(lim_most);
    }
    if (sc.first) {
      low = rv ? max(sc.first[tok], 0) : 0;
      low_max = low;
      low_min = rv ? low : INT32_MAX;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        low_max = max(low_max, __shfl_xor(low_max, o, 64));
        low_min = min(low_min, __shfl_xor(low_min, o, 64));
      }
      low_max = __builtin_amdgcn_readfirstlane(low_max);
      low_wave = __builtin_amdgcn_readfirstlane(low_min);
      if (lane == 0) lows[wave] = low_min;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) low_min = min(low_min, lows[w]);
      low_min = __builtin_amdgcn_readfirstlane(low_min);
    }
  }
  const float slope = (MODE & kBias) != 0 ? sc.slopes[head] * kLog2e : 0.0f;

  const int position = seq.first + ridx / G;

  // units nu0 .. nu - 1, this split's u0 .. u1 - 1
  const int top = SCORED && sc.end ? lim_most : tile_limit(seq, causal, rt, ROWS, G, prefix);
  const int nu = (top + kUnit - 1) / kUnit, nu0 = min(low_min / kUnit, nu);
  const int share = split_units(nu - nu0, splits, units);
  const int u0 = nu0 + split * share, u1 = min(u0 + share, nu);
  if (split > 0 && u0 >= nu) {
    // (scored: the join does not know which splits have units)
    if (SCORED && rv && h == 0) {
      const int64_t at_p = ((int64_t)tok * c.H + head) * splits + split;
      parts.ml[at_p * 2] = kNone;
      parts.ml[at_p * 2 + 1] = 0.0f;
    }
    return;
  }

  half8_t qf[Q_LDS ? 1 : KS];
  uint8_t* q_mine = lds + (NBK + NBV) * BUF + (wave * KS * 64 + lane) * 16;
  auto query = [&](int i) {
    if constexpr (Q_LDS) return *(const half8_t*)(q_mine + i * 1024);
    else return qf[i];
  };
  float f_row = scale * kLog2e;
  {
    u32x4_t w[KS];
    half8_t f[KS];
    const uint16_t* qp = q + (int64_t)tok * q_stride + head * D + 8 * h;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      w[i] = u32x4_t{0, 0, 0, 0};
      if (rv) w[i] = *(const u32x4_t*)(qp + 16 * i);
      if (scale < 0.0f) w[i] ^= 0x80008000u;  // the scores' factor is kept positive
    }
    f_row = fabsf(f_row) * queries_f16<DT, KS, 32>(w, f);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      if constexpr (Q_LDS) *(half8_t*)(q_mine + i * 1024) = f[i];
      else qf[i] = f[i];
    }
  }

  // ---- staging: this lane's piece is 16 bytes at 16 tid of the unit's [4
  // subtiles][16 D]
  const int64_t page_bytes = (int64_t)D << c.lgT;
  const int T = 1 << c.lgT;
  const int32_t* table = c.table + (int64_t)b * c.width;
  u32x4_t kw, vw;
  // table entries of this lane's piece of a unit, and of its 16 tokens of
  // each 32 (WHOLE: one for all), units past the last repeating it; they are
  // brought into range where they are used, a unit later
  constexpr int NSC = WHOLE ? 1 : 2;
  const int sub = tid / D, in_sub = tid % D * 16;
  int of_piece, of_scale[NSC];
  auto entry = [&](int u, int token) {
    return table[min((min(u, nu - 1) * kUnit + token) >> c.lgT, c.width - 1)];
  };
  auto turn_pages = [&](int u_pieces, int u_scales) {
    of_piece = entry(u_pieces, WHOLE ? 0 : 16 * sub);
#pragma unroll
    for (int a = 0; a < NSC; ++a) of_scale[a] = entry(u_scales, WHOLE ? 0 : 32 * a + 16 * h);
  };
  // (the empty statements hold a loaded value's first use where it stands)
  auto fetch = [&](int u) {
    asm volatile("" : "+v"(of_piece));
    const int t = min(u, nu - 1) * kUnit;
    int64_t from;
    if constexpr (WHOLE) {
      const int page = clamp_int(__builtin_amdgcn_readfirstlane(of_piece), 0, c.pages - 1);
      from = ((int64_t)page * c.Hkv + hk) * page_bytes + (int64_t)(t & (T - 1)) * D + tid * 16;
    } else {
      from = ((int64_t)clamp_int(of_piece, 0, c.pages - 1) * c.Hkv + hk) * page_bytes +
             ((t + 16 * sub) & (T - 1)) * D + in_sub;
    }
    kw = *(const u32x4_t*)(c.k + from);
    vw = *(const u32x4_t*)(c.v + from);
  };
  float ks_next[NSC], vs_next[NSC];
  auto fetch_scales = [&]() {
#pragma unroll
    for (int a = 0; a < NSC; ++a) {
      asm volatile("" : "+v"(of_scale[a]));
      const int64_t at_s = (int64_t)clamp_int(of_scale[a], 0, c.pages - 1) * c.Hkv + hk;
      ks_next[a] = c.ks[at_s];
      vs_next[a] = c.vs[at_s];
    }
  };
  // part j of 4: half a piece of keys or values to its buffer.  A key (token 16
  // sub + tk of the unit) is row 32 (sub >> 1) + the bits of its place in 32
  // tokens in the order 0, 1, subtile's parity, 2, 3.
  const int tk = in_sub / D, k_row = 32 * (sub >> 1) + (tk & 3) + 4 * (sub & 1) + 8 * (tk >> 2);
  int k_place = k_row * D * 2 + (((in_sub % D / 8) ^ swizzle<D>(k_row)) << 4);
  int v_place = (sub * 2 * D + tid % D) * 16;
  auto stage = [&](int j, int kbuf, int vbuf) {
    const int e = j & 1;
    if (j & 2)  // a channel's tokens 16 sub + 8 e ..
      *(half8_t*)(lds + (NBK + vbuf) * BUF + v_place + e * D * 16) =
          codes_f16(vw[2 * e], vw[2 * e + 1]);
    else        // a token's channels 16 ch + 8 e ..
      *(half8_t*)(lds + kbuf * BUF + (k_place ^ e << 4)) = codes_f16(kw[2 * e], kw[2 * e + 1]);
  };

  float m = kNone, l = 0.0f, ref = 0.0f;
  bool far = false;  // m of some row of the wave has passed kFar
  float16_t o[DN], even[2], odd[2];  // scores of the units 0, 2, .. and 1, 3, ..
#pragma unroll
  for (int i = 0; i < DN; ++i) o[i] = float16_t{};

  // operand k of the scores of a unit (channels 16 (k >> 1) .., tokens 32 (k &
  // 1) ..), and of the second product (tile k / DN of 16 tokens, channels 32 (k %
  // DN) ..)
  int k_lane = col * D * 2 + ((h ^ swizzle<D>(col)) << 4), v_lane = (2 * h * D + col) * 16;
  auto key = [&](int kbuf, int k) {
    return *(const half8_t*)(lds + kbuf * BUF + (k & 1) * 64 * D + (k_lane ^ (k >> 1) << 5));
  };
  auto value = [&](int vbuf, int k) {
    const int te = k / DN;
    return *(const half8_t*)(lds + (NBK + vbuf) * BUF + v_lane +
                             ((4 * (te >> 1) + (te & 1)) * D + 32 * (k % DN)) * 16);
  };
  // One unit.  EDGE: some row of the wave does not see all of it.
  auto unit = [&](auto edge, float16_t (&s)[2], float16_t (&next)[2], int u, int kbuf, int vbuf,
                  int kbuf_in, int vbuf_in) {
    constexpr bool EDGE = decltype(edge)::value;
    const int t0 = u * kUnit;
    // (renewed each unit, so that the compiler forms addresses from these and
    // does not keep each of them)
    asm volatile("" : "+v"(k_lane), "+v"(v_lane), "+v"(k_place), "+v"(v_place));
    float f[NSC], vs[NSC], vs_top;
#pragma unroll
    for (int a = 0; a < NSC; ++a) {
      asm volatile("" : "+v"(ks_next[a]), "+v"(vs_next[a]));
      // past the sequence's end it may be no page of this sequence
      // (scored: nor does the scale matter of tokens that no row of the wave sees)
      const bool held = ((WHOLE && !SCORED) || t0 + (WHOLE ? 0 : 32 * a + 16 * h) < held_to) &&
                        (!SCORED || t0 + (WHOLE ? 63 : 32 * a + 16 * h + 15) >= low_wave);
      f[a] = held ? f_row * ks_next[a] : 0.0f;
      vs[a] = held ? vs_next[a] : 0.0f;
    }
    auto hidden = [&](int l) { return l >= lim || (SCORED && l < low); };
    if constexpr ((MODE & ~kMasks) != 0) {
      float t[2][16], factor[2] = {f[0], f[NSC - 1]};
#pragma unroll
      for (int i = 0; i < 32; ++i)
        t[i >> 4][i & 15] =
            EDGE && (MODE & kCap) && hidden(t0 + 32 * (i >> 4) + 16 * h + (i & 15)) ? 0.0f : s[i >> 4][i & 15];
      const float back = (float)(position - t0 - 16 * h);
      put_on<MODE>(t, factor, sc, slope, {back, back - 32.0f});
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i >> 4][i & 15] = t[i >> 4][i & 15];
#pragma unroll
      for (int a = 0; a < NSC; ++a) f[a] = factor[a];
    }
#pragma unroll
    for (int a = 0; a < NSC; ++a)
      if (f[a] == 0.0f) f[a] = 1e-37f;  // a hidden key stays at -inf
    vs_top = vs[0];
    if constexpr (!WHOLE) vs_top = both_halves_max(fmaxf(vs[0], vs[1]));
    // ---- the rows' maxima
    float mx = -INFINITY;
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      if (EDGE) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (hidden(t0 + 32 * a + 16 * h + i)) s[a][i] = -INFINITY;
      }
      float t = fmaxf(s[a][0], s[a][1]);
#pragma unroll
      for (int i = 2; i < 16; i += 2) t = fmaxf(fmaxf(t, s[a][i]), s[a][i + 1]);
      mx = fmaxf(mx, t * f[WHOLE ? 0 : a]);
    }
    mx = both_halves_max(mx);
    float back = 1.0f;
    if (vs_top > 2.0f * ref) {
      const float to = fmaxf(vs_top, kRef);
      back = ref * __builtin_amdgcn_rcpf(to);
      ref = to;
    }
    if (__any(mx > m + kLag) || back != 1.0f) {
      const float mn = fmaxf(m, mx), alpha = __builtin_amdgcn_exp2f(m - mn);
      m = mn;
      l *= alpha;
      const float both = alpha * back;
#pragma unroll
      for (int i = 0; i < DN; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) o[i][j] *= both;
      far = far || __any(fabsf(m) > kFar && m != kNone);
    }
    float off = m;
    if (__builtin_expect(far, false)) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
#pragma unroll
        for (int i = 0; i < 16; ++i) s[a][i] = s[a][i] * f[WHOLE ? 0 : a] - m;
      }
#pragma unroll
      for (int a = 0; a < NSC; ++a) f[a] = 1.0f;
      off = 0.0f;
    }
    __builtin_amdgcn_sched_barrier(0);
    // ---- the next unit's scores, one product at a time, and between them this
    // unit's probabilities: operand e of tile a is tokens 16 h + 8 e ..
    half8_t pf[2][2], fr[4];
    const float over = ref > 0.0f ? __builtin_amdgcn_rcpf(ref) : 0.0f;
    float ratio[NSC], shift[NSC], sum[NSC];
#pragma unroll
    for (int a = 0; a < NSC; ++a) {
      const float q_v = vs[a] * over;
      ratio[a] = q_v < kLeast ? kLeast : q_v;
      shift[a] = __builtin_amdgcn_logf(ratio[a]) + kLift - off;
      sum[a] = 0.0f;
    }
    constexpr int N1 = 2 * KS, PER = 32 / N1;
#pragma unroll
    for (int k = 0; k < 3; ++k) fr[k] = key(kbuf, k);
    half8_t qr[2] = {query(0), query(0)};
#pragma unroll
    for (int k = 0; k < N1; ++k) {
      if (k + 3 < N1) fr[(k + 3) & 3] = key(kbuf, k + 3);
      if ((k & 1) == 0 && k + 2 < N1) qr[(k >> 1) + 1 & 1] = query((k >> 1) + 1);
      next[k & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[k & 3], qr[k >> 1 & 1], k < 2 ? float16_t{} : next[k & 1],
                                                           0, 0, 0);
#pragma unroll
      for (int x = k * PER; x < (k + 1) * PER; ++x) {
        const int a = x >> 4, i = x & 15, z = WHOLE ? 0 : a;
        float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[a][i], f[z], shift[z]));
        // exactly 0 where hidden, whatever the page's scales are
        if (EDGE && hidden(t0 + 32 * a + 16 * h + i)) p = 0.0f;
        sum[z] += p;
        pf[a][i >> 3][i & 7] = (_Float16)p;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // ---- the second product, and between its steps the staging of the unit
    // after the next
    constexpr int N2 = 4 * DN, PARTS = 4;
#pragma unroll
    for (int k = 0; k < 3; ++k) fr[k] = value(vbuf, k);
#pragma unroll
    for (int a = 0; a < NSC; ++a)
      l = sum[a] != 0.0f ? __builtin_fmaf(sum[a], __builtin_amdgcn_rcpf(ratio[a]), l) : l;
#pragma unroll
    for (int k = 0; k < N2; ++k) {
      if (k + 3 < N2) fr[(k + 3) & 3] = value(vbuf, k + 3);
      o[k % DN] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fr[k & 3], pf[k / DN >> 1][k / DN & 1],
                                                         o[k % DN], 0, 0, 0);
#pragma unroll
      for (int j = k * PARTS / N2; j < (k + 1) * PARTS / N2; ++j) stage(j, kbuf_in, vbuf_in);
      __builtin_amdgcn_sched_barrier(0);
    }
    fetch_scales();
    fetch(u + 3);
    turn_pages(u + 4, u + 2);
    __builtin_amdgcn_sched_barrier(0);
  };

  // ---- the first units
  if (u0 < u1) {
    turn_pages(u0, u0);
    fetch(u0);
    fetch_scales();
    turn_pages(u0 + 1, u0 + 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) stage(j, 0, 0);
    fetch(u0 + 1);
    turn_pages(u0 + 2, u0 + 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) stage(j, 1, 1);
    fetch(u0 + 2);
    turn_pages(u0 + 3, u0 + 1);
    __syncthreads();
    even[0] = even[1] = float16_t{};
#pragma unroll
    for (int k = 0; k < 2 * KS; ++k)
      even[k & 1] =
          __builtin_amdgcn_mfma_f32_32x32x16_f16(key(0, k), query(k >> 1), even[k & 1], 0, 0, 0);
  }
  int vb = 0;
  auto turn = [&](auto edge, float16_t (&now)[2], float16_t (&next)[2], int u, int parity) {
    // the keys of u + 1 and the values of u are whole in LDS, and nobody reads
    // any more what this iteration overwrites: in the first one the keys of u0,
    // of which every wave has formed its scores just above
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    const int vb2 = vb == 0 ? 2 : vb - 1;  // (vb + 2) % 3
    unit(edge, now, next, u, parity ^ 1, vb, parity, vb2);
    vb = vb == 2 ? 0 : vb + 1;
  };
  int u = u0;
  if constexpr (SCORED) {
    for (; u < u1 && u * kUnit < low_max; u += 2) {
      turn(std::true_type{}, even, odd, u, 0);
      if (u + 1 < u1) turn(std::true_type{}, odd, even, u + 1, 1);
    }
  }
  for (; u + 1 < u1 && (u + 2) * kUnit <= lim_all; u += 2) {
    turn(std::false_type{}, even, odd, u, 0);
    turn(std::false_type{}, odd, even, u + 1, 1);
  }
  for (; u < u1; u += 2) {
    turn(std::true_type{}, even, odd, u, 0);
    if (u + 1 < u1) turn(std::true_type{}, odd, even, u + 1, 1);
  }
  l += __shfl_xor(l, 32, 64);

  // ---- results: register j of o[i] is channel 32 i + (j & 3) + 8 (j >> 2) + 4 h
  if (!rv) return;
  if (splits > 1) {
    const int64_t at_p = ((int64_t)tok * c.H + head) * splits + split;
#pragma unroll
    for (int i = 0; i < DN; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4_t v = {o[i][4 * j], o[i][4 * j + 1], o[i][4 * j + 2], o[i][4 * j + 3]};
        *(float4_t*)(parts.o + at_p * D + 32 * i + 8 * j + 4 * h) = v * kPart * ref;
      }
    if (h == 0) {
      parts.ml[at_p * 2] = m;
      parts.ml[at_p * 2 + 1] = l * kPart;
    }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;  // a row that sees nothing is 0
  uint16_t* dst = out + (int64_t)tok * out_stride + head * D;
#pragma unroll
  for (int i = 0; i < DN; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = round16<DT>(o[i][4 * j + e] * inv * ref);
      *(u32x2_t*)(dst + 32 * i + 8 * j + 4 * h) = u32x2_t{y[0] | y[1] << 16, y[2] | y[3] << 16};
    }
  if (lse && h == 0)
    lse[(int64_t)tok * c.H + head] = lse_of(m, l, 0.0f);
}

// Joins the prompt kernel's splits of a row, in their order: one wave per
// (token, head).
template <int DT, int D, int MODE>
__global__ void __launch_bounds__(256)
kv8_join_kernel(Kv8 c, int causal, uint16_t* __restrict__ out, int64_t out_stride,
                float* __restrict__ lse, Parts parts, int splits, int units, int rows, int max_new) {
  const int lane = threadIdx.x & 63;
  const int G = c.H / c.Hkv;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= (int64_t)c.B * max_new * c.H) return;
  const int hd = (int)(i % c.H), j = (int)(i / c.H % max_new), b = (int)(i / c.H / max_new);
  const Kv8Seq seq = kv8_seq(c, b);
  if (j >= seq.n) return;
  constexpr bool SCORED = MODE != kPlain;
  // (scored: every split has left its sum, those without units a 0)
  int n = splits;
  if constexpr (!SCORED) {
    const int top = tile_limit(seq, causal, (j * G + hd % G) / rows, rows, G);
    const int nu = (top + kUnit - 1) / kUnit;
    const int share = split_units(nu, splits, units);
    n = max((nu + share - 1) / share, 1);
  }
  const int64_t row = (int64_t)(seq.tok + j) * c.H + hd;
  float m = -INFINITY;
  for (int s = 0; s < n; ++s) m = fmaxf(m, parts.ml[(row * splits + s) * 2]);
  const float base = m == -INFINITY ? 0.0f : m;
  constexpr int E = D / 64;
  float l = 0.0f, r[E] = {};
  for (int s = 0; s < n; ++s) {
    const int64_t at = row * splits + s;
    const float w = __builtin_amdgcn_exp2f(parts.ml[at * 2] - base);
    if (SCORED && parts.ml[at * 2 + 1] == 0.0f) continue;  // saw nothing
    l += w * parts.ml[at * 2 + 1];
#pragma unroll
    for (int e = 0; e < E; ++e) r[e] += w * parts.o[at * D + lane * E + e];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    out[(seq.tok + j) * out_stride + hd * D + lane * E + e] = round16<DT>(r[e] * inv);
  if (lse && lane == 0) lse[row] = lse_of(m, l, kShrink);
}

template <int DT, int D, int MODE>
hipError_t launch_attention(const Kv8& c, const Plan& p, const void* q, int64_t q_stride,
                            float scale, int causal, void* out, int64_t out_stride, float* lse,
                            int64_t max_new, void* ws, const Scoring& sc, hipStream_t st) {
  const int64_t rows = (int64_t)c.tokens * c.H * p.splits;
  Parts parts = {(float*)((uint8_t*)ws + kCounters * 4), nullptr, (uint32_t*)ws};
  parts.ml = parts.o + pad256(rows * D * 4) / 4;
  const int64_t groups = (int64_t)c.B * c.Hkv * p.splits;
  auto go = [&](auto kernel, int64_t grid, int threads) {
    launch_timed(kernel, dim3((unsigned)grid), dim3(threads), 0, st, c, (const uint16_t*)q,
                 q_stride, scale, causal, (uint16_t*)out, out_stride, lse, parts, p.row_tiles,
                 p.splits, p.units, sc);
  };
  const int64_t grid = p.waves ? 8 * (groups / 8 * p.row_tiles + ceil_div(groups % 8 * p.row_tiles, 8))
                               : 8 * ceil_div(groups, 8) * p.row_tiles;
  const bool whole = (1 << c.lgT) >= kUnit;
  if (p.waves == 0) go(kv8_decode_kernel<DT, D, MODE>, grid, 256);
  else if (whole) go(kv8_prompt_kernel<DT, D, true, MODE>, grid, 64 * kPromptWaves<D>);
  else go(kv8_prompt_kernel<DT, D, false, MODE>, grid, 64 * kPromptWaves<D>);
  if (p.waves && p.splits > 1)
    hipLaunchKernelGGL((kv8_join_kernel<DT, D, MODE == kPlain ? kPlain : kMasks>),
                       dim3((unsigned)ceil_div((int64_t)c.B * max_new * c.H, 4)), dim3(256), 0,
                       st, c, causal, (uint16_t*)out, out_stride, lse, parts, p.splits, p.units, p.rows,
                       (int)max_new);
  return hipGetLastError();
}

template <int MODE>
AttentionLaunch* launcher(int32_t D, int32_t dtype) {
  return D == 64 ? (dtype == DT_F16 ? launch_attention<DT_F16, 64, MODE>
                                    : launch_attention<DT_BF16, 64, MODE>)
                 : (dtype == DT_F16 ? launch_attention<DT_F16, 128, MODE>
                                    : launch_attention<DT_BF16, 128, MODE>);
}

}  // namespace
}  // namespace w4a16
