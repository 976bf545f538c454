// kv8.hip -- writing the paged 8-bit cache: appending keys and values with
// the position rotation on the way, and reading pages back in 16 bits.
#include "kv8.h"

namespace w4a16 {
namespace {

struct Rope {
  const float* cos;  // [rows, dim / 2] or null: no rotation
  const float* sin;
  int rows, dim, interleaved;
};

// A lane's 16 channels of a row: two pieces of 8, D / 16 lanes to a row.  Lane j
// of a half-split rotation has channels 8 j .. and their partners dim / 2
// further on (the channels past dim, two pieces a lane, come after those); all
// else has channels 16 j ..
struct Place {
  int a, b;     // first channel of each piece
  bool turned;  // rotated
};
__device__ __forceinline__ Place place_of(const Rope& r, int j, bool rotated) {
  const int turning = rotated && r.cos ? r.dim >> 4 : 0;
  if (turning && !r.interleaved && j < turning) return Place{8 * j, 8 * j + (r.dim >> 1), true};
  return Place{16 * j, 16 * j + 8, j < turning};
}

// The angles of a lane's pairs at a position: cos and sin of channels a .. a + 7
// with their partners, or of the 4 pairs in each piece.
struct Angles {
  float4_t c[2], s[2];
};
__device__ __forceinline__ Angles angles_of(const Rope& r, const Place& p, int pos) {
  Angles g{};
  if (p.turned) {
    const int64_t at = (int64_t)clamp_int(pos, 0, r.rows - 1) * (r.dim >> 1) +
                       (r.interleaved ? p.a >> 1 : p.a);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      g.c[i] = *(const float4_t*)(r.cos + at + 4 * i);
      g.s[i] = *(const float4_t*)(r.sin + at + 4 * i);
    }
  }
  return g;
}

// Pair (a, b) becomes (a cos - b sin, b cos + a sin), products and sums in
// fp32, each rounded once.
__device__ __forceinline__ void rotate(float (&x)[16], const Angles& g, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float c = g.c[i >> 2][i & 3], s = g.s[i >> 2][i & 3];
    if (interleaved) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c - b * s;
      x[2 * i + 1] = b * c + a * s;
    } else {
      const float a = x[i], b = x[i + 8];
      x[i] = a * c - b * s;
      x[i + 8] = b * c + a * s;
    }
  }
}

template <int DT>
__device__ __forceinline__ void widen16x(u32x4_t a, u32x4_t b, float (&f)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = i < 4 ? a[i] : b[i - 4];
    f[2 * i] = widen16<DT>((uint16_t)(w & 0xFFFFu));
    f[2 * i + 1] = widen16<DT>((uint16_t)(w >> 16));
  }
}
template <int DT>
__device__ __forceinline__ u32x4_t round8(const float* f) {
  u32x4_t r;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = (uint32_t)round16<DT>(f[2 * i]) | (uint32_t)round16<DT>(f[2 * i + 1]) << 16;
  return r;
}
__device__ __forceinline__ uint32_t mag16(const float (&f)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, mag_bits(f[i]));
  return m;
}

// 16 stored codes requantized to a scale that is 1 / ratio (new / old) times theirs.
__device__ __forceinline__ u32x4_t requantized(u32x4_t w, float ratio) {
  u32x4_t r = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int c = (int)((w[i >> 2] >> (8 * (i & 3))) & 0xFFu) - 128;
    const int n = (int)fminf(fmaxf(rintf((float)c * ratio), -128.0f), 127.0f) + 128;
    r[i >> 2] |= (uint32_t)n << (8 * (i & 3));
  }
  return r;
}

// A page's new scale from the old one (0 if the page begins with this call's
// rows) and the new rows' largest magnitude.  A scale that is NaN stays NaN
// while its page holds older rows.
__device__ __forceinline__ float grown_scale(float old, uint32_t mag) {
  const float fresh = scale_of(mag);
  return old != old || fresh != fresh ? __builtin_nanf("") : fmaxf(old, fresh);
}

// 8 codes as stored, 8 bytes.
__device__ __forceinline__ u32x2_t stored8(const float* f, const Codes8& q) {
  float x[8];
  int c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = f[i];
  if (q.s == 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 0;
  } else {
    q(x, c);
  }
  u32x2_t r = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i >> 2] |= ((uint32_t)(c[i] + 128) & 0xFFu) << (8 * (i & 3));
  return r;
}

// Queries of one token, rotated: 256 lanes, D / 16 to a head, the angles held
// for all heads of the lane.
template <int DT, int D>
__device__ void turn_queries(const Kv8& c, const Rope& rope, const uint16_t* q, int64_t q_stride,
                             uint16_t* out, int64_t o_stride, int tok) {
  constexpr int L = D / 16, R = 256 / L;
  // the token's sequence: the last b with cu[b] <= tok
  int b = tok;
  if (c.cu) {
    int lo = 0, hi = c.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (c.cu[mid] <= tok) lo = mid;
      else hi = mid;
    }
    b = lo;
  }
  const Kv8Seq s = kv8_seq(c, b);
  if (tok - s.tok >= s.n) return;
  const Place p = place_of(rope, threadIdx.x % L, true);
  const Angles g = angles_of(rope, p, s.first + tok - s.tok);
  const uint16_t* src = q + (int64_t)tok * q_stride;
  uint16_t* dst = out + (int64_t)tok * o_stride;
  constexpr int AT_ONCE = 4;
  for (int h0 = threadIdx.x / L; h0 < c.H; h0 += AT_ONCE * R) {
    u32x4_t w[AT_ONCE][2];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int h = h0 + i * R;
      if (h < c.H) {
        w[i][0] = *(const u32x4_t*)(src + h * D + p.a);
        w[i][1] = *(const u32x4_t*)(src + h * D + p.b);
      }
    }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      const int h = h0 + i * R;
      if (h >= c.H) break;
      float f[16];
      widen16x<DT>(w[i][0], w[i][1], f);
      if (p.turned) rotate(f, g, rope.interleaved);
      *(u32x4_t*)(dst + h * D + p.a) = round8<DT>(f);
      *(u32x4_t*)(dst + h * D + p.b) = round8<DT>(f + 8);
    }
  }
}

// Room of the pages that sequences b' < b touch: n new tokens lie in at most
// n / T + 2 pages, so sequence b's pages have the places [at(b), at(b + 1)) of
// tokens / T + 2 B in all.
__device__ __forceinline__ int pages_before(const Kv8& c, int b) {
  return (clamp_int(c.cu[b], 0, c.tokens) >> c.lgT) + 2 * b;
}

// The sequence that has place s, by the whole wave: 64 sequences at a look.
__device__ __forceinline__ int sequence_at(const Kv8& c, int s) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = c.B;
  while (n > 1) {
    const int step = (n + 63) >> 6, i = min(lane * step, n - 1);
    const uint64_t before = __ballot(lane * step < n && pages_before(c, lo + i) <= s);
    const int skip = max(__popcll(before) - 1, 0) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

// Several new tokens.  One workgroup per (sequence, touched page, kv head, keys
// or values), the only one to touch those bytes and that scale.  The new rows
// are read once and kept, rotated, in registers; the page's scale is the larger
// of the old one and the new rows' own; where it grew, the page's older rows
// are requantized to it.
// PASSES: ceil(T D / 16 / 256) rows of lanes.
//
// The bytes bound it: rows in 16 bits are read once, codes and rotated queries
// written once.  MI355X, prompts of 17 k tokens, 40 query and 8 kv heads of 128:
// 97 to 105 us, 145 MB read and 225 MB written by the counters, 3.7 TB/s.  The
// queries of a token are turned by one workgroup, its angles held over its heads;
// that and reading back by 128-byte pieces took the pair from 217 to 136 us.
template <int DT, int D, int PASSES>
__device__ void append_page(const Kv8& c, const Rope& rope, const uint16_t* x, int64_t stride,
                            bool values, int b, int chunk, int head, uint8_t* lds,
                            uint32_t* part) {
  const Kv8Seq q = kv8_seq(c, b);
  const int T = 1 << c.lgT, start = max(q.first, 0), end = q.first + q.n;
  const int p = (start >> c.lgT) + chunk;
  if (q.n == 0 || (p << c.lgT) >= end) return;
  const int r0 = max(start - (p << c.lgT), 0), r1 = min(end - (p << c.lgT), T);
  const int tok0 = q.tok + (p << c.lgT) - q.first;  // new token of the page's row 0
  const int page = kv8_page(c, b, p);
  const int64_t slot = (int64_t)page * c.Hkv + head;
  uint8_t* dst = (values ? c.v : c.k) + slot * ((int64_t)T * D);
  float* scale = (values ? c.vs : c.ks) + slot;

  constexpr int L = D / 16;     // lanes per row
  constexpr int R = 256 / L;    // rows per pass
  const int tid = threadIdx.x;
  const Place at = place_of(rope, tid % L, !values);
  u32x4_t w[PASSES][2];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * R + tid / L;
    const bool in = r >= r0 && r < r1;
    const uint16_t* row = x + (int64_t)(tok0 + r) * stride + head * D;
    w[i][0] = w[i][1] = u32x4_t{0, 0, 0, 0};
    if (in) w[i][0] = *(const u32x4_t*)(row + at.a), w[i][1] = *(const u32x4_t*)(row + at.b);
  }
  float f[PASSES][16];
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    widen16x<DT>(w[i][0], w[i][1], f[i]);
    if (at.turned)
      rotate(f[i], angles_of(rope, at, (p << c.lgT) + i * R + tid / L), rope.interleaved);
    mag = max(mag, mag16(f[i]));
  }
  mag = lanes_max<64>(mag);
  if ((tid & 63) == 0) part[tid >> 6] = mag;
  const float old = r0 > 0 ? *scale : 0.0f;
  __syncthreads();  // (every lane has read the old scale, too)
  mag = max(max(part[0], part[1]), max(part[2], part[3]));
  const float s = grown_scale(old, mag);
  const bool grew = r0 > 0 && s != old;
  const float ratio = s > 0.0f ? old / s : 0.0f;
  if (tid == 0) *scale = s;

  const Codes8 codes(s);
  if (!values) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * R + tid / L;
      if (r >= r0 && r < r1) {
        *(u32x2_t*)(dst + r * D + at.a) = stored8(f[i], codes);
        *(u32x2_t*)(dst + r * D + at.b) = stored8(f[i] + 8, codes);
      }
    }
    if (grew)
      for (int i = tid * 16; i < r0 * D; i += 256 * 16)
        *(u32x4_t*)(dst + i) = requantized(*(const u32x4_t*)(dst + i), ratio);
    return;
  }
  // values: the codes turn in LDS to [T / 16][D][16], then every 16-token
  // piece that holds new rows (or requantized ones) is written whole, its
  // other bytes as they were
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * R + tid / L;
    if (r < T) {
      uint8_t* to = lds + ((r >> 4) * D + at.a) * 16 + (r & 15);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const u32x2_t v = stored8(f[i] + 8 * e, codes);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          to[(8 * e + j) * 16] = (uint8_t)(v[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
  __syncthreads();
  const int sub0 = grew ? 0 : r0 >> 4, sub1 = (r1 + 15) >> 4;
  for (int i = sub0 * D + tid; i < sub1 * D; i += 256) {
    const int t0 = (i / D) * 16;
    u32x4_t v = *(const u32x4_t*)(lds + i * 16);
    if (t0 < r0 || t0 + 16 > r1) {
      const u32x4_t was = *(const u32x4_t*)(dst + i * 16);
      const u32x4_t again = grew ? requantized(was, ratio) : was;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int t = t0 + j;
        const uint32_t m = 0xFFu << (8 * (j & 3));
        const uint32_t from = t < r0 ? again[j >> 2] : t < r1 ? v[j >> 2] : was[j >> 2];
        v[j >> 2] = (v[j >> 2] & ~m) | (from & m);
      }
    }
    *(u32x4_t*)(dst + i * 16) = v;
  }
}

template <int DT, int D, int PASSES>
__global__ void __launch_bounds__(256)
kv8_append_kernel(Kv8 c, Rope rope, const uint16_t* q, int64_t q_stride,
                  uint16_t* q_out, int64_t qo_stride, const uint16_t* __restrict__ k,
                  int64_t k_stride, const uint16_t* __restrict__ v, int64_t v_stride,
                  int64_t blocks) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[PASSES * 4096];
  __shared__ uint32_t part[4];
  const int64_t id = blockIdx.x;
  if (id >= blocks) {
    turn_queries<DT, D>(c, rope, q, q_stride, q_out, qo_stride, (int)(id - blocks));
    return;
  }
  const bool values = id & 1;
  const int64_t j = id >> 1;
  const int head = (int)(j % c.Hkv), place = (int)(j / c.Hkv);
  const int b = __builtin_amdgcn_readfirstlane(sequence_at(c, place));
  const int chunk = max(place - pages_before(c, b), 0);
  append_page<DT, D, PASSES>(c, rope, values ? v : k, values ? v_stride : k_stride, values, b,
                             chunk, head, lds, part);
}

// One new token for each sequence: D / 16 lanes per (sequence, kv head, keys or
// values).  A page whose scale grew is requantized by the whole wave.
//
// A call is a chain of short loads (length, table, scale, page) and bound by
// their latency: 256 sequences, 8 kv heads of 128, 7 us (with its read-back 30;
// 65 with a workgroup per page and head as above, most of its lanes idle).
template <int DT, int D>
__global__ void __launch_bounds__(256)
kv8_append_token_kernel(Kv8 c, Rope rope, const uint16_t* q, int64_t q_stride,
                        uint16_t* q_out, int64_t qo_stride, const uint16_t* __restrict__ k,
                        int64_t k_stride, const uint16_t* __restrict__ v, int64_t v_stride,
                        int64_t blocks) {
  constexpr int L = D / 16, R = 256 / L;
  const int64_t id = blockIdx.x;
  if (id >= blocks) {
    turn_queries<DT, D>(c, rope, q, q_stride, q_out, qo_stride, (int)(id - blocks));
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t row = id * R + threadIdx.x / L;
  const bool values = row & 1;
  const int head = (int)((row >> 1) % c.Hkv);
  const int64_t bq = (row >> 1) / c.Hkv;
  const int b = (int)min(bq, (int64_t)c.B - 1);
  const Kv8Seq sq = kv8_seq(c, b);
  const bool on = bq < c.B && sq.first >= 0 && sq.n > 0;
  const int T = 1 << c.lgT, pos = max(sq.first, 0), r0 = pos & (T - 1);
  const int tok = sq.tok;
  const Place at = place_of(rope, threadIdx.x % L, !values);
  const uint16_t* x = (values ? v + (int64_t)tok * v_stride : k + (int64_t)tok * k_stride) + head * D;
  u32x4_t w0 = {0, 0, 0, 0}, w1 = {0, 0, 0, 0};
  if (on) w0 = *(const u32x4_t*)(x + at.a), w1 = *(const u32x4_t*)(x + at.b);
  const int64_t slot = (int64_t)kv8_page(c, b, pos >> c.lgT) * c.Hkv + head;
  float* scale = (values ? c.vs : c.ks) + slot;
  const float old = on && r0 > 0 ? *scale : 0.0f;
  float f[16];
  widen16x<DT>(w0, w1, f);
  if (at.turned) rotate(f, angles_of(rope, at, pos), rope.interleaved);
  const float s = grown_scale(old, lanes_max<L>(mag16(f)));
  uint8_t* dst = (values ? c.v : c.k) + slot * ((int64_t)T * D);
  const bool grew = on && r0 > 0 && s != old;
  const float ratio = s > 0.0f ? old / s : 0.0f;
  uint64_t todo = __ballot(grew && lane % L == 0);
  if (todo) {
    do {
      const int from = __builtin_ctzll(todo);
      todo &= todo - 1;
      const int rows = __builtin_amdgcn_readlane(r0, from);
      const float rt = __builtin_bit_cast(
          float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, ratio), from));
      const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uintptr_t)dst, from) |
                            (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)((uintptr_t)dst >> 32), from) << 32;
      const bool vals = __builtin_amdgcn_readlane(values, from);
      uint8_t* page = (uint8_t*)base;
      const int bytes = (vals ? (rows + 15) & ~15 : rows) * D;
      for (int i = lane * 16; i < bytes; i += 1024) {
        const u32x4_t was = *(const u32x4_t*)(page + i);
        u32x4_t now = requantized(was, rt);
        const int keep = vals ? rows - i / (16 * D) * 16 : 16;  // older rows of the piece
        if (keep < 16) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const uint32_t m = 0xFFu << (8 * (j & 3));
            if (j >= keep) now[j >> 2] = (now[j >> 2] & ~m) | (was[j >> 2] & m);
          }
        }
        *(u32x4_t*)(page + i) = now;
      }
    } while (todo);
    // the pieces are written before single bytes of them are
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  if (!on) return;
  const Codes8 codes(s);
  const u32x2_t ca = stored8(f, codes), cb = stored8(f + 8, codes);
  if (threadIdx.x % L == 0) *scale = s;
  if (!values) {
    *(u32x2_t*)(dst + r0 * D + at.a) = ca;
    *(u32x2_t*)(dst + r0 * D + at.b) = cb;
  } else {
    uint8_t* to = dst + ((r0 >> 4) * D + at.a) * 16 + (r0 & 15);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      to[j * 16] = (uint8_t)(ca[j >> 2] >> (8 * (j & 3)));
      to[(8 + j) * 16] = (uint8_t)(cb[j >> 2] >> (8 * (j & 3)));
    }
  }
}

// The fp32 product of a code and its scale, rounded to fp32 before it is
// rounded to 16 bits (the empty statement keeps the compiler from making one
// fused multiply-and-convert of the two).
template <int DT>
__device__ __forceinline__ uint32_t value16(uint32_t c, float s) {
  float f = (float)((int)(c & 0xFFu) - 128) * s;
  asm("" : "+v"(f));
  return round16<DT>(f);
}

// Pages read back as [n, Hkv, T, D] in 16 bits.  Keys: a lane turns 16 bytes,
// 16 channels of a token.  Values: a lane turns 8 channels of 16 tokens, whose
// codes are 128 consecutive bytes, and writes 16 bytes of each token.  Bound by
// its bytes, 2 of 3 of them written (MI355X, the pages of 17 k tokens, 8 heads of
// 128: 30.5 us for some 105 MB).
template <int DT>
__global__ void __launch_bounds__(256)
kv8_dequant_kernel(const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
                   const float* __restrict__ ks, const float* __restrict__ vs,
                   const int32_t* __restrict__ pages, int num_pages, int Hkv, int T, int D,
                   int64_t heads, int64_t k_blocks, uint16_t* __restrict__ k_out,
                   uint16_t* __restrict__ v_out) {
  const bool values = blockIdx.x >= k_blocks;
  const int per = values ? T * D / 128 : T * D / 16;  // lanes per (page, head)
  const int64_t at = (int64_t)(blockIdx.x - (values ? k_blocks : 0)) * 256 + threadIdx.x;
  const int64_t ph = at / per;
  const int i = (int)(at - ph * per);
  if (ph >= heads) return;
  const int64_t slot =
      (int64_t)clamp_int(pages[ph / Hkv], 0, num_pages - 1) * Hkv + (int)(ph % Hkv);
  const int64_t src = slot * T * D, dst = ph * T * D;
  if (!values) {
    const float s = ks[slot];
    const u32x4_t w = *(const u32x4_t*)(k + src + i * 16);
    u32x4_t r[2];
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const uint32_t two = w[j >> 2] >> (8 * (j & 3));
      r[j >> 3][(j >> 1) & 3] = value16<DT>(two, s) | value16<DT>(two >> 8, s) << 16;
    }
    *(u32x4_t*)(k_out + dst + i * 16) = r[0];
    *(u32x4_t*)(k_out + dst + i * 16 + 8) = r[1];
    return;
  }
  const float s = vs[slot];
  const int sub = i / (D / 8), d = i % (D / 8) * 8;
  u32x4_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = *(const u32x4_t*)(v + src + (sub * D + d + j) * 16);
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    u32x4_t r;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      r[j] = value16<DT>(w[2 * j][t >> 2] >> (8 * (t & 3)), s) |
             value16<DT>(w[2 * j + 1][t >> 2] >> (8 * (t & 3)), s) << 16;
    *(u32x4_t*)(v_out + dst + (sub * 16 + t) * D + d) = r;
  }
}

template <int DT, int D, int PASSES>
void launch_append_p(const Kv8& c, const Rope& rope, const void* q, int64_t q_stride, void* q_out,
                     int64_t qo_stride, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, int64_t blocks, int64_t qblocks, hipStream_t st) {
  hipLaunchKernelGGL((kv8_append_kernel<DT, D, PASSES>), dim3((unsigned)(blocks + qblocks)),
                     dim3(256), 0, st, c, rope, (const uint16_t*)q, q_stride, (uint16_t*)q_out,
                     qo_stride, (const uint16_t*)k, k_stride, (const uint16_t*)v, v_stride,
                     blocks);
}

// Workgroups of an append (those that turn queries aside).  The places of pages
// go by all new tokens, not by the largest number in a sequence: 256 sequences
// with a few long ones among them have some B places and not B times the longest.
int64_t append_blocks(int64_t tokens, int64_t B, int64_t T, int Hkv, int D, int64_t max_new) {
  return max_new == 1 ? ceil_div(B * Hkv * 2, 256 / (D / 16)) : (tokens / T + 2 * B) * Hkv * 2;
}

template <int DT>
hipError_t launch_append(const Kv8& c, const Rope& rope, int D, const void* q, int64_t q_stride,
                         void* q_out, int64_t qo_stride, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, int64_t max_new, hipStream_t st) {
#define W4A16_APPEND(DD, P)                                                                    \
  launch_append_p<DT, DD, P>(c, rope, q, q_stride, q_out, qo_stride, k, k_stride, v, v_stride, \
                             blocks, qblocks, st)
  const int T = 1 << c.lgT;
  const int64_t blocks = append_blocks(c.tokens, c.B, T, c.Hkv, D, max_new);
  const int64_t qblocks = q ? c.tokens : 0;
  if (max_new == 1) {
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks + qblocks)), dim3(256), 0, st, c, rope,
                         (const uint16_t*)q, q_stride, (uint16_t*)q_out, qo_stride,
                         (const uint16_t*)k, k_stride, (const uint16_t*)v, v_stride, blocks);
    };
    if (D == 64) go(kv8_append_token_kernel<DT, 64>);
    else go(kv8_append_token_kernel<DT, 128>);
  } else if (D == 64) {
    if (T <= 64) W4A16_APPEND(64, 1);
    else W4A16_APPEND(64, 2);
  } else {
    if (T <= 32) W4A16_APPEND(128, 1);
    else if (T == 64) W4A16_APPEND(128, 2);
    else W4A16_APPEND(128, 4);
  }
#undef W4A16_APPEND
  return hipGetLastError();
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int kv8_append(const void* q, int64_t q_stride, void* q_out, int64_t q_out_stride, const void* k,
               int64_t k_stride, const void* v, int64_t v_stride, uint8_t* k_cache,
               uint8_t* v_cache, float* k_scale, float* v_scale, int64_t num_pages,
               int32_t page_size, const int32_t* page_table, int64_t max_pages,
               const int32_t* seq_lens, const int32_t* cu_seqlens, const float* cos,
               const float* sin, int64_t rope_rows, int32_t rope_dim, int32_t interleaved,
               int64_t tokens, int64_t B, int64_t max_new, int32_t H, int32_t Hkv, int32_t D,
               int32_t dtype, void* stream) {
  return guarded([&]() -> int {
    if (int s = validate_kv8(num_pages, page_size, max_pages, tokens, B, max_new, H, Hkv, D,
                             cu_seqlens))
      return s;
    if (int s = validate_dtype(dtype)) return s;
    if ((q == nullptr) != (q_out == nullptr) || (cos == nullptr) != (sin == nullptr))
      return W4A16_ERR_INVALID_ARG;
    if (cos) {
      if (rope_rows <= 0 || rope_rows > (1 << 30) || rope_dim <= 0 || rope_dim > D ||
          rope_dim % 16 != 0)
        return W4A16_ERR_INVALID_ARG;
    }
    if (bad_stride(k_stride, (int64_t)Hkv * D) || bad_stride(v_stride, (int64_t)Hkv * D))
      return W4A16_ERR_INVALID_ARG;
    if (q && (bad_stride(q_stride, (int64_t)H * D) || bad_stride(q_out_stride, (int64_t)H * D)))
      return W4A16_ERR_INVALID_ARG;
    if (tokens == 0 || B == 0 || max_new == 0) return W4A16_OK;
    if (int s = check_ptrs({k, v, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens}))
      return s;
    for (const void* p : {q, (const void*)q_out, (const void*)cu_seqlens, (const void*)cos,
                          (const void*)sin})
      if (!aligned16(p)) return W4A16_ERR_MISALIGNED;
    if (too_large(append_blocks(tokens, B, page_size, Hkv, D, max_new) + (q ? tokens : 0), 256))
      return W4A16_ERR_UNSUPPORTED;
    clear_pending_error();
    const Kv8 c = {k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_seqlens,
                   (int)num_pages, (int)max_pages, (int)B, (int)tokens, (int)max_new, H, Hkv,
                   log2_page(page_size)};
    const Rope rope = {cos, sin, (int)rope_rows, rope_dim, interleaved};
    return hip_status((dtype == DT_F16 ? launch_append<DT_F16> : launch_append<DT_BF16>)(
        c, rope, D, q, q_stride, q_out, q_out_stride, k, k_stride, v, v_stride, max_new,
        (hipStream_t)stream));
  });
}

int kv8_dequant(const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                const float* v_scale, int64_t num_pages, int32_t page_size, int32_t Hkv,
                int32_t D, const int32_t* pages, int64_t n, int32_t dtype, void* k_out,
                void* v_out, void* stream) {
  return guarded([&]() -> int {
    if (int s = validate_kv8(num_pages, page_size, 1, 0, 0, 0, Hkv, Hkv, D, nullptr)) return s;
    if (int s = validate_dtype(dtype)) return s;
    if (n < 0) return W4A16_ERR_INVALID_ARG;
    if (n > (1 << 30)) return W4A16_ERR_UNSUPPORTED;
    if (n == 0) return W4A16_OK;
    if (int s = check_ptrs({k_cache, v_cache, k_scale, v_scale, pages, k_out, v_out})) return s;
    clear_pending_error();
    const int64_t heads = n * Hkv, per = (int64_t)page_size * D;
    const int64_t k_blocks = ceil_div(heads * (per / 16), 256);
    const int64_t blocks = k_blocks + ceil_div(heads * (per / 128), 256);
    if (too_large(blocks, 256)) return W4A16_ERR_UNSUPPORTED;
    const dim3 g((unsigned)blocks), b(256);
    const hipStream_t st = (hipStream_t)stream;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, g, b, 0, st, k_cache, v_cache, k_scale, v_scale, pages,
                         (int)num_pages, Hkv, page_size, D, heads, k_blocks, (uint16_t*)k_out,
                         (uint16_t*)v_out);
    };
    if (dtype == DT_F16) go(kv8_dequant_kernel<DT_F16>);
    else go(kv8_dequant_kernel<DT_BF16>);
    return hip_status(hipGetLastError());
  });
}

}  // extern "C"
