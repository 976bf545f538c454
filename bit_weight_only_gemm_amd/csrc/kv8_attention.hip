// kv8_attention.hip -- attention of 16-bit queries over the paged 8-bit cache:
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
#include "kv8.h"
#include "launch.h"

namespace w4a16 {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kUnit = 64;  // tokens a wave takes at a time

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

// Query rows of a (sequence, kv head): row i is token i / G, head i % G.  A
// row tile is 16 of them; it sees keys up to the largest limit of its rows.
__device__ __forceinline__ int row_limit(const Kv8Seq& s, int causal, int j) {
  return causal ? clamp_int(s.len - s.n + j + 1, 0, s.len) : s.len;
}
__device__ __forceinline__ int tile_limit(const Kv8Seq& s, int causal, int rt, int G) {
  return row_limit(s, causal, min((rt * 16 + 15) / G, s.n - 1));
}

// Partial results of a split: O [row][split][D], then (m, l) [row][split],
// row = token * H + head.
struct Parts {
  float* o;
  float* ml;
};

// One workgroup of 4 waves per (sequence, kv head, row tile, split of the
// keys); its waves take units of 64 tokens in turn and are joined in LDS.
// Scores come out as S^T (16 tokens x 16 rows): lane l holds row l & 15 and
// tokens 16 g + 4 a + i (g = l >> 4) of the unit in register i of product a,
// which is the operand layout of the second product: neither keys, values
// nor probabilities pass through LDS.
template <int DT, int D>
__global__ void __launch_bounds__(256)
kv8_decode_kernel(Kv8 c, const uint16_t* __restrict__ q, int64_t q_stride, float scale, int causal,
                  uint16_t* __restrict__ out, int64_t out_stride, float* __restrict__ lse,
                  Parts parts, int row_tiles, int splits, int units) {
  constexpr int DC = D / 64, DN = D / 16;
  __shared__ float joined[4][16][D + 4];
  __shared__ float stat[4][2][16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;
  int id = blockIdx.x;
  const int split = id % splits;
  id /= splits;
  const int rt = id % row_tiles;
  id /= row_tiles;
  const int hk = id % c.Hkv, b = id / c.Hkv;
  const int G = c.H / c.Hkv;
  const Kv8Seq seq = kv8_seq(c, b);
  if (rt * 16 >= seq.n * G) return;
  const int top = tile_limit(seq, causal, rt, G);
  const int nu = (top + kUnit - 1) / kUnit;
  const int u0 = split * units, u1 = min(u0 + units, nu);
  if (split > 0 && u0 >= nu) return;

  const int ridx = rt * 16 + col;
  const bool rv = ridx < seq.n * G;
  const int tok = seq.tok + (rv ? ridx / G : 0), head = hk * G + (rv ? ridx % G : 0);
  const int lim = rv ? row_limit(seq, causal, ridx / G) : 0;

  // ---- queries: channels 64 c + 16 g + 8 e .. + 7 of this lane's row
  half8_t qf[DC][2];
  float rowscale = scale * kLog2e;
  {
    const uint16_t* qp = q + (int64_t)tok * q_stride + head * D + 16 * g;
    u32x4_t w[DC][2];
#pragma unroll
    for (int i = 0; i < DC; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        w[i][e] = u32x4_t{0, 0, 0, 0};
        if (rv) w[i][e] = *(const u32x4_t*)(qp + 64 * i + 8 * e);
      }
    if constexpr (DT == DT_F16) {
#pragma unroll
      for (int i = 0; i < DC; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) qf[i][e] = __builtin_bit_cast(half8_t, w[i][e]);
    } else {
      uint32_t mag = 0;
      float f[DC][2][8];
#pragma unroll
      for (int i = 0; i < DC; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          widen8<DT>(w[i][e], f[i][e]);
#pragma unroll
          for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(f[i][e][j]));
        }
      mag = max(mag, (uint32_t)__shfl_xor((int)mag, 16, 64));
      mag = max(mag, (uint32_t)__shfl_xor((int)mag, 32, 64));
      // exponent of the row's largest magnitude; 2^(14 - e) brings it to
      // [2^14, 2^15), held to the normal fp32 range
      const int e2 = clamp_int((int)(mag >> 23) - 127, -100, 126);
      const float up = __builtin_bit_cast(float, (uint32_t)(127 + 14 - e2) << 23);
      rowscale *= __builtin_bit_cast(float, (uint32_t)(127 - 14 + e2) << 23);
#pragma unroll
      for (int i = 0; i < DC; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < 8; ++j) qf[i][e][j] = (_Float16)(f[i][e][j] * up);
    }
  }

  float m = -INFINITY, l = 0.0f;
  float4_t o[DN];
#pragma unroll
  for (int i = 0; i < DN; ++i) o[i] = float4_t{};

  const int64_t page_bytes = (int64_t)D << c.lgT;
  auto subtile = [&](int t) -> int64_t {  // of the 16 tokens at t
    const int page = kv8_page(c, b, min(t >> c.lgT, c.width - 1));
    return ((int64_t)page * c.Hkv + hk) * page_bytes + (int64_t)(t & ((1 << c.lgT) - 1)) * D;
  };
  for (int u = u0 + wave; u < u1; u += 4) {
    const int t0 = u * kUnit;
    const uint8_t* kp = c.k + subtile(t0 + 16 * (col >> 2)) + (col & 3) * D + 16 * g;
    const uint8_t* vp = c.v + subtile(t0 + 16 * g) + col * 16;
    const int pg = kv8_page(c, b, min((t0 + 16 * g) >> c.lgT, c.width - 1));
    const bool held = t0 + 16 * g < seq.len;  // else the page may be no page of this sequence
    const float ks = held ? c.ks[(int64_t)pg * c.Hkv + hk] : 0.0f;
    const float vs = held ? c.vs[(int64_t)pg * c.Hkv + hk] : 0.0f;
    u32x4_t kw[4][DC], vw[DN];
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < DC; ++i) kw[a][i] = *(const u32x4_t*)(kp + a * 4 * D + 64 * i);
#pragma unroll
    for (int i = 0; i < DN; ++i) vw[i] = *(const u32x4_t*)(vp + i * 256);

    float s[4][4], mx = -INFINITY;
    const float f = rowscale * ks;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      float4_t acc{};
#pragma unroll
      for (int i = 0; i < DC; ++i) {
        acc = mfma16x16x32<DT_F16>(codes_f16(kw[a][i][0], kw[a][i][1]), qf[i][0], acc);
        acc = mfma16x16x32<DT_F16>(codes_f16(kw[a][i][2], kw[a][i][3]), qf[i][1], acc);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[a][i] = t0 + 16 * g + 4 * a + i < lim ? acc[i] * f : -INFINITY;
        mx = fmaxf(mx, s[a][i]);
      }
    }
    mx = fmaxf(mx, __shfl_xor(mx, 16, 64));
    mx = fmaxf(mx, __shfl_xor(mx, 32, 64));
    const float mn = fmaxf(m, mx), ms = mn == -INFINITY ? 0.0f : mn;
    const float alpha = __builtin_amdgcn_exp2f(m - ms);
    m = mn;
    // the values' scales of the unit's pages, relative to the largest
    float top_v = fmaxf(vs, __shfl_xor(vs, 16, 64));
    top_v = fmaxf(top_v, __shfl_xor(top_v, 32, 64));
    const float rel = top_v > 0.0f ? vs / top_v : (vs == 0.0f ? 1.0f : vs);
    half8_t pf[2];
    float sum = 0.0f;
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = __builtin_amdgcn_exp2f(s[a][i] - ms);
        sum += p;
        pf[a >> 1][4 * (a & 1) + i] = (_Float16)(p * rel);
      }
    l = l * alpha + sum;
#pragma unroll
    for (int i = 0; i < DN; ++i) {
      float4_t acc{};
      acc = mfma16x16x32<DT_F16>(codes_f16(vw[i][0], vw[i][1]), pf[0], acc);
      acc = mfma16x16x32<DT_F16>(codes_f16(vw[i][2], vw[i][3]), pf[1], acc);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = __builtin_fmaf(acc[j], top_v, o[i][j] * alpha);
    }
  }
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);

  // ---- join the waves: lane holds channels 16 i + 4 g + j of row col
#pragma unroll
  for (int i = 0; i < DN; ++i) *(float4_t*)&joined[wave][col][16 * i + 4 * g] = o[i];
  if (g == 0) {
    stat[wave][0][col] = m;
    stat[wave][1][col] = l;
  }
  __syncthreads();
  // 16 lanes per row
  const int row = tid >> 4, part = tid & 15;
  const int rr = rt * 16 + row;
  if (rr >= seq.n * G) return;
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
  constexpr int E = D / 16;  // channels per lane
  float r[E];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    r[j] = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) r[j] += wt[w] * joined[w][row][part * E + j];
  }
  const int64_t tk = seq.tok + rr / G;
  const int hd = hk * G + rr % G;
  if (splits > 1) {
    const int64_t at = (tk * c.H + hd) * splits + split;
#pragma unroll
    for (int j = 0; j < E; ++j) parts.o[at * D + part * E + j] = r[j];
    if (part == 0) {
      parts.ml[at * 2] = mm;
      parts.ml[at * 2 + 1] = ll;
    }
    return;
  }
  const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;  // a row that sees nothing is 0
#pragma unroll
  for (int j = 0; j < E; ++j)
    out[tk * out_stride + hd * D + part * E + j] = round16<DT>(r[j] * inv);
  if (lse && part == 0)
    lse[tk * c.H + hd] = ll == 0.0f ? -INFINITY : (mm + __log2f(ll)) * kLn2;
}

// Joins the splits of a row, in their order: one wave per (token, head).
template <int DT, int D>
__global__ void __launch_bounds__(256)
kv8_join_kernel(Kv8 c, int causal, uint16_t* __restrict__ out, int64_t out_stride,
                float* __restrict__ lse, Parts parts, int splits, int units, int max_new) {
  const int lane = threadIdx.x & 63;
  const int G = c.H / c.Hkv;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= (int64_t)c.B * max_new * c.H) return;
  const int hd = (int)(i % c.H), j = (int)(i / c.H % max_new), b = (int)(i / c.H / max_new);
  const Kv8Seq seq = kv8_seq(c, b);
  if (j >= seq.n) return;
  const int top = tile_limit(seq, causal, (j * G + hd % G) / 16, G);
  const int nu = (top + kUnit - 1) / kUnit;
  const int n = clamp_int((nu + units - 1) / units, 1, splits);
  const int64_t row = (int64_t)(seq.tok + j) * c.H + hd;
  float m = -INFINITY;
  for (int s = 0; s < n; ++s) m = fmaxf(m, parts.ml[(row * splits + s) * 2]);
  const float base = m == -INFINITY ? 0.0f : m;
  constexpr int E = D / 64;
  float l = 0.0f, r[E] = {};
  for (int s = 0; s < n; ++s) {
    const int64_t at = row * splits + s;
    const float w = __builtin_amdgcn_exp2f(parts.ml[at * 2] - base);
    l += w * parts.ml[at * 2 + 1];
#pragma unroll
    for (int e = 0; e < E; ++e) r[e] += w * parts.o[at * D + lane * E + e];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int e = 0; e < E; ++e)
    out[(seq.tok + j) * out_stride + hd * D + lane * E + e] = round16<DT>(r[e] * inv);
  if (lse && lane == 0) lse[row] = l == 0.0f ? -INFINITY : (m + __log2f(l)) * kLn2;
}

struct Plan {
  int row_tiles, splits, units;
};

// Splits of the keys: enough workgroups to fill 256 CUs twice, no split below
// 4 units (one per wave).
Plan plan_attention(int64_t B, int64_t max_new, int64_t max_len, int H, int Hkv) {
  Plan p;
  p.row_tiles = (int)ceil_div(max_new * (H / Hkv), 16);
  const int64_t nu = std::max<int64_t>(1, ceil_div(max_len, kUnit));
  const int64_t groups = B * Hkv * p.row_tiles;
  const int64_t want = std::max<int64_t>(1, ceil_div(1024, groups));
  p.units = (int)std::max<int64_t>(4, ceil_div(nu, want));
  p.splits = (int)ceil_div(nu, p.units);
  return p;
}

int64_t pad256(int64_t b) { return ceil_div(b, 256) * 256; }

int64_t part_bytes(const Plan& p, int64_t tokens, int H, int D) {
  if (p.splits == 1) return 0;
  const int64_t rows = tokens * H * p.splits;
  return pad256(rows * D * 4) + pad256(rows * 8);
}

template <int DT, int D>
hipError_t launch_attention(const Kv8& c, const Plan& p, const void* q, int64_t q_stride,
                            float scale, int causal, void* out, int64_t out_stride, float* lse,
                            int64_t max_new, void* ws, hipStream_t st) {
  Parts parts = {(float*)ws, nullptr};
  parts.ml = parts.o + pad256((int64_t)c.tokens * c.H * p.splits * D * 4) / 4;
  const int64_t grid = (int64_t)c.B * c.Hkv * p.row_tiles * p.splits;
  launch_timed(kv8_decode_kernel<DT, D>, dim3((unsigned)grid), dim3(256), 0, st, c,
               (const uint16_t*)q, q_stride, scale, causal, (uint16_t*)out, out_stride, lse,
               parts, p.row_tiles, p.splits, p.units);
  if (p.splits > 1)
    hipLaunchKernelGGL((kv8_join_kernel<DT, D>),
                       dim3((unsigned)ceil_div((int64_t)c.B * max_new * c.H, 4)), dim3(256), 0,
                       st, c, causal, (uint16_t*)out, out_stride, lse, parts, p.splits, p.units,
                       (int)max_new);
  return hipGetLastError();
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int64_t kv8_attention_workspace_bytes(int64_t tokens, int64_t B, int64_t max_new, int64_t max_len,
                                      int32_t H, int32_t Hkv, int32_t D) {
  if (validate_kv8(1, 64, 1, tokens, B, max_new, H, Hkv, D, &tokens) != W4A16_OK || max_len < 0 ||
      max_len > ((int64_t)1 << 30))
    return -1;
  if (tokens == 0 || B == 0 || max_new == 0) return 0;
  return part_bytes(plan_attention(B, max_new, max_len, H, Hkv), tokens, H, D);
}

int kv8_attention(const void* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                  const float* k_scale, const float* v_scale, int64_t num_pages,
                  int32_t page_size, const int32_t* page_table, int64_t max_pages,
                  const int32_t* seq_lens, const int32_t* cu_seqlens, float scale, int32_t causal,
                  void* out, int64_t out_stride, float* lse, int64_t tokens, int64_t B,
                  int64_t max_new, int64_t max_len, int32_t H, int32_t Hkv, int32_t D,
                  int32_t dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    if (int s = validate_kv8(num_pages, page_size, max_pages, tokens, B, max_new, H, Hkv, D,
                             cu_seqlens))
      return s;
    if (int s = validate_dtype(dtype)) return s;
    if (max_len < 0 || max_len > max_pages * page_size) return W4A16_ERR_INVALID_ARG;
    if (bad_stride(q_stride, (int64_t)H * D) || bad_stride(out_stride, (int64_t)H * D))
      return W4A16_ERR_INVALID_ARG;
    if (tokens == 0 || B == 0 || max_new == 0) return W4A16_OK;
    if (int s = check_ptrs({q, k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, out}))
      return s;
    for (const void* p : {(const void*)cu_seqlens, (const void*)lse, (const void*)workspace})
      if (!aligned16(p)) return W4A16_ERR_MISALIGNED;
    const Plan p = plan_attention(B, max_new, max_len, H, Hkv);
    const int64_t need = part_bytes(p, tokens, H, D);
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
    if (B * Hkv * p.row_tiles * p.splits > ((int64_t)1 << 31) - 1 ||
        B * max_new * H > ((int64_t)1 << 32))
      return W4A16_ERR_UNSUPPORTED;
    clear_pending_error();
    const Kv8 c = {const_cast<uint8_t*>(k_cache), const_cast<uint8_t*>(v_cache),
                   const_cast<float*>(k_scale), const_cast<float*>(v_scale), page_table, seq_lens,
                   cu_seqlens, (int)num_pages, (int)max_pages, (int)B, (int)tokens, H, Hkv,
                   log2_page(page_size)};
    auto* f = D == 64 ? (dtype == DT_F16 ? launch_attention<DT_F16, 64>
                                         : launch_attention<DT_BF16, 64>)
                      : (dtype == DT_F16 ? launch_attention<DT_F16, 128>
                                         : launch_attention<DT_BF16, 128>);
    return hip_status(f(c, p, q, q_stride, scale, causal, out, out_stride, lse, max_new, workspace,
                        (hipStream_t)stream));
  });
}

}  // extern "C"
