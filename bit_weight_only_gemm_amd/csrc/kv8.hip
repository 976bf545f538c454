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

// Rotates 8 consecutive channels d0 .. d0 + 7 of a row, held by the D / 8
// lanes of a group in channel order: pair (a, b) becomes (a cos - b sin,
// b cos + a sin), products and sums in fp32, each rounded once.  Half-split
// pairs are channels (i, i + dim / 2), the partner's 8 channels lying with
// the lane dim / 16 further or before; interleaved pairs are (2 i, 2 i + 1).
// Channels at and past dim pass through.  All lanes of a wave take part.
__device__ __forceinline__ void rotate8(float (&x)[8], const Rope& r, int pos, int d0) {
  if (!r.cos) return;
  const int half = r.dim >> 1, lane = threadIdx.x & 63;
  const int64_t row = (int64_t)clamp_int(pos, 0, r.rows - 1) * half;
  if (r.interleaved) {
    if (d0 >= r.dim) return;
    const float4_t c = *(const float4_t*)(r.cos + row + d0 / 2);
    const float4_t s = *(const float4_t*)(r.sin + row + d0 / 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * s[i];
      x[2 * i + 1] = b * c[i] + a * s[i];
    }
    return;
  }
  const bool first = d0 < half, turned = d0 < r.dim;
  const int from = !turned ? lane : first ? lane + (half >> 3) : lane - (half >> 3);
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __shfl(x[i], from, 64);
  if (!turned) return;
  const int64_t at = row + (first ? d0 : d0 - half);
  float c[8], s[8];
  *(float4_t*)c = *(const float4_t*)(r.cos + at);
  *(float4_t*)(c + 4) = *(const float4_t*)(r.cos + at + 4);
  *(float4_t*)s = *(const float4_t*)(r.sin + at);
  *(float4_t*)(s + 4) = *(const float4_t*)(r.sin + at + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float u = x[i] * c[i], w = y[i] * s[i];
    x[i] = first ? u - w : u + w;
  }
}

// 16 stored codes requantized to a scale `ratio` = old / new times as fine;
// only the bytes of tokens in [0, keep) change when `tokens`, else all.
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

// One workgroup per (sequence, touched page, kv head, keys or values), the
// only one to touch those bytes and that scale.  The new rows are read once
// and kept, rotated, in registers; the page's scale is the larger of the old
// one (none if the page begins with this call's rows) and the new rows' own;
// where it grew, the page's older rows are requantized to it.
// PASSES: ceil(T D / 8 / 256) rows of lanes.
template <int DT, int D, int PASSES>
__device__ void append_page(const Kv8& c, const Rope& rope, const uint16_t* x, int64_t stride,
                            bool values, int b, int chunk, int head, uint8_t* lds,
                            uint32_t* part) {
  const Kv8Seq q = kv8_seq(c, b);
  const int T = 1 << c.lgT, start = max(q.len - q.n, 0);
  const int p = (start >> c.lgT) + chunk;
  if (q.len == 0 || (p << c.lgT) >= q.len || q.n == 0) return;
  const int r0 = max(start - (p << c.lgT), 0), r1 = min(q.len - (p << c.lgT), T);
  const int tok0 = q.tok + q.n - (q.len - (p << c.lgT));  // new token of the page's row 0
  const int page = kv8_page(c, b, p);
  const int64_t slot = (int64_t)page * c.Hkv + head;
  uint8_t* dst = (values ? c.v : c.k) + slot * ((int64_t)T * D);
  float* scale = (values ? c.vs : c.ks) + slot;

  constexpr int L = D / 8;      // lanes per row
  constexpr int R = 256 / L;    // rows per pass
  const int tid = threadIdx.x, d0 = (tid % L) * 8;
  float f[PASSES][8];
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * R + tid / L;
    const bool in = r >= r0 && r < r1;
    u32x4_t w = {0, 0, 0, 0};
    if (in) w = *(const u32x4_t*)(x + (int64_t)(tok0 + r) * stride + head * D + d0);
    widen8<DT>(w, f[i]);
    if (!values) rotate8(f[i], rope, (p << c.lgT) + r, d0);
#pragma unroll
    for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(f[i][j]));
  }
  mag = lanes_max<64>(mag);
  if ((tid & 63) == 0) part[tid >> 6] = mag;
  __syncthreads();
  mag = max(max(part[0], part[1]), max(part[2], part[3]));
  const float old = r0 > 0 ? *scale : 0.0f, fresh = scale_of(mag);
  // a scale that is NaN stays NaN while its page holds older rows
  const float s = old != old || fresh != fresh ? __builtin_nanf("") : fmaxf(old, fresh);
  const bool grew = r0 > 0 && s != old;
  const float ratio = s > 0.0f ? old / s : 0.0f;
  __syncthreads();  // every lane has read the old scale
  if (tid == 0) *scale = s;

  auto codes = [&](const float (&g)[8]) {
    u32x2_t r = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      r[j >> 2] |= (uint32_t)((s == 0.0f ? 0 : code_of(g[j], s)) + 128) << (8 * (j & 3));
    return r;
  };
  if (!values) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * R + tid / L;
      if (r >= r0 && r < r1) *(u32x2_t*)(dst + r * D + d0) = codes(f[i]);
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
      const u32x2_t w = codes(f[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        lds[((r >> 4) * D + d0 + j) * 16 + (r & 15)] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
    }
  }
  __syncthreads();
  const int sub0 = grew ? 0 : r0 >> 4, sub1 = (r1 + 15) >> 4;
  for (int i = sub0 * D + tid; i < sub1 * D; i += 256) {
    const int t0 = (i / D) * 16;
    u32x4_t w = *(const u32x4_t*)(lds + i * 16);
    if (t0 < r0 || t0 + 16 > r1) {
      const u32x4_t was = *(const u32x4_t*)(dst + i * 16);
      const u32x4_t again = grew ? requantized(was, ratio) : was;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int t = t0 + j;
        const uint32_t m = 0xFFu << (8 * (j & 3));
        const uint32_t from = t < r0 ? again[j >> 2] : t < r1 ? w[j >> 2] : was[j >> 2];
        w[j >> 2] = (w[j >> 2] & ~m) | (from & m);
      }
    }
    *(u32x4_t*)(dst + i * 16) = w;
  }
}

template <int DT, int D>
__device__ void rotate_queries(const Kv8& c, const Rope& rope, const uint16_t* q, int64_t stride,
                               uint16_t* out, int64_t out_stride, int64_t block);

template <int DT, int D, int PASSES>
__global__ void __launch_bounds__(256)
kv8_append_kernel(Kv8 c, Rope rope, const uint16_t* __restrict__ q, int64_t q_stride,
                  uint16_t* __restrict__ q_out, int64_t qo_stride,
                  const uint16_t* __restrict__ k, int64_t k_stride,
                  const uint16_t* __restrict__ v, int64_t v_stride, int chunks, int64_t blocks) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[PASSES * 2048];
  __shared__ uint32_t part[4];
  const int64_t id = blockIdx.x;
  if (id < blocks) {
    const bool values = id & 1;
    const int64_t j = id >> 1;
    const int head = (int)(j % c.Hkv), chunk = (int)(j / c.Hkv % chunks);
    const int b = (int)(j / c.Hkv / chunks);
    append_page<DT, D, PASSES>(c, rope, values ? v : k, values ? v_stride : k_stride, values, b,
                               chunk, head, lds, part);
    return;
  }
  // queries: D / 8 lanes per (token, head)
  constexpr int L = D / 8;
  const int64_t at = (id - blocks) * (256 / L) + threadIdx.x / L;
  const int tok = (int)(at / c.H), head = (int)(at % c.H), d0 = (threadIdx.x % L) * 8;
  const bool in = tok < c.tokens;
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
  int pos = 0;
  float f[8];
  u32x4_t w = {0, 0, 0, 0};
  if (in) {
    const Kv8Seq s = kv8_seq(c, b);
    pos = s.len - s.n + tok - s.tok;
    w = *(const u32x4_t*)(q + (int64_t)tok * q_stride + head * D + d0);
  }
  widen8<DT>(w, f);
  rotate8(f, rope, pos, d0);
  if (in) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      r[i] = (uint32_t)round16<DT>(f[2 * i]) | (uint32_t)round16<DT>(f[2 * i + 1]) << 16;
    *(u32x4_t*)(q_out + (int64_t)tok * qo_stride + head * D + d0) = r;
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

// Pages read back as [n, Hkv, T, D] in 16 bits: one workgroup of 64 lanes per
// (page, head).  A lane turns 16 bytes: of k 16 channels of a token, of v one
// channel of 16 tokens.
template <int DT>
__global__ void __launch_bounds__(64)
kv8_dequant_kernel(const uint8_t* __restrict__ k, const uint8_t* __restrict__ v,
                   const float* __restrict__ ks, const float* __restrict__ vs,
                   const int32_t* __restrict__ pages, int num_pages, int Hkv, int T, int D,
                   uint16_t* __restrict__ k_out, uint16_t* __restrict__ v_out) {
  const int head = blockIdx.y, lane = threadIdx.x;
  const int page = clamp_int(pages[blockIdx.x], 0, num_pages - 1);
  const int64_t src = ((int64_t)page * Hkv + head) * T * D;
  const int64_t dst = ((int64_t)blockIdx.x * Hkv + head) * T * D;
  const float sk = ks[(int64_t)page * Hkv + head], sv = vs[(int64_t)page * Hkv + head];
  for (int i = lane * 16; i < T * D; i += 1024) {
    const u32x4_t w = *(const u32x4_t*)(k + src + i);
    u32x4_t r[2];
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const uint32_t two = w[j >> 2] >> (8 * (j & 3));
      r[j >> 3][(j >> 1) & 3] = value16<DT>(two, sk) | value16<DT>(two >> 8, sk) << 16;
    }
    *(u32x4_t*)(k_out + dst + i) = r[0];
    *(u32x4_t*)(k_out + dst + i + 8) = r[1];
  }
  for (int i = lane * 16; i < T * D; i += 1024) {
    const u32x4_t w = *(const u32x4_t*)(v + src + i);
    const int sub = i / (16 * D), d = i / 16 % D;
    for (int j = 0; j < 16; ++j)
      v_out[dst + (sub * 16 + j) * D + d] = (uint16_t)value16<DT>(w[j >> 2] >> (8 * (j & 3)), sv);
  }
}

template <int DT, int D, int PASSES>
void launch_append_p(const Kv8& c, const Rope& rope, const void* q, int64_t q_stride, void* q_out,
                     int64_t qo_stride, const void* k, int64_t k_stride, const void* v,
                     int64_t v_stride, int64_t max_new, hipStream_t st) {
  // a run of max_new tokens touches at most this many pages
  const int64_t T = (int64_t)1 << c.lgT, chunks = (max_new + T - 2) / T + 1;
  const int64_t blocks = chunks * c.B * c.Hkv * 2;
  const int64_t qblocks = q ? ceil_div((int64_t)c.tokens * c.H, 256 / (D / 8)) : 0;
  hipLaunchKernelGGL((kv8_append_kernel<DT, D, PASSES>), dim3((unsigned)(blocks + qblocks)),
                     dim3(256), 0, st, c, rope, (const uint16_t*)q, q_stride, (uint16_t*)q_out,
                     qo_stride, (const uint16_t*)k, k_stride, (const uint16_t*)v, v_stride,
                     (int)chunks, blocks);
}

template <int DT>
hipError_t launch_append(const Kv8& c, const Rope& rope, int D, const void* q, int64_t q_stride,
                         void* q_out, int64_t qo_stride, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, int64_t max_new, hipStream_t st) {
#define W4A16_APPEND(DD, P)                                                                    \
  launch_append_p<DT, DD, P>(c, rope, q, q_stride, q_out, qo_stride, k, k_stride, v, v_stride, \
                             max_new, st)
  const int T = 1 << c.lgT;
  if (D == 64) {
    if (T <= 32) W4A16_APPEND(64, 1);
    else if (T == 64) W4A16_APPEND(64, 2);
    else W4A16_APPEND(64, 4);
  } else {
    if (T == 16) W4A16_APPEND(128, 1);
    else if (T == 32) W4A16_APPEND(128, 2);
    else if (T == 64) W4A16_APPEND(128, 4);
    else W4A16_APPEND(128, 8);
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
    const int64_t T = page_size, chunks = (max_new + T - 2) / T + 1;
    if (chunks * B * Hkv * 2 + tokens * H > ((int64_t)1 << 31) - 1) return W4A16_ERR_UNSUPPORTED;
    clear_pending_error();
    const Kv8 c = {k_cache, v_cache, k_scale, v_scale, page_table, seq_lens, cu_seqlens,
                   (int)num_pages, (int)max_pages, (int)B, (int)tokens, H, Hkv,
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
    const dim3 g((unsigned)n, (unsigned)Hkv), b(64);
    const hipStream_t st = (hipStream_t)stream;
    if (dtype == DT_F16)
      hipLaunchKernelGGL(kv8_dequant_kernel<DT_F16>, g, b, 0, st, k_cache, v_cache, k_scale,
                         v_scale, pages, (int)num_pages, Hkv, page_size, D, (uint16_t*)k_out,
                         (uint16_t*)v_out);
    else
      hipLaunchKernelGGL(kv8_dequant_kernel<DT_BF16>, g, b, 0, st, k_cache, v_cache, k_scale,
                         v_scale, pages, (int)num_pages, Hkv, page_size, D, (uint16_t*)k_out,
                         (uint16_t*)v_out);
    return hip_status(hipGetLastError());
  });
}

}  // extern "C"
