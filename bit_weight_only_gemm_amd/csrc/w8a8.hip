// w8a8.hip -- matrix products of 8-bit integers with one scale per token
// (row of x) and per output channel (row of w), and the quantizer that makes
// such rows:
//
//   y[m, n] = round16( fp32(sum_k cx[m, k] cw[n, k]) * (sx[m] * sw[n]) + b[n] ).
//
// The sum is exact in int32 (|c| <= 127 and K <= 2^17), so it does not depend
// on any split of K.
#include <cstdio>

#include "abi.h"
#include "launch.h"
#include "quant8.h"

namespace w4a16 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

namespace {

// ------------------------------------------------------------- quantizer ---
// One workgroup per row; a row that fits 256 lanes x 8 x kHold values is read
// once and kept in registers between its maximum and its codes, a longer one
// is read again (from cache).
constexpr int kHold = 8;

template <int DT>
__device__ __forceinline__ void load8(const void* x, int64_t i, float (&f)[8]) {
  if constexpr (DT == 2) {
    const float4_t a = *(const float4_t*)((const float*)x + i);
    const float4_t b = *(const float4_t*)((const float*)x + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = a[j], f[4 + j] = b[j];
  } else {
    widen8<DT>(*(const u32x4_t*)((const uint16_t*)x + i), f);
  }
}

__device__ __forceinline__ u32x2_t codes8(const float (&f)[8], float s) {
  u32x2_t r = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    r[j >> 2] |= ((uint32_t)code_of(f[j], s) & 0xFFu) << (8 * (j & 3));
  return r;
}

template <int DT>
__global__ void __launch_bounds__(256)
w8a8_quantize_kernel(const void* __restrict__ x, int64_t stride, int K, int8_t* __restrict__ codes,
                     float* __restrict__ scales) {
  __shared__ uint32_t part[4];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t base = row * stride;
  float f[kHold][8];
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int k = (i * 256 + tid) * 8;
    if (k < K) {
      load8<DT>(x, base + k, f[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(f[i][j]));
    }
  }
  for (int k = (kHold * 256 + tid) * 8; k < K; k += 2048) {
    float g[8];
    load8<DT>(x, base + k, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(g[j]));
  }
  mag = lanes_max<64>(mag);
  if ((tid & 63) == 0) part[tid >> 6] = mag;
  __syncthreads();
  mag = max(max(part[0], part[1]), max(part[2], part[3]));
  float s = scale_of(mag);
  if (s == 0.0f) s = 1.0f;
  int8_t* out = codes + row * (int64_t)K;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int k = (i * 256 + tid) * 8;
    if (k < K) *(u32x2_t*)(out + k) = codes8(f[i], s);
  }
  for (int k = (kHold * 256 + tid) * 8; k < K; k += 2048) {
    float g[8];
    load8<DT>(x, base + k, g);
    *(u32x2_t*)(out + k) = codes8(g, s);
  }
  if (tid == 0) scales[row] = s;
}

hipError_t launch_quantize(const void* x, int64_t M, int64_t K, int64_t stride, int dtype,
                           int8_t* codes, float* scales, hipStream_t st) {
  const dim3 g((unsigned)M), b(256);
  if (dtype == W4A16_F16)
    hipLaunchKernelGGL(w8a8_quantize_kernel<DT_F16>, g, b, 0, st, x, stride, (int)K, codes, scales);
  else if (dtype == W4A16_BF16)
    hipLaunchKernelGGL(w8a8_quantize_kernel<DT_BF16>, g, b, 0, st, x, stride, (int)K, codes, scales);
  else
    hipLaunchKernelGGL(w8a8_quantize_kernel<2>, g, b, 0, st, x, stride, (int)K, codes, scales);
  return hipGetLastError();
}

// ---------------------------------------------------------------- product ---
// One wave per 32 x 32 tile of y on v_mfma_i32_32x32x32_i8, operands straight
// from memory: lane l holds 16 codes of row l & 31 at inputs 16 (l >> 5) of a
// step; rows past the end and inputs past K read 0.
template <int DT>
__global__ void __launch_bounds__(256)
w8a8_gemm_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                 const int8_t* __restrict__ wq, const float* __restrict__ sw,
                 const uint16_t* __restrict__ bias, uint16_t* __restrict__ out, int M, int N,
                 int K) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row0 = (int)blockIdx.y * 64 + 32 * (wave >> 1);
  const int col0 = (int)blockIdx.x * 64 + 32 * (wave & 1);
  if (row0 >= M || col0 >= N) return;
  const int r = lane & 31, h = lane >> 5;
  const rsrc_t rx = make_rsrc(xq + (size_t)row0 * K, (uint32_t)min(32, M - row0) * (uint32_t)K);
  const rsrc_t rw = make_rsrc(wq + (size_t)col0 * K, (uint32_t)min(32, N - col0) * (uint32_t)K);
  i32x16_t acc{};
  for (int k = 16 * h; k < ((K + 31) & ~31); k += 32) {
    const uint32_t off = k < K ? (uint32_t)r * (uint32_t)K + (uint32_t)k : kOutOfRange;
    const i32x4_t a = __builtin_bit_cast(i32x4_t, bld128(rx, off, 0));
    const i32x4_t b = __builtin_bit_cast(i32x4_t, bld128(rw, off, 0));
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc, 0, 0, 0);
  }
  const int col = col0 + r;
  if (col >= N) return;
  const float t = sw[col], b = bias ? widen16<DT>(bias[col]) : 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int row = row0 + (i & 3) + 4 * h + 8 * (i >> 2);
    if (row < M) out[(size_t)row * N + col] = round16<DT>((float)acc[i] * (sx[row] * t) + b);
  }
}

hipError_t launch_gemm(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                       const void* bias, void* out, int64_t M, int64_t N, int64_t K, int dtype,
                       hipStream_t st) {
  const dim3 g((unsigned)ceil_div(N, 64), (unsigned)ceil_div(M, 64)), b(256);
  if (dtype == DT_F16)
    launch_timed(w8a8_gemm_kernel<DT_F16>, g, b, 0, st, xq, sx, wq, sw, (const uint16_t*)bias,
                 (uint16_t*)out, (int)M, (int)N, (int)K);
  else
    launch_timed(w8a8_gemm_kernel<DT_BF16>, g, b, 0, st, xq, sx, wq, sw, (const uint16_t*)bias,
                 (uint16_t*)out, (int)M, (int)N, (int)K);
  return hipGetLastError();
}

// --------------------------------------------------------------- checking ---
constexpr int64_t kMaxM = (int64_t)1 << 21, kMaxN = (int64_t)1 << 24, kMaxK = (int64_t)1 << 17;

int validate_shape(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 16 != 0 || N % 8 != 0) return W4A16_ERR_INVALID_ARG;
  if (M > kMaxM || N > kMaxN || K > kMaxK || M * N > ((int64_t)1 << 36))
    return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

int64_t pad256(int64_t b) { return ceil_div(b, 256) * 256; }

// w8a8_linear's codes and scales
int64_t linear_bytes(int64_t M, int64_t K) { return pad256(M * K) + pad256(M * 4); }

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int w8a8_quantize(const void* x, int64_t M, int64_t K, int64_t x_stride, int32_t dtype,
                  int8_t* codes, float* scales, void* stream) {
  return guarded([&]() -> int {
    if (int s = validate_shape(M, 8, K)) return s;
    if (dtype < W4A16_F16 || dtype > W4A16_F32) return W4A16_ERR_INVALID_ARG;
    if (x_stride < K || x_stride % 8 != 0) return W4A16_ERR_INVALID_ARG;
    if (int s = check_ptrs({x, codes, scales})) return s;
    clear_pending_error();
    return hip_status(launch_quantize(x, M, K, x_stride, dtype, codes, scales,
                                      (hipStream_t)stream));
  });
}

int64_t w8a8_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t linear) {
  if (validate_shape(M, N, K) != W4A16_OK) return -1;
  return linear ? linear_bytes(M, K) : 0;
}

int w8a8_gemm(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
              const void* bias, void* out, int64_t M, int64_t N, int64_t K, int32_t dtype,
              void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    if (int s = validate_shape(M, N, K)) return s;
    if (int s = validate_dtype(dtype)) return s;
    if (int s = check_ptrs({xq, x_scale, wq, w_scale, out})) return s;
    if (!aligned16(bias) || !aligned16(workspace)) return W4A16_ERR_MISALIGNED;
    if (workspace && workspace_bytes < w8a8_workspace_bytes(M, N, K, 0))
      return W4A16_ERR_WORKSPACE;
    clear_pending_error();
    return hip_status(launch_gemm(xq, x_scale, wq, w_scale, bias, out, M, N, K, dtype,
                                  (hipStream_t)stream));
  });
}

int w8a8_linear(const void* x, int64_t x_stride, const int8_t* wq, const float* w_scale,
                const void* bias, void* out, int64_t M, int64_t N, int64_t K, int32_t dtype,
                void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    if (int s = validate_shape(M, N, K)) return s;
    if (int s = validate_dtype(dtype)) return s;
    if (x_stride < K || x_stride % 8 != 0) return W4A16_ERR_INVALID_ARG;
    if (int s = check_ptrs({x, wq, w_scale, out})) return s;
    if (!aligned16(bias) || !aligned16(workspace)) return W4A16_ERR_MISALIGNED;
    const int64_t need = w8a8_workspace_bytes(M, N, K, 1);
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
    clear_pending_error();
    const hipStream_t st = (hipStream_t)stream;
    int8_t* xq = (int8_t*)workspace;
    float* sx = (float*)(xq + pad256(M * K));
    if (int s = hip_status(launch_quantize(x, M, K, x_stride, dtype, xq, sx, st))) return s;
    return hip_status(launch_gemm(xq, sx, wq, w_scale, bias, out, M, N, K, dtype, st));
  });
}

}  // extern "C"
