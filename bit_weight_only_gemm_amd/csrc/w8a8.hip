// w8a8.hip -- matrix products of 8-bit integers with one scale per token
// (row of x) and per output channel (row of w), and the quantizer that makes
// such rows:
//
//   y[m, n] = round16( fp32(sum_k cx[m, k] cw[n, k]) * (sx[m] * sw[n]) + b[n] ).
//
// The sum is exact in int32 (|c| <= 127 and K <= 2^17), so it does not depend
// on any split of K.
#include <stdio.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "abi.h"
#include "launch.h"
#include "quant8.h"

namespace w4a16 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

namespace {

// ------------------------------------------------------------- quantizer ---
// One workgroup of LANES lanes per row.  The first 16384 values are read once,
// every load out before the first is used, and kept in registers between the
// row's maximum and its codes; what a longer row has beyond them is read again
// (from cache).
//
// The bytes bound it where there are many rows (8192 x 5120 in bf16: 29 us,
// 4.3 TB/s), a row's chain of load, maximum, division and store where there are
// few: then 1024 lanes share that chain (MI355X, 256 lanes -> 1024: 16 x 11008
// 5.0 -> 4.5 us, 512 x 11008 7.9 -> 7.3, but 1024 x 4096 6.4 -> 7.5 and 8192 x
// 5120 29 -> 47, where the barriers of large workgroups show).
constexpr int kHeld = 16384, kFewRows = 512 + 1;

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

__device__ __forceinline__ u32x2_t codes8(const float (&f)[8], const Codes8& q) {
  int c[8];
  q(f, c);
  u32x2_t r = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j >> 2] |= ((uint32_t)c[j] & 0xFFu) << (8 * (j & 3));
  return r;
}

template <int DT, int LANES>
__global__ void __launch_bounds__(LANES)
w8a8_quantize_kernel(const void* __restrict__ x, int64_t stride, int K, int8_t* __restrict__ codes,
                     float* __restrict__ scales, uint32_t* __restrict__ counts, int num_counts) {
  constexpr int HOLD = kHeld / (8 * LANES), BYTES = DT == 2 ? 4 : 2, PARTS = BYTES / 2;
  __shared__ uint32_t part[LANES / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t base = row * stride;
  // counters of the product that follows, at zero
  for (int i = (int)blockIdx.x * LANES + tid; i < num_counts; i += (int)gridDim.x * LANES)
    counts[i] = 0;
  // (a load past the row's end gives zeros)
  const rsrc_t r = make_rsrc((const uint8_t*)x + base * BYTES, (uint32_t)K * BYTES);
  u32x4_t raw[HOLD][PARTS];
#pragma unroll
  for (int i = 0; i < HOLD; ++i)
#pragma unroll
    for (int p = 0; p < PARTS; ++p)
      raw[i][p] = bld128(r, (uint32_t)(i * LANES + tid) * 8 * BYTES + 16 * p, 0);
  auto held = [&](int i, float (&f)[8]) {
    if constexpr (DT == 2) {
      const u32x4_t lo = raw[i][0], hi = raw[i][PARTS - 1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = lo[j], b = hi[j];
        f[j] = __builtin_bit_cast(float, a), f[4 + j] = __builtin_bit_cast(float, b);
      }
    } else {
      widen8<DT>(raw[i][0], f);
    }
  };
  uint32_t mag = 0;
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    float f[8];
    held(i, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(f[j]));
  }
  for (int k = kHeld + tid * 8; k < K; k += 8 * LANES) {
    float g[8];
    load8<DT>(x, base + k, g);
#pragma unroll
    for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(g[j]));
  }
  mag = lanes_max<64>(mag);
  if ((tid & 63) == 0) part[tid >> 6] = mag;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < LANES / 64; ++i) mag = max(mag, part[i]);
  float s = scale_of(mag);
  if (s == 0.0f) s = 1.0f;
  const Codes8 q(s);
  int8_t* out = codes + row * (int64_t)K;
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    const int k = (i * LANES + tid) * 8;
    float f[8];
    held(i, f);
    if (k < K) *(u32x2_t*)(out + k) = codes8(f, q);
  }
  for (int k = kHeld + tid * 8; k < K; k += 8 * LANES) {
    float g[8];
    load8<DT>(x, base + k, g);
    *(u32x2_t*)(out + k) = codes8(g, q);
  }
  if (tid == 0) scales[row] = s;
}

template <int DT>
void launch_quantize_dt(const void* x, int64_t M, int64_t K, int64_t stride, int8_t* codes,
                        float* scales, uint32_t* counts, int num_counts, hipStream_t st) {
  if (M < kFewRows)
    hipLaunchKernelGGL((w8a8_quantize_kernel<DT, 1024>), dim3((unsigned)M), dim3(1024), 0, st, x,
                       stride, (int)K, codes, scales, counts, num_counts);
  else
    hipLaunchKernelGGL((w8a8_quantize_kernel<DT, 256>), dim3((unsigned)M), dim3(256), 0, st, x,
                       stride, (int)K, codes, scales, counts, num_counts);
}

hipError_t launch_quantize(const void* x, int64_t M, int64_t K, int64_t stride, int dtype,
                           int8_t* codes, float* scales, hipStream_t st,
                           uint32_t* counts = nullptr, int num_counts = 0) {
  (dtype == W4A16_F16    ? launch_quantize_dt<DT_F16>
   : dtype == W4A16_BF16 ? launch_quantize_dt<DT_BF16>
                         : launch_quantize_dt<2>)(x, M, K, stride, codes, scales, counts,
                                                  num_counts, st);
  return hipGetLastError();
}

// ---------------------------------------------------------------- product ---
// 16 bytes per lane from a buffer straight into LDS: lane l's data lands at
// lds + 16 l (the LDS base is wave-uniform).
__device__ __forceinline__ void dma16(rsrc_t r, uint8_t* lds, uint32_t voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(
      r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
}

// Two fp32 values rounded to 16 bits, in one register.
template <int DT>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  if constexpr (DT == DT_F16) {
    const half2_t v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
  } else {
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
}

// One result in fp32: the sum times the two scales, plus the bias.  Every
// kernel here forms it by these operations, so that the choice of a kernel
// does not show in the result.
__device__ __forceinline__ float result(int acc, float s, float t, float bias) {
  return __builtin_fmaf((float)acc, s * t, bias);
}

// Results 4 g .. 4 g + 3 of a product: 4 channels of one token, in 16 bits.
template <int DT>
__device__ __forceinline__ u32x2_t results4(const i32x16_t& acc, int g, float s, float4_t t,
                                            float4_t bias) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = result(acc[4 * g + e], s, t[e], bias[e]);
  return u32x2_t{pack16<DT>(y[0], y[1]), pack16<DT>(y[2], y[3])};
}

// ------------------------------------------------------ gated product (ACT) ---
// Gated kernels take w as 2 F rows, the gate's and then the up projection's, and
// form F channels y = act(g) u.  They go through w's rows in blocks of 8, the
// gate's and the up projection's in turn, so that a lane whose results are
// channels 8 i + 4 h + e of the gate has the same channels of the up projection in
// its next four registers, whatever the tile; N counts all 2 F rows.
//
// act(g) = g sigmoid(a g + b g^3) for silu (a = 1, b = 0) and for gelu in its tanh
// form (0.5 (1 + tanh z) = sigmoid(2 z)); log2 e is in a and b.  gelu is g Phi(g),
// with Phi(-y) = exp(-y^2 / 2) P(1 / (1 + 0.35 y)), y >= 0: P is a fit of degree 7 to
// erfcx(y / sqrt 2) / 2 over [0, 14.5], 5e-7 off (7e-7 in fp32), and both of its tails
// keep that relative error.  g, u and act are fp32 and rounded once, as y.
enum { kNoGate = 0, kSigmoid = 1, kErf = 2 };
struct Gate {
  int F;
  float a, b;
};
template <int ACT>
__device__ __forceinline__ float gated(float g, float u, const Gate& c) {
  if constexpr (ACT == kSigmoid) {
    const float w = g * __builtin_fmaf(c.b, fminf(g * g, 3e38f), c.a);
    return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-w)) * u;
  } else {
    const float y = fabsf(g), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, y, 1.0f));
    float p = 0.04819544777f;
    p = __builtin_fmaf(p, t, -0.19929255545f);
    p = __builtin_fmaf(p, t, 0.23627594113f);
    p = __builtin_fmaf(p, t, -0.01347748376f);
    p = __builtin_fmaf(p, t, 0.15433320403f);
    p = __builtin_fmaf(p, t, 0.13377590477f);
    p = __builtin_fmaf(p, t, 0.14021381736f);
    p = __builtin_fmaf(p, t, -0.00002427048f);
    p *= __builtin_amdgcn_exp2f(y * (y * -0.72134752044f));
    return g * (g < 0.0f ? p : 1.0f - p) * u;
  }
}

// gated() of results 8 p .. 8 p + 3 of a product (the gate's) and the 4 after.
template <int DT, int ACT>
__device__ __forceinline__ u32x2_t gated4(const i32x16_t& acc, int p, float s, float4_t tg,
                                          float4_t bg, float4_t tu, float4_t bu, const Gate& c) {
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    y[e] = gated<ACT>(result(acc[8 * p + e], s, tg[e], bg[e]),
                      result(acc[8 * p + 4 + e], s, tu[e], bu[e]), c);
  return u32x2_t{pack16<DT>(y[0], y[1]), pack16<DT>(y[2], y[3])};
}

// Scales and bias of the 4 channels from n on.
template <int DT>
__device__ __forceinline__ void channels4(const float* sw, const uint16_t* bias, int64_t n,
                                          float4_t& t, float4_t& b) {
  t = *(const float4_t*)(sw + n);
  b = float4_t{0, 0, 0, 0};
  if (bias) {
    const u32x2_t w = *(const u32x2_t*)(bias + n);
#pragma unroll
    for (int e = 0; e < 4; ++e) b[e] = widen16<DT>((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
  }
}

// K split over workgroups (gated tiles): partial sums in int32, [split][tile][BM BN],
// and a counter for each tile, 0 before the call.  Sums of integers do not depend
// on their order.
struct Split {
  int splits;
  int32_t* parts;
  uint32_t* count;
};
// Two sums past the caches of one die, for a workgroup on another.
__device__ __forceinline__ void send2(int32_t* to, int a, int b) {
  const uint64_t v = (uint64_t)(uint32_t)a | (uint64_t)(uint32_t)b << 32;
  __hip_atomic_store((uint64_t*)to, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t fetch2(const int32_t* from) {
  return __hip_atomic_load((const uint64_t*)from, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Tile shape: WM x WN waves, each MT x NT products of 32 x 32.
template <int MT_, int NT_, int WM_, int WN_, int NS_>
struct Tile {
  static constexpr int MT = MT_, NT = NT_, WM = WM_, WN = WN_, NS = NS_;
  static constexpr int WAVES = WM * WN, BM = 32 * MT * WM, BN = 32 * NT * WN;
  static constexpr int STAGE = (BM + BN) * 128;         // bytes of one step of 128 codes
  static constexpr int LOADS = (BM + BN) / 8 / WAVES;   // 1 KB loads per wave and step
  static_assert((BM + BN) / 8 % WAVES == 0 && NS >= 3, "whole loads per wave");
};

// One workgroup per BM x BN tile of y on v_mfma_i32_32x32x32_i8, the rows of
// w as the first operand (so that a lane's 4 consecutive results are 4
// channels of one token).  For calls of few tiles, which wait for memory:
// nearly all of LDS is steps under way.
//
//  * K goes by in steps of 128 codes.  A step's rows of w and x come straight
//    into LDS (128-byte rows, whole cache lines; the 16-byte chunk q of row r at
//    position q ^ (r >> 1 & 7), so that 16 lanes reading one chunk of 16 rows
//    meet all banks), NS steps deep: the loads of step t + NS - 1 go out in
//    step t.
//  * A step is four quarters of 32 codes.  The operands of a quarter are read
//    while the products of the quarter before run, across the step's boundary
//    too: the wait and the barrier for step t + 1 stand before step t's last.
//  * The results pass through LDS into whole 64 NT-byte pieces of y's rows.
//
// LDS bounds a workgroup: in 128 x 128 a step costs it 32 KB written and 96 KB
// read (1000 cycles at 128 bytes each) against 512 cycles of products.  MI355X:
// 333 x 7168 x 5120 in 23.3 us (1.05 PFLOP/s; 25.1 with 4 waves of 2 x 2, 22.8
// with 16 of 1 x 1, 24.0 with 96 x 128 tiles; reading operands two quarters
// ahead changed nothing), 128 x 4096 x 4096 in 64 x 64 tiles 11.3 us.
template <int DT, class TL, int ACT>
__global__ void __launch_bounds__(64 * TL::WAVES)
w8a8_tile_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                 const int8_t* __restrict__ wq, const float* __restrict__ sw,
                 const uint16_t* __restrict__ bias, uint16_t* __restrict__ out, int M, int N,
                 int K, int mb, int nb, int per_xcd, Gate gate, Split sp) {
  constexpr int MT = TL::MT, NT = TL::NT, NS = TL::NS, L = TL::LOADS;
  __shared__ __attribute__((aligned(16))) uint8_t lds[NS * TL::STAGE];
  // ---- tile of this workgroup: workgroups go to the 8 XCDs in turn, so each
  // XCD takes a contiguous run of tiles, ordered in bands of 8 row blocks
  // (gated: the splits of a tile follow one another)
  const int splits = ACT ? sp.splits : 1;
  const int turn = (int)(blockIdx.x >> 3) / splits, split = (int)(blockIdx.x >> 3) % splits;
  const int at = (int)(blockIdx.x & 7) * per_xcd + turn;
  if (turn >= per_xcd || at >= mb * nb) return;
  const int band = at / (8 * nb), in_band = at % (8 * nb);
  const int bh = min(8, mb - band * 8);
  const int row0 = (band * 8 + in_band % bh) * TL::BM, col0 = in_band / bh * TL::BN;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  // codes of this split, from the k0-th on (every split has some)
  const int share = ACT ? (((K + 127) >> 7) + splits - 1) / splits * 128 : K;
  const int k0 = ACT ? split * share : 0, KS = ACT ? min(share, K - k0) : K;
  const int KT = (KS + 127) >> 7;
  // (gated: the waves being even in number, a wave's blocks are all of the gate's
  // rows or all of the up projection's)
  constexpr int HALVES = ACT ? 2 : 1;
  static_assert(TL::WAVES % 2 == 0, "blocks of w in turn");
  const rsrc_t rw = make_rsrc(wq + (size_t)((ACT && (wave & 1) ? gate.F : 0) + col0 / HALVES) * K + k0,
                              (uint32_t)min(TL::BN, N - col0) / HALVES * (uint32_t)K - (uint32_t)k0);
  const rsrc_t rx = make_rsrc(xq + (size_t)row0 * K + k0,
                              (uint32_t)min(TL::BM, M - row0) * (uint32_t)K - (uint32_t)k0);

  // load i of this wave fills the LDS block WAVES i + wave (8 rows); blocks
  // below BN / 8 are rows of w
  const int lrow = lane >> 3;
  auto load = [&](int t, int i) {
    const int blk = TL::WAVES * i + wave;
    const bool is_w = blk < TL::BN / 8;
    const uint32_t row = 8u * (uint32_t)(is_w ? blk : blk - TL::BN / 8) + (uint32_t)lrow;
    const uint32_t chunk = ((uint32_t)lane & 7u) ^ ((row >> 1) & 7u);
    const uint32_t from = ACT && is_w ? 8u * (uint32_t)(blk >> 1) + (uint32_t)lrow : row;
    const uint32_t off =
        128 * t + 16 * (int)chunk < KS ? from * (uint32_t)K + 16u * chunk : kOutOfRange;
    dma16(is_w ? rw : rx, lds + (t % NS) * TL::STAGE + blk * 1024, off, t * 128);
  };

  const int r = lane & 31, h = lane >> 5;
  const uint32_t swz = (r >> 1) & 7;
  const uint32_t woff = (uint32_t)(wn * NT * 32 + r) * 128, xoff = (uint32_t)(TL::BN + wm * MT * 32 + r) * 128;
  i32x4_t fw[2][NT], fx[2][MT];
  auto read = [&](int t, int quarter, i32x4_t (&w)[NT], i32x4_t (&x)[MT]) {
    const uint8_t* st = lds + (t % NS) * TL::STAGE + (((2 * quarter + h) ^ swz) << 4);
#pragma unroll
    for (int i = 0; i < NT; ++i) w[i] = *(const i32x4_t*)(st + woff + i * 4096);
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = *(const i32x4_t*)(st + xoff + i * 4096);
  };
  i32x16_t acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = i32x16_t{};
  auto products = [&](const i32x4_t (&w)[NT], const i32x4_t (&x)[MT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[i], x[j], acc[i][j], 0, 0, 0);
  };

#pragma unroll
  for (int t = 0; t < NS - 1; ++t)
#pragma unroll
    for (int i = 0; i < L; ++i) load(t, i);
  // step 0 is complete: the loads of NS - 2 later steps may be pending
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NS - 2) * L) : "memory");
  read(0, 0, fw[0], fx[0]);
  for (int t = 0; t < KT; ++t) {
    // the slot of step t - 1 is free: every wave has passed the barrier below
    // with its reads of that step complete
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      read(t, q + 1, fw[(q + 1) & 1], fx[(q + 1) & 1]);
      if (q == 0) {
#pragma unroll
        for (int i = 0; i < L; ++i) load(t + NS - 1, i);
      }
      products(fw[q & 1], fx[q & 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // step t + 1 is complete in LDS (the loads of NS - 2 later steps may be
    // pending), and so are this wave's reads of step t
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NS - 2) * L) : "memory");
    __builtin_amdgcn_sched_barrier(0);
    read(t + 1, 0, fw[0], fx[0]);
    products(fw[1], fx[1]);
    __builtin_amdgcn_sched_barrier(0);
  }
  // the loads past the last step have written their zeros
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");

  // ---- splits: each leaves its sums and counts itself, the last to arrive adds
  // them up.  They have gone past the die's cache before the count does.
  if (ACT && splits > 1) {
    constexpr int SUMS = TL::BM * TL::BN;
    const int tiles = mb * nb, mine = wave * NT * MT * 1024 + lane * 4;
    int32_t* part = sp.parts + ((size_t)split * tiles + at) * SUMS + mine;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 16; e += 2)
          send2(part + ((i * MT + j) * 4 + (e >> 2)) * 256 + (e & 2), acc[i][j][e], acc[i][j][e + 1]);
    // (in the ring, which is free: beside a second variable in LDS the compiler takes
    // the loop's reads to wait for its loads, 0.6 us a step instead of 0.3)
    uint32_t* arrived = (uint32_t*)lds;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (tid == 0)
      *arrived = __hip_atomic_fetch_add(sp.count + at, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    const bool last = *arrived == (uint32_t)splits - 1;
    if (!last) return;
    __syncthreads();  // the results go where it lies
    for (int other = 0; other < splits; ++other) {
      if (other == split) continue;
      const int32_t* from = sp.parts + ((size_t)other * tiles + at) * SUMS + mine;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const uint64_t v = fetch2(from + ((i * MT + j) * 4 + (e >> 2)) * 256 + (e & 2));
            acc[i][j][e] += (int)(uint32_t)v;
            acc[i][j][e + 1] += (int)(uint32_t)(v >> 32);
          }
    }
  }

  // ---- results: register i of product (nt, mt) is channel 8 (i >> 2) + 4 h +
  // (i & 3) of its 32, token lane & 31; one 32-token block of the wave at a time
  constexpr int ROW = NT * 64 / HALVES + 16;  // bytes of a token's row in LDS
  static_assert(TL::WAVES * 32 * ROW <= NS * TL::STAGE, "the results fit");
  uint8_t* mine = lds + wave * 32 * ROW;
  const int width = N / HALVES, wcol = (col0 + wn * NT * 32) / HALVES;  // of y
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int mrow = row0 + (wm * MT + j) * 32;
    const float s = mrow + r < M ? sx[mrow + r] : 0.0f;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int g = 0; g < 4 / HALVES; ++g) {
        const int n = wcol + i * (32 / HALVES) + 8 * g + 4 * h;
        float4_t t = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (n < width) channels4<DT>(sw, bias, n, t, b);
        uint8_t* to = mine + r * ROW + i * (64 / HALVES) + 16 * g + 8 * h;
        if constexpr (ACT != kNoGate) {
          float4_t tu = {0, 0, 0, 0}, bu = {0, 0, 0, 0};
          if (n < width) channels4<DT>(sw, bias, (int64_t)gate.F + n, tu, bu);
          *(u32x2_t*)to = gated4<DT, ACT>(acc[i][j], g, s, t, b, tu, bu, gate);
        } else {
          *(u32x2_t*)to = results4<DT>(acc[i][j], g, s, t, b);
        }
      }
    constexpr int LR = NT * 4 / HALVES;  // lanes per row
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int k = 0; k < 32 / (64 / LR); ++k) {
      const int tr = k * (64 / LR) + lane / LR, c = (lane % LR) * 8;
      const u32x4_t v = *(const u32x4_t*)(mine + tr * ROW + c * 2);
      if (mrow + tr < M && wcol + c < width)
        *(u32x4_t*)(out + (size_t)(mrow + tr) * width + wcol + c) = v;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The same product for many tokens: workgroups stay and take 64 MT x 256 tiles
// in turn, 4 waves of 4 x MT products (MT = 4, and 3 in the gated form).  K goes by
// in steps of 128 codes (whole 128-byte lines of w and x), four quarters of 32 each:
//
//  * The rows of step t + 2 are loaded into registers while step t runs, each
//    register right after its part of step t + 1 went from it to LDS, so a load
//    has a whole step to arrive; LDS holds two steps (64 KB each; chunk q of row
//    r at position q ^ (r >> 1 & 7): 16 lanes reading one chunk of 16 rows meet
//    all banks).  One barrier per step, before its last quarter.
//  * The operands of a quarter are read while the products of the quarter
//    before run.  Steps go on across tiles: a tile's first rows and operands
//    arrive during the last step and the results of the tile before.
//  * The results pass through LDS of their own into whole 128-byte pieces of
//    y's rows; the tile's scales and bias wait there since its first step, in
//    one of two places by the tile's parity: no barrier stands between a tile's
//    results and the first step of the next, which writes the other place, and
//    before a wave writes this one again it passes a barrier that every wave
//    reaches only after these results.
//
// The matrix units bound it, at the clock the card holds under them: 8192 x
// 55296 x 5120 in 1850 to 1950 us by card, 2.5 to 2.4 PFLOP/s, the units busy 68 %
// of the cycles (2.57 with every load from L2, 2.82 without loads; with one tile
// per workgroup and loads straight to LDS it took 2324 us).  The gated form of it, 8192
// x 27648 x 5120, takes 1893 to 2048 us by card, its quantizing among them: half the
// results to write pay for the activations.
constexpr int kWideStage = 512 * 128, kWideTurn = 2 * kWideStage, kWideScales = kWideTurn + 4 * 4096;
// x's scales, w's, the bias as fp32; of this tile and of the one before
constexpr int kWideLds = kWideScales + 2 * 256 * 12;

template <int DT, int ACT, int MT>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
w8a8_wide_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                 const int8_t* __restrict__ wq, const float* __restrict__ sw,
                 const uint16_t* __restrict__ bias, uint16_t* __restrict__ out, int M, int N,
                 int K, int mb, int nb, int per_xcd, Gate gate) {
  constexpr int HALVES = ACT ? 2 : 1, BM = 64 * MT, LOADS = 8 + 2 * MT;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kWideLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const int KT = (K + 127) >> 7;

  // ---- tiles of this workgroup: each XCD has a contiguous run of them, in
  // bands of 8 row blocks; its workgroups take them in turn
  const int run0 = (int)(blockIdx.x & 7) * per_xcd;
  const int run1 = min(run0 + per_xcd, mb * nb);
  const int every = (int)(gridDim.x >> 3);
  const int first = run0 + (int)(blockIdx.x >> 3);
  if (first >= run1) return;
  auto tile_at = [&](int at, int& row0, int& col0) {
    const int band = at / (8 * nb), in_band = at % (8 * nb);
    const int bh = min(8, mb - band * 8);
    row0 = (band * 8 + in_band % bh) * BM;
    col0 = in_band / bh * 256;
  };

  // ---- loads: instruction i of a step fetches 8 rows x 128 bytes, i < 8 rows
  // of w, from 64 wave + 8 i of the tile, i >= 8 rows of x, from 16 MT wave + 8 (i - 8)
  const int lrow = lane >> 3, lchunk = lane & 7;
  // (gated: block 8 wave + i of w is the block (8 wave + i) / 2 of the gate's rows
  // where i is even, of the up projection's where it is odd)
  const uint32_t lane_off = (uint32_t)(64 * wave + lrow) * (uint32_t)K + 16u * lchunk;
  const uint32_t x_off = (uint32_t)(16 * MT * wave + lrow) * (uint32_t)K + 16u * lchunk;
  const uint32_t gate_off = (uint32_t)(32 * wave + lrow) * (uint32_t)K + 16u * lchunk;
  const uint32_t tail = 128 * (KT - 1) + 16 * lchunk >= K ? kOutOfRange : 0u;
  const uint32_t lane_lds = (uint32_t)(64 * wave + lrow) * 128 + 16u * (lchunk ^ ((lrow >> 1) & 3));
  int lat = first, lt = 0;  // the step that is loaded next
  rsrc_t rw, ru, rx;
  auto aim = [&]() {
    int row0 = 0, col0 = 0;
    const bool any = lat < run1;
    if (any) tile_at(lat, row0, col0);
    const uint32_t w_bytes = any ? (uint32_t)min(256, N - col0) / HALVES * (uint32_t)K : 0u;
    rw = make_rsrc(wq + (size_t)(col0 / HALVES) * K, w_bytes);
    if constexpr (ACT != kNoGate) ru = make_rsrc(wq + (size_t)(gate.F + col0 / 2) * K, w_bytes);
    rx = make_rsrc(xq + (size_t)row0 * K, any ? (uint32_t)min(BM, M - row0) * (uint32_t)K : 0u);
  };
  aim();
  i32x4_t held[LOADS];
  auto load = [&](int i) {
    const bool half = ACT && i < 8;
    const uint32_t row = half ? 8 * (i >> 1) : 8 * (i & 7);
    const uint32_t base = half ? gate_off : i < 8 ? lane_off : x_off;
    const uint32_t off = (base + row * (uint32_t)K) | (lt == KT - 1 ? tail : 0u);
    held[i] = __builtin_bit_cast(i32x4_t, bld128(i >= 8 ? rx : half && (i & 1) ? ru : rw, off, lt * 128));
  };
  auto loaded = [&]() {  // every load of a step is out
    if (++lt == KT) {
      lt = 0;
      lat += every;
      aim();
    }
  };
  // row 64 wave + 8 i + lrow (of x 16 MT wave + ..): (row >> 1) & 7 is ((lrow >> 1) &
  // 3) + 4 (i & 1)
  auto store = [&](int slot, int i) {
    *(i32x4_t*)(lds + slot * kWideStage + (i < 8 ? 0 : 32768 - (64 - 16 * MT) * 128 * wave) +
                (i & 7) * 1024 + (lane_lds ^ ((i & 1) << 6))) = held[i];
  };

  const int r = lane & 31, h = lane >> 5;
  i32x4_t fw[2][4], fx[2][MT];
  auto read = [&](int slot, int quarter, i32x4_t (&w)[4], i32x4_t (&x)[MT]) {
    const uint8_t* st = lds + slot * kWideStage + (((2 * quarter + h) ^ ((r >> 1) & 7)) << 4) + r * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *(const i32x4_t*)(st + wn * 16384 + i * 4096);
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = *(const i32x4_t*)(st + 32768 + wm * MT * 4096 + i * 4096);
  };
  i32x16_t acc[4][MT];
  auto products = [&](const i32x4_t (&w)[4], const i32x4_t (&x)[MT], bool anew) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[i], x[j], anew ? i32x16_t{} : acc[i][j],
                                                          0, 0, 0);
  };
  // one quarter: 4 MT products, and between them 4 + MT reads, `n` stores from
  // registers each followed by its load
  auto order = [&](auto n) {
#pragma unroll
    for (int k = 0; k < 4 * MT; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (k < MT) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      else if (k < 4) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      else if (2 * (k - 4) < 2 * decltype(n)::value && k - 4 < decltype(n)::value) {
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // ---- the first step goes to LDS, the second to registers
#pragma unroll
  for (int i = 0; i < LOADS; ++i) load(i);
  loaded();
#pragma unroll
  for (int i = 0; i < LOADS; ++i) store(0, i);
#pragma unroll
  for (int i = 0; i < LOADS; ++i) load(i);
  loaded();
  __syncthreads();
  read(0, 0, fw[0], fx[0]);
  int slot = 0;
  float sx_v = 0.0f, sw_v = 0.0f, bias_v = 0.0f;
  int turn = 0;  // the tile's place of scales
  auto scales_at = [&](int i) { return (float*)(lds + kWideScales + turn * 256 * 12) + i; };
  auto step = [&](auto anew) {
    read(slot, 1, fw[1], fx[1]);
#pragma unroll
    for (int i = 0; i < 6; ++i) store(slot ^ 1, i), load(i);
    products(fw[0], fx[0], decltype(anew)::value);
    order(std::integral_constant<int, 6>{});
    read(slot, 2, fw[0], fx[0]);
#pragma unroll
    for (int i = 6; i < 12; ++i) store(slot ^ 1, i), load(i);
    products(fw[1], fx[1], false);
    order(std::integral_constant<int, 6>{});
    read(slot, 3, fw[1], fx[1]);
#pragma unroll
    for (int i = 12; i < LOADS; ++i) store(slot ^ 1, i), load(i);
    products(fw[0], fx[0], false);
    order(std::integral_constant<int, LOADS - 12>{});
    loaded();
    if (decltype(anew)::value) {
      *scales_at(tid) = sx_v;
      *scales_at(256 + tid) = sw_v;
      *scales_at(512 + tid) = bias_v;
    }
    // the next step is whole in LDS, and nobody reads this one any more
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    slot ^= 1;
    read(slot, 0, fw[0], fx[0]);
    products(fw[1], fx[1], false);
    order(std::integral_constant<int, 0>{});
  };
  uint8_t* mine = lds + kWideTurn + wave * 4096;
  for (int at = first; at < run1; at += every) {
    int row0, col0;
    tile_at(at, row0, col0);
    sx_v = tid < BM && row0 + tid < M ? sx[row0 + tid] : 0.0f;
    // (the channel of w's row tid of the tile)
    const int64_t ch = ACT ? (int64_t)col0 / 2 + (tid >> 4) * 8 + (tid & 7) + (tid & 8 ? gate.F : 0)
                           : col0 + tid;
    sw_v = col0 + tid < N ? sw[ch] : 0.0f;
    bias_v = bias && col0 + tid < N ? widen16<DT>(bias[ch]) : 0.0f;
    step(std::true_type{});
    for (int t = 1; t < KT; ++t) step(std::false_type{});
    // the sums stay in accumulation registers until their block's turn
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) asm volatile("" : "+a"(acc[i][j]));

    // ---- results: register e of product (i, j) is channel 8 (e >> 2) + 4 h +
    // (e & 3) of its 32, token lane & 31; blocks of 32 tokens x 64 channels of y, the
    // 16-byte chunk c of token r at position c ^ (r & 7)
    const int width = N / HALVES, wcol = (col0 + wn * 128) / HALVES;
    // (hidden from the compiler, which would keep every address of this part
    // in registers all through the steps, and spill)
    int at_lane = lane;
    asm volatile("" : "+v"(at_lane));
    const int r = at_lane & 31, h = at_lane >> 5;
#pragma unroll
    for (int i0 = 0; i0 < 4; i0 += 2 * HALVES) {
      const float* sn = scales_at(256 + wn * 128 + i0 * 32 + 4 * h);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const int mrow = row0 + (wm * MT + j) * 32;
        const float s = *scales_at((wm * MT + j) * 32 + r);
#pragma unroll
        for (int i = 0; i < 2 * HALVES; ++i)
#pragma unroll
          for (int g = 0; g < 4 / HALVES; ++g) {
            // (the scales are read again for each block of tokens: held, they
            // would cost the registers that the next tile's rows wait in)
            const float* sg = sn + i * 32 + 8 * HALVES * g;
            const float4_t t = *(const float4_t*)sg, b = *(const float4_t*)(sg + 256);
            uint8_t* to = mine + r * 128 + (((i * (4 / HALVES) + g) ^ (r & 7)) << 4) + 8 * h;
            if constexpr (ACT != kNoGate)
              *(u32x2_t*)to = gated4<DT, ACT>(acc[i0 + i][j], g, s, t, b, *(const float4_t*)(sg + 8),
                                              *(const float4_t*)(sg + 264), gate);
            else
              *(u32x2_t*)to = results4<DT>(acc[i0 + i][j], g, s, t, b);
          }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_wave_barrier();
        const int c = at_lane & 7, n = wcol + i0 * 32 / HALVES + c * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tr = k * 8 + (at_lane >> 3);
          const u32x4_t v = *(const u32x4_t*)(mine + tr * 128 + ((c ^ (tr & 7)) << 4));
          if (mrow + tr < M && n < width)
            *(u32x4_t*)(out + (size_t)(mrow + tr) * width + n) = v;
        }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_wave_barrier();
      }
    }
    turn ^= 1;
  }
}

// Few tokens and channels: the call is the stream of w, spread over all CUs.
// One workgroup of 8 waves per 16 NT channels and all (at most 16 MB) tokens, on
// v_mfma_i32_16x16x64_i8; the waves take the steps of 128 codes (whole lines) in
// turn, straight from memory into registers (lane l: 16 codes of row l & 15),
// AHEAD steps of a wave under way, and their sums are joined in LDS.  MI355X: 16
// x 4096 x 11008 in 12.5 us, of which 4 do not depend on K (launch, first
// rows, join); the rest is w at 5.4 TB/s.
//
// FUSED: the tokens come in 16 bits, every workgroup quantizes them for itself
// into LDS while its first rows of w are on their way; each of 512 lanes holds
// 8 values of up to kRows rows of 4096 (a longer row counts as several).
constexpr int kRows = 4;

template <int DT, int MB, int NT, bool FUSED, int AHEAD>
__global__ void __launch_bounds__(512)
w8a8_stream_kernel(const void* __restrict__ x, int64_t x_stride, const float* __restrict__ sx,
                   const int8_t* __restrict__ wq, const float* __restrict__ sw,
                   const uint16_t* __restrict__ bias, uint16_t* __restrict__ out, int M, int N,
                   int K) {
  constexpr int kSum = 8 * NT * MB * 1024, kCodes = FUSED ? kRows * 4096 + 16 * 16 : 0;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kSum > kCodes ? kSum : kCodes];
  __shared__ uint32_t mags[FUSED ? kRows : 1][8];
  __shared__ float scales[16 * MB];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  const int col0 = (int)blockIdx.x * 16 * NT;
  const int KT = (K + 127) >> 7;
  const rsrc_t rw = make_rsrc(wq + (size_t)col0 * K, (uint32_t)min(16 * NT, N - col0) * (uint32_t)K);
  const uint32_t lane_off = (uint32_t)r * (uint32_t)K + 16u * g;
  auto load_w = [&](int s, i32x4_t (&w)[2][NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        w[e][i] = __builtin_bit_cast(
            i32x4_t, bld128(rw,
                            128 * s + 64 * e + 16 * g < K
                                ? lane_off + (uint32_t)(16 * i) * (uint32_t)K + 64 * e
                                : kOutOfRange,
                            s * 128));
  };
  i32x4_t w[AHEAD][2][NT];
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) load_w(wave + 8 * u, w[u]);

  rsrc_t rx;
  const int pitch = K + 16;  // FUSED: bytes of a row of codes in LDS
  if constexpr (FUSED) {
    const int per = (K + 4095) >> 12;  // pieces of 4096 per row
    u32x4_t raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int m = i / per, k = (i % per) * 4096 + tid * 8;
      raw[i] = u32x4_t{0, 0, 0, 0};
      if (m < M && k < K) raw[i] = *(const u32x4_t*)((const uint16_t*)x + m * x_stride + k);
      uint32_t mag = 0;
      float f[8];
      widen8<DT>(raw[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(f[j]));
      mag = lanes_max<64>(mag);
      if (lane == 0) mags[i][wave] = mag;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int m = i / per, k = (i % per) * 4096 + tid * 8;
      if (m >= M) break;
      uint32_t mag = 0;
      for (int p = m * per; p < (m + 1) * per; ++p)
#pragma unroll
        for (int v = 0; v < 8; ++v) mag = max(mag, mags[p][v]);
      float s = scale_of(mag);
      if (s == 0.0f) s = 1.0f;
      if (k < K) {
        float f[8];
        widen8<DT>(raw[i], f);
        *(u32x2_t*)(lds + m * pitch + k) = codes8(f, Codes8(s));
      }
      if (tid == 0) scales[m] = s;
    }
    __syncthreads();
  } else {
    rx = make_rsrc(x, (uint32_t)M * (uint32_t)K);
    if (tid < 16 * MB) scales[tid] = tid < M ? sx[tid] : 0.0f;
  }
  // tokens past the last repeat it (their results are not written)
  auto load_x = [&](int s, i32x4_t (&v)[2][MB]) {
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int m = min(16 * j + r, M - 1), k = 128 * s + 64 * e + 16 * g;
        if constexpr (FUSED)
          v[e][j] = *(const i32x4_t*)(lds + m * pitch + min(k, K - 16));
        else
          v[e][j] = __builtin_bit_cast(
              i32x4_t, bld128(rx, k < K ? (uint32_t)m * (uint32_t)K + 64 * e + 16u * g : kOutOfRange,
                              s * 128));
      }
  };
  i32x4_t xv[AHEAD][2][MB];
  if constexpr (!FUSED) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) load_x(wave + 8 * u, xv[u]);
  }

  i32x4_t acc[NT][MB];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  for (int s0 = wave; s0 < KT; s0 += 8 * AHEAD) {
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if constexpr (FUSED) load_x(s0 + 8 * u, xv[u]);
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int j = 0; j < MB; ++j)
            acc[i][j] =
                __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][e][i], xv[u][e][j], acc[i][j], 0, 0, 0);
      load_w(s0 + 8 * (u + AHEAD), w[u]);
      if constexpr (!FUSED) load_x(s0 + 8 * (u + AHEAD), xv[u]);
    }
  }

  // ---- join: lane holds channels 4 g .. 4 g + 3 of token r of each product
  if constexpr (FUSED) __syncthreads();  // the codes have been read
  i32x4_t* part = (i32x4_t*)lds;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) part[((wave * NT + i) * MB + j) * 64 + r * 4 + g] = acc[i][j];
  __syncthreads();
  for (int e = tid; e < NT * MB * 64; e += 512) {
    const int i = e / (64 * MB), j = e / 64 % MB, m = 16 * j + (e % 64) / 4, n = col0 + 16 * i + 4 * (e % 4);
    i32x4_t v = part[e];
#pragma unroll
    for (int p = 1; p < 8; ++p) v += part[p * NT * MB * 64 + e];
    if (m < M && n < N) {
      const float4_t t = *(const float4_t*)(sw + n);
      float y[4];
#pragma unroll
      for (int a = 0; a < 4; ++a)
        y[a] = result(v[a], scales[m], t[a], bias ? widen16<DT>(bias[n + a]) : 0.0f);
      *(u32x2_t*)(out + (size_t)m * N + n) = u32x2_t{pack16<DT>(y[0], y[1]), pack16<DT>(y[2], y[3])};
    }
  }
}

// The gated product of up to 16 tokens: the stream of w alone.  Workgroups of 16
// waves, teams of tw = 2, 4 or 8, stay, one on a CU, and each team takes groups of 8
// channels in turn, 8 rows of the gate and 8 of the up projection in one product on
// v_mfma_i32_16x16x64_i8; w is one buffer (less than 2 GB).
//
//  * Each workgroup has the tokens' codes in LDS, up to kCodes of them, brought
//    there once while its first rows of w are on their way (all of the tokens' loads
//    out first).  FUSED: from 16-bit rows of up to kFused values, which it quantizes
//    for itself; more of them (16 x 4096 take every CU 12 us) are quantized by a
//    launch before.
//  * A team's waves take the steps of 128 codes of a group in turn, straight from
//    memory into registers, AHEAD steps of a wave under way, across the groups'
//    borders: no group waits for its first rows.
//  * No wave waits for the others of its team: each leaves its sums of a group in
//    LDS and counts itself, and the last one to arrive joins them.  There are two
//    places in turn, and before a wave writes into one it sees (without a wait,
//    unless it is two groups ahead) that the group before there has been joined;
//    whoever joins that one waits for nobody, so the wait ends.
//
// The stream of w bounds it (MI355X, whole calls, F x K): 1 token 28672 x 8192 80 us, 5.9
// TB/s (95.7 in the form above, workgroups that end with their channels), 11008 x 4096
// 19.9, 16 tokens of that 23.1 (29 in 64 x 64 tiles), 27648 x 5120 57, 5.0 TB/s.
// With all 16 waves on one group and a barrier at its join it took 98 and 38 for the
// first and the third: the joins held up the loads.
constexpr int kCodes = 15 * 8192, kFused = 16384, kAhead = 4;

template <int DT, int ACT, bool FUSED>
__global__ void __launch_bounds__(1024)
w8a8_gated_stream_kernel(const void* __restrict__ x, int64_t x_stride,
                         const float* __restrict__ sx, const int8_t* __restrict__ wq, const float* __restrict__ sw,
                         const uint16_t* __restrict__ bias, uint16_t* __restrict__ out, int M,
                         int K, int tw, Gate gate) {
  constexpr int AHEAD = kAhead;
  __shared__ __attribute__((aligned(16))) uint8_t codes[kCodes + 16 * 16];
  __shared__ __attribute__((aligned(16))) i32x4_t part[2][16][64];
  __shared__ uint32_t arrived[2][8], joined[2][8];  // waves; groups, 1 more than the last
  __shared__ uint32_t mags[16];
  __shared__ float scales[16];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & (tw - 1);
  const int wave0 = __builtin_amdgcn_readfirstlane(tid >> 6) - wave, team = wave0 / tw;
  const int r = lane & 15, g = lane >> 4;
  const int groups = gate.F >> 3, KT = (K + 127) >> 7;
  const int first = (int)(blockIdx.x + gridDim.x * team), every = 16 / tw * (int)gridDim.x;
  // steps of a wave in a group, whole turns of its loads under way
  const int steps = ((KT - 1) / (tw * AHEAD) + 1) * AHEAD;

  // ---- w: the next step that is loaded
  const rsrc_t rw = make_rsrc(wq, (uint32_t)(2 * gate.F) * (uint32_t)K);
  int lgroup = first, lk = 128 * wave;
  uint32_t loff = (uint32_t)(lgroup * 8 + (r & 7) + (r & 8 ? gate.F : 0)) * (uint32_t)K + 16u * g;
  i32x4_t w[AHEAD][2];
  auto load = [&](int u) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
      w[u][e] = __builtin_bit_cast(
          i32x4_t, bld128(rw, lgroup < groups && lk + 64 * e + 16 * g < K ? loff + 64 * e : kOutOfRange, lk));
    lk += 128 * tw;
    if (lk >= 128 * tw * steps) {
      lk = 128 * wave;
      lgroup += every;
      loff += (uint32_t)every * 8u * (uint32_t)K;
    }
  };
#pragma unroll
  for (int u = 0; u < AHEAD; ++u) load(u);

  // ---- tokens: 16 bytes at a time, EACH values, unit i * 1024 + tid.  (its row: at
  // is below 2^13, so (at + 1/2) / per is further from an integer than fp32's
  // rounding moves it)
  constexpr int EACH = FUSED ? 8 : 16, HOLD = (FUSED ? kFused : kCodes) / EACH / 1024 + !FUSED;
  const int per = K / EACH, units = M * per, pitch = K + 16;
  const float rows_per_unit = 1.0f / (float)per;
  auto row_of = [&](int at) { return (int)(((float)at + 0.5f) * rows_per_unit); };
  u32x4_t raw[HOLD];
#pragma unroll
  for (int i = 0; i < HOLD; ++i) {
    const int at = i * 1024 + tid, m = row_of(at);
    raw[i] = u32x4_t{0, 0, 0, 0};
    if (at < units) {
      if constexpr (FUSED)
        raw[i] = *(const u32x4_t*)((const uint16_t*)x + m * x_stride + (at - m * per) * EACH);
      else
        raw[i] = *(const u32x4_t*)((const int8_t*)x + at * EACH);
    }
  }
  if (tid < 16) arrived[tid >> 3][tid & 7] = joined[tid >> 3][tid & 7] = 0;
  if constexpr (FUSED) {
    if (tid < 16) mags[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int at = i * 1024 + tid, m = row_of(at);
      if (i * 1024 >= units) break;
      uint32_t mag = 0;
      float f[8];
      widen8<DT>(raw[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) mag = max(mag, mag_bits(f[j]));
      if (__all(m == __builtin_amdgcn_readfirstlane(m))) {
        mag = lanes_max<64>(mag);
        if (lane == 0 && at < units) atomicMax(mags + m, mag);
      } else if (at < units) {
        atomicMax(mags + m, mag);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int at = i * 1024 + tid, m = row_of(at), k = (at - m * per) * 8;
      if (at >= units) break;
      float s = scale_of(mags[m]), f[8];
      if (s == 0.0f) s = 1.0f;
      widen8<DT>(raw[i], f);
      *(u32x2_t*)(codes + m * pitch + k) = codes8(f, Codes8(s));
      if (k == 0) scales[m] = s;
    }
  } else {
    if (tid < M) scales[tid] = sx[tid];
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int at = i * 1024 + tid, m = row_of(at);
      if (at < units) *(u32x4_t*)(codes + m * pitch + (at - m * per) * EACH) = raw[i];
    }
  }
  __syncthreads();

  // ---- groups.  (tokens past the last repeat it; their results are not written)
  const uint8_t* row = codes + min(r, M - 1) * pitch;
  for (int turn = 0, group = first; group < groups; ++turn, group += every) {
    i32x4_t acc = {0, 0, 0, 0};
    for (int j = 0; j < steps; j += AHEAD) {
      const int k = 128 * tw * j + 128 * wave + 16 * g;
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(
              w[u][e], *(const i32x4_t*)(row + min(k + 128 * tw * u + 64 * e, K - 16)), acc, 0, 0, 0);
        load(u);
      }
    }
    // ---- join: lane holds rows 4 g .. 4 g + 3 of the product, token r
    const int place = turn & 1;
    if (turn >= 2)
      while (__hip_atomic_load(&joined[place][team], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP) <
             (uint32_t)turn - 1)
        __builtin_amdgcn_s_sleep(1);
    asm volatile("" ::: "memory");
    part[place][wave0 + wave][r * 4 + g] = acc;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    uint32_t count = 0;
    if (lane == 0)
      count = __hip_atomic_fetch_add(&arrived[place][team], 1u, __ATOMIC_RELAXED,
                                     __HIP_MEMORY_SCOPE_WORKGROUP);
    count = __builtin_amdgcn_readfirstlane(count);
    asm volatile("" ::: "memory");
    if (count != (uint32_t)(tw * (turn >> 1) + tw - 1)) continue;
    i32x4_t v = part[place][wave0][lane];
    for (int p = 1; p < tw; ++p) v += part[place][wave0 + p][lane];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (lane == 0)
      __hip_atomic_store(&joined[place][team], (uint32_t)turn + 1, __ATOMIC_RELAXED,
                         __HIP_MEMORY_SCOPE_WORKGROUP);
    // lane: token lane / 4, of the gate channels 4 (lane & 1) .., of the up
    // projection where lane & 2
    const int m = lane >> 2, n = group * 8 + 4 * (lane & 1);
    float4_t t, b;
    channels4<DT>(sw, bias, (int64_t)n + (lane & 2 ? gate.F : 0), t, b);
    float y[4];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const float own = result(v[a], scales[min(m, M - 1)], t[a], b[a]);
      y[a] = gated<ACT>(own, __shfl_xor(own, 2, 64), gate);
    }
    if (m < M && !(lane & 2))
      *(u32x2_t*)(out + (size_t)m * gate.F + n) =
          u32x2_t{pack16<DT>(y[0], y[1]), pack16<DT>(y[2], y[3])};
  }
}

// --------------------------------------------------------------- dispatch ---
typedef Tile<2, 1, 2, 4, 4> T128;  // 128 x 128, 8 waves, alone on its CU
typedef Tile<1, 1, 2, 2, 4> T64;   // 64 x 64, 4 waves, two on a CU

// The operands of a call: 16-bit rows (with a stride) or codes with scales.
struct Args {
  const void* x;
  int64_t x_stride;
  const float* sx;
  const int8_t* wq;
  const float* sw;
  const uint16_t* bias;
  uint16_t* out;
  int M, N, K;
  Gate gate;  // of the gated kernels
  Split split;
};

template <int DT, class TL, int ACT>
void launch_tile(const Args& a, hipStream_t st) {
  const int mb = (int)ceil_div(a.M, TL::BM), nb = (int)ceil_div(a.N, TL::BN);
  const int per_xcd = (int)ceil_div((int64_t)mb * nb, 8);
  const unsigned splits = ACT ? (unsigned)a.split.splits : 1u;
  launch_timed(w8a8_tile_kernel<DT, TL, ACT>, dim3(per_xcd * 8 * splits), dim3(64 * TL::WAVES), 0, st,
               (const int8_t*)a.x, a.sx, a.wq, a.sw, a.bias, a.out, a.M, a.N, a.K, mb, nb, per_xcd,
               a.gate, a.split);
}

template <int DT, int MB, int NT, bool FUSED>
void launch_stream(const Args& a, hipStream_t st) {
  // rows of w under way per wave: where there is work before they are used,
  // 4 steps in all (1 x 4096 x 4096: 9.1 us with one step, 8.0 with four);
  // otherwise one, whose few registers leave room for a second workgroup
  // (16 x 4096 x 11008: 12.5 us, 13.4 with four; 8 x 5120 x 16384: 28, 30.2)
  constexpr int AHEAD = FUSED ? 4 / NT : 1;
  launch_timed(w8a8_stream_kernel<DT, MB, NT, FUSED, AHEAD>, dim3((unsigned)ceil_div(a.N, 16 * NT)),
               dim3(512), 0, st, a.x, a.x_stride, a.sx, a.wq, a.sw, a.bias, a.out, a.M, a.N, a.K);
}

// Whether w8a8_linear quantizes inside the product.
bool fused(int64_t M, int64_t K) { return M * ceil_div(K, 4096) <= kRows; }

template <int DT, int ACT, int MT>
void launch_wide(const Args& a, hipStream_t st) {
  const int mb = (int)ceil_div(a.M, 64 * MT), nb = (int)ceil_div(a.N, 256);
  const int per_xcd = (int)ceil_div((int64_t)mb * nb, 8);
  launch_timed(w8a8_wide_kernel<DT, ACT, MT>, dim3((unsigned)std::min(256, per_xcd * 8)), dim3(256), 0, st,
               (const int8_t*)a.x, a.sx, a.wq, a.sw, a.bias, a.out, a.M, a.N, a.K, mb, nb, per_xcd,
               a.gate);
}

// The kernel of a call.  A kernel's time per step of 128 codes was measured on
// MI355X as 0.3 us for 64 x 64 tiles while there is at most one per CU, and in
// proportion to their number beyond (two share a CU); 0.6 us per round of 256
// tiles of 128 x 128; 1.6 us per round of 256 of 256 x 256.  The rule takes the
// least sum.  Both sides of its borders (M x N x K, us):
//   64 / 128:   128 x 16384 x 5120 32.8 / 34.6, 512 x 1016 x 11008 26.3 / 38.1,
//               333 x 7168 x 5120 31.3 / 23.2, 512 x 5120 x 5120 30.8 / 23.6
//   128 / 256:  1024 x 5120 x 5120 46.0 / 55.4, 2048 x 4096 x 4096 46.9 / 50.4,
//               512 x 16384 x 5120 68.2 / 68.6, 2048 x 5120 x 5120 73.6 / 64.1,
//               1024 x 16384 x 5120 121.5 / 84.0
// and for few tokens by few channels, where 64 x 64 tiles are too few to ask
// memory for w at its rate, the stream kernel (stream / 64 x 64):
//   16 x 4096 x 11008 12.5 / 24.6, 16 x 8192 x 4096 11.2 / 11.8,
//   16 x 12288 x 4096 14.7 / 12.0, 32 x 4096 x 4096 8.8 / 11.6,
//   32 x 8192 x 4096 14.5 / 11.7, 64 x 4096 x 4096 12.5 / 12.0
template <int DT>
hipError_t launch_gemm_dt(const Args& a, hipStream_t st) {
  const int64_t t64 = ceil_div(a.M, 64) * ceil_div(a.N, 64);
  const int64_t t128 = ceil_div(a.M, 128) * ceil_div(a.N, 128);
  const int64_t t256 = ceil_div(a.M, 256) * ceil_div(a.N, 256);
  const int64_t c64 = 3 * std::max<int64_t>(t64, 256), c128 = 6 * 256 * ceil_div(t128, 256),
                c256 = 16 * 256 * ceil_div(t256, 256);
  if (a.M <= 64 && ceil_div(a.M, 16) * a.N < 12288) {
    if (a.M > 32) launch_stream<DT, 4, 1, false>(a, st);
    else if (a.M > 16) launch_stream<DT, 2, 1, false>(a, st);
    else launch_stream<DT, 1, 1, false>(a, st);
  } else if (c64 <= c128 && c64 <= c256) {
    launch_tile<DT, T64, kNoGate>(a, st);
  } else if (c128 <= c256) {
    launch_tile<DT, T128, kNoGate>(a, st);
  } else {
    launch_wide<DT, kNoGate, 4>(a, st);
  }
  return hipGetLastError();
}

hipError_t launch_gemm(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                       const void* bias, void* out, int64_t M, int64_t N, int64_t K, int dtype,
                       hipStream_t st) {
  const Args a = {xq, K, sx, wq, sw, (const uint16_t*)bias, (uint16_t*)out, (int)M, (int)N, (int)K, {}, {}};
  return (dtype == DT_F16 ? launch_gemm_dt<DT_F16> : launch_gemm_dt<DT_BF16>)(a, st);
}

// Channels per workgroup: 64 where that leaves two workgroups for each of 256
// CUs, else 32, else 16 (each reads and quantizes the tokens for itself).
template <int DT>
void launch_fused_dt(const Args& a, hipStream_t st) {
  if (a.N >= 512 * 64) launch_stream<DT, 1, 4, true>(a, st);
  else if (a.N >= 512 * 32) launch_stream<DT, 1, 2, true>(a, st);
  else launch_stream<DT, 1, 1, true>(a, st);
}

hipError_t launch_fused(const void* x, int64_t x_stride, const int8_t* wq, const float* sw,
                        const void* bias, void* out, int64_t M, int64_t N, int64_t K, int dtype,
                        hipStream_t st) {
  const Args a = {x, x_stride, nullptr, wq, sw, (const uint16_t*)bias, (uint16_t*)out, (int)M,
                  (int)N, (int)K, {}, {}};
  (dtype == DT_F16 ? launch_fused_dt<DT_F16> : launch_fused_dt<DT_BF16>)(a, st);
  return hipGetLastError();
}

// Whether w8a8_gated takes the kernel for few tokens, and whether that quantizes.
bool few_gated(int64_t M, int64_t F, int64_t K) {
  return M <= 16 && M * K <= kCodes && 2 * F * K < ((int64_t)1 << 31);
}
bool fused_gated(int64_t M, int64_t F, int64_t K) { return few_gated(M, F, K) && M * K <= kFused; }

// How the gated product of more tokens is formed: rows of a tile (64 x 64, 128 x
// 128, 192 x 256 or 256 x 256), and workgroups that share a tile's K.
//
// The rule takes the least sum of us as measured on MI355X: a step of 128 codes of a
// tile of 64 takes 0.3 (for at most one a CU, and in proportion beyond), of 128 0.45,
// or 0.6 in each of several rounds, of 192 1.4 and of 256 1.6 a round; a join of s
// splits 1 + 1.2 s and 4 + s.  Both sides (M x F x K, us, rows / splits):
//   17 x 1696 x 13408 64/1 35.3, 64/4 19.4; 14 x 272 x 19680 64/1 47.6, 64/8 18.8;
//   64 x 1376 x 4096 64/1 15.3, 64/3 12.4, 64/6 14.8; 128 x 2752 x 4096 64/1 15.6, 64/2
//   16.5; 571 x 904 x 10592 64/1 52.1, 128/1 57.2, 128/3 39.0; 139 x 5192 x 16224 64/1
//   95.6, 128/1 87.2; 333 x 13824 x 5120 128/1 96, 192 72.9, 256 81.7; 1024 x 11008 x
//   4096 128/1 141, 192 130, 256 119
struct GatedPlan {
  int rows, splits;
  int64_t tiles;
};
constexpr int64_t kSplit64 = 512, kSplit128 = 256;  // workgroups of a split call, at most
GatedPlan plan_gated(int64_t M, int64_t F, int64_t K) {
  const int64_t N = 2 * F, KT = ceil_div(K, 128);
  GatedPlan best = {0, 1, 0};
  double least = 1e30;
  auto offer = [&](int rows, int splits, int64_t tiles, double us) {
    if (us < least) least = us, best = {rows, splits, tiles};
  };
  const int64_t t64 = ceil_div(M, 64) * ceil_div(N, 64), t128 = ceil_div(M, 128) * ceil_div(N, 128);
  const int64_t t192 = ceil_div(M, 192) * ceil_div(N, 256), t256 = ceil_div(M, 256) * ceil_div(N, 256);
  for (int s = 1; s <= 16 && (s == 1 || 4 * s <= KT); ++s) {
    const double steps = (double)ceil_div(KT, s);
    if (ceil_div(KT, ceil_div(KT, s)) != s) continue;  // a split would have none
    if (s == 1 || t64 * s <= kSplit64)
      offer(64, s, t64, 0.3 * steps * std::max(1.0, t64 * s / 256.0) + (s > 1 ? 1 + 1.2 * s : 0));
    if (s == 1 || t128 * s <= kSplit128)
      offer(128, s, t128, (t128 * s <= 256 ? 0.45 : 0.6 * ceil_div(t128 * s, 256)) * steps +
                              (s > 1 ? 4 + s : 0));
  }
  offer(192, 1, t192, 1.4 * KT * ceil_div(t192, 256));
  offer(256, 1, t256, 1.6 * KT * ceil_div(t256, 256));
  return best;
}
// Bytes of the sums and counters of any plan for up to M tokens (a plan of fewer may
// split K where that of more does not): plan_gated's limits on the tiles of a split call.
int64_t split_bytes(int64_t M, int64_t F, int64_t K) {
  const int64_t N = 2 * F, most = std::min<int64_t>(16, ceil_div(K, 128) / 4);
  if (most < 2) return 0;
  auto sums = [&](int64_t rows, int64_t limit) -> int64_t {
    const int64_t column = ceil_div(N, rows);  // tiles of the least M
    if (2 * column > limit) return 0;
    return std::min(limit, ceil_div(M, rows) * column * most) * rows * rows * 4;
  };
  const int64_t bytes = std::max(sums(64, kSplit64), sums(128, kSplit128));
  return bytes ? pad256(kSplit64 / 2 * 4) + bytes : 0;
}

template <int DT, int ACT, bool FUSED>
void launch_gated_stream(const Args& a, hipStream_t st) {
  // waves of a team: as many as waste the fewest steps (a wave's are padded to
  // turns of kAhead).  MI355X, 8 / 2 of them: 16 tokens by 27648 x 5120 (40 steps)
  // 61.1 / 57.0 us, by 8192 x 4096 (32 steps, none wasted) 19.0 / 21.0
  const int64_t KT = ceil_div(a.K, 128);
  int tw = 2;
  for (int n : {4, 8})
    if (ceil_div(KT, n * kAhead) * n <= ceil_div(KT, tw * kAhead) * tw) tw = n;
  launch_timed(w8a8_gated_stream_kernel<DT, ACT, FUSED>,
               dim3((unsigned)std::min(a.gate.F >> 3, 256)), dim3(1024), 0, st, a.x, a.x_stride, a.sx,
               a.wq, a.sw, a.bias, a.out, a.M, a.K, tw, a.gate);
}
template <int DT, int ACT>
hipError_t launch_gated_dt(const Args& a, const GatedPlan& p, hipStream_t st) {
  if (!a.sx) launch_gated_stream<DT, ACT, true>(a, st);
  else if (few_gated(a.M, a.gate.F, a.K)) launch_gated_stream<DT, ACT, false>(a, st);
  else if (p.rows == 64) launch_tile<DT, T64, ACT>(a, st);
  else if (p.rows == 128) launch_tile<DT, T128, ACT>(a, st);
  else if (p.rows == 192) launch_wide<DT, ACT, 3>(a, st);
  else launch_wide<DT, ACT, 4>(a, st);
  return hipGetLastError();
}

// A gated call on 16-bit rows (sx null) or on codes.
hipError_t launch_gated(const Args& a, const GatedPlan& p, int act, int dtype, hipStream_t st) {
  if (act == W4A16_GELU)
    return (dtype == DT_F16 ? launch_gated_dt<DT_F16, kErf> : launch_gated_dt<DT_BF16, kErf>)(a, p, st);
  return (dtype == DT_F16 ? launch_gated_dt<DT_F16, kSigmoid>
                          : launch_gated_dt<DT_BF16, kSigmoid>)(a, p, st);
}

// --------------------------------------------------------------- checking ---
constexpr int64_t kMaxM = (int64_t)1 << 21, kMaxN = (int64_t)1 << 24, kMaxK = (int64_t)1 << 17;

int validate_shape(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || N <= 0 || K <= 0 || K % 16 != 0 || N % 8 != 0) return W4A16_ERR_INVALID_ARG;
  if (M > kMaxM || N > kMaxN || K > kMaxK || M * N > ((int64_t)1 << 36))
    return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

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
  return linear && !fused(M, K) ? linear_bytes(M, K) : 0;
}

int w8a8_gemm(const int8_t* xq, const float* x_scale, const int8_t* wq, const float* w_scale,
              const void* bias, void* out, int64_t M, int64_t N, int64_t K, int32_t dtype,
              void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    if (int s = validate_shape(M, N, K)) return s;
    if (int s = validate_dtype(dtype)) return s;
    if (int s = check_ptrs({xq, x_scale, wq, w_scale, out})) return s;
    if (!aligned16(bias) || !aligned16(workspace)) return W4A16_ERR_MISALIGNED;
    (void)workspace_bytes;  // none is needed
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
    if (fused(M, K))
      return hip_status(launch_fused(x, x_stride, wq, w_scale, bias, out, M, N, K, dtype, st));
    int8_t* xq = (int8_t*)workspace;
    float* sx = (float*)(xq + pad256(M * K));
    if (int s = hip_status(launch_quantize(x, M, K, x_stride, dtype, xq, sx, st))) return s;
    return hip_status(launch_gemm(xq, sx, wq, w_scale, bias, out, M, N, K, dtype, st));
  });
}

int64_t w8a8_gated_workspace_bytes(int64_t M, int64_t F, int64_t K) {
  if (F <= 0 || F > kMaxN || F % 8 != 0 || validate_shape(M, 2 * F, K) != W4A16_OK) return -1;
  if (fused_gated(M, F, K)) return 0;
  return linear_bytes(M, K) + (few_gated(M, F, K) ? 0 : split_bytes(M, F, K));
}

int w8a8_gated_plan(int64_t M, int64_t F, int64_t K, char* names_host, int64_t names_bytes,
                    int64_t* names_len_host) {
  return guarded([&]() -> int {
    if (F <= 0 || F % 8 != 0) return W4A16_ERR_INVALID_ARG;
    if (F > kMaxN) return W4A16_ERR_UNSUPPORTED;
    if (int s = validate_shape(M, 2 * F, K)) return s;
    if (names_bytes < 0 || (names_bytes > 0 && !names_host)) return W4A16_ERR_INVALID_ARG;
    char names[96];
    const char* quantize = fused_gated(M, F, K) ? "" : "w8a8_quantize_kernel + ";
    const GatedPlan p = plan_gated(M, F, K);
    if (few_gated(M, F, K))
      snprintf(names, sizeof names, "%sw8a8_gated_stream_kernel", quantize);
    else if (p.rows <= 128)
      snprintf(names, sizeof names, "%sw8a8_tile_kernel %dx%d/%d", quantize, p.rows, p.rows, p.splits);
    else
      snprintf(names, sizeof names, "%sw8a8_wide_kernel %dx256", quantize, p.rows);
    if (names_bytes > 0) snprintf(names_host, (size_t)names_bytes, "%s", names);
    if (names_len_host) *names_len_host = (int64_t)strlen(names);
    return W4A16_OK;
  });
}

int w8a8_gated(const void* x, int64_t x_stride, const int8_t* wq, const float* w_scale,
               const void* bias, int32_t act, void* out, int64_t M, int64_t F, int64_t K,
               int32_t dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    if (F <= 0 || F % 8 != 0) return W4A16_ERR_INVALID_ARG;
    if (F > kMaxN) return W4A16_ERR_UNSUPPORTED;
    if (int s = validate_shape(M, 2 * F, K)) return s;
    if (int s = validate_dtype(dtype)) return s;
    if (act < W4A16_SILU || act > W4A16_GELU_TANH) return W4A16_ERR_INVALID_ARG;
    if (x_stride < K || x_stride % 8 != 0) return W4A16_ERR_INVALID_ARG;
    if (int s = check_ptrs({x, wq, w_scale, out})) return s;
    if (!aligned16(bias) || !aligned16(workspace)) return W4A16_ERR_MISALIGNED;
    const int64_t need = w8a8_gated_workspace_bytes(M, F, K);
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
    // x is read while other workgroups write out
    const int64_t from = (int64_t)(intptr_t)x, to = (int64_t)(intptr_t)out;
    if (to < from + 2 * ((M - 1) * x_stride + K) && from < to + 2 * M * F) return W4A16_ERR_INVALID_ARG;
    clear_pending_error();
    const hipStream_t st = (hipStream_t)stream;
    // sigmoid(a g + b g^3): 1 and 0, or 2 sqrt(2 / pi) (1 and 0.044715); times log2 e
    const float log2e = 1.4426950408889634f;
    const float a1 = act == W4A16_SILU ? log2e : 1.5957691216057308f * log2e;
    Args a = {x, x_stride, nullptr, wq, w_scale, (const uint16_t*)bias, (uint16_t*)out, (int)M,
              (int)(2 * F), (int)K, {(int)F, a1, act == W4A16_SILU ? 0.0f : 0.044715f * a1}, {1, nullptr, nullptr}};
    GatedPlan p = {0, 1, 0};
    if (!fused_gated(M, F, K)) {
      if (!few_gated(M, F, K)) p = plan_gated(M, F, K);
      int8_t* xq = (int8_t*)workspace;
      float* sx = (float*)(xq + pad256(M * K));
      uint32_t* count = (uint32_t*)(xq + linear_bytes(M, K));
      if (int s = hip_status(launch_quantize(x, M, K, x_stride, dtype, xq, sx, st, count,
                                             p.splits > 1 ? (int)p.tiles : 0)))
        return s;
      a.x = xq;
      a.sx = sx;
      a.split = {p.splits, (int32_t*)(count + pad256(p.tiles * 4) / 4), count};
    }
    return hip_status(launch_gated(a, p, act, dtype, st));
  });
}

}  // extern "C"
