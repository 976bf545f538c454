// w8a8.hip -- matrix products of 8-bit integers with one scale per token
// (row of x) and per output channel (row of w), and the quantizer that makes
// such rows:
//
//   y[m, n] = round16( fp32(sum_k cx[m, k] cw[n, k]) * (sx[m] * sw[n]) + b[n] ).
//
// The sum is exact in int32 (|c| <= 127 and K <= 2^17), so it does not depend
// on any split of K.
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
                     float* __restrict__ scales) {
  constexpr int HOLD = kHeld / (8 * LANES), BYTES = DT == 2 ? 4 : 2, PARTS = BYTES / 2;
  __shared__ uint32_t part[LANES / 64];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int64_t base = row * stride;
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
                        float* scales, hipStream_t st) {
  if (M < kFewRows)
    hipLaunchKernelGGL((w8a8_quantize_kernel<DT, 1024>), dim3((unsigned)M), dim3(1024), 0, st, x,
                       stride, (int)K, codes, scales);
  else
    hipLaunchKernelGGL((w8a8_quantize_kernel<DT, 256>), dim3((unsigned)M), dim3(256), 0, st, x,
                       stride, (int)K, codes, scales);
}

hipError_t launch_quantize(const void* x, int64_t M, int64_t K, int64_t stride, int dtype,
                           int8_t* codes, float* scales, hipStream_t st) {
  (dtype == W4A16_F16    ? launch_quantize_dt<DT_F16>
   : dtype == W4A16_BF16 ? launch_quantize_dt<DT_BF16>
                         : launch_quantize_dt<2>)(x, M, K, stride, codes, scales, st);
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
template <int DT, class TL>
__global__ void __launch_bounds__(64 * TL::WAVES)
w8a8_tile_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                 const int8_t* __restrict__ wq, const float* __restrict__ sw,
                 const uint16_t* __restrict__ bias, uint16_t* __restrict__ out, int M, int N,
                 int K, int mb, int nb, int per_xcd) {
  constexpr int MT = TL::MT, NT = TL::NT, NS = TL::NS, L = TL::LOADS;
  __shared__ __attribute__((aligned(16))) uint8_t lds[NS * TL::STAGE];
  // ---- tile of this workgroup: workgroups go to the 8 XCDs in turn, so each
  // XCD takes a contiguous run of tiles, ordered in bands of 8 row blocks
  const int at = (int)(blockIdx.x & 7) * per_xcd + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || at >= mb * nb) return;
  const int band = at / (8 * nb), in_band = at % (8 * nb);
  const int bh = min(8, mb - band * 8);
  const int row0 = (band * 8 + in_band % bh) * TL::BM, col0 = in_band / bh * TL::BN;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const int KT = (K + 127) >> 7;
  const rsrc_t rw = make_rsrc(wq + (size_t)col0 * K, (uint32_t)min(TL::BN, N - col0) * (uint32_t)K);
  const rsrc_t rx = make_rsrc(xq + (size_t)row0 * K, (uint32_t)min(TL::BM, M - row0) * (uint32_t)K);

  // load i of this wave fills the LDS block WAVES i + wave (8 rows); blocks
  // below BN / 8 are rows of w
  const int lrow = lane >> 3;
  auto load = [&](int t, int i) {
    const int blk = TL::WAVES * i + wave;
    const bool is_w = blk < TL::BN / 8;
    const uint32_t row = 8u * (uint32_t)(is_w ? blk : blk - TL::BN / 8) + (uint32_t)lrow;
    const uint32_t chunk = ((uint32_t)lane & 7u) ^ ((row >> 1) & 7u);
    const uint32_t off =
        128 * t + 16 * (int)chunk < K ? row * (uint32_t)K + 16u * chunk : kOutOfRange;
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

  // ---- results: register i of product (nt, mt) is channel 8 (i >> 2) + 4 h +
  // (i & 3) of its 32, token lane & 31; one 32-token block of the wave at a time
  constexpr int ROW = NT * 64 + 16;  // bytes of a token's row in LDS
  static_assert(TL::WAVES * 32 * ROW <= NS * TL::STAGE, "the results fit");
  uint8_t* mine = lds + wave * 32 * ROW;
  const int wcol = col0 + wn * NT * 32;
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int mrow = row0 + (wm * MT + j) * 32;
    const float s = mrow + r < M ? sx[mrow + r] : 0.0f;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int n = wcol + i * 32 + 8 * g + 4 * h;
        float4_t t = {0, 0, 0, 0}, b = {0, 0, 0, 0};
        if (n < N) {
          t = *(const float4_t*)(sw + n);
          if (bias) {
            const u32x2_t w = *(const u32x2_t*)(bias + n);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              b[e] = widen16<DT>((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
          }
        }
        *(u32x2_t*)(mine + r * ROW + i * 64 + 16 * g + 8 * h) = results4<DT>(acc[i][j], g, s, t, b);
      }
    constexpr int LR = NT * 4;  // lanes per row
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int k = 0; k < 32 / (64 / LR); ++k) {
      const int tr = k * (64 / LR) + lane / LR, c = (lane % LR) * 8;
      const u32x4_t v = *(const u32x4_t*)(mine + tr * ROW + c * 2);
      if (mrow + tr < M && wcol + c < N) *(u32x4_t*)(out + (size_t)(mrow + tr) * N + wcol + c) = v;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// The same product for many tokens: workgroups stay and take 256 x 256 tiles
// in turn, 4 waves of 4 x 4 products.  K goes by in steps of 128 codes (whole
// 128-byte lines of w and x), four quarters of 32 each:
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
// per workgroup and loads straight to LDS it took 2324 us).
constexpr int kWideStage = 512 * 128, kWideTurn = 2 * kWideStage, kWideScales = kWideTurn + 4 * 4096;
// x's scales, w's, the bias as fp32; of this tile and of the one before
constexpr int kWideLds = kWideScales + 2 * 256 * 12;

template <int DT>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1)))
w8a8_wide_kernel(const int8_t* __restrict__ xq, const float* __restrict__ sx,
                 const int8_t* __restrict__ wq, const float* __restrict__ sw,
                 const uint16_t* __restrict__ bias, uint16_t* __restrict__ out, int M, int N,
                 int K, int mb, int nb, int per_xcd) {
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
    row0 = (band * 8 + in_band % bh) * 256;
    col0 = in_band / bh * 256;
  };

  // ---- loads: instruction i of a step fetches 8 rows x 128 bytes, i < 8 rows
  // of w and i >= 8 rows of x, of rows 64 wave + 8 (i & 7) of the tile
  const int lrow = lane >> 3, lchunk = lane & 7;
  const uint32_t lane_off = (uint32_t)(64 * wave + lrow) * (uint32_t)K + 16u * lchunk;
  const uint32_t tail = 128 * (KT - 1) + 16 * lchunk >= K ? kOutOfRange : 0u;
  const uint32_t lane_lds = (uint32_t)(64 * wave + lrow) * 128 + 16u * (lchunk ^ ((lrow >> 1) & 3));
  int lat = first, lt = 0;  // the step that is loaded next
  rsrc_t rw, rx;
  auto aim = [&]() {
    int row0 = 0, col0 = 0;
    const bool any = lat < run1;
    if (any) tile_at(lat, row0, col0);
    rw = make_rsrc(wq + (size_t)col0 * K, any ? (uint32_t)min(256, N - col0) * (uint32_t)K : 0u);
    rx = make_rsrc(xq + (size_t)row0 * K, any ? (uint32_t)min(256, M - row0) * (uint32_t)K : 0u);
  };
  aim();
  i32x4_t held[16];
  auto load = [&](int i) {
    const uint32_t off = (lane_off + (uint32_t)(8 * (i & 7)) * (uint32_t)K) | (lt == KT - 1 ? tail : 0u);
    held[i] = __builtin_bit_cast(i32x4_t, bld128(i < 8 ? rw : rx, off, lt * 128));
  };
  auto loaded = [&]() {  // every load of a step is out
    if (++lt == KT) {
      lt = 0;
      lat += every;
      aim();
    }
  };
  // row 64 wave + 8 i + lrow: (row >> 1) & 7 is ((lrow >> 1) & 3) + 4 (i & 1)
  auto store = [&](int slot, int i) {
    *(i32x4_t*)(lds + slot * kWideStage + (i < 8 ? 0 : 32768) + (i & 7) * 1024 +
                (lane_lds ^ ((i & 1) << 6))) = held[i];
  };

  const int r = lane & 31, h = lane >> 5;
  i32x4_t fw[2][4], fx[2][4];
  auto read = [&](int slot, int quarter, i32x4_t (&w)[4], i32x4_t (&x)[4]) {
    const uint8_t* st = lds + slot * kWideStage + (((2 * quarter + h) ^ ((r >> 1) & 7)) << 4) + r * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *(const i32x4_t*)(st + wn * 16384 + i * 4096);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *(const i32x4_t*)(st + 32768 + wm * 16384 + i * 4096);
  };
  i32x16_t acc[4][4];
  auto products = [&](const i32x4_t (&w)[4], const i32x4_t (&x)[4], bool anew) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(w[i], x[j], anew ? i32x16_t{} : acc[i][j],
                                                          0, 0, 0);
  };
  // one quarter: 16 products, and between them 8 reads, `n` stores from
  // registers each followed by its load
  auto order = [&](auto n) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (k < 4) __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      else if (2 * (k - 4) < 2 * decltype(n)::value && k - 4 < decltype(n)::value) {
        __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  // ---- the first step goes to LDS, the second to registers
#pragma unroll
  for (int i = 0; i < 16; ++i) load(i);
  loaded();
#pragma unroll
  for (int i = 0; i < 16; ++i) store(0, i);
#pragma unroll
  for (int i = 0; i < 16; ++i) load(i);
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
    for (int i = 12; i < 16; ++i) store(slot ^ 1, i), load(i);
    products(fw[0], fx[0], false);
    order(std::integral_constant<int, 4>{});
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
    sx_v = row0 + tid < M ? sx[row0 + tid] : 0.0f;
    sw_v = col0 + tid < N ? sw[col0 + tid] : 0.0f;
    bias_v = bias && col0 + tid < N ? widen16<DT>(bias[col0 + tid]) : 0.0f;
    step(std::true_type{});
    for (int t = 1; t < KT; ++t) step(std::false_type{});
    // the sums stay in accumulation registers until their block's turn
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) asm volatile("" : "+a"(acc[i][j]));

    // ---- results: register e of product (i, j) is channel 8 (e >> 2) + 4 h +
    // (e & 3) of its 32, token lane & 31; blocks of 32 tokens x 64 channels, the
    // 16-byte chunk c of token r at position c ^ (r & 7)
    const int wcol = col0 + wn * 128;
    // (hidden from the compiler, which would keep every address of this part
    // in registers all through the steps, and spill)
    int at_lane = lane;
    asm volatile("" : "+v"(at_lane));
    const int r = at_lane & 31, h = at_lane >> 5;
#pragma unroll
    for (int i0 = 0; i0 < 4; i0 += 2) {
      const float* sn = scales_at(256 + wn * 128 + i0 * 32 + 4 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int mrow = row0 + (wm * 4 + j) * 32;
        const float s = *scales_at((wm * 4 + j) * 32 + r);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            // (the scales are read again for each block of tokens: held, they
            // would cost the registers that the next tile's rows wait in)
            const float4_t t = *(const float4_t*)(sn + i * 32 + 8 * g);
            const float4_t b = *(const float4_t*)(sn + 256 + i * 32 + 8 * g);
            *(u32x2_t*)(mine + r * 128 + (((i * 4 + g) ^ (r & 7)) << 4) + 8 * h) =
                results4<DT>(acc[i0 + i][j], g, s, t, b);
          }
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_wave_barrier();
        const int c = at_lane & 7, n = wcol + i0 * 32 + c * 8;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int tr = k * 8 + (at_lane >> 3);
          const u32x4_t v = *(const u32x4_t*)(mine + tr * 128 + ((c ^ (tr & 7)) << 4));
          if (mrow + tr < M && n < N)
            *(u32x4_t*)(out + (size_t)(mrow + tr) * N + n) = v;
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
};

template <int DT, class TL>
void launch_tile(const Args& a, hipStream_t st) {
  const int mb = (int)ceil_div(a.M, TL::BM), nb = (int)ceil_div(a.N, TL::BN);
  const int per_xcd = (int)ceil_div((int64_t)mb * nb, 8);
  launch_timed(w8a8_tile_kernel<DT, TL>, dim3((unsigned)per_xcd * 8), dim3(64 * TL::WAVES), 0, st,
               (const int8_t*)a.x, a.sx, a.wq, a.sw, a.bias, a.out, a.M, a.N, a.K, mb, nb, per_xcd);
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

template <int DT>
void launch_wide(const Args& a, hipStream_t st) {
  const int mb = (int)ceil_div(a.M, 256), nb = (int)ceil_div(a.N, 256);
  const int per_xcd = (int)ceil_div((int64_t)mb * nb, 8);
  launch_timed(w8a8_wide_kernel<DT>, dim3((unsigned)std::min(256, per_xcd * 8)), dim3(256), 0, st,
               (const int8_t*)a.x, a.sx, a.wq, a.sw, a.bias, a.out, a.M, a.N, a.K, mb, nb, per_xcd);
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
    launch_tile<DT, T64>(a, st);
  } else if (c128 <= c256) {
    launch_tile<DT, T128>(a, st);
  } else {
    launch_wide<DT>(a, st);
  }
  return hipGetLastError();
}

hipError_t launch_gemm(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw,
                       const void* bias, void* out, int64_t M, int64_t N, int64_t K, int dtype,
                       hipStream_t st) {
  const Args a = {xq, K, sx, wq, sw, (const uint16_t*)bias, (uint16_t*)out, (int)M, (int)N, (int)K};
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
                  (int)N, (int)K};
  (dtype == DT_F16 ? launch_fused_dt<DT_F16> : launch_fused_dt<DT_BF16>)(a, st);
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

}  // extern "C"
