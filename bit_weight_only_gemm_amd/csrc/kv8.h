// kv8.h -- layout and argument checks of the paged 8-bit key/value cache,
// shared by the append, read-back and attention kernels.
//
// A page holds T = 16, 32, 64 or 128 tokens of every kv head; one head of one
// page is T / 16 subtiles of 16 tokens x D channels, 16 D bytes each:
//   k  [page][head][T / 16][16 tokens][D]     (that is [T][D])
//   v  [page][head][T / 16][D][16 tokens]     (tokens innermost)
// so that the attention's matrix instructions take both straight from memory:
// a lane's 16-byte piece of k is 16 channels of one token, of v one channel of
// 16 tokens, in each case along the axis that product sums over.  A code byte c
// stands for (c - 128) * scale, one fp32 scale per (page, head).
#pragma once
#include "abi.h"
#include "quant8.h"

namespace w4a16 {

// Device arguments of a cache and of the sequences in it.  Entries of the
// table, lengths and offsets live in device memory and are not known to the
// host: the kernels bring each into range before an address is formed from
// it, so a wrong one gives unspecified values but no access out of bounds.
struct Kv8 {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  const int32_t* table;  // [B, width]
  const int32_t* lens;   // [B] tokens of each sequence, the new ones included
  const int32_t* cu;     // [B + 1] first new token of each sequence, or null: one each
  int pages, width, B, tokens, max_new, H, Hkv, lgT;
};

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return min(max(v, lo), hi); }

// Sequence b: its first new token, how many of them are processed (at most
// max_new), the first one's position (below 0 where there are more new tokens
// than the sequence has), and its length.
struct Kv8Seq {
  int tok, n, first, len;
};
__device__ __forceinline__ Kv8Seq kv8_seq(const Kv8& c, int b) {
  Kv8Seq s;
  if (c.cu) {
    s.tok = clamp_int(c.cu[b], 0, c.tokens);
    s.n = clamp_int(c.cu[b + 1], s.tok, c.tokens) - s.tok;
  } else {
    s.tok = b;
    s.n = 1;
  }
  s.len = (int)min((int64_t)max(c.lens[b], 0), (int64_t)c.width << c.lgT);
  s.first = s.len - s.n;
  s.n = min(s.n, c.max_new);
  return s;
}
__device__ __forceinline__ int kv8_page(const Kv8& c, int b, int index) {
  return clamp_int(c.table[(int64_t)b * c.width + index], 0, c.pages - 1);
}

inline int log2_page(int32_t T) { return T == 16 ? 4 : T == 32 ? 5 : T == 64 ? 6 : T == 128 ? 7 : -1; }

inline int validate_kv8(int64_t pages, int32_t T, int64_t width, int64_t tokens, int64_t B,
                        int64_t max_new, int32_t H, int32_t Hkv, int32_t D, const void* cu) {
  if (pages <= 0 || width <= 0 || tokens < 0 || B < 0 || max_new < 0 || H <= 0 || Hkv <= 0 ||
      H % Hkv != 0)
    return W4A16_ERR_INVALID_ARG;
  if (!cu && (tokens != B || max_new > 1)) return W4A16_ERR_INVALID_ARG;
  if (log2_page(T) < 0 || (D != 64 && D != 128)) return W4A16_ERR_UNSUPPORTED;
  // 32-bit indices of tokens, pages, table entries and workgroups
  if (pages > (1 << 30) || B > (1 << 20) || tokens > (1 << 24) || H > 1024 ||
      width * T > ((int64_t)1 << 30) || max_new > tokens)
    return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

// A row stride in elements, rows of `row` elements.
inline bool bad_stride(int64_t stride, int64_t row) { return stride < row || stride % 8 != 0; }

}  // namespace w4a16
