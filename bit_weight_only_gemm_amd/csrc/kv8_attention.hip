// kv8_attention.hip -- the entry points of attention over the paged 8-bit cache,
// and its kernels for scores as they are.
#include "kv8_attention.h"

namespace w4a16 {
namespace {

// Up to 128 rows of a kv head go to the decode kernel in tiles of 16, which
// follow one another on one die and find the keys in its cache; more to the
// prompt kernel (MI355X, 24 sequences of 4001 tokens, 4 kv heads of 64: 40 rows
// 28 us against 46 in the prompt kernel's form, 128 rows 45 against 53).
// Splits of the keys: two workgroups for each of 256 CUs in all (64 sequences
// of 8192 tokens, 8 kv heads of 128: 186 us; with 1024 workgroups 192, with thrice
// those 215), no split below 8 units, two a wave (with 4, one sequence of 777
// tokens and 32 kv heads takes 8.7 us instead of 9.7, but 8 of 2000 and 8 kv heads
// 12.6 instead of 11.1 and one of 20000 26.5 instead of 20.1: the join grows with
// the splits); the prompt kernel's 4.
Plan plan_attention(int64_t B, int64_t max_new, int64_t max_len, int H, int Hkv, int D) {
  Plan p;
  const int64_t rows = max_new * (H / Hkv);
  p.waves = rows <= 128 ? 0 : D == 64 ? kPromptWaves<64> : kPromptWaves<128>;
  p.rows = p.waves ? 32 * p.waves : 16;
  p.row_tiles = (int)ceil_div(rows, p.rows);
  const int64_t nu = std::max<int64_t>(1, ceil_div(max_len, kUnit));
  const int64_t groups = B * Hkv * p.row_tiles;
  const int64_t want = ceil_div(kWanted, groups);
  p.units = (int)(p.waves ? std::max<int64_t>(4, ceil_div(nu, want)) : 8);
  p.splits = (int)std::min(ceil_div(nu, p.units), want);
  return p;
}

// The workspace begins with the decode kernel's counters, at the same place
// in every call: they are zero between calls, whatever the calls' sizes.
int64_t part_bytes(const Plan& p, int64_t tokens, int H, int D) {
  if (p.splits == 1) return 0;
  const int64_t rows = tokens * H * p.splits;
  return kCounters * 4 + pad256(rows * D * 4) + pad256(rows * 8);
}

int attention(int mode, const void* q, int64_t q_stride, const uint8_t* k_cache,
              const uint8_t* v_cache,
              const float* k_scale, const float* v_scale, int64_t num_pages, int32_t page_size,
              const int32_t* page_table, int64_t max_pages, const int32_t* seq_lens,
              const int32_t* cu_seqlens, float scale, int32_t causal, const Scoring& sc, void* out,
              int64_t out_stride, float* lse, int64_t tokens, int64_t B, int64_t max_new,
              int64_t max_len, int32_t H, int32_t Hkv, int32_t D, int32_t dtype, void* workspace,
              int64_t workspace_bytes, void* stream) {
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
    for (const void* p : {(const void*)cu_seqlens, (const void*)lse, (const void*)workspace,
                          (const void*)sc.slopes, (const void*)sc.first, (const void*)sc.prefix,
                          (const void*)sc.end})
      if (!aligned16(p)) return W4A16_ERR_MISALIGNED;
    const Plan p = plan_attention(B, max_new, max_len, H, Hkv, D);
    const int64_t need = part_bytes(p, tokens, H, D);
    if (need > 0 && (!workspace || workspace_bytes < need)) return W4A16_ERR_WORKSPACE;
    // (the join's grid is smaller: it runs where there are less than 512 row tiles)
    if (too_large(8 * ceil_div(B * Hkv * p.splits, 8) * p.row_tiles, p.waves ? 64 * p.waves : 256))
      return W4A16_ERR_UNSUPPORTED;
    clear_pending_error();
    const Kv8 c = {const_cast<uint8_t*>(k_cache), const_cast<uint8_t*>(v_cache),
                   const_cast<float*>(k_scale), const_cast<float*>(v_scale), page_table, seq_lens,
                   cu_seqlens, (int)num_pages, (int)max_pages, (int)B, (int)tokens, (int)max_new, H,
                   Hkv, log2_page(page_size)};
    AttentionLaunch* f = mode == kPlain   ? launcher<kPlain>(D, dtype)
                         : (mode & kCap) ? capped_launch(mode, D, dtype)
                                         : scored_launch(mode, D, dtype);
    return hip_status(f(c, p, q, q_stride, scale, causal, out, out_stride, lse, max_new, workspace,
                        sc, (hipStream_t)stream));
  });
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
  return part_bytes(plan_attention(B, max_new, max_len, H, Hkv, D), tokens, H, D);
}

int kv8_attention(const void* q, int64_t q_stride, const uint8_t* k_cache, const uint8_t* v_cache,
                  const float* k_scale, const float* v_scale, int64_t num_pages,
                  int32_t page_size, const int32_t* page_table, int64_t max_pages,
                  const int32_t* seq_lens, const int32_t* cu_seqlens, float scale, int32_t causal,
                  void* out, int64_t out_stride, float* lse, int64_t tokens, int64_t B,
                  int64_t max_new, int64_t max_len, int32_t H, int32_t Hkv, int32_t D,
                  int32_t dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return attention(kPlain, q, q_stride, k_cache, v_cache, k_scale, v_scale, num_pages, page_size,
                          page_table, max_pages, seq_lens, cu_seqlens, scale, causal, Scoring{},
                          out, out_stride, lse, tokens, B, max_new, max_len, H, Hkv, D, dtype,
                          workspace, workspace_bytes, stream);
}

int kv8_attention_scored(const void* q, int64_t q_stride, const uint8_t* k_cache,
                         const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                         int64_t num_pages, int32_t page_size, const int32_t* page_table,
                         int64_t max_pages, const int32_t* seq_lens, const int32_t* cu_seqlens,
                         float scale, int32_t causal, float softcap, const float* slopes,
                         const int32_t* first, const int32_t* prefix, void* out,
                         int64_t out_stride, float* lse, int64_t tokens, int64_t B,
                         int64_t max_new, int64_t max_len, int32_t H, int32_t Hkv, int32_t D,
                         int32_t dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  return kv8_attention_scored_ends(q, q_stride, k_cache, v_cache, k_scale, v_scale, num_pages,
                                   page_size, page_table, max_pages, seq_lens, cu_seqlens, scale,
                                   causal, softcap, slopes, first, nullptr, prefix, out,
                                   out_stride, lse, tokens, B, max_new, max_len, H, Hkv, D, dtype,
                                   workspace, workspace_bytes, stream);
}

int kv8_attention_scored_ends(const void* q, int64_t q_stride, const uint8_t* k_cache,
                              const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                              int64_t num_pages, int32_t page_size, const int32_t* page_table,
                              int64_t max_pages, const int32_t* seq_lens,
                              const int32_t* cu_seqlens, float scale, int32_t causal,
                              float softcap, const float* slopes, const int32_t* first,
                              const int32_t* end, const int32_t* prefix, void* out,
                              int64_t out_stride, float* lse, int64_t tokens, int64_t B,
                              int64_t max_new, int64_t max_len, int32_t H, int32_t Hkv, int32_t D,
                              int32_t dtype, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  // (beyond these the quotients of scores and cap leave fp32)
  if (softcap != 0.0f && !(softcap >= 1e-3f && softcap <= 1e30f)) return W4A16_ERR_INVALID_ARG;
  const float cap = softcap * kLog2e;
  const Scoring sc = {cap, 1.0f / cap, slopes, first, prefix, end};
  const int mode = kMasks | (softcap == 0.0f ? 0 : kCap) | (slopes ? kBias : 0);
  return attention(mode, q, q_stride, k_cache, v_cache, k_scale, v_scale, num_pages, page_size,
                         page_table, max_pages, seq_lens, cu_seqlens, scale, causal, sc, out,
                         out_stride, lse, tokens, B, max_new, max_len, H, Hkv, D, dtype, workspace,
                         workspace_bytes, stream);
}

}  // extern "C"
