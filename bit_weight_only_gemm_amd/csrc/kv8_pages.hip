// kv8_pages.hip -- the pages of a paged 8-bit cache: copying them, sharing
// them between rows of a table (fork), taking and giving them back (reserve,
// free) and moving those in use together (compact).
//
// The state of a pool is refs[page], the number of table rows that hold the
// page, 0 where it is free.  Free pages are taken from the lowest on and in the
// order of the rows, so that what a call leaves is a function of what it found,
// whatever the order its atomics (sums of integers) happen in.
//
// A call that takes pages is planned by one workgroup, which goes through refs
// once or twice, 16 KB at a time (a pool of 288 GB in pages of 128 KB for each of 16
// layers has 140 000 pages, 560 KB), and carried out by a second launch.
//
// The copies are bound by bytes (MI355X: compacting 1.17 GB of 4 caches 247 us, 4.7 TB/s,
// the rate of a 4 GiB copy; a beam's step of 120 children over 16 caches, 302 MB, 76 to
// 89 by card), calls without many by their launches (2 to 11 us each) and the host's
// part: 27 us for the free, fork and reserve of four beams.
#include <algorithm>

#include "kv8.h"

namespace w4a16 {
namespace {

constexpr int kPlan = 1024, kWaves = kPlan / 64;  // lanes and waves of the planning workgroup
constexpr int kLayers = 32;                       // caches a launch takes
constexpr int kChunk = 16384;                     // bytes of a page that a workgroup copies at a time

struct Layers {
  uint8_t* k[kLayers];
  uint8_t* v[kLayers];
  float* ks[kLayers];
  float* vs[kLayers];
};

// A table and its pool.
struct Pool {
  int32_t* refs;
  int32_t* table;  // [B, width]
  int32_t* lens;   // [B]
  int pages, width, B, lgT;
};

__device__ __forceinline__ int len_of(const Pool& p, int row) {
  return (int)min((int64_t)max(p.lens[row], 0), (int64_t)p.width << p.lgT);
}
__device__ __forceinline__ int pages_of(const Pool& p, int len) {
  return (int)(((int64_t)len + (1 << p.lgT) - 1) >> p.lgT);
}
__device__ __forceinline__ bool valid(const Pool& p, int page) {
  return (uint32_t)page < (uint32_t)p.pages;
}

// Sum of v (0 or more) over the lanes before this one in the workgroup; `total`
// over all.  Sums stay at kMany, which is more than there are pages, once they
// reach it.
constexpr uint32_t kMany = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b) { return min(a + b, kMany); }
__device__ __forceinline__ int before_me(int v, int* part, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = (uint32_t)v;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t t = (uint32_t)__shfl_up((int)s, o, 64);
    if (lane >= o) s = plus(s, t);
  }
  const uint32_t mine = (uint32_t)__shfl_up((int)s, 1, 64);
  __syncthreads();  // part is free
  if (lane == 63) part[wave] = (int)s;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w == wave) base = all;
    all = plus(all, (uint32_t)part[w]);
  }
  total = (int)all;
  return (int)(lane ? plus(base, mine) : base);
}

// Counters of the four pages from 4 (turn * kPlan + lane) on: a turn of the planning
// workgroup.  Past the pool's end they are `beyond`.
constexpr int kTurn = 4 * kPlan;
typedef int i32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4_t counters(const Pool& p, int64_t at, int beyond) {
  const int64_t page = at + 4 * (int)threadIdx.x;
  i32x4_t n = {beyond, beyond, beyond, beyond};
  if (page + 4 <= p.pages) {
    n = *(const i32x4_t*)(p.refs + page);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (page + i < p.pages) n[i] = p.refs[page + i];
  }
  return n;
}

// Lists the lowest free pages, as many as wanted; how many there are of those.
__device__ int list_free(const Pool& p, int wanted, int32_t* list, int* part) {
  int found = 0;
  i32x4_t next = counters(p, 0, 1);
  for (int64_t at = 0; at < p.pages && found < wanted; at += kTurn) {
    const i32x4_t n = next;
    next = counters(p, at + kTurn, 1);  // a turn ahead
    int total, rank = found;
    rank += before_me((n[0] == 0) + (n[1] == 0) + (n[2] == 0) + (n[3] == 0), part, total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n[i] == 0 && rank < wanted) list[rank] = (int)at + 4 * (int)threadIdx.x + i;
      rank += n[i] == 0;
    }
    found += total;
  }
  __syncthreads();  // the list is whole
  return min(found, wanted);
}

// Bytes of chunk `chunk` of a page, keys and then values, and with the first
// its scales, read once and written to each page that to(..) names in turn, until
// it names none (-1).
template <class F>
__device__ __forceinline__ void copy_chunk(const Layers& c, int layer, int64_t from, int64_t kb,
                                           int Hkv, int chunk, F&& to) {
  constexpr int N = kChunk / (256 * 16);
  const int tid = threadIdx.x;
  u32x4_t w[N];
  uint8_t* dst[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t off = (int64_t)chunk * kChunk + (i * 256 + tid) * 16;
    dst[i] = nullptr;
    if (off < 2 * kb) {
      dst[i] = off < kb ? c.k[layer] + off : c.v[layer] + (off - kb);
      w[i] = *(const u32x4_t*)(dst[i] + from * kb);
    }
  }
  for (int64_t page = to(); page >= 0; page = to()) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (dst[i]) *(u32x4_t*)(dst[i] + page * kb) = w[i];
    if (chunk == 0)
      for (int h = tid; h < Hkv; h += 256) {
        c.ks[layer][page * Hkv + h] = c.ks[layer][from * Hkv + h];
        c.vs[layer][page * Hkv + h] = c.vs[layer][from * Hkv + h];
      }
  }
}
// To one page.
__device__ __forceinline__ void copy_chunk(const Layers& c, int layer, int64_t from, int64_t to,
                                           int64_t kb, int Hkv, int chunk) {
  copy_chunk(c, layer, from, kb, Hkv, chunk, [next = to]() mutable {
    const int64_t page = next;
    next = -1;
    return page;
  });
}

// ------------------------------------------------------------------- copy ---
__global__ void __launch_bounds__(256)
kv8_copy_pages_kernel(Layers c, int layers, const int32_t* __restrict__ src,
                      const int32_t* __restrict__ dst, int64_t n, int pages, int64_t kb, int Hkv,
                      int chunks) {
  const int64_t items = n * layers * chunks;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int chunk = (int)(it % chunks), layer = (int)(it / chunks % layers);
    const int64_t i = it / chunks / layers;
    const int from = src[i], to = dst[i];
    if ((uint32_t)from >= (uint32_t)pages || (uint32_t)to >= (uint32_t)pages || from == to) continue;
    copy_chunk(c, layer, from, to, kb, Hkv, chunk);
  }
}

// ------------------------------------------------------------------- free ---
// One workgroup per entry of rows.  A row named twice is given back once: the
// first to swap its length for 0 has it.
__global__ void __launch_bounds__(256)
kv8_free_kernel(Pool p, const int32_t* __restrict__ rows) {
  __shared__ int held;
  const int row = rows[blockIdx.x];
  if ((uint32_t)row >= (uint32_t)p.B) return;
  if (threadIdx.x == 0) {
    const int len = atomicExch(p.lens + row, 0);
    held = pages_of(p, (int)min((int64_t)max(len, 0), (int64_t)p.width << p.lgT));
  }
  __syncthreads();
  int32_t* entries = p.table + (int64_t)row * p.width;
  for (int i = threadIdx.x; i < held; i += 256) {
    const int page = entries[i];
    if (valid(p, page)) atomicSub(p.refs + page, 1);
    entries[i] = -1;
  }
}

// ---------------------------------------------------------------- reserve ---
// One workgroup.  ws: the first place in the list of each row's new pages, then
// the list.
__global__ void __launch_bounds__(kPlan)
kv8_reserve_kernel(Pool p, const int32_t* __restrict__ added, int32_t* __restrict__ status,
                   int32_t* __restrict__ ws) {
  __shared__ int part[kWaves];
  __shared__ int bad;  // a row that would be too long, or append to a page of others
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid == 0) bad = 0;
  __syncthreads();
  auto need_of = [&](int b, int& have, int64_t& len) {
    const int old = len_of(p, b);
    len = max((int64_t)old + added[b], (int64_t)0);
    have = pages_of(p, old);
    return (int)min(((len + (1 << p.lgT) - 1) >> p.lgT) - have, (int64_t)p.width + 1);
  };
  int64_t wanted = 0;
  for (int at = 0; at < p.B; at += kPlan) {
    const int b = at + tid;
    int need = 0, have;
    int64_t len = 0;
    if (b < p.B) need = max(need_of(b, have, len), 0);
    if (len > (int64_t)p.width << p.lgT) {
      bad = 1;
      need = 0;
    }
    if (b < p.B && added[b] < 0 && (len & ((1 << p.lgT) - 1)) != 0) {
      const int page = p.table[(int64_t)b * p.width + (len >> p.lgT)];
      if (valid(p, page) && p.refs[page] > 1) bad = 1;
    }
    int total;
    const int first = before_me(need, part, total);
    if (b < p.B) ws[b] = (int)min(wanted + first, (int64_t)p.pages);
    wanted += total;
  }
  __syncthreads();
  int32_t* list = ws + p.B;
  if (bad) {
    if (tid == 0) *status = -1;
    return;
  }
  const int most = (int)min(wanted, (int64_t)p.pages);
  const int found = list_free(p, most, list, part);
  if (found < wanted) {
    if (tid == 0) *status = (int)min(wanted - found, (int64_t)INT32_MAX);
    return;
  }
  for (int b = tid >> 6; b < p.B; b += kWaves) {
    int have;
    int64_t len;
    const int need = need_of(b, have, len);
    for (int i = lane; i < need; i += 64) {
      const int page = list[ws[b] + i];
      p.table[(int64_t)b * p.width + have + i] = page;
      p.refs[page] = 1;
    }
    for (int i = need + lane; i < 0; i += 64) {  // given back: the row's last -need
      int32_t* entry = p.table + (int64_t)b * p.width + have + i;
      if (valid(p, *entry)) atomicSub(p.refs + *entry, 1);
      *entry = -1;
    }
  }
  __syncthreads();  // the lengths have been read
  for (int b = tid; b < p.B; b += kPlan) {
    int have;
    int64_t len;
    need_of(b, have, len);
    p.lens[b] = (int)len;
  }
  if (tid == 0) *status = 0;
}

// ------------------------------------------------------------------- fork ---
// One workgroup: checks the rows and finds a page for every partly filled last
// one.  ws: [n] that page's place in the list or -1, [n] the list, [n] the next pair
// of the same source or -1, [n] a pair of each source with such a page, from which the
// others follow (in whatever order atomics come: all get the same bytes), [4] how many
// those are, [B] marks of the rows.
__global__ void __launch_bounds__(kPlan)
kv8_fork_plan_kernel(Pool p, const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n,
                     int32_t* __restrict__ status, int32_t* __restrict__ ws) {
  __shared__ int part[kWaves];
  __shared__ int bad;
  const int tid = threadIdx.x;
  int32_t *place = ws, *list = ws + n, *link = list + n, *heads = link + n, *marks = heads + n + 4;
  if (tid == 0) bad = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kPlan) {
    const int s = src[i], d = dst[i];
    if ((uint32_t)s >= (uint32_t)p.B || (uint32_t)d >= (uint32_t)p.B || p.lens[d] > 0) bad = 1;
    else marks[s] = marks[d] = 0;
  }
  __syncthreads();
  if (!bad) {
    for (int i = tid; i < n; i += kPlan) atomicOr(marks + src[i], 1);
    __syncthreads();
    for (int i = tid; i < n; i += kPlan)
      if (atomicOr(marks + dst[i], 2) != 0) bad = 1;  // a source, or named before
  }
  __syncthreads();
  if (bad) {
    if (tid == 0) *status = -1;
    return;
  }
  int wanted = 0;
  for (int at = 0; at < n; at += kPlan) {
    const int i = at + tid;
    const int half = i < n && (len_of(p, src[i]) & ((1 << p.lgT) - 1)) != 0;
    int total;
    const int rank = before_me(half, part, total);
    if (i < n) place[i] = half ? wanted + rank : -1;
    wanted += total;
  }
  for (int i = tid; i < n; i += kPlan) marks[src[i]] = -1;
  const int found = list_free(p, wanted, list, part);  // (and a barrier)
  for (int i = tid; i < n; i += kPlan) link[i] = atomicExch(marks + src[i], i);
  if (found == wanted)
    for (int i = tid; i < wanted; i += kPlan) p.refs[list[i]] = 1;
  __syncthreads();
  int count = 0;
  for (int at = 0; at < n; at += kPlan) {
    const int i = at + tid;
    const bool head = i < n && place[i] >= 0 && marks[src[i]] == i;
    int total;
    const int rank = before_me(head, part, total);
    if (head) heads[count + rank] = i;
    count += total;
  }
  if (tid == 0) {
    heads[n] = count;
    *status = wanted - found;
  }
}

// The table's rows (by the first launch of a call: `rows`) and the copies, of each
// source's last page to all of its children at once: 24 pages to 5 children each in 16
// caches, 302 MB, took 79 us with a copy by each child, which reads 240 MB for 50.
__global__ void __launch_bounds__(256)
kv8_fork_kernel(Pool p, Layers c, int layers, const int32_t* __restrict__ src,
                const int32_t* __restrict__ dst, int n, const int32_t* __restrict__ status,
                const int32_t* __restrict__ ws, int rows, int64_t kb, int Hkv, int chunks) {
  if (*status != 0) return;
  const int32_t *place = ws, *list = ws + n, *link = list + n, *heads = link + n;
  if (rows)
    for (int i = blockIdx.x; i < n; i += gridDim.x) {
      const int s = src[i], d = dst[i], len = len_of(p, s), whole = len >> p.lgT;
      const int32_t* from = p.table + (int64_t)s * p.width;
      int32_t* to = p.table + (int64_t)d * p.width;
      for (int j = threadIdx.x; j < whole; j += 256) {
        const int page = from[j];
        to[j] = page;
        if (valid(p, page)) atomicAdd(p.refs + page, 1);
      }
      if (threadIdx.x == 0) {
        if (place[i] >= 0) to[whole] = list[place[i]];
        p.lens[d] = len;
      }
    }
  const int64_t per = (int64_t)layers * chunks, items = per * heads[n];
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int head = heads[it / per], part = (int)(it % per), s = src[head];
    const int page = p.table[(int64_t)s * p.width + (len_of(p, s) >> p.lgT)];
    if (!valid(p, page)) continue;
    copy_chunk(c, part / chunks, page, kb, Hkv, part % chunks, [&, j = head]() mutable {
      const int now = j;
      if (now < 0) return -1;
      j = link[now];
      return list[place[now]];
    });
  }
}

// ---------------------------------------------------------------- compact ---
// One workgroup: pages in use from `used` (their count) on, and the free ones
// below it, both ascending and as many.  ws: [4] how many, [pages] the first,
// [pages] the second, [pages] where each page goes.
__global__ void __launch_bounds__(kPlan)
kv8_compact_plan_kernel(Pool p, int32_t* refs_out, int32_t* __restrict__ used_out,
                        int32_t* __restrict__ ws) {
  __shared__ int part[kWaves];
  const int tid = threadIdx.x;
  int32_t *move = ws + 4, *hole = move + p.pages, *to = hole + p.pages;
  int count = 0;
#pragma unroll 4
  for (int64_t at = 0; at < p.pages; at += kTurn) {
    const i32x4_t n = counters(p, at, 0);
    count += (n[0] > 0) + (n[1] > 0) + (n[2] > 0) + (n[3] > 0);
  }
  int used;
  before_me(count, part, used);
  int moves = 0, holes = 0;
  i32x4_t next = counters(p, 0, 0);
  for (int64_t at = 0; at < p.pages; at += kTurn) {
    const i32x4_t n = next;
    next = counters(p, at + kTurn, 0);  // a turn ahead
    const int page = (int)at + 4 * tid;
    // moves in the low half, holes in the high one: at most kTurn of either
    int mine = 0, total;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mine += page + i >= used ? n[i] > 0 : n[i] <= 0 ? 0x10000 : 0;
    const int before = before_me(mine, part, total);
    int rank_move = moves + (before & 0xFFFF), rank_hole = holes + (before >> 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (page + i >= p.pages) break;
      if (page + i >= used) {
        if (n[i] > 0) move[rank_move++] = page + i;
      } else if (n[i] <= 0) {
        hole[rank_hole++] = page + i;
      }
      refs_out[page + i] = n[i];
      to[page + i] = page + i;
    }
    moves += total & 0xFFFF;
    holes += total >> 16;
  }
  __syncthreads();
  for (int i = tid; i < moves; i += kPlan) {
    const int a = move[i], b = hole[i], n = refs_out[a];
    to[a] = b;
    refs_out[b] = n;
    refs_out[a] = 0;
  }
  if (tid == 0) {
    ws[0] = moves;
    *used_out = used;
  }
}

// The table (by the first launch of a call: `columns` pieces of 256 entries of
// each row) and the copies.
__global__ void __launch_bounds__(256)
kv8_compact_kernel(Pool p, Layers c, int layers, int32_t* table_out, const int32_t* __restrict__ ws,
                   int columns, int64_t kb, int Hkv, int chunks) {
  const int moves = ws[0];
  const int32_t *move = ws + 4, *hole = move + p.pages, *to = hole + p.pages;
  const int64_t pieces = (int64_t)p.B * columns;
  for (int64_t it = blockIdx.x; it < pieces; it += gridDim.x) {
    const int b = (int)(it / columns), i = (int)(it % columns) * 256 + (int)threadIdx.x;
    if (i >= p.width) continue;
    int page = p.table[(int64_t)b * p.width + i];
    if (i < pages_of(p, len_of(p, b)) && valid(p, page)) page = to[page];
    table_out[(int64_t)b * p.width + i] = page;
  }
  const int64_t per = (int64_t)layers * chunks, items = per * moves;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int i = (int)(it / per), part = (int)(it % per);
    copy_chunk(c, part / chunks, move[i], hole[i], kb, Hkv, part % chunks);
  }
}

// --------------------------------------------------------------- checking ---
// Sizes of the caches of a call; their arrays are 4 * count host pointers: k,
// v, k_scale and v_scale of each.
struct Shape {
  int64_t pages, kb;
  int Hkv, chunks;
};

int validate_caches(void* const* arrays, int32_t count, int64_t pages, int32_t T, int32_t Hkv,
                    int32_t D, Shape& s) {
  if (count < 1 || !arrays || pages <= 0 || Hkv <= 0) return W4A16_ERR_INVALID_ARG;
  if (log2_page(T) < 0 || (D != 64 && D != 128) || pages > (1 << 30) || Hkv > 1024 ||
      count > 65536)
    return W4A16_ERR_UNSUPPORTED;
  for (int64_t i = 0; i < 4 * (int64_t)count; ++i) {
    if (!arrays[i]) return W4A16_ERR_INVALID_ARG;
    if (!aligned16(arrays[i])) return W4A16_ERR_MISALIGNED;
  }
  s = {pages, (int64_t)Hkv * T * D, Hkv, (int)ceil_div(2 * (int64_t)Hkv * T * D, kChunk)};
  return W4A16_OK;
}

int validate_pool(int64_t pages, int32_t T, int64_t width, int64_t B, int64_t n) {
  if (pages <= 0 || width <= 0 || B < 0 || n < 0) return W4A16_ERR_INVALID_ARG;
  if (log2_page(T) < 0 || pages > (1 << 30) || B > (1 << 20) || n > (1 << 20) ||
      width * T > ((int64_t)1 << 30))
    return W4A16_ERR_UNSUPPORTED;
  return W4A16_OK;
}

// ints of workspace
int64_t pages_ints(int64_t pages, int64_t B, int64_t n) {
  return std::max(std::max(B + pages, B + 4 * n + 4), 4 + 3 * pages);
}

// Runs launch(layers, count of them, whether they are the call's first) on up
// to kLayers caches at a time.
template <class F>
void each_layers(void* const* arrays, int32_t count, F&& launch) {
  for (int32_t at = 0; at < count; at += kLayers) {
    Layers c = {};
    const int n = std::min(kLayers, count - at);
    for (int i = 0; i < n; ++i) {
      void* const* a = arrays + 4 * (int64_t)(at + i);
      c.k[i] = (uint8_t*)a[0];
      c.v[i] = (uint8_t*)a[1];
      c.ks[i] = (float*)a[2];
      c.vs[i] = (float*)a[3];
    }
    launch(c, n, at == 0);
  }
}

// Workgroups of 256 lanes for so many items, which they take in turn.
dim3 groups_for(int64_t items) {
  return dim3((unsigned)std::max<int64_t>(1, std::min<int64_t>(items, 4096)));
}

}  // namespace
}  // namespace w4a16

using namespace w4a16;

extern "C" {

int64_t kv8_pages_workspace_bytes(int64_t num_pages, int64_t B, int64_t n) {
  if (validate_pool(num_pages, 16, 1, B, n) != W4A16_OK) return -1;
  return pad256(4 * pages_ints(num_pages, B, n));
}

int kv8_copy_pages(void* const* caches_host, int32_t count, int64_t num_pages, int32_t page_size,
                   int32_t Hkv, int32_t D, const int32_t* src, const int32_t* dst, int64_t n,
                   void* stream) {
  return guarded([&]() -> int {
    Shape s;
    if (int e = validate_caches(caches_host, count, num_pages, page_size, Hkv, D, s)) return e;
    if (int e = validate_pool(num_pages, page_size, 1, 0, n)) return e;
    if (n == 0) return W4A16_OK;
    if (int e = check_ptrs({src, dst})) return e;
    clear_pending_error();
    each_layers(caches_host, count, [&](const Layers& c, int layers, bool) {
      hipLaunchKernelGGL(kv8_copy_pages_kernel, groups_for(n * layers * s.chunks), dim3(256), 0,
                         (hipStream_t)stream, c, layers, src, dst, n, (int)num_pages, s.kb, Hkv,
                         s.chunks);
    });
    return hip_status(hipGetLastError());
  });
}

int kv8_free(int32_t* refs, int64_t num_pages, int32_t page_size, int32_t* page_table,
             int64_t max_pages, int32_t* seq_lens, int64_t B, const int32_t* rows, int64_t n,
             void* stream) {
  return guarded([&]() -> int {
    if (int e = validate_pool(num_pages, page_size, max_pages, B, n)) return e;
    if (n == 0) return W4A16_OK;
    if (int e = check_ptrs({refs, rows})) return e;
    if (B == 0) return W4A16_OK;
    if (int e = check_ptrs({page_table, seq_lens})) return e;
    clear_pending_error();
    const Pool p = {refs, page_table, seq_lens, (int)num_pages, (int)max_pages, (int)B,
                    log2_page(page_size)};
    hipLaunchKernelGGL(kv8_free_kernel, dim3((unsigned)n), dim3(256), 0, (hipStream_t)stream, p,
                       rows);
    return hip_status(hipGetLastError());
  });
}

int kv8_reserve(int32_t* refs, int64_t num_pages, int32_t page_size, int32_t* page_table,
                int64_t max_pages, int32_t* seq_lens, int64_t B, const int32_t* added,
                int32_t* status, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    if (int e = validate_pool(num_pages, page_size, max_pages, B, 0)) return e;
    if (int e = check_ptrs({refs, status})) return e;
    if (B > 0)
      if (int e = check_ptrs({page_table, seq_lens, added})) return e;
    if (!aligned16(workspace)) return W4A16_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < kv8_pages_workspace_bytes(num_pages, B, 0))
      return W4A16_ERR_WORKSPACE;
    clear_pending_error();
    const Pool p = {refs, page_table, seq_lens, (int)num_pages, (int)max_pages, (int)B,
                    log2_page(page_size)};
    hipLaunchKernelGGL(kv8_reserve_kernel, dim3(1), dim3(kPlan), 0, (hipStream_t)stream, p, added,
                       status, (int32_t*)workspace);
    return hip_status(hipGetLastError());
  });
}

int kv8_fork(void* const* caches_host, int32_t count, int64_t num_pages, int32_t page_size,
             int32_t Hkv, int32_t D, int32_t* refs, int32_t* page_table, int64_t max_pages,
             int32_t* seq_lens, int64_t B, const int32_t* src, const int32_t* dst, int64_t n,
             int32_t* status, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    Shape s;
    if (int e = validate_caches(caches_host, count, num_pages, page_size, Hkv, D, s)) return e;
    if (int e = validate_pool(num_pages, page_size, max_pages, B, n)) return e;
    if (int e = check_ptrs({refs, status})) return e;
    if (n > 0)
      if (int e = check_ptrs({page_table, seq_lens, src, dst})) return e;
    if (!aligned16(workspace)) return W4A16_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < kv8_pages_workspace_bytes(num_pages, B, n))
      return W4A16_ERR_WORKSPACE;
    clear_pending_error();
    const Pool p = {refs, page_table, seq_lens, (int)num_pages, (int)max_pages, (int)B,
                    log2_page(page_size)};
    const hipStream_t st = (hipStream_t)stream;
    int32_t* ws = (int32_t*)workspace;
    hipLaunchKernelGGL(kv8_fork_plan_kernel, dim3(1), dim3(kPlan), 0, st, p, src, dst, (int)n,
                       status, ws);
    if (n == 0) return hip_status(hipGetLastError());
    each_layers(caches_host, count, [&](const Layers& c, int layers, bool first) {
      hipLaunchKernelGGL(kv8_fork_kernel, groups_for(n * (int64_t)layers * s.chunks),
                         dim3(256), 0, st, p, c, layers, src, dst, (int)n, status, ws, (int)first,
                         s.kb, Hkv, s.chunks);
    });
    return hip_status(hipGetLastError());
  });
}

int kv8_compact(void* const* caches_host, int32_t count, int64_t num_pages, int32_t page_size,
                int32_t Hkv, int32_t D, int32_t* refs, int32_t* refs_out, int32_t* page_table,
                int32_t* page_table_out, int64_t max_pages, const int32_t* seq_lens, int64_t B,
                int32_t* used, void* workspace, int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    Shape s;
    if (int e = validate_caches(caches_host, count, num_pages, page_size, Hkv, D, s)) return e;
    if (int e = validate_pool(num_pages, page_size, max_pages, B, 0)) return e;
    if (int e = check_ptrs({refs, refs_out, used})) return e;
    if (B > 0)
      if (int e = check_ptrs({page_table, page_table_out, seq_lens})) return e;
    if (!aligned16(workspace)) return W4A16_ERR_MISALIGNED;
    if (!workspace || workspace_bytes < kv8_pages_workspace_bytes(num_pages, B, 0))
      return W4A16_ERR_WORKSPACE;
    clear_pending_error();
    const Pool p = {refs, page_table, const_cast<int32_t*>(seq_lens), (int)num_pages,
                    (int)max_pages, (int)B, log2_page(page_size)};
    const hipStream_t st = (hipStream_t)stream;
    int32_t* ws = (int32_t*)workspace;
    hipLaunchKernelGGL(kv8_compact_plan_kernel, dim3(1), dim3(kPlan), 0, st, p, refs_out, used, ws);
    each_layers(caches_host, count, [&](const Layers& c, int layers, bool first) {
      const int columns = first ? (int)ceil_div(max_pages, 256) : 0;
      const int64_t items = std::max((int64_t)B * columns, num_pages / 2 * layers * s.chunks);
      hipLaunchKernelGGL(kv8_compact_kernel, groups_for(items), dim3(256), 0, st, p, c, layers,
                         page_table_out, ws, columns, s.kb, Hkv, s.chunks);
    });
    return hip_status(hipGetLastError());
  });
}

}  // extern "C"
