// The paged KV cache: host checks, inserts of new tokens, and evictions of the
// tokens that received the least attention.
//
// Source: every layer reads and writes a rolling KV cache and old content is
// evicted as new content arrives ("Amazon and Reactor tune Trainium for
// real-time video generation", section "Three problems for generic
// compilers"); here per token instead of per frame (see rkv.h).
#include <algorithm>

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace rkv {
namespace paged {

// ---------------------------------------------------------------------------
// host checks
// ---------------------------------------------------------------------------
int sm_count() {
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 148;
}

static int64_t page_bytes(const rkv_paged_cache* c) { return int64_t(c->page_tokens) * c->H * kRowBytes; }

bool overlaps_pool(const rkv_paged_cache* c, const void* p, uint64_t bytes) {
  const int64_t stride = c->page_stride * 2;
  if (bytes == 0) return false;
  for (const void* base : {c->k, c->v}) {
    // the bytes of p as one row of the pool's own stride where they fit one,
    // so that a neighbour inside the pool's stride is told from an overlap
    const bool one = bytes <= uint64_t(stride);
    if (one ? rows_overlap(p, 1, stride, int64_t(bytes), base, c->n_pages, stride, page_bytes(c))
            : overlaps(p, bytes, base, uint64_t((c->n_pages - 1) * stride + page_bytes(c))))
      return true;
  }
  return false;
}

rkv_status check_cache(const rkv_paged_cache* c) {
  if (!c) return fail(RKV_ERR_INVALID_ARG, "cache is NULL");
  if (!c->k || !c->v) return fail(RKV_ERR_INVALID_ARG, "cache k/v pool is NULL");
  if (!c->page_table) return fail(RKV_ERR_INVALID_ARG, "cache page_table is NULL");
  if (c->D != kHD) return fail(RKV_ERR_INVALID_ARG, "head_dim D must be 128 (got %d)", c->D);
  if (c->n_pages < 1 || c->page_tokens < 1 || c->H < 1 || c->n_seqs < 1 || c->max_pages < 1)
    return fail(RKV_ERR_INVALID_ARG, "cache n_pages/page_tokens/H/n_seqs/max_pages must be >= 1");
  if (c->table_stride < c->max_pages) return fail(RKV_ERR_INVALID_ARG, "cache table_stride < max_pages");
  if (!aligned16(c->k) || !aligned16(c->v)) return fail(RKV_ERR_INVALID_ARG, "cache pools must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(c->page_table) & 3u) || (reinterpret_cast<uintptr_t>(c->status) & 3u))
    return fail(RKV_ERR_INVALID_ARG, "cache page_table/status must be 4-byte aligned");
  if (int64_t(c->page_tokens) * c->H >= (int64_t(1) << 31))
    return fail(RKV_ERR_UNSUPPORTED, "a page holds 2^31 or more head rows");
  if (c->page_stride < int64_t(c->page_tokens) * c->H * kHD)
    return fail(RKV_ERR_INVALID_ARG, "cache page_stride < page_tokens*H*D");
  if (c->page_stride % kHD) return fail(RKV_ERR_INVALID_ARG, "cache page_stride must be a multiple of D");
  if (c->page_stride / kHD >= (int64_t(1) << 32) / c->n_pages)
    return fail(RKV_ERR_UNSUPPORTED, "the pool holds 2^32 or more head rows");
  if (capacity(c) >= (int64_t(1) << 30)) return fail(RKV_ERR_UNSUPPORTED, "a sequence's capacity is 2^30 tokens or more");
  if (rows_overlap(c->k, c->n_pages, c->page_stride * 2, page_bytes(c), c->v, c->n_pages, c->page_stride * 2,
                   page_bytes(c)))
    return fail(RKV_ERR_INVALID_ARG, "cache k and v pools overlap");
  return RKV_OK;
}

CacheDev cache_dev(const rkv_paged_cache* c) {
  CacheDev d;
  d.k = static_cast<uint8_t*>(c->k);
  d.v = static_cast<uint8_t*>(c->v);
  d.table = c->page_table;
  d.table_stride = c->table_stride;
  d.status = c->status;
  d.page_units = uint32_t(c->page_stride / kHD);
  d.n_pages = uint32_t(c->n_pages);
  d.P = uint32_t(c->page_tokens);
  d.div_P = make_fastdiv(d.P);
  d.H = c->H;
  d.n_seqs = c->n_seqs;
  d.capacity = int32_t(capacity(c));
  return d;
}

static uint64_t score_bytes(const rkv_paged_cache* c) { return uint64_t(c->n_seqs) * c->H * capacity(c) * 4; }

// ---------------------------------------------------------------------------
// insert: a copy of n_seqs * n_new rows into their places, 16 bytes a thread
// and step, K and V together; the scores of the new tokens beside it
// ---------------------------------------------------------------------------
struct InsertArgs {
  CacheDev c;
  const uint8_t* k_new;
  const uint8_t* v_new;
  int64_t row_bytes;          // between new rows
  const int32_t* seq_lens;
  const int32_t* next_pos;
  int32_t* pos;
  float* weight;
  int32_t n_new;
  FastDiv div_row, div_new;   // by 16-byte pieces of a row, by n_new
  uint32_t total;             // pieces of K
};

constexpr int kInsertThreads = 256;
constexpr int kInsertUnroll = 4;

__global__ void __launch_bounds__(kInsertThreads) paged_insert_kernel(const __grid_constant__ InsertArgs a) {
  const uint32_t first = blockIdx.x * uint32_t(kInsertThreads * kInsertUnroll) + threadIdx.x;
  uint4 kv[kInsertUnroll], vv[kInsertUnroll];
  uint64_t dst[kInsertUnroll];   // byte offset in the pools, or ~0: nothing to write
#pragma unroll
  for (int u = 0; u < kInsertUnroll; ++u) {
    const uint32_t x = first + uint32_t(u * kInsertThreads);
    dst[u] = ~uint64_t(0);
    if (x >= a.total) continue;
    const uint32_t r = fdiv(x, a.div_row), piece = x - r * a.div_row.d;
    const uint32_t s = fdiv(r, a.div_new), i = r - s * a.div_new.d;
    const uint64_t src = uint64_t(r) * uint64_t(a.row_bytes) + piece * 16u;
    kv[u] = *reinterpret_cast<const uint4*>(a.k_new + src);
    vv[u] = *reinterpret_cast<const uint4*>(a.v_new + src);
    const int j = seq_len(a.c, a.seq_lens, int(s)) - a.n_new + int(i);
    if (j < 0) continue;
    const uint32_t h = piece >> 4;
    if ((piece & 15u) == 0) {
      const int64_t at = (int64_t(s) * a.c.H + h) * a.c.capacity + j;
      if (a.pos) a.pos[at] = a.next_pos[s] - a.n_new + int(i);
      if (a.weight) a.weight[at] = 0.f;
    }
    const uint32_t page = page_of(a.c, int(s), uint32_t(j));
    if (page >= a.c.n_pages) {
      record(a.c, kBadPage);
      continue;
    }
    dst[u] = uint64_t(row_unit(a.c, page, uint32_t(j), int(h))) * kRowBytes + (piece & 15u) * 16u;
  }
#pragma unroll
  for (int u = 0; u < kInsertUnroll; ++u) {
    if (dst[u] == ~uint64_t(0)) continue;
    *reinterpret_cast<uint4*>(a.c.k + dst[u]) = kv[u];
    *reinterpret_cast<uint4*>(a.c.v + dst[u]) = vv[u];
  }
}

// ---------------------------------------------------------------------------
// evict
// ---------------------------------------------------------------------------
struct EvictArgs {
  CacheDev c;
  const int32_t* seq_lens;
  const float* weight;
  const int32_t* pos;
  const int32_t* next_pos;
  int32_t* seq_lens_out;
  float* weight_out;
  int32_t* pos_out;
  int32_t budget, sinks, recent;
  int32_t in_place;
  int32_t smem_keys;   // keys of one head that fit shared memory; the rest are formed again in each pass
  int32_t max_moves;   // moves one head can need: min(budget, capacity - budget)
  int32_t* count;      // [n_seqs * H] moves of each head
  int32_t* src;        // [n_seqs * H][max_moves] token each move takes
  int32_t* dst;        // ... and where it goes
  int32_t blocks_per_item;
};

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kHistCopies = 4;

// Order of the keep rule as an unsigned number: protected tokens above every
// weight, larger weights above smaller, -0 = 0, NaN below every number.
__device__ __forceinline__ uint32_t keep_key(float w, int pos, int sinks, int64_t recent_from) {
  if (pos < sinks || int64_t(pos) >= recent_from) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block of one value a thread; `total` receives
// the sum.  `warp_sums` holds kSelWarps words.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();   // warp_sums of an earlier scan are read
  if (lane == 31) warp_sums[warp] = inc;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w) {
    const uint32_t x = warp_sums[w];
    before += w < warp ? x : 0u;
    total += x;
  }
  return before + inc - v;
}

// One head of one sequence per block: the key of the budget-th largest token
// by radix selection, 8 bits a pass, then the lists of places that fall free
// and of tokens that move into them.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[kHistCopies][256];
  __shared__ uint32_t warp_sums[kSelWarps];
  __shared__ uint32_t found[2];
  const int item = blockIdx.x, tid = threadIdx.x;
  const int s = item / a.c.H;
  ptx::pdl_launch_dependents();   // the move kernel's blocks may take their places; they wait for this grid's end
  const int L = seq_len(a.c, a.seq_lens, s);
  const int64_t base = int64_t(item) * a.c.capacity;
  const float* weight = a.weight + base;
  const int32_t* pos = a.pos + base;
  float* weight_out = a.weight_out + base;
  int32_t* pos_out = a.pos_out + base;
  if (L <= a.budget) {
    if (!a.in_place)
      for (int j = tid; j < L; j += kSelThreads) {
        weight_out[j] = weight[j];
        pos_out[j] = pos[j];
      }
    if (tid == 0) a.count[item] = 0;
    return;
  }
  const int64_t recent_from = int64_t(a.next_pos[s]) - a.recent;
  auto form_key = [&](int j) { return keep_key(weight[j], pos[j], a.sinks, recent_from); };
  auto key = [&](int j) { return j < a.smem_keys ? keys[j] : form_key(j); };
  for (int j = tid; j < min(L, a.smem_keys); j += kSelThreads) keys[j] = form_key(j);

  uint32_t prefix = 0, mask = 0, want = uint32_t(a.budget);   // rank, from the top, among keys that share `prefix`
  uint32_t equal = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < kHistCopies * 256; i += kSelThreads) hist[i >> 8][i & 255] = 0;
    __syncthreads();
    for (int j = tid; j < L; j += kSelThreads) {
      const uint32_t k = key(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(tid >> 5) & (kHistCopies - 1)][(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid < 32) {
      // lane i sums bins 255 - 8i .. 248 - 8i, from the top
      uint32_t n[8], sum = 0;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        n[b] = 0;
#pragma unroll
        for (int c = 0; c < kHistCopies; ++c) n[b] += hist[c][255 - 8 * tid - b];
        sum += n[b];
      }
      uint32_t inc = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, inc, d);
        if (tid >= d) inc += o;
      }
      uint32_t above = inc - sum;
      if (above < want && want <= inc) {
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          if (above < want && want <= above + n[b]) {
            found[0] = uint32_t(255 - 8 * tid - b) | (n[b] << 8);
            found[1] = want - above;
          }
          above += n[b];
        }
      }
    }
    __syncthreads();
    prefix |= (found[0] & 255u) << shift;
    equal = found[0] >> 8;
    mask |= 255u << shift;
    want = found[1];
  }
  // kept: keys above `prefix`, and the first `want` of the `equal` keys at it
  const bool some_ties = equal > want;
  uint32_t ties_before = 0, holes_before = 0, moved_before = 0;
  int32_t* src = a.src + int64_t(item) * a.max_moves;
  int32_t* dst = a.dst + int64_t(item) * a.max_moves;
  for (int j0 = 0; j0 < L; j0 += kSelThreads) {
    const int j = j0 + tid;
    const uint32_t k = j < L ? key(j) : 0u;
    const bool tie = j < L && k == prefix;
    bool keep = j < L && k >= prefix;
    if (some_ties) {
      uint32_t total;
      const uint32_t rank = ties_before + block_scan(tie ? 1u : 0u, warp_sums, total);
      if (tie && rank >= want) keep = false;
      ties_before += total;
    }
    const bool hole = j < a.budget && j < L && !keep, moved = j >= a.budget && keep;
    uint32_t total;
    const uint32_t at = block_scan((hole ? 1u : 0u) | (moved ? 0x10000u : 0u), warp_sums, total);
    if (hole) dst[holes_before + (at & 0xFFFFu)] = j;
    if (moved) src[moved_before + (at >> 16)] = j;
    if (!a.in_place && keep && j < a.budget) {
      weight_out[j] = weight[j];
      pos_out[j] = pos[j];
    }
    holes_before += total & 0xFFFFu;
    moved_before += total >> 16;
  }
  __syncthreads();   // the block's lists are written
  if (tid == 0) a.count[item] = int(moved_before);
  for (int t = tid; t < int(moved_before); t += kSelThreads) {
    const int from = src[t], to = dst[t];
    weight_out[to] = weight[from];   // from >= budget > to: no index is both read and written
    pos_out[to] = pos[from];
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// The K and V rows of the moves: a warp takes kMoveUnroll moves at a time,
// lanes 0-15 the K row's sixteen 16-byte pieces, lanes 16-31 the V row's.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  const int item = int(blockIdx.x) / a.blocks_per_item, part = int(blockIdx.x) - item * a.blocks_per_item;
  const int s = item / a.c.H, h = item - s * a.c.H;
  ptx::pdl_wait();
  if (part == 0 && h == 0 && threadIdx.x == 0) {
    const int L = seq_len(a.c, a.seq_lens, s);
    a.seq_lens_out[s] = min(L, a.budget);
  }
  const int n = a.count[item];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t* src = a.src + int64_t(item) * a.max_moves;
  const int32_t* dst = a.dst + int64_t(item) * a.max_moves;
  uint8_t* pool = (lane < 16 ? a.c.k : a.c.v) + (lane & 15) * 16;
  for (int t0 = (part * (kMoveThreads / 32) + warp) * kMoveUnroll; t0 < n;
       t0 += a.blocks_per_item * (kMoveThreads / 32) * kMoveUnroll) {
    uint4 x[kMoveUnroll];
    uint32_t to[kMoveUnroll];
    bool ok[kMoveUnroll];
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u) {
      ok[u] = t0 + u < n;
      if (!ok[u]) continue;
      const uint32_t js = uint32_t(src[t0 + u]), jd = uint32_t(dst[t0 + u]);
      const uint32_t ps = page_of(a.c, s, js), pd = page_of(a.c, s, jd);
      ok[u] = ps < a.c.n_pages && pd < a.c.n_pages;
      if (!ok[u]) {
        record(a.c, kBadPage);
        continue;
      }
      x[u] = *reinterpret_cast<const uint4*>(pool + uint64_t(row_unit(a.c, ps, js, h)) * kRowBytes);
      to[u] = row_unit(a.c, pd, jd, h);
    }
#pragma unroll
    for (int u = 0; u < kMoveUnroll; ++u)
      if (ok[u]) *reinterpret_cast<uint4*>(pool + uint64_t(to[u]) * kRowBytes) = x[u];
  }
}

static int64_t max_moves(const rkv_paged_cache* c, int32_t budget) {
  return std::max<int64_t>(0, std::min<int64_t>(budget, capacity(c) - budget));
}

}  // namespace paged
}  // namespace rkv

using namespace rkv;
using namespace rkv::paged;

extern "C" rkv_status kvcache_paged_insert(const rkv_paged_cache* cache, const void* k_new, const void* v_new,
                                           int64_t new_row_stride, int32_t n_new, const int32_t* seq_lens,
                                           const int32_t* next_pos, int32_t* pos, float* weight, void* stream) {
  NvtxRange nvtx_range("kvcache_paged_insert");
  clear_error();
  rkv_status st = check_cache(cache);
  if (st != RKV_OK) return st;
  if (n_new < 0 || n_new > capacity(cache))
    return fail(RKV_ERR_INVALID_ARG, "n_new %d must be in [0, capacity=%lld]", n_new, (long long)capacity(cache));
  if (n_new == 0) return RKV_OK;
  if (!k_new || !v_new || !seq_lens) return fail(RKV_ERR_INVALID_ARG, "k_new/v_new/seq_lens is NULL");
  if (!pos != !next_pos) return fail(RKV_ERR_INVALID_ARG, "pos and next_pos go together");
  if (!aligned16(k_new) || !aligned16(v_new)) return fail(RKV_ERR_INVALID_ARG, "k_new/v_new must be 16-byte aligned");
  const int64_t row = int64_t(cache->H) * kHD;
  if (new_row_stride < row) return fail(RKV_ERR_INVALID_ARG, "new_row_stride < H*D");
  if (new_row_stride % 8) return fail(RKV_ERR_INVALID_ARG, "rows of k_new/v_new must be 16-byte aligned");
  if (new_row_stride >= (int64_t(1) << 40)) return fail(RKV_ERR_INVALID_ARG, "new_row_stride too large");
  const int64_t rows = int64_t(cache->n_seqs) * n_new;
  const int64_t pieces = rows * cache->H * 16;
  if (rows >= (int64_t(1) << 31) || pieces >= (int64_t(1) << 31) - kInsertThreads * kInsertUnroll)
    return fail(RKV_ERR_UNSUPPORTED, "insert too large for one launch");
  const uint64_t span = uint64_t((rows - 1) * new_row_stride + row) * 2;
  if (overlaps_pool(cache, k_new, span) || overlaps_pool(cache, v_new, span))
    return fail(RKV_ERR_INVALID_ARG, "new tokens overlap the pool");
  if ((pos && overlaps_pool(cache, pos, score_bytes(cache))) || (weight && overlaps_pool(cache, weight, score_bytes(cache))) ||
      (pos && weight && overlaps(pos, score_bytes(cache), weight, score_bytes(cache))))
    return fail(RKV_ERR_INVALID_ARG, "scores overlap the pool or one another");
  InsertArgs a;
  a.c = cache_dev(cache);
  a.k_new = static_cast<const uint8_t*>(k_new);
  a.v_new = static_cast<const uint8_t*>(v_new);
  a.row_bytes = new_row_stride * 2;
  a.seq_lens = seq_lens;
  a.next_pos = next_pos;
  a.pos = pos;
  a.weight = weight;
  a.n_new = n_new;
  a.div_row = make_fastdiv(uint32_t(cache->H) * 16u);
  a.div_new = make_fastdiv(uint32_t(n_new));
  a.total = uint32_t(pieces);
  const uint32_t per = kInsertThreads * kInsertUnroll;
  paged_insert_kernel<<<(a.total + per - 1) / per, kInsertThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "paged_insert_kernel launch");
  return RKV_OK;
}

extern "C" size_t kvcache_paged_evict_workspace_size(const rkv_paged_cache* cache, int32_t budget) {
  if (check_cache(cache) != RKV_OK || budget < 1) {
    clear_error();
    return 0;
  }
  const uint64_t items = uint64_t(cache->n_seqs) * cache->H;
  return size_t(((items * (1 + 2 * uint64_t(max_moves(cache, budget))) * 4) + 15) / 16 * 16);
}

extern "C" rkv_status kvcache_paged_evict(const rkv_paged_cache* cache, const int32_t* seq_lens, const float* weight,
                                          const int32_t* pos, const int32_t* next_pos, int32_t budget, int32_t sinks,
                                          int32_t recent, int32_t* seq_lens_out, float* weight_out, int32_t* pos_out,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("kvcache_paged_evict");
  clear_error();
  rkv_status st = check_cache(cache);
  if (st != RKV_OK) return st;
  if (!seq_lens || !weight || !pos || !next_pos || !seq_lens_out || !weight_out || !pos_out)
    return fail(RKV_ERR_INVALID_ARG, "seq_lens/weight/pos/next_pos or an output is NULL");
  if (budget < 1) return fail(RKV_ERR_INVALID_ARG, "budget must be >= 1");
  if (sinks < 0 || recent < 0) return fail(RKV_ERR_INVALID_ARG, "sinks and recent must be >= 0");
  const uint64_t sb = score_bytes(cache);
  const bool in_place = weight_out == weight;
  if (in_place != (pos_out == pos)) return fail(RKV_ERR_INVALID_ARG, "weight_out and pos_out are in place both or neither");
  if (overlaps(weight, sb, pos, sb) || overlaps(weight_out, sb, pos_out, sb) ||
      (!in_place && (overlaps(weight, sb, weight_out, sb) || overlaps(weight, sb, pos_out, sb) ||
                     overlaps(pos, sb, weight_out, sb) || overlaps(pos, sb, pos_out, sb))))
    return fail(RKV_ERR_INVALID_ARG, "weight, pos and their outputs overlap");
  if (overlaps_pool(cache, weight_out, sb) || overlaps_pool(cache, pos_out, sb))
    return fail(RKV_ERR_INVALID_ARG, "scores overlap the pool");
  const size_t need = kvcache_paged_evict_workspace_size(cache, budget);
  if (!workspace || !aligned16(workspace) || workspace_bytes < need)
    return fail(RKV_ERR_INVALID_ARG, "workspace must be >= %zu bytes and 16-byte aligned", need);
  const int64_t items = int64_t(cache->n_seqs) * cache->H;
  if (items >= (int64_t(1) << 24)) return fail(RKV_ERR_UNSUPPORTED, "too many heads and sequences for one launch");
  EvictArgs a;
  a.c = cache_dev(cache);
  a.seq_lens = seq_lens;
  a.weight = weight;
  a.pos = pos;
  a.next_pos = next_pos;
  a.seq_lens_out = seq_lens_out;
  a.weight_out = weight_out;
  a.pos_out = pos_out;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.in_place = in_place ? 1 : 0;
  a.max_moves = int32_t(max_moves(cache, budget));
  a.count = static_cast<int32_t*>(workspace);
  a.src = a.count + items;
  a.dst = a.src + items * a.max_moves;
  constexpr int kMaxSmemKeys = 48 * 1024;
  a.smem_keys = int32_t(std::min<int64_t>(capacity(cache), kMaxSmemKeys));
  const int smem = a.smem_keys * 4;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(evict_select_kernel)");
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  evict_select_kernel<<<uint32_t(items), kSelThreads, smem, cs>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "evict_select_kernel launch");
  // enough blocks to fill the machine about twice over, no more than the moves need
  const int64_t per = (kMoveThreads / 32) * kMoveUnroll;
  const int64_t most = std::max<int64_t>(1, (a.max_moves + per - 1) / per);
  const int64_t want = (int64_t(sm_count()) * 16 + items - 1) / items;
  a.blocks_per_item = int32_t(std::min(most, std::max<int64_t>(1, want)));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(uint32_t(items * a.blocks_per_item));
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_move_kernel, a);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "evict_move_kernel launch");
  return RKV_OK;
}

extern "C" rkv_status rkv_paged_status(const rkv_paged_cache* cache, void* stream) {
  NvtxRange nvtx_range("rkv_paged_status");
  clear_error();
  rkv_status st = check_cache(cache);
  if (st != RKV_OK) return st;
  if (!cache->status) return fail(RKV_ERR_INVALID_ARG, "cache has no status word");
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int32_t word = 0;
  cudaError_t e = cudaMemcpyAsync(&word, cache->status, sizeof(word), cudaMemcpyDeviceToHost, cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e != cudaSuccess) return cuda_fail(e, "reading the cache's status word");
  if (word == 0) return RKV_OK;
  e = cudaMemsetAsync(cache->status, 0, sizeof(word), cs);
  if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
  if (e != cudaSuccess) return cuda_fail(e, "clearing the cache's status word");
  return fail(RKV_ERR_DEVICE_CHECK, "a paged cache call met a %s",
              (word >> 8) == kBadLength ? "length outside [0, capacity]" : "page outside [0, n_pages)");
}
