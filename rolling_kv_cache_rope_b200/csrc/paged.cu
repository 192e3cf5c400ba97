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
  static std::atomic<int> known[64];   // by device
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return n;
  if (dev < 64 && known[dev].load(std::memory_order_relaxed) > 0) return known[dev].load(std::memory_order_relaxed);
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 148;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

static int64_t page_bytes(const rkv_paged_cache* c) { return int64_t(c->page_tokens) * c->H * kRowBytes; }

Bytes pool_k(const rkv_paged_cache* c) { return {"the pool k", c->k, c->n_pages, c->page_stride * 2, page_bytes(c)}; }
Bytes pool_v(const rkv_paged_cache* c) { return {"the pool v", c->v, c->n_pages, c->page_stride * 2, page_bytes(c)}; }
Bytes table_of(const rkv_paged_cache* c) {
  const int64_t row = int64_t(c->max_pages) * 4;
  return {"the page table", c->page_table, c->n_seqs, c->n_seqs > 1 ? c->table_stride * 4 : row, row};
}
Bytes status_of(const rkv_paged_cache* c) { return run_of("the status word", c->status, 4); }

static bool meet(Bytes a, Bytes b) {
  if (!a.p || !b.p) return false;
  // rows that fit one of the other's strides count as a single row of it, so
  // that a neighbour between its rows is told from an overlap
  auto fit = [](Bytes& x, const Bytes& y) {
    const int64_t span = (x.rows - 1) * x.stride + x.width;
    if (x.stride != y.stride && span <= y.stride) x = {x.name, x.p, 1, y.stride, span};
  };
  fit(a, b);
  fit(b, a);
  return rows_overlap(a.p, a.rows, a.stride, a.width, b.p, b.rows, b.stride, b.width);
}

rkv_status check_apart(std::initializer_list<Bytes> writes, std::initializer_list<Bytes> reads) {
  for (auto w = writes.begin(); w != writes.end(); ++w) {
    for (const Bytes& r : reads)
      if (meet(*w, r)) return fail(RKV_ERR_INVALID_ARG, "%s overlaps %s", w->name, r.name);
    for (auto x = writes.begin(); x != w; ++x)
      if (meet(*w, *x)) return fail(RKV_ERR_INVALID_ARG, "%s overlaps %s", w->name, x->name);
  }
  return RKV_OK;
}

rkv_status check_cache(const rkv_paged_cache* c) {
  if (!c) return fail(RKV_ERR_INVALID_ARG, "cache is NULL");
  if (!c->k || !c->v) return fail(RKV_ERR_INVALID_ARG, "cache k/v pool is NULL");
  if (!c->page_table) return fail(RKV_ERR_INVALID_ARG, "cache page_table is NULL");
  if (c->D != kHD) return fail(RKV_ERR_INVALID_ARG, "head_dim D must be 128 (got %d)", c->D);
  if (c->n_pages < 1 || c->page_tokens < 1 || c->H < 1 || c->n_seqs < 1 || c->max_pages < 1)
    return fail(RKV_ERR_INVALID_ARG, "cache n_pages/page_tokens/H/n_seqs/max_pages must be >= 1");
  if (c->table_stride < c->max_pages) return fail(RKV_ERR_INVALID_ARG, "cache table_stride < max_pages");
  if (c->n_seqs > 1 && c->table_stride >= (int64_t(1) << 32))
    return fail(RKV_ERR_INVALID_ARG, "cache table_stride too large");
  if (!aligned16(c->k) || !aligned16(c->v)) return fail(RKV_ERR_INVALID_ARG, "cache pools must be 16-byte aligned");
  if (!aligned4(c->page_table) || !aligned4(c->status))
    return fail(RKV_ERR_INVALID_ARG, "cache page_table/status must be 4-byte aligned");
  if (int64_t(c->page_tokens) * c->H >= (int64_t(1) << 31))
    return fail(RKV_ERR_UNSUPPORTED, "a page holds 2^31 or more head rows");
  if (c->page_stride < int64_t(c->page_tokens) * c->H * kHD)
    return fail(RKV_ERR_INVALID_ARG, "cache page_stride < page_tokens*H*D");
  if (c->page_stride % kHD) return fail(RKV_ERR_INVALID_ARG, "cache page_stride must be a multiple of D");
  if (c->page_stride / kHD >= (int64_t(1) << 32) / c->n_pages)
    return fail(RKV_ERR_UNSUPPORTED, "the pool holds 2^32 or more head rows");
  // (the calls' 64-bit counts of rows, pieces and score bytes start from these)
  if (int64_t(c->n_seqs) * c->H >= (int64_t(1) << 28))
    return fail(RKV_ERR_UNSUPPORTED, "2^28 or more key heads of all sequences");
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
// and step, K and V together; the scores of the new tokens beside it.
//
// Bound: HBM for many rows, 1 KB read and 1 KB written per token and key head
// (15,600 tokens of 12 heads, 193 MB counted in K and V read and written: 32.5
// us, 5.9 TB/s); launch latency for a step's (48 tokens of 8 heads: 3.5 us).
// A thread takes four pieces of K and of V, all loaded before the first is
// stored: their page numbers are a load that the loads of the rows do not wait
// for.
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
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
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
    const uint32_t page = page_of(a.c, int(s), uint32_t(j));
    if (page >= a.c.n_pages) {   // no such token: its scores are left as well
      record(a.c, kBadPage);
      continue;
    }
    const uint32_t h = piece >> 4;
    if ((piece & 15u) == 0) {
      const int64_t at = (int64_t(s) * a.c.H + h) * a.c.capacity + j;
      if (a.pos) a.pos[at] = a.next_pos[s] - a.n_new + int(i);
      if (a.weight) a.weight[at] = 0.f;
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
//
// Bound: reading weight and pos (8 bytes a token and key head) and, out of
// place, writing them; then the rows that move (1 KB each).  Two ways to find
// the tokens to drop, by how many there are (E = L - budget):
//   E <= kFew and a block has the head to itself (no cluster, see below): E
//               rounds of a block-wide minimum over (key, index), about 1 us a
//               round, and the block moves the rows itself.  48 streams x 8 heads
//               x 4,096 tokens: 8.7 us for E = 1 (25.6 MB: 3.0 TB/s, the dependent
//               loads of one head's step bound it), 24.8 for E = 16, 24.8 the
//               way below for E = 17
//   otherwise   radix selection of the budget-th largest key, 11 bits a pass,
//               then lists of the places that fall free and of the tokens that
//               move into them; a second launch moves the rows over all SMs
//               (24 heads of 32,760 tokens cut to 7,800: 55 us, of them 22
//               for the selection, a chain of passes, and 21 for the rows, which
//               move at 6.9 TB/s, part of it out of L2; by the selecting blocks
//               themselves the whole took 66 against 58 at that time)
// The second launch is left out where no sequence can have more than kFew
// tokens to drop (capacity - budget <= kFew), blocks have heads to themselves
// and the new lengths are apart from the old; a step's eviction under pages that
// leave more room behind the budget launches it with nothing to move (9.9 us
// against 8.7).
// A head's tokens are shared out over a cluster of blocks where there are too
// few heads and sequences to fill the machine; the blocks' histograms and
// counts meet in distributed shared memory.  That is the faster way for many
// tokens to drop (figures where the host decides) and the slower for one or a
// few: 76 heads of 2,542 tokens, one dropped, 13 us against 4.9; 12 heads of
// 4,097 12.3 against 5.4.
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
  int32_t lens_here;   // the selection writes seq_lens_out (no other block still reads seq_lens there)
  int32_t cluster;     // blocks a head's tokens are shared out over
  int32_t smem_keys;   // keys of one block that fit shared memory; the rest are formed again in each pass
  int32_t max_moves;   // moves one head can need: min(budget, capacity - budget)
  int32_t vec;         // heads' scores start on 16-byte boundaries
  int32_t* count;      // [n_seqs * H] moves of each head left to the second launch
  int32_t* src;        // [n_seqs * H][max_moves] token, then row each move takes
  int32_t* dst;        // ... and where it goes
  int32_t blocks_per_item;
};

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kFew = 16;
constexpr int kMaxCluster = 8;

// Order of the keep rule as an unsigned number: protected tokens above every
// weight, larger weights above smaller, -0 = 0, NaN below every number.
__device__ __forceinline__ uint32_t keep_key(float w, int pos, int sinks, int64_t recent_from) {
  if (pos < sinks || int64_t(pos) >= recent_from) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t v) {   // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (int(threadIdx.x & 31) >= d) v += o;
  }
  return v;
}

__global__ void __launch_bounds__(kSelThreads, 3) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[kBins];     // this block's keys by bin
  __shared__ uint32_t bins[3][kBins];  // the cluster's, one for each pass
  __shared__ uint32_t warp_sums[kSelWarps];
  __shared__ uint32_t found[3];
  __shared__ uint32_t block_sums[3][kMaxCluster];   // free places, moves and ties of each block
  __shared__ uint64_t lowest[2][kSelWarps];
  __shared__ int32_t few_src[kFew], few_dst[kFew], dropped[kFew];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cs = a.cluster, rank = cs > 1 ? int(ptx::cluster_ctarank()) : 0;
  const int item = int(blockIdx.x) / cs;
  const int s = item / a.c.H, h = item - s * a.c.H;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  const int L = seq_len(a.c, a.seq_lens, s);
  const int64_t base = int64_t(item) * a.c.capacity;
  const float* weight = a.weight + base;
  const int32_t* pos = a.pos + base;
  float* weight_out = a.weight_out + base;
  int32_t* pos_out = a.pos_out + base;
  const int E = L - a.budget;
  const bool few = cs == 1 && E <= kFew;
  if (tid == 0 && rank == 0) {
    if (E <= 0 || few) a.count[item] = 0;
    if (a.lens_here && h == 0) a.seq_lens_out[s] = min(L, a.budget);
  }
  if (E <= 0 && a.in_place) return;

  auto sync = [&]() {
    if (cs > 1) {
      ptx::cluster_arrive();
      ptx::cluster_wait();
    } else {
      __syncthreads();
    }
  };
  if (cs > 1 && E > 0) {
    for (int i = tid; i < 3 * kBins; i += kSelThreads) bins[0][i] = 0;
    ptx::cluster_arrive();   // waited for before the first block adds to another's
  }
  // this block's tokens: [j0, j1)
  const int seg = ((L + cs - 1) / cs + 31) & ~31;
  const int j0 = min(L, rank * seg), j1 = min(L, j0 + seg);
  const int64_t recent_from = int64_t(a.next_pos[s]) - a.recent;
  auto key = [&](int j) {
    return j - j0 < a.smem_keys ? keys[j - j0] : keep_key(weight[j], pos[j], a.sinks, recent_from);
  };
  // the lowest key of the thread's tokens; of equal ones the highest index
  uint64_t low = ~uint64_t(0);
  auto packed = [](uint32_t k, int j) { return uint64_t(k) << 32 | uint32_t(~j); };
  // a thread takes four tokens in a row at a time, two times four in flight
  constexpr int kBatch = 2;
  for (int q = tid; j0 + 4 * q < j1; q += kBatch * kSelThreads) {
    float4 w[kBatch];
    int4 p[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + 4 * (q + u * kSelThreads);
      if (a.vec && j + 3 < j1) {
        w[u] = *reinterpret_cast<const float4*>(weight + j);
        p[u] = *reinterpret_cast<const int4*>(pos + j);
      } else {
        float* wu = reinterpret_cast<float*>(&w[u]);
        int* pu = reinterpret_cast<int*>(&p[u]);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          wu[x] = j + x < j1 ? weight[j + x] : 0.f;
          pu[x] = j + x < j1 ? pos[j + x] : 0;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + 4 * (q + u * kSelThreads);
      const float* wu = reinterpret_cast<const float*>(&w[u]);
      const int* pu = reinterpret_cast<const int*>(&p[u]);
      if (j >= j1) break;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (j + x < j1) {
          const uint32_t k = keep_key(wu[x], pu[x], a.sinks, recent_from);
          if (j + x - j0 < a.smem_keys) keys[j + x - j0] = k;
          const uint64_t v = packed(k, j + x);
          low = v < low ? v : low;
        }
      }
      // out of place: the scores below the budget (free places are written over below)
      if (!a.in_place) {
        if (a.vec && j + 3 < min(j1, a.budget)) {
          *reinterpret_cast<float4*>(weight_out + j) = w[u];
          *reinterpret_cast<int4*>(pos_out + j) = p[u];
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (j + x < min(j1, a.budget)) {
              weight_out[j + x] = wu[x];
              pos_out[j + x] = pu[x];
            }
        }
      }
    }
  }
  if (E <= 0) return;

  if (few) {
    auto least = [](uint64_t v) {   // over the warp
      const uint32_t hi = uint32_t(v >> 32), top = __reduce_min_sync(0xffffffffu, hi);
      const uint32_t lo = __reduce_min_sync(0xffffffffu, hi == top ? uint32_t(v) : 0xFFFFFFFFu);
      return uint64_t(top) << 32 | lo;
    };
    for (int e = 0; e < E; ++e) {
      const uint64_t mine = least(low);
      if (lane == 0) lowest[e & 1][warp] = mine;
      __syncthreads();
      const uint64_t all = least(lane < kSelWarps ? lowest[e & 1][lane] : ~uint64_t(0));
      const int j = int(~uint32_t(all));
      if (tid == 0) dropped[e] = j;
      if (j / 4 % kSelThreads == tid) {   // the next lowest of the thread that held it (j0 = 0 here)
        low = ~uint64_t(0);
        for (int x0 = 4 * tid; x0 < j1; x0 += 4 * kSelThreads)
          for (int x = x0; x < min(j1, x0 + 4); ++x) {
            const uint64_t v = packed(key(x), x);
            if (v > all) low = v < low ? v : low;   // those taken before are all below
          }
      }
    }
    __syncthreads();
    if (warp == 0) {
      // places below the budget that fall free, and tokens past it that stay, each in order
      const int mine = lane < E ? dropped[lane] : -1;
      const bool hole = lane < E && mine < a.budget;
      int rank_hole = 0;
      bool stays = lane < E;
      for (int e = 0; e < E; ++e) {
        const int other = __shfl_sync(0xffffffffu, mine, e);
        if (other < mine) rank_hole += other < a.budget ? 1 : 0;
        if (other == a.budget + lane) stays = false;
      }
      if (hole) few_dst[rank_hole] = mine;
      const uint32_t stay = __ballot_sync(0xffffffffu, stays);
      if (stays) few_src[__popc(stay & ((1u << lane) - 1u))] = a.budget + lane;
      if (lane == 0) found[0] = uint32_t(__popc(stay));
    }
    __syncthreads();
    // a warp a move
    for (int i = warp; i < int(found[0]); i += kSelWarps) {
      const int from = few_src[i], to = few_dst[i];
      const uint32_t ps = page_of(a.c, s, uint32_t(from)), pd = page_of(a.c, s, uint32_t(to));
      if (ps < a.c.n_pages && pd < a.c.n_pages) {
        // lanes 0-15 the K row's sixteen 16-byte pieces, lanes 16-31 the V row's
        uint8_t* pool = (lane < 16 ? a.c.k : a.c.v) + (lane & 15) * 16;
        *reinterpret_cast<uint4*>(pool + uint64_t(row_unit(a.c, pd, uint32_t(to), h)) * kRowBytes) =
            *reinterpret_cast<const uint4*>(pool + uint64_t(row_unit(a.c, ps, uint32_t(from), h)) * kRowBytes);
        if (lane == 0) weight_out[to] = weight[from];   // from >= budget > to
        if (lane == 1) pos_out[to] = pos[from];
      } else {   // no move at all: a row keeps its own scores
        record(a.c, kBadPage);
      }
    }
    return;
  }

  // ---- radix selection ----
  uint32_t prefix = 0, mask = 0, want = uint32_t(a.budget);   // rank, from the top, among keys that share `prefix`
  uint32_t equal = 0;
  constexpr int kShift[3] = {21, 10, 0}, kWidth[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = kShift[pass];
    const uint32_t n_bins = 1u << kWidth[pass];
    for (uint32_t i = tid; i < n_bins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int jb = j0 + warp * 32; jb < j1; jb += kSelThreads) {   // whole warps
      const int j = jb + lane;
      const uint32_t k = j < j1 ? key(j) : 0u;
      const bool on = j < j1 && (k & mask) == prefix;
      const uint32_t bin = (k >> shift) & (n_bins - 1u);
      // the first lane's bin is counted by one addition for all that share it
      // (runs of protected tokens or of zeros), the others one by one
      const uint32_t act = __ballot_sync(0xffffffffu, on);
      if (act) {
        const int lead = __ffs(act) - 1;
        const uint32_t bin0 = __shfl_sync(0xffffffffu, bin, lead);
        const uint32_t same = __ballot_sync(0xffffffffu, on && bin == bin0);
        if (lane == lead) atomicAdd(&hist[bin0], uint32_t(__popc(same)));
        else if (on && bin != bin0) atomicAdd(&hist[bin], 1u);
      }
    }
    __syncthreads();
    if (cs > 1) {
      // every block adds its bins to every block's sums
      if (pass == 0) ptx::cluster_wait();
      for (uint32_t i = tid; i < n_bins; i += kSelThreads) {
        const uint32_t n = hist[i];
        if (n == 0) continue;
        const uint32_t at = ptx::smem_u32(&bins[pass][i]);
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < cs) ptx::red_add_cluster(ptx::mapa_shared(at, uint32_t(r)), n);
      }
      sync();
    }
    // bins from the top, four (two in the last pass) a thread
    const uint32_t* all = cs > 1 ? bins[pass] : hist;
    const uint32_t per = n_bins / kSelThreads, top = n_bins - 1u - uint32_t(tid) * per;
    uint32_t sum = 0;
    for (uint32_t b = 0; b < per; ++b) sum += all[top - b];
    const uint32_t inc = warp_scan(sum);
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    const uint32_t sums = lane < kSelWarps ? warp_sums[lane] : 0u;
    uint32_t above = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0u);
    if (above < want && want <= above + sum) {
      for (uint32_t b = 0; b < per; ++b) {
        const uint32_t n = all[top - b];
        if (above < want && want <= above + n) {
          found[0] = top - b;
          found[1] = want - above;
          found[2] = n;
        }
        above += n;
      }
    }
    __syncthreads();
    prefix |= found[0] << shift;
    mask |= (n_bins - 1u) << shift;
    want = found[1];
    equal = found[2];
    if (want == equal) break;   // every key of the bin is kept: its lowest value will do as the bound
  }

  // kept: keys above `prefix`, and the first `want` of the `equal` keys at it.
  // Warp w of block r goes over the w-th part of the block's tokens: it counts
  // ties, then free places and moves, and writes them from where the warps and
  // blocks before it end.
  const int part = (seg / 32 + kSelWarps - 1) / kSelWarps * 32;
  const int wj0 = min(j1, j0 + warp * part), wj1 = min(j1, wj0 + part);
  // exclusive prefix of a warp's count over the warps and blocks before it, and the sum of all
  auto prefix_of = [&](uint32_t mine, int slot, uint32_t& sum) {
    __syncthreads();   // warp_sums of an earlier use are read
    if (lane == 0) warp_sums[warp] = mine;
    __syncthreads();
    const uint32_t sums = lane < kSelWarps ? warp_sums[lane] : 0u;
    uint32_t before = __reduce_add_sync(0xffffffffu, lane < warp ? sums : 0u);
    const uint32_t block = __reduce_add_sync(0xffffffffu, sums);
    sum = block;
    if (cs > 1) {
      if (tid < cs) ptx::st_cluster(ptx::mapa_shared(ptx::smem_u32(&block_sums[slot][rank]), uint32_t(tid)), block);
      sync();
      sum = 0;
      for (int r = 0; r < cs; ++r) {
        before += r < rank ? block_sums[slot][r] : 0u;
        sum += block_sums[slot][r];
      }
    }
    return before;
  };
  uint32_t ties_before = 0;
  if (equal > want) {
    uint32_t n = 0, sum;
    for (int jb = wj0; jb < wj1; jb += 32)
      n += uint32_t(__popc(__ballot_sync(0xffffffffu, jb + lane < wj1 && key(jb + lane) == prefix)));
    ties_before = prefix_of(n, 2, sum);
  }
  // which of a warp's 32 tokens from jb on are kept
  auto kept = [&](int jb, uint32_t& ties) {
    const int j = jb + lane;
    const uint32_t k = j < wj1 ? key(j) : 0u;
    bool keep = j < wj1 && k >= prefix;
    if (equal > want) {
      const uint32_t tie = __ballot_sync(0xffffffffu, j < wj1 && k == prefix);
      if (j < wj1 && k == prefix && ties + __popc(tie & ((1u << lane) - 1u)) >= want) keep = false;
      ties += uint32_t(__popc(tie));
    }
    return keep;
  };
  uint32_t ties = ties_before, holes = 0, moved = 0;
  for (int jb = wj0; jb < wj1; jb += 32) {
    const bool keep = kept(jb, ties);
    const int j = jb + lane;
    holes += uint32_t(__popc(__ballot_sync(0xffffffffu, j < wj1 && j < a.budget && !keep)));
    moved += uint32_t(__popc(__ballot_sync(0xffffffffu, j >= a.budget && keep)));
  }
  // two counts of a head, each below 2^30: one after the other
  uint32_t total = 0;
  uint32_t hole_at = prefix_of(holes, 0, total);
  uint32_t move_at = prefix_of(moved, 1, total);
  int32_t* src = a.src + int64_t(item) * a.max_moves;
  int32_t* dst = a.dst + int64_t(item) * a.max_moves;
  ties = ties_before;
  for (int jb = wj0; jb < wj1; jb += 32) {
    const bool keep = kept(jb, ties);
    const int j = jb + lane;
    const bool hole = j < wj1 && j < a.budget && !keep, move = j >= a.budget && keep;
    const uint32_t hb = __ballot_sync(0xffffffffu, hole), mb = __ballot_sync(0xffffffffu, move);
    if (hole) dst[hole_at + __popc(hb & ((1u << lane) - 1u))] = j;
    if (move) src[move_at + __popc(mb & ((1u << lane) - 1u))] = j;
    hole_at += uint32_t(__popc(hb));
    move_at += uint32_t(__popc(mb));
  }
  sync();   // the head's lists are written, and the kept scores
  if (tid == 0 && rank == 0) a.count[item] = int(total);
  for (int i = rank * kSelThreads + tid; i < int(total); i += cs * kSelThreads) {
    const int from = src[i], to = dst[i];
    // the second launch gets the rows themselves (equal ones: no move at all, a
    // row keeps its own scores)
    const uint32_t ps = page_of(a.c, s, uint32_t(from)), pd = page_of(a.c, s, uint32_t(to));
    const bool ok = ps < a.c.n_pages && pd < a.c.n_pages;
    if (ok) {
      weight_out[to] = weight[from];   // from >= budget > to: no index is both read and written
      pos_out[to] = pos[from];
    } else {
      record(a.c, kBadPage);
    }
    src[i] = ok ? int32_t(row_unit(a.c, ps, uint32_t(from), h)) : 0;
    dst[i] = ok ? int32_t(row_unit(a.c, pd, uint32_t(to), h)) : 0;
  }
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;

// The K and V rows of the moves the selection left, a warp kMoveUnroll rows at
// a time; and the new lengths, where they are in the place of the old.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a) {
  const int item = int(blockIdx.x) / a.blocks_per_item, part = int(blockIdx.x) - item * a.blocks_per_item;
  const int s = item / a.c.H, h = item - s * a.c.H;
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();
  if (!a.lens_here && part == 0 && h == 0 && threadIdx.x == 0) {
    const int L = seq_len(a.c, a.seq_lens, s);
    a.seq_lens_out[s] = min(L, a.budget);
  }
  const int n = a.count[item];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int32_t* src = a.src + int64_t(item) * a.max_moves;
  const int32_t* dst = a.dst + int64_t(item) * a.max_moves;
  // lanes 0-15 the K row's sixteen 16-byte pieces, lanes 16-31 the V row's
  uint8_t* pool = (lane < 16 ? a.c.k : a.c.v) + (lane & 15) * 16;
  for (int t0 = (part * (kMoveThreads / 32) + warp) * 32; t0 < n; t0 += a.blocks_per_item * kMoveThreads) {
    const bool there = t0 + lane < n;
    const uint32_t from = there ? uint32_t(src[t0 + lane]) : 0u, to = there ? uint32_t(dst[t0 + lane]) : 0u;
#pragma unroll 1
    for (int u0 = 0; u0 < 32 && t0 + u0 < n; u0 += kMoveUnroll) {
      uint4 x[kMoveUnroll];
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u)
        x[u] = *reinterpret_cast<const uint4*>(pool + uint64_t(__shfl_sync(0xffffffffu, from, u0 + u)) * kRowBytes);
#pragma unroll
      for (int u = 0; u < kMoveUnroll; ++u) {
        const uint32_t f = __shfl_sync(0xffffffffu, from, u0 + u), d = __shfl_sync(0xffffffffu, to, u0 + u);
        if (f != d) *reinterpret_cast<uint4*>(pool + uint64_t(d) * kRowBytes) = x[u];
      }
    }
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
  if (!aligned4(seq_lens) || !aligned4(next_pos) || !aligned4(pos) || !aligned4(weight))
    return fail(RKV_ERR_INVALID_ARG, "seq_lens/next_pos/pos/weight must be 4-byte aligned");
  const int64_t row = int64_t(cache->H) * kHD;
  if (new_row_stride < row) return fail(RKV_ERR_INVALID_ARG, "new_row_stride < H*D");
  if (new_row_stride % 8) return fail(RKV_ERR_INVALID_ARG, "rows of k_new/v_new must be 16-byte aligned");
  if (new_row_stride >= (int64_t(1) << 40)) return fail(RKV_ERR_INVALID_ARG, "new_row_stride too large");
  const int64_t rows = int64_t(cache->n_seqs) * n_new;
  if (new_row_stride >= kMaxSpan / rows) return fail(RKV_ERR_INVALID_ARG, "new_row_stride too large for the rows");
  const int64_t pieces = rows * cache->H * 16;
  if (rows >= (int64_t(1) << 31) || pieces >= (int64_t(1) << 31) - kInsertThreads * kInsertUnroll)
    return fail(RKV_ERR_UNSUPPORTED, "insert too large for one launch");
  const uint64_t sb = score_bytes(cache), lb = uint64_t(cache->n_seqs) * 4;
  st = check_apart({pool_k(cache), pool_v(cache), run_of("the scores pos", pos, sb), run_of("the scores weight", weight, sb),
                    status_of(cache)},
                   {{"new tokens (k_new)", k_new, rows, new_row_stride * 2, row * 2},
                    {"new tokens (v_new)", v_new, rows, new_row_stride * 2, row * 2},
                    run_of("seq_lens", seq_lens, lb), run_of("next_pos", next_pos, lb), table_of(cache)});
  if (st != RKV_OK) return st;
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
  const cudaError_t e = launch_overlapped(paged_insert_kernel, dim3((a.total + per - 1) / per), kInsertThreads, 0,
                                          static_cast<cudaStream_t>(stream), a);
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
  if (!aligned4(seq_lens) || !aligned4(weight) || !aligned4(pos) || !aligned4(next_pos) || !aligned4(seq_lens_out) ||
      !aligned4(weight_out) || !aligned4(pos_out))
    return fail(RKV_ERR_INVALID_ARG, "seq_lens/weight/pos/next_pos and the outputs must be 4-byte aligned");
  if (budget < 1) return fail(RKV_ERR_INVALID_ARG, "budget must be >= 1");
  if (sinks < 0 || recent < 0) return fail(RKV_ERR_INVALID_ARG, "sinks and recent must be >= 0");
  const bool in_place = weight_out == weight;
  if (in_place != (pos_out == pos)) return fail(RKV_ERR_INVALID_ARG, "weight_out and pos_out are in place both or neither");
  const size_t need = kvcache_paged_evict_workspace_size(cache, budget);
  const uint64_t sb = score_bytes(cache), lb = uint64_t(cache->n_seqs) * 4;
  st = check_apart({pool_k(cache), pool_v(cache), run_of("seq_lens_out", seq_lens_out, lb), run_of("weight_out", weight_out, sb),
                    run_of("pos_out", pos_out, sb), run_of("the workspace", workspace, std::min(need, workspace_bytes)),
                    status_of(cache)},
                   {run_of("seq_lens", seq_lens_out == seq_lens ? nullptr : seq_lens, lb),
                    run_of("weight", in_place ? nullptr : weight, sb), run_of("pos", in_place ? nullptr : pos, sb),
                    run_of("next_pos", next_pos, lb), table_of(cache)});
  if (st != RKV_OK) return st;
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
  a.vec = capacity(cache) % 4 == 0 && aligned16(weight) && aligned16(pos) && aligned16(weight_out) && aligned16(pos_out);
  a.count = static_cast<int32_t*>(workspace);
  a.src = a.count + items;
  a.dst = a.src + items * a.max_moves;
  a.lens_here = seq_lens_out != seq_lens;
  // blocks a head: one where the heads and sequences alone fill the machine
  // (or a head is short), else up to eight: 24 heads cut from 32,760 to 7,800
  // tokens (uniform weights) 63 us, with one block each 112; 12 heads from 4,097 to
  // 2,000 17.2 and 19.4; 76 heads from 2,542 to 1,200 30.1 and 26.5
  const int sms = sm_count();
  a.cluster = 1;
  while (a.cluster < kMaxCluster && items * a.cluster * 2 <= 2 * sms && capacity(cache) >= 2048 * int64_t(a.cluster))
    a.cluster *= 2;
  constexpr int kMaxSmemKeys = 48 * 1024;
  const int64_t seg = ((capacity(cache) + a.cluster - 1) / a.cluster + 31) / 32 * 32;
  a.smem_keys = int32_t(std::min<int64_t>(seg, kMaxSmemKeys));
  cudaError_t e = allow_smem<evict_select_kernel>(kMaxSmemKeys * 4);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(evict_select_kernel)");
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  e = launch_overlapped(evict_select_kernel, dim3(uint32_t(items * a.cluster)), kSelThreads, size_t(a.smem_keys) * 4, cs,
                        a, a.cluster);
  if (e != cudaSuccess) return cuda_fail(e, "evict_select_kernel launch");
  // no second launch where the selection moves every row itself and the new
  // lengths are apart from the old
  if (a.cluster == 1 && capacity(cache) - budget <= kFew && a.lens_here) return RKV_OK;
  // enough blocks to fill the machine about twice over, no more than the moves need
  const int64_t most = std::max<int64_t>(1, (a.max_moves + kMoveThreads - 1) / kMoveThreads);
  const int64_t want = (int64_t(sms) * 16 + items - 1) / items;
  a.blocks_per_item = int32_t(std::min(most, std::max<int64_t>(1, want)));
  e = launch_overlapped(evict_move_kernel, dim3(uint32_t(items * a.blocks_per_item)), kMoveThreads, 0, cs, a);
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
