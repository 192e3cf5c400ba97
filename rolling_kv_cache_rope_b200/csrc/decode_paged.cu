// Attention of the newest tokens of every sequence over a paged KV cache,
// split over the cache's length and joined; optionally the attention weight
// each cached token received is added up.
//
// What it computes (sequence s, query i of Lq, query head h, key head g of H,
// G query heads to a key head, c = L_s - Lq + i):
//   o = sum_j p_j v_j,  p = softmax over the visible j of scale q . k_j,
//   visible: j <= c and (window == 0 or j > c - window or j < sinks)
//   weight_out[s][g][j] = weight_in[s][g][j] + sum of p_j over i and h in g
// Source: attention over a rolling KV cache ("Amazon and Reactor tune Trainium
// for real-time video generation", section "Three problems for generic
// compilers"), here for token streams of different lengths.
//
// Bound: every visible K and V row is read once, 512 bytes for 4 * 128 flops
// per query row; with at most 32 rows to a key head the kernel is bound by
// HBM.  With the queries on M a tcgen05 tile has at least 64 rows, most of them
// empty here; the warp-level m16n8k16 product takes 16 rows and is far from its
// own limit at this bandwidth (16 keys of a head cost 32 of them per 8 KB).  From
// 17 rows on its chains bound the kernel instead (figures at decode_shape); keys
// on M and rows on N would leave no row of a tcgen05 tile empty and is not built:
// it needs every page's rows in swizzled tiles and P^T through shared memory.
//
// Split: the key rows of all (sequence, key head, row block) items, in steps
// of 64 or 32 keys, form one list of T steps, and each of C blocks takes T / C of
// them in a row: every block gets the same bytes whatever the lengths.  An
// item that lies in one block is finished there; of the others each block
// leaves its running maximum, sum and unnormalised O (at most two per block),
// and a second launch joins them in the order of the keys, so the result does
// not depend on timing.  Each kernel derives the list from seq_lens itself:
// nothing is planned on the host, and a captured launch serves growing
// sequences.
//
// Inside a block: four warps, each with 16 of a step's 64 keys (more rows than
// 16: two or four warps share 32 keys, 16 rows each) and its own
// maximum, sum and O in registers, meet only where an item begins or ends.
// Each warp copies its own K and V rows with 16-byte asynchronous copies into
// its part of a ring of stages, so several steps (32 KB each) are in flight
// per SM without registers holding data, across the ends of items too.  A row
// that is not visible to any query (past the end, outside window and sinks, on
// a bad page) is not read but zero-filled, so nothing it holds can enter a sum.
//
// Measured (GPU time alone): one stream of 32,760 tokens, 12 heads, 42 us for
// 201 MB; 64 streams of 1 to 8,192 tokens, 32 / 8 heads, 186 to 194 us from one
// GPU to the next for 1,112 MB (5.7 to 6.0 TB/s).  About 10 us of either do not
// shrink with the bytes: finding the steps 2, the first copies 3, merging the
// warps 2, the join 4; and the SMs end 15 to 20% apart, although each reads the
// same bytes.  With weights (24 streams of 2,000 to 4,097 tokens, 24 / 8 heads,
// 317 MB): 68 us.
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace rkv {
namespace paged {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = kDecWarps * 32;
constexpr int kDecPerSm = 2;                           // blocks of the main launch an SM holds
constexpr int kGroupKeys = 16;                         // keys of one matrix product
constexpr int kGroupBytes = kGroupKeys * int(kRowBytes);
constexpr int kRingBytes = 96 * 1024;                  // K and V stages of a block
constexpr float kMaxSlack = 8.0f;                      // the running maximum moves past 2^8 growth only
constexpr int kMaxRows = 4096;                         // query rows of a key head (Lq * G)
constexpr int kJoinThreads = 256;

struct DecodeArgs {
  CacheDev c;
  const uint8_t* q;
  uint8_t* o;
  int64_t q_row, o_row;          // bytes between rows
  const int32_t* seq_lens;
  const float* weight_in;
  float* weight_out;
  float* part_o;                 // [C][2][rows_blk][kHD]
  float2* part_ml;               // [C][2][rows_blk] running maximum (log2 units) and sum
  float2* item_ml;               // [items][rows_blk] of items finished in one block (weights only)
  float* scores;                 // [T][rows_blk][step_keys] scaled scores, log2 units (weights only)
  struct BlockRec* recs;         // [C]
  float scale_log2;
  int32_t Hq, Lq, G, rows;       // rows = Lq * G
  FastDiv div_G;
  int32_t rows_tile;             // rows a row block has room for: 16, 32 or 64
  int32_t step_keys;             // keys of a step: 64 or 32
  int32_t rows_blk, n_blk;       // rows of a full row block (min(rows, rows_tile)), row blocks
  int32_t window, sinks;
  int32_t main_blocks;           // C
  FastDiv div_blocks;
};

// What a block of the main launch leaves for the join: the place its steps
// began at, and the item it joins (one that began in the block and goes on in
// others; parts = 0: none).
struct alignas(16) BlockRec {
  int32_t s, g, blk, c;         // first step
  int32_t first, n, total;      // ... its number in the whole list, the block's steps, the list's length
  int32_t join_s, join_g, join_blk, parts, slot;
};

// The keys any query of a sequence of length L sees, as a list of `span`
// entries: [0, se), then [lo, L).
struct Span {
  int L, se, lo, span;
  __device__ __forceinline__ int steps(int keys) const { return (span + keys - 1) / keys; }
};

__device__ __forceinline__ Span span_of(const DecodeArgs& a, int L) {
  Span r;
  r.L = L;
  r.lo = a.window > 0 ? max(0, max(0, L - a.Lq) - a.window + 1) : 0;   // of the first query there is
  r.se = min(a.sinks, r.lo);
  r.span = L > 0 ? r.se + L - r.lo : 0;
  return r;
}

__device__ __forceinline__ int seq_steps(const DecodeArgs& a, int s) {
  return span_of(a, seq_len(a.c, a.seq_lens, s)).steps(a.step_keys);
}

// The list of steps: sequence by sequence, `items` times the steps of each.
// Whole warps call these; every lane gets the result.
struct Place {
  int s, base;   // sequence a step falls into, and the steps before that sequence
};
__device__ __forceinline__ int total_steps(const DecodeArgs& a, int items) {
  int total = 0;
  for (int s = threadIdx.x & 31; s < a.c.n_seqs; s += 32) total += seq_steps(a, s);
  return __reduce_add_sync(0xffffffffu, total) * items;
}
__device__ __forceinline__ Place find_step(const DecodeArgs& a, int items, int x) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b = 0; b < a.c.n_seqs; b += 32) {
    const int s = b + lane;
    const int own = s < a.c.n_seqs ? seq_steps(a, s) * items : 0;
    int inc = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, before + inc > x);
    if (hit) {
      const int l = __ffs(hit) - 1;
      return {b + l, __shfl_sync(0xffffffffu, before + inc - own, l)};
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return {a.c.n_seqs, before};   // x is past the list
}

// How T steps are shared out: the first T % C blocks take one more than the
// others.  Blocks past T take none.
struct Split {
  int q, r;   // T / C, T % C
  __device__ __forceinline__ Split(int total, const FastDiv& blocks)
      : q(int(fdiv(uint32_t(total), blocks))), r(total - int(fdiv(uint32_t(total), blocks)) * int(blocks.d)) {}
  __device__ __forceinline__ int first(int b) const { return b * q + min(b, r); }
  __device__ __forceinline__ int count(int b) const { return q + (b < r ? 1 : 0); }
  __device__ __forceinline__ int block_of(int x) const {   // x < T
    const int wide = r * (q + 1);
    return x < wide ? x / (q + 1) : r + (x - wide) / q;
  }
};

// A position in the list of steps: sequence, key head and row block of the
// item, step of the item.
struct Cursor {
  Span sp;
  const int32_t* table;   // the sequence's row of the page table
  int s, g, blk, c, nc;
};

__device__ __forceinline__ void load_seq(const DecodeArgs& a, Cursor& u) {
  while (true) {   // sequences without a visible key have no steps
    u.sp = span_of(a, seq_len(a.c, a.seq_lens, u.s));
    u.nc = u.sp.steps(a.step_keys);
    if (u.nc > 0 || u.s + 1 >= a.c.n_seqs) break;
    ++u.s;
  }
  u.table = a.c.table + int64_t(u.s) * a.c.table_stride;
}

__device__ __forceinline__ void advance(const DecodeArgs& a, Cursor& u) {
  if (++u.c < u.nc) return;
  u.c = 0;
  if (++u.blk < a.n_blk) return;
  u.blk = 0;
  if (++u.g < a.c.H) return;
  u.g = 0;
  if (u.s + 1 >= a.c.n_seqs) return;   // past the last step: not used
  ++u.s;
  load_seq(a, u);
}

// Entry x of a sequence's visible list -> its token.
__device__ __forceinline__ int token_of(const Span& sp, int x) { return x < sp.se ? x : x - sp.se + sp.lo; }

// Shared memory of a block whose warps split into NR row tiles: 4 / NR key
// tiles a step, each read by NR warps.  A tile is 16 keys, or two groups of 16
// where warps share it: they then meet, and form addresses and masks, half as
// often, and two chains of products run side by side (16 streams of 8,000
// tokens, 4 key heads: 32 rows 61 us, 73 with one group; 64 rows 93, 121).
// With one row tile HBM is the bound, and smaller tiles keep more steps in
// flight.
template <int NR>
struct DecSmem {
  static constexpr int kKeyTiles = kDecWarps / NR;
  static constexpr int kGroups = NR == 1 ? 1 : 2;
  static constexpr int kTileKeys = kGroups * kGroupKeys;
  static constexpr int kTileBytes = kGroups * kGroupBytes;   // of K, and of V
  static constexpr int kStepKeys = kKeyTiles * kTileKeys;
  static constexpr int kStageBytes = kKeyTiles * 2 * kTileBytes;
  static constexpr int kStages = kRingBytes / kStageBytes;
  static constexpr int kOffMl = kRingBytes;
  static constexpr int kOffMask = kOffMl + kDecWarps * 16 * 8;
  static constexpr int kBytes = kOffMask + kStages * kDecWarps * 4;
  // the stage an item's last step was in serves as the buffer its warps' O
  // meet in: so many floats per warp
  static constexpr int kMergeFloats = kStageBytes / 4 / kDecWarps;
  static_assert(kDecPerSm * (kBytes + 1024) <= 228 * 1024, "blocks of one SM");
};

template <int NR, bool kWeights>
__global__ void __launch_bounds__(kDecThreads, kDecPerSm) decode_paged_kernel(const __grid_constant__ DecodeArgs a) {
  using SM = DecSmem<NR>;
  constexpr int kStages = SM::kStages, kKeyTiles = SM::kKeyTiles;
  constexpr int kGroups = SM::kGroups, kTileKeys = SM::kTileKeys, kTileBytes = SM::kTileBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kt = warp % kKeyTiles, rt = warp / kKeyTiles;   // the warp's key tile and row tile
  const int per_step = a.c.H * a.n_blk;
  // nothing is read before the launches ahead are complete, nor may the join
  // read the lengths before
  ptx::pdl_wait();
  ptx::pdl_launch_dependents();

  const int total = total_steps(a, per_step);
  const Split split(total, a.div_blocks);
  const int n_steps = split.count(blockIdx.x);
  const int c0 = split.first(blockIdx.x);
  BlockRec& rec = a.recs[blockIdx.x];
  if (n_steps == 0 && tid == 0) {
    rec.n = 0;
    rec.parts = 0;
  }
  if (n_steps > 0) {
    Cursor cu;   // the step computed next
    {
      const Place pl = find_step(a, per_step, c0);
      cu.s = pl.s;
      load_seq(a, cu);
      const int it = (c0 - pl.base) / cu.nc;
      cu.c = (c0 - pl.base) - it * cu.nc;
      cu.g = a.n_blk == 1 ? it : it / a.n_blk;
      cu.blk = it - cu.g * a.n_blk;
    }
    if (tid == 0) {
      rec.s = cu.s;
      rec.g = cu.g;
      rec.blk = cu.blk;
      rec.c = cu.c;
      rec.first = c0;
      rec.n = n_steps;
      rec.total = total;
    }
    Cursor is = cu;   // the step copied next
    int issued = 0;
    uint32_t st_is = 0, st = 0;   // stage of the issued / computed step
    float2* ml = reinterpret_cast<float2*>(smem + SM::kOffMl);
    uint32_t* vmask = reinterpret_cast<uint32_t*>(smem + SM::kOffMask);

    // Rows of 256 bytes lie in shared memory as sixteen 16-byte pieces, piece
    // p of row r at place p ^ (r % 8), so that eight rows' pieces of one
    // column block fall into different banks.  Of the places a lane touches
    // only four differ beyond a constant: x ^ 2c for c = 0..3.
    constexpr int kCopies = kTileKeys / NR / 2;             // row pairs of a tile this warp copies
    constexpr int kDistinct = kCopies < 4 ? kCopies : 4;
    constexpr uint32_t kAllKeys = kTileKeys == 32 ? 0xFFFFFFFFu : (1u << (kTileKeys & 31)) - 1u;
    uint32_t dofs[kDistinct], kofs[4], vofs[4];
    {
      const uint32_t hi = uint32_t(lane) >> 4, low = uint32_t(lane) & 7u, piece = uint32_t(lane) & 15u;
      const uint32_t tile = sbase + uint32_t(kt) * (2 * kTileBytes);
#pragma unroll
      for (int c = 0; c < kDistinct; ++c) {
        // copies: rows 2c + hi of the warp's share of the tile, piece `piece`
        const uint32_t r = uint32_t(rt * (kTileKeys / NR) + 2 * c) + hi;
        dofs[c] = tile + r * kRowBytes + ((piece ^ (r & 7u)) << 4);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        // K operand: keys 0-7 and 8-15, column pieces 2kk and 2kk + 1
        kofs[c] = tile + (low + (hi << 3)) * kRowBytes + ((((uint32_t(lane) >> 3) & 1u) ^ low ^ (2u * c)) << 4);
        // V operand: keys 0-15, column pieces 2np and 2np + 1
        vofs[c] = tile + kTileBytes + piece * kRowBytes + ((hi ^ low ^ (2u * c)) << 4);
      }
    }
    const uint8_t* const k_lane = a.c.k + (lane & 15) * 16;
    const uint8_t* const v_lane = a.c.v + (lane & 15) * 16;

    // Copy this warp's share of its key tile of step `is` into its stage.
    auto issue = [&]() {
      if (issued < n_steps) {
        const int x0 = is.c * SM::kStepKeys + kt * kTileKeys, x = x0 + (lane & (kTileKeys - 1));
        if (x0 < is.sp.span) {   // a tile past the list's end is not computed either
          bool ok = x < is.sp.span;
          uint32_t unit = 0;
          if (ok) {
            const uint32_t j = uint32_t(token_of(is.sp, x));
            const uint32_t pg = fdiv(j, a.c.div_P);
            const uint32_t page = uint32_t(is.table[pg]);
            ok = page < a.c.n_pages;
            unit = page * a.c.page_units + (j - pg * a.c.P) * uint32_t(a.c.H) + uint32_t(is.g);
            if (!ok) record(a.c, kBadPage);
          }
          const uint32_t mask = __ballot_sync(0xffffffffu, ok) & kAllKeys;
          if (lane == 0) vmask[st_is * kDecWarps + warp] = mask;
          const uint32_t so = st_is * SM::kStageBytes;
          const int kk0 = rt * (kTileKeys / NR) + (lane >> 4);
          unit = ok ? unit : 0u;
          auto rows = [&](auto ic) {
            constexpr int i = decltype(ic)::value;
            if constexpr (i < kCopies) {
              constexpr int kOff = (i / 4) * 8 * int(kRowBytes);   // rows 8 apart swizzle alike
              const uint32_t d = dofs[i % kDistinct] + so;
              const uint64_t off = uint64_t(__shfl_sync(0xffffffffu, unit, kk0 + 2 * i)) * kRowBytes;
              if (mask == kAllKeys) {
                ptx::cp_async16<kOff>(d, k_lane + off);
                ptx::cp_async16<kOff + kTileBytes>(d, v_lane + off);
              } else {   // rows that are not there are zeros
                const uint32_t bytes = ((mask >> (kk0 + 2 * i)) & 1u) << 4;
                ptx::cp_async16_fill<kOff>(d, k_lane + off, bytes);
                ptx::cp_async16_fill<kOff + kTileBytes>(d, v_lane + off, bytes);
              }
            }
          };
          rows(std::integral_constant<int, 0>());
          rows(std::integral_constant<int, 1>());
          rows(std::integral_constant<int, 2>());
          rows(std::integral_constant<int, 3>());
          rows(std::integral_constant<int, 4>());
          rows(std::integral_constant<int, 5>());
          rows(std::integral_constant<int, 6>());
          rows(std::integral_constant<int, 7>());
        }
        st_is = st_is + 1 == kStages ? 0 : st_is + 1;
        ++issued;
        if (issued < n_steps) advance(a, is);
      }
      ptx::cp_async_commit();
    };

    uint32_t qf[8][4];   // the warp's 16 Q rows as A operands
    float O[16][4];
    float m[2], l[2];    // of rows lane / 4 and 8 + lane / 4
    int all_lo = 0, all_hi = 0;         // keys in [all_lo, all_hi) are visible to every row
    int frag_c0 = 0, frag_t0 = 0;       // step of the item, and of the block, this part of the item began at
    bool first = true;

#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) issue();

#pragma unroll 1
    for (int t = 0; t < n_steps; ++t) {
      if constexpr (NR == 1) {
        issue();
        ptx::cp_async_wait<kStages - 1>();
        __syncwarp();
      } else {
        // the warps of a key tile: all their shares of this step have landed,
        // and all are done with the stage that is filled next
        ptx::cp_async_wait<kStages - 2>();
        ptx::named_sync(1 + kt, 32 * NR);
        issue();
      }
      if (first) {
        first = false;
        frag_c0 = cu.c;
        frag_t0 = t;
        const int last_q = min(a.rows, (cu.blk + 1) * (NR * 16)) - 1, first_q = cu.blk * (NR * 16);
        all_hi = max(0, cu.sp.L - a.Lq + int(fdiv(uint32_t(first_q), a.div_G)) + 1);
        all_lo = a.window > 0 ? max(0, cu.sp.L - a.Lq + int(fdiv(uint32_t(last_q), a.div_G)) - a.window + 1) : 0;
        // Q straight from global memory: its latency is a small part of an
        // item's time, and the stages under way keep the memory busy
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = cu.blk * (NR * 16) + rt * 16 + e * 8 + (lane >> 2);
          const bool there = row < a.rows;
          const int qi = there ? int(fdiv(uint32_t(row), a.div_G)) : 0;
          const int h = there ? cu.g * a.G + row - qi * a.G : 0;
          const uint32_t* src = reinterpret_cast<const uint32_t*>(
              a.q + (int64_t(cu.s) * a.Lq + qi) * a.q_row + int64_t(h) * kRowBytes + (lane & 3) * 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            qf[kk][e] = there ? __ldg(src + 8 * kk) : 0u;
            qf[kk][2 + e] = there ? __ldg(src + 8 * kk + 4) : 0u;
          }
        }
#pragma unroll
        for (int n = 0; n < 16; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[n][e] = 0.f;
        m[0] = m[1] = -INFINITY;
        l[0] = l[1] = 0.f;
      }

      const int x0 = cu.c * SM::kStepKeys + kt * kTileKeys;
      if (x0 < cu.sp.span) {
        const uint32_t mask = vmask[st * kDecWarps + warp];
        const uint32_t so = st * SM::kStageBytes;
        // S = Q K^T, 16 rows x 16 or 32 keys, eight to an accumulator
        constexpr int kCols = 2 * kGroups;
        float S[kCols][4];
#pragma unroll
        for (int n = 0; n < kCols; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) S[n][e] = 0.f;
        auto s_step = [&](auto kc) {
          constexpr int kk = decltype(kc)::value;
          uint32_t b[4];   // keys 0-7 of columns 16kk.. and 16kk + 8.., then keys 8-15
          ptx::ldsm4<(kk >> 2) * 128>(kofs[kk & 3] + so, b);
          ptx::mma_bf16(S[0], qf[kk], b[0], b[1]);
          ptx::mma_bf16(S[1], qf[kk], b[2], b[3]);
          if constexpr (kGroups == 2) {
            ptx::ldsm4<(kk >> 2) * 128 + kGroupBytes>(kofs[kk & 3] + so, b);
            ptx::mma_bf16(S[kCols - 2], qf[kk], b[0], b[1]);
            ptx::mma_bf16(S[kCols - 1], qf[kk], b[2], b[3]);
          }
        };
        s_step(std::integral_constant<int, 0>());
        s_step(std::integral_constant<int, 1>());
        s_step(std::integral_constant<int, 2>());
        s_step(std::integral_constant<int, 3>());
        s_step(std::integral_constant<int, 4>());
        s_step(std::integral_constant<int, 5>());
        s_step(std::integral_constant<int, 6>());
        s_step(std::integral_constant<int, 7>());
        // the tile holds the tokens from j0 on unless the list jumps from the
        // sinks to the window inside it; no mask is needed where every row sees all
        const int j0 = token_of(cu.sp, x0);
        const bool plain = mask == kAllKeys && (x0 >= cu.sp.se || x0 + kTileKeys <= cu.sp.se) &&
                           j0 + kTileKeys <= all_hi && (j0 >= all_lo || j0 + kTileKeys <= a.sinks);
        if (!plain) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the row sees keys <= c that are past c - window or among the sinks
            const int row = cu.blk * (NR * 16) + rt * 16 + e * 8 + (lane >> 2);
            const int c = row < a.rows ? cu.sp.L - a.Lq + int(fdiv(uint32_t(row), a.div_G)) : -1;
            const int from = a.window > 0 ? c - a.window + 1 : 0;
#pragma unroll
            for (int n = 0; n < kCols; ++n)
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const int kk = n * 8 + 2 * (lane & 3) + f;
                const int j = token_of(cu.sp, x0 + kk);
                const bool vis = ((mask >> kk) & 1u) && j <= c && (j >= from || j < a.sinks);
                if (!vis) S[n][2 * e + f] = -INFINITY;
              }
          }
        }
        if constexpr (kWeights) {
          const int64_t step = int64_t(c0) + t;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = rt * 16 + e * 8 + (lane >> 2);
            if (r < a.rows_blk) {
              float* dst = a.scores + (step * a.rows_blk + r) * SM::kStepKeys + kt * kTileKeys + 2 * (lane & 3);
#pragma unroll
              for (int n = 0; n < kCols; ++n)
                *reinterpret_cast<float2*>(dst + 8 * n) =
                    make_float2(S[n][2 * e] * a.scale_log2, S[n][2 * e + 1] * a.scale_log2);
            }
          }
        }
        // a lane sees a quarter of a row's scores; only where one of them
        // outgrows the running maximum do the row's lanes find the tile's
        float mx[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[e] = fmaxf(fmaxf(S[0][2 * e], S[0][2 * e + 1]), fmaxf(S[1][2 * e], S[1][2 * e + 1]));
          if constexpr (kGroups == 2)
            mx[e] = fmaxf(mx[e], fmaxf(fmaxf(S[kCols - 2][2 * e], S[kCols - 2][2 * e + 1]),
                                       fmaxf(S[kCols - 1][2 * e], S[kCols - 1][2 * e + 1])));
          mx[e] *= a.scale_log2;
        }
        if (__any_sync(0xffffffffu, mx[0] > m[0] + kMaxSlack || mx[1] > m[1] + kMaxSlack)) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
            const float nm = mx[e] > m[e] + kMaxSlack ? mx[e] : m[e];
            f[e] = m[e] == nm ? 1.f : ptx::ex2_approx(m[e] - nm);
            m[e] = nm;
            l[e] *= f[e];
          }
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            O[n][0] *= f[0];
            O[n][1] *= f[0];
            O[n][2] *= f[1];
            O[n][3] *= f[1];
          }
        }
        // P = exp2(S - m): summed in fp32, rounded to bf16 for P V (at most
        // half a step of bf16, 2^-8 of each weight, as the output's own
        // rounding).  S's accumulator layout is the A operand's as it stands.
        uint32_t P[kGroups][4];
        const float u0 = m[0] == -INFINITY ? 0.f : m[0], u1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
        for (int n = 0; n < kCols; ++n) {
          const float p0 = ptx::ex2_approx(fmaf(S[n][0], a.scale_log2, -u0));
          const float p1 = ptx::ex2_approx(fmaf(S[n][1], a.scale_log2, -u0));
          const float p2 = ptx::ex2_approx(fmaf(S[n][2], a.scale_log2, -u1));
          const float p3 = ptx::ex2_approx(fmaf(S[n][3], a.scale_log2, -u1));
          l[0] += p0 + p1;
          l[1] += p2 + p3;
          P[n / 2][2 * (n & 1)] = pack_bf16x2(p0, p1);
          P[n / 2][2 * (n & 1) + 1] = pack_bf16x2(p2, p3);
        }
        // O += P V
        auto o_step = [&](auto nc) {
          constexpr int np = decltype(nc)::value;
          uint32_t b[4];   // keys 0-7 / 8-15 of columns 16np.., then of 16np + 8..
          ptx::ldsm4_trans<(np >> 2) * 128>(vofs[np & 3] + so, b);
          ptx::mma_bf16(O[2 * np], P[0], b[0], b[1]);
          ptx::mma_bf16(O[2 * np + 1], P[0], b[2], b[3]);
          if constexpr (kGroups == 2) {
            ptx::ldsm4_trans<(np >> 2) * 128 + kGroupBytes>(vofs[np & 3] + so, b);
            ptx::mma_bf16(O[2 * np], P[kGroups - 1], b[0], b[1]);
            ptx::mma_bf16(O[2 * np + 1], P[kGroups - 1], b[2], b[3]);
          }
        };
        o_step(std::integral_constant<int, 0>());
        o_step(std::integral_constant<int, 1>());
        o_step(std::integral_constant<int, 2>());
        o_step(std::integral_constant<int, 3>());
        o_step(std::integral_constant<int, 4>());
        o_step(std::integral_constant<int, 5>());
        o_step(std::integral_constant<int, 6>());
        o_step(std::integral_constant<int, 7>());
      }
      if constexpr (NR == 1) __syncwarp();   // the warp is done with the stage issue() fills next

      if (cu.c + 1 == cu.nc || t + 1 == n_steps) {
        // ---- the item ends here, in this block: join the key tiles' parts ----
        const bool whole = frag_c0 == 0 && cu.c + 1 == cu.nc;
        const int rows_here = min(a.rows - cu.blk * (NR * 16), NR * 16);
        const int part = frag_t0 == 0 ? 0 : 1;
        const int64_t slot = (int64_t(blockIdx.x) * 2 + part) * a.rows_blk;
        if (t + 1 == n_steps && tid == 0) {
          // the item goes on in other blocks: this one joins it if it began here
          rec.parts = frag_c0 == 0 && !whole ? split.block_of(c0 + t - cu.c + cu.nc - 1) - int(blockIdx.x) + 1 : 0;
          rec.join_s = cu.s;
          rec.join_g = cu.g;
          rec.join_blk = cu.blk;
          rec.slot = part;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
          l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
          if ((lane & 3) == 0) ml[warp * 16 + e * 8 + (lane >> 2)] = make_float2(m[e], l[e]);
        }
        __syncthreads();   // and every warp is done with the stage: it holds the O parts from here
        auto joined = [&](int r, float& M, float& sum) {   // row r of the block, over its key tiles
          const float2* x = ml + (r >> 4) * kKeyTiles * 16 + (r & 15);
          M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kKeyTiles; ++w) M = fmaxf(M, x[w * 16].x);
          sum = 0.f;
#pragma unroll
          for (int w = 0; w < kKeyTiles; ++w)
            sum += x[w * 16].x == -INFINITY ? 0.f : x[w * 16].y * ptx::ex2_approx(x[w * 16].x - M);
        };
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float M, sum;
          joined(rt * 16 + e * 8 + (lane >> 2), M, sum);
          f[e] = m[e] == -INFINITY ? 0.f : ptx::ex2_approx(m[e] - M);
        }
        if (tid < rows_here && (!whole || kWeights)) {
          float M, sum;
          joined(tid, M, sum);
          if (!whole)
            a.part_ml[slot + tid] = make_float2(M, sum);
          else
            a.item_ml[(int64_t(cu.s) * per_step + cu.g * a.n_blk + cu.blk) * a.rows_blk + tid] = make_float2(M, sum);
        }
        // rows of cw columns at a time, padded by 8 floats so that four rows
        // fall into different banks
        float* const merge = reinterpret_cast<float*>(smem + st * SM::kStageBytes);
        const int tile_rows = min(rows_here, 16);
        int cw = 128;
        while (tile_rows * (cw + 8) > SM::kMergeFloats) cw >>= 1;
        const int pad = cw + 8;
        for (int cb = 0; cb < kHD; cb += cw) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = e * 8 + (lane >> 2);
            if (rt * 16 + r < rows_here) {
              float* dst = merge + warp * SM::kMergeFloats + r * pad + 2 * (lane & 3) - cb;
#pragma unroll
              for (int n = 0; n < 16; ++n)
                if (n * 8 >= cb && n * 8 < cb + cw)
                  *reinterpret_cast<float2*>(dst + n * 8) = make_float2(O[n][2 * e] * f[e], O[n][2 * e + 1] * f[e]);
            }
          }
          __syncthreads();
          for (int idx = tid; idx < rows_here * (cw / 2); idx += kDecThreads) {
            const int r = idx / (cw / 2), col = 2 * (idx - r * (cw / 2));
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kKeyTiles; ++w) {
              const float2 x = *reinterpret_cast<const float2*>(
                  merge + ((r >> 4) * kKeyTiles + w) * SM::kMergeFloats + (r & 15) * pad + col);
              sum.x += x.x;
              sum.y += x.y;
            }
            if (whole) {
              float M, ls;
              joined(r, M, ls);
              const float inv = ls > 0.f ? 1.f / ls : 0.f;
              const int row = cu.blk * (NR * 16) + r, qi = int(fdiv(uint32_t(row), a.div_G));
              const int h = cu.g * a.G + row - qi * a.G;
              *reinterpret_cast<uint32_t*>(a.o + (int64_t(cu.s) * a.Lq + qi) * a.o_row + int64_t(h) * kRowBytes +
                                           (cb + col) * 2) = pack_bf16x2(sum.x * inv, sum.y * inv);
            } else {
              *reinterpret_cast<float2*>(a.part_o + (slot + r) * kHD + cb + col) = sum;
            }
          }
          __syncthreads();
        }
        first = true;
      }
      st = st + 1 == kStages ? 0 : st + 1;
      if (t + 1 < n_steps) advance(a, cu);
    }
  }

  // outputs of sequences without a visible key
  for (int s = blockIdx.x; s < a.c.n_seqs; s += a.main_blocks) {
    if (span_of(a, seq_len(a.c, a.seq_lens, s)).span > 0) continue;
    for (int x = tid; x < a.Lq * a.Hq * 16; x += kDecThreads) {
      const int qi = x / (a.Hq * 16), rest = x - qi * (a.Hq * 16);
      *reinterpret_cast<uint4*>(a.o + (int64_t(s) * a.Lq + qi) * a.o_row + rest * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
}

// ---------------------------------------------------------------------------
// join: the items that lie in several blocks, and the weights
// ---------------------------------------------------------------------------

// Row r of part i of an item whose first part is slot `first` of the parts and
// begins in block b0.
__device__ __forceinline__ int64_t part_row(const DecodeArgs& a, int b0, int slot, int i, int r) {
  return (int64_t(b0 + i) * 2 + (i == 0 ? slot : 0)) * a.rows_blk + r;
}

// (blocks per SM: four without weights, in 64 registers.  Four query tokens of
// 16 streams, 32 rows: 43.1 us, with three blocks 43.7; but 8 rows of 3 streams
// of 31,012 tokens, one key head, take 37 where three blocks take 26, because the
// path over many parts spills.  Three with weights: 24 streams measure 66.1
// either way, 40 rows of one stream 67.4 and with four blocks 62.)
template <bool kWeights>
__global__ void __launch_bounds__(kJoinThreads, kWeights ? 3 : 4) decode_join_kernel(const __grid_constant__ DecodeArgs a) {
  __shared__ float4 part[kJoinThreads / 32][32];
  __shared__ float2 part_sum[kJoinThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  ptx::pdl_wait();   // the main launch's parts are written
  ptx::pdl_launch_dependents();
  // Main block b = blockIdx.x may hold the first part of an item that goes on in
  // the blocks after it.  A row is joined by `per` warps (all eight where there
  // is one row), each with every per-th part; they meet in order in shared
  // memory.  The first parts are loaded beside the record that says whether and
  // how many there are: what is not a part is not used.  One row: 42.2 us for a
  // stream of 32,760 tokens and 12 heads, 42.9 with one warp a row.  From five
  // rows on a warp has a row to itself: 8 rows of 16 streams of 2,000 tokens 32.4
  // us, with eight warps a row 35.9, 32 rows 43.2 and 57.9.  Where few key heads
  // leave an item a hundred parts it is the slower way, 37 us against 21.7 (3
  // streams of 31,012 tokens, one key head, 8 rows).
  const int per = a.rows_blk == 1 ? 8 : (a.rows_blk == 2 ? 4 : (a.rows_blk <= 4 ? 2 : 1));
  const int b0 = blockIdx.x, w0 = warp % per, r = int(blockIdx.y) * (8 / per) + warp / per;
  const bool row_ok = r < a.rows_blk;
  constexpr int kAheadParts = 4;
  float2 ml0 = make_float2(-INFINITY, 0.f), ml1 = ml0;   // part w0 + lane * per; slot 1 of the first block
  float4 o_ahead[kAheadParts], o1 = make_float4(0.f, 0.f, 0.f, 0.f);
  if (row_ok) {
    if (b0 + w0 + lane * per < a.main_blocks) ml0 = a.part_ml[part_row(a, b0, 0, w0 + lane * per, r)];
    if (w0 == 0) {
      ml1 = a.part_ml[part_row(a, b0, 1, 0, r)];
      o1 = *reinterpret_cast<const float4*>(a.part_o + part_row(a, b0, 1, 0, r) * kHD + 4 * lane);
    }
#pragma unroll
    for (int i = 0; i < kAheadParts; ++i)
      if (b0 + w0 + i * per < a.main_blocks)
        o_ahead[i] = *reinterpret_cast<const float4*>(a.part_o + part_row(a, b0, 0, w0 + i * per, r) * kHD + 4 * lane);
  }
  const BlockRec rec = a.recs[blockIdx.x];

  if (rec.parts > 0) {
    const int n = rec.parts;
    const int rows_here = min(a.rows - rec.join_blk * a.rows_tile, a.rows_tile);
    float M = -INFINITY, sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows_here) {
      if (w0 == 0 && rec.slot == 1) {
        if (lane == 0) ml0 = ml1;
        o_ahead[0] = o1;
      }
      for (int i0 = w0; i0 < n; i0 += 32 * per) {   // 32 parts at a time, one a lane
        const int mine = i0 + lane * per;
        float2 x = ml0;
        if (i0 != w0 && mine < n) x = a.part_ml[part_row(a, b0, rec.slot, mine, r)];
        if (mine >= n) x = make_float2(-INFINITY, 0.f);
        float nm = x.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) nm = fmaxf(nm, __shfl_xor_sync(0xffffffffu, nm, d));
        nm = fmaxf(nm, M);
        const float old = M == nm ? 1.f : ptx::ex2_approx(M - nm);   // 0 for the first
        const float f = x.x == -INFINITY ? 0.f : ptx::ex2_approx(x.x - nm);
        M = nm;
        float add = f * x.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) add += __shfl_xor_sync(0xffffffffu, add, d);
        sum = sum * old + add;
        acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
        const int count = min(32, (n - i0 + per - 1) / per);
        auto take = [&](int i, float4 y) {
          const float g = __shfl_sync(0xffffffffu, f, i);
          acc.x += y.x * g;
          acc.y += y.y * g;
          acc.z += y.z * g;
          acc.w += y.w * g;
        };
        int i1 = 0;
        if (i0 == w0) {
#pragma unroll
          for (int i = 0; i < kAheadParts; ++i)
            if (i < count) take(i, o_ahead[i]);
          i1 = min(count, kAheadParts);
        }
#pragma unroll 4
        for (int i = i1; i < count; ++i)
          take(i, *reinterpret_cast<const float4*>(a.part_o + part_row(a, b0, rec.slot, i0 + i * per, r) * kHD + 4 * lane));
      }
    }
    if (per > 1) {
      part[warp][lane] = acc;
      if (lane == 0) part_sum[warp] = make_float2(M, sum);
      __syncthreads();
      if (w0 == 0) {
        float top = M;
        for (int w = 1; w < per; ++w) top = fmaxf(top, part_sum[warp + w].x);
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        sum = 0.f;
        for (int w = 0; w < per; ++w) {
          const float2 s = part_sum[warp + w];
          const float f = s.x == -INFINITY ? 0.f : ptx::ex2_approx(s.x - top);
          const float4 y = part[warp + w][lane];
          sum += s.y * f;
          acc.x += y.x * f;
          acc.y += y.y * f;
          acc.z += y.z * f;
          acc.w += y.w * f;
        }
      }
    }
    if (r < rows_here && w0 == 0) {
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
      const int row = rec.join_blk * a.rows_tile + r, qi = int(fdiv(uint32_t(row), a.div_G));
      const int h = rec.join_g * a.G + row - qi * a.G;
      *reinterpret_cast<uint2*>(a.o + (int64_t(rec.join_s) * a.Lq + qi) * a.o_row + int64_t(h) * kRowBytes + lane * 8) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    }
  }

  if constexpr (kWeights) {
    // The steps of main block b once more, a step to a warp, of each item's
    // first row block only: p = exp2(score - maximum) / sum, added up over the
    // token's rows in their order, lane i taking tokens 2i and 2i + 1 (64 keys
    // a step; with fewer only the first lanes work).  Tokens that no query
    // sees are copied, shared out over the item's steps.
    if (rec.n == 0) return;
    const Split split(rec.total, a.div_blocks);
    Cursor cu;
    cu.s = rec.s;
    cu.g = rec.g;
    cu.blk = rec.blk;
    cu.c = rec.c;
    load_seq(a, cu);
    const int stride = int(gridDim.y) * (kJoinThreads / 32);
    int loaded_x0 = -1;
    // lane i: maximum and 1 / sum of rows i and 32 + i of the row block that begins at step loaded_x0
    float2 mrs[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    int skip = int(blockIdx.y) * (kJoinThreads / 32) + warp;
    for (int t = skip; t < rec.n; t += stride) {
      // forward to step t
      cu.c += skip;
      skip = stride;
      while (cu.c >= cu.nc) {
        cu.c -= cu.nc;
        if (++cu.blk < a.n_blk) continue;
        cu.blk = 0;
        if (++cu.g < a.c.H) continue;
        cu.g = 0;
        ++cu.s;
        load_seq(a, cu);
      }
      if (cu.blk != 0) continue;
      const int64_t out = (int64_t(cu.s) * a.c.H + cu.g) * a.c.capacity;
      const int x = cu.c * a.step_keys + 2 * lane;
      const bool live = 2 * lane < a.step_keys;
      float2 sum = make_float2(0.f, 0.f);
      // what is added to, and the first rows' scores, are under way before the
      // rows' maxima are known
      const int64_t at0 = out + token_of(cu.sp, x), at1 = out + token_of(cu.sp, x + 1);
      const bool on0 = live && x < cu.sp.span, on1 = live && x + 1 < cu.sp.span;
      float2 old = make_float2(0.f, 0.f);
      if (a.weight_in && on0) old.x = a.weight_in[at0];
      if (a.weight_in && on1) old.y = a.weight_in[at1];
      constexpr int kAhead = 4;
      float2 ahead[kAhead];
      const int rows_first = min(min(a.rows, a.rows_tile), kAhead);
#pragma unroll
      for (int r = 0; r < kAhead; ++r)
        if (live && r < rows_first)
          ahead[r] = *reinterpret_cast<const float2*>(a.scores + ((int64_t(rec.first) + t) * a.rows_blk + r) * a.step_keys +
                                                      2 * lane);
      for (int blk = 0; blk < a.n_blk; ++blk) {
        const int x0 = rec.first + t - cu.c + blk * cu.nc;   // the item's first step in the whole list
        const int rows_here = min(a.rows - blk * a.rows_tile, a.rows_tile);
        if (x0 != loaded_x0) {
          loaded_x0 = x0;
          const int b0 = split.block_of(x0), n = split.block_of(x0 + cu.nc - 1) - b0 + 1;
          const int slot = split.first(b0) == x0 ? 0 : 1;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int r = 32 * half + lane;
            mrs[half] = make_float2(0.f, 0.f);
            if (r < rows_here) {
              float M = -INFINITY, ls = 0.f;
              if (n == 1) {
                const float2 y = a.item_ml[(int64_t(cu.s) * a.c.H + cu.g) * a.n_blk * a.rows_blk +
                                           int64_t(blk) * a.rows_blk + r];
                M = y.x;
                ls = y.y;
              } else {
#pragma unroll 4
                for (int i = 0; i < n; ++i) {
                  const float2 y = a.part_ml[part_row(a, b0, slot, i, r)];
                  const float nm = fmaxf(M, y.x);
                  if (nm != -INFINITY) ls = ls * ptx::ex2_approx(M - nm) + y.y * ptx::ex2_approx(y.x - nm);
                  M = nm;
                }
              }
              if (ls > 0.f) mrs[half] = make_float2(M, 1.f / ls);
            }
          }
        }
        for (int r0 = 0; r0 < rows_here; r0 += 32) {
          const float2 mr = r0 == 0 ? mrs[0] : mrs[1];
          const float* sc = a.scores + ((int64_t(x0) + cu.c) * a.rows_blk + r0) * a.step_keys + 2 * lane;
          const int rows = min(rows_here - r0, 32);
          int r1 = 0;
          if (blk == 0 && r0 == 0) {
            r1 = rows_first;
#pragma unroll
            for (int r = 0; r < kAhead; ++r) {
              const float M = __shfl_sync(0xffffffffu, mr.x, r), inv = __shfl_sync(0xffffffffu, mr.y, r);
              if (live && r < rows_first) {
                sum.x += ptx::ex2_approx(ahead[r].x - M) * inv;
                sum.y += ptx::ex2_approx(ahead[r].y - M) * inv;
              }
            }
          }
#pragma unroll 4
          for (int r = r1; r < rows; ++r) {
            const float M = __shfl_sync(0xffffffffu, mr.x, r), inv = __shfl_sync(0xffffffffu, mr.y, r);
            if (live) {
              const float2 y = *reinterpret_cast<const float2*>(sc + int64_t(r) * a.step_keys);
              sum.x += ptx::ex2_approx(y.x - M) * inv;
              sum.y += ptx::ex2_approx(y.y - M) * inv;
            }
          }
        }
      }
      if (on0) a.weight_out[at0] = old.x + sum.x;
      if (on1) a.weight_out[at1] = old.y + sum.y;
      if (cu.sp.lo > cu.sp.se && a.weight_in != a.weight_out) {
        const int64_t gap = cu.sp.lo - cu.sp.se;
        const int64_t from = cu.sp.se + gap * cu.c / cu.nc, to = cu.sp.se + gap * (cu.c + 1) / cu.nc;
        for (int64_t j = from + lane; j < to; j += 32) a.weight_out[out + j] = a.weight_in ? a.weight_in[out + j] : 0.f;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct DecodeShape {
  int64_t rows, rows_tile, rows_blk, n_blk, items, steps, blocks;
  int64_t step_keys;
  size_t part_o, part_ml, recs, item_ml, scores, bytes;   // offsets into the workspace, and its size
};

static rkv_status decode_shape(const rkv_paged_cache* c, int32_t Hq, int32_t Lq, bool weights, DecodeShape& d) {
  if (Hq < 1 || Hq % c->H) return fail(RKV_ERR_INVALID_ARG, "Hq %d must be a multiple of the cache's H %d", Hq, c->H);
  if (Lq < 1 || Lq > RKV_DECODE_MAX_LQ)
    return fail(RKV_ERR_INVALID_ARG, "Lq %d must be in [1, %d]", Lq, RKV_DECODE_MAX_LQ);
  d.rows = int64_t(Lq) * (Hq / c->H);
  if (d.rows > kMaxRows) return fail(RKV_ERR_UNSUPPORTED, "more than %d query rows to a key head", kMaxRows);
  // A row block is as many 16-row tiles as the rows need, up to the four that a
  // block's warps can take: K and V are read once for all of them.  16 streams
  // of 8,000 tokens, 4 key heads: 16 rows 55 us, 32 rows 61 (in two blocks of
  // 16 rows 94), 64 rows 93, 128 rows 155
  d.rows_tile = d.rows <= 16 ? 16 : (d.rows <= 32 ? 32 : 64);
  d.step_keys = d.rows_tile == 16   ? DecSmem<1>::kStepKeys
                : d.rows_tile == 32 ? DecSmem<2>::kStepKeys
                                    : DecSmem<4>::kStepKeys;
  d.rows_blk = std::min(d.rows, d.rows_tile);
  d.n_blk = (d.rows + d.rows_tile - 1) / d.rows_tile;
  d.items = int64_t(c->n_seqs) * c->H * d.n_blk;
  d.steps = d.items * ((capacity(c) + d.step_keys - 1) / d.step_keys);
  // step counts are 32-bit, and so is Lq * Hq * 16 in the zero fill
  if (d.steps >= (int64_t(1) << 30) || int64_t(c->n_seqs) * Lq >= (int64_t(1) << 31) || int64_t(Hq) * Lq >= (1 << 26))
    return fail(RKV_ERR_UNSUPPORTED, "too many sequences, heads and tokens for one launch");
  d.blocks = std::min<int64_t>(kDecPerSm * sm_count(), std::max<int64_t>(d.steps, 1));
  auto up = [](size_t x) { return (x + 15) / 16 * 16; };
  d.part_o = 0;
  d.part_ml = d.part_o + up(size_t(d.blocks * 2 * d.rows_blk) * kHD * 4);
  d.recs = d.part_ml + up(size_t(d.blocks * 2 * d.rows_blk) * 8);
  d.item_ml = d.recs + size_t(d.blocks) * sizeof(BlockRec);
  d.scores = d.item_ml + (weights ? up(size_t(d.items * d.rows_blk) * 8) : 0);
  d.bytes = d.scores + (weights ? size_t(d.steps * d.rows_blk * d.step_keys) * 4 : 0);
  return RKV_OK;
}

template <int NR, bool kWeights>
static rkv_status launch_decode(const DecodeArgs& a, cudaStream_t cs) {
  constexpr int smem = DecSmem<NR>::kBytes;
  cudaError_t e = allow_smem<decode_paged_kernel<NR, kWeights>>(smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(decode_paged_kernel)");
  e = launch_overlapped(decode_paged_kernel<NR, kWeights>, dim3(uint32_t(a.main_blocks)), kDecThreads, smem, cs, a);
  if (e != cudaSuccess) return cuda_fail(e, "decode_paged_kernel launch");
  // a block per main block and eight rows of a row block (its warps: see the
  // kernel); the weights pass shares a main block's steps out over them
  const int rows = a.rows_blk <= 4 ? 1 : (a.rows_blk + 7) / 8;
  const dim3 grid(uint32_t(a.main_blocks), uint32_t(kWeights ? std::max(rows, 2) : rows));
  e = launch_overlapped(decode_join_kernel<kWeights>, grid, kJoinThreads, 0, cs, a);
  if (e != cudaSuccess) return cuda_fail(e, "decode_join_kernel launch");
  return RKV_OK;
}

}  // namespace paged
}  // namespace rkv

using namespace rkv;
using namespace rkv::paged;

extern "C" size_t attn_decode_paged_workspace_size(const rkv_paged_cache* cache, int32_t Hq, int32_t Lq,
                                                   int32_t weights) {
  DecodeShape d;
  if (check_cache(cache) != RKV_OK || decode_shape(cache, Hq, Lq, weights != 0, d) != RKV_OK) {
    clear_error();
    return 0;
  }
  return d.bytes;
}

extern "C" rkv_status attn_decode_paged(const rkv_paged_cache* cache, const void* q, void* o, int64_t q_row_stride,
                                        int64_t o_row_stride, int32_t Hq, int32_t Lq, const int32_t* seq_lens,
                                        float softmax_scale, int32_t window, int32_t sinks, const float* weight_in,
                                        float* weight_out, void* workspace, size_t workspace_bytes, void* stream) {
  NvtxRange nvtx_range("attn_decode_paged");
  clear_error();
  rkv_status st = check_cache(cache);
  if (st != RKV_OK) return st;
  DecodeShape d;
  st = decode_shape(cache, Hq, Lq, weight_out != nullptr, d);
  if (st != RKV_OK) return st;
  if (!q || !o || !seq_lens) return fail(RKV_ERR_INVALID_ARG, "q/o/seq_lens is NULL");
  if (!aligned16(q) || !aligned16(o)) return fail(RKV_ERR_INVALID_ARG, "q/o must be 16-byte aligned");
  if (!aligned4(seq_lens) || !aligned4(weight_in) || !aligned4(weight_out))
    return fail(RKV_ERR_INVALID_ARG, "seq_lens/weight_in/weight_out must be 4-byte aligned");
  const int64_t row = int64_t(Hq) * kHD, n_rows = int64_t(cache->n_seqs) * Lq;
  for (int64_t stride : {q_row_stride, o_row_stride}) {
    if (stride < row) return fail(RKV_ERR_INVALID_ARG, "row stride < Hq*D");
    if (stride % 8) return fail(RKV_ERR_INVALID_ARG, "rows of q/o must be 16-byte aligned");
    if (stride >= (int64_t(1) << 40) || stride >= kMaxSpan / n_rows)
      return fail(RKV_ERR_INVALID_ARG, "row stride too large");
  }
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return fail(RKV_ERR_INVALID_ARG, "softmax_scale must be > 0");
  if (window < 0 || sinks < 0) return fail(RKV_ERR_INVALID_ARG, "window and sinks must be >= 0");
  if (weight_in && !weight_out) return fail(RKV_ERR_INVALID_ARG, "weight_in without weight_out");
  const uint64_t sb = uint64_t(cache->n_seqs) * cache->H * capacity(cache) * 4;
  if (weight_in && weight_in != weight_out && overlaps(weight_in, sb, weight_out, sb))
    return fail(RKV_ERR_INVALID_ARG, "weight_in and weight_out overlap in part");
  st = check_apart({{"o", o, n_rows, o_row_stride * 2, row * 2}, run_of("weight_out", weight_out, sb),
                    run_of("the workspace", workspace, std::min(d.bytes, workspace_bytes)), status_of(cache)},
                   {{"q", q, n_rows, q_row_stride * 2, row * 2}, pool_k(cache), pool_v(cache), table_of(cache),
                    run_of("seq_lens", seq_lens, uint64_t(cache->n_seqs) * 4),
                    run_of("weight_in", weight_in == weight_out ? nullptr : weight_in, sb)});
  if (st != RKV_OK) return st;
  if (!workspace || !aligned16(workspace) || workspace_bytes < d.bytes)
    return fail(RKV_ERR_INVALID_ARG, "workspace must be >= %zu bytes and 16-byte aligned", d.bytes);
  DecodeArgs a;
  a.c = cache_dev(cache);
  a.q = static_cast<const uint8_t*>(q);
  a.o = static_cast<uint8_t*>(o);
  a.q_row = q_row_stride * 2;
  a.o_row = o_row_stride * 2;
  a.seq_lens = seq_lens;
  a.weight_in = weight_in;
  a.weight_out = weight_out;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + d.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + d.part_ml);
  a.recs = reinterpret_cast<BlockRec*>(ws + d.recs);
  a.item_ml = reinterpret_cast<float2*>(ws + d.item_ml);
  a.scores = reinterpret_cast<float*>(ws + d.scores);
  a.scale_log2 = float(double(softmax_scale) * 1.4426950408889634);
  a.Hq = Hq;
  a.Lq = Lq;
  a.G = Hq / cache->H;
  a.div_G = make_fastdiv(uint32_t(a.G));
  a.rows = int32_t(d.rows);
  a.rows_tile = int32_t(d.rows_tile);
  a.step_keys = int32_t(d.step_keys);
  a.rows_blk = int32_t(d.rows_blk);
  a.n_blk = int32_t(d.n_blk);
  a.window = std::min(window, 1 << 30);   // more than any capacity: all tokens
  a.sinks = sinks;
  a.main_blocks = int32_t(d.blocks);
  a.div_blocks = make_fastdiv(uint32_t(d.blocks));
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (weight_out) {
    return d.rows_tile == 16   ? launch_decode<1, true>(a, cs)
           : d.rows_tile == 32 ? launch_decode<2, true>(a, cs)
                               : launch_decode<4, true>(a, cs);
  }
  return d.rows_tile == 16   ? launch_decode<1, false>(a, cs)
         : d.rows_tile == 32 ? launch_decode<2, false>(a, cs)
                             : launch_decode<4, false>(a, cs);
}
