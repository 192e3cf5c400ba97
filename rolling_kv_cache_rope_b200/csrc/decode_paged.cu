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
// HBM.  A tcgen05 tile has at least 64 query rows, most of them empty here, and
// needs its operands in whole swizzled tiles where pages end anywhere; the
// warp-level m16n8k16 product takes 16 rows and is far from its own limit at
// this bandwidth (16 keys of a head cost 32 of them per 8 KB).
//
// Split: the key rows of all (sequence, key head, row block) items, in steps
// of 128 keys, form one list of T steps, and block b of C takes the steps
// [b T / C, (b + 1) T / C): every block gets the same bytes whatever the
// lengths.  An item that lies in one block is finished there; of the others
// each block leaves its running maximum, sum and unnormalised O (at most two
// per block), and a second launch joins them in the order of the keys, so the
// result does not depend on timing.  Each kernel derives the list from
// seq_lens itself: nothing is planned on the host, and a captured launch
// serves growing sequences.
//
// Inside a block: eight warps, each with 16 of a step's 128 keys and its own
// maximum, sum and O in registers, meet only where an item begins or ends.
// Each warp copies its own K and V rows with 16-byte asynchronous copies into
// its part of a ring of stages, so several steps (64 KB each) are in flight
// per SM without registers holding data, across the ends of items too.  A row
// that is not visible to any query (past the end, outside window and sinks, on
// a bad page) is not read but zero-filled, so nothing it holds can enter a sum.
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "sm100_ptx.cuh"

namespace rkv {
namespace paged {

constexpr int kDecThreads = 256;
constexpr int kDecWarps = kDecThreads / 32;
constexpr int kTileKeys = 16;                          // keys of a step one warp takes
constexpr int kStepKeys = kDecWarps * kTileKeys;       // 128
constexpr int kTileBytes = kTileKeys * int(kRowBytes); // 4 KB of K, as much of V
constexpr int kStepBytes = kDecWarps * 2 * kTileBytes; // 64 KB
constexpr float kMaxSlack = 8.0f;                      // the running maximum moves past 2^8 growth only
constexpr int kMaxRows = 4096;                         // query rows of a key head (Lq * G)
constexpr int kJoinThreads = 256;
constexpr int kWeightTokens = kJoinThreads;            // tokens of a step of the weights pass

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
  float* scores;                 // [T][rows_blk][kStepKeys] scaled scores, log2 units (weights only)
  float scale_log2;
  int32_t Hq, Lq, G, rows;       // rows = Lq * G
  int32_t rows_tile;             // rows a row block has room for (16 or 32)
  int32_t rows_blk, n_blk;       // rows of a full row block (min(rows, rows_tile)), row blocks
  int32_t window, sinks;
  int32_t main_blocks;           // C
};

// The keys any query of a sequence of length L sees, as a list of `span`
// entries: [0, se), then [lo, L).
struct Span {
  int L, se, lo, span;
  __device__ __forceinline__ int steps() const { return (span + kStepKeys - 1) / kStepKeys; }
};

__device__ __forceinline__ Span span_of(const DecodeArgs& a, int L) {
  Span r;
  r.L = L;
  r.lo = a.window > 0 ? max(0, max(0, L - a.Lq) - a.window + 1) : 0;   // of the first query there is
  r.se = min(a.sinks, r.lo);
  r.span = L > 0 ? r.se + L - r.lo : 0;
  return r;
}

// Steps of a sequence in the list of visible keys (main launch), per item.
struct MainSteps {
  __device__ __forceinline__ static int of(const DecodeArgs& a, int s) {
    return span_of(a, seq_len(a.c, a.seq_lens, s)).steps();
  }
};
// Steps of a sequence's tokens, visible or not, in the weights pass, per key head.
struct TokenSteps {
  __device__ __forceinline__ static int of(const DecodeArgs& a, int s) {
    return (seq_len(a.c, a.seq_lens, s) + kWeightTokens - 1) / kWeightTokens;
  }
};

// Steps of the whole list: `items` times each sequence's.  Whole warps call
// these two; every lane gets the result.
template <class Steps>
__device__ __forceinline__ int total_steps(const DecodeArgs& a, int items) {
  int total = 0;
  for (int s = threadIdx.x & 31; s < a.c.n_seqs; s += 32) total += Steps::of(a, s);
  return __reduce_add_sync(0xffffffffu, total) * items;
}

// The sequence that step x of the list falls into and the steps before it.
struct Place {
  int s, base;
};

template <class Steps>
__device__ __forceinline__ Place find_step(const DecodeArgs& a, int items, int x) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int b = 0; b < a.c.n_seqs; b += 32) {
    const int s = b + lane;
    const int own = s < a.c.n_seqs ? Steps::of(a, s) * items : 0;
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

// Blocks that take part (each with at least one step), the first step of one,
// and the block whose range holds step x.
__device__ __forceinline__ int blocks_used(const DecodeArgs& a, int total) { return min(a.main_blocks, total); }
__device__ __forceinline__ int block_first(int total, int b, int blocks) {
  return int(int64_t(total) * b / blocks);
}
// the block whose range holds step x
__device__ __forceinline__ int block_of(int total, int x, int blocks) {
  return int((int64_t(x + 1) * blocks - 1) / total);
}

// A position in the list of steps: sequence, item of the sequence (key head
// major, row block minor), step of the item.
struct Cursor {
  Span sp;
  int s, it, c, nc;
};

__device__ __forceinline__ void load_seq(const DecodeArgs& a, Cursor& u) {
  while (true) {   // sequences without a visible key have no steps
    u.sp = span_of(a, seq_len(a.c, a.seq_lens, u.s));
    u.nc = u.sp.steps();
    if (u.nc > 0 || u.s + 1 >= a.c.n_seqs) return;
    ++u.s;
  }
}

__device__ __forceinline__ void advance(const DecodeArgs& a, Cursor& u) {
  if (++u.c < u.nc) return;
  u.c = 0;
  if (++u.it < a.c.H * a.n_blk) return;
  u.it = 0;
  if (u.s + 1 >= a.c.n_seqs) return;   // past the last step: not used
  ++u.s;
  load_seq(a, u);
}

// Entry x of a sequence's visible list -> its token.
__device__ __forceinline__ int token_of(const Span& sp, int x) { return x < sp.se ? x : x - sp.se + sp.lo; }

template <int MT, int kStages>
struct DecSmem {
  static constexpr int kQBytes = MT * 16 * int(kRowBytes);
  // merge buffer: per warp 640 floats a 16-row tile (16 rows of 32 columns
  // padded to 40, or 8 of 64 to 72, or 4 of 128 to 136)
  static constexpr int kMergeFloats = MT * 640;
  static constexpr int kOffQ = kStages * kStepBytes;
  static constexpr int kOffMerge = kOffQ + kStages * kQBytes;
  static constexpr int kOffMl = kOffMerge + kDecWarps * kMergeFloats * 4;
  static constexpr int kOffMask = kOffMl + kDecWarps * MT * 16 * 8;
  static constexpr int kBytes = kOffMask + kStages * kDecWarps * 4;
  static_assert(kBytes <= 232448, "shared memory of one block");
};

template <int MT, int kStages, bool kWeights>
__global__ void __launch_bounds__(kDecThreads, 1) decode_paged_kernel(const __grid_constant__ DecodeArgs a) {
  using SM = DecSmem<MT, kStages>;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per_step = a.c.H * a.n_blk;
  ptx::pdl_launch_dependents();

  const int total = total_steps<MainSteps>(a, per_step);
  const int blocks = blocks_used(a, total);

  if (int(blockIdx.x) < blocks) {
    const int c0 = block_first(total, blockIdx.x, blocks);
    const int n_steps = block_first(total, blockIdx.x + 1, blocks) - c0;   // >= 1
    const Place pl = find_step<MainSteps>(a, per_step, c0);
    Cursor cu;   // the step computed next
    cu.s = pl.s;
    load_seq(a, cu);
    cu.it = (c0 - pl.base) / cu.nc;
    cu.c = (c0 - pl.base) - cu.it * cu.nc;
    Cursor is = cu;   // the step copied next
    int issued = 0;
    uint32_t q_slot_is = 0, q_slot = 0;   // Q ring position of the issued / computed item
    float* merge = reinterpret_cast<float*>(smem + SM::kOffMerge);
    float2* ml = reinterpret_cast<float2*>(smem + SM::kOffMl);
    uint32_t* vmask = reinterpret_cast<uint32_t*>(smem + SM::kOffMask);

    // Copy this warp's 16 keys of step `is` into stage issued % kStages, and,
    // where an item begins, its Q rows (all threads together).
    auto issue = [&]() {
      if (issued < n_steps) {
        const uint32_t st = uint32_t(issued) % kStages;
        const int g = is.it / a.n_blk;
        const int x0 = is.c * kStepKeys + warp * kTileKeys, x = x0 + (lane & 15);
        bool ok = x < is.sp.span;
        uint32_t unit = 0;
        if (ok) {
          const uint32_t j = uint32_t(token_of(is.sp, x));
          const uint32_t page = page_of(a.c, is.s, j);
          ok = page < a.c.n_pages;
          if (ok) unit = row_unit(a.c, page, j, g);
          else record(a.c, kBadPage);
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, ok) & 0xFFFFu;
        if (lane == 0) vmask[st * kDecWarps + warp] = mask;
        const uint32_t dst = sbase + st * kStepBytes + uint32_t(warp) * (2 * kTileBytes);
        const uint32_t piece = uint32_t(lane) & 15u;
        if (x0 < is.sp.span) {   // a tile past the list's end is not computed either
#pragma unroll
          for (int i = 0; i < kTileKeys / 2; ++i) {
            const int kk = 2 * i + (lane >> 4);
            const uint32_t un = __shfl_sync(0xffffffffu, unit, kk);
            const uint32_t bytes = (mask >> kk) & 1u ? 16u : 0u;
            const uint64_t off = uint64_t(un) * kRowBytes + piece * 16u;
            const uint32_t d = dst + uint32_t(kk) * kRowBytes + ((piece ^ (uint32_t(kk) & 7u)) << 4);
            ptx::cp_async16(d, a.c.k + off, bytes);
            ptx::cp_async16(d + kTileBytes, a.c.v + off, bytes);
          }
        }
        if (issued == 0 || is.c == 0) {
          if (issued > 0) q_slot_is = (q_slot_is + 1) % kStages;
          const int blk = is.it - g * a.n_blk;
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            const int r = i * 16 + (tid >> 4);
            const int row = blk * (MT * 16) + r;
            const bool there = row < a.rows;
            const int qi = there ? row / a.G : 0;
            const int h = there ? g * a.G + row - qi * a.G : 0;
            const uint32_t pc = uint32_t(tid) & 15u;
            ptx::cp_async16(sbase + SM::kOffQ + q_slot_is * SM::kQBytes + uint32_t(r) * kRowBytes +
                                ((pc ^ (uint32_t(r) & 7u)) << 4),
                            a.q + (int64_t(is.s) * a.Lq + qi) * a.q_row + int64_t(h) * kRowBytes + pc * 16u,
                            there ? 16u : 0u);
          }
        }
        ++issued;
        if (issued < n_steps) advance(a, is);
      }
      ptx::cp_async_commit();
    };

    // Q as A operands: in registers where one row tile leaves room, else read
    // from shared memory in every step
    constexpr bool kQRegs = MT == 1;
    uint32_t qf[kQRegs ? MT : 1][8][4];
    auto load_q = [&](uint32_t qb, int i, int kk, uint32_t (&r4)[4]) {
      // matrices of an A tile: rows 0-7 / 8-15, then the next 8 columns
      const uint32_t r = uint32_t(i * 16 + (lane & 15)), pc = uint32_t(2 * kk + (lane >> 4));
      ptx::ldsm4(qb + r * kRowBytes + ((pc ^ (r & 7u)) << 4), r4);
    };
    float O[MT][16][4];
    float m[MT][2], l[MT][2];
    int row_hi[MT][2], row_lo[MT][2];   // this lane's rows (g, g + 8 of each tile): keys < hi, >= lo or a sink
    int all_lo = 0, all_hi = 0;         // keys in [all_lo, all_hi) are visible to every row
    int frag_c0 = 0, frag_t0 = 0;       // step of the item, and of the block, this part of the item began at
    bool first = true;

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    for (int t = 0; t < n_steps; ++t) {
      issue();
      ptx::cp_async_wait<kStages - 1>();
      __syncwarp();
      const int g = cu.it / a.n_blk, blk = cu.it - g * a.n_blk;
      const uint32_t qb = sbase + SM::kOffQ + q_slot * SM::kQBytes;
      if (first) {
        __syncthreads();   // every warp's share of the item's Q rows has landed
        first = false;
        frag_c0 = cu.c;
        frag_t0 = t;
        const int last_q = min(a.rows, (blk + 1) * (MT * 16)) - 1, first_q = blk * (MT * 16);
        const int c_first = cu.sp.L - a.Lq + first_q / a.G, c_last = cu.sp.L - a.Lq + last_q / a.G;
        all_hi = max(0, c_first + 1);
        all_lo = a.window > 0 ? max(0, c_last - a.window + 1) : 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          if constexpr (kQRegs) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) load_q(qb, i, kk, qf[i][kk]);
          }
#pragma unroll
          for (int n = 0; n < 16; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) O[i][n][e] = 0.f;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            m[i][e] = -INFINITY;
            l[i][e] = 0.f;
            const int row = blk * (MT * 16) + i * 16 + e * 8 + (lane >> 2);
            const int c = cu.sp.L - a.Lq + row / a.G;
            row_hi[i][e] = row < a.rows ? max(0, c + 1) : 0;
            row_lo[i][e] = a.window > 0 ? max(0, c - a.window + 1) : 0;
          }
        }
      }

      const uint32_t st = uint32_t(t) % kStages;
      const int x0 = cu.c * kStepKeys + warp * kTileKeys;
      if (x0 < cu.sp.span) {
        const uint32_t mask = vmask[st * kDecWarps + warp];
        const uint32_t sk = sbase + st * kStepBytes + uint32_t(warp) * (2 * kTileBytes), sv = sk + kTileBytes;
        // S = Q K^T: two chains of four products per 8-key tile and row tile
        float S[MT][2][4], S2[MT][2][4];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i][n][e] = S2[i][n][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          // matrices: keys 0-7 of columns 16kk.. and 16kk + 8.., then keys 8-15
          uint32_t b[4];
          const uint32_t r = uint32_t((lane & 7) + ((lane >> 4) << 3)), pc = uint32_t(2 * kk + ((lane >> 3) & 1));
          ptx::ldsm4(sk + r * kRowBytes + ((pc ^ (r & 7u)) << 4), b);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            uint32_t qa[4];
            if constexpr (kQRegs) {
#pragma unroll
              for (int e = 0; e < 4; ++e) qa[e] = qf[i][kk][e];
            } else {
              load_q(qb, i, kk, qa);
            }
            ptx::mma_bf16(kk & 1 ? S2[i][0] : S[i][0], qa, b[0], b[1]);
            ptx::mma_bf16(kk & 1 ? S2[i][1] : S[i][1], qa, b[2], b[3]);
          }
        }
        // the tile holds tokens j0 .. j0 + 15 unless the list jumps from the
        // sinks to the window inside it; no mask is needed where every row sees all
        const int j0 = token_of(cu.sp, x0);
        const bool plain = mask == 0xFFFFu && (x0 >= cu.sp.se || x0 + kTileKeys <= cu.sp.se) &&
                           j0 + kTileKeys <= all_hi && (j0 >= all_lo || j0 + kTileKeys <= a.sinks);
        uint32_t P[MT][4];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i][n][e] = (S[i][n][e] + S2[i][n][e]) * a.scale_log2;
          if (!plain) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int kk = n * 8 + 2 * (lane & 3) + (e & 1);
                const int j = token_of(cu.sp, x0 + kk);
                const bool vis = ((mask >> kk) & 1u) && j < row_hi[i][e >> 1] &&
                                 (j >= row_lo[i][e >> 1] || j < a.sinks);
                if (!vis) S[i][n][e] = -INFINITY;
              }
          }
          if constexpr (kWeights) {
            const int64_t step = int64_t(c0) + t;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = i * 16 + e * 8 + (lane >> 2);
              if (r < a.rows_blk) {
                float* dst = a.scores + (step * a.rows_blk + r) * kStepKeys + warp * kTileKeys + 2 * (lane & 3);
                *reinterpret_cast<float2*>(dst) = make_float2(S[i][0][2 * e], S[i][0][2 * e + 1]);
                *reinterpret_cast<float2*>(dst + 8) = make_float2(S[i][1][2 * e], S[i][1][2 * e + 1]);
              }
            }
          }
          float mx[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            mx[e] = fmaxf(fmaxf(S[i][0][2 * e], S[i][0][2 * e + 1]), fmaxf(S[i][1][2 * e], S[i][1][2 * e + 1]));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
            mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
          }
          const bool move = mx[0] > m[i][0] + kMaxSlack || mx[1] > m[i][1] + kMaxSlack;
          if (__any_sync(0xffffffffu, move)) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float nm = mx[e] > m[i][e] + kMaxSlack ? mx[e] : m[i][e];
              f[e] = m[i][e] == nm ? 1.f : ptx::ex2_approx(m[i][e] - nm);
              m[i][e] = nm;
              l[i][e] *= f[e];
            }
#pragma unroll
            for (int n = 0; n < 16; ++n) {
              O[i][n][0] *= f[0];
              O[i][n][1] *= f[0];
              O[i][n][2] *= f[1];
              O[i][n][3] *= f[1];
            }
          }
          // P = exp2(S - m): summed in fp32, rounded to bf16 for P V (at most
          // half a step of bf16, 2^-8 of each weight, as the output's own
          // rounding).  S's accumulator layout is the A operand's as it stands.
          const float u0 = m[i][0] == -INFINITY ? 0.f : m[i][0], u1 = m[i][1] == -INFINITY ? 0.f : m[i][1];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float p0 = ptx::ex2_approx(S[i][n][0] - u0), p1 = ptx::ex2_approx(S[i][n][1] - u0);
            const float p2 = ptx::ex2_approx(S[i][n][2] - u1), p3 = ptx::ex2_approx(S[i][n][3] - u1);
            l[i][0] += p0 + p1;
            l[i][1] += p2 + p3;
            P[i][2 * n] = pack_bf16x2(p0, p1);
            P[i][2 * n + 1] = pack_bf16x2(p2, p3);
          }
        }
        // O += P V
#pragma unroll
        for (int np = 0; np < 8; ++np) {
          // matrices: keys 0-7 / 8-15 of columns 16np.., then of 16np + 8..
          uint32_t b[4];
          const uint32_t r = uint32_t(lane & 15), pc = uint32_t(2 * np + (lane >> 4));
          ptx::ldsm4_trans(sv + r * kRowBytes + ((pc ^ (r & 7u)) << 4), b);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            ptx::mma_bf16(O[i][2 * np], P[i], b[0], b[1]);
            ptx::mma_bf16(O[i][2 * np + 1], P[i], b[2], b[3]);
          }
        }
      }
      __syncwarp();   // the warp is done with the stage issue() fills next

      if (cu.c + 1 == cu.nc || t + 1 == n_steps) {
        // ---- the item ends here, in this block: join the warps' parts ----
        const bool whole = frag_c0 == 0 && cu.c + 1 == cu.nc;
        const int rows_here = min(a.rows - blk * (MT * 16), MT * 16);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 1);
            l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], 2);
            if ((lane & 3) == 0) ml[warp * (MT * 16) + i * 16 + e * 8 + (lane >> 2)] = make_float2(m[i][e], l[i][e]);
          }
        __syncthreads();
        auto joined = [&](int r, float& M, float& sum) {
          M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) M = fmaxf(M, ml[w * (MT * 16) + r].x);
          sum = 0.f;
#pragma unroll
          for (int w = 0; w < kDecWarps; ++w) {
            const float2 x = ml[w * (MT * 16) + r];
            sum += x.x == -INFINITY ? 0.f : x.y * ptx::ex2_approx(x.x - M);
          }
        };
        float f[MT][2];
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float M, sum;
            joined(i * 16 + e * 8 + (lane >> 2), M, sum);
            f[i][e] = m[i][e] == -INFINITY ? 0.f : ptx::ex2_approx(m[i][e] - M);
          }
        const int64_t slot = (int64_t(blockIdx.x) * 2 + (frag_t0 == 0 ? 0 : 1)) * a.rows_blk;
        if (tid < rows_here && (!whole || kWeights)) {
          float M, sum;
          joined(tid, M, sum);
          if (!whole)
            a.part_ml[slot + tid] = make_float2(M, sum);
          else
            a.item_ml[(int64_t(cu.s) * per_step + cu.it) * a.rows_blk + tid] = make_float2(M, sum);
        }
        const int cw = rows_here <= 4 ? 128 : (rows_here <= 8 ? 64 : 32), pad = cw + 8;
        for (int cb = 0; cb < kHD; cb += cw) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = i * 16 + e * 8 + (lane >> 2);
              if (r < rows_here) {
                float* dst = merge + warp * SM::kMergeFloats + r * pad + 2 * (lane & 3) - cb;
#pragma unroll
                for (int n = 0; n < 16; ++n)
                  if (n * 8 >= cb && n * 8 < cb + cw)
                    *reinterpret_cast<float2*>(dst + n * 8) =
                        make_float2(O[i][n][2 * e] * f[i][e], O[i][n][2 * e + 1] * f[i][e]);
              }
            }
          __syncthreads();
          for (int idx = tid; idx < rows_here * (cw / 2); idx += kDecThreads) {
            const int r = idx / (cw / 2), col = 2 * (idx - r * (cw / 2));
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kDecWarps; ++w) {
              const float2 x = *reinterpret_cast<const float2*>(merge + w * SM::kMergeFloats + r * pad + col);
              sum.x += x.x;
              sum.y += x.y;
            }
            if (whole) {
              float M, ls;
              joined(r, M, ls);
              const float inv = ls > 0.f ? 1.f / ls : 0.f;
              const int row = blk * (MT * 16) + r, qi = row / a.G, h = g * a.G + row - qi * a.G;
              *reinterpret_cast<uint32_t*>(a.o + (int64_t(cu.s) * a.Lq + qi) * a.o_row + int64_t(h) * kRowBytes +
                                           (cb + col) * 2) = pack_bf16x2(sum.x * inv, sum.y * inv);
            } else {
              *reinterpret_cast<float2*>(a.part_o + (slot + r) * kHD + cb + col) = sum;
            }
          }
          __syncthreads();
        }
        first = true;
        q_slot = (q_slot + 1) % kStages;
      }
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

// The parts of the item with steps [x0, x1): blocks b0 .. b1 of the main
// launch, the first one's part in slot `first`, the others' in slot 2 b.
struct Parts {
  int b0, b1;
  int64_t first;
};
__device__ __forceinline__ Parts parts_of(int total, int blocks, int x0, int x1) {
  Parts p;
  p.b0 = block_of(total, x0, blocks);
  p.b1 = block_of(total, x1 - 1, blocks);
  p.first = int64_t(p.b0) * 2 + (block_first(total, p.b0, blocks) == x0 ? 0 : 1);
  return p;
}
__device__ __forceinline__ int64_t part_row(const DecodeArgs& a, const Parts& p, int b, int r) {
  return (b == p.b0 ? p.first : int64_t(b) * 2) * a.rows_blk + r;
}

// Running maximum and sum of row r of an item over its parts.
__device__ __forceinline__ void join_ml(const DecodeArgs& a, const Parts& p, int r, float& M, float& sum) {
  M = -INFINITY;
  sum = 0.f;
  for (int b = p.b0; b <= p.b1; ++b) M = fmaxf(M, a.part_ml[part_row(a, p, b, r)].x);
  for (int b = p.b0; b <= p.b1; ++b) {
    const float2 x = a.part_ml[part_row(a, p, b, r)];
    sum += x.x == -INFINITY ? 0.f : x.y * ptx::ex2_approx(x.x - M);
  }
}

template <bool kWeights>
__global__ void __launch_bounds__(kJoinThreads) decode_join_kernel(const __grid_constant__ DecodeArgs a) {
  extern __shared__ float2 row_ml[];   // weights: maximum and 1 / sum of the rows of the step's key head
  const int tid = threadIdx.x;
  const int per_step = a.c.H * a.n_blk;
  const int total = total_steps<MainSteps>(a, per_step);
  const int blocks = blocks_used(a, total);

  Place pl = {0, 0};
  int c0 = 0, c1 = 0;
  if (int(blockIdx.x) < blocks) {
    c0 = block_first(total, blockIdx.x, blocks);
    c1 = block_first(total, blockIdx.x + 1, blocks);
    pl = find_step<MainSteps>(a, per_step, c1 - 1);
  }
  ptx::pdl_wait();   // the main launch's parts are written
  if (int(blockIdx.x) < blocks) {
    // the item this block's last step lies in, where it began here and goes on
    const int nc = MainSteps::of(a, pl.s);
    const int it = (c1 - 1 - pl.base) / nc, x0 = pl.base + it * nc, x1 = x0 + nc;
    if (x1 > c1 && x0 >= c0) {
      const Parts p = parts_of(total, blocks, x0, x1);
      const int g = it / a.n_blk, blk = it - g * a.n_blk;
      const int rows_here = min(a.rows - blk * a.rows_tile, a.rows_tile);
      for (int idx = tid; idx < rows_here * (kHD / 4); idx += kJoinThreads) {
        const int r = idx / (kHD / 4), col = 4 * (idx - r * (kHD / 4));
        float M, ls;
        join_ml(a, p, r, M, ls);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int b = p.b0; b <= p.b1; ++b) {
          const int64_t at = part_row(a, p, b, r);
          const float mb = a.part_ml[at].x;
          const float f = mb == -INFINITY ? 0.f : ptx::ex2_approx(mb - M);
          const float4 x = *reinterpret_cast<const float4*>(a.part_o + at * kHD + col);
          sum.x += x.x * f;
          sum.y += x.y * f;
          sum.z += x.z * f;
          sum.w += x.w * f;
        }
        const float inv = ls > 0.f ? 1.f / ls : 0.f;
        const int row = blk * a.rows_tile + r, qi = row / a.G, h = g * a.G + row - qi * a.G;
        *reinterpret_cast<uint2*>(a.o + (int64_t(pl.s) * a.Lq + qi) * a.o_row + int64_t(h) * kRowBytes + col * 2) =
            make_uint2(pack_bf16x2(sum.x * inv, sum.y * inv), pack_bf16x2(sum.z * inv, sum.w * inv));
      }
    }
  }

  if constexpr (kWeights) {
    // p = exp2(score - maximum) / sum, added up over a token's rows in their
    // order; one thread a token, the scores of 128 tokens of a row side by side
    const int all = total_steps<TokenSteps>(a, a.c.H);
    const int w0 = block_first(all, blockIdx.x, gridDim.x), w1 = block_first(all, blockIdx.x + 1, gridDim.x);
    if (w0 == w1) return;
    Place wp = find_step<TokenSteps>(a, a.c.H, w0);
    int s = wp.s, at = w0 - wp.base;   // step of the sequence
    int main_base = 0;                 // main steps before sequence s
    for (int i = tid & 31; i < s; i += 32) main_base += MainSteps::of(a, i) * per_step;
    main_base = __reduce_add_sync(0xffffffffu, main_base);
    int loaded = -1;
    for (int w = w0; w < w1; ++w, ++at) {
      int ns = TokenSteps::of(a, s);
      while (at >= ns * a.c.H) {
        at -= ns * a.c.H;
        main_base += MainSteps::of(a, s) * per_step;
        ns = TokenSteps::of(a, ++s);
        loaded = -1;
      }
      const Span sp = span_of(a, seq_len(a.c, a.seq_lens, s));
      const int nc = sp.steps();
      const int h = at / ns;
      if (h != loaded) {
        __syncthreads();   // the last head's rows are no longer read
        for (int r = tid; r < a.rows; r += kJoinThreads) {
          const int blk = r / a.rows_tile, rb = r - blk * a.rows_tile;
          const int x0 = main_base + (h * a.n_blk + blk) * nc;
          const Parts p = parts_of(total, blocks, x0, x0 + nc);
          float M, ls;
          if (p.b0 == p.b1) {
            const float2 x = a.item_ml[(int64_t(s) * per_step + h * a.n_blk + blk) * a.rows_blk + rb];
            M = x.x;
            ls = x.y;
          } else {
            join_ml(a, p, rb, M, ls);
          }
          row_ml[r] = ls > 0.f ? make_float2(M, 1.f / ls) : make_float2(0.f, 0.f);
        }
        __syncthreads();
        loaded = h;
      }
      const int j = (at - h * ns) * kWeightTokens + tid;
      if (j >= sp.L) continue;
      const int64_t out = (int64_t(s) * a.c.H + h) * a.c.capacity + j;
      const float before = a.weight_in ? a.weight_in[out] : 0.f;
      float sum = 0.f;
      if (j < sp.se || j >= sp.lo) {
        const int x = j < sp.se ? j : j - sp.lo + sp.se;
        for (int blk = 0; blk < a.n_blk; ++blk) {
          const int64_t step = int64_t(main_base) + (h * a.n_blk + blk) * nc + x / kStepKeys;
          const float* sc = a.scores + step * a.rows_blk * kStepKeys + x % kStepKeys;
          const int rows_here = min(a.rows - blk * a.rows_tile, a.rows_tile);
#pragma unroll 4
          for (int r = 0; r < rows_here; ++r) {
            const float2 mr = row_ml[blk * a.rows_tile + r];
            sum += ptx::ex2_approx(sc[int64_t(r) * kStepKeys] - mr.x) * mr.y;
          }
        }
      }
      a.weight_out[out] = before + sum;
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
struct DecodeShape {
  int64_t rows, rows_tile, rows_blk, n_blk, items, steps, blocks;
  size_t part_o, part_ml, item_ml, scores, bytes;   // offsets into the workspace, and its size
};

static rkv_status decode_shape(const rkv_paged_cache* c, int32_t Hq, int32_t Lq, bool weights, DecodeShape& d) {
  if (Hq < 1 || Hq % c->H) return fail(RKV_ERR_INVALID_ARG, "Hq %d must be a multiple of the cache's H %d", Hq, c->H);
  if (Lq < 1 || Lq > RKV_DECODE_MAX_LQ)
    return fail(RKV_ERR_INVALID_ARG, "Lq %d must be in [1, %d]", Lq, RKV_DECODE_MAX_LQ);
  d.rows = int64_t(Lq) * (Hq / c->H);
  if (d.rows > kMaxRows) return fail(RKV_ERR_UNSUPPORTED, "more than %d query rows to a key head", kMaxRows);
  d.rows_tile = d.rows <= 16 ? 16 : 32;
  d.rows_blk = std::min(d.rows, d.rows_tile);
  d.n_blk = (d.rows + d.rows_tile - 1) / d.rows_tile;
  d.items = int64_t(c->n_seqs) * c->H * d.n_blk;
  d.steps = d.items * ((capacity(c) + kStepKeys - 1) / kStepKeys);
  // step counts are 32-bit, and so is Lq * Hq * 16 in the zero fill
  if (d.steps >= (int64_t(1) << 30) || int64_t(c->n_seqs) * Lq >= (int64_t(1) << 31) || int64_t(Hq) * Lq >= (1 << 26))
    return fail(RKV_ERR_UNSUPPORTED, "too many sequences, heads and tokens for one launch");
  d.blocks = std::min<int64_t>(sm_count(), std::max<int64_t>(d.steps, 1));
  auto up = [](size_t x) { return (x + 15) / 16 * 16; };
  d.part_o = 0;
  d.part_ml = d.part_o + up(size_t(d.blocks * 2 * d.rows_blk) * kHD * 4);
  d.item_ml = d.part_ml + up(size_t(d.blocks * 2 * d.rows_blk) * 8);
  d.scores = d.item_ml + (weights ? up(size_t(d.items * d.rows_blk) * 8) : 0);
  d.bytes = d.scores + (weights ? size_t(d.steps * d.rows_blk) * kStepKeys * 4 : 0);
  return RKV_OK;
}

template <int MT, int kStages, bool kWeights>
static rkv_status launch_decode(const DecodeArgs& a, cudaStream_t cs) {
  auto kern = decode_paged_kernel<MT, kStages, kWeights>;
  constexpr int smem = DecSmem<MT, kStages>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(decode_paged_kernel)");
  kern<<<uint32_t(a.main_blocks), kDecThreads, smem, cs>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "decode_paged_kernel launch");
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  // the weights pass takes more blocks than the join needs
  cfg.gridDim = dim3(uint32_t(kWeights ? 4 * sm_count() : a.main_blocks));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = kWeights ? size_t(a.rows) * 8 : 0;
  cfg.stream = cs;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, decode_join_kernel<kWeights>, a);
  if (e == cudaSuccess) e = cudaGetLastError();
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
  const int64_t row = int64_t(Hq) * kHD;
  for (int64_t stride : {q_row_stride, o_row_stride}) {
    if (stride < row) return fail(RKV_ERR_INVALID_ARG, "row stride < Hq*D");
    if (stride % 8) return fail(RKV_ERR_INVALID_ARG, "rows of q/o must be 16-byte aligned");
    if (stride >= (int64_t(1) << 40)) return fail(RKV_ERR_INVALID_ARG, "row stride too large");
  }
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return fail(RKV_ERR_INVALID_ARG, "softmax_scale must be > 0");
  if (window < 0 || sinks < 0) return fail(RKV_ERR_INVALID_ARG, "window and sinks must be >= 0");
  if (weight_in && !weight_out) return fail(RKV_ERR_INVALID_ARG, "weight_in without weight_out");
  const int64_t n_rows = int64_t(cache->n_seqs) * Lq;
  if (rows_overlap(o, n_rows, o_row_stride * 2, row * 2, q, n_rows, q_row_stride * 2, row * 2))
    return fail(RKV_ERR_INVALID_ARG, "o overlaps q");
  const uint64_t o_bytes = uint64_t((n_rows - 1) * o_row_stride + row) * 2;
  if (overlaps_pool(cache, o, o_bytes)) return fail(RKV_ERR_INVALID_ARG, "o overlaps the pool");
  const uint64_t sb = uint64_t(cache->n_seqs) * cache->H * capacity(cache) * 4;
  if (weight_out) {
    if (weight_in && weight_in != weight_out && overlaps(weight_in, sb, weight_out, sb))
      return fail(RKV_ERR_INVALID_ARG, "weight_in and weight_out overlap in part");
    if (overlaps(weight_out, sb, o, o_bytes) ||
        overlaps(weight_out, sb, q, uint64_t((n_rows - 1) * q_row_stride + row) * 2) ||
        overlaps_pool(cache, weight_out, sb))
      return fail(RKV_ERR_INVALID_ARG, "weight_out overlaps q, o or the pool");
  }
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
  a.item_ml = reinterpret_cast<float2*>(ws + d.item_ml);
  a.scores = reinterpret_cast<float*>(ws + d.scores);
  a.scale_log2 = float(double(softmax_scale) * 1.4426950408889634);
  a.Hq = Hq;
  a.Lq = Lq;
  a.G = Hq / cache->H;
  a.rows = int32_t(d.rows);
  a.rows_tile = int32_t(d.rows_tile);
  a.rows_blk = int32_t(d.rows_blk);
  a.n_blk = int32_t(d.n_blk);
  a.window = window;
  a.sinks = sinks;
  a.main_blocks = int32_t(d.blocks);
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (d.rows_tile == 16) return weight_out ? launch_decode<1, 3, true>(a, cs) : launch_decode<1, 3, false>(a, cs);
  return weight_out ? launch_decode<2, 2, true>(a, cs) : launch_decode<2, 2, false>(a, cs);
}
