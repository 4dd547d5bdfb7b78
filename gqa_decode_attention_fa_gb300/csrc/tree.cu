// Attention for a tree of drafted tokens over a KV cache (include/gqa_tree.h) on the
// 5th-generation tensor core, and the tree's masks and positions.
//
// Rows.  The n_b nodes of a sequence and the G query heads of a KV head make n_b G rows that
// all read the same keys; a row tile is Tt = 128 / G nodes, 128 rows, the M of every MMA.  Every
// row sees the whole context, so the work is one pass over K and V per row tile; only the last
// tiles, which hold the nodes' own slots, are masked, by the bits of the node's mask.
//
// Work.  The batch's tokens, in tiles of 64 (one page) sequence after sequence, are cut into W
// contiguous ranges of equal cost whatever the sequence boundaries, so ragged batches and single
// long sequences both fill the GPU; the lengths are read on the device.  CTA (w, kv, r) streams KV
// head kv of range w for row tile r, or for two of them.  The CTAs of a range run side by side: the
// heads of a token lie next to each other in the cache, and streamed together they read HBM in
// whole rows (8 x 32k single tokens 182 us with the heads of a tile read at different times, 177 us
// so), and the row tiles share their tiles in L2.  A piece of a range that is a whole sequence
// writes its output rows; one that is cut leaves (O, m, l) in the workspace and tree_merge_kernel
// joins the parts in order.
//
// Attention CTA, one per SM: a TMA warp streams the K and V tiles through deep rings; two streams of
// an MMA warp and four softmax warps each work on them, so that one stream's softmax overlaps the
// other's products.  Where the CTA has two row tiles (R >= 2) each stream takes one and both use
// every tile: a tile's way through TMA, whose rows of 128 bytes an SM takes at about 50 GB/s, is
// paid once for 256 rows.  Where it has one, the streams take the even and the odd tiles and join
// their O at the end (a softmax thread finds both in its own tensor-memory lane).
//   A stream's MMA warp issues S = Q K^T into one of two tensor-memory buffers and O += P V, P
// read from tensor memory as bf16 hi + lo (rounding P to one bf16 would add an error as large as
// the output's own rounding); a softmax thread holds a row.  The maximum is raised lazily (by more
// than 2^8), so most tiles rescale nothing.  The pipeline runs on across the pieces of a range.
//
// Bounds.  One row tile: HBM (K and V once); 8 x 32k single tokens 160 us = 6.7 TB/s, 0.99 of the
// measured copy rate; 32 ragged drafts of up to 16 nodes 105 us, 0.87 (start, the ends of the
// sequences, the merge).  Many short sequences: their ends; 256 single tokens on 200 each 78 us, 0.41.
// More row tiles: the tensor core with P as hi + lo, 1.5 x the products of the formula; 64 nodes on 128k
// tokens 263 us = 1.05 PFLOP/s of the formula's, 1.57 issued, and 280 us where calls follow each other for
// more than 5 ms or so (the card's power limit: 1.93 GHz instead of 2.07).  Small calls: latency,
// 8 us for the shortest (2.3 us to find the range and set up, 1.7 to the first scores).  Slower and
// not kept (the last case, us): two CTAs an SM with shorter rings 297; 128-token stages with one S
// buffer (an MMA of N = 64 takes as long as one of N = 128, but the softmax then waits for it) 312; S
// and P in buffers of their own 297; sixteen softmax warps of 16 rows each, through the 16-lane shapes of
// tensor memory, 283 (ragged drafts 108, the shortest call 9.7), with stages of 128 tokens 417; tiles
// brought to L2 by TMA prefetches 3 to 12 ahead, the second pass through TMA costing more than it hides
// (single tokens 208 to 309).
#include <math.h>
#include <string.h>

#include <atomic>

#include "../../include/gqa_tree.h"
#include "op_args.h"
#include "pairmath.cuh"
#include "tc05.cuh"

namespace gqa {

struct TreeParams {
  const int32_t *page_table, *ctx_lens, *counts;
  const uint64_t *mask;
  const uint16_t *v_cache;
  uint16_t *out;
  float *part;                  // [W * Hkv * R * 2][130][128]: O columns, m, l of a cut piece
  uint32_t *err;
  int B, T, Hq, Hkv, G, Tt, R;  // R row tiles of Tt nodes
  int words;                    // 64-bit words of a mask row
  int paged, max_seq, max_blocks, num_blocks;
  int W;                        // ranges the grid is sized for
  int out_wide;                 // `out` is 32-byte aligned
  int merge_by_sequence;        // the merge's first index is a sequence, else a boundary between ranges
  float scale_log2;
};

namespace {

constexpr int kTrRows = 128;                 // M of every MMA
constexpr int kTrStreams = 2;
constexpr int kTrMmaWarp = 8;                // and 9: a stream's each
constexpr int kTrProducerWarp = 10;
constexpr int kTrThreads = 32 * 11;
// Tensor memory: a stream's two S buffers (64 fp32 columns each; P overwrites S as bf16 pairs, each 32
// keys' hi in 16 columns, their lo in the next 16) and its O (128 columns).
constexpr uint32_t kTrTmemStream = 256;
constexpr uint32_t kTrTmemCols = kTrStreams * kTrTmemStream;
constexpr uint32_t kTrTmemO = 128;
constexpr float kTrRescaleLog2 = 8.f;

constexpr int kTrQBytes = 2 * kTrRows * kHalfRowBytes;  // 32 KiB: two 64-dim panels
constexpr int kTrTileBytes = 2 * kHalfTileBytes;         // 16 KiB: a K or V tile's two halves
constexpr int kTrPartFloats = (kHeadDim + 2) * kTrRows;

// Shared memory of the kernel with NQ query tiles: what they leave is the K and V rings.
template <int NQ>
struct TreeSmem {
  static constexpr int kStages = NQ == 1 ? 6 : 5;  // of K and of V
  static constexpr int kOffK = NQ * kTrQBytes;
  static constexpr int kOffV = kOffK + kStages * kTrTileBytes;
  static constexpr int kOffMl = kOffV + kStages * kTrTileBytes;  // [2 streams][128] (m, l)
  // barriers: k_full, k_empty, v_full, v_empty [kStages], s_full, p_full [2 streams][2],
  // pv_done, o_full, o_free, drain [2 streams], q_full, q_empty, meet
  static constexpr int kNumBars = 4 * kStages + 2 * 4 + 4 * 2 + 3;
  static constexpr int kOffBar = kOffMl + kTrStreams * kTrRows * 8;
  static constexpr int kBytes = kOffBar + 8 * kNumBars + 4 * 5 + 12;
  static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
  static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0, "swizzled tiles 1024-aligned");
};

// Nodes of sequence b, or -1 when its lengths are invalid.
__device__ __forceinline__ int tree_nodes(const TreeParams &p, int b, int ctx) {
  const int n = p.counts ? p.counts[b] : p.T;
  return (ctx >= 0 && n >= 0 && n <= p.T && static_cast<long long>(ctx) + n <= p.max_seq) ? n : -1;
}
// KV tiles of sequence b: those up to its last node's slot, none when it has no node.
__device__ __forceinline__ int tree_tiles(const TreeParams &p, int b) {
  const int ctx = p.ctx_lens[b], n = tree_nodes(p, b, ctx);
  return n > 0 ? (ctx + n - 1) / kTile + 1 : 0;
}

// How the batch is cut.  Tiles are numbered sequence after sequence; behind each sequence with tiles
// but the last, `gap` numbers are left out, the cost of a piece's end in tiles, so that a range with many
// short sequences gets fewer tiles.  (The streams run dry, O goes out: about 3 us of a CTA, four tiles
// at HBM's pace.  7 counts the end of two row tiles alike, and was the faster: 32 ragged drafts 103.7 us and 64
// sequences of 300 to 3000 tokens 80.7, against 104.7 and 82.3 with 10.)  The
// numbers, fewer than 2^31, go to the ranges in order, `each` to a range, one more to the first `more`.
//   Batches of few short sequences are not cut: a range is a sequence where none is longer, in tiles,
// than a range, the ends in it and the merge (about kTrMergeCost tiles) would cost otherwise.  (15
// sequences of 8 tiles, 8 KV heads: 26 us cut, 15 us whole.)  The numbers are then those of the sequences.
constexpr int kTrPieceCost = 7;
constexpr int kTrMergeCost = 8;
constexpr int kTrMinTiles = 4;  // of a range, so that small batches leave few partials
struct TreeCut {
  int ranges, gap, each, more;
  bool whole;      // a range is a sequence
  int lane_first;  // first number of the warp's lane's sequences [lane per, lane per + per)

  __device__ __forceinline__ int begin(int w) const { return w * each + min(w, more); }
  __device__ __forceinline__ int range_of(int x) const {
    const int wide = (each + 1) * more;
    return x < wide ? x / (each + 1) : more + (x - wide) / each;
  }
};
// Every lane of a warp calls these alike.
__device__ __forceinline__ TreeCut tree_cut(const TreeParams &p, int lane) {
  const int per = (p.B + 31) / 32, b0 = lane * per, b1 = min(p.B, b0 + per);
  int tiles = 0, seqs = 0, longest = 0;
  for (int b = b0; b < b1; ++b) {
    const int nt = tree_tiles(p, b);
    tiles += nt;
    seqs += nt > 0;
    longest = max(longest, nt);
  }
  const int own_tiles = tiles, own_seqs = seqs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, tiles, o), z = __shfl_up_sync(0xffffffffu, seqs, o);
    if (lane >= o) tiles += y, seqs += z;
  }
  const int all = __shfl_sync(0xffffffffu, tiles, 31), all_seqs = __shfl_sync(0xffffffffu, seqs, 31);
  TreeCut c;
  c.ranges = all < 1 ? 0 : max(1, min(p.W, all / kTrMinTiles));
  const int quarter = c.ranges > 0 ? all / c.ranges / 4 : 0;  // of a range
  c.gap = min(quarter, kTrPieceCost);
  longest = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(longest)));
  c.whole = c.ranges > 0 && all_seqs <= p.W &&
            longest <= all / c.ranges + kTrPieceCost * all_seqs / c.ranges + kTrMergeCost;
  if (c.whole) c.ranges = all_seqs;
  const int total = c.whole ? all_seqs : all + c.gap * max(0, all_seqs - 1);
  c.each = c.ranges > 0 ? total / c.ranges : 0;
  c.more = total - c.each * c.ranges;
  c.lane_first = c.whole ? seqs - own_seqs : tiles - own_tiles + c.gap * (seqs - own_seqs);
  return c;
}
__device__ __forceinline__ int tree_span(const TreeParams &p, const TreeCut &c, int b) {
  const int nt = tree_tiles(p, b);
  return nt < 1 ? 0 : c.whole ? 1 : nt + c.gap;
}
// The sequence whose numbers (or the gap behind them) hold `at`, below their end, and its first number.
__device__ __forceinline__ void tree_find(const TreeParams &p, const TreeCut &c, int at, int *b, int *seq0) {
  // the last lane whose first number is <= at (lanes without tiles share their successor's)
  const uint32_t le = __ballot_sync(0xffffffffu, c.lane_first <= at);
  const int owner = 31 - __clz(le);
  const int per = (p.B + 31) / 32;
  int s = __shfl_sync(0xffffffffu, c.lane_first, owner);
  int x = owner * per;
  while (x + 1 < p.B) {
    const int nxt = s + tree_span(p, c, x);
    if (nxt > at) break;
    s = nxt;
    ++x;
  }
  *b = x;
  *seq0 = s;
}

// Walks the sequences a range [pos, end) covers.  Every warp of the CTA runs its own copy, all
// lanes alike.
struct TreeWalk {
  int pos, end;         // numbers still to do
  int seq0;             // first number of sequence b
  int b, gap;
  int ctx, n, nt;       // sequence b: context, nodes (-1: invalid lengths), tiles
  int ctx_next, n_next; // of sequence b + 1, on the way while b is worked on
  // of the piece at hand
  int j0, j1;
  bool whole;  // the piece is its whole sequence

  __device__ __forceinline__ void start(const TreeParams &p, int begin, int stop, int b0, int s0, int g) {
    pos = begin;
    end = stop;
    b = b0;
    seq0 = s0;
    gap = g;
    nt = 0;
    if (pos < end) {
      fetch(p, b);
      enter(p);
    }
  }
  __device__ __forceinline__ void fetch(const TreeParams &p, int x) {
    ctx_next = x < p.B ? p.ctx_lens[x] : 0;
    n_next = x < p.B && p.counts ? p.counts[x] : p.T;
  }
  __device__ __forceinline__ void enter(const TreeParams &p) {  // sequence b, whose lengths were fetched
    ctx = ctx_next;
    n = (ctx >= 0 && n_next >= 0 && n_next <= p.T && static_cast<long long>(ctx) + n_next <= p.max_seq) ? n_next : -1;
    nt = n > 0 ? (ctx + n - 1) / kTile + 1 : 0;
    fetch(p, b + 1);
  }
  // The next piece; false when the range is done.
  __device__ __forceinline__ bool next(const TreeParams &p) {
    while (pos < end && pos >= seq0 + nt) {  // on to the next sequence
      seq0 += nt > 0 ? nt + gap : 0;
      if (pos < seq0) pos = seq0;
      if (pos >= end) break;
      ++b;
      enter(p);
    }
    if (pos >= end) return false;
    j0 = pos - seq0;
    j1 = min(nt, j0 + end - pos);
    whole = j0 == 0 && j1 == nt;
    pos += j1 - j0;
    return true;
  }
};

__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}
// 32 bytes to global memory: a thread's whole sector, in one store where the address allows it.
__device__ __forceinline__ void store_32b(uint16_t *dst, const uint32_t (&x)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
                 "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}
// 16 columns of the thread's row, as tmem_ld32 and tmem_st32.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

}  // namespace

// ------------------------------------------------------------------------- masks, positions
// A CTA per sequence, a thread per node: pointer jumping.  After each round a node's mask holds
// the path up to (not including) the node `up` points at, so ceil(log2 depth) rounds suffice.
__global__ void __launch_bounds__(GQA_MAX_TREE) tree_prepare_kernel(const int32_t *parents, const int32_t *ctx_lens,
                                                                    const int32_t *counts, uint64_t *mask,
                                                                    int32_t *positions, int T, uint32_t *err) {
  __shared__ uint64_t s_mask[4][GQA_MAX_TREE];
  __shared__ int s_up[GQA_MAX_TREE], s_len[GQA_MAX_TREE];
  griddep_wait();
  const int b = blockIdx.x, t = threadIdx.x, words = (T + 63) / 64;
  const int ctx = ctx_lens[b], n = counts ? counts[b] : T;
  if (ctx < 0 || n < 0 || n > T || static_cast<long long>(ctx) + n > 0x7fffffffLL) {
    if (t == 0) flag_error(err, GQA_DEVERR_SEQLEN);
    return;
  }
  int up = -1, len = 1;
  uint64_t m[4] = {0, 0, 0, 0};
  if (t < n) {
    up = parents[static_cast<long long>(b) * T + t];
    if (up < -1 || up >= t) {
      flag_error(err, GQA_DEVERR_POSITION);
      up = -1;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) m[w] = (t >> 6) == w ? 1ull << (t & 63) : 0ull;
  }
  while (__syncthreads_or(up >= 0)) {
    s_up[t] = up;
    s_len[t] = len;
#pragma unroll
    for (int w = 0; w < 4; ++w) s_mask[w][t] = m[w];
    __syncthreads();
    if (up >= 0) {
      len += s_len[up];
#pragma unroll
      for (int w = 0; w < 4; ++w) m[w] |= s_mask[w][up];
      up = s_up[up];
    }
  }
  if (t < n) {
    const long long row = static_cast<long long>(b) * T + t;
    positions[row] = ctx + len - 1;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (w < words) mask[row * words + w] = m[w];
  }
}

// ------------------------------------------------------------------------------- attention
// The values of the seen nodes u0 <= u < u1 that are not finite, which the products left out, come to
// dims d0 .. d1 - 1 of a node's row after all: p x inf for some p > 0.  The row, which this thread has just
// written, is the output's, scaled by inv, or column-major in the workspace.
__device__ __noinline__ void add_nonfinite(const TreeParams &p, int b, int t, int kv, int ctx, int u0, int u1, int d0, int d1,
                                           uint16_t *out, float *part, float inv) {
  const uint64_t *mrow = p.mask + (static_cast<long long>(b) * p.T + t) * p.words;
  for (int u = u0; u < u1; ++u) {
    if (!((mrow[u >> 6] >> (u & 63)) & 1ull)) continue;
    const int slot = ctx + u;
    long long crow = static_cast<long long>(b) * p.max_seq + slot;
    if (p.paged) {
      const int pg = p.page_table[static_cast<long long>(b) * p.max_blocks + slot / kTile];
      if (pg < 0 || pg >= p.num_blocks) continue;
      crow = static_cast<long long>(pg) * kTile + (slot & (kTile - 1));
    }
    const uint16_t *v = p.v_cache + (crow * p.Hkv + kv) * kHeadDim;
#pragma unroll 1
    for (int d = d0; d < d1; ++d) {
      const uint32_t y = v[d];
      if ((y & 0x7f80u) != 0x7f80u) continue;
      if (out)
        out[d] = static_cast<uint16_t>(pack_bf16(bf16_lo_to_float(out[d]) + bf16_lo_to_float(y) * inv, 0.f) & 0xffffu);
      else
        part[d * kTrRows] += bf16_lo_to_float(y);
    }
  }
}

template <int NQ>
__global__ void __launch_bounds__(kTrThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeParams p) {
  using Smem = TreeSmem<NQ>;
  constexpr int kStages = Smem::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_addr(smem_raw) & 1023u) != 0u) {  // a launch assumption broken: no work at all
    if (threadIdx.x == 0) flag_error(p.err, GQA_DEVERR_LAUNCH);
    return;
  }
  uint8_t *smem = smem_raw;
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + Smem::kOffBar);
  uint64_t *k_empty = k_full + kStages;
  uint64_t *v_full = k_empty + kStages;
  uint64_t *v_empty = v_full + kStages;
  uint64_t *s_full = v_empty + kStages;  // [stream][buffer]
  uint64_t *p_full = s_full + 4;
  uint64_t *pv_done = p_full + 4;  // [stream]
  uint64_t *o_full = pv_done + 2;
  uint64_t *o_free = o_full + 2;
  uint64_t *drain = o_free + 2;
  uint64_t *q_full = drain + 2;
  uint64_t *q_empty = q_full + 1;
  uint64_t *meet = q_full + 2;  // all eight softmax warps
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(k_full + Smem::kNumBars);
  // the last piece (from 1) of those with piece % 4 = i that had a non-finite value in a node's V
  // row (a stream is at most two pieces ahead of the other: the queries are given back by both)
  uint32_t *v_bad = tmem_slot + 1;
  float2 *s_ml = reinterpret_cast<float2 *>(smem + Smem::kOffMl);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = (p.R + NQ - 1) / NQ;  // row tiles, NQ at a time
  const int r0 = static_cast<int>(blockIdx.x) % units * NQ, kv = static_cast<int>(blockIdx.x) / units % p.Hkv,
            w = static_cast<int>(blockIdx.x) / units / p.Hkv;

  griddep_wait();  // everything below may come from the preceding kernel
  if (p.W > 1) griddep_launch_dependents();  // tree_merge_kernel follows, and it waits
  // Tensor memory, barriers and maps are set up by a warp each, while the others look for the range.
  if (warp == kTrMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), kTrTmemCols);
    tmem_relinquish();
  } else if (warp == kTrMmaWarp + 1) {
    for (int i = lane; i < Smem::kNumBars; i += 32) {
      uint64_t *bar = k_full + i;
      // the queries, and tiles that both streams use, are given back by both; P comes from a stream's
      // four softmax warps; O is read by all eight
      int count = 1;
      if ((bar >= k_empty && bar < v_full) || (bar >= v_empty && bar < s_full)) count = NQ;
      if (bar == q_empty) count = 2;
      if (bar >= p_full && bar < pv_done) count = 4;
      if ((bar >= o_free && bar < drain) || bar == meet) count = 8;
      mbar_init(smem_addr(bar), count);
    }
    if (lane < 4) v_bad[lane] = 0;
    fence_barrier_init();
    __syncwarp();
  } else if (warp == kTrProducerWarp && lane == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  TreeWalk walk;
  {
    const TreeCut cut = tree_cut(p, lane);
    int begin = 0, stop = 0, seq0 = 0, b = 0;
    if (w < cut.ranges) {
      begin = cut.begin(w);
      stop = cut.begin(w + 1);
      tree_find(p, cut, begin, &b, &seq0);
      if (cut.whole) begin = seq0 = 0, stop = tree_tiles(p, b);
    }
    walk.start(p, begin, stop, b, seq0, cut.gap);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Sequences with invalid lengths: flagged, zeros in all their rows.
  for (int b = static_cast<int>(blockIdx.x); b < p.B; b += static_cast<int>(gridDim.x)) {
    const int ctx = p.ctx_lens[b];
    if (tree_nodes(p, b, ctx) >= 0) continue;
    if (tid == 0) flag_error(p.err, ctx < 0 ? GQA_DEVERR_POSITION : GQA_DEVERR_SEQLEN);
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + static_cast<long long>(b) * p.T * p.Hq * kHeadDim);
    const long long n = static_cast<long long>(p.T) * p.Hq * kHeadDim / 8;
    for (long long c = tid; c < n; c += kTrThreads) dst[c] = make_uint4(0, 0, 0, 0);
  }

  auto k_ptr = [&](int s) { return smem + Smem::kOffK + s * kTrTileBytes; };
  auto v_ptr = [&](int s) { return smem + Smem::kOffV + s * kTrTileBytes; };
  // A piece's streams: 0 if the CTA's row tiles have no node in the sequence, 1 if only the first
  // has (the streams share its tiles), 2 if both have (each stream takes all tiles for its own).
  auto row_tiles = [&](const TreeWalk &x) {
    return r0 * p.Tt >= x.n ? 0 : (NQ == 2 && (r0 + 1) * p.Tt < x.n) ? 2 : 1;
  };

  if (warp == kTrProducerWarp) {
    // ------------------------------------------------------------------ TMA producer
    // The whole warp walks (a lane holds the cache row of one of the next 32 tiles, the 32 after
    // them are fetched ahead); lane 0 issues the loads.
    int it = 0, piece = 0, queries = 0;  // KV tiles, pieces, loads of queries so far: stages and phases
    bool ok = true;
    while (ok && walk.next(p)) {
      const int b = walk.b, j0 = walk.j0, j1 = walk.j1, nr = row_tiles(walk);
      if (nr == 0) continue;
      auto row_of = [&](int j) -> int {  // -kTile where there is none: TMA fills zeros
        if (j >= j1) return -kTile;
        if (!p.paged) return b * p.max_seq + j * kTile;
        const int pg = p.page_table[static_cast<long long>(b) * p.max_blocks + j];
        if (pg < 0 || pg >= p.num_blocks) {
          flag_error(p.err, GQA_DEVERR_PAGE);
          return -kTile;
        }
        return pg * kTile;
      };
      int rows = row_of(j0 + lane), rows_next = row_of(j0 + 32 + lane), base = j0;
      // The queries, once the last S of the piece before has read its own; until then the piece's
      // first tiles, as far as the rings take them without an S of this piece.
      bool q_sent = false;
      auto send_q = [&](bool wait) {
        bool free = piece == 0;
        if (!free) {
          const uint32_t bar = smem_addr(q_empty), phase = static_cast<uint32_t>((piece - 1) & 1);
          free = __all_sync(0xffffffffu, wait ? mbar_wait(bar, phase) : mbar_try_wait(bar, phase));
        }
        if (!free) return !wait;
        q_sent = true;
        if (lane == 0) {
          mbar_arrive_expect_tx(smem_addr(q_full), 2u * 64u * 2u * static_cast<uint32_t>(p.G * p.Tt * nr));
          for (int x = 0; x < nr; ++x) {
            const uint32_t qd = smem_addr(smem) + x * kTrQBytes;
            tma_load_4d(qd, &tmQ, smem_addr(q_full), 0, kv * p.G, (r0 + x) * p.Tt, b);
            tma_load_4d(qd + kTrRows * kHalfRowBytes, &tmQ, smem_addr(q_full), 64, kv * p.G, (r0 + x) * p.Tt, b);
          }
        }
        return true;
      };
      for (int j = j0; j < j1; ++j, ++it) {
        if (!q_sent) ok = send_q(j - j0 == kStages - 1);
        if (!ok) break;
        if (j - base == 32) {
          base += 32;
          rows = rows_next;
          rows_next = row_of(base + 32 + lane);
        }
        const int row = __shfl_sync(0xffffffffu, rows, j - base);
        const int st = it % kStages;
        const uint32_t free_phase = static_cast<uint32_t>((it / kStages - 1) & 1);
        if (it >= kStages) ok = mbar_wait(smem_addr(&k_empty[st]), free_phase);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t kb = smem_addr(&k_full[st]), kd = smem_addr(k_ptr(st));
          mbar_arrive_expect_tx(kb, kTrTileBytes);
          tma_load_3d(kd, &tmK, kb, 0, kv, row);
          tma_load_3d(kd + kHalfTileBytes, &tmK, kb, 64, kv, row);
        }
        if (it >= kStages) ok = mbar_wait(smem_addr(&v_empty[st]), free_phase);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          const uint32_t vb = smem_addr(&v_full[st]), vd = smem_addr(v_ptr(st));
          mbar_arrive_expect_tx(vb, kTrTileBytes);
          tma_load_3d(vd, &tmV, vb, 0, kv, row);
          tma_load_3d(vd + kHalfTileBytes, &tmV, vb, 64, kv, row);
        }
      }
      if (ok && !q_sent) ok = send_q(true);
      queries += q_sent;
      ++piece;
    }
    if (!ok && lane == 0) {
      flag_error(p.err, GQA_DEVERR_TIMEOUT);
      // Do not leave while copies into this CTA's shared memory may still be in flight: wait out
      // every phase that a load was issued for (tile `it` may have its K loads alone).
      if (queries > 0) (void)mbar_wait(smem_addr(q_full), static_cast<uint32_t>((queries - 1) & 1));
      for (int i = (it + 1 > kStages ? it + 1 - kStages : 0); i <= it; ++i)
        (void)mbar_wait(smem_addr(&k_full[i % kStages]), static_cast<uint32_t>((i / kStages) & 1));
      for (int i = (it > kStages ? it - kStages : 0); i < it; ++i)
        (void)mbar_wait(smem_addr(&v_full[i % kStages]), static_cast<uint32_t>((i / kStages) & 1));
    }
  } else if (warp >= kTrMmaWarp) {
    // ------------------------------------------------------------------ MMA issuer of a stream
    // Issue order within a piece: S_0, S_1, PV_0, S_2, PV_1, ..., PV_last (of the stream's tiles).
    // S overwrites the buffer that held the P of two tiles before; that P V was issued before it
    // and the tensor pipe runs them in order.  With one row tile the tiles are given back by
    // commits, at once: HBM is the bound.  With two the products are, and a commit holds the pipe up
    // for about 100 cycles: there is one a tile, after S, which also says that every P V before is
    // done, and the softmax warps that see it give the tiles back (64 nodes on 128k: 338 -> 291 us;
    // done so with one row tile, 8 x 32k single tokens take 186 us instead of 176).
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(kTrRows, kTile, false, false);
      constexpr uint32_t kIdO = idesc_bf16_f32(kTrRows, kHeadDim, false, true);
      const int st = warp - kTrMmaWarp;
      const uint32_t tm = tmem + st * kTrTmemStream;
      uint64_t *const sf = s_full + 2 * st, *const pf = p_full + 2 * st;
      // descriptors of the first tiles; the others differ in the start address alone (16-byte units,
      // below 2^14 anywhere in shared memory), so one addition gives each: the issue must keep up
      const uint64_t qd0 = sdesc_sw128(smem_addr(smem), 16, 1024), kd0 = sdesc_sw128(smem_addr(k_ptr(0)), 16, 1024),
                     vd0 = sdesc_sw128(smem_addr(v_ptr(0)), kHalfTileBytes, 1024);
      int it0 = 0, is = 0, piece = 0;  // the CTA's tiles before the piece, the stream's own, pieces
      bool ok = true;
      // O += P V for the stream's tile number x, the CTA's tile number t
      auto issue_pv = [&](int x, int t, bool first) -> bool {
        const int pb = x & 1, sv = t % kStages;
        if (!mbar_wait(smem_addr(&v_full[sv]), static_cast<uint32_t>((t / kStages) & 1))) return false;
        if (!mbar_wait(smem_addr(&pf[pb]), static_cast<uint32_t>((x >> 1) & 1))) return false;
        tc_fence_after();
        const uint64_t vd = vd0 + static_cast<uint64_t>(sv * (kTrTileBytes / 16));
        const uint32_t pt = tm + 64 * pb;
#pragma unroll
        for (int k = 0; k < 2 * kTile / 16; ++k) {  // 16 keys each: hi of all, then lo
          const int x = k % (kTile / 16);
          umma_bf16_ts(tm + kTrTmemO, pt + 32 * (x >> 1) + 8 * (x & 1) + 16 * (k / (kTile / 16)), vd + 128 * x, kIdO,
                       k > 0 || !first ? 1u : 0u);
        }
        if (NQ == 1) umma_commit(smem_addr(&v_empty[sv]));
        return true;
      };
      while (ok && walk.next(p)) {
        const int nr = row_tiles(walk);
        if (nr == 0) continue;
        const int nt = walk.j1 - walk.j0, step = nr == 1 ? 2 : 1, first = nr == 1 ? st : 0;
        const uint64_t qd = qd0 + (nr == 2 ? st * (kTrQBytes / 16) : 0);
        ok = mbar_wait(smem_addr(q_full), static_cast<uint32_t>(piece & 1));
        for (int i = first; i < nt && ok; i += step, ++is) {
          const int t = it0 + i, sk = t % kStages, sb = is & 1;
          ok = mbar_wait(smem_addr(&k_full[sk]), static_cast<uint32_t>((t / kStages) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = kd0 + static_cast<uint64_t>(sk * (kTrTileBytes / 16));
#pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k)
            umma_bf16(tm + 64 * sb, qd + (k >> 2) * (kTrRows * kHalfRowBytes / 16) + 2 * (k & 3),
                      kd + (k >> 2) * (kHalfTileBytes / 16) + 2 * (k & 3), kIdS, k > 0 ? 1u : 0u);
          umma_commit(smem_addr(&sf[sb]));
          if (NQ == 1) umma_commit(smem_addr(&k_empty[sk]));
          if (i > first) {
            ok = issue_pv(is - 1, t - step, i - step == first);
            if (i + step >= nt && ok) umma_commit(smem_addr(&pv_done[st]));  // all but the last P V
          } else if (piece > 0) {
            // O of the piece before must have been read before this piece's first P V
            ok = mbar_wait(smem_addr(&o_free[st]), static_cast<uint32_t>((piece - 1) & 1));
          }
        }
        if (first < nt) {
          if (ok) {
            const int last = first + (nt - 1 - first) / step * step;
            ok = issue_pv(is - 1, it0 + last, last == first);
          }
          if (ok) umma_commit(smem_addr(&o_full[st]));
        } else if (ok) {  // one tile, the other stream's
          if (piece > 0) ok = mbar_wait(smem_addr(&o_free[st]), static_cast<uint32_t>((piece - 1) & 1));
          mbar_arrive(smem_addr(&o_full[st]));
        }
        it0 += nt;
        ++piece;
      }
      if (!ok) flag_error(p.err, GQA_DEVERR_TIMEOUT);
      if (is > 0) {  // nothing is deallocated while an MMA runs
        umma_commit(smem_addr(&drain[st]));
        if (!mbar_wait(smem_addr(&drain[st]), 0)) flag_error(p.err, GQA_DEVERR_TIMEOUT);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax warps of a stream
    const int st = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int tl = row / p.G, g = row - tl * p.G;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm = tmem + lane_base + st * kTrTmemStream;
    uint64_t *const sf = s_full + 2 * st, *const pf = p_full + 2 * st;
    int it0 = 0, is = 0, piece = 0, met = 0, pv = 0;  // (pv: pieces with more than one tile of the stream's)
    bool ok = true;
    // A barrier of the eight softmax warps, with a limit to the wait (a warp that gave up on
    // another wait does not come).
    auto softmax_barrier = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(meet));
      return mbar_wait(smem_addr(meet), static_cast<uint32_t>(met++ & 1));
    };
    while (ok && walk.next(p)) {
      const int b = walk.b, j0 = walk.j0, j1 = walk.j1;
      const int ctx = walk.ctx, n = walk.n, nr = row_tiles(walk);
      if (nr == 0) continue;
      const int r = r0 + (nr == 2 ? st : 0), step = nr == 1 ? 2 : 1, first = nr == 1 ? st : 0;
      const int t = r * p.Tt + tl;  // this row's node
      const bool valid = tl < p.Tt && t < n;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const uint64_t *mrow = p.mask + (static_cast<long long>(b) * p.T + t) * p.words;
      const uint64_t mask0 = valid ? mrow[0] : 0ull;  // on the way while the context is streamed
      // bits 64 x .. 64 x + 63 of the node's mask, none from n on
      auto mask_word = [&](int x) -> uint64_t {
        const int left = n - 64 * x;
        if (left <= 0) return 0ull;
        const uint64_t m = x == 0 ? mask0 : mrow[x];
        return left >= 64 ? m : m & ((1ull << left) - 1ull);
      };
      float m_run = -INFINITY, l_run = 0.f;
      const uint32_t shares = nr == 1 ? 2 : 1;  // of the tiles' two users, those this stream stands for
      for (int j = j0 + first; j < j1; j += step, ++is) {
        const int sb = is & 1;
        const int o0 = j * kTile - ctx;  // the node at the tile's first slot; negative: context
        const bool tail = o0 > -kTile;   // the tile holds slots of nodes
        uint64_t see = ~0ull;
        if (tail) {
          see = 0ull;
          if (valid) {
            if (o0 < 0) {
              see = ((1ull << -o0) - 1ull) | (mask_word(0) << -o0);
            } else {
              const int x = o0 >> 6, sh = o0 & 63;
              see = mask_word(x) >> sh;
              if (sh) see |= mask_word(x + 1) << (64 - sh);
            }
          }
          // This tile's V: rows that no node owns (nothing has written them) are cleared, and
          // so is a non-finite value in a node's row, which would reach the rows that do not see the
          // node as 0 x inf; the epilogue gives it to those that do.  When both streams use the
          // tile, each looks at half of it.
          const int tt = it0 + (j - j0), vs = tt % kStages;
          ok = mbar_wait(smem_addr(&v_full[vs]), static_cast<uint32_t>((tt / kStages) & 1));
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          // 16-byte chunks: slot, half, chunk, from the first node's slot on
          bool bad = false;
          const int c1 = kTile * 16, each = nr * kTrRows;
          for (int c = 16 * max(0, -o0) + row + (nr == 2 ? st * kTrRows : 0); c < c1; c += each) {
            const int slot = c >> 4;
            uint4 *at = reinterpret_cast<uint4 *>(v_ptr(vs)) + ((c & 8) << 6) + slot * 8 + (c & 7);
            if (o0 + slot >= n) {
              *at = make_uint4(0, 0, 0, 0);
              continue;
            }
            const uint4 q = *at;
            // an exponent of all ones carries into the sign's place
            const uint32_t ones = (((q.x & 0x7f807f80u) + 0x00800080u) | ((q.y & 0x7f807f80u) + 0x00800080u) |
                                   ((q.z & 0x7f807f80u) + 0x00800080u) | ((q.w & 0x7f807f80u) + 0x00800080u)) &
                                  0x80008000u;
            if (ones) {
              uint32_t y[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((y[k] & 0x7f80u) == 0x7f80u) y[k] &= 0xffff0000u;
                if ((y[k] & 0x7f800000u) == 0x7f800000u) y[k] &= 0xffffu;
              }
              *at = make_uint4(y[0], y[1], y[2], y[3]);
              bad = true;
            }
          }
          if (bad) atomicMax(&v_bad[piece & 3], static_cast<uint32_t>(piece + 1));
          fence_proxy_async_smem();
          if (nr == 2) ok = softmax_barrier();
        }
        ok = ok && mbar_wait(smem_addr(&sf[sb]), static_cast<uint32_t>((is >> 1) & 1));
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if ((warp & 3) == 0 && lane == 0) {
          // S is done with the K tile, the P V of two tiles before with its V tile, and the last S
          // of the piece with the queries
          const int i = j - j0;
          if (NQ == 2) {
            mbar_arrive_n(smem_addr(&k_empty[(it0 + i) % kStages]), shares);
            if (i >= first + 2 * step) mbar_arrive_n(smem_addr(&v_empty[(it0 + i - 2 * step) % kStages]), shares);
          }
          if (j + step >= j1) mbar_arrive(smem_addr(q_empty));
        }
        if (!warp_valid) {  // no node in this warp's rows: what P holds there reaches no output
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&pf[sb]));
          continue;
        }
        tc_fence_after();
        float sv[64];
        {
          float a[32], c[32];
          tmem_ld32(tm + 64 * sb, a);
          tmem_ld32(tm + 64 * sb + 32, c);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            sv[e] = a[e];
            sv[32 + e] = c[e];
          }
        }
        if (tail) {
          const uint32_t s0 = static_cast<uint32_t>(see), s1 = static_cast<uint32_t>(see >> 32);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            sv[c] = (s0 >> c) & 1u ? sv[c] : -INFINITY;
            sv[32 + c] = (s1 >> c) & 1u ? sv[32 + c] : -INFINITY;
          }
        }
        float m4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], sv[c + e], sv[c + 4 + e]);
#pragma unroll
        for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], sv[60 + e]);
        const float mx = max3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
        const float m_new = fmaxf(m_run, mx * p.scale_log2);
        float corr = 1.f;
        bool resc = false;
        if (valid && m_new > m_run + kTrRescaleLog2) {
          corr = fast_exp2(m_run - m_new);  // 0 before the row's first seen key
          m_run = m_new;
          l_run *= corr;
          resc = j > j0 + first;
        }
        if (__any_sync(0xffffffffu, resc)) {
          // O must hold every P V before this tile's when it is scaled: the next S comes after them,
          // or, behind the piece's last S, a commit of their own.
          if (j + step < j1)
            ok = mbar_wait(smem_addr(&sf[sb ^ 1]), static_cast<uint32_t>(((is + 1) >> 1) & 1));
          else
            ok = mbar_wait(smem_addr(&pv_done[st]), static_cast<uint32_t>(pv & 1));
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 16) {
            uint32_t o[16];
            tmem_ld16(tm + kTrTmemO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
            tmem_st16(tm + kTrTmemO + c, o);
          }
        }
        // P = 2^(s - m) as bf16 hi + lo pairs into the S buffer's columns: hi the leading 8 bits of the
        // significand as they are, lo the rest rounded (to 2^-16 of the weight in all)
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;  // a row that has seen no key yet: P = 0
        const f2 scale2 = make_f2(p.scale_log2, p.scale_log2), neg2 = make_f2(neg_m, neg_m), minus = make_f2(-1.f, -1.f);
        f2 rs[4] = {{0}, {0}, {0}, {0}};
#pragma unroll
        for (int x = 0; x < kTile; x += 32) {  // 32 keys at a time, or the registers do not hold it all
          uint32_t ph[16], pl[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float v0, v1, e0, e1;
            split_f2(fma_f2(make_f2(sv[x + 2 * c], sv[x + 2 * c + 1]), scale2, neg2), v0, v1);
            v0 = fast_exp2(v0);
            v1 = fast_exp2(v1);
            const f2 v = make_f2(v0, v1);
            rs[c & 3] = add_f2(rs[c & 3], v);
            const uint32_t h0 = __float_as_uint(v0) & 0xffff0000u, h1 = __float_as_uint(v1) & 0xffff0000u;
            ph[c] = __byte_perm(h0, h1, 0x7632);
            split_f2(fma_f2(make_f2(__uint_as_float(h0), __uint_as_float(h1)), minus, v), e0, e1);
            pl[c] = pack_bf16(e0, e1);
          }
          tmem_st16(tm + 64 * sb + x, ph);
          tmem_st16(tm + 64 * sb + x + 16, pl);
        }
        float l0, l1;
        split_f2(add_f2(add_f2(rs[0], rs[1]), add_f2(rs[2], rs[3])), l0, l1);
        l_run += l0 + l1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&pf[sb]));
      }
      float f_own = 1.f, f_other = 0.f;
      if (ok) ok = mbar_wait(smem_addr(&o_full[st]), static_cast<uint32_t>(piece & 1));
      if (j0 + first + step < j1) ++pv;
      if ((warp & 3) == 0 && lane == 0 && ok) {  // every P V is done: the last two V tiles
        const int nt = j1 - j0, last = first + (nt - 1 - first) / step * step;
        if (NQ == 2 && first < nt) mbar_arrive_n(smem_addr(&v_empty[(it0 + last) % kStages]), shares);
        if (NQ == 2 && first + step < nt) mbar_arrive_n(smem_addr(&v_empty[(it0 + last - step) % kStages]), shares);
        if (first >= nt) mbar_arrive(smem_addr(q_empty));  // this stream had no tile
      }
      ok = __all_sync(0xffffffffu, ok);
      if (ok && nr == 1) {
        // Join the streams: each thread learns its row's (m, l) in the other one.  (Both threads of a
        // row have read the last joined piece's before this stream's O was free for this one.)
        s_ml[st * kTrRows + row] = make_float2(m_run, l_run);
        ok = softmax_barrier();
        const float2 x = s_ml[(st ^ 1) * kTrRows + row];
        if (x.y != 0.f) {
          const float M = l_run != 0.f ? fmaxf(m_run, x.x) : x.x;
          f_own = l_run != 0.f ? fast_exp2(m_run - M) : 0.f;
          f_other = fast_exp2(x.x - M);
          l_run = st == 0 ? fmaf(x.y, f_other, l_run * f_own) : fmaf(l_run, f_own, x.y * f_other);
          m_run = M;
        }
        if (ok) ok = mbar_wait(smem_addr(&o_full[st ^ 1]), static_cast<uint32_t>(piece & 1));
      }
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      // The piece's O: to the output if the piece is its whole sequence, else to its slot of the
      // workspace (a range has at most two cut pieces, its first and its last).  Streams that
      // share the row tile write half of the dims each.
      tc_fence_after();
      if (warp_valid) {
        bool bad = false;
        const int o1 = (j1 - 1) * kTile - ctx + kTile;  // the node at the slot behind the piece (j1 kTile may be 2^31)
        if (o1 > 0)  // every softmax warp's look at V came before its P, which came before this O
          bad = *reinterpret_cast<volatile uint32_t *>(&v_bad[piece & 3]) == static_cast<uint32_t>(piece + 1);
        const float inv = l_run != 0.f ? 1.f / l_run : 0.f;  // (NaN stays NaN)
        uint16_t *dst = p.out + ((static_cast<long long>(b) * p.T + t) * p.Hq + kv * p.G + g) * kHeadDim;
        float *mine = p.part + (((static_cast<long long>(w) * p.Hkv + kv) * p.R + r) * 2 + (j0 > 0 ? 0 : 1)) * kTrPartFloats;
        // 64 dims at a time, of both O where the streams share the rows: the end of a piece is time that
        // neither stream works (with 32 at a time ragged drafts took 113 us).
        const int c0 = nr == 1 ? 2 * st : 0, c1 = nr == 1 ? c0 + 2 : 4;
        const bool two = nr == 1 && j1 - j0 > 1;  // both streams have an O
        const uint32_t from = nr == 1 ? tmem + lane_base : tm;
        const float f0 = st == 0 ? f_own : f_other, f1 = st == 0 ? f_other : f_own;
#pragma unroll 1
        for (int c4 = c0; c4 < c1; c4 += 2) {
          float o[2][32];
          tmem_ld32(from + kTrTmemO + 32 * c4, o[0]);
          tmem_ld32(from + kTrTmemO + 32 * c4 + 32, o[1]);
          if (two) {
            float o1[2][32];
            tmem_ld32(from + kTrTmemO + kTrTmemStream + 32 * c4, o1[0]);
            tmem_ld32(from + kTrTmemO + kTrTmemStream + 32 * c4 + 32, o1[1]);
            tmem_wait_ld();
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int e = 0; e < 32; ++e) o[x][e] = fmaf(o1[x][e], f1, o[x][e] * f0);
          } else {
            tmem_wait_ld();
          }
          if (!walk.whole) {
#pragma unroll
            for (int e = 0; e < 64; ++e) mine[(32 * c4 + e) * kTrRows + row] = o[e >> 5][e & 31];
          } else if (valid) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t x[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                x[e] = pack_bf16(o[q >> 1][16 * (q & 1) + 2 * e] * inv, o[q >> 1][16 * (q & 1) + 2 * e + 1] * inv);
              store_32b(dst + 32 * c4 + 16 * q, x, p.out_wide);
            }
          }
        }
        if (bad && valid)
          add_nonfinite(p, b, t, kv, ctx, max(0, j0 * kTile - ctx), min(n, o1), 32 * c0, 32 * c1,
                        walk.whole ? dst : nullptr, mine + row, inv);
        if (!walk.whole && (nr == 2 || st == 0)) {
          mine[kHeadDim * kTrRows + row] = m_run;
          mine[(kHeadDim + 1) * kTrRows + row] = l_run;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {  // both streams' O have been read by a warp of each, or one by its own alone
        mbar_arrive(smem_addr(&o_free[st]));
        mbar_arrive(smem_addr(&o_free[nr == 1 ? st ^ 1 : st]));
      }
      it0 += j1 - j0;
      ++piece;
    }
    if (!ok && lane == 0) flag_error(p.err, GQA_DEVERR_TIMEOUT);
  }

  // ------------------------------------------------------------------ teardown
  __syncwarp();  // the MMA warps ran their loops on lane 0 alone
  tc_fence_before();
  __syncthreads();
  if (warp == kTrMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTrTmemCols);
  }
}

// ----------------------------------------------------------------------------------- merge
// out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k over the parts k of a cut sequence, in the order
// of the ranges, kChunk parts at a time with a running (M, sum, sum).  A CTA joins kDims dims of one
// (sequence, KV head, row tile); its first index is the sequence or, where there are more sequences
// than cuts, a boundary between ranges, whose CTA joins the sequence that it is the first to cut.  A
// warp takes kDims / 8 dims, a lane four rows of the column-major partials (512 contiguous bytes a
// load).  All loads of a chunk go out together; (m, l) pass through shared memory, where a thread
// takes a row and makes its weights for half of the chunk.  What to join follows from the lengths,
// which the attention kernel has waited for before it let this one start, so that is found before
// the wait.
//   Few cut sequences take 8 dims a CTA and 16 parts a chunk (8 tokens on one 4k sequence, 16 parts:
// 16.3 us the call, against 26.6 with one part after the other), many take 32 dims and 4 parts (8 x 32k
// single tokens, 64 joins of 3 to 4 parts: 160 us the call, against 178 with 8 dims).
constexpr int kTrMergeThreads = 256;
template <int kDims>
__global__ void __launch_bounds__(kTrMergeThreads, 2) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  constexpr int kPer = kDims / 8, kChunk = 16 / kPer;
  constexpr int kPitch = kDims + 8;  // of the output rows staged in shared memory
  static_assert(kChunk % 2 == 0 && kChunk <= 16, "a thread makes the weights of half a chunk");
  __shared__ __align__(16) float s_m[kChunk][kTrRows], s_l[kChunk][kTrRows], s_f[kChunk][kTrRows];
  __shared__ __align__(16) float s_corr[kTrRows], s_sum[2][kTrRows];
  __shared__ __align__(16) uint16_t s_out[kTrRows][kPitch];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = static_cast<int>(blockIdx.x) % (p.Hkv * p.R), index = static_cast<int>(blockIdx.x) / (p.Hkv * p.R);
  const int r = unit % p.R, kv = unit / p.R;
  const TreeCut all = tree_cut(p, lane);
  int b = 0, n = 0, w0 = 0, w1 = -1;
  if (!all.whole && all.ranges > 1) {
    int first = 0, at = 0;
    bool mine = true;
    if (p.merge_by_sequence) {
      b = index;
      const int per = (p.B + 31) / 32;
      first = __shfl_sync(0xffffffffu, all.lane_first, b / per);
      for (int x = b / per * per; x < b; ++x) first += tree_span(p, all, x);
    } else {
      at = all.begin(index + 1);
      mine = index + 1 < all.ranges;
      if (mine) tree_find(p, all, at, &b, &first);
    }
    if (mine) {
      n = tree_nodes(p, b, p.ctx_lens[b]);
      const int nt = tree_tiles(p, b);
      if (nt > 0 && r * p.Tt < n) {
        w0 = all.range_of(first);
        w1 = all.range_of(first + nt - 1);
        // one range, or another boundary is the first in the sequence: nothing to do here
        if (w0 == w1 || (!p.merge_by_sequence && w0 != index)) w1 = w0 - 1;
      }
    }
  }
  griddep_wait();  // the attention kernel's partials
  if (w1 < w0) return;
  const int rows = min(p.Tt, n - r * p.Tt) * p.G;  // of the row tile
  const bool live = 4 * lane < rows;
  const int d0 = kDims * static_cast<int>(blockIdx.y) + kPer * warp;
  const int row = tid & (kTrRows - 1), side = tid >> 7;  // of the weights
  float M = -INFINITY, L = 0.f;  // of `row`, alike on both sides
  float A[kPer][4];
#pragma unroll
  for (int e = 0; e < kPer; ++e)
#pragma unroll
    for (int k = 0; k < 4; ++k) A[e][k] = 0.f;
  auto part = [&](int w) {
    return p.part + ((static_cast<long long>(w) * p.Hkv * p.R + unit) * 2 + (w == w0 ? 1 : 0)) * kTrPartFloats + 4 * lane;
  };
  for (int wb = w0; wb <= w1; wb += kChunk) {
    const int parts = min(kChunk, w1 - wb + 1);
    float4 o[kChunk][kPer];
#pragma unroll
    for (int k = 0; k < kChunk; ++k)
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        o[k][e] = live && k < parts ? __ldcg(reinterpret_cast<const float4 *>(part(wb + k) + (d0 + e) * kTrRows))
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = warp; k < parts; k += 8) {
      const float *sp = part(wb + k);
      *reinterpret_cast<float4 *>(&s_m[k][4 * lane]) =
          live ? __ldcg(reinterpret_cast<const float4 *>(sp + kHeadDim * kTrRows)) : make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4 *>(&s_l[k][4 * lane]) =
          live ? __ldcg(reinterpret_cast<const float4 *>(sp + (kHeadDim + 1) * kTrRows)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    float m2 = M;
    for (int k = 0; k < parts; ++k)
      if (s_l[k][row] != 0.f) m2 = fmaxf(m2, s_m[k][row]);  // (l = 0: a part that saw none of the row's keys)
    float sum = 0.f;
    for (int k = side * (kChunk / 2); k < min(parts, (side + 1) * (kChunk / 2)); ++k) {
      const float l = s_l[k][row], f = l != 0.f ? fast_exp2(s_m[k][row] - m2) : 0.f;
      s_f[k][row] = f;
      sum = fmaf(l, f, sum);
    }
    s_sum[side][row] = sum;
    const float corr = M == -INFINITY ? 0.f : fast_exp2(M - m2);
    if (side == 0) s_corr[row] = corr;
    M = m2;
    __syncthreads();
    L = fmaf(L, corr, s_sum[0][row] + s_sum[1][row]);
    const float4 c4 = *reinterpret_cast<const float4 *>(&s_corr[4 * lane]);
    const float cc[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
    for (int e = 0; e < kPer; ++e)
#pragma unroll
      for (int k = 0; k < 4; ++k) A[e][k] *= cc[k];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) {
      if (k >= parts) break;
      const float4 f4 = *reinterpret_cast<const float4 *>(&s_f[k][4 * lane]);
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        // A part with weight 0 too: its O is finite, and adds nothing, unless a value that the row sees is not
        A[e][0] = fmaf(f4.x, o[k][e].x, A[e][0]);
        A[e][1] = fmaf(f4.y, o[k][e].y, A[e][1]);
        A[e][2] = fmaf(f4.z, o[k][e].z, A[e][2]);
        A[e][3] = fmaf(f4.w, o[k][e].w, A[e][3]);
      }
    }
    __syncthreads();  // before the next chunk's (m, l), and for the sums below
  }
  if (side == 0) s_corr[row] = L != 0.f ? 1.f / L : 0.f;
  __syncthreads();
  const float4 i4 = *reinterpret_cast<const float4 *>(&s_corr[4 * lane]);
  const float inv[4] = {i4.x, i4.y, i4.z, i4.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      s_out[4 * lane + k][kPer * warp + e] = static_cast<uint16_t>(pack_bf16(A[e][k] * inv[k], 0.f) & 0xffffu);
  __syncthreads();
  constexpr int kChunks = kDims / 8;  // of 16 bytes
  for (int x = tid; x < rows * kChunks; x += kTrMergeThreads) {
    const int y = x / kChunks, c = x % kChunks, tl = y / p.G, g = y - tl * p.G;
    *reinterpret_cast<uint4 *>(p.out + ((static_cast<long long>(b) * p.T + r * p.Tt + tl) * p.Hq + kv * p.G + g) * kHeadDim +
                               kDims * blockIdx.y + 8 * c) = *reinterpret_cast<const uint4 *>(&s_out[y][8 * c]);
  }
}

// --------------------------------------------------------------------------------- host side

namespace {

constexpr int kTrMaxDevices = 64;
std::atomic<int> g_tree_sms[kTrMaxDevices];  // 0: the kernels are not configured on the device yet

// First call on the current device: the attention kernel's shared memory, the SM count.
gqa_status_t tree_device(int device, int *sms) {
  if (device >= kTrMaxDevices) return GQA_ERR_UNSUPPORTED;
  *sms = g_tree_sms[device].load(std::memory_order_acquire);
  if (*sms > 0) return GQA_OK;
  int n = 0;
  if (cudaFuncSetAttribute(tree_attn_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeSmem<1>::kBytes) !=
          cudaSuccess ||
      cudaFuncSetAttribute(tree_attn_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize, TreeSmem<2>::kBytes) !=
          cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  g_tree_sms[device].store(n, std::memory_order_release);
  *sms = n;
  return GQA_OK;
}

int tree_row_tiles(const gqa_tree_desc_t &d) {
  const int per = kTrRows / (d.num_q_heads / d.num_kv_heads);
  return (d.tree_len + per - 1) / per;
}

gqa_status_t tree_check(const gqa_tree_desc_t &d) {
  const gqa_status_t st = check_cache_geometry(d.batch, d.num_q_heads, d.num_kv_heads, d.head_dim, d.tree_len,
                                               d.block_size, d.max_seq_len, d.num_cache_blocks);
  if (st != GQA_OK) return st;
  if (d.tree_len > GQA_MAX_TREE) return GQA_ERR_INVALID_ARG;
  // (grid sizes, and the numbers of the batch's tiles with their gaps, are int32)
  const long long tiles = static_cast<long long>(d.batch) * (capacity_tiles(d.max_seq_len) + kTrPieceCost);
  return static_cast<long long>(d.batch) * d.num_kv_heads * tree_row_tiles(d) > 0x7fffffffLL || tiles > 0x7fffffffLL
             ? GQA_ERR_UNSUPPORTED
             : GQA_OK;
}

// CTAs a range: one per KV head and row tile, or pair of row tiles.
int tree_units(const gqa_tree_desc_t &d) {
  const int r = tree_row_tiles(d);
  return d.num_kv_heads * (r > 1 ? (r + 1) / 2 : 1);
}
// Ranges of a call: as many as the GPU holds at once, a CTA per SM; where that leaves more than a
// tenth of it idle (many heads or row tiles), as many as fill two or three rounds, if that is better.
int tree_max_ranges(const gqa_tree_desc_t &d, int sms) {
  const long long slots = sms, units = tree_units(d);
  long long best = 1, best_rounds = (units + slots - 1) / slots;
  for (long long rounds = 1; rounds <= 3; ++rounds) {
    const long long w = slots * rounds / units;
    // of the slots of the rounds, the share that has work: w units / (rounds slots)
    if (w >= 1 && 10 * w * best_rounds > 11 * best * rounds) best = w, best_rounds = rounds;
  }
  // never more than the batch at full capacity could use
  long long most = static_cast<long long>(d.batch) * capacity_tiles(d.max_seq_len) / kTrMinTiles;
  most = most > d.batch ? most : d.batch;
  best = best < most ? best : most;
  return static_cast<int>(best < 1 ? 1 : best);
}
size_t tree_part_bytes(const gqa_tree_desc_t &d, int sms) {
  const int w = tree_max_ranges(d, sms);
  if (w == 1) return 256;  // nothing is cut
  return static_cast<size_t>(w) * d.num_kv_heads * tree_row_tiles(d) * 2 * kTrPartFloats * sizeof(float);
}

}  // namespace

}  // namespace gqa

using namespace gqa;

extern "C" gqa_status_t gqa_tree_prepare(int batch, int tree_len, const int32_t *parents, const int32_t *ctx_lens,
                                         const int32_t *counts, uint64_t *mask, int32_t *positions, int device,
                                         uint32_t *device_errors, void *stream) {
  if (batch < 1 || batch > GQA_MAX_BATCH || tree_len < 1 || tree_len > GQA_MAX_TREE) return GQA_ERR_INVALID_ARG;
  if (!parents || !ctx_lens || !mask || !positions) return GQA_ERR_INVALID_ARG;
  if (!aligned_to(parents, 4) || !aligned_to(ctx_lens, 4) || !aligned_to(counts, 4) || !aligned_to(mask, 8) ||
      !aligned_to(positions, 4) || !aligned_to(device_errors, 4))
    return GQA_ERR_INVALID_ARG;
  gqa_status_t st = check_device(device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(device);
  if (!guard.ok) return GQA_ERR_CUDA;
  const unsigned threads = static_cast<unsigned>((tree_len + 31) / 32 * 32);
  if (launch_pdl(tree_prepare_kernel, dim3(static_cast<unsigned>(batch)), dim3(threads), 0,
                 static_cast<cudaStream_t>(stream), parents, ctx_lens, counts, mask, positions, tree_len,
                 device_errors) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

extern "C" gqa_status_t gqa_tree_workspace_bytes(const gqa_tree_desc_t *desc, size_t *bytes) {
  if (!desc || !bytes) return GQA_ERR_INVALID_ARG;
  const gqa_tree_desc_t d = *desc;
  gqa_status_t st = tree_check(d);
  if (st != GQA_OK) return st;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  int sms = 0;
  st = tree_device(d.device, &sms);
  if (st != GQA_OK) return st;
  *bytes = tree_part_bytes(d, sms);
  return GQA_OK;
}

extern "C" gqa_status_t gqa_tree_attn(const gqa_tree_desc_t *desc, const void *q, const void *k_cache,
                                      const void *v_cache, const int32_t *page_table, const int32_t *ctx_lens,
                                      const int32_t *counts, const uint64_t *mask, void *out, void *workspace,
                                      uint32_t *device_errors, void *stream) {
  if (!desc) return GQA_ERR_INVALID_ARG;
  const gqa_tree_desc_t d = *desc;
  gqa_status_t st = tree_check(d);
  if (st != GQA_OK) return st;
  if (!q || !k_cache || !v_cache || !ctx_lens || !mask || !out || !workspace) return GQA_ERR_INVALID_ARG;
  const bool paged = d.block_size > 0;
  if (paged != (page_table != nullptr)) return GQA_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(out, 16) ||
      !aligned_to(workspace, 256) || !aligned_to(mask, 8) || !aligned_to(page_table, 4) || !aligned_to(ctx_lens, 4) ||
      !aligned_to(counts, 4) || !aligned_to(device_errors, 4))
    return GQA_ERR_INVALID_ARG;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  int sms = 0;
  st = tree_device(d.device, &sms);
  if (st != GQA_OK) return st;

  TreeParams p;
  memset(&p, 0, sizeof p);
  p.page_table = page_table;
  p.ctx_lens = ctx_lens;
  p.counts = counts;
  p.mask = mask;
  p.v_cache = static_cast<const uint16_t *>(v_cache);
  p.out = static_cast<uint16_t *>(out);
  p.part = static_cast<float *>(workspace);
  p.err = device_errors;
  p.B = d.batch;
  p.T = d.tree_len;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.G = d.num_q_heads / d.num_kv_heads;
  p.Tt = kTrRows / p.G;
  p.R = tree_row_tiles(d);
  p.words = (d.tree_len + 63) / 64;
  p.paged = paged ? 1 : 0;
  p.max_seq = d.max_seq_len;
  p.max_blocks = capacity_tiles(d.max_seq_len);
  p.num_blocks = paged ? d.num_cache_blocks : 0;
  p.W = tree_max_ranges(d, sms);
  p.out_wide = aligned_to(out, 32) ? 1 : 0;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(kHeadDim)));

  const long long rows = paged ? static_cast<long long>(d.num_cache_blocks) * kTile
                               : static_cast<long long>(d.batch) * d.max_seq_len;
  CUtensorMap tq, tk, tv;
  // queries viewed as [B][T][H_q][128]; box = 64 dims x G heads x Tt nodes x 1
  const cuuint64_t qdims[4] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(p.Hq),
                               static_cast<cuuint64_t>(p.T), static_cast<cuuint64_t>(p.B)};
  const cuuint64_t qstrides[3] = {static_cast<cuuint64_t>(kHeadDim) * 2, static_cast<cuuint64_t>(p.Hq) * kHeadDim * 2,
                                  static_cast<cuuint64_t>(p.T) * p.Hq * kHeadDim * 2};
  const cuuint32_t qbox[4] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(p.Tt), 1};
  if (!encode_bf16_map(&tq, 4, q, qdims, qstrides, qbox) || !make_cache_map(&tk, k_cache, p.Hkv, rows) ||
      !make_cache_map(&tv, v_cache, p.Hkv, rows))
    return GQA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool pairs = p.R > 1;
  p.merge_by_sequence = p.B <= p.W - 1;
  const long long joins = static_cast<long long>(p.merge_by_sequence ? p.B : p.W - 1) * p.Hkv * p.R;
  // the fewest dims a CTA with which the joins still run at once (two CTAs an SM), 8 to 32
  const int dims = joins * (kHeadDim / 8) <= 2LL * sms ? 8 : joins * (kHeadDim / 16) <= 2LL * sms ? 16 : 32;
  auto *merge = dims == 8 ? tree_merge_kernel<8> : dims == 16 ? tree_merge_kernel<16> : tree_merge_kernel<32>;
  if (launch_pdl(pairs ? tree_attn_kernel<2> : tree_attn_kernel<1>, dim3(static_cast<unsigned>(p.W * tree_units(d))),
                 dim3(kTrThreads), static_cast<size_t>(pairs ? TreeSmem<2>::kBytes : TreeSmem<1>::kBytes), s, tq, tk, tv,
                 p) != cudaSuccess ||
      (p.W > 1 && launch_pdl(merge, dim3(static_cast<unsigned>(joins), static_cast<unsigned>(kHeadDim / dims)),
                             dim3(kTrMergeThreads), 0, s, p) != cudaSuccess)) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}
