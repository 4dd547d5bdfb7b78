// Attention for a tree of drafted tokens over a KV cache (include/gqa_tree.h) on the
// 5th-generation tensor core, and the tree's masks and positions.
//
// Rows.  The n_b nodes of a sequence and the G query heads of a KV head make n_b G rows that
// all read the same keys; a row tile is Tt = 128 / G nodes, 128 rows, the M of every MMA.  Every
// row sees the whole context, so the work is one pass over K and V per row tile; only the last
// tiles, which hold the nodes' own slots, are masked, by the bits of the node's mask.
//
// Work.  The batch's KV tiles (sequence-major, then KV head, then 64 tokens) are cut into W
// equal contiguous ranges whatever the sequence boundaries, so ragged batches and single long
// sequences both fill the GPU; the lengths are read on the device.  CTA (w, r) streams range w
// for row tile r; the row tiles of one range run side by side and share its tiles in L2.  A piece
// of a range that is a whole (sequence, KV head) segment writes its output rows; one that is
// cut leaves (O, m, l) in the workspace and tree_merge_kernel joins the parts in order.
//
// Attention CTA: as in prefill.cu.  A TMA warp streams K (2 stages) and V (3 stages) tiles; an
// MMA warp issues S = Q K^T into one of two tensor-memory buffers and O += P V, P read from
// tensor memory as bf16 hi + lo (rounding P to one bf16 would double the output's error: its
// 2^-9 relative error a weight is as large as the output's own rounding); four softmax warps
// hold a row a thread.  The maximum is raised lazily (by more than 2^8), so most tiles rescale
// nothing.  The pipeline runs on across the pieces of a range.
#include <math.h>
#include <string.h>

#include <atomic>

#include "../../include/gqa_tree.h"
#include "op_args.h"
#include "tc05.cuh"

namespace gqa {

struct TreeParams {
  const int32_t *page_table, *ctx_lens, *counts;
  const uint64_t *mask;
  const uint16_t *v_cache;
  uint16_t *out;
  float *part;                  // [W * R * 2][130][128]: O columns, m, l of a cut piece
  uint32_t *err;
  int B, T, Hq, Hkv, G, Tt, R;  // R row tiles of Tt nodes
  int words;                    // 64-bit words of a mask row
  int paged, max_seq, max_blocks, num_blocks;
  int W;                        // ranges the grid is sized for
  float scale_log2;
};

namespace {

constexpr int kTrKStages = 2;
constexpr int kTrVStages = 3;
constexpr int kTrSoftmaxWarps = 4;
constexpr int kTrThreads = 32 * (kTrSoftmaxWarps + 2);
constexpr int kTrProducerWarp = kTrSoftmaxWarps;
constexpr int kTrMmaWarp = kTrSoftmaxWarps + 1;
constexpr int kTrCtasPerSm = 2;
constexpr int kTrRows = 128;
// Tensor memory per CTA: two S buffers (64 fp32 columns each; P overwrites S as bf16 pairs, hi
// in the first 32 columns, lo in the next) and O (128 columns); two CTAs fill the SM's 512.
constexpr uint32_t kTrTmemCols = 256;
constexpr uint32_t kTrTmemO = 128;
constexpr float kTrRescaleLog2 = 8.f;

constexpr int kTrQBytes = 2 * kTrRows * kHalfRowBytes;  // 32 KiB: two 64-dim panels
constexpr int kTrTileBytes = 2 * kHalfTileBytes;         // 16 KiB: a K or V tile's two halves
constexpr int kTrOffK = kTrQBytes;
constexpr int kTrOffV = kTrOffK + kTrKStages * kTrTileBytes;
constexpr int kTrOffBar = kTrOffV + kTrVStages * kTrTileBytes;
// barriers: k_full[2], k_empty[2], v_full[3], v_empty[3], s_full[2], p_full[2], q_full, q_empty,
// pv_done, o_full, o_free, drain
constexpr int kTrNumBars = 2 * kTrKStages + 2 * kTrVStages + 2 + 2 + 6;
constexpr int kTrSmemBytes = kTrOffBar + 8 * kTrNumBars + 16;
constexpr int kTrPartFloats = (kHeadDim + 2) * kTrRows;
static_assert(kTrCtasPerSm * (kTrSmemBytes + 1024) <= 228 * 1024, "two CTAs must share an SM");
static_assert(kTrOffK % 1024 == 0 && kTrOffV % 1024 == 0 && kTrTileBytes % 1024 == 0, "swizzled tiles 1024-aligned");

// Nodes of sequence b, or -1 when its lengths are invalid.
__device__ __forceinline__ int tree_nodes(const TreeParams &p, int b, int ctx) {
  const int n = p.counts ? p.counts[b] : p.T;
  return (ctx >= 0 && n >= 0 && n <= p.T && static_cast<long long>(ctx) + n <= p.max_seq) ? n : -1;
}
// KV tiles of each segment of sequence b: those up to its last node's slot, none when it has no node.
__device__ __forceinline__ int tree_tiles(const TreeParams &p, int b) {
  const int ctx = p.ctx_lens[b], n = tree_nodes(p, b, ctx);
  return n > 0 ? (ctx + n + kTile - 1) / kTile : 0;
}

// Walks the segments a range [pos, end) of KV tiles covers.  Every warp of the CTA runs its own
// copy, all lanes alike.
struct TreeWalk {
  long long pos, end;  // tiles still to do
  long long seq0;      // first tile of sequence b
  int b, nt;           // sequence, its tiles a segment
  // of the piece at hand
  int kv, j0, j1;
  bool whole;          // the piece is its whole segment

  __device__ __forceinline__ void start(const TreeParams &p, long long begin, long long stop, int b0, long long s0) {
    pos = begin;
    end = stop;
    b = b0;
    seq0 = s0;
    nt = pos < end ? tree_tiles(p, b) : 0;
  }
  // The next piece; false when the range is done.
  __device__ __forceinline__ bool next(const TreeParams &p) {
    if (pos >= end) return false;
    while (pos >= seq0 + static_cast<long long>(nt) * p.Hkv) {
      seq0 += static_cast<long long>(nt) * p.Hkv;
      ++b;
      nt = tree_tiles(p, b);
    }
    const long long off = pos - seq0;
    kv = static_cast<int>(off / nt);
    j0 = static_cast<int>(off - static_cast<long long>(kv) * nt);
    const long long left = end - pos;
    j1 = left < nt - j0 ? j0 + static_cast<int>(left) : nt;
    whole = j0 == 0 && j1 == nt;
    pos += j1 - j0;
    return true;
  }
};

// The batch's KV tiles, and the sequence (and its first tile) that holds tile `at`: a warp sums
// its lanes' sequences, then looks into the lane that holds it.  All lanes get the same answer.
__device__ __forceinline__ long long tree_total(const TreeParams &p, int lane, long long *lane_first) {
  const int per = (p.B + 31) / 32, b0 = lane * per, b1 = min(p.B, b0 + per);
  long long sum = 0;
  for (int b = b0; b < b1; ++b) sum += static_cast<long long>(tree_tiles(p, b)) * p.Hkv;
  long long x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  *lane_first = x - sum;
  return __shfl_sync(0xffffffffu, x, 31);
}
__device__ __forceinline__ void tree_find(const TreeParams &p, int lane, long long lane_first, long long at, int *b,
                                          long long *seq0) {
  // the last lane whose first tile is <= at (lanes without tiles share their successor's first)
  const uint32_t le = __ballot_sync(0xffffffffu, lane_first <= at);
  const int owner = 31 - __clz(le);
  const int per = (p.B + 31) / 32;
  long long s = __shfl_sync(0xffffffffu, lane_first, owner);
  int x = owner * per;
  while (x + 1 < p.B) {
    const long long nxt = s + static_cast<long long>(tree_tiles(p, x)) * p.Hkv;
    if (nxt > at) break;
    s = nxt;
    ++x;
  }
  *b = x;
  *seq0 = s;
}

// Ranges in use: at least kTrMinTiles tiles each, so that small batches leave few partials.
constexpr int kTrMinTiles = 2;
__device__ __forceinline__ int tree_ranges(const TreeParams &p, long long total) {
  const long long most = (total + kTrMinTiles - 1) / kTrMinTiles;
  return static_cast<int>(most < p.W ? most : p.W);
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
__global__ void __launch_bounds__(kTrThreads, kTrCtasPerSm)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_addr(smem_raw) & 1023u) != 0u) {  // a launch assumption broken: no work at all
    if (threadIdx.x == 0) flag_error(p.err, GQA_DEVERR_LAUNCH);
    return;
  }
  uint8_t *smem = smem_raw;
  uint64_t *k_full = reinterpret_cast<uint64_t *>(smem + kTrOffBar);
  uint64_t *k_empty = k_full + kTrKStages;
  uint64_t *v_full = k_empty + kTrKStages;
  uint64_t *v_empty = v_full + kTrVStages;
  uint64_t *s_full = v_empty + kTrVStages;
  uint64_t *p_full = s_full + 2;
  uint64_t *q_full = p_full + 2;
  uint64_t *q_empty = q_full + 1;
  uint64_t *pv_done = q_full + 2;
  uint64_t *o_full = q_full + 3;
  uint64_t *o_free = q_full + 4;
  uint64_t *drain = q_full + 5;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(k_full + kTrNumBars);
  uint32_t *v_bad = tmem_slot + 1;  // a non-finite value in a node's V row of the piece at hand

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = static_cast<int>(blockIdx.x) % p.R, w = static_cast<int>(blockIdx.x) / p.R;

  if (tid == 0) {
    for (int i = 0; i < kTrNumBars; ++i) {
      uint64_t *bar = k_full + i;
      const bool from_softmax = bar == &p_full[0] || bar == &p_full[1] || bar == o_free;
      mbar_init(smem_addr(bar), from_softmax ? kTrSoftmaxWarps : 1);
    }
    *v_bad = 0;
    fence_barrier_init();
  }
  if (warp == kTrProducerWarp && lane == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == kTrMmaWarp) {
    tmem_alloc(smem_addr(tmem_slot), kTrTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // everything below may come from the preceding kernel
  griddep_launch_dependents();  // only tree_merge_kernel follows, and it waits

  // Sequences with invalid lengths: flagged, zeros in all their rows.
  for (int b = static_cast<int>(blockIdx.x); b < p.B; b += static_cast<int>(gridDim.x)) {
    const int ctx = p.ctx_lens[b];
    if (tree_nodes(p, b, ctx) >= 0) continue;
    if (tid == 0) flag_error(p.err, ctx < 0 ? GQA_DEVERR_POSITION : GQA_DEVERR_SEQLEN);
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + static_cast<long long>(b) * p.T * p.Hq * kHeadDim);
    const long long n = static_cast<long long>(p.T) * p.Hq * kHeadDim / 8;
    for (long long c = tid; c < n; c += kTrThreads) dst[c] = make_uint4(0, 0, 0, 0);
  }

  long long lane_first = 0;
  const long long total = tree_total(p, lane, &lane_first);
  const int ranges = tree_ranges(p, total);
  TreeWalk walk;
  {
    long long begin = 0, stop = 0, seq0 = 0;
    int b = 0;
    if (w < ranges) {
      begin = total * w / ranges;
      stop = total * (w + 1) / ranges;
      tree_find(p, lane, lane_first, begin, &b, &seq0);
    }
    walk.start(p, begin, stop, b, seq0);
  }
  uint8_t *const qs = smem;
  auto k_ptr = [&](int s) { return smem + kTrOffK + s * kTrTileBytes; };
  auto v_ptr = [&](int s) { return smem + kTrOffV + s * kTrTileBytes; };
  // Does row tile r have a node in sequence b?
  auto has_rows = [&](int b) { return r * p.Tt < tree_nodes(p, b, p.ctx_lens[b]); };

  if (warp == kTrProducerWarp) {
    // ------------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int it = 0, piece = 0;  // KV tiles and pieces so far: their stages and phases
      bool ok = true;
      while (ok && walk.next(p)) {
        if (!has_rows(walk.b)) continue;
        const int b = walk.b, kv = walk.kv;
        auto row_of = [&](int j) {
          if (!p.paged) return b * p.max_seq + j * kTile;
          const int pg = p.page_table[static_cast<long long>(b) * p.max_blocks + j];
          if (pg < 0 || pg >= p.num_blocks) {
            flag_error(p.err, GQA_DEVERR_PAGE);
            return -kTile;  // the whole box out of bounds: TMA fills zeros
          }
          return pg * kTile;
        };
        // the queries, once the last S of the piece before has read its own
        if (piece > 0) ok = mbar_wait(smem_addr(q_empty), static_cast<uint32_t>((piece - 1) & 1));
        if (!ok) break;
        mbar_arrive_expect_tx(smem_addr(q_full), 2u * 64u * 2u * static_cast<uint32_t>(p.G * p.Tt));
        tma_load_4d(smem_addr(qs), &tmQ, smem_addr(q_full), 0, kv * p.G, r * p.Tt, b);
        tma_load_4d(smem_addr(qs + kTrRows * kHalfRowBytes), &tmQ, smem_addr(q_full), 64, kv * p.G, r * p.Tt, b);
        ++piece;
        for (int j = walk.j0; j < walk.j1; ++j, ++it) {
          const int row = row_of(j);
          const int ks = it % kTrKStages, vs = it % kTrVStages;
          if (it >= kTrKStages) ok = mbar_wait(smem_addr(&k_empty[ks]), static_cast<uint32_t>((it / kTrKStages - 1) & 1));
          if (!ok) break;
          const uint32_t kb = smem_addr(&k_full[ks]), kd = smem_addr(k_ptr(ks));
          mbar_arrive_expect_tx(kb, kTrTileBytes);
          tma_load_3d(kd, &tmK, kb, 0, kv, row);
          tma_load_3d(kd + kHalfTileBytes, &tmK, kb, 64, kv, row);
          if (it >= kTrVStages) ok = mbar_wait(smem_addr(&v_empty[vs]), static_cast<uint32_t>((it / kTrVStages - 1) & 1));
          if (!ok) break;
          const uint32_t vb = smem_addr(&v_full[vs]), vd = smem_addr(v_ptr(vs));
          mbar_arrive_expect_tx(vb, kTrTileBytes);
          tma_load_3d(vd, &tmV, vb, 0, kv, row);
          tma_load_3d(vd + kHalfTileBytes, &tmV, vb, 64, kv, row);
        }
      }
      if (!ok) {
        flag_error(p.err, GQA_DEVERR_TIMEOUT);
        // Do not leave while copies into this CTA's shared memory may still be in flight: wait out
        // every phase that a load was issued for (tile `it` may have its K loads alone).
        if (piece > 0) (void)mbar_wait(smem_addr(q_full), static_cast<uint32_t>((piece - 1) & 1));
        for (int i = (it + 1 > kTrKStages ? it + 1 - kTrKStages : 0); i <= it; ++i)
          (void)mbar_wait(smem_addr(&k_full[i % kTrKStages]), static_cast<uint32_t>((i / kTrKStages) & 1));
        for (int i = (it > kTrVStages ? it - kTrVStages : 0); i < it; ++i)
          (void)mbar_wait(smem_addr(&v_full[i % kTrVStages]), static_cast<uint32_t>((i / kTrVStages) & 1));
      }
    }
  } else if (warp == kTrMmaWarp) {
    // ------------------------------------------------------------------ MMA issuer
    // Issue order within a piece: S_0, S_1, PV_0, S_2, PV_1, ..., PV_last.  S overwrites the buffer
    // that held the P of two tiles before; that P V was issued before it and the tensor pipe runs
    // them in order.
    if (lane == 0) {
      constexpr uint32_t kIdS = idesc_bf16_f32(kTrRows, kTile, false, false);
      constexpr uint32_t kIdO = idesc_bf16_f32(kTrRows, kHeadDim, false, true);
      const uint32_t qa = smem_addr(qs);
      int it = 0, piece = 0;
      bool ok = true;
      auto issue_pv = [&](int t, bool first) -> bool {
        const int pb = t & 1, s = t % kTrVStages;
        if (!mbar_wait(smem_addr(&v_full[s]), static_cast<uint32_t>((t / kTrVStages) & 1))) return false;
        if (!mbar_wait(smem_addr(&p_full[pb]), static_cast<uint32_t>((t >> 1) & 1))) return false;
        tc_fence_after();
        const uint32_t va = smem_addr(v_ptr(s));
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_bf16_ts(tmem + kTrTmemO, tmem + 64 * pb + 8 * k, sdesc_sw128(va + 2048 * k, kHalfTileBytes, 1024), kIdO,
                       (!first || k > 0) ? 1u : 0u);
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          umma_bf16_ts(tmem + kTrTmemO, tmem + 64 * pb + 32 + 8 * k, sdesc_sw128(va + 2048 * k, kHalfTileBytes, 1024),
                       kIdO, 1u);
        umma_commit(smem_addr(&v_empty[s]));
        umma_commit(smem_addr(pv_done));
        return true;
      };
      while (ok && walk.next(p)) {
        if (!has_rows(walk.b)) continue;
        ok = mbar_wait(smem_addr(q_full), static_cast<uint32_t>(piece & 1));
        for (int j = walk.j0; j < walk.j1 && ok; ++j, ++it) {
          const int s = it % kTrKStages, sb = it & 1;
          ok = mbar_wait(smem_addr(&k_full[s]), static_cast<uint32_t>((it / kTrKStages) & 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t ka = smem_addr(k_ptr(s));
#pragma unroll
          for (int k = 0; k < kHeadDim / 16; ++k)
            umma_bf16(tmem + 64 * sb, sdesc_sw128(qa + (k >> 2) * (kTrRows * kHalfRowBytes) + 32 * (k & 3), 16, 1024),
                      sdesc_sw128(ka + (k >> 2) * kHalfTileBytes + 32 * (k & 3), 16, 1024), kIdS, k > 0 ? 1u : 0u);
          umma_commit(smem_addr(&k_empty[s]));
          umma_commit(smem_addr(&s_full[sb]));
          if (j == walk.j1 - 1) umma_commit(smem_addr(q_empty));
          if (j > walk.j0) ok = issue_pv(it - 1, j - 1 == walk.j0);
          // O of the piece before must have been read before this piece's first P V
          if (j == walk.j0 && piece > 0 && ok) ok = mbar_wait(smem_addr(o_free), static_cast<uint32_t>((piece - 1) & 1));
        }
        if (ok) ok = issue_pv(it - 1, walk.j1 - walk.j0 == 1);
        if (ok) umma_commit(smem_addr(o_full));
        ++piece;
      }
      if (!ok) flag_error(p.err, GQA_DEVERR_TIMEOUT);
      if (it > 0) {  // nothing is deallocated while an MMA runs
        umma_commit(smem_addr(drain));
        if (!mbar_wait(smem_addr(drain), 0)) flag_error(p.err, GQA_DEVERR_TIMEOUT);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax warps
    const int row = warp * 32 + lane;
    const int tl = row / p.G, g = row - tl * p.G;
    const int t = r * p.Tt + tl;  // this row's node
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    int it = 0, piece = 0;
    bool ok = true;
    while (ok && walk.next(p)) {
      const int b = walk.b, j0 = walk.j0, j1 = walk.j1;
      const int ctx = p.ctx_lens[b], n = tree_nodes(p, b, ctx);
      if (r * p.Tt >= n) continue;
      const bool valid = tl < p.Tt && t < n;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const uint64_t *mrow = p.mask + (static_cast<long long>(b) * p.T + t) * p.words;
      // bits 64 x .. 64 x + 63 of the node's mask, none from n on
      auto mask_word = [&](int x) -> uint64_t {
        const int left = n - 64 * x;
        if (left <= 0) return 0ull;
        const uint64_t m = mrow[x];
        return left >= 64 ? m : m & ((1ull << left) - 1ull);
      };
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = j0; j < j1; ++j, ++it) {
        const int sb = it & 1;
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
          // node as 0 x inf; the epilogue gives it to those that do.
          const int vs = it % kTrVStages;
          ok = mbar_wait(smem_addr(&v_full[vs]), static_cast<uint32_t>((it / kTrVStages) & 1));
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          bool bad = false;
          for (int c = row; c < 2 * kTile * 8; c += kTrRows) {  // 16-byte chunks: half, row, chunk
            const int slot = (c >> 3) & (kTile - 1), node = o0 + slot;
            if (node < 0) continue;
            uint4 *at = reinterpret_cast<uint4 *>(v_ptr(vs)) + c;
            if (node >= n) {
              *at = make_uint4(0, 0, 0, 0);
              continue;
            }
            const uint4 x = *at;
            uint32_t y[4] = {x.x, x.y, x.z, x.w};
            bool hit = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((y[e] & 0x7f80u) == 0x7f80u) y[e] &= 0xffff0000u, hit = true;
              if ((y[e] & 0x7f800000u) == 0x7f800000u) y[e] &= 0xffffu, hit = true;
            }
            if (hit) {
              *at = make_uint4(y[0], y[1], y[2], y[3]);
              bad = true;
            }
          }
          if (bad) atomicMax(v_bad, static_cast<uint32_t>(piece + 1));
          fence_proxy_async_smem();
        }
        ok = mbar_wait(smem_addr(&s_full[sb]), static_cast<uint32_t>((it >> 1) & 1));
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (!warp_valid) {  // no node in this warp's rows: what P holds there reaches no output
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&p_full[sb]));
          continue;
        }
        tc_fence_after();
        float sv[64];
        {
          float a[32], c[32];
          tmem_ld32(tmem + lane_base + 64 * sb, a);
          tmem_ld32(tmem + lane_base + 64 * sb + 32, c);
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
        float m8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) m8[e] = fmaxf(sv[e], sv[e + 8]);
#pragma unroll
        for (int c = 16; c < 64; c += 8)
#pragma unroll
          for (int e = 0; e < 8; ++e) m8[e] = fmaxf(m8[e], sv[c + e]);
        const float mx =
            fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
        const float m_new = fmaxf(m_run, mx * p.scale_log2);
        float corr = 1.f;
        bool resc = false;
        if (valid && m_new > m_run + kTrRescaleLog2) {
          corr = fast_exp2(m_run - m_new);  // 0 before the row's first seen key
          m_run = m_new;
          l_run *= corr;
          resc = j > j0;
        }
        if (__any_sync(0xffffffffu, resc)) {
          // O must hold every P V before this tile's when it is scaled.  (S was issued after the P V
          // of two tiles before, so the parity wait is never more than one phase ahead.)
          ok = mbar_wait(smem_addr(pv_done), static_cast<uint32_t>((it - 1) & 1));
          if (!__all_sync(0xffffffffu, ok)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c4 = 0; c4 < 4; ++c4) {
            float o[32];
            tmem_ld32(tmem + lane_base + kTrTmemO + 32 * c4, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= corr;
            tmem_st32(tmem + lane_base + kTrTmemO + 32 * c4, o);
          }
        }
        // P = 2^(s - m) as bf16 hi + lo pairs into the S buffer's columns
        uint32_t ph[32], pl[32];
        float rs8[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;  // a row that has seen no key yet: P = 0
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float v0 = fast_exp2(fmaf(sv[2 * c], p.scale_log2, neg_m));
          const float v1 = fast_exp2(fmaf(sv[2 * c + 1], p.scale_log2, neg_m));
          rs8[c & 7] += v0 + v1;
          ph[c] = pack_bf16(v0, v1);
          pl[c] = pack_bf16(v0 - bf16_lo_to_float(ph[c]), v1 - bf16_hi_to_float(ph[c]));
        }
        tmem_st32(tmem + lane_base + 64 * sb, ph);
        tmem_st32(tmem + lane_base + 64 * sb + 32, pl);
        l_run += ((rs8[0] + rs8[1]) + (rs8[2] + rs8[3])) + ((rs8[4] + rs8[5]) + (rs8[6] + rs8[7]));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&p_full[sb]));
      }
      if (!ok) break;

      // The piece's O: to the output if the piece is its whole segment, else to its slot of the
      // workspace (a range has at most two cut pieces, its first and its last).
      ok = mbar_wait(smem_addr(o_full), static_cast<uint32_t>(piece & 1));
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (warp_valid) {
        bool bad = false;
        if (j1 * kTile > ctx) {
          // every softmax warp's look at V came before its P, which came before this O
          bad = *reinterpret_cast<volatile uint32_t *>(v_bad) == static_cast<uint32_t>(piece + 1);
        }
        const float inv = l_run != 0.f ? 1.f / l_run : 0.f;  // (NaN stays NaN)
        uint16_t *dst = p.out + ((static_cast<long long>(b) * p.T + t) * p.Hq + walk.kv * p.G + g) * kHeadDim;
        float *mine = p.part + (static_cast<long long>(blockIdx.x) * 2 + (j0 > 0 ? 0 : 1)) * kTrPartFloats;
#pragma unroll 1
        for (int c4 = 0; c4 < 4; ++c4) {
          float o[32];
          tmem_ld32(tmem + lane_base + kTrTmemO + 32 * c4, o);
          tmem_wait_ld();
          if (bad && valid) {
            // values of seen nodes that are not finite: p x inf for some p > 0
#pragma unroll 1
            for (int u = max(0, j0 * kTile - ctx); u < min(n, j1 * kTile - ctx); ++u) {
              if (!((mask_word(u >> 6) >> (u & 63)) & 1ull)) continue;
              const int slot = ctx + u;
              long long crow = static_cast<long long>(b) * p.max_seq + slot;
              if (p.paged) {
                const int pg = p.page_table[static_cast<long long>(b) * p.max_blocks + slot / kTile];
                if (pg < 0 || pg >= p.num_blocks) continue;
                crow = static_cast<long long>(pg) * kTile + (slot & (kTile - 1));
              }
              const uint32_t *v = reinterpret_cast<const uint32_t *>(p.v_cache + (crow * p.Hkv + walk.kv) * kHeadDim) + 16 * c4;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const uint32_t y = v[e];
                if ((y & 0x7f80u) == 0x7f80u) o[2 * e] += bf16_lo_to_float(y);
                if ((y & 0x7f800000u) == 0x7f800000u) o[2 * e + 1] += bf16_hi_to_float(y);
              }
            }
          }
          if (!walk.whole) {
#pragma unroll
            for (int e = 0; e < 32; ++e) mine[(32 * c4 + e) * kTrRows + row] = o[e];
          } else if (valid) {
            uint4 *d4 = reinterpret_cast<uint4 *>(dst + 32 * c4);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              d4[q] = make_uint4(pack_bf16(o[8 * q] * inv, o[8 * q + 1] * inv),
                                 pack_bf16(o[8 * q + 2] * inv, o[8 * q + 3] * inv),
                                 pack_bf16(o[8 * q + 4] * inv, o[8 * q + 5] * inv),
                                 pack_bf16(o[8 * q + 6] * inv, o[8 * q + 7] * inv));
          }
        }
        if (!walk.whole) {
          mine[kHeadDim * kTrRows + row] = m_run;
          mine[(kHeadDim + 1) * kTrRows + row] = l_run;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(o_free));
      ++piece;
    }
    if (!ok && lane == 0) flag_error(p.err, GQA_DEVERR_TIMEOUT);
  }

  // ------------------------------------------------------------------ teardown
  __syncwarp();  // the producer and MMA warps ran their loops on lane 0 alone
  tc_fence_before();
  __syncthreads();
  if (warp == kTrMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTrTmemCols);
  }
}

// ----------------------------------------------------------------------------------- merge
// One CTA per (segment, row tile, 16 dims); a thread takes four rows and a dim.  A segment that
// one range held whole is already written.  The parts are joined in the order of the ranges:
// out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k, kept as a running (M, sum, sum) pair.
constexpr int kTrMergeDims = 16;
constexpr int kTrMergeThreads = 32 * kTrMergeDims;
constexpr int kTrMergeAhead = 4;
__global__ void __launch_bounds__(kTrMergeThreads) tree_merge_kernel(const __grid_constant__ TreeParams p) {
  griddep_wait();  // the attention kernel's partials
  const int lane = threadIdx.x & 31;
  const int seg = static_cast<int>(blockIdx.x) / p.R, r = static_cast<int>(blockIdx.x) % p.R;
  const int b = seg / p.Hkv, kv = seg - b * p.Hkv;
  const int ctx = p.ctx_lens[b], n = tree_nodes(p, b, ctx);
  if (r * p.Tt >= n) return;
  long long lane_first = 0;
  const long long total = tree_total(p, lane, &lane_first);
  const int ranges = tree_ranges(p, total);
  const int per = (p.B + 31) / 32;
  long long first = __shfl_sync(0xffffffffu, lane_first, b / per);
  for (int x = b / per * per; x < b; ++x) first += static_cast<long long>(tree_tiles(p, x)) * p.Hkv;
  const int nt = tree_tiles(p, b);
  first += static_cast<long long>(kv) * nt;
  const int w0 = worker_of(total, ranges, first), w1 = worker_of(total, ranges, first + nt - 1);
  if (w0 == w1) return;
  const int rq = lane, d = kTrMergeDims * static_cast<int>(blockIdx.y) + static_cast<int>(threadIdx.x) / 32;
  if (4 * rq >= min(p.Tt, n - r * p.Tt) * p.G) return;  // rows past the tile's last node
  float M[4], L[4], A[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) M[k] = -INFINITY, L[k] = 0.f, A[k] = 0.f;
  for (int wb = w0; wb <= w1; wb += kTrMergeAhead) {
    float4 m[kTrMergeAhead], l[kTrMergeAhead], o[kTrMergeAhead];
#pragma unroll
    for (int e = 0; e < kTrMergeAhead; ++e) {
      const int w = wb + e;
      if (w > w1) continue;
      const float *sp = p.part + ((static_cast<long long>(w) * p.R + r) * 2 + (w == w0 ? 1 : 0)) * kTrPartFloats + 4 * rq;
      m[e] = __ldcg(reinterpret_cast<const float4 *>(sp + kHeadDim * kTrRows));
      l[e] = __ldcg(reinterpret_cast<const float4 *>(sp + (kHeadDim + 1) * kTrRows));
      o[e] = __ldcg(reinterpret_cast<const float4 *>(sp + d * kTrRows));
    }
#pragma unroll
    for (int e = 0; e < kTrMergeAhead; ++e) {
      if (wb + e > w1) continue;
      const float mm[4] = {m[e].x, m[e].y, m[e].z, m[e].w}, ll[4] = {l[e].x, l[e].y, l[e].z, l[e].w},
                  oo[4] = {o[e].x, o[e].y, o[e].z, o[e].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (ll[k] == 0.f) continue;  // a part that saw none of the row's keys
        const float m2 = fmaxf(M[k], mm[k]);
        const float f = fast_exp2(M[k] - m2), h = fast_exp2(mm[k] - m2);
        L[k] = fmaf(L[k], f, ll[k] * h);
        A[k] = fmaf(A[k], f, oo[k] * h);
        M[k] = m2;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int row = 4 * rq + k, tl = row / p.G, g = row - tl * p.G, t = r * p.Tt + tl;
    if (tl >= p.Tt || t >= n) continue;
    const float inv = L[k] != 0.f ? 1.f / L[k] : 0.f;
    p.out[((static_cast<long long>(b) * p.T + t) * p.Hq + kv * p.G + g) * kHeadDim + d] =
        static_cast<uint16_t>(pack_bf16(A[k] * inv, 0.f) & 0xffffu);
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
  if (cudaFuncSetAttribute(tree_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTrSmemBytes) != cudaSuccess ||
      cudaFuncSetAttribute(tree_attn_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                           cudaSharedmemCarveoutMaxShared) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  g_tree_sms[device].store(n, std::memory_order_release);
  *sms = n;
  return GQA_OK;
}

gqa_status_t tree_check(const gqa_tree_desc_t &d) {
  const gqa_status_t st = check_cache_geometry(d.batch, d.num_q_heads, d.num_kv_heads, d.head_dim, d.tree_len,
                                               d.block_size, d.max_seq_len, d.num_cache_blocks);
  if (st != GQA_OK) return st;
  return d.tree_len > GQA_MAX_TREE ? GQA_ERR_INVALID_ARG : GQA_OK;
}

int tree_row_tiles(const gqa_tree_desc_t &d) {
  const int per = kTrRows / (d.num_q_heads / d.num_kv_heads);
  return (d.tree_len + per - 1) / per;
}
int tree_max_ranges(const gqa_tree_desc_t &d, int sms) {
  const int w = kTrCtasPerSm * sms / tree_row_tiles(d);
  return w > 1 ? w : 1;
}
size_t tree_part_bytes(const gqa_tree_desc_t &d, int sms) {
  return static_cast<size_t>(tree_max_ranges(d, sms)) * tree_row_tiles(d) * 2 * kTrPartFloats * sizeof(float);
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
  p.max_blocks = (d.max_seq_len + kTile - 1) / kTile;
  p.num_blocks = paged ? d.num_cache_blocks : 0;
  p.W = tree_max_ranges(d, sms);
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
  if (launch_pdl(tree_attn_kernel, dim3(static_cast<unsigned>(p.W * p.R)), dim3(kTrThreads),
                 static_cast<size_t>(kTrSmemBytes), s, tq, tk, tv, p) != cudaSuccess ||
      launch_pdl(tree_merge_kernel, dim3(static_cast<unsigned>(p.B * p.Hkv * p.R), kHeadDim / kTrMergeDims),
                 dim3(kTrMergeThreads), 0, s, p) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}
