// Attention over prompts packed one behind the other (include/gqa_packed.h) on the 5th-generation tensor
// core.
//
// Rows.  Tt = 128 / G tokens and the G query heads of a KV head make the 128 rows of a tile, the M of
// every MMA; a unit of work is two such tiles, neighbours in one sequence, and the 128-key tiles that the
// later of the two sees.  Keys behind a row's last are masked by the row, those behind the unit's never
// loaded.
//
// Units are numbered from the one with the most key tiles to the one with the fewest, over all sequences and
// KV heads, and dealt to the CTAs, one an SM, to and fro; the numbering follows from the lengths, which are read on the
// device: the units with at least D key tiles are counted in closed form for each sequence.
//
// A CTA: a warp finds the units and tells the others, a TMA warp streams Q, K and V; two streams of four softmax
// warps hold a tile each and an MMA warp serves them in turn, so that one stream's softmax overlaps the other's
// products; a warp looks over the values that some rows must not see.  A stream's S = Q K^T (128 x 128) and its O += P V lie in tensor
// memory, P over S as bf16 pairs in two halves, the first multiplied while the second is made.  A softmax thread holds a
// row.  The maximum is raised lazily (by more than 2^8), so most tiles rescale nothing; S of a tile is issued behind P V of
// the one before, so a thread that sees S finds O at rest.
//   P is rounded to bf16 (at most 2^-8 of a weight) and the row divided by the sum of the weights as they were: over the
// keys that adds about as much to a row as the output's own rounding; a second term for what is cut, as the chunked
// prefill and the draft trees have, would add half to the products.
//
// Bounds and figures (a GB300 whose bf16 library products run at 1908 TFLOP/s in bursts, 1719 for seconds).  Two chunks
// of 6000 tokens over prefixes of 1500 to 2000, 64 query over 8 KV heads: 1030 us in short bursts, 1.74 PFLOP/s of
// products that a row needs (ncu: tensor pipe active 74 % of the time, issue 43 %); in long trains the card's power
// limit lowers the clock from 1.9 to 1.72 GHz and a call takes 1145 us, 0.91 of the rate for seconds.  16 prompts of 64 to
// 2000, 40 over 8 heads: 233 us, where the needed products alone are 139 and tiles on the diagonal make them 155 (S over all
// 128 keys, P V up to the last sixteen seen); a unit's first scores, last products and output wait for each other (0.9, 0.5 and 1.1 us
// of the 11 that a unit takes here), and the dealing leaves the slowest CTA 10 % behind the middle one.  One prompt of 150 tokens
// takes 8.4 us, latency.
//   Tried and slower or no faster: units taken as CTAs come free (16 prompts -0.5 %, 64 short ones +14 %, one of 3000 tokens
// +4 %), warps of their own for the output (16 prompts 267 us), P from the maximum of the tile before (longer code),
// output rows turned through shuffles (no gain), through shared memory (16 prompts 2 % slower) or copied from there by TMA
// (4 %), V in three stages, the issue of MMAs rolled over the streams (64 short prompts -4 %, the two chunks +6 %), S of the
// next unit before the other stream's last P V (no change); scores rounded before m is taken off them where m is beyond 2^26, so that
// scores of any size keep their largest (8 % on the 16 prompts, the code again).
#include <math.h>
#include <string.h>

#include <atomic>

#include "../../include/gqa_packed.h"
#include "divisor.cuh"
#include "op_args.h"
#include "pairmath.cuh"
#include "tc05.cuh"

namespace gqa {

struct PackedParams {
  const int32_t *q_offsets, *k_offsets;
  const uint16_t *v;
  uint16_t *out;
  uint32_t *err;
  long long v_stride;
  int B, Nq, Nk, Hq, Hkv, G, Tt;
  Divisor by_heads, by_unit;  // Hkv, 2 Tt
  int causal;
  int out_wide;  // `out` is 32-byte aligned
  float scale_log2;
};

namespace {

constexpr int kPkRows = 128;
constexpr int kPkKeys = 128;
constexpr int kPkMmaWarp = 8;
constexpr int kPkUnitWarp = 9;
constexpr int kPkProducerWarp = 10;
constexpr int kPkCheckWarp = 11;
constexpr int kPkThreads = 32 * 12;
constexpr int kPkKStages = 2, kPkVStages = 2;
constexpr int kPkPanelBytes = kPkRows * kHalfRowBytes;  // 64 dims of 128 rows: 16 KiB
constexpr int kPkTileBytes = 2 * kPkPanelBytes;
constexpr int kPkSlots = 4;  // units told ahead
// Tensor memory: a stream's S (128 columns; P in the first 64) and its O (128).
constexpr uint32_t kPkTmemStream = 256, kPkTmemO = 128, kPkTmemCols = 512;
constexpr float kPkRescaleLog2 = 8.f;
// Registers a thread: 168 at launch; the softmax warpgroups take what the third gives up.
constexpr int kPkRegsSoftmax = 200, kPkRegsOther = 104;
static_assert(2 * kPkRegsSoftmax + kPkRegsOther <= 3 * 168, "registers of the launch");

constexpr int kPkOffK = 2 * kPkTileBytes;
constexpr int kPkOffV = kPkOffK + kPkKStages * kPkTileBytes;
constexpr int kPkOffBar = kPkOffV + kPkVStages * kPkTileBytes;

// A place in a ring of N stages and the parity of its barriers' phase.
template <int N>
struct Ring {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void step() {
    if (++at == N) at = 0, phase ^= 1u;
  }
};

// A unit as it is told.
struct PackedUnit {
  int q0, k0;      // packed rows of the unit's first query and of its sequence's first key
  int tokens;      // queries of the unit, up to 2 Tt; 0: no unit is left
  int see0;        // keys that the first query sees (causal: each next one sees one more), may be negative
  int keys;        // m of the sequence
  int nt[2];       // key tiles of each stream's tile
  int steps[2];    // of the last one, sixteens of keys that some row sees
  int kv;
  uint32_t bad;    // a value that not all rows see, or none does, is not finite (known once unit_looked says so)
};

struct PackedShared {
  uint64_t k_full[kPkKStages], k_empty[kPkKStages], v_full[kPkVStages], v_clean[kPkVStages], v_empty[kPkVStages];
  uint64_t s_full[2], p_full[2][2], o_full[2], o_free[2], drain, q_full[2], q_empty[2];
  uint64_t unit_full[kPkSlots], unit_empty[kPkSlots], unit_looked[kPkSlots], unit_checked[kPkSlots][2];
  PackedUnit unit[kPkSlots];
  uint32_t tmem;
};
constexpr int kPkNumBars = 2 * kPkKStages + 3 * kPkVStages + 2 + 4 + 5 + 4 + 5 * kPkSlots;
constexpr int kPkSmemBytes = kPkOffBar + static_cast<int>(sizeof(PackedShared));
static_assert(kPkSmemBytes <= 227 * 1024, "shared memory of a CTA");

// True in one lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
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

// The larger sizes of two bf16 pairs, NaN where either is one; the signs mean nothing.
__device__ __forceinline__ uint32_t max_abs_bf16(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// Queries and keys of sequence b; n = 0 where the offsets of the queries, m = 0 where those of the keys are
// not in order.
struct PackedSeq {
  int q0, k0, n, m;
};
__device__ __forceinline__ PackedSeq packed_seq(const PackedParams &p, int b) {
  PackedSeq s = {0, 0, 0, 0};
  if (b >= p.B) return s;
  s.q0 = p.q_offsets[b];
  const int q1 = p.q_offsets[b + 1];
  s.k0 = p.k_offsets[b];
  const int k1 = p.k_offsets[b + 1];
  s.n = s.q0 >= 0 && q1 >= s.q0 && q1 <= p.Nq ? q1 - s.q0 : 0;
  s.m = s.k0 >= 0 && k1 >= s.k0 && k1 <= p.Nk ? k1 - s.k0 : 0;
  return s;
}
__device__ __forceinline__ int units_of(const PackedParams &p, const PackedSeq &s) {
  return static_cast<int>(p.by_unit.divide(static_cast<uint32_t>(s.n) + 2u * p.Tt - 1u));
}
// Units a KV head of a sequence of `all` units whose key tiles are at least D.
__device__ __forceinline__ int units_of_depth(const PackedParams &p, const PackedSeq &s, int all, int D) {
  if (D <= 0) return all;
  const int need = (D - 1) * kPkKeys + 1;  // keys that the unit's last query has to see
  if (s.m < need) return 0;
  if (!p.causal) return all;
  const int last = need - (s.m - s.n);  // queries, counted from the sequence's first, up to the unit's last
  if (last <= 0) return all;
  return last > s.n ? 0 : all - static_cast<int>(p.by_unit.divide(static_cast<uint32_t>(last - 1)));
}

// Finds units by their number, which grows from call to call.  Every lane of a warp alike; the lanes keep
// the first 32 sequences.
struct PackedWalk {
  PackedSeq mine;
  int mine_all;
  int all;             // units a KV head
  bool by_depth;       // numbered by their key tiles, else by their sequences
  int D, upto, above;  // units a KV head with at least D key tiles, and with more
  int base, before;    // the 32 sequences looked at, and units of exactly D tiles in those before them

  __device__ __forceinline__ int count(const PackedParams &p, int d, int lane) const {
    int c = units_of_depth(p, mine, mine_all, d);
    for (int b = 32 + lane; b < p.B; b += 32) {
      const PackedSeq s = packed_seq(p, b);
      c += units_of_depth(p, s, units_of(p, s), d);
    }
    return __reduce_add_sync(0xffffffffu, c);
  }
  // ctas: where one round takes all units their order does not matter.
  __device__ __forceinline__ void start(const PackedParams &p, int lane, int ctas) {
    mine = packed_seq(p, lane);
    mine_all = units_of(p, mine);
    unsigned most = static_cast<unsigned>(mine.m);
    for (int b = 32 + lane; b < p.B; b += 32) most = max(most, static_cast<unsigned>(packed_seq(p, b).m));
    all = count(p, 0, lane);
    by_depth = static_cast<long long>(all) * p.Hkv > ctas;
    D = by_depth ? static_cast<int>((__reduce_max_sync(0xffffffffu, most) + kPkKeys - 1) / kPkKeys) + 1 : 0;
    upto = by_depth ? 0 : all;
    above = base = before = 0;
  }
  // The unit of number `at` (a KV head's); false if there are fewer.
  __device__ __forceinline__ bool find(const PackedParams &p, int at, int lane, PackedSeq *seq, int *index) {
    if (at >= all) return false;
    if (at >= upto) {
      // the largest depth with more than `at` units: down in growing steps, then between the last two
      int hi = D - 1, lo = hi, step = 1, c = count(p, lo, lane), c_hi = upto;
      while (c <= at) {
        hi = lo - 1;
        c_hi = c;
        lo = max(0, lo - step);
        step *= 2;
        c = count(p, lo, lane);
      }
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2, x = count(p, mid, lane);
        if (x > at) lo = mid, c = x;
        else hi = mid - 1, c_hi = x;
      }
      D = lo;
      upto = c;
      above = c_hi;  // the count at lo + 1, where the search ended
      base = before = 0;
    }
    const int want = at - above;
    for (; base < p.B; base += 32) {
      const PackedSeq s = base == 0 ? mine : packed_seq(p, base + lane);
      const int mine_units = base == 0 ? mine_all : units_of(p, s);
      const int deeper = by_depth ? units_of_depth(p, s, mine_units, D + 1) : 0;
      const int c = units_of_depth(p, s, mine_units, D) - deeper;
      int sum = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      const int total = __shfl_sync(0xffffffffu, sum, 31);
      if (want >= before + total) {
        before += total;
        continue;
      }
      const int x = want - before;
      const int who = __ffs(__ballot_sync(0xffffffffu, sum > x)) - 1;
      // units of a sequence get deeper with their index: those of D tiles end where the deeper ones begin
      const int i = mine_units - deeper - c + (x - (sum - c));
      *index = __shfl_sync(0xffffffffu, i, who);
      seq->q0 = __shfl_sync(0xffffffffu, s.q0, who);
      seq->k0 = __shfl_sync(0xffffffffu, s.k0, who);
      seq->n = __shfl_sync(0xffffffffu, s.n, who);
      seq->m = __shfl_sync(0xffffffffu, s.m, who);
      return true;
    }
    return false;
  }
};

// Values of keys [from, to) of a row's sequence that are not finite, which the products left out, come to
// the row after all.
__device__ __noinline__ void packed_add_nonfinite(const PackedParams &p, int k0, int kv, int from, int to, uint16_t *out,
                                                  float inv) {
  for (int j = from; j < to; ++j) {
    const uint16_t *v = p.v + (k0 + j) * p.v_stride + kv * kHeadDim;
#pragma unroll 1
    for (int d = 0; d < kHeadDim; ++d) {
      const uint32_t y = v[d];
      if ((y & 0x7f80u) != 0x7f80u) continue;
      out[d] = static_cast<uint16_t>(pack_bf16(bf16_lo_to_float(out[d]) + bf16_lo_to_float(y) * inv, 0.f) & 0xffffu);
    }
  }
}

}  // namespace

__global__ void __launch_bounds__(kPkThreads, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PackedParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_addr(smem) & 1023u) != 0u) {  // a launch assumption broken: no work at all
    if (threadIdx.x == 0) flag_error(p.err, GQA_DEVERR_LAUNCH);
    return;
  }
  PackedShared &sh = *reinterpret_cast<PackedShared *>(smem + kPkOffBar);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  griddep_wait();
  if (warp == kPkMmaWarp) {
    tmem_alloc(smem_addr(&sh.tmem), kPkTmemCols);
    tmem_relinquish();
  } else if (warp == kPkCheckWarp) {
    uint64_t *bars = sh.k_full;
    for (int i = lane; i < kPkNumBars; i += 32) {
      uint64_t *bar = bars + i;
      int count = 1;
      if ((bar >= sh.p_full[0] && bar < sh.o_full) || (bar >= sh.o_free && bar < &sh.drain)) count = 4;
      if (bar >= sh.unit_empty && bar < sh.unit_looked) count = 11;  // every warp but the one that finds them
      mbar_init(smem_addr(bar), count);
    }
    fence_barrier_init();
    __syncwarp();
  } else if (warp == kPkProducerWarp && lane == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;

  auto k_ptr = [&](int s) { return smem_addr(smem) + kPkOffK + s * kPkTileBytes; };
  auto v_ptr = [&](int s) { return smem_addr(smem) + kPkOffV + s * kPkTileBytes; };
  // The unit told in a slot; false when a wait ran out.  Whoever has read a slot gives it back.
  auto take_unit = [&](const Ring<kPkSlots> &slot, PackedUnit &x) -> bool {
    if (!mbar_wait(smem_addr(&sh.unit_full[slot.at]), slot.phase)) return false;
    x = sh.unit[slot.at];
    return true;
  };
  bool ok = true;

  if (warp >= kPkMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPkRegsOther));
    if (warp == kPkUnitWarp) {
      // ---------------------------------------------------------------- units, ahead of the others
      if (blockIdx.x == 0)
        for (int b = lane; b < p.B; b += 32) {
          const int q0 = p.q_offsets[b], q1 = p.q_offsets[b + 1], k0 = p.k_offsets[b], k1 = p.k_offsets[b + 1];
          if (q0 < 0 || q1 < q0 || q1 > p.Nq || k0 < 0 || k1 < k0 || k1 > p.Nk) flag_error(p.err, GQA_DEVERR_SEQLEN);
        }
      const int c = static_cast<int>(blockIdx.x), W = static_cast<int>(gridDim.x);
      PackedWalk walk;
      walk.start(p, lane, W);
      Ring<kPkSlots> slot;
      for (int u = 0; ok; ++u, slot.step()) {
        const long long number = static_cast<long long>(u) * W + (u & 1 ? W - 1 - c : c);  // to and fro
        PackedUnit x = {};
        PackedSeq s;
        int index = 0;
        const uint32_t at = p.by_heads.divide(static_cast<uint32_t>(number));
        if (number < 0x7fffffffLL && walk.find(p, static_cast<int>(at), lane, &s, &index)) {
          const int t0 = index * 2 * p.Tt;
          x.q0 = s.q0 + t0;
          x.k0 = s.k0;
          x.tokens = min(2 * p.Tt, s.n - t0);
          x.see0 = p.causal ? t0 + 1 + s.m - s.n : s.m;
          x.keys = s.m;
          x.kv = static_cast<int>(static_cast<uint32_t>(number) - at * p.Hkv);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int rows = min(p.Tt, x.tokens - i * p.Tt);  // tokens of the tile
            const int sees = p.causal ? x.see0 + i * p.Tt + rows - 1 : s.m;
            x.nt[i] = rows > 0 && sees > 0 ? (sees + kPkKeys - 1) / kPkKeys : 0;
            x.steps[i] = x.nt[i] > 0 ? ((sees - 1) % kPkKeys) / 16 + 1 : 0;
          }
        }
        if (u >= kPkSlots) ok = mbar_wait(smem_addr(&sh.unit_empty[slot.at]), slot.phase ^ 1u);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          sh.unit[slot.at] = x;
          mbar_arrive(smem_addr(&sh.unit_full[slot.at]));
        }
        if (x.tokens == 0) break;
        // Behind the first query's last key a row of V is seen by some rows of the unit or, from the sequence's end to the last
        // sixteen that is multiplied, by none: P is 0 there, but 0 x inf is not.  Looked at here, ahead of time and in global
        // memory: shared memory is the MMAs' (a warp that looked at the tiles there took up to 5900 cycles a unit).
        const int nt = x.nt[1] > 0 ? x.nt[1] : x.nt[0], steps = x.nt[1] > 0 ? x.steps[1] : x.steps[0];
        const int first = max(x.see0, 0);
        const int last = min(nt > 0 ? (nt - 1) * kPkKeys + 16 * steps : 0, p.Nk - x.k0);
        constexpr int kAhead = 8;
        uint32_t most = 0;  // the largest sizes in its halves
        const uint16_t *row = p.v + (x.k0 + first + (lane >> 4)) * p.v_stride + x.kv * kHeadDim + 8 * (lane & 15);
        for (int left = last - first - (lane >> 4); left > 0; left -= 2 * kAhead) {
          uint4 y[kAhead];
#pragma unroll
          for (int i = 0; i < kAhead; ++i, row += 2 * p.v_stride)
            y[i] = 2 * i < left ? __ldg(reinterpret_cast<const uint4 *>(row)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < kAhead; ++i) most = max_abs_bf16(most, max_abs_bf16(max_abs_bf16(y[i].x, y[i].y), max_abs_bf16(y[i].z, y[i].w)));
        }
        most &= 0x7fff7fffu;
        bool bad = max(most & 0xffffu, most >> 16) >= 0x7f80u;
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
          if (bad) sh.unit[slot.at].bad = 1;
          mbar_arrive(smem_addr(&sh.unit_looked[slot.at]));
        }
      }
      if (!ok && lane == 0) flag_error(p.err, GQA_DEVERR_TIMEOUT);
    } else if (warp == kPkProducerWarp) {
      // ---------------------------------------------------------------- TMA
      if (lane == 0) {
        int it = 0, queries[2] = {0, 0};  // key tiles and loads of a stream's queries so far
        Ring<kPkKStages> ks;
        Ring<kPkVStages> vs;
        Ring<kPkSlots> slot;
        for (; ok; slot.step()) {
          PackedUnit x;
          ok = take_unit(slot, x);
          if (!ok || x.tokens == 0) break;
          mbar_arrive(smem_addr(&sh.unit_empty[slot.at]));
          const int nt = max(x.nt[0], x.nt[1]);
          for (int j = 0; j < nt; ++j, ++it, ks.step(), vs.step()) {
            const int row = x.k0 + j * kPkKeys;
            if (it >= kPkKStages) ok = mbar_wait(smem_addr(&sh.k_empty[ks.at]), ks.phase ^ 1u);
            if (!ok) break;
            const uint32_t kb = smem_addr(&sh.k_full[ks.at]), kd = k_ptr(ks.at);
            mbar_arrive_expect_tx(kb, kPkTileBytes);
            tma_load_3d(kd, &tmK, kb, 0, x.kv, row);
            tma_load_3d(kd + kPkPanelBytes, &tmK, kb, 64, x.kv, row);
            if (j == 0) {  // a stream's queries, once every S of the stream has read those before
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (!ok || x.nt[i] == 0) continue;
                if (queries[i] > 0) ok = mbar_wait(smem_addr(&sh.q_empty[i]), static_cast<uint32_t>((queries[i] - 1) & 1));
                if (!ok) continue;
                const uint32_t qb = smem_addr(&sh.q_full[i]), qd = smem_addr(smem) + i * kPkTileBytes;
                mbar_arrive_expect_tx(qb, 2u * 64u * 2u * static_cast<uint32_t>(p.G * p.Tt));
                tma_load_3d(qd, &tmQ, qb, 0, x.kv * p.G, x.q0 + i * p.Tt);
                tma_load_3d(qd + kPkPanelBytes, &tmQ, qb, 64, x.kv * p.G, x.q0 + i * p.Tt);
                ++queries[i];
              }
              if (!ok) break;
            }
            if (it >= kPkVStages) ok = mbar_wait(smem_addr(&sh.v_empty[vs.at]), vs.phase ^ 1u);
            if (!ok) break;
            const uint32_t vb = smem_addr(&sh.v_full[vs.at]), vd = v_ptr(vs.at);
            mbar_arrive_expect_tx(vb, kPkTileBytes);
            tma_load_3d(vd, &tmV, vb, 0, x.kv, row);
            tma_load_3d(vd + kPkPanelBytes, &tmV, vb, 64, x.kv, row);
          }
        }
        if (!ok) {
          flag_error(p.err, GQA_DEVERR_TIMEOUT);
          // Do not leave while copies into this CTA's shared memory may still be in flight: wait out every
          // phase that a load was issued for (tile `it` may have its K loads alone).
          for (int i = 0; i < 2; ++i)
            if (queries[i] > 0) (void)mbar_wait(smem_addr(&sh.q_full[i]), static_cast<uint32_t>((queries[i] - 1) & 1));
          for (int i = (it + 1 > kPkKStages ? it + 1 - kPkKStages : 0); i <= it; ++i)
            (void)mbar_wait(smem_addr(&sh.k_full[i % kPkKStages]), static_cast<uint32_t>((i / kPkKStages) & 1));
          for (int i = (it > kPkVStages ? it - kPkVStages : 0); i < it; ++i)
            (void)mbar_wait(smem_addr(&sh.v_full[i % kPkVStages]), static_cast<uint32_t>((i / kPkVStages) & 1));
        }
      }
    } else if (warp == kPkCheckWarp) {
      // ---------------------------------------------------------------- values that some rows must not see
      // Where such a value was found, rows of V behind the sequence's end are cleared in the tiles, and so is a
      // value before it that is not finite, which the epilogue gives to the rows that see it.
      Ring<kPkVStages> vs;
      Ring<kPkSlots> slot;
      for (; ok; slot.step()) {
        PackedUnit x;
        ok = __all_sync(0xffffffffu, take_unit(slot, x));
        if (!ok || x.tokens == 0) break;
        const int nt = max(x.nt[0], x.nt[1]);
        if (lane == 0) {
          if (x.nt[0] == 0) mbar_arrive(smem_addr(&sh.unit_checked[slot.at][0]));
          if (x.nt[1] == 0) mbar_arrive(smem_addr(&sh.unit_checked[slot.at][1]));
        }
        for (int j = 0; j < nt; ++j, vs.step()) {
          ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&sh.v_full[vs.at]), vs.phase));
          if (!ok) break;
          // rows from r0 on, to r2; the sequence's end
          const int r0 = max(0, max(x.see0, 0) - j * kPkKeys), r1 = x.keys - j * kPkKeys;
          const int r2 = j + 1 < nt ? kPkKeys : 16 * (x.nt[1] == nt ? x.steps[1] : x.steps[0]);
          bool bad = false;
          if (r0 < r2) {
            ok = __all_sync(0xffffffffu, mbar_wait(smem_addr(&sh.unit_looked[slot.at]), slot.phase));
            if (!ok) break;
            bad = *reinterpret_cast<volatile uint32_t *>(&sh.unit[slot.at].bad) != 0;
          }
          if (bad) {
            uint4 *tile = reinterpret_cast<uint4 *>(smem + kPkOffV + vs.at * kPkTileBytes);
            auto at = [&](int c) { return tile + ((c & 8) << 7) + (c >> 4) * 8 + (c & 7); };  // chunk: row, panel, 16 bytes
            for (int c = 16 * r0 + lane; c < 16 * r2; c += 32) {
              if (c >= 16 * r1) {
                *at(c) = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint32_t *z = reinterpret_cast<uint32_t *>(at(c));
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if ((z[k] & 0x7f80u) == 0x7f80u) z[k] &= 0xffff0000u;
                if ((z[k] & 0x7f800000u) == 0x7f800000u) z[k] &= 0xffffu;
              }
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&sh.v_clean[vs.at]));
            if (j + 1 == x.nt[0]) mbar_arrive(smem_addr(&sh.unit_checked[slot.at][0]));
            if (j + 1 == x.nt[1]) mbar_arrive(smem_addr(&sh.unit_checked[slot.at][1]));
          }
        }
        if (lane == 0) mbar_arrive(smem_addr(&sh.unit_empty[slot.at]));
      }
      if (!ok && lane == 0) flag_error(p.err, GQA_DEVERR_TIMEOUT);
    } else if (warp == kPkMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer
      // For each key tile, of stream 0 and then of stream 1: P V of the tile before, in two halves, and S, which
      // overwrites P; the tensor pipe runs what a thread issues in order.  One thread for both streams
      // keeps them half a tile apart: with an issuer each they fell into step, the tensor core idle while both
      // made their P (the two chunks took 1616 us then, 1328 with one).  A commit holds the pipe up, so
      // there is one to a stream and tile, and the softmax warps that see it give the tiles back.
      //   The whole warp walks, on values that are known to be alike in its lanes, so that descriptors are made in
      // uniform registers; one lane issues.
      constexpr uint32_t kIdS = idesc_bf16_f32(kPkRows, kPkKeys, false, false);
      constexpr uint32_t kIdO = idesc_bf16_f32(kPkRows, kHeadDim, false, true);
      const uint64_t qd0 = sdesc_sw128(smem_addr(smem), 16, 1024), kd0 = sdesc_sw128(k_ptr(0), 16, 1024),
                     vd0 = sdesc_sw128(v_ptr(0), kPkPanelBytes, 1024);
      //   The walk runs on across the units: a unit's last P V come right before the next unit's first S.
      Ring<kPkKStages> ks;                                 // of the tile at hand
      Ring<kPkVStages> vs;                                 // of the tile before
      Ring<kPkSlots> slot;
      int pj = 0, pn[2] = {0, 0}, ps[2] = {0, 0};          // the tile before: its place in its unit, that unit's tiles, the last one's steps
      uint32_t phase_p[2] = {0, 0}, phase_q[2] = {0, 0};   // P made, queries loaded so far (mod 2)
      uint32_t mine[2] = {0, 0};                           // units of a stream whose P V is all issued
      bool issued = false;
      for (; ok; slot.step()) {
        PackedUnit x;
        ok = __all_sync(0xffffffffu, take_unit(slot, x));
        if (!ok) break;
        const bool end = __reduce_max_sync(0xffffffffu, x.tokens) == 0;
        const int tiles[2] = {__reduce_max_sync(0xffffffffu, x.nt[0]), __reduce_max_sync(0xffffffffu, x.nt[1])};
        const int steps[2] = {__reduce_max_sync(0xffffffffu, x.steps[0]), __reduce_max_sync(0xffffffffu, x.steps[1])};
        if (!end && elect_one()) mbar_arrive(smem_addr(&sh.unit_empty[slot.at]));
        const int n0 = max(max(tiles[0], tiles[1]), end ? 1 : 0);  // (the last P V is issued at the end)
        // O += P V of the tile before, the sixteens of keys below `steps`
        auto issue_pv = [&](int st, uint64_t vd, int place, int steps, bool last) -> bool {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!mbar_wait(smem_addr(&sh.p_full[st][half]), phase_p[st])) return false;
            tc_fence_after();
            if (elect_one()) {
              const uint32_t tm = tmem + st * kPkTmemStream;
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (4 * half + k < steps)
                  umma_bf16_ts(tm + kPkTmemO, tm + 32 * half + 8 * k, vd + 128 * (4 * half + k), kIdO,
                               place > 0 || half > 0 || k > 0 ? 1u : 0u);
              if (half == 1 && last) umma_commit(smem_addr(&sh.o_full[st]));
            }
            __syncwarp();
          }
          phase_p[st] ^= 1;
          return true;
        };
        auto issue_s = [&](int st, uint64_t kd) {
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kHeadDim / 16; ++k)
              umma_bf16(tmem + st * kPkTmemStream, qd0 + st * (kPkTileBytes / 16) + (k >> 2) * (kPkPanelBytes / 16) + 2 * (k & 3),
                        kd + (k >> 2) * (kPkPanelBytes / 16) + 2 * (k & 3), kIdS, k > 0 ? 1u : 0u);
            umma_commit(smem_addr(&sh.s_full[st]));
          }
          __syncwarp();
        };
        auto o_free = [&](int st) {  // the O of the unit before has been read
          return mine[st] == 0 || mbar_wait(smem_addr(&sh.o_free[st]), (mine[st] - 1) & 1);
        };
        const int both = min(tiles[0], tiles[1]);
        for (int j = 0; j < n0;) {
          const bool pv = pj < max(pn[0], pn[1]);
          const uint64_t vd = vd0 + static_cast<uint64_t>(vs.at * (kPkTileBytes / 16));
          const uint64_t kd = kd0 + static_cast<uint64_t>(ks.at * (kPkTileBytes / 16));
          if (pv) ok = mbar_wait(smem_addr(&sh.v_clean[vs.at]), vs.phase);
          if (!ok) break;
          if (j == 0 || j >= both) {
            // The unit's first tile, before which come the last P V of the unit before, or one that a stream uses alone.
#pragma unroll
            for (int st = 0; st < 2; ++st)
              if (ok && pj < pn[st]) {
                const bool last = pj + 1 == pn[st];
                if (pj == 0) ok = o_free(st);
                ok = ok && issue_pv(st, vd, pj, last ? ps[st] : kPkKeys / 16, last);
                if (last) ++mine[st];
              }
            if (ok && !end) ok = mbar_wait(smem_addr(&sh.k_full[ks.at]), ks.phase);
#pragma unroll
            for (int st = 0; st < 2; ++st)
              if (ok && j < tiles[st]) {
                if (j == 0) {
                  ok = mbar_wait(smem_addr(&sh.q_full[st]), phase_q[st]);
                  phase_q[st] ^= 1;
                }
                tc_fence_after();
                if (ok) issue_s(st, kd);
                issued = true;
              }
          } else {  // both streams have P V and S of a tile in the middle
            ok = mbar_wait(smem_addr(&sh.k_full[ks.at]), ks.phase);
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              if (j == 1) ok = ok && o_free(st);
              ok = ok && issue_pv(st, vd, j - 1, kPkKeys / 16, false);
              if (!ok) break;
              issue_s(st, kd);
            }
          }
          if (!ok) break;
          pj = j;
          pn[0] = tiles[0];
          pn[1] = tiles[1];
          ps[0] = steps[0];
          ps[1] = steps[1];
          if (pv) vs.step();
          ks.step();
          ++j;
        }
        if (end) break;
      }
      if (!ok && lane == 0) flag_error(p.err, GQA_DEVERR_TIMEOUT);
      __syncwarp();
      if (issued) {  // nothing is deallocated while an MMA runs
        if (elect_one()) umma_commit(smem_addr(&sh.drain));
        if (!mbar_wait(smem_addr(&sh.drain), 0)) flag_error(p.err, GQA_DEVERR_TIMEOUT);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax warps of a stream
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPkRegsSoftmax));
    const int st = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const int tl = row / p.G, g = row - tl * p.G;
    const uint32_t tm = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + st * kPkTmemStream;
    uint32_t phase_s = 0, phase_o = 0;
    int it = 0;  // the CTA's key tiles before the unit
    Ring<kPkSlots> slot;
    for (; ok; slot.step()) {
      ok = mbar_wait(smem_addr(&sh.unit_full[slot.at]), slot.phase);
      const PackedUnit &x = sh.unit[slot.at];
      ok = __all_sync(0xffffffffu, ok);
      if (!ok || x.tokens == 0) break;
      const int nt = x.nt[st];
      const int token = st * p.Tt + tl;
      const bool valid = tl < p.Tt && token < x.tokens;
      const bool warp_valid = __any_sync(0xffffffffu, valid);
      const int sees = valid ? max(0, min(x.keys, x.see0 + (p.causal ? token : 0))) : 0;
      const int all_see = x.see0 + (p.causal ? st * p.Tt : 0);  // keys that every row of the tile sees
      // The unit's tiles are given back by the stream that has S and P V of a tile behind the other's: the later one, if
      // it has any tile (it has at least as many as the other then).
      const bool gives = (warp & 3) == 0 && lane == 0 && st == (x.nt[1] > 0 ? 1 : 0);
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < nt; ++j, phase_s ^= 1u) {
        ok = mbar_wait(smem_addr(&sh.s_full[st]), phase_s);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        if (gives) {
          mbar_arrive(smem_addr(&sh.k_empty[(it + j) % kPkKStages]));
          if (j > 0) mbar_arrive(smem_addr(&sh.v_empty[(it + j - 1) % kPkVStages]));
        }
        if ((warp & 3) == 0 && lane == 0 && j + 1 == nt) mbar_arrive(smem_addr(&sh.q_empty[st]));
        if (!warp_valid) {  // what P holds in these rows reaches no output
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(smem_addr(&sh.p_full[st][0]));
            mbar_arrive(smem_addr(&sh.p_full[st][1]));
          }
          continue;
        }
        tc_fence_after();
        float sv[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tm + 32 * c, sv[c]);
        tmem_wait_ld();
        if ((j + 1) * kPkKeys > all_see) {
          const int left = sees - j * kPkKeys;
#pragma unroll
          for (int c = 0; c < kPkKeys; c += 32) {
            const int here = min(max(left - c, 0), 32);
            const uint32_t seen = here == 32 ? 0xffffffffu : (1u << here) - 1;
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[c >> 5][e] = seen & (1u << e) ? sv[c >> 5][e] : -INFINITY;
          }
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          m4[c] = max3(sv[c][0], sv[c][1], sv[c][2]);
#pragma unroll
          for (int e = 3; e < 31; e += 2) m4[c] = max3(m4[c], sv[c][e], sv[c][e + 1]);
          m4[c] = fmaxf(m4[c], sv[c][31]);
        }
        const float m_new = max3(m_run, fmaxf(m4[0], m4[1]) * p.scale_log2, fmaxf(m4[2], m4[3]) * p.scale_log2);
        float corr = 1.f;
        bool resc = false;
        if (m_new > m_run + kPkRescaleLog2) {
          corr = fast_exp2(m_run - m_new);  // 0 before the row's first seen key
          m_run = m_new;
          l_run *= corr;
          resc = j > 0;
        }
        if (__any_sync(0xffffffffu, resc)) {
#pragma unroll 1
          for (int c = 0; c < kHeadDim; c += 32) {
            float o[32];
            tmem_ld32(tm + kPkTmemO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= corr;
            tmem_st32(tm + kPkTmemO + c, o);
          }
        }
        const float neg_m = m_run == -INFINITY ? 0.f : -m_run;  // a row that has seen no key yet: P = 0
        const f2 scale2 = make_f2(p.scale_log2, p.scale_log2), neg2 = make_f2(neg_m, neg_m);
        f2 rs[4] = {{0}, {0}, {0}, {0}};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t ph[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int at = 64 * half + 2 * c;
            float v0, v1;
            split_f2(fma_f2(make_f2(sv[at >> 5][at & 31], sv[at >> 5][(at & 31) + 1]), scale2, neg2), v0, v1);
            v0 = fast_exp2(v0);
            v1 = fast_exp2(v1);
            ph[c] = pack_bf16(v0, v1);
            rs[c & 3] = add_f2(rs[c & 3], make_f2(v0, v1));
          }
          tmem_st32(tm + 32 * half, ph);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_addr(&sh.p_full[st][half]));
        }
        float l0, l1;
        split_f2(add_f2(add_f2(rs[0], rs[1]), add_f2(rs[2], rs[3])), l0, l1);
        l_run += l0 + l1;
      }
      if (!ok) break;
      // ---------------------------------------------------------------- the unit's rows
      if (nt > 0) {
        ok = mbar_wait(smem_addr(&sh.o_full[st]), phase_o);
        phase_o ^= 1u;
        if (ok && gives) mbar_arrive(smem_addr(&sh.v_empty[(it + nt - 1) % kPkVStages]));
      }
      it += max(x.nt[0], x.nt[1]);
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      if (warp_valid) {
        const float inv = l_run != 0.f ? 1.f / l_run : 0.f;  // (NaN stays NaN)
        uint16_t *dst = p.out + (static_cast<long long>(x.q0 + token) * p.Hq + x.kv * p.G + g) * kHeadDim;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < kHeadDim; c += 32) {
          float o[32];
          tmem_ld32(tm + kPkTmemO + c, o);  // (not used where there was no tile)
          tmem_wait_ld();
          if (c == kHeadDim - 32 && nt > 0) {  // the next unit's P V may come
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&sh.o_free[st]));
          }
          if (valid) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t y[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                y[e] = l_run != 0.f ? pack_bf16(o[16 * i + 2 * e] * inv, o[16 * i + 2 * e + 1] * inv) : 0u;
              store_32b(dst + c + 16 * i, y, p.out_wide);
            }
          }
        }
        ok = mbar_wait(smem_addr(&sh.unit_checked[slot.at][st]), slot.phase);
        const bool bad = *reinterpret_cast<volatile uint32_t *>(&sh.unit[slot.at].bad) != 0;
        if (bad && valid && ok && l_run != 0.f) packed_add_nonfinite(p, x.k0, x.kv, max(0, x.see0), sees, dst, inv);
      } else if (nt > 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&sh.o_free[st]));
      }
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0) mbar_arrive(smem_addr(&sh.unit_empty[slot.at]));
    }
    if (!ok && lane == 0) flag_error(p.err, GQA_DEVERR_TIMEOUT);
  }

  // ------------------------------------------------------------------ teardown
  __syncwarp();  // the producer ran its loop on lane 0 alone
  tc_fence_before();
  __syncthreads();
  if (warp == kPkMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kPkTmemCols);
  }
}

// --------------------------------------------------------------------------------- host side

namespace {

constexpr int kPkMaxDevices = 64;
std::atomic<int> g_packed_sms[kPkMaxDevices];  // 0: the kernel is not configured on the device yet

gqa_status_t packed_device(int device, int *sms) {
  if (device >= kPkMaxDevices) return GQA_ERR_UNSUPPORTED;
  *sms = g_packed_sms[device].load(std::memory_order_acquire);
  if (*sms > 0) return GQA_OK;
  int n = 0;
  if (cudaFuncSetAttribute(packed_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPkSmemBytes) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  g_packed_sms[device].store(n, std::memory_order_release);
  *sms = n;
  return GQA_OK;
}

// Packed rows viewed as [N][H][128] with a stride of `stride` elements; box = 64 dims x heads x tokens.
bool packed_map(CUtensorMap *m, const void *base, int tokens, int heads, long long stride, int box_heads, int box_tokens) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(kHeadDim), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(kHeadDim) * 2, static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_tokens)};
  return encode_bf16_map(m, 3, base, dims, strides, box);
}

}  // namespace

}  // namespace gqa

using namespace gqa;

extern "C" gqa_status_t gqa_packed_attn(const gqa_packed_desc_t *desc, const void *q, const void *k, const void *v,
                                        const int32_t *q_offsets, const int32_t *k_offsets, void *out,
                                        uint32_t *device_errors, void *stream) {
  if (!desc) return GQA_ERR_INVALID_ARG;
  const gqa_packed_desc_t d = *desc;
  gqa_status_t st = check_cache_geometry(d.batch, d.num_q_heads, d.num_kv_heads, d.head_dim, 1, 0, 1, 0);
  if (st != GQA_OK) return st;
  if (d.num_queries < 1 || d.num_keys < 1) return GQA_ERR_INVALID_ARG;
  const long long dense_q = static_cast<long long>(d.num_q_heads) * kHeadDim, dense_k = static_cast<long long>(d.num_kv_heads) * kHeadDim;
  if ((d.q_stride && (d.q_stride < dense_q || d.q_stride % 8)) || (d.k_stride && (d.k_stride < dense_k || d.k_stride % 8)) ||
      (d.v_stride && (d.v_stride < dense_k || d.v_stride % 8)))
    return GQA_ERR_INVALID_ARG;
  if (static_cast<long long>(d.num_queries) * d.num_q_heads > 0x7fffffffLL ||
      static_cast<long long>(d.num_keys) * d.num_kv_heads > 0x7fffffffLL || dense_q > 0x7fffffffLL)
    return GQA_ERR_UNSUPPORTED;
  if (d.num_keys > 1 << 26) return GQA_ERR_UNSUPPORTED;  // a unit stays well within the limit of a wait (2 s)
  if (!q || !k || !v || !q_offsets || !out) return GQA_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(out, 16) || !aligned_to(q_offsets, 4) ||
      !aligned_to(k_offsets, 4) || !aligned_to(device_errors, 4))
    return GQA_ERR_INVALID_ARG;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  int sms = 0;
  st = packed_device(d.device, &sms);
  if (st != GQA_OK) return st;

  PackedParams p;
  memset(&p, 0, sizeof p);
  p.q_offsets = q_offsets;
  p.k_offsets = k_offsets ? k_offsets : q_offsets;
  p.v = static_cast<const uint16_t *>(v);
  p.v_stride = d.v_stride ? d.v_stride : dense_k;
  p.out = static_cast<uint16_t *>(out);
  p.err = device_errors;
  p.B = d.batch;
  p.Nq = d.num_queries;
  p.Nk = d.num_keys;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.G = d.num_q_heads / d.num_kv_heads;
  p.Tt = kPkRows / p.G;
  p.by_heads.set(p.Hkv);
  p.by_unit.set(2 * p.Tt);
  p.causal = d.causal ? 1 : 0;
  p.out_wide = aligned_to(out, 32) ? 1 : 0;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(kHeadDim)));
  CUtensorMap tq, tk, tv;
  if (!packed_map(&tq, q, p.Nq, p.Hq, d.q_stride ? d.q_stride : dense_q, p.G, p.Tt) ||
      !packed_map(&tk, k, p.Nk, p.Hkv, d.k_stride ? d.k_stride : dense_k, 1, kPkKeys) ||
      !packed_map(&tv, v, p.Nk, p.Hkv, p.v_stride, 1, kPkKeys))
    return GQA_ERR_CUDA;
  // units at most: every sequence ends one
  const long long units = (static_cast<long long>(p.Nq) / (2 * p.Tt) + p.B) * p.Hkv;
  if (launch_pdl(packed_attn_kernel, dim3(static_cast<unsigned>(units < sms ? units : sms)), dim3(kPkThreads),
                 static_cast<size_t>(kPkSmemBytes), static_cast<cudaStream_t>(stream), tq, tk, tv, p) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}
