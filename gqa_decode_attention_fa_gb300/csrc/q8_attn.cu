// Attention of one new token a sequence over an 8-bit KV cache (include/gqa_q8.h).
//
// out = sum_j p_j vs_j vc_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = (q . kc_j) ks_j log2(e) / sqrt(128).
//
// Work.  The batch's tokens, in units of 16, sequence after sequence, are cut into W ranges of equal
// cost whatever the sequence boundaries; the lengths are read on the device.  A CTA streams a range for
// `hg` neighbouring KV heads: its eight warps take a head each, or share a head's units in turn.  A piece
// of a range that is a whole sequence writes its output rows, one that is cut leaves its normalised
// output, its maximum and its sum in the workspace for q8_merge_kernel.  (The two apart: beside a large maximum the
// logarithm of a sum has no bits left.)
//
// A warp works alone between the ends of its pieces: a ring of stages of its own in shared memory, filled by
// asynchronous 16-byte copies (16 tokens of K, of V and their scales a stage; rows in 16-byte chunks permuted by
// chunk ^ (row mod 8), so that no load below meets a bank conflict; what lies beyond the
// sequence is filled with zeros), and mma.sync with the G query heads as the N of both products, S^T = K q^T and
// O^T += V^T P^T.  The codes become binary16 exactly (two to a conversion); the order of the 128 dims in a
// product is free, so a lane takes 32 neighbouring bytes of a K row, and of V rows 16 neighbouring dims
// of its four tokens.
//   q is scaled to binary16's range by a power of two a row (exact but for elements 2^-29 below the
// largest).  The scale of K multiplies the score, that of V the weight: x = p vs 2^(m - E), rounded to
// binary16 (at most 2^-11 of each weight, where the output's own rounding is 2^-8) under a power of two 2^E of its own
// that follows the largest weight seen, so that neither p nor the scale can pass binary16's range: weights down
// to 2^-22 of the largest keep 11 bits, those below 2^-32 are lost.  The maximum m is raised lazily, where a score
// passes it by 8; sums are binary32.
//
// Bounds and figures (a GB300 that copies 6.77 TB/s; 40 query over 8 KV heads where nothing else is said).  A token's K and V
// of a head are 264 bytes, so the cache bounds long calls: 8 sequences of 32768 take 90 us (88 to 92 on different GPUs), 6.2 TB/s, 0.91 of the copy rate;
// one of 131072 with 64 query heads over int8 codes 50 us, 5.5 TB/s, where the fixed costs show: 5.5 us from the launch to the first products
// (1.7 of them the cut, the rest the first copies' way), 3 us from a range's last products to its partials, 6 us for the
// join of 38 parts a head.  32 sequences of 512 to 8192 in pages take 52 us, 5.4 TB/s.  One sequence of 256 takes 5.0 us on the
// device and 8.2 from one call to the next, which is the host's.  At the long calls neither the
// instruction issue (45 % used) nor the MMAs (16 %) is near a limit.
#include <float.h>
#include <math.h>
#include <string.h>

#include <atomic>

#include "q8.cuh"

namespace gqa {

struct Q8AttnParams {
  const uint16_t *q;
  const uint8_t *k_codes, *v_codes;
  const float *k_scale, *v_scale;
  const int32_t *page_table, *seq_lens;
  uint16_t *out;
  float *part;  // [W][Hkv][2] (G x 128 outputs, G maxima, G sums, 2 G unused) of cut pieces
  uint32_t *err;
  int B, Hq, Hkv, G;
  int hg;       // KV heads of a CTA
  int paged, max_seq, max_blocks, num_blocks;
  int W;        // ranges the grid is sized for
  int whole;    // a range is a sequence, W = B
  int merge_by_sequence;
  float scale_log2;
};

namespace {

constexpr int kQaWarps = 8;
constexpr int kQaThreads = 32 * kQaWarps;
constexpr int kQaUnit = 16;                              // tokens of a stage
constexpr int kQaStageBytes = 2 * kQaUnit * 128 + 2 * kQaUnit * 4;  // K, V, scales of K, of V
constexpr int kQaMaxRanges = 640;
constexpr int kQaPieceCost = 3;     // of a piece's end, in units of a warp
constexpr float kQaRaise = 8.f;     // log2: how far a score may pass m
constexpr float kQaMostLog2 = 14.f; // of x (binary16 holds 65504)
constexpr float kQaFreshLog2 = 8.f; // of the largest x when E is set
// Of 2^(m - E): a product p vs below 2^-150, which is 0 in binary32 and cannot be seen by E, is an x below 2^7 then.
constexpr float kQaUpMost = 157.f;

template <int NT>
struct Q8Smem {
  static constexpr int kStages = NT == 1 ? 3 : 6;
  static constexpr int kRing = kQaWarps * kStages * kQaStageBytes;
  static constexpr int kRow = kHeadDim + 4;  // floats of a head's row in the merge
  static constexpr int kMerge = kQaWarps * 8 * NT * (kRow + 2) * 4;
  static constexpr int kBytes = kRing > kMerge ? kRing : kMerge;
};

__device__ __forceinline__ int q8_units(const Q8AttnParams &p, int b) {
  const int n = p.seq_lens[b];
  return n > 0 && n <= p.max_seq ? (n - 1) / kQaUnit + 1 : 0;
}

// How the batch is cut: as for draft trees (tree.cu), in units of 16 tokens.  Behind each sequence but the
// last `gap` numbers are left out, the cost of a piece's end.
struct Q8Cut {
  int ranges, gap, each, more;
  bool whole;
  int lane_first;

  __device__ __forceinline__ int begin(int w) const { return w * each + min(w, more); }
  __device__ __forceinline__ int range_of(int x) const {
    const int wide = (each + 1) * more;
    return x < wide ? x / (each + 1) : more + (x - wide) / each;
  }
};
__device__ __forceinline__ Q8Cut q8_cut(const Q8AttnParams &p, int lane) {
  const int per = (p.B + 31) / 32, b0 = lane * per, b1 = min(p.B, b0 + per);
  int units = 0, seqs = 0, longest = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = q8_units(p, b);
    units += n;
    seqs += n > 0;
    longest = max(longest, n);
  }
  const int own_units = units, own_seqs = seqs;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, units, o), z = __shfl_up_sync(0xffffffffu, seqs, o);
    if (lane >= o) units += y, seqs += z;
  }
  const int all = __shfl_sync(0xffffffffu, units, 31), all_seqs = __shfl_sync(0xffffffffu, seqs, 31);
  longest = static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(longest)));
  const int wph = kQaWarps / p.hg;  // a warp's unit is 1 / wph of a range's
  Q8Cut c;
  c.ranges = all < 1 ? 0 : max(1, min(p.W, all / (2 * wph)));
  const int quarter = c.ranges > 0 ? all / c.ranges / 4 : 0;
  c.gap = min(quarter, kQaPieceCost * wph);
  c.whole = c.ranges > 0 && all_seqs <= p.W && longest <= all / c.ranges + c.gap * all_seqs / c.ranges + 2 * wph;
  if (c.whole) c.ranges = all_seqs;
  const int total = c.whole ? all_seqs : all + c.gap * max(0, all_seqs - 1);
  c.each = c.ranges > 0 ? total / c.ranges : 0;
  c.more = total - c.each * c.ranges;
  c.lane_first = c.whole ? seqs - own_seqs : units - own_units + c.gap * (seqs - own_seqs);
  return c;
}
__device__ __forceinline__ int q8_span(const Q8AttnParams &p, const Q8Cut &c, int b) {
  const int n = q8_units(p, b);
  return n < 1 ? 0 : c.whole ? 1 : n + c.gap;
}
// The sequence whose numbers (or the gap behind them) hold `at`, below their end, and its first number.
__device__ __forceinline__ void q8_find(const Q8AttnParams &p, const Q8Cut &c, int at, int *b, int *seq0) {
  const uint32_t le = __ballot_sync(0xffffffffu, c.lane_first <= at);
  const int owner = 31 - __clz(le);
  const int per = (p.B + 31) / 32;
  int s = __shfl_sync(0xffffffffu, c.lane_first, owner);
  int x = owner * per;
  while (x + 1 < p.B) {
    const int nxt = s + q8_span(p, c, x);
    if (nxt > at) break;
    s = nxt;
    ++x;
  }
  *b = x;
  *seq0 = s;
}

// Of 16 (or 4) bytes the first `bytes` copied, the others zero.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
// D = A(16x16, row) * B(16x8, col) + D, binary16 inputs, binary32 sums.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
__device__ __forceinline__ float power_of_two(int e) { return __int_as_float((e + 127) << 23); }  // -126 .. 127
__device__ __forceinline__ uint32_t word(const uint4 &x, int i) { return i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w; }

// Largest over the lanes of the same t (lane = 4 g + t).
__device__ __forceinline__ float max_over_g(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

}  // namespace

// NT: the heads of a KV head in eights.  Two CTAs an SM leave 128 threads' registers, so that CTAs of the merge start
// beside them and have found their parts by their end (one sequence of 4000 tokens 10.1 us; with 128 registers 10.8, with 96
// and three CTAs' room 10.6, and 8 sequences of 32k 99).
template <int FMT, int NT>
__global__ void __launch_bounds__(kQaThreads) __maxnreg__(NT == 1 ? 112 : 255) q8_attn_kernel(const __grid_constant__ Q8AttnParams p) {
  using Smem = Q8Smem<NT>;
  constexpr int kStages = Smem::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int groups = p.Hkv / p.hg, wph = kQaWarps / p.hg;
  const int w = static_cast<int>(blockIdx.x) / groups, h0 = (static_cast<int>(blockIdx.x) - w * groups) * p.hg;
  const int hl = warp % p.hg, share = warp / p.hg, kv = h0 + hl;

  griddep_wait();
  if (!p.whole && p.W > 1) griddep_launch_dependents();  // q8_merge_kernel follows, and it waits

  int pos, end, b, seq0, gap = 0;  // numbers of the range still to do; the sequence at hand and its first number
  if (p.whole) {
    b = w;
    pos = seq0 = 0;
    end = q8_units(p, b);
  } else {
    const Q8Cut cut = q8_cut(p, lane);
    pos = end = b = seq0 = 0;
    gap = cut.gap;
    if (w < cut.ranges) {
      pos = cut.begin(w);
      end = cut.begin(w + 1);
      q8_find(p, cut, pos, &b, &seq0);
      if (cut.whole) pos = seq0 = 0, end = q8_units(p, b);
    }
  }

  const uint32_t ring = smem_addr(smem_raw) + warp * kStages * kQaStageBytes;
  const int cp_row = lane >> 3, cp_chunk = lane & 7;
  const long long row_bytes = static_cast<long long>(p.Hkv) * kHeadDim;
  const uint8_t *const k_lane = p.k_codes + static_cast<long long>(kv) * kHeadDim + 16 * cp_chunk;
  const uint8_t *const v_lane = p.v_codes + static_cast<long long>(kv) * kHeadDim + 16 * cp_chunk;
  const float *const s_lane = (lane < 16 ? p.k_scale : p.v_scale) + kv;
  const uint32_t cp_dst0 = cp_row * 128 + ((cp_chunk ^ cp_row) << 4);        // rows cp_row and cp_row + 8
  const uint32_t cp_dst1 = cp_row * 128 + 512 + ((cp_chunk ^ (cp_row + 4)) << 4);  // cp_row + 4 and + 12

  while (pos < end) {
    int n = p.seq_lens[b], nu = q8_units(p, b);
    while (pos >= seq0 + nu) {  // on to the next sequence
      seq0 += nu > 0 ? nu + gap : 0;
      if (pos < seq0) pos = seq0;
      if (pos >= end) break;
      ++b;
      n = p.seq_lens[b];
      nu = q8_units(p, b);
    }
    if (pos >= end) break;
    const int j0 = pos - seq0, j1 = min(nu, j0 + end - pos);
    pos += j1 - j0;

    // The queries are asked for ahead of the copies, which they would wait behind.
    const uint16_t *const q_row = p.q + (static_cast<long long>(b) * p.Hq + kv * p.G + g) * kHeadDim + 32 * t;
    uint4 raw[NT][4];
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        raw[x][i] = 8 * x + g < p.G ? reinterpret_cast<const uint4 *>(q_row + 8 * x * kHeadDim)[i] : make_uint4(0, 0, 0, 0);

    // ------------------------------------------------------------- copies
    int pg_base = -1, pg = 0;  // the lane's page id among 32 from pg_base on
    auto issue = [&](int j, int stage) {
      if (j < j1) {
        const int tok = j * kQaUnit;
        long long crow;
        bool there = true;
        if (p.paged) {
          const int page = tok / kTile;
          if (pg_base < 0 || page >= pg_base + 32) {
            pg_base = page;
            const int at = page + lane;
            pg = at <= (n - 1) / kTile ? p.page_table[static_cast<long long>(b) * p.max_blocks + at] : 0;
            if (pg < 0 || pg >= p.num_blocks) {
              flag_error(p.err, GQA_DEVERR_PAGE);
              pg = -1;
            }
          }
          const int id = __shfl_sync(0xffffffffu, pg, page - pg_base);
          there = id >= 0;
          crow = (there ? static_cast<long long>(id) * kTile : 0) + (tok & (kTile - 1));
        } else {
          crow = static_cast<long long>(b) * p.max_seq + tok;
        }
        const int left = there ? n - tok : 0;  // tokens of the unit that there are; the others' rows are zero
        const uint32_t st = ring + stage * kQaStageBytes;
        const uint8_t *const kp = k_lane + crow * row_bytes, *const vp = v_lane + crow * row_bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = cp_row + 4 * i;
          const long long from = max(0, min(row, left - 1)) * row_bytes;
          const uint32_t dst = st + (i & 1 ? cp_dst1 : cp_dst0) + (i >> 1) * 1024, bytes = row < left ? 16u : 0u;
          cp_async16(dst, kp + from, bytes);
          cp_async16(dst + kQaUnit * 128, vp + from, bytes);
        }
        const int row = lane & 15;
        cp_async4(st + 2 * kQaUnit * 128 + 4 * lane, s_lane + (crow + max(0, min(row, left - 1))) * p.Hkv, row < left ? 4u : 0u);
      }
      cp_async_commit();
    };

    int jl = j0 + share;
#pragma unroll 1
    for (int s = 0; s < kStages - 1; ++s, jl += wph) issue(jl, s);  // on their way while the queries are made

    // ------------------------------------------------------------- the queries, as B of the first product
    uint32_t qf[NT][8][2];
    float qs1[NT][2], qs2[NT][2];  // of heads 2t, 2t + 1: together 2^-shift log2(e) / sqrt(128)
#pragma unroll
    for (int x = 0; x < NT; ++x) {
      const int head = 8 * x + g;
      const uint4 (&r)[4] = raw[x];
      uint32_t most = 0;  // the largest |q|, as bf16 bits
#pragma unroll
      for (int i = 0; i < 4; ++i)
        most = __vmaxu2(most, __vmaxu2(__vmaxu2(r[i].x & 0x7fff7fffu, r[i].y & 0x7fff7fffu),
                                       __vmaxu2(r[i].z & 0x7fff7fffu, r[i].w & 0x7fff7fffu)));
      most = max(most & 0xffffu, most >> 16);
      if (most >= 0x7f80u) {  // the largest finite one
        most = 0;
#pragma unroll 1
        for (int i = 0; i < 32; ++i) {
          const uint32_t y = head < p.G ? q_row[8 * x * kHeadDim + i] & 0x7fffu : 0u;
          if (y < 0x7f80u) most = max(most, y);
        }
      }
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = max(most, __shfl_xor_sync(0xffffffffu, most, 2));
      const int shift = most == 0 ? 0 : min(126, 14 - (static_cast<int>(most >> 7) - 127));
      const float f = power_of_two(shift);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint32_t y = word(r[i >> 2], i & 3);
        qf[x][i >> 1][i & 1] = pack_f16(bf16_lo_to_float(y) * f, bf16_hi_to_float(y) * f);
      }
      const int h1 = shift >> 1;
      const float a1 = power_of_two(-h1) * p.scale_log2, a2 = power_of_two(h1 - shift);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        qs1[x][e] = __shfl_sync(0xffffffffu, a1, (2 * t + e) * 4);
        qs2[x][e] = __shfl_sync(0xffffffffu, a2, (2 * t + e) * 4);
      }
    }

    float o[8][NT][4], m[NT][2], top[NT][2], l[NT][2], up[NT][2], lim[NT][2], wt[NT][2];
#pragma unroll
    for (int x = 0; x < NT; ++x) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][x][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[x][e] = 0.f;                         // 0 until a score is finite
        top[x][e] = -INFINITY;                 // m + 8
        up[x][e] = kQaUpMost;                  // m - E, kept for E: beside a large m, E would be too coarse
        l[x][e] = lim[x][e] = wt[x][e] = 0.f;  // lim: 2^(14 + E - m), wt: 2^((m - E) / 2)
      }
    }
    auto follow = [&](int x, int e, float d) {  // m or E has changed
      up[x][e] = d;
      lim[x][e] = fminf(fast_exp2(kQaMostLog2 - d), FLT_MAX);  // (a p vs that is infinite passes it)
      wt[x][e] = fast_exp2(0.5f * d);
    };

    int stage = 0;
    for (int j = j0 + share; j < j1; j += wph) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      issue(jl, stage == 0 ? kStages - 1 : stage - 1);  // the stage read last
      jl += wph;
      const uint32_t st = ring + stage * kQaStageBytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;

      float acc[NT][4];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[x][e] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t a = st + g * 128 + (((2 * t + i) ^ g) << 4);
        const uint4 ka = lds128(a), kb = lds128(a + 1024);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t a0, a1, a2, a3;
          codes_to_f16<FMT>(word(ka, c), a0, a2);
          codes_to_f16<FMT>(word(kb, c), a1, a3);
#pragma unroll
          for (int x = 0; x < NT; ++x) mma_f16(acc[x], a0, a1, a2, a3, qf[x][4 * i + c][0], qf[x][4 * i + c][1]);
        }
      }
      const uint32_t sc = st + 2 * kQaUnit * 128 + 4 * g;
      const float ks[2] = {lds_f32(sc), lds_f32(sc + 32)}, vs[2] = {lds_f32(sc + 64), lds_f32(sc + 96)};
      bool raise = false;
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          acc[x][e] = acc[x][e] * qs1[x][e & 1] * ks[e >> 1] * qs2[x][e & 1];
        }
      if (const int left = n - j * kQaUnit; left < kQaUnit) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (g + 8 * (e >> 1) >= left) acc[x][e] = -INFINITY;
      }
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) raise |= acc[x][e] > top[x][e & 1];
      bool far = false;  // m has risen so that 2^(m - E) is beyond what it may be
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mx = max_over_g(fmaxf(acc[x][e], acc[x][e + 2]));
            if (mx > top[x][e]) {  // (a head's result does not depend on the others)
              const bool first = top[x][e] == -INFINITY;  // nothing has been summed
              l[x][e] *= first ? 0.f : fast_exp2(m[x][e] - mx);
              follow(x, e, first ? kQaUpMost : up[x][e] + (mx - m[x][e]));
              m[x][e] = mx;
              top[x][e] = mx + kQaRaise;
              far |= up[x][e] > kQaUpMost;
            }
          }
      }
      float y[NT][4];
      raise = far;
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float pr = fast_exp2(acc[x][e] - m[x][e & 1]);
          l[x][e & 1] += pr;
          y[x][e] = pr * vs[e >> 1];
          raise |= fabsf(y[x][e]) > lim[x][e & 1];
          acc[x][e] = pr;
        }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // the largest p vs, by its logarithm: it may pass binary32's range where the result does not
            const float most = max_over_g(fmaxf(log2f(acc[x][e]) + log2f(fabsf(vs[0])), log2f(acc[x][e + 2]) + log2f(fabsf(vs[1]))));
            float fresh = fminf(up[x][e], kQaUpMost);
            if (most + fresh > kQaMostLog2 && most < INFINITY) fresh = kQaFreshLog2 - most;  // the largest x is about 2^8 then
            if (fresh < up[x][e]) {
              const float f = fast_exp2(fresh - up[x][e]);
              follow(x, e, fresh);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                o[i][x][e] *= f;
                o[i][x][e + 2] *= f;
              }
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          pb[x][r] = movmatrix_t(pack_f16(acc[x][2 * r] * wt[x][0] * vs[r] * wt[x][0],
                                          acc[x][2 * r + 1] * wt[x][1] * vs[r] * wt[x][1]));
      const uint32_t vb = st + kQaUnit * 128 + 2 * t * 128;
      const uint4 v0 = lds128(vb + ((g ^ (2 * t)) << 4)), v1 = lds128(vb + 128 + ((g ^ (2 * t + 1)) << 4)),
                  v2 = lds128(vb + 1024 + ((g ^ (2 * t)) << 4)), v3 = lds128(vb + 1152 + ((g ^ (2 * t + 1)) << 4));
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a0, a1, a2, a3;
          codes_to_f16<FMT>(__byte_perm(word(v0, c), word(v1, c), i ? 0x7362 : 0x5140), a0, a1);
          codes_to_f16<FMT>(__byte_perm(word(v2, c), word(v3, c), i ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
          for (int x = 0; x < NT; ++x) mma_f16(o[2 * c + i][x], a0, a1, a2, a3, pb[x][0], pb[x][1]);
        }
    }

    // ------------------------------------------------------------- the piece's end
    // Each warp's output over its own sum, then the warps of a head joined through shared memory.
    cp_async_wait<0>();
    __syncthreads();
    float *const rows = reinterpret_cast<float *>(smem_raw);
    constexpr int kHeads = 8 * NT;
    float *const ml = rows + kQaWarps * kHeads * Smem::kRow, *const sl = ml + kQaWarps * kHeads;  // maxima and sums
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[x][e];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        const int head = 8 * x + 2 * t + e;
        const float f = fast_exp2(-0.5f * up[x][e]);
        const float fl = sum != 0.f ? f / sum : 0.f;
        float *row = rows + (warp * kHeads + head) * Smem::kRow + 16 * g;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y0 = o[i][x][e] * f * fl, y1 = o[i][x][e + 2] * f * fl;
          *reinterpret_cast<float2 *>(row + 2 * i) = sum != 0.f ? make_float2(y0, y1) : make_float2(0.f, 0.f);
        }
        if (g == 0) {
          ml[warp * kHeads + head] = sum != 0.f ? m[x][e] : -INFINITY;  // nothing counts
          sl[warp * kHeads + head] = sum;
        }
      }
    __syncthreads();
    const bool whole = j0 == 0 && j1 == nu;
    for (int c = tid; c < p.hg * p.G * (kHeadDim / 4); c += kQaThreads) {
      const int d = 4 * (c & 31), hh = c >> 5, hq = hh / p.G, head = hh - hq * p.G;
      float M = -INFINITY, sum = 0.f;
      for (int s = 0; s < wph; ++s) M = fmaxf(M, ml[(s * p.hg + hq) * kHeads + head]);
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      const float mm = M == -INFINITY ? 0.f : M;
      for (int s = 0; s < wph; ++s) {
        const int from = (s * p.hg + hq) * kHeads + head;
        sum = fmaf(fast_exp2(ml[from] - mm), sl[from], sum);
      }
      const float inv = sum != 0.f ? 1.f / sum : 0.f;
      for (int s = 0; s < wph; ++s) {  // (weights of 1 in all: values near the largest number stay below it)
        const int from = (s * p.hg + hq) * kHeads + head;
        const float f = fast_exp2(ml[from] - mm) * sl[from] * inv;
        const float4 y = *reinterpret_cast<const float4 *>(rows + from * Smem::kRow + d);
        a.x = fmaf(f, y.x, a.x);
        a.y = fmaf(f, y.y, a.y);
        a.z = fmaf(f, y.z, a.z);
        a.w = fmaf(f, y.w, a.w);
      }
      const int h = h0 + hq;
      if (whole) {
        *reinterpret_cast<uint2 *>(p.out + (static_cast<long long>(b) * p.Hq + h * p.G + head) * kHeadDim + d) =
            make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
      } else {
        float *mine = p.part + ((static_cast<long long>(w) * p.Hkv + h) * 2 + (j0 > 0 ? 0 : 1)) * p.G * (kHeadDim + 4);
        *reinterpret_cast<float4 *>(mine + head * kHeadDim + d) = a;
        if (d == 0) {
          mine[p.G * kHeadDim + head] = M;
          mine[p.G * (kHeadDim + 1) + head] = sum;
        }
      }
    }
    __syncthreads();  // the ring is filled anew
  }

  for (int b = static_cast<int>(blockIdx.x); b < p.B; b += static_cast<int>(gridDim.x)) {  // sequences without tokens
    const int n = p.seq_lens[b];
    if (n > 0 && n <= p.max_seq) continue;
    if (n != 0 && tid == 0) flag_error(p.err, GQA_DEVERR_SEQLEN);
    uint4 *dst = reinterpret_cast<uint4 *>(p.out + static_cast<long long>(b) * p.Hq * kHeadDim);
    for (int c = tid; c < p.Hq * (kHeadDim / 8); c += kQaThreads) dst[c] = make_uint4(0, 0, 0, 0);
  }
}

// ------------------------------------------------------------------------------------ merge
// out = sum_k 2^(m_k - M) l_k o_k / sum_k 2^(m_k - M) l_k over the parts k of a cut sequence (m_k: maximum, l_k: sum, o_k: its
// normalised output), in the order of the ranges.  A CTA joins one (sequence, query head): warp x of kWarps takes the parts x, x +
// kWarps, ..., a lane four dims; the warps' sums are added in order.  One warp finds what to join: with all of them
// looking, the 32 ragged sequences above took 56.5 us.
template <int kWarps>
__global__ void __launch_bounds__(32 * kWarps) q8_merge_kernel(const __grid_constant__ Q8AttnParams p) {
  __shared__ float s_w[kQaMaxRanges];
  __shared__ float4 s_o[kWarps][32];
  __shared__ int s_what[3];  // sequence, first range, parts
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hq = static_cast<int>(blockIdx.x) % p.Hq, index = static_cast<int>(blockIdx.x) / p.Hq;
  const int kv = hq / p.G, head = hq - kv * p.G;
  // What to join follows from the lengths, which the attention kernel has waited for before it let this one start.
  if (warp == 0) {
    const Q8Cut all = q8_cut(p, lane);
    int b = 0, first = 0, w0 = 0, w1 = 0;
    if (!all.whole && all.ranges > 1 && (p.merge_by_sequence || index + 1 < all.ranges)) {
      if (p.merge_by_sequence) {
        b = index;
        const int per = (p.B + 31) / 32;
        first = __shfl_sync(0xffffffffu, all.lane_first, b / per);
        for (int x = b / per * per; x < b; ++x) first += q8_span(p, all, x);
      } else {
        q8_find(p, all, all.begin(index + 1), &b, &first);
      }
      const int nu = q8_units(p, b);
      if (nu > 0) {
        w0 = all.range_of(first);
        w1 = all.range_of(first + nu - 1);
        if (!p.merge_by_sequence && w0 != index) w1 = w0;  // another boundary is its first
      }
    }
    if (lane == 0) {
      s_what[0] = b;
      s_what[1] = w0;
      s_what[2] = w1 - w0 + 1;
    }
  }
  __syncthreads();
  const int b = s_what[0], w0 = s_what[1], parts = s_what[2];
  griddep_wait();  // the attention kernel's partials; without any, too, or this kernel could end before that one
  if (parts < 2) return;  // not cut, or joined by another CTA
  const long long each = static_cast<long long>(p.G) * (kHeadDim + 4);
  auto part = [&](int k) { return p.part + ((static_cast<long long>(w0 + k) * p.Hkv + kv) * 2 + (k == 0 ? 1 : 0)) * each; };
  constexpr int kAhead = 8;
  float4 y[kAhead];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + i * kWarps;
      y[i] = k < parts ? __ldcg(reinterpret_cast<const float4 *>(part(k) + head * kHeadDim + 4 * lane))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  fetch(warp);
  if (warp == 0) {  // the weights, 1 in all, so that values near the largest number stay below it
    constexpr int kHeld = 2;  // of a lane's parts in registers
    float x[kHeld], l[kHeld];
    auto max_of = [&](int k) { return __ldcg(part(k) + p.G * kHeadDim + head); };
    auto sum_of = [&](int k) { return __ldcg(part(k) + p.G * (kHeadDim + 1) + head); };
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      x[i] = lane + 32 * i < parts ? max_of(lane + 32 * i) : -INFINITY;
      l[i] = lane + 32 * i < parts ? sum_of(lane + 32 * i) : 0.f;
    }
    float M = fmaxf(x[0], x[1]);
    for (int k = lane + 32 * kHeld; k < parts; k += 32) M = fmaxf(M, s_w[k] = max_of(k));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) sum += x[i] = fast_exp2(x[i] - M) * l[i];
    for (int k = lane + 32 * kHeld; k < parts; k += 32) sum += s_w[k] = fast_exp2(s_w[k] - M) * sum_of(k);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (lane + 32 * i < parts) s_w[lane + 32 * i] = x[i] * inv;
    for (int k = lane + 32 * kHeld; k < parts; k += 32) s_w[k] *= inv;
  }
  __syncthreads();
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = warp; k0 < parts; k0 += kAhead * kWarps) {
    if (k0 > warp) fetch(k0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int k = k0 + i * kWarps;
      if (k >= parts) break;
      const float f = s_w[k];
      a.x = fmaf(f, y[i].x, a.x);
      a.y = fmaf(f, y[i].y, a.y);
      a.z = fmaf(f, y[i].z, a.z);
      a.w = fmaf(f, y[i].w, a.w);
    }
  }
  s_o[warp][lane] = a;
  __syncthreads();
  if (warp != 0) return;
  for (int x = 1; x < kWarps; ++x) {
    const float4 y = s_o[x][lane];
    a.x += y.x, a.y += y.y, a.z += y.z, a.w += y.w;
  }
  *reinterpret_cast<uint2 *>(p.out + (static_cast<long long>(b) * p.Hq + hq) * kHeadDim + 4 * lane) =
      make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
}

// --------------------------------------------------------------------------------- host side

namespace {

constexpr int kQaMaxDevices = 64;
std::atomic<int> g_qa_sms[kQaMaxDevices];  // 0: the kernels are not configured on the device yet

template <int FMT, int NT>
cudaError_t qa_configure() {
  return cudaFuncSetAttribute(q8_attn_kernel<FMT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Q8Smem<NT>::kBytes);
}
gqa_status_t qa_device(int device, int *sms) {
  if (device >= kQaMaxDevices) return GQA_ERR_UNSUPPORTED;
  *sms = g_qa_sms[device].load(std::memory_order_acquire);
  if (*sms > 0) return GQA_OK;
  int n = 0;
  if (qa_configure<GQA_Q8_E4M3, 1>() != cudaSuccess || qa_configure<GQA_Q8_E4M3, 2>() != cudaSuccess ||
      qa_configure<GQA_Q8_INT8, 1>() != cudaSuccess || qa_configure<GQA_Q8_INT8, 2>() != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  g_qa_sms[device].store(n, std::memory_order_release);
  *sms = n;
  return GQA_OK;
}

// How a call of this geometry is laid out over the SMs.
struct QaLayout {
  int hg, W;
  bool whole;
};
// A CTA to a sequence and KV head, its eight warps sharing the tokens, and nothing to join, where no sequence can be
// long: 5 ns a token against 3 to 8 us for cuts, their ends and the merge.  (8 KV heads, us whole / cut: one sequence of
// 500 tokens 7.0 / 8.7, of 700 8.2 / 9.0, of 850 9.0 / 8.8, of 1015 9.8 / 8.4; 4 of up to 1015 8.9 / 11.8; 16 of up to 1015
// 9.6 / 15.0, of up to 1500 12.2 / 15.5, of up to 2500 18.7 / 19.5; 64 of up to 2500 42.8 / 40.6; 200 of up to 2500 96.9 / 97.7.)
// The host knows the capacity alone, so short sequences in a cache for long ones are cut (unless the lengths let the device
// take them whole): 16 of 1000 tokens take 12.3 us in a cache for 2048 tokens and 18.8 in one for 32768.
constexpr int kQaWholeTokensOne = 768;  // of a single sequence
constexpr int kQaWholeTokens = 1024;
constexpr int kQaWholeTokensMany = 2560, kQaMany = 128;  // where there are as many sequences and heads
// KV heads of a CTA where sequences are cut: one, so that few parts are to be joined, but in wide caches, whose rows are
// better read, and whose scales lie 32 bytes to eight heads (8 KV heads, 8 x 32k tokens: 92.6 us with 1, 93.0 with 2, 93.6
// with 4, 99 with 8; one 128k sequence 52 / 56 / 59 / 69; 16 KV heads, 2 x 30k: 50 / 50 / 51 / 55; 32, 4 x 8k: 66 / 60 / 54 / 52).
QaLayout qa_layout(const gqa_q8_desc_t &d, int sms) {
  QaLayout y;
  const int G = d.num_q_heads / d.num_kv_heads;
  y.whole = d.max_seq_len <= (d.batch == 1 ? kQaWholeTokensOne : kQaWholeTokens) ||
            (d.max_seq_len <= kQaWholeTokensMany && static_cast<long long>(d.batch) * d.num_kv_heads >= kQaMany);
  y.hg = 1;
  if (!y.whole)
    while (y.hg < kQaWarps && d.num_kv_heads % (2 * y.hg) == 0 && d.num_kv_heads / y.hg > (d.num_kv_heads < 32 ? 8 : 4))
      y.hg *= 2;
  const long long units = d.num_kv_heads / y.hg, slots = static_cast<long long>(sms) * (G > 8 ? 1 : 2);
  if (y.whole) {
    y.W = d.batch;
    return y;
  }
  long long best = 1, best_rounds = (units + slots - 1) / slots;
  for (long long rounds = 1; rounds <= 3; ++rounds) {
    const long long w = slots * rounds / units;
    if (w >= 1 && 10 * w * best_rounds > 11 * best * rounds) best = w, best_rounds = rounds;
  }
  const long long most = static_cast<long long>(d.batch) * ((d.max_seq_len - 1) / kQaUnit + 1);
  best = best < most ? best : most;
  best = best < kQaMaxRanges ? best : kQaMaxRanges;
  y.W = static_cast<int>(best < 1 ? 1 : best);
  return y;
}

gqa_status_t qa_check(const gqa_q8_desc_t &d) {
  const gqa_status_t st = q8_check(d, true);
  if (st != GQA_OK) return st;
  // grid sizes, and the numbers of the batch's units with their gaps, are int32
  const long long units = static_cast<long long>(d.batch) * ((d.max_seq_len - 1) / kQaUnit + 1 + kQaPieceCost * kQaWarps);
  return units > 0x7fffffffLL || static_cast<long long>(d.batch > kQaMaxRanges ? d.batch : kQaMaxRanges) * d.num_q_heads > 0x7fffffffLL
             ? GQA_ERR_UNSUPPORTED
             : GQA_OK;
}

}  // namespace

}  // namespace gqa

using namespace gqa;

extern "C" gqa_status_t gqa_q8_workspace_bytes(const gqa_q8_desc_t *desc, size_t *bytes) {
  if (!desc || !bytes) return GQA_ERR_INVALID_ARG;
  const gqa_q8_desc_t d = *desc;
  gqa_status_t st = qa_check(d);
  if (st != GQA_OK) return st;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  int sms = 0;
  st = qa_device(d.device, &sms);
  if (st != GQA_OK) return st;
  const QaLayout y = qa_layout(d, sms);
  *bytes = y.whole || y.W < 2 ? 256
                              : static_cast<size_t>(y.W) * 2 * d.num_q_heads * (kHeadDim + 4) * sizeof(float);
  return GQA_OK;
}

extern "C" gqa_status_t gqa_q8_attn(const gqa_q8_desc_t *desc, const void *q, const void *k_codes, const void *v_codes,
                                    const float *k_scale, const float *v_scale, const int32_t *page_table,
                                    const int32_t *seq_lens, void *out, void *workspace, uint32_t *device_errors,
                                    void *stream) {
  if (!desc) return GQA_ERR_INVALID_ARG;
  const gqa_q8_desc_t d = *desc;
  gqa_status_t st = qa_check(d);
  if (st != GQA_OK) return st;
  if (!q || !k_codes || !v_codes || !k_scale || !v_scale || !seq_lens || !out || !workspace) return GQA_ERR_INVALID_ARG;
  const bool paged = d.block_size > 0;
  if (paged != (page_table != nullptr)) return GQA_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k_codes, 16) || !aligned_to(v_codes, 16) || !aligned_to(out, 16) ||
      !aligned_to(workspace, 256) || !aligned_to(k_scale, 4) || !aligned_to(v_scale, 4) || !aligned_to(page_table, 4) ||
      !aligned_to(seq_lens, 4) || !aligned_to(device_errors, 4))
    return GQA_ERR_INVALID_ARG;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  int sms = 0;
  st = qa_device(d.device, &sms);
  if (st != GQA_OK) return st;

  const QaLayout y = qa_layout(d, sms);
  Q8AttnParams p;
  memset(&p, 0, sizeof p);
  p.q = static_cast<const uint16_t *>(q);
  p.k_codes = static_cast<const uint8_t *>(k_codes);
  p.v_codes = static_cast<const uint8_t *>(v_codes);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.out = static_cast<uint16_t *>(out);
  p.part = static_cast<float *>(workspace);
  p.err = device_errors;
  p.B = d.batch;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.G = d.num_q_heads / d.num_kv_heads;
  p.hg = y.hg;
  p.paged = paged ? 1 : 0;
  p.max_seq = d.max_seq_len;
  p.max_blocks = capacity_tiles(d.max_seq_len);
  p.num_blocks = paged ? d.num_cache_blocks : 0;
  p.W = y.W;
  p.whole = y.whole ? 1 : 0;
  p.merge_by_sequence = p.B <= p.W - 1;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(kHeadDim)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = p.G > 8, e4m3 = d.format == GQA_Q8_E4M3;
  auto *kernel = e4m3 ? (wide ? q8_attn_kernel<GQA_Q8_E4M3, 2> : q8_attn_kernel<GQA_Q8_E4M3, 1>)
                      : (wide ? q8_attn_kernel<GQA_Q8_INT8, 2> : q8_attn_kernel<GQA_Q8_INT8, 1>);
  const long long joins = static_cast<long long>(p.merge_by_sequence ? p.B : p.W - 1) * p.Hq;
  if (launch_pdl(kernel, dim3(static_cast<unsigned>(p.W * (p.Hkv / p.hg))), dim3(kQaThreads),
                 static_cast<size_t>(wide ? Q8Smem<2>::kBytes : Q8Smem<1>::kBytes), s, p) != cudaSuccess ||
      (!y.whole && p.W > 1 &&
       (p.W <= 4LL * p.B ? launch_pdl(q8_merge_kernel<2>, dim3(static_cast<unsigned>(joins)), dim3(64), 0, s, p)
                         : launch_pdl(q8_merge_kernel<4>, dim3(static_cast<unsigned>(joins)), dim3(128), 0, s, p)) != cudaSuccess)) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}
