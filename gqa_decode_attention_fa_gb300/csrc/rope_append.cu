// QK RMSNorm + rotary embedding + KV append of any number of tokens (include/gqa_rope.h).
//
// One CTA per token.  Its rows, one contiguous block each of queries, keys and values, come to shared
// memory by three bulk copies while the CTA computes the token's cosines and sines; the values go on
// to the cache by another one.  Half a warp takes a head row, a lane 8 of its dims with their
// partners among them: two chunks of 4 dims that are r / 2 apart (half; r / 2 is a multiple of 4) or
// follow each other (interleaved).
//
// The floor is HBM's (a token is read once and written once, 28 KB at 40/8 heads: 8000 tokens 34 us at
// the measured copy rate); the kernel comes within 1.2 of it, 3460 instructions a token and the waits
// for its rows: 8000 tokens take 41 us = 5.5 TB/s with a token on two warps (47 with one, 44 with
// three, 46 with four; 49 with the partners of the half layout in another lane, reached by shuffles).
// Where the tokens are few, up to 1024, a token has four warps (40/8 heads, four against two: 128 tokens 4.1 us
// against 5.5, 1024 9.3 against 9.7; 1280 12.1 against 11.2; eight warps are no faster at 32 tokens and
// slower from 256 on).  The crossing is the same with 8/8 heads (1024 6.1 against 5.8, 2048 11.0 against 9.4)
// and 16/1; with 64/8 the two are close from there on (1280 14.8 against 14.0, 2048 19.2 against 21.7, 8192 57.4
// against 58.0).  With the most rows a token four would be faster throughout (320/40, two CTAs an SM:
// 8192 tokens 346 us against 531): the rule does not look at the heads.
// What keeps the instructions few:
//   * the norm weights are folded into the lane's cosines and sines, z = r (x_i (w_i c) + x_j
//     (-+ w_j s)), in pairs (fma.rn.f32x2);
//   * the angle p f modulo a turn.  f / 2 pi is kept as a 64-bit fraction of a turn, so p times
//     it modulo 2^64 is the angle's place in the turn, exact but for 2^-65 p turns -- an integer
//     product instead of binary64's (1/64 of the binary32 rate here); sine and cosine of the rest
//     (at most 1/8 turn) are Taylor sums, the large terms in double-word binary32;
//   * the key rows, which stay in the cache and round as the exact value does (rowmath.cuh).
//     An element is first computed in binary32 (only the row's r in double-word) with a bound on
//     its error; where both ends of the interval round to the same bf16 that is the exact value's
//     rounding too, else the warp repeats the element in double-word (the method of Ziv, "Fast
//     evaluation of elementary mathematical functions with correctly rounded last bit", ACM TOMS
//     17(3), 1991): about one pair of rows in ten has such an element.
// Query rows are computed in binary32 and rounded once.
#include <math.h>
#include <string.h>

#include "../../include/gqa_rope.h"
#include "op_args.h"
#include "pairmath.cuh"
#include "rowmath.cuh"

namespace gqa {

struct RopeAppendParams {
  const uint16_t *q, *k, *v;
  uint16_t *k_cache, *v_cache, *q_out;
  const int32_t *page_table, *slot_start, *positions, *counts;
  const uint16_t *q_norm_w, *k_norm_w;
  uint32_t *err;
  long long q_stride, k_stride, v_stride;
  int T, Hq, Hkv;
  int paged, max_seq, max_blocks, num_blocks;
  int rotary;                    // r
  float eps;
  float mag_hi, mag_lo;          // magnitude as a double-word
  uint64_t turns[kHeadDim / 2];  // f_i / (2 pi) modulo 1, in units of 2^-64
};

namespace {

// Cache row of slot `slot` of sequence b, or -1 when its page id is out of range.
__device__ __forceinline__ long long append_row(const RopeAppendParams &p, int b, int slot) {
  if (!p.paged) return static_cast<long long>(b) * p.max_seq + slot;
  const int pg = p.page_table[static_cast<long long>(b) * p.max_blocks + slot / kTile];
  if (pg < 0 || pg >= p.num_blocks) return -1;
  return static_cast<long long>(pg) * kTile + (slot & (kTile - 1));
}

// Bulk copy of this CTA's shared memory to global memory (both 16-byte aligned, a multiple of 16
// bytes); bulk_wait returns once the thread's committed copies are complete.
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)),
               "r"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// c + v for |c| >= 2 |v|, both double-words (no cancellation): relative error about 2^-46.
__device__ __forceinline__ dw dw_add_big(dw c, dw v) {
  const dw s = fast_two_sum(c.hi, v.hi);
  return fast_two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(c.lo, v.lo)));
}

// cos and sin of frac 2^-64 turns as double-words (relative error about 2^-44).
__device__ __forceinline__ void cos_sin_turn(uint64_t frac, dw *c, dw *s) {
  const uint64_t quarter = (frac + (1ull << 61)) >> 62;                // nearest quarter turn
  const int64_t rest = static_cast<int64_t>(frac - (quarter << 62));   // within an eighth of a turn
  const float hi = static_cast<float>(rest);
  const float lo = static_cast<float>(rest - static_cast<int64_t>(hi));
  const dw x = dw_mul(dw{hi, lo}, dw{0x1.921fb6p-62f, -0x1.777a5cp-87f});  // 2 pi / 2^64
  const dw z = dw_mul(x, x);
  // sin x = x + x z (-1/3! + z (1/5! + z (-1/7! + z (1/9! - z/11! + z^2/13! - z^3/15!))))
  float t = fmaf(z.hi, fmaf(z.hi, fmaf(z.hi, -0x1.ae7f3ep-41f, 0x1.612462p-33f), -0x1.ae6456p-26f), 0x1.71de3ap-19f);
  dw p = dw_add_big(dw{-0x1.a01a02p-13f, 0x1.7f97fap-39f}, dw{z.hi * t, 0.f});
  p = dw_add_big(dw{0x1.111112p-7f, -0x1.ddddep-32f}, dw_mul(z, p));
  p = dw_add_big(dw{-0x1.555556p-3f, 0x1.555556p-28f}, dw_mul(z, p));
  const dw sx = dw_add_big(x, dw_mul(x, dw_mul(z, p)));
  // cos x = 1 + z (-1/2! + z (1/4! + z (-1/6! + z (1/8! - z/10! + z^2/12! - z^3/14!))))
  t = fmaf(z.hi, fmaf(z.hi, -0x1.93974ap-37f, 0x1.1eed8ep-29f), -0x1.27e4fcp-22f);
  p = dw_add_big(dw{0x1.a01a02p-16f, -0x1.7f97fap-42f}, dw{z.hi * t, 0.f});
  p = dw_add_big(dw{-0x1.6c16c2p-10f, 0x1.27d27ep-35f}, dw_mul(z, p));
  p = dw_add_big(dw{0x1.555556p-5f, -0x1.555556p-30f}, dw_mul(z, p));
  p = dw_add_big(dw{-0.5f, 0.f}, dw_mul(z, p));
  const dw cx = dw_add_big(dw{1.f, 0.f}, dw_mul(z, p));
  const dw a = quarter & 1 ? sx : cx, b = quarter & 1 ? cx : sx;  // of the angle, but for their signs
  *c = (quarter + 1) & 2 ? dw_neg(a) : a;
  *s = quarter & 2 ? dw_neg(b) : b;
}

__device__ __forceinline__ f2 unpack_f2(uint32_t w) { return make_f2(bf16_lo_to_float(w), bf16_hi_to_float(w)); }
__device__ __forceinline__ f2 abs_f2(f2 x) {
  f2 r;
  r.v = x.v & 0x7fffffff7fffffffull;
  return r;
}

__device__ __forceinline__ f2 swap_f2(f2 x) {
  float a, b;
  split_f2(x, a, b);
  return make_f2(b, a);
}

// A lane's 8 dims of a row, as two chunks of 4 whose partners the lane holds too: in the half layout
// chunk l of the first elements and the one r / 2 dims on, for l < r / 8, else two chunks that do
// not turn; in the interleaved layout, where partners are neighbours, chunks 2 l and 2 l + 1.
template <bool kInterleaved, bool kFull>
struct RopeLane {
  int chunk[2], pair[2];  // and the chunk's first pair
  bool turns[2];

  __device__ __forceinline__ void init(int rotary, int l) {
    const int m = kFull ? kHeadDim / 8 : rotary / 8;  // chunks of the first elements
    const bool split = !kInterleaved && (kFull || l < m);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      chunk[h] = split ? l + h * m : 2 * l + h;
      turns[h] = kFull || (kInterleaved ? chunk[h] < 2 * m : split);
      pair[h] = kInterleaved ? 2 * chunk[h] : 4 * l;
    }
  }
  // the lane's words (bf16 pairs) of a row: of its 32 uint2 chunks
  __device__ __forceinline__ void load(const uint2 *row, uint32_t (&w)[4]) const {
    if (kInterleaved) {
      const uint4 x = *reinterpret_cast<const uint4 *>(row + chunk[0]);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
      const uint2 x = row[chunk[0]], y = row[chunk[1]];
      w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
    }
  }
  __device__ __forceinline__ void store(uint2 *row, const uint32_t (&w)[4]) const {
    if (kInterleaved) {
      *reinterpret_cast<uint4 *>(row + chunk[0]) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      row[chunk[0]] = make_uint2(w[0], w[1]);
      row[chunk[1]] = make_uint2(w[2], w[3]);
    }
  }
  // The partners of values 2 e and 2 e + 1; zeros in chunks that do not turn, which have no sine
  // term (and must not meet 0 x inf).
  __device__ __forceinline__ f2 partners(const f2 (&v)[4], int e) const {
    const f2 x = kInterleaved ? swap_f2(v[e]) : v[e ^ 2];
    return kFull || turns[e >> 1] ? x : make_f2(0.f, 0.f);
  }
  // The sign of dim 4 h + e's sine term is minus.  Chunks that do not turn have it too: x - 0 is x.
  __device__ __forceinline__ bool negative(int h, int e) const {
    return (kInterleaved ? (e & 1) == 0 : h == 0) || !(kFull || turns[h]);
  }
  __device__ __forceinline__ int pair_of(int h, int e) const { return pair[h] + (kInterleaved ? e >> 1 : e); }
};

// One key element in double-word arithmetic, the rounding of its exact value: y its own product x w, yp
// its partner's with the sign of the sine term, c its pair's (cos_hi, sin_hi, cos_lo, sin_lo).
__device__ __noinline__ uint32_t key_element_exact(float y, float yp, float4 c, bool turns, dw rn, bool norm) {
  dw z = {y, 0.f};
  if (turns) z = dw_add(dw_mul_f(dw{c.x, c.z}, y), dw_mul_f(dw{c.y, c.w}, yp));
  return round_dw_bf16(norm ? dw_mul(z, rn) : z);
}

// r = 1 / sqrt(ss / 128 + eps) of the half warp's row as a double-word, from a lane's 8 values: the squares
// are exact in binary32 (those of values below 2^-67 are not, which a mean of 2^-100 and more hides) and
// are summed with the errors of every addition (Knuth's TwoSum, in pairs), a binary32 seed takes one
// Newton step with its residual.
__device__ __forceinline__ dw row_inv_rms(const f2 (&v)[4], float eps) {
  f2 s = mul_f2(v[0], v[0]), err = make_f2(0.f, 0.f);
  const f2 minus = make_f2(-1.f, -1.f);
#pragma unroll
  for (int e = 1; e < 4; ++e) {
    const f2 q = mul_f2(v[e], v[e]), t = add_f2(s, q);
    const f2 bb = fma_f2(s, minus, t);                                        // t - s
    const f2 lost = add_f2(fma_f2(fma_f2(bb, minus, t), minus, s), fma_f2(bb, minus, q));  // (s - (t - bb)) + (q - bb)
    err = add_f2(err, lost);
    s = t;
  }
  float a, b, ea, eb;
  split_f2(s, a, b);
  split_f2(err, ea, eb);
  dw ss = two_sum(a, b);
  ss.lo = __fadd_rn(ss.lo, __fadd_rn(ea, eb));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, ss.hi, o), lo = __shfl_xor_sync(0xffffffffu, ss.lo, o);
    const dw t = two_sum(ss.hi, hi);
    ss = dw{t.hi, __fadd_rn(t.lo, __fadd_rn(ss.lo, lo))};
  }
  const dw m = dw_add(fast_two_sum(__fmul_rn(ss.hi, 1.0f / 128.0f), __fmul_rn(ss.lo, 1.0f / 128.0f)), dw{eps, 0.f});
  // r of m 4^-h, in [1, 4), so that no low word is subnormal (that of r0^2 would lose bits from m of 2^101 on)
  const int h = max(-63, min(63, ((__float_as_int(m.hi) >> 23) - 127) >> 1));
  const float scale = __int_as_float((127 - 2 * h) << 23), back = __int_as_float((127 - h) << 23);
  const dw u = {__fmul_rn(m.hi, scale), __fmul_rn(m.lo, scale)};
  const float r0 = rsqrtf(u.hi);
  const dw p = two_prod(r0, r0);
  // 1 - u r0^2: u.hi p.hi is near 1, so the fma gives its difference exactly rounded
  const float e = __fmaf_rn(-u.lo, p.hi, __fmaf_rn(-u.hi, p.lo, __fmaf_rn(-u.hi, p.hi, 1.f)));
  const dw r = fast_two_sum(r0, __fmul_rn(__fmul_rn(0.5f, r0), e));
  return dw{__fmul_rn(r.hi, back), __fmul_rn(r.lo, back)};
}

// Tokens up to which a CTA has four warps, and above which two.
constexpr int kRopeFew = 1024;
// A CTA holds its token's H_q + 2 H_kv rows in shared memory (256 bytes each), as the prefill prologue.
constexpr int kRopeMaxSmem = 200 * 1024;
// Error of a key element computed in binary32, relative to r (|x_i w_i cos| + |x_j w_j sin|), in
// units of 2^-24: the rounding of r to binary32, cos or sin, its product with w, the product with x,
// the fma and the product with r, 1 each.  8 leaves room for the rounding of the interval's own ends.
constexpr float kKeyWindow = 8.f * 0x1p-24f;

}  // namespace

template <bool kInterleaved, bool kFull, int kRopeWarps>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeWarps == 2 ? 13 : 7) rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
  constexpr int kRopeThreads = 32 * kRopeWarps;
  __shared__ float4 cs[kHeadDim / 2];  // m (cos_hi, sin_hi, cos_lo, sin_lo) of pair i
  __shared__ __align__(8) uint64_t arrived;
  extern __shared__ __align__(128) uint4 rows[];  // the token's H_q + 2 H_kv rows, 16 chunks each
  const uint32_t bar = smem_addr(&arrived);
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    fence_barrier_init();
  }
  griddep_wait();  // everything below may come from the preceding kernel
  const int b = static_cast<int>(blockIdx.x) / p.T, t = static_cast<int>(blockIdx.x) - b * p.T;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, half = lane >> 4, hl = lane & 15;
  const long long tok = static_cast<long long>(blockIdx.x);
  const int n = p.counts ? p.counts[b] : p.T;
  const int s0 = p.slot_start[b];
  int pos = p.positions ? p.positions[tok] : s0 + t;
  const bool seq_ok = n >= 0 && n <= p.T && s0 >= 0 && static_cast<long long>(s0) + n <= p.max_seq;
  if (seq_ok && t >= n) return;
  if (!seq_ok || pos < 0) {
    if (tid == 0 && (seq_ok || t == 0))
      flag_error(p.err, (seq_ok || s0 < 0) ? GQA_DEVERR_POSITION : GQA_DEVERR_SEQLEN);
    uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + tok * p.Hq * kHeadDim);
    for (int c = tid; c < p.Hq * kHeadDim / 8; c += kRopeThreads) dst[c] = make_uint4(0, 0, 0, 0);
    return;
  }

  const uint32_t qbytes = static_cast<uint32_t>(p.Hq) * kHeadDim * 2, kbytes = static_cast<uint32_t>(p.Hkv) * kHeadDim * 2;
  if (tid == 0) {
    const uint32_t dst = smem_addr(rows);
    mbar_arrive_expect_tx(bar, qbytes + 2 * kbytes);
    bulk_load(dst, p.q + tok * p.q_stride, qbytes, bar);
    bulk_load(dst + qbytes, p.k + tok * p.k_stride, kbytes, bar);
    bulk_load(dst + qbytes + kbytes, p.v + tok * p.v_stride, kbytes, bar);
  }
  for (int i = tid; i < p.rotary / 2; i += kRopeThreads) {
    dw c, s;
    cos_sin_turn(static_cast<uint64_t>(pos) * p.turns[i], &c, &s);
    if (p.mag_hi != 1.f || p.mag_lo != 0.f) {
      c = dw_mul(c, dw{p.mag_hi, p.mag_lo});
      s = dw_mul(s, dw{p.mag_hi, p.mag_lo});
    }
    cs[i] = make_float4(c.hi, s.hi, c.lo, s.lo);
  }
  const long long crow = append_row(p, b, s0 + t);
  if (crow < 0 && tid == 0) flag_error(p.err, GQA_DEVERR_PAGE);
  RopeLane<kInterleaved, kFull> l;
  l.init(p.rotary, hl);
  __syncthreads();  // cos and sin, and the barrier's initialisation
  if (!__all_sync(0xffffffffu, mbar_wait(bar, 0))) {  // the rows never arrived: flag, write nothing
    if (lane == 0) flag_error(p.err, GQA_DEVERR_TIMEOUT);
    (void)mbar_wait(bar, 0);  // do not leave while copies into this CTA's shared memory may be in flight
    return;
  }
  if (tid == 0 && crow >= 0) {  // the values go to the cache as they are
    bulk_store(p.v_cache + crow * p.Hkv * kHeadDim, smem_addr(rows) + qbytes + kbytes, kbytes);
    bulk_commit();
  }

  // The lane's cosines and sines with the norm weights folded in (w: its own weights).
  f2 A[4], S[4], w[4];
  auto fold = [&](const uint16_t *weights) {
    uint32_t words[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};  // ones
    if (weights) l.load(reinterpret_cast<const uint2 *>(weights), words);
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = unpack_f2(words[e]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float c[2], s[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int h = e >> 1, d = 2 * (e & 1) + k;
        const float4 v = kFull || l.turns[h] ? cs[l.pair_of(h, d)] : make_float4(1.f, 0.f, 0.f, 0.f);
        c[k] = v.x;
        s[k] = l.negative(h, d) ? -v.y : v.y;
      }
      A[e] = mul_f2(w[e], make_f2(c[0], c[1]));
      S[e] = mul_f2(l.partners(w, e), make_f2(s[0], s[1]));
    }
  };
  // r of a row (1 where there is no norm), from its values
  auto inv_rms = [&](const f2 (&v)[4]) {
    f2 q = mul_f2(v[0], v[0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) q = fma_f2(v[e], v[e], q);
    float a, c;
    split_f2(q, a, c);
    float ss = a + c;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    return rsqrtf(ss * (1.0f / 128.0f) + p.eps);
  };

  // Row pairs, a half warp a row: rows 2 i + half of the queries, then of the keys.
  const uint2 *const held = reinterpret_cast<const uint2 *>(rows);  // 32 chunks of 4 dims a row
  fold(p.q_norm_w);
  uint2 *qdst = reinterpret_cast<uint2 *>(p.q_out + tok * p.Hq * kHeadDim);
  for (int i = warp; 2 * i < p.Hq; i += kRopeWarps) {
    uint32_t x[4], out[4];
    l.load(held + min(2 * i + half, p.Hq - 1) * 32, x);
    f2 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = unpack_f2(x[e]);
    const float rn = p.q_norm_w ? inv_rms(v) : 1.f;
    const f2 rn2 = make_f2(rn, rn);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float a, c;
      split_f2(mul_f2(rn2, fma_f2(v[e], A[e], mul_f2(l.partners(v, e), S[e]))), a, c);
      out[e] = pack_bf16(a, c);
    }
    if (2 * i + half < p.Hq) l.store(qdst + (2 * i + half) * 32, out);
  }
  if (crow < 0) return;
  uint2 *kdst = reinterpret_cast<uint2 *>(p.k_cache + crow * p.Hkv * kHeadDim);
  fold(p.k_norm_w);
  for (int i = warp; 2 * i < p.Hkv; i += kRopeWarps) {
    uint32_t x[4];
    l.load(held + (p.Hq + min(2 * i + half, p.Hkv - 1)) * 32, x);
    f2 v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = unpack_f2(x[e]);
    const dw rn = p.k_norm_w ? row_inv_rms(v, p.eps) : dw{1.f, 0.f};
    const f2 rn2 = make_f2(rn.hi, rn.hi), up = make_f2(kKeyWindow, kKeyWindow), down = make_f2(-kKeyWindow, -kKeyWindow);
    uint32_t out[4], unsure = 0u;  // a bit per element
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f2 t = mul_f2(l.partners(v, e), S[e]);
      const f2 z = mul_f2(rn2, fma_f2(v[e], A[e], t));
      const f2 size = mul_f2(rn2, fma_f2(abs_f2(v[e]), abs_f2(A[e]), abs_f2(t)));
      float a, c;
      split_f2(fma_f2(size, down, z), a, c);
      out[e] = pack_bf16(a, c);
      split_f2(fma_f2(size, up, z), a, c);
      const uint32_t differ = out[e] ^ pack_bf16(a, c);
      // tiny values, whose binary32 steps are not relative, take the exact path, and so does
      // what is not finite
      split_f2(size, a, c);
      if ((differ & 0xffffu) || !(a == 0.f || (a > 0x1p-80f && a < 0x1p100f))) unsure |= 1u << (2 * e);
      if ((differ >> 16) || !(c == 0.f || (c > 0x1p-80f && c < 0x1p100f))) unsure |= 2u << (2 * e);
    }
    const uint32_t any = __reduce_or_sync(0xffffffffu, unsure);
    if (any) {  // the warp repeats those elements exactly
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (!(any >> e & 1u)) continue;
        const int h = e >> 2, x2 = e >> 1;
        const f2 y2 = mul_f2(v[x2], w[x2]), yp2 = mul_f2(l.partners(v, x2), l.partners(w, x2));  // exact: 8-bit significands
        float y[2], yp[2];
        split_f2(y2, y[0], y[1]);
        split_f2(yp2, yp[0], yp[1]);
        const float4 c = l.turns[h] ? cs[l.pair_of(h, e & 3)] : make_float4(1.f, 0.f, 0.f, 0.f);
        const uint32_t z = key_element_exact(y[e & 1], l.negative(h, e & 3) ? -yp[e & 1] : yp[e & 1], c, l.turns[h], rn,
                                             p.k_norm_w != nullptr);
        out[x2] = e & 1 ? (out[x2] & 0xffffu) | (z << 16) : (out[x2] & 0xffff0000u) | z;
      }
    }
    if (2 * i + half < p.Hkv) l.store(kdst + (2 * i + half) * 32, out);
  }
  if (tid == 0) bulk_wait();  // the values have left shared memory and are written
}

}  // namespace gqa

using namespace gqa;

namespace {

// f / (2 pi) modulo 1 in units of 2^-64, rounded: the 53-bit significand of f times the first 128
// bits of 1 / (2 pi), shifted into place.  |f| <= 2^16.
uint64_t turns_of(double f) {
  int e = 0;
  const double a = frexp(fabs(f), &e);  // |f| = a 2^e, a in [1/2, 1) or 0
  const uint64_t m = static_cast<uint64_t>(ldexp(a, 53));
  const int shift = 117 - e;            // |f| / (2 pi) 2^64 = m c 2^-shift, c = 2^128 / (2 pi)
  if (m == 0 || shift >= 191) return 0;
  const unsigned __int128 lo = static_cast<unsigned __int128>(m) * 0x7f09d5f47d4d3770ull;
  const unsigned __int128 hi = static_cast<unsigned __int128>(m) * 0x28be60db9391054aull + (lo >> 64);
  // m c = hi 2^64 + (lo mod 2^64); shift is above 64, so the low word only rounds
  const int s = shift - 64;             // 36 .. 126
  const uint64_t t = static_cast<uint64_t>(hi >> s) + static_cast<uint64_t>((hi >> (s - 1)) & 1);
  return f < 0 ? 0 - t : t;
}

}  // namespace

extern "C" gqa_status_t gqa_rope_freqs(const gqa_rope_t *rope, double *freqs, double *magnitude) {
  if (!rope) return GQA_ERR_INVALID_ARG;
  const gqa_rope_t &s = *rope;
  const int r = s.rotary_dim;
  if (s.layout != GQA_ROPE_HALF && s.layout != GQA_ROPE_INTERLEAVED) return GQA_ERR_INVALID_ARG;
  if (r < 8 || r > kHeadDim || r % 8 != 0) return GQA_ERR_INVALID_ARG;
  if (s.scaling < GQA_ROPE_NONE || s.scaling > GQA_ROPE_CUSTOM) return GQA_ERR_INVALID_ARG;
  if (!isfinite(s.magnitude) || s.magnitude < 0.f) return GQA_ERR_INVALID_ARG;
  double f[kHeadDim / 2], m = 1.0;
  if (s.scaling == GQA_ROPE_CUSTOM) {
    if (!s.freqs) return GQA_ERR_INVALID_ARG;
    for (int i = 0; i < r / 2; ++i) {
      if (!isfinite(s.freqs[i])) return GQA_ERR_INVALID_ARG;
      f[i] = s.freqs[i];
    }
  } else {
    if (!(isfinite(s.theta) && s.theta > 0.f)) return GQA_ERR_INVALID_ARG;
    for (int i = 0; i < r / 2; ++i) f[i] = pow(static_cast<double>(s.theta), -2.0 * i / static_cast<double>(r));
    if (s.scaling != GQA_ROPE_NONE && !(isfinite(s.factor) && s.factor > 0.f)) return GQA_ERR_INVALID_ARG;
    if ((s.scaling == GQA_ROPE_BANDED || s.scaling == GQA_ROPE_YARN) && s.original_max_len < 1)
      return GQA_ERR_INVALID_ARG;
    const double factor = s.factor, two_pi = 6.283185307179586476925;
    if (s.scaling == GQA_ROPE_LINEAR) {
      for (int i = 0; i < r / 2; ++i) f[i] /= factor;
    } else if (s.scaling == GQA_ROPE_BANDED) {
      if (!(isfinite(s.low_freq_factor) && isfinite(s.high_freq_factor) && s.low_freq_factor > 0.f &&
            s.high_freq_factor > s.low_freq_factor))
        return GQA_ERR_INVALID_ARG;
      for (int i = 0; i < r / 2; ++i) {
        const double periods = s.original_max_len * f[i] / two_pi;  // of the pair in the trained length
        double keep = (periods - s.low_freq_factor) /
                      (static_cast<double>(s.high_freq_factor) - s.low_freq_factor);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        f[i] = keep * f[i] + (1.0 - keep) * f[i] / factor;
      }
    } else if (s.scaling == GQA_ROPE_YARN) {
      if (!(isfinite(s.beta_fast) && isfinite(s.beta_slow) && s.beta_slow > 0.f && s.beta_fast > s.beta_slow) ||
          s.theta <= 1.f || s.factor < 1.f)
        return GQA_ERR_INVALID_ARG;
      auto dim_of = [&](double beta) {  // the pair with `beta` periods in the trained length
        return r * log(s.original_max_len / (beta * two_pi)) / (2.0 * log(static_cast<double>(s.theta)));
      };
      const double low = fmax(floor(dim_of(s.beta_fast)), 0.0), high = fmin(ceil(dim_of(s.beta_slow)), r - 1.0);
      for (int i = 0; i < r / 2; ++i) {
        double ramp = (i - low) / fmax(high - low, 0.001);
        ramp = ramp < 0.0 ? 0.0 : ramp > 1.0 ? 1.0 : ramp;
        f[i] = ramp * f[i] / factor + (1.0 - ramp) * f[i];
      }
      m = 0.1 * log(factor) + 1.0;
    }
  }
  for (int i = 0; i < r / 2; ++i)
    if (!(fabs(f[i]) <= 65536.0)) return GQA_ERR_INVALID_ARG;
  if (s.magnitude > 0.f) m = s.magnitude;
  if (freqs) memcpy(freqs, f, sizeof(double) * (r / 2));
  if (magnitude) *magnitude = m;
  return GQA_OK;
}

namespace {

// What the kernel takes of a rotary embedding.  The thread's last one is kept (a model has one for
// all layers and steps, and its 64 powers take longer than a launch): it follows from the fields
// alone, but for CUSTOM, whose table is read at every call.
struct RopeTurns {
  gqa_rope_t of;
  bool valid = false;
  uint64_t turns[kHeadDim / 2];
  float mag_hi, mag_lo;
};

bool same_rope(const gqa_rope_t &a, const gqa_rope_t &b) {
  return a.layout == b.layout && a.rotary_dim == b.rotary_dim && a.scaling == b.scaling &&
         a.original_max_len == b.original_max_len && a.theta == b.theta && a.factor == b.factor &&
         a.low_freq_factor == b.low_freq_factor && a.high_freq_factor == b.high_freq_factor &&
         a.beta_fast == b.beta_fast && a.beta_slow == b.beta_slow && a.magnitude == b.magnitude;
}

gqa_status_t rope_turns(const gqa_rope_t *rope, const RopeTurns **out) {
  static thread_local RopeTurns last;
  *out = &last;
  if (rope && last.valid && rope->scaling != GQA_ROPE_CUSTOM && same_rope(*rope, last.of)) return GQA_OK;
  last.valid = false;
  double freqs[kHeadDim / 2], magnitude;
  const gqa_status_t st = gqa_rope_freqs(rope, freqs, &magnitude);
  if (st != GQA_OK) return st;
  for (int i = 0; i < kHeadDim / 2; ++i) last.turns[i] = i < rope->rotary_dim / 2 ? turns_of(freqs[i]) : 0;
  last.mag_hi = static_cast<float>(magnitude);
  last.mag_lo = static_cast<float>(magnitude - last.mag_hi);
  last.of = *rope;
  last.valid = true;
  return GQA_OK;
}

}  // namespace

namespace {

// First call on the current device: the kernels' shared memory.
bool rope_configure(int device) {
  static std::atomic<bool> done[64];
  if (device < 64 && done[device].load(std::memory_order_acquire)) return true;
  auto raise = [](void (*kernel)(const RopeAppendParams)) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRopeMaxSmem) == cudaSuccess &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) ==
               cudaSuccess;
  };
  const bool ok = raise(rope_append_kernel<true, true, 2>) && raise(rope_append_kernel<true, true, 4>) &&
                  raise(rope_append_kernel<true, false, 2>) && raise(rope_append_kernel<true, false, 4>) &&
                  raise(rope_append_kernel<false, true, 2>) && raise(rope_append_kernel<false, true, 4>) &&
                  raise(rope_append_kernel<false, false, 2>) && raise(rope_append_kernel<false, false, 4>);
  if (!ok) cudaGetLastError();
  if (ok && device < 64) done[device].store(true, std::memory_order_release);
  return ok;
}

}  // namespace

extern "C" gqa_status_t gqa_rope_append(const gqa_rope_desc_t *desc, const void *q, const void *k, const void *v,
                                        void *k_cache, void *v_cache, const int32_t *page_table,
                                        const int32_t *slot_start, const int32_t *positions, const int32_t *counts,
                                        const void *q_norm_w, const void *k_norm_w, const gqa_rope_t *rope, float eps,
                                        void *q_out, uint32_t *device_errors, void *stream) {
  if (!desc) return GQA_ERR_INVALID_ARG;
  const gqa_rope_desc_t d = *desc;
  gqa_status_t st = check_cache_geometry(d.batch, d.num_q_heads, d.num_kv_heads, d.head_dim, d.num_tokens,
                                         d.block_size, d.max_seq_len, d.num_cache_blocks);
  if (st != GQA_OK) return st;
  if ((static_cast<long long>(d.num_q_heads) + 2LL * d.num_kv_heads) * kHeadDim * 2 > kRopeMaxSmem) return GQA_ERR_UNSUPPORTED;
  if (!q || !k || !v || !k_cache || !v_cache || !slot_start || !q_out) return GQA_ERR_INVALID_ARG;
  const bool paged = d.block_size > 0;
  if (paged != (page_table != nullptr)) return GQA_ERR_INVALID_ARG;
  if (!isfinite(eps) || eps < 0.f) return GQA_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_cache, 16) ||
      !aligned_to(v_cache, 16) || !aligned_to(q_out, 16) || !aligned_to(q_norm_w, 16) || !aligned_to(k_norm_w, 16) ||
      !aligned_to(page_table, 4) || !aligned_to(slot_start, 4) || !aligned_to(positions, 4) ||
      !aligned_to(counts, 4) || !aligned_to(device_errors, 4))
    return GQA_ERR_INVALID_ARG;
  const long long qd = static_cast<long long>(d.num_q_heads) * kHeadDim;
  const long long kd = static_cast<long long>(d.num_kv_heads) * kHeadDim;
  auto stride_ok = [](long long s, long long dense) { return s == 0 || (s >= dense && s % 8 == 0); };
  if (!stride_ok(d.q_stride, qd) || !stride_ok(d.k_stride, kd) || !stride_ok(d.v_stride, kd)) return GQA_ERR_INVALID_ARG;
  if (q_out == q && d.q_stride != 0 && d.q_stride != qd) return GQA_ERR_INVALID_ARG;
  RopeAppendParams p;
  memset(&p, 0, sizeof p);
  const RopeTurns *turns = nullptr;
  st = rope_turns(rope, &turns);
  if (st != GQA_OK) return st;
  memcpy(p.turns, turns->turns, sizeof p.turns);
  p.mag_hi = turns->mag_hi;
  p.mag_lo = turns->mag_lo;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  p.k_cache = static_cast<uint16_t *>(k_cache);
  p.v_cache = static_cast<uint16_t *>(v_cache);
  p.q_out = static_cast<uint16_t *>(q_out);
  p.page_table = page_table;
  p.slot_start = slot_start;
  p.positions = positions;
  p.counts = counts;
  p.q_norm_w = static_cast<const uint16_t *>(q_norm_w);
  p.k_norm_w = static_cast<const uint16_t *>(k_norm_w);
  p.err = device_errors;
  p.q_stride = d.q_stride ? d.q_stride : qd;
  p.k_stride = d.k_stride ? d.k_stride : kd;
  p.v_stride = d.v_stride ? d.v_stride : kd;
  p.T = d.num_tokens;
  p.Hq = d.num_q_heads;
  p.Hkv = d.num_kv_heads;
  p.paged = paged ? 1 : 0;
  p.max_seq = d.max_seq_len;
  p.max_blocks = capacity_tiles(d.max_seq_len);
  p.num_blocks = paged ? d.num_cache_blocks : 0;
  p.rotary = rope->rotary_dim;
  p.eps = eps;
  const dim3 grid(static_cast<unsigned>(d.batch) * static_cast<unsigned>(d.num_tokens));
  const long long tokens = static_cast<long long>(d.batch) * d.num_tokens;
  const bool full = p.rotary == kHeadDim, many = tokens > kRopeFew;
  const int warps = many ? 2 : 4;
  const size_t smem = static_cast<size_t>(d.num_q_heads + 2 * d.num_kv_heads) * kHeadDim * 2;
  if (!rope_configure(d.device)) return GQA_ERR_CUDA;
  void (*kernel)(const RopeAppendParams);
  if (rope->layout == GQA_ROPE_INTERLEAVED)
    kernel = full ? (many ? rope_append_kernel<true, true, 2> : rope_append_kernel<true, true, 4>)
                  : (many ? rope_append_kernel<true, false, 2> : rope_append_kernel<true, false, 4>);
  else
    kernel = full ? (many ? rope_append_kernel<false, true, 2> : rope_append_kernel<false, true, 4>)
                  : (many ? rope_append_kernel<false, false, 2> : rope_append_kernel<false, false, 4>);
  if (launch_pdl(kernel, grid, dim3(32 * warps), smem, static_cast<cudaStream_t>(stream), p) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}
