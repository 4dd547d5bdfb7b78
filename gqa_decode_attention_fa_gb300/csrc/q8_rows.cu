// Rows of an 8-bit KV cache (include/gqa_q8.h): quantised as they are appended, and read back.
//
// The rows of all tokens are numbered, a token's 2 H_kv (K heads, then V heads) behind each other.  A warp takes 8 of
// them (4 where there are few), eight lanes to a row and 16 of its values to a lane, all of its loads on their way
// before the first is used; a lane finds one row's place in the cache.
//
// Quantising.  scale = max |x| / Q (1 + d), |d| <= 2^-24.  The codes change at quotients x / scale on the borders
// of levels, which have few bits (5 for e4m3, 8 for int8), as x and max |x| have (8): x Q / max |x| is either
// on a border or at least 2^-16 of it away.  So any quotient within 2^-17 gives the right code, but on
// the borders, where the sign of d decides, the same one for the row, and where d is 0 the tie is a tie.
// q = x (1 / scale) in two terms, multiplied by 1 - 2^-21 sign(d), falls on the right side, or on
// the border itself (checked for all significands of x and max |x|).  Rows below 2^-60, whose scale may have lost bits, are
// divided exactly: q cut to binary32 with its last bit set where anything was cut.
//   Bounds.  HBM, and the append its arithmetic too (20 instructions a value when each was divided: 32 us where this takes
// 23): 19k tokens of 8 KV heads appended 23 us = 5.2 TB/s, 0.77 of the measured copy rate, 28k rows read back 28.6 us =
// 6.0 TB/s, 0.88; small calls 2.2 to 2.8 us.  What counts is that many warps are on their way: an SM's 64 take 32
// registers each (with 40 and 48 warps 26.8 us; held to 32 the append of 8 rows a warp stores seven words in local memory and
// loads two), a CTA has four (8: 23.1 us and 28.7, 16: 23.7 and 29.0), and one of its warps looks for the places of all its
// rows (each warp for its own: 24.6 us).  Warps that stay and load ahead took 30 to 45 us, 16 rows a warp 2 % more than 8, 32 a
// third more.
#include <string.h>

#include "divisor.cuh"
#include "pairmath.cuh"
#include "q8.cuh"

namespace gqa {

struct Q8RowsParams {
  const uint16_t *k, *v;  // append: the packed rows
  uint16_t *k_out, *v_out;  // read: the packed rows
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;
  const int32_t *page_table, *offsets, *slot_start;
  uint32_t *err;
  long long k_stride, v_stride;
  int B, N, Hkv;
  int paged, max_seq, max_blocks, num_blocks;
  Divisor by_rows;  // 2 Hkv
};

namespace {

constexpr int kRowWarps = 4;

// Where packed row n lives in the cache: its row, -1 if nothing is to be done, -2 if its page id is
// outside the pool.
__device__ __forceinline__ long long q8_cache_row(const Q8RowsParams &p, int n) {
  int b = n, first = n, end = n + 1;
  if (p.offsets) b = sequence_of_row(p.offsets, p.B, n, &first, &end);
  if (b < 0 || first < 0 || end > p.N) return -1;  // (flagged by the first CTA, or no sequence's row)
  const int start = p.slot_start ? p.slot_start[b] : 0;
  if (start < 0 || static_cast<long long>(start) + (end - first) > p.max_seq) {
    flag_error(p.err, start < 0 ? GQA_DEVERR_POSITION : GQA_DEVERR_SEQLEN);
    return -1;
  }
  const int slot = start + (n - first);
  if (!p.paged) return static_cast<long long>(b) * p.max_seq + slot;
  const int pg = p.page_table[static_cast<long long>(b) * p.max_blocks + slot / kTile];
  if (pg < 0 || pg >= p.num_blocks) {
    flag_error(p.err, GQA_DEVERR_PAGE);
    return -2;
  }
  return static_cast<long long>(pg) * kTile + (slot & (kTile - 1));
}

// The rows of a warp, R of them: lane r % R knows the r-th one's token and place in it, and finds its place in the cache.
template <int R>
struct Q8Rows {
  int n, r;  // token and row of the token; n = -1 behind the last one

  __device__ __forceinline__ Q8Rows(const Q8RowsParams &p, int warp, int lane) {
    const uint32_t rows = 2u * p.Hkv;  // N rows < 2^32
    const uint64_t all = static_cast<uint64_t>(blockIdx.x * kRowWarps + warp) * R + (lane % R);
    const uint32_t at = static_cast<uint32_t>(all), t = p.by_rows.divide(at);
    n = all < static_cast<uint64_t>(rows) * p.N ? static_cast<int>(t) : -1;
    r = static_cast<int>(at - t * rows);
  }
  // The row of codes, or -1 or -2 as above.
  __device__ __forceinline__ long long find(const Q8RowsParams &p) const {
    if (n < 0) return -1;
    const long long crow = q8_cache_row(p, n);
    return crow < 0 ? crow : crow * p.Hkv + (r < p.Hkv ? r : r - p.Hkv);
  }
};

// Sequences whose offsets are not in order, flagged once a call.
__device__ __forceinline__ void q8_check_offsets(const Q8RowsParams &p) {
  if (blockIdx.x != 0 || !p.offsets) return;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const int x = p.offsets[b], y = p.offsets[b + 1];
    if (x < 0 || x > y || y > p.N) flag_error(p.err, GQA_DEVERR_SEQLEN);
  }
}

// a / s, a >= 0 and s > 0, cut to binary32 with the last bit set where something was cut.
__device__ __forceinline__ float quotient(float a, float s, float inv) {
  float q = a * inv;
  q = fmaf(fmaf(-q, s, a), inv, q);
  const float r = fmaf(-q, s, a);
  int bits = __float_as_int(q) + (__float_as_int(r) >> 31);
  if (r != 0.f) bits |= 1;
  return __int_as_float(bits);
}

// The larger sizes of two bf16 pairs, NaN where either is one; the signs mean nothing.
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// The codes of a lane's 16 values (bf16 pairs); `largest` is max |x| of the row as bits.
template <int FMT>
__device__ __forceinline__ uint4 quantise16(const uint4 (&raw)[2], uint32_t largest, float *scale) {
  constexpr float kMost = FMT == GQA_Q8_E4M3 ? 448.f : 127.f;
  const float most = __uint_as_float(largest << 16);
  float s = __fdiv_rn(most, kMost);
  const bool usable = largest - 1u < 0x7f7fu;  // not zero, finite
  *scale = usable ? s : largest == 0 ? 0.f : __uint_as_float(0x7fc00000u);
  if (!usable) return make_uint4(0, 0, 0, 0);
  const bool small = largest < 0x2180u;  // below 2^-60
  if (small) s *= 0x1p80f;
  const float inv = __frcp_rn(s);
  const float d = fmaf(s, kMost, -most);  // its sign is that of the scale's rounding
  float e = fmaf(-inv, s, 1.f);
  if (d != 0.f) e -= copysignf(0x1p-21f, d);
  const f2 hi = make_f2(inv, inv), lo = make_f2(inv * e, inv * e);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 &x = raw[i >> 1];
    const uint32_t w[2] = {i & 1 ? x.z : x.x, i & 1 ? x.w : x.y};
    f2 q[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const f2 a = make_f2(bf16_lo_to_float(w[k]), bf16_hi_to_float(w[k]));
      q[k] = fma_f2(a, hi, mul_f2(a, lo));
    }
    if (small) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float a0 = bf16_lo_to_float(w[k]) * 0x1p80f, a1 = bf16_hi_to_float(w[k]) * 0x1p80f;
        q[k] = make_f2(copysignf(fminf(quotient(fabsf(a0), s, inv), kMost), a0),
                       copysignf(fminf(quotient(fabsf(a1), s, inv), kMost), a1));
      }
    }
    uint32_t y[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float q0, q1;
      if (FMT == GQA_Q8_E4M3) {
        split_f2(q[k], q0, q1);
        uint16_t z;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(z) : "f"(q1), "f"(q0));
        y[k] = z;
      } else {  // added to 1.5 2^23 the quotient is rounded to a whole number, ties to even, in the low bits
        split_f2(add_f2(q[k], make_f2(12582912.f, 12582912.f)), q0, q1);
        y[k] = __byte_perm(__float_as_uint(q0), __float_as_uint(q1), 0x0040);
      }
    }
    c[i] = __byte_perm(y[0], y[1], 0x5410);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

}  // namespace

// U groups of four rows a warp.
template <int FMT, int U>
__global__ void __launch_bounds__(32 * kRowWarps, 64 / kRowWarps) q8_append_kernel(const Q8RowsParams p) {
  griddep_wait();
  q8_check_offsets(p);
  __shared__ long long place[kRowWarps * 4 * U];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> 3, ql = lane & 7;
  const Q8Rows<4 * U> mine(p, warp, lane);
  uint4 x[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = __shfl_sync(0xffffffffu, mine.n, 4 * u + sub), r = __shfl_sync(0xffffffffu, mine.r, 4 * u + sub);
    x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
    if (n >= 0) {
      const uint16_t *src = r < p.Hkv ? p.k + n * p.k_stride + static_cast<long long>(r) * kHeadDim
                                      : p.v + n * p.v_stride + static_cast<long long>(r - p.Hkv) * kHeadDim;
      x[u][0] = reinterpret_cast<const uint4 *>(src + 16 * ql)[0];
      x[u][1] = reinterpret_cast<const uint4 *>(src + 16 * ql)[1];
    }
  }
  // a lane to a row looks for its place, for the whole CTA, while the rows are on their way
  if (threadIdx.x < kRowWarps * 4 * U)
    place[threadIdx.x] = Q8Rows<4 * U>(p, threadIdx.x / (4 * U), threadIdx.x).find(p);
  uint4 c[U];
  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t m = max_abs(max_abs(max_abs(x[u][0].x, x[u][0].y), max_abs(x[u][0].z, x[u][0].w)),
                         max_abs(max_abs(x[u][1].x, x[u][1].y), max_abs(x[u][1].z, x[u][1].w)));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max_abs(m, __shfl_xor_sync(0xffffffffu, m, o));
    m &= 0x7fff7fffu;
    c[u] = quantise16<FMT>(x[u], max(m & 0xffffu, m >> 16), &scale[u]);
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long to = place[4 * (U * warp + u) + sub];
    const bool is_k = __shfl_sync(0xffffffffu, mine.r, 4 * u + sub) < p.Hkv;
    if (to >= 0) {
      *reinterpret_cast<uint4 *>((is_k ? p.k_codes : p.v_codes) + to * kHeadDim + 16 * ql) = c[u];
      if (ql == 0) (is_k ? p.k_scale : p.v_scale)[to] = scale[u];
    }
  }
}

template <int FMT, int U>
__global__ void __launch_bounds__(32 * kRowWarps) q8_read_kernel(const Q8RowsParams p) {
  griddep_wait();
  q8_check_offsets(p);
  const int lane = threadIdx.x & 31, sub = lane >> 3, ql = lane & 7;
  const Q8Rows<4 * U> mine(p, threadIdx.x >> 5, lane);
  const long long found = mine.find(p);
  uint4 x[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long from = __shfl_sync(0xffffffffu, found, 4 * u + sub);
    const bool is_k = __shfl_sync(0xffffffffu, mine.r, 4 * u + sub) < p.Hkv;
    x[u] = make_uint4(0, 0, 0, 0);
    s[u] = 0.f;
    if (from >= 0) {
      x[u] = *reinterpret_cast<const uint4 *>((is_k ? p.k_codes : p.v_codes) + from * kHeadDim + 16 * ql);
      s[u] = (is_k ? p.k_scale : p.v_scale)[from];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int n = __shfl_sync(0xffffffffu, mine.n, 4 * u + sub), r = __shfl_sync(0xffffffffu, mine.r, 4 * u + sub);
    const bool ours = __shfl_sync(0xffffffffu, found, 4 * u + sub) != -1;
    const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
    uint32_t y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t h[2];
      codes_to_f16<FMT>(w[i], h[0], h[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
        y[2 * i + e] = pack_bf16(f.x * s[u], f.y * s[u]);
      }
    }
    if (ours) {
      uint16_t *dst = r < p.Hkv ? p.k_out + n * p.k_stride + static_cast<long long>(r) * kHeadDim
                                : p.v_out + n * p.v_stride + static_cast<long long>(r - p.Hkv) * kHeadDim;
      reinterpret_cast<uint4 *>(dst + 16 * ql)[0] = make_uint4(y[0], y[1], y[2], y[3]);
      reinterpret_cast<uint4 *>(dst + 16 * ql)[1] = make_uint4(y[4], y[5], y[6], y[7]);
    }
  }
}

// --------------------------------------------------------------------------------- host side

gqa_status_t q8_check(const gqa_q8_desc_t &d, bool attn) {
  const gqa_status_t st =
      check_cache_geometry(d.batch, attn ? d.num_q_heads : d.num_kv_heads, d.num_kv_heads, d.head_dim, 1, d.block_size,
                           d.max_seq_len, d.num_cache_blocks);
  if (st != GQA_OK) return st;
  return d.format == GQA_Q8_E4M3 || d.format == GQA_Q8_INT8 ? GQA_OK : GQA_ERR_INVALID_ARG;
}

namespace {

// Checks that append and read share, and their parameters.
gqa_status_t q8_rows_params(const gqa_q8_desc_t &d, const void *k, const void *v, const void *k_codes, const void *v_codes,
                            const float *k_scale, const float *v_scale, const int32_t *page_table, const int32_t *offsets,
                            const int32_t *slot_start, uint32_t *err, Q8RowsParams *p) {
  gqa_status_t st = q8_check(d, false);
  if (st != GQA_OK) return st;
  if (d.num_tokens < 1 || (!offsets && d.num_tokens != d.batch)) return GQA_ERR_INVALID_ARG;
  const long long dense = static_cast<long long>(d.num_kv_heads) * kHeadDim;
  for (const int s : {d.k_stride, d.v_stride})
    if (s != 0 && (s < dense || s % 8 != 0)) return GQA_ERR_INVALID_ARG;
  if (static_cast<long long>(d.num_tokens) * d.num_kv_heads > 0x7fffffffLL || dense > 0x7fffffffLL)
    return GQA_ERR_UNSUPPORTED;
  if (!k || !v || !k_codes || !v_codes || !k_scale || !v_scale) return GQA_ERR_INVALID_ARG;
  if ((d.block_size > 0) != (page_table != nullptr)) return GQA_ERR_INVALID_ARG;
  for (const void *t : {k, v, k_codes, v_codes})
    if (!aligned_to(t, 16)) return GQA_ERR_INVALID_ARG;
  for (const void *t : {static_cast<const void *>(k_scale), static_cast<const void *>(v_scale),
                        static_cast<const void *>(page_table), static_cast<const void *>(offsets),
                        static_cast<const void *>(slot_start), static_cast<const void *>(err)})
    if (!aligned_to(t, 4)) return GQA_ERR_INVALID_ARG;
  memset(p, 0, sizeof *p);
  p->k_codes = static_cast<uint8_t *>(const_cast<void *>(k_codes));
  p->v_codes = static_cast<uint8_t *>(const_cast<void *>(v_codes));
  p->k_scale = const_cast<float *>(k_scale);
  p->v_scale = const_cast<float *>(v_scale);
  p->page_table = page_table;
  p->offsets = offsets;
  p->slot_start = slot_start;
  p->err = err;
  p->k_stride = d.k_stride ? d.k_stride : dense;
  p->v_stride = d.v_stride ? d.v_stride : dense;
  p->B = d.batch;
  p->N = d.num_tokens;
  p->Hkv = d.num_kv_heads;
  p->by_rows.set(2u * d.num_kv_heads);
  p->paged = d.block_size > 0 ? 1 : 0;
  p->max_seq = d.max_seq_len;
  p->max_blocks = capacity_tiles(d.max_seq_len);
  p->num_blocks = p->paged ? d.num_cache_blocks : 0;
  return check_device(d.device);
}

// Launches `few` (4 rows a warp) where the rows are few, else `many` (8).
template <typename Kernel>
gqa_status_t q8_launch_rows(const Q8RowsParams &p, int device, Kernel *few, Kernel *many, void *stream) {
  DeviceGuard guard(device);
  if (!guard.ok) return GQA_ERR_CUDA;
  const long long rows = 2LL * p.N * p.Hkv;
  const bool small = rows <= 4096;
  const long long per = kRowWarps * (small ? 4 : 8);
  if (launch_pdl(small ? few : many, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(32 * kRowWarps), 0,
                 static_cast<cudaStream_t>(stream), p) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

}  // namespace

}  // namespace gqa

using namespace gqa;

extern "C" gqa_status_t gqa_q8_append(const gqa_q8_desc_t *desc, const void *k, const void *v, void *k_codes,
                                      void *v_codes, float *k_scale, float *v_scale, const int32_t *page_table,
                                      const int32_t *offsets, const int32_t *slot_start, uint32_t *device_errors,
                                      void *stream) {
  if (!desc || !slot_start) return GQA_ERR_INVALID_ARG;
  const gqa_q8_desc_t d = *desc;
  Q8RowsParams p;
  const gqa_status_t st = q8_rows_params(d, k, v, k_codes, v_codes, k_scale, v_scale, page_table, offsets, slot_start,
                                         device_errors, &p);
  if (st != GQA_OK) return st;
  p.k = static_cast<const uint16_t *>(k);
  p.v = static_cast<const uint16_t *>(v);
  return d.format == GQA_Q8_E4M3 ? q8_launch_rows(p, d.device, q8_append_kernel<GQA_Q8_E4M3, 1>,
                                                  q8_append_kernel<GQA_Q8_E4M3, 2>, stream)
                                 : q8_launch_rows(p, d.device, q8_append_kernel<GQA_Q8_INT8, 1>,
                                                  q8_append_kernel<GQA_Q8_INT8, 2>, stream);
}

extern "C" gqa_status_t gqa_q8_read(const gqa_q8_desc_t *desc, const void *k_codes, const void *v_codes,
                                    const float *k_scale, const float *v_scale, const int32_t *page_table,
                                    const int32_t *offsets, const int32_t *slot_start, void *k_out, void *v_out,
                                    uint32_t *device_errors, void *stream) {
  if (!desc) return GQA_ERR_INVALID_ARG;
  const gqa_q8_desc_t d = *desc;
  Q8RowsParams p;
  const gqa_status_t st = q8_rows_params(d, k_out, v_out, k_codes, v_codes, k_scale, v_scale, page_table, offsets,
                                         slot_start, device_errors, &p);
  if (st != GQA_OK) return st;
  p.k_out = static_cast<uint16_t *>(k_out);
  p.v_out = static_cast<uint16_t *>(v_out);
  return d.format == GQA_Q8_E4M3 ? q8_launch_rows(p, d.device, q8_read_kernel<GQA_Q8_E4M3, 1>,
                                                  q8_read_kernel<GQA_Q8_E4M3, 2>, stream)
                                 : q8_launch_rows(p, d.device, q8_read_kernel<GQA_Q8_INT8, 1>,
                                                  q8_read_kernel<GQA_Q8_INT8, 2>, stream);
}
