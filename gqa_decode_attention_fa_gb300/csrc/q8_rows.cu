// Rows of an 8-bit KV cache (include/gqa_q8.h): quantised as they are appended, and read back.
//
// A warp takes one token, or a part of its 2 H_kv rows (K heads, then V heads): 16 lanes to a row of
// 128 bf16 values when appending, 8 lanes to a row of 128 codes when reading, 16 bytes a lane either way, all of a
// part's loads on their way before the first is used.
//
// Quantising: scale = max |x| / Q.  The level next to x / scale, ties to even, follows from the
// quotient cut to binary32 with its last bit set where anything was cut (so that a quotient next to
// the border of two levels stays on its side): q = x (1 / scale) improved once, and the sign of its
// exact remainder x - q scale.  Rows so small that the remainder would underflow are scaled by 2^80
// with their scale.
#include <string.h>

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
  int parts;  // warps a token
};

namespace {

constexpr int kRowWarps = 8;

// Where packed row n lives in the cache: its row, -1 if nothing is to be done, -2 if its page id is
// outside the pool.  Every lane alike.
__device__ __forceinline__ long long q8_cache_row(const Q8RowsParams &p, int n, int lane) {
  int b = n, first = n, end = n + 1;
  if (p.offsets) b = sequence_of_row(p.offsets, p.B, n, lane, &first, &end);
  if (b < 0 || first < 0 || end > p.N) return -1;  // (flagged by the first CTA, or no sequence's row)
  const int start = p.slot_start ? p.slot_start[b] : 0;
  if (start < 0 || static_cast<long long>(start) + (end - first) > p.max_seq) {
    if (lane == 0) flag_error(p.err, start < 0 ? GQA_DEVERR_POSITION : GQA_DEVERR_SEQLEN);
    return -1;
  }
  const int slot = start + (n - first);
  if (!p.paged) return static_cast<long long>(b) * p.max_seq + slot;
  const int pg = p.page_table[static_cast<long long>(b) * p.max_blocks + slot / kTile];
  if (pg < 0 || pg >= p.num_blocks) {
    if (lane == 0) flag_error(p.err, GQA_DEVERR_PAGE);
    return -2;
  }
  return static_cast<long long>(pg) * kTile + (slot & (kTile - 1));
}

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

// The codes of a row: the lane's 8 values (bf16 pairs), the row's 16 lanes alike in `largest` (max |x| as bits).
template <int FMT>
__device__ __forceinline__ uint2 quantise8(const uint4 &raw, uint32_t largest, float *scale) {
  constexpr float kMost = FMT == GQA_Q8_E4M3 ? 448.f : 127.f;
  float s = __fdiv_rn(__uint_as_float(largest << 16), kMost);
  const bool usable = largest - 1u < 0x7f7fu;  // not zero, finite
  *scale = usable ? s : largest == 0 ? 0.f : __uint_as_float(0x7fc00000u);
  if (!usable) return make_uint2(0, 0);
  float up = 1.f;
  if (largest < 0x2180u) up = 0x1p80f;  // below 2^-60
  s *= up;
  const float inv = __frcp_rn(s);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = bf16_lo_to_float(w[i]) * up, x1 = bf16_hi_to_float(w[i]) * up;
    const float q0 = quotient(fabsf(x0), s, inv), q1 = quotient(fabsf(x1), s, inv);
    if (FMT == GQA_Q8_E4M3) {
      uint16_t y;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(copysignf(q1, x1)), "f"(copysignf(q0, x0)));
      c[i] = y;
    } else {  // added to 1.5 2^23 the quotient is rounded to a whole number, ties to even, in the low bits
      const uint32_t y0 = __float_as_uint(copysignf(fminf(q0, kMost), x0) + 12582912.f);
      const uint32_t y1 = __float_as_uint(copysignf(fminf(q1, kMost), x1) + 12582912.f);
      c[i] = __byte_perm(y0, y1, 0x0040);
    }
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

}  // namespace

// U pairs of rows a warp, those from 2 U part on.
template <int FMT, int U>
__global__ void __launch_bounds__(32 * kRowWarps) q8_append_kernel(const Q8RowsParams p) {
  griddep_wait();
  q8_check_offsets(p);
  const int lane = threadIdx.x & 31, half = lane >> 4, hl = lane & 15;
  const long long at = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int n = static_cast<int>(at / p.parts), part = static_cast<int>(at - static_cast<long long>(n) * p.parts);
  if (n >= p.N) return;
  const int r0 = 2 * U * part + half, rows = 2 * p.Hkv;
  uint4 x[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 2 * u;
    x[u] = make_uint4(0, 0, 0, 0);
    if (r < rows) {
      const uint16_t *src = r < p.Hkv ? p.k + n * p.k_stride + static_cast<long long>(r) * kHeadDim
                                      : p.v + n * p.v_stride + static_cast<long long>(r - p.Hkv) * kHeadDim;
      x[u] = *reinterpret_cast<const uint4 *>(src + 8 * hl);
    }
  }
  const long long crow = q8_cache_row(p, n, lane);
  if (crow < 0) return;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 2 * u;
    uint32_t m = __vmaxu2(__vmaxu2(x[u].x & 0x7fff7fffu, x[u].y & 0x7fff7fffu),
                          __vmaxu2(x[u].z & 0x7fff7fffu, x[u].w & 0x7fff7fffu));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    float scale;
    const uint2 c = quantise8<FMT>(x[u], max(m & 0xffffu, m >> 16), &scale);
    if (r < rows) {
      const int h = r < p.Hkv ? r : r - p.Hkv;
      const long long to = crow * p.Hkv + h;
      *reinterpret_cast<uint2 *>((r < p.Hkv ? p.k_codes : p.v_codes) + to * kHeadDim + 8 * hl) = c;
      if (hl == 0) (r < p.Hkv ? p.k_scale : p.v_scale)[to] = scale;
    }
  }
}

// U groups of four rows a warp, those from 4 U part on.
template <int FMT, int U>
__global__ void __launch_bounds__(32 * kRowWarps) q8_read_kernel(const Q8RowsParams p) {
  griddep_wait();
  q8_check_offsets(p);
  const int lane = threadIdx.x & 31, sub = lane >> 3, ql = lane & 7;
  const long long at = static_cast<long long>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int n = static_cast<int>(at / p.parts), part = static_cast<int>(at - static_cast<long long>(n) * p.parts);
  if (n >= p.N) return;
  const long long crow = q8_cache_row(p, n, lane);
  if (crow == -1) return;
  const int r0 = 4 * U * part + sub, rows = 2 * p.Hkv;
  uint4 x[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 4 * u;
    x[u] = make_uint4(0, 0, 0, 0);
    s[u] = 0.f;
    if (r < rows && crow >= 0) {
      const long long from = crow * p.Hkv + (r < p.Hkv ? r : r - p.Hkv);
      x[u] = *reinterpret_cast<const uint4 *>((r < p.Hkv ? p.k_codes : p.v_codes) + from * kHeadDim + 16 * ql);
      s[u] = (r < p.Hkv ? p.k_scale : p.v_scale)[from];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 4 * u;
    if (r >= rows) break;
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
    uint16_t *dst = r < p.Hkv ? p.k_out + n * p.k_stride + static_cast<long long>(r) * kHeadDim
                              : p.v_out + n * p.v_stride + static_cast<long long>(r - p.Hkv) * kHeadDim;
    reinterpret_cast<uint4 *>(dst + 16 * ql)[0] = make_uint4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<uint4 *>(dst + 16 * ql)[1] = make_uint4(y[4], y[5], y[6], y[7]);
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
  p->paged = d.block_size > 0 ? 1 : 0;
  p->max_seq = d.max_seq_len;
  p->max_blocks = capacity_tiles(d.max_seq_len);
  p->num_blocks = p->paged ? d.num_cache_blocks : 0;
  return check_device(d.device);
}

// Launches `few` (a pair or a group of rows a warp) where the rows are few, else `many` (kMany of them).
template <typename Kernel>
gqa_status_t q8_launch_rows(Q8RowsParams &p, int device, Kernel *few, Kernel *many, int rows_few, int rows_many,
                            void *stream) {
  DeviceGuard guard(device);
  if (!guard.ok) return GQA_ERR_CUDA;
  const bool small = static_cast<long long>(p.N) * p.Hkv <= 2048;
  const int per = small ? rows_few : rows_many;
  p.parts = (2 * p.Hkv + per - 1) / per;
  const long long ctas = (static_cast<long long>(p.N) * p.parts + kRowWarps - 1) / kRowWarps;
  if (launch_pdl(small ? few : many, dim3(static_cast<unsigned>(ctas)), dim3(32 * kRowWarps), 0,
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
                                                  q8_append_kernel<GQA_Q8_E4M3, 4>, 2, 8, stream)
                                 : q8_launch_rows(p, d.device, q8_append_kernel<GQA_Q8_INT8, 1>,
                                                  q8_append_kernel<GQA_Q8_INT8, 4>, 2, 8, stream);
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
                                                  q8_read_kernel<GQA_Q8_E4M3, 4>, 4, 16, stream)
                                 : q8_launch_rows(p, d.device, q8_read_kernel<GQA_Q8_INT8, 1>,
                                                  q8_read_kernel<GQA_Q8_INT8, 4>, 4, 16, stream);
}
