// QK RMSNorm + rotary embedding + KV append of any number of tokens (include/gqa_rope.h).
//
// One CTA per token.  The token's cos/sin (binary64, kept as double-word hi + lo) go through
// shared memory; then a warp takes a head row at a time, lane l holding dims 4l .. 4l + 3 (one
// 8-byte access).  In the interleaved layout both pairs of a lane are in the lane; in the half
// layout the partners are r/8 lanes apart and come by a shuffle (r is a multiple of 8, so that a
// lane's four dims are on one side).  Query rows are computed in binary32 and rounded
// once; key rows, which stay in the cache, in double-word arithmetic, so that they round as
// the exact value does (rowmath.cuh).
#include <math.h>
#include <string.h>

#include "../../include/gqa_rope.h"
#include "op_args.h"
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
  double magnitude;
  double freq[kHeadDim / 2];
};

namespace {

constexpr int kRopeThreads = 256;

// Cache row of slot `slot` of sequence b, or -1 when its page id is out of range.
__device__ __forceinline__ long long append_row(const RopeAppendParams &p, int b, int slot) {
  if (!p.paged) return static_cast<long long>(b) * p.max_seq + slot;
  const int pg = p.page_table[static_cast<long long>(b) * p.max_blocks + slot / kTile];
  if (pg < 0 || pg >= p.num_blocks) return -1;
  return static_cast<long long>(pg) * kTile + (slot & (kTile - 1));
}

}  // namespace

template <bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const __grid_constant__ RopeAppendParams p) {
  __shared__ float4 cs[kHeadDim / 2];  // m (cos_hi, sin_hi, cos_lo, sin_lo) of pair i
  griddep_wait();  // everything below may come from the preceding kernel
  const int b = static_cast<int>(blockIdx.x) / p.T, t = static_cast<int>(blockIdx.x) - b * p.T;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long tok = static_cast<long long>(blockIdx.x);
  const int n = p.counts ? p.counts[b] : p.T;
  const int s0 = p.slot_start[b];
  const bool seq_ok = n >= 0 && n <= p.T && s0 >= 0 && static_cast<long long>(s0) + n <= p.max_seq;
  if (seq_ok && t >= n) return;
  const int pos = !seq_ok ? 0 : p.positions ? p.positions[tok] : s0 + t;
  if (!seq_ok || pos < 0) {
    if (tid == 0 && (seq_ok || t == 0))
      flag_error(p.err, (seq_ok || s0 < 0) ? GQA_DEVERR_POSITION : GQA_DEVERR_SEQLEN);
    uint4 *dst = reinterpret_cast<uint4 *>(p.q_out + tok * p.Hq * kHeadDim);
    for (int c = tid; c < p.Hq * kHeadDim / 8; c += kRopeThreads) dst[c] = make_uint4(0, 0, 0, 0);
    return;
  }
  if (tid < p.rotary / 2) {
    double sv, cv;
    sincos(static_cast<double>(pos) * p.freq[tid], &sv, &cv);
    sv *= p.magnitude;
    cv *= p.magnitude;
    const float ch = static_cast<float>(cv), sh = static_cast<float>(sv);
    cs[tid] = make_float4(ch, sh, static_cast<float>(cv - ch), static_cast<float>(sv - sh));
  }
  const long long crow = append_row(p, b, s0 + t);
  if (crow < 0 && tid == 0) flag_error(p.err, GQA_DEVERR_PAGE);
  __syncthreads();

  // This lane's place in the rotation: dims 4l .. 4l + 3.
  const bool turns = 4 * lane < p.rotary;
  const int span = p.rotary / 8;  // half layout: lanes between partners
  const bool first = lane < span;
  const int partner = (kInterleaved || !turns) ? lane : first ? lane + span : lane - span;
  float4 c4[kInterleaved ? 2 : 4];
#pragma unroll
  for (int e = 0; e < (kInterleaved ? 2 : 4); ++e) {
    const int i = kInterleaved ? 2 * lane + e : 4 * (first ? lane : lane - span) + e;
    c4[e] = turns ? cs[i] : make_float4(1.f, 0.f, 0.f, 0.f);
  }
  const uint2 none = make_uint2(0x3f803f80u, 0x3f803f80u);  // ones
  const uint2 qw = p.q_norm_w ? reinterpret_cast<const uint2 *>(p.q_norm_w)[lane] : none;
  const uint2 kw = p.k_norm_w ? reinterpret_cast<const uint2 *>(p.k_norm_w)[lane] : none;

  const int rows = p.Hq + (crow >= 0 ? 2 * p.Hkv : 0);
  for (int r = warp; r < rows; r += kRopeThreads / 32) {
    if (r >= p.Hq + p.Hkv) {  // value row: stored as it is
      const int h = r - p.Hq - p.Hkv;
      reinterpret_cast<uint2 *>(p.v_cache + (crow * p.Hkv + h) * kHeadDim)[lane] =
          reinterpret_cast<const uint2 *>(p.v + tok * p.v_stride + h * kHeadDim)[lane];
      continue;
    }
    const bool isq = r < p.Hq;
    const int h = isq ? r : r - p.Hq;
    const uint2 xw = isq ? reinterpret_cast<const uint2 *>(p.q + tok * p.q_stride + h * kHeadDim)[lane]
                         : reinterpret_cast<const uint2 *>(p.k + tok * p.k_stride + h * kHeadDim)[lane];
    const uint2 ww = isq ? qw : kw;
    const bool norm = isq ? p.q_norm_w != nullptr : p.k_norm_w != nullptr;
    const float x[4] = {bf16_lo_to_float(xw.x), bf16_hi_to_float(xw.x), bf16_lo_to_float(xw.y),
                        bf16_hi_to_float(xw.y)};
    float y[4] = {x[0] * bf16_lo_to_float(ww.x), x[1] * bf16_hi_to_float(ww.x), x[2] * bf16_lo_to_float(ww.y),
                  x[3] * bf16_hi_to_float(ww.y)};  // exact: 8-bit significands
    float yp[4];                                   // the partners, with the sign of their term
    if (kInterleaved) {
      yp[0] = -y[1], yp[1] = y[0], yp[2] = -y[3], yp[3] = y[2];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float o = __shfl_sync(0xffffffffu, y[e], partner);
        yp[e] = first ? -o : o;
      }
    }
    if (isq) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float rn = norm ? 1.0f / sqrtf(ss * (1.0f / 128.0f) + p.eps) : 1.0f;
      float z[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 c = c4[kInterleaved ? e >> 1 : e];
        z[e] = rn * (turns ? fmaf(y[e], c.x, yp[e] * c.y) : y[e]);
      }
      reinterpret_cast<uint2 *>(p.q_out + (tok * p.Hq + h) * kHeadDim)[lane] =
          make_uint2(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]));
    } else {
      dw rn = {1.f, 0.f};
      if (norm) {
        dw ss = {0.f, 0.f};
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = dw_add(ss, dw{__fmul_rn(x[e], x[e]), 0.f});
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          ss = dw_add(ss, dw{__shfl_xor_sync(0xffffffffu, ss.hi, o), __shfl_xor_sync(0xffffffffu, ss.lo, o)});
        const dw m = dw_add(dw{__fmul_rn(ss.hi, 1.0f / 128.0f), __fmul_rn(ss.lo, 1.0f / 128.0f)}, dw{p.eps, 0.f});
        const float r0 = __frcp_rn(__fsqrt_rn(m.hi));
        const dw e1 = dw_add(dw{1.f, 0.f}, dw_neg(dw_mul(m, two_prod(r0, r0))));  // 1 - m r0^2
        rn = fast_two_sum(r0, __fmul_rn(__fmul_rn(0.5f, r0), e1.hi));
      }
      uint16_t z[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 c = c4[kInterleaved ? e >> 1 : e];
        const dw turned = turns ? dw_add(dw_mul_f(dw{c.x, c.z}, y[e]), dw_mul_f(dw{c.y, c.w}, yp[e])) : dw{y[e], 0.f};
        z[e] = round_dw_bf16(norm ? dw_mul(turned, rn) : turned);
      }
      reinterpret_cast<uint2 *>(p.k_cache + (crow * p.Hkv + h) * kHeadDim)[lane] =
          make_uint2(static_cast<uint32_t>(z[0]) | (static_cast<uint32_t>(z[1]) << 16),
                     static_cast<uint32_t>(z[2]) | (static_cast<uint32_t>(z[3]) << 16));
    }
  }
}

}  // namespace gqa

using namespace gqa;

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
  if (s.magnitude > 0.f) m = s.magnitude;
  if (freqs) memcpy(freqs, f, sizeof(double) * (r / 2));
  if (magnitude) *magnitude = m;
  return GQA_OK;
}

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
  st = gqa_rope_freqs(rope, p.freq, &p.magnitude);
  if (st != GQA_OK) return st;
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
  p.max_blocks = (d.max_seq_len + kTile - 1) / kTile;
  p.num_blocks = paged ? d.num_cache_blocks : 0;
  p.rotary = rope->rotary_dim;
  p.eps = eps;
  const dim3 grid(static_cast<unsigned>(d.batch) * static_cast<unsigned>(d.num_tokens));
  auto *kernel = rope->layout == GQA_ROPE_INTERLEAVED ? rope_append_kernel<true> : rope_append_kernel<false>;
  if (launch_pdl(kernel, grid, dim3(kRopeThreads), 0, static_cast<cudaStream_t>(stream), p) != cudaSuccess) {
    cudaGetLastError();
    return GQA_ERR_CUDA;
  }
  return GQA_OK;
}
