// What the kernels over an 8-bit KV cache (include/gqa_q8.h) share: the formats, and where a
// packed row or a slot lies.
#pragma once

#include "../../include/gqa_q8.h"
#include <cuda_fp16.h>

#include "op_args.h"

namespace gqa {

// Geometry and format checks of a call (q8_rows.cu).
gqa_status_t q8_check(const gqa_q8_desc_t &d, bool attn);

// Four e4m3 codes as binary16 pairs; exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// Four codes, c0 in the low byte, as binary16 pairs (c0, c1) and (c2, c3); exact.  An int8 code c
// is put, as c + 128, under the exponent of 1024: 1024 + 128 + c, less 1152.
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
  if (FMT == GQA_Q8_E4M3) {
    e4m3x4_to_f16(x, lo, hi);
  } else {
    const uint32_t u = x ^ 0x80808080u;
    lo = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
  }
}

// The sequence that packed row n belongs to, or -1: the last b of the batch with offsets[b] <= n, if n
// is below offsets[b + 1] too.
__device__ __forceinline__ int sequence_of_row(const int32_t *offsets, int B, int n, int *first, int *end) {
  int b = 0, above = B;
  while (above - b > 1) {
    const int mid = (b + above) / 2;
    if (offsets[mid] <= n) b = mid;
    else above = mid;
  }
  *first = offsets[b];
  *end = offsets[b + 1];
  return *first <= n && n < *end ? b : -1;
}

}  // namespace gqa
