// The pages of a paged KV cache: fork, resize, copy, keep rows (include/gqa_pages.h).
//
// fork and resize are bookkeeping over a few thousand integers: one CTA each, so that the order
// in which pages are handed out is fixed and the call is one launch.  copy and keep_rows move
// bytes and are bound by HBM: each byte is read once and written once, in 16-byte accesses.
#include <string.h>

#include "../../include/gqa_pages.h"
#include "op_args.h"

namespace gqa {

struct PageState {
  int32_t *refs, *table, *lens;
  uint32_t *err;
  int B, max_blocks, num_blocks;
};

struct PoolSet {
  uint8_t *base[GQA_MAX_POOLS];
  int32_t row16[GQA_MAX_POOLS];  // row_bytes / 16
};

namespace {

constexpr int kStateThreads = 1024;
static_assert(GQA_MAX_BATCH <= kStateThreads, "a thread per sequence");
static_assert(kStateThreads == 1024, "block_scan sums the words of 32 warps");
constexpr int kPageList = 4096;  // free pages handed out per round

__device__ __forceinline__ int pages_of(int len) { return len / kTile + (len % kTile != 0); }

// Reference counts change within the kernel through atomics; read them from L2.
__device__ __forceinline__ int ref_of(const PageState &s, int page) { return __ldcg(s.refs + page); }

// Exclusive prefix sum of one value a thread over the CTA, and the total.  `scratch` holds
// 33 words.  Ends with every thread past its use of scratch.
__device__ __forceinline__ int block_scan(int v, int *scratch, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    scratch[lane] = w;
  }
  __syncthreads();
  const int before = warp > 0 ? scratch[warp - 1] : 0;
  *total = scratch[31];
  __syncthreads();
  return before + x - v;
}

}  // namespace

// ------------------------------------------------------------------------------------ fork
// One CTA: thread i decides whether pair i is valid, then a warp a pair copies table rows and
// counts the pages up.  A source is never any pair's destination, so the pairs do not interact.
__global__ void __launch_bounds__(kStateThreads) pages_fork_kernel(const PageState s, const int32_t *src,
                                                                   const int32_t *dst, int n) {
  __shared__ int s_src[GQA_MAX_BATCH], s_dst[GQA_MAX_BATCH], s_have[GQA_MAX_BATCH];
  griddep_wait();
  const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
  if (i < n) {
    s_src[i] = src[i];
    s_dst[i] = dst[i];
  }
  __syncthreads();
  if (i < n) {
    const int a = s_src[i], b = s_dst[i];
    int have = -1;
    if (a >= 0) {
      if (a >= s.B || b < 0 || b >= s.B) {
        flag_error(s.err, GQA_DEVERR_POSITION);
      } else {
        bool clash = a == b;
        for (int j = 0; j < n; ++j) clash |= s_src[j] >= 0 && ((j < i && s_dst[j] == b) || s_src[j] == b);
        const int la = s.lens[a], lb = s.lens[b];
        if (clash) {
          flag_error(s.err, GQA_DEVERR_CONFLICT);
        } else if (lb != 0 || la < 0 || pages_of(la) > s.max_blocks) {
          flag_error(s.err, GQA_DEVERR_SEQLEN);
        } else {
          have = pages_of(la);
        }
      }
    }
    s_have[i] = have;
  }
  __syncthreads();
  for (int j = warp; j < n; j += kStateThreads / 32) {
    const int have = s_have[j];
    if (have < 0) continue;
    const int32_t *from = s.table + static_cast<long long>(s_src[j]) * s.max_blocks;
    int32_t *to = s.table + static_cast<long long>(s_dst[j]) * s.max_blocks;
    bool ok = true;
    for (int c = lane; c < have; c += 32) {
      const int page = from[c];
      ok = ok && page >= 0 && page < s.num_blocks && ref_of(s, page) > 0;
    }
    if (!__all_sync(0xffffffffu, ok)) {
      if (lane == 0) flag_error(s.err, GQA_DEVERR_PAGE);
      continue;
    }
    for (int c = lane; c < have; c += 32) {
      const int page = from[c];
      to[c] = page;
      atomicAdd(s.refs + page, 1);
    }
    if (lane == 0) s.lens[s_dst[j]] = s.lens[s_src[j]];
  }
}

// ---------------------------------------------------------------------------------- resize
// One CTA, a thread a sequence for its lengths, a warp a sequence for the pages it drops:
//   1 which sequences change, and whether the pages they drop are theirs to drop
//   2 drop them (counts only)
//   3 which growing sequences need their last page split, the pages each one needs, their sum
//   4 the free pages, counted a contiguous chunk a thread; too few: put 2 back and stop
//   5 the free pages in ascending order to the sequences in order
//   6 table entries of dropped pages, lengths, the counts of split pages
__global__ void __launch_bounds__(kStateThreads) pages_resize_kernel(const PageState s, const int32_t *new_lens,
                                                                     int32_t *cow_src, int32_t *cow_dst) {
  __shared__ int s_have[GQA_MAX_BATCH], s_need[GQA_MAX_BATCH], s_last[GQA_MAX_BATCH], s_first[GQA_MAX_BATCH + 1];
  __shared__ int s_list[kPageList];
  __shared__ int scratch[33];
  griddep_wait();
  const int b = threadIdx.x, lane = b & 31, warp = b >> 5;
  int len = 0, want = 0, have = 0, need = 0;
  bool active = false;
  if (b < s.B) {
    len = s.lens[b];
    want = new_lens[b];
    if (want >= 0) {
      have = len >= 0 ? pages_of(len) : 0;
      need = pages_of(want);
      active = len >= 0 && have <= s.max_blocks && need <= s.max_blocks;
      if (!active) flag_error(s.err, GQA_DEVERR_SEQLEN);
    }
    if (!active) have = need = 0;
    s_have[b] = have;
    s_need[b] = need;
    cow_src[b] = -1;
    cow_dst[b] = -1;
  }
  __syncthreads();
  for (int j = warp; j < s.B; j += kStateThreads / 32) {
    const int lo = s_need[j], hi = s_have[j];
    if (lo >= hi) continue;
    bool ok = true;
    for (int c = lo + lane; c < hi; c += 32) {
      const int page = s.table[static_cast<long long>(j) * s.max_blocks + c];
      ok = ok && page >= 0 && page < s.num_blocks && ref_of(s, page) > 0;
    }
    if (!__all_sync(0xffffffffu, ok) && lane == 0) {
      flag_error(s.err, GQA_DEVERR_PAGE);
      s_have[j] = s_need[j] = -1;  // left as it is
    }
  }
  __syncthreads();
  if (b < s.B && s_have[b] < 0) active = false, have = need = 0, s_have[b] = s_need[b] = 0;
  __syncthreads();
  for (int j = warp; j < s.B; j += kStateThreads / 32)
    for (int c = s_need[j] + lane; c < s_have[j]; c += 32)
      atomicAdd(s.refs + s.table[static_cast<long long>(j) * s.max_blocks + c], -1);
  int last = -1;  // (the barrier below orders the counts before they are read; no fence: it costs 2 us)
  if (active && want > len && len % kTile != 0) {
    last = s.table[static_cast<long long>(b) * s.max_blocks + have - 1];
    if (last < 0 || last >= s.num_blocks) last = -2;
  }
  __syncthreads();  // the counts are down
  if (last >= 0 && ref_of(s, last) < 1) last = -2;
  if (last == -2) {
    flag_error(s.err, GQA_DEVERR_PAGE);
    active = false;
    last = -1;
    have = need = 0;
    s_have[b] = s_need[b] = 0;
  }
  if (b < s.B) s_last[b] = last;
  __syncthreads();
  bool cow = false;
  if (last >= 0) {
    const int held = ref_of(s, last);
    if (held > 1) {
      int before = 0;  // sequences before this one that leave the page
      for (int j = 0; j < b; ++j) before += s_last[j] == last;
      cow = held - before > 1;
    }
  }
  int total = 0;
  const int adds = (need > have ? need - have : 0) + (cow ? 1 : 0);
  const int first = block_scan(adds, scratch, &total);
  if (b < s.B) s_first[b] = first;
  if (b == 0) s_first[s.B] = total;
  if (total > 0) {
    const int chunk = (s.num_blocks + kStateThreads - 1) / kStateThreads;
    const long long p0 = static_cast<long long>(b) * chunk;
    const int pages = static_cast<int>(p0 >= s.num_blocks ? 0 : min(static_cast<long long>(chunk), s.num_blocks - p0));
    int mine = 0, nfree = 0;
    for (int c = 0; c < pages; ++c) mine += ref_of(s, static_cast<int>(p0) + c) <= 0;
    const int rank0 = block_scan(mine, scratch, &nfree);
    if (nfree < total) {
      for (int j = warp; j < s.B; j += kStateThreads / 32)
        for (int c = s_need[j] + lane; c < s_have[j]; c += 32)
          atomicAdd(s.refs + s.table[static_cast<long long>(j) * s.max_blocks + c], 1);
      if (b == 0) flag_error(s.err, GQA_DEVERR_NOPAGE);
      return;
    }
    for (int base = 0; base < total; base += kPageList) {
      const int upto = min(total, base + kPageList);
      if (rank0 < upto && rank0 + mine > base) {
        int rank = rank0;
        for (int c = 0; c < pages && rank < upto; ++c) {
          const int page = static_cast<int>(p0) + c;
          if (ref_of(s, page) > 0) continue;
          if (rank >= base) s_list[rank - base] = page;
          ++rank;
        }
      }
      __syncthreads();
      for (int k = base + b; k < upto; k += kStateThreads) {
        int lo = 0, hi = s.B - 1;  // the sequence that takes the k-th page: s_first[lo] <= k < s_first[lo + 1]
        while (lo < hi) {
          const int mid = (lo + hi + 1) / 2;
          if (s_first[mid] <= k) lo = mid; else hi = mid - 1;
        }
        const int page = s_list[k - base], idx = k - s_first[lo];
        const int grow = max(0, s_need[lo] - s_have[lo]);
        const bool split = s_first[lo + 1] - s_first[lo] > grow;
        const int col = split ? s_have[lo] - 1 + idx : s_have[lo] + idx;
        s.table[static_cast<long long>(lo) * s.max_blocks + col] = page;
        if (split && idx == 0) cow_dst[lo] = page;
      }
      __syncthreads();
    }
    // the counts of the pages taken, once every round has seen which were free
    for (int c = 0, rank = rank0; c < pages && rank < total; ++c) {
      const int page = static_cast<int>(p0) + c;
      if (ref_of(s, page) > 0) continue;
      s.refs[page] = 1;
      ++rank;
    }
  }
  __syncthreads();
  if (cow) {
    cow_src[b] = last;
    atomicAdd(s.refs + last, -1);
  }
  for (int j = warp; j < s.B; j += kStateThreads / 32)
    for (int c = s_need[j] + lane; c < s_have[j]; c += 32) {
      int32_t *at = s.table + static_cast<long long>(j) * s.max_blocks + c;
      if (atomicMax(s.refs + *at, 0) < 0) flag_error(s.err, GQA_DEVERR_PAGE);  // more holders than its count said
      *at = -1;
    }
  if (active) s.lens[b] = want;
}

// ------------------------------------------------------------------------------------ copy
// One CTA per (pair, pool): 64 rows, 16 bytes a thread and access, eight accesses in flight.
constexpr int kCopyThreads = 256;
constexpr int kCopyDepth = 8;
__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const __grid_constant__ PoolSet pools,
                                                                  const int32_t *src, const int32_t *dst, int n,
                                                                  int num_blocks, uint32_t *err) {
  griddep_wait();
  const int i = static_cast<int>(blockIdx.x), tid = threadIdx.x;
  const int a = src[i], b = dst[i];
  if (a < 0) return;
  if (a >= num_blocks || b < 0 || b >= num_blocks) {
    if (tid == 0 && blockIdx.y == 0) flag_error(err, GQA_DEVERR_PAGE);
    return;
  }
  if (a == b) return;
  bool clash = false;
  for (int j = tid; j < n; j += kCopyThreads) {
    const int aj = src[j];
    clash |= aj >= 0 && j != i && ((j < i && dst[j] == b) || aj == b);
  }
  if (__syncthreads_or(clash)) {
    if (tid == 0 && blockIdx.y == 0) flag_error(err, GQA_DEVERR_CONFLICT);
    return;
  }
  const long long page16 = static_cast<long long>(pools.row16[blockIdx.y]) * kTile;
  const uint4 *from = reinterpret_cast<const uint4 *>(pools.base[blockIdx.y]) + a * page16;
  uint4 *to = reinterpret_cast<uint4 *>(pools.base[blockIdx.y]) + b * page16;
  for (long long c = tid; c < page16; c += kCopyThreads * kCopyDepth) {
    uint4 x[kCopyDepth];
#pragma unroll
    for (int e = 0; e < kCopyDepth; ++e)
      if (c + e * kCopyThreads < page16) x[e] = __ldcs(from + c + e * kCopyThreads);
#pragma unroll
    for (int e = 0; e < kCopyDepth; ++e)
      if (c + e * kCopyThreads < page16) to[c + e * kCopyThreads] = x[e];
  }
}

// ------------------------------------------------------------------------------- keep rows
struct KeepParams {
  const int32_t *table, *start, *keep, *counts;
  uint32_t *err;
  int max_keep, max_seq, max_blocks, num_blocks, paged;
  int pools, per;  // pools, and those of a CTA
  int cols;        // 16-byte columns of a row that a CTA moves
};

// One CTA per (some pools, sequence, slice of the row's columns).  Row keep[i] goes to row
// i <= keep[i]: rows taken in ascending order, a group at a time, a group read whole before it is
// written, never overwrite one that is still to be read (the reads left have keep[j] >= j > every
// row written), so the next group is read before the group at hand is written.  Entries with
// keep[i] = i, a prefix of the list, move nothing.
//   Bound by HBM when CTAs enough have work: the host cuts the rows into slices (of 256 bytes at
// least) where there are few pools and sequences (16 pools x 4 sequences, half of 8000 rows kept:
// 493 us with whole rows, 175 us in slices), and gives a CTA several pools where there are many,
// so that a list is checked less often (80 pools x 32 sequences, 5 rows each: 15 us with a CTA a
// pool, 10.7 us with five pools a CTA).
constexpr int kKeepThreads = 256;
constexpr int kKeepDepth = 4;   // rows a thread holds of a group
constexpr int kKeepLanes = 64;  // rows side by side, at most
constexpr int kKeepRing = 2048; // entries whose rows are known, in shared memory; filled by halves
static_assert(3 * kKeepDepth * kKeepLanes <= kKeepRing / 2, "three groups are in use while a half is filled");
__global__ void __launch_bounds__(kKeepThreads) keep_rows_kernel(const __grid_constant__ PoolSet pools,
                                                                 const KeepParams p) {
  __shared__ int s_still;
  __shared__ int2 s_rows[kKeepRing];  // (from, to) cache rows of entry i at i % kKeepRing
  griddep_wait();
  const int b = static_cast<int>(blockIdx.y), tid = threadIdx.x;
  const int n = p.counts[b], s0 = p.start[b];
  const bool lead = tid == 0 && blockIdx.x == 0 && blockIdx.z == 0;
  if (n == 0) return;
  if (n < 0 || n > p.max_keep) {
    if (lead) flag_error(p.err, GQA_DEVERR_SEQLEN);
    return;
  }
  const int32_t *list = p.keep + static_cast<long long>(b) * p.max_keep;
  const int32_t *pages = p.table + static_cast<long long>(b) * p.max_blocks;
  if (tid == 0) s_still = 0;
  // cache row of a slot (below 2^31); the page ids have been checked
  auto row_of = [&](int slot) {
    if (!p.paged) return b * p.max_seq + slot;
    return pages[slot / kTile] * kTile + (slot & (kTile - 1));
  };
  auto page_ok = [&](int slot) {
    const int pg = pages[slot / kTile];
    return pg >= 0 && pg < p.num_blocks;
  };
  bool bad = s0 < 0, bad_page = false;
  int still = 0;  // entries with keep[i] == i
  if (!bad)
    for (int i = tid; i < n; i += kKeepThreads) {
      const int at = list[i], before = i > 0 ? list[i - 1] : -1;
      if (at <= before || static_cast<long long>(s0) + at >= p.max_seq) {
        bad = true;
      } else {
        still += at == i;
        if (p.paged && at != i) bad_page = bad_page || !page_ok(s0 + at) || !page_ok(s0 + i);
      }
    }
  if (__syncthreads_or(bad || bad_page)) {
    const int any_bad = __syncthreads_or(bad);
    if (lead) flag_error(p.err, any_bad ? GQA_DEVERR_POSITION : GQA_DEVERR_PAGE);
    return;
  }
  // the prefix that stays (ascending entries: keep[i] == i implies it for all before)
  if (still) atomicAdd(&s_still, still);
  __syncthreads();
  const int i0 = s_still;
  if (i0 >= n) return;

  int filled = i0;  // entries below it have been put into the ring
  auto fill = [&](int count) {
    const int upto = min(n, filled + count);
    for (int i = filled + tid; i < upto; i += kKeepThreads)
      s_rows[i % kKeepRing] = make_int2(row_of(s0 + list[i]), row_of(s0 + i));
    filled = upto;
  };
  fill(kKeepRing);
  __syncthreads();

  // The groups to move, one after another: pool k, columns from cb, entries from g on.  rl and col are the
  // thread's row in the group's first `lanes` and its column.
  struct Group {
    int k, cb, g, lanes, rl, col;
  };
  const int k1 = min(p.pools, (static_cast<int>(blockIdx.x) + 1) * p.per);
  const int c0 = static_cast<int>(blockIdx.z) * p.cols;
  auto place = [&](Group &x) {  // the thread's place once k and cb are set; past pools narrower than cb
    while (x.k < k1) {
      const int c1 = min(pools.row16[x.k], c0 + p.cols);
      if (x.cb < c1) {
        const int width = min(c1 - x.cb, kKeepThreads);
        x.lanes = min(kKeepLanes, kKeepThreads / width);
        x.rl = tid / width;
        x.col = x.cb + tid - x.rl * width;
        return;
      }
      ++x.k;
      x.cb = c0;
    }
  };
  auto next = [&](Group x) {
    x.g += x.lanes * kKeepDepth;
    if (x.g >= n) {
      x.g = i0;
      x.cb += kKeepThreads;
      place(x);
    }
    return x;
  };
  auto at = [&](const Group &x, int row) {
    return reinterpret_cast<uint4 *>(pools.base[x.k]) + static_cast<long long>(row) * pools.row16[x.k] + x.col;
  };
  auto read = [&](const Group &x, uint4 (&v)[kKeepDepth]) {
#pragma unroll
    for (int e = 0; e < kKeepDepth; ++e) {
      const int i = x.g + e * x.lanes + x.rl;
      if (x.rl < x.lanes && i < n) v[e] = __ldcg(at(x, s_rows[i % kKeepRing].x));
    }
  };
  auto write = [&](const Group &x, const uint4 (&v)[kKeepDepth]) {
#pragma unroll
    for (int e = 0; e < kKeepDepth; ++e) {
      const int i = x.g + e * x.lanes + x.rl;
      if (x.rl < x.lanes && i < n) __stcg(at(x, s_rows[i % kKeepRing].y), v[e]);
    }
  };
  // One step: group x is in u; the group after it is read into v, x is written, and the rows the group
  // after that will need are looked up.  Where a new pool or column block starts over and its first
  // entries have left the ring, the ring is filled anew first.
  const bool once = n - i0 <= kKeepRing;
  auto step = [&](const Group &x, const uint4 (&u)[kKeepDepth], uint4 (&v)[kKeepDepth]) {
    const Group y = next(x);
    __syncthreads();  // every thread has read group x, and the rows of group y are known
    const bool over = y.k < k1 && y.g <= x.g && !once;
    if (y.k < k1 && !over) read(y, v);
    write(x, u);
    if (over) {
      __syncthreads();
      filled = i0;
      fill(kKeepRing);
      __syncthreads();
      read(y, v);
    } else if (y.k < k1 && filled < n && y.g + 2 * y.lanes * kKeepDepth > filled) {
      fill(kKeepRing / 2);
    }
    return y;
  };
  Group x{static_cast<int>(blockIdx.x) * p.per, c0, i0, 1, 0, 0};
  place(x);
  uint4 u[kKeepDepth], v[kKeepDepth];
  if (x.k < k1) read(x, u);
  while (x.k < k1) {
    x = step(x, u, v);
    if (x.k >= k1) break;
    x = step(x, v, u);
  }
}

// --------------------------------------------------------------------------------- host side

namespace {

gqa_status_t check_state(const gqa_pages_desc_t *desc, const void *refs, const void *table, const void *lens,
                         const void *err) {
  if (!desc || !refs || !table || !lens) return GQA_ERR_INVALID_ARG;
  if (desc->batch < 1 || desc->batch > GQA_MAX_BATCH || desc->max_blocks < 1 || desc->num_blocks < 1 ||
      desc->num_blocks >= (1 << 25) || static_cast<long long>(desc->batch) * desc->max_blocks > 0x7fffffffLL)
    return GQA_ERR_INVALID_ARG;
  if (!aligned_to(refs, 4) || !aligned_to(table, 4) || !aligned_to(lens, 4) || !aligned_to(err, 4))
    return GQA_ERR_INVALID_ARG;
  return GQA_OK;
}

gqa_status_t take_pools(const gqa_pool_t *pools, int n, PoolSet *set) {
  if (!pools || n < 1 || n > GQA_MAX_POOLS) return GQA_ERR_INVALID_ARG;
  memset(set, 0, sizeof *set);
  for (int i = 0; i < n; ++i) {
    if (!pools[i].base || !aligned_to(pools[i].base, 16)) return GQA_ERR_INVALID_ARG;
    if (pools[i].row_bytes < 16 || pools[i].row_bytes > (1 << 20) || pools[i].row_bytes % 16 != 0)
      return GQA_ERR_INVALID_ARG;
    set->base[i] = static_cast<uint8_t *>(pools[i].base);
    set->row16[i] = static_cast<int32_t>(pools[i].row_bytes / 16);
  }
  return GQA_OK;
}

PageState state_of(const gqa_pages_desc_t &d, int32_t *refs, int32_t *table, int32_t *lens, uint32_t *err) {
  return PageState{refs, table, lens, err, d.batch, d.max_blocks, d.num_blocks};
}

gqa_status_t launched(cudaError_t e) {
  if (e == cudaSuccess) return GQA_OK;
  cudaGetLastError();
  return GQA_ERR_CUDA;
}

}  // namespace

}  // namespace gqa

using namespace gqa;

extern "C" gqa_status_t gqa_pages_fork(const gqa_pages_desc_t *desc, int32_t *ref_counts, int32_t *page_table,
                                       int32_t *seq_lens, const int32_t *src, const int32_t *dst, int num_pairs,
                                       uint32_t *device_errors, void *stream) {
  gqa_status_t st = check_state(desc, ref_counts, page_table, seq_lens, device_errors);
  if (st != GQA_OK) return st;
  if (!src || !dst || !aligned_to(src, 4) || !aligned_to(dst, 4) || num_pairs < 1 || num_pairs > GQA_MAX_BATCH)
    return GQA_ERR_INVALID_ARG;
  const gqa_pages_desc_t d = *desc;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  return launched(launch_pdl(pages_fork_kernel, dim3(1), dim3(kStateThreads), 0, static_cast<cudaStream_t>(stream),
                             state_of(d, ref_counts, page_table, seq_lens, device_errors), src, dst, num_pairs));
}

extern "C" gqa_status_t gqa_pages_resize(const gqa_pages_desc_t *desc, int32_t *ref_counts, int32_t *page_table,
                                         int32_t *seq_lens, const int32_t *new_lens, int32_t *cow_src,
                                         int32_t *cow_dst, uint32_t *device_errors, void *stream) {
  gqa_status_t st = check_state(desc, ref_counts, page_table, seq_lens, device_errors);
  if (st != GQA_OK) return st;
  if (!new_lens || !cow_src || !cow_dst || !aligned_to(new_lens, 4) || !aligned_to(cow_src, 4) ||
      !aligned_to(cow_dst, 4))
    return GQA_ERR_INVALID_ARG;
  const gqa_pages_desc_t d = *desc;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  return launched(launch_pdl(pages_resize_kernel, dim3(1), dim3(kStateThreads), 0, static_cast<cudaStream_t>(stream),
                             state_of(d, ref_counts, page_table, seq_lens, device_errors), new_lens, cow_src,
                             cow_dst));
}

extern "C" gqa_status_t gqa_pages_copy(const gqa_pool_t *pools, int num_pools, int num_blocks, const int32_t *src,
                                       const int32_t *dst, int num_pairs, int device, uint32_t *device_errors,
                                       void *stream) {
  PoolSet set;
  gqa_status_t st = take_pools(pools, num_pools, &set);
  if (st != GQA_OK) return st;
  if (!src || !dst || !aligned_to(src, 4) || !aligned_to(dst, 4) || !aligned_to(device_errors, 4) || num_pairs < 1 ||
      num_pairs > GQA_MAX_PAGE_PAIRS || num_blocks < 1 || num_blocks >= (1 << 25))
    return GQA_ERR_INVALID_ARG;
  st = check_device(device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(device);
  if (!guard.ok) return GQA_ERR_CUDA;
  return launched(launch_pdl(pages_copy_kernel, dim3(static_cast<unsigned>(num_pairs), static_cast<unsigned>(num_pools)),
                             dim3(kCopyThreads), 0, static_cast<cudaStream_t>(stream), set, src, dst, num_pairs,
                             num_blocks, device_errors));
}

extern "C" gqa_status_t gqa_cache_keep_rows(const gqa_keep_desc_t *desc, const gqa_pool_t *pools, int num_pools,
                                            const int32_t *page_table, const int32_t *start, const int32_t *keep,
                                            const int32_t *counts, uint32_t *device_errors, void *stream) {
  if (!desc) return GQA_ERR_INVALID_ARG;
  const gqa_keep_desc_t d = *desc;
  if (d.batch < 1 || d.batch > GQA_MAX_BATCH || d.max_seq_len < 1 || d.max_keep < 1 || d.max_keep > d.max_seq_len)
    return GQA_ERR_INVALID_ARG;
  if (d.block_size != 0 && d.block_size != GQA_BLOCK_SIZE) return GQA_ERR_UNSUPPORTED;
  const bool paged = d.block_size > 0;
  if (paged && d.num_blocks < 1) return GQA_ERR_INVALID_ARG;
  const long long rows = paged ? static_cast<long long>(d.num_blocks) * kTile
                               : static_cast<long long>(d.batch) * d.max_seq_len;
  if (rows > 0x7fffffffLL || d.max_keep > (1 << 30)) return GQA_ERR_UNSUPPORTED;  // (entries are counted in int32 steps)
  if (paged != (page_table != nullptr) || !start || !keep || !counts) return GQA_ERR_INVALID_ARG;
  if (!aligned_to(page_table, 4) || !aligned_to(start, 4) || !aligned_to(keep, 4) || !aligned_to(counts, 4) ||
      !aligned_to(device_errors, 4))
    return GQA_ERR_INVALID_ARG;
  PoolSet set;
  gqa_status_t st = take_pools(pools, num_pools, &set);
  if (st != GQA_OK) return st;
  st = check_device(d.device);
  if (st != GQA_OK) return st;
  DeviceGuard guard(d.device);
  if (!guard.ok) return GQA_ERR_CUDA;
  KeepParams p;
  memset(&p, 0, sizeof p);
  p.table = page_table;
  p.start = start;
  p.keep = keep;
  p.counts = counts;
  p.err = device_errors;
  p.max_keep = d.max_keep;
  p.max_seq = d.max_seq_len;
  p.max_blocks = capacity_tiles(d.max_seq_len);
  p.num_blocks = paged ? d.num_blocks : 0;
  p.paged = paged ? 1 : 0;
  int widest = 1, sms = 0;
  for (int i = 0; i < num_pools; ++i) widest = set.row16[i] > widest ? set.row16[i] : widest;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d.device) != cudaSuccess) return launched(cudaErrorUnknown);
  // three CTAs an SM: pools together where there are more (pool, sequence) pairs, slices of the rows
  // (16 columns, 256 bytes, at least) where there are fewer
  const long long pairs = static_cast<long long>(num_pools) * d.batch, want = 3LL * sms;
  long long per = pairs / want, slices = (want + pairs - 1) / pairs;
  per = per < 1 ? 1 : per > num_pools ? num_pools : per;
  const long long most = (widest + 15) / 16;
  slices = slices > most ? most : slices;
  p.pools = num_pools;
  p.per = static_cast<int>(per);
  p.cols = static_cast<int>((widest + slices - 1) / slices);
  slices = (widest + p.cols - 1) / p.cols;
  return launched(launch_pdl(keep_rows_kernel, dim3(static_cast<unsigned>((num_pools + per - 1) / per), static_cast<unsigned>(d.batch),
                                                    static_cast<unsigned>(slices)),
                             dim3(kKeepThreads), 0, static_cast<cudaStream_t>(stream), set, p));
}
