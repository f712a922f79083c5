// fa_tokens.cuh -- where the rows of packed sequences and the new tokens of a paged cache belong, and
// the codes in which E4M3 pools hold them: one rule for all kernels that write them, so that the appends
// with and without norms leave out the same tokens and quantise alike.
#pragma once
#include "fa_internal.h"

#include <cuda_fp8.h>

namespace fa {

// The sequence b that a thread has looked up last, with rows [lo, hi) of the packed ones, and the row up
// to which the look-ups of later rows end there, too (hi, where the offsets ascend).
struct Sequence {
  int lo, hi, b, to;
};
// Whether packed row n lies in the last sequence that begins at n or before; then seq is that one.  A
// thread asks for rows in ascending order, beginning with to = 0.  Offsets that are not ascending may
// lead to a sequence that does not hold n, which the comparison refuses, or to one of several that do,
// whatever rows were asked for before: below `to` every comparison goes the way it went.
__device__ __forceinline__ bool find_sequence(const int* cu, int n_seq, int n, Sequence& seq) {
  if (n < seq.to) return true;
  int lo = 0, hi = n_seq, to = 0x7fffffff;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1, c = cu[mid];
    if (c <= n) {
      lo = mid;
    } else {
      hi = mid;
      to = min(to, c);
    }
  }
  seq = {cu[lo], cu[lo + 1], lo, 0};
  if (n < seq.lo || n >= seq.hi) return false;
  seq.to = min(to, seq.hi);
  return true;
}

// The sequence b and key position pos of new token t: its sequence's last token is its last key.
// Without offsets every sequence has one.  false: the token belongs to no sequence or lies before its
// sequence's first key.
__device__ __forceinline__ bool locate_token(const PagedView& pg, const int* cu, int n_seq, int t,
                                             Sequence& seq, int& b, int& pos) {
  b = t;
  int end = t + 1;
  if (cu) {
    if (!find_sequence(cu, n_seq, t, seq)) return false;
    b = seq.b;
    end = seq.hi;
  }
  const long long p = static_cast<long long>(pg.seqlens[b]) - (end - t);
  pos = static_cast<int>(p);
  return p >= 0;
}
// The page that holds key pos of sequence b, page pi of its table, as the table has it; -1 past the table.
__device__ __forceinline__ int page_id(const PagedView& pg, int b, int pos, int& pi) {
  pi = static_cast<int>(pg.page.quot(pos));
  return pi < pg.max_pages ? pg.table[b * pg.table_stride + pi] : -1;
}

// 8 values times inv as E4M3 codes, nearest even, saturated to +-448 (NaN stays NaN).
__device__ __forceinline__ uint2 codes8(const float2 (&x)[4], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[i].x * inv, x[i].y * inv), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

}  // namespace fa
