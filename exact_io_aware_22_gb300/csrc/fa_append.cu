// fa_append.cu -- new tokens' keys and values into a paged cache, with the rotary position
// rotation applied on the way, and the same tokens' queries rotated by the same launch.
//
// Mathematics.  A token at position p turns each pair (x, y) of the first `rot` columns of
// its query and key heads by the pair's angle a(p), read from the caller's table:
//     x' = x cos a - y sin a,    y' = y cos a + x sin a
// with pairs (i, i + rot/2) or, interleaved, (2i, 2i + 1).  Values and the other columns
// are copied.  fp32 arithmetic, one rounding to 16 bits, or (E4M3 caches) one rounding of
// x' / scale to E4M3.
//
// Bound: bytes.  Every input and output element moves once; the table row of a token is read
// by all its heads and stays in L1.  One thread carries 16 elements (two 16-byte loads, two
// stores) -- both halves of 8 pairs -- so a rotation needs no exchange between threads.
// The token's data are loaded before its position is known: finding the sequence, its length
// and the page is a chain of dependent loads that the data loads then hide.  All loads are
// plain ones, not read-only-path ones: earlier work in the stream may still be writing their
// sources when this kernel starts, and nothing may move them above grid_dep_wait().
#include "fa_internal.h"
#include "fa_ptx.cuh"

#include <cuda_fp8.h>

namespace fa {

namespace {

constexpr int APP_THREADS = 128;

// The sequence b and key position pos of token t; false for a token that belongs to no
// sequence or lies before its sequence's first key.
__device__ __forceinline__ bool locate(const AppendArgs& a, int t, int& b, int& pos) {
  int end;
  if (!a.cu) {
    b = t;
    end = t + 1;
  } else {
    // last b with cu[b] <= t; offsets that are not ascending may lead to a sequence that
    // does not hold t, which the comparison below refuses
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    b = lo;
    end = a.cu[b + 1];
    if (a.cu[b] > t || end <= t) return false;
  }
  const long long p = static_cast<long long>(a.pg.seqlens[b]) - (end - t);
  pos = static_cast<int>(p);
  return p >= 0;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8], bool bf16) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = bf16 ? unpack2<true>(u[i]) : unpack2<false>(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                    pack2<BF16>(x[6], x[7]));
}
// 8 values times inv as E4M3 codes, nearest even, saturated to +-448 (NaN stays NaN).
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * inv, x[2 * i + 1] * inv), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// One thread per (token, head of Q|K|V, 16 columns).
template <int D, bool BF16, bool C8, bool INTER>
__global__ void __launch_bounds__(APP_THREADS) append_kernel(const AppendArgs a) {
  grid_dep_wait();                               // inputs written, cache rows free to overwrite
  constexpr int IPH = D / 16;                    // items per head
  const int heads = (a.Q ? a.H : 0) + 2 * a.Hkv;
  const long long item = static_cast<long long>(blockIdx.x) * APP_THREADS + threadIdx.x;
  const int per_tok = heads * IPH;
  const long long tl = item / per_tok;
  if (tl >= a.T) return;
  const int t = static_cast<int>(tl);
  const int rem = static_cast<int>(item - tl * per_tok);
  int head = rem / IPH;
  const int j = rem % IPH;
  // which tensor: keys first, then values, then queries
  const int kind = head < a.Hkv ? 0 : head < 2 * a.Hkv ? 1 : 2;
  head -= kind * a.Hkv;
  const bool turn = kind != 1 && j < a.rot / 16;
  // the item's two 8-column chunks
  const int c0 = !INTER && turn ? 8 * j : 16 * j;
  const int c1 = !INTER && turn ? 8 * j + a.rot / 2 : 16 * j + 8;

  const uint16_t* src = static_cast<const uint16_t*>(kind == 0 ? a.K : kind == 1 ? a.V : a.Q) +
                        t * (kind == 0 ? a.k_stride : kind == 1 ? a.v_stride : a.q_stride) +
                        static_cast<long long>(head) * D;
  const uint4 w0 = *reinterpret_cast<const uint4*>(src + c0);
  const uint4 w1 = *reinterpret_cast<const uint4*>(src + c1);

  int b, pos;
  if (!locate(a, t, b, pos)) return;
  float x[8], y[8];
  unpack8(w0, x, BF16);
  unpack8(w1, y, BF16);
  if (turn) {
    const int ang = a.positions ? a.positions[t] : pos;
    if (ang < 0 || ang >= a.max_pos) {
      atomicOr(a.ctl.status, FA_DEV_BAD_INDEX);
      return;
    }
    const float* cs = a.cos_sin + static_cast<long long>(ang) * a.rot + 8 * j;
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 cc = *reinterpret_cast<const float4*>(cs + i);
      const float4 ss = *reinterpret_cast<const float4*>(cs + a.rot / 2 + i);
      c[i] = cc.x; c[i + 1] = cc.y; c[i + 2] = cc.z; c[i + 3] = cc.w;
      s[i] = ss.x; s[i + 1] = ss.y; s[i + 2] = ss.z; s[i + 3] = ss.w;
    }
    if constexpr (INTER) {                       // pairs inside a chunk: x holds 4 pairs, y 4
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float p = x[i], q = x[i + 1], u = y[i], v = y[i + 1];
        x[i] = p * c[i / 2] - q * s[i / 2];
        x[i + 1] = q * c[i / 2] + p * s[i / 2];
        y[i] = u * c[4 + i / 2] - v * s[4 + i / 2];
        y[i + 1] = v * c[4 + i / 2] + u * s[4 + i / 2];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = x[i], q = y[i];
        x[i] = p * c[i] - q * s[i];
        y[i] = q * c[i] + p * s[i];
      }
    }
  }
  if (kind == 2) {
    uint16_t* dst = static_cast<uint16_t*>(a.Qout) + (static_cast<long long>(t) * a.H + head) * D;
    *reinterpret_cast<uint4*>(dst + c0) = pack8<BF16>(x);
    *reinterpret_cast<uint4*>(dst + c1) = pack8<BF16>(y);
    return;
  }
  const int pi = static_cast<int>(a.pg.page.quot(pos));
  const int id = pi < a.pg.max_pages ? a.pg.table[b * a.pg.table_stride + pi] : -1;
  if (id < 0 || id >= a.pg.pages) {
    atomicOr(a.ctl.status, FA_DEV_BAD_INDEX);
    return;
  }
  const long long at = id * a.page_stride + head * a.head_stride +
                       (pos - pi * static_cast<int>(a.pg.page.div)) * a.row_stride;
  void* pool = kind == 0 ? a.Kc : a.Vc;
  if constexpr (C8) {
    uint8_t* dst = static_cast<uint8_t*>(pool) + at;
    const float inv = kind == 0 ? a.k_inv : a.v_inv;
    *reinterpret_cast<uint2*>(dst + c0) = codes8(x, inv);
    *reinterpret_cast<uint2*>(dst + c1) = codes8(y, inv);
  } else {
    uint16_t* dst = static_cast<uint16_t*>(pool) + at;
    *reinterpret_cast<uint4*>(dst + c0) = pack8<BF16>(x);
    *reinterpret_cast<uint4*>(dst + c1) = pack8<BF16>(y);
  }
}

template <int D, bool BF16, bool C8>
cudaError_t launch_append_t(const AppendArgs& a, bool interleaved, cudaStream_t st) {
  const long long items =
      static_cast<long long>(a.T) * ((a.Q ? a.H : 0) + 2 * a.Hkv) * (D / 16);
  const long long grid = (items + APP_THREADS - 1) / APP_THREADS;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = interleaved ? append_kernel<D, BF16, C8, true> : append_kernel<D, BF16, C8, false>;
  return launch_dependent(kern, static_cast<unsigned>(grid), APP_THREADS, 0, st, a);
}

template <int D>
cudaError_t launch_append_d(const AppendArgs& a, bool bf16, bool c8, bool inter, cudaStream_t st) {
  if constexpr (D == 128)
    if (c8)
      return bf16 ? launch_append_t<D, true, true>(a, inter, st)
                  : launch_append_t<D, false, true>(a, inter, st);
  return bf16 ? launch_append_t<D, true, false>(a, inter, st)
              : launch_append_t<D, false, false>(a, inter, st);
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, int d, bool bf16, bool c8, bool interleaved,
                          cudaStream_t st) {
  if (c8 && d != 128) return cudaErrorInvalidValue;
  if (d == 32) return launch_append_d<32>(a, bf16, c8, interleaved, st);
  if (d == 64) return launch_append_d<64>(a, bf16, c8, interleaved, st);
  if (d == 128) return launch_append_d<128>(a, bf16, c8, interleaved, st);
  return cudaErrorInvalidValue;
}

}  // namespace fa
