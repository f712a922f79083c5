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
// Bound: bytes.  Every input and output element moves once.  An item is 16 elements of a head
// (two 16-byte loads, two stores) -- both halves of 8 pairs -- so a rotation needs no exchange
// between threads.  A thread carries the same 16 columns of up to M heads of one token, which
// share the 16 table values that turn them; a token takes as many threads as that needs, and
// a CTA as many tokens as fit (or a slice of one).  The data are loaded before the token's
// position is known: finding the sequence, its length and the page is a chain of dependent
// loads that the data loads then hide.  All loads are plain ones, not read-only-path ones:
// earlier work in the stream may still be writing their sources when this kernel starts, and
// nothing may move them above grid_dep_wait().
// Measured, 32/8 heads, d = 128, bf16: 16 prompts of 600-1100 tokens 55 us (6.3 TB/s), one token
// 1.9 us, 64 tokens 2.2 us.
#include "fa_internal.h"
#include "fa_ptx.cuh"
#include "fa_tokens.cuh"

namespace fa {

namespace {

constexpr int APP_THREADS = 128;
constexpr int APP_CTAS = 8;                       // CTAs per SM up to which a thread has one head

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<BF16>(u[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3]), pack2<BF16>(x[4], x[5]),
                    pack2<BF16>(x[6], x[7]));
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  const float2 p[4] = {make_float2(x[0], x[1]), make_float2(x[2], x[3]), make_float2(x[4], x[5]),
                       make_float2(x[6], x[7])};
  return fa::codes8(p, inv);
}

// How the heads of a token (K's, V's, then Q's) go to threads: `lanes` threads per column group
// in each of `slices` CTAs, M heads each; `tokens` tokens per CTA.
struct AppendSplit {
  int lanes, slices, tokens;
};

template <int D, bool BF16, bool C8, bool INTER, int M>
__global__ void __launch_bounds__(APP_THREADS) append_kernel(const AppendArgs a,
                                                             const AppendSplit sp) {
  grid_dep_wait();                               // inputs written, cache rows free to overwrite
  constexpr int IPH = D / 16;                    // items per head
  const int heads = (a.Q ? a.H : 0) + 2 * a.Hkv;
  const int per_tok = sp.lanes * IPH, slot = static_cast<int>(threadIdx.x) / per_tok;
  const int lane = static_cast<int>(threadIdx.x) - slot * per_tok;
  const int t = static_cast<int>(blockIdx.x) / sp.slices * sp.tokens + slot;
  if (slot >= sp.tokens || t >= a.T) return;
  const int h0 = static_cast<int>(blockIdx.x) % sp.slices * (sp.lanes * M) + lane / IPH;
  const int j = lane % IPH;
  const bool rot = j < a.rot / 16;               // columns that keys and queries turn
  // the item's two 8-column chunks: plain, and turned
  const int p0 = 16 * j, p1 = 16 * j + 8;
  const int r0 = INTER ? p0 : 8 * j, r1 = INTER ? p1 : 8 * j + a.rot / 2;

  uint4 w0[M], w1[M];
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int head = h0 + m * sp.lanes;
    if (head >= heads) break;
    // which tensor: keys first, then values, then queries
    const int kind = head < a.Hkv ? 0 : head < 2 * a.Hkv ? 1 : 2;
    const uint16_t* src = static_cast<const uint16_t*>(kind == 0 ? a.K : kind == 1 ? a.V : a.Q) +
                          t * (kind == 0 ? a.k_stride : kind == 1 ? a.v_stride : a.q_stride) +
                          static_cast<long long>(head - kind * a.Hkv) * D;
    const bool turn = rot && kind != 1;
    w0[m] = *reinterpret_cast<const uint4*>(src + (turn ? r0 : p0));
    w1[m] = *reinterpret_cast<const uint4*>(src + (turn ? r1 : p1));
  }

  int b, pos, pi;
  Sequence seq = {0, 0, 0, 0};
  if (!locate_token(a.pg, a.cu, a.B, t, seq, b, pos)) return;
  const int id = page_id(a.pg, b, pos, pi);
  float c[8], s[8];
  if (a.rot > 0) {
    // a token whose angle lies outside the table is left out whole
    const int ang = a.positions ? a.positions[t] : pos;
    if (ang < 0 || ang >= a.max_pos) {
      atomicOr(a.ctl.status, FA_DEV_BAD_INDEX);
      return;
    }
    if (rot) {
      const float* cs = a.cos_sin + static_cast<long long>(ang) * a.rot + 8 * j;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 cc = *reinterpret_cast<const float4*>(cs + i);
        const float4 ss = *reinterpret_cast<const float4*>(cs + a.rot / 2 + i);
        c[i] = cc.x; c[i + 1] = cc.y; c[i + 2] = cc.z; c[i + 3] = cc.w;
        s[i] = ss.x; s[i + 1] = ss.y; s[i + 2] = ss.z; s[i + 3] = ss.w;
      }
    }
  }
  const bool in_pool = id >= 0 && id < a.pg.pages;
  if (!in_pool) atomicOr(a.ctl.status, FA_DEV_BAD_INDEX);
  const long long row = id * a.page_stride +
                        (pos - pi * static_cast<int>(a.pg.page.div)) * a.row_stride;
#pragma unroll
  for (int m = 0; m < M; ++m) {
    const int at = h0 + m * sp.lanes;
    if (at >= heads) break;
    const int kind = at < a.Hkv ? 0 : at < 2 * a.Hkv ? 1 : 2, head = at - kind * a.Hkv;
    const bool turn = rot && kind != 1;
    float x[8], y[8];
    unpack8<BF16>(w0[m], x);
    unpack8<BF16>(w1[m], y);
    if (turn) {
      if constexpr (INTER) {                     // pairs inside a chunk: x holds 4 pairs, y 4
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float p = x[e], q = x[e + 1], u = y[e], v = y[e + 1];
          x[e] = p * c[e / 2] - q * s[e / 2];
          x[e + 1] = q * c[e / 2] + p * s[e / 2];
          y[e] = u * c[4 + e / 2] - v * s[4 + e / 2];
          y[e + 1] = v * c[4 + e / 2] + u * s[4 + e / 2];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = x[e], q = y[e];
          x[e] = p * c[e] - q * s[e];
          y[e] = q * c[e] + p * s[e];
        }
      }
    }
    const int c0 = turn ? r0 : p0, c1 = turn ? r1 : p1;
    if (kind == 2) {
      uint16_t* dst = static_cast<uint16_t*>(a.Qout) + (static_cast<long long>(t) * a.H + head) * D;
      *reinterpret_cast<uint4*>(dst + c0) = pack8<BF16>(x);
      *reinterpret_cast<uint4*>(dst + c1) = pack8<BF16>(y);
    } else if (in_pool) {
      void* pool = kind == 0 ? a.Kc : a.Vc;
      if constexpr (C8) {
        uint8_t* dst = static_cast<uint8_t*>(pool) + row + head * a.head_stride;
        const float inv = kind == 0 ? a.k_inv : a.v_inv;
        *reinterpret_cast<uint2*>(dst + c0) = codes8(x, inv);
        *reinterpret_cast<uint2*>(dst + c1) = codes8(y, inv);
      } else {
        uint16_t* dst = static_cast<uint16_t*>(pool) + row + head * a.head_stride;
        *reinterpret_cast<uint4*>(dst + c0) = pack8<BF16>(x);
        *reinterpret_cast<uint4*>(dst + c1) = pack8<BF16>(y);
      }
    }
  }
}

template <int D, bool BF16, bool C8, bool INTER, int M>
cudaError_t launch_append_m(const AppendArgs& a, int heads, cudaStream_t st) {
  constexpr int IPH = D / 16, MOST = APP_THREADS / IPH;   // lanes of a whole CTA
  AppendSplit sp;
  sp.slices = (heads + MOST * M - 1) / (MOST * M);
  sp.lanes = ((heads + sp.slices - 1) / sp.slices + M - 1) / M;
  sp.tokens = MOST / sp.lanes;
  const long long grid =
      (static_cast<long long>(a.T) + sp.tokens - 1) / sp.tokens * sp.slices;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_dependent(append_kernel<D, BF16, C8, INTER, M>, static_cast<unsigned>(grid),
                          APP_THREADS, 0, st, a, sp);
}

template <int D, bool BF16, bool C8, bool INTER>
cudaError_t launch_append_t(const AppendArgs& a, cudaStream_t st) {
  const long long heads = (a.Q ? a.H : 0) + 2LL * a.Hkv;
  if (heads > (1 << 28)) return cudaErrorInvalidConfiguration;
  // few tokens: one head per thread, so that they spread over more SMs (64 tokens of 32/8
  // heads: 2.1 against 2.4 us); many: four, or three where the codes' conversion adds to the
  // work (16384 tokens, 1 / 2 / 3 / 4 heads: bf16 76.4 / 71.6 / 65.6 / 63.4 us, E4M3 76.5 /
  // 70.3 / 63.9 / 65.2 us)
  if (a.T * heads * (D / 16) <= 152LL * APP_CTAS * APP_THREADS)
    return launch_append_m<D, BF16, C8, INTER, 1>(a, static_cast<int>(heads), st);
  return launch_append_m<D, BF16, C8, INTER, C8 ? 3 : 4>(a, static_cast<int>(heads), st);
}

template <int D, bool BF16, bool C8>
cudaError_t launch_append_i(const AppendArgs& a, bool interleaved, cudaStream_t st) {
  return interleaved ? launch_append_t<D, BF16, C8, true>(a, st)
                     : launch_append_t<D, BF16, C8, false>(a, st);
}

template <int D>
cudaError_t launch_append_d(const AppendArgs& a, bool bf16, bool c8, bool inter, cudaStream_t st) {
  if constexpr (D == 128)
    if (c8)
      return bf16 ? launch_append_i<D, true, true>(a, inter, st)
                  : launch_append_i<D, false, true>(a, inter, st);
  return bf16 ? launch_append_i<D, true, false>(a, inter, st)
              : launch_append_i<D, false, false>(a, inter, st);
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
