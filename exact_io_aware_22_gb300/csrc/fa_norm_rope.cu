// fa_norm_rope.cu -- query and key heads normed and turned by their positions before attention, the
// gradient of both, and the same on the way into a paged cache.
//
// Mathematics.  A head x of d columns is divided by its root mean square and weighted,
//     xn = x r,  r = 1 / sqrt(mean x^2 + eps),    z = w xn
// and the pairs (a, b) of its first `rot` columns turn by the token's angles,
//     y = (a cos - b sin, b cos + a sin).
// Backward, for the gradient dy of y: the turn's transpose gives the gradient g of z, then
//     dw = sum over tokens and heads of g xn,    dx = r (h - xn mean(h xn)),  h = w g.
// fp32 arithmetic, one rounding to 16 bits; r is formed again from x, so that nothing is stored
// between the passes.  Without norm the gradient is the forward with the sines negated.
// Appending (fa_append.cu without norms): y of the new tokens' keys, and their values as they are, go
// to their rows of the pools, to E4M3 as y / scale rounded once, to nearest, saturated at +-448.
//
// Bound: bytes.  Every element moves once: two tensors' worth forward and appending, three backward.
// Threads hold items (fa_heads.cuh), 16 columns of one head of one token, a head's neighbouring lanes
// its sums.  The CTAs are as many as fit, and each warp takes a few heads of a token at a time, whose
// angles stay in registers from head to head; queries and keys have CTAs of their own, so that a
// thread has one set of weights (and of sums of dw).  A thread copies its coming items' data, and with
// a new token its angles, to shared memory itself, asynchronously, a ring of them ahead: what is in
// flight takes no registers, needs no barrier, and nothing waits for a look-up.
// Measured, 32/8 heads, d = 128, bf16: 4 x 8192 tokens forward 108 us (6.3 TB/s, 92 % of the copy
// rate), backward 159 us (6.3 TB/s) with the weights' gradients; appending 16 prompts of 600-1100
// tokens 66 us (5.2 TB/s), to E4M3 pages 68 (4.7 TB/s), about as much the instructions of a warp's items
// as bytes.  So are smaller heads: d = 64 forward 63 us (5.3 TB/s), backward 91 (5.6); d = 32 40 (4.2) and
// 54 (4.7).
#include "fa_internal.h"
#include "fa_heads.cuh"
#include "fa_tokens.cuh"

#include <type_traits>

namespace fa {

namespace {

constexpr int NR_THREADS = 128, SMS = 152;
// FWD: y from x; BWD: the gradient with norm, BWD_DW: and of the weights, the CTA's share of it; APPEND,
// APPEND8: y, with values beside queries and keys, into pools of 16-bit numbers or codes.
enum Mode { FWD, BWD, BWD_DW, APPEND, APPEND8 };
// CTAS per SM: more of them with shorter rings, or fewer with longer ones, are slower (appending 16
// prompts of 600-1100 tokens, 32/8 heads: 3 CTAs 82 us, 4 66, 5 71): what counts is warps to
// switch between.  RING: a thread's items in shared memory, of parts of 16 bytes: angles (4), x (2),
// and dy (2) or an appended token's place.
template <Mode MODE>
struct Shape {
  static constexpr bool GRAD = MODE == BWD || MODE == BWD_DW, APP = MODE == APPEND || MODE == APPEND8;
  static constexpr int CTAS = 4, RING = GRAD || APP ? 3 : 4;
  static constexpr int PARTS = GRAD ? 8 : APP ? 7 : 6;
  static constexpr int PART = 16 * NR_THREADS, SMEM = RING * PARTS * PART;
};

// Row of the angles' table for row n of batch entry b (packed: token n); false: it belongs to no
// sequence.
__device__ __forceinline__ bool token_angle(const NormRopeArgs& a, int b, int n, Sequence& seq,
                                            int& ang) {
  ang = n;
  if (a.cu) {
    if (!find_sequence(a.cu, a.n_seq, n, seq)) return false;
    ang = n - seq.lo;
  }
  if (a.positions) ang = a.positions[b * a.pos_stride + n];
  return true;
}

// The place of an appended token: its row of the pools (elements; -1: its page is absent) and its row of
// the angles' table; false: it belongs to no sequence or lies before its sequence's first key.
struct Slot {
  long long row;
};
__device__ __forceinline__ bool append_place(const NormRopeArgs& a, int t, Sequence& seq, Slot& slot,
                                             int& ang) {
  int b, pos, pi;
  if (!locate_token(a.pg, a.cu, a.n_seq, t, seq, b, pos)) return false;
  const int id = page_id(a.pg, b, pos, pi);
  ang = a.positions ? a.positions[t] : pos;
  const bool in_pool = id >= 0 && id < a.pg.pages;
  slot.row = !in_pool ? -1 : id * a.page_stride +
                             (pos - pi * static_cast<int>(a.pg.page.div)) * a.row_stride;
  return true;
}

// An item's chunks begin at columns c0 and c1, apart so that a head's lanes read and write runs of
// neighbouring 16 bytes; t0 and t1 tell whether they turn, by the angles of the pairs a0 .. a0 + 3 and
// a1 .. a1 + 3.  Halves: both chunks of one item turn, c0 with c1; interleaved: each by itself.
struct Item {
  int c0, c1, a0, a1;
  bool t0, t1;
};
template <int D, bool INTER>
__device__ __forceinline__ Item item_of(int j, int rot) {
  if (INTER) {
    const int c0 = 8 * j, c1 = 8 * j + D / 2;
    return {c0, c1, c0 / 2, c1 / 2, c0 < rot, c1 < rot};
  }
  const int k = j - rot / 16;                    // from the first item that does not turn
  if (k >= 0) return {rot + 8 * k, rot + 8 * k + (D - rot) / 2, 0, 0, false, false};
  return {8 * j, 8 * j + rot / 2, 8 * j, 8 * j + 4, true, true};
}
// Turns an item: c, s are the cosines and sines of its 8 pairs.  (Keeping the negated sines too
// spills in the gradient: 4 x 8192 tokens 225 us when this took 161.)
template <bool INTER>
__device__ __forceinline__ void rotate(const Item& it, float2 (&x)[4], float2 (&y)[4],
                                       const float2 (&c)[4], const float2 (&s)[4]) {
  if constexpr (INTER) {
    auto turn = [](float2& p, float c, float s) {
      p = make_float2(p.x * c - p.y * s, p.y * c + p.x * s);
    };
    if (it.t0) {
      turn(x[0], c[0].x, s[0].x);
      turn(x[1], c[0].y, s[0].y);
      turn(x[2], c[1].x, s[1].x);
      turn(x[3], c[1].y, s[1].y);
    }
    if (it.t1) {
      turn(y[0], c[2].x, s[2].x);
      turn(y[1], c[2].y, s[2].y);
      turn(y[2], c[3].x, s[3].x);
      turn(y[3], c[3].y, s[3].y);
    }
  } else if (it.t0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 p = x[i], q = y[i];
      x[i] = fma2(p, c[i], mul2(q, make_float2(-s[i].x, -s[i].y)));
      y[i] = fma2(q, c[i], mul2(p, s[i]));
    }
  }
}

__device__ __forceinline__ void copy16(uint32_t smem, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16_l1(uint32_t smem, const void* src) {   // heads share them
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until all but the last N groups of this thread's copies have landed.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, bool BF16, bool INTER, bool NORM, Mode MODE>
__global__ void __launch_bounds__(NR_THREADS, Shape<MODE>::CTAS)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  grid_dep_wait();                               // inputs written, outputs free to overwrite
  using S = Shape<MODE>;
  constexpr bool GRAD = S::GRAD, DW = MODE == BWD_DW, APP = S::APP;
  constexpr int IPH = D / 16, SLOTS = 32 / IPH;  // lanes of a head, heads of a warp
  constexpr int RING = S::RING;
  constexpr uint32_t PART = S::PART, STAGE = S::PARTS * S::PART;
  __shared__ __align__(16) uint8_t ring[S::SMEM];
  // queries, keys, and of appended tokens values
  int bx = static_cast<int>(blockIdx.x), kind = 0, blocks = a.blocks[0];
  if (bx >= blocks) {
    bx -= blocks;
    blocks = a.blocks[kind = 1];
    if (APP && bx >= blocks) {
      bx -= blocks;
      blocks = a.blocks[kind = 2];
    }
  }
  const HeadView vx = a.x[kind], vo = a.y[kind], vg = a.dy[GRAD ? kind : 0];
  const FastDiv heads = a.heads[kind];
  const int rot = APP && kind == 2 ? 0 : a.rot;  // columns that turn
  const int tid = static_cast<int>(threadIdx.x), j = tid % IPH;
  const Item it = item_of<D, INTER>(j, rot);
  // The heads of all tokens, a token's one after another, are cut into chunks of chunk * SLOTS;
  // warp w of W takes chunks w, w + W, ..., SLOTS heads at a time.
  const int H = static_cast<int>(heads.div), chunk = a.chunk[kind];
  const uint32_t total = static_cast<uint32_t>(a.T) * heads.div;
  const uint32_t stride = static_cast<uint32_t>(blocks) * (NR_THREADS / 32) * (chunk * SLOTS);
  const int dt = SLOTS / H, dh = SLOTS % H;
  struct Place {                                 // of an item of this thread
    uint32_t u0;                                 // its slot's head in the chunk's first step
    int k, t, h;                                 // step, token, head
  };
  auto seek = [&](Place& p) {
    p.k = 0;
    p.t = static_cast<int>(heads.quot(p.u0));
    p.h = static_cast<int>(p.u0) - p.t * H;
  };
  auto there = [&](const Place& p) { return p.u0 + p.k * SLOTS < total; };
  auto advance = [&](Place& p) {
    if (++p.k == chunk) {
      p.u0 += stride;
      seek(p);
      return;
    }
    p.t += dt;
    p.h += dh;
    if (p.h >= H) {
      p.h -= H;
      ++p.t;
    }
  };
  auto token_at = [&](const HeadView& v, int b, int n) {
    return static_cast<uint16_t*>(v.data) + b * v.batch_stride + n * v.row_stride;
  };
  Place pf, p;                                   // of the next item to fetch, and to compute
  pf.u0 = (static_cast<uint32_t>(bx) * (NR_THREADS / 32) + tid / 32) * (chunk * SLOTS) + tid % 32 / IPH;
  seek(pf);
  p = pf;
  const uint32_t mine = smem_u32(ring) + 16 * tid;
  Sequence seq = {0, 0, 0, 0};
  const uint16_t *fx = nullptr, *fg = nullptr;   // the token's first head
  int t_fetched = -1;
  bool known = false;                            // its token is to be computed
  uint32_t have = 0;                             // bit i: so is the item in stage i
  auto fetch = [&](int stage) {
    if (there(pf)) {
      const uint32_t dst = mine + stage * STAGE;
      if (pf.t != t_fetched) {
        t_fetched = pf.t;
        const int b = static_cast<int>(a.rows.quot(pf.t));
        const int n = pf.t - b * static_cast<int>(a.rows.div);
        fx = token_at(vx, b, n) + it.c0;
        if constexpr (GRAD) fg = token_at(vg, b, n) + it.c0;
        int ang;
        if constexpr (APP) {
          Slot slot = {-1};
          known = append_place(a, n, seq, slot, ang);
          if (known && slot.row < 0) {
            atomicOr(a.ctl.status, FA_DEV_BAD_INDEX);
            known = kind == 0;                   // only its query is left
          }
          asm volatile("st.shared.b64 [%0], %1;" ::"r"(dst + 6 * PART), "l"(slot.row) : "memory");
        } else {
          known = token_angle(a, b, n, seq, ang);
        }
        if (known && a.rot > 0) {
          if (ang < 0 || ang >= a.max_pos) {     // such a token is left out whole
            atomicOr(a.ctl.status, FA_DEV_BAD_INDEX);
            known = false;
          } else {
            const float* cs = a.cos_sin + static_cast<long long>(ang) * a.rot;
            if (it.t0) {
              copy16_l1(dst, cs + it.a0);
              copy16_l1(dst + PART, cs + a.rot / 2 + it.a0);
            }
            if (it.t1) {
              copy16_l1(dst + 2 * PART, cs + it.a1);
              copy16_l1(dst + 3 * PART, cs + a.rot / 2 + it.a1);
            }
          }
        }
        if (!APP && !known && (kind ? a.y[1].zero_rest : a.y[0].zero_rest)) {
          // zeros to all that this thread, or another warp's in its place, has of the token: here, once a
          // token, and not where its items are skipped below (the gradient of 4 x 8192 tokens 159
          // against 162 us)
          uint16_t* y = token_at(vo, b, n);
          for (int h = pf.h; h < H; h += SLOTS) {
            *reinterpret_cast<uint4*>(y + h * vo.head_stride + it.c0) = make_uint4(0u, 0u, 0u, 0u);
            *reinterpret_cast<uint4*>(y + h * vo.head_stride + it.c1) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
      }
      have = (have & ~(1u << stage)) | (static_cast<uint32_t>(known) << stage);
      const uint16_t* x = fx + pf.h * vx.head_stride;
      copy16(dst + 4 * PART, x);
      copy16(dst + 5 * PART, x + (it.c1 - it.c0));
      if constexpr (GRAD) {
        const uint16_t* g = fg + pf.h * vg.head_stride;
        copy16(dst + 6 * PART, g);
        copy16(dst + 7 * PART, g + (it.c1 - it.c0));
      }
      advance(pf);
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < RING - 1; ++i) fetch(i);
  // weights, sums of dw, angles
  float2 wx[4], wy[4], ax[4], ay[4], c[4], s[4];
  if constexpr (NORM) {
    load_weights8<BF16>(kind ? a.w[1] : a.w[0], a.w_fp32, it.c0, wx);
    load_weights8<BF16>(kind ? a.w[1] : a.w[0], a.w_fp32, it.c1, wy);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) ax[e] = ay[e] = c[e] = s[e] = make_float2(0.f, 0.f);

  uint16_t* out = nullptr;                       // the token's first head
  uint8_t* out8 = nullptr;                       // the same in a pool of codes
  const bool pool = APP && kind > 0;
  int t_turned = -1;
  for (int stage = 0; there(p); stage = stage + 1 == RING ? 0 : stage + 1, advance(p)) {
    fetch(stage == 0 ? RING - 1 : stage - 1);
    copies_wait<RING - 1>();
    auto part = [&](int i) -> const uint4& {
      return *reinterpret_cast<const uint4*>(ring + stage * STAGE + i * PART + 16 * tid);
    };
    if (p.t != t_turned) {                       // a token's first item has its angles
      t_turned = p.t;
      const int b = static_cast<int>(a.rows.quot(p.t));
      out = token_at(vo, b, p.t - b * static_cast<int>(a.rows.div));
      if (pool) {
        long long row;
        asm volatile("ld.shared.b64 %0, [%1];"
                     : "=l"(row)
                     : "r"(mine + stage * STAGE + 6 * PART)
                     : "memory");
        out = static_cast<uint16_t*>(vo.data) + row;
        out8 = static_cast<uint8_t*>(vo.data) + row;
      }
      if (it.t0 || it.t1) {
        const float4 c0 = *reinterpret_cast<const float4*>(&part(0)),
                     s0 = *reinterpret_cast<const float4*>(&part(1)),
                     c1 = *reinterpret_cast<const float4*>(&part(2)),
                     s1 = *reinterpret_cast<const float4*>(&part(3));
        const float2 sg = make_float2(a.sin_sign, a.sin_sign);
        c[0] = make_float2(c0.x, c0.y);
        c[1] = make_float2(c0.z, c0.w);
        c[2] = make_float2(c1.x, c1.y);
        c[3] = make_float2(c1.z, c1.w);
        s[0] = mul2(make_float2(s0.x, s0.y), sg);
        s[1] = mul2(make_float2(s0.z, s0.w), sg);
        s[2] = mul2(make_float2(s1.x, s1.y), sg);
        s[3] = mul2(make_float2(s1.z, s1.w), sg);
      }
    }
    if (!((have >> stage) & 1u)) continue;
    if constexpr (MODE == APPEND) {
      if (kind == 2) {                           // values as they are
        uint16_t* dst = out + p.h * vo.head_stride;
        *reinterpret_cast<uint4*>(dst + it.c0) = part(4);
        *reinterpret_cast<uint4*>(dst + it.c1) = part(5);
        continue;
      }
    }
    float2 x[4], y[4];
    unpack8<BF16>(part(4), x);
    unpack8<BF16>(part(5), y);
    if constexpr (!GRAD) {
      if (NORM && !(APP && kind == 2)) {
        const float r = head_rrms<D>(x, y, a.eps);
        weigh8(x, r, wx);
        weigh8(y, r, wy);
      }
      rotate<INTER>(it, x, y, c, s);
      if constexpr (MODE == APPEND8) {
        if (pool) {
          uint8_t* dst = out8 + p.h * vo.head_stride;
          const float inv = kind == 1 ? a.k_inv : a.v_inv;
          *reinterpret_cast<uint2*>(dst + it.c0) = codes8(x, inv);
          *reinterpret_cast<uint2*>(dst + it.c1) = codes8(y, inv);
          continue;
        }
      }
    } else {
      float2 gx[4], gy[4];
      unpack8<BF16>(part(6), gx);
      unpack8<BF16>(part(7), gy);
      rotate<INTER>(it, gx, gy, c, s);
      const float r = head_rrms<D>(x, y, a.eps);
      const float2 r2 = make_float2(r, r);
      float2 dx = make_float2(0.f, 0.f), dy = dx;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = mul2(x[e], r2);
        y[e] = mul2(y[e], r2);
        if constexpr (DW) {
          ax[e] = fma2(gx[e], x[e], ax[e]);
          ay[e] = fma2(gy[e], y[e], ay[e]);
        }
        gx[e] = mul2(gx[e], wx[e]);
        gy[e] = mul2(gy[e], wy[e]);
        dx = fma2(gx[e], x[e], dx);
        dy = fma2(gy[e], y[e], dy);
      }
      const float dot = head_sum<D>((dx.x + dx.y) + (dy.x + dy.y)) * (-1.f / D);
      const float2 d2 = make_float2(dot, dot);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = mul2(r2, fma2(x[e], d2, gx[e]));
        y[e] = mul2(r2, fma2(y[e], d2, gy[e]));
      }
    }
    uint16_t* dst = out + p.h * vo.head_stride;
    *reinterpret_cast<uint4*>(dst + it.c0) = pack8<BF16>(x);
    *reinterpret_cast<uint4*>(dst + it.c1) = pack8<BF16>(y);
  }
  if constexpr (DW) {
    // threads IPH apart have the same columns: first the warp's, then the four warps'
    __shared__ float sums[NR_THREADS / 32][IPH][16];
    const int wl = tid % 32, warp = tid / 32;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int w = IPH; w < 32; w *= 2) {
        ax[e].x += __shfl_xor_sync(0xffffffffu, ax[e].x, w);
        ax[e].y += __shfl_xor_sync(0xffffffffu, ax[e].y, w);
        ay[e].x += __shfl_xor_sync(0xffffffffu, ay[e].x, w);
        ay[e].y += __shfl_xor_sync(0xffffffffu, ay[e].y, w);
      }
      if (wl < IPH) {
        sums[warp][wl][2 * e] = ax[e].x;
        sums[warp][wl][2 * e + 1] = ax[e].y;
        sums[warp][wl][8 + 2 * e] = ay[e].x;
        sums[warp][wl][8 + 2 * e + 1] = ay[e].y;
      }
    }
    __syncthreads();
    if (tid < D) {
      const int jj = tid / 16, e = tid % 16;
      const Item cc = item_of<D, INTER>(jj, a.rot);
      const int col = e < 8 ? cc.c0 + e : cc.c1 + e - 8;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < NR_THREADS / 32; ++w) v += sums[w][jj][e];
      a.part[static_cast<size_t>(blockIdx.x) * D + col] = v;
    }
  }
}

// dw of queries (blockIdx.y 0) and keys: 32 columns, the CTAs' sums of rows 32 apart to a warp.
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* part, int blocks_q,
                                                            int blocks, int d, float* dwq,
                                                            float* dwk) {
  grid_dep_wait();
  __shared__ float sums[32][33];
  float* dst = blockIdx.y ? dwk : dwq;
  if (!dst) return;
  const int lane = static_cast<int>(threadIdx.x) & 31, warp = static_cast<int>(threadIdx.x) >> 5;
  const int col = static_cast<int>(blockIdx.x) * 32 + lane;
  const int r0 = blockIdx.y ? blocks_q : 0, r1 = blockIdx.y ? blocks : blocks_q;
  // ten loads of a thread together, so that most calls wait for memory twice; few rows in fours
  float v = 0.f;
  auto add = [&](auto n, int r) {
    constexpr int N = decltype(n)::value;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = r + 32 * i < r1 ? part[static_cast<size_t>(r + 32 * i) * d + col] : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) v += x[i];
  };
  if (r1 - r0 > 128)
    for (int r = r0 + warp; r < r1; r += 320) add(std::integral_constant<int, 10>(), r);
  else
    add(std::integral_constant<int, 4>(), r0 + warp);
  sums[warp][lane] = v;
  __syncthreads();
  v = sums[lane][warp];                          // column `warp`, row group `lane`
#pragma unroll
  for (int w = 16; w > 0; w /= 2) v += __shfl_xor_sync(0xffffffffu, v, w);
  if (lane == 0) dst[static_cast<int>(blockIdx.x) * 32 + warp] = v;
}

// Steps of a warp's piece of a token's heads, of which it has `steps` in all.  Output planes of (B, heads,
// N, d) want the tokens in work close together: 2 (1 / 2 / 4 / 8 steps, 4 x 8192 tokens, 32/8 heads, d = 128:
// 134 / 110 / 122 / 127 us forward, 193 / 162 / 174 / 181 backward).  Where a token has a sequence to be
// found, its heads in a row pay for that: 8 for the append (90 / 72 / 71 / 68) and, where there is work
// for two pieces, for packed sequences with norms (13 000 tokens: 58 / 50 / 48 / 47.5 forward, 86 / 75 / 73 /
// 71 backward; 1200 tokens backward 13.2 / 12.3 / 13.1 / 14.6; without norms 49 / 44.5 / 46 / 49).  No longer
// pieces than a warp has steps (64 tokens into E4M3 pages 2.9 against 7.2 us).
template <Mode MODE, bool NORM>
int piece_steps(const NormRopeArgs& a, long long steps) {
  const bool look_ups = Shape<MODE>::APP || (NORM && a.cu && steps >= 16);
  const long long most = look_ups ? 8 : 2;
  return static_cast<int>(steps < 1 ? 1 : steps < most ? steps : most);
}

// CTAs for queries, keys and appended values, in proportion to their heads: at most `most` in all (or one
// each), and no more than have work.
template <int D, bool NORM, Mode MODE>
bool plan(NormRopeArgs& a, int& all) {
  constexpr int most = SMS * Shape<MODE>::CTAS;
  constexpr int SLOTS = NR_THREADS / (D / 16);   // heads that a CTA holds at a time
  long long heads = 0;
  for (const HeadView& x : a.x) heads += x.heads;
  all = 0;
  for (int i = 0; i < 3; ++i) {
    const long long n = static_cast<long long>(a.T) * a.x[i].heads;
    if (n > 0x7fffffffLL) return false;
    a.blocks[i] = 0;
    if (n == 0) continue;
    const long long share = most * static_cast<long long>(a.x[i].heads) / heads;
    const long long need = (n + SLOTS - 1) / SLOTS;
    a.blocks[i] = static_cast<int>(need < share ? need : share < 1 ? 1 : share);
    a.chunk[i] = piece_steps<MODE, NORM>(a, need / (share < 1 ? 1 : share));
    a.heads[i] = make_fast_div(static_cast<uint32_t>(a.x[i].heads));
    all += a.blocks[i];
  }
  return true;
}

template <int D, bool BF16, bool INTER, bool NORM, Mode MODE>
cudaError_t launch_t(NormRopeArgs a, cudaStream_t st) {
  int all;
  if (!plan<D, NORM, MODE>(a, all)) return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_dependent(norm_rope_kernel<D, BF16, INTER, NORM, MODE>,
                                   static_cast<unsigned>(all), NR_THREADS, 0, st, a);
  if (MODE != BWD_DW || e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(D / 32, 2, 1);
  cfg.blockDim = dim3(1024, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_rope_dw_kernel, static_cast<const float*>(a.part),
                            a.blocks[0], all, D, a.dw[0], a.dw[1]);
}

template <int D, bool BF16, bool INTER>
cudaError_t launch_i(const NormRopeArgs& a, NormRopeOp op, cudaStream_t st) {
  if (op == NormRopeOp::Append) return launch_t<D, BF16, INTER, true, APPEND>(a, st);
  if constexpr (D == 128)
    if (op == NormRopeOp::Append8) return launch_t<D, BF16, INTER, true, APPEND8>(a, st);
  if (!a.norm) return launch_t<D, BF16, INTER, false, FWD>(a, st);
  if (op == NormRopeOp::Forward) return launch_t<D, BF16, INTER, true, FWD>(a, st);
  if (a.dw[0] || a.dw[1]) return launch_t<D, BF16, INTER, true, BWD_DW>(a, st);
  return launch_t<D, BF16, INTER, true, BWD>(a, st);
}
template <int D>
cudaError_t launch_d(const NormRopeArgs& a, bool bf16, bool inter, NormRopeOp op, cudaStream_t st) {
  if (inter) return bf16 ? launch_i<D, true, true>(a, op, st) : launch_i<D, false, true>(a, op, st);
  return bf16 ? launch_i<D, true, false>(a, op, st) : launch_i<D, false, false>(a, op, st);
}

}  // namespace

size_t norm_rope_bwd_ws_bytes(int d) { return static_cast<size_t>(SMS * Shape<BWD>::CTAS + 2) * d * 4; }

cudaError_t launch_norm_rope(const NormRopeArgs& a, int d, bool bf16, bool interleaved,
                             NormRopeOp op, cudaStream_t st) {
  if (op == NormRopeOp::Append8 && d != 128) return cudaErrorInvalidValue;
  if (d == 32) return launch_d<32>(a, bf16, interleaved, op, st);
  if (d == 64) return launch_d<64>(a, bf16, interleaved, op, st);
  if (d == 128) return launch_d<128>(a, bf16, interleaved, op, st);
  return cudaErrorInvalidValue;
}

}  // namespace fa
