// fa_decode_paged.cu -- one new query row per (sequence, head) over a paged key/value cache.
//
// Mathematics.  Softmax over disjoint key ranges is carried as partial states (m, l, acc)
// that merge exactly (m' = max(m1, m2), l' = l1 2^(m1-m') + l2 2^(m2-m'), acc likewise), in
// base 2 with scale * log2(e) applied to the fp32 scores: the tutorial page "What is
// FlashAttention?", "Softmax in pieces".  A state without keys is (-inf, 0, 0).
//
// Bound: the cache's bytes.  Each K and V row is read once from HBM and serves all query
// heads of its group (up to 16 per CTA; the CTAs of a larger group's parts walk the same keys
// side by side, so that all but one find them in L2).  The products are kept off the critical
// path: they run as warp-level tensor-core products (m16n8k16) with the *keys* as the rows,
//     S^T (16 keys x 8 heads) = K Q^T,      O^T (16 columns x 8 heads) += V^T P^T,
// so a group of up to 8 heads pads nothing but n = 8, K and V^T are fragments that ldmatrix
// reads from the tiles as TMA laid them down, and S^T becomes the second product's operand by
// transposing 8 x 8 blocks between lanes (movmatrix).  P goes in as two 16-bit terms (its
// rounding and the remainder's), so that rounding P costs the result nothing.
//
// Work split.  Lengths live on the device and are ragged.  The keys of all rows (sequence,
// K/V head) are laid end to end in units of one ring stage of every warp, and
// the grid's CTAs take equal ranges; a range may end inside a row.  A row inside one CTA's
// range is finished there; a row cut by range borders leaves one partial state per CTA, and
// decode_paged_merge_kernel joins them in CTA order, so results do not depend on timing.
// CTA c keeps at most two such states: of the row that began in an earlier CTA (slot 0) and of
// the row that goes on in the next one (slot 1).  Ranges are equal in cost: a row of u units
// counts 2u + 1, since beginning and ending a row takes about as long as half a unit.  Unit i
// of a row then sits at the row's position 2i + 1, and a CTA has the units at its positions.
// Where the table (or the window) bounds every row to a few units, each row has a CTA of its
// own instead: nothing to scan, nothing to join.
//
// Measured, 32/8 heads, d = 128: 16 sequences of 16384-32768 keys 0.238 ms in bf16 (6.8 TB/s,
// the rate of a copy) and 0.130 ms in E4M3 (6.2 TB/s); one sequence of 130049 keys 0.090 ms
// (5.9 TB/s).  About 10 us of every call that cuts rows do not depend on the bytes: 3 us until
// the first load is out, 3 to 4 us of join, and ranges that end up to 10 % apart.  Short rows
// that are not cut: one sequence of 60 keys 3.7 us, 256 of 250-500 keys 63 us (5.8 TB/s).
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

namespace {

constexpr int DP_WARPS = 4;
constexpr int DP_MERGE_THREADS = 128;
// Ring stages per warp and CTAs per SM, by column blocks NT (8 heads each): 192 KiB of ring on
// an SM either way.  Two blocks need more than the 168 registers that three CTAs leave.
__host__ __device__ constexpr int stages_of(int NT) { return NT == 1 ? 2 : 3; }
__host__ __device__ constexpr int ctas_of(int NT) { return NT == 1 ? 3 : 2; }
__host__ __device__ constexpr int grid_of(int NT) { return 152 * ctas_of(NT); }   // one wave

// One ring stage of a warp: KEYS keys of K, then of V, about 4 KiB each.
template <int D, bool C8>
struct Geom {
  static constexpr int ELEM = C8 ? 1 : 2;
  static constexpr int BOXC = C8 ? D : (D == 32 ? 32 : 64);   // columns of one TMA box
  static constexpr int ROWB = BOXC * ELEM;                    // bytes of a box row (swizzle span)
  static constexpr int SWM = ROWB == 128 ? 7 : 3;             // 16-byte chunk bits ^= row bits
  static constexpr int HALVES = D / BOXC;
  static constexpr int KEYS = 4096 / (D * ELEM);              // 16, 32 or 64
  static constexpr int BOXB = KEYS * ROWB;
  static constexpr int TILEB = HALVES * BOXB;                 // 4 KiB
  static constexpr int STAGEB = 2 * TILEB;
  static constexpr int UNIT = DP_WARPS * KEYS;                // keys of one work unit
};

template <int D, bool C8, int NT>
__host__ __device__ constexpr int ring_bytes() {
  return DP_WARPS * stages_of(NT) * Geom<D, C8>::STAGEB;
}
// two warps' states of 8 heads: m, l, then acc, heads 16 bytes apart mod 128
template <int D>
__host__ __device__ constexpr int red_bytes() { return 2 * 8 * (D + 4) * 4; }
template <int D, bool C8, int NT>
constexpr int smem_bytes() {
  return 1024 + ring_bytes<D, C8, NT>() + red_bytes<D>() + DP_WARPS * stages_of(NT) * 8 + 64;
}

// Workspace: one header per CTA, then two slots of `rows` partial states per CTA.
struct Header {
  int row;     // the row (b * Hkv + hk) that range x shares with range x - 1, or -1
  int c0, c1;  // first and last range of that row
};
__host__ __device__ constexpr size_t hdr_bytes(int NT) {
  return (grid_of(NT) * sizeof(Header) + 15) / 16 * 16;
}

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
// Transpose of an 8 x 8 block of 16-bit values held as (row lane / 4, columns 2 (lane % 4)).
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E4M3 codes (the low or high half of w) as f16 values, exactly.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}"
      : "=r"(r)
      : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t even_odd(uint32_t w) {   // bytes 0, 2, 1, 3
  uint32_t r;
  asm("prmt.b32 %0, %1, %1, 0x3120;" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ float ld_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_f32(uint32_t a, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}
// 2^(m - ref) of a state with maximum m relative to a larger one; a state without keys weighs 0.
__device__ __forceinline__ float weight(float m, float ref) {
  return m == -INFINITY ? 0.f : ex2(m - ref);
}

// Keys [lo, n) of a sequence are attended; its units start at key a0 = lo rounded down to
// whole stages.  A window counts from the length as it is given, and may lie past the table.
struct SeqKeys {
  int lo, n, a0, units;
};
template <int KEYS, int UNIT>
__device__ __forceinline__ SeqKeys seq_keys(const PagedView& pg, int b, int window) {
  const long long cap = static_cast<long long>(pg.max_pages) * pg.page.div;
  SeqKeys s;
  const int len = max(pg.seqlens[b], 0);
  s.n = static_cast<int>(min(static_cast<long long>(len), cap));
  s.lo = window > 0 && window < len ? len - window : 0;
  s.a0 = s.lo & ~(KEYS - 1);
  s.units = s.lo < s.n ? (s.n - s.a0 + UNIT - 1) / UNIT : 0;
  return s;
}

// Cost of a row of `units` units (see above).
__host__ __device__ constexpr int row_cost(int units) { return units > 0 ? 2 * units + 1 : 0; }

// A place in a CTA's range: row r (K/V head) of sequence b, unit u of the row; the range
// covers the row's units up to ue, and `left` positions after the row's.
struct Cursor {
  int b, r, u, ue, left;
  SeqKeys s;
};

template <int D, bool BF16, bool C8, int NT>
__global__ void __launch_bounds__(32 * DP_WARPS, ctas_of(NT))
    decode_paged_kernel(const __grid_constant__ CUtensorMap tmK,
                        const __grid_constant__ CUtensorMap tmV, const void* Q, void* O, float* L,
                        uint8_t* ws, int B, int H, int Hkv, int window, int direct, int box_log2,
                        float c_log2, float o_scale, const PagedView pg, KernelCtl ctl) {
  using G = Geom<D, C8>;
  constexpr int KEYS = G::KEYS, MT = KEYS / 16, KS = D / 16, RG = 8 * NT, STAGES = stages_of(NT);
  constexpr bool MB = BF16 && !C8;               // operands of the products: bf16 or f16
  // A state's m is the maximum less SH: p <= 2^(SH + 8) = 2^15 where P is f16, so that the
  // small p of a long context, which add up, stay clear of f16's subnormals: a weight of less than
  // 2^-21 of the largest is off by up to 2^-32 of that, others by 2^-16 of themselves or less.
  constexpr float SH = MB ? 0.f : 7.f;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;         // fragment row, column pair
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw), sb = (raw + 1023u) & ~1023u;
  const uint32_t ring = sb + warp * STAGES * G::STAGEB;
  const uint32_t red = sb + ring_bytes<D, C8, NT>();
  const uint32_t bars = red + red_bytes<D>() + warp * STAGES * 8;
  const uint32_t scan = red + red_bytes<D>() + DP_WARPS * STAGES * 8;
  if (lane == 0) {
    for (int st = 0; st < STAGES; ++st) mbar_init(bars + st * 8, 1);
    fence_mbar_init();
  }
  __syncwarp();
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  // Finding the first keys is a chain of dependent loads (lengths, page table); what they
  // will read is brought to L2 at once: one 128-byte line of the table per thread of the grid.
  {
    const long long i = static_cast<long long>(blockIdx.x) * (32 * DP_WARPS) + threadIdx.x;
    const int lpr = (pg.max_pages + 31) >> 5;    // lines per table row
    if (i < static_cast<long long>(B) * lpr)
      prefetch_l2(pg.table + (i / lpr) * pg.table_stride + (i % lpr) * 32);
    if (i < (B + 31) >> 5) prefetch_l2(pg.seqlens + i * 32);
  }
  grid_dep_launch();                             // the merge kernel may set up
  grid_dep_wait();                               // lengths, table, cache and q are written

  // ---------------------------------------------------------------- this CTA's range
  // CTA = (range, part of the head group); the range's rows are (sequence, K/V head)
  const int grp = H / Hkv, n_rg = (grp + RG - 1) / RG, rg = blockIdx.x % n_rg;
  const int nrow = min(RG, grp - rg * RG);       // heads of this part
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  // rows of this part of the head group without keys: O = 0, L = -inf
  auto empty_heads = [&](int b, int h_first, int n_heads) {
    const size_t at = static_cast<size_t>(b) * H + h_first;
    uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<T*>(O) + at * D);
    for (int i = threadIdx.x; i < n_heads * (D / 2); i += 32 * DP_WARPS) o[i] = 0u;
    for (int i = threadIdx.x; i < n_heads; i += 32 * DP_WARPS) L[at + i] = -INFINITY;
  };
  const int cta = blockIdx.x / n_rg;             // range index (direct: row)
  Header* hdr = reinterpret_cast<Header*>(ws);
  float* part = reinterpret_cast<float*>(ws + hdr_bytes(NT));
  Cursor cur;
  if (direct) {
    cur.b = cta / Hkv;
    cur.r = cta % Hkv;
    cur.s = seq_keys<KEYS, G::UNIT>(pg, cur.b, window);
    cur.u = cur.left = 0;
    cur.ue = cur.s.units;
    if (cur.ue == 0) {
      empty_heads(cur.b, cur.r * grp + rg * RG, nrow);
      return;
    }
  } else {
    const int per = (B + 32 * DP_WARPS - 1) / (32 * DP_WARPS);   // sequences per thread
    int mine = 0;
    for (int i = 0; i < per; ++i) {
      const int b = threadIdx.x * per + i;
      if (b < B) mine += row_cost(seq_keys<KEYS, G::UNIT>(pg, b, window).units) * Hkv;
    }
    int incl = mine;
#pragma unroll
    for (int w = 1; w < 32; w *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, incl, w);
      if (lane >= w) incl += o;
    }
    // [4] warps' sums, then the sequence that holds the range's start and its position
    volatile int* sc = reinterpret_cast<volatile int*>(smem_raw + (scan - raw));
    if (lane == 31) sc[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < DP_WARPS; ++w) {
      if (w < warp) before += sc[w];
      total += sc[w];
    }
    incl += before;
    const int n_cta = gridDim.x / n_rg;
    const int per_cta = max((total - 1) / n_cta + 1, 2);          // positions per CTA
    const int x0 = static_cast<int>(min(static_cast<long long>(cta) * per_cta,
                                        static_cast<long long>(total)));
    const int x1 = x0 + min(per_cta, total - x0);
    if (x0 < x1 && incl > x0 && incl - mine <= x0) {              // one thread holds position x0
      int at = incl - mine;
      for (int i = 0; i < per; ++i) {
        const int b = threadIdx.x * per + i;
        const int n = b < B ? row_cost(seq_keys<KEYS, G::UNIT>(pg, b, window).units) * Hkv : 0;
        if (at + n > x0) {
          sc[4] = b;
          sc[5] = at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    for (int b = blockIdx.x; b < B; b += gridDim.x)
      if (seq_keys<KEYS, G::UNIT>(pg, b, window).units == 0) empty_heads(b, 0, H);
    if (x0 >= x1) {
      if (threadIdx.x == 0) hdr[blockIdx.x].row = -1;
      return;
    }
    cur.b = sc[4];
    cur.s = seq_keys<KEYS, G::UNIT>(pg, cur.b, window);
    const int w = row_cost(cur.s.units), x = (x0 - sc[5]) % w, take = min(w - x, x1 - x0);
    cur.r = (x0 - sc[5]) / w;
    cur.u = x / 2;
    cur.ue = min(cur.s.units, (x + take) / 2);
    cur.left = x1 - x0 - take;
    Header h = {-1, 0, 0};
    if (cur.u > 0 && cur.u < cur.ue) {           // its unit 0 lies in an earlier CTA
      h.row = cur.b * Hkv + cur.r;
      h.c0 = (x0 - x + 1) / per_cta;
      h.c1 = (x0 - x + 2 * cur.s.units - 1) / per_cta;
    }
    if (threadIdx.x == 0) hdr[blockIdx.x] = h;
  }
  // to the range's units of the next row that has some; false at its end
  auto next_row = [&](Cursor& x) -> bool {
    do {
      if (x.left <= 0) return false;
      if (++x.r == Hkv) {
        x.r = 0;
        do {
          if (++x.b >= B) return false;          // not reached: `left` counts existing rows
          x.s = seq_keys<KEYS, G::UNIT>(pg, x.b, window);
        } while (x.s.units == 0);
      }
      const int take = min(row_cost(x.s.units), x.left);
      x.u = 0;
      x.ue = min(x.s.units, take / 2);
      x.left -= take;
    } while (x.u == x.ue);
    return true;
  };
  if (cur.u == cur.ue && !next_row(cur)) return;  // only positions without a unit

  // ---------------------------------------------------------------- this warp's ring
  // Tiles go out in the range's order, STAGES ahead of their use and across row borders.
  // Lane i fetches the page of the stage's box i one tile before it issues it.
  const int box = 1 << box_log2, n_box = KEYS >> box_log2;
  Cursor pr = cur;
  bool pr_more = true;
  int issued = 0, used = 0;
  int pid = -1, prow = 0, phk = 0;               // this lane's box of the tile to issue next
  bool p_has = false;
  // moves pr to the next tile this warp has, and starts the fetch of its pages
  auto fetch = [&]() {
    p_has = false;
    while (pr_more) {
      if (pr.u == pr.ue) {
        pr_more = next_row(pr);
        continue;
      }
      const int k0 = pr.s.a0 + (pr.u * DP_WARPS + warp) * KEYS;
      ++pr.u;
      if (k0 >= pr.s.n) continue;
      const int k = k0 + (lane << box_log2);
      const uint32_t p = pg.page.quot(k);
      prow = k - static_cast<int>(p * pg.page.div);
      phk = pr.r;
      pid = lane < n_box && k < pr.s.n ? pg.table[pr.b * pg.table_stride + p] : -1;
      p_has = true;
      return;
    }
  };
  // boxes of the tile in stage st whose page exists
  uint32_t okm[STAGES];
  auto issue = [&](int st) {
    const uint32_t bar = bars + st * 8, dst = ring + st * G::STAGEB;
    const bool ok = pid >= 0 && pid < pg.pages;
    okm[st] = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) mbar_arrive_expect_tx(bar, G::STAGEB);
    __syncwarp();
    if (lane < n_box) {
      const int w = ok ? pid : pg.pages;         // past the pool: the box reads as zeros
      const uint32_t d0 = dst + (lane << box_log2) * G::ROWB;
#pragma unroll
      for (int hf = 0; hf < G::HALVES; ++hf) {
        tma_load_4d(d0 + hf * G::BOXB, &tmK, bar, hf * G::BOXC, prow, phk, w);
        tma_load_4d(d0 + G::TILEB + hf * G::BOXB, &tmV, bar, hf * G::BOXC, prow, phk, w);
      }
    }
    ++issued;
  };
#pragma unroll
  for (int st = 0; st < STAGES; ++st) okm[st] = 0;
  {
    // the first stages' look-ups go out together
    int id0[STAGES], row0[STAGES], hk0[STAGES];
    bool has0[STAGES];
#pragma unroll
    for (int st = 0; st < STAGES; ++st) {
      fetch();
      id0[st] = pid;
      row0[st] = prow;
      hk0[st] = phk;
      has0[st] = p_has;
    }
    fetch();
    const int id1 = pid, row1 = prow, hk1 = phk;
#pragma unroll
    for (int st = 0; st < STAGES; ++st) {
      pid = id0[st];
      prow = row0[st];
      phk = hk0[st];
      if (has0[st]) issue(st);
    }
    pid = id1;
    prow = row1;
    phk = hk1;
  }

  // shared-memory byte offsets of this lane's ldmatrix rows: lane i gives row i % 8 of block
  // i / 8.  K blocks: (keys 0-7 | 8-15) x (chunk 0 | 1); V blocks for 16-bit caches: chunks
  // vary first, then keys; for codes: keys first, as for K.
  const int mr = lane & 7, m0 = (lane >> 3) & 1, m1 = lane >> 4;
  auto tile_off = [&](int key, int chunk) -> uint32_t {
    // 16-byte chunk `chunk` of a key's row, in the swizzled box layout
    const uint32_t off = key * G::ROWB + (chunk % (G::ROWB / 16)) * 16;
    return (chunk / (G::ROWB / 16)) * G::BOXB + (off ^ (((off >> 7) & G::SWM) << 4));
  };

  // Words of q of a row's heads 8 nt + g as they lie in memory: columns 16 ks + 2c (+ 1) and
  // + 8, or for codes 16 ks + 4c (+ 3), the order in which ldmatrix hands out the codes of K.
  // A row's words are loaded before the previous row is joined, which hides their latency.
  uint32_t qw[NT][KS][2];
  auto load_q = [&](const Cursor& x) {
    const size_t h0 = static_cast<size_t>(x.b) * H + x.r * grp + rg * RG;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t* q = static_cast<const uint32_t*>(Q) + (h0 + 8 * nt + g) * (D / 2);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qw[nt][ks][0] = qw[nt][ks][1] = 0u;
        if (8 * nt + g < nrow) {
          qw[nt][ks][0] = q[8 * ks + (C8 ? 2 : 1) * c];
          qw[nt][ks][1] = q[8 * ks + (C8 ? 2 * c + 1 : c + 4)];
        }
      }
    }
  };
  load_q(cur);

  bool ok = true, more = true;
  while (more) {
    // ---- one row segment: units [u, ue) of row r of sequence b
    const int seg_u = cur.u;
    const size_t h0 = static_cast<size_t>(cur.b) * H + cur.r * grp + rg * RG;
    // q as the products' second operand
    uint32_t qf[NT][KS][2];
    float cs[NT][2];                             // scale * log2(e) of this lane's heads 2c, 2c + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (C8 && BF16) {
        // bf16 q as f16 after an exact power-of-two scaling that brings the head's largest
        // magnitude to [1, 2), or below 4: no entry overflows, and an entry's 8 bits stay whole
        // down to 2^-17.  A smaller entry is off by at most 2^-25 (half of f16's least step):
        // times a code k, less than fp32's rounding of the largest entry times k.
        float mx = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = unpack2<true>(qw[nt][ks][e]);
            mx = fmax3(mx, fabsf(f.x), fabsf(f.y));
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the power of two at mx: its exponent bits, up to 2^126, whose reciprocal is a normal
        // number (0 and infinities: no scaling)
        uint32_t eb = __float_as_uint(mx) & 0x7f800000u;
        eb = eb == 0u || eb == 0x7f800000u ? 0x3f800000u : min(eb, 0x7e800000u);
        const float dn = __uint_as_float(0x7f000000u - eb);     // 1 / 2^e
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 f = unpack2<true>(qw[nt][ks][e]);
            qf[nt][ks][e] = pack2<false>(f.x * dn, f.y * dn);
          }
        // lane 4h holds head h's; never 0, which would make a masked score NaN (the least
        // normal number in its place moves no score by 2^-100), nor infinite, which would a
        // score of 0
        const float up = fminf(fmaxf(__uint_as_float(eb) * c_log2, 0x1p-126f), 0x1.fffffep127f);
        cs[nt][0] = __shfl_sync(0xffffffffu, up, 8 * c);
        cs[nt][1] = __shfl_sync(0xffffffffu, up, 8 * c + 4);
      } else {
        cs[nt][0] = cs[nt][1] = c_log2;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          qf[nt][ks][0] = qw[nt][ks][0];
          qf[nt][ks][1] = qw[nt][ks][1];
        }
      }
    }
    float m[NT][2], l[NT][2], acc[NT][KS][4];    // heads 8 nt + 2c, + 1; columns g (+ 8) of each 16
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][i][e] = 0.f;
    }

    for (; cur.u < cur.ue && ok; ++cur.u) {
      const int k0 = cur.s.a0 + (cur.u * DP_WARPS + warp) * KEYS;
      if (k0 >= cur.s.n) continue;
      const int st = used % STAGES;
      if (!(ok = mbar_wait_warp(bars + st * 8, (used / STAGES) & 1, ctl))) break;
      const uint32_t kt = ring + st * G::STAGEB, vt = kt + G::TILEB;
      uint32_t have = okm[0];
#pragma unroll
      for (int i = 1; i < STAGES; ++i)
        if (st == i) have = okm[i];
      // keys of the tile that are attended: [klo, khi), less those of absent pages
      const int klo = max(cur.s.lo - k0, 0), khi = min(cur.s.n - k0, KEYS);
      const uint32_t all = n_box == 32 ? 0xffffffffu : (1u << n_box) - 1u;
      const bool edge = klo > 0 || khi < KEYS || have != all;
      if (klo > 0 || khi < KEYS) {
        // V rows outside may hold anything, and 0 x NaN is NaN: clear them
        for (int i = lane; i < KEYS * (D * G::ELEM / 16); i += 32) {
          const int key = i % KEYS, ch = i / KEYS;
          if (key < klo || key >= khi)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + tile_off(key, ch)),
                         "r"(0u)
                         : "memory");
        }
        fence_proxy_async_smem();                // before a later copy into this stage
        __syncwarp();
      }

      // S^T of the tile: keys 16 mt + g (+ 8), heads 8 nt + 2c, + 1
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
        if constexpr (C8) {
#pragma unroll
          for (int kp = 0; kp < KS / 2; ++kp) {
            uint32_t w[4];
            ldsm4(kt + tile_off(16 * mt + mr + 8 * m0, 2 * kp + m1), w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a[4] = {codes_lo(w[2 * h]), codes_lo(w[2 * h + 1]),
                                     codes_hi(w[2 * h]), codes_hi(w[2 * h + 1])};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma<MB>(s[mt][nt], a, qf[nt][2 * kp + h][0], qf[nt][2 * kp + h][1]);
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            uint32_t a[4];
            ldsm4(kt + tile_off(16 * mt + mr + 8 * m0, 2 * ks + m1), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma<MB>(s[mt][nt], a, qf[nt][ks][0], qf[nt][ks][1]);
          }
        }
      }
      if (edge) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const int key = 16 * mt + 8 * hf + g;
            if (key < klo || key >= khi || !((have >> (key >> box_log2)) & 1u)) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) s[mt][nt][2 * hf] = s[mt][nt][2 * hf + 1] = -INFINITY;
            }
          }
      }
      // Running maximum, moved only when some score of the warp exceeds it by 2^8 (then
      // every lane of a head takes the head's new maximum): numerator and denominator carry
      // the same m, so a stale one changes nothing, and p <= 2^(SH + 8).
      bool rise = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = -INFINITY;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) v = fmax3(v, s[mt][nt][e], s[mt][nt][2 + e]);
          mx[nt][e] = v * cs[nt][e];
          rise |= mx[nt][e] > m[nt][e] + (SH + 8.0f);
        }
      if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = mx[nt][e];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            const float mn = fmaxf(m[nt][e], v - SH), al = weight(m[nt][e], mn);
            m[nt][e] = mn;
            l[nt][e] *= al;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              acc[nt][i][e] *= al;
              acc[nt][i][2 + e] *= al;
            }
          }
      }
      // p = 2^(s c - m); P^T as 16-bit hi + lo terms, transposed into the second operand
      uint32_t ph[MT][NT][2], pl[MT][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float ma = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
        const float mb = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const float pa = ex2(fmaf(s[mt][nt][2 * hf], cs[nt][0], -ma));
            const float pb = ex2(fmaf(s[mt][nt][2 * hf + 1], cs[nt][1], -mb));
            l[nt][0] += pa;
            l[nt][1] += pb;
            const uint32_t hi = pack2<MB>(pa, pb);
            const float2 back = unpack2<MB>(hi);
            ph[mt][nt][hf] = movm_t(hi);
            pl[mt][nt][hf] = movm_t(pack2<MB>(pa - back.x, pb - back.y));
          }
      }
      // O^T += V^T P^T over the tile's 16-key steps
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if constexpr (C8) {
          // blocks: (keys 0-7 | 8-15) x (chunk 2j | 2j + 1); a transposed block of code pairs
          // holds columns 2g, 2g + 1 of its chunk for keys 2c, 2c + 1: the even columns make
          // one fragment of 16 output columns, the odd ones the next
#pragma unroll
          for (int j = 0; j < KS / 2; ++j) {
            uint32_t w[4];
            ldsm4_t(vt + tile_off(16 * mt + mr + 8 * m0, 2 * j + m1), w);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = even_odd(w[i]);
            const uint32_t ae[4] = {codes_lo(w[0]), codes_lo(w[2]), codes_lo(w[1]), codes_lo(w[3])};
            const uint32_t ao[4] = {codes_hi(w[0]), codes_hi(w[2]), codes_hi(w[1]), codes_hi(w[3])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<MB>(acc[nt][2 * j], ae, ph[mt][nt][0], ph[mt][nt][1]);
              mma<MB>(acc[nt][2 * j], ae, pl[mt][nt][0], pl[mt][nt][1]);
              mma<MB>(acc[nt][2 * j + 1], ao, ph[mt][nt][0], ph[mt][nt][1]);
              mma<MB>(acc[nt][2 * j + 1], ao, pl[mt][nt][0], pl[mt][nt][1]);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            uint32_t a[4];
            ldsm4_t(vt + tile_off(16 * mt + mr + 8 * m1, 2 * i + m0), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma<MB>(acc[nt][i], a, ph[mt][nt][0], ph[mt][nt][1]);
              mma<MB>(acc[nt][i], a, pl[mt][nt][0], pl[mt][nt][1]);
            }
          }
        }
      }
      __syncwarp();                              // stage read by every lane
      ++used;
      if (p_has) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i)
          if (st == i) issue(i);
        fetch();
      }
    }

    const bool whole = seg_u == 0 && cur.ue == cur.s.units;
    // warps that had keys: all, or the first few of a segment shorter than a unit
    const int n_warps = cur.ue - seg_u > 1 ? DP_WARPS
        : (cur.s.n - cur.s.a0 - seg_u * G::UNIT + KEYS - 1) / KEYS;
    cur.u = cur.ue;
    more = next_row(cur);
    if (more) load_q(cur);
    // ---- join the warps: 2, 3 into 0, 1, then 1 into 0, through shared memory
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int w = 4; w <= 16; w *= 2) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], w);
    constexpr int HS = (D + 4) * 4;              // bytes of a head's state
    auto put = [&](uint32_t at, int nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t p = at + (2 * c + e) * HS;
        if (g == 0) {
          st_f32(p, m[nt][e]);
          st_f32(p + 4, l[nt][e]);
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          st_f32(p + (4 + 16 * i + g) * 4, acc[nt][i][e]);
          st_f32(p + (4 + 16 * i + 8 + g) * 4, acc[nt][i][2 + e]);
        }
      }
    };
    auto join = [&](uint32_t at, int nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t p = at + (2 * c + e) * HS;
        const float mo = ld_f32(p), lo = ld_f32(p + 4);
        const float mn = fmaxf(m[nt][e], mo);
        const float wa = weight(m[nt][e], mn), wb = weight(mo, mn);
        m[nt][e] = mn;
        l[nt][e] = l[nt][e] * wa + lo * wb;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          acc[nt][i][e] = acc[nt][i][e] * wa + ld_f32(p + (4 + 16 * i + g) * 4) * wb;
          acc[nt][i][2 + e] = acc[nt][i][2 + e] * wa + ld_f32(p + (4 + 16 * i + 8 + g) * 4) * wb;
        }
      }
    };
    static_assert(DP_WARPS == 4, "two-level join of four warps");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (nt * 8 >= nrow || n_warps == 1) continue;   // the same for the whole CTA
      __syncthreads();                           // earlier readers of the two buffers are done
      if (n_warps > 2) {
        if (warp >= 2) put(red + (warp - 2) * 8 * HS, nt);
        __syncthreads();
        if (warp < 2) join(red + warp * 8 * HS, nt);
        __syncthreads();
      }
      if (warp == 1) put(red, nt);
      __syncthreads();
      if (warp == 0) join(red, nt);
    }
    // ---- a row that is whole in this CTA gives its result, one cut by a border its state
    if (warp == 0) {
      const int slot = seg_u > 0 ? 0 : 1;
      float* rec = part + (static_cast<size_t>(blockIdx.x) * 2 + slot) * RG * (D + 4);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 8 * nt + 2 * c + e;
          if (row >= nrow) continue;
          const float lr = l[nt][e], f = whole ? (lr == 0.f ? 0.f : o_scale / lr) : 1.f;
          T* o = static_cast<T*>(O) + (h0 + row) * D;
          float* pr_ = rec + row * (D + 4);
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              const int col = C8 ? 32 * (i / 2) + 16 * hf + 2 * g + (i & 1) : 16 * i + 8 * hf + g;
              const float v = lr == 0.f ? 0.f : acc[nt][i][2 * hf + e] * f;
              if (whole) {
                if constexpr (BF16) o[col] = __float2bfloat16_rn(v);
                else o[col] = __float2half_rn(v);
              } else {
                pr_[4 + col] = v;
              }
            }
          if (g == 0) {
            if (whole) {
              L[h0 + row] = lr == 0.f ? -INFINITY : (m[nt][e] + log2f(lr)) * 0.69314718055994531f;
            } else {
              pr_[0] = m[nt][e];
              pr_[1] = lr;
            }
          }
        }
    }
  }
  // after a wait that ran out (recorded in the status word): the copies still in flight land
  // (bounded) before the CTA's shared memory is released
  for (int i = used; i < issued; ++i)
    mbar_wait_warp(bars + (i % STAGES) * 8, (i / STAGES) & 1, ctl);
}

// Joins the states of a row cut by range borders: CTA c takes part for the row it shares with
// CTA c - 1.  The CTAs of one row divide its outputs among them, four columns at a time; the
// states of one output are divided among 2^gs threads, so that a thread has few loads, all
// in flight at once (their latency is what this kernel takes), and joined through shared
// memory in a fixed order.  It does not let the next kernel start early: CTAs of the next
// call's split kernel, three to an SM with all of its registers, would be placed around this
// kernel's, and where a hole of the wrong size is left between them the third has to wait for
// another to end (0.276 against 0.240 ms a call with 16 caches of up to 32768 keys).
template <int D, bool BF16>
__global__ void __launch_bounds__(DP_MERGE_THREADS)
    decode_paged_merge_kernel(const uint8_t* ws, void* O, float* L, int H, int Hkv, int NT,
                              float o_scale) {
  constexpr int PER = 8;                         // states a thread loads at once
  __shared__ float sh[DP_MERGE_THREADS][7];      // m, l, acc; rows of 7 words: no bank conflicts
  grid_dep_wait();                               // the split kernel's states
  const Header h = reinterpret_cast<const Header*>(ws)[blockIdx.x];
  if (h.row < 0) return;
  const float* part = reinterpret_cast<const float*>(ws + hdr_bytes(NT));
  const int RG = 8 * NT, grp = H / Hkv, n_rg = (grp + RG - 1) / RG;
  const int x = blockIdx.x / n_rg, rg = blockIdx.x % n_rg;
  const int b = h.row / Hkv, hk = h.row % Hkv;
  const int nrow = min(RG, grp - rg * RG);
  const size_t h0 = static_cast<size_t>(b) * H + hk * grp + rg * RG;
  const int n_sl = h.c1 - h.c0, sl = x - h.c0 - 1, n = n_sl + 1;
  int gs = 0;                                    // up to 16 threads per output, PER / 2 states each
  while (gs < 4 && (PER / 2 << gs) < n) ++gs;
  const int tg = threadIdx.x & ((1 << gs) - 1), outs = DP_MERGE_THREADS >> gs;
  const int n_out = nrow * (D / 4);
  const size_t step = static_cast<size_t>(2) * n_rg * RG * (D + 4);
  for (int base = sl * outs; base < n_out; base += n_sl * outs) {   // the same for the whole CTA
    const int i = base + (threadIdx.x >> gs);
    const int row = i / (D / 4), col = 4 * (i % (D / 4));
    float m = -INFINITY, l = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < n_out) {
      const float* p1 =
          part + (static_cast<size_t>(h.c0) * n_rg + rg) * 2 * RG * (D + 4) + row * (D + 4);
      for (int k0 = tg; k0 < n; k0 += PER << gs) {
        float2 ml[PER];
        float4 v[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const int k = k0 + (e << gs);
          ml[e] = make_float2(-INFINITY, 0.f);
          v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < n) {
            const float* p = p1 + k * step + (k == 0 ? RG * (D + 4) : 0);   // the first: slot 1
            ml[e] = *reinterpret_cast<const float2*>(p);
            v[e] = *reinterpret_cast<const float4*>(p + 4 + col);
          }
        }
        float mn = m;
#pragma unroll
        for (int e = 0; e < PER; ++e) mn = fmaxf(mn, ml[e].x);
        float w = weight(m, mn);
        m = mn;
        l *= w;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] *= w;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          w = weight(ml[e].x, mn);
          l = fmaf(ml[e].y, w, l);
          a[0] = fmaf(v[e].x, w, a[0]);
          a[1] = fmaf(v[e].y, w, a[1]);
          a[2] = fmaf(v[e].z, w, a[2]);
          a[3] = fmaf(v[e].w, w, a[3]);
        }
      }
    }
    if (gs > 0) {
      float* s = sh[threadIdx.x];
      s[0] = m; s[1] = l;
#pragma unroll
      for (int e = 0; e < 4; ++e) s[2 + e] = a[e];
      __syncthreads();
      if (tg == 0) {
        float mn = m;
        for (int k = 1; k < 1 << gs; ++k) mn = fmaxf(mn, s[7 * k]);
        float w = weight(m, mn);
        m = mn;
        l *= w;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] *= w;
        for (int k = 1; k < 1 << gs; ++k) {
          w = weight(s[7 * k], mn);
          l = fmaf(s[7 * k + 1], w, l);
#pragma unroll
          for (int e = 0; e < 4; ++e) a[e] = fmaf(s[7 * k + 2 + e], w, a[e]);
        }
      }
      __syncthreads();
    }
    if (tg == 0 && i < n_out) {
      const float f = l == 0.f ? 0.f : o_scale / l;
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = l == 0.f ? 0.f : a[e] * f;
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(O) + (h0 + row) * D + col) =
          make_uint2(pack2<BF16>(a[0], a[1]), pack2<BF16>(a[2], a[3]));
      if (col == 0) L[h0 + row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
  }
}

// Column blocks of a CTA's products: two when a group has more than 8 heads.
int n_blocks(int H, int Hkv) { return H / Hkv > 8 ? 2 : 1; }

// Whether each of `rows` rows of at most `units` units gets a CTA of its own.  Measured with
// 32/8 heads, d = 128, bf16, lengths up to 64 `units`, rows cut against whole (us):
//   8 units     1 sequence 7.7 / 7.7     8: 9.4 / 9.4     32: 16.8 / 13.0   256: 71.8 / 63.3
//   16 units    1: 8.2 / 11.5            16: 16.6 / 17.4  32: 24.5 / 21.2   256: 127 / 115
//   32 units    16: 24.5 / 30.1          64: 67.4 / 68.3  128: 123 / 119    256: 239 / 222
// Longer rows are cut however many there are: one that is much longer than the others would
// keep one CTA busy after all the rest.
bool rows_direct(long long units, long long rows, int slots) {
  return units <= 8 || (units <= 16 && rows >= 152) || (units <= 32 && rows >= 2 * slots);
}

// Ranges of a call, and whether they are its rows.
struct Plan {
  long long ranges;
  bool direct;
};
Plan plan(const DecodePagedArgs& a, int d, bool c8, int nt) {
  const long long cap = static_cast<long long>(a.pg.max_pages) * a.pg.page.div;
  const long long longest = a.window > 0 && a.window < cap ? a.window : cap;
  const long long cost = decode_paged_cost(a.Hkv, d, c8, longest), rows = 1LL * a.B * a.Hkv;
  const int n_rg = (a.H / a.Hkv + 8 * nt - 1) / (8 * nt);
  if (rows_direct((cost / a.Hkv - 1) / 2, rows * n_rg, grid_of(nt))) return {rows, true};
  // at least two positions per range, ranges no more than run at once
  const long long most = a.B * cost / 2, fit = grid_of(nt) / n_rg;
  return {most < fit ? (most > 1 ? most : 1) : fit, false};
}

template <int D, bool BF16, bool C8, int NT>
cudaError_t launch_t(const DecodePagedArgs& a, cudaStream_t st) {
  auto kern = decode_paged_kernel<D, BF16, C8, NT>;
  constexpr int smem = smem_bytes<D, C8, NT>();
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const Plan pl = plan(a, D, C8, NT);
  const int n_rg = (a.H / a.Hkv + 8 * NT - 1) / (8 * NT);
  const long long ranges = pl.ranges;
  const bool direct = pl.direct;
  if (ranges * n_rg > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(ranges * n_rg);
  uint8_t* ws = static_cast<uint8_t*>(a.ws);
  trace_begin(TR_DEC_SPLIT, st);
  e = launch_dependent(kern, grid, 32 * DP_WARPS, smem, st, a.tmK, a.tmV, a.Q, a.O, a.L, ws, a.B,
                       a.H, a.Hkv, a.window, static_cast<int>(direct), a.box_log2, a.c_log2, a.o_scale,
                       a.pg, a.ctl);
  trace_end(TR_DEC_SPLIT, st);
  if (e != cudaSuccess || direct || ranges == 1) return e;   // no row is cut
  trace_begin(TR_DEC_MERGE, st);
  e = launch_dependent(decode_paged_merge_kernel<D, BF16>, grid, DP_MERGE_THREADS, 0, st,
                       static_cast<const uint8_t*>(ws), a.O, a.L, a.H, a.Hkv, NT, a.o_scale);
  trace_end(TR_DEC_MERGE, st);
  return e;
}

template <int D, bool BF16, bool C8>
cudaError_t launch_nt(const DecodePagedArgs& a, cudaStream_t st) {
  return n_blocks(a.H, a.Hkv) == 2 ? launch_t<D, BF16, C8, 2>(a, st)
                                   : launch_t<D, BF16, C8, 1>(a, st);
}

}  // namespace

int decode_paged_keys(int d, bool c8) { return 4096 / (d * (c8 ? 1 : 2)); }

long long decode_paged_cost(int Hkv, int d, bool c8, long long n) {
  // a window may start inside a stage: up to KEYS - 1 more keys
  const int keys = decode_paged_keys(d, c8), unit = DP_WARPS * keys;
  return (2 * ((n + keys - 1 + unit - 1) / unit) + 1) * Hkv;
}

bool decode_paged_group_fits(int H, int Hkv) {
  const int nt = n_blocks(H, Hkv);
  return (H / Hkv + 8 * nt - 1) / (8 * nt) <= grid_of(nt);
}

bool decode_paged_cuts_rows(const DecodePagedArgs& a, int d, bool c8) {
  return !plan(a, d, c8, n_blocks(a.H, a.Hkv)).direct;
}

size_t decode_paged_ws_bytes(int H, int Hkv, int d) {
  const int nt = n_blocks(H, Hkv);
  return hdr_bytes(nt) + static_cast<size_t>(grid_of(nt)) * 2 * 8 * nt * (d + 4) * 4;
}

cudaError_t launch_decode_paged(const DecodePagedArgs& a, int d, bool bf16, bool c8,
                                cudaStream_t st) {
  if (c8) {
    if (d != 128) return cudaErrorInvalidValue;
    return bf16 ? launch_nt<128, true, true>(a, st) : launch_nt<128, false, true>(a, st);
  }
  if (d == 32) return bf16 ? launch_nt<32, true, false>(a, st) : launch_nt<32, false, false>(a, st);
  if (d == 64) return bf16 ? launch_nt<64, true, false>(a, st) : launch_nt<64, false, false>(a, st);
  if (d == 128)
    return bf16 ? launch_nt<128, true, false>(a, st) : launch_nt<128, false, false>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace fa
