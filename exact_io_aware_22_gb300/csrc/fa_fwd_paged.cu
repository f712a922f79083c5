// fa_fwd_paged.cu -- the forward of many new tokens over a paged key/value cache.
//
// Mathematics: the forward's (running maximum m, running sum l, correction alpha applied to l
// and the accumulator together, one divide at the end, L = m + log l; "flash-attn-triton" docs
// page, "Tiling softmax is exact algebra" and Fig. 3), in base 2.  The new tokens of a sequence
// are its last positions: query i of nq sees keys up to i + (keys - nq).
//
// Two kernels, as in the dense forward: at d = 128 one CTA per SM with two query tiles, at
// d <= 64 a persistent one, two CTAs per SM, one query tile at a time.  Their pipelines are the
// dense kernels' (TMA producer, one MMA issuer, a softmax thread per query row; S, P and O in
// tensor memory).  What pages change:
//   producer   a whole warp.  Each lane looks up the pages of its boxes (the largest power of
//              two of rows that divides the page size) one tile ahead and loads them; a 128-row
//              tile lies in shared memory as one box would.  Boxes of absent pages read as
//              zeros and their keys are masked; V rows past the last key, which may hold
//              anything, are cleared before the product that reads them (0 x NaN).
//   tiles      A query tile holds the rows of 2^pack heads that share a K/V head, heads fastest:
//              the tile of a few new tokens is better filled, K and V pass once for those
//              heads, and less of a tile lies beyond the diagonal (5 tokens of 4 sequences of
//              2000 keys, 32/8 heads, d = 128: 33.4 against 17.7 us with the split below;
//              8 prompts of 1000: 110 against 100 us).
//   split      Where there are fewer query tiles than the GPU runs at once, the KV tiles of
//              each are cut into ranges of equal length for as many CTAs, whose results, each
//              normalised with its own L, fwd_paged_merge_kernel joins by their weights
//              2^(L_s - L).
//
// Bound: at d = 128 the tensor pipe and the exponentials (2 x 2048 tokens on 8192 keys, 32/8
// heads: 0.342 ms, 1394 TFLOP/s), at d <= 64 the exponentials and the softmax threads' issue
// slots; with few tokens the latency of start, split and join (the 5 tokens above: 17.3 us for
// 34 MB of keys).
//
// The kernels stand apart from fa_fwd.cu's although the pipelines are alike: pages, packed heads
// and ranges reach into every role, and the dense kernels' code does not change with them.
#include "fa_internal.h"
#include "fa_ptx.cuh"

namespace fa {

namespace {

constexpr int BM = 128;       // query rows per Q tile (= TMEM lanes)
constexpr int BN = 128;       // keys per K/V tile
constexpr int NT = 2;         // Q tiles per CTA
constexpr int THREADS = 384;
constexpr float RESCALE_LOG2 = 8.0f;   // the running maximum moves in steps of 2^8 or more
// P is formed with 2^7 times its weight where it is f16 (p <= 2^15), so that the small p of a
// long context, which add up, stay clear of f16's subnormals; l carries the same factor.
template <bool BF16>
constexpr float P_LOG2 = BF16 ? 0.f : 7.f;
constexpr int kMaskSlots = 8;         // ring of 128-bit key masks, one per KV tile

template <int D>
struct Cfg {
  static constexpr int STAGES = D == 128 ? 2 : 3;
  static constexpr int SW = D == 32 ? 64 : 128;        // swizzle width in bytes
  static constexpr int ATOM = SW / 2;                  // elements per swizzled row
  static constexpr int NCHUNK = D / ATOM;              // swizzle-width column blocks per tile
  static constexpr int CHUNK_BYTES = 128 * SW;         // one column block of a 128-row tile
  static constexpr int TILE_BYTES = 128 * D * 2;
  static constexpr uint32_t SWZ = D == 32 ? UMMA_SW64 : UMMA_SW128;
  static constexpr int Q_OFF = 0;
  static constexpr int K_OFF = Q_OFF + NT * TILE_BYTES;
  static constexpr int V_OFF = K_OFF + STAGES * TILE_BYTES;
  static constexpr int BAR_OFF = V_OFF + STAGES * TILE_BYTES;
  // q_full, k_full[S], k_empty[S], v_full[S], v_empty[S], s_full[2], p_full[2], o_full[2], done
  static constexpr int NBARS = 1 + 4 * STAGES + 7;
  static constexpr int SLOT_OFF = BAR_OFF + NBARS * 8;
  static constexpr int MASK_OFF = (SLOT_OFF + 16 + 15) / 16 * 16;
  static constexpr int SMEM_BYTES = MASK_OFF + kMaskSlots * 16 + 1024;   // + alignment slack
  static constexpr int TMEM_COLS = 512;
  static constexpr int S_COL = 0;                           // S_t at t * 128
  static constexpr int O_COL = 256;                         // O_t at 256 + t * D
};

// byte offset of k-step kk (16 elements along K) inside a K-major tile
template <int D>
__device__ __forceinline__ uint32_t kmajor_koff(int kk) {
  using C = Cfg<D>;
  const int e = kk * 16;
  return (e / C::ATOM) * C::CHUNK_BYTES + (e % C::ATOM) * 2;
}

struct PagedArgs {
  PagedView pg;
  int box_log2, causal, window;    // window: kNoLimit for none
  int pack;                        // log2 of the heads in a query tile
  int n_split;                     // KV ranges per query tile (1: no workspace)
  size_t rows;                     // (query, head) pairs of all sequences: B * max_seqlen * H
  float* part;                     // [n_split][rows][D] results of the ranges
  float* part_l;                   // [n_split][rows] their logsumexp (natural log)
};
constexpr int kNoLimit = 1 << 30;
// Keys of a sequence with nq query rows: query row i is at key position i + off and sees keys
// up to i + hi (all of them unless causal) and from i + off - window + 1.
struct KeyRows {
  int n, off, hi;
};
// Query and key rows of sequence b; the three loads go out together.
__device__ __forceinline__ void rows_of(const PagedArgs& px, const int* cu, int b, int N,
                                        int total, SeqRows& sr, KeyRows& k) {
  const int c0 = cu[b], c1 = cu[b + 1], len = px.pg.seqlens[b];
  const int a = min(max(c0, 0), total), e = min(max(c1, a), total);
  sr = {a, min(e - a, N), true};
  const long long cap = static_cast<long long>(px.pg.max_pages) * px.pg.page.div;
  k.n = static_cast<int>(min(static_cast<long long>(max(len, 0)), cap));
  k.off = k.n - (e - a);                         // rows past N are left out, the others stay
  k.hi = px.causal ? k.off : kNoLimit;
}
// KV tiles [lo, hi) of the query tile at rows r .. r + BM - 1 of a sequence's nr; row i is
// a head of query i >> pack.
__device__ __forceinline__ void paged_tiles(const KeyRows& k, int r, int nr, int window, int pack,
                                            int& lo, int& hi) {
  const int last = (min(r + BM - 1, nr - 1) >> pack) + k.hi;
  hi = r >= nr || last < 0 ? 0 : min((k.n + BN - 1) / BN, last / BN + 1);
  lo = min(max(0, (r >> pack) + k.off - window + 1) / BN, hi);
}
// How the KV tiles [lo, hi) of `TILES` query tiles from row r are cut: ranges of `per` tiles,
// `used` of them (at least one).
struct SplitRange {
  int lo, hi, per, used;
};
template <int TILES>
__device__ __forceinline__ SplitRange split_range(const KeyRows& k, int r, int nr, int window,
                                                  int pack, int n_split) {
  SplitRange s;
  paged_tiles(k, r, nr, window, pack, s.lo, s.hi);
#pragma unroll
  for (int t = 1; t < TILES; ++t) {
    int lo, hi;
    paged_tiles(k, r + t * BM, nr, window, pack, lo, hi);
    if (hi > s.hi) s.hi = hi;                    // lo rises with the row
  }
  // two tiles at least: the join costs about as much as one
  s.per = max((s.hi - s.lo + n_split - 1) / n_split, n_split > 1 ? 2 : 1);
  s.used = max((s.hi - s.lo + s.per - 1) / s.per, 1);
  return s;
}

// One warp's loads of 128-key tiles of a paged cache.  Lane i handles boxes i, i + 32, ...
struct PagedTile {
  int id[4], row[4];               // page id as the table has it, and first row in the page
  int past;                        // bit i: box lane + 32 i lies past the keys
};
// Starts the tile's table loads.  Nothing here uses what they return: the warp would stand
// still for a load's latency instead of issuing the tile before this one.
__device__ __forceinline__ void paged_fetch(const PagedArgs& px, int b, const KeyRows& k,
                                            int krow, int lane, PagedTile& t) {
  const int n_box = BN >> px.box_log2;
  t.past = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int bx = lane + 32 * i, key = krow + (bx << px.box_log2);
    t.id[i] = -1;
    t.row[i] = 0;
    if (bx < n_box && key < k.n) {
      const int p = static_cast<int>(px.pg.page.quot(key));
      t.row[i] = key - p * static_cast<int>(px.pg.page.div);
      t.id[i] = px.pg.table[b * px.pg.table_stride + p];
    } else {
      t.past |= 1 << i;
    }
  }
}
__device__ __forceinline__ bool paged_in_pool(const PagedArgs& px, int id) {
  return id >= 0 && id < px.pg.pages;
}
// Keys of the tile that exist, as 128 bits, to the ring slot at `slot` (all lanes call).
__device__ __forceinline__ void paged_mask(const PagedArgs& px, int lane, const PagedTile& t,
                                           uint32_t slot) {
  uint32_t have = t.past;                        // keys past the end are masked by their index
#pragma unroll
  for (int i = 0; i < 4; ++i) have |= (paged_in_pool(px, t.id[i]) ? 1u : 0u) << i;
  uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
  if (__any_sync(0xffffffffu, have != 15u)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int bx = (32 * i + lane) >> px.box_log2;      // the box of key 32 i + lane
      const uint32_t h = __shfl_sync(0xffffffffu, have, bx & 31);
      w[i] = __ballot_sync(0xffffffffu, (h >> (bx >> 5)) & 1u);
    }
  }
  if (lane == 0)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(slot),
                 "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                 : "memory");
}
template <int D>
__device__ __forceinline__ void paged_load(const PagedArgs& px, const CUtensorMap* map,
                                           uint32_t dst, uint32_t bar, int hk, int lane,
                                           const PagedTile& t) {
  using C = Cfg<D>;
  const int n_box = BN >> px.box_log2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int bx = lane + 32 * i;
    if (bx < n_box) {
      const int w = paged_in_pool(px, t.id[i]) ? t.id[i] : px.pg.pages;   // past the pool: zeros
#pragma unroll
      for (int c = 0; c < C::NCHUNK; ++c)
        tma_load_4d(dst + c * C::CHUNK_BYTES + (bx << px.box_log2) * C::SW, map, bar, c * C::ATOM,
                    t.row[i], hk, w);
    }
  }
}
// Which keys a row of a paged query tile may attend, [lo, lim), and where a KV tile needs
// masks at all: above `full` for the tile's first row, below `past` for its last.
struct RowKeys {
  int lo, lim, past, full;
};
__device__ __forceinline__ RowKeys row_keys(const KeyRows& k, int row0, int row, int pack,
                                            int window) {
  RowKeys r;
  r.lim = min((row >> pack) + k.hi + 1, k.n);
  r.lo = (row >> pack) + k.off - window + 1;
  r.full = min((row0 >> pack) + k.hi + 1, k.n);
  r.past = ((row0 + BM - 1) >> pack) + k.off - window + 1;
  return r;
}
// A KV tile's mask in the ring, a bit per key whose page is there.  The d = 128 kernel reads it
// before it waits for the scores (2 x 2048 tokens: 350 against 345 us); at d <= 64 the order
// made no difference.
__device__ __forceinline__ void load_mask(uint32_t slot, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "r"(slot)
               : "memory");
}
// Masks a row's scores with the keys kbase .. kbase + BN - 1: those outside [lo, lim) and those
// of absent pages (w).  One block for all of them, entered for
// few tiles: separate ones cost the unmasked tiles more (1 x 8192, 32 heads, d = 128: 393
// against 371 us).  At d <= 64 words of 32 keys that are whole are skipped, which most of a
// diagonal tile's are (ragged prompts, window 512: 38.4 against 36.4 us); the branches cost
// the d = 128 kernel more than they save (2 x 2048 tokens: 350 against 355 us).
template <bool WORDS>
__device__ __forceinline__ void paged_masks(const RowKeys& r, int kbase, uint32_t (&w)[4],
                                            uint32_t (&s)[BN]) {
  if (kbase + BN <= r.full && kbase >= r.past && (w[0] & w[1] & w[2] & w[3]) == ~0u) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int hi = r.lim - kbase - 32 * i, lo = r.lo - kbase - 32 * i;   // bits [lo, hi) stay
    if (hi < 32) w[i] &= hi > 0 ? (1u << hi) - 1u : 0u;
    if (lo > 0) w[i] &= lo < 32 ? ~0u << lo : 0u;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (WORDS && w[i] == ~0u) continue;
#pragma unroll
    for (int c = 32 * i; c < 32 * i + 32; ++c)
      if (!((w[i] >> (c % 32)) & 1u)) s[c] = __float_as_uint(-INFINITY);
  }
}
// Clears row r of a V tile (all its columns, so the swizzle does not matter).
template <int D>
__device__ __forceinline__ void clear_row(uint32_t tile, int r) {
  using C = Cfg<D>;
#pragma unroll
  for (int c = 0; c < C::NCHUNK; ++c)
#pragma unroll
    for (int i = 0; i < C::SW / 16; ++i)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                       tile + c * C::CHUNK_BYTES + r * C::SW + 16 * i),
                   "r"(0u)
                   : "memory");
}

template <int D, bool BF16>
__global__ void __launch_bounds__(THREADS, 1)
    fwd_paged_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, void* __restrict__ Out,
                     float* __restrict__ Lout, int N, int n_qblk, int group, const int* cu_seqlens,
                     int H, int total, float c_log2, KernelCtl ctl, const PagedArgs px) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sg = smem_raw + (sb - raw);

  grid_dep_launch();                            // the next kernel may start setting up
  grid_dep_wait();                              // offsets, lengths, table and inputs are written
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const BlockPos bp = block_pos(n_qblk);        // bp.bh: (sequence, block of heads, KV range)
  const int pack = px.pack, blocks = H >> pack;
  const int split = bp.bh % px.n_split, bh = bp.bh / px.n_split;
  const int b = bh / blocks;
  const int hq = (bh % blocks) << pack, hk = hq / group;   // the tile's first head, its K/V head
  const int qblk = n_qblk - 1 - bp.rank;        // the last query tiles have the most work
  SeqRows sr;
  KeyRows kr;
  rows_of(px, cu_seqlens, b, N, total, sr, kr);
  const int Nr = sr.n << pack, Nk = kr.n;       // query rows, keys
  const int row0 = qblk * (NT * BM);
  // KV tiles [lo_t[t], n_t[t]) of Q tile t, cut to this CTA's range of those of both
  const SplitRange sp = split_range<NT>(kr, row0, Nr, px.window, pack, px.n_split);
  if (split >= sp.used) return;
  const bool shared = sp.used > 1;              // the tile's other ranges are other CTAs'
  const int j0 = sp.lo + split * sp.per, n_max = min(j0 + sp.per, sp.hi);
  int n_t[NT], lo_t[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    paged_tiles(kr, row0 + t * BM, Nr, px.window, pack, lo_t[t], n_t[t]);
    lo_t[t] = min(max(lo_t[t], j0), n_max);
    n_t[t] = min(max(n_t[t], j0), n_max);
  }
  const int n_stream = n_max - j0;              // KV tiles loaded, j0 .. n_max - 1
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  // where row `grow` lies in O, in the workspace, and in L or the workspace's L
  auto row_at = [&](int grow) -> size_t {
    return static_cast<size_t>(sr.base + (grow >> pack)) * H + hq + (grow & ((1 << pack) - 1));
  };
  auto part_at = [&](int grow) -> size_t {
    return split * px.rows + (static_cast<size_t>(b) * N + (grow >> pack)) * H + hq +
           (grow & ((1 << pack) - 1));
  };
  auto lse_at = [&](int grow) -> float* {
    if (shared) return px.part_l + part_at(grow);
    return Lout + static_cast<size_t>(hq + (grow & ((1 << pack) - 1))) * total + sr.base +
           (grow >> pack);
  };
  // row `grow` sees no key here: O = 0, L = -inf (a range's O is not read where its L is -inf)
  auto empty_row = [&](int grow) {
    if (!shared) {
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<T*>(Out) + row_at(grow) * D);
      for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
    *lse_at(grow) = -INFINITY;
  };
  if (n_stream <= 0) {                          // past the sequence's queries, or before its keys
    for (int r = row0 + threadIdx.x; r < min(row0 + NT * BM, Nr); r += THREADS) empty_row(r);
    return;
  }

  auto bar = [&](int i) -> uint32_t { return sb + C::BAR_OFF + 8 * i; };
  const int B_QF = 0;
  auto B_KF = [&](int s) { return 1 + s; };
  auto B_KE = [&](int s) { return 1 + C::STAGES + s; };
  auto B_VF = [&](int s) { return 1 + 2 * C::STAGES + s; };
  auto B_VE = [&](int s) { return 1 + 3 * C::STAGES + s; };
  auto B_SF = [&](int t) { return 1 + 4 * C::STAGES + t; };
  auto B_PF = [&](int t) { return 3 + 4 * C::STAGES + t; };
  auto B_OF = [&](int t) { return 5 + 4 * C::STAGES + t; };
  const int B_DONE = 7 + 4 * C::STAGES;

  PagedTile first_tile;                         // its look-up passes under the set-up
  if (warp == 0) paged_fetch(px, b, kr, j0 * BN, lane, first_tile);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NBARS; ++i) mbar_init(bar(i), 1);
    for (int t = 0; t < NT; ++t) mbar_init(bar(B_PF(t)), 128);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + C::SLOT_OFF, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sg + C::SLOT_OFF);

  if (warp == 0) {
    regs_dec<kRegsLow>();                          // warpgroup 0 (TMA, MMA issue): few registers
    // ------------------------------------------------------------ producer
    {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(B_QF), NT * C::TILE_BYTES);
        for (int t = 0; t < NT; ++t)
          for (int c = 0; c < C::NCHUNK; ++c)
            tma_load_3d(sb + C::Q_OFF + t * C::TILE_BYTES + c * C::CHUNK_BYTES, &tmQ, bar(B_QF),
                        c * C::ATOM, hq, sr.base + ((row0 + t * BM) >> pack));
      }
      bool ok = true;
      PagedTile next = first_tile;
      int j = 0;
      for (; j < n_stream; ++j) {
        const int s = j % C::STAGES;
        const uint32_t ph = (j / C::STAGES) & 1;
        const PagedTile cur = next;
        if (j + 1 < n_stream) paged_fetch(px, b, kr, (j0 + j + 1) * BN, lane, next);
        if (!(ok = mbar_wait_warp(bar(B_KE(s)), ph ^ 1, ctl))) break;
        // the slot's last readers were the softmax threads of tile j - 8: they are done,
        // since S(j - 2), whose K tile has just been released, waited for their P
        paged_mask(px, lane, cur, sb + C::MASK_OFF + (j % kMaskSlots) * 16);
        if (lane == 0) mbar_arrive_expect_tx(bar(B_KF(s)), C::TILE_BYTES);
        __syncwarp();
        paged_load<D>(px, &tmK, sb + C::K_OFF + s * C::TILE_BYTES, bar(B_KF(s)), hk, lane, cur);
        if (!(ok = mbar_wait_warp(bar(B_VE(s)), ph ^ 1, ctl))) { ++j; break; }
        if (lane == 0) mbar_arrive_expect_tx(bar(B_VF(s)), C::TILE_BYTES);
        __syncwarp();
        paged_load<D>(px, &tmV, sb + C::V_OFF + s * C::TILE_BYTES, bar(B_VF(s)), hk, lane, cur);
      }
      if (!ok) {
        // drain: wait (bounded) for the copies in flight, so that none lands in shared memory
        // after the CTA has gone
        mbar_wait_warp(bar(B_QF), 0, ctl);
        for (int jj = max(0, j - C::STAGES); jj < j; ++jj) {
          const int s = jj % C::STAGES;
          const uint32_t ph = (jj / C::STAGES) & 1;
          mbar_wait_warp(bar(B_KF(s)), ph, ctl);
          mbar_wait_warp(bar(B_VF(s)), ph, ctl);
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    regs_dec<kRegsLow>();
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_stream > 0) {
      constexpr uint32_t idS = umma_idesc_f16(BM, BN, BF16, false, false);
      constexpr uint32_t idO = umma_idesc_f16(BM, D, BF16, false, true);
      // descriptor low words of Q tile 0 and of stage 0 of the K and V rings (K-major
      // with LBO 16; V MN-major with LBO = one swizzle-width chunk); tiles and stages
      // are TILE_BYTES apart
      constexpr uint32_t HI = sdesc_hi(8 * C::SW, C::SWZ), STAGE_W = C::TILE_BYTES >> 4;
      const uint32_t q_lo = sdesc_lo(sb + C::Q_OFF, 16), k_lo = sdesc_lo(sb + C::K_OFF, 16);
      const uint32_t v_lo = sdesc_lo(sb + C::V_OFF, C::CHUNK_BYTES);
      auto issue_S = [&](int t, int s) {
        const uint32_t qa = q_lo + t * STAGE_W, ka = k_lo + s * STAGE_W;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = kmajor_koff<D>(kk) >> 4;
          umma_ss_w(tmem + C::S_COL + t * BN, qa + o, ka + o, HI, idS, kk > 0);
        }
      };
      auto issue_PV = [&](int t, int s, bool acc) {
        const uint32_t va = v_lo + s * STAGE_W, acc0 = acc ? 1u : 0u;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk) {
          umma_ts_w(tmem + C::O_COL + t * D, tmem + C::S_COL + t * BN + kk * 8,
                    va + ((kk * 16 * C::SW) >> 4), HI, idO, kk > 0 ? 1u : acc0);
        }
      };
      bool ok = mbar_wait(bar(B_QF), 0, ctl) && mbar_wait(bar(B_KF(0)), 0, ctl);
      if (ok) {
        tc_fence_after();
        for (int t = 0; t < NT; ++t)
          if (lo_t[t] == j0 && n_t[t] > j0) {
            issue_S(t, 0);
            umma_commit(bar(B_SF(t)));
          }
        umma_commit(bar(B_KE(0)));
      }
      // stream position jj holds KV tile j = j0 + jj; Q tile t takes part while
      // lo_t[t] <= j < n_t[t], its own iteration index being j - lo_t[t]
      for (int jj = 0; ok && jj < n_stream; ++jj) {
        const int j = j0 + jj;
        const int s = jj % C::STAGES;
        const int s1 = (jj + 1) % C::STAGES;
        const uint32_t ph = (jj / C::STAGES) & 1, ph1 = ((jj + 1) / C::STAGES) & 1;
        if (!(ok = mbar_wait(bar(B_VF(s)), ph, ctl))) break;
        bool k_next = false;
        for (int t = 0; t < NT && ok; ++t) {
          const bool in_t = j >= lo_t[t] && j < n_t[t];
          if (in_t) {
            if (!(ok = mbar_wait(bar(B_PF(t)), (j - lo_t[t]) & 1, ctl))) break;
            tc_fence_after();
            issue_PV(t, s, j > lo_t[t]);
          }
          if (j + 1 >= lo_t[t] && j + 1 < n_t[t]) {
            if (!k_next) {
              if (!(ok = mbar_wait(bar(B_KF(s1)), ph1, ctl))) break;
              tc_fence_after();
              k_next = true;
            }
            issue_S(t, s1);
            umma_commit(bar(B_SF(t)));
          } else if (in_t) {
            umma_commit(bar(B_OF(t)));
          }
        }
        if (!ok) break;
        umma_commit(bar(B_VE(s)));
        if (k_next) umma_commit(bar(B_KE(s1)));
      }
      // every MMA this thread issued has completed before TMEM is released
      umma_commit(bar(B_DONE));
      mbar_wait(bar(B_DONE), 0, ctl);
    }
    __syncwarp();
  } else if (warp >= 4) {
    regs_inc<kRegsHigh>();                         // the compute warpgroups take what it gives back
    // ------------------------------------------------------------ softmax
    const int t = (warp - 4) >> 2;
    const int rit = (warp & 3) * 32 + lane;              // row within the tile (= TMEM lane)
    const int grow = row0 + t * BM + rit;                // query row
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::S_COL + t * BN;
    const uint32_t tO = tmem + lane_off + C::O_COL + t * D;
    const int nt = n_t[t] - lo_t[t];             // this tile's KV tiles, from lo_t[t]
    const int tile_row0 = row0 + t * BM;
    const RowKeys rk = row_keys(kr, tile_row0, grow, pack, px.window);
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < nt; ++j) {
      if (!(ok = mbar_wait_warp(bar(B_SF(t)), j & 1, ctl))) break;
      tc_fence_after();
      uint32_t mask[4], sr[BN];
      load_mask(sb + C::MASK_OFF + ((lo_t[t] + j - j0) % kMaskSlots) * 16, mask);
      tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
      tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
      tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
      tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
      tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
      tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
      tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
      const int kbase = (lo_t[t] + j) * BN;
      paged_masks<false>(rk, kbase, mask, sr);
      if (kbase + BN > Nk) {                     // the last tile's V rows past the keys
        const int jj = lo_t[t] + j - j0;         // stream position
        if (!(ok = mbar_wait_warp(bar(B_VF(jj % C::STAGES)), (jj / C::STAGES) & 1, ctl))) break;
        if (kbase + rit >= Nk) clear_row<D>(sb + C::V_OFF + (jj % C::STAGES) * C::TILE_BYTES, rit);
        fence_proxy_async_smem();                // before this thread's arrival on p_full
      }
      // row maximum: four independent chains of 3-input max
      const float mx = row_max128(sr);
      const float m_tile = mx * c_log2;
      const bool grow_m = m_tile > m_run + RESCALE_LOG2;
      const float m_use = grow_m ? m_tile : m_run;
      const float alpha = grow_m ? ex2(m_run - m_use) : 1.f;
      const float m_sub = (m_use == -INFINITY) ? 0.f : m_use;
      const float2 c2 = make_float2(c_log2, c_log2), nm2 = make_float2(P_LOG2<BF16> - m_sub, P_LOG2<BF16> - m_sub);
      float2 rs2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int c = 32 * h + 2 * i;
          const float2 t = fma2(make_float2(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), c2, nm2);
          const float2 pp = make_float2(ex2(t.x), ex2(t.y));
          rs2[i & 1] = add2(rs2[i & 1], pp);
          pk[i] = pack2<BF16>(pp.x, pp.y);
        }
        tmem_st16(tS + 16 * h, pk);
      }
      const float rs = (rs2[0].x + rs2[0].y) + (rs2[1].x + rs2[1].y);
      l_run = l_run * alpha + rs;
      if (j > 0 && __any_sync(0xffffffffu, grow_m)) {
        // O holds sum over tiles < j; PV(j-1) has completed because S(j) was
        // issued after it and its commit was observed above.
#pragma unroll
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * cc, o);
          tmem_ld_wait_regs(o);
          const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 v = mul2(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), a2);
            o[2 * i] = __float_as_uint(v.x);
            o[2 * i + 1] = __float_as_uint(v.y);
          }
          tmem_st32(tO + 32 * cc, o);
        }
      }
      m_run = m_use;
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(bar(B_PF(t)));
    }
    if (ok && nt > 0 && mbar_wait_warp(bar(B_OF(t)), 0, ctl)) {
      tc_fence_after();
      const bool none = l_run == 0.f;            // a row whose keys are all masked: acc = 0
      const float inv_l = none ? 0.f : 1.f / l_run;
      const bool valid = grow < Nr;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * cc, o);
        tmem_ld_wait_regs(o);
        if (shared) {
          if (valid) {
            float4* dst = reinterpret_cast<float4*>(px.part + part_at(grow) * D + 32 * cc);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(
                  __uint_as_float(o[4 * i]) * inv_l, __uint_as_float(o[4 * i + 1]) * inv_l,
                  __uint_as_float(o[4 * i + 2]) * inv_l, __uint_as_float(o[4 * i + 3]) * inv_l);
          }
          continue;
        }
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = pack2<BF16>(__uint_as_float(o[2 * i]) * inv_l,
                             __uint_as_float(o[2 * i + 1]) * inv_l);
        if (valid) {
          uint4* dst =
              reinterpret_cast<uint4*>(reinterpret_cast<T*>(Out) + row_at(grow) * D + 32 * cc);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
      }
      if (valid)
        *lse_at(grow) = none ? -INFINITY : (m_run - P_LOG2<BF16> + log2f(l_run)) * 0.69314718055994531f;
    } else if (nt <= 0 && grow < Nr) {
      empty_row(grow);
    }
  } else {
    regs_dec<kRegsLow>();                          // warps 2 and 3: idle
  }
  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

PagedArgs paged_args(const FwdArgs& a) {
  PagedArgs px;
  px.pg = a.pg;
  px.box_log2 = a.box_log2;
  px.causal = a.causal;
  px.window = a.window;
  px.pack = a.pack;
  px.n_split = a.n_split;
  px.rows = static_cast<size_t>(a.B) * a.N * a.H;
  px.part = a.part;
  px.part_l = a.part_l;
  return px;
}

template <int D, bool BF16>
cudaError_t launch_fwd_paged2_t(const FwdArgs& a, cudaStream_t st) {
  using C = Cfg<D>;
  constexpr int smem = C::SMEM_BYTES;
  auto kern = fwd_paged_kernel<D, BF16>;
  cudaError_t e = check_split_regs(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return e;
  e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int n_qblk =
      static_cast<int>(((static_cast<long long>(a.N) << a.pack) + NT * BM - 1) / (NT * BM));
  const long long grid = static_cast<long long>(n_qblk) * a.BH;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  trace_begin(TR_FWD, st);
  e = launch_dependent(kern, static_cast<unsigned>(grid), THREADS, smem, st, a.tmQ, a.tmK, a.tmV,
                       a.O, a.L, a.N, n_qblk, a.group, a.cu_seqlens, a.H, a.total, a.c_log2, a.ctl,
                       paged_args(a));
  trace_end(TR_FWD, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ============================================================== head dim <= 64
// One 128-row query tile at a time per CTA, two CTAs per SM, each persistent: it takes further
// tiles from CTAs that have not been launched yet (cluster launch control).
//   warp 0      TMA producer and scheduler: publishes each tile, with what its look-ups gave
//               (lengths, ranges), in a two-slot ring, loads its Q tile (double-buffered) and
//               streams K_j / V_j into a ring that runs on across tiles, then asks for the next
//               tile.
//   warp 1      TMEM allocator; lane 0 issues every tcgen05.mma and commit.
//   warps 2-5   softmax, one thread per query row (TMEM lane quadrant = warp % 4),
//               and the epilogue of each tile.
// TMEM (256 columns): S (128 fp32) | P (64: 128 keys as 16-bit pairs) | O (d fp32).
// P has columns of its own, so S(g+1) is issued as soon as the softmax threads hold
// S(g), and runs under their exponentials; P.V(g) then runs under softmax(g+1), which
// waits for it only before storing P(g+1) (and before an O rescale).  The step index
// g runs on across tiles, so the MMA issue order is S(0), S(1), PV(0), S(2), PV(1), ...
// whatever tile each step belongs to.  The first P.V of a tile overwrites O; the
// softmax threads arrive on p_full only after their epilogue has read the previous
// tile's O out of TMEM, so that order is kept without a barrier of its own.
namespace one {
constexpr int THREADS = 192;
template <int D>
struct Cfg1 {
  using C = Cfg<D>;                                         // swizzle geometry of a tile
  static constexpr int STAGES = D == 64 ? 2 : 4;
  static constexpr int TILE_BYTES = C::TILE_BYTES;
  static constexpr int Q_OFF = 0;                           // two Q buffers
  static constexpr int K_OFF = 2 * TILE_BYTES;
  static constexpr int V_OFF = K_OFF + STAGES * TILE_BYTES;
  static constexpr int O_OFF = V_OFF + STAGES * TILE_BYTES;   // O rows staged for the store
  static constexpr int BAR_OFF = O_OFF + TILE_BYTES;
  // q_full[2], q_empty[2], k_full[S], k_empty[S], v_full[S], v_empty[S], s_full, s_free,
  // p_full, pv_done, o_full, done, tile_full[2], tile_empty[2], clc
  static constexpr int NBARS = 4 + 4 * STAGES + 6 + 5;
  static constexpr int CLC_OFF = (BAR_OFF + NBARS * 8 + 15) / 16 * 16;   // 16-byte response
  static constexpr int SLOT_OFF = CLC_OFF + 16;             // TMEM base, tile slots[2]
  static constexpr int MASK_OFF = SLOT_OFF + 16;            // key masks
  static constexpr int INFO_OFF = MASK_OFF + kMaskSlots * 16;   // two Tile1
  static constexpr int SMEM_BYTES = INFO_OFF + 2 * 64;
  static constexpr int TMEM_COLS = 256;
  static constexpr uint32_t S_COL = 0, P_COL = 128, O_COL = 192;
  // two CTAs per SM, each with the 1 KiB the system reserves per CTA
  static_assert(2 * (SMEM_BYTES + 1024) <= 233472, "two CTAs per SM must fit");
  static_assert(O_COL + D <= TMEM_COLS, "TMEM layout");
};

// One query tile of the grid: its first head, K/V head and first row, and its KV tiles
// [lo, lo + nt).
struct Tile1 {
  int b, hq, hk, row0, lo, nt;
  int base, nr;                                  // first token and query rows of the sequence
  KeyRows kr;
  int split;                                     // its KV range, if it has one of several
  bool shared;
};
static_assert(sizeof(Tile1) <= 64, "a slot of the tile ring");
__device__ __forceinline__ Tile1 tile1(int id, int n_qt, int N, int group, const int* cu_seqlens,
                                       int H, int total, const PagedArgs& px) {
  Tile1 t;
  const BlockPos bp = block_pos(n_qt, id);       // bp.bh: sequence, block of heads, KV range
  const int blocks = H >> px.pack, bh = bp.bh / px.n_split;
  t.split = bp.bh % px.n_split;
  t.b = bh / blocks;
  t.hq = (bh % blocks) << px.pack;
  t.hk = t.hq / group;
  t.row0 = (n_qt - 1 - bp.rank) * BM;            // the last query tiles have the most work
  SeqRows sr;
  rows_of(px, cu_seqlens, t.b, N, total, sr, t.kr);
  t.base = sr.base;
  t.nr = sr.n << px.pack;
  const SplitRange sp = split_range<1>(t.kr, t.row0, t.nr, px.window, px.pack, px.n_split);
  t.shared = sp.used > 1;
  t.lo = sp.lo + t.split * sp.per;
  t.nt = max(min(sp.per, sp.hi - t.lo), 0);
  if (t.split >= sp.used) t.nr = t.nt = 0;       // nothing to do or to write
  return t;
}
}  // namespace one

template <int D, bool BF16>
__global__ void __launch_bounds__(one::THREADS, 2)
    fwd1_paged_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, void* __restrict__ Out,
                      float* __restrict__ Lout, int N, int n_qt, int group, const int* cu_seqlens,
                      int H, int total, float c_log2, KernelCtl ctl, const PagedArgs px) {
  using C = Cfg<D>;
  using C1 = one::Cfg1<D>;
  constexpr int STAGES = C1::STAGES;
  extern __shared__ __align__(1024) uint8_t sg[];
  const uint32_t sb = smem_u32(sg);
  grid_dep_launch();                            // the next kernel may start setting up
  if (sb & 1023u) {                             // see FA_DEV_SMEM_ALIGN
    grid_dep_wait();
    if (threadIdx.x == 0) atomicOr(ctl.status, FA_DEV_SMEM_ALIGN);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pack = px.pack;

  auto bar = [&](int i) -> uint32_t { return sb + C1::BAR_OFF + 8 * i; };
  auto B_QF = [&](int b) { return b; };
  auto B_QE = [&](int b) { return 2 + b; };
  auto B_KF = [&](int st) { return 4 + st; };
  auto B_KE = [&](int st) { return 4 + STAGES + st; };
  auto B_VF = [&](int st) { return 4 + 2 * STAGES + st; };
  auto B_VE = [&](int st) { return 4 + 3 * STAGES + st; };
  const int B_SF = 4 + 4 * STAGES, B_SFREE = B_SF + 1, B_PF = B_SF + 2, B_PVD = B_SF + 3,
            B_OF = B_SF + 4, B_DONE = B_SF + 5;
  auto B_TF = [&](int b) { return B_SF + 6 + b; };
  auto B_TE = [&](int b) { return B_SF + 8 + b; };
  const int B_CLC = B_SF + 10;
  volatile int* slot = reinterpret_cast<volatile int*>(sg + C1::SLOT_OFF + 4);
  const uint32_t clc_resp = sb + C1::CLC_OFF;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C1::NBARS; ++i) mbar_init(bar(i), 1);
    mbar_init(bar(B_SFREE), 128);
    mbar_init(bar(B_PF), 128);
    mbar_init(bar(B_TE(0)), 5);                 // the MMA thread and one lane per softmax warp
    mbar_init(bar(B_TE(1)), 5);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + C1::SLOT_OFF, C1::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sg + C1::SLOT_OFF);
  grid_dep_wait();                              // inputs written, outputs free to overwrite

  auto info = [&](int b) -> one::Tile1* {
    return reinterpret_cast<one::Tile1*>(sg + C1::INFO_OFF + 64 * b);
  };
  // Consumers read tile k from slot k & 1; the last tile published is -1.
  auto next_tile = [&](int k, bool& ok) -> int {
    if (!(ok = mbar_wait(bar(B_TF(k & 1)), (k >> 1) & 1, ctl))) return -1;
    return slot[k & 1];
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer, scheduler
    {
      const bool lead = lane == 0;               // does what is done once
      auto wait = [&](uint32_t b, uint32_t parity) -> bool {
        return mbar_wait_warp(b, parity, ctl);
      };
      bool ok = true;
      int tile = static_cast<int>(blockIdx.x);
      int g = 0, kq = 0, nk = 0, nv = 0;         // steps, Q tiles, K and V tiles loaded
      bool pending = false;                       // a request for the next tile is out
      int n_req = 0;                               // requests made
      for (int k = 0; ok; ++k) {
        if (!(ok = wait(bar(B_TE(k & 1)), ((k >> 1) & 1) ^ 1))) break;
        one::Tile1 t;
        if (tile >= 0) {
          t = one::tile1(tile, n_qt, N, group, cu_seqlens, H, total, px);
          if (lead) *info(k & 1) = t;
        }
        if (lead) {
          slot[k & 1] = tile;
          mbar_arrive(bar(B_TF(k & 1)));        // release: the slot write is seen with the phase
        }
        if (tile < 0) break;
        // ask for the next tile together with this tile's last loads: early enough that
        // the answer is there when they complete, late enough that a CTA takes a tile
        // only when it is nearly free (asking at a tile's start handed the last tiles to
        // CTAs that still had most of a long tile ahead, and took tiles from CTAs that had
        // not started yet when all would have fit at once)
        auto request = [&]() {
          if (lead) {
            mbar_arrive_expect_tx(bar(B_CLC), 16);
            clc_try_cancel(clc_resp, bar(B_CLC));
          }
          pending = true;
          ++n_req;
        };
        if (t.nt <= 0) request();
        if (t.nt > 0) {
          const int qb = kq & 1;
          if (!(ok = wait(bar(B_QE(qb)), ((kq >> 1) & 1) ^ 1))) break;
          if (lead) {
            mbar_arrive_expect_tx(bar(B_QF(qb)), C1::TILE_BYTES);
            for (int c = 0; c < C::NCHUNK; ++c)
              tma_load_3d(sb + C1::Q_OFF + qb * C1::TILE_BYTES + c * C::CHUNK_BYTES, &tmQ,
                          bar(B_QF(qb)), c * C::ATOM, t.hq, t.base + (t.row0 >> pack));
          }
          ++kq;
          PagedTile next;
          paged_fetch(px, t.b, t.kr, t.lo * BN, lane, next);
          for (int j = 0; j < t.nt; ++j, ++g) {
            const int st = g % STAGES;
            const uint32_t ph = (g / STAGES) & 1;
            const int krow = (t.lo + j) * BN;
            const PagedTile cur = next;
            if (j + 1 < t.nt) paged_fetch(px, t.b, t.kr, krow + BN, lane, next);
            if (!(ok = wait(bar(B_KE(st)), ph ^ 1))) break;
            // the mask slot's last readers were the softmax threads of step g - 8: they are
            // done, since S(g - STAGES), whose K tile has just been released, came two steps
            // or more after theirs
            paged_mask(px, lane, cur, sb + C1::MASK_OFF + (g % kMaskSlots) * 16);
            if (lead) mbar_arrive_expect_tx(bar(B_KF(st)), C1::TILE_BYTES);
            __syncwarp();
            paged_load<D>(px, &tmK, sb + C1::K_OFF + st * C1::TILE_BYTES, bar(B_KF(st)), t.hk, lane,
                          cur);
            ++nk;
            if (!(ok = wait(bar(B_VE(st)), ph ^ 1))) break;
            if (lead) mbar_arrive_expect_tx(bar(B_VF(st)), C1::TILE_BYTES);
            __syncwarp();
            paged_load<D>(px, &tmV, sb + C1::V_OFF + st * C1::TILE_BYTES, bar(B_VF(st)), t.hk, lane,
                          cur);
            ++nv;
            if (j + 1 == t.nt) request();
          }
          if (!ok) break;
        }
        // the next tile: a CTA that had not started, if any was left
        if (!(ok = wait(bar(B_CLC), k & 1))) break;
        pending = false;
        tile = clc_result(clc_resp);
      }
      if (!ok) {
        if (pending) wait(bar(B_CLC), (n_req - 1) & 1);   // the response lands in smem
        // drain: wait (bounded) for the copies this thread may still have in flight, so
        // no bulk copy lands in shared memory after the CTA has gone
        for (int i = max(0, kq - 2); i < kq; ++i) wait(bar(B_QF(i & 1)), (i >> 1) & 1);
        for (int i = max(0, nk - STAGES); i < nk; ++i)
          wait(bar(B_KF(i % STAGES)), (i / STAGES) & 1);
        for (int i = max(0, nv - STAGES); i < nv; ++i)
          wait(bar(B_VF(i % STAGES)), (i / STAGES) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = umma_idesc_f16(BM, BN, BF16, false, false);
      constexpr uint32_t idO = umma_idesc_f16(BM, D, BF16, false, true);
      constexpr uint32_t HI = sdesc_hi(8 * C::SW, C::SWZ), STAGE_W = C1::TILE_BYTES >> 4;
      const uint32_t q_lo = sdesc_lo(sb + C1::Q_OFF, 16), k_lo = sdesc_lo(sb + C1::K_OFF, 16);
      const uint32_t v_lo = sdesc_lo(sb + C1::V_OFF, C::CHUNK_BYTES);
      // the pending P.V: step, stage, whether it is its tile's first / last
      int pv_g = -1, pv_st = 0;
      bool pv_first = false, pv_last = false;
      bool ok = true;
      auto issue_pv = [&]() -> bool {
        if (!mbar_wait(bar(B_VF(pv_st)), (pv_g / STAGES) & 1, ctl)) return false;
        if (!mbar_wait(bar(B_PF), pv_g & 1, ctl)) return false;
        tc_fence_after();
        const uint32_t va = v_lo + pv_st * STAGE_W;
#pragma unroll
        for (int kk = 0; kk < BN / 16; ++kk)
          umma_ts_w(tmem + C1::O_COL, tmem + C1::P_COL + kk * 8,
                    va + ((kk * 16 * C::SW) >> 4), HI, idO, (kk > 0 || !pv_first) ? 1u : 0u);
        umma_commit(bar(B_VE(pv_st)));
        umma_commit(bar(B_PVD));
        if (pv_last) umma_commit(bar(B_OF));
        return true;
      };
      int g = 0, kq = 0;
      for (int k = 0; ok; ++k) {
        const int tile = next_tile(k, ok);
        if (!ok) break;
        const int nt = info(k & 1)->nt;
        mbar_arrive(bar(B_TE(k & 1)));
        if (tile < 0) break;
        if (nt == 0) continue;
        const int qb = kq & 1;
        if (!(ok = mbar_wait(bar(B_QF(qb)), (kq >> 1) & 1, ctl))) break;
        const uint32_t qa = q_lo + qb * STAGE_W;
        for (int j = 0; j < nt; ++j, ++g) {
          // S(g) once K_g is in and the softmax threads hold S(g - 1)
          const int st = g % STAGES;
          if (!(ok = mbar_wait(bar(B_KF(st)), (g / STAGES) & 1, ctl))) break;
          if (g > 0 && !(ok = mbar_wait(bar(B_SFREE), (g - 1) & 1, ctl))) break;
          tc_fence_after();
          const uint32_t ka = k_lo + st * STAGE_W;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = kmajor_koff<D>(kk) >> 4;
            umma_ss_w(tmem + C1::S_COL, qa + o, ka + o, HI, idS, kk > 0);
          }
          umma_commit(bar(B_SF));
          umma_commit(bar(B_KE(st)));
          if (j + 1 == nt) umma_commit(bar(B_QE(qb)));   // Q free once its last S is done
          // then P(g - 1).V
          if (pv_g >= 0 && !(ok = issue_pv())) break;
          pv_g = g;
          pv_st = st;
          pv_first = j == 0;
          pv_last = j + 1 == nt;
        }
        // the tile's last P.V goes out before this thread waits for the next tile, so
        // the epilogue never waits on the next tile's loads
        if (ok && pv_g >= 0) ok = issue_pv();
        pv_g = -1;
        ++kq;
      }
      // every MMA this thread issued has completed before TMEM is released
      umma_commit(bar(B_DONE));
      mbar_wait(bar(B_DONE), 0, ctl);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax, epilogue
    const int rit = (warp & 3) * 32 + lane;      // row within the tile (= TMEM lane)
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C1::S_COL;
    const uint32_t tP = tmem + lane_off + C1::P_COL;
    const uint32_t tO = tmem + lane_off + C1::O_COL;
    bool ok = true;
    int g = 0, kq = 0;
    for (int k = 0; ok; ++k) {
      int tile = next_tile(k, ok);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // the tile's slot is read again by the epilogue and given back after it
      auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_TE(k & 1)));
      };
      if (tile < 0) release();
      if (tile < 0) break;
      const one::Tile1* ti = info(k & 1);
      const int nt = ti->nt, lo = ti->lo, row0 = ti->row0, Nk = ti->kr.n;
      const RowKeys rk = row_keys(ti->kr, row0, row0 + rit, pack, px.window);
      const int grow = row0 + rit;               // query row
      // where a row lies in O, in the workspace, and in L or the workspace's L
      auto row_at = [&](int r) -> size_t {
        return static_cast<size_t>(ti->base + (r >> pack)) * H + ti->hq + (r & ((1 << pack) - 1));
      };
      auto part_at = [&](int r) -> size_t {
        return ti->split * px.rows + (static_cast<size_t>(ti->b) * N + (r >> pack)) * H + ti->hq +
               (r & ((1 << pack) - 1));
      };
      auto lse_at = [&](int r) -> float* {
        if (ti->shared) return px.part_l + part_at(r);
        return Lout + static_cast<size_t>(ti->hq + (r & ((1 << pack) - 1))) * total + ti->base +
               (r >> pack);
      };
      if (nt == 0) {
        if (grow < ti->nr) {                     // a row before the first key: O = 0, L = -inf
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(Out) + row_at(grow) * D);
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
          *lse_at(grow) = -INFINITY;
        }
        release();
        continue;
      }
      float m_run = -INFINITY, l_run = 0.f;
      for (int j = 0; j < nt; ++j, ++g) {
        if (!(ok = mbar_wait_warp(bar(B_SF), g & 1, ctl))) break;
        tc_fence_after();
        uint32_t sr_[BN];
        tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr_[0]));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr_[32]));
        tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr_[64]));
        tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr_[96]));
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr_[0]));
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr_[32]));
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr_[64]));
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr_[96]));
        tc_fence_before();
        mbar_arrive(bar(B_SFREE));               // S may now receive the next step
        const int kbase = (lo + j) * BN;
        uint32_t mask[4];
        load_mask(sb + C1::MASK_OFF + (g % kMaskSlots) * 16, mask);
        paged_masks<true>(rk, kbase, mask, sr_);
        if (kbase + BN > Nk) {                   // the last tile's V rows past the keys
          const int st = g % STAGES;
          if (!(ok = mbar_wait_warp(bar(B_VF(st)), (g / STAGES) & 1, ctl))) break;
          if (kbase + rit >= Nk) clear_row<D>(sb + C1::V_OFF + st * C1::TILE_BYTES, rit);
          fence_proxy_async_smem();              // before this thread's arrival on p_full
        }
        const float mx = row_max128(sr_);
        const float m_tile = mx * c_log2;
        const bool grow_m = m_tile > m_run + RESCALE_LOG2;
        const float m_use = grow_m ? m_tile : m_run;
        const float alpha = grow_m ? ex2(m_run - m_use) : 1.f;
        const float m_sub = (m_use == -INFINITY) ? 0.f : m_use;
        const float2 c2 = make_float2(c_log2, c_log2), nm2 = make_float2(P_LOG2<BF16> - m_sub, P_LOG2<BF16> - m_sub);
        float2 rs2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        // p for keys [32h, 32h + 32) as 16 packed pairs
        auto exp_pairs = [&](int h, uint32_t (&pk)[16]) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = 32 * h + 2 * i;
            const float2 tt = fma2(make_float2(__uint_as_float(sr_[c]), __uint_as_float(sr_[c + 1])),
                                   c2, nm2);
            const float2 pp = make_float2(ex2(tt.x), ex2(tt.y));
            rs2[i & 1] = add2(rs2[i & 1], pp);
            pk[i] = pack2<BF16>(pp.x, pp.y);
          }
        };
        // the first half of P before waiting for P(g-1).V; the second half is stored as
        // it is formed, so no more than half of P is held in registers
        uint32_t pa[16], pb[16];
        exp_pairs(0, pa);
        exp_pairs(1, pb);
        // P(g-1).V has completed: P's columns are free and O holds the sum over the
        // tile's earlier steps (at a tile's first step, the epilogue before it waited
        // for the previous tile's last P.V)
        if (j > 0) {
          if (!(ok = mbar_wait_warp(bar(B_PVD), (g - 1) & 1, ctl))) break;
          tc_fence_after();
        }
        tmem_st16(tP, pa);
        tmem_st16(tP + 16, pb);
        exp_pairs(2, pa);
        tmem_st16(tP + 32, pa);
        exp_pairs(3, pb);
        tmem_st16(tP + 48, pb);
        if (j > 0 && __any_sync(0xffffffffu, grow_m)) {
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * cc, o);
            tmem_ld_wait_regs(o);
            const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 v = mul2(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), a2);
              o[2 * i] = __float_as_uint(v.x);
              o[2 * i + 1] = __float_as_uint(v.y);
            }
            tmem_st32(tO + 32 * cc, o);
          }
        }
        m_run = m_use;
        const float rs = (rs2[0].x + rs2[0].y) + (rs2[1].x + rs2[1].y);
        l_run = l_run * alpha + rs;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(B_PF));
      }
      if (!ok) break;
      // epilogue: O = acc / l and L once the tile's last P.V has completed
      if (!(ok = mbar_wait_warp(bar(B_OF), kq & 1, ctl))) break;
      ++kq;
      tc_fence_after();
      const int Nr = ti->nr;
      const bool shared = ti->shared;
      const bool none = l_run == 0.f;            // a row whose keys are all masked: acc = 0
      const float inv_l = none ? 0.f : 1.f / l_run;
      const bool valid = grow < Nr;
      // Each thread writes its row of O (16-bit) to this warp's 32 staging rows in shared
      // memory, 16-byte chunk c of row r at chunk c ^ (r mod CPR), so the eight lanes of
      // a store phase hit distinct banks; the warp then writes rows to global memory
      // 512 contiguous bytes per instruction.
      constexpr int CPR = D / 8;                 // 16-byte chunks per row
      uint4* stage = reinterpret_cast<uint4*>(sg + C1::O_OFF) + (warp & 3) * 32 * CPR;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * cc, o);
        tmem_ld_wait_regs(o);
        if (shared) {
          if (valid) {
            float4* dst = reinterpret_cast<float4*>(px.part + part_at(grow) * D + 32 * cc);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[i] = make_float4(
                  __uint_as_float(o[4 * i]) * inv_l, __uint_as_float(o[4 * i + 1]) * inv_l,
                  __uint_as_float(o[4 * i + 2]) * inv_l, __uint_as_float(o[4 * i + 3]) * inv_l);
          }
          continue;
        }
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w[i] = pack2<BF16>(__uint_as_float(o[2 * i]) * inv_l,
                             __uint_as_float(o[2 * i + 1]) * inv_l);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          stage[lane * CPR + ((4 * cc + i) ^ (lane % CPR))] =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      }
      tc_fence_before();                         // O read before the next tile's p_full
      if (valid)
        *lse_at(grow) = none ? -INFINITY : (m_run - P_LOG2<BF16> + log2f(l_run)) * 0.69314718055994531f;
      if (shared) {                              // nothing staged
        release();
        continue;
      }
      __syncwarp();
      using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
      constexpr int RPI = 32 / CPR;              // rows per store instruction
#pragma unroll
      for (int i = 0; i < 32 / RPI; ++i) {
        const int r = i * RPI + lane / CPR, c = lane % CPR;   // row within the warp, chunk
        const int orow_g = row0 + (warp & 3) * 32 + r;
        if (orow_g < Nr) {
          T* dst = reinterpret_cast<T*>(Out) + row_at(orow_g) * D + 8 * c;
          *reinterpret_cast<uint4*>(dst) = stage[r * CPR + (c ^ (r % CPR))];
        }
      }
      release();                                 // staging rows free for the next tile, too
    }
  }
  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C1::TMEM_COLS);
  }
}

template <int D, bool BF16>
cudaError_t launch_fwd_paged1_t(const FwdArgs& a, cudaStream_t st) {
  using C1 = one::Cfg1<D>;
  constexpr int smem = C1::SMEM_BYTES;
  auto kern = fwd1_paged_kernel<D, BF16>;
  cudaError_t e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const int n_qt = static_cast<int>(((static_cast<long long>(a.N) << a.pack) + BM - 1) / BM);
  const long long grid = static_cast<long long>(n_qt) * a.BH;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  trace_begin(TR_FWD, st);
  e = launch_dependent(kern, static_cast<unsigned>(grid), one::THREADS, smem, st, a.tmQ,
                       a.tmK, a.tmV, a.O, a.L, a.N, n_qt, a.group, a.cu_seqlens, a.H, a.total,
                       a.c_log2, a.ctl, paged_args(a));
  trace_end(TR_FWD, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Joins the KV ranges of a query tile: one warp per (query, head) of a sequence, which is
// left alone where its tile was not cut.  TILES: query tiles of 128 rows that are cut together.
constexpr int MERGE_THREADS = 128;
template <int D, bool BF16, int TILES>
__global__ void __launch_bounds__(MERGE_THREADS)
    fwd_paged_merge_kernel(void* Out, float* Lout, const int* cu_seqlens, int N, int H, int total,
                           const PagedArgs px) {
  grid_dep_wait();                               // the ranges' results
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  SeqRows sr;
  KeyRows kr;
  rows_of(px, cu_seqlens, b, N, total, sr, kr);
  const long long i =
      static_cast<long long>(blockIdx.x) * (MERGE_THREADS / 32) + (threadIdx.x >> 5);
  if (i >= static_cast<long long>(sr.n) * H) return;
  const int q = static_cast<int>(i / H), h = static_cast<int>(i % H);
  // the row in its block of packed heads, and the first row of its tiles
  const int row = (q << px.pack) + (h & ((1 << px.pack) - 1));
  const SplitRange sp = split_range<TILES>(kr, row / (TILES * BM) * (TILES * BM), sr.n << px.pack,
                                           px.window, px.pack, px.n_split);
  if (sp.used <= 1) return;
  const size_t rows = px.rows, at = (static_cast<size_t>(b) * N + q) * H + h;   // in the workspace
  float l_max = -INFINITY;
  for (int s = lane; s < sp.used; s += 32) l_max = fmaxf(l_max, px.part_l[s * rows + at]);
#pragma unroll
  for (int w = 16; w >= 1; w /= 2) l_max = fmaxf(l_max, __shfl_xor_sync(0xffffffffu, l_max, w));
  // weights of 32 ranges at a time, one per lane; their rows in batches of 8 loads that do not
  // wait for one another (a range without keys has weight 0 and left nothing to read)
  constexpr int E = D / 32;
  float sum = 0.f, acc[E] = {};
  for (int s0 = 0; s0 < sp.used; s0 += 32) {
    const float ls = s0 + lane < sp.used ? px.part_l[(s0 + lane) * rows + at] : -INFINITY;
    const float wl = ls == -INFINITY ? 0.f : ex2((ls - l_max) * 1.4426950408889634f);
    sum += wl;
    for (int k0 = 0; k0 < min(32, sp.used - s0); k0 += 8) {
      float v[8][E], w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        w[k] = __shfl_sync(0xffffffffu, wl, k0 + k);
        const float* src = px.part + ((s0 + k0 + k) * rows + at) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; ++e) v[k][e] = w[k] > 0.f ? src[e] : 0.f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(v[k][e], w[k], acc[e]);
    }
  }
#pragma unroll
  for (int w = 16; w >= 1; w /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, w);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  T* dst = static_cast<T*>(Out) + (static_cast<size_t>(sr.base + q) * H + h) * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (BF16) dst[e] = __float2bfloat16_rn(acc[e] * inv);
    else dst[e] = __float2half_rn(acc[e] * inv);
  }
  if (lane == 0)
    Lout[static_cast<size_t>(h) * total + sr.base + q] =
        sum == 0.f ? -INFINITY : l_max + log2f(sum) * 0.69314718055994531f;
}

template <int D, bool BF16>
cudaError_t launch_fwd_paged_t(const FwdArgs& a, cudaStream_t st) {
  cudaError_t e;
  if constexpr (D == 128) e = launch_fwd_paged2_t<D, BF16>(a, st);
  else e = launch_fwd_paged1_t<D, BF16>(a, st);
  if (e != cudaSuccess || a.n_split == 1) return e;
  const long long warps = static_cast<long long>(a.N) * a.H;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps * 32 + MERGE_THREADS - 1) / MERGE_THREADS),
                     static_cast<unsigned>(a.B));
  cfg.blockDim = dim3(MERGE_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fwd_paged_merge_kernel<D, BF16, D == 128 ? NT : 1>, a.O, a.L,
                            a.cu_seqlens, a.N, a.H, a.total, paged_args(a));
}

template <bool BF16>
cudaError_t launch_fwd_paged_b(const FwdArgs& a, int d, cudaStream_t st) {
  if (d == 32) return launch_fwd_paged_t<32, BF16>(a, st);
  if (d == 64) return launch_fwd_paged_t<64, BF16>(a, st);
  if (d == 128) return launch_fwd_paged_t<128, BF16>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace

int fwd_paged_pack(int group) {
  int p = 0;
  while (p < 7 && group % (2 << p) == 0) ++p;
  return p;
}

// Ranges per query tile: none where the tiles fill half the GPU or more (152 SMs; two CTAs
// each at d <= 64), else as many as fill it once.
int fwd_paged_splits(int B, int H, int Hkv, int max_seqlen, int d) {
  const int pack = fwd_paged_pack(H / Hkv), rows = d == 128 ? NT * BM : BM;
  const long long tiles = static_cast<long long>(B) * (H >> pack) *
                          (((static_cast<long long>(max_seqlen) << pack) + rows - 1) / rows);
  const long long slots = d == 128 ? 152 : 304;
  return tiles * 2 > slots ? 1 : static_cast<int>(slots / tiles);
}

cudaError_t launch_fwd_paged(const FwdArgs& args, int d, bool bf16, bool causal, cudaStream_t st) {
  FwdArgs a = args;
  a.causal = causal;
  if (!causal || a.window == 0) a.window = kNoLimit;
  a.BH = a.B * (a.H >> a.pack) * a.n_split;
  return bf16 ? launch_fwd_paged_b<true>(a, d, st) : launch_fwd_paged_b<false>(a, d, st);
}

}  // namespace fa
