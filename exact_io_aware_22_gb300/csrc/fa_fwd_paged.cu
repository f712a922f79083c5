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
//   producer   a whole warp, or up to three (d = 128).  Each lane looks up the pages of its boxes
//              (the largest power of two of rows that divides the page size) one tile ahead and
//              loads them; a 128-row tile lies in shared memory as one box would.  Boxes of
//              absent pages read as zeros and their keys are masked; V rows past the last key,
//              which may hold anything, are cleared before the product that reads them (0 x NaN).
//   tiles      A query tile holds the rows of 2^pack heads that share a K/V head, heads fastest:
//              the tile of a few new tokens is better filled, K and V pass once for those
//              heads, and less of a tile lies beyond the diagonal (5 tokens of 4 sequences of
//              2000 keys, 32/8 heads, d = 128: 33.4 against 17.7 us with the keys split; 8
//              prompts of 1000: 110 against 99 us).
//   ranges     Where there are few query tiles, or uneven ones, the KV tiles of all are laid
//              end to end and every CTA takes an equal range of them, which may begin and end
//              inside a query tile.  The lengths lie on the device, so every CTA finds its range
//              by a scan over the tiles, and decides there whether cutting pays.  A tile cut by
//              range borders leaves in each of its CTAs a result normalised with its own L, and
//              fwd_paged_merge_kernel joins these in order, by their weights 2^(L_s - L).  5
//              tokens of 10 / 16 sequences of 16384-32768 keys: 163 / 252 us (6.2 and 6.4 TB/s);
//              a CTA for each tile: 355 / 356 us.
//
// Bound: at d = 128 the products and exponentials of a KV tile, 1.55 us where the products alone
// take 1.35 at the rate of a large matrix product, and the last, part-filled round of query tiles
// (2 x 2048 tokens on 8192 keys, 32/8 heads: 0.335 ms, 1422 TFLOP/s; 512 tiles on 152 SMs give a
// CTA up to 216 KV tiles where the mean is 189); at d <= 64 the latency of a KV tile's chain (S,
// maximum, exponentials, P, P.V) under two CTAs per SM; with few tokens that of start, split and
// join (the 5 tokens above: 18 us for 34 MB of keys), with few tokens on long caches the cache's
// bytes.
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
// P is rounded to 16 bits once, as the tensor cores take it and as in the dense forward: each
// weight is off by at most half a step (2^-8 of it in bf16, 2^-11 in f16), l sums them unrounded.
// Against 64 bits the result is off by 1.4 times the rounding of O alone (0.0023 of its size
// against 0.0017 in bf16).  Two terms, as decoding has them, would take half as many products
// again, and the tensor pipe is what long prompts wait for.
// P is formed with 2^7 times its weight where it is f16 (p <= 2^15), so that the small p of a
// long context, which add up, stay clear of f16's subnormals (weights below 2^-21 of the largest
// are off by up to 2^-32 of that); l carries the same factor.
template <bool BF16>
constexpr float P_LOG2 = BF16 ? 0.f : 7.f;
constexpr int kMaskSlots = 8;         // ring of 128-bit key masks, one per KV tile

template <int D, bool C8 = false>
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
  // C8: tiles K(0), V(0), K(1), ... go through a ring of codes and then one of f16 tiles from K_OFF
  static constexpr int CODES = 4, TILES16 = 3;
  static constexpr int CODE_OFF = K_OFF + TILES16 * TILE_BYTES, CODE_BYTES = 128 * D;
  static constexpr int BAR_OFF = C8 ? CODE_OFF + CODES * CODE_BYTES : V_OFF + STAGES * TILE_BYTES;
  // q_full, k_full[S], k_empty[S], v_full[S], v_empty[S], s_full[2], p_full[2], o_full[2], done,
  // q_empty, piece_full[2], piece_empty[2], and C8: code_full[4], code_empty[4], q_turned,
  // half_full, half_empty (and of the first 4S, tile_full[3], tile_empty[3])
  static constexpr int NBARS = 1 + 4 * STAGES + 7 + 5 + (C8 ? 2 * CODES + 3 : 0);
  static constexpr int SLOT_OFF = BAR_OFF + NBARS * 8;
  static constexpr int MASK_OFF = (SLOT_OFF + 16 + 15) / 16 * 16;
  static constexpr int INFO_OFF = MASK_OFF + kMaskSlots * 16;            // two Pieces
  static constexpr int HALF_OFF = INFO_OFF + 2 * 64;                     // C8: m and l of 128 rows
  static constexpr int SMEM_BYTES = HALF_OFF + (C8 ? 1024 : 0) + 1024;   // + alignment slack
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

// The query tile that range x shares with range x - 1: its sequence's first token, its first head,
// first row and rows (0: there is none), and the first and last range that have parts of it.
// Range 0 shares none; its header's `base` says whether the call is cut at all, and where it is
// not, no other header is written: at d <= 64 a CTA that has not started may be cancelled and its
// tile taken by another.  So every CTA that starts stores it, before anything that may fail.
struct RangeHeader {
  int base, hq, row0, rows, c0, c1;
};
struct PagedArgs {
  PagedView pg;
  int box_log2, causal, window;    // window: 0 for none
  int pack;                        // log2 of the heads in a query tile
  int B, n_qt;                     // sequences, query tiles of the longest
  int ranges;                      // CTAs that may share the KV tiles of all query tiles (0: none)
  RangeHeader* hdr;                // workspace, with ranges: [ranges], then
  float* part;                     // [2 * ranges][rows of a query tile][D] results of pieces
  float* part_l;                   // [2 * ranges][rows of a query tile] their L (natural log)
  float o_scale;                   // 1 (codes: v_scale)
};
constexpr int kNoLimit = 1 << 30;  // no table has room for more keys
// Keys of a sequence: query row i sees keys i + lo up to i + hi of its n.
struct KeyRows {
  int n, lo, hi;
};
// Query and key rows of sequence b; the three loads go out together.
__device__ __forceinline__ void rows_of(const PagedArgs& px, const int* cu, int b, int N,
                                        int total, SeqRows& sr, KeyRows& k) {
  const int c0 = cu[b], c1 = cu[b + 1], len = max(px.pg.seqlens[b], 0);
  const int a = min(max(c0, 0), total), e = min(max(c1, a), total);
  sr = {a, min(e - a, N), true};
  const long long cap = static_cast<long long>(px.pg.max_pages) * px.pg.page.div;
  k.n = static_cast<int>(min(static_cast<long long>(len), cap));
  // Row i is at position i + off, which goes by the length and the offsets as they are given: rows
  // past N and keys past the table are left out, the others stay where they are.  Rows are below
  // 2^29 (the call refuses more), so sums with the limits stay in 32 bits.
  const long long none = kNoLimit, off = static_cast<long long>(len) - c1 + a;
  const long long lo = px.window > 0 ? off - px.window + 1 : -none;
  k.lo = static_cast<int>(max(min(lo, none), -none));
  k.hi = px.causal ? static_cast<int>(min(off, none)) : kNoLimit;
}
// KV tiles [lo, hi) of the query tile at rows r .. r + BM - 1 of a sequence's nr; row i is
// a head of query i >> pack.
__device__ __forceinline__ void paged_tiles(const KeyRows& k, int r, int nr, int pack, int& lo,
                                            int& hi) {
  const int last = (min(r + BM - 1, nr - 1) >> pack) + k.hi;
  hi = r >= nr || last < 0 ? 0 : min((k.n + BN - 1) / BN, last / BN + 1);
  lo = min(max(0, (r >> pack) + k.lo) / BN, hi);
}
// KV tiles [lo, hi) of a query tile of TILES * BM rows from row r.
struct Span {
  int lo, hi;
};
template <int TILES>
__device__ __forceinline__ Span tile_span(const PagedArgs& px, const KeyRows& k, int r, int nr) {
  Span s;
  paged_tiles(k, r, nr, px.pack, s.lo, s.hi);
#pragma unroll
  for (int t = 1; t < TILES; ++t) {
    int lo, hi;
    paged_tiles(k, r + t * BM, nr, px.pack, lo, hi);
    if (hi > s.hi) s.hi = hi;                    // lo rises with the row
  }
  return s;
}
// Positions of a query tile of n KV tiles on the line that ranges are cut from: beginning and
// ending a piece takes about as long as kTileCost KV tiles (1, 2 and 4 differ by up to 2 %, but
// 4, of which a range has at least twice as much, leaves 4 x 5 tokens on 2000 keys at 25 us
// instead of 18).  KV tile i is at position kTileCost + i.
constexpr int kTileCost = 2;
// What cutting costs a call, in KV tiles, besides moving the rows that are cut: 16 rows take
// about as long as one.  5 tokens of 16 sequences, whole / cut: 500-2000 keys 31 / 33.5 us,
// 4096-8192 keys 94 / 79; 8 x 128 tokens on 8192 keys 106 / 129.
constexpr int kJoinCost = 8;
__host__ __device__ constexpr int join_cost(int rows) { return kJoinCost + rows / 16; }
// What cutting saves a call of `tiles` query tiles: whole ones take as long as the longest, or
// where there are more of them than the `ranges` CTAs, end about half of it apart.
__host__ __device__ constexpr long long cut_saves(long long tiles, int ranges, int longest,
                                                  int mean) {
  return tiles <= ranges ? longest - mean : longest / 2;
}
__device__ __forceinline__ int tile_cost(const Span& s) {
  return s.hi > s.lo ? s.hi - s.lo + kTileCost : 0;
}

// A piece of work: KV tiles [j0, j1) of the query tile of one block of packed heads at rows
// row0 .. of a sequence.
struct Piece {
  int b, base, nr;                               // sequence, its first token and query rows
  KeyRows kr;
  int hq, hk, row0, j0, j1;                      // first head, its K/V head, first row
  int part;                                      // place in the workspace, -1: the tile is whole
};
// The pieces of one CTA, found by one warp.
template <int TILES>
struct Work {
  static constexpr int ROWS = TILES * BM;
  int b, qt, blk;                                // the current query tile
  SeqRows sr;
  KeyRows kr;
  Span span;
  int u, ue;                                     // its KV tiles of this CTA, from span.lo
  int left;                                      // positions of the range after them

  // The whole of query tile `id`, in the order of block_pos; nothing past the last one.
  __device__ __forceinline__ void whole(const PagedArgs& px, const int* cu, int N, int H, int total,
                                        int id) {
    const int blocks = H >> px.pack, heads = px.B * blocks;
    b = blk = qt = u = ue = left = 0;
    sr = {0, 0, true};
    kr = {0, 0, 0};
    span = {0, 0};
    if (id >= heads * px.n_qt) return;
    const int g0 = id / (8 * px.n_qt) * 8, gsz = min(8, heads - g0), w = id - g0 * px.n_qt;
    const int bh = g0 + w % gsz;
    b = bh / blocks;
    blk = bh % blocks;
    qt = px.n_qt - 1 - w / gsz;                  // the last query tiles have the most work
    rows_of(px, cu, b, N, total, sr, kr);
    span = tile_span<TILES>(px, kr, qt * ROWS, sr.n << px.pack);
    ue = max(span.hi - span.lo, 0);
  }
  // To this CTA's first piece, where the work may be cut; false: there is none.  `cut` tells
  // whether it is: then the CTA has range blockIdx.x of px.ranges equal ones of all query
  // tiles' KV tiles, laid end to end (sequences, their query tiles, blocks of heads).
  __device__ __forceinline__ bool first(const PagedArgs& px, const int* cu, int N, int H, int total,
                                        bool& cut) {
    const int lane = threadIdx.x & 31, blocks = H >> px.pack, cta = static_cast<int>(blockIdx.x);
    auto cost = [&](int i) -> int {              // of query tile i of all sequences, every block
      SeqRows r;
      KeyRows k;
      rows_of(px, cu, i / px.n_qt, N, total, r, k);
      return tile_cost(tile_span<TILES>(px, k, i % px.n_qt * ROWS, r.n << px.pack)) * blocks;
    };
    const int n_i = px.B * px.n_qt, per = (n_i + 31) / 32;   // query tiles per lane
    int mine = 0, most = 0;
    for (int i = lane * per; i < min(lane * per + per, n_i); ++i) {
      const int c = cost(i);
      mine += c;
      most = max(most, c);
    }
    int incl = mine;
#pragma unroll
    for (int w = 1; w < 32; w *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, incl, w);
      if (lane >= w) incl += o;
    }
    const int sum = __shfl_sync(0xffffffffu, incl, 31);
    most = __reduce_max_sync(0xffffffffu, most) / blocks;
    cut = cut_saves(n_i * blocks, px.ranges, most, sum / px.ranges) >
          join_cost(min(N << px.pack, ROWS));
    if (!cut) {
      if (lane == 0) px.hdr[0].base = 0;
      whole(px, cu, N, H, total, cta);
      return cta < n_i * blocks;
    }
    if (cta >= px.ranges) return false;
    const int per_cta = max((sum - 1) / px.ranges + 1, 2 * kTileCost);
    const int x0 = static_cast<int>(min(static_cast<long long>(cta) * per_cta,
                                        static_cast<long long>(sum)));
    const int x1 = x0 + min(per_cta, sum - x0);
    RangeHeader h = {cta == 0, 0, 0, 0, 0, 0};
    if (x0 < x1) {
      const bool here = incl > x0 && incl - mine <= x0;            // one lane has position x0
      int at = incl - mine, i = lane * per;
      if (here)
        for (int c; at + (c = cost(i)) <= x0; ++i) at += c;
      const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
      i = __shfl_sync(0xffffffffu, i, src);
      at = __shfl_sync(0xffffffffu, at, src);
      b = i / px.n_qt;
      qt = i % px.n_qt;
      rows_of(px, cu, b, N, total, sr, kr);
      span = tile_span<TILES>(px, kr, qt * ROWS, sr.n << px.pack);
      const int c = tile_cost(span);
      blk = (x0 - at) / c;
      at += blk * c;                             // the query tile's first position
      const int off = x0 - at, take = min(c - off, x1 - x0);
      u = max(off - kTileCost, 0);
      ue = max(off + take - kTileCost, 0);
      left = x1 - x0 - take;
      if (u > 0 && u < ue)                       // its first KV tile lies in an earlier range
        h = {sr.base, blk << px.pack, qt * ROWS, min(ROWS, (sr.n << px.pack) - qt * ROWS),
             (at + kTileCost) / per_cta, (at + c - 1) / per_cta};
    }
    if (lane == 0) px.hdr[cta] = h;
    return x0 < x1 && (u < ue || next(px, cu, N, H, total));
  }
  // To the next piece.
  __device__ __forceinline__ bool next(const PagedArgs& px, const int* cu, int N, int H,
                                       int total) {
    do {
      if (left <= 0) return false;
      if (++blk == H >> px.pack) {
        blk = 0;
        do {
          if ((++qt) * ROWS >= sr.n << px.pack) {
            qt = 0;
            if (++b >= px.B) return false;       // not reached: `left` counts existing tiles
            rows_of(px, cu, b, N, total, sr, kr);
          }
          span = tile_span<TILES>(px, kr, qt * ROWS, sr.n << px.pack);
        } while (span.hi <= span.lo);
      }
      const int take = min(tile_cost(span), left);
      u = 0;
      ue = max(take - kTileCost, 0);
      left -= take;
    } while (ue == 0);
    return true;
  }
  __device__ __forceinline__ Piece piece(const PagedArgs& px, int group) const {
    Piece p;
    p.b = b;
    p.base = sr.base;
    p.nr = sr.n << px.pack;
    p.kr = kr;
    p.hq = blk << px.pack;
    p.hk = p.hq / group;
    p.row0 = qt * ROWS;
    p.j0 = span.lo + u;
    p.j1 = span.lo + ue;
    // a range has at most two pieces of cut tiles: one that it goes on with, one it begins
    p.part = ue - u == max(span.hi - span.lo, 0) ? -1 : 2 * static_cast<int>(blockIdx.x) + (u == 0);
    return p;
  }
};
// Rows of query tiles that see no key, which no range has: O = 0, L = -inf.  Thread i of n.
template <int TILES, int D>
__device__ __forceinline__ void rows_without_keys(const PagedArgs& px, const int* cu, int N, int H,
                                                  int total, uint16_t* Out, float* Lout, int i0,
                                                  int n) {
  constexpr int ROWS = TILES * BM;
  const int heads = 1 << px.pack, blocks = H >> px.pack;
  for (int b = static_cast<int>(blockIdx.x); b < px.B; b += static_cast<int>(gridDim.x)) {
    SeqRows sr;
    KeyRows kr;
    rows_of(px, cu, b, N, total, sr, kr);
    const int nr = sr.n << px.pack;
    for (int row0 = 0; row0 < nr; row0 += ROWS) {
      const Span s = tile_span<TILES>(px, kr, row0, nr);
      if (s.hi > s.lo) continue;
      const int rows = min(ROWS, nr - row0);
      for (int i = i0; i < rows * blocks; i += n) {
        const int r = row0 + i / blocks, h = i % blocks * heads + (r & (heads - 1));
        const size_t tok = static_cast<size_t>(sr.base + (r >> px.pack));
        uint4* dst = reinterpret_cast<uint4*>(Out + (tok * H + h) * D);
        for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
        Lout[static_cast<size_t>(h) * total + tok] = -INFINITY;
      }
    }
  }
}

// One warp's loads of 128-key tiles of a paged cache.  Lane i handles boxes i, i + 32, ..., NB of them (4
// for any page size; the call of codes takes 1 where boxes have 4 rows or more: the producer's
// instructions count there, 5 tokens of 16 sequences of 16384-32768 keys 187 against 170 us).
template <int NB>
struct PagedBoxes {
  int id[NB], row[NB];             // page id as the table has it, and first row in the page
  int past;                        // bit i: box lane + 32 i lies past the keys
};
using PagedTile = PagedBoxes<4>;
// Starts the tile's table loads.  Nothing here uses what they return: the warp would stand
// still for a load's latency instead of issuing the tile before this one.
template <int NB>
__device__ __forceinline__ void paged_fetch(const PagedArgs& px, int b, const KeyRows& k,
                                            int krow, int lane, PagedBoxes<NB>& t) {
  const int n_box = BN >> px.box_log2;
  t.past = 0;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
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
template <int NB>
__device__ __forceinline__ void paged_mask(const PagedArgs& px, int lane, const PagedBoxes<NB>& t,
                                           uint32_t slot) {
  uint32_t have = t.past;                        // keys past the end are masked by their index
#pragma unroll
  for (int i = 0; i < NB; ++i) have |= (paged_in_pool(px, t.id[i]) ? 1u : 0u) << i;
  uint32_t w[4] = {~0u, ~0u, ~0u, ~0u};
  if (__any_sync(0xffffffffu, have != (1u << NB) - 1u)) {
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
// Of `shares` warps (1 or 3), `share` issues every shares-th box.
template <int D>
__device__ __forceinline__ void paged_load(const PagedArgs& px, const CUtensorMap* map,
                                           uint32_t dst, uint32_t bar, int hk, int lane,
                                           const PagedTile& t, int share = 0, int shares = 1) {
  using C = Cfg<D>;
  const int n_box = BN >> px.box_log2;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int bx = lane + 32 * i;
    if (bx < n_box && (shares == 1 || bx % 3 == share)) {
      const int w = paged_in_pool(px, t.id[i]) ? t.id[i] : px.pg.pages;   // past the pool: zeros
#pragma unroll
      for (int c = 0; c < C::NCHUNK; ++c)
        tma_load_4d(dst + c * C::CHUNK_BYTES + (bx << px.box_log2) * C::SW, map, bar, c * C::ATOM,
                    t.row[i], hk, w);
    }
  }
}
// The same for a tile of codes, whose rows are one swizzle width.
template <int NB>
__device__ __forceinline__ void paged_load_codes(const PagedArgs& px, const CUtensorMap* map,
                                                 uint32_t dst, uint32_t bar, int hk, int lane,
                                                 const PagedBoxes<NB>& t) {
  const int n_box = BN >> px.box_log2;
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int bx = lane + 32 * i;
    if (bx < n_box) {
      const int w = paged_in_pool(px, t.id[i]) ? t.id[i] : px.pg.pages;   // past the pool: zeros
      tma_load_4d(dst + (bx << px.box_log2) * 128, map, bar, 0, t.row[i], hk, w);
    }
  }
}
// E4M3 codes to f16, which holds every one of them exactly.
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t w, bool upper) {
  uint32_t r;
  if (upper)
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
// A tile of 128 x 128 codes at `src` to f16 at `dst`, laid out as two boxes of 64 columns.  Of 64 threads
// the first 32 turn the left columns, 16 of every eighth row each; eight neighbours have eight
// rows, whose swizzled chunks lie in distinct banks.  Rows from `keys` on become zeros.
__device__ __forceinline__ void convert_tile(uint32_t src, uint32_t dst, int x, int keys) {
  using C = Cfg<128>;
  const int r0 = x & 7, c = x >> 3;              // row of each eight, 16-column chunk
  const uint32_t from = src + r0 * 128 + ((c ^ r0) << 4);
  const uint32_t to = dst + (c >> 2) * C::CHUNK_BYTES + r0 * 128;
  const uint32_t to0 = to + (((2 * c & 6) ^ r0) << 4), to1 = to + (((2 * c & 6 | 1) ^ r0) << 4);
#pragma unroll 1
  for (int i0 = 0; i0 < 16; i0 += 8) {
    uint32_t w[8][4];                            // loads first: they do not wait for one another
#pragma unroll
    for (int i = 0; i < 8; ++i)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[i][0]), "=r"(w[i][1]), "=r"(w[i][2]), "=r"(w[i][3])
                   : "r"(from + 1024 * (i0 + i))
                   : "memory");
    if (8 * i0 + 64 > keys) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * (i0 + i) + r0 >= keys) w[i][0] = w[i][1] = w[i][2] = w[i][3] = 0u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to0 + 1024 * (i0 + i)),
                   "r"(codes_to_f16(w[i][0], false)), "r"(codes_to_f16(w[i][0], true)),
                   "r"(codes_to_f16(w[i][1], false)), "r"(codes_to_f16(w[i][1], true))
                   : "memory");
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to1 + 1024 * (i0 + i)),
                   "r"(codes_to_f16(w[i][2], false)), "r"(codes_to_f16(w[i][2], true)),
                   "r"(codes_to_f16(w[i][3], false)), "r"(codes_to_f16(w[i][3], true))
                   : "memory");
    }
  }
}
// Row r of a bf16 query tile to f16, in place, times the power of two that brings its largest value
// to [2^14, 2^15): bf16's 8 bits fit f16's 11, and what falls below f16's normal numbers is
// 2^-28 of the row's largest value or less.  Returns the inverse power.
__device__ __forceinline__ float query_row_to_f16(uint32_t tile, int r) {
  using C = Cfg<128>;
  // Loops, read twice: the code runs once or a few times in a CTA, and unrolled it waits for its
  // instructions longer than for the data.
  auto at = [&](int i) {
    return tile + (i >> 3) * C::CHUNK_BYTES + r * 128 + (((i & 7) ^ (r & 7)) << 4);
  };
  auto load = [&](int i, uint32_t (&w)[4]) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at(i))
                 : "memory");
  };
  uint32_t top = 0;                              // largest absolute values of the 16-bit halves
#pragma unroll 1
  for (int i = 0; i < 16; i += 4) {
    uint32_t w[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) load(i + k, w[k]);
#pragma unroll
    for (int k = 0; k < 16; ++k) top = __vmaxu2(top, w[k / 4][k % 4] & 0x7fff7fffu);
  }
  // exponent of the largest value; 2^(14 - e) and its inverse stay normal numbers
  const int e = max(static_cast<int>(max(top & 0xffffu, top >> 16) >> 7) - 127, -112);
  const float f = __int_as_float((14 - e + 127) << 23);
#pragma unroll 1
  for (int i = 0; i < 16; i += 4) {
    uint32_t w[4][4];
#pragma unroll
    for (int k = 0; k < 4; ++k) load(i + k, w[k]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 v = unpack2<true>(w[k][m]);
        w[k][m] = pack2<false>(v.x * f, v.y * f);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(i + k)), "r"(w[k][0]),
                   "r"(w[k][1]), "r"(w[k][2]), "r"(w[k][3])
                   : "memory");
    }
  }
  return __int_as_float((e - 14 + 127) << 23);
}
// Which keys a row of a paged query tile may attend: [lo, lim).
struct RowKeys {
  int lo, lim;
};
__device__ __forceinline__ RowKeys row_keys(const KeyRows& k, int row, int pack) {
  return {(row >> pack) + k.lo, min((row >> pack) + k.hi + 1, k.n)};
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
// The unmasked tile's test is the thread's own row, voted on: limits of the whole tile beside the
// row's are two more registers (1 x 8192, 32 heads, d = 64: 280.1 against 285.6 us).
template <bool WORDS>
__device__ __forceinline__ void paged_masks(const RowKeys& r, int kbase, uint32_t (&w)[4],
                                            uint32_t (&s)[BN]) {
  const bool all = kbase + BN <= r.lim && kbase >= r.lo && (w[0] & w[1] & w[2] & w[3]) == ~0u;
  if (__all_sync(0xffffffffu, all)) return;
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

// RANGES: the CTA may have several pieces of work, which warp 0 finds and hands on; otherwise it
// has one query tile, found by every thread.  The loop over pieces costs tiles that are not cut
// 2 to 9 % (8 prompts of 1000 tokens 108 against 99 us, 2 x 2048 on 8192 keys 345 against 338).
// C8: pools of E4M3 codes.  The products take f16: warps 2 and 3 turn each tile of codes, which lands in
// a ring of its own, into a ring of f16 tiles, and the softmax threads turn bf16 query rows when a
// tile of them arrives.  Every code is an f16 value, so K and V lose nothing; P is f16 for both
// types of queries.  Bound: as with 16-bit pools for many rows (2 x 2048 tokens on 8192 keys, 32/8
// heads: 337 against 335 us); for few the shared memory's port, which a KV tile's copy, conversion
// and products hold for 1790 of its 2040 cycles, not the codes' bytes (16 x 5 tokens on
// 16384-32768 keys: 167 us, 4.8 TB/s of codes, from 16-bit pools 258).  Other splits, measured when the
// two took 343 and 186 us: one converter warp for K and one for V 432 us for the former (a tile's
// conversion is waited for), four converter warps in a warpgroup of their own 358 and 213 (they share
// the one port, and leave the softmax threads 184 registers); two tiles of codes ahead instead of four
// 220 for the latter.  With ranges 40 bytes of a thread's registers spill (8 from 16-bit pools),
// which costs little: 4800 of the 2.1 million warp instructions of 4 x 5 tokens on 1500-2500 keys move
// them, and 31 thousand of the 56 million of the long ones.
// SCALE_LAST: v_scale multiplies means of the codes, which are at most 448.  Whole tiles otherwise take
// v_scale / l_run for 1 / l_run, which costs nothing but falls below fp32's normal numbers for a very
// small one (the multiplication costs 2 x 2048 tokens on 8192 keys 1 to 2 %: 342 to 346 against 338 us).
template <int D, bool BF16, bool RANGES, bool C8, bool SCALE_LAST>
__global__ void __launch_bounds__(THREADS, 1)
    fwd_paged_kernel(const __grid_constant__ CUtensorMap tmQ,
                     const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, void* __restrict__ Out,
                     float* __restrict__ Lout, int N, int group, const int* cu_seqlens, int H,
                     int total, float c_log2, KernelCtl ctl, const PagedArgs px) {
  using C = Cfg<D, C8>;
  constexpr bool PB = BF16 && !C8;              // the products' operands are bf16
  constexpr bool HALVES = C8 && RANGES;         // few rows: see halved()
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sg = smem_raw + (sb - raw);

  grid_dep_launch();                            // the next kernel may start setting up
  grid_dep_wait();                              // offsets, lengths, table and inputs are written
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pack = px.pack;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  Work<NT> work;
  bool have = true, cuts = false;
  Piece mine = {};                              // without ranges
  if (!RANGES) {
    work.whole(px, cu_seqlens, N, H, total, static_cast<int>(blockIdx.x));
    mine = work.piece(px, group);
    mine.part = -1;
  }
  if (!RANGES && mine.j0 >= mine.j1) {          // past the sequence's queries, or before its keys
    const int heads = 1 << pack;
    for (int r = mine.row0 + threadIdx.x; r < min(mine.row0 + NT * BM, mine.nr); r += THREADS) {
      const int h = mine.hq + (r & (heads - 1));
      const size_t tok = static_cast<size_t>(mine.base + (r >> pack));
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<T*>(Out) + (tok * H + h) * D);
      for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
      Lout[static_cast<size_t>(h) * total + tok] = -INFINITY;
    }
    return;
  }
  // Pieces pass to the warps that need them through two slots.
  static_assert(sizeof(Piece) <= 64, "a slot of the ring");
  auto info = [&](int k) -> volatile Piece* {
    return reinterpret_cast<volatile Piece*>(sg + C::INFO_OFF + 64 * (k & 1));
  };
  // KV tiles [lo, hi) of Q tile t that a piece has
  auto tiles_of = [&](const volatile Piece& p, int t, int& lo, int& hi) {
    const KeyRows kr = {p.kr.n, p.kr.lo, p.kr.hi};
    paged_tiles(kr, p.row0 + t * BM, p.nr, pack, lo, hi);
    lo = min(max(lo, p.j0), p.j1);
    hi = min(max(hi, p.j0), p.j1);
  };

  // A piece of codes whose query tile has rows in its first half only: both softmax warpgroups work on
  // these rows, on every other KV tile each, and the first one joins the two results.  That costs
  // about what two KV tiles take: 16 x 5 tokens on 16384-32768 keys 167 against 229 us; pieces of
  // four too, 4 x 5 tokens on 1500-2500 keys 18.6 against 17.7 (on 2000 each 16.8 against 17.8).
  auto halved = [&](const volatile Piece& p) {
    return HALVES && p.nr - p.row0 <= BM && p.j1 - p.j0 >= 6;
  };

  auto bar = [&](int i) -> uint32_t { return sb + C::BAR_OFF + 8 * i; };
  const int B_QF = 0;
  // K and V tiles of step g: their place in the order in which the rings' stages are filled, the
  // stage, and how often it has been filled before.  Codes: both take stages of one ring in turn,
  // K(0), V(0), K(1), V(1), ... of a piece, or where it is halved, as its products go,
  // K(0), K(1), V(0), K(2), V(1), ..., V(n - 1).
  auto k_place = [](int g) { return C8 ? 2 * g : g; };
  auto v_place = [](int g) { return C8 ? 2 * g + 1 : g; };
  auto k_place2 = [](int g0, int jj) { return 2 * g0 + max(2 * jj - 1, 0); };
  auto v_place2 = [](int g0, int jj, int n) { return 2 * g0 + min(2 * jj + 2, 2 * n - 1); };
  constexpr int RING = C8 ? C::TILES16 : C::STAGES;
  auto stage = [](int place) { return place % RING; };
  auto phase = [](int place) -> uint32_t { return (place / RING) & 1; };
  auto B_KF = [&](int s) { return 1 + s; };
  auto B_KE = [&](int s) { return 1 + RING + s; };
  auto B_VF = [&](int s) { return C8 ? 1 + s : 1 + 2 * C::STAGES + s; };
  auto B_VE = [&](int s) { return C8 ? 1 + RING + s : 1 + 3 * C::STAGES + s; };
  auto B_SF = [&](int t) { return 1 + 4 * C::STAGES + t; };
  auto B_PF = [&](int t) { return 3 + 4 * C::STAGES + t; };
  auto B_OF = [&](int t) { return 5 + 4 * C::STAGES + t; };
  const int B_DONE = 7 + 4 * C::STAGES, B_QE = B_DONE + 1;
  // Producers: issuing a box takes a warp about 50 cycles, small ones more in all than the products
  // take.  Boxes of 32 rows and more: warp 0 alone; of 16: warp 2 issues V's; of 8 and fewer: warps
  // 0, 2 and 3 a third of them each.  One / two / three warps, 2 x 1024 tokens on 4096 keys: pages
  // of 32 rows 94.7 / 96.2 / 101.6 us, of 16 105 / 96.5 / 100.6, of 8 152 / - / 103, of one
  // 820 / - / 341; 5 tokens of 16 sequences of 16384-32768 keys, pages of 16: 306 / 257 / 308.
  // Codes: warp 0 alone (half as many boxes), the other two convert.
  const int producers = C8 ? 1 : px.box_log2 <= 3 ? 3 : px.box_log2 == 4 ? 2 : 1;
  auto B_TF = [&](int k) { return B_DONE + 2 + (k & 1); };
  auto B_TE = [&](int k) { return B_DONE + 4 + (k & 1); };
  auto B_CF = [&](int c) { return B_DONE + 6 + c; };
  auto B_CE = [&](int c) { return B_DONE + 6 + C::CODES + c; };
  const int B_QT = B_DONE + 6 + 2 * C::CODES, B_HF = B_QT + 1, B_HE = B_QT + 2;

  if (threadIdx.x == 0) {
    if (!RANGES) *const_cast<Piece*>(info(0)) = mine;
    for (int i = 0; i < C::NBARS; ++i) mbar_init(bar(i), 1);
    for (int t = 0; t < NT; ++t) mbar_init(bar(B_PF(t)), 128);
    // readers of a piece: the MMA thread, 8 softmax warps, and the other producers or converters
    for (int k = 0; k < 2; ++k) mbar_init(bar(B_TE(k)), C8 ? 11 : 8 + producers);
    if (C8) {
      for (int s = 0; s < C::TILES16; ++s) mbar_init(bar(B_KF(s)), 2);
      for (int c = 0; c < C::CODES; ++c) mbar_init(bar(B_CE(c)), 2);
      mbar_init(bar(B_QT), NT * 128);
      mbar_init(bar(B_HF), 128);
      mbar_init(bar(B_HE), 128);
    }
    fence_mbar_init();
  }
  PagedTile first_tile;                         // its look-up passes under the set-up
  if (warp == 0) {
    if (RANGES) have = work.first(px, cu_seqlens, N, H, total, cuts);
    if (have && work.u < work.ue)
      paged_fetch(px, work.b, work.kr, (work.span.lo + work.u) * BN, lane, first_tile);
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
      bool ok = true;
      int g = 0, nk = 0, nv = 0, nq = 0;         // KV steps, K, V and Q tiles loaded
      int n_pieces = 0;
      for (int k = 0; !RANGES || have; ++k) {
        const Piece p = RANGES ? work.piece(px, group) : mine;
        if (RANGES) {
          if (!(ok = mbar_wait_warp(bar(B_TE(k)), ((k >> 1) & 1) ^ 1, ctl))) break;
          if (lane == 0) {
            *const_cast<Piece*>(info(k)) = p;
            mbar_arrive(bar(B_TF(k)));           // release: the piece is seen with the phase
          }
        }
        if (p.j0 < p.j1) {
          // Q free once the previous piece's last S is done
          if (RANGES && !(ok = mbar_wait_warp(bar(B_QE), (nq & 1) ^ 1, ctl))) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_QF), NT * C::TILE_BYTES);
            for (int t = 0; t < NT; ++t)
              for (int c = 0; c < C::NCHUNK; ++c)
                tma_load_3d(sb + C::Q_OFF + t * C::TILE_BYTES + c * C::CHUNK_BYTES, &tmQ, bar(B_QF),
                            c * C::ATOM, p.hq,
                            p.base + ((p.row0 + (halved(p) ? 0 : t * BM)) >> pack));
          }
          ++nq;
          PagedTile next;
          if (k == 0) next = first_tile;
          else paged_fetch(px, work.b, p.kr, p.j0 * BN, lane, next);
          if constexpr (C8) {
            const int n = p.j1 - p.j0;
            const bool ahead = halved(p);
            auto load = [&](const CUtensorMap* map, const auto& t, int at) -> bool {
              // at: step whose mask goes with the tile, or -1.  The codes' buffer is free once the
              // tile four places before is converted, for which PV of four steps before or more
              // had to be done: so are the steps whose slots of the masks are taken.
              const int c = nk % C::CODES;         // nk: tiles loaded, K and V
              if (!mbar_wait_warp(bar(B_CE(c)), ((nk / C::CODES) & 1) ^ 1, ctl)) return false;
              // the boxes first: their bytes may come before they are announced, the phase lasts
              // until they have been
              paged_load_codes(px, map, sb + C::CODE_OFF + c * C::CODE_BYTES, bar(B_CF(c)), p.hk, lane, t);
              if (at >= 0) paged_mask(px, lane, t, sb + C::MASK_OFF + (at % kMaskSlots) * 16);
              __syncwarp();
              if (lane == 0) mbar_arrive_expect_tx(bar(B_CF(c)), C::CODE_BYTES);
              ++nk;
              return true;
            };
            auto load_all = [&](auto ahead_of) {   // the first tile's boxes
              auto before = ahead_of, cur = ahead_of;   // of V, a step behind where K goes ahead, and of K
              for (int jj = 0; jj < n + ahead && ok; ++jj) {
                before = cur;
                cur = ahead_of;
                if (jj < n) ok = load(&tmK, cur, g + jj);
                if (jj + 1 < n) paged_fetch(px, work.b, p.kr, (p.j0 + jj + 1) * BN, lane, ahead_of);
                if (ok && jj >= ahead) ok = load(&tmV, ahead ? before : cur, -1);
              }
            };
            if (px.box_log2 >= 2) load_all(PagedBoxes<1>{{next.id[0]}, {next.row[0]}, next.past & 1});
            else load_all(next);
            g += n;
          }
          for (int j = p.j0; !C8 && j < p.j1; ++j, ++g) {
            const int s = g % C::STAGES;
            const uint32_t ph = (g / C::STAGES) & 1;
            const PagedTile cur = next;
            if (j + 1 < p.j1) paged_fetch(px, work.b, p.kr, (j + 1) * BN, lane, next);
            if (!(ok = mbar_wait_warp(bar(B_KE(s)), ph ^ 1, ctl))) break;
            // the slot's last readers were the softmax threads of step g - 8: they are done,
            // since S(g - 2), whose K tile has just been released, waited for their P
            paged_mask(px, lane, cur, sb + C::MASK_OFF + (g % kMaskSlots) * 16);
            if (lane == 0) mbar_arrive_expect_tx(bar(B_KF(s)), C::TILE_BYTES);
            __syncwarp();
            paged_load<D>(px, &tmK, sb + C::K_OFF + s * C::TILE_BYTES, bar(B_KF(s)), p.hk, lane, cur,
                          0, producers == 3 ? 3 : 1);
            ++nk;
            if (producers == 2) continue;
            if (!(ok = mbar_wait_warp(bar(B_VE(s)), ph ^ 1, ctl))) break;
            if (lane == 0) mbar_arrive_expect_tx(bar(B_VF(s)), C::TILE_BYTES);
            __syncwarp();
            paged_load<D>(px, &tmV, sb + C::V_OFF + s * C::TILE_BYTES, bar(B_VF(s)), p.hk, lane, cur,
                          0, producers);
            ++nv;
          }
          if (!ok) break;
        }
        if (!RANGES) break;
        have = cuts && work.next(px, cu_seqlens, N, H, total);
        n_pieces = k + 1;
      }
      if (RANGES && ok && (ok = mbar_wait_warp(bar(B_TE(n_pieces)), ((n_pieces >> 1) & 1) ^ 1, ctl))) {
        if (lane == 0) {
          info(n_pieces)->nr = -1;               // the end
          mbar_arrive(bar(B_TF(n_pieces)));
        }
      }
      if (!ok) {
        // drain: wait (bounded) for the copies in flight, so that none lands in shared memory
        // after the CTA has gone
        if (nq > 0) mbar_wait_warp(bar(B_QF), (nq - 1) & 1, ctl);
        if (C8) {
          for (int i = max(0, nk - C::CODES); i < nk; ++i)
            mbar_wait_warp(bar(B_CF(i % C::CODES)), (i / C::CODES) & 1, ctl);
          nk = 0;
        }
        for (int i = max(0, nk - C::STAGES); i < nk; ++i)
          mbar_wait_warp(bar(B_KF(i % C::STAGES)), (i / C::STAGES) & 1, ctl);
        for (int i = max(0, nv - C::STAGES); i < nv; ++i)
          mbar_wait_warp(bar(B_VF(i % C::STAGES)), (i / C::STAGES) & 1, ctl);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    regs_dec<kRegsLow>();
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      constexpr uint32_t idS = umma_idesc_f16(BM, BN, PB, false, false);
      constexpr uint32_t idO = umma_idesc_f16(BM, D, PB, false, true);
      // descriptor low words of Q tile 0 and of stage 0 of the K and V rings (K-major
      // with LBO 16; V MN-major with LBO = one swizzle-width chunk); tiles and stages
      // are TILE_BYTES apart
      constexpr uint32_t HI = sdesc_hi(8 * C::SW, C::SWZ), STAGE_W = C::TILE_BYTES >> 4;
      const uint32_t q_lo = sdesc_lo(sb + C::Q_OFF, 16), k_lo = sdesc_lo(sb + C::K_OFF, 16);
      const uint32_t v_lo = sdesc_lo(sb + (C8 ? C::K_OFF : C::V_OFF), C::CHUNK_BYTES);
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
      // The step index g of the K and V rings runs on across pieces; p_full[t] has had np[t]
      // phases before the current piece.
      bool ok = true;
      int g = 0, nq = 0, np[NT] = {};
      for (int k = 0;; ++k) {
        if (RANGES && !(ok = mbar_wait(bar(B_TF(k)), (k >> 1) & 1, ctl))) break;
        const volatile Piece& p = *info(k);
        if (p.nr < 0) break;
        const int j0 = p.j0, n = p.j1 - j0, g0 = g;
        const bool halved_piece = halved(p);
        int lo_t[NT], n_t[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) tiles_of(p, t, lo_t[t], n_t[t]);
        if (RANGES) mbar_arrive(bar(B_TE(k)));
        if (RANGES && n <= 0) continue;
        if (!(ok = mbar_wait(bar(C8 && BF16 ? B_QT : B_QF), nq & 1, ctl) &&
                   mbar_wait(bar(B_KF(stage(k_place(g)))), phase(k_place(g)), ctl)))
          break;
        ++nq;
        tc_fence_after();
        if (HALVES && halved_piece) {              // Q tile jj % 2 takes part in step jj
          auto step_S = [&](int jj) {            // of step g + jj - j, whose K tile is there
            const int s = stage(k_place2(g0, jj));
            issue_S(jj & 1, s);
            umma_commit(bar(B_SF(jj & 1)));
            umma_commit(bar(B_KE(s)));
            if (RANGES && jj + 1 == n) umma_commit(bar(B_QE));
          };
          auto wait_K = [&](int jj) {
            const int at = k_place2(g0, jj);
            if (!(ok = mbar_wait(bar(B_KF(stage(at))), phase(at), ctl))) return false;
            tc_fence_after();
            return true;
          };
          step_S(0);
          if (wait_K(1)) step_S(1);
          for (int jj = 0; jj < n && ok; ++jj, ++g) {
            const int t = jj & 1, at = v_place2(g0, jj, n), s = stage(at);
            if (!(ok = mbar_wait(bar(B_VF(s)), phase(at), ctl) &&
                       mbar_wait(bar(B_PF(t)), (np[t] + (jj >> 1)) & 1, ctl)))
              break;
            tc_fence_after();
            issue_PV(t, s, jj > 1);
            umma_commit(bar(B_VE(s)));
            if (jj + 2 >= n) umma_commit(bar(B_OF(t)));
            else if (wait_K(jj + 2)) step_S(jj + 2);
          }
          np[0] += (n + 1) / 2;
          np[1] += n / 2;
          if (!RANGES || !ok) break;
          continue;
        }
        for (int t = 0; t < NT; ++t)
          if (lo_t[t] == j0 && n_t[t] > j0) {
            issue_S(t, stage(k_place(g)));
            umma_commit(bar(B_SF(t)));
          }
        umma_commit(bar(B_KE(stage(k_place(g)))));
        if (RANGES && n == 1) umma_commit(bar(B_QE));
        // step g holds KV tile j = j0 + jj; Q tile t takes part while
        // lo_t[t] <= j < n_t[t], its own iteration index being j - lo_t[t]
        for (int jj = 0; jj < n; ++jj, ++g) {
          const int j = j0 + jj;
          const int s = stage(v_place(g)), s1 = stage(k_place(g + 1));
          const uint32_t ph = phase(v_place(g)), ph1 = phase(k_place(g + 1));
          if (!(ok = mbar_wait(bar(B_VF(s)), ph, ctl))) break;
          bool k_next = false;
          for (int t = 0; t < NT && ok; ++t) {
            const bool in_t = j >= lo_t[t] && j < n_t[t];
            if (in_t) {
              if (!(ok = mbar_wait(bar(B_PF(t)), (np[t] + j - lo_t[t]) & 1, ctl))) break;
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
          if (RANGES && jj + 2 == n) umma_commit(bar(B_QE));   // the piece's last S is on its way
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) np[t] += n_t[t] - lo_t[t];
        if (!RANGES || !ok) break;
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
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::S_COL + t * BN;
    const uint32_t tO = tmem + lane_off + C::O_COL + t * D;
    bool ok = true;
    int g = 0, ns = 0, no = 0;                   // ring steps, phases of s_full and o_full so far
    // C8: query tiles turned to f16, halves joined, phases of the second o_full
    int nq = 0, nh = 0, no1 = 0;
    float c_row = c_log2;
    for (int k = 0;; ++k) {
      if (RANGES && !mbar_wait_warp(bar(B_TF(k)), (k >> 1) & 1, ctl)) break;
      const volatile Piece& p = *info(k);
      if (p.nr < 0) break;
      int lo, hi;
      tiles_of(p, t, lo, hi);
      const bool half = halved(p);
      int nt = hi - lo, row = p.row0 + t * BM + rit, by = 1;   // its KV tiles, the thread's row
      if (HALVES && half) {
        lo = p.j0 + t;
        nt = (p.j1 - p.j0 + 1 - t) / 2;
        row = p.row0 + rit;
        by = 2;
      }
      const int g0 = g + lo - p.j0;                // its first step
      // rows past the sequence's end: nothing is computed for a warp of them, what its rows of S and
      // O hold is not read
      const bool idle = C8 && row - lane >= p.nr;
      const int Nk = p.kr.n;
      const KeyRows kr = {Nk, p.kr.lo, p.kr.hi};
      const RowKeys rk = row_keys(kr, row, pack);
      float m_run = -INFINITY, l_run = 0.f;
      if constexpr (C8 && BF16) {
        if (p.j0 < p.j1) {
          if (!(ok = mbar_wait_warp(bar(B_QF), nq & 1, ctl))) break;
          ++nq;
          // the row's power of two goes to its scores' factor, which stays a normal number: masked
          // scores are -inf and have to stay so
          if (!idle) {
            const float back = query_row_to_f16(sb + C::Q_OFF + t * C::TILE_BYTES, rit);
            c_row = fminf(fmaxf(c_log2 * back, 0x1p-126f), 0x1.fffffep127f);
            fence_proxy_async_smem();
          }
          mbar_arrive(bar(B_QT));
        }
      }
      for (int j = 0; j < nt; ++j) {
        if (!(ok = mbar_wait_warp(bar(B_SF(t)), (ns + j) & 1, ctl))) break;
        tc_fence_after();
        if (C8 && idle) {
          tc_fence_before();
          mbar_arrive(bar(B_PF(t)));
          continue;
        }
        uint32_t mask[4], sr[BN];
        load_mask(sb + C::MASK_OFF + ((g0 + (HALVES ? j * by : j)) % kMaskSlots) * 16, mask);
        tmem_ld32(tS + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_ld32(tS + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
        tmem_ld32(tS + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
        tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
        const int kbase = (lo + (HALVES ? j * by : j)) * BN;
        paged_masks<false>(rk, kbase, mask, sr);
        if (!C8 && kbase + BN > Nk) {              // the last tile's V rows past the keys
          const int jj = g0 + j;                   // step of the rings
          if (!(ok = mbar_wait_warp(bar(B_VF(jj % C::STAGES)), (jj / C::STAGES) & 1, ctl))) break;
          if (kbase + rit >= Nk) clear_row<D>(sb + C::V_OFF + (jj % C::STAGES) * C::TILE_BYTES, rit);
          fence_proxy_async_smem();                // before this thread's arrival on p_full
        }
        // row maximum: four independent chains of 3-input max
        const float mx = row_max128(sr);
        const float cl = C8 && BF16 ? c_row : c_log2;
        const float m_tile = mx * cl;
        const bool grow_m = m_tile > m_run + RESCALE_LOG2;
        const float m_use = grow_m ? m_tile : m_run;
        const float alpha = grow_m ? ex2(m_run - m_use) : 1.f;
        const float m_sub = (m_use == -INFINITY) ? 0.f : m_use;
        const float2 c2 = make_float2(cl, cl), nm2 = make_float2(P_LOG2<PB> - m_sub, P_LOG2<PB> - m_sub);
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
            pk[i] = pack2<PB>(pp.x, pp.y);
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
      if (!ok) break;
      // where the row lies in O, in the workspace, and in L or the workspace's L
      const int grow = HALVES ? row : p.row0 + t * BM + rit, Nr = p.nr, part = RANGES ? p.part : -1;
      const int h = p.hq + (grow & ((1 << pack) - 1));
      const size_t tok = static_cast<size_t>(p.base + (grow >> pack)), row_at = tok * H + h;
      const size_t part_at = static_cast<size_t>(part) * (NT * BM) + (t * BM + rit);
      float* lse_at = part >= 0 ? px.part_l + part_at : Lout + static_cast<size_t>(h) * total + tok;
      // the second warpgroup's half of the KV tiles: its m and l go to shared memory, its O is read
      // where it lies, in the same lanes of tensor memory
      const bool join = HALVES && half;
      float2* const ml = reinterpret_cast<float2*>(sg + C::HALF_OFF) + rit;
      float a0 = 1.f, a1 = 0.f;
      if (HALVES && half && t == 1) {
        ++no;                                      // the other one waits for its O
        *ml = make_float2(m_run, l_run);
        mbar_arrive(bar(B_HF));
        if (!(ok = mbar_wait_warp(bar(B_HE), nh & 1, ctl))) break;
        ++nh;
        tc_fence_after();
      } else if (nt > 0) {
        if (!(ok = mbar_wait_warp(bar(B_OF(t)), no & 1, ctl))) break;
        ++no;
        if (HALVES && join) {
          // its arrival first: it has then seen its o_full phases up to this piece's
          if (!(ok = mbar_wait_warp(bar(B_HF), nh & 1, ctl) && mbar_wait_warp(bar(B_OF(1)), no1 & 1, ctl)))
            break;
          ++nh;
          const float2 other = *ml;
          const float m = fmaxf(m_run, other.x), base = m == -INFINITY ? 0.f : m;
          a0 = ex2(m_run - base);
          a1 = ex2(other.x - base);
          // a row none of whose keys is in a half: that half's O may be 0 x NaN
          if (l_run == 0.f) a0 = 0.f;
          if (other.y == 0.f) a1 = 0.f;
          l_run = l_run * a0 + other.y * a1;
          m_run = m;
        }
        tc_fence_after();
        // a row whose keys are all masked: 0, whatever its tiles' values (0 x NaN) left in acc
        const bool none = l_run == 0.f;
        const float inv_l = none ? 0.f : (C8 && !SCALE_LAST ? px.o_scale : 1.f) / l_run;
        auto out = [&](uint32_t x) {
          const float y = __uint_as_float(x) * inv_l;
          return SCALE_LAST ? y * px.o_scale : y;
        };
        const bool valid = grow < Nr;
#pragma unroll (HALVES ? 1 : D / 32)         // few tokens wait for instructions: 160 against 162 us
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * cc, o);
          tmem_ld_wait_regs(o);
          if (HALVES && join) {
            uint32_t o1[32];
            tmem_ld32(tO + D + 32 * cc, o1);
            tmem_ld_wait_regs(o1);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float u = a0 > 0.f ? __uint_as_float(o[i]) * a0 : 0.f;
              o[i] = __float_as_uint(a1 > 0.f ? fmaf(__uint_as_float(o1[i]), a1, u) : u);
            }
          }
          if (part >= 0) {
            if (valid) {
              float4* dst = reinterpret_cast<float4*>(px.part + part_at * D + 32 * cc);
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
            w[i] = none ? 0u
                        : pack2<BF16>(out(o[2 * i]), out(o[2 * i + 1]));
          if (valid) {
            uint4* dst =
                reinterpret_cast<uint4*>(reinterpret_cast<T*>(Out) + row_at * D + 32 * cc);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              dst[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          }
        }
        if (valid)
          *lse_at = none ? -INFINITY : (m_run - P_LOG2<PB> + log2f(l_run)) * 0.69314718055994531f;
        tc_fence_before();                         // O read before the next piece's p_full
        if (HALVES && join) mbar_arrive(bar(B_HE));
      } else if (grow < Nr) {
        // the row sees no key here: O = 0, L = -inf (a piece's O is not read where its L is -inf)
        if (part < 0) {
          uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<T*>(Out) + row_at * D);
          for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        *lse_at = -INFINITY;
      }
      ns += nt;
      if (HALVES && t == 0) {                      // whether the second Q tile had KV tiles
        int lo1 = 0, hi1 = p.j1 - p.j0 - 1;
        if (!half) tiles_of(p, 1, lo1, hi1);
        no1 += hi1 > lo1;
      }
      g += p.j1 - p.j0;
      if (!RANGES) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_TE(k)));  // the slot may take the piece after the next
    }
  } else {
    regs_dec<kRegsLow>();
    // ------------------------------------------------------------ converters of codes
    if constexpr (C8) {
      bool ok = true;
      int g = 0;                                 // tiles converted
      const int x = static_cast<int>(threadIdx.x) - 64;
      for (int k = 0;; ++k) {
        if (RANGES && !(ok = mbar_wait_warp(bar(B_TF(k)), (k >> 1) & 1, ctl))) break;
        const volatile Piece& p = *info(k);
        if (p.nr < 0) break;
        const int n = p.kr.n, j0 = p.j0, steps = p.j1 - j0;
        const bool ahead = halved(p);
        if (RANGES) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_TE(k)));
        }
        for (int i = 0; i < 2 * steps; ++i, ++g) {
          // the piece's i-th tile: which it is, and of V the keys, past which rows are cleared
          const bool last = i == 2 * steps - 1, is_v = ahead ? i > 0 && ((i & 1) == 0 || last) : i & 1;
          const int jj = !is_v ? 0 : !ahead ? i >> 1 : last ? steps - 1 : (i >> 1) - 1;
          const int c = g % C::CODES, s = stage(g);
          if (!(ok = mbar_wait_warp(bar(B_CF(c)), (g / C::CODES) & 1, ctl) &&
                     mbar_wait_warp(bar(B_KE(s)), phase(g) ^ 1, ctl)))
            break;
          convert_tile(sb + C::CODE_OFF + c * C::CODE_BYTES, sb + C::K_OFF + s * C::TILE_BYTES, x,
                       is_v ? n - (j0 + jj) * BN : BN);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar(B_CE(c)));
            mbar_arrive(bar(B_KF(s)));
          }
        }
        if (!RANGES || !ok) break;
      }
    }
    // ------------------------------------------------------------ further producers
    if (!C8 && warp <= producers) {
      bool ok = true;
      int g = 0, nk = 0, nv = 0;
      for (int k = 0;; ++k) {
        if (RANGES && !(ok = mbar_wait_warp(bar(B_TF(k)), (k >> 1) & 1, ctl))) break;
        const volatile Piece& p = *info(k);
        if (p.nr < 0) break;
        const KeyRows kr = {p.kr.n, p.kr.lo, p.kr.hi};
        const int b = p.b, hk = p.hk, j0 = p.j0, j1 = p.j1;
        if (RANGES) {
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_TE(k)));
        }
        PagedTile next;
        if (j0 < j1) paged_fetch(px, b, kr, j0 * BN, lane, next);
        for (int j = j0; j < j1; ++j, ++g) {
          const int s = g % C::STAGES;
          const uint32_t ph = (g / C::STAGES) & 1;
          const PagedTile cur = next;
          if (j + 1 < j1) paged_fetch(px, b, kr, (j + 1) * BN, lane, next);
          // of three producers warp 0 announces the bytes, which may come before: the phase lasts
          // until it has
          if (producers == 3) {
            if (!(ok = mbar_wait_warp(bar(B_KE(s)), ph ^ 1, ctl))) break;
            paged_load<D>(px, &tmK, sb + C::K_OFF + s * C::TILE_BYTES, bar(B_KF(s)), hk, lane, cur,
                          warp - 1, 3);
            ++nk;
          }
          if (!(ok = mbar_wait_warp(bar(B_VE(s)), ph ^ 1, ctl))) break;
          if (producers == 2 && lane == 0) mbar_arrive_expect_tx(bar(B_VF(s)), C::TILE_BYTES);
          __syncwarp();
          paged_load<D>(px, &tmV, sb + C::V_OFF + s * C::TILE_BYTES, bar(B_VF(s)), hk, lane, cur,
                        producers == 3 ? warp - 1 : 0, producers == 3 ? 3 : 1);
          ++nv;
        }
        if (!RANGES || !ok) break;
      }
      if (!ok) {                                   // as warp 0
        for (int i = max(0, nk - C::STAGES); i < nk; ++i)
          mbar_wait_warp(bar(B_KF(i % C::STAGES)), (i / C::STAGES) & 1, ctl);
        for (int i = max(0, nv - C::STAGES); i < nv; ++i)
          mbar_wait_warp(bar(B_VF(i % C::STAGES)), (i / C::STAGES) & 1, ctl);
      }
    }
    // ------------------------------------------------------------ rows without keys
    if (RANGES)
      rows_without_keys<NT, D>(px, cu_seqlens, N, H, total, static_cast<uint16_t*>(Out), Lout,
                               static_cast<int>(threadIdx.x) - 64, 64);
  }
  // ------------------------------------------------------------ teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

size_t hdr_bytes(int ranges) { return (ranges * sizeof(RangeHeader) + 15) / 16 * 16; }

PagedArgs paged_args(const FwdArgs& a, int rows, int d) {
  PagedArgs px;
  px.n_qt = static_cast<int>(((static_cast<long long>(a.N) << a.pack) + rows - 1) / rows);
  px.pg = a.pg;
  px.box_log2 = a.box_log2;
  px.causal = a.causal;
  px.window = a.window;
  px.pack = a.pack;
  px.B = a.B;
  px.ranges = a.ranges;
  px.hdr = static_cast<RangeHeader*>(a.ws);
  px.part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + hdr_bytes(a.ranges));
  px.part_l = px.part + static_cast<size_t>(2 * a.ranges) * rows * d;
  px.o_scale = a.o_scale;
  return px;
}

template <int D, bool BF16, bool RANGES, bool C8, bool SCALE_LAST>
cudaError_t launch_fwd_paged2_t(const FwdArgs& a, cudaStream_t st) {
  using C = Cfg<D, C8>;
  constexpr int smem = C::SMEM_BYTES;
  static_assert(smem <= 232448, "shared memory of a CTA");
  auto kern = fwd_paged_kernel<D, BF16, RANGES, C8, SCALE_LAST>;
  cudaError_t e = check_split_regs(reinterpret_cast<const void*>(kern));
  if (e != cudaSuccess) return e;
  e = ensure_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const PagedArgs px = paged_args(a, NT * BM, D);
  const long long tiles = static_cast<long long>(px.n_qt) * a.BH;
  const long long grid = tiles > a.ranges ? tiles : a.ranges;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  trace_begin(TR_FWD, st);
  e = launch_dependent(kern, static_cast<unsigned>(grid), THREADS, smem, st, a.tmQ, a.tmK, a.tmV,
                       a.O, a.L, a.N, a.group, a.cu_seqlens, a.H, a.total, a.c_log2, a.ctl, px);
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
  static constexpr int INFO_OFF = MASK_OFF + kMaskSlots * 16;   // two Pieces
  static constexpr int SMEM_BYTES = INFO_OFF + 2 * 64;
  static constexpr int TMEM_COLS = 256;
  static constexpr uint32_t S_COL = 0, P_COL = 128, O_COL = 192;
  // two CTAs per SM, each with the 1 KiB the system reserves per CTA
  static_assert(2 * (SMEM_BYTES + 1024) <= 233472, "two CTAs per SM must fit");
  static_assert(O_COL + D <= TMEM_COLS, "TMEM layout");
};

}  // namespace one

template <int D, bool BF16>
__global__ void __launch_bounds__(one::THREADS, 2)
    fwd1_paged_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, void* __restrict__ Out,
                      float* __restrict__ Lout, int N, int group, const int* cu_seqlens, int H,
                      int total, float c_log2, KernelCtl ctl, const PagedArgs px) {
  using C = Cfg<D>;
  using C1 = one::Cfg1<D>;
  constexpr int STAGES = C1::STAGES;
  extern __shared__ __align__(1024) uint8_t sg[];
  const uint32_t sb = smem_u32(sg);
  grid_dep_launch();                            // the next kernel may start setting up
  if (sb & 1023u) {                             // see FA_DEV_SMEM_ALIGN
    grid_dep_wait();
    if (threadIdx.x == 0) {
      atomicOr(ctl.status, FA_DEV_SMEM_ALIGN);
      if (px.ranges) px.hdr[0].base = 0;
    }
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

  auto info = [&](int b) -> Piece* {
    return reinterpret_cast<Piece*>(sg + C1::INFO_OFF + 64 * b);
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
      Work<1> work;
      int tile = static_cast<int>(blockIdx.x);   // in a range: >= 0 while there are pieces
      bool cuts = false;
      if (px.ranges && !work.first(px, cu_seqlens, N, H, total, cuts)) tile = -1;
      int g = 0, kq = 0, nk = 0, nv = 0;         // steps, Q tiles, K and V tiles loaded
      bool pending = false;                       // a request for the next tile is out
      int n_req = 0;                               // requests made
      for (int k = 0; ok; ++k) {
        if (!(ok = wait(bar(B_TE(k & 1)), ((k >> 1) & 1) ^ 1))) break;
        if (tile >= 0 && (k > 0 ? !cuts : !px.ranges)) work.whole(px, cu_seqlens, N, H, total, tile);
        const Piece t = work.piece(px, group);
        const int nt = t.j1 - t.j0;
        if (lead && tile >= 0) *info(k & 1) = t;
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
        if (nt <= 0 && !cuts) request();
        if (nt > 0) {
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
          paged_fetch(px, work.b, t.kr, t.j0 * BN, lane, next);
          for (int j = 0; j < nt; ++j, ++g) {
            const int st = g % STAGES;
            const uint32_t ph = (g / STAGES) & 1;
            const int krow = (t.j0 + j) * BN;
            const PagedTile cur = next;
            if (j + 1 < nt) paged_fetch(px, work.b, t.kr, krow + BN, lane, next);
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
            if (j + 1 == nt && !cuts) request();
          }
          if (!ok) break;
        }
        if (cuts) {
          if (!work.next(px, cu_seqlens, N, H, total)) tile = -1;
          continue;
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
        const int nt = info(k & 1)->j1 - info(k & 1)->j0;
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
    if (px.ranges)
      rows_without_keys<1, D>(px, cu_seqlens, N, H, total, static_cast<uint16_t*>(Out), Lout,
                              static_cast<int>(threadIdx.x) - 64, 128);
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
      const Piece* ti = info(k & 1);
      const int lo = ti->j0, nt = ti->j1 - lo, row0 = ti->row0, Nk = ti->kr.n;
      const RowKeys rk = row_keys(ti->kr, row0 + rit, pack);
      const int grow = row0 + rit;               // query row
      // where a row lies in O, in the workspace, and in L or the workspace's L
      auto row_at = [&](int r) -> size_t {
        return static_cast<size_t>(ti->base + (r >> pack)) * H + ti->hq + (r & ((1 << pack) - 1));
      };
      auto part_at = [&](int r) -> size_t {
        return static_cast<size_t>(ti->part) * BM + (r - row0);
      };
      auto lse_at = [&](int r) -> float* {
        if (ti->part >= 0) return px.part_l + part_at(r);
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
      const bool shared = ti->part >= 0;
      const bool none = l_run == 0.f;            // a row whose keys are all masked
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
      // O = 0 as in the d = 128 kernel, over what was staged: choosing each word costs the rows with
      // keys more here (1 x 8192, d = 64: 284.3 against 283.0 us; there 336.4 against 338.7)
      if (none && !shared)
        for (int i = 0; i < CPR; ++i) stage[lane * CPR + i] = make_uint4(0u, 0u, 0u, 0u);
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
  const PagedArgs px = paged_args(a, BM, D);
  const long long tiles = static_cast<long long>(px.n_qt) * a.BH;
  const long long grid = tiles > a.ranges ? tiles : a.ranges;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  trace_begin(TR_FWD, st);
  e = launch_dependent(kern, static_cast<unsigned>(grid), one::THREADS, smem, st, a.tmQ,
                       a.tmK, a.tmV, a.O, a.L, a.N, a.group, a.cu_seqlens, a.H, a.total,
                       a.c_log2, a.ctl, px);
  trace_end(TR_FWD, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Joins the pieces of a query tile cut by range borders, a warp per row: the CTAs of range x
// take part for the tile that it shares with range x - 1.
constexpr int MERGE_THREADS = 128;
template <int D, bool BF16, int TILES>
__global__ void __launch_bounds__(MERGE_THREADS)
    fwd_paged_merge_kernel(void* Out, float* Lout, int H, int total, const PagedArgs px) {
  constexpr int ROWS = TILES * BM, WARPS = MERGE_THREADS / 32;
  grid_dep_wait();                               // the pieces' results
  const int cut = px.hdr[0].base;
  const RangeHeader hd = px.hdr[blockIdx.x];
  if (cut == 0 || hd.rows == 0) return;          // not cut: the other headers are not written
  const int lane = threadIdx.x & 31, n_sl = hd.c1 - hd.c0, used = n_sl + 1;
  const int first = ((static_cast<int>(blockIdx.x) - hd.c0 - 1) * static_cast<int>(gridDim.y) +
                     static_cast<int>(blockIdx.y)) * WARPS + (static_cast<int>(threadIdx.x) >> 5);
  // piece s of row r: the first one is the second of its range, the others the first
  auto at = [&](int s, int r) -> size_t {
    return (2 * static_cast<size_t>(hd.c0 + s) + (s == 0)) * ROWS + r;
  };
  for (int r = first; r < hd.rows; r += n_sl * static_cast<int>(gridDim.y) * WARPS) {
    float l_max = -INFINITY;
    for (int s = lane; s < used; s += 32) l_max = fmaxf(l_max, px.part_l[at(s, r)]);
#pragma unroll
    for (int w = 16; w >= 1; w /= 2) l_max = fmaxf(l_max, __shfl_xor_sync(0xffffffffu, l_max, w));
    // weights of 32 ranges at a time, one per lane; their rows in batches of 8 loads that do not
    // wait for one another (a range without keys has weight 0 and left nothing to read)
    constexpr int E = D / 32;
    float sum = 0.f, acc[E] = {};
    for (int s0 = 0; s0 < used; s0 += 32) {
      const float ls = s0 + lane < used ? px.part_l[at(s0 + lane, r)] : -INFINITY;
      const float wl = ls == -INFINITY ? 0.f : ex2((ls - l_max) * 1.4426950408889634f);
      sum += wl;
      for (int k0 = 0; k0 < min(32, used - s0); k0 += 8) {
        float v[8][E], w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          w[k] = __shfl_sync(0xffffffffu, wl, k0 + k);
          const float* src = px.part + at(s0 + k0 + k, r) * D + lane * E;
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
    const int row = hd.row0 + r, h = hd.hq + (row & ((1 << px.pack) - 1));
    const size_t tok = static_cast<size_t>(hd.base + (row >> px.pack));
    T* dst = static_cast<T*>(Out) + (tok * H + h) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float y = acc[e] * inv * px.o_scale;   // pieces of codes: v_scale is still to come
      if constexpr (BF16) dst[e] = __float2bfloat16_rn(y);
      else dst[e] = __float2half_rn(y);
    }
    if (lane == 0)
      Lout[static_cast<size_t>(h) * total + tok] =
          sum == 0.f ? -INFINITY : l_max + log2f(sum) * 0.69314718055994531f;
  }
}

template <int D, bool BF16, bool C8>
cudaError_t launch_fwd_paged_t(const FwdArgs& a, cudaStream_t st) {
  cudaError_t e;
  if constexpr (D == 128)
    // the weights' sum is below 2^46 (2^30 keys, at most 2^15 each): 2^-64 over it is a normal number
    e = a.ranges ? launch_fwd_paged2_t<D, BF16, true, C8, C8>(a, st)
        : C8 && !(a.o_scale >= 0x1p-64f && a.o_scale <= 0x1p64f)
            ? launch_fwd_paged2_t<D, BF16, false, C8, C8>(a, st)
            : launch_fwd_paged2_t<D, BF16, false, C8, false>(a, st);
  else e = launch_fwd_paged1_t<D, BF16>(a, st);
  if (e != cudaSuccess || !a.ranges) return e;
  constexpr int TILES = D == 128 ? NT : 1, ROWS = TILES * BM;
  const long long rows = static_cast<long long>(a.N) << a.pack;
  // CTAs per range: a warp for four of a query tile's rows
  const unsigned y = static_cast<unsigned>(((rows < ROWS ? rows : ROWS) + 15) / 16);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.ranges), y);
  cfg.blockDim = dim3(MERGE_THREADS);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fwd_paged_merge_kernel<D, BF16, TILES>, a.O, a.L, a.H, a.total,
                            paged_args(a, ROWS, D));
}

template <bool BF16>
cudaError_t launch_fwd_paged_b(const FwdArgs& a, int d, bool c8, cudaStream_t st) {
  if (c8) return d == 128 ? launch_fwd_paged_t<128, BF16, true>(a, st) : cudaErrorInvalidValue;
  if (d == 32) return launch_fwd_paged_t<32, BF16, false>(a, st);
  if (d == 64) return launch_fwd_paged_t<64, BF16, false>(a, st);
  if (d == 128) return launch_fwd_paged_t<128, BF16, false>(a, st);
  return cudaErrorInvalidValue;
}

}  // namespace

int fwd_paged_pack(int group) {
  int p = 0;
  while (p < 7 && group % (2 << p) == 0) ++p;
  return p;
}

// Which calls may cut: those whose tiles the GPU runs at once (152 SMs; two CTAs each at
// d <= 64), or in up to four rounds where a tile holds all rows of a sequence: more tiles, or
// those of long prompts, of which the short ones come last, even out by themselves (2 x 2048
// tokens on 8192 keys, 512 tiles: 337 whole, 342 us cut).  Whether they do the device decides by
// the lengths (Work::first).
FwdPagedPlan fwd_paged_plan(int B, int H, int Hkv, int max_seqlen, int d) {
  const int pack = fwd_paged_pack(H / Hkv), rows = d == 128 ? NT * BM : BM;
  const int slots = d == 128 ? 152 : 304;
  const long long n_qt = ((static_cast<long long>(max_seqlen) << pack) + rows - 1) / rows;
  const long long r = static_cast<long long>(max_seqlen) << pack;
  FwdPagedPlan p = {static_cast<long long>(B) * (H >> pack) * n_qt, 0,
                    static_cast<int>(r < rows ? r : rows), 0};
  if (p.tiles > (n_qt == 1 ? 4 : 1) * slots) return p;
  p.ranges = slots;
  p.ws_bytes = hdr_bytes(slots) + 2 * sizeof(float) * slots * rows * (d + 1);
  return p;
}

// Not where the longest tile possible is too short, nor where the lengths may not add up in 32 bits.
bool fwd_paged_may_cut(const FwdPagedPlan& p, long long keys) {
  const long long most = (keys + BN - 1) / BN + kTileCost;
  return p.ranges > 0 && p.tiles * most <= 0x7fffffffLL &&
         cut_saves(p.tiles, p.ranges, static_cast<int>(most), 0) > join_cost(p.rows);
}

cudaError_t launch_fwd_paged(const FwdArgs& args, int d, bool bf16, bool c8, bool causal,
                             cudaStream_t st) {
  FwdArgs a = args;
  a.causal = causal;
  a.BH = a.B * (a.H >> a.pack);
  return bf16 ? launch_fwd_paged_b<true>(a, d, c8, st) : launch_fwd_paged_b<false>(a, d, c8, st);
}

}  // namespace fa
