// fa_internal.h -- host-side interface between the C ABI (fa_api.cu) and the
// kernel launchers (fa_fwd.cu, fa_bwd.cu).  Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <mutex>

#include "fa_ptx.cuh"

namespace fa {

// Kernel kinds for the optional per-kernel CUDA-event trace (fa_trace_* in fa.h).
enum TraceKind {
  TR_FWD = 0,
  TR_BWD_PRE = 1,
  TR_BWD_DKDV = 2,
  TR_BWD_DQ = 3,
  TR_DEC_SPLIT = 4,
  TR_DEC_MERGE = 5,
  TR_FWD8 = 6,
  TR_NKINDS = 7
};
// Record an event before / after one kernel launch on `st` (no-op unless tracing).
void trace_begin(int kind, cudaStream_t st);
void trace_end(int kind, cudaStream_t st);

// Launch `kern` with programmatic stream serialisation: its CTAs may be scheduled
// while the previous kernel in `st` finishes its last wave, so launch latency and the
// kernel's set-up overlap that kernel's tail.  The kernel must call grid_dep_wait()
// before its first access to global memory that earlier work in the stream writes or
// reads (fa_ptx.cuh).
template <typename... KArgs, typename... Args>
inline cudaError_t launch_dependent(void (*kern)(KArgs...), unsigned grid, unsigned block,
                                    size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// Heads per ordering group (block_pos) of a persistent kernel whose work items stream
// `bytes_per_head` bytes of one head's tiles: all heads (the whole grid longest-first)
// when they fit in about half of L2 together, else as many as do, at least 8.
inline int order_group(long long heads, long long bytes_per_head) {
  const long long budget = 64ll << 20;
  long long g = bytes_per_head > 0 ? budget / bytes_per_head : heads;
  if (g < 8) g = 8;
  if (g > heads) g = heads;
  return static_cast<int>(g < 1 ? 1 : g);
}

// Raise a kernel's dynamic shared-memory limit to `bytes`, once per kernel (later
// calls only look it up; launches from several host threads share the record).
inline cudaError_t ensure_smem(const void* kern, int bytes) {
  static std::mutex mu;
  static const void* seen[512];
  static int n_seen = 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < n_seen; ++i)
    if (seen[i] == kern) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && n_seen < 512) seen[n_seen++] = kern;
  return e;
}

// TMA box of one 128-row tile: box_cols elements (one swizzle width) per row.
struct FwdTileInfo {
  int box_cols;
  int box_rows;
  int swizzle_bytes;
};
FwdTileInfo fwd_tile_info(int d);

// Paged caches (fa_paged_cache in fa.h): pages of page.div rows, addressed through a table of
// max_pages ids per sequence.
struct PagedView {
  const int* table;            // device int32, rows table_stride entries apart
  const int* seqlens;          // device int32 [B]: keys per sequence
  long long table_stride;
  int pages, max_pages;        // pages in the pools, ids per sequence
  FastDiv page;                // page size
};

struct FwdArgs {
  CUtensorMap tmQ, tmK, tmV;   // 3-D maps (d, N, B*H) of Q; (d, N, B*Hkv) of K and V
  void* O;
  float* L;
  int N, BH;
  int group;                   // query heads per K/V head (H / Hkv; 1 without sharing)
  int window;                  // causal sliding window of this many keys (0: none)
  // packed variable-length sequences (NULL: dense (B, H, N, d)): device int32
  // offsets [B+1]; Q, O (total, H, d), K, V (total, H/group, d), L (H, total); N is
  // then the longest sequence
  const int* cu_seqlens;
  int H, total;
  // paged keys (launch_fwd_paged): tmK, tmV are then 4-D maps (d, page_size, Hkv, pages) with
  // boxes of 1 << box_log2 rows
  PagedView pg;
  int box_log2;
  int causal;
  int B;
  int pack;                    // log2 of the heads that share a query tile (0 elsewhere)
  int ranges;                  // CTAs that may share the KV tiles of all query tiles (0: none)
  void* ws;                    // their workspace
  float c_log2;                // scale * log2(e) (E4M3 caches: times k_scale)
  float o_scale;               // E4M3 caches: v_scale
  KernelCtl ctl;
};
cudaError_t launch_fwd(const FwdArgs& a, int d, bool bf16, bool causal, cudaStream_t st);
cudaError_t launch_fwd_paged(const FwdArgs& a, int d, bool bf16, bool c8, bool causal,
                             cudaStream_t st);
// log2 of the heads packed in a query tile of a paged call.
int fwd_paged_pack(int group);
// Query tiles of a paged call, and the CTAs that may share their KV tiles, with their workspace.
struct FwdPagedPlan {
  long long tiles;
  int ranges, rows;            // CTAs; rows of a tile that are used, at most
  size_t ws_bytes;
};
FwdPagedPlan fwd_paged_plan(int B, int H, int Hkv, int max_seqlen, int d);
// Whether they do if a row may see up to `keys` keys.
bool fwd_paged_may_cut(const FwdPagedPlan& p, long long keys);

struct BwdArgs {
  CUtensorMap tmQ, tmK, tmV, tmO, tmdO;
  const void* Q;
  const void* O;
  const void* dO;
  const float* L;
  float* Dvec;                 // workspace: rowsum(dO o O), (B*H, N) fp32
  void* dQ;
  void* dK;
  void* dV;
  int N, BH;                   // BH = B*H query heads
  int group;                   // query heads per K/V head; B*H/group K/V heads
  int window;                  // causal sliding window of this many keys (0: none)
  const int* cu_seqlens;       // packed variable-length sequences, as in FwdArgs
  int H, total;
  float scale, c_log2;
  KernelCtl ctl;
};
cudaError_t launch_bwd(const BwdArgs& a, int d, bool bf16, bool causal, cudaStream_t st);
// dK/dV and dQ kernels after the pre-pass: the TMEM-resident kernels of fa_bwd128.cu
// (every head dim) and the persistent ones of fa_bwd64.cu (head dims 32 and 64)
cudaError_t launch_dkdv128(const BwdArgs& a, int d, bool bf16, bool causal, cudaStream_t st);
cudaError_t launch_dq128(const BwdArgs& a, int d, bool bf16, bool causal, cudaStream_t st);
cudaError_t launch_dkdv64(const BwdArgs& a, int d, bool bf16, bool causal, cudaStream_t st);
cudaError_t launch_dq64(const BwdArgs& a, int d, bool bf16, bool causal, cudaStream_t st);
// Workspace: D and L*log2(e) per padded row.
size_t bwd_workspace_bytes(long long BH, int N, int d);

struct DecodeArgs {
  CUtensorMap tmK, tmV;        // 3-D maps (d, Nmax, B*Hkv) of the caches, box decode_key_rows(d) rows
  const void* Q;               // (B, H, d) one query row per head
  const int* seqlens;          // device int32 [B]: cached keys per sequence
  void* O;                     // (B, H, d)
  float* L;                    // (B, H) fp32, natural log
  float* part;                 // workspace: (B*H, n_splits, d+4) partial states
  int B, H, Hkv, Nmax;
  int n_splits, chunk;         // splits of the cache and keys per split
  float c_log2;                // scale * log2(e) (E4M3 caches: times k_scale)
  float o_scale;               // 1 (E4M3 caches: v_scale)
  KernelCtl ctl;
};
// Query rows that one decode CTA serves from each K/V row (a power of two dividing H/Hkv).
int decode_rows(int H, int Hkv);
// Keys per ring stage of the decode kernel (the TMA box height); c8: E4M3 caches.
int decode_key_rows(int d, bool c8);
// Splits and keys per split (written to *chunk) for caches of Nmax keys.
int decode_parts(int B, int H, int Hkv, int Nmax, int* chunk);
cudaError_t launch_decode(const DecodeArgs& a, int d, bool bf16, bool c8, cudaStream_t st);

// Appending new tokens' keys and values, rotated on the way; queries rotated beside them.
struct AppendArgs {
  const void* K;               // (T, Hkv, d), tokens k_stride elements apart; V and Q likewise
  const void* V;
  const void* Q;               // NULL: keys and values only
  void* Qout;                  // (T, H, d)
  void* Kc;                    // pools, element (page, head, row, c) at the strides below
  void* Vc;
  const int* cu;               // device int32 [B+1]: new tokens of each sequence (NULL: one each)
  const int* positions;        // device int32 [T]: angle positions (NULL: key positions)
  const float* cos_sin;        // (max_pos, rot): cos then sin of each pair's angle
  long long k_stride, v_stride, q_stride;
  long long page_stride, head_stride, row_stride;
  int B, T, H, Hkv, rot, max_pos;
  float k_inv, v_inv;          // E4M3 caches: 1 / descale factors
  PagedView pg;
  KernelCtl ctl;
};
cudaError_t launch_append(const AppendArgs& a, int d, bool bf16, bool c8, bool interleaved,
                          cudaStream_t st);

// Heads of a (batch, heads, rows, d) tensor, columns contiguous; strides in elements.
struct HeadView {
  void* data;
  long long batch_stride, head_stride, row_stride;
  int heads;
  bool zero_rest;              // of an output: rows that are left out get zeros
};
// Norms of query ([0]) and key ([1]) heads and their rotation, the gradient of both, or appending
// them and values ([2]) to a paged cache.
struct NormRopeArgs {
  HeadView x[3], y[3], dy[2];  // inputs; outputs (backward: dx; appending: queries, then the pools with
                               // their head strides); backward: gradients of the outputs
  const void* w[2];            // norm weights (d), fp32 or of the inputs' type; NULL: ones
  float* dw[2];                // their gradients, or NULL
  const int* cu;               // device int32 [n_seq + 1]: packed sequences (one batch entry), or NULL
  const int* positions;        // rows of the angles' table, batch entries pos_stride apart, or NULL
  const float* cos_sin;        // (max_pos, rot): cos then sin of each pair's angle
  float* part;                 // workspace: the CTAs' sums of dw
  long long pos_stride;
  FastDiv rows;                // rows of a batch entry
  int T, n_seq, rot, max_pos;  // T: rows of all batch entries
  bool norm, w_fp32;
  float eps, sin_sign;         // sin_sign -1: the rotation's transpose
  PagedView pg;                // appending, as in AppendArgs
  long long page_stride, row_stride;
  float k_inv, v_inv;
  FastDiv heads[3];            // set by the launch
  int blocks[3], chunk[3];
  KernelCtl ctl;
};
size_t norm_rope_bwd_ws_bytes(int d);
enum class NormRopeOp { Forward, Backward, Append, Append8 };
cudaError_t launch_norm_rope(const NormRopeArgs& a, int d, bool bf16, bool interleaved,
                             NormRopeOp op, cudaStream_t st);

// One query row per (sequence, head) over a paged cache.
struct DecodePagedArgs {
  CUtensorMap tmK, tmV;        // 4-D maps (d, page_size, Hkv, pages), box 1 << box_log2 rows
  const void* Q;               // (B, H, d)
  void* O;
  float* L;
  void* ws;                    // headers and partial states (decode_paged_ws_bytes)
  int B, H, Hkv, window;       // window 0: every key
  int box_log2;
  float c_log2, o_scale;       // scale * log2(e) (E4M3: times k_scale); 1 (E4M3: v_scale)
  PagedView pg;
  KernelCtl ctl;
};
// Keys per ring stage of one warp: what the TMA box's height has to divide.
int decode_paged_keys(int d, bool c8);
// Cost of one sequence of n keys as the split counts it (an upper bound for windows).
long long decode_paged_cost(int Hkv, int d, bool c8, long long n);
// Whether a group of H / Hkv heads fits the grid.
bool decode_paged_group_fits(int H, int Hkv);
size_t decode_paged_ws_bytes(int H, int Hkv, int d);
// Whether a call's ranges may cut rows, so that it touches its workspace.
bool decode_paged_cuts_rows(const DecodePagedArgs& a, int d, bool c8);
cudaError_t launch_decode_paged(const DecodePagedArgs& a, int d, bool bf16, bool c8,
                                cudaStream_t st);

// Forward on 8-bit E4M3 inputs, d = 128, dense (B, H, N, 128) layout.
struct Fwd8Args {
  CUtensorMap tmQ, tmK;        // 3-D byte maps (128, N, B*H) / (128, N, B*Hkv), box 128 x 128
  CUtensorMap tmVt;            // 3-D byte map (N, 128, B*Hkv) of V^T, box 128 x 128
  void* O;                     // (B, H, N, 128) bf16
  float* L;                    // (B, H, N) fp32
  int N, BH, group;
  float c_log2;                // scale * q_scale * k_scale * log2(e)
  float o_scale;               // v_scale
  KernelCtl ctl;
};
cudaError_t launch_fwd8(const Fwd8Args& a, bool causal, cudaStream_t st);
// E4M3 codes of x * inv_scale for `mats` row-major rows x cols matrices of 16-bit
// values, optionally transposing each matrix.
cudaError_t launch_quant8(const void* X, void* Y, long long mats, int rows, int cols,
                          float inv_scale, bool transpose, bool bf16, cudaStream_t st);

}  // namespace fa
