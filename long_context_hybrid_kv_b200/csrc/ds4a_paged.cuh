// Decode attention over a paged K=V cache: the arguments and the work
// schedule that the attention and the joining kernels share.
//
// One query per sequence.  Sequence b at position p has closed (p + 1) / m
// entries; drop[b] of them have been evicted, the others lie in the slots
// 0 .. n - 1 of its pages.  Its keys are those slots (or the listed ones)
// and then the window rows.
//
// Work is counted in tiles of kt keys.  The tiles of all items (sequence,
// group of hn heads) stand in one row, item after item, and block c of G
// takes the tiles [c total / G, (c + 1) total / G): every block gets the same
// number of tiles (give or take one) whatever the lengths are, and the host
// needs to know none of them, so a captured launch serves growing sequences.
// A block's piece of an item is a segment; an item that one block holds
// whole is finished there, the others are joined from their segments.
#pragma once

#include "ds4a_internal.cuh"
#include "ds4a_mx.cuh"

namespace ds4a {

struct PagedArgs {
  int B, H, D, R, W, m, k, cap, sparse;
  float scale, eps;
  // cache
  const uint8_t* pages;
  int fmt, row_bytes;  // 0: bf16 rows of D; 1: DS4A_MX_KV_FP8 rows
  int n_pages, page_size;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* drop;  // nullable
  // query side
  const int32_t* q_pos;
  const uint16_t* q;
  const float* q_norm_g;
  const int32_t* idx;
  const uint16_t* win;
  int win_cap;
  int64_t win_bstride;
  const float* sink;
  uint16_t* out;
  uint16_t* weights;  // nullable: bf16 [B][w_stride], slots below w_len
  int64_t w_stride;
  int w_len;
  // schedule and workspace
  int hn, hgroups, kt, G;
  int32_t* first;   // [B hgroups + 1] tiles before each item
  float* part;      // [2 G][2 hn + hn D] segments: max (natural log), sum, accumulator
  float* whole_ml;  // [B hgroups][2 hn] max and sum of items that one block holds (weights only)
  float* tile_ref;  // [tiles][hn] reference of each tile's probabilities, log2 (weights only)
  uint16_t* tile_p; // [tiles][kt][hn] probabilities against it, bf16 (weights only)
  unsigned int* err;
  RopeTheta rope;
};

// Entries in the cache of sequence b (0 at a negative position).
__device__ __forceinline__ int paged_entries(const PagedArgs& a, int b, int pos) {
  if (pos < 0) return 0;
  const int gone = a.drop ? a.drop[b] : 0;
  // (pos + 1) / m without leaving 32 bits at the largest position
  const int closed = (int)(((int64_t)pos + 1) / a.m);
  return max(0, min(closed - gone, a.cap));
}

// Key slots of a sequence: the cache's (all, or the listed ones, of which at
// most n can be distinct), then the window's.
struct PagedSeq {
  int pos, n, n_sel, win_start, n_keys;
};
__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
  PagedSeq s;
  s.pos = a.q_pos[b];
  s.n = paged_entries(a, b, s.pos);
  s.n_sel = a.sparse ? min(a.k, s.n) : s.n;
  s.win_start = max(0, s.pos - a.W + 1);
  s.n_keys = s.pos < 0 ? 0 : s.n_sel + (a.W > 0 ? s.pos - s.win_start + 1 : 0);
  return s;
}

// Row of key j of sequence b: its address, whether it is an FP8 row, or
// nullptr (an unused or bad index, a bad page: recorded).
__device__ __forceinline__ const uint8_t* paged_key(const PagedArgs& a, int b, const PagedSeq& s, int j, bool* fp8) {
  *fp8 = false;
  if (j < s.n_sel) {
    int e = j;
    if (a.sparse) {
      e = a.idx[(int64_t)b * a.k + j];
      if (e == -1) return nullptr;
      if (e < 0 || e >= s.n) {
        raise_err(a.err, DS4A_DEV_BAD_INDEX);
        return nullptr;
      }
    }
    const int pg = e / a.page_size;
    const int ph = a.table[(int64_t)b * a.table_stride + pg];
    if (ph < 0 || ph >= a.n_pages) {
      raise_err(a.err, DS4A_DEV_BAD_INDEX);
      return nullptr;
    }
    *fp8 = a.fmt != 0;
    return a.pages + ((int64_t)ph * a.page_size + (e - pg * a.page_size)) * a.row_bytes;
  }
  const int p = s.win_start + (j - s.n_sel);
  return reinterpret_cast<const uint8_t*>(a.win + (int64_t)b * a.win_bstride + (int64_t)(p % a.win_cap) * a.D);
}

__device__ __forceinline__ int paged_tiles(const PagedArgs& a, const PagedSeq& s) { return (s.n_keys + a.kt - 1) / a.kt; }

// The blocks that take part (with fewer tiles than blocks, one a tile), the
// first tile of block c, and the block that holds tile t.
__device__ __forceinline__ int paged_start(int c, int total, int G) {
  const int g = min(G, total);
  return c >= g ? total : (int)((int64_t)c * total / g);
}
__device__ __forceinline__ int paged_block_of(int t, int total, int G) {
  return (int)((((int64_t)t + 1) * min(G, total) - 1) / total);
}

// A block's place in the schedule, found by one warp (all 32 lanes): the
// tiles before every item are summed 32 sequences at a time.  Block 0 also
// writes them down for the joining kernel.
struct PagedRange {
  int total, t0, t1;  // this block's tiles
  int item, item_t0;  // the item of tile t0 and the tiles before it
};
__device__ __forceinline__ PagedRange paged_range(const PagedArgs& a, int c) {
  const int lane = threadIdx.x & 31;
  PagedRange r;
  int total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int b = b0 + lane;
    int v = 0;
    if (b < a.B) {
      const PagedSeq s = paged_seq(a, b);
      if (s.pos < 0 && c == 0) raise_err(a.err, DS4A_DEV_BAD_POS);
      v = paged_tiles(a, s) * a.hgroups;
    }
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (c == 0 && b < a.B)
      for (int g = 0; g < a.hgroups; ++g) a.first[b * a.hgroups + g] = total + inc - v + v / a.hgroups * g;
    total += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (c == 0 && lane == 0) a.first[a.B * a.hgroups] = total;
  r.total = total;
  r.t0 = paged_start(c, total, a.G);
  r.t1 = paged_start(c + 1, total, a.G);
  r.item = a.B * a.hgroups;
  r.item_t0 = total;
  int before = 0;
  for (int b0 = 0; b0 < a.B && r.t0 < r.t1; b0 += 32) {
    const int b = b0 + lane;
    const int v = b < a.B ? paged_tiles(a, paged_seq(a, b)) * a.hgroups : 0;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const unsigned int here = __ballot_sync(0xffffffffu, before + inc > r.t0);
    if (here) {
      const int l = __ffs(here) - 1;
      const int v_l = __shfl_sync(0xffffffffu, v, l), inc_l = __shfl_sync(0xffffffffu, inc, l);
      const int per = v_l / a.hgroups, b_t0 = before + inc_l - v_l;
      const int g = (r.t0 - b_t0) / per;
      r.item = (b0 + l) * a.hgroups + g;
      r.item_t0 = b_t0 + g * per;
      break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return r;
}

// head group, tile and grid of the two kernels
void paged_shape_generic(PagedArgs* a);
void paged_shape_tc(PagedArgs* a);
bool paged_tc_supported(const PagedArgs& a, int fmt);
cudaError_t launch_paged_attend_generic(const PagedArgs& a, cudaStream_t s);
cudaError_t launch_paged_attend_tc(const PagedArgs& a, cudaStream_t s);
cudaError_t launch_paged_join(const PagedArgs& a, cudaStream_t s);

}  // namespace ds4a
