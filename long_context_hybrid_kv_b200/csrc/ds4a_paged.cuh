// Decode attention over a paged K=V cache: the arguments and the work
// schedule that the attention and the joining kernels share.
//
// One query per sequence.  Sequence b at position p has closed (p + 1) / m
// entries; drop[b] of them have been evicted, the others lie in the slots
// 0 .. n - 1 of its pages.  Its keys are those slots (or the listed ones)
// and then the window rows.
//
// Work is counted in tiles of kt keys.  The tiles of all items (sequence,
// group of hn heads) stand in one row, item after item, and are cut into as
// many equal ranges as there are blocks, so that every block gets the same
// number of tiles (give or take one) whatever the lengths are, and the host
// needs to know none of them: a captured launch serves growing sequences.
// A block's piece of an item is a segment; an item that one block holds whole
// is finished there, the others are joined from their segments.  As a segment
// costs its block a float accumulator written (128 KiB for 64 heads x 512) and
// the joining kernel one read, a cut that would fall into a short item moves
// to its nearer end, and a block gets at least two tiles.
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
  int32_t* total;    // tiles of all items
  int4* cut;         // [G] the item that begins in the block and is cut: item or -1, its last block, its slot
  float* part;       // [2 G][2 hn + hn D] segments: max (natural log), sum, accumulator
  float* lse2;       // [items][hn] log2 of the softmax denominator (weights only)
  int2* tile_of;     // [tiles] item, tile within it (weights only)
  float* tile_ref;   // [tiles][hn] reference of each tile's probabilities, log2 (weights only)
  uint16_t* tile_p;  // [tiles][kt][hn] probabilities against it, bf16 (weights only)
  int p_swizzled;    // 16-byte piece c of a key's row of tile_p lies at c ^ (key % 8)
  unsigned int* err;
  RopeTheta rope;
};

// Entries in the cache of sequence b (0 at a negative position).
__device__ __forceinline__ int paged_entries(const PagedArgs& a, int b, int pos) {
  if (pos < 0) return 0;
  const int gone = a.drop ? a.drop[b] : 0;
  const int closed = (int)(((unsigned)pos + 1u) / (unsigned)a.m);
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

// (kt: a.kt, as a constant where the caller has one)
__device__ __forceinline__ int paged_tiles(const PagedSeq& s, int kt) { return (int)((unsigned)(s.n_keys + kt - 1) / (unsigned)kt); }
__device__ __forceinline__ int paged_item_seq(const PagedArgs& a, int item) {
  return a.hgroups == 1 ? item : item / a.hgroups;
}

// Items of at most this many tiles are not cut.
constexpr int kPagedWhole = 4;

// The blocks that take part, where block c's range begins before its ends
// are moved, and the block that holds tile t.
__device__ __forceinline__ int paged_blocks(int total, int G) { return min(G, (total + 1) / 2); }
__device__ __forceinline__ int paged_start(int c, int total, int ge) {
  const unsigned q = (unsigned)total / (unsigned)ge, rem = (unsigned)total - q * (unsigned)ge;
  return c >= ge ? total : (int)((unsigned)c * q + min((unsigned)c, rem));
}
__device__ __forceinline__ int paged_block_of(int t, int total, int ge) {
  const unsigned q = (unsigned)total / (unsigned)ge, rem = (unsigned)total - q * (unsigned)ge, wide = rem * (q + 1);
  return (unsigned)t < wide ? (int)((unsigned)t / (q + 1)) : (int)(rem + ((unsigned)t - wide) / q);
}

// A block's place in the schedule, found by one warp (all 32 lanes): the
// tiles before every item are summed 32 sequences at a time.
struct PagedRange {
  int total, ge, raw0;  // tiles of all items, blocks that take part, start before moving
  int t0, t1;           // this block's tiles
  int item, item_t0;    // the item of tile t0 and the tiles before it
};
__device__ __forceinline__ PagedRange paged_range(const PagedArgs& a, int c, int kt) {
  const int lane = threadIdx.x & 31;
  auto tiles_at = [&](int b0) {
    const int b = b0 + lane;
    if (b >= a.B) return 0;
    const PagedSeq s = paged_seq(a, b);
    if (s.pos < 0 && c == 0) raise_err(a.err, DS4A_DEV_BAD_POS);
    return paged_tiles(s, kt) * a.hgroups;
  };
  auto scan = [&](int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    return v;
  };
  PagedRange r;
  int v = 0, inc = 0, total = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    v = tiles_at(b0);
    inc = scan(v);
    total += __shfl_sync(0xffffffffu, inc, 31);
  }
  r.total = total;
  r.ge = max(1, paged_blocks(total, a.G));
  r.raw0 = paged_start(c, total, r.ge);
  r.t0 = r.raw0;
  r.t1 = paged_start(c + 1, total, r.ge);
  r.item = a.B * a.hgroups;
  r.item_t0 = total;
  if (r.t0 >= r.t1) return r;
  // an end that lies in a short item moves to the nearer end of it
  int before = 0, found = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B && found < 2; b0 += 32) {
    if (a.B > 32) {
      v = tiles_at(b0);
      inc = scan(v);
    }
    const int upto = before + __shfl_sync(0xffffffffu, inc, 31);
#pragma unroll 1
    while (found < 2) {
      const int t = found == 0 ? r.raw0 : r.t1;
      if (t >= upto) break;  // (t = total: not found, not moved)
      const int l = __ffs(__ballot_sync(0xffffffffu, before + inc > t)) - 1;
      const int v_l = __shfl_sync(0xffffffffu, v, l), inc_l = __shfl_sync(0xffffffffu, inc, l);
      const int n = paged_item_seq(a, v_l), b_t0 = before + inc_l - v_l, g = a.hgroups == 1 ? 0 : (t - b_t0) / n;
      const int i_t0 = b_t0 + g * n;
      const int to = n > kPagedWhole ? t : 2 * (t - i_t0) < n ? i_t0 : i_t0 + n;
      if (found == 0) {
        r.t0 = to;
        r.item = (b0 + l) * a.hgroups + g + (to == i_t0 + n ? 1 : 0);
        r.item_t0 = to == i_t0 + n ? to : i_t0;
      } else {
        r.t1 = to;
      }
      ++found;
    }
    before = upto;
  }
  return r;
}

// The segments of a block one after the other.
struct PagedWalk {
  int t, t1, item, item_t0, raw0, total, ge;
  __device__ __forceinline__ explicit PagedWalk(const PagedRange& r)
      : t(r.t0), t1(r.t1), item(r.item), item_t0(r.item_t0), raw0(r.raw0), total(r.total), ge(r.ge) {}
};
struct PagedSegment {
  int item, b, g;
  int t, tile0, n_tiles;  // first tile in the row of all tiles and in the item; how many
  bool whole;
  int slot;      // of a partial result: 0 if the item began in an earlier block, else 1
  int cut_last;  // the item's last block if it begins here and goes on, else -1
  PagedSeq seq;
};
__device__ __forceinline__ bool paged_next(const PagedArgs& a, PagedWalk& w, PagedSegment& s, int kt) {
  while (w.t < w.t1) {
    s.item = w.item;
    s.b = paged_item_seq(a, w.item);
    s.g = w.item - s.b * a.hgroups;
    s.seq = paged_seq(a, s.b);
    const int n = paged_tiles(s.seq, kt), end = w.item_t0 + n;
    if (w.t >= end) {  // no tiles
      w.item_t0 = end;
      ++w.item;
      continue;
    }
    const int stop = min(w.t1, end);
    s.t = w.t;
    s.tile0 = w.t - w.item_t0;
    s.n_tiles = stop - w.t;
    s.whole = s.n_tiles == n;
    s.slot = w.item_t0 > w.raw0 ? 1 : 0;
    s.cut_last = s.tile0 == 0 && !s.whole ? paged_block_of(end - 1, w.total, w.ge) : -1;
    w.t = stop;
    w.item_t0 = end;
    ++w.item;
    return true;
  }
  return false;
}
__device__ __forceinline__ float* paged_part(const PagedArgs& a, int c, int slot) {
  return a.part + (int64_t)(2 * c + slot) * (2 * a.hn + (int64_t)a.hn * a.D);
}

// head group, tile and grid of the two kernels
void paged_shape_generic(PagedArgs* a);
void paged_shape_tc(PagedArgs* a);
bool paged_tc_supported(const PagedArgs& a, int fmt);
cudaError_t launch_paged_attend_generic(const PagedArgs& a, cudaStream_t s);
cudaError_t launch_paged_attend_tc(const PagedArgs& a, cudaStream_t s);
// tiles: at most that many
cudaError_t launch_paged_join(const PagedArgs& a, int tiles, cudaStream_t s);

}  // namespace ds4a
