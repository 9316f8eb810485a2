// Decode attention over a paged K=V cache: the arguments and the work
// schedule that the attention and the joining kernels share.
//
// One query per sequence.  Sequence b at position p has closed (p + 1) / m
// entries; drop[b] of them have been evicted, the others lie in the slots
// 0 .. n - 1 of its pages.  Its keys are those slots (or the listed ones)
// and then the window rows.
//
// Work is counted in tiles of kt keys; an item is a sequence and a group of hn
// heads.  The host knows no length, so a captured launch serves growing
// sequences: every block of the attention finds its own place.
//   Up to as many items as blocks: the shortest T for which the blocks do when
//   an item of n tiles is cut into ceil(n / T) equal pieces, a block each, and
//   items of up to T / 2 tiles share blocks, whole, each counted six tiles
//   longer: that is about what a segment costs besides its tiles (its q^, the
//   filling of the pipeline, the output), and why pieces a little longer than
//   the average beat equal shares.  A piece costs, on top, a float accumulator
//   written (128 KiB for 64 heads x 512) and read by the joining kernel.
//   More items: whole items share the blocks in the same way, if the longest
//   block that this makes is no longer than with the third way:
//   The tiles of all items stand in one row, cut into equal ranges (a cut that
//   would fall into a short item moves to its nearer end).  This is also for
//   lengths with which T would exceed the average by more than a segment costs.
// A block's piece of an item is a segment; an item that one block holds whole
// is finished there, the others are joined from their segments.
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
  int4* cut;         // [G] the item that begins in the block and is cut: item or -1, its last block, its slot
  float* part;       // [2 G][2 hn + hn D] segments: max (natural log), sum, accumulator
  float* lse2;       // [items][hn] log2 of the softmax denominator, +inf if no key counts (weights only)
  int item_tiles;    // at most that many tiles an item
  float* tile_ref;   // [items][item_tiles][hn] reference of each tile's probabilities, log2 (weights only)
  uint16_t* tile_p;  // [items][item_tiles][kt][hn] probabilities against it (weights only), bf16: half the
                     // bytes, and their sum over the heads, which averages the roundings, goes out as bf16;
                     // of the tensor-core kernel the 16-byte piece c of a key's row at c ^ (key % 8)
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

// Items of at most this many tiles are not cut, and no piece is shorter.
constexpr int kPagedWhole = 4, kPagedLeast = 2;
constexpr int kPagedCost = 6;  // of a segment besides its tiles, in tiles (a second segment takes 7 to 8 us, four tiles; 4 to 6 measure alike)
constexpr int kPagedJoin = 4;  // of the joining, in tiles

// Where piece j of an item of n tiles in p equal pieces begins: floor(j n / p)
// for j <= p, by quotient and remainder, since 296 pieces of 2^25 tiles pass 32
// bits (j rem < p^2 does not).
__host__ __device__ constexpr int paged_piece(int j, int n, int p) {
  const unsigned q = (unsigned)n / (unsigned)p, rem = (unsigned)n - q * (unsigned)p;
  return (int)((unsigned)j * q + (unsigned)j * rem / (unsigned)p);
}

// More items than blocks: the blocks that take part, where block c's range
// begins before its ends are moved, and the block that holds tile t.
__device__ __forceinline__ int paged_blocks(int total, int G) { return min(G, (total + 1) / 2); }
__device__ __forceinline__ int paged_start(int c, int total, int ge) {
  const unsigned q = (unsigned)total / (unsigned)ge, rem = (unsigned)total - q * (unsigned)ge;
  return c >= ge ? total : (int)((unsigned)c * q + min((unsigned)c, rem));
}
__device__ __forceinline__ int paged_block_of(int t, int total, int ge) {
  const unsigned q = (unsigned)total / (unsigned)ge, rem = (unsigned)total - q * (unsigned)ge, wide = rem * (q + 1);
  return (unsigned)t < wide ? (int)((unsigned)t / (q + 1)) : (int)(rem + ((unsigned)t - wide) / q);
}

// A block's place in the schedule.
struct PagedRange {
  int kind;           // 0: a piece of an item, 1: whole items that share the block, 2: a range of the row of all tiles
  int item;           // the first
  int t0, t1;         // 0: tiles of the item.  2: tiles of the row
  int last;           // 0: the item's last block
  int T, stop, done;  // 1: items above T / 2 are left out; twice the cost at which to stop, cost before the first
  int item_t0, raw0, total, ge;  // 2: tiles before the first item, start before moving, tiles and blocks in all
};

// Found by the whole block, the result valid in its warp 0.  s_n: room for
// `staged` lengths (at least the number of blocks), s_fit: 32 ints.  It stands
// before the first product of every launch, so it is short: all lengths are
// fetched at once, T is searched by up to 16 warps side by side, and no loop
// is unrolled (at a first pass instructions cost more than their work).
__device__ __forceinline__ PagedRange paged_range(const PagedArgs& a, int c, int kt, int* s_n, int staged, int* s_fit) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, hg = a.hgroups, items = a.B * hg;
  auto tiles_of = [&](int b) {
    const PagedSeq s = paged_seq(a, b);
    if (s.pos < 0 && c == 0) raise_err(a.err, DS4A_DEV_BAD_POS);
    return paged_tiles(s, kt);
  };
#pragma unroll 1
  for (int b = tid; b < min(a.B, staged); b += blockDim.x) s_n[b] = tiles_of(b);
  __syncthreads();
  auto tiles_at = [&](int b0) {  // of sequence b0 + lane
    const int b = b0 + lane;
    return b >= a.B ? 0 : b < staged ? s_n[b] : tiles_of(b);
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
  r.kind = 1;
  r.item = items;  // nothing to do
  r.t0 = r.t1 = r.last = r.T = r.stop = r.done = r.item_t0 = r.raw0 = r.total = r.ge = 0;
  if (items > a.G && warp > 0) return r;
  int total = 0, most = 0, some = 0;  // tiles, the longest item's, items that have any
#pragma unroll 1
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int v = tiles_at(b0);
    total += v;
    most = max(most, v);
    some += v > 0;
  }
  total = __reduce_add_sync(0xffffffffu, total) * hg;
  some = __reduce_add_sync(0xffffffffu, some) * hg;
  most = __reduce_max_sync(0xffffffffu, most);
  bool rows = false;
  if (items <= a.G) {
    int T = 0, big = 0;
    auto pieces = [&](int v) {  // 0: none, or small
      return 2 * v <= T ? 0 : v <= kPagedWhole ? 1 : (int)((unsigned)(v + T - 1) / (unsigned)T);
    };
    auto cost = [&](int v) { return v > 0 && 2 * v <= T ? v + kPagedCost : 0; };
    auto fits = [&](int t) {
      T = t;
      big = 0;
      int small = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int v = tiles_at(b0);
        big += pieces(v);
        small += cost(v);
      }
      big = __reduce_add_sync(0xffffffffu, big) * hg;
      small = __reduce_add_sync(0xffffffffu, small) * hg;
      return big + (small + T + kPagedCost - 1) / (T + kPagedCost) <= a.G;
    };
    // T = the longest item's tiles fits: one block an item or fewer.  (The sum
    // of n / T + 1 over the items bounds the pieces: look up to there first.)
    const int lo = max(kPagedLeast, (total + a.G - 1) / a.G), nc = min(16, (int)blockDim.x >> 5);
    int no = lo - 1, yes = max(most, lo);
    int top = a.G > items ? max(lo, min(yes, (total + a.G - items - 1) / (a.G - items))) : yes;
#pragma unroll 1
    while (yes - no > 1) {
      auto cand = [&](int w) { return no + 1 + (int)((int64_t)(top - no - 1) * w / (nc - 1)); };
      if (warp < nc) {
        const bool f = fits(cand(warp));
        if (lane == 0) s_fit[warp] = f;
      }
      __syncthreads();
      const unsigned int m = __ballot_sync(0xffffffffu, lane < nc && s_fit[lane] != 0);
      if (m == 0) {
        no = top;
      } else {
        const int w = __ffs(m) - 1, hi = cand(w);
        if (w > 0) no = cand(w - 1);
        yes = hi;
      }
      top = yes;
      __syncthreads();
    }
    if (warp > 0) return r;
    fits(yes);
    // (lengths that do not fit well: the row of tiles is better, although its
    // blocks have two segments)
    rows = T > (total + a.G - 1) / a.G + kPagedCost && most > kPagedWhole;
    if (!rows) {
      int blocks = 0, before = 0;
      const int share = T + kPagedCost, s0 = (c - big) * 2 * share;  // a shared block takes the items whose middle lies in its share
      r.T = T;
      r.stop = s0 + 2 * share;
#pragma unroll 1
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int n = tiles_at(b0);
        if (c < big) {
          const int p = pieces(n) * hg, pi = scan(p);
          const unsigned int here = __ballot_sync(0xffffffffu, blocks + pi > c);
          if (here) {
            const int l = __ffs(here) - 1;
            const int n_l = __shfl_sync(0xffffffffu, n, l), p_l = __shfl_sync(0xffffffffu, p, l) / hg;
            const int at = c - blocks - __shfl_sync(0xffffffffu, pi - p, l), g = at / p_l, j = at - g * p_l;
            r.kind = 0;
            r.item = (b0 + l) * hg + g;
            r.t0 = paged_piece(j, n_l, p_l);
            r.t1 = paged_piece(j + 1, n_l, p_l);
            r.last = c - j + p_l - 1;
            break;
          }
          blocks += __shfl_sync(0xffffffffu, pi, 31);
        } else {
          const int w = cost(n), wi = scan(w * hg);
          // the sequence's last group lies behind the share's begin
          const unsigned int here = __ballot_sync(0xffffffffu, w > 0 && 2 * (before + wi) - w >= s0);
          if (here) {
            const int l = __ffs(here) - 1;
            int g = 0, d = before + __shfl_sync(0xffffffffu, wi - w * hg, l);
            const int w_l = __shfl_sync(0xffffffffu, w, l);
            for (; 2 * d + w_l < s0; d += w_l) ++g;
            r.item = (b0 + l) * hg + g;
            r.done = d;
            break;
          }
          before += __shfl_sync(0xffffffffu, wi, 31);
        }
      }
      return r;
    }
  }
  int v = 0, inc = 0;
  if (items > a.G) {
    const int64_t costs = (int64_t)total + (int64_t)some * kPagedCost;
    const int share = (int)((costs + a.G - 1) / a.G), longest = most + kPagedCost;
    // with items that are long next to a share, as many of the longest as one takes
    const int64_t shared = 4 * longest > share ? (int64_t)((share + longest - 1) / longest) * longest : (int64_t)share + longest / 2;
    if (shared <= total / a.G + 2 * kPagedCost + kPagedJoin) {
      const int64_t s0 = (int64_t)c * 2 * share;
      if (s0 > 2 * costs) return r;
      r.T = 2 * most;
      r.stop = (int)(s0 + 2 * share);
      int before = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < a.B; b0 += 32) {
        v = tiles_at(b0);
        const int w = v > 0 ? v + kPagedCost : 0, wi = scan(w * hg);
        // the sequence's last group lies behind the share's begin
        const unsigned int here = __ballot_sync(0xffffffffu, w > 0 && 2 * (before + wi) - w >= (int)s0);
        if (here) {
          const int l = __ffs(here) - 1;
          int g = 0, d = before + __shfl_sync(0xffffffffu, wi - w * hg, l);
          const int w_l = __shfl_sync(0xffffffffu, w, l);
          for (; 2 * d + w_l < (int)s0; d += w_l) ++g;
          r.item = (b0 + l) * hg + g;
          r.done = d;
          return r;
        }
        before += __shfl_sync(0xffffffffu, wi, 31);
      }
      return r;
    }
  }
  r.kind = 2;
  r.total = total;
  r.ge = max(1, paged_blocks(total, a.G));
  r.raw0 = paged_start(c, total, r.ge);
  r.t0 = r.raw0;
  r.t1 = paged_start(c + 1, total, r.ge);
  r.item_t0 = total;
  if (r.t0 >= r.t1) return r;
  // an end that lies in a short item moves to the nearer end of it
  int before = 0, found = 0;
#pragma unroll 1
  for (int b0 = 0; b0 < a.B && found < 2; b0 += 32) {
    v = tiles_at(b0) * hg;
    inc = scan(v);
    const int upto = before + __shfl_sync(0xffffffffu, inc, 31);
#pragma unroll 1
    while (found < 2) {
      const int t = found == 0 ? r.raw0 : r.t1;
      if (t >= upto) break;  // (t = total: not found, not moved)
      const int l = __ffs(__ballot_sync(0xffffffffu, before + inc > t)) - 1;
      const int v_l = __shfl_sync(0xffffffffu, v, l), inc_l = __shfl_sync(0xffffffffu, inc, l);
      const int n = paged_item_seq(a, v_l), b_t0 = before + inc_l - v_l, g = hg == 1 ? 0 : (t - b_t0) / n;
      const int i_t0 = b_t0 + g * n;
      const int to = n > kPagedWhole ? t : 2 * (t - i_t0) < n ? i_t0 : i_t0 + n;
      if (found == 0) {
        r.t0 = to;
        r.item = (b0 + l) * hg + g + (to == i_t0 + n ? 1 : 0);
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

// The segments of a block one after the other: paged_next takes the next one.
struct PagedSegment {
  int item, b, g;
  int tile0, n_tiles;  // first tile in the item; how many
  bool whole;
  bool alone;    // the block's only segment, a piece
  int slot;      // of a partial result: 1 if the item begins behind the start of the block's range, else 0
  int cut_last;  // the item's last block if it begins here and goes on, else -1
  PagedSeq seq;
};
__device__ __forceinline__ bool paged_next(const PagedArgs& a, PagedRange& w, PagedSegment& s, int kt) {
  const int items = a.B * a.hgroups;
  while (w.item < items) {
    s.item = w.item;
    s.b = paged_item_seq(a, w.item);
    s.g = w.item - s.b * a.hgroups;
    if (w.kind == 2 && w.t0 >= w.t1) return false;
    s.seq = paged_seq(a, s.b);
    const int n = paged_tiles(s.seq, kt);
    s.slot = 0;
    s.cut_last = -1;
    s.alone = w.kind == 0;
    if (w.kind == 0) {
      s.tile0 = w.t0;
      s.n_tiles = w.t1 - w.t0;
      s.whole = s.n_tiles == n;
      if (s.tile0 == 0 && !s.whole) s.cut_last = w.last;
      w.item = items;
      return true;
    }
    ++w.item;
    if (w.kind == 1) {
      if (n == 0 || 2 * n > w.T) continue;
      const int cost = n + kPagedCost;
      if (2 * w.done + cost >= w.stop) {
        w.item = items;
        return false;
      }
      w.done += cost;
      s.tile0 = 0;
      s.n_tiles = n;
      s.whole = true;
      return true;
    }
    const int end = w.item_t0 + n, stop = min(w.t1, end);
    if (w.t0 < end) {
      s.tile0 = w.t0 - w.item_t0;
      s.n_tiles = stop - w.t0;
      s.whole = s.n_tiles == n;
      s.slot = w.item_t0 > w.raw0 ? 1 : 0;
      if (s.tile0 == 0 && !s.whole) s.cut_last = paged_block_of(end - 1, w.total, w.ge);
      w.t0 = stop;
      w.item_t0 = end;
      return true;
    }
    w.item_t0 = end;  // no tiles
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
cudaError_t launch_paged_join(const PagedArgs& a, cudaStream_t s);

}  // namespace ds4a
