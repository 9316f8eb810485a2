// Eviction from a bounded paged cache by accumulated attention weight.
//
//   acc[s] += w[s]                               for the n slots in use
//   if n > budget: keep the `recent` youngest entries and, of the others,
//   those of the largest acc (ties: the lower slot), `budget` in all
//
// A softmax over the cache does not ask for its order (each entry carries
// its own position), so nothing is shifted: the kept entries that lie in
// slots >= budget move into the slots below budget that the evicted ones
// leave, in order.  Sources and destinations are disjoint, every row moves at
// most once, and one entry in, one entry out moves a single row.
//
// evict_select_kernel, one block per sequence: a radix select over the order-
// preserving integer form of acc, then one ordered walk that ranks holes and
// movers.  evict_move_kernel, over the whole GPU: the rows.
#include "ds4a_evict.cuh"

namespace ds4a {
namespace {

constexpr int kThreads = 1024;

// larger = kept first; a protected entry is above all weights, NaN above the
// others, -0 as 0
__device__ __forceinline__ unsigned int evict_key(float acc, bool protect) {
  const unsigned int u = __float_as_uint(acc);
  if (protect) return 0xFFFFFFFFu;
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFEu;
  return u == 0x80000000u ? f2key(0.f) : f2key(acc);
}

// exclusive prefix of two 16-bit-safe counts over the block, and their totals
__device__ __forceinline__ int2 block_scan(int x, int y, int2* sums, int2* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) {
      ix += ux;
      iy += uy;
    }
  }
  __syncthreads();
  if (lane == 31) sums[warp] = make_int2(ix, iy);
  __syncthreads();
  int bx = 0, by = 0, tx = 0, ty = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    const int2 v = sums[w];
    if (w < warp) {
      bx += v.x;
      by += v.y;
    }
    tx += v.x;
    ty += v.y;
  }
  *total = make_int2(tx, ty);
  return make_int2(bx + ix - x, by + iy - y);
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictArgs a) {
  __shared__ unsigned int hist[256];
  __shared__ unsigned int s_digit, s_above;
  __shared__ int2 sums[kThreads / 32];
  const int b = blockIdx.x, tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int pos = a.q_pos[b];
  if (pos < 0) {
    if (tid == 0) {
      raise_err(a.err, DS4A_DEV_BAD_POS);
      a.moves[b] = 0;
    }
    return;
  }
  const int gone = a.drop[b];
  const int closed = (int)(((int64_t)pos + 1) / a.m);
  const int n = max(0, min(closed - gone, a.cap));
  float* acc = a.acc + (int64_t)b * a.stride;
  int32_t* entry = a.entry + (int64_t)b * a.stride;
  const uint16_t* w = a.w ? a.w + (int64_t)b * a.w_stride : nullptr;
  if (w)
    for (int s = tid; s < n; s += kThreads) acc[s] += bf2f(w[s]);
  if (n <= a.budget) {
    if (tid == 0) a.moves[b] = 0;
    return;
  }
  const int oldest_kept = closed - a.recent;  // entries from here on are protected
  auto key_of = [&](int s) {
    const int e = entry[s];
    return evict_key(acc[s], (e < 0 ? s + gone : e) >= oldest_kept);
  };
  __syncthreads();
  // the budget-th largest key, digit by digit
  unsigned int prefix = 0, need = (unsigned int)a.budget;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    const unsigned int mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    for (int s = tid; s < n; s += kThreads) {
      const unsigned int k = key_of(s);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (tid == 0) {
      unsigned int above = 0;
      int d = 255;
      while (d > 0 && above + hist[d] < need) above += hist[d--];
      s_digit = (unsigned int)d;
      s_above = above;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    need -= s_above;
    __syncthreads();
  }
  // slots in order: a key above the threshold is kept, of the equal ones the
  // first `need`
  int32_t* dst = a.list + (int64_t)b * 2 * a.budget;
  int32_t* src = dst + a.budget;
  unsigned int ties = 0;
  int holes = 0, movers = 0;
  for (int s0 = 0; s0 < n; s0 += kThreads) {
    const int s = s0 + tid;
    const unsigned int k = s < n ? key_of(s) : 0u;
    const bool tie = s < n && k == prefix;
    int2 total;
    const int2 rank = block_scan(tie, 0, sums, &total);
    const bool keep = s < n && (k > prefix || (tie && ties + (unsigned int)rank.x < need));
    ties += (unsigned int)total.x;
    const bool hole = s < a.budget && !keep, mover = s >= a.budget && keep;
    const int2 at = block_scan(hole, mover, sums, &total);
    if (hole) dst[holes + at.x] = s;
    if (mover) src[movers + at.y] = s;
    holes += total.x;
    movers += total.y;
  }
  __syncthreads();
  for (int s = tid; s < a.budget; s += kThreads)
    if (entry[s] < 0) entry[s] = s + gone;
  __syncthreads();
  for (int r = tid; r < movers; r += kThreads) {
    const int from = src[r], to = dst[r], e = entry[from];
    acc[to] = acc[from];
    entry[to] = e < 0 ? from + gone : e;
  }
  __syncthreads();
  // slots behind the kept ones start over (n may stop short of stale ones of a longer cache)
  for (int s = a.budget + tid; s < a.cap; s += kThreads) {
    acc[s] = 0.f;
    entry[s] = -1;
  }
  if (tid == 0) {
    a.moves[b] = movers;
    a.drop[b] = gone + (n - a.budget);
  }
}

// rows in 16-byte pieces, a warp a row
__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int moves = a.moves[b];
  const int32_t* dst = a.list + (int64_t)b * 2 * a.budget;
  const int32_t* src = dst + a.budget;
  auto row = [&](int slot) -> uint8_t* {
    const int pg = slot / a.page_size;
    const int ph = a.table[(int64_t)b * a.table_stride + pg];
    if (ph < 0 || ph >= a.n_pages) return nullptr;
    return a.pages + ((int64_t)ph * a.page_size + (slot - pg * a.page_size)) * a.row_bytes;
  };
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < moves; r += gridDim.x * 8) {
    uint8_t* to = row(dst[r]);
    const uint8_t* from = row(src[r]);
    if (!to || !from) {
      if (lane == 0) raise_err(a.err, DS4A_DEV_BAD_INDEX);
      continue;
    }
    for (int i = lane * 16; i < a.row_bytes; i += 512)
      *reinterpret_cast<uint4*>(to + i) = *reinterpret_cast<const uint4*>(from + i);
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  {
    TraceScope tr("evict_select", s);
    const cudaError_t e = launch_pdl(evict_select_kernel, dim3(a.B), dim3(kThreads), 0, s, a);
    if (e != cudaSuccess) return e;
  }
  TraceScope tr("evict_move", s);
  const int most = min(a.budget, a.cap - a.budget);
  const int blocks = max(1, min((most + 7) / 8, 148 * 8 / a.B));
  return launch_pdl(evict_move_kernel, dim3(blocks, a.B), dim3(256), 0, s, a);
}

}  // namespace ds4a
