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
// evict_keep_kernel, one block per sequence of up to 32768 slots, a thread up
// to 32 slots in a row: the budget-th largest weight by bisection over its
// order-preserving integer form, the keys in registers (a count of all of them
// is a few instructions a key and one barrier, without the contention that a
// histogram of weights, which share their exponents, has; it ends as soon as a
// bound leaves exactly `budget`), then two scans rank holes and movers.
// evict_select_kernel does the same by radix select from memory, for more
// slots.  evict_move_kernel, over the whole GPU: the rows; few are moved by the
// first kernel itself.
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
    // the digit at which the keys from the top on reach `need`: lane l of
    // the first warp sums the digits 255 - 8l .. 248 - 8l
    if (tid < 32) {
      unsigned int h[8], c = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = hist[255 - 8 * tid - i];
        c += h[i];
      }
      unsigned int up = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned int u = __shfl_up_sync(0xffffffffu, up, o);
        if (tid >= o) up += u;
      }
      up -= c;  // above this lane's digits
      if (up < need && up + c >= need) {
        int i = 0;
        while (up + h[0] < need) {
          up += h[0];
#pragma unroll
          for (int q = 0; q < 7; ++q) h[q] = h[q + 1];
          ++i;
        }
        s_digit = (unsigned int)(255 - 8 * tid - i);
        s_above = up;
      }
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

// row of a slot, or nullptr (a bad page)
__device__ __forceinline__ uint8_t* evict_row(const EvictArgs& a, int b, int slot) {
  const int pg = slot / a.page_size;
  const int ph = a.table[(int64_t)b * a.table_stride + pg];
  if (ph < 0 || ph >= a.n_pages) return nullptr;
  return a.pages + ((int64_t)ph * a.page_size + (slot - pg * a.page_size)) * a.row_bytes;
}
// a warp moves a row, in 16-byte pieces
__device__ __forceinline__ void evict_move_row(const EvictArgs& a, int b, int from, int to) {
  const int lane = threadIdx.x & 31;
  const uint8_t* src = evict_row(a, b, from);
  uint8_t* dst = evict_row(a, b, to);
  if (!src || !dst) {
    if (lane == 0) raise_err(a.err, DS4A_DEV_BAD_INDEX);
    return;
  }
  for (int i = lane * 16; i < a.row_bytes; i += 512)
    *reinterpret_cast<uint4*>(dst + i) = *reinterpret_cast<const uint4*>(src + i);
}

// kPer slots a thread
template <int kPer>
__global__ void __launch_bounds__(kThreads, 1) evict_keep_kernel(const EvictArgs a, int move_here) {
  extern __shared__ unsigned int keys[];  // slot s at s + s / 32 (a thread's run of 32 would be one bank)
  __shared__ int2 sums[kThreads / 32];
  __shared__ int counts[2][kThreads / 32];
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_trigger();
  pdl_wait();
  const int pos = a.q_pos[b], gone = a.drop[b];
  if (pos < 0) {
    if (tid == 0) {
      raise_err(a.err, DS4A_DEV_BAD_POS);
      a.moves[b] = 0;
    }
    return;
  }
  const int closed = (int)(((unsigned)pos + 1u) / (unsigned)a.m);
  const int n = max(0, min(closed - gone, a.cap)), budget = a.budget;
  float* acc = a.acc + (int64_t)b * a.stride;
  int32_t* entry = a.entry + (int64_t)b * a.stride;
  const uint16_t* w = a.w ? a.w + (int64_t)b * a.w_stride : nullptr;
  const bool full = n > budget;
  const int oldest_kept = closed - a.recent;  // entries from here on are protected
#pragma unroll 4
  for (int s = tid; s < n; s += kThreads) {
    float x = acc[s];
    if (w) {
      x += bf2f(w[s]);
      acc[s] = x;
    }
    if (full) {
      int e = entry[s];
      if (e < 0) {
        e = s + gone;
        entry[s] = e;
      }
      keys[s + (s >> 5)] = evict_key(x, e >= oldest_kept);
    }
  }
  if (!full) {
    if (tid == 0) a.moves[b] = 0;
    return;
  }
  __syncthreads();
  const int s0 = tid * kPer;
  unsigned int key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = s0 + i < n ? keys[s0 + i + ((s0 + i) >> 5)] : 0u;
  int round = 0;
  auto count = [&](unsigned int bound) {  // keys >= bound (> 0), over the block
    int c = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c += key[i] >= bound;
    c = __reduce_add_sync(0xffffffffu, c);
    int* buf = counts[round++ & 1];
    if (lane == 0) buf[warp] = c;
    __syncthreads();
    return __reduce_add_sync(0xffffffffu, buf[lane]);
  };
  // the largest bound that leaves `budget` keys or more; `above`: keys over it
  unsigned int bound = 0;
  int above = n;
  bool exact = false;
  for (int bit = 31; bit >= 0; --bit) {
    const unsigned int b2 = bound | (1u << bit);
    const int c = count(b2);
    if (c >= budget) bound = b2;
    else above = c;
    if (c == budget) {
      exact = true;
      break;
    }
  }
  // a key above the bound is kept, of the equal ones the lowest `need`
  const int need = exact ? 0x7FFFFFFF : budget - (above == n ? 0 : above);
  int2 total;
  int ties = 0;
  if (!exact) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += s0 + i < n && key[i] == bound;
    ties = block_scan(mine, 0, sums, &total).x;
  }
  unsigned int keep = 0;
  int holes = 0, movers = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = s0 + i;
    if (s >= n) break;
    const bool k = key[i] > bound || (key[i] == bound && ties++ < need);
    keep |= (k ? 1u : 0u) << i;
    holes += s < budget && !k;
    movers += s >= budget && k;
  }
  int2 at = block_scan(holes, movers, sums, &total);
  int32_t* dst = a.list + (int64_t)b * 2 * budget;
  int32_t* src = dst + budget;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int s = s0 + i;
    if (s >= n) break;
    const bool k = keep >> i & 1u;
    if (s < budget && !k) dst[at.x++] = s;
    if (s >= budget && k) src[at.y++] = s;
  }
  __syncthreads();
  const int moved = total.y;
  for (int r = tid; r < moved; r += kThreads) {
    const int from = src[r], to = dst[r];
    acc[to] = acc[from];
    entry[to] = entry[from];
  }
  if (move_here)
    for (int r = warp; r < moved; r += kThreads / 32) evict_move_row(a, b, src[r], dst[r]);
  __syncthreads();
  // slots behind the kept ones start over
  for (int s = budget + tid; s < a.cap; s += kThreads) {
    acc[s] = 0.f;
    entry[s] = -1;
  }
  if (tid == 0) {
    a.moves[b] = moved;
    a.drop[b] = gone + (n - budget);
  }
}

__global__ void __launch_bounds__(256) evict_move_kernel(const EvictArgs a) {
  const int b = blockIdx.y;
  pdl_trigger();
  pdl_wait();
  const int moves = a.moves[b];
  const int32_t* dst = a.list + (int64_t)b * 2 * a.budget;
  const int32_t* src = dst + a.budget;
  for (int r = blockIdx.x * 8 + (threadIdx.x >> 5); r < moves; r += gridDim.x * 8) evict_move_row(a, b, src[r], dst[r]);
}

template <int kPer>
cudaError_t launch_keep(const EvictArgs& a, int move_here, cudaStream_t s) {
  const int slots = kPer * kThreads, smem = (slots + slots / 32) * 4;
  static std::atomic<int> cache[kMaxDevices];
  const cudaError_t e = ensure_smem(evict_keep_kernel<kPer>, smem, cache);
  if (e != cudaSuccess) return e;
  TraceScope tr("evict_keep", s);
  return launch_pdl(evict_keep_kernel<kPer>, dim3(a.B), dim3(kThreads), smem, s, a, move_here);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const int most = min(a.budget, a.cap - a.budget);  // rows that a sequence may move
  const int move_here = most <= 64;                  // two rows a warp: less than a launch
  const int per = (a.cap + kThreads - 1) / kThreads;
  cudaError_t e;
  if (per <= 1) e = launch_keep<1>(a, move_here, s);
  else if (per <= 4) e = launch_keep<4>(a, move_here, s);
  else if (per <= 8) e = launch_keep<8>(a, move_here, s);
  else if (per <= 16) e = launch_keep<16>(a, move_here, s);
  else if (per <= 32) e = launch_keep<32>(a, move_here, s);
  else {
    TraceScope tr("evict_select", s);
    e = launch_pdl(evict_select_kernel, dim3(a.B), dim3(kThreads), 0, s, a);
  }
  if (e != cudaSuccess || (move_here && per <= 32)) return e;
  TraceScope tr("evict_move", s);
  const int blocks = max(1, min((most + 7) / 8, 148 * 8 / a.B));
  return launch_pdl(evict_move_kernel, dim3(blocks, a.B), dim3(256), 0, s, a);
}

}  // namespace ds4a
