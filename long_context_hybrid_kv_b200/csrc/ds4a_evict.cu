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
// evict_keep_kernel, one block or, for more than 16384 slots, a cluster of up
// to eight per sequence, a thread up to 32 slots in a row: the budget-th
// largest weight by bisection over its order-preserving integer form, the keys
// in registers (a count of all of them is a few instructions a key and one
// barrier, without the contention that a histogram of weights, which share
// their exponents, has; it ends as soon as a bound leaves exactly `budget`),
// then two scans rank holes and movers.  Bound by that chain of barriers: 9.4
// us for 32 sequences of 1024 slots, 24 for 8 of 7596, 66 for 32 of 32768.
// evict_select_kernel does the same by radix select from memory, one block a
// sequence, where that leaves a thread more than 32 slots: above 262144 slots,
// and from 32769 slots on in batches that leave no SM for larger clusters (37
// sequences have four blocks each up to 131072 slots, 74 two up to 65536, 75
// one up to 32768).  evict_move_kernel, over the whole GPU: the rows, bound by
// memory; few are moved by the first kernel itself.
#include "ds4a_evict.cuh"

namespace ds4a {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxTeam = 8;  // blocks of a cluster

// larger = kept first; a protected entry is above all weights, NaN above the
// others, -0 as 0
__device__ __forceinline__ unsigned int evict_key(float acc, bool protect) {
  const unsigned int u = __float_as_uint(acc);
  if (protect) return 0xFFFFFFFFu;
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFEu;
  return u == 0x80000000u ? f2key(0.f) : f2key(acc);
}

// A sequence that is left as it is: at a negative position, or with more
// entries than slots (those behind cannot be told apart from free ones, and a
// cut of the others would hand out their numbers); recorded.  The same in all
// blocks of a cluster.
__device__ __forceinline__ bool evict_refuses(const EvictArgs& a, int b, int pos, int closed, int gone) {
  const bool bad_pos = pos < 0;
  if (!bad_pos && (int64_t)closed - gone <= a.cap) return false;
  if (threadIdx.x == 0) {
    raise_err(a.err, bad_pos ? DS4A_DEV_BAD_POS : DS4A_DEV_BAD_INDEX);
    a.moves[b] = 0;
  }
  return true;
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
  const int pos = a.q_pos[b], gone = a.drop[b];
  const int closed = (int)(((unsigned)pos + 1u) / (unsigned)a.m);
  if (evict_refuses(a, b, pos, closed, gone)) return;
  const int n = max(0, closed - gone);
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
  // slots behind the kept ones start over
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
// The blocks of a cluster, each with its part of one sequence's slots.
template <bool kMany>
struct Team {
  uint32_t rank = 0, size = 1;
  __device__ Team() {
    if (!kMany) return;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
  }
  __device__ void sync() const {
    if (kMany)
      asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
    else
      __syncthreads();
  }
  // v into place `rank` of every block's array at (shared) at; one warp
  __device__ void tell(const uint4* at, uint4 v) const {
    const uint32_t r = threadIdx.x & 31;
    if (r < size) {
      const uint32_t here = (uint32_t)__cvta_generic_to_shared(at + rank);
      asm volatile(
          "{\n .reg .b32 there;\n mapa.shared::cluster.u32 there, %0, %1;\n"
          " st.shared::cluster.v4.b32 [there], {%2, %3, %4, %5};\n}\n" ::"r"(here),
          "r"(r), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
          : "memory");
    }
  }
};

template <int kPer, bool kMany>
__global__ void __launch_bounds__(kThreads, 1) evict_keep_kernel(const EvictArgs a, int move_here) {
  extern __shared__ unsigned int keys[];  // slot s of the block at s + s / 32 (a thread's run of 32 would be one bank)
  __shared__ int2 sums[kThreads / 32];
  __shared__ __align__(16) uint4 counts[2][kThreads / 32], told[2][kMaxTeam];
  const Team<kMany> team;
  const int b = blockIdx.x / team.size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int all = kThreads * team.size, first = kThreads * kPer * team.rank;
  pdl_trigger();
  pdl_wait();
  const int pos = a.q_pos[b], gone = a.drop[b];
  const int closed = (int)(((unsigned)pos + 1u) / (unsigned)a.m);
  if (evict_refuses(a, b, pos, closed, gone)) return;
  const int n = max(0, closed - gone), budget = a.budget;
  float* acc = a.acc + (int64_t)b * a.stride;
  int32_t* entry = a.entry + (int64_t)b * a.stride;
  const uint16_t* w = a.w ? a.w + (int64_t)b * a.w_stride : nullptr;
  const bool full = n > budget;
  const int oldest_kept = closed - a.recent;  // entries from here on are protected
  const int n_here = min(kThreads * kPer, n - first);
#pragma unroll 4
  for (int i = tid; i < n_here; i += kThreads) {
    const int s = first + i;
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
      keys[i + (i >> 5)] = evict_key(x, e >= oldest_kept);
    }
  }
  if (!full) {
    if (tid == 0 && team.rank == 0) a.moves[b] = 0;
    return;
  }
  team.sync();  // (and every block of the cluster has begun)
  const int i0 = tid * kPer, s0 = first + i0;
  unsigned int key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = s0 + i < n ? keys[i0 + i + ((i0 + i) >> 5)] : 0u;
  // The largest bound that leaves `budget` keys or more; `above`: keys over it.
  unsigned int bound = 0;
  int above = 0, round = 0;
  bool exact = false;
  // One block: a bit a round.
#pragma unroll 1
  for (int shift = 31; shift >= 0 && !kMany && !exact; --shift) {
    const unsigned int b2 = bound | (1u << shift);
    int c = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) c += key[i] >= b2;
    c = __reduce_add_sync(0xffffffffu, c);
    unsigned int* buf = reinterpret_cast<unsigned int*>(counts[round++ & 1]);
    if (lane == 0) buf[warp] = c;
    __syncthreads();
    c = __reduce_add_sync(0xffffffffu, (int)buf[lane]);
    if (c >= budget) bound = b2;
    else above = c;
    exact = c == budget;
  }
  // A cluster, whose rounds take longer: three bits a round, the keys at or
  // over seven bounds counted at once, two counts of up to 32768 in a word.
#pragma unroll 1
  for (int shift = 30; shift >= 0 && kMany && !exact; shift -= 3) {
    const unsigned int most = shift == 30 ? 3u : 7u;
    unsigned int c[4] = {0, 0, 0, 0};  // bounds 1, 2 | 3, 4 | 5, 6 | 7
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      // how many of the bounds the key reaches
      const unsigned int d = key[i] < bound ? 0u : min((key[i] - bound) >> shift, most);
      c[0] += (d >= 1) | (d >= 2) << 16;
      c[1] += (d >= 3) | (d >= 4) << 16;
      c[2] += (d >= 5) | (d >= 6) << 16;
      c[3] += d >= 7;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) c[q] = __reduce_add_sync(0xffffffffu, c[q]);
    const int buf = round++ & 1;
    if (lane == 0) counts[buf][warp] = make_uint4(c[0], c[1], c[2], c[3]);
    __syncthreads();
    const uint4 v = counts[buf][lane];
    c[0] = __reduce_add_sync(0xffffffffu, v.x);
    c[1] = __reduce_add_sync(0xffffffffu, v.y);
    c[2] = __reduce_add_sync(0xffffffffu, v.z);
    c[3] = __reduce_add_sync(0xffffffffu, v.w);
    if (warp == 0) team.tell(told[buf], make_uint4(c[0], c[1], c[2], c[3]));
    team.sync();
    int k[7] = {0, 0, 0, 0, 0, 0, 0};
#pragma unroll 1
    for (uint32_t r = 0; r < team.size; ++r) {
      const uint4 t = told[buf][r];
      const unsigned int u[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
      for (int q = 0; q < 7; ++q) k[q] += (int)(q & 1 ? u[q >> 1] >> 16 : u[q >> 1] & 0xFFFFu);
    }
    unsigned int j = 0;
#pragma unroll
    for (unsigned int q = 1; q <= 7; ++q)
      if (q <= most) {
        if (k[q - 1] >= budget) {
          j = q;
          exact = k[q - 1] == budget;
        } else if (j == q - 1) {
          above = k[q - 1];
        }
      }
    bound += j << shift;
  }
  // a key above the bound is kept, of the equal ones the lowest `need`
  const int need = exact ? 0x7FFFFFFF : budget - above;
  // the sums of the blocks before this one, and of all
  auto join = [&](int2 total, int2* before) {
    *before = make_int2(0, 0);
    if (!kMany) return total;
    const int buf = round++ & 1;
    if (warp == 0) team.tell(told[buf], make_uint4((unsigned)total.x, (unsigned)total.y, 0, 0));
    team.sync();
    int2 sum = make_int2(0, 0);
#pragma unroll 1
    for (uint32_t r = 0; r < team.size; ++r) {
      const uint4 t = told[buf][r];
      if (r == team.rank) *before = sum;
      sum.x += (int)t.x;
      sum.y += (int)t.y;
    }
    return sum;
  };
  int2 total, before;
  int ties = 0;
  if (!exact) {
    int mine = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mine += s0 + i < n && key[i] == bound;
    ties = block_scan(mine, 0, sums, &total).x;
    join(total, &before);
    ties += before.x;
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
  total = join(total, &before);
  at.x += before.x;
  at.y += before.y;
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
  team.sync();
  const int moved = total.y;
  for (int r = kThreads * team.rank + tid; r < moved; r += all) {
    const int from = src[r], to = dst[r];
    acc[to] = acc[from];
    entry[to] = entry[from];
  }
  if (move_here)
    for (int r = (kThreads * team.rank + tid) / 32; r < moved; r += all / 32) evict_move_row(a, b, src[r], dst[r]);
  team.sync();
  // slots behind the kept ones start over
  for (int s = budget + kThreads * team.rank + tid; s < a.cap; s += all) {
    acc[s] = 0.f;
    entry[s] = -1;
  }
  if (tid == 0 && team.rank == 0) {
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

template <int kPer, bool kMany>
cudaError_t launch_keep(const EvictArgs& a, int team, int move_here, cudaStream_t s) {
  const int slots = kPer * kThreads, smem = (slots + slots / 32) * 4;
  static std::atomic<int> cache[kMaxDevices];
  const cudaError_t e = ensure_smem(evict_keep_kernel<kPer, kMany>, smem, cache);
  if (e != cudaSuccess) return e;
  TraceScope tr("evict_keep", s);
  return launch_pdl_cluster(evict_keep_kernel<kPer, kMany>, dim3(a.B * team), dim3(kThreads), smem, s, team, a, move_here);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const int most = min(a.budget, a.cap - a.budget);  // rows that a sequence may move
  const int move_here = most <= 64;                  // two rows a warp: less than a launch
  // A thread of one block holds up to 16 slots; above that a cluster, whose
  // rounds take longer, pays: until a thread has four or all SMs have a block
  // (32 sequences of 32768 slots, one block and four: 91 and 66 us; of 16384:
  // 36 and 38).  A large batch has one block a sequence.
  int team = 1;
  while (team < kMaxTeam && a.cap > 16 * kThreads && (int64_t)team * 4 * kThreads < a.cap && (int64_t)a.B * team * 2 <= 148)
    team *= 2;
  const int per = (a.cap + kThreads * team - 1) / (kThreads * team);
  cudaError_t e;
  if (team == 1) {
    if (per <= 1) e = launch_keep<1, false>(a, team, move_here, s);
    else if (per <= 4) e = launch_keep<4, false>(a, team, move_here, s);
    else if (per <= 8) e = launch_keep<8, false>(a, team, move_here, s);
    else if (per <= 16) e = launch_keep<16, false>(a, team, move_here, s);
    else if (per <= 32) e = launch_keep<32, false>(a, team, move_here, s);
  } else {
    if (per <= 4) e = launch_keep<4, true>(a, team, move_here, s);
    else if (per <= 8) e = launch_keep<8, true>(a, team, move_here, s);
    else if (per <= 16) e = launch_keep<16, true>(a, team, move_here, s);
    else if (per <= 32) e = launch_keep<32, true>(a, team, move_here, s);
  }
  if (per > 32) {
    TraceScope tr("evict_select", s);
    e = launch_pdl(evict_select_kernel, dim3(a.B), dim3(kThreads), 0, s, a);
  }
  if (e != cudaSuccess || (move_here && per <= 32)) return e;
  TraceScope tr("evict_move", s);
  const int blocks = max(1, min((most + 7) / 8, 148 * 8 / a.B));
  return launch_pdl(evict_move_kernel, dim3(blocks, a.B), dim3(256), 0, s, a);
}

}  // namespace ds4a
