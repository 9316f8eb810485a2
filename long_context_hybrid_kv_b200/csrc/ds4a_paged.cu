// Decode attention of one new token per sequence over a paged K=V cache
// ("DeepSeek-v4 Beyond Basics" 3.2.2 eq. 19 and 3.3 eqs. 24-27 over a paged
// pool; schedule in ds4a_paged.cuh): the CUDA-core kernel for any head shape,
// and the kernel that joins the segments and sums the attention weights.
#include "ds4a_paged.cuh"

namespace ds4a {
namespace {

constexpr int kGenThreads = 256;
constexpr int kGenHeads = 8;   // heads of an item
constexpr int kGenKeys = 32;   // keys of a tile: 8 heads x 32 keys, one logit a thread
constexpr float kLog2e = 1.4426950408889634f;

// dims d, d + 1 of a cache row
__device__ __forceinline__ float2 row_pair(const PagedArgs& a, const uint8_t* row, bool fp8, int d) {
  if (!fp8) return bf2x2_to_f2(reinterpret_cast<const unsigned int*>(row)[d >> 1]);
  const int n = a.D - a.R;
  if (d >= n) return bf2x2_to_f2(*reinterpret_cast<const unsigned int*>(row + n + 2 * (d - n)));
  const float s = mx_scale(row[n + 2 * a.R + d / kMxBlock]);
  return mul_f2(e4m3x2_to_f2(*reinterpret_cast<const uint16_t*>(row + d)), make_float2(s, s));
}

// One pass over the keys with a running maximum and sum per head; float32
// throughout.  It serves the head shapes that the tensor-core kernel does not.
__global__ void __launch_bounds__(kGenThreads) paged_attend_generic_kernel(const __grid_constant__ PagedArgs a) {
  extern __shared__ float sm[];
  const int D = a.D, LD = D + 1;
  float* qs = sm;                        // [8][D] prepared query
  float* ks = qs + kGenHeads * D;        // [32][D + 1] rows
  float* ps = ks + kGenKeys * LD;        // [8][32] probabilities
  float* ml = ps + kGenHeads * kGenKeys; // [8] max (log2), [8] sum, [8] factor
  __shared__ PagedRange s_r;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  if (warp == 0) {
    const PagedRange r = paged_range(a, blockIdx.x);
    if (lane == 0) s_r = r;
  }
  __syncthreads();
  const PagedRange r = s_r;
  const float scale2 = a.scale * kLog2e;
  int item = r.item, item_t0 = r.item_t0;
  for (int t = r.t0; t < r.t1;) {
    const int b = item / a.hgroups, g = item % a.hgroups;
    const PagedSeq s = paged_seq(a, b);
    const int n_tiles = paged_tiles(a, s);
    if (t >= item_t0 + n_tiles) {  // an item without tiles, or the next one
      item_t0 += n_tiles;
      ++item;
      continue;
    }
    const int t_end = min(r.t1, item_t0 + n_tiles);
    const bool whole = t == item_t0 && t_end == item_t0 + n_tiles;
    const int hb = g * kGenHeads, nh = min(kGenHeads, a.H - hb);
    __syncthreads();
    // q^ = RoPE(RMSNorm(q) g): a warp a head
    if (warp < nh) {
      const uint16_t* qr = a.q + ((int64_t)b * a.H + hb + warp) * D;
      float ss = 0.f;
      for (int d = lane; d < D; d += 32) ss = fmaf(bf2f(qr[d]), bf2f(qr[d]), ss);
      const float rstd = rsqrtf(warp_sum(ss) / (float)D + a.eps);
      for (int d = 2 * lane; d < D; d += 64) {
        float x0 = bf2f(qr[d]) * rstd * a.q_norm_g[d], x1 = bf2f(qr[d + 1]) * rstd * a.q_norm_g[d + 1];
        if (d >= D - a.R) {
          float c, sn;
          rope_cos_sin(s.pos, a.rope.t[(d - (D - a.R)) >> 1], &c, &sn);
          const float y0 = x0 * c - x1 * sn;
          x1 = x0 * sn + x1 * c;
          x0 = y0;
        }
        qs[warp * D + d] = x0;
        qs[warp * D + d + 1] = x1;
      }
    }
    if (tid < kGenHeads) {
      ml[tid] = -INFINITY;
      ml[kGenHeads + tid] = 0.f;
    }
    constexpr int kAcc = kGenHeads * 512 / kGenThreads;
    float acc[kAcc];
#pragma unroll
    for (int i = 0; i < kAcc; ++i) acc[i] = 0.f;
    for (; t < t_end; ++t) {
      const int j0 = (t - item_t0) * kGenKeys;
      __syncthreads();
      bool live = false;
      for (int j = warp; j < kGenKeys; j += kGenThreads / 32) {
        bool fp8 = false;
        const uint8_t* row = nullptr;
        if (lane == 0 && j0 + j < s.n_keys) row = paged_key(a, b, s, j0 + j, &fp8);
        row = reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(row), 0));
        fp8 = __shfl_sync(0xffffffffu, (int)fp8, 0) != 0;
        for (int d = 2 * lane; d < D; d += 64) {
          const float2 v = row ? row_pair(a, row, fp8, d) : make_float2(0.f, 0.f);
          ks[j * LD + d] = v.x;
          ks[j * LD + d + 1] = v.y;
        }
        if (lane == 0) ps[j] = row ? 0.f : -INFINITY;  // (read before the probabilities go in)
      }
      __syncthreads();
      // thread: head warp, key lane
      live = ps[lane] == 0.f;
      __syncthreads();
      float z = -INFINITY;
      if (warp < nh && live) {
        float dot = 0.f;
        for (int d = 0; d < D; ++d) dot = fmaf(qs[warp * D + d], ks[lane * LD + d], dot);
        z = dot * scale2;
      }
      float mt = z;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      const float mo = ml[warp], mn = fmaxf(mo, mt);
      const float p = mn == -INFINITY ? 0.f : exp2f(z - mn);
      const float l = warp_sum(p);
      ps[warp * kGenKeys + lane] = p;
      __syncwarp();
      if (lane == 0) {
        const float f = mn == -INFINITY ? 1.f : exp2f(mo - mn);
        ml[warp] = mn;
        ml[kGenHeads + warp] = ml[kGenHeads + warp] * f + l;
        ml[2 * kGenHeads + warp] = f;
        if (a.weights) a.tile_ref[(int64_t)t * kGenHeads + warp] = mn;
      }
      if (a.weights) a.tile_p[((int64_t)t * kGenKeys + lane) * kGenHeads + warp] = f2bf(p);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kAcc; ++i) {
        const int e = tid + i * kGenThreads;
        if (e >= kGenHeads * D) break;
        const int h = e / D, d = e % D;
        float x = acc[i] * ml[2 * kGenHeads + h];
        for (int j = 0; j < kGenKeys; ++j) x = fmaf(ps[h * kGenKeys + j], ks[j * LD + d], x);
        acc[i] = x;
      }
    }
    __syncthreads();
    if (whole) {
      // finished here: the sink joins the denominator, the rope slice turns back
      if (tid < nh) {
        const float mx = ml[tid] / kLog2e;
        const float den = ml[tid] == -INFINITY ? 0.f : ml[kGenHeads + tid] + expf(a.sink[hb + tid] - mx);
        ml[2 * kGenHeads + tid] = den > 0.f ? 1.f / den : 0.f;
        if (a.weights) {
          a.whole_ml[(int64_t)item * 2 * kGenHeads + tid] = mx;
          a.whole_ml[(int64_t)item * 2 * kGenHeads + kGenHeads + tid] = ml[kGenHeads + tid];
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kAcc; ++i) {
        const int e = tid + i * kGenThreads;
        if (e < kGenHeads * D) ks[e] = acc[i] * ml[2 * kGenHeads + e / D];
      }
      __syncthreads();
      for (int e = 2 * tid; e < nh * D; e += 2 * kGenThreads) {
        const int h = e / D, d = e % D;
        float x0 = ks[e], x1 = ks[e + 1];
        if (d >= D - a.R) {
          float c, sn;
          rope_cos_sin(s.pos, a.rope.t[(d - (D - a.R)) >> 1], &c, &sn);
          const float y0 = x0 * c + x1 * sn;
          x1 = -x0 * sn + x1 * c;
          x0 = y0;
        }
        *reinterpret_cast<unsigned int*>(a.out + ((int64_t)b * a.H + hb + h) * D + d) = f2_to_bf2x2(x0, x1);
      }
    } else {
      const int slot = 2 * blockIdx.x + (item == r.item ? 0 : 1);
      float* part = a.part + (int64_t)slot * (2 * kGenHeads + kGenHeads * D);
      if (tid < kGenHeads) {
        part[tid] = ml[tid] / kLog2e;  // -inf stays
        part[kGenHeads + tid] = ml[kGenHeads + tid];
      }
#pragma unroll
      for (int i = 0; i < kAcc; ++i) {
        const int e = tid + i * kGenThreads;
        if (e < kGenHeads * D) part[2 * kGenHeads + e] = acc[i];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Joining: out = sum_s e^(m_s - M) acc_s / (sum_s e^(m_s - M) l_s + e^(sink -
// M)) over an item's segments s, then the rope slice turned back.  One block
// per (head, sequence), a thread a pair of dims.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

struct JoinItem {
  int t0, t1, total, c0, c1;  // tiles; blocks that hold segments
};
__device__ __forceinline__ JoinItem join_item(const PagedArgs& a, int item) {
  JoinItem j;
  j.t0 = a.first[item];
  j.t1 = a.first[item + 1];
  j.total = a.first[a.B * a.hgroups];
  j.c0 = j.c1 = 0;
  if (j.t1 > j.t0) {
    j.c0 = paged_block_of(j.t0, j.total, a.G);
    j.c1 = paged_block_of(j.t1 - 1, j.total, a.G);
  }
  return j;
}
// segment of block c: in its first slot if the block's tiles begin inside the item
__device__ __forceinline__ const float* join_part(const PagedArgs& a, const JoinItem& j, int c) {
  const int slot = 2 * c + (paged_start(c, j.total, a.G) >= j.t0 ? 0 : 1);
  return a.part + (int64_t)slot * (2 * a.hn + (int64_t)a.hn * a.D);
}

__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedArgs a) {
  const int h = blockIdx.x, b = blockIdx.y, g = h / a.hn, hl = h % a.hn;
  pdl_trigger();
  pdl_wait();
  const int pos = a.q_pos[b];
  if (pos < 0) return;
  const JoinItem j = join_item(a, b * a.hgroups + g);
  const int D = a.D;
  uint16_t* orow = a.out + ((int64_t)b * a.H + h) * D;
  if (j.t1 == j.t0) {  // no keys at all: nothing but the sink
    for (int d = 2 * threadIdx.x; d < D; d += 2 * kJoinThreads) *reinterpret_cast<unsigned int*>(orow + d) = 0u;
    return;
  }
  if (j.c0 == j.c1) return;  // finished by its block
  float M = -INFINITY;
  for (int c = j.c0; c <= j.c1; ++c) M = fmaxf(M, join_part(a, j, c)[hl]);
  for (int d = 2 * threadIdx.x; d < D; d += 2 * kJoinThreads) {
    float L = 0.f, x0 = 0.f, x1 = 0.f;
    if (M != -INFINITY) {
      for (int c = j.c0; c <= j.c1; ++c) {
        const float* p = join_part(a, j, c);
        const float e = __expf(p[hl] - M);  // 0 for a segment without keys
        if (e == 0.f) continue;
        const float2 v = *reinterpret_cast<const float2*>(p + 2 * a.hn + (int64_t)hl * D + d);
        L = fmaf(p[a.hn + hl], e, L);
        x0 = fmaf(v.x, e, x0);
        x1 = fmaf(v.y, e, x1);
      }
      const float inv = 1.f / (L + __expf(a.sink[h] - M));
      x0 *= inv;
      x1 *= inv;
    }
    if (d >= D - a.R) {
      float c, sn;
      rope_cos_sin(pos, a.rope.t[(d - (D - a.R)) >> 1], &c, &sn);
      const float y0 = x0 * c + x1 * sn;
      x1 = -x0 * sn + x1 * c;
      x0 = y0;
    }
    *reinterpret_cast<unsigned int*>(orow + d) = f2_to_bf2x2(x0, x1);
  }
}

// Attention weight of a slot: sum over the heads of p e^(ref - lse), from the
// probabilities that the attention left per tile.  A warp a key.
__global__ void __launch_bounds__(kJoinThreads) paged_weights_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ float lse2[128];
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  const int pos = a.q_pos[b];
  const int n = paged_entries(a, b, pos);
  if (n > a.w_len && blockIdx.x == 0 && tid == 0) raise_err(a.err, DS4A_DEV_BAD_INDEX);
  const int n_w = min(n, a.w_len);
  if ((int)blockIdx.x * a.kt >= n_w) return;
  for (int h = tid; h < a.H; h += kJoinThreads) {
    const int item = b * a.hgroups + h / a.hn, hl = h % a.hn;
    const JoinItem j = join_item(a, item);
    float M = -INFINITY, L = 0.f;
    if (j.c0 == j.c1) {
      M = a.whole_ml[(int64_t)item * 2 * a.hn + hl];
      L = a.whole_ml[(int64_t)item * 2 * a.hn + a.hn + hl];
    } else {
      for (int c = j.c0; c <= j.c1; ++c) M = fmaxf(M, join_part(a, j, c)[hl]);
      for (int c = j.c0; c <= j.c1; ++c) {
        const float* p = join_part(a, j, c);
        if (p[hl] != -INFINITY) L = fmaf(p[a.hn + hl], expf(p[hl] - M), L);
      }
    }
    // log of the denominator, sink included, in log2 units
    const float sk = a.sink[h], top = fmaxf(M, sk);
    lse2[h] = (top + logf(L * expf(M - top) + expf(sk - top))) * kLog2e;
  }
  __syncthreads();
  for (int s0 = blockIdx.x * a.kt; s0 < n_w; s0 += gridDim.x * a.kt) {
    const int tile = s0 / a.kt;
    for (int i = warp; i < a.kt && s0 + i < n_w; i += kJoinThreads / 32) {
      float w = 0.f;
      for (int h = lane; h < a.H; h += 32) {
        const int64_t t = a.first[b * a.hgroups + h / a.hn] + tile;
        const float p = bf2f(a.tile_p[(t * a.kt + i) * a.hn + h % a.hn]);
        const float ref = a.tile_ref[t * a.hn + h % a.hn];
        if (p > 0.f) w += p * exp2f(ref - lse2[h]);
      }
      w = warp_sum(w);
      if (lane == 0) a.weights[(int64_t)b * a.w_stride + s0 + i] = f2bf(w);
    }
  }
}

}  // namespace

cudaError_t launch_paged_attend_generic(const PagedArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)(kGenHeads * a.D + kGenKeys * (a.D + 1) + kGenHeads * kGenKeys + 3 * kGenHeads) * sizeof(float);
  static std::atomic<int> cache[kMaxDevices];
  cudaError_t e = ensure_smem(paged_attend_generic_kernel, (int)smem, cache);
  if (e != cudaSuccess) return e;
  TraceScope tr("paged_attend_generic", s);
  return launch_pdl(paged_attend_generic_kernel, dim3(a.G), dim3(kGenThreads), smem, s, a);
}

cudaError_t launch_paged_join(const PagedArgs& a, cudaStream_t s) {
  {
    TraceScope tr("paged_join", s);
    const cudaError_t e = launch_pdl(paged_join_kernel, dim3(a.H, a.B), dim3(kJoinThreads), 0, s, a);
    if (e != cudaSuccess || !a.weights) return e;
  }
  TraceScope tr("paged_weights", s);
  const int tiles = (a.cap + a.kt - 1) / a.kt;
  return launch_pdl(paged_weights_kernel, dim3(min(tiles, max(1, 148 * 8 / a.B)), a.B), dim3(kJoinThreads), 0, s, a);
}

void paged_shape_generic(PagedArgs* a) {
  a->hn = kGenHeads;
  a->kt = kGenKeys;
  a->G = 148 * 2;
}

}  // namespace ds4a
