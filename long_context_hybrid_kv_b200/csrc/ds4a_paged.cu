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
constexpr float kNoMax = -1e30f;  // maximum of a segment whose logits are all NaN: finite, below any logit

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
  {
    __shared__ int s_n[512], s_fit[32];
    const PagedRange r = paged_range(a, blockIdx.x, kGenKeys, s_n, 512, s_fit);
    if (tid == 0) s_r = r;
  }
  __syncthreads();
  const PagedRange r = s_r;
  const float scale2 = a.scale * kLog2e;
  if (tid == 0) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  PagedRange walk = r;
  PagedSegment sg;
  while (paged_next(a, walk, sg, kGenKeys)) {
    const int b = sg.b;
    const PagedSeq& s = sg.seq;
    const int hb = sg.g * kGenHeads, nh = min(kGenHeads, a.H - hb);
    if (tid == 0 && sg.cut_last >= 0) a.cut[blockIdx.x] = make_int4(sg.item, sg.cut_last, sg.slot, 0);
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
    for (int i = 0; i < sg.n_tiles; ++i) {
      const int j0 = (sg.tile0 + i) * kGenKeys;
      const int64_t t = (int64_t)sg.item * a.item_tiles + sg.tile0 + i;
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
      // (the maximum passes NaN over, the probabilities and their sum do not)
      const float mo = ml[warp], mn = fmaxf(mo, mt);
      const float p = exp2f(z - (mn == -INFINITY ? 0.f : mn));
      const float l = warp_sum(p);
      ps[warp * kGenKeys + lane] = p;
      __syncwarp();
      if (lane == 0) {
        const float f = mn == -INFINITY ? 1.f : exp2f(mo - mn);
        ml[warp] = mn;
        ml[kGenHeads + warp] = ml[kGenHeads + warp] * f + l;
        ml[2 * kGenHeads + warp] = f;
        if (a.weights) a.tile_ref[t * kGenHeads + warp] = mn;
      }
      if (a.weights) a.tile_p[(t * kGenKeys + lane) * kGenHeads + warp] = f2bf(p);
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
    if (sg.whole) {
      // finished here: the sink joins the denominator, the rope slice turns back
      if (tid < nh) {
        const float mx = ml[tid] / kLog2e, l = ml[kGenHeads + tid];
        const bool none = ml[tid] == -INFINITY && l == 0.f;  // no key counts
        const float den = l + expf(a.sink[hb + tid] - mx);
        ml[2 * kGenHeads + tid] = none ? 0.f : 1.f / den;
        if (a.weights)
          a.lse2[(int64_t)sg.item * kGenHeads + tid] = none ? INFINITY : ml[tid] + log2f(den);
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
      float* part = paged_part(a, blockIdx.x, sg.slot);
      if (tid < kGenHeads) {
        // -inf stays, unless the logits are all NaN: -inf says that no key counts
        const float l = ml[kGenHeads + tid];
        part[tid] = ml[tid] == -INFINITY && l != 0.f ? kNoMax : ml[tid] / kLog2e;
        part[kGenHeads + tid] = l;
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
// M)) over a cut item's segments s in order, then the rope slice turned back.
// At most one item is cut behind each block of the attention.  The common
// item, of up to eight segments, takes two warps a head: the lanes hold the
// segments' maxima, and a lane sums 8 dims of half a head.  An item of more
// segments (few long sequences) takes a block for each half head, its warps an
// eighth of the segments each, added in order.  Bound by latency: two dependent
// reads from L2 (the cut; the maxima with the accumulators), 5 to 6 us behind
// the attention for 19 MB of segments; three blocks an SM (two: 2 us more for
// b24, four, which spill: 4 us more).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;
constexpr int kFewSegments = 8;

__device__ __forceinline__ const float* join_part(const PagedArgs& a, int c0, int slot0, int s) {
  return paged_part(a, c0 + s, s == 0 ? slot0 : 0);
}

// A warp's share of one head: the segments [s0, s1) of n, half of the dims.
// M, L: maximum and sum over all n segments; x: 8 dims of a lane, d + 128 k ..
// + 3, d = d0 + 4 lane, k < 2.
struct JoinSum {
  float M, L, x[8];
};
__device__ __forceinline__ void join_sum(const PagedArgs& a, int c0, int slot0, int n, int hl, int d0, int s0, int s1,
                                         JoinSum& j) {
  const int lane = threadIdx.x & 31, d = d0 + 4 * lane;
  constexpr int kBatch = 4;
  float4 v[kBatch][2];
  float m[kBatch];
  auto load = [&](int s) {  // out before the maxima are known
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      m[i] = -INFINITY;
      v[i][0] = v[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s + i < s1) {
        const float* p = join_part(a, c0, slot0, s + i);
        m[i] = p[hl];
        if (d < a.D) v[i][0] = *reinterpret_cast<const float4*>(p + 2 * a.hn + (int64_t)hl * a.D + d);
        if (d + 128 < a.D) v[i][1] = *reinterpret_cast<const float4*>(p + 2 * a.hn + (int64_t)hl * a.D + d + 128);
      }
    }
  };
  load(s0);
  j.M = -INFINITY;
  j.L = 0.f;
  for (int t = 0; t < n; t += 32) {
    float mt = -INFINITY, lt = 0.f;
    if (t + lane < n) {
      const float* p = join_part(a, c0, slot0, t + lane);
      mt = p[hl];
      lt = p[a.hn + hl];
    }
    float mx = mt;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float M = fmaxf(j.M, mx);
    if (M == -INFINITY) continue;
    j.L = j.L * __expf(j.M - M) + warp_sum(lt * __expf(mt - M));
    j.M = M;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) j.x[i] = 0.f;
  for (int s = s0; s < s1; s += kBatch) {
    if (s > s0) load(s);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // (a segment without a key that counts holds zeros, or NaN where an infinite row gave a logit of -inf)
      const float e = m[i] == -INFINITY ? 0.f : __expf(m[i] - j.M);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        j.x[4 * k] = fmaf(v[i][k].x, e, j.x[4 * k]);
        j.x[4 * k + 1] = fmaf(v[i][k].y, e, j.x[4 * k + 1]);
        j.x[4 * k + 2] = fmaf(v[i][k].z, e, j.x[4 * k + 2]);
        j.x[4 * k + 3] = fmaf(v[i][k].w, e, j.x[4 * k + 3]);
      }
    }
  }
}
__device__ __forceinline__ void join_out(const PagedArgs& a, int item, int hl, int d0, const JoinSum& j, int pos, float sk) {
  const int lane = threadIdx.x & 31, D = a.D;
  const int b = paged_item_seq(a, item), h = (item - b * a.hgroups) * a.hn + hl;
  float x[8];
  const float inv = j.M == -INFINITY ? 0.f : 1.f / (j.L + __expf(sk - j.M));
  if (a.weights && lane == 0 && d0 == 0) {
    const float top = fmaxf(j.M, sk);
    a.lse2[(int64_t)item * a.hn + hl] =
        j.M == -INFINITY ? INFINITY : (top + logf(j.L * expf(j.M - top) + expf(sk - top))) * kLog2e;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = j.x[i] * inv;
  // rotation by -pos: a lane finds the angle of one pair in 32 and has the
  // others' from its neighbours (one place that computes angles, not four: a
  // short kernel waits for its instructions)
  const int r0 = D - a.R;
  if (d0 + 256 > r0) {
#pragma unroll 1
    for (int p0 = 0; 2 * p0 < a.R; p0 += 32) {
      float cs, sn;
      rope_cos_sin(pos, a.rope.t[min(p0 + lane, kMaxRopePairs - 1)], &cs, &sn);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int dd = d0 + 4 * lane + 128 * (i >> 1) + 2 * (i & 1) - r0, pr = dd >> 1;
        const float c1 = __shfl_sync(0xffffffffu, cs, pr & 31), s1 = __shfl_sync(0xffffffffu, sn, pr & 31);
        if (dd >= 0 && (pr & ~31) == p0) {
          const float x0 = x[2 * i], x1 = x[2 * i + 1];
          x[2 * i] = x0 * c1 + x1 * s1;
          x[2 * i + 1] = -x0 * s1 + x1 * c1;
        }
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int d = d0 + 4 * lane + 128 * k;
    if (d < D)
      *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.H + h) * D + d) =
          make_uint2(f2_to_bf2x2(x[4 * k], x[4 * k + 1]), f2_to_bf2x2(x[4 * k + 2], x[4 * k + 3]));
  }
}

// One wave of blocks: each lists the cuts, then their warps take (cut, head,
// half of the dims) in turn, then the blocks (head, half) of the items of many
// segments.
constexpr int kMaxBlocks = 296;  // of the attention's grid

__global__ void __launch_bounds__(kJoinThreads, 3) paged_join_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ __align__(16) float s_x[kJoinWarps][256];
  __shared__ int4 s_cut[kMaxBlocks];  // item, first block, segments, slot of the first
  __shared__ int s_few, s_all;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  if (warp == 0) {  // few segments from the front on, many behind them
    int4 v[(kMaxBlocks + 31) / 32];
#pragma unroll
    for (int k = 0; k < (kMaxBlocks + 31) / 32; ++k) {
      const int c = 32 * k + lane;
      v[k] = c < a.G ? a.cut[c] : make_int4(-1, 0, 0, 0);
    }
    int at = 0;
#pragma unroll
    for (int many = 0; many < 2; ++many) {
#pragma unroll
      for (int k = 0; k < (kMaxBlocks + 31) / 32; ++k) {
        const int c = 32 * k + lane, n = v[k].y - c + 1;
        const bool mine = v[k].x >= 0 && (n > kFewSegments) == (many == 1);
        const unsigned int m = __ballot_sync(0xffffffffu, mine);
        if (mine) s_cut[at + __popc(m & ((1u << lane) - 1u))] = make_int4(v[k].x, c, n, v[k].z);
        at += __popc(m);
      }
      if (lane == 0) (many ? s_all : s_few) = at;
    }
  }
  if (a.W == 0)  // sequences without any key: nothing but the sink
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      const PagedSeq s = paged_seq(a, b);
      if (s.pos >= 0 && s.n_keys == 0)
        for (int e = tid; e < a.H * a.D / 2; e += kJoinThreads)
          reinterpret_cast<unsigned int*>(a.out + (int64_t)b * a.H * a.D)[e] = 0u;
    }
  __syncthreads();
  const int few = s_few, all = s_all, halves = a.D > 256 ? 2 : 1, per = a.hn * halves;
  JoinSum j;
  for (int u = blockIdx.x * kJoinWarps + warp; u < few * per; u += gridDim.x * kJoinWarps) {
    const int4 cut = s_cut[u / per];
    const int w = u % per, hl = w / halves, d0 = (w % halves) * 256;
    const int b = paged_item_seq(a, cut.x), h = (cut.x - b * a.hgroups) * a.hn + hl;
    if (h >= a.H) continue;
    const int pos = a.q_pos[b];
    const float sk = a.sink[h];
    join_sum(a, cut.y, cut.w, cut.z, hl, d0, 0, cut.z, j);
    join_out(a, cut.x, hl, d0, j, pos, sk);
  }
  for (int u = few * per + blockIdx.x; u < all * per; u += gridDim.x) {
    const int4 cut = s_cut[u / per];
    const int w = u % per, hl = w / halves, d0 = (w % halves) * 256;
    const int b = paged_item_seq(a, cut.x), h = (cut.x - b * a.hgroups) * a.hn + hl;
    if (h >= a.H) continue;
    const int pos = a.q_pos[b];
    const float sk = a.sink[h];
    join_sum(a, cut.y, cut.w, cut.z, hl, d0, warp * cut.z / kJoinWarps, (warp + 1) * cut.z / kJoinWarps, j);
    __syncthreads();
    *reinterpret_cast<float4*>(&s_x[warp][4 * lane]) = make_float4(j.x[0], j.x[1], j.x[2], j.x[3]);
    *reinterpret_cast<float4*>(&s_x[warp][4 * lane + 128]) = make_float4(j.x[4], j.x[5], j.x[6], j.x[7]);
    __syncthreads();
    if (warp != 0) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      for (int q = 1; q < kJoinWarps; ++q) {
        const float4 y = *reinterpret_cast<const float4*>(&s_x[q][4 * lane + 128 * k]);
        j.x[4 * k] += y.x;
        j.x[4 * k + 1] += y.y;
        j.x[4 * k + 2] += y.z;
        j.x[4 * k + 3] += y.w;
      }
    join_out(a, cut.x, hl, d0, j, pos, sk);
  }
}

// Attention weight of a slot: sum over the heads of p 2^(ref - lse2), from
// the probabilities that the attention left per tile.  A block a tile; the factors 2^(ref - lse2) once a tile, four
// threads a key.
__global__ void __launch_bounds__(kJoinThreads) paged_weights_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ float f[128];
  const int tid = threadIdx.x, hn = a.hn;
  pdl_trigger();
  pdl_wait();
  for (int u = blockIdx.x; u < a.B * a.item_tiles; u += gridDim.x) {
    const int b = u / a.item_tiles, tile = u - b * a.item_tiles, j0 = tile * a.kt;
    const int item = b * a.hgroups;
    const PagedSeq s = paged_seq(a, b);
    if (tile == 0 && tid == 0 && s.n > a.w_len) raise_err(a.err, DS4A_DEV_BAD_INDEX);
    if (j0 >= min(s.n, a.w_len)) continue;
    __syncthreads();
    for (int h = tid; h < a.H; h += kJoinThreads) {
      const int g = h / hn;
      f[h] = exp2f(a.tile_ref[((int64_t)(item + g) * a.item_tiles + tile) * hn + h % hn] - a.lse2[(int64_t)(item + g) * hn + h % hn]);
    }
    __syncthreads();
    for (int i0 = 0; i0 < a.kt; i0 += kJoinThreads / 4) {
      const int i = i0 + (tid >> 2), q = tid & 3;
      float w = 0.f;
      if (i < a.kt)
        for (int g = 0; g < a.hgroups; ++g) {
          const uint16_t* p = a.tile_p + (((int64_t)(item + g) * a.item_tiles + tile) * a.kt + i) * hn;
          for (int c = 8 * q; c < hn; c += 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + c);
            const unsigned int x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 y = bf2x2_to_f2(x[k]);
              const int h = g * hn + c + 2 * k;
              if (h < a.H) w = fmaf(y.x, f[h], w);
              if (h + 1 < a.H) w = fmaf(y.y, f[h + 1], w);
            }
          }
        }
      w += __shfl_xor_sync(0xffffffffu, w, 1);
      w += __shfl_xor_sync(0xffffffffu, w, 2);
      const int j = j0 + i;
      if (q == 0 && i < a.kt && j < s.n && j < a.w_len) a.weights[(int64_t)b * a.w_stride + j] = f2bf(w);
    }
  }
}

// bits of the heads h, h + 1 in a word that lie below nh
__device__ __forceinline__ unsigned int head_pair(int h, int nh) { return (h < nh ? 0xFFFFu : 0u) | (h + 1 < nh ? 0xFFFF0000u : 0u); }

// The same for the tensor-core kernel's tiles (64 keys x 64 heads, swizzled),
// a warp a tile and no block barrier: a load covers four keys' rows, lane l
// the piece l % 8 of key l / 8, so that a lane's heads alternate between two
// sets of eight.
__global__ void __launch_bounds__(kJoinThreads) paged_weights64_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ __align__(16) float fs[kJoinWarps][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = lane >> 3, piece = lane & 7;
  pdl_trigger();
  pdl_wait();
  float* f = fs[warp];
  for (int u = blockIdx.x * kJoinWarps + warp; u < a.B * a.item_tiles; u += gridDim.x * kJoinWarps) {
    const int b = u / a.item_tiles, tile = u - b * a.item_tiles, j0 = tile * 64;
    const PagedSeq s = paged_seq(a, b);
    if (tile == 0 && lane == 0 && s.n > a.w_len) raise_err(a.err, DS4A_DEV_BAD_INDEX);
    const int n = min(s.n, a.w_len);
    if (j0 >= n) continue;
    float w[2] = {0.f, 0.f};  // of the keys 32 i + 4 piece + row
    for (int g = 0; g < a.hgroups; ++g) {
      const int64_t item = (int64_t)b * a.hgroups + g, t = item * a.item_tiles + tile;
      const uint4* p = reinterpret_cast<const uint4*>(a.tile_p + t * 64 * 64) + lane;
      uint4 v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = p[32 * i];
      if ((g + 1) * 64 > a.H) {
        // heads that the group does not have: their query is 0, and 0 times an infinite row is NaN
        const int nh = a.H - g * 64;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int h0 = 8 * (piece ^ (row + 4 * (i & 1)));
          v[i].x &= head_pair(h0, nh);
          v[i].y &= head_pair(h0 + 2, nh);
          v[i].z &= head_pair(h0 + 4, nh);
          v[i].w &= head_pair(h0 + 6, nh);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int h = lane + 32 * i;
        f[h] = g * 64 + h < a.H ? exp2f(a.tile_ref[t * 64 + h] - a.lse2[item * 64 + h]) : 0.f;
      }
      __syncwarp();
      float f0[8], f1[8];  // keys 8k + row: piece ^ row; keys 8k + 4 + row: piece ^ (4 + row)
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        f0[q] = f[8 * (piece ^ row) + q];
        f1[q] = f[8 * (piece ^ (row + 4)) + q];
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const unsigned int y[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float z = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 x = bf2x2_to_f2(y[q]);
          z = fmaf(x.x, i & 1 ? f1[2 * q] : f0[2 * q], z);
          z = fmaf(x.y, i & 1 ? f1[2 * q + 1] : f0[2 * q + 1], z);
        }
        z += __shfl_xor_sync(0xffffffffu, z, 1);
        z += __shfl_xor_sync(0xffffffffu, z, 2);
        z += __shfl_xor_sync(0xffffffffu, z, 4);
        if (piece == (i & 7)) w[i >> 3] += z;
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int j = j0 + 32 * i + 4 * piece + row;
      if (j < n) a.weights[(int64_t)b * a.w_stride + j] = f2bf(w[i]);
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
  if (a.item_tiles > kPagedWhole || a.W == 0) {  // else nothing is cut
    TraceScope tr("paged_join", s);
    const int blocks = (a.G * a.hn * 2 + kJoinWarps - 1) / kJoinWarps;
    const cudaError_t e = launch_pdl(paged_join_kernel, dim3(min(148 * 3, blocks)), dim3(kJoinThreads), 0, s, a);
    if (e != cudaSuccess) return e;
  }
  if (!a.weights) return cudaSuccess;
  TraceScope tr("paged_weights", s);
  const int64_t tiles = (int64_t)a.B * a.item_tiles;
  if (a.hn == 64) {
    const int64_t blocks = (tiles + kJoinWarps - 1) / kJoinWarps;
    return launch_pdl(paged_weights64_kernel, dim3((int)(blocks < 148 * 2 ? blocks : 148 * 2)), dim3(kJoinThreads), 0, s, a);
  }
  return launch_pdl(paged_weights_kernel, dim3((int)(tiles < 148 * 8 ? tiles : 148 * 8)), dim3(kJoinThreads), 0, s, a);
}

void paged_shape_generic(PagedArgs* a) {
  a->hn = kGenHeads;
  a->kt = kGenKeys;
  a->G = 148 * 2;
}

}  // namespace ds4a
