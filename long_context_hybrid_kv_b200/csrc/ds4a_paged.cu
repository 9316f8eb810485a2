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
    const PagedRange r = paged_range(a, blockIdx.x, kGenKeys);
    if (lane == 0) s_r = r;
  }
  __syncthreads();
  const PagedRange r = s_r;
  const float scale2 = a.scale * kLog2e;
  if (blockIdx.x == 0 && tid == 0) *a.total = r.total;
  if (tid == 0) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  PagedWalk walk(r);
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
      const int64_t t = sg.t + i;
      if (a.weights && tid == 0) a.tile_of[t] = make_int2(sg.item, sg.tile0 + i);
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
        const float mx = ml[tid] / kLog2e;
        const float den = ml[tid] == -INFINITY ? 0.f : ml[kGenHeads + tid] + expf(a.sink[hb + tid] - mx);
        ml[2 * kGenHeads + tid] = den > 0.f ? 1.f / den : 0.f;
        if (a.weights)
          a.lse2[(int64_t)sg.item * kGenHeads + tid] =
              den > 0.f ? ml[tid] + log2f(den) : a.sink[hb + tid] * kLog2e;
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
// M)) over a cut item's segments s in order, then the rope slice turned back.
// At most one item is cut behind each block of the attention.  The common
// item, of up to eight segments, takes a warp a head: the lanes hold the
// segments' maxima, and a lane sums 16 dims.  An item of more segments (few
// long sequences) takes a block a head, its warps an eighth of the segments
// each, added in order.  Bound by latency: three dependent reads from L2 (the
// cut, the maxima, the accumulators).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8, kJoinThreads = 32 * kJoinWarps;
constexpr int kFewSegments = 8;

// the weights of the segments [s0, s0 + 32) in the lanes: e^(m - M) (0 for
// one without keys), with M and the denominator's sum L of all segments
struct JoinHead {
  float M, L;
};
__device__ __forceinline__ const float* join_part(const PagedArgs& a, int c0, int slot0, int s) {
  return paged_part(a, c0 + s, s == 0 ? slot0 : 0);
}
__device__ __forceinline__ JoinHead join_head(const PagedArgs& a, int c0, int slot0, int n_seg, int hl) {
  const int lane = threadIdx.x & 31;
  JoinHead j;
  j.M = -INFINITY;
  j.L = 0.f;
  for (int s0 = 0; s0 < n_seg; s0 += 32) {
    float m = -INFINITY, l = 0.f;
    if (s0 + lane < n_seg) {
      const float* p = join_part(a, c0, slot0, s0 + lane);
      m = p[hl];
      l = p[a.hn + hl];
    }
    float mx = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float M = fmaxf(j.M, mx);
    if (M == -INFINITY) continue;
    j.L = j.L * __expf(j.M - M) + warp_sum(l * __expf(m - M));
    j.M = M;
  }
  return j;
}
// 16 dims of a lane: 4 lane + 128 k .. + 3, k < 4 (D <= 512)
__device__ __forceinline__ void join_sum(const PagedArgs& a, int c0, int slot0, int hl, int s0, int s1, float M,
                                         float (&x)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.f;
#pragma unroll 4
  for (int s = s0; s < s1; ++s) {
    const float* p = join_part(a, c0, slot0, s);
    const float m = p[hl];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (4 * lane + 128 * k < a.D) v[k] = *reinterpret_cast<const float4*>(p + 2 * a.hn + (int64_t)hl * a.D + 4 * lane + 128 * k);
    }
    if (m == -INFINITY) continue;  // (a segment without a key that counts may hold anything)
    const float e = __expf(m - M);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[4 * k] = fmaf(v[k].x, e, x[4 * k]);
      x[4 * k + 1] = fmaf(v[k].y, e, x[4 * k + 1]);
      x[4 * k + 2] = fmaf(v[k].z, e, x[4 * k + 2]);
      x[4 * k + 3] = fmaf(v[k].w, e, x[4 * k + 3]);
    }
  }
}
__device__ __forceinline__ void join_out(const PagedArgs& a, int item, int hl, const JoinHead& j, float (&x)[16]) {
  const int lane = threadIdx.x & 31, D = a.D;
  const int b = paged_item_seq(a, item), h = (item - b * a.hgroups) * a.hn + hl;
  const float sk = a.sink[h];
  const float inv = j.M == -INFINITY ? 0.f : 1.f / (j.L + __expf(sk - j.M));
  if (a.weights && lane == 0) {
    const float top = fmaxf(j.M, sk);
    a.lse2[(int64_t)item * a.hn + hl] = (top + logf(j.L * expf(j.M - top) + expf(sk - top))) * kLog2e;
  }
  const int pos = a.q_pos[b];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int d = 4 * lane + 128 * k;
    if (d >= D) continue;
    unsigned int w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float x0 = x[4 * k + 2 * i] * inv, x1 = x[4 * k + 2 * i + 1] * inv;
      const int dd = d + 2 * i;
      if (dd >= D - a.R) {
        float cs, sn;
        rope_cos_sin(pos, a.rope.t[(dd - (D - a.R)) >> 1], &cs, &sn);
        const float y0 = x0 * cs + x1 * sn;
        x1 = -x0 * sn + x1 * cs;
        x0 = y0;
      }
      w[i] = f2_to_bf2x2(x0, x1);
    }
    *reinterpret_cast<uint2*>(a.out + ((int64_t)b * a.H + h) * D + d) = make_uint2(w[0], w[1]);
  }
}

// blocks 0 .. few - 1: eight heads of a cut; from there on: heads of the
// items of many segments
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedArgs a, int few) {
  __shared__ __align__(16) float s_x[kJoinWarps][512];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  float x[16];
  if ((int)blockIdx.x < few) {
    if (a.W == 0)  // sequences without any key: nothing but the sink
      for (int b = blockIdx.x; b < a.B; b += few) {
        const PagedSeq s = paged_seq(a, b);
        if (s.pos >= 0 && s.n_keys == 0)
          for (int e = tid; e < a.H * a.D / 2; e += kJoinThreads)
            reinterpret_cast<unsigned int*>(a.out + (int64_t)b * a.H * a.D)[e] = 0u;
      }
    const int per = a.hn / kJoinWarps, c0 = blockIdx.x / per, hl = (blockIdx.x - c0 * per) * kJoinWarps + warp;
    const int4 cut = a.cut[c0];
    const int n_seg = cut.y - c0 + 1;
    if (cut.x < 0 || n_seg > kFewSegments) return;
    const int b = paged_item_seq(a, cut.x);
    if ((cut.x - b * a.hgroups) * a.hn + hl >= a.H) return;
    const JoinHead j = join_head(a, c0, cut.z, n_seg, hl);
    join_sum(a, c0, cut.z, hl, 0, n_seg, j.M, x);
    join_out(a, cut.x, hl, j, x);
    return;
  }
  // the (blockIdx.x - few) / hn-th item of many segments
  const int want = (blockIdx.x - few) / a.hn, hl = (blockIdx.x - few) % a.hn;
  int seen = 0, c0 = -1;
  int4 cut = make_int4(-1, 0, 0, 0);
  for (int c = 0; c < a.G && c0 < 0; c += 160) {
    int4 v[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) v[k] = c + 32 * k + lane < a.G ? a.cut[c + 32 * k + lane] : make_int4(-1, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int ck = c + 32 * k;
      const unsigned int m = __ballot_sync(0xffffffffu, v[k].x >= 0 && v[k].y - (ck + lane) + 1 > kFewSegments);
      const int n = __popc(m);
      if (c0 < 0 && seen + n > want) {
        unsigned int r = m;
        for (int i = seen; i < want; ++i) r &= r - 1;
        const int l = __ffs(r) - 1;
        c0 = ck + l;
        cut.x = __shfl_sync(0xffffffffu, v[k].x, l);
        cut.y = __shfl_sync(0xffffffffu, v[k].y, l);
        cut.z = __shfl_sync(0xffffffffu, v[k].z, l);
      }
      seen += n;
    }
  }
  if (c0 < 0) return;
  const int b = paged_item_seq(a, cut.x), n_seg = cut.y - c0 + 1;
  if ((cut.x - b * a.hgroups) * a.hn + hl >= a.H) return;
  const JoinHead j = join_head(a, c0, cut.z, n_seg, hl);
  join_sum(a, c0, cut.z, hl, warp * n_seg / kJoinWarps, (warp + 1) * n_seg / kJoinWarps, j.M, x);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<float4*>(&s_x[warp][4 * lane + 128 * k]) = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    for (int w = 1; w < kJoinWarps; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(&s_x[w][4 * lane + 128 * k]);
      x[4 * k] += v.x;
      x[4 * k + 1] += v.y;
      x[4 * k + 2] += v.z;
      x[4 * k + 3] += v.w;
    }
  join_out(a, cut.x, hl, j, x);
}

// Attention weight of a slot: sum over the heads of p 2^(ref - lse2), from
// the probabilities that the attention left per tile (128 bytes a key for 64
// heads).  A block a tile; the factors 2^(ref - lse2) once a tile, four
// threads a key.
__global__ void __launch_bounds__(kJoinThreads) paged_weights_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ float f[128];
  const int tid = threadIdx.x, hn = a.hn;
  pdl_trigger();
  pdl_wait();
  const int total = *a.total;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const int2 at = a.tile_of[t];
    const int b = paged_item_seq(a, at.x);
    if (at.x != b * a.hgroups) continue;  // the sequence's first group sums them all
    const PagedSeq s = paged_seq(a, b);
    const int n_tiles = paged_tiles(s, a.kt), j0 = at.y * a.kt;
    if (at.y == 0 && tid == 0 && s.n > a.w_len) raise_err(a.err, DS4A_DEV_BAD_INDEX);
    __syncthreads();
    for (int h = tid; h < a.H; h += kJoinThreads) {
      const int g = h / hn;
      f[h] = exp2f(a.tile_ref[((int64_t)t + (int64_t)g * n_tiles) * hn + h % hn] - a.lse2[(int64_t)(at.x + g) * hn + h % hn]);
    }
    __syncthreads();
    for (int i0 = 0; i0 < a.kt; i0 += kJoinThreads / 4) {
      const int i = i0 + (tid >> 2), q = tid & 3;
      float w = 0.f;
      if (i < a.kt)
        for (int g = 0; g < a.hgroups; ++g) {
          const uint16_t* p = a.tile_p + (((int64_t)t + (int64_t)g * n_tiles) * a.kt + i) * hn;
          for (int c = 8 * q; c < hn; c += 32) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + (a.p_swizzled ? c ^ ((i & 7) << 3) : c));
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

}  // namespace

cudaError_t launch_paged_attend_generic(const PagedArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)(kGenHeads * a.D + kGenKeys * (a.D + 1) + kGenHeads * kGenKeys + 3 * kGenHeads) * sizeof(float);
  static std::atomic<int> cache[kMaxDevices];
  cudaError_t e = ensure_smem(paged_attend_generic_kernel, (int)smem, cache);
  if (e != cudaSuccess) return e;
  TraceScope tr("paged_attend_generic", s);
  return launch_pdl(paged_attend_generic_kernel, dim3(a.G), dim3(kGenThreads), smem, s, a);
}

cudaError_t launch_paged_join(const PagedArgs& a, int tiles, cudaStream_t s) {
  if (a.G > 1 || a.W == 0) {  // (one block cuts nothing)
    TraceScope tr("paged_join", s);
    const int few = a.G * (a.hn / kJoinWarps), many = (a.G - 1) / kFewSegments * a.hn;
    // (neighbours share a block, so such an item takes eight blocks or more of its own)
    const cudaError_t e = launch_pdl(paged_join_kernel, dim3(few + many), dim3(kJoinThreads), 0, s, a, few);
    if (e != cudaSuccess) return e;
  }
  if (!a.weights) return cudaSuccess;
  TraceScope tr("paged_weights", s);
  return launch_pdl(paged_weights_kernel, dim3(min(tiles, 148 * 6)), dim3(kJoinThreads), 0, s, a);
}

void paged_shape_generic(PagedArgs* a) {
  a->hn = kGenHeads;
  a->kt = kGenKeys;
  a->G = 148 * 2;
  a->p_swizzled = 0;
}

}  // namespace ds4a
