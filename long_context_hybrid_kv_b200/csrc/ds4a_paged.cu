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
  if (blockIdx.x == 0 && tid == 0) *a.total = r.total;
  if (tid == 0) a.cut[blockIdx.x] = make_int4(-1, 0, 0, 0);
  PagedWalk walk(r);
  PagedSegment sg;
  while (paged_next(a, walk, sg)) {
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
// M)) over a cut item's segments s, then the rope slice turned back.  Only
// cut items are looked at (at most one a block of the attention): every block
// lists them and takes (item, head) pairs in turn.  Four groups of 64 threads
// take the segments in turn, a thread eight dims, and are added in order.
// Bound by L2: an accumulator is read once, half a microsecond or more after
// it was written.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256, kJoinGroups = 4;
constexpr int kMaxBlocks = 512;  // of the attention's grid

__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const __grid_constant__ PagedArgs a) {
  __shared__ int4 cuts[kMaxBlocks];
  __shared__ int from[kMaxBlocks];
  __shared__ float wt[kMaxBlocks];
  __shared__ int n_cuts;
  __shared__ float s_l;
  __shared__ __align__(16) float acc[kJoinGroups][512];
  const int tid = threadIdx.x, D = a.D;
  pdl_trigger();
  pdl_wait();
  if (tid < 32) {
    int n = 0;
    for (int c0 = 0; c0 < a.G; c0 += 32) {
      const int c = c0 + tid;
      const int4 v = c < a.G ? a.cut[c] : make_int4(-1, 0, 0, 0);
      const unsigned int m = __ballot_sync(0xffffffffu, v.x >= 0);
      if (v.x >= 0) {
        const int at = n + __popc(m & ((1u << tid) - 1u));
        cuts[at] = v;
        from[at] = c;
      }
      n += __popc(m);
    }
    if (tid == 0) n_cuts = n;
  }
  if (a.W == 0)  // sequences without any key: nothing but the sink
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
      const PagedSeq s = paged_seq(a, b);
      if (s.pos >= 0 && s.n_keys == 0)
        for (int e = tid; e < a.H * D / 2; e += kJoinThreads)
          reinterpret_cast<unsigned int*>(a.out + (int64_t)b * a.H * D)[e] = 0u;
    }
  __syncthreads();
  const int grp = tid >> 6, l64 = tid & 63;
  for (int u = blockIdx.x; u < n_cuts * a.hn; u += gridDim.x) {
    const int4 cut = cuts[u / a.hn];
    const int c0 = from[u / a.hn], hl = u % a.hn, n_seg = cut.y - c0 + 1;
    const int b = cut.x / a.hgroups, h = (cut.x - b * a.hgroups) * a.hn + hl;
    if (h >= a.H) continue;
    auto part_of = [&](int s) { return paged_part(a, c0 + s, s == 0 ? cut.z : 0); };
    __syncthreads();
    if (tid < 32) {
      float M = -INFINITY, L = 0.f;
      for (int s = tid; s < n_seg; s += 32) {
        wt[s] = part_of(s)[hl];
        M = fmaxf(M, wt[s]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      for (int s = tid; s < n_seg; s += 32) {
        const float e = M == -INFINITY ? 0.f : __expf(wt[s] - M);
        wt[s] = e;
        L = fmaf(part_of(s)[a.hn + hl], e, L);
      }
      L = warp_sum(L);
      if (tid == 0) {
        const float sk = a.sink[h], top = fmaxf(M, sk);
        s_l = M == -INFINITY ? 0.f : 1.f / (L + __expf(sk - M));
        if (a.weights) a.lse2[(int64_t)cut.x * a.hn + hl] = (top + logf(L * expf(M - top) + expf(sk - top))) * kLog2e;
      }
    }
    __syncthreads();
    const float inv = s_l;
    const int pos = a.q_pos[b];
    for (int d0 = 0; d0 < D; d0 += 512) {
      const int d = d0 + 8 * l64;
      if (d < D) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
#pragma unroll 4
        for (int s = grp; s < n_seg; s += kJoinGroups) {
          const float4* p = reinterpret_cast<const float4*>(part_of(s) + 2 * a.hn + (int64_t)hl * D + d);
          const float4 v = p[0], w = p[1];
          const float e = wt[s];
          if (e != 0.f) {  // (a segment without a key that counts may hold anything)
            x[0] = fmaf(v.x, e, x[0]); x[1] = fmaf(v.y, e, x[1]); x[2] = fmaf(v.z, e, x[2]); x[3] = fmaf(v.w, e, x[3]);
            x[4] = fmaf(w.x, e, x[4]); x[5] = fmaf(w.y, e, x[5]); x[6] = fmaf(w.z, e, x[6]); x[7] = fmaf(w.w, e, x[7]);
          }
        }
        *reinterpret_cast<float4*>(&acc[grp][8 * l64]) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(&acc[grp][8 * l64 + 4]) = make_float4(x[4], x[5], x[6], x[7]);
      }
      __syncthreads();
      const int e = 2 * tid, dd = d0 + e;
      if (e < 512 && dd < D) {
        float x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int g = 0; g < kJoinGroups; ++g) {
          x0 += acc[g][e];
          x1 += acc[g][e + 1];
        }
        x0 *= inv;
        x1 *= inv;
        if (dd >= D - a.R) {
          float cs, sn;
          rope_cos_sin(pos, a.rope.t[(dd - (D - a.R)) >> 1], &cs, &sn);
          const float y0 = x0 * cs + x1 * sn;
          x1 = -x0 * sn + x1 * cs;
          x0 = y0;
        }
        *reinterpret_cast<unsigned int*>(a.out + ((int64_t)b * a.H + h) * D + dd) = f2_to_bf2x2(x0, x1);
      }
    }
  }
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
    const int b = at.x / a.hgroups;
    if (at.x != b * a.hgroups) continue;  // the sequence's first group sums them all
    const PagedSeq s = paged_seq(a, b);
    const int n_tiles = paged_tiles(a, s), j0 = at.y * a.kt;
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
    const cudaError_t e = launch_pdl(paged_join_kernel, dim3(min(148 * 6, a.G * a.hn)), dim3(kJoinThreads), 0, s, a);
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
}

}  // namespace ds4a
