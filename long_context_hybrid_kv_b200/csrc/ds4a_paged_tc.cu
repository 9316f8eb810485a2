// Decode attention over a paged K=V cache on the tensor cores (tcgen05), for
// rows of 512: "DeepSeek-v4 Beyond Basics" 3.2.2 eq. 19 and 3.3 eqs. 24-27 for
// one new token per sequence; schedule in ds4a_paged.cuh.
//
// All heads read the same rows, so a tile of 64 keys is two dense products with
// the keys, then the dims, on the MMA's M side and 64 heads on N:
//   S^T[key][h]  = KV[key][:] . q^[h][:]      K = 512, A K-major, M = 64
//   O^T[d][h]   += KV[key][d]^T . P^T[key][h]  K = 64 keys, A MN-major, M = 128
// The products are bound by the shared memory that an MMA reads (32 and 48
// cycles each): 0.95 us a tile; at 44 GB/s of HBM an SM its rows take 1.5 us.
// 64 keys, not 128, leave room for nine 128-dim chunks of rows (2.25 tiles)
// next to the 64 KiB of q^, so that the next tile is there and its first
// product runs during this tile's softmax.  What is left is the chain: a slot
// of the ring is free after the second product, its new rows take about 1 us,
// the first product, the softmax and the second product 0.6 + 1.1 + 0.6, and
// the ring holds two tiles of that: 1.9 us a tile (FP8 2.6: the expansion of
// the codes).  (A ring of 48-key tiles, or MMAs of two warps in turn, were
// slower; integer expansion of the codes 114 us instead of 89.)
//
// q^ and P are rounded to bf16, which the MMA takes with bf16 rows (at most
// half a step, 2^-8, each, which the softmax and the sum over keys average: an
// output is off by 0.0024 to 0.0027, root mean square, against the 0.0017 of
// its own rounding; the low halves would take 64 KiB of the ring, and as many
// MMAs again of the second product); logits, maxima, sums and O stay in float32.
//
// Thread block (one per SM, 640 threads):
//   warps 0-7    q^ of every segment, softmax, epilogue: two warps per TMEM
//                lane quarter with 32 heads each.  S^T of M = 64 has 16 keys
//                in each quarter; a thread holds two keys x 8 heads of it, and
//                later a dim row of O^T.
//   warp 8       TMEM allocation; an elected lane issues the MMAs.
//   warps 9-10   find the segments and tell the others; one key a thread, up to
//                four tiles ahead: index, page, row address, and a prefetch of
//                the row into L2, so that HBM keeps streaming while the ring
//                is full.
//   warps 11-18  gather the rows by cp.async, a chunk (16 KiB) at a time, into
//                a ring of nine, in the 128-byte swizzle.  FP8 rows go through
//                registers, a tile ahead, and are expanded on the way.
//   warp 19      fences landed chunks for the MMAs; angles and sinks of the
//                segments to come.
// Of a small call the prologue is half: code that runs once waits for its
// instructions, so it is short and not unrolled (b1 x 64 entries 13.9 -> 11.4
// us).  In a graph of calls with the window of 128: b1 x 8192 entries 21 us,
// b32 x 1024 32 us, b32 x 8192 86 to 109 us from GPU to GPU (272 MB of rows: 2.5
// to 3.2 TB/s), b256 x 512 selected 68 us.
#include "ds4a_paged.cuh"
#include "ds4a_tc.cuh"

namespace ds4a {
namespace {

using namespace tc;

constexpr int kH = 64, kD = 512;
constexpr int kKT = 64;               // keys per tile
constexpr int kThreads = 640;
constexpr int kMmaWarp = 8;
constexpr int kPtr0 = 288;            // first address thread (warps 9-10)
constexpr int kPG0 = 352;             // first gathering thread (warps 11-18)
constexpr int kGather = 256;
constexpr int kFenceWarp = 19;
constexpr int kSlots = 9;             // ring of 128-dim chunks
constexpr int kAhead = 4;             // tiles of row addresses
constexpr int kSegs = 8;              // segments made known: the address warps are at most five tiles, so segments, ahead of the rest
// cos, sin and sinks of four segments: while one is in its epilogue the ring
// can hold the next two's rows and the first of the third's
constexpr int kTabs = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;  // O^T is rescaled when a head's maximum grows by more than 2^8
constexpr float kNoRef = -1e30f;      // reference of a head that has seen no key: finite, below any logit

constexpr uint32_t kBlk = kKT * 128;   // 64 dims of a tile's keys
constexpr uint32_t kSlot = 2 * kBlk;   // 128 dims
constexpr uint32_t kOffKV = 0;
constexpr uint32_t kOffQ = kSlots * kSlot;       // 8 blocks x [64 heads][128 B]
constexpr uint32_t kOffP = kOffQ + 65536;        // [64 keys][128 B]
constexpr uint32_t kOffBar = kOffP + kBlk;
constexpr uint32_t kOffSeg = kOffBar + 480;         // segments
constexpr uint32_t kOffMisc = kOffSeg + kSegs * 64;     // abort flag, TMEM address, the block's range
constexpr uint32_t kOffRow = kOffMisc + 128;      // [4 tiles][64] row addresses, bit 0: FP8
constexpr uint32_t kOffRed = kOffRow + kAhead * kKT * 8;  // [4][64] floats
constexpr uint32_t kOffMrun = kOffRed + 1024;
constexpr uint32_t kOffAlpha = kOffMrun + 256;
constexpr uint32_t kOffInv = kOffAlpha + 256;
constexpr uint32_t kOffSink = kOffInv + 256;
constexpr uint32_t kOffRope = kOffSink + kTabs * 256;  // [4 segments][128] (cos, sin) of the position
constexpr uint32_t kSmemBytes = kOffRope + kTabs * 1024 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of a block");
// The finished output goes out through the q^ and P^T buffers, a head's 1024
// bytes 1088 apart (the two heads that a warp writes at a time then lie in
// different banks).
constexpr uint32_t kStagePitch = 1088;
static_assert(kH * kStagePitch <= 65536 + kBlk && kH * kD * 4 <= kSlots * kSlot, "output stages");

enum Bar {
  kKVLanded = 0, kKVFull = kKVLanded + kSlots, kKVEmpty = kKVFull + kSlots, kRowFull = kKVEmpty + kSlots, kRowEmpty = kRowFull + kAhead,
  kSegFull = kRowEmpty + kAhead, kTabFull = kSegFull + kSegs, kQFull = kTabFull + kTabs, kSFull0, kSFull1, kPFull, kPVDone, kEpiDone, kDrain, kNumBars
};
static_assert(kNumBars * 8 <= 480 && sizeof(PagedSegment) <= 64, "barriers");

constexpr uint32_t kIdescQK = idesc_bf16(64, 64, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16(128, 64, 1, 1);

// MMAs and commits by one elected lane of a converged warp.  The election gives
// the same lane each time, so that the commits cover the MMAs.  A chunk's MMAs
// are one statement, with the low words of the descriptors (the high words are
// the same): da and db in 16-byte units, and what each MMA adds to them.
// (go = 0 issues nothing)
#define DS4A_MMA(off, pred)                                                            \
  " add.u32 x, %1, " #off ";\n add.u32 y, %2, " #off ";\n"                             \
  " mov.b64 da, {x, %3};\n mov.b64 db, {y, %3};\n"                                     \
  " @q tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, " pred ";\n"
// S^T += 128 dims: eight MMAs, 32 bytes of a 128-byte row each, then the next 64 dims' block
__device__ __forceinline__ void mma_qk_chunk(uint32_t d_tmem, uint32_t da, uint32_t db, uint32_t hi, uint32_t idesc,
                                             uint32_t accumulate, uint32_t go) {
  asm volatile(
      "{\n .reg .pred p, t, q, g;\n .reg .b64 da, db;\n .reg .b32 x, y;\n"
      " setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 g, %6, 0;\n and.pred q, q, g;\n"
      DS4A_MMA(0, "p") DS4A_MMA(2, "t") DS4A_MMA(4, "t") DS4A_MMA(6, "t")
      DS4A_MMA(512, "t") DS4A_MMA(514, "t") DS4A_MMA(516, "t") DS4A_MMA(518, "t")
      "}\n" ::"r"(d_tmem), "r"(da), "r"(db), "r"(hi), "r"(idesc), "r"(accumulate), "r"(go)
      : "memory");
}
// O^T of 128 dims += 64 keys: four MMAs, 16 keys each
__device__ __forceinline__ void mma_pv_chunk(uint32_t d_tmem, uint32_t da, uint32_t db, uint32_t hi, uint32_t idesc,
                                             uint32_t accumulate, uint32_t go) {
  asm volatile(
      "{\n .reg .pred p, t, q, g;\n .reg .b64 da, db;\n .reg .b32 x, y;\n"
      " setp.ne.b32 p, %5, 0;\n setp.eq.b32 t, 0, 0;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 g, %6, 0;\n and.pred q, q, g;\n"
      DS4A_MMA(0, "p") DS4A_MMA(128, "t") DS4A_MMA(256, "t") DS4A_MMA(384, "t")
      "}\n" ::"r"(d_tmem), "r"(da), "r"(db), "r"(hi), "r"(idesc), "r"(accumulate), "r"(go)
      : "memory");
}
#undef DS4A_MMA
__device__ __forceinline__ void mma_commit_elect(uint32_t bar, uint32_t go = 1u) {
  asm volatile(
      "{\n .reg .pred q, g;\n elect.sync _|q, 0xffffffff;\n setp.ne.b32 g, %1, 0;\n and.pred q, q, g;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar),
      "r"(go)
      : "memory");
}

// S^T of M = 64: 16 lanes x 32 columns; thread t gets, of each 8 columns j,
// v[4j], v[4j + 1]: lane t / 4, columns 2 (t % 4), + 1; v[4j + 2], v[4j + 3]:
// lane t / 4 + 8, the same columns
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// smem -> global, 16-byte aligned, in the thread's bulk group
__device__ __forceinline__ void bulk_s2g(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t src) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
  return v;
}

// the low half at dst, the high half kPitch behind it
template <uint32_t kPitch>
__device__ __forceinline__ void st_shared_halves(uint32_t dst, uint32_t v) {
  asm volatile("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n st.shared.b16 [%0], l;\n st.shared.b16 [%0 + %2], h;\n}\n" ::"r"(dst),
               "r"(v), "n"(kPitch)
               : "memory");
}

// Arrive on the mbarrier when this thread's cp.async so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// 16 bytes, or (bytes = 0) zeros without a read
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1) paged_attend_tc_kernel(const __grid_constant__ PagedArgs a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* smem =
      reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t sbase = smem_u32(smem);
  const uint32_t kv_base = sbase + kOffKV, q_base = sbase + kOffQ, p_base = sbase + kOffP;
  auto bar = [&](int i) { return sbase + kOffBar + 8u * (uint32_t)i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffMisc + 8);
  unsigned long long* rows = reinterpret_cast<unsigned long long*>(smem + kOffRow);
  float* red = reinterpret_cast<float*>(smem + kOffRed);
  float* mrun = reinterpret_cast<float*>(smem + kOffMrun);
  float* alpha_s = reinterpret_cast<float*>(smem + kOffAlpha);
  float* inv_s = reinterpret_cast<float*>(smem + kOffInv);
  float* sink_s = reinterpret_cast<float*>(smem + kOffSink);
  float2* rope_s = reinterpret_cast<float2*>(smem + kOffRope);

  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (the same in the warp, as the compiler sees it)
  unsigned int* err = a.err;

  pdl_trigger();
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(bar(kKVLanded + i), kFp8 ? kGather / 2 : kGather);
      mbar_init(bar(kKVFull + i), 1);
      mbar_init(bar(kKVEmpty + i), 1);
    }
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(bar(kRowFull + i), kKT);
      mbar_init(bar(kRowEmpty + i), kGather + 64);  // the gatherers, and 64 softmax threads for all
    }
    for (int i = 0; i < kSegs; ++i) mbar_init(bar(kSegFull + i), 1);
    for (int i = 0; i < kTabs; ++i) mbar_init(bar(kTabFull + i), 1);
    mbar_init(bar(kQFull), 256);
    mbar_init(bar(kSFull0), 1);
    mbar_init(bar(kSFull1), 1);
    mbar_init(bar(kPFull), 256);
    mbar_init(bar(kPVDone), 1);
    mbar_init(bar(kEpiDone), 256);
    mbar_init(bar(kDrain), 1);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  // Positions and queries are inputs that no kernel of the chain writes: the
  // schedule (unless entries were evicted) and the first q^ are made while the
  // preceding kernel finishes.
  if (a.drop != nullptr) pdl_wait();
  PagedRange* s_range = reinterpret_cast<PagedRange*>(smem + kOffMisc + 16);
  PagedSegment* segs = reinterpret_cast<PagedSegment*>(smem + kOffSeg);
  PagedSegment sg;
  PagedRange r0 = paged_range(a, blockIdx.x, kKT, reinterpret_cast<int*>(smem + kOffKV), kSlots * kSlot / 4,
                              reinterpret_cast<int*>(smem + kOffRed));
  if (warp == 0) {
    if (!paged_next(a, r0, sg, kKT)) sg.n_tiles = 0;
    if (lane == 0) {
      *s_range = r0;
      segs[0] = sg;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  uint32_t seg = 0;
  auto wait = [&](int b, uint32_t parity) {
    if (!mbar_test(bar(b), parity)) mbar_wait(bar(b), parity, abort_flag, err);
  };
  // the next segment, as the address warps found it
  auto next_seg = [&]() {
    if (seg > 0) {  // (the first is there)
      wait(kSegFull + seg % kSegs, (seg / kSegs - (seg % kSegs == 0)) & 1u);
      if (*abort_flag) return false;
    }
    sg = segs[seg++ % kSegs];
    return sg.n_tiles > 0;
  };

  if (warp < 8) {
    // =================== q^, softmax, epilogue ===================
    const int q4 = warp & 3, hf = warp >> 2;
    const int r = 32 * q4 + lane;  // dim row of O^T within a chunk
    const int key0 = 16 * q4 + (lane >> 2), col0 = 2 * (lane & 3);  // keys key0, key0 + 8; columns col0, + 1 of each 8
    const int st = tid;            // 0..255
    const int h0 = 32 * hf;
    const uint32_t t_lane = tmem + ((uint32_t)(32 * q4) << 16);
    const float scale2 = a.scale * kLog2e;
    const int R = a.R;
    uint32_t gt = 0;
    int4 cut = make_int4(-1, 0, 0, 0);
    bool more = next_seg();
    while (more) {
      const int nh = min(kH, a.H - sg.g * kH);
      const int64_t head0 = (int64_t)sg.b * a.H + sg.g * kH;
      if (sg.cut_last >= 0) cut = make_int4(sg.item, sg.cut_last, sg.slot, 0);
      const float2* rope_t = rope_s + (seg - 1) % kTabs * 128;
      const float* sink_t = sink_s + (seg - 1) % kTabs * 64;
      // q^ = RoPE_pos(RMSNorm(q) g), rounded to bf16 (the MMA's operand), in
      // the K-major operand layout: warp w takes heads w, w + 8, ..., lane l
      // dims 8l .. 8l+7 and 256+8l .., which are copied to where q^ will be and
      // changed there; heads that the group does not have are 0.
      const uint32_t qA = q_base + (uint32_t)(lane >> 3) * 8192u, qB = qA + 4u * 8192u;
      {
        const uint16_t* qrow = a.q + head0 * kD + 8 * lane;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int h = warp + 8 * u;
          const uint32_t sw = sw128((uint32_t)h, (uint32_t)(lane & 7)), bytes = h < nh ? 16u : 0u;
          const uint16_t* src = h < nh ? qrow + h * kD : a.q;
          cp_async16_or_zero(qA + sw, src, bytes);
          cp_async16_or_zero(qB + sw, src + 256, bytes);
        }
        cp_async_commit();
      }
      if (st < kH) mrun[st] = kNoRef;
      {
        float2 g[8], rope[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          g[k] = *reinterpret_cast<const float2*>(a.q_norm_g + 8 * lane + 2 * k);
          g[4 + k] = *reinterpret_cast<const float2*>(a.q_norm_g + 256 + 8 * lane + 2 * k);
        }
        wait(kTabFull + (seg - 1) % kTabs, ((seg - 1) / kTabs) & 1u);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int d = 256 + 8 * lane + 2 * k - (kD - R);
          rope[k] = d >= 0 ? rope_t[d >> 1] : make_float2(1.f, 0.f);
        }
        cp_async_wait<0>();
#pragma unroll 1
        for (int u0 = 0; u0 < 8; u0 += 2) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int h = warp + 8 * (u0 + u);
            const uint32_t sw = sw128((uint32_t)h, (uint32_t)(lane & 7));
            const uint4 va = ld_shared16(qA + sw), vb = ld_shared16(qB + sw);
            const unsigned int wv[8] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const float2 f = bf2x2_to_f2(wv[q]);
              acc = fma_f2(f, f, acc);
            }
            // (a head that is not there: 0 rather than 0 / sqrt(eps))
            const float ss = warp_sum(acc.x + acc.y);
            const float rstd = h < nh ? rsqrtf(ss * (1.f / kD) + a.eps) : 0.f;
            uint32_t pq[8];
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              float2 x = mul_f2(mul_f2(bf2x2_to_f2(wv[q]), make_float2(rstd, rstd)), g[q]);
              if (q >= 4) {
                const float2 cs = rope[q - 4];
                x = fma_f2(make_float2(x.x, x.x), cs, mul_f2(make_float2(x.y, x.y), make_float2(-cs.y, cs.x)));
              }
              pq[q] = f2_to_bf2x2(x.x, x.y);
            }
            st_shared16(qA + sw, pq[0], pq[1], pq[2], pq[3]);
            st_shared16(qB + sw, pq[4], pq[5], pq[6], pq[7]);
          }
        }
      }
      fence_async_smem();
      mbar_arrive(bar(kQFull));
      if (gt == 0) pdl_wait();
      float lpart[8];  // columns col0, + 1 of each 8, both keys
#pragma unroll
      for (int i = 0; i < 8; ++i) lpart[i] = 0.f;
      for (int tile = 0; tile < sg.n_tiles; ++tile) {
        wait(kSFull0 + (gt & 1u), (gt >> 1) & 1u);
        wait(kRowFull + gt % kAhead, (gt / kAhead) & 1u);  // (the tile's addresses)
        tc_fence_after();
        float z[16];
        tmem_ld_16x32(t_lane + (gt & 1u) * 64u + (uint32_t)h0, z);
        // a key slot without a row (zero-filled, so its S^T row is 0) gets
        // -inf through the bias of the scaling FMA
        const unsigned long long* rp = rows + (gt % kAhead) * kKT + key0;
        const float ba = rp[0] != 0 ? 0.f : -INFINITY, bb = rp[8] != 0 ? 0.f : -INFINITY;
        tmem_ld_wait();
        const float2 sc2 = make_float2(scale2, scale2);
        float lead = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 m2 = *reinterpret_cast<const float2*>(mrun + h0 + 8 * j + col0);
          const float2 za = fma_f2(make_float2(z[4 * j], z[4 * j + 1]), sc2, make_float2(ba, ba));
          const float2 zb = fma_f2(make_float2(z[4 * j + 2], z[4 * j + 3]), sc2, make_float2(bb, bb));
          z[4 * j] = za.x;
          z[4 * j + 1] = za.y;
          z[4 * j + 2] = zb.x;
          z[4 * j + 3] = zb.y;
          const float2 da = sub_f2(za, m2), db = sub_f2(zb, m2);
          lead = fmaxf(lead, fmaxf(fmaxf(da.x, da.y), fmaxf(db.x, db.y)));
        }
        const bool rescale = bar_or(1, 256, lead > kRescaleLog2);
        if (hf == 0 && lane < 16) mbar_arrive(bar(kRowEmpty + gt % kAhead));  // every thread has read its keys' addresses
        if (rescale) {
          // the tile's largest logit of each head (lanes of equal lane % 4)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float a0 = fmaxf(z[4 * j], z[4 * j + 2]), a1 = fmaxf(z[4 * j + 1], z[4 * j + 3]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, o));
              a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
            }
            if (lane < 4) *reinterpret_cast<float2*>(red + q4 * 64 + h0 + 8 * j + col0) = make_float2(a0, a1);
          }
          named_bar(1, 256);
          if (st < kH) {
            const float mt = fmaxf(fmaxf(red[st], red[64 + st]), fmaxf(red[128 + st], red[192 + st]));
            const float mo = mrun[st];
            float al = 1.f;
            if (mt > mo + kRescaleLog2) {  // a -inf tile maximum never moves it
              al = exp2f(mo - mt);         // 0 from the no-key reference
              mrun[st] = mt;
            }
            alpha_s[st] = al;
          }
          named_bar(1, 256);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 al = *reinterpret_cast<const float2*>(alpha_s + h0 + 8 * j + col0);
            lpart[2 * j] *= al.x;
            lpart[2 * j + 1] *= al.y;
          }
        }
        if (a.weights && st < kH) a.tile_ref[((int64_t)sg.item * a.item_tiles + sg.tile0 + tile) * kH + st] = mrun[st];
        uint32_t pa[4], pb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 m2 = *reinterpret_cast<const float2*>(mrun + h0 + 8 * j + col0);
          // a -inf logit gives 0 (the reference is always finite); P is
          // rounded to bf16 (the MMA's operand) and summed as rounded
          const float2 da = sub_f2(make_float2(z[4 * j], z[4 * j + 1]), m2);
          const float2 db = sub_f2(make_float2(z[4 * j + 2], z[4 * j + 3]), m2);
          pa[j] = f2_to_bf2x2(ex2_approx(da.x), ex2_approx(da.y));
          pb[j] = f2_to_bf2x2(ex2_approx(db.x), ex2_approx(db.y));
          const float2 l2 = add_f2(make_float2(lpart[2 * j], lpart[2 * j + 1]),
                                   add_f2(bf2x2_to_f2(pa[j]), bf2x2_to_f2(pb[j])));
          lpart[2 * j] = l2.x;
          lpart[2 * j + 1] = l2.y;
        }
        if (tile > 0) {
          // the previous tile's PV must be done before P^T and O^T change
          wait(kPVDone, (gt - 1) & 1u);
          tc_fence_after();
        }
        // heads h0 + 8j .. + 7 are the 16-byte piece 4 hf + j of the key's row
        // (key0 and key0 + 8 share their place in the swizzle)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t at = p_base + sw128((uint32_t)key0, (uint32_t)(4 * hf + j)) + 2u * (uint32_t)col0;
          st_shared32(at, pa[j]);
          st_shared32(at + 1024u, pb[j]);
        }
        if (tile > 0 && rescale) {
          const float4* al4 = reinterpret_cast<const float4*>(alpha_s + h0);
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            // 16 head columns of one 128-dim chunk at a time
            float v[16];
            const uint32_t addr = t_lane + 128u + 64u * (c >> 1) + (uint32_t)h0 + 16u * (c & 1);
            tmem_ld16(addr, v);
            tmem_ld_wait();
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              const float4 a4 = al4[4 * (c & 1) + i4];
              v[4 * i4] *= a4.x;
              v[4 * i4 + 1] *= a4.y;
              v[4 * i4 + 2] *= a4.z;
              v[4 * i4 + 3] *= a4.w;
            }
            tmem_st16(addr, v);
          }
          tmem_st_wait();
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(bar(kPFull));
        ++gt;
      }
      // ---------------- epilogue ----------------
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a0 = lpart[2 * j], a1 = lpart[2 * j + 1];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          a0 += __shfl_xor_sync(0xffffffffu, a0, o);
          a1 += __shfl_xor_sync(0xffffffffu, a1, o);
        }
        if (lane < 4) *reinterpret_cast<float2*>(red + q4 * 64 + h0 + 8 * j + col0) = make_float2(a0, a1);
      }
      named_bar(1, 256);
      float* part = paged_part(a, blockIdx.x, sg.slot);
      if (st < kH) {
        const float l = red[st] + red[64 + st] + red[128 + st] + red[192 + st], m = mrun[st];
        // (a head whose logits are all NaN has no reference either: its sum, NaN, is handed on)
        const bool none = m <= kNoRef && l == 0.f;  // no key counts
        if (sg.whole) {
          const float den = l + exp2f(sink_t[st] - m);
          inv_s[st] = none ? 0.f : 1.f / den;
          if (a.weights) a.lse2[(int64_t)sg.item * kH + st] = none ? INFINITY : m + log2f(den);
        } else {
          part[st] = none ? -INFINITY : m * 0.6931471805599453f;  // natural-log units
          part[kH + st] = l;
        }
      }
      named_bar(1, 256);
      wait(kPVDone, (gt - 1) & 1u);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        const int d = 128 * c + r;
        float v[32];
        tmem_ld32(t_lane + 128u + 64u * c + (uint32_t)h0, v);
        tmem_ld_wait();
        if (sg.whole) {
          if (128 * c + 32 * q4 + 31 >= kD - R) {
            // the rope slice, rotated by -pos: lanes r and r^1 hold dims d and
            // d^1 (x0 cs + x1 sn, -x0 sn + x1 cs)
            float cs = 1.f, sn = 0.f;
            if (d >= kD - R) {
              cs = rope_t[(d - (kD - R)) >> 1].x;
              sn = rope_t[(d - (kD - R)) >> 1].y;
              if (r & 1) sn = -sn;
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = v[i] * cs + __shfl_xor_sync(0xffffffffu, v[i], 1) * sn;
          }
          const float4* inv4 = reinterpret_cast<const float4*>(inv_s + h0);
          const uint32_t at = q_base + (uint32_t)h0 * kStagePitch + 2u * (uint32_t)d;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 s4 = inv4[i];
            st_shared_halves<kStagePitch>(at + 4u * i * kStagePitch, f2_to_bf2x2(v[4 * i] * s4.x, v[4 * i + 1] * s4.y));
            st_shared_halves<kStagePitch>(at + (4u * i + 2u) * kStagePitch, f2_to_bf2x2(v[4 * i + 2] * s4.z, v[4 * i + 3] * s4.w));
          }
        } else if (sg.alone) {  // through the ring, which this only segment has left
#pragma unroll
          for (int i = 0; i < 32; ++i) st_shared32(kv_base + (uint32_t)((h0 + i) * kD + d) * 4u, __float_as_uint(v[i]));
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) part[2 * kH + (h0 + i) * kD + d] = v[i];
        }
      }
      if (!sg.whole && sg.alone) {
        fence_async_smem();
        named_bar(1, 256);
        if (st < 8) {
          bulk_s2g(part + 2 * kH + st * 8 * kD, kv_base + (uint32_t)st * 8u * kD * 4u, 8 * kD * 4);
          bulk_commit();
        }
      }
      tc_fence_before();
      mbar_arrive(bar(kEpiDone));
      const bool staged = sg.whole;
      if (staged) {
        fence_async_smem();
        named_bar(1, 256);
        if (st < nh) {
          bulk_s2g(a.out + (head0 + st) * kD, q_base + (uint32_t)st * kStagePitch, kD * 2);
          bulk_commit();
        }
      }
      more = !sg.alone && next_seg();
      if (staged && st < kH) bulk_wait_read0();  // the stage is read before the next segment's q^ goes in
      named_bar(1, 256);
    }
    pdl_wait();
    if (st == 0) a.cut[blockIdx.x] = cut;
    if (st < kH) bulk_wait0();
  } else if (warp == kMmaWarp) {
    // =================== MMA issuer ===================
    // low words of the descriptors; the strides between 8-row groups, the
    // swizzle and the rest of the high words are the same
    const uint32_t qk_a = (uint32_t)sdesc_sw128(kv_base, 16, 1024), qk_b = (uint32_t)sdesc_sw128(q_base, 16, 1024);
    const uint32_t pv_a = (uint32_t)sdesc_sw128(kv_base, kBlk, 1024), pv_b = (uint32_t)sdesc_sw128(p_base, kBlk, 1024);
    const uint32_t sd_hi = (uint32_t)(sdesc_sw128(kv_base, 16, 1024) >> 32);
    // The whole warp runs this loop and an elected lane issues: with operands
    // that are the same in all lanes an MMA of this shape goes out every 48
    // cycles, what its 6 KiB of shared memory take; from a branch of one lane
    // it was 54 to 90.
    uint32_t gt = 0, active = 0;
    uint32_t qs = 0, qph = 0, ps = 0;  // slot and phase of the next chunk of the first product, slot of the second's
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    // (The first pass is dry: nothing is issued and nothing waits, but the code
    // comes in while the schedule is made; on a busy memory its first pass
    // waits 2 to 3 us for instructions.)
    for (uint32_t go = 0;; go = 1) {
      if (go && !__any_sync(0xffffffffu, next_seg())) break;
      const int n_tiles = go ? __shfl_sync(0xffffffffu, sg.n_tiles, 0) : 1;
      int qc = 0;  // half tiles whose first product is issued
      if (go) wait(kQFull, active & 1u);
      for (int tile = 0; tile < n_tiles; ++tile) {
        const int now = 2 * (tile + 1), end = go ? 2 * min(tile + 2, n_tiles) : 1;
        // the tile's first product, and until P^T comes the next tile's, as it
        // arrives, two chunks at a time (asking costs as much as four MMAs;
        // chunks become full in order, so the second stands for both)
        int q = qc;
        while (q < end) {
          const uint32_t s1 = qs + 1 == kSlots ? 0u : qs + 1, ph1 = s1 == 0 ? qph ^ 1u : qph;
          const uint32_t t = gt + (q >= now ? 1u : 0u);
          if (go) {
            if (q < now) {
              wait(kKVFull + s1, ph1);
            } else if (!__all_sync(0xffffffffu, mbar_test(bar(kKVFull + s1), ph1))) {
              if (__any_sync(0xffffffffu, mbar_test(bar(kPFull), gt & 1u) || *abort_flag)) break;
              continue;
            }
            __syncwarp();
            tc_fence_after();
          }
          const uint32_t d_s = tm + (t & 1u) * 64u, db = qk_b + ((q & 1u) ? 2048u : 0u);
          mma_qk_chunk(d_s, qk_a + qs * (kSlot >> 4), db, sd_hi, kIdescQK, q & 1, go);
          mma_qk_chunk(d_s, qk_a + s1 * (kSlot >> 4), db + 1024u, sd_hi, kIdescQK, 1, go);
          mma_commit_elect(bar(kSFull0 + (t & 1u)), go & q);
          if (go) {
            qph = s1 + 1 == kSlots ? ph1 ^ 1u : ph1;
            qs = s1 + 1 == kSlots ? 0u : s1 + 1;
          }
          ++q;
        }
        if (go) {
          qc = q;
          wait(kPFull, gt & 1u);
          if (tile == 0 && active > 0) wait(kEpiDone, (active - 1) & 1u);
          __syncwarp();
          tc_fence_after();
          if (a.weights && lane == 0) {  // P^T as it lies, for the weights
            bulk_s2g(a.tile_p + ((int64_t)sg.item * a.item_tiles + sg.tile0 + tile) * kKT * kH, p_base, kKT * kH * 2);
            bulk_commit();
          }
          __syncwarp();
        }
        const uint32_t acc0 = tile == 0 ? 0u : 1u;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mma_pv_chunk(tm + 128u + 64u * c, pv_a + ps * (kSlot >> 4), pv_b, sd_hi, kIdescPV, acc0, go);
          mma_commit_elect(bar(kKVEmpty + ps), go);
          ps += go;
          if (ps == kSlots) ps = 0;
        }
        if (go && a.weights) {
          if (lane == 0) bulk_wait_read0();  // before P^T changes
          __syncwarp();
        }
        mma_commit_elect(bar(kPVDone), go);
        if (!go) pdl_wait();
        gt += go;
      }
      active += go;
    }
    pdl_wait();
    // drain: every MMA issued has finished before the block exits
    mma_commit_elect(bar(kDrain));
    mbar_wait(bar(kDrain), 0, abort_flag, err);
    if (lane == 0) bulk_wait0();
    __syncwarp();
  } else if (tid < kPG0) {
    // =================== row addresses ===================
    // (positions and the table are inputs; the listed slots a kernel may have
    // just written)
    const int key = tid - kPtr0;  // 0..63
    uint32_t gt = 0;
    PagedRange walk = *s_range;
    sg = segs[0];
    bool more = sg.n_tiles > 0;
    while (more) {
      if (a.sparse && gt == 0) pdl_wait();
      // the segment's query into L2 as well, a head a thread
      if (key < min(kH, a.H - sg.g * kH)) prefetch_l2_bulk(a.q + ((int64_t)sg.b * a.H + sg.g * kH + key) * kD, kD * 2u);
      for (int tile = 0; tile < sg.n_tiles; ++tile, ++gt) {
        const int j = (sg.tile0 + tile) * kKT + key;
        bool fp8 = false;
        const uint8_t* row = j < sg.seq.n_keys ? paged_key(a, sg.b, sg.seq, j, &fp8) : nullptr;
        if (row) prefetch_l2_bulk(row, fp8 ? (uint32_t)a.row_bytes : kD * 2u);
        if (gt >= kAhead) wait(kRowEmpty + gt % kAhead, (gt / kAhead - 1) & 1u);
        rows[(gt % kAhead) * kKT + key] = reinterpret_cast<unsigned long long>(row) | (fp8 ? 1ull : 0ull);
        mbar_arrive(bar(kRowFull + gt % kAhead));
      }
      more = paged_next(a, walk, sg, kKT);
      ++seg;
      if (key == 0) {
        if (!more) sg.n_tiles = 0;
        segs[seg % kSegs] = sg;
        mbar_arrive(bar(kSegFull + seg % kSegs));
      }
    }
  } else if (warp != kFenceWarp) {
    // =================== gather ===================
    pdl_wait();
    const int pt = tid - kPG0;  // 0..255
    int left = 0;               // tiles of the segment
    auto next_tile = [&]() {
      if (left == 0) {
        if (!next_seg()) return false;
        left = sg.n_tiles;
      }
      --left;
      return true;
    };
    auto acquire = [&](uint32_t u) {  // chunk u's slot
      if (u >= kSlots) wait(kKVEmpty + u % kSlots, (u / kSlots - 1) & 1u);
    };
    if (!kFp8) {
      // a thread takes the 16-byte piece pt % 16 of four rows' 256 bytes; a
      // key without a row gets zeros (no branch: the copies go out together)
      constexpr int kN = kKT * 16 / kGather;
      const int piece = pt & 15, row0 = pt >> 4;
      // (rows 16 apart share their place in the swizzle)
      const uint32_t at = (uint32_t)(piece >> 3) * kBlk + sw128(row0, piece & 7);
      for (uint32_t gt = 0; next_tile(); ++gt) {
        const uint32_t rs = gt % kAhead;
        wait(kRowFull + rs, (gt / kAhead) & 1u);
        const uint16_t* src[kN];
        uint32_t bytes[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const unsigned long long v = rows[rs * kKT + row0 + (kGather / 16) * i];
          bytes[i] = v ? 16u : 0u;
          src[i] = (v ? reinterpret_cast<const uint16_t*>(v) : a.q) + piece * 8;
        }
        mbar_arrive(bar(kRowEmpty + rs));
        for (int c = 0; c < 4; ++c) {
          const uint32_t u = 4 * gt + c;
          acquire(u);
          const uint32_t dst = kv_base + (u % kSlots) * kSlot + at;
#pragma unroll
          for (int i = 0; i < kN; ++i) cp_async16_or_zero(dst + (kGather / 16) * 128u * i, src[i] + c * 128, bytes[i]);
          cp_async_arrive(bar(kKVLanded + u % kSlots));
        }
      }
      cp_async_wait<0>();  // nothing of this block is in flight at exit
    } else {
      // FP8 rows: two warps a chunk, a thread 16 dims of eight rows.  The codes
      // are loaded a tile ahead, when the tile's own have been expanded (code
      // times the block's power of two, exact in bf16) and stored; the RoPE
      // dims and the window's rows are bf16 and copied as they are.
      constexpr int kN = 8;
      const int c = pt >> 6, p8 = pt & 7, row0 = (pt >> 3) & 7;  // rows row0 + 8 i (which share their place in the swizzle)
      const bool rope = c == 3 && p8 >= 4;  // dims 448 + 16 (p8 - 4) ..
      uint4 w[kN];
      uint32_t sc[kN];
      auto load = [&](uint32_t gt) {
        const uint32_t rs = gt % kAhead;
        wait(kRowFull + rs, (gt / kAhead) & 1u);
        if (rope) return;
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const unsigned long long v = rows[rs * kKT + row0 + 8 * i];
          if (v & 1ull) {
            const uint8_t* src = reinterpret_cast<const uint8_t*>(v & ~1ull);
            w[i] = *reinterpret_cast<const uint4*>(src + c * 128 + p8 * 16);
            sc[i] = src[kD + 64 + 4 * c + (p8 >> 1)];
          }
        }
      };
      const uint32_t blk = (uint32_t)(p8 >> 2) * kBlk;
      const uint32_t at0 = blk + sw128(row0, (2 * p8) & 7), at1 = blk + sw128(row0, ((2 * p8) & 7) + 1);
      bool have = next_tile();
      if (have) load(0);
      for (uint32_t gt = 0; have; ++gt) {
        const uint32_t u = 4 * gt + c, slot = kv_base + (u % kSlots) * kSlot;
        acquire(u);
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const unsigned long long v = rows[(gt % kAhead) * kKT + row0 + 8 * i];
          const uint32_t d0 = slot + at0 + 1024u * i, d1 = slot + at1 + 1024u * i;
          if ((v & 1ull) && !rope) {
            const float s = mx_scale((int)sc[i]);
            const uint32_t wd[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float2 f = mul_f2(e4m3x2_to_f2(wd[k >> 1] >> (16 * (k & 1))), make_float2(s, s));
              o[k] = f2_to_bf2x2(f.x, f.y);
            }
            st_shared16(d0, o[0], o[1], o[2], o[3]);
            st_shared16(d1, o[4], o[5], o[6], o[7]);
          } else {
            const uint8_t* src = reinterpret_cast<const uint8_t*>(v & ~1ull) +
                                 ((v & 1ull) ? 448 + (p8 - 4) * 32 : c * 256 + p8 * 32);
            cp_async16_or_zero(d0, v ? src : reinterpret_cast<const uint8_t*>(a.q), v ? 16u : 0u);
            cp_async16_or_zero(d1, v ? src + 16 : reinterpret_cast<const uint8_t*>(a.q), v ? 16u : 0u);
          }
        }
        mbar_arrive(bar(kRowEmpty + gt % kAhead));
        mbar_arrive(bar(kKVLanded + u % kSlots));
        cp_async_arrive(bar(kKVLanded + u % kSlots));
        have = next_tile();
        if (have) load(gt + 1);
      }
      cp_async_wait<0>();
    }
  } else {
    // =================== landed rows to the MMAs ===================
    // The rows are written in the generic proxy.  The fence between the proxies
    // costs 0.2 us a chunk in the issuing warp; here it is off its path.
    // It also makes the tables of a segment, ahead of the softmax.
    uint32_t u = 0;
    while (next_seg()) {
      const uint32_t tab = (seg - 1) % kTabs;
      const int nh = min(kH, a.H - sg.g * kH);
      float2* rope_t = rope_s + tab * 128;
      float* sink_t = sink_s + tab * 64;
      float snk[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) snk[i] = lane + 32 * i < nh ? a.sink[sg.g * kH + lane + 32 * i] : 0.f;
#pragma unroll 1
      for (int i = lane; i < a.R / 2; i += 32) {
        float cs, sn;
        rope_cos_sin(sg.seq.pos, a.rope.t[i], &cs, &sn);
        rope_t[i] = make_float2(cs, sn);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) sink_t[lane + 32 * i] = snk[i] * kLog2e;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kTabFull + tab));
      for (int i = 4 * sg.n_tiles; i > 0; --i, ++u) {
        wait(kKVLanded + u % kSlots, (u / kSlots) & 1u);
        fence_async_smem();
        if (lane == 0) mbar_arrive(bar(kKVFull + u % kSlots));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace

// FP8 rows: 448 codes in blocks of 32 and 64 RoPE dims, as the gather reads them
bool paged_tc_supported(const PagedArgs& a, int fmt) {
  return a.D == kD && (a.R % 2) == 0 && a.R <= 256 && (fmt == 0 || a.R == 64);
}

void paged_shape_tc(PagedArgs* a) {
  a->hn = kH;
  a->kt = kKT;
  a->G = 148;
}

cudaError_t launch_paged_attend_tc(const PagedArgs& a, cudaStream_t s) {
  static std::atomic<int> cache[kMaxDevices], cache8[kMaxDevices];
  const bool fp8 = a.fmt != 0;
  const cudaError_t e = fp8 ? ensure_smem(paged_attend_tc_kernel<true>, (int)kSmemBytes, cache8)
                            : ensure_smem(paged_attend_tc_kernel<false>, (int)kSmemBytes, cache);
  if (e != cudaSuccess) return e;
  TraceScope tr("paged_attend_tc", s);
  return fp8 ? launch_pdl(paged_attend_tc_kernel<true>, dim3(a.G), dim3(kThreads), kSmemBytes, s, a)
             : launch_pdl(paged_attend_tc_kernel<false>, dim3(a.G), dim3(kThreads), kSmemBytes, s, a);
}

}  // namespace ds4a
