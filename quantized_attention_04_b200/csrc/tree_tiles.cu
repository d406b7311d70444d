// Attention of drafted tokens over a paged cache, many rows: k_tree_tiles.
//
// Row tiles of 128 against key tiles of 64 on the 5th-generation tensor cores.
// A block holds two row tiles ("slots", eight softmax warps each):
//   SHARE   (more than 128 rows a pair): both slots walk the same run of key
//           tiles with the two halves of up to 256 rows; K and V are loaded once.
//   !SHARE  (up to 128 rows): each slot has a run of its own, as if it were a
//           block, and its own K and V tiles.
// Per slot and key tile: S = Q K^T (both in shared memory, fp32 S in TMEM), softmax,
// P (16 bits) written over S in TMEM, O += P V with P as the TMEM operand and V as it is
// cached ([key][d], the "MN-major" form), O in TMEM for the whole run of a pair.  S is
// double-buffered: S of the next tile is there when the softmax of this one ends, so
// that the exponentials (16 a cycle and SM: 1024 cycles for 256 rows x 64 keys) and
// the tensor cores (as many for both products, d = 128) run side by side.
//
// The softmax passes over S once: exponentials are taken against the reference
// left by the earlier keys, and only if some score of the warp's rows lies far above
// it (kRefGrow) the reference moves, and O and the row sums are rescaled.  A P above 1
// keeps its relative precision.
//
// 16-bit caches: K and V arrive by TMA, a box a page.  e4m3 caches: eight warps load
// the codes (16 bytes a lane, in registers), widen them to fp16
// (exact) and store them in the same layout, while a warp ahead of them brings the rows
// into L2.  Q enters as fp16 scaled by a power of two a row; the key scales multiply
// the scores and the value scales multiply P, whose reference is the largest of score +
// log2(value scale) among the keys that the row attends.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_index.h"
#include "sage2.h"
#include "sage2_internal.h"
#include "sm100_ptx.cuh"

namespace sage2 {

constexpr int kTR = 128;                  // rows of a slot
constexpr int kTK = 64;                   // keys of a tile
constexpr int kTAhead = 8;                // tiles between the L2 prefetch and the loaders
// Warps: 16 softmax, 4 loaders (one a ring; e4m3: 8, 4 or 2 a ring), 2 MMA warps, with e4m3 one
// that prefetches and one that loads the scales.
template <bool E4M3>
constexpr int kTLoad = E4M3 ? 8 : 4;
template <bool E4M3>
constexpr int kTThreads = (16 + kTLoad<E4M3> + 4) * 32;

template <int D, bool E4M3>
struct TilesCfg {
  static constexpr int kBlk = D / 64;                    // 128-byte blocks of a row
  static constexpr int kQBytes = kTR * D * 2;            // a tile of Q
  static constexpr int kTileBytes = kTK * D * 2;         // a 16-bit tile of K or V
  static constexpr int kBufs = D == 128 ? 8 : 16;        // rings of K and V (SHARE), or of each slot's K and V
  // Tiles of scales that a slot keeps.  When K(t) is stored, K(t - kBufs/2), whose buffer it takes (or
  // a later one), has been freed, so S of it and P V of the second tile before that are done: the
  // softmax reads scales of the kBufs/2 + 2 tiles up to t at most.
  static constexpr int kScales = kBufs;
  static_assert(kScales >= kBufs / 2 + 2, "scales in use");
};

template <int D, bool E4M3>
struct __align__(1024) TilesSmem {
  using C = TilesCfg<D, E4M3>;
  uint8_t q[2][C::kQBytes];
  uint8_t kv[C::kBufs][C::kTileBytes];
  // scales of a slot's last tiles; keys 2i, 2i+1: key scales at 4i, 4i+1, value scales at 4i+2, 4i+3
  float scl[E4M3 ? 2 : 1][C::kScales][E4M3 ? 2 * kTK : 4];
  float lv[E4M3 ? 2 : 1][C::kScales];   // log2 of the tile's largest value scale
  uint64_t full[C::kBufs];   // the loader warps of the ring, with K the scale warp (or the TMA's bytes)
  uint64_t empty[C::kBufs];  // commit of the MMAs that read the buffer (SHARE: of both slots)
  uint64_t tail[C::kBufs];   // bytes of a V tile that is checked before use
  uint64_t q_full[2];        // the slot's eight softmax warps
  uint64_t s_full[2][2];     // the MMA warp (it has seen the tile's scales) and the commit of S
  uint64_t p_full[2][2];     // the slot's eight softmax warps: S read, P written
  uint64_t o_done[2][2];     // commit of O += P V (by the tile's parity, as the two above)
  uint64_t drain[2];
  uint32_t tmem;
  int starts[C::kBufs];      // the K tile is a piece's first
  int bad_v;                 // a drafted token's V row or scale was not finite
  int progress[2];           // by slot: V tiles stored
  int abort_flag;
};

static_assert(sizeof(TilesSmem<128, false>) + 1024 <= 232448 && sizeof(TilesSmem<128, true>) + 1024 <= 232448,
              "shared memory of a block");

// MMAs and commits of one elected lane as predicated instructions: the whole converged warp passes them, so
// that descriptors stay in uniform registers (inside a branch of one lane each operand costs moves).
// D[tmem] (+)= A[tmem] * B[smem], 16-bit A (two values a column), fp32 D.
__device__ __forceinline__ void mma_f16_ts_if(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead));
}
// D[tmem] (+)= A[smem] * B[smem]^T, 16-bit floats.
__device__ __forceinline__ void mma_f16_ss_if(uint32_t lead, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                              uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead));
}
// The same of 8-bit floats.
__device__ __forceinline__ void mma_f8_ss_if(uint32_t lead, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead));
}
__device__ __forceinline__ void tc_commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(lead) : "memory");
}
__device__ __forceinline__ void mbar_arrive_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(lead) : "memory");
}
// Descriptor of a [k][n] operand (n contiguous): 128-byte rows of 64 n, 128-byte
// swizzle, 8-row groups 1024 bytes apart, the next 64 n `block` bytes on.
__device__ __forceinline__ uint64_t smem_desc_nmajor(const void* p, uint32_t block) {
  const uint32_t addr = smem_u32(p);
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(block >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
// Lane 0's value, which the compiler then knows to be alike in all lanes.
template <typename T>
__device__ __forceinline__ T uniform(T x) {
  return __shfl_sync(0xffffffffu, x, 0);
}
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p;
}

// Byte offset of 16-byte chunk `ch` (of D/8) of row `r` in a 16-bit tile of ROWS rows.
template <int ROWS>
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
  return (ch >> 3) * (ROWS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// A warp waits for the phase with the given parity, with no more than a poll and a branch a try: the
// waiting warps share the issue slots with those that work.  Gives up as mbar_wait does.
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  bool ok = mbar_try_wait(bar, parity);
  if (!__all_sync(0xffffffffu, ok)) {
    const uint64_t t0 = globaltimer_ns();
    while (!ok) {
#pragma unroll 1
      for (int i = 0; i < 256 && !ok; ++i) ok = mbar_try_wait(bar, parity);
      if (ok || (abort_flag && *abort_flag)) break;
      if (globaltimer_ns() - t0 > kWaitLimitNs) {
        atomicOr(&g_device_error, DEVERR_TIMEOUT);
        if (abort_flag) *abort_flag = 1;
        break;
      }
    }
    ok = __all_sync(0xffffffffu, ok);
  }
  return ok;
}

// 32 lanes x 16 consecutive columns: thread t gets lane (base + t).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// .16x256b.x4: 16 lanes x 32 columns.  Thread t gets, for k = 0..3, the columns 8k + 2(t%4) + {0,1}
// of lane t/4 (registers 4k, 4k+1) and of lane t/4 + 8 (4k+2, 4k+3).
__device__ __forceinline__ void tmem_ld16x256_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// .16x128b.x8: 16 lanes x 32 columns.  Thread t has, for k = 0..7, column 4k + t%4 of lane t/4
// (register 2k) and of lane t/4 + 8 (2k+1).
__device__ __forceinline__ void tmem_st16x128_16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
      : "memory");
}

// Does the V row of slot `slot`, or one of its scales, hold an infinity or NaN?
template <int D, bool E4M3, bool BF>
__device__ __noinline__ bool v_row_bad(const TreeArgs& a, int b, int h, int slot) {
  const int page = __ldg(a.table + (size_t)b * a.MP + (slot >> a.c.page_shift));
  if (!page_inside(page, a.c.pages)) return false;
  const long long row = row_of(page, a.c.Hkv, h, a.c.page_shift, slot);
  bool bad = E4M3 && !(fabsf(__ldg(a.c.vs + row)) < INFINITY && fabsf(__ldg(a.c.ks + row)) < INFINITY);
  for (int i = 0; i < D * (E4M3 ? 1 : 2) / 16; ++i)
    bad = bad || not_finite16<E4M3, BF>(
                     __ldg(reinterpret_cast<const uint4*>(a.c.v + row * D * (E4M3 ? 1 : 2)) + i));
  return bad;
}

// Scores of an edge tile that the mask or the length leaves out become -inf where they lie (the two rows
// of a thread, drafted tokens i0, i1).
template <int UNROLL>
__device__ __forceinline__ void mask_scores(const TreeArgs& a, SeqLen s, int b, uint32_t tS, int key0, int i0,
                                            int i1) {
  const uint8_t* mask = a.mask ? a.mask + b * a.mask_sb : nullptr;
  const int g = threadIdx.x & 3;
#pragma unroll 1
  for (int c = 0; c < kTK; c += 32) {
    uint32_t bits = 0;
#pragma unroll UNROLL
    for (int y = 0; y < 16; ++y)
      bits |= (slot_allowed(a, mask, s, y & 2 ? i1 : i0, key0 + c + 8 * (y >> 2) + 2 * g + (y & 1)) ? 1u : 0u) << y;
    uint32_t x[16];
    tmem_ld16x256_16(tS + c, x);
    tmem_ld_wait();
#pragma unroll
    for (int y = 0; y < 16; ++y)
      if (!((bits >> y) & 1u)) x[y] = 0xff800000u;
    tmem_st16x256_16(tS + c, x);
  }
  tmem_st_wait();
}

__device__ __noinline__ void mask_scores_apart(const TreeArgs& a, SeqLen s, int b, uint32_t tS, int key0, int i0,
                                               int i1) {
  mask_scores<16>(a, s, b, tS, key0, i0, i1);
}

// The two rows of a thread (.16x256b) of O times f0, f1.  Rare: not inlined, so that the loop that
// calls it keeps its registers.
template <int D>
__device__ __noinline__ void scale_rows(uint32_t o, float f0, float f1) {
#pragma unroll 1
  for (int d0 = 0; d0 < D; d0 += 32) {
    uint32_t y[16];
    tmem_ld16x256_16(o + d0, y);
    tmem_ld_wait();
#pragma unroll
    for (int z = 0; z < 16; ++z) y[z] = __float_as_uint(__uint_as_float(y[z]) * ((z & 2) ? f1 : f0));
    tmem_st16x256_16(o + d0, y);
  }
  tmem_st_wait();
}

// e4m3: where the references of a thread's two rows move to (x, y): the largest of score + log2(value scale)
// among the keys so far; and the factors of their sums and O (z, w).  qs0, qs1: log2 units of a score.  Rare: not
// inlined, and the tile's P is taken anew after it (inlined and with P kept, the loop around it spilled: 1145 us
// instead of 862 for 16 x 48 tokens over 32768 slots).
__device__ __noinline__ float4 moved_refs(uint32_t tS, const float* sc, float qs0, float qs1, float ref0, float ref1) {
  const int g = threadIdx.x & 3;
  float2 top = make_float2(ref0, ref1);
#pragma unroll 1
  for (int c = 0; c < kTK; c += 32) {
    uint32_t x[16];
    tmem_ld16x256_16(tS + c, x);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 f = *reinterpret_cast<const float4*>(sc + 2 * (c + 8 * k + 2 * g));
      const float v0 = vref_log2(f.z), v1 = vref_log2(f.w);
      top.x = max3f(top.x, __uint_as_float(x[4 * k]) * f.x * qs0 + v0, __uint_as_float(x[4 * k + 1]) * f.y * qs0 + v1);
      top.y = max3f(top.y, __uint_as_float(x[4 * k + 2]) * f.x * qs1 + v0,
                    __uint_as_float(x[4 * k + 3]) * f.y * qs1 + v1);
    }
  }
#pragma unroll
  for (int o = 1; o <= 2; o *= 2) {
    top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, o));
    top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, o));
  }
  return make_float4(top.x, top.y, ref0 == -INFINITY ? 0.f : ex2(ref0 - top.x), ref1 == -INFINITY ? 0.f : ex2(ref1 - top.y));
}

template <int D, bool E4M3, bool QBF, bool SHARE>
__global__ void __launch_bounds__(kTThreads<E4M3>, 1)
    k_tree_tiles(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ TreeArgs a, int rows_unit) {
  using C = TilesCfg<D, E4M3>;
  using Smem = TilesSmem<D, E4M3>;
  constexpr int kRing = SHARE ? C::kBufs / 2 : C::kBufs / 4;     // buffers of a ring
  constexpr int kGroup = !E4M3 ? 1 : (SHARE ? 4 : 2);            // loader warps of a ring
  constexpr bool BF = QBF && !E4M3;              // type of the MMA operands
  constexpr int kMma = 16 + kTLoad<E4M3>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = a.G * a.T, pairs = a.c.Hkv * a.RT;
  volatile int* abort_flag = &sm.abort_flag;
  if (tid == 0) {
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&sm.full[i], kGroup + (E4M3 && !((i / kRing) & 1) ? 1 : 0));
      mbar_init(&sm.empty[i], SHARE ? 2 : 1);
      mbar_init(&sm.tail[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 8);
      for (int p = 0; p < 2; ++p) {
        mbar_init(&sm.s_full[s][p], 2);
        mbar_init(&sm.p_full[s][p], 8);
        mbar_init(&sm.o_done[s][p], 1);
      }
    }
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.abort_flag = 0;
    sm.bad_v = 0;
    sm.progress[0] = sm.progress[1] = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  // slot and ring of this warp
  const int ring = warp < 16 ? 0 : (warp < kMma ? (warp - 16) / kGroup : (warp - kMma) * 2);
  const int slot = warp < 16 ? warp >> 3 : (SHARE && warp < kMma ? 0 : ring >> 1);
  auto run_of_slot = [&](int s) {
    return warp_run(a, kTK, pairs, SHARE ? gridDim.x : 2 * gridDim.x, SHARE ? blockIdx.x : 2 * blockIdx.x + s, 1);
  };
  const Run run = run_of_slot(slot & 1);
  if (blockIdx.x == gridDim.x - 1 && warp == kMma + 2) write_before(a, kTK, pairs);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  // registers at launch and by role: 768 x 80 = 512 x 88 + 128 x 64 + 128 x 64, and with e4m3
  // 896 x 72 = 512 x 80 + 256 x 72 + 128 x 40
  constexpr int kRegSoft = E4M3 ? 80 : 88, kRegMma = E4M3 ? 40 : 64;
  if (warp >= 16 && warp < 16 + kTLoad<E4M3>) {
    // ------------------------------------------------------------ loaders
    if (!E4M3) setmaxnreg_dec<64>();
    // One ring of tiles each: (slot 0:) K, V, !SHARE: of slot 1 as well.
    const bool v = ring & 1;
    const int n = ring < (SHARE ? 2 : 4) ? run.n : 0, base = ring * kRing;
    Cursor at;
    if (n > 0) at.start(run, kTK);
    // lane j: the page of the slots from key0 + j * (at most 16) on; -1 behind the last key
    const int chunk = E4M3 ? 16 : min(kTK, 1 << a.c.page_shift);
    auto page_of = [&]() {
      const int key = at.tile * kTK + lane * chunk;
      return lane * chunk < kTK && key < at.s.len + at.s.n
                 ? __ldg(a.table + (size_t)at.b * a.MP + (key >> a.c.page_shift))
                 : -1;
    };
    int page = n > 0 ? page_of() : -1;
    bool ok = true;
    if (!E4M3) {
      unsigned tails = 0;          // parity of the next phase of each buffer's tail barrier
      int t = 0;
      for (; t < n; ++t) {
        const int buf = base + t % kRing;
        const int key0 = at.tile * kTK, len = at.s.len, L = len + at.s.n, h = at.pair / a.RT;
        const bool starts = t == 0 || at.tile == 0, edge = v && key0 + kTK > len;
        const bool in = lane * chunk < kTK && key0 + lane * chunk < L;
        int pg = page;
        if (in && !page_inside(pg, a.c.pages)) {
          atomicOr(&g_device_error, DEVERR_BOUNDS);
          pg = 0;           // any rows: the outputs are not meaningful
        }
        if (t + 1 < n) {
          at.next(a, pairs, kTK);
          page = page_of();
        }
        if (t >= kRing && !tile_wait(&sm.empty[buf], (t / kRing - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        uint64_t* bar = edge ? &sm.tail[buf] : &sm.full[buf];
        uint8_t* dst = sm.kv[buf];
        const int cnt = __popc(__ballot_sync(0xffffffffu, in));
        if (lane == 0) {
          if (!v) sm.starts[buf] = starts;
          mbar_expect_tx(bar, cnt * chunk * D * 2);
        }
        __syncwarp();
        if (in) {
          const int row = (int)row_of(pg, a.c.Hkv, h, a.c.page_shift, key0 + lane * chunk);
#pragma unroll
          for (int x = 0; x < C::kBlk; ++x)
            tma_load_2d(dst + x * kTK * 128 + lane * chunk * 128, v ? &tm_v : &tm_k, bar, x * 64, row);
        }
        if (edge) {
          // rows behind the last key and drafted rows that are not finite become zeros
          if (!tile_wait(&sm.tail[buf], (tails >> (t % kRing)) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tails ^= 1u << (t % kRing);
          for (int r = lane; r < kTK; r += 32) {
            if (key0 + r < len) continue;
            bool zero = key0 + r >= L;
            if (!zero) {
#pragma unroll
              for (int ch = 0; ch < D / 8; ++ch)
                zero = not_finite16<false, QBF>(*reinterpret_cast<const uint4*>(dst + tile_off<kTK>(r, ch))) || zero;
              if (zero) sm.bad_v = 1;
            }
            if (zero)
              for (int ch = 0; ch < D / 8; ++ch)
                *reinterpret_cast<uint4*>(dst + tile_off<kTK>(r, ch)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[buf]);
        }
      }
      if (!ok) {
        // let the copies already issued land before the block exits
        for (int u = t > kRing ? t - kRing : 0; u < t; ++u)
          mbar_wait(&sm.full[base + u % kRing], (u / kRing) & 1, nullptr);
      }
    } else {
      // A row is 8 lanes with 8 bytes each (D = 128: and 8 more 64 codes on), so that they store the 8
      // chunks of a 128-byte line.  In units of NU passes over the tile's rows; one unit is on its way
      // while the one before it is stored.
      constexpr int RPP = 4 * kGroup, NP = kTK / RPP, NU = kGroup == 4 || D == 64 ? NP : NP / 2;
      constexpr int kUnits = NP / NU;
      const int lt = (tid - 16 * 32) % (32 * kGroup), lr = lt >> 3, lc = lt & 7;
      const uint8_t* pool = (v ? a.c.v : a.c.k) + 8 * lc;
      struct Unit {
        uint2 u[NU][C::kBlk];
        int first;                 // row of the tile from which on they are drafted ones
        bool starts;
      };
      int at_t = 0, row16 = -1;    // lane j: row of slot 16 j of the tile
      auto fetch = [&](Unit& x, int sub) {
        if (at_t >= n) return;
        const int key0 = at.tile * kTK, L = at.s.len + at.s.n;
        if (sub == 0) {
          row16 = -1;
          if (lane < kTK / 16 && key0 + 16 * lane < L) {
            if (page_inside(page, a.c.pages))
              row16 = (int)row_of(page, a.c.Hkv, at.pair / a.RT, a.c.page_shift, key0 + 16 * lane);
            else
              atomicOr(&g_device_error, DEVERR_BOUNDS);
          }
        }
        x.first = at.s.len - key0;
        x.starts = at_t == 0 || at.tile == 0;
        const bool full = key0 + kTK <= L && __all_sync(0xffffffffu, lane >= kTK / 16 || row16 >= 0);
#pragma unroll
        for (int p = 0; p < NU; ++p) {
          const int r = (sub * NU + p) * RPP + lr, row = __shfl_sync(0xffffffffu, row16, r >> 4);
          const uint2* src = reinterpret_cast<const uint2*>(pool + (size_t)(uint32_t)(row + (r & 15)) * D);
#pragma unroll
          for (int c = 0; c < C::kBlk; ++c) {
            if (full) x.u[p][c] = __ldg(src + 8 * c);
            else x.u[p][c] = row >= 0 && key0 + r < L ? __ldg(src + 8 * c) : make_uint2(0u, 0u);
          }
        }
        if (sub == kUnits - 1 && ++at_t < n) {
          at.next(a, pairs, kTK);
          page = page_of();
        }
      };
      const uint32_t off = tile_off<kTK>(lr, lc);      // of row r + 8 i: 1024 i more
      auto put = [&](Unit& x, int t, int sub) -> bool {
        const int buf = base + t % kRing;
        if (sub == 0 && t >= kRing && !tile_wait(&sm.empty[buf], (t / kRing - 1) & 1, abort_flag)) return false;
        uint8_t* dst = sm.kv[buf] + off;
        if (sub == 0 && !v && lt == 0) sm.starts[buf] = x.starts;
        if (v && x.first < kTK) {
          // drafted rows that are not finite become zeros
#pragma unroll
          for (int p = 0; p < NU; ++p) {
            const int r = (sub * NU + p) * RPP + lr;
            unsigned bad = 0;
#pragma unroll
            for (int c = 0; c < C::kBlk; ++c)
              bad |= not_finite16<true, false>(make_uint4(x.u[p][c].x, x.u[p][c].y, 0u, 0u)) ? 1u : 0u;
#pragma unroll
            for (int o = 4; o; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
            if (bad && r >= x.first) {
#pragma unroll
              for (int c = 0; c < C::kBlk; ++c) x.u[p][c] = make_uint2(0u, 0u);
              sm.bad_v = 1;
            }
          }
        }
#pragma unroll
        for (int p = 0; p < NU; ++p)
#pragma unroll
          for (int c = 0; c < C::kBlk; ++c) {
            uint4 w;
            widen4(x.u[p][c].x, w.x, w.y);
            widen4(x.u[p][c].y, w.z, w.w);
            *reinterpret_cast<uint4*>(dst + (sub * NU + p) * RPP * 128 + c * (kTK * 128)) = w;
          }
        if (sub == kUnits - 1) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[buf]);
          if (v && lt == 0) *static_cast<volatile int*>(&sm.progress[slot]) = t;
        }
        return true;
      };
      Unit x0, x1;
      fetch(x0, 0);
      if (kUnits == 1) {
        for (int t = 0; t < n; t += 2) {
          fetch(x1, 0);
          if (!put(x0, t, 0)) break;
          if (t + 1 == n) break;
          fetch(x0, 0);
          if (!put(x1, t + 1, 0)) break;
        }
      } else {
        for (int t = 0; t < n; ++t) {
          fetch(x1, 1);
          if (!put(x0, t, 0)) break;
          fetch(x0, 0);
          if (!put(x1, t, kUnits - 1)) break;
        }
      }
    }
  } else if (warp >= 16) {
    // ------------------------------------------------------------ MMA issuer
    setmaxnreg_dec<kRegMma>();
    if (warp < kMma + 2) {
      // One warp a slot.  The whole warp walks the tiles with values that the compiler knows to be
      // alike in all lanes (shuffled from lane 0), so that descriptors and addresses live in
      // uniform registers, and one elected lane issues.  This warp's instructions are
      // on the path of every tile: what it would have to work out (which tile starts a piece)
      // comes with the tile.
      constexpr uint32_t idesc_s = idesc_f16_f32(kTR, kTK, BF);
      constexpr uint32_t idesc_o = idesc_f16_f32(kTR, D, BF) | (1u << 16);   // B is [k][n]
      constexpr uint32_t kBuf16 = C::kTileBytes >> 4;
      const int s = uniform(warp - kMma);
      const int kb0 = (SHARE ? 0 : 2 * s) * kRing, vb0 = kb0 + kRing;      // the rings' first buffers
      const uint64_t dk0 = smem_desc_kmajor(sm.kv[kb0], 128);
      const uint64_t dv0 = smem_desc_nmajor(sm.kv[vb0], kTK * 128);
      const uint32_t k_hi = uniform((uint32_t)(dk0 >> 32)), k_lo = uniform((uint32_t)dk0);
      const uint32_t v_hi = uniform((uint32_t)(dv0 >> 32)), v_lo = uniform((uint32_t)dv0);
      const uint32_t q_lo = uniform((uint32_t)smem_desc_kmajor(sm.q[s], 128));
      const uint32_t tm = uniform(tmem) + s * 128, to = uniform(tmem) + 256 + s * 128;
      const uint32_t leader = elect_one();
      const int n = uniform(run.n);
      int first = 0;               // bit p: the last tile of parity p starts a piece
      int q_ph = 0;
      // S of tile k, whose K has landed
      auto scores = [&](int k, int buf, int start) -> bool {
        const int p = k & 1;
        if (start) {
          if (!tile_wait(&sm.q_full[s], q_ph, abort_flag)) return false;
          q_ph ^= 1;
        }
        first = (first & ~(1 << p)) | (start << p);
        tc_fence_after();
        const uint32_t kb = uniform(k_lo + buf * kBuf16);
        mbar_arrive_if(leader, &sm.s_full[s][p]);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_f16_ss_if(leader, tm + p * 64, desc_of(q_lo + (kk >> 2) * ((kTR * 128) >> 4) + (kk & 3) * 2, k_hi),
                        desc_of(kb + (kk >> 2) * ((kTK * 128) >> 4) + (kk & 3) * 2, k_hi), idesc_s, kk > 0);
        tc_commit_if(leader, &sm.s_full[s][p]);
        tc_commit_if(leader, &sm.empty[kb0 + buf]);
        __syncwarp();
        return true;
      };
      // S(t+2) follows P V of t, whose P it overwrites.  A tile that starts a piece waits until every
      // P V of the piece before is issued (its Q is loaded after that piece's softmax), the ones
      // behind it wait for it.
      int ns = 0;
      bool ok = true;
#pragma unroll 1
      for (int t = -1; ok && t < n; ++t) {
        if (t >= 0) {
          const int p = t & 1, buf = t % kRing;
          if (!tile_wait(&sm.p_full[s][p], (t >> 1) & 1, abort_flag) ||
              !tile_wait(&sm.full[vb0 + buf], (t / kRing) & 1, abort_flag))
            break;
          tc_fence_after();
          const uint32_t vb = uniform(v_lo + buf * kBuf16), keep = ((first >> p) & 1) ^ 1;
#pragma unroll
          for (int kk = 0; kk < kTK / 16; ++kk)
            mma_f16_ts_if(leader, to, tm + p * 64 + 8 * kk, desc_of(vb + kk * (16 * 128 >> 4), v_hi), idesc_o,
                          kk > 0 ? 1u : keep);
          tc_commit_if(leader, &sm.o_done[s][p]);
          tc_commit_if(leader, &sm.empty[vb0 + buf]);
          __syncwarp();
        }
#pragma unroll 1
        while (ns < n && ns <= t + 2) {
          const int buf = ns % kRing;
          if (!tile_wait(&sm.full[kb0 + buf], (ns / kRing) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const int start = uniform(sm.starts[kb0 + buf]);
          if (start && ns != t + 1) break;
          if (!scores(ns, buf, start)) {
            ok = false;
            break;
          }
          ++ns;
        }
      }
      // every MMA issued so far completes before the block frees TMEM
      tc_commit_if(leader, &sm.drain[s]);
      __syncwarp();
      tile_wait(&sm.drain[s], 0, nullptr);
    } else if (E4M3 && warp == kMma + 2) {
      // the rows of the tiles ahead, to L2: a 128-byte line (D = 64: half of one) a row
      const Run r0 = run_of_slot(0), r1 = SHARE ? r0 : run_of_slot(1);
      Cursor c0, c1;
      if (r0.n > 0) c0.start(r0, kTK);
      if (!SHARE && r1.n > 0) c1.start(r1, kTK);
      for (int t = 0; t < max(r0.n, r1.n); ++t) {
#pragma unroll
        for (int s = 0; s < (SHARE ? 1 : 2); ++s) {
          if (t >= (s ? r1.n : r0.n)) continue;
          Cursor& c = s ? c1 : c0;
          // no further ahead of the loaders than kTAhead tiles (a bounded wait: running ahead is no fault)
          for (int x = 0; x < 100000 && !*abort_flag; ++x) {
            if (*static_cast<volatile int*>(&sm.progress[s]) + kTAhead >= t) break;
            __nanosleep(100);
          }
          __syncwarp();
          const int L = c.s.len + c.s.n, h = c.pair / a.RT;
#pragma unroll
          for (int x = 0; x < kTK; x += 32) {
            const int key = c.tile * kTK + x + lane;
            const int page = key < L ? __ldg(a.table + (size_t)c.b * a.MP + (key >> a.c.page_shift)) : -1;
            if (page_inside(page, a.c.pages)) {
              const long long row = row_of(page, a.c.Hkv, h, a.c.page_shift, key);
              prefetch_l2(a.c.k + row * D);
              prefetch_l2(a.c.v + row * D);
              if (lane % 16 == 0) {
                prefetch_l2(a.c.ks + row);
                prefetch_l2(a.c.vs + row);
              }
            }
          }
          if (t + 1 < (s ? r1.n : r0.n)) c.next(a, pairs, kTK);
        }
      }
    } else if (E4M3 && warp == kMma + 3) {
      // the scales, two keys a lane; those of the next tile are on their way while these are stored
      const Run r0 = run_of_slot(0), r1 = SHARE ? r0 : run_of_slot(1);
      Cursor c0, c1;
      struct Ahead {
        float2 ks, vs;
        int page, key, len, L;
      };
      Ahead x0, x1;
      auto page_at = [&](const Cursor& c, Ahead& x) {       // the page of the cursor's tile
        x.key = c.tile * kTK + 2 * lane;
        x.len = c.s.len;
        x.L = x.len + c.s.n;
        x.page = x.key < x.L ? __ldg(a.table + (size_t)c.b * a.MP + (x.key >> a.c.page_shift)) : -1;
      };
      auto fetch = [&](const Cursor& c, Ahead& x) {
        x.ks = x.vs = make_float2(0.f, 0.f);
        if (page_inside(x.page, a.c.pages)) {
          const long long row = row_of(x.page, a.c.Hkv, c.pair / a.RT, a.c.page_shift, x.key);
          x.ks = __ldg(reinterpret_cast<const float2*>(a.c.ks + row));
          x.vs = __ldg(reinterpret_cast<const float2*>(a.c.vs + row));
        }
      };
      if (r0.n > 0) {
        c0.start(r0, kTK);
        page_at(c0, x0);
        fetch(c0, x0);
      }
      if (!SHARE && r1.n > 0) {
        c1.start(r1, kTK);
        page_at(c1, x1);
        fetch(c1, x1);
      }
      bool go = true;
      for (int t = 0; go && t < max(r0.n, r1.n); ++t) {
#pragma unroll
        for (int s = 0; s < (SHARE ? 1 : 2); ++s) {
          const int n = s ? r1.n : r0.n;
          if (!go || t >= n) continue;
          Cursor& c = s ? c1 : c0;
          Ahead& x = s ? x1 : x0;
          const int buf = 2 * s * kRing + t % kRing;
          Ahead y = x;
          if (t + 1 < n) {
            c.next(a, pairs, kTK);
            page_at(c, x);
          }
          // masked scores are -inf before the key scale multiplies them, and P is 0 before the value
          // scale does: the scales of drafted rows become finite, a key's not 0 (a row of scale 0
          // has codes 0); those behind the last key are 1 and 0
          auto clean = [&](float w, bool is_key, int k) {
            if (k < y.len) return w;
            if (k >= y.L) w = 0.f;
            if (!(fabsf(w) < INFINITY)) {
              w = 0.f;
              sm.bad_v = 1;
            }
            return is_key && w == 0.f ? 1.f : w;
          };
          if (y.key + 2 > y.len) {
            y.ks.x = clean(y.ks.x, true, y.key);
            y.ks.y = clean(y.ks.y, true, y.key + 1);
            y.vs.x = clean(y.vs.x, false, y.key);
            y.vs.y = clean(y.vs.y, false, y.key + 1);
          }
          float m = fmaxf(y.vs.x, y.vs.y);
#pragma unroll
          for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          if (t + 1 < n) fetch(c, x);
          if (t >= kRing && !tile_wait(&sm.empty[buf], (t / kRing - 1) & 1, abort_flag)) {
            go = false;
            continue;
          }
          *reinterpret_cast<float4*>(sm.scl[s][t % C::kScales] + 4 * lane) =
              make_float4(y.ks.x, y.ks.y, y.vs.x, y.vs.y);
          if (lane == 0) sm.lv[s][t % C::kScales] = log2f(fmaxf(m, kVrefLeast));
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[buf]);
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    // Eight warps a slot.  The .16x256b loads give a warp 16 TMEM lanes and each of its
    // quads two rows, t/4 and t/4 + 8, so that four warps share a scheduler.  Row r
    // of the slot is on lane 32 (r/16 % 4) + 16 (r/64) + r%16: any number of rows is
    // spread evenly over the schedulers.
    setmaxnreg_inc<kRegSoft>();
    const int s = warp >> 3, quad = warp & 3, hf = (warp >> 2) & 1, g = lane & 3;
    const int lo = (SHARE ? s * kTR : 0) + 64 * hf + 16 * quad + (lane >> 2);   // of the unit's rows: lo, lo + 8
    const int ml = 32 * quad + 16 * hf + (lane >> 2);                           // TMEM lane: ml, ml + 8
    const int nt = run.n;
    const uint32_t lanes = static_cast<uint32_t>(32 * quad + 16 * hf) << 16;
    const uint32_t tO = tmem + lanes + 256 + s * 128;
    const float kL2E = 1.4426950408889634f;
    Cursor at;
    if (nt > 0) at.start(run, kTK);
    bool ok = true;
    float ref[2], l[2], qs[2];
    int r[2];
    bool active = false;
    for (int t = 0; t < nt; ++t) {
      const bool first = t == 0 || at.tile == 0;
      if (first) {
        // a piece starts: the slot's rows of Q.  The last S of the piece before has been waited
        // for, so nothing reads the buffer.
        const int unit0 = (at.pair % a.RT) * rows_unit, h = at.pair / a.RT;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint4 u[D / 32];
          r[e] = lo + 8 * e < rows_unit ? min(unit0 + lo + 8 * e, R) : R;
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(a.q) + at.b * a.sb + (long long)(h * a.G + r[e] / a.T) * a.sh +
              (long long)(r[e] % a.T) * a.st);
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
            u[c] = r[e] < R ? __ldg(src + 4 * c + g) : make_uint4(0u, 0u, 0u, 0u);
          qs[e] = a.sm_scale * kL2E;
          ref[e] = -INFINITY;
          l[e] = 0.f;
          if (E4M3) {
            float amax = 0.f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              const uint32_t w4[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float2 f = halves<QBF>(w4[y]);
                amax = max3f(amax, fabsf(f.x), fabsf(f.y));
              }
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // an exact power of two that puts the largest value at 2^13
            const int ex = (int)(__float_as_uint(amax) >> 23);
            const int sh = (ex == 0 || ex == 255) ? 0 : max(-114, min(60, 13 + 127 - ex));
            const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
            qs[e] *= __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t w4[4] = {u[c].x, u[c].y, u[c].z, u[c].w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float2 f = halves<QBF>(w4[y]);
                w4[y] = pack2<false>(f.x * up, f.y * up);
              }
              u[c] = make_uint4(w4[0], w4[1], w4[2], w4[3]);
            }
          }
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
            *reinterpret_cast<uint4*>(sm.q[s] + tile_off<kTR>(ml + 8 * e, 4 * c + g)) = u[c];
        }
        active = __any_sync(0xffffffffu, r[0] < R);
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_lane0(&sm.q_full[s], lane);
      }
      if (!tile_wait(&sm.s_full[s][t & 1], (t >> 1) & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int key0 = at.tile * kTK;
      const uint32_t tS = tmem + lanes + s * 128 + (t & 1) * 64;
      if (active) {
        const float* sc = sm.scl[E4M3 && !SHARE ? s : 0][E4M3 ? t % C::kScales : 0];
        float lv = 0.f;
        if (E4M3) {
          lv = sm.lv[SHARE ? 0 : s][t % C::kScales];
        }
        if (key0 + kTK > at.s.len) {
          // inlined or not, the rest of the loop is compiled otherwise.  Inlined | apart, us, 32 heads over 8: 16 x 48
          // tokens over 32768 slots, e4m3 861 | 1041 (d = 64: 833 | 816), bf16 573 | 575 (447 | 448); 4 x 61 over 8192,
          // e4m3 105 | 112 (87 | 89), bf16 73.1 | 72.0 (64.4 | 63.4)
          if (E4M3) mask_scores<4>(a, at.s, at.b, tS, key0, r[0] % a.T, r[1] % a.T);
          else mask_scores_apart(a, at.s, at.b, tS, key0, r[0] % a.T, r[1] % a.T);
        }
        {
          uint32_t p[16];
          float2 sum[2];
          while (true) {
            const float n0 = ref[0] == -INFINITY ? 0.f : -ref[0], n1 = ref[1] == -INFINITY ? 0.f : -ref[1];
            const float2 q0 = make_float2(qs[0], qs[0]), q1 = make_float2(qs[1], qs[1]);
            const float2 m0 = make_float2(n0, n0), m1 = make_float2(n1, n1);
            float mx[2] = {-INFINITY, -INFINITY};
            sum[0] = sum[1] = make_float2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t x[16];
              tmem_ld16x256_16(tS + 32 * c, x);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                float2 x0 = make_float2(__uint_as_float(x[4 * k]), __uint_as_float(x[4 * k + 1]));
                float2 x1 = make_float2(__uint_as_float(x[4 * k + 2]), __uint_as_float(x[4 * k + 3]));
                float4 f4;
                if (E4M3) {
                  // two key scales and two value scales
                  f4 = *reinterpret_cast<const float4*>(sc + 2 * (32 * c + 8 * k + 2 * g));
                  x0 = __fmul2_rn(x0, make_float2(f4.x, f4.y));
                  x1 = __fmul2_rn(x1, make_float2(f4.x, f4.y));
                }
                mx[0] = max3f(mx[0], x0.x, x0.y);
                mx[1] = max3f(mx[1], x1.x, x1.y);
                float2 e0 = __ffma2_rn(x0, q0, m0), e1 = __ffma2_rn(x1, q1, m1);
                e0.x = ex2(e0.x);
                e0.y = ex2(e0.y);
                e1.x = ex2(e1.x);
                e1.y = ex2(e1.y);
                sum[0] = __fadd2_rn(sum[0], e0);
                sum[1] = __fadd2_rn(sum[1], e1);
                if (E4M3) {
                  e0 = __fmul2_rn(e0, make_float2(f4.z, f4.w));
                  e1 = __fmul2_rn(e1, make_float2(f4.z, f4.w));
                }
                p[8 * c + 2 * k] = pack2<BF>(e0.x, e0.y);
                p[8 * c + 2 * k + 1] = pack2<BF>(e1.x, e1.y);
              }
            }
            // e4m3: a bound, the largest score and the tile's largest value scale
            const bool over = (mx[0] > -INFINITY && mx[0] * qs[0] + lv > ref[0] + kRefGrow) ||
                              (mx[1] > -INFINITY && mx[1] * qs[1] + lv > ref[1] + kRefGrow);
            if (!__any_sync(0xffffffffu, over)) break;
            // the references move to the largest scores so far: the sums and O (at rest once P V of
            // the tile before is done) follow, and the tile is done again
            float f[2];
            if (E4M3) {
              const float4 w = moved_refs(tS, sc, qs[0], qs[1], ref[0], ref[1]);
              lv = -INFINITY;                     // the tile's bound is settled
              ref[0] = w.x;
              ref[1] = w.y;
              f[0] = w.z;
              f[1] = w.w;
              l[0] *= f[0];
              l[1] *= f[1];
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
                mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
                const float now = mx[e] == -INFINITY ? ref[e] : fmaxf(ref[e], mx[e] * qs[e]);
                f[e] = ref[e] == -INFINITY ? 0.f : ex2(ref[e] - now);
                ref[e] = now;
                l[e] *= f[e];
              }
            }
            if (!first) {
              if (!tile_wait(&sm.o_done[s][(t - 1) & 1], ((t - 1) >> 1) & 1, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
              scale_rows<D>(tO, f[0], f[1]);
            }
          }
          if (!ok) break;
          tmem_st16x128_16(tS, p);
          l[0] += sum[0].x + sum[0].y;
          l[1] += sum[1].x + sum[1].y;
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      mbar_arrive_lane0(&sm.p_full[s][t & 1], lane);

      if (at.tile + 1 == at.tiles || t + 1 == nt) {
        // ---- the piece ends
        if (!tile_wait(&sm.o_done[s][t & 1], (t >> 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (active) {
          const int start = at.tile - min(t, at.tile);     // the piece's first tile of the pair
          const bool whole = start == 0 && at.tile + 1 == at.tiles;
          const int vb = SHARE ? blockIdx.x : 2 * blockIdx.x + s, h = at.pair / a.RT;
          float inv[2];
          bool none[2];
          size_t row[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = r[e] % a.T;
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
            if (*static_cast<volatile int*>(&sm.bad_v) && r[e] < R) {
              // a drafted token's V was not finite somewhere: rows that attend such a one get NaN
              const uint8_t* mask = a.mask ? a.mask + at.b * a.mask_sb : nullptr;
              for (int j = 0; j < at.s.n; ++j)
                if (tree_allows(mask, a.T, i, j) && v_row_bad<D, E4M3, QBF>(a, at.b, h, at.s.len + j))
                  l[e] = __int_as_float(0x7fffffff);
            }
            none[e] = i >= at.s.n || l[e] == 0.f;
            inv[e] = none[e] ? 0.f : 1.f / l[e];
            row[e] = whole ? ((size_t)at.b * a.Hq + h * a.G + r[e] / a.T) * a.T + i
                           : (size_t)(2 * vb + (start == 0 ? 1 : 0)) * rows_unit + lo + 8 * e;
            if (r[e] < R && g == 0) {
              if (!whole) a.part_ml[row[e]] = make_float2(ref[e], l[e]);
              else if (a.lse) a.lse[row[e]] = none[e] ? -INFINITY : row_lse(ref[e], l[e]);
            }
          }
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t x[16];
            tmem_ld16x256_16(tO + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 16; y += 2) {
              const int e = (y >> 1) & 1;
              if (r[e] < R) {
                float f0 = __uint_as_float(x[y]), f1 = __uint_as_float(x[y + 1]);
                const size_t idx = row[e] * D + c + 8 * (y >> 2) + 2 * g;
                if (whole) store2(a.o, a.o_dtype, idx, none[e] ? 0.f : f0 * inv[e], none[e] ? 0.f : f1 * inv[e]);
                else store2(a.part, 2, idx, f0, f1);
              }
            }
          }
        }
      }
      if (t + 1 < nt) at.next(a, pairs, kTK);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool E4M3, bool QBF, bool SHARE>
static cudaError_t launch_tiles(TreeArgs a, int dev, cudaMemPool_t pool, cudaStream_t st) {
  using C = TilesCfg<D, E4M3>;
  const int R = a.G * a.T, most = SHARE ? 2 * kTR : kTR;
  a.RT = (R + most - 1) / most;
  const int unit = (R + a.RT - 1) / a.RT;          // rows of a unit
  const int grid = sm_count(dev), vgrid = SHARE ? grid : 2 * grid;
  CUtensorMap tk{}, tv{};
  cudaError_t e = cudaSuccess;
  if (!E4M3) {
    const uint64_t rows = (uint64_t)a.c.pages * a.c.Hkv << a.c.page_shift;
    const uint64_t dims[2] = {(uint64_t)D, rows};
    const uint64_t strides[1] = {(uint64_t)D * 2};
    const uint32_t box[2] = {64, min(1u << a.c.page_shift, (unsigned)kTK)};
    e = make_tmap(&tk, a.c.k, 2, dims, strides, box, 2, 128);
    if (e == cudaSuccess) e = make_tmap(&tv, a.c.v, 2, dims, strides, box, 2, 128);
    if (e != cudaSuccess) return e;
  }
  const size_t prow = (size_t)2 * vgrid * unit;
  e = split_workspace(&a, prow, D, pool, st);
  if (e != cudaSuccess) return e;
  auto kern = k_tree_tiles<D, E4M3, QBF, SHARE>;
  const int smem = sizeof(TilesSmem<D, E4M3>) + 1024;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) {
    kern<<<grid, kTThreads<E4M3>, smem, st>>>(tk, tv, a, unit);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    e = launch_join<D>(a, kTK, unit, vgrid, 1, st);
  }
  const cudaError_t e2 = cudaFreeAsync(a.part, st);
  return e != cudaSuccess ? e : e2;
}

}  // namespace sage2
