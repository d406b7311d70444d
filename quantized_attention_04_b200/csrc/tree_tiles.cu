// Attention of drafted tokens over a paged cache, many rows: k_tree_tiles.
//
// Row tiles of 128 against key tiles of 128 on the 5th-generation tensor cores.
// A block holds two row tiles ("slots", one softmax warpgroup each), so that one
// slot's softmax runs while the tensor cores work for the other:
//   SHARE   (more than 128 rows a pair): both slots walk the same run of key
//           tiles with the two halves of up to 256 rows; K and V are loaded once.
//   !SHARE  (up to 128 rows): each slot has a run of its own, as if it were a
//           block, and its own K and V tiles.
// Per slot and key tile: S = Q K^T (both in shared memory, fp32 S in TMEM),
// softmax by a thread per row, P (16 bits) written over S in TMEM, O += P V with
// P as the TMEM operand and V as it is cached ([key][d], the "MN-major" form), O in
// TMEM for the whole run of a pair.
//
// The softmax passes over S once: exponentials are taken against the reference
// left by the earlier keys, and only if some score of the warp's rows lies far above
// it (kGrow) the reference moves, and O, the row sums and the tile's P so far are
// rescaled.  A P above 1 keeps its relative precision.
//
// 16-bit caches: K and V arrive by TMA, a box a page.  e4m3 caches: eight warps load
// the codes (16 bytes a lane, in registers, two groups in turn), widen them to fp16
// (exact) and store them in the same layout.  Q enters as fp16 scaled by a power of
// two a row; the key scales multiply the scores and the value scales multiply P,
// whose reference includes the tile's largest value scale.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_index.h"
#include "sage2.h"
#include "sage2_internal.h"
#include "sm100_ptx.cuh"

namespace sage2 {

constexpr int kTT = 128;                  // keys of a tile, rows of a slot
// Warps: 16 softmax, 4 loaders (e4m3: two groups of 4, which take turns), the MMA warp and 3 idle ones.
template <bool E4M3>
constexpr int kTLoad = E4M3 ? 8 : 4;
template <bool E4M3>
constexpr int kTThreads = (16 + kTLoad<E4M3> + 4) * 32;
constexpr int kTScales = 4;               // tiles of scales that a slot keeps

template <int D, bool E4M3>
struct TilesCfg {
  static constexpr int kBlk = D / 64;                    // 128-byte blocks of a row
  static constexpr int kTileBytes = kTT * D * 2;         // a 16-bit tile of Q, K or V
  static constexpr int kBufs = D == 128 ? (E4M3 ? 4 : 5) : 6;
};

template <int D, bool E4M3>
struct __align__(1024) TilesSmem {
  using C = TilesCfg<D, E4M3>;
  uint8_t q[2][C::kTileBytes];
  uint8_t kv[C::kBufs][C::kTileBytes];
  // scales of a slot's last tiles; keys 2i, 2i+1: key scales at 4i, 4i+1, value scales at 4i+2, 4i+3
  float scl[E4M3 ? 2 : 1][kTScales][E4M3 ? 2 * kTT : 4];
  uint64_t full[C::kBufs];   // the four loader warps (and the TMA's bytes)
  uint64_t empty[C::kBufs];  // commit of the last MMA that reads the buffer
  uint64_t q_full[2];        // the slot's eight softmax warps
  uint64_t s_full[2];        // the MMA thread (it has seen the tile's scales) and the commit of S
  uint64_t p_full[2];        // the slot's eight softmax warps: S read, P written
  uint64_t o_done[2];        // commit of O += P V
  uint64_t tail[C::kBufs];   // bytes of a V tile that is checked before use
  uint64_t drain;
  long long scratch[28];
  Run run[2];
  Cursor mma_at[2];          // the MMA thread's: the piece that each slot is in
  uint32_t tmem;
  int bad_v;                 // a drafted token's V row or scale was not finite
  int abort_flag;
};

// D[tmem] (+)= A[tmem] * B[smem], 16-bit A (two values a column), fp32 D.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate));
}
// Descriptor of a [k][n] operand (n contiguous): 128-byte rows of 64 n, 128-byte
// swizzle, 8-row groups 1024 bytes apart, the next 64 n `block` bytes on.
__device__ __forceinline__ uint64_t smem_desc_nmajor(const void* p, uint32_t block) {
  const uint32_t addr = smem_u32(p);
  return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | (static_cast<uint64_t>(block >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

// Byte offset of 16-byte chunk `ch` (of D/8) of row `r` in a 128-row 16-bit tile.
__device__ __forceinline__ uint32_t tile_off(int r, int ch) {
  return (ch >> 3) * (kTT * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
}

// The order in which K and V tiles are loaded and used.  A slot's tiles go
// K(0), V(0), K(1), V(1), ..; with two runs the slots take turns after K(0) of each:
// V0(t) K0(t+1) V1(t) K1(t+1).
template <bool SHARE>
struct Walk {
  Cursor c[SHARE ? 1 : 2];
  int t[2], nt[2];
  bool v, pro, more;
  int s;
  __device__ __forceinline__ void start(const TreeArgs& a, const Run* run) {
    nt[0] = (int)(run[0].t1 - run[0].t0);
    nt[1] = SHARE ? 0 : (int)(run[1].t1 - run[1].t0);
    t[0] = t[1] = 0;
    if (nt[0] > 0) c[0].start(a, run[0], kTT);
    if (!SHARE && nt[1] > 0) c[SHARE ? 0 : 1].start(a, run[1], kTT);
    v = false;
    pro = !SHARE;
    s = 0;
    more = nt[0] > 0;      // slot 1 has work only if slot 0 has
  }
  __device__ __forceinline__ void step(const TreeArgs& a, int pairs) {
    if (SHARE) {
      if (!v) {
        v = true;
      } else {
        v = false;
        if (++t[0] < nt[0]) c[0].next(a, pairs, kTT);
        else more = false;
      }
      return;
    }
    if (pro) {
      if (s == 0 && nt[1] > 0) {
        s = 1;
        return;
      }
      pro = false;
      s = 0;
      v = true;
      return;
    }
    if (v) {
      bool k = false;
      if (s == 0) {
        if (++t[0] < nt[0]) {
          c[0].next(a, pairs, kTT);
          k = true;
        }
      } else {
        if (++t[1] < nt[1]) {
          c[SHARE ? 0 : 1].next(a, pairs, kTT);
          k = true;
        }
      }
      if (k) {
        v = false;
        return;
      }
    }
    v = true;
    const bool l0 = t[0] < nt[0], l1 = t[1] < nt[1];
    if (s == 0) s = l1 ? 1 : 0;
    else s = l0 ? 0 : 1;
    more = l0 || l1;
  }
  __device__ __forceinline__ Cursor cur() const { return SHARE || s == 0 ? c[0] : c[SHARE ? 0 : 1]; }
};

// Which of the 32 slots from `key` on a row of drafted token i attends, as bits.
__device__ __forceinline__ uint32_t allowed32(const TreeArgs& a, const uint8_t* mask, SeqLen s, int i,
                                              int key) {
  const int ctx = s.len - key;                 // of them in the context
  if (ctx >= 32) return 0xffffffffu;
  uint32_t bits = ctx > 0 ? (1u << ctx) - 1u : 0u;
  if (key >= s.len + s.n) return bits;
#pragma unroll
  for (int c = 0; c < 32; ++c) {
    const int j = c - ctx;
    const bool in = j >= 0 && j < s.n;
    if (in && tree_allows(mask, a.T, i, j)) bits |= 1u << c;
  }
  return bits;
}

// Does drafted token i of a sequence attend slot `key`?
__device__ __forceinline__ bool slot_allowed(const TreeArgs& a, const uint8_t* mask, SeqLen s, int i, int key) {
  const int j = key - s.len;
  return j < 0 || (j < s.n && tree_allows(mask, a.T, i, j));
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
__device__ __forceinline__ void tmem_ld16x128_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x128b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Two consecutive values (index of the first, even) in the output type.
__device__ __forceinline__ void store2(void* out, int dtype, size_t idx, float x, float y) {
  if (dtype == 2) *reinterpret_cast<float2*>(static_cast<float*>(out) + idx) = make_float2(x, y);
  else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + idx) = dtype == 1 ? pack2<true>(x, y) : pack2<false>(x, y);
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

template <int D, bool E4M3, bool QBF, bool SHARE>
__global__ void __launch_bounds__(kTThreads<E4M3>, 1)
    k_tree_tiles(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ TreeArgs a, int rows_unit) {
  using C = TilesCfg<D, E4M3>;
  using Smem = TilesSmem<D, E4M3>;
  constexpr bool BF = QBF && !E4M3;              // type of the MMA operands
  // log2 of how far P may exceed 1 before the reference moves: fp16 ends at 2^16; a bf16 P of
  // 2^40 leaves its sums and O (fp32) far from their end
  constexpr float kGrow = BF ? 40.f : 14.f;
  constexpr int kMma = 16 + kTLoad<E4M3>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = a.G * a.T, pairs = a.c.Hkv * a.RT;
  volatile int* abort_flag = &sm.abort_flag;
  if (tid == 0) {
    for (int i = 0; i < C::kBufs; ++i) {
      mbar_init(&sm.full[i], 4);
      mbar_init(&sm.empty[i], 1);
      mbar_init(&sm.tail[i], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 8);
      mbar_init(&sm.s_full[s], 2);
      mbar_init(&sm.p_full[s], 8);
      mbar_init(&sm.o_done[s], 1);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    sm.bad_v = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  const int vgrid = SHARE ? gridDim.x : 2 * gridDim.x;
  find_run(a, kTT, pairs, vgrid, SHARE ? blockIdx.x : 2 * blockIdx.x, 1, &sm.run[0], sm.scratch);
  if (!SHARE) find_run(a, kTT, pairs, vgrid, 2 * blockIdx.x + 1, 1, &sm.run[1], sm.scratch);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  const Run& run0 = sm.run[0];
  const Run& run1 = sm.run[SHARE ? 0 : 1];

  // registers at launch and by role: 768 x 80 = 512 x 96 + 128 x 48 + 128 x 48, and with
  // e4m3, whose loaders hold a tile, 896 x 72 = 512 x 80 + 256 x 72 + 128 x 40
  constexpr int kRegSoft = E4M3 ? 80 : 96, kRegMma = E4M3 ? 40 : 48;
  if (warp >= 16 && warp < 16 + kTLoad<E4M3>) {
    // ------------------------------------------------------------ loaders
    if (!E4M3) setmaxnreg_dec<48>();
    Walk<SHARE> w;
    w.start(a, sm.run);
    const int lw = (warp - 16) & 3, lgroup = (warp - 16) >> 2;
    bool ok = true;
    if (!E4M3) {
      int e = 0;
      unsigned tails = 0;          // parity of the next phase of each buffer's tail barrier
      for (; w.more; w.step(a, pairs), ++e) {
        const Cursor c = w.cur();
        const int buf = e % C::kBufs;
        if (e >= C::kBufs && !mbar_wait_warp(&sm.empty[buf], (e / C::kBufs - 1) & 1, abort_flag)) {
          ok = false;
          break;
        }
        const int key0 = c.tile * kTT, L = c.s.len + c.s.n, h = c.pair / a.RT;
        const bool edge = w.v && key0 + kTT > c.s.len;
        uint64_t* bar = edge ? &sm.tail[buf] : &sm.full[buf];
        uint8_t* dst = sm.kv[buf];
        if (lw == 0) {
          // lane p: page chunk p of the tile (the pages of rows behind the last key are not read)
          const int prow = 1 << a.c.page_shift, chunk = key0 + lane * prow;
          const bool in = lane * prow < kTT && chunk < L;
          int page = -1;
          if (in) {
            page = __ldg(a.table + (size_t)c.b * a.MP + (chunk >> a.c.page_shift));
            if (!page_inside(page, a.c.pages)) {
              atomicOr(&g_device_error, DEVERR_BOUNDS);
              page = 0;     // any rows: the outputs are not meaningful
            }
          }
          const int n = __popc(__ballot_sync(0xffffffffu, in));
          if (lane == 0) mbar_expect_tx(bar, n * prow * D * 2);
          __syncwarp();
          if (in) {
            const int row = (int)row_of(page, a.c.Hkv, h, a.c.page_shift, chunk);
#pragma unroll
            for (int x = 0; x < C::kBlk; ++x)
              tma_load_2d(dst + x * kTT * 128 + lane * prow * 128, w.v ? &tm_v : &tm_k, bar, x * 64, row);
          }
        }
        if (edge) {
          // rows behind the last key and drafted rows that are not finite become zeros
          if (!mbar_wait_warp(&sm.tail[buf], (tails >> buf) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tails ^= 1u << buf;
          const int r = tid - 16 * 32;
          if (key0 + r >= c.s.len) {
            bool zero = key0 + r >= L;
            if (!zero) {
#pragma unroll
              for (int ch = 0; ch < D / 8; ++ch)
                zero = not_finite16<false, QBF>(*reinterpret_cast<const uint4*>(dst + tile_off(r, ch))) || zero;
              if (zero) sm.bad_v = 1;
            }
            if (zero)
              for (int ch = 0; ch < D / 8; ++ch)
                *reinterpret_cast<uint4*>(dst + tile_off(r, ch)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.full[buf]);
        } else if (lw != 0 && lane == 0) {
          mbar_arrive(&sm.full[buf]);
        }
      }
      if (!ok && lw == 0) {
        // let the copies already issued land before the block exits
        for (int u = e > C::kBufs ? e - C::kBufs : 0; u < e; ++u)
          mbar_wait(&sm.full[u % C::kBufs], (u / C::kBufs) & 1, nullptr);
      }
    } else {
      constexpr int LPR = D / 16, RPP = 128 / LPR, NP = kTT / RPP;   // lanes of a row, rows of a pass
      const int lt = (tid - 16 * 32) & 127, lr = lt / LPR, lc = lt % LPR;
      struct Ahead {
        uint4 u[NP];
        float ks, vs;
        int key0, len, n, t, s;
        bool v, there;
      };
      auto fetch = [&](Ahead& x) {
        x.there = w.more;
        if (!w.more) return;
        const Cursor c = w.cur();
        x.v = w.v;
        x.s = w.s;
        x.t = w.s ? w.t[1] : w.t[0];
        x.key0 = c.tile * kTT;
        x.len = c.s.len;
        x.n = c.s.n;
        const int h = c.pair / a.RT, L = c.s.len + c.s.n;
        const int* tab = a.table + (size_t)c.b * a.MP;
        const uint8_t* pool = w.v ? a.c.v : a.c.k;
        int pg[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int key = x.key0 + p * RPP + lr;
          pg[p] = key < L ? __ldg(tab + (key >> a.c.page_shift)) : -1;
        }
        int spg = -1;
        const int skey = x.key0 + lt;
        if (!w.v && skey < L) spg = __ldg(tab + (skey >> a.c.page_shift));
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int key = x.key0 + p * RPP + lr;
          x.u[p] = make_uint4(0u, 0u, 0u, 0u);
          if (key < L) {
            if (page_inside(pg[p], a.c.pages)) {
              const long long row = row_of(pg[p], a.c.Hkv, h, a.c.page_shift, key);
              x.u[p] = __ldg(reinterpret_cast<const uint4*>(pool + row * D) + lc);
            } else {
              atomicOr(&g_device_error, DEVERR_BOUNDS);
            }
          }
        }
        x.ks = x.vs = 0.f;
        if (!w.v && page_inside(spg, a.c.pages)) {
          const long long row = row_of(spg, a.c.Hkv, h, a.c.page_shift, skey);
          x.ks = __ldg(a.c.ks + row);
          x.vs = __ldg(a.c.vs + row);
        }
        w.step(a, pairs);
      };
      auto put = [&](Ahead& x, int e) -> bool {
        const int buf = e % C::kBufs;
        if (e >= C::kBufs && !mbar_wait_warp(&sm.empty[buf], (e / C::kBufs - 1) & 1, abort_flag)) return false;
        uint8_t* dst = sm.kv[buf];
        const bool edge = x.key0 + kTT > x.len;
        if (!x.v) {
          // the scales of both; slot x.t % kTScales was last read kTScales tiles ago, and a
          // V tile later than that one has been freed
          float ks = x.ks, vs = x.vs;
          if (x.key0 + lt >= x.len) {
            // masked scores are -inf before the key scale multiplies them, and P is 0 before the
            // value scale does: the scales of drafted rows become finite, a key's not 0 (a row of
            // scale 0 has codes 0), those behind the last key are 0
            if (!(fabsf(vs) < INFINITY) || !(fabsf(ks) < INFINITY)) {
              if (!(fabsf(vs) < INFINITY)) vs = 0.f;
              if (!(fabsf(ks) < INFINITY)) ks = 1.f;
              sm.bad_v = 1;
            }
            if (ks == 0.f) ks = 1.f;
          }
          float* sc = sm.scl[x.s][x.t % kTScales] + 4 * (lt >> 1) + (lt & 1);
          sc[0] = ks;
          sc[2] = vs;
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          const int r = p * RPP + lr;
          if (x.v && edge) {
            const bool dr = x.key0 + r >= x.len;
            unsigned bad = dr && not_finite16<true, false>(x.u[p]) ? 1u : 0u;
#pragma unroll
            for (int o = LPR / 2; o; o >>= 1) bad |= __shfl_xor_sync(0xffffffffu, bad, o);
            if (bad) {
              x.u[p] = make_uint4(0u, 0u, 0u, 0u);
              sm.bad_v = 1;
            }
          }
          const uint32_t cw[4] = {x.u[p].x, x.u[p].y, x.u[p].z, x.u[p].w};
          uint4 lo, hi;
          lo.x = e4m3x2_f16x2(cw[0] & 0xffffu);
          lo.y = e4m3x2_f16x2(cw[0] >> 16);
          lo.z = e4m3x2_f16x2(cw[1] & 0xffffu);
          lo.w = e4m3x2_f16x2(cw[1] >> 16);
          hi.x = e4m3x2_f16x2(cw[2] & 0xffffu);
          hi.y = e4m3x2_f16x2(cw[2] >> 16);
          hi.z = e4m3x2_f16x2(cw[3] & 0xffffu);
          hi.w = e4m3x2_f16x2(cw[3] >> 16);
          // the two halves of a row store different chunks at a time: no bank conflicts
          const bool sw = D == 128 && (lc >> 2);
          *reinterpret_cast<uint4*>(dst + tile_off(r, 2 * lc + (sw ? 1 : 0))) = sw ? hi : lo;
          *reinterpret_cast<uint4*>(dst + tile_off(r, 2 * lc + (sw ? 0 : 1))) = sw ? lo : hi;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[buf]);
        return true;
      };
      // the two groups take every other tile: one loads while the other stores
      if (lgroup && w.more) w.step(a, pairs);
      int e = lgroup;
      Ahead x;
      for (fetch(x); x.there; fetch(x)) {
        if (!put(x, e)) break;
        e += 2;
        if (w.more) w.step(a, pairs);
      }
    }
  } else if (warp >= 16) {
    // ------------------------------------------------------------ MMA issuer
    setmaxnreg_dec<kRegMma>();
    if (warp == kMma && lane == 0) {
      constexpr uint32_t idesc_s = idesc_f16_f32(kTT, kTT, BF);
      constexpr uint32_t idesc_o = idesc_f16_f32(kTT, D, BF) | (1u << 16);   // B is [k][n]
      const uint64_t dq = smem_desc_kmajor(sm.q[0], 128);
      const uint64_t dk = smem_desc_kmajor(sm.kv[0], 128);
      const uint64_t dv = smem_desc_nmajor(sm.kv[0], kTT * 128);
      constexpr uint32_t kBuf16 = C::kTileBytes >> 4;
      int nt[2] = {(int)(run0.t1 - run0.t0), (int)(run1.t1 - run1.t0)};
      // tiles of the slot's piece from the current one on; a piece's first tile is next
      int left0 = 0, left1 = 0;
      bool new0 = true, new1 = true;
      if (nt[0] > 0) {
        sm.mma_at[0].start(a, run0, kTT);
        left0 = sm.mma_at[0].tiles - sm.mma_at[0].tile;
      }
      if (nt[1] > 0) {
        sm.mma_at[1].start(a, run1, kTT);
        left1 = sm.mma_at[1].tiles - sm.mma_at[1].tile;
      }
      int e = 0;                   // buffers taken
      int pieces = 0;              // parity of each slot's piece
      bool ok = true;
      auto wait_full = [&](int u) {
        return mbar_wait(&sm.full[u % C::kBufs], (u / C::kBufs) & 1, abort_flag);
      };
      // S of slot s; entry u; `first`: a piece starts with this tile
      auto scores = [&](int s, int u, bool first, bool release) -> bool {
        if (first) {
          if (!mbar_wait(&sm.q_full[s], (pieces >> s) & 1, abort_flag)) return false;
          pieces ^= 1 << s;
        }
        if (!wait_full(u)) return false;
        mbar_arrive(&sm.s_full[s]);
        tc_fence_after();
        const uint64_t qb = dq + s * kBuf16, kb = dk + (u % C::kBufs) * kBuf16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * ((kTT * 128) >> 4) + (kk & 3) * 2;
          mma_f16_ss(tmem + s * 128, qb + off, kb + off, idesc_s, kk > 0);
        }
        tc_commit(&sm.s_full[s]);
        if (release) tc_commit(&sm.empty[u % C::kBufs]);
        return true;
      };
      auto values = [&](int s, int t, int u, bool first, bool release) -> bool {
        if (!mbar_wait(&sm.p_full[s], t & 1, abort_flag)) return false;
        if (!wait_full(u)) return false;
        tc_fence_after();
        const uint64_t vb = dv + (u % C::kBufs) * kBuf16;
#pragma unroll
        for (int kk = 0; kk < kTT / 16; ++kk)
          mma_f16_ts(tmem + 256 + s * 128, tmem + s * 128 + 8 * kk, vb + kk * (16 * 128 >> 4), idesc_o,
                     !first || kk > 0);
        tc_commit(&sm.o_done[s]);
        if (release) tc_commit(&sm.empty[u % C::kBufs]);
        return true;
      };
      // prologue: the first S of both slots
      if (SHARE) {
        if (nt[0] > 0) {
          ok = scores(0, 0, true, false) && scores(1, 0, true, true);
          e = 1;
        }
      } else {
        if (nt[0] > 0) ok = scores(0, e++, true, true);
        if (ok && nt[1] > 0) ok = scores(1, e++, true, true);
      }
      const int nt0 = nt[0], nt1 = nt[1];
#pragma unroll 1
      for (int ts = 0; ok && ts < 2 * nt0; ++ts) {
        const int t = ts >> 1, s = ts & 1, n = s ? nt1 : nt0;
        if (t >= n) continue;
        int left = s ? left1 : left0;
        bool fresh = s ? new1 : new0;
        const int u = SHARE ? 2 * t + 1 : e;       // this V; K of the next tile is u + 1
        const bool more = t + 1 < n;
        const bool rel = SHARE ? s == 1 : true;
        ok = values(s, t, u, fresh, rel);
        fresh = false;
        if (ok && more) {
          if (--left == 0) {
            Cursor c = sm.mma_at[s];
            c.tile = c.tiles - 1;
            c.next(a, pairs, kTT);
            sm.mma_at[s] = c;
            left = c.tiles;
            fresh = true;
          }
          ok = scores(s, u + 1, fresh, rel);
        }
        if (s) {
          left1 = left;
          new1 = fresh;
        } else {
          left0 = left;
          new0 = fresh;
        }
        if (!SHARE) e += more ? 2 : 1;
      }
      // every MMA issued so far completes before the block frees TMEM
      tc_commit(&sm.drain);
      mbar_wait(&sm.drain, 0, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    // Eight warps a slot.  The .16x256b loads give a warp 16 TMEM lanes and each of its
    // quads two rows, t/4 and t/4 + 8, so that four warps share a scheduler.  Row r
    // of the slot is on lane 32 (r/16 % 4) + 16 (r/64) + r%16: any number of rows is
    // spread evenly over the schedulers.
    setmaxnreg_inc<kRegSoft>();
    const int s = warp >> 3, quad = warp & 3, hf = (warp >> 2) & 1, g = lane & 3;
    const int lo = (SHARE ? s * kTT : 0) + 64 * hf + 16 * quad + (lane >> 2);   // of the unit's rows: lo, lo + 8
    const int ml = 32 * quad + 16 * hf + (lane >> 2);                           // TMEM lane: ml, ml + 8
    const Run& run = s ? run1 : run0;
    const int nt = (int)(run.t1 - run.t0);
    const uint32_t lanes = static_cast<uint32_t>(32 * quad + 16 * hf) << 16;
    const uint32_t tS = tmem + lanes + s * 128, tO = tmem + lanes + 256 + s * 128;
    const float kL2E = 1.4426950408889634f;
    Cursor at;
    if (nt > 0) at.start(a, run, kTT);
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
          r[e] = lo + 8 * e < rows_unit ? min(unit0 + lo + 8 * e, R) : R;
          qs[e] = a.sm_scale * kL2E;
          ref[e] = -INFINITY;
          l[e] = 0.f;
          uint4 u[D / 32];
          const uint4* src = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(a.q) + at.b * a.sb + (long long)(h * a.G + r[e] / a.T) * a.sh +
              (long long)(r[e] % a.T) * a.st);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) u[c] = r[e] < R ? __ldg(src + 4 * c + g) : make_uint4(0u, 0u, 0u, 0u);
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
            *reinterpret_cast<uint4*>(sm.q[s] + tile_off(ml + 8 * e, 4 * c + g)) = u[c];
        }
        active = __any_sync(0xffffffffu, r[0] < R);
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_lane0(&sm.q_full[s], lane);
      }
      if (!mbar_wait_warp(&sm.s_full[s], t & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const int key0 = at.tile * kTT;
      if (active) {
        const float* sc = sm.scl[E4M3 && !SHARE ? s : 0][E4M3 ? t % kTScales : 0];
        float lv = 0.f;
        if (E4M3) {
          const float4 v0 = *reinterpret_cast<const float4*>(sc + 8 * lane);
          const float4 v1 = *reinterpret_cast<const float4*>(sc + 8 * lane + 4);
          float m = fmaxf(fmaxf(v0.z, v0.w), fmaxf(v1.z, v1.w));
#pragma unroll
          for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          lv = log2f(fmaxf(m, kVrefLeast));
        }
        if (key0 + kTT > at.s.len) {
          // scores that the mask or the length leaves out become -inf where they lie
          const uint8_t* mask = a.mask ? a.mask + at.b * a.mask_sb : nullptr;
          const int i0 = r[0] % a.T, i1 = r[1] % a.T;
#pragma unroll 1
          for (int c = 0; c < kTT; c += 32) {
            uint32_t x[16];
            tmem_ld16x256_16(tS + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 16; ++y) {
              const int key = key0 + c + 8 * (y >> 2) + 2 * g + (y & 1);
              if (!slot_allowed(a, mask, at.s, y & 2 ? i1 : i0, key)) x[y] = 0xff800000u;
            }
            tmem_st16x256_16(tS + c, x);
          }
          tmem_st_wait();
        }
        // P of chunk c (64 keys, 32 columns) goes over scores that have been read
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t p[16];
          float2 sum[2];
          while (true) {
            const float n0 = ref[0] == -INFINITY ? 0.f : -ref[0], n1 = ref[1] == -INFINITY ? 0.f : -ref[1];
            const float2 q0 = make_float2(qs[0], qs[0]), q1 = make_float2(qs[1], qs[1]);
            const float2 m0 = make_float2(n0, n0), m1 = make_float2(n1, n1);
            float mx[2] = {-INFINITY, -INFINITY};
            sum[0] = sum[1] = make_float2(0.f, 0.f);
            uint32_t x[32];
            tmem_ld16x256_32(tS + 64 * c, x);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float2 x0 = make_float2(__uint_as_float(x[4 * k]), __uint_as_float(x[4 * k + 1]));
              float2 x1 = make_float2(__uint_as_float(x[4 * k + 2]), __uint_as_float(x[4 * k + 3]));
              float4 f4;
              if (E4M3) {
                // two key scales and two value scales
                f4 = *reinterpret_cast<const float4*>(sc + 2 * (64 * c + 8 * k + 2 * g));
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
              p[2 * k] = pack2<BF>(e0.x, e0.y);
              p[2 * k + 1] = pack2<BF>(e1.x, e1.y);
            }
            const bool over = (mx[0] > -INFINITY && mx[0] * qs[0] + lv > ref[0] + kGrow) ||
                              (mx[1] > -INFINITY && mx[1] * qs[1] + lv > ref[1] + kGrow);
            if (!__any_sync(0xffffffffu, over)) break;
            // the references move to the largest scores so far: the sums, O (at rest once P V of the
            // tile before is done) and the P of chunk 0 follow, and this chunk is done again
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
              mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
              const float now = mx[e] == -INFINITY ? ref[e] : fmaxf(ref[e], mx[e] * qs[e] + lv);
              f[e] = ref[e] == -INFINITY ? 0.f : ex2(ref[e] - now);
              ref[e] = now;
              l[e] *= f[e];
            }
            if (!first) {
              if (!mbar_wait_warp(&sm.o_done[s], (t - 1) & 1, abort_flag)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int d0 = 0; d0 < D; d0 += 32) {
                uint32_t y[16];
                tmem_ld16x256_16(tO + d0, y);
                tmem_ld_wait();
#pragma unroll
                for (int z = 0; z < 16; ++z) y[z] = __float_as_uint(__uint_as_float(y[z]) * f[(z >> 1) & 1]);
                tmem_st16x256_16(tO + d0, y);
              }
            }
            tmem_st_wait();
            if (c == 1) {
              uint32_t y[16];
              tmem_ld16x128_16(tS, y);
              tmem_ld_wait();
#pragma unroll
              for (int z = 0; z < 16; ++z) {
                const float2 w2 = halves<BF>(y[z]);
                y[z] = pack2<BF>(w2.x * f[z & 1], w2.y * f[z & 1]);
              }
              tmem_st16x128_16(tS, y);
            }
          }
          if (!ok) break;
          tmem_st16x128_16(tS + 32 * c, p);
          l[0] += sum[0].x + sum[0].y;
          l[1] += sum[1].x + sum[1].y;
        }
        if (!ok) break;
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      mbar_arrive_lane0(&sm.p_full[s], lane);

      if (at.tile + 1 == at.tiles || t + 1 == nt) {
        // ---- the piece ends
        if (!mbar_wait_warp(&sm.o_done[s], t & 1, abort_flag)) {
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
      if (t + 1 < nt) at.next(a, pairs, kTT);
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
  const int R = a.G * a.T, most = SHARE ? 2 * kTT : kTT;
  a.RT = (R + most - 1) / most;
  const int unit = (R + a.RT - 1) / a.RT;          // rows of a unit
  const int grid = sm_count(dev), vgrid = SHARE ? grid : 2 * grid;
  CUtensorMap tk{}, tv{};
  cudaError_t e = cudaSuccess;
  if (!E4M3) {
    const uint64_t rows = (uint64_t)a.c.pages * a.c.Hkv << a.c.page_shift;
    const uint64_t dims[2] = {(uint64_t)D, rows};
    const uint64_t strides[1] = {(uint64_t)D * 2};
    const uint32_t box[2] = {64, 1u << a.c.page_shift};
    e = make_tmap(&tk, a.c.k, 2, dims, strides, box, 2, 128);
    if (e == cudaSuccess) e = make_tmap(&tv, a.c.v, 2, dims, strides, box, 2, 128);
    if (e != cudaSuccess) return e;
  }
  const size_t prow = (size_t)2 * vgrid * unit;
  uint8_t* ws = nullptr;
  e = cudaMallocFromPoolAsync(reinterpret_cast<void**>(&ws), up256(prow * D * 4) + prow * 8, pool, st);
  if (e != cudaSuccess) return e;
  a.part = reinterpret_cast<float*>(ws);
  a.part_ml = reinterpret_cast<float2*>(ws + up256(prow * D * 4));
  auto kern = k_tree_tiles<D, E4M3, QBF, SHARE>;
  const int smem = sizeof(TilesSmem<D, E4M3>) + 1024;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) {
    kern<<<grid, kTThreads<E4M3>, smem, st>>>(tk, tv, a, unit);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    k_tree_join<D><<<dim3((R + 3) / 4, a.c.Hkv, a.B), 128, 0, st>>>(a, kTT, unit, vgrid, 1);
    e = cudaGetLastError();
  }
  const cudaError_t e2 = cudaFreeAsync(ws, st);
  return e != cudaSuccess ? e : e2;
}

}  // namespace sage2
