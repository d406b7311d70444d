// Attention of drafted tokens over a paged cache (sage2_attn_tree) and the
// tally of attention weight per cached token (sage2_cache_weights).
//
// Row r = g*T + i of key/value head h is drafted token i of query head h*G + g
// (G = Hq/Hkv); its keys are the slots [0, lens[b]) and, of the drafted tokens'
// slots lens[b] + j (j < n[b]), those that the mask allows (no mask: j <= i).
//
// Work split.  The tiles of all (sequence, head, row tile) pairs, in that order,
// form one sequence that the blocks cut into equal runs, so unequal lengths
// need no plan from the host, which does not know them.  A pair that one block
// covers whole is written at once; the pieces of the others go to a
// workspace with their row maxima and sums and k_tree_join adds them.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cache_index.h"
#include "sage2.h"
#include "sage2_internal.h"
#include "sm100_ptx.cuh"

namespace sage2 {

struct TreeArgs {
  CacheView c;
  const int* table;
  const int* lens;
  const int* n;             // null: T
  const uint8_t* mask;      // null: j <= i
  long long mask_sb;        // bytes between the masks of consecutive sequences
  const void* q;
  long long sb, sh, st;     // strides of q in elements
  void* o;
  int o_dtype;
  float* lse;
  int B, Hq, G, T, MP;
  float sm_scale;
  int RT;                   // row tiles of a (sequence, head) pair
  float* part;              // [2*grid][rows of a tile][d]
  float2* part_ml;          // [2*grid][rows of a tile]: (max in log2 units, sum)
  long long* before;        // [B + 1]: tiles of the sequences before b; the last: of all
};

// Context length and drafted tokens of sequence b, held to what the table can hold.
__device__ __forceinline__ SeqLen seq_len(const int* lens, const int* ns, int b, int T, int MP,
                                          int page_shift) {
  SeqLen s;
  s.len = __ldg(lens + b);
  s.n = ns ? __ldg(ns + b) : T;
  const int cap = MP << page_shift;
  if (!seq_fits(s.len, s.n, T, cap)) {
    atomicOr(&g_device_error, DEVERR_BOUNDS);
    s = seq_clamped(s.len, s.n, T, cap);
  }
  return s;
}

// Is drafted token j among the keys of drafted token i?  (j < n)
__device__ __forceinline__ bool tree_allows(const uint8_t* mask, int T, int i, int j) {
  return mask ? __ldg(mask + (size_t)i * T + j) != 0 : j <= i;
}
// Does drafted token i of a sequence (n > 0) attend slot `key`?  The byte of the mask is asked for in any case,
// at the nearest drafted slot, so that many such loads are on their way at once (behind a condition each
// waited for the one before: 16 us for the 128 keys and 256 rows of an edge tile of the tally).
__device__ __forceinline__ bool slot_allowed(const TreeArgs& a, const uint8_t* mask, SeqLen s, int i, int key) {
  const int j = key - s.len;
  const bool in = tree_allows(mask, a.T, i, min(max(j, 0), s.n - 1));
  return j < 0 || (j < s.n && in);
}

// ------------------------------------------------------------ the work split
// A block's run of the global tile sequence and the pair it starts in.
struct Run {
  int n;                   // tiles
  int b, pair, tile;       // the first one
  SeqLen s;                // of sequence b
};

// The run of block `c` of `grid`, by a whole warp (every warp that needs it works it out
// for itself: no barrier).  No block takes fewer than `least` tiles while others have none.
// `pairs`: pairs of one sequence (Hkv*RT).
__device__ __forceinline__ Run warp_run(const TreeArgs& a, int tile, int pairs, int grid, int c, int least) {
  const int lane = threadIdx.x & 31;
  Run r{0, 0, 0, 0, {0, 0}};
  SeqLen s{0, 0};
  int tl = 0;
  long long total = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    tl = 0;
    if (b0 + lane < a.B) {
      s = seq_len(a.lens, a.n, b0 + lane, a.T, a.MP, a.c.page_shift);
      tl = pair_tiles(s, tile);
    }
    total += tl;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  total *= pairs;
  const int g = run_blocks(total, grid, least);
  if (c >= g) return r;
  const long long t0 = run_start(total, g, c);
  r.n = (int)(run_start(total, g, c + 1) - t0);
  if (r.n == 0) return r;
  long long before = 0;    // tiles of the sequences before b0
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    if (a.B > 32) {        // else s and tl are at hand
      tl = 0;
      if (b0 + lane < a.B) {
        s = seq_len(a.lens, a.n, b0 + lane, a.T, a.MP, a.c.page_shift);
        tl = pair_tiles(s, tile);
      }
    }
    long long incl = (long long)tl * pairs;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const long long off = t0 - before - (incl - (long long)tl * pairs);
    const unsigned here = __ballot_sync(0xffffffffu, off >= 0 && off < (long long)tl * pairs);
    if (here) {
      const int src = __ffs(here) - 1;
      int pair = 0, at = 0;
      if (lane == src) {
        if (off <= INT_MAX) {
          pair = (int)off / tl;
          at = (int)off % tl;
        } else {
          pair = (int)(off / tl);
          at = (int)(off % tl);
        }
      }
      r.b = b0 + src;
      r.pair = __shfl_sync(0xffffffffu, pair, src);
      r.tile = __shfl_sync(0xffffffffu, at, src);
      r.s.len = __shfl_sync(0xffffffffu, s.len, src);
      r.s.n = __shfl_sync(0xffffffffu, s.n, src);
      break;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  return r;
}

// What the join needs of the split: the tiles before each sequence.  By one warp of the launch.
__device__ __forceinline__ void write_before(const TreeArgs& a, int tile, int pairs) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    long long incl = 0;
    if (b0 + lane < a.B)
      incl = (long long)pair_tiles(seq_len(a.lens, a.n, b0 + lane, a.T, a.MP, a.c.page_shift), tile) * pairs;
    const long long mine = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (b0 + lane < a.B) a.before[b0 + lane] = before + incl - mine;
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) a.before[a.B] = before;
}

// Walks the tiles of a run.
struct Cursor {
  int b, pair, tile, tiles;
  SeqLen s;
  __device__ __forceinline__ void start(const Run& r, int tl) {
    b = r.b;
    pair = r.pair;
    tile = r.tile;
    s = r.s;
    tiles = pair_tiles(s, tl);
  }
  // to the next tile of the run, which exists
  __device__ __forceinline__ void next(const TreeArgs& a, int pairs, int tl) {
    if (++tile < tiles) return;
    tile = 0;
    if (++pair < pairs) return;
    pair = 0;
    do {
      ++b;
      s = seq_len(a.lens, a.n, b, a.T, a.MP, a.c.page_shift);
      tiles = pair_tiles(s, tl);
    } while (tiles == 0 && b + 1 < a.B);
  }
};

// ------------------------------------------------------------ legacy-path MMA
// D (16x8, fp32) += A (16x16) * B (16x8), fp16 or bf16.
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Four e4m3 codes to two packed fp16 pairs, exact.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& a, uint32_t& b) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
      : "=r"(a), "=r"(b)
      : "r"(w));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The two values of a packed pair.
template <bool BF>
__device__ __forceinline__ float2 halves(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
// Does a 16-byte piece of a cached row hold an infinity or NaN?
template <bool E4M3, bool BF>
__device__ __forceinline__ bool not_finite16(uint4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (E4M3) {
      bad = bad || (((w[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u);
    } else {
      constexpr uint32_t e = BF ? 0x7f80u : 0x7c00u;
      bad = bad || (w[i] & e) == e || ((w[i] >> 16) & e) == e;
    }
  }
  return bad;
}

// Four consecutive values (index of the first, a multiple of 4) in the output type.
__device__ __forceinline__ void store4(void* out, int dtype, size_t idx, const float (&f)[4]) {
  if (dtype == 2) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + idx) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
    const uint2 w = dtype == 1 ? make_uint2(pack2<true>(f[0], f[1]), pack2<true>(f[2], f[3]))
                               : make_uint2(pack2<false>(f[0], f[1]), pack2<false>(f[2], f[3]));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + idx) = w;
  }
}
// Two consecutive values (index of the first, even) in the output type.
__device__ __forceinline__ void store2(void* out, int dtype, size_t idx, float x, float y) {
  if (dtype == 2) *reinterpret_cast<float2*>(static_cast<float*>(out) + idx) = make_float2(x, y);
  else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + idx) = dtype == 1 ? pack2<true>(x, y) : pack2<false>(x, y);
}
// Value scales outside of these count as one of them in P's reference: 2^-80, as a sum of 2^30 exponentials, each
// 2^14 above the reference at most, is then below 2^124; and 2^107, as the exponential of a key with such a
// scale is then still a normal number.
constexpr float kVrefLeast = 8.2718061e-25f, kVrefMost = 1.6225928e32f;
// log2 of how far P may exceed 1 before the reference moves: an fp16 P ends at 2^16, and O, a sum of P V over
// N keys, stays finite up to |V| N = 2^114.
constexpr float kRefGrow = 14.f;
// log2 of a value scale as P's reference counts it (NaN: the least).
__device__ __forceinline__ float vref_log2(float scale) {
  return __log2f(fminf(fmaxf(scale, kVrefLeast), kVrefMost));
}
// ln of a row's sum of exponentials from its maximum (log2 units) and the sum relative to it.
__device__ __forceinline__ float row_lse(float m, float sum) {
  return (m + log2f(sum)) * 0.6931471805599453f;
}

// ------------------------------------------------------------ few rows
// k_tree_rows: a tile of 16 rows (all the rows of a pair where T*G is small, up to 16
// with a 16-bit cache and 48, three tiles, with an e4m3 one) against the keys.  The legacy
// tensor path (no TMEM round trip, P stays in registers): two tiles a warp spilled with
// e4m3 (64 us against 48 to 53 for 20 rows of 8 heads).  Four warps; warp w owns keys
// 16w..16w+15 of each 64-key tile, with its own ring of TMA-filled stages, its own
// running maximum and sum and its own accumulator, so that nothing in the loop waits for
// another warp; they are added when the piece ends.
//
// Bound by issue and latency of each warp's chain (load, products, exponentials), not by the
// cache's bytes: one token over 32768 e4m3 slots of 8 heads takes 28 us here for 69 MB (2.5
// TB/s), half of its instructions widen codes, and a warp issues in one of five cycles.
//
// e4m3 cache: codes become fp16 in registers (exact).  Q (fp16 or bf16) enters as
// fp16 scaled by a power of two that puts the row's largest value at 2^13 (what
// falls below fp16's range is under 2^-37 of it).  The key scales multiply the
// scores; the value scales multiply P, whose reference is the largest of score + log2(value scale) among the
// keys that the row attends: a large value row that weighs nothing takes no bits from the others.
constexpr int kRowsWarps = 4;
constexpr int kRowsTile = 16 * kRowsWarps;
constexpr int kRowsLeast = 2;          // tiles that a block takes at least

template <int D, bool E4M3>
struct RowsCfg {
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kBoxBytes = kRowBytes < 128 ? kRowBytes : 128;   // swizzle span
  static constexpr int kBoxes = kRowBytes / kBoxBytes;
  static constexpr int kTileBytes = 16 * kRowBytes;                     // K or V of a warp's 16 keys
  static constexpr int kStageBytes = 2 * kTileBytes;
  // Blocks of an SM, and stages of a warp in the shared memory that leaves them.  A warp's chain of
  // waits, products and exponentials is long, so that more warps keep more bytes coming than deeper rings.
  static constexpr int kBlocks = D == 64 ? 4 : (E4M3 ? 3 : 2);
  static constexpr int kStages = E4M3 && D == 64 ? 4 : 2;
};

template <int D, bool E4M3>
struct __align__(1024) RowsSmem {
  using C = RowsCfg<D, E4M3>;
  uint8_t kv[kRowsWarps][C::kStages][C::kStageBytes];
  float sc[kRowsWarps][C::kStages][E4M3 ? 32 : 4];  // key scales, value scales
  float red[kRowsWarps][16][D + 4];                 // O of the rows of an m-tile
  float2 ml[kRowsWarps][16];
  uint64_t full[kRowsWarps][C::kStages];
  int bad[kRowsWarps][C::kStages];                  // the stage's page was out of range
  int abort_flag;
};

// Byte offset of 16-byte chunk `ch` of row `r` in a tile of 16 rows.
template <int D, bool E4M3>
__device__ __forceinline__ uint32_t rows_off(int r, int ch) {
  using C = RowsCfg<D, E4M3>;
  if (C::kBoxBytes == 128)
    return (ch >> 3) * (16 * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
  return r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
}

template <int D, bool E4M3, bool QBF>
__global__ void __launch_bounds__(32 * kRowsWarps, (RowsCfg<D, E4M3>::kBlocks))
    k_tree_rows(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ TreeArgs a) {
  using C = RowsCfg<D, E4M3>;
  constexpr bool BF = QBF && !E4M3;           // type of the MMA operands
  constexpr int NT = D / 8;                   // n-tiles of O
  extern __shared__ uint8_t smem_raw[];
  RowsSmem<D, E4M3>& sm = *reinterpret_cast<RowsSmem<D, E4M3>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int R = a.G * a.T, pairs = a.c.Hkv * a.RT;
  if (tid == 0) {
    for (int w = 0; w < kRowsWarps; ++w)
      for (int s = 0; s < C::kStages; ++s) mbar_init(&sm.full[w][s], 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  const Run run = warp_run(a, kRowsTile, pairs, gridDim.x, blockIdx.x, kRowsLeast);
  if (blockIdx.x == gridDim.x - 1 && warp == 0) write_before(a, kRowsTile, pairs);
  __syncthreads();
  const int nt = run.n;
  if (nt == 0) return;
  Cursor in, at;                              // where loads are issued; where work is done
  in.start(run, kRowsTile);
  at = in;
  int issued = 0, used = 0, in_t = 0;         // tiles with keys of this warp
  int page = -1;                              // of the tile to be issued next, asked for one tile ahead
  // On to the next tile in which this warp has keys.
  auto seek = [&]() {
    while (in_t < nt) {
      const int key0 = in.tile * kRowsTile + warp * 16;
      if (key0 < in.s.len + in.s.n) {
        page = __ldg(a.table + (size_t)in.b * a.MP + (key0 >> a.c.page_shift));
        return;
      }
      if (++in_t < nt) in.next(a, pairs, kRowsTile);
    }
  };
  // Issues the loads of that tile, if the run has one.
  auto issue = [&]() {
    if (in_t >= nt) return;
    if (lane == 0) {
      const int key0 = in.tile * kRowsTile + warp * 16;
      const int st = issued % C::kStages;
      const bool ok = page_inside(page, a.c.pages);
      if (!ok) atomicOr(&g_device_error, DEVERR_BOUNDS);
      sm.bad[warp][st] = !ok;
      const int row = (int)row_of(ok ? page : 0, a.c.Hkv, in.pair / a.RT, a.c.page_shift, key0);
      uint64_t* bar = &sm.full[warp][st];
      uint8_t* dst = sm.kv[warp][st];
      mbar_expect_tx(bar, C::kStageBytes + (E4M3 ? 128 : 0));
#pragma unroll
      for (int x = 0; x < C::kBoxes; ++x) {
        tma_load_2d(dst + x * 2048, &tm_k, bar, x * 64, row);
        tma_load_2d(dst + C::kTileBytes + x * 2048, &tm_v, bar, x * 64, row);
      }
      if (E4M3) {
        bulk_load(sm.sc[warp][st], a.c.ks + row, 64, bar);
        bulk_load(sm.sc[warp][st] + 16, a.c.vs + row, 64, bar);
      }
    }
    ++issued;
    if (++in_t < nt) in.next(a, pairs, kRowsTile);
    seek();
  };
  seek();
  for (int s = 0; s < C::kStages; ++s) issue();
  __syncwarp();                               // lane 0's sm.bad

  uint32_t qf[D / 16][4];
  float acc[NT][4];
  float m[2], l[2], qs[2];        // m: the reference (log2 units)
  const float kL2E = 1.4426950408889634f;

  for (int t = 0; t < nt; ++t) {
    const int L = at.s.len + at.s.n;
    const int row0 = (at.pair % a.RT) * 16;
    const int h = at.pair / a.RT;
    if (t == 0 || at.tile == 0) {
      // a piece starts: its rows' Q fragments
      const uint16_t* src[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row0 + g + 8 * e;
        src[e] = r < R ? static_cast<const uint16_t*>(a.q) + at.b * a.sb +
                             (long long)(h * a.G + r / a.T) * a.sh + (long long)(r % a.T) * a.st
                       : nullptr;
        m[e] = -INFINITY;
        l[e] = 0.f;
        qs[e] = a.sm_scale * kL2E;
      }
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          // 16 bit: k = 16 ks + 2c (+8).  e4m3: the thread's bytes of a key are
          // contiguous (D/4 of them), so k-step ks takes d = (D/4) c + 4 ks + {0,1}, {2,3}
          const int dd = E4M3 ? (D / 4) * c + 4 * ks + 2 * (u >> 1) : 16 * ks + 2 * c + 8 * (u >> 1);
          qf[ks][u] = src[u & 1] ? __ldg(reinterpret_cast<const uint32_t*>(src[u & 1] + dd)) : 0u;
        }
      if (E4M3) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float amax = 0.f;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int u = e; u < 4; u += 2) {
              const float2 f = halves<QBF>(qf[ks][u]);
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          // 2^(13 - exponent): an exact power of two; left alone where the row is 0 or not finite
          const int ex = (int)(__float_as_uint(amax) >> 23);
          const int sh = (ex == 0 || ex == 255) ? 0 : max(-114, min(60, 13 + 127 - ex));
          const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
          qs[e] *= __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
            for (int u = e; u < 4; u += 2) {
              const float2 f = halves<QBF>(qf[ks][u]);
              qf[ks][u] = pack2<false>(f.x * up, f.y * up);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[j][u] = 0.f;
    }

    const int key0 = at.tile * kRowsTile + warp * 16;
    if (key0 < L) {
      const int st = used % C::kStages;
      if (!mbar_wait_warp(&sm.full[warp][st], (used / C::kStages) & 1, &sm.abort_flag)) {
        // let the copies already issued land before the block exits
        for (int u = used; u < issued; ++u)
          mbar_wait(&sm.full[warp][u % C::kStages], (u / C::kStages) & 1, nullptr);
        return;
      }
      const uint8_t* kt = sm.kv[warp][st];
      const uint8_t* vt = kt + C::kTileBytes;
      const int live = sm.bad[warp][st] ? 0 : min(16, L - key0);   // keys of this tile that exist
      // Edge tiles: rows behind the last key may hold anything, and V there must not be
      // NaN under P = 0; nor in a drafted token's row, which some rows do not attend: such
      // a row becomes zeros, and the rows that do attend it get NaN from their scores.
      const bool edge = key0 + 16 > at.s.len || live < 16;
      unsigned badrows = 0;
      if (edge) {
        constexpr int PPR = C::kRowBytes / 16;
        uint8_t* vz = sm.kv[warp][st] + C::kTileBytes;
        const int first = max(0, at.s.len - key0);
        for (int i = lane; i < 16 * PPR; i += 32) {
          const int r = i / PPR;
          if (r >= first && r < live && not_finite16<E4M3, QBF>(*reinterpret_cast<const uint4*>(
                                            vz + rows_off<D, E4M3>(r, i % PPR))))
            badrows |= 1u << r;
        }
        if (E4M3 && lane < 16) {
          if (lane >= live) sm.sc[warp][st][lane] = 0.f;
          const float w = sm.sc[warp][st][16 + lane];
          if (lane >= first && lane < live && !(fabsf(w) < INFINITY)) badrows |= 1u << lane;
        }
        badrows = __reduce_or_sync(0xffffffffu, badrows);
        for (int i = lane; i < 16 * PPR; i += 32)
          if (i / PPR >= live || (badrows >> (i / PPR)) & 1u)
            *reinterpret_cast<uint4*>(vz + rows_off<D, E4M3>(i / PPR, i % PPR)) =
                make_uint4(0u, 0u, 0u, 0u);
        if (E4M3 && lane < 16 && (lane >= live || (badrows >> lane) & 1u)) sm.sc[warp][st][16 + lane] = 0.f;
        __syncwarp();
      }
      // ---- S = Q K^T
      float s[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) s[j][u] = 0.f;
      if (!E4M3) {
        const uint32_t base = smem_u32(kt);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t b[4];
          const int key = (lane >> 4) * 8 + (lane & 7), ch = 2 * ks + ((lane >> 3) & 1);
          ldsm4(base + rows_off<D, E4M3>(key, ch), b);
          mma16816<BF>(s[0], qf[ks], b[0], b[1]);
          mma16816<BF>(s[1], qf[ks], b[2], b[3]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            // 16 bytes of key 8j + g: d = (D/4) c + 16 x ..
            const uint4 w = *reinterpret_cast<const uint4*>(
                kt + rows_off<D, E4M3>(8 * j + g, (D / 64) * c + x));
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              uint32_t b0, b1;
              widen4(ww[y], b0, b1);
              mma16816<BF>(s[j], qf[4 * x + y], b0, b1);
            }
          }
      }
      // ---- softmax of the 16 keys: this thread has keys 8j + 2c + {0,1} of rows g, g+8.  The
      // exponentials are taken against the reference that the earlier keys have left; it moves (and
      // the sums and O with it) only when a score of the warp lies far above it.  e4m3: whether it does is
      // asked of a bound, the largest score and the tile's largest value scale (lv); where it moves to, of
      // each key's own.
      float kscl[2][2], vscl[2][2], lv = 0.f;
      if (E4M3) {
        float vm = kVrefLeast;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 k2 = *reinterpret_cast<const float2*>(&sm.sc[warp][st][8 * j + 2 * c]);
          const float2 v2 = *reinterpret_cast<const float2*>(&sm.sc[warp][st][16 + 8 * j + 2 * c]);
          kscl[j][0] = k2.x;
          kscl[j][1] = k2.y;
          vscl[j][0] = v2.x;
          vscl[j][1] = v2.y;
          vm = fmaxf(vm, fmaxf(v2.x, v2.y));
        }
        vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
        vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
        lv = __log2f(vm);
      }
      float x[2][2][2];
      bool over = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int y = 0; y < 2; ++y)
            x[e][j][y] = s[j][2 * e + y] * (E4M3 ? qs[e] * kscl[j][y] : qs[e]);
        if (edge) {
          const int r = row0 + g + 8 * e;
          const int i = r % a.T;
          const uint8_t* mask = a.mask ? a.mask + at.b * a.mask_sb : nullptr;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int k = 8 * j + 2 * c + y;
              const bool in = slot_allowed(a, mask, at.s, i, key0 + k);
              if (!(in && k < live && r < R)) x[e][j][y] = -INFINITY;
              else if ((badrows >> k) & 1u) x[e][j][y] = __int_as_float(0x7fffffff);
            }
        }
        const float mx = fmaxf(fmaxf(x[e][0][0], x[e][0][1]), fmaxf(x[e][1][0], x[e][1][1]));
        over = over || (mx > -INFINITY && mx + lv > m[e] + kRefGrow);
      }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              mx = fmaxf(mx, E4M3 ? x[e][j][y] + vref_log2(vscl[j][y]) : x[e][j][y]);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const float now = fmaxf(m[e], mx);
          const float f = m[e] == -INFINITY ? 0.f : ex2(m[e] - now);
          m[e] = now;
          l[e] *= f;
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            acc[j][2 * e] *= f;
            acc[j][2 * e + 1] *= f;
          }
        }
      }
      uint32_t pf[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mb = m[e] == -INFINITY ? 0.f : m[e];
        float p[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int y = 0; y < 2; ++y) p[j][y] = ex2(x[e][j][y] - mb);
        l[e] += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
        if (E4M3) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y) p[j][y] *= vscl[j][y];
        }
        pf[e] = pack2<BF>(p[0][0], p[0][1]);
        pf[2 + e] = pack2<BF>(p[1][0], p[1][1]);
      }
      // ---- O += P V
      if (!E4M3) {
        const uint32_t base = smem_u32(vt);
#pragma unroll
        for (int jj = 0; jj < NT / 2; ++jj) {
          uint32_t b[4];
          const int key = ((lane >> 3) & 1) * 8 + (lane & 7), ch = 2 * jj + (lane >> 4);
          ldsm4_t(base + rows_off<D, E4M3>(key, ch), b);
          mma16816<BF>(acc[2 * jj], pf, b[0], b[1]);
          mma16816<BF>(acc[2 * jj + 1], pf, b[2], b[3]);
        }
      } else {
        // keys 2c, 2c+1, 2c+8, 2c+9; column g of n-tile j is d = (D/8) g + j
        uint32_t w[4][D / 32];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 2 * c + (k & 1) + 8 * (k >> 1);
          if (D == 128) {
            *reinterpret_cast<uint4*>(w[k]) =
                *reinterpret_cast<const uint4*>(vt + rows_off<D, E4M3>(key, g));
          } else {
            *reinterpret_cast<uint2*>(w[k]) =
                *reinterpret_cast<const uint2*>(vt + rows_off<D, E4M3>(key, g >> 1) + 8 * (g & 1));
          }
        }
#pragma unroll
        for (int x = 0; x < D / 32; ++x)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const uint32_t sel = hh ? 0x7362u : 0x5140u;
            uint32_t b0[2], b1[2];
            widen4(__byte_perm(w[0][x], w[1][x], sel), b0[0], b0[1]);
            widen4(__byte_perm(w[2][x], w[3][x], sel), b1[0], b1[1]);
#pragma unroll
            for (int y = 0; y < 2; ++y)
              mma16816<BF>(acc[4 * x + 2 * hh + y], pf, b0[y], b1[y]);
          }
      }
      __syncwarp();
      if (edge) fence_proxy_async_smem();        // the zeros above, before the next TMA write
      __syncwarp();
      ++used;
      issue();
    }

    // ---- the piece ends with the pair's last tile or the run's
    if (at.tile + 1 == at.tiles || t + 1 == nt) {
      const int first = at.tile - min(t, at.tile);   // the piece's first tile of the pair
      const bool whole = first == 0 && at.tile + 1 == at.tiles;
      const int slot = 2 * blockIdx.x + (first == 0 ? 1 : 0);
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[e];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (c == 0) sm.ml[warp][g + 8 * e] = make_float2(m[e], x);
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, sm.ml[w][g + 8 * e].x);
        f[e] = ex2(m[e] - (M == -INFINITY ? 0.f : M));
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (row0 + g + 8 * e >= R) continue;
        float* to = sm.red[warp][g + 8 * e];
        if (!E4M3) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            *reinterpret_cast<float2*>(to + 8 * j + 2 * c) =
                make_float2(acc[j][2 * e] * f[e], acc[j][2 * e + 1] * f[e]);
        } else {
          // column y of n-tile j is d = (D/8) (2c + y) + j
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < NT; j += 4)
              *reinterpret_cast<float4*>(to + NT * (2 * c + y) + j) =
                  make_float4(acc[j][2 * e + y] * f[e], acc[j + 1][2 * e + y] * f[e],
                              acc[j + 2][2 * e + y] * f[e], acc[j + 3][2 * e + y] * f[e]);
        }
      }
      __syncthreads();
      // eight threads a row, every eighth float4
      const int rr = tid >> 3, r = row0 + rr;
      if (r < R) {
        float M = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) M = fmaxf(M, sm.ml[w][rr].x);
        const float mb = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int w = 0; w < kRowsWarps; ++w) sum += ex2(sm.ml[w][rr].x - mb) * sm.ml[w][rr].y;
        const int i = r % a.T;
        const bool none = i >= at.s.n || sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum;
        const size_t row = whole ? ((size_t)at.b * a.Hq + h * a.G + r / a.T) * a.T + i
                                 : (size_t)slot * 16 + rr;
#pragma unroll
        for (int col = 4 * (tid & 7); col < D; col += 32) {
          float4 v = *reinterpret_cast<const float4*>(&sm.red[0][rr][col]);
#pragma unroll
          for (int w = 1; w < kRowsWarps; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(&sm.red[w][rr][col]);
            v.x += y.x;
            v.y += y.y;
            v.z += y.z;
            v.w += y.w;
          }
          float o4[4] = {v.x, v.y, v.z, v.w};
          if (whole) {
#pragma unroll
            for (int x = 0; x < 4; ++x) o4[x] = none ? 0.f : o4[x] * inv;
            store4(a.o, a.o_dtype, row * D + col, o4);
          } else {
            store4(a.part, 2, row * D + col, o4);
          }
        }
        if ((tid & 7) == 0) {
          if (!whole) a.part_ml[row] = make_float2(M, sum);
          else if (a.lse) a.lse[row] = none ? -INFINITY : row_lse(M, sum);
        }
      }
      __syncthreads();
    }
    if (t + 1 < nt) at.next(a, pairs, kRowsTile);
  }
}

// ------------------------------------------------------------ adding pieces
// Rows of a pair that one block covered are done; the others (and the pairs without any tile) are
// written here.  The pieces' maxima and sums are read at once, then the channels of all pieces with
// loads that do not wait for one another (a warp that went from piece to piece took 23 us for
// the 37 pieces of one token's heads).  k_tree_join: a block a row, thread d for channel d; for
// rows of many pieces.  k_tree_join_few: a warp a row.
constexpr int kMostBlocks = 1024;       // of a split
// Blocks a pair from which on a row has a block.  Whole call, block / warp a row, us: bf16, d = 128, 1 row a pair (a grid
// of 296): 1 pair of 32768 slots 28 / 66, 8 pairs 34 / 39, 32 pairs of 16384 51.5 / 52.8, 48 pairs of 8000 43.3 / 43.1;
// 200 rows (a grid of 148): 8 pairs 68 / 69, 16 pairs 103 / 100, 64 pairs of 8192 126 / 105.
constexpr int kJoinFew = 8;
template <int D>
__global__ void __launch_bounds__(128) k_tree_join_few(const __grid_constant__ TreeArgs a, int tile,
                                                       int rows_tile, int grid, int least) {
  const int b = blockIdx.z, h = blockIdx.y, lane = threadIdx.x & 31;
  const int R = a.G * a.T, r = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (r >= R) return;
  const SeqLen s = seq_len(a.lens, a.n, b, a.T, a.MP, a.c.page_shift);
  const int tiles = pair_tiles(s, tile);
  const int i = r % a.T;
  const size_t orow = ((size_t)b * a.Hq + h * a.G + r / a.T) * a.T + i;
  constexpr int PER = D / 32;
  float o[PER] = {};
  float M = -INFINITY, sum = 0.f;
  if (tiles > 0) {
    const long long total = a.before[a.B];
    const int gr = run_blocks(total, grid, least);
    const long long P0 = a.before[b] + (long long)(h * a.RT + r / rows_tile) * tiles;
    const int c0 = run_of(P0, total, gr), np = run_of(P0 + tiles - 1, total, gr) - c0 + 1;
    if (np == 1) return;
    const size_t prow0 = (size_t)2 * c0 * rows_tile + r % rows_tile;
    for (int x0 = 0; x0 < np; x0 += 32) {
      const int x = x0 + lane, m = min(32, np - x0);
      const float2 ml = x < np ? a.part_ml[prow0 + (size_t)(2 * x + (x == 0 ? 1 : 0)) * rows_tile]
                               : make_float2(-INFINITY, 0.f);
      float mn = ml.x;
#pragma unroll
      for (int k = 16; k; k >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, k));
      mn = fmaxf(mn, M);
      const float mb = mn == -INFINITY ? 0.f : mn;
      const float f0 = ex2(M - mb), f1 = ex2(ml.x - mb);
      float part = f1 * ml.y;
#pragma unroll
      for (int k = 16; k; k >>= 1) part += __shfl_xor_sync(0xffffffffu, part, k);
      sum = sum * f0 + part;
      M = mn;
#pragma unroll
      for (int y = 0; y < PER; ++y) o[y] *= f0;
#pragma unroll 4
      for (int z = 0; z < m; ++z) {
        const int xx = x0 + z;
        const float f = __shfl_sync(0xffffffffu, f1, z);
        const float* src = a.part + (prow0 + (size_t)(2 * xx + (xx == 0 ? 1 : 0)) * rows_tile) * D + lane * PER;
        if (PER == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          o[0] += f * v.x;
          o[1] += f * v.y;
          o[PER - 2] += f * v.z;
          o[PER - 1] += f * v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          o[0] += f * v.x;
          o[1] += f * v.y;
        }
      }
    }
  }
  const bool none = i >= s.n || sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
#pragma unroll
  for (int y = 0; y < PER; ++y) o[y] = none ? 0.f : o[y] * inv;
  const size_t idx = orow * D + lane * PER;
  if (PER == 4) {
    const float f4[4] = {o[0], o[1], o[PER - 2], o[PER - 1]};
    store4(a.o, a.o_dtype, idx, f4);
  } else {
    store2(a.o, a.o_dtype, idx, o[0], o[1]);
  }
  if (a.lse && lane == 0) a.lse[orow] = none ? -INFINITY : row_lse(M, sum);
}

template <int D>
__global__ void __launch_bounds__(128) k_tree_join(const __grid_constant__ TreeArgs a, int tile,
                                                   int rows_tile, int grid, int least) {
  __shared__ float fac[kMostBlocks];
  __shared__ float red[2][4];
  __shared__ float half[D];
  const int b = blockIdx.z, h = blockIdx.y, r = blockIdx.x;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const SeqLen s = seq_len(a.lens, a.n, b, a.T, a.MP, a.c.page_shift);
  const int tiles = pair_tiles(s, tile);
  const int i = r % a.T;
  const size_t orow = ((size_t)b * a.Hq + h * a.G + r / a.T) * a.T + i;
  float M = -INFINITY, sum = 0.f, o = 0.f;
  if (tiles > 0) {
    const long long total = a.before[a.B];
    const int gr = run_blocks(total, grid, least);
    const long long P0 = a.before[b] + (long long)(h * a.RT + r / rows_tile) * tiles;
    const int c0 = run_of(P0, total, gr), np = run_of(P0 + tiles - 1, total, gr) - c0 + 1;
    if (np == 1) return;
    const size_t prow0 = (size_t)2 * c0 * rows_tile + r % rows_tile;
    auto prow = [&](int x) { return prow0 + (size_t)(2 * x + (x == 0 ? 1 : 0)) * rows_tile; };
    for (int x = tid; x < np; x += 128) M = fmaxf(M, a.part_ml[prow(x)].x);
#pragma unroll
    for (int k = 16; k; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
    M = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
    const float mb = M == -INFINITY ? 0.f : M;
    for (int x = tid; x < np; x += 128) {
      const float2 ml = a.part_ml[prow(x)];
      fac[x] = ex2(ml.x - mb);
      sum += fac[x] * ml.y;
    }
#pragma unroll
    for (int k = 16; k; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
    if (lane == 0) red[1][warp] = sum;
    __syncthreads();
    sum = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
    // D = 64: the two halves of the block take every other piece
    constexpr int kStep = 128 / D;
    const float* src = a.part + tid % D;
#pragma unroll 8
    for (int x = tid / D; x < np; x += kStep) o += fac[x] * src[prow(x) * D];
    if (kStep == 2) {
      if (tid >= D) half[tid - D] = o;
      __syncthreads();
      if (tid < D) o += half[tid];
    }
  }
  if (tid >= D) return;
  const bool none = i >= s.n || sum == 0.f;
  const float v = none ? 0.f : o / sum;
  const size_t idx = orow * D + tid;
  if (a.o_dtype == 0) static_cast<__half*>(a.o)[idx] = __float2half_rn(v);
  else if (a.o_dtype == 1) static_cast<__nv_bfloat16*>(a.o)[idx] = __float2bfloat16_rn(v);
  else static_cast<float*>(a.o)[idx] = v;
  if (a.lse && tid == 0) a.lse[orow] = none ? -INFINITY : row_lse(M, sum);
}

// ------------------------------------------------------------ launches
static int sm_count(int dev) {
  static int n[64] = {};
  if (dev < 0 || dev >= 64) return 148;
  if (n[dev] == 0) {
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0)
      v = 148;
    n[dev] = v < kMostBlocks / 4 ? v : kMostBlocks / 4;
  }
  return n[dev];
}

// Workspace of a split: partial rows, their maxima and sums, the tiles before each sequence.
static cudaError_t split_workspace(TreeArgs* a, size_t prow, int D, cudaMemPool_t pool, cudaStream_t st) {
  const size_t p = up256(prow * D * 4), m = up256(prow * 8);
  uint8_t* ws = nullptr;
  const cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void**>(&ws), p + m + (size_t)(a->B + 1) * 8,
                                                pool, st);
  if (e != cudaSuccess) return e;
  a->part = reinterpret_cast<float*>(ws);
  a->part_ml = reinterpret_cast<float2*>(ws + p);
  a->before = reinterpret_cast<long long*>(ws + p + m);
  return cudaSuccess;
}

template <int D>
static cudaError_t launch_join(const TreeArgs& a, int tile, int rows_tile, int grid, int least, cudaStream_t st) {
  const int R = a.G * a.T;
  if ((int64_t)a.B * a.c.Hkv * a.RT * kJoinFew <= grid)
    k_tree_join<D><<<dim3(R, a.c.Hkv, a.B), 128, 0, st>>>(a, tile, rows_tile, grid, least);
  else
    k_tree_join_few<D><<<dim3((R + 3) / 4, a.c.Hkv, a.B), 128, 0, st>>>(a, tile, rows_tile, grid, least);
  return cudaGetLastError();
}

template <int D, bool E4M3, bool QBF>
static cudaError_t launch_rows(TreeArgs a, int dev, cudaMemPool_t pool, cudaStream_t st) {
  using C = RowsCfg<D, E4M3>;
  a.RT = (a.G * a.T + 15) / 16;
  const int grid = C::kBlocks * sm_count(dev);
  CUtensorMap tk, tv;
  const uint64_t rows = (uint64_t)a.c.pages * a.c.Hkv << a.c.page_shift;
  const int eb = E4M3 ? 1 : 2;
  const uint64_t dims[2] = {(uint64_t)D, rows};
  const uint64_t strides[1] = {(uint64_t)D * eb};
  const uint32_t box[2] = {(uint32_t)(C::kBoxBytes / eb), 16};
  cudaError_t e = make_tmap(&tk, a.c.k, 2, dims, strides, box, eb, C::kBoxBytes);
  if (e == cudaSuccess) e = make_tmap(&tv, a.c.v, 2, dims, strides, box, eb, C::kBoxBytes);
  if (e != cudaSuccess) return e;
  const size_t prow = (size_t)2 * grid * 16;
  e = split_workspace(&a, prow, D, pool, st);
  if (e != cudaSuccess) return e;
  auto kern = k_tree_rows<D, E4M3, QBF>;
  const int smem = sizeof(RowsSmem<D, E4M3>) + 1024;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) {
    kern<<<grid, 32 * kRowsWarps, smem, st>>>(tk, tv, a);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess) {
    e = launch_join<D>(a, kRowsTile, 16, grid, kRowsLeast, st);
  }
  const cudaError_t e2 = cudaFreeAsync(a.part, st);
  return e != cudaSuccess ? e : e2;
}

}  // namespace sage2
#include "tree_tiles.cu"
#include "weights_tiles.cu"
namespace sage2 {

template <int D, bool E4M3, bool QBF>
static cudaError_t tree_pick(const TreeArgs& a, int dev, cudaMemPool_t pool, cudaStream_t st) {
  // A row tile of 16 reads the cache once more, from L2 mostly; k_tree_tiles reads it once and costs the same
  // for 17 rows as for 128.  Measured, us (1 x 32768 / 8 x 4096 / 32 x 1000 slots), tiles of 16 | k_tree_tiles:
  //   16 bits  d = 128   8 heads  16 rows  36 / 37 / 36 | 37 / 39 / 40       20 rows  53 / 51 / 55 | 38 / 40 / 41
  //                     32 heads  16 rows  95 / 95 / 105 | 96 / 98 / 112     20 rows  167 / 172 / 182 | 96 / 98 / 116
  //            d = 64    8 heads  16 rows  24 / 24 / 23 | 28 / 31 / 31       20 rows  31 / 32 / 32 | 29 / 32 / 32
  //   e4m3     d = 128   8 heads  48 rows  70 / 72 / 85 | 77 / 87 / 118      64 rows  85 / 87 / 109 | 79 / 89 / 123
  //                     32 heads  48 rows  216 / 229 / 281 | 269 / 315 / 415  64 rows  277 / 299 / 380 | 275 / 320 / 425
  //            d = 64    8 heads  48 rows  50 / 52 / 60 | 69 / 73 / 100      64 rows  62 / 65 / 77 | 69 / 74 / 103
  // Past the limits tiles of 16 lead still for one head of 16 bits (64 rows over 32768 slots 25 | 36), and with e4m3
  // up to 64 rows for d = 64 and for many short sequences.
  const int R = a.G * a.T;
  if (R <= (E4M3 ? 48 : 16)) return launch_rows<D, E4M3, QBF>(a, dev, pool, st);
  if (R <= kTR) return launch_tiles<D, E4M3, QBF, false>(a, dev, pool, st);
  return launch_tiles<D, E4M3, QBF, true>(a, dev, pool, st);
}

// What sage2_attn_tree and sage2_cache_weights check alike.
static sage2_status tree_args(const void* q, int dtype, const int64_t* q_strides,
                              const sage2_cache* cache, const int* table, int max_pages,
                              const int* lens, const int* n, const uint8_t* mask,
                              int64_t mask_stride, int B, int Hq, int T, float sm_scale, TreeArgs* a) {
  sage2_status s = check_cache(cache, &a->c);
  if (s != SAGE2_OK) return s;
  s = check_table(a->c, B, max_pages);
  if (s != SAGE2_OK) return s;
  if (dtype != SAGE2_F16 && dtype != SAGE2_BF16) return SAGE2_ERR_INVALID_ARG;
  if (a->c.kv_dtype != SAGE2_E4M3 && dtype != a->c.kv_dtype) return SAGE2_ERR_INVALID_ARG;
  if (Hq <= 0 || Hq % a->c.Hkv != 0 || T <= 0) return SAGE2_ERR_INVALID_ARG;
  if (T > 1024 || (int64_t)Hq * T > INT32_MAX) return SAGE2_ERR_UNSUPPORTED;
  if (!(sm_scale >= 1e-20f) || sm_scale > 1e20f) return SAGE2_ERR_INVALID_ARG;
  if (mask_stride < 0) return SAGE2_ERR_INVALID_ARG;
  s = check_ptrs(q);
  if (s != SAGE2_OK) return s;
  s = check_words(table, lens);
  if (s != SAGE2_OK) return s;
  if (n && !aligned4(n)) return SAGE2_ERR_MISALIGNED;
  long long st[3];
  s = take_strides(q_strides, Hq, T, a->c.d, st);
  if (s != SAGE2_OK) return s;
  a->sb = st[0];
  a->sh = st[1];
  a->st = st[2];
  a->table = table;
  a->lens = lens;
  a->n = n;
  a->mask = mask;
  a->mask_sb = mask_stride;
  a->q = q;
  a->B = B;
  a->Hq = Hq;
  a->G = Hq / a->c.Hkv;
  a->T = T;
  a->MP = max_pages;
  a->sm_scale = sm_scale;
  a->RT = 1;
  return SAGE2_OK;
}

}  // namespace sage2

extern "C" {

sage2_status sage2_attn_tree(const void* q, int dtype, const int64_t* q_strides,
                             const sage2_cache* cache, const int* table, int max_pages,
                             const int* lens, const int* n, const uint8_t* mask,
                             int64_t mask_stride, void* o, int o_dtype, float* lse, int B, int Hq,
                             int T, float sm_scale, sage2_stream_t stream) {
  using namespace sage2;
  TreeArgs a{};
  sage2_status s = tree_args(q, dtype, q_strides, cache, table, max_pages, lens, n, mask, mask_stride,
                             B, Hq, T, sm_scale, &a);
  if (s != SAGE2_OK) return s;
  if (o_dtype < SAGE2_F16 || o_dtype > SAGE2_F32) return SAGE2_ERR_INVALID_ARG;
  s = check_ptrs(o);
  if (s != SAGE2_OK) return s;
  if (lse && !aligned4(lse)) return SAGE2_ERR_MISALIGNED;
  a.o = o;
  a.o_dtype = o_dtype;
  a.lse = lse;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAGE2_ERR_CUDA;
  cudaMemPool_t pool = device_pool(dev);
  if (!pool) return SAGE2_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf = dtype == SAGE2_BF16, e4 = a.c.kv_dtype == SAGE2_E4M3;
  cudaError_t e;
  if (a.c.d == 64)
    e = e4 ? (bf ? tree_pick<64, true, true>(a, dev, pool, st) : tree_pick<64, true, false>(a, dev, pool, st))
           : (bf ? tree_pick<64, false, true>(a, dev, pool, st) : tree_pick<64, false, false>(a, dev, pool, st));
  else
    e = e4 ? (bf ? tree_pick<128, true, true>(a, dev, pool, st) : tree_pick<128, true, false>(a, dev, pool, st))
           : (bf ? tree_pick<128, false, true>(a, dev, pool, st) : tree_pick<128, false, false>(a, dev, pool, st));
  return from_cuda(e);
}

sage2_status sage2_cache_weights(const void* q, int dtype, const int64_t* q_strides,
                                 const float* lse, const sage2_cache* cache, const int* table,
                                 int max_pages, const int* lens, const int* n, const uint8_t* mask,
                                 int64_t mask_stride, float* acc, const int64_t* acc_strides, int S,
                                 int B, int Hq, int T, float sm_scale, sage2_stream_t stream) {
  using namespace sage2;
  TreeArgs a{};
  sage2_status s = tree_args(q, dtype, q_strides, cache, table, max_pages, lens, n, mask, mask_stride,
                             B, Hq, T, sm_scale, &a);
  if (s != SAGE2_OK) return s;
  s = check_words(lse, acc);
  if (s != SAGE2_OK) return s;
  if (S <= 0 || !acc_strides || !heads_apart(acc_strides, B, a.c.Hkv, S)) return SAGE2_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return SAGE2_ERR_CUDA;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const long long ab = acc_strides[0], ah = acc_strides[1];
  const bool bf = dtype == SAGE2_BF16, e4 = a.c.kv_dtype == SAGE2_E4M3;
  cudaError_t e;
  if (a.c.d == 64)
    e = e4 ? (bf ? launch_weights_tiles<64, true, true>(a, lse, acc, ab, ah, S, dev, st)
                 : launch_weights_tiles<64, true, false>(a, lse, acc, ab, ah, S, dev, st))
           : (bf ? launch_weights_tiles<64, false, true>(a, lse, acc, ab, ah, S, dev, st)
                 : launch_weights_tiles<64, false, false>(a, lse, acc, ab, ah, S, dev, st));
  else
    e = e4 ? (bf ? launch_weights_tiles<128, true, true>(a, lse, acc, ab, ah, S, dev, st)
                 : launch_weights_tiles<128, true, false>(a, lse, acc, ab, ah, S, dev, st))
           : (bf ? launch_weights_tiles<128, false, true>(a, lse, acc, ab, ah, S, dev, st)
                 : launch_weights_tiles<128, false, false>(a, lse, acc, ab, ah, S, dev, st));
  return from_cuda(e);
}

}  // extern "C"
