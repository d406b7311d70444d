// Paged key/value cache: writing new tokens (sage2_cache_append), choosing the
// tokens to keep by accumulated attention weight and moving rows
// (sage2_cache_evict, sage2_cache_compact).
//
// Slot s of sequence b is row s % page of page table[b][s / page]; a page holds
// `page` rows of d values for each head, head-major, so a head's rows of one
// page are contiguous.
//
// Device-side integers (table, lens, n, idx) are checked where they are used:
// one that points outside the pools or the table sets DEVERR_BOUNDS and the
// row it names is skipped.
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cache_index.h"
#include "sage2.h"
#include "sage2_internal.h"
#include "sm100_ptx.cuh"

namespace sage2 {

// Row (in units of one head's rows over the pool) of slot `slot`; -1 (and the
// error word) if the slot or its page is out of range.
__device__ __forceinline__ long long cache_row(const CacheView& c, const int* table, int MP, int b,
                                               int h, int slot) {
  if (!slot_inside(slot, c.page_shift, MP)) {
    atomicOr(&g_device_error, DEVERR_BOUNDS);
    return -1;
  }
  const int page = __ldg(table + (size_t)b * MP + (slot >> c.page_shift));
  if (!page_inside(page, c.pages)) {
    atomicOr(&g_device_error, DEVERR_BOUNDS);
    return -1;
  }
  return row_of(page, c.Hkv, h, c.page_shift, slot);
}

// The 16-bit value with these bits.
template <typename T>
__device__ __forceinline__ float to_float(uint32_t bits);
template <>
__device__ __forceinline__ float to_float<__half>(uint32_t bits) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(uint32_t bits) {
  return __uint_as_float(bits << 16);
}

// Data that this kernel alone reads, and once: not kept in L1.
__device__ __forceinline__ uint4 ld_once(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// ---------------------------------------------------------------------------
// Append.  D/16 lanes own one row of K or V (32 bytes each) and have kAppendRows of them in
// flight; a block works for one head of one sequence.  4 x 32 heads x 8192 tokens, d = 128: 16 bits 165 us
// (6.5 TB/s, memory), e4m3 147 us (5.5 TB/s; bound by instruction issue, 80% of its slots: 53 instructions
// for 16 bytes of input).  e4m3: scale = amax/448, code = e4m3(x * (448/amax)), all fp32 RN, the
// same rounding as the quantized V; a row of zeros has scale 0, a row with an
// infinity or NaN has scale NaN, so that whatever reads it sees NaN.
struct AppendArgs {
  const void* x[2];        // k, v
  long long sb[2], sh[2], st[2];  // strides in elements
  CacheView c;
  const int* table;
  const int* lens;
  const int* n;            // null: T
  int B, T, MP;
};

constexpr int kAppendRows = 2;           // rows that a thread has in flight

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(256) k_cache_append(AppendArgs a) {
  constexpr int LPR = D / 16;           // lanes of a row, two 16-byte pieces each
  constexpr int RPB = 256 / LPR;        // rows of a pass
  const int kv = blockIdx.z, h = blockIdx.x % a.c.Hkv, b = blockIdx.x / a.c.Hkv;
  const int lane = threadIdx.x % LPR;
  const int len = __ldg(a.lens + b);
  int n = a.T;
  if (a.n) {
    n = __ldg(a.n + b);
    if (static_cast<unsigned>(n) > static_cast<unsigned>(a.T)) {
      atomicOr(&g_device_error, DEVERR_BOUNDS);
      return;
    }
  }
  if (len < 0 || len > INT_MAX - a.T) {
    if (n > 0) atomicOr(&g_device_error, DEVERR_BOUNDS);
    return;
  }
  const T* x0 = static_cast<const T*>(a.x[kv]) + b * a.sb[kv] + h * a.sh[kv];
  uint8_t* pool = kv ? a.c.v : a.c.k;
  // whole rows take part, so that the shuffles stay among lanes that are there
  const unsigned act = ((1u << LPR) - 1u) << (threadIdx.x % 32 / LPR * LPR);
  const int step = gridDim.y * RPB * kAppendRows;
  for (int t0 = blockIdx.y * RPB * kAppendRows + threadIdx.x / LPR; t0 < n; t0 += step) {
    uint4 u[kAppendRows][2];
    long long dst[kAppendRows];
#pragma unroll
    for (int r = 0; r < kAppendRows; ++r) {
      const int t = t0 + r * RPB;
      dst[r] = -1;
      if (t < n) {
        const uint4* src = reinterpret_cast<const uint4*>(x0 + (long long)t * a.st[kv]) + lane;
        u[r][0] = ld_once(src);
        u[r][1] = ld_once(src + LPR);
        dst[r] = cache_row(a.c, a.table, a.MP, b, h, len + t);
      }
    }
#pragma unroll
    for (int r = 0; r < kAppendRows; ++r) {
      if (t0 + r * RPB >= n || dst[r] < 0) continue;
      if (!E4M3) {
        uint4* to = reinterpret_cast<uint4*>(pool + dst[r] * D * 2) + lane;
        to[0] = u[r][0];
        to[LPR] = u[r][1];
        continue;
      }
      // largest magnitude as integers, two 16-bit values a word (their order is that of the bits; an
      // infinity or NaN is the largest of all)
      uint32_t m2 = 0;
#pragma unroll
      for (int p = 0; p < 2; ++p)
        m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(u[r][p].x & 0x7fff7fffu, u[r][p].y & 0x7fff7fffu),
                                   __vmaxu2(u[r][p].z & 0x7fff7fffu, u[r][p].w & 0x7fff7fffu)));
#pragma unroll
      for (int o = LPR / 2; o; o >>= 1) m2 = __vmaxu2(m2, __shfl_xor_sync(act, m2, o));
      const uint32_t mb = max(m2 & 0xffffu, m2 >> 16);
      const bool bad = mb >= (std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u);
      const float amax = to_float<T>(mb);
      // below 2^-100 the inverse would pass fp32's range: such a row is zero
      const bool nz = amax >= 7.8886e-31f;
      // one division a lane: the even ones' 448 / amax goes into the codes, the odd ones' amax / 448
      // is the scale
      const float q = nz ? __fdiv_rn(lane & 1 ? amax : 448.f, lane & 1 ? 448.f : amax) : 0.f;
      const float inv = __shfl_sync(act, q, 0, LPR);
      const float2 inv2 = make_float2(inv, inv);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        float x[8];
        unpack8<T>(u[r][p], x);
        uint32_t w[2];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const float2 lo = __fmul2_rn(make_float2(x[4 * g], x[4 * g + 1]), inv2);
          const float2 hi = __fmul2_rn(make_float2(x[4 * g + 2], x[4 * g + 3]), inv2);
          w[g] = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
                 static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16;
        }
        reinterpret_cast<uint2*>(pool + dst[r] * D)[lane + p * LPR] = make_uint2(w[0], w[1]);
      }
      if (lane == 1) (kv ? a.c.vs : a.c.ks)[dst[r]] = bad ? __int_as_float(0x7fffffff) : q;
    }
  }
}

template <typename T, int D, bool E>
static cudaError_t append_go(const AppendArgs& a, cudaStream_t st) {
  const int rows = 256 / (D / 16) * kAppendRows;
  const int blocks = (a.T + rows - 1) / rows;
  k_cache_append<T, D, E><<<dim3((unsigned)(a.B * a.c.Hkv), blocks < 65535 ? blocks : 65535, 2), 256, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t append_pick(const AppendArgs& a, int d, bool e4m3, cudaStream_t st) {
  if (d == 64) return e4m3 ? append_go<T, 64, true>(a, st) : append_go<T, 64, false>(a, st);
  return e4m3 ? append_go<T, 128, true>(a, st) : append_go<T, 128, false>(a, st);
}

// ---------------------------------------------------------------------------
// Choice of the tokens to keep.  One block per (sequence, head).  The tallies
// of the middle (neither among the first `sinks` nor the last `recent`) are
// mapped to integers of the same order (NaN lowest, -0 like +0) and kept in shared
// memory while they fit there (SMEM: one pass over the tally).  The
// (keep - sinks - recent)-th largest is found by three radix passes of 11, 11 and 10
// bits; then each thread counts its run of consecutive slots, a scan over the block gives
// where its choices go, and the chosen slots are written ascending, the equal ones
// from the lowest slot on.  Bound by the latency of its passes, one block a head: 14 us for 24 heads of 17776
// tallies, 23 us for 128 heads of 32768.
struct SelectArgs {
  const float* acc;
  long long sb, sh;        // strides of acc in elements
  const int* lens;
  int* idx;                // [B, Hkv, keep]
  int* new_lens;           // [B]
  int Hkv, S, keep, sinks, recent;
};

__device__ __forceinline__ uint32_t tally_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(__fadd_rn(x, 0.f));  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelKeys = 54000;          // of the middle that fit beside the rest (227 KB)

// Exclusive sums over the block (1024 threads); *all: the total.
__device__ __forceinline__ uint2 scan_block(uint2 v, uint2 (&part)[32], uint2* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint2 incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) {
      incl.x += x;
      incl.y += y;
    }
  }
  __syncthreads();                       // part is free
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  uint2 w = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, w.x, o), y = __shfl_up_sync(0xffffffffu, w.y, o);
    if (lane >= o) {
      w.x += x;
      w.y += y;
    }
  }
  all->x = __shfl_sync(0xffffffffu, w.x, 31);
  all->y = __shfl_sync(0xffffffffu, w.y, 31);
  uint2 before = make_uint2(__shfl_sync(0xffffffffu, w.x, (warp + 31) & 31),
                            __shfl_sync(0xffffffffu, w.y, (warp + 31) & 31));
  if (warp == 0) before = make_uint2(0u, 0u);
  return make_uint2(before.x + incl.x - v.x, before.y + incl.y - v.y);
}

template <bool SMEM>
__global__ void __launch_bounds__(kSelThreads) k_cache_select(SelectArgs a) {
  extern __shared__ uint32_t keys[];     // SMEM: the middle
  __shared__ uint32_t hist[kSelBins];
  __shared__ uint2 part[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  int len = __ldg(a.lens + b);
  if (len < 0 || len > a.S) {
    if (tid == 0) atomicOr(&g_device_error, DEVERR_BOUNDS);
    len = len < 0 ? 0 : a.S;
  }
  const int m = min(len, a.keep);
  int* out = a.idx + ((size_t)b * a.Hkv + h) * a.keep;
  if (h == 0 && tid == 0) a.new_lens[b] = m;
  for (int i = m + tid; i < a.keep; i += kSelThreads) out[i] = -1;
  if (len <= a.keep) {
    for (int i = tid; i < m; i += kSelThreads) out[i] = i;
    return;
  }
  const int lo = a.sinks, n = len - a.recent - lo;   // the middle: n slots from lo on, more than `want`
  const int want = a.keep - a.sinks - a.recent;
  for (int i = tid; i < lo; i += kSelThreads) out[i] = i;
  for (int i = tid; i < a.recent; i += kSelThreads) out[lo + want + i] = lo + n + i;
  if (want == 0) return;
  const float* acc = a.acc + b * a.sb + h * a.sh + lo;
  auto key = [&](int i) { return SMEM ? keys[i] : tally_key(__ldg(acc + i)); };
  for (int i = tid; i < kSelBins; i += kSelThreads) hist[i] = 0;
  __syncthreads();
  uint32_t prefix = 0;
  int need = want;                       // still to take among those with the prefix
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    if (pass == 0 && SMEM) {
#pragma unroll 8
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t k = tally_key(__ldg(acc + i));
        keys[i] = k;
        atomicAdd(&hist[k >> 21], 1u);
      }
    } else {
#pragma unroll 4
      for (int i = tid; i < n; i += kSelThreads) {
        const uint32_t k = key(i);
        if (pass == 0 || (k >> (shift + bits)) == prefix) atomicAdd(&hist[(k >> shift) & ((1 << bits) - 1)], 1u);
      }
    }
    __syncthreads();
    // the bins from the largest on, two a thread
    const int top = kSelBins - 1 - 2 * tid;
    const uint32_t v0 = hist[top], v1 = hist[top - 1];
    uint2 all;
    const uint32_t before = scan_block(make_uint2(v0 + v1, 0u), part, &all).x;
    if (before < (uint32_t)need && before + v0 + v1 >= (uint32_t)need) {
      const bool first = before + v0 >= (uint32_t)need;
      s_prefix = (prefix << bits) | (uint32_t)(first ? top : top - 1);
      s_need = need - (int)(before + (first ? 0u : v0));
    }
    hist[top] = 0;
    hist[top - 1] = 0;
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
  }
  // prefix is now the threshold key; `need` of the equal ones are kept.  An odd run of slots a
  // thread: the threads of a warp read different banks.
  const int per = ((n + kSelThreads - 1) / kSelThreads) | 1;
  const int i0 = tid * per < n ? tid * per : n, i1 = min(n, i0 + per);
  uint2 mine = make_uint2(0u, 0u);       // larger, equal
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    mine.x += k > prefix;
    mine.y += k == prefix;
  }
  uint2 all;
  uint2 at = scan_block(mine, part, &all);
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = key(i);
    if (k > prefix) out[lo + at.x++ + min(at.y, (uint32_t)need)] = lo + i;
    else if (k == prefix) {
      if (at.y < (uint32_t)need) out[lo + at.x + at.y] = lo + i;
      ++at.y;
    }
  }
}

static cudaError_t launch_select(const SelectArgs& a, int B, cudaStream_t st) {
  // the longest middle that the tally's extent allows
  const long long n = (long long)a.S - a.sinks - a.recent;
  if (n <= kSelKeys) {
    const int smem = (int)(n > 0 ? n : 0) * 4;
    const cudaError_t e =
        cudaFuncSetAttribute(k_cache_select<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
    if (e != cudaSuccess) return e;
    k_cache_select<true><<<dim3(a.Hkv, B), kSelThreads, smem, st>>>(a);
  } else {
    k_cache_select<false><<<dim3(a.Hkv, B), kSelThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Row moves: slot base[b]+i of out_table <- slot idx[b][h][i] of table, i < n[b].
//
// In place (out_table is table) a row may only move towards the front (idx[i] >= base + i).
// A block then owns one slice (64 bytes) of the rows of one head and walks them in order, a chunk at a time.  What chunk j writes lies before everything
// that the chunks after it read, so chunk j + 1 is read before chunk j is written, with
// one barrier between: all of chunk j has been read by then.  Slices do not touch each other.
// Otherwise the pages do not overlap and every chunk has its own block.
// Bound by memory where rows are 256 bytes and many (in place, 8 x 32 heads, 4096 of 8192 rows: 179 us, 6.0 TB/s); a
// gather of one row of 128 bytes in four runs at 70% of that.
struct MoveArgs {
  CacheView c;
  const int* table;
  const int* out_table;
  int MP, MO;
  const int* idx;
  long long ib, ih;        // strides of idx in elements
  const int* n;            // rows to move, per sequence; null: M
  const int* base;         // null: 0
  const float* acc;        // null: none
  long long ab, ah;
  float* acc_out;
  long long ob, oh;
  int S, SO;               // extent of acc and acc_out along the slots
  int M, row_bytes;        // row_bytes: bytes of one cached row of K or V
  int slice_bytes;         // bytes of a row that one block moves
  int piece_blocks;        // blocks that move them; the others move the 4-byte values
  int in_place;
  int clear;               // acc_out behind the last row becomes 0
};

constexpr int kMoveThreads = 256;
constexpr int kMovePieces = 4;           // 16-byte pieces of a row that one thread moves
// Rows of a thread and chunk; in place a thread holds two chunks.
template <bool INPLACE>
constexpr int kMoveRows = INPLACE ? 1 : 2;

// A block's part of a head's rows: one slice of K or V, or the 4-byte values (scales, tally; a row a
// thread).  A slice's row is slice/64 lanes with four pieces each, so that the look-up of a row (its
// index and two pages) is shared by 64 bytes a lane.  Four things follow one another, each a chunk
// behind: the indices, the pages they name, the data, the writing; none waits for what it has just
// asked for.
template <bool INPLACE>
__global__ void __launch_bounds__(kMoveThreads, 4) k_cache_move(MoveArgs a) {
  constexpr int NR = kMoveRows<INPLACE>;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  // blocks: the slices of K and of V chunk by chunk, then the words
  const int slices = a.row_bytes / a.slice_bytes;
  const bool words = (int)blockIdx.x >= a.piece_blocks;
  const int what = words ? 0 : blockIdx.x % (2 * slices);
  const int chunk0 = words ? blockIdx.x - a.piece_blocks : blockIdx.x / (2 * slices);
  const int n = a.n ? __ldg(a.n + b) : a.M;
  const int base = a.base ? __ldg(a.base + b) : 0;
  if (static_cast<unsigned>(n) > static_cast<unsigned>(a.M) || base < 0 || base > INT_MAX - a.M) {
    if (tid == 0) atomicOr(&g_device_error, DEVERR_BOUNDS);
    return;
  }
  const int* idx = a.idx + b * a.ib + h * a.ih;
  const int* table = a.table + (size_t)b * a.MP;
  const int* out_table = a.out_table + (size_t)b * a.MO;
  const int lanes = words ? 1 : a.slice_bytes / (16 * kMovePieces), shift = 31 - __clz(lanes);
  const int pass = kMoveThreads >> shift, rpc = pass * NR;       // rows of a pass, of a chunk
  const int lane = tid & (lanes - 1), row0 = tid >> shift;
  uint8_t* pool = (what < slices ? a.c.k : a.c.v) + (size_t)(what % slices) * a.slice_bytes + 16 * lane;
  const float* acc = a.acc ? a.acc + b * a.ab + h * a.ah : nullptr;
  float* acc_out = a.acc_out ? a.acc_out + b * a.ob + h * a.oh : nullptr;
  const int last = INPLACE ? n : min(n, (chunk0 + 1) * rpc);
  auto ask_idx = [&](int (&s)[NR], int i0) {
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      const int i = i0 + u * pass + row0;
      s[u] = i < last ? __ldg(idx + i) : 0;
    }
  };
  struct Pages {
    int slot[NR];                        // -1: nothing to move
    int src[NR], dst[NR];
  };
  auto ask_pages = [&](Pages& p, const int (&s)[NR], int i0) {
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      const int i = i0 + u * pass + row0, to = base + i;
      p.slot[u] = -1;
      if (i >= last) continue;
      if (!slot_inside(s[u], a.c.page_shift, a.MP) || !slot_inside(to, a.c.page_shift, a.MO) ||
          (INPLACE && s[u] < to)) {
        atomicOr(&g_device_error, DEVERR_BOUNDS);
        continue;
      }
      p.slot[u] = s[u];
      p.src[u] = __ldg(table + (s[u] >> a.c.page_shift));
      p.dst[u] = __ldg(out_table + (to >> a.c.page_shift));
    }
  };
  struct Data {
    uint4 v[NR][kMovePieces];            // words: key scale, value scale, tally in the first
    int to[NR];                          // row written (rows over the pool are 31-bit); -1: none
  };
  auto ask_data = [&](Data& x, const Pages& p, int i0) {
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      x.to[u] = -1;
      if (p.slot[u] < 0) continue;
      if (!page_inside(p.src[u], a.c.pages) || !page_inside(p.dst[u], a.c.pages)) {
        atomicOr(&g_device_error, DEVERR_BOUNDS);
        continue;
      }
      const int to = base + i0 + u * pass + row0;
      const long long src = row_of(p.src[u], a.c.Hkv, h, a.c.page_shift, p.slot[u]);
      x.to[u] = (int)row_of(p.dst[u], a.c.Hkv, h, a.c.page_shift, to);
      if (!words) {
        if (INPLACE && p.slot[u] == to) {
          x.to[u] = -1;                                           // it stays
        } else {
          const uint8_t* from = pool + src * a.row_bytes;
#pragma unroll
          for (int y = 0; y < kMovePieces; ++y)
            x.v[u][y] = *reinterpret_cast<const uint4*>(from + ((16 * y) << shift));
        }
      } else {
        if (a.c.ks) {
          x.v[u][0].x = __float_as_uint(a.c.ks[src]);
          x.v[u][0].y = __float_as_uint(a.c.vs[src]);
        }
        if (acc) {
          const bool in = p.slot[u] < a.S;
          x.v[u][0].z = in ? __float_as_uint(acc[p.slot[u]]) : 0u;
          if (!in || to >= a.SO) atomicOr(&g_device_error, DEVERR_BOUNDS);
        }
      }
    }
  };
  auto write = [&](const Data& x, int i0) {
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      if (x.to[u] < 0) continue;
      if (!words) {
        uint8_t* into = pool + (long long)x.to[u] * a.row_bytes;
#pragma unroll
        for (int y = 0; y < kMovePieces; ++y)
          *reinterpret_cast<uint4*>(into + ((16 * y) << shift)) = x.v[u][y];
      } else {
        if (a.c.ks) {
          a.c.ks[x.to[u]] = __uint_as_float(x.v[u][0].x);
          a.c.vs[x.to[u]] = __uint_as_float(x.v[u][0].y);
        }
        const int to = base + i0 + u * pass + row0;
        if (acc_out && to < a.SO) acc_out[to] = __uint_as_float(x.v[u][0].z);
      }
    }
  };
  // Each word block its share.  In place all of them have been read by the last barrier.
  auto clear_rest = [&]() {
    if (!words || !a.clear || !acc_out) return;
    const int step = INPLACE ? kMoveThreads : ((int)gridDim.x - a.piece_blocks) * kMoveThreads;
    for (long long i = (long long)base + n + (INPLACE ? 0 : chunk0 * kMoveThreads) + tid; i < a.SO; i += step)
      acc_out[i] = 0.f;
  };
  int s[NR];
  Pages p;
  Data x0;
  if (!INPLACE) {
    const int i0 = chunk0 * rpc;
    ask_idx(s, i0);
    ask_pages(p, s, i0);
    ask_data(x0, p, i0);
    write(x0, i0);
    clear_rest();
    return;
  }
  Data x1;
  ask_idx(s, 0);
  ask_pages(p, s, 0);
  ask_idx(s, rpc);
  ask_data(x0, p, 0);
  ask_pages(p, s, rpc);
  ask_idx(s, 2 * rpc);
  // the data of chunk i0 is on its way, with the pages of the one after it and the indices of the next
  for (int i0 = 0; i0 < n; i0 += 2 * rpc) {
    ask_data(x1, p, i0 + rpc);
    ask_pages(p, s, i0 + 2 * rpc);
    ask_idx(s, i0 + 3 * rpc);
    __syncthreads();
    write(x0, i0);
    if (i0 + rpc >= n) break;
    ask_data(x0, p, i0 + 2 * rpc);
    ask_pages(p, s, i0 + 3 * rpc);
    ask_idx(s, i0 + 4 * rpc);
    __syncthreads();
    write(x1, i0 + rpc);
  }
  clear_rest();
}

static cudaError_t launch_move(MoveArgs a, int B, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  // In place a block walks all rows of its slice: whole rows where the heads fill the SMs twice, else
  // slices down to 64 bytes.
  a.slice_bytes = a.row_bytes;
  while (a.in_place && a.slice_bytes > 64 &&
         (int64_t)B * a.c.Hkv * 2 * (a.row_bytes / a.slice_bytes) < 2 * 148)
    a.slice_bytes /= 2;
  const int slices = a.row_bytes / a.slice_bytes;
  const int per = kMoveThreads * (a.in_place ? kMoveRows<true> : kMoveRows<false>);
  const int rpc = per / (a.slice_bytes / (16 * kMovePieces));
  a.piece_blocks = (a.in_place ? 1 : (a.M + rpc - 1) / rpc) * 2 * slices;
  const int word_blocks = a.c.ks || a.acc ? (a.in_place ? 1 : (a.M + per - 1) / per) : 0;
  const dim3 grid((unsigned)(a.piece_blocks + word_blocks), a.c.Hkv, B);
  if (a.in_place) k_cache_move<true><<<grid, kMoveThreads, 0, st>>>(a);
  else k_cache_move<false><<<grid, kMoveThreads, 0, st>>>(a);
  return cudaGetLastError();
}

// ------------------------------------------------------------ validation
static bool pow2(int x) { return x > 0 && (x & (x - 1)) == 0; }

static sage2_status check_cache(const sage2_cache* c, CacheView* out) {
  if (!c) return SAGE2_ERR_INVALID_ARG;
  if (c->pages <= 0 || c->Hkv <= 0 || c->page_size <= 0) return SAGE2_ERR_INVALID_ARG;
  if (c->kv_dtype != SAGE2_F16 && c->kv_dtype != SAGE2_BF16 && c->kv_dtype != SAGE2_E4M3)
    return SAGE2_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return SAGE2_ERR_UNSUPPORTED;
  if (!pow2(c->page_size) || c->page_size < 16 || c->page_size > 128) return SAGE2_ERR_UNSUPPORTED;
  if (c->Hkv > 65535) return SAGE2_ERR_UNSUPPORTED;
  // rows over the pool are 32-bit TMA coordinates
  if ((int64_t)c->pages * c->Hkv > INT32_MAX / c->page_size) return SAGE2_ERR_UNSUPPORTED;
  sage2_status s = check_ptrs(c->k, c->v);
  if (s != SAGE2_OK) return s;
  const bool e4m3 = c->kv_dtype == SAGE2_E4M3;
  if (e4m3) {
    s = check_ptrs(c->k_scale, c->v_scale);
    if (s != SAGE2_OK) return s;
  }
  out->k = static_cast<uint8_t*>(c->k);
  out->v = static_cast<uint8_t*>(c->v);
  out->ks = e4m3 ? c->k_scale : nullptr;
  out->vs = e4m3 ? c->v_scale : nullptr;
  out->pages = c->pages;
  out->Hkv = c->Hkv;
  out->page_shift = __builtin_ctz(c->page_size);
  out->d = c->d;
  out->kv_dtype = c->kv_dtype;
  return SAGE2_OK;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Device integer arrays and fp32 tallies only need their natural alignment.
template <typename... P>
static sage2_status check_words(P... ps) {
  const void* arr[] = {static_cast<const void*>(ps)...};
  for (const void* p : arr)
    if (!p) return SAGE2_ERR_INVALID_ARG;
  for (const void* p : arr)
    if (!aligned4(p)) return SAGE2_ERR_MISALIGNED;
  return SAGE2_OK;
}

// B sequences and a table of MP pages each: sizes that the grids and the int32
// slots can hold.
static sage2_status check_table(const CacheView& c, int B, int MP) {
  if (B <= 0 || MP <= 0) return SAGE2_ERR_INVALID_ARG;
  if (B > 65535) return SAGE2_ERR_UNSUPPORTED;
  if ((int64_t)MP << c.page_shift > INT32_MAX / 2) return SAGE2_ERR_UNSUPPORTED;
  return SAGE2_OK;
}

// Does every head of a tally that is written ({batch, head} strides, S slots a head) have slots of its own?
// Nested either way: what several blocks write at once may not be shared.
static bool heads_apart(const int64_t* st, int B, int H, int S) {
  if (st[0] < 0 || st[1] < 0) return false;
  const __int128 b = st[0], h = st[1];
  if (B == 1 && H == 1) return true;
  if (B == 1) return h >= S;
  if (H == 1) return b >= S;
  return h <= b ? h >= S && b >= h * (H - 1) + S : b >= S && h >= b * (B - 1) + S;
}

// Strides of a [B, H, T, d] tensor (elements; null: contiguous): rows must
// start on 16-byte boundaries.
static sage2_status take_strides(const int64_t* s, int64_t H, int64_t T, int64_t d, long long* out) {
  if (!s) {
    out[0] = H * T * d;
    out[1] = T * d;
    out[2] = d;
    return SAGE2_OK;
  }
  for (int i = 0; i < 3; ++i) {
    if (s[i] < 0) return SAGE2_ERR_INVALID_ARG;
    if (s[i] % 8 != 0) return SAGE2_ERR_MISALIGNED;
    out[i] = s[i];
  }
  return SAGE2_OK;
}

}  // namespace sage2

using namespace sage2;

extern "C" {

sage2_status sage2_cache_append(const void* k, const void* v, int dtype, const int64_t* k_strides,
                                const int64_t* v_strides, const sage2_cache* cache,
                                const int* table, int max_pages, const int* lens, const int* n,
                                int B, int T, sage2_stream_t stream) {
  AppendArgs a{};
  sage2_status s = check_cache(cache, &a.c);
  if (s != SAGE2_OK) return s;
  s = check_table(a.c, B, max_pages);
  if (s != SAGE2_OK) return s;
  if (dtype != SAGE2_F16 && dtype != SAGE2_BF16) return SAGE2_ERR_INVALID_ARG;
  const bool e4m3 = a.c.kv_dtype == SAGE2_E4M3;
  if (!e4m3 && dtype != a.c.kv_dtype) return SAGE2_ERR_INVALID_ARG;
  if (T <= 0) return SAGE2_ERR_INVALID_ARG;
  if (!n && T > (max_pages << a.c.page_shift)) return SAGE2_ERR_INVALID_ARG;   // n: a padded batch
  if ((int64_t)B * a.c.Hkv > INT32_MAX) return SAGE2_ERR_UNSUPPORTED;
  s = check_ptrs(k, v);
  if (s != SAGE2_OK) return s;
  s = check_words(table, lens);
  if (s != SAGE2_OK) return s;
  if (n && !aligned4(n)) return SAGE2_ERR_MISALIGNED;
  const int64_t* strides[2] = {k_strides, v_strides};
  for (int i = 0; i < 2; ++i) {
    long long st[3];
    s = take_strides(strides[i], a.c.Hkv, T, a.c.d, st);
    if (s != SAGE2_OK) return s;
    a.sb[i] = st[0];
    a.sh[i] = st[1];
    a.st[i] = st[2];
  }
  a.x[0] = k;
  a.x[1] = v;
  a.table = table;
  a.lens = lens;
  a.n = n;
  a.B = B;
  a.T = T;
  a.MP = max_pages;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return from_cuda(dtype == SAGE2_F16 ? append_pick<__half>(a, a.c.d, e4m3, st)
                                      : append_pick<__nv_bfloat16>(a, a.c.d, e4m3, st));
}

// One move of rows, the arguments checked but for idx.  padded: of the M indices a count on the device is in use.
static sage2_status move_args(const sage2_cache* cache, const int* table, int max_pages,
                              const int* out_table, int out_max_pages, const float* acc,
                              const int64_t* acc_strides, int S, float* acc_out,
                              const int64_t* acc_out_strides, int SO, int B, int M, bool padded,
                              MoveArgs* a) {
  sage2_status s = check_cache(cache, &a->c);
  if (s != SAGE2_OK) return s;
  s = check_table(a->c, B, max_pages);
  if (s != SAGE2_OK) return s;
  if (M < 0) return SAGE2_ERR_INVALID_ARG;
  s = check_words(table);
  if (s != SAGE2_OK) return s;
  if (!out_table || out_table == table) {
    out_table = table;
    out_max_pages = max_pages;
  }
  s = check_table(a->c, B, out_max_pages);
  if (s != SAGE2_OK) return s;
  if (!padded && M > (out_max_pages << a->c.page_shift)) return SAGE2_ERR_INVALID_ARG;
  s = check_words(out_table);
  if (s != SAGE2_OK) return s;
  if ((acc == nullptr) != (acc_out == nullptr)) return SAGE2_ERR_INVALID_ARG;
  if (acc) {
    s = check_words(acc, acc_out);
    if (s != SAGE2_OK) return s;
    if (S <= 0 || SO <= 0 || !acc_strides || !acc_out_strides) return SAGE2_ERR_INVALID_ARG;
    if (acc_strides[0] < 0 || acc_strides[1] < 0 || !heads_apart(acc_out_strides, B, a->c.Hkv, SO))
      return SAGE2_ERR_INVALID_ARG;
    // onto itself: in place, and laid out alike
    if (acc == acc_out &&
        (out_table != table || (B > 1 && acc_strides[0] != acc_out_strides[0]) ||
         (a->c.Hkv > 1 && acc_strides[1] != acc_out_strides[1])))
      return SAGE2_ERR_INVALID_ARG;
    a->ab = acc_strides[0];
    a->ah = acc_strides[1];
    a->ob = acc_out_strides[0];
    a->oh = acc_out_strides[1];
  }
  a->table = table;
  a->out_table = out_table;
  a->MP = max_pages;
  a->MO = out_max_pages;
  a->acc = acc;
  a->acc_out = acc_out;
  a->S = S;
  a->SO = SO;
  a->M = M;
  a->row_bytes = a->c.d * (a->c.kv_dtype == SAGE2_E4M3 ? 1 : 2);
  a->in_place = out_table == table;
  return SAGE2_OK;
}

sage2_status sage2_cache_compact(const sage2_cache* cache, const int* table, int max_pages,
                                 const int* out_table, int out_max_pages, const int* idx,
                                 const int64_t* idx_strides, const int* n, const int* base,
                                 const float* acc, const int64_t* acc_strides, int S, float* acc_out,
                                 const int64_t* acc_out_strides, int SO, int B, int M,
                                 sage2_stream_t stream) {
  MoveArgs a{};
  sage2_status s = move_args(cache, table, max_pages, out_table, out_max_pages, acc, acc_strides, S,
                             acc_out, acc_out_strides, SO, B, M, n != nullptr, &a);
  if (s != SAGE2_OK) return s;
  if (M == 0) return SAGE2_OK;
  s = check_words(idx);
  if (s != SAGE2_OK) return s;
  if ((n && !aligned4(n)) || (base && !aligned4(base))) return SAGE2_ERR_MISALIGNED;
  if (idx_strides && (idx_strides[0] < 0 || idx_strides[1] < 0)) return SAGE2_ERR_INVALID_ARG;
  a.idx = idx;
  a.ib = idx_strides ? idx_strides[0] : (long long)a.c.Hkv * M;
  a.ih = idx_strides ? idx_strides[1] : M;
  a.n = n;
  a.base = base;
  return from_cuda(launch_move(a, B, reinterpret_cast<cudaStream_t>(stream)));
}

sage2_status sage2_cache_evict(const sage2_cache* cache, const int* table, int max_pages,
                               const int* out_table, int out_max_pages, const int* lens,
                               const float* acc, const int64_t* acc_strides, int S, float* acc_out,
                               const int64_t* acc_out_strides, int SO, int B, int keep, int sinks,
                               int recent, int* idx, int* new_lens, sage2_stream_t stream) {
  if (!acc) return SAGE2_ERR_INVALID_ARG;
  if (keep <= 0 || sinks < 0 || recent < 0 || sinks > keep || recent > keep - sinks)
    return SAGE2_ERR_INVALID_ARG;
  MoveArgs a{};
  sage2_status s = move_args(cache, table, max_pages, out_table, out_max_pages, acc, acc_strides, S,
                             acc_out, acc_out_strides, SO, B, keep, false, &a);
  if (s != SAGE2_OK) return s;
  if (SO < keep) return SAGE2_ERR_INVALID_ARG;
  s = check_words(lens, idx, new_lens);
  if (s != SAGE2_OK) return s;
  if (new_lens == lens) return SAGE2_ERR_INVALID_ARG;   // other blocks still read them
  a.idx = idx;
  a.ib = (long long)a.c.Hkv * keep;
  a.ih = keep;
  a.n = new_lens;
  a.base = nullptr;
  a.clear = 1;             // a token that takes one of these slots starts from 0
  SelectArgs sel{acc, a.ab, a.ah, lens, idx, new_lens, a.c.Hkv, S, keep, sinks, recent};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_select(sel, B, st);
  if (e == cudaSuccess) e = launch_move(a, B, st);
  return from_cuda(e);
}

}  // extern "C"
