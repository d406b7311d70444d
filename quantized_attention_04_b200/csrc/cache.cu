// Paged key/value cache: writing new tokens (sage2_cache_append), choosing the
// tokens to keep by accumulated attention weight and moving rows
// (sage2_cache_evict, sage2_cache_compact).
//
// Slot s of sequence b is row s % page of page table[b][s / page]; a page holds
// `page` rows of d values for each head, head-major, so a head's rows of one
// page are contiguous.  Everything here is bound by memory or by latency.
//
// Device-side integers (table, lens, n, idx) are checked where they are used:
// one that points outside the pools or the table sets DEVERR_BOUNDS and the
// row it names is skipped.
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

// ---------------------------------------------------------------------------
// Append.  D/8 lanes own one row of K or V (16 bytes each); a warp holds 2 or 4
// rows.  e4m3: scale = amax/448, code = e4m3(x * (448/amax)), all fp32 RN, the
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

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(256) k_cache_append(AppendArgs a) {
  constexpr int LPR = D / 8;            // lanes of a row
  constexpr int RPB = 256 / LPR;        // rows of a block
  const int kv = blockIdx.y;
  const long long row = (long long)blockIdx.x * RPB + threadIdx.x / LPR;
  const int lane = threadIdx.x % LPR;
  const long long rows = (long long)a.B * a.c.Hkv * a.T;
  if (row >= rows) return;              // whole rows, and the shuffles stay inside a row
  const int t = (int)(row % a.T);
  const long long bh = row / a.T;
  const int h = (int)(bh % a.c.Hkv), b = (int)(bh / a.c.Hkv);
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(
                            static_cast<const T*>(a.x[kv]) + b * a.sb[kv] + h * a.sh[kv] +
                            (long long)t * a.st[kv]) + lane);
  const int len = __ldg(a.lens + b);
  int n = a.T;
  if (a.n) {
    n = __ldg(a.n + b);
    if (static_cast<unsigned>(n) > static_cast<unsigned>(a.T)) {
      atomicOr(&g_device_error, DEVERR_BOUNDS);
      return;
    }
  }
  if (t >= n) return;
  if (len < 0 || len > INT_MAX - a.T) {
    atomicOr(&g_device_error, DEVERR_BOUNDS);
    return;
  }
  const long long dst = cache_row(a.c, a.table, a.MP, b, h, len + t);
  if (dst < 0) return;
  uint8_t* pool = kv ? a.c.v : a.c.k;
  if (!E4M3) {
    reinterpret_cast<uint4*>(pool + dst * D * 2)[lane] = u;
  } else {
    float x[8];
    unpack8<T>(u, x);
    float amax = 0.f;
    bool fin = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      amax = fmaxf(amax, fabsf(x[i]));
      fin = fin && fabsf(x[i]) < __int_as_float(0x7f800000);
    }
    // the lanes of this row, which are all here: whole rows leave above
    const unsigned act = (LPR == 32 ? 0xffffffffu : ((1u << LPR) - 1u)) << (threadIdx.x % 32 / LPR * LPR);
    float bad = fin ? 0.f : 1.f;
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) {
      amax = fmaxf(amax, __shfl_xor_sync(act, amax, o));
      bad = fmaxf(bad, __shfl_xor_sync(act, bad, o));
    }
    // below 2^-100 the inverse would pass fp32's range: such a row is zero
    const bool nz = amax >= 7.8886e-31f;
    const float inv = nz ? __fdiv_rn(448.f, amax) : 0.f;
    uint32_t w[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      w[g] = 0;
#pragma unroll
      for (int i = 0; i < 4; i += 2)
        w[g] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                    make_float2(__fmul_rn(x[4 * g + i], inv), __fmul_rn(x[4 * g + i + 1], inv)),
                    __NV_SATFINITE, __NV_E4M3))
                << (8 * i);
    }
    reinterpret_cast<uint2*>(pool + dst * D)[lane] = make_uint2(w[0], w[1]);
    if (lane == 0)
      (kv ? a.c.vs : a.c.ks)[dst] = bad > 0.f ? __int_as_float(0x7fffffff)
                                              : (nz ? __fdiv_rn(amax, 448.f) : 0.f);
  }
}

template <typename T, int D, bool E>
static cudaError_t append_go(const AppendArgs& a, cudaStream_t st) {
  const long long rows = (long long)a.B * a.c.Hkv * a.T;
  const long long blocks = (rows + 256 / (D / 8) - 1) / (256 / (D / 8));
  k_cache_append<T, D, E><<<dim3((unsigned)blocks, 2), 256, 0, st>>>(a);
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
// mapped to integers of the same order (NaN lowest, -0 like +0), the
// (keep - sinks - recent)-th largest is found by four 8-bit radix passes, and one
// pass in slot order writes the chosen slots ascending, the equal ones from the
// lowest slot on.
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

__global__ void __launch_bounds__(kSelThreads) k_cache_select(SelectArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int wsum[2][kSelThreads / 32];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
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
  const float* acc = a.acc + b * a.sb + h * a.sh;
  const int lo = a.sinks, hi = len - a.recent;     // the middle: [lo, hi), longer than `want`
  const int want = a.keep - a.sinks - a.recent;
  for (int i = tid; i < lo; i += kSelThreads) out[i] = i;
  for (int i = tid; i < a.recent; i += kSelThreads) out[lo + want + i] = hi + i;
  if (want == 0) return;
  uint32_t prefix = 0;
  int need = want;                                  // still to take among those with the prefix
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int s = lo + tid; s < hi; s += kSelThreads) {
      const uint32_t key = tally_key(__ldg(acc + s));
      if (pass == 0 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1u);
    }
    __syncthreads();
    if (tid < 32) {
      // lane L sums bins 255-8L .. 248-8L; the largest bins come first
      uint32_t v[8], sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = hist[255 - 8 * lane - i];
        sum += v[i];
      }
      uint32_t incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      uint32_t before = incl - sum;
      if (before < (uint32_t)need && incl >= (uint32_t)need) {
        int i = 0;
        while (before + v[i] < (uint32_t)need) before += v[i++];
        s_prefix = (prefix << 8) | (255 - 8 * lane - i);
        s_need = need - (int)before;
      }
    }
    __syncthreads();
    prefix = s_prefix;
    need = s_need;
    __syncthreads();
  }
  // prefix is now the threshold key; `need` of the equal ones are kept
  int taken = 0, ties = 0;
  for (int s0 = lo; s0 < hi; s0 += kSelThreads) {
    const int s = s0 + tid;
    const uint32_t key = s < hi ? tally_key(__ldg(acc + s)) : 0u;
    const bool gt = s < hi && key > prefix, eq = s < hi && key == prefix;
    const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      wsum[0][warp] = __popc(bg);
      wsum[1][warp] = __popc(be);
    }
    __syncthreads();
    int g0 = 0, e0 = 0, gall = 0, eall = 0;
    for (int w = 0; w < kSelThreads / 32; ++w) {
      const int cg = wsum[0][w], ce = wsum[1][w];
      if (w < warp) {
        g0 += cg;
        e0 += ce;
      }
      gall += cg;
      eall += ce;
    }
    const unsigned below = (1u << lane) - 1u;
    const int eqs = ties + e0 + __popc(be & below);        // equal ones before this slot
    const int gts = taken + g0 + __popc(bg & below);       // larger ones before this slot
    if (gt || (eq && eqs < need)) out[lo + gts + min(eqs, need)] = s;
    taken += gall;
    ties += eall;
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Row moves: slot base[b]+i of out_table <- slot idx[b][h][i] of table, i < n[b].
//
// In place (out_table is table) a row may only move towards the front
// (idx[i] >= base + i).  A block then owns one slice of the rows' bytes and walks
// all its rows in order, a chunk at a time: a chunk is read whole before any of
// it is written, and what a chunk writes lies before everything that the later
// chunks read.  Slices do not touch each other, so they run side by side.
// Otherwise the pages do not overlap and every chunk has its own block.
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
  int in_place;
};

constexpr int kMoveThreads = 256;
constexpr int kMovePer = 4;              // 16-byte pieces of a thread and chunk

__global__ void __launch_bounds__(kMoveThreads) k_cache_move(MoveArgs a) {
  const int slices = a.row_bytes / a.slice_bytes;
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  int what = blockIdx.x % (2 * slices + 1);      // K slices, V slices, the 4-byte values
  const int chunk0 = blockIdx.x / (2 * slices + 1);
  int n = a.n ? __ldg(a.n + b) : a.M;
  const int base = a.base ? __ldg(a.base + b) : 0;
  if (static_cast<unsigned>(n) > static_cast<unsigned>(a.M) || base < 0 || base > INT_MAX - a.M) {
    if (tid == 0) atomicOr(&g_device_error, DEVERR_BOUNDS);
    return;
  }
  const int* idx = a.idx + b * a.ib + h * a.ih;
  if (what < 2 * slices) {
    uint8_t* pool = what < slices ? a.c.k : a.c.v;
    const int off = (what % slices) * a.slice_bytes;
    const int ppr = a.slice_bytes / 16;              // pieces of a row
    const int rpc = kMoveThreads * kMovePer / ppr;   // rows of a chunk
    const int step = a.in_place ? rpc : rpc * (gridDim.x / (2 * slices + 1));
    for (int i0 = chunk0 * rpc; i0 < n; i0 += step) {
      uint4 v[kMovePer];
      long long dst[kMovePer];
#pragma unroll
      for (int u = 0; u < kMovePer; ++u) {
        const int p = u * kMoveThreads + tid;
        const int i = i0 + p / ppr;
        dst[u] = -1;
        if (i < n) {
          const int s = __ldg(idx + i);
          if (a.in_place && s < base + i) {
            atomicOr(&g_device_error, DEVERR_BOUNDS);
          } else if (!(a.in_place && s == base + i)) {
            const long long src = cache_row(a.c, a.table, a.MP, b, h, s);
            const long long to = cache_row(a.c, a.out_table, a.MO, b, h, base + i);
            if (src >= 0 && to >= 0) {
              dst[u] = to * a.row_bytes + off + 16 * (p % ppr);
              v[u] = *reinterpret_cast<const uint4*>(pool + src * a.row_bytes + off + 16 * (p % ppr));
            }
          }
        }
      }
      if (a.in_place) __syncthreads();
#pragma unroll
      for (int u = 0; u < kMovePer; ++u)
        if (dst[u] >= 0) *reinterpret_cast<uint4*>(pool + dst[u]) = v[u];
    }
    return;
  }
  // the scales and the tally: one block walks all rows
  if (chunk0 != 0) return;
  const float* acc = a.acc ? a.acc + b * a.ab + h * a.ah : nullptr;
  float* acc_out = a.acc_out ? a.acc_out + b * a.ob + h * a.oh : nullptr;
  for (int i0 = 0; i0 < n; i0 += kMoveThreads) {
    const int i = i0 + tid;
    long long to = -1;
    int s = -1;
    float ks = 0.f, vs = 0.f, t = 0.f;
    if (i < n) {
      s = __ldg(idx + i);
      if (s < 0 || (a.in_place && s < base + i)) {
        atomicOr(&g_device_error, DEVERR_BOUNDS);
        s = -1;
      } else {
        if (a.c.ks) {
          const long long src = cache_row(a.c, a.table, a.MP, b, h, s);
          to = cache_row(a.c, a.out_table, a.MO, b, h, base + i);
          if (src < 0) to = -1;
          if (to >= 0) {
            ks = a.c.ks[src];
            vs = a.c.vs[src];
          }
        }
        if (acc && s < a.S) t = acc[s];
      }
    }
    __syncthreads();
    if (to >= 0) {
      a.c.ks[to] = ks;
      a.c.vs[to] = vs;
    }
    if (acc_out && s >= 0 && base + i < a.SO) acc_out[base + i] = t;
    __syncthreads();
  }
}

static cudaError_t launch_move(MoveArgs a, int B, cudaStream_t st) {
  if (a.M == 0) return cudaSuccess;
  a.slice_bytes = a.in_place ? (a.row_bytes >= 64 ? 64 : a.row_bytes) : a.row_bytes;
  const int slices = a.row_bytes / a.slice_bytes;
  const int rpc = kMoveThreads * kMovePer / (a.slice_bytes / 16);
  const int chunks = a.in_place ? 1 : (a.M + rpc - 1) / rpc;
  k_cache_move<<<dim3((unsigned)(chunks * (2 * slices + 1)), a.c.Hkv, B), kMoveThreads, 0, st>>>(a);
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
  if (T > (max_pages << a.c.page_shift)) return SAGE2_ERR_INVALID_ARG;
  if ((int64_t)B * a.c.Hkv * T > (int64_t)INT32_MAX * 8) return SAGE2_ERR_UNSUPPORTED;
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

// One move of rows, the arguments checked but for idx.
static sage2_status move_args(const sage2_cache* cache, const int* table, int max_pages,
                              const int* out_table, int out_max_pages, const float* acc,
                              const int64_t* acc_strides, int S, float* acc_out,
                              const int64_t* acc_out_strides, int SO, int B, int M, MoveArgs* a) {
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
  if (M > (out_max_pages << a->c.page_shift)) return SAGE2_ERR_INVALID_ARG;
  s = check_words(out_table);
  if (s != SAGE2_OK) return s;
  if ((acc == nullptr) != (acc_out == nullptr)) return SAGE2_ERR_INVALID_ARG;
  if (acc) {
    s = check_words(acc, acc_out);
    if (s != SAGE2_OK) return s;
    if (S <= 0 || SO <= 0 || !acc_strides || !acc_out_strides) return SAGE2_ERR_INVALID_ARG;
    if (acc_strides[0] < 0 || acc_strides[1] < 0 || acc_out_strides[0] < 0 || acc_out_strides[1] < 0)
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
                             acc_out, acc_out_strides, SO, B, M, &a);
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
                             acc_out, acc_out_strides, SO, B, keep, &a);
  if (s != SAGE2_OK) return s;
  if (SO < keep) return SAGE2_ERR_INVALID_ARG;
  s = check_words(lens, idx, new_lens);
  if (s != SAGE2_OK) return s;
  a.idx = idx;
  a.ib = (long long)a.c.Hkv * keep;
  a.ih = keep;
  a.n = new_lens;
  a.base = nullptr;
  SelectArgs sel{acc, a.ab, a.ah, lens, idx, new_lens, a.c.Hkv, S, keep, sinks, recent};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  k_cache_select<<<dim3(a.c.Hkv, B), kSelThreads, 0, st>>>(sel);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_move(a, B, st);
  return from_cuda(e);
}

}  // extern "C"
