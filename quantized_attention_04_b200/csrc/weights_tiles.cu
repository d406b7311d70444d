// Tally of attention weight per cached token on the tensor cores: k_weights_tiles.
//
//   acc[b][h][s] += sum over the rows r that attend slot s of exp2(c_s q_r . K_s - z_r),
// z = lse / ln 2.  S^T = K Q^T: 128 keys are the MMA's rows (TMEM lanes) and up to 256 rows of Q
// its columns, so that a thread owns a key and adds up its own columns: no sum crosses
// lanes, and a slot's sum has a fixed order.  S^T is double-buffered in TMEM; eight warps take the even
// tiles and eight the odd ones, each half of the columns in chunks of 16, and the two that share a key
// meet once a tile.
// Bound, where rows are many, by products and exponentials in turn: both score buffers are full while a group
// reads them (8 x 48 tokens, 32 heads over 8, 32768 e4m3 slots: 73 us of products in three terms, 68 of exponentials,
// 150 to 165 in all); where few, by launch and latency (13 tokens, 24 heads, d = 64, 17776 fp16 slots: 23 us against
// 9 of K's bytes).
//
// e4m3 caches go to the tensor cores as they are (kind::f8f6f4).  The rows of Q, scaled
// by one power of two for all of them, are split into e5m2 terms that add up to them exactly (3
// for bf16, 4 for fp16: each takes 3 bits of the significand; what lies below 2^-31 of
// the largest value is rounded there), and their products accumulate in the same fp32 sums: the
// codes need no widening.  The key scale multiplies the score.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "cache_index.h"
#include "sage2.h"
#include "sage2_internal.h"
#include "sm100_ptx.cuh"

namespace sage2 {

constexpr int kWK = 128;                 // keys of a tile
constexpr int kWR = 256;                 // rows of a unit at most
constexpr int kWExp = 16;                // warps that take exponentials
constexpr int kWThreads = (kWExp + 2) * 32;
constexpr int kWStages = 4;

template <int D, bool E4M3, bool QBF>
struct WeightsCfg {
  static constexpr int kTerms = !E4M3 ? 1 : (QBF ? 3 : 4);
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kLine = kRowBytes < 128 ? kRowBytes : 128;     // swizzle span
  static constexpr int kBlk = kRowBytes / kLine;                      // lines of a row
  static constexpr int kTileBytes = kWK * kRowBytes;
  static constexpr int kTermBytes = kWR * kRowBytes;
};

template <int D, bool E4M3, bool QBF>
struct __align__(1024) WeightsSmem {
  using C = WeightsCfg<D, E4M3, QBF>;
  uint8_t q[C::kTerms][C::kTermBytes];
  uint8_t k[kWStages][C::kTileBytes];
  float z[kWR];              // -lse in log2 units; -inf: the row does not count
  int tok[kWR];              // drafted token of the row
  float red[2][2][kWK];      // sums of the second half of the columns, by tile parity and its turn
  float amax[kWExp];
  uint64_t full[kWStages], empty[kWStages];
  uint64_t q_full;           // the exponential warps
  uint64_t d_full[2], d_empty[2];           // by tile parity
  uint64_t drain;
  uint32_t tmem;
  int abort_flag;
};

// Byte offset of 16-byte chunk `ch` of row `r` in a tile of ROWS rows.
template <typename C, int ROWS>
__device__ __forceinline__ uint32_t line_off(int r, int ch) {
  if (C::kLine == 128) return (ch >> 3) * (ROWS * 128) + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
  return r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
}
__device__ __forceinline__ void bar_exp() { asm volatile("bar.sync 1, %0;" ::"n"(kWExp * 32) : "memory"); }
__device__ __forceinline__ void bar_half(int group) {      // the eight warps of a tile parity
  asm volatile("bar.sync %0, %1;" ::"r"(2 + group), "n"(kWExp * 16) : "memory");
}
__host__ __device__ constexpr uint32_t idesc_e4m3_e5m2(int M, int N) {
  return (1u << 4) | (0u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

template <int D, bool E4M3, bool QBF>
__global__ void __launch_bounds__(kWThreads, 1)
    k_weights_tiles(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ TreeArgs a,
                    const float* __restrict__ lse, float* __restrict__ tally, long long ab, long long ah,
                    int S, int rows_unit) {
  using C = WeightsCfg<D, E4M3, QBF>;
  using Smem = WeightsSmem<D, E4M3, QBF>;
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                      ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = a.G * a.T, cols = (rows_unit + 15) & ~15;
  const int cols0 = ((cols >> 4) + 1) / 2 * 16;      // columns of the first half
  volatile int* abort_flag = &sm.abort_flag;
  if (tid == 0) {
    for (int i = 0; i < kWStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    mbar_init(&sm.q_full, kWExp);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.d_full[i], 1);
      mbar_init(&sm.d_empty[i], kWExp / 2);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWExp + 1) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  const Run run = warp_run(a, kWK, a.c.Hkv, gridDim.x, blockIdx.x, 1);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  // All roles walk alike: the pieces of the run (tiles of one pair), for each its row units, for each
  // its tiles.
  Cursor at;
  if (run.n > 0) at.start(run, kWK);
  int left = run.n, t = 0;               // t: steps so far
  bool ok = true;
  auto piece_tiles = [&]() { return min(left, at.tiles - at.tile); };
  auto next_piece = [&](int cnt) {
    left -= cnt;
    if (left > 0) {
      at.tile = at.tiles - 1;
      at.next(a, a.c.Hkv, kWK);
    }
  };

  if (warp == kWExp) {
    // ------------------------------------------------------------ loader
    while (ok && left > 0) {
      const int cnt = piece_tiles(), L = at.s.len + at.s.n;
      const int prow = min(kWK, 1 << a.c.page_shift);
      for (int u = 0; ok && u < a.RT; ++u)
        for (int k = 0; k < cnt; ++k, ++t) {
          const int key0 = (at.tile + k) * kWK, chunk = key0 + lane * prow, st = t % kWStages;
          const bool in = lane * prow < kWK && chunk < L;
          int page = -1;
          if (in) {
            page = __ldg(a.table + (size_t)at.b * a.MP + (chunk >> a.c.page_shift));
            if (!page_inside(page, a.c.pages)) {
              atomicOr(&g_device_error, DEVERR_BOUNDS);
              page = 0;     // any rows: the tally is not meaningful
            }
          }
          if (t >= kWStages && !tile_wait(&sm.empty[st], (t / kWStages - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const int n = __popc(__ballot_sync(0xffffffffu, in));
          if (lane == 0) mbar_expect_tx(&sm.full[st], n * prow * C::kRowBytes);
          __syncwarp();
          if (in) {
            const int row = (int)row_of(page, a.c.Hkv, at.pair, a.c.page_shift, chunk);
#pragma unroll
            for (int x = 0; x < C::kBlk; ++x)
              tma_load_2d(sm.k[st] + x * kWK * 128 + lane * prow * C::kLine, &tm_k, &sm.full[st], x * 64, row);
          }
        }
      next_piece(cnt);
    }
    if (!ok) {
      // let the copies already issued land before the block exits
      for (int u = t > kWStages ? t - kWStages : 0; u < t; ++u)
        mbar_wait(&sm.full[u % kWStages], (u / kWStages) & 1, nullptr);
    }
  } else if (warp == kWExp + 1) {
    // ------------------------------------------------------------ MMA issuer (values alike in all lanes)
    auto idesc_of = [&](int n) { return E4M3 ? idesc_e4m3_e5m2(kWK, n) : idesc_f16_f32(kWK, n, QBF); };
    const uint64_t dk0 = smem_desc_kmajor(sm.k[0], C::kLine), dq0 = smem_desc_kmajor(sm.q[0], C::kLine);
    const uint32_t hi = uniform((uint32_t)(dk0 >> 32)), k_lo = uniform((uint32_t)dk0), q_lo = uniform((uint32_t)dq0);
    const uint32_t tm = uniform(tmem), id = uniform(idesc_of(cols));
    const uint32_t leader = elect_one();
    int units = 0;
    while (ok && left > 0) {
      const int cnt = piece_tiles();
      for (int u = 0; ok && u < a.RT; ++u, ++units) {
        if (!tile_wait(&sm.q_full, units & 1, abort_flag)) {
          ok = false;
          break;
        }
        for (int k = 0; k < cnt; ++k, ++t) {
          const int st = t % kWStages, p = t & 1;
          if (!tile_wait(&sm.full[st], (t / kWStages) & 1, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t kb = uniform(k_lo + st * (C::kTileBytes >> 4));
          if (t >= 2 && !tile_wait(&sm.d_empty[p], ((t >> 1) - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = uniform(tm + p * 256);
#pragma unroll
            for (int x = 0; x < C::kTerms; ++x)
#pragma unroll
              for (int kk = 0; kk < C::kRowBytes / 32; ++kk) {
                const uint32_t qo = (kk >> 2) * ((kWR * 128) >> 4) + (kk & 3) * 2 + x * (C::kTermBytes >> 4);
                const uint32_t ko = (kk >> 2) * ((kWK * 128) >> 4) + (kk & 3) * 2;
                if (E4M3) mma_f8_ss_if(leader, d, desc_of(kb + ko, hi), desc_of(q_lo + qo, hi), id, x > 0 || kk > 0);
                else mma_f16_ss_if(leader, d, desc_of(kb + ko, hi), desc_of(q_lo + qo, hi), id, kk > 0);
              }
          tc_commit_if(leader, &sm.d_full[p]);
          tc_commit_if(leader, &sm.empty[st]);
        }
      }
      next_piece(cnt);
    }
    tc_commit_if(leader, &sm.drain);
    __syncwarp();
    tile_wait(&sm.drain, 0, nullptr);
  } else {
    // ------------------------------------------------------------ exponentials
    // After a wait that gave up every barrier is still passed, so that no warp is left waiting.
    const int quad = warp & 3, part = (warp >> 2) & 1, group = warp >> 3, key_l = 32 * quad + lane;
    const uint32_t tD = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    const float kL2E = 1.4426950408889634f;
    while (left > 0) {
      const int cnt = piece_tiles(), h = at.pair, L = at.s.len + at.s.n;
      const uint8_t* mask = a.mask ? a.mask + at.b * a.mask_sb : nullptr;
      if (L > S && tid == 0 && h == 0) atomicOr(&g_device_error, DEVERR_BOUNDS);
      for (int u = 0; u < a.RT; ++u) {
        // this group's tiles: every other one; the page of the thread's key two of them ahead, the key
        // scale one
        const int k0 = (t & 1) == group ? 0 : 1;
        auto page_of = [&](int k) {
          const int key = (at.tile + k) * kWK + key_l;
          return E4M3 && k < cnt && key < L ? __ldg(a.table + (size_t)at.b * a.MP + (key >> a.c.page_shift)) : -1;
        };
        auto scale_of = [&](int k, int page) {
          const int key = (at.tile + k) * kWK + key_l;
          return E4M3 && page_inside(page, a.c.pages)
                     ? __ldg(a.c.ks + row_of(page, a.c.Hkv, h, a.c.page_shift, key)) : 0.f;
        };
        auto old_of = [&](int k) {
          const int key = (at.tile + k) * kWK + key_l;
          return part == 0 && k < cnt && key < L && key < S ? tally[at.b * ab + h * ah + key] : 0.f;
        };
        const int page0 = page_of(k0);
        int page = page_of(k0 + 2);
        // ---- the unit's rows: two threads a row.  Rows that do not count become zeros with z = +inf; a row
        // whose lse is NaN gives NaN whatever its Q, which becomes zeros too (an infinity there is not
        // to set the scale of the others).
        const int rl = tid >> 1, half = tid & 1, r = u * rows_unit + rl;
        const int i = r % a.T;
        float z = INFINITY;
        const bool there = rl < rows_unit && r < R && i < at.s.n;
        const bool mine_q = 16 * warp < cols;           // this warp's rows are among the MMA's columns
        if (there) {
          z = __ldg(lse + ((size_t)at.b * a.Hq + h * a.G + r / a.T) * a.T + i) * kL2E;
          if (z == -INFINITY) z = INFINITY;
        }
        uint4 w[D / 16];
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + at.b * a.sb +
                                                          (long long)(h * a.G + (there ? r / a.T : 0)) * a.sh +
                                                          (long long)(there ? i : 0) * a.st) + half * (D / 16);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) w[c] = there ? __ldg(src + c) : make_uint4(0u, 0u, 0u, 0u);
        float ks = scale_of(k0, page0);
        if (!(z < INFINITY)) {
#pragma unroll
          for (int c = 0; c < D / 16; ++c) w[c] = make_uint4(0u, 0u, 0u, 0u);
        }
        float qs = a.sm_scale * kL2E;
        // everyone is done with the last unit's rows: the threads have all read its last tile, and its
        // MMAs are over (d_full has been waited for)
        bar_exp();
        // (after it: with an odd count of tiles the other group has added the unit before to them)
        float next_old = old_of(k0);
        if (!E4M3) {
          if (mine_q) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
              *reinterpret_cast<uint4*>(sm.q[0] + line_off<C, kWR>(rl, half * (D / 16) + c)) = w[c];
          }
        } else {
          float amax = 0.f;
          if (mine_q) {
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
              const uint32_t w4[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const float2 f = halves<QBF>(w4[y]);
                amax = max3f(amax, fabsf(f.x), fabsf(f.y));
              }
            }
          }
#pragma unroll
          for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          if (lane == 0) sm.amax[warp] = amax;
          bar_exp();
          amax = sm.amax[lane & (kWExp - 1)];
#pragma unroll
          for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // an exact power of two that puts the unit's largest value at 2^14
          const int ex = (int)(__float_as_uint(amax) >> 23);
          const int sh = (ex == 0 || ex == 255) ? 0 : max(-113, min(60, 14 + 127 - ex));
          const float up = __uint_as_float((uint32_t)(127 + sh) << 23);
          qs *= __uint_as_float((uint32_t)(127 - sh) << 23);
          // 16 bytes of each term at a time, in packed fp16: the scaled values, what each term leaves of
          // them and the terms themselves are exact there (but for what lies below 2^-24)
          if (mine_q) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t v[8];
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const uint4& ww = w[2 * c + (y >> 2)];
                const float2 f = halves<QBF>((y & 3) == 0 ? ww.x : (y & 3) == 1 ? ww.y : (y & 3) == 2 ? ww.z : ww.w);
                v[y] = pack2<false>(f.x * up, f.y * up);
              }
#pragma unroll
              for (int x = 0; x < C::kTerms; ++x) {
                uint32_t o4[4];
#pragma unroll
                for (int y = 0; y < 8; ++y) {
                  __half2_raw hv;
                  hv.x = static_cast<unsigned short>(v[y]);
                  hv.y = static_cast<unsigned short>(v[y] >> 16);
                  const __nv_fp8x2_storage_t e = __nv_cvt_halfraw2_to_fp8x2(hv, __NV_SATFINITE, __NV_E5M2);
                  if (x + 1 < C::kTerms) {
                    const __half2 rest = __hsub2(__half2(hv), __half2(__nv_cvt_fp8x2_to_halfraw2(e, __NV_E5M2)));
                    v[y] = *reinterpret_cast<const uint32_t*>(&rest);
                  }
                  if (y & 1) o4[y >> 1] |= static_cast<uint32_t>(e) << 16;
                  else o4[y >> 1] = static_cast<uint32_t>(e);
                }
                *reinterpret_cast<uint4*>(sm.q[x] + line_off<C, kWR>(rl, half * (D / 32) + c)) =
                    make_uint4(o4[0], o4[1], o4[2], o4[3]);
              }
            }
          }
        }
        if (half == 0) {
          sm.z[rl] = -z;
          sm.tok[rl] = i;
        }
        fence_proxy_async_smem();
        bar_exp();
        if (lane == 0) mbar_arrive(&sm.q_full);

        const int c0 = part ? cols0 : 0, c1st = part ? cols : cols0;      // this warp's columns
        for (int k = k0; k < cnt; k += 2) {
          const int tt = t + k, key0 = (at.tile + k) * kWK, key = key0 + key_l, p = group;
          const float c1 = E4M3 ? qs * ks : qs;
          ks = scale_of(k + 2, page);
          page = page_of(k + 4);
          const bool edge = key0 + kWK > at.s.len, mine = part == 0 && key < L && key < S;
          float* out = tally + at.b * ab + h * ah + key;
          const float old = next_old;
          next_old = old_of(k + 2);
          ok = ok && tile_wait(&sm.d_full[p], (tt >> 1) & 1, abort_flag);
          tc_fence_after();
          float2 sum = make_float2(0.f, 0.f), sum2 = sum;
          const float2 c2 = make_float2(c1, c1);
          const uint32_t d = tD + p * 256;
          if (!edge && ok) {
            auto add = [&](const uint32_t (&x)[16], int c) {
#pragma unroll
              for (int y = 0; y < 16; y += 4) {
                const float4 zz = *reinterpret_cast<const float4*>(sm.z + c + y);
                float2 e0 = __ffma2_rn(make_float2(__uint_as_float(x[y]), __uint_as_float(x[y + 1])), c2,
                                       make_float2(zz.x, zz.y));
                float2 e1 = __ffma2_rn(make_float2(__uint_as_float(x[y + 2]), __uint_as_float(x[y + 3])), c2,
                                       make_float2(zz.z, zz.w));
                e0.x = ex2(e0.x);
                e0.y = ex2(e0.y);
                e1.x = ex2(e1.x);
                e1.y = ex2(e1.y);
                sum = __fadd2_rn(sum, e0);
                sum2 = __fadd2_rn(sum2, e1);
              }
            };
            uint32_t xa[16], xb[16];
            int c = c0;
            if (c < c1st) tmem_ld16(d + c, xa);
#pragma unroll 1
            while (c < c1st) {
              tmem_ld_wait();
              if (c + 16 < c1st) tmem_ld16(d + c + 16, xb);
              add(xa, c);
              c += 16;
              if (c >= c1st) break;
              tmem_ld_wait();
              if (c + 16 < c1st) tmem_ld16(d + c + 16, xa);
              add(xb, c);
              c += 16;
            }
          } else if (ok) {
#pragma unroll 1
            for (int c = c0; c < c1st; c += 16) {
              // which rows attend this key: 16 bytes of the mask on their way at a time
              uint32_t in = 0;
#pragma unroll
              for (int y = 0; y < 16; ++y)
                in |= (slot_allowed(a, mask, at.s, sm.tok[c + y], key) ? 1u : 0u) << y;
              if (key >= L) in = 0;
              uint32_t x[16];
              tmem_ld16(d + c, x);
              tmem_ld_wait();
#pragma unroll
              for (int y = 0; y < 16; ++y) {
                const float zz = sm.z[c + y], e = ex2(fmaf(__uint_as_float(x[y]), c1, zz));
                if (((in >> y) & 1u) && zz != -INFINITY) sum.x += e;
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          mbar_arrive_lane0(&sm.d_empty[p], lane);
          const float half_sum = (sum.x + sum.y) + (sum2.x + sum2.y);
          const int turn = (tt >> 1) & 1;
          if (part == 1) sm.red[p][turn][key_l] = half_sum;
          bar_half(group);
          if (mine) *out = old + (half_sum + sm.red[p][turn][key_l]);
        }
        t += cnt;
      }
      next_piece(cnt);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWExp + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool E4M3, bool QBF>
static cudaError_t launch_weights_tiles(TreeArgs a, const float* lse, float* acc, long long ab, long long ah,
                                        int S, int dev, cudaStream_t st) {
  using C = WeightsCfg<D, E4M3, QBF>;
  const int R = a.G * a.T;
  a.RT = (R + kWR - 1) / kWR;
  const int unit = (R + a.RT - 1) / a.RT;
  CUtensorMap tk{};
  const uint64_t rows = (uint64_t)a.c.pages * a.c.Hkv << a.c.page_shift;
  const int eb = E4M3 ? 1 : 2;
  const uint64_t dims[2] = {(uint64_t)D, rows};
  const uint64_t strides[1] = {(uint64_t)D * eb};
  const uint32_t box[2] = {(uint32_t)(C::kLine / eb), min(1u << a.c.page_shift, (unsigned)kWK)};
  cudaError_t e = make_tmap(&tk, a.c.k, 2, dims, strides, box, eb, C::kLine);
  if (e != cudaSuccess) return e;
  auto kern = k_weights_tiles<D, E4M3, QBF>;
  const int smem = sizeof(WeightsSmem<D, E4M3, QBF>) + 1024;
  static_assert(sizeof(WeightsSmem<D, E4M3, QBF>) + 1024 <= 232448, "shared memory of a block");
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<sm_count(dev), kWThreads, smem, st>>>(tk, a, lse, acc, ab, ah, S, unit);
  return cudaGetLastError();
}

}  // namespace sage2
