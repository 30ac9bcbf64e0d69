// Matrix product with its dequantisation, bias, activation and residual in the
// epilogue: Y = act((X W^T) * sx sw + b) + R, bf16 or e4m3 operands, f32
// accumulation in tensor memory, nothing of the product written but Y.
//
// Both operands are K-major and move as 128-byte-wide swizzled boxes (64 bf16 or
// 128 e4m3 values), and one tcgen05.mma reads 32 bytes of every operand row
// whatever the type, so one kernel text serves both types; e4m3 does twice the
// products per byte moved.
//
// Two kernels:
//   k_linear_split  few tokens. Bound by streaming W, so the 128 rows of the MMA's
//                   M are output features and the tokens are its N (16..256): no
//                   accumulator row is padding, and a stage is 16 KB of W and 128
//                   bytes a token of X, which leaves eight and more stages (about
//                   190 KB) in flight per SM. Too few feature tiles to fill the
//                   SMs split K over a cluster; the f32 partials are summed through
//                   distributed shared memory in rank order, so results repeat.
//   k_linear_pair   many tokens. Bound by the tensor cores: persistent SM pairs on
//                   256 x 256 tiles (cta_group::2), two accumulators in TMEM, so
//                   the epilogue of a tile runs under the products of the next.
// Warp roles in both: warp 0 loads (TMA), warp 1 issues the MMAs, warps 2-5 are
// the epilogue. Every wait is bounded, as in the grouped GEMM.
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "op_util.h"
#include "sm100_ptx.cuh"

namespace tpgqa {
namespace {

using namespace op;

constexpr int kThreads = 192;
constexpr int kMaxParts = 16;  // weight shards (column) or K slices (row)
constexpr int kSmemLimit = 227 * 1024;
constexpr int kWTile = 128 * 128;  // bytes of one 128-row, 128-byte-wide box

struct LinearParams {
  CUtensorMap x[kMaxParts];  // one per K slice
  CUtensorMap w[kMaxParts];  // one per K slice, or one per weight shard
  int k_tiles[kMaxParts];    // 128-byte-wide k-tiles of each slice
  int n[kMaxParts];          // output features of each shard
  int n_tile0[kMaxParts];    // its first feature tile
  long long col0[kMaxParts];  // its first output column
  int n_slices, n_shards, kt_total, n_tiles, rows, m_tiles;
  int act, y_f32, res_f32, bias_f32;
  const float *x_scale, *w_scale;  // null: no scales
  const void *bias, *res;          // null: none
  void *y;
  long long y_ld, res_ld;
  int tok_tile, stages, split, early_w;
  int *status;
  long long wait_ns;
};

__device__ __forceinline__ void record(int *status, int code) { atomicCAS(status, 0, code); }

// Shard of a feature tile (shards are laid out in tile order).
__device__ __forceinline__ int shard_of(const LinearParams &p, int nt) {
  int s = 0;
  while (s + 1 < p.n_shards && nt >= p.n_tile0[s + 1]) ++s;
  return s;
}

// The activations by their formulas, in f32: relu, x Phi(x) with the error
// function, x / (1 + e^-x) (at x < -88 the quotient is -0, its limit).
template <int N>
__device__ __forceinline__ void activate(float (&f)[N], int act) {
  if (act == TP_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = f[i] < 0.0f ? 0.0f : f[i];  // keeps NaN
  } else if (act == TP_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = 0.5f * f[i] * (1.0f + erff(f[i] * 0.70710678118654752f));
  } else if (act == TP_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = __fdividef(f[i], 1.0f + __expf(-f[i]));
  }
}

// Four neighbouring features of one token: acc -> y. col: output column (bias, scales, y, residual).
__device__ __forceinline__ void finish4(const LinearParams &p, long long tok, long long col, int left, float (&f)[4]) {
  if (p.w_scale) {
    const float sx = __ldg(p.x_scale + tok);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) f[i] *= sx * __ldg(p.w_scale + col + i);
  }
  if (p.bias) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left)
        f[i] += p.bias_f32 ? __ldg(static_cast<const float *>(p.bias) + col + i)
                           : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.bias)[col + i]);
  }
  activate(f, p.act);
  if (p.res) {
    const long long at = tok * p.res_ld + col;
    if (p.res_f32) {
      const float *r = static_cast<const float *>(p.res) + at;
      if (left >= 4) {
        const float4 v = *reinterpret_cast<const float4 *>(r);
        f[0] += v.x; f[1] += v.y; f[2] += v.z; f[3] += v.w;
      } else {
        for (int i = 0; i < left; ++i) f[i] += r[i];
      }
    } else {
      const __nv_bfloat16 *r = static_cast<const __nv_bfloat16 *>(p.res) + at;
      if (left >= 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(r);
        f[0] += bf16_lo(v.x); f[1] += bf16_hi(v.x); f[2] += bf16_lo(v.y); f[3] += bf16_hi(v.y);
      } else {
        for (int i = 0; i < left; ++i) f[i] += __bfloat162float(r[i]);
      }
    }
  }
  const long long at = tok * p.y_ld + col;
  if (p.y_f32) {
    float *y = static_cast<float *>(p.y) + at;
    if (left >= 4) *reinterpret_cast<float4 *>(y) = make_float4(f[0], f[1], f[2], f[3]);
    else
      for (int i = 0; i < left; ++i) y[i] = f[i];
  } else {
    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(p.y) + at;
    if (left >= 4) *reinterpret_cast<uint2 *>(y) = make_uint2(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]));
    else
      for (int i = 0; i < left; ++i) y[i] = __float2bfloat16_rn(f[i]);
  }
}

// ---------------------------------------------------------------------------
// Few tokens: features on the MMA's M, tokens on its N, K split over a cluster.
// ---------------------------------------------------------------------------
template <bool F8>
__global__ void __launch_bounds__(kThreads, 1) k_linear_split(const __grid_constant__ LinearParams p) {
  constexpr int kElems = F8 ? 128 : 64;  // values of a 128-byte box row
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int S = p.stages, NT = p.tok_tile;
  const uint32_t stage_bytes = kWTile + static_cast<uint32_t>(NT) * 128u;
  const uint32_t sbase = ptx::smem_addr(smem);
  auto w_slot = [&](int st) { return sbase + static_cast<uint32_t>(st) * stage_bytes; };
  auto x_slot = [&](int st) { return w_slot(st) + kWTile; };
  uint8_t *bar_area = smem + static_cast<uint32_t>(S) * stage_bytes;
  const uint32_t bar0 = ptx::smem_addr(bar_area);
  auto full_bar = [&](int i) { return bar0 + 8u * i; };
  auto empty_bar = [&](int i) { return bar0 + 8u * (S + i); };
  const uint32_t done_bar = bar0 + 8u * (2 * S);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bar_area + 8 * (2 * S + 1));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bar_area + 8 * (2 * S + 1) + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = p.split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int tile = blockIdx.x / p.split;
  const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;  // token tiles of one feature tile are neighbours
  const int shard = shard_of(p, nt);
  const int feat0 = (nt - p.n_tile0[shard]) * 128;  // within the shard
  const int kb0 = static_cast<int>(static_cast<long long>(p.kt_total) * part / p.split);
  const int kb1 = static_cast<int>(static_cast<long long>(p.kt_total) * (part + 1) / p.split);
  uint32_t tmem_cols = 32;
  while (tmem_cols < static_cast<uint32_t>(NT)) tmem_cols *= 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(full_bar(i), 1);
      ptx::mbar_init(empty_bar(i), 1);
    }
    ptx::mbar_init(done_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t *>(tmem_slot)), tmem_cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // k-tile kb of the whole K range -> (slice, k-tile in it)
    auto seek = [&](int kb, int &sl, int &kt) {
      sl = 0;
      kt = kb;
      while (kt >= p.k_tiles[sl]) kt -= p.k_tiles[sl++];
    };
    auto load_w = [&](int st, int sl, int kt) {
      ptx::tma_load_2d(w_slot(st), &p.w[p.n_shards > 1 ? shard : sl], kt * kElems, feat0, full_bar(st));
    };
    // W does not come from the previous kernel: its first stages start before
    // the grid-dependency wait, each barrier already expecting the X bytes.
    int pre = 0;
    if (p.early_w) {
      int sl, kt;
      seek(kb0, sl, kt);
      for (; pre < S && kb0 + pre < kb1; ++pre) {
        ptx::mbar_arrive_expect_tx(full_bar(pre), stage_bytes);
        load_w(pre, sl, kt);
        if (++kt == p.k_tiles[sl]) {
          kt = 0;
          ++sl;
        }
      }
    }
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
    int sl, kt;
    seek(kb0, sl, kt);
    for (int i = 0; kb0 + i < kb1; ++i) {
      const int st = i % S;
      if (i >= pre) {
        if (*abort_flag) break;
        if (!ptx::mbar_wait(empty_bar(st), ((i / S) & 1) ^ 1, p.wait_ns)) {
          record(p.status, kDevTimeoutProducer);
          *abort_flag = 1;
          break;
        }
        ptx::mbar_arrive_expect_tx(full_bar(st), stage_bytes);
        load_w(st, sl, kt);
      }
      ptx::tma_load_2d(x_slot(st), &p.x[sl], kt * kElems, mt * NT, full_bar(st));
      if (++kt == p.k_tiles[sl]) {
        kt = 0;
        ++sl;
      }
    }
  } else {
    ptx::griddep_wait();
    ptx::griddep_launch_dependents();
  }
  if (warp == 1 && lane == 0) {
    const uint32_t idesc = F8 ? ptx::idesc_e4m3_f32(128, NT) : ptx::idesc_bf16_f32(128, NT);
    for (int i = 0; kb0 + i < kb1; ++i) {
      const int st = i % S;
      if (*abort_flag) break;
      if (!ptx::mbar_wait(full_bar(st), (i / S) & 1, p.wait_ns)) {
        record(p.status, kDevTimeoutMma);
        *abort_flag = 1;
        break;
      }
      ptx::tc_fence_after();
      const uint64_t wd = ptx::smem_desc_sw128(w_slot(st)), xd = ptx::smem_desc_sw128(x_slot(st));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (F8) ptx::mma_f8(tmem, wd + 2 * k, xd + 2 * k, idesc, (i | k) != 0 ? 1u : 0u);
        else ptx::mma_bf16(tmem, wd + 2 * k, xd + 2 * k, idesc, (i | k) != 0 ? 1u : 0u);
      }
      ptx::mma_commit(empty_bar(st));
    }
    ptx::mma_commit(done_bar);
  }
  __syncwarp();
  // Every warp waits for the last product; the stage buffers are free from then on.
  const bool ready = __all_sync(0xffffffffu, ptx::mbar_wait(done_bar, 0, p.wait_ns));
  if (!ready && lane == 0) {
    record(p.status, kDevTimeoutEpilogue);
    *abort_flag = 1;
  }
  ptx::tc_fence_after();
  float *red = reinterpret_cast<float *>(smem);  // [token][128 features] f32
  if (warp >= 2 && ready) {
    const int q = warp & 3;
    for (int c = 0; c < NT; c += 16) {
      uint32_t v[16];
      ptx::tmem_ld_16cols(tmem + c + (static_cast<uint32_t>(q * 32) << 16), v);
      ptx::tmem_ld_wait();
      ptx::tmem_regs_ready(v);
#pragma unroll
      for (int j = 0; j < 16; ++j) red[(c + j) * 128 + q * 32 + lane] = __uint_as_float(v[j]);
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, tmem_cols);
  }
  if (*abort_flag && threadIdx.x == 0) {
    // copies already in flight land before the shared memory goes away
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  if (p.split > 1) ptx::cluster_sync();
  else __syncthreads();
  // The cluster's CTAs share the tile's tokens; a warp finishes one token at a
  // time, four features a lane, the partials added in cluster order.
  if (*abort_flag == 0) {
    const int t1 = NT * (part + 1) / p.split;
    const int left = p.n[shard] - feat0 - lane * 4;
    const uint32_t red_addr = ptx::smem_addr(red);
    for (int t = NT * part / p.split + warp; t < t1; t += kThreads / 32) {
      const long long tok = static_cast<long long>(mt) * NT + t;
      if (tok >= p.rows) break;
      float f[4];
      if (p.split == 1) {
        const float4 v = *reinterpret_cast<const float4 *>(red + t * 128 + lane * 4);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
      } else {
        float4 v[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < p.split)
            v[r] = ptx::ld_shared_cluster_f4(ptx::mapa_shared(red_addr + static_cast<uint32_t>(t * 128 + lane * 4) * 4u, r));
        f[0] = v[0].x; f[1] = v[0].y; f[2] = v[0].z; f[3] = v[0].w;
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < p.split) {
            f[0] += v[r].x; f[1] += v[r].y; f[2] += v[r].z; f[3] += v[r].w;
          }
      }
      if (left > 0) finish4(p, tok, p.col0[shard] + feat0 + lane * 4, left, f);
    }
  }
  __syncwarp();
  if (p.split > 1) ptx::cluster_sync();  // peers have read this CTA's partials
}

// ---------------------------------------------------------------------------
// Many tokens: persistent SM pairs, 256 tokens x 256 features per tile.
// ---------------------------------------------------------------------------
constexpr int kSub = 2;                                   // k-tiles per stage
constexpr int kPairStage = kSub * 2 * kWTile;              // 64 KB per CTA
constexpr int kPairStages = 3;
constexpr int kPairSmem = 1024 + kPairStages * kPairStage + 256;
constexpr int kGroup = 16;  // token tiles walked for one feature tile before the next (keeps both in L2)

// Tile -> (token tile, feature tile): groups of kGroup token tiles, token tile fastest.
__device__ __forceinline__ void pair_tile(const LinearParams &p, int tile, int &mt, int &nt) {
  const int per_group = kGroup * p.n_tiles;
  const int grp = tile / per_group, r = tile - grp * per_group;
  const int rows = min(kGroup, p.m_tiles - grp * kGroup);
  mt = grp * kGroup + r % rows;
  nt = r / rows;
}

template <bool F8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_linear_pair(const __grid_constant__ LinearParams p) {
  constexpr int kElems = F8 ? 128 : 64;
  constexpr int S = kPairStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sX = ptx::smem_addr(smem), sW = sX + S * kSub * kWTile;
  uint8_t *bar_area = smem + S * kPairStage;
  const uint32_t bar0 = ptx::smem_addr(bar_area);
  auto full_bar = [&](int i) { return bar0 + 8u * i; };
  auto empty_bar = [&](int i) { return bar0 + 8u * (S + i); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 4);
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bar_area + 8 * (2 * S + 5));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bar_area + 8 * (2 * S + 5) + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int tiles = p.m_tiles * p.n_tiles;
  auto slice_stages = [&](int sl) { return (p.k_tiles[sl] + kSub - 1) / kSub; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(full_bar(i), 1);
      ptx::mbar_init(empty_bar(i), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(tfull_bar(a), 1);
      ptx::mbar_init(tempty_bar(a), 8);  // 4 epilogue warps in each CTA
    }
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_addr(const_cast<uint32_t *>(tmem_slot)), 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      int kb = 0;
      bool go = true;
      for (int tile = pair; go && tile < tiles; tile += npairs) {
        int mt, nt;
        pair_tile(p, tile, mt, nt);
        const int shard = shard_of(p, nt);
        const int x_row = mt * 256 + static_cast<int>(rank) * 128;
        const int w_row = (nt - p.n_tile0[shard]) * 256 + static_cast<int>(rank) * 128;
        for (int sl = 0; go && sl < p.n_slices; ++sl) {
          const CUtensorMap *wm = &p.w[p.n_shards > 1 ? shard : sl];
          for (int ks = 0; ks < slice_stages(sl); ++ks, ++kb) {
            const int st = kb % S;
            if (*abort_flag || !ptx::mbar_wait(empty_bar(st), ((kb / S) & 1) ^ 1, p.wait_ns)) {
              if (!*abort_flag) record(p.status, kDevTimeoutProducer);
              *abort_flag = 1;
              go = false;
              break;
            }
            const uint32_t lead_full = ptx::mapa_shared(full_bar(st), 0);
            if (leader) ptx::mbar_arrive_expect_tx(full_bar(st), 2 * kPairStage);
#pragma unroll
            for (int j = 0; j < kSub; ++j) {  // a k-tile past the slice's end reads zeros
              ptx::tma_load_2d_pair(sX + (st * kSub + j) * kWTile, &p.x[sl], (ks * kSub + j) * kElems, x_row, lead_full);
              ptx::tma_load_2d_pair(sW + (st * kSub + j) * kWTile, wm, (ks * kSub + j) * kElems, w_row, lead_full);
            }
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = F8 ? ptx::idesc_e4m3_f32(256, 256) : ptx::idesc_bf16_f32(256, 256);
      int nk = 0;
      for (int sl = 0; sl < p.n_slices; ++sl) nk += slice_stages(sl);
      int kb = 0;
      bool ok = true;
      for (int tile = pair, j = 0; ok && tile < tiles; tile += npairs, ++j) {
        const int a = j & 1;
        if (*abort_flag || !ptx::mbar_wait(tempty_bar(a), ((j >> 1) & 1) ^ 1, p.wait_ns)) {
          if (!*abort_flag) record(p.status, kDevTimeoutMma);
          *abort_flag = 1;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(a * 256);
        for (int k0 = 0; k0 < nk; ++k0, ++kb) {
          const int st = kb % S;
          if (*abort_flag || !ptx::mbar_wait(full_bar(st), (kb / S) & 1, p.wait_ns)) {
            if (!*abort_flag) record(p.status, kDevTimeoutMma);
            *abort_flag = 1;
            ok = false;
            break;
          }
          ptx::tc_fence_after();
#pragma unroll
          for (int i = 0; i < kSub; ++i) {
            const uint64_t xd = ptx::smem_desc_sw128(sX + (st * kSub + i) * kWTile);
            const uint64_t wd = ptx::smem_desc_sw128(sW + (st * kSub + i) * kWTile);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (F8) ptx::mma_f8_pair(d, xd + 2 * k, wd + 2 * k, idesc, (k0 | i | k) != 0 ? 1u : 0u);
              else ptx::mma_bf16_pair(d, xd + 2 * k, wd + 2 * k, idesc, (k0 | i | k) != 0 ? 1u : 0u);
            }
          }
          ptx::mma_commit_pair_multicast(empty_bar(st), 0x3);
        }
        if (!ok) break;
        ptx::mma_commit_pair_multicast(tfull_bar(a), 0x3);
      }
      ptx::mma_commit_pair_multicast(drain_bar, 0x1);
      if (!ptx::mbar_wait(drain_bar, 0, p.wait_ns)) record(p.status, kDevTimeoutDrain);
    }
  } else {
    const int q = warp & 3;
    for (int tile = pair, j = 0; tile < tiles; tile += npairs, ++j) {
      const int a = j & 1;
      const bool ready = ptx::mbar_wait(tfull_bar(a), (j >> 1) & 1, p.wait_ns);
      if (!ready && lane == 0) record(p.status, kDevTimeoutEpilogue);
      ptx::tc_fence_after();
      if (!__all_sync(0xffffffffu, ready && (*abort_flag == 0))) {
        if (lane == 0) *abort_flag = 1;
        break;
      }
      int mt, nt;
      pair_tile(p, tile, mt, nt);
      const int shard = shard_of(p, nt);
      const long long tok = static_cast<long long>(mt) * 256 + rank * 128 + q * 32 + lane;
      const int feat0 = (nt - p.n_tile0[shard]) * 256;
      const uint32_t tb = tmem + static_cast<uint32_t>(a * 256) + (static_cast<uint32_t>(q * 32) << 16);
      const uint32_t lead_tempty = ptx::mapa_shared(tempty_bar(a), 0);
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        uint32_t v[32];
        ptx::tmem_ld_32cols(tb + c, v);
        ptx::tmem_ld_wait();
        ptx::tmem_regs_ready(v);
        if (c + 32 == 256) {
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_remote(lead_tempty);
        }
        const int left = p.n[shard] - feat0 - c;
        if (tok < p.rows && left > 0) {
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float f[4] = {__uint_as_float(v[i]), __uint_as_float(v[i + 1]), __uint_as_float(v[i + 2]),
                          __uint_as_float(v[i + 3])};
            if (left - i > 0) finish4(p, tok, p.col0[shard] + feat0 + c + i, left - i, f);
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// Dynamic shared memory above 48 KB, granted once per device and kernel.
template <typename K>
cudaError_t allow_smem(K kernel, unsigned &mask, std::mutex &mu) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> g(mu);
  if (dev < 32 && (mask & (1u << dev))) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
  if (e == cudaSuccess && dev < 32) mask |= 1u << dev;
  return e;
}

template <bool F8>
tp_status launch_split(const LinearParams &p, size_t smem, cudaStream_t s) {
  static unsigned mask = 0;
  static std::mutex mu;
  const cudaError_t e = allow_smem(k_linear_split<F8>, mask, mu);
  if (e != cudaSuccess) return cuda_fail(e);
  return launched(launch_kernel(k_linear_split<F8>, dim3(static_cast<unsigned>(p.m_tiles * p.n_tiles * p.split)),
                                dim3(kThreads), smem, s, static_cast<unsigned>(p.split), p));
}
template <bool F8>
tp_status launch_pair(const LinearParams &p, cudaStream_t s) {
  static unsigned mask = 0;
  static std::mutex mu;
  const cudaError_t e = allow_smem(k_linear_pair<F8>, mask, mu);
  if (e != cudaSuccess) return cuda_fail(e);
  const int tiles = p.m_tiles * p.n_tiles, most = num_sms() / 2;
  return launched(launch_kernel(k_linear_pair<F8>, dim3(2u * static_cast<unsigned>(tiles < most ? tiles : most)),
                                dim3(kThreads), kPairSmem, s, 1, p));
}

// Whether view b continues view a to the right (same rows, next columns) or below.
bool continues_right(const tp_tensor &a, const tp_tensor &b) {
  return a.rows == b.rows && (a.ld == b.ld || a.rows == 1) &&
         static_cast<const char *>(a.ptr) + a.cols * elem_size(a.dtype) == b.ptr;
}
bool continues_below(const tp_tensor &a, const tp_tensor &b) {
  return a.ld == b.ld && static_cast<const char *>(a.ptr) + a.rows * a.ld * elem_size(a.dtype) == b.ptr;
}

}  // namespace
}  // namespace tpgqa

using namespace tpgqa;
using namespace tpgqa::op;

extern "C" tp_status tp_linear_epilogue(int32_t n, int32_t shard, const tp_tensor *x, const float *x_scale,
                                        const tp_tensor *w, const float *w_scale, const tp_tensor *bias,
                                        int32_t activation, const tp_tensor *residual, tp_tensor *y, tp_stream_t stream) {
  if (n < 1 || n > 64) return TP_ERR_INVALID_ARG;
  if (n & (n - 1)) return TP_ERR_TP_SIZE_NOT_POW2;
  if (!x || !w || !y || (shard != TP_SHARD_COLUMN && shard != TP_SHARD_ROW)) return TP_ERR_INVALID_ARG;
  if (activation < TP_ACT_NONE || activation > TP_ACT_SILU) return TP_ERR_INVALID_ARG;
  const bool row = shard == TP_SHARD_ROW;
  const int32_t dt = x[0].dtype;
  const long long T = x[0].rows;
  long long total_n = 0;
  for (int32_t r = 0; r < n; ++r) {
    const tp_tensor &xr = x[row ? r : 0];
    if (!view_ok(xr) || !view_ok(w[r])) return TP_ERR_INVALID_ARG;
    if ((dt != TP_BF16 && dt != TP_E4M3) || xr.dtype != dt || w[r].dtype != dt) return TP_ERR_DTYPE;
    if (xr.rows != T || w[r].cols != xr.cols || (row && w[r].rows != w[0].rows)) return TP_ERR_INVALID_ARG;
    if (!row) total_n += w[r].rows;
  }
  if (row) total_n = w[0].rows;
  if (total_n > 0x7fffffffLL) return TP_ERR_INVALID_ARG;
  if (!view_ok(*y) || y->rows != T || y->cols != total_n) return TP_ERR_INVALID_ARG;
  if (y->dtype != TP_F32 && y->dtype != TP_BF16) return TP_ERR_DTYPE;
  if (bias) {
    if (!view_ok(*bias) || bias->rows != 1 || bias->cols != total_n) return TP_ERR_INVALID_ARG;
    if (bias->dtype != TP_F32 && bias->dtype != TP_BF16) return TP_ERR_DTYPE;
    if (!elem_aligned(*bias)) return TP_ERR_ALIGNMENT;
  }
  if (residual) {
    if (!view_ok(*residual) || residual->rows != T || residual->cols != total_n) return TP_ERR_INVALID_ARG;
    if (residual->dtype != TP_F32 && residual->dtype != TP_BF16) return TP_ERR_DTYPE;
  }
  const bool empty = T == 0 || total_n == 0;
  // scales exactly where the operands are 8-bit
  if (!empty && ((dt == TP_E4M3) != (x_scale != nullptr) || (dt == TP_E4M3) != (w_scale != nullptr)))
    return TP_ERR_INVALID_ARG;
  if (!ptr_aligned(x_scale, 4) || !ptr_aligned(w_scale, 4)) return TP_ERR_ALIGNMENT;
  if (!empty) {
    for (int32_t r = 0; r < n; ++r) {
      const bool some = w[r].rows > 0 && w[r].cols > 0;  // an empty slice is skipped
      if (some && (!vec_aligned(x[row ? r : 0]) || !vec_aligned(w[r]))) return TP_ERR_ALIGNMENT;
      if (!row && r + 1 < n && (w[r].rows * elem_size(y->dtype)) % 16) return TP_ERR_ALIGNMENT;
      if (!row && r + 1 < n && residual && (w[r].rows * elem_size(residual->dtype)) % 16) return TP_ERR_ALIGNMENT;
    }
    if (!vec_aligned(*y) || (residual && !vec_aligned(*residual))) return TP_ERR_ALIGNMENT;
  }
  tp_status st = check_rank_health(n);
  if (st != TP_OK) return st;
  if (empty) return TP_OK;

  // Neighbouring slices (or shards) of one tensor are one K range (or one weight):
  // fewer tensor maps, and no tile or k-tile ends at a rank's border.
  tp_tensor xs[64], ws[64];
  int parts = 0;
  for (int32_t r = 0; r < n; ++r) {
    if (row ? w[r].cols == 0 : w[r].rows == 0) continue;
    if (parts > 0) {
      tp_tensor &px = xs[parts - 1], &pw = ws[parts - 1];
      if (row && continues_right(px, x[r]) && continues_right(pw, w[r]) && px.cols + x[r].cols <= 0x7fffffffLL) {
        px.cols += x[r].cols;
        pw.cols += w[r].cols;
        continue;
      }
      if (!row && continues_below(pw, w[r])) {
        pw.rows += w[r].rows;
        continue;
      }
    }
    xs[parts] = x[row ? r : 0];
    ws[parts++] = w[r];
  }
  if (parts == 0 || xs[0].cols == 0) return TP_ERR_UNSUPPORTED;  // no input features at all
  if (parts > kMaxParts) return TP_ERR_UNSUPPORTED;
  for (int i = 0; i < parts; ++i)  // the pitch of a single row is free: any legal one for its tensor map
    for (tp_tensor *t : {&xs[i], &ws[i]})
      if (t->rows == 1) t->ld = (t->cols + 15) / 16 * 16;
  DevCtx ctx;
  const cudaError_t e = get_dev_ctx(&ctx);
  if (e != cudaSuccess) return cuda_fail(e);
  static thread_local LinearParams p;  // tensor maps: kept off the stack
  std::memset(&p, 0, sizeof(p));
  p.n_slices = row ? parts : 1;
  p.n_shards = row ? 1 : parts;
  const int elems = dt == TP_E4M3 ? 128 : 64;
  for (int i = 0; i < p.n_slices; ++i) {
    p.k_tiles[i] = static_cast<int>((xs[i].cols + elems - 1) / elems);
    p.kt_total += p.k_tiles[i];
  }
  long long col = 0;
  auto lay_out = [&](int tile_n) {
    p.n_tiles = 0;
    col = 0;
    for (int i = 0; i < p.n_shards; ++i) {
      p.n[i] = static_cast<int>(ws[i].rows);
      p.n_tile0[i] = p.n_tiles;
      p.col0[i] = col;
      p.n_tiles += static_cast<int>((ws[i].rows + tile_n - 1) / tile_n);
      col += ws[i].rows;
    }
  };
  p.rows = static_cast<int>(T);
  p.act = activation;
  p.y_f32 = y->dtype == TP_F32;
  p.res_f32 = residual && residual->dtype == TP_F32;
  p.bias_f32 = bias && bias->dtype == TP_F32;
  p.x_scale = x_scale;
  p.w_scale = w_scale;
  p.bias = bias ? bias->ptr : nullptr;
  p.res = residual ? residual->ptr : nullptr;
  p.res_ld = residual ? residual->ld : 0;
  p.y = y->ptr;
  p.y_ld = y->ld;
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  const char *env = getenv("TPGQA_EARLY_B");
  p.early_w = !(env && env[0] == '0');
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);

  // The pair kernel from half a wave of its tiles on; below that the split kernel's
  // smaller tiles and its split of K put more SMs to work.
  lay_out(256);
  const long long m256 = (T + 255) / 256;
  const bool pair = T > 128 && m256 * p.n_tiles >= num_sms() / 4;
  int x_box, w_box = 128;
  if (pair) {
    x_box = 128;
    p.m_tiles = static_cast<int>(m256);
    if (m256 * p.n_tiles > 0x7fffffffLL) return TP_ERR_UNSUPPORTED;
  } else {
    lay_out(128);
    p.m_tiles = static_cast<int>(m256);
    const long long per = (T + p.m_tiles - 1) / p.m_tiles;
    p.tok_tile = static_cast<int>((per + 15) / 16 * 16);
    x_box = p.tok_tile;
    const int stage = kWTile + p.tok_tile * 128;
    p.stages = (kSmemLimit - 1024 - 512) / stage;
    if (p.stages > 12) p.stages = 12;
    // the largest cluster that one wave holds, with at least two k-tiles a CTA
    const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles;
    p.split = 1;
    for (int c = 2; c <= 8; ++c)
      if (tiles * c <= num_sms() && tiles <= max_active_clusters(c) && p.kt_total >= 2 * c) p.split = c;
    if (tiles * p.split > 0x7fffffffLL) return TP_ERR_UNSUPPORTED;
  }
  for (int i = 0; i < p.n_slices; ++i)
    if (!encode_rows_map(&p.x[i], xs[i], x_box)) return TP_ERR_INVALID_ARG;
  for (int i = 0; i < parts; ++i)
    if (!encode_rows_map(&p.w[i], ws[i], w_box)) return TP_ERR_INVALID_ARG;
  if (pair) return dt == TP_E4M3 ? launch_pair<true>(p, s) : launch_pair<false>(p, s);
  const size_t smem = 1024 + static_cast<size_t>(p.stages) * (kWTile + p.tok_tile * 128) + 8 * (2 * p.stages + 2) + 64;
  return dt == TP_E4M3 ? launch_split<true>(p, smem, s) : launch_split<false>(p, smem, s);
}
