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
//                   bytes a token of X, 170 to 220 KB in flight per SM. Too few
//                   feature tiles to fill the SMs split K over a cluster; the f32
//                   partials are summed through distributed shared memory in rank
//                   order, so results repeat.
//   k_linear_pair   many tokens. Bound by the tensor cores: persistent SM pairs on
//                   tiles of 256 tokens x BN features (cta_group::2). The tile's sum
//                   lives in the epilogue warps' registers, so both accumulators
//                   in TMEM stay with the MMAs, under which the whole epilogue runs.
//
// The tensor core truncates where it adds a step's products into the f32
// accumulator: an error of one sign that grows with the steps. So no accumulator
// runs for more than kChunkSteps steps (1024 bf16 or 2048 e4m3 values of K): both
// kernels add a chunk's products to the sum outside the tensor core, rounding to
// nearest. k_linear_pair's epilogue keeps the sum in registers. k_linear_split gives
// each chunk its own columns of TMEM and adds them at the end; what does not fit (half
// of the columns, where two CTAs share an SM) is added to the first chunk's columns
// under the products. Over K = 8192 in bf16 this takes the error of an f32 output,
// relative to its size, from 8e-6 to 1e-6, an f32 sum's.
// Warp roles in both: warp 0 loads (TMA), warp 1 issues the MMAs, the others are
// the epilogue. Every wait is bounded, as in the grouped GEMM.
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "op_util.h"
#include "sm100_ptx.cuh"

namespace tpgqa {
namespace {

using namespace op;

constexpr int kThreads = 256;       // k_linear_split
constexpr int kChunkSteps = 64;     // MMA steps (32 bytes of K each) of one accumulator
constexpr int kMaxRegions = 8;      // accumulators of k_linear_split: 256 columns of 32
constexpr int kMaxParts = 16;  // weight shards (column) or K slices (row)
constexpr int kSmemLimit = 227 * 1024;
constexpr int kWTile = 128 * 128;  // bytes of one 128-row, 128-byte-wide box

// The scalars come first and lie together: a kernel's first read of each 64-byte
// line of its parameters is a miss of a few hundred nanoseconds.
struct LinearParams {
  int tok_tile, stages, split;       // k_linear_split: token tile, stages (one k-tile each), CTAs sharing K
  int box3;                          // k_linear_pair: one copy of a 3-D box brings a stage's k-tiles of an operand
  int regions, region_cols, tmem_cols;  // its accumulators in TMEM, their stride, and what it allocates
  int early_w;                       // W loads before the dependency wait
  int n_slices, n_shards, kt_total, n_tiles, rows, m_tiles;
  int act, y_f32, res_f32, bias_f32, wide32;  // wide32: f32 rows of residual and y in 32-byte accesses
  const float *x_scale, *w_scale;  // null: no scales
  const void *bias, *res;          // null: none
  void *y;
  long long y_ld, res_ld;
  int *status;
  long long wait_ns;
  struct {
    int n;       // output features of a shard
    int tile0;   // its first feature tile
    long long col0;  // its first output column
  } shard[kMaxParts];
  int k_tiles[kMaxParts];    // 128-byte-wide k-tiles of each K slice
  CUtensorMap w[kMaxParts];  // one per K slice, or one per weight shard
  CUtensorMap x[kMaxParts];  // one per K slice
};

__device__ __forceinline__ void record(int *status, int code) { atomicCAS(status, 0, code); }

// Shard of a feature tile (shards are laid out in tile order).
__device__ __forceinline__ int shard_of(const LinearParams &p, int nt) {
  int s = 0;
  while (s + 1 < p.n_shards && nt >= p.shard[s + 1].tile0) ++s;
  return s;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// x Phi(x) of two values, from h = Phi(-|x|) = t P(t) e^(-x^2/2) with t = 1 / (1 + 0.27 |x|):
// x h below 0, where x/2 (1 + erf) would cancel (below -4.5 it keeps fewer bits than bf16), x (1 - h)
// above. P is the polynomial of degree 8 nearest to erfc(|x| / sqrt 2) e^(x^2/2) / (2 t)
// relative to it (2.4e-8), by a weighted least-squares fit over |x| <= 14.
__device__ __forceinline__ void gelu2(float &x0, float &x1) {
  const float t0 = rcp(fmaf(fabsf(x0), 0.27f, 1.0f)), t1 = rcp(fmaf(fabsf(x1), 0.27f, 1.0f));
  const uint64_t t = pack2(t0, t1);
  uint64_t q = pack2(0.028915392f, 0.028915392f);
  q = fma2(q, t, pack2(-0.12625581f, -0.12625581f));
  q = fma2(q, t, pack2(0.16929251f, 0.16929251f));
  q = fma2(q, t, pack2(-0.068622246f, -0.068622246f));
  q = fma2(q, t, pack2(0.1074003f, 0.1074003f));
  q = fma2(q, t, pack2(0.072239928f, 0.072239928f));
  q = fma2(q, t, pack2(0.10175926f, 0.10175926f));
  q = fma2(q, t, pack2(0.10755049f, 0.10755049f));
  q = fma2(q, t, pack2(0.10772019f, 0.10772019f));
  float q0, q1;
  unpack2(q, q0, q1);
  const float h0 = q0 * t0 * ex2(x0 * x0 * -0.72134752f), h1 = q1 * t1 * ex2(x1 * x1 * -0.72134752f);
  x0 *= x0 < 0.0f ? h0 : 1.0f - h0;
  x1 *= x1 < 0.0f ? h1 : 1.0f - h1;
}
// x / (1 + e^-x) for an f32 output, within 6 2^-24 of it: e^-x is 2^t, and the rounding of
// t = -x log2(e), up to 2^-18 of e^-x, is brought in again behind it; the quotient is corrected
// by its remainder. From 20 on it is x; t stops at 126, so below -88 it is 2^-126 x.
__device__ __forceinline__ float silu_f32(float x) {
  const float c = 1.442695041f, c_low = 1.925963033e-8f;  // log2(e), and what f32 leaves of it
  const float t = x * -c, e0 = ex2(fminf(t, 126.0f));
  const float low = fmaf(x, -c_low, fmaf(x, -c, -t)) * 0.6931471806f;
  const float d = 1.0f + fmaf(e0, low, e0), r = rcp(d), q = x * r;
  return x > 20.0f ? x : fmaf(fmaf(-q, d, x), r, q);
}

// The activations by their formulas, in f32: relu, x Phi(x), x / (1 + e^-x). For a bf16 output
// the last by the hardware's exponential and reciprocal alone, off by up to 2^-23 |x| of its
// value (at x < -88 it is -0, its limit): far below bf16's half step of 2^-9, and the exact
// form costs 4096 x 8192 x 28672 in e4m3 7%.
template <int N>
__device__ __forceinline__ void activate(float (&f)[N], int act, bool f32) {
  if (act == TP_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = f[i] < 0.0f ? 0.0f : f[i];  // keeps NaN
  } else if (act == TP_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; i += 2) gelu2(f[i], f[i + 1]);
  } else if (act == TP_ACT_SILU && f32) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = silu_f32(f[i]);
  } else if (act == TP_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] *= rcp(1.0f + ex2(f[i] * -1.442695041f));
  }
}

// 32 bytes in one access.
__device__ __forceinline__ void load32(const float *p, float (&v)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store32(float *p, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// N neighbouring values of a row of f32 or bf16 as f32; `left` of them exist, the
// rest read as 0. Whole groups are aligned for vector loads.
template <int N>
__device__ __forceinline__ void load_row(const void *base, bool f32, long long at, int left, float (&v)[N]) {
  if (f32) {
    const float *r = static_cast<const float *>(base) + at;
    if (left >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 w = *reinterpret_cast<const float4 *>(r + i);
        v[i] = w.x; v[i + 1] = w.y; v[i + 2] = w.z; v[i + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = i < left ? r[i] : 0.f;
    }
  } else {
    const __nv_bfloat16 *r = static_cast<const __nv_bfloat16 *>(base) + at;
    if (left >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint2 w = *reinterpret_cast<const uint2 *>(r + i);
        v[i] = bf16_lo(w.x); v[i + 1] = bf16_hi(w.x); v[i + 2] = bf16_lo(w.y); v[i + 3] = bf16_hi(w.y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = i < left ? __bfloat162float(r[i]) : 0.f;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_row(void *base, bool f32, long long at, int left, const float (&v)[N]) {
  if (f32) {
    float *r = static_cast<float *>(base) + at;
    if (left >= N) {
#pragma unroll
      for (int i = 0; i < N; i += 4) *reinterpret_cast<float4 *>(r + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) r[i] = v[i];
    }
  } else {
    __nv_bfloat16 *r = static_cast<__nv_bfloat16 *>(base) + at;
    if (left >= N) {
      if constexpr (N % 8 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 8)
          *reinterpret_cast<uint4 *>(r + i) = make_uint4(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]),
                                                         pack_bf16(v[i + 4], v[i + 5]), pack_bf16(v[i + 6], v[i + 7]));
      } else {
#pragma unroll
        for (int i = 0; i < N; i += 4)
          *reinterpret_cast<uint2 *>(r + i) = make_uint2(pack_bf16(v[i], v[i + 1]), pack_bf16(v[i + 2], v[i + 3]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < left) r[i] = __float2bfloat16_rn(v[i]);
    }
  }
}

// Scale of the weight's feature and bias at output column c; 1 and 0 where there is none.
__device__ __forceinline__ float2 column_terms(const LinearParams &p, long long c, bool there) {
  float2 t = make_float2(1.f, 0.f);
  if (there) {
    if (p.w_scale) t.x = __ldg(p.w_scale + c);
    if (p.bias)
      t.y = p.bias_f32 ? __ldg(static_cast<const float *>(p.bias) + c)
                       : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.bias)[c]);
  }
  return t;
}

// ---------------------------------------------------------------------------
// Few tokens: features on the MMA's M, tokens on its N, K split over a cluster.
// 61 tokens, 4096 -> 14336 in e4m3 with GELU: 15.3 us for 61 MB; its weights stream in
// 7 us (8 TB/s), the rest is the start (2 us to the first stage), the partials'
// exchange (2 us) and the output (2 us). One token, 4096 -> 4096 in bf16: 9.0 us.
// ---------------------------------------------------------------------------
// ADD: a CTA's K has more chunks than accumulators (a kernel of its own: the code costs the others 0.15 us).
template <bool F8, bool ADD>
__global__ void __launch_bounds__(kThreads, 2) k_linear_split(const __grid_constant__ LinearParams p) {
  constexpr int kElems = F8 ? 128 : 64;  // values of a 128-byte box row
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int S = p.stages, NT = p.tok_tile;
  const uint32_t stage_bytes = kWTile + static_cast<uint32_t>(NT) * 128u;
  const uint32_t sbase = ptx::smem_addr(smem);
  auto w_slot = [&](int st) { return sbase + static_cast<uint32_t>(st) * stage_bytes; };
  uint8_t *bar_area = smem + max(static_cast<uint32_t>(S) * stage_bytes, static_cast<uint32_t>(NT) * 512u);
  const uint32_t bar0 = ptx::smem_addr(bar_area);
  auto full_bar = [&](int i) { return bar0 + 8u * i; };
  auto empty_bar = [&](int i) { return bar0 + 8u * (S + i); };
  const uint32_t done_bar = bar0 + 8u * (2 * S);
  auto chunk_bar = [&](int r) { return bar0 + 8u * (2 * S + 1 + r); };  // an accumulator is whole
  auto added_bar = [&](int r) { return bar0 + 8u * (2 * S + 1 + kMaxRegions + r); };  // and added to the first
  constexpr int kBars = 1 + 2 * kMaxRegions;  // beside the stages'
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bar_area + 8 * (2 * S + kBars));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bar_area + 8 * (2 * S + kBars) + 4);
  float *s_scale = reinterpret_cast<float *>(bar_area + 8 * (2 * S + kBars + 1));  // [token]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int part = p.split > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int tile = blockIdx.x / p.split;
  const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;  // token tiles of one feature tile are neighbours
  const int shard = shard_of(p, nt);
  const int feat0 = (nt - p.shard[shard].tile0) * 128;  // within the shard
  const int kb0 = static_cast<int>(static_cast<long long>(p.kt_total) * part / p.split);
  const int kb1 = static_cast<int>(static_cast<long long>(p.kt_total) * (part + 1) / p.split);
  const uint32_t tmem_cols = static_cast<uint32_t>(p.tmem_cols);
  const int nkb = kb1 - kb0;
  // Chunks of K. The first p.regions of them have an accumulator each. Accumulator 0 keeps the
  // first; a later chunk takes the place of an earlier one in the others, which warps 4 to 7
  // have added to accumulator 0 by then: chunks 1 to to_add.
  constexpr int kChunkKt = kChunkSteps / 4;
  const int to_add = ADD ? max((nkb + kChunkKt - 1) / kChunkKt - p.regions, 0) : 0;
  const int chunk_kt = ADD ? kChunkKt : (nkb + p.regions - 1) / p.regions;

  // The loading thread's cursors over the k-tiles, (slice, k-tile in it), of W and of X.
  struct Cursor {
    int sl, kt;
  };
  auto next = [&](Cursor &c) {
    if (++c.kt == p.k_tiles[c.sl]) {
      c.kt = 0;
      ++c.sl;
    }
  };
  Cursor wc = {0, kb0};
  while (wc.kt >= p.k_tiles[wc.sl]) wc.kt -= p.k_tiles[wc.sl++];
  Cursor xc = wc;
  int pre = 0;
  // The loops of the issuing warps hold no division: a remainder by the run-time
  // stage count costs as much as the rest of a step.
  auto load_w = [&](int st, bool issue) {
    if (issue) {
      ptx::mbar_arrive_expect_tx(full_bar(st), kWTile);
      ptx::tma_load_2d(w_slot(st), &p.w[p.n_shards > 1 ? shard : wc.sl], wc.kt * kElems, feat0, full_bar(st));
    }
    next(wc);
  };
  auto load_x = [&](int st, bool issue) {
    if (issue) {
      ptx::mbar_arrive_expect_tx(full_bar(st), stage_bytes - kWTile);
      ptx::tma_load_2d(w_slot(st) + kWTile, &p.x[xc.sl], xc.kt * kElems, mt * NT, full_bar(st));
    }
    next(xc);
  };
  if (warp == 0) {
    const bool leader = ptx::elect_one();
    if (leader) {
      for (int i = 0; i < S; ++i) {
        ptx::mbar_init(full_bar(i), 2);  // W's and X's loading warps
        ptx::mbar_init(empty_bar(i), 1);
      }
      ptx::mbar_init(done_bar, 1);
      if (ADD)
        for (int r = 1; r < p.regions; ++r) {
          ptx::mbar_init(chunk_bar(r), 1);
          ptx::mbar_init(added_bar(r), 4);
        }
      *abort_flag = 0;
      ptx::fence_barrier_init();
      ptx::fence_proxy_async_smem();
    }
    // W does not come from the previous kernel: its first stages start before the
    // grid-dependency wait and before anything else of this CTA.
    if (p.early_w)
      for (; pre < S && pre < nkb; ++pre) load_w(pre, leader);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t *>(tmem_slot)), tmem_cols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  // Warp 0 loads W, warp 2 loads X; the other warps fetch the tokens' scales. A warp
  // walks its stages converged and one lane issues: with a branch on the lane index
  // around the whole walk an issue took about 300 ns, which set the kernel's pace.
  if (warp == 0 || warp == 2) {
    const bool leader = ptx::elect_one();
    int st = 0;
    uint32_t parity = 1;  // of the stage's empty barrier
    for (int i = 0; i < nkb; ++i) {
      if (i >= S && !__all_sync(0xffffffffu, ptx::mbar_wait(empty_bar(st), parity, p.wait_ns))) {
        record(p.status, kDevTimeoutProducer);
        *abort_flag = 1;
        break;
      }
      if (warp == 2) load_x(st, leader);
      else if (i >= pre) load_w(st, leader);
      if (++st == S) {
        st = 0;
        parity ^= 1;
      }
    }
  } else if (warp >= 3) {
    for (int t = threadIdx.x - 96; t < NT; t += kThreads - 96) {
      const long long tok = static_cast<long long>(mt) * NT + t;
      s_scale[t] = p.x_scale && tok < p.rows ? __ldg(p.x_scale + tok) : 1.f;
    }
    if (ADD && warp >= 4) {  // a warp per quarter of the TMEM lanes
      const uint32_t sum_at = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      int region = 1;
      uint32_t parity = 0;
      for (int i = 0; i < to_add; ++i) {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(chunk_bar(region), parity, p.wait_ns))) {
          record(p.status, kDevTimeoutEpilogue);
          *abort_flag = 1;
          break;
        }
        ptx::tc_fence_after();
        for (int c = 0; c < NT; c += 32) {  // 32 columns' loads in flight; an odd 16 at the end twice
          const int c2 = c + 16 < NT ? c + 16 : c;
          uint32_t v[2][16], sum[2][16];
          ptx::tmem_ld_16cols(sum_at + region * p.region_cols + c, v[0]);
          ptx::tmem_ld_16cols(sum_at + c, sum[0]);
          ptx::tmem_ld_16cols(sum_at + region * p.region_cols + c2, v[1]);
          ptx::tmem_ld_16cols(sum_at + c2, sum[1]);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ptx::tmem_regs_ready(v[h]);
            ptx::tmem_regs_ready(sum[h]);
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[h][j] = __float_as_uint(__uint_as_float(sum[h][j]) + __uint_as_float(v[h][j]));
            ptx::tmem_st_16cols(sum_at + (h ? c2 : c), sum[h]);
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(added_bar(region));
        if (++region == p.regions) {
          region = 1;
          parity ^= 1;
        }
      }
    }
  }
  if (warp == 1) {  // the whole warp walks the stages, one lane issues
    const uint32_t idesc = F8 ? ptx::idesc_e4m3_f32(128, NT) : ptx::idesc_bf16_f32(128, NT);
    const bool leader = ptx::elect_one();
    int st = 0, region = 0;
    uint32_t parity = 0, reuse = 1, d = tmem;  // reuse: parity of the additions that the present accumulator waits for
    bool go = true;
    for (int i = 0, chunk = 0; go && i < nkb; ++chunk) {
      if (ADD && chunk >= p.regions && !__all_sync(0xffffffffu, ptx::mbar_wait(added_bar(region), reuse, p.wait_ns))) {
        record(p.status, kDevTimeoutMma);
        *abort_flag = 1;
        break;
      }
      const int end = min(nkb, i + chunk_kt);
      for (uint32_t more = 0; i < end; ++i, more = 1) {
        if (!__all_sync(0xffffffffu, ptx::mbar_wait(full_bar(st), parity, p.wait_ns))) {
          record(p.status, kDevTimeoutMma);
          *abort_flag = 1;
          go = false;
          break;
        }
        ptx::tc_fence_after();
        const uint64_t wd = ptx::smem_desc_sw128(w_slot(st)), xd = ptx::smem_desc_sw128(w_slot(st) + kWTile);
        if (leader) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (F8) ptx::mma_f8(d, wd + 2 * k, xd + 2 * k, idesc, k != 0 ? 1u : more);
            else ptx::mma_bf16(d, wd + 2 * k, xd + 2 * k, idesc, k != 0 ? 1u : more);
          }
        }
        if (leader) ptx::mma_commit(empty_bar(st));
        __syncwarp();
        if (++st == S) {
          st = 0;
          parity ^= 1;
        }
      }
      d += static_cast<uint32_t>(p.region_cols);  // the next accumulator
      if (ADD) {
        if (leader && chunk > 0 && chunk <= to_add) ptx::mma_commit(chunk_bar(region));
        __syncwarp();
        if (++region == p.regions) {
          region = 1;
          reuse ^= 1;
          d = tmem + static_cast<uint32_t>(p.region_cols);
        }
      }
    }
    if (leader) ptx::mma_commit(done_bar);
  }
  __syncwarp();
  // this lane's four features: their terms load under the products
  const int left = p.shard[shard].n - feat0 - lane * 4;
  const long long col = p.shard[shard].col0 + feat0 + lane * 4;
  float2 terms[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) terms[i] = column_terms(p, col + i, i < left);
  // Every warp waits for the last product; the stage buffers are free from then on.
  const bool ready = __all_sync(0xffffffffu, ptx::mbar_wait(done_bar, 0, p.wait_ns));
  if (!ready && lane == 0) {
    record(p.status, kDevTimeoutEpilogue);
    *abort_flag = 1;
  }
  ptx::tc_fence_after();
  float *red = reinterpret_cast<float *>(smem);  // [token][128 features] f32
  if (ready) {  // two warps per quarter of the TMEM lanes, every other 16 tokens each
    const int q = warp & 3;
    const int used = min((nkb + chunk_kt - 1) / chunk_kt, p.regions);
    for (int c = 16 * (warp >> 2); c < NT; c += 32) {
      float f[16];
      for (int r = 0; r < used; r += 2) {  // two accumulators' loads in flight
        uint32_t v[16], w[16];
        const uint32_t at = tmem + r * p.region_cols + c + (static_cast<uint32_t>(q * 32) << 16);
        const bool two = r + 1 < used;
        ptx::tmem_ld_16cols(at, v);
        ptx::tmem_ld_16cols(two ? at + p.region_cols : at, w);
        ptx::tmem_ld_wait();
        ptx::tmem_regs_ready(v);
        ptx::tmem_regs_ready(w);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          f[j] = r == 0 ? __uint_as_float(v[j]) : f[j] + __uint_as_float(v[j]);
          if (two) f[j] += __uint_as_float(w[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) red[(c + j) * 128 + q * 32 + lane] = f[j];
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
  // The cluster's CTAs share the tile's tokens. A warp finishes two tokens at a
  // time, four features a lane; the partials are added in cluster order.
  if (*abort_flag == 0) {
    constexpr int kWarps = kThreads / 32, kTok = 2;
    const int t1 = min(NT * (part + 1) / p.split, static_cast<int>(p.rows - static_cast<long long>(mt) * NT));
    const uint32_t red_addr = ptx::smem_addr(red) + static_cast<uint32_t>(lane * 16);
#pragma unroll 1
    for (int t0 = NT * part / p.split + warp; t0 < t1; t0 += kTok * kWarps) {
      float f[kTok][4], res[kTok][4], sx[kTok];
      const long long tok0 = static_cast<long long>(mt) * NT + t0;
#pragma unroll
      for (int u = 0; u < kTok; ++u) {
        const bool on = t0 + u * kWarps < t1 && left > 0;
        sx[u] = on ? s_scale[t0 + u * kWarps] : 1.f;
        if (p.res && on) load_row(p.res, p.res_f32, (tok0 + u * kWarps) * p.res_ld + col, left, res[u]);
      }
      if (p.split == 1) {
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
          const float4 v = ptx::ld_shared_f4(red_addr + static_cast<uint32_t>(min(t0 + u * kWarps, t1 - 1)) * 512u);
          f[u][0] = v.x; f[u][1] = v.y; f[u][2] = v.z; f[u][3] = v.w;
        }
      } else {
        float4 v[8][kTok];  // every partial's load is in flight before the first is added
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (r < p.split)
#pragma unroll
            for (int u = 0; u < kTok; ++u)
              v[r][u] = ptx::ld_shared_cluster_f4(
                  ptx::mapa_shared(red_addr + static_cast<uint32_t>(min(t0 + u * kWarps, t1 - 1)) * 512u, r));
#pragma unroll
        for (int u = 0; u < kTok; ++u) {
          f[u][0] = v[0][u].x; f[u][1] = v[0][u].y; f[u][2] = v[0][u].z; f[u][3] = v[0][u].w;
        }
#pragma unroll
        for (int r = 1; r < 8; ++r)
          if (r < p.split)
#pragma unroll
            for (int u = 0; u < kTok; ++u) {
              f[u][0] += v[r][u].x; f[u][1] += v[r][u].y; f[u][2] += v[r][u].z; f[u][3] += v[r][u].w;
            }
      }
#pragma unroll
      for (int u = 0; u < kTok; ++u) {
        if (t0 + u * kWarps >= t1 || left <= 0) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[u][i] = f[u][i] * (sx[u] * terms[i].x) + terms[i].y;
        activate(f[u], p.act, p.y_f32);
        if (p.res) {
#pragma unroll
          for (int i = 0; i < 4; ++i) f[u][i] += res[u][i];
        }
        store_row(p.y, p.y_f32, (tok0 + u * kWarps) * p.y_ld + col, left, f[u]);
      }
    }
  }
  __syncwarp();
  if (p.split > 1) ptx::cluster_sync_relaxed();  // peers have read this CTA's partials
}

// ---------------------------------------------------------------------------
// Many tokens: persistent SM pairs, 256 tokens x BN features per tile. Each CTA
// holds its 128 tokens' accumulator rows and loads its half of the W rows. Eight
// epilogue warps: two per quarter of the TMEM lanes, each with half of the columns.
// BN is at most 224: the 128 sums a lane of BN = 256 spill (4096 x 8192 x 28672 in e4m3:
// 638 us against 578). That product runs at 2.9-3.3 PFLOP/s, by the clock the power
// cap leaves; the tensor pipe is active 66% of the cycles on 2048 x 8192 x 8192, where
// a CTA takes in 69 bytes a clock, near what its copies bring. 2047 x 8192 x 8192 in
// bf16: 168 us with an f32 output, 199 with an f32 residual too.
// ---------------------------------------------------------------------------
constexpr int kSub = 2;           // k-tiles per stage
constexpr int kPairThreads = 320;
constexpr int kChunkStages = kChunkSteps / 4 / kSub;
constexpr int kGroup = 16;  // token tiles walked for one feature tile before the next (keeps both in L2)

template <int BN>
struct PairCfg {
  static constexpr int kWBytes = BN / 2 * 128;  // this CTA's rows of one k-tile of W
  static constexpr int kStage = kSub * (kWTile + kWBytes);
  static constexpr int kTerms = 8 * (BN / 2) * 8;  // scale and bias of each epilogue warp's columns
  static constexpr int kFit = (kSmemLimit - 1024 - 256 - kTerms) / kStage;
  static constexpr int kStages = kFit > 4 ? 4 : kFit;
  static constexpr int kSmem = 1024 + kStages * kStage + kTerms + 256;
  static_assert(kWBytes % 1024 == 0, "k-tiles keep the swizzle's alignment");
};

// Tile -> (token tile, feature tile): groups of kGroup token tiles, token tile fastest.
__device__ __forceinline__ void pair_tile(const LinearParams &p, int tile, int &mt, int &nt) {
  const int per_group = kGroup * p.n_tiles;
  const int grp = tile / per_group, r = tile - grp * per_group;
  const int rows = min(kGroup, p.m_tiles - grp * kGroup);
  mt = grp * kGroup + r % rows;
  nt = r / rows;
}

// Y32: an f32 output. As a template parameter it halves the epilogue's unrolled code, whose length
// shows: with both kinds of output in one kernel the widest product takes 2% more.
template <bool F8, int BN, bool Y32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_linear_pair(const __grid_constant__ LinearParams p) {
  using C = PairCfg<BN>;
  constexpr int kElems = F8 ? 128 : 64;
  constexpr int S = C::kStages;
  constexpr int kHalf = BN / 2;  // columns of an epilogue warp
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sX = ptx::smem_addr(smem), sW = sX + S * kSub * kWTile;
  float2 *terms_area = reinterpret_cast<float2 *>(smem + S * C::kStage);
  uint8_t *bar_area = smem + S * C::kStage + C::kTerms;
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
  int nk = 0;  // stages of a tile, and the chunks they make
  for (int sl = 0; sl < p.n_slices; ++sl) nk += slice_stages(sl);
  const int chunks = (nk + kChunkStages - 1) / kChunkStages;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(full_bar(i), 1);
      ptx::mbar_init(empty_bar(i), 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(tfull_bar(a), 1);
      ptx::mbar_init(tempty_bar(a), 16);  // 8 epilogue warps in each CTA
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

  if (warp == 0) {  // converged, one lane issues
    const bool issue = ptx::elect_one();
    int st = 0;
    uint32_t parity = 1;
    bool go = true;
    for (int tile = pair; go && tile < tiles; tile += npairs) {
      int mt, nt;
      pair_tile(p, tile, mt, nt);
      const int shard = shard_of(p, nt);
      const int x_row = mt * 256 + static_cast<int>(rank) * 128;
      const int w_row = (nt - p.shard[shard].tile0) * BN + static_cast<int>(rank) * kHalf;
      for (int sl = 0; go && sl < p.n_slices; ++sl) {
        const CUtensorMap *wm = &p.w[p.n_shards > 1 ? shard : sl], *xm = &p.x[sl];
        const int stages = slice_stages(sl);
        for (int ks = 0; ks < stages; ++ks) {
          if (!__all_sync(0xffffffffu, ptx::mbar_wait(empty_bar(st), parity, p.wait_ns) && *abort_flag == 0)) {
            if (*abort_flag == 0) record(p.status, kDevTimeoutProducer);
            *abort_flag = 1;
            go = false;
            break;
          }
          const uint32_t lead_full = ptx::mapa_shared(full_bar(st), 0);
          if (issue) {
            if (leader) ptx::mbar_arrive_expect_tx(full_bar(st), 2 * C::kStage);
            // k-tiles past the slice's end read zeros
            if (p.box3) {
              ptx::tma_load_3d_pair(sX + st * kSub * kWTile, xm, 0, x_row, ks * kSub, lead_full);
              ptx::tma_load_3d_pair(sW + st * kSub * C::kWBytes, wm, 0, w_row, ks * kSub, lead_full);
            } else {
#pragma unroll
              for (int j = 0; j < kSub; ++j) {
                ptx::tma_load_2d_pair(sX + (st * kSub + j) * kWTile, xm, (ks * kSub + j) * kElems, x_row, lead_full);
                ptx::tma_load_2d_pair(sW + (st * kSub + j) * C::kWBytes, wm, (ks * kSub + j) * kElems, w_row, lead_full);
              }
            }
          }
          if (++st == S) {
            st = 0;
            parity ^= 1;
          }
        }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      const bool issue = ptx::elect_one();
      constexpr uint32_t idesc = F8 ? ptx::idesc_e4m3_f32(256, BN) : ptx::idesc_bf16_f32(256, BN);
      int st = 0, g = 0;  // stage; chunks over all tiles
      uint32_t parity = 0;
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t par) {
        if (__all_sync(0xffffffffu, ptx::mbar_wait(bar, par, p.wait_ns) && *abort_flag == 0)) return true;
        if (*abort_flag == 0) record(p.status, kDevTimeoutMma);
        *abort_flag = 1;
        ok = false;
        return false;
      };
      for (int tile = pair; ok && tile < tiles; tile += npairs) {
        for (int k0 = 0; ok && k0 < nk; k0 += kChunkStages, ++g) {
          const int a = g & 1;
          if (!wait(tempty_bar(a), ((g >> 1) & 1) ^ 1)) break;
          ptx::tc_fence_after();
          const uint32_t d = tmem + static_cast<uint32_t>(a * 256);
          const int n = min(kChunkStages, nk - k0);
          for (int i = 0; i < n; ++i) {
            if (!wait(full_bar(st), parity)) break;
            ptx::tc_fence_after();
            if (issue) {
#pragma unroll
              for (int j = 0; j < kSub; ++j) {
                const uint64_t xd = ptx::smem_desc_sw128(sX + (st * kSub + j) * kWTile);
                const uint64_t wd = ptx::smem_desc_sw128(sW + (st * kSub + j) * C::kWBytes);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (F8) ptx::mma_f8_pair(d, xd + 2 * k, wd + 2 * k, idesc, (i | j | k) != 0 ? 1u : 0u);
                  else ptx::mma_bf16_pair(d, xd + 2 * k, wd + 2 * k, idesc, (i | j | k) != 0 ? 1u : 0u);
                }
              }
              ptx::mma_commit_pair_multicast(empty_bar(st), 0x3);
            }
            __syncwarp();
            if (++st == S) {
              st = 0;
              parity ^= 1;
            }
          }
          if (ok && issue) ptx::mma_commit_pair_multicast(tfull_bar(a), 0x3);
        }
      }
      if (issue) {
        ptx::mma_commit_pair_multicast(drain_bar, 0x1);
        if (!ptx::mbar_wait(drain_bar, 0, p.wait_ns)) record(p.status, kDevTimeoutDrain);
      }
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    float2 *terms = terms_area + (warp - 2) * kHalf;  // this warp's own: no barrier beyond the warp
    const uint32_t lane_off = (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * kHalf);
    int g = 0;
    bool ok = true;
    for (int tile = pair; ok && tile < tiles; tile += npairs) {
      int mt, nt;
      pair_tile(p, tile, mt, nt);
      const int shard = shard_of(p, nt);
      const long long tok = static_cast<long long>(mt) * 256 + rank * 128 + q * 32 + lane;
      const int feat0 = (nt - p.shard[shard].tile0) * BN + half * kHalf;
      const long long col = p.shard[shard].col0 + feat0;
      const int n_left = p.shard[shard].n - feat0;  // columns of this warp's half that exist
      const bool row_on = tok < p.rows;
      __syncwarp();
      for (int c = lane; c < kHalf; c += 32) terms[c] = column_terms(p, col + c, c < n_left);
      __syncwarp();
      const float sx = p.x_scale && row_on ? __ldg(p.x_scale + tok) : 1.f;
      if (p.res && row_on) {  // the residual comes into L2 under the products
        const int es = p.res_f32 ? 4 : 2;
        const char *r = static_cast<const char *>(p.res) + (tok * p.res_ld + col) * es;
        for (int c = 0; c < min(kHalf, n_left) * es; c += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(r + c));
      }
      float sum[kHalf];
      for (int ch = 0; ch < chunks; ++ch, ++g) {
        const int a = g & 1;
        const bool ready = ptx::mbar_wait(tfull_bar(a), (g >> 1) & 1, p.wait_ns);
        if (!ready && lane == 0) record(p.status, kDevTimeoutEpilogue);
        ptx::tc_fence_after();
        if (!__all_sync(0xffffffffu, ready && (*abort_flag == 0))) {
          if (lane == 0) *abort_flag = 1;
          ok = false;
          break;
        }
        const uint32_t tb = tmem + static_cast<uint32_t>(a * 256) + lane_off;
#pragma unroll
        for (int c = 0; c < kHalf; c += 16) {
          uint32_t v[16];
          ptx::tmem_ld_16cols(tb + c, v);
          ptx::tmem_ld_wait();
          ptx::tmem_regs_ready(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[c + i] = ch == 0 ? __uint_as_float(v[i]) : sum[c + i] + __uint_as_float(v[i]);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(ptx::mapa_shared(tempty_bar(a), 0));
      }
      if (!ok) break;
      if (row_on) {
#pragma unroll
        for (int c = 0; c < kHalf; c += 8) {
          if (c >= n_left) break;
          float res[8], f[8];
          const bool wide = p.wide32 && n_left - c >= 8;
          if (p.res) {
            if (wide && p.res_f32) load32(static_cast<const float *>(p.res) + tok * p.res_ld + col + c, res);
            else load_row(p.res, p.res_f32, tok * p.res_ld + col + c, n_left - c, res);
          }
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float4 t = *reinterpret_cast<const float4 *>(terms + c + i);
            f[i] = sum[c + i] * (sx * t.x) + t.y;
            f[i + 1] = sum[c + i + 1] * (sx * t.z) + t.w;
          }
          activate(f, p.act, Y32);
          if (p.res) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] += res[i];
          }
          if (wide && Y32) store32(static_cast<float *>(p.y) + tok * p.y_ld + col + c, f);
          else store_row(p.y, Y32, tok * p.y_ld + col + c, n_left - c, f);
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

template <bool F8, bool ADD>
tp_status launch_split(const LinearParams &p, size_t smem, cudaStream_t s) {
  static unsigned mask = 0;
  static std::mutex mu;
  const cudaError_t e = allow_smem(k_linear_split<F8, ADD>, mask, mu);
  if (e != cudaSuccess) return cuda_fail(e);
  return launched(launch_kernel(k_linear_split<F8, ADD>, dim3(static_cast<unsigned>(p.m_tiles * p.n_tiles * p.split)),
                                dim3(kThreads), smem, s, static_cast<unsigned>(p.split), p));
}
template <bool F8, int BN, bool Y32>
tp_status launch_pair(const LinearParams &p, cudaStream_t s) {
  static unsigned mask = 0;
  static std::mutex mu;
  const cudaError_t e = allow_smem(k_linear_pair<F8, BN, Y32>, mask, mu);
  if (e != cudaSuccess) return cuda_fail(e);
  const int tiles = p.m_tiles * p.n_tiles, most = num_sms() / 2;
  return launched(launch_kernel(k_linear_pair<F8, BN, Y32>, dim3(2u * static_cast<unsigned>(tiles < most ? tiles : most)),
                                dim3(kPairThreads), PairCfg<BN>::kSmem, s, 1, p));
}
template <bool F8, bool Y32>
tp_status launch_pair_bn(const LinearParams &p, int bn, cudaStream_t s) {
  switch (bn) {
    case 128: return launch_pair<F8, 128, Y32>(p, s);
    case 160: return launch_pair<F8, 160, Y32>(p, s);
    case 192: return launch_pair<F8, 192, Y32>(p, s);
    default: return launch_pair<F8, 224, Y32>(p, s);
  }
}
template <bool F8>
tp_status launch_pair_y(const LinearParams &p, int bn, cudaStream_t s) {
  return p.y_f32 ? launch_pair_bn<F8, true>(p, bn, s) : launch_pair_bn<F8, false>(p, bn, s);
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
      p.shard[i].n = static_cast<int>(ws[i].rows);
      p.shard[i].tile0 = p.n_tiles;
      p.shard[i].col0 = col;
      p.n_tiles += static_cast<int>((ws[i].rows + tile_n - 1) / tile_n);
      col += ws[i].rows;
    }
  };
  p.rows = static_cast<int>(T);
  p.act = activation;
  p.y_f32 = y->dtype == TP_F32;
  p.res_f32 = residual && residual->dtype == TP_F32;
  p.bias_f32 = bias && bias->dtype == TP_F32;
  // every f32 row and first column on 32 bytes
  p.wide32 = 1;
  for (const tp_tensor *t : {static_cast<const tp_tensor *>(y), residual})
    if (t && t->dtype == TP_F32) p.wide32 = p.wide32 && ptr_aligned(t->ptr, 32) && t->ld % 8 == 0;
  for (int i = 0; !row && i + 1 < parts; ++i) p.wide32 = p.wide32 && ws[i].rows % 8 == 0;
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

  // The pair kernel from a quarter wave of its tiles on; below that the split kernel's
  // smaller tiles and its split of K put more SMs to work.
  const long long m256 = (T + 255) / 256;
  lay_out(256);
  const bool pair = T > 128 && m256 * p.n_tiles >= num_sms() / 4;
  bool add = false;
  int x_box = 128, w_box = 128, bn = 224;
  if (pair) {
    // The tile width whose last wave wastes least: the busiest pair's columns,
    // the wider tile (fewer bytes loaded per product) where two are equal.
    long long best = -1;
    for (int w = 224; w >= 128; w -= 32) {
      lay_out(w);
      const long long tiles = m256 * p.n_tiles, pairs = num_sms() / 2;
      const long long cost = (tiles + pairs - 1) / pairs * w;
      if (best < 0 || cost < best) {
        best = cost;
        bn = w;
      }
    }
    lay_out(bn);
    w_box = bn / 2;
    p.m_tiles = static_cast<int>(m256);
    if (m256 * p.n_tiles > 0x7fffffffLL) return TP_ERR_UNSUPPORTED;
  } else {
    lay_out(128);
    p.m_tiles = static_cast<int>(m256);
    const long long per = (T + p.m_tiles - 1) / p.m_tiles;
    p.tok_tile = static_cast<int>((per + 15) / 16 * 16);
    x_box = p.tok_tile;
    // Half of an SM's shared memory, so that two CTAs share it (the next kernel's first
    // weights load beside this one's end): six stages for 16 tokens, four for 64, three
    // from 81 to 128; beyond 128 tokens all of it. At 61 tokens, 4096 -> 14336 in e4m3: 15.9 us with two
    // CTAs an SM of 110 KB, 16.5 with one of 222 KB, 18.7 with three of 72 KB.
    const int stage = kWTile + p.tok_tile * 128;
    const bool two = p.tok_tile <= 128;
    p.stages = ((two ? 110 : 222) * 1024 - 2048) / stage;
    // the largest cluster that leaves every CTA its place, with at least two k-tiles a CTA
    const long long tiles = static_cast<long long>(p.m_tiles) * p.n_tiles, per_sm = two ? 2 : 1;
    p.split = 1;
    for (int c = 2; c <= 8; ++c)
      if (tiles * c <= num_sms() * per_sm && tiles <= max_active_clusters(c) * per_sm && p.kt_total >= 2 * c) p.split = c;
    if (tiles * p.split > 0x7fffffffLL) return TP_ERR_UNSUPPORTED;
    // Accumulators of kChunkSteps steps each, a power of two of them for TMEM's allocation, in
    // the columns that a CTA has (half of the SM's where two share it); where they do not
    // suffice, as many as those columns hold, and chunks are added under the products.
    const int most = two ? 256 : 512;
    p.region_cols = 32;
    while (p.region_cols < p.tok_tile) p.region_cols *= 2;
    const int steps = (p.kt_total + p.split - 1) / p.split * 4;
    p.regions = 1;
    while (p.regions * kChunkSteps < steps && 2 * p.regions * p.region_cols <= most) p.regions *= 2;
    p.tmem_cols = p.regions * p.region_cols;
    add = p.regions * kChunkSteps < steps;
    if (add) {
      p.region_cols = (p.tok_tile + 31) / 32 * 32;
      p.regions = most / p.region_cols < kMaxRegions ? most / p.region_cols : kMaxRegions;
      p.tmem_cols = most;
    }
  }
  // A copy costs its issue whatever its size, so where every slice is whole k-tiles one
  // box spans a stage's k-tiles (2048 x 4096 x 8192 in e4m3: 56.1 us, 57.8 with one copy
  // a k-tile; k_linear_split, whose weights come at memory's rate, gains nothing).
  p.box3 = pair;
  for (int i = 0; i < p.n_slices; ++i) p.box3 = p.box3 && xs[i].cols % elems == 0;
  auto encode = [&](CUtensorMap *m, const tp_tensor &t, int rows) {
    return p.box3 ? encode_rows_map_3d(m, t, rows, kSub) : encode_rows_map(m, t, rows);
  };
  for (int i = 0; i < p.n_slices; ++i)
    if (!encode(&p.x[i], xs[i], x_box)) return TP_ERR_INVALID_ARG;
  for (int i = 0; i < parts; ++i)
    if (!encode(&p.w[i], ws[i], w_box)) return TP_ERR_INVALID_ARG;
  if (pair) return dt == TP_E4M3 ? launch_pair_y<true>(p, bn, s) : launch_pair_y<false>(p, bn, s);
  size_t smem = 1024 + static_cast<size_t>(p.stages) * (kWTile + p.tok_tile * 128);
  const size_t out = 1024 + static_cast<size_t>(p.tok_tile) * 512;  // the partials lie over the stages
  smem = (smem > out ? smem : out) + 8 * (2 * p.stages + 2 + 2 * kMaxRegions) + p.tok_tile * 4 + 64;
  if (add) return dt == TP_E4M3 ? launch_split<true, true>(p, smem, s) : launch_split<false, true>(p, smem, s);
  return dt == TP_E4M3 ? launch_split<true, false>(p, smem, s) : launch_split<false, false>(p, smem, s);
}
