// Attention of one new token per sequence over a prefix that the whole batch
// shares and each sequence's own cache, with GQA:
//   A[b, h] = softmax([q K_prefix^T, q K_own(b)^T] / sqrt(d)) [V_prefix ; V_own(b)]
// and, on request, every own key's softmax weight summed over its q heads and
// added to its accumulated weight.
//
// Every query row of a kv head (B sequences x G heads of its group) sees the same
// prefix, so the prefix part is one dense product of B*G rows against P keys and
// K/V are read once, not B times: k_prefix_part runs it on the tensor cores
// (tcgen05) in tiles of 128 rows, split over the keys where there are too few
// rows to fill the SMs. The own part differs per sequence and is bound by reading
// the cache: k_own_part streams it through shared memory (cp.async) into
// m16n8k16 products whose 16 rows are the group's heads; P stays in registers.
// Both leave unnormalised f32 sums with their reference maximum m and sum l per
// (split, row); k_combine joins them: sum of 2^(m_s - M) O_s over sum of
// 2^(m_s - M) l_s, which is the softmax over all keys, whatever the split. No m is below
// f32's lowest value: with it in place of -inf, keys that score -inf (and masked ones) get
// weight 0 where no other has been seen yet, and what is seen later moves m as usual.
//
// The two parts bound different things, so they run at the same time: k_prefix_part
// leaves some SMs free, and k_own_part, which shares nothing with it, does not wait
// for it: it starts on those SMs, goes on where that kernel's CTAs leave, and waits
// for it only in its last CTA, so that what follows it on the stream follows both.
// Its inputs were written before k_prefix_part, whose every CTA has waited for what is
// before it on the stream when the first CTA of k_own_part starts: they are in L2, and
// what reads them without a wait of its own (k_own_part, and k_combine the lengths)
// reads them there, past L1 (61 sequences: 33.1 us, 32.4 through L1).
//
// Few keys and sequences, where three launches cost more than the work, take one:
// k_direct.
#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>

#include "op_util.h"
#include "sm100_ptx.cuh"

namespace tpgqa {
namespace {

using namespace op;

constexpr int kMaxRanks32 = 32;
constexpr int kSms = 152;  // a GB300's; splits and workspace sizes follow it, not the device at hand

// The scalars come first and lie together: a kernel's first read of each 64-byte
// line of its parameters is a miss of a few hundred nanoseconds.
struct PrefixAttnParams {
  int batch, heads_q, heads_kv, group, heads_per_rank, heads_per_source, d;
  int prefix, blocks, split_p, pairs, ctas_p;  // 128-key blocks; key splits; 256-row tile pairs per kv head; CTAs
  int cap, chunk, split_o;             // own cache: rows a sequence, keys a split, splits
  int score_ld;                        // floats of a row of scores: a multiple of four
  int has_prev;                        // k_own_part runs behind k_prefix_part
  int direct;                          // above 0: k_direct runs instead, with this many CTAs a cluster
  int one_prefix;                      // every source's prefix lies in one tensor, in head order: one map of each
  float scale_log2;
  const int *lengths;
  float *part_o;    // [split][row][d]
  float2 *part_ml;  // [split][row] (m in log2 units, l)
  float *scores;    // [row][score_ld], s * log2(e) / sqrt(d) of the own keys; null: not wanted
  int *status;
  long long wait_ns;
  const void *q[kMaxRanks32];
  long long q_ld[kMaxRanks32];
  const void *k_own[kMaxRanks32], *v_own[kMaxRanks32];
  long long ko_ld[kMaxRanks32], vo_ld[kMaxRanks32];
  const void *k_prefix[kMaxRanks32], *v_prefix[kMaxRanks32];
  long long kp_ld[kMaxRanks32], vp_ld[kMaxRanks32];
  void *a[kMaxRanks32];
  long long a_ld[kMaxRanks32];
  const float *w_in[kMaxRanks32];
  float *w_out[kMaxRanks32];
  long long wi_ld[kMaxRanks32], wo_ld[kMaxRanks32];
};
struct PrefixMaps {
  CUtensorMap k[kMaxRanks32], v[kMaxRanks32];  // prefix K and V of each kv source
};

// q row (or output row) of sequence b, global q head h.
__device__ __forceinline__ const __nv_bfloat16 *q_row(const PrefixAttnParams &p, int b, int h) {
  const int r = h / p.heads_per_rank;
  return static_cast<const __nv_bfloat16 *>(p.q[r]) + b * p.q_ld[r] + static_cast<long long>(h - r * p.heads_per_rank) * p.d;
}
// Row of the partial results: the rows of a kv head are neighbours.
__device__ __forceinline__ long long part_row(const PrefixAttnParams &p, int kv, int b, int g) {
  return (static_cast<long long>(kv) * p.batch + b) * p.group + g;
}
__device__ __forceinline__ int own_length(const PrefixAttnParams &p, int b) {
  return min(max(__ldcg(p.lengths + b), 0), p.cap);
}

// ---------------------------------------------------------------------------
// The shared prefix. A work item is (kv head, pair of adjacent 128-row tiles, key
// split); both tiles use every K and V tile that is loaded. Warp roles:
//   warp 0     TMA: lane 0 the K ring, lane 1 the V ring (two 128-key stages each);
//   warp 1     MMA issuer: S_A, S_B, P_A V, S_A of the next block, P_B V, ...;
//   warps 2-5  softmax of tile A, 6-9 of tile B, one thread per row; each thread
//              also gathers its own q row into the swizzled Q tile (a group's
//              heads may lie on several ranks, so no one tensor map covers them).
// TMEM: S of A at columns 0, of B at 128 (P overwrites its first half as bf16, the type
// of the product with V, and is read from there; with the bf16 output's own rounding that
// makes an error of 2.3e-3 of the output, against 1.7e-3 from the latter alone), O at 256
// and 384. V is used as it lies, [keys x d], as an
// MN-major operand, so no transposed copy is made. The running reference maximum
// m moves only on a split's first block or when a block's sum of p passes 2^64.
// A block step of both tiles takes 1.6 us (the MMAs alone 1.1): its period is the chain
// S, softmax, P V of the two tiles. With the MMAs issued under a branch on the lane
// index, which holds operands outside the uniform registers, it took 0.2
// us more. Halving the chain costs more than it hides: products of P's halves 0.2 us, S
// by halves of 64 keys too (four chains) 0.5. P stored 16 keys at a time in place of
// 32, for the registers, is worth 3%; columns loaded under the exponentials of those
// before cost 10% (spills). An item's start and end move q and O between rows
// and threads through shared memory (61 sequences, 4099 keys: 28.9 -> 26.1 us a call).
// ---------------------------------------------------------------------------
constexpr int kPrefThreads = 320;
constexpr uint32_t kSubTile = 128u * 128u;  // [128 rows x 64 bf16], swizzled
constexpr float kSumLimit = 0x1p64f;

__device__ __forceinline__ void st_shared(uint32_t at, const uint4 &v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <int D>
struct PrefCfg {
  static constexpr int kCh = D / 64;                      // 64-column sub-tiles of a head
  static constexpr uint32_t kTile = kCh * kSubTile;       // a [128 x D] tile
  static constexpr uint32_t kK = 2 * kTile, kV = 4 * kTile, kBar = 6 * kTile;
  static constexpr size_t kSmem = kBar + 256 + 1024;
};

template <int D>
__global__ void __launch_bounds__(kPrefThreads, 1) k_prefix_part(const __grid_constant__ PrefixAttnParams p, const __grid_constant__ PrefixMaps maps) {
  using C = PrefCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = ptx::smem_addr(smem), sK0 = sQ + C::kK, sV0 = sQ + C::kV;
  uint8_t *bar_area = smem + C::kBar;
  const uint32_t bar0 = ptx::smem_addr(bar_area);
  const uint32_t q_full0 = bar0, k_full0 = bar0 + 16, k_empty0 = bar0 + 32, v_full0 = bar0 + 48, v_empty0 = bar0 + 64,
                 s_full0 = bar0 + 80, p_full0 = bar0 + 96, o_full0 = bar0 + 112, o_free0 = bar0 + 128, drain = bar0 + 144;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bar_area + 152);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bar_area + 156);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.batch * p.group;
  const int items = p.heads_kv * p.pairs * p.split_p;
  // item -> (kv head, tile pair, split, its blocks); splits of one head are neighbours
  auto item = [&](int it, int &kv, int &pair, int &split, int &b0, int &b1) {
    split = it % p.split_p;
    const int r = it / p.split_p;
    pair = r % p.pairs;
    kv = r / p.pairs;
    b0 = static_cast<int>(static_cast<long long>(p.blocks) * split / p.split_p);
    b1 = static_cast<int>(static_cast<long long>(p.blocks) * (split + 1) / p.split_p);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(q_full0 + 8 * s, 128);
      ptx::mbar_init(k_full0 + 8 * s, 1);
      ptx::mbar_init(k_empty0 + 8 * s, 1);
      ptx::mbar_init(v_full0 + 8 * s, 1);
      ptx::mbar_init(v_empty0 + 8 * s, 1);
      ptx::mbar_init(s_full0 + 8 * s, 1);
      ptx::mbar_init(p_full0 + 8 * s, 4);
      ptx::mbar_init(o_full0 + 8 * s, 1);
      ptx::mbar_init(o_free0 + 8 * s, 128);
    }
    ptx::mbar_init(drain, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t *>(tmem_slot)), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  int issued[2] = {0, 0};
  if (warp == 0) {
    if (lane < 2) {
      const uint32_t full0 = lane == 0 ? k_full0 : v_full0, empty0 = lane == 0 ? k_empty0 : v_empty0;
      const uint32_t dst0 = lane == 0 ? sK0 : sV0;
      bool run = true;
      int g = 0;
      for (int it = blockIdx.x; run && it < items; it += gridDim.x) {
        int kv, pair, split, b0, b1;
        item(it, kv, pair, split, b0, b1);
        const int src = p.one_prefix ? 0 : kv / p.heads_per_source;
        const int col = (kv - src * p.heads_per_source) * D;
        const CUtensorMap *map = lane == 0 ? &maps.k[src] : &maps.v[src];
        for (int j = b0; j < b1; ++j, ++g) {
          const int s = g & 1;
          if (*abort_flag || !ptx::mbar_wait(empty0 + 8 * s, ((g >> 1) & 1) ^ 1, p.wait_ns)) {
            if (!*abort_flag) record(p.status, kDevTimeoutProducer);
            *abort_flag = 1;
            run = false;
            break;
          }
          ptx::mbar_arrive_expect_tx(full0 + 8 * s, C::kTile);
          for (int c = 0; c < C::kCh; ++c)
            ptx::tma_load_2d(dst0 + s * C::kTile + c * kSubTile, map, col + c * 64, j * 128, full0 + 8 * s);
          ++issued[s];
        }
      }
    }
  } else if (warp == 1) {  // converged; one lane issues (see elect_one)
    constexpr uint32_t idesc_s = ptx::idesc_bf16_f32(128, 128);
    constexpr uint32_t idesc_o = ptx::idesc_bf16_f32(128, D) | ptx::kIdescBMn;
    const bool leader = ptx::elect_one();
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (__all_sync(0xffffffffu, ptx::mbar_wait(bar, parity, p.wait_ns))) return true;  // an abort elsewhere ends in a timeout here
      if (*abort_flag == 0) record(p.status, kDevTimeoutMma);
      ok = false;
      return false;
    };
    auto commit = [&](uint32_t bar) {
      if (leader) ptx::mma_commit(bar);
      __syncwarp();
    };
    auto issue_s = [&](int x, int g) {  // S_X = Q_X K^T
      const uint32_t qa = sQ + static_cast<uint32_t>(x) * C::kTile, ka = sK0 + static_cast<uint32_t>(g & 1) * C::kTile;
      const uint32_t d = tmem + static_cast<uint32_t>(x * 128);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          ptx::mma_bf16(d, ptx::smem_desc_sw128(qa + (kk >> 2) * kSubTile) + 2 * (kk & 3),
                        ptx::smem_desc_sw128(ka + (kk >> 2) * kSubTile) + 2 * (kk & 3), idesc_s, kk > 0 ? 1u : 0u);
        ptx::mma_commit(s_full0 + 8 * x);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int x, int g, bool first) {  // O_X += P_X V, 16 keys (2048 bytes of V) a step
      const uint32_t va = sV0 + static_cast<uint32_t>(g & 1) * C::kTile;
      const uint32_t d = tmem + 256u + static_cast<uint32_t>(x * 128), a = tmem + static_cast<uint32_t>(x * 128);
      const uint32_t more = first ? 0u : 1u;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          ptx::mma_bf16_ts(d, a + 8u * kk, ptx::smem_desc_mn_sw128(va + kk * 2048u, kSubTile), idesc_o, kk > 0 ? 1u : more);
      }
      __syncwarp();
    };
    int g = 0;
    uint32_t np[2] = {0, 0}, nact[2] = {0, 0};
    for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
      int kv, pair, split, b0, b1;
      item(it, kv, pair, split, b0, b1);
      const int nb = b1 - b0;
      const int tiles = (2 * pair + 1) * 128 < rows ? 2 : 1;
      if (!wait(k_full0 + 8 * (g & 1), (g >> 1) & 1)) break;
      for (int x = 0; ok && x < tiles; ++x) {
        if (!wait(q_full0 + 8 * x, nact[x] & 1)) break;
        ptx::tc_fence_after();
        issue_s(x, g);
      }
      if (!ok) break;
      commit(k_empty0 + 8 * (g & 1));
      for (int j = 0; ok && j < nb; ++j) {
        const int gj = g + j;
        const bool last = j + 1 == nb;
        if (!wait(v_full0 + 8 * (gj & 1), (gj >> 1) & 1)) break;
        if (!last && !wait(k_full0 + 8 * ((gj + 1) & 1), ((gj + 1) >> 1) & 1)) break;
        for (int x = 0; ok && x < tiles; ++x) {
          if (!wait(p_full0 + 8 * x, np[x] & 1)) break;
          ++np[x];
          if (j == 0 && !wait(o_free0 + 8 * x, (nact[x] & 1) ^ 1)) break;
          ptx::tc_fence_after();
          issue_pv(x, gj, j == 0);
          if (last) commit(o_full0 + 8 * x);
          else issue_s(x, gj + 1);
        }
        if (!ok) break;
        commit(v_empty0 + 8 * (gj & 1));
        if (!last) commit(k_empty0 + 8 * ((gj + 1) & 1));
      }
      for (int x = 0; x < tiles; ++x) ++nact[x];
      g += nb;
    }
    if (!ok) *abort_flag = 1;
    if (leader) {
      ptx::mma_commit(drain);
      if (!ptx::mbar_wait(drain, 0, p.wait_ns)) record(p.status, kDevTimeoutDrain);
    }
    __syncwarp();
  } else {
    const int x = (warp - 2) >> 2;
    const int qw = warp & 3;
    const int row = qw * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(qw * 32) << 16;
    const uint32_t sb = tmem + lane_off + static_cast<uint32_t>(x * 128);
    const uint32_t ob = tmem + lane_off + 256u + static_cast<uint32_t>(x * 128);
    const uint32_t s_full = s_full0 + 8 * x, p_full = p_full0 + 8 * x;
    const uint32_t warp_q = sQ + static_cast<uint32_t>(x) * C::kTile + static_cast<uint32_t>(qw) * 4096u;  // its 32 rows
    bool ok = true;
    auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
      const bool ready = ptx::mbar_wait(bar, parity, p.wait_ns);
      if (__all_sync(0xffffffffu, ready)) return true;  // an abort elsewhere ends in a timeout here
      if (lane == 0) {
        if (*abort_flag == 0) record(p.status, kDevTimeoutEpilogue);
        *abort_flag = 1;
      }
      return false;
    };
    uint32_t gs = 0, nact = 0;
    for (int it = blockIdx.x; ok && it < items; it += gridDim.x) {
      int kv, pair, split, b0, b1;
      item(it, kv, pair, split, b0, b1);
      const int nb = b1 - b0;
      const int m_row = (2 * pair + x) * 128 + row;  // row of the kv head: sequence * group + head
      if ((2 * pair + x) * 128 >= rows) continue;
      // the warp's q rows into the Q tile, a row's 16-byte pieces by neighbouring lanes; the
      // previous item's products have read it (its o_full was waited for)
      {
        constexpr int kPieces = D / 8;
        const int b = m_row < rows ? m_row / p.group : 0, gq = m_row < rows ? m_row - b * p.group : 0;
        const unsigned long long mine = m_row < rows ? reinterpret_cast<unsigned long long>(q_row(p, b, kv * p.group + gq)) : 0;
        const int c = lane % kPieces;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
          const int r = i * (32 / kPieces) + lane / kPieces;
          const uint4 *src = reinterpret_cast<const uint4 *>(__shfl_sync(0xffffffffu, mine, r));
          const uint4 v = src ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          st_shared(warp_q + (c >> 3) * kSubTile + r * 128 + ((c & 7) ^ (r & 7)) * 16, v);
        }
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(q_full0 + 8 * x);
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < nb; ++j, ++gs) {
        if (!wait_all(s_full, gs & 1)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const int lim = p.prefix - (b0 + j) * 128;  // keys of the block that exist
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          ptx::tmem_ld_16cols(sb + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&v[16 * c]));
        ptx::tmem_ld_wait();
        ptx::tmem_regs_ready(v);
        if (lim < 128) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= lim) v[i] = __float_as_uint(-INFINITY);
        }
        const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
        bool find_max = j == 0, move = false;
        float m_new = m, s0, s1;
#pragma unroll 1
        for (;;) {
          if (find_max) {
            float mq[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              mq[q] = __uint_as_float(v[32 * q + 31]);
#pragma unroll
              for (int i = 0; i < 30; i += 2)
                mq[q] = max3(mq[q], __uint_as_float(v[32 * q + i]), __uint_as_float(v[32 * q + i + 1]));
              mq[q] = fmaxf(mq[q], __uint_as_float(v[32 * q + 30]));
            }
            const float m_blk = fmaxf(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])) * p.scale_log2, -FLT_MAX);
            move = m_blk > m + 8.f;
            m_new = move ? m_blk : m;
          }
          const uint64_t nm2 = pack2(-m_new, -m_new);
          uint64_t sumh[4];
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint64_t &sum2 = sumh[h];
            sum2 = pack2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 32; e += 16) {  // P leaves in pieces of 16 keys: v holds most registers
              uint32_t pk[8];
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const int k = 32 * h + e + i;
                float y0, y1;
                unpack2(fma2(pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2, nm2), y0, y1);
                const float a0 = ex2(y0), a1 = ex2(y1);
                sum2 = add2(sum2, pack2(a0, a1));
                pk[i >> 1] = pack_bf16(a0, a1);
              }
              ptx::tmem_st_8cols(sb + 16 * h + e / 2, pk);
            }
          }
          unpack2(add2(add2(sumh[0], sumh[1]), add2(sumh[2], sumh[3])), s0, s1);
          if (find_max || !__any_sync(0xffffffffu, !(s0 + s1 <= kSumLimit))) break;
          find_max = true;
          ptx::tmem_st_wait();
        }
        const float alpha = move ? exp2f(m - m_new) : 1.f;
        m = m_new;
        if (find_max && j > 0 && __any_sync(0xffffffffu, move)) {
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            ptx::tmem_ld_32cols(ob + c * 32, o);
            ptx::tmem_ld_wait();
            ptx::tmem_regs_ready(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            ptx::tmem_st_32cols(ob + c * 32, o);
          }
        }
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full);
        l += s0 + s1;
      }
      if (!ok) break;
      if (!wait_all(o_full0 + 8 * x, nact & 1)) {
        ok = false;
        break;
      }
      ++nact;
      ptx::tc_fence_after();
      const long long at = static_cast<long long>(split) * p.batch * p.heads_q + static_cast<long long>(kv) * rows + m_row;
      if (m_row < rows) p.part_ml[at] = make_float2(m, l);
      // out by rows of 128 bytes, turned in the warp's part of the Q tile, which nothing
      // reads any more: a lane that stores its own row touches 32 lines an instruction
      const int there = rows - (m_row - lane);  // of the warp's rows
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        ptx::tmem_ld_32cols(ob + c * 32, v);
        ptx::tmem_ld_wait();
        ptx::tmem_regs_ready(v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared(warp_q + lane * 128 + (i ^ (lane & 7)) * 16, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3), q = lane & 7;
          const uint4 w = ld_shared(warp_q + r * 128 + (q ^ (r & 7)) * 16);
          if (r < there) *reinterpret_cast<uint4 *>(p.part_o + (at - lane + r) * D + c * 32 + q * 4) = w;
        }
        __syncwarp();
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(o_free0 + 8 * x);
    }
  }

  __syncthreads();
  if (warp == 0 && lane < 2) {
    const uint32_t full0 = lane == 0 ? k_full0 : v_full0;
    for (int s = 0; s < 2; ++s)
      if (issued[s] > 0 && !ptx::mbar_wait(full0 + 8 * s, (issued[s] - 1) & 1, p.wait_ns)) record(p.status, kDevTimeoutDrain);
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// The own caches. CTA (sequence and kv head, key split, 16-head tile). The four
// warps walk by themselves, 32 keys a step, each through its own ring of three slots (K
// of the step, V of the step, K of the next), and keep their own m, l and O, which
// are joined at the end. Keys past the length are zero-filled in shared memory,
// never read from the cache (stale values there may be anything), and masked.
// Bound by memory on all SMs (268 MB in 45 us, 6 TB/s) and by latency on the SMs that
// the prefix part leaves: a step's chain (85 KB/us an SM with two CTAs of 1000
// keys), a CTA's start and join (44 KB/us with 256 keys). Measured and slower: stages
// of 64 keys shared by the warps, 16 a warp (62 KB/us; 61 sequences 36.1 us in place
// of 33.4: twice the shuffles and dependent products a key, and a barrier); rings of
// 16 keys (35.6); three CTAs an SM with two shared stages (33.9, but 90 in place of 85
// for 128 sequences of 1025 keys: too little in flight); eight warps that share
// a step's maximum and P and own output columns (three barriers a step, 23 KB/us); runs
// of steps across sequences in place of a CTA a split (no better balance than the
// scheduler's, and a join and a q load in the run).
// ---------------------------------------------------------------------------
constexpr int kOwnThreads = 128;
constexpr int kOwnKeys = 64;   // keys of a k_direct tile; an own split is a multiple of it
constexpr int kWarpKeys = 32;  // keys of a warp's step in k_own_part

// A warp's ring: three slots of kWarpKeys keys' K or V.
template <int D>
struct OwnCfg {
  static constexpr int kSlot = kWarpKeys * D * 2;
  static constexpr int kRing = 3 * kSlot;
  static constexpr int kSmem = 4 * kRing;
  static_assert(kRing >= 16 * D * 4, "a warp's outputs fit over its ring");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One warp's share of a head tile: the q rows as the A operand (rows lane/4 and lane/4
// + 8), the outputs over all of D, and the rows' running maximum and sum.
template <int D>
struct WarpRows {
  uint32_t qa[D / 16][4];
  float o[D / 8][4];
  float m[2], l[2];

  __device__ __forceinline__ void start(const PrefixAttnParams &p, int b, int kv, int g0) {
    const int lane = threadIdx.x & 31, r_lo = g0 + (lane >> 2), r_hi = r_lo + 8;
    const uint32_t *q_lo = r_lo < p.group ? reinterpret_cast<const uint32_t *>(q_row(p, b, kv * p.group + r_lo)) : nullptr;
    const uint32_t *q_hi = r_hi < p.group ? reinterpret_cast<const uint32_t *>(q_row(p, b, kv * p.group + r_hi)) : nullptr;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const int at = kk * 8 + (lane & 3);
      qa[kk][0] = q_lo ? __ldcg(q_lo + at) : 0u;
      qa[kk][1] = q_hi ? __ldcg(q_hi + at) : 0u;
      qa[kk][2] = q_lo ? __ldcg(q_lo + at + 4) : 0u;
      qa[kk][3] = q_hi ? __ldcg(q_hi + at + 4) : 0u;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    m[0] = m[1] = -FLT_MAX;
    l[0] = l[1] = 0.f;
  }

  // Scores of the KEYS keys at shared-memory rows row0 .., in log2 units; keys from the
  // `left`-th on are masked. s[n][0,1]: row lane/4, keys 8n + 2 (lane%4) + {0, 1};
  // s[n][2,3]: row lane/4 + 8.
  template <int KEYS>
  __device__ __forceinline__ void scores(uint32_t ks, int row0, int left, float scale_log2, float (&s)[KEYS / 8][4]) const {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int n = 0; n < KEYS / 8; n += 2) {
        const int r = row0 + n * 8 + ((lane >> 4) << 3) + (lane & 7), c = 2 * kk + ((lane >> 3) & 1);
        uint32_t kb[4];
        ldsm4(ks + static_cast<uint32_t>(r * D * 2 + (c ^ (r & 7)) * 16), kb);
        mma16816(s[n], qa[kk], kb[0], kb[1]);
        mma16816(s[n + 1], qa[kk], kb[2], kb[3]);
      }
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[n][i] = 8 * n + 2 * (lane & 3) + (i & 1) < left ? s[n][i] * scale_log2 : -INFINITY;
  }

  // Turns scores into softmax terms p, rescaling what came before; at least one key is there.
  template <int KEYS>
  __device__ __forceinline__ void softmax(float (&s)[KEYS / 8][4]) {
    float alpha[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(s[0][2 * h], s[0][2 * h + 1]);
#pragma unroll
      for (int n = 1; n < KEYS / 8; ++n) mx = fmaxf(mx, fmaxf(s[n][2 * h], s[n][2 * h + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m[h], mx);
      alpha[h] = m[h] == m_new ? 1.f : ex2(m[h] - m_new);
      l[h] *= alpha[h];
      m[h] = m_new;
    }
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= alpha[0];
        o[i][1] *= alpha[0];
        o[i][2] *= alpha[1];
        o[i][3] *= alpha[1];
      }
    }
#pragma unroll
    for (int n = 0; n < KEYS / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[n][i] = ex2(s[n][i] - m[i >> 1]);
        l[i >> 1] += s[n][i];
      }
  }

  // Adds p V. P is rounded to bf16 for the product, as every GEMM operand here; l sums the
  // unrounded p.
  template <int KEYS>
  __device__ __forceinline__ void add_pv(uint32_t vs, int row0, const float (&s)[KEYS / 8][4]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 0; n < KEYS / 8; n += 2) {
      const uint32_t pa[4] = {pack_bf16(s[n][0], s[n][1]), pack_bf16(s[n][2], s[n][3]), pack_bf16(s[n + 1][0], s[n + 1][1]),
                              pack_bf16(s[n + 1][2], s[n + 1][3])};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const int r = row0 + n * 8 + ((lane >> 3) & 1) * 8 + (lane & 7), c = 2 * i + (lane >> 4);
        uint32_t vb[4];
        ldsm4_t(vs + static_cast<uint32_t>(r * D * 2 + (c ^ (r & 7)) * 16), vb);
        mma16816(o[2 * i], pa, vb[0], vb[1]);
        mma16816(o[2 * i + 1], pa, vb[2], vb[3]);
      }
    }
  }

  // Puts the warp's m and l into ml[16] and its outputs into so[16][D].
  __device__ __forceinline__ void put(float2 *ml, float *so) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      const int r = (lane >> 2) + 8 * h;
      if ((lane & 3) == 0) ml[r] = make_float2(m[h], l[h]);
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2 *>(so + r * D + i * 8 + 2 * (lane & 3)) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
    }
  }
};
// Four columns of a row over the CTA's four warps (`stride` floats apart): their common
// maximum, sum and outputs. A warp without keys has zeros, and a factor of 0 still multiplies: a warp
// whose only scores are no numbers has the lowest maximum (fmaxf passes over them) and such a sum.
template <int D>
__device__ __forceinline__ float4 join_warps(const float2 (*s_ml)[16], const float *so, int stride, int r, int c, float2 &ml) {
  float top = -INFINITY;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, s_ml[w][r].x);
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float f = ex2(s_ml[w][r].x - top);
    const float4 ov = *reinterpret_cast<const float4 *>(so + w * stride + r * D + c);
    sum += f * s_ml[w][r].y;
    acc.x += f * ov.x;
    acc.y += f * ov.y;
    acc.z += f * ov.z;
    acc.w += f * ov.w;
  }
  ml = make_float2(top, sum);
  return acc;
}
// A thread's walk over 64-key tiles of a cache: 16-byte pieces of rows r0, r0 + kRows,
// ... of K and V into a stage, zeros past the last key.
template <int D>
struct TileLoader {
  static constexpr int kPieces = D / 8;                // 16-byte pieces of a row
  static constexpr int kRows = kOwnThreads / kPieces;  // rows that the CTA loads at a time: 8 or 16
  const char *k, *v;
  long long k_step, v_step;  // bytes of kRows rows
  int left;                  // keys from this thread's next row on
  uint32_t to0;              // its place in a stage (rows kRows apart share the swizzle)

  // `row` is the first key's row; `keys` follow.
  __device__ __forceinline__ void start(const void *kc, long long k_ld, const void *vc, long long v_ld, long long col,
                                        long long row, int keys) {
    const int c0 = threadIdx.x % kPieces, r0 = threadIdx.x / kPieces;
    k = reinterpret_cast<const char *>(static_cast<const __nv_bfloat16 *>(kc) + (row + r0) * k_ld + col + c0 * 8);
    v = reinterpret_cast<const char *>(static_cast<const __nv_bfloat16 *>(vc) + (row + r0) * v_ld + col + c0 * 8);
    k_step = kRows * k_ld * 2;
    v_step = kRows * v_ld * 2;
    left = keys - r0;
    to0 = static_cast<uint32_t>(r0 * D * 2 + (c0 ^ (r0 & 7)) * 16);
  }
  // safe: any readable address, for the copies that read nothing.
  __device__ __forceinline__ void tile(uint32_t stage, const void *safe) {
    const uint32_t to = stage + to0;
#pragma unroll
    for (int i = 0; i < kOwnKeys / kRows; ++i) {
      const bool valid = left > 0;
      cp_async16(to + i * kRows * D * 2, valid ? static_cast<const void *>(k) : safe, valid);
      cp_async16(to + kOwnKeys * D * 2 + i * kRows * D * 2, valid ? static_cast<const void *>(v) : safe, valid);
      k += k_step;
      v += v_step;
      left -= kRows;
    }
  }
};
// A warp's walk down one matrix of a cache, kWarpKeys of every 4 kWarpKeys keys: copies
// into a slot, zeros past the last key.
template <int D>
struct KeyWalk {
  static constexpr int kPieces = D / 8;        // 16-byte pieces of a row
  static constexpr int kRows = 32 / kPieces;   // rows that a warp copies at a time: 2 or 4
  const char *at;
  long long step;  // bytes of kRows rows
  int left;        // keys from this lane's next row on
  uint32_t to0;    // the lane's place in a slot, of its first row

  // `row` is the warp's first row; `keys` follow it, others' among them.
  __device__ __forceinline__ void start(const void *cache, long long ld, long long col, long long row, int keys) {
    const int lane = threadIdx.x & 31, c0 = lane % kPieces, r0 = lane / kPieces;
    at = reinterpret_cast<const char *>(static_cast<const __nv_bfloat16 *>(cache) + (row + r0) * ld + col + c0 * 8);
    step = kRows * ld * 2;
    left = keys - r0;
    to0 = static_cast<uint32_t>(r0 * D * 2 + (c0 ^ r0) * 16);
  }
  // safe: any readable address, for the copies that read nothing.
  __device__ __forceinline__ void load(uint32_t slot, const void *safe) {
#pragma unroll
    for (int i = 0; i < kWarpKeys / kRows; ++i) {
      const bool valid = left > i * kRows;
      // row r0 + i kRows: r0 < kRows, a power of two, so its swizzle is r0's with the bits of i kRows flipped
      cp_async16(slot + (to0 ^ (((i * kRows) & 7) << 4)) + i * kRows * D * 2, valid ? static_cast<const void *>(at) : safe,
                 valid);
      at += step;
    }
    at += step * (3 * kWarpKeys / kRows);
    left -= 4 * kWarpKeys;
  }
};
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kOwnThreads, 2) k_own_part(const __grid_constant__ PrefixAttnParams p) {
  using C = OwnCfg<D>;
  extern __shared__ __align__(128) uint8_t own_smem[];
  __shared__ float2 s_ml[4][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kv = blockIdx.x % p.heads_kv, b = blockIdx.x / p.heads_kv;
  const int split = blockIdx.y, g0 = blockIdx.z * 16;
  if (!p.has_prev) grid_dep_wait();
  grid_dep_launch();
  const int len = own_length(p, b);
  if (kv == 0 && split == 0 && g0 == 0 && tid == 0 && len != __ldcg(p.lengths + b)) atomicCAS(p.status, 0, kDevBadLength);
  const int j0 = split * p.chunk, j1 = min(len, j0 + p.chunk);
  if (j0 < j1) {
    const int src = kv / p.heads_per_source;
    const long long col = static_cast<long long>(kv - src * p.heads_per_source) * D;
    const uint32_t sbase = ptx::smem_addr(own_smem);
    const int mine = j1 - j0 - warp * kWarpKeys;  // keys from the warp's first on
    const int steps = mine > 0 ? (mine + 4 * kWarpKeys - 1) / (4 * kWarpKeys) : 0;
    KeyWalk<D> kw, vw;
    kw.start(p.k_own[src], p.ko_ld[src], col, static_cast<long long>(b) * p.cap + j0 + warp * kWarpKeys, mine);
    vw.start(p.v_own[src], p.vo_ld[src], col, static_cast<long long>(b) * p.cap + j0 + warp * kWarpKeys, mine);
    // K and V of a step take the ring's next two slots; what follows them goes where they were
    uint32_t ks = sbase + static_cast<uint32_t>(warp * C::kRing), vs = ks + C::kSlot, next = vs + C::kSlot;
    if (steps > 0) kw.load(ks, p.k_own[src]);
    cp_async_commit();
    if (steps > 0) vw.load(vs, p.k_own[src]);
    cp_async_commit();
    if (steps > 1) kw.load(next, p.k_own[src]);
    cp_async_commit();
    WarpRows<D> rows;
    rows.start(p, b, kv, g0);
    for (int step = 0; step < steps; ++step) {
      const int key0 = j0 + (step * 4 + warp) * kWarpKeys;
      cp_async_wait<2>();  // this K
      __syncwarp();
      float s[kWarpKeys / 8][4];
      rows.template scores<kWarpKeys>(ks, 0, j1 - key0, p.scale_log2, s);
      __syncwarp();  // every lane has read the slot
      if (step + 1 < steps) vw.load(ks, p.k_own[src]);
      cp_async_commit();
      if (p.scores) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int g = g0 + (lane >> 2) + 8 * h;
          if (g < p.group) {
            float *dst = p.scores + part_row(p, kv, b, g) * p.score_ld;
#pragma unroll
            for (int n = 0; n < kWarpKeys / 8; ++n) {
              const int key = key0 + 8 * n + 2 * (lane & 3);  // even, and so is the row's pitch
              if (key < j1) *reinterpret_cast<float2 *>(dst + key) = make_float2(s[n][2 * h], s[n][2 * h + 1]);
            }
          }
        }
      }
      rows.template softmax<kWarpKeys>(s);
      cp_async_wait<2>();  // this V
      __syncwarp();
      rows.template add_pv<kWarpKeys>(vs, 0, s);
      __syncwarp();
      if (step + 2 < steps) kw.load(vs, p.k_own[src]);
      cp_async_commit();
      const uint32_t k_next = next;
      next = vs;
      vs = ks;
      ks = k_next;
    }
    cp_async_wait<0>();
    __syncwarp();  // the ring is read and nothing is on its way to it
    float *so = reinterpret_cast<float *>(own_smem);  // each warp's [16][D] over its ring
    rows.put(s_ml[warp], so + warp * (C::kRing / 4));
    __syncthreads();
    const int n_rows = min(16, p.group - g0);
    for (int i = tid; i < n_rows * (D / 4); i += kOwnThreads) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4;
      float2 ml;
      const float4 acc = join_warps<D>(s_ml, so, C::kRing / 4, r, c, ml);
      const long long at = static_cast<long long>(p.split_p + split) * p.batch * p.heads_q + part_row(p, kv, b, g0 + r);
      *reinterpret_cast<float4 *>(p.part_o + at * D + c) = acc;
      if (c == 0) p.part_ml[at] = ml;
    }
  }
  // What follows this kernel on the stream follows the prefix kernel too: the grid
  // ends with its last CTA, which waits for it (the others leave their SMs).
  if (p.has_prev && blockIdx.x + 1 == gridDim.x && blockIdx.y + 1 == gridDim.y && blockIdx.z + 1 == gridDim.z) grid_dep_wait();
}

// ---------------------------------------------------------------------------
// Few keys and few sequences: one launch in place of three. A cluster of CTAs takes a
// (sequence, kv head); its CTAs share the 64-key tiles of the prefix and then of
// the own cache (each sequence reads the prefix by itself, from L2 after the first),
// join through distributed shared memory in cluster order, and finish: outputs by
// columns, weights by the CTA whose keys they are, from the scores it kept. Bound by
// latency: 6.6 us for one sequence of 16 heads on 4 kv heads behind 100 + 64 keys, of
// which a launch and the first loads are about 4.
// ---------------------------------------------------------------------------
constexpr int kDirectTiles = 16;                           // tiles of a CTA at most
constexpr int kScoreRow = kDirectTiles * kOwnKeys + 4;     // floats of a row of kept scores

template <int D>
struct DirectCfg {
  static constexpr int kMat = kOwnKeys * D * 2;  // bytes of a stage's K (or V)
  static constexpr int kStages = 3;
  static constexpr int kTiles = kStages * 2 * kMat;
  static constexpr int kSmem = kTiles + 16 * kScoreRow * 4;
  static_assert(kTiles >= 5 * 16 * D * 4, "the warps' and the CTA's outputs fit over the stages");
};

template <int D>
__global__ void __launch_bounds__(kOwnThreads, 1) k_direct(const __grid_constant__ PrefixAttnParams p) {
  using C = DirectCfg<D>;
  extern __shared__ __align__(128) uint8_t own_smem[];
  __shared__ float2 s_ml[4][16];
  __shared__ __align__(16) float4 s_cta[16];  // the CTA's (m, l) of each row; 16 bytes for the cluster's loads
  __shared__ float s_lse[16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = p.direct;
  const int part = parts > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int unit = blockIdx.x / parts, kv = unit % p.heads_kv, b = unit / p.heads_kv;
  grid_dep_wait();
  grid_dep_launch();
  const int len = own_length(p, b);
  if (kv == 0 && part == 0 && tid == 0 && len != __ldcg(p.lengths + b)) atomicCAS(p.status, 0, kDevBadLength);
  const int tiles_p = (p.prefix + kOwnKeys - 1) / kOwnKeys, tiles = tiles_p + (len + kOwnKeys - 1) / kOwnKeys;
  const int t0 = tiles * part / parts, t1 = tiles * (part + 1) / parts;
  const int own0 = max(t0, tiles_p);  // the CTA's first own tile
  const int src = kv / p.heads_per_source;
  const long long col = static_cast<long long>(kv - src * p.heads_per_source) * D;
  const uint32_t sbase = ptx::smem_addr(own_smem);
  float *s_scores = reinterpret_cast<float *>(own_smem + C::kTiles);  // [16][kScoreRow] of the own tiles
  TileLoader<D> loader;
  int load_stage = 0;
  auto load = [&](int t) {
    if (t < t1) {
      if (t < tiles_p) {
        if (t == t0)
          loader.start(p.k_prefix[src], p.kp_ld[src], p.v_prefix[src], p.vp_ld[src], col, static_cast<long long>(t) * kOwnKeys,
                       p.prefix - t * kOwnKeys);
      } else if (t == own0) {
        const int j = (t - tiles_p) * kOwnKeys;
        loader.start(p.k_own[src], p.ko_ld[src], p.v_own[src], p.vo_ld[src], col, static_cast<long long>(b) * p.cap + j, len - j);
      }
      loader.tile(sbase + static_cast<uint32_t>(load_stage) * 2 * C::kMat, t < tiles_p ? p.k_prefix[src] : p.k_own[src]);
      if (++load_stage == C::kStages) load_stage = 0;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < C::kStages - 1; ++i) load(t0 + i);
  WarpRows<D> rows;
  rows.start(p, b, kv, 0);
  int stage = 0;
  for (int t = t0; t < t1; ++t) {
    asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
    __syncthreads();
    load(t + C::kStages - 1);
    const uint32_t ks = sbase + static_cast<uint32_t>(stage) * 2 * C::kMat, vs = ks + C::kMat;
    if (++stage == C::kStages) stage = 0;
    const int left = (t < tiles_p ? p.prefix - t * kOwnKeys : len - (t - tiles_p) * kOwnKeys) - warp * 16;
    if (left <= 0) continue;
    float s[2][4];
    rows.template scores<16>(ks, warp * 16, left, p.scale_log2, s);
    if (p.w_out[0] && t >= tiles_p) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          *reinterpret_cast<float2 *>(s_scores + ((lane >> 2) + 8 * h) * kScoreRow + (t - own0) * kOwnKeys + warp * 16 + 8 * n +
                                      2 * (lane & 3)) = make_float2(s[n][2 * h], s[n][2 * h + 1]);
    }
    rows.template softmax<16>(s);
    rows.template add_pv<16>(vs, warp * 16, s);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float *so = reinterpret_cast<float *>(own_smem);  // [warp][16][D], then the CTA's [16][D]
  float *cta_o = so + 4 * 16 * D;
  rows.put(s_ml[warp], so + warp * 16 * D);
  __syncthreads();
  for (int i = tid; i < 16 * (D / 4); i += kOwnThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float2 ml;
    *reinterpret_cast<float4 *>(cta_o + r * D + c) = join_warps<D>(s_ml, so, 16 * D, r, c, ml);
    if (c == 0) s_cta[r] = make_float4(ml.x, ml.y, 0.f, 0.f);
  }
  if (parts > 1) ptx::cluster_sync();
  else __syncthreads();
  // Every CTA sees every part; the outputs are dealt by column groups, in cluster order.
  const uint32_t ml_addr = ptx::smem_addr(s_cta), o_addr = ptx::smem_addr(cta_o);
  auto far = [&](uint32_t addr, int q) { return ptx::ld_shared_cluster_f4(ptx::mapa_shared(addr, static_cast<uint32_t>(q))); };
  const bool any = tiles > 0;
  const int pieces = p.group * (D / 4);
  for (int i = part * kOwnThreads + tid; i < pieces; i += parts * kOwnThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float2 ml[8];
    float4 ov[8];
    float top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < parts) {
        const float4 v = far(ml_addr + r * 16, q);
        ml[q] = make_float2(v.x, v.y);
        ov[q] = far(o_addr + static_cast<uint32_t>(r * D + c) * 4u, q);
      }
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < parts) top = fmaxf(top, ml[q].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < parts) {
        const float f = ex2(ml[q].x - top);
        sum += f * ml[q].y;
        acc.x += f * ov[q].x;
        acc.y += f * ov[q].y;
        acc.z += f * ov[q].z;
        acc.w += f * ov[q].w;
      }
    // no key at all: the row is zero
    const float inv = any ? 1.f / sum : 0.f;
    const int h = kv * p.group + r, rank = h / p.heads_per_rank;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.a[rank]) + b * p.a_ld[rank] +
                         static_cast<long long>(h - rank * p.heads_per_rank) * D + c;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  }
  if (p.w_out[0]) {
    if (tid < p.group) {
      float top = -INFINITY, sum = 0.f;
      for (int q = 0; q < parts; ++q) top = fmaxf(top, far(ml_addr + tid * 16, q).x);
      for (int q = 0; q < parts; ++q) {
        const float4 v = far(ml_addr + tid * 16, q);
        sum += ex2(v.x - top) * v.y;
      }
      s_lse[tid] = top + log2f(sum);
    }
    __syncthreads();
    const long long wrow = static_cast<long long>(b) * p.heads_per_source + (kv - src * p.heads_per_source);
    const float *wi = p.w_in[src] ? p.w_in[src] + wrow * p.wi_ld[src] : nullptr;
    float *wo = p.w_out[src] + wrow * p.wo_ld[src];
    const int first = (own0 - tiles_p) * kOwnKeys, keys = t1 > own0 ? min(len, (t1 - tiles_p) * kOwnKeys) - first : 0;
    for (int x = tid; x < keys; x += kOwnThreads) {
      float w = 0.f;
#pragma unroll 8
      for (int g = 0; g < p.group; ++g) w += ex2(s_scores[g * kScoreRow + x] - s_lse[g]);
      if (wi) w += wi[first + x];
      wo[first + x] = w;
    }
    for (int j = len + part * kOwnThreads + tid; j < p.cap; j += parts * kOwnThreads) wo[j] = 0.f;
  }
  __syncwarp();
  if (parts > 1) ptx::cluster_sync_relaxed();  // the other CTAs have read this one's results
}

// ---------------------------------------------------------------------------
// Joins the splits of a (sequence, kv head): one warp per head of the group, then
// the own keys' weights. Bound by latency: 5 us for 61 sequences' 488 heads of six
// splits, and 2.5 us for their weights, four keys a thread (4.6 with one: too few loads
// in flight). With few (sequence, kv head)s, SHARED spreads the
// weights over blockIdx.y, each CTA with the sums of its own reading (two heads, 2048
// own keys: the call takes 10.3 us in place of 17.6; a form for both costs 61
// sequences 0.3 us).
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <int D, bool SHARED>
__global__ void __launch_bounds__(kJoinThreads, 4) k_combine(const __grid_constant__ PrefixAttnParams p) {
  constexpr int kPer = D / 32;  // output columns of a lane
  __shared__ float s_lse[kJoinThreads];
  // The lengths were written before the kernels whose results this one joins, and those
  // began after them: they can be read while the last of them still runs.
  if (p.split_p + p.split_o == 0) grid_dep_wait();
  const int kv = blockIdx.x % p.heads_kv, b = blockIdx.x / p.heads_kv;
  const int share = SHARED ? gridDim.y : 1, at = SHARED ? blockIdx.y : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = own_length(p, b);
  grid_dep_wait();
  grid_dep_launch();
  if (p.split_o == 0 && kv == 0 && at == 0 && threadIdx.x == 0 && len != __ldcg(p.lengths + b)) atomicCAS(p.status, 0, kDevBadLength);
  const int own = len > 0 ? (len + p.chunk - 1) / p.chunk : 0;
  const int n = p.split_p + own;
  const long long stride = static_cast<long long>(p.batch) * p.heads_q;
  if (at > 0) {  // the weights need the sums alone
    for (int g = warp; g < p.group; g += kJoinThreads / 32) {
      const long long row = part_row(p, kv, b, g);
      float m = -INFINITY, l = 0.f;
      for (int i = lane; i < n; i += 32) {
        const float2 ml = p.part_ml[i * stride + row];
        const float m_new = fmaxf(m, ml.x);
        l = (m == m_new ? l : l * ex2(m - m_new)) + ex2(ml.x - m_new) * ml.y;
        m = m_new;
      }
      float mt = m;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
      l *= m == mt ? 1.f : ex2(m - mt);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (lane == 0) s_lse[g] = mt + log2f(l);
    }
  }
  for (int g = warp; g < p.group && at == 0; g += kJoinThreads / 32) {
    const long long row = part_row(p, kv, b, g);
    float mt = -INFINITY, lt = 0.f, acc[kPer] = {};
    for (int s0 = 0; s0 < n; s0 += 32) {  // a lane per split, then every lane its columns of all of them
      float2 ml = make_float2(-INFINITY, 0.f);
      if (s0 + lane < n) ml = p.part_ml[(s0 + lane) * stride + row];
      float mx = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float m_new = fmaxf(mt, mx);
      const float back = mt == m_new ? 1.f : ex2(mt - m_new);
      const float f = s0 + lane < n ? ex2(ml.x - m_new) : 0.f;
      float sum = f * ml.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      lt = lt * back + sum;
#pragma unroll
      for (int c = 0; c < kPer; ++c) acc[c] *= back;
      mt = m_new;
      const int here = min(32, n - s0);
      const float *src = p.part_o + (s0 * stride + row) * D + lane * kPer;
#pragma unroll 8
      for (int j = 0; j < here; ++j) {
        const float w = __shfl_sync(0xffffffffu, f, j);
#pragma unroll
        for (int c = 0; c < kPer; c += 2) {
          const float2 v = *reinterpret_cast<const float2 *>(src + j * stride * D + c);
          acc[c] += w * v.x;
          acc[c + 1] += w * v.y;
        }
      }
    }
    // no key at all: the row is zero, and no key has a weight
    const float inv = n > 0 ? 1.f / lt : 0.f;
    const int h = kv * p.group + g;
    const int r = h / p.heads_per_rank;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.a[r]) + b * p.a_ld[r] +
                         static_cast<long long>(h - r * p.heads_per_rank) * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t *>(dst + i) = pack_bf16(acc[i] * inv, acc[i + 1] * inv);
    if (lane == 0) s_lse[g] = mt + log2f(lt);
  }
  if (!p.w_out[0]) return;
  __syncthreads();
  const int src = kv / p.heads_per_source;
  const long long wrow = static_cast<long long>(b) * p.heads_per_source + (kv - src * p.heads_per_source);
  const float *wi = p.w_in[src] ? p.w_in[src] + wrow * p.wi_ld[src] : nullptr;
  float *wo = p.w_out[src] + wrow * p.wo_ld[src];
  const float *sc = p.scores + part_row(p, kv, b, 0) * p.score_ld;
  for (int j = 4 * (at * kJoinThreads + threadIdx.x); j < p.cap; j += 4 * share * kJoinThreads) {
    float w[4] = {};
    if (j < len) {
      float old[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) old[i] = wi && j + i < len ? wi[j + i] : 0.f;
#pragma unroll 8
      for (int g = 0; g < p.group; ++g) {
        const float4 v = *reinterpret_cast<const float4 *>(sc + static_cast<long long>(g) * p.score_ld + j);
        w[0] += ex2(v.x - s_lse[g]);
        w[1] += ex2(v.y - s_lse[g]);
        w[2] += ex2(v.z - s_lse[g]);
        w[3] += ex2(v.w - s_lse[g]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = j + i < len ? w[i] + old[i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (j + i < p.cap) wo[j + i] = w[i];
  }
}

// The launch shape: pure functions of the sizes, shared by the workspace's size.
struct Shape {
  int pairs, blocks, split_p, ctas_p, chunk, split_o;
};
Shape shape_of(long long batch, long long group, long long heads_kv, long long prefix, long long cap, long long d) {
  Shape s = {};
  const long long rows = batch * group;
  s.pairs = static_cast<int>((rows + 255) / 256);
  s.blocks = static_cast<int>((prefix + 127) / 128);
  s.ctas_p = kSms;
  if (prefix > 0) {
    const long long bases = heads_kv * s.pairs;
    if (cap > 0) {
      // The prefix part leaves SMs to the own part, which runs beside it: its share of
      // the two parts' SM time, 2.4 us for a block step with its part of an item's start
      // and end (1.5 with one tile of rows) and 0.5 us for 64 own keys, if the caches are
      // half full (the lengths are the device's). Fuller caches go on after the prefix,
      // on all SMs. 128 sequences, 32768 + 1025 keys on average: 85 us on 96 SMs, 108 on
      // 112; 61 sequences, 4099 + 256 keys: 34 on 64 or 80, 39 on 96.
      const double t_p = bases * s.blocks * (rows > 128 ? 2.4 : 1.5);
      const double t_o = 0.5 * batch * heads_kv * ((group + 15) / 16) * cap / 64 * 0.50 * d / 128;
      s.ctas_p = static_cast<int>(kSms * t_p / (t_p + t_o) + 0.5);
      if (s.ctas_p < kSms / 4) s.ctas_p = kSms / 4;
    }
    // key splits: the fewest block steps of the busiest CTA, counting about four
    // blocks' time for an item's start and its partial results
    long long best = -1;
    for (int c = 1; c <= s.blocks && c <= 2 * kSms; ++c) {
      const long long waves = (bases * c + s.ctas_p - 1) / s.ctas_p;
      const long long cost = waves * ((s.blocks + c - 1) / c + 4);
      if (best < 0 || cost < best) {
        best = cost;
        s.split_p = c;
      }
      if (bases * c >= 2 * s.ctas_p) break;
    }
  }
  if (cap > 0) {
    // own keys per split: 2048, halved while the grid leaves SMs idle
    s.chunk = 2048;
    const long long units = batch * heads_kv * ((group + 15) / 16);
    while (s.chunk > kOwnKeys && units * ((cap + s.chunk - 1) / s.chunk) < 2 * kSms) s.chunk /= 2;
    s.split_o = static_cast<int>((cap + s.chunk - 1) / s.chunk);
  } else {
    s.chunk = 1;
  }
  return s;
}
long long score_pitch(long long cap) { return (cap + 3) / 4 * 4; }
struct Regions {
  size_t o, ml, scores, total;
};
Regions regions_of(const Shape &s, long long batch, long long heads_q, long long d, long long cap, bool weights) {
  Regions r;
  const size_t rows = static_cast<size_t>(s.split_p + s.split_o) * batch * heads_q;
  r.o = 0;
  r.ml = round256(rows * d * 4);
  r.scores = r.ml + round256(rows * 8);
  r.total = r.scores + (weights ? round256(static_cast<size_t>(batch) * heads_q * score_pitch(cap) * 4) : 0);
  return r;
}

template <int D>
tp_status launch_all(const PrefixAttnParams &p, const PrefixMaps &maps, cudaStream_t s) {
  static unsigned mask_p = 0, mask_o = 0, mask_d = 0;
  static std::mutex mu;
  if (p.direct > 0) {
    const cudaError_t de = allow_smem(k_direct<D>, DirectCfg<D>::kSmem, mask_d, mu);
    if (de != cudaSuccess) return cuda_fail(de);
    return launched(launch_kernel(k_direct<D>, dim3(static_cast<unsigned>(p.batch * p.heads_kv * p.direct)),
                                  dim3(kOwnThreads), DirectCfg<D>::kSmem, s, static_cast<unsigned>(p.direct), p));
  }
  cudaError_t e = allow_smem(k_prefix_part<D>, static_cast<int>(PrefCfg<D>::kSmem), mask_p, mu);
  if (e == cudaSuccess) e = allow_smem(k_own_part<D>, OwnCfg<D>::kSmem, mask_o, mu);
  if (e != cudaSuccess) return cuda_fail(e);
  tp_status st = TP_OK;
  if (p.split_p > 0) {
    const int items = p.heads_kv * p.pairs * p.split_p;
    st = launched(launch_kernel(k_prefix_part<D>, dim3(static_cast<unsigned>(items < p.ctas_p ? items : p.ctas_p)),
                                dim3(kPrefThreads), PrefCfg<D>::kSmem, s, 1, p, maps));
    if (st != TP_OK) return st;
  }
  if (p.split_o > 0) {
    const dim3 grid(static_cast<unsigned>(p.batch * p.heads_kv), static_cast<unsigned>(p.split_o),
                    static_cast<unsigned>((p.group + 15) / 16));
    st = launched(launch_kernel(k_own_part<D>, grid, dim3(kOwnThreads), OwnCfg<D>::kSmem, s, 1, p));
    if (st != TP_OK) return st;
  }
  // CTAs a (sequence, kv head): they share the weights while SMs are idle
  const long long units = static_cast<long long>(p.batch) * p.heads_kv;
  const int most = p.w_out[0] ? (p.cap + 4 * kJoinThreads - 1) / (4 * kJoinThreads) : 1;
  int share = 1;
  while (share < most && share < 32 && units * share * 2 <= 2 * kSms) share *= 2;
  return launched(launch_kernel(share > 1 ? k_combine<D, true> : k_combine<D, false>,
                                dim3(static_cast<unsigned>(units), static_cast<unsigned>(share)), dim3(kJoinThreads), 0, s,
                                1, p));
}

// CTAs a (sequence, kv head) for k_direct, or 0 where the three kernels run: all
// clusters resident at once, one 16-head tile, and few tiles a CTA, since every
// sequence reads the prefix again. Groups of four, d = 128, us here and with the three
// kernels: 1 sequence of 8 kv heads, 100 + 64 keys 6.7 and 8.5, 4032 + 64 keys 11.1
// and 14.7; 9 sequences, 1024 + 64 keys (9 tiles a CTA) 11.0 and 12.0, 512 own
// keys 10.8 and 15.2; 18 sequences, 512 + 64 keys (9) 10.5 and 12.7, 1024 + 64 keys
// (17) 15.3 and 13.4.
int direct_parts(long long units, long long group, long long prefix, long long cap) {
  const long long tiles = (prefix + kOwnKeys - 1) / kOwnKeys + (cap + kOwnKeys - 1) / kOwnKeys;
  if (group > 16 || tiles == 0 || units > num_sms()) return 0;
  int parts = 1;
  for (int c = 2; c <= 8; c *= 2)
    if (c <= tiles && units * c <= num_sms() && units <= max_active_clusters(c)) parts = c;
  return (tiles + parts - 1) / parts <= kDirectTiles ? parts : 0;
}

// Sizes that the launch shape's 32-bit arithmetic and the kernels take.
bool sizes_ok(const tp_dims &d, long long batch, long long prefix, long long cap) {
  const long long group = d.num_q_heads / d.num_kv_heads;
  return (d.head_dim == 64 || d.head_dim == 128) && d.tp_size <= kMaxRanks32 && group <= kJoinThreads &&
         batch <= 0x7fffffffLL / 256 / d.num_q_heads && prefix <= 0x7fffffffLL - 256 &&
         (cap + kOwnKeys - 1) / kOwnKeys <= 65535;
}

}  // namespace
}  // namespace tpgqa

using namespace tpgqa;
using namespace tpgqa::op;

extern "C" size_t tp_prefix_attn_workspace_size(const tp_plan *plan, int64_t batch, int64_t prefix, int64_t capacity,
                                                int32_t weights) {
  tp_dims d;
  if (!plan || batch < 0 || prefix < 0 || capacity < 0 || tp_plan_dims(plan, &d) != TP_OK) return 0;
  if (batch == 0 || !sizes_ok(d, batch, prefix, capacity)) return 0;
  const Shape s = shape_of(batch, d.num_q_heads / d.num_kv_heads, d.num_kv_heads, prefix, capacity, d.head_dim);
  return regions_of(s, batch, d.num_q_heads, d.head_dim, capacity, weights != 0).total;
}

extern "C" tp_status tp_prefix_attn(const tp_plan *plan, int64_t batch, const tp_tensor *q, const tp_tensor *k_prefix,
                                    const tp_tensor *v_prefix, const tp_tensor *k_own, const tp_tensor *v_own,
                                    const int32_t *lengths, const tp_tensor *weight_in, tp_tensor *weight_out,
                                    tp_tensor *a, void *workspace, size_t workspace_bytes, tp_stream_t stream) {
  tp_dims dims;
  tp_rank_shard sh;
  if (!plan || tp_plan_dims(plan, &dims) != TP_OK || tp_plan_query_rank(plan, 0, &sh) != TP_OK) return TP_ERR_INVALID_ARG;
  if (!q || !k_prefix || !v_prefix || !k_own || !v_own || !a || batch < 0) return TP_ERR_INVALID_ARG;
  if (weight_in && !weight_out) return TP_ERR_INVALID_ARG;
  const int n = dims.tp_size;
  const long long hd = dims.head_dim;
  if ((hd != 64 && hd != 128) || n > kMaxRanks32) return TP_ERR_UNSUPPORTED;
  const int sources = sh.kv_replicated ? 1 : n;
  const long long kvc = (sh.kv_head_end - sh.kv_head_begin) * hd, qc = dims.num_q_heads / n * hd;
  const long long P = k_prefix[0].rows, cap = batch ? k_own[0].rows / batch : 0;
  auto check = [&](const tp_tensor &t, long long rows, long long cols) -> tp_status {
    if (!view_ok(t)) return TP_ERR_INVALID_ARG;
    if (t.dtype != TP_BF16) return TP_ERR_DTYPE;
    if (t.rows != rows || t.cols != cols) return TP_ERR_INVALID_ARG;
    return rows > 0 && !vec_aligned(t) ? TP_ERR_ALIGNMENT : TP_OK;
  };
  tp_status st;
  for (int r = 0; r < n; ++r) {
    if ((st = check(q[r], batch, qc)) != TP_OK) return st;
    if ((st = check(a[r], batch, qc)) != TP_OK) return st;
  }
  for (int r = 0; r < sources; ++r) {
    if ((st = check(k_prefix[r], P, kvc)) != TP_OK || (st = check(v_prefix[r], P, kvc)) != TP_OK) return st;
    if ((st = check(k_own[r], batch * cap, kvc)) != TP_OK || (st = check(v_own[r], batch * cap, kvc)) != TP_OK) return st;
    for (const tp_tensor *w : {weight_in, static_cast<const tp_tensor *>(weight_out)}) {
      if (!w) continue;
      if (!view_ok(w[r]) || w[r].rows != batch * (kvc / hd) || w[r].cols != cap) return TP_ERR_INVALID_ARG;
      if (w[r].dtype != TP_F32) return TP_ERR_DTYPE;
      if (!ptr_aligned(w[r].ptr, 4)) return TP_ERR_ALIGNMENT;
    }
  }
  if (batch > 0 && !lengths) return TP_ERR_INVALID_ARG;
  if (!ptr_aligned(lengths, 4)) return TP_ERR_ALIGNMENT;
  if (!sizes_ok(dims, batch, P, cap)) return TP_ERR_UNSUPPORTED;
  const bool weights = weight_out && cap > 0;
  const long long group = dims.num_q_heads / dims.num_kv_heads;
  const Shape shape = shape_of(batch, group, dims.num_kv_heads, P, cap, hd);
  const Regions reg = regions_of(shape, batch, dims.num_q_heads, hd, cap, weights);
  if (batch > 0 && reg.total > 0) {
    if (!workspace || workspace_bytes < reg.total) return TP_ERR_WORKSPACE;
    if (!ptr_aligned(workspace, 16)) return TP_ERR_ALIGNMENT;
  }
  if ((st = check_rank_health(n)) != TP_OK) return st;
  if (batch == 0) return TP_OK;
  DevCtx ctx;
  const cudaError_t e = get_dev_ctx(&ctx);
  if (e != cudaSuccess) return cuda_fail(e);
  static thread_local PrefixAttnParams p;
  static thread_local PrefixMaps maps;  // 8 KB: kept off the stack
  std::memset(&p, 0, sizeof(p));
  for (int r = 0; r < n; ++r) {
    p.q[r] = q[r].ptr;
    p.q_ld[r] = q[r].ld;
    p.a[r] = a[r].ptr;
    p.a_ld[r] = a[r].ld;
  }
  p.direct = direct_parts(batch * dims.num_kv_heads, group, P, cap);
  // Sources whose prefixes are neighbouring columns of one tensor need one map together.
  p.one_prefix = 1;
  for (int r = 1; r < sources; ++r)
    for (const tp_tensor *t : {k_prefix, v_prefix})
      if (t[r].ld != t[0].ld || static_cast<const char *>(t[0].ptr) + r * kvc * 2 != t[r].ptr) p.one_prefix = 0;
  for (int r = 0; r < sources; ++r) {
    p.k_prefix[r] = k_prefix[r].ptr;
    p.v_prefix[r] = v_prefix[r].ptr;
    p.kp_ld[r] = k_prefix[r].ld;
    p.vp_ld[r] = v_prefix[r].ld;
    if (p.direct == 0 && P > 0 && (r == 0 || !p.one_prefix)) {
      tp_tensor k = k_prefix[r], v = v_prefix[r];
      if (p.one_prefix) k.cols = v.cols = kvc * sources;
      if (P == 1) k.ld = v.ld = kvc * sources;  // the pitch of a single row is free
      if (!encode_rows_map(&maps.k[r], k, 128) || !encode_rows_map(&maps.v[r], v, 128)) return TP_ERR_INVALID_ARG;
    }
    p.k_own[r] = k_own[r].ptr;
    p.v_own[r] = v_own[r].ptr;
    p.ko_ld[r] = k_own[r].ld;
    p.vo_ld[r] = v_own[r].ld;
    if (weights) {
      p.w_out[r] = static_cast<float *>(weight_out[r].ptr);
      p.wo_ld[r] = weight_out[r].ld;
      if (weight_in) {
        p.w_in[r] = static_cast<const float *>(weight_in[r].ptr);
        p.wi_ld[r] = weight_in[r].ld;
      }
    }
  }
  char *ws = static_cast<char *>(workspace);
  p.lengths = lengths;
  p.part_o = reinterpret_cast<float *>(ws + reg.o);
  p.part_ml = reinterpret_cast<float2 *>(ws + reg.ml);
  p.scores = weights ? reinterpret_cast<float *>(ws + reg.scores) : nullptr;
  p.batch = static_cast<int>(batch);
  p.heads_q = dims.num_q_heads;
  p.heads_kv = dims.num_kv_heads;
  p.group = static_cast<int>(group);
  p.heads_per_rank = dims.num_q_heads / n;
  p.heads_per_source = dims.num_kv_heads / sources;
  p.d = static_cast<int>(hd);
  p.prefix = static_cast<int>(P);
  p.blocks = shape.blocks;
  p.split_p = shape.split_p;
  p.pairs = shape.pairs;
  p.ctas_p = shape.ctas_p;
  p.cap = static_cast<int>(cap);
  p.score_ld = static_cast<int>(score_pitch(cap));
  p.chunk = shape.chunk;
  p.split_o = shape.split_o;
  p.has_prev = p.split_p > 0 && pdl_enabled();
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(hd)));
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return hd == 128 ? launch_all<128>(p, maps, s) : launch_all<64>(p, maps, s);
}
