// Attention of the last T of S positions over a sliding window and the first tokens, with GQA:
// the query at position i sees key j when j <= i and (j > i - window or j < sinks);
//   A[t, h] = softmax(q K_g^T / sqrt(d)) V_g over these keys.
//
// All query rows of a kv head (T tokens x G heads of its group, token by token) read the same K
// and V, so they are packed into tiles of 128 rows: 128 / G tokens a tile, which move the
// window by that little, and every K and V tile serves the whole group. A work item is (kv
// head, pair of adjacent row tiles, key split). Its keys are two runs, the pair's window from its first
// row's first key on and the first tokens before it, each in units of 16 keys; blocks are 8
// neighbouring units of the two runs together, so that only the last one is short (its products are
// as narrow as it is) and a few first tokens cost a unit, not a block. Masks are applied
// in the blocks where a row's limits lie.
//
// k_window's roles (one CTA an SM, persistent):
//   warp 0        TMA: lane 0 the K ring, lane 1 the V ring (two 128-key stages each);
//   warp 1        MMA issuer (tcgen05): S_A, S_B, P_A V, S_A of the next block, P_B V, ..., over
//                 the items' ends: the next item's first S follows this one's last P V;
//   warps 4-7     softmax of tile A, 8-11 of tile B, one thread a row; they store the output;
//   warps 2, 3    gather the q rows of tile A and B of the next item into the swizzled Q tile (a row is
//                 a token's head, which no one tensor map covers when a group lies on several
//                 ranks) as soon as this item's last S has read it.
// TMEM: S of A at columns 0, of B at 128 (P overwrites its first half as bf16 and is read from
// there), O at 256 and 384. V is used as it lies, [keys x d], as an MN-major operand.
// The reference maximum m of a row is found on its item's first block and moves later only when
// a block's sum of p passes 2^64 or is not finite, as when the row's first keys were masked:
// m is then f32's lowest value, the masked keys weigh 0, and the first key that is seen moves m.
//
// Where there are too few items for the SMs (few tokens), the blocks of an item are
// split, the splits leave f32 sums, and k_window_join joins them.
#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>

#include "op_util.h"
#include "sm100_ptx.cuh"
#include "split_join.cuh"

namespace tpgqa {
namespace {

using namespace op;

constexpr int kWinRanks = 32;
constexpr int kWinThreads = 384;
// Registers a thread: 168 at launch; the softmax's warpgroups take what the first one gives up
// (128 * (104 + 2 * 200) of 384 * 168).
constexpr int kRegsOthers = 104, kRegsSoftmax = 200;
static_assert(kRegsOthers + 2 * kRegsSoftmax <= 3 * 168, "the split fits the launch's registers");
constexpr uint32_t kSubTile = 128u * 128u;  // [128 rows x 64 bf16], swizzled
constexpr float kSumLimit = 0x1p64f;

struct WindowParams {
  int tokens, keys, window, sinks;
  int group, heads_q, heads_kv, heads_per_rank, heads_per_source;
  int rows, pairs, split;           // rows of a kv head, pairs of row tiles, key splits
  int one_map;                      // every source's K (and V) lies in one tensor, in head order
  float scale_log2;
  float *part_o;                    // [split][row][d]
  float2 *part_ml;                  // [split][row]: m (log2 units), l
  int *status;
  long long wait_ns;
  const void *q[kWinRanks];
  long long q_ld[kWinRanks];
  void *a[kWinRanks];
  long long a_ld[kWinRanks];
};
struct WindowMaps {
  CUtensorMap k[kWinRanks], v[kWinRanks];      // boxes of 128 keys
  CUtensorMap k16[kWinRanks], v16[kWinRanks];  // of 16, for blocks of both runs
};

// The keys of a pair of row tiles in units of 16: the window run (w_units units from key w0 on), then the
// first tokens (units from key 0 on, keys below `sinks`, which end before w0).
struct Keys {
  int w0, w_units, sinks, units, blocks;
};
__host__ __device__ inline Keys keys_of(int pair, int rows, int group, int tokens, int keys, int window, int sinks) {
  const int last = 256 * pair + 255 < rows ? 256 * pair + 255 : rows - 1;
  const int p0 = keys - tokens + 256 * pair / group, p1 = keys - tokens + last / group;
  Keys k;
  k.w0 = p0 >= window ? p0 - window + 1 : 0;  // first key of the first row's window
  k.w_units = (p1 - k.w0) / 16 + 1;
  k.sinks = sinks < k.w0 ? sinks : k.w0;
  k.units = k.w_units + (k.sinks + 15) / 16;
  k.blocks = (k.units + 7) / 8;
  return k;
}

__device__ __forceinline__ void record(int *status, int code) { atomicCAS(status, 0, code); }
__device__ __forceinline__ uint64_t desc_mn_sw128(uint32_t saddr, uint32_t mn_stride) {
  // MN-major bf16 tile: rows of 64 MN values (128 bytes, swizzled) a k index, 8-row groups
  // 1024 bytes apart, the next 64 MN values mn_stride bytes on
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(mn_stride >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
constexpr uint32_t kIdescBMn = 1u << 16;  // B operand MN-major

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void st_shared(uint32_t at, const uint4 &v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

template <int D>
struct WinCfg {
  static constexpr int kCh = D / 64;                 // 64-column sub-tiles of a head
  static constexpr uint32_t kTile = kCh * kSubTile;  // a [128 x D] tile
  static constexpr uint32_t kK = 2 * kTile, kV = 4 * kTile, kOut = 6 * kTile, kBar = kOut + 8 * 4096;
  static constexpr size_t kSmem = kBar + 256 + 1024;
};

// n low bits, for any n.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

template <int D>
__global__ void __launch_bounds__(kWinThreads, 1) k_window(const __grid_constant__ WindowParams p, const __grid_constant__ WindowMaps maps) {
  using C = WinCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = ptx::smem_addr(smem), sK0 = sQ + C::kK, sV0 = sQ + C::kV;
  uint8_t *bar_area = smem + C::kBar;
  const uint32_t bar0 = ptx::smem_addr(bar_area);
  const uint32_t q_full0 = bar0, k_full0 = bar0 + 16, k_empty0 = bar0 + 32, v_full0 = bar0 + 48, v_empty0 = bar0 + 64,
                 s_full0 = bar0 + 80, p_full0 = bar0 + 96, o_full0 = bar0 + 112, o_free0 = bar0 + 128, q_empty0 = bar0 + 144,
                 drain = bar0 + 160;
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bar_area + 168);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bar_area + 172);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.rows;
  const int items = p.heads_kv * p.pairs * p.split;
  // An item: (kv head, tile pair, split) and its part [j0, j1) of the pair's blocks.
  struct Item {
    int kv, pair, split, j0, j1;
    Keys k;
    __device__ int units(int j) const { return min(8, k.units - 8 * j); }
  };
  // This CTA's r-th item in snake order over the CTAs, so that with the longest items first
  // (an open window's last tokens) every CTA's total stays close to the mean; those without a block
  // (more splits than blocks) are passed over. False past the last.
  auto next_item = [&](int &r, Item &it) {
    for (;; ++r) {
      const int at = (r & 1) ? static_cast<int>(gridDim.x) - 1 - static_cast<int>(blockIdx.x) : static_cast<int>(blockIdx.x);
      const long long i = static_cast<long long>(r) * gridDim.x + at;
      if (static_cast<long long>(r) * gridDim.x >= items) return false;
      if (i >= items) continue;
      const int first = static_cast<int>(i) / p.split;
      it.split = static_cast<int>(i) - first * p.split;
      it.pair = first / p.heads_kv;
      it.kv = first - it.pair * p.heads_kv;
      it.pair = p.pairs - 1 - it.pair;
      it.k = keys_of(it.pair, rows, p.group, p.tokens, p.keys, p.window, p.sinks);
      const int n = min(p.split, it.k.blocks);
      if (it.split >= n) continue;
      it.j0 = static_cast<int>(static_cast<long long>(it.k.blocks) * it.split / n);
      it.j1 = static_cast<int>(static_cast<long long>(it.k.blocks) * (it.split + 1) / n);
      ++r;
      return true;
    }
  };
  auto tiles_of = [&](const Item &it) { return (2 * it.pair + 1) * 128 < rows ? 2 : 1; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(q_full0 + 8 * s, 32);
      ptx::mbar_init(q_empty0 + 8 * s, 1);
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
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOthers));
  if (warp == 0) {
    if (lane < 2) {
      const uint32_t full0 = lane == 0 ? k_full0 : v_full0, empty0 = lane == 0 ? k_empty0 : v_empty0;
      const uint32_t dst0 = lane == 0 ? sK0 : sV0;
      bool run = true;
      int g = 0;
      Item it;
      for (int r = 0; run && next_item(r, it);) {
        const int src = p.one_map ? 0 : it.kv / p.heads_per_source;
        const int col = (it.kv - src * p.heads_per_source) * D;
        const CUtensorMap *map = lane == 0 ? &maps.k[src] : &maps.v[src];
        const CUtensorMap *map16 = lane == 0 ? &maps.k16[src] : &maps.v16[src];
        for (int j = it.j0; j < it.j1; ++j, ++g) {
          const int s = g & 1;
          if (*abort_flag || !ptx::mbar_wait(empty0 + 8 * s, ((g >> 1) & 1) ^ 1, p.wait_ns)) {
            if (!*abort_flag) record(p.status, kDevTimeoutProducer);
            *abort_flag = 1;
            run = false;
            break;
          }
          const int n = it.units(j), w = min(8, it.k.w_units - 8 * j);  // units of the block; of the window run
          const uint32_t dst = dst0 + s * C::kTile;
          if (w > 0 && w < n) {  // of both runs: unit by unit
            ptx::mbar_arrive_expect_tx(full0 + 8 * s, n * 2048u * C::kCh);
            for (int u = 0; u < n; ++u) {
              const int key = u < w ? it.k.w0 + 128 * j + 16 * u : 128 * j - 16 * it.k.w_units + 16 * u;
              for (int c = 0; c < C::kCh; ++c)
                ptx::tma_load_2d(dst + c * kSubTile + u * 2048u, map16, col + c * 64, key, full0 + 8 * s);
            }
          } else {
            ptx::mbar_arrive_expect_tx(full0 + 8 * s, C::kTile);
            const int key = w > 0 ? it.k.w0 + 128 * j : 128 * j - 16 * it.k.w_units;
            for (int c = 0; c < C::kCh; ++c) ptx::tma_load_2d(dst + c * kSubTile, map, col + c * 64, key, full0 + 8 * s);
          }
          ++issued[s];
        }
      }
    }
  } else if (warp == 1) {  // converged; one lane issues (see elect_one)
    constexpr uint32_t idesc_s0 = ptx::idesc_bf16_f32(128, 0);  // + 2 units << 17: 16 columns a unit
    constexpr uint32_t idesc_o = ptx::idesc_bf16_f32(128, D) | kIdescBMn;
    // descriptors of the tiles' starts; the address field counts 16 bytes
    const uint64_t qd = ptx::smem_desc_sw128(sQ), kd = ptx::smem_desc_sw128(sK0), vd = desc_mn_sw128(sV0, kSubTile);
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
    auto issue_s = [&](int x, int g, int n) {  // S_X = Q_X K^T, 16 n columns
      const uint64_t qa = qd + static_cast<uint32_t>(x) * (C::kTile >> 4), ka = kd + static_cast<uint32_t>(g & 1) * (C::kTile >> 4);
      const uint32_t d = tmem + static_cast<uint32_t>(x * 128);
      const uint32_t idesc = idesc_s0 + (static_cast<uint32_t>(2 * n) << 17);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          ptx::mma_bf16(d, qa + ((kk >> 2) * (kSubTile >> 4) + 2 * (kk & 3)), ka + ((kk >> 2) * (kSubTile >> 4) + 2 * (kk & 3)),
                        idesc, kk > 0 ? 1u : 0u);
        ptx::mma_commit(s_full0 + 8 * x);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int x, int g, bool first, int n) {  // O_X += P_X V, 16 keys (2048 bytes of V) a step
      const uint64_t va = vd + static_cast<uint32_t>(g & 1) * (C::kTile >> 4);
      const uint32_t d = tmem + 256u + static_cast<uint32_t>(x * 128), a = tmem + static_cast<uint32_t>(x * 128);
      const uint32_t more = first ? 0u : 1u;
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (kk < n) ptx::mma_bf16_ts(d, a + 8u * kk, va + kk * (2048u >> 4), idesc_o, kk > 0 ? 1u : more);
      }
      __syncwarp();
    };
    int g = 0, r = 0;
    uint32_t np[2] = {0, 0}, nact[2] = {0, 0};
    Item it, next;
    bool have = next_item(r, it);
    if (have) {  // the first item's first S
      const int tiles = tiles_of(it);
      if (wait(k_full0, 0)) {
        for (int x = 0; ok && x < tiles; ++x) {
          if (!wait(q_full0 + 8 * x, 0)) break;
          ptx::tc_fence_after();
          issue_s(x, 0, it.units(it.j0));
        }
        if (ok) {
          commit(k_empty0);
          if (it.j1 - it.j0 == 1)
            for (int x = 0; x < tiles; ++x) commit(q_empty0 + 8 * x);
        }
      }
    }
    while (ok && have) {
      const int nb = it.j1 - it.j0, tiles = tiles_of(it);
      const bool more = next_item(r, next);
      const int next_tiles = more ? tiles_of(next) : 0;
      for (int j = 0; ok && j < nb; ++j) {
        const int gj = g + j, n = it.units(it.j0 + j);
        const bool last = j + 1 == nb;
        const int n_next = last ? (more ? next.units(next.j0) : 0) : it.units(it.j0 + j + 1);
        if (!wait(v_full0 + 8 * (gj & 1), (gj >> 1) & 1)) break;
        if (n_next > 0 && !wait(k_full0 + 8 * ((gj + 1) & 1), ((gj + 1) >> 1) & 1)) break;
        for (int x = 0; ok && x < 2; ++x) {
          if (x < tiles) {
            if (!wait(p_full0 + 8 * x, np[x] & 1)) break;
            ++np[x];
            if (j == 0 && !wait(o_free0 + 8 * x, (nact[x] & 1) ^ 1)) break;
            ptx::tc_fence_after();
            issue_pv(x, gj, j == 0, n);
            if (last) {
              commit(o_full0 + 8 * x);
              ++nact[x];
            } else {
              issue_s(x, gj + 1, n_next);
            }
          }
          if (last && x < next_tiles) {  // this tile's P has been read by the products before
            if (!wait(q_full0 + 8 * x, nact[x] & 1)) break;
            ptx::tc_fence_after();
            issue_s(x, gj + 1, n_next);
          }
        }
        if (!ok) break;
        commit(v_empty0 + 8 * (gj & 1));
        if (n_next > 0) commit(k_empty0 + 8 * ((gj + 1) & 1));
        // the last S of an item frees its Q
        if (!last && j + 2 == nb)
          for (int x = 0; x < tiles; ++x) commit(q_empty0 + 8 * x);
        if (last && more && next.j1 - next.j0 == 1)
          for (int x = 0; x < next_tiles; ++x) commit(q_empty0 + 8 * x);
      }
      g += nb;
      it = next;
      have = more;
    }
    if (!ok) *abort_flag = 1;
    if (leader) {
      ptx::mma_commit(drain);
      if (!ptx::mbar_wait(drain, 0, p.wait_ns)) record(p.status, kDevTimeoutDrain);
    }
    __syncwarp();
  } else {
    // ---- q rows, 16-byte pieces of a row by neighbouring lanes ----
    const int x = warp - 2;
    constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;
    const int c = lane % kPieces, sub = lane / kPieces;
    Item it;
    uint32_t n = 0;
    for (int r = 0; next_item(r, it);) {
      if ((2 * it.pair + x) * 128 >= rows) continue;
      const bool ready = *abort_flag == 0 && ptx::mbar_wait(q_empty0 + 8 * x, (n & 1) ^ 1, p.wait_ns);
      if (!__all_sync(0xffffffffu, ready)) {
        if (lane == 0) {
          if (*abort_flag == 0) record(p.status, kDevTimeoutProducer);
          *abort_flag = 1;
        }
        break;
      }
      ++n;
#pragma unroll 1
      for (int quarter = 0; quarter < 4; ++quarter) {
        const int m_row = (2 * it.pair + x) * 128 + quarter * 32 + lane;  // row of the kv head: token * group + head
        unsigned long long mine = 0;
        if (m_row < rows) {
          const int token = m_row / p.group, head = it.kv * p.group + m_row - token * p.group, rank = head / p.heads_per_rank;
          mine = reinterpret_cast<unsigned long long>(static_cast<const __nv_bfloat16 *>(p.q[rank]) + token * p.q_ld[rank] +
                                                      static_cast<long long>(head - rank * p.heads_per_rank) * D);
        }
        const uint32_t to = sQ + static_cast<uint32_t>(x) * C::kTile + static_cast<uint32_t>(quarter) * 4096u + (c >> 3) * kSubTile;
#pragma unroll 4
        for (int i = 0; i < kPieces; ++i) {
          const int rr = i * kAtOnce + sub;
          const unsigned long long src = __shfl_sync(0xffffffffu, mine, rr);
          // rows past the last token are zeros
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + rr * 128 + ((c & 7) ^ (rr & 7)) * 16),
                       "l"(src ? src + c * 16 : reinterpret_cast<unsigned long long>(p.q[0])), "r"(src ? 16 : 0)
                       : "memory");
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(q_full0 + 8 * x);
    }
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int x = (warp - 4) >> 2;
    const int qw = warp & 3;
    const int row = qw * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(qw * 32) << 16;
    const uint32_t sb = tmem + lane_off + static_cast<uint32_t>(x * 128);
    const uint32_t ob = tmem + lane_off + 256u + static_cast<uint32_t>(x * 128);
    const uint32_t s_full = s_full0 + 8 * x, p_full = p_full0 + 8 * x;
    const uint32_t turn = sQ + C::kOut + static_cast<uint32_t>(warp - 4) * 4096u;  // where this warp turns its output
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
    Item it;
    for (int r = 0; ok && next_item(r, it);) {
      if ((2 * it.pair + x) * 128 >= rows) continue;
      const int m_row = (2 * it.pair + x) * 128 + row;  // row of the kv head: token * group + head
      const bool there = m_row < rows;
      const int token = there ? m_row / p.group : 0;
      // the row sees keys [w0, pos] and [0, sinks)
      const int pos = p.keys - p.tokens + token;
      const int w0 = pos >= p.window ? pos - p.window + 1 : 0;
      float m = -INFINITY, l = 0.f;
      for (int j = it.j0; j < it.j1; ++j, ++gs) {
        // the block's columns: its window run's up to 16 wu, its first tokens' from there to 16 n
        const int n = it.units(j), wu = max(0, min(8, it.k.w_units - 8 * j));
        const int k0 = it.k.w0 + 128 * j;  // key of column 0 of the window run
        const int hi = min(pos - k0 + 1, 16 * wu), lo = w0 - k0, first = p.sinks - k0;  // seen: i < hi and (i >= lo or i < first)
        const int hs = it.k.sinks - (128 * j - 16 * it.k.w_units);                     // seen of the first tokens: i < hs
        if (!wait_all(s_full, gs & 1)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        uint32_t v[128];
#pragma unroll
        for (int c = 0; c < 8; ++c)
          ptx::tmem_ld_16cols(sb + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&v[16 * c]));
        ptx::tmem_ld_wait();
        ptx::tmem_regs_ready(v);
        if (__any_sync(0xffffffffu, hi < 128 || (lo > 0 && first < 128))) {
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            const uint32_t win = low_bits(16 * wu - 32 * h);
            const uint32_t see = (low_bits(hi - 32 * h) & (~low_bits(lo - 32 * h) | low_bits(first - 32 * h))) |
                                 (low_bits(min(hs, 16 * n) - 32 * h) & ~win);
            if (__any_sync(0xffffffffu, see != 0xffffffffu)) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!(see & (1u << i))) v[32 * h + i] = __float_as_uint(-INFINITY);
            }
          }
        }
        const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
        bool find_max = j == it.j0, move = false;
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
        if (find_max && j > it.j0 && __any_sync(0xffffffffu, move)) {
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
      // out by pieces of 128 bytes, turned through shared memory: a lane that stores its own row
      // touches 32 lines an instruction
      if (p.split > 1) {
        const long long at = (static_cast<long long>(it.split) * p.heads_kv + it.kv) * rows + m_row;
        const int left = rows - (m_row - lane);  // of the warp's rows
        if (there) p.part_ml[at] = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t v[32];
          ptx::tmem_ld_32cols(ob + c * 32, v);
          ptx::tmem_ld_wait();
          ptx::tmem_regs_ready(v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            st_shared(turn + lane * 128 + (i ^ (lane & 7)) * 16, make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3), q = lane & 7;
            const uint4 w = ld_shared(turn + rr * 128 + (q ^ (rr & 7)) * 16);
            if (rr < left) *reinterpret_cast<uint4 *>(p.part_o + (at - lane + rr) * D + c * 32 + q * 4) = w;
          }
          __syncwarp();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(o_free0 + 8 * x);
      } else {
        const float inv = 1.f / l;
        const int head = it.kv * p.group + (there ? m_row - token * p.group : 0), rank = head / p.heads_per_rank;
        const unsigned long long mine =
            there ? reinterpret_cast<unsigned long long>(static_cast<__nv_bfloat16 *>(p.a[rank]) + token * p.a_ld[rank] +
                                                         static_cast<long long>(head - rank * p.heads_per_rank) * D)
                  : 0;
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t v[32];
            ptx::tmem_ld_32cols(ob + c * 64 + hh * 32, v);
            ptx::tmem_ld_wait();
            ptx::tmem_regs_ready(v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16(__uint_as_float(v[8 * i + 2 * e]) * inv, __uint_as_float(v[8 * i + 2 * e + 1]) * inv);
              st_shared(turn + lane * 128 + ((4 * hh + i) ^ (lane & 7)) * 16, make_uint4(w[0], w[1], w[2], w[3]));
            }
          }
          if (c == D / 64 - 1) {  // O has been read
            ptx::tc_fence_before();
            ptx::mbar_arrive(o_free0 + 8 * x);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 4 * i + (lane >> 3), q = lane & 7;
            const uint4 w = ld_shared(turn + rr * 128 + (q ^ (rr & 7)) * 16);
            __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(__shfl_sync(0xffffffffu, mine, rr));
            if (dst) *reinterpret_cast<uint4 *>(dst + c * 64 + q * 8) = w;
          }
          __syncwarp();
        }
      }
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

constexpr int kJoinThreads = 256;

// Joins the splits: one warp a row (token and head).
template <int D>
__global__ void __launch_bounds__(kJoinThreads) k_window_join(const __grid_constant__ WindowParams p) {
  constexpr int kPer = D / 32;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const long long all = static_cast<long long>(p.heads_kv) * p.rows;
  if (row >= all) return;
  const int kv = static_cast<int>(row / p.rows), m_row = static_cast<int>(row - static_cast<long long>(kv) * p.rows);
  const int blocks = keys_of(m_row / 256, p.rows, p.group, p.tokens, p.keys, p.window, p.sinks).blocks;
  float acc[kPer];
  const float l = join_splits<D>(p.part_ml, p.part_o, all, row, min(p.split, blocks), lane, acc);
  const int token = m_row / p.group, head = kv * p.group + (m_row - token * p.group), rank = head / p.heads_per_rank;
  __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.a[rank]) + token * p.a_ld[rank] +
                       static_cast<long long>(head - rank * p.heads_per_rank) * D + lane * kPer;
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t *>(dst + i) = pack_bf16(acc[i] * inv, acc[i + 1] * inv);
}

// Key splits of an item: the fewest block steps of the busiest CTA, counting about four blocks'
// time for an item's start and its partial results. One where the items fill the SMs.
int splits_of(long long rows, int group, int heads_kv, int tokens, int keys, int window, int sinks) {
  const int pairs = static_cast<int>((rows + 255) / 256);
  const long long bases = static_cast<long long>(pairs) * heads_kv;
  const int sms = num_sms();
  if (bases >= sms) return 1;
  const int most = keys_of(pairs - 1, static_cast<int>(rows), group, tokens, keys, window, sinks).blocks;
  int split = 1;
  long long best = -1;
  for (int c = 1; c <= most && bases * c <= 2LL * sms; ++c) {
    const long long cost = (bases * c + sms - 1) / sms * ((most + c - 1) / c + 4);
    if (best < 0 || cost < best) {
      best = cost;
      split = c;
    }
  }
  return split;
}

// Sizes that the item arithmetic takes in 32 bits.
bool sizes_ok(const tp_dims &d, long long tokens, long long keys) {
  return (d.head_dim == 64 || d.head_dim == 128) && d.tp_size <= kWinRanks && tokens <= 0x7fffffffLL / 8 / d.num_q_heads &&
         keys <= 0x7fffffffLL - 256;
}

template <typename K>
cudaError_t allow_smem(K kernel, int bytes, unsigned &mask, std::mutex &mu) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> g(mu);
  if (dev < 32 && (mask & (1u << dev))) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 32) mask |= 1u << dev;
  return e;
}

template <int D>
tp_status launch_window(const WindowParams &p, const WindowMaps &maps, cudaStream_t s) {
  static unsigned mask = 0;
  static std::mutex mu;
  const cudaError_t e = allow_smem(k_window<D>, static_cast<int>(WinCfg<D>::kSmem), mask, mu);
  if (e != cudaSuccess) return cuda_fail(e);
  const long long items = static_cast<long long>(p.heads_kv) * p.pairs * p.split;
  const unsigned grid = static_cast<unsigned>(items < num_sms() ? items : num_sms());
  tp_status st = launched(launch_kernel(k_window<D>, dim3(grid), dim3(kWinThreads), WinCfg<D>::kSmem, s, 1, p, maps));
  if (st != TP_OK || p.split == 1) return st;
  const long long all = static_cast<long long>(p.heads_kv) * p.rows;
  return launched(launch_kernel(k_window_join<D>, dim3(static_cast<unsigned>((all + kJoinThreads / 32 - 1) / (kJoinThreads / 32))),
                                dim3(kJoinThreads), 0, s, 1, p));
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }
// Bytes of the splits' sums before their (m, l), and of both.
size_t sums_bytes(int split, long long rows_all, long long d) { return split > 1 ? round256(static_cast<size_t>(split) * rows_all * d * 4) : 0; }
size_t workspace_bytes_of(int split, long long rows_all, long long d) {
  return split > 1 ? sums_bytes(split, rows_all, d) + round256(static_cast<size_t>(split) * rows_all * 8) : 0;
}

}  // namespace
}  // namespace tpgqa

using namespace tpgqa;
using namespace tpgqa::op;

extern "C" size_t tp_window_attn_workspace_size(const tp_plan *plan, int64_t tokens, int64_t keys, int32_t window,
                                                int32_t sinks) {
  tp_dims d;
  if (!plan || tokens < 1 || keys < tokens || window < 1 || sinks < 0 || tp_plan_dims(plan, &d) != TP_OK) return 0;
  if (!sizes_ok(d, tokens, keys)) return 0;
  const int group = d.num_q_heads / d.num_kv_heads;
  const int split = splits_of(tokens * group, group, d.num_kv_heads, static_cast<int>(tokens), static_cast<int>(keys), window, sinks);
  return workspace_bytes_of(split, tokens * d.num_q_heads, d.head_dim);
}

extern "C" tp_status tp_window_attn(const tp_plan *plan, const tp_tensor *q, const tp_tensor *k, const tp_tensor *v,
                                    int32_t window, int32_t sinks, tp_tensor *a, void *workspace, size_t workspace_bytes,
                                    tp_stream_t stream) {
  tp_dims dims;
  tp_rank_shard sh;
  if (!plan || tp_plan_dims(plan, &dims) != TP_OK || tp_plan_query_rank(plan, 0, &sh) != TP_OK) return TP_ERR_INVALID_ARG;
  if (!q || !k || !v || !a || window < 1 || sinks < 0) return TP_ERR_INVALID_ARG;
  const int n = dims.tp_size;
  const long long hd = dims.head_dim;
  if ((hd != 64 && hd != 128) || n > kWinRanks) return TP_ERR_UNSUPPORTED;
  const int sources = sh.kv_replicated ? 1 : n;
  const long long qc = dims.num_q_heads / n * hd, kvc = dims.num_kv_heads / sources * hd;
  const long long T = q[0].rows, S = k[0].rows;
  auto check = [&](const tp_tensor &t, long long rows, long long cols) -> tp_status {
    if (!view_ok(t)) return TP_ERR_INVALID_ARG;
    if (t.dtype != TP_BF16) return TP_ERR_DTYPE;
    if (t.rows != rows || t.cols != cols) return TP_ERR_INVALID_ARG;
    return rows > 0 && !vec_aligned(t) ? TP_ERR_ALIGNMENT : TP_OK;
  };
  tp_status st;
  for (int r = 0; r < n; ++r)
    if ((st = check(q[r], T, qc)) != TP_OK || (st = check(a[r], T, qc)) != TP_OK) return st;
  for (int r = 0; r < sources; ++r)
    if ((st = check(k[r], S, kvc)) != TP_OK || (st = check(v[r], S, kvc)) != TP_OK) return st;
  if (S < T) return TP_ERR_INVALID_ARG;
  if (!sizes_ok(dims, T, S)) return TP_ERR_UNSUPPORTED;
  const int group = dims.num_q_heads / dims.num_kv_heads;
  const long long rows_all = T * dims.num_q_heads;
  const int split = T > 0 ? splits_of(T * group, group, dims.num_kv_heads, static_cast<int>(T), static_cast<int>(S), window, sinks) : 1;
  const size_t need = workspace_bytes_of(split, rows_all, hd);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return TP_ERR_WORKSPACE;
    if (!ptr_aligned(workspace, 16)) return TP_ERR_ALIGNMENT;
  }
  if ((st = check_rank_health(n)) != TP_OK) return st;
  if (T == 0) return TP_OK;
  DevCtx ctx;
  const cudaError_t e = get_dev_ctx(&ctx);
  if (e != cudaSuccess) return cuda_fail(e);
  static thread_local WindowParams p;
  static thread_local WindowMaps maps;  // 16 KB: kept off the stack
  std::memset(&p, 0, sizeof(p));
  for (int r = 0; r < n; ++r) {
    p.q[r] = q[r].ptr;
    p.q_ld[r] = q[r].ld;
    p.a[r] = a[r].ptr;
    p.a_ld[r] = a[r].ld;
  }
  // Sources that are neighbouring columns of one tensor need one map together.
  p.one_map = 1;
  for (int r = 1; r < sources; ++r)
    for (const tp_tensor *t : {k, v})
      if (t[r].ld != t[0].ld || static_cast<const char *>(t[0].ptr) + r * kvc * 2 != t[r].ptr) p.one_map = 0;
  for (int r = 0; r < (p.one_map ? 1 : sources); ++r) {
    tp_tensor kr = k[r], vr = v[r];
    if (p.one_map) kr.cols = vr.cols = kvc * sources;
    if (S == 1) kr.ld = vr.ld = kvc * sources;  // the pitch of a single row is free
    if (!encode_rows_map(&maps.k[r], kr, 128) || !encode_rows_map(&maps.v[r], vr, 128)) return TP_ERR_INVALID_ARG;
    if (sinks > 0 && (!encode_rows_map(&maps.k16[r], kr, 16) || !encode_rows_map(&maps.v16[r], vr, 16))) return TP_ERR_INVALID_ARG;
  }
  p.tokens = static_cast<int>(T);
  p.keys = static_cast<int>(S);
  p.window = window;
  p.sinks = sinks;
  p.group = group;
  p.heads_q = dims.num_q_heads;
  p.heads_kv = dims.num_kv_heads;
  p.heads_per_rank = dims.num_q_heads / n;
  p.heads_per_source = dims.num_kv_heads / sources;
  p.rows = static_cast<int>(T * group);
  p.pairs = (p.rows + 255) / 256;
  p.split = split;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(hd)));
  p.part_o = static_cast<float *>(workspace);
  p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + sums_bytes(split, rows_all, hd));
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return hd == 128 ? launch_window<128>(p, maps, s) : launch_window<64>(p, maps, s);
}
