// Attention of the last T of S positions over a sliding window and the first tokens, with GQA:
// the query at position i sees key j when j <= i and (j > i - window or j < sinks);
//   A[t, h] = softmax(q K_g^T / sqrt(d)) V_g over these keys.
//
// The query rows of the heads of a group read the same K and V, so they are packed into tiles of 128
// rows, token by token: with G heads 128 / G tokens a tile, which move the window by
// that little, and every K and V tile serves all of them. G is the largest power of two that divides
// both the plan's group and a rank's heads, so that one copy of a 3-D tensor map (values, heads, tokens) brings
// a tile in this order. A work item is (such a set of heads, two adjacent row tiles or, where there are few, one,
// key split). Its keys are two runs, the window of its rows from the first row's first key
// on and the first tokens before it, each in units of 16 keys; blocks are 8
// neighbouring units of the two runs together, so that only the last one is short (its products are
// as narrow as it is) and a few first tokens cost a unit, not a block. The units of the first tokens end with the
// last of these, so that what fills the first one up are rows before key 0, which the copy makes zeros: rows behind
// them would be keys that maybe no query sees, whose memory holds anything, and 0 * NaN is NaN in P V.
// Masks are applied in the blocks where a row's limits lie.
//
// k_window's roles (one CTA an SM, persistent):
//   warp 0        TMA: one lane, K and V tiles of 128 keys in turn through one ring of five slots
//                 (d = 128; eight for d = 64): a tile is asked for one to two steps before it is needed;
//   warps 1, 2    MMA issuers (tcgen05) of tile A and of tile B: S, P V, S of the next block, ..., over
//                 the items' ends: the next item's first S follows this one's last P V. One warp
//                 for both tiles bounds the whole: a product of 128 x 128 x 16 takes the tensor core
//                 64 cycles and its issue about 80 (2.1 us a step of both tiles in place of 1.55);
//   warp 3        TMA of the next item's q tiles as soon as this item's last S has read them;
//   warps 4-7     softmax of tile A, 8-11 of tile B, one thread a row;
//   warps 12-15   store the outputs, while the softmax is at the next item already.
// TMEM: S of A at columns 0, of B at 128 (P overwrites its first half as bf16 and is read from
// there), O at 256 and 384. V is used as it lies, [keys x d], as an MN-major operand.
// The reference maximum m of a row is found on its item's first block and moves later only when
// a block's sum of p passes 2^64 or is not finite, as when the row's first keys were masked:
// m is then f32's lowest value, the masked keys weigh 0, and the first key that is seen moves m.
//
// Bounds. A step (128 keys of both tiles, d = 128) is 32 products of 128 x 128 x 16: 1.0 us at 64 cycles
// each, 1.35 us at the rate of a large library product (1895 TFLOP/s); and 256 x 128 exponentials, 0.5 us
// of their unit (its counter reads 27%). It takes 1.55 us: 0.5 us of a tile's own products, then 1.05 us from S to
// P, one thread's chain of waits, loads, about 350 instructions and stores, while the other tile's products
// run. More instructions lengthen it: an eighth of the exponentials as polynomials 1.72 us. Every item adds
// about 4.4 us (its first S, a short block, masked blocks at both of the window's ends, the output), so a
// window of 1024 and 4 first tokens over 16384 tokens, 64 heads on 8 (9 blocks an item), takes 455 us,
// 1.17 PFLOP/s over the keys that are seen (in bursts at 2070 MHz; 467 for seconds on end, when the power cap
// holds the clock at 2000 to 2025). With heads of 64 it takes 385 us (floor 141): half the products behind the same
// chain. Small calls are bound by one item's latency: 2047 tokens of 16 heads of 64, window 300: 9.8 us; one token,
// 64 heads, 4100 keys: 9.8. Groups that are no power of two are taken in parts: one token over 4100 keys of 4 kv
// heads takes 9.1 us with 8 heads each, 10.8 with 6 (in pairs), 15.8 with 7 (one by one); 4096 tokens, window
// 1024, take 57, 54 and 73.
//
// Where there are too few items for the SMs (few tokens), items have one row tile, or their blocks are
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
constexpr int kWinThreads = 512;
// Registers a thread: 128 at launch; the softmax's two warpgroups take what the other two give up.
constexpr int kRegsOthers = 64, kRegsSoftmax = 192;
static_assert(kRegsOthers + kRegsSoftmax <= 2 * 128, "the split fits the launch's registers");
constexpr uint32_t kSubTile = 128u * 128u;  // [128 rows x 64 bf16], swizzled
constexpr float kSumLimit = 0x1p64f;

struct WindowParams {
  int tokens, keys, window, sinks;
  int group, sets;                  // heads that share a tile; such sets
  int sets_per_kv, heads_per_rank, heads_per_source;
  int rows, parts, split;           // rows of a set, parts of one or two row tiles, key splits
  Divider by_sets, by_split;
  int group_shift;
  int one_map;                      // every source's K (and V) lies in one tensor, in head order
  float scale_log2;
  float *part_o;                    // [split][row][d]
  float2 *part_ml;                  // [split][row]: m (log2 units), l
  int *status;
  long long wait_ns;
  void *a[kWinRanks];
  long long a_ld[kWinRanks];
};
struct WindowMaps {
  CUtensorMap q[kWinRanks];                    // boxes of 64 values, the set's heads, 128 / group tokens
  CUtensorMap k[kWinRanks], v[kWinRanks];      // boxes of 128 keys
  CUtensorMap k16[kWinRanks], v16[kWinRanks];  // of 16, for blocks of both runs
};

// The keys of an item's rows in units of 16: the window run (w_units units from key w0 on), then the
// first tokens (units that end with key sinks - 1, at w0 - 1 or before; the first one's first `pad` keys are below 0).
struct Keys {
  int w0, w_units, sinks, units, blocks;
  __host__ __device__ int pad() const { return -sinks & 15; }
  // the key of column 0 of block j where that lies in the first tokens' run, or would if it went on to the left
  __host__ __device__ int first(int j) const { return 128 * j - 16 * w_units - pad(); }
};
// Of tokens t0 .. t1, the item's first and last.
__host__ __device__ inline Keys keys_of(int t0, int t1, int tokens, int keys, int window, int sinks) {
  const int p0 = keys - tokens + t0, p1 = keys - tokens + t1;
  Keys k;
  k.w0 = p0 >= window ? p0 - window + 1 : 0;  // first key of the first row's window
  k.w_units = (p1 - k.w0) / 16 + 1;
  k.sinks = sinks < k.w0 ? sinks : k.w0;
  k.units = k.w_units + (k.sinks + 15) / 16;
  k.blocks = (k.units + 7) / 8;
  return k;
}

// Of part `part` of the rows: TILES row tiles.
template <int TILES>
__device__ __forceinline__ Keys keys_of_part(const WindowParams &p, int part) {
  constexpr int kRows = 128 * TILES;
  return keys_of(kRows * part >> p.group_shift, min(kRows * part + kRows - 1, p.rows - 1) >> p.group_shift, p.tokens, p.keys, p.window, p.sinks);
}

template <int D>
struct WinCfg {
  static constexpr int kCh = D / 64;                 // 64-column sub-tiles of a head
  static constexpr uint32_t kTile = kCh * kSubTile;  // a [128 x D] tile
  static constexpr int kSlots = D == 128 ? 5 : 8;    // of the K and V ring
  static constexpr uint32_t kRing = 2 * kTile, kL = kRing + kSlots * kTile, kBar = kL + 1024;
  static constexpr size_t kSmem = kBar + 288 + 64 + 1024;
};
// A place in the ring: K of block g is tile 2g, V is tile 2g + 1.
template <int SLOTS>
struct Slot {
  int at;
  uint32_t phase;
  __device__ __forceinline__ void on(int n) {
    at += n;
    if (at >= SLOTS) {
      at -= SLOTS;
      phase ^= 1;
    }
  }
};

// n low bits, for any n.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

// TILES: row tiles of an item.
template <int D, int TILES>
__global__ void __launch_bounds__(kWinThreads, 1) k_window(const __grid_constant__ WindowParams p, const __grid_constant__ WindowMaps maps) {
  using C = WinCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = ptx::smem_addr(smem), sR = sQ + C::kRing;
  uint8_t *bar_area = smem + C::kBar;
  const uint32_t bar0 = ptx::smem_addr(bar_area);
  const uint32_t q_full0 = bar0, q_empty0 = bar0 + 16, s_full0 = bar0 + 32, p_full0 = bar0 + 48, o_full0 = bar0 + 64,
                 o_free0 = bar0 + 80, l_full0 = bar0 + 96, drain0 = bar0 + 112, turn0 = bar0 + 128, full0 = bar0 + 144, empty0 = full0 + 8 * C::kSlots;
  static_assert(144 + 16 * C::kSlots <= 272, "barriers, TMEM slot and abort flag fit");
  volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(bar_area + 272);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(bar_area + 276);
  float *row_l = reinterpret_cast<float *>(smem + C::kL);  // l of the rows of both tiles

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = p.rows;
  const int items = p.sets * p.parts * p.split;
  // An item: (set of heads, part of the rows, split) and its own [j0, j1) of the part's blocks.
  struct Item {
    int set, part, split, j0, j1;
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
      const int first = p.by_split.of(static_cast<int>(i));
      it.split = static_cast<int>(i) - first * p.split;
      it.part = p.by_sets.of(first);
      it.set = first - it.part * p.sets;
      it.part = p.parts - 1 - it.part;
      it.k = keys_of_part<TILES>(p, it.part);
      it.j0 = 0;
      it.j1 = it.k.blocks;
      if (p.split > 1) {
        const int n = min(p.split, it.k.blocks);
        if (it.split >= n) continue;
        it.j0 = static_cast<int>(static_cast<long long>(it.k.blocks) * it.split / n);
        it.j1 = static_cast<int>(static_cast<long long>(it.k.blocks) * (it.split + 1) / n);
      }
      ++r;
      return true;
    }
  };
  auto row_of = [&](const Item &it, int x) { return (TILES * it.part + x) * 128; };  // first row of a tile
  auto has = [&](const Item &it, int x) { return x < TILES && row_of(it, x) < rows; };
  auto tiles_of = [&](const Item &it) { return has(it, 1) ? 2 : 1; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      ptx::mbar_init(q_full0 + 8 * s, 1);
      ptx::mbar_init(q_empty0 + 8 * s, 1);
      ptx::mbar_init(s_full0 + 8 * s, 1);
      ptx::mbar_init(p_full0 + 8 * s, 4);
      ptx::mbar_init(o_full0 + 8 * s, 1);
      ptx::mbar_init(o_free0 + 8 * s, 4);
      ptx::mbar_init(l_full0 + 8 * s, 4);
      ptx::mbar_init(drain0 + 8 * s, 1);
      ptx::mbar_init(turn0 + 8 * s, 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      ptx::mbar_init(full0 + 8 * s, 1);
      ptx::mbar_init(empty0 + 8 * s, 2);  // both tiles' products have read it
    }
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t *>(tmem_slot)), 512);
    ptx::tmem_relinquish();
  }
  // Before the wait for the kernel before: the first item, for all roles (from the wait to the first K tile
  // 1.3 us, 2.6 where each role finds it for itself), and the maps, whose first reads are misses too.
  struct First {
    Item it;
    int r, have;
  };
  static_assert(sizeof(First) <= 64, "the first item fits");
  if (threadIdx.x == 96) {
    First f;
    f.r = 0;
    f.have = next_item(f.r, f.it);
    int *to = reinterpret_cast<int *>(bar_area + 288);
    if (!f.have) f.it = Item{};
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(First) / 4); ++i) to[i] = reinterpret_cast<const int *>(&f)[i];
    if (f.have) {
      const int kv = f.it.set / p.sets_per_kv, src = p.one_map ? 0 : kv / p.heads_per_source;
      ptx::prefetch_tensormap(&maps.q[f.it.set * p.group / p.heads_per_rank]);
      ptx::prefetch_tensormap(&maps.k[src]);
      ptx::prefetch_tensormap(&maps.v[src]);
      if (f.it.k.sinks > 0) {
        ptx::prefetch_tensormap(&maps.k16[src]);
        ptx::prefetch_tensormap(&maps.v16[src]);
      }
    }
  }
  auto first_item = [&](int &r, Item &it) {
    First f;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(First) / 4); ++i)
      reinterpret_cast<int *>(&f)[i] = reinterpret_cast<const int *>(bar_area + 288)[i];
    it = f.it;
    r = f.r;
    return f.have != 0;
  };
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOthers));
    if (warp == 0) {
      if (lane == 0) {
        bool run = true;
        Slot<C::kSlots> at = {0, 0};
        int filled = 0;
        Item it;
        int r;
        for (bool have = first_item(r, it); run && have; have = next_item(r, it)) {
          const int kv = it.set / p.sets_per_kv, src = p.one_map ? 0 : kv / p.heads_per_source;
          const int col = (kv - src * p.heads_per_source) * D;
          for (int t = 2 * it.j0; run && t < 2 * it.j1; ++t) {  // K, V of block t / 2
            const int j = t >> 1, v = t & 1;
            if (*abort_flag || !ptx::mbar_wait(empty0 + 8 * at.at, at.phase ^ 1, p.wait_ns)) {
              if (!*abort_flag) record(p.status, kDevTimeoutProducer);
              *abort_flag = 1;
              run = false;
              break;
            }
            const int n = it.units(j), w = min(8, it.k.w_units - 8 * j);  // units of the block; of the window run
            const uint32_t dst = sR + at.at * C::kTile, bar = full0 + 8 * at.at;
            if (w > 0 && w < n) {  // of both runs: unit by unit
              const CUtensorMap *map = v ? &maps.v16[src] : &maps.k16[src];
              ptx::mbar_arrive_expect_tx(bar, n * 2048u * C::kCh);
              for (int u = 0; u < n; ++u) {
                const int key = (u < w ? it.k.w0 + 128 * j : it.k.first(j)) + 16 * u;
                for (int c = 0; c < C::kCh; ++c) ptx::tma_load_2d(dst + c * kSubTile + u * 2048u, map, col + c * 64, key, bar);
              }
            } else {
              const CUtensorMap *map = v ? &maps.v[src] : &maps.k[src];
              ptx::mbar_arrive_expect_tx(bar, C::kTile);
              const int key = w > 0 ? it.k.w0 + 128 * j : it.k.first(j);
              for (int c = 0; c < C::kCh; ++c) ptx::tma_load_2d(dst + c * kSubTile, map, col + c * 64, key, bar);
            }
            at.on(1);
            ++filled;
          }
        }
        // every load has landed before the CTA may end: the last fill of each slot
        Slot<C::kSlots> last = {0, 0};
        for (int i = 0; i < filled; ++i, last.on(1))
          if (i + C::kSlots >= filled && !ptx::mbar_wait(full0 + 8 * last.at, last.phase, p.wait_ns)) record(p.status, kDevTimeoutDrain);
      }
    } else if (warp < 3) {  // converged; one lane issues (see elect_one)
      const int x = warp - 1;
      constexpr uint32_t idesc_s0 = ptx::idesc_bf16_f32(128, 0);  // + 2 units << 17: 16 columns a unit
      constexpr uint32_t idesc_o = ptx::idesc_bf16_f32(128, D) | ptx::kIdescBMn;
      // descriptors of the tiles' starts; the address field counts 16 bytes
      const uint64_t qd = ptx::smem_desc_sw128(sQ), kd = ptx::smem_desc_sw128(sR), vd = ptx::smem_desc_mn_sw128(sR, kSubTile);
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
      const uint64_t qa = qd + static_cast<uint32_t>(x) * (C::kTile >> 4);
      const uint32_t td_s = tmem + static_cast<uint32_t>(x * 128), td_o = tmem + 256u + static_cast<uint32_t>(x * 128);
      auto issue_s = [&](int slot, int n) {  // S = Q K^T, 16 n columns
        const uint64_t ka = kd + static_cast<uint32_t>(slot) * (C::kTile >> 4);
        const uint32_t idesc = idesc_s0 + (static_cast<uint32_t>(2 * n) << 17);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            ptx::mma_bf16(td_s, qa + ((kk >> 2) * (kSubTile >> 4) + 2 * (kk & 3)), ka + ((kk >> 2) * (kSubTile >> 4) + 2 * (kk & 3)),
                          idesc, kk > 0 ? 1u : 0u);
          ptx::mma_commit(s_full0 + 8 * x);
        }
        __syncwarp();
      };
      auto issue_pv = [&](int slot, bool first, int n) {  // O += P V, 16 keys (2048 bytes of V) a step
        const uint64_t va = vd + static_cast<uint32_t>(slot) * (C::kTile >> 4);
        const uint32_t more = first ? 0u : 1u;
        if (n == 8) {
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) ptx::mma_bf16_ts(td_o, td_s + 8u * kk, va + kk * (2048u >> 4), idesc_o, kk > 0 ? 1u : more);
          }
        } else if (leader) {
#pragma unroll 1
          for (int kk = 0; kk < n; ++kk) ptx::mma_bf16_ts(td_o, td_s + 8u * kk, va + kk * (2048u >> 4), idesc_o, kk > 0 ? 1u : more);
        }
        __syncwarp();
      };
      // a slot is free of this tile: at once where the tile has no rows, else when its products are done
      auto release = [&](int slot, bool used) {
        if (leader) {
          if (used) ptx::mma_commit(empty0 + 8 * slot);
          else ptx::mbar_arrive(empty0 + 8 * slot);
        }
        __syncwarp();
      };
      // what of an item these products need
      struct Work {
        int units, nb;  // from its first block on; its blocks, 0: no item
        bool mine;      // the tile has rows
      };
      auto work = [&](const Item &it, bool have) {
        Work w = {0, 0, false};
        if (have) w = {it.k.units - 8 * it.j0, it.j1 - it.j0, x < tiles_of(it)};
        return w;
      };
      // The tiles' products are issued in turn, A's P V and next S, then B's. As they come, both tiles would
      // fall into step: in their softmax together, then in the tensor core's queue.
      uint32_t turn = 0;
      uint32_t np = 0, nact = 0;                     // P tiles consumed; items with rows in the tile
      Slot<C::kSlots> ks = {0, 0}, vs = {1, 0};      // the next block of each
      auto first_s = [&](const Work &w) {  // the S of an item's first block
        if (!wait(full0 + 8 * ks.at, ks.phase)) return;
        if (w.mine) {
          if (!wait(q_full0 + 8 * x, nact & 1)) return;
          ptx::tc_fence_after();
          issue_s(ks.at, min(8, w.units));
          if (w.nb == 1) commit(q_empty0 + 8 * x);  // the last S of an item frees its Q
        }
        release(ks.at, w.mine);
        ks.on(2);
      };
      Item it;
      int r;
      const bool any = first_item(r, it);
      Work w = work(it, any);
      if (w.nb > 0) first_s(w);
      while (ok && w.nb > 0) {
        const bool more = next_item(r, it);
        const Work next = work(it, more);
        for (int j = 0; ok && j < w.nb; ++j, vs.on(2)) {
          const bool last = j + 1 == w.nb;
          // what is there early is waited for before P, which is there last
          if (!wait(full0 + 8 * vs.at, vs.phase) || (!last && !wait(full0 + 8 * ks.at, ks.phase))) break;
          if (!wait(turn0 + 8 * x, turn ^ (x == 0 ? 1 : 0))) break;
          if (w.mine) {
            if (j == 0 && !wait(o_free0 + 8 * x, (nact & 1) ^ 1)) break;
            if (!wait(p_full0 + 8 * x, np & 1)) break;
            ++np;
            ptx::tc_fence_after();
            issue_pv(vs.at, j == 0, min(8, w.units - 8 * j));
            if (last) {
              commit(o_full0 + 8 * x);
              ++nact;
            } else {
              issue_s(ks.at, min(8, w.units - 8 * (j + 1)));
            }
          }
          if (leader) ptx::mbar_arrive(turn0 + 8 * (x ^ 1));
          turn ^= 1;
          release(vs.at, w.mine);
          if (last) {
            if (next.nb > 0) first_s(next);  // this tile's P has been read by the products before
          } else {
            if (w.mine && j + 2 == w.nb) commit(q_empty0 + 8 * x);
            release(ks.at, w.mine);
            ks.on(2);
          }
        }
        w = next;
      }
      if (!ok) *abort_flag = 1;
      if (leader) {
        ptx::mma_commit(drain0 + 8 * x);
        if (!ptx::mbar_wait(drain0 + 8 * x, 0, p.wait_ns)) record(p.status, kDevTimeoutDrain);
      }
      __syncwarp();
    } else {
      // ---- the q tiles ----
      if (lane == 0) {
        Item it;
        uint32_t n[2] = {0, 0};
        int r;
        bool have = first_item(r, it), ok = true;
        auto place = [&](const Item &i, int &rank, int &head) {
          rank = i.set * p.group / p.heads_per_rank;
          head = i.set * p.group - rank * p.heads_per_rank;
        };
        while (have && ok) {
          int rank, head;
          place(it, rank, head);
          for (int x = 0; x < tiles_of(it); ++x) {
            if (*abort_flag || !ptx::mbar_wait(q_empty0 + 8 * x, (n[x] & 1) ^ 1, p.wait_ns)) {
              if (!*abort_flag) record(p.status, kDevTimeoutProducer);
              *abort_flag = 1;
              ok = false;
              break;
            }
            ++n[x];
            ptx::mbar_arrive_expect_tx(q_full0 + 8 * x, C::kTile);
            for (int c = 0; c < C::kCh; ++c)
              ptx::tma_load_3d(sQ + x * C::kTile + c * kSubTile, &maps.q[rank], c * 64, head, row_of(it, x) >> p.group_shift,
                               q_full0 + 8 * x);
          }
          have = ok && next_item(r, it);
          if (have) {  // into L2 meanwhile
            place(it, rank, head);
            for (int x = 0; x < tiles_of(it); ++x)
              for (int c = 0; c < C::kCh; ++c)
                ptx::tma_prefetch_l2_3d(&maps.q[rank], c * 64, head, row_of(it, x) >> p.group_shift);
          }
        }
        // every load has landed before the CTA may end
        for (int x = 0; x < 2; ++x)
          if (n[x] > 0 && !ptx::mbar_wait(q_full0 + 8 * x, (n[x] - 1) & 1, p.wait_ns)) record(p.status, kDevTimeoutDrain);
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int x = (warp - 4) >> 2;
    const int qw = warp & 3;
    const int row = qw * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(qw * 32) << 16;
    const uint32_t sb = tmem + lane_off + static_cast<uint32_t>(x * 128);
    const uint32_t ob = tmem + lane_off + 256u + static_cast<uint32_t>(x * 128);
    const uint32_t s_full = s_full0 + 8 * x, p_full = p_full0 + 8 * x;
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
    // the next item with rows in this tile
    auto next_rows = [&](int &r, Item &i) {
      while (next_item(r, i))
        if (has(i, x)) return true;
      return false;
    };
    Item it, next;
    int r;
    bool have = first_item(r, it), more = false;
    if (have && !has(it, x)) have = next_rows(r, it);
    for (; ok && have; it = next, have = more) {
      const int m_row = row_of(it, x) + row;  // row of the set: token * group + head
      const bool there = m_row < rows;
      const int token = there ? m_row >> p.group_shift : 0;
      // the row sees keys [w0, pos] and [0, sinks)
      const int pos = p.keys - p.tokens + token;
      const int w0 = pos >= p.window ? pos - p.window + 1 : 0;
      float m = -INFINITY, l = 0.f;
      for (int j = it.j0; j < it.j1; ++j, ++gs) {
        // the block's columns: its window run's up to 16 wu, its first tokens' from there to 16 n
        const int n = it.units(j), wu = max(0, min(8, it.k.w_units - 8 * j));
        const int k0 = it.k.w0 + 128 * j;  // key of column 0 of the window run
        const int hi = min(pos - k0 + 1, 16 * wu), lo = w0 - k0, first = p.sinks - k0;  // seen: i < hi and (i >= lo or i < first)
        const int ls = -it.k.first(j);                                                 // seen of the first tokens: i >= ls
        if (j + 1 == it.j1) more = next_rows(r, next);  // while S is on its way
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
            if (__all_sync(0xffffffffu, hi >= 32 * h + 32 && lo <= 32 * h)) continue;
            const uint32_t see = (low_bits(hi - 32 * h) & (~low_bits(lo - 32 * h) | low_bits(first - 32 * h))) |
                                 (low_bits(16 * n - 32 * h) & ~low_bits(ls - 32 * h));
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see & (1u << i))) v[32 * h + i] = __float_as_uint(-INFINITY);
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
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const int k = 32 * h + i;
              float y0, y1;
              unpack2(fma2(pack2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), c2, nm2), y0, y1);
              const float a0 = ex2(y0), a1 = ex2(y1);
              sum2 = add2(sum2, pack2(a0, a1));
              pk[i >> 1] = pack_bf16(a0, a1);
            }
            ptx::tmem_st_16cols(sb + 16 * h, pk);
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
      // the output of the tile's item before has read its l
      if (nact > 0 && !wait_all(o_free0 + 8 * x, (nact - 1) & 1)) {
        ok = false;
        break;
      }
      ++nact;
      row_l[x * 128 + row] = l;
      if (p.split > 1 && there) p.part_ml[(static_cast<long long>(it.split) * p.sets + it.set) * rows + m_row] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(l_full0 + 8 * x);
    }
  } else {
    // ---- output: warp w has TMEM lanes [32 * (w % 4), +32) of both tiles ----
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOthers));
    const int qw = warp & 3;
    const int row = qw * 32 + lane;
    uint32_t nact[2] = {0, 0};
    bool ok = true;
    Item it;
    int r;
    for (bool have = first_item(r, it); ok && have; have = next_item(r, it)) {
      for (int x = 0; x < 2; ++x) {
        if (!has(it, x)) continue;
        const int m_row = row_of(it, x) + row;
        const bool there = m_row < rows;
        const uint32_t ob = tmem + (static_cast<uint32_t>(qw * 32) << 16) + 256u + static_cast<uint32_t>(x * 128);
        const int token = there ? m_row >> p.group_shift : 0;
        const int head = it.set * p.group + (m_row & (p.group - 1)), rank = it.set * p.group / p.heads_per_rank;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.a[rank]) + token * p.a_ld[rank] +
                             static_cast<long long>(head - rank * p.heads_per_rank) * D;
        const bool ready = ptx::mbar_wait_asleep(l_full0 + 8 * x, nact[x] & 1, p.wait_ns) &&
                           ptx::mbar_wait(o_full0 + 8 * x, nact[x] & 1, p.wait_ns);
        if (!__all_sync(0xffffffffu, ready)) {
          if (lane == 0) {
            if (*abort_flag == 0) record(p.status, kDevTimeoutEpilogue);
            *abort_flag = 1;
          }
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        ++nact[x];
        const bool split = p.split > 1;
        const float inv = split ? 1.f : 1.f / row_l[x * 128 + row];
        float *part = split ? p.part_o + ((static_cast<long long>(it.split) * p.sets + it.set) * rows + m_row) * D : nullptr;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {  // a lane its row: the lines fill up in L2
          uint32_t v[32];
          ptx::tmem_ld_32cols(ob + c * 32, v);
          ptx::tmem_ld_wait();
          ptx::tmem_regs_ready(v);
          if (c == D / 32 - 1) {  // O has been read
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(o_free0 + 8 * x);
          }
          if (!there) continue;
          if (split) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4 *>(part + c * 32 + 4 * i) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16(__uint_as_float(v[8 * i + 2 * e]) * inv, __uint_as_float(v[8 * i + 2 * e + 1]) * inv);
              *reinterpret_cast<uint4 *>(dst + c * 32 + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

constexpr int kJoinThreads = 256;

// Joins the splits: one warp a row (token and head).
template <int D, int TILES>
__global__ void __launch_bounds__(kJoinThreads) k_window_join(const __grid_constant__ WindowParams p) {
  constexpr int kPer = D / 32;
  grid_dep_wait();
  grid_dep_launch();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const long long all = static_cast<long long>(p.sets) * p.rows;
  if (row >= all) return;
  const int set = static_cast<int>(row / p.rows), m_row = static_cast<int>(row - static_cast<long long>(set) * p.rows);
  const int blocks = keys_of_part<TILES>(p, m_row / (128 * TILES)).blocks;
  float acc[kPer];
  const float l = join_splits<D>(p.part_ml, p.part_o, all, row, min(p.split, blocks), lane, acc);
  const int token = m_row >> p.group_shift, head = set * p.group + (m_row & (p.group - 1)), rank = head / p.heads_per_rank;
  __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.a[rank]) + token * p.a_ld[rank] +
                       static_cast<long long>(head - rank * p.heads_per_rank) * D + lane * kPer;
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t *>(dst + i) = pack_bf16(acc[i] * inv, acc[i + 1] * inv);
}

// Row tiles and key splits of an item: the least time of the busiest CTA and the join, with 1.5 us a block step
// of two tiles and 1.35 of one, 5 us for an item's start and end, 3 us for the join and its traffic at 4
// TB/s. Two tiles and no splits where those items fill the SMs. One token, 64 heads, 4100 keys: 17 splits, 9.8 us (one:
// 50); 515 tokens, 32 heads, 513 keys in sight: items of one tile 12.8, of two 14.3, in two splits 25.
struct Shape {
  int tiles, parts, split;
};
Shape shape_of(int group, int sets, int tokens, int keys, int window, int sinks, long long d) {
  const int sms = num_sms();
  const long long rows = static_cast<long long>(tokens) * group;
  Shape best = {2, static_cast<int>((rows + 255) / 256), 1};
  if (static_cast<long long>(best.parts) * sets >= sms) return best;
  double least = -1;
  for (int tiles = 2; tiles >= 1; --tiles) {
    const int per = 128 * tiles, parts = static_cast<int>((rows + per - 1) / per);
    const long long bases = static_cast<long long>(parts) * sets;
    const int most = keys_of(static_cast<int>(static_cast<long long>(per) * (parts - 1) / group), tokens - 1, tokens, keys, window, sinks).blocks;
    for (int c = 1; c <= most && bases * c <= 2LL * sms; ++c) {
      double us = (bases * c + sms - 1) / sms * ((most + c - 1) / c * (tiles == 2 ? 1.5 : 1.35) + 5);
      if (c > 1) us += 3 + 8e-6 / 4 * rows * sets * c * d;
      if (least < 0 || us < least) {
        least = us;
        best = {tiles, parts, c};
      }
    }
  }
  return best;
}

// Heads that share a tile.
int group_of(const tp_dims &d) {
  const int a = d.num_q_heads / d.num_kv_heads, b = d.num_q_heads / d.tp_size;
  int g = 1;
  while (g < 128 && a % (2 * g) == 0 && b % (2 * g) == 0) g *= 2;
  return g;
}

// Sizes that the item arithmetic takes in 32 bits.
bool sizes_ok(const tp_dims &d, long long tokens, long long keys) {
  return (d.head_dim == 64 || d.head_dim == 128) && d.tp_size <= kWinRanks && tokens <= (1LL << 28) / d.num_q_heads &&
         keys <= 0x7fffffffLL - 256;
}

template <int D, int TILES>
tp_status launch_window(const WindowParams &p, const WindowMaps &maps, cudaStream_t s) {
  static unsigned mask = 0;
  static std::mutex mu;
  const cudaError_t e = allow_smem(k_window<D, TILES>, static_cast<int>(WinCfg<D>::kSmem), mask, mu);
  if (e != cudaSuccess) return cuda_fail(e);
  const long long items = static_cast<long long>(p.sets) * p.parts * p.split;
  const unsigned grid = static_cast<unsigned>(items < num_sms() ? items : num_sms());
  tp_status st = launched(launch_kernel(k_window<D, TILES>, dim3(grid), dim3(kWinThreads), WinCfg<D>::kSmem, s, 1, p, maps));
  if (st != TP_OK || p.split == 1) return st;
  const long long all = static_cast<long long>(p.sets) * p.rows;
  return launched(launch_kernel(k_window_join<D, TILES>, dim3(static_cast<unsigned>((all + kJoinThreads / 32 - 1) / (kJoinThreads / 32))),
                                dim3(kJoinThreads), 0, s, 1, p));
}

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
  const int group = group_of(d);
  const Shape shape = shape_of(group, d.num_q_heads / group, static_cast<int>(tokens), static_cast<int>(keys), window, sinks, d.head_dim);
  return workspace_bytes_of(shape.split, tokens * d.num_q_heads, d.head_dim);
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
  const int group = group_of(dims), sets = dims.num_q_heads / group;
  const long long rows_all = T * dims.num_q_heads;
  const Shape shape = T > 0 ? shape_of(group, sets, static_cast<int>(T), static_cast<int>(S), window, sinks, hd) : Shape{2, 0, 1};
  const size_t need = workspace_bytes_of(shape.split, rows_all, hd);
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
  static thread_local WindowMaps maps;  // 20 KB: kept off the stack
  std::memset(&p, 0, sizeof(p));
  for (int r = 0; r < n; ++r) {
    tp_tensor qr = q[r];
    if (T == 1) qr.ld = qc;  // the pitch of a single row is free
    if (!encode_heads_map(&maps.q[r], qr, static_cast<int>(hd), group, 128 / group)) return TP_ERR_INVALID_ARG;
    p.a[r] = a[r].ptr;
    p.a_ld[r] = a[r].ld;
  }
  // Sources that are neighbouring columns of one tensor need one map together.
  p.one_map = S == 1 || (k[0].ld >= kvc * sources && v[0].ld >= kvc * sources);
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
  while ((1 << p.group_shift) < group) ++p.group_shift;
  p.sets = sets;
  p.sets_per_kv = sets / dims.num_kv_heads;
  p.heads_per_rank = dims.num_q_heads / n;
  p.heads_per_source = dims.num_kv_heads / sources;
  p.rows = static_cast<int>(T * group);
  p.parts = shape.parts;
  p.split = shape.split;
  p.by_sets.set(sets);
  p.by_split.set(shape.split);
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(hd)));
  p.part_o = static_cast<float *>(workspace);
  p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + sums_bytes(shape.split, rows_all, hd));
  p.status = ctx.status;
  p.wait_ns = ctx.wait_ns;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (shape.tiles == 1) return hd == 128 ? launch_window<128, 1>(p, maps, s) : launch_window<64, 1>(p, maps, s);
  return hd == 128 ? launch_window<128, 2>(p, maps, s) : launch_window<64, 2>(p, maps, s);
}
