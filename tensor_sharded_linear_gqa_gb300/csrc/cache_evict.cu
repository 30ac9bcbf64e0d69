// Eviction from the sequences' caches by accumulated attention weight.
//
// Per (sequence, kv head): of the positions between the first n_first and the
// last n_recent, the m = budget - n_first - n_recent with the largest weight
// stay (equal weights: the lower position). The threshold, the m-th largest
// weight, is found by a radix selection over the weights' order-preserving 32-bit
// keys (three passes of 11, 11 and 10 bits, one histogram in shared memory each),
// which reads each weight from shared memory and needs no sort. A second pass
// over the positions in order turns "above the threshold" and "the first few
// equal to it" into output places by a block-wide prefix sum, so the kept
// positions come out in rising order.
//
// The move of the K and V rows is a gather bound by memory: 2 d bytes per (row,
// head), each read and written once. In place (outputs = inputs) one CTA owns a
// column slice of a (sequence, head) and walks the kept rows upwards in chunks:
// a row's new place is never above its old one, so a chunk whose loads have all
// returned can be stored without touching a row that a later chunk reads.
#include "op_util.h"

namespace tpgqa {
namespace {

using namespace op;

constexpr int kMaxSources = 32;
constexpr int kSelThreads = 512;
constexpr int kSelPer = 4;                          // positions per thread and chunk
constexpr int kSelChunk = kSelThreads * kSelPer;
constexpr int kBins = 2048;                         // 11 bits a pass
constexpr int kMaxSmemKeys = 48 * 1024;             // keys held in shared memory (192 KB); longer caches re-read

struct EvictParams {
  const void *k[kMaxSources], *v[kMaxSources];
  void *k_out[kMaxSources], *v_out[kMaxSources];
  const float *weight[kMaxSources];
  float *weight_out[kMaxSources];
  long long k_ld[kMaxSources], v_ld[kMaxSources], ko_ld[kMaxSources], vo_ld[kMaxSources];
  long long w_ld[kMaxSources], wo_ld[kMaxSources];
  const int *lengths;
  int *lengths_out, *kept, *status;
  long long cap, cap_out;  // rows per sequence of the caches read and written
  long long wo_cols;       // columns of weight_out
  int places;              // places a sequence can fill: min(budget, cap)
  int chunks;              // of them per sequence in the gather's grid
  int batch, heads, sources, budget, n_first, n_recent, d, keys_in_smem;
};

// Larger weight, larger key; NaN lowest, -0 with +0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sums of two counters over the CTA's threads, and their totals.
__device__ __forceinline__ void block_scan2(int a, int b, int &ea, int &eb, int &ta, int &tb) {
  __shared__ int2 part[kSelThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ua = __shfl_up_sync(0xffffffffu, ia, o), ub = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += ua;
      ib += ub;
    }
  }
  if (lane == 31) part[warp] = make_int2(ia, ib);
  __syncthreads();
  int2 p = lane < kSelThreads / 32 ? part[lane] : make_int2(0, 0);
  int pa = p.x, pb = p.y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ua = __shfl_up_sync(0xffffffffu, pa, o), ub = __shfl_up_sync(0xffffffffu, pb, o);
    if (lane >= o) {
      pa += ua;
      pb += ub;
    }
  }
  ta = __shfl_sync(0xffffffffu, pa, 31);
  tb = __shfl_sync(0xffffffffu, pb, 31);
  const int ba = __shfl_sync(0xffffffffu, pa, warp) - __shfl_sync(0xffffffffu, p.x, warp);
  const int bb = __shfl_sync(0xffffffffu, pb, warp) - __shfl_sync(0xffffffffu, p.y, warp);
  ea = ba + ia - a;
  eb = bb + ib - b;
  __syncthreads();  // part may be written again
}

// Exclusive prefix sum of one counter over the CTA's threads. The next use of `part`
// comes after another barrier of the caller's.
__device__ __forceinline__ int block_scan(int a, int *part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int ia = a;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, ia, o);
    if (lane >= o) ia += u;
  }
  if (lane == 31) part[warp] = ia;
  __syncthreads();
  int p = lane < warp ? part[lane] : 0;  // the warps before this one
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
  return __shfl_sync(0xffffffffu, p, 0) + ia - a;
}

// One CTA per (sequence, source, head): kept positions and weights. A cache of one
// chunk keeps its weights and keys in registers from the first read on; a longer one
// its keys in shared memory, or, beyond that, reads the weights again. Bound by
// latency: about ten barriers and three dependent reads, some 7 us before the gather
// whatever the number of caches that one wave holds (256 threads with eight positions
// each issue half the instructions and take as long).
__global__ void __launch_bounds__(kSelThreads) k_evict_select(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t s_keys[];
  __shared__ __align__(16) int s_hist[kBins];
  __shared__ int s_bin, s_above, s_part[kSelThreads / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x;
  const int h = blockIdx.x % p.heads, src = (blockIdx.x / p.heads) % p.sources;
  const int b = blockIdx.x / (p.heads * p.sources);
  const int given = p.lengths[b];
  const int cap = static_cast<int>(p.cap);
  if ((given < 0 || given > cap) && tid == 0) atomicCAS(p.status, 0, kDevBadLength);
  const int len = min(max(given, 0), cap);
  const long long wrow = static_cast<long long>(b) * p.heads + h;
  const float *w = p.weight[src] + wrow * p.w_ld[src];
  float *wo = p.weight_out[src] + wrow * p.wo_ld[src];
  int *kept = p.kept + (static_cast<long long>(src) * p.batch * p.heads + wrow) * p.budget;
  const int n_new = min(len, p.budget);

  if (len > p.budget) {
    const int lo = p.n_first, hi = len - p.n_recent;  // candidates [lo, hi)
    int want = p.budget - p.n_first - p.n_recent;     // of them stay; hi - lo > want
    const bool one = len <= kSelChunk;
    float val[kSelPer];
    uint32_t key[kSelPer];
    auto read_chunk = [&](int c0) {
#pragma unroll
      for (int i = 0; i < kSelPer; ++i) {
        const int j = c0 + tid * kSelPer + i;
        val[i] = j < len ? w[j] : 0.0f;
        key[i] = weight_key(val[i]);
      }
    };
    if (one) {
      read_chunk(0);
    } else if (p.keys_in_smem) {
      for (int j = tid; j < len; j += kSelThreads) s_keys[j] = weight_key(w[j]);
    }
    uint32_t prefix = 0;
    int equal = 0;  // how many of the keys equal to the threshold stay
    if (want > 0) {
#pragma unroll
      for (int pass = 0; pass < 3; ++pass) {
        // digits of 11, 11 and 10 bits; a key counts while its higher digits are the threshold's
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bins = pass == 2 ? 1024 : 2048;
        const uint32_t mask = pass == 0 ? 0u : (pass == 1 ? 0xffe00000u : 0xfffffc00u);
        for (int i = tid * 4; i < kBins; i += kSelThreads * 4) *reinterpret_cast<int4 *>(s_hist + i) = make_int4(0, 0, 0, 0);
        __syncthreads();
        auto count = [&](uint32_t k) {
          if ((k & mask) == prefix) atomicAdd(&s_hist[(k >> shift) & (bins - 1)], 1);
        };
        if (one) {
#pragma unroll
          for (int i = 0; i < kSelPer; ++i) {
            const int j = tid * kSelPer + i;
            if (j >= lo && j < hi) count(key[i]);
          }
        } else {
          for (int j = lo + tid; j < hi; j += kSelThreads) count(p.keys_in_smem ? s_keys[j] : weight_key(w[j]));
        }
        __syncthreads();
        // thread t owns the four bins below bins - 4t: a prefix sum from the top
        const int top = bins - 1 - tid * 4;
        int c[4] = {0, 0, 0, 0};
        if (top >= 0) {
          const int4 v = *reinterpret_cast<const int4 *>(s_hist + top - 3);
          c[0] = v.w; c[1] = v.z; c[2] = v.y; c[3] = v.x;
        }
        const int sum = c[0] + c[1] + c[2] + c[3];
        const int before = block_scan(sum, s_part);
        // the bin in which the want-th largest lies
        if (before < want && before + sum >= want) {
          int above = before;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (above < want && above + c[i] >= want) {
              s_bin = top - i;
              s_above = above;
              break;
            }
            above += c[i];
          }
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(s_bin) << shift;
        want -= s_above;
      }
      equal = want;
    }
    const bool none = p.budget == p.n_first + p.n_recent;
    // Places, in position order. weight_out may be weight: a chunk's weights are
    // read before any of its places (all at or below their positions) is written.
    int kept_before = 0, equal_before = 0;
    for (int c0 = 0; c0 < len; c0 += kSelChunk) {
      if (!one) read_chunk(c0);
      bool sure[kSelPer], tie[kSelPer];
      int n_sure = 0, n_tie = 0;
#pragma unroll
      for (int i = 0; i < kSelPer; ++i) {
        const int j = c0 + tid * kSelPer + i;
        const bool forced = j < lo || j >= hi;
        sure[i] = j < len && (forced || (!none && key[i] > prefix));
        tie[i] = j < len && !forced && !none && key[i] == prefix;
        n_sure += sure[i];
        n_tie += tie[i];
      }
      int es, et, ts, tt;
      block_scan2(n_sure, n_tie, es, et, ts, tt);  // its barriers also close the chunk's reads
      int ties = equal_before + et;  // ties before this position
      int place = kept_before + es + min(ties, equal) - min(equal_before, equal);
#pragma unroll
      for (int i = 0; i < kSelPer; ++i) {
        const int j = c0 + tid * kSelPer + i;
        bool keep = sure[i];
        if (tie[i]) {
          keep = ties < equal;
          ++ties;
        }
        if (keep) {
          kept[place] = j;
          wo[place] = val[i];
          ++place;
        }
      }
      kept_before += ts + min(equal_before + tt, equal) - min(equal_before, equal);
      equal_before += tt;
    }
  } else {
    for (int j = tid; j < len; j += kSelThreads) {
      kept[j] = j;
      wo[j] = w[j];
    }
  }
  for (int j = n_new + tid; j < p.budget; j += kSelThreads) kept[j] = -1;
  __syncthreads();  // in place: every weight has been read
  for (long long j = n_new + tid; j < p.wo_cols; j += kSelThreads) wo[j] = 0.0f;
}

// Sequence b's new length, written after the selection (this grid waited for it),
// so lengths_out may be lengths.
__device__ __forceinline__ void write_length(const EvictParams &p, int b) {
  p.lengths_out[b] = min(min(max(p.lengths[b], 0), static_cast<int>(p.cap)), p.budget);
}

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;    // rows in flight per thread, gather
constexpr int kPlaceUnroll = 4;   // the same, in place

// Gather into another buffer. CTA: (sequence, chunk of kept places) with (source,
// head, K or V) fastest, so that the heads of a row, which lie side by side in
// memory, are read and written at about the same time; a thread keeps one 16-byte
// piece of the head's row and steps over the places, four loads in flight. Each
// CTA waits twice (for kept, then for the rows), so full occupancy, 32 registers a
// thread, carries it: when that was set, 64 caches of up to 2048 keys (8 kv heads of
// 128) went to 1024 in 93 us in all, against 104 with eight loads a thread and 126
// with sixteen at the occupancy that those leave. It is 91 us now, 5.7 TB/s; the
// gather alone takes 81 at 72% of DRAM's peak. Rows are read and written once:
// streaming accesses.
__global__ void __launch_bounds__(kMoveThreads, 8) k_evict_gather(const __grid_constant__ EvictParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const int lanes = p.d / 8;  // 16-byte pieces of a head's row
  const int columns = 2 * p.sources * p.heads;
  const int group = blockIdx.x / columns, column = blockIdx.x - group * columns;
  const int b = group / p.chunks, chunk = group - b * p.chunks;
  const int src = (column >> 1) % p.sources, h = (column >> 1) / p.sources;
  const bool is_v = column & 1;
  if (column == 0 && chunk == 0 && threadIdx.x == 0) write_length(p, b);
  const int rows = kMoveThreads / lanes;
  const int piece = threadIdx.x % lanes, row0 = threadIdx.x / lanes;
  if (row0 >= rows) return;
  const long long in_ld = (is_v ? p.v_ld[src] : p.k_ld[src]) * 2, out_ld = (is_v ? p.vo_ld[src] : p.ko_ld[src]) * 2;
  const long long col = (static_cast<long long>(h) * lanes + piece) * 16;
  const char *in = static_cast<const char *>(is_v ? p.v[src] : p.k[src]) + b * p.cap * in_ld + col;
  char *out = static_cast<char *>(is_v ? p.v_out[src] : p.k_out[src]) + b * p.cap_out * out_ld + col;
  const int *kept =
      p.kept + (static_cast<long long>(src) * p.batch * p.heads + static_cast<long long>(b) * p.heads + h) * p.budget;
  const int c0 = chunk * rows * kMoveUnroll;
  int from[kMoveUnroll];
  uint4 x[kMoveUnroll];
#pragma unroll
  for (int i = 0; i < kMoveUnroll; ++i) {
    const int place = c0 + i * rows + row0;
    from[i] = place < p.places ? __ldg(kept + place) : -1;
  }
#pragma unroll
  for (int i = 0; i < kMoveUnroll; ++i)
    if (from[i] >= 0) x[i] = __ldcs(reinterpret_cast<const uint4 *>(in + from[i] * in_ld));
#pragma unroll
  for (int i = 0; i < kMoveUnroll; ++i)
    if (from[i] >= 0) __stcs(reinterpret_cast<uint4 *>(out + (c0 + i * rows + row0) * out_ld), x[i]);
}

// In place: CTA x = (sequence, source, head, K or V), y = one 64-byte column slice
// of the head. The barrier separates a chunk's loads from its stores.
__global__ void __launch_bounds__(kMoveThreads) k_evict_in_place(const __grid_constant__ EvictParams p) {
  grid_dep_wait();
  grid_dep_launch();
  const bool is_v = blockIdx.x & 1;
  const int unit = blockIdx.x >> 1;
  const int h = unit % p.heads, src = (unit / p.heads) % p.sources, b = unit / (p.heads * p.sources);
  if (blockIdx.y == 0 && !is_v && h == 0 && src == 0 && threadIdx.x == 0) write_length(p, b);
  const int lanes = p.d / 8, first = blockIdx.y * 4, width = min(4, lanes - first);
  char *buf = static_cast<char *>(is_v ? p.v_out[src] : p.k_out[src]);
  const long long ld = (is_v ? p.vo_ld[src] : p.ko_ld[src]) * 2;
  buf += b * p.cap * ld + (static_cast<long long>(h) * lanes + first) * 16;
  const int *kept =
      p.kept + (static_cast<long long>(src) * p.batch * p.heads + static_cast<long long>(b) * p.heads + h) * p.budget;
  const int piece = threadIdx.x % 4, row0 = threadIdx.x / 4;
  constexpr int kRows = kMoveThreads / 4;
  for (int c0 = 0; c0 < p.places; c0 += kRows * kPlaceUnroll) {
    if (kept[c0] < 0) break;  // rising, then -1: nothing further to move (same for every thread)
    uint4 x[kPlaceUnroll];
    int from[kPlaceUnroll];
#pragma unroll
    for (int i = 0; i < kPlaceUnroll; ++i) {
      const int place = c0 + i * kRows + row0;
      from[i] = place < p.places && piece < width ? kept[place] : -1;
      if (from[i] == place) from[i] = -1;  // stays where it is
      if (from[i] >= 0) x[i] = *reinterpret_cast<uint4 *>(buf + from[i] * ld + piece * 16);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPlaceUnroll; ++i)
      if (from[i] >= 0) *reinterpret_cast<uint4 *>(buf + (c0 + i * kRows + row0) * ld + piece * 16) = x[i];
  }
}

}  // namespace
}  // namespace tpgqa

using namespace tpgqa;
using namespace tpgqa::op;

extern "C" tp_status tp_cache_evict(const tp_plan *plan, int64_t batch, const int32_t *lengths, const tp_tensor *k,
                                    const tp_tensor *v, const tp_tensor *weight, int32_t budget, int32_t n_first,
                                    int32_t n_recent, tp_tensor *k_out, tp_tensor *v_out, tp_tensor *weight_out,
                                    int32_t *lengths_out, int32_t *kept, tp_stream_t stream) {
  tp_dims dims;
  tp_rank_shard sh;
  if (!plan || tp_plan_dims(plan, &dims) != TP_OK || tp_plan_query_rank(plan, 0, &sh) != TP_OK) return TP_ERR_INVALID_ARG;
  if (!k || !v || !weight || !k_out || !v_out || !weight_out || batch < 0) return TP_ERR_INVALID_ARG;
  if (budget < 1 || n_first < 0 || n_recent < 0 || static_cast<long long>(n_first) + n_recent > budget)
    return TP_ERR_INVALID_ARG;
  const int sources = sh.kv_replicated ? 1 : dims.tp_size;
  const long long heads = sh.kv_head_end - sh.kv_head_begin, d = dims.head_dim, cols = heads * d;
  if (sources > kMaxSources || d % 8 != 0) return TP_ERR_UNSUPPORTED;
  if (d > 2048 || 2 * heads * sources > 65535 || batch > 0x7fffffff / (2 * heads * sources))
    return TP_ERR_UNSUPPORTED;  // a head's row within one CTA's threads; grid sizes
  if (batch > 0 && (!lengths || !lengths_out || !kept)) return TP_ERR_INVALID_ARG;
  if (!ptr_aligned(lengths, 4) || !ptr_aligned(lengths_out, 4) || !ptr_aligned(kept, 4)) return TP_ERR_ALIGNMENT;
  const long long cap = batch ? k[0].rows / batch : 0, cap_out = batch ? k_out[0].rows / batch : 0;
  const long long need = budget < cap ? budget : cap;  // rows that a sequence can keep
  bool same = true, apart = true;  // outputs are the inputs for every source / for none
  for (int r = 0; r < sources; ++r) {
    const tp_tensor *in[2] = {&k[r], &v[r]}, *out[2] = {&k_out[r], &v_out[r]};
    for (int i = 0; i < 2; ++i) {
      if (!view_ok(*in[i]) || !view_ok(*out[i])) return TP_ERR_INVALID_ARG;
      if (in[i]->dtype != TP_BF16 || out[i]->dtype != TP_BF16) return TP_ERR_DTYPE;
      if (in[i]->rows != batch * cap || in[i]->cols != cols || out[i]->rows != batch * cap_out || out[i]->cols != cols)
        return TP_ERR_INVALID_ARG;
      if ((in[i]->rows > 0 && !vec_aligned(*in[i])) || (out[i]->rows > 0 && !vec_aligned(*out[i]))) return TP_ERR_ALIGNMENT;
      const bool eq = in[i]->ptr == out[i]->ptr;
      if (eq && batch * cap > 0 && (in[i]->ld != out[i]->ld || cap != cap_out)) return TP_ERR_INVALID_ARG;
      same = same && eq;
      apart = apart && (!eq || batch * cap == 0);
    }
    if (!view_ok(weight[r]) || !view_ok(weight_out[r])) return TP_ERR_INVALID_ARG;
    if (weight[r].dtype != TP_F32 || weight_out[r].dtype != TP_F32) return TP_ERR_DTYPE;
    if (weight[r].rows != batch * heads || weight[r].cols != cap || weight_out[r].rows != batch * heads ||
        weight_out[r].cols < need || weight_out[r].cols != weight_out[0].cols)
      return TP_ERR_INVALID_ARG;
    if (!ptr_aligned(weight[r].ptr, 4) || !ptr_aligned(weight_out[r].ptr, 4)) return TP_ERR_ALIGNMENT;
    if (weight[r].ptr == weight_out[r].ptr && weight[r].ptr && weight[r].ld != weight_out[r].ld) return TP_ERR_INVALID_ARG;
  }
  if (!same && !apart) return TP_ERR_INVALID_ARG;  // in place for all of K and V, or for none
  if (cap_out < need) return TP_ERR_INVALID_ARG;
  const long long rows_per_cta = kMoveThreads / (d / 8) * kMoveUnroll;
  const long long chunks = need > 0 ? (need + rows_per_cta - 1) / rows_per_cta : 1;
  if (batch > 0 && chunks > 0x7fffffff / (batch * 2 * heads * sources)) return TP_ERR_UNSUPPORTED;
  tp_status st = check_rank_health(dims.tp_size);
  if (st != TP_OK) return st;
  if (batch == 0) return TP_OK;
  DevCtx ctx;
  const cudaError_t e = get_dev_ctx(&ctx);
  if (e != cudaSuccess) return cuda_fail(e);
  EvictParams p = {};
  for (int r = 0; r < sources; ++r) {
    p.k[r] = k[r].ptr;
    p.v[r] = v[r].ptr;
    p.k_out[r] = k_out[r].ptr;
    p.v_out[r] = v_out[r].ptr;
    p.k_ld[r] = k[r].ld;
    p.v_ld[r] = v[r].ld;
    p.ko_ld[r] = k_out[r].ld;
    p.vo_ld[r] = v_out[r].ld;
    p.weight[r] = static_cast<const float *>(weight[r].ptr);
    p.weight_out[r] = static_cast<float *>(weight_out[r].ptr);
    p.w_ld[r] = weight[r].ld;
    p.wo_ld[r] = weight_out[r].ld;
  }
  p.lengths = lengths;
  p.lengths_out = lengths_out;
  p.kept = kept;
  p.status = ctx.status;
  p.cap = cap;
  p.cap_out = cap_out;
  p.wo_cols = weight_out[0].cols;
  p.batch = static_cast<int>(batch);
  p.heads = static_cast<int>(heads);
  p.sources = sources;
  p.places = static_cast<int>(need);
  p.chunks = static_cast<int>(chunks);
  p.budget = budget;
  p.n_first = n_first;
  p.n_recent = n_recent;
  p.d = static_cast<int>(d);
  // keys in shared memory where a cache can lose keys, outgrows the registers and fits
  p.keys_in_smem = cap > budget && cap > kSelChunk && cap <= kMaxSmemKeys;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const size_t smem = p.keys_in_smem ? static_cast<size_t>(cap) * 4 : 0;
  cudaError_t ce = cudaFuncSetAttribute(k_evict_select, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmemKeys * 4);
  if (ce != cudaSuccess) return cuda_fail(ce);
  const unsigned units = static_cast<unsigned>(batch * sources * heads);
  st = launched(launch_kernel(k_evict_select, dim3(units), dim3(kSelThreads), smem, s, 1, p));
  if (st != TP_OK) return st;
  const int lanes = p.d / 8;
  if (same && cap > 0)
    return launched(launch_kernel(k_evict_in_place, dim3(units * 2, static_cast<unsigned>((lanes + 3) / 4)),
                                  dim3(kMoveThreads), 0, s, 1, p));
  return launched(launch_kernel(k_evict_gather, dim3(static_cast<unsigned>(batch * p.chunks * 2 * sources * heads)),
                                dim3(kMoveThreads), 0, s, 1, p));
}
