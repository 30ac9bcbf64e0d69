// Rotary positions of q and k with one or several axes. For pair i of a head with the values
// (a, b), at token t:
//   angle = position[axis(i)][t] * freq[i],  a' = a cos - b sin,  b' = a sin + b cos
// (inverse: the angle negated, which turns the gradient back). The pairs are (i, i + pairs) or
// (2i, 2i + 1); values past 2 * pairs are copied.
//
// Bound by memory: every value is read and written once. A thread owns a token and a few pairs
// (those of one 16-byte piece), takes their sines and cosines into registers, and walks the
// heads of its CTA's share of q and k, two heads' pieces in flight: neither a table nor a
// barrier stands between the loads and the stores. Values that do not turn have threads of their own.
// 8192 tokens of 72 heads of 128 (302 MB): 51 us, 6.0 TB/s; with four heads in flight a thread 57,
// with the values that do not turn copied by the threads of those that do 2047 f32 tokens, half of
// whose values turn, 7.9 us in place of 5.3.
//
// Angles. In f32 the angle of position 10^6 is off by 0.03 already. A turn is therefore a
// 64-bit fixed-point fraction: F = freq / (2 pi) mod 1 in units of 2^-64, once a CTA and pair, and
// position * F wraps by itself as an integer product, whatever the position's sign. F is the frequency's 24-bit
// significand times the digits of 1 / (2 pi) from its exponent on (M. Payne and R. Hanek, "Radian reduction for
// trigonometric functions", 1983), off by little more than a unit, so a turn by 2^-33 at position 2^31; its upper 32 bits go on
// as f32. A 64-bit float product is off by 2^-52 of the angle (5e-5 at frequency 100 and position 2^31); one of two
// 64-bit floats is not, but takes longer (2047 f32 tokens 6.1 us, 5.3 here).
#include <cmath>
#include <type_traits>

#include "op_util.h"

namespace tpgqa {
namespace {

using namespace op;

constexpr int kRotThreads = 256;
constexpr int kMaxPairs = 256, kMaxAxes = 8, kRotRanks = 32;
constexpr int kHeadsInFlight = 2;

struct RotaryParams {
  const int *positions;  // [axes][tokens]
  const float *freq;
  int tokens, pairs, still, d;      // still: pieces of a head that are copied
  int heads_q, heads_kv;            // 0: not given
  int heads_per_rank, heads_per_source, heads_per_cta;
  int inverse;
  const void *in[2 * kRotRanks];    // q of the ranks, then k of the sources
  void *out[2 * kRotRanks];
  long long ld_in[2 * kRotRanks], ld_out[2 * kRotRanks];
  uint8_t axis[kMaxPairs];
};

// E neighbouring values as f32: E * sizeof(T) is 16 (one load) or E is 1.
template <typename T, int E>
struct Piece;
template <typename T>
struct Piece<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T *p) { raw = *p; }
  __device__ __forceinline__ void store(T *p) const { *p = raw; }
  __device__ __forceinline__ float get(int) const { return static_cast<float>(raw); }
  __device__ __forceinline__ void set(int, float x) { raw = static_cast<T>(x); }
};
template <>
struct Piece<float, 4> {
  float v[4];
  __device__ __forceinline__ void load(const float *p) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  }
  __device__ __forceinline__ void store(float *p) const { *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]); }
  __device__ __forceinline__ float get(int i) const { return v[i]; }
  __device__ __forceinline__ void set(int i, float x) { v[i] = x; }
};
template <>
struct Piece<__nv_bfloat16, 8> {
  __nv_bfloat162 v[4];
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(v); }
  __device__ __forceinline__ float get(int i) const { return i & 1 ? __high2float(v[i >> 1]) : __low2float(v[i >> 1]); }
  __device__ __forceinline__ void set(int i, float x) {
    if (i & 1) v[i >> 1].y = __float2bfloat16_rn(x);
    else v[i >> 1].x = __float2bfloat16_rn(x);
  }
};

// freq / (2 pi) modulo 1, in units of 2^-64, of a frequency below 2^56.
__device__ __forceinline__ unsigned long long turn_a_position(float freq) {
  const uint32_t bits = __float_as_uint(freq), field = bits >> 23 & 255;
  // freq = m * 2^e; the digits from 2^-(e + 96) up, of which those above 2^-e are whole turns and overflow
  const uint32_t m = (bits & 0x7fffff) | (field ? 0x800000 : 0);
  const int e = static_cast<int>(max(field, 1u)) - 150, down = max(32 - e, 0);
  // 2^128 / (2 pi) in 32-bit words, the lowest first, and its 96 bits from bit `down` up
  const uint32_t w[4] = {0x7d4d3770u, 0x7f09d5f4u, 0x9391054au, 0x28be60dbu};
  const int by = down >> 5;
  uint32_t x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = 0;
#pragma unroll
    for (int k = i; k < 4; ++k)
      if (k - i == by) x[i] = w[k];
  }
  const uint32_t d0 = __funnelshift_r(x[0], x[1], down), d1 = __funnelshift_r(x[1], x[2], down), d2 = __funnelshift_r(x[2], x[3], down);
  const unsigned long long turn = (static_cast<unsigned long long>(d2) << 32 | d1) * m + (static_cast<unsigned long long>(d0) * m >> 32);
  return bits >> 31 ? 0 - turn : turn;
}
// A turn's sine and cosine, the turn in units of 2^-64.
__device__ __forceinline__ void turn_sincos(unsigned long long turn, float *s, float *c) {
  const int top = static_cast<int>((turn + 0x80000000ull) >> 32);  // in [-2^31, 2^31): half turns of 2^-31
  sincospif(static_cast<float>(top) * 0x1p-31f, s, c);
}

template <typename T, int E, bool HALVES>
__global__ void __launch_bounds__(kRotThreads) k_rotary(const __grid_constant__ RotaryParams p) {
  __shared__ unsigned long long s_turn[kMaxPairs];
  grid_dep_wait();
  grid_dep_launch();
  for (int i = threadIdx.x; i < p.pairs; i += kRotThreads) s_turn[i] = turn_a_position(p.freq[i]);
  __syncthreads();
  // of a head: pieces that turn, E pairs each, then pieces of 2 E values that do not
  const int turning = p.pairs / E, pieces = turning + p.still;
  const long long item = static_cast<long long>(blockIdx.x) * kRotThreads + threadIdx.x;
  const long long t = item / pieces;
  if (t >= p.tokens) return;
  const int piece = static_cast<int>(item - t * pieces);
  const bool turns = piece < turning;
  float sn[E], cs[E];
  if (turns) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = piece * E + e;
      const long long pos = p.positions[static_cast<long long>(p.axis[i]) * p.tokens + t];
      turn_sincos(static_cast<unsigned long long>(pos) * s_turn[i], &sn[e], &cs[e]);
      if (p.inverse) sn[e] = -sn[e];
    }
  }
  const int heads = p.heads_q + p.heads_kv;
  const int h0 = blockIdx.y * p.heads_per_cta, h1 = min(heads, h0 + p.heads_per_cta);
  int at0 = HALVES ? piece * E : 2 * piece * E, at1 = HALVES ? p.pairs + piece * E : at0 + E;
  if (!turns) {
    at0 = 2 * p.pairs + 2 * E * (piece - turning);
    at1 = at0 + E < p.d ? at0 + E : at0;  // an odd last piece: its only half twice
  }
  // N heads from h on; their loads go out together
  auto heads_from = [&](int h, auto count) {
    constexpr int N = decltype(count)::value;
    Piece<T, E> x0[N], x1[N];
    T *dst[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const bool key = h + u >= p.heads_q;
      const int local = key ? h + u - p.heads_q : h + u, per = key ? p.heads_per_source : p.heads_per_rank;
      const int r = local / per, slot = key ? kRotRanks + r : r;
      const long long col = static_cast<long long>(local - r * per) * p.d;
      const T *src = static_cast<const T *>(p.in[slot]) + t * p.ld_in[slot] + col;
      dst[u] = static_cast<T *>(p.out[slot]) + t * p.ld_out[slot] + col;
      x0[u].load(src + at0);
      x1[u].load(src + at1);
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (turns) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          // value e of the first and of the second members: pieces of their own, or neighbours over both
          const int j = 2 * e;
          const float a = HALVES ? x0[u].get(e) : (j < E ? x0[u].get(j % E) : x1[u].get(j % E));
          const float b = HALVES ? x1[u].get(e) : (j + 1 < E ? x0[u].get((j + 1) % E) : x1[u].get((j + 1) % E));
          const float ra = a * cs[e] - b * sn[e], rb = a * sn[e] + b * cs[e];
          if (HALVES) {
            x0[u].set(e, ra);
            x1[u].set(e, rb);
          } else {
            if (j < E) x0[u].set(j % E, ra);
            else x1[u].set(j % E, ra);
            if (j + 1 < E) x0[u].set((j + 1) % E, rb);
            else x1[u].set((j + 1) % E, rb);
          }
        }
      }
      x0[u].store(dst[u] + at0);
      x1[u].store(dst[u] + at1);
    }
  };
  int h = h0;
  for (; h + kHeadsInFlight <= h1; h += kHeadsInFlight) heads_from(h, std::integral_constant<int, kHeadsInFlight>());
  for (; h < h1; ++h) heads_from(h, std::integral_constant<int, 1>());
}

template <typename T, int E>
tp_status launch_rotary(const RotaryParams &p, bool halves, dim3 grid, cudaStream_t s) {
  if (halves) return launched(launch_kernel(k_rotary<T, E, true>, grid, dim3(kRotThreads), 0, s, 1, p));
  return launched(launch_kernel(k_rotary<T, E, false>, grid, dim3(kRotThreads), 0, s, 1, p));
}

}  // namespace
}  // namespace tpgqa

using namespace tpgqa;
using namespace tpgqa::op;

extern "C" tp_status tp_rotary(const tp_plan *plan, int64_t tokens, const int32_t *positions, int32_t n_axes,
                               const float *freq, int32_t pairs, const int32_t *axis, int32_t layout, int32_t inverse,
                               const tp_tensor *q, const tp_tensor *k, tp_tensor *q_out, tp_tensor *k_out,
                               tp_stream_t stream) {
  tp_dims dims;
  tp_rank_shard sh;
  if (!plan || tp_plan_dims(plan, &dims) != TP_OK || tp_plan_query_rank(plan, 0, &sh) != TP_OK) return TP_ERR_INVALID_ARG;
  if ((!q && !k) || !q != !q_out || !k != !k_out || tokens < 0 || tokens > 0x7fffffffLL) return TP_ERR_INVALID_ARG;
  if (layout != TP_ROTARY_HALVES && layout != TP_ROTARY_NEIGHBOURS) return TP_ERR_INVALID_ARG;
  const int n = dims.tp_size;
  const long long hd = dims.head_dim;
  if (pairs < 1 || 2LL * pairs > hd || n_axes < 1) return TP_ERR_INVALID_ARG;
  if (n > kRotRanks || pairs > kMaxPairs || n_axes > kMaxAxes) return TP_ERR_UNSUPPORTED;
  for (int i = 0; axis && i < pairs; ++i)
    if (axis[i] < 0 || axis[i] >= n_axes) return TP_ERR_INVALID_ARG;
  const int sources = sh.kv_replicated ? 1 : n;
  const tp_tensor *first = q ? q : k;
  RotaryParams p = {};
  bool vec = true, in_place = true;
  auto take = [&](const tp_tensor *in, const tp_tensor *out, int count, long long heads, int slot) -> tp_status {
    for (int r = 0; r < count; ++r) {
      for (const tp_tensor *t : {in + r, out + r}) {
        if (!view_ok(*t)) return TP_ERR_INVALID_ARG;
        if (t->dtype != first->dtype || (t->dtype != TP_F32 && t->dtype != TP_BF16)) return TP_ERR_DTYPE;
        if (t->rows != tokens || t->cols != heads * hd) return TP_ERR_INVALID_ARG;
        if (!elem_aligned(*t)) return TP_ERR_ALIGNMENT;
        vec = vec && vec_aligned(*t);
      }
      if (tokens > 1 && in[r].ptr == out[r].ptr && in[r].ld != out[r].ld) return TP_ERR_INVALID_ARG;  // rows would meet others
      in_place = in_place && in[r].ptr == out[r].ptr;
      p.in[slot + r] = in[r].ptr;
      p.out[slot + r] = out[r].ptr;
      p.ld_in[slot + r] = in[r].ld;
      p.ld_out[slot + r] = out[r].ld;
    }
    return TP_OK;
  };
  p.heads_per_rank = dims.num_q_heads / n;
  p.heads_per_source = dims.num_kv_heads / sources;
  tp_status st;
  if (q && (st = take(q, q_out, n, p.heads_per_rank, 0)) != TP_OK) return st;
  if (k && (st = take(k, k_out, sources, p.heads_per_source, kRotRanks)) != TP_OK) return st;
  if (tokens > 0 && (!positions || !freq)) return TP_ERR_INVALID_ARG;
  if (!ptr_aligned(positions, 4) || !ptr_aligned(freq, 4)) return TP_ERR_ALIGNMENT;
  if ((st = check_rank_health(n)) != TP_OK) return st;
  if (tokens == 0) return TP_OK;
  p.positions = positions;
  p.freq = freq;
  p.tokens = static_cast<int>(tokens);
  p.pairs = pairs;
  p.d = static_cast<int>(hd);
  p.heads_q = q ? dims.num_q_heads : 0;
  p.heads_kv = k ? dims.num_kv_heads : 0;
  p.inverse = inverse != 0;
  for (int i = 0; i < pairs; ++i) p.axis[i] = static_cast<uint8_t>(axis ? axis[i] : 0);
  const int per16 = first->dtype == TP_F32 ? 4 : 8;
  vec = vec && pairs % per16 == 0 && hd % per16 == 0;
  const int e = vec ? per16 : 1;
  // Heads are spread over CTAs until there are about eight CTAs an SM; with 16 CTAs an SM more angles
  // are taken than that gains.
  p.still = in_place ? 0 : static_cast<int>((hd - 2 * pairs + 2 * e - 1) / (2 * e));
  const long long blocks = (tokens * (pairs / e + p.still) + kRotThreads - 1) / kRotThreads;
  const int heads = p.heads_q + p.heads_kv;
  if (blocks > 0x7fffffffLL) return TP_ERR_UNSUPPORTED;
  long long share = 8LL * num_sms() / blocks;
  if (share < 1) share = 1;
  if (share > heads) share = heads;
  p.heads_per_cta = static_cast<int>((heads + share - 1) / share);
  const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((heads + p.heads_per_cta - 1) / p.heads_per_cta));
  const bool halves = layout == TP_ROTARY_HALVES;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (first->dtype == TP_F32) return vec ? launch_rotary<float, 4>(p, halves, grid, s) : launch_rotary<float, 1>(p, halves, grid, s);
  return vec ? launch_rotary<__nv_bfloat16, 8>(p, halves, grid, s) : launch_rotary<__nv_bfloat16, 1>(p, halves, grid, s);
}
