// Caches of keys and values held in 4 bits: storing, reading back, and attention of one new token
// per sequence over them.
//
// Format. The 32 neighbouring values of a head that form a group share a bf16 scale,
//   scale = bf16(max|x| / 7),  code = clamp(rint(x / scale), -8, 7) + 8,  value = (code - 8) * scale
// (all codes 8 where the scale is 0; a group with an infinity or a NaN has the scale NaN). Row (b * heads + h) * C + j
// of a kv source's tensors is position j of sequence b's head h: d/2 bytes of codes and d/32
// scales, 4.5 bits a value. A row's bytes are ordered for the attention kernel's registers: a
// group's 32 values are cut into pieces (4 of 8 values for keys, 8 of 4 for values), the row
// holds the first pieces of all groups, then the second ones, and so on, two codes a byte, the
// lower value's in the lower half.
//
// k_cache4_attn. The floor is reading the cache once: 4.5 bits a value leave 41 codes a clock and SM
// at the measured copy rate, so what counts is instructions a code; a warp's step of 32 keys, 8 heads of 128 has
// about 600, of which 32 are tensor products. Those are m16n8k16 with the KEYS as
// rows: S^T = K q^T (16 keys x 8 heads), O^T += V^T P^T (16 dims x 8 heads). A group of 8 heads then
// fills a product, where rows of heads would leave half of it empty, and both operands that come
// from the cache are A fragments made in registers:
//   K  a word of 8 codes gives four f16 pairs by one shift and four masks: the code's bits in the
//      low mantissa bits are the subnormal code * 2^-24, or 16 times it, which q makes good
//      (f16, scaled by a power of two for each head so that its largest value is near 2^14). No -8 is
//      taken off the codes: the accumulators start at -8 * sum(q). Products of one group
//      share the key's scale, which multiplies the accumulators, not the codes.
//   V  codes of two keys are paired by byte permutes, 0x4300 | code is the bf16 128 + code, and
//      136 is taken off exactly. The values' scales multiply p before it is rounded to bf16,
//      once a group; movmatrix turns it from S^T's layout into the B operand's.
// A warp walks 32 keys at a time by itself, through its own ring of cp.async stages; its m, l
// and O are joined with the other warps' at the end of the CTA's keys. Where they are few, the CTAs
// of a (sequence, kv head) are a cluster and join their sums through distributed shared memory; else
// they leave them in memory for k_cache4_join. Either way they share a sequence's keys evenly.
//
// Measured: 64 sequences of 5000 to 16384 keys, 64 heads on 8 (790 MB): 142 us, 5.6 TB/s, 0.83 of the copy rate;
// issue slots 58% busy, the integer pipe 55%, the tensor cores 25%. Three CTAs of four warps an SM: when
// that took 153 us, four CTAs (128 registers) took 159 and CTAs of three warps 173. Other ways to the operands: V's
// -136 as a product of its own 167 for 157 us, shifts as products 167 to 172, K's codes as e4m3 numbers
// 185 for 151. Short caches are bound by starts and ends (about 7 us a CTA): 61 sequences with up to
// 1028 keys in sight 20.4 us (floor 9.7), one of 577 4.6 us. Heads of 64: the long batch 91 us (floor 59), the short
// caches 14.5 (4.8).
#include <cuda_fp16.h>

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

constexpr int kC4Ranks = 32;
constexpr int kGroup = 32;  // values that share a scale

struct Cache4 {
  uint8_t *k_codes[kC4Ranks], *v_codes[kC4Ranks];
  __nv_bfloat16 *k_scale[kC4Ranks], *v_scale[kC4Ranks];
};

// The codes at bits 0-3 and 16-19 of w, less 8, as a bf16 pair: 0x4300 | code is 128 + code, and 136 goes off
// exactly.
__device__ __forceinline__ uint32_t bf16_codes(uint32_t w) {
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(r) : "r"(w));  // (w & a) | b
  const uint32_t off = 0xc308c308u;  // -136 twice
  const __nv_bfloat162 x = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&r), *reinterpret_cast<const __nv_bfloat162 *>(&off));
  return *reinterpret_cast<const uint32_t *>(&x);
}

// ---------------------------------------------------------------------------
// Storing and reading back. A thread has 32 values of a row, whose codes are 16 neighbouring bytes: 8 of
// each of four groups (d = 128) or 16 of each of two (d = 64). Bound by memory and, nearly as much, by
// issue (slots 66% busy): 16384 tokens of 8 heads take 31.8 us to store and read back (172 MB, 5.4 TB/s; heads of 64 21.9), 51
// with 8 neighbouring values a thread, whose addresses and scales cost as much and whose codes are words apart.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;

struct CopyParams {
  Cache4 cache;
  const void *in[2][kC4Ranks];   // store: keys and values; load: unused
  void *out[2][kC4Ranks];        // load: keys and values
  long long ld[2][kC4Ranks];
  const int *starts, *counts;
  int batch, n, cap, heads_kv, heads_per_source;
  Divider by_heads, by_source;
  int *status;
};

// A thread's four chunks of 8 values: chunk i of thread c of a row.
template <int D>
__device__ __forceinline__ constexpr int chunk_group(int i) { return D == 128 ? i : i >> 1; }
template <int D>
__device__ __forceinline__ int chunk_at(int i, int c) { return D == 128 ? i * kGroup + c * 8 : (i >> 1) * kGroup + c * 16 + (i & 1) * 8; }
// The 16 bytes of a row from the chunks' codes (8 a word), and back. Both are their own inverses: words change
// places (K, d = 64), or halves of words, the two pieces of 4 values (V).
template <int D>
__device__ __forceinline__ uint4 k_order(const uint4 &w) { return D == 128 ? w : make_uint4(w.x, w.z, w.y, w.w); }
template <int D>
__device__ __forceinline__ uint4 v_to_row(const uint4 &w) {
  const uint32_t a = D == 128 ? w.y : w.z, b = D == 128 ? w.z : w.y;  // what lies beside the first and the last chunk's codes
  const uint32_t p0 = __byte_perm(w.x, a, 0x5410), p1 = __byte_perm(w.x, a, 0x7632);
  const uint32_t p2 = __byte_perm(b, w.w, 0x5410), p3 = __byte_perm(b, w.w, 0x7632);
  return D == 128 ? make_uint4(p0, p2, p1, p3) : make_uint4(p0, p1, p2, p3);
}
template <int D>
__device__ __forceinline__ uint4 v_from_row(const uint4 &w) {
  const uint32_t p0 = w.x, p1 = D == 128 ? w.z : w.y, p2 = D == 128 ? w.y : w.z, p3 = w.w;
  const uint32_t x = __byte_perm(p0, p1, 0x5410), a = __byte_perm(p0, p1, 0x7632);
  const uint32_t b = __byte_perm(p2, p3, 0x5410), last = __byte_perm(p2, p3, 0x7632);
  return D == 128 ? make_uint4(x, a, b, last) : make_uint4(x, b, a, last);
}

// Rows of sequence blockIdx.z: n tokens by heads, the heads of a token neighbours.
struct RowAt {
  int i, src, h;  // token, kv source, head of the source
};
__device__ __forceinline__ RowAt row_at(int row, const CopyParams &p) {
  RowAt r;
  r.i = p.by_heads.of(row);
  const int kv = row - r.i * p.heads_kv;
  r.src = p.by_source.of(kv);
  r.h = kv - r.src * p.heads_per_source;
  return r;
}

// x / s rounded to f32, which the definition asks for and a product with r = 1 / s does not give where
// x / s lies halfway between two codes: one step of Newton's method on the product's remainder.
__device__ __forceinline__ float rounded_quotient(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The scale of a group whose largest size has these bf16 bits.
__device__ __forceinline__ __nv_bfloat16 scale_of(uint32_t bits) {
  const float top = __uint_as_float(bits << 16);
  // below, f32's smallest values are near: up by 2^80 for the division
  const bool tiny = top < 0x1p-60f;
  float q = rounded_quotient(tiny ? top * 0x1p80f : top, 7.f, 1.f / 7.f);
  if (tiny) q *= 0x1p-80f;
  return __float2bfloat16_rn(bits >= 0x7f80u ? NAN : q);  // infinities and NaN
}
// 8 codes of 8 values. TINY: the scale is so small that it has no reciprocal, and the group goes up by 2^80.
template <bool TINY>
__device__ __forceinline__ uint32_t codes_of(const uint4 &v, float s) {
  if (TINY) s *= 0x1p80f;
  float r = rcp_approx(s);
  if (!(s > 0.f)) s = r = 0.f;  // all codes 8
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    float c = rounded_quotient(TINY ? x * 0x1p80f : x, s, r);
    if (TINY) c = fminf(fmaxf(c, -8.f), 7.f);  // elsewhere |c| < 7.1: a scale is off by 2^-8 at most
    // 1.5 * 2^23 + 8 + c rounds c to even and has the code in its low bits; what it has above them
    // adds up to a constant over the eight
    codes += __float_as_uint(c + 12582920.f) * (1u << (4 * i));
  }
  return codes - 0x4b400000u * 0x11111111u;  // of 1.5 * 2^23
}

template <int D>
__global__ void __launch_bounds__(kCopyThreads) k_cache4_store(const __grid_constant__ CopyParams p) {
  constexpr int G = D / kGroup, kPer = D / 32;  // groups, threads a row
  constexpr int kRows = kCopyThreads / kPer;    // rows of a CTA
  grid_dep_wait();
  grid_dep_launch();
  const int which = blockIdx.y, b = blockIdx.z;  // keys or values; sequence
  const int c = threadIdx.x % kPer, row = blockIdx.x * kRows + threadIdx.x / kPer;
  const int start = p.starts[b], given = p.counts ? p.counts[b] : p.n;
  const bool start_ok = start >= 0 && start <= p.cap;
  const int count = start_ok ? min(min(max(given, 0), p.n), p.cap - start) : 0;
  if ((!start_ok || count != given) && blockIdx.x == 0 && which == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, kDevBadLength);
  const RowAt r = row_at(row, p);
  const bool there = row < p.n * p.heads_kv && r.i < count;
  uint4 v[4] = {};
  if (there) {
    const __nv_bfloat16 *from = static_cast<const __nv_bfloat16 *>(p.in[which][r.src]) +
                                (static_cast<long long>(b) * p.n + r.i) * p.ld[which][r.src] + r.h * D;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4 *>(from + chunk_at<D>(i, c));
  }
  // the groups' largest sizes as bf16 bits, in whose order infinities and then NaN come last; two groups a word
  uint32_t m[G];
#pragma unroll
  for (int g = 0; g < G; ++g) m[g] = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu), __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
    m[chunk_group<D>(i)] = __vmaxu2(m[chunk_group<D>(i)], x);
  }
  uint32_t pair[G / 2];
#pragma unroll
  for (int g = 0; g < G; g += 2) {
    uint32_t x = __vmaxu2(__byte_perm(m[g], m[g + 1], 0x5410), __byte_perm(m[g], m[g + 1], 0x7632));
#pragma unroll
    for (int o = 1; o < kPer; o *= 2) x = __vmaxu2(x, __shfl_xor_sync(0xffffffffu, x, o));
    pair[g / 2] = x;
  }
  if (!there) return;
  __nv_bfloat162 scale[G / 2];
#pragma unroll
  for (int g = 0; g < G / 2; ++g) scale[g] = __halves2bfloat162(scale_of(pair[g] & 0xffffu), scale_of(pair[g] >> 16));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = chunk_group<D>(i);
    const float one = __bfloat162float(g & 1 ? scale[g / 2].y : scale[g / 2].x);
    if (one < 0x1p-60f && one > 0.f)
      w[i] = codes_of<true>(v[i], one);
    else
      w[i] = codes_of<false>(v[i], one);
  }
  const uint4 codes = make_uint4(w[0], w[1], w[2], w[3]);
  const long long to = (static_cast<long long>(b) * p.heads_per_source + r.h) * p.cap + start + r.i;
  *reinterpret_cast<uint4 *>((which ? p.cache.v_codes : p.cache.k_codes)[r.src] + to * (D / 2) + c * 16) =
      which ? v_to_row<D>(codes) : k_order<D>(codes);
  if (c == 0) {
    __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>((which ? p.cache.v_scale : p.cache.k_scale)[r.src] + to * G);
    if (G == 4)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(*reinterpret_cast<const uint32_t *>(&scale[0]), *reinterpret_cast<const uint32_t *>(&scale[G / 2 - 1]));
    else
      dst[0] = scale[0];
  }
}

template <int D, typename T>
__global__ void __launch_bounds__(kCopyThreads) k_cache4_load(const __grid_constant__ CopyParams p) {
  constexpr int G = D / kGroup, kPer = D / 32;
  constexpr int kRows = kCopyThreads / kPer;
  grid_dep_wait();
  grid_dep_launch();
  const int which = blockIdx.y, b = blockIdx.z;
  const int c = threadIdx.x % kPer, row = blockIdx.x * kRows + threadIdx.x / kPer;
  const int start = p.starts[b];
  if ((start < 0 || start > p.cap) && blockIdx.x == 0 && which == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, kDevBadLength);
  if (row >= p.n * p.heads_kv) return;
  const RowAt r = row_at(row, p);
  uint4 codes = make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u);
  uint32_t scale[G / 2] = {};
  if (start >= 0 && r.i < p.cap - start) {  // positions that do not exist are zeros
    const long long from = (static_cast<long long>(b) * p.heads_per_source + r.h) * p.cap + start + r.i;
    codes = *reinterpret_cast<const uint4 *>((which ? p.cache.v_codes : p.cache.k_codes)[r.src] + from * (D / 2) + c * 16);
    codes = which ? v_from_row<D>(codes) : k_order<D>(codes);
    const uint32_t *s = reinterpret_cast<const uint32_t *>((which ? p.cache.v_scale : p.cache.k_scale)[r.src] + from * G);
    if (G == 4) {
      const uint2 two = *reinterpret_cast<const uint2 *>(s);
      scale[0] = two.x, scale[G / 2 - 1] = two.y;
    } else {
      scale[0] = *s;
    }
  }
  T *dst = static_cast<T *>(p.out[which][r.src]) + (static_cast<long long>(b) * p.n + r.i) * p.ld[which][r.src] + r.h * D;
  const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int g = chunk_group<D>(i);
    uint32_t pr[4];  // codes e and e + 4, less 8, as bf16 (exact)
#pragma unroll
    for (int e = 0; e < 4; ++e) pr[e] = bf16_codes(w[i] >> (4 * e));
    if (sizeof(T) == 4) {
      const float s = g & 1 ? bf16_hi(scale[g / 2]) : bf16_lo(scale[g / 2]);
      float4 *to = reinterpret_cast<float4 *>(dst + chunk_at<D>(i, c));
      to[0] = make_float4(bf16_lo(pr[0]) * s, bf16_lo(pr[1]) * s, bf16_lo(pr[2]) * s, bf16_lo(pr[3]) * s);
      to[1] = make_float4(bf16_hi(pr[0]) * s, bf16_hi(pr[1]) * s, bf16_hi(pr[2]) * s, bf16_hi(pr[3]) * s);
    } else {
      const uint32_t twice = __byte_perm(scale[g / 2], 0, g & 1 ? 0x3232 : 0x1010);
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // one rounding of the product
        const __nv_bfloat162 x = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&pr[e]), *reinterpret_cast<const __nv_bfloat162 *>(&twice));
        pr[e] = *reinterpret_cast<const uint32_t *>(&x);
      }
      *reinterpret_cast<uint4 *>(dst + chunk_at<D>(i, c)) = make_uint4(__byte_perm(pr[0], pr[1], 0x5410), __byte_perm(pr[2], pr[3], 0x5410),
                                                                       __byte_perm(pr[0], pr[1], 0x7632), __byte_perm(pr[2], pr[3], 0x7632));
    }
  }
}

// ---------------------------------------------------------------------------
// Attention.
// ---------------------------------------------------------------------------
constexpr int kAttnWarps = 4, kAttnThreads4 = 32 * kAttnWarps;
constexpr int kTileKeys = 32;  // keys of a warp's step: two products' rows
constexpr int kStages = 3;     // of a ring: 143 us on the long batch, with two 145 and with four 144
constexpr int kOrdered = 256;  // sequences that are put in order at most

struct Attn4Params {
  Cache4 cache;
  int batch, cap, heads_q, heads_kv, group, heads_per_rank, heads_per_source;
  int window, sinks;
  int chunk;               // without clusters: tiles a split has at most
  int splits;              // CTAs of a (sequence, kv head) and head tile
  int cluster;             // whether they are a cluster
  int longest_first;       // the order in which the sequences' CTAs start; else as they come
  float scale_log2;
  const int *lengths;
  float *part_o;    // [split][row][d], rows kv head by kv head
  float2 *part_ml;  // [split][row]: m (log2 units), l
  int *status;
  const void *q[kC4Ranks];
  long long q_ld[kC4Ranks];
  void *a[kC4Ranks];
  long long a_ld[kC4Ranks];
};

// The 32-key tiles that a sequence's new token sees: those of the first tokens, then those of the
// window. One run from 0 where the two meet.
struct Tiles {
  int sink_tiles, first, count;
  __device__ __forceinline__ int at(int j) const { return j < sink_tiles ? j : j - sink_tiles + first; }
};
__device__ __forceinline__ Tiles tiles_of(int len, int window, int sinks) {
  const int w0 = len > window ? len - window : 0;
  Tiles t;
  t.first = w0 / kTileKeys;
  const int st = (min(sinks, w0) + kTileKeys - 1) / kTileKeys;
  t.sink_tiles = min(st, t.first);
  t.count = len > 0 ? t.sink_tiles + (len + kTileKeys - 1) / kTileKeys - t.first : 0;
  return t;
}
__device__ __forceinline__ int splits_here(const Tiles &t, int chunk) { return (t.count + chunk - 1) / chunk; }

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void cp_small_or_zero(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(there ? N : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// D = A B + C, 16 x 8 x 16.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
__device__ __forceinline__ void mma_bf(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int D>
struct Attn4Cfg {
  static constexpr int kG = D / kGroup;
  static constexpr int kRow = D / 2;                             // bytes of a row of codes
  static constexpr int kV = kTileKeys * kRow, kKs = 2 * kV;      // stage: K codes, V codes, K scales, V scales
  static constexpr int kVs = kKs + kTileKeys * 2 * kG;
  static constexpr int kStage = kVs + kTileKeys * 2 * kG;
  static constexpr int kWarp = kStages * kStage;
  static constexpr int kJoinRow = D + 4;                         // floats of a head's sums while warps are joined
  // Where a tile's K row lies in a stage: rows j and j + 4, read by neighbouring rows of a fragment,
  // are no multiple of 128 bytes apart.
  static __device__ __forceinline__ int k_slot(int row) { return row ^ (D == 128 ? row >> 2 & 1 : row >> 1 & 2); }
  // Where byte `in` of a V row lies: rows 2, 3 mod 4 have their halves exchanged.
  static __device__ __forceinline__ int v_in(int row, int in) { return D == 128 ? in ^ ((row >> 1 & 1) * 32) : in; }
};
template <int D, int NT>
constexpr int attn4_smem() {
  const int sums = kAttnWarps * 8 * NT * Attn4Cfg<D>::kJoinRow * 4, ring = kAttnWarps * Attn4Cfg<D>::kWarp;
  return sums > ring ? sums : ring;
}

// The sequence whose CTAs have the place-th most tiles (those with the same number in order). All threads of
// the CTA; s_key has kOrdered entries.
__device__ __forceinline__ int sequence_at(int place, const Attn4Params &p, int *s_key) {
  __shared__ int s_found;  // not in the ring, which the first warps fill while others read it
  for (int i = threadIdx.x; i < kOrdered; i += kAttnThreads4) {
    int key = -1;
    if (i < p.batch) {
      const Tiles t = tiles_of(min(max(p.lengths[i], 0), p.cap), p.window, p.sinks);
      const int n = splits_here(t, p.chunk);
      key = (n > 0 ? (t.count + n - 1) / n : 0) * kOrdered + (kOrdered - 1 - i);
    }
    s_key[i] = key;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.batch; i += kAttnThreads4) {
    const int key = s_key[i];
    int before = 0;
#pragma unroll 4
    for (int j = 0; j < p.batch; j += 4) {
      const int4 o = *reinterpret_cast<const int4 *>(s_key + j);
      before += (o.x > key) + (o.y > key) + (o.z > key) + (o.w > key);
    }
    if (before == place) s_found = i;
  }
  __syncthreads();
  return s_found;
}

// NT: products of 8 heads a key fragment serves (the CTA has up to 8 NT heads of the group).
template <int D, int NT>
__global__ void __launch_bounds__(kAttnThreads4, NT == 1 ? 3 : 2) k_cache4_attn(const __grid_constant__ Attn4Params p) {
  using C = Attn4Cfg<D>;
  constexpr int G = C::kG;
  extern __shared__ __align__(128) uint8_t smem[];  // 16 bytes past a line: 147 us in place of 143
  __shared__ float2 s_ml[kAttnWarps][8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  const int unit = blockIdx.x / p.splits, split = blockIdx.x - unit * p.splits;
  const int place = unit / p.heads_kv, kv = unit - place * p.heads_kv;
  const int h0 = blockIdx.y * 8 * NT;  // first head of the group here
  grid_dep_wait();
  grid_dep_launch();
  const int b = p.longest_first ? sequence_at(place, p, reinterpret_cast<int *>(smem)) : place;
  const int given = p.lengths[b], len = min(max(given, 0), p.cap);
  if (given != len && kv == 0 && split == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicCAS(p.status, 0, kDevBadLength);
  const Tiles tl = tiles_of(len, p.window, p.sinks);
  const int n_splits = p.cluster ? (len > 0 ? p.splits : 0) : splits_here(tl, p.chunk);
  if (split >= n_splits) {  // a whole cluster, or a split that this sequence has not
    if (len > 0 || split > 0) return;
    // no key at all: the heads' outputs are zero
    for (int i = threadIdx.x; i < 8 * NT * (D / 2); i += kAttnThreads4) {
      const int g = h0 + i / (D / 2);
      if (g >= p.group) break;
      const int head = kv * p.group + g, rank = head / p.heads_per_rank;
      reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.a[rank]) + b * p.a_ld[rank] +
                                   static_cast<long long>(head - rank * p.heads_per_rank) * D)[i % (D / 2)] = 0;
    }
    return;
  }
  const int t0 = static_cast<int>(static_cast<long long>(tl.count) * split / n_splits);
  const int t1 = static_cast<int>(static_cast<long long>(tl.count) * (split + 1) / n_splits);
  const int w0 = len > p.window ? len - p.window : 0;

  const int src = kv / p.heads_per_source;
  const long long row0 = (static_cast<long long>(b) * p.heads_per_source + (kv - src * p.heads_per_source)) * p.cap;
  // this lane's first pieces: 16 bytes of codes of row lane / kLanes, the scales of row lane
  constexpr int kLanes = C::kRow / 16, kRowsAtOnce = 32 / kLanes;
  const int my_row = lane / kLanes, my_in = lane % kLanes * 16;
  const uint8_t *k_codes = p.cache.k_codes[src] + row0 * C::kRow + lane * 16, *v_codes = p.cache.v_codes[src] + row0 * C::kRow + lane * 16;
  const __nv_bfloat16 *k_scale = p.cache.k_scale[src] + (row0 + lane) * G, *v_scale = p.cache.v_scale[src] + (row0 + lane) * G;
  const uint32_t ring = ptx::smem_addr(smem) + warp * C::kWarp;
  const uint32_t to_k = ring + C::k_slot(my_row) * C::kRow + my_in, to_v = ring + C::kV + my_row * C::kRow + C::v_in(my_row, my_in);
  const uint32_t to_s = ring + C::kKs + lane * 2 * G;

  // A tile's rows into a stage; rows that the token does not see are zeros (their scales too), so
  // that nothing stale is read, however it is encoded.
  auto seen = [&](int j) { return j < len && (j >= w0 || j < p.sinks); };
  auto whole = [&](int j0) { return j0 + kTileKeys <= len && (j0 >= w0 || j0 + kTileKeys <= p.sinks); };  // all rows are seen
  auto fetch = [&](int t, int stage) {
    if (t < t1) {
      const int j0 = tl.at(t) * kTileKeys;
      const uint32_t off = stage * C::kStage;
      const long long at = static_cast<long long>(j0) * C::kRow, at_s = static_cast<long long>(j0) * G;
      if (whole(j0)) {
#pragma unroll
        for (int i = 0; i < kTileKeys / kRowsAtOnce; ++i) {
          cp16(to_k + off + i * 512, k_codes + at + i * 512);
          cp16(to_v + off + i * 512, v_codes + at + i * 512);
        }
        cp_small<2 * G>(to_s + off, k_scale + at_s);
        cp_small<2 * G>(to_s + off + C::kVs - C::kKs, v_scale + at_s);
      } else {
#pragma unroll
        for (int i = 0; i < kTileKeys / kRowsAtOnce; ++i) {
          const bool there = seen(j0 + my_row + i * kRowsAtOnce);
          cp16_or_zero(to_k + off + i * 512, there ? k_codes + at + i * 512 : p.cache.k_codes[src], there);
          cp16_or_zero(to_v + off + i * 512, there ? v_codes + at + i * 512 : p.cache.v_codes[src], there);
        }
        const bool there = seen(j0 + lane);
        cp_small_or_zero<2 * G>(to_s + off, there ? k_scale + at_s : p.cache.k_scale[src], there);
        cp_small_or_zero<2 * G>(to_s + off + C::kVs - C::kKs, there ? v_scale + at_s : p.cache.v_scale[src], there);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(t0 + warp + i * kAttnWarps, i);

  // q of the heads as B fragments: step 2g + h of the product over group g takes, from thread c, the
  // values 8c + 2h, 8c + 2h + 4 (first pair) and 8c + 2h + 1, 8c + 2h + 5 (second), as the codes' masks
  // bring them up. The second pairs' codes are 16 times as large.
  uint32_t qf[NT][2 * G][2];
  float start[NT][G][2];  // the accumulators' first values: -8 * 2^-24 * sum of q over the group, heads 2c and 2c + 1
  float f[NT][2];         // log2(e) / sqrt(d) * 2^24 / the head's factor
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int g = h0 + 8 * nt + r;
    uint4 raw[G];
    float top = 0.f;
    const int head = kv * p.group + (g < p.group ? g : 0), rank = head / p.heads_per_rank;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q[rank]) + b * p.q_ld[rank] +
                             static_cast<long long>(head - rank * p.heads_per_rank) * D;
#pragma unroll
    for (int i = 0; i < G; ++i) {
      raw[i] = g < p.group ? *reinterpret_cast<const uint4 *>(q + i * kGroup + c * 8) : make_uint4(0, 0, 0, 0);
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[e])), fabsf(bf16_hi(w[e]))));
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // the power of two that brings the largest value into [2^14, 2^15); within [2^-100, 2^100] for the
    // factor's own range
    const int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    const int up = min(max(14 - ex, -100), 100);
    const float scale = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
    const float mine = p.scale_log2 * 0x1p24f * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
    f[nt][0] = __shfl_sync(0xffffffffu, mine, 8 * c);
    f[nt][1] = __shfl_sync(0xffffffffu, mine, 8 * c + 4);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      float x[8], sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = (e & 1 ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1])) * scale;
        // what the product will use: values far below the head's largest lose bits in f16
        x[e] = __half2float(__float2half_rn(e & 1 ? x[e] * 0.0625f : x[e]));
        sum += e & 1 ? 16.f * x[e] : x[e];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const __half2 pr = __floats2half2_rn(x[2 * h + e], x[2 * h + e + 4]);
          qf[nt][2 * i + h][e] = *reinterpret_cast<const uint32_t *>(&pr);
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum *= -8.f * 0x1p-24f;
      start[nt][i][0] = __shfl_sync(0xffffffffu, sum, 8 * c);
      start[nt][i][1] = __shfl_sync(0xffffffffu, sum, 8 * c + 4);
    }
  }

  float m[NT][2], l[NT][2], o[NT][2 * G][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    m[nt][0] = m[nt][1] = 0.f;
    l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * G; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
  }

  // Row r of a fragment's upper half is the product's key r/2 + 4 (r & 1), of its lower half that key
  // + 8: the pairs of keys (2c, 2c + 1) of the second product are then the rows c and c + 4, and
  // each of the values' loads takes four neighbouring rows.
  const int key = (r >> 1) + 4 * (r & 1);
  int stage = 0;
  // The heads 2 nt + e that have no reference yet, a bit each: until a tile has a score above -infinity theirs is 0,
  // and nothing is lost (every p is 0).
  uint32_t none = (1u << 2 * NT) - 1;
  for (int t = t0 + warp; t < t1; t += kAttnWarps) {
    cp_wait<kStages - 2>();
    __syncwarp();  // the tile has landed, and every lane has read the one before, whose stage is filled next
    fetch(t + (kStages - 1) * kAttnWarps, stage == 0 ? kStages - 1 : stage - 1);
    const uint8_t *st = smem + warp * C::kWarp + stage * C::kStage;
    stage = stage + 1 == kStages ? 0 : stage + 1;
    const int j0 = tl.at(t) * kTileKeys;
    // ---- scores ----
    float s[2][NT][4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t kw[2][G];
      float ks[2][G];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int row = key + 8 * u + 16 * half;
        const uint8_t *at = st + C::k_slot(key) * C::kRow + (8 * u + 16 * half) * C::kRow + c * 4 * G;
        if (G == 4) {
          const uint4 w = *reinterpret_cast<const uint4 *>(at);
          kw[u][0] = w.x, kw[u][1] = w.y, kw[u][2 % G] = w.z, kw[u][3 % G] = w.w;
          const uint2 v = *reinterpret_cast<const uint2 *>(st + C::kKs + row * 2 * G);
          ks[u][0] = bf16_lo(v.x), ks[u][1] = bf16_hi(v.x), ks[u][2 % G] = bf16_lo(v.y), ks[u][3 % G] = bf16_hi(v.y);
        } else {
          const uint2 w = *reinterpret_cast<const uint2 *>(at);
          kw[u][0] = w.x, kw[u][1] = w.y;
          const uint32_t v = *reinterpret_cast<const uint32_t *>(st + C::kKs + row * 2 * G);
          ks[u][0] = bf16_lo(v), ks[u][1] = bf16_hi(v);
        }
      }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const uint32_t a = kw[0][i], a8 = a >> 8, d = kw[1][i], d8 = d >> 8;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float acc[4] = {start[nt][i][0], start[nt][i][1], start[nt][i][0], start[nt][i][1]};
          mma_f16(acc, a & 0x000f000fu, d & 0x000f000fu, a & 0x00f000f0u, d & 0x00f000f0u, qf[nt][2 * i][0], qf[nt][2 * i][1], acc);
          mma_f16(acc, a8 & 0x000f000fu, d8 & 0x000f000fu, a8 & 0x00f000f0u, d8 & 0x00f000f0u, qf[nt][2 * i + 1][0],
                  qf[nt][2 * i + 1][1], acc);
#pragma unroll
          for (int e = 0; e < 4; ++e) s[half][nt][e] = i == 0 ? ks[e >> 1][0] * acc[e] : s[half][nt][e] + ks[e >> 1][i] * acc[e];
        }
      }
    }
    // less the reference maximum, in log2 units: p = 2^s
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[half][nt][e] = fmaf(s[half][nt][e], f[nt][e & 1], -m[nt][e & 1]);
    if (!whole(j0)) {
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (!seen(j0 + key + 8 * u + 16 * half))
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) s[half][nt][2 * u] = s[half][nt][2 * u + 1] = -INFINITY;
    }
    // p, and its sums; the references move when a sum says that some p is large, which is rare after
    // the first tile, whose maximum is the first reference
    float pr[2][NT][4], sum[NT][2];
    auto weights = [&]() {
      bool fine = true;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
          for (int e = 0; e < 4; ++e) pr[half][nt][e] = ex2(s[half][nt][e]);
#pragma unroll
        for (int e = 0; e < 2; ++e) sum[nt][e] = (pr[0][nt][e] + pr[0][nt][e + 2]) + (pr[1][nt][e] + pr[1][nt][e + 2]);
        fine = fine && sum[nt][0] + sum[nt][1] <= 1024.f;
      }
      return fine;
    };
    if (__any_sync(0xffffffffu, !weights() || none != 0)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(fmaxf(s[0][nt][e], s[0][nt][e + 2]), fmaxf(s[1][nt][e], s[1][nt][e + 2]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const uint32_t bit = 1u << (2 * nt + e);
          const bool had = !(none & bit), any = mx > -INFINITY;  // NaN are no references
          const float up = fmaxf(any ? mx : 0.f, had ? 0.f : -FLT_MAX), alpha = had ? ex2(-up) : 1.f;
          if (any) none &= ~bit;
          m[nt][e] += up;
          l[nt][e] *= alpha;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            s[half][nt][e] -= up;
            s[half][nt][e + 2] -= up;
          }
#pragma unroll
          for (int i = 0; i < 2 * G; ++i) {
            o[nt][i][e] *= alpha;
            o[nt][i][e + 2] *= alpha;
          }
        }
      weights();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      l[nt][0] += sum[nt][0];
      l[nt][1] += sum[nt][1];
    }
    // ---- values ----
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float vs[2][G];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint8_t *at = st + C::kVs + (key + 8 * u + 16 * half) * 2 * G;
        if (G == 4) {
          const uint2 w = *reinterpret_cast<const uint2 *>(at);
          vs[u][0] = bf16_lo(w.x), vs[u][1] = bf16_hi(w.x), vs[u][2 % G] = bf16_lo(w.y), vs[u][3 % G] = bf16_hi(w.y);
        } else {
          const uint32_t w = *reinterpret_cast<const uint32_t *>(at);
          vs[u][0] = bf16_lo(w), vs[u][1] = bf16_hi(w);
        }
      }
      uint32_t vw[4][G / 2];  // rows c, c + 4, c + 8, c + 12: keys 2c, 2c + 1, 2c + 8, 2c + 9 of the product
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint8_t *at = st + C::kV + c * C::kRow + (4 * u + 16 * half) * C::kRow + C::v_in(c, r * 2 * G);
        if (G == 4) {
          const uint2 w = *reinterpret_cast<const uint2 *>(at);
          vw[u][0] = w.x, vw[u][G / 2 - 1] = w.y;
        } else {
          vw[u][0] = *reinterpret_cast<const uint32_t *>(at);
        }
      }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pb[nt][0] = turn8x8(pack_bf16(pr[half][nt][0] * vs[0][i], pr[half][nt][1] * vs[0][i]));
          pb[nt][1] = turn8x8(pack_bf16(pr[half][nt][2] * vs[1][i], pr[half][nt][3] * vs[1][i]));
        }
        const uint32_t lo = __byte_perm(vw[0][i >> 1], vw[1][i >> 1], i & 1 ? 0x7632 : 0x5410);
        const uint32_t hi = __byte_perm(vw[2][i >> 1], vw[3][i >> 1], i & 1 ? 0x7632 : 0x5410);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a0 = bf16_codes(lo >> (8 * h)), a1 = bf16_codes(lo >> (8 * h + 4));
          const uint32_t a2 = bf16_codes(hi >> (8 * h)), a3 = bf16_codes(hi >> (8 * h + 4));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_bf(o[nt][2 * i + h], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
        }
      }
    }
  }
  cp_wait<0>();

  // ---- the warps' sums are joined through shared memory ----
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 4; x < 32; x *= 2) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], x);
      if (r == 0) s_ml[warp][8 * nt + 2 * c + e] = make_float2(none >> (2 * nt + e) & 1 ? -FLT_MAX : m[nt][e], l[nt][e]);
    }
  __syncthreads();  // the rings are free
  float *sums = reinterpret_cast<float *>(smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float *row = sums + (warp * 8 * NT + 8 * nt + 2 * c + e) * C::kJoinRow;
#pragma unroll
      for (int i = 0; i < G; ++i)  // values 4r .. 4r + 3 of group i
        *reinterpret_cast<float4 *>(row + i * kGroup + 4 * r) =
            make_float4(o[nt][2 * i][e], o[nt][2 * i][e + 2], o[nt][2 * i + 1][e], o[nt][2 * i + 1][e + 2]);
    }
  __syncthreads();
  constexpr int kAll = 8 * NT * (D / 4), kMine = (kAll + kAttnThreads4 - 1) / kAttnThreads4;  // float4s of the CTA's sums; a thread's
  float4 acc[kMine];
  float2 ml[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = k * kAttnThreads4 + threadIdx.x, hl = i / (D / 4), col = i % (D / 4) * 4;
    if (i >= kAll) break;
    float top = -FLT_MAX, sum = 0.f;
    acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_ml[w][hl].x);
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
      const float2 one = s_ml[w][hl];
      const float fw = ex2(one.x - top);
      const float4 v = *reinterpret_cast<const float4 *>(sums + (w * 8 * NT + hl) * C::kJoinRow + col);
      sum += fw * one.y;
      acc[k].x += fw * v.x;
      acc[k].y += fw * v.y;
      acc[k].z += fw * v.z;
      acc[k].w += fw * v.w;
    }
    ml[k] = make_float2(top, sum);
  }
  auto store = [&](int hl, int col, const float4 &v, float sum) {
    const int head = kv * p.group + h0 + hl, rank = head / p.heads_per_rank;
    const float inv = 1.f / sum;
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.a[rank]) + b * p.a_ld[rank] +
                         static_cast<long long>(head - rank * p.heads_per_rank) * D + col;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
  };
  if (n_splits > 1 && p.cluster) {
    // the CTA's sums in place of the warps', then every CTA joins a part of them
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = k * kAttnThreads4 + threadIdx.x, hl = i / (D / 4), col = i % (D / 4) * 4;
      if (i >= kAll) break;
      *reinterpret_cast<float4 *>(sums + hl * C::kJoinRow + col) = acc[k];
      if (col == 0) *reinterpret_cast<float4 *>(sums + hl * C::kJoinRow + D) = make_float4(ml[k].x, ml[k].y, 0.f, 0.f);
    }
    ptx::cluster_sync();
    const uint32_t mine = ptx::smem_addr(sums);
    for (int i = split * kAttnThreads4 + threadIdx.x; i < kAll; i += p.splits * kAttnThreads4) {
      const int hl = i / (D / 4), col = i % (D / 4) * 4;
      float4 v[8], m8[8];
#pragma unroll
      for (int r8 = 0; r8 < 8; ++r8) {
        const uint32_t at = ptx::mapa_shared(mine, r8 < p.splits ? r8 : 0) + hl * C::kJoinRow * 4;
        v[r8] = ptx::ld_shared_cluster_f4(at + col * 4);
        m8[r8] = ptx::ld_shared_cluster_f4(at + D * 4);
      }
      float top = -FLT_MAX, sum = 0.f;
      float4 all = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int r8 = 0; r8 < 8; ++r8) top = r8 < p.splits ? fmaxf(top, m8[r8].x) : top;
#pragma unroll
      for (int r8 = 0; r8 < 8; ++r8) {
        if (r8 >= p.splits) continue;
        const float fw = ex2(m8[r8].x - top);
        sum += fw * m8[r8].y;
        all.x += fw * v[r8].x;
        all.y += fw * v[r8].y;
        all.z += fw * v[r8].z;
        all.w += fw * v[r8].w;
      }
      if (h0 + hl < p.group) store(hl, col, all, sum);
    }
    ptx::cluster_sync();  // nothing is read of a CTA that has ended
    return;
  }
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int i = k * kAttnThreads4 + threadIdx.x, hl = i / (D / 4), col = i % (D / 4) * 4;
    if (i >= kAll || h0 + hl >= p.group) break;
    if (n_splits == 1) {
      store(hl, col, acc[k], ml[k].y);
    } else {
      const long long row = (static_cast<long long>(split) * p.batch + b) * p.heads_q + kv * p.group + h0 + hl;
      *reinterpret_cast<float4 *>(p.part_o + row * D + col) = acc[k];
      if (col == 0) p.part_ml[row] = ml[k];
    }
  }
}

// One warp a (sequence, head); those whose keys one CTA had are done already.
template <int D>
__global__ void __launch_bounds__(256) k_cache4_join(const __grid_constant__ Attn4Params p) {
  constexpr int kPer = D / 32;
  grid_dep_wait();
  grid_dep_launch();
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<long long>(p.batch) * p.heads_q) return;
  const int b = static_cast<int>(row / p.heads_q), head = static_cast<int>(row - static_cast<long long>(b) * p.heads_q);
  const Tiles tl = tiles_of(min(max(p.lengths[b], 0), p.cap), p.window, p.sinks);
  const int n = splits_here(tl, p.chunk);
  if (n < 2) return;
  float acc[kPer];
  const float l = join_splits<D>(p.part_ml, p.part_o, static_cast<long long>(p.batch) * p.heads_q, row, n, lane, acc);
  const int rank = head / p.heads_per_rank;
  __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.a[rank]) + b * p.a_ld[rank] +
                       static_cast<long long>(head - rank * p.heads_per_rank) * D + lane * kPer;
  const float inv = 1.f / l;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) *reinterpret_cast<uint32_t *>(dst + i) = pack_bf16(acc[i] * inv, acc[i + 1] * inv);
}

// CTAs a (sequence, kv head), and the tiles that each has at most.
struct Shape4 {
  int chunk, splits, cluster, longest_first, head_tiles, nt;
};
Shape4 shape4_of(const tp_dims &d, long long batch, long long cap, long long window, long long sinks) {
  Shape4 s;
  const int group = d.num_q_heads / d.num_kv_heads;
  s.nt = group > 8 ? 2 : 1;
  s.head_tiles = (group + 8 * s.nt - 1) / (8 * s.nt);
  long long tiles = (cap + kTileKeys - 1) / kTileKeys;
  if (window < cap) {
    // the first tokens' tiles and the window's, whose ends may both lie inside one
    const long long some = (window + kTileKeys - 1) / kTileKeys + 1 + (sinks + kTileKeys - 1) / kTileKeys;
    if (some < tiles) tiles = some;
  }
  const long long units = batch * d.num_kv_heads * s.head_tiles, room = (s.nt == 1 ? 3LL : 2LL) * num_sms();
  auto ctas = [&]() { return units * ((tiles + s.chunk - 1) / s.chunk); };
  // Up to 256 tiles (8192 keys) a CTA, halved while there is room on the SMs for more CTAs, down to a tile a
  // warp. Where CTAs start in the order of their length and there are two of them for each place, else 128:
  // 64 sequences of 5000 to 16384 keys, 8 heads: 142 us with 256 tiles, 150 with 128, 146 with
  // 256 as they come; 32 such ones 82 with 128, 91 with 256.
  s.chunk = batch <= kOrdered ? 256 : 128;
  while (s.chunk > kAttnWarps && ctas() < room) s.chunk /= 2;
  if (s.chunk > 128 && ctas() < 2 * room) s.chunk = 128;
  // At most 64 splits a sequence: one warp of the join reads all of a row's, eight at a time. One sequence of
  // 131072 keys: 1 kv head 18.7 us (128 splits 17.8, 256 26, 512 47), 4 kv heads 26.2 (128: 33.8); of 16384, 10.1
  // (128: 13.4). Only 2^20 keys of 1 or 2 kv heads would gain: 88 and 89 us, with 128 splits 53 and 76.
  while ((tiles + s.chunk - 1) / s.chunk > 64) s.chunk *= 2;
  s.splits = static_cast<int>((tiles + s.chunk - 1) / s.chunk);
  if (s.splits < 1) s.splits = 1;
  // Clusters where all of them are resident at once: one launch in place of two (577 keys of 4 heads 4.5 us
  // and 5.0). With more they wait for SMs to have room for a whole one (64 sequences of
  // 5000 to 16384 keys, 8 heads: 159 us and 151).
  int c = 2;
  while (c < s.splits) c *= 2;
  s.cluster = s.splits > 1 && c <= 8 && units * c <= room;
  if (s.cluster) s.splits = c;
  // 61 sequences with up to 1028 keys in sight: 20.5 us, 21.8 as they come; 128 of 1 to 4096 keys: 64 and 74
  s.longest_first = !s.cluster && batch <= kOrdered && units * s.splits > room;
  return s;
}

template <int D, int NT>
tp_status launch_attn4(const Attn4Params &p, dim3 grid, cudaStream_t s) {
  static std::mutex mu;
  static unsigned mask = 0;
  constexpr int kSmem = attn4_smem<D, NT>();
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  {
    std::lock_guard<std::mutex> g(mu);
    if (dev >= 32 || !(mask & (1u << dev))) {
      e = cudaFuncSetAttribute(k_cache4_attn<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e == cudaSuccess)  // room for as many CTAs as the registers hold
        e = cudaFuncSetAttribute(k_cache4_attn<D, NT>, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
      if (e != cudaSuccess) return cuda_fail(e);
      if (dev < 32) mask |= 1u << dev;
    }
  }
  return launched(launch_kernel(k_cache4_attn<D, NT>, grid, dim3(kAttnThreads4), kSmem, s, p.cluster ? p.splits : 1, p));
}

size_t sums_bytes(const Shape4 &s, long long rows, long long d) { return s.splits > 1 && !s.cluster ? round256(static_cast<size_t>(s.splits) * rows * d * 4) : 0; }
size_t workspace_bytes_of(const Shape4 &s, long long rows, long long d) {
  return s.splits > 1 && !s.cluster ? sums_bytes(s, rows, d) + round256(static_cast<size_t>(s.splits) * rows * 8) : 0;
}

// Head sizes that the format's layouts cover, and capacities whose positions are in range.
bool cache_ok(const tp_dims &d, long long cap) {
  return (d.head_dim == 64 || d.head_dim == 128) && d.tp_size <= kC4Ranks && cap <= 0x7fffffffLL - 256;
}
// The attention's own: a row is a (sequence, q head), and its grid has up to 64 splits of each.
bool attn_sizes_ok(const tp_dims &d, long long batch, long long cap) {
  return cache_ok(d, cap) && batch <= (1LL << 23) / d.num_q_heads && d.num_q_heads / d.num_kv_heads <= 65535;
}

// The four tensors of a kv source's cache.
tp_status check_cache(const tp_tensor *t, int sources, long long rows, long long cols, int32_t dtype) {
  for (int r = 0; r < sources; ++r) {
    if (t[r].dtype != dtype) return TP_ERR_DTYPE;
    if (t[r].rows != rows || t[r].cols != cols || (rows > 1 && t[r].ld != cols)) return TP_ERR_INVALID_ARG;
    if (rows > 0 && !t[r].ptr) return TP_ERR_INVALID_ARG;
    // 16-byte pieces of codes; a row's scales at once
    if (!ptr_aligned(t[r].ptr, dtype == TP_U8 ? 16 : 2 * cols)) return TP_ERR_ALIGNMENT;
  }
  return TP_OK;
}

struct Given {
  tp_dims dims;
  int n, sources;
  long long hd, heads, cap;  // heads of a source, positions of a sequence
};
tp_status check_call(const tp_plan *plan, int64_t batch, const tp_tensor *kc, const tp_tensor *ks, const tp_tensor *vc,
                     const tp_tensor *vs, Given &g, Cache4 &out) {
  tp_rank_shard sh;
  if (!plan || tp_plan_dims(plan, &g.dims) != TP_OK || tp_plan_query_rank(plan, 0, &sh) != TP_OK) return TP_ERR_INVALID_ARG;
  if (!kc || !ks || !vc || !vs || batch < 0 || batch > 0x7fffffffLL) return TP_ERR_INVALID_ARG;
  g.n = g.dims.tp_size;
  g.hd = g.dims.head_dim;
  if ((g.hd != 64 && g.hd != 128) || g.n > kC4Ranks) return TP_ERR_UNSUPPORTED;
  g.sources = sh.kv_replicated ? 1 : g.n;
  g.heads = g.dims.num_kv_heads / g.sources;
  g.cap = batch > 0 ? kc[0].rows / (batch * g.heads) : 0;
  if (g.cap < 0 || g.cap > 0x7fffffffLL) return TP_ERR_INVALID_ARG;
  const long long rows = batch * g.heads * g.cap;
  tp_status st;
  if ((st = check_cache(kc, g.sources, rows, g.hd / 2, TP_U8)) != TP_OK || (st = check_cache(vc, g.sources, rows, g.hd / 2, TP_U8)) != TP_OK ||
      (st = check_cache(ks, g.sources, rows, g.hd / kGroup, TP_BF16)) != TP_OK ||
      (st = check_cache(vs, g.sources, rows, g.hd / kGroup, TP_BF16)) != TP_OK)
    return st;
  if (!cache_ok(g.dims, g.cap)) return TP_ERR_UNSUPPORTED;
  for (int r = 0; r < g.sources; ++r) {
    out.k_codes[r] = static_cast<uint8_t *>(kc[r].ptr);
    out.v_codes[r] = static_cast<uint8_t *>(vc[r].ptr);
    out.k_scale[r] = static_cast<__nv_bfloat16 *>(ks[r].ptr);
    out.v_scale[r] = static_cast<__nv_bfloat16 *>(vs[r].ptr);
  }
  return TP_OK;
}

tp_status copy_call(const Given &g, CopyParams &p, int64_t batch, const int32_t *starts, const tp_tensor *k, const tp_tensor *v,
                    bool store, cudaStream_t s) {
  if (!k || !v) return TP_ERR_INVALID_ARG;
  const long long n = batch > 0 ? k[0].rows / batch : 0;
  const int32_t dt = k[0].dtype;
  for (int r = 0; r < g.sources; ++r)
    for (int w = 0; w < 2; ++w) {
      const tp_tensor &t = w ? v[r] : k[r];
      if (!view_ok(t)) return TP_ERR_INVALID_ARG;
      if (t.dtype != dt || (dt != TP_BF16 && (store || dt != TP_F32))) return TP_ERR_DTYPE;
      if (t.rows != batch * n || t.cols != g.heads * g.hd) return TP_ERR_INVALID_ARG;
      if (t.rows > 0 && !vec_aligned(t)) return TP_ERR_ALIGNMENT;
      p.in[w][r] = t.ptr;
      p.out[w][r] = t.ptr;
      p.ld[w][r] = t.ld;
    }
  const long long rows = batch * n;
  if (n * g.dims.num_kv_heads > 0x7fffffffLL - 1023 || batch > 65535) return TP_ERR_UNSUPPORTED;
  if (rows > 0 && !starts) return TP_ERR_INVALID_ARG;
  if (!ptr_aligned(starts, 4)) return TP_ERR_ALIGNMENT;
  tp_status st = check_rank_health(g.n);
  if (st != TP_OK || rows == 0) return st;
  DevCtx ctx;
  const cudaError_t e = get_dev_ctx(&ctx);
  if (e != cudaSuccess) return cuda_fail(e);
  p.starts = starts;
  p.batch = static_cast<int>(batch);
  p.n = static_cast<int>(n);
  p.cap = static_cast<int>(g.cap);
  p.heads_kv = g.dims.num_kv_heads;
  p.heads_per_source = static_cast<int>(g.heads);
  p.by_heads.set(p.heads_kv);
  p.by_source.set(p.heads_per_source);
  p.status = ctx.status;
  const long long per = kCopyThreads / (g.hd / 32), blocks = (n * p.heads_kv + per - 1) / per;
  const dim3 grid(static_cast<unsigned>(blocks), 2, static_cast<unsigned>(batch));
  if (store) return launched(launch_kernel(g.hd == 128 ? k_cache4_store<128> : k_cache4_store<64>, grid, dim3(kCopyThreads), 0, s, 1, p));
  if (dt == TP_F32)
    return launched(launch_kernel(g.hd == 128 ? k_cache4_load<128, float> : k_cache4_load<64, float>, grid, dim3(kCopyThreads), 0, s, 1, p));
  return launched(launch_kernel(g.hd == 128 ? k_cache4_load<128, __nv_bfloat16> : k_cache4_load<64, __nv_bfloat16>, grid,
                                dim3(kCopyThreads), 0, s, 1, p));
}

}  // namespace
}  // namespace tpgqa

using namespace tpgqa;
using namespace tpgqa::op;

extern "C" tp_status tp_cache4_store(const tp_plan *plan, int64_t batch, const int32_t *lengths, const int32_t *counts,
                                     const tp_tensor *k, const tp_tensor *v, tp_tensor *k_codes, tp_tensor *k_scale,
                                     tp_tensor *v_codes, tp_tensor *v_scale, tp_stream_t stream) {
  Given g;
  CopyParams p = {};
  const tp_status st = check_call(plan, batch, k_codes, k_scale, v_codes, v_scale, g, p.cache);
  if (st != TP_OK) return st;
  if (!ptr_aligned(counts, 4)) return TP_ERR_ALIGNMENT;
  p.counts = counts;
  return copy_call(g, p, batch, lengths, k, v, true, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" tp_status tp_cache4_load(const tp_plan *plan, int64_t batch, const int32_t *first, const tp_tensor *k_codes,
                                    const tp_tensor *k_scale, const tp_tensor *v_codes, const tp_tensor *v_scale,
                                    tp_tensor *k_out, tp_tensor *v_out, tp_stream_t stream) {
  Given g;
  CopyParams p = {};
  const tp_status st = check_call(plan, batch, k_codes, k_scale, v_codes, v_scale, g, p.cache);
  if (st != TP_OK) return st;
  return copy_call(g, p, batch, first, k_out, v_out, false, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" size_t tp_cache4_attn_workspace_size(const tp_plan *plan, int64_t batch, int64_t capacity, int32_t window,
                                                int32_t sinks) {
  tp_dims d;
  if (!plan || batch < 1 || capacity < 1 || window < 1 || sinks < 0 || tp_plan_dims(plan, &d) != TP_OK) return 0;
  if (!attn_sizes_ok(d, batch, capacity)) return 0;
  return workspace_bytes_of(shape4_of(d, batch, capacity, window, sinks), batch * d.num_q_heads, d.head_dim);
}

extern "C" tp_status tp_cache4_attn(const tp_plan *plan, int64_t batch, const tp_tensor *q, const tp_tensor *k_codes,
                                    const tp_tensor *k_scale, const tp_tensor *v_codes, const tp_tensor *v_scale,
                                    const int32_t *lengths, int32_t window, int32_t sinks, tp_tensor *a, void *workspace,
                                    size_t workspace_bytes, tp_stream_t stream) {
  Given g;
  Attn4Params p = {};
  tp_status st = check_call(plan, batch, k_codes, k_scale, v_codes, v_scale, g, p.cache);
  if (st != TP_OK) return st;
  if (!q || !a || window < 1 || sinks < 0) return TP_ERR_INVALID_ARG;
  if (!attn_sizes_ok(g.dims, batch, g.cap)) return TP_ERR_UNSUPPORTED;
  const long long qc = g.dims.num_q_heads / g.n * g.hd;
  for (int r = 0; r < g.n; ++r) {
    for (const tp_tensor *t : {q + r, static_cast<const tp_tensor *>(a + r)}) {
      if (!view_ok(*t)) return TP_ERR_INVALID_ARG;
      if (t->dtype != TP_BF16) return TP_ERR_DTYPE;
      if (t->rows != batch || t->cols != qc) return TP_ERR_INVALID_ARG;
      if (batch > 0 && !vec_aligned(*t)) return TP_ERR_ALIGNMENT;
    }
    p.q[r] = q[r].ptr;
    p.q_ld[r] = q[r].ld;
    p.a[r] = a[r].ptr;
    p.a_ld[r] = a[r].ld;
  }
  if (batch > 0 && !lengths) return TP_ERR_INVALID_ARG;
  if (!ptr_aligned(lengths, 4)) return TP_ERR_ALIGNMENT;
  const Shape4 s = shape4_of(g.dims, batch, g.cap, window, sinks);
  const long long rows = batch * g.dims.num_q_heads;
  const size_t need = workspace_bytes_of(s, rows, g.hd);
  if (batch > 0 && need > 0) {
    if (!workspace || workspace_bytes < need) return TP_ERR_WORKSPACE;
    if (!ptr_aligned(workspace, 16)) return TP_ERR_ALIGNMENT;
  }
  if ((st = check_rank_health(g.n)) != TP_OK) return st;
  if (batch == 0) return TP_OK;
  DevCtx ctx;
  const cudaError_t e = get_dev_ctx(&ctx);
  if (e != cudaSuccess) return cuda_fail(e);
  p.batch = static_cast<int>(batch);
  p.cap = static_cast<int>(g.cap);
  p.heads_q = g.dims.num_q_heads;
  p.heads_kv = g.dims.num_kv_heads;
  p.group = p.heads_q / p.heads_kv;
  p.heads_per_rank = p.heads_q / g.n;
  p.heads_per_source = static_cast<int>(g.heads);
  p.window = window;
  p.sinks = sinks;
  p.chunk = s.chunk;
  p.splits = s.splits;
  p.cluster = s.cluster;
  p.longest_first = s.longest_first;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(g.hd)));
  p.lengths = lengths;
  p.part_o = static_cast<float *>(workspace);
  p.part_ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + sums_bytes(s, rows, g.hd));
  p.status = ctx.status;
  cudaStream_t str = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid(static_cast<unsigned>(batch * p.heads_kv * p.splits), static_cast<unsigned>(s.head_tiles));
  st = g.hd == 128 ? (s.nt == 2 ? launch_attn4<128, 2>(p, grid, str) : launch_attn4<128, 1>(p, grid, str))
                   : (s.nt == 2 ? launch_attn4<64, 2>(p, grid, str) : launch_attn4<64, 1>(p, grid, str));
  if (st != TP_OK || s.splits < 2 || s.cluster) return st;
  return launched(launch_kernel(g.hd == 128 ? k_cache4_join<128> : k_cache4_join<64>, dim3(static_cast<unsigned>((rows + 7) / 8)),
                                dim3(256), 0, str, 1, p));
}
