// Residual addition and root-mean-square norm of one activation or of the N
// ranks' f32 partials, with a bf16 output or e4m3 codes and one scale per token.
//
// z = sum_r x_r + residual; y = z * rsqrt(mean(z^2) + eps) * w. One CTA owns one
// row and holds it in registers between the two uses of z, so every input is
// read once and every output written once: the kernel is bound by memory, and
// by latency below a few hundred rows. The sum of squares and, for the 8-bit
// output, the largest |z w| come out of one block reduction: the row maximum of
// |y| is that times the row's factor, so no second reduction waits for the first.
// Sums and statistics are f32; the normalised value is taken from the unrounded
// z, so the residual stream's rounding to bf16 does not enter y.
#include <cuda_fp8.h>

#include <cmath>

#include "op_util.h"

namespace tpgqa {
namespace {

using namespace op;

constexpr int kMaxX = 64;
constexpr float kScaleFloor = 0x1p-96f;  // keeps 1 / scale finite for rows of (near) zeros
constexpr float kE4m3Max = 448.0f;

struct NormParams {
  const void *x[kMaxX];
  long long x_ld[kMaxX];
  const void *res;
  void *res_out;
  const void *w;
  void *y;
  float *scale;
  long long res_ld, res_out_ld, y_ld;
  int n_x, rows, cols, w_f32;
  float eps;
};

// Eight consecutive elements as f32; `left` (1..8) of them exist.
__device__ __forceinline__ void load8(const float *p, int left, float (&v)[8]) {
  if (left >= 8) {
    const float4 a = *reinterpret_cast<const float4 *>(p), b = *reinterpret_cast<const float4 *>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
  }
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int left, float (&v)[8]) {
  if (left >= 8) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p);
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? __bfloat162float(p[i]) : 0.0f;
  }
}
__device__ __forceinline__ void store8(float *p, int left, const float (&v)[8]) {
  if (left >= 8) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int left, const float (&v)[8]) {
  if (left >= 8) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                               pack_bf16(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = __float2bfloat16_rn(v[i]);
  }
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3 *p, int left, const float (&v)[8]) {
  if (left >= 8) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i], v[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2], v[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
      w[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i].__x = __nv_cvt_float_to_fp8(v[i], __NV_SATFINITE, __NV_E4M3);
  }
}

__device__ __forceinline__ float load1(const float *p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store1(__nv_fp8_e4m3 *p, float v) {
  p->__x = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

struct NoRes {};  // "no residual" as a type

template <typename T>
struct IsFp8 {
  static constexpr bool value = false;
};
template <>
struct IsFp8<__nv_fp8_e4m3> {
  static constexpr bool value = true;
};

// The larger of two; NaN if either is (fmaxf would pass over it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}
// A token's scale from its largest |z w| and its factor. A row whose largest |y| is
// no number (a NaN, or an infinity times the factor 0 of an infinite mean) has no scale.
__device__ __forceinline__ float row_scale(float top, float rstd) {
  return max_nan(top * rstd, kScaleFloor) / kE4m3Max;
}

// Sum and maximum over the CTA, in every thread. The order of the additions is
// fixed by the thread count, so results do not change from run to run.
__device__ __forceinline__ float2 block_sum_max(float sum, float mx) {
  __shared__ float2 part[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const int warps = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(sum, mx);
  __syncthreads();
  float2 r = (threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : make_float2(0.0f, 0.0f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    r.x += __shfl_xor_sync(0xffffffffu, r.x, o);
    r.y = max_nan(r.y, __shfl_xor_sync(0xffffffffu, r.y, o));
  }
  return r;
}

// The row in registers: thread t holds the 8-element groups t, t + blockDim, ...
// (ITEMS of them). Bases and pitches are 16-byte aligned; a row's last group may
// be partial and is moved by elements.
// ONE: a single x, whose few registers let three CTAs share an SM: with rows that
// load, reduce and store at different times memory stays busy (4096 x 8192, f32 x and
// bf16 residual: 56 us, 5.95 TB/s, against 69 us with two CTAs of up to 64 registers). Four
// groups a thread (rows of 8193 to 16384) leave room for two, and read the weight again, from
// L1, where it would take half of the registers: 2048 x 16384 takes 64 us, 69 with the weight
// kept (spills) and 84 with three CTAs (more of them). The loads of several partials
// need more registers (64 x 4096, eight partials: 5.4 us, 8.3 with three CTAs).
template <typename XT, typename RT, typename YT, int ITEMS, bool ONE>
__global__ void __launch_bounds__(512, ONE ? (ITEMS <= 2 ? 3 : 2) : 1) k_add_rmsnorm(const __grid_constant__ NormParams p) {
  constexpr bool kRes = !std::is_same<RT, NoRes>::value;
  grid_dep_wait();
  grid_dep_launch();
  const long long row = blockIdx.x;
  float z[ITEMS][8];
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int c = (threadIdx.x + j * blockDim.x) * 8;
    if (c < p.cols) load8(static_cast<const XT *>(p.x[0]) + row * p.x_ld[0] + c, p.cols - c, z[j]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) z[j][i] = 0.0f;
  }
  // four partials' loads in flight at a time; added in rank order
  for (int r0 = 1; !ONE && r0 < p.n_x; r0 += 4) {
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * 8;
      if (c < p.cols) {
        float v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r0 + u < p.n_x) load8(static_cast<const XT *>(p.x[r0 + u]) + row * p.x_ld[r0 + u] + c, p.cols - c, v[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r0 + u < p.n_x)
#pragma unroll
            for (int i = 0; i < 8; ++i) z[j][i] += v[u][i];
      }
    }
  }
  if constexpr (kRes) {
#pragma unroll
    for (int j = 0; j < ITEMS; ++j) {
      const int c = (threadIdx.x + j * blockDim.x) * 8;
      if (c < p.cols) {
        float v[8];
        load8(static_cast<const RT *>(p.res) + row * p.res_ld + c, p.cols - c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) z[j][i] += v[i];
      }
    }
  }
  constexpr bool kKeep = ITEMS <= 2;  // the weight in registers
  float kept[kKeep ? ITEMS : 1][8];
  auto weight = [&](int c, float (&w)[8]) {
    if (p.w_f32) load8(static_cast<const float *>(p.w) + c, p.cols - c, w);
    else load8(static_cast<const __nv_bfloat16 *>(p.w) + c, p.cols - c, w);
  };
  float sum = 0.0f, mx = 0.0f;
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int c = (threadIdx.x + j * blockDim.x) * 8;
    if (c < p.cols) {
      float (&w)[8] = kept[kKeep ? j : 0];
      if (kKeep || IsFp8<YT>::value) weight(c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum = fmaf(z[j][i], z[j][i], sum);
        if (IsFp8<YT>::value) mx = max_nan(mx, fabsf(z[j][i] * w[i]));
      }
    }
  }
  const float2 st = block_sum_max(sum, mx);
  const float rstd = rsqrtf(st.x / static_cast<float>(p.cols) + p.eps);
  float inv = 1.0f;
  if (IsFp8<YT>::value) {
    const float scale = row_scale(st.y, rstd);
    inv = 1.0f / scale;
    if (threadIdx.x == 0) p.scale[row] = scale;
  }
#pragma unroll
  for (int j = 0; j < ITEMS; ++j) {
    const int c = (threadIdx.x + j * blockDim.x) * 8;
    if (c < p.cols) {
      if constexpr (kRes) {
        if (p.res_out) store8(static_cast<RT *>(p.res_out) + row * p.res_out_ld + c, p.cols - c, z[j]);
      }
      float (&w)[8] = kept[kKeep ? j : 0];
      if (!kKeep) weight(c, w);
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = z[j][i] * rstd * w[i] * inv;
      store8(static_cast<YT *>(p.y) + row * p.y_ld + c, p.cols - c, v);
    }
  }
}

// Any alignment and row length, element by element: z is computed twice, the
// second time for the outputs. residual_out is written in the second pass only,
// each element after its own last read, so it may be the residual.
template <typename XT, typename RT, typename YT>
__global__ void __launch_bounds__(512) k_add_rmsnorm_elems(const __grid_constant__ NormParams p) {
  constexpr bool kRes = !std::is_same<RT, NoRes>::value;
  grid_dep_wait();
  grid_dep_launch();
  const long long row = blockIdx.x;
  auto z_at = [&](int c) {
    float z = load1(static_cast<const XT *>(p.x[0]) + row * p.x_ld[0] + c);
    for (int r = 1; r < p.n_x; ++r) z += load1(static_cast<const XT *>(p.x[r]) + row * p.x_ld[r] + c);
    if constexpr (kRes) z += load1(static_cast<const RT *>(p.res) + row * p.res_ld + c);
    return z;
  };
  auto w_at = [&](int c) {
    return p.w_f32 ? static_cast<const float *>(p.w)[c] : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.w)[c]);
  };
  float sum = 0.0f, mx = 0.0f;
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float z = z_at(c);
    sum = fmaf(z, z, sum);
    if (IsFp8<YT>::value) mx = max_nan(mx, fabsf(z * w_at(c)));
  }
  const float2 st = block_sum_max(sum, mx);
  const float rstd = rsqrtf(st.x / static_cast<float>(p.cols) + p.eps);
  float inv = 1.0f;
  if (IsFp8<YT>::value) {
    const float scale = row_scale(st.y, rstd);
    inv = 1.0f / scale;
    if (threadIdx.x == 0) p.scale[row] = scale;
  }
  for (int c = threadIdx.x; c < p.cols; c += blockDim.x) {
    const float z = z_at(c);
    if constexpr (kRes) {
      if (p.res_out) store1(static_cast<RT *>(p.res_out) + row * p.res_out_ld + c, z);
    }
    store1(static_cast<YT *>(p.y) + row * p.y_ld + c, z * rstd * w_at(c) * inv);
  }
}

template <typename XT, typename RT, typename YT, bool ONE>
tp_status launch_vec(const NormParams &p, int groups, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(p.rows));
  auto threads_for = [](int per) { return dim3(static_cast<unsigned>(per <= 32 ? 32 : (per + 31) / 32 * 32)); };
  // The fewest groups per thread that keep the CTA within 512 threads.
  if (groups <= 512)
    return launched(launch_kernel(k_add_rmsnorm<XT, RT, YT, 1, ONE>, grid, threads_for(groups), 0, s, 1, p));
  if (groups <= 1024)
    return launched(launch_kernel(k_add_rmsnorm<XT, RT, YT, 2, ONE>, grid, threads_for((groups + 1) / 2), 0, s, 1, p));
  return launched(launch_kernel(k_add_rmsnorm<XT, RT, YT, 4, ONE>, grid, threads_for((groups + 3) / 4), 0, s, 1, p));
}

template <typename XT, typename RT, typename YT>
tp_status launch_typed(const NormParams &p, bool vec, cudaStream_t s) {
  const int groups = (p.cols + 7) / 8;
  if (vec && groups <= 2048)
    return p.n_x == 1 ? launch_vec<XT, RT, YT, true>(p, groups, s) : launch_vec<XT, RT, YT, false>(p, groups, s);
  return launched(launch_kernel(k_add_rmsnorm_elems<XT, RT, YT>, dim3(static_cast<unsigned>(p.rows)), dim3(512), 0, s, 1, p));
}

template <typename XT, typename RT>
tp_status launch_y(const NormParams &p, int32_t y_dt, bool vec, cudaStream_t s) {
  return y_dt == TP_E4M3 ? launch_typed<XT, RT, __nv_fp8_e4m3>(p, vec, s) : launch_typed<XT, RT, __nv_bfloat16>(p, vec, s);
}

template <typename XT>
tp_status launch_r(const NormParams &p, const tp_tensor *res, int32_t y_dt, bool vec, cudaStream_t s) {
  if (!res) return launch_y<XT, NoRes>(p, y_dt, vec, s);
  return res->dtype == TP_F32 ? launch_y<XT, float>(p, y_dt, vec, s) : launch_y<XT, __nv_bfloat16>(p, y_dt, vec, s);
}

}  // namespace
}  // namespace tpgqa

using namespace tpgqa;
using namespace tpgqa::op;

extern "C" tp_status tp_add_rmsnorm(int32_t n_x, const tp_tensor *x, const tp_tensor *residual, const tp_tensor *weight,
                                    float eps, tp_tensor *residual_out, tp_tensor *y, float *y_scale,
                                    tp_stream_t stream) {
  if (n_x < 1 || n_x > kMaxX || !x || !weight || !y) return TP_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return TP_ERR_INVALID_ARG;
  if (residual_out && !residual) return TP_ERR_INVALID_ARG;
  const long long T = x[0].rows, D = x[0].cols;
  auto float_like = [](int32_t dt) { return dt == TP_F32 || dt == TP_BF16; };
  bool vec = true;
  auto check = [&](const tp_tensor &t, long long rows, bool dt_ok) -> tp_status {
    if (!view_ok(t) || t.rows != rows || t.cols != D) return TP_ERR_INVALID_ARG;
    if (!dt_ok) return TP_ERR_DTYPE;
    if (!elem_aligned(t)) return TP_ERR_ALIGNMENT;
    vec = vec && vec_aligned(t);
    return TP_OK;
  };
  tp_status st;
  for (int32_t r = 0; r < n_x; ++r)
    if ((st = check(x[r], T, float_like(x[r].dtype) && x[r].dtype == x[0].dtype)) != TP_OK) return st;
  if (residual && (st = check(*residual, T, float_like(residual->dtype))) != TP_OK) return st;
  if (residual_out && (st = check(*residual_out, T, residual_out->dtype == residual->dtype)) != TP_OK) return st;
  if (!view_ok(*weight) || weight->rows != 1 || weight->cols != D) return TP_ERR_INVALID_ARG;
  if (!float_like(weight->dtype)) return TP_ERR_DTYPE;
  if (!elem_aligned(*weight)) return TP_ERR_ALIGNMENT;
  vec = vec && ptr_aligned(weight->ptr, 16);
  if ((st = check(*y, T, y->dtype == TP_BF16 || y->dtype == TP_E4M3)) != TP_OK) return st;
  if ((y->dtype == TP_E4M3) != (y_scale != nullptr)) {
    if (!(y->dtype == TP_E4M3 && T == 0)) return TP_ERR_INVALID_ARG;
  }
  if (!ptr_aligned(y_scale, 4)) return TP_ERR_ALIGNMENT;
  if ((st = check_rank_health(n_x)) != TP_OK) return st;
  if (T == 0 || D == 0) return TP_OK;
  NormParams p = {};
  for (int32_t r = 0; r < n_x; ++r) {
    p.x[r] = x[r].ptr;
    p.x_ld[r] = x[r].ld;
  }
  p.res = residual ? residual->ptr : nullptr;
  p.res_ld = residual ? residual->ld : 0;
  p.res_out = residual_out ? residual_out->ptr : nullptr;
  p.res_out_ld = residual_out ? residual_out->ld : 0;
  p.w = weight->ptr;
  p.w_f32 = weight->dtype == TP_F32;
  p.y = y->ptr;
  p.y_ld = y->ld;
  p.scale = y_scale;
  p.n_x = n_x;
  p.rows = static_cast<int>(T);
  p.cols = static_cast<int>(D);
  p.eps = eps;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return x[0].dtype == TP_F32 ? launch_r<float>(p, residual, y->dtype, vec, s)
                              : launch_r<__nv_bfloat16>(p, residual, y->dtype, vec, s);
}
