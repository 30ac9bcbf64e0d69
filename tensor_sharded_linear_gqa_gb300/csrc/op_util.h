// Argument checks and small device helpers shared by the operators between the
// projections and for long contexts (rmsnorm.cu, cache_evict.cu, linear_epilogue.cu,
// prefix_attention.cu, rotary.cu, window_attention.cu, cache4.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "tp_internal.h"

namespace tpgqa {
namespace op {

// Bytes of an element; 0 for an unknown type.
inline long long elem_size(int32_t dt) {
  return dt == TP_F32 ? 4 : (dt == TP_BF16 ? 2 : (dt == TP_E4M3 ? 1 : 0));
}

// A view with sane extents: rows and columns below 2^31 (TMA and tile coordinates
// are 32-bit), a pitch of at least a row, a base unless it is empty.
inline bool view_ok(const tp_tensor &t) {
  if (elem_size(t.dtype) == 0) return false;
  if (t.rows < 0 || t.cols < 0 || t.ld < t.cols || t.ld < 1) return false;
  if (t.rows > 0x7fffffffLL || t.cols > 0x7fffffffLL) return false;
  return t.rows == 0 || t.cols == 0 || t.ptr != nullptr;
}
inline bool ptr_aligned(const void *p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
inline bool elem_aligned(const tp_tensor &t) { return ptr_aligned(t.ptr, elem_size(t.dtype)); }
// Base and row pitch (of more than one row) on 16-byte boundaries.
inline bool vec_aligned(const tp_tensor &t) {
  return ptr_aligned(t.ptr, 16) && (t.rows <= 1 || (t.ld * elem_size(t.dtype)) % 16 == 0);
}

inline tp_status launched(cudaError_t e) {
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? TP_OK : cuda_fail(e);
}

// Dynamic shared memory above 48 KB, granted once per device and kernel.
template <typename K>
inline cudaError_t allow_smem(K kernel, int bytes, unsigned &mask, std::mutex &mu) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> g(mu);
  if (dev < 32 && (mask & (1u << dev))) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 32) mask |= 1u << dev;
  return e;
}

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }  // regions of a workspace

// Division by a number that the host knows: x / d = (umulhi(x, mul) + x) >> shift for x < 2^31.
struct Divider {
  uint32_t mul, shift;
  __host__ void set(uint32_t d) {
    shift = 0;
    while ((1ull << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ int of(int x) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(x), mul) + static_cast<uint32_t>(x)) >> shift);
  }
};

__device__ __forceinline__ void grid_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ void record(int *status, int code) { atomicCAS(status, 0, code); }

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two f32 in one register pair.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t r, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

}  // namespace op
}  // namespace tpgqa
