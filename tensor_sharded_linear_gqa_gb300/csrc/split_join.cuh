// Joining the key splits of an attention row. Each split left its unnormalised f32 sums O_s, its
// reference maximum m_s (log2 units) and its sum l_s; the softmax over all keys is
//   sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s,  M = max m_s,
// whatever the splits. One warp joins a row, each lane its D / 32 columns.
#pragma once

#include "op_util.h"

namespace tpgqa {
namespace op {

// Split s of the row has its sums at part_o + (s * stride + row) * D. acc receives the
// lane's columns of the sum, the result is the sum of l; with n = 0 both are zero.
template <int D>
__device__ __forceinline__ float join_splits(const float2 *part_ml, const float *part_o, long long stride, long long row,
                                             int n, int lane, float (&acc)[D / 32]) {
  constexpr int kPer = D / 32;
  float mt = -INFINITY, lt = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
  for (int s0 = 0; s0 < n; s0 += 32) {  // a lane per split, then every lane its columns of all of them
    float2 ml = make_float2(-INFINITY, 0.f);
    if (s0 + lane < n) ml = part_ml[(s0 + lane) * stride + row];
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
    const float *src = part_o + (s0 * stride + row) * D + lane * kPer;
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
  return lt;
}

}  // namespace op
}  // namespace tpgqa
