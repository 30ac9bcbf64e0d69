// Joining the key splits of an attention row. Each split left its unnormalised f32 sums O_s, its
// reference maximum m_s (log2 units) and its sum l_s; the softmax over all keys is
//   sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s,  M = max m_s,
// whatever the splits. One warp joins a row, each lane its D / 32 columns, eight splits at a
// time whose loads all go out together: the join is bound by their latency.
#pragma once

#include "op_util.h"

namespace tpgqa {
namespace op {

// Split s of the row has its sums at part_o + (s * stride + row) * D. acc receives the
// lane's columns of the sum, the result is the sum of l; with n = 0 both are zero.
template <int D>
__device__ __forceinline__ float join_splits(const float2 *part_ml, const float *part_o, long long stride, long long row,
                                             int n, int lane, float (&acc)[D / 32]) {
  constexpr int kPer = D / 32, kAtOnce = 8;
  float mt = -INFINITY, lt = 0.f;
#pragma unroll
  for (int c = 0; c < kPer; ++c) acc[c] = 0.f;
  for (int s0 = 0; s0 < n; s0 += kAtOnce) {
    float2 ml[kAtOnce], o[kAtOnce][kPer / 2];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const bool there = s0 + j < n;
      const long long at = (s0 + j) * stride + row;
      ml[j] = there ? part_ml[at] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int c = 0; c < kPer / 2; ++c)
        o[j][c] = there ? *reinterpret_cast<const float2 *>(part_o + at * D + lane * kPer + 2 * c) : make_float2(0.f, 0.f);
    }
    float m_new = mt;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) m_new = fmaxf(m_new, ml[j].x);
    const float back = mt == m_new ? 1.f : ex2(mt - m_new);
    mt = m_new;
    lt *= back;
#pragma unroll
    for (int c = 0; c < kPer; ++c) acc[c] *= back;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const float f = ex2(ml[j].x - m_new);
      lt += f * ml[j].y;
#pragma unroll
      for (int c = 0; c < kPer / 2; ++c) {
        acc[2 * c] += f * o[j][c].x;
        acc[2 * c + 1] += f * o[j][c].y;
      }
    }
  }
  return lt;
}

}  // namespace op
}  // namespace tpgqa
