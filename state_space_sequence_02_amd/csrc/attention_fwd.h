// The forward's parts that prompts and single tokens share (attention.hip,
// attention_step.hip).  Per row i and the keys j that it sees,
//
//     s_j = scale q_i . k_j,   m = max s_j,   l = sum exp(s_j - m)
//     o_i = sum exp(s_j - m) v_j / l,   lse_i = m + log l
//
// in one pass over the keys: the sums so far are scaled down when a larger s
// appears.  A wavefront holds 32 packed rows as columns: S^T = K Q^T puts a
// row's weights into one lane and its other half, so the maximum, the sum and
// the scaling are that lane's own, and the weights are at once the operand of
// O^T += V^T P^T (attention.h).  Exponentials are base 2 with scale * log2(e)
// in the multiply-add before them.
#pragma once

#include "attention.h"

namespace m2 {

template <typename T, int DP>
struct RowState {
  f32x16 o[DP / 32];
  float m, l;  // m in units of s before the scale; l: this half's keys

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) o[d] = zero16();
    m = -__builtin_inff();
    l = 0.f;
  }

  // One tile of 32 SUBS keys.  lim: keys of the tile that this lane's row sees;
  // mask: whether that is not all of them for some lane (uniform).
  template <int SUBS>
  __device__ __forceinline__ void step(const head_frag<T> (&q)[TileCfg<T, DP>::STEPS],
                                       const TileReader<T, DP>& kr, const TileReader<T, DP>& vr,
                                       bool mask, int lim, float c) {
    f32x16 s[SUBS];
#pragma unroll
    for (int u = 0; u < SUBS; ++u) {
      s[u] = zero16();
#pragma unroll
      for (int d = 0; d < TileCfg<T, DP>::STEPS; ++d)
        s[u] = mma_head(kr.head(0, 32 * u, d), q[d], s[u]);
    }
    if (mask) {
      const int left = lim - 4 * (lane_id() >> 5);
#pragma unroll
      for (int u = 0; u < SUBS; ++u)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * u + 8 * (r / 4) + r % 4 >= left) s[u][r] = -__builtin_inff();
    }
    float top = s[0][0];
#pragma unroll
    for (int u = 0; u < SUBS; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) top = __builtin_fmaxf(top, s[u][r]);
    top = max_halves(top);
    if (__ballot(top > m)) {
      const float now = __builtin_fmaxf(m, top);
      const float a = m == now ? 1.f : fast_exp2((m - now) * c);
      m = now;
      l *= a;
#pragma unroll
      for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] *= a;
    }
    // a row that has seen nothing yet: weights of exp2(-infinity - 0)
    const float mc = m == -__builtin_inff() ? 0.f : m * c;
#pragma unroll
    for (int u = 0; u < SUBS; ++u) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[u][r] = fast_exp2(__builtin_fmaf(s[u][r], c, -mc));
        l += s[u][r];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const row_frag<T> p = acc_frag<T>(s[u], h);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
          o[d] = mma_rows(vr.cols(0, 32 * u + 16 * h, d), p, o[d]);
      }
    }
  }
};

}  // namespace m2
