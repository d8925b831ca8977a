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

// Rows of K and V of one (sequence, group).
template <typename T>
struct Keys {
  const T *k, *v;            // row 0
  int64_t ks, vs;            // elements between rows
  int n;                     // rows, >= 1
  const T *k_last, *v_last;  // row n - 1, where it stands elsewhere; else NULL
};

// Starts the loads of rows r0 .. r0 + ROWS - 1 into an LDS tile, by NT
// threads.  Rows behind the last are the last again: finite values under
// weights of zero, and nothing behind the sequence is read.
template <typename T, int DP, int ROWS, int NT>
__device__ __forceinline__ void stage_rows(uint32_t lds, const T* base, int64_t stride, int n,
                                           const T* last, int r0, int D, int thread) {
  using K = TileCfg<T, DP>;
#pragma unroll
  for (int i = 0; i < ROWS * K::CH / NT; ++i) {
    const int slot = i * NT + thread;
    const int r = slot / K::CH, c = (slot % K::CH) ^ swz<K::CH>(r);
    const int at = r0 + r < n - 1 ? r0 + r : n - 1;
    const T* p = base + at * stride;
    if (last && at == n - 1) p = last;
    if (c * K::E < D) dma16(p + c * K::E, lds + (slot & ~63) * 16);
  }
}

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

  // One tile of 32 SUBS keys.  lim: keys of the tile that this lane's row sees.
  template <int SUBS, bool MASK>
  __device__ __forceinline__ void step(const head_frag<T> (&q)[TileCfg<T, DP>::STEPS],
                                       const char* kt, const char* vt, int lim, float c) {
    using R = TileReader<T, DP>;
    f32x16 s[SUBS];
#pragma unroll
    for (int u = 0; u < SUBS; ++u) {
      s[u] = zero16();
#pragma unroll
      for (int d = 0; d < TileCfg<T, DP>::STEPS; ++d)
        s[u] = mma_head(R::head(kt, 32 * u, d), q[d], s[u]);
    }
    if constexpr (MASK) {
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
          o[d] = mma_rows(R::cols(vt, 32 * u + 16 * h, d), p, o[d]);
      }
    }
  }
};

}  // namespace m2
