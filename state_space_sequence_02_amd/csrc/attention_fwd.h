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

// A row's sum of weights, with m its maximum.  A score beyond float32 leaves
// NaN in it, or 0 or infinity where only m c is beyond: o and lse of the row
// are then NaN.  0 is left to rows that have seen no key (m = -infinity).
__device__ __forceinline__ float row_sum(float l, float m) {
  return m == -__builtin_inff() || (l > 0.f && l < __builtin_inff()) ? l : __builtin_nanf("");
}

template <typename T, int DP, int SUBS>
struct RowState {
  static constexpr int STEPS = TileCfg<T, DP>::STEPS, COLS = DP / 32;
  typedef f32x16 Scores[SUBS];       // of a tile of 32 SUBS keys
  typedef row_frag<T> Weights[SUBS][2];

  f32x16 o[COLS];
  float m, l;  // m: what the exponents are taken from, in units of s before the scale; l: this
               // half's keys

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int d = 0; d < COLS; ++d) o[d] = zero16();
    m = -__builtin_inff();
    l = 0.f;
  }

  __device__ __forceinline__ static void scores(const head_frag<T> (&q)[STEPS],
                                                const TileReader<T, DP>& kr, Scores& s) {
#pragma unroll
    for (int u = 0; u < SUBS; ++u) {
      s[u] = zero16();
#pragma unroll
      for (int d = 0; d < STEPS; ++d) s[u] = mma_head(kr.head(0, 32 * u, d), q[d], s[u]);
    }
  }

  // Keys from `lim` on are not seen by this lane's row.
  __device__ __forceinline__ static void mask(Scores& s, int lim) {
    const int left = lim - 4 * (lane_id() >> 5);
#pragma unroll
    for (int u = 0; u < SUBS; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r)
        if (32 * u + 8 * (r / 4) + r % 4 >= left) s[u][r] = -__builtin_inff();
  }

  __device__ __forceinline__ static float top(const Scores& s) {
    float t = s[0][0];
#pragma unroll
    for (int u = 0; u < SUBS; ++u)
#pragma unroll
      for (int r = 0; r < 16; ++r) t = __builtin_fmaxf(t, s[u][r]);
    return max_halves(t);
  }

  // How far above m a score may be: until then the weights are at most 2^8,
  // which costs no digits, and the sums need no scaling.  Finite for any scale,
  // so that the first tile (m = -infinity) always counts.
  __device__ __forceinline__ static float slack_of(float c) {
    return __builtin_fminf(8.f / c, 1e30f);
  }
  // Takes m to the tile's top where that is more than `slack` above.
  __device__ __forceinline__ void raise(float top, float slack, float c) {
    if (__ballot(top > m + slack)) {
      const float now = __builtin_fmaxf(m, top);
      const float a = m == now ? 1.f : fast_exp2((m - now) * c);
      m = now;
      l *= a;
#pragma unroll
      for (int d = 0; d < COLS; ++d)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[d][r] *= a;
    }
  }

  __device__ __forceinline__ void weigh(Scores& s, float c, Weights& p) {
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
      for (int h = 0; h < 2; ++h) p[u][h] = acc_frag<T>(s[u], h);
    }
  }

  __device__ __forceinline__ void take(const TileReader<T, DP>& vr, const Weights& p) {
#pragma unroll
    for (int u = 0; u < SUBS; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < COLS; ++d)
          o[d] = mma_rows(vr.cols(0, 32 * u + 16 * h, d), p[u][h], o[d]);
  }

  // scores() of the next tile with weigh() of this one between its products:
  // the matrix cores and the vector ALU work at the same time.  Fragments are
  // read kAhead products before their own.  The barriers hold the order that
  // is written here (left alone, the compiler puts every read first and runs
  // out of registers).
  static constexpr int kAhead = 3;
  __device__ __forceinline__ void scores_and_weigh(const head_frag<T> (&q)[STEPS],
                                                   const TileReader<T, DP>& kr, Scores& next,
                                                   Scores& s, float c, Weights& p) {
    constexpr int N = SUBS * STEPS, E = SUBS * 16 / N;  // products, weights beside each
    static_assert(SUBS * 16 % N == 0, "every product has as many weights beside it");
    const float mc = m == -__builtin_inff() ? 0.f : m * c;
    head_frag<T> f[N];
#pragma unroll
    for (int i = 0; i < kAhead && i < N; ++i) f[i] = kr.head(0, 32 * (i / STEPS), i % STEPS);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int u = i / STEPS, ahead = i + kAhead;
      if (ahead < N) f[ahead] = kr.head(0, 32 * (ahead / STEPS), ahead % STEPS);
      if (i % STEPS == 0) next[u] = zero16();
      next[u] = mma_head(f[i], q[i % STEPS], next[u]);
#pragma unroll
      for (int e = i * E; e < (i + 1) * E; ++e) {
        s[e / 16][e % 16] = fast_exp2(__builtin_fmaf(s[e / 16][e % 16], c, -mc));
        l += s[e / 16][e % 16];
        if (e % 8 == 7) {
          p[e / 16][e % 16 / 8] = acc_frag<T>(s[e / 16], e % 16 / 8);
          pin(p[e / 16][e % 16 / 8]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    pin(l);
  }

  // take() with top() of the next tile between its products.
  __device__ __forceinline__ float take_and_top(const TileReader<T, DP>& vr, const Weights& p,
                                                const Scores& next) {
    constexpr int N = SUBS * 2 * COLS, E = SUBS * 16 / N;
    static_assert(SUBS * 16 % N == 0, "every product has as many scores beside it");
    row_frag<T> f[N];
    const auto read = [&](int i) { return vr.cols(0, 16 * (i / COLS), i % COLS); };
    float t = next[0][0];
#pragma unroll
    for (int i = 0; i < kAhead && i < N; ++i) f[i] = read(i);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i + kAhead < N) f[i + kAhead] = read(i + kAhead);
      const int d = i % COLS, h = i / COLS;
      o[d] = mma_rows(f[i], p[h / 2][h % 2], o[d]);
#pragma unroll
      for (int e = i * E; e < (i + 1) * E; ++e) t = __builtin_fmaxf(t, next[e / 16][e % 16]);
      __builtin_amdgcn_sched_barrier(0);
    }
    return max_halves(t);
  }
};

}  // namespace m2
