// Backward pass of the selective scan.  With q = dy silu(z) (dy without a
// gate), d the time step, w = d u, a = exp(d A), per token t, channel and
// state n:
//
//     g[t] = q[t] C[t] + a[t+1] g[t+1]          (the gradient of h[t]; dfinal at the end)
//     dC = sum over channels q h                dB = sum over channels g w
//     du = d sum_n g B + D q                    dD = sum q u
//     dd = sum_n A g (a h[t-1]) + u sum_n g B   dA = sum over tokens d g (a h[t-1])
//     ddt = dd softplus'(dt + bias)             ddt_bias = sum over tokens ddt
//     dz = dy silu'(z) (sum_n C h + D u)        dinit = a[0] g[0]
//
// The states are recomputed.  The sequence is cut into short chunks (64
// tokens at 16 states) that run at once:
//   1. scan_bwd_ends: per chunk the state reached from zero, the sum of d (the
//      decay over the chunk is exp(A sum d)), and the gradient its tokens send
//      to its start.  All go forward in time, from one exponential per (token,
//      channel, state): the last is sum_t (a[0] .. a[t]) q[t] C[t].
//   2. scan_bwd_carry: start states forward over the chunks, end gradients
//      backward over them.
//   3. scan_bwd_main: per chunk the states at the start of each tile of
//      tokens (kept in LDS), then the tiles in reverse, each with its states
//      and decays in registers.  Tiles behind a sequence's end get zeros.
//   4. scan_bwd_sums: the sums over channel tiles (dB, dC) and over chunks
//      (dA, dD, ddt_bias).
//
// A lane holds K of a channel's 4 K states, four lanes (a quad) a channel, a
// wavefront 16 channels, a workgroup 64 of one group.  Each lane of a quad
// loads every fourth token and hands it to the other three through the quad
// permutation that an instruction's operand can carry; sums over a channel's
// states cross the quad the same way, so nothing waits for another wavefront
// inside a chunk.  Sums over the channels of a wavefront (dB, dC) exchange
// halves of the values while they add: the count of values halves with the
// count of lanes, two operations per value instead of eight.
#include "partial_sums.h"
#include "selective_scan.h"

namespace m2 {

namespace {

// Tokens of a tile whose states and decays stay in registers, and the longest
// chunk: the workgroup's tile-start states take 32 KB of LDS at 16 states, 64
// at 32, 128 at 64 (2 x 2048 x 1536 x 64: 749 us, 949 with half the chunk).
constexpr int bwd_tile(int K) { return K <= 4 ? 8 : 4; }
constexpr int bwd_chunk(int K) { return K <= 4 ? 64 : 32; }

// The value of the lane 8 and 4 lanes away (exclusive or) in a row of 16: a
// rotation by 8; the mirror of 8 lanes after that of each quad.
__device__ __forceinline__ float from_xor8(float v) { return dpp<0x128>(v); }
__device__ __forceinline__ float from_xor4(float v) { return dpp<0x141>(dpp<0x1B>(v)); }

// Sums v over the 16 lanes of the wavefront that hold the same quarter of the
// states.  M values per lane become ceil(M / 16): lane (b5 b4 b3 b2 j) ends
// with the totals of v[b5 M/2 + b4 M/4 + b3 M/8 + b2 M/16 + r].
template <int M>
__device__ __forceinline__ void sum_channels(float (&v)[M], int lane) {
  static_assert(M >= 8, "");
#pragma unroll
  for (int m = 0; m < M / 2; ++m) {
    const auto s = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v[m]),
                                                    __builtin_bit_cast(unsigned, v[m + M / 2]),
                                                    false, false);
    const unsigned x = s[0], y = s[1];  // a bit cast of s[1] itself reads s[0]
    v[m] = __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
  }
#pragma unroll
  for (int m = 0; m < M / 4; ++m) {
    const auto s = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v[m]),
                                                    __builtin_bit_cast(unsigned, v[m + M / 4]),
                                                    false, false);
    const unsigned x = s[0], y = s[1];
    v[m] = __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
  }
#pragma unroll
  for (int m = 0; m < M / 8; ++m) {
    const bool hi = lane & 8;
    const float keep = hi ? v[m + M / 8] : v[m], send = hi ? v[m] : v[m + M / 8];
    v[m] = keep + from_xor8(send);
  }
  if constexpr (M >= 16) {
#pragma unroll
    for (int m = 0; m < M / 16; ++m) {
      const bool hi = lane & 4;
      const float keep = hi ? v[m + M / 16] : v[m], send = hi ? v[m] : v[m + M / 16];
      v[m] = keep + from_xor4(send);
    }
  } else {
    v[0] += from_xor4(v[0]);
  }
}

// Stores what sum_channels left: v[m] is state m % K of this lane's quarter,
// token m / K of rows of 4 K states.
template <int M, int K>
__device__ __forceinline__ void store_sums(float* rows, const float (&v)[M], int lane) {
  const int m = (lane >> 5) * (M / 2) + (lane >> 4 & 1) * (M / 4) + (lane >> 3 & 1) * (M / 8) +
                (M >= 16 ? (lane >> 2 & 1) * (M / 16) : 0);
#pragma unroll
  for (int r = 0; r < (M >= 16 ? M / 16 : 1); ++r)
    rows[(m + r) / K * (4 * K) + K * (lane & 3) + (m + r) % K] = v[r];
}

// B and C of a chunk into LDS as float32, zero past N and past the sequence.
template <typename T, int NP, int Q>
__device__ __forceinline__ void stage_bc(const ScanArgs& a, const ScanPlace& p, int valid,
                                         float (*sB)[NP], float (*sC)[NP]) {
  const int64_t row0 = p.b * a.L + p.t0;
  const T* Bb = (const T*)a.B + row0 * a.bs + (int64_t)p.g * a.N;
  const T* Cb = (const T*)a.C + row0 * a.cs + (int64_t)p.g * a.N;
#pragma unroll
  for (int i = threadIdx.x; i < Q * NP; i += 64 * kQuadWaves) {
    const int t = i / NP, n = i % NP;
    const bool in = n < a.N && t < valid;
    sB[t][n] = in ? to_f32(Bb[t * a.bs + n]) : 0.f;
    sC[t][n] = in ? to_f32(Cb[t * a.cs + n]) : 0.f;
  }
}

template <typename T, int K, bool GATE>
__global__ void __launch_bounds__(64 * kQuadWaves) scan_bwd_ends_kernel(
    ScanArgs a, const T* __restrict__ dy, float* __restrict__ hs, float* __restrict__ sum_d,
    float* __restrict__ ge) {
  constexpr int NP = 4 * K, Q = bwd_chunk(K), TT = Q < 16 ? Q : 16, OWN = TT / 4;
  __shared__ __align__(16) float sB[Q][NP], sC[Q][NP];
  const int j = lane_id() & 3;
  const ScanPlace p = scan_place(a);
  const Rows<T> r(a, p, dy, j);
  stage_bc<T, NP, Q>(a, p, r.valid, sB, sC);
  const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f;
  States<K> A2, h, P, e;
  A2.load_n(a.A + p.c * a.N, K * j, a.N, kLog2e);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    h.v[k] = e.v[k] = 0.f;
    P.v[k] = 1.f;
  }
  float total = 0.f;
  Tokens<T, TT, GATE> cur, nxt;
  cur.template load<true, true>(a, p, r, 0);
  __syncthreads();
  for (int t = 0; t < r.valid; t += TT) {
    if (t + TT < r.valid) nxt.template load<true, true>(a, p, r, t + TT);
    float raw[OWN], d[OWN], w[OWN], q[OWN];
    cur.steps(a, r, t, bias, raw, d);
    cur.grads(q);
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      w[i] = d[i] * to_f32(cur.u[i]);
      total += d[i];
    }
    auto token = [&](int i, float dv, float wv, float qv) {
      States<K> B, C;
      B.load(&sB[t + i][K * j]);
      C.load(&sC[t + i][K * j]);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float x = fast_exp2(dv * A2.v[k]);
        h.v[k] = __builtin_fmaf(x, h.v[k], wv * B.v[k]);
        P.v[k] *= x;
        e.v[k] = __builtin_fmaf(P.v[k], qv * C.v[k], e.v[k]);
      }
    };
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      token(4 * i, of_lane<0>(d[i]), of_lane<0>(w[i]), of_lane<0>(q[i]));
      token(4 * i + 1, of_lane<1>(d[i]), of_lane<1>(w[i]), of_lane<1>(q[i]));
      token(4 * i + 2, of_lane<2>(d[i]), of_lane<2>(w[i]), of_lane<2>(q[i]));
      token(4 * i + 3, of_lane<3>(d[i]), of_lane<3>(w[i]), of_lane<3>(q[i]));
    }
    cur = nxt;
  }
  total = quad_sum(total);
  if (!p.live) return;
  const int64_t col = (p.b * a.chunks + p.chunk) * a.Dm + p.c;
  h.store(hs + col * NP + K * j);
  e.store(ge + col * NP + K * j);
  if (j == 0) sum_d[col] = total;
}

// Over the chunks, per (batch, channel, state): hs from "reached from zero" to
// "starts from", ge from "sent to its start" to "arrives at its end".  Shares
// of the chunks as in the forward's carry.
__global__ void __launch_bounds__(64 * kCarryWaves) scan_bwd_carry_kernel(
    ScanArgs a, int NP, float* __restrict__ hs, const float* __restrict__ sum_d,
    float* __restrict__ ge, const float* __restrict__ dfinal) {
  __shared__ float sh[kCarryWaves][64], sg[kCarryWaves][64], sp[kCarryWaves][64];
  const int lane = lane_id(), wave = wave_id(), waves = blockDim.x >> 6;
  const int64_t cols = a.Dm * NP, col = (int64_t)blockIdx.x * 64 + lane, b = blockIdx.y;
  const bool live = col < cols;
  const int n = (int)(col % NP);
  const int64_t c = live ? col / NP : 0;
  const int64_t share = (a.chunks + waves - 1) / waves;
  const int64_t c0 = wave * share, c1 = c0 + share < a.chunks ? c0 + share : a.chunks;
  const int64_t base = b * a.chunks * cols + (live ? col : 0);
  const float A2 = n < a.N ? a.A[c * a.N + n] * kLog2e : 0.f;
  const float* dp = sum_d + b * a.chunks * a.Dm + c;
  float x[kCarryLoads], hl[kCarryLoads], el[kCarryLoads];
  auto load = [&](int64_t q) {
#pragma unroll
    for (int k = 0; k < kCarryLoads; ++k) {
      const int64_t i = q + k < c1 ? q + k : c1 - 1;
      x[k] = dp[i * a.Dm];
      hl[k] = hs[base + i * cols];
      el[k] = ge[base + i * cols];
    }
#pragma unroll
    for (int k = 0; k < kCarryLoads; ++k) x[k] = fast_exp2(A2 * x[k]);
  };
  // this share as one chunk: state reached, decay, gradient sent to its start
  float h = 0.f, P = 1.f, e = 0.f;
  for (int64_t q = c0; q < c1; q += kCarryLoads) {
    load(q);
#pragma unroll
    for (int k = 0; k < kCarryLoads; ++k) {
      if (q + k < c1) {
        e = __builtin_fmaf(P, el[k], e);
        h = __builtin_fmaf(x[k], h, hl[k]);
        P *= x[k];
      }
    }
  }
  sh[wave][lane] = h;
  sg[wave][lane] = e;
  sp[wave][lane] = P;
  __syncthreads();
  if (!live) return;
  const int64_t st = (b * a.Dm + c) * a.N + n;
  float run = a.init && n < a.N ? a.init[st] : 0.f;
  for (int w = 0; w < wave; ++w) run = __builtin_fmaf(sp[w][lane], run, sh[w][lane]);
  float back = dfinal && n < a.N ? dfinal[st] : 0.f;
  for (int w = waves - 1; w > wave; --w) back = __builtin_fmaf(sp[w][lane], back, sg[w][lane]);
  const bool again = share > kCarryLoads;  // else the share is still in registers
  for (int64_t q = c0; q < c1; q += kCarryLoads) {
    if (again) load(q);
#pragma unroll
    for (int k = 0; k < kCarryLoads; ++k) {
      if (q + k < c1) {
        hs[base + (q + k) * cols] = run;
        run = __builtin_fmaf(x[k], run, hl[k]);
      }
    }
  }
  const int64_t last = c0 < c1 ? c0 + (c1 - 1 - c0) / kCarryLoads * kCarryLoads : c0 - 1;
  for (int64_t q = last; q >= c0; q -= kCarryLoads) {
    if (again) load(q);
#pragma unroll
    for (int k = kCarryLoads - 1; k >= 0; --k) {
      if (q + k < c1) {
        ge[base + (q + k) * cols] = back;
        back = __builtin_fmaf(x[k], back, el[k]);
      }
    }
  }
}

// part_bc: [2][tiles][B][L][G][NP] parts of dB and dC, one for each channel
// tile of a group.  part_a: [B * chunks][D (N + 2)] parts of dA, dD and
// ddt_bias.
template <typename T, int K, bool GATE>
__global__ void __launch_bounds__(64 * kQuadWaves) scan_bwd_main_kernel(
    ScanArgs a, const T* __restrict__ dy, const float* __restrict__ dfinal,
    const float* __restrict__ hs, const float* __restrict__ ge, T* __restrict__ du,
    T* __restrict__ ddt, T* __restrict__ dz, int64_t dzs, float* __restrict__ dinit,
    float* __restrict__ part_bc, float* __restrict__ part_a) {
  constexpr int NP = 4 * K, Q = bwd_chunk(K), TT = bwd_tile(K), OWN = TT / 4, NT = Q / TT;
  constexpr int GT = K == 1 ? 8 : 16 / K, M = GT * K;  // tokens and values summed over channels at once
  __shared__ __align__(16) float sB[Q][NP], sC[Q][NP];
  // per wavefront and tile: the states at its start, then its dB and dC
  __shared__ __align__(16) float slot[kQuadWaves][NT][64 * K];
  const int lane = lane_id(), wave = wave_id(), j = lane & 3;
  const ScanPlace p = scan_place(a);
  const Rows<T> rows(a, p, dy, j);
  stage_bc<T, NP, Q>(a, p, rows.valid, sB, sC);
  const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f;
  const float Dv = a.D ? a.D[p.c] : 0.f;
  const int64_t srow = (p.b * a.Dm + p.c) * a.N;
  const int64_t row = ((p.b * a.chunks + p.chunk) * a.Dm + p.c) * NP + K * j;
  States<K> A2, h, ag, dA;
  // a lane without a channel: decay 1, state and gradient 0.  With the tile's
  // first channel's instead, a negative bias (its time step, without softplus)
  // makes them grow, and 0 * infinity is no 0 in the sums over channels
#pragma unroll
  for (int k = 0; k < K; ++k) A2.v[k] = h.v[k] = ag.v[k] = dA.v[k] = 0.f;
  if (p.live) {
    A2.load_n(a.A + p.c * a.N, K * j, a.N, kLog2e);
    if (a.chunks > 1) {
      h.load(hs + row);
      ag.load(ge + row);
    } else {
      if (a.init) h.load_n(a.init + srow, K * j, a.N);
      if (dfinal) ag.load_n(dfinal + srow, K * j, a.N);
    }
  }
  const int tiles = (rows.valid + TT - 1) / TT;  // those that hold a token
  Tokens<T, TT, GATE> cur, nxt;
  cur.template load<false, false>(a, p, rows, 0);
  __syncthreads();

  // states at the start of every tile
  for (int i = 0; i + 1 < tiles; ++i) {
    h.store(&slot[wave][i][lane * K]);
    const int t = i * TT;
    nxt.template load<false, false>(a, p, rows, t + TT);
    float raw[OWN], d[OWN], w[OWN];
    cur.steps(a, rows, t, bias, raw, d);
#pragma unroll
    for (int o = 0; o < OWN; ++o) w[o] = d[o] * to_f32(cur.u[o]);
    auto token = [&](int r, float dv, float wv) {
      States<K> B;
      B.load(&sB[i * TT + r][K * j]);
#pragma unroll
      for (int k = 0; k < K; ++k)
        h.v[k] = __builtin_fmaf(fast_exp2(dv * A2.v[k]), h.v[k], wv * B.v[k]);
    };
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      token(4 * o, of_lane<0>(d[o]), of_lane<0>(w[o]));
      token(4 * o + 1, of_lane<1>(d[o]), of_lane<1>(w[o]));
      token(4 * o + 2, of_lane<2>(d[o]), of_lane<2>(w[o]));
      token(4 * o + 3, of_lane<3>(d[o]), of_lane<3>(w[o]));
    }
    cur = nxt;
  }
  float dDs = 0.f, dbs = 0.f;
  if (tiles > 0) {
    h.store(&slot[wave][tiles - 1][lane * K]);
    cur.template load<true, true>(a, p, rows, (tiles - 1) * TT);
  }
  T* dub = du + (p.b * a.L + p.t0) * a.Dm + p.c0;
  T* ddtb = ddt + (p.b * a.L + p.t0) * a.Dm + p.c0;
  T* dzb = GATE ? dz + (p.b * a.L + p.t0) * dzs + p.c0 : nullptr;
  const unsigned dzoff = ((unsigned)j * (unsigned)dzs + p.at) * (unsigned)sizeof(T);
  for (int i = tiles - 1; i >= 0; --i) {
    const int t = i * TT;
    if (i > 0) nxt.template load<true, true>(a, p, rows, t - TT);
    float d[OWN], w[OWN], q[OWN], raw[OWN], s1[OWN], s2[OWN], s3[OWN];
    cur.steps(a, rows, t, bias, raw, d);
    cur.grads(q);
#pragma unroll
    for (int o = 0; o < OWN; ++o) w[o] = d[o] * to_f32(cur.u[o]);
    // forward: states and decays of the tile, dC and the gate's sum C h
    float x[TT][K], hh[TT][K], v[M];
    States<K> h0;
    h0.load(&slot[wave][i][lane * K]);
    float* res = &slot[wave][i][0];  // dB and dC take the place of the states just read
    float part[4];
    auto forward = [&](int r, float dv, float wv, float qv) {
      States<K> B, C;
      B.load(&sB[t + r][K * j]);
      C.load(&sC[t + r][K * j]);
      float y = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        x[r][k] = fast_exp2(dv * A2.v[k]);
        hh[r][k] = __builtin_fmaf(x[r][k], r ? hh[r ? r - 1 : 0][k] : h0.v[k], wv * B.v[k]);
        v[r % GT * K + k] = qv * hh[r][k];
        if constexpr (GATE) y = __builtin_fmaf(C.v[k], hh[r][k], y);
      }
      part[r & 3] = y;
      if ((r + 1) % GT == 0) {
        sum_channels<M>(v, lane);
        store_sums<M, K>(res + (TT + r + 1 - GT) * NP, v, lane);
      }
    };
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      forward(4 * o, of_lane<0>(d[o]), of_lane<0>(w[o]), of_lane<0>(q[o]));
      forward(4 * o + 1, of_lane<1>(d[o]), of_lane<1>(w[o]), of_lane<1>(q[o]));
      forward(4 * o + 2, of_lane<2>(d[o]), of_lane<2>(w[o]), of_lane<2>(q[o]));
      forward(4 * o + 3, of_lane<3>(d[o]), of_lane<3>(w[o]), of_lane<3>(q[o]));
      s3[o] = GATE ? quad_sums(part, j) : 0.f;
    }
    // tokens behind the sequence keep its last state and add nothing to dA: the
    // states before them are taken as 0, or an infinite one would be 0 * infinity.
    // The branch also keeps the two halves of a tile apart: scheduled into each
    // other they take 228 registers instead of 167, two wavefronts per SIMD instead
    // of three (2 x 4096 x 1536 x 16: 225 us, 200 with it)
    if (t + TT > rows.valid) {
#pragma unroll
      for (int r = 0; r < TT; ++r) {
        if (t + r + 1 >= rows.valid) {
#pragma unroll
          for (int k = 0; k < K; ++k) hh[r][k] = 0.f;
        }
      }
    }
    // reverse: the gradients of the states
    float gAs[4];
    auto reverse = [&](int r, float dv, float wv, float qv) {
      States<K> B, C;
      B.load(&sB[t + r][K * j]);
      C.load(&sC[t + r][K * j]);
      float gB = 0.f, gA = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float g = __builtin_fmaf(qv, C.v[k], ag.v[k]);
        v[r % GT * K + k] = g * wv;
        gB = __builtin_fmaf(g, B.v[k], gB);
        ag.v[k] = x[r][k] * g;
        const float m = ag.v[k] * (r ? hh[r ? r - 1 : 0][k] : h0.v[k]);
        gA = __builtin_fmaf(A2.v[k], m, gA);
        dA.v[k] = __builtin_fmaf(dv, m, dA.v[k]);
      }
      part[r & 3] = gB;
      gAs[r & 3] = gA;
      if (r % GT == 0) {
        sum_channels<M>(v, lane);
        store_sums<M, K>(res + r * NP, v, lane);
      }
    };
#pragma unroll
    for (int o = OWN - 1; o >= 0; --o) {
      reverse(4 * o + 3, of_lane<3>(d[o]), of_lane<3>(w[o]), of_lane<3>(q[o]));
      reverse(4 * o + 2, of_lane<2>(d[o]), of_lane<2>(w[o]), of_lane<2>(q[o]));
      reverse(4 * o + 1, of_lane<1>(d[o]), of_lane<1>(w[o]), of_lane<1>(q[o]));
      reverse(4 * o, of_lane<0>(d[o]), of_lane<0>(w[o]), of_lane<0>(q[o]));
      s1[o] = quad_sums(part, j);
      s2[o] = quad_sums(gAs, j);
    }
    const bool full = rows.whole && t + TT <= rows.valid;
    const int ty = fresh(t);
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
      const int tq = t + 4 * o + j;
      const float u = to_f32(cur.u[o]);
      float dd = __builtin_fmaf(s1[o], u, s2[o] * (1.f / kLog2e));
      if (a.softplus) dd *= sigmoid_f32(raw[o]);
      float dzv = 0.f;
      if constexpr (GATE) {
        const float zv = to_f32(cur.z[o]), sg = sigmoid_f32(zv);
        dzv = to_f32(cur.dy[o]) * __builtin_fmaf(Dv, u, s3[o]) *
              (sg * __builtin_fmaf(zv, 1.f - sg, 1.f));
      }
      float duv = __builtin_fmaf(s1[o], d[o], Dv * q[o]);
      dDs = __builtin_fmaf(q[o], u, dDs);
      const int64_t at = (int64_t)(ty + 4 * o) * a.Dm, zat = (int64_t)(ty + 4 * o) * dzs;
      if (full) {
        dbs += dd;
        lane_at(dub + at, rows.off) = from_f32<T>(duv);
        lane_at(ddtb + at, rows.off) = from_f32<T>(dd);
        if constexpr (GATE) lane_at(dzb + zat, dzoff) = from_f32<T>(dzv);
      } else if (p.live && tq < rows.n) {
        if (tq >= rows.valid) dd = duv = dzv = 0.f;
        dbs += dd;
        lane_at(dub + at, rows.off) = from_f32<T>(duv);
        lane_at(ddtb + at, rows.off) = from_f32<T>(dd);
        if constexpr (GATE) lane_at(dzb + zat, dzoff) = from_f32<T>(dzv);
      }
    }
    cur = nxt;
  }

  // what is left of the chunk lies behind the sequence
  if (p.live) {
    for (int t = tiles * TT; t + j < rows.n; t += 4) {
      lane_at(dub + (int64_t)t * a.Dm, rows.off) = (T)0.f;
      lane_at(ddtb + (int64_t)t * a.Dm, rows.off) = (T)0.f;
      if constexpr (GATE) lane_at(dzb + (int64_t)t * dzs, dzoff) = (T)0.f;
    }
    if (dinit && p.chunk == 0) ag.store_n(dinit + srow, K * j, a.N);
    float* pa = part_a + (p.b * a.chunks + p.chunk) * (a.Dm * (a.N + 2));
    dA.store_n(pa + p.c * a.N, K * j, a.N);
    dDs = quad_sum(dDs);
    dbs = quad_sum(dbs);
    if (j == 0) {
      pa[a.Dm * a.N + p.c] = dDs;
      pa[a.Dm * (a.N + 1) + p.c] = dbs;
    }
  }

  // dB and dC of the chunk: the four wavefronts' sums
  __syncthreads();
  const int64_t tile = blockIdx.x % (unsigned)(a.G * a.tiles) % (unsigned)a.tiles;
  const int64_t B = gridDim.y;
#pragma unroll
  for (int arr = 0; arr < 2; ++arr) {
    float* out = part_bc + ((arr * a.tiles + tile) * B + p.b) * a.L * a.G * NP;
    for (int i = threadIdx.x; i < Q * NP; i += 64 * kQuadWaves) {
      const int t = i / NP, n = i % NP;
      if (p.t0 + t < p.t1) {
        float s = 0.f;
        if (t < rows.valid) {
#pragma unroll
          for (int w = 0; w < kQuadWaves; ++w)
            s += slot[w][t / TT][arr * TT * NP + t % TT * NP + n];
        }
        out[((p.t0 + t) * a.G + p.g) * NP + n] = s;
      }
    }
  }
}

// The last sums in one launch: the first `first` workgroups add dB and dC
// [B, L, G, N] from the channel tiles' parts, the others dA, dD and ddt_bias
// from the chunks'.
template <typename T>
__global__ void __launch_bounds__(64 * kSumWaves) scan_bwd_sums_kernel(
    const float* __restrict__ part, int64_t tiles, int64_t count, int NP, int N,
    T* __restrict__ dB, T* __restrict__ dC, unsigned first, const float* __restrict__ sums,
    int64_t P, int64_t M, SumOuts out) {
  __shared__ float red[kSumWaves][64];
  if (blockIdx.x >= first) {
    sum_columns(sums, P, M, out, blockIdx.x - first, red);
    return;
  }
  const int64_t id = (int64_t)blockIdx.x * (64 * kSumWaves) + threadIdx.x;
  if (id >= 2 * count) return;
  const int64_t arr = id / count, i = id % count;
  const int n = (int)(i % NP);
  if (n >= N) return;
  const float* p = part + arr * tiles * count + i;
  float s = 0.f;
#pragma unroll 8
  for (int64_t t = 0; t < tiles; ++t) s += p[t * count];
  (arr ? dC : dB)[i / NP * N + n] = from_f32<T>(s);
}

// Chunks: as long as the tile-start states fit in LDS (a chunk's states are
// written and read five times), shorter, down to 16 tokens, where that leaves
// fewer than two workgroups for each CU.
ScanSplit backward_split(const ScanDims& d) {
  ScanSplit p;
  p.len = bwd_chunk(scan_k(d.N));
  const int64_t per = d.B * scan_channel_tiles(d);
  while (p.len > 16 && per * ((d.L + p.len - 1) / p.len) < 512) p.len /= 2;
  p.chunks = (d.L + p.len - 1) / p.len;
  return p;
}

struct BwdParts {
  size_t states, steps, bc, sums, total;  // bytes; states: each of hs and ge; steps: sum_d
};

BwdParts backward_parts(const ScanDims& d) {
  const ScanSplit p = backward_split(d);
  const int64_t NP = 4 * scan_k(d.N), tiles = (d.D / d.G + 63) / 64;
  auto round = [](int64_t n) { return ((size_t)n * sizeof(float) + 255) & ~(size_t)255; };
  BwdParts w;
  w.states = p.chunks > 1 ? round(d.B * p.chunks * d.D * NP) : 0;
  w.steps = p.chunks > 1 ? round(d.B * p.chunks * d.D) : 0;
  w.bc = round(2 * tiles * d.B * d.L * d.G * NP);
  w.sums = round(d.B * p.chunks * d.D * (d.N + 2));
  w.total = 2 * w.states + w.steps + w.bc + w.sums;
  return w;
}

template <typename T, int K>
hipError_t backward_t(const ScanDims& d, const ScanSplit& p, const ScanArgs& a, const void* dy,
                      const float* dfinal, void* du, void* ddt, float* dA, void* dB, void* dC,
                      float* dD, void* dz, float* ddt_bias, float* dinit, char* ws,
                      hipStream_t s) {
  constexpr int NP = 4 * K, threads = 64 * kQuadWaves;
  const BwdParts w = backward_parts(d);
  float* hs = (float*)ws;
  float* ge = (float*)(ws + w.states);
  float* sum_d = (float*)(ws + 2 * w.states);
  float* bc = (float*)(ws + 2 * w.states + w.steps);
  float* sums = (float*)(ws + 2 * w.states + w.steps + w.bc);
  const dim3 grid((unsigned)(p.chunks * scan_channel_tiles(d)), (unsigned)d.B);
  if (p.chunks > 1) {
    if (a.z)
      scan_bwd_ends_kernel<T, K, true><<<grid, threads, 0, s>>>(a, (const T*)dy, hs, sum_d, ge);
    else
      scan_bwd_ends_kernel<T, K, false><<<grid, threads, 0, s>>>(a, (const T*)dy, hs, sum_d, ge);
    const dim3 cols((unsigned)((d.D * NP + 63) / 64), (unsigned)d.B);
    scan_bwd_carry_kernel<<<cols, 64 * carry_waves(p.chunks), 0, s>>>(a, NP, hs, sum_d, ge, dfinal);
  }
  if (a.z)
    scan_bwd_main_kernel<T, K, true><<<grid, threads, 0, s>>>(
        a, (const T*)dy, dfinal, hs, ge, (T*)du, (T*)ddt, (T*)dz, d.dzs, dinit, bc, sums);
  else
    scan_bwd_main_kernel<T, K, false><<<grid, threads, 0, s>>>(
        a, (const T*)dy, dfinal, hs, ge, (T*)du, (T*)ddt, nullptr, 0, dinit, bc, sums);
  const int64_t count = d.B * d.L * d.G * NP, M = d.D * (d.N + 2);
  const int64_t ends[3] = {d.D * d.N, d.D * (d.N + 1), M};
  float* const outs[3] = {dA, dD, ddt_bias};
  const unsigned first = (unsigned)((2 * count + 64 * kSumWaves - 1) / (64 * kSumWaves));
  scan_bwd_sums_kernel<T><<<first + (unsigned)((M + 63) / 64), 64 * kSumWaves, 0, s>>>(
      bc, a.tiles, count, NP, a.N, (T*)dB, (T*)dC, first, sums, d.B * p.chunks, M,
      sum_outs(ends, outs));
  return hipGetLastError();
}

template <typename T, typename... R>
hipError_t backward_by_k(const ScanDims& d, R... r) {
  switch (scan_k(d.N)) {
    case 1: return backward_t<T, 1>(d, r...);
    case 2: return backward_t<T, 2>(d, r...);
    case 4: return backward_t<T, 4>(d, r...);
    case 8: return backward_t<T, 8>(d, r...);
    default: return backward_t<T, 16>(d, r...);
  }
}

}  // namespace

size_t scan_backward_bytes(const ScanDims& d) { return backward_parts(d).total; }

hipError_t launch_selective_scan_backward(
    const ScanDims& d, const void* u, const void* dt, const float* A, const void* B, const void* C,
    const float* D, const void* z, const float* dt_bias, const float* init, const int32_t* lengths,
    const void* dy, const float* dfinal, void* du, void* ddt, float* dA, void* dB, void* dC,
    float* dD, void* dz, float* ddt_bias, float* dinit, void* ws, hipStream_t s) {
  const ScanSplit p = backward_split(d);
  const ScanArgs a = scan_args(d, p, u, dt, A, B, C, D, z, dt_bias, init, lengths);
  return d.bf16 ? backward_by_k<bf16>(d, p, a, dy, dfinal, du, ddt, dA, dB, dC, dD, dz, ddt_bias,
                                      dinit, (char*)ws, s)
                : backward_by_k<float>(d, p, a, dy, dfinal, du, ddt, dA, dB, dC, dD, dz, ddt_bias,
                                       dinit, (char*)ws, s);
}

}  // namespace m2
