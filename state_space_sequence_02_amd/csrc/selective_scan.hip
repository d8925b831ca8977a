// selective_scan: the SSD's recurrence with a decay of its own for every
// (channel, state), where the SSD has one per head:
//
//     d = softplus(dt + dt_bias) (or dt);  h[n] = exp(d A[n]) h[n] + d u B[n]
//     s = sum_n C[n] h[n] + D u;           y = s silu(z) (or s)
//
// The decays of a token differ by state, so no matrix product forms the
// interaction of two tokens as in the SSD; what is left is one step per
// (token, channel, state): an exponential and four float32 operations.  The
// counters put a wavefront's exponential at two issue slots of the vector ALU
// and the others at one: six slots, against 6-8 bytes of HBM traffic per
// (token, channel).  At 16 states the vector ALU bounds it; with a token's
// own work (softplus, gate, loads, the sum over states) the pass that writes
// the outputs takes 9.1 slots per step, the one for the chunks' ends 6.7.
//
// Where batch * channels fill the device, one pass walks all tokens.  Where
// they do not (a long prompt, a small batch) the sequence is cut into
// chunks: a first pass finds the state each chunk reaches from zero and its
// sum of d (the decay over the chunk is exp(A sum d)), a small kernel carries
// the state over the chunks, and the full pass runs on all chunks at once
// from their start states.  That computes the exponentials twice.
#include "selective_scan.h"

#include <type_traits>

namespace m2 {

namespace {

constexpr int kStageTokens = 32;  // tokens whose B and C are in LDS at once (twice)
constexpr int fwd_tile(int K) { return K <= 8 ? 16 : 8; }

// OUT: the outputs, from the chunks' start states; else the states that the
// chunks reach from zero and their sums of d.
template <typename T, int K, bool GATE, bool OUT>
__global__ void __launch_bounds__(64 * kQuadWaves) scan_fwd_kernel(
    ScanArgs a, T* __restrict__ y, float* __restrict__ hs, float* __restrict__ sum_d,
    float* final_state) {
  constexpr int NP = 4 * K, TT = fwd_tile(K), OWN = TT / 4, S = kStageTokens;
  constexpr int THREADS = 64 * kQuadWaves, EACH = S * NP > THREADS ? S * NP / THREADS : 1;
  __shared__ __align__(16) float sB[2][S][NP], sC[2][OUT ? S : 1][NP];
  const int j = lane_id() & 3;
  const ScanPlace p = scan_place(a);
  const Rows<T> r(a, p, (const T*)a.u, j);
  const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f;
  const float Dv = OUT && a.D ? a.D[p.c] : 0.f;
  States<K> A2, h;
  A2.load_n(a.A + p.c * a.N, K * j, a.N, kLog2e);
#pragma unroll
  for (int k = 0; k < K; ++k) h.v[k] = 0.f;
  const int64_t hrow = ((p.b * a.chunks + p.chunk) * a.Dm + p.c) * NP + K * j;
  const int64_t srow = (p.b * a.Dm + p.c) * a.N;
  if constexpr (OUT) {
    if (a.chunks > 1)
      h.load(hs + hrow);
    else if (a.init)
      h.load_n(a.init + srow, K * j, a.N);
  }
  T* yb = OUT ? y + (p.b * a.L + p.t0) * a.Dm + p.c0 : nullptr;

  // B and C: thread -> state bn of tokens bt, bt + THREADS / NP, ..
  const int bt = threadIdx.x / NP, bn = threadIdx.x % NP;
  const T* Bb = (const T*)a.B + (p.b * a.L + p.t0) * a.bs + (int64_t)p.g * a.N;
  const T* Cb = (const T*)a.C + (p.b * a.L + p.t0) * a.cs + (int64_t)p.g * a.N;
  const bool state = bn < a.N && bt < S;
  const unsigned boff = state ? ((unsigned)bt * (unsigned)a.bs + bn) * (unsigned)sizeof(T) : 0u;
  const unsigned coff = state ? ((unsigned)bt * (unsigned)a.cs + bn) * (unsigned)sizeof(T) : 0u;
  T hb[EACH], hc[EACH];
  auto load_bc = [&](int t) {
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
      const int q = t + i * (THREADS / NP);
      hb[i] = hc[i] = (T)0.f;
      if (state && q + bt < r.valid) {
        hb[i] = lane_at(Bb + (int64_t)q * a.bs, boff);
        if constexpr (OUT) hc[i] = lane_at(Cb + (int64_t)q * a.cs, coff);
      }
    }
  };
  auto stage_bc = [&](int buf) {
    if (bt < S) {
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        sB[buf][bt + i * (THREADS / NP)][bn] = to_f32(hb[i]);
        if constexpr (OUT) sC[buf][bt + i * (THREADS / NP)][bn] = to_f32(hc[i]);
      }
    }
  };

  Tokens<T, TT, GATE> cur, nxt;
  float total = 0.f;
  load_bc(0);
  cur.template load<false, OUT>(a, p, r, 0);
  stage_bc(0);
  __syncthreads();
  int buf = 0;
  for (int s0 = 0; s0 < r.n; s0 += S, buf ^= 1) {
    if (s0 + S < r.n) load_bc(s0 + S);
    const int s1 = s0 + S < r.n ? s0 + S : r.n;
    for (int t = s0; t < s1; t += TT) {
      if (t + TT < r.n) nxt.template load<false, OUT>(a, p, r, t + TT);
      float raw[OWN], d[OWN], w[OWN], part[4];
      cur.steps(a, r, t, bias, raw, d);
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        w[i] = d[i] * to_f32(cur.u[i]);
        if constexpr (!OUT) total += d[i];
      }
      auto token = [&](int i, float dv, float wv) {
        States<K> B, C;
        B.load(&sB[buf][t - s0 + i][K * j]);
        if constexpr (OUT) C.load(&sC[buf][t - s0 + i][K * j]);
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          h.v[k] = __builtin_fmaf(fast_exp2(dv * A2.v[k]), h.v[k], wv * B.v[k]);
          if constexpr (OUT) s = __builtin_fmaf(h.v[k], C.v[k], s);
        }
        part[i & 3] = s;
      };
      float out[OWN];
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        token(4 * i, of_lane<0>(d[i]), of_lane<0>(w[i]));
        token(4 * i + 1, of_lane<1>(d[i]), of_lane<1>(w[i]));
        token(4 * i + 2, of_lane<2>(d[i]), of_lane<2>(w[i]));
        token(4 * i + 3, of_lane<3>(d[i]), of_lane<3>(w[i]));
        if constexpr (OUT) {
          out[i] = __builtin_fmaf(Dv, to_f32(cur.u[i]), quad_sums(part, j));
          if constexpr (GATE) {
            const float zv = to_f32(cur.z[i]);
            out[i] *= zv * sigmoid_f32(zv);
          }
        }
      }
      if constexpr (OUT) {
        const int ty = fresh(t);
        if (r.whole && t + TT <= r.valid) {
#pragma unroll
          for (int i = 0; i < OWN; ++i)
            lane_at(yb + (int64_t)(ty + 4 * i) * a.Dm, r.off) = from_f32<T>(out[i]);
        } else if (p.live) {
#pragma unroll
          for (int i = 0; i < OWN; ++i)
            if (t + 4 * i + j < r.n)
              lane_at(yb + (int64_t)(ty + 4 * i) * a.Dm, r.off) =
                  from_f32<T>(t + 4 * i + j < r.valid ? out[i] : 0.f);
        }
      }
      cur = nxt;
    }
    if (s0 + S < r.n) stage_bc(buf ^ 1);
    __syncthreads();
  }

  if constexpr (OUT) {
    if (final_state && p.live && p.chunk == a.chunks - 1)
      h.store_n(final_state + srow, K * j, a.N);
  } else {
    total = quad_sum(total);
    if (p.live) {
      h.store(hs + hrow);
      if (j == 0) sum_d[(p.b * a.chunks + p.chunk) * a.Dm + p.c] = total;
    }
  }
}

// hs: the states the chunks reach from zero -> the states they start from.  A
// workgroup takes 64 columns of (channel, padded state); each of its
// wavefronts composes its share of the chunks into one (decay, state reached),
// the shares are carried through LDS, and each wavefront walks its share
// again, from registers where it is at most kCarryLoads chunks (up to 16
// wavefronts: 256 chunks).
__global__ void __launch_bounds__(64 * kCarryWaves) scan_carry_kernel(
    ScanArgs a, int NP, float* __restrict__ hs, const float* __restrict__ sum_d) {
  __shared__ float sh[kCarryWaves][64], sp[kCarryWaves][64];
  const int lane = lane_id(), wave = wave_id(), waves = blockDim.x >> 6;
  const int64_t cols = a.Dm * NP, col = (int64_t)blockIdx.x * 64 + lane, b = blockIdx.y;
  const bool live = col < cols;
  const int n = (int)(col % NP);
  const int64_t c = live ? col / NP : 0;
  const float A2 = n < a.N ? a.A[c * a.N + n] * kLog2e : 0.f;
  const int64_t share = (a.chunks + waves - 1) / waves;
  const int64_t c0 = wave * share, c1 = c0 + share < a.chunks ? c0 + share : a.chunks;
  float* hp = hs + b * a.chunks * cols + (live ? col : 0);
  const float* dp = sum_d + b * a.chunks * a.Dm + c;
  float reached[kCarryLoads], d[kCarryLoads];
  auto load = [&](int64_t q) {
#pragma unroll
    for (int k = 0; k < kCarryLoads; ++k) {
      const int64_t i = q + k < c1 ? q + k : c1 - 1;
      reached[k] = hp[i * cols];
      d[k] = dp[i * a.Dm];
    }
  };
  float h = 0.f, total = 0.f;
  for (int64_t q = c0; q < c1; q += kCarryLoads) {
    load(q);
#pragma unroll
    for (int k = 0; k < kCarryLoads; ++k) {
      if (q + k < c1) {
        h = __builtin_fmaf(fast_exp2(A2 * d[k]), h, reached[k]);
        total += d[k];
      }
    }
  }
  sh[wave][lane] = h;
  sp[wave][lane] = fast_exp2(A2 * total);
  __syncthreads();
  if (!live) return;
  float run = a.init && n < a.N ? a.init[(b * a.Dm + c) * a.N + n] : 0.f;
  for (int w = 0; w < wave; ++w) run = __builtin_fmaf(sp[w][lane], run, sh[w][lane]);
  for (int64_t q = c0; q < c1; q += kCarryLoads) {
    if (share > kCarryLoads) load(q);
#pragma unroll
    for (int k = 0; k < kCarryLoads; ++k) {
      if (q + k < c1) {
        hp[(q + k) * cols] = run;
        run = __builtin_fmaf(fast_exp2(A2 * d[k]), run, reached[k]);
      }
    }
  }
}

// One token.  State rows of 4 LPR states: LPR lanes of 16 bytes each.  A thread
// takes its channel's row of SEQS sequences: their states are all requested
// before the first is used, and the channel's parameters are read once.
template <typename T, int LPR, int SEQS>
__global__ void __launch_bounds__(256) scan_step_kernel(ScanArgs a, int B, float* state,
                                                        T* __restrict__ y, int wide) {
  const int n0 = (int)(threadIdx.x % LPR) * 4;
  const unsigned c = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  if (c >= (unsigned)a.Dm) return;  // the lanes of a row leave together
  const unsigned g = a.G == 1 ? 0u : c / (unsigned)(a.Dm / a.G);
  const int b0 = (int)blockIdx.y * SEQS;
  f32x4 h[SEQS];
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    h[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (b0 + i < B) h[i] = *(const f32x4*)(state + ((int64_t)(b0 + i) * a.Dm + c) * a.N + n0);
  }
  const f32x4 A2 = *(const f32x4*)(a.A + (int64_t)c * a.N + n0) * kLog2e;
  const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, Dv = a.D ? a.D[c] : 0.f;
#pragma unroll
  for (int i = 0; i < SEQS; ++i) {
    const int64_t b = b0 + i, row = b * a.Dm + c;
    if (b >= B) return;
    const T* Bp = (const T*)a.B + b * a.bs + (int64_t)g * a.N + n0;
    const T* Cp = (const T*)a.C + b * a.cs + (int64_t)g * a.N + n0;
    float Bv[4], Cv[4];
    if (wide) {
      load_row<T, 4>(Bp, Bv);
      load_row<T, 4>(Cp, Cv);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        Bv[k] = to_f32(Bp[k]);
        Cv[k] = to_f32(Cp[k]);
      }
    }
    const float u = to_f32(((const T*)a.u)[row]);
    float d = to_f32(((const T*)a.dt)[row]) + bias;
    if (a.softplus) d = softplus_f32(d);
    const float w = d * u;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      h[i][k] = __builtin_fmaf(fast_exp2(d * A2[k]), h[i][k], w * Bv[k]);
      s = __builtin_fmaf(h[i][k], Cv[k], s);
    }
    *(f32x4*)(state + row * a.N + n0) = h[i];
#pragma unroll
    for (int off = 1; off < LPR; off <<= 1) s += __shfl_xor(s, off, 64);
    if (n0 == 0) {
      s = __builtin_fmaf(Dv, u, s);
      if (a.z) {
        const float zv = to_f32(((const T*)a.z)[b * a.zs + c]);
        s *= zv * sigmoid_f32(zv);
      }
      y[row] = from_f32<T>(s);
    }
  }
}

// One token, any number of states: 16 lanes per row.
template <typename T>
__global__ void __launch_bounds__(256) scan_step_any_kernel(ScanArgs a, int64_t rows, float* state,
                                                            T* __restrict__ y) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = id / 16;
  if (row >= rows) return;
  const int l = (int)(id % 16);
  const int64_t b = row / a.Dm, c = row % a.Dm;
  const int64_t g = c / (a.Dm / a.G);
  const float u = to_f32(((const T*)a.u)[row]);
  float d = to_f32(((const T*)a.dt)[row]) + (a.dt_bias ? a.dt_bias[c] : 0.f);
  if (a.softplus) d = softplus_f32(d);
  float s = 0.f;
  for (int n = l; n < a.N; n += 16) {
    const float Bv = to_f32(((const T*)a.B)[b * a.bs + g * a.N + n]);
    const float Cv = to_f32(((const T*)a.C)[b * a.cs + g * a.N + n]);
    const float v = __builtin_fmaf(fast_exp2(d * kLog2e * a.A[c * a.N + n]), state[row * a.N + n],
                                   d * u * Bv);
    state[row * a.N + n] = v;
    s = __builtin_fmaf(v, Cv, s);
  }
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) s += __shfl_xor(s, off, 64);
  if (l == 0) {
    if (a.D) s = __builtin_fmaf(a.D[c], u, s);
    if (a.z) {
      const float zv = to_f32(((const T*)a.z)[b * a.zs + c]);
      s *= zv * sigmoid_f32(zv);
    }
    y[row] = from_f32<T>(s);
  }
}

// Chunks of the forward.  One pass over whole sequences where the channel
// tiles nearly fill the device (2048 tokens x 2048 channels x 16 states:
// batch 16, 512 workgroups, 385 us in one pass and 460 in chunks; batch 12,
// 384 workgroups, 380 and 356), or where there is little to divide; else
// chunks of 64 tokens (1 x 512 x 2048: 25 us, 37 with 128) and, from 4096
// workgroups on, longer ones.
ScanSplit forward_split(const ScanDims& d) {
  const int64_t blocks = d.B * scan_channel_tiles(d);
  ScanSplit p;
  if (d.L <= 128 || blocks >= 448) {
    p.len = (d.L + 15) / 16 * 16;
  } else {
    p.len = 64;
    while (blocks * ((d.L + p.len - 1) / p.len) > 4096) p.len *= 2;
  }
  p.chunks = (d.L + p.len - 1) / p.len;
  return p;
}

template <typename T, int K>
hipError_t forward_t(const ScanDims& d, const ScanSplit& p, const ScanArgs& a, void* y,
                     float* final_state, float* hs, float* sum_d, hipStream_t s) {
  constexpr int threads = 64 * kQuadWaves;
  const dim3 grid((unsigned)(p.chunks * scan_channel_tiles(d)), (unsigned)d.B);
  if (p.chunks > 1) {
    scan_fwd_kernel<T, K, false, false><<<grid, threads, 0, s>>>(a, nullptr, hs, sum_d, nullptr);
    const dim3 cols((unsigned)((d.D * 4 * K + 63) / 64), (unsigned)d.B);
    scan_carry_kernel<<<cols, 64 * carry_waves(p.chunks), 0, s>>>(a, 4 * K, hs, sum_d);
  }
  if (a.z)
    scan_fwd_kernel<T, K, true, true><<<grid, threads, 0, s>>>(a, (T*)y, hs, nullptr, final_state);
  else
    scan_fwd_kernel<T, K, false, true><<<grid, threads, 0, s>>>(a, (T*)y, hs, nullptr, final_state);
  return hipGetLastError();
}

template <typename T, typename... R>
hipError_t forward_by_k(const ScanDims& d, R... r) {
  switch (scan_k(d.N)) {
    case 1: return forward_t<T, 1>(d, r...);
    case 2: return forward_t<T, 2>(d, r...);
    case 4: return forward_t<T, 4>(d, r...);
    case 8: return forward_t<T, 8>(d, r...);
    default: return forward_t<T, 16>(d, r...);
  }
}

size_t states_bytes(const ScanDims& d, const ScanSplit& p) {
  return (size_t)(d.B * p.chunks * d.D * 4 * scan_k(d.N)) * sizeof(float);
}

constexpr int kStepSeqs = 2;
constexpr int64_t kStepThreads = 1 << 19;

template <typename T>
hipError_t step_t(const ScanDims& d, const ScanArgs& a, float* state, void* y, hipStream_t s) {
  const int64_t rows = d.B * d.D;
  const int wide = d.bs % 4 == 0 && d.cs % 4 == 0;
  auto vec = [&](auto lanes) {
    constexpr int LPR = decltype(lanes)::value, SEQS = kStepSeqs;
    const unsigned x = (unsigned)((d.D + 256 / LPR - 1) / (256 / LPR));
    if (rows * LPR >= kStepThreads)
      scan_step_kernel<T, LPR, SEQS><<<dim3(x, (unsigned)((d.B + SEQS - 1) / SEQS)), 256, 0, s>>>(
          a, (int)d.B, state, (T*)y, wide);
    else
      scan_step_kernel<T, LPR, 1>
          <<<dim3(x, (unsigned)d.B), 256, 0, s>>>(a, (int)d.B, state, (T*)y, wide);
  };
  switch (d.N) {
    case 4: vec(std::integral_constant<int, 1>()); break;
    case 8: vec(std::integral_constant<int, 2>()); break;
    case 16: vec(std::integral_constant<int, 4>()); break;
    case 32: vec(std::integral_constant<int, 8>()); break;
    case 64: vec(std::integral_constant<int, 16>()); break;
    default:
      scan_step_any_kernel<T><<<(unsigned)((rows * 16 + 255) / 256), 256, 0, s>>>(a, rows, state,
                                                                                  (T*)y);
  }
  return hipGetLastError();
}

}  // namespace

// [batch, chunk, channel, padded state] chunk states, then the chunks' sums
// of d; nothing where one chunk is the sequence.
size_t scan_forward_bytes(const ScanDims& d) {
  const ScanSplit p = forward_split(d);
  if (p.chunks == 1) return 0;
  return states_bytes(d, p) + (size_t)(d.B * p.chunks * d.D) * sizeof(float);
}

hipError_t launch_selective_scan(const ScanDims& d, const void* u, const void* dt, const float* A,
                                 const void* B, const void* C, const float* D, const void* z,
                                 const float* dt_bias, const float* init, const int32_t* lengths,
                                 void* y, float* final_state, void* ws, hipStream_t s) {
  const ScanSplit p = forward_split(d);
  const ScanArgs a = scan_args(d, p, u, dt, A, B, C, D, z, dt_bias, init, lengths);
  float* hs = (float*)ws;
  float* sum_d = p.chunks > 1 ? (float*)((char*)ws + states_bytes(d, p)) : nullptr;
  return d.bf16 ? forward_by_k<bf16>(d, p, a, y, final_state, hs, sum_d, s)
                : forward_by_k<float>(d, p, a, y, final_state, hs, sum_d, s);
}

hipError_t launch_selective_scan_step(const ScanDims& d, const void* u, const void* dt,
                                      const float* A, const void* B, const void* C, const float* D,
                                      const void* z, const float* dt_bias, float* state, void* y,
                                      hipStream_t s) {
  const ScanArgs a = scan_args(d, {1, 1}, u, dt, A, B, C, D, z, dt_bias, nullptr, nullptr);
  return d.bf16 ? step_t<bf16>(d, a, state, y, s) : step_t<float>(d, a, state, y, s);
}

}  // namespace m2
