// selective_scan: the SSD's recurrence with a decay of its own for every
// (channel, state), where the SSD has one per head:
//
//     d = softplus(dt + dt_bias) (or dt);  h[n] = exp(d A[n]) h[n] + d u B[n]
//     s = sum_n C[n] h[n] + D u;           y = s silu(z) (or s)
//
// The decays of a token differ by state, so no matrix product forms the
// interaction of two tokens as in the SSD; what is left is one step per
// (token, channel, state): an exponential and four float32 operations, eight
// issue slots on the vector ALU (the exponential takes four), against 6-8
// bytes of HBM traffic per (token, channel).  At 16 states it is bound by
// the vector ALU.
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

// Tokens of a tile that one thread loads: raw values of u, dt and z, and one
// element of B and of C.
template <typename T, int ROWS>
struct Held {
  T u[ROWS], dt[ROWS], z[ROWS], b, c;
};

// The vector ALU bounds this kernel, so what is the same for a wavefront stays
// off it: a row's address is scalar and lanes add a constant 32-bit offset;
// token counts are 32-bit and scalar; tiles inside the sequence skip the
// masks; two tiles per round alternate the registers of the tile in hand and
// of the one being loaded.
template <typename T, int WV, bool GATE, bool OUT>
__global__ void __launch_bounds__(64 * WV) scan_fwd_kernel(ScanArgs a, T* __restrict__ y,
                                                           float* __restrict__ hs,
                                                           float* __restrict__ sum_d,
                                                           float* final_state) {
  constexpr int TT = scan_tile(WV);
  constexpr int ROWS = TT > WV ? TT / WV : 1;
  constexpr int NP = kScanK * WV;  // states, padded
  constexpr int LOADERS = TT / ROWS;  // wavefronts that load rows
  __shared__ float sd[2][TT][64], su[2][TT][64];
  __shared__ __align__(16) float sB[2][TT][NP], sC[2][OUT ? TT : 1][NP];
  __shared__ float sy[2][OUT ? WV : 1][OUT ? TT : 1][64];
  const int lane = lane_id(), wave = wave_id();
  const ScanPlace p = scan_place(a);
  const int n = (int)(p.t1 - p.t0);  // tokens of this chunk, and those that are no padding
  const int64_t left = p.len - p.t0;
  const int valid = left <= 0 ? 0 : left < n ? (int)left : n;
  const int64_t row0 = p.b * a.L + p.t0;
  const T* ub = (const T*)a.u + row0 * a.Dm + p.c0;
  const T* db = (const T*)a.dt + row0 * a.Dm + p.c0;
  const T* zb = GATE ? (const T*)a.z + row0 * a.zs + p.c0 : nullptr;
  T* yb = OUT ? y + row0 * a.Dm + p.c0 : nullptr;
  const unsigned off = p.at * (unsigned)sizeof(T);
  const int bt = threadIdx.x / NP, bn = threadIdx.x % NP;  // the element of B and C it loads
  const bool bc = bt < TT && bn < a.N;
  const T* Bb = (const T*)a.B + row0 * a.bs + (int64_t)p.g * a.N;
  const T* Cb = (const T*)a.C + row0 * a.cs + (int64_t)p.g * a.N;
  const unsigned boff = bc ? (unsigned)(bt * (int)a.bs + bn) * (unsigned)sizeof(T) : 0u;
  const unsigned coff = bc ? (unsigned)(bt * (int)a.cs + bn) * (unsigned)sizeof(T) : 0u;
  const float bias = a.dt_bias ? a.dt_bias[p.c] : 0.f;
  const float Dv = OUT && a.D ? a.D[p.c] : 0.f;
  const int n0 = kScanK * wave;
  const f32x4 A2 = load_A2(a, p.c, n0);

  f32x4 h = {0.f, 0.f, 0.f, 0.f};
  const int64_t hrow = ((p.b * a.chunks + p.chunk) * a.Dm + p.c) * NP + n0;
  if constexpr (OUT) {
    if (a.chunks > 1)
      h = *(const f32x4*)(hs + hrow);
    else if (a.init)
      h = load_states(a.init + (p.b * a.Dm + p.c) * a.N, n0, a.N);
  }

  auto load = [&](Held<T, ROWS>& r, int t) {
    const int first = t + wave * ROWS;
    if (t + TT <= valid) {
      if (wave < LOADERS) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          r.u[i] = lane_at(ub + (int64_t)(first + i) * a.Dm, off);
          r.dt[i] = lane_at(db + (int64_t)(first + i) * a.Dm, off);
          if constexpr (GATE && OUT) r.z[i] = lane_at(zb + (int64_t)(first + i) * a.zs, off);
        }
      }
      if (bc) {
        r.b = lane_at(Bb + (int64_t)t * a.bs, boff);
        if constexpr (OUT) r.c = lane_at(Cb + (int64_t)t * a.cs, coff);
      }
    } else {
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        r.u[i] = r.dt[i] = r.z[i] = (T)0.f;
        if (wave < LOADERS && first + i < valid) {
          r.u[i] = lane_at(ub + (int64_t)(first + i) * a.Dm, off);
          r.dt[i] = lane_at(db + (int64_t)(first + i) * a.Dm, off);
          if constexpr (GATE && OUT) r.z[i] = lane_at(zb + (int64_t)(first + i) * a.zs, off);
        }
      }
      r.b = r.c = (T)0.f;
      if (bc && t + bt < valid) {
        r.b = lane_at(Bb + (int64_t)t * a.bs, boff);
        if constexpr (OUT) r.c = lane_at(Cb + (int64_t)t * a.cs, coff);
      }
    }
  };
  float total = 0.f;  // sum of d over the chunk's tokens that this thread loaded
  auto stage = [&](const Held<T, ROWS>& r, int t, int buf) {
    if (wave < LOADERS) {
      float d[ROWS];
#pragma unroll
      for (int i = 0; i < ROWS; ++i) d[i] = to_f32(r.dt[i]) + bias;
      if (a.softplus) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) d[i] = softplus_f32(d[i]);
      }
      if (t + TT > valid) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) d[i] = t + wave * ROWS + i < valid ? d[i] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        sd[buf][wave * ROWS + i][lane] = d[i];
        su[buf][wave * ROWS + i][lane] = d[i] * to_f32(r.u[i]);
        if constexpr (!OUT) total += d[i];
      }
    }
    if (bt < TT) {
      sB[buf][bt][bn] = bc ? to_f32(r.b) : 0.f;
      if constexpr (OUT) sC[buf][bt][bn] = bc ? to_f32(r.c) : 0.f;
    }
  };
  // One tile: `cur` is staged in buffer `buf`, the next tile is loaded into
  // `nxt` meanwhile and staged in the other buffer.
  auto tile = [&](const Held<T, ROWS>& cur, Held<T, ROWS>& nxt, int t, int buf) {
    const bool more = t + TT < n;
    if (more) load(nxt, t + TT);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const float d = sd[buf][i][lane], w = su[buf][i][lane];
      const f32x4 Bv = *(const f32x4*)&sB[buf][i][n0];
      f32x4 Cv;
      if constexpr (OUT) Cv = *(const f32x4*)&sC[buf][i][n0];
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kScanK; ++k) {
        h[k] = __builtin_fmaf(fast_exp2(d * A2[k]), h[k], w * Bv[k]);
        if constexpr (OUT) s = __builtin_fmaf(h[k], Cv[k], s);
      }
      if constexpr (OUT) sy[buf][wave][i][lane] = s;
    }
    if (more) stage(nxt, t + TT, buf ^ 1);
    __syncthreads();
    if constexpr (OUT) {
      if (wave < LOADERS && p.live) {
        float s[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
          s[i] = Dv * to_f32(cur.u[i]);
#pragma unroll
          for (int w = 0; w < WV; ++w) s[i] += sy[buf][w][wave * ROWS + i][lane];
          if constexpr (GATE) {
            const float zv = to_f32(cur.z[i]);
            s[i] *= zv * sigmoid_f32(zv);
          }
        }
        const int first = t + wave * ROWS;
        if (t + TT <= valid) {
#pragma unroll
          for (int i = 0; i < ROWS; ++i)
            lane_at(yb + (int64_t)(first + i) * a.Dm, off) = from_f32<T>(s[i]);
        } else {
#pragma unroll
          for (int i = 0; i < ROWS; ++i)
            if (first + i < n)
              lane_at(yb + (int64_t)(first + i) * a.Dm, off) =
                  from_f32<T>(first + i < valid ? s[i] : 0.f);
        }
      }
    }
  };

  Held<T, ROWS> r0, r1;
  load(r0, 0);
  stage(r0, 0, 0);
  __syncthreads();
  for (int t = 0; t < n; t += 2 * TT) {
    tile(r0, r1, t, 0);
    if (t + TT < n) tile(r1, r0, t + TT, 1);
  }

  if constexpr (OUT) {
    if (final_state && p.live && p.chunk == a.chunks - 1)
      store_states(final_state + (p.b * a.Dm + p.c) * a.N, n0, a.N, h);
  } else {
    if (p.live) *(f32x4*)(hs + hrow) = h;
    // the sums of the loading wavefronts, through LDS that no wavefront reads any more
    if (wave < LOADERS) sd[0][wave][lane] = total;
    __syncthreads();
    if (wave == 0 && p.live) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < LOADERS; ++w) s += sd[0][w][lane];
      sum_d[(p.b * a.chunks + p.chunk) * a.Dm + p.c] = s;
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

// Chunks of the forward: one where the channel tiles alone keep the device
// busy, else enough for about 6 workgroups per CU, of at least 64 tokens.
ScanSplit forward_split(const ScanDims& d) {
  const int64_t tile = scan_tile(scan_waves(d.N));
  const int64_t blocks = d.B * scan_channel_tiles(d);
  int64_t chunks = 1;
  if (blocks < 512) chunks = 1536 / blocks;
  const int64_t most = (d.L + 63) / 64;
  if (chunks > most) chunks = most;
  ScanSplit p;
  p.len = ((d.L + chunks - 1) / chunks + tile - 1) / tile * tile;
  p.chunks = (d.L + p.len - 1) / p.len;
  return p;
}

template <typename T, int WV>
hipError_t forward_t(const ScanDims& d, const ScanSplit& p, const ScanArgs& a, void* y,
                     float* final_state, float* hs, float* sum_d, hipStream_t s) {
  const dim3 grid((unsigned)(p.chunks * scan_channel_tiles(d)), (unsigned)d.B);
  if (p.chunks > 1) {
    scan_fwd_kernel<T, WV, false, false><<<grid, 64 * WV, 0, s>>>(a, nullptr, hs, sum_d, nullptr);
    const dim3 cols((unsigned)((d.D * kScanK * WV + 63) / 64), (unsigned)d.B);
    scan_carry_kernel<<<cols, 64 * carry_waves(p.chunks), 0, s>>>(a, kScanK * WV, hs, sum_d);
  }
  if (a.z)
    scan_fwd_kernel<T, WV, true, true><<<grid, 64 * WV, 0, s>>>(a, (T*)y, hs, nullptr, final_state);
  else
    scan_fwd_kernel<T, WV, false, true><<<grid, 64 * WV, 0, s>>>(a, (T*)y, hs, nullptr,
                                                                 final_state);
  return hipGetLastError();
}

template <typename T>
hipError_t forward_by_waves(const ScanDims& d, const ScanSplit& p, const ScanArgs& a, void* y,
                            float* final_state, float* hs, float* sum_d, hipStream_t s) {
  switch (scan_waves(d.N)) {
    case 1: return forward_t<T, 1>(d, p, a, y, final_state, hs, sum_d, s);
    case 2: return forward_t<T, 2>(d, p, a, y, final_state, hs, sum_d, s);
    case 4: return forward_t<T, 4>(d, p, a, y, final_state, hs, sum_d, s);
    case 8: return forward_t<T, 8>(d, p, a, y, final_state, hs, sum_d, s);
    default: return forward_t<T, 16>(d, p, a, y, final_state, hs, sum_d, s);
  }
}

size_t states_bytes(const ScanDims& d, const ScanSplit& p) {
  return (size_t)(d.B * p.chunks * d.D * kScanK * scan_waves(d.N)) * sizeof(float);
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
  return d.bf16 ? forward_by_waves<bf16>(d, p, a, y, final_state, hs, sum_d, s)
                : forward_by_waves<float>(d, p, a, y, final_state, hs, sum_d, s);
}

hipError_t launch_selective_scan_step(const ScanDims& d, const void* u, const void* dt,
                                      const float* A, const void* B, const void* C, const float* D,
                                      const void* z, const float* dt_bias, float* state, void* y,
                                      hipStream_t s) {
  const ScanArgs a = scan_args(d, {1, 1}, u, dt, A, B, C, D, z, dt_bias, nullptr, nullptr);
  return d.bf16 ? step_t<bf16>(d, a, state, y, s) : step_t<float>(d, a, state, y, s);
}

}  // namespace m2
