// norm: layer norm or RMS norm over groups of channels, optionally of
// x * silu(z) (the gate of an SSD layer's output), and its backward pass.
// Per row and group of Dg channels:
//
//     v = x silu(z) or x
//     layer: xh = (v - mean(v)) rstd, rstd = 1 / sqrt(mean((v - mean)^2) + eps)
//     RMS:   xh = v rstd,             rstd = 1 / sqrt(mean(v^2) + eps)
//     y = xh w + bias
//     d = dy w;  dv = rstd (d - mean(d) [layer only] - xh mean(d xh))
//     dx = dv silu(z), dz = dv x silu'(z);  dw = sum over rows dy xh, dbias = sum dy
//
// Both are bound by HBM: every row is read once, held in registers across
// the reductions (a second pass over the registers forms the variance from
// the centred values, so a large mean costs no digits), and written once.
// The backward recomputes the statistics from the row it has to read anyway.
// A team of lanes (32 to 1024, the smallest whose registers hold a group)
// takes one group of channels and walks rows with it: the weights and the
// weights' gradients stay in the lanes that own their columns.
#include <type_traits>

#include "launch.h"
#include "rowvec.h"

namespace m2 {

namespace {

// Sums N values over the team; every lane of it ends with the totals.
template <int TEAM, int N>
__device__ __forceinline__ void team_sum(float (&s)[N], float (*red)[N]) {
  constexpr int LANES = TEAM < 64 ? TEAM : 64;
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = lanes_sum<LANES>(s[i]);
  if constexpr (TEAM > 64) {
    const int wave = wave_id();
    if (lane_id() == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) red[wave][i] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int w = 0; w < TEAM / 64; ++w) s[i] += red[w][i];
    }
    __syncthreads();  // red is free for the next sum
  }
}

template <typename T, int V, int NV>
struct Row {
  raw_t<T, V> r[NV];
  __device__ __forceinline__ float at(int k, int e) const { return elem<T, V>(r[k], e); }
  __device__ __forceinline__ void load(const T* p, int lane, int team, int64_t n) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int64_t c = (int64_t)(k * team + lane) * V;
      r[k] = raw_t<T, V>{};
      if (c < n) r[k] = *(const raw_t<T, V>*)(p + c);
    }
  }
};

template <typename T, int V, int NV>
__device__ __forceinline__ void store(T* p, int lane, int team, int64_t n,
                                      const float (&v)[NV][V]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t c = (int64_t)(k * team + lane) * V;
    if (c < n) store_row<T, V>(p + c, v[k]);
  }
}

// Float parameters of this lane's columns (0 past the group).  With vectors
// the columns start at a multiple of 16 bytes.
template <int V, int NV>
__device__ __forceinline__ void params(const float* p, int lane, int team, int64_t n,
                                       float (&v)[NV][V]) {
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int64_t c = (int64_t)(k * team + lane) * V;
#pragma unroll
    for (int e = 0; e < V; ++e) v[k][e] = 0.f;
    if (p && c < n) {
      if constexpr (V == 1) {
        v[k][0] = p[c];
      } else {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          const f32x4 q = *(const f32x4*)(p + c + e);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[k][e + i] = q[i];
        }
      }
    }
  }
}

constexpr int block_of(int team) { return team < 256 ? 256 : team; }

template <typename T, int V, int NV, int TEAM, bool GATE>
__global__ void __launch_bounds__(block_of(TEAM)) norm_fwd_kernel(
    const T* __restrict__ x, const T* __restrict__ z, const float* __restrict__ w,
    const float* __restrict__ bias, T* __restrict__ y, int64_t R, int64_t D, int64_t Dg,
    int64_t xs, int64_t zs, unsigned G, float eps, int layer) {
  constexpr int TEAMS = block_of(TEAM) / TEAM;
  __shared__ float red1[TEAM / 64 + 1][1];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int64_t g0 = blockIdx.x % G * Dg;
  const int64_t step = (int64_t)(gridDim.x / G) * TEAMS;
  const float inv = 1.f / (float)Dg;
  float wv[NV][V], bv[NV][V];
  params<V, NV>(w + g0, lane, TEAM, Dg, wv);
  params<V, NV>(bias ? bias + g0 : nullptr, lane, TEAM, Dg, bv);
  // every team of a workgroup makes the same number of rounds: the sums of
  // teams over 64 lanes meet at barriers
  const int64_t first = (int64_t)(blockIdx.x / G) * TEAMS;
  for (int64_t r0 = first; r0 < R; r0 += step) {
    const int64_t r = r0 + team;
    const bool live = r < R;
    Row<T, V, NV> rx, rz;
    rx.load(x + r * xs + g0, lane, TEAM, live ? Dg : 0);
    if constexpr (GATE) rz.load(z + r * zs + g0, lane, TEAM, live ? Dg : 0);
    float v[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        v[k][e] = rx.at(k, e);
        if constexpr (GATE) v[k][e] *= rz.at(k, e) * sigmoid_f32(rz.at(k, e));
      }
    float s[1];
    if (layer) {
      s[0] = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += v[k][e];
      team_sum<TEAM, 1>(s, red1);
      const float mean = s[0] * inv;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e)
          v[k][e] = (int64_t)(k * TEAM + lane) * V + e < Dg ? v[k][e] - mean : 0.f;
    }
    s[0] = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) s[0] = __builtin_fmaf(v[k][e], v[k][e], s[0]);
    team_sum<TEAM, 1>(s, red1);
    const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(s[0], inv, eps));
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e)
        v[k][e] = __builtin_fmaf(v[k][e] * rstd, wv[k][e], bv[k][e]);
    if (live) store<T, V, NV>(y + r * D + g0, lane, TEAM, Dg, v);
  }
}

template <typename T, int V, int NV, int TEAM, bool GATE>
__global__ void __launch_bounds__(block_of(TEAM)) norm_bwd_kernel(
    const T* __restrict__ x, const T* __restrict__ z, const float* __restrict__ w,
    const T* __restrict__ dy, T* __restrict__ dx, T* __restrict__ dz, float* __restrict__ part,
    int64_t R, int64_t D, int64_t Dg, int64_t xs, int64_t zs, int64_t dzs, unsigned G, float eps,
    int layer, int with_bias) {
  constexpr int TEAMS = block_of(TEAM) / TEAM;
  __shared__ float red1[TEAM / 64 + 1][1], red3[TEAM / 64 + 1][3];
  __shared__ float cols[TEAMS > 1 ? TEAMS - 1 : 1][TEAMS > 1 ? NV * V : 1][TEAM];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int64_t g0 = blockIdx.x % G * Dg;
  const int64_t step = (int64_t)(gridDim.x / G) * TEAMS;
  const float inv = 1.f / (float)Dg;
  float wv[NV][V], dw[NV][V], db[NV][V];
  params<V, NV>(w + g0, lane, TEAM, Dg, wv);
  params<V, NV>(nullptr, lane, TEAM, Dg, dw);
  params<V, NV>(nullptr, lane, TEAM, Dg, db);
  const int64_t first = (int64_t)(blockIdx.x / G) * TEAMS;
  for (int64_t r0 = first; r0 < R; r0 += step) {
    const int64_t r = r0 + team;
    const bool live = r < R;
    Row<T, V, NV> rx, rz, rg;
    rx.load(x + r * xs + g0, lane, TEAM, live ? Dg : 0);
    rg.load(dy + r * D + g0, lane, TEAM, live ? Dg : 0);
    if constexpr (GATE) rz.load(z + r * zs + g0, lane, TEAM, live ? Dg : 0);
    // the gate's sigmoid is used twice: kept where there are registers for it
    constexpr bool KEEP = GATE && NV * V <= 8;
    float v[NV][V], sg[KEEP ? NV : 1][KEEP ? V : 1];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        v[k][e] = rx.at(k, e);
        if constexpr (GATE) {
          const float q = sigmoid_f32(rz.at(k, e));
          v[k][e] *= rz.at(k, e) * q;
          if constexpr (KEEP) sg[k][e] = q;
        }
      }
    if (layer) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += v[k][e];
      team_sum<TEAM, 1>(s, red1);
      const float mean = s[0] * inv;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e)
          v[k][e] = (int64_t)(k * TEAM + lane) * V + e < Dg ? v[k][e] - mean : 0.f;
    }
    float s[3] = {0.f, 0.f, 0.f};  // v^2, d, d v
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = rg.at(k, e) * wv[k][e];
        s[0] = __builtin_fmaf(v[k][e], v[k][e], s[0]);
        s[1] += d;
        s[2] = __builtin_fmaf(d, v[k][e], s[2]);
      }
    team_sum<TEAM, 3>(s, red3);
    // a team without a row: 0, else eps = 0 makes it infinite and its 0 * xh
    // a NaN in the weights' gradients
    const float rstd = live ? __builtin_amdgcn_rsqf(__builtin_fmaf(s[0], inv, eps)) : 0.f;
    const float md = layer ? s[1] * inv : 0.f;
    const float mx = s[2] * inv * rstd;  // mean(d xh)
    float gx[NV][V], gz[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xh = v[k][e] * rstd, g = rg.at(k, e);
        dw[k][e] = __builtin_fmaf(g, xh, dw[k][e]);
        db[k][e] += g;
        const float dv = rstd * (__builtin_fmaf(g, wv[k][e], -md) - xh * mx);
        if constexpr (GATE) {
          const float zv = rz.at(k, e);
          float q;
          if constexpr (KEEP)
            q = sg[k][e];
          else
            q = sigmoid_f32(zv);
          gx[k][e] = dv * (zv * q);
          gz[k][e] = dv * rx.at(k, e) * (q * __builtin_fmaf(zv, 1.f - q, 1.f));
        } else {
          gx[k][e] = dv;
        }
      }
    if (live) {
      store<T, V, NV>(dx + r * D + g0, lane, TEAM, Dg, gx);
      if constexpr (GATE) store<T, V, NV>(dz + r * dzs + g0, lane, TEAM, Dg, gz);
    }
  }

  // this workgroup's row of gradient parts: [D] for w, then [D] for the bias
  float* row = part + (int64_t)(blockIdx.x / G) * D * (with_bias ? 2 : 1) + g0;
  for (int o = 0; o < (with_bias ? 2 : 1); ++o, row += D) {
    if constexpr (TEAMS > 1) {
      __syncthreads();
      if (team) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) cols[team - 1][k * V + e][lane] = o ? db[k][e] : dw[k][e];
      }
      __syncthreads();
    }
    if (team == 0) {
      float out[NV][V];
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float s = o ? db[k][e] : dw[k][e];
          if constexpr (TEAMS > 1) {
#pragma unroll
            for (int q = 0; q < TEAMS - 1; ++q) s += cols[q][k * V + e][lane];
          }
          out[k][e] = s;
        }
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int64_t c = (int64_t)(k * TEAM + lane) * V;
        if (c < Dg) {
          if constexpr (V == 1) {
            row[c] = out[k][0];
          } else {
#pragma unroll
            for (int e = 0; e < V; e += 4)
              *(f32x4*)(row + c + e) =
                  f32x4{out[k][e], out[k][e + 1], out[k][e + 2], out[k][e + 3]};
          }
        }
      }
    }
  }
}

struct Shape {
  int v, nv, team;
};

// Vectors per lane of a team of up to 256 lanes.
constexpr int most_vectors(int v, bool back) { return v == 1 || back ? 16 / v : 4; }

// The smallest team whose registers hold a group.  The forward holds up to 32
// values per lane (a wavefront for 2048 bfloat16 channels), the backward 16:
// with the weights, their two gradients and the rows of x, z and dy beside
// them, 32 spill.  A team of 1024 lanes has 128 registers per lane and takes
// 8 values.  One stride that is no multiple of 16 bytes makes every access one
// element (16384 x 2048 bf16, gated: 31 us, 86 with rows of 2049 for z;
// backward 57 and 263).
Shape shape_of(const NormDims& d, bool back) {
  const int v = d.bf16 ? vec_of<bf16>() : vec_of<float>();
  const int64_t dg = d.D / d.G;
  const bool vec = dg % v == 0 && d.D % v == 0 && d.xs % v == 0 && d.zs % v == 0 &&
                   (!back || d.dzs % v == 0);
  Shape s;
  s.v = vec ? v : 1;
  const int64_t n = (dg + s.v - 1) / s.v;  // vectors of a group
  const int most = most_vectors(s.v, back);
  if (n <= 32) {
    s.team = 32;
    s.nv = 1;
  } else if (n <= 64 * most) {
    s.team = 64;
    s.nv = n <= 64 ? 1 : n <= 64 * (most / 2) ? most / 2 : most;
  } else if (n <= 256 * most) {
    s.team = 256;
    s.nv = n <= 256 * (most / 2) ? most / 2 : most;
  } else {
    s.team = 1024;
    s.nv = 8 / s.v;
  }
  return s;
}

// Workgroups along the rows.  Forward: enough teams to fill the device
// several times over.  Backward: each workgroup leaves a row of parts that is
// read again, so about two resident sets of them, and four rows per team where
// that leaves a workgroup for each CU (1000 x 4096 bf16: 20 us, 38 with one).
int64_t row_blocks(const NormDims& d, int team, bool back) {
  const int64_t teams = block_of(team) / team;
  const int64_t most = (back ? 1024 : 4096) * 256 / block_of(team) / d.G;
  int64_t want = (d.R + teams - 1) / teams;
  if (back && want > 256) want = (want + 3) / 4 < 256 ? 256 : (want + 3) / 4;
  return want < most ? want : most < 1 ? 1 : most;
}

template <typename T, int V, int NV, int TEAM, typename F>
hipError_t call(F&& f) {
  return f((T*)nullptr, std::integral_constant<int, V>(), std::integral_constant<int, NV>(),
           std::integral_constant<int, TEAM>());
}

template <bool BACK, typename T, int V, typename F>
hipError_t by_shape(const Shape& s, F&& f) {
  constexpr int MOST = most_vectors(V, BACK);
  if (s.team == 32) return call<T, V, 1, 32>(f);
  if (s.team == 64)
    return s.nv == 1 ? call<T, V, 1, 64>(f)
                     : s.nv == MOST / 2 ? call<T, V, MOST / 2, 64>(f) : call<T, V, MOST, 64>(f);
  if (s.team == 256)
    return s.nv == MOST / 2 ? call<T, V, MOST / 2, 256>(f) : call<T, V, MOST, 256>(f);
  return call<T, V, 8 / V, 1024>(f);
}

template <bool BACK, typename F>
hipError_t dispatch(const NormDims& d, const Shape& s, F&& f) {
  if (d.bf16)
    return s.v == 1 ? by_shape<BACK, bf16, 1>(s, f) : by_shape<BACK, bf16, vec_of<bf16>()>(s, f);
  return s.v == 1 ? by_shape<BACK, float, 1>(s, f) : by_shape<BACK, float, vec_of<float>()>(s, f);
}

}  // namespace

hipError_t launch_norm(const NormDims& d, const void* x, const void* z, const float* w,
                       const float* bias, void* y, hipStream_t s) {
  const Shape sh = shape_of(d, false);
  return dispatch<false>(d, sh, [&](auto* tp, auto v, auto nv, auto tm) {
    typedef std::remove_pointer_t<decltype(tp)> T;
    constexpr int V = decltype(v)::value, NV = decltype(nv)::value, TEAM = decltype(tm)::value;
    const unsigned grid = (unsigned)(row_blocks(d, TEAM, false) * d.G);
    if (z)
      norm_fwd_kernel<T, V, NV, TEAM, true><<<grid, block_of(TEAM), 0, s>>>(
          (const T*)x, (const T*)z, w, bias, (T*)y, d.R, d.D, d.D / d.G, d.xs, d.zs, (unsigned)d.G,
          d.eps, d.layer);
    else
      norm_fwd_kernel<T, V, NV, TEAM, false><<<grid, block_of(TEAM), 0, s>>>(
          (const T*)x, nullptr, w, bias, (T*)y, d.R, d.D, d.D / d.G, d.xs, d.zs, (unsigned)d.G,
          d.eps, d.layer);
    return hipGetLastError();
  });
}

// The vector and the scalar form use other teams: the larger of the two.
size_t norm_part_bytes(const NormDims& d) {
  int64_t rows = 0;
  for (int team : {32, 64, 256, 1024}) {
    const int64_t n = row_blocks(d, team, true);
    rows = n > rows ? n : rows;
  }
  return (size_t)(rows * d.D * 2) * sizeof(float);
}

hipError_t launch_norm_backward(const NormDims& d, const void* x, const void* z, const float* w,
                                const void* dy, void* dx, void* dz, float* dw, float* dbias,
                                float* part, hipStream_t s) {
  const Shape sh = shape_of(d, true);
  const int64_t rows = row_blocks(d, sh.team, true);
  const hipError_t err = dispatch<true>(d, sh, [&](auto* tp, auto v, auto nv, auto tm) {
    typedef std::remove_pointer_t<decltype(tp)> T;
    constexpr int V = decltype(v)::value, NV = decltype(nv)::value, TEAM = decltype(tm)::value;
    const unsigned grid = (unsigned)(rows * d.G);
    if (z)
      norm_bwd_kernel<T, V, NV, TEAM, true><<<grid, block_of(TEAM), 0, s>>>(
          (const T*)x, (const T*)z, w, (const T*)dy, (T*)dx, (T*)dz, part, d.R, d.D, d.D / d.G,
          d.xs, d.zs, d.dzs, (unsigned)d.G, d.eps, d.layer, dbias != nullptr);
    else
      norm_bwd_kernel<T, V, NV, TEAM, false><<<grid, block_of(TEAM), 0, s>>>(
          (const T*)x, nullptr, w, (const T*)dy, (T*)dx, nullptr, part, d.R, d.D, d.D / d.G, d.xs,
          d.zs, d.dzs, (unsigned)d.G, d.eps, d.layer, dbias != nullptr);
    return hipGetLastError();
  });
  if (err != hipSuccess) return err;
  const int64_t m = d.D * (dbias ? 2 : 1);
  const int64_t ends[3] = {d.D, m, m};
  float* const outs[3] = {dw, dbias, nullptr};
  return launch_partial_sums(part, rows, m, ends, outs, s);
}

}  // namespace m2
