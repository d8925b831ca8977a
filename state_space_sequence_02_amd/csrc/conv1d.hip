// conv1d: the short causal depthwise convolution that makes x, B and C of an
// SSD call (and u of a selective scan), its backward pass and its one-token
// form.  Per channel c, with W taps and x before the first token taken from
// the first state (zeros without one):
//
//     p[t] = bias + sum_k w[k] x[t - (W-1) + k]        y[t] = silu(p[t]) or p[t]
//     g[t] = dy[t] act'(p[t])
//     dx[s] = sum_k w[k] g[s + (W-1) - k]              (+ dfinal at the last W-1 rows)
//     dw[k] = sum_t g[t] x[t - (W-1) + k]              dbias = sum_t g[t]
//
// About 2 W + 6 operations for every element read and written: the forward is
// bound by HBM, one token by the launch.  The backward's 6 W + 12 (the
// convolution again, silu's slope, W products each for dx and dw) keep the
// vector ALU 79 % busy (2 x 8192 x 1792 bf16: 43 us, 29 for its bytes).  A
// thread owns four channels and walks the tokens of a tile with the last W-1
// rows in registers, so each row is read once but for the W-1 rows before a
// tile; neighbouring lanes own neighbouring channels, so every access of a
// wavefront is 512 bytes (bfloat16) or 1 KB of one row or of two.  Eight
// bfloat16 channels per thread make 16-byte accesses and are slower (65536 x
// 2560: 147 us, 137 with four; backward 2 x 8192 x 1792: 51 and 48): their
// weights, rows and gradient sums leave two wavefronts per SIMD.  Where a row,
// part or stride is no multiple of four, a thread owns one channel (16384 x
// 2048 bf16: 30 us, 55 with rows of 2049; backward 44 and 77).
#include <type_traits>

#include "launch.h"
#include "rowvec.h"

namespace m2 {

namespace {

constexpr int kVec = 4;           // channels of a thread (1 where rows or parts are no multiple)
constexpr int kLoads = 8;         // rows in flight per thread
constexpr int kBwdWaves = 4;      // wavefronts (token tiles) per workgroup of the backward

struct Parts {
  void* p[3];
  int64_t n[3];
};

// The part that channel c falls into: its base pointer at c and its row length.
template <typename T>
__device__ __forceinline__ void part_of(const Parts& y, int64_t c, T** base, int64_t* width) {
  int64_t at = c;
  int i = 0;
  if (at >= y.n[0]) {
    at -= y.n[0];
    i = 1;
    if (at >= y.n[1]) {
      at -= y.n[1];
      i = 2;
    }
  }
  *base = (T*)y.p[i] + at;
  *width = y.n[i];
}

__device__ __forceinline__ int64_t length_of(const int32_t* lengths, int64_t b, int64_t L) {
  if (!lengths) return L;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > L ? L : n;
}

template <typename T, int V>
__device__ __forceinline__ void zero(float (&v)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = 0.f;
}

// Weights of V channels from w[C, W].
template <int V, int W>
__device__ __forceinline__ void load_weights(const float* __restrict__ w,
                                             const float* __restrict__ bias, int64_t c,
                                             float (&wk)[W][V], float (&bv)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int k = 0; k < W; ++k) wk[k][e] = w[(c + e) * W + k];
    bv[e] = bias ? bias[c + e] : 0.f;
  }
}

// Row `pos` of [first state; x] for this thread's channels.
template <typename T, int V, int W>
__device__ __forceinline__ raw_t<T, V> row_at(const T* xb, int64_t xs, const T* ib, int64_t C,
                                              int64_t pos) {
  if (pos >= 0) return *(const raw_t<T, V>*)(xb + pos * xs);
  if (ib) return *(const raw_t<T, V>*)(ib + (W - 1 + pos) * C);
  return raw_t<T, V>{};
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(256) conv1d_fwd_kernel(
    const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ bias,
    const T* init, const int32_t* __restrict__ lengths, Parts y, T* final_state, int64_t B,
    int64_t L, int64_t C, int64_t xs, int tile, int64_t ntiles, int silu) {
  const int64_t ncv = C / V;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= ncv * ntiles * B) return;
  const int64_t c = id % ncv * V;
  const int64_t bt = id / ncv;
  const int64_t t0 = bt % ntiles * tile;
  const int64_t b = bt / ntiles;
  const int64_t len = length_of(lengths, b, L);

  float wk[W][V], bv[V];
  load_weights<V, W>(w, bias, c, wk, bv);
  const T* xb = x + b * L * xs + c;
  const T* ib = init ? init + b * (W - 1) * C + c : nullptr;
  T* yb;
  int64_t ys;
  part_of(y, c, &yb, &ys);
  yb += b * L * ys;

  // first tile: the state after the last token, before anything is written
  // (the caller may pass the first state's own buffer for it)
  raw_t<T, V> fin[W - 1];
  if (t0 == 0 && final_state) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) fin[j] = row_at<T, V, W>(xb, xs, ib, C, len - (W - 1) + j);
  }

  float h[W - 1][V];  // h[j] = row t - (W-1) + j
  if (t0 < len) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const raw_t<T, V> q = row_at<T, V, W>(xb, xs, ib, C, t0 - (W - 1) + j);
#pragma unroll
      for (int e = 0; e < V; ++e) h[j][e] = elem<T, V>(q, e);
    }
  }
  const int64_t t1 = t0 + tile < L ? t0 + tile : L;
  for (int64_t t = t0; t < t1; t += kLoads) {
    raw_t<T, V> r[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      r[i] = raw_t<T, V>{};
      if (t + i < len && t + i < t1) r[i] = *(const raw_t<T, V>*)(xb + (t + i) * xs);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      float out[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float xv = elem<T, V>(r[i], e);
        float p = bv[e];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) p = __builtin_fmaf(wk[k][e], h[k][e], p);
        p = __builtin_fmaf(wk[W - 1][e], xv, p);
        if (silu) p *= sigmoid_f32(p);
        out[e] = t + i < len ? p : 0.f;
#pragma unroll
        for (int k = 0; k < W - 2; ++k) h[k][e] = h[k + 1][e];
        h[W - 2][e] = xv;
      }
      if (t + i < t1) store_row<T, V>(yb + (t + i) * ys, out);
    }
  }
  if (t0 == 0 && final_state) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      *(raw_t<T, V>*)(final_state + (b * (W - 1) + j) * C + c) = fin[j];
  }
}

// Backward: a wavefront walks a tile of tokens and the W-1 after them (whose g
// it recomputes for its last dx rows).  The workgroup's kBwdWaves tiles are
// summed in LDS into one row of weight-gradient parts [C * W | C]; the rows
// are summed by partial_sums.
template <typename T, int V, int W>
__global__ void __launch_bounds__(64 * kBwdWaves) conv1d_bwd_kernel(
    const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ bias,
    const T* __restrict__ init, const int32_t* __restrict__ lengths, Parts dy,
    const T* __restrict__ dfinal, T* __restrict__ dx, T* __restrict__ dinit,
    float* __restrict__ part, int64_t L, int64_t C, int64_t xs, int64_t dxs, unsigned ncb,
    int tile_len, int silu) {
  constexpr int NS = (W + 1) * V;
  __shared__ float red[kBwdWaves - 1][NS][64];
  const int lane = lane_id(), wave = wave_id();
  // channel blocks of a tile are neighbouring workgroups: together they read whole rows
  const unsigned tile = blockIdx.x / ncb;
  const int64_t c = ((int64_t)(blockIdx.x % ncb) * 64 + lane) * V;
  const int64_t b = blockIdx.y;
  const int64_t t0 = ((int64_t)tile * kBwdWaves + wave) * tile_len;
  const bool live = c < C;
  const int64_t len = length_of(lengths, b, L);

  float acc[W + 1][V];
#pragma unroll
  for (int k = 0; k <= W; ++k) zero<T, V>(acc[k]);

  if (live && t0 < L) {
    float wk[W][V], bv[V];
    load_weights<V, W>(w, bias, c, wk, bv);
    const T* xb = x + b * L * xs + c;
    const T* ib = init ? init + b * (W - 1) * C + c : nullptr;
    T* dyb;
    int64_t dys;
    part_of(dy, c, &dyb, &dys);
    dyb += b * L * dys;
    T* dxb = dx + b * L * dxs + c;
    float xw[W][V], gw[W][V];  // xw[k] = row t - (W-1) + k; gw[k] = g[t - k]
#pragma unroll
    for (int k = 0; k < W; ++k) {
      zero<T, V>(xw[k]);
      zero<T, V>(gw[k]);
    }
    if (t0 < len) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const raw_t<T, V> q = row_at<T, V, W>(xb, xs, ib, C, t0 - (W - 1) + j);
#pragma unroll
        for (int e = 0; e < V; ++e) xw[j + 1][e] = elem<T, V>(q, e);
      }
    }
    const int64_t own = t0 + tile_len < L ? t0 + tile_len : L;
    const int64_t end = own + W - 1;
    constexpr int U = 4;
    for (int64_t t = t0; t < end; t += U) {
      raw_t<T, V> rx[U], rg[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        rx[i] = raw_t<T, V>{};
        rg[i] = raw_t<T, V>{};
        if (t + i < len && t + i < end) {
          rx[i] = *(const raw_t<T, V>*)(xb + (t + i) * xs);
          rg[i] = *(const raw_t<T, V>*)((const T*)dyb + (t + i) * dys);
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const bool mine = t + i < own && t + i < len;  // g is 0 behind len, but x may be infinite
        float out[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
          for (int k = 0; k < W - 1; ++k) {
            xw[k][e] = xw[k + 1][e];
            gw[W - 1 - k][e] = gw[W - 2 - k][e];
          }
          xw[W - 1][e] = elem<T, V>(rx[i], e);
          float g = elem<T, V>(rg[i], e);
          if (silu) {
            float p = bv[e];
#pragma unroll
            for (int k = 0; k < W; ++k) p = __builtin_fmaf(wk[k][e], xw[k][e], p);
            const float sg = sigmoid_f32(p);
            g *= sg * __builtin_fmaf(p, 1.f - sg, 1.f);
          }
          if (t + i >= len) g = 0.f;
          gw[0][e] = g;
          if (mine) {
#pragma unroll
            for (int k = 0; k < W; ++k) acc[k][e] = __builtin_fmaf(g, xw[k][e], acc[k][e]);
            acc[W][e] += g;
          }
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < W; ++k) s = __builtin_fmaf(wk[k][e], gw[k][e], s);
          out[e] = s;
        }
        const int64_t s = t + i - (W - 1);
        // rows before the tile are the previous tile's, but before the first they are dinit's
        if (s < own && (s >= t0 || t0 == 0) && t + i < end) {
          if (s < len) {
            const int64_t j = s - (len - (W - 1));
            if (dfinal && j >= 0) {
              float f[V];
              load_row<T, V>(dfinal + (b * (W - 1) + j) * C + c, f);
#pragma unroll
              for (int e = 0; e < V; ++e) out[e] += f[e];
            }
          } else {
            zero<T, V>(out);
          }
          if (s >= 0)
            store_row<T, V>(dxb + s * dxs, out);
          else if (dinit)
            store_row<T, V>(dinit + (b * (W - 1) + (W - 1 + s)) * C + c, out);
        }
      }
    }
  }

  if (wave) {
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) red[wave - 1][k * V + e][lane] = acc[k][e];
  }
  __syncthreads();
  if (wave || !live) return;
  float* row = part + ((int64_t)b * (gridDim.x / ncb) + tile) * C * (W + 1);
  auto sum = [&](int k, int e) {
    float s = acc[k][e];
#pragma unroll
    for (int o = 0; o < kBwdWaves - 1; ++o) s += red[o][k * V + e][lane];
    return s;
  };
#pragma unroll
  for (int e = 0; e < V; ++e)
#pragma unroll
    for (int k = 0; k < W; ++k) row[(c + e) * W + k] = sum(k, e);
#pragma unroll
  for (int e = 0; e < V; ++e) row[C * W + c + e] = sum(W, e);
}

template <typename T, int V, int W>
__global__ void __launch_bounds__(256) conv1d_step_kernel(
    const T* __restrict__ x, const float* __restrict__ w, const float* __restrict__ bias, T* state,
    Parts y, int64_t B, int64_t C, int64_t xs, int silu) {
  const int64_t ncv = C / V;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= ncv * B) return;
  const int64_t c = id % ncv * V;
  const int64_t b = id / ncv;
  T* sb = state + b * (W - 1) * C + c;
  raw_t<T, V> r[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) r[j] = *(const raw_t<T, V>*)(sb + j * C);
  r[W - 1] = *(const raw_t<T, V>*)(x + b * xs + c);
  float wk[W][V], bv[V], out[V];
  load_weights<V, W>(w, bias, c, wk, bv);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    float p = bv[e];
#pragma unroll
    for (int k = 0; k < W; ++k) p = __builtin_fmaf(wk[k][e], elem<T, V>(r[k], e), p);
    out[e] = silu ? p * sigmoid_f32(p) : p;
  }
  T* yb;
  int64_t ys;
  part_of(y, c, &yb, &ys);
  store_row<T, V>(yb + b * ys, out);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) *(raw_t<T, V>*)(sb + j * C) = r[j + 1];
}

bool vectors(const ConvDims& d, bool back) {
  return d.C % kVec == 0 && d.part[0] % kVec == 0 && d.part[1] % kVec == 0 &&
         d.part[2] % kVec == 0 && d.xs % kVec == 0 && (!back || d.dxs % kVec == 0);
}

Parts parts_of(const ConvDims& d, void* const* p) {
  Parts y;
  for (int i = 0; i < 3; ++i) {
    y.p[i] = p[i];
    y.n[i] = d.part[i];
  }
  return y;
}

// Calls f with the element type, the vector length and the width as types.
template <typename T, int V, typename F>
hipError_t by_width(const ConvDims& d, F&& f) {
  switch (d.W) {
    case 2: return f((T*)nullptr, std::integral_constant<int, V>(), std::integral_constant<int, 2>());
    case 3: return f((T*)nullptr, std::integral_constant<int, V>(), std::integral_constant<int, 3>());
    default: return f((T*)nullptr, std::integral_constant<int, V>(), std::integral_constant<int, 4>());
  }
}

template <typename F>
hipError_t dispatch(const ConvDims& d, bool back, F&& f) {
  const bool vec = vectors(d, back);
  if (d.bf16) return vec ? by_width<bf16, kVec>(d, f) : by_width<bf16, 1>(d, f);
  return vec ? by_width<float, kVec>(d, f) : by_width<float, 1>(d, f);
}

// Tokens of a backward tile: 32, or 16 or 8 where that leaves less than two
// wavefronts for each SIMD (2 x 2048 x 2560 bf16: 32 tokens 30 us, 16 tokens
// 25; 1 x 38 x 2560: 8 tokens 11 us, 32 tokens 30).  By the sizes alone, so
// that the workspace is known before the pointers.
int bwd_tile(const ConvDims& d) {
  const int64_t lanes = d.C / (vectors(d, true) ? kVec : 1);
  const int64_t per = (lanes + 63) / 64 * d.B;
  for (int n = 32; n > 8; n /= 2)
    if (per * ((d.L + n - 1) / n) >= 2048) return n;
  return 8;
}

int64_t bwd_tiles(const ConvDims& d) {
  const int n = bwd_tile(d) * kBwdWaves;
  return (d.L + n - 1) / n;
}

}  // namespace

size_t conv1d_part_bytes(const ConvDims& d) {
  return (size_t)(d.B * bwd_tiles(d) * d.C * (d.W + 1)) * sizeof(float);
}

hipError_t launch_conv1d(const ConvDims& d, const void* x, const float* w, const float* bias,
                         const void* init, const int32_t* lengths, void* const* y,
                         void* final_state, hipStream_t s) {
  return dispatch(d, false, [&](auto* tp, auto v, auto wd) {
    typedef std::remove_pointer_t<decltype(tp)> T;
    constexpr int V = decltype(v)::value, W = decltype(wd)::value;
    // long tiles read fewer rows and weights again, short ones fill the device
    // (65536 x 2560 bf16: 137 us with 32 rows, 141 with 64, 157 with 128)
    const int64_t per = d.C / V * d.B;
    const int tile = per * ((d.L + 31) / 32) >= (1 << 17) ? 32 : 8;
    const int64_t ntiles = (d.L + tile - 1) / tile;
    const unsigned grid = (unsigned)((per * ntiles + 255) / 256);
    conv1d_fwd_kernel<T, V, W><<<grid, 256, 0, s>>>((const T*)x, w, bias, (const T*)init, lengths,
                                                    parts_of(d, y), (T*)final_state, d.B, d.L, d.C,
                                                    d.xs, tile, ntiles, d.silu);
    return hipGetLastError();
  });
}

hipError_t launch_conv1d_backward(const ConvDims& d, const void* x, const float* w,
                                  const float* bias, const void* init, const int32_t* lengths,
                                  void* const* dy, const void* dfinal, void* dx, void* dinit,
                                  float* dw, float* dbias, float* part, hipStream_t s) {
  hipError_t e = dispatch(d, true, [&](auto* tp, auto v, auto wd) {
    typedef std::remove_pointer_t<decltype(tp)> T;
    constexpr int V = decltype(v)::value, W = decltype(wd)::value;
    const unsigned ncb = (unsigned)((d.C / V + 63) / 64);
    const dim3 grid((unsigned)(ncb * bwd_tiles(d)), (unsigned)d.B);
    conv1d_bwd_kernel<T, V, W><<<grid, 64 * kBwdWaves, 0, s>>>(
        (const T*)x, w, bias, (const T*)init, lengths, parts_of(d, dy), (const T*)dfinal, (T*)dx,
        (T*)dinit, part, d.L, d.C, d.xs, d.dxs, ncb, bwd_tile(d), d.silu);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  const int64_t ends[3] = {d.C * d.W, d.C * (d.W + 1), d.C * (d.W + 1)};
  float* const outs[3] = {dw, dbias, nullptr};
  return launch_partial_sums(part, d.B * bwd_tiles(d), d.C * (d.W + 1), ends, outs, s);
}

hipError_t launch_conv1d_step(const ConvDims& d, const void* x, const float* w, const float* bias,
                              void* state, void* const* y, hipStream_t s) {
  return dispatch(d, false, [&](auto* tp, auto v, auto wd) {
    typedef std::remove_pointer_t<decltype(tp)> T;
    constexpr int V = decltype(v)::value, W = decltype(wd)::value;
    const unsigned grid = (unsigned)((d.C / V * d.B + 255) / 256);
    conv1d_step_kernel<T, V, W><<<grid, 256, 0, s>>>((const T*)x, w, bias, (T*)state,
                                                     parts_of(d, y), d.B, d.C, d.xs, d.silu);
    return hipGetLastError();
  });
}

}  // namespace m2
