// rotary: queries and keys turned by their positions.  Pair i of a head's
// first R elements, with a = position * inv_freq[i]:
//
//     (x1, x2) -> scale * (x1 cos a - x2 sin a, x1 sin a + x2 cos a)
//
// where the pair is (x[i], x[i + R/2]) or (x[2i], x[2i+1]); the elements
// behind R are copied.  The backward is the transpose: the same with -a.
//
// Bound by HBM: each element is read and written once.  The angle is formed in
// float64 and reduced to a part of a turn there, so positions far out keep
// their digits (in float32 a position of 10^6 would leave 0.06 rad); sine and
// cosine are then float32 functions of that part.  A workgroup forms them once
// for its tokens in LDS; then neighbouring threads take neighbouring vectors of
// a token's heads, so that a wavefront reads and writes whole rows.
#include "launch.h"
#include "rowvec.h"

namespace m2 {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;    // of a workgroup
constexpr int kMaxTable = 1024;  // pairs of a workgroup's tokens
constexpr int64_t kMaxBlocks = 1 << 20;

struct RotaryArgs {
  const void *q, *k;
  void *yq, *yk;
  const float* inv_freq;
  const int32_t* positions;
  int64_t tokens, L, qs, ks, yqs, yks;
  int H, G, D, R;     // G = 0: no keys
  int units, up, per;  // units of a head, threads for them (a power of two), tokens of a workgroup
  float scale, sign;
};

// Unit u of a head: V pairs, or, behind the turned part, V elements.
// Tokens t0 .. t0 + count - 1; table: [token][cosines, then sines of the pairs].
template <typename T, int V, bool HALF>
__device__ __forceinline__ void turn_tokens(const RotaryArgs& a, float* table, int64_t t0,
                                            int count) {
  const int pairs = a.R / 2;
  for (int i = threadIdx.x; i < count * pairs; i += kThreads) {
    const int tok = i / pairs, p = i - tok * pairs;
    const int64_t t = t0 + tok;
    const int64_t pos = a.positions ? a.positions[t] : t % a.L;
    const double turns = (double)pos * (double)a.inv_freq[p] * 0.15915494309189533577;
    const float x = (float)(turns - __builtin_rint(turns));
    float sn, cs;
    sincospif(2.f * x, &sn, &cs);
    table[2 * tok * pairs + p] = a.scale * cs;
    table[(2 * tok + 1) * pairs + p] = a.sign * a.scale * sn;
  }
  __syncthreads();
  const int rot = pairs / V, heads = a.H + a.G, slots = kThreads / a.up;
  const float over = 1.f / (float)heads;
  for (int i = threadIdx.x / a.up; i < count * heads; i += slots) {
    // i < 2^15: the half keeps the quotient clear of whole numbers
    const int tok = (int)(((float)i + 0.5f) * over), h = i - tok * heads;
    const int64_t t = t0 + tok;
    const bool key = h >= a.H;
    const T* x = (const T*)(key ? a.k : a.q) + t * (key ? a.ks : a.qs) +
                 (int64_t)(key ? h - a.H : h) * a.D;
    T* y = (T*)(key ? a.yk : a.yq) + t * (key ? a.yks : a.yqs) +
           (int64_t)(key ? h - a.H : h) * a.D;
    const float* cs = table + 2 * tok * pairs;
    const float* sn = cs + pairs;
    for (int u = threadIdx.x % a.up; u < a.units; u += a.up) {
      if (u >= rot) {
        const int o = a.R + (u - rot) * V;
        *(raw_t<T, V>*)(y + o) = *(const raw_t<T, V>*)(x + o);
        continue;
      }
      // half: V pairs are two vectors of V; neighbours: a vector of 2 V
      // elements as two of V
      const int o1 = HALF ? u * V : 2 * u * V;
      const int o2 = HALF ? o1 + pairs : o1 + V;
      float x1[V], x2[V], y1[V], y2[V], c[V], s[V];
      load_row<T, V>(x + o1, x1);
      load_row<T, V>(x + o2, x2);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        c[e] = cs[u * V + e];
        s[e] = sn[u * V + e];
      }
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (HALF || V == 1) {
          y1[e] = x1[e] * c[e] - x2[e] * s[e];
          y2[e] = x1[e] * s[e] + x2[e] * c[e];
        } else {
          // element e of the 2 V belongs to pair e / 2
          const int j1 = e / 2, j2 = (V + e) / 2;
          y1[e] = e % 2 ? x1[e - 1] * s[j1] + x1[e] * c[j1] : x1[e] * c[j1] - x1[e + 1] * s[j1];
          y2[e] = e % 2 ? x2[e - 1] * s[j2] + x2[e] * c[j2] : x2[e] * c[j2] - x2[e + 1] * s[j2];
        }
      }
      store_row<T, V>(y + o1, y1);
      store_row<T, V>(y + o2, y2);
    }
  }
}

template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
  __shared__ __align__(16) float table[2 * kMaxTable];
  const int64_t step = (int64_t)gridDim.x * a.per;
  for (int64_t t0 = (int64_t)blockIdx.x * a.per; t0 < a.tokens; t0 += step) {
    turn_tokens<T, V, HALF>(a, table, t0, (int)(a.tokens - t0 < a.per ? a.tokens - t0 : a.per));
    __syncthreads();  // the table is free
  }
}

template <typename T, int V>
void go(const RotaryArgs& a, bool half, unsigned blocks, hipStream_t s) {
  if (half)
    rotary_kernel<T, V, true><<<blocks, kThreads, 0, s>>>(a);
  else
    rotary_kernel<T, V, false><<<blocks, kThreads, 0, s>>>(a);
}

template <typename T>
void run(RotaryArgs a, bool half, hipStream_t s) {
  constexpr int V = vec_of<T>();
  // vectors where every row, head, half and the end of the rotated part begin
  // at one (base pointers are at 16 bytes)
  const auto fits = [](int64_t v) { return v % V == 0; };
  const bool vec = fits(a.D) && fits(a.R / 2) && fits(a.qs) && fits(a.yqs) &&
                   (!a.G || (fits(a.ks) && fits(a.yks)));
  const int v = vec ? V : 1;
  a.units = a.R / 2 / v + (a.D - a.R) / v;
  a.up = 1;
  while (a.up < a.units && a.up < kThreads) a.up *= 2;
  // Tokens of a workgroup: one while that gives no four workgroups for each
  // CU, then as many as share a table.
  a.per = 1;
  while (2 * a.per <= kMaxTokens && 2 * a.per * (a.R / 2) <= kMaxTable &&
         a.tokens >= 1024 * 2 * a.per)
    a.per *= 2;
  const int64_t groups = (a.tokens + a.per - 1) / a.per;
  const unsigned blocks = (unsigned)(groups < kMaxBlocks ? groups : kMaxBlocks);
  if (vec)
    go<T, V>(a, half, blocks, s);
  else
    go<T, 1>(a, half, blocks, s);
}

}  // namespace

hipError_t launch_rotary(const RotaryDims& d, const void* q, const void* k, const float* inv_freq,
                         const int32_t* positions, void* yq, void* yk, bool back, hipStream_t s) {
  RotaryArgs a = {};
  a.q = q;
  a.k = k;
  a.yq = yq;
  a.yk = yk;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.tokens = d.B * d.L;
  a.L = d.L;
  a.qs = d.qs;
  a.ks = d.ks;
  a.yqs = d.yqs;
  a.yks = d.yks;
  a.H = (int)d.H;
  a.G = (int)d.G;
  a.D = (int)d.D;
  a.R = (int)d.R;
  a.scale = d.scale;
  a.sign = back ? -1.f : 1.f;
  if (d.bf16)
    run<bf16>(a, d.half, s);
  else
    run<float>(a, d.half, s);
  return hipGetLastError();
}

}  // namespace m2
