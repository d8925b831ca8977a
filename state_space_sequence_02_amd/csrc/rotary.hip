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
// cosine are then float32 functions of that part.  A thread takes one unit (a
// vector of pairs, or a vector behind R) of every S-th head of a token, so a
// sine serves (H + G) / S heads.
#include "launch.h"
#include "rowvec.h"

namespace m2 {

namespace {

constexpr int kThreads = 256;

struct RotaryArgs {
  const void *q, *k;
  void *yq, *yk;
  const float* inv_freq;
  const int32_t* positions;
  int64_t tokens, L, qs, ks, yqs, yks;
  int H, G, D, R;    // G = 0: no keys
  int units, up, S;  // units of a head, threads for them (a power of two), threads for its heads
  float scale, sign;
};

template <typename T, int V, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(RotaryArgs a) {
  const int team = threadIdx.x / a.up, slot = team % a.S;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / a.up / a.S) + team / a.S;
  if (t >= a.tokens) return;
  const int pairs = a.R / 2;
  // half: V pairs are two vectors of V; neighbours: a vector of 2 V elements
  // as two of V.  Either way a thread holds two vectors of a rotated unit.
  const int rot = (pairs + V - 1) / V;
  const int64_t pos = a.positions ? a.positions[t] : t % a.L;
  for (int u = threadIdx.x % a.up; u < a.units; u += a.up) {
    const bool turn = u < rot;
    float c[V], s[V];
    int o1, o2;
    if (turn) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const double turns = (double)pos * (double)a.inv_freq[u * V + e] * 0.15915494309189533577;
        const float x = (float)(turns - __builtin_rint(turns));
        float sn, cs;
        sincospif(2.f * x, &sn, &cs);
        c[e] = a.scale * cs;
        s[e] = a.sign * a.scale * sn;
      }
      o1 = HALF ? u * V : 2 * u * V;
      o2 = HALF ? o1 + pairs : o1 + V;
    } else {
      o1 = o2 = a.R + (u - rot) * V;
    }
    for (int h = slot; h < a.H + a.G; h += a.S) {
      const bool key = h >= a.H;
      const T* x = (const T*)(key ? a.k : a.q) + t * (key ? a.ks : a.qs) +
                   (int64_t)(key ? h - a.H : h) * a.D;
      T* y = (T*)(key ? a.yk : a.yq) + t * (key ? a.yks : a.yqs) +
             (int64_t)(key ? h - a.H : h) * a.D;
      if (!turn) {
        *(raw_t<T, V>*)(y + o1) = *(const raw_t<T, V>*)(x + o1);
        continue;
      }
      float x1[V], x2[V], y1[V], y2[V];
      load_row<T, V>(x + o1, x1);
      load_row<T, V>(x + o2, x2);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (HALF || V == 1) {
          y1[e] = x1[e] * c[e] - x2[e] * s[e];
          y2[e] = x1[e] * s[e] + x2[e] * c[e];
        } else {
          // element j of the 2 V: pair j / 2
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
  const bool vec = fits(a.D) && fits(a.R) && fits(a.R / 2) && fits(a.qs) && fits(a.yqs) &&
                   (!a.G || (fits(a.ks) && fits(a.yks)));
  const int v = vec ? V : 1;
  a.units = a.R / 2 / v + (a.D - a.R) / v;
  a.up = 1;
  while (a.up < a.units && a.up < kThreads) a.up *= 2;
  // Threads per token for its heads: one (a sine serves all heads) once the
  // tokens alone fill the device, more while they do not.
  const int slots = kThreads / a.up;
  a.S = 1;
  while (2 * a.S <= slots && a.S < a.H + a.G && a.tokens * a.up * a.S < 256 * 2048) a.S *= 2;
  const int64_t per = slots / a.S;
  const unsigned blocks = (unsigned)((a.tokens + per - 1) / per);
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
