// What the forward and the backward pass of the selective scan share: how a
// workgroup divides channels and states, and the loads of a tile of tokens.
//
// A lane holds K of a channel's 4 K states, four lanes (a quad) a channel, a
// wavefront 16 channels, a workgroup 64 neighbouring channels of one group.
// Each lane of a quad loads every fourth token of its channel and hands the
// values to the other three through the quad permutation that an
// instruction's operand can carry; sums over a channel's states cross the
// quad the same way.  B and C are the same for all channels and come from LDS
// as float32.  So the recurrence runs down the tokens with no exchange between
// wavefronts.  The vector ALU bounds these kernels: what is the same for a
// wavefront stays off it (scalar row addresses with constant 32-bit lane
// offsets, 32-bit token counts), and tiles inside a sequence skip the masks.
#pragma once

#include "launch.h"
#include "rowvec.h"

namespace m2 {

constexpr int kQuadWaves = 4;

// States per lane for N states of a channel: 1, 2, 4, 8 or 16.
inline int scan_k(int64_t N) {
  int k = 1;
  while (4 * k < N) k *= 2;
  return k;
}

// Workgroups along the channels: tiles never straddle two groups.
inline int64_t scan_channel_tiles(const ScanDims& d) {
  return d.G * ((d.D / d.G + 63) / 64);
}

// The kernels that carry states over the chunks: wavefronts of a workgroup, and
// chunks whose loads a wavefront has in flight together.
constexpr int kCarryWaves = 16;
constexpr int kCarryLoads = 16;
inline unsigned carry_waves(int64_t chunks) {
  const int64_t w = (chunks + 7) / 8;
  return (unsigned)(w < kCarryWaves ? w : kCarryWaves);
}

struct ScanArgs {
  const void *u, *dt, *B, *C, *z;
  const float *A, *D, *dt_bias, *init;
  const int32_t* lengths;
  int64_t L, Dm, zs, bs, cs;  // tokens, channels and token strides
  int N, G, tiles;            // states, groups, channel tiles of a group
  int softplus;
  int64_t chunks, chunk;      // chunks of the sequence and tokens of each (a multiple of the tile)
};

inline ScanArgs scan_args(const ScanDims& d, const ScanSplit& p, const void* u, const void* dt,
                          const float* A, const void* B, const void* C, const float* D,
                          const void* z, const float* dt_bias, const float* init,
                          const int32_t* lengths) {
  ScanArgs a;
  a.u = u;
  a.dt = dt;
  a.B = B;
  a.C = C;
  a.z = z;
  a.A = A;
  a.D = D;
  a.dt_bias = dt_bias;
  a.init = init;
  a.lengths = lengths;
  a.L = d.L;
  a.Dm = d.D;
  a.zs = d.zs;
  a.bs = d.bs;
  a.cs = d.cs;
  a.N = (int)d.N;
  a.G = (int)d.G;
  a.tiles = (int)((d.D / d.G + 63) / 64);
  a.softplus = d.softplus;
  a.chunks = p.chunks;
  a.chunk = p.len;
  return a;
}

// Where this workgroup is (blockIdx.x = chunk * (G * tiles) + group * tiles +
// tile, blockIdx.y = batch) and this lane's channel.
struct ScanPlace {
  int64_t b, chunk, c;  // c: this lane's channel, c0 + at
  int64_t c0;           // the tile's first channel
  unsigned at;          // this lane's channel in the tile (0 where there is none)
  int g;
  bool live;            // the channel exists
  int64_t t0, t1, len;  // this chunk's tokens, and the sequence's length
};

__device__ __forceinline__ ScanPlace scan_place(const ScanArgs& a) {
  ScanPlace p;
  const unsigned per = (unsigned)(a.G * a.tiles);
  p.b = blockIdx.y;
  p.chunk = blockIdx.x / per;
  const unsigned r = blockIdx.x % per;
  p.g = (int)(r / (unsigned)a.tiles);
  const int64_t dg = a.Dm / a.G;
  const int64_t first = (int64_t)(r % (unsigned)a.tiles) * 64;
  const unsigned in = (unsigned)(wave_id() * 16 + (lane_id() >> 2));
  p.live = first + in < dg;
  p.c0 = (int64_t)p.g * dg + first;
  p.at = p.live ? in : 0u;
  p.c = p.c0 + p.at;
  p.t0 = p.chunk * a.chunk;
  p.t1 = p.t0 + a.chunk < a.L ? p.t0 + a.chunk : a.L;
  p.len = a.L;
  if (a.lengths) {
    const int64_t n = a.lengths[p.b];
    p.len = n < 0 ? 0 : n < a.L ? n : a.L;
  }
  return p;
}

// The value of lane J of this lane's quad.
template <int J>
__device__ __forceinline__ float of_lane(float v) { return dpp<J * 0x55>(v); }
__device__ __forceinline__ float quad_sum(float v) {
  v += dpp<0xB1>(v);  // lanes 1 0 3 2
  v += dpp<0x4E>(v);  // lanes 2 3 0 1
  return v;
}
// Lane j of the quad gets the sum over the quad of v[j]: nine operations for
// four sums.
__device__ __forceinline__ float quad_sums(const float (&v)[4], int j) {
  const bool hi2 = j & 2, hi1 = j & 1;
  const float a = (hi2 ? v[2] : v[0]) + dpp<0x4E>(hi2 ? v[0] : v[2]);
  const float b = (hi2 ? v[3] : v[1]) + dpp<0x4E>(hi2 ? v[1] : v[3]);
  return (hi1 ? b : a) + dpp<0xB1>(hi1 ? a : b);
}
// K states of one channel.  load / store: rows padded to 4 K states, 16-byte
// aligned; load_n / store_n: the caller's rows of N, zero past them.
template <int K>
struct States {
  float v[K];
  __device__ __forceinline__ void load(const float* p) {
    if constexpr (K >= 4) {
#pragma unroll
      for (int k = 0; k < K; k += 4) {
        const f32x4 q = *(const f32x4*)(p + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[k + e] = q[e];
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] = p[k];
    }
  }
  __device__ __forceinline__ void store(float* p) const {
    if constexpr (K >= 4) {
#pragma unroll
      for (int k = 0; k < K; k += 4) *(f32x4*)(p + k) = f32x4{v[k], v[k + 1], v[k + 2], v[k + 3]};
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) p[k] = v[k];
    }
  }
  __device__ __forceinline__ void load_n(const float* p, int n0, int N, float by = 1.f) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = n0 + k < N ? by * p[n0 + k] : 0.f;
  }
  __device__ __forceinline__ void store_n(float* p, int n0, int N) const {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (n0 + k < N) p[n0 + k] = v[k];
  }
};

// A lane's rows of a chunk: scalar addresses of the chunk's first token, this
// lane's offsets in bytes from the first token of a group of four, and the
// counts of tokens (those of the chunk; those that are no padding).
template <typename T>
struct Rows {
  const T *u, *dt, *dy, *z;
  unsigned off, zoff;
  int n, valid, j;
  bool whole;  // every lane of the workgroup has a channel
  __device__ __forceinline__ Rows(const ScanArgs& a, const ScanPlace& p, const T* dyp, int jj) {
    const int64_t row0 = p.b * a.L + p.t0;
    u = (const T*)a.u + row0 * a.Dm + p.c0;
    dt = (const T*)a.dt + row0 * a.Dm + p.c0;
    dy = dyp + row0 * a.Dm + p.c0;
    z = (const T*)a.z + row0 * a.zs + p.c0;  // not read where there is none
    j = jj;
    off = ((unsigned)j * (unsigned)a.Dm + p.at) * (unsigned)sizeof(T);
    zoff = ((unsigned)j * (unsigned)a.zs + p.at) * (unsigned)sizeof(T);
    n = (int)(p.t1 - p.t0);
    const int64_t left = p.len - p.t0;
    valid = left <= 0 ? 0 : left < n ? (int)left : n;
    whole = p.c0 + 64 <= (int64_t)(p.g + 1) * (a.Dm / a.G);
  }
};

// A token count that the compiler takes as new: addresses formed from it stay
// scalar.  Else it turns every row's address of a loop into a 64-bit pointer
// in vector registers, advanced by vector instructions.
__device__ __forceinline__ int fresh(int t) {
  asm("" : "+s"(t));
  return t;
}

// What a lane loads of its tokens of a tile (token 4 i + j of it).
template <typename T, int TT, bool GATE>
struct Tokens {
  static constexpr int OWN = TT / 4;
  T u[OWN], dt[OWN], dy[OWN], z[OWN];
  template <bool DY, bool Z>
  __device__ __forceinline__ void load(const ScanArgs& a, const ScanPlace& p, const Rows<T>& r,
                                       int t0) {
    const int t = fresh(t0);
    auto one = [&](int i) {
      const int64_t at = (int64_t)(t + 4 * i) * a.Dm;
      u[i] = lane_at(r.u + at, r.off);
      dt[i] = lane_at(r.dt + at, r.off);
      if constexpr (DY) dy[i] = lane_at(r.dy + at, r.off);
      if constexpr (Z && GATE) z[i] = lane_at(r.z + (int64_t)(t + 4 * i) * a.zs, r.zoff);
    };
    if (r.whole && t + TT <= r.valid) {
#pragma unroll
      for (int i = 0; i < OWN; ++i) one(i);
    } else {
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        u[i] = dt[i] = dy[i] = z[i] = (T)0.f;
        if (p.live && t + 4 * i + r.j < r.valid) one(i);
      }
    }
  }
  // the time steps, zero where there is no token
  __device__ __forceinline__ void steps(const ScanArgs& a, const Rows<T>& r, int t, float bias,
                                        float (&raw)[OWN], float (&d)[OWN]) const {
#pragma unroll
    for (int i = 0; i < OWN; ++i) d[i] = raw[i] = to_f32(dt[i]) + bias;
    if (a.softplus) {
#pragma unroll
      for (int i = 0; i < OWN; ++i) d[i] = softplus_f32(raw[i]);
    }
    if (t + TT > r.valid) {
#pragma unroll
      for (int i = 0; i < OWN; ++i) d[i] = t + 4 * i + r.j < r.valid ? d[i] : 0.f;
    }
  }
  // dy, times silu(z) with a gate
  __device__ __forceinline__ void grads(float (&q)[OWN]) const {
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
      q[i] = to_f32(dy[i]);
      if constexpr (GATE) {
        const float zv = to_f32(z[i]);
        q[i] *= zv * sigmoid_f32(zv);
      }
    }
  }
};

}  // namespace m2
