// What the forward and the backward pass of the selective scan share: how a
// workgroup divides channels and states, its tile of tokens, and the loads
// that turn a tile of the inputs into float32 values in LDS.
//
// A workgroup takes 64 neighbouring channels of one group (lane = channel)
// and every state of them: wavefront w of WV holds states 4 w .. 4 w + 3 of
// its lane's channel in registers.  B and C are then the same for all lanes
// and come from LDS as broadcast reads of 16 bytes; the recurrence runs down
// the tokens with no exchange between lanes, and only the sum over a
// channel's states crosses wavefronts, through LDS, once per token.
#pragma once

#include "launch.h"
#include "rowvec.h"

namespace m2 {

constexpr int kScanK = 4;           // states of one channel in one lane
constexpr int kScanMaxState = 64;   // 16 wavefronts

// Wavefronts of a workgroup for N states: 1, 2, 4, 8 or 16.
inline int scan_waves(int64_t N) {
  int w = 1;
  while (w * kScanK < N) w *= 2;
  return w;
}

// Tokens of a tile: what 64 KB of LDS hold twice over.
constexpr int scan_tile(int wv) { return wv <= 4 ? 16 : wv == 8 ? 8 : 4; }

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

// Where this workgroup is: blockIdx.x = chunk * (G * tiles) + group * tiles +
// tile, blockIdx.y = batch.
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
  p.live = first + lane_id() < dg;
  p.c0 = (int64_t)p.g * dg + first;
  p.at = p.live ? (unsigned)lane_id() : 0u;
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

// A state array of the caller's, [.., N] float32: four states of one channel,
// zero past N.
__device__ __forceinline__ f32x4 load_states(const float* p, int n0, int N) {
  f32x4 v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = n0 + k < N ? p[n0 + k] : 0.f;
  return v;
}
__device__ __forceinline__ void store_states(float* p, int n0, int N, const f32x4& v) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (n0 + k < N) p[n0 + k] = v[k];
}

// A[c, n] log2(e) of this lane's four states (0 past N: such a state stays
// what it is, zero).
__device__ __forceinline__ f32x4 load_A2(const ScanArgs& a, int64_t c, int n0) {
  return load_states(a.A + c * a.N, n0, a.N) * kLog2e;
}

}  // namespace m2
