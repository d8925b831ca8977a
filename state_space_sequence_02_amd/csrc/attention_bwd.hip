// Backward pass of attention.  With P_ij = exp(s_ij - lse_i) and the gradient
// dO of the output,
//
//     delta_i = sum_d dO_id O_id
//     dV_j = sum_i P_ij dO_i            dP_ij = dO_i . V_j
//     dS_ij = P_ij (dP_ij - delta_i)
//     dQ_i = scale sum_j dS_ij K_j      dK_j = scale sum_i dS_ij Q_i
//
// The weights are formed again from q, k and lse.  One kernel owns rows and
// walks the keys (dQ, 3 products), one owns keys and walks the rows (dK and
// dV, 4 products): seven products instead of five, but every gradient is a sum
// in one place and in a fixed order, without atomics and without float32
// partial dQ in memory.  dK and dV of a group are sums over the packed rows of
// all its heads.  P and dS are rounded to the inputs' type before the products
// that take them (bfloat16: 2^-8 at most for each term of a sum).
#include "attention_fwd.h"

namespace m2 {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 128;     // packed rows of a workgroup of the dQ kernel
constexpr int kKeys = 64;       // keys of a tile in the dQ kernel
constexpr int kTileKeys = 128;  // keys of a workgroup of the dK and dV kernel

struct BwdArgs {
  const void *q, *k, *v, *o, *dout;
  const float* lse;
  void *dq, *dk, *dv;
  float *lse2, *delta;  // [rows of q][H]; lse in log2 units, 0 for rows without keys
  Side qside, kside;
  int64_t qs, ks, vs, dqs, dks, dvs, slots;
  int64_t q_rows, k_rows;
  float* part;  // where a walk is split: [gridDim.y][rows][heads][D], of dK and then of dV
  int H, G, rep, D;
  unsigned div_m;
  int div_l;
  bool causal;
  float c, scale;
};

// r / rep for 0 <= r < 2^31: M = ceil(2^(31 + l) / rep), l = ceil(log2 rep).
__device__ __forceinline__ int over_rep(const BwdArgs& a, int r) {
  return (int)(__umulhi(2u * (unsigned)r, a.div_m) >> a.div_l);
}

// Starts the loads of packed rows r0 .. r0 + ROWS - 1 of a group; rows behind
// the last are the last again.
template <typename T, int DP, int ROWS, int NT>
__device__ __forceinline__ void stage_packed(uint32_t lds, const T* base, int64_t stride, int rows,
                                             int r0, const BwdArgs& a, int thread) {
  using K = TileCfg<T, DP>;
#pragma unroll
  for (int i = 0; i < ROWS * K::CH / NT; ++i) {
    const int slot = i * NT + thread;
    const int r = slot / K::CH, c = (slot % K::CH) ^ swz<K::CH>(r);
    const int at = r0 + r < rows ? r0 + r : rows - 1;
    const int tok = over_rep(a, at);
    const T* p = base + tok * stride + (at - tok * a.rep) * a.D;
    if (c * K::E < a.D) dma16(p + c * K::E, lds + (slot & ~63) * 16);
  }
}

// 4 bytes a lane, as dma16.
__device__ __forceinline__ void dma4(const void* src, uint32_t lds_base) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_base);
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" : : "v"(src), "{m0}"(m0) : "memory");
}

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) attention_dq_kernel(BwdArgs a) {
  using K = TileCfg<T, DP>;
  constexpr int TILE = kKeys * K::ROWB;
  extern __shared__ __align__(16) char lds[];
  const int lane = lane_id(), wave = wave_id(), hh = lane >> 5;
  const int g = blockIdx.x % a.G;
  const Tile tile = tile_of<false>(a.qside, a.rep, kRows, (int)a.slots, blockIdx.x / a.G);
  const int span = tile.seq.span * a.rep;
  if (tile.r0 >= span) return;
  const int nq = tile.seq.n, rows = nq * a.rep;
  Seq ks = {0, 0, 0};
  if (tile.b >= 0) ks = seq_of(a.kside, tile.b);
  const int nk = ks.n;
  const int row = tile.r0 + wave * 32 + (lane & 31);
  const int token = row / a.rep;
  const int head = g * a.rep + row % a.rep;
  const auto seen = [&](int tok) {
    const int64_t n = (int64_t)tok + nk - nq + 1;
    return a.causal ? (int)clamp64(n, nk) : nk;
  };
  const int lim = row < rows ? seen(token) : 0;
  const int last = min(tile.r0 + kRows, rows) - 1;
  const int most = last >= tile.r0 ? seen(last / a.rep) : 0;
  const int all = (most + kKeys - 1) / kKeys;
  const int per = (all + gridDim.y - 1) / gridDim.y;
  const int t0 = blockIdx.y * per, tiles = t0 + per < all ? t0 + per : all;

  f32x16 acc[DP / 32];
#pragma unroll
  for (int d = 0; d < DP / 32; ++d) acc[d] = zero16();
  if (tile.r0 < rows) {
    head_frag<T> q[K::STEPS], dout[K::STEPS];
    const int safe = row < rows ? row : rows - 1;
    const int64_t tok = tile.seq.row0 + safe / a.rep;
    const int hd = g * a.rep + safe % a.rep;
    const int64_t at = tok * a.H + hd;
    load_row_frags<T, DP>((const T*)a.q + tok * a.qs + (int64_t)hd * a.D, a.D, q);
    load_row_frags<T, DP>((const T*)a.dout + at * a.D, a.D, dout);
    // delta and lse of a row, also for the other kernel
    head_frag<T> o[K::STEPS];
    load_row_frags<T, DP>((const T*)a.o + at * a.D, a.D, o);
    float delta = 0.f;
#pragma unroll
    for (int s = 0; s < K::STEPS; ++s)
#pragma unroll
      for (int e = 0; e < K::E; ++e)
        delta = __builtin_fmaf(to_f32(o[s][e]), to_f32(dout[s][e]), delta);
    delta = add_xor32(delta);
    float lse2 = a.lse[at];
    lse2 = lse2 == -__builtin_inff() ? 0.f : lse2 * kLog2e;
    if (row < rows && hh == 0 && blockIdx.y == 0) {
      a.lse2[at] = lse2;
      a.delta[at] = delta;
    }
    const T* k = (const T*)a.k + (int64_t)ks.row0 * a.ks + (int64_t)g * a.D;
    const T* v = (const T*)a.v + (int64_t)ks.row0 * a.vs + (int64_t)g * a.D;
    const uint32_t base = lds_addr(lds);
    clear_ends<T, DP>(lds, 4 * kKeys, a.D, threadIdx.x, kThreads);
    int low = lim, high = lim;
#pragma unroll
    for (int m = 1; m < 32; m *= 2) {
      low = min(low, __shfl_xor(low, m));
      high = max(high, __shfl_xor(high, m));
    }
    low = __builtin_amdgcn_readfirstlane(low);
    high = __builtin_amdgcn_readfirstlane(high);
    using St = Stager<T, DP, kKeys, kThreads>;
    const St ks_(a.ks, threadIdx.x), vs_(a.vs, threadIdx.x);
    const auto stage = [&](int t) {
      const uint32_t to = base + (t & 1) * 2 * TILE;
      const int r0 = t * kKeys;
      if (r0 + kKeys <= nk) {
        ks_.load(to, k + r0 * a.ks, a.D, threadIdx.x);
        vs_.load(to + TILE, v + r0 * a.vs, a.D, threadIdx.x);
      } else {
        St::load_tail(to, k, a.ks, r0, nk, nullptr, a.D, threadIdx.x);
        St::load_tail(to + TILE, v, a.vs, r0, nk, nullptr, a.D, threadIdx.x);
      }
    };
    const TileReader<T, DP> rd(base);
    if (t0 < tiles) stage(t0);
    for (int t = t0; t < tiles; ++t) {
      wait_vm(0);
      lds_barrier();
      if (t + 1 < tiles) stage(t + 1);
      const TileReader<T, DP> kr = rd.later((t & 1) * 2 * TILE), vr = kr.later(TILE);
      const int k0 = t * kKeys;
#pragma unroll
      for (int u = 0; u < kKeys / 32; ++u) {
        const int ku = k0 + 32 * u;
        if (high <= ku) break;
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int d = 0; d < K::STEPS; ++d) s = mma_head(kr.head(0, 32 * u, d), q[d], s);
#pragma unroll
        for (int d = 0; d < K::STEPS; ++d) dp = mma_head(vr.head(0, 32 * u, d), dout[d], dp);
        if (low < ku + 32) {
          const int left = lim - ku - 4 * hh;
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (8 * (r / 4) + r % 4 >= left) s[r] = -__builtin_inff();
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] = fast_exp2(__builtin_fmaf(s[r], a.c, -lse2));
        if (ku == 0) {
          // All keys of rows that see no more than these: their delta without
          // o's rounding, which is what such rows' gradients feel (its share
          // falls with the number of keys).  The weights are good to lse's
          // rounding, |lse| 2^-24 times a few, one factor for a row: over
          // their own sum it leaves dP - delta, and only scales dS.
          float sum = 0.f, total = 0.f;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            sum = __builtin_fmaf(s[r], dp[r], sum);
            total += s[r];
          }
          sum = add_xor32(sum);
          total = add_xor32(total);
          sum = total == 0.f ? 0.f : sum / total;  // no key: no weights
          if (lim <= 32) delta = sum;
          if (lim <= 32 && row < rows && hh == 0) a.delta[at] = sum;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) s[r] *= dp[r] - delta;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const row_frag<T> ds = acc_frag<T>(s, h);
#pragma unroll
          for (int d = 0; d < DP / 32; ++d)
            acc[d] = mma_rows(kr.cols(0, 32 * u + 16 * h, d), ds, acc[d]);
        }
      }
    }
  }
  if (row >= span) return;
  if (a.part) {
    const int64_t to = (blockIdx.y * a.q_rows + tile.seq.row0 + token) * a.H + head;
    store_column<float, DP>(a.part + to * a.D, acc, a.scale, a.D);
    return;
  }
  store_column<T, DP>((T*)a.dq + (int64_t)(tile.seq.row0 + token) * a.dqs + (int64_t)head * a.D, acc,
                      a.scale, a.D);
}

// The dK and dV kernel: 4 wavefronts along the keys, 32 each, and in bfloat16
// two such sets that share the rows of a tile and add their sums at the end:
// one workgroup fills a CU and the longest walk (the first keys of a causal
// sequence) takes half as long.  With one set, and two workgroups on a CU, the
// training step of 2 x 4096 tokens, 32 heads of 128, took 1691 us (1240 with
// two sets), packed 8192 x 24 x 64 385 us (297); tiles of 64 keys with four
// sets 1347 and 305.
template <typename T, int DP>
struct DkvCfg {
  static constexpr int SETS = sizeof(T) == 2 ? 2 : 1;
  static constexpr int THREADS = 256 * SETS;
  static constexpr int SUBS = sizeof(T) == 2 ? 2 / SETS : 1;  // 32 packed rows each, of a set
  static constexpr int ROWS = 32 * SETS * SUBS;               // packed rows of a tile
  static constexpr int TILE = ROWS * TileCfg<T, DP>::ROWB;
  static constexpr int BUF = 2 * TILE + 512;  // Q, dO, lse2 and delta
  static constexpr int JOIN = (SETS - 1) * 4 * 32 * DP * 4;
  static constexpr int LDS = 2 * BUF > JOIN ? 2 * BUF : JOIN;
};

template <typename T, int DP>
__global__ void __launch_bounds__((DkvCfg<T, DP>::THREADS), (sizeof(T) == 2 ? 2 : 1))
    attention_dkv_kernel(BwdArgs a) {
  using K = TileCfg<T, DP>;
  using C = DkvCfg<T, DP>;
  extern __shared__ __align__(16) char lds[];
  const int lane = lane_id(), wave = wave_id() & 3, set = wave_id() >> 2, hh = lane >> 5;
  const int g = blockIdx.x % a.G;
  const Tile tile = tile_of<true>(a.kside, 1, kTileKeys, (int)a.slots, blockIdx.x / a.G);
  if (tile.r0 >= tile.seq.span) return;
  const int nk = tile.seq.n;
  Seq qs = {0, 0, 0};
  if (tile.b >= 0) qs = seq_of(a.qside, tile.b);
  const int nq = qs.n, rows = nq * a.rep;
  const int k0 = tile.r0, key = k0 + wave * 32 + (lane & 31);
  // the first packed row that sees a key; all see the keys before the first token
  const auto first_of = [&](int kk) {
    const int64_t tok = (int64_t)kk - ((int64_t)nk - nq);
    return !a.causal || tok < 0 ? 0 : (int)(tok < nq ? tok * a.rep : rows);
  };
  const int first = first_of(key < nk ? key : nk - 1);
  const int wave_last = k0 + wave * 32 + 31;
  const int low = first_of(k0 + wave * 32);                        // the wavefront's earliest row
  const int high = first_of(wave_last < nk ? wave_last : nk - 1);  // all its keys are seen from here
  const int begin0 = k0 < nk ? first_of(k0) / C::ROWS : 0;
  const int all = k0 < nk ? (rows + C::ROWS - 1) / C::ROWS : 0;
  const int per = (all - begin0 + gridDim.y - 1) / gridDim.y;
  const int begin = begin0 + blockIdx.y * per, tiles = begin + per < all ? begin + per : all;

  f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int d = 0; d < DP / 32; ++d) dk[d] = dv[d] = zero16();
  if (begin < tiles) {
    head_frag<T> kf[K::STEPS], vf[K::STEPS];
    const int64_t at = tile.seq.row0 + (key < nk ? key : nk - 1);
    load_row_frags<T, DP>((const T*)a.k + at * a.ks + (int64_t)g * a.D, a.D, kf);
    load_row_frags<T, DP>((const T*)a.v + at * a.vs + (int64_t)g * a.D, a.D, vf);
    const T* q = (const T*)a.q + (int64_t)qs.row0 * a.qs + (int64_t)g * a.rep * a.D;
    const T* dout = (const T*)a.dout + ((int64_t)qs.row0 * a.H + g * a.rep) * a.D;
    const float* lse2 = a.lse2 + (int64_t)qs.row0 * a.H + g * a.rep;
    const float* delta = a.delta + (int64_t)qs.row0 * a.H + g * a.rep;
    const uint32_t base = lds_addr(lds);
    clear_ends<T, DP>(lds, 2 * C::ROWS, a.D, threadIdx.x, C::THREADS);
    clear_ends<T, DP>(lds + C::BUF, 2 * C::ROWS, a.D, threadIdx.x, C::THREADS);
    const auto stage = [&](int t) {
      const uint32_t to = base + (t & 1) * C::BUF;
      const int r0 = t * C::ROWS;
      stage_packed<T, DP, C::ROWS, C::THREADS>(to, q, a.qs, rows, r0, a, threadIdx.x);
      stage_packed<T, DP, C::ROWS, C::THREADS>(to + C::TILE, dout, (int64_t)a.H * a.D, rows, r0, a,
                                               threadIdx.x);
      // wavefront 0: lse2, wavefront 1: delta of the tile's rows, 64 at a time
      const int w = wave_id();
#pragma unroll
      for (int i = 0; i < (C::ROWS + 63) / 64; ++i) {
        if (w < 2 && lane < C::ROWS) {
          const int r = r0 + 64 * i + lane < rows ? r0 + 64 * i + lane : rows - 1;
          const int tok = over_rep(a, r);
          const float* p = (w ? delta : lse2) + (int64_t)tok * a.H + (r - tok * a.rep);
          dma4(p, to + 2 * C::TILE + w * C::ROWS * 4 + i * 256);
        }
      }
    };
    const TileReader<T, DP> rd(base);
    stage(begin);
    for (int t = begin; t < tiles; ++t) {
      wait_vm(0);
      lds_barrier();
      if (t + 1 < tiles) stage(t + 1);
      const int mine = set * 32 * C::SUBS;  // this set's rows of the tile
      const TileReader<T, DP> qr = rd.later((t & 1) * C::BUF + mine * K::ROWB),
                              dr = qr.later(C::TILE);
      const float* st = (const float*)(lds + (t & 1) * C::BUF + 2 * C::TILE) + mine;
      const int r0 = t * C::ROWS + mine;
#pragma unroll
      for (int u = 0; u < C::SUBS; ++u) {
        const int ru = r0 + 32 * u;
        if (ru >= rows || low >= ru + 32) continue;
        f32x16 s = zero16(), dp = zero16();
#pragma unroll
        for (int d = 0; d < K::STEPS; ++d) s = mma_head(qr.head(0, 32 * u, d), kf[d], s);
#pragma unroll
        for (int d = 0; d < K::STEPS; ++d) dp = mma_head(dr.head(0, 32 * u, d), vf[d], dp);
        if (high > ru || ru + 32 > rows) {
          const int lo = first - ru - 4 * hh, hi = rows - ru - 4 * hh;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int i = 8 * (r / 4) + r % 4;
            if (i < lo || i >= hi) s[r] = -__builtin_inff();
          }
        }
        f32x16 ds;
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const f32x4 l4 = *(const f32x4*)(st + 32 * u + 2 * r + 4 * hh);
          const f32x4 d4 = *(const f32x4*)(st + C::ROWS + 32 * u + 2 * r + 4 * hh);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            s[r + i] = fast_exp2(__builtin_fmaf(s[r + i], a.c, -l4[i]));
            ds[r + i] = s[r + i] * (dp[r + i] - d4[i]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const row_frag<T> pf = acc_frag<T>(s, h), df = acc_frag<T>(ds, h);
#pragma unroll
          for (int d = 0; d < DP / 32; ++d) {
            dv[d] = mma_rows(dr.cols(0, 32 * u + 16 * h, d), pf, dv[d]);
            dk[d] = mma_rows(qr.cols(0, 32 * u + 16 * h, d), df, dk[d]);
          }
        }
      }
    }
  }
  if constexpr (C::SETS > 1) {
    if (begin < tiles) {  // the first set takes dV, the last dK
      const auto join = [&](f32x16 (&v)[DP / 32], int to) {
        __syncthreads();
        const int place = (set < to ? set : set - 1) * 4 + wave;
        if (set != to) put_sums(lds, place, v);
        __syncthreads();
        if (set == to)
          for (int i = 0; i < C::SETS - 1; ++i) add_scaled_sums(lds, i * 4 + wave, v, 1.f, 1.f);
      };
      join(dv, 0);
      join(dk, C::SETS - 1);
    }
  }
  if (key >= tile.seq.span) return;
  if (key >= nk) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) dk[d] = dv[d] = zero16();
  }
  const int64_t to = tile.seq.row0 + key;
  if (a.part) {
    float* p = a.part + ((blockIdx.y * a.k_rows + to) * a.G + g) * a.D;
    if (set == C::SETS - 1) store_column<float, DP>(p, dk, a.scale, a.D);
    if (set == 0)
      store_column<float, DP>(p + gridDim.y * a.k_rows * a.G * a.D, dv, 1.f, a.D);
    return;
  }
  if (set == C::SETS - 1)
    store_column<T, DP>((T*)a.dk + to * a.dks + (int64_t)g * a.D, dk, a.scale, a.D);
  if (set == 0) store_column<T, DP>((T*)a.dv + to * a.dvs + (int64_t)g * a.D, dv, 1.f, a.D);
}

// The sum of a split walk's parts in their order, 4 elements a thread; the
// second of two outputs where gridDim.y is 2.
template <typename T>
__global__ void __launch_bounds__(kThreads) sum_kernel(const float* __restrict__ part, T* out0,
                                                       T* out1, int64_t s0, int64_t s1, int64_t rows,
                                                       int width, int parts) {
  const int quads = width / 4;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= rows * quads) return;
  const int64_t row = i / quads, e = i % quads * 4;
  const float* p = part + (int64_t)blockIdx.y * parts * rows * width + row * width + e;
  f32x4 sum = {};
  for (int k = 0; k < parts; ++k) {
    const f32x4 v = *(const f32x4*)(p + k * rows * width);
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] += v[j];
  }
  const float v[4] = {sum[0], sum[1], sum[2], sum[3]};
  store_row<T, 4>((blockIdx.y ? out1 + row * s1 : out0 + row * s0) + e, v);
}

template <typename T>
hipError_t launch_sum(const float* part, T* out0, T* out1, int64_t s0, int64_t s1, int64_t rows,
                      int width, int parts, hipStream_t s) {
  const int64_t n = rows * (width / 4);
  sum_kernel<T><<<dim3((unsigned)((n + kThreads - 1) / kThreads), out1 ? 2 : 1), kThreads, 0, s>>>(
      part, out0, out1, s0, s1, rows, width, parts);
  return hipGetLastError();
}

// Ranges that the walks are split into, with float32 parts: one (no parts)
// where the tiles are 128 workgroups or more, else as many as fill the device,
// of at least 4 steps each (float32, whose steps take 16 times as long: one).  5
// x 301 rows on 203 keys in float32: dK and dV 18 + 3 us (99 in one walk), dQ 15
// + 3 (27).  The rule counts workgroups, not the lengths of causal walks: those
// of one sequence of 2048 or 4096 tokens, 8 groups (128 and 256 workgroups of dK
// and dV), are as long as the longest of 2 x 4096, so its training step takes
// 364 or 842 us where 2 x 4096 takes 1307.
struct Splits {
  int dq, dkv;
};
int split_of(int64_t blocks, int64_t steps, int64_t least) {
  int64_t n = blocks < 128 ? 256 / blocks : 1;
  if (n > steps / least) n = steps / least;
  if (n > 32) n = 32;
  return n < 2 ? 1 : (int)n;
}
Splits splits_of(const AttentionDims& d) {
  const int64_t rep = d.H / d.G, lq = d.qpacked ? d.Lq / d.B : d.Lq;
  const int64_t lk = d.kpacked ? d.Lk / d.B : d.Lk, least = d.bf16 ? 4 : 1;
  const int64_t rows = d.bf16 ? 64 : 32;
  return {split_of(attention_blocks(d), lk / kKeys, least),
          split_of(attention_key_blocks(d), lq * rep / rows, least)};
}
size_t part_bytes(const AttentionDims& d) {
  const Splits n = splits_of(d);
  const size_t q = n.dq > 1 ? (size_t)n.dq * d.q_rows() * d.H * d.D * 4 : 0;
  const size_t kv = n.dkv > 1 ? (size_t)n.dkv * 2 * d.k_rows() * d.G * d.D * 4 : 0;
  return q > kv ? q : kv;
}

template <typename F>
hipError_t launch_lds(F kernel, int64_t blocks, int splits, int threads, int bytes,
                      const BwdArgs& a, hipStream_t s) {
  const hipError_t e =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)blocks, splits), threads, bytes, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DP>
hipError_t go(BwdArgs a, float* part, Splits n, hipStream_t s) {
  using C = DkvCfg<T, DP>;
  a.slots = tile_slots(a.qside, a.rep, kRows);
  a.part = n.dq > 1 ? part : nullptr;
  hipError_t e = launch_lds(attention_dq_kernel<T, DP>, a.slots * a.G, n.dq, kThreads,
                            4 * kKeys * TileCfg<T, DP>::ROWB, a, s);
  if (e != hipSuccess) return e;
  if (a.part) {
    e = launch_sum<T>(part, (T*)a.dq, nullptr, a.dqs, 0, a.q_rows, a.H * a.D, n.dq, s);
    if (e != hipSuccess) return e;
  }
  a.part = n.dkv > 1 ? part : nullptr;
  a.slots = tile_slots(a.kside, 1, kTileKeys);
  e = launch_lds(attention_dkv_kernel<T, DP>, a.slots * a.G, n.dkv, C::THREADS, C::LDS, a, s);
  if (e != hipSuccess || !a.part) return e;
  return launch_sum<T>(part, (T*)a.dk, (T*)a.dv, a.dks, a.dvs, a.k_rows, a.G * a.D, n.dkv, s);
}

size_t row_bytes(const AttentionDims& d) {
  return ((size_t)d.q_rows() * d.H * 2 * sizeof(float) + 255) & ~(size_t)255;
}

}  // namespace

int64_t attention_key_blocks(const AttentionDims& d) {
  return tile_slots({nullptr, d.Lk, d.B, d.kpacked}, 1, kTileKeys) * d.G;
}

size_t attention_backward_bytes(const AttentionDims& d) {
  return row_bytes(d) + part_bytes(d);
}

hipError_t launch_attention_backward(const AttentionDims& d, const void* q, const void* k,
                                     const void* v, const int32_t* q_seqs, const int32_t* k_seqs,
                                     const void* o, const float* lse, const void* dout, void* dq,
                                     void* dk, void* dv, void* ws, hipStream_t s) {
  const int64_t rows = d.q_rows() * d.H;
  float* lse2 = (float*)ws;
  float* delta = lse2 + rows;
  BwdArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  a.dout = dout;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.lse2 = lse2;
  a.delta = delta;
  a.qside = {q_seqs, d.Lq, d.B, d.qpacked};
  a.kside = {k_seqs, d.Lk, d.B, d.kpacked};
  a.qs = d.qs;
  a.ks = d.ks;
  a.vs = d.vs;
  a.dqs = d.dqs;
  a.dks = d.dks;
  a.dvs = d.dvs;
  a.q_rows = d.q_rows();
  a.k_rows = d.k_rows();
  a.H = (int)d.H;
  a.G = (int)d.G;
  a.rep = (int)(d.H / d.G);
  a.D = (int)d.D;
  a.div_l = 0;
  while ((1 << a.div_l) < a.rep) ++a.div_l;
  a.div_m = (unsigned)((((uint64_t)1 << (31 + a.div_l)) + a.rep - 1) / a.rep);
  a.causal = d.causal;
  a.c = d.scale * kLog2e;
  a.scale = d.scale;
  float* part = (float*)((char*)ws + row_bytes(d));
  const Splits n = splits_of(d);
  if (d.bf16)
    return d.D <= 64 ? go<bf16, 64>(a, part, n, s) : go<bf16, 128>(a, part, n, s);
  return d.D <= 64 ? go<float, 64>(a, part, n, s) : go<float, 128>(a, part, n, s);
}

}  // namespace m2
