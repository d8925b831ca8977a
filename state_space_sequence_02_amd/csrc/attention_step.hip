// attention_step: one token of every sequence against its cache of keys and
// values, with or without a prefix that all sequences share.  Sequence b sees
// the prefix, rows 0 .. n - 1 of its cache (n = lengths[b]) and the token
// itself, whose key and value go to row n of the cache (if it has one: a full
// cache keeps what it holds, the token is still seen).  They are read from the
// call's inputs, never from the cache, so no workgroup waits for the one that
// writes them.
//
// Bound by HBM on the caches, which are read once: a workgroup takes the rep
// rows of one (sequence, group) and a range of the keys; its 4 or 8 wavefronts
// walk tiles of 32 keys on their own, each next K and V on its way into LDS as
// soon as the last is used, and join at the end.  The prefix is one product for
// the whole batch: batch * rep packed rows against the prefix's keys
// (attention.hip), so it is read once for all sequences and not once for each.
// Ranges and prefix leave float32 parts that one more kernel joins; a single
// range without a prefix needs none.
// 128 sequences of up to 4096 rows of 8 x 128, 1.1 GB: 215 us, 5.1 TB/s.
#include "attention_fwd.h"

namespace m2 {

namespace {

struct StepArgs {
  const void *q, *k, *v;
  void *k_cache, *v_cache;
  const int32_t* lengths;
  void* o;
  float *part_o, *part_lse;  // NULL: o is written
  int64_t qs, ks, vs, rows;  // rows of a cache
  int B, H, G, rep, D, tiles;  // tiles of 32 packed rows
  float c;
};

// Workgroup n of slots * G: its slot and group.  Workgroups go to the 8 XCDs in
// turn; eight neighbours take eight slots of one group, so that an XCD reads
// whole rows of the caches, in which the groups lie side by side (128 x 4096
// rows of 8 x 128: 215 us; group n % G: 219).
struct Place {
  int slot, g;
};
__device__ __forceinline__ Place place_of(unsigned n, unsigned slots, unsigned G) {
  constexpr unsigned X = 8;
  const unsigned block = n / (X * G), first = block * X;
  const unsigned wide = slots - first < X ? slots - first : X;  // slots of the last block
  const unsigned r = n - block * X * G;
  const unsigned g = r / wide;
  return {(int)(first + r - g * wide), (int)g};
}

// W wavefronts, 4 or 8, of which a CU holds 8 (float32 heads above 64: 4).
template <typename T, int DP, int W>
__global__ void __launch_bounds__((64 * W), (sizeof(T) * DP > 256 ? 1 : 2))
    attention_step_kernel(StepArgs a) {
  using K = TileCfg<T, DP>;
  constexpr int TILE = 32 * K::ROWB;
  extern __shared__ __align__(16) char lds[];  // [W][K tile, V tile]
  const int lane = lane_id(), wave = wave_id(), hh = lane >> 5;
  const Place at = place_of(blockIdx.x, a.B * a.tiles, a.G);
  const int g = at.g;
  const int b = at.slot / a.tiles, r0 = at.slot % a.tiles * 32;
  const int64_t cap = a.rows;
  const int n = (int)clamp64(uniform_at(a.lengths, b), cap);
  const int64_t cs = (int64_t)a.G * a.D;
  const int64_t cache = (int64_t)b * cap * cs + (int64_t)g * a.D;
  const T* kn = (const T*)a.k + b * a.ks + (int64_t)g * a.D;
  const T* vn = (const T*)a.v + b * a.vs + (int64_t)g * a.D;
  T* kc = (T*)a.k_cache + cache;
  T* vc = (T*)a.v_cache + cache;
  const int row = r0 + (lane & 31);
  const int head = g * a.rep + (row < a.rep ? row : a.rep - 1);
  const int nk = n + 1;
  const int tiles = (nk + 31) / 32;
  const int per = (tiles + gridDim.y - 1) / gridDim.y;
  const int t0 = blockIdx.y * per, t1 = t0 + per < tiles ? t0 + per : tiles;
  char* mine = lds + wave * 2 * TILE;
  const uint32_t base = lds_addr(mine);
  using State = RowState<T, DP, 1>;
  State st;
  st.clear();
  if (t0 + wave < t1) {
    head_frag<T> q[K::STEPS];
    load_row_frags<T, DP>((const T*)a.q + b * a.qs + (int64_t)head * a.D, a.D, q);
    clear_ends<T, DP>(mine, 2 * 32, a.D, lane, 64);
    using St = Stager<T, DP, 32, 64>;
    const St off(cs, lane);
    const auto load = [&](const T* cache, const T* token, uint32_t to, int t) {
      if (t * 32 + 32 <= n)
        off.load(to, cache + t * 32 * cs, a.D, lane);
      else
        St::load_tail(to, cache, cs, t * 32, nk, token, a.D, lane);
    };
    // Waits for a load and for the reads before the next one into its place.
    const auto here = [&](int later) {
      wait_vm(later);
      asm volatile("" ::: "memory");
    };
    const auto read = [&] {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
      asm volatile("" ::: "memory");
    };
    const TileReader<T, DP> kr(base), vr = kr.later(TILE);
    load(kc, kn, base, t0 + wave);
    load(vc, vn, base + TILE, t0 + wave);
    for (int t = t0 + wave; t < t1; t += W) {
      typename State::Scores s;
      typename State::Weights p;
      here(St::PER);
      State::scores(q, kr, s);
      read();
      const bool more = t + W < t1;
      if (more) load(kc, kn, base, t + W);
      if (t * 32 + 32 > nk) State::mask(s, nk - t * 32);
      st.raise(State::top(s), State::slack_of(a.c), a.c);
      st.weigh(s, a.c, p);
      here(more ? St::PER : 0);
      st.take(vr, p);
      read();
      if (more) load(vc, vn, base + TILE, t + W);
    }
  }

  // the token's own row of the cache, which nothing here reads
  if (blockIdx.y == 0 && r0 == 0 && n < cap) {
    for (int i = threadIdx.x * 4; i < a.D; i += 64 * W * 4) {
      *(raw_t<T, 4>*)(kc + n * cs + i) = *(const raw_t<T, 4>*)(kn + i);
      *(raw_t<T, 4>*)(vc + n * cs + i) = *(const raw_t<T, 4>*)(vn + i);
    }
  }

  // Join the wavefronts: each scales its sums to the common maximum.
  __syncthreads();
  float* tops = (float*)lds;            // [W][32]
  float* sums = tops + W * 32;          // [W][32]
  float* outs = sums + W * 32;          // [W][32][DP + 4]
  constexpr int LD = DP + 4;
  const int x = lane & 31;
  const float l = st.l + __shfl_xor(st.l, 32);
  const int left = a.rep - r0 < 32 ? a.rep - r0 : 32;
  if (x < left) {
    if (hh == 0) {
      tops[wave * 32 + x] = st.m;
      sums[wave * 32 + x] = l;
    }
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const float v[4] = {st.o[d][r], st.o[d][r + 1], st.o[d][r + 2], st.o[d][r + 3]};
        store_row<float, 4>(outs + (wave * 32 + x) * LD + 32 * d + 2 * r + 4 * hh, v);
      }
  }
  __syncthreads();
  const int quads = a.D / 4;
  for (int i = threadIdx.x; i < left * quads; i += 64 * W) {
    const int rr = i / quads, e = i % quads * 4;
    float top = tops[rr];
#pragma unroll
    for (int w = 1; w < W; ++w) top = __builtin_fmaxf(top, tops[w * 32 + rr]);
    const float ref = top == -__builtin_inff() ? 0.f : top;
    float sum = 0.f;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = fast_exp2((tops[w * 32 + rr] - ref) * a.c);
      sum += f * sums[w * 32 + rr];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += f * outs[(w * 32 + rr) * LD + e + j];
    }
    sum = row_sum(sum, top);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] *= inv;
    const int64_t at = (int64_t)b * a.H + g * a.rep + r0 + rr;
    if (a.part_o) {
      const int64_t p = (int64_t)blockIdx.y * a.B * a.H + at;
      store_row<float, 4>(a.part_o + p * a.D + e, v);
      if (e == 0)
        a.part_lse[p] = sum == 0.f ? -__builtin_inff() : top * a.c + __builtin_amdgcn_logf(sum);
    } else {
      store_row<T, 4>((T*)a.o + at * a.D + e, v);
    }
  }
}

template <typename T, int DP, int W>
hipError_t go(const StepArgs& a, int splits, hipStream_t s) {
  constexpr int tiles = W * 2 * 32 * TileCfg<T, DP>::ROWB, join = (W * 64 + W * 32 * (DP + 4)) * 4;
  constexpr int bytes = tiles > join ? tiles : join;
  static_assert(bytes <= 160 * 1024, "a CU's LDS");
  const auto kernel = attention_step_kernel<T, DP, W>;
  const hipError_t e =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)((int64_t)a.B * a.tiles * a.G), splits), 64 * W, bytes, s>>>(a);
  return hipGetLastError();
}

template <typename T, int DP>
hipError_t go(const StepArgs& a, int splits, hipStream_t s) {
  if constexpr (sizeof(T) * DP <= 256) {
    // Long walks: one workgroup on a CU, whose wavefronts share a row's groups
    // (128 x 4096 rows: 215 us; with two workgroups of 4 wavefronts 242).
    // Short ones are mostly their beginning and end, which two overlap (64
    // sequences of up to 512 rows: 17 us instead of 20; 4 of 1100: 8.1, 8.4).
    // Around the border the rates of full caches are near: 64 of 1024 rows (four
    // wavefronts) 6.1 TB/s and of 1100 (eight) 5.7, 128 of either 5.3.
    if (a.rows > 1024 * (int64_t)splits) return go<T, DP, 8>(a, splits, s);
  }
  return go<T, DP, 4>(a, splits, s);
}

int64_t row_tiles(const AttentionStepDims& d) { return (d.H / d.G + 31) / 32; }

// Ranges of the cache: as many as fit in one workgroup for each CU, of at least
// one tile for each wavefront where the cache is full.  Workgroups that are no
// divisor of 256 leave CUs idle in the last turn: full caches of 4096 rows of 8
// x 128 stream at 5.3 TB/s for 32 sequences, 5.6 for 64, 5.0 for 17, 4.2 for 33
// and 4.4 for 40.
int splits_of(const AttentionStepDims& d) {
  const int64_t blocks = attention_step_blocks(d);
  const int64_t most = (d.rows + 255) / 256;
  int64_t n = 256 / blocks;
  if (n > most) n = most;
  if (n > 32) n = 32;
  return n < 2 ? 1 : (int)n;
}

AttentionDims prefix_dims(const AttentionStepDims& d) {
  AttentionDims p = {};
  p.B = 1;
  p.Lq = d.B;
  p.Lk = d.prefix;
  p.H = d.H;
  p.G = d.G;
  p.D = d.D;
  p.qs = d.qs;
  p.ks = p.vs = d.G * d.D;
  p.scale = d.scale;
  p.bf16 = d.bf16;
  return p;
}

}  // namespace

int64_t attention_step_blocks(const AttentionStepDims& d) { return d.B * row_tiles(d) * d.G; }

AttentionDims attention_step_prefix(const AttentionStepDims& d) { return prefix_dims(d); }

size_t attention_step_bytes(const AttentionStepDims& d) {
  int n = splits_of(d);
  if (n == 1 && !d.prefix) return 0;
  if (d.prefix) n += attention_parts(prefix_dims(d));
  return (size_t)n * d.B * d.H * (d.D + 1) * 4;
}

hipError_t launch_attention_step(const AttentionStepDims& d, const void* q, const void* k,
                                 const void* v, void* k_cache, void* v_cache,
                                 const int32_t* lengths, const void* k_prefix,
                                 const void* v_prefix, void* o, void* ws, hipStream_t s) {
  StepArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.lengths = lengths;
  a.o = o;
  a.qs = d.qs;
  a.ks = d.ks;
  a.vs = d.vs;
  a.rows = d.rows;
  a.B = (int)d.B;
  a.H = (int)d.H;
  a.G = (int)d.G;
  a.rep = (int)(d.H / d.G);
  a.D = (int)d.D;
  a.tiles = (int)row_tiles(d);
  a.c = d.scale * kLog2e;
  const int splits = splits_of(d);
  const int more = d.prefix ? attention_parts(prefix_dims(d)) : 0;
  const int64_t rows = d.B * d.H;
  if (splits + more > 1) {
    a.part_o = (float*)ws;
    a.part_lse = a.part_o + (splits + more) * rows * d.D;
  }
  hipError_t e;
  if (d.bf16)
    e = d.D <= 64 ? go<bf16, 64>(a, splits, s) : go<bf16, 128>(a, splits, s);
  else
    e = d.D <= 64 ? go<float, 64>(a, splits, s) : go<float, 128>(a, splits, s);
  if (e != hipSuccess || splits + more == 1) return e;
  if (more) {
    e = launch_attention_parts(prefix_dims(d), q, k_prefix, v_prefix,
                               a.part_o + splits * rows * d.D, a.part_lse + splits * rows, s);
    if (e != hipSuccess) return e;
  }
  return launch_attention_join(a.part_o, a.part_lse, o, nullptr, rows, d.D, splits + more, d.bf16,
                               s);
}

}  // namespace m2
