// attention: softmax attention of a prompt, causal or not, with grouped heads,
// over padded or packed sequences.  The mathematics of a row stands in
// attention_fwd.h.
//
// Bound by the matrix cores where rows are many: a workgroup takes 128 packed
// rows of a group and walks the keys in tiles of 64, K and V double-buffered in
// LDS by direct loads; the exponentials (5 vector instructions for a score)
// run between the matrix instructions of the same wavefront.  16384 tokens, 32
// heads of 128 in 8 groups, causal: 2.02 ms, 1090 TFLOP/s (a bfloat16 library
// product reaches 1280); heads of 64: 910.  Matrix cores busy 56 % of the
// cycles, vector ALU 52 %.  Steps without that interleaving: 2.18 ms; with
// every LDS read ahead of the products instead: 2.20.
#include "attention_fwd.h"

namespace m2 {

namespace {

constexpr int kRows = 128;  // packed rows of a workgroup: 4 wavefronts of 32
constexpr int kKeys = 64;   // keys of a tile
constexpr int kThreads = 256;
constexpr int kMaxParts = 64;

struct FwdArgs {
  const void *q, *k, *v;
  void* o;
  float* lse;
  float *part_o, *part_lse;  // [splits][rows of q][H][D] and [..][H]; NULL: o and lse are written
  Side qside, kside;
  int64_t qs, ks, vs, slots, q_rows;
  int H, G, rep, D, splits;
  bool causal;
  float c;  // scale * log2(e)
};

// SETS = 2: two sets of 4 wavefronts take every other tile and join at the
// end, so that few rows walk their keys in half the time.
template <typename T, int DP, int SETS>
struct FwdCfg {
  static constexpr int TILE = kKeys * TileCfg<T, DP>::ROWB;
  static constexpr int BUF = 2 * SETS * TILE;  // K and V of a tile for each set
  static constexpr int JOIN = SETS == 2 ? (4 * 32 * DP + 4 * 128) * 4 : 0;
  static constexpr int LDS = 2 * BUF > JOIN ? 2 * BUF : JOIN;
  static constexpr int WAVES_PER_SIMD = sizeof(T) == 2 ? 2 : 1;
};

template <typename T, int DP, int SETS>
__global__ void __launch_bounds__((kThreads * SETS), (FwdCfg<T, DP, SETS>::WAVES_PER_SIMD))
    attention_kernel(FwdArgs a) {
  using K = TileCfg<T, DP>;
  using C = FwdCfg<T, DP, SETS>;
  extern __shared__ __align__(16) char lds[];  // [2][SETS][K tile, V tile]
  const int lane = lane_id(), wave = wave_id() & 3, set = wave_id() >> 2, hh = lane >> 5;
  const int thread = threadIdx.x & (kThreads - 1);
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
  // keys that a row sees; none for rows behind the sequence
  const auto seen = [&](int tok) {
    const int64_t n = (int64_t)tok + nk - nq + 1;
    return a.causal ? (int)clamp64(n, nk) : nk;
  };
  const int lim = row < rows ? seen(token) : 0;
  const int last = min(tile.r0 + kRows, rows) - 1;
  const int most = last >= tile.r0 ? seen(last / a.rep) : 0;  // of the workgroup's rows
  const int tiles = (most + kKeys - 1) / kKeys;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int t0 = blockIdx.y * per, t1 = t0 + per < tiles ? t0 + per : tiles;

  RowState<T, DP, kKeys / 32> st;
  st.clear();
  if (t0 < t1) {
    head_frag<T> q[K::STEPS];
    const int safe = row < rows ? row : rows - 1;
    load_row_frags<T, DP>((const T*)a.q + (tile.seq.row0 + safe / a.rep) * a.qs +
                              (int64_t)(g * a.rep + safe % a.rep) * a.D,
                          a.D, q);
    const T* k = (const T*)a.k + (int64_t)ks.row0 * a.ks + (int64_t)g * a.D;
    const T* v = (const T*)a.v + (int64_t)ks.row0 * a.vs + (int64_t)g * a.D;
    const uint32_t base = lds_addr(lds) + set * 2 * C::TILE;
    clear_ends<T, DP>(lds, 4 * SETS * kKeys, a.D, threadIdx.x, kThreads * SETS);
    int low = lim;  // the fewest keys of this wavefront's rows
#pragma unroll
    for (int m = 1; m < 32; m *= 2) low = min(low, __shfl_xor(low, m));
    low = min(__builtin_amdgcn_readfirstlane(low), t1 * kKeys);
    using St = Stager<T, DP, kKeys, kThreads>;
    const St ks_(a.ks, thread), vs_(a.vs, thread);
    const int steps = (t1 - t0 + SETS - 1) / SETS;
    // the last set may have no tile in its last step: keys that no row sees
    const int end = min(lim, t1 * kKeys);
    const auto tile_at = [&](int i) { return (t0 + i * SETS + set) * kKeys; };
    const auto load = [&](const T* x, int64_t stride, const St& st_, uint32_t to, int i) {
      const int r0 = tile_at(i);
      if (r0 + kKeys <= nk)
        st_.load(to, x + r0 * stride, a.D, thread);
      else
        St::load_tail(to, x, stride, r0, nk, nullptr, a.D, thread);
    };
    const TileReader<T, DP> kr(base), vr = kr.later(C::TILE);
    using State = RowState<T, DP, kKeys / 32>;
    const float slack = State::slack_of(a.c);
    typename State::Scores s0, s1;  // s1: the next tile's
    if constexpr (sizeof(T) == 4) {
      // Products in float32 take 16 times as long as in bfloat16: nothing to
      // put beside them matters.
      load(k, a.ks, ks_, base, 0);
      load(v, a.vs, vs_, base + C::TILE, 0);
      for (int i = 0; i < steps; ++i) {
        const int buf = (i & 1) * C::BUF;
        wait_vm(0);
        lds_barrier();  // tile i is there, and tile i - 1 is not read any more
        if (i + 1 < steps) {
          load(k, a.ks, ks_, base + (C::BUF - buf), i + 1);
          load(v, a.vs, vs_, base + C::TILE + (C::BUF - buf), i + 1);
        }
        typename State::Weights p;
        State::scores(q, kr.later(buf), s0);
        if (low < tile_at(i) + kKeys) State::mask(s0, end - tile_at(i));
        st.raise(State::top(s0), slack, a.c);
        st.weigh(s0, a.c, p);
        st.take(vr.later(buf), p);
      }
    } else {
      load(k, a.ks, ks_, base, 0);
      wait_vm(0);
      lds_barrier();
      if (steps > 1) load(k, a.ks, ks_, base + C::BUF, 1);
      load(v, a.vs, vs_, base + C::TILE, 0);
      State::scores(q, kr, s0);
      if (low < tile_at(0) + kKeys) State::mask(s0, end - tile_at(0));
      st.raise(State::top(s0), slack, a.c);
      const auto arrive = [&](int i, int buf) {
        wait_vm(0);
        lds_barrier();  // K of step i + 1 and V of step i are there, and none is read any more
        if (i + 2 < steps) load(k, a.ks, ks_, base + buf, i + 2);
        if (i + 1 < steps) load(v, a.vs, vs_, base + C::TILE + (C::BUF - buf), i + 1);
      };
      // Step i: the next tile's scores beside this tile's exponentials, then this
      // tile's values beside the next one's maximum.
      const auto step = [&](typename State::Scores& s, typename State::Scores& next, int i, int buf) {
        typename State::Weights p;
        arrive(i, buf);
        st.scores_and_weigh(q, kr.fresh(C::BUF - buf), next, s, a.c, p);
        if (low < tile_at(i + 1) + kKeys) State::mask(next, end - tile_at(i + 1));
        st.raise(st.take_and_top(vr.fresh(buf), p, next), slack, a.c);
      };
      int i = 0;
      for (; i + 2 < steps; i += 2) {
        step(s0, s1, i, 0);
        step(s1, s0, i + 1, C::BUF);
      }
      typename State::Weights p;
      if (i + 1 < steps) {
        step(s0, s1, i, 0);
        arrive(i + 1, C::BUF);
        st.weigh(s1, a.c, p);
        st.take(vr.fresh(C::BUF), p);
      } else {
        arrive(i, 0);
        st.weigh(s0, a.c, p);
        st.take(vr.fresh(0), p);
      }
    }
  }

  float l = st.l + __shfl_xor(st.l, 32);
  if constexpr (SETS == 2) {
    if (t0 < t1) {  // the first set takes the second's sums
      __syncthreads();
      float* stats = (float*)lds + 4 * 32 * DP + wave * 128;
      if (set == 1) {
        put_sums(lds, wave, st.o);
        stats[lane] = st.m;
        stats[64 + lane] = l;
      }
      __syncthreads();
      if (set == 0) {
        const float m1 = stats[lane], l1 = stats[64 + lane];
        const float top = __builtin_fmaxf(st.m, m1);
        const float ref = top == -__builtin_inff() ? 0.f : top;
        const float f0 = fast_exp2((st.m - ref) * a.c), f1 = fast_exp2((m1 - ref) * a.c);
        l = l * f0 + l1 * f1;
        st.m = top;
        add_scaled_sums(lds, wave, st.o, f0, f1);
      }
    }
    if (set == 1) return;
  }
  l = row_sum(l, st.m);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (row >= span) return;
  const int64_t at = (int64_t)(tile.seq.row0 + token) * a.H + head;
  // log2 units until the end
  const float lse = l == 0.f ? -__builtin_inff() : st.m * a.c + __builtin_amdgcn_logf(l);
  if (a.part_o) {
    const int64_t p = (int64_t)blockIdx.y * a.q_rows * a.H + at;
    if (hh == 0) a.part_lse[p] = lse;
    store_column<float, DP>(a.part_o + p * a.D, st.o, inv, a.D);
    return;
  }
  if (hh == 0) a.lse[at] = lse * kLn2;
  store_column<T, DP>((T*)a.o + at * a.D, st.o, inv, a.D);
}

// Joins the parts of `rows` (token, head) rows: 32 lanes a row, 4 elements
// each.  A lane weighs parts lane and lane + 32; rows without keys in a part
// left zeros there.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(const float* __restrict__ part_o,
                                                        const float* __restrict__ part_lse,
                                                        T* __restrict__ o, float* __restrict__ lse,
                                                        int64_t rows, int D, int parts) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, e = lane * 4;
  if (row >= rows) return;
  const float none = -__builtin_inff();
  const float l0 = lane < parts ? part_lse[lane * rows + row] : none;
  const float l1 = lane + 32 < parts ? part_lse[(lane + 32) * rows + row] : none;
  float top = __builtin_fmaxf(l0, l1);
#pragma unroll
  for (int m = 1; m < 32; m *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, m, 32));
  const float base = top == none ? 0.f : top;
  const float w0 = fast_exp2(l0 - base), w1 = fast_exp2(l1 - base);
  const float sum = lanes_sum<32>(w0 + w1);
  f32x4 acc = {};
  const int last = parts - 1;
  const float* p = part_o + row * D + (e < D ? e : 0);
  for (int k = 0; k < parts; k += 4) {
    f32x4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *(const f32x4*)(p + min(k + i, last) * rows * D);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float w = __shfl(k + i < 32 ? w0 : w1, (k + i) & 31, 32);
      if (k + i > last) w = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = __builtin_fmaf(w, v[i][j], acc[j]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (lse && lane == 0) lse[row] = sum == 0.f ? none : (base + __builtin_amdgcn_logf(sum)) * kLn2;
  if (e < D) {
    const float v[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
    store_row<T, 4>(o + row * D + e, v);
  }
}

template <typename T, int DP, int SETS>
hipError_t go(const FwdArgs& a, hipStream_t s) {
  constexpr int bytes = FwdCfg<T, DP, SETS>::LDS;
  const auto kernel = attention_kernel<T, DP, SETS>;
  const hipError_t e =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)(a.slots * a.G), a.splits), kThreads * SETS, bytes, s>>>(a);
  return hipGetLastError();
}

Side query_side(const AttentionDims& d, const int32_t* seqs) {
  return {seqs, d.Lq, d.B, d.qpacked};
}
Side key_side(const AttentionDims& d, const int32_t* seqs) { return {seqs, d.Lk, d.B, d.kpacked}; }

// While the rows give at most one workgroup for each CU (256; packed rows count
// with the slots that may stay empty): two sets in each, and the keys split into
// as many parts as give one workgroup to each CU, of at least 4 tiles for each
// set.  One set in two workgroups for each CU has twice the parts: 64 rows of 32
// heads on a prefix of 16384 took 28 + 7 us with the join instead of 29 + 5, 128
// tokens on 32768 keys 79 + 7 instead of 84 + 5.  Above 256 workgroups one set.
// From 257 to 512 two sets would gain where one causal sequence's walks differ
// (1152, 1536 and 2048 tokens, 32 heads of 128: 26, 34 and 50 us instead of 29,
// 37 and 52; 2048 tokens, 24 heads of 64: 27 instead of 33) and lose where they
// are equal or short (the same without a causal limit: 48, 60, 83 and 49 instead
// of 39, 52, 75 and 42; 4 x 400 tokens: 23 instead of 19).  float32
// products take 16 times as long: one set, so that a workgroup has its CU's
// matrix cores alone, and parts of at least one tile (5 x 301 rows on 203 keys:
// 12 + 3 us, 23 with two sets and no parts).
struct Plan {
  int sets, splits;
};
Plan plan_of(const AttentionDims& d) {
  const int64_t blocks = tile_slots(query_side(d, nullptr), d.H / d.G, kRows) * d.G;
  if (blocks > 256) return {1, 1};
  const int sets = d.bf16 ? 2 : 1;
  const int64_t keys = d.kpacked ? d.Lk / d.B : d.Lk;
  const int64_t most = keys / ((d.bf16 ? 4 : 1) * sets * kKeys);
  int64_t n = 256 / blocks;
  if (n > most) n = most;
  if (n > kMaxParts / 2) n = kMaxParts / 2;
  return {sets, n < 2 ? 1 : (int)n};
}
int splits_of(const AttentionDims& d) { return plan_of(d).splits; }

}  // namespace

int64_t attention_blocks(const AttentionDims& d) {
  return tile_slots(query_side(d, nullptr), d.H / d.G, kRows) * d.G;
}

size_t attention_forward_bytes(const AttentionDims& d) {
  const int n = splits_of(d);
  if (n == 1) return 0;
  const size_t rows = (size_t)d.q_rows() * d.H;
  return (size_t)n * rows * (d.D + 1) * 4;
}

int attention_parts(const AttentionDims& d) { return splits_of(d); }

hipError_t launch_attention_join(const float* part_o, const float* part_lse, void* o, float* lse,
                                 int64_t rows, int64_t D, int parts, bool bf, hipStream_t s) {
  const unsigned blocks = (unsigned)((rows + kThreads / 32 - 1) / (kThreads / 32));
  if (bf)
    join_kernel<bf16>
        <<<blocks, kThreads, 0, s>>>(part_o, part_lse, (bf16*)o, lse, rows, (int)D, parts);
  else
    join_kernel<float>
        <<<blocks, kThreads, 0, s>>>(part_o, part_lse, (float*)o, lse, rows, (int)D, parts);
  return hipGetLastError();
}

namespace {

FwdArgs args_of(const AttentionDims& d, const void* q, const void* k, const void* v,
                const int32_t* q_seqs, const int32_t* k_seqs) {
  FwdArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.qside = query_side(d, q_seqs);
  a.kside = key_side(d, k_seqs);
  a.qs = d.qs;
  a.ks = d.ks;
  a.vs = d.vs;
  a.slots = attention_blocks(d) / d.G;
  a.q_rows = d.q_rows();
  a.H = (int)d.H;
  a.G = (int)d.G;
  a.rep = (int)(d.H / d.G);
  a.D = (int)d.D;
  a.splits = splits_of(d);
  a.causal = d.causal;
  a.c = d.scale * kLog2e;
  return a;
}

hipError_t run(const AttentionDims& d, const FwdArgs& a, hipStream_t s) {
  const bool narrow = d.D <= 64;
  if (plan_of(d).sets == 2) return narrow ? go<bf16, 64, 2>(a, s) : go<bf16, 128, 2>(a, s);
  if (d.bf16) return narrow ? go<bf16, 64, 1>(a, s) : go<bf16, 128, 1>(a, s);
  return narrow ? go<float, 64, 1>(a, s) : go<float, 128, 1>(a, s);
}

}  // namespace

hipError_t launch_attention_parts(const AttentionDims& d, const void* q, const void* k,
                                  const void* v, float* part_o, float* part_lse, hipStream_t s) {
  FwdArgs a = args_of(d, q, k, v, nullptr, nullptr);
  a.part_o = part_o;
  a.part_lse = part_lse;
  return run(d, a, s);
}

hipError_t launch_attention(const AttentionDims& d, const void* q, const void* k, const void* v,
                            const int32_t* q_seqs, const int32_t* k_seqs, void* o, float* lse,
                            void* ws, hipStream_t s) {
  FwdArgs a = args_of(d, q, k, v, q_seqs, k_seqs);
  a.o = o;
  a.lse = lse;
  if (a.splits == 1) return run(d, a, s);
  const int64_t rows = a.q_rows * a.H;
  a.part_o = (float*)ws;
  a.part_lse = a.part_o + a.splits * rows * a.D;
  const hipError_t e = run(d, a, s);
  if (e != hipSuccess) return e;
  return launch_attention_join(a.part_o, a.part_lse, o, lse, rows, d.D, a.splits, d.bf16, s);
}

}  // namespace m2
