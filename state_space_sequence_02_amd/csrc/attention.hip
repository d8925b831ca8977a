// attention: softmax attention of a prompt, causal or not, with grouped heads,
// over padded or packed sequences.  The mathematics of a row stands in
// attention_fwd.h.
#include "attention_fwd.h"

namespace m2 {

namespace {

constexpr int kRows = 128;  // packed rows of a workgroup: 4 wavefronts of 32
constexpr int kKeys = 64;   // keys of a tile
constexpr int kThreads = 256;

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

template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) attention_kernel(FwdArgs a) {
  using K = TileCfg<T, DP>;
  constexpr int TILE = kKeys * K::ROWB;
  extern __shared__ __align__(16) char lds[];  // [2][K tile, V tile]
  const int lane = lane_id(), wave = wave_id(), hh = lane >> 5;
  const int g = blockIdx.x % a.G;
  // causal rows at the end of a sequence see most keys: they go first
  const Tile tile = tile_of(a.qside, a.rep, kRows, a.slots - 1 - blockIdx.x / a.G);
  const int64_t span = tile.seq.span * a.rep;
  if (tile.r0 >= span) return;
  const int nq = (int)tile.seq.n, rows = nq * a.rep;
  Seq ks = {0, 0, 0};
  if (tile.b >= 0) ks = seq_of(a.kside, tile.b);
  const int nk = (int)ks.n;

  const int row = (int)tile.r0 + wave * 32 + (lane & 31);
  const int token = row / a.rep;
  const int head = g * a.rep + row % a.rep;
  // keys that a row sees; none for rows behind the sequence
  const auto seen = [&](int tok) {
    const int64_t n = (int64_t)tok + nk - nq + 1;
    return a.causal ? (int)clamp64(n, nk) : nk;
  };
  const int lim = row < rows ? seen(token) : 0;
  const int last = (int)(tile.r0 + kRows < rows ? tile.r0 + kRows : rows) - 1;
  const int most = last >= tile.r0 ? seen(last / a.rep) : 0;  // of the workgroup's rows
  const int tiles = (most + kKeys - 1) / kKeys;
  const int per = (tiles + a.splits - 1) / a.splits;
  const int t0 = blockIdx.y * per, t1 = t0 + per < tiles ? t0 + per : tiles;

  RowState<T, DP> st;
  st.clear();
  if (t0 < t1) {
    head_frag<T> q[K::STEPS];
    const int safe = row < rows ? row : rows - 1;
    load_row_frags<T, DP>((const T*)a.q + (tile.seq.row0 + safe / a.rep) * a.qs +
                              (int64_t)(g * a.rep + safe % a.rep) * a.D,
                          a.D, q);
    const T* k = (const T*)a.k + ks.row0 * a.ks + (int64_t)g * a.D;
    const T* v = (const T*)a.v + ks.row0 * a.vs + (int64_t)g * a.D;
    const uint32_t base = lds_addr(lds);
    clear_ends<T, DP>(lds, 4 * kKeys, a.D, threadIdx.x, kThreads);
    // the fewest and the most keys of this wavefront's rows
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
    const TileReader<T, DP> first(base);
    stage(t0);
    for (int t = t0; t < t1; ++t) {
      wait_vm(0);
      lds_barrier();  // tile t is there, and every wavefront is done with tile t - 1
      if (t + 1 < t1) stage(t + 1);
      const int k0 = t * kKeys;
      if (high > k0) {
        const TileReader<T, DP> kr = first.later((t & 1) * 2 * TILE);
        st.template step<kKeys / 32>(q, kr, kr.later(TILE), low < k0 + kKeys, lim - k0, a.c);
      }
    }
  }

  const float l = st.l + __shfl_xor(st.l, 32);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  if (row >= span) return;
  const int64_t at = (tile.seq.row0 + token) * a.H + head;
  // log2 units until the end
  const float lse = l > 0.f ? st.m * a.c + __builtin_amdgcn_logf(l) : -__builtin_inff();
  if (a.part_o) {
    const int64_t p = (int64_t)blockIdx.y * a.q_rows * a.H + at;
    if (hh == 0) a.part_lse[p] = lse;
    float* o = a.part_o + p * a.D;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int r = 0; r < 16; r += 4) {
        const int e = 32 * d + 2 * r + 4 * hh;
        const float v[4] = {st.o[d][r] * inv, st.o[d][r + 1] * inv, st.o[d][r + 2] * inv,
                            st.o[d][r + 3] * inv};
        if (e < a.D) store_row<float, 4>(o + e, v);
      }
    return;
  }
  if (hh == 0) a.lse[at] = lse * kLn2;
  T* o = (T*)a.o + at * a.D;
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int e = 32 * d + 2 * r + 4 * hh;
      const float v[4] = {st.o[d][r] * inv, st.o[d][r + 1] * inv, st.o[d][r + 2] * inv,
                          st.o[d][r + 3] * inv};
      if (e < a.D) store_row<T, 4>(o + e, v);
    }
}

// Joins the parts of `rows` (token, head) rows: 32 lanes a row, 4 elements each.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(const float* __restrict__ part_o,
                                                        const float* __restrict__ part_lse,
                                                        T* __restrict__ o, float* __restrict__ lse,
                                                        int64_t rows, int D, int parts) {
  const int64_t row = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int e = threadIdx.x % 32 * 4;
  if (row >= rows) return;
  float top = -__builtin_inff();
  for (int p = 0; p < parts; ++p) top = __builtin_fmaxf(top, part_lse[p * rows + row]);
  const float base = top == -__builtin_inff() ? 0.f : top;
  float sum = 0.f;
  f32x4 acc = {};
  for (int p = 0; p < parts; ++p) {
    const float w = fast_exp2(part_lse[p * rows + row] - base);
    sum += w;
    if (e < D && w > 0.f) {
      const f32x4 v = *(const f32x4*)(part_o + (p * rows + row) * D + e);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  if (lse && e == 0)
    lse[row] = sum > 0.f ? (base + __builtin_amdgcn_logf(sum)) * kLn2 : -__builtin_inff();
  if (e < D) {
    const float v[4] = {acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv};
    store_row<T, 4>(o + row * D + e, v);
  }
}

template <typename T, int DP>
hipError_t go(const FwdArgs& a, hipStream_t s) {
  constexpr int bytes = 4 * kKeys * TileCfg<T, DP>::ROWB;
  const auto kernel = attention_kernel<T, DP>;
  const hipError_t e =
      hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)(a.slots * a.G), a.splits), kThreads, bytes, s>>>(a);
  return hipGetLastError();
}

Side query_side(const AttentionDims& d, const int32_t* seqs) {
  return {seqs, d.Lq, d.B, d.qpacked};
}
Side key_side(const AttentionDims& d, const int32_t* seqs) { return {seqs, d.Lk, d.B, d.kpacked}; }

// Parts that the keys are split into: one where the rows alone fill the
// device, else as many as do, but at least 4 tiles of keys for each.
int splits_of(const AttentionDims& d) {
  const int64_t blocks = tile_slots(query_side(d, nullptr), d.H / d.G, kRows) * d.G;
  const int64_t keys = d.kpacked ? d.Lk / d.B : d.Lk;
  const int64_t most = keys / (4 * kKeys);
  int64_t n = 512 / blocks;
  if (n > most) n = most;
  if (n > 64) n = 64;
  return n < 2 ? 1 : (int)n;
}

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
  if (d.bf16) return d.D <= 64 ? go<bf16, 64>(a, s) : go<bf16, 128>(a, s);
  return d.D <= 64 ? go<float, 64>(a, s) : go<float, 128>(a, s);
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
