// What the attention kernels share: sequences and tiles of packed rows, the
// tiles in LDS, and the matrix products on fragments.
//
// Packed rows.  Head h reads the keys and values of group g = h / rep
// (rep = H/G).  The rep rows that one token has for a group are rows of the
// same product, so the kernels see, per (sequence, group), n * rep packed
// rows: row r is head g rep + r % rep of token r / rep.  Keys are then read
// once for the heads that share them, and their gradients are sums over the
// packed rows like any other.
//
// Fragments (gfx950, 32x32 products, checked on the device).  Lane l has
// x = l & 31 and half hh = l >> 5.  An accumulator holds column x, rows
// 8 (r / 4) + 4 hh + r % 4 for r = 0 .. 15.
//   Along the head: a fragment is what one lane gives to a product over 16
//   (bfloat16) or 8 (float32) elements of a row of 32 rows: 16 bytes of row x
//   at 16-byte chunk 2 s + hh.  Which elements meet in which instruction does
//   not matter as long as both operands agree.
//   Along the rows: 8 accumulator registers (8 s .. 8 s + 7) of a lane are the
//   elements of its column at 8 of 16 rows; taken as the operand of a product
//   over those rows, the other operand has to hold the same rows: 16 s + 4 hh
//   + j and 16 s + 8 + 4 hh + j, j = 0 .. 3.  For bfloat16 that is what two
//   transposing reads return, so the weights never change lanes.
#pragma once

#include "common.h"
#include "launch.h"
#include "rowvec.h"

namespace m2 {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// ------------------------------------------------------------------ sequences

// One side (queries, or keys and values) of a call.
struct Side {
  const int32_t* seqs;  // lengths [B] or NULL (padded); starts [B + 1] (packed)
  int64_t len;          // rows of a sequence (padded), of all together (packed)
  int64_t B;
  bool packed;
};

struct Seq {
  int row0;  // its first row in the tensor
  int span;  // rows of the tensor that are its own, padding among them
  int n;     // tokens
};

__device__ __forceinline__ int64_t clamp64(int64_t v, int64_t hi) {
  return v < 0 ? 0 : v > hi ? hi : v;
}

// An element that is the same for all lanes, in a scalar register.
__device__ __forceinline__ int uniform_at(const int32_t* p, int64_t i) {
  return __builtin_amdgcn_readfirstlane(p[i]);
}

__device__ __forceinline__ Seq seq_of(const Side& s, int64_t b) {
  const int len = (int)s.len;
  Seq q;
  if (!s.packed) {
    q.row0 = (int)b * len;
    q.span = len;
    q.n = s.seqs ? min(max(uniform_at(s.seqs, b), 0), len) : len;
  } else {
    q.row0 = min(max(uniform_at(s.seqs, b), 0), len);
    q.span = q.n = max(min(uniform_at(s.seqs, b + 1), len) - q.row0, 0);
  }
  return q;
}

// A tile of `tile` packed rows.  Packed: between and behind the sequences there
// are rows that belong to none, so the tensor is cut at 0, starts[0 .. B], len:
// B + 2 pieces of which the first and the last hold no tokens.  The tiles of
// all pieces are at most floor(len rep / tile) + B + 2, whatever the lengths, so
// the number of workgroups follows from the sizes alone (no list is made,
// nothing is copied to the host).
struct Tile {
  Seq seq;
  int b;   // sequence; -1: rows of none
  int r0;  // first packed row
};

inline int64_t tile_slots(const Side& s, int64_t rep, int64_t tile) {
  return s.packed ? s.len * rep / tile + s.B + 2 : s.B * ((s.len * rep + tile - 1) / tile);
}

__device__ __forceinline__ int64_t cut_of(const Side& s, int64_t i) {
  return i == 0 ? 0 : i > s.B + 1 ? s.len : clamp64(s.seqs[i - 1], s.len);
}

__device__ __forceinline__ Tile piece_tile(const Side& s, int piece, int cut, int next, int r0) {
  Tile t;
  t.r0 = __builtin_amdgcn_readfirstlane(r0);
  t.b = __builtin_amdgcn_readfirstlane(piece) - 1;
  t.seq.row0 = __builtin_amdgcn_readfirstlane(cut);
  t.seq.span = max(__builtin_amdgcn_readfirstlane(next) - t.seq.row0, 0);
  t.seq.n = t.seq.span;
  if (t.b == (int)s.B) t.b = -1;
  if (t.b < 0) t.seq.n = 0;
  return t;
}

// The tile that workgroup `slot` takes, the same for all lanes; a tile behind
// its sequence's end is none.  In causal attention a tile's work grows with
// its number in the sequence (queries; of keys, with its number from the
// end): the longest walks have to begin first, or the last of them runs on
// alone.  Padded sequences are gone through tile number by tile number,
// longest walks first.  So are packed ones while their pieces fit a
// wavefront's lanes: F(i) = the tiles that are at least number i is a sum over
// the lanes, workgroup n has the number i with F(i + 1) <= n < F(i), and takes
// the (n - F(i + 1))-th piece that is so long.  With more sequences than that
// no single one holds much of the work; they are taken as they lie.
template <bool KEYS>
__device__ __forceinline__ Tile tile_of(const Side& s, int rep, int tile, int slots, int slot) {
  const int B = (int)s.B;
  if (!s.packed) {
    const uint32_t n = KEYS ? slot : slots - 1 - slot;
    const uint32_t i = n / (uint32_t)B;
    Tile t;
    t.b = n - i * B;
    t.r0 = i * tile;
    t.seq = seq_of(s, t.b);
    return t;
  }
  const int lane = lane_id();
  const int pieces = B + 2;
  if (pieces <= 64) {
    const int cut = (int)cut_of(s, lane), next = (int)cut_of(s, lane + 1);
    int have = 0;
    if (lane < pieces && next > cut) have = (int)(((int64_t)(next - cut) * rep + tile - 1) / tile);
    // sums of counts below 2^24 are exact in float32
    const auto f = [&](int i) {
      return __builtin_amdgcn_readfirstlane((int)lanes_sum<64>((float)max(have - i, 0)));
    };
    int lo = 0, hi = have;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) hi = max(hi, __shfl_xor(hi, m));
    hi = __builtin_amdgcn_readfirstlane(hi);
    if (slot >= f(0)) return piece_tile(s, 0, 0, 0, 0);
    while (hi - lo > 1) {  // F(lo) > slot >= F(hi)
      const int mid = (lo + hi) / 2;
      if (f(mid) > slot)
        lo = mid;
      else
        hi = mid;
    }
    uint64_t mask = __ballot(have > lo);
    for (int k = slot - f(lo + 1); k > 0; --k) mask &= mask - 1;
    const int p = __builtin_ctzll(mask);
    return piece_tile(s, p, __builtin_amdgcn_readlane(cut, p), __builtin_amdgcn_readlane(next, p),
                      (KEYS ? __builtin_amdgcn_readlane(have, p) - 1 - lo : lo) * tile);
  }
  // Piece i takes the slots from floor(cut_i rep / tile) + i on: the next one's
  // first is at least as far as its rows need.  64 pieces are looked at at once.
  int lo = 0, count = pieces;
  while (count > 1) {
    const int step = (count + 63) / 64;
    const int i = lo + lane * step;
    const bool at = i < lo + count && cut_of(s, i) * rep / tile + i <= slot;
    const uint64_t mask = __ballot(at);
    const int last = mask ? 63 - __builtin_clzll(mask) : 0;
    const int left = count - last * step;
    lo += last * step;
    count = left < step ? left : step;
  }
  const int i = __builtin_amdgcn_readfirstlane(lo);
  const int64_t cut = cut_of(s, i);
  return piece_tile(s, i, (int)cut, (int)cut_of(s, i + 1),
                    (int)((slot - (cut * rep / tile + i)) * tile));
}

// ------------------------------------------------------------------ LDS tiles

// A tile's rows hold DP elements (64 or 128, the head's size rounded up) in
// 16-byte chunks; chunk c of row r stands at position c ^ swz(r).  Row reads
// (16 rows, one chunk) then meet every bank once, and so do transposing reads
// (4 rows, 4 chunks of each).
template <typename T, int DP>
struct TileCfg {
  static constexpr int E = 16 / (int)sizeof(T);     // elements of a chunk
  static constexpr int CH = DP / E;                 // chunks of a row: 8, 16 or 32
  static constexpr int ROWB = DP * (int)sizeof(T);  // bytes of a row
  static constexpr int STEPS = CH / 2;              // products along a row
};

template <int CH>
__device__ __forceinline__ int swz(int r) {
  if constexpr (CH == 8)
    return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
  else
    return (r & 3) << 2 | ((r >> 2) & 3);
}

template <int CH>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  return (uint32_t)(r * CH + (c ^ swz<CH>(r))) * 16;
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// A lane's part of a fragment along the head: 16 bytes.
template <typename T>
using head_frag = raw_t<T, 16 / (int)sizeof(T)>;

// c += A B over one step along the head.
__device__ __forceinline__ f32x16 mma_head(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma_head(f32x4 a, f32x4 b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], b[j], c, 0, 0, 0);
  return c;
}

// Operand of a product over 16 rows: 8 values of a lane.
struct f32v8 {
  float v[8];
};
template <typename T>
struct RowFrag;
template <>
struct RowFrag<bf16> {
  typedef bf16x8 type;
};
template <>
struct RowFrag<float> {
  typedef f32v8 type;
};
template <typename T>
using row_frag = typename RowFrag<T>::type;

typedef float at_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 at_bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ at_bf16x2 pack2(float a, float b) {
  return __builtin_convertvector((at_f32x2){a, b}, at_bf16x2);
}
__device__ __forceinline__ bf16x4 pack4(float a, float b, float c, float d) {
  return __builtin_shufflevector(pack2(a, b), pack2(c, d), 0, 1, 2, 3);
}

// Registers 8 s .. 8 s + 7 of an accumulator as such an operand.  bfloat16
// products take bfloat16 weights: one rounding (at most 2^-8 relative) of each
// weight, independent over a sum's terms.
template <typename T>
__device__ __forceinline__ row_frag<T> acc_frag(const f32x16& p, int s) {
  if constexpr (sizeof(T) == 2) {
    return cat(pack4(p[8 * s], p[8 * s + 1], p[8 * s + 2], p[8 * s + 3]),
               pack4(p[8 * s + 4], p[8 * s + 5], p[8 * s + 6], p[8 * s + 7]));
  } else {
    f32v8 f;
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] = p[8 * s + j];
    return f;
  }
}

// Holds a value's computation where it is written (the compiler would move it
// behind a branch, next to its use).
__device__ __forceinline__ void pin(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void pin(bf16x8& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void pin(f32v8& f) {
#pragma unroll
  for (int j = 0; j < 8; ++j) pin(f.v[j]);
}

__device__ __forceinline__ f32x16 mma_rows(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma_rows(const f32v8& a, const f32v8& b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    c = __builtin_amdgcn_mfma_f32_32x32x2f32(a.v[j], b.v[j], c, 0, 0, 0);
  return c;
}

// A lane's reads of LDS tiles.  What a step or a column range changes of an
// address are bits of the chunk, and the swizzle only flips bits, so each
// address is one exclusive or away from the lane's own; rows and tiles are
// constants of the instruction.  Tiles begin at multiples of a row.
template <typename T, int DP>
struct TileReader {
  using K = TileCfg<T, DP>;
  uint32_t row, col;

  __device__ __forceinline__ TileReader(uint32_t tile) {
    const int lane = lane_id(), hh = lane >> 5;
    row = tile + chunk_at<K::CH>(lane & 31, hh);
    if constexpr (sizeof(T) == 2) {
      const int i = lane & 15;
      col = tile + chunk_at<K::CH>(4 * hh + (i >> 2), ((lane >> 4) & 1) * 2 + ((i & 3) >> 1)) +
            (i & 1) * 8;
    } else {
      // row 4 hh + j adds j << 2 to the chunk's flips
      col = tile + chunk_at<K::CH>(4 * hh, (lane & 31) >> 2) + (lane & 3) * 4;
    }
  }
  template <typename V>
  __device__ __forceinline__ static V at(uint32_t a, int offset) {
    typedef __attribute__((address_space(3))) const V* lds_ptr;
    return *(lds_ptr)(uintptr_t)(a + offset);
  }
  // The same reads of a tile that begins `bytes` (multiples of a row) later.
  __device__ __forceinline__ TileReader later(uint32_t bytes) const {
    TileReader r = *this;
    r.row += bytes;
    r.col += bytes;
    return r;
  }
  // The same, where `bytes` is a constant of an unrolled step: the empty asm
  // keeps the addresses from being held in registers across the steps.
  __device__ __forceinline__ TileReader fresh(uint32_t bytes) const {
    TileReader r = later(bytes);
    asm volatile("" : "+v"(r.row), "+v"(r.col));
    return r;
  }
  // Rows r32 .. r32 + 31 at step s along the head; `offset`: bytes from the
  // reader's tile, a constant.
  __device__ __forceinline__ head_frag<T> head(int offset, int r32, int s) const {
    return at<head_frag<T>>(row ^ (32 * s), offset + r32 * K::ROWB);
  }
  // Column 32 dt + x at rows r16 .. r16 + 15, those of acc_frag.
  __device__ __forceinline__ row_frag<T> cols(int offset, int r16, int dt) const {
    const int o = offset + r16 * K::ROWB;
    if constexpr (sizeof(T) == 2) {
      typedef __attribute__((address_space(3))) s16x4* lds_ptr;
      const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_ptr)(uintptr_t)((col ^ (64 * dt)) + o));
      const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_ptr)(uintptr_t)((col ^ (64 * dt + 32)) + o + 8 * K::ROWB));
      return cat(__builtin_bit_cast(bf16x4, lo), __builtin_bit_cast(bf16x4, hi));
    } else {
      f32v8 f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // 8 rows on flip bit 1 of the chunk, row j bits 2 and 3
        const uint32_t a = col ^ (128 * dt) ^ ((j & 3) * 64) ^ ((j >> 2) * 32);
        f.v[j] = at<float>(a, o + ((j >> 2) * 8 + (j & 3)) * K::ROWB);
      }
      return f;
    }
  }
};

// A column's accumulators as a row of a tensor.
template <typename T, int DP>
__device__ __forceinline__ void store_column(T* row, const f32x16 (&acc)[DP / 32], float scale,
                                             int D) {
  const int hh = lane_id() >> 5;
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int r = 0; r < 16; r += 4) {
      const int e = 32 * d + 2 * r + 4 * hh;
      const float v[4] = {acc[d][r] * scale, acc[d][r + 1] * scale, acc[d][r + 2] * scale,
                          acc[d][r + 3] * scale};
      if (e < D) store_row<T, 4>(row + e, v);
    }
}

// A wavefront's sums to LDS, and v = f0 v + f1 those of another.
template <int N>
__device__ __forceinline__ void put_sums(char* lds, int wave, const f32x16 (&v)[N]) {
  f32x4* to = (f32x4*)lds + wave * (N * 4 * 64) + lane_id();
#pragma unroll
  for (int d = 0; d < N; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      to[(d * 4 + r) * 64] = f32x4{v[d][4 * r], v[d][4 * r + 1], v[d][4 * r + 2], v[d][4 * r + 3]};
}
template <int N>
__device__ __forceinline__ void add_scaled_sums(const char* lds, int wave, f32x16 (&v)[N], float f0,
                                                float f1) {
  const f32x4* from = (const f32x4*)lds + wave * (N * 4 * 64) + lane_id();
#pragma unroll
  for (int d = 0; d < N; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const f32x4 x = from[(d * 4 + r) * 64];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[d][4 * r + i] = f0 * v[d][4 * r + i] + f1 * x[i];
    }
}

// The larger of a lane's value and its other half's.
__device__ __forceinline__ float max_halves(float v) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const unsigned x = s[0], y = s[1];
  return __builtin_fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y));
}

// Fragments along the head of one row in memory, zeros behind the head's D
// elements.
template <typename T, int DP>
__device__ __forceinline__ void load_row_frags(const T* row, int D,
                                               head_frag<T> (&f)[TileCfg<T, DP>::STEPS]) {
  using K = TileCfg<T, DP>;
  const int hh = lane_id() >> 5;
#pragma unroll
  for (int s = 0; s < K::STEPS; ++s) {
    const int e = (2 * s + hh) * K::E;
    f[s] = head_frag<T>{};
    if (e < D) f[s] = *(const head_frag<T>*)(row + e);
  }
}

// 16-byte direct-to-LDS load from a uniform base plus this lane's 32-bit
// offset; otherwise as dma16.  The wait states are those that a vector memory
// instruction needs behind a vector instruction that wrote its scalar base,
// which the compiler does not insert ahead of inline asm.
__device__ __forceinline__ void dma16_at(const void* base, uint32_t offset, uint32_t lds_base) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_base);
  const uint64_t a = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(offset), "s"((uint64_t)hi << 32 | lo), "{m0}"(m0)
               : "memory");
}

// Loads of ROWS rows of a tensor into an LDS tile by NT threads.
template <typename T, int DP, int ROWS, int NT>
struct Stager {
  using K = TileCfg<T, DP>;
  static constexpr int PER = ROWS * K::CH / NT;  // loads of a thread
  uint32_t off[PER];

  __device__ __forceinline__ static int row_of(int i, int thread) {
    return (i * NT + thread) / K::CH;
  }
  __device__ __forceinline__ static int chunk_of(int i, int thread) {
    return ((i * NT + thread) % K::CH) ^ swz<K::CH>(row_of(i, thread));
  }
  __device__ __forceinline__ Stager(int64_t stride, int thread) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      off[i] = (uint32_t)(row_of(i, thread) * (uint32_t)stride * (uint32_t)sizeof(T) +
                          chunk_of(i, thread) * 16);
  }
  // The rows from `at` on, all of them there.
  __device__ __forceinline__ void load(uint32_t lds, const T* at, int D, int thread) const {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (chunk_of(i, thread) * K::E < D)
        dma16_at(at, off[i], lds + ((i * NT + thread) & ~63) * 16);
  }
  // Rows r0 on of n (at least one); those behind the last are the last again:
  // finite values under weights of zero, and nothing behind the sequence is
  // read.  `last`: where row n - 1 stands if not with the others, else NULL.
  __device__ __forceinline__ static void load_tail(uint32_t lds, const T* base, int64_t stride,
                                                   int r0, int n, const T* last, int D,
                                                   int thread) {
    asm volatile("" : "+v"(thread));  // rare: nothing of it is kept in registers
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = chunk_of(i, thread), r = r0 + row_of(i, thread);
      const int at = r < n - 1 ? r : n - 1;
      const T* p = base + at * stride;
      if (last && at == n - 1) p = last;
      if (c * K::E < D) dma16(p + c * K::E, lds + ((i * NT + thread) & ~63) * 16);
    }
  }
};

// Clears a tile's chunks behind the head's end; loads never touch them.
template <typename T, int DP>
__device__ __forceinline__ void clear_ends(char* tile, int rows, int D, int thread, int threads) {
  using K = TileCfg<T, DP>;
  if (D == DP) return;
  for (int i = thread; i < rows * K::CH; i += threads) {
    const int r = i / K::CH, c = i % K::CH;
    if (c * K::E >= D) *(f32x4*)(tile + chunk_at<K::CH>(r, c)) = f32x4{};
  }
}

}  // namespace m2
