// Tiles, masks and matrix-core fragments shared by the jagged attention's
// forward and backward kernels.
//
// Fragments of v_mfma_f32_32x32x16 (lane = 32 g + c, g in {0, 1}):
//   A  row c,    k = 8 g + e,  e = 0..7      (16 bytes of one row)
//   B  column c, k = 8 g + e
//   C  column c, row 8 (i / 4) + 4 g + i % 4, i = 0..15
// A product's C holds, for a fixed column, rows 4 g .. 4 g + 3 of every
// group of 8. Read as the B operand of a second product over those rows,
// accumulators 8 s .. 8 s + 7 are k-slots of chunk s in the order
//   k-slot (g, e)  <->  row 16 s + 8 (e / 4) + 4 g + e % 4,
// and the sum over k does not care about the order as long as A uses the same.
// So probabilities go from the first product's accumulators to the second
// product's operand by rounding alone, with no shared memory and no shuffles,
// and A is read from a row-major tile with the transposing 8-byte LDS read
// (16 lanes read 4 rows x 16 columns, lane c receives column c's 4 rows).
#pragma once

#include <cmath>

#include "common.hpp"

namespace fs {
namespace attn {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// LDS tiles are filled and read in pieces of 16 bytes, their addresses formed
// by exclusive-or below that
constexpr int kTileAlign = 16;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 8 elements of either type travel as four 32-bit registers.
template <typename T>
struct Elem;
template <>
struct Elem<__bf16> {
  static constexpr bool kNarrow = false;  // of fewer exponents than fp32
  static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {  // to nearest even
    const f32x2 v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
  }
  static __device__ __forceinline__ f32x2 unpack(uint32_t u) {
    return __builtin_convertvector(__builtin_bit_cast(bf16x2, u), f32x2);
  }
};
template <>
struct Elem<_Float16> {
  static constexpr bool kNarrow = true;
  static __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float x, float y) {
    const f32x2 v = {x, y};
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
  }
  static __device__ __forceinline__ f32x2 unpack(uint32_t u) {
    return __builtin_convertvector(__builtin_bit_cast(f16x2, u), f32x2);
  }
};

// the wave's number, in a scalar register
__device__ __forceinline__ int wave_id() {
  return __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
}

__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t x = (uint64_t)p;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (const char*)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// accumulators 8 s .. 8 s + 7 as the B operand of chunk s
template <typename T>
__device__ __forceinline__ u32x4 to_operand(const f32x16& x, int s) {
  u32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = Elem<T>::pack(x[8 * s + 2 * e], x[8 * s + 2 * e + 1]);
  return r;
}

// the two lanes that hold one column's rows (c and c + 32): both get both
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float add_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// ---------------------------------------------------------------- LDS tiles
// A tile of rows of DP elements (2 bytes each; DP = 32, 64 or 128) without
// padding. The 16-byte pieces of a row are permuted by the row, so that both
// reads below meet every bank equally often (a row of 256 bytes spans the
// banks once): piece p of row r lies at p ^ swz(r).
//  - A read of one piece of 16 neighbouring rows should find 16 different
//    places in 256 bytes. Rows are 1, 2 or 4 to 256 bytes; the row's higher
//    bits choose among the pieces of its part.
//  - The transposing read takes 64 bytes of 4 neighbouring rows, which should
//    lie in 4 different quarters: the row's lowest bits go to the piece's
//    highest.
// Measured (forward, 4 x 8192 tokens, 4 heads of 128): with a permutation by
// three row bits 3.4e7 of 8.5e7 LDS cycles were bank conflicts, with this none.
template <int DP>
__device__ __forceinline__ int swz(int r) {
  if constexpr (DP == 32) return (r >> 2) & 3;
  if constexpr (DP == 64) return (r & 2) << 1 | ((r >> 2) & 3);
  return (r & 3) << 2 | ((r >> 2) & 3);
}

// piece p (8 elements) of row r, as an element offset
template <int DP>
__device__ __forceinline__ int piece(int r, int p) {
  return r * DP + ((p ^ swz<DP>(r)) << 3);
}

// The two operand reads. Rows enter as multiples of 16, which do not change
// the permutation, so what depends on the lane is one offset, and pieces
// differ from it by exclusive-or with constants.
template <int DP>
struct Operands {
  int rows_at, cols_at;
  __device__ __forceinline__ Operands() {
    const int l = lane(), g = l >> 5, j = l & 15;
    rows_at = piece<DP>(l & 31, g);
    const int col = (l & 16) + 4 * (j & 3);
    cols_at = piece<DP>(4 * g + (j >> 2), col >> 3) + (col & 7);
  }
  // A operand: rows r0 .. r0 + 31 (r0 a multiple of 32), elements 16 kk .. + 15
  __device__ __forceinline__ u32x4 rows(const uint16_t* tile, int r0, int kk) const {
    return *(const u32x4*)(tile + (rows_at ^ (16 * kk)) + r0 * DP);
  }
  // A operand of the transposed tile: its rows are the tile's columns c0 ..
  // c0 + 31, its k-slots the tile's rows r0 .. r0 + 15 in the order of
  // to_operand. Rows 8 apart differ in bit 1 of the permutation alone.
  __device__ __forceinline__ u32x4 cols(const uint16_t* tile, int r0, int c0) const {
    const uint16_t* a = tile + (cols_at ^ c0) + r0 * DP;
    const uint16_t* b = tile + (cols_at ^ c0 ^ 16) + (r0 + 8) * DP;
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)b));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
};

// ---------------------------------------------------------------- samples
// One tile of rows of one sample: rows t0 .. of the sample whose tokens start
// at lo; len tokens, of which the first hist are history.
struct Tile {
  int32_t lo, len, hist, t0;
};

// The table lists a sample's tiles by their rows to the sample's end (most
// first). The kernels that pass over the tokens before their rows take the
// mirrored tile: as many rows from the start.
__device__ __forceinline__ Tile tile_by_end(Tile t, int rows) {
  t.t0 = (t.len - 1) / rows * rows - t.t0;
  return t;
}

// A thread's rows of a staged tile lie less than 64 tokens behind a uniform
// address, so 32 bits hold their distance.
constexpr int64_t kMaxStride = (int64_t)1 << 26;

// Tiles of `rows` rows, the number of them on the device
struct TileTable {
  Tile* tiles;
  int32_t* n;
  int32_t rows;
};

// A [n_tok, heads, D] array: bytes between tokens and between heads
struct View {
  char* p;
  int64_t tok, head;
};

struct Shape {
  TileTable tab;
  const uint8_t* valid;  // nullable
  int64_t n_tok;
  int32_t heads;         // query heads
  int32_t group;         // query heads per key head
  int32_t pack;          // query heads per workgroup, see pack_of
  int32_t dim;           // elements of a head, at most DP
  int32_t causal;
  float scale;           // of the scores
};

__device__ __forceinline__ bool live_row(const Shape& a, const Tile& t, int r) {
  if (r >= t.len) return false;
  return a.valid == nullptr || a.valid[(int64_t)t.lo + r] != 0;
}

// the lowest n bits (n may lie outside 0..32)
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? ~0u : ((1u << n) - 1u));
}
__device__ __forceinline__ uint32_t one_bit(int n) { return n >= 0 && n < 32 ? 1u << n : 0u; }

// keys j0 .. j0 + 31 that row i sees: the history, up to itself where causal,
// and itself
__device__ __forceinline__ uint32_t seen_keys(int i, int j0, int hist, bool causal) {
  const int lim = causal ? min(hist, i + 1) : hist;
  return low_bits(lim - j0) | one_bit(i - j0);
}
// rows i0 .. i0 + 31 that see key j
__device__ __forceinline__ uint32_t seeing_rows(int j, int i0, int hist, bool causal) {
  const uint32_t self = one_bit(j - i0);
  if (j >= hist) return self;
  return causal ? ~low_bits(j - i0) : ~0u;
}

// 16 bytes of row r of one head, elements 8 p .. 8 p + 7. A row past the
// sample loads its last one and a piece past the head's width the first, so
// that no load waits for a condition.
__device__ __forceinline__ u32x4 load_piece(const char* head, int64_t tok_bytes, const Shape& a,
                                            const Tile& t, int r, int p) {
  return *(const u32x4*)(head + ((int64_t)t.lo + min(r, t.len - 1)) * tok_bytes +
                         (8 * p < a.dim ? 16 * p : 0));
}

// Which rows r0 .. r0 + 63 of a sample exist and are valid, one row per lane,
// and as bits.
__device__ __forceinline__ uint32_t live_byte(const Shape& a, const Tile& t, int r0) {
  const int r = r0 + lane();
  if (r >= t.len) return 0;
  return a.valid == nullptr ? 1 : a.valid[(int64_t)t.lo + r];
}
__device__ __forceinline__ uint64_t live_bits(uint32_t byte) { return __ballot(byte != 0); }

// A tile of 64 rows on its way from memory to LDS, NT threads: load() lets
// memory write to LDS as it arrives (no registers hold it in between), finish()
// puts zeros in the place of what is not live or lies past the head's width.
// Rows past the sample load its last one and pieces past the width the first,
// so every load is in bounds and none is conditional. A wave's load fills 1024
// bytes of LDS in the order of its lanes, so a lane loads the piece that
// belongs at its place. Measured against a passage through registers: forward
// 327 -> 290 us, backward 1197 -> 1036 us on long samples with heads of 128.
// The instruction is written out because the compiler otherwise waits
// for it before the next read of any LDS, which is where the other tile's
// products start: wait() is the one wait, before the barrier that lets the
// tile be read, and nothing reads or writes the tile between load() and that.
template <int DP, int NT>
struct Direct {
  static constexpr int kRows = 64;
  static constexpr int kPieces = DP / 8;
  static constexpr int kPer = kRows * kPieces / NT;
  static constexpr int kStepRows = NT / kPieces;
  static_assert(kPer >= 1 && kRows * kPieces % NT == 0, "whole pieces per thread");
  static_assert(kStepRows % 16 == 0, "a thread's rows share the permutation");

  static __device__ __forceinline__ int piece_of() {
    return ((int)threadIdx.x % kPieces) ^ swz<DP>(threadIdx.x / kPieces);
  }
  // 16 bytes per lane from base + at to LDS address `to` + 16 lane; base and
  // `to` are uniform. The instruction takes `to` from M0, one idle cycle after it
  // is written. The compiler does not let an asm declare that it changes M0, so
  // what was there is put back.
  static __device__ __forceinline__ void load16(const char* base, uint32_t at, uint32_t to) {
    uint32_t m0;
    asm volatile(
        "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(m0)
        : "s"(to), "v"(at), "s"(base)
        : "memory");
  }
  static __device__ __forceinline__ void load(uint16_t* tile, const char* head, int64_t tok_bytes,
                                              const Shape& a, const Tile& t, int r0) {
    typedef __attribute__((address_space(3))) uint16_t* lds_ptr;
    const int row = threadIdx.x / kPieces, p = piece_of();
    const char* base = uniform(head + ((int64_t)t.lo + r0) * tok_bytes);
    const uint32_t to = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(lds_ptr)tile + threadIdx.x / kWave * (kWave * 16));
    if (r0 + kRows <= t.len && a.dim == DP) {
      const uint32_t at = (uint32_t)row * (uint32_t)tok_bytes + 16 * p;
#pragma unroll
      for (int x = 0; x < kPer; ++x)
        load16(uniform(base + (int64_t)x * kStepRows * tok_bytes), at, to + x * NT * 16);
    } else {
      const int last = t.len - 1 - r0, pc = 8 * p < a.dim ? 16 * p : 0;
#pragma unroll
      for (int x = 0; x < kPer; ++x)
        load16(base, (uint32_t)min(row + x * kStepRows, last) * (uint32_t)tok_bytes + pc,
               to + x * NT * 16);
    }
  }
  // before the barrier that lets the tile be read, after wait()
  static __device__ __forceinline__ void finish(uint16_t* tile, const Shape& a, uint64_t live) {
    if (live == ~0ull && a.dim == DP) return;
    const int row = threadIdx.x / kPieces;
    const bool in = 8 * piece_of() < a.dim;
#pragma unroll
    for (int x = 0; x < kPer; ++x)
      if (!in || !((live >> (row + x * kStepRows)) & 1))
        *(u32x4*)(tile + (x * NT + threadIdx.x) * 8) = u32x4{0, 0, 0, 0};
  }
  static __device__ __forceinline__ void wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
};

// What a score of each key of a tile starts from: 0, or -inf for keys that
// are not live. In the scores' accumulators keys run down the rows, so both
// halves of the wave read theirs as they are, and no score is masked later.
__device__ __forceinline__ void store_off(float* off, uint64_t live) {
  if (threadIdx.x < 64) off[threadIdx.x] = (live >> threadIdx.x) & 1 ? 0.f : -INFINITY;
}
__device__ __forceinline__ f32x16 load_off(const float* off, int k0) {
  const int g = lane() >> 5;
  f32x16 r;
#pragma unroll
  for (int y = 0; y < 4; ++y) {
    const f32x4 x = *(const f32x4*)(off + k0 + 8 * y + 4 * g);
#pragma unroll
    for (int z = 0; z < 4; ++z) r[4 * y + z] = x[z];
  }
  return r;
}

// B operands of 32 rows of one head: column c = row r0 + c. Rows that are not
// live bring whatever memory holds: a column of a product depends on no other
// column, and those of such rows are cleared before they are stored. Pieces
// past the width meet zeros of the staged tile.
template <int DP>
__device__ __forceinline__ void load_columns(u32x4 (&f)[DP / 16], const char* head,
                                             int64_t tok_bytes, const Shape& a, const Tile& t,
                                             int r) {
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk)
    f[kk] = load_piece(head, tok_bytes, a, t, r, 2 * kk + (lane() >> 5));
}

// The kernels scale scores by a positive number (a maximum may be scaled
// after it is taken, and a masked score stays -inf). The sign of `scale` goes
// into one operand of S, and a scale of 0 makes that operand zero.
template <int DP>
__device__ __forceinline__ void load_scaled_columns(u32x4 (&f)[DP / 16], const char* head,
                                                    int64_t tok_bytes, const Shape& a,
                                                    const Tile& t, int r) {
  load_columns<DP>(f, head, tok_bytes, a, t, r);
  if (a.scale <= 0.f) {
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) f[kk] = a.scale < 0.f ? f[kk] ^ 0x80008000u : f[kk] & 0u;
  }
}
__device__ __forceinline__ float log2_scale(const Shape& a) {
  return a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
}

// ---------------------------------------------------------------- host side
__host__ inline bool type_ok(int32_t dtype) { return dtype == FS_BF16 || dtype == FS_F16; }

// Exponents are scaled by scale log2(e), which has to be finite too: 0 times an
// infinity is no score.
__host__ inline bool scale_ok(float scale) { return std::isfinite(scale * kLog2e); }

// the width of the kernel's rows for heads of dim elements
__host__ inline int32_t padded(int32_t dim) { return dim <= 32 ? 32 : (dim <= 64 ? 64 : 128); }

// tiles of `rows` rows that n samples of n_tok tokens can need
__host__ inline int64_t tile_cap(int64_t n_tok, int32_t n, int32_t rows) { return n_tok / rows + n; }

// checks of one argument array; dense strides filled in
__host__ int make_view(const fs_heads* x, int32_t heads, int32_t dim, View* v);

// Query heads that one workgroup of the forward and the dQ kernel takes: its
// four waves share key tiles, so they may as well be four heads of one key
// head over 32 rows as one head over 128. Heads leave no wave without rows at
// a sample's end and none waiting at the diagonal. Measured on 128 samples of
// 428 tokens on average, 8/2 heads of 64, forward: one head 90 us, four 83;
// on samples of 8192 tokens both the same.
__host__ inline int32_t pack_of(int32_t group) { return group % 4 == 0 ? 4 : (group % 2 == 0 ? 2 : 1); }

// Fills one or two tables (see attention.hip).
int launch_tiles(const int64_t* offsets, int32_t n, int64_t n_tok, const int32_t* n_cand,
                 int32_t causal, const TileTable* t, int32_t tables, int32_t* err,
                 hipStream_t stream);

}  // namespace attn
}  // namespace fs
