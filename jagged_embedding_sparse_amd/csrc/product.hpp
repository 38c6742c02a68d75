// Tile products of 16-bit matrices on the matrix cores: a workgroup's waves compute
// out[n][m] = sum over k of A(m, k) B(n, k) for BM columns m and BN rows n of the
// output, with fp32 sums in registers.
//
// An operand lies in memory in one of two ways: Rows, its row m (or n) holding
// the k's one after another, or Cols, its row k holding the m's. Either travels
// to LDS as it lies, 64 k's a step, without registers, and is read into the
// layout of v_mfma_f32_32x32x16 (see attention.hpp): a row's 16 bytes for Rows,
// two transposing 8-byte reads for Cols. Pieces of 16 bytes are permuted by
// exclusive-or with bits of the row so that neither read meets a bank twice.
//
// The pipeline: two stages in LDS. A step has four chunks of 16 k's; the next
// chunk's operands are read while this one's products run, and the one barrier
// of a step stands before its last chunk's products, which cover the first reads
// of the next stage. Loads are asked for right behind the barrier, a whole step
// before they are waited for.
//
// Measured (256 x 256, eight waves, K = 32768, 16384 x 1024 sums, bf16): 845 to 884 us by
// card, 1245 to 1300 TFLOP/s, the matrix units busy 70% of the time at a clock that the card has
// brought down from 2.4 to 1.7 GHz, so what bounds it is power. A library product of these
// shapes reaches 960 to 1070, one of 8192^3 1380 to 1410. Four waves of 128 x 128 instead of
// eight of 128 x 64 do not fit the registers (737 against 613 us for 16384 x 16384 x
// 1024); left to the compiler's order of reads and products, 470 against 458.
#pragma once

#include <type_traits>

#include "attention.hpp"

namespace fs {
namespace prod {

using attn::Elem;
using attn::f32x16;
using attn::f32x4;
using attn::u32x2;
using attn::u32x4;

constexpr int kK = 64;        // k's of a step

typedef __attribute__((address_space(3))) uint16_t* lds_ptr;

// A value that the compiler takes for new each time, so that what follows from it
// is not kept in registers over a loop.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// 16 bytes per lane from base + at to LDS address `to` + 16 lane. M0 is put back:
// the compiler does not let an asm declare that it changes it.
__device__ __forceinline__ void load_piece(const char* base, uint32_t at, uint32_t to) {
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(m0)
      : "s"(to), "v"(at), "s"(base)
      : "memory");
}

// the same for 4 bytes per lane
__device__ __forceinline__ void load_words(const void* base, uint32_t at, uint32_t to) {
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, %3\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(m0)
      : "s"(to), "v"(at), "s"(base)
      : "memory");
}

// A operand reads of a tile in LDS: rows r0 .. r0 + 31 (r0 a multiple of 32), k's
// 16 kk + 8 g .. of a tile of rows of 64 k's,
struct ReadRows {
  int rows_at;
  __device__ __forceinline__ ReadRows() { rows_at = attn::piece<kK>(lane() & 31, lane() >> 5); }
  __device__ __forceinline__ u32x4 operator()(const uint16_t* tile, int r0, int kk) const {
    return *(const u32x4*)(tile + (rows_at ^ (16 * kk)) + r0 * kK);
  }
};
// columns c0 .. c0 + 31 (a multiple of 32) of a tile of 64 rows of R elements.
template <int R>
constexpr int kColsSwz = R == 64 ? 64 : 128;
template <int R>
struct ReadCols {
  int cols_at;
  __device__ __forceinline__ ReadCols() {
    // rows 8 g + j / 4 and 4 more (the permutation of those differs in bit 0)
    const int l = lane(), g = l >> 5, j = l & 15, col = (l & 16) + 4 * (j & 3), row = 8 * g + (j >> 2);
    cols_at = row * R + 8 * ((col >> 3) ^ attn::swz<kColsSwz<R>>(row)) + (col & 7);
  }
  __device__ __forceinline__ u32x4 operator()(const uint16_t* tile, int c0, int kk) const {
    const uint16_t* a = tile + (cols_at ^ c0) + 16 * kk * R;
    const uint16_t* b = tile + (cols_at ^ c0 ^ 8) + (16 * kk + 4) * R;
    const u32x2 lo = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((attn::lds_s16x4*)a));
    const u32x2 hi = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((attn::lds_s16x4*)b));
    return u32x4{lo[0], lo[1], hi[0], hi[1]};
  }
};

// k's together: a tile of R rows and 64 k's, rows of 128 bytes.
template <int R, int NT>
struct Rows {
  static constexpr int kElems = R * kK;
  static constexpr int kPer = R * 8 / NT;  // loads of a thread
  static_assert(kPer >= 1 && R * 8 % NT == 0, "whole pieces per thread");
  const char* base;  // of the tile's first row, at the next step's first k
  uint32_t at[kPer];
  uint32_t row_bytes;
  int32_t last;

  static __device__ __forceinline__ int row_of(int x, int t) { return x * (NT / 8) + t / 8; }
  static __device__ __forceinline__ int piece_of(int t) { return (t % 8) ^ attn::swz<kK>(t / 8); }
  // rows row0 .. of `rows` rows; rows past the last load it again
  __device__ __forceinline__ Rows(const char* p, int64_t stride, int64_t row0, int64_t rows, int64_t k0) {
    base = attn::uniform(p + row0 * stride + k0 * 2);
    row_bytes = (uint32_t)stride;
    last = (int32_t)min((int64_t)R, rows - row0) - 1;
    limit(kK);
  }
  // pieces of k's past `left` load the step's first
  __device__ __forceinline__ void limit(int left) {
    const int t = here(threadIdx.x), p = 8 * piece_of(t) < left ? piece_of(t) : 0;
#pragma unroll
    for (int x = 0; x < kPer; ++x) at[x] = (uint32_t)min(row_of(x, t), last) * row_bytes + 16 * p;
  }
  // piece x of the next step's tile; then the step after it
  __device__ __forceinline__ void load(uint32_t tile, int x) const {
    load_piece(base, at[x], tile + attn::wave_id() * (kWave * 16) + x * NT * 16);
  }
  __device__ __forceinline__ void advance() { base = attn::uniform(base + kK * 2); }
  using Read = ReadRows;
};

// k's apart: a tile of 64 k's, rows of R elements. Piece p of row r lies at
// p ^ ((r & 3) << 2 | (r >> 2) & 3), of rows of 128 bytes at p ^ ((r & 2) << 1 |
// (r >> 2) & 3): see attention.hpp.
template <int R, int NT, int Hold = 1>
struct Cols {
  static constexpr int kElems = R * kK;
  static constexpr int kPieces = R / 8;
  static constexpr int kPer = R * 8 / NT;
  static constexpr int kStepRows = NT / kPieces;
  static_assert(kPer >= 1 && R * 8 % NT == 0 && NT % kPieces == 0, "whole rows per step");
  const char* base;  // of the next step's first row, at the tile's first column
  uint32_t at[kPer];
  uint32_t row_bytes;
  int32_t cols, turn = 0;  // a step's tile is loaded Hold times

  static __device__ __forceinline__ int row_of(int x) { return x * kStepRows + (int)threadIdx.x / kPieces; }
  static __device__ __forceinline__ int piece_of(int x) {
    return ((int)threadIdx.x % kPieces) ^ attn::swz<kColsSwz<R>>(row_of(x));
  }
  // columns col0 .. of `cols_` (a multiple of 8); pieces past the last load the tile's first
  __device__ __forceinline__ Cols(const char* p, int64_t stride, int64_t col0, int64_t cols_, int64_t k0) {
    base = attn::uniform(p + k0 * stride + col0 * 2);
    row_bytes = (uint32_t)stride;
    cols = (int32_t)min((int64_t)R, cols_ - col0);
    limit(kK);
  }
  // rows past `left` load the step's first
  __device__ __forceinline__ void limit(int left) {
#pragma unroll
    for (int x = 0; x < kPer; ++x)
      at[x] = (row_of(x) < left ? (uint32_t)row_of(x) * row_bytes : 0u) +
              (8 * piece_of(x) < cols ? 16 * piece_of(x) : 0);
  }
  __device__ __forceinline__ void load(uint32_t tile, int x) const {
    load_piece(base, at[x], tile + attn::wave_id() * (kWave * 16) + x * NT * 16);
  }
  __device__ __forceinline__ void advance() {
    if (Hold > 1 && ++turn < Hold) return;
    turn = 0;
    base = attn::uniform(base + (int64_t)kK * row_bytes);
  }
  using Read = ReadCols<R>;
};

// Matrices of this library's own making lie in blocks of 64 x 64, a block's rows
// one after another, so that what a step loads is a few runs of 8 KiB: whole rows
// of a power of two apart would meet the same memory channels. Both kinds of tile
// load from blocks; rows and columns are padded to whole blocks.
constexpr int kBlock = kK * kK;  // elements

__host__ __device__ __forceinline__ int64_t blocked(int64_t row, int64_t col, int64_t cols) {
  return (row / kK * (cols / kK) + col / kK) * kBlock + row % kK * kK + col % kK;
}

template <int R, int NT>
struct BlockRows {
  static constexpr int kElems = R * kK;
  static constexpr int kPer = R * 8 / NT;
  static_assert(kPer >= 1 && R * 8 % NT == 0, "whole pieces per thread");
  const char* base;
  uint32_t at[kPer];
  // row0 and k0: multiples of 64
  __device__ __forceinline__ BlockRows(const char* p, int64_t cols, int64_t row0, int64_t k0) {
    base = attn::uniform(p + 2 * blocked(row0, k0, cols));
    const int piece = ((int)threadIdx.x % 8) ^ attn::swz<kK>((int)threadIdx.x / 8);
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int row = x * (NT / 8) + (int)threadIdx.x / 8;
      at[x] = (uint32_t)(row / kK) * (uint32_t)(cols * kK * 2) + row % kK * (kK * 2) + 16 * piece;
    }
  }
  __device__ __forceinline__ void limit(int) {}
  __device__ __forceinline__ void load(uint32_t tile, int x) const {
    load_piece(base, at[x], tile + attn::wave_id() * (kWave * 16) + x * NT * 16);
  }
  __device__ __forceinline__ void advance() { base = attn::uniform(base + kBlock * 2); }
  using Read = ReadRows;
};

// Hold: a step's tile is loaded so often. Parts: a block of columns is so many
// blocks beside each other, of which a step takes one (the parts of a sum of
// matrices, a step of each in turn).
template <int R, int NT, int Hold = 1, int Parts = 1>
struct BlockCols {
  static constexpr int kElems = R * kK;
  static constexpr int kPieces = R / 8, kPer = R * 8 / NT;
  static_assert(kPer >= 1 && R * 8 % NT == 0 && NT % kPieces == 0, "whole rows per step");
  static_assert(Hold == 1 || Parts == 1, "one or the other");
  const char* base;
  uint32_t at[kPer];
  int64_t step;
  int32_t turn = 0;
  // col0 and k0: multiples of 64; columns past `cols` are the tile's first block again
  __device__ __forceinline__ BlockCols(const char* p, int64_t cols, int64_t col0, int64_t k0) {
    base = attn::uniform(p + 2 * blocked(k0, col0 * Parts, cols * Parts));
    step = cols * Parts * kK * 2;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int row = x * (NT / kPieces) + (int)threadIdx.x / kPieces;
      const int piece = ((int)threadIdx.x % kPieces) ^ attn::swz<kColsSwz<R>>(row);
      const int block = col0 + 8 * piece < cols ? piece / 8 * Parts : 0;
      at[x] = block * (kBlock * 2) + row * (kK * 2) + 16 * (piece % 8);
    }
  }
  __device__ __forceinline__ void limit(int) {}
  __device__ __forceinline__ void load(uint32_t tile, int x) const {
    load_piece(base, at[x], tile + attn::wave_id() * (kWave * 16) + x * NT * 16);
  }
  __device__ __forceinline__ void advance() {
    if (Hold > 1 && ++turn < Hold) return;
    if (Parts > 1 && ++turn < Parts) {
      base = attn::uniform(base + kBlock * 2);
      return;
    }
    turn = 0;
    base = attn::uniform(base + step - (Parts - 1) * (kBlock * 2));
  }
  using Read = ReadCols<R>;
};

// (Turns: 64 k's are so many steps, with another part of one operand each.)
// WM x WN waves, each of MI x NI blocks of 32 x 32. Register i of a lane's block
// (mi, ni) is column m = m_of(mi) + 8 (i / 4) + i % 4 of row n = n_of(ni).
// Stages: tiles of so many steps fit LDS, so the loads of all but one are in flight.
template <typename T, typename A, typename B, int BM, int BN, int WM, int WN, int Turns = 1, int Stages = 2>
struct Tile {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int MI = BM / WM / 32, NI = BN / WN / 32;
  static constexpr int kStage = (BM + BN) * kK;  // elements
  static_assert(MI >= 1 && NI >= 1, "whole blocks");
  f32x16 acc[MI][NI];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = attn::zero16();
  }
  static __device__ __forceinline__ int m_of(int mi, int l = lane()) {
    return (attn::wave_id() % WM * MI + mi) * 32 + 4 * (l >> 5);
  }
  static __device__ __forceinline__ int n_of(int ni, int l = lane()) {
    return (attn::wave_id() / WM * NI + ni) * 32 + (l & 31);
  }

  struct Operands {
    u32x4 a[MI], b[NI];
  };
  // operand x of a chunk, in the order in which the products ask for them
  static constexpr int kOperands = MI + NI, kProducts = MI * NI, kLoads = A::kPer + B::kPer;
  __device__ __forceinline__ void read(Operands& o, const typename A::Read& ra, const typename B::Read& rb,
                                       const uint16_t* stage, int kk, int x) const {
    const int w = attn::wave_id();
    if (x > 0 && x <= NI) o.b[x - 1] = rb(stage + BM * kK, (w / WM * NI + x - 1) * 32, kk);
    else o.a[x ? x - NI : 0] = ra(stage, (w % WM * MI + (x ? x - NI : 0)) * 32, kk);
  }
  __device__ __forceinline__ void multiply(const Operands& o, int x) {
    acc[x / NI][x % NI] = Elem<T>::mfma(o.a[x / NI], o.b[x % NI], acc[x / NI][x % NI]);
  }

  // Asks for the first 64 of `k` k's, from where a and b stand. The first stage
  // must be free; run() may follow after other work that leaves it alone (with more
  // than two stages that work has stored nothing: loads are counted, stores are not).
  template <bool LimA, bool LimB>
  static __device__ __forceinline__ void ask(A& a, B& b, int64_t k, uint16_t* lds) {
    if (k > 0) ask_step<LimA, LimB>(a, b, k, 0, lds_address(lds));
  }

  // Adds the product over `k` k's in steps of 64, behind ask(); in the last step the
  // operands are told how many are left where Lim says so. lds: Stages kStage
  // elements. They are free again when it returns, all but the first before it begins.
  //
  // Products, reads and loads are issued in this order and no other (left to
  // itself the compiler reads a chunk's operands right before its products and
  // waits for them there).
  template <bool LimA, bool LimB>
  __device__ __forceinline__ void run(A& a, B& b, int64_t k, uint16_t* lds) {
    const typename A::Read ra;
    const typename B::Read rb;
    const uint32_t lds0 = lds_address(lds);
    const int steps = (int)cdiv(k, (int64_t)kK) * Turns;
    if (steps <= 0) return;
    if constexpr (Stages == 2) landed();
#pragma unroll
    for (int t = 1; t < Stages; ++t)
      if (t < steps) ask_step<LimA, LimB>(a, b, k, t, lds0 + t * (kStage * 2));
    if constexpr (Stages > 2) {
      if (steps >= Stages) landed<(Stages - 1) * kLoads>();
      else landed();
    }
    Operands o[2];
#pragma unroll
    for (int x = 0; x < kOperands; ++x) read(o[0], ra, rb, lds, 0, x);
    constexpr int kMost = kProducts > kOperands ? kProducts : kOperands;
    // one step on stage `buf`; the one behind it holds the next step's tiles
    int buf = 0;
    auto step = [&](auto more) {
      const uint16_t* here = lds + buf * kStage;
      const int then = Stages == 2 ? buf ^ 1 : buf + 1 < Stages ? buf + 1 : 0;
      const uint16_t* next = lds + then * kStage;
#pragma unroll
      for (int kk = 0; kk < 3; ++kk)
#pragma unroll
        for (int x = 0; x < kMost; ++x) {
          if (x < kOperands) read(o[(kk + 1) & 1], ra, rb, here, kk + 1, x);
          if (x < kProducts) multiply(o[kk & 1], x);
          __builtin_amdgcn_sched_barrier(0);
        }
      // the last chunk's operands are here, so this stage may be written again; of the
      // loads, those of the next step are
      landed<decltype(more)::value ? (Stages - 2) * kLoads : 0>();
#pragma unroll
      for (int x = 0; x < kLoads || x < kMost; ++x) {
        if (x < kOperands) read(o[0], ra, rb, next, 0, x);  // behind the last step: of no use
        if (more && x < kLoads) load(a, b, lds0 + buf * (kStage * 2), x);
        if (x < kProducts) multiply(o[1], x);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (more) {
        a.advance();
        b.advance();
      }
      buf = then;
    };
    int t = 0;
    for (; t + Stages < steps; ++t) {
      limit<LimA, LimB>(a, b, k, t + Stages);
      step(std::true_type());
    }
    for (; t < steps; ++t) step(std::false_type());
    landed();
  }

  static __device__ __forceinline__ uint32_t lds_address(uint16_t* lds) {
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_ptr)lds);
  }
  template <bool LimA, bool LimB>
  static __device__ __forceinline__ void limit(A& a, B& b, int64_t k, int step) {
    const int64_t k0 = step / Turns * (int64_t)kK;
    if ((LimA || LimB) && k0 + kK > k) {
      if (LimA) a.limit((int)(k - k0));
      if (LimB) b.limit((int)(k - k0));
    }
  }
  static __device__ __forceinline__ void load(const A& a, const B& b, uint32_t stage, int x) {
    if (x < A::kPer) a.load(stage, x);
    else b.load(stage + BM * kK * 2, x - A::kPer);
  }
  template <bool LimA, bool LimB>
  static __device__ __forceinline__ void ask_step(A& a, B& b, int64_t k, int step, uint32_t stage) {
    limit<LimA, LimB>(a, b, k, step);
#pragma unroll
    for (int x = 0; x < kLoads; ++x) load(a, b, stage, x);
    a.advance();
    b.advance();
  }

  // every wave's loads but its last `Flying` have landed (loads land in order) and
  // every wave's reads of LDS are done
  template <int Flying = 0>
  static __device__ __forceinline__ void landed() {
    static_assert(Flying < 64, "what the counter holds");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"i"(Flying) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }
};

// LDS written before it is read behind it; loads in flight stay in flight
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------- output
// Rows of a tile pass through LDS so that memory sees whole rows: 4 neighbouring
// columns of a lane are 8 (16-bit) or 16 bytes (fp32), and a row's 16-byte pieces
// are permuted by the row, so neither side meets a bank twice.
//
// put(n, m, v): columns m .. m + 3 of row n of the staged rows; at: a thread's
// pieces in turn.
template <int BM>
struct Stage16 {  // rows of BM elements of 2 bytes
  static constexpr int kPieces = BM / 8;
  static __device__ __forceinline__ void put(uint16_t* lds, int n, int m, u32x2 v) {
    const int p = (m >> 3) ^ (n & (kPieces - 1));
    *(u32x2*)(lds + n * BM + 8 * p + (m & 7)) = v;
  }
  static __device__ __forceinline__ void put1(uint16_t* lds, int n, int m, uint32_t v) {
    lds[n * BM + 8 * ((m >> 3) ^ (n & (kPieces - 1))) + (m & 7)] = (uint16_t)v;
  }
  static __device__ __forceinline__ u32x4 get(const uint16_t* lds, int n, int piece) {
    return *(const u32x4*)(lds + n * BM + 8 * (piece ^ (n & (kPieces - 1))));
  }
};
template <int BM>
struct Stage32 {  // rows of BM floats
  static constexpr int kPieces = BM / 4;
  static __device__ __forceinline__ void put(float* lds, int n, int m, f32x4 v) {
    *(f32x4*)(lds + n * BM + 4 * ((m >> 2) ^ (n & (kPieces - 1)))) = v;
  }
  static __device__ __forceinline__ f32x4 get(const float* lds, int n, int piece) {
    return *(const f32x4*)(lds + n * BM + 4 * (piece ^ (n & (kPieces - 1))));
  }
};

// Elements at any alignment, 16 bytes at a time where they are whole.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// Order of a grid's tiles: XCD x runs an eighth of them in a row, and inside
// that blocks of `group` row tiles go by column tile, so that the tiles of an XCD
// at one time share operands in its L2.
struct Order {
  int32_t rows, cols;  // tiles
  __device__ __forceinline__ void at(int32_t id, int32_t group, int32_t* row, int32_t* col) const {
    const int32_t whole = rows / group * group * cols;
    if (id < whole) {
      const int32_t block = group * cols, b = id / block, r = id % block;
      *row = b * group + r % group;
      *col = r / group;
    } else {
      const int32_t left = rows % group, r = id - whole;
      *row = rows / group * group + r % left;
      *col = r / left;
    }
  }
};
// workgroup to position: neighbours in order on one XCD
__device__ __forceinline__ int32_t in_order(int32_t bid, int32_t n) {
  const int32_t per = n / kXcd, cut = n % kXcd, x = bid % kXcd, i = bid / kXcd;
  return x < cut ? x * (per + 1) + i : cut * (per + 1) + (x - cut) * per + i;
}

}  // namespace prod
}  // namespace fs
