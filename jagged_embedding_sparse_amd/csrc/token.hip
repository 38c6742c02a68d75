// Token embedding: scaled lookup of a vocabulary's rows, and the gradient of
// the rows by the sorted tokens (token_sort.hip).
//
//   out[i] = scale w[ids[i]]        g[v] = scale sum over i with ids[i] = v of dout[i]
#include <algorithm>

#include "common.hpp"
#include "divu32.hpp"

namespace fs {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// ---------------------------------------------------------------- elements
template <typename T>
struct Num;
template <>
struct Num<float> {
  static __device__ __forceinline__ float up(float x) { return x; }
  static __device__ __forceinline__ float down(float x) { return x; }
};
template <>
struct Num<__bf16> {
  static __device__ __forceinline__ float up(__bf16 x) { return (float)x; }
  static __device__ __forceinline__ __bf16 down(float x) { return (__bf16)x; }
};
template <>
struct Num<_Float16> {
  static __device__ __forceinline__ float up(_Float16 x) { return (float)x; }
  static __device__ __forceinline__ _Float16 down(float x) { return (_Float16)x; }
};

// A 64-bit sum to a table's type in one rounding. To 16 bits it goes by way of
// fp32 rounded to odd: where fp32 is not exact, its last bit is set, 13 bits or
// more below the 16-bit type's, so that a sum beside a midpoint stays on its side
// of it. Infinities and NaN stay.
template <typename T>
__device__ __forceinline__ T round_sum(double x) {
  const float f = (float)x;
  if constexpr (sizeof(T) == 4) {
    return f;
  } else {
    const double back = fabs((double)f), size = fabs(x);
    uint32_t u = __float_as_uint(f);
    if (!(u & 1)) u += size > back ? 1 : (size < back ? -1 : 0);
    return Num<T>::down(__uint_as_float(u));
  }
}

template <typename T>
struct Pair {
  T a, b;
};

// N elements of a row. Rows may start anywhere an element may: global accesses
// of 4, 8 and 16 bytes need no alignment on this hardware, so odd widths and
// strides take the same wide accesses as even ones.
template <typename T, int N>
struct Pack {
  T v[N];
};

// Streams past the caches: written once, read by nobody soon, and not in the
// way of the rows that the caches hold. Measured: a lookup of 200003 rows of
// 636 (fp32 to bf16) 125 -> 71 us.
template <typename P>
__device__ __forceinline__ void put_through(P* to, const P& v) {
  typedef u32x4 v4 __attribute__((aligned(2)));
  typedef u32x2 v2 __attribute__((aligned(2)));
  if constexpr (sizeof(P) == 32) {
    const auto x = __builtin_bit_cast(Pair<u32x4>, v);
    __builtin_nontemporal_store(x.a, (v4*)to);
    __builtin_nontemporal_store(x.b, (v4*)to + 1);
  } else if constexpr (sizeof(P) == 16) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), (v4*)to);
  } else if constexpr (sizeof(P) == 8) {
    __builtin_nontemporal_store(__builtin_bit_cast(u32x2, v), (v2*)to);
  } else {
    *to = v;
  }
}

// ---------------------------------------------------------------- lookup
struct TokLookupArgs {
  const char* table;
  const int64_t* ids;
  char* out;
  int32_t* err;
  int64_t n, rows, in_stride, out_stride;
  float scale;
  int32_t dim;
  int32_t pieces;          // pieces of a row; the last may overlap the one before
  int32_t rows_per_block;
  DivU32 by_pieces;
};

constexpr int kLookupPer = 4;  // pieces per thread
constexpr int64_t kLookupBlocks = (int64_t)1 << 23;  // workgroups at most

// A workgroup takes rows_per_block tokens; its threads run over the pieces
// (N elements) of their rows, all of a thread's pieces in flight. Bound by HBM:
// the kernel takes 15.6 us for 32768 x 1024 bf16 and 71.5 for 200003 x 636 fp32
// to bf16, where copying the same bytes (each distinct row read once) takes 16.8
// and 70.8; 1.7 us for one token of 2048.
template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(kThreads) k_token_lookup(TokLookupArgs a) {
  const int64_t i0 = (int64_t)blockIdx.x * a.rows_per_block;
  const int32_t nr = (int32_t)min((int64_t)a.rows_per_block, a.n - i0);
  const uint32_t total = (uint32_t)nr * a.pieces;
  for (uint32_t base = 0; base < total; base += kThreads * kLookupPer) {  // uniform
    Pack<TI, N> x[kLookupPer];
    int64_t to[kLookupPer];
    bool bad = false;
#pragma unroll
    for (int u = 0; u < kLookupPer; ++u) {
      const uint32_t id = base + u * kThreads + threadIdx.x;
      to[u] = -1;
#pragma unroll
      for (int e = 0; e < N; ++e) x[u].v[e] = (TI)0.f;
      if (id < total) {
        const uint32_t r = divu32(id, a.by_pieces);
        const int32_t col = min((int32_t)(id - r * a.pieces) * N, a.dim - N);
        const int64_t row = a.ids[i0 + r];
        to[u] = (i0 + r) * a.out_stride + col * (int64_t)sizeof(TO);
        if (row >= 0 && row < a.rows)
          x[u] = *(const Pack<TI, N>*)(a.table + row * a.in_stride + col * (int64_t)sizeof(TI));
        else
          bad = true;
      }
    }
    flag_err(a.err, bad, FS_EF_ID_RANGE);
#pragma unroll
    for (int u = 0; u < kLookupPer; ++u) {
      if (to[u] < 0) continue;
      Pack<TO, N> y;
#pragma unroll
      for (int e = 0; e < N; ++e) y.v[e] = Num<TO>::down(Num<TI>::up(x[u].v[e]) * a.scale);
      put_through((Pack<TO, N>*)(a.out + to[u]), y);
    }
  }
}

// ---------------------------------------------------------------- gradient
struct TokGradArgs {
  const int64_t* unique;
  const int64_t* unique_offsets;
  const int32_t* seg;
  const int32_t* occ_bm;
  const int32_t* occ_uid;
  const char* dout;
  char* grad;
  double* part;  // [workgroups][2][cols]
  int64_t n, rows, in_stride, out_stride;
  float scale;
  int32_t W, dim, accumulate;
  int32_t lanes;       // lanes per chunk, a power of two
  int32_t chunk;       // sorted tokens per chunk
  int32_t spans;       // workgroups' shares of all n tokens
  int32_t col_tiles;
  int32_t cols;        // col_tiles * lanes * N
  int64_t sum_blocks;  // workgroups that sum; the rest clear rows
  int32_t clear_rows;  // rows per clearing workgroup
  int32_t clear_pieces;  // 16-byte pieces of a row; the last may overlap the one before
  DivU32 by_clear_pieces;
};

// A lane's columns: N of them from `at`, the first `skip` of which are another
// lane's too (the last piece of a row whose width is not a multiple of N) and
// are left to it. `part` numbers the columns of the sums in scratch memory.
struct Cols {
  int32_t part, at, skip;
  bool any;
};
template <int N>
__device__ __forceinline__ Cols cols_of(const TokGradArgs& a, int32_t tile, int32_t li) {
  Cols c;
  c.part = (tile * a.lanes + li) * N;
  c.any = c.part < a.dim;
  c.at = min(c.part, a.dim - N);
  c.skip = c.part - c.at;
  return c;
}

template <typename TO, int N>
__device__ __forceinline__ void put_row(const TokGradArgs& a, int64_t row, const Cols& c,
                                        const double (&s)[N]) {
  if (row < 0 || row >= a.rows) return;  // the sort of a larger table
  Pack<TO, N>* p = (Pack<TO, N>*)(a.grad + row * a.out_stride + c.at * (int64_t)sizeof(TO));
  Pack<TO, N> y;
  if (a.accumulate) {
    y = *p;
#pragma unroll
    for (int e = 0; e < N; ++e)
      y.v[e] = round_sum<TO>((double)Num<TO>::up(y.v[e]) + (double)a.scale * s[e]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) y.v[e] = round_sum<TO>((double)a.scale * s[e]);
  }
  if (c.skip == 0) {
    put_through(p, y);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e >= c.skip) p->v[e] = y.v[e];
  }
}

constexpr int kAhead = 8;   // tokens whose gradients are in flight
// Rows of at most this many tokens are summed whole (measured on 16384 tokens x
// 1024 with their sort: 32 / 64 / 128: 60 / 60 / 64 us).
constexpr int kShort = 64;
constexpr int kClearMax = 1024;
constexpr int kMinLanes = 8;    // lanes of a chunk, at least
constexpr int kChunkMax = 64;   // tokens of a chunk, at most
constexpr int kStage = kThreads / kMinLanes * kChunkMax + kShort;  // tokens of a workgroup

// rows of [row0, row0 + clear_rows) that no token names
template <typename TO>
__device__ void clear_rows(const TokGradArgs& a, int64_t row0, int64_t U) {
  __shared__ uint32_t named[kClearMax / 32];
  const int64_t row1 = min(row0 + a.clear_rows, a.rows);
  if (threadIdx.x < kClearMax / 32) named[threadIdx.x] = 0;
  __syncthreads();
  const int64_t* unique = a.unique;
  const int64_t u0 = wave_partition_point(0, U, [&](int64_t p) { return unique[p] < row0; });
  for (int64_t u = u0 + threadIdx.x; u < U && unique[u] < row1; u += kThreads)
    atomicOr(&named[(unique[u] - row0) >> 5], 1u << ((unique[u] - row0) & 31));
  __syncthreads();
  // 16 bytes per thread, rows one after the other
  const uint32_t pieces = (uint32_t)a.clear_pieces, total = (uint32_t)(row1 - row0) * pieces;
  for (uint32_t x = threadIdx.x; x < total; x += kThreads) {
    const uint32_t r = divu32(x, a.by_clear_pieces), p = x - r * pieces;
    if ((named[r >> 5] >> (r & 31)) & 1u) continue;
    char* row = a.grad + (row0 + r) * a.out_stride;
    constexpr int kPer = 16 / sizeof(TO);
    if (a.dim >= kPer) {
      put_through((Pack<TO, kPer>*)((TO*)row + min((int32_t)p * kPer, a.dim - kPer)), Pack<TO, kPer>{});
    } else {
      for (int32_t y = 0; y < a.dim; ++y) ((TO*)row)[y] = Num<TO>::down(0.f);
    }
  }
}

// A lane group takes a chunk of the sorted tokens and N columns per lane and
// sums row after row in 64 bits. Rows of at most kShort tokens belong whole to
// the chunk they begin in, which reads on past its end for the last one, so
// nearly every row is written at once. Of a longer row each chunk sums its own
// tokens: the workgroup adds its chunks' sums in LDS and writes the rows that
// begin and end in it; the rest goes to `part` ([0] of a row that came in, [1]
// of one that goes on), which k_token_join adds. A workgroup's tokens and rows
// are read together into LDS first: between its start and its first gradient
// stand two dependent reads (row index, row), not one per token. Bound by HBM:
// the kernel takes 162 us for 262139 x 1000 bf16 into 131072 rows (copying the
// bytes takes 152) and 28 for 16384 x 1024 bf16 into 32000 fp32 rows (28); with
// `accumulate` into the rows that have tokens, the call (with k_token_join) takes
// 185 instead of 180 and 28 instead of 33 us.
struct TokStage {
  int32_t bm[kStage], uid[kStage];
  uint32_t row[kStage];
};

// What a lane group leaves of its long rows
constexpr int32_t kCame = 1;     // [0]: of a row that came in and ends here
constexpr int32_t kGoes = 2;     // [1]: of a row that begins here and goes on
constexpr int32_t kThrough = 4;  // [0]: of a row that came in and goes on

template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(kThreads) k_token_grad(TokGradArgs a) {
  // the sums take the place of the tokens when these are done with
  constexpr size_t kSums = (size_t)2 * kThreads * N * sizeof(double);
  __shared__ __attribute__((aligned(16))) char
      lds[kSums > sizeof(TokStage) ? kSums : sizeof(TokStage)];
  __shared__ int32_t s_has[kThreads / kMinLanes];
  __shared__ uint32_t s_last[kThreads / kMinLanes];
  __shared__ int32_t s_any;
  if ((int64_t)blockIdx.x >= a.sum_blocks) {
    const int64_t U = max((int64_t)0, min(a.unique_offsets[a.W], a.n));
    clear_rows<TO>(a, ((int64_t)blockIdx.x - a.sum_blocks) * a.clear_rows, U);
    return;
  }
  TokStage& st = *(TokStage*)lds;
  const int32_t groups = kThreads / a.lanes, gi = threadIdx.x / a.lanes;
  const int32_t li = threadIdx.x % a.lanes;
  const int32_t tile = (int32_t)(blockIdx.x % a.col_tiles);
  const int64_t wg = blockIdx.x / a.col_tiles;
  const int64_t base = wg * groups * a.chunk;  // the workgroup's first token
  const int32_t staged = groups * a.chunk + kShort;
  const int64_t U = max((int64_t)0, min(a.unique_offsets[a.W], a.n));
  for (int32_t x = threadIdx.x; x < staged; x += kThreads) {
    const bool in = base + x < a.n;
    // past the last sorted token the arrays hold anything: clamped to be read
    const int32_t u = in ? a.occ_uid[base + x] : 0;
    st.uid[x] = u;
    st.bm[x] = in ? min(max(a.occ_bm[base + x], 0), (int32_t)a.n - 1) : 0;
    st.row[x] = (uint32_t)a.unique[min(max(u, 0), (int32_t)a.n - 1)];
  }
  if (threadIdx.x == 0) s_any = 0;
  if (threadIdx.x < kThreads / kMinLanes) s_has[threadIdx.x] = 0;
  const int32_t n = min(a.seg[U], (int32_t)a.n);
  __syncthreads();
  const int32_t off = gi * a.chunk;
  const int64_t e0 = base + off;
  const Cols col = cols_of<N>(a, tile, li);
  double s[N], came_sum[N];
#pragma unroll
  for (int x = 0; x < N; ++x) s[x] = came_sum[x] = 0;
  int32_t has = 0;
  uint32_t row = 0;
  if (e0 < n && col.any) {
    const int32_t e1 = (int32_t)min((int64_t)n, e0 + a.chunk);
    // the rows at the chunk's two ends
    const int32_t uf = st.uid[off], ul = st.uid[off + (e1 - (int32_t)e0) - 1];
    const int32_t f0 = a.seg[uf], f1 = a.seg[uf + 1], l0 = a.seg[ul], l1 = a.seg[ul + 1];
    const bool came = f0 < (int32_t)e0, goes = l1 > e1;
    const bool long_f = f1 - f0 > kShort, long_l = l1 - l0 > kShort;
    const int32_t p0 = came && !long_f ? f1 : (int32_t)e0;  // its chunk sums it
    const int32_t p1 = goes && !long_l ? (l0 < (int32_t)e0 ? e1 : l1) : e1;
    const char* src = a.dout + col.at * (int64_t)sizeof(TI);
    int32_t at = p0 - (int32_t)base;
    const int32_t stop = p1 - (int32_t)base;
    bool first = came && long_f;  // the row being summed came in
    if (at < stop) {
      row = st.row[at];
      for (; at < stop; at += kAhead) {
        Pack<TI, N> v[kAhead];
        uint32_t r[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          const int32_t x = min(at + k, stop - 1);
          r[k] = st.row[x];
          v[k] = *(const Pack<TI, N>*)(src + (int64_t)st.bm[x] * a.in_stride);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
          if (at + k < stop) {
            if (r[k] != row) {
              if (first) {
                has = kCame;
#pragma unroll
                for (int x = 0; x < N; ++x) came_sum[x] = s[x];
              } else {
                put_row<TO, N>(a, row, col, s);
              }
              first = false;
              row = r[k];
#pragma unroll
              for (int x = 0; x < N; ++x) s[x] = 0;
            }
#pragma unroll
            for (int x = 0; x < N; ++x) s[x] += (double)Num<TI>::up(v[k].v[x]);
          }
        }
      }
      if (first) {
        has = goes ? kThrough : kCame;
#pragma unroll
        for (int x = 0; x < N; ++x) came_sum[x] = s[x];
      } else if (goes && long_l) {
        has |= kGoes;
      } else {
        put_row<TO, N>(a, row, col, s);
      }
    }
  }
  if (has) s_any = 1;  // the same for every lane of a group that has a column
  __syncthreads();
  if (!s_any) return;
  // the groups' sums, then each column's in the order of the groups
  double* sums = (double*)lds;
  if (col.any) {
    if (li == 0) {
      s_has[gi] = has;
      s_last[gi] = row;
    }
#pragma unroll
    for (int x = 0; x < N; ++x) {
      sums[(gi * 2 + 0) * a.lanes * N + li * N + x] = came_sum[x];
      sums[(gi * 2 + 1) * a.lanes * N + li * N + x] = s[x];
    }
  }
  __syncthreads();
  if (gi != 0 || !col.any) return;
#pragma unroll
  for (int x = 0; x < N; ++x) s[x] = 0;
  auto keep = [&](int32_t which) {
    double* p = a.part + (wg * 2 + which) * a.cols + col.part;
#pragma unroll
    for (int x = 0; x < N; ++x) p[x] = s[x];
  };
  bool open = false, began = false;  // a row is being added; it began in this workgroup
  uint32_t open_row = 0;
  for (int32_t y = 0; y < groups; ++y) {
    const int32_t h = s_has[y];
    const double* p = sums + y * 2 * a.lanes * N + li * N;
    if (h & (kCame | kThrough)) {
      open = true;
#pragma unroll
      for (int x = 0; x < N; ++x) s[x] += p[x];
    }
    if (h & kCame) {
      if (began) put_row<TO, N>(a, open_row, col, s); else keep(0);
      open = began = false;
#pragma unroll
      for (int x = 0; x < N; ++x) s[x] = 0;
    }
    if (h & kGoes) {
      open = began = true;
      open_row = s_last[y];
#pragma unroll
      for (int x = 0; x < N; ++x) s[x] = p[a.lanes * N + x];
    }
  }
  if (open) keep(began ? 1 : 0);
}

// Rows of more than kShort tokens over several workgroups: that of the
// workgroup where such a row begins adds the workgroups' sums, every lane
// group a run of them, then the groups in order.
template <typename TO, int N>
__global__ void __launch_bounds__(kThreads) k_token_join(TokGradArgs a) {
  __shared__ double stage[kThreads][N];
  const int64_t U = max((int64_t)0, min(a.unique_offsets[a.W], a.n));
  const int32_t tile = (int32_t)(blockIdx.x % a.col_tiles);
  const int32_t groups = kThreads / a.lanes, gi = threadIdx.x / a.lanes;
  const int32_t span = groups * a.chunk;  // tokens of a workgroup
  const int32_t c = (int32_t)(blockIdx.x / a.col_tiles);
  const int64_t end = ((int64_t)c + 1) * span;  // below n: see the grid
  const int32_t u = min(max(a.occ_uid[end - 1], 0), (int32_t)a.n - 1);
  if (end >= a.seg[U]) return;
  const int32_t l0 = a.seg[u], l1 = a.seg[u + 1];
  if (l0 < (int64_t)c * span || l1 <= end || l1 - l0 <= kShort) return;  // uniform
  const int32_t last = (l1 - 1) / span;
  const int32_t li = threadIdx.x % a.lanes;
  const Cols col = cols_of<N>(a, tile, li);
  double s[N];
#pragma unroll
  for (int x = 0; x < N; ++x) s[x] = 0;
  if (col.any) {
    const double* p = a.part + col.part;
    if (gi == 0) {
#pragma unroll
      for (int x = 0; x < N; ++x) s[x] = p[((int64_t)c * 2 + 1) * a.cols + x];
    }
    const int32_t all = last - c;
    const int32_t k0 = c + 1 + (int32_t)((int64_t)all * gi / groups);
    const int32_t k1 = c + 1 + (int32_t)((int64_t)all * (gi + 1) / groups);
    for (int32_t k = k0; k < k1; k += kAhead) {
      double v[kAhead][N];
#pragma unroll
      for (int y = 0; y < kAhead; ++y)
#pragma unroll
        for (int x = 0; x < N; ++x) v[y][x] = p[(int64_t)min(k + y, k1 - 1) * 2 * a.cols + x];
#pragma unroll
      for (int y = 0; y < kAhead; ++y)
        if (k + y < k1)
#pragma unroll
          for (int x = 0; x < N; ++x) s[x] += v[y][x];
    }
  }
#pragma unroll
  for (int x = 0; x < N; ++x) stage[threadIdx.x][x] = s[x];
  __syncthreads();
  if (gi != 0 || !col.any) return;
  for (int32_t y = 1; y < groups; ++y)
#pragma unroll
    for (int x = 0; x < N; ++x) s[x] += stage[y * a.lanes + li][x];
  put_row<TO, N>(a, a.unique[u], col, s);
}

// ---------------------------------------------------------------- host side
int32_t elem_bytes(int32_t dtype) { return dtype == FS_F32 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == FS_F32 || dtype == FS_BF16 || dtype == FS_F16; }

// Elements per access: as many as the wider type's 16 bytes hold, or the
// narrower's where the two differ, of a row that has them
int32_t piece_elems(int32_t dim, int32_t most) {
  while (most > dim) most /= 2;
  return most;
}

template <typename TI, typename TO>
void launch_lookup(const TokLookupArgs& a, int32_t elems, unsigned grid, hipStream_t stream) {
  switch (elems) {
    case 8:
      if constexpr (sizeof(TI) + sizeof(TO) < 8)  // 16 bytes of a 2-byte type
        hipLaunchKernelGGL((k_token_lookup<TI, TO, 8>), dim3(grid), dim3(kThreads), 0, stream, a);
      break;
    case 4: hipLaunchKernelGGL((k_token_lookup<TI, TO, 4>), dim3(grid), dim3(kThreads), 0, stream, a); break;
    case 2: hipLaunchKernelGGL((k_token_lookup<TI, TO, 2>), dim3(grid), dim3(kThreads), 0, stream, a); break;
    default: hipLaunchKernelGGL((k_token_lookup<TI, TO, 1>), dim3(grid), dim3(kThreads), 0, stream, a);
  }
}

template <typename TI>
void launch_lookup(const TokLookupArgs& a, int32_t elems, int32_t out_dtype, unsigned grid,
                   hipStream_t stream) {
  if (out_dtype == FS_F32) launch_lookup<TI, float>(a, elems, grid, stream);
  else if (out_dtype == FS_BF16) launch_lookup<TI, __bf16>(a, elems, grid, stream);
  else launch_lookup<TI, _Float16>(a, elems, grid, stream);
}

template <typename TI, typename TO, int N>
int launch_grad(const TokGradArgs& a, int64_t blocks, hipStream_t stream) {
  if (blocks > 0) {
    hipLaunchKernelGGL((k_token_grad<TI, TO, N>), dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    FS_LAUNCH_CHECK();
  }
  if (a.n > kShort && a.spans > 1) {
    hipLaunchKernelGGL((k_token_join<TO, N>), dim3((unsigned)((a.spans - 1) * a.col_tiles)),
                       dim3(kThreads), 0, stream, a);
    FS_LAUNCH_CHECK();
  }
  return FS_OK;
}

template <typename TI, typename TO>
int launch_grad(const TokGradArgs& a, int32_t elems, int64_t blocks, hipStream_t stream) {
  switch (elems) {
    case 8:
      if constexpr (sizeof(TI) == 2) return launch_grad<TI, TO, 8>(a, blocks, stream);
      break;
    case 4: return launch_grad<TI, TO, 4>(a, blocks, stream);
    case 2: return launch_grad<TI, TO, 2>(a, blocks, stream);
  }
  return launch_grad<TI, TO, 1>(a, blocks, stream);
}

template <typename TI>
int launch_grad(const TokGradArgs& a, int32_t elems, int32_t out_dtype, int64_t blocks,
                hipStream_t stream) {
  if (out_dtype == FS_F32) return launch_grad<TI, float>(a, elems, blocks, stream);
  if (out_dtype == FS_BF16) return launch_grad<TI, __bf16>(a, elems, blocks, stream);
  return launch_grad<TI, _Float16>(a, elems, blocks, stream);
}

// Sorted tokens per chunk of a gradient call: as long as about 4096 waves of
// 512 columns each still share the work, and at least 16. Measured with the
// sort: 16384 tokens x 1024, chunks of 8 / 16 / 32: 60 / 57 / 57 us; 262139 x
// 1000, chunks of 64 by the rule, the same time with 16 at least as with 8.
constexpr int32_t kChunkMin = 16;
int32_t grad_chunk(int64_t n, int32_t dim) {
  int32_t c = kChunkMin;
  while (c < kChunkMax && n * dim >= (int64_t)c * 2 * 512 * 4096) c *= 2;
  return c;
}
// the most chunks of any call of at most n tokens
int64_t grad_chunks_cap(int64_t n, int32_t dim) {
  int64_t most = cdiv(n, grad_chunk(n, dim));
  for (int32_t c = kChunkMin; c < kChunkMax; c *= 2) {  // the largest call of each chunk size
    const int64_t last = std::min(n, ((int64_t)c * 2 * 512 * 4096 - 1) / dim);
    most = std::max(most, cdiv(last, c));
  }
  return most;
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" int fs_token_lookup(const fs_table* table, const int64_t* ids, int64_t n, float scale,
                               void* out, int32_t out_dtype, int64_t out_stride, int32_t* err,
                               hipStream_t stream) {
  if (!table || table->rows < 1 || table->dim < 1 || n < 0 || n >= (int64_t)INT32_MAX ||
      !dtype_ok(table->dtype) || !dtype_ok(out_dtype))
    return FS_ERR_INVALID_ARG;
  if (table->dim > FS_MAX_TOKEN_DIM) return FS_ERR_UNSUPPORTED;
  if (n == 0) return FS_OK;
  if (!table->weights || !ids || !out) return FS_ERR_INVALID_ARG;
  const int32_t ei = elem_bytes(table->dtype), eo = elem_bytes(out_dtype);
  TokLookupArgs a;
  a.in_stride = table->stride ? table->stride : (int64_t)table->dim * ei;
  a.out_stride = out_stride ? out_stride : (int64_t)table->dim * eo;
  if (a.in_stride < (int64_t)table->dim * ei || a.in_stride % ei || (uintptr_t)table->weights % ei ||
      a.out_stride < (int64_t)table->dim * eo || a.out_stride % eo || (uintptr_t)out % eo)
    return FS_ERR_INVALID_ARG;
  a.table = (const char*)table->weights;
  a.ids = ids;
  a.out = (char*)out;
  a.err = err;
  a.n = n;
  a.rows = table->rows;
  a.scale = scale;
  const int32_t elems = piece_elems(table->dim, ei == 4 && eo == 4 ? 4 : 8);
  a.dim = table->dim;
  a.pieces = (int32_t)cdiv(table->dim, elems);
  // more rows than fill a workgroup where the grid would pass 2^32 threads
  a.rows_per_block = (int32_t)std::max<int64_t>({1, kThreads * kLookupPer / a.pieces,
                                                 cdiv(n, kLookupBlocks)});
  a.by_pieces = make_divu32((uint32_t)a.pieces);
  const unsigned grid = (unsigned)cdiv(n, a.rows_per_block);
  if (table->dtype == FS_F32) launch_lookup<float>(a, elems, out_dtype, grid, stream);
  else if (table->dtype == FS_BF16) launch_lookup<__bf16>(a, elems, out_dtype, grid, stream);
  else launch_lookup<_Float16>(a, elems, out_dtype, grid, stream);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

extern "C" size_t fs_token_grad_workspace_size(int64_t n, int32_t dim) {
  if (n < 0 || dim < 1) return 0;
  Carve c(nullptr);
  // a workgroup has at least four chunks, and fewer columns where it has more
  c.take<double>((size_t)cdiv(grad_chunks_cap(n, dim), kThreads / kWave) * 2 * align_up((size_t)dim, 512));
  return c.used + 256;
}

extern "C" int fs_token_grad(const int64_t* unique, const int64_t* unique_offsets, int32_t W,
                             const int32_t* seg_offsets, const int32_t* occ_bm,
                             const int32_t* occ_uid, int64_t n, const void* dout,
                             int32_t dout_dtype, int64_t dout_stride, float scale, int64_t rows,
                             int32_t dim, void* grad, int32_t grad_dtype, int64_t grad_stride,
                             int32_t accumulate, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (n < 0 || n >= (int64_t)INT32_MAX || rows < 1 || dim < 1 || W < 1 || W > FS_MAX_RANKS ||
      !unique_offsets || !seg_offsets || !grad || !dtype_ok(dout_dtype) || !dtype_ok(grad_dtype))
    return FS_ERR_INVALID_ARG;
  if (n > 0 && (!unique || !occ_bm || !occ_uid || !dout)) return FS_ERR_INVALID_ARG;
  if (rows >= (int64_t)UINT32_MAX || dim > FS_MAX_TOKEN_DIM) return FS_ERR_UNSUPPORTED;
  const int32_t ei = elem_bytes(dout_dtype), eo = elem_bytes(grad_dtype);
  TokGradArgs a;
  a.in_stride = dout_stride ? dout_stride : (int64_t)dim * ei;
  a.out_stride = grad_stride ? grad_stride : (int64_t)dim * eo;
  if (a.in_stride < (int64_t)dim * ei || a.in_stride % ei || (uintptr_t)dout % ei ||
      a.out_stride < (int64_t)dim * eo || a.out_stride % eo || (uintptr_t)grad % eo)
    return FS_ERR_INVALID_ARG;
  if (!ws || ws_bytes < fs_token_grad_workspace_size(n, dim)) return FS_ERR_WORKSPACE;
  a.unique = unique;
  a.unique_offsets = unique_offsets;
  a.seg = seg_offsets;
  a.occ_bm = occ_bm;
  a.occ_uid = occ_uid;
  a.dout = (const char*)dout;
  a.grad = (char*)grad;
  Carve c(ws);
  a.part = c.take<double>(1);
  a.n = n;
  a.rows = rows;
  a.scale = scale;
  a.W = W;
  a.dim = dim;
  a.accumulate = accumulate != 0;
  const int32_t elems = piece_elems(dim, ei == 4 ? 4 : 8);
  const int32_t pieces = (int32_t)cdiv(dim, elems);
  a.lanes = kMinLanes;
  while (a.lanes < kWave && a.lanes < pieces) a.lanes *= 2;
  a.chunk = grad_chunk(n, dim);
  // few tokens in one workgroup need no second launch (about 4 us); beyond 32
  // tokens one after the other a group takes as long itself
  const int32_t groups = kThreads / a.lanes;
  while (a.chunk < 32 && (int64_t)a.chunk * groups < n && n <= (int64_t)32 * groups) a.chunk *= 2;
  a.spans = (int32_t)cdiv(n, (int64_t)a.chunk * groups);
  a.col_tiles = (int32_t)cdiv(pieces, a.lanes);
  a.cols = a.col_tiles * a.lanes * elems;
  a.sum_blocks = (int64_t)a.spans * a.col_tiles;
  const int64_t row_bytes = (int64_t)dim * eo;
  a.clear_pieces = (int32_t)cdiv(row_bytes, 16);
  a.by_clear_pieces = make_divu32((uint32_t)a.clear_pieces);
  a.clear_rows = (int32_t)std::min<int64_t>(kClearMax, std::max<int64_t>(4, 32768 / row_bytes));
  const int64_t clear_blocks = a.accumulate ? 0 : cdiv(rows, a.clear_rows);
  const int64_t blocks = a.sum_blocks + clear_blocks;
  if (!grid_fits(blocks, kThreads)) return FS_ERR_UNSUPPORTED;
  if (dout_dtype == FS_F32) return launch_grad<float>(a, elems, grad_dtype, blocks, stream);
  if (dout_dtype == FS_BF16) return launch_grad<__bf16>(a, elems, grad_dtype, blocks, stream);
  return launch_grad<_Float16>(a, elems, grad_dtype, blocks, stream);
}
