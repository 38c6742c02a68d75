// Token embedding: scaled lookup of a vocabulary's rows, the tokens sorted by
// row, and the gradient of the rows by the sorted tokens.
//
//   out[i] = scale w[ids[i]]        g[v] = scale sum over i with ids[i] = v of dout[i]
#include <algorithm>

#include "common.hpp"
#include "divu32.hpp"

namespace fs {
namespace {

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

// N elements that lie at a multiple of their size (at most 16 bytes)
template <typename T, int N>
struct alignas(sizeof(T) * N > 16 ? 16 : sizeof(T) * N) Pack {
  T v[N];
};

// ---------------------------------------------------------------- lookup
struct TokLookupArgs {
  const char* table;
  const int64_t* ids;
  char* out;
  int32_t* err;
  int64_t n, rows, in_stride, out_stride;
  float scale;
  int32_t pieces;          // pieces of a row
  int32_t rows_per_block;
  DivU32 by_pieces;
};

constexpr int kLookupPer = 4;  // pieces per thread

// A workgroup takes rows_per_block tokens; its threads run over the pieces
// (N elements) of their rows, all of a thread's pieces in flight.
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
        const uint32_t r = divu32(id, a.by_pieces), p = id - r * a.pieces;
        const int64_t row = a.ids[i0 + r];
        to[u] = (i0 + r) * a.out_stride + (int64_t)p * (int64_t)(sizeof(TO) * N);
        if (row >= 0 && row < a.rows)
          x[u] = *(const Pack<TI, N>*)(a.table + row * a.in_stride + (int64_t)p * (int64_t)(sizeof(TI) * N));
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
      *(Pack<TO, N>*)(a.out + to[u]) = y;
    }
  }
}

// ---------------------------------------------------------------- sort
// The tokens as the items of a one-shard batch: dropped ones (padding, outside
// the table) go to one more row behind the last, which the sort puts last.
__global__ void __launch_bounds__(kThreads)
k_token_items(const int64_t* __restrict__ ids, int64_t n, int64_t rows, int64_t padding,
              int64_t* __restrict__ keys, int32_t* __restrict__ bm, int64_t* __restrict__ bounds,
              int32_t* __restrict__ err) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  bool bad = false;
  if (i < n) {
    const int64_t id = ids[i];
    bad = id != padding && (id < 0 || id >= rows);
    keys[i] = id == padding || bad ? rows : id;
    bm[i] = (int32_t)i;
  }
  flag_err(err, bad, FS_EF_ID_RANGE);
  if (i == 0) {
    bounds[0] = 0;
    bounds[1] = n;
  }
}

// takes the row of the dropped tokens off the end
__global__ void k_token_drop(const int64_t* __restrict__ unique, int64_t rows, int64_t n,
                             int64_t* __restrict__ unique_offsets, int64_t* __restrict__ counts) {
  const int64_t u = counts[0];
  if (threadIdx.x == 0 && u > 0 && u <= n && unique[u - 1] >= rows) {
    counts[0] = u - 1;
    counts[2] = u - 1;
    unique_offsets[1] = u - 1;
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
  double* part;  // [chunks][2][cols]
  int64_t n, rows, in_stride, out_stride;
  float scale;
  int32_t W, dim, accumulate;
  int32_t lanes;       // lanes per chunk, a power of two
  int32_t chunk;       // sorted tokens per chunk
  int32_t chunks;      // of all n tokens
  int32_t col_tiles;
  int32_t cols;        // col_tiles * lanes * N
  int64_t sum_blocks;  // workgroups that sum; the rest clear rows
  int32_t clear_rows;  // rows per clearing workgroup
};

template <typename TO, int N>
__device__ __forceinline__ void put_row(const TokGradArgs& a, int64_t row, int32_t col,
                                        const double (&s)[N]) {
  Pack<TO, N>* p = (Pack<TO, N>*)(a.grad + row * a.out_stride + (int64_t)col * (int64_t)sizeof(TO));
  Pack<TO, N> y;
  if (a.accumulate) {
    y = *p;
#pragma unroll
    for (int e = 0; e < N; ++e)
      y.v[e] = Num<TO>::down((float)((double)Num<TO>::up(y.v[e]) + (double)a.scale * s[e]));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) y.v[e] = Num<TO>::down((float)((double)a.scale * s[e]));
  }
  *p = y;
}

constexpr int kAhead = 8;  // tokens whose gradients are in flight
constexpr int kClearMax = 1024;

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
  const int64_t bytes = (int64_t)a.dim * (int64_t)sizeof(TO);
  const bool wide = (bytes & 15) == 0 && (a.out_stride & 15) == 0 && ((uintptr_t)a.grad & 15) == 0;
  const int w = threadIdx.x / kWave;
  for (int64_t r = row0 + w; r < row1; r += kThreads / kWave) {
    if ((named[(r - row0) >> 5] >> ((r - row0) & 31)) & 1u) continue;
    char* p = a.grad + r * a.out_stride;
    if (wide) {
      for (int64_t x = lane() * 16; x < bytes; x += kWave * 16) *(uint4*)(p + x) = uint4{0, 0, 0, 0};
    } else {
      for (int64_t x = lane(); x < a.dim; x += kWave) ((TO*)p)[x] = Num<TO>::down(0.f);
    }
  }
}

// A lane group takes a chunk of the sorted tokens and N columns per lane,
// sums row after row in 64 bits, and writes the rows that begin and end in
// the chunk; the sums of rows that cross a chunk's bound go to `part`: [0] of
// the row that came in, [1] of the row that goes on.
template <typename TI, typename TO, int N>
__global__ void __launch_bounds__(kThreads) k_token_grad(TokGradArgs a) {
  const int64_t U = max((int64_t)0, min(a.unique_offsets[a.W], a.n));
  if ((int64_t)blockIdx.x >= a.sum_blocks) {
    clear_rows<TO>(a, ((int64_t)blockIdx.x - a.sum_blocks) * a.clear_rows, U);
    return;
  }
  const int32_t n = min(a.seg[U], (int32_t)a.n);
  const int32_t groups = kThreads / a.lanes;
  const int32_t tile = (int32_t)(blockIdx.x % a.col_tiles);
  const int64_t c = (int64_t)(blockIdx.x / a.col_tiles) * groups + threadIdx.x / a.lanes;
  const int32_t col = (tile * a.lanes + (int32_t)(threadIdx.x % a.lanes)) * N;
  const int64_t e0 = c * a.chunk;
  if (e0 >= n || col >= a.dim) return;
  const int32_t e1 = (int32_t)min((int64_t)n, e0 + a.chunk);
  double s[N];
#pragma unroll
  for (int x = 0; x < N; ++x) s[x] = 0;
  const char* base = a.dout + (int64_t)col * (int64_t)sizeof(TI);
  int32_t u = a.occ_uid[e0];
  auto close = [&](bool goes_on) {  // row u ends here, or at the chunk's end
    if (a.seg[u] < (int32_t)e0 || goes_on) {
      double* p = a.part + ((int64_t)c * 2 + (a.seg[u] < (int32_t)e0 ? 0 : 1)) * a.cols + col;
#pragma unroll
      for (int x = 0; x < N; ++x) p[x] = s[x];
    } else {
      put_row<TO, N>(a, a.unique[u], col, s);
    }
#pragma unroll
    for (int x = 0; x < N; ++x) s[x] = 0;
  };
  for (int32_t e = (int32_t)e0; e < e1; e += kAhead) {
    Pack<TI, N> v[kAhead];
    int32_t uid[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int32_t x = min(e + k, e1 - 1);
      uid[k] = a.occ_uid[x];
      v[k] = *(const Pack<TI, N>*)(base + (int64_t)a.occ_bm[x] * a.in_stride);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (e + k < e1) {
        if (uid[k] != u) {
          close(false);
          u = uid[k];
        }
#pragma unroll
        for (int x = 0; x < N; ++x) s[x] += (double)Num<TI>::up(v[k].v[x]);
      }
    }
  }
  close(a.seg[u + 1] > e1);
}

// Rows over several chunks: the workgroup of the chunk where a row begins
// adds the chunks' sums, each lane group every groups-th one, then the groups
// in order.
template <typename TO, int N>
__global__ void __launch_bounds__(kThreads) k_token_join(TokGradArgs a) {
  __shared__ double stage[kThreads][N];
  const int64_t U = max((int64_t)0, min(a.unique_offsets[a.W], a.n));
  const int32_t n = min(a.seg[U], (int32_t)a.n);
  const int32_t tile = (int32_t)(blockIdx.x % a.col_tiles);
  const int64_t c = blockIdx.x / a.col_tiles;
  const int64_t end = (c + 1) * a.chunk;
  if (end >= n) return;
  const int32_t u = a.occ_uid[end - 1];
  if (a.seg[u] < c * a.chunk || a.seg[u + 1] <= end) return;  // uniform
  const int64_t last = (a.seg[u + 1] - 1) / a.chunk;
  const int32_t groups = kThreads / a.lanes, gi = threadIdx.x / a.lanes;
  const int32_t li = threadIdx.x % a.lanes;
  const int32_t col = (tile * a.lanes + li) * N;
  double s[N];
#pragma unroll
  for (int x = 0; x < N; ++x) s[x] = 0;
  if (col < a.dim) {
    for (int64_t k = c + gi; k <= last; k += groups) {
      const double* p = a.part + (k * 2 + (k == c ? 1 : 0)) * a.cols + col;
#pragma unroll
      for (int x = 0; x < N; ++x) s[x] += p[x];
    }
  }
#pragma unroll
  for (int x = 0; x < N; ++x) stage[threadIdx.x][x] = s[x];
  __syncthreads();
  if (gi != 0 || col >= a.dim) return;
  for (int32_t y = 1; y < groups; ++y)
#pragma unroll
    for (int x = 0; x < N; ++x) s[x] += stage[y * a.lanes + li][x];
  put_row<TO, N>(a, a.unique[u], col, s);
}

// ---------------------------------------------------------------- host side
int32_t elem_bytes(int32_t dtype) { return dtype == FS_F32 ? 4 : 2; }
bool dtype_ok(int32_t dtype) { return dtype == FS_F32 || dtype == FS_BF16 || dtype == FS_F16; }

// Elements per access: the most, up to `most`, that divide the row and keep
// both arrays' accesses aligned.
int32_t piece_elems(int32_t dim, int32_t most, const void* a, int64_t a_stride, int32_t a_elem,
                    const void* b, int64_t b_stride, int32_t b_elem) {
  int32_t n = most;
  auto fits = [&](const void* p, int64_t stride, int32_t elem) {
    const int64_t al = n * elem > 16 ? 16 : n * elem;
    return (uintptr_t)p % al == 0 && stride % al == 0;
  };
  while (n > 1 && (dim % n || !fits(a, a_stride, a_elem) || !fits(b, b_stride, b_elem))) n /= 2;
  return n;
}

template <typename TI, typename TO>
void launch_lookup(const TokLookupArgs& a, int32_t elems, unsigned grid, hipStream_t stream) {
  switch (elems) {
    case 8: hipLaunchKernelGGL((k_token_lookup<TI, TO, 8>), dim3(grid), dim3(kThreads), 0, stream, a); break;
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
  if (a.chunks > 1) {
    hipLaunchKernelGGL((k_token_join<TO, N>), dim3((unsigned)(a.chunks * a.col_tiles)),
                       dim3(kThreads), 0, stream, a);
    FS_LAUNCH_CHECK();
  }
  return FS_OK;
}

template <typename TI, typename TO>
int launch_grad(const TokGradArgs& a, int32_t elems, int64_t blocks, hipStream_t stream) {
  switch (elems) {
    case 8: return launch_grad<TI, TO, 8>(a, blocks, stream);
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

// Sorted tokens per chunk of a gradient call: a rule on the token count alone,
// so that the workspace query and every alignment agree.
int32_t grad_chunk(int64_t n) { return n <= 4096 ? 8 : (n <= 65536 ? 16 : 64); }
// chunks of any call with at most n tokens
int64_t grad_chunks_cap(int64_t n) {
  int64_t most = cdiv(n, grad_chunk(n));
  if (n > 4096) most = std::max(most, cdiv((int64_t)4096, (int64_t)8));
  if (n > 65536) most = std::max(most, cdiv((int64_t)65536, (int64_t)16));
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
  const int32_t elems = piece_elems(table->dim, ei == 4 && eo == 4 ? 4 : 8, table->weights,
                                    a.in_stride, ei, out, a.out_stride, eo);
  a.pieces = table->dim / elems;
  a.rows_per_block = std::max(1, kThreads * kLookupPer / a.pieces);
  a.by_pieces = make_divu32((uint32_t)a.pieces);
  const unsigned grid = (unsigned)cdiv(n, a.rows_per_block);
  if (table->dtype == FS_F32) launch_lookup<float>(a, elems, out_dtype, grid, stream);
  else if (table->dtype == FS_BF16) launch_lookup<__bf16>(a, elems, out_dtype, grid, stream);
  else launch_lookup<_Float16>(a, elems, out_dtype, grid, stream);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

extern "C" size_t fs_token_sort_workspace_size(int64_t n) {
  if (n < 0) return 0;
  const size_t cap = (size_t)(n > 0 ? n : 1);
  Carve c(nullptr);
  c.take<int64_t>(cap);
  c.take<int32_t>(cap);
  c.take<int64_t>(2);
  c.take<uint8_t>(cap);
  return c.used + 256 + fs_unique_workspace_size(n, 0, 1, 1);
}

extern "C" int fs_token_sort(const int64_t* ids, int64_t n, int64_t rows, int64_t padding_id,
                             int64_t* unique, int64_t* unique_offsets, int32_t* seg_offsets,
                             int32_t* occ_bm, int32_t* occ_uid, int64_t* counts, int32_t* err,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  if (n < 0 || n >= (int64_t)INT32_MAX || rows < 1 || !unique_offsets || !seg_offsets || !counts)
    return FS_ERR_INVALID_ARG;
  if (rows >= (int64_t)UINT32_MAX) return FS_ERR_UNSUPPORTED;
  if (n > 0 && (!ids || !unique || !occ_bm || !occ_uid)) return FS_ERR_INVALID_ARG;
  if (!ws || ws_bytes < fs_token_sort_workspace_size(n)) return FS_ERR_WORKSPACE;
  const size_t cap = (size_t)(n > 0 ? n : 1);
  Carve c(ws);
  int64_t* keys = c.take<int64_t>(cap);
  int32_t* bm = c.take<int32_t>(cap);
  int64_t* bounds = c.take<int64_t>(2);
  uint8_t* cls = c.take<uint8_t>(cap);
  char* rest = (char*)ws + align_up(c.used, 256);
  hipLaunchKernelGGL(k_token_items, dim3((unsigned)cdiv((int64_t)cap, kThreads)), dim3(kThreads), 0,
                     stream, ids, n, rows, padding_id, keys, bm, bounds, err);
  FS_LAUNCH_CHECK();
  fs_table tab = {};
  tab.rows = rows + 1;
  const int rc = fs_unique_collision_split(
      keys, bm, bounds, n, &tab, 1, 1, nullptr, nullptr, nullptr, 0, unique, unique_offsets,
      seg_offsets, occ_bm, occ_uid, cls, nullptr, counts, rest,
      fs_unique_workspace_size(n, 0, 1, 1), stream);
  if (rc) return rc;
  hipLaunchKernelGGL(k_token_drop, dim3(1), dim3(kWave), 0, stream, unique, rows, n,
                     unique_offsets, counts);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

extern "C" size_t fs_token_grad_workspace_size(int64_t n, int32_t dim) {
  if (n < 0 || dim < 0) return 0;
  Carve c(nullptr);
  c.take<double>((size_t)grad_chunks_cap(n) * 2 * align_up((size_t)dim, 512));
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
  const int32_t elems = piece_elems(dim, ei == 4 ? 4 : 8, dout, a.in_stride, ei, grad,
                                    a.out_stride, eo);
  const int32_t pieces = dim / elems;
  a.lanes = 1;
  while (a.lanes < kWave && a.lanes < pieces) a.lanes *= 2;
  a.chunk = grad_chunk(n);
  a.chunks = (int32_t)cdiv(n, a.chunk);
  a.col_tiles = (int32_t)cdiv(pieces, a.lanes);
  a.cols = a.col_tiles * a.lanes * elems;
  a.sum_blocks = cdiv(a.chunks, kThreads / a.lanes) * a.col_tiles;
  const int64_t row_bytes = (int64_t)dim * eo;
  a.clear_rows = (int32_t)std::min<int64_t>(kClearMax, std::max<int64_t>(4, 32768 / row_bytes));
  const int64_t clear_blocks = a.accumulate ? 0 : cdiv(rows, a.clear_rows);
  const int64_t blocks = a.sum_blocks + clear_blocks;
  if (blocks >= (int64_t)INT32_MAX || (int64_t)a.chunks * a.col_tiles >= (int64_t)INT32_MAX)
    return FS_ERR_UNSUPPORTED;
  if (dout_dtype == FS_F32) return launch_grad<float>(a, elems, grad_dtype, blocks, stream);
  if (dout_dtype == FS_BF16) return launch_grad<__bf16>(a, elems, grad_dtype, blocks, stream);
  return launch_grad<_Float16>(a, elems, grad_dtype, blocks, stream);
}
