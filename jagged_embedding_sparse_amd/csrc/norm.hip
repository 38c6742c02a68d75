// Layer norm over the rows of [n, dim], forward and backward.
//
//   mean = sum x / dim,  rstd = (sum (x - mean)^2 / dim + eps)^-1/2,
//   h = (x - mean) rstd,  out = h weight + bias
//   g = dout weight,  dx = rstd (g - sum g / dim - h sum (g h) / dim),
//   dweight = sum over the rows of dout h,  dbias = of dout
//
// A row stays in the registers of the lanes that share it, so memory is read
// once and the variance is that of the centred values. Both directions are
// bound by memory.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.hpp"

namespace fs {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <typename T, int N>
struct Pack {  // anywhere an element may be: wide accesses need no alignment here
  T v[N];
};

struct NormRows {
  char* p;
  int64_t stride;
  int32_t type;
};

// A lane's share of a row: C pieces of E elements, L lanes apart. The last piece
// of a row may overlap the one before it and pieces past the row are its last
// one again, so that no access waits for a condition; `first` is the piece's
// first element that is this lane's own (E: none). Only sums ask for it: what
// two lanes compute of one element is the same, and so is what they store.
template <int E, int L, int C>
struct Share {
  int32_t at[C], first[C], dim;
  __device__ __forceinline__ Share(int32_t l, int32_t dim_) : dim(dim_) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int32_t col = (c * L + l) * E;
      at[c] = max(min(col, dim - E), 0);
      first[c] = col < dim ? col - at[c] : E;
    }
  }
  // this lane's element, counted once (rows of fewer than E elements have one piece)
  __device__ __forceinline__ bool mine(int c, int e) const { return e >= first[c] && at[c] + e < dim; }

  template <typename T>
  __device__ __forceinline__ void load_as(float (&v)[C][E], const char* row) const {
    if (dim >= E) {  // uniform
      Pack<T, E> x[C];
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] = *(const Pack<T, E>*)(row + at[c] * (int)sizeof(T));
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) v[c][e] = (float)x[c].v[e];
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) v[c][e] = mine(c, e) ? (float)((const T*)row)[at[c] + e] : 0.f;
    }
  }
  __device__ __forceinline__ void load(float (&v)[C][E], const char* row, int32_t type) const {
    if (type == FS_F32) load_as<float>(v, row);
    else if (type == FS_BF16) load_as<__bf16>(v, row);
    else load_as<_Float16>(v, row);
  }

  // A row as it lies, B bytes an element, for a later look at it: the loads of the
  // next row are in flight while this one is worked on.
  template <int B>
  struct Raw {
    Pack<uint32_t, E * B / 4> v[C];
  };
  template <int B>
  __device__ __forceinline__ void load_raw(Raw<B>& r, const char* row) const {
    struct __attribute__((packed, aligned(2))) Any {
      uint32_t v[E * B / 4];
    };
    if (dim >= E) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const Any x = *(const Any*)(row + at[c] * B);
        r.v[c] = __builtin_bit_cast(Pack<uint32_t, E * B / 4>, x);
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < E * B / 4; ++e) {
          if constexpr (B == 4) r.v[c].v[e] = mine(c, e) ? ((const uint32_t*)row)[at[c] + e] : 0u;
          else
            r.v[c].v[e] = (mine(c, 2 * e) ? ((const uint16_t*)row)[at[c] + 2 * e] : 0u) |
                          (mine(c, 2 * e + 1) ? (uint32_t)((const uint16_t*)row)[at[c] + 2 * e + 1] << 16 : 0u);
        }
    }
  }
  template <int B>
  __device__ __forceinline__ void values(float (&v)[C][E], const Raw<B>& r, int32_t type) const {
    if constexpr (B == 4) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) v[c][e] = __uint_as_float(r.v[c].v[e]);
    } else if (type == FS_BF16) {  // uniform
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e) v[c][e] = bf16_bits_to_f32(e & 1 ? r.v[c].v[e / 2] >> 16 : r.v[c].v[e / 2] & 0xffffu);
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e)
          v[c][e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r.v[c].v[e / 2] >> (16 * (e & 1))));
    }
  }

  template <typename T>
  __device__ __forceinline__ void store_as(const float (&v)[C][E], char* row) const {
    if (dim >= E) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        Pack<T, E> y;
#pragma unroll
        for (int e = 0; e < E; ++e) y.v[e] = (T)v[c][e];
        if (first[c] < E) *(Pack<T, E>*)(row + at[c] * (int)sizeof(T)) = y;
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (mine(c, e)) ((T*)row)[at[c] + e] = (T)v[c][e];
    }
  }
  __device__ __forceinline__ void store(const float (&v)[C][E], char* row, int32_t type) const {
    if (type == FS_F32) store_as<float>(v, row);
    else if (type == FS_BF16) store_as<__bf16>(v, row);
    else store_as<_Float16>(v, row);
  }
};

// Sum over groups of W lanes (8 to 64), the same bits in each of them: exchanges
// inside 16 lanes cost no instruction of their own, the two wider ones one each.
template <int W>
__device__ __forceinline__ float lanes_sum(float x) {
  auto dpp = [](float v, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  x += dpp(x, std::integral_constant<int, 0xb1>());   // lanes 1 0 3 2
  x += dpp(x, std::integral_constant<int, 0x4e>());   // lanes 2 3 0 1
  x += dpp(x, std::integral_constant<int, 0x141>());  // 8 lanes mirrored
  if constexpr (W >= 16) x += dpp(x, std::integral_constant<int, 0x140>());  // 16 lanes mirrored
  if constexpr (W >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  if constexpr (W >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  return x;
}

// N sums over the L lanes of a row; with more than a wave the whole workgroup
// shares the row. `tmp` holds 2 x 16 pairs, taken in turn: a pair is written again
// only behind the other's barrier.
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&s)[N], float (*tmp)[2], int turn) {
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = lanes_sum<L < kWave ? L : kWave>(s[k]);
  if constexpr (L > kWave) {
    float(*t)[2] = tmp + 16 * turn;
    if (lane() == 0) {
#pragma unroll
      for (int k = 0; k < N; ++k) t[threadIdx.x / kWave][k] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
      s[k] = 0.f;
#pragma unroll
      for (int i = 0; i < L / kWave; ++i) s[k] += t[i][k];
    }
  }
}

struct NormArgs {
  NormRows x, out;  // backward: out is dout
  char* dx;
  int64_t dx_stride, n;
  const char *weight, *bias;
  float *mean, *rstd;
  float* part;               // backward: [workgroups][2][dim], or null: one workgroup writes
  char *dweight, *dbias;
  int32_t dim, param;        // type of weight, bias and their gradients
  float inv_dim, count, eps;  // count: dim
};

// A sum over a row by its length, rounded once: the product with 1 / dim, and what that
// leaves of the sum by 1 / dim once more. The product alone may be off by a step, and a row
// of one number c would keep what is left of c - mean times rstd (0.02 for 1000 columns of
// 1000 with an eps of 1e-5). 4096 x 16384 bf16 backward: 126.6 us with the product alone, 127.3
// like this, 133 with a division; 32768 x 1024 fp32 to bf16 forward 42 and 43 to 44, others
// within 1%. The length comes with the call: made here it would take a register of rows that
// have none left (4096 x 9000, fp32 with a bf16 dout, backward 161 and 175 us).
__device__ __forceinline__ float by_dim(float sum, const NormArgs& a) {
  const float q = sum * a.inv_dim, left = __builtin_fmaf(-q, a.count, sum);
  return left == left ? __builtin_fmaf(left, a.inv_dim, q) : q;  // none of an infinity
}

// 32768 x 1024 fp32 to bf16: 33 us on one set of rows, part of them in the caches, 40
// on changing ones, where copying the bytes takes 41.
template <int E, int L, int C>
__global__ void __launch_bounds__(L > 256 ? L : 256) k_norm(NormArgs a) {
  __shared__ float tmp[32][2];
  const Share<E, L, C> s(threadIdx.x % L, a.dim);
  float w[C][E], b[C][E];
  if (a.weight) {
    s.load(w, a.weight, a.param);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) w[c][e] = 1.f;
  }
  if (a.bias) {
    s.load(b, a.bias, a.param);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) b[c][e] = 0.f;
  }
  const int per = blockDim.x / L;
  for (int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / L; r < a.n; r += (int64_t)gridDim.x * per) {
    float v[C][E];
    s.load(v, a.x.p + r * a.x.stride, a.x.type);
    float sum[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) sum[0] += s.mine(c, e) ? v[c][e] : 0.f;
    row_sums<L>(sum, tmp, 0);
    const float mean = by_dim(sum[0], a);
    float sq[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[c][e] -= mean;
        sq[0] += s.mine(c, e) ? v[c][e] * v[c][e] : 0.f;
      }
    row_sums<L>(sq, tmp, 1);
    const float rstd = 1.f / sqrtf(by_dim(sq[0], a) + a.eps);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) v[c][e] = v[c][e] * rstd * w[c][e] + b[c][e];
    s.store(v, a.out.p + r * a.out.stride, a.out.type);
    if (threadIdx.x % L == 0) {
      if (a.mean) a.mean[r] = mean;
      if (a.rstd) a.rstd[r] = rstd;
    }
  }
}

__device__ __forceinline__ void put_param(char* p, int32_t type, int64_t i, float v) {
  if (type == FS_F32) ((float*)p)[i] = v;
  else if (type == FS_BF16) ((__bf16*)p)[i] = (__bf16)v;
  else ((_Float16*)p)[i] = (_Float16)v;
}

// The sums of a workgroup's groups of L lanes, in order, in the first group's
// registers. `join` holds C E floats for every thread.
template <int E, int L, int C>
__device__ __forceinline__ void join_groups(float (&v)[C][E], float* join) {
  const int T = blockDim.x, l = threadIdx.x % L, per = T / L;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e) join[(c * E + e) * T + threadIdx.x] = v[c][e];
  __syncthreads();
  // the groups take a lane's C E sums in turn
  for (int k = threadIdx.x / L; k < C * E; k += per) {
    float sum = 0.f;
    for (int g = 0; g < per; ++g) sum += join[k * T + g * L + l];
    join[k * T + l] = sum;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e) v[c][e] = join[(c * E + e) * T + l];
  __syncthreads();
}

// Each group of L lanes adds its rows' parts of dweight and dbias in registers;
// a workgroup's groups are joined in LDS, in order, and the workgroups' sums by
// k_norm_params, in order: equal calls give equal bits. A row is asked for before the
// one in front of it is worked on (65537 x 1000 bf16: 147 -> 95 us; 78 with kParts
// workgroups, 5 TB/s, what a copy reaches).
template <int E, int L, int C, int B>
__global__ void __launch_bounds__(L > 256 ? L : C * E > 8 ? 512 : 1024) k_norm_back(NormArgs a) {
  extern __shared__ float join[];  // [C E][threads], where a workgroup has more groups than one
  __shared__ float tmp[32][2];
  constexpr int BX = 16 / E;  // bytes of an element of x; B: of dout
  const int l = threadIdx.x % L, per = blockDim.x / L;
  const Share<E, L, C> s(l, a.dim);
  float w[C][E], dw[C][E], db[C][E];
  if (a.weight) {
    s.load(w, a.weight, a.param);
  } else {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) w[c][e] = 1.f;
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e) dw[c][e] = db[c][e] = 0.f;
  int turn = 0;
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t r = (int64_t)blockIdx.x * per + threadIdx.x / L;
  typename Share<E, L, C>::template Raw<BX> xr;
  typename Share<E, L, C>::template Raw<B> gr;
  float mean_r = 0.f, rstd_r = 0.f;
  auto ask = [&](int64_t row) {
    s.load_raw(xr, a.x.p + row * a.x.stride);
    s.load_raw(gr, a.out.p + row * a.out.stride);
    mean_r = a.mean[row];
    rstd_r = a.rstd[row];
  };
  if (r < a.n) ask(r);
  for (; r < a.n; r += step) {
    float h[C][E], g[C][E];
    s.values(h, xr, a.x.type);
    s.values(g, gr, a.out.type);
    const float mean = mean_r, rstd = rstd_r;
    constexpr bool kAhead = L < 1024 || C == 1;  // as registers allow
    if (kAhead) ask(min(r + step, a.n - 1));
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        h[c][e] = (h[c][e] - mean) * rstd;
        dw[c][e] += g[c][e] * h[c][e];
        db[c][e] += g[c][e];
        g[c][e] *= w[c][e];
        sum[0] += s.mine(c, e) ? g[c][e] : 0.f;
        sum[1] += s.mine(c, e) ? g[c][e] * h[c][e] : 0.f;
      }
    row_sums<L>(sum, tmp, turn);
    turn ^= 1;
    const float sg = by_dim(sum[0], a), sgh = by_dim(sum[1], a);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < E; ++e) g[c][e] = rstd * (g[c][e] - sg - h[c][e] * sgh);
    s.store(g, a.dx + r * a.dx_stride, a.x.type);
    if (!kAhead) ask(min(r + step, a.n - 1));
  }
  if (!a.dweight && !a.dbias) return;
  if (per > 1) {
    join_groups<E, L, C>(dw, join);
    join_groups<E, L, C>(db, join);
    if (threadIdx.x >= L) return;
  }
  float* part = a.part ? a.part + (int64_t)blockIdx.x * 2 * a.dim : nullptr;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (s.mine(c, e)) {
        const int32_t col = s.at[c] + e;
        if (part) {
          part[col] = dw[c][e];
          part[a.dim + col] = db[c][e];
        } else {
          if (a.dweight) put_param(a.dweight, a.param, col, dw[c][e]);
          if (a.dbias) put_param(a.dbias, a.param, col, db[c][e]);
        }
      }
}

constexpr int kParamCols = 16;

// dweight and dbias: the workgroups' sums, added in the same order by 64 threads a
// column (few columns a workgroup: 768 sums of 2000 columns, 64 columns 5.9 us, 16
// 4.8).
__global__ void __launch_bounds__(1024)
k_norm_params(const float* __restrict__ part, int32_t parts, int32_t dim, char* dweight, char* dbias,
              int32_t type) {
  __shared__ float sh[16][kParamCols];
  const int x = threadIdx.x % kParamCols, y = threadIdx.x / kParamCols;
  const int32_t col = blockIdx.x * kParamCols + x, width = 2 * dim;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  if (col < width) {
    int32_t i = y;
    for (; i + 192 < parts; i += 256)
#pragma unroll
      for (int u = 0; u < 4; ++u) s[u] += part[(int64_t)(i + 64 * u) * width + col];
    for (; i < parts; i += 64) s[0] += part[(int64_t)i * width + col];
  }
  float sum = (s[0] + s[1]) + (s[2] + s[3]);
  sum += __shfl_xor(sum, 16, kWave);
  sum += __shfl_xor(sum, 32, kWave);
  if (lane() < kParamCols) sh[threadIdx.x / kWave][x] = sum;
  __syncthreads();
  if (y || col >= width) return;
  sum = 0.f;
  for (int i = 0; i < 16; ++i) sum += sh[i][x];
  if (col < dim) {
    if (dweight) put_param(dweight, type, col, sum);
  } else if (dbias) {
    put_param(dbias, type, col - dim, sum);
  }
}

// ---------------------------------------------------------------- host
int32_t elem_bytes(int32_t type) { return type == FS_F32 ? 4 : 2; }
bool type_known(int32_t type) { return type == FS_F32 || type == FS_BF16 || type == FS_F16; }

// strides filled in, null pointers and layouts refused
int rows_of(const void* p, int32_t type, int64_t stride, int32_t dim, NormRows* r) {
  const int32_t e = elem_bytes(type);
  r->p = (char*)p;
  r->type = type;
  r->stride = stride ? stride : (int64_t)dim * e;
  if (!p || r->stride < (int64_t)dim * e || r->stride % e || (uintptr_t)p % e) return FS_ERR_INVALID_ARG;
  return FS_OK;
}

// Workgroups that sum dweight and dbias: as many as the chip holds at once, one of
// 1024 threads a CU, two of 512, four of 256, three where a lane has 16 elements, one
// of 512 where it has more than 8 (65537 x 1000 bf16: 768 workgroups 80 us, 1024 96,
// 512 85; fewer also mean fewer sums to add).
template <int E, int L, int C>
constexpr int32_t kParts = L > 512 ? 256 : L > 256 ? (C * E > 8 ? 256 : 512) : C * E > 8 ? 768 : 1024;
constexpr int32_t kMaxParts = 1024;

// Lanes and pieces of a row by its width in pieces, calls launch.template go<E, L, C>().
// Wide rows: fewer lanes with more pieces each mean more rows under way in a CU, more
// lanes more registers for each; the last piece of a narrower row is mostly idle. us
// with 1024 lanes and with those taken: forward fp32 to bf16 16384 x 2560 82 and 47,
// 16384 x 4096 95 and 76, 8192 x 5120 90 and 46, 4096 x 8192 59 and 46; bf16 8192 x 5120
// 52 and 41, x 8192 60 and 55, x 12288 129 and 84. Backward fp32 16384 x 2560 148 and
// 84, x 4096 159 and 138, 8192 x 5120 103 and 84; bf16 8192 x 12288 174 and 133; bf16
// 8192 x 8192 86, with 512 105. The widest rows' backward sums (16 bits above 12288 columns,
// fp32 above 8192) do not fit the registers of 1024 lanes and spill: 4096 x 16384 bf16 127 us,
// 3.2 TB/s, fp32 235, 3.4; 4096 x 9000 fp32 173, 2.6.
template <int E, bool Back, typename F>
void by_width(int32_t dim, const F& launch) {
  const int32_t q = (int32_t)cdiv(dim, E);
  if (q <= 8) return launch.template go<E, 8, 1>();
  if (q <= 16) return launch.template go<E, 16, 1>();
  if (q <= 32) return launch.template go<E, 32, 1>();
  if (q <= 64) return launch.template go<E, 64, 1>();
  if (q <= 128) return launch.template go<E, 64, 2>();
  if (q <= 256) return launch.template go<E, 256, 1>();
  if (q <= 512) return launch.template go<E, 256, 2>();
  if constexpr (Back) {
    if constexpr (E == 4) {
      if (q <= 1024) return launch.template go<E, 512, 2>();
    } else {
      if (q <= 1024) return launch.template go<E, 1024, 1>();
    }
  } else {
    if (q <= 768) return launch.template go<E, 256, 3>();
    if constexpr (E == 4) {
      if (q <= 1024) return launch.template go<E, 256, 4>();
    } else {
      if (q <= 1024) return launch.template go<E, 512, 2>();
    }
  }
  if (q <= 1536) return launch.template go<E, 512, 3>();
  if constexpr (E == 4) {  // 16 bits have half as many pieces
    if constexpr (Back) {
      if (q <= 2048) return launch.template go<E, 1024, 2>();
    } else {
      if (q <= 2048) return launch.template go<E, 512, 4>();
    }
    launch.template go<E, 1024, 4>();
  } else {
    launch.template go<E, 1024, 2>();
  }
}

template <bool Back, typename F>
void by_type(const NormArgs& a, const F& launch) {
  if (a.x.type == FS_F32) by_width<4, Back>(a.dim, launch);
  else by_width<8, Back>(a.dim, launch);
}

struct Forward {
  const NormArgs& a;
  hipStream_t stream;
  template <int E, int L, int C>
  void go() const {
    constexpr int T = L > 256 ? L : 256;
    const int64_t blocks = std::min<int64_t>(cdiv(a.n, T / L), 4096);
    hipLaunchKernelGGL((k_norm<E, L, C>), dim3((unsigned)blocks), dim3(T), 0, stream, a);
  }
};

// Few rows are one workgroup's, whose sums need no second launch and no workspace:
// threads it has, or 0 where all of them share each row. There that is for up to 4 rows
// (us of a call and, in a graph, of its kernels, with a second launch and without: 4 x
// 1216 fp16 20 and 6.5, 14.5 and 6.8; 4 x 8152 20 and 14.3, 14.3 and 11.5; 8 x 8152 20
// and 14.3, 16.6 and 16.9).
template <int E, int L, int C>
constexpr int few_threads() { return L >= 256 ? 0 : C * E > 8 ? 512 : 1024; }
struct Few {
  int64_t n;
  bool* all;
  template <int E, int L, int C>
  void go() const {
    constexpr int T = few_threads<E, L, C>();
    *all = *all && (T ? cdiv(n, std::max(T, 1) / L) <= 8 : n <= 4);
  }
};

struct Backward {
  NormArgs& a;
  float* part;
  int32_t* parts;
  hipStream_t stream;
  template <int E, int L, int C>
  void go() const {
    int T = L > 256 ? L : 256;
    int64_t blocks = std::min<int64_t>(cdiv(a.n, T / L), kParts<E, L, C>);
    bool few = true;
    Few{a.n, &few}.template go<E, L, C>();
    if (few) {
      if (few_threads<E, L, C>()) T = few_threads<E, L, C>();
      blocks = 1;
    }
    blocks = std::max<int64_t>(blocks, 1);
    a.part = blocks > 1 ? part : nullptr;
    *parts = (int32_t)blocks;
    const size_t lds = T > L ? sizeof(float) * C * E * T : 0;
    if (a.out.type == FS_F32)
      hipLaunchKernelGGL((k_norm_back<E, L, C, 4>), dim3((unsigned)blocks), dim3(T), lds, stream, a);
    else
      hipLaunchKernelGGL((k_norm_back<E, L, C, 2>), dim3((unsigned)blocks), dim3(T), lds, stream, a);
  }
};

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" int fs_layer_norm(const void* x, int32_t x_dtype, int64_t x_stride, int64_t n, int32_t dim,
                             const void* weight, const void* bias, int32_t param_dtype, float eps,
                             void* out, int32_t out_dtype, int64_t out_stride, float* mean,
                             float* rstd, hipStream_t stream) {
  if (n < 0 || n >= (int64_t)INT32_MAX || dim < 1 || !type_known(x_dtype) || !type_known(out_dtype) ||
      !type_known(param_dtype) || !std::isfinite(eps) || eps < 0.f)
    return FS_ERR_INVALID_ARG;
  if (dim > FS_MAX_NORM_DIM) return FS_ERR_UNSUPPORTED;
  if (n == 0) return FS_OK;
  NormArgs a = {};
  int rc;
  if ((rc = rows_of(x, x_dtype, x_stride, dim, &a.x)) || (rc = rows_of(out, out_dtype, out_stride, dim, &a.out)))
    return rc;
  const int32_t e = elem_bytes(param_dtype);
  if ((uintptr_t)weight % e || (uintptr_t)bias % e) return FS_ERR_INVALID_ARG;
  a.n = n;
  a.weight = (const char*)weight;
  a.bias = (const char*)bias;
  a.mean = mean;
  a.rstd = rstd;
  a.dim = dim;
  a.param = param_dtype;
  a.inv_dim = 1.f / (float)dim;
  a.count = (float)dim;
  a.eps = eps;
  by_type<false>(a, Forward{a, stream});
  FS_LAUNCH_CHECK();
  return FS_OK;
}

extern "C" size_t fs_layer_norm_backward_workspace_size(int64_t n, int32_t dim) {
  if (n < 0 || dim < 1 || dim > FS_MAX_NORM_DIM) return 0;
  bool few = true;
  by_width<4, true>(dim, Few{n, &few});
  by_width<8, true>(dim, Few{n, &few});
  if (few) return 0;
  return sizeof(float) * 2 * (size_t)dim * (size_t)std::min<int64_t>(n, kMaxParts) + 256;
}

extern "C" int fs_layer_norm_backward(const void* x, int32_t x_dtype, int64_t x_stride, int64_t n,
                                      int32_t dim, const float* mean, const float* rstd,
                                      const void* dout, int32_t dout_dtype, int64_t dout_stride,
                                      const void* weight, int32_t param_dtype, void* dx,
                                      int64_t dx_stride, void* dweight, void* dbias, void* ws,
                                      size_t ws_bytes, hipStream_t stream) {
  if (n < 0 || n >= (int64_t)INT32_MAX || dim < 1 || !type_known(x_dtype) || !type_known(dout_dtype) ||
      !type_known(param_dtype))
    return FS_ERR_INVALID_ARG;
  if (dim > FS_MAX_NORM_DIM) return FS_ERR_UNSUPPORTED;
  NormArgs a = {};
  NormRows to = {};
  int rc;
  if (n > 0 && ((rc = rows_of(x, x_dtype, x_stride, dim, &a.x)) ||
                (rc = rows_of(dout, dout_dtype, dout_stride, dim, &a.out)) ||
                (rc = rows_of(dx, x_dtype, dx_stride, dim, &to))))
    return rc;
  const int32_t e = elem_bytes(param_dtype);
  if ((n > 0 && (!mean || !rstd)) || (uintptr_t)weight % e || (uintptr_t)dweight % e || (uintptr_t)dbias % e)
    return FS_ERR_INVALID_ARG;
  const size_t need = fs_layer_norm_backward_workspace_size(n, dim);
  if (need > 0 && (!ws || ws_bytes < need)) return FS_ERR_WORKSPACE;
  if (n == 0 && !dweight && !dbias) return FS_OK;
  a.dx = to.p;
  a.dx_stride = to.stride;
  a.n = n;
  a.weight = (const char*)weight;
  a.mean = (float*)mean;
  a.rstd = (float*)rstd;
  a.dweight = (char*)dweight;
  a.dbias = (char*)dbias;
  a.dim = dim;
  a.param = param_dtype;
  a.inv_dim = 1.f / (float)dim;
  a.count = (float)dim;
  a.x.type = x_dtype;
  a.out.type = dout_dtype;
  float* part = Carve(ws).take<float>(1);
  part = (float*)align_up((size_t)part, 256);
  int32_t parts = 1;
  by_type<true>(a, Backward{a, part, &parts, stream});
  FS_LAUNCH_CHECK();
  if (parts > 1 && (dweight || dbias)) {
    hipLaunchKernelGGL(k_norm_params, dim3((unsigned)cdiv(2 * (int64_t)dim, kParamCols)), dim3(1024), 0,
                       stream, part, parts, dim, (char*)dweight, (char*)dbias, param_dtype);
    FS_LAUNCH_CHECK();
  }
  return FS_OK;
}
