// Jagged softmax attention, forward, and the tile table both directions use.
//
// Sample s owns the tokens [offsets[s], offsets[s+1]); its last n_cand[s] are
// candidates. With S = scale q k^T over the keys a row sees,
//   out = softmax(S) v,   lse = log(sum exp S).
// The scores are never written: a workgroup holds 32 query rows per wave and
// passes over the keys once, in tiles of 64, with the running maximum m and
// sum l of each row (base 2):
//   m' = max(m, max S),  l = l 2^(m - m') + sum 2^(S - m'),  O = O 2^(m - m') + 2^(S - m') v.
// Bound by how far one wave's exponentials overlap another's products: at 4 x
// 8192 tokens, 4 heads of 128, causal, the kernel takes 289 us (952 TFLOP/s; a
// library product of 8192^3 reaches 1239), matrix units busy 43% and vector
// units 43% of the time at two waves per SIMD. In 128 samples of 428 tokens on
// average, 8/2 heads of 64, 67 us (22% and 56%), where loads and joins of short
// samples weigh as much.
#include <cmath>

#include "attention.hpp"

namespace fs {
namespace attn {
namespace {

constexpr int kBuckets = 256;

// One workgroup per table: one descriptor per tile of each sample, those with
// the most steps first, so that the last ones to start are short and the
// workgroups end together. A tile's steps are what a causal pass over rows t0
// + rows - 1 and before, or t0 and after, takes (tile_by_end turns one into
// the other); without causal every tile of a sample takes as many as its
// sample has. Tiles with equally many (or kBuckets and more) come in any
// order, which changes no result. Offsets that do not rise inside [0, n_tok]
// would let samples overlap (and outgrow the table): then there are no tiles.
// Threads run over tiles, not samples, so one long sample takes no longer
// than many short ones.
template <int NT>
__global__ void __launch_bounds__(NT)
k_attn_tiles(const int64_t* __restrict__ offsets, int32_t n, int64_t n_tok,
             const int32_t* __restrict__ n_cand, int32_t causal, TileTable t0, TileTable t1,
             int32_t* __restrict__ err) {
  __shared__ int32_t first[kBuckets], tmp[17];
  __shared__ int32_t s_lo[NT], s_len[NT], s_cand[NT];
  __shared__ int32_t s_at[NT + 1];
  const TileTable t = blockIdx.x ? t1 : t0;
  bool bad = false, order = true;
  static_assert(NT >= kBuckets, "a thread per bucket");
  if (threadIdx.x < kBuckets) first[threadIdx.x] = 0;
  for (int32_t s = threadIdx.x; s < n; s += NT)
    order &= offsets[s] >= 0 && offsets[s] <= offsets[s + 1] && offsets[s + 1] <= n_tok;
  if (__syncthreads_or(!order)) {
    flag_err(err, !order, FS_EF_SHAPE);
    if (threadIdx.x == 0) *t.n = 0;
    return;
  }
  // pass 0 counts the tiles of each bucket, pass 1 places them
  for (int pass = 0; pass < 2; ++pass) {
    for (int32_t c0 = 0; c0 < n; c0 += NT) {  // uniform
      const int32_t s = c0 + threadIdx.x, left = min(n - c0, NT);
      if (n > NT || pass == 0) {  // one chunk stays in LDS for the second pass
        int32_t lo = 0, len = 0, cand = 0;
        if (s < n) {
          lo = (int32_t)offsets[s];
          len = (int32_t)(offsets[s + 1] - lo);
          cand = n_cand ? n_cand[s] : 0;
          bad |= cand < 0 || cand > len;
          cand = min(max(cand, 0), len);
        }
        int32_t total;
        const int32_t at = block_excl_scan<int32_t>((int32_t)cdiv(len, t.rows), tmp, &total);
        s_lo[threadIdx.x] = lo;
        s_len[threadIdx.x] = len;
        s_cand[threadIdx.x] = cand;
        s_at[threadIdx.x] = at;
        if (threadIdx.x == 0) s_at[NT] = total;
        __syncthreads();
      }
      for (int32_t e = threadIdx.x; e < s_at[NT]; e += NT) {
        int32_t a = 0, b = left - 1;  // the last sample that starts at or before tile e
        while (a < b) {
          const int32_t mid = (a + b + 1) >> 1;
          if (s_at[mid] <= e) a = mid; else b = mid - 1;
        }
        const int32_t len = s_len[a], k = e - s_at[a], cnt = (int32_t)cdiv(len, t.rows);
        const int32_t at = atomicAdd(&first[kBuckets - min(causal ? cnt - k : cnt, kBuckets)], 1);
        if (pass) t.tiles[at] = Tile{s_lo[a], len, len - s_cand[a], k * t.rows};
      }
      __syncthreads();
    }
    if (pass == 0) {
      int32_t total;
      const int32_t x = threadIdx.x < kBuckets ? first[threadIdx.x] : 0;
      const int32_t ex = block_excl_scan<int32_t>(x, tmp, &total);
      if (threadIdx.x < kBuckets) first[threadIdx.x] = ex;
      if (threadIdx.x == 0) *t.n = total;
      __syncthreads();
    }
  }
  flag_err(err, bad, FS_EF_SHAPE);
}

struct FwdArgs {
  Shape s;
  View q, k, v, o;
  float* lse;
};

constexpr int kKeys = 64;    // keys per step
// A row's running maximum m moves where 2^(S - m) would pass 2^kMost, to where
// its largest is 2^kTo. fp16's largest value is just below 2^16 and its smallest
// step 2^-24, so there the largest stays in 2^8 .. 2^15: what lies 2^22 below it
// and more is rounded to a multiple of 2^-32 of it, not to one of 2^-24.
template <typename T>
constexpr float kMost = Elem<T>::kNarrow ? 15.f : 8.f;
template <typename T>
constexpr float kTo = Elem<T>::kNarrow ? 8.f : 0.f;

template <typename T, int DP, int NW>
__global__ void __launch_bounds__(NW * kWave, 2) k_attn_fwd(FwdArgs a) {
  constexpr int NT = NW * kWave;
  __shared__ __attribute__((aligned(kTileAlign))) uint16_t sk[2][kKeys * DP], sv[2][kKeys * DP];
  static_assert(__alignof__(sk) >= kTileAlign && __alignof__(sv) >= kTileAlign, "16-byte pieces");
  __shared__ __attribute__((aligned(16))) float s_off[2][kKeys];
  const int l = lane(), w = wave_id(), g = l >> 5;
  const int rows = 32 * NW / a.s.pack, packs = a.s.heads / a.s.pack;  // see pack_of
  const int at = blockIdx.x / packs, head = blockIdx.x % packs * a.s.pack + w % a.s.pack;
  const Tile entry = a.s.tab.tiles[at];  // in the table's memory, beside the count
  if (at >= *a.s.tab.n) return;
  const Tile t = tile_by_end(entry, rows);
  const int kvh = head / a.s.group;
  const char* kp = a.k.p + kvh * a.k.head;
  const char* vp = a.v.p + kvh * a.v.head;
  const int t1 = min(t.t0 + rows, t.len);  // the workgroup's rows: [t0, t1)
  const int i0 = t.t0 + 32 * (w / a.s.pack), i = i0 + (l & 31);
  const bool on = live_row(a.s, t, i);
  const bool causal = a.s.causal != 0;

  u32x4 qf[DP / 16];
  load_scaled_columns<DP>(qf, a.q.p + head * a.q.head, a.q.tok, a.s, t, i);
  f32x16 o[DP / 32];
#pragma unroll
  for (int d = 0; d < DP / 32; ++d) o[d] = zero16();
  // finite, so that a row that sees nothing keeps 2^(-inf - m) = 0
  float m = -3e38f, sum = 0.f;
  const float c = log2_scale(a.s);
  const Operands<DP> op;

  // key tiles: the history, then the workgroup's own candidates
  const int hist_end = (int)cdiv(causal ? min(t.hist, t1) : t.hist, kKeys);
  const int own_lo = max(hist_end, max(t.t0, t.hist) / kKeys);
  const int own_end = t1 > t.hist ? (int)cdiv(t1, kKeys) : 0;
  const int steps = hist_end + max(0, own_end - own_lo);
  auto key0 = [&](int step) { return (step < hist_end ? step : own_lo + step - hist_end) * kKeys; };

  using Tiles = Direct<DP, NT>;
  // The bytes that say which keys are live are read two steps ahead and made
  // bits one step ahead, before the next tiles are asked for: made after the
  // tiles' wait, as in the backward pass, they cost this kernel 5% (302 against
  // 318 us on 4 x 8192 tokens, 4 heads of 128).
  uint64_t keys = 0;
  uint32_t ahead = 0;
  auto load = [&](int step) {
    const int j = key0(step);
    keys = live_bits(ahead);
    Tiles::load(sk[step & 1], kp, a.k.tok, a.s, t, j);
    Tiles::load(sv[step & 1], vp, a.v.tok, a.s, t, j);
    if (step + 1 < steps) ahead = live_byte(a.s, t, key0(step + 1));
  };
  if (steps > 0) {
    ahead = live_byte(a.s, t, key0(0));
    load(0);
  }
  for (int step = 0; step < steps; ++step) {
    const int j0 = key0(step), b = step & 1;
    const uint64_t live = keys;
    Tiles::wait();
    Tiles::finish(sk[b], a.s, live);
    Tiles::finish(sv[b], a.s, live);
    if (live != ~0ull) store_off(s_off[b], live);
    __syncthreads();
    if (step + 1 < steps) load(step + 1);
    // tiles that none of this wave's rows sees
    const bool past = causal ? j0 > i0 + 31 : j0 >= t.hist;
    if (i0 >= t1 || (past && (j0 > i0 + 31 || j0 + kKeys <= i0))) continue;
    const bool whole = j0 + kKeys <= t.hist && (!causal || j0 + kKeys <= i0 + 1);
    f32x16 s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      // both start a product, the first with a zero that takes no registers
      if (live == ~0ull)
        s[kb] = Elem<T>::mfma(op.rows(sk[b], 32 * kb, 0), qf[0], zero16());
      else
        s[kb] = Elem<T>::mfma(op.rows(sk[b], 32 * kb, 0), qf[0], load_off(s_off[b], 32 * kb));
#pragma unroll
      for (int kk = 1; kk < DP / 16; ++kk)
        s[kb] = Elem<T>::mfma(op.rows(sk[b], 32 * kb, kk), qf[kk], s[kb]);
    }
    if (!whole) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        const uint32_t see = seen_keys(i, j0 + 32 * kb, t.hist, causal) >> (4 * g);
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (!((see >> (8 * (x >> 2) + (x & 3))) & 1u)) s[kb][x] = -INFINITY;
      }
    }
    float top = s[0][0];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int x = 0; x < 16; ++x) top = fmaxf(top, s[kb][x]);
    top = max_halves(top) * c;
    // The running maximum only has to keep 2^(S - m) in range: it moves when a
    // row passes it by more than kMost, so the sums are rescaled in few steps
    // instead of nearly all (some of 32 rows has a new maximum in most).
    if (__any(top > m + kMost<T>)) {
      // rows that need not move keep theirs: a row's bits depend on no other row
      const float to = top > m + kMost<T> ? top - kTo<T> : m, f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      sum *= f;
#pragma unroll
      for (int d = 0; d < DP / 32; ++d) o[d] *= f;
    }
    float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        s[kb][x] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kb][x], c, -m));
        part[x & 3] += s[kb][x];
      }
    sum += (part[0] + part[1]) + (part[2] + part[3]);
    // probabilities are rounded to the operand's type (half a step each)
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const u32x4 p = to_operand<T>(s[kb], ch);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
          o[d] = Elem<T>::mfma(op.cols(sv[b], 32 * kb + 16 * ch, 32 * d), p, o[d]);
      }
  }
  if (i >= t.len) return;
  sum = add_halves(sum);
  if (!on) {  // a row that is not live has summed what it does not see
    sum = 0.f;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) o[d] = zero16();
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // a sum that is NaN stays NaN
  char* dst = a.o.p + head * a.o.head + ((int64_t)t.lo + i) * a.o.tok;
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int col = 32 * d + 8 * x + 4 * g;
      if (col < a.s.dim) {
        u32x2 v;
        v[0] = Elem<T>::pack(o[d][4 * x] * inv, o[d][4 * x + 1] * inv);
        v[1] = Elem<T>::pack(o[d][4 * x + 2] * inv, o[d][4 * x + 3] * inv);
        *(u32x2*)(dst + 2 * col) = v;
      }
    }
  if (g == 0)
    a.lse[(int64_t)head * a.s.n_tok + t.lo + i] =
        sum == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <typename T>
void launch_fwd(const FwdArgs& a, dim3 grid, hipStream_t stream) {
  constexpr int NW = 4;
  if (padded(a.s.dim) == 32)
    hipLaunchKernelGGL((k_attn_fwd<T, 32, NW>), grid, dim3(NW * kWave), 0, stream, a);
  else if (padded(a.s.dim) == 64)
    hipLaunchKernelGGL((k_attn_fwd<T, 64, NW>), grid, dim3(NW * kWave), 0, stream, a);
  else
    hipLaunchKernelGGL((k_attn_fwd<T, 128, NW>), grid, dim3(NW * kWave), 0, stream, a);
}

}  // namespace

int make_view(const fs_heads* x, int32_t heads, int32_t dim, View* v) {
  if (!x) return FS_ERR_INVALID_ARG;
  const int64_t row = (int64_t)dim * 2;
  v->p = (char*)x->data;
  v->head = x->head_stride ? x->head_stride : row;
  v->tok = x->token_stride ? x->token_stride : row * heads;
  if (v->tok > kMaxStride || v->head > ((int64_t)1 << 40)) return FS_ERR_UNSUPPORTED;
  if (v->head < 0 || v->tok < 0 || (v->head & 15) || (v->tok & 15) || ((uintptr_t)v->p & 15))
    return FS_ERR_INVALID_ARG;
  if (v->tok < row || (heads > 1 && v->head < row)) return FS_ERR_INVALID_ARG;
  return FS_OK;
}

int launch_tiles(const int64_t* offsets, int32_t n, int64_t n_tok, const int32_t* n_cand,
                 int32_t causal, const TileTable* t, int32_t tables, int32_t* err,
                 hipStream_t stream) {
  // few samples and tiles: barriers of four waves instead of sixteen (6.3 -> 5.0 us)
  if (n <= 256 && tile_cap(n_tok, n, t[0].rows) <= 1024)
    hipLaunchKernelGGL(k_attn_tiles<256>, dim3((unsigned)tables), dim3(256), 0, stream, offsets, n,
                       n_tok, n_cand, causal, t[0], t[tables - 1], err);
  else
    hipLaunchKernelGGL(k_attn_tiles<1024>, dim3((unsigned)tables), dim3(1024), 0, stream, offsets, n,
                       n_tok, n_cand, causal, t[0], t[tables - 1], err);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

}  // namespace attn
}  // namespace fs

using namespace fs;
using namespace fs::attn;

extern "C" size_t fs_jagged_attention_workspace_size(int64_t n_tok, int32_t n) {
  if (n_tok < 0 || n < 0) return 0;
  Carve c(nullptr);
  c.take<int32_t>(1);
  c.take<Tile>((size_t)tile_cap(n_tok, n, 32));
  return c.used + 256;
}

extern "C" int fs_jagged_attention(const fs_heads* q, const fs_heads* k, const fs_heads* v,
                                   const int64_t* offsets, int32_t n, int64_t n_tok,
                                   const int32_t* n_cand, const uint8_t* valid, int32_t heads,
                                   int32_t kv_heads, int32_t dim, int32_t dtype, int32_t causal,
                                   float scale, const fs_heads* out, float* lse, int32_t* err,
                                   void* ws, size_t ws_bytes, hipStream_t stream) {
  if (n < 0 || n > FS_MAX_SAMPLES || n_tok < 0 || n_tok >= (int64_t)INT32_MAX || heads < 1 ||
      kv_heads < 1 || heads % kv_heads || !offsets || !scale_ok(scale))
    return FS_ERR_INVALID_ARG;
  if (!type_ok(dtype) || dim < 8 || dim > 128 || dim % 8 || heads > FS_MAX_HEADS)
    return FS_ERR_UNSUPPORTED;
  FwdArgs a;
  int rc;
  if ((rc = make_view(q, heads, dim, &a.q)) || (rc = make_view(k, kv_heads, dim, &a.k)) ||
      (rc = make_view(v, kv_heads, dim, &a.v)) || (rc = make_view(out, heads, dim, &a.o)))
    return rc;
  if (n_tok > 0 && n > 0 && (!a.q.p || !a.k.p || !a.v.p || !a.o.p || !lse))
    return FS_ERR_INVALID_ARG;
  if (!ws || ws_bytes < fs_jagged_attention_workspace_size(n_tok, n)) return FS_ERR_WORKSPACE;
  if (n == 0 || n_tok == 0) return FS_OK;
  const int32_t pack = pack_of(heads / kv_heads), rows = 128 / pack;
  const int64_t cap = tile_cap(n_tok, n, rows), grid = cap * (heads / pack);
  if (!grid_fits(grid, 256)) return FS_ERR_UNSUPPORTED;
  Carve c(ws);
  TileTable tab;
  tab.rows = rows;
  tab.n = c.take<int32_t>(1);
  tab.tiles = c.take<Tile>((size_t)cap);
  if ((rc = launch_tiles(offsets, n, n_tok, n_cand, causal, &tab, 1, err, stream))) return rc;
  a.s = Shape{tab, valid, n_tok, heads, heads / kv_heads, pack, dim, causal, scale};
  a.lse = lse;
  if (dtype == FS_BF16)
    launch_fwd<__bf16>(a, dim3((unsigned)grid), stream);
  else
    launch_fwd<_Float16>(a, dim3((unsigned)grid), stream);
  FS_LAUNCH_CHECK();
  return FS_OK;
}
