// Jagged softmax attention, backward. The probabilities are recomputed from
// the forward pass's log-sum-exp:
//   P = exp(S - lse),  delta_i = sum_d dO_id O_id,  dP = dO v^T,
//   dS = P (dP - delta),  dV = P^T dO,  dQ = scale dS k,  dK = scale dS^T q.
//
// Two kernels, because dQ sums over keys and dK, dV over rows: each keeps its
// sums in registers and recomputes S and dP (7 products instead of the least
// 5), so no sum crosses workgroups, nothing is added atomically and equal
// calls give equal bits. The first writes delta for the second. Bound as the
// forward pass is: at 2 x 8192 tokens, 8/2 heads of 128, causal, bf16, the
// kernels take 406 us for dQ (matrix units busy 48% of the time), 605 for dK and
// dV (35%) and 16 for the sum of parts, where the seven products would take 777
// at a library product's rate; in 128 samples of 428 tokens on average, 8/2
// heads of 64, 102 us (24%) and 117 (26%).
#include <algorithm>
#include <cmath>

#include "attention.hpp"

namespace fs {
namespace attn {
namespace {

constexpr int kStep = 64;  // rows or keys per step

struct BwdArgs {
  Shape s;
  View q, k, v, o, d_o, dq, dk, dv;
  TileTable keys;    // 128 keys each
  const float* lse;  // [heads][n_tok]
  float* delta;      // [heads][n_tok]
  float* factor;     // [heads][n_tok], fp16: of every 32 rows of a sample, see kDsTop
  float* part;       // [splits][2][kv_heads][n_tok][DP]: dK (unscaled) and dV
  int32_t splits;
};

// The grid of the dK / dV kernel is one workgroup per 128 keys and key head.
// Causal tiles differ in length by up to the sample's, so with fewer than
// about two workgroups per CU the longest one decides; then each tile's steps
// are cut into equal parts, whose sums a second kernel adds in order. Measured
// at 2 x 8192 tokens, 8/2 heads of 128 (256 tiles): 2028 us whole, 1103 and 16
// for the sum in two parts; in 64 short samples (5644 tokens, one key head)
// eight parts take 15 and 6 us, one 20, and a launch less.
constexpr int64_t kParts = 512;   // workgroups to reach
constexpr int64_t kSplitMax = 8;  // parts of one tile
constexpr int64_t kPartSteps = 4;  // steps that a part of a tile of average length has, at least
__host__ inline int32_t splits_of(int64_t n_tok, int32_t n, int32_t kv_heads, int32_t group) {
  const int64_t tiles = std::max<int64_t>(1, n_tok / 128 * kv_heads);
  const int64_t steps = n_tok / n * group / kStep;
  return (int32_t)std::max<int64_t>(1, std::min({kSplitMax, cdiv(kParts, tiles), steps / kPartSteps}));
}
// The most tokens times splits of any call with at most n_tok tokens: a call
// has s splits or more while its tiles are at most (kParts - 1) / (s - 1).
__host__ inline int64_t split_tokens(int64_t n_tok, int32_t kv_heads) {
  int64_t most = 0;
  for (int64_t s = 2; s <= kSplitMax; ++s)
    most = std::max(most, s * std::min(n_tok, ((kParts - 1) / (s - 1) / kv_heads + 1) * 128 - 1));
  return most;
}

// fp16 has 5 bits of exponent, and P and dS leave its range where inputs and
// outputs do not: P is about 1 / length, dS = P (dP - delta) that times the size
// of a gradient. So both are rounded times a power of two that the sums lose
// again (bf16 has fp32's exponents and needs none):
//  - P of dV times 2^kPUp;
//  - dS of dQ times a row's own factor, which is a lane's: it takes the largest
//    of the row's dS so far to 2^(kDsTop - 2) .. 2^kDsTop, and moves (with the
//    sums) where one passes 2^kDsMost. It starts from delta, so that a row
//    whose dS cancel to rounding errors of delta has a factor for these too;
//  - dS of dK and dV's kernel times one factor per tile of keys, from the
//    smallest of the rows that meet it, which the dQ kernel leaves for every 32
//    rows: dS is at most 2^kDsMost over that factor, up to the two kernels'
//    rounding of P, which has three bits here.
// What is too small for fp16 even so is rounded to a multiple of 2^-24, off by
// at most 2^-25: 2^-37 of P's 1, of dS 2^-36 of the row's largest (dQ) or 2^-34
// of the largest of the rows that the tile meets (dK). Measured against dS and
// P rounded as they are, which at gradients of 1e-4 over thousands of tokens are
// off by several percent: whole calls take 240 us instead of 229 (128 samples,
// 8/2 heads of 64), 1094 instead of 1051 (2 x 8192 tokens, 8/2 heads of 128) and
// 36 instead of 34 (64 short samples, 2/1 heads of 40): a row's largest dS is
// looked for at every step.
constexpr int kPUp = 12, kDsTop = 13, kDsMost = 15;
constexpr int kFactorMost = 60;  // bits of a factor: products with dP stay inside fp32

__device__ __forceinline__ int factor_bits(int bits) {
  return min(max(bits, -kFactorMost), kFactorMost);
}
__device__ __forceinline__ float wave_min(float x) {
#pragma unroll
  for (int d = kWave / 2; d > 0; d >>= 1) x = fminf(x, __shfl_xor(x, d, kWave));
  return x;
}

// The factor of dS for the rows [r0, r1) of a sample (r0 a multiple of 32) and a
// key head's query heads
__device__ __forceinline__ float rows_factor(const BwdArgs& a, const Tile& t, int kvh, int r0,
                                             int r1) {
  const int per = (int)cdiv(r1 - r0, 32);
  float f = INFINITY;
#pragma unroll 4
  for (int x = lane(); x < per * a.s.group; x += kWave)
    f = fminf(f, a.factor[(int64_t)(kvh * a.s.group + x / per) * a.s.n_tok + t.lo + r0 + x % per * 32]);
  f = wave_min(f);
  // times 2^kPUp, which comes with P
  return f == INFINITY ? 1.f : ldexpf(f, kDsTop - kDsMost - kPUp);
}

// 32 columns x DP rows of sums to one row of memory per lane, scaled
template <typename T, int DP>
__device__ __forceinline__ void store_rows(char* row, const f32x16 (&x)[DP / 32], int dim,
                                           float f) {
  const int g = lane() >> 5;
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int col = 32 * d + 8 * y + 4 * g;
      if (col < dim) {
        u32x2 v;
        v[0] = Elem<T>::pack(x[d][4 * y] * f, x[d][4 * y + 1] * f);
        v[1] = Elem<T>::pack(x[d][4 * y + 2] * f, x[d][4 * y + 3] * f);
        *(u32x2*)(row + 2 * col) = v;
      }
    }
}

// dQ: 32 rows per wave, keys in steps. S^T = k q^T and dP^T = v dO^T have one
// row per lane, so lse and delta are one register each and dS^T is the operand
// of dQ^T = k^T dS^T.
template <typename T, int DP, int NW>
__global__ void __launch_bounds__(NW * kWave, DP == 128 ? 2 : 3) k_attn_dq(BwdArgs a) {
  constexpr int NT = NW * kWave;
  __shared__ __attribute__((aligned(kTileAlign))) uint16_t sk[2][kStep * DP], sv[2][kStep * DP];
  static_assert(__alignof__(sk) >= kTileAlign && __alignof__(sv) >= kTileAlign, "16-byte pieces");
  __shared__ __attribute__((aligned(16))) float s_off[2][kStep];
  const int l = lane(), w = wave_id(), g = l >> 5;
  const int rows = 32 * NW / a.s.pack, packs = a.s.heads / a.s.pack;  // see pack_of
  const int at = blockIdx.x / packs, head = blockIdx.x % packs * a.s.pack + w % a.s.pack;
  const Tile entry = a.s.tab.tiles[at];  // in the table's memory, beside the count
  if (at >= *a.s.tab.n) return;
  const Tile t = tile_by_end(entry, rows);
  const int kvh = head / a.s.group;
  const char* kp = a.k.p + kvh * a.k.head;
  const char* vp = a.v.p + kvh * a.v.head;
  const int t1 = min(t.t0 + rows, t.len);
  const int i0 = t.t0 + 32 * (w / a.s.pack), i = i0 + (l & 31);
  const bool on = live_row(a.s, t, i);
  const bool causal = a.s.causal != 0;

  u32x4 qf[DP / 16], df[DP / 16];
  load_scaled_columns<DP>(qf, a.q.p + head * a.q.head, a.q.tok, a.s, t, i);
  load_columns<DP>(df, a.d_o.p + head * a.d_o.head, a.d_o.tok, a.s, t, i);
  // delta, the diagonal of out dO^T: by the product that makes dP, in its order,
  // so that a row that sees itself alone, whose out is its v, has delta = dP to
  // the bit and dS = 0, whatever its P of about 1 is
  float delta = 0.f;
  {
    const char* outp = a.o.p + head * a.o.head;
    f32x16 x = zero16();
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      u32x4 o = load_piece(outp, a.o.tok, a.s, t, i, 2 * kk + g);
      if (8 * (2 * kk + g) >= a.s.dim) o = u32x4{0, 0, 0, 0};
      x = Elem<T>::mfma(o, df[kk], x);
    }
#pragma unroll
    for (int y = 0; y < 16; ++y)  // row l & 31 of the diagonal is in one of the halves
      if ((l & 31) == 8 * (y >> 2) + 4 * g + (y & 3)) delta = x[y];
    delta = add_halves(delta);
  }
  // a row that sees nothing has lse = -inf: 2^(S - inf) = 0
  float lse = INFINITY;
  const int64_t lse_at = (int64_t)head * a.s.n_tok + t.lo + i;
  if (on) lse = a.lse[lse_at];
  lse = lse == -INFINITY ? INFINITY : lse * kLog2e;
  const float c = log2_scale(a.s);
  const Operands<DP> op;

  const int hist_end = (int)cdiv(causal ? min(t.hist, t1) : t.hist, kStep);
  const int own_lo = max(hist_end, max(t.t0, t.hist) / kStep);
  const int own_end = t1 > t.hist ? (int)cdiv(t1, kStep) : 0;
  const int steps = hist_end + max(0, own_end - own_lo);
  auto key0 = [&](int step) { return (step < hist_end ? step : own_lo + step - hist_end) * kStep; };
  // The scores of 32 keys of a staged tile and their dP, masked
  auto scores = [&](int j0, int b, int kb, uint64_t live, f32x16& s, f32x16& dp) {
    s = live == ~0ull ? zero16() : load_off(s_off[b], 32 * kb);
    dp = zero16();
#pragma unroll
    for (int kk = 0; kk < DP / 16; ++kk) {
      s = Elem<T>::mfma(op.rows(sk[b], 32 * kb, kk), qf[kk], s);
      dp = Elem<T>::mfma(op.rows(sv[b], 32 * kb, kk), df[kk], dp);
    }
    if (j0 + kStep > t.hist || (causal && j0 + kStep > i0 + 1)) {
      const uint32_t see = seen_keys(i, j0 + 32 * kb, t.hist, causal) >> (4 * g);
#pragma unroll
      for (int x = 0; x < 16; ++x)
        if (!((see >> (8 * (x >> 2) + (x & 3))) & 1u)) s[x] = -INFINITY;
    }
  };

  using Tiles = Direct<DP, NT>;
  // delta comes with the rounding of out to 16 bits. Where a row sees few keys,
  // out is as large as v and that is as much as all of dS's own rounding: rows
  // of at most two steps sum delta = sum_j P_ij dP_ij first, in fp32, unless they
  // see one key.
  if (steps <= 2) {
    float sum = 0.f;
    int seen = 0;
    for (int step = 0; step < steps; ++step) {
      const int j0 = key0(step);
      Tiles::load(sk[0], kp, a.k.tok, a.s, t, j0);
      Tiles::load(sv[0], vp, a.v.tok, a.s, t, j0);
      const uint32_t byte = live_byte(a.s, t, j0);
      Tiles::wait();
      const uint64_t live = live_bits(byte);
      Tiles::finish(sk[0], a.s, live);
      Tiles::finish(sv[0], a.s, live);
      if (live != ~0ull) store_off(s_off[0], live);
      __syncthreads();
#pragma unroll 1
      for (int kb = 0; kb < 2; ++kb) {
        f32x16 s, dp;
        scores(j0, 0, kb, live, s, dp);
#pragma unroll
        for (int x = 0; x < 16; ++x)
          sum = __builtin_fmaf(__builtin_amdgcn_exp2f(__builtin_fmaf(s[x], c, -lse)), dp[x], sum);
        seen += __popc(seen_keys(i, j0 + 32 * kb, t.hist, causal) & (uint32_t)(live >> (32 * kb)));
      }
      __syncthreads();
    }
    sum = add_halves(sum);
    if (seen != 1) delta = sum;
  }
  if (g == 0 && i < t.len) a.delta[lse_at] = delta;
  f32x16 dq[DP / 32];
#pragma unroll
  for (int d = 0; d < DP / 32; ++d) dq[d] = zero16();
  // fp16: the row's factor 2^up, and whether no dS other than 0 has come yet
  int up = 0;
  bool fresh = true;
  if (Elem<T>::kNarrow && delta != 0.f) {
    up = factor_bits(kDsMost + kDsTop - 1 - __builtin_amdgcn_frexp_expf(delta));
    fresh = false;
  }
  float factor = ldexpf(1.f, up), scaled_delta = delta * factor;

  uint32_t live_of = 0;
  auto load = [&](int step) {
    const int j = key0(step);
    Tiles::load(sk[step & 1], kp, a.k.tok, a.s, t, j);
    Tiles::load(sv[step & 1], vp, a.v.tok, a.s, t, j);
    live_of = live_byte(a.s, t, j);
  };
  if (steps > 0) load(0);
  for (int step = 0; step < steps; ++step) {
    const int j0 = key0(step), b = step & 1;
    Tiles::wait();
    const uint64_t live = live_bits(live_of);
    Tiles::finish(sk[b], a.s, live);
    Tiles::finish(sv[b], a.s, live);
    if (live != ~0ull) store_off(s_off[b], live);
    __syncthreads();
    if (step + 1 < steps) load(step + 1);
    const bool past = causal ? j0 > i0 + 31 : j0 >= t.hist;
    if (i0 >= t1 || (past && (j0 > i0 + 31 || j0 + kStep <= i0))) continue;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb) {
      f32x16 s, dp;
      scores(j0, b, kb, live, s, dp);
#pragma unroll
      for (int x = 0; x < 16; ++x)
        s[x] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x], c, -lse)) *
               (Elem<T>::kNarrow ? __builtin_fmaf(dp[x], factor, -scaled_delta) : dp[x] - delta);
      if constexpr (Elem<T>::kNarrow) {
        float top = 0.f;
#pragma unroll
        for (int x = 0; x < 16; ++x) top = fmaxf(top, fabsf(s[x]));
        top = max_halves(top);
        const bool move = top > (float)(1 << kDsMost) || (fresh && top > 0.f);
        if (__any(move)) {
          const int to = move ? factor_bits(up + kDsTop - __builtin_amdgcn_frexp_expf(top)) : up;
          const float by = ldexpf(1.f, to - up);
          s *= by;
#pragma unroll
          for (int d = 0; d < DP / 32; ++d) dq[d] *= by;
          up = to;
          factor = ldexpf(1.f, up);
          scaled_delta = delta * factor;
          fresh = fresh && !move;
        }
      }
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const u32x4 ds = to_operand<T>(s, ch);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
          dq[d] = Elem<T>::mfma(op.cols(sk[b], 32 * kb + 16 * ch, 32 * d), ds, dq[d]);
      }
    }
  }
  if constexpr (Elem<T>::kNarrow) {
    const float least = wave_min(on && !fresh ? factor : INFINITY);
    if (l == 0 && i0 < t.len) a.factor[(int64_t)head * a.s.n_tok + t.lo + i0] = least;
  }
  if (i >= t.len) return;
  if (!on) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) dq[d] = zero16();
  }
  store_rows<T, DP>(a.dq.p + head * a.dq.head + ((int64_t)t.lo + i) * a.dq.tok, dq, a.s.dim,
                    ldexpf(a.s.scale, -up));
}

// dK and dV: 32 keys per wave, the rows of every query head of the key head
// in steps. S = q k^T and dP = dO v^T have one key per lane, so P and dS are
// the operands of dV^T = dO^T P and dK^T = q^T dS.
template <typename T, int DP, int NW>
__global__ void __launch_bounds__(NW * kWave, DP == 64 ? 2 : 3) k_attn_dkv(BwdArgs a) {
  constexpr int NT = NW * kWave;
  __shared__ __attribute__((aligned(kTileAlign))) uint16_t sq[2][kStep * DP], sd[2][kStep * DP];
  static_assert(__alignof__(sq) >= kTileAlign && __alignof__(sd) >= kTileAlign, "16-byte pieces");
  __shared__ __attribute__((aligned(16))) float s_lse[2][kStep], s_delta[2][kStep];
  const int kv_heads = a.s.heads / a.s.group;
  const int kvh = blockIdx.x % kv_heads, part = blockIdx.x / kv_heads % a.splits;
  const int at = blockIdx.x / kv_heads / a.splits;
  const Tile t = a.keys.tiles[at];
  if (at >= *a.keys.n) return;
  const int l = lane(), w = wave_id(), g = l >> 5;
  const int t1 = min(t.t0 + 32 * NW, t.len);
  const int j0 = t.t0 + 32 * w, j = j0 + (l & 31);
  const bool on = live_row(a.s, t, j);
  const bool causal = a.s.causal != 0;

  u32x4 kf[DP / 16], vf[DP / 16];
  load_scaled_columns<DP>(kf, a.k.p + kvh * a.k.head, a.k.tok, a.s, t, j);
  load_columns<DP>(vf, a.v.p + kvh * a.v.head, a.v.tok, a.s, t, j);
  f32x16 dk[DP / 32], dv[DP / 32];
#pragma unroll
  for (int d = 0; d < DP / 32; ++d) dk[d] = dv[d] = zero16();
  const float c = log2_scale(a.s);
  const Operands<DP> op;

  // rows that see a key of this tile: from the tile on where causal, all of
  // them otherwise; only its own where it holds candidates alone
  const bool own = t.t0 >= t.hist;
  const int first = (own || causal ? t.t0 : 0) / kStep;
  const int last = (int)cdiv(own ? t1 : t.len, kStep);
  const int per = last - first, all = per * a.s.group;
  const int step0 = (int)((int64_t)all * part / a.splits);
  const int steps = (int)((int64_t)all * (part + 1) / a.splits);

  using Tiles = Direct<DP, NT>;
  uint32_t live_of = 0;
  float st_lse = INFINITY, st_delta = 0.f;  // threads 0 .. 63: one row each
  auto row0 = [&](int step) { return (first + step % per) * kStep; };
  auto load = [&](int step) {
    const int head = kvh * a.s.group + step / per, i0 = row0(step);
    Tiles::load(sq[step & 1], a.q.p + head * a.q.head, a.q.tok, a.s, t, i0);
    Tiles::load(sd[step & 1], a.d_o.p + head * a.d_o.head, a.d_o.tok, a.s, t, i0);
    if (threadIdx.x < kStep) {
      const int i = min(i0 + (int)threadIdx.x, t.len - 1);
      const int64_t at = (int64_t)head * a.s.n_tok + t.lo + i;
      st_lse = a.lse[at];
      st_delta = a.delta[at];
    }
    live_of = live_byte(a.s, t, i0);
  };
  if (step0 < steps) load(step0);
  // beside the first tiles' way
  const float factor =
      Elem<T>::kNarrow ? rows_factor(a, t, kvh, first * kStep, own ? t1 : t.len) : 1.f;
  constexpr float p_up = Elem<T>::kNarrow ? kPUp : 0;
  for (int step = step0; step < steps; ++step) {
    const int i0 = row0(step), b = step & 1;
    Tiles::wait();
    const uint64_t live = live_bits(live_of);
    Tiles::finish(sq[b], a.s, live);
    Tiles::finish(sd[b], a.s, live);
    if (threadIdx.x < kStep) {
      const bool in = (live >> threadIdx.x) & 1;
      s_lse[b][threadIdx.x] = !in || st_lse == -INFINITY ? INFINITY : st_lse * kLog2e - p_up;
      s_delta[b][threadIdx.x] = in ? st_delta * factor : 0.f;
    }
    __syncthreads();
    if (step + 1 < steps) load(step + 1);
    // steps whose rows see none of this wave's keys
    if (j0 >= t1 || (causal && i0 + kStep <= j0)) continue;
    if (j0 >= t.hist && (i0 + kStep <= j0 || i0 > j0 + 31)) continue;
    // rows that are not live have lse = inf, so P = 0; keys that are not live
    // spoil only their own column, which is not stored
    const bool whole = j0 + 32 <= t.hist && (!causal || i0 >= j0 + 31);
#pragma unroll
    for (int ib = 0; ib < 2; ++ib) {
      f32x16 s = zero16(), dp = zero16();
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        s = Elem<T>::mfma(op.rows(sq[b], 32 * ib, kk), kf[kk], s);
        dp = Elem<T>::mfma(op.rows(sd[b], 32 * ib, kk), vf[kk], dp);
      }
      if (!whole) {
        const uint32_t see = seeing_rows(j, i0 + 32 * ib, t.hist, causal) >> (4 * g);
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (!((see >> (8 * (x >> 2) + (x & 3))) & 1u)) s[x] = -INFINITY;
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const f32x4 ls = *(const f32x4*)&s_lse[b][32 * ib + 8 * y + 4 * g];
        const f32x4 de = *(const f32x4*)&s_delta[b][32 * ib + 8 * y + 4 * g];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int z = 4 * y + x;
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[z], c, -ls[x]));
          s[z] = p;
          dp[z] = p * (Elem<T>::kNarrow ? __builtin_fmaf(dp[z], factor, -de[x]) : dp[z] - de[x]);
        }
      }
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const u32x4 pb = to_operand<T>(s, ch), db = to_operand<T>(dp, ch);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d) {
          dv[d] = Elem<T>::mfma(op.cols(sd[b], 32 * ib + 16 * ch, 32 * d), pb, dv[d]);
          dk[d] = Elem<T>::mfma(op.cols(sq[b], 32 * ib + 16 * ch, 32 * d), db, dk[d]);
        }
      }
    }
  }
  if (j >= t.len) return;
  if (!on) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) dk[d] = dv[d] = zero16();
  }
  // what takes the powers of two out again: exact in fp32
  const float dv_by = ldexpf(1.f, Elem<T>::kNarrow ? -kPUp : 0), dk_by = dv_by / factor;
  const int64_t tok = (int64_t)t.lo + j;
  if (a.splits > 1) {
    if constexpr (Elem<T>::kNarrow) {
#pragma unroll
      for (int d = 0; d < DP / 32; ++d) {
        dk[d] *= dk_by;
        dv[d] *= dv_by;
      }
    }
    float* to = a.part + (((int64_t)part * 2 * kv_heads + kvh) * a.s.n_tok + tok) * DP;
    const int64_t dv_at = (int64_t)kv_heads * a.s.n_tok * DP;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int col = 32 * d + 8 * y + 4 * g;
        *(f32x4*)(to + col) = f32x4{dk[d][4 * y], dk[d][4 * y + 1], dk[d][4 * y + 2], dk[d][4 * y + 3]};
        *(f32x4*)(to + dv_at + col) = f32x4{dv[d][4 * y], dv[d][4 * y + 1], dv[d][4 * y + 2], dv[d][4 * y + 3]};
      }
    return;
  }
  store_rows<T, DP>(a.dk.p + kvh * a.dk.head + tok * a.dk.tok, dk, a.s.dim,
                    a.s.scale * dk_by);
  store_rows<T, DP>(a.dv.p + kvh * a.dv.head + tok * a.dv.tok, dv, a.s.dim, dv_by);
}

// dK and dV of heads wider than 64: the sums alone take 128 registers per
// lane, which leaves one wave per SIMD. So two waves share 32 keys: of each
// step's 64 rows, each computes P and dS of 32, then one sums dV over all 64
// and the other dK, each with its own operand and its partner's, which travels
// through LDS as rounded operands (2 KB a step). The sums of a step are taken
// one step later, beside the next step's scores: their products do not wait
// for the exponentials, and one barrier per step serves both the tiles (three
// in turn) and the exchange.
template <typename T, int DP>
__global__ void __launch_bounds__(512, 2) k_attn_dkv2(BwdArgs a) {
  constexpr int NT = 512;
  __shared__ __attribute__((aligned(kTileAlign))) uint16_t sq[3][kStep * DP], sd[3][kStep * DP];
  static_assert(__alignof__(sq) >= kTileAlign && __alignof__(sd) >= kTileAlign, "16-byte pieces");
  __shared__ u32x4 ex[2][8][2][kWave];
  __shared__ __attribute__((aligned(16))) float s_lse[3][kStep], s_delta[3][kStep];
  const int kv_heads = a.s.heads / a.s.group;
  const int kvh = blockIdx.x % kv_heads, part = blockIdx.x / kv_heads % a.splits;
  const int at = blockIdx.x / kv_heads / a.splits;
  const Tile t = a.keys.tiles[at];
  if (at >= *a.keys.n) return;
  const int l = lane(), w = wave_id(), g = l >> 5;
  const int half = w >> 2;  // which 32 rows of a step, and dV (0) or dK (1)
  const int t1 = min(t.t0 + 128, t.len);
  const int j0 = t.t0 + 32 * (w & 3), j = j0 + (l & 31);
  const bool on = live_row(a.s, t, j);
  const bool causal = a.s.causal != 0;

  u32x4 kf[DP / 16], vf[DP / 16];
  load_scaled_columns<DP>(kf, a.k.p + kvh * a.k.head, a.k.tok, a.s, t, j);
  load_columns<DP>(vf, a.v.p + kvh * a.v.head, a.v.tok, a.s, t, j);
  f32x16 sum[DP / 32];
#pragma unroll
  for (int d = 0; d < DP / 32; ++d) sum[d] = zero16();
  const float c = log2_scale(a.s);
  const Operands<DP> op;

  const bool own = t.t0 >= t.hist;
  const int first = (own || causal ? t.t0 : 0) / kStep;
  const int last = (int)cdiv(own ? t1 : t.len, kStep);
  const int per = last - first, all = per * a.s.group;
  const int step0 = (int)((int64_t)all * part / a.splits);
  const int steps = (int)((int64_t)all * (part + 1) / a.splits);

  using Tiles = Direct<DP, NT>;
  uint32_t live_of = 0;
  float st_lse = INFINITY, st_delta = 0.f;  // threads 0 .. 63: one row each
  auto row0 = [&](int step) { return (first + step % per) * kStep; };
  auto load = [&](int step, int to) {
    const int head = kvh * a.s.group + step / per, i0 = row0(step);
    Tiles::load(sq[to], a.q.p + head * a.q.head, a.q.tok, a.s, t, i0);
    Tiles::load(sd[to], a.d_o.p + head * a.d_o.head, a.d_o.tok, a.s, t, i0);
    if (threadIdx.x < kStep) {
      const int i = min(i0 + (int)threadIdx.x, t.len - 1);
      const int64_t at = (int64_t)head * a.s.n_tok + t.lo + i;
      st_lse = a.lse[at];
      st_delta = a.delta[at];
    }
    live_of = live_byte(a.s, t, i0);
  };
  if (step0 < steps) load(step0, 0);
  // beside the first tiles' way
  const float factor =
      Elem<T>::kNarrow ? rows_factor(a, t, kvh, first * kStep, own ? t1 : t.len) : 1.f;
  constexpr float p_up = Elem<T>::kNarrow ? kPUp : 0;
  bool have = false;       // the last step's operands wait to be summed
  u32x4 mine[2];           // this wave's own of them
  int b = 0, before = 2;   // this step's tiles, the last step's
  for (int step = step0; step <= steps; ++step) {  // one more, for the last sums
    const int e = step & 1, i0 = row0(step), r0 = i0 + 32 * half;
    if (step < steps) {
      Tiles::wait();
      const uint64_t live = live_bits(live_of);
      Tiles::finish(sq[b], a.s, live);
      Tiles::finish(sd[b], a.s, live);
      if (threadIdx.x < kStep) {
        const bool in = (live >> threadIdx.x) & 1;
        s_lse[b][threadIdx.x] = !in || st_lse == -INFINITY ? INFINITY : st_lse * kLog2e - p_up;
        s_delta[b][threadIdx.x] = in ? st_delta * factor : 0.f;
      }
    }
    __syncthreads();
    if (step + 1 < steps) load(step + 1, b == 2 ? 0 : b + 1);
    // steps whose rows see none of these keys (the same for both waves)
    const bool none = step >= steps || j0 >= t1 || (causal && i0 + kStep <= j0) ||
                      (j0 >= t.hist && (i0 + kStep <= j0 || i0 > j0 + 31));
    f32x16 s, dp;
    if (!none) {
      s = dp = zero16();
#pragma unroll
      for (int kk = 0; kk < DP / 16; ++kk) {
        s = Elem<T>::mfma(op.rows(sq[b], 32 * half, kk), kf[kk], s);
        dp = Elem<T>::mfma(op.rows(sd[b], 32 * half, kk), vf[kk], dp);
      }
      // rows that are not live have lse = inf, so P = 0; keys that are not
      // live spoil only their own column, which is not stored
      if (j0 + 32 > t.hist || (causal && r0 < j0 + 31)) {
        const uint32_t see = seeing_rows(j, r0, t.hist, causal) >> (4 * g);
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (!((see >> (8 * (x >> 2) + (x & 3))) & 1u)) s[x] = -INFINITY;
      }
    }
    if (have) {
      const uint16_t* tile = half ? sq[before] : sd[before];
#pragma unroll
      for (int ib = 0; ib < 2; ++ib)
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          const u32x4 x = ib == half ? mine[ch] : ex[e ^ 1][w ^ 4][ch][l];
#pragma unroll
          for (int d = 0; d < DP / 32; ++d)
            sum[d] = Elem<T>::mfma(op.cols(tile, 32 * ib + 16 * ch, 32 * d), x, sum[d]);
        }
    }
    if (!none) {
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const f32x4 ls = *(const f32x4*)&s_lse[b][32 * half + 8 * y + 4 * g];
        const f32x4 de = *(const f32x4*)&s_delta[b][32 * half + 8 * y + 4 * g];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int z = 4 * y + x;
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[z], c, -ls[x]));
          s[z] = p;
          dp[z] = p * (Elem<T>::kNarrow ? __builtin_fmaf(dp[z], factor, -de[x]) : dp[z] - de[x]);
        }
      }
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        const u32x4 pb = to_operand<T>(s, ch), db = to_operand<T>(dp, ch);
        mine[ch] = half ? db : pb;
        ex[e][w][ch][l] = half ? pb : db;
      }
    }
    have = !none;
    before = b;
    b = b == 2 ? 0 : b + 1;
  }
  if (j >= t.len) return;
  if (!on) {
#pragma unroll
    for (int d = 0; d < DP / 32; ++d) sum[d] = zero16();
  }
  // what takes the powers of two out again: exact in fp32
  const float dv_by = ldexpf(1.f, Elem<T>::kNarrow ? -kPUp : 0), by = half ? dv_by / factor : dv_by;
  const int64_t tok = (int64_t)t.lo + j;
  if (a.splits > 1) {
    if constexpr (Elem<T>::kNarrow) {
#pragma unroll
      for (int d = 0; d < DP / 32; ++d) sum[d] *= by;
    }
    float* to = a.part + (((int64_t)part * 2 + 1 - half) * kv_heads + kvh) * a.s.n_tok * DP + tok * DP;
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
      for (int y = 0; y < 4; ++y)
        *(f32x4*)(to + 32 * d + 8 * y + 4 * g) =
            f32x4{sum[d][4 * y], sum[d][4 * y + 1], sum[d][4 * y + 2], sum[d][4 * y + 3]};
    return;
  }
  const View& o = half ? a.dk : a.dv;
  store_rows<T, DP>(o.p + kvh * o.head + tok * o.tok, sum, a.s.dim,
                    half ? a.s.scale * by : by);
}

// Sums of the parts, part by part: one thread per 4 columns of dK or dV.
template <typename T, int DP>
__global__ void __launch_bounds__(256) k_attn_join(BwdArgs a, const int64_t* __restrict__ offsets,
                                                   int32_t n) {
  constexpr int kPer = DP / 4;
  if (*a.keys.n == 0) return;  // no samples, or offsets that do not rise
  const int kv_heads = a.s.heads / a.s.group;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int col = (int)(id % kPer) * 4;
  const int64_t tok = id / kPer % a.s.n_tok;
  const int64_t row = id / kPer / a.s.n_tok;  // which * kv_heads + key head
  if (row >= 2 * kv_heads || col >= a.s.dim || tok < offsets[0] || tok >= offsets[n]) return;
  f32x4 s = {0, 0, 0, 0};
  for (int p = 0; p < a.splits; ++p)
    s += *(const f32x4*)(a.part + (((int64_t)p * 2 * kv_heads + row) * a.s.n_tok + tok) * DP + col);
  const bool is_v = row >= kv_heads;
  const View& o = is_v ? a.dv : a.dk;
  if (!is_v) s *= a.s.scale;
  *(u32x2*)(o.p + (row - (is_v ? kv_heads : 0)) * o.head + tok * o.tok + 2 * col) =
      u32x2{Elem<T>::pack(s[0], s[1]), Elem<T>::pack(s[2], s[3])};
}

template <typename T, int DP>
int launch_bwd(const BwdArgs& a, const int64_t* offsets, int32_t n, int64_t row_cap, int64_t key_cap,
               hipStream_t stream) {
  constexpr int NW = 4;
  const int64_t kv_heads = a.s.heads / a.s.group;
  hipLaunchKernelGGL((k_attn_dq<T, DP, NW>), dim3((unsigned)(row_cap * (a.s.heads / a.s.pack))),
                     dim3(NW * kWave), 0, stream, a);
  FS_LAUNCH_CHECK();
  const dim3 grid((unsigned)(key_cap * kv_heads * a.splits));
  if constexpr (DP == 128)
    hipLaunchKernelGGL((k_attn_dkv2<T, DP>), grid, dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((k_attn_dkv<T, DP, NW>), grid, dim3(NW * kWave), 0, stream, a);
  FS_LAUNCH_CHECK();
  if (a.splits > 1) {
    const int64_t threads = 2 * kv_heads * a.s.n_tok * (DP / 4);
    hipLaunchKernelGGL((k_attn_join<T, DP>), dim3((unsigned)cdiv(threads, 256)), dim3(256), 0, stream,
                       a, offsets, n);
    FS_LAUNCH_CHECK();
  }
  return FS_OK;
}

template <typename T>
int launch_bwd(const BwdArgs& a, const int64_t* offsets, int32_t n, int64_t row_cap, int64_t key_cap,
               hipStream_t stream) {
  if (padded(a.s.dim) == 32) return launch_bwd<T, 32>(a, offsets, n, row_cap, key_cap, stream);
  if (padded(a.s.dim) == 64) return launch_bwd<T, 64>(a, offsets, n, row_cap, key_cap, stream);
  return launch_bwd<T, 128>(a, offsets, n, row_cap, key_cap, stream);
}

}  // namespace
}  // namespace attn
}  // namespace fs

using namespace fs;
using namespace fs::attn;

extern "C" size_t fs_jagged_attention_backward_workspace_size(int64_t n_tok, int32_t n,
                                                              int32_t heads, int32_t kv_heads,
                                                              int32_t dim) {
  if (n_tok < 0 || n < 0 || heads < 0 || kv_heads < 1 || dim < 0) return 0;
  Carve c(nullptr);
  c.take<int32_t>(1);
  c.take<Tile>((size_t)tile_cap(n_tok, n, 32));
  c.take<int32_t>(1);
  c.take<Tile>((size_t)tile_cap(n_tok, n, 128));
  c.take<float>((size_t)heads * (size_t)n_tok);
  c.take<float>((size_t)heads * (size_t)n_tok);
  c.take<float>((size_t)split_tokens(n_tok, kv_heads) * 2 * kv_heads * padded(dim));
  return c.used + 256;
}

extern "C" int fs_jagged_attention_backward(
    const fs_heads* q, const fs_heads* k, const fs_heads* v, const fs_heads* out,
    const float* lse, const fs_heads* dout, const int64_t* offsets, int32_t n, int64_t n_tok,
    const int32_t* n_cand, const uint8_t* valid, int32_t heads, int32_t kv_heads, int32_t dim,
    int32_t dtype, int32_t causal, float scale, const fs_heads* dq, const fs_heads* dk,
    const fs_heads* dv, int32_t* err, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (n < 0 || n > FS_MAX_SAMPLES || n_tok < 0 || n_tok >= (int64_t)INT32_MAX || heads < 1 ||
      kv_heads < 1 || heads % kv_heads || !offsets || !scale_ok(scale))
    return FS_ERR_INVALID_ARG;
  if (!type_ok(dtype) || dim < 8 || dim > 128 || dim % 8 || heads > FS_MAX_HEADS)
    return FS_ERR_UNSUPPORTED;
  BwdArgs a;
  int rc;
  if ((rc = make_view(q, heads, dim, &a.q)) || (rc = make_view(k, kv_heads, dim, &a.k)) ||
      (rc = make_view(v, kv_heads, dim, &a.v)) || (rc = make_view(out, heads, dim, &a.o)) ||
      (rc = make_view(dout, heads, dim, &a.d_o)) || (rc = make_view(dq, heads, dim, &a.dq)) ||
      (rc = make_view(dk, kv_heads, dim, &a.dk)) || (rc = make_view(dv, kv_heads, dim, &a.dv)))
    return rc;
  if (n_tok > 0 && n > 0 &&
      (!a.q.p || !a.k.p || !a.v.p || !a.o.p || !a.d_o.p || !a.dq.p || !a.dk.p || !a.dv.p || !lse))
    return FS_ERR_INVALID_ARG;
  if (!ws || ws_bytes < fs_jagged_attention_backward_workspace_size(n_tok, n, heads, kv_heads, dim))
    return FS_ERR_WORKSPACE;
  if (n == 0 || n_tok == 0) return FS_OK;
  const int32_t pack = pack_of(heads / kv_heads), rows = 128 / pack;
  const int64_t row_cap = tile_cap(n_tok, n, rows), key_cap = tile_cap(n_tok, n, 128);
  a.splits = splits_of(n_tok, n, kv_heads, heads / kv_heads);
  if (!grid_fits(row_cap * (heads / pack), 256) ||
      !grid_fits(key_cap * kv_heads * a.splits, padded(dim) == 128 ? 512 : 256))
    return FS_ERR_UNSUPPORTED;
  Carve c(ws);
  TileTable tabs[2];
  tabs[0].rows = rows;
  tabs[0].n = c.take<int32_t>(1);
  tabs[0].tiles = c.take<Tile>((size_t)tile_cap(n_tok, n, 32));
  tabs[1].rows = 128;
  tabs[1].n = c.take<int32_t>(1);
  tabs[1].tiles = c.take<Tile>((size_t)key_cap);
  a.lse = lse;
  a.delta = c.take<float>((size_t)heads * (size_t)n_tok);
  a.factor = c.take<float>((size_t)heads * (size_t)n_tok);
  a.part = c.take<float>((size_t)split_tokens(n_tok, kv_heads) * 2 * kv_heads * padded(dim));
  if ((rc = launch_tiles(offsets, n, n_tok, n_cand, causal, tabs, 2, err, stream))) return rc;
  a.s = Shape{tabs[0], valid, n_tok, heads, heads / kv_heads, pack, dim, causal, scale};
  a.keys = tabs[1];
  return dtype == FS_BF16 ? launch_bwd<__bf16>(a, offsets, n, row_cap, key_cap, stream)
                          : launch_bwd<_Float16>(a, offsets, n, row_cap, key_cap, stream);
}
