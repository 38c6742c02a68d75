// Softmax losses of tokens against a vocabulary's table, without their logits.
//
//   z_iv = scale x_i . w_v,  lse_i = log sum_v exp z_iv
//   loss:     loss_i = lse_i - z_i,label(i)
//   distill:  q_i = softmax of scale teacher_i over the token's entries,
//             loss_i = sum_k q_ik (log q_ik - z_i,id(k) + lse_i)
//   back:     e_iv = dloss_i scale (exp(z_iv - lse_i) - target_iv),  dx = e w,  dw = e^T x
//             target: 1 at the label; the sum of the q of the entries with id v
//
// Tokens that take part are first packed together (k_head_pack; the forward
// pass reads few tokens as they lie). The forward
// pass is one product whose tiles keep a maximum and a sum per token instead of
// scores. The backward pass goes over the table in pieces: scores again, e in 16
// bits, and the two products that sum it; what it holds of a piece is bounded
// whatever the vocabulary's size.
#include <algorithm>
#include <cmath>

#include "product.hpp"

namespace fs {
namespace {

using namespace prod;

constexpr float kLog2e = attn::kLog2e, kLn2 = attn::kLn2;
constexpr int kV = 256;                           // table rows of a tile
// e of one piece of the table: every piece adds to dx's fp32 sums in memory (16384 x
// 131072 x 1024: pieces of 2^29 bytes 11.5 ms, 2^30 11.4, 2^27 13.3)
constexpr int64_t kPieceBytes = (int64_t)1 << 30;
constexpr int64_t kPackBytes = (int64_t)1 << 26;   // a piece of a table that has to be laid out
constexpr int64_t kPartBytes = (int64_t)1 << 28;   // sums of a cut product
constexpr int kMostParts = 256;
constexpr int64_t kFew = 256;                      // tokens, see ScoreArgs::e
constexpr int64_t kStayMost = 1024;                // tokens that may keep their places
// Tokens whose tiles are joined by many threads each, a distillation's where its entries are
// (a launch of 4 us less). Calls with that and without, us: distillation of 2100 tokens, 4000
// rows of 512, 46 and 39, 4096 64 and 48, 8192 100 and 68; of 1500 34 and 30, so 1025 would do
// as well. Cross entropy 8192 x 4000 x 512 59 and 56, 1500 24 and 22.
constexpr int64_t kFewRows = 2048;
static_assert(kFewRows > kStayMost, "tokens that keep their places have no list of them for k_loss");
constexpr int64_t kCacheBytes = (int64_t)1 << 27;  // half of the last level

// What the kernels of one call share, in its workspace.
struct Head {
  int32_t* n_live;  // tokens that take part
  float* mul;       // [2]: e is rounded times mul[0], sums of it come times mul[1]
  int32_t* pos;     // [n] a token's place among them, or -1
  int32_t* label;   // [npad] by place, as are lse2 and coef
  float* lse2;      // lse log2(e)
  float* coef;      // dloss scale
  char* x;          // [npad][dp] 16 bits in blocks: their rows, zeros past dim and n_live
  int64_t n, npad;
  int32_t dim, dp;
};

// 8 elements of a row of `dim`, zeros past it, from any alignment
__device__ __forceinline__ u32x4 row_piece(const char* row, int32_t col, int32_t dim) {
  if (col + 8 <= dim) return *(const u32x4_any*)(row + 2 * (int64_t)col);
  uint16_t v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = col + e < dim ? ((const uint16_t*)row)[col + e] : (uint16_t)0;
  u32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) r[e] = v[2 * e] | (uint32_t)v[2 * e + 1] << 16;
  return r;
}

// A teacher's entries, [n][top]. One takes part where its id is a row of the table
// and not the padding, and its logit is not -inf.
struct Entries {
  const int64_t* ids;
  const char* teacher;
  int32_t type, top;
  int64_t rows, pad;
  __device__ __forceinline__ float logit(int64_t i) const {
    if (type == FS_F32) return ((const float*)teacher)[i];
    if (type == FS_BF16) return (float)((const __bf16*)teacher)[i];
    return (float)((const _Float16*)teacher)[i];
  }
  __device__ __forceinline__ bool on(int64_t id, float t) const {
    return id >= 0 && id < rows && id != pad && t != -INFINITY;
  }
  __device__ __forceinline__ bool bad(int64_t id) const { return (id < 0 || id >= rows) && id != pad; }
  // whether token i has one, four at a time
  __device__ __forceinline__ bool any(int64_t i) const {
    for (int k = 0; k < top; k += 4) {
      bool found = false;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t at = i * top + min(k + u, top - 1);
        found |= on(ids[at], logit(at));
      }
      if (found) return true;
    }
    return false;
  }
};

// ---------------------------------------------------------------- packing
struct PackArgs {
  Head h;
  const char* x;
  int64_t x_stride;
  const int64_t* labels;  // or null: live says which tokens take part,
  const uint8_t* live;    // or, of tokens that stay, their entries
  Entries entries;
  int32_t stay;           // few tokens: each keeps its place, with a row of zeros where it takes no part
  int64_t rows, pad;
  const float *lse, *dloss;  // backward
  int32_t back;
  float scale;
  int32_t per;     // tokens of a workgroup
  int32_t pad_to;  // zero rows up to a multiple of this
  int32_t narrow;  // fp16
  int32_t* err;
};

constexpr int kPackThreads = 256;

__device__ __forceinline__ bool takes_part(const PackArgs& a, int64_t i, bool* bad) {
  if (!a.labels) return a.stay ? a.entries.any(i) : a.live[i] != 0;
  const int64_t v = a.labels[i];
  const bool in = v >= 0 && v < a.rows;
  *bad = !in && v != a.pad;
  return in && v != a.pad;
}
// Which of tokens i, i + 256, .. take part, eight with their loads in flight
// together; tokens from `end` on do not.
constexpr int kAtOnce = 8;
__device__ __forceinline__ uint32_t take_part(const PackArgs& a, int64_t i, int64_t end) {
  uint32_t on = 0;
  if (a.labels) {
    int64_t v[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) v[u] = a.labels[min(i + u * kPackThreads, end - 1)];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) on |= (uint32_t)(v[u] >= 0 && v[u] < a.rows && v[u] != a.pad) << u;
  } else {
    uint8_t v[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) v[u] = a.live[min(i + u * kPackThreads, end - 1)];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) on |= (uint32_t)(v[u] != 0) << u;
  }
  const int64_t left = cdiv(end - i, kPackThreads);
  return left < kAtOnce ? on & ((1u << left) - 1) : on;
}

// What e is rounded times, and its inverse, by one workgroup. fp16's exponents end
// where e's do not: there it is a power of two that takes the largest coefficient to
// 2^13 .. 2^14, and the sums lose it again.
__device__ void put_mul(const PackArgs& a) {
  __shared__ float s_max[kPackThreads / kWave];
  bool bad = false;
  float top = 0.f;
  if (a.narrow) {
    if (a.stay) {  // few tokens a thread
      for (int64_t i = threadIdx.x; i < a.h.n; i += kPackThreads)
        if (takes_part(a, i, &bad)) top = fmaxf(top, fabsf(a.dloss[i] * a.scale));
    }
    for (int64_t i = threadIdx.x; !a.stay && i < a.h.n; i += kAtOnce * kPackThreads) {
      float d[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) d[u] = a.dloss[min(i + u * kPackThreads, a.h.n - 1)];
      const uint32_t on = take_part(a, i, a.h.n);
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) top = fmaxf(top, on >> u & 1 ? fabsf(d[u] * a.scale) : 0.f);
    }
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
    if (lane() == 0) s_max[threadIdx.x / kWave] = top;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    float m = 1.f, back = 1.f;
    if (a.narrow) {
      for (int w = 0; w < kPackThreads / kWave; ++w) top = fmaxf(top, s_max[w]);
      int ex = 0;
      if (top > 0.f && top < INFINITY) frexpf(top, &ex);
      // powers of two that fp32 has on both sides
      const int s = min(max(14 - ex, -120), 120);
      m = ldexpf(1.f, s);
      back = ldexpf(1.f, -s);
    }
    a.h.mul[0] = m;
    a.h.mul[1] = back;
  }
}

// Each workgroup counts the tokens before its own that take part (labels are few
// bytes beside the rows), so one launch does it without waiting for another
// workgroup. The last of them writes the count and the zero rows behind it. 16384 x
// 1024: 25 us, where copying the rows takes 13; the counting is the rest. There are at most
// 1024 workgroups, so it grows with the tokens: rows of 64, 2^17 tokens 57 us, 2^20 520 and
// 2^23 4.1 ms, more than the forward scores of 300 table rows (2^20: 250).
__global__ void __launch_bounds__(kPackThreads) k_head_pack(PackArgs a) {
  __shared__ int32_t tmp[17], s_row[kPackThreads];
  const int32_t groups = gridDim.x - a.back;
  if ((int32_t)blockIdx.x == groups) {  // backward: one workgroup more
    put_mul(a);
    return;
  }
  const int64_t i0 = (int64_t)blockIdx.x * a.per, i1 = min(a.h.n, i0 + a.per);
  bool bad = false;
  int32_t base = (int32_t)i0;
  if (!a.stay) {
    int32_t count = 0;
    for (int64_t i = threadIdx.x; i < i0; i += kAtOnce * kPackThreads) count += __popc(take_part(a, i, i0));
    block_excl_scan<int32_t>(count, tmp, &base);
  }
  const int32_t pieces = a.h.dp / 8;
  const bool whole = a.h.dim % 8 == 0;
  for (int64_t c = i0; c < i1; c += kPackThreads) {  // uniform
    const int64_t i = c + threadIdx.x;
    bad = false;
    bool on;
    int32_t at = threadIdx.x, total = (int32_t)min((int64_t)kPackThreads, i1 - c);
    if (a.stay && !a.labels) {  // the threads share the tokens' entries
      s_row[threadIdx.x] = 0;
      __syncthreads();
      const int32_t top = a.entries.top, all = total * top;
      for (int32_t u0 = threadIdx.x; u0 < all; u0 += 4 * kPackThreads) {  // four in flight
        int64_t id[4];
        float t[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const int64_t at = c * top + min(u0 + y * kPackThreads, all - 1);
          id[y] = a.entries.ids[at];
          t[y] = a.entries.logit(at);
        }
#pragma unroll
        for (int y = 0; y < 4; ++y) {  // past the last one: it again
          bad |= a.entries.bad(id[y]);
          if (a.entries.on(id[y], t[y])) s_row[min(u0 + y * kPackThreads, all - 1) / top] = 1;
        }
      }
      __syncthreads();
      on = i < i1 && s_row[threadIdx.x];
      __syncthreads();
    } else {
      on = i < i1 && takes_part(a, i, &bad);
    }
    flag_err(a.err, bad, FS_EF_ID_RANGE);
    if (!a.stay) at = block_excl_scan<int32_t>(on ? 1 : 0, tmp, &total);
    if (i < i1) a.h.pos[i] = on ? base + at : -1;
    if (a.stay ? i < i1 : on) {
      s_row[at] = on ? (int32_t)(i - i0) : -1;
      a.h.label[base + at] = a.labels && on ? (int32_t)a.labels[i] : -1;
      if (a.back) {
        a.h.lse2[base + at] = on ? a.lse[i] * kLog2e : 0.f;
        a.h.coef[base + at] = on ? a.dloss[i] * a.scale : 0.f;
      }
    }
    __syncthreads();
    const int32_t all = total * pieces;
    for (int32_t u0 = 0; u0 < all; u0 += 4 * kPackThreads) {  // four pieces of a thread in flight
      u32x4 v[4];
      int32_t r[4], p[4];
      bool on_row[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int32_t u = min(u0 + y * kPackThreads + (int32_t)threadIdx.x, all - 1);
        r[y] = u / pieces;
        p[y] = u - r[y] * pieces;
        on_row[y] = s_row[r[y]] >= 0;
        const char* row = a.x + (i0 + max(s_row[r[y]], 0)) * a.x_stride;
        if (whole) v[y] = *(const u32x4_any*)(row + 16 * (8 * p[y] < a.h.dim ? p[y] : 0));
        else v[y] = row_piece(row, 8 * p[y], a.h.dim);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y)
        *(u32x4*)(a.h.x + 2 * blocked(base + r[y], 8 * p[y], a.h.dp)) =
            on_row[y] && 8 * p[y] < a.h.dim ? v[y] : u32x4{0, 0, 0, 0};
    }
    base += total;
    __syncthreads();
  }
  if ((int32_t)blockIdx.x == groups - 1) {
    const int32_t end = (int32_t)cdiv(base, a.pad_to) * a.pad_to, rest = end - base;
    if (threadIdx.x == 0) *a.h.n_live = base;
    for (int32_t r = base + threadIdx.x; r < end; r += kPackThreads) {
      a.h.label[r] = -1;
      a.h.lse2[r] = a.h.coef[r] = 0.f;
    }
    for (int32_t u = threadIdx.x; u < rest * pieces; u += kPackThreads)
      *(u32x4*)(a.h.x + 2 * blocked(base + u / pieces, 8 * (u % pieces), a.h.dp)) = u32x4{0, 0, 0, 0};
  }
}

// Table rows that the tiles cannot load as they lie, [rows][dp] with zeros past dim.
__global__ void __launch_bounds__(kPackThreads)
k_table_pack(const char* w, int64_t stride, int64_t rows, int32_t dim, int32_t dp, char* to) {
  const int32_t pieces = dp / 8;
  for (int64_t u = (int64_t)blockIdx.x * kPackThreads + threadIdx.x; u < rows * pieces;
       u += (int64_t)gridDim.x * kPackThreads) {
    const int64_t r = u / pieces;
    *(u32x4*)(to + u * 16) = row_piece(w + r * stride, 8 * (int32_t)(u - r * pieces), dim);
  }
}

// ---------------------------------------------------------------- scores
struct ScoreArgs {
  Head h;
  const char* w;     // the piece's first row
  int64_t w_stride;
  int64_t v0;        // its number in the table
  int64_t rows;      // rows of the piece
  int32_t k;         // elements of a row
  int32_t v_tile0;   // forward: tiles of the pieces before
  Order order;
  float scale2;      // scale log2(e)
  const char* x;     // forward of few tokens: their rows as they lie, with
  int64_t x_stride;
  const int64_t* labels;  // (null: none)
  int64_t all_rows, pad;
  float2* part;      // forward: [tiles of the table][npad] maximum and sum, base 2
  float2* at_label;  // forward: [npad] the label's score, base 2, and what its rounding left
  // backward: [npad][e_cols] 16 bits in blocks. Up to kFew tokens e is two numbers,
  // rounded and what the rounding left, in blocks beside each other: few tokens'
  // gradients have few terms to average a rounding over (64 tokens: dx off by 3.2e-4
  // of its size in one number, fp16, where its own rounding is 2.1e-4).
  char* e;
  int64_t e_cols;
  int32_t past;      // e outgrows the caches
};

// a label's row, or -1 where its token takes no part
__device__ __forceinline__ int32_t label_of(int64_t v, int64_t rows, int64_t pad) {
  return v >= 0 && v < rows && v != pad ? (int32_t)v : -1;
}

// element (token, row) of a half of e
__device__ __forceinline__ int64_t place_of_e(int64_t n, int64_t v, int64_t cols, int half, int halves) {
  return blocked(n, (v / kK * halves + half) * kK + v % kK, cols * halves);
}

// waves of a tile: 256 x 256 and 256 x 64
constexpr int kWM = 2, kWN = 4;
constexpr int kMostThreads = 512;
constexpr int kCus = 256;
constexpr int kGroup = 8;  // token tiles that go by a table tile together

// label, lse2 and coef of a tile's tokens, to LDS without registers: a wait for
// them would wait for the next tile's loads as well
template <int BN, int NW, bool Back>
__device__ __forceinline__ void ask_info(const Head& h, int64_t n0, float (*info)[BN]) {
  const uint32_t to = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float*)&info[0][0]);
  constexpr int kGroups = BN / kWave;
#pragma unroll
  for (int t0 = 0; t0 < (Back ? 3 : 1) * kGroups; t0 += NW) {
    const int t = t0 + attn::wave_id(), which = t / kGroups, g = t % kGroups;
    if (which >= (Back ? 3 : 1)) break;
    const char* from = (const char*)(which == 0 ? (const void*)h.label : which == 1 ? h.lse2 : h.coef);
    load_words(attn::uniform(from + 4 * (n0 + g * kWave)), 4 * lane(), to + 4 * (which * BN + g * kWave));
  }
}

// A tile's tokens' label, lse2 and coef: in LDS, or where a workgroup has one tile in
// registers, a lane's NI tokens, read ahead of its product.
template <int BN>
struct TokenInfo {
  const float (*lds)[BN];
  int32_t labels[2];
  float lse2s[2], coefs[2];
  __device__ __forceinline__ int32_t label(int n, int j) const {
    return BN == 256 ? __float_as_int(lds[0][n]) : labels[j];
  }
  __device__ __forceinline__ float lse2(int n, int j) const { return BN == 256 ? lds[1][n] : lse2s[j]; }
  __device__ __forceinline__ float coef(int n, int j) const { return BN == 256 ? lds[2][n] : coefs[j]; }
};

// What a tile's scores leave behind, by way of the stage that the next tile's
// first loads do not write.
template <typename T, int BN, int WM, int WN, int Halves, typename P>
__device__ __forceinline__ void finish_scores(const ScoreArgs& a, P& p, uint16_t* lds, int64_t n0, int64_t v0,
                                              int32_t tv, const TokenInfo<BN>& info, float mul) {
  constexpr int NT = WM * WN * kWave;
  const int l = here(lane()), tid = here(threadIdx.x);
  const int left = (int)min((int64_t)kV, a.rows - v0);  // rows of this tile
  // from here on the scale is positive, so the largest product's score is the
  // largest (a scale of 0 makes the products zeros)
  if (a.scale2 <= 0.f) {
#pragma unroll
    for (int i = 0; i < P::MI; ++i)
#pragma unroll
      for (int j = 0; j < P::NI; ++j) p.acc[i][j] = a.scale2 < 0.f ? -p.acc[i][j] : attn::zero16();
  }
  const float scale2 = a.scale2 == 0.f ? 1.f : fabsf(a.scale2);
  if (left < kV) {  // rows past the table: exp 0
    const int d = left - P::m_of(0, l);
#pragma unroll
    for (int i = 0; i < P::MI; ++i)
#pragma unroll
      for (int j = 0; j < P::NI; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * i + 8 * (r >> 2) + (r & 3) >= d) p.acc[i][j][r] = -INFINITY;
  }
  // the product at column m of a lane's row, where the lane has it
  auto product_at = [&](int j, int m) {
    const int d = here(m - P::m_of(0, l));
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < P::MI; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) v = 32 * i + 8 * (r >> 2) + (r & 3) == d ? p.acc[i][j][r] : v;
    return v;
  };
  auto has = [&](int m) {  // m of the tile
    return m / 32 / P::MI == attn::wave_id() % WM && (m >> 2 & 1) == l >> 5;
  };
  if constexpr (Halves == 0) {
    float2(*s_part)[BN] = (float2(*)[BN])lds;
    static_assert(2 * P::kStage >= WM * BN * 8, "a stage holds them");
#pragma unroll
    for (int j = 0; j < P::NI; ++j) {
      const int n = P::n_of(j, l);
      const int64_t lab = (int64_t)info.label(n, j) - a.v0 - v0;
      if (lab >= 0 && lab < kV && has((int)lab)) {
        const float p_lab = product_at(j, (int)lab), z = p_lab * scale2, rest = __builtin_fmaf(p_lab, scale2, -z);
        a.at_label[n0 + n] = make_float2(z, rest == rest ? rest : 0.f);  // none of an infinity
      }
      float top = p.acc[0][j][0];
#pragma unroll
      for (int i = 0; i < P::MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, p.acc[i][j][r]);
      // finite, so that scores of -inf add 0
      top = fmaxf(attn::max_halves(top) * scale2, -3e38f);
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < P::MI; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          sum[r & 3] += __builtin_amdgcn_exp2f(__builtin_fmaf(p.acc[i][j][r], scale2, -top));
      const float total = attn::add_halves((sum[0] + sum[1]) + (sum[2] + sum[3]));
      if (l < 32) s_part[attn::wave_id() % WM][n] = make_float2(top, total);
    }
    lds_barrier();
    for (int n = tid; n < BN; n += NT) {
      float top = s_part[0][n].x;
#pragma unroll
      for (int i = 1; i < WM; ++i) top = fmaxf(top, s_part[i][n].x);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < WM; ++i) sum += s_part[i][n].y * __builtin_amdgcn_exp2f(s_part[i][n].x - top);
      a.part[(int64_t)(a.v_tile0 + tv) * a.h.npad + n0 + n] = make_float2(top, sum);
    }
  } else {
    // Rows of e that pass through LDS at once: all of them and both halves where no
    // next tile's loads are under way, else a block of 32 a wave.
    constexpr bool kWhole = BN == 64;
    constexpr int kRows = kWhole ? BN : WN * 32, kPieces = kV / 8;
    static_assert((kWhole ? 2 * P::kStage : P::kStage) >= (kWhole ? Halves : 1) * kRows * kV, "LDS holds a pass of e");
    uint16_t* const at0 = kWhole ? lds - P::kStage : lds;
    auto store = [&](int half, int j) {
#pragma unroll 4
      for (int y = 0; y < kRows * kPieces / NT; ++y) {  // block by block
        const int u = y * NT + tid, r = u / 8 % kRows, piece = u / (8 * kRows) * 8 + u % 8;
        const int n = kWhole ? r : (r / 32 * P::NI + j) * 32 + r % 32;
        const u32x4 v = Stage16<kV>::get(at0 + (kWhole ? half * kRows * kV : 0), r, piece);
        u32x4* to = (u32x4*)(a.e + 2 * place_of_e(n0 + n, v0 + 8 * piece, a.e_cols, half, Halves));
        // what outgrows the caches goes past them: they hold the operands of the
        // tiles beside this one (597 -> 565 us, and the product that reads e 503
        // -> 479); less is read from them soon
        if (Halves == 1 && a.past) __builtin_nontemporal_store(v, to);
        else *to = v;
      }
    };
#pragma unroll
    for (int j = 0; j < P::NI; ++j) {
      if (j && !kWhole) lds_barrier();
      const int n = P::n_of(j, l), s = kWhole ? n : attn::wave_id() / WM * 32 + (l & 31);
      const int64_t lab = (int64_t)info.label(n, j) - a.v0 - v0;
      const float lse2 = info.lse2(n, j), c = info.coef(n, j) * mul;
      // c exp2(s) = exp2(s + log2 c): the factor costs no instruction of its own
      const float at = __builtin_amdgcn_logf(fabsf(c)) - lse2;
      const uint32_t sign = c < 0.f ? 0x80008000u : 0u;
      // two values rounded, and what that leaves of them
      auto rounded = [](float x, float y, uint32_t* u) {
        u[0] = Elem<T>::pack(x, y);
        if (Halves > 1) {
          const auto back = Elem<T>::unpack(u[0]);
          u[1] = Elem<T>::pack(x - back[0], y - back[1]);
        }
      };
#pragma unroll
      for (int i = 0; i < P::MI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int m = P::m_of(i, l) + 8 * q;
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(p.acc[i][j][4 * q + r], scale2, at));
          uint32_t y0[2], y1[2];
          rounded(v[0], v[1], y0);
          rounded(v[2], v[3], y1);
#pragma unroll
          for (int half = 0; half < Halves; ++half)
            Stage16<kV>::put(at0 + half * kRows * kV, s, m, u32x2{y0[half] ^ sign, y1[half] ^ sign});
        }
      // the label's place, from the difference
      if (lab >= 0 && lab < kV && has((int)lab)) {
        const float v = __builtin_amdgcn_exp2f(__builtin_fmaf(product_at(j, (int)lab), scale2, -lse2)) - 1.f;
        uint32_t y[2];
        rounded(v * c, 0.f, y);
#pragma unroll
        for (int half = 0; half < Halves; ++half) Stage16<kV>::put1(at0 + half * kRows * kV, s, (int)lab, y[half]);
      }
      if (!kWhole) {
        lds_barrier();
        store(0, j);
      }
    }
    if (kWhole) {
      lds_barrier();
#pragma unroll
      for (int half = 0; half < Halves; ++half) store(half, 0);
    }
  }
}

// Tiles of scores. Columns of the product are table rows, its rows tokens: a lane's
// registers hold one token's scores, so their maximum and sum need one exchange
// between two lanes and one between waves. Workgroups of 256 tokens are as many as
// CUs and take tiles in turn; the next tile's first loads are asked for before this
// one's exponentials.
// Bound by power where rows are long, as the products are: forward, 14746 tokens x
// 100000 x 1024, 2.42 to 2.55 ms by card (1185 to 1250 TFLOP/s, matrix units busy 64%).
// Backward, 16384 x 32768 x 1024, 1.12 to 1.17 ms (940 to 980; 49%, 1.88 GHz): of that a fifth
// is what follows the product and does not overlap it, 140 us of
// it the 1 GiB of e that it writes, 36 the exponentials. Tiles begun half a tile apart
// on half of the CUs, so that fewer write at once: 1143 against 1134 us, not kept. With
// rows of 64 (one step a tile) the exponentials bound it: 8778 x 104994 x 64 takes 300
// us, the products alone 100.
template <typename T, int BN, int WM, int WN, int Halves, int Stages, bool Direct>
__global__ void __launch_bounds__(WM * WN * kWave) k_scores(ScoreArgs a) {
  constexpr bool Back = Halves > 0;
  constexpr int NT = WM * WN * kWave;
  using X = std::conditional_t<Direct, Rows<BN, NT>, BlockRows<BN, NT>>;
  using P = Tile<T, Rows<kV, NT>, X, kV, BN, WM, WN, 1, Stages>;
  auto tokens = [&](int32_t tn) {
    if constexpr (Direct) return X(a.x, a.x_stride, (int64_t)tn * BN, a.h.n, 0);
    else return X(a.h.x, a.h.dp, (int64_t)tn * BN, 0);
  };
  __shared__ __attribute__((aligned(16))) uint16_t lds[Stages * P::kStage];
  uint16_t* const second = lds + P::kStage;
  const int32_t live = Direct ? (int32_t)a.h.n : *a.h.n_live;
  // tiles of tokens that take part, dealt to all XCDs alike
  const Order order{(int32_t)cdiv(live, BN), a.order.cols};
  const int32_t tiles = order.rows * order.cols;
  if ((int32_t)blockIdx.x >= tiles) return;
  int32_t tn, tv;
  order.at(in_order(blockIdx.x, tiles), kGroup, &tn, &tv);
  Rows<kV, NT> w(a.w, a.w_stride, (int64_t)tv * kV, a.rows, 0);
  X x = tokens(tn);
  // tiles of 64 tokens are one to a workgroup, and LDS holds two such
  constexpr bool kMany = BN == 256;
  static_assert(Stages == 2 || !kMany, "a workgroup with more stages has one tile");
  float(*info)[Back ? 3 : 1][BN] = nullptr;
  if constexpr (kMany) {
    __shared__ float two[2][Back ? 3 : 1][BN];
    info = two;
  }
  if constexpr (kMany) ask_info<BN, WM * WN, Back>(a.h, (int64_t)tn * BN, info[0]);
  const float mul = Back ? __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(a.h.mul[0]))) : 1.f;
  P::template ask<true, false>(w, x, a.k, lds);
  int turn = 0;
  for (int32_t id = blockIdx.x; id < tiles; id += gridDim.x) {  // uniform
    const int64_t n0 = (int64_t)tn * BN, v0 = (int64_t)tv * kV;
    const int32_t tile = tv;
    TokenInfo<BN> its;
    if constexpr (kMany) {
      its.lds = (const float(*)[BN])info[turn];
    } else {
#pragma unroll
      for (int j = 0; j < P::NI; ++j) {
        const int64_t n = n0 + P::n_of(j);
        if constexpr (Direct) its.labels[j] = a.labels && n < a.h.n ? label_of(a.labels[n], a.all_rows, a.pad) : -1;
        else its.labels[j] = a.h.label[n];
        its.lse2s[j] = Back ? a.h.lse2[n] : 0.f;
        its.coefs[j] = Back ? a.h.coef[n] : 0.f;
      }
    }
    P p;
    p.clear();
    p.template run<true, false>(w, x, a.k, lds);
    if (id + (int32_t)gridDim.x < tiles) {  // the next tile's first loads, behind this one's scores
      order.at(in_order(id + gridDim.x, tiles), kGroup, &tn, &tv);
      w = Rows<kV, NT>(a.w, a.w_stride, (int64_t)tv * kV, a.rows, 0);
      x = tokens(tn);
      if constexpr (kMany) ask_info<BN, WM * WN, Back>(a.h, (int64_t)tn * BN, info[turn ^ 1]);
      P::template ask<true, false>(w, x, a.k, lds);
    }
    finish_scores<T, BN, WM, WN, Halves>(a, p, second, n0, v0, tile, its, mul);
    if (kMany) turn ^= 1;
  }
}

// ---------------------------------------------------------------- gradients
struct SumArgs {
  Head h;
  const char* w;     // dx: the piece's first row
  int64_t w_stride;
  int64_t rows;      // rows of the piece
  int32_t w_cols;
  const char* e;
  int64_t e_cols;
  Order order;       // of the output's tiles
  int32_t parts;     // of the sum
  int32_t steps;     // of 64, of a part (dx)
  int32_t add;       // to what the parts hold
  float* part;       // [parts][rows of the output][dp], or
  char* out;         // the output itself
  int64_t out_stride, out_rows;
  int32_t out_type;
};

// A tile's sums, fp32, to [row][dp] floats or to an output of any type.
template <typename P, int DM, int BN, int WM>
__device__ __forceinline__ void put_sums(P& p, uint16_t* lds, const SumArgs& a, float* part, int64_t row0,
                                         int64_t rows, int32_t col0) {
  const int32_t cols = part ? a.h.dp : a.h.dim;
  if (part || a.out_type == FS_F32) {
    const float back = part ? 1.f : a.h.mul[1];
    constexpr int kRows = P::kThreads / kWave / WM * 32, kPieces = DM / 4;
    float* f = (float*)lds;
#pragma unroll
    for (int j = 0; j < P::NI; ++j) {
      if (j) __syncthreads();
      const int n = attn::wave_id() / WM * 32 + (lane() & 31);
#pragma unroll
      for (int i = 0; i < P::MI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          Stage32<DM>::put(f, n, P::m_of(i) + 8 * q,
                           f32x4{p.acc[i][j][4 * q] * back, p.acc[i][j][4 * q + 1] * back,
                                 p.acc[i][j][4 * q + 2] * back, p.acc[i][j][4 * q + 3] * back});
      __syncthreads();
#pragma unroll 4
      for (int u = threadIdx.x; u < kRows * kPieces; u += P::kThreads) {
        const int s = u / kPieces, piece = u % kPieces;
        const int64_t row = row0 + (s / 32 * P::NI + j) * 32 + s % 32;
        const int32_t col = col0 + 4 * piece;
        if (row >= rows || col >= cols) continue;
        f32x4 v = Stage32<DM>::get(f, s, piece);
        if (part) {
          f32x4* to = (f32x4*)(part + row * a.h.dp + col);
          if (a.add) v += *to;
          *to = v;
        } else {
          float* to = (float*)(a.out + row * a.out_stride) + col;
          if (col + 4 <= cols) {
            *(f32x4_any*)to = v;
          } else {
            for (int e = 0; e < cols - col; ++e) to[e] = v[e];
          }
        }
      }
    }
    return;
  }
  const float back = a.h.mul[1];
  constexpr int kPieces = DM / 8;
#pragma unroll
  for (int j = 0; j < P::NI; ++j)
#pragma unroll
    for (int i = 0; i < P::MI; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = p.acc[i][j][4 * q + r] * back;
        u32x2 y;
        if (a.out_type == FS_BF16) {
          y[0] = Elem<__bf16>::pack(v[0], v[1]);
          y[1] = Elem<__bf16>::pack(v[2], v[3]);
        } else {
          y[0] = Elem<_Float16>::pack(v[0], v[1]);
          y[1] = Elem<_Float16>::pack(v[2], v[3]);
        }
        Stage16<DM>::put(lds, P::n_of(j), P::m_of(i) + 8 * q, y);
      }
  __syncthreads();
#pragma unroll 4
  for (int u = threadIdx.x; u < BN * kPieces; u += P::kThreads) {
    const int n = u / kPieces, piece = u % kPieces;
    const int64_t row = row0 + n;
    const int32_t col = col0 + 8 * piece;
    if (row >= rows || col >= cols) continue;
    const u32x4 v = Stage16<DM>::get(lds, n, piece);
    uint16_t* to = (uint16_t*)(a.out + row * a.out_stride) + col;
    if (col + 8 <= cols) {
      *(u32x4_any*)to = v;
    } else {
      for (int e = 0; e < cols - col; ++e) to[e] = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
    }
  }
}

// Waves of a tile of DM columns and BN rows.
template <int DM, int BN>
struct Waves {
  static constexpr int WM = BN == 256 ? 2 : DM / 32 < 4 ? 2 : DM == 128 ? 4 : 8;
  static constexpr int WN = BN == 256 ? 4 : DM == 256 ? 1 : 2;
  static constexpr int kThreads = WM * WN * kWave;
};

// dx = e w over a part of the piece's rows, by tokens' places: workgroup `bid` of
// the product's. lds: two stages. 16384 x 32768 x 1024: 854 to 884 us by card (1245 to 1290
// TFLOP/s, matrix units busy 69%: power, see product.hpp), with the fp32 sums that it adds to.
template <typename T, int DM, int BN, int Halves>
struct GradX : Waves<DM, BN> {
  using V = Waves<DM, BN>;
  using W = Cols<DM, V::kThreads, Halves>;
  using E = BlockRows<BN, V::kThreads>;
  using P = Tile<T, W, E, DM, BN, V::WM, V::WN, Halves>;
  static_assert(4 * P::kStage >= V::WN * 32 * DM * 4, "the stages hold rows of sums");
  static __device__ __forceinline__ void run(const SumArgs& a, int32_t bid, uint16_t* lds) {
    const Order order{(int32_t)cdiv(*a.h.n_live, BN), a.order.cols};
    const int32_t tiles = order.rows * order.cols;
    if ((int64_t)bid >= (int64_t)tiles * a.parts) return;
    const int32_t id = in_order(bid, tiles * a.parts);
    int32_t tn, td;
    // parts of one tile run apart, tiles of one part together
    order.at(id % tiles, kGroup, &tn, &td);
    const int32_t part = id / tiles;
    const int64_t n0 = (int64_t)tn * BN;
    const int64_t k0 = (int64_t)part * a.steps * kK, k1 = min(a.rows, k0 + (int64_t)a.steps * kK);
    P p;
    p.clear();
    W w(a.w, a.w_stride, td * DM, a.w_cols, k0);
    E e(a.e, a.e_cols * Halves, n0, k0 * Halves);
    P::template ask<true, false>(w, e, k1 - k0, lds);
    p.template run<true, false>(w, e, k1 - k0, lds);
    put_sums<P, DM, BN, V::WM>(p, lds, a, a.part + (int64_t)part * a.h.npad * a.h.dp, n0, a.h.npad, td * DM);
  }
};

// dw = e^T x over a part of the tokens. 16384 x 32768 x 1024: 845 to 877 us by card (1255 to
// 1300 TFLOP/s, matrix units busy 72%: power).
template <typename T, int DM, int BV, int Halves>
struct GradW : Waves<DM, BV> {
  using V = Waves<DM, BV>;
  using X = BlockCols<DM, V::kThreads, Halves>;
  using E = BlockCols<BV, V::kThreads, 1, Halves>;
  using P = Tile<T, X, E, DM, BV, V::WM, V::WN, Halves>;
  static_assert(4 * P::kStage >= V::WN * 32 * DM * 4 && 2 * P::kStage >= BV * DM, "the stages hold rows of sums");
  static __device__ __forceinline__ void run(const SumArgs& a, int32_t bid, int32_t grid, uint16_t* lds) {
    const int32_t tiles = a.order.rows * a.order.cols, id = in_order(bid, grid);
    int32_t tv, td;
    a.order.at(id % tiles, kGroup, &tv, &td);
    const int32_t part = id / tiles;
    // rows of e and x are zeros from n_live to the next multiple of 64
    const int64_t steps = cdiv(*a.h.n_live, kK), per = cdiv(steps, a.parts);
    const int64_t s0 = min(steps, part * per), s1 = min(steps, s0 + per);
    P p;
    p.clear();
    X x(a.h.x, a.h.dp, td * DM, s0 * kK);
    E e(a.e, a.e_cols, (int64_t)tv * BV, s0 * kK);
    P::template ask<false, false>(x, e, (s1 - s0) * kK, lds);
    p.template run<false, false>(x, e, (s1 - s0) * kK, lds);
    float* to = a.part ? a.part + (int64_t)part * a.out_rows * a.h.dp : nullptr;
    put_sums<P, DM, BV, V::WM>(p, lds, a, to, (int64_t)tv * BV, a.out_rows, td * DM);
  }
};

template <typename T, int DM>
__global__ void __launch_bounds__((Waves<DM, 256>::kThreads)) k_grad_x(SumArgs a) {
  using G = GradX<T, DM, 256, 1>;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * G::P::kStage];
  G::run(a, blockIdx.x, lds);
}
template <typename T, int DM, int BV>
__global__ void __launch_bounds__((Waves<DM, BV>::kThreads)) k_grad_w(SumArgs a) {
  using G = GradW<T, DM, BV, 1>;
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * G::P::kStage];
  G::run(a, blockIdx.x, gridDim.x, lds);
}
// Few tokens: both in one launch, dx's x_grid workgroups first, so that neither
// waits for the other to leave the chip half empty. Bound by latency: a start, a few
// steps and a way through LDS (64 tokens, 32000 rows of 64: 9 us; 499 tokens, 10007 of
// 200: 15.5).
template <typename T, int DM, int Halves>
__global__ void __launch_bounds__((Waves<DM, 64>::kThreads)) k_grads(SumArgs x, SumArgs w, int32_t x_grid) {
  using X = GradX<T, DM, 64, Halves>;
  using W = GradW<T, DM, 64, Halves>;
  static_assert(X::P::kStage == W::P::kStage, "one pair of stages");
  __shared__ __attribute__((aligned(16))) uint16_t lds[2 * X::P::kStage];
  if ((int32_t)blockIdx.x < x_grid) X::run(x, blockIdx.x, lds);
  else W::run(w, blockIdx.x - x_grid, gridDim.x - x_grid, lds);
}

// The parts of a sum, added in order and rounded once. Rows of pos < 0 are zeros.
struct JoinArgs {
  const float* part;
  int64_t part_rows;
  int32_t parts, dp, dim;
  const int32_t* pos;  // null: every row is its own
  int64_t rows;
  const float* mul;
  char* out;
  int64_t out_stride;
};
// PL lanes share the parts of 4 columns of a row.
template <typename T, int PL>
__global__ void __launch_bounds__(256) k_join(JoinArgs a) {
  constexpr int kPer = 256 / PL;
  __shared__ f32x4 sh[PL][kPer];
  const int32_t pieces = (int32_t)cdiv(a.dim, 4);
  const float back = a.mul[1];
  const int x = threadIdx.x % kPer, y = threadIdx.x / kPer;
  for (int64_t u0 = (int64_t)blockIdx.x * kPer; u0 < a.rows * pieces; u0 += (int64_t)gridDim.x * kPer) {  // uniform
    const int64_t u = u0 + x, row = u / pieces;
    const bool in = u < a.rows * pieces;
    const int32_t col = 4 * (int32_t)(u - row * pieces);
    const int64_t r = !in ? -1 : a.pos ? a.pos[row] : row;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (r >= 0) {
      const f32x4* p = (const f32x4*)(a.part + r * a.dp + col);
      const int64_t step = a.part_rows * a.dp / 4;
      int i = y;
      for (; i + 3 * PL < a.parts; i += 4 * PL) {
        f32x4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = p[(i + k * PL) * step];
        s += (v[0] + v[1]) + (v[2] + v[3]);
      }
      for (; i < a.parts; i += PL) s += p[i * step];
    }
    if constexpr (PL > 1) {
      __syncthreads();
      sh[y][x] = s;
      __syncthreads();
      if (y || !in) continue;
      for (int i = 1; i < PL; ++i) s += sh[i][x];
    }
    if (!in) continue;
    s *= back;
    T* to = (T*)(a.out + row * a.out_stride) + col;
    struct __attribute__((packed, aligned(sizeof(T)))) Four {
      T v[4];
    };
    if (col + 4 <= a.dim) {
      *(Four*)to = Four{{(T)s[0], (T)s[1], (T)s[2], (T)s[3]}};
    } else {
      for (int e = 0; e < a.dim - col; ++e) to[e] = (T)s[e];
    }
  }
}

// ---------------------------------------------------------------- losses
struct LossArgs {
  Head h;
  const float2* part;
  int64_t tiles;
  const float2* at_label;  // null: no loss here
  float *loss, *lse;
  const int64_t* labels;  // of tokens that were read as they lie, or null
  int64_t rows, pad;
  int32_t* err;
};

// A token's tiles joined: R tokens a workgroup, 256 / R threads each. 16384 tokens of
// 391 tiles: 16 us, the 51 MB that the scores left in the caches at 3.2 TB/s.
template <int R>
__global__ void __launch_bounds__(256) k_loss(LossArgs a) {
  constexpr int Q = 256 / R;
  __shared__ float2 sh[Q][R];
  const int r = threadIdx.x % R, q = threadIdx.x / R;
  const int64_t i = (int64_t)blockIdx.x * R + r;
  int32_t pos = -1;
  if (i < a.h.n && a.labels) {
    const int64_t v = a.labels[i];
    if (label_of(v, a.rows, a.pad) >= 0) pos = (int32_t)i;
    flag_err(a.err, q == 0 && pos < 0 && v != a.pad, FS_EF_ID_RANGE);
  } else if (i < a.h.n) {
    pos = a.h.pos[i];
  }
  float top = -3e38f, sum = 0.f;
  if (pos >= 0) {
    int64_t t = q;
    for (; t + 3 * Q < a.tiles; t += 4 * Q) {
      float2 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = a.part[(t + u * Q) * a.h.npad + pos];
      const float m = fmaxf(fmaxf(fmaxf(x[0].x, x[1].x), fmaxf(x[2].x, x[3].x)), top);
      sum *= __builtin_amdgcn_exp2f(top - m);
#pragma unroll
      for (int u = 0; u < 4; ++u) sum += x[u].y * __builtin_amdgcn_exp2f(x[u].x - m);
      top = m;
    }
    for (; t < a.tiles; t += Q) {
      const float2 x = a.part[t * a.h.npad + pos];
      const float m = fmaxf(x.x, top);
      sum = sum * __builtin_amdgcn_exp2f(top - m) + x.y * __builtin_amdgcn_exp2f(x.x - m);
      top = m;
    }
  }
  sh[q][r] = make_float2(top, sum);
  __syncthreads();
  if (q || i >= a.h.n) return;
  float m = top;
  for (int u = 1; u < Q; ++u) m = fmaxf(m, sh[u][r].x);
  sum = 0.f;
  for (int u = 0; u < Q; ++u) sum += sh[u][r].y * __builtin_amdgcn_exp2f(sh[u][r].x - m);
  const float log = __builtin_amdgcn_logf(sum);  // base 2
  a.lse[i] = pos >= 0 ? (m + log) * kLn2 : 0.f;
  // The sum is that of the scores' distances from m, which is rounded: the label's own
  // distance counts its rounding too, or a loss near 0 would be off by half a step of the
  // score (8e-5 at scores of 1600). The label is one of the sum's terms, so what is left
  // below 0 is rounding. NaN stays.
  if (a.at_label) {
    float loss = 0.f;
    if (pos >= 0) {
      const float2 z = a.at_label[pos];
      loss = (((m - z.x) - z.y) + log) * kLn2;
      loss = loss < 0.f ? 0.f : loss;
    }
    a.loss[i] = loss;
  }
}

// ---------------------------------------------------------------- distillation
struct TeacherArgs {
  Head h;
  Entries in;
  float scale;
  uint8_t* live;
  int32_t* err;
  // forward
  const char* w;
  int64_t w_stride;
  const char* x;  // tokens as they lie, or null
  int64_t x_stride;
  float *loss, *logits, *lse;
  const float2* part;  // null: lse is there, else it is made of these tiles
  int64_t tiles;
  // backward
  const float* logits_in;
  char* e;
  int64_t e_cols, v0, piece_rows;
  int32_t halves;
};

constexpr int kRowsPerGroup = 4;  // tokens of a workgroup, a wave each

__global__ void __launch_bounds__(kRowsPerGroup * kWave) k_teacher_live(TeacherArgs a) {
  const int64_t i = (int64_t)blockIdx.x * kRowsPerGroup + threadIdx.x / kWave;
  if (i >= a.h.n) return;
  bool on = false, bad = false;
  for (int k = lane(); k < a.in.top; k += kWave) {
    const int64_t id = a.in.ids[i * a.in.top + k];
    bad |= a.in.bad(id);
    on |= a.in.on(id, a.in.logit(i * a.in.top + k));
  }
  flag_err(a.err, bad, FS_EF_ID_RANGE);
  const bool any = __any(on);
  if (lane() == 0) a.live[i] = any;
}

constexpr int kPerLane = FS_MAX_TOP / kWave;

// The teacher's distribution over a token's entries, one wave: q and log q of
// entry lane + 64 u (0 where it takes no part). The scale goes to the distance from the
// logit of the largest product, halves of both taken, so that neither a product nor a
// distance of the type's largest and lowest values leaves fp32.
struct Teacher {
  float q[kPerLane], logq[kPerLane];
  int64_t id[kPerLane];
  bool on[kPerLane];
  __device__ __forceinline__ Teacher(const TeacherArgs& a, int64_t i) {
    float t[kPerLane], top = -INFINITY, sum = 0.f;
    const float sign = a.scale < 0.f ? -1.f : 1.f;
#pragma unroll
    for (int u = 0; u < kPerLane; ++u) {
      const int k = lane() + kWave * u;
      on[u] = false;
      id[u] = -1;
      t[u] = 0.f;
      if (k < a.in.top) {
        id[u] = a.in.ids[i * a.in.top + k];
        const float x = a.in.logit(i * a.in.top + k);
        on[u] = a.in.on(id[u], x);
        t[u] = x * (0.5f * sign);
      }
      if (on[u]) top = fmaxf(top, t[u]);
    }
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, kWave));
#pragma unroll
    for (int u = 0; u < kPerLane; ++u) {
      t[u] = 2.f * ((t[u] - top) * (a.scale * sign));
      q[u] = on[u] ? expf(t[u]) : 0.f;
      sum += q[u];
    }
    sum = wave_sum(sum);
    const float log = logf(sum);
#pragma unroll
    for (int u = 0; u < kPerLane; ++u) {
      logq[u] = on[u] ? t[u] - log : 0.f;
      q[u] = on[u] ? q[u] / sum : 0.f;
    }
  }
};

// What one wave wrote to LDS before what it reads behind
__device__ __forceinline__ void wave_lds() {
  __builtin_amdgcn_wave_barrier();
  __threadfence_block();
}

// Scores of a token's entries, and its loss. W waves have a token: 4 where tokens are
// few, which join its tiles as well, 1 where they are many. They take the entries in
// turn; LP lanes share a row's elements, so narrow rows go several to an access, and
// 8 accesses are in flight. Bound by the latency of a token's few dependent reads, so by
// how many tokens are under way: 5135 tokens of 56 entries, rows of 32, 51 us with 4
// waves of whole rows, 11 like this; 10813 x 5, rows of 440, 30 and 13; 8192 x 64, rows
// of 1024, 116 and 87.
template <typename T, int LP, int W>
__global__ void __launch_bounds__(kRowsPerGroup * kWave) k_distill(TeacherArgs a) {
  constexpr int kTokens = kRowsPerGroup / W, kRows = 8, kGroups = kWave / LP;
  __shared__ int32_t s_id[kRowsPerGroup][FS_MAX_TOP];
  __shared__ float s_z[kTokens][FS_MAX_TOP];
  const int wave = attn::wave_id(), w = wave % W, l = lane();
  const int64_t i = (int64_t)blockIdx.x * kTokens + wave / W;
  if (W == 1 && i >= a.h.n) return;
  float* const z_of = s_z[wave / W];
  const int32_t top = a.in.top;
  const Teacher t(a, i);
  int32_t pos;
  if (a.x) {
    bool on = false, bad = false;
#pragma unroll
    for (int u = 0; u < kPerLane; ++u) {
      on |= t.on[u];
      bad |= l + kWave * u < top && a.in.bad(t.id[u]);
    }
    flag_err(a.err, w == 0 && bad, FS_EF_ID_RANGE);
    pos = __any(on) ? (int32_t)i : -1;
  } else {
    pos = a.h.pos[i];
  }
  if (pos < 0) {  // uniform where waves share a token
    for (int k = w * kWave + l; k < top; k += W * kWave) a.logits[i * top + k] = 0.f;
    if (w == 0 && l == 0) {
      a.loss[i] = 0.f;
      if (W > 1) a.lse[i] = 0.f;
    }
    return;
  }
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) s_id[wave][l + kWave * u] = t.on[u] ? (int32_t)t.id[u] : -1;
  wave_lds();
  const int g = l / LP, c0 = 8 * (l % LP);
  for (int k0 = w * kGroups; k0 < top; k0 += kRows * W * kGroups) {  // uniform in a wave
    int32_t id[kRows];
    float sum[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int k = k0 + u * W * kGroups + g;
      id[u] = k < top ? s_id[wave][k] : -1;
      sum[u] = 0.f;
    }
    for (int c = c0; c < a.h.dim; c += 8 * LP) {
      const u32x4 xv = *(const u32x4*)(a.x ? a.x + i * a.x_stride + 2 * c : a.h.x + 2 * blocked(pos, c, a.h.dp));
      u32x4 wv[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) {
        wv[u] = u32x4{0, 0, 0, 0};
        if (id[u] >= 0) wv[u] = row_piece(a.w + id[u] * a.w_stride, c, a.h.dim);
      }
#pragma unroll
      for (int u = 0; u < kRows; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const auto p = Elem<T>::unpack(xv[e]), y = Elem<T>::unpack(wv[u][e]);
          sum[u] = __builtin_fmaf(p[0], y[0], sum[u]);
          sum[u] = __builtin_fmaf(p[1], y[1], sum[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float z = sum[u];
#pragma unroll
      for (int d = LP / 2; d > 0; d >>= 1) z += __shfl_xor(z, d, kWave);
      const int k = k0 + u * W * kGroups + g;
      if (l % LP == 0 && k < top) z_of[k] = id[u] >= 0 ? z * a.scale : 0.f;
    }
  }
  float lse;
  if constexpr (W > 1) {
    __shared__ float2 s_part[W];
    float top2 = -3e38f, sum = 0.f;
    for (int64_t q = threadIdx.x; q < a.tiles; q += W * kWave) {
      const float2 x = a.part[q * a.h.npad + pos];
      const float m = fmaxf(x.x, top2);
      sum = sum * __builtin_amdgcn_exp2f(top2 - m) + x.y * __builtin_amdgcn_exp2f(x.x - m);
      top2 = m;
    }
    float m = top2;
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, kWave));
    sum = wave_sum(sum * __builtin_amdgcn_exp2f(top2 - m));
    if (l == 0) s_part[w] = make_float2(m, sum);
    __syncthreads();
    if (w) return;
    m = s_part[0].x;
    sum = 0.f;
#pragma unroll
    for (int q = 1; q < W; ++q) m = fmaxf(m, s_part[q].x);
#pragma unroll
    for (int q = 0; q < W; ++q) sum += s_part[q].y * __builtin_amdgcn_exp2f(s_part[q].x - m);
    lse = (m + __builtin_amdgcn_logf(sum)) * kLn2;
    if (l == 0) a.lse[i] = lse;
  } else {
    wave_lds();
    lse = a.lse[i];
  }
  float loss = 0.f;
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int k = l + kWave * u;
    if (k < top) {
      const float z = z_of[k];
      a.logits[i * top + k] = z;
      if (t.on[u] && t.q[u] != 0.f) loss += t.q[u] * (t.logq[u] - z + lse);
    }
  }
  loss = wave_sum(loss);
  if (l == 0) a.loss[i] = loss;
}

template <typename T, int W>
void launch_distill(const TeacherArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)cdiv(a.h.n, kRowsPerGroup / W)), block(kRowsPerGroup * kWave);
  if (a.h.dim <= 64) hipLaunchKernelGGL((k_distill<T, 8, W>), grid, block, 0, stream, a);
  else if (a.h.dim <= 128) hipLaunchKernelGGL((k_distill<T, 16, W>), grid, block, 0, stream, a);
  else if (a.h.dim <= 256) hipLaunchKernelGGL((k_distill<T, 32, W>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_distill<T, 64, W>), grid, block, 0, stream, a);
}

// The entries' places of e in a piece: target off the softmax before the one
// rounding. Entries of one id write the same value.
template <typename T>
__global__ void __launch_bounds__(kRowsPerGroup * kWave) k_distill_entries(TeacherArgs a) {
  __shared__ uint2 s_own[kRowsPerGroup][FS_MAX_TOP];  // id and q
  const int w = threadIdx.x / kWave, l = lane();
  const int64_t i = (int64_t)blockIdx.x * kRowsPerGroup + w;
  if (i >= a.h.n) return;
  const int32_t pos = a.h.pos[i];
  if (pos < 0) return;
  const Teacher t(a, i);
#pragma unroll
  for (int u = 0; u < kPerLane; ++u)
    s_own[w][l + kWave * u] = make_uint2(t.on[u] ? (uint32_t)t.id[u] : ~0u, __float_as_uint(t.q[u]));
  wave_lds();
  const float c = a.h.coef[pos] * a.h.mul[0], lse2 = a.h.lse2[pos];
  float q[kPerLane] = {};
#pragma unroll 8
  for (int k = 0; k < a.in.top; ++k) {  // the q of each id's entries, in order (84 x 124: 16 us one by one, 9)
    const uint2 own = s_own[w][k];
#pragma unroll
    for (int u = 0; u < kPerLane; ++u) q[u] += own.x == (uint32_t)t.id[u] ? __uint_as_float(own.y) : 0.f;
  }
#pragma unroll
  for (int u = 0; u < kPerLane; ++u) {
    const int64_t v = t.id[u] - a.v0;
    if (!t.on[u] || v < 0 || v >= a.piece_rows) continue;
    const float z = a.logits_in[i * a.in.top + l + kWave * u];
    const float e = (__builtin_amdgcn_exp2f(__builtin_fmaf(z, kLog2e, -lse2)) - q[u]) * c;
    ((T*)a.e)[place_of_e(pos, v, a.e_cols, 0, a.halves)] = (T)e;
    if (a.halves > 1) ((T*)a.e)[place_of_e(pos, v, a.e_cols, 1, 2)] = (T)(e - (float)(T)e);
  }
}

// ---------------------------------------------------------------- host
struct Sizes {
  int64_t n, rows, npad, vpad, piece, pack_rows, pack_bytes, e_bytes, dx_part, dw_part, tiles;
  int32_t dim, dp, bn, halves, stay, dm;  // tiles of bn tokens, gradients' of dm columns
};

int64_t most_parts(int64_t steps) { return std::min<int64_t>(kMostParts, std::max<int64_t>(1, steps / 4)); }

// In how many parts a product is cut, so that few tiles do not leave CUs idle: the
// number for which its rounds of workgroups take the least time, with the sums that
// every part writes and somebody reads. Measured: a step of 64 takes a workgroup 1.8
// us in tiles of 256 x 256 (one to a CU) and 0.9 in tiles of 64 rows (two to a CU),
// less as there are fewer columns to load; its start and end take about 6, memory
// gives 5 bytes in a ps. 256 tiles of 256 steps: in two parts 479 us, in one 453.
int32_t parts_of(int64_t tiles, int64_t steps, int32_t rows, int32_t cols, int64_t bytes_each, int64_t bytes) {
  const int64_t most = std::min(most_parts(steps), std::max<int64_t>(1, bytes / std::max<int64_t>(bytes_each, 1)));
  const int64_t at_once = kCus * std::min<int64_t>(4, std::max<int64_t>(1, 640 / (rows + cols)));
  const double step = 1.8 * (rows + cols) / 512.0 * (rows == 64 ? 1.4 : 1.0);
  int32_t best = 1;
  double least = 1e300;
  for (int64_t p = 1; p <= most; p += 1 + p / 8) {
    const double us = (double)cdiv(tiles * p, at_once) * ((double)cdiv(steps, p) * step + 6.0) +
                      (p > 1 ? 5.0 : 0.0) + 2e-6 * (double)(p * bytes_each) / 5.0;
    if (us < least) {
      least = us;
      best = (int32_t)p;
    }
  }
  return best;
}

Sizes sizes_of(int64_t n, int64_t rows, int32_t dim) {
  Sizes s;
  s.n = n;
  s.rows = rows;
  s.dim = dim;
  s.dp = (int32_t)align_up((size_t)dim, kK);
  // Tiles of 64 tokens where those of 256 would be few or mostly empty: of 512 tiles and
  // more those of 256 win forward (4096 tokens, 8192 rows of 256: 35 us against 41; 2048, 32000
  // of 512: 81 and 99) and both ways of the largest (263 and 273), below them those of 64
  // mostly backward (512, 32000 of 256: 69 and 73; 1024, 32000 of 256: 104 and 108; of 1024
  // columns 260 and 238). Long rows' forward alone would have those of 256 from 128 tiles on
  // (1024, 32000 of 1024: 94 and 76 us).
  s.bn = n > kFew && cdiv(n, 256) * cdiv(rows, kV) >= 512 ? 256 : 64;
  s.dm = dim <= 64 ? 64 : (dim <= 128 ? 128 : 256);
  s.npad = (int64_t)align_up((size_t)std::max<int64_t>(n, 1), n > 128 ? 256 : 64);
  s.vpad = (int64_t)align_up((size_t)rows, kV);
  s.tiles = s.vpad / kV;
  // e: all of it, or pieces of kPieceBytes, or of one tile's width
  s.halves = n <= kFew ? 2 : 1;
  const int64_t e_rows = s.npad * s.halves;
  // Tokens that take no part cost as much as others where all keep their places, so
  // that is for what takes little time. us of a call's kernels, places kept and not, all
  // tokens taking part and half of them: forward 1000 tokens, 8000 rows of 256, 14 and 20, 14
  // and 17; 32000 of 128 27 and 32, 27 and 22; 32000 of 512 54 and 58, 52 and 36. Backward of a
  // distillation, 499 tokens, 10007 of 200, 43 and 47, 40 and 38; 1000, 32000 of 128 83 and 88,
  // 76 and 60; 32000 of 512 160 and 163, 150 and 98.
  s.stay = n <= kFew || (n <= kStayMost && n * rows * dim <= ((int64_t)1 << 32));
  s.e_bytes = e_rows <= kPieceBytes / 2 / s.vpad ? e_rows * s.vpad * 2 : std::max(kPieceBytes, e_rows * kV * 2);
  s.piece = std::min(s.vpad, std::max<int64_t>(kV, s.e_bytes / (e_rows * 2) / kV * kV));
  s.pack_bytes = std::max(std::min(s.vpad * s.dp * 2, kPackBytes), (int64_t)kV * s.dp * 2);
  s.pack_rows = std::min(s.vpad, std::max<int64_t>(kV, s.pack_bytes / (s.dp * 2) / kV * kV));
  const int64_t dx = s.npad * s.dp * 4, dw = s.vpad * s.dp * 4;
  const int64_t x_most = most_parts(s.vpad / kK), w_most = most_parts(s.npad / kK);
  s.dx_part = std::max(dx, std::min(dx * x_most, kPartBytes));
  s.dw_part = w_most > 1 ? std::min(dw * w_most, kPartBytes) : 0;
  return s;
}

struct Space {
  Head h;
  uint8_t* live;
  char* pack;
  float2* part;      // forward
  float2* at_label;
  char* e;           // backward
  float *dx_part, *dw_part;
};

size_t carve(void* ws, const Sizes& s, bool back, Space* o) {
  Carve c(ws);
  Head& h = o->h;
  h.n_live = c.take<int32_t>(1);
  h.mul = c.take<float>(2);
  h.pos = c.take<int32_t>((size_t)s.npad);
  h.label = c.take<int32_t>((size_t)s.npad);
  h.lse2 = c.take<float>((size_t)s.npad);
  h.coef = c.take<float>((size_t)s.npad);
  h.x = c.take<char>((size_t)(s.npad * s.dp * 2));
  o->live = c.take<uint8_t>((size_t)s.npad);
  o->pack = c.take<char>((size_t)s.pack_bytes);
  if (back) {
    o->e = c.take<char>((size_t)s.e_bytes);
    o->dx_part = c.take<float>((size_t)s.dx_part / 4);
    o->dw_part = c.take<float>((size_t)s.dw_part / 4);
  } else {
    o->part = c.take<float2>((size_t)(s.tiles * s.npad));
    o->at_label = c.take<float2>((size_t)s.npad);
  }
  h.n = s.n;
  h.npad = s.npad;
  h.dim = s.dim;
  h.dp = s.dp;
  return c.used + 512;
}

void* aligned(void* ws) { return (void*)align_up((size_t)ws, 256); }

// The table as the tiles load it: rows that lie 16-byte aligned as they are.
struct Table {
  const char* w;
  int64_t stride;
  bool direct;
};

bool loads_directly(const char* w, int64_t stride, int32_t dim) {
  return dim % 8 == 0 && stride % 16 == 0 && (uintptr_t)w % 16 == 0 && stride <= ((int64_t)1 << 23);
}

// rows v0 .. of a table, laid out in `pack` where the tiles cannot load them
int piece_of(const Table& t, const Sizes& s, int64_t v0, int64_t rows, char* pack, const char** w,
             int64_t* stride, int32_t* k, hipStream_t stream) {
  *w = t.w + v0 * t.stride;
  *stride = t.stride;
  *k = s.dim;
  if (t.direct) return FS_OK;
  const int64_t blocks = std::min<int64_t>(cdiv(rows * (s.dp / 8), kPackThreads), 8192);
  hipLaunchKernelGGL(k_table_pack, dim3((unsigned)blocks), dim3(kPackThreads), 0, stream, *w, t.stride, rows,
                     s.dim, s.dp, pack);
  FS_LAUNCH_CHECK();
  *w = pack;
  *stride = 2 * (int64_t)s.dp;
  *k = s.dp;
  return FS_OK;
}

int pack_tokens(PackArgs a, hipStream_t stream) {
  const int64_t per = std::max<int64_t>(16, cdiv(a.h.n, 1024));
  a.per = (int32_t)per;
  const int64_t blocks = std::max<int64_t>(1, cdiv(a.h.n, per));
  hipLaunchKernelGGL(k_head_pack, dim3((unsigned)(blocks + a.back)), dim3(kPackThreads), 0, stream, a);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

// Halves: 0 forward, else of e. Two go with tiles of 64 tokens.
template <typename T, int Halves>
void launch_scores(const ScoreArgs& a, const Sizes& s, int64_t tiles, hipStream_t stream) {
  if constexpr (Halves < 2) {
    if (s.bn == 256) {
      hipLaunchKernelGGL((k_scores<T, 256, kWM, kWN, Halves, 2, false>), dim3((unsigned)std::min<int64_t>(tiles, kCus)),
                         dim3(kWM * kWN * kWave), 0, stream, a);
      return;
    }
  }
  const dim3 grid((unsigned)tiles), block(8 * kWave);
  // No more tiles than CUs: LDS of a whole CU, three steps' loads in flight instead of
  // one (162 tokens, 1474 rows of 1472: 19.8 -> 16.7 us; 2 tokens, 48218 of 1176: 22.8 ->
  // 19.9; rows of 512 and 192 gain nothing)
  const bool deep = tiles <= kCus && a.k > 8 * kK;
  auto go = [&](auto direct) {
    constexpr bool D = decltype(direct)::value;
    if (deep) hipLaunchKernelGGL((k_scores<T, 64, 8, 1, Halves, 4, D>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((k_scores<T, 64, 8, 1, Halves, 2, D>), grid, block, 0, stream, a);
  };
  if constexpr (Halves == 0) {
    if (a.x) return go(std::true_type());
  }
  go(std::false_type());
}
template <int Halves>
int launch_scores(const ScoreArgs& a, const Sizes& s, int32_t dtype, hipStream_t stream) {
  const int64_t tiles = (int64_t)a.order.rows * a.order.cols;
  if (!grid_fits(tiles, kMostThreads)) return FS_ERR_UNSUPPORTED;
  if (dtype == FS_BF16) launch_scores<__bf16, Halves>(a, s, tiles, stream);
  else launch_scores<_Float16, Halves>(a, s, tiles, stream);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

// dx's and dw's products of a piece; a grid of 0 is left out.
template <typename T, int DM>
void launch_grads(const SumArgs& x, int64_t x_grid, const SumArgs& w, int64_t w_grid, const Sizes& s,
                  int32_t bv, hipStream_t stream) {
  const dim3 many(Waves<DM, 256>::kThreads), few(Waves<DM, 64>::kThreads);
  if (s.bn == 64) {
    const dim3 grid((unsigned)(x_grid + w_grid));
    if (s.halves == 1) hipLaunchKernelGGL((k_grads<T, DM, 1>), grid, few, 0, stream, x, w, (int32_t)x_grid);
    else hipLaunchKernelGGL((k_grads<T, DM, 2>), grid, few, 0, stream, x, w, (int32_t)x_grid);
    return;
  }
  const dim3 gx((unsigned)x_grid), gw((unsigned)w_grid);
  if (x_grid > 0) hipLaunchKernelGGL((k_grad_x<T, DM>), gx, many, 0, stream, x);
  if (w_grid > 0) {
    if (bv == 256) hipLaunchKernelGGL((k_grad_w<T, DM, 256>), gw, many, 0, stream, w);
    else hipLaunchKernelGGL((k_grad_w<T, DM, 64>), gw, few, 0, stream, w);
  }
}
template <typename T>
void launch_grads(const SumArgs& x, int64_t x_grid, const SumArgs& w, int64_t w_grid, const Sizes& s,
                  int32_t bv, hipStream_t stream) {
  if (s.dm == 64) launch_grads<T, 64>(x, x_grid, w, w_grid, s, bv, stream);
  else if (s.dm == 128) launch_grads<T, 128>(x, x_grid, w, w_grid, s, bv, stream);
  else launch_grads<T, 256>(x, x_grid, w, w_grid, s, bv, stream);
}

template <typename T>
void launch_join_as(const JoinArgs& a, hipStream_t stream) {
  // many parts, few rows: 8 lanes share them (63 parts of 64 x 64: 19 -> 4.6 us; 8
  // parts of 8192 x 768: 38 by one lane, 53 by eight)
  const bool share = a.parts >= 8 && a.rows * a.dim <= ((int64_t)1 << 19);
  const int64_t per = share ? 32 : 256, work = cdiv(a.rows * cdiv(a.dim, 4), per);
  const dim3 g((unsigned)std::max<int64_t>(1, std::min<int64_t>(work, 16384))), b(256);
  if (share) hipLaunchKernelGGL((k_join<T, 8>), g, b, 0, stream, a);
  else hipLaunchKernelGGL((k_join<T, 1>), g, b, 0, stream, a);
}

int launch_join(const JoinArgs& a, int32_t type, hipStream_t stream) {
  if (type == FS_F32) launch_join_as<float>(a, stream);
  else if (type == FS_BF16) launch_join_as<__bf16>(a, stream);
  else launch_join_as<_Float16>(a, stream);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

// What both losses' calls are checked for alike.
int check(const void* x, int64_t* x_stride, int64_t n, const fs_table* table, float scale, Table* t) {
  if (!table || n < 0 || n >= (int64_t)INT32_MAX - 256 || table->rows < 1 || table->dim < 1 ||
      !attn::scale_ok(scale))
    return FS_ERR_INVALID_ARG;
  if ((table->dtype != FS_BF16 && table->dtype != FS_F16) || table->dim > FS_MAX_TOKEN_DIM ||
      table->rows >= (int64_t)INT32_MAX - 256)
    return FS_ERR_UNSUPPORTED;
  const int64_t row = 2 * (int64_t)table->dim;
  if (!*x_stride) *x_stride = row;
  t->w = (const char*)table->weights;
  t->stride = table->stride ? table->stride : row;
  if (*x_stride < row || *x_stride % 2 || t->stride < row || t->stride % 2 || !t->w || (uintptr_t)t->w % 2 ||
      (n > 0 && (!x || (uintptr_t)x % 2)))
    return FS_ERR_INVALID_ARG;
  t->direct = loads_directly(t->w, t->stride, table->dim);
  return FS_OK;
}

// Tokens of a forward call that the tiles can read as they lie.
struct Tokens {
  const char* x;  // null: packed
  int64_t stride;
};

// Few tokens' rows of whole steps need no packing: what a token's row holds reaches no
// other's score (17 tokens, 100000 rows of 256: 20.3 -> 17.5 us).
Tokens as_they_lie(const void* x, int64_t stride, const Sizes& s) {
  const bool can = s.stay && s.bn == 64 && s.dim % kK == 0 && loads_directly((const char*)x, stride, s.dim);
  return can ? Tokens{(const char*)x, stride} : Tokens{};
}

// Scores of all tiles, then lse and the losses of labels.
int forward(const Sizes& s, const Space& o, const Table& t, int32_t dtype, float scale, const Tokens& x,
            const int64_t* labels, int64_t padding_id, int32_t* err, float* loss, float* lse,
            hipStream_t stream) {
  int rc;
  const int64_t step = t.direct ? s.vpad : s.pack_rows;
  for (int64_t v0 = 0; v0 < s.rows; v0 += step) {
    ScoreArgs a = {};
    a.h = o.h;
    a.v0 = v0;
    a.rows = std::min(step, s.rows - v0);
    a.v_tile0 = (int32_t)(v0 / kV);
    if ((rc = piece_of(t, s, v0, a.rows, o.pack, &a.w, &a.w_stride, &a.k, stream))) return rc;
    a.order = Order{(int32_t)cdiv(s.n, s.bn), (int32_t)cdiv(a.rows, kV)};
    a.scale2 = scale * kLog2e;
    a.x = x.x;
    a.x_stride = x.stride;
    a.labels = labels;
    a.all_rows = s.rows;
    a.pad = padding_id;
    a.part = o.part;
    a.at_label = o.at_label;
    if ((rc = launch_scores<0>(a, s, dtype, stream))) return rc;
  }
  // few tokens' tiles are joined where their entries are (a launch of 4 us less; of
  // many tokens a token's tiles lie too far apart for that)
  if (!labels && s.n < kFewRows) return FS_OK;
  const LossArgs l{o.h, o.part, s.tiles, labels ? o.at_label : nullptr, loss, lse, x.x ? labels : nullptr,
                   s.rows, padding_id, err};
  if (s.n < kFewRows) hipLaunchKernelGGL(k_loss<4>, dim3((unsigned)cdiv(s.n, 4)), dim3(256), 0, stream, l);
  else hipLaunchKernelGGL(k_loss<16>, dim3((unsigned)cdiv(s.n, 16)), dim3(256), 0, stream, l);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

struct Grads {
  void* dx;
  int64_t dx_stride;
  void* dw;
  int32_t dw_type;
  int64_t dw_stride;
};

int check_grads(Grads* g, int64_t n, int32_t dim) {
  if (g->dw_type != FS_F32 && g->dw_type != FS_BF16 && g->dw_type != FS_F16) return FS_ERR_INVALID_ARG;
  const int32_t e = g->dw_type == FS_F32 ? 4 : 2;
  if (!g->dx_stride) g->dx_stride = 2 * (int64_t)dim;
  if (!g->dw_stride) g->dw_stride = e * (int64_t)dim;
  if (g->dx_stride < 2 * (int64_t)dim || g->dx_stride % 2 || (uintptr_t)g->dx % 2 ||
      g->dw_stride < e * (int64_t)dim || g->dw_stride % e || (uintptr_t)g->dw % e || (n > 0 && !g->dx && !g->dw))
    return FS_ERR_INVALID_ARG;
  return FS_OK;
}

int backward(const Sizes& s, const Space& o, const Table& t, int32_t dtype, float scale, const Grads& g,
             TeacherArgs* entries, hipStream_t stream) {
  int rc;
  const int64_t step = t.direct ? s.piece : std::min(s.piece, s.pack_rows);
  const int32_t token_tiles = (int32_t)cdiv(s.n, s.bn), col_tiles = (int32_t)cdiv(s.dim, s.dm);
  const int32_t x_parts = parts_of((int64_t)token_tiles * col_tiles, cdiv(std::min(step, s.rows), kK) * s.halves,
                                   s.bn, s.dm, s.npad * s.dp * 4, s.dx_part);
  for (int64_t v0 = 0; v0 < s.rows; v0 += step) {
    ScoreArgs a = {};
    a.h = o.h;
    a.v0 = v0;
    a.rows = std::min(step, s.rows - v0);
    a.e = o.e;
    a.e_cols = (int64_t)align_up((size_t)a.rows, kV);
    a.past = 2 * s.npad * a.e_cols > kCacheBytes;
    if ((rc = piece_of(t, s, v0, a.rows, o.pack, &a.w, &a.w_stride, &a.k, stream))) return rc;
    const int32_t table_tiles = (int32_t)cdiv(a.rows, kV);
    a.order = Order{token_tiles, table_tiles};
    a.scale2 = scale * kLog2e;
    if (s.n > 0) {
      rc = s.halves == 2 ? launch_scores<2>(a, s, dtype, stream) : launch_scores<1>(a, s, dtype, stream);
      if (rc) return rc;
      if (entries) {
        entries->e = a.e;
        entries->e_cols = a.e_cols;
        entries->halves = s.halves;
        entries->v0 = v0;
        entries->piece_rows = a.rows;
        const dim3 grid((unsigned)cdiv(s.n, kRowsPerGroup)), block(kRowsPerGroup * kWave);
        if (dtype == FS_BF16) hipLaunchKernelGGL(k_distill_entries<__bf16>, grid, block, 0, stream, *entries);
        else hipLaunchKernelGGL(k_distill_entries<_Float16>, grid, block, 0, stream, *entries);
        FS_LAUNCH_CHECK();
      }
    }
    SumArgs b = {};
    b.h = o.h;
    b.w = a.w;
    b.w_stride = a.w_stride;
    b.rows = a.rows;
    b.w_cols = a.k;
    b.e = a.e;
    b.e_cols = a.e_cols;
    SumArgs c = b;
    int64_t x_grid = 0, w_grid = 0;
    if (g.dx && s.n > 0) {
      b.order = Order{token_tiles, col_tiles};
      b.parts = x_parts;
      b.steps = (int32_t)cdiv(cdiv(a.rows, kK), x_parts);
      b.add = v0 > 0;
      b.part = o.dx_part;
      x_grid = (int64_t)token_tiles * col_tiles * x_parts;
    }
    // tiles of 64 rows beside tiles of 64 tokens, and where those of 256 would leave
    // CUs idle (us of the call with 64 and 256: 4096 tokens, 8192 rows of 256, 121 and 125,
    // 32768 of 512 522 and 470; 16384 tokens, 16384 of 1024 1677 and 1508. Many tokens' tiles of
    // 256 are cut into parts and win below that too: 16384, 8192 of 1024 866 and 814, of
    // 256 364 and 350)
    const int32_t bv = s.bn == 64 || (int64_t)table_tiles * col_tiles < kCus ? 64 : kV;
    if (g.dw) {
      const int32_t row_tiles = (int32_t)cdiv(a.rows, bv);
      const int64_t tiles = (int64_t)row_tiles * col_tiles;
      c.order = Order{row_tiles, col_tiles};
      c.parts = parts_of(tiles, cdiv(s.n, kK) * s.halves, bv, s.dm, a.rows * s.dp * 4, s.dw_part);
      c.part = c.parts > 1 ? o.dw_part : nullptr;
      c.out = (char*)g.dw + v0 * g.dw_stride;
      c.out_stride = g.dw_stride;
      c.out_rows = a.rows;
      c.out_type = g.dw_type;
      w_grid = tiles * c.parts;
    }
    if (!grid_fits(x_grid + w_grid, kMostThreads)) return FS_ERR_UNSUPPORTED;
    if (dtype == FS_BF16) launch_grads<__bf16>(b, x_grid, c, w_grid, s, bv, stream);
    else launch_grads<_Float16>(b, x_grid, c, w_grid, s, bv, stream);
    FS_LAUNCH_CHECK();
    if (g.dw && c.parts > 1) {
      const JoinArgs j{o.dw_part, a.rows, c.parts, s.dp, s.dim, nullptr, a.rows, o.h.mul, c.out, g.dw_stride};
      if ((rc = launch_join(j, g.dw_type, stream))) return rc;
    }
  }
  if (g.dx && s.n > 0) {
    const JoinArgs j{o.dx_part, s.npad, x_parts, s.dp, s.dim, o.h.pos, s.n, o.h.mul, (char*)g.dx, g.dx_stride};
    if ((rc = launch_join(j, dtype, stream))) return rc;
  }
  return FS_OK;
}

// a grid of any launch of a call, by its sizes
bool too_many(const Sizes& s) {
  return !grid_fits(cdiv(s.npad, 64) * s.tiles, kMostThreads) || !grid_fits(s.npad, kRowsPerGroup * kWave);
}

PackArgs pack_args(const Space& o, const Sizes& s, const void* x, int64_t x_stride, const int64_t* labels,
                   int64_t padding_id, float scale, int32_t dtype, int32_t* err) {
  PackArgs p = {};
  p.h = o.h;
  p.x = (const char*)x;
  p.x_stride = x_stride;
  p.labels = labels;
  p.live = o.live;
  p.rows = s.rows;
  p.pad = padding_id;
  p.scale = scale;
  p.pad_to = s.bn;
  p.stay = s.stay;
  p.narrow = dtype == FS_F16;
  p.err = err;
  return p;
}

bool top_ok(int32_t top, int32_t type) {
  return top >= 1 && (type == FS_F32 || type == FS_BF16 || type == FS_F16);
}

TeacherArgs teacher_args(const Space& o, const Sizes& s, const int64_t* ids, int32_t top, const void* teacher,
                         int32_t type, float scale, int64_t padding_id, int32_t* err) {
  TeacherArgs t = {};
  t.h = o.h;
  t.in = Entries{ids, (const char*)teacher, type, top, s.rows, padding_id};
  t.scale = scale;
  t.live = o.live;
  t.err = err;
  return t;
}

// Packs a distillation's tokens; those that stay need no launch for who takes part
// (few tokens' calls are a launch of 4 us shorter).
int pack_entries(const TeacherArgs& t, PackArgs p, hipStream_t stream) {
  p.entries = t.in;
  if (p.stay) return pack_tokens(p, stream);
  hipLaunchKernelGGL(k_teacher_live, dim3((unsigned)cdiv(t.h.n, kRowsPerGroup)), dim3(kRowsPerGroup * kWave), 0,
                     stream, t);
  FS_LAUNCH_CHECK();
  return pack_tokens(p, stream);
}

}  // namespace
}  // namespace fs

using namespace fs;

extern "C" size_t fs_token_loss_workspace_size(int64_t n, int64_t rows, int32_t dim) {
  if (n < 0 || rows < 1 || dim < 1) return 0;
  Space o;
  return carve(nullptr, sizes_of(n, rows, dim), false, &o);
}

extern "C" size_t fs_token_loss_backward_workspace_size(int64_t n, int64_t rows, int32_t dim) {
  if (n < 0 || rows < 1 || dim < 1) return 0;
  Space o;
  return carve(nullptr, sizes_of(n, rows, dim), true, &o);
}

extern "C" int fs_token_loss(const void* x, int64_t x_stride, int64_t n, const fs_table* table,
                             const int64_t* labels, float scale, int64_t padding_id, float* loss,
                             float* lse, int32_t* err, void* ws, size_t ws_bytes, hipStream_t stream) {
  Table t;
  int rc;
  if ((rc = check(x, &x_stride, n, table, scale, &t))) return rc;
  if (n > 0 && (!labels || !loss || !lse)) return FS_ERR_INVALID_ARG;
  const Sizes s = sizes_of(n, table->rows, table->dim);
  if (too_many(s)) return FS_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < fs_token_loss_workspace_size(n, table->rows, table->dim)) return FS_ERR_WORKSPACE;
  if (n == 0) return FS_OK;
  Space o;
  carve(aligned(ws), s, false, &o);
  const Tokens lie = as_they_lie(x, x_stride, s);
  if (!lie.x &&
      (rc = pack_tokens(pack_args(o, s, x, x_stride, labels, padding_id, scale, table->dtype, err), stream)))
    return rc;
  return forward(s, o, t, table->dtype, scale, lie, labels, padding_id, err, loss, lse, stream);
}

extern "C" int fs_token_loss_backward(const void* x, int64_t x_stride, int64_t n, const fs_table* table,
                                      const int64_t* labels, const float* lse, const float* dloss,
                                      float scale, int64_t padding_id, void* dx, int64_t dx_stride,
                                      void* dweight, int32_t dweight_dtype, int64_t dweight_stride,
                                      int32_t* err, void* ws, size_t ws_bytes, hipStream_t stream) {
  Table t;
  int rc;
  Grads g{dx, dx_stride, dweight, dweight_dtype, dweight_stride};
  if ((rc = check(x, &x_stride, n, table, scale, &t)) || (rc = check_grads(&g, n, table->dim))) return rc;
  if (n > 0 && (!labels || !lse || !dloss)) return FS_ERR_INVALID_ARG;
  const Sizes s = sizes_of(n, table->rows, table->dim);
  if (too_many(s)) return FS_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < fs_token_loss_backward_workspace_size(n, table->rows, table->dim))
    return FS_ERR_WORKSPACE;
  if (n == 0 && !dweight) return FS_OK;
  Space o;
  carve(aligned(ws), s, true, &o);
  PackArgs p = pack_args(o, s, x, x_stride, labels, padding_id, scale, table->dtype, err);
  p.lse = lse;
  p.dloss = dloss;
  p.back = 1;
  if ((rc = pack_tokens(p, stream))) return rc;
  return backward(s, o, t, table->dtype, scale, g, nullptr, stream);
}

extern "C" int fs_token_distill(const void* x, int64_t x_stride, int64_t n, const fs_table* table,
                                const int64_t* ids, int32_t top, const void* teacher,
                                int32_t teacher_dtype, float scale, int64_t padding_id, float* loss,
                                float* lse, float* logits, int32_t* err, void* ws, size_t ws_bytes,
                                hipStream_t stream) {
  Table t;
  int rc;
  if ((rc = check(x, &x_stride, n, table, scale, &t))) return rc;
  if (!top_ok(top, teacher_dtype)) return FS_ERR_INVALID_ARG;
  if (top > FS_MAX_TOP) return FS_ERR_UNSUPPORTED;
  if (n > 0 && (!ids || !teacher || !loss || !lse || !logits)) return FS_ERR_INVALID_ARG;
  const Sizes s = sizes_of(n, table->rows, table->dim);
  if (too_many(s)) return FS_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < fs_token_loss_workspace_size(n, table->rows, table->dim)) return FS_ERR_WORKSPACE;
  if (n == 0) return FS_OK;
  Space o;
  carve(aligned(ws), s, false, &o);
  TeacherArgs a = teacher_args(o, s, ids, top, teacher, teacher_dtype, scale, padding_id, err);
  const Tokens lie = as_they_lie(x, x_stride, s);
  if (!lie.x &&
      (rc = pack_entries(a, pack_args(o, s, x, x_stride, nullptr, padding_id, scale, table->dtype, err), stream)))
    return rc;
  if ((rc = forward(s, o, t, table->dtype, scale, lie, nullptr, padding_id, err, loss, lse, stream))) return rc;
  a.x = lie.x;
  a.x_stride = lie.stride;
  a.w = t.w;
  a.w_stride = t.stride;
  a.loss = loss;
  a.logits = logits;
  a.lse = lse;
  a.part = n < kFewRows ? o.part : nullptr;
  a.tiles = s.tiles;
  const bool few = n < kFewRows;
  if (table->dtype == FS_BF16) few ? launch_distill<__bf16, 4>(a, stream) : launch_distill<__bf16, 1>(a, stream);
  else few ? launch_distill<_Float16, 4>(a, stream) : launch_distill<_Float16, 1>(a, stream);
  FS_LAUNCH_CHECK();
  return FS_OK;
}

extern "C" int fs_token_distill_backward(const void* x, int64_t x_stride, int64_t n, const fs_table* table,
                                         const int64_t* ids, int32_t top, const void* teacher,
                                         int32_t teacher_dtype, const float* lse, const float* logits,
                                         const float* dloss, float scale, int64_t padding_id, void* dx,
                                         int64_t dx_stride, void* dweight, int32_t dweight_dtype,
                                         int64_t dweight_stride, int32_t* err, void* ws,
                                         size_t ws_bytes, hipStream_t stream) {
  Table t;
  int rc;
  Grads g{dx, dx_stride, dweight, dweight_dtype, dweight_stride};
  if ((rc = check(x, &x_stride, n, table, scale, &t)) || (rc = check_grads(&g, n, table->dim))) return rc;
  if (!top_ok(top, teacher_dtype)) return FS_ERR_INVALID_ARG;
  if (top > FS_MAX_TOP) return FS_ERR_UNSUPPORTED;
  if (n > 0 && (!ids || !teacher || !lse || !logits || !dloss)) return FS_ERR_INVALID_ARG;
  const Sizes s = sizes_of(n, table->rows, table->dim);
  if (too_many(s)) return FS_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < fs_token_loss_backward_workspace_size(n, table->rows, table->dim))
    return FS_ERR_WORKSPACE;
  if (n == 0 && !dweight) return FS_OK;
  Space o;
  carve(aligned(ws), s, true, &o);
  TeacherArgs a = teacher_args(o, s, ids, top, teacher, teacher_dtype, scale, padding_id, err);
  a.logits_in = logits;
  PackArgs p = pack_args(o, s, x, x_stride, nullptr, padding_id, scale, table->dtype, err);
  p.lse = lse;
  p.dloss = dloss;
  p.back = 1;
  if ((rc = pack_entries(a, p, stream))) return rc;
  return backward(s, o, t, table->dtype, scale, g, &a, stream);
}
